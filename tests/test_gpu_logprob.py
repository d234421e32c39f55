"""Log probabilities of tokens, entropies, top tokens and their gradient on the
GPU against 64-bit references.

Tolerances. u = 2^-24, z = x / temperature, r = z - max z <= 0. The exponent of a
term has five roundings (1 / temperature, log2 e, their product, x - max, the last
product), v_exp_f32 one unit, 2 u: a term is within (6 |r| + 2) u of itself, and a
thread adds at most c terms in a row (c = V / 256 rounded up to whole vectors, 16,
and 16 to join and rescale). With A = sum p |r| and B = sum p r^2:
  log S within (6 A + c + 34) u + 2 u |log S|,
  a log probability within that + 4 u |r| + u |log p| (|log p| <= |r| + |log S|),
  the entropy within (6 A + 6 B + 2 (c + 36) (1 + A)) u + 2 u |log S|.
In the gradient p is within E = (6 A + c + 40 + 6 |r| + 4 |log S|) u of itself,
log p within E too, so dx within |dlp| (E p + 4 u) + |dH| p (E (|log p| + H + 2)
+ 2 error of H), over the temperature, 4 u of its own and the output's half step."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]
TINY = {torch.float32: 1e-38, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38}


def within(got, want, tol):
    same = (got.double() == want) | ((got.double() - want).abs() <= tol)
    assert bool(same.all()), (int((~same).sum()), (~same).nonzero()[:3].tolist(), got[~same][:3], want[~same][:3])


def bits(lp):
    """All it says, as whole numbers: an id of -1 would be a NaN among the floats."""
    return lp.buf.view(torch.int32)


class Exact:
    """The 64-bit answers of rows with at least one token, and the bounds."""

    def __init__(self, X, tokens, temperature):
        T, V = X.shape
        z = X.double() / temperature
        r = z - z.amax(1, keepdim=True)
        e = torch.exp(r)
        S = e.sum(1, keepdim=True)
        self.p, self.logp = e / S, r - torch.log(S)
        fin = torch.where(self.p > 0, r, 0.0)
        A, B = (self.p * fin.abs()).sum(1), (self.p * fin * fin).sum(1)
        self.H = -(self.p * torch.where(self.p > 0, self.logp, 0.0)).sum(1)
        c = -(-V // 256) + 16 + 16
        ls = torch.log(S)[:, 0].abs()
        self.tol_s = (6 * A + c + 34) * U + 2 * U * ls
        far = torch.where(r.isfinite(), r.abs(), 0.0)  # also where p has left the range
        self.tol_p = self.tol_s[:, None] + 5 * U * far + U * ls[:, None]
        self.tol_H = (6 * A + 6 * B + 2 * (c + 36) * (1 + A)) * U + 2 * U * ls
        self.E = (6 * A + c + 40 + 4 * ls)[:, None] * U + 6 * fin.abs() * U
        self.t = tokens.long()
        self.pad = (self.t < 0) | (self.t >= V)
        at = self.t.clamp(0, V - 1)[:, None]
        self.lp = torch.where(self.pad, 0.0, self.logp.gather(1, at)[:, 0])
        self.tol_lp = torch.where(self.pad, 0.0, self.tol_p.gather(1, at)[:, 0])

    def gradient(self, dl, dh, temperature, dtype):
        dl = torch.where(self.pad, 0.0, torch.zeros_like(self.H) if dl is None else dl.double())[:, None]
        dh = (torch.zeros_like(self.H) if dh is None else dh.double())[:, None]
        hit = torch.zeros_like(self.p)
        live = (~self.pad).nonzero()[:, 0]
        hit[live, self.t[live]] = 1
        lp = torch.where(self.p > 0, self.logp, 0.0)
        H = self.H[:, None]
        dx = (dl * (hit - self.p) - dh * self.p * (lp + H)) / temperature
        tol = dl.abs() * (self.E * self.p + 4 * U) + dh.abs() * self.p * (self.E * (lp.abs() + H + 2) + 2 * self.tol_H[:, None])
        tol = tol / temperature + 4 * U * dx.abs() + torch.finfo(dtype).eps / 2 * dx.abs() + TINY[dtype]
        return dx, tol


def tops(X, k):
    """By value, then by the lower index: sorted stably on the CPU."""
    v, i = torch.sort(X.float().cpu(), dim=1, descending=True, stable=True)
    return i[:, :k].to(torch.int32)


def check(fp, X, tokens, top, temperature=1.0, out=None):
    lp = fp.token_logprobs(X, tokens, temperature=temperature, top=top, out=out)
    ex = Exact(X, tokens, temperature)
    within(lp.logprob, ex.lp, ex.tol_lp)
    within(lp.entropy, ex.H, ex.tol_H)
    within(lp.max, X.double().amax(1), 0)
    if top:
        k = min(top, X.shape[1])
        ids = tops(X, k)
        assert torch.equal(lp.top_ids[:, :k].cpu(), ids)
        at = ids.long().cuda()
        within(lp.top_logprobs[:, :k], ex.logp.gather(1, at), ex.tol_p.gather(1, at))
        assert bool((lp.top_ids[:, k:] == -1).all()) and bool((lp.top_logprobs[:, k:] == -math.inf).all())
    return lp, ex


def logits(g, T, V, dtype, ld=None, offset=0, spread=2.5):
    ld = ld or V
    buf = torch.zeros(T * ld + offset + 16, dtype=dtype, device="cuda")
    v = torch.as_strided(buf, (T, V), (ld, 1), offset)
    v.copy_(spread * torch.randn((T, V), generator=g, device="cuda"))
    return v


SHAPES = [(1, 1), (2, 2), (3, 5), (1, 31), (4, 33), (2, 255), (3, 1000), (1, 4096), (2, 4097), (5, 8191), (1, 16384), (2, 16385), (3, 32769),
          (1, 50001), (70, 131), (300, 2000), (600, 5000), (1100, 4100), (600, 20000), (40, 100003), (1, 262144)]


@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_forward(fp, T, V, dtype):
    g = torch.Generator("cuda").manual_seed(T + V)
    X = logits(g, T, V, dtype)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    tokens[1::5] = -100
    tokens[2::7] = V
    for top, temp in ((0, 1.0), (1, 0.7), (20, 1.0), (32, 1.5)):
        lp, _ = check(fp, X, tokens, top, temp)
    lp32 = fp.token_logprobs(X, tokens.to(torch.int32), temperature=1.5, top=32)
    assert torch.equal(bits(lp32), bits(lp))  # int32 tokens, and the same bits again


@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_gradient(fp, T, V, dtype):
    g = torch.Generator("cuda").manual_seed(T * 3 + V)
    X = logits(g, T, V, dtype)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    tokens[1::5] = -1
    dl, dh = torch.randn(T, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")
    lp, ex = check(fp, X, tokens, 0, 0.8)
    for a, b in ((dl, dh), (dl, None), (None, dh)):
        dx, tol = ex.gradient(a, b, 0.8, dtype)
        within(fp.token_logprobs_backward(a, b, X, tokens, lp, temperature=0.8), dx, tol)
    got = fp.token_logprobs_backward(dl, dh, X, tokens, lp, temperature=0.8)
    x = X.clone()
    assert fp.token_logprobs_backward(dl, dh, x, tokens.int(), lp, temperature=0.8, out=x) is x and torch.equal(x, got)
    assert bool((fp.token_logprobs_backward(None, None, X, tokens, lp) == 0).all())


@pytest.mark.parametrize("V", [40, 3000, 40000])
def test_gradient_by_differences(fp, V):
    """Along a random direction, the difference of the call's own outputs; the formula's curvature is taken from 64 bits."""
    g = torch.Generator("cuda").manual_seed(V)
    T, e = 3, 2.0 ** -6
    X, v = logits(g, T, V, torch.float32), torch.randn((T, V), generator=g, device="cuda")
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    dl, dh = torch.randn(T, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")
    lp = fp.token_logprobs(X, tokens)
    along = (fp.token_logprobs_backward(dl, dh, X, tokens, lp).double() * v.double()).sum(1)
    base = Exact(X, tokens, 1.0)
    d64, tol = base.gradient(dl, dh, 1.0, torch.float32)
    got, exact, noise = [], [], 0
    for s in (1, -1):
        x = X + s * e * v
        ex, at = Exact(x, tokens, 1.0), fp.token_logprobs(x, tokens)
        got.append(dl.double() * at.logprob.double() + dh.double() * at.entropy.double())
        exact.append(dl.double() * ex.lp + dh.double() * ex.H)
        noise = noise + dl.double().abs() * ex.tol_lp + dh.double().abs() * ex.tol_H
    bend = ((exact[0] - exact[1]) / (2 * e) - (d64 * v.double()).sum(1)).abs()
    moved = 2 * U / e * (d64.abs() * (X.double().abs() + 1)).sum(1)  # x + e v is rounded
    assert bool((((got[0] - got[1]) / (2 * e) - along).abs() <= bend + noise / (2 * e) + moved + (tol * v.double().abs()).sum(1)).all())


@pytest.mark.parametrize("T,V", [(3, 700), (2, 40000), (700, 3000), (520, 40000)])
@pytest.mark.parametrize("dtype", TYPES)
def test_masks(fp, T, V, dtype):
    """Banned tokens (-infinity), rows with few left, one left and none, and the type's lowest value as a mask."""
    g = torch.Generator("cuda").manual_seed(T + V)
    X = logits(g, T, V, dtype)
    X[torch.rand((T, V), generator=g, device="cuda") < 0.5] = -math.inf
    X[0] = -math.inf
    X[0, [V - 1, V // 2, 3]] = torch.tensor([1.0, 2.0, 1.0], device="cuda", dtype=dtype)
    X[1] = torch.finfo(dtype).min
    X[1, V // 3] = 0.5
    tokens = torch.zeros(T, dtype=torch.int64, device="cuda")
    tokens[0] = V // 2
    lp, ex = check(fp, X, tokens, 20)
    dl, dh = torch.randn(T, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")
    live = ~torch.isneginf(ex.lp)  # where the token is banned, p = 0 and the gradient of its log probability is -p elsewhere
    dx, tol = ex.gradient(dl, dh, 1.0, dtype)
    got = fp.token_logprobs_backward(dl, dh, X, tokens, lp)
    within(got[live], dx[live], tol[live])
    assert bool(got.isfinite().all())
    # a row without any token
    X[0] = -math.inf
    lp = fp.token_logprobs(X, tokens, top=5)
    assert float(lp.logprob[0]) == -math.inf and float(lp.entropy[0]) == 0 and float(lp.logsum[0]) == 0
    assert lp.top_ids[0].tolist() == [0, 1, 2, 3, 4] and bool((lp.top_logprobs[0] == -math.inf).all())
    got = fp.token_logprobs_backward(dl, dh, X, tokens, lp)
    assert bool((got[0] == 0).all()) and bool(got.isfinite().all())
    tokens[0] = -1
    assert float(fp.token_logprobs(X, tokens).logprob[0]) == 0


@pytest.mark.parametrize("T,V", [(3, 700), (2, 40000), (520, 40000)])
def test_infinities_and_nan(fp, T, V):
    g = torch.Generator("cuda").manual_seed(V)
    X = logits(g, T, V, torch.float32)
    clean = fp.token_logprobs(X, torch.full((T,), 4, device="cuda"), top=7)
    for bad in (math.inf, math.nan):
        x = X.clone()
        x[1, V // 2] = bad
        tokens = torch.full((T,), 4, device="cuda")
        lp = fp.token_logprobs(x, tokens, top=7)
        assert math.isnan(lp.logprob[1]) and math.isnan(lp.entropy[1]) and bool(lp.top_logprobs[1].isnan().all())
        assert bool((lp.top_ids[1] == -1).all())
        for k in ("logprob", "entropy", "top_logprobs", "top_ids"):
            assert torch.equal(getattr(lp, k)[0], getattr(clean, k)[0])
        dx = fp.token_logprobs_backward(torch.ones(T, device="cuda"), None, x, tokens, lp)
        assert bool(dx[1].isnan().any()) and bool(dx[0].isfinite().all())
    x = torch.full((T, V), math.nan, device="cuda")
    lp = fp.token_logprobs(x, tokens, top=3)
    assert bool(lp.logprob.isnan().all()) and bool((lp.top_ids == -1).all())


@pytest.mark.parametrize("T,V", [(1, 3000), (2, 70000), (700, 20000)])
@pytest.mark.parametrize("kind", ["equal", "two values", "ascending", "descending", "blocks", "thread", "zeros"])
def test_top_orders(fp, T, V, kind):
    """Rows that make many candidates: ties, sorted rows, and the greatest values all in one thread's places."""
    i = torch.arange(V, device="cuda")
    x = {"equal": torch.full((V,), 2.5, device="cuda"), "two values": (i % 2).float(), "ascending": i.float() / 64,
         "descending": (V - i).float() / 64, "blocks": ((i // 997) % 13).float(),
         "thread": torch.where((i // 8) % 256 < 40, 10.0, 0.0) + (i * 7919 % 1013).float() / 512,
         "zeros": torch.where(i % 3 == 0, -0.0, 0.0)}[kind]
    X = x.expand(T, V).contiguous()
    tokens = torch.full((T,), V - 1, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        for top in (1, 20, 32):
            check(fp, X.to(dtype), tokens, top)


@pytest.mark.parametrize("V", [50, 1023, 20001])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (8, 8), (3, 5)])
@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_guards(fp, V, pad, offset, dtype):
    g = torch.Generator("cuda").manual_seed(V)
    T = 4
    X = logits(g, T, V, dtype, V + pad, offset)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    a, b = fp.token_logprobs(X, tokens, top=9), fp.token_logprobs(X.contiguous(), tokens, top=9)
    assert torch.equal(bits(a), bits(b))
    big = torch.full((T + 2, V + 2 * pad + 2), 5.0, dtype=dtype, device="cuda")
    dx = big[1:T + 1, pad + 1:pad + 1 + V]
    d = torch.randn(T, generator=g, device="cuda")
    fp.token_logprobs_backward(d, d, X, tokens, a, out=dx)
    assert torch.equal(dx, fp.token_logprobs_backward(d, d, X.contiguous(), tokens, b))
    dx.fill_(5)
    assert bool((big == 5).all())


def test_large_logits(fp):
    """Logits of 10^4 with a narrow spread: the largest is taken off before anything is rounded."""
    g = torch.Generator("cuda").manual_seed(1)
    X = logits(g, 3, 5000, torch.float32) + 1e4
    lp, ex = check(fp, X, torch.tensor([1, 2, 3], device="cuda"), 5)
    d = torch.ones(3, device="cuda")
    dx, tol = ex.gradient(d, d, 1.0, torch.float32)
    within(fp.token_logprobs_backward(d, d, X, torch.tensor([1, 2, 3], device="cuda"), lp), dx, tol)


def test_empty(fp):
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    lp = fp.token_logprobs(torch.zeros((0, 50), device="cuda"), none, top=3)
    assert lp.logprob.shape == (0,) and lp.top_ids.shape == (0, 3)
    assert fp.token_logprobs_backward(None, None, torch.zeros((0, 50), device="cuda"), none, lp).shape == (0, 50)
    X, t = torch.zeros((2, 0), device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    lp = fp.token_logprobs(X, t, top=3)
    assert lp.logprob.tolist() == [0, 0] and lp.entropy.tolist() == [0, 0] and bool((lp.top_ids == -1).all())
    assert fp.token_logprobs_backward(None, None, X, t, lp).shape == (2, 0)


def test_rows_past_32_bits(fp):
    ld = 1 << 21
    buf = torch.zeros((1030, ld), dtype=torch.bfloat16, device="cuda")
    X = buf[:, :700]
    X.copy_(2 * torch.randn((1030, 700), device="cuda"))
    tokens = torch.randint(0, 700, (1030,), device="cuda")
    lp = fp.token_logprobs(X, tokens, top=5)
    assert torch.equal(bits(lp), bits(fp.token_logprobs(X.contiguous(), tokens, top=5)))
    d = torch.randn(1030, device="cuda")
    dx = fp.token_logprobs_backward(d, d, X, tokens, lp, out=buf[:, 1000:1700])
    assert torch.equal(dx, fp.token_logprobs_backward(d, d, X.contiguous(), tokens, lp))


@pytest.mark.parametrize("T", [2, 700])
def test_streams_and_graphs(fp, T):
    """A training step captured and replayed beside the same calls on another stream, each against the eager result."""
    g = torch.Generator("cuda").manual_seed(T)
    V = 20000
    sets = [(logits(g, T, V, torch.bfloat16), torch.randint(0, V, (T,), generator=g, device="cuda")) for _ in range(4)]
    d = torch.randn(T, generator=g, device="cuda")

    def step(X, t):
        lp = fp.token_logprobs(X, t, top=20)
        return bits(lp), fp.token_logprobs_backward(d, d, X, t, lp)
    want = [step(*s) for s in sets]
    X, t = sets[0][0].clone(), sets[0][1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(X, t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(X, t)
    for i in (1, 2, 3, 0):
        X.copy_(sets[i][0])
        t.copy_(sets[i][1])
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            other = step(*sets[(i + 1) % 4])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(other, want[(i + 1) % 4]))


@pytest.mark.parametrize("T,V", [(4, 700), (4, 40000), (520, 40000)])
@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_of_bad_rows(fp, T, V, dtype):
    """A row with a NaN or +infinity has a gradient of NaN throughout, whichever gradients come in and whatever its token; the
    rows beside it keep theirs."""
    g = torch.Generator("cuda").manual_seed(V)
    X = logits(g, T, V, dtype)
    d = torch.randn(T, generator=g, device="cuda")
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    rest = [0] + list(range(4, T))
    clean = fp.token_logprobs(X, tokens)
    X[1, V // 2], X[2, 0], X[3, V - 1] = math.nan, math.inf, math.nan
    X[3, :V - 1] = -math.inf
    for token in (4, V // 2, -1):
        tokens[1:4] = token
        lp = fp.token_logprobs(X, tokens)
        for a, b in ((d, d), (d, None), (None, d), (None, None)):
            dx = fp.token_logprobs_backward(a, b, X, tokens, lp)
            assert bool(dx[1:4].isnan().all())
            assert torch.equal(dx[rest], fp.token_logprobs_backward(a, b, torch.where(X.isfinite(), X, 0), tokens, clean)[rest])
