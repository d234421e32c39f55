"""The mixture layer for a few tokens on the GPU against 64-bit references, and a
decoding step's operators strung together.

Tolerances. u = 2^-24. The int8 rows of X are quantize_rows' bit for bit, so the
hidden products are exact. g and v = (Z x_scale) w_scale have two roundings each;
silu(g) = g / (1 + exp(-g)) is within (3 |g| + 12) u of itself (exp of an argument
that is off by 2 u |g|, of at most 4 units itself, the sum and the quotient), and a
with its product within e_a = (3 |g| + 16) u. A row's scale is within e = max e_a +
2 u; an element's step can differ from the reference's only where a 127 / max |a| is
within 127 (2 e + 5 u) of the middle between two, which adds a step of it to the
bound. What follows is linear: a term w[t, k] (Z scale) d_scale has e and three
roundings, their sum over k one each, and the output half a step, eps / 2."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = {torch.float32: 1e-38, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38}


class Layer:
    def __init__(self, fp, g, E, d, ff, gate, pad=0):
        maps = {"up": (ff, d), "down": (d, ff)}
        if gate:
            maps["gate"] = (ff, d)
        self.W = {k: torch.randint(-128, 128, (E,) + s, generator=g, device="cuda", dtype=torch.int8) for k, s in maps.items()}
        self.s = {}
        for k, s in maps.items():
            wide = torch.zeros((E, s[0] + pad), device="cuda")
            wide[:, :s[0]] = (0.5 + torch.rand((E, s[0]), generator=g, device="cuda")) / (74 * s[1] ** 0.5)
            self.s[k] = wide[:, :s[0]]
        self.P = {k: fp.pack_experts(w) for k, w in self.W.items()}
        self.E, self.d, self.ff, self.gate = E, d, ff, gate

    def __call__(self, fp, X, ids, w, **kw):
        if self.gate:
            kw.update(gate=self.P["gate"], gate_scale=self.s["gate"])
        return fp.moe_layer(X, ids, w, self.P["up"], self.s["up"], self.P["down"], self.s["down"], **kw)

    def check(self, Y, Xq, xs, ids, w):
        """Y against 64 bits, from the int8 rows."""
        T, K = ids.shape
        want = torch.zeros((T, self.d), dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(want)
        q, xs = Xq.double(), xs.double()
        for e in range(self.E):
            t, k = (ids == e).nonzero(as_tuple=True)
            if not t.numel():
                continue

            def product(name):
                return (q[t] @ self.W[name][e].double().t()) * xs[t][:, None] * self.s[name][e].double()
            v = product("up")
            g = product("gate") if self.gate else v
            a = torch.nn.functional.silu(g)
            if self.gate:
                a = a * v
            e_a = (3 * g.abs() + 16) * U
            err = e_a.amax(1, keepdim=True) + 2 * U
            top = a.abs().amax(1, keepdim=True)
            x = torch.where(top > 0, a * 127 / top, 0.0)
            n = torch.round(x)
            between = ((x - torch.floor(x) - 0.5).abs() <= 127 * (2 * err + 5 * U)).double()
            D = self.W["down"][e].double().t()
            f = w[t, k].double()[:, None] * (top / 127) * self.s["down"][e].double()
            y = (n @ D) * f
            want.index_add_(0, t, y)
            tol.index_add_(0, t, y.abs() * (err + (4 + K) * U) + f.abs() * (between @ D.abs()))
        dt = Y.dtype
        tol = tol + torch.finfo(dt).eps / 2 * (want.abs() + tol) + TINY[dt]
        bad = ~((Y.double() - want).abs() <= tol)
        assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:3].tolist(), Y[bad][:3], want[bad][:3], tol[bad][:3])


def tokens(g, T, d, dtype, ld=None, offset=0):
    ld = ld or d
    buf = torch.zeros(T * ld + offset + 16, dtype=dtype, device="cuda")
    v = torch.as_strided(buf, (T, d), (ld, 1), offset)
    v.copy_(torch.randn((T, d), generator=g, device="cuda") * torch.exp(torch.randn((T, 1), generator=g, device="cuda")))
    return v


def route(g, T, K, E, drop=0.0, wide=False):
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:K] for _ in range(T)]) if K <= E else \
        torch.randint(0, E, (T, K), generator=g, device="cuda")
    ids[torch.rand((T, K), generator=g, device="cuda") < drop] = -1
    return ids if wide else ids.to(torch.int32), torch.softmax(torch.randn((T, K), generator=g, device="cuda"), 1)


# one token to as many slots as there are; one expert to more than a word of the bitmap; ragged widths around every tile and unit
CASES = [(1, 1, 1, 64, 64), (1, 8, 128, 256, 128), (2, 2, 4, 1, 1), (3, 2, 5, 15, 17), (8, 2, 16, 512, 768), (5, 4, 33, 63, 31),
         (9, 1, 3, 65, 33), (16, 2, 4, 100, 257), (33, 1, 1, 128, 96), (61, 3, 20, 200, 333), (64, 16, 40, 48, 64), (64, 1, 2, 1000, 130),
         (1, 16, 600, 40, 40), (7, 3, 1024, 24, 40), (1024, 1, 12, 32, 64), (10, 100, 7, 64, 32), (4, 2, 6, 2100, 1029), (12, 5, 9, 129, 2050), (2, 1, 3, 64, 5000), (8, 8, 64, 640, 2100),
         (20, 1, 3, 64, 5000), (40, 2, 60, 640, 1100), (32, 4, 64, 96, 160), (32, 1, 16, 200, 130), (16, 2, 16, 64, 3000)]


@pytest.mark.parametrize("T,K,E,d,ff", CASES)
@pytest.mark.parametrize("gate", [True, False])
def test_layer(fp, T, K, E, d, ff, gate):
    g = torch.Generator("cuda").manual_seed(T * 7 + E + d)
    L = Layer(fp, g, E, d, ff, gate)
    for i, dtype in enumerate((torch.bfloat16, torch.float16, torch.float32)):
        X = tokens(g, T, d, dtype)
        ids, w = route(g, T, K, E, drop=(0.0, 0.2, 0.6)[i], wide=i == 1)
        q, s = fp.quantize_rows(X)
        for out in (dtype, torch.float32):
            Y = L(fp, X, ids, w, dtype=out)
            assert Y.dtype == out
            L.check(Y, q, s, ids, w)
        assert torch.equal(L(fp, q, ids, w, x_scale=s, dtype=torch.float32), Y)  # the same rows, quantized before the call
    assert L(fp, q, ids, w, x_scale=s).dtype == torch.bfloat16


def test_same_experts(fp):
    """A token that names an expert twice, and every token the same ones."""
    g = torch.Generator("cuda").manual_seed(4)
    L = Layer(fp, g, 6, 96, 160, True)
    X = tokens(g, 40, 96, torch.float32)
    for T in (40, 8, 3):  # with few tokens too an expert has more than eight rows
        ids = torch.tensor([[2, 2, 5]], dtype=torch.int32, device="cuda").repeat(T, 1)
        w = torch.rand((T, 3), generator=g, device="cuda")
        q, s = fp.quantize_rows(X[:T])
        L.check(L(fp, X[:T], ids, w), q, s, ids, w)
    L = Layer(fp, g, 64, 96, 160, False)  # 32 tokens, two rows an expert on average, all of them with two experts
    ids = torch.tensor([[7, 60, 7, 60]], device="cuda").repeat(32, 1)
    w = torch.rand((32, 4), generator=g, device="cuda")
    q, s = fp.quantize_rows(X[:32])
    L.check(L(fp, X[:32], ids, w), q, s, ids, w)


@pytest.mark.parametrize("wide", [False, True])
def test_without_experts(fp, wide):
    """Ids outside the experts, some or all of them; tokens without any get zeros."""
    g = torch.Generator("cuda").manual_seed(5)
    L = Layer(fp, g, 3, 70, 50, True)
    X = tokens(g, 6, 70, torch.float32)
    ids = torch.tensor([[0, 2], [-1, 3], [3, 1], [-7, -1], [2 ** 31 - 1, -2 ** 31], [1, 1000]], device="cuda")
    if wide:
        ids[4] = torch.tensor([2 ** 32, -2 ** 32 + 1], device="cuda")  # 0 and 1 in their low halves
    ids = ids if wide else ids.to(torch.int32)
    w = torch.rand((6, 2), generator=g, device="cuda")
    q, s = fp.quantize_rows(X)
    Y = L(fp, X, ids, w)
    L.check(Y, q, s, ids, w)
    assert bool((Y[[1, 3, 4]] == 0).all()) and bool((Y[0] != 0).any())
    out = torch.full((6, 70), 3.0, device="cuda")
    L(fp, X, torch.full_like(ids, -1), w, out=out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (16, 16), (5, 7)])
@pytest.mark.parametrize("dtype", [torch.int8, torch.bfloat16, torch.float32])
def test_strides_and_guards(fp, pad, offset, dtype):
    """Rows of X, scales and Y at strides and addresses of their own; nothing beside Y is written."""
    g = torch.Generator("cuda").manual_seed(6)
    d = 150
    L = Layer(fp, g, 5, d, 77, True, pad=3)
    ids, w = route(g, 9, 2, 5)
    if dtype == torch.int8:
        buf = torch.randint(-127, 128, (9 * (d + pad) + offset,), generator=g, device="cuda", dtype=torch.int8)  # the last row ends the storage
        X, kw = torch.as_strided(buf, (9, d), (d + pad, 1), offset)[:, :], {"x_scale": torch.rand(9, generator=g, device="cuda") / 50}
    else:
        X, kw = tokens(g, 9, d, dtype, d + pad, offset), {}
    want = L(fp, X.contiguous(), ids, w, dtype=torch.float32, **kw)
    for out in (torch.float32, torch.bfloat16, torch.float16):
        big = torch.full((11, d + 2 * pad + 3), 5.0, dtype=out, device="cuda")
        Y = big[1:10, pad + 1:pad + 1 + d]
        L(fp, X, ids, w, out=Y, **kw)
        assert torch.equal(Y, want.to(out))
        Y.fill_(5)
        assert bool((big == 5).all())


def test_bad_rows_stay_alone(fp):
    """An infinity, a NaN, zeros and huge values in a token's row do not reach the others."""
    g = torch.Generator("cuda").manual_seed(7)
    L = Layer(fp, g, 4, 128, 64, True)
    X = tokens(g, 12, 128, torch.float32)
    ids, w = route(g, 12, 2, 4)
    want = L(fp, X, ids, w)
    x = X.clone()
    x[1, 5], x[3, 100], x[4], x[6] = float("inf"), float("nan"), 0, 1e30
    Y = L(fp, x, ids, w)
    same = [0, 2, 5, 7, 8, 9, 10, 11]
    assert torch.equal(Y[same], want[same])
    assert bool(Y[[1, 3]].isnan().all()) and bool((Y[4] == 0).all())


@pytest.mark.parametrize("T", [5, 40])
def test_over_its_input(fp, T):
    """Y written over X."""
    g = torch.Generator("cuda").manual_seed(14)
    L = Layer(fp, g, 6, 200, 90, True)
    X = tokens(g, T, 200, torch.bfloat16)
    ids, w = route(g, T, 2, 6)
    want = L(fp, X, ids, w)
    x = X.clone()
    assert L(fp, x, ids, w, out=x) is x and torch.equal(x, want)


def test_no_tokens(fp):
    g = torch.Generator("cuda").manual_seed(8)
    L = Layer(fp, g, 4, 64, 64, False)
    Y = L(fp, torch.zeros((0, 64), device="cuda"), torch.zeros((0, 2), dtype=torch.int32, device="cuda"), torch.zeros((0, 2), device="cuda"))
    assert Y.shape == (0, 64)


def test_same_as_strung_together(fp):
    """The layer from the calls for many tokens, with torch's activation between: the same up to an element's step here and there
    (a quantized value next to the middle of two), which is bounded as in Layer.check against the same 64-bit answer."""
    g = torch.Generator("cuda").manual_seed(9)
    T, K, E, d, ff = 48, 4, 12, 320, 272
    L = Layer(fp, g, E, d, ff, True)
    X = tokens(g, T, d, torch.bfloat16)
    ids, w = route(g, T, K, E)
    q, s = fp.quantize_rows(X)
    plan = fp.moe_sort(ids, E)
    up = fp.scaled_matmul_grouped(q, s, L.P["up"], L.s["up"], plan.offsets, rows=plan.tokens, dtype=torch.float32)
    gt = fp.scaled_matmul_grouped(q, s, L.P["gate"], L.s["gate"], plan.offsets, rows=plan.tokens, dtype=torch.float32)
    aq, a_s = fp.quantize_rows(torch.nn.functional.silu(gt) * up)
    O = fp.scaled_matmul_grouped(aq, a_s, L.P["down"], L.s["down"], plan.offsets, dtype=torch.float32)  # noqa: E741
    L.check(fp.moe_combine(O, plan, w), q, s, ids, w)
    L.check(L(fp, X, ids, w, dtype=torch.float32), q, s, ids, w)


def test_streams_and_graphs(fp):
    """Captured and replayed beside the same call on another stream: arrivals and scratch of the two do not meet."""
    g = torch.Generator("cuda").manual_seed(10)
    L = Layer(fp, g, 16, 512, 320, True)
    sets = [(tokens(g, 8, 512, torch.bfloat16),) + route(g, 8, 2, 16, drop=0.1) for _ in range(4)]
    want = [L(fp, *s) for s in sets]
    args = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L(fp, *args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = L(fp, *args)
    for i in (1, 2, 3, 0, 2):
        for a, b in zip(args, sets[i]):
            a.copy_(b)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            other = L(fp, *sets[(i + 1) % 4])
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]) and torch.equal(other, want[(i + 1) % 4])


def test_table_of_experts(fp):
    """The addresses that the layer reads on the device are those of the packed weights."""
    W = torch.randint(-8, 8, (5, 40, 70), device="cuda", dtype=torch.int8)
    P = fp.pack_experts(W)
    assert P.table.tolist() == [w.data.data_ptr() for w in P.weights] == [ctypes.c_void_p(p).value for p in P.ptrs]


def test_experts_put_together_inside_a_capture(fp):
    """The packed weights as experts again, inside a capture: the grouped product's launch needs no table, the layer's refuses
    there, and has it afterwards."""
    g = torch.Generator("cuda").manual_seed(13)
    L = Layer(fp, g, 3, 64, 96, False)
    X = tokens(g, 5, 64, torch.bfloat16)
    q, s = fp.quantize_rows(X)
    ids, w = route(g, 5, 2, 3)
    plan = fp.moe_sort(ids, 3)
    want, layer = fp.scaled_matmul_grouped(q, s, L.P["up"], L.s["up"], plan.offsets, rows=plan.tokens), L(fp, X, ids, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        up = fp.PackedExperts(L.P["up"].weights)
        Y = fp.scaled_matmul_grouped(q, s, up, L.s["up"], plan.offsets, rows=plan.tokens)
        with pytest.raises(ValueError, match="capture"):
            fp.moe_layer(X, ids, w, up, L.s["up"], L.P["down"], L.s["down"])
    for _ in range(2):
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)
    assert torch.equal(fp.moe_layer(X, ids, w, up, L.s["up"], L.P["down"], L.s["down"]), layer)


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, fp, X, w):
        ctx.fp = fp
        ctx.save_for_backward(X, w)
        return fp.rms_norm(X, w)

    @staticmethod
    def backward(ctx, dY):
        dX, dw = ctx.fp.rms_norm_backward(dY.contiguous(), *ctx.saved_tensors)
        return None, dX, dw


class _Logprob(torch.autograd.Function):
    @staticmethod
    def forward(ctx, fp, logits, tokens):
        lp = fp.token_logprobs(logits, tokens)
        ctx.fp, ctx.lp = fp, lp
        ctx.save_for_backward(logits, tokens)
        return lp.logprob, lp.entropy

    @staticmethod
    def backward(ctx, dl, dh):
        logits, t = ctx.saved_tensors
        return None, ctx.fp.token_logprobs_backward(dl.contiguous(), dh.contiguous(), logits, t, ctx.lp), None


def test_training_through_them(fp):
    """Norm, head and log probabilities as autograd Functions: the gradients of a loss against 64 bits. The forward errors of
    the logits (fp32 products of 96 terms, at most 100 u of their absolute sums) reach the gradients through a softmax, whose
    slopes are at most 1 a unit of logit and token: 1e-4 of each gradient's largest value bounds all with room."""
    g = torch.Generator("cuda").manual_seed(11)
    T, d, V = 24, 96, 500
    X, w, head = (torch.randn(s, generator=g, device="cuda") * c for s, c in (((T, d), 1.0), ((d,), 1.0), ((V, d), d ** -0.5)))
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    a = [v.clone().requires_grad_() for v in (X, w, head)]
    lp, h = _Logprob.apply(fp, _Norm.apply(fp, a[0], a[1]) @ a[2].t(), t)
    (-lp.mean() - 0.1 * h.mean()).backward()
    b = [v.double().requires_grad_() for v in (X, w, head)]
    n = b[0] * torch.rsqrt((b[0] * b[0]).mean(1, keepdim=True) + 1e-5) * b[1]
    log = torch.log_softmax(n @ b[2].t(), 1)
    (-log.gather(1, t[:, None]).mean() + 0.1 * (log.exp() * log).sum(1).mean()).backward()
    for x, y in zip(a, b):
        assert float((x.grad.double() - y.grad).abs().max()) <= 1e-4 * float(y.grad.abs().max())


def test_decoding_step(fp):
    """A decoding step after attention: norm with the residual, router, mixture, norm with the residual, head, log
    probabilities; each against what it stands for, and the whole captured and replayed with other inputs."""
    g = torch.Generator("cuda").manual_seed(12)
    T, d, ff, E, K, V = 6, 256, 192, 10, 2, 3001
    L = Layer(fp, g, E, d, ff, True)
    w1, w2 = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    router = torch.randn((d, E), generator=g, device="cuda") / d ** 0.5
    W = torch.randint(-128, 128, (V, d), generator=g, device="cuda", dtype=torch.int8)
    head, hs = fp.pack_weights(W), torch.full((V,), 3 / (74 * d ** 0.5), device="cuda")

    def step(x, stream, sampled):
        n = torch.empty_like(x)
        q, s, h = fp.rms_norm_quantize(x, w1, residual=stream, Y=n)
        weights, ids = torch.softmax(n.float() @ router, 1).topk(K, dim=1)
        y = L(fp, q, ids, weights, x_scale=s)
        q2, s2, h2 = fp.rms_norm_quantize(y, w2, residual=h)
        logits = fp.scaled_matmul(q2, s2, head, hs, dtype=torch.float32)
        lp = fp.token_logprobs(logits, sampled, top=5)
        return q, s, h, n, ids, weights, y, q2, s2, h2, logits, lp.logprob, lp.top_ids
    sets = [tuple((torch.randn((T, d), generator=g, device="cuda")).bfloat16() for _ in range(2)) + (torch.randint(0, V, (T,), generator=g, device="cuda"),)
            for _ in range(3)]
    eager = [step(*s) for s in sets]
    x, stream, sampled = sets[0]
    q, s, h, n, ids, weights, y, q2, s2, h2, logits, lp, top = eager[0]
    hd = x.double() + stream.double()
    nd = hd * torch.rsqrt((hd * hd).mean(1, keepdim=True) + 1e-5) * w1.double()
    assert bool(((q.double() * s.double()[:, None] - nd).abs() <= (0.5 + 2.0 ** -13) * s.double()[:, None]).all())
    L.check(y, q, s, ids, weights)
    assert torch.equal(h2, (y.float() + h.float()).bfloat16())
    want = (q2.double() @ W.double().t()) * s2.double()[:, None] * hs.double()
    assert bool(((logits.double() - want).abs() <= 4 * U * want.abs() + 1e-38).all())
    log = torch.log_softmax(logits.double(), 1)
    assert float((lp.double() - log.gather(1, sampled[:, None])[:, 0]).abs().max()) <= 200 * U
    assert torch.equal(top.cpu().long(), torch.sort(logits.cpu(), dim=1, descending=True, stable=True)[1][:, :5])
    args = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*args)
    for i in (1, 2, 0):
        for a, b in zip(args, sets[i]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager[i]))


def test_packing_does_not_wait(fp):
    """Packing the experts leaves the host free: neither the weights nor the addresses wait for the device."""
    W = torch.randint(-8, 8, (5, 40, 70), device="cuda", dtype=torch.int8)
    torch.cuda.synchronize()
    torch.cuda.set_sync_debug_mode("error")
    try:
        P = fp.pack_experts(W)
        Q = fp.PackedExperts(P.weights)
    finally:
        torch.cuda.set_sync_debug_mode("default")
    for experts in (P, Q):
        assert experts.table.tolist() == [w.data.data_ptr() for w in P.weights]


def test_packed_on_another_stream(fp):
    """Experts put together behind other work on one stream and used at once on another: the layer waits for their addresses."""
    g = torch.Generator("cuda").manual_seed(21)
    L = Layer(fp, g, 6, 96, 160, True)
    X = tokens(g, 5, 96, torch.bfloat16)
    ids, w = route(g, 5, 2, 6)
    want = L(fp, X, ids, w)
    A = torch.randn((4096, 4096), generator=g, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            A = A @ A / 64
        again = {k: fp.PackedExperts(p.weights) for k, p in L.P.items()}
    Y = fp.moe_layer(X, ids, w, again["up"], L.s["up"], again["down"], L.s["down"], gate=again["gate"], gate_scale=L.s["gate"])
    assert torch.equal(Y, want)
    torch.cuda.synchronize()


def test_packed_and_captured_at_once(fp):
    """The first call with newly packed experts is inside a capture."""
    g = torch.Generator("cuda").manual_seed(22)
    L, M = (Layer(fp, g, 6, 96, 160, True) for _ in range(2))
    X = tokens(g, 5, 96, torch.bfloat16)
    ids, w = route(g, 5, 2, 6)
    M(fp, X, ids, w)  # (libraries are loaded outside of captures)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = L(fp, X, ids, w)
    want = L(fp, X, ids, w)
    for _ in range(3):
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)


def panels_of(ids, d):
    """How many 32-output panels the second launch has: all of those of every expert that a token meets."""
    return ids[ids >= 0].unique().numel() * ((d + 31) // 32)


# ff short of eight units of K, so that no panel is cut, and more panels than the 768 (float rows) or 1024 (int8 rows) workgroups
@pytest.mark.parametrize("T,K,E,d,ff,held", [(16, 4, 64, 1024, 512, 768), (32, 4, 64, 2048, 1024, 768), (5, 8, 40, 1100, 270, 768), (40, 4, 64, 1024, 512, 1024),
                                             (64, 8, 48, 1000, 333, 1024)])
@pytest.mark.parametrize("gate", [True, False])
def test_whole_panels_several_to_a_workgroup(fp, T, K, E, d, ff, held, gate):
    g = torch.Generator("cuda").manual_seed(T + d + ff)
    L = Layer(fp, g, E, d, ff, gate, pad=5)
    for dtype, drop in ((torch.bfloat16, 0.0), (torch.float32, 0.1)):
        X = tokens(g, T, d, dtype)
        ids, w = route(g, T, K, E, drop=drop)
        assert panels_of(ids, d) > held
        q, s = fp.quantize_rows(X)
        Y = L(fp, X, ids, w, dtype=torch.float32)
        L.check(Y, q, s, ids, w)
        assert torch.equal(L(fp, q, ids, w, x_scale=s, dtype=torch.float32), Y)


@pytest.mark.parametrize("T,K,E,d,ff", [(8, 2, 16, 512, 2048), (16, 4, 64, 1024, 512), (40, 2, 16, 512, 320), (40, 2, 16, 256, 1100)])
def test_streams_and_graphs_of_every_way(fp, T, K, E, d, ff):
    """Cut sums, several whole panels to a workgroup, and both of them with the rows quantized between: captured and replayed
    beside the same calls on another stream, int8 rows too."""
    g = torch.Generator("cuda").manual_seed(T + ff)
    L = Layer(fp, g, E, d, ff, True)
    sets = []
    for i in range(3):
        X = tokens(g, T, d, torch.bfloat16)
        sets.append((X,) + route(g, T, K, E, drop=0.1 * i) + fp.quantize_rows(X))

    def both(X, ids, w, q, s):
        return L(fp, X, ids, w), L(fp, q, ids, w, x_scale=s)
    want = [both(*s) for s in sets]
    for (X, ids, w, q, s), (a, b) in zip(sets, want):
        L.check(a, q, s, ids, w)
        assert torch.equal(a, b)
    args = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(*args)
    for i in (1, 2, 0, 2, 1):
        for a, b in zip(args, sets[i]):
            a.copy_(b)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            other = both(*sets[(i + 1) % 3])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(other, want[(i + 1) % 3]))


def test_values_that_leave_fp32(fp):
    """A row of huge values: with a gate the hidden values leave fp32, which makes the token's output NaN; without one they do
    not, and the output is as exact as any."""
    g = torch.Generator("cuda").manual_seed(23)
    for gate in (True, False):
        L = Layer(fp, g, 4, 128, 64, gate)
        X = tokens(g, 12, 128, torch.float32)
        X[6] = 1e30
        ids, w = route(g, 12, 2, 4)
        q, s = fp.quantize_rows(X)
        Y = L(fp, X, ids, w)
        if gate:
            assert bool(Y[6].isnan().all())
            X[6] = 0
            q, s = fp.quantize_rows(X)
            Y[6] = L(fp, X, ids, w)[6]
        L.check(Y, q, s, ids, w)
