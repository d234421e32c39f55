"""Tokens sorted by expert, gathered and combined on the GPU, with their
gradients, against 64-bit references; and a whole expert layer strung together
from them and the grouped scaled products.

Tolerances, with u = 2^-24: a sum of n fp32 fused multiply-adds is off by at
most ((1 + u)^n - 1) sum |terms| <= 1.01 n u sum |terms| in any order, a product
by u of itself; rounding to the output's type adds eps / 2 of the value (fp16:
at least 2^-25)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def within(got, want, fp32_err, dtype):
    got = got.double().cpu().numpy()
    tol = fp32_err + torch.finfo(dtype).eps / 2 * (np.abs(want) + fp32_err) + 2.0 ** -25 * (dtype == torch.float16) + 1e-38
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


def sorted_slots(ids, E):
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    rows = np.empty(len(flat), np.int64)
    rows[order] = np.arange(len(flat))
    rows[key == E] = -1
    slots = np.where(key[order] < E, order, -1)
    offsets = np.searchsorted(key[order], np.arange(E + 1))
    return offsets, slots, rows.reshape(ids.shape)


def check_plan(plan, ids, E):
    offsets, slots, rows = sorted_slots(ids, E)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.slots.cpu().numpy(), slots)
    assert np.array_equal(plan.tokens.cpu().numpy(), np.where(slots >= 0, slots // ids.shape[1], -1))
    assert np.array_equal(plan.rows.cpu().numpy(), rows)
    return offsets, slots, rows


def draw_ids(rng, T, K, E, kind):
    if kind == "one":        # every slot to the last expert
        return np.full((T, K), E - 1)
    if kind == "none":       # no slot has an expert
        return np.where(rng.random((T, K)) < 0.5, -1, E)
    if kind == "wild":       # ids outside [0, E) of every size, repeated experts in a token
        ids = rng.integers(-2, E + 2, (T, K))
        ids[rng.random((T, K)) < 0.05] = -2 ** 31
        ids[rng.random((T, K)) < 0.05] = 2 ** 31 - 1
        return ids
    p = 1.0 / np.arange(1, E + 1)
    return rng.choice(E, size=(T, K), p=p / p.sum())


@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (1, 8, 128), (3, 2, 5), (63, 1, 2), (64, 4, 64), (65, 3, 7), (1000, 8, 128), (1024, 8, 60),
                                   (1025, 8, 60), (4100, 2, 1000), (5000, 6, 1024), (40000, 8, 256), (300000, 1, 16), (0, 4, 8)])
@pytest.mark.parametrize("kind", ["skewed", "one", "none", "wild"])
def test_sort(fp, T, K, E, kind):
    rng = np.random.default_rng(T + K + E)
    ids = draw_ids(rng, T, K, E, kind)
    for dt in (torch.int32, torch.int64):
        check_plan(fp.moe_sort(torch.from_numpy(ids).cuda().to(dt), E), ids, E)
    if kind == "wild" and T:  # 64-bit ids that 32 bits would cut to experts
        far = ids.astype(np.int64) + (1 << 32)
        plan = fp.moe_sort(torch.from_numpy(far).cuda(), E)
        assert int(plan.offsets[-1]) == 0 and bool((plan.rows == -1).all()) and bool((plan.slots == -1).all())


def test_sort_agrees_with_the_host_plan(fp):
    rng = np.random.default_rng(0)
    route = rng.integers(0, 12, 500).astype(np.int32)
    counts, offsets, perm = fp.moe_plan(route, 12)
    plan = fp.moe_sort(torch.from_numpy(route[:, None]).cuda(), 12)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets) and np.array_equal(plan.tokens.cpu().numpy(), perm)
    X = torch.from_numpy(rng.integers(-128, 128, (500, 96), dtype=np.int8)).cuda()
    assert torch.equal(fp.moe_permute(X, plan), fp.gather_rows(X, torch.from_numpy(perm).cuda()))


MOVES = [(1, 1, 1, 1), (1, 8, 128, 5120), (3, 2, 4, 7), (65, 3, 7, 96), (300, 6, 60, 1111), (129, 2, 9, 4096), (700, 8, 32, 200), (5, 16, 20, 24),
         (2, 1, 3, 20000), (1200, 8, 64, 64),
         (20, 4, 1000, 33), (3, 20, 30, 40), (512, 4, 700, 16)]


@pytest.mark.parametrize("T,K,E,d", MOVES)
@pytest.mark.parametrize("dt", TYPES + [torch.int8])
def test_dispatch(fp, T, K, E, d, dt):
    rng = np.random.default_rng(T + d)
    ids = draw_ids(rng, T, K, E, "wild" if T % 2 else "skewed")
    _, slots, rows = sorted_slots(ids, E)
    for left, right in ((0, 0), (1, 2)):
        big = (torch.from_numpy(rng.standard_normal((T, left + d + right)).astype(np.float32)).cuda() * 50).to(dt)
        X = big[:, left:left + d]
        out = torch.full((T * K + 2, left + d + right), 9, dtype=dt, device="cuda")
        Xs, plan = fp.moe_dispatch(X, torch.from_numpy(ids).cuda(), E, out=out[1:-1, left:left + d])
        check_plan(plan, ids, E)
        live = torch.from_numpy(slots >= 0).cuda()
        tok = torch.from_numpy(np.maximum(slots, 0) // K).cuda()
        assert torch.equal(Xs[live], X[tok][live]) and bool((Xs[~live] == 9).all())
        again = fp.moe_permute(X, plan)
        assert torch.equal(again[live], Xs[live])
        Xs.fill_(9)
        assert bool((out == 9).all())


@pytest.mark.parametrize("T,K", [(6, 3), (1100, 4)])
@pytest.mark.parametrize("d,pad", [(1, 0), (2, 0), (3, 0), (1023, 0), (1025, 0), (4098, 0), (4103, 0), (2052, 4), (4111, 1), (8210, 2)])
@pytest.mark.parametrize("dt", [torch.int8, torch.bfloat16])
def test_rows_of_every_length(fp, T, K, d, pad, dt):
    """Rows that end in each part of a word, over several pieces, in both launches."""
    E = 7
    rng = np.random.default_rng(d + T)
    ids = draw_ids(rng, T, K, E, "wild")
    _, slots, _ = sorted_slots(ids, E)
    X = torch.from_numpy(rng.integers(-128, 128, (T, d + pad), dtype=np.int8)).cuda().to(dt)[:, :d]
    out = torch.full((T * K, d + pad), 99, dtype=dt, device="cuda")
    fp.moe_dispatch(X, torch.from_numpy(ids).cuda(), E, out=out[:, :d])
    want = torch.full((T * K, d + pad), 99, dtype=dt, device="cuda")
    live = torch.from_numpy(slots >= 0).cuda()
    want[live, :d] = X[torch.from_numpy(slots[slots >= 0] // K).cuda()]
    assert torch.equal(out, want)


@pytest.mark.parametrize("T,K,E,d", MOVES)
@pytest.mark.parametrize("dt", TYPES)
def test_combine_and_gradients(fp, T, K, E, d, dt):
    rng = np.random.default_rng(T * 3 + d)
    ids = draw_ids(rng, T, K, E, "wild" if d % 2 else "skewed")
    plan = fp.moe_sort(torch.from_numpy(ids).cuda(), E)
    _, slots, rows = sorted_slots(ids, E)
    n = T * K
    for left, right in ((0, 0), (1, 2)):
        def mat(r):
            return torch.from_numpy(rng.standard_normal((r, left + d + right)).astype(np.float32)).cuda().to(dt)[:, left:left + d]
        O, dY, dXs = mat(n), mat(T), mat(n)  # noqa: E741
        w = torch.from_numpy(rng.random((T, K)).astype(np.float32)).cuda()
        o64, dy64, dx64, w64 = (t.double().cpu().numpy() for t in (O, dY, dXs, w))
        live = rows >= 0
        pick = np.maximum(rows, 0)
        terms = np.where(live[:, :, None], w64[:, :, None] * o64[pick], 0)
        err = 1.01 * K * U * np.abs(terms).sum(1)
        within(fp.moe_combine(O, plan, w), terms.sum(1), err, dt)
        terms = np.where(live[:, :, None], o64[pick], 0)
        within(fp.moe_combine(O, plan), terms.sum(1), 1.01 * K * U * np.abs(terms).sum(1), dt)
        terms = np.where(live[:, :, None], dx64[pick], 0)
        within(fp.moe_dispatch_backward(dXs, plan), terms.sum(1), 1.01 * K * U * np.abs(terms).sum(1), dt)
        # gradients of the combination, into rows of a wider buffer
        buf = torch.full((n + 2, left + d + right), 9.0, dtype=dt, device="cuda")
        dO = buf[1:-1, left:left + d]
        got, dw = fp.moe_combine_backward(dY, O, plan, w, dO=dO)
        has = slots >= 0
        s = np.maximum(slots, 0)
        want = w64.reshape(-1)[s][:, None] * dy64[s // K]
        within(got[torch.from_numpy(has).cuda()], want[has], U * np.abs(want[has]), dt)
        assert bool((got[torch.from_numpy(~has).cuda()] == 9.0).all())
        prod = np.where(live[:, :, None], dy64[:, None, :] * o64[pick], 0)
        within(dw, prod.sum(2), 1.01 * d * U * np.abs(prod).sum(2), torch.float32)
        assert bool((dw[torch.from_numpy(~live).cuda()] == 0).all())
        got2, dw2 = fp.moe_combine_backward(dY, O, plan, w)
        assert torch.equal(dw, dw2)  # a fixed order of summation
        dO.fill_(9.0)
        assert bool((buf == 9.0).all())


def test_rows_past_32_bits(fp):
    """Sorted rows that start more than 2^31 elements into their tensor, there and back."""
    T, K, E, d = 270000, 2, 16, 4096  # Xs: 2.2 G elements
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    X = torch.randn((T, d), generator=g, device="cuda", dtype=torch.bfloat16)
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((T, K), generator=g, device="cuda")
    Xs, plan = fp.moe_dispatch(X, ids, E)
    at = torch.cat([torch.arange(0, 50), torch.arange(T * K - 50, T * K), torch.randint(0, T * K, (200,))]).cuda()
    assert torch.equal(Xs[at], X[plan.tokens[at].long()])
    Y = fp.moe_combine(Xs, plan, w)          # both choices hold the token's own row
    t = torch.cat([torch.arange(0, 20), torch.arange(T - 20, T)]).cuda()
    x64, w64 = X[t].double().cpu().numpy(), w[t].double().cpu().numpy()
    terms = w64[:, :, None] * x64[:, None, :]
    within(Y[t], terms.sum(1), 1.01 * K * U * np.abs(terms).sum(1), torch.bfloat16)
    dO, dw = fp.moe_combine_backward(X, Xs, plan, w)
    rows = plan.rows[t].long()
    for k in range(K):
        want = w64[:, k, None] * x64
        within(dO[rows[:, k]], want, U * np.abs(want), torch.bfloat16)
        within(dw[t, k], (x64 * x64).sum(1), 1.01 * d * U * (x64 * x64).sum(1), torch.float32)


def test_combine_infinities_and_no_rows(fp):
    """An infinity or a NaN stays with the tokens that have its row; a weight of zero does not hide a NaN; tokens whose
    slots all were dropped get zeros."""
    ids = torch.tensor([[0, 1], [-1, 2], [-1, -1]], device="cuda")
    plan = fp.moe_sort(ids, 2)
    O = torch.ones((6, 40), device="cuda")  # noqa: E741
    O[1, 3], O[0, 5] = float("nan"), float("inf")
    O[2:] = float("nan")  # rows of no slot
    y = fp.moe_combine(O, plan, torch.tensor([[1.0, 0.0], [1, 1], [1, 1]], device="cuda"))
    assert bool(torch.isnan(y[0, 3])) and bool(torch.isinf(y[0, 5])) and float(y[0, 0]) == 1.0
    assert bool((y[1:] == 0).all())


def test_gradients_by_differences(fp):
    """The loss sum G * combine(O(X), w), O linear in the gathered rows, is linear in each argument, so differences of
    the 64-bit plain form give its derivatives up to rounding."""
    T, K, E, d = 7, 3, 5, 12
    rng = np.random.default_rng(2)
    ids = draw_ids(rng, T, K, E, "wild")
    offsets, slots, rows = sorted_slots(ids, E)
    X, G, w = rng.standard_normal((T, d)), rng.standard_normal((T, d)), rng.random((T, K))
    X, G, w = (a.astype(np.float32).astype(np.float64) for a in (X, G, w))
    gain = np.repeat(np.arange(1.0, E + 1), np.diff(offsets)).tolist() + [0.0] * (T * K - offsets[-1])  # expert e: (e + 1) x

    def loss(X, w):
        out = 0.0
        for t in range(T):
            for k in range(K):
                if rows[t, k] >= 0:
                    out += w[t, k] * gain[rows[t, k]] * float(X[t] @ G[t])
        return out
    c = lambda a: torch.from_numpy(np.asarray(a, np.float32)).cuda()  # noqa: E731
    Xs, plan = fp.moe_dispatch(c(X), torch.from_numpy(ids).cuda(), E, out=torch.zeros((T * K, d), device="cuda"))
    O = Xs * c(gain)[:, None]  # noqa: E741
    dO, dw = fp.moe_combine_backward(c(G), O, plan, c(w), dO=torch.zeros_like(O))
    dX = fp.moe_dispatch_backward(dO * c(gain)[:, None], plan)
    # each derivative: at most K d products and sums of four fp32 roundings each, of terms of size below 200
    tol = 1.01 * U * (4 + d + K) * 200 * K
    for t, i in [(0, 0), (3, 5), (6, 11)]:
        e = np.zeros_like(X)
        e[t, i] = 0.5
        assert abs((loss(X + e, w) - loss(X - e, w)) - float(dX[t, i])) < tol
    for t, k in [(0, 0), (2, 1), (6, 2)]:
        e = np.zeros_like(w)
        e[t, k] = 0.5
        assert abs((loss(X, w + e) - loss(X, w - e)) - float(dw[t, k])) < tol


def layer(fp, X, ids, w, E, up, down, wu, wd, plan=None):
    """An expert layer from its router's choices on: every step on the device."""
    plan = fp.moe_sort(ids, E, plan=plan)
    Xq, xs = fp.quantize_rows(X)
    n = ids.numel()
    H = fp.scaled_matmul_grouped(Xq, xs, up, wu, plan.offsets, rows=plan.tokens,
                                 out=torch.zeros((n, up.d_out), dtype=X.dtype, device=X.device))
    Hq, hs = fp.quantize_rows(H)
    O = fp.scaled_matmul_grouped(Hq, hs, down, wd, plan.offsets,  # noqa: E741
                                 out=torch.zeros((n, down.d_out), dtype=X.dtype, device=X.device))
    return fp.moe_combine(O, plan, w), (plan, Xq, xs, H, Hq, hs, O)


@pytest.mark.parametrize("T,K,E,d,dff,dt", [(1, 2, 8, 64, 96, torch.bfloat16), (40, 2, 8, 96, 160, torch.float16), (300, 4, 16, 128, 200, torch.float32)])
def test_expert_layer(fp, T, K, E, d, dff, dt):
    """Sort, quantization, grouped products and combination strung together: each step against 64 bits on what the step
    before it wrote, the whole also as graph replays with other inputs and eager work between them."""
    rng = np.random.default_rng(T)
    W1 = torch.from_numpy(rng.integers(-7, 8, (E, dff, d), dtype=np.int8)).cuda()
    W2 = torch.from_numpy(rng.integers(-7, 8, (E, d, dff), dtype=np.int8)).cuda()
    up, down = fp.pack_experts(W1), fp.pack_experts(W2)
    wu, wd = (torch.from_numpy(rng.uniform(0.01, 0.02, s).astype(np.float32)).cuda() for s in ((E, dff), (E, d)))
    sets = []
    for k in range(3):
        ids = draw_ids(rng, T, K, E, "wild" if k else "skewed")
        w = torch.from_numpy(rng.random((T, K)).astype(np.float32)).cuda()
        X = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda().to(dt)
        sets.append((X, torch.from_numpy(ids).cuda(), w))
    want = []
    for X, ids, w in sets:
        Y, (plan, Xq, xs, H, Hq, hs, O) = layer(fp, X, ids, w, E, up, down, wu, wd)  # noqa: E741
        off, slots, rows = check_plan(plan, ids.cpu().numpy(), E)
        for (q, s, W, ws, y, by_token) in ((Xq, xs, W1, wu, H, True), (Hq, hs, W2, wd, O, False)):
            q64, s64, W64, w64 = (t.cpu().numpy().astype(np.float64) for t in (q, s, W, ws))
            for g in range(E):
                for i in range(off[g], off[g + 1]):
                    r = slots[i] // K if by_token else i
                    ref = (W64[g] @ q64[r]) * s64[r] * w64[g]
                    within(y[i], ref, 3.1 * U * np.abs(ref), dt)
        o64, w64 = O.double().cpu().numpy(), w.double().cpu().numpy()
        terms = np.where((rows >= 0)[:, :, None], w64[:, :, None] * o64[np.maximum(rows, 0)], 0)
        within(Y, terms.sum(1), 1.01 * K * U * np.abs(terms).sum(1), dt)
        want.append(Y)
    X, ids, w = (t.clone() for t in sets[0])
    y = torch.empty_like(X)
    kept = fp.MoePlan(T, K, E)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y.copy_(layer(fp, X, ids, w, E, up, down, wu, wd, plan=kept)[0])
    for k in range(6):
        for a, b in zip((X, ids, w), sets[k % 3]):
            a.copy_(b)
        y.zero_()
        g.replay()
        assert torch.equal(layer(fp, *sets[(k + 1) % 3], E, up, down, wu, wd)[0], want[(k + 1) % 3])
        torch.cuda.synchronize()
        assert torch.equal(y, want[k % 3])


def test_other_stream(fp):
    rng = np.random.default_rng(9)
    ids = torch.from_numpy(draw_ids(rng, 2000, 8, 64, "skewed")).cuda()
    X = torch.from_numpy(rng.standard_normal((2000, 64)).astype(np.float32)).cuda()
    want, plan = fp.moe_dispatch(X, ids, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, plan2 = fp.moe_dispatch(X, ids, 64)
        y = fp.moe_combine(got, plan2)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(y, fp.moe_combine(want, plan))


def test_as_functions_of_autograd(fp):
    """The calls and their gradients as torch's Functions, as a program that trains through them has them: the same
    gradients as the calls by themselves; outside a Function, a tensor that asks for a gradient is refused."""
    T, K, E, d = 50, 3, 7, 72
    rng = np.random.default_rng(4)
    ids = torch.from_numpy(draw_ids(rng, T, K, E, "wild")).cuda()

    class Gather(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X, plan):
            ctx.plan = plan
            return fp.moe_permute(X, plan, out=X.new_zeros((T * K, d)))

        @staticmethod
        def backward(ctx, dXs):
            return fp.moe_dispatch_backward(dXs.contiguous(), ctx.plan), None

    class Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, O, w, plan):  # noqa: E741
            ctx.save_for_backward(O, w)
            ctx.plan = plan
            return fp.moe_combine(O, plan, w)

        @staticmethod
        def backward(ctx, dY):
            O, w = ctx.saved_tensors  # noqa: E741
            return (*fp.moe_combine_backward(dY.contiguous(), O, ctx.plan, w, dO=torch.zeros_like(O)), None)

    plan = fp.moe_sort(ids, E)
    X = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda()
    w = torch.from_numpy(rng.random((T, K)).astype(np.float32)).cuda()
    G = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda()
    Xs = fp.moe_permute(X, plan, out=torch.zeros((T * K, d), device="cuda"))
    dO, dw = fp.moe_combine_backward(G, Xs * 3, plan, w, dO=torch.zeros_like(Xs))
    dX = fp.moe_dispatch_backward(dO * 3, plan)
    x, v = X.clone().requires_grad_(), w.clone().requires_grad_()
    y = Combine.apply(Gather.apply(x, plan) * 3, v, plan)
    gx, gv = torch.autograd.grad(y, (x, v), G)
    assert torch.equal(y, fp.moe_combine(Xs * 3, plan, w)) and torch.equal(gx, dX) and torch.equal(gv, dw)
    for f in (lambda: fp.moe_permute(x, plan), lambda: fp.moe_dispatch(x, ids, E), lambda: fp.moe_combine(Xs, plan, v)):
        with pytest.raises(ValueError, match="backward"):
            f()
    with torch.no_grad():
        assert torch.equal(fp.moe_combine(Xs, plan, v), fp.moe_combine(Xs, plan, w))
        assert torch.equal(fp.moe_dispatch(x, ids, E)[0][:int(plan.offsets[-1])], Xs[:int(plan.offsets[-1])])


def test_gradients_replayed(fp):
    """There and back and both gradients captured with a kept plan, replayed on other choices and values, with the same
    calls on another stream and another plan between the replays: each replay against the calls by themselves."""
    T, K, E, d = 70, 3, 9, 75
    rng = np.random.default_rng(6)

    def step(plan, X, ids, w, G):
        Xs, _ = fp.moe_dispatch(X, ids, E, plan=plan, out=torch.zeros((T * K, d), dtype=X.dtype, device="cuda"))
        Y = fp.moe_combine(Xs, plan, w)
        dO, dw = fp.moe_combine_backward(G, Xs, plan, w, dO=torch.zeros_like(Xs))
        return Xs, Y, dO, dw, fp.moe_dispatch_backward(dO, plan), *fp.quantize_rows(Y)

    def values(kind):
        X, G = (torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda().bfloat16() for _ in range(2))
        return (X, torch.from_numpy(draw_ids(rng, T, K, E, kind)).cuda(),
                torch.from_numpy(rng.random((T, K)).astype(np.float32)).cuda(), G)
    sets = [values(kind) for kind in ("skewed", "wild", "none", "one")]
    want = [step(fp.MoePlan(T, K, E), *s) for s in sets]
    held = [t.clone() for t in sets[0]]
    plan = fp.MoePlan(T, K, E)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(plan, *held)
    side = torch.cuda.Stream()
    for k in range(8):
        for a, b in zip(held, sets[k % 4]):
            a.copy_(b)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            beside = step(fp.MoePlan(T, K, E), *sets[(k + 1) % 4])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[k % 4]):
            assert torch.equal(a, b)
        for a, b in zip(beside, want[(k + 1) % 4]):
            assert torch.equal(a, b)
