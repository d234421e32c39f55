"""The scaled products and the sort by expert refuse bad arguments before any
launch: at the C ABI with their error codes, in the binding with exceptions.
CPU only (the pointers are never read)."""
import ctypes

import pytest
import torch

import zero_knowledge_proof_amd as fp

D = ctypes.c_void_p(256)   # an aligned address that is never dereferenced
ODD = ctypes.c_void_p(257)
F32, F16, BF16 = fp.FP_F32, fp.FP_F16, fp.FP_BF16
EARG, ESHAPE, EWS = 1, 2, 4


def mm(X=D, ldx=64, xs=D, Wp=D, ws=D, bias=None, T=4, d_in=64, d_out=32, dt=BF16, Y=D, ldy=32, Z=None, ldz=32):
    return fp.lib().fp_scaled_matmul(X, ldx, xs, Wp, ws, bias, T, d_in, d_out, dt, Y, ldy, Z, ldz, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EARG), (dict(d_in=-1), EARG), (dict(d_out=-1), EARG), (dict(dt=0), EARG), (dict(dt=5), EARG),
    (dict(X=None), EARG), (dict(xs=None), EARG), (dict(ws=None), EARG), (dict(Y=None), EARG), (dict(Wp=None), EARG),
    (dict(ldx=63), ESHAPE), (dict(ldy=31), ESHAPE), (dict(Z=D, ldz=31), ESHAPE), (dict(d_in=131072, ldx=131072), ESHAPE),
    (dict(Wp=ctypes.c_void_p(264)), EARG), (dict(Y=ODD), EARG), (dict(Y=ctypes.c_void_p(258), dt=F32), EARG),
    (dict(Z=ctypes.c_void_p(258)), EARG), (dict(bias=ODD), EARG),
    (dict(T=1 << 30, d_out=1 << 20, ldy=1 << 20), ESHAPE)])
def test_scaled_matmul(kw, code):
    assert mm(**kw) == code
    assert fp.lib().fp_last_error()


def test_empty_products_are_no_launches():
    assert mm(T=0, X=None, xs=None, Wp=None, ws=None, Y=None) == 0
    assert mm(d_out=0, Wp=None, ws=None, Y=None) == 0
    assert fp.lib().fp_quantize_rows(F32, None, 8, 0, 8, None, 8, None, None) == 0
    assert fp.lib().fp_moe_permute(2, None, 8, 0, 2, 8, None, None, 8, None) == 0
    assert fp.lib().fp_moe_combine(BF16, None, 8, 0, None, None, 0, 2, 8, None, 8, None) == 0


def test_quantize_rows():
    q = lambda dt=BF16, X=D, ldx=8, T=2, c=8, Q=D, ldq=8, s=D: fp.lib().fp_quantize_rows(dt, X, ldx, T, c, Q, ldq, s, None)  # noqa: E731
    assert q(dt=1) == EARG and q(T=-1) == EARG and q(X=None) == EARG and q(Q=None) == EARG and q(s=None) == EARG
    assert q(ldx=7) == ESHAPE and q(ldq=7) == ESHAPE and q(X=ODD) == EARG and q(s=ODD) == EARG


def test_scaled_linear():
    need = fp.lib().fp_scaled_linear_workspace(4, 64)
    assert need >= 4 * 64 + 16 and fp.lib().fp_scaled_linear_workspace(-1, 64) == 0

    def call(dt=BF16, X=D, ldx=64, Wp=D, ws=D, T=4, d_in=64, d_out=32, y=BF16, Y=D, ldy=32, w=D, n=need):
        return fp.lib().fp_scaled_linear(dt, X, ldx, Wp, ws, None, T, d_in, d_out, y, Y, ldy, None, 32, w, n, None)
    assert call(n=need - 1) == EWS and call(w=None) == EWS and call(w=ctypes.c_void_p(128)) == EARG
    assert call(dt=1) == EARG and call(y=1) == EARG and call(X=None) == EARG and call(Wp=None) == EARG
    assert call(ldx=63) == ESHAPE and call(ldy=31) == ESHAPE
    assert call(T=0, X=None, w=None, n=0) == 0


def test_scaled_matmul_grouped():
    W = (ctypes.c_void_p * 300)(*([256] * 300))

    def call(x_rows=4, rows=D, n=8, W=W, lds=32, off=D, G=3, T=None, Z=None, d_out=32, ldy=32):
        return fp.lib().fp_scaled_matmul_grouped(D, 64, D, x_rows, rows, n, W, D, None, lds, off, G, 64, d_out, BF16, D,
                                                 ldy, Z, 32, None)
    assert call(G=0) == EARG and call(G=257) == EARG and call(off=None) == EARG and call(W=None) == EARG
    assert call(rows=None) == ESHAPE  # X has fewer rows than the output
    assert call(x_rows=-1) == ESHAPE and call(lds=31) == ESHAPE and call(ldy=31) == ESHAPE and call(n=-1) == EARG
    assert call(W=(ctypes.c_void_p * 3)(256, None, 256)) == EARG and b"group 1" in fp.lib().fp_last_error()
    assert call(W=(ctypes.c_void_p * 3)(256, 256, 264)) == EARG and b"group 2" in fp.lib().fp_last_error()
    assert call(n=0) == 0


def test_moe_sort():
    L = fp.lib()
    assert L.fp_moe_sort_workspace(1, 8, 128) == 0           # one workgroup needs none
    need = L.fp_moe_sort_workspace(16384, 8, 128)
    assert need > 0

    def call(ids=D, b=4, T=16384, K=8, E=128, o=D, s=D, t=D, r=D, w=D, n=need):
        return L.fp_moe_sort(ids, b, T, K, E, o, s, t, r, w, n, None)
    assert call(n=need - 4) == EWS and call(w=None) == EWS and call(w=ODD) == EARG
    assert call(E=0) == EARG and call(E=1025) == EARG and call(K=0) == EARG and call(T=-1) == EARG and call(b=2) == EARG
    assert call(T=1 << 30, K=2) == ESHAPE
    for k in ("ids", "o", "s", "t", "r"):
        assert call(**{k: None}) == EARG
    assert call(ids=ctypes.c_void_p(260), b=8) == EARG


def test_moe_rows():
    L = fp.lib()
    per = lambda b=2, X=D, ldx=8, T=2, K=2, d=8, r=D, Xs=D, lds=8: L.fp_moe_permute(b, X, ldx, T, K, d, r, Xs, lds, None)  # noqa: E731
    assert per(b=3) == EARG and per(X=None) == EARG and per(r=None) == EARG and per(Xs=None) == EARG and per(X=ODD) == EARG
    assert per(ldx=7) == ESHAPE and per(lds=7) == ESHAPE and per(T=1 << 30) == ESHAPE and per(d=-1) == EARG
    com = lambda dt=BF16, O=D, ldo=8, n=4, r=D, T=2, K=2, d=8, Y=D, ldy=8: L.fp_moe_combine(dt, O, ldo, n, r, None, T, K, d, Y, ldy, None)  # noqa: E731,E741
    assert com(dt=0) == EARG and com(O=None) == EARG and com(r=None) == EARG and com(Y=None) == EARG and com(n=-1) == EARG
    assert com(ldo=7) == ESHAPE and com(ldy=7) == ESHAPE and com(Y=ODD) == EARG

    def bwd(dt=BF16, dY=D, ldd=8, O=D, ldo=8, n=4, r=D, w=D, T=2, K=2, d=8, dO=D, lddo=8, dw=D):  # noqa: E741
        return L.fp_moe_combine_backward(dt, dY, ldd, O, ldo, n, r, w, T, K, d, dO, lddo, dw, None)
    assert bwd(dt=1) == EARG and bwd(ldd=7) == ESHAPE and bwd(ldo=7) == ESHAPE and bwd(lddo=7) == ESHAPE
    for k in ("dY", "O", "r", "w", "dO", "dw"):
        assert bwd(**{k: None}) == EARG
    assert bwd(dO=ODD) == EARG and bwd(n=-1) == EARG


def test_moe_rows_of_2_31_bytes():
    L, d = fp.lib(), 1 << 30
    assert L.fp_moe_permute(2, D, d, 2, 2, d, D, D, d, None) == ESHAPE
    assert L.fp_moe_combine(BF16, D, d, 4, D, None, 2, 2, d, D, d, None) == ESHAPE
    assert L.fp_moe_combine_backward(F32, D, d, D, d, 4, D, D, 2, 2, d, D, d, D, None) == ESHAPE
    ok = (1 << 31) - 16  # the widest row
    assert L.fp_moe_permute(1, None, ok, 0, 2, ok, None, None, ok, None) == 0
    assert L.fp_moe_permute(1, None, ok + 1, 0, 2, ok + 1, None, None, ok + 1, None) == ESHAPE


def test_binding():
    """Shapes, types and strides are checked before anything reaches the device."""
    Wp = fp.PackedWeights(torch.zeros(64 * 64, dtype=torch.int8), 40, 64)
    X, xs, ws = torch.zeros(3, 64, dtype=torch.int8), torch.ones(3), torch.ones(40)
    for args, kw in [((X.float(), xs, Wp, ws), {}), ((X[:, :63], xs, Wp, ws), {}), ((X, xs[:2], Wp, ws), {}),
                     ((X, xs.double(), Wp, ws), {}), ((X, xs, Wp, ws[:39]), {}), ((X.t().contiguous().t(), xs, Wp, ws), {}),
                     ((X, xs, Wp, ws), dict(bias=torch.ones(41))), ((X, xs, Wp, ws), dict(out=torch.zeros(3, 41))),
                     ((X, xs, Wp, ws), dict(out=torch.zeros(3, 40, dtype=torch.int32))), ((X, xs, Wp, ws), dict(dtype=torch.int8)),
                     ((X, xs, Wp, ws), dict(Z=torch.zeros(3, 40))), ((X, xs, Wp, ws), dict(out=torch.zeros(1, 40).expand(3, 40)))]:
        with pytest.raises(ValueError):
            fp.scaled_matmul(*args, **kw)
    with pytest.raises(ValueError):
        fp.scaled_linear(X, Wp, ws)               # int8 activations have scales already
    with pytest.raises(ValueError):
        fp.scaled_linear(torch.zeros(3, 63), Wp, ws)
    with pytest.raises(ValueError):
        fp.quantize_rows(X)
    with pytest.raises(ValueError):
        fp.quantize_rows(torch.zeros(3, 64), out=torch.zeros(3, 63, dtype=torch.int8))
    with pytest.raises(ValueError):
        fp.PackedExperts([])
    with pytest.raises(ValueError):
        fp.PackedExperts([Wp, fp.PackedWeights(Wp.data, 39, 64)])
    We = fp.PackedExperts([Wp, Wp])
    off, ws2 = torch.zeros(3, dtype=torch.int32), torch.ones(2, 40)
    for args, kw in [((X, xs, We, ws2, off.long()), {}), ((X, xs, We, ws2, off[:2]), {}), ((X, xs, We, ws, off), {}),
                     ((X, xs, We, ws2, off), dict(rows=torch.zeros(4))), ((X, xs, We, ws2, off), dict(bias=torch.ones(2, 41))),
                     ((X, xs, We, ws2, off), dict(out=torch.zeros(4, 40)))]:
        with pytest.raises(ValueError):
            fp.scaled_matmul_grouped(*args, **kw)
    # a last row whose 16-byte chunk leaves its storage
    s = torch.zeros(2 * 32 + 20, dtype=torch.int8)
    if s.data_ptr() % 16 == 0:
        with pytest.raises(ValueError, match="storage"):
            fp._whole_rows(torch.as_strided(s, (3, 20), (32, 1)), 32)
        assert fp._whole_rows(torch.as_strided(s, (1, 20), (32, 1), 64), 32) == 20  # one row: to its end only
        assert fp._whole_rows(torch.as_strided(s, (2, 20), (32, 1)), 32) == 32
    assert fp._whole_rows(torch.zeros(3, 32, dtype=torch.int8)[:, :20], 32) == 32


def test_binding_moe():
    plan = fp.MoePlan(3, 2, 4, device="cpu")
    assert plan.offsets.numel() == 5 and plan.rows.shape == (3, 2) and plan.slots.numel() == plan.tokens.numel() == 6
    ids = torch.zeros(3, 2, dtype=torch.int32)
    for bad in (ids.float(), ids.reshape(-1), torch.zeros(2, 3, dtype=torch.int32).t()):
        with pytest.raises(ValueError):
            fp.moe_sort(bad, 4)
    with pytest.raises(ValueError, match="plan"):
        fp.moe_sort(ids, 5, plan=plan)
    with pytest.raises(ValueError):
        fp.MoePlan(3, 0, 4, device="cpu")
    X = torch.zeros(3, 8)
    for x, kw in [(X.double(), {}), (X[:2], {}), (X, dict(out=torch.zeros(5, 8))), (X, dict(out=torch.zeros(6, 8).half()))]:
        with pytest.raises(ValueError):
            fp.moe_permute(x, plan, **kw)
    O, w = torch.zeros(6, 8), torch.zeros(3, 2)  # noqa: E741
    for o, ww, kw in [(O[:5], w, {}), (O.int(), w, {}), (O, w.half(), {}), (O, w[:2], {}), (O, w, dict(out=torch.zeros(3, 7)))]:
        with pytest.raises(ValueError):
            fp.moe_combine(o, plan, ww, **kw)
    with pytest.raises(ValueError):
        fp.moe_combine_backward(X.half(), O, plan, w)
    with pytest.raises(ValueError):
        fp.moe_combine_backward(X, O, plan, w, dw=torch.zeros(2, 3))


def test_grouped_without_tokens():
    """X of no rows, as a batch of padding rows alone has it: nothing to do, and no pointers to X and its scales needed."""
    W = (ctypes.c_void_p * 3)(256, 256, 256)

    def call(X=None, xs=None, x_rows=0, ws=D, Y=D):
        return fp.lib().fp_scaled_matmul_grouped(X, 64, xs, x_rows, D, 8, W, ws, None, 32, D, 3, 64, 32, BF16, Y, 32, None, 32, None)
    assert call() == 0
    assert call(ws=None) == EARG and call(Y=None) == EARG
    assert call(X=D, x_rows=4) == EARG and call(xs=D, x_rows=4) == EARG


def test_gradients_are_not_lost_silently():
    """The calls record no graph, so those that have gradients refuse tensors that ask for one."""
    plan = fp.MoePlan(3, 2, 4, device="cpu")
    ids = torch.zeros(3, 2, dtype=torch.int32)
    X, O, w = torch.zeros(3, 8), torch.zeros(6, 8), torch.zeros(3, 2)  # noqa: E741
    g = lambda t: t.clone().requires_grad_()  # noqa: E731
    for f in (lambda: fp.moe_permute(g(X), plan), lambda: fp.moe_dispatch(g(X), ids, 4, plan=plan),
              lambda: fp.moe_combine(g(O), plan, w), lambda: fp.moe_combine(O, plan, g(w)), lambda: fp.moe_combine(g(O), plan),
              lambda: fp.moe_combine(O, plan, torch.softmax(g(w), 1))):
        with pytest.raises(ValueError, match="backward"):
            f()
        with torch.no_grad(), pytest.raises(Exception) as e:  # on to the next check: these are no device tensors
            f()
        assert "backward" not in str(e.value)


@pytest.mark.parametrize("T", [1, 9, 300, 2 ** 31 - 1])
@pytest.mark.parametrize("d_out", [2 ** 31 - 1, 2 ** 31 - 33, 2 ** 31 - 200])
@pytest.mark.parametrize("ldx", [64, 65])
def test_sizes_next_to_32_bits(T, d_out, ldx):
    """Outputs whose number leaves 32 bits when it is rounded up to tiles."""
    assert mm(T=T, d_out=d_out, ldx=ldx, ldy=d_out, ldz=d_out) == ESHAPE
    W = (ctypes.c_void_p * 3)(256, 256, 256)
    assert fp.lib().fp_scaled_matmul_grouped(D, ldx, D, T, D, T, W, D, None, d_out, D, 3, 64, d_out, BF16, D, d_out, None, d_out,
                                             None) == ESHAPE
