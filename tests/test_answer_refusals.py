"""The norm, the mixture layer for a few tokens and the log probabilities refuse
bad arguments before any launch: at the C ABI with their error codes, in the
binding with exceptions. CPU only (the pointers are never read)."""
import ctypes

import pytest
import torch

import zero_knowledge_proof_amd as fp

D = ctypes.c_void_p(256)   # an aligned address that is never dereferenced
ODD = ctypes.c_void_p(257)
TWO = ctypes.c_void_p(258)
I8, F32, F16, BF16 = fp.FP_I8, fp.FP_F32, fp.FP_F16, fp.FP_BF16
EARG, ESHAPE, EWS = 1, 2, 4
NAN, INF = float("nan"), float("inf")


def norm(dt=BF16, X=D, ldx=64, R=D, ldr=64, wdt=BF16, w=D, eps=1e-5, T=4, d=64, H=D, ldh=64, Y=D, ldy=64, Q=D, ldq=64, s=D):
    return fp.lib().fp_rms_norm(dt, X, ldx, R, ldr, wdt, w, eps, T, d, H, ldh, Y, ldy, Q, ldq, s, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EARG), (dict(dt=1), EARG), (dict(dt=5), EARG), (dict(T=-1), EARG), (dict(d=-1), EARG), (dict(wdt=F16), EARG), (dict(wdt=I8), EARG),
    (dict(dt=F32, wdt=BF16), EARG), (dict(eps=0.0), EARG), (dict(eps=-1.0), EARG), (dict(eps=NAN), EARG), (dict(eps=INF), EARG), (dict(eps=1.5), EARG),
    (dict(eps=1e-31), EARG), (dict(X=None), EARG), (dict(Y=None, Q=None, s=None), EARG), (dict(s=None), EARG), (dict(Q=None), EARG),
    (dict(X=ODD), EARG), (dict(R=ODD), EARG), (dict(w=ODD), EARG), (dict(w=TWO, wdt=F32), EARG), (dict(H=ODD), EARG), (dict(Y=ODD), EARG), (dict(s=TWO), EARG),
    (dict(dt=F32, wdt=F32, X=TWO), EARG), (dict(ldx=63), ESHAPE), (dict(ldr=63), ESHAPE), (dict(ldh=63), ESHAPE), (dict(ldy=63), ESHAPE), (dict(ldq=63), ESHAPE),
    (dict(d=131072, ldx=131072, ldr=131072, ldh=131072, ldy=131072, ldq=131072), ESHAPE)])
def test_norm(kw, code):
    assert norm(**kw) == code
    assert b"fp_rms_norm" in fp.lib().fp_last_error()


def norm_bwd(dt=BF16, dY=D, lddy=64, H=D, ldh=64, wdt=BF16, w=D, eps=1e-5, dH=D, lddh=64, T=4, d=64, dX=D, lddx=64, dw=D, ws=D, n=1 << 20):
    return fp.lib().fp_rms_norm_backward(dt, dY, lddy, H, ldh, wdt, w, eps, dH, lddh, T, d, dX, lddx, dw, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EARG), (dict(T=-1), EARG), (dict(d=-1), EARG), (dict(wdt=F16), EARG), (dict(eps=0.0), EARG), (dict(dY=None), EARG), (dict(H=None), EARG),
    (dict(dX=None), EARG), (dict(dY=ODD), EARG), (dict(H=ODD), EARG), (dict(dH=ODD), EARG), (dict(dX=ODD), EARG), (dict(dw=TWO), EARG), (dict(ws=TWO), EARG),
    (dict(lddy=63), ESHAPE), (dict(ldh=63), ESHAPE), (dict(lddh=63), ESHAPE), (dict(lddx=63), ESHAPE), (dict(ws=None), EWS), (dict(n=4 * 64 * 4 // 4 - 1), EWS),
    (dict(d=16385, lddy=16385, ldh=16385, lddh=16385, lddx=16385), ESHAPE)])
def test_norm_backward(kw, code):
    assert norm_bwd(**kw) == code
    assert b"fp_rms_norm_backward" in fp.lib().fp_last_error()


def test_norm_workspace():
    L = fp.lib()
    assert L.fp_rms_norm_backward_workspace(4, 64) >= 64 * 4
    assert L.fp_rms_norm_backward_workspace(-1, 64) == L.fp_rms_norm_backward_workspace(4, -1) == L.fp_rms_norm_backward_workspace(4, 16385) == 0


def layer(x=BF16, X=D, ldx=64, xs=None, ids=D, b=4, w=D, T=4, K=2, E=8, g=D, gs=D, ldg=96, u=D, us=D, ldu=96, dn=D, ds=D, ldd=64, d=64, ff=96, y=BF16, Y=D, ldy=64,
          ws=D, n=1 << 30):
    return fp.lib().fp_moe_layer(x, X, ldx, xs, ids, b, w, T, K, E, g, gs, ldg, u, us, ldu, dn, ds, ldd, d, ff, y, Y, ldy, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EARG), (dict(K=0), EARG), (dict(d=-1), EARG), (dict(ff=-1), EARG), (dict(E=0), EARG), (dict(E=1025), EARG), (dict(x=1), EARG), (dict(x=5), EARG),
    (dict(y=0), EARG), (dict(y=5), EARG), (dict(b=2), EARG), (dict(x=I8), EARG), (dict(g=None), EARG), (dict(gs=None), EARG),
    (dict(X=None), EARG), (dict(ids=None), EARG), (dict(w=None), EARG), (dict(u=None), EARG), (dict(us=None), EARG), (dict(dn=None), EARG), (dict(ds=None), EARG),
    (dict(Y=None), EARG), (dict(X=ODD), EARG), (dict(Y=ODD), EARG), (dict(ids=TWO), EARG), (dict(ids=ctypes.c_void_p(260), b=8), EARG), (dict(w=TWO), EARG),
    (dict(xs=TWO), EARG), (dict(gs=TWO), EARG), (dict(us=TWO), EARG), (dict(ds=TWO), EARG), (dict(g=ctypes.c_void_p(260)), EARG), (dict(u=ctypes.c_void_p(260)), EARG),
    (dict(dn=ctypes.c_void_p(260)), EARG), (dict(ws=ctypes.c_void_p(128)), EARG), (dict(ws=None), EWS), (dict(n=4096), EWS),
    (dict(T=513), ESHAPE), (dict(T=1 << 30, K=1 << 30), ESHAPE), (dict(d=0), ESHAPE), (dict(ff=0), ESHAPE), (dict(d=131072, ldx=131072, ldy=131072, ldd=131072), ESHAPE),
    (dict(ff=131072, ldu=131072, ldg=131072), ESHAPE),
    (dict(T=1024, K=1, E=1024, d=131071, ff=131071, ldx=131071, ldy=131071, ldd=131071, ldu=131071, ldg=131071), ESHAPE), (dict(ldx=63), ESHAPE), (dict(ldy=63), ESHAPE), (dict(ldu=95), ESHAPE), (dict(ldg=95), ESHAPE), (dict(ldd=63), ESHAPE)])
def test_moe_layer(kw, code):
    assert layer(**kw) == code
    assert b"fp_moe_layer" in fp.lib().fp_last_error()


def test_moe_layer_workspace():
    L = fp.lib()
    need = L.fp_moe_layer_workspace(4, 2, 64, 96)
    assert need >= 8 * (64 + 96) * 4 and layer(n=need - 1) == EWS
    assert L.fp_moe_layer_workspace(513, 2, 64, 96) == L.fp_moe_layer_workspace(4, 0, 64, 96) == L.fp_moe_layer_workspace(4, 2, 0, 96) == 0
    assert layer(T=0, X=None, ids=None, w=None, u=None, us=None, dn=None, ds=None, Y=None, ws=None, n=0) == 0


def logp(dt=BF16, X=D, ldx=500, T=4, V=500, t=D, b=4, temp=1.0, top=5, lp=D, h=D, m=D, ls=D, tl=D, ti=D, ws=D, n=1 << 20):
    return fp.lib().fp_token_logprobs(dt, X, ldx, T, V, t, b, temp, top, lp, h, m, ls, tl, ti, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EARG), (dict(dt=5), EARG), (dict(T=-1), EARG), (dict(V=-1), EARG), (dict(b=2), EARG), (dict(temp=0.0), EARG), (dict(temp=-1.0), EARG),
    (dict(temp=NAN), EARG), (dict(temp=INF), EARG), (dict(temp=2.0 ** -21), EARG), (dict(temp=2.0 ** 21), EARG), (dict(top=-1), EARG), (dict(top=33), EARG),
    (dict(X=None), EARG), (dict(t=None), EARG), (dict(lp=None), EARG), (dict(h=None), EARG), (dict(m=None), EARG), (dict(ls=None), EARG), (dict(tl=None), EARG),
    (dict(ti=None), EARG), (dict(X=ODD), EARG), (dict(t=TWO), EARG), (dict(t=ctypes.c_void_p(260), b=8), EARG), (dict(lp=TWO), EARG), (dict(ti=TWO), EARG),
    (dict(ldx=499), ESHAPE), (dict(V=0x7FFFFF01, ldx=0x7FFFFF01), ESHAPE),
    (dict(V=100000, ldx=100000, ws=None), EWS), (dict(V=100000, ldx=100000, n=64), EWS), (dict(V=100000, ldx=100000, ws=ctypes.c_void_p(260)), EARG)])
def test_logprobs(kw, code):
    assert logp(**kw) == code
    assert b"fp_token_logprobs" in fp.lib().fp_last_error()


def test_logprobs_workspace():
    L = fp.lib()
    need = L.fp_token_logprobs_workspace(BF16, 4, 100000, 5)
    assert need > 0 and logp(V=100000, ldx=100000, n=need - 1) == EWS
    assert L.fp_token_logprobs_workspace(BF16, 5000, 100000, 5) == 0  # a workgroup to a row
    assert L.fp_token_logprobs_workspace(BF16, 4, 100000, 33) == L.fp_token_logprobs_workspace(0, 4, 100000, 5) == L.fp_token_logprobs_workspace(BF16, -4, 9, 5) == 0
    assert logp(T=0, X=None, t=None, lp=None, h=None, m=None, ls=None, tl=None, ti=None, ws=None, n=0) == 0


def test_logprobs_backward():
    def call(dt=BF16, X=D, ldx=500, T=4, V=500, t=D, b=4, temp=1.0, dl=D, dh=D, m=D, ls=D, h=D, dX=D, ldd=500):
        return fp.lib().fp_token_logprobs_backward(dt, X, ldx, T, V, t, b, temp, dl, dh, m, ls, h, dX, ldd, None)
    for kw in (dict(dt=0), dict(T=-1), dict(V=-1), dict(b=3), dict(temp=0.0), dict(X=None), dict(t=None), dict(m=None), dict(ls=None), dict(h=None), dict(dX=None),
               dict(X=ODD), dict(dX=ODD), dict(dl=TWO), dict(dh=TWO), dict(m=TWO), dict(t=TWO)):
        assert call(**kw) == EARG, kw
    assert call(ldx=499) == ESHAPE and call(ldd=499) == ESHAPE
    assert call(T=0, X=None, t=None, m=None, ls=None, h=None, dX=None) == 0 and call(V=0, X=None, m=None, ls=None, h=None, dX=None) == 0


def refused(f, *args, match=None, **kw):
    with pytest.raises(ValueError, match=match):
        f(*args, **kw)


def test_binding_norm():
    X, w = torch.zeros(3, 64), torch.ones(64)
    for f in (fp.rms_norm, fp.rms_norm_quantize):
        for a, kw in [((X[0], w), {}), ((X.double(), w), {}), ((X.to(torch.int8), w), {}), ((X, w[:63]), {}), ((X, w.half()), {}), ((X.half(), w.bfloat16()), {}),
                      ((X, w[None]), {}), ((X, torch.ones(128)[::2]), {}), ((X.t().contiguous().t(), w), {}), ((X[:1].expand(3, 64), w), {}),
                      ((X, w), dict(residual=X[:2])), ((X, w), dict(residual=X.half())), ((X, w), dict(residual_out=X)),
                      ((X, w), dict(residual=X, residual_out=X[:, :63])), ((X, w), dict(residual=X, residual_out=X.half()))]:
            refused(f, *a, **kw)
    refused(fp.rms_norm, X, w, out=torch.zeros(3, 63))
    refused(fp.rms_norm, X, w, out=X.half())
    refused(fp.rms_norm, X, w, out=torch.zeros(1, 64).expand(3, 64))
    for kw in (dict(out=X), dict(out=torch.zeros(3, 63, dtype=torch.int8)), dict(scale=torch.zeros(2)), dict(scale=torch.zeros(3).half()), dict(Y=X.half()), dict(Y=X[:2])):
        refused(fp.rms_norm_quantize, X, w, **kw)
    for a, kw in [((X[:2], X, w), {}), ((X.half(), X, w), {}), ((X, X, w.half()), {}), ((X, X, w), dict(dH=X[:2])), ((X, X, w), dict(dw=torch.zeros(63))),
                  ((X, X, w), dict(dw=torch.zeros(64).half())), ((X, X, None), dict(dw=torch.zeros(64))), ((X, X, w), dict(out=X.half()))]:
        refused(fp.rms_norm_backward, *a, **kw)


def test_binding_moe_layer():
    def pack(E, o, i):
        return fp.PackedExperts([fp.PackedWeights(torch.zeros(64 * 64, dtype=torch.int8), o, i) for _ in range(E)])
    up, down = pack(4, 40, 64), pack(4, 64, 40)
    us, ds = torch.ones(4, 40), torch.ones(4, 64)
    X, ids, w = torch.zeros(3, 64), torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, 2)
    ok = dict(X=X, ids=ids, weights=w, up=up, up_scale=us, down=down, down_scale=ds)
    for kw in (dict(X=X[0]), dict(X=X.double()), dict(X=X[:, :63]), dict(X=X.to(torch.int8)), dict(x_scale=torch.ones(3)),
               dict(X=X.to(torch.int8), x_scale=torch.ones(2)), dict(X=X.to(torch.int8), x_scale=torch.ones(3).double()), dict(X=X.t().contiguous().t()),
               dict(ids=ids[:2]), dict(ids=ids.float()), dict(ids=ids[0]), dict(ids=torch.zeros(2, 3, dtype=torch.int32).t()), dict(weights=w.half()), dict(weights=w[:2]),
               dict(up=pack(4, 40, 63)), dict(down=pack(4, 63, 40)), dict(down=pack(4, 64, 41)), dict(down=pack(3, 64, 40)), dict(up_scale=us[:, :39]), dict(up_scale=us[:3]),
               dict(up_scale=us.half()), dict(down_scale=ds[:3]), dict(gate=up), dict(gate_scale=us), dict(gate=pack(3, 40, 64), gate_scale=us),
               dict(gate=pack(4, 41, 64), gate_scale=us), dict(gate=up, gate_scale=us[:, 1:]), dict(out=torch.zeros(3, 63)), dict(out=torch.zeros(3, 64, dtype=torch.int8)),
               dict(dtype=torch.int8)):
        refused(fp.moe_layer, **dict(ok, **kw))
    for kw in (dict(X=X.clone().requires_grad_()), dict(weights=w.clone().requires_grad_()), dict(up_scale=us.clone().requires_grad_()),
               dict(down_scale=ds.clone().requires_grad_()), dict(gate=up, gate_scale=us.clone().requires_grad_())):
        refused(fp.moe_layer, match="gradient", **dict(ok, **kw))
    if not torch.cuda.is_available():
        with pytest.raises(Exception):  # tensors that are on no device
            fp.moe_layer(**ok)


def test_binding_logprobs():
    X, t = torch.zeros(3, 50), torch.zeros(3, dtype=torch.int64)
    lp = fp.TokenLogprobs(3, 4, device="cpu")
    assert lp.logprob.shape == lp.entropy.shape == (3,) and lp.top_ids.shape == lp.top_logprobs.shape == (3, 4) and lp.top_ids.dtype == torch.int32
    ends = [(v.data_ptr(), v.data_ptr() + 4 * v.numel()) for v in (lp.logprob, lp.entropy, lp.max, lp.logsum, lp.top_logprobs, lp.top_ids)]
    assert all(a[1] == b[0] for a, b in zip(ends, ends[1:])) and ends[-1][1] == lp.buf.data_ptr() + 4 * lp.buf.numel()
    refused(fp.TokenLogprobs, -1, 2, device="cpu")
    refused(fp.TokenLogprobs, 1, -2, device="cpu")
    for a, kw in [((X[0], t), {}), ((X.double(), t), {}), ((X, t[:2]), {}), ((X, t.float()), {}), ((X, t[:, None]), {}), ((X.t().contiguous().t(), t), {}),
                  ((X, torch.zeros(6, dtype=torch.int64)[::2]), {}), ((X, t), dict(top=3, out=lp)), ((X[:2], t[:2]), dict(top=4, out=lp))]:
        refused(fp.token_logprobs, *a, **kw)
    d = torch.zeros(3)
    for a, kw in [((d.half(), d, X, t, lp), {}), ((d, d[:2], X, t, lp), {}), ((d, d, X[:2], t[:2], lp), {}), ((d, d, X, t[:2], lp), {}),
                  ((d, d, X, t, lp), dict(out=X.half())), ((d, d, X, t, lp), dict(out=X[:, :49])), ((d[:2], d[:2], X[:2], t[:2], lp), {})]:
        refused(fp.token_logprobs_backward, *a, **kw)


def test_gradients_are_not_lost_silently():
    X, w, t = torch.zeros(3, 8), torch.ones(8), torch.zeros(3, dtype=torch.int64)
    g = lambda v: v.clone().requires_grad_()  # noqa: E731
    for f in (lambda: fp.rms_norm(g(X), w), lambda: fp.rms_norm(X, g(w)), lambda: fp.rms_norm(X, w, residual=g(X)), lambda: fp.rms_norm_quantize(g(X), w),
              lambda: fp.token_logprobs(g(X), t)):
        with pytest.raises(ValueError, match="backward"):
            f()
        with torch.no_grad(), pytest.raises(Exception) as e:  # on to the next check: these are no device tensors
            f()
        assert "backward" not in str(e.value)


A, B = (ctypes.c_void_p(256 * i) for i in (2, 3))  # other addresses that are never dereferenced


@pytest.mark.parametrize("call,kw", [
    (norm, dict(Y=A, H=B, X=B, ldh=65)), (norm, dict(Y=A, H=B, R=B, ldh=65)), (norm, dict(Y=A, H=B, X=A, ldy=72)), (norm, dict(Y=A, H=None, R=A, ldr=72)),
    (norm_bwd, dict(dX=A, dY=A, lddx=65)), (norm_bwd, dict(dX=A, H=A, lddx=65)), (norm_bwd, dict(dX=A, dH=A, lddh=65)),
    (norm_bwd, dict(dX=A, dY=A, H=B, dH=None, lddy=72))])
def test_in_place_needs_the_same_rows(call, kw):
    """An output at an input's address has its rows where the input has its own: else a row is overwritten before it is read."""
    assert call(**kw) == EARG
    assert b"leading dimension" in fp.lib().fp_last_error()


def test_logits_in_place_need_the_same_rows():
    assert fp.lib().fp_token_logprobs_backward(BF16, A, 500, 4, 500, D, 4, 1.0, D, D, D, D, D, A, 512, None) == EARG
    assert b"leading dimension" in fp.lib().fp_last_error()


def test_stream_and_norm_need_places_of_their_own():
    """H may be X and Y may be X, but not both: one of them would be lost."""
    assert norm(X=A, H=A, Y=A) == EARG and norm(R=A, H=A, Y=A) == EARG and norm(H=A, Y=A) == EARG
    assert b"same place" in fp.lib().fp_last_error()
