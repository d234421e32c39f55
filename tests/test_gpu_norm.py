"""The root-mean-square norm, its int8 form and its gradients on the GPU against
64-bit references.

Tolerances. u = 2^-24. A sum of squares adds at most c values in a row in a
thread (c <= 80 for rows of up to 20480: 16 to 256 threads take a row), then
log2 and 3 more: relative error at most 92 u, with h's own rounding 94 u; its
root has half of that, and mean, eps, root and quotient add one rounding each, so
s is within 52 u, and y = (h s) w within 56 u, before the output's rounding of
half a step, eps / 2. A scale of int8 rows adds one division; a value is then
within (1/2 + 2^-14) steps of y. Gradients: the sums of g h have at most 92
roundings relative to sum |g h|, so dx is within 64 u s |g| + 160 u s |n| mean |g
n|, and dw's sum over T rows (at most ceil(T / 256) + 48 + 16 + 16 in a row)
within (56 + that) u sum |dy n|."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def half_step(want, dtype):
    return torch.finfo(dtype).eps / 2 * want.abs() + TINY[dtype]


def within(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:3].tolist(), got[bad][:3], want[bad][:3])


def rows(g, T, d, dtype, ld=None, offset=0):
    """Rows of magnitudes of their own, as a view with this row stride and offset."""
    ld = ld or d
    x = torch.randn((T, max(ld, 1)), generator=g, device="cuda") * torch.exp(torch.randn((T, 1), generator=g, device="cuda"))
    buf = torch.zeros(T * ld + offset + 16, device="cuda", dtype=dtype)
    v = torch.as_strided(buf, (T, d), (ld, 1), offset)
    v.copy_(x[:, :d])
    return v


def exact(X, w, eps, R=None):
    h = X.double() if R is None else X.double() + R.double()
    s = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h, h * s * (1 if w is None else w.double())


# rows of one value to many times the registers' capacity, next to every change of the threads to a row
SHAPES = [(1, 1), (3, 2), (1, 5120), (2, 7), (5, 8), (7, 63), (300, 64), (33, 127), (20, 128), (1000, 128), (9, 255), (6, 256), (11, 257),
          (5, 511), (4, 512), (5, 513), (130, 1000), (9, 1023), (3, 1025), (70, 1111), (5, 2047), (6, 2049), (40, 4096), (3, 4097),
          (2, 8191), (3, 8192), (3, 8200), (2, 16384), (2, 20000), (4100, 40)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_norm(fp, T, d, dtype):
    g = torch.Generator("cuda").manual_seed(T * 31 + d)
    X, R = rows(g, T, d, dtype), rows(g, T, d, dtype)
    for wt in {dtype, torch.float32}:
        w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(wt)
        _, want = exact(X, w, 1e-5)
        within(fp.rms_norm(X, w, eps=1e-5), want, 56 * U * want.abs() + half_step(want, dtype))
        h, want = exact(X, w, 1e-5, R)
        Y, H = fp.rms_norm(X, w, eps=1e-5, residual=R)
        within(H, h, U * h.abs() + half_step(h, dtype))
        within(Y, want, 56 * U * want.abs() + half_step(want, dtype))
    h, want = exact(X, None, 0.5, R)
    within(fp.rms_norm(X, None, eps=0.5, residual=R)[0], want, 56 * U * want.abs() + half_step(want, dtype))


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_int8_rows(fp, T, d, dtype):
    g = torch.Generator("cuda").manual_seed(T * 37 + d)
    X, R = rows(g, T, d, dtype), rows(g, T, d, dtype)
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    Y = torch.empty_like(X)
    q, scale, H = fp.rms_norm_quantize(X, w, residual=R, Y=Y)
    h, want = exact(X, w, 1e-5, R)
    top = want.abs().amax(1)
    within(scale, top / 127, 58 * U * top / 127 + 1e-45)
    step = scale.double()[:, None]
    within(q.double() * step, want, (0.5 + 2.0 ** -14) * step + 57 * U * want.abs())
    assert bool((q.double().abs().amax(1) == 127).all())
    # the float rows beside them, and the stream, are those of the float call
    y, hh = fp.rms_norm(X, w, residual=R)
    assert torch.equal(y, Y) and torch.equal(hh, H)
    if dtype == torch.float32:  # the same rows, rounded to int8 by the call for float rows
        q2, s2 = fp.quantize_rows(Y)
        assert torch.equal(q, q2) and torch.equal(scale, s2)
    q3, s3 = fp.rms_norm_quantize(X, w)
    q4, s4 = fp.rms_norm_quantize(X, w, residual=torch.zeros_like(X))[:2]
    assert torch.equal(q3, q4) and torch.equal(s3, s4)


@pytest.mark.parametrize("d", [60, 130, 1111, 2600, 9001])
@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (8, 8), (5, 7)])
@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_guards(fp, d, pad, offset, dtype):
    """Rows and outputs with strides and addresses of their own: nothing beside the outputs is written."""
    g = torch.Generator("cuda").manual_seed(d + pad)
    T = 5
    X, R = rows(g, T, d, dtype, d + pad, offset), rows(g, T, d, dtype, d + pad + 1, offset + 2)
    w = torch.randn(d, generator=g, device="cuda")
    q0, s0, H0 = fp.rms_norm_quantize(X.contiguous(), w, residual=R.contiguous())
    Y0 = fp.rms_norm(X.contiguous(), w, residual=R.contiguous())[0]

    def guarded(dt):
        big = torch.full((T + 2, d + 2 * pad + 3), 5, dtype=dt, device="cuda")
        return big, big[1:T + 1, pad + 1:pad + 1 + d]
    (bh, H), (by, Y), (bq, q) = guarded(dtype), guarded(dtype), guarded(torch.int8)
    s = torch.empty(T, device="cuda")
    fp.rms_norm_quantize(X, w, residual=R, residual_out=H, out=q, scale=s, Y=Y)
    assert torch.equal(H, H0) and torch.equal(Y, Y0) and torch.equal(q, q0) and torch.equal(s, s0)
    for b, v in ((bh, H), (by, Y), (bq, q)):
        v.fill_(5)
        assert bool((b == 5).all())
    dY, dH = rows(g, T, d, dtype, d + pad, offset), rows(g, T, d, dtype, d + pad + 3, offset)
    dx0, dw0 = fp.rms_norm_backward(dY.contiguous(), X.contiguous(), w, dH=dH.contiguous())
    bx, dx = guarded(dtype)
    _, dw = fp.rms_norm_backward(dY, X, w, dH=dH, out=dx)
    assert torch.equal(dx, dx0) and torch.equal(dw, dw0)
    dx.fill_(5)
    assert bool((bx == 5).all())


@pytest.mark.parametrize("d", [100, 700, 1500, 8000, 11000, 20000])
@pytest.mark.parametrize("dtype", TYPES)
def test_in_place(fp, d, dtype):
    """The stream updated in place, the norm written over its input, the gradient over its own."""
    g = torch.Generator("cuda").manual_seed(d)
    X, R, w = rows(g, 6, d, dtype), rows(g, 6, d, dtype), torch.randn(d, generator=g, device="cuda")
    Y0, H0 = fp.rms_norm(X, w, residual=R)
    q0, s0 = fp.rms_norm_quantize(X, w, residual=R)[:2]
    r, x = R.clone(), X.clone()
    Y, H = fp.rms_norm(x, w, residual=r, residual_out=r, out=x)
    assert H is r and torch.equal(r, H0) and Y is x and torch.equal(x, Y0)
    r, x = R.clone(), X.clone()
    q, s, _ = fp.rms_norm_quantize(x, w, residual=r, residual_out=x, Y=r)
    assert torch.equal(x, H0) and torch.equal(r, Y0) and torch.equal(q, q0) and torch.equal(s, s0)
    if d <= 16384:
        dY, dH = rows(g, 6, d, dtype), rows(g, 6, d, dtype)
        dx0, dw0 = fp.rms_norm_backward(dY, X, w, dH=dH)
        for which in range(3):
            t = [dY.clone(), X.clone(), dH.clone()]
            dx, dw = fp.rms_norm_backward(t[0], t[1], w, dH=t[2], out=t[which])
            assert torch.equal(dx, dx0) and torch.equal(dw, dw0)


@pytest.mark.parametrize("d", [40, 300, 1200, 3000, 9000, 20000])
def test_extremes(fp, d):
    """Zeros, tiny and huge values, infinities and NaN, next to ordinary rows."""
    g = torch.Generator("cuda").manual_seed(d)
    X = torch.randn((9, d), generator=g, device="cuda")
    X[1] = 0
    X[2] *= 1e-18
    X[3] *= 2.0 ** 90   # its squares' sum leaves fp32
    X[4] = 3e38
    X[5, d // 2] = float("inf")
    X[6, d - 1] = float("nan")
    X[7, 0] = 3.3e38
    w = 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    dY = torch.randn((9, d), generator=g, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        x, dy = X.to(dtype), dY.to(dtype)
        Y = torch.empty_like(x)
        q, scale = fp.rms_norm_quantize(x, w, Y=Y)
        fine = [0, 1, 2, 3, 4, 7, 8]
        _, want = exact(x[fine], w, 1e-5)
        within(Y[fine], want, 60 * U * want.abs() + half_step(want, dtype))
        assert torch.equal(Y[fine], fp.rms_norm(x, w)[fine])  # NaN is not equal to itself
        assert bool((q[1] == 0).all()) and float(scale[1]) == 0
        top = want.abs().amax(1)
        within(scale[fine], top / 127, 62 * U * top / 127 + 1e-45)
        inf = torch.zeros(d, dtype=torch.bool, device="cuda")
        inf[d // 2] = True
        assert bool(Y[5][inf].isnan().all()) and bool((Y[5][~inf] == 0).all())
        assert bool(Y[6].isnan().all())
        assert bool(scale[[5, 6]].isnan().all()) and bool((q[[5, 6]] == 0).all())
        if d <= 16384:
            dx, dw = fp.rms_norm_backward(dy[fine], x[fine], w)
            check_gradients(dx, dw, dy[fine], x[fine], w, 1e-5, None)


def check_gradients(dx, dw, dY, H, w, eps, dH):
    h, dy, dtype = H.double(), dY.double(), H.dtype
    s = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    n, gr = h * s, dy if w is None else dy * w.double()
    mean, size = (gr * n).mean(1, keepdim=True), (gr * n).abs().mean(1, keepdim=True)
    want = s * (gr - n * mean) + (0 if dH is None else dH.double())
    own = 64 * U * s * gr.abs() + 160 * U * s * n.abs() * size
    within(dx, want, own + 2 * U * want.abs() + half_step(want, dtype))
    if w is not None:
        T = H.shape[0]
        c = 56 + -(-T // 256) + 48 + 16 + 16
        within(dw, (dy * n).sum(0), c * U * (dy * n).abs().sum(0) + 1e-44)


@pytest.mark.parametrize("T,d", [s for s in SHAPES if s[1] <= 16384] + [(3000, 300), (2000, 1025), (900, 5000)])
@pytest.mark.parametrize("dtype", TYPES)
def test_gradients(fp, T, d, dtype):
    g = torch.Generator("cuda").manual_seed(T * 41 + d)
    H, dY, dH = rows(g, T, d, dtype), rows(g, T, d, dtype), rows(g, T, d, dtype)
    for wt in {dtype, torch.float32}:
        w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(wt)
        check_gradients(*fp.rms_norm_backward(dY, H, w, eps=1e-5), dY, H, w, 1e-5, None)
    dx, dw = fp.rms_norm_backward(dY, H, w, eps=1e-3, dH=dH)
    check_gradients(dx, dw, dY, H, w, 1e-3, dH)
    dx, dw = fp.rms_norm_backward(dY, H, None, dH=dH)
    assert dw is None
    check_gradients(dx, None, dY, H, None, 1e-5, dH)


@pytest.mark.parametrize("d", [12, 400, 5000])
def test_gradients_by_differences(fp, d):
    """Along random directions of x and w: the difference of the call's own outputs. Its error is that of the outputs (56 u
    each) over the step, and the formula's own curvature, which is taken from 64 bits."""
    g = torch.Generator("cuda").manual_seed(d)
    T, e = 3, 2.0 ** -8
    X, w = torch.randn((T, d), generator=g, device="cuda"), 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    dY = torch.randn((T, d), generator=g, device="cuda")
    dx, dw = fp.rms_norm_backward(dY, X, w)
    vx, vw = torch.randn((T, d), generator=g, device="cuda"), torch.randn(d, generator=g, device="cuda")
    for ax, aw, grad, v in ((e, 0, dx, vx), (0, e, dw, vw)):
        ends, curves, noise = [], [], 0.0
        for sign in (1, -1):
            x, ww = X + sign * ax * vx, w + sign * aw * vw
            y = fp.rms_norm(x, ww).double() * dY.double()
            ends.append(y.sum())
            want = exact(x, ww, 1e-5)[1] * dY.double()
            curves.append(want.sum())
            noise += float(57 * U * want.abs().sum())
        along = (grad.double() * v.double()).sum()
        x = X.double().requires_grad_()
        ww = w.double().requires_grad_()
        (x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-5) * ww * dY.double()).sum().backward()
        g64 = ((x.grad if ax else ww.grad) * v.double()).sum()
        bend = abs(float((curves[0] - curves[1]) / (2 * e) - g64))
        size = float((grad.double() * v.double()).abs().sum())
        step = float(U * 4 * size)  # the rounding of x + e v itself: e v is known to 2 u |x| / e
        moved = float(2 * U / e * ((x.grad if ax else ww.grad).abs() * ((X if ax else w).double().abs() + 1)).sum())
        assert abs(float((ends[0] - ends[1]) / (2 * e) - along)) <= bend + noise / (2 * e) + step + moved + 200 * U * size


def test_empty(fp):
    w = torch.ones(64, device="cuda")
    X = torch.zeros((0, 64), device="cuda")
    assert fp.rms_norm(X, w).shape == (0, 64)
    q, s = fp.rms_norm_quantize(X, w)
    assert q.shape == (0, 64) and s.shape == (0,)
    dx, dw = fp.rms_norm_backward(X, X, w)
    assert dx.shape == (0, 64) and bool((dw == 0).all())
    E = torch.zeros((3, 0), device="cuda")
    s = torch.full((3,), 7.0, device="cuda")
    assert fp.rms_norm(E, torch.zeros(0, device="cuda")).shape == (3, 0)
    fp.rms_norm_quantize(E, None, scale=s)
    assert bool((s == 0).all())


def test_rows_past_32_bits(fp):
    """Rows whose offset leaves 32 bits (2^31 elements and more), forward and backward."""
    ld = 1 << 21
    buf = torch.zeros((1030, ld), dtype=torch.bfloat16, device="cuda")
    X = buf[:, :500]
    X.copy_(torch.randn((1030, 500), device="cuda"))
    w = torch.randn(500, device="cuda")
    assert torch.equal(fp.rms_norm(X, w), fp.rms_norm(X.contiguous(), w))
    out = buf[:, 1000:1500]
    dx, dw = fp.rms_norm_backward(X, X, w, out=out)
    dx0, dw0 = fp.rms_norm_backward(X.contiguous(), X.contiguous(), w)
    assert torch.equal(dx, dx0) and torch.equal(dw, dw0)


def test_streams_and_graphs(fp):
    """A step captured and replayed several times beside the same calls on another stream, each against the eager result."""
    g = torch.Generator("cuda").manual_seed(3)
    sets = [(rows(g, 300, 1000, torch.bfloat16), rows(g, 300, 1000, torch.bfloat16)) for _ in range(4)]
    w = torch.randn(1000, generator=g, device="cuda")

    def step(X, R):
        q, s, H = fp.rms_norm_quantize(X, w, residual=R)
        dx, dw = fp.rms_norm_backward(X, H, w, dH=R)
        return q, s, H, dx, dw
    want = [step(*s) for s in sets]
    X, R = sets[0][0].clone(), sets[0][1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(X, R)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(X, R)
    for i in (1, 2, 3, 0):
        X.copy_(sets[i][0])
        R.copy_(sets[i][1])
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            other = step(*sets[(i + 1) % 4])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(other, want[(i + 1) % 4]))


@pytest.mark.parametrize("size_h,size_g,eps", [(1e15, 1e25, 1e-5), (1.0, 1e37, 1e-5), (2.0 ** 90, 1e25, 1e-5), (2.0 ** 66, 1e-15, 1e-5), (1e15, 0.0, 1e-5), (1e30, 0.0, 1e-5),
                                               (1e-15, 1e-28, 1e-30)])
@pytest.mark.parametrize("d", [1, 40, 300, 1200, 4096, 16384])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_far_from_one(fp, size_h, size_g, eps, d, dtype):
    """A row whose products with its gradient leave fp32's range, or fall below it, where the row's own gradient does not;
    the ordinary rows beside it keep theirs."""
    g = torch.Generator("cuda").manual_seed(d)
    H, dY = torch.randn((3, d), generator=g, device="cuda"), torch.randn((3, d), generator=g, device="cuda").clamp(-3, 3)
    w = 1 + 0.3 * torch.rand(d, generator=g, device="cuda")
    plain = fp.rms_norm_backward(dY.to(dtype), H.to(dtype), w, eps=eps)[0]
    H[1] *= size_h
    dY[1] *= size_g
    H, dY = H.to(dtype), dY.to(dtype)
    dx, dw = fp.rms_norm_backward(dY, H, w, eps=eps)
    assert torch.equal(dx[[0, 2]], plain[[0, 2]])
    check_gradients(dx, dw, dY, H, w, eps, None)


@pytest.mark.parametrize("T,d", [(9000, 300), (2100, 1500), (512, 5000), (513, 5000), (2100, 5000), (513, 2100), (600, 9001), (1100, 20000)])
@pytest.mark.parametrize("dtype", TYPES)
def test_more_rows_than_workgroups(fp, T, d, dtype):
    """Every form for many rows, each workgroup with several of them, bad ones between: floats, stream and int8 rows."""
    g = torch.Generator("cuda").manual_seed(T + d)
    X, R = rows(g, T, d, dtype), rows(g, T, d, dtype)
    X[5::97, d // 3] = float("nan")
    if dtype != torch.float16:
        X[6::97] = 1e30
        R[6::97] = 0
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    Y = torch.empty_like(X)
    q, scale, H = fp.rms_norm_quantize(X, w, residual=R, Y=Y)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[5::97] = True
    assert bool(Y[bad].isnan().all()) and bool(scale[bad].isnan().all()) and bool((q[bad] == 0).all())
    h, want = exact(X[~bad], w, 1e-5, R[~bad])
    within(H[~bad], h, U * h.abs() + half_step(h, dtype))
    within(Y[~bad], want, 60 * U * want.abs() + half_step(want, dtype))
    step = scale[~bad].double()[:, None]
    within(scale[~bad], want.abs().amax(1) / 127, 62 * U * want.abs().amax(1) / 127)
    within(q[~bad].double() * step, want, (0.5 + 2.0 ** -14) * step + 61 * U * want.abs())
