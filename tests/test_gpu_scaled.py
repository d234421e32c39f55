"""Scaled int8 products, row quantization and the grouped form on the GPU
against 64-bit references.

Tolerances. With u = 2^-24, S = Z x_scale w_scale and B the bias, the kernel
rounds Z, Z x_scale and the fused last step once each, so before the output's
rounding |y - (S + B)| <= ((1 + u)^3 - 1) |S| + u |B| <= 3.1 u (|S| + |B|); the
output's type then adds half a step, eps / 2 of the value, or half of its
smallest step (fp16: 2^-25; fp32 and bf16 as fp32's subnormals: 2^-134 and below)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def close(y, want, mag, dtype, extra=0.0):
    """|y - want| within the bound above (mag: |S| + |B|)."""
    got = y.double().cpu().numpy()
    if dtype == torch.float16:
        lim = np.abs(want) < 65504 * (1 - 2.0 ** -12)  # beyond: infinity or the largest value
        got, want, mag = got[lim], want[lim], mag[lim]
    tol = (3.1 * U + extra) * mag + torch.finfo(dtype).eps / 2 * (np.abs(want) + 4 * U * mag) + 2.0 ** -25 * (dtype == torch.float16) + 1e-38
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


def inputs(rng, T, d_in, d_out, ldx=None, offset=0):
    """int8 X (a view with this row stride and offset), W, scales and a bias."""
    ldx = ldx or (d_in + 15) // 16 * 16
    buf = torch.from_numpy(rng.integers(-128, 128, size=T * ldx + offset + 16, dtype=np.int8)).cuda()
    X = torch.as_strided(buf, (T, d_in), (ldx, 1), offset)
    W = torch.from_numpy(rng.integers(-128, 128, size=(d_out, d_in), dtype=np.int8)).cuda()
    xs = torch.from_numpy(rng.uniform(0.001, 0.1, T).astype(np.float32)).cuda()
    ws = torch.from_numpy(rng.uniform(1e-4, 1e-2, d_out).astype(np.float32)).cuda()
    return X, W, xs, ws, torch.from_numpy(rng.normal(size=d_out).astype(np.float32)).cuda()


def reference(X, W, xs, ws, bias=None):
    """(Z, Y, |S| + |B|) in 64 bits (Z exact: below 2^53)."""
    Z = X.cpu().numpy().astype(np.float64) @ W.cpu().numpy().astype(np.float64).T
    S = Z * xs.cpu().numpy().astype(np.float64)[:, None] * ws.cpu().numpy().astype(np.float64)
    B = np.zeros_like(S) if bias is None else np.broadcast_to(bias.cpu().numpy().astype(np.float64), S.shape)
    return Z, S + B, np.abs(S) + np.abs(B)


# one token to many, one output to many, ragged in every direction, K from nothing to several hundred blocks
SHAPES = [(1, 1, 1), (1, 64, 32), (1, 4096, 100), (2, 17, 33), (5, 100, 257), (16, 128, 16), (17, 640, 1000), (31, 63, 129),
          (32, 1000, 512), (33, 65, 255), (64, 2048, 96), (65, 96, 300), (100, 4096, 64), (128, 64, 128), (129, 192, 513),
          (200, 1111, 777), (256, 512, 1024), (500, 320, 260), (700, 160, 2100), (3, 14336, 48), (40, 8192, 40), (7, 0, 9)]


@pytest.mark.parametrize("T,d_in,d_out", SHAPES)
def test_scaled_matmul(fp, T, d_in, d_out):
    rng = np.random.default_rng(T * 7919 + d_in * 31 + d_out)
    X, W, xs, ws, bias = inputs(rng, T, d_in, d_out)
    Z, Y, mag = reference(X, W, xs, ws, bias)
    _, Y0, mag0 = reference(X, W, xs, ws)
    Wp = fp.pack_weights(W)
    for dt in TYPES:
        z = torch.full((T, d_out), 7, dtype=torch.int32, device="cuda")
        y = fp.scaled_matmul(X, xs, Wp, ws, bias=bias, dtype=dt, Z=z)
        assert y.dtype == dt and np.array_equal(z.cpu().numpy(), Z.astype(np.int64))
        close(y, Y, mag, dt)
        close(fp.scaled_matmul(X, xs, Wp, ws, dtype=dt), Y0, mag0, dt)


@pytest.mark.parametrize("T,d_in,d_out", [(1, 100, 70), (20, 333, 90), (70, 1000, 130), (300, 65, 515)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 3), (16, 1), (28, 0)])
def test_scaled_matmul_any_rows(fp, T, d_in, d_out, pad, offset):
    """Row strides and addresses of X that are no multiple of 16."""
    rng = np.random.default_rng(T + d_in + pad)
    X, W, xs, ws, bias = inputs(rng, T, d_in, d_out, ldx=d_in + pad, offset=offset)
    Z, Y, mag = reference(X, W, xs, ws, bias)
    z = torch.zeros((T, d_out), dtype=torch.int32, device="cuda")
    y = fp.scaled_matmul(X, xs, fp.pack_weights(W), ws, bias=bias, dtype=torch.float32, Z=z)
    assert np.array_equal(z.cpu().numpy(), Z.astype(np.int64))
    close(y, Y, mag, torch.float32)


def test_one_row_at_the_end_of_its_storage(fp):
    """A single row whose last 16-byte chunk would leave its storage is read to its end only."""
    rng = np.random.default_rng(8)
    _, W, _, ws, _ = inputs(rng, 1, 100, 70)
    buf = torch.from_numpy(rng.integers(-128, 128, size=3 * 128 + 100, dtype=np.int8)).cuda()
    X = torch.as_strided(buf, (1, 100), (128, 1), 3 * 128)
    xs = torch.ones(1, device="cuda")
    Z, Y, mag = reference(X, W, xs, ws)
    close(fp.scaled_matmul(X, xs, fp.pack_weights(W), ws, dtype=torch.float32), Y, mag, torch.float32)


@pytest.mark.parametrize("T,d_out", [(1, 96), (9, 100), (40, 31), (150, 260)])
@pytest.mark.parametrize("dt", TYPES)
def test_scaled_matmul_strided_out(fp, T, d_out, dt):
    """Outputs that are columns of wider rows: nothing beside them is written."""
    rng = np.random.default_rng(T)
    X, W, xs, ws, _ = inputs(rng, T, 128, d_out)
    Z, Y, mag = reference(X, W, xs, ws)
    Wp = fp.pack_weights(W)
    for left, right in ((0, 0), (16, 16), (3, 2)):
        big = torch.full((T + 2, left + d_out + right), 5.0, dtype=dt, device="cuda")
        zig = torch.full((T + 2, left + d_out + right), 5, dtype=torch.int32, device="cuda")
        y, z = big[1:T + 1, left:left + d_out], zig[1:T + 1, left:left + d_out]
        fp.scaled_matmul(X, xs, Wp, ws, out=y, Z=z)
        assert np.array_equal(z.cpu().numpy(), Z.astype(np.int64))
        close(y, Y, mag, dt)
        y.fill_(5.0)
        z.fill_(5)
        assert bool((big == 5.0).all()) and bool((zig == 5).all())


@pytest.mark.parametrize("T,d_in,d_out,dt", [(1000, 2000, 8000, torch.bfloat16), (900, 1999, 8100, torch.float32),
                                             (4200, 640, 4200, torch.bfloat16), (2100, 1111, 8200, torch.float16),
                                             (513, 4096, 14336, torch.bfloat16)])
def test_large_tiles(fp, T, d_in, d_out, dt):
    """Products of whole tiles, of half tiles, of both, with ragged last ones in every direction (references by a 64-bit
    product on the GPU, exact for these integers)."""
    rng = np.random.default_rng(T + d_out)
    X, W, xs, ws, bias = inputs(rng, T, d_in, d_out)
    big = torch.full((T + 2, d_out + 8), 5.0, dtype=dt, device="cuda")
    z = torch.full((T, d_out), 7, dtype=torch.int32, device="cuda")
    fp.scaled_matmul(X, xs, fp.pack_weights(W), ws, bias=bias, out=big[1:T + 1, :d_out], Z=z)
    Z = X.double() @ W.double().t().contiguous()
    assert torch.equal(z, Z.to(torch.int32))
    S = Z * xs.double()[:, None] * ws.double()
    close(big[1:T + 1, :d_out], (S + bias.double()).cpu().numpy(), (S.abs() + bias.double().abs()).cpu().numpy(), dt)
    assert bool((big[0] == 5.0).all()) and bool((big[T + 1] == 5.0).all()) and bool((big[:, d_out:] == 5.0).all())


def test_rows_past_32_bits(fp):
    """Rows of X, Y and Z that start more than 2^31 bytes (and elements) into their tensors: the last rows equal those of
    a call on them alone, which takes another kernel."""
    T, d_in, d_out = 540000, 4096, 4100  # X: 2.2 G bytes; Y: 2.2 G elements
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    X = torch.randint(-128, 128, (T, d_in), generator=g, device="cuda", dtype=torch.int8)
    W = torch.randint(-128, 128, (d_out, d_in), generator=g, device="cuda", dtype=torch.int8)
    xs, ws = torch.rand(T, generator=g, device="cuda"), torch.rand(d_out, generator=g, device="cuda")
    Wp = fp.pack_weights(W)
    y, z = torch.zeros((T, d_out), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, d_out), dtype=torch.int32, device="cuda")
    fp.scaled_matmul(X, xs, Wp, ws, out=y, Z=z)
    for a, b in ((T - 5, T), (262000, 262007), (0, 8)):
        z2 = torch.zeros((b - a, d_out), dtype=torch.int32, device="cuda")
        y2 = fp.scaled_matmul(X[a:b], xs[a:b], Wp, ws, Z=z2)
        assert torch.equal(y[a:b], y2) and torch.equal(z[a:b], z2)
    # the same rows picked by index for a group, and quantized
    rows = torch.tensor([T - 1, 0, T - 2], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    y3 = fp.scaled_matmul_grouped(X, xs, fp.PackedExperts([Wp]), ws[None], off, rows=rows)
    assert torch.equal(y3, y[rows.long()])
    q, s = fp.quantize_rows(y)
    q2, s2 = fp.quantize_rows(y[T - 3:].clone())
    assert torch.equal(q[T - 3:], q2) and torch.equal(s[T - 3:], s2)


def test_extremes(fp):
    """The largest |Z| (every product (-128)^2 over d_in = 131071), zero scales, infinities and NaN in the scales, and
    values beyond fp16."""
    X = torch.full((3, 131071), -128, dtype=torch.int8, device="cuda")
    W = torch.full((40, 131071), -128, dtype=torch.int8, device="cuda")
    xs = torch.tensor([1.0, 0.0, float("nan")], device="cuda")
    ws = torch.ones(40, device="cuda")
    ws[1] = float("inf")
    Wp = fp.pack_weights(W)
    z = torch.zeros((3, 40), dtype=torch.int32, device="cuda")
    y = fp.scaled_matmul(X, xs, Wp, ws, dtype=torch.float32, Z=z)
    assert bool((z == 2 ** 14 * 131071).all())
    assert float(y[0, 0]) == float(np.float32(2 ** 14 * 131071)) and bool(torch.isinf(y[0, 1]))
    assert float(y[1, 0]) == 0.0 and bool(torch.isnan(y[1, 1])) and bool(torch.isnan(y[2]).all())
    h = fp.scaled_matmul(X, xs, Wp, ws, dtype=torch.float16)
    assert bool(torch.isinf(h[0]).all()) and float(h[1, 0]) == 0.0
    # scales whose product leaves fp32 while the answer does not
    tiny = torch.full((3,), 1e-25, device="cuda")
    y = fp.scaled_matmul(X, tiny, Wp, torch.full((40,), 1e-20, device="cuda"), dtype=torch.float32)
    want = 2 ** 14 * 131071 * float(np.float32(1e-25)) * float(np.float32(1e-20))
    assert abs(float(y[0, 0]) - want) <= 3.1 * U * want + 2.0 ** -149


def test_z_is_the_witness(fp):
    """The product beside the answer is the one the layer's proof is about."""
    rng = np.random.default_rng(3)
    for T, d_in, d_out in ((4, 256, 96), (100, 320, 700)):
        X, W, xs, ws, _ = inputs(rng, T, d_in, d_out)
        Wp = fp.pack_weights(W)
        Zw, _, _ = fp.witness_linear_packed(X, Wp, 8)
        z = torch.zeros_like(Zw)
        fp.scaled_matmul(X, xs, Wp, ws, Z=z)
        assert torch.equal(z, Zw)


# ------------------------------------------------------------ quantization --
def quantized(x):
    """The definition in fp32, step by step (x: float32 array)."""
    top = np.abs(x).max(axis=1, initial=0).astype(np.float32)
    pre = np.where(top < np.float32(2.0 ** -100), np.float32(2.0 ** 64), np.float32(1)).astype(np.float32)
    with np.errstate(all="ignore"):
        inv = np.where(top > 0, np.float32(127) * (np.float32(1) / (top * pre)), np.float32(0)).astype(np.float32)
        q = np.rint((x * pre[:, None]).astype(np.float32) * inv[:, None]).astype(np.float32)
        scale = (top / np.float32(127)).astype(np.float32)
    bad = ~np.isfinite(x).all(axis=1)
    q[bad] = 0
    scale[bad] = np.nan
    return np.clip(q, -127, 127).astype(np.int8), scale


@pytest.mark.parametrize("T,d", [(1, 1), (1, 4096), (1, 5), (3, 16), (17, 1000), (64, 1111), (5, 14336), (300, 256), (2, 40000), (9, 0)])
@pytest.mark.parametrize("dt", TYPES)
def test_quantize_rows(fp, T, d, dt):
    rng = np.random.default_rng(T + d)
    for left, right in ((0, 0), (3, 6)):
        big = torch.from_numpy((rng.standard_normal((T, left + d + right)) * np.exp(rng.normal(size=(T, 1)) * 3)).astype(np.float32)).cuda().to(dt)
        X = big[:, left:left + d]
        q, s = fp.quantize_rows(X)
        wq, ws = quantized(X.float().cpu().numpy())
        assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), wq)
        if d:  # within half a step of the value, and the largest magnitude is met
            x = X.double().cpu().numpy()
            step = s.double().cpu().numpy()[:, None]
            assert (np.abs(x - q.cpu().numpy() * step) <= step * (0.5 + 127 * 4 * U)).all()
            assert (np.abs(q.cpu().numpy().astype(int)).max(axis=1) == 127).all()
        # into columns of a wider buffer
        out = torch.full((T, d + 9), 77, dtype=torch.int8, device="cuda")
        fp.quantize_rows(X, out=out[:, 4:4 + d], scale=s)
        assert np.array_equal(out[:, 4:4 + d].cpu().numpy(), wq)
        assert bool((out[:, :4] == 77).all()) and bool((out[:, 4 + d:] == 77).all())


def test_quantize_special_rows(fp):
    """Zeros, one nonzero, subnormal and huge rows, infinities and NaN, ties."""
    d = 200
    x = np.zeros((10, d), np.float32)
    x[1, 7] = -3.0
    x[2] = np.linspace(-1, 1, d) * 2.0 ** -140
    x[3] = np.linspace(-1, 1, d) * 3e38
    x[4] = 1.0
    x[4, 5] = np.inf
    x[5] = 1.0
    x[5, 199] = np.nan
    x[6, 0], x[6, 1:128] = 127.0, np.arange(127) + 0.5  # ties to even
    x[7] = 2.0 ** -126
    x[8] = np.linspace(-1, 1, d) * 2.0 ** -101
    x[9, 0] = 2.0 ** -149
    q, s = fp.quantize_rows(torch.from_numpy(x).cuda())
    wq, ws = quantized(x)
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(q, wq) and np.array_equal(s, ws, equal_nan=True)
    assert not q[0].any() and s[0] == 0 and np.isnan(s[4]) and np.isnan(s[5]) and q[6, 1] == 0 and q[6, 2] == 2
    W = torch.ones((3, d), dtype=torch.int8, device="cuda")
    y = fp.scaled_linear(torch.from_numpy(x).cuda(), fp.pack_weights(W), torch.ones(3, device="cuda")).cpu().numpy()
    assert not y[0].any() and np.isnan(y[4]).all() and np.isnan(y[5]).all() and np.isfinite(y[[0, 1, 2, 6, 7, 8, 9]]).all()


@pytest.mark.parametrize("T,d_in,d_out", [(1, 4096, 300), (1, 1, 1), (4, 100, 64), (33, 1000, 130), (16, 2048, 4096), (150, 640, 257), (0, 64, 32), (3, 0, 5)])
@pytest.mark.parametrize("dt", TYPES)
def test_scaled_linear(fp, T, d_in, d_out, dt):
    """The same as the two calls, whatever path a few tokens take."""
    rng = np.random.default_rng(T + d_in)
    _, W, _, ws, bias = inputs(rng, 1, d_in, d_out)
    X = torch.from_numpy(rng.standard_normal((T, d_in)).astype(np.float32)).cuda().to(dt)
    Wp = fp.pack_weights(W)
    q, s = fp.quantize_rows(X)
    z, z2 = (torch.full((T, d_out), 3, dtype=torch.int32, device="cuda") for _ in range(2))
    y = fp.scaled_linear(X, Wp, ws, bias=bias, Z=z)
    assert y.dtype == dt
    assert torch.equal(y, fp.scaled_matmul(q, s, Wp, ws, bias=bias, dtype=dt, Z=z2)) and torch.equal(z, z2)
    Z, Y, mag = reference(q, W, s, ws, bias)
    assert np.array_equal(z.cpu().numpy(), Z.astype(np.int64))
    close(y, Y, mag, dt)


# ----------------------------------------------------------------- grouped --
def group_inputs(rng, counts, x_rows, d_in, d_out, index=True, stray=0):
    G = len(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(off[-1]) + stray
    X, _, xs, _, _ = inputs(rng, x_rows, d_in, 1)
    W = [torch.from_numpy(rng.integers(-128, 128, size=(d_out, d_in), dtype=np.int8)).cuda() for _ in range(G)]
    ws = torch.from_numpy(rng.uniform(1e-4, 1e-2, (G, d_out)).astype(np.float32)).cuda()
    bias = torch.from_numpy(rng.normal(size=(G, d_out)).astype(np.float32)).cuda()
    rows = torch.from_numpy(rng.integers(0, x_rows, n).astype(np.int32)).cuda() if index else None
    return X, xs, W, ws, bias, torch.from_numpy(off).cuda(), rows, n


@pytest.mark.parametrize("counts,x_rows,d_in,d_out,index", [
    ([1], 1, 64, 32, True), ([0, 3, 0, 0, 5, 1, 0], 6, 100, 70, True), ([40, 0, 33, 32, 31, 1], 137, 320, 300, False),
    ([0, 0, 0], 4, 64, 64, True), ([300, 2, 0, 129], 50, 192, 130, True), ([700, 900], 512, 128, 520, True),
    ([int(c) for c in np.random.default_rng(1).integers(0, 4, 256)], 40, 64, 40, True),
    ([2] * 100, 9, 2048, 96, True), ([1, 1, 1, 1, 1, 1, 1, 1], 2, 4096, 512, True), ([5, 0, 7], 12, 0, 33, True)])
def test_grouped(fp, counts, x_rows, d_in, d_out, index):
    rng = np.random.default_rng(sum(counts) + d_in)
    stray = 3 if index else 0  # rows behind the last group
    X, xs, W, ws, bias, off, rows, n = group_inputs(rng, counts, x_rows, d_in, d_out, index, stray)
    We = fp.pack_experts(W)
    for dt, b in ((torch.float32, bias), (torch.bfloat16, None), (torch.float16, bias)):
        y = torch.full((n, d_out), 9.0, dtype=dt, device="cuda")
        z = torch.full((n, d_out), 9, dtype=torch.int32, device="cuda")
        fp.scaled_matmul_grouped(X, xs, We, ws, off, rows=rows, bias=b, out=y, Z=z)
        o = off.tolist()
        for g in range(len(counts)):
            if counts[g] == 0:
                continue
            sl = slice(o[g], o[g + 1])
            pick = rows[sl].long() if index else torch.arange(o[g], o[g + 1], device="cuda")
            Z, Y, mag = reference(X[pick], W[g], xs[pick], ws[g], None if b is None else b[g])
            assert np.array_equal(z[sl].cpu().numpy(), Z.astype(np.int64)), g
            close(y[sl], Y, mag, dt)
        assert bool((y[o[-1]:] == 9.0).all()) and bool((z[o[-1]:] == 9).all())


def test_grouped_large_tiles(fp):
    """Groups of several tiles, of one row and of none, whose last tiles are of every width, over many weight panels."""
    rng = np.random.default_rng(77)
    counts = [600, 0, 1, 257, 130, 65, 0, 64, 512, 33]
    X, xs, W, ws, bias, off, rows, n = group_inputs(rng, counts, 400, 448, 1500, True, 5)
    y = torch.full((n, 1500), 9.0, dtype=torch.bfloat16, device="cuda")
    z = torch.full((n, 1500), 9, dtype=torch.int32, device="cuda")
    fp.scaled_matmul_grouped(X, xs, fp.pack_experts(W), ws, off, rows=rows, bias=bias, out=y, Z=z)
    o = off.tolist()
    for g, c in enumerate(counts):
        if c:
            pick = rows[o[g]:o[g + 1]].long()
            Z, Y, mag = reference(X[pick], W[g], xs[pick], ws[g], bias[g])
            assert np.array_equal(z[o[g]:o[g + 1]].cpu().numpy(), Z.astype(np.int64)), g
            close(y[o[g]:o[g + 1]], Y, mag, torch.bfloat16)
    assert bool((y[o[-1]:] == 9.0).all()) and bool((z[o[-1]:] == 9).all())


def test_grouped_unaligned_and_index_out_of_range(fp):
    """X's rows of no multiple of 16 bytes; rows whose index is no row of X are left as they were."""
    rng = np.random.default_rng(11)
    for counts, d_in in (([3, 2, 6], 77), ([60, 90, 41], 333)):
        X, xs, W, ws, bias, off, rows, n = group_inputs(rng, counts, 10, d_in, 50)
        X = X.contiguous()
        rows[1], rows[4] = -1, 10
        y = torch.full((n, 50), 9.0, device="cuda")
        fp.scaled_matmul_grouped(X, xs, fp.pack_experts(W), ws, off, rows=rows, out=y)
        o, r = off.tolist(), rows.tolist()
        for g in range(3):
            for i in range(o[g], o[g + 1]):
                if 0 <= r[i] < 10:
                    _, Y, mag = reference(X[r[i]:r[i] + 1], W[g], xs[r[i]:r[i] + 1], ws[g])
                    close(y[i:i + 1], Y, mag, torch.float32)
                else:
                    assert bool((y[i] == 9.0).all())


def test_grouped_offsets_beyond_the_rows(fp):
    """Offsets past the rows, and ends before their starts, are cut to what there is: nothing outside is touched."""
    rng = np.random.default_rng(12)
    X, xs, W, ws, bias, off, rows, n = group_inputs(rng, [4, 4, 4], 8, 64, 40)
    We = fp.pack_experts(W)
    big = torch.full((n + 4, 40), 9.0, device="cuda")
    off2 = torch.tensor([0, 4, 4, 100], dtype=torch.int32, device="cuda")
    fp.scaled_matmul_grouped(X, xs, We, ws, off2, rows=rows, out=big[2:n + 2])
    assert bool((big[:2] == 9).all()) and bool((big[n + 2:] == 9).all())
    _, Y, mag = reference(X[rows[4:].long()], W[2], xs[rows[4:].long()], ws[2])
    close(big[6:n + 2], Y, mag, torch.float32)
    off3 = torch.tensor([8, 3, -5, 6], dtype=torch.int32, device="cuda")
    y = torch.full((n, 40), 9.0, device="cuda")
    fp.scaled_matmul_grouped(X, xs, We, ws, off3, rows=rows, out=y)
    assert bool((y[6:] == 9).all())
    _, Y, mag = reference(X[rows[:6].long()], W[2], xs[rows[:6].long()], ws[2])
    close(y[:6], Y, mag, torch.float32)


def test_streams_and_graph_replays(fp):
    """On a stream of its own, and captured (scratch of the capture apart from the eager calls'), replayed with eager
    work between on other inputs of the same buffers."""
    rng = np.random.default_rng(5)
    _, W, _, ws, bias = inputs(rng, 1, 512, 320)
    Wp = fp.pack_weights(W)
    for T in (1, 20, 200):
        xs = [torch.from_numpy(rng.standard_normal((T, 512)).astype(np.float32)).cuda().bfloat16() for _ in range(3)]
        want = [fp.scaled_linear(x, Wp, ws, bias=bias) for x in xs]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = fp.scaled_linear(xs[0], Wp, ws, bias=bias)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(got, want[0])
        x, y = xs[0].clone(), torch.empty((T, 320), dtype=torch.bfloat16, device="cuda")
        graphs = []
        for _ in range(2):  # two graphs of the same call
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                fp.scaled_linear(x, Wp, ws, bias=bias, out=y)
            graphs.append(g)
        for k in range(6):
            x.copy_(xs[k % 3])
            y.zero_()
            graphs[k % 2].replay()
            assert torch.equal(fp.scaled_linear(xs[(k + 1) % 3], Wp, ws, bias=bias), want[(k + 1) % 3])
            torch.cuda.synchronize()
            assert torch.equal(y, want[k % 3])


def test_wrong_device(fp):
    Wp = fp.pack_weights(torch.zeros((32, 64), dtype=torch.int8, device="cuda"))
    with pytest.raises(ValueError, match="device"):
        fp.scaled_matmul(torch.zeros((2, 64), dtype=torch.int8), torch.ones(2), Wp, torch.ones(32, device="cuda"),
                         out=torch.zeros((2, 32), device="cuda"))


def test_grouped_without_tokens(fp):
    """X of no rows: every row's index is outside it, so all are left as they were."""
    rng = np.random.default_rng(14)
    _, _, W, ws, bias, off, rows, n = group_inputs(rng, [2, 3], 4, 64, 40)
    X, xs = torch.empty((0, 64), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    y = torch.full((n, 40), 9.0, device="cuda")
    fp.scaled_matmul_grouped(X, xs, fp.pack_experts(W), ws, off, rows=torch.full_like(rows, -1), bias=bias, out=y)
    assert bool((y == 9).all())


def test_one_group_with_rows_of_scales_apart(fp):
    """One group's scales and bias may be rows of matrices of any width."""
    rng = np.random.default_rng(15)
    X, xs, W, ws, bias, off, rows, n = group_inputs(rng, [7], 5, 64, 40)
    wide = torch.zeros((3, 50), device="cuda")
    wide[1, :40] = bias[0]
    _, Y, mag = reference(X[rows.long()], W[0], xs[rows.long()], ws[0], bias[0])
    for b, w in ((wide[1:2, :40], ws), (bias, torch.cat([ws, ws], 1)[:, :40])):
        close(fp.scaled_matmul_grouped(X, xs, fp.pack_experts(W), w, off, rows=rows, bias=b, dtype=torch.float32), Y, mag, torch.float32)


@pytest.mark.parametrize("T,d_in,d_out", [(2, 100, 70), (9, 20, 96), (40, 1000, 60), (300, 333, 515), (700, 65, 1300)])
def test_rows_that_end_with_their_storage(fp, T, d_in, d_out):
    """Rows 16 bytes apart whose last one ends with the storage, in the middle of a 16-byte chunk."""
    rng = np.random.default_rng(T)
    ld = (d_in + 15) // 16 * 16
    _, W, xs, ws, bias = inputs(rng, T, d_in, d_out)
    buf = torch.from_numpy(rng.integers(-128, 128, size=(T - 1) * ld + d_in, dtype=np.int8)).cuda()
    X = torch.as_strided(buf, (T, d_in), (ld, 1))
    assert X.data_ptr() % 16 == 0 and buf.untyped_storage().nbytes() < T * ld
    Z, Y, mag = reference(X, W, xs, ws, bias)
    z = torch.zeros((T, d_out), dtype=torch.int32, device="cuda")
    Wp = fp.pack_weights(W)
    close(fp.scaled_matmul(X, xs, Wp, ws, bias=bias, dtype=torch.float32, Z=z), Y, mag, torch.float32)
    assert np.array_equal(z.cpu().numpy(), Z.astype(np.int64))
    off = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    back = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    y = fp.scaled_matmul_grouped(X, xs, fp.PackedExperts([Wp, Wp]), torch.stack([ws, ws]), off, rows=back,
                                 bias=torch.stack([bias, bias]), dtype=torch.float32, Z=z)
    close(y, Y[::-1], mag[::-1], torch.float32)
    assert np.array_equal(z.cpu().numpy(), Z[::-1].astype(np.int64))


@pytest.mark.parametrize("G,most,d_in", [(257, 3, 64), (300, 9, 100), (1024, 2, 33), (512, 0, 64)])
def test_grouped_of_many_experts(fp, G, most, d_in):
    """More groups than one launch takes; rows behind the last group are left as they were."""
    rng = np.random.default_rng(G)
    counts = rng.integers(0, most + 1, G)
    X, xs, W, ws, bias, off, rows, n = group_inputs(rng, counts, 20, d_in, 40, True, 3)
    rows[n // 2] = -1
    y = torch.full((n, 40), 9.0, device="cuda")
    z = torch.full((n, 40), 9, dtype=torch.int32, device="cuda")
    fp.scaled_matmul_grouped(X, xs, fp.pack_experts(W), ws, off, rows=rows, bias=bias, out=y, Z=z)
    o, r = off.tolist(), rows.tolist()
    left = np.ones(n, bool)
    for g in range(G):
        for i in range(o[g], o[g + 1]):
            if r[i] < 0:
                continue
            left[i] = False
            Z, Y, mag = reference(X[r[i]:r[i] + 1], W[g], xs[r[i]:r[i] + 1], ws[g], bias[g])
            assert np.array_equal(z[i:i + 1].cpu().numpy(), Z.astype(np.int64))
            close(y[i:i + 1], Y, mag, torch.float32)
    left = torch.from_numpy(left).cuda()
    assert int(left.sum()) >= 3 and bool((y[left] == 9).all()) and bool((z[left] == 9).all())
