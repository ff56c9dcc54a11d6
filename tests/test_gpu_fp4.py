"""The 4-bit operators on the GPU against the float64 oracle (oracle/fp4.py).

Quantiser and inverse: equality (codes, scales, tensor scale, values).

Products: |y - y64| <= (n / 16 + 4) 2^-22 S + h |y64| with S = sum |x w|.
Products of two E2M1 values are exact; a block's 16 of them are summed and
scaled, and at most n / 16 float32 additions follow, each off by at most one
unit in the last place (2^-23 of a sum no larger than S, truncation
included); the factor two covers the rounding of the block sums, the 4 the
tensor scales' and the output's float32 roundings and float32 tokens, which
enter the product as two or three parts (2^-22 S at most).  h is the output type's
half step (bf16 2^-8, float32 2^-24)."""
import numpy as np
import pytest
import torch

import post_quantization_kronq_b200 as kq
from oracle import fp4

pytestmark = pytest.mark.gpu
DEV = "cuda"
MX, NV = kq.MXFP4, kq.NVFP4
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def stored(x, fmt, g=None):
    """(codes, scales, g) on the device and the float64 values, by the oracle."""
    codes, sb, g = fp4.quantize(x, fmt, g)
    c, s = fp4.store(codes, sb, fmt)
    return dev(c), dev(s), None if g is None else dev(np.array([g], np.float32)), fp4.values(codes, sb, fmt)


def quantized(x, fmt, g=None, deq=None, **kw):
    """kronq_fp4_quantize's outputs as numpy arrays, the arrays poisoned before."""
    rows, n = x.shape
    c = torch.full((rows, kq.kronq_fp4_code_row_bytes(n)), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((rows, kq.kronq_fp4_scale_row_bytes(fmt, n)), 0xA5, dtype=torch.uint8, device=DEV)
    gs = None if fmt == MX else torch.tensor([7.0 if g is None else g], device=DEV)
    kq.kronq_fp4_quantize(x, fmt, c, s, gscale=gs, gscale_given=g is not None, deq=deq, **kw)
    torch.cuda.synchronize()
    return c.cpu().numpy(), s.cpu().numpy(), None if gs is None else gs.cpu().numpy()[0]


def check_quantize(x, fmt, g=None):
    deq = torch.full_like(x, 3.0)
    c, s, gs = quantized(x, fmt, g, deq)
    codes, sb, g64 = fp4.quantize(x.float().cpu().numpy(), fmt, g)
    want_c, want_s = fp4.store(codes, sb, fmt)
    assert np.array_equal(s, want_s)
    assert np.array_equal(c, want_c)
    if fmt == NV:
        assert gs == g64
    with np.errstate(over="ignore"):
        v = torch.from_numpy(fp4.values_f32(codes, sb, fmt, g64)).to(x.dtype)
    assert torch.equal(deq.cpu().nan_to_num(nan=12345.0), v.nan_to_num(nan=12345.0))


# ------------------------------------------------------------ quantiser
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 15), (2, 16), (5, 17), (1, 33), (7, 255), (4, 4100), (129, 512), (33, 1000)])
def test_quantize_matches_oracle(fmt, dt, rows, n):
    g = torch.Generator().manual_seed(rows * 1000 + n)
    x = (torch.randn(rows, n, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))).to(dt).to(DEV)
    check_quantize(x, fmt)
    if fmt == NV:
        check_quantize(x, fmt, 0.037)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("g", [1.0, 2.0 ** -9, 0.0123, 3e38, 2.0 ** -126, 1e-30])
def test_nv_borders_are_exact(dt, g):
    # values on the rounding borders of codes and of block scales, and their neighbours
    rng = np.random.default_rng(3)
    g = np.float32(g)
    s = fp4.e4m3_table()[rng.integers(1, 127, size=(512, 1))]
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])[rng.integers(0, 8, size=(512, 32))]
    with np.errstate(over="ignore"):
        x = (mids * s * np.float64(g)).astype(np.float32)
    smid = (fp4.e4m3_table()[1:] + fp4.e4m3_table()[:-1]) / 2 * 6 * np.float64(g)
    with np.errstate(over="ignore"):
        x[:, 5] = smid[rng.integers(0, 126, size=512)].astype(np.float32)
    x = np.clip(x, 0, 3e38)
    step = rng.integers(-1, 2, size=x.shape)
    x = np.where(step < 0, np.nextafter(x, np.float32(0)), np.where(step > 0, np.nextafter(x, np.float32(3e38)), x))
    x *= rng.choice(np.array([-1, 1], np.float32), size=x.shape)
    check_quantize(torch.from_numpy(x).to(dt).to(DEV), NV, g)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("g", [None, 1.0, 2.0 ** -9, 0.0123, 2.0 ** 100, 2.0 ** -100, 3e38, 2.0 ** -126, 1.7e-7])
def test_nv_borders_are_exact_in_a_large_tensor(dt, g):
    # as above with more than two blocks a thread, for every scale byte; a
    # ragged last block; a row of NaN, a row of zeros
    rng = np.random.default_rng(6)
    rows, n = 20000, 250
    gv = np.float32(0.31 if g is None else g)
    table = fp4.e4m3_table()
    s = table[(np.arange(rows) % 126 + 1)][:, None]
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])[rng.integers(0, 8, size=(rows, n))]
    with np.errstate(over="ignore"):
        x = np.clip(mids * s * np.float64(gv), 0, 3e38).astype(np.float32)
        smid = np.clip((table[1:] + table[:-1]) / 2 * 6 * np.float64(gv), 0, 3e38).astype(np.float32)
    x[:, 16:32] *= 0.25
    x[:, 20] = smid[rng.integers(0, 126, size=rows)]
    step = rng.integers(-1, 2, size=x.shape)
    x = np.where(step < 0, np.nextafter(x, np.float32(0)), np.where(step > 0, np.nextafter(x, np.float32(3e38)), x))
    x *= rng.choice(np.array([-1, 1], np.float32), size=x.shape)
    x[7], x[9], x[11, 40] = np.nan, 0.0, np.inf
    check_quantize(torch.from_numpy(x).to(dt).to(DEV), NV, None if g is None else gv)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_mx_borders_and_extreme_exponents(dt):
    rng = np.random.default_rng(4)
    e = rng.integers(-149, 128, size=(2048, 1)).astype(np.float64)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.5])[rng.integers(0, 8, size=(2048, 64))]
    with np.errstate(over="ignore"):
        x = np.clip(mids * 2.0 ** (e - 2), 0, 3e38).astype(np.float32)
    step = rng.integers(-1, 2, size=x.shape)
    x = np.where(step < 0, np.nextafter(x, np.float32(0)), np.where(step > 0, np.nextafter(x, np.float32(3e38)), x))
    x *= rng.choice(np.array([-1, 1], np.float32), size=x.shape)
    check_quantize(torch.from_numpy(x).to(dt).to(DEV), MX)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_quantize_non_finite_zero_and_negative_zero(fmt, dt):
    x = torch.randn(6, 200, generator=torch.Generator().manual_seed(0))
    x[0, 5], x[1, 40], x[2, 199], x[3], x[4, :64] = float("nan"), float("inf"), float("-inf"), 0.0, -0.0
    check_quantize(x.to(dt).to(DEV), fmt)
    check_quantize(torch.zeros(2, 48, dtype=dt, device=DEV), fmt)
    check_quantize(torch.full((2, 48), float("nan"), dtype=dt, device=DEV), fmt)


@pytest.mark.parametrize("g", [0.0, -1.0, float("nan"), float("inf"), 1e-40])
def test_bad_given_scale_makes_every_block_nan(g):
    x = torch.randn(3, 40, device=DEV)
    c, s, _ = quantized(x, NV, g)
    assert (s[:, :3] == 127).all() and c.max() == 0 and s[:, 3:].max() == 0


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_quantize_strided_and_misaligned_rows(fmt, dt):
    base = torch.randn(9, 413, generator=torch.Generator().manual_seed(1)).to(dt).to(DEV)
    for x in (base[:, 1:300], base[:, 8:200], base[::2, 3:67], base[4:5, 7:]):
        d = torch.zeros(x.shape[0], x.shape[1] + 3, dtype=dt, device=DEV)[:, 1:-2]
        c, s, g = quantized(x, fmt, deq=d)
        c2, s2, g2 = quantized(x.contiguous(), fmt)
        assert np.array_equal(c, c2) and np.array_equal(s, s2) and g == g2
        out = torch.empty(x.shape, dtype=dt, device=DEV)
        kq.kronq_fp4_dequantize(dev(c), dev(s), fmt, out, gscale=None if g is None else dev(np.array([g])))
        assert torch.equal(out, d)


def test_quantize_in_place_and_no_rows():
    x = torch.randn(40, 300, device=DEV)
    want = torch.empty_like(x)
    c0, s0, g0 = quantized(x, NV, deq=want)
    y = x.clone()
    c1, s1, g1 = quantized(y, NV, deq=y)
    assert np.array_equal(c0, c1) and np.array_equal(s0, s1) and g0 == g1 and torch.equal(y, want)
    c, s, g = quantized(torch.empty(0, 64, device=DEV), NV)
    assert c.shape == (0, 32) and g == 1.0


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n,ld,first", [(1300, 4096, 4096, 0), (1300, 4099, 4099, 0), (1300, 4096, 4110, 3),
                                             (190, 8192, 8192, 0), (2500, 2000, 2016, 0)])
def test_dequantize_of_many_rows(fmt, dt, rows, n, ld, first):
    """Sizes on both sides of the number of runs that a step takes, aligned and
    unaligned rows; what lies between the rows stays."""
    gen = torch.Generator(device=DEV).manual_seed(rows + n)
    c, s = (torch.empty(rows, b, dtype=torch.uint8, device=DEV)
            for b in (kq.kronq_fp4_code_row_bytes(n), kq.kronq_fp4_scale_row_bytes(fmt, n)))
    c.random_(0, 256, generator=gen)
    s.random_(100, 130, generator=gen) if fmt == MX else s.random_(0, 127, generator=gen)
    g = torch.full((1,), 0.37, device=DEV) if fmt == NV else None
    big = torch.full((rows, ld), 7.0, dtype=dt, device=DEV)
    out = big[:, first:first + n]
    kq.kronq_fp4_dequantize(c, s, fmt, out, gscale=g)
    nib = torch.stack([c & 15, c >> 4], 2).reshape(rows, -1)[:, :n].long()
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    value = torch.where(nib >= 8, -table[nib & 7], table[nib & 7])
    sb = s.repeat_interleave(fp4.BLOCK[fmt], 1)[:, :n]
    # a code times its scale is exact in float32, and one rounding for each of the scale and the type remains
    scale = (sb.int() << 23).view(torch.float32) if fmt == MX else sb.view(torch.float8_e4m3fn).float()
    want = value * scale if g is None else value * scale * g
    assert torch.equal(out, want.to(dt))
    big[:, first:first + n] = 7.0
    assert (big == 7.0).all()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_dequantize_every_code_and_scale(fmt, dt):
    rng = np.random.default_rng(5)
    bs = fp4.BLOCK[fmt]
    sb = np.arange(256 if fmt == MX else 128, dtype=np.uint8)
    codes = np.tile(np.arange(16, dtype=np.uint8), len(sb) * bs // 16)[None, :].repeat(3, 0)
    sb = np.stack([sb, sb[::-1], rng.permutation(sb)])
    c, s = fp4.store(codes, sb, fmt)
    g = np.float32(0.0371)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(fp4.values_f32(codes, sb, fmt, g if fmt == NV else None)).to(dt)
    out = torch.empty(want.shape, dtype=dt, device=DEV)
    kq.kronq_fp4_dequantize(dev(c), dev(s), fmt, out, gscale=dev(np.array([g])) if fmt == NV else None)
    assert torch.equal(out.cpu().nan_to_num(nan=777.0), want.nan_to_num(nan=777.0))


# ------------------------------------------------------------ products
def tolerance(n, S, y64, dt):
    return (n / 16 + 4) * 2.0 ** -22 * S + HALF[dt] * np.abs(y64)


def matmul(xq, wq, fmt, n, y, **kw):
    kq.kronq_fp4_matmul(xq[0], xq[1], wq[0], wq[1], fmt, n, y, xg=xq[2], wg=wq[2], **kw)


def check(y, y64, S, n):
    got = y.double().cpu().numpy()
    assert (np.abs(got - y64) <= tolerance(n, S, y64, y.dtype)).all()


def g_of(q):
    return None if q[2] is None else float(q[2].cpu()[0])


SHAPES = [(1, 1, 1), (1, 64, 64), (3, 130, 33), (17, 257, 255), (128, 128, 256), (65, 300, 1000), (200, 129, 4095),
          (256, 512, 512), (257, 1000, 1030), (16, 4096, 2048), (600, 700, 1536), (5, 8, 8192)]


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,m,n", SHAPES)
def test_matmul_matches_oracle(fmt, dt, T, m, n):
    rng = np.random.default_rng(T + m + n)
    x = stored(rng.standard_normal((T, n)) * np.exp(rng.standard_normal((1, n))), fmt)
    w = stored(0.02 * rng.standard_normal((m, n)), fmt)
    y = torch.full((T, m), float("nan"), dtype=dt, device=DEV)
    matmul(x, w, fmt, n, y)
    check(y, *fp4.product(x[3], w[3], g_of(x), g_of(w)), n)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("T,m,n", [(128, 256, 256), (70, 200, 1024), (300, 513, 2080)])
def test_matmul_is_exact_where_sums_are(fmt, T, m, n):
    # codes and power-of-two scales whose sums fit 24 bits: any misplaced code
    # or scale shows as a wrong whole number
    rng = np.random.default_rng(n)
    def pick(rows):
        codes = rng.integers(0, 16, size=(rows, n)).astype(np.uint8)
        nb = -(-n // fp4.BLOCK[fmt])
        e = rng.integers(-2, 3, size=(rows, nb))
        sb = ((127 + e) if fmt == MX else (7 + e) * 8).astype(np.uint8)
        c, s = fp4.store(codes, sb, fmt)
        return dev(c), dev(s), None if fmt == MX else torch.ones(1, device=DEV), fp4.values(codes, sb, fmt)
    x, w = pick(T), pick(m)
    y = torch.empty(T, m, device=DEV)
    matmul(x, w, fmt, n, y)
    assert np.array_equal(y.cpu().numpy().astype(np.float64), x[3] @ w[3].T)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_matmul_padding_is_not_data(fmt):
    # what lies behind a row's codes and scales (the half byte of an odd n apart) may be anything
    rng = np.random.default_rng(8)
    T, m, n = 40, 150, 330
    x, w = stored(rng.standard_normal((T, n)), fmt), stored(rng.standard_normal((m, n)), fmt)
    y = torch.empty(T, m, device=DEV)
    matmul(x, w, fmt, n, y)
    nb = -(-n // fp4.BLOCK[fmt])
    for q in (x, w):
        q[0][:, n // 2:] = 0x77
        q[1][:, nb:] = 0xFF if fmt == MX else 0x7F
    z = torch.empty_like(y)
    matmul(x, w, fmt, n, z)
    assert torch.equal(y, z)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_matmul_nan_blocks_stay_in_their_rows_and_columns(fmt):
    rng = np.random.default_rng(9)
    T, m, n = 70, 140, 512
    xv, wv = rng.standard_normal((T, n)), rng.standard_normal((m, n))
    xv[3, 100], wv[77, 5] = np.nan, np.inf
    x, w = stored(xv, fmt), stored(wv, fmt)
    y = torch.empty(T, m, device=DEV)
    matmul(x, w, fmt, n, y)
    bad = torch.isnan(y.cpu())
    want = torch.zeros(T, m, dtype=torch.bool)
    want[3], want[:, 77] = True, True
    assert torch.equal(bad, want)


def test_matmul_strided_output_and_untouched_surroundings():
    rng = np.random.default_rng(10)
    T, m, n = 67, 131, 320
    x, w = stored(rng.standard_normal((T, n)), NV), stored(rng.standard_normal((m, n)), NV)
    for dt in (torch.bfloat16, torch.float32):
        big = torch.full((T + 2, m + 5), 9.0, dtype=dt, device=DEV)
        matmul(x, w, NV, n, big[1:-1, 3:-2])
        y = torch.empty(T, m, dtype=dt, device=DEV)
        matmul(x, w, NV, n, y)
        assert torch.equal(big[1:-1, 3:-2], y)
        big[1:-1, 3:-2] = 9.0
        assert (big == 9.0).all()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("xdt,dt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                    (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("T,m,n", [(1, 1, 1), (1, 4096, 4096), (2, 130, 33), (3, 257, 1000), (5, 64, 28672), (8, 513, 2048),
                                   (9, 100, 4095), (16, 1000, 768), (16, 17, 20000)])
def test_matvec_matches_oracle(fmt, xdt, dt, T, m, n):
    rng = np.random.default_rng(T + m + n)
    x = torch.from_numpy(rng.standard_normal((T, n)).astype(np.float32)).to(xdt)
    w = stored(0.02 * rng.standard_normal((m, n)), fmt)
    y = torch.full((T, m), float("nan"), dtype=dt, device=DEV)
    kq.kronq_fp4_matvec(x.to(DEV), w[0], w[1], fmt, y, wg=w[2])
    check(y, *fp4.product(x.double().numpy(), w[3], None, g_of(w)), n)


@pytest.mark.parametrize("xdt", [torch.bfloat16, torch.float32])
def test_matvec_extreme_tokens(xdt):
    # tokens near the type's largest and smallest values, next to a NaN one
    rng = np.random.default_rng(11)
    n, m = 512, 96
    x = rng.standard_normal((4, n)).astype(np.float32)
    x[0] *= 1e34
    x[1] *= 1e-36
    x[2, 7] = np.nan
    xt = torch.from_numpy(x).to(xdt)
    w = stored(rng.standard_normal((m, n)), MX)
    y = torch.empty(4, m, device=DEV)
    kq.kronq_fp4_matvec(xt.to(DEV), w[0], w[1], MX, y)
    y64, S = fp4.product(np.nan_to_num(xt.double().numpy()), w[3])
    got = y.double().cpu().numpy()
    assert np.isnan(got[2]).all()
    for t in (0, 1, 3):   # 2^-149 n: products below the smallest float32
        assert (np.abs(got[t] - y64[t]) <= tolerance(n, S[t], y64[t], torch.float32) + n * 2.0 ** -149).all()


@pytest.mark.parametrize("fmt", [MX, NV])
def test_matvec_nan_blocks_infinite_tokens_and_padding(fmt):
    rng = np.random.default_rng(18)
    n, m = 650, 90
    wv = rng.standard_normal((m, n))
    wv[7, 300], wv[11] = np.inf, 0.0
    w = stored(wv, fmt)
    nb = -(-n // fp4.BLOCK[fmt])
    w[0][:, n // 2:] = 0x77                      # what lies behind the row's data may be anything
    w[1][:, nb:] = 0xFF if fmt == MX else 0x7F
    x = rng.standard_normal((3, n)).astype(np.float32)
    x[1, 5] = np.inf
    y = torch.empty(3, m, device=DEV)
    kq.kronq_fp4_matvec(torch.from_numpy(x).to(DEV), w[0], w[1], fmt, y, wg=w[2])
    y = y.cpu()
    assert torch.isnan(y[:, 7]).all()
    col = torch.from_numpy(w[3][:, 5])
    for r in range(m):
        if r != 7:   # infinity times the weight's sign, NaN for a zero weight
            v = float(y[1, r])
            assert np.isnan(v) if col[r] == 0 else v == np.sign(float(col[r])) * np.inf
    rest = np.delete(np.arange(m), 7)
    y64, S = fp4.product(x[[0, 2]], w[3][rest], None, g_of(w))
    got = y.double().numpy()[[0, 2]][:, rest]
    assert (np.abs(got - y64) <= tolerance(n, S, y64, torch.float32)).all()


def test_matvec_strided_tokens_and_output():
    rng = np.random.default_rng(12)
    for fmt, n in ((NV, 333), (MX, 640)):
        big = torch.from_numpy(rng.standard_normal((12, n + 9)).astype(np.float32)).to(DEV)
        w = stored(rng.standard_normal((200, n)), fmt)
        for dt in (torch.float32, torch.bfloat16):
            x = big.to(dt)[::2, 5:5 + n]
            y, z = torch.empty(6, 200, device=DEV), torch.zeros(6, 207, device=DEV)
            kq.kronq_fp4_matvec(x, w[0], w[1], fmt, z[:, 3:203], wg=w[2])
            kq.kronq_fp4_matvec(x.contiguous(), w[0], w[1], fmt, y, wg=w[2])
            assert torch.equal(z[:, 3:203], y) and (z[:, :3] == 0).all() and (z[:, 203:] == 0).all()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes,m,n,pad", [
    ([5], 64, 64, 0), ([0, 0, 3], 130, 100, 2), ([1, 0, 300, 17, 0, 256, 64], 257, 512, 7), ([0, 0], 64, 64, 4),
    ([33] * 12, 96, 1025, 0), ([257, 1, 511], 600, 768, 1)])
def test_grouped_matches_oracle(fmt, dt, sizes, m, n, pad):
    rng = np.random.default_rng(sum(sizes) + m)
    E, T = len(sizes), sum(sizes) + pad
    x = stored(rng.standard_normal((T, n)), fmt)
    ws = [stored(0.02 * (e + 1) * rng.standard_normal((m, n)), fmt) for e in range(E)]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    y = torch.full((T, m), 5.0, dtype=dt, device=DEV)
    kq.kronq_fp4_grouped_matmul(x[0], x[1], dev(off), torch.stack([w[0] for w in ws]), torch.stack([w[1] for w in ws]),
                                fmt, n, y, xg=x[2], wg=torch.cat([w[2] for w in ws]) if fmt == NV else None)
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a < b:
            check(y[a:b], *fp4.product(x[3][a:b], ws[e][3], g_of(x), g_of(ws[e])), n)
    assert (y[T - pad:] == 5.0).all() if pad else True


def test_grouped_offsets_out_of_range_are_taken_as_the_nearest():
    rng = np.random.default_rng(13)
    E, T, m, n = 4, 50, 70, 128
    x = stored(rng.standard_normal((T, n)), MX)
    ws = [stored(rng.standard_normal((m, n)), MX) for _ in range(E)]
    wc, wsc = torch.stack([w[0] for w in ws]), torch.stack([w[1] for w in ws])
    for off in ([-7, 20, 10, 90, 60], [3, 3, 3, 3, 3], [60, 70, 80, 90, 100], [5, 2 ** 31 - 1, -2 ** 31, 9, 1]):
        y = torch.full((T, m), 5.0, device=DEV)
        kq.kronq_fp4_grouped_matmul(x[0], x[1], dev(np.array(off, np.int32)), wc, wsc, MX, n, y)
        b = fp4.group_bounds(off, T)
        want = np.full((T, m), 5.0)
        S = np.zeros((T, m))
        for e in range(E):
            if b[e] < b[e + 1]:
                want[b[e]:b[e + 1]], S[b[e]:b[e + 1]] = fp4.product(x[3][b[e]:b[e + 1]], ws[e][3])
        check(y, want, S, n)


def test_many_experts_some_empty():
    rng = np.random.default_rng(14)
    E, m, n = 1024, 32, 64
    sizes = rng.integers(0, 3, size=E)
    T = int(sizes.sum())
    x = stored(rng.standard_normal((T, n)), NV)
    w = stored(rng.standard_normal((E * m, n)), NV)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    y = torch.empty(T, m, device=DEV)
    g = torch.linspace(0.5, 2.0, E, device=DEV)
    kq.kronq_fp4_grouped_matmul(x[0], x[1], dev(off), w[0].view(E, m, -1), w[1].view(E, m, -1), NV, n, y, xg=x[2], wg=g)
    who = np.repeat(np.arange(E), sizes)
    wv = w[3].reshape(E, m, n)[who]
    f = g_of(x) * g.double().cpu().numpy()[who][:, None]
    check(y, np.einsum("tn,tmn->tm", x[3], wv) * f, np.einsum("tn,tmn->tm", np.abs(x[3]), np.abs(wv)) * f, n)


# ------------------------------------------------------------ together, streams, graphs
def test_quantised_layer_as_served():
    """Weights of a rotated layer quantised once, then a prompt (quantised
    tokens) and a decode step (full-precision token) through them, with the
    BiIP rotation on both sides; the calls captured and replayed."""
    torch.manual_seed(0)
    m, n, T = 384, 512, 96
    W = 0.02 * torch.randn(m, n, device=DEV)
    X = torch.randn(T, n, device=DEV)
    HX, HG = X.T @ X, torch.eye(m, device=DEV)
    Wt, d_in, d_out = torch.empty(m, n, device=DEV), torch.empty(n, device=DEV), torch.empty(m, device=DEV)
    kq.kronq_biip_forward(W, Wt, HX, HG, 3, 0.25, "full", d_in, d_out)
    wc = torch.empty(m, kq.kronq_fp4_code_row_bytes(n), dtype=torch.uint8, device=DEV)
    ws = torch.empty(m, kq.kronq_fp4_scale_row_bytes(NV, n), dtype=torch.uint8, device=DEV)
    wg, deq = torch.empty(1, device=DEV), torch.empty_like(Wt)
    kq.kronq_fp4_quantize(Wt, NV, wc, ws, gscale=wg, deq=deq)
    # unrotated weights from the quantised ones: off by the formats' error
    What = deq.clone()
    kq.kronq_biip_inverse(What, 3, "full", d_in, d_out)
    assert (What - W).norm() < 0.2 * W.norm()
    xc = torch.empty(T, wc.shape[1], dtype=torch.uint8, device=DEV)
    xs = torch.empty(T, ws.shape[1], dtype=torch.uint8, device=DEV)
    xg, xd, y, y1 = torch.empty(1, device=DEV), torch.empty_like(X), torch.empty(T, m, device=DEV), torch.empty(1, m, device=DEV)
    qws = kq.workspace(kq.kronq_fp4_quantize_workspace_bytes(T, n, NV), DEV)
    mws = kq.workspace(max(kq.kronq_fp4_matmul_workspace_bytes(T, m, n, NV), kq.kronq_fp4_matvec_workspace_bytes(1, m, n, NV)), DEV)

    def step():
        kq.kronq_fp4_quantize(X, NV, xc, xs, gscale=xg, deq=xd, ws=qws)
        kq.kronq_fp4_matmul(xc, xs, wc, ws, NV, n, y, xg=xg, wg=wg, ws=mws)
        kq.kronq_fp4_matvec(X[-1:], wc, ws, NV, y1, wg=wg, ws=mws)

    def right():
        y64, S = fp4.product(xd.double().cpu().numpy(), deq.double().cpu().numpy())
        # xd and deq are rounded to float32 once: 2^-24 each
        assert (np.abs(y.double().cpu().numpy() - y64) <= tolerance(n, S, y64, y.dtype)).all()
        y64, S = fp4.product(X[-1:].double().cpu().numpy(), deq.double().cpu().numpy())
        assert (np.abs(y1.double().cpu().numpy() - y64) <= tolerance(n, S, y64, y.dtype)).all()

    step()
    right()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    right()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        X.copy_(torch.randn(T, n, device=DEV) * (k + 1))
        y.fill_(float("nan")), y1.fill_(float("nan"))
        graph.replay()
        right()
    assert kq.kronq_device_status() == 0


def test_calls_on_two_streams_at_once():
    rng = np.random.default_rng(15)
    jobs = []
    for T, m, n, fmt in ((300, 700, 1024, NV), (40, 1100, 4096, MX)):
        x, w = stored(rng.standard_normal((T, n)), fmt), stored(rng.standard_normal((m, n)), fmt)
        want = torch.empty(T, m, device=DEV)
        matmul(x, w, fmt, n, want)
        jobs.append((x, w, fmt, n, want, torch.empty_like(want), torch.cuda.Stream(),
                     kq.workspace(kq.kronq_fp4_matmul_workspace_bytes(T, m, n, fmt), DEV)))
    torch.cuda.synchronize()
    for _ in range(20):
        for x, w, fmt, n, _, y, s, ws in jobs:
            matmul(x, w, fmt, n, y, ws=ws, stream=s)
    torch.cuda.synchronize()
    for job in jobs:
        assert torch.equal(job[5], job[4])


def test_scratch_of_a_call_belongs_to_its_stream(monkeypatch):
    """A workspace that a call allocates is freed when the call returns: on
    another stream than the call's it could be handed out while in use."""
    rng = np.random.default_rng(19)
    T, m, n = 16, 256, 14336
    x, w = stored(rng.standard_normal((T, n)), NV), stored(rng.standard_normal((m, n)), NV)
    xf = torch.randn(T, n, device=DEV)
    side, at, make = torch.cuda.Stream(), [], kq.workspace

    def spy(nbytes, device="cuda"):
        at.append(torch.cuda.current_stream().cuda_stream)
        return make(nbytes, device)

    want, y = torch.empty(2, T, m, device=DEV), torch.empty(2, T, m, device=DEV)
    matmul(x, w, NV, n, want[0])
    kq.kronq_fp4_matvec(xf, w[0], w[1], NV, want[1], wg=w[2])
    torch.cuda.synchronize()
    monkeypatch.setattr(kq, "workspace", spy)
    g = torch.empty(1, device=DEV)
    codes, scales = torch.empty_like(x[0]), torch.empty_like(x[1])
    side.wait_stream(torch.cuda.current_stream())
    matmul(x, w, NV, n, y[0], stream=side)
    kq.kronq_fp4_matvec(xf, w[0], w[1], NV, y[1], wg=w[2], stream=side)
    kq.kronq_fp4_quantize(xf, NV, codes, scales, gscale=g, stream=side)
    assert at == [side.cuda_stream] * 3
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_repeats_are_bitwise_equal():
    rng = np.random.default_rng(16)
    x, w = stored(rng.standard_normal((33, 4096)), NV), stored(rng.standard_normal((520, 4096)), NV)
    ys = [torch.empty(33, 520, device=DEV) for _ in range(6)]
    vs = [torch.empty(4, 520, device=DEV) for _ in range(6)]
    xf = torch.randn(4, 4096, device=DEV)
    for y, v in zip(ys, vs):
        matmul(x, w, NV, 4096, y)
        kq.kronq_fp4_matvec(xf, w[0], w[1], NV, v, wg=w[2])
    assert all(torch.equal(y, ys[0]) for y in ys) and all(torch.equal(v, vs[0]) for v in vs)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,m,n", [(40, 300, 20000), (257, 200, 9000), (1, 256, 40000), (64, 1030, 8224)])
def test_matmul_with_split_columns(fmt, dt, T, m, n):
    assert kq.kronq_fp4_matmul_workspace_bytes(T, m, n, fmt) > 0
    rng = np.random.default_rng(T + n)
    x, w = stored(rng.standard_normal((T, n)), fmt), stored(0.02 * rng.standard_normal((m, n)), fmt)
    big = torch.full((T, m + 3), 9.0, dtype=dt, device=DEV)
    matmul(x, w, fmt, n, big[:, 1:-2])
    check(big[:, 1:-2], *fp4.product(x[3], w[3], g_of(x), g_of(w)), n)
    assert (big[:, 0] == 9.0).all() and (big[:, -2:] == 9.0).all()


@pytest.mark.parametrize("fmt, dt, T, m, n", [
    (NV, torch.float32, 5, 64, 20000), (MX, torch.bfloat16, 300, 300, 8191), (NV, torch.bfloat16, 100, 1000, 4095),
    (MX, torch.float32, 17, 1100, 4352)])
def test_matmul_in_many_short_parts(fmt, dt, T, m, n):
    parts = kq.kronq_fp4_matmul_workspace_bytes(T, m, n, fmt) // (T * m * 4)
    assert parts >= 4
    rng = np.random.default_rng(T + n + m)
    x, w = stored(rng.standard_normal((T, n)), fmt), stored(0.02 * rng.standard_normal((m, n)), fmt)
    out = torch.full((T + 1, m), 9.0, dtype=dt, device=DEV)
    matmul(x, w, fmt, n, out[:T])
    check(out[:T], *fp4.product(x[3], w[3], g_of(x), g_of(w)), n)
    assert (out[T] == 9.0).all()


@pytest.mark.parametrize("T", [1, 4, 11, 16])
@pytest.mark.parametrize("xdt", [torch.bfloat16, torch.float32])
def test_matvec_ranges_within_a_token(T, xdt):
    # spans of 128 columns whose values differ by more than fp16 parts cover,
    # next to plain ones; E8M0 scales beyond the fp16 range
    rng = np.random.default_rng(17 + T)
    n, m = 1300, 200
    x = rng.standard_normal((T, n)).astype(np.float32)
    x[0, 130:140] *= 1e-12
    x[T - 1, 300] = 1e20
    x[T // 2, 600:728] = 0.0
    x[0, 1290] = 1e-40
    w = 0.02 * rng.standard_normal((m, n))
    w[3, 256:288] *= 1e-15
    w[5, 640:672] *= 1e12
    xt = torch.from_numpy(x).to(xdt)
    for fmt in (MX, NV):
        q = stored(w, fmt)
        y = torch.empty(T, m, device=DEV)
        kq.kronq_fp4_matvec(xt.to(DEV), q[0], q[1], fmt, y, wg=q[2])
        y64, S = fp4.product(xt.double().numpy(), q[3], None, g_of(q))
        # 2^-149: products below the smallest float32
        assert (np.abs(y.double().cpu().numpy() - y64) <= tolerance(n, S, y64, torch.float32) + n * 2.0 ** -149).all()


def test_matvec_loud_column_with_zero_weights():
    # a column 2^40 times the others whose weights are all zero: the others count in full
    n, m = 256, 64
    w = torch.randn(m, n, dtype=torch.float64, generator=torch.Generator().manual_seed(3)).numpy()
    w[:, 17] = 0.0
    x = np.ones((2, n), np.float32)
    x[:, 17] = 2.0 ** 40
    for fmt in (MX, NV):
        for xdt in (torch.bfloat16, torch.float32):
            q = stored(w, fmt)
            y = torch.empty(2, m, device=DEV)
            kq.kronq_fp4_matvec(torch.from_numpy(x).to(xdt).to(DEV), q[0], q[1], fmt, y, wg=q[2])
            check(y, *fp4.product(x, q[3], None, g_of(q)), n)


def test_offsets_beyond_32_bits():
    """Arrays of more than 2^32 bytes and elements: each call's last rows equal
    those of the same call on these rows alone."""
    rows, n = 70000, 65536
    x = torch.empty(rows, n, dtype=torch.bfloat16, device=DEV).normal_()
    c = torch.empty(rows, kq.kronq_fp4_code_row_bytes(n), dtype=torch.uint8, device=DEV)
    s = torch.empty(rows, kq.kronq_fp4_scale_row_bytes(NV, n), dtype=torch.uint8, device=DEV)
    g = torch.full((1,), 0.002, device=DEV)
    kq.kronq_fp4_quantize(x, NV, c, s, gscale=g, gscale_given=True, deq=x)
    tail = x[-5:].clone()
    x.zero_()
    kq.kronq_fp4_dequantize(c, s, NV, x, gscale=g)
    assert torch.equal(x[-5:], tail) and bool(torch.isfinite(tail).all()) and float(tail.float().std()) > 0.5
    del x
    # the last rows' product with two tokens, alone and among all rows
    xf = torch.randn(2, n, device=DEV)
    y, z = torch.empty(2, rows, device=DEV), torch.empty(2, 64, device=DEV)
    kq.kronq_fp4_matvec(xf, c, s, NV, y, wg=g)
    kq.kronq_fp4_matvec(xf, c[-64:], s[-64:], NV, z, wg=g)
    # the columns may be split otherwise: (n / 16 + 4) 2^-22 of sum |x w|, whose mean is n 0.8 0.8
    assert float((y[:, -64:] - z).abs().max()) < (n / 16 + 4) * 2.0 ** -22 * n
    # two experts, the second's rows beyond 2^31 bytes of codes
    xc, xs = c[:3].clone(), s[:3].clone()
    off = torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV)
    gg = torch.ones(2, device=DEV)
    out = torch.empty(3, rows // 2, device=DEV)
    kq.kronq_fp4_grouped_matmul(xc, xs, off, c.view(2, rows // 2, -1), s.view(2, rows // 2, -1), NV, n, out, xg=g, wg=gg)
    want = torch.empty(3, 64, device=DEV)
    kq.kronq_fp4_matmul(xc, xs, c[-64:], s[-64:], NV, n, want, xg=g, wg=gg[:1])
    assert float((out[1:, -64:] - want[1:]).abs().max()) < (n / 16 + 4) * 2.0 ** -22 * n * 500 * 0.002
    del out, c, s
    # an output of more than 2^31 elements
    T, m, n = 66000, 34000, 64
    wc = torch.randint(0, 256, (m, 32), dtype=torch.uint8, device=DEV)
    xc = torch.randint(0, 256, (T, 32), dtype=torch.uint8, device=DEV)
    one = torch.full((m, 16), 127, dtype=torch.uint8, device=DEV)
    ones = torch.full((T, 16), 127, dtype=torch.uint8, device=DEV)
    y = torch.empty(T, m, dtype=torch.bfloat16, device=DEV)
    kq.kronq_fp4_matmul(xc, ones, wc, one, MX, n, y)
    z = torch.empty(9, m, dtype=torch.bfloat16, device=DEV)
    kq.kronq_fp4_matmul(xc[-9:], ones[-9:], wc, one, MX, n, z)
    assert torch.equal(y[-9:], z)


def test_first_call_inside_a_capture():
    """In a process of its own, the first 4-bit calls of all are captured ones."""
    import subprocess
    import sys
    code = """
import torch
import post_quantization_kronq_b200 as kq
d = "cuda"
x = torch.randn(24, 512, device=d); w = torch.randn(96, 512, device=d)
q = lambda r, b: torch.zeros(r, b, dtype=torch.uint8, device=d)
xc, xs, wc, ws = q(24, 256), q(24, 16), q(96, 256), q(96, 16)
y, v, dx, dw = torch.zeros(24, 96, device=d), torch.zeros(3, 96, device=d), torch.empty_like(x), torch.empty_like(w)
off = torch.tensor([0, 24], dtype=torch.int32, device=d)
z = torch.zeros(24, 96, device=d)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    kq.kronq_fp4_quantize(x, kq.MXFP4, xc, xs, deq=dx)
    kq.kronq_fp4_quantize(w, kq.MXFP4, wc, ws, deq=dw)
    kq.kronq_fp4_matmul(xc, xs, wc, ws, kq.MXFP4, 512, y)
    kq.kronq_fp4_grouped_matmul(xc, xs, off, wc[None], ws[None], kq.MXFP4, 512, z)
    kq.kronq_fp4_matvec(x[:3], wc, ws, kq.MXFP4, v)
g.replay()
torch.cuda.synchronize()
assert torch.equal(y, z)
assert (y - dx @ dw.T).abs().max() < 1e-2 and (v - x[:3] @ dw.T).abs().max() < 1e-2
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=__file__.rsplit("/", 2)[0])
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_expanded_rows_are_refused():
    c = torch.zeros(4, 32, dtype=torch.uint8, device=DEV)
    s = torch.zeros(4, 16, dtype=torch.uint8, device=DEV)
    x = torch.zeros(1, 64, device=DEV).expand(4, 64)
    for call in (lambda: kq.kronq_fp4_quantize(x, MX, c, s), lambda: kq.kronq_fp4_dequantize(c, s, MX, x),
                 lambda: kq.kronq_fp4_matvec(x, c, s, MX, torch.zeros(4, 4, device=DEV)),
                 lambda: kq.kronq_fp4_matmul(c, s, c, s, MX, 64, torch.zeros(1, 4, device=DEV).expand(4, 4))):
        with pytest.raises(kq.KronqError):
            call()


def test_python_refusals_on_the_device():
    c = torch.zeros(4, 32, dtype=torch.uint8, device=DEV)
    s = torch.zeros(4, 16, dtype=torch.uint8, device=DEV)
    x = torch.zeros(4, 64, device=DEV)
    with pytest.raises(ValueError):
        kq.kronq_fp4_quantize(x, NV, c, s)                                  # no tensor scale
    with pytest.raises(ValueError):
        kq.kronq_fp4_quantize(x, MX, c[:, :16], s)                          # row bytes
    with pytest.raises(ValueError):
        kq.kronq_fp4_quantize(x.T, MX, c, s)                                # rows not dense
    with pytest.raises(TypeError):
        kq.kronq_fp4_quantize(x.half(), MX, c, s)
    with pytest.raises(ValueError):
        kq.kronq_fp4_quantize(x, MX, c, s, deq=x.bfloat16())
    with pytest.raises(ValueError):
        kq.kronq_fp4_matmul(c, s, c, s, MX, 64, torch.empty(3, 4, device=DEV))
    with pytest.raises(ValueError):
        kq.kronq_fp4_grouped_matmul(c, s, torch.zeros(2, device=DEV), c[None], s[None], MX, 64, x)
    with pytest.raises(kq.KronqError):
        kq.kronq_fp4_matvec(torch.zeros(17, 64, device=DEV), c, s, MX, torch.zeros(17, 4, device=DEV))
