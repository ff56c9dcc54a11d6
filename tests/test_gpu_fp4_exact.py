"""The 4-bit products on whole numbers: codes, and scales that are powers of two,
whose sums are whole multiples of a unit and fit float32's 24 bits in any order,
so that the products have to be equal to the float64 ones.  One code, scale or
column that is left out, taken twice or misplaced shows."""
import numpy as np
import pytest
import torch

import post_quantization_kronq_b200 as kq
from oracle import fp4

pytestmark = pytest.mark.gpu
DEV = "cuda"
MX, NV = kq.MXFP4, kq.NVFP4


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def whole(rng, rows, n, fmt):
    """(codes, scales, tensor scale, float64 values on the device): any code under scales of 2^-1 .. 2^1, another
    one in every block."""
    codes = rng.integers(0, 16, size=(rows, n)).astype(np.uint8)
    e = rng.integers(-1, 2, size=(rows, -(-n // fp4.BLOCK[fmt])))
    sb = ((127 + e) if fmt == MX else (7 + e) * 8).astype(np.uint8)
    c, s = fp4.store(codes, sb, fmt)
    return dev(c), dev(s), None if fmt == MX else torch.ones(1, device=DEV), dev(fp4.values(codes, sb, fmt))


def product(x, w):
    """X W^T in float64; values are multiples of 2^-2, so partial sums fit where sum |x w| is below 2^20."""
    assert float((x.abs() @ w.abs().T).max()) < 2.0 ** 20
    return x @ w.T


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("T,m,n", [(256, 512, 28672), (300, 700, 8192), (2048, 4096, 4096)])
def test_scales_of_both_halves_of_a_pair_in_every_repeat(fmt, T, m, n):
    """Rows 0 - 127 and 128 - 255 of a tile of W, and halves of its tokens, come
    by way of two SMs; one of them multiplies.  Long rows, so that every slot
    of scales is filled many times over, and many repeats."""
    rng = np.random.default_rng(n)
    x, w = whole(rng, T, n, fmt), whole(rng, m, n, fmt)
    want = product(x[3], w[3])
    y = torch.empty(T, m, device=DEV)
    ws = kq.workspace(kq.kronq_fp4_matmul_workspace_bytes(T, m, n, fmt), DEV)
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(60):
        y.fill_(float("nan"))
        kq.kronq_fp4_matmul(x[0], x[1], w[0], w[1], fmt, n, y, xg=x[2], wg=w[2], ws=ws)
        wrong += (y != want).sum()
    assert int(wrong) == 0
    assert kq.kronq_device_status() == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,m,n,split", [(100, 1000, 4095, True), (16, 300, 20000, True), (300, 5000, 512, False)])
def test_tensor_scales_far_apart(dt, T, m, n, split):
    """Tensor scales whose product is an ordinary number count as that number,
    also where a sum times one of them would leave float32's range."""
    rng = np.random.default_rng(T)
    x, w = whole(rng, T, n, NV), whole(rng, m, n, NV)
    assert (kq.kronq_fp4_matmul_workspace_bytes(T, m, n, NV) > 0) == split
    one, y = (torch.empty(T, m, dtype=dt, device=DEV) for _ in range(2))
    kq.kronq_fp4_matmul(x[0], x[1], w[0], w[1], NV, n, one, xg=x[2], wg=w[2])
    for a, b in ((-126, 100), (100, -126), (120, -100), (-100, 120)):
        ga, gb = torch.tensor([2.0 ** a], device=DEV), torch.tensor([2.0 ** b], device=DEV)
        kq.kronq_fp4_matmul(x[0], x[1], w[0], w[1], NV, n, y, xg=ga, wg=gb)
        assert torch.equal(y, one * 2.0 ** (a + b))


@pytest.mark.parametrize("T,m,n", [(130, 300, 1056), (20, 200, 8192)])
def test_e8m0_scales_at_the_ends(T, m, n):
    """Scales from 2^-127 to 2^127, those of tokens against those of weights:
    their product is 1 in every block, and the sums are whole."""
    rng = np.random.default_rng(n)
    xc, wc = (rng.integers(0, 16, size=(r, n)).astype(np.uint8) for r in (T, m))
    e = rng.integers(0, 255, size=(1, -(-n // 32)))
    e[0, :4] = 0, 254, 1, 253
    xq = fp4.store(xc, np.repeat(e, T, 0).astype(np.uint8), MX)
    wq = fp4.store(wc, np.repeat(254 - e, m, 0).astype(np.uint8), MX)
    one = np.full((1, e.shape[1]), 127, np.uint8)
    want = product(*(dev(fp4.values(c, np.repeat(one, len(c), 0), MX)) for c in (xc, wc)))
    y = torch.empty(T, m, device=DEV)
    kq.kronq_fp4_matmul(dev(xq[0]), dev(xq[1]), dev(wq[0]), dev(wq[1]), MX, n, y)
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,m,n", [(1, 256, 40001), (100, 1000, 4095), (300, 300, 8191), (17, 520, 20033)])
def test_split_columns(fmt, dt, T, m, n):
    assert kq.kronq_fp4_matmul_workspace_bytes(T, m, n, fmt) > 0
    rng = np.random.default_rng(n)
    x, w = whole(rng, T, n, fmt), whole(rng, m, n, fmt)
    y = torch.empty(T, m, dtype=dt, device=DEV)
    kq.kronq_fp4_matmul(x[0], x[1], w[0], w[1], fmt, n, y, xg=x[2], wg=w[2])
    assert torch.equal(y, product(x[3], w[3]).to(dt))


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes,m,n,pad", [([0, 200, 33, 0, 300, 1], 300, 4095, 3), ([64] * 9, 70, 545, 0), ([5, 7], 513, 28672, 2)])
def test_groups(fmt, dt, sizes, m, n, pad):
    rng = np.random.default_rng(n)
    E, T = len(sizes), sum(sizes) + pad
    x, w = whole(rng, T, n, fmt), whole(rng, E * m, n, fmt)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    y = torch.full((T, m), 5.0, dtype=dt, device=DEV)
    g = None if fmt == MX else 2.0 ** (torch.arange(E, device=DEV) % 3)
    kq.kronq_fp4_grouped_matmul(x[0], x[1], dev(off), w[0].view(E, m, -1), w[1].view(E, m, -1), fmt, n, y, xg=x[2], wg=g)
    want = torch.full((T, m), 5.0, dtype=torch.float64, device=DEV)
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        if off[e] < off[e + 1]:
            want[rows] = product(x[3][rows], w[3][e * m:(e + 1) * m]) * (1.0 if g is None else float(g[e]))
    assert torch.equal(y, want.to(dt))


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("xdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 2, 8, 9, 16])
@pytest.mark.parametrize("m,n", [(100, 28672), (33, 20001), (300, 1030), (5000, 130)])
def test_few_tokens(fmt, xdt, T, m, n):
    """Whole tokens: one in 64 has more bits than one fp16 part holds (float32), the others few."""
    rng = np.random.default_rng(T + n)
    w = whole(rng, m, n, fmt)
    if n > 20000 and xdt is torch.float32 and T > 8:
        assert kq.kronq_fp4_matvec_workspace_bytes(T, m, n, fmt) >= 16 * T * m * 4   # many slices
    big = 4095 if xdt is torch.float32 else 127
    k = np.where(rng.random((T, n)) < 1 / 64, rng.integers(-big, big + 1, size=(T, n)), rng.integers(-4, 5, size=(T, n)))
    x = dev(k.astype(np.float32)).to(xdt)
    # values of W are multiples of 2^-2: sums of these fit below 2^22
    assert float((x.double().abs() @ w[3].abs().T).max()) < 2.0 ** 22
    y = torch.empty(T, m, device=DEV)
    kq.kronq_fp4_matvec(x, w[0], w[1], fmt, y, wg=w[2])
    assert torch.equal(y.double(), x.double() @ w[3].T)
