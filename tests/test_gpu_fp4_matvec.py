"""kronq_fp4_matvec: a result depends on its own token and row (and the sizes),
whatever stands beside them in the call."""
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


def weights(rng, m, n, fmt):
    codes, sb, g = fp4.quantize(0.02 * rng.standard_normal((m, n)), fmt)
    c, s = fp4.store(codes, sb, fmt)
    return dev(c), dev(s), None if fmt == MX else torch.tensor([float(g)], device=DEV)


def matvec(x, w, fmt):
    y = torch.full((x.shape[0], w[0].shape[0]), float("nan"), device=DEV)
    kq.kronq_fp4_matvec(x, w[0], w[1], fmt, y, wg=w[2])
    return y.view(torch.int32)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("xdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,m,n", [(2, 200, 1300), (7, 97, 20000), (16, 200, 1300), (11, 33, 9000)])
def test_a_token_does_not_depend_on_the_others(fmt, xdt, T, m, n):
    rng = np.random.default_rng(T)
    w = weights(rng, m, n, fmt)
    x = dev(rng.standard_normal((T, n)).astype(np.float32)).to(xdt)
    want = matvec(x, w, fmt)
    for odd in (float("nan"), float("inf"), 1e-30, 1e38):
        for j in (0, T - 1):
            z = x.clone()
            z[j, ::100] = odd
            keep = torch.arange(T, device=DEV) != j
            assert torch.equal(matvec(z, w, fmt)[keep], want[keep]), (odd, j)


@pytest.mark.parametrize("xdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,m,n", [(1, 100, 1300), (3, 90, 20000), (16, 100, 1300)])
def test_a_row_does_not_depend_on_its_neighbours(xdt, T, m, n):
    rng = np.random.default_rng(m + T)
    c, s, _ = weights(rng, m, n, MX)
    x = dev(rng.standard_normal((T, n)).astype(np.float32)).to(xdt)
    want = matvec(x, (c, s, None), MX)
    for byte in (255, 3, 200, 0):
        for r in (0, 21, m - 1):
            s2 = s.clone()
            s2[r, : -(-n // 32) : 7] = byte
            keep = torch.arange(m, device=DEV) != r
            assert torch.equal(matvec(x, (c, s2, None), MX)[:, keep], want[:, keep]), (byte, r)


@pytest.mark.parametrize("xdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 5, 16])
def test_blocks_of_zeros(xdt, T):
    """The quantiser gives a block of zeros the lowest scale: the result is that
    under any other scale, and NaN under NaN."""
    rng = np.random.default_rng(20 + T)
    m, n = 70, 1300
    w = 0.02 * rng.standard_normal((m, n))
    zero = rng.random((m, -(-n // 32))) < 0.2
    zero[13] = True
    w[np.repeat(zero, 32, axis=1)[:, :n]] = 0.0
    codes, sb, _ = fp4.quantize(w, MX)
    assert (sb[zero] == 0).all()
    x = dev(rng.standard_normal((T, n)).astype(np.float32)).to(xdt)
    got = []
    for byte in (0, 127, 254):
        c, s = fp4.store(codes, np.where(zero, byte, sb).astype(np.uint8), MX)
        got.append(matvec(x, (dev(c), dev(s), None), MX))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    assert not got[0][:, 13].any()
    sb[13, 5] = 255
    c, s = fp4.store(codes, sb, MX)
    y = matvec(x, (dev(c), dev(s), None), MX).view(torch.float32)
    assert bool(torch.isnan(y[:, 13]).all()) and int(torch.isnan(y).sum()) == T


@pytest.mark.parametrize("T", [1, 16])
def test_blocks_of_zeros_cost_no_more_than_others(T):
    """One zero block in a hundred, as pruned weights and padded rows have:
    about the time of dense weights (2.6 to 33 times it when such blocks were
    computed one weight at a time)."""
    m, n = 28672, 8192
    x = torch.randn(T, n, device=DEV).to(torch.bfloat16)
    y = torch.empty(T, m, dtype=torch.bfloat16, device=DEV)
    W = 0.02 * torch.randn(m, n, device=DEV)
    ws = kq.workspace(kq.kronq_fp4_matvec_workspace_bytes(T, m, n, MX), DEV)
    calls = []
    for share in (0.0, 0.01):
        keep = torch.rand(m, n // 32, device=DEV) >= share
        c = torch.empty(m, n // 2, dtype=torch.uint8, device=DEV)
        s = torch.empty(m, n // 32, dtype=torch.uint8, device=DEV)
        kq.kronq_fp4_quantize((W.view(m, -1, 32) * keep[:, :, None]).view(m, n), MX, c, s)
        calls.append(lambda c=c, s=s: kq.kronq_fp4_matvec(x, c, s, MX, y, ws=ws))
    times = [[], []]
    for call in calls:
        call()
    for _ in range(9):
        for call, t in zip(calls, times):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                call()
            b.record()
            b.synchronize()
            t.append(a.elapsed_time(b))
    dense, zeros = (sorted(t)[4] for t in times)
    assert zeros < 1.5 * dense


@pytest.mark.parametrize("xdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 3, 16])
@pytest.mark.parametrize("byte", [0, 1, 60, 200, 251, 252, 253, 254])
def test_e8m0_scales_at_the_ends(xdt, T, byte):
    """Weights up to 6 * 2^127, beyond float32 themselves: whole tokens times a
    power of two bring the products back to whole numbers, which sum exactly.
    A token that is zero under such weights takes nothing from them."""
    rng = np.random.default_rng(byte)
    m, n = 50, 700
    codes = rng.integers(0, 16, size=(m, n)).astype(np.uint8)
    sb = np.full((m, -(-n // 32)), byte, np.uint8)
    c, s = fp4.store(codes, sb, MX)
    k = rng.integers(-8, 9, size=(T, n)).astype(np.float64)
    x = k * 2.0 ** min(max(127 - byte, -120), 120)   # tokens are normal numbers
    y64 = x @ fp4.values(codes, sb, MX).T
    y = matvec(dev(x.astype(np.float32)).to(xdt), (dev(c), dev(s), None), MX).view(torch.float32)
    assert np.array_equal(y.double().cpu().numpy(), y64)
    if T > 1:
        x[1] = 0.0
        y = matvec(dev(x.astype(np.float32)).to(xdt), (dev(c), dev(s), None), MX).view(torch.float32)
        assert not y[1].any()
