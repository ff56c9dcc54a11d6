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
