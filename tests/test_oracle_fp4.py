"""The 4-bit oracle against the formats' definitions, by exhaustive search in
exact rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fp4


def _e2m1_exact(x, s):
    """Nearest E2M1 index of |x| / s by Fractions, ties to even."""
    y = abs(Fraction(float(x))) / s
    d = [abs(y - Fraction(float(v))) for v in fp4.E2M1]
    best = min(d)
    near = [i for i in range(8) if d[i] == best]
    return near[0] if len(near) == 1 else next(i for i in near if i % 2 == 0)


def test_e4m3_table_is_torchs():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp4.e4m3_table(), t)


@pytest.mark.parametrize("g", [1.0, 2.0 ** -7, 0.0123, 3.3e-5])
def test_nv_decisions_are_those_of_exact_arithmetic(g):
    rng = np.random.default_rng(0)
    g = np.float32(g)
    s0 = fp4.e4m3_table()[rng.integers(1, 127, size=40)]
    # values on and next to the borders under some block scale
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = np.float32(mids[rng.integers(0, 7, size=(40, 16))] * s0[:, None] * np.float64(g))
    x = np.nextafter(x, np.where(rng.random(x.shape) < 0.5, np.float32(0), np.float32(np.inf)) * 1,
                     where=rng.random(x.shape) < 0.5, out=x.copy())
    codes, sb, _ = fp4.quantize(x, fp4.NV, g)
    table = [Fraction(float(v)) for v in fp4.e4m3_table()]
    for r in range(x.shape[0]):
        t = Fraction(float(np.abs(x[r]).max())) / (6 * Fraction(float(g)))
        d = [abs(min(t, table[-1]) - v) for v in table]
        near = [i for i in range(127) if d[i] == min(d)]
        want = near[0] if len(near) == 1 else next(i for i in near if i % 2 == 0)
        assert sb[r, 0] == want
        s = table[want] * Fraction(float(g))
        for j in range(16):
            assert codes[r, j] & 7 == (_e2m1_exact(x[r, j], s) if s else 0)


def test_mx_scale_and_codes():
    x = np.zeros((4, 40), np.float32)
    x[0, 0], x[0, 1], x[0, 2] = 6.0, 5.0, -2.5        # scale 1; ties 5 -> 4, 2.5 -> 2
    x[1, 35] = 7.9                                    # saturates at 6
    x[2, :] = 2.0 ** -140                             # below the smallest scale's border
    codes, sb, g = fp4.quantize(x, fp4.MX)
    assert g is None and sb[0, 0] == 127 and sb[1, 0] == 0 and sb[1, 1] == 127 and sb[2, 0] == 0
    assert list(codes[0, :3]) == [7, 6, 8 + 4] and codes[1, 35] == 7 and codes[2].max() == 0


def test_non_finite_blocks_and_tensor_scale():
    x = np.ones((1, 48), np.float32)
    x[0, 3], x[0, 20] = np.nan, -np.inf
    codes, sb, g = fp4.quantize(x, fp4.NV)
    assert list(sb[0, :2]) == [127, 127] and codes[0, :32].max() == 0 and g == np.float32(1 / 2688)
    v = fp4.values(codes, sb, fp4.NV)
    assert np.isnan(v[0, :32]).all() and np.isfinite(v[0, 32:]).all()
    assert fp4.tensor_scale(np.zeros((2, 2))) == 1 and fp4.tensor_scale(np.full((1, 1), 1e-44)) == np.float32(2.0 ** -126)


@pytest.mark.parametrize("fmt", [fp4.MX, fp4.NV])
def test_relative_error_of_a_block(fmt):
    # half a step of E2M1 next to 6 is 1/6 of the block's maximum at most; the
    # block scale adds its own half step (NVFP4) or the saturation of (6, 8) (MXFP4)
    x = np.random.default_rng(1).standard_normal((64, 256)).astype(np.float32)
    codes, sb, g = fp4.quantize(x, fmt)
    v = fp4.values_f32(codes, sb, fmt, g)
    bs = fp4.BLOCK[fmt]
    amax = np.abs(x).reshape(64, -1, bs).max(axis=2)
    err = np.abs(x - v).reshape(64, -1, bs).max(axis=2)
    assert (err <= amax * (0.25 if fmt == fp4.MX else 1 / 6 + 1 / 16)).all()


def test_store_layout():
    codes = (np.arange(37)[None, :] % 16).astype(np.uint8)
    c, s = fp4.store(codes, np.arange(1, 4, dtype=np.uint8)[None, :], fp4.NV)
    assert c.shape == (1, 32) and s.shape == (1, 16)
    assert c[0, 0] == 0x10 and c[0, 18] == 0x04 and c[0, 19:].max() == 0 and list(s[0, :4]) == [1, 2, 3, 0]


def test_group_bounds():
    assert list(fp4.group_bounds([0, 4, 2, 9, 7], 6)) == [0, 4, 4, 6, 6]
    assert list(fp4.group_bounds([-3, 4], 6)) == [0, 4]
