"""GPU tests of how near rows that are rotated as they are appended come to exact rotation.

The frequency of a pair is the float64 number theta^(-2i / head_dim); its product with a position, as a fraction of a turn, is formed
here in integers of any length with 400 bits of 1 / (2 pi), so that the float64 result below is within 2^-50 of the pair's length
for every position (the fraction's, the sine's and the products' roundings)."""
import math

import numpy as np
import pytest

from test_gpu_kv8 import Case, f64, i32

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def cb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import cacheblend_selective_kv_gb300 as cbm
    return cbm


BITS = 400


def over_two_pi():
    """2^BITS / (2 pi), by Machin's formula."""
    one = 1 << (2 * BITS)

    def arctan_of_inverse(x):
        term, total, n, sign = one // x, 0, 1, 1
        while term:
            total += sign * (term // n)
            term //= x * x
            n, sign = n + 2, -sign
        return total
    pi = 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))
    return (one << BITS) // (2 * pi)


def angles(positions, theta, hd):
    """float64 angles [position][pair] within half a turn."""
    inverse, out = over_two_pi(), np.empty((len(positions), hd // 2))
    for i in range(hd // 2):
        m, e = math.frexp(math.pow(theta, -2.0 * i / hd))
        turn = (int(math.ldexp(m, 53)) * inverse) >> (53 - e)        # in 2^-BITS turns
        keep = turn >> (BITS - 160)                     # 160 bits are enough for a position of 32
        half = 1 << 159
        for j, p in enumerate(positions):
            out[j, i] = (((int(p) * keep + half) & ((1 << 160) - 1)) - half) / (1 << 160)
    return out * (2 * math.pi)


def turned(x, angle):
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = x[..., 0::2], x[..., 1::2]
    y = np.empty_like(x)
    y[..., 0::2], y[..., 1::2] = a * c - b * s, a * s + b * c
    return y


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1])
def test_rotation_at_far_positions(cb, far):
    """An fp32 q is off by at most 2.5e-7 of its pair's length at every position: cosine and sine by 1.266e-7 as a vector, over all phases of 32
    bits; the cut to those 1.5e-9; the frequency's 64 bits 0.7e-9; product and sum by 2^-24 of the length each."""
    n, hd, theta = 2048, 128, 1.5e4
    c = Case(cb, [n], H=1, G=2, hd=hd, P=64, dtype="f32", seed=17)
    q, q64 = c.values(n, 2, hd)
    k, _ = c.values(n, 1, hd)
    pos = c.rng.integers(-far - 1, far + 1, n)
    pos[:3] = far, -far - 1, far - 1
    out = c.cache.append(c.table, c.lens_t, q, k, k, theta, positions=i32(pos))
    torch.cuda.synchronize()
    y = turned(q64, angles(pos, theta, hd))
    length = np.sqrt(q64[..., 0::2] ** 2 + q64[..., 1::2] ** 2).repeat(2, axis=-1)
    off = np.abs(f64(out) - y) / length
    assert off.max() <= 2.5e-7, off.max()
    c.done()
