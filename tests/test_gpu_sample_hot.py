"""GPU tests of cb_sample where numbers near the end of fp32 meet in it: the highest temperatures and logits of their size.  The
tolerances are those of tests/test_gpu_sample.py.  At temperatures above 2^120 the remainder of 256 log2(e) / T is below the normal numbers
and off by up to 2^-150, which 2^128 makes 2^-22 in 256ths: 2^-30.5 of a weight, inside the 2^-29 of a probability and the 2^-30 of
a border that are allowed there."""
import numpy as np
import pytest

from test_gpu_sample import check

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


@pytest.mark.parametrize("v", [700, 40000])
def test_highest_temperatures(cb, v):
    n = 24
    rng = np.random.default_rng(v)
    t = np.concatenate([rng.uniform(1.2e38, 3.4e38, n - 8), [1e34, 1e35, 1e36, 1e37, 2e37, 5e37, 8e37, 1e38]]).astype(np.float32)
    x = rng.uniform(-3.3e38, 3.3e38, (n, v)).astype(np.float32)
    x[n - 8:] = np.clip(rng.normal(size=(8, v)) * t[n - 8:, None], -3.4e38, 3.4e38)
    x = torch.from_numpy(x).cuda()
    u = rng.random(n)
    check(cb, x, u, t=t)
    check(cb, x, u, t=t, p=rng.uniform(0.05, 0.95, n))
    check(cb, x, u, t=t, k=np.full(n, 300), m=np.full(n, 0.2))
    check(cb, x, u, t=t, k=np.full(n, 20), p=np.full(n, 0.7))
    check(cb, -x.abs(), u, t=t, m=np.full(n, 0.3))


def test_min_p_whose_value_passes_fp32(cb):
    """The logit below which min-p keeps nothing lies beyond the lowest fp32 number when it is counted from 0, and still cuts: of tokens with
    2^-38 of the largest weight, min-p 2^-31 keeps none, and the last uniform number below 1 takes the only one that is left."""
    v, t, top = 128256, 1.6e37, 3.3e38
    low = top + t * np.log(2.0 ** -38)
    x = torch.full((4, v), low, device="cuda")
    x[:2, 0], x[2:, v - 1] = top, top
    u, m = np.array([1 - 2.0 ** -24, 0.0, 1 - 2.0 ** -24, 0.0]), np.array([2.0 ** -31, 2.0 ** -31, 2.0 ** -31, 2.0 ** -40])
    tokens, probs = check(cb, x, u, t=np.full(4, t), m=m, compared=0.75)       # (the last row's border is nearer than float64 sums tell)
    assert tokens.tolist() == [0, 0, v - 1, 0] and (probs[:3] == 1.0).all()


@pytest.mark.parametrize("v", [600, 30000])
def test_lowest_temperatures(cb, v):
    """Temperatures down to the smallest that is not greedy, with logits of their size, below the normal numbers among them, and with logits
    thousands of temperatures away from 0 or below anything that 2^32 leaves within fp32."""
    n = 24
    rng = np.random.default_rng(v)
    t = np.concatenate([10.0 ** rng.uniform(-37.9, -30, n - 2), [1.1754944e-38, 7.8e-31]]).astype(np.float32)
    x = (rng.normal(size=(n, v)) * 3 * t[:, None]).astype(np.float32)
    x[3:6] += np.float32(20000) * t[3:6, None]
    x[6:9, ::3] = -3e38
    x[9] -= np.float32(5000) * t[9]
    u = rng.random(n)
    x = torch.from_numpy(x).cuda()
    check(cb, x, u, t=t)
    check(cb, x, u, t=t, p=rng.uniform(0.05, 0.95, n))
    check(cb, x, u, t=t, k=np.full(n, 300), m=np.full(n, 0.2))
    check(cb, x, u, t=t, k=np.full(n, 20), p=np.full(n, 0.7))
    check(cb, x, u, t=t, k=np.full(n, v - 1), p=np.full(n, 0.99), m=np.full(n, 1e-4))
