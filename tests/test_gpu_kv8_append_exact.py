"""GPU tests of the codes and scales of rows that are rotated as they are appended: those of exact rotation.

The frequency of a pair is the float64 number theta^(-2i / head_dim); its product with a position, as a fraction of a turn, is formed
here in integers of any length with 400 bits of 1 / (2 pi), so that the float64 result below is within 2^-50 of the pair's length
for every position (the fraction's, the sine's and the products' roundings).  The library turns what fp32 does not decide within 1e-13
of the pair's length, and within 2^31 2^-64 turns for the farthest positions (7e-10).  A value nearer than that to the middle between
two codes could fall to either side: none of the values here is (`margin` says how near one comes, and is asserted)."""
import math

import numpy as np
import pytest

import kv8_model as km
from test_gpu_kv8 import Case, f64, i32, starts_of

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


def margin(y, scale):
    """How near a value comes to the middle between two codes or to the largest of its scale, relative to its pair's length."""
    z = np.abs(y) / scale
    middles = np.concatenate([(km._POS[:-1] + km._POS[1:]) / 2, [km.F8_MAX]])
    at = np.clip(np.searchsorted(middles, z), 1, len(middles) - 1)
    near = np.minimum(np.abs(middles[at] - z), np.abs(middles[at - 1] - z))
    length = np.sqrt(z[..., 0::2] ** 2 + z[..., 1::2] ** 2).repeat(2, axis=-1)
    return near / np.maximum(length, 1e-300)


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


def same_k(c):
    """K's scales and codes against the model's (a zero of either sign is one value)."""
    assert np.array_equal(c.scales[:, 0].cpu().numpy(), c.model.scales[:, 0].astype(np.float32))
    got, want = km.VALUES[c.codes[:, 0].cpu().numpy()], km.VALUES[c.model.codes[:, 0]]
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    assert same.all(), (int((~same).sum()), np.argwhere(~same)[:5])


@pytest.mark.parametrize("n,hd,dtype,far", [(8192, 128, "bf16", None), (4096, 64, "f32", None), (2048, 128, "f32", 1 << 20), (2048, 64, "bf16", (1 << 31) - 1)])
def test_random_rows(cb, n, hd, dtype, far):
    """Every code and scale of a long prompt, at its rows' places, at positions of both signs up to 2^20, and at the farthest."""
    H, P = 4, 64
    c = Case(cb, [n], H=H, G=1, hd=hd, P=P, dtype=dtype, seed=n + hd)
    k, k64 = c.values(n, H, hd)
    pos = np.arange(n) if far is None else c.rng.integers(-far, far + 1, n)
    y = turned(k64, angles(pos, 5e5, hd))
    c.model.write(c.table_np, c.lens, y[None], k64[None], [0, n])
    used = c.model.scales[0, 0, c.table_np[0]].repeat(P, axis=0)                # [rows][H]
    m = margin(y, used[..., None])
    assert m[m > 0].min() > (2e-9 if far and far > 1 << 24 else 1e-12)         # (0: a row at position 0, which is not turned)
    c.cache.append(c.table, c.lens_t, None, k, k, 5e5, positions=None if far is None else i32(pos))
    torch.cuda.synchronize()
    same_k(c)
    c.done()


def bf16(x):
    """float64 numbers cut off to bf16."""
    return (np.asarray(x, np.float32).view(np.uint32) & 0xffff0000).view(np.float32).astype(np.float64)


def near_middles(rng, n, hd, dtype, angle):
    """Rows [n][1][hd] whose values, turned and at a scale of 1, lie next to the middle between two codes, small codes and values far below
    their pair's length among them; the first pair holds the scale at 1."""
    x = np.zeros((n, 1, hd))
    f = hd // 2
    if dtype == "f32":
        # turned back from the wanted values and rounded to fp32, which leaves them some 1e-8 of the pair's length away
        middles = (km._POS[:-1] + km._POS[1:])[:-8] / 2
        want = rng.choice(middles, (2, n, f)) * rng.choice([-1.0, 1.0], (2, n, f))
        c, s = np.cos(angle), np.sin(angle)
        x[:, 0, 0::2], x[:, 0, 1::2] = want[0] * c + want[1] * s, want[1] * c - want[0] * s
        x = x.astype(np.float32).astype(np.float64)
    else:
        # bf16 pairs of which one or the other turns out that near: found by trying
        for r in range(n):
            for i in range(1, f):
                a, b = bf16(rng.normal(size=(2, 4000)) * 2.0 ** rng.integers(-6, 7, 4000))
                c, s = np.cos(angle[r, i]), np.sin(angle[r, i])
                y = np.stack([a * c - b * s, a * s + b * c], axis=-1)
                m = np.where(np.abs(y).max(axis=-1) < 440, margin(y, 1.0).min(axis=-1), 1.0)
                m[m < 1e-11] = 1.0
                at = int(m.argmin())
                x[r, 0, 2 * i:2 * i + 2] = a[at], b[at]
    x[:, 0, :2] = 320.0, 0.0                             # its larger value is from 226 to 320
    return x


@pytest.mark.parametrize("dtype,hd,P,given", [("f32", 64, 16, None), ("f32", 128, 64, "both signs"), ("f32", 128, 256, "far"), ("bf16", 64, 32, "both signs")])
def test_values_next_to_a_middle(cb, dtype, hd, P, given):
    """Nearly every pair needs more than fp32: as whole blocks, as rows behind others in a block, whose codes are rounded to a scale that
    grows, and one row at a time."""
    rng = np.random.default_rng(hd + P)
    n = 3 * P if dtype == "f32" else 24
    pos = np.arange(n) if given is None else rng.integers(-4000, 4000, n) if given == "both signs" else rng.integers(-2 ** 31, 2 ** 31, n)
    angle = angles(pos, 1e4, hd)
    x = near_middles(rng, n, hd, dtype, angle)
    y = turned(x, angle)
    near = margin(y, 1.0).min(axis=(1, 2)) if given != "far" else np.full(n, 1.0)
    keep = near > 1e-12                                  # (rows with a value nearer than the library's 64 bits tell are left out)
    assert keep.mean() > 0.8
    n, pos, x, y = int(keep.sum()), pos[keep], x[keep], y[keep]
    if given == "far":
        z = margin(y, 1.0) > 2e-9                        # at the farthest positions a turn is known within 7e-10
        pairs = (z[..., 0::2] & z[..., 1::2]).repeat(2, axis=-1)
        x, y = np.where(pairs, x, 0.0), np.where(pairs, y, 0.0)
        assert pairs.mean() > 0.5
    c = Case(cb, [P // 2 + n, n], H=1, G=1, hd=hd, P=P, dtype=dtype, seed=5, spare=4)
    m = margin(y, 1.0)
    if dtype == "f32":
        assert (m[..., 2:] < 1e-7).mean() > 0.7          # that near fp32 decides by chance
    else:
        assert (m[..., 2:].reshape(n, -1, 2).min(axis=-1) < 3e-7).mean() > 0.1
    k = torch.from_numpy(x.astype(np.float32)).to(c.td).cuda()
    assert np.array_equal(f64(k), x)
    # sequence 0: behind P / 2 rows of its own, at a smaller scale; sequence 1: from its first page's first row on
    c.scales[:, 0] = 2.0 ** -9
    c.model.scales[:, 0] = 2.0 ** -9
    both = torch.cat((k, k))
    c.cache.append(c.table, c.lens_t, None, both, both, 1e4, positions=i32(np.r_[pos, pos]), row_start=i32([0, n, 2 * n]))
    torch.cuda.synchronize()
    x2 = np.concatenate((x, x))
    c.model.write(c.table_np, c.lens, np.concatenate((y, y))[None], x2[None], [0, n, 2 * n])
    same_k(c)
    # single rows behind what is there
    for step in range(3):
        lens = [P // 2 + n + step + 1, n + step + 1]
        rows, at = [step, n - 1 - step], pos[[step, n - 1 - step]]
        one = k[rows].contiguous()
        c.cache.append(c.table, i32(lens), None, one, one, 1e4, positions=i32(at), max_len=P // 2 + n + 4)
        torch.cuda.synchronize()
        c.model.write(c.table_np, lens, y[rows][None], x[rows][None], [0, 1, 2])
        same_k(c)
    c.done()


@pytest.mark.parametrize("dtype,P,rows", [("f32", 16, 16), ("f32", 256, 256), ("f32", 64, 1), ("bf16", 32, 32)])
def test_maxima_next_to_a_scale(cb, dtype, P, rows):
    """Blocks whose largest value lies next to 448 times a power of two: the exact maximum decides, and with it all codes of the block.
    A value that is equal to the border (a row at position 0) does not pass it."""
    hd, blocks = 64, 48
    rng = np.random.default_rng(P + rows)
    n = blocks * rows
    pos = rng.integers(-3000, 3000, n)
    angle = angles(pos, 1e4, hd)
    x = rng.normal(size=(n, 1, hd)) * 60
    x = bf16(np.clip(x, -200, 200))
    for b in range(blocks):
        r, i = b * rows + int(rng.integers(0, rows)), int(rng.integers(1, hd // 2))
        if b % 6 == 0:
            pos[r], angle[r] = 0, 0.0
            x[r, 0, 2 * i:2 * i + 2] = 448.0, 3.0
        elif dtype == "f32":
            want, other = 448.0, rng.uniform(-300, 300)
            c, s = np.cos(angle[r, i]), np.sin(angle[r, i])
            x[r, 0, 2 * i:2 * i + 2] = np.float32([want * c + other * s, other * c - want * s])
        else:
            # of all bf16 numbers and pairs the one that, with the nearest partner, comes nearest
            a = bf16(np.concatenate([np.geomspace(1, 500, 2000), -np.geomspace(1, 500, 2000)]))[:, None]
            c, s = np.cos(angle[r, 1:]), np.sin(angle[r, 1:])
            d = bf16((a * c - 448.0) / s)
            y0, y1 = a * c - d * s, a * s + d * c
            at, i = np.unravel_index(np.where(np.abs(y1) < 440, np.abs(np.abs(y0) - 448.0), 1e9).argmin(), d.shape)
            x[r, 0, 2 * i + 2:2 * i + 4] = a[at, 0], d[at, i]
    y = turned(x, angle)
    tops = np.abs(y).reshape(blocks, -1).max(axis=1)
    off = np.abs(tops - 448) / 448
    assert (off[np.arange(blocks) % 6 > 0] > 1e-11).all() and (off < 5e-7).mean() > 0.6
    wide = (tops > 448).sum()
    assert wide >= 5 and (tops <= 448).sum() >= 5
    c = Case(cb, [rows] * blocks, H=1, G=1, hd=hd, P=P, dtype=dtype, seed=6)
    k = torch.from_numpy(x.astype(np.float32)).to(c.td).cuda()
    assert np.array_equal(f64(k), x)
    c.cache.append(c.table, c.lens_t, None, k, k, 1e4, positions=i32(pos))
    torch.cuda.synchronize()
    c.model.write(c.table_np, c.lens, y[None], x[None], starts_of([rows] * blocks))
    assert sorted(set(c.model.scales[0, 0, c.table_np[:, 0], 0])) == [1.0, 2.0]
    used = np.repeat(c.model.scales[0, 0, c.table_np[:, 0], 0], rows)[:, None, None]
    m = margin(y, used)
    assert m[m > 0].min() > 1e-12
    same_k(c)
    c.done()


def test_zero_rows(cb):
    """Rows and pairs of zeros stay zeros beside others, whatever their sign."""
    c = Case(cb, [64], H=2, G=1, hd=64, P=16, dtype="f32", seed=1)
    x = c.rng.normal(size=(64, 2, 64)).astype(np.float32)
    x[:16] = 0
    x[16:32] = -0.0
    x[32:, :, 10:20] = 0
    x[40:, :, 1::2] = -0.0
    k = torch.from_numpy(x).cuda()
    y = turned(f64(k), angles(np.arange(64), 1e4, 64))
    c.cache.append(c.table, c.lens_t, None, k, k, 1e4)
    torch.cuda.synchronize()
    c.model.write(c.table_np, c.lens, y[None], f64(k)[None], [0, 64])
    same_k(c)
    assert (c.scales[0, 0, c.table[0, :2].long()] == 0).all()
    c.done()
