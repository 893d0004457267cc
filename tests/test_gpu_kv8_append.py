"""GPU tests of rows appended to the 8-bit paged cache with q and k rotated on the way, against float64.

Tolerance of a rotated value.  The phase is exact to the float64 frequency's rounding (at most 2^-56 of a turn per position,
2^-36 for positions up to 2^20, 2^-25 for the largest) and is cut to 2^-32 turns, 1.5e-9; its fp32 conversion, the constant and
their product are off by at most 3 * 2^-25 of an angle within pi / 4: 7.0e-8.  The series are evaluated within 2 * 2^-24 and
truncated by 2e-9; the two products and their sum round three times at most, 3 * 2^-24 of the pair's magnitude.  Together
less than 3.8e-7, so 2^-21 (|a| + |b|) for positions up to 2^20.  The largest positions add 2 pi 2^-25 = 1.9e-7 here and, in
the float64 reference, 2^31 * 2^-53 of a radian, 2.4e-7: 2^-20 holds for every position.  A code is right if it lies
between the codes of the exact value less and plus that error, a scale if it lies between the scales of such maxima."""
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


def rotate(x, positions, theta):
    """float64 x [rows][heads][dim]; (rotated, |a| + |b| of each value's pair)."""
    i = np.arange(x.shape[-1] // 2)
    angle = np.asarray(positions, np.float64)[:, None] * theta ** (-2.0 * i / x.shape[-1])
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = x[..., 0::2], x[..., 1::2]
    out, size = np.empty_like(x), np.empty_like(x)
    out[..., 0::2], out[..., 1::2] = a * c - b * s, a * s + b * c
    size[..., 0::2] = size[..., 1::2] = np.abs(a) + np.abs(b)
    return out, size


def scale_between(top, err, was, got):
    lo, hi = km.scale_of(np.array([max(top - err, 0.0)])), km.scale_of(np.array([top + err]))
    return max(lo, was) <= got <= max(hi, was)


EPS = {"bf16": 2.0 ** -21, "f32": 2.0 ** -21}           # positions up to 2^20


def check_k(c, before, table, lens, k, size, starts, eps, layer=0):
    """The pool's K blocks that got rows, against exact rotated rows k and their pairs' sizes; other K blocks as before."""
    codes, scales = c.codes.cpu().numpy(), c.scales.cpu().numpy().astype(np.float64)
    seen = np.zeros((c.model.n_pages, c.H, c.P), bool)
    for s, n in enumerate(lens):
        rows = starts[s + 1] - starts[s]
        first = n - rows
        for b in range(first // c.P, -(-n // c.P)) if rows else ():
            lo, hi = max(first - b * c.P, 0), min(n - b * c.P, c.P)
            pg = table[s][b]
            src = slice(starts[s] + b * c.P + lo - first, starts[s] + b * c.P + hi - first)
            for h in range(c.H):
                x, e = k[src, h], eps * size[src, h]
                sc = scales[layer, 0, pg, h]
                at = np.unravel_index(np.abs(x).argmax(), x.shape)
                was = before.scales[layer, 0, pg, h] if lo > 0 else 0.0
                assert scale_between(abs(x[at]), e.max(), was, sc), (s, b, h)
                got = km.VALUES[codes[layer, 0, pg, h, lo:hi]]
                if sc == 0:
                    assert not x.any()
                else:
                    low, high = (km.VALUES[km.encode(v / sc)] for v in (x - e, x + e))
                    assert ((low <= got) & (got <= high)).all(), (s, b, h)
                old = before.codes[layer, 0, pg, h, :lo]
                if lo and was not in (sc, 0.0):
                    old = km.encode(km.VALUES[old] * was / sc)
                assert np.array_equal(codes[layer, 0, pg, h, :lo], old)
                seen[pg, h, :hi] = True
    rest = ~seen
    assert np.array_equal(codes[layer, 0][rest], before.codes[layer, 0][rest])


def check_q(out, exact, size, eps, dtype, untouched=()):
    half = 2.0 ** (-8 if dtype == "bf16" else -24)
    rows = [r for r in range(len(exact)) if r not in set(untouched)]
    err = np.abs(f64(out)[rows] - exact[rows])
    lim = half * np.abs(exact[rows]) + (1 + half) * eps * size[rows]
    assert (err <= lim).all(), float((err - lim).max())


@pytest.mark.parametrize("hd,dtype,P,H,G", [(128, "bf16", 64, 2, 4), (64, "bf16", 16, 3, 1), (128, "f32", 256, 1, 3), (64, "f32", 32, 2, 8),
                                            (128, "bf16", 256, 1, 2), (64, "bf16", 128, 2, 7)])
@pytest.mark.parametrize("given", [False, True])
def test_append_ragged(cb, hd, dtype, P, H, G, given):
    """Ragged rows that begin and end inside pages, rows of no sequence, a sequence without rows, an empty one; positions given
    (negative ones among them) or the rows' places."""
    lens = [5 * P // 2 + 3, 1, 7, 3 * P, 0, P + 1, 2 * P]
    rows = [P + 5, 1, 0, 3 * P, 0, 1, P]
    c = Case(cb, lens, L=2, H=H, G=G, hd=hd, P=P, dtype=dtype, seed=hd + P + given)
    st = starts_of(rows, 2)
    n = st[-1] + 3
    theta = 5e5 if given else 1e4
    place = np.zeros(n, np.int64)
    for s, m in enumerate(lens):
        place[st[s]:st[s + 1]] = np.arange(m - rows[s], m)
    pos = c.rng.integers(-(1 << 20), 1 << 20, n) if given else place
    q, q64 = c.values(n, H * G, hd)
    k, k64 = c.values(n, H, hd, size=3.0)
    v, v64 = c.values(n, H, hd, size=50.0)
    before = km.Model(c.model.codes, c.model.scales)
    kr, ks = rotate(k64, pos, theta)
    qr, qs = rotate(q64, pos, theta)
    out = torch.full_like(q, 9.0)
    got = c.cache.append(c.table, c.lens_t, q, k, v, theta, out_q=out, layer=1, positions=i32(pos) if given else None, row_start=i32(st))
    assert got is out
    torch.cuda.synchronize()
    own = [r for s in range(len(lens)) for r in range(st[s], st[s + 1])]
    none = [r for r in range(n) if r not in own]
    check_q(out, qr, qs, EPS[dtype], dtype, none)
    assert (f64(out)[none] == 9.0).all()
    check_k(c, before, c.table_np, lens, kr, ks, st, EPS[dtype], layer=1)
    # V as write puts it there, and nothing in the other layer
    c.model.write(c.table_np, lens, v64[None], v64[None], st, layer=1)
    codes, scales = c.codes.cpu().numpy(), c.scales.cpu().numpy()
    assert np.array_equal(codes[1, 1], c.model.codes[1, 1]) and np.array_equal(codes[0], before.codes[0])
    assert np.array_equal(scales[1, 1], c.model.scales[1, 1].astype(np.float32)) and np.array_equal(scales[0], before.scales[0].astype(np.float32))
    c.done()


def test_append_far_positions(cb):
    """The largest positions of both signs, and the exact rotation by 0."""
    H, hd, P = 1, 64, 16
    pos = [0, 1, (1 << 31) - 1, -(1 << 31), 1 << 30, (1 << 24) + 1, -1, 131071, 8, 9, 10]
    c = Case(cb, [len(pos)], H=H, G=1, hd=hd, P=P, dtype="f32", seed=5)
    q, q64 = c.values(len(pos), 1, hd)
    out = c.cache.append(c.table, c.lens_t, q, q, q, 1e4, positions=i32(pos))
    exact, size = rotate(q64, pos, 1e4)
    check_q(out, exact, size, 2.0 ** -20, "f32")
    assert torch.equal(out[0], q[0])
    c.done()


def test_append_steps_and_slices(cb):
    """Forty single-row steps whose blocks' scales grow: q, k and v are slices of one projection's rows, q rotated in place; the
    rows that a graph appends follow lens and positions."""
    H, G, hd, P, B = 2, 4, 128, 16, 3
    c = Case(cb, [5, 16, 31], H=H, G=G, hd=hd, P=P, seed=8, spare=40)
    width = (H * G + 2 * H) * hd
    proj = torch.zeros((B, width), dtype=torch.bfloat16, device="cuda")
    q, k, v = proj.split([H * G * hd, H * hd, H * hd], dim=1)
    q, k, v = q.view(B, H * G, hd), k.view(B, H, hd), v.view(B, H, hd)
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens_np = np.array(c.lens)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        for warm in range(2):
            c.cache.append(c.table, torch.zeros_like(c.lens_t), q, k, v, 5e5, out_q=q, positions=pos, max_len=71)
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        c.cache.append(c.table, c.lens_t, q, k, v, 5e5, out_q=q, positions=pos, max_len=71)
    st = [0, 1, 2, 3]
    for step in range(40):
        lens_np = lens_np + 1
        new = torch.from_numpy((c.rng.normal(size=(B, width)) * 1.3 ** (step % 17)).astype(np.float32)).cuda().bfloat16()
        at = lens_np - 1 + 4000 * np.arange(B)
        proj.copy_(new)
        c.lens_t.copy_(i32(lens_np))
        pos.copy_(i32(at))
        graph.replay()
        torch.cuda.synchronize()
        x = f64(new)
        q64, k64, v64 = x[:, :H * G * hd].reshape(B, -1, hd), x[:, H * G * hd:-H * hd].reshape(B, H, hd), x[:, -H * hd:].reshape(B, H, hd)
        qr, qs = rotate(q64, at, 5e5)
        check_q(q, qr, qs, EPS["bf16"], "bf16")
        assert np.array_equal(f64(k), k64) and np.array_equal(f64(v), v64)
        kr, ks = rotate(k64, at, 5e5)
        check_k(c, c.model, c.table_np, lens_np, kr, ks, st, EPS["bf16"])
        c.model.write(c.table_np, lens_np, v64[None], v64[None], st)
        c.model.codes[:, 0], c.model.scales[:, 0] = c.codes[:, 0].cpu().numpy(), c.scales[:, 0].cpu().numpy()
        c.check_pool()
    c.done()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_special_values(cb, dtype):
    """Rows of zeros, NaN and infinities, the largest and smallest numbers: as write stores them, both of a pair that meets a NaN
    or an infinity being NaN after a rotation by an angle that is not 0."""
    P, H, hd = 16, 1, 64
    c = Case(cb, [4 * P], H=H, G=1, hd=hd, P=P, dtype=dtype, seed=3)
    x = c.rng.normal(size=(4 * P, H, hd)).astype(np.float32)
    x[:P] = 0
    x[P, 0, 0] = np.nan
    x[P, 0, 6] = np.inf
    x[2 * P:3 * P] *= 1e-39
    x[3 * P:] = np.clip(x[3 * P:], -1.9, 1.9) * 1e38
    k = torch.from_numpy(x).to(c.td).cuda()
    c.cache.append(c.table, c.lens_t, None, k, k, 1e4)
    torch.cuda.synchronize()
    k64 = f64(k)
    c.model.write(c.table_np, c.lens, k64[None], k64[None], [0, 4 * P])
    codes, scales = c.codes.cpu().numpy()[0], c.scales.cpu().numpy()[0]
    pages = c.table_np[0]
    assert np.array_equal(scales[1], c.model.scales[0, 1].astype(np.float32))
    same = (codes[1] == c.model.codes[0, 1]) | (np.isnan(km.VALUES[codes[1]]) & np.isnan(km.VALUES[c.model.codes[0, 1]]))
    assert same.all()
    kv = km.VALUES[codes[0]]
    assert scales[0, pages[0], 0] == 0 and not kv[pages[0]].any()
    nan = np.isnan(kv[pages[1], 0])
    assert nan[0, [0, 1, 6, 7]].all() and nan.sum() == 4
    for b in (2, 3):
        exact, size = rotate(k64[b * P:(b + 1) * P], np.arange(b * P, (b + 1) * P), 1e4)
        got = kv[pages[b], 0] * scales[0, pages[b], 0].astype(np.float64)
        step = 2.0 ** -4 * np.abs(exact[:, 0]) + 2.0 ** -9 * scales[0, pages[b], 0]
        flush = 2.0 ** -126 * 4                          # fp32 products below the normal numbers may be 0
        # (at a scale of 2^120 codes end at 240)
        assert (np.abs(got - np.clip(exact[:, 0], -240 * 2.0 ** 120, 240 * 2.0 ** 120)) <= step + EPS[dtype] * size[:, 0] + flush).all()
    c.done()


def test_append_bad_rows(cb):
    """A page id outside the pool, a length below the rows' number and one out of range: recorded, their rows left as they were."""
    P, H, G, hd = 16, 1, 2, 64
    c = Case(cb, [20, 3, 40, 10], H=H, G=G, hd=hd, P=P, seed=2)
    table = c.table_np.copy()
    table[0, 1] = 1 << 20
    lens = [20, 3, 4000, 10]
    st = [0, 6, 10, 15, 17]                               # sequence 1 has four rows and a length of 3
    q, q64 = c.values(17, H * G, hd)
    k, k64 = c.values(17, H, hd)
    out = torch.full_like(q, 9.0)
    before_codes = c.codes.cpu().numpy()
    c.cache.append(i32(table), i32(lens), q, k, k, 1e4, out_q=out, row_start=i32(st), max_len=48)
    torch.cuda.synchronize()
    assert c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    got = f64(out)
    assert (got[6:15] == 9.0).all()
    place = np.r_[np.arange(14, 20), np.zeros(9), [8, 9]]
    qr, qs = rotate(q64, place, 1e4)
    check_q(out, qr, qs, EPS["bf16"], "bf16", untouched=range(6, 15))       # q is rotated whether its page is good or not
    kr, ks = rotate(k64, place, 1e4)
    codes = c.codes.cpu().numpy()
    changed = (codes != before_codes).any(axis=(0, 1, 3, 5))               # [pages][rows]
    allowed = np.zeros_like(changed)
    allowed[table[0, 0], :16] = True
    allowed[table[3, 0], :10] = True
    assert not (changed & ~allowed).any() and changed[table[0, 0], 14:16].all() and changed[table[3, 0], 8:10].all()
    c.done()


def test_append_on_a_stream_of_its_own(cb):
    """Outputs that the call makes are made on its stream; write and attention behind it there need no further wait."""
    P, H, G, hd = 32, 2, 4, 64
    c = Case(cb, [40, 70], H=H, G=G, hd=hd, P=P, seed=12)
    q, q64 = c.values(4, H * G, hd)
    k, k64 = c.values(4, H, hd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = c.cache.append(c.table, c.lens_t, q, k, k, 1e4, stream=side)
    o = c.cache.attention(c.table, c.lens_t, out, stream=side)
    side.synchronize()
    place = [38, 39, 68, 69]
    qr, qs = rotate(q64, place, 1e4)
    check_q(out, qr, qs, EPS["bf16"], "bf16")
    m = km.Model(c.codes.cpu().numpy(), c.scales.cpu().numpy())
    ref, _, spread, _ = m.attention(c.table_np, c.lens, f64(out), [0, 2, 4], 0, hd ** -0.5)
    assert (np.abs(f64(o) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * spread).all()
    c.done()


def test_append_refusals(cb):
    """Tensors of another shape, type or layout, and numbers out of range, are refused before anything is enqueued."""
    c = Case(cb, [40, 20], H=2, G=2, hd=64, P=16)
    k, v, q = (c.values(2, h, 64)[0] for h in (2, 2, 4))
    wide = torch.zeros((2, 2, 128), dtype=k.dtype, device="cuda")
    before = c.codes.clone()

    def refused(what, *args, **kw):
        with pytest.raises((ValueError, cb.CacheBlendError), match=what):
            c.cache.append(c.table, c.lens_t, *args, **{"rope_theta": 1e4, **kw})
    refused("k must", q, k.float(), v)
    refused("v must", q, k, v.cpu())
    refused("k must", q, k[:, :1], v)
    refused("contiguous", q, wide[:, :, ::2], v)
    refused("contiguous", q, k, wide[:, :, :64])
    refused("same number of rows", q, k, v[:1])
    refused("q must", q[:, :3], k, v)
    refused("rows", q[:1], k, v)
    refused("rows", q, k, v, out_q=q[:1].clone())
    refused("out_q without q", None, k, v, out_q=q)
    refused("positions", q, k, v, positions=i32([1, 2, 3]))
    refused("row_start", q, k, v, row_start=i32([0, 2]))
    refused("theta", q, k, v, rope_theta=0.0)
    refused("theta", q, k, v, rope_theta=float("nan"))
    refused("layer", q, k, v, layer=1)
    torch.cuda.synchronize()
    assert torch.equal(c.codes, before)
    c.done()


def test_append_codes_of_exact_rotation(cb):
    """Codes are those of the rotation in 64 bits, also next to the middle between two codes.  A value's fp32 error is at most
    1.7 2^-23 (|a| + |b|) of its pair (sine and cosine within 2^-23.5, a product's and the result's rounding), which is less than the 5
    units in its last place that are looked at anew where the value is at least 0.8 (|a| + |b|)."""
    P, H, hd, n = 64, 8, 128, 8192
    c = Case(cb, [n], H=H, G=1, hd=hd, P=P, seed=31)
    k = torch.randn((n, H, hd), device="cuda", generator=torch.Generator("cuda").manual_seed(5)).to(c.td)
    c.cache.append(c.table, c.lens_t, None, k, k, 5e5)
    torch.cuda.synchronize()
    i = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 5e5 ** (-2.0 * i / hd)
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = k[..., 0::2].double(), k[..., 1::2].double()
    y = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    size = (a.abs() + b.abs()).repeat_interleave(2, dim=-1)
    pages = c.table[0, :n // P].long()
    scale = c.scales[0, 0, pages].double()                                           # [blocks][H]
    y = y.view(n // P, P, H, hd) / scale[:, None, :, None]
    got = c.codes[0, 0, pages].view(torch.float8_e4m3fn).float().double().transpose(1, 2)
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(y.abs().clamp_min(1e-30))), min=-6) - 3)
    want = torch.round(y / step) * step                                              # (ties to even)
    sure = y.abs() >= 0.8 * (size.view_as(y) / scale[:, None, :, None])
    assert sure.float().mean() > 0.1 and torch.equal(got[sure], want[sure])
    assert (got != want).sum() < 8.4e6 * 2.0 ** -18                                  # and of the others hardly one
    c.done()
