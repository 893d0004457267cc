"""GPU tests of the 8-bit paged K/V cache against the float64 model of tests/kv8_model.py: rows written and read back,
appends, attention (causal, ragged, weights, NaN behind the mask), eviction, bad ids, graphs, streams, and the
operators run together as a request uses them.

Tolerances.  Codes, scales, rows read back, kept rows and moved weights are exact.  Attention: with u = 2^-24, a
score's error is at most ds = (head_dim + 8) u max sum|q k| scale (products and sums in fp32, whatever their order); a
softmax weight is then off by a factor e^(2 ds), about 2 ds, plus at most 16 u of its own evaluation.  out adds a sum
over keys in fp32 (at most (128 + len / 128) u of sum p|v|: 128 keys at a time, then the steps' partial sums), the
representation of p by the matrix unit's operands (2^-11 of it in bf16 calls, 2^-23 in fp32 ones) and one rounding of
the result (half a step: 2^-8 |out| in bf16, 2^-24 in fp32).

That representation has a floor too.  p times V's block scale stands as T e4m3 terms, term t in units of 16^-t, of numbers
scaled so that the largest of a tile of 128 keys lies between 128 and 256.  A term's last place is 2^-9, so a number
below the terms' range is off by at most half of it in the last term, 2^-10 16^-(T-1): relative to the tile's largest
p * scale, Y >= 128 in those units, at most 2^-17 16^-(T-1), that is 2^-25 for T = 3 (bf16) and 2^-37 for T = 6 (fp32).
An output element meets it once per key, times the key's code: 2^-25 or 2^-37 of the sum over tiles of
Y sum|code| (the model's `floor`).  It shows only where keys of one tile differ by 2^14 and more in p * scale.
With many query rows (bf16, more than 32 rows times heads of a group) p times the scale is an fp16 number, 2^7 times its
size relative to a reference that is at most the largest so far: half of fp16's last place is 2^-25, so an element is off
by at most 2^-32 of (largest p * scale) * sum|code| over all keys (`floor_all`), besides 2^-12 of p."""
import numpy as np
import pytest

import kv8_model as km

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24


@pytest.fixture(scope="module")
def cb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import cacheblend_selective_kv_gb300 as cbm
    return cbm


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Case:
    """A pool of random codes, a shuffled block table and its model."""

    def __init__(self, cb, lens, *, L=1, H=2, G=2, hd=64, P=16, dtype="bf16", seed=0, extra=4, cells=0, spare=0):
        self.rng = np.random.default_rng(seed)
        self.cb, self.lens, self.L, self.H, self.G, self.hd, self.P, self.dtype = cb, list(lens), L, H, G, hd, P, dtype
        self.td = torch.bfloat16 if dtype == "bf16" else torch.float32
        top = max(max(lens), 1) + spare
        width = -(-top // P)
        n_pages = width * len(lens) + extra
        order = self.rng.permutation(n_pages).astype(np.int32)
        self.table_np = order[:width * len(lens)].reshape(len(lens), width)
        self.free = list(order[width * len(lens):])
        codes = self.rng.integers(0, 256, (L, 2, n_pages, H, P, hd)).astype(np.uint8)
        codes[(codes & 0x7F) == 0x7F] = 3
        codes &= 0xEF                                   # a spread of a few octaves
        codes[(codes & 0x7F) == 0x7F] = 3
        scales = 2.0 ** self.rng.integers(-9, -5, (L, 2, n_pages, H))
        # rows behind a sequence's last one, and pages of no sequence, hold NaN codes
        used = np.zeros((n_pages, P), bool)
        for s, n in enumerate(lens):
            for b in range(-(-n // P)):
                used[self.table_np[s, b], :min(P, n - b * P)] = True
        codes[:, :, ~used.reshape(n_pages, P)[:, 0]] = 0x7F
        for pg in range(n_pages):
            codes[:, :, pg][:, :, :, ~used[pg]] = 0x7F
        self.model = km.Model(codes, scales)
        self.codes = torch.from_numpy(codes).cuda()
        self.scales = torch.from_numpy(scales.astype(np.float32)).cuda()
        self.table, self.lens_t = i32(self.table_np), i32(self.lens)
        self.cache = cb.KV8Cache(self.codes, self.scales, n_heads=H * G, dtype=dtype, weight_cells=cells)

    def values(self, *shape, size=1.0):
        """Random values of the rows' type, as (tensor, float64)."""
        t = torch.from_numpy((self.rng.normal(size=shape) * size).astype(np.float32)).to(self.td).cuda()
        return t, f64(t)

    def check_pool(self):
        assert np.array_equal(self.scales.cpu().numpy(), self.model.scales.astype(np.float32))
        got, ref = self.codes.cpu().numpy(), self.model.codes
        same = (got == ref) | (((got & 0x7F) == 0x7F) & ((ref & 0x7F) == 0x7F))
        assert same.all(), np.argwhere(~same)[:5]

    def done(self, status=0):
        torch.cuda.synchronize()
        assert self.cache.status(clear=True) == status
        self.cache.close()


def starts_of(rows, first=0):
    return [first + int(x) for x in np.concatenate([[0], np.cumsum(rows)])]


# ------------------------------------------------------------------------------------------------
# write and read
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("hd,dtype,P,H", [(64, "f32", 16, 2), (128, "bf16", 16, 3), (64, "bf16", 32, 1), (128, "f32", 64, 2),
                                          (128, "bf16", 128, 2), (64, "f32", 256, 3), (128, "f32", 256, 1)])
def test_write_and_read_ragged(cb, hd, dtype, P, H):
    """Ragged rows that begin and end inside pages, in two of three layers, sizes that force both kinds of scale."""
    lens = [5 * P // 2 + 3, 1, 7, 3 * P, 0, P + 1]
    rows = [P + 5, 1, 0, 3 * P, 0, 1]
    c = Case(cb, lens, L=3, H=H, hd=hd, P=P, dtype=dtype, seed=hd + P)
    st = starts_of(rows, 2)
    n = st[-1] + 3                                      # rows 0, 1 and the last three belong to no sequence
    k, k64 = c.values(2, n, H, hd)
    v, v64 = c.values(2, n, H, hd, size=100.0)
    k[:, 3] *= 1e4
    k64 = f64(k)
    c.cache.write(c.table, c.lens_t, k, v, layer=1, n_layers=2, row_start=i32(st))
    c.model.write(c.table_np, lens, k64, v64, st, layer=1)
    torch.cuda.synchronize()
    c.check_pool()
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    c.cache.read(c.table, c.lens_t, ko, vo, layer=1, n_layers=2, row_start=i32(st))
    for l in range(2):
        for out, kv in ((f64(ko), 0), (f64(vo), 1)):
            ref = np.full((n, H, hd), 7.0)
            for s, m in enumerate(lens):
                ref[st[s]:st[s + 1]] = c.model.rows(c.table_np[s], m, 1 + l)[kv][m - rows[s]:]
            assert np.array_equal(out[l], ref)
    c.done()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_special_values(cb, dtype):
    """Blocks of zeros, NaN, infinities, the smallest and largest numbers, and values at 448 times a power of two."""
    P, H, hd = 16, 1, 64
    c = Case(cb, [8 * P], H=H, hd=hd, P=P, dtype=dtype, seed=3)
    x = c.rng.normal(size=(1, 8 * P, H, hd)).astype(np.float32)
    x[0, :P] = 0
    x[0, P, 0, 0] = np.nan
    x[0, P, 0, 1] = np.inf
    x[0, P, 0, 2] = -np.inf
    x[0, 2 * P:3 * P] = 0
    x[0, 2 * P, 0, 5] = np.nan
    x[0, 3 * P:4 * P] *= 1e-39
    x[0, 4 * P:5 * P] *= 1e38 / 4
    x[0, 5 * P, 0, 0] = 448.0 * 4
    x[0, 6 * P:7 * P] = np.clip(x[0, 6 * P:7 * P], -1, 1)
    x[0, 6 * P, 0, 0] = np.float32(1.7578125)           # just above 448 * 2^-8
    x[0, 7 * P:, 0, :32] = 2.0 ** -20
    t = torch.from_numpy(x).to(c.td).cuda()
    ref = f64(t)
    c.cache.write(c.table, c.lens_t, t, t)
    c.model.write(c.table_np, c.lens, ref, ref, [0, 8 * P])
    torch.cuda.synchronize()
    c.check_pool()
    ko, vo = torch.zeros_like(t), torch.zeros_like(t)
    c.cache.read(c.table, c.lens_t, ko, vo)
    want = c.model.rows(c.table_np[0], 8 * P, 0)
    assert np.array_equal(f64(ko)[0], want[0], equal_nan=True) and np.array_equal(f64(vo)[0], want[1], equal_nan=True)
    c.done()


def test_append_grows_the_scale_captured(cb):
    """One token per sequence and step through one captured graph: sizes that grow and shrink, so that blocks are
    rounded to larger scales, pages begin, and shared buffers and lengths change between replays."""
    H, hd, P, steps = 2, 128, 16, 40
    start = [0, 15, 16, 33, 5]
    c = Case(cb, start, H=H, hd=hd, P=P, seed=9, spare=steps)
    k = torch.zeros((1, 5, H, hd), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    lens = i32(start)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.cache.write(c.table, lens, k, v)
    c.check_pool()                                      # capturing runs nothing
    now = list(start)
    for step in range(steps):
        size = 2.0 ** c.rng.integers(-12, 12)
        kk, k64 = c.values(1, 5, H, hd, size=size)
        vv, v64 = c.values(1, 5, H, hd, size=1.0 / size)
        now = [n + 1 for n in now]
        k.copy_(kk)
        v.copy_(vv)
        lens.copy_(i32(now))
        g.replay()
        c.model.write(c.table_np, now, k64, v64, list(range(6)))
    torch.cuda.synchronize()
    c.check_pool()
    c.done()


def test_rows_with_strides(cb):
    """K and V as slices of a fused projection's rows, and as the halves of a [layers][2][rows] buffer."""
    H, hd, P, n = 2, 64, 16, 37
    c = Case(cb, [n], H=H, hd=hd, P=P, seed=4)
    qkv = torch.from_numpy(c.rng.normal(size=(n, 4 * H + 2 * H, hd)).astype(np.float32)).to(torch.bfloat16).cuda()
    k, v = qkv[:, 4 * H:5 * H], qkv[:, 5 * H:]
    c.cache.write(c.table, c.lens_t, k, v)
    c.model.write(c.table_np, c.lens, f64(k)[None], f64(v)[None], [0, n])
    both = torch.zeros((1, 2, n, H, hd), dtype=torch.bfloat16, device="cuda")
    c.cache.read(c.table, c.lens_t, both[:, 0], both[:, 1])
    torch.cuda.synchronize()
    c.check_pool()
    want = c.model.rows(c.table_np[0], n, 0)
    assert np.array_equal(f64(both)[0, 0], want[0]) and np.array_equal(f64(both)[0, 1], want[1])
    c.done()


# ------------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------------
def check_attention(c, q, q64, starts, out, w=None, layer=0, w_before=0.0, scale=None):
    scale = c.hd ** -0.5 if scale is None else scale
    ref, ws, spread, big = c.model.attention(c.table_np, c.lens, q64, starts, layer, scale)
    ds = (c.hd + 8) * U * big
    steps = 128 + max(c.lens) / 128
    p_rep, rnd, last = (2.0 ** -11, 2.0 ** -8, 2.0 ** -25) if c.dtype == "bf16" else (2.0 ** -23, 2.0 ** -24, 2.0 ** -37)
    got = f64(out)
    owned = np.zeros(len(q64), bool)
    for s in range(len(c.lens)):
        owned[starts[s]:starts[s + 1]] = True
    tol = rnd * np.abs(ref) + (2 * ds + (16 + steps) * U + p_rep) * spread + last * c.model.floor + 2.0 ** -32 * c.model.floor_all
    err = np.abs(got - ref)[owned]
    assert np.all(err <= tol[owned] + 1e-30), (err.max(), float((err / (tol[owned] + 1e-30)).max()))
    if w is not None:
        G, wg = q64.shape[1] // c.H, f64(w)
        for s, n in enumerate(c.lens):
            rows = starts[s + 1] - starts[s]
            r = ws[s] + w_before
            tol = (2 * ds + (16 + steps + rows * G) * U) * r
            e = np.abs(wg[s, :, :n] - r)
            assert np.all(e <= tol + 1e-30), (s, e.max(), float((e / (tol + 1e-30)).max()))
    return owned


ATTN = [  # hd, dtype, H, G, P, lens, rows per sequence
    (128, "bf16", 2, 4, 16, [1, 17, 128, 129, 300], [1, 1, 1, 1, 1]),
    (64, "bf16", 2, 2, 32, [5, 700, 0, 64], [1, 1, 1, 1]),
    (128, "bf16", 1, 8, 64, [513, 40], [3, 7]),
    (64, "bf16", 3, 1, 16, [90, 256, 33], [5, 33, 2]),
    (128, "bf16", 2, 3, 128, [400, 3, 129], [17, 9, 0]),
    (128, "bf16", 1, 7, 256, [1025], [13]),
    (64, "f32", 2, 4, 16, [200, 12, 385], [2, 20, 1]),
    (128, "f32", 1, 5, 32, [260, 31], [33, 1]),
    (128, "f32", 2, 1, 64, [129, 1], [1, 1]),
    (64, "f32", 1, 8, 256, [511], [16]),
    (128, "bf16", 1, 4, 32, [150], [150]),
    (64, "bf16", 1, 6, 64, [70], [70]),
]


@pytest.mark.parametrize("hd,dtype,H,G,P,lens,rows", ATTN)
def test_attention(cb, hd, dtype, H, G, P, lens, rows):
    n = sum(rows) + 5
    c = Case(cb, lens, L=2, H=H, G=G, hd=hd, P=P, dtype=dtype, seed=hd + G + P, cells=cb.KV8Cache.cells(n, H * G, max(lens)))
    st = starts_of(rows, 2)
    q, q64 = c.values(n, H * G, hd)
    out = torch.full_like(q, 9.0)
    w = torch.full((len(lens), H, max(lens) + 3), -5.0, device="cuda")
    c.cache.attention(c.table, c.lens_t, q, out, layer=1, q_start=i32(st), weights=w, max_len=max(lens))
    owned = check_attention(c, q, q64, st, out, w, layer=1)
    assert np.all(f64(out)[~owned] == 9.0)
    for s, m in enumerate(lens):
        assert torch.all(w[s, :, m:] == -5.0)
    again = torch.empty_like(q)
    c.cache.attention(c.table, c.lens_t, q, again, layer=1, q_start=i32(st), max_len=max(lens))
    o = torch.from_numpy(owned).cuda()
    assert torch.equal(again[o], out[o])                # the weights change nothing, and the bits repeat
    before = w.clone()
    c.cache.attention(c.table, c.lens_t, q, again, layer=1, q_start=i32(st), weights=w, add=True, max_len=max(lens))
    for s, m in enumerate(lens):
        assert torch.equal(w[s, :, :m], 2 * before[s, :, :m])
    c.done()


@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("f32", 3), ("bf16", 40)])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.5])
def test_attention_scale_of_any_sign(cb, dtype, rows, scale):
    """A negative scale turns the order of the keys round; with 0 every key that is seen weighs the same."""
    lens = [150, 300]
    c = Case(cb, lens, H=2, G=2, hd=64, P=32, dtype=dtype, seed=rows, cells=cb.KV8Cache.cells(2 * rows, 4, 300))
    q, q64 = c.values(2 * rows, 4, 64)
    out, w = torch.empty_like(q), torch.zeros((2, 2, 300), device="cuda")
    c.cache.attention(c.table, c.lens_t, q, out, scale=scale, weights=w, max_len=300)
    check_attention(c, q, q64, [0, rows, 2 * rows], out, w, scale=scale)
    c.done()


@pytest.mark.parametrize("rows", [[2, 0, 1, 3], [40, 9, 0, 70]])
def test_attention_with_empty_sequences(cb, rows):
    """Sequences without rows, without keys, and with more rows than keys, in one call; and calls without rows or keys."""
    lens = [400, 0, 129, 3]
    n, G = sum(rows), 3
    c = Case(cb, lens, H=2, G=G, hd=64, P=16, seed=sum(rows), cells=cb.KV8Cache.cells(n, 6, 400))
    q, q64 = c.values(n, 2 * G, 64)
    st, out = starts_of(rows), torch.full_like(q, 7.0)
    w = torch.full((4, 2, 400), 3.0, device="cuda")
    c.cache.attention(c.table, c.lens_t, q, out, q_start=i32(st), weights=w, max_len=400)
    check_attention(c, q, q64, st, out, w)
    assert torch.count_nonzero(out[st[1]:st[2]]) == 0   # no keys
    for s, m in enumerate(lens):
        assert torch.all(w[s, :, m:] == 3.0)
    assert torch.count_nonzero(w[[s for s in range(4) if rows[s] == 0], :, :0]) == 0
    # no keys at all: zeros, and nothing of the weights (nor of the scratch, which holds fewer rows than these)
    many = torch.ones((4 * 1000, 2 * G, 64), dtype=q.dtype, device="cuda")
    o = c.cache.attention(c.table, i32([0] * 4), many, weights=w, max_len=0)
    assert torch.count_nonzero(o) == 0 and torch.all(w[1] == 3.0)
    # no rows: every key's weight is 0, or what it was
    before = w.clone()
    none = q[:0]
    c.cache.attention(c.table, c.lens_t, none, weights=w, add=True, max_len=400)
    assert torch.equal(w, before)
    c.cache.attention(c.table, c.lens_t, none, weights=w, max_len=400)
    for s, m in enumerate(lens):
        assert torch.count_nonzero(w[s, :, :m]) == 0 and torch.all(w[s, :, m:] == 3.0)
    c.done()


@pytest.mark.parametrize("rows", [1, 40])
def test_two_handles_on_one_pool_at_once(cb, rows):
    lens = [3000, 1500]
    c = Case(cb, lens, H=2, G=4, hd=128, P=64, seed=3, cells=cb.KV8Cache.cells(2 * rows, 8, 3000))
    other = cb.KV8Cache(c.codes, c.scales, n_heads=8, weight_cells=cb.KV8Cache.cells(2 * rows, 8, 3000))
    qs = [c.values(2 * rows, 8, 128)[0] for _ in range(2)]
    ws = [torch.zeros((2, 2, 3000), device="cuda") for _ in range(4)]
    want = [c.cache.attention(c.table, c.lens_t, qs[i], weights=ws[i], max_len=3000) for i in range(2)]
    outs, streams = [torch.empty_like(q) for q in qs], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, cache in enumerate((c.cache, other)):
            cache.attention(c.table, c.lens_t, qs[i], outs[i], weights=ws[2 + i], max_len=3000, stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], want[i]) and torch.equal(ws[2 + i], ws[i])
    assert other.status() == 0
    other.close()
    c.done()


@pytest.mark.parametrize("dtype,rows", [("bf16", 2), ("f32", 2), ("bf16", 25)])
def test_attention_large_scores_and_scales(cb, dtype, rows):
    """Scores spread over hundreds (most weights vanish), a sink that outweighs the rest, and V blocks whose scales
    differ by 2^20."""
    lens = [900, 400]
    c = Case(cb, lens, H=1, G=4, hd=128, P=16, dtype=dtype, seed=21, cells=cb.KV8Cache.cells(2 * rows, 4, 900))
    sc = c.model.scales
    sc[0, 1] = 2.0 ** c.rng.integers(-20, 1, sc[0, 1].shape)
    sc[0, 0, c.table_np[1, 0]] *= 64
    c.scales.copy_(torch.from_numpy(sc.astype(np.float32)))
    q, q64 = c.values(2 * rows, 4, 128, size=4.0)
    out = torch.empty_like(q)
    w = torch.zeros((2, 1, 900), device="cuda")
    c.cache.attention(c.table, c.lens_t, q, out, weights=w, max_len=900)
    check_attention(c, q, q64, [0, rows, 2 * rows], out, w)
    c.done()


@pytest.mark.parametrize("rows", [1, 17])
def test_attention_one_key_outweighs_a_long_cache(cb, rows):
    """A first key whose weight is about 2^17 times any other's, over a cache long enough for the others to count."""
    n = 20000
    c = Case(cb, [n], H=1, G=2, hd=64, P=64, seed=5)
    m = c.model
    m.scales[:] = 2.0 ** -9
    m.codes[0, 0, c.table_np[0], :, :, 0] = 0x38        # 1.0 in every key's first channel
    m.codes[0, 0, :, :, :, 1:] = 0
    m.codes[0, 0, c.table_np[0, 0], 0, 0, 0] = 0x7E     # 448 in the first key's
    c.codes.copy_(torch.from_numpy(m.codes))
    c.scales.copy_(torch.from_numpy(m.scales.astype(np.float32)))
    q = torch.zeros((rows, 2, 64), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 108.0                                  # (448 - 1) * 2^-9 * 108 / 8 = 11.8 = ln 2^17
    out = torch.empty_like(q)
    c.cache.attention(c.table, c.lens_t, q, out)
    check_attention(c, q, f64(q), [0, rows], out)
    c.done()


@pytest.mark.parametrize("dtype,hd,G", [("bf16", 128, 2), ("f32", 64, 2), ("bf16", 128, 4), ("bf16", 64, 8)])
def test_nan_does_not_pass_the_mask(cb, dtype, hd, G):
    """NaN in the K or V of a row reaches the query rows that see it and no others."""
    lens, rows = [140, 60], [20, 4]
    c = Case(cb, lens, H=2, G=G, hd=hd, P=16, dtype=dtype, seed=8)
    m = c.model

    def spoil(kv, s, j, h, d):
        m.codes[0, kv, c.table_np[s, j // 16], h, j % 16, d] = 0xFF
    spoil(1, 0, 130, 0, 3)                              # V: seen from row 130 - 120 = 10 on
    spoil(1, 0, 134, 1, 5)
    spoil(1, 0, 125, 1, 5)
    spoil(0, 1, 58, 1, 0)                               # K: seen by rows 2 and 3 of the second sequence
    c.codes.copy_(torch.from_numpy(m.codes))
    q, q64 = c.values(24, 2 * G, hd)
    out = torch.empty_like(q)
    st = starts_of(rows)
    c.cache.attention(c.table, c.lens_t, q, out, q_start=i32(st))
    got = f64(out)
    want_nan = np.zeros(got.shape, bool)
    want_nan[10:20, 0:G, 3] = True
    want_nan[5:20, G:, 5] = True
    want_nan[22:24, G:] = True
    assert np.array_equal(np.isnan(got), want_nan)
    clean = km.Model(np.where((m.codes & 0x7F) == 0x7F, 0, m.codes).astype(np.uint8), m.scales)
    # without the spoiled numbers (their weights stay): every other output is the same sum
    c.model = clean
    ref, _, spread, big = clean.attention(c.table_np, lens, q64, st, 0, hd ** -0.5)
    seen_k = np.zeros(got.shape, bool)
    seen_k[22:24, G:] = True
    ok = ~want_nan & ~seen_k
    tol = 2.0 ** -8 * np.abs(ref) + (2 * (hd + 8) * U * big + 2.0 ** -11 + 200 * U) * spread
    assert np.all(np.abs(got - ref)[ok] <= tol[ok])
    c.done()


def test_attention_strides_and_uneven_heads(cb):
    """Queries as a slice of a fused projection, outputs into a wider buffer, rows shared evenly."""
    H, G, hd = 2, 4, 64
    c = Case(cb, [77, 300, 4], H=H, G=G, hd=hd, P=32, seed=6)
    wide = torch.from_numpy(c.rng.normal(size=(6, H * G + 2 * H, hd)).astype(np.float32)).to(torch.bfloat16).cuda()
    q = wide[:, :H * G]
    buf = torch.full((6, H * G + 1, hd), 3.0, dtype=torch.bfloat16, device="cuda")
    c.cache.attention(c.table, c.lens_t, q, buf[:, 1:], scale=0.2)
    check_attention(c, q, f64(q), [0, 2, 4, 6], buf[:, 1:], scale=0.2)
    assert torch.all(buf[:, 0] == 3.0)
    c.done()


@pytest.mark.parametrize("G", [1, 4])
def test_many_sequences(cb, G):
    """Enough sequences of every length that work is divided inside and between them; lengths far below max_len."""
    rng = np.random.default_rng(G)
    lens = [int(x) for x in rng.integers(0, 260, 90)]
    lens[7], lens[80] = 2500, 1300
    c = Case(cb, lens, H=2, G=G, hd=128, P=16, seed=11, cells=cb.KV8Cache.cells(90, 2 * G, 4000))
    q, q64 = c.values(90, 2 * G, 128)
    out = torch.empty_like(q)
    w = torch.zeros((90, 2, 4000), device="cuda")
    tab = torch.zeros((90, 250), dtype=torch.int32, device="cuda")
    tab[:, :c.table.shape[1]] = c.table
    tab[:, c.table.shape[1]:] = 10 ** 6                 # never read: behind every length
    c.cache.attention(tab, c.lens_t, q, out, weights=w, max_len=4000)
    check_attention(c, q, q64, list(range(91)), out, w)
    c.done()


@pytest.mark.parametrize("G,hd,P", [(4, 128, 16), (8, 64, 128), (5, 128, 256)])
def test_many_rows_of_many_sequences(cb, G, hd, P):
    """Query rows in numbers that end anywhere in a tile, over sequences of every length and some without rows or keys:
    items of one tile and of many, divided between CTAs."""
    rng = np.random.default_rng(G)
    lens = [0, 1, 700, 127, 128, 129, 30, 2100, 64, 300, 1]
    rows = [3, 1, 60, 40, 128, 2, 30, 33, 0, 90, 5]
    n = sum(rows)
    c = Case(cb, lens, H=2, G=G, hd=hd, P=P, seed=hd, cells=cb.KV8Cache.cells(n + 1, 2 * G, max(lens)))
    st = starts_of(rows, 1)
    q, q64 = c.values(n + 1, 2 * G, hd)
    out = torch.full_like(q, 2.0)
    w = torch.zeros((len(lens), 2, max(lens)), device="cuda")
    c.cache.attention(c.table, c.lens_t, q, out, q_start=i32(st), weights=w, max_len=max(lens))
    check_attention(c, q, q64, st, out, w)
    assert torch.all(out[0] == 2.0)
    again = torch.empty_like(out)
    c.cache.attention(c.table, c.lens_t, q, again, q_start=i32(st), max_len=max(lens))
    assert torch.equal(again[1:], out[1:])
    c.done()


def test_large_pool_offsets(cb):
    """Blocks beyond 2^32 bytes of the pool: the second layer of a pool of 5 GB, at its last pages."""
    n_pages, H, P, hd = 36000, 2, 256, 128
    codes = torch.zeros((2, 2, n_pages, H, P, hd), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((2, 2, n_pages, H), device="cuda")
    assert codes.numel() // 2 > 2 ** 32
    cache = cb.KV8Cache(codes, scales, n_heads=2 * H)
    rng = np.random.default_rng(1)
    pages = [n_pages - 1, 5, n_pages - 3]
    n = 700
    k = torch.from_numpy(rng.normal(size=(1, n, H, hd)).astype(np.float32)).to(torch.bfloat16).cuda()
    v = torch.from_numpy(rng.normal(size=(1, n, H, hd)).astype(np.float32)).to(torch.bfloat16).cuda()
    table, lens = i32([pages]), i32([n])
    cache.write(table, lens, k, v, layer=1)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    cache.read(table, lens, ko, vo, layer=1)
    q = torch.from_numpy(rng.normal(size=(1, 2 * H, hd)).astype(np.float32)).to(torch.bfloat16).cuda()
    out = cache.attention(table, lens, q, layer=1)
    small = cb.KV8Cache.empty(1, 3, H, P, hd, 2 * H)
    t3 = i32([[2, 0, 1]])
    small.write(t3, lens, k, v)
    ref = small.attention(t3, lens, q)
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    small.read(t3, lens, k2, v2)
    torch.cuda.synchronize()
    assert torch.equal(ko, k2) and torch.equal(vo, v2) and torch.equal(out, ref)
    assert torch.count_nonzero(codes[0]) == 0 and cache.status() == 0
    assert set(torch.nonzero(scales[1].sum(dim=(0, 2))).flatten().tolist()) == set(pages)
    cache.close()
    small.close()


# ------------------------------------------------------------------------------------------------
# eviction
# ------------------------------------------------------------------------------------------------
EVICT = [  # hd, H, P, lens, keep, sink, recent, in place
    (64, 2, 16, [100, 37, 200, 16, 0, 50], 50, 4, 13, False),
    (128, 1, 32, [513, 129], 128, 0, 0, True),
    (128, 2, 64, [300], 70, 70, 0, False),
    (64, 1, 16, [90, 33], 33, 0, 33, True),
    (64, 2, 256, [700, 300], 257, 1, 5, False),
    (128, 1, 16, [1500, 20], 1, 0, 0, False),
    (64, 1, 128, [129], 128, 3, 4, True),
]


@pytest.mark.parametrize("hd,H,P,lens,keep,sink,recent,in_place", EVICT)
def test_evict(cb, hd, H, P, lens, keep, sink, recent, in_place):
    L, top = 3, max(lens)
    need = [-(-min(n, keep) // P) for n in lens]
    c = Case(cb, lens, L=L, H=H, hd=hd, P=P, seed=keep + P, extra=sum(need) + 2)
    w = np.exp(c.rng.normal(size=(2, len(lens), H, top + 2))).astype(np.float32)
    w[0, :, :, 3::4] = 0.25                             # ties on both sides of the threshold
    w[1, :, :, ::3] = 0.0
    w[1, :, :, 1::7] = -1.0
    w[1, 0, 0, 5] = np.nan
    w[:, :, :, 11 % top] = np.inf
    if in_place:
        dst_np, dst = c.table_np, c.table
    else:
        dst_np = np.full((len(lens), max(need)), 10 ** 6, np.int32)
        for s in range(len(lens)):
            for b in range(need[s]):
                dst_np[s, b] = c.free.pop()
        dst = i32(dst_np)
    wt = torch.from_numpy(w).cuda()
    ow = wt if in_place else torch.full_like(wt, 8.0)
    lens_t = c.lens_t.clone()
    rows = torch.full((2, len(lens), H, keep), 77, dtype=torch.int32, device="cuda")
    c.cache.evict(c.table, lens_t, dst, wt, keep, sink, recent, out_rows=rows, out_weights=ow, layer=1, n_layers=2, max_len=top,
                  out_lens=lens_t if in_place else None)
    torch.cuda.synchronize()
    r_rows, r_lens, r_w = c.model.evict(c.table_np, lens, dst_np, w, keep, sink, recent, layer=1)
    assert np.array_equal(rows.cpu().numpy(), r_rows)
    got = ow.cpu().numpy()
    for s, n in enumerate(lens):
        assert np.array_equal(got[:, s, :, :n], r_w[:, s, :, :n], equal_nan=True)
        assert np.array_equal(got[:, s, :, n:], (w if in_place else np.full_like(w, 8.0))[:, s, :, n:], equal_nan=True)
    if in_place:
        assert lens_t.tolist() == r_lens
    c.check_pool()
    c.done()


def test_evict_long_sequence_selects_like_a_sort(cb):
    """30 000 rows with many equal weights: the kept rows against a stable sort."""
    n, keep, sink, recent = 30001, 4096, 4, 100
    cache = cb.KV8Cache.empty(1, 2 * (n // 64 + 1), 2, 64, 64, 4)
    table = torch.arange(n // 64 + 1, dtype=torch.int32, device="cuda")[None]
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(0, 300, (1, 1, 2, n), generator=g, device="cuda").float() / 16
    out = cache.evict(table, i32([n]), table + table.shape[1], w.clone(), keep, sink, recent, max_len=n)
    for h in range(2):
        r = w[0, 0, h].clone()
        r[:sink] = float("inf")
        r[n - recent:] = float("inf")
        want = torch.sort(r, descending=True, stable=True).indices[:keep].sort().values.int()
        assert torch.equal(out["rows"][0, 0, h], want)
        assert torch.equal(out["weights"][0, 0, h, :keep], w[0, 0, h][want.long()])
        assert torch.all(out["weights"][0, 0, h, keep:] == 0)
    assert out["lens"].tolist() == [keep] and cache.status() == 0
    cache.close()


@pytest.mark.parametrize("n", [16384, 16385, 20000])
def test_evict_long_sequence_in_place(cb, n):
    """In place, through a view of the table that is only as wide as what is kept."""
    keep, P = 5000, 64
    cache = cb.KV8Cache.empty(1, n // P + 1, 1, P, 64, 4)
    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.randn((n, 1, 64), generator=g, device="cuda").bfloat16()
    table = torch.randperm(n // P + 1, generator=g, device="cuda").int()[None]
    cache.write(table, i32([n]), k, -k, max_len=n)
    back = [torch.empty_like(k) for _ in range(2)]
    cache.read(table, i32([n]), *back, max_len=n)
    w = torch.randint(0, 2000, (1, 1, 1, n), generator=g, device="cuda").float() / 128
    was, lens = w.clone(), i32([n])
    out = cache.evict(table, lens, table[:, :-(-keep // P)], w, keep, 3, 30, max_len=n, out_lens=lens)
    r = was[0, 0, 0].clone()
    r[:3] = r[n - 30:] = float("inf")
    want = torch.sort(r, descending=True, stable=True).indices[:keep].sort().values
    assert torch.equal(out["rows"][0, 0, 0], want.int()) and lens.tolist() == [keep]
    assert torch.equal(w[0, 0, 0, :keep], was[0, 0, 0, want]) and torch.count_nonzero(w[0, 0, 0, keep:]) == 0
    got = [torch.empty_like(k[:keep]) for _ in range(2)]
    cache.read(table, lens, *got, max_len=n)
    # a value that meets a larger scale is off by half a step at most: 2^-4 of it, or 2^-10 of the scale, which is
    # below 2^-4 here (448 times a scale is less than twice the block's largest value, itself less than 8)
    for a, b in zip(got, back):
        x, y = a.double(), b[want].double()
        assert torch.all((x - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -10 * 2.0 ** -4)
    assert cache.status() == 0
    cache.close()


# ------------------------------------------------------------------------------------------------
# bad ids, streams, devices
# ------------------------------------------------------------------------------------------------
def test_bad_pages_with_many_rows(cb):
    """Keys of bad pages are not seen: the rows give what the remaining keys give."""
    c = Case(cb, [192], H=1, G=4, hd=128, P=16, seed=13, cells=cb.KV8Cache.cells(12, 4, 192))
    bad = c.table.clone()
    bad[0, 2] = 10 ** 6
    bad[0, 5] = -7
    q, q64 = c.values(12, 4, 128)
    out = torch.empty_like(q)
    w = torch.zeros((1, 1, 192), device="cuda")
    c.cache.attention(bad, c.lens_t, q, out, weights=w)
    torch.cuda.synchronize()
    assert c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    assert torch.all(w[0, 0, 32:48] == 0) and torch.all(w[0, 0, 80:96] == 0)
    c.table_np = np.delete(c.table_np, [2, 5], axis=1)
    c.lens = [160]
    check_attention(c, q, q64, [0, 12], out)
    c.done()


def test_bad_ids_are_recorded_not_faulted(cb):
    H, hd, P = 2, 64, 16
    c = Case(cb, [64, 40, 20], H=H, G=2, hd=hd, P=P, seed=12, cells=cb.KV8Cache.cells(3, 4, 64))
    bad = c.table.clone()
    bad[0, 1] = 10 ** 6                                 # rows 16 .. 31 of the first sequence
    bad[1, 2] = -1                                      # the last rows of the second
    q, q64 = c.values(3, 4, hd)
    out = torch.empty_like(q)
    w = torch.zeros((3, H, 64), device="cuda")
    c.cache.attention(bad, c.lens_t, q, out, weights=w, max_len=64)
    torch.cuda.synchronize()
    assert c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    assert torch.all(w[0, :, 16:32] == 0) and torch.all(w[1, :, 32:40] == 0) and torch.isfinite(out).all()
    # what the remaining keys give: the first sequence without its second page
    m = c.model
    ref = km.Model(m.codes, m.scales)
    t2 = c.table_np.copy()
    t2[0, 1:3] = c.table_np[0, 2:4]
    r, _, spread, big = ref.attention(t2, [48, 32, 20], q64, [0, 1, 2, 3], 0, hd ** -0.5)
    tol = 2.0 ** -8 * np.abs(r) + (2 * (hd + 8) * U * big + 2.0 ** -11 + 200 * U) * spread
    assert np.all(np.abs(f64(out) - r) <= tol)
    # lengths above max_len, negative lengths, offsets out of range: skipped, the others as usual
    k, k64 = c.values(1, 3, H, hd)
    lens = i32([65, -2, 20])
    c.cache.write(c.table, lens, k, k, max_len=64)
    m.write(c.table_np, [0, 0, 20], k64, k64, [2, 2, 2, 3])
    torch.cuda.synchronize()
    assert c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    c.check_pool()
    keep = torch.full_like(out, 4.0)
    c.cache.attention(c.table, lens, q, keep, max_len=64)
    c.cache.attention(c.table, c.lens_t, q, keep, q_start=i32([0, 9, -3, 2]), max_len=64)
    torch.cuda.synchronize()
    assert c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    assert torch.all(keep[:2] == 4.0)
    e = c.cache.evict(c.table, lens, c.table, torch.ones((1, 3, H, 64), device="cuda"), 8, max_len=64)
    assert e["lens"][2].item() == 8
    m.evict(c.table_np[2:], [20], c.table_np[2:], np.ones((1, 1, H, 64), np.float32), 8, 0, 0)
    torch.cuda.synchronize()
    assert c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    c.check_pool()
    c.done()


def test_other_stream_and_graph(cb):
    """The call runs on the stream it is given; a captured append + attention follows the lengths and tables that stand
    in its buffers at replay, two graphs sharing one handle."""
    H, G, hd, P = 2, 2, 128, 16
    c = Case(cb, [40, 130], H=H, G=G, hd=hd, P=P, seed=14, spare=20, cells=cb.KV8Cache.cells(2, 4, 150))
    q, _ = c.values(2, 4, hd)
    kv, _ = c.values(1, 2, H, hd)
    lens, out = i32([40, 130]), torch.zeros_like(q)
    w = torch.zeros((2, H, 160), device="cuda")
    graphs = []
    for weights in (None, w):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            c.cache.write(c.table, lens, kv, kv)
            c.cache.attention(c.table, lens, q, out, weights=weights, add=True, max_len=150)
        graphs.append(g)
    total = [np.zeros((H, 160)) for _ in range(2)]
    side = torch.cuda.Stream()
    for step in range(6):
        qq, q64 = c.values(2, 4, hd)
        kk, k64 = c.values(1, 2, H, hd)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            q.copy_(qq)
            kv.copy_(kk)
            lens += 1
            graphs[step % 2].replay()
        c.lens = [n + 1 for n in c.lens]
        c.model.write(c.table_np, c.lens, k64, k64, [0, 1, 2])
        side.synchronize()
        check_attention(c, q, q64, [0, 1, 2], out)
        if step % 2:
            _, ws, _, _ = c.model.attention(c.table_np, c.lens, q64, [0, 1, 2], 0, hd ** -0.5)
            for s in range(2):
                total[s][:, :c.lens[s]] += ws[s]
    for s in range(2):
        assert np.allclose(f64(w)[s], total[s], rtol=1e-4, atol=1e-6)
    other = torch.empty_like(out)
    c.cache.attention(c.table, lens, q, other, max_len=150, stream=side)
    side.synchronize()
    assert torch.equal(other, out)
    c.done()


def test_free_places_of_a_captured_batch(cb):
    """A decoding step captured for four places, of which some are free at each replay: length 0, a table of no pages."""
    H, G, hd, P = 2, 4, 64, 16
    c = Case(cb, [20, 30, 15, 33], H=H, G=G, hd=hd, P=P, seed=41, spare=10, cells=cb.KV8Cache.cells(4, 8, 43))
    kv, kv64 = c.values(1, 4, H, hd)
    q, q64 = c.values(4, H * G, hd)
    lens, table, out = c.lens_t.clone(), c.table.clone(), torch.empty_like(q)
    w, rows, kept = torch.zeros((1, 4, H, 48), device="cuda"), i32(np.zeros((1, 4, H, 40))), i32([0] * 4)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.cache.write(table, lens, kv, kv, max_len=43)
        c.cache.attention(table, lens, q, out, weights=w[0], max_len=43)
        c.cache.evict(table, lens, table, w, 40, 1, 2, out_rows=rows, out_lens=kept, max_len=43)
    now = [20, 30, 15, 33]
    for free in ([1], [0, 2, 3], [], [0, 1, 2, 3], [2]):
        t = c.table_np.copy()
        t[free] = -5
        step = [0 if s in free else now[s] + 1 for s in range(4)]
        lens.copy_(i32(step))
        table.copy_(i32(t))
        out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        c.lens = step
        for s in range(4):
            if s in free:
                assert torch.count_nonzero(out[s]) == 0 and kept[s].item() == 0 and torch.all(rows[0, s] == -1)
            else:
                c.model.write(c.table_np[s:s + 1], step[s:s + 1], kv64[:, s:s + 1], kv64[:, s:s + 1], [0, 1])
                now[s] += 1
                assert kept[s].item() == step[s]
        check_attention(c, q, q64, [0, 1, 2, 3, 4], out)
        for s in set(range(4)) - set(free):             # all rows stay, quantised anew
            c.model.evict(c.table_np[s:s + 1], step[s:s + 1], c.table_np[s:s + 1], np.zeros((1, 1, H, 48), np.float32), 40, 1, 2)
        c.check_pool()
    c.done()


def test_python_refusals(cb):
    c = Case(cb, [40, 20], H=2, G=2, hd=64, P=16, seed=1)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((1, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    a = c.cache
    for f in (lambda: a.attention(c.table.long(), c.lens_t, q), lambda: a.attention(c.table.cpu(), c.lens_t, q),
              lambda: a.attention(c.table, c.lens_t[:1], q), lambda: a.attention(c.table, c.lens_t, q.float()),
              lambda: a.attention(c.table, c.lens_t, q[:, :3]), lambda: a.attention(c.table, c.lens_t, q.transpose(1, 2)),
              lambda: a.attention(c.table, c.lens_t, q, weights=torch.zeros((2, 4, 40), device="cuda")),
              lambda: a.attention(c.table, c.lens_t, q, out=torch.zeros_like(q)[:1]),
              lambda: a.write(c.table, c.lens_t, kv, kv[:, :1]), lambda: a.write(c.table, c.lens_t, kv.cpu(), kv),
              lambda: a.write(c.table, c.lens_t, kv, kv, n_layers=2), lambda: a.write(c.table[:, ::2], c.lens_t, kv, kv),
              lambda: a.evict(c.table, c.lens_t, c.table, torch.zeros((1, 2, 2, 48), device="cuda"), 4, out_rows=i32([1])),
              lambda: a.evict(c.table, c.lens_t, c.table, torch.zeros((2, 2, 48), device="cuda"), 4),
              lambda: cb.KV8Cache(c.codes[:, :, ::2], c.scales, 4), lambda: cb.KV8Cache(c.codes, c.scales[:, :1], 4)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: a.attention(c.table, c.lens_t, q, layer=1), lambda: a.attention(c.table, c.lens_t, q, max_len=49),
              lambda: a.attention(c.table, c.lens_t, q, out=q),
              lambda: a.attention(c.table, c.lens_t, q, weights=torch.zeros((2, 2, 48), device="cuda")),
              lambda: a.write(c.table, c.lens_t, kv[:, :1], kv[:, :1]),
              lambda: a.read(c.table, c.lens_t, kv, kv),
              lambda: a.evict(c.table, c.lens_t, c.table.view(-1)[:4].view(2, 2), torch.zeros((1, 2, 2, 48), device="cuda"), 4),
              lambda: a.evict(c.table, c.lens_t, c.table, torch.zeros((1, 2, 2, 48), device="cuda"), 4, 3, 2)):
        with pytest.raises(cb.CacheBlendError) as ei:
            f()
        assert ei.value.code == cb.CB_ERR_INVALID_ARG
    torch.cuda.synchronize()
    c.check_pool()
    c.done()


# ------------------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("P", [16, 64])
def test_blend_over_the_8bit_pool(cb, P):
    """cb_blend_kv8 is the read, the gradual blend in place and the write, bit for bit; shared pages are only read."""
    import test_gpu_gradual as tg
    w, toks, chunks, caches = tg.tiny5_case()
    ratios = (0.5, 0.35, 0.35, 0.2)
    n_ctx, N = sum(x[2] for x in chunks), len(toks)
    model = cb.BlendModel(tg.TINY5.as_dict(), w, max_tokens=N, max_chunks=len(chunks))
    nb = -(-N // P)
    cache = cb.KV8Cache.empty(5, 3 * nb, 2, P, 64, n_heads=tg.TINY5.n_heads, dtype="f32")
    order = torch.randperm(3 * nb, generator=torch.Generator().manual_seed(P)).to(torch.int32).cuda()
    src, dst = order[:nb].contiguous(), order[nb:2 * nb].contiguous()
    ctx = tg.device_cache(caches, "f32")
    cache.write(src[None, :-(-n_ctx // P)].contiguous(), None, ctx[:, 0], ctx[:, 1], n_layers=5, max_len=n_ctx)
    before = cache.codes[:, :, src.long()].clone()
    t = torch.from_numpy(toks).cuda()
    work, logits = model.kv_buffer(N), torch.empty(1024, device="cuda")
    st = cb.cb_blend_kv8(model.handle, t, N, cache, src, dst, chunks, ratios, work, logits, stats=True)
    ref = model.kv_buffer(N)
    cache.read(src[None].contiguous(), None, ref[:, 0, :n_ctx], ref[:, 1, :n_ctx], n_layers=5, max_len=n_ctx)
    out = model.blend_gradual(t, ref, chunks, ratios, out_kv=ref, stats=True)
    torch.cuda.synchronize()
    assert torch.equal(work, ref) and torch.equal(logits, out["logits"])
    assert st["kernel_launches"] == out["stats"]["kernel_launches"] + 2
    assert torch.equal(cache.codes[:, :, src.long()], before)
    fresh = cb.KV8Cache.empty(5, nb, 2, P, 64, n_heads=tg.TINY5.n_heads, dtype="f32")
    fresh.write(torch.arange(nb, dtype=torch.int32, device="cuda")[None], None, ref[:, 0], ref[:, 1], n_layers=5, max_len=N)
    torch.cuda.synchronize()
    full = N // P                                       # whole pages; the last one's tail was never written
    assert torch.equal(cache.codes[:, :, dst.long()[:full]], fresh.codes[:, :, :full])
    assert torch.equal(cache.scales[:, :, dst.long()], fresh.scales)
    assert model.status() == 0 and cache.status() == 0
    bad = cb.KV8Cache.empty(5, nb, 2, P, 64, n_heads=tg.TINY5.n_heads, dtype="bf16")
    with pytest.raises(cb.CacheBlendError):
        cb.cb_blend_kv8(model.handle, t, N, bad, src, dst, chunks, ratios, work, logits)
    for x in (bad, fresh, cache, model):
        x.close()


def test_prompt_decode_evict_decode(cb):
    """A request's life on the cache: the prompt's rows written, its last rows' window ranks the keys, decoding adds to
    the weights, the cache shrinks in place, decoding goes on in the freed rows; the model follows every step."""
    L, H, G, hd, P, n0, keep = 2, 2, 2, 64, 16, 90, 41
    c = Case(cb, [0, 0], L=L, H=H, G=G, hd=hd, P=P, dtype="f32", seed=30, spare=n0 + 12, cells=cb.KV8Cache.cells(40, 4, 112))
    top, now = 112, [n0, 57]
    st = starts_of(now)
    k, k64 = c.values(L, st[-1], H, hd)
    v, v64 = c.values(L, st[-1], H, hd)
    lens = i32(now)
    c.cache.write(c.table, lens, k, v, n_layers=L, row_start=i32(st), max_len=top)
    c.model.write(c.table_np, now, k64, v64, st)
    w = torch.zeros((L, 2, H, top), device="cuda")
    w64 = np.zeros((L, 2, H, top))

    def attend(rows, add):
        qs = starts_of(rows)
        q, q64 = c.values(qs[-1], H * G, hd)
        for l in range(L):
            out = c.cache.attention(c.table, lens, q, layer=l, q_start=i32(qs), weights=w[l], add=add, max_len=top)
            c.lens = now
            check_attention(c, q, q64, qs, out, layer=l)
            _, ws, _, _ = c.model.attention(c.table_np, now, q64, qs, l, hd ** -0.5)
            for s, n in enumerate(now):
                w64[l, s, :, :n] = ws[s] + (w64[l, s, :, :n] if add else 0)

    def step():
        now[0] += 1
        now[1] += 1
        lens.copy_(i32(now))
        kk, kk64 = c.values(L, 2, H, hd, size=3.0)
        vv, vv64 = c.values(L, 2, H, hd)
        c.cache.write(c.table, lens, kk, vv, n_layers=L, max_len=top)
        c.model.write(c.table_np, now, kk64, vv64, [0, 1, 2])
        attend([1, 1], True)

    attend([24, 16], False)
    for _ in range(4):
        step()
    assert np.allclose(f64(w), w64, rtol=1e-4, atol=1e-7)
    wn = w.cpu().numpy()
    e = c.cache.evict(c.table, lens, c.table, w, keep, 4, 8, out_lens=lens, n_layers=L, max_len=top)
    rows, new_lens, new_w = c.model.evict(c.table_np, now, c.table_np, wn, keep, 4, 8)
    torch.cuda.synchronize()
    assert np.array_equal(e["rows"].cpu().numpy(), rows) and lens.tolist() == new_lens and np.array_equal(w.cpu().numpy(), new_w)
    now[:] = new_lens
    w64 = new_w.astype(np.float64)
    c.check_pool()
    for _ in range(9):
        step()
    assert np.allclose(f64(w), w64, rtol=1e-4, atol=1e-7)
    c.check_pool()
    c.done()
