"""GPU tests of attention over a prefix that sequences share, against the float64 model of tests/kv8_model.py on the joined
keys.

Tolerances are those of tests/test_gpu_kv8.py for attention over the joined keys (its docstring derives them: scores, weights and
fp32 sums, the representation of p with its floors, one rounding of the result).  Joining the two parts multiplies each
by a power of two of a difference of references (ex2.approx, 2 ulp, and the difference's rounding, at most 2^-24 of a
reference's size) and adds them: at most 8 u and ln 2 u of the largest score more on each side, inside the 16 u and the ds
that `limit` already counts twice."""
import numpy as np
import pytest

import kv8_model as km
from test_gpu_kv8 import Case, f64, i32, starts_of

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


@pytest.fixture(params=["one launch", "two launches"], autouse=True)
def path(request, monkeypatch):
    """Both ways of a call: the prefix read again for each sequence in one launch, or once in a launch of its own."""
    monkeypatch.setenv("CB_SHARED_AGAIN", "1e15" if request.param == "one launch" else "-1e15")


class Shared(Case):
    """A Case whose first sequences are the groups' prefixes, the others the batch."""

    def __init__(self, cb, prefixes, lens, first, rows, **kw):
        n_q = sum(rows) + 5
        cells = cb.KV8Cache.shared_cells(n_q, kw.get("H", 2) * kw.get("G", 2), kw.get("hd", 64))
        super().__init__(cb, list(prefixes) + list(lens), cells=cells, **kw)
        self.n_pre, self.own, self.first, self.rows = len(prefixes), list(lens), list(first), list(rows)
        self.pre_table, self.pre_lens = self.table[:self.n_pre].contiguous(), i32(prefixes)
        self.own_table, self.own_lens = self.table[self.n_pre:].contiguous(), i32(lens)
        self.start = starts_of(rows, 2)                 # rows 0, 1 and the last three belong to no sequence
        self.n_q = self.start[-1] + 3

    def run(self, q, out=None, **kw):
        return self.cache.attention_shared(self.pre_table, self.pre_lens, self.own_table, self.own_lens, q, out, prefix_start=i32(self.first),
                                           q_start=i32(self.start), **kw)

    def exact(self, q64, scale, layer=0):
        """out, spread, floors of each row, and the largest sum |q k| scale: row by row over its prefix and own keys."""
        shape = q64.shape
        out, spread, floor, floor_all = (np.zeros(shape) for _ in range(4))
        big = 0.0
        parts = {}
        for g in range(self.n_pre):
            parts["p", g] = self.keys(g, layer)
        for s in range(len(self.own)):
            g = next((g for g in range(self.n_pre) if self.first[g] <= s < self.first[g + 1]), None)
            own = self.keys(self.n_pre + s, layer)
            n, m = self.rows[s], self.own[s]
            for i in range(n):
                seen = max(0, m - n + i + 1)
                use = ([parts["p", g]] if g is not None else []) + [tuple(x[:seen] for x in own)]
                k, v, sv = (np.concatenate([u[j] for u in use]) for j in range(3))
                if not len(k):
                    continue
                r = self.start[s] + i
                for h in range(shape[1]):
                    kv = h // self.G
                    x = k[:, kv] @ q64[r, h] * scale
                    big = max(big, float(np.max(np.abs(k[:, kv]) @ np.abs(q64[r, h]) * abs(scale))))
                    p = np.exp(x - x.max())
                    p /= p.sum()
                    out[r, h], spread[r, h] = p @ v[:, kv], p @ np.abs(v[:, kv])
                    ps, code = p * sv[:, kv], np.abs(v[:, kv]) / np.where(sv[:, kv] > 0, sv[:, kv], 1.0)[:, None]
                    floor_all[r, h] = ps.max() * code.sum(axis=0)
                    at = 0
                    for u in use:                        # tiles of 128 keys begin anew behind the prefix
                        for t in range(0, len(u[0]), 128):
                            e = min(t + 128, len(u[0]))
                            if e > t:
                                floor[r, h] += ps[at + t:at + e].max() * code[at + t:at + e].sum(axis=0)
                        at += len(u[0])
        return out, spread, floor, floor_all, big

    def keys(self, s, layer):
        n = self.lens[s]
        k, v = self.model.rows(self.table_np[s], n, layer)
        sv = np.zeros((n, self.H))
        for b in range(-(-n // self.P)):
            sv[b * self.P:(b + 1) * self.P] = self.model.scales[layer, 1, self.table_np[s][b]]
        return k, v, sv

    def check(self, out, q64, scale=None, layer=0):
        scale = self.hd ** -0.5 if scale is None else scale
        ref, spread, floor, floor_all, big = self.exact(q64, scale, layer)
        ds = (self.hd + 8) * U * big
        bf = self.dtype == "bf16"
        keys = max(self.lens) * 2
        lim = (2 * ds + 16 * U + (128 + keys / 128) * U + (2.0 ** -11 if bf else 2.0 ** -23)) * spread + (2.0 ** -8 if bf else U) * np.abs(ref)
        lim += (2.0 ** -25 if bf else 2.0 ** -37) * floor + (2.0 ** -32 * floor_all if bf else 0.0)
        got = f64(out)
        own = list(range(self.start[0], self.start[-1]))
        err = np.abs(got[own] - ref[own])
        assert (err <= lim[own]).all(), (float(err.max()), float((err - lim[own]).max()))
        return got, own


SHAPES = [
    # prefixes, own lengths, first sequence of each group, rows, and the pool
    ([300], [40, 17, 1], [0, 3], [1, 1, 1], dict(H=2, G=4, hd=128, P=64)),
    ([300, 1, 513], [40, 17, 1, 0, 130, 129, 64], [1, 3, 3, 6], [1, 1, 1, 1, 1, 1, 1], dict(H=2, G=2, hd=64, P=16)),
    ([129, 0], [40, 200, 5, 16], [0, 2, 4], [3, 2, 5, 0], dict(H=1, G=3, hd=128, P=32)),
    ([260], [9, 300], [0, 2], [7, 3], dict(H=2, G=1, hd=64, P=128)),
    ([1000], [70] * 9, [0, 9], [1] * 9, dict(H=1, G=8, hd=128, P=256)),          # 72 columns: the kernel for many rows
    ([700, 90], [40] * 12, [0, 11, 12], [2] * 12, dict(H=2, G=4, hd=64, P=64)),
    ([260], [128, 90, 257], [0, 3], [64, 40, 90], dict(H=1, G=4, hd=128, P=64)),     # many rows of their own too
    ([400], [30, 40, 50, 20], [0, 4], [1, 1, 1, 1], dict(H=2, G=4, hd=64, P=32, dtype="f32")),
    ([150, 33], [30, 1, 50], [0, 1, 3], [5, 1, 4], dict(H=1, G=5, hd=128, P=16, dtype="f32")),
]


@pytest.mark.parametrize("prefixes,lens,first,rows,kw", SHAPES)
def test_shared(cb, prefixes, lens, first, rows, kw):
    """Groups of any size, empty ones, sequences of no group, prefixes and own lengths that end inside tiles and pages, lengths
    of 0 and 1; rows of no sequence stay as they were; the same bits twice."""
    c = Shared(cb, prefixes, lens, first, rows, seed=len(lens) + sum(prefixes), L=2, **kw)
    q, q64 = c.values(c.n_q, c.H * c.G, c.hd)
    out = torch.full_like(q, 9.0)
    assert c.run(q, out, layer=1) is out
    got, own = c.check(out, q64, layer=1)
    rest = [r for r in range(c.n_q) if r not in own]
    assert (got[rest] == 9.0).all()
    again = torch.full_like(q, 9.0)
    c.run(q, again, layer=1)
    assert torch.equal(out, again)
    c.done()


def test_shared_equals_attention_over_joined_pages(cb):
    """A prefix that fills its pages and the sequences' own pages in one table are the same keys for cb_kv8_attention: both
    results are within their roundings of each other; with no prefix the results are the same bits."""
    P = 64
    c = Shared(cb, [4 * P], [70, 128, 1], [0, 3], [2, 2, 1], H=2, G=4, hd=128, P=P, seed=4)
    q, q64 = c.values(c.n_q, 8, 128)
    joined = torch.cat((c.pre_table[:, :4].expand(3, -1), c.own_table), dim=1).contiguous()
    lens = c.own_lens + 4 * P
    a = c.cache.attention(joined, lens, q, q_start=i32(c.start), max_len=128 + 4 * P)
    b = c.run(q, max_len=128)
    c.check(b, q64)
    c.check(a, q64)
    assert (a - b).abs().max() <= 2.0 ** -7 * a.abs().max()
    for kw in (dict(prefix_max_len=0), dict()):
        empty = c.pre_table[:0] if not kw else c.pre_table
        none = c.cache.attention_shared(empty, None, c.own_table, c.own_lens, q, q_start=i32(c.start), prefix_start=i32([0, 3][:len(empty) + 1]), **kw)
        assert torch.equal(none, c.cache.attention(c.own_table, c.own_lens, q, q_start=i32(c.start)))
    c.done()


@pytest.mark.parametrize("n,rows", [(6, 1), (8, 9)])
def test_shared_scores_far_apart(cb, n, rows):
    """A prefix whose largest score lies far above or below that of the own keys, and V scales far apart in the two parts."""
    for up in (40.0, -40.0):
        c = Shared(cb, [200], [150] * n, [0, n], [rows] * n, H=1, G=2, hd=64, P=16, seed=int(up) + 50)
        pre = set(int(x) for x in c.table_np[0][:-(-200 // 16)])
        for pg in range(c.model.n_pages):
            f = 2.0 ** (6 if (pg in pre) == (up > 0) else -2)
            c.model.scales[0, 0, pg] *= f
            c.model.scales[0, 1, pg] *= 2.0 ** (20 if pg in pre else -20)
        c.scales.copy_(torch.from_numpy(c.model.scales.astype(np.float32)))
        q, q64 = c.values(c.n_q, 2, 64)
        c.check(c.run(q), q64)
        c.done()


@pytest.mark.parametrize("G,n", [(2, 3), (8, 12)])
def test_shared_nan(cb, G, n):
    """NaN behind what a row sees does not reach it; NaN in a seen V of the prefix reaches the group's rows in its dims; a NaN or
    an infinity in a row of q makes that head NaN."""
    c = Shared(cb, [130, 40], [20 + s for s in range(n)], [0, n - 1, n], [1] * n, H=1, G=G, hd=64, P=16, seed=9)
    pg, row = int(c.table_np[0][130 // 16]), 130 % 16
    codes = c.codes.clone()
    codes[0, 1, int(c.table_np[0][3]), 0, 5, 7] = 0x7F
    c.codes.copy_(codes)
    assert (codes[0, 0, pg, 0, row:] == 0x7F).all()               # behind the prefix's last row: NaN, and not seen
    q, q64 = c.values(c.n_q, G, 64)
    r = c.start[1]
    q[r, G - 1, 3] = float("nan")
    q[r + 1, 0, 3] = float("inf")
    got = f64(c.run(q))
    own = np.array(range(c.start[0], c.start[-1]))
    nan = np.isnan(got[own])
    want = np.zeros_like(nan)
    want[:n - 1, :, 7] = True
    want[1, G - 1] = want[2, 0] = True
    assert np.array_equal(nan, want)
    c.done()


def test_shared_bad_ids_and_lengths(cb):
    """Bad pages' keys are not seen, a prefix of a bad length has no rows; offsets that decrease compute nothing; all are recorded."""
    c = Shared(cb, [100, 60], [30, 20, 40], [0, 2, 3], [1, 2, 1], H=1, G=2, hd=64, P=16, seed=6)
    q, q64 = c.values(c.n_q, 2, 64)
    ref_none = c.cache.attention(c.own_table, c.own_lens, q, q_start=i32(c.start))
    good = c.run(q)
    assert c.cache.status() == 0
    bad = c.pre_lens.clone()
    bad[0] = 10 ** 6
    out = c.cache.attention_shared(c.pre_table, bad, c.own_table, c.own_lens, q, prefix_start=i32(c.first), q_start=i32(c.start), prefix_max_len=112)
    torch.cuda.synchronize()
    assert c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    a, b = c.start[0], c.start[2]
    assert torch.allclose(out[a:b].float(), ref_none[a:b].float(), rtol=2.0 ** -7, atol=0) and torch.equal(out[b:c.start[3]], good[b:c.start[3]])
    table = c.pre_table.clone()
    table[0] = -1
    out = c.cache.attention_shared(table, c.pre_lens, c.own_table, c.own_lens, q, prefix_start=i32(c.first), q_start=i32(c.start))
    torch.cuda.synchronize()
    assert c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    assert torch.allclose(out[a:b].float(), ref_none[a:b].float(), rtol=2.0 ** -7, atol=0)
    for first, start in (([0, 3, 2], c.start), ([0, 2, 4], c.start), ([-1, 2, 3], c.start), (c.first, [2, 4, 3, 6]), (c.first, [2, 3, 5, 90])):
        out = torch.full_like(q, 9.0)
        c.cache.attention_shared(c.pre_table, c.pre_lens, c.own_table, c.own_lens, q, out, prefix_start=i32(first), q_start=i32(start))
        torch.cuda.synchronize()
        assert (out == 9.0).all() and c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    assert torch.equal(c.run(q), good)
    c.done()


def test_shared_graph_follows_lengths(cb):
    """A captured call follows lengths, tables and group offsets; an eager call of the same handle in between changes nothing."""
    n = 6
    c = Shared(cb, [200, 90], [60] * n, [0, 4, n], [1] * n, H=2, G=4, hd=64, P=16, seed=3, spare=8)
    q, q64 = c.values(c.n_q, 8, 64)
    first, start = i32(c.first), i32(c.start)
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call():
        c.cache.attention_shared(c.pre_table, c.pre_lens, c.own_table, c.own_lens, q, out, prefix_start=first, q_start=start, stream=side)
    call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for pre, lens, groups in (([200, 90], [60] * n, [0, 4, n]), ([17, 1], [1, 60, 33, 2, 16, 59], [0, 1, n]), ([150, 90], [60] * n, [2, 4, 5])):
        c.lens, c.own, c.first = pre + lens, lens, groups
        c.pre_lens.copy_(i32(pre))
        c.own_lens.copy_(i32(lens))
        first.copy_(i32(groups))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, q64)
        c.cache.attention(c.own_table, c.own_lens, q, q_start=start)
    c.done()


@pytest.mark.parametrize("G,dtype,rows", [(7, "f32", [1950, 3]), (5, "f32", [2700, 1]), (1, "f32", [9, 66000]), (7, "bf16", [1900] + [1] * 500)])
def test_shared_one_sequence_of_many_rows(cb, G, dtype, rows):
    """A batch of few rows on average in which one sequence has more columns (rows x heads of a group) than small divisions reach: the
    results are those of attention over joined pages.  Both lie within 2 (hd + 8) 2^-24 sum |q k| scale of the scores (at most 60 here) and
    170 2^-24 more of the values' spread, 2^-9 in all, and in bf16 calls within another 2^-8 of the value; a row in another's place
    differs by the values themselves."""
    P, pre = 64, 128
    lens = [max(n, 20) for n in rows]
    L = max(lens)
    n_q, width = sum(rows), -(-L // P)
    rng = np.random.default_rng(G)
    pages = -(-pre // P) + sum(-(-n // P) for n in lens)
    codes = torch.from_numpy(rng.integers(0, 112, (1, 2, pages, 1, P, 64)).astype(np.uint8) | (rng.integers(0, 2, (1, 2, pages, 1, P, 64)) * 128).astype(np.uint8)).cuda()
    scales = torch.full((1, 2, pages, 1), 2.0 ** -7, device="cuda")
    table = np.zeros((len(lens), width), np.int32)
    at = -(-pre // P)
    for s, n in enumerate(lens):
        table[s, :-(-n // P)] = np.arange(at, at - (-n // P))
        at += -(-n // P)
    cache = cb.KV8Cache(codes, scales, n_heads=G, dtype=dtype, weight_cells=cb.KV8Cache.shared_cells(n_q, G, 64))
    q = torch.from_numpy(rng.normal(size=(n_q, G, 64)).astype(np.float32)).cuda().to(cache.dtype)
    start, own, t = i32(starts_of(rows, 0)), i32(lens), i32(table)
    head = i32(np.arange(pre // P)[None])
    a = cache.attention_shared(head, i32([pre]), t, own, q, torch.zeros_like(q), q_start=start)
    b = cache.attention(torch.cat((head.expand(len(lens), -1), t), dim=1).contiguous(), own + pre, q, torch.zeros_like(q), q_start=start)
    torch.cuda.synchronize()
    assert cache.status() == 0
    assert (a.float() - b.float()).abs().max() <= (2.0 ** -8 if dtype == "f32" else 2.0 ** -6) * b.float().abs().max()
    cache.close()


def test_shared_after_calls_of_other_sizes(cb):
    """What an earlier call of other sizes left in the cache's scratch does not reach a result (here 27 tiles of the prefix, whose items
    span CTAs, after calls with more)."""
    lens, rows = [19, 178, 167, 9, 176, 140, 127], [29, 19, 32, 1, 8, 14, 29]
    c = Shared(cb, [256], [max(a, b) for a, b in zip(lens, rows)], [0, 7], rows, H=3, G=2, hd=128, P=64, seed=21)
    q, q64 = c.values(c.n_q, 6, 128)
    for _ in range(2):
        c.check(c.run(q), q64)
        c.cache.attention(c.own_table, c.own_lens, q, q_start=i32(c.start))
        c.cache.attention(c.table[:1], i32([256]), q)
        c.cache.attention_shared(c.pre_table, i32([200]), c.own_table, c.own_lens, q, prefix_start=i32([2, 5]), q_start=i32(c.start))
    c.done()


def test_shared_right_behind_what_it_reads(cb):
    """Captured steps without a wait between them, each of which lengthens the sequences, appends their rows and attends at once: the
    same bits as when every call is waited for.  (The launch over the own keys starts before the launch over the prefix ends.)"""
    n, steps, P = 64, 10, 64
    c = Shared(cb, [1500, 700], [130 + s for s in range(n)], [0, 40, n], [1] * n, H=4, G=4, hd=128, P=P, seed=12, spare=64)
    kv = [c.values(n, 4, 128)[0] for _ in range(2 * steps)]
    qs = [c.values(n, 16, 128)[0] for _ in range(steps)]
    first, most = i32(c.first), 130 + n + steps
    codes, scales, lens = c.codes.clone(), c.scales.clone(), c.own_lens.clone()
    outs = [torch.zeros_like(x) for x in qs]
    side = torch.cuda.Stream()

    def step(i, wait):
        c.own_lens.add_(1)
        wait()
        c.cache.append(c.own_table, c.own_lens, None, kv[2 * i], kv[2 * i + 1], 1e4, max_len=most, stream=side)
        wait()
        c.cache.attention_shared(c.pre_table, c.pre_lens, c.own_table, c.own_lens, qs[i], outs[i], prefix_start=first, max_len=most, stream=side)
        wait()

    def back():
        for a, b in ((c.codes, codes), (c.scales, scales), (c.own_lens, lens)):
            a.copy_(b)
        torch.cuda.synchronize()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for i in range(steps):
            step(i, side.synchronize)
    want = [o.clone() for o in outs]
    back()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for i in range(steps):
            step(i, lambda: None)
    for _ in range(5):
        back()
        for o in outs:
            o.fill_(9.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert c.cache.status() == 0
    c.done()


def test_shared_python_refusals(cb):
    c = Shared(cb, [40], [20, 20], [0, 2], [1, 1], H=1, G=2, hd=64, P=16)
    q, _ = c.values(c.n_q, 2, 64)
    call = dict(prefix_start=i32([0, 2]), q_start=i32(c.start))
    with pytest.raises(ValueError, match="prefix_start"):
        c.cache.attention_shared(c.pre_table, c.pre_lens, c.own_table, c.own_lens, q, prefix_start=i32([0, 1, 2]), q_start=i32(c.start))
    with pytest.raises(ValueError, match="lens"):
        c.cache.attention_shared(c.pre_table, c.own_lens, c.own_table, c.own_lens, q, **call)
    with pytest.raises(ValueError, match="out must have"):
        c.cache.attention_shared(c.pre_table, c.pre_lens, c.own_table, c.own_lens, q, q[:2].clone(), **call)
    with pytest.raises(cb.CacheBlendError, match="cells"):
        big = torch.zeros((c.n_q + 1, 2, 64), dtype=q.dtype, device="cuda")
        c.cache.attention_shared(c.pre_table, c.pre_lens, c.own_table, c.own_lens, big, **call)
    c.done()
