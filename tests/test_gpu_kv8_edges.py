"""GPU tests of the 8-bit paged K/V cache at the edges of what its calls accept: values of any finite size in q, K and
V, keys that cannot be read, offsets and lengths out of order, outputs that a call makes on a stream of its own.  The
model, the cases and the attention tolerances are those of test_gpu_kv8.py; what a test adds to them is derived at it."""
import numpy as np
import pytest

import kv8_model as km
from test_gpu_kv8 import Case, U, cb, check_attention, f64, i32, starts_of                  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def set_pool(c):
    """The model's pool onto the device."""
    c.codes.copy_(torch.from_numpy(c.model.codes))
    c.scales.copy_(torch.from_numpy(c.model.scales.astype(np.float32)))


def attend(c, rows, size=1.0, q=None, weights=True):
    """One call with `rows` query rows per sequence, checked against the model."""
    n, heads = rows * len(c.lens), c.H * c.G
    if q is None:
        q, _ = c.values(n, heads, c.hd, size=size)
    out = torch.full_like(q, 9.0)
    w = torch.zeros((len(c.lens), c.H, max(c.lens)), device="cuda") if weights else None
    c.cache.attention(c.table, c.lens_t, q, out, weights=w, max_len=max(c.lens))
    check_attention(c, q, f64(q), [rows * s for s in range(len(c.lens) + 1)], out, w)
    return q, out, w


def v_scales(c, s, j0, j1, value):
    """V's scale of the blocks that hold rows j0 .. j1 - 1 of sequence s."""
    for b in range(j0 // c.P, -(-j1 // c.P)):
        c.model.scales[0, 1, c.table_np[s, b]] = value


# every kernel: query columns of 4, 8, 16 and 32, fp32 ones of 4 and 8, and many rows
KERNELS = [("bf16", 1), ("bf16", 2), ("bf16", 4), ("bf16", 8), ("f32", 1), ("f32", 2), ("bf16", 40)]


@pytest.mark.parametrize("dtype,rows", KERNELS)
@pytest.mark.parametrize("ahead,scale", [(130, 2.0 ** -3), (130, 4.0), (90, 2.0 ** 20), (170, 2.0 ** 20), (230, 2.0 ** 100)])
def test_attention_first_key_far_ahead(cb, dtype, rows, ahead, scale):
    """A first key whose score is `ahead` octaves (a factor 2^ahead in weight) above the others', whose V blocks have large
    scales: what vanishes beside it is 0 and not 0 times an overflow.  With (230, 2^100) a weight is below the smallest
    number of fp32."""
    n, hd = 400, 64
    c = Case(cb, [n], H=1, G=4, hd=hd, P=16, dtype=dtype, seed=rows, cells=cb.KV8Cache.cells(rows, 4, n))
    m = c.model
    m.scales[0, 0] = 2.0 ** -9
    m.codes[0, 0, :, :, :, 0] = 0
    m.codes[0, 0, c.table_np[0, 0], 0, 0, 0] = 0x7E     # 448 * 2^-9 = 0.875 in the first key's first channel
    v_scales(c, 0, 0, 128, 2.0 ** -3)
    v_scales(c, 0, 128, n, scale)
    # in the last page only the last row is not 0: its scale is another one, and most rows do not see what it stands for
    m.codes[0, 1, c.table_np[0, n // 16 - 1], :, :15] = 0
    v_scales(c, 0, n - 16, n, scale * 2.0 ** 6)
    set_pool(c)
    q, _ = c.values(rows, 4, hd)
    q[:, :, 0] = ahead * np.log(2.0) * 8 / 0.875
    attend(c, rows, q=q)
    c.done()


def largest_values(cb, dtype, rows, n):
    c = Case(cb, [n], H=1, G=4, hd=64, P=32, dtype=dtype, seed=rows, cells=cb.KV8Cache.cells(rows, 4, n))
    for scale in (2.0 ** 120, 2.0 ** 119, 2.0 ** 70):
        c.model.scales[0, 1] = scale
        set_pool(c)
        attend(c, rows)
    c.model.codes[0, 1, c.table_np[0]] &= 0x7F           # all of one sign: nothing cancels
    c.model.scales[0, 1] = 2.0 ** 120
    set_pool(c)
    attend(c, rows)
    c.done()


@pytest.mark.parametrize("dtype,rows", KERNELS[:-1])
@pytest.mark.parametrize("n", [300, 5000])
def test_attention_largest_values(cb, dtype, rows, n):
    """V near the largest finite number (codes up to 120 at a scale of 2^120): means of such values are finite, whatever the
    number of keys, and as exact as any other."""
    largest_values(cb, dtype, rows, n)


@pytest.mark.parametrize("dtype,rows", KERNELS)
@pytest.mark.parametrize("n", [100, 3000])
def test_rows_that_see_only_bad_pages(cb, dtype, rows, n):
    """Keys of bad pages are not seen, and a row that sees nothing gives 0: a whole sequence of bad pages, and one whose first
    pages are bad, so that its first rows see nothing; items of one CTA and of many."""
    H, G, hd, P = 2, 4, 64, 16
    c = Case(cb, [n, rows + 5, n], H=H, G=G, hd=hd, P=P, dtype=dtype, seed=rows, cells=cb.KV8Cache.cells(3 * rows, H * G, n))
    bad = c.table.clone()
    bad[0] = -1
    blind = min(rows, max(0, P - 5))                     # rows of the second sequence at positions below P
    bad[1, 0] = 10 ** 6
    q, q64 = c.values(3 * rows, H * G, hd)
    out = torch.full_like(q, 9.0)
    w = torch.full((3, H, n), 5.0, device="cuda")
    c.cache.attention(bad, c.lens_t, q, out, weights=w, max_len=n)
    torch.cuda.synchronize()
    assert c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    got, wg = f64(out), f64(w)
    assert not got[:rows].any() and not got[rows:rows + blind].any()
    assert not wg[0].any() and not wg[1, :, :min(P, rows + 5)].any()
    # the rows that see something: the second sequence without its first page, and the third as it is
    c.table_np = np.concatenate([c.table_np[:1], np.roll(c.table_np[1:2], -1, axis=1), c.table_np[2:]])
    c.lens = [n, max(0, rows + 5 - P), n]
    st = [0, rows, 2 * rows, 3 * rows]
    ref, ws, spread, big = c.model.attention(c.table_np, c.lens, q64, st, 0, hd ** -0.5)
    lo = rows + blind
    p_rep, rnd, last = (2.0 ** -11, 2.0 ** -8, 2.0 ** -25) if dtype == "bf16" else (2.0 ** -23, 2.0 ** -24, 2.0 ** -37)
    tol = rnd * np.abs(ref) + (2 * (hd + 8) * U * big + (144 + n / 128) * U + p_rep) * spread + last * c.model.floor + \
        2.0 ** -32 * c.model.floor_all
    assert np.all(np.abs(got - ref)[lo:] <= tol[lo:] + 1e-30)
    assert np.allclose(wg[2], ws[2], rtol=1e-4, atol=1e-12)
    assert np.allclose(wg[1, :, P:rows + 5], ws[1], rtol=1e-4, atol=1e-12)
    c.done()


@pytest.mark.parametrize("dtype,rows", KERNELS)
def test_queries_with_infinities_and_nan(cb, dtype, rows):
    """An infinity or a NaN in a query head's row makes that result NaN, and no other."""
    n = 200
    c = Case(cb, [n], H=2, G=4, hd=64, P=16, dtype=dtype, seed=rows, cells=cb.KV8Cache.cells(rows, 8, n))
    codes = c.model.codes[0, 0, c.table_np[0]]
    c.model.codes[0, 0, c.table_np[0]] = np.where((codes & 0x7F) == 0x7F, codes, codes & 0x7F | 0x08)
    # (keys above 0: against an infinite q every score would be -inf, as if nothing were seen)
    set_pool(c)
    q, _ = c.values(rows, 8, 64)
    r = rows - 1
    q[r, 1, :] = -float("inf")
    q[0, 2, 7] = float("nan")
    q[r, 6, 3] = float("inf")
    out, w = torch.empty_like(q), torch.zeros((1, 2, n), device="cuda")
    c.cache.attention(c.table, c.lens_t, q, out, weights=w, max_len=n)
    want = np.zeros((rows, 8), bool)
    want[r, 1] = want[0, 2] = want[r, 6] = True
    got = f64(out)
    assert np.array_equal(np.isnan(got), np.repeat(want[:, :, None], 64, axis=2))
    clean = torch.where(torch.isfinite(q), q, torch.zeros_like(q))
    ref = torch.empty_like(q)
    c.cache.attention(c.table, c.lens_t, clean, ref, max_len=n)
    keep = torch.from_numpy(want).cuda()[:, :, None]
    check_attention(c, clean, f64(clean), [0, rows], torch.where(keep, ref, out))
    assert torch.isnan(w[0]).all()
    c.done()


@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("bf16", 8), ("bf16", 9), ("f32", 3)])
def test_attention_tiny_queries(cb, dtype, rows):
    """Rows of q from the smallest numbers up, on either side of 32 columns: their scores are next to 0 and their weights
    next to equal."""
    sizes = (1e-36, 1e-39, 2e-37, 0.0, 1.0, 1e-30, 3e-36, 8e-35)
    c = Case(cb, [260], H=1, G=4, hd=64, P=16, dtype=dtype, seed=rows, cells=cb.KV8Cache.cells(rows, 4, 260))
    for first in range(0, len(sizes), 4):
        x = c.rng.normal(size=(rows, 4, 64))
        for r in range(rows):
            for h in range(4):
                x[r, h] *= sizes[(first + r * 4 + h) % len(sizes)]
        x[:, :, 5] = 0.0
        attend(c, rows, q=torch.from_numpy(x.astype(np.float32)).to(c.td).cuda())
    c.done()


@pytest.mark.parametrize("dtype,rows", KERNELS)
@pytest.mark.parametrize("n", [200, 4000])
@pytest.mark.parametrize("low,high", [(0.0, 2.0 ** 30), (0.0, 2.0 ** 120), (2.0 ** -90, 2.0 ** 40), (2.0 ** -126, 2.0 ** 100),
                                      (2.0 ** -90, 2.0 ** -90), (2.0 ** 110, 2.0 ** 110)])
def test_attention_scales_far_apart(cb, dtype, rows, n, low, high):
    """V blocks of very different sizes beside each other: half of the keys low, half high, in one order and the other, and
    in turn.  Each key's weight counts in the sum whatever its V."""
    c = Case(cb, [n], H=1, G=4, hd=64, P=16, dtype=dtype, seed=rows, cells=cb.KV8Cache.cells(rows, 4, n))
    was = c.model.codes.copy()
    h = n // 2 // 16 * 16
    for order in range(3):
        c.model.codes = was.copy()
        v_scales(c, 0, 0, h, (low, high, high)[order])
        v_scales(c, 0, h, n, (high, low, low)[order])
        if order == 2:
            for b in range(0, -(-n // 16), 2):
                v_scales(c, 0, 16 * b, 16 * b + 16, low)
        zero = c.model.scales[0, 1] == 0                 # a block whose scale is 0 holds zeros
        c.model.codes[0, 1][zero] = 0
        set_pool(c)
        attend(c, rows)
    c.done()


@pytest.mark.parametrize("gap", [60, 100])
@pytest.mark.parametrize("dtype,rows", KERNELS)
def test_attention_large_v_behind_a_small_weight(cb, dtype, rows, gap):
    """Keys of a weight 2^-gap, beside one of weight 1, whose V is as much larger: both count in the result."""
    n, hd = 200, 64
    for top, rest in ((2.0 ** -100, 2.0 ** (gap - 100)), (1.0, 2.0 ** gap), (2.0 ** 15, 2.0 ** 115)):
        c = Case(cb, [n], H=1, G=4, hd=hd, P=16, dtype=dtype, seed=rows, cells=cb.KV8Cache.cells(rows, 4, n))
        m = c.model
        m.scales[0, 0] = 2.0 ** -9
        m.codes[0, 0, :, :, :, 0] = 0
        m.codes[0, 0, c.table_np[0, 0], 0, 0, 0] = 0x7E
        v_scales(c, 0, 0, 16, top)
        v_scales(c, 0, 16, n, rest)
        m.codes[0, 1, c.table_np[0, 0], 0, 1:] = 0       # in the first block only the first key's V
        set_pool(c)
        q, _ = c.values(rows, 4, hd)
        q[:, :, 0] = gap * np.log(2.0) * 8 / 0.875
        attend(c, rows, q=q)
        c.done()


@pytest.mark.parametrize("n", [300, 5000])
def test_many_rows_largest_values(cb, n):
    largest_values(cb, "bf16", 40, n)


def busy(ms_of_work=16):
    """Work that keeps the current stream busy for some milliseconds."""
    x = torch.ones(1 << 28, device="cuda")
    for _ in range(3 * ms_of_work):
        x.add_(1.0)
    return x


@pytest.mark.parametrize("rows", [1, 40])
def test_outputs_made_by_a_call_on_a_stream(cb, rows):
    """out left to the call, on another stream than the current one, which has work to do: rows of no sequence are 0, the
    others are what the call gives on the current stream."""
    c = Case(cb, [150, 90], H=2, G=4, hd=64, P=16, seed=rows)
    n = 2 * rows + 3
    q, _ = c.values(n, 8, 64)
    st = i32([1, 1 + rows, 1 + 2 * rows])
    want = c.cache.attention(c.table, c.lens_t, q, q_start=st)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        # blocks that the allocator may give out again, full of NaN
        trash = [torch.full_like(q, float("nan")) for _ in range(4)]
        torch.cuda.synchronize()
        del trash
        keep = busy()
        out = c.cache.attention(c.table, c.lens_t, q, q_start=st, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.count_nonzero(out[0]) == 0 and torch.count_nonzero(out[-2:]) == 0
        del keep
    c.done()


def test_evict_outputs_made_by_a_call_on_a_stream(cb):
    """Blocks that the current stream still writes are not handed to another stream's eviction."""
    c = Case(cb, [150, 90], H=2, G=4, hd=64, P=16, seed=3)
    w = torch.rand((1, 2, 2, 160), device="cuda")
    side = torch.cuda.Stream()
    want = None
    for stream in (None, side, side.cuda_stream):
        ow = torch.empty_like(w)
        t, held = torch.empty(25000, dtype=torch.int32, device="cuda"), []
        was = torch.cuda.memory_reserved()
        while torch.cuda.memory_reserved() == was:       # so that t's is the smallest free block
            held.append(torch.empty(128, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        keep = busy() if stream is not None else None
        t.fill_(-77)                                     # behind that work
        del t
        e = c.cache.evict(c.table, c.lens_t, c.table, w, 40, 2, 5, out_weights=ow, stream=stream)
        torch.cuda.synchronize()
        got = [e["rows"].clone(), e["lens"].clone()]
        if want is None:
            want = got
        set_pool(c)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del keep, e, held
    c.done()


@pytest.mark.parametrize("rows", [4, 40])
def test_offsets_that_decrease(cb, rows):
    """Offsets that go back would give rows to two sequences: nothing is computed and the call is recorded."""
    lens = [100, 60, 300, 80]
    c = Case(cb, lens, H=2, G=4, hd=64, P=16, seed=rows, cells=cb.KV8Cache.cells(2 * rows, 8, 300))
    q, q64 = c.values(2 * rows, 8, 64)
    for st in ([0, rows, 0, rows, 2 * rows], [0, 2 * rows, rows, rows, 2 * rows], [5, 4, 4, 4, 4]):
        out = torch.full_like(q, 3.0)
        w = torch.full((4, 2, 300), 6.0, device="cuda")
        c.cache.attention(c.table, c.lens_t, q, out, q_start=i32(st), weights=w, max_len=300)
        torch.cuda.synchronize()
        assert c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
        assert torch.all(out == 3.0) and torch.all(w == 6.0)
    # the next call is as any other
    st, out = [0, rows, rows, rows + 2, 2 * rows], torch.empty_like(q)
    w = torch.zeros((4, 2, 300), device="cuda")
    c.cache.attention(c.table, c.lens_t, q, out, q_start=i32(st), weights=w, max_len=300)
    check_attention(c, q, q64, st, out, w)
    # offsets that pass the number of rows without going back: those sequences are skipped, the others computed
    out = torch.full_like(q, 3.0)
    c.cache.attention(c.table, c.lens_t, q, out, q_start=i32([0, rows, rows + 2, 2 * rows + 1, 2 * rows + 7]), max_len=300)
    torch.cuda.synchronize()
    assert c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    ref = torch.empty_like(q[:rows + 2])
    c.cache.attention(c.table[:2].contiguous(), c.lens_t[:2].contiguous(), q[:rows + 2], ref, q_start=i32([0, rows, rows + 2]), max_len=300)
    torch.cuda.synchronize()
    assert torch.allclose(out[:rows + 2].float(), ref.float(), rtol=2.0 ** -7, atol=1e-6) and torch.all(out[rows + 2:] == 3.0)
    c.done()


@pytest.mark.parametrize("start", [[0, 64, 0, 8], [0, 64, 64, 1], [9, 8, 8, 8]])
def test_write_and_read_record_offsets_that_decrease(cb, start):
    c = Case(cb, [64, 64, 64], H=2, hd=64, P=16, seed=3)
    k, _ = c.values(1, 64, 2, 64)
    for f in (c.cache.write, c.cache.read):
        f(c.table, c.lens_t, k, k.clone(), row_start=i32(start))
        torch.cuda.synchronize()
        assert c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    c.done()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_largest_finite_values_stay_finite(cb, dtype):
    """A scale of 2^120 ends at the code 240, the last whose value is finite: values above 248 * 2^120 round to it.  Written
    as whole pages and appended to a block that has that scale, or a smaller one, already."""
    P, H, hd = 16, 2, 64
    c = Case(cb, [3 * P], H=H, hd=hd, P=P, dtype=dtype, seed=2)
    top = float(torch.finfo(c.td).max)
    x = c.rng.uniform(2.0 ** 126, top, size=(1, 3 * P, H, hd)) * c.rng.choice([-1, 1], size=(1, 3 * P, H, hd))
    x[0, 0, 0, :4] = top, -top, 247.9 * 2.0 ** 120, -248.1 * 2.0 ** 120
    x[0, 1, 1, :2] = np.nan, np.inf
    x[0, P:P + 7] *= 2.0 ** -30
    t = torch.from_numpy(x.astype(np.float32)).to(c.td)
    t[0, 2, 0, 0] = top                                  # (as the type rounds it, not beyond)
    t = torch.where(torch.isinf(t) & torch.tensor(np.isfinite(x)), torch.sign(t) * top, t).cuda()
    x = f64(t)
    lens = []
    for n, m in ((P + 7, P + 7), (3 * P, 2 * P - 7)):     # the second call's rows begin inside the second page
        c.cache.write(c.table, i32([n]), t[:, n - m:n].contiguous(), t[:, n - m:n].contiguous(), max_len=3 * P)
        lens.append(n)
    ko, vo = torch.zeros_like(t), torch.zeros_like(t)
    c.cache.read(c.table, i32([3 * P]), ko, vo, max_len=3 * P)
    torch.cuda.synchronize()
    want = np.zeros_like(x)
    for b in range(3):
        for h in range(H):
            rows = x[0, b * P:(b + 1) * P, h]
            parts = [rows] if b != 1 else [rows[:7], rows[7:]]
            was = 0.0
            done = np.zeros((0, hd))
            for p in parts:
                s = max(km.scale_of(p), was)
                if was:
                    done = km.VALUES[km.encode(done / s)] * s
                limit = 240.0 if s == 2.0 ** 120 else 448.0
                new = km.VALUES[km.encode(np.clip(km.divide(p, s), -limit, limit))] * s
                done, was = np.concatenate([done, new]), s
            want[0, b * P:(b + 1) * P, h] = done
    for got in (f64(ko), f64(vo)):
        assert np.array_equal(got, want, equal_nan=True)
    assert np.isfinite(want).sum() == want.size - 2 and (np.abs(want) == 240 * 2.0 ** 120).sum() > 10
    c.done()


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_with_lengths_out_of_range(cb, in_place):
    """A sequence whose length is out of range is recorded and keeps nothing: 0 rows, -1 for each, whatever stood in the
    outputs before."""
    lens = [65, 50, -3, 20]
    c = Case(cb, [64, 50, 30, 20], H=2, hd=64, P=16, seed=7, extra=12)
    dst = c.table if in_place else i32(np.array(c.free[:12]).reshape(4, 3))
    w = torch.rand((1, 4, 2, 64), device="cuda")
    w0 = w.cpu().numpy()
    rows, new = torch.full((1, 4, 2, 33), 12345, dtype=torch.int32, device="cuda"), i32([9, 9, 9, 9])
    c.cache.evict(c.table, i32(lens), dst, w, 33, 1, 2, out_rows=rows, out_lens=new, max_len=64)
    torch.cuda.synchronize()
    assert c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    assert new.tolist() == [0, 33, 0, 20]
    assert torch.all(rows[:, 0] == -1) and torch.all(rows[:, 2] == -1)
    assert np.array_equal(w.cpu().numpy()[:, [0, 2]], w0[:, [0, 2]])
    tab = c.table_np if in_place else np.array(c.free[:12]).reshape(4, 3)
    for s in (1, 3):
        r, _, nw = c.model.evict(c.table_np[s:s + 1], lens[s:s + 1], tab[s:s + 1], w0[:, s:s + 1], 33, 1, 2)
        assert np.array_equal(rows[:, s:s + 1].cpu().numpy(), r) and np.array_equal(w[:, s:s + 1].cpu().numpy(), nw)
    c.check_pool()
    # the lengths themselves as the output
    ln = i32(lens)
    c.cache.evict(c.table, ln, c.table, w, 33, 1, 2, out_lens=ln, max_len=64)
    torch.cuda.synchronize()
    assert ln.tolist() == [0, 33, 0, 20] and c.cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    c.done()


@pytest.mark.parametrize("which", ["src", "dst"])
def test_blend_records_bad_pages_in_the_model(cb, which):
    """A page id outside the pool in cb_blend_kv8's tables: in the model's status, where cb_blend_paged's are, and in the
    cache's."""
    import test_gpu_gradual as tg
    w, toks, chunks, caches = tg.tiny5_case()
    n_ctx, N, P = sum(x[2] for x in chunks), len(toks), 32
    nb = -(-N // P)
    model = cb.BlendModel(tg.TINY5.as_dict(), w, max_tokens=N, max_chunks=len(chunks))
    cache = cb.KV8Cache.empty(5, 2 * nb, 2, P, 64, n_heads=tg.TINY5.n_heads, dtype="f32")
    tabs = dict(src=torch.arange(nb, dtype=torch.int32, device="cuda"), dst=torch.arange(nb, 2 * nb, dtype=torch.int32, device="cuda"))
    ctx = tg.device_cache(caches, "f32")
    cache.write(tabs["src"][None, :-(-n_ctx // P)].contiguous(), None, ctx[:, 0], ctx[:, 1], n_layers=5, max_len=n_ctx)
    t, work, logits = torch.from_numpy(toks).cuda(), model.kv_buffer(N), torch.empty(1024, device="cuda")
    work.zero_()
    args = (chunks, (0.4,) * 4, work, logits)
    cb.cb_blend_kv8(model.handle, t, N, cache, tabs["src"], tabs["dst"], *args)
    assert model.status() == 0 and cache.status() == 0
    work.zero_()
    tabs[which][1] = 2 * nb
    cb.cb_blend_kv8(model.handle, t, N, cache, tabs["src"], tabs["dst"], *args)
    assert model.status(clear=True) == cb.CB_STATUS_BAD_ROW and cache.status(clear=True) == cb.CB_STATUS_BAD_ROW
    # the cache's own calls are recorded in the cache alone
    cache.read(tabs[which][None].contiguous(), None, work[:, 0], work[:, 1], n_layers=5, max_len=N)
    assert cache.status(clear=True) == cb.CB_STATUS_BAD_ROW and model.status() == 0
    cache.close()
    model.close()


def test_cleared_status_does_not_lose_the_next_call(cb):
    """What a call on any stream records after status(clear=True) has returned stays recorded."""
    c = Case(cb, [20], H=1, hd=64, P=16, seed=1)
    kv, _ = c.values(1, 1, 1, 64)
    side, bad = torch.cuda.Stream(), i32([-1])
    torch.cuda.synchronize()
    for _ in range(200):
        c.cache.status(clear=True)
        c.cache.write(c.table, bad, kv, kv, stream=side)
        assert c.cache.status() == cb.CB_STATUS_BAD_ROW
    c.cache.status(clear=True)
    c.done()


@pytest.mark.parametrize("dtype,rows", KERNELS)
def test_queries_with_an_outlier_channel(cb, dtype, rows):
    """One channel of q 2^11 .. 2^16 times the others, over keys that are 0 there, so that the scores are the small channels'.
    A bf16 q of few rows is two e4m3 terms, scaled by the row's largest value to at most 448: an element below 2^-6 in
    those units is off by up to 2^-14, that is 2^-14 / 224 < 2^-21 of the row's largest.  (fp32: six terms, 2^-37; many
    rows: fp16, exact down to 2^-29 of it.)"""
    n = 300
    for size in (2.0 ** 11, 2.0 ** 14, 2.0 ** 16):
        c = Case(cb, [n], H=2, G=4, hd=64, P=16, dtype=dtype, seed=rows, cells=cb.KV8Cache.cells(rows, 8, n))
        m = c.model
        m.codes[0, 0, :, :, :, 9] = 0
        m.scales[0, 0] = 2.0 ** -3
        set_pool(c)
        q, _ = c.values(rows, 8, 64, size=0.25)
        q[:, :, 9] = size
        q64 = f64(q)
        out = torch.empty_like(q)
        c.cache.attention(c.table, c.lens_t, q, out, max_len=n)
        ref, _, spread, big = m.attention(c.table_np, c.lens, q64, [0, rows], 0, 0.125)
        k = m.rows(c.table_np[0], n, 0)[0]
        ds = 72 * U * big + (2.0 ** -21 * size * np.abs(k).sum(axis=2).max() * 0.125 if dtype == "bf16" and rows <= 8 else 0.0)
        p_rep, rnd, last = (2.0 ** -11, 2.0 ** -8, 2.0 ** -25) if dtype == "bf16" else (2.0 ** -23, 2.0 ** -24, 2.0 ** -37)
        tol = rnd * np.abs(ref) + (np.expm1(2 * ds) + 160 * U + p_rep) * spread + last * m.floor + 2.0 ** -32 * m.floor_all
        assert np.all(np.abs(f64(out) - ref) <= tol)
        c.done()


@pytest.mark.parametrize("rows", [[2, 0, 1, 0, 3], [40, 0, 9, 0, 70]])
def test_weights_of_sequences_without_rows(cb, rows):
    """Their keys have received nothing: 0 where the call writes, what was there where it adds."""
    lens = [400, 77, 129, 256, 90]
    n = sum(rows)
    c = Case(cb, lens, H=2, G=3, hd=64, P=16, seed=n, cells=cb.KV8Cache.cells(n, 6, 400))
    q, q64 = c.values(n, 6, 64)
    st, out = starts_of(rows), torch.empty_like(q)
    for add in (False, True):
        w = torch.full((5, 2, 400), 3.0, device="cuda")
        c.cache.attention(c.table, c.lens_t, q, out, q_start=i32(st), weights=w, add=add, max_len=400)
        check_attention(c, q, q64, st, out, w, w_before=3.0 if add else 0.0)
        for s in (1, 3):
            assert torch.all(w[s, :, :lens[s]] == (3.0 if add else 0.0)) and torch.all(w[s, :, lens[s]:] == 3.0)
    c.done()


@pytest.mark.parametrize("P,dtype", [(16, "bf16"), (64, "f32"), (256, "bf16")])
def test_ragged_rows_that_begin_anywhere(cb, P, dtype):
    """Many sequences whose rows begin and end at any place of a page, in an order of lengths that moves every sequence's
    blocks: all are written, and read back."""
    rng = np.random.default_rng(P)
    for _ in range(4):
        rows = (rng.integers(0, 3 * P, 40) * rng.integers(0, 2, 40)).tolist()
        lens = [r + int(rng.integers(0, P + 1)) for r in rows]
        c = Case(cb, lens, H=1, G=1, hd=64, P=P, dtype=dtype, seed=int(rng.integers(1000)))
        st = starts_of(rows, int(rng.integers(0, 5)))
        k, k64 = c.values(1, st[-1] + 1, 1, 64)
        v, v64 = c.values(1, st[-1] + 1, 1, 64, size=8.0)
        c.cache.write(c.table, c.lens_t, k, v, row_start=i32(st))
        c.model.write(c.table_np, lens, k64, v64, st)
        torch.cuda.synchronize()
        c.check_pool()
        ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
        c.cache.read(c.table, c.lens_t, ko, vo, row_start=i32(st))
        for got, kv in ((f64(ko)[0], 0), (f64(vo)[0], 1)):
            want = np.full((st[-1] + 1, 1, 64), 7.0)
            for s, n in enumerate(lens):
                if rows[s]:
                    want[st[s]:st[s + 1]] = c.model.rows(c.table_np[s], n, 0)[kv][n - rows[s]:]
            assert np.array_equal(got, want)
        c.done()


def test_fp32_heads_of_128_of_many_sequences(cb):
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 700, 70)]
    lens[3] = 3000
    c = Case(cb, lens, H=2, G=2, hd=128, P=32, dtype="f32", seed=5, cells=cb.KV8Cache.cells(70, 4, 3000))
    q, q64 = c.values(70, 4, 128)
    out, w = torch.empty_like(q), torch.zeros((70, 2, 3000), device="cuda")
    c.cache.attention(c.table, c.lens_t, q, out, weights=w, max_len=3000)
    check_attention(c, q, q64, list(range(71)), out, w)
    c.done()


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_long_sequences_of_several_layers(cb, in_place):
    """More rows than a selecting block keeps in shared memory, of several layers and sequences at once: rows and weights against
    a stable sort, and the rows' codes, which a page of one scale keeps."""
    lens, keep, sink, recent, P, L, H = [20000, 16384, 17001, 500], 3000, 4, 60, 64, 2, 2
    width = -(-max(lens) // P)
    need = -(-keep // P)
    n_pages = 4 * width + 4 * need
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = cb.KV8Cache.empty(L, n_pages, H, P, 64, 2 * H)
    cache.codes.copy_(torch.randint(0, 0x77, cache.codes.shape, generator=g, device="cuda", dtype=torch.uint8))
    cache.codes[..., 0] = 0x78                           # 256 in every row: each page has the scale of its values
    cache.scales.fill_(2.0 ** -5)
    before = cache.codes.clone()
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = order[:4 * width].view(4, width).contiguous()
    dst = table if in_place else order[4 * width:].view(4, need).contiguous()
    w = torch.randint(0, 500, (L, 4, H, max(lens)), generator=g, device="cuda").float() / 64
    was, lt = w.clone(), i32(lens)
    e = cache.evict(table, lt, dst, w, keep, sink, recent, n_layers=L, max_len=max(lens))
    torch.cuda.synchronize()
    assert e["lens"].tolist() == [min(n, keep) for n in lens] and cache.status() == 0
    for l in range(L):
        for s, n in enumerate(lens):
            m = min(n, keep)
            for h in range(H):
                r = was[l, s, h, :n].clone()
                r[:sink] = r[n - recent:] = float("inf")
                want = torch.sort(r, descending=True, stable=True).indices[:m].sort().values
                assert torch.equal(e["rows"][l, s, h, :m], want.int()) and torch.all(e["rows"][l, s, h, m:] == -1)
                assert torch.equal(w[l, s, h, :m], was[l, s, h, want]) and torch.count_nonzero(w[l, s, h, m:n]) == 0
                assert torch.equal(w[l, s, h, n:], was[l, s, h, n:])
                at = torch.arange(m, device="cuda")
                for kv in range(2):
                    got = cache.codes[l, kv, dst[s, at // P].long(), h, at % P]
                    ref = before[l, kv, table[s, want // P].long(), h, want % P]
                    assert torch.equal(got, ref)
                    assert torch.all(cache.scales[l, kv, dst[s, :-(-m // P)].long(), h] == 2.0 ** -5)
    cache.close()


def test_blend_over_the_8bit_pool_in_bf16(cb):
    """cb_blend_kv8 of a bf16 model on the tensor cores is the read, the gradual blend in place and the write, bit for bit."""
    import workload
    shape = workload.ModelShape(3, 1024, 8, 2, 128, 2816, 4096, 5e5, "bf16")
    w = workload.make_weights(shape, 7)
    chunks, P = [(0, 256 * i, 256) for i in range(3)], 32
    n_ctx, N = 768, 768 + 40
    toks = torch.from_numpy(workload.tokens(0, 5, N, 4096)).cuda()
    model = cb.BlendModel(shape.as_dict(), w, max_tokens=N, max_chunks=3)
    nb = -(-N // P)
    cache = cb.KV8Cache.empty(3, 2 * nb, 2, P, 128, n_heads=8)
    src = torch.arange(nb, dtype=torch.int32, device="cuda")
    dst = src + nb
    g = torch.Generator(device="cuda").manual_seed(4)
    ctx = torch.randn((3, 2, n_ctx, 2, 128), generator=g, device="cuda").bfloat16()
    cache.write(src[None, :n_ctx // P].contiguous(), None, ctx[:, 0], ctx[:, 1], n_layers=3, max_len=n_ctx)
    work, ratios = model.kv_buffer(N), (0.3, 0.2)
    logits = torch.empty(4096, device="cuda", dtype=torch.float32)
    cb.cb_blend_kv8(model.handle, toks, N, cache, src, dst, chunks, ratios, work, logits)
    ref = model.kv_buffer(N)
    cache.read(src[None].contiguous(), None, ref[:, 0, :n_ctx], ref[:, 1, :n_ctx], n_layers=3, max_len=n_ctx)
    out = model.blend_gradual(toks, ref, chunks, ratios, out_kv=ref)
    fresh = cb.KV8Cache.empty(3, nb, 2, P, 128, n_heads=8)
    fresh.write(src[None].contiguous(), None, ref[:, 0], ref[:, 1], n_layers=3, max_len=N)
    torch.cuda.synchronize()
    assert torch.equal(work, ref) and torch.equal(logits, out["logits"].float())
    full = N // P                                        # whole pages, and of the last one the rows that were written
    assert torch.equal(cache.codes[:, :, nb:nb + full], fresh.codes[:, :, :full])
    assert torch.equal(cache.codes[:, :, nb + full, :, :N % P], fresh.codes[:, :, full, :, :N % P])
    assert torch.equal(cache.scales[:, :, nb:], fresh.scales) and model.status() == 0 and cache.status() == 0
    for x in (fresh, cache, model):
        x.close()


def test_most_sequences(cb):
    """65535 sequences, one page each: written, attended to with weights, read back, evicted."""
    n, P, hd, G = 65535, 16, 64, 2
    cache = cb.KV8Cache.empty(1, n, 1, P, hd, G, weight_cells=cb.KV8Cache.cells(n, G, P))
    g = torch.Generator(device="cuda").manual_seed(9)
    table = torch.randperm(n, generator=g, device="cuda").int()[:, None].contiguous()
    lens = torch.randint(0, P + 1, (n,), generator=g, device="cuda").int()
    start = torch.cat([torch.zeros(1, device="cuda"), lens.cumsum(0)]).int()
    total = int(start[-1])
    k = torch.randn((total, 1, hd), generator=g, device="cuda").bfloat16()
    v = torch.randn((total, 1, hd), generator=g, device="cuda").bfloat16()
    cache.write(table, lens, k, v, row_start=start)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    cache.read(table, lens, ko, vo, row_start=start)
    # half a step of a number (2^-4), or of a block's scale (2^-10 of 2^-6: its largest value is below 7)
    for a, b in ((ko, k), (vo, v)):
        assert torch.all((a.float() - b.float()).abs() <= 2.0 ** -4 * b.float().abs() + 2.0 ** -16)
    q = torch.randn((n, G, hd), generator=g, device="cuda").bfloat16()
    w = torch.full((n, 1, P), -1.0, device="cuda")
    out = cache.attention(table, lens, q, weights=w)
    seen = torch.arange(P, device="cuda")[None, :] < lens[:, None]
    kk, vv = (torch.zeros((n, P, hd), device="cuda", dtype=torch.float64) for _ in range(2))
    kk[seen], vv[seen] = ko[:, 0].double(), vo[:, 0].double()
    x = torch.einsum("nhd,npd->nhp", q.double(), kk) * hd ** -0.5
    p = torch.softmax(x.masked_fill(~seen[:, None], -torch.inf), dim=2).nan_to_num(0.0)
    ref, spread = torch.einsum("nhp,npd->nhd", p, vv), torch.einsum("nhp,npd->nhd", p, vv.abs())
    # (as in test_gpu_kv8.py, with scores of sum |q k| scale below 64; P's floor: 2^-25 of at most 448 * 16 codes * scale)
    tol = 2.0 ** -8 * ref.abs() + (2 * 72 * U * 64 + 160 * U + 2.0 ** -11) * spread + 2.0 ** -25 * 448 * 16 * 2.0 ** -6
    assert torch.all((out.double() - ref).abs() <= tol)
    assert torch.all(torch.where(seen, (w[:, 0] - p.sum(1)).abs() <= 1e-3 * p.sum(1) + 1e-12, w[:, 0] == -1.0))
    e = cache.evict(table, lens, table, w[None], 5, 1, 1)
    torch.cuda.synchronize()
    assert torch.equal(e["lens"], lens.clamp(max=5)) and cache.status() == 0
    rows = e["rows"][0, :, 0]
    kept = torch.arange(5, device="cuda")[None, :] < e["lens"][:, None]
    assert torch.all((rows >= 0) == kept)
    assert torch.all((rows[:, 1:] > rows[:, :-1]) | (rows[:, 1:] < 0))
    cache.close()


def test_scores_of_more_than_32_bits(cb):
    """1024 rows of 32 heads over 140 000 keys with weights: 4.6e9 scores.  The same rows in two calls, the second of which
    adds, give the same sums."""
    n, rows, P, hd = 140000, 1024, 256, 64
    cells = cb.KV8Cache.cells(rows, 32, n)
    assert cells > 2 ** 32
    cache = cb.KV8Cache.empty(1, n // P + 1, 8, P, hd, 32, weight_cells=cells)
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.randn((n, 8, hd), generator=g, device="cuda").bfloat16()
    table = torch.randperm(n // P + 1, generator=g, device="cuda").int()[None]
    cache.write(table, i32([n]), k, k.flip(0).contiguous(), max_len=n)
    q = torch.randn((rows, 32, hd), generator=g, device="cuda").bfloat16()
    w, two = torch.zeros((1, 8, n), device="cuda"), torch.zeros((1, 8, n), device="cuda")
    out = cache.attention(table, i32([n]), q, weights=w, max_len=n)
    h = rows // 2
    a = cache.attention(table, i32([n - h]), q[:h], weights=two, max_len=n)
    b = cache.attention(table, i32([n]), q[h:], weights=two, add=True, max_len=n)
    torch.cuda.synchronize()
    assert cache.status() == 0
    # both within (2 ds + (16 + 128 + n / 128 + columns) u) of the weight, ds = 72 u 64 at most
    assert torch.all((w - two).abs() <= 2 * (2 * 72 * 64 + 144 + n / 128 + 4096) * U * two)
    assert abs(float(w.double().sum()) / (rows * 32) - 1) < 1e-3
    both = torch.cat([a, b]).float()
    assert torch.all((out.float() - both).abs() <= 2 * 2.0 ** -8 * both.abs() + 2.0 ** -10)
    cache.close()


def test_numbers_beyond_32_bits_are_refused(cb):
    """2^32 + 40 keys or layer 2^32 are not 40 keys and layer 0."""
    c = Case(cb, [40], H=1, hd=64, P=16, seed=1)
    q, _ = c.values(1, 2, 64)
    kv, _ = c.values(1, 1, 1, 64)
    w = torch.zeros((1, 1, 1, 48), device="cuda")
    for top in (2 ** 31, 2 ** 32, 2 ** 32 + 40, -2 ** 32 + 40, -1):
        for f in (lambda: c.cache.attention(c.table, c.lens_t, q, max_len=top), lambda: c.cache.write(c.table, c.lens_t, kv, kv, max_len=top),
                  lambda: c.cache.read(c.table, c.lens_t, kv, kv.clone(), max_len=top),
                  lambda: c.cache.evict(c.table, c.lens_t, c.table, w, 4, max_len=top)):
            with pytest.raises((ValueError, cb.CacheBlendError)):
                f()
    big = 2 ** 32
    for f in (lambda: c.cache.attention(c.table, c.lens_t, q, layer=big), lambda: c.cache.write(c.table, c.lens_t, kv, kv, layer=big),
              lambda: c.cache.read(c.table, c.lens_t, kv, kv.clone(), layer=-big),
              lambda: c.cache.evict(c.table, c.lens_t, c.table, w, 4, layer=big),
              lambda: c.cache.evict(c.table, c.lens_t, c.table, w, 4, big + 1), lambda: c.cache.evict(c.table, c.lens_t, c.table, w, 4, 0, big),
              lambda: c.cache.evict(c.table, c.lens_t, c.table, w, big + 4)):
        with pytest.raises((ValueError, cb.CacheBlendError)):
            f()
    c.check_pool()
    # numbers of numpy's are numbers
    a = c.cache.attention(c.table, c.lens_t, q, layer=np.int64(0), max_len=np.int32(40))
    assert torch.equal(a, c.cache.attention(c.table, c.lens_t, q, max_len=40))
    c.done()
