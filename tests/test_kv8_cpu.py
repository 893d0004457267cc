"""8-bit paged K/V cache without a GPU: the numpy model against torch's e4m3 cast, the block addressing of ragged
rows, and the refusals of the C ABI (argument checks come before the first CUDA call of an entry point; the handle
used here names no device, so that nothing is ever launched)."""
import ctypes

import numpy as np
import pytest

import cacheblend_selective_kv_gb300 as cb
import kv8_model as km

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return cb.lib()


def test_encode_matches_torch_cast():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-14, 9, 4000), km.VALUES[~np.isnan(km.VALUES)],
                        (km._POS[1:] + km._POS[:-1]) / 2, [0.0, -0.0, 448.0, -448.0, 2.0 ** -10, 2.0 ** -11]])
    x = x[np.abs(x) <= 448].astype(np.float32)
    got = km.encode(x.astype(np.float64))
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, ref)
    back = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(back, km.VALUES.astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("P", [16, 64])
def test_slots_of_ragged_rows_cover_every_block(P):
    """The slot base start / P + 2 s gives each sequence room for every block its rows touch, wherever they begin."""
    rng = np.random.default_rng(P)
    for _ in range(200):
        n = rng.integers(1, 12)
        rows = rng.integers(0, 3 * P, n) * rng.integers(0, 2, n)
        start = np.concatenate([[0], np.cumsum(rows)])
        total = start[-1] // P + 2 * n
        base = [start[s] // P + 2 * s for s in range(n)] + [total]
        for s in range(n):
            for first in range(P):
                if rows[s]:
                    touched = (first + rows[s] - 1) // P - first // P + 1
                    assert base[s + 1] - base[s] >= touched, (start, s, first)


class FakeHandle(ctypes.Structure):
    """The leading fields of a cache handle: its configuration and a device that is never the current one."""
    _fields_ = [("cfg", cb.CbKV8Config), ("device", ctypes.c_int), ("num_sms", ctypes.c_int), ("shift", ctypes.c_int), ("pdl", ctypes.c_bool),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("scores", ctypes.c_void_p), ("room", ctypes.c_uint8 * 256)]


def fake(**kw):
    c = dict(n_layers=4, n_heads=8, n_kv_heads=2, head_dim=64, dtype=cb.CB_BF16, page_size=32, n_pages=100, weight_cells=5000)
    c.update(kw)
    h = FakeHandle()
    h.cfg = cb.CbKV8Config(*[c[f] for f, _ in cb.CbKV8Config._fields_])
    h.device, h.num_sms = -1, 152
    while (1 << h.shift) < c["page_size"]:
        h.shift += 1
    return h


A = 1 << 20                                            # an aligned address that no check dereferences


def seqs(n=3, table=A, ld=4, lens=A, top=100):
    return cb.CbKV8Seqs(n, table, ld, lens, top)


def refused(code, word):
    assert code == cb.CB_ERR_INVALID_ARG, (code, cb.cb_last_error())
    assert word in cb.cb_last_error(), cb.cb_last_error()


def reaches_device(code):
    """Every argument check passed: what stops the call is the handle's device."""
    assert code == cb.CB_ERR_CUDA and "CUDA device -1 is not available" in cb.cb_last_error()


@pytest.mark.parametrize("bad,code", [
    (dict(head_dim=96), cb.CB_ERR_UNSUPPORTED), (dict(n_heads=18), cb.CB_ERR_UNSUPPORTED),
    (dict(n_heads=7), cb.CB_ERR_INVALID_ARG), (dict(page_size=8), cb.CB_ERR_INVALID_ARG),
    (dict(page_size=512), cb.CB_ERR_INVALID_ARG), (dict(page_size=48), cb.CB_ERR_INVALID_ARG),
    (dict(n_pages=0), cb.CB_ERR_INVALID_ARG), (dict(n_pages=1 << 25), cb.CB_ERR_INVALID_ARG),
    (dict(n_layers=0), cb.CB_ERR_INVALID_ARG), (dict(dtype=2), cb.CB_ERR_INVALID_ARG),
    (dict(weight_cells=-1), cb.CB_ERR_INVALID_ARG), (dict(n_layers=1000, n_kv_heads=64, n_heads=64), cb.CB_ERR_UNSUPPORTED),
])
def test_create_refuses(lib, bad, code):
    out = ctypes.c_void_p()
    assert lib.cb_kv8_create(ctypes.byref(fake(**bad).cfg), A, A, ctypes.byref(out)) == code
    assert not out.value and cb.cb_last_error()


def test_create_refuses_pointers(lib):
    out = ctypes.c_void_p()
    for codes, scales in ((0, A), (A, 0), (A + 16, A), (A, A + 2)):
        assert lib.cb_kv8_create(ctypes.byref(fake().cfg), codes, scales, ctypes.byref(out)) == cb.CB_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["cb_kv8_write", "cb_kv8_read"])
def test_rows_refusals(lib, name):
    f, h = getattr(lib, name), fake()

    def call(sq=None, layer=1, n_layers=2, k=A, v=2 * A, ls=10 * 128, rs=128, start=A, rows=10, handle=h):
        return f(ctypes.addressof(handle) if handle else None, sq or seqs(), layer, n_layers, k, v, ls, rs, start, rows, None)

    reaches_device(call())
    reaches_device(call(start=None, rows=9))
    reaches_device(call(ls=128, rs=2 * 128))           # layers interleaved row by row
    refused(call(handle=None), "null cache")
    refused(call(layer=3), "layers")
    refused(call(layer=-1), "layers")
    refused(call(n_layers=-1), "layers")
    refused(call(sq=seqs(n=-1)), "n_seqs")
    refused(call(sq=seqs(n=65536)), "n_seqs")
    refused(call(sq=seqs(top=129)), "max_len")
    refused(call(sq=seqs(top=-1)), "max_len")
    refused(call(sq=seqs(table=None)), "block table")
    refused(call(start=None), "shared evenly")
    refused(call(rows=-1), "rows")
    refused(call(k=None), "null k or v")
    refused(call(k=A + 8), "16 bytes")
    refused(call(rs=132), "16 bytes")
    refused(call(rs=64), "row stride")
    refused(call(ls=5 * 128), "overlap")
    assert call(rows=0, k=None) == cb.CB_OK            # nothing to do
    assert call(n_layers=0, k=None) == cb.CB_OK


def test_attention_refusals(lib):
    h = fake()

    def call(sq=None, layer=3, q=A, qs=512, start=A, nq=5, scale=0.125, out=3 * A, os=512, w=None, ld=0, handle=h):
        return lib.cb_kv8_attention(ctypes.addressof(handle) if handle else None, sq or seqs(), layer, q, qs, start, nq, scale, out,
                                    os, w, ld, 0, None)

    reaches_device(call())
    reaches_device(call(nq=4, w=A, ld=100))            # 4 * 8 * 129 cells
    refused(call(handle=None), "null cache")
    refused(call(layer=4), "layers")
    refused(call(scale=float("nan")), "scale")
    refused(call(scale=float("inf")), "scale")
    refused(call(q=None), "null q or out")
    refused(call(out=None), "null q or out")
    refused(call(q=A + 2), "16 bytes")
    refused(call(os=516), "16 bytes")
    refused(call(qs=256), "row stride")
    refused(call(out=A + 4 * 512 * 2), "overlap")
    refused(call(w=A, ld=99), "weights_ld")
    refused(call(nq=5, w=A, ld=100), "cells")
    refused(call(start=None), "shared evenly")
    refused(call(sq=seqs(ld=3)), "max_len")
    assert call(nq=0, q=None, out=None) == cb.CB_OK
    assert call(sq=seqs(n=0), nq=0) == cb.CB_OK


def test_evict_refusals(lib):
    h = fake()

    def call(sq=None, dst=2 * A, dld=4, layer=0, nl=4, w=A, ld=100, keep=50, sink=4, recent=8, ow=A, rows=9 * A, lens=A, handle=h):
        return lib.cb_kv8_evict(ctypes.addressof(handle) if handle else None, sq or seqs(), dst, dld, layer, nl, w, ld, keep, sink,
                                recent, ow, rows, lens, None)

    reaches_device(call())
    reaches_device(call(dst=A))
    reaches_device(call(keep=1000, dld=4))             # more than any sequence has
    refused(call(handle=None), "null cache")
    refused(call(nl=5), "layers")
    refused(call(keep=0), "n_keep")
    refused(call(sink=-1), "n_keep")
    refused(call(sink=40, recent=11), "n_keep")
    refused(call(dld=1), "destination")
    refused(call(ld=99), "weights_ld")
    refused(call(ow=A + 400), "overlap")
    for name in ("dst", "w", "ow", "rows", "lens"):
        refused(call(**{name: None}), "null destination")


def test_blend_kv8_refuses_null(lib):
    assert lib.cb_blend_kv8(None, None, 1, None, None, None, None, 0, None, 0, None, None, None, None, None, None) == \
        cb.CB_ERR_INVALID_ARG


def unsupported(code, word):
    assert code == cb.CB_ERR_UNSUPPORTED and word in cb.cb_last_error(), (code, cb.cb_last_error())


@pytest.mark.parametrize("name", ["cb_kv8_write", "cb_kv8_read"])
def test_rows_overlaps_and_counts(lib, name):
    f, h = getattr(lib, name), fake(n_kv_heads=2)
    read = name == "cb_kv8_read"

    def call(n_layers=2, k=A, v=2 * A, ls=10 * 128, rs=128, rows=10, handle=h, sq=None):
        return f(ctypes.addressof(handle), sq or seqs(), 0, n_layers, k, v, ls, rs, A, rows, None)

    one_for_all = call(ls=0)                           # an input may be one layer for all, an output may not
    refused(one_for_all, "overlap") if read else reaches_device(one_for_all)
    one_for_all = call(ls=0, rs=2 * 128)
    refused(one_for_all, "overlap") if read else reaches_device(one_for_all)
    refused(call(ls=64, rs=2 * 128), "overlap")        # interleaved, but not by a whole row
    same = call(v=A)
    refused(same, "k and v overlap") if read else reaches_device(same)
    reaches_device(call(v=A + 256, rs=256, ls=10 * 256))           # K and V side by side in a row
    many = fake(n_kv_heads=1024, n_heads=1024, n_layers=4, page_size=16, n_pages=1000)
    w = 1024 * 64                                      # blocks: (n_rows / 16 + 2 * 3) * 1024 below 2^31
    reaches_device(call(n_layers=1, rs=w, rows=16 * ((1 << 21) - 8), handle=many, sq=seqs(top=60)))
    unsupported(call(n_layers=1, rs=w, rows=1 << 26, handle=many, sq=seqs(top=60)), "rows")
    unsupported(call(n_layers=1, rs=w, rows=1 << 30, handle=many, sq=seqs(top=60)), "rows")


def test_attention_counts_pass_64_bits(lib):
    """Sizes whose products pass 32 or 64 bits are refused and do not wrap around to small ones."""
    h = fake(n_kv_heads=1024, n_heads=8192, weight_cells=5000)
    w = 8192 * 64

    def call(n, top, weights=None, handle=h, qs=w):
        return lib.cb_kv8_attention(ctypes.addressof(handle), seqs(n=1, ld=1 << 26, top=top), 0, A, qs, None, n, 0.125, 1 << 55, qs, weights,
                                    1 << 30, 0, None)

    reaches_device(call(1, 4096))
    for n, top in ((1 << 30, 1 << 30), (1 << 30, (1 << 30) - 256), (1 << 20, 1 << 20), (1 << 21, 0), (1 << 12, 1 << 16)):
        unsupported(call(n, top), "too many")
    for n, top in ((1 << 30, 1 << 30), (1 << 28, (1 << 23) - 1), (1, 4096), (1 << 30, 1)):
        refused(call(n, top, weights=A), "cells")
    small = fake(weight_cells=5000)
    # no keys: no weights to return, and no scratch
    reaches_device(lib.cb_kv8_attention(ctypes.addressof(small), seqs(n=1, top=0), 0, A, 512, None, 5000, 0.125, 1 << 50, 512, A, 0, 0, None))


def test_evict_refuses_overlapping_tables(lib):
    h = fake()

    def call(n=3, dst=2 * A, dld=4, ld=4, keep=50):
        return lib.cb_kv8_evict(ctypes.addressof(h), seqs(n=n, ld=ld), dst, dld, 0, 4, A, 100, keep, 4, 8, A, 9 * A, A, None)

    reaches_device(call(dst=A))
    refused(call(dst=A, dld=2), "overlaps")            # the same table at another width names other pages
    refused(call(dst=A + 4), "overlaps")
    refused(call(dst=A + 2 * 4 * 4), "overlaps")
    reaches_device(call(dst=A, dld=2, n=1))            # one sequence: its first pages, in place
    reaches_device(call(dst=A + 3 * 4 * 4))


def test_read_refuses_overlapping_outputs(lib):
    """k and v that meet in any of their rows, against a search over all pairs of rows."""
    h = fake(n_kv_heads=2)                             # rows of 128 elements, 256 bytes

    def call(apart, ls, rs, rows=6, n_layers=3):
        return lib.cb_kv8_read(ctypes.addressof(h), seqs(), 0, n_layers, 8 * A, 8 * A + 2 * apart, ls, rs, A, rows, None)

    def distances(ls, rs, rows=6, n_layers=3):
        at = [l * ls + r * rs for l in range(n_layers) for r in range(rows)]
        return sorted({b - a for a in at for b in at})

    for ls, rs in ((6 * 128, 128), (12 * 128, 128), (6 * 256, 256), (128, 3 * 128), (256, 6 * 128), (7 * 192, 192), (128, 4 * 128)):
        both, far = set(), distances(ls, rs)
        for apart in range(-40 * 128, 40 * 128 + 1, 8):
            want = any(abs(apart + d) < 128 for d in far)
            both.add(want)
            code = call(apart, ls, rs)
            refused(code, "k and v overlap") if want else reaches_device(code)
        assert both == {True, False}
    refused(call(128, 6 * 128, 128), "k and v overlap")                # v is k without its first row
    refused(call(6 * 128, 6 * 128, 128), "k and v overlap")            # ... without its first layer
    reaches_device(call(6 * 128, 12 * 128, 128))                       # the halves of [layers][2][rows]
    reaches_device(call(128, 6 * 256, 256))                            # halves of a row
    reaches_device(call(3 * 128, 128, 6 * 128))                        # layers interleaved row by row, then K and V
    # a write's inputs may meet
    code = lib.cb_kv8_write(ctypes.addressof(h), seqs(), 0, 3, 8 * A, 8 * A + 256, 6 * 128, 128, A, 6, None)
    reaches_device(code)
