"""Operators of a decoding step without a GPU: the refusals of the C ABI (argument checks come before the first CUDA call;
the handle used here names no device, so that nothing is ever launched)."""
import ctypes

import pytest

import cacheblend_selective_kv_gb300 as cb
from test_kv8_cpu import A, fake, lib, reaches_device, refused, seqs, unsupported   # noqa: F401 (lib is a fixture)

torch = pytest.importorskip("torch")


def test_append_refusals(lib):
    h = fake()                                         # rows of 512 elements of q, 128 of k and v, bf16

    def call(sq=None, layer=3, q=A, qs=512, oq=2 * A, os=512, k=4 * A, v=5 * A, ks=128, pos=A, theta=1e4, start=A, rows=10, handle=h):
        return lib.cb_kv8_append(ctypes.addressof(handle) if handle else None, sq or seqs(), layer, q, qs, oq, os, k, v, ks, pos, theta,
                                 start, rows, None)

    reaches_device(call())
    reaches_device(call(q=None, oq=None, qs=0, os=0))
    reaches_device(call(oq=A))                         # in place
    reaches_device(call(start=None, rows=9, pos=None))
    reaches_device(call(qs=768, os=768, ks=768, oq=A, k=A + 1024, v=A + 1280))     # slices of one projection's rows, in place
    reaches_device(call(k=4 * A, v=4 * A))             # what is only read may meet
    refused(call(handle=None), "null cache")
    refused(call(layer=4), "layers")
    refused(call(layer=-1), "layers")
    refused(call(sq=seqs(n=65536)), "n_seqs")
    refused(call(sq=seqs(top=129)), "max_len")
    refused(call(start=None), "shared evenly")
    refused(call(rows=-1), "rows")
    for theta in (0.0, -1.0, 0.5, float("nan"), float("inf")):
        refused(call(theta=theta), "rope_theta")
    refused(call(k=None), "null k or v")
    refused(call(v=A + 8), "16 bytes")
    refused(call(ks=64), "row stride")
    refused(call(ks=132), "16 bytes")
    refused(call(q=None), "both")
    refused(call(oq=None), "both")
    refused(call(q=A + 2), "16 bytes")
    refused(call(os=516), "16 bytes")
    refused(call(qs=256), "row stride")
    refused(call(oq=A + 512), "q and out_q overlap")
    refused(call(oq=A, os=768), "q and out_q overlap")
    refused(call(qs=768, os=768, ks=768, oq=A, k=A + 1008, v=A + 1280), "out_q overlaps")
    refused(call(qs=768, os=768, ks=768, oq=A, k=A + 1024, v=A + 1536 - 16), "out_q overlaps")
    refused(call(oq=4 * A - 512, os=512), "out_q overlaps")
    assert call(rows=0, k=None) == cb.CB_OK            # nothing to do
    assert call(sq=seqs(n=0), rows=0, k=None) == cb.CB_OK
    big = fake(n_heads=512, n_kv_heads=64, page_size=256, n_pages=1000)
    unsupported(lib.cb_kv8_append(ctypes.addressof(big), seqs(n=1, ld=1 << 23, top=1 << 30), 0, A, 1 << 15, 1 << 55, 1 << 15, 1 << 58, 1 << 59,
                                  1 << 12, None, 1e4, None, 1 << 25, None), "rows of q")


def test_shared_attention_refusals(lib):
    h = fake(weight_cells=5 * 8 * 134)                 # rows of 8 heads of 64: five of them

    def call(pre=None, first=A, sq=None, layer=3, q=A, qs=512, start=A, nq=5, scale=0.125, out=3 * A, os=512, handle=h):
        return lib.cb_kv8_attention_shared(ctypes.addressof(handle) if handle else None, pre or seqs(n=2), first, sq or seqs(), layer, q, qs,
                                           start, nq, scale, out, os, None)

    reaches_device(call())
    reaches_device(call(pre=seqs(n=3), first=None))
    reaches_device(call(pre=seqs(n=0), nq=9, first=None))          # no prefix: no scratch
    reaches_device(call(pre=seqs(n=2, top=0), nq=9))
    refused(call(handle=None), "null cache")
    refused(call(layer=4), "layers")
    refused(call(pre=seqs(n=-1)), "n_seqs")
    refused(call(pre=seqs(ld=3)), "max_len")
    refused(call(pre=seqs(table=None)), "block table")
    refused(call(sq=seqs(ld=3)), "max_len")
    refused(call(first=None), "shared evenly by 2 prefixes")
    refused(call(start=None), "shared evenly by 3 sequences")
    refused(call(nq=6), "cells")
    refused(call(scale=float("nan")), "scale")
    refused(call(q=None), "null q or out")
    refused(call(q=A + 2), "16 bytes")
    refused(call(qs=256), "row stride")
    refused(call(out=A + 4 * 512 * 2), "overlap")
    assert call(nq=0, q=None, out=None) == cb.CB_OK
    assert call(sq=seqs(n=0), nq=0, first=None) == cb.CB_OK
    big = fake(n_kv_heads=1024, n_heads=8192, weight_cells=1 << 36)

    def large(n, top, own):
        return lib.cb_kv8_attention_shared(ctypes.addressof(big), seqs(n=1, ld=1 << 26, top=top), None, seqs(n=1, ld=1 << 26, top=own), 0, A,
                                           8192 * 64, None, n, 0.125, 1 << 55, 8192 * 64, None)
    reaches_device(large(1, 4096, 4096))
    unsupported(large(1 << 12, 1 << 16, 1), "too many")
    unsupported(large(1 << 12, 1, 1 << 16), "too many")


def test_sample_refusals(lib):
    def call(x=A, dtype=cb.CB_F32, n=3, v=100, ld=100, t=A, k=A, p=A, m=A, u=A, out=A, probs=A):
        return lib.cb_sample(x, dtype, n, v, ld, t, k, p, m, u, out, probs, None)

    assert call(n=0, x=None, u=None, out=None) == cb.CB_OK
    refused(call(dtype=2), "dtype")
    refused(call(n=-1), "n_rows")
    refused(call(n=(1 << 24) + 1), "n_rows")
    refused(call(v=0), "vocab")
    refused(call(v=-5), "vocab")
    unsupported(call(v=cb.CB_SAMPLE_MAX_VOCAB + 1, ld=1 << 20), "vocabulary")
    refused(call(ld=99), "stride")
    refused(call(ld=1 << 41), "stride")
    for name in ("x", "u", "out"):
        refused(call(**{name: None}), "null")
    for name in ("t", "k", "p", "m", "u", "out", "probs", "x"):
        refused(call(**{name: A + 2}), "aligned")
    refused(call(x=A + 1, dtype=cb.CB_BF16), "aligned")
