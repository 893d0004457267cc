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
