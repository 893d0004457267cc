"""GPU tests of the layouts of k and v that append takes: those that write takes too."""
import pytest

from test_gpu_kv8 import Case

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


def layouts(H, n, k, v):
    """Pairs of tensors with the values of k and v whose strides differ where there is one row or one head."""
    hd = k.shape[2]
    if n == 1:
        wide = torch.zeros((3, 2 * H, hd), dtype=k.dtype, device="cuda")
        wide[1, :H] = k[0]
        yield wide[1:2, :H], v                          # a slice of a projection's row beside a tensor of its own
        yield v, wide[1:2, :H]
    if H == 1:
        yield k.as_strided((n, 1, hd), (hd, 8, 1)), v
        yield k, v.as_strided((n, 1, hd), (hd, 0, 1))


@pytest.mark.parametrize("H,n,dtype", [(2, 1, "bf16"), (1, 1, "f32"), (1, 3, "bf16")])
def test_strides_that_say_nothing(cb, H, n, dtype):
    """One row, or one KV head: k and v whose other strides differ are taken, and give what contiguous tensors give."""
    hd, P = 64, 16
    c = Case(cb, [20], H=H, G=2, hd=hd, P=P, dtype=dtype, seed=H + n)
    k, v = c.values(n, H, hd)[0], c.values(n, H, hd)[0]
    codes, scales = c.codes.clone(), c.scales.clone()
    seen = 0
    for a, b in layouts(H, n, k, v):
        assert a.stride() != b.stride()
        pools = []
        for x, y in ((a, b), (a.contiguous().clone(), b.contiguous().clone())):
            c.codes.copy_(codes)
            c.scales.copy_(scales)
            c.cache.append(c.table, c.lens_t, None, x, y, 1e4)
            c.cache.append(c.table, c.lens_t, None, x, y, 1e4, row_start=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
            torch.cuda.synchronize()
            pools.append((c.codes.clone(), c.scales.clone()))
        assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
        assert not torch.equal(pools[0][0], codes)
        c.cache.write(c.table, c.lens_t, a, b)          # takes the same
        seen += 1
    assert seen >= 2
    c.done()


def test_strides_that_differ_are_refused(cb):
    c = Case(cb, [20], H=2, G=2, hd=64, P=16)
    k = c.values(3, 2, 64)[0]
    wide = torch.zeros((3, 256), dtype=k.dtype, device="cuda")[:, :128].view(3, 2, 64)
    for a, b in ((k, wide), (wide, k), (k[None], k[None]), (k, k[None])):
        with pytest.raises(ValueError, match="same number of rows and the same strides"):
            c.cache.append(c.table, c.lens_t, None, a, b, 1e4)
    c.done()
