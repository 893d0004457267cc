"""GPU tests of how attention over a shared prefix chooses between one launch and several: what a handle was created with
decides, and the choice that it makes by itself gives the results of one of the two ways, which tests/test_gpu_kv8_shared.py compares with
float64 for both."""
import pytest

from test_gpu_kv8_shared import Shared

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


def result(monkeypatch, cb, again, shape, check=False):
    """The rows of a call of a handle that was created with CB_SHARED_AGAIN = again (None: unset); then the same call with the
    variable changed."""
    prefixes, lens, first, rows, kw = shape
    if again is None:
        monkeypatch.delenv("CB_SHARED_AGAIN", raising=False)
    else:
        monkeypatch.setenv("CB_SHARED_AGAIN", again)
    c = Shared(cb, prefixes, lens, first, rows, seed=len(lens), **kw)
    q, q64 = c.values(c.n_q, c.H * c.G, c.hd)
    out = torch.zeros_like(q)
    c.run(q, out, max_len=max(lens), prefix_max_len=max(prefixes))
    if check:
        c.check(out, q64)
    monkeypatch.setenv("CB_SHARED_AGAIN", "-1e15" if again != "-1e15" else "1e15")
    later = torch.zeros_like(q)
    c.run(q, later, max_len=max(lens), prefix_max_len=max(prefixes))
    torch.cuda.synchronize()
    assert torch.equal(out, later)
    c.done()
    return out


def shape(prefixes, n, own, rows, groups=None, **kw):
    per = n // len(prefixes)
    return prefixes, [own + s % 3 for s in range(n)], groups or [per * g for g in range(len(prefixes) + 1)], [rows] * n, {**dict(H=2, G=4, hd=64, P=64), **kw}


# on both sides of where several launches are estimated to take less: few rows and many, one group and several, both types
FEW = [shape([300], 3, 40, 1), shape([900], 64, 200, 1), shape([8192], 64, 200, 1), shape([2100, 2000, 2048, 70], 32, 30, 1, P=16),
       shape([6000, 6100], 48, 300, 2, hd=128), shape([8192], 64, 200, 1, dtype="f32", G=2), shape([700], 12, 100, 5, dtype="f32", G=1)]
MANY = [shape([500], 4, 90, 40), shape([700, 600], 8, 120, 16, hd=128), shape([16384], 16, 60, 16, H=1, G=8), shape([30000], 24, 40, 12, P=256)]


@pytest.mark.parametrize("shapes,small", [(FEW, 3), (MANY, 2)])
def test_choice_by_estimate(monkeypatch, cb, shapes, small):
    taken = set()
    for i, s in enumerate(shapes):
        one, two, chosen = (result(monkeypatch, cb, again, s, check=again is None and i < small) for again in ("1e15", "-1e15", None))
        assert not torch.equal(one, two)               # (else this test could not tell)
        assert torch.equal(chosen, one) or torch.equal(chosen, two), i
        taken.add(torch.equal(chosen, one))
    assert taken == {True, False}


def test_batches_of_single_sequences(monkeypatch, cb):
    """Groups of one sequence, a group for every sequence, and sequences of no group at all, by the handle's own choice."""
    for first, n_pre in (([0, 1, 2, 3, 4], 4), ([0, 0, 0, 0, 0], 4), ([4, 4], 1), ([0, 4], 1)):
        result(monkeypatch, cb, None, ([130 + 7 * g for g in range(n_pre)], [20, 1, 0, 128], first, [1, 1, 1, 1], dict(H=2, G=2, hd=64, P=16)), check=True)


def test_scratch_without_shared_calls(monkeypatch, cb):
    """A cache without cells for a row of attention over a shared prefix holds no pieces for a second launch, and refuses such a call."""
    def size(cells):
        codes, scales = torch.zeros((1, 2, 4, 8, 16, 128), dtype=torch.uint8, device="cuda"), torch.zeros((1, 2, 4, 8), device="cuda")
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        caches = [cb.KV8Cache(codes, scales, n_heads=32, dtype="bf16", weight_cells=cells) for _ in range(8)]
        used = before - torch.cuda.mem_get_info()[0]
        for c in caches:
            c.close()
        return used / 8
    row = cb.KV8Cache.shared_cells(1, 32, 128)
    none, shared = size(0), size(row)
    assert shared - none >= 4 << 20
    assert size(row - 1) - none < 2 << 20
    table, lens, q = torch.zeros((1, 2), dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda"), torch.zeros((1, 32, 128), device="cuda").bfloat16()
    for cells in (0, row - 1, row):
        codes, scales = torch.zeros((1, 2, 4, 8, 16, 128), dtype=torch.uint8, device="cuda"), torch.zeros((1, 2, 4, 8), device="cuda")
        c = cb.KV8Cache(codes, scales, n_heads=32, dtype="bf16", weight_cells=cells)
        if cells < row:
            with pytest.raises(cb.CacheBlendError, match="cells"):
                c.attention_shared(table, lens, table + 1, lens, q)
        else:
            assert not c.attention_shared(table, lens, table + 1, lens, q).any()
        torch.cuda.synchronize()
        assert c.status() == 0
        c.close()
