"""GPU tests of what the launch over the sequences' own keys reads while the launch over their prefixes runs beside it: queries, lengths,
tables, offsets and rows that were written right before the call.  Results are compared bit by bit with those of the same calls
when each is waited for, which other tests compare with float64."""
import pytest

from test_gpu_kv8 import i32
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


@pytest.fixture(autouse=True)
def two_launches(monkeypatch):
    monkeypatch.setenv("CB_SHARED_AGAIN", "-1e15")


@pytest.mark.parametrize("dtype,G,prefixes,rows", [("bf16", 4, [600, 300], 1), ("bf16", 8, [1500, 40], 2), ("f32", 2, [500, 0], 1), ("bf16", 1, [90, 3000], 5)])
def test_inputs_written_right_before(cb, dtype, G, prefixes, rows):
    """Steps of one handle without a wait between them, as a graph and as calls: q is projected into one buffer and rotated there by the
    append, the sequences' lengths grow, the groups and the table's rows change places.  The kernels before are the framework's own, which
    let the next one start early, and torch's, which do not."""
    n, steps, H, hd, P = 40, 8, 2, 64, 16
    c = Shared(cb, prefixes, [60 + 3 * s for s in range(n)], [0, 25, n], [rows] * n, H=H, G=G, hd=hd, P=P, seed=G, spare=steps * rows, dtype=dtype)
    qs = [c.values(n * rows, H * G, hd)[0] for _ in range(steps)]
    kv = [c.values(n * rows, H, hd)[0] for _ in range(2 * steps)]
    tables = [c.own_table.clone() for _ in range(steps)]
    groups = [i32([i % 3, 10 + 3 * i, n - i % 2]) for i in range(steps)]
    lengths = [i32([60 + 3 * s + rows * (i + 1) for s in range(n)]) for i in range(steps)]
    for i in range(1, steps, 2):                       # pairs of sequences trade places
        for a in range(0, n - 1, 2):
            tables[i][[a, a + 1]] = tables[i][[a + 1, a]]
            lengths[i][[a, a + 1]] = lengths[i][[a + 1, a]]
    most = 60 + 3 * n + rows * steps
    first, q = groups[0].clone(), torch.zeros_like(qs[0])
    codes, scales = c.codes.clone(), c.scales.clone()
    outs = [torch.zeros_like(x) for x in qs]
    side = torch.cuda.Stream()

    def step(i, wait):
        with torch.cuda.stream(side):
            c.own_table.copy_(tables[i])
            c.own_lens.copy_(lengths[i])
            first.copy_(groups[i])
            q.copy_(qs[i])
        wait()
        c.cache.append(c.own_table, c.own_lens, q, kv[2 * i], kv[2 * i + 1], 1e4, out_q=q, max_len=most, stream=side)
        wait()
        c.cache.attention_shared(c.pre_table, c.pre_lens, c.own_table, c.own_lens, q, outs[i], prefix_start=first, max_len=most, stream=side)
        wait()

    def back():
        c.codes.copy_(codes)
        c.scales.copy_(scales)
        for o in outs:
            o.fill_(9.0)
        q.zero_()
        torch.cuda.synchronize()
    back()
    for i in range(steps):
        step(i, side.synchronize)
    want = [o.clone() for o in outs]
    assert not any((w == 9.0).all() for w in want)
    for _ in range(4):
        back()
        for i in range(steps):
            step(i, lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    back()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for i in range(steps):
            step(i, lambda: None)
    for _ in range(4):
        back()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert c.cache.status() == 0
    c.done()


def test_calls_behind_each_other(cb):
    """Two calls of one handle with nothing between them, the second with other inputs, also on two streams of which one waits for the
    other, and replays of a captured call behind eager ones: each call's own results."""
    n = 24
    c = Shared(cb, [400], [100 + s for s in range(n)], [0, n], [1] * n, H=2, G=4, hd=64, P=32, seed=2)
    a, b = (c.values(c.n_q, 8, 64)[0] for _ in range(2))
    start, first = i32(c.start), i32(c.first)
    few = i32([3 + s for s in range(n)])
    main, other = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros_like(a) for _ in range(3)]

    def call(q, lens, out, stream):
        c.cache.attention_shared(c.pre_table, c.pre_lens, c.own_table, lens, q, out, prefix_start=first, q_start=start, max_len=100 + n, stream=stream)
    torch.cuda.synchronize()
    want = []
    for q, lens in ((a, c.own_lens), (b, few), (b, c.own_lens)):
        call(q, lens, outs[0], main)
        main.synchronize()
        want.append(outs[0].clone())
    torch.cuda.synchronize()
    x, lens = a.clone(), c.own_lens.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        call(x, lens, outs[2], main)
    for _ in range(20):
        with torch.cuda.stream(main):
            x.copy_(a)
            lens.copy_(c.own_lens)
        call(a, c.own_lens, outs[0], main)
        call(b, few, outs[1], main)
        other.wait_stream(main)
        call(a, c.own_lens, outs[0], other)
        main.wait_stream(other)
        with torch.cuda.stream(main):
            x.copy_(b)
            graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert torch.equal(got, w)
    assert c.cache.status() == 0
    c.done()
