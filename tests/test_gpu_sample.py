"""GPU tests of cb_sample against its definition in float64.

Tolerance.  A weight of the library is off by at most 2^-31 of itself (the table's and the series' roundings 2^-32 and 2^-32.4, the
remainder's 2^-34, its constants' 2^-38) and by one unit of at least 2^-45 of the largest.  A sum of weights is then off by at
most 2^-31 of the sum S and n units, and so is the total it is compared with a fraction of: a border nearer to the exact one
than 2^-30 S + 2 n 2^-45 (times the largest weight) may fall to either side.  Where an exact sum lies that near to a border that
decides (of top-p, of min-p or of the uniform number), the row is not compared; every test says how many it compares.
Probabilities are off by 2^-30 + 2 n 2^-45 / S and a rounding to fp32, relative, and by a unit of their own weight: units are
2^-44 of a power of two that is at most the largest weight, and S is at least that, so 2^-44 of 1."""
import numpy as np
import pytest

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


def exact(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """(token, probability, whether a border is too near to tell) of one row of float64 logits."""
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if top == -np.inf:
        return -1, 0.0, False
    if not t >= 2.0 ** -126:
        return int(np.argmax(x)), 1.0, False
    if top == np.inf:
        w = (x == np.inf).astype(np.float64)
    else:
        with np.errstate(over="ignore"):
            w = np.exp((x - top) / t)
    n = len(x)
    order = np.argsort(-x, kind="stable")
    keep = order[:k] if 0 < k < n else order
    near = False
    if p < 1:
        s = np.cumsum(w[keep])
        before, total = s - w[keep], s[-1]
        target = max(p, 0.0) * total
        gap = np.abs(before[1:] - target)
        # (equal weights sum exactly: a border that is met exactly is no rounding)
        near |= bool(((gap < 2.0 ** -30 * total + n * 2.0 ** -44) & (gap > 0) & (w[keep][1:] > 2.0 ** -40)).any())
        ok = before < target
        ok[0] = True
        keep = keep[ok]
    if m > 0:
        m = min(m, 1.0)
        gap = np.abs(w[keep] - m)
        near |= bool(((gap < 2.0 ** -29 * m + 2.0 ** -43) & (gap > 0)).any())
        keep = keep[w[keep] >= m]
    kept = np.zeros(n, bool)
    kept[keep] = True
    c = np.cumsum(np.where(kept, w, 0.0))
    u = 0.0 if not u > 0 else u
    if u >= 1:
        i = int(np.nonzero(kept & (w > 2.0 ** -43))[0][-1])
        return i, w[i] / c[-1], near or bool((kept & (w > 2.0 ** -47) & (w < 2.0 ** -42)).any())
    i = min(int(np.searchsorted(c, u * c[-1], side="right")), n - 1)
    gap = np.abs(c[max(i - 1, 0):i + 1] - u * c[-1])
    near |= bool(((gap < 2.0 ** -30 * c[-1] + n * 2.0 ** -44) & (gap > 0)).any())
    return i, w[i] / c[-1], near


def dev(a, dtype=torch.float32):
    return None if a is None else torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def check(cb, logits, u, t=None, k=None, p=None, m=None, compared=0.9):
    """Runs the call and compares every row that can be told; settings are numpy arrays or None."""
    n, v = logits.shape
    f32 = [None if a is None else np.asarray(a, np.float32) for a in (u, t, p, m)]
    probs = torch.full((n,), 7.0, device="cuda")
    got = cb.cb_sample(logits, dev(f32[0]), temperature=dev(f32[1]), top_k=dev(k, torch.int32), top_p=dev(f32[2]), min_p=dev(f32[3]), out_probs=probs)
    tokens, probs = got.cpu().numpy(), probs.cpu().numpy()
    x = logits.float().cpu().numpy().astype(np.float64)
    told = 0
    for r in range(n):
        s = [d if a is None else float(a[r]) for a, d in zip((f32[1], f32[2], f32[3]), (1.0, 1.0, 0.0))]
        token, prob, near = exact(x[r], float(f32[0][r]), s[0], 0 if k is None else int(k[r]), s[1], s[2])
        if near:
            continue
        told += 1
        assert tokens[r] == token, (r, tokens[r], token, s, None if k is None else k[r], f32[0][r])
        assert abs(probs[r] - prob) <= (2.0 ** -24 + 2.0 ** -29 + v * 2.0 ** -43) * prob + 2.0 ** -44, (r, probs[r], prob)
    assert told >= compared * n, f"{told} of {n} rows could be compared"
    return tokens, probs


def rows_of(rng, n, v, dtype, spread=2.0):
    x = rng.normal(size=(n, v)) * spread
    for r in range(n):
        at = rng.integers(0, v, min(v, 40))
        x[r, at] += rng.exponential(3.0, len(at)) + 2 * spread
    return torch.from_numpy(x.astype(np.float32)).cuda().to(dtype)


F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("n,v,dtype", [(7, 1, F32), (9, 2, BF16), (20, 33, F32), (40, 1000, BF16), (30, 4097, F32), (64, 4096, F32), (12, 8200, BF16),
                                       (40, 32000, F32), (24, 50001, BF16), (20, 128256, F32), (2, 128256, BF16), (1, 128256, F32),
                                       (3, 393216, F32), (80, 20000, F32), (76, 131069, F32), (146, 65533, BF16)])
def test_settings(cb, n, v, dtype):
    """Every row its own settings, each of them off in some rows; clusters of 1 to 8 CTAs, parts of a row that end anywhere."""
    rng = np.random.default_rng(n * 1000 + v)
    for spread in (0.5, 3.0):
        x = rows_of(rng, n, v, dtype, spread)
        u = rng.random(n)
        t = np.where(rng.random(n) < 0.15, 0.0, rng.uniform(0.3, 1.6, n))
        k = np.where(rng.random(n) < 0.4, 0, np.minimum(np.exp(rng.uniform(0, 8, n)), 10 ** 6).astype(np.int64))
        p = np.where(rng.random(n) < 0.3, 1.0, rng.uniform(0.05, 0.999, n))
        m = np.where(rng.random(n) < 0.5, 0.0, rng.uniform(0, 0.3, n))
        check(cb, x, u, t, k, p, m)
        check(cb, x, u)
        check(cb, x, u, k=np.full(n, min(50, v)))
        check(cb, x, u, p=np.full(n, 0.9))


def test_every_token_has_its_share(cb):
    """Equally spaced uniform numbers give every token as many rows as its probability says."""
    rng = np.random.default_rng(5)
    n, v = 4000, 50
    one = torch.from_numpy((rng.normal(size=v) * 2).astype(np.float32)).cuda()
    x = one.expand(n, v).contiguous()
    u = (np.arange(n) + 0.5) / n
    for kw in (dict(), dict(p=np.full(n, 0.8)), dict(k=np.full(n, 7)), dict(m=np.full(n, 0.1)), dict(t=np.full(n, 0.5))):
        tokens, _ = check(cb, x, u, **kw)
        assert (np.diff(tokens) >= 0).all()
    w = np.exp(one.cpu().numpy().astype(np.float64))
    tokens, _ = check(cb, x, u)
    assert (np.abs(np.bincount(tokens, minlength=v) - n * w / w.sum()) <= 1).all()


@pytest.mark.parametrize("v", [3, 500, 5000, 70000])
def test_equal_logits(cb, v):
    """All logits equal: top-k and top-p keep the lowest tokens, to the exact border."""
    n = 40
    rng = np.random.default_rng(v)
    x = torch.full((n, v), 1.25, device="cuda")
    u = rng.random(n)
    check(cb, x, u)
    check(cb, x, u, k=np.arange(1, n + 1) * max(1, v // 50))
    check(cb, x, u, p=np.arange(1, n + 1) / 64)
    check(cb, x, u, m=np.full(n, 1.0))
    # v / 2 tokens sum to exactly half: the next is not kept
    if v % 2 == 0:
        tokens, _ = check(cb, x, np.full(n, 1.0), p=np.full(n, 0.5))
        assert (tokens == v // 2 - 1).all()


def test_many_ties(cb):
    """bf16 logits of few different values: the cut falls among thousands of equal ones, also after another cut among them."""
    rng = np.random.default_rng(1)
    n, v = 48, 100000
    x = torch.from_numpy(rng.integers(-6, 3, (n, v)).astype(np.float32) / 2).cuda().to(BF16)
    u = rng.random(n)
    k = rng.integers(1, v, n)
    check(cb, x, u, k=k)
    check(cb, x, u, p=rng.uniform(0.01, 0.99, n))
    check(cb, x, u, k=k, p=rng.uniform(0.1, 0.99, n), t=rng.uniform(0.3, 3, n))
    check(cb, x, u, k=rng.integers(1, 2000, n), p=rng.uniform(0.1, 0.99, n), m=np.full(n, 0.3))


def test_values_of_all_sizes(cb):
    """Outliers that leave all other values in one step of the histogram, again and again, and values next to each other."""
    rng = np.random.default_rng(2)
    n, v = 12, 30000
    x = np.empty((n, v), np.float32)
    for r in range(n):
        scale = 10.0 ** rng.integers(-30, 3, v) if r % 3 == 0 else np.full(v, 1e-6 if r % 3 == 1 else 1.0)
        x[r] = rng.normal(size=v) * scale
        if r % 2:
            x[r, rng.integers(0, v)] = 30.0 if r % 3 else 5.0
    x[3] = np.float32(1.0) + np.arange(v, dtype=np.float32) * np.float32(2.0 ** -23)         # all different, one step apart
    x[7] = -np.float32(2.0) ** -rng.integers(0, 140, v)                                       # crowded towards 0
    x = torch.from_numpy(x).cuda()
    u = rng.random(n)
    for kw in (dict(k=rng.integers(1, v, n)), dict(k=np.full(n, 3000)), dict(p=rng.uniform(0.1, 0.99, n)),
               dict(k=rng.integers(100, v, n), p=rng.uniform(0.1, 0.99, n)), dict(t=np.full(n, 1e3), k=np.full(n, 700), p=np.full(n, 0.7))):
        check(cb, x, u, **kw)


def test_masks_infinities_nan(cb):
    n, v = 16, 9000
    rng = np.random.default_rng(3)
    x = (rng.normal(size=(n, v)) * 2).astype(np.float32)
    low = np.finfo(np.float32).min
    x[0] = -np.inf
    x[1] = np.nan
    x[2], x[2, 77] = -np.inf, -5.0
    x[3], x[3, [5, 8000]] = low, [1.0, 1.5]
    x[4] = low                                          # equal, finite: all alike
    x[5, [3, 4000, 8999]] = np.inf
    x[6, 10] = np.inf
    x[7, ::2] = np.nan
    x[8, 1:] = -np.inf
    x[9] = 3e38
    x[10, :4500] = -np.inf
    x[11], x[11, [1, 2]] = -0.0, 0.0
    x[12] = -np.inf
    x[12, 4096:4100] = [1, 2, 2, 1]
    x[13] = low
    x[13, 1] = 3e38
    u = rng.random(n)
    for dtype in (F32, BF16):
        t = torch.from_numpy(x).cuda().to(dtype)
        tokens, probs = check(cb, t, u)
        assert (tokens[:2] == -1).all() and (probs[:2] == 0).all() and tokens[2] == 77 and tokens[8] == 0
        for kw in (dict(k=np.full(n, 2)), dict(k=np.full(n, 8000), p=np.full(n, 0.6)), dict(p=np.full(n, 0.9)), dict(m=np.full(n, 0.5)), dict(t=np.zeros(n))):
            check(cb, t, u, **kw)


def test_settings_out_of_range(cb):
    """Temperatures from nothing to infinity, uniform numbers outside [0, 1), settings that are off or beyond."""
    rng = np.random.default_rng(4)
    t = [0.0, -1.0, np.nan, 1e-45, 1.2e-38, 1e-20, 1e-4, 0.01, 50.0, 1e5, 1e30, np.inf]
    n, v = len(t), 5000
    x = rows_of(rng, n, v, F32)
    x[:, 17] = x[:, 4011] = x.max(dim=1).values         # three likeliest tokens with the one whose value it is
    u = rng.random(n)
    tokens, probs = check(cb, x, u, t=np.where(np.isinf(t), 3.4e38, t))
    again = cb.cb_sample(x, dev(u), temperature=dev(t)).cpu().numpy()
    assert (again[:11] == tokens[:11]).all() and (tokens[:4] == x[:4].argmax(dim=1).cpu().numpy()).all() and 0 <= again[11] < v
    assert (probs[4:6] == np.float32(1 / 3)).all()
    for odd, like in ((-3.0, 0.0), (np.nan, 0.0), (1.0, 1.0), (7.0, 1.0), (np.inf, 1.0)):
        got, _ = check(cb, x, np.full(n, odd), t=np.full(n, 0.7), k=np.full(n, 5))
        same, _ = check(cb, x, np.full(n, like), t=np.full(n, 0.7), k=np.full(n, 5))
        assert (got == same).all()
    plain, _ = check(cb, x, u)
    for kw in (dict(k=np.full(n, -5)), dict(k=np.full(n, v)), dict(k=np.full(n, 2 ** 31 - 1)), dict(p=np.full(n, 1.5)), dict(p=np.full(n, np.nan)),
               dict(m=np.full(n, -1.0)), dict(m=np.full(n, np.nan))):
        got = cb.cb_sample(x, dev(u), top_k=dev(kw.get("k"), torch.int32), top_p=dev(kw.get("p")), min_p=dev(kw.get("m"))).cpu().numpy()
        assert (got == plain).all()
    first = x.argmax(dim=1).cpu().numpy()
    for kw in (dict(k=np.ones(n, int)), dict(p=np.zeros(n)), dict(p=np.full(n, -1.0)), dict(p=np.full(n, 1e-30))):
        got, _ = check(cb, x, u, **kw)
        assert (got == first).all()
    check(cb, x, u, m=np.full(n, 5.0))


def test_rows_anywhere(cb):
    """Rows that begin at any element, strides of any size, one row as a vector; what lies between rows is not read."""
    rng = np.random.default_rng(6)
    for dtype in (F32, BF16):
        for v, stride, first in ((1001, 1003, 1), (4099, 4100, 3), (777, 777, 2), (5000, 5008, 0)):
            n = 5
            buf = torch.full((n * stride + 8,), float("inf"), dtype=dtype, device="cuda")
            x = buf[first:first + n * stride].view(n, stride)[:, :v]
            x.copy_(rows_of(rng, n, v, dtype))
            check(cb, x, rng.random(n), p=np.full(n, 0.9))
    x = rows_of(rng, 1, 2000, F32)
    assert cb.cb_sample(x[0], dev([0.3])).tolist() == cb.cb_sample(x, dev([0.3])).tolist()
    assert cb.cb_sample(x[:0], dev([])).shape == (0,)


def test_streams_graphs_and_repeats(cb):
    """Two calls at once on two streams, a captured call that follows its inputs, and the same result every time."""
    rng = np.random.default_rng(7)
    n, v = 30, 60000
    a, b = rows_of(rng, n, v, F32), rows_of(rng, n, v, BF16)
    u, t, p, k = dev(rng.random(n)), dev(rng.uniform(0.5, 1.5, n)), dev(np.full(n, 0.95)), dev(np.full(n, 400), torch.int32)
    kw = dict(temperature=t, top_p=p, top_k=k)
    ref_a, ref_b = cb.cb_sample(a, u, **kw), cb.cb_sample(b, u, **kw)
    s, z = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        ta, tb = cb.cb_sample(a, u, stream=s, **kw), cb.cb_sample(b, u, stream=z, **kw)
        s.synchronize()
        z.synchronize()
        assert torch.equal(ta, ref_a) and torch.equal(tb, ref_b)
    out, probs, x = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, device="cuda"), a.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cb.cb_sample(x, u, out_tokens=out, out_probs=probs, stream=s, **kw)
    for src in (a, b, -a):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, cb.cb_sample(x, u, **kw))


def test_refusals(cb):
    x, u = torch.zeros((3, 100), device="cuda"), torch.zeros(3, device="cuda")
    for bad, word in ((dict(logits=x.half()), "logits"), (dict(logits=x.cpu()), "logits"), (dict(logits=x.t()), "logits"), (dict(logits=x[:, ::2]), "contiguous"),
                      (dict(uniform=None), "uniform"), (dict(uniform=u[:2]), "uniform"), (dict(uniform=u.double()), "uniform"),
                      (dict(temperature=u.cpu()), "temperature"), (dict(top_k=u), "top_k"), (dict(top_p=u[:1]), "top_p"), (dict(min_p=u.int()), "min_p"),
                      (dict(out_tokens=u), "out_tokens"), (dict(out_probs=u[::2]), "out_probs")):
        with pytest.raises(ValueError, match=word):
            cb.cb_sample(**{**dict(logits=x, uniform=u), **bad})
    with pytest.raises(cb.CacheBlendError) as e:
        cb.cb_sample(torch.zeros((1, cb.CB_SAMPLE_MAX_VOCAB + 1), device="cuda"), u[:1])
    assert e.value.code == cb.CB_ERR_UNSUPPORTED
    with pytest.raises(cb.CacheBlendError, match="stride"):
        cb.cb_sample(x[:1].expand(3, 100), u)
