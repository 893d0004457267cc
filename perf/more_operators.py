"""Measured cases of the operators of a decoding step on a blended context: new rows rotated and appended to the 8-bit
paged K/V cache, attention of sequences that share a prefix, and the choice of the next token.

The cache holds e4m3 codes ``[layer][K|V][page][KV head][row of the page][head_dim]`` and one float32 scale, a power of
two, for each block (a page's rows of one KV head, in one layer's K or V).  Logical row j of a sequence is row j % P of
page ``table[j // P]``.  Sequence lengths, block tables, positions and offsets are device arrays.

  append  new rows of q, k and v as the projections give them: q and k are rotated at their rows' positions, pair
          (2i, 2i + 1) of a head by the angle position * theta^(-2i / head_dim), and k and v become the last rows of
          their sequences.  A row's position is given, or is its place in its sequence.  Scale of a block: 0 when every
          value is 0, else the smallest power of two s with max|x| <= 448 s; a block that already holds rows of the
          sequence keeps the larger of its old scale and the new rows' one, and its old codes are rounded to it.
  shared  softmax(q k / sqrt(head_dim)) v, where the sequences of a group see all rows of the group's prefix (stored
          once) and then their own: query row i of a sequence's n sees its own rows 0 .. len - n + i.
  sample  a token per row of logits x: weights exp((x - max) / temperature), in descending order (ties to the lower
          token); of the first top_k those before which the weights sum to less than top_p of theirs; of those the ones
          of at least min_p times the largest.  The token is the lowest i whose kept weights up to i pass
          uniform * (their sum); its probability is its weight over that sum.  Temperature 0 takes the most likely.
"""
import numpy as np
import torch

own = False

SUPPORTED_PAGES = (16, 32, 64, 128, 256)


# --------------------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------------------
def _rows_case(op, *, heads=32, kv_heads=8, head_dim=128, dtype="bf16", page=64, seqs=1, length=8192, ragged=False, rows=1,
               theta=5e5, far=False, groups=1, prefix=0, name=None):
    c = dict(op=op, heads=heads, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, page=page, seqs=seqs, length=length,
             ragged=ragged, rows=rows, theta=theta, far=far, groups=groups, prefix=prefix)
    if name:
        c["name"] = name
    return c


def _sample_case(*, rows=1, vocab=128256, dtype="f32", temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, mixed=False, spread=2.0, name=None):
    c = dict(op="sample", rows=rows, vocab=vocab, dtype=dtype, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p,
             mixed=mixed, spread=spread)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decoding step of a batch, one layer: each sequence's new token joins its last page
        _rows_case("append", seqs=64, length=8256, ragged=True, name="append 64 x 1"),
        # a prompt of 8K tokens, one layer
        _rows_case("append", length=8192, rows=8192, name="append 8k"),
        # a few speculated tokens of a small fp32 model on a cache from which rows were evicted: positions far behind places
        _rows_case("append", heads=16, kv_heads=4, head_dim=64, dtype="f32", page=32, seqs=8, length=2080, ragged=True, rows=5,
                   theta=1e4, far=True, name="append 8 x 5 far f32"),
        # three short answers to one short context: latency
        _rows_case("shared", seqs=3, length=40, ragged=True, prefix=300, name="shared 3 x (300 + 40)"),
        # a decoding step of a server's batch: all requests on one retrieved context of 8K
        _rows_case("shared", seqs=64, length=256, ragged=True, prefix=8192, name="shared 64 x (8k + 256)"),
        # four documents, sixteen requests on each, answers of any length so far
        _rows_case("shared", seqs=64, length=512, ragged=True, prefix=4096, groups=4, page=32, name="shared 4 x 16 x (4k + 512)"),
        # few requests on a very long context in small pages
        _rows_case("shared", seqs=8, length=1000, ragged=True, prefix=131071, page=16, name="shared 8 x (128k + 1000)"),
        # speculated tokens of a small fp32 model
        _rows_case("shared", heads=16, kv_heads=4, head_dim=64, dtype="f32", page=32, seqs=4, length=100, ragged=True, rows=5,
                   prefix=2080, name="shared 4 x 5 x (2k + 100) f32"),
        # the next token of one request, usual settings: latency
        _sample_case(temperature=0.8, top_k=50, top_p=0.95, name="sample 1 top-k top-p"),
        # a batch, the nucleus of a wide distribution
        _sample_case(rows=64, top_p=0.9, name="sample 64 top-p"),
        # a large batch of bf16 logits of a small vocabulary: ties
        _sample_case(rows=256, vocab=32000, dtype="bf16", temperature=1.3, min_p=0.02, name="sample 256 min-p bf16"),
        # a server's batch, every request with settings of its own
        _sample_case(rows=40, mixed=True, spread=2.5, name="sample 40 mixed"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    largest = {}
    for c in listed():
        w = work(c)
        for k in w:
            largest[c["op"], k] = max(largest.get((c["op"], k), 0), w[k])
    while True:
        op = rng.choice(["append", "shared", "shared", "sample", "sample"])
        if op == "sample":
            c = _sample_case(rows=_log_int(rng, 1, 256), vocab=_log_int(rng, 700, 200000), dtype=rng.choice(["f32", "f32", "bf16"]),
                             temperature=rng.choice([1.0, round(rng.uniform(0.3, 2.0), 2)]), spread=round(rng.uniform(1.0, 4.0), 2))
            c["top_k"] = rng.choice([0, 0, _log_int(rng, 1, 2000)])
            c["top_p"] = rng.choice([1.0, round(rng.uniform(0.3, 0.99), 3)])
            c["min_p"] = rng.choice([0.0, 0.0, round(rng.uniform(0.001, 0.3), 4)])
            c["mixed"] = rng.random() < 0.3
        else:
            kv_heads = rng.choice([1, 2, 4, 8, 8])
            group = rng.choice([1, 2, 3, 4, 4, 7, 8])
            c = _rows_case(op, heads=kv_heads * group, kv_heads=kv_heads, head_dim=rng.choice([64, 128, 128]), page=rng.choice(SUPPORTED_PAGES),
                           dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), theta=rng.choice([1e4, 5e5, 1e6]))
            c["ragged"] = rng.random() < 0.7
            c["seqs"] = _log_int(rng, 1, 64)
            c["rows"] = rng.choice([1, 1, 1, 2, 5])
            if op == "append":
                c["far"] = rng.random() < 0.4
                c["length"] = _log_int(rng, 17, 8192)
                c["rows"] = rng.choice([c["rows"], rng.randint(1, c["length"]), c["length"]])
            else:
                c["length"] = _log_int(rng, 5, 2000)
                c["prefix"] = _log_int(rng, 17, 131071)
                c["groups"] = rng.choice([1, 1, 1, rng.randint(1, min(8, c["seqs"]))])
            c["rows"] = min(c["rows"], c["length"])
        w = work(c)
        pool = 0 if op == "sample" else (c["seqs"] * c["length"] + c["groups"] * c["prefix"]) * c["kv_heads"] * c["head_dim"] * 2
        if all(w[k] <= largest[op, k] for k in w) and pool <= 2 * 10 ** 9:
            return c


def _lengths(case):
    """Row count of each sequence: `length`, or ragged ones up to it (the first is the longest), from the case alone."""
    n, top = case["seqs"], case["length"]
    if not case["ragged"] or n == 1:
        return [top] * n
    r = np.random.RandomState(n * 7919 + top)
    return [top] + [int(v) for v in r.randint(max(case["rows"], top // 16), top + 1, n - 1)]


def _prefixes(case):
    """(rows of each group's prefix, first sequence of each group and their number)."""
    n, g, top = case["seqs"], case["groups"], case["prefix"]
    if g == 1:
        return [top], [0, n]
    r = np.random.RandomState(g * 104729 + top)
    lens = [top] + [int(v) for v in r.randint(max(1, top // 4), top + 1, g - 1)]
    return lens, [0] + sorted(int(v) for v in r.choice(np.arange(1, n), g - 1, replace=False)) + [n]


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (4.0 if case["dtype"] == "f32" else 2.0) + 28.0 * case["rows"], "flops": 4.0 * n}
    lens, rows = _lengths(case), case["rows"]
    hq, hkv, hd, es = case["heads"], case["kv_heads"], case["head_dim"], 2 if case["dtype"] == "bf16" else 4
    n = rows * case["seqs"]
    if case["op"] == "append":
        blocks = sum(-(-l // case["page"]) - (l - rows) // case["page"] for l in lens)
        return {"bytes": 2.0 * n * hq * hd * es + 2.0 * hkv * (n * hd * (es + 1) + blocks * 4), "flops": 3.0 * n * (hq + hkv) * hd}
    shared, first = _prefixes(case)
    keys = sum(lens) + sum(shared)
    blocks = sum(-(-l // case["page"]) for l in lens + shared)
    seen = sum(l - rows + i + 1 for l in lens for i in range(rows))
    seen += sum(l * (first[g + 1] - first[g]) * rows for g, l in enumerate(shared))
    return {"bytes": 2.0 * hkv * (keys * hd + blocks * 4) + 2.0 * n * hq * hd * es, "flops": 4.0 * hd * hq * seen}


# --------------------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------------------
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _logits(case, g):
    """Normal logits with a number of likely tokens above them, as a language model gives them."""
    n, v = case["rows"], case["vocab"]
    x = torch.randn((n, v), generator=g, device="cuda") * case["spread"]
    at = torch.randint(0, v, (n, 48), generator=g, device="cuda")
    lift = torch.empty((n, 48), device="cuda").exponential_(1.0, generator=g) * 3.0
    return (x.scatter_add_(1, at, lift + 2.0 * case["spread"])).to(_dtype(case))


def _settings(case, cpu):
    """Temperature, top-k, top-p and min-p of each row, None where no row has one."""
    n = case["rows"]
    if not case["mixed"]:
        def one(v, off, t):
            return None if v == off else torch.full((n,), v, dtype=t, device="cuda")
        return dict(temperature=one(case["temperature"], 1.0, torch.float32), top_k=one(case["top_k"], 0, torch.int32),
                    top_p=one(case["top_p"], 1.0, torch.float32), min_p=one(case["min_p"], 0.0, torch.float32))
    u = torch.rand((5, n), generator=cpu)
    t = torch.where(u[0] < 0.2, 0.0, 0.3 + 1.2 * u[0])                       # a fifth of the requests are greedy
    k = torch.where(u[1] < 0.5, 0, torch.exp(7.0 * u[2])).to(torch.int32)    # off, or up to a thousand
    p = torch.where(u[2] < 0.4, 1.0, 0.5 + 0.49 * u[3])
    m = torch.where(u[4] < 0.6, 0.0, 0.2 * u[4] * u[3])
    return dict(temperature=t.cuda(), top_k=k.cuda(), top_p=p.cuda(), min_p=m.cuda())


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    cpu = torch.Generator()
    cpu.manual_seed(int(seed) * 999983 + 7)
    if case["op"] == "sample":
        n = case["rows"]
        return dict(case=case, logits=_logits(case, g), uniform=torch.rand(n, generator=g, device="cuda"), **_settings(case, cpu),
                    tokens=torch.zeros(n, dtype=torch.int32, device="cuda"), probs=torch.zeros(n, device="cuda"))
    B, P, hkv, hd, hq = case["seqs"], case["page"], case["kv_heads"], case["head_dim"], case["heads"]
    lens, (shared, first) = _lengths(case), _prefixes(case)
    if case["op"] == "append":
        shared = []
    used = [-(-l // P) for l in lens + shared]
    n_pages = sum(used) + 3
    order = torch.randperm(n_pages, generator=cpu, dtype=torch.int64).to(torch.int32)
    table = torch.zeros((B, max(used[:B])), dtype=torch.int32)
    above = torch.zeros((len(shared), max(used[B:] + [1])), dtype=torch.int32)
    at = 0
    for s, u in enumerate(used):
        row = table[s] if s < B else above[s - B]
        row[:u] = order[at:at + u]
        at += u
    gain = torch.ones((hkv, hd), device="cuda")                   # a few channels of keys are much larger
    gain[:, torch.randperm(hd, generator=cpu)[:4].cuda()] = 6.0
    # the pool as it stands: every block quantised from normal values, their size drifting from page to page
    codes = torch.empty((1, 2, n_pages, hkv, P, hd), dtype=torch.uint8, device="cuda")
    scales = torch.empty((1, 2, n_pages, hkv), dtype=torch.float32, device="cuda")
    for kv in range(2):
        x = torch.randn((n_pages, hkv, P, hd), generator=g, device="cuda")
        x *= torch.exp2(torch.randn((n_pages, 1, 1, 1), generator=g, device="cuda") * 0.7)
        if kv == 0:
            x *= gain[None, :, None, :]
        s = _scale_of(x.abs().amax(dim=(2, 3)))
        scales[0, kv] = s
        codes[0, kv] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        del x
    n = B * case["rows"]
    state = dict(case=case, codes=codes, scales=scales, table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                 max_len=max(lens), q=torch.randn((n, hq, hd), generator=g, device="cuda").to(_dtype(case)),
                 out=torch.zeros((n, hq, hd), dtype=_dtype(case), device="cuda"))
    if case["op"] == "append":
        state["k"] = (torch.randn((n, hkv, hd), generator=g, device="cuda") * gain).to(_dtype(case))
        state["v"] = torch.randn((n, hkv, hd), generator=g, device="cuda").to(_dtype(case))
        place = (state["lens"] - case["rows"])[:, None] + torch.arange(case["rows"], device="cuda", dtype=torch.int32)
        behind = torch.randint(0, 120000, (B, 1), generator=g, device="cuda", dtype=torch.int32) if case["far"] else 0
        state["positions"] = (place + behind).reshape(-1).contiguous() if case["far"] else None
    else:
        state["above"] = above.cuda()
        state["above_lens"] = torch.tensor(shared, dtype=torch.int32).cuda()
        state["first"] = torch.tensor(first, dtype=torch.int32).cuda()
        state["members"] = first                                  # the same on the host: a scheduler has both
        state["longest"] = shared
    if own:
        import cacheblend_selective_kv_gb300 as cb
        cells = cb.KV8Cache.shared_cells(n, hq, hd) if case["op"] == "shared" else 0
        state["cache"] = cb.KV8Cache(codes, scales, n_heads=hq, dtype=case["dtype"], weight_cells=cells)
    return state


# --------------------------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------------------------
def run(state):
    return {"append": _append, "shared": _shared, "sample": _sample}[state["case"]["op"]](state)


def _scale_of(top):
    """The smallest power of two s with top <= 448 s (0 for 0): 448 = 0.875 * 2^9."""
    m, e = torch.frexp(top)
    s = torch.ldexp(torch.ones_like(top), torch.clamp(e - 9 + (m > 0.875).to(e.dtype), min=-126))
    return torch.where(top > 0, s, torch.zeros_like(s))


def _to_codes(x, s):
    return torch.where(s > 0, x / torch.where(s > 0, s, 1.0), torch.zeros_like(x)).to(torch.float8_e4m3fn)


def _rotated(x, cos, sin):
    """float32 x [rows][heads][dim] with pairs (2i, 2i + 1) turned; cos, sin [rows][dim / 2]."""
    a, b, c, s = x[..., 0::2], x[..., 1::2], cos[:, None], sin[:, None]
    return torch.stack((a * c - b * s, a * s + b * c), dim=-1).flatten(-2)


def _append(state):
    case, codes, scales = state["case"], state["codes"], state["scales"]
    if own:
        state["cache"].append(state["table"], state["lens"], state["q"], state["k"], state["v"], case["theta"], out_q=state["out"],
                              positions=state["positions"], max_len=state["max_len"])
        return {"q": state["out"], "codes": codes.view(torch.float8_e4m3fn), "scales": scales}
    B, P, rows, hkv, hd = case["seqs"], case["page"], case["rows"], case["kv_heads"], case["head_dim"]
    lens = state["lens"].long()
    new = lens[:, None] - rows + torch.arange(rows, device="cuda")                # places of the new rows [B][rows]
    pos = new.reshape(-1) if state["positions"] is None else state["positions"]
    i = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    angle = pos.double()[:, None] * torch.pow(torch.tensor(case["theta"], dtype=torch.float64, device="cuda"), -2.0 * i / hd)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    state["out"].copy_(_rotated(state["q"].float(), cos, sin).to(state["out"].dtype))
    first = (lens - rows) // P                                                    # first block of each sequence that gets a row
    block = first[:, None] + torch.arange((rows + P - 2) // P + 1, device="cuda")
    live = block * P < lens[:, None]
    page = state["table"].long().gather(1, torch.where(live, block, torch.zeros_like(block)))
    j = block[:, :, None] * P + torch.arange(P, device="cuda")                    # row of each row of those blocks [B][n][P]
    fresh = (j >= (lens - rows)[:, None, None]) & (j < lens[:, None, None])
    old = j < (lens - rows)[:, None, None]
    src = torch.where(fresh, j - (lens - rows)[:, None, None] + (torch.arange(B, device="cuda") * rows)[:, None, None], torch.zeros_like(j))
    f = fresh[..., None, None]
    for kv, x in ((0, _rotated(state["k"].float(), cos, sin)), (1, state["v"].float())):
        x = torch.where(f, x[src], 0.0)                                           # [B][n][P][heads][dim]
        s = _scale_of(x.abs().amax(dim=(2, 4)))                                   # [B][n][heads]
        was = torch.where(old.any(2)[..., None], scales[0, kv][page], 0.0)
        s = torch.maximum(s, was)
        before = codes[0, kv][page].transpose(2, 3)
        held = torch.where(old[..., None, None], before.view(torch.float8_e4m3fn).float() * was[:, :, None, :, None], x)
        c = _to_codes(held, s[:, :, None, :, None]).view(torch.uint8)
        c = torch.where(f | old[..., None, None], c, before)
        codes[0, kv][page[live]] = c.transpose(2, 3)[live]
        scales[0, kv][page[live]] = s[live]
    return {"q": state["out"], "codes": codes.view(torch.float8_e4m3fn), "scales": scales}


def _values(state, kv, page, row):
    """Rows of the pool as the float32 values they stand for: page and row [...] -> [...][KV heads][head_dim]."""
    c = state["codes"][0, kv].transpose(1, 2)[page, row]
    return c.view(torch.float8_e4m3fn).float() * state["scales"][0, kv][page][..., None]


def _shared(state):
    case = state["case"]
    if own:
        state["cache"].attention_shared(state["above"], state["above_lens"], state["table"], state["lens"], state["q"], state["out"],
                                        prefix_start=state["first"], prefix_max_len=max(state["longest"]), max_len=state["max_len"])
        return {"out": state["out"]}
    P, rows, hkv, hd, hq, top = case["page"], case["rows"], case["kv_heads"], case["head_dim"], case["heads"], state["max_len"]
    G = hq // hkv
    j, i = torch.arange(top, device="cuda"), torch.arange(rows, device="cuda")
    for g, n_prefix in enumerate(state["longest"]):
        lo, hi = state["members"][g], state["members"][g + 1]
        B = hi - lo
        lens = state["lens"][lo:hi].long()
        q = state["q"][lo * rows:hi * rows].float().view(B, rows, hkv, G, hd).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * rows, hd) / hd ** 0.5
        # scores with the prefix, whose keys all of the group's rows see, and with each sequence's own rows
        a = torch.arange(n_prefix, device="cuda")
        page = state["above"][g].long()[a // P]
        shared = torch.matmul(q.transpose(0, 1).reshape(hkv, -1, hd), _values(state, 0, page, a % P).permute(1, 2, 0))
        valid = j < lens[:, None]
        mine = torch.where(valid, state["table"][lo:hi].long().gather(1, (j // P).expand(B, top)), 0)
        k = _values(state, 0, mine, (j % P).expand(B, top)).transpose(1, 2)       # [B][heads][keys][dim]
        x = torch.matmul(q, k.transpose(2, 3))
        sees = (j <= (lens - rows)[:, None, None] + i[:, None]).repeat(1, G, 1)[:, None]
        x = torch.where(sees, x, -torch.inf)
        shared = shared.view(hkv, B, G * rows, n_prefix).transpose(0, 1)
        m = torch.maximum(shared.amax(dim=3, keepdim=True), x.amax(dim=3, keepdim=True))
        shared, x = torch.exp(shared - m), torch.exp(x - m)
        total = shared.sum(dim=3, keepdim=True) + x.sum(dim=3, keepdim=True)
        v = torch.where(valid[:, None, :, None], _values(state, 1, mine, (j % P).expand(B, top)).transpose(1, 2), 0.0)
        o = torch.matmul(x, v)
        over = torch.matmul(shared.transpose(0, 1).reshape(hkv, -1, n_prefix), _values(state, 1, page, a % P).transpose(0, 1))
        o = (o + over.view(hkv, B, G * rows, hd).transpose(0, 1)) / total
        o = o.view(B, hkv, G, rows, hd).permute(0, 3, 1, 2, 4).reshape(B * rows, hq, hd)
        state["out"][lo * rows:hi * rows] = o.to(state["out"].dtype)
    return {"out": state["out"]}


def _sample(state):
    if own:
        import cacheblend_selective_kv_gb300 as cb
        cb.cb_sample(state["logits"], state["uniform"], temperature=state["temperature"], top_k=state["top_k"], top_p=state["top_p"],
                     min_p=state["min_p"], out_tokens=state["tokens"], out_probs=state["probs"])
        return {"tokens": state["tokens"], "probs": state["probs"]}
    # in 64 bits: a sum over the vocabulary decides between neighbouring tokens
    x = state["logits"].double()
    n, v = x.shape
    t = torch.ones(n, device="cuda") if state["temperature"] is None else state["temperature"]
    greedy = t <= 0
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((x - x[:, :1]) / torch.where(greedy, 1.0, t).double()[:, None])
    keep = torch.ones((n, v), dtype=torch.bool, device="cuda")
    rank = torch.arange(v, device="cuda")
    if state["top_k"] is not None:
        keep &= (rank < state["top_k"][:, None]) | (state["top_k"] <= 0)[:, None]
    if state["top_p"] is not None:
        of = torch.where(keep, w, 0.0)
        upto = torch.cumsum(of, dim=1)
        keep &= (upto - of < state["top_p"].double()[:, None] * upto[:, -1:]) | (state["top_p"] >= 1)[:, None]
    if state["min_p"] is not None:
        keep &= w >= state["min_p"].double()[:, None]
    keep &= (rank == 0) | ~greedy[:, None]
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))         # back in the tokens' order
    upto = torch.cumsum(w, dim=1)
    token = torch.searchsorted(upto, state["uniform"].double()[:, None] * upto[:, -1:], right=True)
    state["tokens"].copy_(token[:, 0])
    state["probs"].copy_((w.gather(1, token) / upto[:, -1:])[:, 0])
    return {"tokens": state["tokens"], "probs": state["probs"]}


# --------------------------------------------------------------------------------------------------------------
# the definition in 64 bits, row by row
# --------------------------------------------------------------------------------------------------------------
def _grid(x):
    """float64 x (|x| <= 448) rounded to the nearest number with a sign, four significant bits and a last place of at
    least 2^-9, ties to the even one."""
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -60))), min=-6.0) - 3.0)
    return torch.round(x / step) * step


def _pow2_at_least(top):
    """Per element the smallest power of two s with top <= 448 s, by trying the neighbours of the logarithm; 0 for 0."""
    e = torch.floor(torch.log2(torch.clamp(top, min=2.0 ** -140) / 448.0)) - 1.0
    for _ in range(3):
        e = torch.where(top > 448.0 * torch.exp2(e), e + 1.0, e)
    return torch.where(top > 0, torch.exp2(torch.clamp(e, min=-126.0)), 0.0)


def _numbers():
    """Codes as float64 numbers, through a table of the 256 codes."""
    i = torch.arange(256, dtype=torch.float64)
    sign, e, m = torch.where(i >= 128, -1.0, 1.0), (i % 128) // 8, i % 8
    t = sign * torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
    t[127] = t[255] = float("nan")
    t = t.cuda()
    return lambda c: t[c.long()]


def _exact_sample(state):
    n = state["case"]["rows"]
    settings = [None if state[s] is None else state[s].tolist() for s in ("temperature", "top_k", "top_p", "min_p")]
    tokens = torch.zeros(n, dtype=torch.int32, device="cuda")
    probs = torch.zeros(n, dtype=torch.float64, device="cuda")
    for r, u in enumerate(state["uniform"].tolist()):
        t, k, p, m = (s[r] if s is not None else d for s, d in zip(settings, (1.0, 0, 1.0, 0.0)))
        x = state["logits"][r].double()
        if t <= 0:
            tokens[r], probs[r] = int(torch.nonzero(x == x.max())[0, 0]), 1.0
            continue
        w = torch.exp((x - x.max()) / t)
        by = torch.argsort(x, descending=True, stable=True)
        if k > 0:
            by = by[:k]
        if p < 1:
            s = torch.cumsum(w[by], 0)
            before = torch.cat((s.new_zeros(1), s[:-1]))
            by = by[before < p * s[-1]]
        by = by[w[by] >= m].sort().values
        s = torch.cumsum(w[by], 0)
        i = min(int((s <= u * s[-1]).sum()), len(by) - 1)
        tokens[r], probs[r] = int(by[i]), float(w[by[i]] / s[-1])
    return {"tokens": tokens, "probs": probs}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(state)
    number = _numbers()
    P, hkv, hd, hq, rows = case["page"], case["kv_heads"], case["head_dim"], case["heads"], case["rows"]
    G = hq // hkv
    lens, table = _lengths(case), state["table"].tolist()
    codes, scales = state["codes"], state["scales"]
    if case["op"] == "append":
        place = torch.cat([torch.arange(n - rows, n, device="cuda") for n in lens])
        pos = (place if state["positions"] is None else state["positions"]).double()
        turn = torch.stack([pos * case["theta"] ** (-2.0 * i / hd) for i in range(hd // 2)], dim=1)
        z = torch.polar(torch.ones_like(turn), turn)[:, None]                     # a pair as one complex number

        def rotate(x):
            return torch.view_as_real(torch.view_as_complex(x.double().unflatten(-1, (hd // 2, 2))) * z).flatten(-2)
        new_codes, new_scales = number(codes[0]), scales[0].double()
        for kv, x in ((0, rotate(state["k"])), (1, state["v"].double())):
            for s, n in enumerate(lens):
                lo = (n - rows) // P * P
                have = n - rows - lo                                              # rows of the first block that stay
                pg = torch.tensor(table[s][lo // P:-(-n // P)], device="cuda")
                b = torch.zeros((len(pg) * P, hkv, hd), dtype=torch.float64, device="cuda")
                b[have:have + rows] = x[s * rows:(s + 1) * rows]
                b = b.view(len(pg), P, hkv, hd).transpose(1, 2)
                sc = _pow2_at_least(b.abs().amax(dim=(2, 3)))
                if have:
                    was = scales[0, kv, pg[0]].double()
                    sc[0] = torch.maximum(sc[0], was)
                    b[0, :, :have] = number(codes[0, kv, pg[0]])[:, :have] * was[:, None, None]
                c = _grid(b / torch.where(sc > 0, sc, 1.0)[..., None, None]).transpose(1, 2).reshape(-1, hkv, hd)
                kept = new_codes[kv][pg].transpose(1, 2).reshape(-1, hkv, hd)
                kept[:have + rows] = c[:have + rows]
                new_codes[kv][pg] = kept.view(len(pg), P, hkv, hd).transpose(1, 2)
                new_scales[kv][pg] = sc
        return {"q": rotate(state["q"]), "codes": new_codes[None], "scales": new_scales[None]}

    def whole(kv, pages, n):
        """The n rows of these pages as [rows][heads][dim]."""
        pg = torch.tensor(pages[:-(-n // P)], device="cuda")
        x = number(codes[0, kv][pg]) * scales[0, kv][pg].double()[..., None, None]
        return x.transpose(1, 2).reshape(-1, hkv, hd)[:n]
    shared, first = _prefixes(case)
    above = state["above"].tolist()
    out = torch.zeros(state["out"].shape, dtype=torch.float64, device="cuda")
    for g, n_prefix in enumerate(shared):
        kp, vp = whole(0, above[g], n_prefix), whole(1, above[g], n_prefix)
        for s in range(first[g], first[g + 1]):
            n = lens[s]
            ks, vs = whole(0, table[s], n), whole(1, table[s], n)
            unseen = torch.arange(n, device="cuda")[None] > n - rows + torch.arange(rows, device="cuda")[:, None]
            q = state["q"][s * rows:(s + 1) * rows].double()
            for h in range(hkv):
                qh = q[:, h * G:(h + 1) * G].transpose(0, 1)                      # [G][rows][dim]
                x = torch.cat((qh @ kp[:, h].T, (qh @ ks[:, h].T).masked_fill(unseen, -torch.inf)), dim=2) * hd ** -0.5
                p = torch.softmax(x, dim=2)
                o = p[:, :, :n_prefix] @ vp[:, h] + p[:, :, n_prefix:] @ vs[:, h]
                out[s * rows:(s + 1) * rows, h * G:(h + 1) * G] = o.transpose(0, 1)
    return {"out": out}
