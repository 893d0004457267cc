"""Measured cases of the operators on the 8-bit paged K/V cache: writing rows into it, reading them back,
attention over it (with the weight every key received), and eviction by accumulated weight.

The cache holds e4m3 codes ``[layer][K|V][page][KV head][row of the page][head_dim]`` and one float32 scale, a
power of two, for each block (a page's rows of one KV head, in one layer's K or V).  Logical row j of a sequence
is row j % P of page ``table[j // P]``.  Sequence lengths, block tables and row offsets are device arrays.

  write      new rows become the last rows of their sequences.  Scale of a block: 0 when every value is 0, else the
             smallest power of two s with max|x| <= 448 s; a block that already holds rows of the sequence keeps the
             larger of its old scale and the new rows' one, and its old codes are rounded to it.  code = e4m3(x / s).
  read       the last rows of their sequences as code * scale.
  attention  query row i of a sequence's n sees rows 0 .. len - n + i: softmax(q k / sqrt(head_dim)) v over those,
             query heads sharing a KV head in groups; a row that sees nothing gives 0.  The weight of a key is the
             sum of its softmax weights over the call's query rows and the group's heads.
  evict      each KV head of each layer keeps its first rows, its last rows, and of the others those with the
             largest accumulated weight (ties to the lower row); the kept rows, in order, fill the destination
             pages as a write of their values would, and their weights move along (0 behind them).
"""
import numpy as np
import torch

own = False

SUPPORTED_PAGES = (16, 32, 64, 128, 256)


# --------------------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------------------
def _case(op, *, layers=1, heads=32, kv_heads=8, head_dim=128, dtype="bf16", page=64, seqs=1, length=8192, ragged=False,
          rows=1, weights=False, keep=0, sink=0, recent=0, name=None):
    c = dict(op=op, layers=layers, heads=heads, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, page=page, seqs=seqs,
             length=length, ragged=ragged, rows=rows, weights=weights, keep=keep, sink=sink, recent=recent)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a blended request (8K context and its query, 32 layers of the 8B shape) goes into the 8-bit pool
        _case("write", layers=32, length=8256, rows=8256, name="write blended 8k"),
        # one decoding step of a batch: each sequence's new token joins its last page, in one layer
        _case("write", seqs=64, length=8256, ragged=True, rows=1, name="write append 64"),
        # the cached context comes back as rows for the next blend
        _case("read", layers=32, length=8192, rows=8192, name="read context 8k"),
        # the same of a small fp32 model, with a length that ends inside a page
        _case("read", layers=5, heads=4, kv_heads=2, head_dim=64, dtype="f32", page=16, length=197, rows=197, name="read small f32"),
        # the first decoded token after a short prompt: latency
        _case("attention", length=200, name="decode 1 x 200"),
        # one decoding step of a server's batch, every length its own
        _case("attention", seqs=64, length=8256, ragged=True, name="decode 64 x 8k"),
        # one request with a very long context in small pages
        _case("attention", length=131071, page=16, name="decode 1 x 128k"),
        # the query's 64 rows over the blended context: the window whose weights choose what to evict
        _case("attention", length=8256, rows=64, weights=True, name="query 64 x 8k weights"),
        # a decoding step that keeps the keys' weights
        _case("attention", seqs=16, length=4096, ragged=True, weights=True, page=32, name="decode 16 x 4k weights"),
        # a few speculated tokens of a small fp32 model (head_dim 64)
        _case("attention", heads=16, kv_heads=4, head_dim=64, dtype="f32", seqs=8, length=2080, ragged=True, rows=5, page=32,
              name="verify 8 x 5 x 2k f32"),
        # the whole cache of a blended request shrinks to a quarter
        _case("evict", layers=32, length=8256, keep=2048, sink=4, recent=64, name="evict 8k to 2k"),
        # a small model's batch, lengths on both sides of what is kept
        _case("evict", layers=2, heads=16, kv_heads=4, head_dim=64, seqs=5, length=700, ragged=True, page=16, keep=200, sink=4, recent=33, name="evict 5 x 700"),
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
        op = rng.choice(["write", "read", "attention", "attention", "attention", "evict"])
        head_dim = rng.choice([64, 128, 128])
        kv_heads = rng.choice([1, 2, 4, 8, 8])
        group = rng.choice([1, 2, 3, 4, 4, 7, 8])
        page = rng.choice(SUPPORTED_PAGES)
        c = _case(op, heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, page=page)
        c["ragged"] = rng.random() < 0.7
        c["seqs"] = _log_int(rng, 1, 64)
        c["length"] = _log_int(rng, 17, 131071 if op == "attention" else 16384)
        if op == "attention":
            c["rows"] = rng.choice([1, 1, 1, 2, 5, _log_int(rng, 1, 64)])
            c["weights"] = rng.random() < 0.3
            c["dtype"] = rng.choice(["bf16", "bf16", "bf16", "f32"])
        else:
            c["layers"] = _log_int(rng, 1, 32)
            c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
            if op == "evict":
                c["dtype"] = "bf16"
                c["keep"] = _log_int(rng, 16, max(17, c["length"]))
                c["sink"] = min(4, c["keep"])
                c["recent"] = rng.randint(0, c["keep"] - c["sink"])
            else:
                c["rows"] = rng.choice([1, rng.randint(1, c["length"]), c["length"]])
        c["rows"] = min(c["rows"], c["length"])
        w = work(c)
        pool = c["layers"] * c["seqs"] * c["length"] * kv_heads * head_dim * 2
        if all(w[k] <= largest[op, k] for k in w) and pool <= 2 * 10 ** 9:
            return c


def _lengths(case):
    """Row count of each sequence: `length`, or ragged ones up to it (the first is the longest), from the case alone."""
    n, top = case["seqs"], case["length"]
    if not case["ragged"] or n == 1:
        return [top] * n
    r = np.random.RandomState(n * 7919 + top)
    lo = max(case["rows"] if case["op"] in ("write", "read") else 1, top // 16)
    return [top] + [int(v) for v in r.randint(lo, top + 1, n - 1)]


def work(case):
    lens, rows, L = _lengths(case), case["rows"], case["layers"]
    hkv, hd, es = case["kv_heads"], case["head_dim"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("write", "read"):
        n = rows * case["seqs"]
        blocks = sum(-(-l // case["page"]) - (l - rows) // case["page"] for l in lens)
        return {"bytes": 2.0 * L * hkv * (n * hd * (es + 1) + blocks * 4), "flops": 2.0 * L * hkv * n * hd}
    if case["op"] == "attention":
        keys = sum(lens)
        blocks = sum(-(-l // case["page"]) for l in lens)
        seen = sum(max(0, l - rows + i + 1) for l in lens for i in range(rows))
        out = case["seqs"] * rows * case["heads"] * hd * es
        return {"bytes": 2.0 * hkv * (keys * hd + blocks * 4) + 2.0 * out + (4.0 * hkv * keys if case["weights"] else 0.0),
                "flops": 4.0 * hd * case["heads"] * seen}
    kept = sum(min(l, case["keep"]) for l in lens)
    return {"bytes": float(L) * hkv * (4 * sum(lens) + 4 * sum(lens) + 4 * kept + 2 * 2 * kept * hd),
            "flops": float(L) * hkv * sum(lens)}


# --------------------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------------------
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _rows(case, g, n, gain):
    """K or V rows [layers][n][KV heads][head_dim]: normal values, a few channels of each head much larger (as keys have
    them) and a slow drift of the size along the rows, so that neighbouring blocks get other scales."""
    shape = (n, case["kv_heads"], case["head_dim"])
    drift = torch.exp2(2.0 * torch.sin(torch.arange(n, device="cuda", dtype=torch.float32) / 173.0))[:, None, None]
    out = torch.empty((case["layers"],) + shape, dtype=_dtype(case), device="cuda")
    for l in range(case["layers"]):
        out[l] = (torch.randn(shape, generator=g, device="cuda") * gain * drift).to(out.dtype)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    cpu = torch.Generator()
    cpu.manual_seed(int(seed) * 999983 + 5)
    L, B, P, hkv, hd, hq = case["layers"], case["seqs"], case["page"], case["kv_heads"], case["head_dim"], case["heads"]
    lens = _lengths(case)
    width = -(-max(lens) // P)
    used = [-(-l // P) for l in lens]
    more = [-(-min(l, case["keep"]) // P) for l in lens] if case["op"] == "evict" else [0] * B
    n_pages = sum(used) + sum(more) + 3
    order = torch.randperm(n_pages, generator=cpu, dtype=torch.int64).to(torch.int32)
    table = torch.zeros((B, width), dtype=torch.int32)
    dst = torch.zeros((B, max(more + [1])), dtype=torch.int32)
    at = 0
    for s in range(B):
        table[s, :used[s]] = order[at:at + used[s]]
        at += used[s]
    for s in range(B):
        dst[s, :more[s]] = order[at:at + more[s]]
        at += more[s]
    gain = torch.ones((hkv, hd), device="cuda")
    gain[:, torch.randperm(hd, generator=cpu)[:4].cuda()] = 6.0
    # the pool as it stands: every block quantised from normal values, its size drifting from page to page
    codes = torch.empty((L, 2, n_pages, hkv, P, hd), dtype=torch.uint8, device="cuda")
    scales = torch.empty((L, 2, n_pages, hkv), dtype=torch.float32, device="cuda")
    for l in range(L):
        for kv in range(2):
            drift = torch.exp2(torch.randn((n_pages, 1, 1, 1), generator=g, device="cuda") * 0.7)
            x = torch.randn((n_pages, hkv, P, hd), generator=g, device="cuda") * drift
            if kv == 0:
                x *= gain[None, :, None, :]
            top = x.abs().amax(dim=(2, 3))
            s = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
            scales[l, kv] = s
            codes[l, kv] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            del x
    state = dict(case=case, codes=codes, scales=scales, table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                 max_len=max(lens))
    n = B * case["rows"]
    if case["op"] == "write":
        state["k"] = _rows(case, g, n, gain)
        state["v"] = _rows(case, g, n, 1.0)
    elif case["op"] == "read":
        state["k"] = torch.empty((L, n, hkv, hd), dtype=_dtype(case), device="cuda")
        state["v"] = torch.empty_like(state["k"])
    elif case["op"] == "attention":
        state["q"] = torch.randn((n, hq, hd), generator=g, device="cuda").to(_dtype(case))
        state["out"] = torch.zeros((n, hq, hd), dtype=_dtype(case), device="cuda")
        if case["weights"]:
            state["w"] = torch.zeros((B, hkv, max(lens)), dtype=torch.float32, device="cuda")
    else:
        state["dst"] = dst.cuda()
        state["w"] = torch.exp(2.0 * torch.randn((L, B, hkv, max(lens)), generator=g, device="cuda"))
        state["w_out"] = torch.zeros_like(state["w"])
        state["kept"] = torch.full((L, B, hkv, case["keep"]), -1, dtype=torch.int32, device="cuda")
        state["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if own:
        import cacheblend_selective_kv_gb300 as cb
        cells = n * hq * (-(-max(lens) // 128) * 128 + 1) if case["weights"] else 0
        state["cache"] = cb.KV8Cache(codes, scales, n_heads=hq, dtype=case["dtype"], weight_cells=cells)
    return state


# --------------------------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------------------------
def run(state):
    return {"write": _write, "read": _read, "attention": _attention, "evict": _evict}[state["case"]["op"]](state)


def _pool(state):
    return {"codes": state["codes"].view(torch.float8_e4m3fn), "scales": state["scales"]}


def _scale_of(top):
    """The smallest power of two s with top <= 448 s (0 for 0): 448 = 0.875 * 2^9."""
    m, e = torch.frexp(top)
    s = torch.ldexp(torch.ones_like(top), torch.clamp(e - 9 + (m > 0.875).to(e.dtype), min=-126))
    return torch.where(top > 0, s, torch.zeros_like(s))


def _to_codes(x, s):
    return torch.where(s > 0, x / torch.where(s > 0, s, 1.0), torch.zeros_like(x)).to(torch.float8_e4m3fn)


def _write(state):
    case, codes, scales = state["case"], state["codes"], state["scales"]
    if own:
        state["cache"].write(state["table"], state["lens"], state["k"], state["v"], n_layers=case["layers"], max_len=state["max_len"])
        return _pool(state)
    L, B, P, rows, hkv, hd = case["layers"], case["seqs"], case["page"], case["rows"], case["kv_heads"], case["head_dim"]
    lens = state["lens"].long()
    first = (lens - rows) // P                                         # first block of each sequence that gets a row
    n_blocks = (rows + P - 2) // P + 1
    block = first[:, None] + torch.arange(n_blocks, device="cuda")     # [B][n]
    live = block * P < lens[:, None]
    page = state["table"].long().gather(1, torch.where(live, block, torch.zeros_like(block)))
    j = block[:, :, None] * P + torch.arange(P, device="cuda")         # logical row of each row of those blocks
    fresh = (j >= (lens - rows)[:, None, None]) & (j < lens[:, None, None]) & live[:, :, None]
    old = (j < (lens - rows)[:, None, None]) & live[:, :, None]
    src = torch.where(fresh, j - (lens - rows)[:, None, None] + (torch.arange(B, device="cuda") * rows)[:, None, None], torch.zeros_like(j))
    f = fresh[..., None, None]
    pages = page[live]
    for l in range(L):
        for kv, x in ((0, state["k"][l]), (1, state["v"][l])):
            x = torch.where(f, x[src].float(), 0.0)                    # [B][n][P][heads][dim]
            s = _scale_of(x.abs().amax(dim=(2, 4)))                    # [B][n][heads]
            was = torch.where(old.any(2)[..., None], scales[l, kv][page], 0.0)
            s = torch.maximum(s, was)
            before = codes[l, kv][page].transpose(2, 3)
            kept = before.view(torch.float8_e4m3fn).float() * was[:, :, None, :, None]
            held = torch.where(old[..., None, None], kept, x)
            c = _to_codes(held, s[:, :, None, :, None]).view(torch.uint8)
            c = torch.where(f | old[..., None, None], c, before)
            codes[l, kv][pages] = c.transpose(2, 3)[live]
            scales[l, kv][pages] = s[live]
    return _pool(state)


def _values(state, l, kv, page, row):
    """Rows of the pool as the float32 values they stand for: page and row [...] -> [...][KV heads][head_dim]."""
    c = state["codes"][l, kv].transpose(1, 2)[page, row]
    return c.view(torch.float8_e4m3fn).float() * state["scales"][l, kv][page][..., None]


def _read(state):
    case = state["case"]
    if own:
        state["cache"].read(state["table"], state["lens"], state["k"], state["v"], n_layers=case["layers"], max_len=state["max_len"])
        return {"k": state["k"], "v": state["v"]}
    rows, P = case["rows"], case["page"]
    j = (state["lens"].long() - rows)[:, None] + torch.arange(rows, device="cuda")
    page = state["table"].long().gather(1, j // P).reshape(-1)
    row = (j % P).reshape(-1)
    for l in range(case["layers"]):
        state["k"][l] = _values(state, l, 0, page, row).to(state["k"].dtype)
        state["v"][l] = _values(state, l, 1, page, row).to(state["v"].dtype)
    return {"k": state["k"], "v": state["v"]}


def _attention(state):
    case = state["case"]
    if own:
        state["cache"].attention(state["table"], state["lens"], state["q"], state["out"], max_len=state["max_len"], weights=state.get("w"))
        return {"out": state["out"], **({"weights": state["w"]} if case["weights"] else {})}
    B, P, rows, hkv, hd, top = case["seqs"], case["page"], case["rows"], case["kv_heads"], case["head_dim"], state["max_len"]
    G = case["heads"] // hkv
    lens = state["lens"].long()
    j = torch.arange(top, device="cuda")
    valid = j < lens[:, None]                                                    # [B][keys]
    page = torch.where(valid, state["table"].long().gather(1, (j // P).expand(B, top)), 0)
    k = _values(state, 0, 0, page, (j % P).expand(B, top)).transpose(1, 2)       # [B][heads][keys][dim]
    q = state["q"].float().view(B, rows, hkv, G, hd).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * rows, hd)
    s = torch.matmul(q, k.transpose(2, 3)) / hd ** 0.5
    del k
    i = torch.arange(rows, device="cuda")
    sees = (j <= (lens - rows)[:, None, None] + i[:, None]).repeat(1, G, 1)[:, None]    # [B][1][G rows][keys]
    s = torch.where(sees, s, -torch.inf)
    m = s.amax(dim=3, keepdim=True)
    e = torch.where(sees, torch.exp(s - torch.where(m > -torch.inf, m, 0.0)), 0.0)
    del s
    total = e.sum(dim=3, keepdim=True)
    p = torch.where(total > 0, e / total, 0.0)
    del e
    v = torch.where(valid[:, None, :, None], _values(state, 0, 1, page, (j % P).expand(B, top)).transpose(1, 2), 0.0)
    o = torch.matmul(p, v).view(B, hkv, G, rows, hd).permute(0, 3, 1, 2, 4).reshape(B * rows, hkv * G, hd)
    state["out"].copy_(o.to(state["out"].dtype))
    if not case["weights"]:
        return {"out": state["out"]}
    state["w"].copy_(torch.where(valid[:, None], p.sum(dim=2), state["w"]))
    return {"out": state["out"], "weights": state["w"]}


def _evict(state):
    case, codes, scales = state["case"], state["codes"], state["scales"]
    if own:
        state["cache"].evict(state["table"], state["lens"], state["dst"], state["w"], case["keep"], n_sink=case["sink"],
                             n_recent=case["recent"], out_rows=state["kept"], out_lens=state["new_lens"],
                             out_weights=state["w_out"], n_layers=case["layers"], max_len=state["max_len"])
        return {**_pool(state), "weights": state["w_out"], "rows": state["kept"], "lens": state["new_lens"]}
    L, B, P, hkv, hd, keep = case["layers"], case["seqs"], case["page"], case["kv_heads"], case["head_dim"], case["keep"]
    top = state["max_len"]
    lens = state["lens"].long()
    j = torch.arange(top, device="cuda")
    n = torch.clamp(lens, max=keep)                                              # rows kept of each sequence
    state["new_lens"].copy_(n)
    valid = j < lens[:, None]
    always = valid & ((j < case["sink"]) | (j >= (lens - case["recent"])[:, None]))     # [B][rows]
    w = state["w"]
    rank = torch.where(w > 0, w, 0.0)
    rank = torch.where(always[:, None], torch.inf, torch.where(valid[:, None], rank, -1.0))
    by_rank = torch.sort(rank, dim=3, descending=True, stable=True).indices
    width = min(keep, top)
    slot = torch.arange(width, device="cuda")
    live = (slot < n[:, None])[:, None]                                          # [B][1][slots]
    kept = torch.where(live, by_rank[..., :width], top).sort(dim=3).values       # [L][B][heads][slots], ascending
    at = torch.where(live, kept, 0)
    state["kept"].fill_(-1)
    state["kept"][..., :width] = torch.where(live, kept, -1).to(torch.int32)
    new_w = torch.where(live, w.gather(3, at), 0.0)
    state["w_out"][..., :width] = torch.where(valid[:, None, :width], new_w, state["w_out"][..., :width])
    state["w_out"][..., width:] = torch.where(valid[:, None, width:], 0.0, state["w_out"][..., width:])
    blocks = -(-width // P)
    pad = blocks * P - width
    live_b = torch.nn.functional.pad(live.expand(B, 1, width), (0, pad)).view(B, 1, blocks, P)
    full = torch.arange(blocks, device="cuda") * P < n[:, None]                  # [B][blocks] a block that gets a row
    pages = state["dst"].long()[:, :blocks][full]
    heads = torch.arange(hkv, device="cuda")[None, :, None]
    for l in range(L):
        page = state["table"].long()[:, None].expand(B, hkv, -1).gather(2, at[l] // P)
        for kv in range(2):
            x = codes[l, kv][page, heads, at[l] % P].view(torch.float8_e4m3fn).float() * scales[l, kv][page, heads][..., None]
            x = torch.nn.functional.pad(torch.where(live[..., None], x, 0.0), (0, 0, 0, pad)).view(B, hkv, blocks, P, hd)
            s = _scale_of(x.abs().amax(dim=(3, 4)))                              # [B][heads][blocks]
            c = _to_codes(x, s[..., None, None]).view(torch.uint8).permute(0, 2, 1, 3, 4)
            before = codes[l, kv][state["dst"].long()[:, :blocks]]
            c = torch.where(live_b.permute(0, 2, 1, 3)[..., None], c, before)
            codes[l, kv][pages] = c[full]
            scales[l, kv][pages] = s.transpose(1, 2)[full]
    return {**_pool(state), "weights": state["w_out"], "rows": state["kept"], "lens": state["new_lens"]}


# --------------------------------------------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence
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


def _block(rows):
    """(codes, scales) of blocks [...][rows][dim] of float64 values, a scale for each."""
    s = _pow2_at_least(rows.abs().amax(dim=(-2, -1)))
    return _grid(rows / torch.where(s > 0, s, 1.0)[..., None, None]), s


def _numbers(state):
    """The pool's codes as float64 numbers, through a table of the 256 codes."""
    i = torch.arange(256, dtype=torch.float64)
    sign, e, m = torch.where(i >= 128, -1.0, 1.0), (i % 128) // 8, i % 8
    t = sign * torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
    t[127] = t[255] = float("nan")
    t = t.cuda()
    return lambda c: t[c.long()]


def exact(case, seed):
    state = prepare(case, seed)
    number = _numbers(state)
    P, hkv, hd, rows = case["page"], case["kv_heads"], case["head_dim"], case["rows"]
    lens, table = _lengths(case), state["table"].tolist()
    codes, scales = state["codes"], state["scales"]

    def whole(l, kv, s, lo, hi):
        """Rows lo..hi-1 of sequence s as [rows][heads][dim]; lo is a multiple of P."""
        pg = torch.tensor(table[s][lo // P:-(-hi // P)], device="cuda")
        x = number(codes[l, kv][pg]) * scales[l, kv][pg].double()[..., None, None]
        return x.transpose(1, 2).reshape(-1, hkv, hd)[:hi - lo]

    if case["op"] == "read":
        out = [torch.empty(state["k"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
        for l in range(case["layers"]):
            for kv in range(2):
                for s, n in enumerate(lens):
                    lo = (n - rows) // P * P
                    out[kv][l, s * rows:(s + 1) * rows] = whole(l, kv, s, lo, n)[n - rows - lo:]
        return {"k": out[0], "v": out[1]}
    if case["op"] == "write":
        new_codes = torch.empty(codes.shape, dtype=torch.float64, device="cuda")
        new_scales = scales.double()
        for l in range(case["layers"]):
            for kv, x in ((0, state["k"]), (1, state["v"])):
                new_codes[l, kv] = number(codes[l, kv])
                for s, n in enumerate(lens):
                    lo = (n - rows) // P * P
                    have = n - rows - lo                                   # rows of the first block that stay
                    x_s = x[l, s * rows:(s + 1) * rows].double()
                    pg = torch.tensor(table[s][lo // P:-(-n // P)], device="cuda")
                    b = torch.zeros((len(pg) * P, hkv, hd), dtype=torch.float64, device="cuda")
                    b[have:have + rows] = x_s
                    b = b.view(len(pg), P, hkv, hd).transpose(1, 2)
                    sc = _pow2_at_least(b.abs().amax(dim=(2, 3)))
                    if have:
                        was = scales[l, kv][pg[0]].double()
                        sc[0] = torch.maximum(sc[0], was)
                        b[0, :, :have] = number(codes[l, kv][pg[0]])[:, :have] * was[:, None, None]
                    c = _grid(b / torch.where(sc > 0, sc, 1.0)[..., None, None])
                    c = c.transpose(1, 2).reshape(-1, hkv, hd)
                    kept = new_codes[l, kv][pg].transpose(1, 2).reshape(-1, hkv, hd)
                    kept[:have + rows] = c[:have + rows]
                    new_codes[l, kv][pg] = kept.view(len(pg), P, hkv, hd).transpose(1, 2)
                    new_scales[l, kv][pg] = sc
        return {"codes": new_codes, "scales": new_scales}
    if case["op"] == "attention":
        G = case["heads"] // hkv
        out = torch.zeros(state["out"].shape, dtype=torch.float64, device="cuda")
        weights = torch.zeros((case["seqs"], hkv, max(lens)), dtype=torch.float64, device="cuda")
        for s, n in enumerate(lens):
            k, v = whole(0, 0, s, 0, n), whole(0, 1, s, 0, n)
            q = state["q"][s * rows:(s + 1) * rows].double()
            pos = n - rows + torch.arange(rows, device="cuda")
            seen = torch.arange(n, device="cuda")[None] <= pos[:, None]
            for h in range(case["heads"]):
                x = (q[:, h] @ k[:, h // G].T) * hd ** -0.5
                x = torch.where(seen, x, torch.full_like(x, -torch.inf))
                p = torch.where((pos >= 0)[:, None], torch.softmax(x, dim=1), 0.0)
                out[s * rows:(s + 1) * rows, h] = p @ v[:, h // G]
                weights[s, h // G, :n] += p.sum(dim=0)
        return {"out": out, **({"weights": weights} if case["weights"] else {})}
    # evict
    keep, L = case["keep"], case["layers"]
    dst = state["dst"].tolist()
    new_codes = torch.empty(codes.shape, dtype=torch.float64, device="cuda")
    for l in range(L):
        for kv in range(2):
            new_codes[l, kv] = number(codes[l, kv])
    new_scales, new_w = scales.double(), torch.zeros_like(state["w"], dtype=torch.float64)
    for l in range(L):
        for s, n in enumerate(lens):
            m = min(n, keep)
            w = state["w"][l, s, :, :n].double()
            order = w.clone()
            order[:, :case["sink"]] = torch.inf
            order[:, max(0, n - case["recent"]):] = torch.inf
            idx = torch.argsort(order, dim=1, descending=True, stable=True)[:, :m].sort(dim=1).values
            new_w[l, s, :, :m] = w.gather(1, idx)
            pg = torch.tensor(dst[s][:-(-m // P)], device="cuda")
            for kv in range(2):
                x = whole(l, kv, s, 0, n).transpose(0, 1).gather(1, idx[..., None].expand(-1, -1, hd))   # [heads][m][dim]
                b = torch.zeros((hkv, len(pg) * P, hd), dtype=torch.float64, device="cuda")
                b[:, :m] = x
                c, sc = _block(b.view(hkv, len(pg), P, hd))
                was = new_codes[l, kv][pg].transpose(0, 1).reshape(hkv, -1, hd)
                was[:, :m] = c.reshape(hkv, -1, hd)[:, :m]
                new_codes[l, kv][pg] = was.view(hkv, len(pg), P, hd).transpose(0, 1)
                new_scales[l, kv][pg] = sc.transpose(0, 1)
    return {"codes": new_codes, "scales": new_scales, "weights": new_w, "rows": None, "lens": None}
