"""GPU test of the operators of a decoding step as a program runs them: requests on one blended context, each step new rows
rotated and appended, attention over the shared context and the request's own rows, logits, the next token; eviction in
between, after which positions run on; the step captured into a graph.  Every stage is compared with float64 from the
stage's own inputs (the tolerances are those of the stages' own tests)."""
import numpy as np
import pytest

import kv8_model as km
from test_gpu_kv8 import Case, f64, i32
from test_gpu_kv8_append import EPS, check_k, check_q, rotate
from test_gpu_sample import exact as exact_token

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


@pytest.mark.parametrize("B", [3, 11])
def test_decode_on_a_shared_context(cb, B):
    H, G, hd, P, V, theta, top = 2, 4, 64, 16, 700, 1e4, 64
    context = 150
    cells = max(cb.KV8Cache.shared_cells(B, H * G, hd), cb.KV8Cache.cells(B, H * G, top))
    c = Case(cb, [context] + [0] * B, H=H, G=G, hd=hd, P=P, seed=B, cells=cells)
    width = -(-top // P)
    rng = np.random.default_rng(B)
    own = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    # the requests' pages: of those that the context does not take
    free = [p for p in range(c.model.n_pages) if p not in set(c.table_np[0][:-(-context // P)].tolist())]
    assert len(free) >= B * width
    own_np = np.array(rng.permutation(free)[:B * width], np.int32).reshape(B, width)
    own.copy_(i32(own_np))
    pre, pre_lens = c.table[:1].contiguous(), i32([context])
    lens, pos = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), context, dtype=torch.int32, device="cuda")
    d = 96
    hidden = torch.zeros((B, d), dtype=torch.bfloat16, device="cuda")
    w_qkv = torch.from_numpy((rng.normal(size=((H * G + 2 * H) * hd, d)) * 0.3).astype(np.float32)).cuda().bfloat16()
    w_out = torch.from_numpy((rng.normal(size=(V, H * G * hd)) * 0.1).astype(np.float32)).cuda().bfloat16()
    qkv = torch.zeros((B, (H * G + 2 * H) * hd), dtype=torch.bfloat16, device="cuda")
    q, k, v = (t.view(B, -1, hd) for t in qkv.split([H * G * hd, H * hd, H * hd], dim=1))
    out, q_rot = torch.zeros((B, H * G, hd), dtype=torch.bfloat16, device="cuda"), torch.zeros((B, H * G, hd), dtype=torch.bfloat16, device="cuda")
    weights = torch.zeros((1, B, H, top), device="cuda")
    logits = torch.zeros((B, V), device="cuda")
    u, t = torch.zeros(B, device="cuda"), torch.full((B,), 0.8, device="cuda")
    top_k, top_p = torch.full((B,), 40, dtype=torch.int32, device="cuda"), torch.full((B,), 0.95, device="cuda")
    token, prob = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, device="cuda")

    def step():
        torch.mm(hidden, w_qkv.t(), out=qkv)
        c.cache.append(own, lens, q, k, v, theta, out_q=q_rot, positions=pos)
        c.cache.attention_shared(pre, pre_lens, own, lens, q_rot, out)
        c.cache.attention(own, lens, q_rot, weights=weights[0], add=True)          # what the requests' own keys receive, for eviction
        logits.copy_(torch.mm(out.view(B, -1), w_out.t()))
        cb.cb_sample(logits, u, temperature=t, top_k=top_k, top_p=top_p, out_tokens=token, out_probs=prob)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                          # no sequence has a length: nothing is stored
    side.synchronize()
    weights.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    weights.zero_()
    told = 0
    lens_np, pos_np = np.zeros(B, int), np.full(B, context - 1)
    for n in range(24):
        lens_np, pos_np = lens_np + 1, pos_np + 1
        if n >= 3:
            lens_np[1] = 0                              # a place of the batch that became free
        lens.copy_(i32(lens_np))
        pos.copy_(i32(pos_np))
        hidden.copy_(torch.from_numpy(rng.normal(size=(B, d)).astype(np.float32)))
        u.copy_(torch.from_numpy(rng.random(B).astype(np.float32)))
        c.model.codes[:], c.model.scales[:] = c.codes.cpu().numpy(), c.scales.cpu().numpy()
        graph.replay()
        torch.cuda.synchronize()
        st, live = list(range(B + 1)), [s for s in range(B) if lens_np[s]]
        qr, qs = rotate(f64(q), pos_np, theta)
        check_q(q_rot, qr, qs, EPS["bf16"], "bf16", untouched=[s for s in range(B) if not lens_np[s]])
        kr, ks = rotate(f64(k), pos_np, theta)
        rows = [0]
        for s in range(B):
            rows.append(rows[-1] + (lens_np[s] > 0))
        check_k(c, c.model, own_np, lens_np, kr[live], ks[live], rows, EPS["bf16"])
        now = km.Model(c.codes.cpu().numpy(), c.scales.cpu().numpy())
        kp, vp = now.rows(c.table_np[0], context, 0)
        for s in live:
            ko, vo = now.rows(own_np[s], lens_np[s], 0)
            kk, vv, qq = np.concatenate((kp, ko)), np.concatenate((vp, vo)), f64(q_rot)[s]
            for h in range(H * G):
                x = kk[:, h // G] @ qq[h] * hd ** -0.5
                p = np.exp(x - x.max())
                p /= p.sum()
                ref, spread = p @ vv[:, h // G], p @ np.abs(vv[:, h // G])
                assert (np.abs(f64(out)[s, h] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * spread).all()
        x = logits.cpu().numpy().astype(np.float64)
        for s in range(B):
            tok, pr, near = exact_token(x[s], float(u[s]), float(t[s]), 40, float(top_p[s]))
            if not near:
                told += 1
                assert int(token[s]) == tok and abs(float(prob[s]) - pr) <= 2.0 ** -22 * pr
        if n == 15:
            # requests keep 6 of their rows, in place; their positions run on
            c.cache.evict(own, lens, own, weights, n_keep=6, n_sink=1, n_recent=2, out_lens=lens)
            torch.cuda.synchronize()
            lens_np = np.minimum(lens_np, 6)
            assert lens.tolist() == lens_np.tolist()
    assert told >= 0.9 * 24 * B
    c.done()
