"""Plain numpy / float64 model of the 8-bit paged K/V cache: what cb_kv8_write, read, attention and evict compute,
row by row, from their definition.  Shares no code with the library."""
import numpy as np

F8_MAX = 448.0


def code_values():
    """The value of each of the 256 e4m3 codes."""
    out = np.zeros(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        out[c] = -v if s else v
    out[0x7F] = out[0xFF] = np.nan
    return out


VALUES = code_values()
_POS = VALUES[:127]                       # ascending, codes 0 .. 126


def encode(x):
    """float64 array -> e4m3 codes, to nearest, ties to the even code; NaN -> 0x7F; |x| above 448 -> 448."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), F8_MAX)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    up, dn = _POS[hi] - a, a - _POS[lo]
    c = np.where((up < dn) | ((up == dn) & (hi % 2 == 0)), hi, lo)
    c = np.where(np.signbit(x), c + 128, c)
    return np.where(np.isnan(x), 0x7F, c).astype(np.uint8)


def scale_of(x):
    """Scale of a block of values: by trying powers of two."""
    fin = np.abs(x[np.isfinite(x)])
    top = float(fin.max()) if fin.size else 0.0
    if top == 0.0:
        return 0.0
    e = -126
    while top > F8_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def divide(x, s):
    """x / s for the encoder: infinities become NaN; a block of zeros has s = 0."""
    x = np.where(np.isfinite(x), x, np.nan)
    return x / s if s else x * 0.0


class Model:
    """codes [L][2][n_pages][Hkv][P][hd] uint8 and scales [L][2][n_pages][Hkv] (float64), modified in place."""

    def __init__(self, codes, scales):
        self.codes, self.scales = codes.copy(), scales.astype(np.float64)
        self.L, _, self.n_pages, self.H, self.P, self.hd = codes.shape

    def write(self, table, lens, k, v, starts, layer=0):
        """k, v [layers][rows][H][hd] float64."""
        P = self.P
        for s, n in enumerate(lens):
            r0, r1 = starts[s], starts[s + 1]
            first = n - (r1 - r0)
            for b in range(first // P, -(-n // P)) if r1 > r0 else ():
                lo, hi = max(first - b * P, 0), min(n - b * P, P)
                pg = table[s][b]
                for l in range(k.shape[0]):
                    for kv, src in ((0, k), (1, v)):
                        for h in range(self.H):
                            x = src[l, r0 + b * P + lo - first:r0 + b * P + hi - first, h]
                            sc, was = scale_of(x), self.scales[layer + l, kv, pg, h]
                            blk = self.codes[layer + l, kv, pg, h]
                            if lo > 0:
                                if was >= sc:
                                    sc = was
                                elif was > 0:
                                    blk[:lo] = encode(VALUES[blk[:lo]] * was / sc)
                            blk[lo:hi] = encode(divide(x, sc))
                            self.scales[layer + l, kv, pg, h] = sc

    def rows(self, table_row, n, layer):
        """(K, V) of a sequence's first n rows, float64 [n][H][hd]."""
        out = []
        for kv in range(2):
            x = np.zeros((n, self.H, self.hd))
            for b in range(-(-n // self.P)):
                pg = table_row[b]
                blk = VALUES[self.codes[layer, kv, pg]] * self.scales[layer, kv, pg][:, None, None]
                m = min(self.P, n - b * self.P)
                x[b * self.P:b * self.P + m] = blk[:, :m].transpose(1, 0, 2)
            out.append(x)
        return out

    def attention(self, table, lens, q, starts, layer, scale):
        """out [n_q][Hq][hd], weights list of [H][len] per sequence, and for error bounds: spread, sum p|v|
        [n_q][Hq][hd]; the largest sum |q k| scale of any row and key; self.floor [n_q][Hq][hd], the sum over tiles of
        128 keys of (largest p * scale of V in the tile) * (sum of |codes of V|); self.floor_all, the same with all keys
        as one tile."""
        out, spread = np.zeros(q.shape), np.zeros(q.shape)
        self.floor, self.floor_all = np.zeros(q.shape), np.zeros(q.shape)
        ws, big = [], 0.0
        G = q.shape[1] // self.H
        for s, n in enumerate(lens):
            k, v = self.rows(table[s], n, layer)
            sv = np.zeros((n, self.H))
            for b in range(-(-n // self.P)):
                sv[b * self.P:(b + 1) * self.P] = self.scales[layer, 1, table[s][b]]
            w = np.zeros((self.H, n))
            r0, r1 = starts[s], starts[s + 1]
            for i in range(r0, r1):
                seen = n - (r1 - r0) + (i - r0) + 1
                if seen <= 0:
                    continue
                for h in range(q.shape[1]):
                    kk, vv = k[:seen, h // G], v[:seen, h // G]
                    x = kk @ q[i, h] * scale
                    mag = np.abs(kk) @ np.abs(q[i, h]) * abs(scale)
                    big = max(big, float(np.nanmax(mag)))
                    p = np.exp(x - x.max())
                    p /= p.sum()
                    out[i, h] = p @ vv
                    spread[i, h] = p @ np.abs(vv)
                    w[h // G, :seen] += p
                    ss = sv[:seen, h // G]
                    code = np.abs(vv) / np.where(ss > 0, ss, 1.0)[:, None]
                    self.floor_all[i, h] = (p * ss).max() * code.sum(axis=0)
                    for t in range(0, seen, 128):
                        self.floor[i, h] += (p * ss)[t:t + 128].max() * code[t:t + 128].sum(axis=0)
            ws.append(w)
        return out, ws, spread, big

    def evict(self, table, lens, dst, weights, keep, sink, recent, layer=0):
        """weights [layers][n][H][ld]; returns (rows, new_lens, new_weights) and moves the rows into dst's pages."""
        nl = weights.shape[0]
        rows = np.full((nl, len(lens), self.H, keep), -1, np.int32)
        new_w = weights.copy()
        before = Model(self.codes, self.scales)
        new_lens = [min(n, keep) for n in lens]
        for l in range(nl):
            for s, n in enumerate(lens):
                m = new_lens[s]
                k, v = before.rows(table[s], n, layer + l)
                for h in range(self.H):
                    w = weights[l, s, h, :n]
                    if n <= keep:
                        idx = list(range(n))
                    else:
                        must = set(range(sink)) | set(range(n - recent, n))
                        rest = [j for j in range(n) if j not in must]
                        rest.sort(key=lambda j: (-(w[j] if w[j] > 0 else 0.0), j))
                        idx = sorted(must | set(rest[:keep - len(must)]))
                    rows[l, s, h, :m] = idx
                    new_w[l, s, h, :m] = w[idx]
                    new_w[l, s, h, m:n] = 0
                    for kv, x in ((0, k), (1, v)):
                        for b in range(-(-m // self.P)):
                            part = x[idx[b * self.P:(b + 1) * self.P], h]
                            sc = scale_of(part)
                            pg = dst[s][b]
                            self.codes[layer + l, kv, pg, h, :len(part)] = encode(divide(part, sc))
                            self.scales[layer + l, kv, pg, h] = sc
        return rows, new_lens, new_w
