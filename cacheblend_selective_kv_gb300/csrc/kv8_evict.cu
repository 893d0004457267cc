// Eviction from the 8-bit paged K/V cache by accumulated attention weight.  Each KV head of each layer keeps its first
// `sink` rows, its last `recent` rows and, of the others, those with the largest weight (ties to the lower row; a
// weight that is not positive ranks as 0), `keep` rows in all; a sequence with at most `keep` rows keeps them all.
// The kept rows, in order, become rows 0 .. of the destination pages, quantised anew as a write of their values
// would be, and their weights move along.
//
//   select   one CTA per (layer, sequence, KV head): the weights' bits order as unsigned integers, so four rounds of a
//            256-bin histogram fix the threshold (and, when more rows equal it than are wanted, rounds over the row
//            numbers of those fix the last one taken); a warp then counts and writes the kept rows of its own stretch.
//   move     one CTA per (layer, K|V, KV head, sequence) and destination page; a page's rows are in registers before it is
//            written.  Destination row r comes from a row >= r, so with equal tables (in place) one CTA does a head's
//            pages in order and nothing is overwritten before it is read.
// The moved rows are most of the bytes: move is bound by HBM, at the latency of rows -> table -> codes, which many
// small CTAs (or, in place, the next page's addresses fetched ahead) cover.
#include <climits>

#include "cb_kv8.cuh"

namespace cb {

namespace {

constexpr int ST = 512;       // select threads
constexpr int MT = 128;       // move threads

struct EvictArgs {
    Kv8Seqs q;
    Kv8Evict e;
    uint8_t* codes;
    float* scales;
    int Hkv, hd, layer;
};

__device__ __forceinline__ unsigned rank_bits(float w) { return w > 0.f ? __float_as_uint(w) : 0u; }

// In a 256-bin histogram, the bin in which a running count from the top (or the bottom) reaches `want`, and how many of
// that bin are wanted.  Called by warp 0.
template <bool TOP> __device__ __forceinline__ void find_bin(const int* hist, int want, unsigned* pick) {
    const int lane = threadIdx.x & 31;
    int h[8], sum = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {                      // lane 0 holds the first bins in counting order
        const int i = lane * 8 + k;
        h[k] = hist[TOP ? 255 - i : i];
        sum += h[k];
    }
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
    }
    before -= sum;
    if (before < want && want <= before + sum) {
        int k = 0;
        while (before + h[k] < want) before += h[k++];
        pick[0] = (unsigned)(TOP ? 255 - (lane * 8 + k) : lane * 8 + k);
        pick[1] = (unsigned)(want - before);
    }
}

__global__ void __launch_bounds__(ST) kv8_select_kernel(const EvictArgs a) {
    __shared__ int hist[256];
    __shared__ int sm[ST / 32];
    __shared__ unsigned pick[2];                       // bin chosen, rows wanted of it
    grid_dep_launch();
    grid_dep_wait();
    const int g = blockIdx.x, s = blockIdx.y, l = blockIdx.z, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int len = kv8_len(a.q, s);
    if (len < 0 || len > a.q.max_len) {
        if (t == 0) atomicOr(a.q.status, ST_BAD_ROW);
        return;
    }
    const int64_t seg = ((int64_t)l * a.q.n + s) * a.Hkv + g;
    const float* w = a.e.weights + seg * a.e.weights_ld;
    float* ow = a.e.out_weights + seg * a.e.weights_ld;
    int* rows = a.e.out_rows + seg * a.e.keep;
    const int kept = min(len, a.e.keep);
    const int c0 = a.e.sink, c1 = len - a.e.recent;    // candidates [c0, c1)
    unsigned thr = 0;                                  // candidates with rank bits above it are kept ...
    int cut = -1;                                      // ... and those equal to it up to this row
    if (len > a.e.keep) {
        int want = a.e.keep - a.e.sink - a.e.recent;   // fewer than the candidates
        // rounds of eight bits: a row counts when its bits above `shift + 8` are `prefix`; ties by row number
        const auto round = [&](int shift, unsigned prefix, bool by_row) {
            for (int i = t; i < 256; i += ST) hist[i] = 0;
            __syncthreads();
            const unsigned mask = shift == 24 ? 0u : ~0u << (shift + 8);
#pragma unroll 4
            for (int j = c0 + t; j < c1; j += ST) {
                const unsigned b = rank_bits(w[j]), v = by_row ? (unsigned)j : b;
                if ((v & mask) == prefix && (!by_row || b == thr)) atomicAdd(&hist[(v >> shift) & 255u], 1);
            }
            __syncthreads();
            if (warp == 0) {
                if (by_row) find_bin<false>(hist, want, pick);
                else find_bin<true>(hist, want, pick);
            }
            __syncthreads();
            want = (int)pick[1];
            return prefix | (pick[0] << shift);
        };
        if (want > 0) {
            for (int shift = 24; shift >= 0; shift -= 8) thr = round(shift, thr, false);
            cut = INT_MAX;
            if (hist[thr & 255u] > want) {             // more rows equal the threshold than are wanted
                __syncthreads();
                unsigned last = 0;
                for (int shift = 24; shift >= 0; shift -= 8) last = round(shift, last, true);
                cut = (int)last;
            }
        } else {
            thr = ~0u;
        }
    }
    const auto keeps = [&](int j) {
        if (j >= len) return false;
        if (len <= a.e.keep || j < c0 || j >= c1) return true;
        const unsigned b = rank_bits(w[j]);
        return b > thr || (b == thr && j <= cut);
    };
    // a warp's stretch of rows: count what it keeps, then write it behind the stretches before
    const int per = (len + ST - 1) / ST * 32, j_lo = warp * per, j_hi = min(len, j_lo + per);
    int n = 0;
#pragma unroll 4
    for (int j = j_lo; j < j_hi; j += 32) n += __popc(__ballot_sync(0xffffffffu, keeps(j + lane)));
    if (lane == 0) sm[warp] = n;
    __syncthreads();
    int at = 0;
    for (int k = 0; k < warp; ++k) at += sm[k];
#pragma unroll 4
    for (int j = j_lo; j < j_hi; j += 32) {
        const bool k = keeps(j + lane);
        const unsigned who = __ballot_sync(0xffffffffu, k);
        if (k) rows[at + __popc(who & ((1u << lane) - 1))] = j + lane;
        at += __popc(who);
    }
    for (int j = kept + t; j < a.e.keep; j += ST) rows[j] = -1;
    __syncthreads();
    // the kept rows' weights; in place a weight moves down (rows[i] >= i), so a step reads before it writes
    constexpr int STEP = 4;
    for (int i0 = 0; i0 < kept; i0 += STEP * ST) {
        float v[STEP];
#pragma unroll
        for (int k = 0; k < STEP; ++k) {
            const int i = i0 + k * ST + t;
            v[k] = i < kept ? w[rows[i]] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < STEP; ++k) {
            const int i = i0 + k * ST + t;
            if (i < kept) ow[i] = v[k];
        }
    }
    __syncthreads();
    for (int j = kept + t; j < len; j += ST) ow[j] = 0.f;
}

// NP 16-byte vectors of codes per thread: a page of P rows is P * hd / 16 = tpb * NP vectors
template <int NP>
__global__ void __launch_bounds__(MT) kv8_move_kernel(const EvictArgs a, int tpb, int ranges) {
    __shared__ float sm[2][MT / 32];
    grid_dep_launch();
    grid_dep_wait();
    const int g = blockIdx.y % a.Hkv, lk = blockIdx.y / a.Hkv, s = blockIdx.z, t = threadIdx.x;
    const int l = lk >> 1, kv = lk & 1, P = 1 << a.q.shift, vpr_shift = a.hd == 128 ? 3 : 2;
    const int len = kv8_len(a.q, s);
    if (len < 0 || len > a.q.max_len) return;
    const int kept = min(len, a.e.keep), pages = (kept + P - 1) >> a.q.shift;
    // out_lens may be the lengths read above: a CTA that sees the new one finds the same `kept`
    if (blockIdx.x == 0 && blockIdx.y == 0 && t == 0) a.e.out_lens[s] = kept;
    const int64_t seg = ((int64_t)l * a.q.n + s) * a.Hkv + g;
    const int* rows = a.e.out_rows + seg * a.e.keep;
    const int64_t base = (int64_t)((a.layer + l) * 2 + kv) * a.q.n_pages;
    const int per = (pages + ranges - 1) / ranges, b_hi = min(pages, ((int)blockIdx.x + 1) * per);
    // source of vector t + i * tpb of page b: its pool row (page * P + row in page), or -1
    int64_t from[NP];
    const auto sources = [&](int b) {
        int j[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int row = b * P + ((t + i * tpb) >> vpr_shift);
            j[i] = t < tpb && b < b_hi && row < kept ? rows[row] : -1;
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int pg = j[i] >= 0 ? kv8_page(a.q, s, j[i] >> a.q.shift) : -1;
            from[i] = pg >= 0 ? ((int64_t)pg << a.q.shift) + (j[i] & (P - 1)) : -1;
        }
    };
    int b = blockIdx.x * per, flip = 0;
    sources(b);
    for (; b < b_hi; ++b, flip ^= 1) {
        uint4 x[NP];
        float sc[NP];
        const int n = min(P, kept - b * P);
        const int dst = a.e.dst_table[(int64_t)s * a.e.dst_ld + b];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            x[i] = make_uint4(0, 0, 0, 0);
            sc[i] = 0.f;
            if (from[i] >= 0) {
                const int64_t blk = (base + (from[i] >> a.q.shift)) * a.Hkv + g;
                x[i] = reinterpret_cast<const uint4*>(a.codes + (blk * P + (from[i] & (P - 1))) * a.hd)[(t + i * tpb) & ((1 << vpr_shift) - 1)];
                sc[i] = a.scales[blk];
            }
        }
        sources(b + 1);
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            // the largest code without its sign (a NaN code counts as 0), times the scale
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t c = w[k] & 0x7f7f7f7fu;
                c &= ~__vcmpeq4(c, 0x7f7f7f7fu);
                m = __vmaxu4(m, c);
            }
            m = __vmaxu4(m, m >> 16);
            m = __vmaxu4(m, m >> 8);
            top = fmaxf(top, kv8_value2(m & 0xffu).x * sc[i]);
        }
        top = warp_max(top);
        if ((t & 31) == 0) sm[flip][t >> 5] = top;
        __syncthreads();                               // also: every row of this page has been read
        for (int i = 0; i < MT / 32; ++i) top = fmaxf(top, sm[flip][i]);
        const float ns = kv8_scale(top), inv = kv8_inverse(ns);
        if (dst < 0 || dst >= a.q.n_pages) {
            if (t == 0) atomicOr(a.q.status, ST_BAD_ROW);
            continue;
        }
        const int64_t blk = (base + dst) * a.Hkv + g;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int v = t + i * tpb;
            if (t >= tpb || (v >> vpr_shift) >= n) continue;
            if (sc[i] != ns) {
                const float f = sc[i] * inv;
                x[i].x = kv8_rescale4(x[i].x, f);
                x[i].y = kv8_rescale4(x[i].y, f);
                x[i].z = kv8_rescale4(x[i].z, f);
                x[i].w = kv8_rescale4(x[i].w, f);
            }
            reinterpret_cast<uint4*>(a.codes + blk * P * a.hd)[v] = x[i];
        }
        if (t == 0) a.scales[blk] = ns;
    }
}

}  // namespace

cudaError_t launch_kv8_evict(const Kv8& c, const Kv8Seqs& q, const Kv8Evict& e, int layer, int n_layers, cudaStream_t s) {
    EvictArgs a{q, e, c.codes, c.scales, c.cfg.n_kv_heads, c.cfg.head_dim, layer};
    if (q.n == 0 || n_layers == 0) return cudaSuccess;
    const cudaError_t err = launch_ex(c.pdl, kv8_select_kernel, dim3(a.Hkv, q.n, n_layers), dim3(ST), 0, s, a);
    if (err != cudaSuccess) return err;
    const int P = 1 << q.shift, vecs = P * a.hd / 16;
    const int tpb = vecs < MT ? vecs : MT, np = vecs / tpb;             // 64 .. 2048 vectors
    const int pages = ((e.keep < q.max_len ? e.keep : q.max_len) + P - 1) / P;
    // in place the pages of a head are done in order by one CTA; between two tables each has its own
    const bool in_place = e.dst_table == q.table && e.dst_ld == q.table_ld;
    const int ranges = in_place || pages == 0 ? 1 : pages;
    const dim3 grid(ranges, 2 * n_layers * a.Hkv, q.n);
    switch (np) {
        case 1: return launch_ex(c.pdl, kv8_move_kernel<1>, grid, dim3(MT), 0, s, a, tpb, ranges);
        case 2: return launch_ex(c.pdl, kv8_move_kernel<2>, grid, dim3(MT), 0, s, a, tpb, ranges);
        case 4: return launch_ex(c.pdl, kv8_move_kernel<4>, grid, dim3(MT), 0, s, a, tpb, ranges);
        case 8: return launch_ex(c.pdl, kv8_move_kernel<8>, grid, dim3(MT), 0, s, a, tpb, ranges);
        default: return launch_ex(c.pdl, kv8_move_kernel<16>, grid, dim3(MT), 0, s, a, tpb, ranges);
    }
}

}  // namespace cb
