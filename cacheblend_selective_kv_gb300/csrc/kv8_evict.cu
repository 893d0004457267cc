// Eviction from the 8-bit paged K/V cache by accumulated attention weight.  Each KV head of each layer keeps its first
// `sink` rows, its last `recent` rows and, of the others, those with the largest weight (ties to the lower row; a
// weight that is not positive ranks as 0), `keep` rows in all; a sequence with at most `keep` rows keeps them all.
// The kept rows, in order, become rows 0 .. of the destination pages, quantised anew as a write of their values
// would be, and their weights move along.
//
//   select   one CTA per (layer, sequence, KV head): the weights' bits order as unsigned integers, so four rounds of a
//            256-bin histogram fix the threshold, then one pass in row order writes the kept rows and their weights.
//   move     one CTA per (layer, K|V, KV head, sequence) and range of destination pages; each page's rows are in
//            registers before the page is written.  Destination row r comes from a row >= r, so with equal tables (in
//            place) and the pages done in order nothing is overwritten before it is read.
#include "cb_kv8.cuh"

namespace cb {

namespace {

constexpr int ST = 512;       // select threads
constexpr int MT = 256;       // move threads

struct EvictArgs {
    Kv8Seqs q;
    Kv8Evict e;
    uint8_t* codes;
    float* scales;
    int Hkv, hd, layer;
};

__device__ __forceinline__ unsigned rank_bits(float w) { return w > 0.f ? __float_as_uint(w) : 0u; }

// exclusive prefix of v over the CTA's ST threads, and the total; sm holds ST / 32 + 1 ints
__device__ __forceinline__ int block_prefix(int v, int* sm, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                                   // sm is free again
    if (lane == 31) sm[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < ST / 32; ++w) {
        const int t = sm[w];
        if (w < warp) before += t;
        all += t;
    }
    total = all;
    return before + x - v;
}

__global__ void __launch_bounds__(ST) kv8_select_kernel(const EvictArgs a) {
    __shared__ int hist[256];
    __shared__ int sm[ST / 32 + 1];
    __shared__ unsigned pick[2];                       // digit chosen, rows still wanted below it
    const int g = blockIdx.x, s = blockIdx.y, l = blockIdx.z, t = threadIdx.x;
    int len = kv8_len(a.q, s);
    if (len < 0 || len > a.q.max_len) {
        if (t == 0) atomicOr(a.q.status, ST_BAD_ROW);
        return;
    }
    const int64_t seg = ((int64_t)l * a.q.n + s) * a.Hkv + g;
    const float* w = a.e.weights + seg * a.e.weights_ld;
    float* ow = a.e.out_weights + seg * a.e.weights_ld;
    int* rows = a.e.out_rows + seg * a.e.keep;
    const int kept = min(len, a.e.keep);
    unsigned thr = 0;                                  // rows with rank bits above it are kept ...
    int ties = 0;                                      // ... and the first `ties` rows equal to it
    const int c0 = a.e.sink, c1 = len - a.e.recent;    // candidates [c0, c1)
    if (len > a.e.keep) {
        int want = a.e.keep - a.e.sink - a.e.recent;   // > = 0; fewer than the candidates
        unsigned prefix = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = t; i < 256; i += ST) hist[i] = 0;
            __syncthreads();
            const unsigned mask = shift == 24 ? 0u : ~0u << (shift + 8);
            for (int j = c0 + t; j < c1; j += ST) {
                const unsigned b = rank_bits(w[j]);
                if ((b & mask) == prefix) atomicAdd(&hist[(b >> shift) & 255u], 1);
            }
            __syncthreads();
            if (t == 0) {                              // the digit that holds the want-th largest
                int left = want, d = 255;
                while (d > 0 && hist[d] < left) left -= hist[d--];
                pick[0] = (unsigned)d;
                pick[1] = (unsigned)left;
            }
            __syncthreads();
            prefix |= pick[0] << shift;
            want = (int)pick[1];
        }
        thr = prefix;
        ties = want;
    }
    int n_out = 0, n_tie = 0;
    for (int j0 = 0; j0 < len; j0 += ST) {
        const int j = j0 + t;
        const float wj = j < len ? w[j] : 0.f;
        const unsigned b = rank_bits(wj);
        const bool cand = j >= c0 && j < c1;
        bool keep = j < len && (!cand || len <= a.e.keep || b > thr);
        const bool tie = j < len && !keep && b == thr;
        int total;
        const int before = block_prefix(tie ? 1 : 0, sm, total);
        if (tie && n_tie + before < ties) keep = true;
        n_tie += total;
        const int at = n_out + block_prefix(keep ? 1 : 0, sm, total);
        if (keep && at < kept) {                       // in place: at <= j, and this step's weights are in registers
            rows[at] = j;
            ow[at] = wj;
        }
        n_out += total;
    }
    __syncthreads();
    for (int j = kept + t; j < len; j += ST) ow[j] = 0.f;
    for (int j = kept + t; j < a.e.keep; j += ST) rows[j] = -1;
}

// NP 16-byte vectors of codes per thread: a page of P rows is P * hd / 16 vectors
template <int NP>
__global__ void __launch_bounds__(MT) kv8_move_kernel(const EvictArgs a, int tpb, int ranges) {
    __shared__ float sm[MT / 32];
    const int g = blockIdx.y % a.Hkv, lk = blockIdx.y / a.Hkv, s = blockIdx.z, t = threadIdx.x;
    const int l = lk >> 1, kv = lk & 1, P = 1 << a.q.shift, vpr = a.hd / 16;
    const int len = kv8_len(a.q, s);
    if (len < 0 || len > a.q.max_len) return;
    const int kept = min(len, a.e.keep), pages = (kept + P - 1) >> a.q.shift;
    // out_lens may be the lengths read above: a CTA that sees the new one finds the same `kept`
    if (blockIdx.x == 0 && blockIdx.y == 0 && t == 0) a.e.out_lens[s] = kept;
    const int64_t seg = ((int64_t)l * a.q.n + s) * a.Hkv + g;
    const int* rows = a.e.out_rows + seg * a.e.keep;
    const int64_t base = (int64_t)((a.layer + l) * 2 + kv) * a.q.n_pages;
    const int per = (pages + ranges - 1) / ranges;
    for (int b = blockIdx.x * per; b < min(pages, ((int)blockIdx.x + 1) * per); ++b) {
        uint4 x[NP];
        float sc[NP];
        float top = 0.f;
        const int n = min(P, kept - b * P);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int v = t + i * tpb, row = v / vpr, e = v - row * vpr;
            x[i] = make_uint4(0, 0, 0, 0);
            sc[i] = 0.f;
            if (t < tpb && row < n) {
                const int j = rows[b * P + row];
                const int pg = kv8_page(a.q, s, j >> a.q.shift);
                if (pg >= 0) {
                    const int64_t blk = (base + pg) * a.Hkv + g;
                    x[i] = reinterpret_cast<const uint4*>(a.codes + (blk * P + (j & (P - 1))) * a.hd)[e];
                    sc[i] = a.scales[blk];
                }
            }
        }
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
        if ((t & 31) == 0) sm[t >> 5] = top;
        __syncthreads();                               // also: every row of this page has been read
        for (int i = 0; i < MT / 32; ++i) top = fmaxf(top, sm[i]);
        const float ns = kv8_scale(top), inv = kv8_inverse(ns);
        const int pg = a.e.dst_table[(int64_t)s * a.e.dst_ld + b];
        if (pg < 0 || pg >= a.q.n_pages) {
            if (t == 0) atomicOr(a.q.status, ST_BAD_ROW);
        } else {
            const int64_t blk = (base + pg) * a.Hkv + g;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int v = t + i * tpb, row = v / vpr;
                if (t >= tpb || row >= n) continue;
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
        __syncthreads();                               // the page and sm are done with before the next one
    }
}

}  // namespace

cudaError_t launch_kv8_evict(const Kv8& c, const Kv8Seqs& q, const Kv8Evict& e, int layer, int n_layers, cudaStream_t s) {
    EvictArgs a{q, e, c.codes, c.scales, c.cfg.n_kv_heads, c.cfg.head_dim, layer};
    if (q.n == 0 || n_layers == 0) return cudaSuccess;
    kv8_select_kernel<<<dim3(a.Hkv, q.n, n_layers), ST, 0, s>>>(a);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const int P = 1 << q.shift, vecs = P * a.hd / 16;
    const int tpb = vecs < MT ? vecs : MT, np = vecs / tpb;
    const int pages = ((e.keep < q.max_len ? e.keep : q.max_len) + P - 1) / P;
    // in place the pages of a head are done in order by one CTA; between two tables they are split
    const bool in_place = e.dst_table == q.table && e.dst_ld == q.table_ld;
    const int64_t heads = (int64_t)2 * n_layers * a.Hkv * q.n;
    int64_t ranges = in_place ? 1 : ((int64_t)c.num_sms * 16 + heads - 1) / heads;
    if (ranges > pages) ranges = pages > 0 ? pages : 1;
    const dim3 grid((unsigned)ranges, 2 * n_layers * a.Hkv, q.n);
    switch (np) {
        case 1: kv8_move_kernel<1><<<grid, MT, 0, s>>>(a, tpb, (int)ranges); break;
        case 2: kv8_move_kernel<2><<<grid, MT, 0, s>>>(a, tpb, (int)ranges); break;
        case 4: kv8_move_kernel<4><<<grid, MT, 0, s>>>(a, tpb, (int)ranges); break;
        default: kv8_move_kernel<8><<<grid, MT, 0, s>>>(a, tpb, (int)ranges); break;
    }
    return cudaGetLastError();
}

}  // namespace cb
