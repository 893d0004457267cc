// Eviction from the 8-bit paged K/V cache by accumulated attention weight.  Each KV head of each layer keeps its first
// `sink` rows, its last `recent` rows and, of the others, those with the largest weight (ties to the lower row; a
// weight that is not positive ranks as 0), `keep` rows in all; a sequence with at most `keep` rows keeps them all.
// The kept rows, in order, become rows 0 .. of the destination pages, quantised anew as a write of their values
// would be, and their weights move along.
//
//   select   one CTA per (layer, sequence, KV head): the weights' bits order as unsigned integers, so three rounds of
//            histograms of 11 and 10 bits fix the threshold (and, when more rows equal it than are wanted, rounds over the row
//            numbers of those fix the last one taken); a warp then counts and writes the kept rows of its own stretch.
//   move     one CTA per (layer, K|V, KV head, sequence) and destination page; a page's rows are in registers before it is
//            written.  Destination row r comes from a row >= r, so with equal tables (in place) one CTA does a head's
//            pages in order and nothing is overwritten before it is read.
// The moved rows are most of the bytes: move is bound by HBM, at the latency of rows -> table -> codes, which many
// small CTAs (or, in place, the next page's addresses fetched ahead) cover.  8K to 2K rows, 32 layers x 8 heads of 128: select
// 19 us, move 51 us for 268 MB of kept codes read and written (5.3 TB/s; a kept row is 128 scattered bytes).  Fewer CTAs per SM, the next
// page's codes loaded ahead and fewer instructions per code were all slower (72 .. 100 us in all against 70).
#include <climits>

#include "cb_kv8.cuh"

namespace cb {

namespace {

constexpr int ST = 512;       // select threads
constexpr int BINS = 2048;    // of select's histogram: digits of 11, 10 and 10 bits
constexpr int CACHE = 32 * ST;  // weights that a select CTA keeps in shared memory (two CTAs per SM)
constexpr int NP = 4;         // 16-byte vectors of codes per move thread
constexpr int MT = 512;       // move threads, at most: a page of 256 rows of 128 codes

struct EvictArgs {
    Kv8Seqs q;
    Kv8Evict e;
    uint8_t* codes;
    float* scales;
    int Hkv, hd, layer;
};

__device__ __forceinline__ unsigned rank_bits(float w) { return w > 0.f ? __float_as_uint(w) : 0u; }

struct Pick {
    int bin, want, count;     // the bin chosen, how many of its rows are wanted, how many it has
};

// In the histogram, the bin in which a running count from the top (or the bottom) reaches `want`.  Called by all threads,
// each with BINS / ST bins that follow each other in counting order; leaves the histogram zero.
template <bool TOP> __device__ __forceinline__ Pick find_bin(int* hist, int* totals, Pick* found, int want) {
    constexpr int PER = BINS / ST;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    int4& mine = reinterpret_cast<int4*>(hist)[TOP ? ST - 1 - t : t];
    static_assert(PER == 4, "one vector per thread");
    const int4 x = mine;
    mine = make_int4(0, 0, 0, 0);
    const int h[4] = {TOP ? x.w : x.x, TOP ? x.z : x.y, TOP ? x.y : x.z, TOP ? x.x : x.w};
    const int sum = h[0] + h[1] + h[2] + h[3];
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
    }
    if (lane == 31) totals[warp] = before;
    before -= sum;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ST / 32; ++k) before += k < warp ? totals[k] : 0;
    if (before < want && want <= before + sum) {
        int k = 0;
        while (before + h[k] < want) before += h[k++];
        *found = Pick{TOP ? BINS - 1 - (t * PER + k) : t * PER + k, want - before, h[k]};
    }
    __syncthreads();
    return *found;
}

// exclusive prefix sums over N ints in shared memory, by warp 0 (N a multiple of 32)
template <int N> __device__ __forceinline__ void warp_scan(int* v) {
    const int lane = threadIdx.x & 31;
    constexpr int PER = N / 32;
    int x[PER], sum = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        x[k] = v[lane * PER + k];
        sum += x[k];
    }
    int at = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += y;
    }
    at -= sum;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        v[lane * PER + k] = at;
        at += x[k];
    }
}

// The rows of one head.  CACHED: the weights are brought into shared memory first; otherwise each round reads them again
// (from L2).  The loops stay short: with the weights in registers, hence everything unrolled, the instructions of so many
// lines run once took longer to fetch than to execute (5 sequences of 700 rows, 2 layers: 10.1 us in all, 8.6 this way).
template <bool CACHED>
__device__ __forceinline__ void select_rows(const EvictArgs& a, const float* w, float* cache, float* ow, int* rows, int len) {
    __shared__ __align__(16) int hist[BINS];
    __shared__ int totals[ST / 32];
    __shared__ Pick found;
    __shared__ int count[32];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int kept = min(len, a.e.keep), c0 = a.e.sink, c1 = len - a.e.recent;       // candidates [c0, c1)
    // rank bits of the candidates; NONE for every other row (above all bits of a float that is not negative)
    constexpr unsigned NONE = ~0u;
    const float* src = CACHED ? cache : w;
    const auto rank_of = [&](int j) { return j >= c0 && j < c1 ? rank_bits(src[j]) : NONE; };
    if (CACHED) {
#pragma unroll 8
        for (int j = t; j < len; j += ST) cache[j] = w[j];
    }
    for (int i = t; i < BINS; i += ST) hist[i] = 0;
    __syncthreads();
    unsigned thr = 0;                                  // candidates with rank bits above it are kept ...
    int cut = -1;                                      // ... and those equal to it up to this row
    if (len > a.e.keep) {
        int want = a.e.keep - a.e.sink - a.e.recent;   // fewer than the candidates
        // rounds of a digit: a row counts when its bits above the digit are `prefix`; ties by row number.  No rank and no row
        // number has the sign bit, which keeps NONE out.
        Pick got{0, 0, 0};
        const auto round = [&](int shift, unsigned prefix, bool by_row) {
            const unsigned mask = shift == 20 ? 0x80000000u : ~0u << (shift + 10), digit = shift == 20 ? 2047u : 1023u;
            const auto add = [&](int j, unsigned b) {
                const unsigned y = by_row ? (unsigned)j : b;
                if ((y & mask) == prefix && (!by_row || b == thr)) atomicAdd(&hist[(y >> shift) & digit], 1);
            };
#pragma unroll 4
            for (int j = c0 + t; j < c1; j += ST) add(j, rank_of(j));
            __syncthreads();
            got = by_row ? find_bin<false>(hist, totals, &found, want) : find_bin<true>(hist, totals, &found, want);
            want = got.want;
            return prefix | ((unsigned)got.bin << shift);
        };
        if (want > 0) {
            for (int shift = 20; shift >= 0; shift -= 10) thr = round(shift, thr, false);
            cut = INT_MAX;
            if (got.count > want) {                    // more rows equal the threshold than are wanted
                unsigned last = 0;
                for (int shift = 20; shift >= 0; shift -= 10) last = round(shift, last, true);
                cut = (int)last;
            }
        } else {
            thr = ~0u;
        }
    }
    const auto keeps = [&](int j, unsigned b) {
        return j < len && (len <= a.e.keep || b == NONE || b > thr || (b == thr && j <= cut));
    };
    // a warp's stretch of rows: count, scan, write
    const int per = (len + ST - 1) / ST * 32, j_lo = min(len, warp * per), j_hi = min(len, j_lo + per);
    int n = 0;
#pragma unroll 4
    for (int j = j_lo; j < j_hi; j += 32) n += __popc(__ballot_sync(0xffffffffu, keeps(j + lane, rank_of(j + lane))));
    if (lane == 0) count[warp] = n;
    if (t >= ST / 32 && t < 32) count[t] = 0;
    __syncthreads();
    if (warp == 0) warp_scan<32>(count);
    __syncthreads();
    int at = count[warp];
#pragma unroll 4
    for (int j = j_lo; j < j_hi; j += 32) {
        const bool k = keeps(j + lane, rank_of(j + lane));
        const unsigned who = __ballot_sync(0xffffffffu, k);
        if (k) {
            const int to = at + __popc(who & ((1u << lane) - 1));
            rows[to] = j + lane;
            if (CACHED) ow[to] = src[j + lane];        // (in place too: all were read before one is written)
        }
        at += __popc(who);
    }
    if (!CACHED) {
        __syncthreads();
        // the kept rows' weights; in place a weight moves down (rows[i] >= i), so a step reads before it writes
        constexpr int STEP = 4;
        for (int i0 = 0; i0 < kept; i0 += STEP * ST) {
            float x[STEP];
#pragma unroll
            for (int k = 0; k < STEP; ++k) {
                const int i = i0 + k * ST + t;
                x[k] = i < kept ? w[rows[i]] : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < STEP; ++k) {
                const int i = i0 + k * ST + t;
                if (i < kept) ow[i] = x[k];
            }
        }
        __syncthreads();
    }
    for (int j = kept + t; j < a.e.keep; j += ST) rows[j] = -1;
    for (int j = kept + t; j < len; j += ST) ow[j] = 0.f;
}

__global__ void __launch_bounds__(ST, 2) kv8_select_kernel(const EvictArgs a, int cached) {
    extern __shared__ float cache[];                    // [cached]
    grid_dep_launch();
    grid_dep_wait();
    const int g = blockIdx.x, s = blockIdx.y, l = blockIdx.z;
    const int len = kv8_len(a.q, s);
    const int64_t seg = ((int64_t)l * a.q.n + s) * a.Hkv + g;
    const float* w = a.e.weights + seg * a.e.weights_ld;
    float* ow = a.e.out_weights + seg * a.e.weights_ld;
    int* rows = a.e.out_rows + seg * a.e.keep;
    if (len < 0 || len > a.q.max_len) {                 // keeps nothing
        if (threadIdx.x == 0) atomicOr(a.q.status, ST_BAD_ROW);
        for (int j = threadIdx.x; j < a.e.keep; j += ST) rows[j] = -1;
        return;
    }
    if (len <= cached) select_rows<true>(a, w, cache, ow, rows, len);
    else select_rows<false>(a, w, cache, ow, rows, len);
}

// Codes are worked on four to a word: the conversions to and from fp16 cost several times as much.  The magnitudes of
// codes compare as integers, and a factor 2^k adds k to every exponent field as long as all values are and stay normal;
// zeros, subnormals and NaN go through the conversions.
__device__ __forceinline__ unsigned largest_code(const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    unsigned m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        m = kv8_max_u16x2(m, w[k] & 0x007f007fu);
        m = kv8_max_u16x2(m, (w[k] >> 8) & 0x007f007fu);
    }
    m = max(m & 0xffffu, m >> 16);
    if (m == 0x7f) {                                   // a NaN: the largest of the others
        m = 0;
        for (int k = 0; k < 4; ++k)
            for (int n = 0; n < 32; n += 8) {
                const unsigned c = w[k] >> n & 0x7fu;
                if (c != 0x7f && c > m) m = c;
            }
    }
    return m;
}
__device__ __forceinline__ void times_power(uint4& x, float from, float inv_to) {
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    const float f = from * inv_to;
    const int k = (int)(__float_as_uint(f) >> 23) - 127;
    if (k == 0) return;
    bool fast = f > 0.f && k >= -14 && k <= 14;
    if (fast) {
        const uint32_t least = (uint32_t)(k < 0 ? 1 - k : 1) * 0x08080808u;      // smallest code that stays normal
        uint32_t all = 0x80808080u, nan = 0;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            all &= (w[n] | 0x80808080u) - least;
            nan |= (w[n] & 0x7f7f7f7fu) + 0x01010101u;
        }
        fast = (all & 0x80808080u) == 0x80808080u && !(nan & 0x80808080u);
    }
    if (fast) {
#pragma unroll
        for (int n = 0; n < 4; ++n) w[n] += (uint32_t)k * 0x08080808u;
    } else {
        const Kv8Factor f2 = kv8_factor(f);
#pragma unroll
        for (int n = 0; n < 4; ++n) w[n] = kv8_rescale4(w[n], f2);
    }
    x = make_uint4(w[0], w[1], w[2], w[3]);
}

// A page of P rows is P * hd / 16 vectors: NP for each of the CTA's threads (half the warp's, for 16 rows of 64)
__global__ void __launch_bounds__(MT) kv8_move_kernel(const EvictArgs a, int vecs, int ranges) {
    // a page's rows: index among the pool's rows of this layer's K or V (-1: none) and scale, for this page and the next
    __shared__ int from[2][256];
    __shared__ float scale[2][256];
    __shared__ float sm[MT / 32];
    grid_dep_launch();
    grid_dep_wait();
    const int g = blockIdx.y % a.Hkv, lk = blockIdx.y / a.Hkv, s = blockIdx.z, t = threadIdx.x, threads = blockDim.x;
    const int l = lk >> 1, kv = lk & 1, P = 1 << a.q.shift, vpr_shift = a.hd == 128 ? 3 : 2;
    const int len = kv8_len(a.q, s);
    const int kept = len < 0 || len > a.q.max_len ? 0 : min(len, a.e.keep), pages = (kept + P - 1) >> a.q.shift;
    // out_lens may be the lengths read above: a CTA that sees the new one finds the same `kept`
    if (blockIdx.x == 0 && blockIdx.y == 0 && t == 0) a.e.out_lens[s] = kept;
    const int* rows = a.e.out_rows + (((int64_t)l * a.q.n + s) * a.Hkv + g) * a.e.keep;
    const int64_t base = (int64_t)((a.layer + l) * 2 + kv) * a.q.n_pages * a.Hkv;
    uint8_t* codes = a.codes + base * P * a.hd;
    float* scales = a.scales + base;
    const int per = (pages + ranges - 1) / ranges, b_lo = blockIdx.x * per, b_hi = min(pages, b_lo + per);
    // Rows of a page by thread: the addresses go to shared memory at once, the scales, which only the next step needs,
    // when the codes have been asked for.
    float sc = 0.f;                                    // (there are at least as many threads as rows)
    const auto resolve = [&](int b, int buf) {
        int at = -1;
        sc = 0.f;
        if (t < P && b * P + t < kept) {
            const int j = rows[b * P + t], pg = kv8_page(a.q, s, j >> a.q.shift);
            if (pg >= 0) {
                at = (pg * a.Hkv + g) * P + (j & (P - 1));
                sc = scales[pg * a.Hkv + g];
            }
        }
        if (t < P) from[buf][t] = at;
    };
    if (b_lo >= b_hi) return;
    resolve(b_lo, 0);
    for (int b = b_lo, buf = 0; b < b_hi; ++b, buf ^= 1) {
        const int dst = a.e.dst_table[(int64_t)s * a.e.dst_ld + b];
        __syncthreads();                               // this page's addresses are there, the page before is written
        uint4 x[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int v = t + i * threads, at = v < vecs ? from[buf][v >> vpr_shift] : -1;
            x[i] = make_uint4(0, 0, 0, 0);
            if (at >= 0) x[i] = reinterpret_cast<const uint4*>(codes + (int64_t)at * a.hd)[v & ((1 << vpr_shift) - 1)];
        }
        if (t < P) scale[buf][t] = sc;
        if (b + 1 < b_hi) resolve(b + 1, buf ^ 1);
        __syncthreads();
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int v = t + i * threads;
            top = fmaxf(top, kv8_value2(largest_code(x[i])).x * (v < vecs ? scale[buf][v >> vpr_shift] : 0.f));
        }
        top = warp_max(top);
        if ((t & 31) == 0) sm[t >> 5] = top;
        __syncthreads();                               // also: every row of this page has been read
        for (int i = 0; i < threads / 32; ++i) top = fmaxf(top, sm[i]);
        const float ns = kv8_scale(top), inv = kv8_inverse(ns);
        if (dst < 0 || dst >= a.q.n_pages) {
            if (t == 0) atomicOr(a.q.status, ST_BAD_ROW);
            continue;
        }
        const int n = min(P, kept - b * P), blk = dst * a.Hkv + g;
        uint4* out = reinterpret_cast<uint4*>(codes + (int64_t)blk * P * a.hd);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int v = t + i * threads, row = v >> vpr_shift;
            if (v >= vecs || row >= n) continue;
            times_power(x[i], scale[buf][row], inv);
            out[v] = x[i];
        }
        if (t == 0) scales[blk] = ns;
    }
}

}  // namespace

cudaError_t launch_kv8_evict(const Kv8& c, const Kv8Seqs& q, const Kv8Evict& e, int layer, int n_layers, cudaStream_t s) {
    EvictArgs a{q, e, c.codes, c.scales, c.cfg.n_kv_heads, c.cfg.head_dim, layer};
    if (q.n == 0 || n_layers == 0) return cudaSuccess;
    static std::atomic<uint64_t> done{0};
    cudaError_t err = smem_limit_once(kv8_select_kernel, CACHE * 4, done);
    if (err != cudaSuccess) return err;
    const int cached = q.max_len < CACHE ? q.max_len : CACHE;
    err = launch_ex(c.pdl, kv8_select_kernel, dim3(a.Hkv, q.n, n_layers), dim3(ST), cached * 4, s, a, cached);
    if (err != cudaSuccess) return err;
    const int P = 1 << q.shift, vecs = P * a.hd / 16;                    // 64 .. 2048 vectors
    const int threads = vecs / NP < 32 ? 32 : vecs / NP;                 // P or 2 P, at least 32
    const int pages = ((e.keep < q.max_len ? e.keep : q.max_len) + P - 1) / P;
    // In place the pages of a head are done in order by one CTA.  Between two tables they are divided until there are 24
    // CTAs per SM: a CTA that has several looks up the next one's rows while it moves one (8K to 2K, 32 layers: one page
    // per CTA 57 us, four 53 us).
    const bool in_place = e.dst_table == q.table && e.dst_ld == q.table_ld;
    const int64_t heads = (int64_t)2 * n_layers * a.Hkv * q.n, most = ((int64_t)24 * c.num_sms + heads - 1) / heads;
    const int ranges = in_place || pages == 0 ? 1 : (int)(pages < most ? pages : most);
    return launch_ex(c.pdl, kv8_move_kernel, dim3(ranges, 2 * n_layers * a.Hkv, q.n), dim3(threads), 0, s, a, vecs, ranges);
}

}  // namespace cb
