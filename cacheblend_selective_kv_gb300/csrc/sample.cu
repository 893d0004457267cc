// The next token from a row of logits: temperature, top-k, top-p, min-p and a given uniform number (cb_sample).
//
// With weights w_i = 2^((x_i - max) log2(e) / T), in descending order of x (ties to the lower token): top-k keeps the first k,
// top-p of those the ones before which the weights sum to less than p of theirs, min-p of those w_i >= p_min w_max.  The
// token is the lowest i whose kept weights up to i pass u times their sum.
//
// The result is a whole number, so sums have to be where the exact ones are: at a vocabulary of 128K a border that is off by
// 2^-24 of the sum would pick a neighbour in one row of a hundred.  Weights are therefore 64-bit integers, in units of
// 2^-44 to 2^-45 of the largest, and their sums are exact and independent of the order of adding.  A weight is good to about
// 2^-32 of itself: x / T as a sum of two fp32 numbers, its integer part in 256ths by rounding, 2^(j / 256) from a table of
// 32-bit integers, and 2^r - 1 for the rest (|r| <= 2^-9) by three terms of the series, all in fp32 and one wide integer product.
// A weight below 2^-45 of the largest is 0.
//
// A row is a cluster's: its CTAs hold the row in shared memory, as fp32, and every pass over it reads it there.  What passes
// find out is left in shared memory for all CTAs of the cluster, and each works out the same next step from it.
// Threshold of top-k or top-p: a histogram of the values (of counts, or of weights as two 32-bit words and a carry) over 1024
// equal steps from the largest value down, the step in which the sum crosses, and the items of that step one by one; a step with
// too many of them is divided again, and equal values are counted off in the tokens' order.
#include <cstdarg>
#include <cstdio>

#include "cb_ptx.cuh"

using namespace cb;

namespace {

constexpr int THREADS = 1024, WARPS = THREADS / 32;
constexpr int BINS = THREADS;            // a thread per bin where they are summed
constexpr int CAP = 256;                 // items of a bin that are looked at one by one
constexpr int GRAIN = 4 * THREADS;       // a CTA's part of a row is a multiple of it
constexpr int MOST_CTAS = 8;
constexpr int MOST_PART = 49152;         // floats of a row in a CTA
constexpr float MAGIC = 12582912.f;      // 1.5 * 2^23: adding it rounds to a whole number
constexpr int MAGIC_BITS = 0x4B400000;

// 2^(j / 256) in units of 2^-31, rounded
struct PowerTable {
    unsigned of[256];
};
constexpr double power_of(double x) {    // e^x for x in [0, ln 2), by its series
    double sum = 1.0, term = 1.0;
    for (int n = 1; n < 30; ++n) {
        term *= x / n;
        sum += term;
    }
    return sum;
}
constexpr PowerTable make_powers() {
    PowerTable t{};
    for (int j = 0; j < 256; ++j) t.of[j] = (unsigned)(power_of(j * (0.69314718055994530942 / 256)) * 2147483648.0 + 0.5);
    return t;
}
__device__ constexpr PowerTable kPowers = make_powers();

struct SampleArgs {
    const void* logits;
    int64_t stride;                      // elements between rows
    int vocab, part, ctas;               // part: floats of a row per CTA; CTAs per row
    const float* temperature;
    const int* top_k;
    const float* top_p;
    const float* min_p;
    const float* uniform;
    int* out_tokens;
    float* out_probs;
};

struct Item {
    float x;
    int i;
};
struct Shared {
    unsigned power[256];
    // left for the cluster
    unsigned long long best;             // key of the CTA's largest value and its first token
    unsigned low;                        // key of its smallest finite value
    unsigned hist[2][2][BINS];           // counts, or weights' low and high words; two buffers
    unsigned found[2], low_of[2], high_of[2];      // items of the bin: how many, keys of the smallest and the largest value
    Item list[2][CAP];
    int tie;                             // the token at which equal values are cut off
    unsigned long long warp_sum[WARPS];
    // of the CTA
    unsigned long long scan[WARPS];
    int bin;
    unsigned long long above;
    Item joined[CAP];
    unsigned long long weight[CAP];
    float cut_x;
    int cut_i;
    int segment;
};

__device__ __forceinline__ unsigned ld_cluster(uint32_t caddr) {
    unsigned v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(caddr));
    return v;
}
__device__ __forceinline__ unsigned long long ld_cluster64(uint32_t caddr) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(caddr));
    return v;
}
template <typename V> __device__ __forceinline__ uint32_t of_rank(const V* p, int rank) {
    return ptx::map_to_rank(ptx::smem_u32(p), (uint32_t)rank);
}

__device__ __forceinline__ void sync_cluster() {
    __syncwarp();
    ptx::cluster_sync();
}

// unsigned integers that order like the floats (no NaN, no -0)
__device__ __forceinline__ unsigned key_of(float x) {
    const unsigned b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(unsigned k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }

__device__ __forceinline__ unsigned long long shfl64(unsigned long long v, int lane) {
    const unsigned lo = __shfl_sync(0xffffffffu, (unsigned)v, lane), hi = __shfl_sync(0xffffffffu, (unsigned)(v >> 32), lane);
    return ((unsigned long long)hi << 32) | lo;
}
__device__ __forceinline__ unsigned long long warp_sum64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ unsigned long long warp_scan64(unsigned long long v) {        // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}
// inclusive sum over the block's threads, and the sum of all
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* sm, unsigned long long& total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v = warp_scan64(v);
    __syncthreads();
    if (lane == 31) sm[warp] = v;
    __syncthreads();
    const unsigned long long sums = warp_scan64(sm[lane]);
    total = shfl64(sums, 31);
    const unsigned long long before = shfl64(sums, warp > 0 ? warp - 1 : 0);
    return warp > 0 ? v + before : v;
}

// Weights of a row: 2^(x t - m t) in units of 2^-44 of the power of two at or below the largest.
struct Weigh {
    float th, tl, shift;                 // t = log2(e) / T as a sum; x is taken relative to `shift`
    int top;                             // floor of the largest x t
    const unsigned* power;
    __device__ __forceinline__ int split(float x, float& r) const {             // x t = k / 256 + r
        x -= shift;
        const float hi = fmaxf(x * th, -16000.f);
        const float lo = fmaf(x, tl, fmaf(x, th, -hi));
        const float km = fmaf(hi, 256.f, MAGIC);
        r = fmaf(km - MAGIC, -1.f / 256.f, hi) + lo;
        return __float_as_int(km) - MAGIC_BITS;
    }
    __device__ __forceinline__ unsigned long long operator()(float x) const {
        float r;
        const int k = split(x, r);
        const float q = fmaf(r, fmaf(r, 5.5504109e-2f, 2.4022651e-1f), 6.9314718e-1f);
        const int v = __float_as_int(fmaf(r * 2147483648.f, q, MAGIC)) - MAGIC_BITS;     // (2^r - 1) 2^31
        const unsigned long long product = (unsigned long long)power[k & 255] * (0x80000000u + (unsigned)v);
        const int down = 18 + top - (k >> 8);
        return down < 64 ? product >> down : 0ull;
    }
};

// ceil(f s) and floor(f s) for f in [0, 1) (multiples of 2^-64, as every fp32 from 2^-40 on is)
__device__ __forceinline__ unsigned long long fraction(float f) {
    return f > 0.f ? (unsigned long long)(f * 18446744073709551616.f) : 0ull;
}
__device__ __forceinline__ unsigned long long floor_of(float f, unsigned long long s) { return __umul64hi(fraction(f), s); }
__device__ __forceinline__ unsigned long long ceil_of(float f, unsigned long long s) {
    return __umul64hi(fraction(f), s) + (fraction(f) * s != 0ull);
}

// what is kept: x above the cut's, or equal to it and a token up to the cut's
struct Cut {
    float x;
    int i;
    __device__ __forceinline__ bool keeps(float y, int j) const { return y > x || (y == x && j <= i); }
};

struct Row {
    const float* x;                      // this CTA's part
    int part, first, ctas, rank;         // first: its first token
    template <typename F> __device__ __forceinline__ void each(F f) const {      // in the tokens' order within a warp's steps
        const int per = part / WARPS;
        const float* from = x + (threadIdx.x >> 5) * per;
        const int j0 = first + (threadIdx.x >> 5) * per;
        for (int at = (threadIdx.x & 31) * 4; at < per; at += 128) {
            const float4 v = *reinterpret_cast<const float4*>(from + at);
            f(v.x, j0 + at);
            f(v.y, j0 + at + 1);
            f(v.z, j0 + at + 2);
            f(v.w, j0 + at + 3);
        }
    }
};

// Lowers the cut to the first kept item, in descending order, at which the sum of counts (MASS: of weights) reaches the target:
// `most` items, or p of the sum.  All CTAs of the cluster come to the same cut.  `phase` alternates the buffers that others
// read: one is written again only when all have passed the next barrier of the cluster.
template <bool MASS>
__device__ __forceinline__ void select(const Row& row, const Weigh& w, Shared& s, float m, float low, int most, float p, Cut& cut, int& phase) {
    const int tid = threadIdx.x, lane = tid & 31;
    float high = m;
    float range = fminf(m - low, 3.4e38f);
    const float reach = 47.f / w.th;                   // below it weights are 0
    const bool cut_off = reach < range;
    range = cut_off ? reach : range;
    unsigned long long above = 0, target = MASS ? 0ull : (unsigned long long)most;
    // The largest and the smallest value of a level never share a step and a step is at most 1 / 1022 of its level's range, so
    // that 28 levels lead from the largest difference of two fp32 numbers to the smallest.
    for (int level = 0; level < 40; ++level) {
        const int b = phase++ & 1;
        // (differences of small numbers are brought up first: 1 / range could pass fp32, and all values be in one step for ever)
        const float up = range < 0x1p-60f ? 0x1p100f : 1.f, step = range > 0.f ? (BINS - 1) / (range * up) : 0.f;
        const auto bin_of = [&](float x) { return (int)fminf(fminf(high - x, 3.4e38f) * up * step, BINS - 1); };
        const auto inside = [&](float x, int j) { return cut.keeps(x, j) && (level == 0 || (x <= high && x >= low)); };
        s.hist[b][0][tid] = 0;
        s.hist[b][1][tid] = 0;
        if (tid == 0) {
            s.found[b] = 0;
            s.low_of[b] = 0xffffffffu;
            s.high_of[b] = 0;
        }
        __syncthreads();
        row.each([&](float x, int j) {
            if (!inside(x, j)) return;
            const int at = bin_of(x);
            if constexpr (MASS) {
                const unsigned long long y = w(x);
                const unsigned lo = (unsigned)y, was = atomicAdd(&s.hist[b][0][at], lo);
                const unsigned hi = (unsigned)(y >> 32) + (was + lo < was);
                if (hi) atomicAdd(&s.hist[b][1][at], hi);
            } else {
                atomicAdd(&s.hist[b][0][at], 1u);
            }
        });
        sync_cluster();
        unsigned long long here = 0;
        for (int r = 0; r < row.ctas; ++r) {
            here += ld_cluster(of_rank(&s.hist[b][0][tid], r));
            if (MASS) here += (unsigned long long)ld_cluster(of_rank(&s.hist[b][1][tid], r)) << 32;
        }
        unsigned long long total;
        const unsigned long long upto = above + block_scan(here, s.scan, total);
        if (MASS && level == 0) target = max(ceil_of(p, total), 1ull);
        if (level == 0 && total < target) return;      // fewer items than top-k keeps
        if (upto - here < target && target <= upto) {
            s.bin = tid;
            s.above = upto - here;
        }
        __syncthreads();
        const int bin = s.bin;
        above = s.above;
        if (level == 0 && cut_off && bin == BINS - 1) return;      // what is cut has no weight
        // the bin's items
        float least = INFINITY, largest = -INFINITY;
        row.each([&](float x, int j) {
            if (!inside(x, j) || bin_of(x) != bin) return;
            const unsigned n = atomicAdd(&s.found[b], 1u);
            if (n < CAP) s.list[b][n] = Item{x, j};
            least = fminf(least, x);
            largest = fmaxf(largest, x);
        });
        if (largest >= least) {
            atomicMin(&s.low_of[b], key_of(least));
            atomicMax(&s.high_of[b], key_of(largest));
        }
        sync_cluster();
        unsigned n = 0, before = 0, mine = 0, lo_key = 0xffffffffu, hi_key = 0;
        int from = 0;
        for (int r = 0; r < row.ctas; ++r) {
            const unsigned k = ld_cluster(of_rank(&s.found[b], r));
            if ((unsigned)tid >= n && (unsigned)tid < n + k) {
                from = r;
                mine = tid - n;
            }
            if (r < row.rank) before += k;
            n += k;
            lo_key = min(lo_key, ld_cluster(of_rank(&s.low_of[b], r)));
            hi_key = max(hi_key, ld_cluster(of_rank(&s.high_of[b], r)));
        }
        if (n <= CAP) {
            if (tid < (int)n) {
                const uint32_t at = of_rank(&s.list[b][mine], from);
                const Item it{__uint_as_float(ld_cluster(at)), (int)ld_cluster(at + 4)};
                s.joined[tid] = it;
                s.weight[tid] = MASS ? w(it.x) : 1ull;
            }
            __syncthreads();
            if (tid < (int)n) {
                const Item it = s.joined[tid];
                unsigned long long sum = above;
                for (int k = 0; k < (int)n; ++k) {
                    const Item o = s.joined[k];
                    if (o.x > it.x || (o.x == it.x && o.i < it.i)) sum += s.weight[k];
                }
                if (sum < target && target <= sum + s.weight[tid]) {
                    s.cut_x = it.x;
                    s.cut_i = it.i;
                }
            }
            __syncthreads();
            cut = Cut{s.cut_x, s.cut_i};
            return;
        }
        low = of_key(lo_key);
        high = of_key(hi_key);
        range = fminf(high - low, 3.4e38f);
        if (low == high) {                             // equal values: the first of them in the tokens' order
            const unsigned long long each = MASS ? w(high) : 1ull;
            const unsigned long long keep = (target - above + each - 1) / each;
            if (keep >= n) {
                if (cut.x != high) cut = Cut{high, 0x7fffffff};
                return;
            }
            const unsigned here_n = s.found[b];
            if (keep > before && keep <= before + here_n) {
                // this CTA has the token: by warp, then step by step
                int count = 0;
                row.each([&](float x, int j) { count += x == high && cut.keeps(x, j); });
                const unsigned long long warps = __reduce_add_sync(0xffffffffu, (unsigned)count);
                unsigned long long all;
                const unsigned long long end = before + block_scan(lane == 31 ? warps : 0ull, s.scan, all);
                // (the sum up to lane 31 of this warp; other lanes have what stands before the warp)
                const unsigned long long begin = shfl64(end, 0);
                if (keep > begin && keep <= begin + warps) {
                    unsigned left = (unsigned)(keep - begin);
                    const int per = row.part / WARPS, w0 = (tid >> 5) * per;
                    for (int at = w0; at < w0 + per; at += 32) {
                        const int j = row.first + at + lane;
                        const bool is = row.x[at + lane] == high && cut.keeps(high, j);
                        const unsigned votes = __ballot_sync(0xffffffffu, is);
                        if ((unsigned)__popc(votes) >= left) {
                            if (is && __popc(votes & ((2u << lane) - 1u)) == (int)left) s.tie = j;
                            break;
                        }
                        left -= __popc(votes);
                    }
                }
            }
            sync_cluster();
            int owner = 0;
            unsigned upto_r = 0;
            for (int r = 0; r < row.ctas; ++r) {
                const unsigned k = ld_cluster(of_rank(&s.found[b], r));
                if (keep > upto_r && keep <= upto_r + k) owner = r;
                upto_r += k;
            }
            cut = Cut{high, (int)ld_cluster(of_rank(&s.tie, owner))};
            return;
        }
        __syncthreads();                               // bin, above and the scan's sums are written again
    }
}

__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float4 load_four(const float* p) { return __ldcs(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load_four(const bf16* p) {
    const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}

template <typename T>
__global__ void __launch_bounds__(THREADS, 1) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) float xs[];        // [part]
    __shared__ Shared s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ctas = a.ctas, rank = (int)ptx::cluster_rank();
    const int r = blockIdx.x / ctas;
    if (tid < 256) s.power[tid] = kPowers.of[tid];
    const float temperature = a.temperature ? a.temperature[r] : 1.f;
    const int top_k = a.top_k ? a.top_k[r] : 0;
    const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f, u = a.uniform[r];

    // The row into shared memory, a NaN as -inf and -0 as 0; its largest value and that one's first token
    const Row row{xs, a.part, rank * a.part, ctas, rank};
    float best = -INFINITY, low = INFINITY;
    int best_i = 0x7fffffff;
    {
        const T* src = (const T*)a.logits + (int64_t)r * a.stride;
        const int per = a.part / WARPS, n = a.vocab;
        const bool wide = ((uintptr_t)src & (4 * sizeof(T) - 1)) == 0;
#pragma unroll 4
        for (int at = lane * 4; at < per; at += 128) {
            const int to = warp * per + at, j = row.first + to;
            float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (wide && j + 4 <= n) {
                const float4 f = load_four(src + j);
                v[0] = f.x;
                v[1] = f.y;
                v[2] = f.z;
                v[3] = f.w;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (j + k < n) v[k] = load_one(src + j + k);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = v[k] == v[k] ? v[k] + 0.f : -INFINITY;
                if (v[k] > best) {
                    best = v[k];
                    best_i = j + k;
                }
                if (v[k] > -INFINITY) low = fminf(low, v[k]);
            }
            *reinterpret_cast<float4*>(xs + to) = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
    if (tid == 0) {
        s.best = 0;
        s.low = 0xffffffffu;
    }
    __syncthreads();
    {
        unsigned long long k = ((unsigned long long)key_of(best) << 32) | (unsigned)~best_i;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) k = max(k, __shfl_xor_sync(0xffffffffu, k, o));
        const unsigned l = __reduce_min_sync(0xffffffffu, key_of(low));
        if (lane == 0) {
            atomicMax(&s.best, k);
            atomicMin(&s.low, l);
        }
    }
    sync_cluster();
    unsigned long long k_best = 0;
    unsigned k_low = 0xffffffffu;
    for (int c = 0; c < ctas; ++c) {
        k_best = max(k_best, ld_cluster64(of_rank(&s.best, c)));
        k_low = min(k_low, ld_cluster(of_rank(&s.low, c)));
    }
    float m = of_key((unsigned)(k_best >> 32));
    low = of_key(k_low);
    const bool greedy = !(temperature >= 1.1754944e-38f);
    if (m == -INFINITY || greedy) {                    // no token, or the most likely one
        if (rank == 0 && tid == 0) {
            a.out_tokens[r] = m == -INFINITY ? -1 : (int)~(unsigned)k_best;
            if (a.out_probs) a.out_probs[r] = m == -INFINITY ? 0.f : 1.f;
        }
        sync_cluster();                           // no CTA exits while another reads its shared memory
        return;
    }
    if (m == INFINITY) {                               // infinities share all the weight (a thread reads what it has written)
        const int per = a.part / WARPS;
        for (int at = lane * 4; at < per; at += 128)
            for (int k = 0; k < 4; ++k) {
                float& x = xs[warp * per + at + k];
                x = x == INFINITY ? 0.f : -INFINITY;
            }
        m = low = 0.f;
        __syncthreads();
    }
    Weigh w;
    {
        const float T1 = fminf(temperature, 3.4e38f);
        w.th = 1.44269502f / T1;                       // log2(e) = 1.44269502 + 1.92596299e-8
        w.tl = (fmaf(-w.th, T1, 1.44269502f) + 1.92596299e-8f) / T1;
        w.shift = fabsf(m) * w.th >= 8192.f ? m : 0.f; // (what has weight lies so near to m then that x - m is exact)
        w.power = s.power;
        float rest;
        w.top = w.split(m, rest) >> 8;
    }
    Cut cut{-INFINITY, -1};
    int phase = 0;
    if (top_k > 0 && top_k < a.vocab) select<false>(row, w, s, m, low, top_k, 1.f, cut, phase);
    if (top_p < 1.f) select<true>(row, w, s, m, low, 0, top_p, cut, phase);
    const unsigned long long least = min_p >= 1.f ? w(m) : ceil_of(min_p, w(m));

    // sums of what is kept, per warp; the warp in which they pass u of their sum; the token in it
    const auto kept = [&](float x, int j) {
        if (!cut.keeps(x, j)) return 0ull;
        const unsigned long long y = w(x);
        return y >= least ? y : 0ull;
    };
    {
        unsigned long long sum = 0;
        row.each([&](float x, int j) { sum += kept(x, j); });
        sum = warp_sum64(sum);
        if (lane == 0) s.warp_sum[warp] = sum;
    }
    sync_cluster();
    unsigned long long total;
    const unsigned long long part = tid < ctas * WARPS ? ld_cluster64(of_rank(&s.warp_sum[lane], warp)) : 0ull;
    const unsigned long long upto = block_scan(part, s.scan, total);
    const unsigned long long target = u >= 1.f ? total - 1 : floor_of(u, total);
    if (upto - part <= target && target < upto) {
        s.segment = tid;
        s.above = upto - part;
    }
    __syncthreads();
    if (s.segment / WARPS == rank && s.segment % WARPS == warp) {
        unsigned long long before = s.above;
        const int per = a.part / WARPS;
        for (int at = 0; at < per; at += 128) {
            const int to = warp * per + at + lane * 4;
            const float4 v = *reinterpret_cast<const float4*>(xs + to);
            const float x[4] = {v.x, v.y, v.z, v.w};
            unsigned long long y[4], sum = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[k] = kept(x[k], row.first + to + k);
                sum += y[k];
            }
            const unsigned long long end = before + warp_scan64(sum);
            unsigned long long c = end - sum;
            if (c <= target && target < end) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (c <= target && target < c + y[k]) {
                        a.out_tokens[r] = row.first + to + k;
                        if (a.out_probs) a.out_probs[r] = (float)((double)y[k] / (double)total);
                    }
                    c += y[k];
                }
            }
            before = shfl64(end, 31);
            if (target < before) break;
        }
    }
    sync_cluster();
}

template <typename T> cudaError_t launch_sample(const SampleArgs& a, int n_rows, int ctas, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = smem_limit_once(sample_kernel<T>, MOST_PART * 4, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n_rows * ctas));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = (size_t)a.part * 4;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
}

cb_status fail(cb_status code, const char* fmt, ...) {
    char msg[300];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    set_last_error(msg);
    return code;
}

}  // namespace

extern "C" cb_status cb_sample(const void* logits, int32_t dtype, int32_t n_rows, int32_t vocab, int64_t row_stride,
                               const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                               const float* uniform, int32_t* out_tokens, float* out_probs, void* stream) {
    set_last_error("");
    if (dtype != CB_F32 && dtype != CB_BF16) return fail(CB_ERR_INVALID_ARG, "cb_sample: dtype must be CB_F32 or CB_BF16");
    if (n_rows < 0 || n_rows > (1 << 24)) return fail(CB_ERR_INVALID_ARG, "cb_sample: n_rows %d outside [0, 2^24]", n_rows);
    if (vocab <= 0) return fail(CB_ERR_INVALID_ARG, "cb_sample: vocab %d is not positive", vocab);
    if (vocab > CB_SAMPLE_MAX_VOCAB) return fail(CB_ERR_UNSUPPORTED, "cb_sample: a vocabulary of %d is above %d", vocab, CB_SAMPLE_MAX_VOCAB);
    if (n_rows == 0) return CB_OK;
    if (row_stride < vocab || row_stride > ((int64_t)1 << 40))
        return fail(CB_ERR_INVALID_ARG, "cb_sample: row stride %lld below the vocabulary's %d, or out of range", (long long)row_stride, vocab);
    if (!logits || !uniform || !out_tokens) return fail(CB_ERR_INVALID_ARG, "cb_sample: null logits, uniform or out_tokens");
    const int es = dtype == CB_BF16 ? 2 : 4;
    if ((uintptr_t)logits % es || ((uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p | (uintptr_t)uniform |
                                   (uintptr_t)out_tokens | (uintptr_t)out_probs) % 4)
        return fail(CB_ERR_INVALID_ARG, "cb_sample: a pointer is not aligned to its elements");
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return fail(CB_ERR_CUDA, "cb_sample: no CUDA device");
    }
    // as few CTAs per row as hold it, and more while that leaves SMs idle
    int ctas = 1;
    const auto part = [&](int c) { return ((vocab + c - 1) / c + GRAIN - 1) / GRAIN * GRAIN; };
    while (ctas < MOST_CTAS && (part(ctas) > MOST_PART || ((int64_t)n_rows * ctas * 2 <= sms && part(ctas) > GRAIN))) ctas *= 2;
    const SampleArgs a{logits, row_stride, vocab, part(ctas), ctas, temperature, top_k, top_p, min_p, uniform, out_tokens, out_probs};
    const cudaError_t e = dtype == CB_BF16 ? launch_sample<bf16>(a, n_rows, ctas, (cudaStream_t)stream)
                                           : launch_sample<float>(a, n_rows, ctas, (cudaStream_t)stream);
    if (e == cudaSuccess) return CB_OK;
    cudaGetLastError();
    return fail(CB_ERR_CUDA, "cb_sample: %s", cudaGetErrorString(e));
}
