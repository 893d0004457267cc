// The next token from a row of logits: temperature, top-k, top-p, min-p and a given uniform number (cb_sample).
//
// With weights w_i = 2^((x_i - max) log2(e) / T), in descending order of x (ties to the lower token): top-k keeps the first k,
// top-p of those the ones before which the weights sum to less than p of theirs, min-p of those w_i >= p_min w_max.  The
// token is the lowest i whose kept weights up to i pass u times their sum.
//
// The result is a whole number, so sums have to be where the exact ones are: at a vocabulary of 128K a border that is off by
// 2^-24 of the sum would pick a neighbour in one row of a hundred.  Weights are therefore 64-bit integers, in units of
// 2^-44 to 2^-45 of the largest, and their sums are exact and independent of the order of adding.  A weight is good to
// 2^-31 of itself: x / T as a sum of two fp32 numbers, its integer part in 256ths by rounding, 2^(j / 256) from a table of
// 32-bit integers, and 2^r - 1 for the rest (|r| <= 2^-9) by three terms of the series, all in fp32 and one wide integer product.
// A weight below 2^-45 of the largest is 0.
//
// A row is a cluster's, each of whose CTAs has a part of it.  Only the first pass over a row meets HBM: the rows under way fit in
// L2, so that passes read them there again, and CTAs need little shared memory and are many (held in shared memory, 64 rows of
// 128K came in two waves of clusters: 32 us without a filter, 20 this way).  What a pass finds out is left in shared memory for all
// CTAs of the cluster, and each works out the same next step from it.
//   few candidates   With c CTAs, at least k values reach the smallest of their ceil(k / c)-th largest thread maxima, and hardly
//                    more than twice as many do.  They go to the first CTA, which compares each with each and draws; more of them (or all
//                    that top-k leaves) are listed in shared memory first, and what follows reads the lists.
//   top-p            sums all weights, and their upper bits by steps of 2^(1 / 16), which leaves a window of a step or two where the sum can
//                    cross.  What reaches it is weighed by whole warps; the window's items are listed, and what lies above them is
//                    summed by warp.  Few items down to the window's end are candidates as above.
//   thresholds       else: the items' counts (top-p: weights, as three words of 16 bits) over equal steps from the largest value down, the step
//                    in which the sum crosses, and the items of that step one by one; a step with too many of them is divided again, and
//                    equal values are counted off in the tokens' order.
//   the token        the kept weights' sums by warp, then the warp's part by the CTA's warps, then a warp's items in their order.
//
// Vocabulary of 128256 in fp32 on the device: 1 row 10 us without a filter, 13 with top-k 50 and top-p, 16 with top-p; 64 rows 21, 18 (top-k),
// 47 to 58 (top-p).  Bound by the instructions of the exact weights (94 per logit with top-p, issue slots half busy) and by the passes'
// latencies with a barrier of the cluster each; HBM sees a row once (33 MB for 64 rows: 4.8 us).
#include <cstdarg>
#include <cstdio>

#include "cb_ptx.cuh"

using namespace cb;

namespace {

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int BINS = THREADS;            // a thread per bin where they are summed
constexpr int CAP = 256;                 // items that are compared each with each
constexpr int MOST_K = 128;              // top-k up to which there are few candidates
constexpr int LISTED = 8192, PER_WARP = LISTED / WARPS;          // candidates that a CTA, and a warp of it, may list
constexpr int WAITING = 160;             // of a warp's, how many may wait to be looked at: less than 32, and four for each lane
constexpr int DYNAMIC = (LISTED + WARPS * WAITING) * 6;          // values, and places in the part
constexpr int MOST_CTAS = 8;
constexpr int MOST_PART = 65536;         // places of a CTA: 16 bits in its list, and see the histograms
static_assert(CB_SAMPLE_MAX_VOCAB + 3 <= MOST_PART * MOST_CTAS && MOST_PART % (4 * THREADS) == 0, "the largest vocabulary");
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
    int vocab, part, ctas;               // part: elements of a row per CTA; CTAs per row
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
    unsigned low;                        // key of the smallest of its threads' maxima
    unsigned bound;                      // key of its share of the top-k's lower bound
    unsigned hist[2][4][BINS];           // counts, and weights in words of 16 bits; two buffers
    unsigned long long mass[2][BINS];    // those as one
    unsigned long long over[2], rest[2]; // weights above the window, and of all
    unsigned found[2], low_of[2], high_of[2];      // items of the step: how many, keys of the smallest and the largest value
    unsigned listed[2];
    Item list[2][CAP];
    int tie;                             // the token at which equal values are cut off
    unsigned full;                       // a warp's list has overflowed
    unsigned long long warp_sum[WARPS];
    // of the CTA
    unsigned long long over_warp[WARPS];           // weights above the window, by warp
    unsigned long long scan[WARPS];
    int bin, items, first, last;
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

__device__ __forceinline__ unsigned long long warp_sum64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// a value of every CTA: lane r has rank r's (lanes behind the last: `none`)
__device__ __forceinline__ unsigned of_all(const unsigned* p, int ctas, unsigned none) {
    const int lane = threadIdx.x & 31;
    return lane < ctas ? ld_cluster(of_rank(p, lane)) : none;
}
__device__ __forceinline__ unsigned long long of_all(const unsigned long long* p, int ctas) {
    const int lane = threadIdx.x & 31;
    return lane < ctas ? ld_cluster64(of_rank(p, lane)) : 0ull;
}
// the sum over all CTAs
template <typename V> __device__ __forceinline__ unsigned long long sum_of_all(const V* p, int ctas) {
    unsigned long long v[MOST_CTAS], sum = 0;
#pragma unroll
    for (int r = 0; r < MOST_CTAS; ++r) {                        // all under way together
        if constexpr (sizeof(V) == 8) v[r] = r < ctas ? ld_cluster64(of_rank(p, r)) : 0ull;
        else v[r] = r < ctas ? ld_cluster(of_rank(p, r)) : 0u;
    }
#pragma unroll
    for (int r = 0; r < MOST_CTAS; ++r) sum += v[r];
    return sum;
}
__device__ __forceinline__ unsigned long long total_of_all(const unsigned long long* p, int ctas) { return warp_sum64(of_all(p, ctas)); }
// adds to a 64-bit word in shared memory by its halves
__device__ __forceinline__ void add64(unsigned long long* to, unsigned long long v) {
    unsigned* w = reinterpret_cast<unsigned*>(to);
    const unsigned lo = (unsigned)v, was = atomicAdd(w, lo), hi = (unsigned)(v >> 32) + (was + lo < was);
    if (hi) atomicAdd(w + 1, hi);
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
    const unsigned long long sums = warp_scan64(lane < WARPS ? sm[lane] : 0ull);
    total = shfl64(sums, 31);
    const unsigned long long before = shfl64(sums, warp > 0 ? warp - 1 : 0);
    return warp > 0 ? v + before : v;
}

// Weights of a row: 2^(x t) in units of 2^-44 of the power of two at or below the largest, t = log2(e) / T.
struct Weigh {
    float t, rest;                       // 256 t as a sum
    float lowest;                        // a value whose weight is 0 and stands for all lower ones (and for NaN)
    int base;                            // `bits` >> 8 from which a weight is a product shifted by nothing
    const unsigned* power;
    // 256 x t rounded to a whole number k, as the bits of MAGIC + k
    __device__ __forceinline__ int bits(float x) const { return __float_as_int(fmaf(fmaxf(x, lowest), t, MAGIC)); }
    // a weight as a product of 2^62 .. 2^63, to be shifted by 18 .. 63
    __device__ __forceinline__ unsigned long long product(float x, int b) const {            // b: its bits
        x = fmaxf(x, lowest);
        const float r = fmaf(x, rest, fmaf(x, t, -(__int_as_float(b) - MAGIC)));             // in 256ths, |r| <= 1 / 2
        // (2^(r / 256) - 1) 2^31 by the series: (ln 2 / 256)^n / n!
        const float v = fmaf(r, fmaf(r, fmaf(r, 7.1045254f, 7871.7417f), 5814540.f), MAGIC);
        return (unsigned long long)power[b & 255] * ((unsigned)(__float_as_int(v) - MAGIC_BITS) + 0x80000000u);
    }
    __device__ __forceinline__ unsigned long long operator()(float x, int b) const { return product(x, b) >> (base - (b >> 8)); }
    __device__ __forceinline__ unsigned long long operator()(float x) const { return (*this)(x, bits(x)); }
    // a sum of products, in units of 2^48, as a sum of weights
    __device__ __forceinline__ unsigned long long of_sum(unsigned long long sum, int b) const {
        const int s = base - (b >> 8) - 48;
        return s <= 0 ? sum << -s : s < 64 ? sum >> s : 0ull;
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

__device__ __forceinline__ float4 four_of(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 four_of(const bf16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}

// A row and this CTA's part of it.  Places are tokens counted from the last 16 (8) bytes boundary at or before the row's first:
// place j + off is token j, and vectors of four places are aligned.
template <typename T> struct Row {
    const T* x;                          // token 0
    int vocab, off;
    int part, first, ctas, rank;         // places of this CTA: first .. first + part - 1
    int start;                           // token of its first place
    // or the part's candidates in the tokens' order, when they have been listed: places are those of the list
    const float* values;
    const unsigned short* places;        // from the part's first place on
    // Rows whose values stand for others.  Infinities share all the weight: they become 0, all others -inf.  Where the largest is thousands
    // of temperatures from 0, values are taken less the largest (what has weight lies so near to it that the difference is exact), and at
    // the very lowest temperatures times 2^32, so that 1 / T stays within fp32.
    bool special, infinite;
    float less, times;
    __device__ __forceinline__ float see(float v) const {
        return !special ? v : !infinite ? (v - less) * times : v == INFINITY ? 0.f : -INFINITY;
    }
    __device__ __forceinline__ float4 raw(int place) const {     // four from here on; -inf where there is no token
        if (values) return *reinterpret_cast<const float4*>(values + place);
        const int j = place - off;
        if (j >= 0 && j + 4 <= vocab) return four_of(x + j);
        const auto one = [&](int k) { return k >= 0 && k < vocab ? to_f(x[k]) : -INFINITY; };
        return make_float4(one(j), one(j + 1), one(j + 2), one(j + 3));
    }
    __device__ __forceinline__ void tokens_of(int place, int* j) const {
        if (places) {
            const uint2 v = *reinterpret_cast<const uint2*>(places + place);
            j[0] = start + (v.x & 0xffffu);
            j[1] = start + (v.x >> 16);
            j[2] = start + (v.y & 0xffffu);
            j[3] = start + (v.y >> 16);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) j[k] = place - off + k;
        }
    }
    // f(four values, the place of the first) for the places of [from, from + n) that this thread of a warp has, n a multiple of
    // 128: in the tokens' order within a step of the warp, all lanes together.  Two vectors are under way beside the one that
    // is worked on (a third made nothing faster).
    template <typename F> __device__ __forceinline__ void each_of(int from, int n, F f) const {
        const int end = from + n;
        int p = from + (threadIdx.x & 31) * 4;
        const auto load = [&](int q) { return q < end ? raw(q) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); };
        float4 v0 = load(p), v1 = load(p + 128);
#pragma unroll 1
        for (; p < end; p += 128) {
            float v[4] = {v0.x, v0.y, v0.z, v0.w};
            v0 = v1;
            v1 = load(p + 256);
            if (special) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = see(v[k]);
            }
            f(v, p);
        }
    }
    template <typename F> __device__ __forceinline__ void each(F f) const {
        const int per = part / WARPS;
        each_of(first + (threadIdx.x >> 5) * per, per, f);
    }
};
// whether a lane of the warp has a value from `low` on
__device__ __forceinline__ bool any_from(const float* x, float low) {
    return __any_sync(0xffffffffu, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= low);
}

// steps of equal size from `high` down over `range`
struct Steps {
    float high, up, step;
    __device__ __forceinline__ Steps(float high_, float range) : high(high_) {
        // (differences of small numbers are brought up first: 1 / range could pass fp32, and all values be in one step for ever)
        up = range < 0x1p-60f ? 0x1p100f : 1.f;
        step = range > 0.f ? (BINS - 1) / (range * up) : 0.f;
    }
    __device__ __forceinline__ int operator()(float x) const { return (int)fminf(fminf(high - x, 3.4e38f) * up * step, BINS - 1); }
};

// what ranks below make of the first CTAs' lists: which list and entry thread tid takes, and how many there are in all
struct Gathered {
    unsigned n, before, mine;            // before: in the lists of lower ranks
    int from;
    __device__ __forceinline__ Gathered(unsigned by_lane, int rank) : n(0), before(0), mine(0), from(0) {
#pragma unroll
        for (int r = 0; r < MOST_CTAS; ++r) {
            const unsigned k = __shfl_sync(0xffffffffu, by_lane, r);
            if (threadIdx.x >= n && threadIdx.x < n + k) {
                from = r;
                mine = threadIdx.x - n;
            }
            if (r < rank) before += k;
            n += k;
        }
    }
};
__device__ __forceinline__ Item remote_item(const Item* p, int rank) {
    const uint32_t at = of_rank(p, rank);
    return Item{__uint_as_float(ld_cluster(at)), (int)ld_cluster(at + 4)};
}

// Steps of weights: 2^shift 256ths of log2 each, from the largest value's down, each within an octave; a value and its weight share
// the bits they are found by.
struct Scale {
    int top, shift;                      // top: the largest value's bits >> shift
    __device__ __forceinline__ int operator()(int bits) const { return min(top - (bits >> shift), BINS - 1); }
    __device__ __forceinline__ int lowest_of(int step) const { return (top - step) << shift; }       // bits
};
// Where a search begins: the items whose step is first .. last.  It divides them into equal steps from `high` down over `range`;
// none of them lies below `low`.  What lies above sums to what the search's first level finds, of `target` to be reached.
struct Window {
    Scale scale;
    int first, last;
    float high, range, low;
    unsigned long long target;
    unsigned items;                      // in the window and above it
    bool listed;                         // the row is the list of the window's items, and what lies above weighs `over`
    unsigned long long over;
};

// The window of top-p: all weights are summed, and the upper 15 to 16 bits of their products by step, in 32 bits.  A step's weights are
// known within 2^-14 of themselves that way, and the sum must cross within the steps (mostly one) where the sum of what they are at most has
// reached the target and that of what they are at least has not.  (With counts of items in place of products a step's weights were known within
// 4.4 %: half of a row's items could lie in the window, or all below a few heavy ones, 40 rows of mixed settings 65 to 87 us.)
template <typename T>
__device__ __forceinline__ Window nucleus(const Row<T>& row, const Weigh& w, Shared& s, float m, float p, const Cut& cut, int& phase) {
    const int tid = threadIdx.x, lane = tid & 31, b = phase++ & 1;
    // weights below (1 - p) / n of the largest sum to less than 1 - p of all
    const float covers = 256.f * fminf(fmaxf(1.f - log2f(fmaxf(1.f - p, 1e-9f) / row.vocab), 1.f), 47.f);
    Window win{};
    int shift = 0;
    while ((int)covers >> shift >= BINS - 2) ++shift;
    const Scale scale{w.bits(m) >> shift, shift};
    win.scale = scale;
    s.hist[b][0][tid] = 0;
    if (tid == 0) {
        s.rest[b] = 0;
        s.first = s.last = BINS - 1;
        s.above = 0;
    }
    __syncthreads();
    unsigned long long sum = 0;
    const float from = cut.x > -INFINITY ? cut.x : w.lowest;     // (below the lowest there is no weight)
    if (cut.x == -INFINITY && w.lowest > -3.4e38f) {             // what is not kept has no weight
        row.each([&](const float* x, int) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int bits = w.bits(x[k]), at = scale.top - (bits >> scale.shift);
                const unsigned long long y = w.product(x[k], bits);
                sum += y >> (w.base - (bits >> 8));
                if (at < BINS - 1 && x[k] >= w.lowest) atomicAdd(&s.hist[b][0][at], (unsigned)(y >> 48));
            }
        });
    } else {
        row.each([&](const float* x, int place) {
            if (!any_from(x, from)) return;
            int j[4];
            row.tokens_of(place, j);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int bits = w.bits(x[k]), at = scale(bits);
                const unsigned long long y = w.product(x[k], bits);
                if (!cut.keeps(x[k], j[k])) continue;
                sum += y >> (w.base - (bits >> 8));
                if (at < BINS - 1) atomicAdd(&s.hist[b][0][at], (unsigned)(y >> 48));
            }
        });
    }
    sum = warp_sum64(sum);
    if (lane == 0 && sum) add64(&s.rest[b], sum);
    sync_cluster();
    win.target = max(ceil_of(p, total_of_all(&s.rest[b], row.ctas)), 1ull);
    // of n items at most (a value is within half of a 256th of its whole number: a factor of 1 - 2^-9 or more), each cut off by less than 1
    const unsigned long long sum_at = sum_of_all(&s.hist[b][0][tid], row.ctas);
    const int edge = scale.lowest_of(tid);
    const unsigned least = s.power[edge & 255] >> 17;
    const unsigned long long n = tid < BINS - 1 ? sum_at / (least - (least >> 9) - 2u) : 0ull;
    const unsigned long long most = n ? w.of_sum(sum_at + n, edge) + 1 : 0ull, less = w.of_sum(sum_at, edge);
    unsigned long long total;
    if (block_scan(most, s.scan, total) >= win.target) atomicMin(&s.first, tid);
    if (block_scan(less > n ? less - n : 0ull, s.scan, total) >= win.target) atomicMin(&s.last, tid);
    __syncthreads();
    win.first = s.first;
    win.last = s.last;
    const unsigned long long upto = block_scan(n, s.scan, total);
    if (tid == win.last) s.above = upto;
    __syncthreads();
    win.items = (unsigned)s.above;
    const auto value = [&](int bits) { return (float)(bits - MAGIC_BITS) / w.t; };           // about where x t 256 is that whole number
    const float bottom = value(scale.lowest_of(win.last) - 2);
    win.high = value(scale.lowest_of(win.first - 1) + 2);
    win.low = win.last == BINS - 1 ? -INFINITY : bottom - fabsf(m) * 1e-6f;
    win.range = win.high - bottom;
    return win;
}

// Lists the part's values from `from` on, in the tokens' order, a warp's share in a piece of its own; what is done then reads
// the list.  The row stays as it is where a warp of the cluster has more of them than its piece holds.  The first CAP of a CTA
// stand in s.list[b] too; returns how many there are in the cluster (more than CAP: or more than that).
template <typename T> __device__ __forceinline__ unsigned list_from(Row<T>& row, Shared& s, float from, float* values, unsigned short* places, int b) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, base = warp * PER_WARP;
    if (threadIdx.x == 0) s.full = s.found[b] = 0;
    __syncthreads();
    int n = 0;
    row.each([&](const float* x, int place) {
        if (!any_from(x, from)) return;
        int at = n;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const unsigned votes = __ballot_sync(0xffffffffu, x[k] >= from);
            at += __popc(votes & ((1u << lane) - 1u));
            n += __popc(votes);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (!(x[k] >= from)) continue;
            if (at < PER_WARP) {
                values[base + at] = x[k];
                places[base + at] = (unsigned short)(place - row.first + k);
            }
            ++at;
            if (s.found[b] <= CAP) {                   // (a look at the count spares the additions behind)
                const unsigned i = atomicAdd(&s.found[b], 1u);
                if (i < CAP) s.list[b][i] = Item{x[k], place - row.off + k};
            }
        }
    });
    for (int i = n + lane; i < PER_WARP; i += 32) values[base + i] = -INFINITY;
    if (n > PER_WARP && lane == 0) s.full = 1;
    sync_cluster();
    if (__any_sync(0xffffffffu, of_all(&s.full, row.ctas, 0u))) return CAP + 1;
    row.values = values;
    row.places = places;
    row.part = LISTED;
    row.first = 0;
    row.special = false;
    return __reduce_add_sync(0xffffffffu, of_all(&s.found[b], row.ctas, 0u));
}

// For a wide nucleus: sums the weights above the window, by warp, and lists the window's items, which are few in any case; `use`
// becomes that list.  False (and `use` as it was) where a warp's piece does not hold its share.
template <typename T>
__device__ __forceinline__ bool list_window(const Row<T>& row, Row<T>& use, const Weigh& w, Shared& s, Window& win, const Cut& cut, float* values,
                                            unsigned short* places, float* waiting, int b) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, base = warp * PER_WARP;
    if (threadIdx.x == 0) {
        s.full = 0;
        s.over[b] = 0;
    }
    __syncthreads();
    // What may be kept is brought together first, in the tokens' order, and looked at by whole warps.
    float* wait = waiting + warp * WAITING;
    unsigned short* wait_at = places + LISTED + warp * WAITING;
    int n = 0, waits = 0;
    unsigned long long over = 0;
    const auto look = [&](int from, int k) {           // at k of them
        const Item v = lane < k ? Item{wait[from + lane], wait_at[from + lane]} : Item{-INFINITY, 0};
        const int bits = w.bits(v.x), of_weight = win.scale(bits);
        const bool keep = lane < k && cut.keeps(v.x, row.start + v.i);
        if (keep && of_weight < win.first) over += w(v.x, bits);
        const bool in = keep && of_weight >= win.first && of_weight <= win.last;
        const unsigned votes = __ballot_sync(0xffffffffu, in);
        const int at = n + __popc(votes & ((1u << lane) - 1u));
        if (in && at < PER_WARP) {
            values[base + at] = v.x;
            places[base + at] = (unsigned short)v.i;
        }
        n += __popc(votes);
    };
    row.each([&](const float* x, int place) {
        if (!any_from(x, win.low)) return;
        int at = waits;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const unsigned votes = __ballot_sync(0xffffffffu, x[k] >= win.low);
            at += __popc(votes & ((1u << lane) - 1u));
            waits += __popc(votes);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (x[k] >= win.low) {
                wait[at] = x[k];
                wait_at[at++] = (unsigned short)(place - row.first + k);
            }
        __syncwarp();
        if (waits < 32) return;
        int done = 0;
#pragma unroll 1
        for (; waits - done >= 32; done += 32) look(done, 32);
        waits -= done;
        const Item last = lane < waits ? Item{wait[done + lane], wait_at[done + lane]} : Item{0.f, 0};
        __syncwarp();
        if (lane < waits) {
            wait[lane] = last.x;
            wait_at[lane] = (unsigned short)last.i;
        }
        __syncwarp();
    });
    if (waits > 0) look(0, waits);
    __syncwarp();
    for (int i = n + lane; i < PER_WARP; i += 32) values[base + i] = -INFINITY;
    over = warp_sum64(over);
    if (lane == 0) {
        s.over_warp[warp] = over;
        if (over) add64(&s.over[b], over);
        if (n > PER_WARP) s.full = 1;
    }
    sync_cluster();
    if (__any_sync(0xffffffffu, of_all(&s.full, row.ctas, 0u))) return false;
    win.over = total_of_all(&s.over[b], row.ctas);
    win.listed = true;
    use.values = values;
    use.places = places;
    use.part = LISTED;
    use.first = 0;
    use.special = false;
    return true;
}

// Lowers the cut to the first kept item, in descending order, at which the sum of counts (MASS: of weights) reaches the target.
// All CTAs of the cluster come to the same cut.  `phase` alternates the buffers that others read: one is written again only
// when all have passed the next barrier of the cluster.
template <bool MASS, typename T>
__device__ __forceinline__ void select(const Row<T>& row, const Weigh& w, Shared& s, const Window& win, Cut& cut, int& phase) {
    const int tid = threadIdx.x, lane = tid & 31;
    float high = win.high, low = win.low, range = win.range;
    unsigned long long above = 0;
    const unsigned long long target = win.target;
    // The largest and the smallest value of a level never share a step and a step is at most 1 / 510 of its level's range, so
    // that 31 levels lead from the largest difference of two fp32 numbers to the smallest.
    for (int level = 0; level < 40; ++level) {
        const int b = phase++ & 1;
        const Steps step_of(high, range);
        // -1: not of this level; -2: above the window
        const auto step = [&](float x, int j, int at) {
            if (!cut.keeps(x, j)) return -1;
            if (level == 0) {
                if (MASS && !win.listed) {
                    if (at < win.first) return -2;
                    if (at > win.last) return -1;
                }
            } else if (!(x <= high && x >= low)) {
                return -1;
            }
            return max(step_of(x), 0);
        };
        for (int k = 0; k < (MASS ? 4 : 1); ++k) s.hist[b][k][tid] = 0;
        if (tid == 0) {
            s.over[b] = s.rest[b] = 0;
            s.found[b] = s.listed[b] = 0;
            s.low_of[b] = 0xffffffffu;
            s.high_of[b] = 0;
        }
        __syncthreads();
        unsigned long long over = 0;
        row.each([&](const float* x, int place) {
            if (!any_from(x, low)) return;
            int j[4];
            row.tokens_of(place, j);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                unsigned long long y = 0;
                int of_weight = 0;
                if constexpr (MASS) {
                    const int bits = w.bits(x[k]);
                    of_weight = win.scale(bits);
                    y = w(x[k], bits);
                    const bool above_it = level == 0 && !win.listed && of_weight < win.first;
                    over += above_it && cut.keeps(x[k], j[k]) ? y : 0ull;
                    if (above_it) continue;
                }
                const int at = step(x[k], j[k], of_weight);
                if (at < 0) continue;
                if (MASS || at < BINS - 1) atomicAdd(&s.hist[b][0][at], 1u);
                if constexpr (MASS) {              // (a part has 2^16 items at most: no word overflows)
                    atomicAdd(&s.hist[b][1][at], (unsigned)y & 0xffffu);
                    atomicAdd(&s.hist[b][2][at], (unsigned)(y >> 16) & 0xffffu);
                    atomicAdd(&s.hist[b][3][at], (unsigned)(y >> 32));
                }
            }
        });
        if constexpr (MASS) {
            over = warp_sum64(over);
            if (lane == 0 && over) add64(&s.over[b], over);
            if (lane == 0 && level == 0 && !win.listed) s.over_warp[tid >> 5] = over;
        }
        if constexpr (MASS) {                          // a step's three words as one
            __syncthreads();
            s.mass[b][tid] = s.hist[b][1][tid] + ((unsigned long long)s.hist[b][2][tid] << 16) + ((unsigned long long)s.hist[b][3][tid] << 32);
        }
        sync_cluster();
        // (counts: the last step, which holds whatever lies below, is not counted)
        const unsigned long long items = !MASS && tid == BINS - 1 ? 1ull << 32 : sum_of_all(&s.hist[b][0][tid], row.ctas);
        unsigned long long here = items;
        if constexpr (MASS) {
            here = sum_of_all(&s.mass[b][tid], row.ctas);
            if (level == 0) above = win.listed ? win.over : total_of_all(&s.over[b], row.ctas);
        }
        unsigned long long total;
        const unsigned long long upto = above + block_scan(here, s.scan, total);
        if (upto - here < target && target <= upto) {
            s.bin = tid;
            s.above = upto - here;
            s.items = items > CAP ? CAP + 1 : (int)items;
        }
        __syncthreads();
        const int bin = s.bin;
        const bool few = s.items <= CAP;
        above = s.above;
        // the step's items
        float least = INFINITY, largest = -INFINITY;
        unsigned count = 0;
        // (values that may be in the step; the last one reaches to the window's end, and a step is off by its rounding)
        const float size = range / (BINS - 1), margin = fabsf(high) * 1e-6f;
        const bool narrow = range > 0x1p-100f && range < 0x1p100f;
        const float no_more = narrow ? high - (bin - 0.01f) * size + margin : INFINITY;
        const float no_less = narrow && bin < BINS - 1 ? fmaxf(high - (bin + 1.01f) * size - margin, low) : low;
        row.each([&](const float* x, int place) {
            bool in = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) in |= x[k] >= no_less && (bin == 0 || x[k] <= no_more);
            if (!__any_sync(0xffffffffu, in)) return;
            int j[4];
            row.tokens_of(place, j);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (!(x[k] >= no_less) || step(x[k], j[k], MASS && level == 0 ? win.scale(w.bits(x[k])) : 0) != bin) continue;
                ++count;
                least = fminf(least, x[k]);
                largest = fmaxf(largest, x[k]);
                if (few) s.list[b][min(atomicAdd(&s.listed[b], 1u), CAP - 1u)] = Item{x[k], j[k]};
            }
        });
        count = __reduce_add_sync(0xffffffffu, count);
        const unsigned lo = __reduce_min_sync(0xffffffffu, key_of(least + 0.f)), hi = __reduce_max_sync(0xffffffffu, key_of(largest + 0.f));
        if (lane == 0 && count) {                      // (-0 counts as 0)
            atomicAdd(&s.found[b], count);
            atomicMin(&s.low_of[b], lo);
            atomicMax(&s.high_of[b], hi);
        }
        sync_cluster();
        const unsigned mine_n = of_all(&s.found[b], row.ctas, 0u);               // by lane: of each rank
        const unsigned lo_key = __reduce_min_sync(0xffffffffu, of_all(&s.low_of[b], row.ctas, 0xffffffffu));
        const unsigned hi_key = __reduce_max_sync(0xffffffffu, of_all(&s.high_of[b], row.ctas, 0u));
        const Gathered g(mine_n, row.rank);
        const unsigned n = g.n, before = g.before;
        if (!MASS && above + n < target) return;       // fewer items than top-k keeps
        if (few) {
            if (tid < (int)n) {
                const Item it = remote_item(&s.list[b][g.mine], g.from);
                s.joined[tid] = it;
                s.weight[tid] = MASS ? w(it.x) : 1ull;
            }
            __syncthreads();
            if (tid < (int)n) {
                const Item it = s.joined[tid];
                unsigned long long sum = above;
#pragma unroll 8
                for (int k = 0; k < (int)n; ++k) {
                    const Item o = s.joined[k];
                    const unsigned long long z = s.weight[k];
                    sum += o.x > it.x || (o.x == it.x && o.i < it.i) ? z : 0ull;
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
                int mine = 0;
                row.each([&](const float* x, int place) {
                    int j[4];
                    row.tokens_of(place, j);
#pragma unroll
                    for (int k = 0; k < 4; ++k) mine += x[k] == high && cut.keeps(x[k], j[k]);
                });
                const unsigned long long warps = __reduce_add_sync(0xffffffffu, (unsigned)mine);
                unsigned long long all;
                const unsigned long long end = before + block_scan(lane == 31 ? warps : 0ull, s.scan, all);
                // (the sum up to lane 31 of this warp; other lanes have what stands before the warp)
                const unsigned long long begin = shfl64(end, 0);
                if (keep > begin && keep <= begin + warps) {
                    unsigned left = (unsigned)(keep - begin);
                    const int per = row.part / WARPS, p0 = row.first + (tid >> 5) * per;
                    for (int p = p0; p < p0 + per; p += 128) {
                        const float4 v = row.raw(p + lane * 4);
                        const float x[4] = {row.see(v.x), row.see(v.y), row.see(v.z), row.see(v.w)};
                        int j[4];
                        row.tokens_of(p + lane * 4, j);
                        unsigned own = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) own += x[k] == high && cut.keeps(high, j[k]);
                        const unsigned stop = (unsigned)warp_scan64(own);
                        if (stop - own < left && left <= stop) {
                            unsigned at = stop - own;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (x[k] == high && cut.keeps(high, j[k]) && ++at == left) s.tie = j[k];
                        }
                        const unsigned all_of = __shfl_sync(0xffffffffu, stop, 31);
                        if (all_of >= left) break;
                        left -= all_of;
                    }
                }
            }
            sync_cluster();
            int owner = 0;
            unsigned upto_r = 0;
#pragma unroll
            for (int r = 0; r < MOST_CTAS; ++r) {
                const unsigned k = __shfl_sync(0xffffffffu, mine_n, r);
                if (keep > upto_r && keep <= upto_r + k) owner = r;
                upto_r += k;
            }
            cut = Cut{high, (int)ld_cluster(of_rank(&s.tie, owner))};
            return;
        }
        __syncthreads();                               // bin, above and the scan's sums are written again
    }
}

// y / total for 64-bit integers, rounded once (nearly): both as sums of two fp32 numbers
__device__ __forceinline__ float share_of(unsigned long long y, unsigned long long total) {
    const float yh = (float)y, th = (float)total;
    const float yl = (float)(long long)(y - (unsigned long long)yh), tl = (float)(long long)(total - (unsigned long long)th);
    const float q = yh / th;
    return q + ((fmaf(-q, th, yh) + yl) - q * tl) / th;
}

// The first CTA draws from the items in all CTAs' lists, which hold every item above their last: those that the cut keeps, of
// them the first top_k, of them the ones before which the weights sum to less than `target` (0: top_p of theirs).
__device__ __forceinline__ void draw_listed(const Weigh& w, Shared& s, int b, const Gathered& g, float m, const Cut& cut, int top_k, float top_p,
                                            unsigned long long target_p, float min_p, float u, const SampleArgs& a, int r_out) {
    const int tid = threadIdx.x, n = (int)g.n;
    Item it{0.f, 0};
    unsigned long long y = 0;
    bool keep = false;
    if (tid < n) {
        it = remote_item(&s.list[b][g.mine], g.from);
        keep = cut.keeps(it.x, it.i);
        y = keep ? w(it.x) : 0ull;
        s.joined[tid] = it;
        s.weight[tid] = y;
    }
    __syncthreads();
    int ahead = 0;
    unsigned long long before = 0;
    if (tid < n) {
#pragma unroll 8
        for (int k = 0; k < n; ++k) {
            const Item o = s.joined[k];
            const unsigned long long z = s.weight[k];
            const bool first = o.x > it.x || (o.x == it.x && o.i < it.i);
            ahead += first;
            before += first ? z : 0ull;
        }
    }
    keep = keep && ahead < top_k;
    unsigned long long sum;
    if (target_p == 0 && top_p < 1.f) {
        block_scan(keep ? y : 0ull, s.scan, sum);
        target_p = max(ceil_of(top_p, sum), 1ull);
    }
    if (target_p > 0) keep = keep && before < target_p;
    if (min_p > 0.f) {
        const unsigned long long most = w(m);
        keep = keep && y >= (min_p >= 1.f ? most : ceil_of(min_p, most));
    }
    __syncthreads();                                   // every weight has been read
    if (tid < n) s.weight[tid] = keep ? y : 0ull;
    block_scan(keep ? y : 0ull, s.scan, sum);
    const unsigned long long target = u >= 1.f ? sum - 1 : floor_of(u, sum);
    if (!keep) return;
    before = 0;
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
        const unsigned long long z = s.weight[k];
        before += s.joined[k].i < it.i ? z : 0ull;
    }
    if (before <= target && target < before + y) {
        a.out_tokens[r_out] = it.i;
        if (a.out_probs) a.out_probs[r_out] = share_of(y, sum);
    }
}

// The part's items from `from` on into s.list[b], as far as they fit; how many there are in the cluster.  `own`: the largest of
// the thread's values in the row, or infinity where it is not known (a thread whose largest lies below has none).
template <typename T>
__device__ __forceinline__ unsigned collect(const Row<T>& row, Shared& s, float from, float own, int b) {
    const int tid = threadIdx.x;
    if (tid == 0) s.found[b] = 0;
    __syncthreads();
    if (own >= from) {
        const int per = row.part / WARPS, end = row.first + (tid >> 5) * per + per;
        for (int p = end - per + (tid & 31) * 4; p < end; p += 128) {
            const float4 v = row.raw(p);
            const float x[4] = {row.see(v.x), row.see(v.y), row.see(v.z), row.see(v.w)};
            if (!(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= from)) continue;
            int j[4];
            row.tokens_of(p, j);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (!(x[k] >= from) || s.found[b] > CAP) continue;
                const unsigned n = atomicAdd(&s.found[b], 1u);
                if (n < CAP) s.list[b][n] = Item{x[k], j[k]};
            }
        }
    }
    sync_cluster();
    return __reduce_add_sync(0xffffffffu, of_all(&s.found[b], row.ctas, 0u));
}

// key of the j-th largest of the threads' maxima, or less; 0 where there are fewer
__device__ __forceinline__ unsigned jth_largest(Shared& s, float own, int j) {
    const int tid = threadIdx.x;
    s.hist[1][0][tid] = 0;                             // (not yet anyone's)
    if (tid == 0) s.bound = 0xffffffffu;
    const float most = of_key((unsigned)(s.best >> 32));
    const float least = s.low == 0xffffffffu ? most : of_key(s.low);
    __syncthreads();
    const Steps step_of(most, fminf(most - least, 3.4e38f));
    const bool some = own > -INFINITY;
    const int bin = some && most < INFINITY ? step_of(own) : 0;
    if (some) atomicAdd(&s.hist[1][0][bin], 1u);
    __syncthreads();
    unsigned long long total;
    const unsigned long long here = s.hist[1][0][tid], upto = block_scan(here, s.scan, total);
    if (upto - here < (unsigned)j && (unsigned)j <= upto) s.bin = tid;
    __syncthreads();
    if (total < (unsigned)j) return 0;
    const unsigned l = __reduce_min_sync(0xffffffffu, some && bin <= s.bin ? key_of(own + 0.f) : 0xffffffffu);
    if ((tid & 31) == 0) atomicMin(&s.bound, l);
    __syncthreads();
    return s.bound;
}

template <typename T>
__global__ void __launch_bounds__(THREADS, 2) sample_kernel(const SampleArgs a) {
    __shared__ Shared s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ctas = a.ctas, rank = (int)ptx::cluster_rank();
    const int r = blockIdx.x / ctas;
    if (tid < 256) s.power[tid] = kPowers.of[tid];
    if (tid == 0) {
        s.best = 0;
        s.low = 0xffffffffu;
    }
    const float temperature = a.temperature ? a.temperature[r] : 1.f;
    const int top_k = a.top_k ? a.top_k[r] : 0;
    const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f, u = a.uniform[r];
    const T* src = (const T*)a.logits + (int64_t)r * a.stride;
    Row<T> row{src, a.vocab, (int)((uintptr_t)src / sizeof(T) & 3), a.part, rank * a.part, ctas, rank, 0, nullptr, nullptr, false, false, 0.f, 1.f};

    // the largest value and its first token (a NaN is never larger)
    float own = -INFINITY;                             // of this thread's values
    int own_i = 0x7fffffff;
    {
        constexpr int AHEAD = 4;                       // vectors under way
        const int per = a.part / WARPS, end = row.first + warp * per + per;
        int own_p = -1;                                // the first place of the vector that has it
#pragma unroll 1
        for (int p = end - per + lane * 4; p < end; p += AHEAD * 128) {
            float4 v[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) v[k] = p + k * 128 < end ? row.raw(p + k * 128) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const float x = fmaxf(fmaxf(v[k].x, v[k].y), fmaxf(v[k].z, v[k].w));
                if (x > own) {
                    own = x;
                    own_p = p + k * 128;
                }
            }
        }
        if (own_p >= 0) {
            const float4 v = row.raw(own_p);
            own_i = own_p - row.off + (v.x == own ? 0 : v.y == own ? 1 : v.z == own ? 2 : 3);
        }
    }
    __syncthreads();
    {
        const unsigned k = key_of(own + 0.f), top = __reduce_max_sync(0xffffffffu, k);       // (-0 counts as 0)
        const unsigned i = __reduce_min_sync(0xffffffffu, k == top ? (unsigned)own_i : 0xffffffffu);
        const unsigned l = __reduce_min_sync(0xffffffffu, own > -INFINITY ? k : 0xffffffffu);
        if (lane == 0) {
            atomicMax(&s.best, ((unsigned long long)top << 32) | ~i);
            atomicMin(&s.low, l);
        }
    }
    const bool greedy = !(temperature >= 1.1754944e-38f), cuts = top_k > 0 && top_k < a.vocab;
    // (a share of the threads' maxima bounds the k-th value while it is not all of them)
    const int share = (top_k + ctas - 1) / ctas;
    const bool few = cuts && share <= THREADS - THREADS / 8 && !greedy;
    if (few) {
        __syncthreads();
        const unsigned k = jth_largest(s, own, share);
        if (tid == 0) s.bound = k;
    }
    sync_cluster();
    const unsigned long long bests = of_all(&s.best, ctas);
    const unsigned top = __reduce_max_sync(0xffffffffu, (unsigned)(bests >> 32));
    const unsigned best_i = ~__reduce_max_sync(0xffffffffu, (unsigned)(bests >> 32) == top ? (unsigned)bests : 0u);
    float m = of_key(top), low = of_key(__reduce_min_sync(0xffffffffu, of_all(&s.low, ctas, 0xffffffffu)));
    if (m == -INFINITY || greedy) {                    // no token, or the most likely one
        if (rank == 0 && tid == 0) {
            a.out_tokens[r] = m == -INFINITY ? -1 : (int)best_i;
            if (a.out_probs) a.out_probs[r] = m == -INFINITY ? 0.f : 1.f;
        }
        sync_cluster();                                // no CTA exits while another reads its shared memory
        return;
    }
    unsigned bound = few ? __reduce_min_sync(0xffffffffu, of_all(&s.bound, ctas, 0xffffffffu)) : 0u;     // 0: a CTA has fewer values
    Weigh w;
    {
        float T1 = fminf(temperature, 3.4e38f);
        const bool far = !(fabsf(m) * (1.442695f / T1) < 8192.f);
        if (m == INFINITY) {
            row.special = row.infinite = true;
            m = low = 0.f;
            bound = 0;
        } else if (far || T1 < 0x1p-100f) {
            row.special = true;
            row.less = far ? m : 0.f;                  // (nearer to 0 the difference would be rounded)
            row.times = T1 < 0x1p-100f ? 0x1p32f : 1.f;
            T1 *= row.times;
            own = row.see(own);
            low = row.see(low);
            m = row.see(m);
        }
        // log2(e) = 1.44269502 + 1.92596299e-8 (times 256 before it is divided: at the highest temperatures 1 / T1 is below the normal numbers)
        w.t = 256.f * 1.44269502f / T1;
        w.rest = (fmaf(-w.t, T1, 256.f * 1.44269502f) + 256.f * 1.92596299e-8f) / T1;
        w.power = s.power;
        w.lowest = -INFINITY;
        const int top8 = (w.bits(m) - MAGIC_BITS) >> 8;
        w.base = 18 + top8 + (MAGIC_BITS >> 8);
        w.lowest = fmaxf((top8 - 44.5f) * 256.f / w.t, -3.402823466e38f);
    }
    Cut cut{-INFINITY, -0x7fffffff - 1};               // (-inf, where there is no token among others, is not kept)
    int phase = 0;
    extern __shared__ __align__(16) float lists[];     // values [LISTED], [WARPS][WAITING]; places [LISTED], [WARPS][WAITING]
    float* waiting = lists + LISTED;
    unsigned short* places = reinterpret_cast<unsigned short*>(waiting + WARPS * WAITING);
    row.start = row.first - row.off;
    // a value below which min-p keeps nothing
    const float from_min = min_p > 0.f ? m + 256.f * (log2f(fminf(min_p, 1.f)) - 0.01f) / w.t - fabsf(m) * 1e-6f : -INFINITY;
    // where few candidates are left, the buffer they stand in; how many of them top-k keeps; what top-p's weights sum to
    int listed = -1, first_k = 0x7fffffff;
    unsigned long long target_p = 0;
    // after top-p: its window's first step, and a value above the window
    int window_first = -1;
    bool window_listed = false;
    Scale scale{};
    float below = INFINITY;
    Row<T> use = row;                                  // what is left to be looked at of it
    if (bound > 0) {
        const float from = row.see(of_key(bound));
        if (top_k <= MOST_K) {
            listed = phase++ & 1;
            if (collect(row, s, from, own, listed) > CAP) listed = -1;
        }
        if (listed < 0) {
            listed = phase++ & 1;
            if (list_from(row, s, from, lists, places, listed) > CAP) listed = -1;
        }
        if (listed >= 0) first_k = top_k;
    }
    if (listed < 0 && cuts) {
        // As many items as there are threads reach the smallest of the threads' maxima, and below 2^-47 of the largest weight
        // there is none to cut.
        const float range = fminf(fminf(m - low, 47.f * 256.f / w.t), 3.4e38f);
        select<false>(row, w, s, Window{Scale{}, 0, 0, m, range, -INFINITY, (unsigned long long)top_k, 0u, false, 0ull}, cut, phase);
    }
    if (listed < 0 && top_p < 1.f) {
        use = row;
        Window win = nucleus(row, w, s, m, top_p, cut, phase);
        // (of what lies below the window, or below min-p, nothing is kept)
        if (from_min > win.low || (win.low > -INFINITY && win.items <= CAP)) {
            listed = phase++ & 1;
            if (collect(row, s, fmaxf(win.low, from_min), INFINITY, listed) <= CAP) target_p = win.target; else listed = -1;
        }
        if (listed < 0 && win.low > -INFINITY && !row.values) {
            window_listed = list_window(row, use, w, s, win, cut, lists, places, waiting, phase++ & 1);
        }
        if (listed < 0) {
            select<true>(use, w, s, win, cut, phase);
            window_first = win.first;
            scale = win.scale;
            below = win.first > 0 ? win.high + fabsf(m) * 1e-6f : INFINITY;
        }
    }
    if (listed >= 0) {
        const Gathered g(of_all(&s.found[listed], ctas, 0u), rank);
        if (rank == 0) draw_listed(w, s, listed, g, m, cut, first_k, top_p, target_p, min_p, u, a, r);
        sync_cluster();
        return;
    }
    const unsigned long long least = min_p >= 1.f ? w(m) : ceil_of(min_p, w(m));

    // sums of what is kept, per warp; the warp's part in which they pass u of their sum; the token in it
    const float from = fmaxf(cut.x, from_min);         // nothing below is kept
    // (then -inf has no weight by itself; the value below which min-p keeps nothing may have passed fp32)
    const bool all = from == -INFINITY && w.lowest > -3.4e38f && !(min_p > 0.f);
    const auto kept = [&](const float* x, int place, unsigned long long* y) {  // false: none of the warp's
        if (!all && !any_from(x, from)) return false;
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = w(x[k]);
        if (!all) {
            int j[4];
            row.tokens_of(place, j);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = cut.keeps(x[k], j[k]) && y[k] >= least ? y[k] : 0ull;
        }
        return true;
    };
    // What lies above top-p's window has been summed by warp (without min-p): only the window's weights are left.
    const auto kept_of_window = [&](const float* x, int place, unsigned long long* y) {
        bool in = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) in |= x[k] >= from && x[k] <= below;
        if (!__any_sync(0xffffffffu, in)) return false;
        int j[4];
        row.tokens_of(place, j);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int bits = w.bits(x[k]);
            y[k] = cut.keeps(x[k], j[k]) && scale(bits) >= window_first ? w(x[k], bits) : 0ull;
        }
        return true;
    };
    const auto sum_of = [&](int at, int n) {
        unsigned long long sum = 0;
        row.each_of(at, n, [&](const float* x, int place) {
            unsigned long long y[4];
            if (kept(x, place, y)) sum += (y[0] + y[1]) + (y[2] + y[3]);
        });
        return warp_sum64(sum);
    };
    const int per = row.part / WARPS;
    {
        unsigned long long sum = 0;
        if (window_listed && min_p <= 0.f) {
            use.each([&](const float* x, int place) {
                if (!any_from(x, from)) return;
                int j[4];
                use.tokens_of(place, j);
#pragma unroll
                for (int k = 0; k < 4; ++k) sum += cut.keeps(x[k], j[k]) ? w(x[k]) : 0ull;
            });
            sum = warp_sum64(sum) + s.over_warp[warp];
        } else if (window_first >= 0 && min_p <= 0.f) {
            row.each([&](const float* x, int place) {
                unsigned long long y[4];
                if (kept_of_window(x, place, y)) sum += (y[0] + y[1]) + (y[2] + y[3]);
            });
            sum = warp_sum64(sum) + s.over_warp[warp];
        } else {
            sum = sum_of(row.first + warp * per, per);
        }
        if (lane == 0) s.warp_sum[warp] = sum;
    }
    sync_cluster();
    unsigned long long total;
    const unsigned long long part = tid < ctas * WARPS ? ld_cluster64(of_rank(&s.warp_sum[tid % WARPS], tid / WARPS)) : 0ull;
    const unsigned long long upto = block_scan(part, s.scan, total);
    const unsigned long long target = u >= 1.f ? total - 1 : floor_of(u, total);
    if (upto - part <= target && target < upto) {
        s.segment = tid;
        s.above = upto - part;
    }
    __syncthreads();
    if (s.segment / WARPS == rank) {                   // in this CTA: the part again, by all its warps
        const int small = (per / 128 + WARPS - 1) / WARPS * 128, piece = row.first + s.segment % WARPS * per;
        const int at = min(warp * small, per), n = min(small, per - at);
        const unsigned long long mine = sum_of(piece + at, n), above = s.above;
        unsigned long long of_piece;
        const unsigned long long end = above + block_scan(lane == 31 ? mine : 0ull, s.scan, of_piece);
        unsigned long long before = shfl64(end, 0);    // what stands before this warp's piece
        if (before <= target && target < before + mine) {
            for (int p = piece + at; p < piece + at + n; p += 128) {
                const float4 v = row.raw(p + lane * 4);
                int j[4];
                row.tokens_of(p + lane * 4, j);
                const float x[4] = {row.see(v.x), row.see(v.y), row.see(v.z), row.see(v.w)};
                unsigned long long y[4], sum = 0;
                if (kept(x, p + lane * 4, y)) sum = (y[0] + y[1]) + (y[2] + y[3]);
                else y[0] = y[1] = y[2] = y[3] = 0ull;
                const unsigned long long stop = before + warp_scan64(sum);
                unsigned long long c = stop - sum;
                if (c <= target && target < stop) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (c <= target && target < c + y[k]) {
                            a.out_tokens[r] = j[k];
                            if (a.out_probs) a.out_probs[r] = share_of(y[k], total);
                        }
                        c += y[k];
                    }
                }
                before = shfl64(stop, 31);
                if (target < before) break;
            }
        }
    }
    sync_cluster();
}

template <typename T> cudaError_t launch_sample(const SampleArgs& a, int n_rows, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = smem_limit_once(sample_kernel<T>, DYNAMIC, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n_rows * a.ctas));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = DYNAMIC;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.ctas;
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
    // Threads of a row: as many as all rows' find room for at once (two CTAs to an SM, and fewer the larger the clusters are, which have to
    // lie together), up to a cluster of eight; a CTA more only for every 4096 tokens.  Device us of 128256 tokens with 2, 4 and 8 CTAs, without
    // a filter and with top-p: 1 row 22, 14, 10; 24 rows 23, 15, 15 and 66, 44, 40; 38 rows 23, 21, 23 and 64, 48, 52; 64 rows 23, 21, 29 and
    // 65, 59, 62; 76 rows 23, 32, 36 and 66, 68, 81.
    const auto room = [&](int c) { return (int64_t)n_rows * c <= 2 * sms - sms * c / 20; };
    const int places = vocab + 3;                      // (a row may begin up to three elements behind a boundary)
    int ctas = 1;
    while (ctas < MOST_CTAS && (places > MOST_PART * ctas || (room(2 * ctas) && vocab > 4096 * ctas))) ctas *= 2;
    const int grain = 4 * THREADS, part = ((places + ctas - 1) / ctas + grain - 1) / grain * grain;
    const SampleArgs a{logits, row_stride, vocab, part, ctas, temperature, top_k, top_p, min_p, uniform, out_tokens, out_probs};
    const cudaError_t e = dtype == CB_BF16 ? launch_sample<bf16>(a, n_rows, (cudaStream_t)stream) : launch_sample<float>(a, n_rows, (cudaStream_t)stream);
    if (e == cudaSuccess) return CB_OK;
    cudaGetLastError();
    return fail(CB_ERR_CUDA, "cb_sample: %s", cudaGetErrorString(e));
}
