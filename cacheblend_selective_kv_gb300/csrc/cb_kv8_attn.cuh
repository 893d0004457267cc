// What the two kernels of attention over the 8-bit cache share: their arguments and the list of tiles that divides the
// work.  An item is (sequence, tile of QT query rows, KV head), cut into tiles of 128 keys; the tiles of all items form one
// list, in this order, and every CTA takes an equal, contiguous piece of it.  What an item costs besides its tiles (its Q,
// its output, a pipeline that runs empty) stands in the list as places before its first tile, so that a CTA of many short
// items gets fewer of them.  An item that spans CTAs leaves a partial result per CTA, and the partial results are joined
// in their order.
#pragma once
#include <climits>

#include "cb_kv8.cuh"
#include "cb_ptx.cuh"

namespace cb {

namespace {

constexpr int TK = 128;                  // keys per tile

// What a launch computes.  Attention over a prefix that sequences share is two launches:
//   PLAIN   the rows' results over their sequence's keys
//   PREFIX  a sequence is a group's prefix, its rows are those of all the group's sequences and see all of it; their sums,
//           not divided, go to scratch with their references
//   OWN     many rows: PLAIN, and what PREFIX has left is added to a row's sums before they are divided
//   BESIDE  few rows: PLAIN, on SMs that PREFIX leaves free and at the same time; its sums go to scratch too, and a third launch
//           joins both
// or one, where reading the prefix again for each sequence costs less than the other launches:
//   JOINT   PLAIN, and a sequence's tiles begin with those of its prefix, which all its rows see
enum : int { PLAIN, PREFIX, OWN, JOINT, BESIDE };

// 16 bytes to shared memory, past L1
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

struct AttnArgs {
    Kv8Seqs q;
    Kv8Rows r;
    Kv8Attn a;
    const float* ks;                     // this layer's scales [n_pages][Hkv]
    const float* vs;
    int Hq, Hkv, G, QT;                  // QT = query rows per item
    unsigned inv_g;                      // ceil(2^16 / G): k / G for k below 2^13
    int kz;                              // z coordinate of this layer's K in the map (V is kz + 1)
    int box;                             // rows of a TMA box: min(page_size, 128)
    int ahead;                           // places before an item's first tile
    int min_places;                      // places per CTA, at least
    float* part;                         // [cta][2][NC][HD + 2] pieces of items that span CTAs
    unsigned* arrived;                   // [cta] pieces finished of the item that begins in this CTA (0 between calls)
    int* todo;                           // many rows: [cta] what the joining kernel has to do (4 ints)
    float* scores;                       // weights: scores in the exp2 domain (score_of), score_ld per column
    int score_ld;                        // max_len rounded up to TK
    float2* stats;                       // weights: [Hkv][n_q][G] (max, 1 / sum)
    unsigned* voided;                    // weights: the call's offsets decrease, nothing was computed (NULL: no query rows)
    int sms;                             // SMs that the launch is for
    // all but PLAIN
    Kv8Seqs pre;                         // JOINT: the groups' prefixes
    const int* first;                    // [groups + 1] first sequence of each group, or NULL: `per_group` each
    int per_group, groups, members;      // members: sequences
    float* side_sum;                     // [n_q][Hq][HD] of the prefix (BESIDE: of a sequence's own keys)
    float2* side_stat;                   // [n_q][Hq] reference and sum of the exponentials
    int2* pieces_of;                     // PREFIX, beside BESIDE: [n_q][Hq] where a row's sums stand
    int piece_cols, piece_ctas;          // columns of a piece, CTAs that have pieces
    const unsigned* prefix_voided;       // OWN: PREFIX has computed nothing
    unsigned* opened;                    // PREFIX, BESIDE: see open_for_beside (NULL: no BESIDE)
};

// BESIDE starts when all CTAs of PREFIX have let it, and reads what the kernels before PREFIX have written.  That those are complete
// PREFIX has waited for, which makes their writes visible to PREFIX; a release by one of its threads, before it lets BESIDE start, and an
// acquire in each CTA of BESIDE, behind which a barrier stands, pass it on.  The launch that joins both sets the word back, so that it is 0
// when a call's PREFIX starts; a CTA that reads 0 waits for all of PREFIX.
__device__ __forceinline__ void open_for_beside(const AttnArgs& p) {
    if (p.opened && blockIdx.x == 0 && threadIdx.x == 0) asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p.opened), "r"(1u) : "memory");
}
__device__ __forceinline__ void wait_beside(const AttnArgs& p) {
    unsigned open = 1u;
    if (threadIdx.x == 0) asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(open) : "l"(p.opened) : "memory");
    if (__syncthreads_or(open != 1u)) grid_dep_wait();
    asm volatile("fence.proxy.async.global;" ::: "memory");      // codes are read by TMA
}

// k / G and k % G of a column or row of an item
__device__ __forceinline__ int div_g(const AttnArgs& p, int k) { return (int)(((unsigned)k * p.inv_g) >> 16); }
__device__ __forceinline__ int mod_g(const AttnArgs& p, int k) { return k - div_g(p, k) * p.G; }

__device__ __forceinline__ float exp2_fast(float x) {          // special-function unit, about 2 ulp
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// ------------------------------------------------------------------------------------------------
// the list of tiles
// ------------------------------------------------------------------------------------------------
struct Seq {                             // one sequence: its query rows and length (-1: its offsets decrease)
    int r0, n, len;
    int pre, group;                      // JOINT: rows of its prefix, and whose they are
    template <int MODE> __device__ __forceinline__ int pre_tiles() const { return MODE == JOINT ? (pre + TK - 1) / TK : 0; }
    __device__ __forceinline__ int q_tiles(int QT) const { return (n + QT - 1) / QT; }
    // keys that the last row of query tile qt sees
    template <int MODE> __device__ __forceinline__ int visible(int qt, int QT) const {
        return MODE == PREFIX ? len : max(0, len - n + min((qt + 1) * QT, n));
    }
    template <int MODE> __device__ __forceinline__ int tiles(int qt, int QT) const { return max(1, pre_tiles<MODE>() + (visible<MODE>(qt, QT) + TK - 1) / TK); }
    // the last key that row q0 sees (PREFIX: and every other row)
    template <int MODE> __device__ __forceinline__ int position(int q0) const { return MODE == PREFIX ? len - 1 : len - n + q0; }
};
// the rows of a group: those of its sequences, which see a prefix of no rows where its length is out of range
__device__ __forceinline__ Seq group_at(const AttnArgs& p, int g) {
    const int s0 = p.first ? p.first[g] : g * p.per_group, s1 = p.first ? p.first[g + 1] : s0 + p.per_group;
    if (s0 >= 0 && s1 >= s0 && s1 <= p.members) {
        const int r0 = p.r.start ? p.r.start[s0] : s0 * p.r.each, r1 = p.r.start ? p.r.start[s1] : s1 * p.r.each;
        if (r0 >= 0 && r1 >= r0 && r1 <= p.r.n_rows) {
            const int len = kv8_len(p.q, g);
            const bool good = len >= 0 && len <= p.q.max_len;
            if (!good) atomicOr(p.q.status, ST_BAD_ROW);
            return Seq{r0, r1 - r0, good ? len : 0};
        }
    }
    atomicOr(p.q.status, ST_BAD_ROW);
    return Seq{0, 0, -1};
}
// a sequence with its prefix
__device__ __forceinline__ Seq joint_at(const AttnArgs& p, int s) {
    Seq q{0, 0, 0, 0, 0};
    int r1;
    if (!kv8_rows(p.q, p.r, s, q.r0, r1, q.len)) return Seq{0, 0, q.r0 < 0 || r1 < q.r0 || r1 > p.r.n_rows ? -1 : 0};
    q.n = r1 - q.r0;
    if (p.first) {
        if (s < p.first[0] || s >= p.first[p.groups]) return q;
        int z = p.groups - 1;                                    // the last group that begins at or before it
        while (q.group < z) {
            const int m = (q.group + z + 1) >> 1;
            if (p.first[m] <= s) q.group = m; else z = m - 1;
        }
    } else {
        q.group = s / p.per_group;
    }
    const int pre = kv8_len(p.pre, q.group);
    if (pre >= 0 && pre <= p.pre.max_len) q.pre = pre;
    else atomicOr(p.q.status, ST_BAD_ROW);
    return q;
}
// (JOINT) whether the groups' first sequences are in order
__device__ __forceinline__ bool bad_groups(const AttnArgs& p, int g) {
    const int a = p.first[g], b = p.first[g + 1];
    const bool bad = a < 0 || b < a || b > p.members;
    if (bad) atomicOr(p.q.status, ST_BAD_ROW);
    return bad;
}
template <int MODE = PLAIN> __device__ __forceinline__ Seq seq_at(const AttnArgs& p, int s) {
    if constexpr (MODE == PREFIX) return group_at(p, s);
    if constexpr (MODE == JOINT) return joint_at(p, s);
    Seq q;
    int r1;
    if (!kv8_rows(p.q, p.r, s, q.r0, r1, q.len)) return Seq{0, 0, r1 < q.r0 ? -1 : 0};
    q.n = r1 - q.r0;
    return q;
}
template <int MODE> __device__ __forceinline__ int seq_places(const AttnArgs& p, const Seq& q) {
    int t = 0;
#pragma unroll 1
    for (int qt = 0; qt < q.q_tiles(p.QT); ++qt) t += p.ahead + q.tiles<MODE>(qt, p.QT);
    return t * p.Hkv;
}

// Scores of a column (query row of the sequence x head of the group) with the keys of tile t: a tile's columns lie together,
// so that what sums over them reads one contiguous piece.
__device__ __forceinline__ float* score_of(const AttnArgs& p, const Seq& q, int g, int t, int col) {
    return p.scores + ((int64_t)g * p.r.n_rows + q.r0) * p.G * p.score_ld + ((int64_t)t * q.n * p.G + col) * TK;
}

// A tile in the list: item (s, query tile qt, g) and tile t of its nt.
template <int MODE> struct Cursor {
    int s, qt, g, t, nt;
    Seq q;
    __device__ __forceinline__ void settle(const AttnArgs& p) { nt = q.tiles<MODE>(qt, p.QT); }
    // to the first tile of the next item
    __device__ __forceinline__ void next_item(const AttnArgs& p) {
        t = 0;
        if (++g < p.Hkv) return;
        g = 0;
        if (++qt >= q.q_tiles(p.QT)) {
            qt = 0;
            do {
                q = ++s < p.q.n ? seq_at<MODE>(p, s) : Seq{0, 1, 0};
            } while (q.n == 0);
        }
        settle(p);
    }
};

// Joins one row of an item's pieces in their order, by a warp: piece u holds the row's HD sums at offset `row` and its
// (maximum, sum) at offset `stat` of piece_at(u).  Lanes below HD / 4 return four dims each, every lane the joint m and l.
// NB loads of a lane are under way together, the first of them with the maxima; they land in `buf` (shared memory, NB * 32
// vectors of this warp), because the attention kernel has no registers to spare for them.
template <int HD, int NB, typename F>
__device__ __forceinline__ float4 join_pieces(const F& piece_at, int n_pieces, int row, int stat, float& m, float& l, float4* buf) {
    constexpr int LANES = HD / 4, SIDE = 32 / LANES, STEP = NB * SIDE;      // lanes of a row; pieces side by side, per step
    static_assert(STEP % 32 == 0 || 32 % STEP == 0, "steps and the factors' blocks of 32 pieces");
    const int lane = threadIdx.x & 31, side = lane / LANES, d = (lane % LANES) * 4;
    const auto stat_of = [&](int u) {
        return u < n_pieces ? __ldcg(reinterpret_cast<const float2*>(piece_at(u) + stat)) : make_float2(-INFINITY, 0.f);
    };
    float2 ml = stat_of(lane);
    float f = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    m = -INFINITY;
    l = 0.f;
#pragma unroll 1
    for (int u0 = 0; u0 < n_pieces; u0 += STEP) {
        float4* to = buf + lane;
        const int nv = min(NB, (n_pieces - u0 + SIDE - 1) / SIDE);
#pragma unroll 1
        for (int v = 0; v < nv; ++v) {
            const int u = u0 + v * SIDE + side;
            if (u < n_pieces) cp_async16(ptx::smem_u32(to + v * 32), piece_at(u) + row + d);
        }
        if (u0 % 32 == 0) {                                      // the factors of 32 pieces
            if (u0 == 0) {
                m = ml.x;
#pragma unroll 1
                for (int u = lane + 32; u < n_pieces; u += 32) m = fmaxf(m, __ldcg(piece_at(u) + stat));
                m = warp_max(m);
            } else {
                ml = stat_of(u0 + lane);
            }
            f = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - m);
            l = fmaf(ml.y, f, l);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");         // a lane reads what it has asked for itself
#pragma unroll 1
        for (int v = 0; v < nv; ++v) {
            const int k = v * SIDE + side;
            const float w = __shfl_sync(0xffffffffu, f, (u0 + k) & 31);
            if (u0 + k >= n_pieces) continue;
            const float4 o = to[v * 32];
            a.x = fmaf(o.x, w, a.x);
            a.y = fmaf(o.y, w, a.y);
            a.z = fmaf(o.z, w, a.z);
            a.w = fmaf(o.w, w, a.w);
        }
    }
    l = warp_sum(l);
    if (SIDE == 2) {
        a.x += __shfl_xor_sync(0xffffffffu, a.x, 16);
        a.y += __shfl_xor_sync(0xffffffffu, a.y, 16);
        a.z += __shfl_xor_sync(0xffffffffu, a.z, 16);
        a.w += __shfl_xor_sync(0xffffffffu, a.w, 16);
    }
    return a;
}
// four dims of a result row: a / l, or 0 for a row that sees nothing
template <typename T> __device__ __forceinline__ void store4(T* o, const float4& a, float l) {
    const float inv = 1.f / l;
    const bool sees = l != 0.f;                        // (a NaN is one that sees)
    o[0] = from_f<T>(sees ? a.x * inv : 0.f);
    o[1] = from_f<T>(sees ? a.y * inv : 0.f);
    o[2] = from_f<T>(sees ? a.z * inv : 0.f);
    o[3] = from_f<T>(sees ? a.w * inv : 0.f);
}

// This CTA's piece of the list: `per` places for every CTA but the last, `count` tiles among them.
struct Piece {
    int per, count;
};
template <int MODE> struct Find {        // shared memory of find_piece
    Cursor<MODE> cur;
    int begin, count;                    // place at which the first tile's item begins
    int sums[32];
};
// Of an item of nt tiles, of which this CTA has n_here from tile `first` on but not all: the CTA it begins in, and how many
// CTAs have a piece of it.  One that began before is this CTA's first; of one that begins here the others have what is left.
template <int MODE> __device__ __forceinline__ int first_cta(const AttnArgs& p, const Find<MODE>& f, int per, int first) {
    return first > 0 ? (int)((unsigned)(f.begin + p.ahead) / (unsigned)per) : (int)blockIdx.x;
}
template <int MODE>
__device__ __forceinline__ int piece_count(const AttnArgs& p, const Find<MODE>& f, int per, int first, int n_here, int nt) {
    const unsigned rest = first > 0 ? (unsigned)(f.begin + p.ahead) % (unsigned)per + nt : (unsigned)(per + nt - n_here);
    return (int)((rest + per - 1) / (unsigned)per);
}

// Finds it and the cursor at its first tile, THREADS sequences at a time (the first step's are kept); before and after run
// around the first barrier, which also publishes what the caller has set up in shared memory.  The host refuses calls of
// 2^31 places, counted for rows that each belong to one sequence at most; offsets that decrease could give rows to
// several, whose scores would lie on one another and whose places could pass 32 bits, and then every CTA gets an empty
// piece.  (This and what ends an item run once or twice per CTA, from instructions that have to be fetched first: short
// loops and 32-bit arithmetic are worth more here than fewer steps.)
template <int THREADS, int MODE, typename F, typename H>
__device__ __forceinline__ void find_piece(const AttnArgs& p, Find<MODE>& f, Piece& mine, Cursor<MODE>& cur, F before_sync, H after_sync) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Seq q_own = tid < p.q.n ? seq_at<MODE>(p, tid) : Seq{0, 0, 0};
    const int n_own = seq_places<MODE>(p, q_own);
    bool decrease = q_own.len < 0;
    if constexpr (MODE == OWN) decrease |= *p.prefix_voided != 0;
    if constexpr (MODE == JOINT) {
        if (p.first)
#pragma unroll 1
            for (int g = tid; g < p.groups; g += THREADS) decrease |= bad_groups(p, g);
    }
    {
        int sum = n_own;
#pragma unroll 1
        for (int s = tid + THREADS; s < p.q.n; s += THREADS) {
            const Seq q = seq_at<MODE>(p, s);
            decrease |= q.len < 0;
            sum += seq_places<MODE>(p, q);
        }
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) f.sums[warp] = sum;
    }
    before_sync();
    decrease = __syncthreads_or(decrease);
    after_sync();
    if (blockIdx.x == 0 && tid == 0) *p.voided = decrease;
    const int total = __reduce_add_sync(0xffffffffu, lane < THREADS / 32 ? f.sums[lane] : 0);
    mine.per = max((int)(((unsigned)total + gridDim.x - 1) / gridDim.x), p.min_places);
    mine.count = 0;
    if (decrease) return;
    const long long at = (long long)blockIdx.x * mine.per;
    if (at >= total) return;
    const int p0 = (int)at;
    int base = 0;                                                // places of the sequences before this step's
#pragma unroll 1
    for (int s0 = 0; s0 < p.q.n; s0 += THREADS) {
        const int s = s0 + tid;
        Seq q = q_own;
        int n = n_own;
        if (s0 > 0) {
            q = s < p.q.n ? seq_at<MODE>(p, s) : Seq{0, 0, 0};
            n = seq_places<MODE>(p, q);
        }
        int x = n;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();                                         // sums has been read
        if (lane == 31) f.sums[warp] = x;
        __syncthreads();
        const int w = lane < THREADS / 32 ? f.sums[lane] : 0;
        const int before = base + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + x - n;
        base += __reduce_add_sync(0xffffffffu, w);
        if (n > 0 && before <= p0 && p0 < before + n) {
            int left = p0 - before;
            Cursor<MODE> u{s, 0, 0, 0, 0, q};
            u.settle(p);
#pragma unroll 1
            while (left >= (p.ahead + u.nt) * p.Hkv) {
                left -= (p.ahead + u.nt) * p.Hkv;
                ++u.qt;
                u.settle(p);
            }
            u.g = left / (p.ahead + u.nt);
            left -= u.g * (p.ahead + u.nt);                      // place within the item
            f.begin = p0 - left;
            u.t = max(left - p.ahead, 0);
            f.cur = u;
            int count = 0, room = min(mine.per, total - p0) + left;      // places from the item's first one on
#pragma unroll 1
            while (true) {                                       // the tiles among them
                count += max(0, min(u.nt, room - p.ahead) - u.t);
                room -= p.ahead + u.nt;
                if (room <= 0) break;
                u.next_item(p);
            }
            f.count = count;
        }
        if (base > p0) break;
    }
    __syncthreads();
    cur = f.cur;
    mine.count = f.count;
}

// byte `b` of row `row` of a tile of codes: rows of ROW bytes in the ROW-byte swizzle
template <int ROW> __device__ __forceinline__ uint32_t f8_at(uint32_t row, uint32_t b) {
    return ROW == 128 ? row * 128 + ((((b >> 4) ^ row) & 7) << 4) + (b & 15)
                      : row * 64 + ((((b >> 4) ^ (row >> 1)) & 3) << 4) + (b & 15);
}

// A row's sums over its own keys and over the prefix, relative to their references m and pre.x: the factors that bring
// both to the larger one, and the joint sum of exponentials.
struct Merge {
    float own, pre, l;
    __device__ __forceinline__ Merge(float m, float l_own, float2 before) {
        const float top = fmaxf(m, before.x);
        own = m == -INFINITY ? 0.f : exp2_fast(m - top);
        pre = before.x == -INFINITY ? 0.f : exp2_fast(before.x - top);
        l = l_own * own + before.y * pre;
    }
    __device__ __forceinline__ float operator()(float o, float before) const { return o * own + before * pre; }
    __device__ __forceinline__ float4 operator()(const float4& o, const float4& b) const {
        return make_float4((*this)(o.x, b.x), (*this)(o.y, b.y), (*this)(o.z, b.z), (*this)(o.w, b.w));
    }
};
// whether sequence s has a prefix (OWN; its group's offsets were in order)
__device__ __forceinline__ bool has_prefix(const AttnArgs& p, int s) {
    return !p.first || (s >= p.first[0] && s < p.first[p.groups]);
}
__device__ __forceinline__ int64_t prefix_at(const AttnArgs& p, int row, int head) { return (int64_t)row * p.Hq + head; }

// where a row's sums stand: row k of `pieces` pieces of the item that begins in CTA u0; none of them: in side_sum
__device__ __forceinline__ int2 place_of_sums(int u0, int k, int pieces) { return make_int2(u0 << 7 | k, pieces); }

// One CTA per SM, in clusters of two: the two SMs of a pair share what they fetch instructions through, and the SMs that this launch leaves
// free for another are whole pairs (64 sequences of up to 256 keys beside 8192 shared ones: 42.2 us in all without clusters, 34.1 with).
inline unsigned in_pairs(unsigned ctas) { return ctas > 2 ? ctas / 2 * 2 : 2; }
template <typename... KArgs, typename... Args>
cudaError_t launch_pairs(bool pdl, void (*k)(KArgs...), unsigned ctas, int threads, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

inline AttnArgs attn_args(const Kv8& c, const Kv8Seqs& q, const Kv8Rows& r, const Kv8Attn& a, int layer) {
    const int64_t blocks = c.cfg.n_pages * c.cfg.n_kv_heads, k0 = (int64_t)layer * 2 * blocks;
    AttnArgs p{};
    p.q = q;
    p.r = r;
    p.a = a;
    p.ks = c.scales + k0;
    p.vs = p.ks + blocks;
    p.Hq = c.cfg.n_heads;
    p.Hkv = c.cfg.n_kv_heads;
    p.G = p.Hq / p.Hkv;
    p.inv_g = (65536 + p.G - 1) / p.G;
    p.kz = 2 * layer;
    p.box = c.cfg.page_size < TK ? c.cfg.page_size : TK;
    p.part = c.part;
    p.arrived = c.arrived;
    p.sms = c.num_sms;
    p.stats = c.stats;
    p.score_ld = (q.max_len + TK - 1) / TK * TK;
    return p;
}
// Up to 32 columns (rows of a sequence, on average, times heads of a group) stand in one item of the kernel for few rows, and
// beyond that keys and values are read and P is formed once per item of 32 (64 sequences of 2K: 32 columns 111 us there, 121
// in the kernel for many rows; 48 columns 205 and 122).
inline bool many_rows(const Kv8& c, const AttnArgs& p) {
    const int rows = (p.r.n_rows + p.q.n - 1) / p.q.n;
    return c.cfg.dtype == CB_BF16 && rows * p.G > 32;
}

// ------------------------------------------------------------------------------------------------
// tiles of codes and their scales into shared memory
// ------------------------------------------------------------------------------------------------
// 4 bytes to shared memory; the barrier is arrived at once this thread's copies so far have landed
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

constexpr int LOOK = 2;                  // tiles by which the scales are asked for ahead of the codes
template <int N> struct ScaleRing {      // scales of N tiles, under way or in use
    static constexpr int SLOTS = N;
    float scale[N][2][8];                // K's and V's scale of each box of a tile; -1: not loaded
    uint64_t full[N];                    // one arrival per box
};

// The TMA warp: this CTA's tiles of K and V codes into rings of KS and VS stages (swizzled as the tensor map says).  A lane
// looks after one box (at most a page) of a tile.  Its page id is loaded LOOK + 1 tiles ahead and the scales are asked for
// LOOK tiles ahead, so that neither is waited for when memory is busy.  Rows that belong to no page of the pool or lie
// behind the sequence's last page are not loaded.  Returns when every copy has landed.
template <int HD, int KS, int VS, int RING, int MODE>
__device__ __forceinline__ void produce_tiles(const AttnArgs& p, const CUtensorMap& map, Cursor<MODE> cur, int count, uint8_t* sK,
                                              uint8_t* sV, uint64_t* k_full, uint64_t* k_empty, uint64_t* v_full,
                                              uint64_t* v_empty, ScaleRing<RING>& ring, volatile int* abort) {
    const int lane = threadIdx.x & 31, boxes = TK / p.box, rows = p.box, in_page = (1 << p.q.shift) - 1;
    unsigned* status = p.q.status;
    struct Ahead {
        int page, g, off;                                        // off: first row in the page
        bool need;                                               // the box holds rows of the sequence
    };
    auto look = [&](const Cursor<MODE>& u) {
        const int own_t = u.t - u.q.template pre_tiles<MODE>();
        if (MODE == JOINT && own_t < 0) {
            const int j = u.t * TK + lane * rows;
            Ahead a{0, u.g, j & in_page, lane < boxes && j < u.q.pre};
            if (a.need) a.page = p.pre.table[(int64_t)u.q.group * p.pre.table_ld + (j >> p.q.shift)];
            return a;
        }
        const int j = own_t * TK + lane * rows;
        Ahead a{0, u.g, j & in_page, lane < boxes && j < u.q.len};
        if (a.need) a.page = p.q.table[(int64_t)u.s * p.q.table_ld + (j >> p.q.shift)];
        return a;
    };
    auto ask_scales = [&](Ahead& a, int i) {                     // (the page id was loaded a tile ago)
        if (a.need && (a.page < 0 || a.page >= p.q.n_pages)) {
            atomicOr(status, ST_BAD_ROW);
            a.need = false;
        }
        if (lane >= boxes) return;
        float* dst = &ring.scale[i % RING][0][lane];
        const uint32_t bar = ptx::smem_u32(&ring.full[i % RING]);
        if (a.need) {
            const int64_t at = (int64_t)a.page * p.Hkv + a.g;
            cp_async4(ptx::smem_u32(dst), p.ks + at);
            cp_async4(ptx::smem_u32(dst + 8), p.vs + at);
            cp_async_arrive(bar);
        } else {
            dst[0] = dst[8] = -1.f;
            ptx::mbar_arrive(bar);
        }
    };
    int k_issued = 0, v_issued = 0;
    Ahead box[LOOK + 2];
    int at = 0;                                                  // tile that `cur` stands at
    auto advance = [&] {
        if (++at < count && ++cur.t == cur.nt) cur.next_item(p);
    };
    if (count > 0) {
#pragma unroll
        for (int k = 0; k <= LOOK; ++k) {                        // tiles 0 .. LOOK
            box[k] = look(cur);
            if (at >= count) box[k].need = false;
            advance();
        }
#pragma unroll
        for (int k = 0; k < LOOK; ++k)
            if (k < count) ask_scales(box[k], k);
    }
    for (int i = 0; i < count; ++i) {
        box[LOOK + 1] = Ahead{0, 0, 0, false};
        if (at < count) box[LOOK + 1] = look(cur);               // tile i + LOOK + 1
        advance();
        if (i + LOOK < count) ask_scales(box[LOOK], i + LOOK);
        const bool load = box[0].need;
        const int row = (box[0].page * p.Hkv + box[0].g) * (in_page + 1) + box[0].off;
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, load)) * rows * HD;
#pragma unroll
        for (int k = 0; k <= LOOK; ++k) box[k] = box[k + 1];
        // K and V have barriers of their own: a K tile is free as soon as its S is computed, a V tile a softmax later
        const int sk = i % KS, sv = i % VS;
        bool ok = ptx::mbar_wait(ptx::smem_u32(&k_empty[sk]), ((i / KS) & 1) ^ 1, abort, status);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lane == 0) ptx::mbar_arrive_expect_tx(ptx::smem_u32(&k_full[sk]), bytes);
        __syncwarp();
        k_issued = i + 1;
        if (load)
            tma_3d(ptx::smem_u32(sK + (sk * TK + lane * rows) * HD), &map, 0, row, p.kz, ptx::smem_u32(&k_full[sk]));
        ok = ptx::mbar_wait(ptx::smem_u32(&v_empty[sv]), ((i / VS) & 1) ^ 1, abort, status);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lane == 0) ptx::mbar_arrive_expect_tx(ptx::smem_u32(&v_full[sv]), bytes);
        __syncwarp();
        v_issued = i + 1;
        if (load)
            tma_3d(ptx::smem_u32(sV + (sv * TK + lane * rows) * HD), &map, 0, row, p.kz + 1, ptx::smem_u32(&v_full[sv]));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    int never = 0;
    for (int i = max(0, k_issued - KS); i < k_issued; ++i)
        ptx::mbar_wait(ptx::smem_u32(&k_full[i % KS]), (i / KS) & 1, &never, status);
    for (int i = max(0, v_issued - VS); i < v_issued; ++i)
        ptx::mbar_wait(ptx::smem_u32(&v_full[i % VS]), (i / VS) & 1, &never, status);
}

}  // namespace

}  // namespace cb
