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
};

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
    __device__ __forceinline__ int q_tiles(int QT) const { return (n + QT - 1) / QT; }
    // keys that the last row of query tile qt sees
    __device__ __forceinline__ int visible(int qt, int QT) const { return max(0, len - n + min((qt + 1) * QT, n)); }
    __device__ __forceinline__ int tiles(int qt, int QT) const { return max(1, (visible(qt, QT) + TK - 1) / TK); }
};
__device__ __forceinline__ Seq seq_at(const AttnArgs& p, int s) {
    Seq q;
    int r1;
    if (!kv8_rows(p.q, p.r, s, q.r0, r1, q.len)) return Seq{0, 0, r1 < q.r0 ? -1 : 0};
    q.n = r1 - q.r0;
    return q;
}
__device__ __forceinline__ int seq_places(const AttnArgs& p, const Seq& q) {
    int t = 0;
#pragma unroll 1
    for (int qt = 0; qt < q.q_tiles(p.QT); ++qt) t += p.ahead + q.tiles(qt, p.QT);
    return t * p.Hkv;
}

// Scores of a column (query row of the sequence x head of the group) with the keys of tile t: a tile's columns lie together,
// so that what sums over them reads one contiguous piece.
__device__ __forceinline__ float* score_of(const AttnArgs& p, const Seq& q, int g, int t, int col) {
    return p.scores + ((int64_t)g * p.r.n_rows + q.r0) * p.G * p.score_ld + ((int64_t)t * q.n * p.G + col) * TK;
}

// A tile in the list: item (s, query tile qt, g) and tile t of its nt.
struct Cursor {
    int s, qt, g, t, nt;
    Seq q;
    __device__ __forceinline__ void settle(const AttnArgs& p) { nt = q.tiles(qt, p.QT); }
    // to the first tile of the next item
    __device__ __forceinline__ void next_item(const AttnArgs& p) {
        t = 0;
        if (++g < p.Hkv) return;
        g = 0;
        if (++qt >= q.q_tiles(p.QT)) {
            qt = 0;
            do {
                q = ++s < p.q.n ? seq_at(p, s) : Seq{0, 1, 0};
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
struct Find {                            // shared memory of find_piece
    Cursor cur;
    int begin, count;                    // place at which the first tile's item begins
    int sums[32];
};
// Of an item of nt tiles, of which this CTA has n_here from tile `first` on but not all: the CTA it begins in, and how many
// CTAs have a piece of it.  One that began before is this CTA's first; of one that begins here the others have what is left.
__device__ __forceinline__ int first_cta(const AttnArgs& p, const Find& f, int per, int first) {
    return first > 0 ? (int)((unsigned)(f.begin + p.ahead) / (unsigned)per) : (int)blockIdx.x;
}
__device__ __forceinline__ int piece_count(const AttnArgs& p, const Find& f, int per, int first, int n_here, int nt) {
    const unsigned rest = first > 0 ? (unsigned)(f.begin + p.ahead) % (unsigned)per + nt : (unsigned)(per + nt - n_here);
    return (int)((rest + per - 1) / (unsigned)per);
}

// Finds it and the cursor at its first tile, THREADS sequences at a time (the first step's are kept); before and after run
// around the first barrier, which also publishes what the caller has set up in shared memory.  The host refuses calls of
// 2^31 places, counted for rows that each belong to one sequence at most; offsets that decrease could give rows to
// several, whose scores would lie on one another and whose places could pass 32 bits, and then every CTA gets an empty
// piece.  (This and what ends an item run once or twice per CTA, from instructions that have to be fetched first: short
// loops and 32-bit arithmetic are worth more here than fewer steps.)
template <int THREADS, typename F, typename H>
__device__ __forceinline__ void find_piece(const AttnArgs& p, Find& f, Piece& mine, Cursor& cur, F before_sync, H after_sync) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Seq q_own = tid < p.q.n ? seq_at(p, tid) : Seq{0, 0, 0};
    const int n_own = seq_places(p, q_own);
    bool decrease = q_own.len < 0;
    {
        int sum = n_own;
#pragma unroll 1
        for (int s = tid + THREADS; s < p.q.n; s += THREADS) {
            const Seq q = seq_at(p, s);
            decrease |= q.len < 0;
            sum += seq_places(p, q);
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
            q = s < p.q.n ? seq_at(p, s) : Seq{0, 0, 0};
            n = seq_places(p, q);
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
            Cursor u{s, 0, 0, 0, 0, q};
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
template <int HD, int KS, int VS, int RING>
__device__ __forceinline__ void produce_tiles(const AttnArgs& p, const CUtensorMap& map, Cursor cur, int count, uint8_t* sK,
                                              uint8_t* sV, uint64_t* k_full, uint64_t* k_empty, uint64_t* v_full,
                                              uint64_t* v_empty, ScaleRing<RING>& ring, volatile int* abort) {
    const int lane = threadIdx.x & 31, boxes = TK / p.box, rows = p.box, in_page = (1 << p.q.shift) - 1;
    unsigned* status = p.q.status;
    struct Ahead {
        int page, g, off;                                        // off: first row in the page
        bool need;                                               // the box holds rows of the sequence
    };
    auto look = [&](const Cursor& u) {
        const int j = u.t * TK + lane * rows;
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
