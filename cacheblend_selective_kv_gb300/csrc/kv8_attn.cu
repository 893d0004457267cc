// Attention over the 8-bit paged K/V cache on the sm_103a tensor cores.  Query row i of a sequence's n sits at position
// len - n + i and sees keys 0 .. that position: out = softmax(q k * scale) v, the G query heads of a group sharing a KV
// head.  A row that sees nothing (its position is negative, or all its keys lie in bad pages) gives 0.  With weights,
// every key gets the sum of its softmax weights over the call's query rows and the group's heads.
//
// A decoding step reads every cached byte once and does 4 G FLOPs for it, so it is bound by HBM as long as the codes
// reach the matrix unit without being touched.  They do: tcgen05 kind::f8f6f4 takes e4m3 operands, so the keys are the
// A operand of S^T = K Q^T (M = 128 keys, N = query columns) and the values, read MN-major from the same [key][dim]
// tile, the A operand of O^T = V^T P^T (M = dims, K = 128 keys); block scales multiply S and P in fp32.  With the
// queries in N, a column costs only what it uses: 16 columns for a decoded token where a 128-row tile would waste 120.
//
// q and P are not 8-bit values.  Each is written as a sum of e4m3 numbers c_0 + c_1 / 16 + c_2 / 256 + .., every term the
// rounding of 16 times the residue before it, as columns of their own (column t * NC + c holds term t of column c), and
// the columns of a sum are added in fp32 after the MMA.  A term carries 4 bits: a bf16 q is two terms, exactly for elements
// down to 2^-14 of the row's largest and within 2^-21 of that largest below (where e4m3 runs out of exponents); P gets
// three (2^-12 relative), which keeps the result's error well below its bf16 rounding.  fp32 calls use six of each.
// e4m3 products and their fp32 accumulation were checked to be as exact as an fp32 sum of the same products.
//
// Work: an item is (sequence, tile of NC / G query rows, KV head), cut into tiles of 128 keys.  All tiles of all items
// form one list; every CTA takes an equal, contiguous piece of it, so that any mix of lengths is balanced.  An item that
// spans several CTAs is joined by the CTA that finishes last, in the order of the pieces (the result does not depend on
// which one that is).  Which items a CTA has follows from the lengths on the device, so a captured graph stays valid.
//
// Roles: softmax and output warps in groups of four (thread = key, then thread = dim; a group owns NC / GR of the columns,
// so that many columns get more warps and not more registers per thread), one TMA warp (page by page through the block
// table), one MMA warp.  S of the next tile is computed while P of this one is formed; O of a tile is read back from
// tensor memory and added in registers while the next tile's P is formed, which rescales it exactly and makes every
// tile's sum its own.  P is stored [key][column], the B operand MN-major, so that a thread's terms are a few vector
// stores instead of a byte store for each; what belongs to a column (its maximum, its factors) is computed by one lane
// per warp and read back from shared memory.
//
// Measured (32 heads, 8 KV heads of 128, bf16): 64 sequences of up to 8K keys, each its own length, 97 us, 88 % of the measured
// copy rate; 64 x 8192 keys 167 us, 95 %; 1 x 131071 keys 54 us, 73 %; 1 x 200 keys 7 us.  Bound by HBM in the long run (the
// difference between two lengths is read at the copy rate), with about 7 us for the launch, the first tile and the end.
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cstring>
#include <iterator>

#include "cb_kv8_attn.cuh"

namespace cb {

namespace {


constexpr int round16(int x) { return (x + 15) / 16 * 16; }
constexpr int pow2_cols(int x) { return x <= 32 ? 32 : x <= 64 ? 64 : x <= 128 ? 128 : x <= 256 ? 256 : 512; }

__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// D[tmem] (+)= A[smem] B[smem]^T, e4m3 operands, fp32 accumulator; one thread issues it
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Shared-memory operand descriptor: rows of 128 bytes in the 128-byte swizzle, or of 64 bytes in the 64-byte one; eight
// rows are one atom and the next eight follow it directly.
template <int ROW> __device__ __forceinline__ uint64_t f8_desc(uint32_t saddr, uint32_t lbo) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)((8 * ROW) >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)(ROW == 128 ? 2 : 4) << 61);
}
// B operand MN-major: rows (keys) of PITCH bytes = columns in the PITCH-byte swizzle; more than 128 columns are further
// blocks of 128 rows
template <int PITCH> __device__ __forceinline__ uint64_t p_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((TK * PITCH) >> 4) << 16) | ((uint64_t)((8 * PITCH) >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)(PITCH == 128 ? 2 : PITCH == 64 ? 4 : 6) << 61);
}
template <int PITCH> __device__ __forceinline__ uint32_t p_at(uint32_t key, uint32_t col) {
    const uint32_t c = col % PITCH, ch = c >> 4;
    const uint32_t x = PITCH == 128 ? (ch ^ key) & 7 : PITCH == 64 ? (ch ^ (key >> 1)) & 3 : (ch ^ (key >> 2)) & 1;
    return col / PITCH * (TK * PITCH) + key * PITCH + x * 16 + (c & 15);
}
__host__ __device__ constexpr uint32_t f8_idesc(int N, bool mn) {       // M = 128; mn: both operands MN-major
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24) | (mn ? 3u << 15 : 0u);
}
// N consecutive columns of this thread's lane, without the wait
template <int N> __device__ __forceinline__ void tmem_ld_cols(uint32_t addr, uint32_t* r) {
    if constexpr (N == 4) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
    } else if constexpr (N == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(addr));
    } else {
        ptx::tmem_ld16_issue(addr, r);
    }
}
// ... and the wait, through which the registers pass so that no use of them moves above it
template <int N> __device__ __forceinline__ void tmem_ld_done(uint32_t* r) {
#pragma unroll
    for (int k = 0; k < N; k += 4)
        asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[k]), "+r"(r[k + 1]), "+r"(r[k + 2]), "+r"(r[k + 3])::"memory");
}
constexpr int MAX_STAGES = 3;
constexpr int RING = 8;
struct Open {                            // an item of which this CTA has a piece
    int u0, pieces;                      // the CTA it begins in, how many have a piece of it
    int row0, cols, g;
};
struct Shared {
    ScaleRing<RING> ring;
    uint64_t k_full[MAX_STAGES], v_full[MAX_STAGES], k_empty[MAX_STAGES], v_empty[MAX_STAGES];
    uint64_t s_full[2], s_free[2];
    uint64_t p_full, o_full, q_full, drain;
    uint32_t tmem;
    int abort;
    Find find;
    Cursor next;                         // the softmax warps' next item
    Open open[2];                        // at the beginning of this CTA's tiles, at their end
    int last[2];                         // this CTA joins it
};

// ------------------------------------------------------------------------------------------------
// HD: head_dim; NC: query columns; GR: softmax groups; TQ, TP: terms of q and P; CTAS per SM; STAGES: K and V tiles in flight
// ------------------------------------------------------------------------------------------------
template <int HD_, int NC_, int GR_, int TQ_, int TP_, int CTAS_, int STAGES_> struct Shape {
    static constexpr int HD = HD_, NC = NC_, GR = GR_, TQ = TQ_, TP = TP_, CTAS = CTAS_, STAGES = STAGES_;
    static constexpr int NW = NC / GR;                                     // columns of a group
    static constexpr int SOFT = 128 * GR, THREADS = SOFT + 64;
    static constexpr int NQ = round16(TQ * NC), NP = round16(TP * NC);     // MMA columns
    static constexpr int KV_BYTES = TK * HD, Q_BYTES = NQ * HD;
    static constexpr int PITCH = NP <= 32 ? 32 : NP <= 64 ? 64 : 128;
    static constexpr int P_BYTES = (NP + 127) / 128 * TK * PITCH;
    static constexpr int O_COL = 2 * NQ;
    static constexpr int TMEM = pow2_cols(2 * NQ + NP);
    // K/V stages, Q (two), P (all 1024-byte aligned), then the softmax exchange and the control block
    static constexpr int OFF_Q = 2 * STAGES * KV_BYTES;
    static constexpr int OFF_P = (OFF_Q + 2 * Q_BYTES + 1023) / 1024 * 1024;
    static constexpr int OFF_X = (OFF_P + P_BYTES + 1023) / 1024 * 1024;
    // floats: wmax, ymax [2][GR][4][NW]; cols [2][4 GR][4][NW]; qscale [2][NC]; wsum, colm [4][NC]; nan_from [2][HD]
    static constexpr int X_FLOATS = 2 * 8 * NC + 2 * 4 * GR * 4 * NW + 2 * NC + 8 * NC + 2 * HD;
    static constexpr int OFF_C = (OFF_X + X_FLOATS * 4 + 63) / 64 * 64;
    static constexpr int BYTES = OFF_C + (int)sizeof(Shared);
    static constexpr int PIECE = NC * (HD + 2);                            // floats of an unfinished item
    // vectors per lane that a joining warp has under way, where K and V were
    static constexpr int JOIN = HD / 4 / GR;
    static_assert(JOIN * 512 * (SOFT / 32) <= OFF_Q, "joining buffers");
    static_assert(TMEM * CTAS <= 512 && 2 * NQ + NP <= 512, "tensor memory");
    static_assert((BYTES + 1024) * CTAS <= 228 * 1024 && STAGES <= MAX_STAGES, "shared memory");
    static_assert(NW == 4 || NW == 8 || NW == 16, "columns of a group");
};

// piece u of the item that begins in CTA u0: a CTA's first one is of an item that began before
template <typename S> __device__ __forceinline__ float* piece_at(const AttnArgs& p, int u0, int u) {
    return p.part + (int64_t)((u0 + u) * 2 + (u == 0 ? 1 : 0)) * S::PIECE;
}

// Kept out of the tile loop, whose instructions have to stay close together:

// Q of an item as terms: column r = (query row, head of the group), lane = HD / 32 of its dims.  An item's Q is written
// (into one of two buffers) while the first tile of the item before it is worked on, so that the MMA warp runs on across
// items.
template <typename T, typename S>
__device__ __noinline__ void q_terms(const AttnArgs& p, const Cursor& u, uint8_t* sQ, float* qscale, float to_exp2) {
    constexpr int HD = S::HD, E = HD / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q0 = u.qt * p.QT, cols = min(p.QT, u.q.n - q0) * p.G;
    const T* qbase = (const T*)p.a.q + (int64_t)(u.q.r0 + q0) * p.a.q_stride + (int64_t)u.g * p.G * HD;
    for (int r = warp; r < S::NC; r += S::SOFT / 32) {
        float x[E];
        float top = 0.f;
        const T* src = qbase + (int64_t)(div_g(p, r)) * p.a.q_stride + (mod_g(p, r)) * HD + lane * E;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            x[k] = r < cols ? to_f(src[k]) : 0.f;
            top = fmaxf(top, kv8_mag(x[k]));
        }
        const float sc = kv8_scale(warp_max(top)), inv = kv8_inverse(sc);
#pragma unroll
        for (int k = 0; k < E; ++k) x[k] = kv8_nan_inf(x[k]) * inv;
#pragma unroll
        for (int t = 0; t < S::TQ; ++t) {
            uint32_t w = 0;
#pragma unroll
            for (int k = 0; k < E; k += 2) {
                const uint32_t c2 = kv8_code2(x[k], x[k + 1]);
                const float2 v = kv8_value2(c2);
                x[k] = (x[k] - v.x) * 16.f;
                x[k + 1] = (x[k + 1] - v.y) * 16.f;
                w |= c2 << (8 * k);
            }
            uint8_t* d = sQ + f8_at<HD>(t * S::NC + r, lane * E);
            if (E == 4) *reinterpret_cast<uint32_t*>(d) = w;
            else *reinterpret_cast<uint16_t*>(d) = (uint16_t)w;
        }
        if (lane == 0) qscale[r] = sc * to_exp2;
    }
    fence_async_smem();
    __syncwarp();
}

// A V row that no weight may meet: one that was not loaded or lies behind the sequence is zeroed (0 times NaN would be
// NaN); in one that only later query rows see, NaN codes are taken out and remembered.
template <int HD> __device__ __noinline__ void clean_v_row(uint8_t* tile, int key, bool have, int j, int* nan_from) {
    for (int d = 0; d < HD; d += 16) {
        uint4* v = reinterpret_cast<uint4*>(tile + f8_at<HD>(key, d));
        if (!have) {
            *v = make_uint4(0, 0, 0, 0);
            continue;
        }
        uint32_t* w = reinterpret_cast<uint32_t*>(v);
        for (int k = 0; k < 4; ++k) {
            const uint32_t bad = __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
            if (bad == 0) continue;
            w[k] &= ~bad;
            for (int n = 0; n < 4; ++n)
                if (bad >> (8 * n) & 1) atomicMin(&nan_from[d + 4 * k + n], j);
        }
    }
}

template <typename T, typename S>
__global__ void __launch_bounds__(S::THREADS, S::CTAS)
    kv8_attn_kernel(const __grid_constant__ CUtensorMap map, const AttnArgs p) {
    constexpr int HD = S::HD, NC = S::NC, NW = S::NW, GR = S::GR, TQ = S::TQ, TP = S::TP, NQ = S::NQ, NP = S::NP;
    constexpr int STAGES = S::STAGES, SOFT = S::SOFT, THREADS = S::THREADS, TMA_WARP = SOFT / 32, MMA_WARP = TMA_WARP + 1;
    extern __shared__ __align__(1024) uint8_t sm[];     // no static shared memory: the window starts on 1024 bytes
    uint8_t* sK = sm;                                   // [STAGES][TK][HD]
    uint8_t* sV = sm + STAGES * S::KV_BYTES;
    uint8_t* sQ = sm + S::OFF_Q;
    uint8_t* sP = sm + S::OFF_P;
    float* wmax = reinterpret_cast<float*>(sm + S::OFF_X);
    float* ymax = wmax + 8 * NC;
    float* cols_of = ymax + 8 * NC;
    float* qscale = cols_of + 2 * 4 * GR * 4 * NW;
    float* wsum = qscale + 2 * NC;
    float* colm = wsum + 4 * NC;
    int* nan_marks = reinterpret_cast<int*>(colm + 4 * NC);
    Shared& c = *reinterpret_cast<Shared*>(sm + S::OFF_C);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned* status = p.q.status;
    volatile int* abort = &c.abort;
    if (ptx::smem_u32(sm) & 1023) {                     // (the swizzled layouts would not hold)
        if (tid == 0) atomicOr(status, ST_WAIT_TIMEOUT);
        return;
    }

    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            ptx::mbar_init(ptx::smem_u32(&c.k_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&c.v_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&c.k_empty[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&c.v_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_u32(&c.s_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&c.s_free[i]), SOFT / 32);
        }
        for (int i = 0; i < RING; ++i) ptx::mbar_init(ptx::smem_u32(&c.ring.full[i]), TK / p.box);
        ptx::mbar_init(ptx::smem_u32(&c.p_full), SOFT / 32);
        ptx::mbar_init(ptx::smem_u32(&c.o_full), 1);
        ptx::mbar_init(ptx::smem_u32(&c.q_full), SOFT / 32);
        ptx::mbar_init(ptx::smem_u32(&c.drain), 1);
        c.abort = 0;
        ptx::fence_barrier_init();
        ptx::prefetch_tmap(&map);
    }
    if (warp == MMA_WARP) {
        ptx::tmem_alloc(ptx::smem_u32(&c.tmem), S::TMEM);
        ptx::tmem_relinquish();
    }

    grid_dep_launch();
    grid_dep_wait();                                     // lengths, tables, queries and the cache of the kernels before
    Piece mine;
    Cursor cur;
    find_piece<THREADS>(p, c.find, mine, cur, [] { ptx::tc_fence_before(); }, [] { ptx::tc_fence_after(); });
    const int count = mine.count;                        // tiles of this CTA
    const uint32_t tmem = c.tmem;

    if (warp == TMA_WARP) {
        // ------------------------------------------------------------------------------------ TMA
        // A scale slot is free again without a barrier of its own: K of tile i - 1 waited for S of tile i - 1 - STAGES, which
        // waited for the softmax to have read tile i - 3 - STAGES, and slot i + LOOK was last used for tile i + LOOK - RING.
        static_assert(RING - LOOK >= STAGES + 3, "scale ring");
        produce_tiles<HD, STAGES, STAGES>(p, map, cur, count, sK, sV, c.k_full, c.k_empty, c.v_full, c.v_empty, c.ring, abort);
    } else if (warp == MMA_WARP) {
        // ------------------------------------------------------------------------------------ MMA
        if (lane == 0) {
            constexpr uint32_t id_s = f8_idesc(NQ, false), id_o = f8_idesc(NP, true);
            uint64_t qd = 0;
            const uint64_t pd = p_desc<S::PITCH>(ptx::smem_u32(sP));
            int left = 0, item = 0;
            bool ok = true;
            auto values = [&](int i) {                           // O^T = V^T P^T of tile i
                const int st = i % STAGES;
                if (!ptx::mbar_wait(ptx::smem_u32(&c.v_full[st]), (i / STAGES) & 1, abort, status) ||
                    !ptx::mbar_wait(ptx::smem_u32(&c.p_full), i & 1, abort, status)) return false;
                ptx::tc_fence_after();
                // head_dim 64: the 128 rows of A are the 64 dims twice (the second half is not read back)
                const uint64_t vd = f8_desc<HD>(ptx::smem_u32(sV + st * S::KV_BYTES), 0);
#pragma unroll
                for (int k = 0; k < TK / 32; ++k)
                    mma_e4m3(tmem + S::O_COL, vd + (uint64_t)(k * 32 * HD >> 4), pd + (uint64_t)(k * 32 * S::PITCH >> 4), id_o, k > 0);
                ptx::mma_commit(ptx::smem_u32(&c.v_empty[st]));
                ptx::mma_commit(ptx::smem_u32(&c.o_full));
                return true;
            };
            for (int i = 0; i < count && ok; ++i) {
                if (left == 0) {                                 // an item's first tile waits for its Q
                    if (i > 0) cur.next_item(p);
                    left = cur.nt - cur.t;
                    if (!ptx::mbar_wait(ptx::smem_u32(&c.q_full), item & 1, abort, status)) break;
                    qd = f8_desc<HD>(ptx::smem_u32(sQ + (item & 1) * S::Q_BYTES), 16);
                    ++item;
                }
                const int st = i % STAGES, b = i & 1;
                if (!ptx::mbar_wait(ptx::smem_u32(&c.k_full[st]), (i / STAGES) & 1, abort, status) ||
                    !ptx::mbar_wait(ptx::smem_u32(&c.s_free[b]), ((i >> 1) & 1) ^ 1, abort, status)) break;
                ptx::tc_fence_after();
                const uint64_t kd = f8_desc<HD>(ptx::smem_u32(sK + st * S::KV_BYTES), 16);
#pragma unroll
                for (int k = 0; k < HD / 32; ++k)
                    mma_e4m3(tmem + b * NQ, kd + (uint64_t)(k * 32 >> 4), qd + (uint64_t)(k * 32 >> 4), id_s, k > 0);
                ptx::mma_commit(ptx::smem_u32(&c.s_full[b]));
                ptx::mma_commit(ptx::smem_u32(&c.k_empty[st]));
                if (i > 0) ok = values(i - 1);
                --left;
                if (ok && i == count - 1) ok = values(i);
            }
            ptx::mma_commit(ptx::smem_u32(&c.drain));            // nothing runs on when the CTA leaves
            int never = 0;
            ptx::mbar_wait(ptx::smem_u32(&c.drain), 0, &never, status);
        }
    } else {
        // ------------------------------------------------------------------------------------ softmax, output
        // A wait that gives up raises `abort`, after which every wait returns at once: these warps then run on to
        // their last tile (their barriers stay in step, the counters stay whole) with results that are not valid.
        const int gr = warp >> 2, quarter = warp & 3, key = tid & 127, c0 = gr * NW;     // this group's first column
        const uint32_t my_lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const float to_exp2 = p.a.scale * 1.4426950408889634f;
        const int box_shift = min(p.q.shift, 7);
        auto write_q = [&](const Cursor& u, int buf) {
            q_terms<T, S>(p, u, sQ + buf * S::Q_BYTES, qscale + buf * NC, to_exp2);
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&c.q_full));
        };
        int item = 0, n_open = 0;
        for (int i = 0; i < count; ++item) {
            const int first = cur.t, n_here = min(cur.nt - first, count - i), g = cur.g;
            const Seq q = cur.q;
            const int q0 = cur.qt * p.QT, rows = min(p.QT, q.n - q0), cols = rows * p.G;
            const int pos0 = q.len - q.n + q0;                   // position of the item's first query row
            const int64_t stat0 = ((int64_t)g * p.r.n_rows + q.r0 + q0) * p.G;     // the item's first column in scores, stats

            int* nan_from = nan_marks + (item & 1) * HD;         // (the item before's may still be read)
            if (tid < HD) nan_from[tid] = INT_MAX;
            if (item == 0) write_q(cur, 0);
            ptx::named_bar_sync(1, SOFT);                        // nan_from, the first item's qscale
            const float* qsc = qscale + (item & 1) * NC + c0;

            float acc[NW], lsum[NW];
            float mrun = -INFINITY;                              // running reference of column c0 + lane
#pragma unroll
            for (int k = 0; k < NW; ++k) acc[k] = lsum[k] = 0.f;
            // factors of this warp's columns in a tile: [0] reference, [1] scale of P, [2] factor of what was summed
            // before, [3] scale of O
            auto col = [&](int i_, int what) { return cols_of + (((i_ & 1) * 4 * GR + warp) * 4 + what) * NW; };
            auto add_tile = [&](int done) {                      // acc = acc * factor + O of a finished tile
                ptx::mbar_wait(ptx::smem_u32(&c.o_full), done & 1, abort, status);
                ptx::tc_fence_after();
                uint32_t o[TP][NW];
#pragma unroll
                for (int t = 0; t < TP; ++t) tmem_ld_cols<NW>(my_lanes + S::O_COL + t * NC + c0, o[t]);
#pragma unroll
                for (int t = 0; t < TP; ++t) tmem_ld_done<NW>(o[t]);
                const float4* al = reinterpret_cast<const float4*>(col(done, 2));
                const float4* os = reinterpret_cast<const float4*>(col(done, 3));
#pragma unroll
                for (int k = 0; k < NW; k += 4) {
                    const float4 a4 = al[k / 4], o4 = os[k / 4];
                    const float av[4] = {a4.x, a4.y, a4.z, a4.w}, ov[4] = {o4.x, o4.y, o4.z, o4.w};
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        float v = __uint_as_float(o[TP - 1][k + n]);
#pragma unroll
                        for (int t = TP - 2; t >= 0; --t) v = fmaf(v, 0.0625f, __uint_as_float(o[t][k + n]));
                        acc[k + n] = fmaf(v, ov[n], acc[k + n] * av[n]);
                    }
                }
            };

            for (int t = first; t < first + n_here; ++t, ++i) {
                const int b = i & 1, j = t * TK + key;
                ptx::mbar_wait(ptx::smem_u32(&c.ring.full[i % RING]), (i / RING) & 1, abort, status);
                const float ks_now = c.ring.scale[i % RING][0][key >> box_shift], vs_now = c.ring.scale[i % RING][1][key >> box_shift];
                const bool have = ks_now >= 0.f && j < q.len;

                ptx::mbar_wait(ptx::smem_u32(&c.s_full[b]), (i >> 1) & 1, abort, status);
                ptx::tc_fence_after();
                float x[NW];
                {
                    uint32_t w[TQ][NW];
#pragma unroll
                    for (int n = 0; n < TQ; ++n) tmem_ld_cols<NW>(my_lanes + b * NQ + n * NC + c0, w[n]);
#pragma unroll
                    for (int n = 0; n < TQ; ++n) tmem_ld_done<NW>(w[n]);
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&c.s_free[b]));
#pragma unroll
                    for (int k = 0; k < NW; ++k) {
                        float v = __uint_as_float(w[TQ - 1][k]);
#pragma unroll
                        for (int n = TQ - 2; n >= 0; --n) v = fmaf(v, 0.0625f, __uint_as_float(w[n][k]));
                        x[k] = v * (ks_now * qsc[k]);
                    }
                }
                // column k (query row k / G) sees key j from its own position on: k >= (j - pos0) G
                const int hidden = have ? min(max(j - pos0, 0), NC) * p.G - c0 : NC;
                if (hidden > 0) {
#pragma unroll
                    for (int k = 0; k < NW; ++k)
                        if (k < hidden) x[k] = -INFINITY;
                }
                if (p.scores) {
                    float* score = score_of(p, q, g, t, q0 * p.G + c0) + key;
#pragma unroll
                    for (int k = 0; k < NW; ++k)
                        if (c0 + k < cols)
                            score[k * TK] = x[k];
                }
                // maxima over the tile's keys of the scores, and of scores with V's scale: y = x + log2(scale), which says
                // how far a column's P can be scaled up.  A warp's keys lie in one block unless pages have 16 rows.
                float* wm = wmax + ((b * GR + gr) * 4) * NW;
                float* wy = ymax + ((b * GR + gr) * 4) * NW;
                const float ev = have && vs_now > 0.f ? (float)((int)(__float_as_uint(vs_now) >> 23) - 127) : -INFINITY;
                const float ew = redux_max(ev);
#pragma unroll
                for (int k = 0; k < NW; k += 4) {
                    float m[4], y[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        m[n] = redux_max(x[k + n]);
                        y[n] = p.box >= 32 ? m[n] + ew : redux_max(x[k + n] + ev);
                    }
                    if (lane == 0) {
                        *reinterpret_cast<float4*>(wm + quarter * NW + k) = make_float4(m[0], m[1], m[2], m[3]);
                        *reinterpret_cast<float4*>(wy + quarter * NW + k) = make_float4(y[0], y[1], y[2], y[3]);
                    }
                }
                ptx::named_bar_sync(2 + gr, 128);
                if (lane < NW) {
                    const float mt = fmaxf(fmaxf(wm[lane], wm[NW + lane]), fmaxf(wm[2 * NW + lane], wm[3 * NW + lane]));
                    const float yt = fmaxf(fmaxf(wy[lane], wy[NW + lane]), fmaxf(wy[2 * NW + lane], wy[3 * NW + lane]));
                    // The reference of the exponentials: the largest score, or what keeps exponential times V's scale within
                    // 2^60, so that a sum of the largest values does not pass fp32 before it is divided.
                    const float mn = fmaxf(fmaxf(mrun, mt), yt - 60.f), ref = mn == -INFINITY ? 0.f : mn;
                    // P of the column times V's scale, scaled by the power of two that brings its largest value to 128 .. 256
                    const int up = 8 + (yt == -INFINITY ? 0 : (int)floorf(fminf(ref - yt, 118.f)));          // 2^-52 .. 2^126
                    col(i, 0)[lane] = ref;
                    col(i, 1)[lane] = __uint_as_float((unsigned)(127 + up) << 23);
                    col(i, 2)[lane] = mn == mrun ? 1.f : exp2_fast(mrun - ref);
                    col(i, 3)[lane] = __uint_as_float((unsigned)(127 - up) << 23);
                    mrun = mn;
                }
                __syncwarp();
                const float v_mul = have ? vs_now : 0.f;
#pragma unroll
                for (int k = 0; k < NW; k += 4) {
                    const float4 r4 = *reinterpret_cast<const float4*>(col(i, 0) + k), p4 = *reinterpret_cast<const float4*>(col(i, 1) + k),
                                 a4 = *reinterpret_cast<const float4*>(col(i, 2) + k);
                    const float rv[4] = {r4.x, r4.y, r4.z, r4.w}, pv[4] = {p4.x, p4.y, p4.z, p4.w}, av[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float e = exp2_fast(x[k + n] - rv[n]);
                        lsum[k + n] = fmaf(lsum[k + n], av[n], e);
                        x[k + n] = (e * pv[n]) * v_mul;          // (pv * v_mul may pass fp32 where e has vanished)
                    }
                }
                if (t > first) add_tile(i - 1);
                // P as terms (sP is free: O of the tile before is complete)
#pragma unroll
                for (int n = 0; n < TP; ++n) {
                    uint32_t w[NW / 4];
#pragma unroll
                    for (int k = 0; k < NW; k += 4) {
                        const uint32_t lo = kv8_code2(x[k], x[k + 1]), hi = kv8_code2(x[k + 2], x[k + 3]);
                        w[k / 4] = lo | (hi << 16);
                        const float2 u = kv8_value2(lo), v = kv8_value2(hi);
                        x[k] = (x[k] - u.x) * 16.f;
                        x[k + 1] = (x[k + 1] - u.y) * 16.f;
                        x[k + 2] = (x[k + 2] - v.x) * 16.f;
                        x[k + 3] = (x[k + 3] - v.y) * 16.f;
                    }
                    uint8_t* d = sP + p_at<S::PITCH>(key, n * NC + c0);
                    if constexpr (NW == 4) *reinterpret_cast<uint32_t*>(d) = w[0];
                    else if constexpr (NW == 8) *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
                    else *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (gr == 0 && (!have || j > pos0)) {
                    const int st = i % STAGES;
                    ptx::mbar_wait(ptx::smem_u32(&c.v_full[st]), (i / STAGES) & 1, abort, status);
                    clean_v_row<HD>(sV + st * S::KV_BYTES, key, have, j, nan_from);
                }
                fence_async_smem();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&c.p_full));
                // (S of this item's first tile is there, so its own Q has been taken and the barrier is a phase behind)
                if (t == first && i + n_here < count + t - first) {
                    Cursor next = cur;
                    next.next_item(p);
                    write_q(next, (item + 1) & 1);
                    if (tid == 0) c.next = next;                 // (kept there: registers are short in the tile loop)
                }
            }
            add_tile(i - 1);
            ptx::tc_fence_before();
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                const float v = warp_sum(lsum[k]);
                if (lane == 0) wsum[quarter * NC + c0 + k] = v;
            }
            if (quarter == 0 && lane < NW) colm[c0 + lane] = mrun;
            ptx::named_bar_sync(1, SOFT);                        // sums, maxima and nan_from of all groups
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                const float* w = wsum + c0 + k;
                lsum[k] = (w[0] + w[NC]) + (w[2 * NC] + w[3 * NC]);
            }
            if (key < HD && nan_from[key] != INT_MAX) {
                const int k0 = (nan_from[key] - pos0) * p.G - c0;        // columns from the row that sees the NaN on
#pragma unroll
                for (int k = 0; k < NW; ++k)
                    if (k >= k0) acc[k] = __int_as_float(0x7fc00000);
            }
            const auto out_at = [&](int k) {                     // output row of column k
                return (T*)p.a.out + (int64_t)(q.r0 + q0 + div_g(p, k)) * p.a.out_stride + (int64_t)(g * p.G + mod_g(p, k)) * HD;
            };
            if (first == 0 && n_here == cur.nt) {
#pragma unroll
                for (int k = 0; k < NW; ++k) {
                    if (c0 + k >= cols) continue;
                    const float inv = 1.f / lsum[k];
                    if (key < HD) out_at(c0 + k)[key] = from_f<T>(lsum[k] != 0.f ? acc[k] * inv : 0.f);
                    if (p.scores && key == 0) p.stats[stat0 + c0 + k] = make_float2(colm[c0 + k], inv);
                }
            } else {
                // A piece.  It is announced, and joined if it was the last, when the CTA has done all its tiles: here every warp
                // would wait for the fence and the count (decode of 64 x 8K: 100.5 us that way, 96 this way).
                const int u0 = first_cta(p, c.find, mine.per, first), n_pieces = piece_count(p, c.find, mine.per, first, n_here, cur.nt);
                float* piece = piece_at<S>(p, u0, blockIdx.x - u0);
                if (key < HD) {
#pragma unroll
                    for (int k = 0; k < NW; ++k) piece[(c0 + k) * HD + key] = acc[k];
                }
                if (key == 0) {
#pragma unroll
                    for (int k = 0; k < NW; ++k)
                        *reinterpret_cast<float2*>(piece + NC * HD + 2 * (c0 + k)) = make_float2(colm[c0 + k], lsum[k]);
                }
                if (tid == 0) c.open[n_open] = Open{u0, n_pieces, q.r0 + q0, cols, g};
                ++n_open;
            }
            if (i < count) cur = c.next;                         // written before the last barrier, again behind the next
        }
        if (n_open > 0) {
            ptx::named_bar_sync(1, SOFT);
            if (tid < n_open) {
                const Open& o = c.open[tid];
                __threadfence();                                 // the whole CTA's pieces, ordered by the barrier
                c.last[tid] = atomicAdd(p.arrived + o.u0, 1u) == (unsigned)o.pieces - 1;
                if (c.last[tid]) atomicExch(p.arrived + o.u0, 0u);
                __threadfence();
            }
            ptx::named_bar_sync(1, SOFT);
            // (K and V of all tiles have been used: O of the last tile has been read)
            float4* buf = reinterpret_cast<float4*>(sm) + warp * S::JOIN * 32;
#pragma unroll 1
            for (int n = 0; n < n_open; ++n) {
                if (!c.last[n]) continue;
                const Open o = c.open[n];                        // join the pieces in their order, a warp per column
#pragma unroll 1
                for (int k = warp; k < o.cols; k += SOFT / 32) {
                    float m, l;
                    const auto at = [&](int u) { return piece_at<S>(p, o.u0, u); };
                    const float4 a = join_pieces<HD, S::JOIN>(at, o.pieces, k * HD, NC * HD + 2 * k, m, l, buf);
                    T* out = (T*)p.a.out + (int64_t)(o.row0 + div_g(p, k)) * p.a.out_stride + (int64_t)(o.g * p.G + mod_g(p, k)) * HD;
                    if (lane < HD / 4) store4(out + lane * 4, a, l);
                    if (p.scores && lane == 0) p.stats[((int64_t)o.g * p.r.n_rows + o.row0) * p.G + k] = make_float2(m, 1.f / l);
                }
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, S::TMEM);
    }
}

// weights[s][g][j] = sum over the sequence's rows and the group's heads of exp2(score - max) / sum: four keys per thread,
// blockDim.x threads side by side (one key per thread took 64 sequences of 4K, one row, from 106 us in all to 125).  With
// blockDim.y > 1 there are that many sums of every so-manieth column, joined in order.
__global__ void __launch_bounds__(512) kv8_weights_kernel(const AttnArgs p) {
    extern __shared__ __align__(16) float4 part[];      // [blockDim.y][blockDim.x]; none for one sum, to fit in beside the attention's CTAs
    grid_dep_launch();
    grid_dep_wait();
    const int x = threadIdx.x, y = threadIdx.y, bx = blockDim.x, by = blockDim.y, g = blockIdx.y;
    const int quad = blockIdx.x * bx + x, t = quad / (TK / 4), j = quad * 4;
    const Seq q = seq_at(p, blockIdx.z);
    if (blockIdx.x * 4 * bx >= q.len || (p.voided && *p.voided)) return;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    if (j < q.len) {
        const float* score = score_of(p, q, g, t, 0) + (j - t * TK);
        const float2* st = p.stats + ((int64_t)g * p.r.n_rows + q.r0) * p.G;
        const int seen = max(0, j - (q.len - q.n)) * p.G, cols = q.n * p.G;      // columns that see key j: [seen, cols)
#pragma unroll 4
        for (int k = seen + y; k < cols; k += by) {
            const float4 s4 = __ldcs(reinterpret_cast<const float4*>(score + (int64_t)k * TK));
            const float2 m = st[k];
            w[0] += s4.x == -INFINITY ? 0.f : exp2_fast(s4.x - m.x) * m.y;
            w[1] += s4.y == -INFINITY ? 0.f : exp2_fast(s4.y - m.x) * m.y;
            w[2] += s4.z == -INFINITY ? 0.f : exp2_fast(s4.z - m.x) * m.y;
            w[3] += s4.w == -INFINITY ? 0.f : exp2_fast(s4.w - m.x) * m.y;
        }
    }
    if (by > 1) {
        part[y * bx + x] = make_float4(w[0], w[1], w[2], w[3]);
        __syncthreads();
        if (y > 0) return;
#pragma unroll 1
        for (int k = 1; k < by; ++k) {
            const float4 o = part[k * bx + x];
            w[0] += o.x;
            w[1] += o.y;
            w[2] += o.z;
            w[3] += o.w;
        }
    }
    float* dst = p.a.weights + ((int64_t)blockIdx.z * p.Hkv + g) * p.a.weights_ld + j;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (j + k < q.len) dst[k] = p.a.add ? dst[k] + w[k] : w[k];
}

template <typename T, typename S>
cudaError_t launch_shape(const Kv8& c, AttnArgs& p, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = smem_limit_once(kv8_attn_kernel<T, S>, S::BYTES, done);
    if (e != cudaSuccess) return e;
    p.QT = S::NC / p.G;
    p.ahead = 2;                         // (64 x 8K decode 102 us with 0, 100 with 1, 98 with 2 and 3)
    p.min_places = 2 + p.ahead;
    const int64_t items = ((int64_t)p.r.n_rows / p.QT + p.q.n) * p.Hkv;
    const int64_t tiles = items * ((p.q.max_len + TK - 1) / TK + 1);
    const int64_t most = (int64_t)c.num_sms * S::CTAS;
    CUtensorMap map;
    memcpy(&map, c.map, sizeof map);
    return launch_ex(c.pdl, kv8_attn_kernel<T, S>, dim3((unsigned)(tiles < most ? tiles : most)), dim3(S::THREADS), S::BYTES, s, map, p);
}

//                           columns, groups, terms of q and P, CTAs per SM, stages
template <int HD> using C4 = Shape<HD, 4, 1, 2, 3, 3, 2>;
template <int HD> using C8 = Shape<HD, 8, 1, 2, 3, 2, 3>;
template <int HD> using C16 = Shape<HD, 16, 2, 2, 3, 2, 2>;
template <int HD> using C32 = Shape<HD, 32, 4, 2, 3, 1, 3>;
template <int HD> using F4 = Shape<HD, 4, 1, 6, 6, 2, 3>;
template <int HD> using F8 = Shape<HD, 8, 1, 6, 6, 2, 2>;

template <int HD> cudaError_t launch_dim(const Kv8& c, AttnArgs& p, cudaStream_t s) {
    // Query columns per item: what a sequence's rows need on average, within what tensor memory holds.  Fewer columns leave
    // room for more CTAs on an SM and shorter tiles, too few double the tiles (64 x 8K, us with shapes of 4 / 8 / 16 / 32: 4 columns
    // 167 / 171 / 188 / 328, 8 columns 322 / 175 / 192 / 334, 16 columns 626 / 328 / 197 / 335).
    const int rows = (p.r.n_rows + p.q.n - 1) / p.q.n, need = rows * p.G;
    if (c.cfg.dtype == CB_BF16) {
        if (need <= 4) return launch_shape<bf16, C4<HD>>(c, p, s);
        if (need <= 8) return launch_shape<bf16, C8<HD>>(c, p, s);
        if (need <= 16) return launch_shape<bf16, C16<HD>>(c, p, s);
        return launch_shape<bf16, C32<HD>>(c, p, s);
    }
    return need <= 4 ? launch_shape<float, F4<HD>>(c, p, s) : launch_shape<float, F8<HD>>(c, p, s);
}

}  // namespace

// scratch: two pieces for every CTA of the largest launch
template <typename S> constexpr size_t pieces() { return (size_t)S::CTAS * 2 * S::PIECE; }
size_t kv8_part_floats(int num_sms) {
    const size_t sizes[] = {pieces<C4<128>>(), pieces<C8<128>>(), pieces<C16<128>>(), pieces<C32<128>>(),
                            pieces<F4<128>>(), pieces<F8<128>>()};
    return std::max(*std::max_element(std::begin(sizes), std::end(sizes)) * num_sms, kv8_rows_part_floats(num_sms));
}
int kv8_most_ctas(int num_sms) { return 3 * num_sms; }

bool kv8_make_map(const Kv8& c, void* out) {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
        return false;
    const cuuint64_t hd = c.cfg.head_dim, rows = (cuuint64_t)c.cfg.n_pages * c.cfg.n_kv_heads * c.cfg.page_size;
    const cuuint64_t dims[3] = {hd, rows, 2ull * c.cfg.n_layers};
    const cuuint64_t strides[2] = {hd, rows * hd};
    const cuuint32_t box[3] = {(cuuint32_t)hd, (cuuint32_t)(c.cfg.page_size < TK ? c.cfg.page_size : TK), 1};
    const cuuint32_t one[3] = {1, 1, 1};
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
               reinterpret_cast<CUtensorMap*>(out), CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c.codes, dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_kv8_attention(const Kv8& c, const Kv8Seqs& q, const Kv8Rows& r, const Kv8Attn& a, int layer,
                                 cudaStream_t s) {
    const int Hkv = c.cfg.n_kv_heads;
    const int64_t blocks = c.cfg.n_pages * Hkv, k0 = (int64_t)layer * 2 * blocks;
    AttnArgs p{};
    p.q = q;
    p.r = r;
    p.a = a;
    p.ks = c.scales + k0;
    p.vs = p.ks + blocks;
    p.Hq = c.cfg.n_heads;
    p.Hkv = Hkv;
    p.G = p.Hq / Hkv;
    p.inv_g = (65536 + p.G - 1) / p.G;
    p.kz = 2 * layer;
    p.box = c.cfg.page_size < TK ? c.cfg.page_size : TK;
    p.part = c.part;
    p.arrived = c.arrived;
    p.voided = r.n_rows > 0 ? c.voided : nullptr;
    p.scores = a.weights && q.max_len > 0 ? c.scores : nullptr;      // (no keys: no weights to return)
    p.stats = c.stats;
    p.score_ld = (q.max_len + TK - 1) / TK * TK;
    if (r.n_rows > 0) {
        const int rows = (r.n_rows + q.n - 1) / q.n;             // of a sequence, on average
        // Up to 32 columns of a sequence stand in one item here, and beyond that keys and values are read and P is formed once
        // per item of 32 (64 sequences of 2K: 32 columns 111 us here, 121 there; 48 columns 205 here, 122 there).
        const bool many = c.cfg.dtype == CB_BF16 && rows * p.G > 32;
        if (many) return launch_kv8_rows(c, &p, s);              // sums its weights too
        const cudaError_t e = c.cfg.head_dim == 128 ? launch_dim<128>(c, p, s) : launch_dim<64>(c, p, s);
        if (e != cudaSuccess) return e;
    }
    if (a.weights && q.max_len > 0) {
        // A block sums 512 keys of a head.  Where those blocks are few and have several columns each, a block has 128 keys and 16
        // sums side by side (64 fp32 rows over 4K: 66 us in all against 115); many blocks fill the SMs as they are (16 sequences, 8
        // rows: 82 us, 114 split).
        const int64_t wide = ((int64_t)q.max_len + 511) / 512;
        const bool few = wide * Hkv * q.n <= c.num_sms && (int64_t)r.n_rows * p.G > 8 * (int64_t)q.n;
        if (few) return launch_ex(c.pdl, kv8_weights_kernel, dim3((q.max_len + 127) / 128, Hkv, q.n), dim3(32, 16), 512 * sizeof(float4), s, p);
        return launch_ex(c.pdl, kv8_weights_kernel, dim3((unsigned)wide, Hkv, q.n), dim3(128), 0, s, p);
    }
    return cudaSuccess;
}

}  // namespace cb
