// Attention over the 8-bit paged K/V cache on the sm_103a tensor cores.  Query row i of a sequence's n sits at position
// len - n + i and sees keys 0 .. that position: out = softmax(q k * scale) v, the G query heads of a group sharing a KV
// head.  A row that sees nothing (its position is negative) gives 0.  With weights, every key gets the sum of its
// softmax weights over the call's query rows and the group's heads.
//
// A decoding step reads every cached byte once and does 4 G FLOPs for it, so it is bound by HBM as long as the codes
// reach the matrix unit without being touched.  They do: tcgen05 kind::f8f6f4 takes e4m3 operands, so the keys are the
// A operand of S^T = K Q^T (M = 128 keys, N = query columns) and the values, read MN-major from the same [key][dim]
// tile, the A operand of O^T = V^T P^T (M = dims, K = 128 keys); block scales multiply S and P in fp32.  With the
// queries in N, a column costs only what it uses: 16 columns for a decoded token where a 128-row tile would waste 120.
//
// q and P are not 8-bit values.  Each is written as a sum of e4m3 numbers c_0 + c_1 / 16 + c_2 / 256 + .., every term the
// rounding of 16 times the residue before it, as columns of their own (column t * NC + c holds term t of column c), and
// the columns of a sum are added in fp32 after the MMA.  A term carries 4 bits: a bf16 q is two terms, exactly; P gets
// three (2^-12 relative), which keeps the result's error well below its bf16 rounding.  fp32 calls use six of each.
// e4m3 products and their fp32 accumulation were checked to be as exact as an fp32 sum of the same products.
//
// Work: an item is (sequence, tile of NC / G query rows, KV head), cut into tiles of 128 keys.  All tiles of all items
// form one list; every CTA takes an equal, contiguous piece of it, so that any mix of lengths is balanced.  An item that
// spans several CTAs is joined by the CTA that finishes last, in the order of the pieces (the result does not depend on
// which one that is).  Which items a CTA has follows from the lengths on the device, so a captured graph stays valid.
//
// Roles: warps 0-3 softmax and output (thread = key, then thread = dim), warp 4 TMA (page by page through the block
// table), warp 5 MMA.  S of the next tile is computed while P of this one is formed; O of a tile is read back from
// tensor memory and added in registers while the next tile's P is formed, which rescales it exactly and makes every
// tile's sum its own.
#include <cudaTypedefs.h>

#include <climits>
#include <cstring>

#include "cb_kv8.cuh"
#include "cb_ptx.cuh"

namespace cb {

namespace {

constexpr int TK = 128;                  // keys per tile
constexpr int SOFT = 128;                // softmax threads
constexpr int THREADS = SOFT + 64;
constexpr int STAGES = 2;                // K and V tiles in flight

struct AttnArgs {
    Kv8Seqs q;
    Kv8Rows r;
    Kv8Attn a;
    const float* ks;                     // this layer's scales [n_pages][Hkv]
    const float* vs;
    int Hq, Hkv, G, QT;                  // QT = query rows per item
    int kz;                              // z coordinate of this layer's K in the map (V is kz + 1)
    int box;                             // rows of a TMA box: min(page_size, 128)
    int min_tiles;                       // tiles per CTA, at least
    float* part;                         // [cta][2][NC][HD + 2] pieces of items that span CTAs
    unsigned* arrived;                   // [cta] pieces finished of the item that begins in this CTA (0 between calls)
    float* scores;                       // weights: [n_q][Hq][score_ld] scores in the exp2 domain
    int score_ld;
    float2* stats;                       // weights: [n_q][Hq] (max, 1 / sum)
};

constexpr int round16(int x) { return (x + 15) / 16 * 16; }
constexpr int pow2_cols(int x) { return x <= 32 ? 32 : x <= 64 ? 64 : x <= 128 ? 128 : x <= 256 ? 256 : 512; }

__device__ __forceinline__ float exp2_fast(float x) {          // special-function unit, about 2 ulp
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

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
__host__ __device__ constexpr uint32_t f8_idesc(int N, bool a_mn) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24) | (a_mn ? 1u << 15 : 0u);   // M = 128
}
// byte `b` of row `row` in that swizzled layout
template <int ROW> __device__ __forceinline__ uint32_t f8_at(uint32_t row, uint32_t b) {
    return ROW == 128 ? row * 128 + ((((b >> 4) ^ row) & 7) << 4) + (b & 15)
                      : row * 64 + ((((b >> 4) ^ (row >> 1)) & 3) << 4) + (b & 15);
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// ------------------------------------------------------------------------------------------------
// the list of tiles
// ------------------------------------------------------------------------------------------------
struct Seq {                             // one sequence: its query rows and length
    int r0, n, len;
    __device__ __forceinline__ int q_tiles(int QT) const { return (n + QT - 1) / QT; }
    // keys that the last row of query tile qt sees
    __device__ __forceinline__ int visible(int qt, int QT) const { return max(0, len - n + min((qt + 1) * QT, n)); }
    __device__ __forceinline__ int tiles(int qt, int QT) const { return max(1, (visible(qt, QT) + TK - 1) / TK); }
};
__device__ __forceinline__ Seq seq_at(const AttnArgs& p, int s) {
    Seq q;
    int r1;
    if (!kv8_rows(p.q, p.r, s, q.r0, r1, q.len)) return Seq{0, 0, 0};
    q.n = r1 - q.r0;
    return q;
}
__device__ __forceinline__ long long seq_tiles(const AttnArgs& p, const Seq& q) {
    long long t = 0;
    for (int qt = 0; qt < q.q_tiles(p.QT); ++qt) t += q.tiles(qt, p.QT);
    return t * p.Hkv;
}

// A position in the list: item (s, qt, g) and tile t of its nt.
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

struct Shared {
    uint64_t k_full[STAGES], v_full[STAGES], empty[STAGES];
    uint64_t s_full[2], s_free[2];
    uint64_t p_full, o_full, q_full, drain;
    uint32_t tmem;
    int abort;
    long long total;                     // tiles of all items
    int s0, qt0, g0, tile0;              // where this CTA begins
    int last;                            // this CTA joins the item
    int prefix[THREADS / 32];
    long long sums[THREADS / 32];
};

// ------------------------------------------------------------------------------------------------
// HD: head_dim; NC: query columns; TQ, TP: terms of q and P
// ------------------------------------------------------------------------------------------------
template <int HD, int NC, int TQ, int TP> struct Shape {
    static constexpr int NQ = round16(TQ * NC), NP = round16(TP * NC);     // MMA columns
    static constexpr int KV_BYTES = TK * HD;
    static constexpr int Q_BYTES = NQ * HD, P_BYTES = NP * TK;
    static constexpr int O_COL = 2 * NQ;
    static constexpr int TMEM = pow2_cols(2 * NQ + NP);
    // K/V stages, Q, P (all 1024-byte aligned), then the softmax exchange and the control block
    static constexpr int OFF_Q = 2 * STAGES * KV_BYTES;
    static constexpr int OFF_P = (OFF_Q + Q_BYTES + 1023) / 1024 * 1024;
    static constexpr int OFF_X = (OFF_P + P_BYTES + 1023) / 1024 * 1024;
    // floats: wmax [2][4][NC], ymax [2][4][NC], qscale [NC], wsum [4][NC], nan_from [HD]
    static constexpr int X_FLOATS = 8 * NC + 8 * NC + NC + 4 * NC + HD;
    static constexpr int OFF_C = (OFF_X + X_FLOATS * 4 + 63) / 64 * 64;
    static constexpr int BYTES = OFF_C + (int)sizeof(Shared) + 1024;       // + alignment of the base
    // CTAs per SM: what registers and tensor memory allow
    static constexpr int CTAS = NC <= 8 && TMEM <= 128 ? 3 : 2;
    static_assert(TMEM * CTAS <= 512 && 2 * NQ + NP <= 512, "tensor memory");
};

template <typename T, int HD, int NC, int TQ, int TP>
__global__ void __launch_bounds__(THREADS, Shape<HD, NC, TQ, TP>::CTAS)
    kv8_attn_kernel(const __grid_constant__ CUtensorMap map, const AttnArgs p) {
    using S = Shape<HD, NC, TQ, TP>;
    constexpr int NQ = S::NQ, NP = S::NP;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sK = sm;                                   // [STAGES][TK][HD]
    uint8_t* sV = sm + STAGES * S::KV_BYTES;
    uint8_t* sQ = sm + S::OFF_Q;
    uint8_t* sP = sm + S::OFF_P;
    float* wmax = reinterpret_cast<float*>(sm + S::OFF_X);
    float* ymax = wmax + 8 * NC;
    float* qscale = ymax + 8 * NC;
    float* wsum = qscale + NC;
    int* nan_from = reinterpret_cast<int*>(wsum + 4 * NC);
    Shared& c = *reinterpret_cast<Shared*>(sm + S::OFF_C);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned* status = p.q.status;
    volatile int* abort = &c.abort;

    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            ptx::mbar_init(ptx::smem_u32(&c.k_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&c.v_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&c.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_u32(&c.s_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&c.s_free[i]), 4);
        }
        ptx::mbar_init(ptx::smem_u32(&c.p_full), 4);
        ptx::mbar_init(ptx::smem_u32(&c.o_full), 1);
        ptx::mbar_init(ptx::smem_u32(&c.q_full), 4);
        ptx::mbar_init(ptx::smem_u32(&c.drain), 1);
        c.abort = 0;
        ptx::fence_barrier_init();
        ptx::prefetch_tmap(&map);
    }
    if (warp == 5) {
        ptx::tmem_alloc(ptx::smem_u32(&c.tmem), S::TMEM);
        ptx::tmem_relinquish();
    }

    // ---- this CTA's piece of the list: two passes over the sequences, THREADS at a time
    {
        long long mine = 0;
        for (int s = tid; s < p.q.n; s += THREADS) mine += seq_tiles(p, seq_at(p, s));
        for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
        if (lane == 0) c.sums[warp] = mine;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    long long total = 0;
    for (int w = 0; w < THREADS / 32; ++w) total += c.sums[w];
    const long long per = max((total + gridDim.x - 1) / gridDim.x, (long long)p.min_tiles);
    const long long t0 = blockIdx.x * per;
    const int count = (int)min(per, max(0ll, total - t0));       // tiles of this CTA
    if (count > 0) {
        long long base = 0;                                      // tiles of the sequences before this step's
        for (int s0 = 0; s0 < p.q.n; s0 += THREADS) {
            const int s = s0 + tid;
            const Seq q = s < p.q.n ? seq_at(p, s) : Seq{0, 0, 0};
            const long long mine = seq_tiles(p, q);
            long long x = mine;
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            __syncthreads();                                     // sums has been read
            if (lane == 31) c.sums[warp] = x;
            __syncthreads();
            long long before = base, all = base;
            for (int w = 0; w < THREADS / 32; ++w) {
                if (w < warp) before += c.sums[w];
                all += c.sums[w];
            }
            before += x - mine;
            if (mine > 0 && before <= t0 && t0 < before + mine) {
                long long left = t0 - before;
                int qt = 0, nt = q.tiles(0, p.QT);
                while (left >= (long long)nt * p.Hkv) {
                    left -= (long long)nt * p.Hkv;
                    nt = q.tiles(++qt, p.QT);
                }
                c.s0 = s;
                c.qt0 = qt;
                c.g0 = (int)(left / nt);
                c.tile0 = (int)(left % nt);
            }
            if (all > t0) break;
            base = all;
        }
        __syncthreads();
    }
    const uint32_t tmem = c.tmem;
    Cursor cur;
    if (count > 0) {
        cur.s = c.s0;
        cur.qt = c.qt0;
        cur.g = c.g0;
        cur.t = c.tile0;
        cur.q = seq_at(p, cur.s);
        cur.settle(p);
    }

    if (warp == 4) {
        // ------------------------------------------------------------------------------------ TMA
        const int boxes = TK / p.box, rows = p.box;              // boxes per tile, one lane each
        const int per_page = 1 << p.q.shift;
        uint32_t issued = 0;
        auto page_of = [&](const Cursor& u) -> int {             // this lane's page (-1: nothing to load)
            const int j = u.t * TK + lane * rows;
            if (lane >= boxes || j >= u.q.len) return -1;
            return kv8_page(p.q, u.s, j >> p.q.shift);
        };
        int page = count > 0 ? page_of(cur) : -1;
        for (int i = 0; i < count; ++i) {
            const int st = i % STAGES;
            const int row = (page * p.Hkv + cur.g) * per_page + ((cur.t * TK + lane * rows) & (per_page - 1));
            const bool load = page >= 0;
            const unsigned who = __ballot_sync(0xffffffffu, load);
            if (i + 1 < count) {                                 // the next tile's pages, before this one's wait
                if (++cur.t == cur.nt) cur.next_item(p);
                page = page_of(cur);
            }
            const bool ok = ptx::mbar_wait(ptx::smem_u32(&c.empty[st]), ((i / STAGES) & 1) ^ 1, abort, status);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t kb = ptx::smem_u32(&c.k_full[st]), vb = ptx::smem_u32(&c.v_full[st]);
            if (lane == 0) {
                const uint32_t bytes = (uint32_t)__popc(who) * rows * HD;
                ptx::mbar_arrive_expect_tx(kb, bytes);
                ptx::mbar_arrive_expect_tx(vb, bytes);
            }
            __syncwarp();
            issued = (uint32_t)(i + 1);
            if (load) tma_3d(ptx::smem_u32(sK + st * S::KV_BYTES + lane * rows * HD), &map, 0, row, p.kz, kb);
            if (load) tma_3d(ptx::smem_u32(sV + st * S::KV_BYTES + lane * rows * HD), &map, 0, row, p.kz + 1, vb);
        }
        // every copy has landed before the CTA may leave
        for (int k = 0; k < STAGES; ++k) {
            if (issued <= (uint32_t)k) continue;
            const uint32_t i = (issued - 1 - k), st = i % STAGES, par = (i / STAGES) & 1;
            int never = 0;
            ptx::mbar_wait(ptx::smem_u32(&c.k_full[st]), par, &never, status);
            ptx::mbar_wait(ptx::smem_u32(&c.v_full[st]), par, &never, status);
        }
    } else if (warp == 5) {
        // ------------------------------------------------------------------------------------ MMA
        if (lane == 0) {
            constexpr uint32_t id_s = f8_idesc(NQ, false), id_o = f8_idesc(NP, true);
            const uint64_t qd = f8_desc<HD>(ptx::smem_u32(sQ), 16), pd = f8_desc<128>(ptx::smem_u32(sP), 16);
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
                    mma_e4m3(tmem + S::O_COL, vd + (uint64_t)(k * 32 * HD >> 4), pd + (uint64_t)(k * 32 >> 4), id_o, k > 0);
                ptx::mma_commit(ptx::smem_u32(&c.empty[st]));
                ptx::mma_commit(ptx::smem_u32(&c.o_full));
                return true;
            };
            for (int i = 0; i < count && ok; ++i) {
                const bool begins = left == 0;                   // an item's first tile waits for its Q, which is
                if (begins) {                                    // written after the item before it is done
                    if (i > 0) {
                        if (!values(i - 1)) break;
                        cur.next_item(p);
                    }
                    left = cur.nt - cur.t;
                    if (!ptx::mbar_wait(ptx::smem_u32(&c.q_full), item & 1, abort, status)) break;
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
                if (!begins) ok = values(i - 1);
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
        const uint32_t my_lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const float to_exp2 = p.a.scale * 1.4426950408889634f;
        int item = 0;
        for (int i = 0; i < count; ++item) {
            const int first = cur.t, n_here = min(cur.nt - first, count - i), g = cur.g, s = cur.s;
            const Seq q = cur.q;
            const int q0 = cur.qt * p.QT, rows = min(p.QT, q.n - q0), cols = rows * p.G;
            const int pos0 = q.len - q.n + q0;                   // position of the item's first query row
            const T* qbase = (const T*)p.a.q + (int64_t)(q.r0 + q0) * p.a.q_stride + (int64_t)g * p.G * HD;

            auto page_of = [&](int t) -> int {                   // page of this thread's key in tile t of the item
                const int j = t * TK + tid;
                return t < first + n_here && j < q.len ? kv8_page(p.q, s, j >> p.q.shift) : -1;
            };
            int page = page_of(first), page_next = page_of(first + 1);
            float ksc = page >= 0 ? p.ks[(int64_t)page * p.Hkv + g] : 0.f, vsc = page >= 0 ? p.vs[(int64_t)page * p.Hkv + g] : 0.f;

            // Q as terms: column r = (query row, head of the group), lane = HD / 32 of its dims
            for (int r = warp; r < NC; r += 4) {
                constexpr int E = HD / 32;
                float x[E];
                float top = 0.f;
                const T* src = qbase + (int64_t)(r / p.G) * p.a.q_stride + (r % p.G) * HD + lane * E;
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    x[k] = r < cols ? to_f(src[k]) : 0.f;
                    top = fmaxf(top, kv8_mag(x[k]));
                }
                const float sc = kv8_scale(warp_max(top)), inv = kv8_inverse(sc);
#pragma unroll
                for (int k = 0; k < E; ++k) x[k] = kv8_nan_inf(x[k]) * inv;
#pragma unroll
                for (int t = 0; t < TQ; ++t) {
                    uint32_t w = 0;
#pragma unroll
                    for (int k = 0; k < E; k += 2) {
                        const uint32_t c2 = kv8_code2(x[k], x[k + 1]);
                        const float2 v = kv8_value2(c2);
                        x[k] = (x[k] - v.x) * 16.f;
                        x[k + 1] = (x[k + 1] - v.y) * 16.f;
                        w |= c2 << (8 * k);
                    }
                    uint8_t* d = sQ + f8_at<HD>(t * NC + r, lane * E);
                    if (E == 4) *reinterpret_cast<uint32_t*>(d) = w;
                    else *reinterpret_cast<uint16_t*>(d) = (uint16_t)w;
                }
                if (lane == 0) qscale[r] = sc * to_exp2;
            }
            if (tid < HD) nan_from[tid] = INT_MAX;
            fence_async_smem();
            ptx::named_bar_sync(1, SOFT);
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&c.q_full));

            float acc[NC], lsum[NC], mrun[NC], alpha[NC], oscale[NC];
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                acc[k] = 0.f;
                lsum[k] = 0.f;
                mrun[k] = -INFINITY;
                alpha[k] = 1.f;
                oscale[k] = 0.f;
            }
            // acc = acc * alpha + O of the tile before
            auto add_tile = [&](int done) {
                ptx::mbar_wait(ptx::smem_u32(&c.o_full), done & 1, abort, status);
                ptx::tc_fence_after();
                uint32_t o[NP];
#pragma unroll
                for (int k = 0; k < NP; k += 16) ptx::tmem_ld16_issue(my_lanes + S::O_COL + k, o + k);
#pragma unroll
                for (int k = 0; k < NP; k += 16) ptx::tmem_ld_wait16(o + k);
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    float v = __uint_as_float(o[(TP - 1) * NC + k]);
#pragma unroll
                    for (int t = TP - 2; t >= 0; --t) v = fmaf(v, 0.0625f, __uint_as_float(o[t * NC + k]));
                    acc[k] = fmaf(v, oscale[k], acc[k] * alpha[k]);
                }
            };

            for (int t = first; t < first + n_here; ++t, ++i) {
                const int b = i & 1, j = t * TK + tid;
                const bool have = page >= 0;
                const float ks_now = ksc, vs_now = vsc;
                // the next tile's scales and the page after it, while this one is worked on
                page = page_next;
                page_next = page_of(t + 2);
                ksc = page >= 0 ? p.ks[(int64_t)page * p.Hkv + g] : 0.f;
                vsc = page >= 0 ? p.vs[(int64_t)page * p.Hkv + g] : 0.f;

                ptx::mbar_wait(ptx::smem_u32(&c.s_full[b]), (i >> 1) & 1, abort, status);
                ptx::tc_fence_after();
                float x[NC];
                {
                    uint32_t w[NQ];
#pragma unroll
                    for (int k = 0; k < NQ; k += 16) ptx::tmem_ld16_issue(my_lanes + b * NQ + k, w + k);
#pragma unroll
                    for (int k = 0; k < NQ; k += 16) ptx::tmem_ld_wait16(w + k);
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&c.s_free[b]));
#pragma unroll
                    for (int k = 0; k < NC; ++k) {
                        float v = __uint_as_float(w[(TQ - 1) * NC + k]);
#pragma unroll
                        for (int n = TQ - 2; n >= 0; --n) v = fmaf(v, 0.0625f, __uint_as_float(w[n * NC + k]));
                        x[k] = v * (ks_now * qscale[k]);
                    }
                }
                // column k (query row k / G) sees key j from its own position on: k >= (j - pos0) G
                const int hidden = have ? min(max(j - pos0, 0), NC) * p.G : NC;
                if (hidden > 0) {
#pragma unroll
                    for (int k = 0; k < NC; ++k)
                        if (k < hidden) x[k] = -INFINITY;
                }
                if (p.scores) {
#pragma unroll
                    for (int k = 0; k < NC; ++k)
                        if (k < cols)
                            p.scores[((int64_t)(q.r0 + q0 + k / p.G) * p.Hq + g * p.G + k % p.G) * p.score_ld + j] = x[k];
                }
                // maxima over the tile's keys of the scores, and of scores with V's scale: y = x + log2(scale), which says
                // how far a column's P can be scaled up.  A warp's keys lie in one block unless pages have 16 rows.
                float* wm = wmax + b * 4 * NC;
                float* wy = ymax + b * 4 * NC;
                const float ev = have && vs_now > 0.f ? (float)((int)(__float_as_uint(vs_now) >> 23) - 127) : -INFINITY;
                if (p.box >= 32) {
                    const float ew = redux_max(ev);
#pragma unroll
                    for (int k = 0; k < NC; ++k) {
                        const float m = redux_max(x[k]);
                        if (lane == 0) {
                            wm[warp * NC + k] = m;
                            wy[warp * NC + k] = m + ew;
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < NC; ++k) {
                        const float m = redux_max(x[k]), y = redux_max(x[k] + ev);
                        if (lane == 0) {
                            wm[warp * NC + k] = m;
                            wy[warp * NC + k] = y;
                        }
                    }
                }
                ptx::named_bar_sync(1, SOFT);
                float a_now[NC], os_now[NC];
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    const float mt = fmaxf(fmaxf(wm[k], wm[NC + k]), fmaxf(wm[2 * NC + k], wm[3 * NC + k]));
                    const float yt = fmaxf(fmaxf(wy[k], wy[NC + k]), fmaxf(wy[2 * NC + k], wy[3 * NC + k]));
                    const float mn = fmaxf(mrun[k], mt), ref = mn == -INFINITY ? 0.f : mn;
                    a_now[k] = mn == mrun[k] ? 1.f : exp2_fast(mrun[k] - ref);
                    mrun[k] = mn;
                    const float e = exp2_fast(x[k] - ref);
                    lsum[k] = fmaf(lsum[k], a_now[k], e);
                    // P of the column times V's scale, scaled by the power of two that brings its largest value to 128 .. 256
                    const int up = 8 + (yt == -INFINITY ? 0 : (int)floorf(fminf(fmaxf(ref - yt, -118.f), 118.f)));
                    x[k] = e * (have ? vs_now * __uint_as_float((unsigned)(127 + up) << 23) : 0.f);
                    os_now[k] = __uint_as_float((unsigned)(127 - up) << 23);
                }
                if (t > first) add_tile(i - 1);
                // P as terms, one byte per column and term (sP is free: O of the tile before is complete)
#pragma unroll
                for (int k = 0; k < NC; k += 2) {
                    alpha[k] = a_now[k];
                    alpha[k + 1] = a_now[k + 1];
                    oscale[k] = os_now[k];
                    oscale[k + 1] = os_now[k + 1];
#pragma unroll
                    for (int n = 0; n < TP; ++n) {
                        const uint32_t c2 = kv8_code2(x[k], x[k + 1]);
                        const float2 v = kv8_value2(c2);
                        x[k] = (x[k] - v.x) * 16.f;
                        x[k + 1] = (x[k + 1] - v.y) * 16.f;
                        sP[f8_at<TK>(n * NC + k, tid)] = (uint8_t)c2;
                        sP[f8_at<TK>(n * NC + k + 1, tid)] = (uint8_t)(c2 >> 8);
                    }
                }
                // V rows that no weight may meet: one that was not loaded or lies behind the sequence is zeroed (0 times
                // NaN would be NaN); in one that only later query rows see, NaN codes are taken out and remembered
                if (!have || (j > pos0 && q.n > 1)) {
                    const int st = i % STAGES;
                    ptx::mbar_wait(ptx::smem_u32(&c.v_full[st]), (i / STAGES) & 1, abort, status);
                    uint8_t* row = sV + st * S::KV_BYTES;
                    for (int d = 0; d < HD; d += 16) {
                        uint4* v = reinterpret_cast<uint4*>(row + f8_at<HD>(tid, d));
                        if (!have) {
                            *v = make_uint4(0, 0, 0, 0);
                        } else {
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
                }
                fence_async_smem();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&c.p_full));
            }
            add_tile(i - 1);
            ptx::tc_fence_before();
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const float v = warp_sum(lsum[k]);
                if (lane == 0) wsum[warp * NC + k] = v;
            }
            ptx::named_bar_sync(1, SOFT);
#pragma unroll
            for (int k = 0; k < NC; ++k) lsum[k] = (wsum[k] + wsum[NC + k]) + (wsum[2 * NC + k] + wsum[3 * NC + k]);
            if (tid < HD && nan_from[tid] != INT_MAX) {
                const int k0 = (nan_from[tid] - pos0) * p.G;     // columns from the row that sees the NaN on
#pragma unroll
                for (int k = 0; k < NC; ++k)
                    if (k >= k0) acc[k] = __int_as_float(0x7fc00000);
            }
            bool mine = true;                                    // this CTA writes the item's result
            if (first > 0 || first + n_here < cur.nt) {
                constexpr int PIECE = NC * (HD + 2);
                const long long begin = t0 + (i - n_here) - first;           // the item's first tile in the list
                const int c_first = (int)(begin / per), c_last = (int)((begin + cur.nt - 1) / per);
                float* piece = p.part + (int64_t)(blockIdx.x * 2 + (first > 0 ? 0 : 1)) * PIECE;
                if (tid < HD) {
#pragma unroll
                    for (int k = 0; k < NC; ++k) piece[k * HD + tid] = acc[k];
                }
                if (tid == 0) {
#pragma unroll
                    for (int k = 0; k < NC; ++k) {
                        piece[NC * HD + 2 * k] = mrun[k];
                        piece[NC * HD + 2 * k + 1] = lsum[k];
                    }
                }
                __threadfence();
                ptx::named_bar_sync(1, SOFT);
                if (tid == 0) {
                    const unsigned n = (unsigned)(c_last - c_first + 1);
                    c.last = atomicAdd(p.arrived + c_first, 1u) == n - 1;
                    if (c.last) atomicExch(p.arrived + c_first, 0u);
                    __threadfence();
                }
                ptx::named_bar_sync(1, SOFT);
                mine = c.last != 0;
                if (mine) {                                      // join the pieces in their order
#pragma unroll
                    for (int k = 0; k < NC; ++k) {
                        acc[k] = 0.f;
                        lsum[k] = 0.f;
                        mrun[k] = -INFINITY;
                    }
                    for (int u = c_first; u <= c_last; ++u) {
                        const float* o = p.part + (int64_t)(u * 2 + (u == c_first ? 1 : 0)) * PIECE;
#pragma unroll
                        for (int k = 0; k < NC; ++k) mrun[k] = fmaxf(mrun[k], __ldcg(o + NC * HD + 2 * k));
                    }
                    for (int u = c_first; u <= c_last; ++u) {
                        const float* o = p.part + (int64_t)(u * 2 + (u == c_first ? 1 : 0)) * PIECE;
#pragma unroll
                        for (int k = 0; k < NC; ++k) {
                            const float2 ml = __ldcg(reinterpret_cast<const float2*>(o + NC * HD + 2 * k));
                            const float f = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - mrun[k]);
                            lsum[k] = fmaf(ml.y, f, lsum[k]);
                            if (tid < HD) acc[k] = fmaf(__ldcg(o + k * HD + tid), f, acc[k]);
                        }
                    }
                }
            }
            if (mine) {
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    if (k >= cols) continue;
                    const int row = k / p.G, h = k % p.G;
                    const float inv = 1.f / lsum[k];
                    if (tid < HD)
                        ((T*)p.a.out)[(int64_t)(q.r0 + q0 + row) * p.a.out_stride + (int64_t)(g * p.G + h) * HD + tid] =
                            from_f<T>(pos0 + row >= 0 ? acc[k] * inv : 0.f);
                    if (p.scores && tid == 0)
                        p.stats[(int64_t)(q.r0 + q0 + row) * p.Hq + g * p.G + h] = make_float2(mrun[k], inv);
                }
            }
            if (i < count) cur.next_item(p);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, S::TMEM);
    }
}

// weights[s][g][j] = sum over the sequence's rows and the group's heads of exp2(score - max) / sum, in row order
__global__ void __launch_bounds__(128) kv8_weights_kernel(const AttnArgs p) {
    const int j = blockIdx.x * 128 + threadIdx.x, g = blockIdx.y;
    const Seq q = seq_at(p, blockIdx.z);
    if (j >= q.len) return;
    float w = 0.f;
    for (int i = max(0, j - (q.len - q.n)); i < q.n; ++i) {
        const int64_t at = (int64_t)(q.r0 + i) * p.Hq + g * p.G;
        for (int h = 0; h < p.G; ++h) {
            const float x = p.scores[(at + h) * p.score_ld + j];
            const float2 st = p.stats[at + h];
            w += x == -INFINITY ? 0.f : exp2_fast(x - st.x) * st.y;
        }
    }
    float* dst = p.a.weights + ((int64_t)blockIdx.z * p.Hkv + g) * p.a.weights_ld + j;
    *dst = p.a.add ? *dst + w : w;
}

template <typename T, int HD, int NC, int TQ, int TP>
cudaError_t launch_shape(const Kv8& c, AttnArgs& p, cudaStream_t s) {
    using S = Shape<HD, NC, TQ, TP>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = smem_limit_once(kv8_attn_kernel<T, HD, NC, TQ, TP>, S::BYTES, done);
    if (e != cudaSuccess) return e;
    p.QT = NC / p.G;
    const int64_t items = ((int64_t)p.r.n_rows / p.QT + p.q.n) * p.Hkv;
    const int64_t tiles = items * ((p.q.max_len + TK - 1) / TK + 1);
    const int64_t most = (int64_t)c.num_sms * S::CTAS;
    CUtensorMap map;
    memcpy(&map, c.map, sizeof map);
    kv8_attn_kernel<T, HD, NC, TQ, TP><<<(int)(tiles < most ? tiles : most), THREADS, S::BYTES, s>>>(map, p);
    return cudaGetLastError();
}

template <int HD> cudaError_t launch_dim(const Kv8& c, AttnArgs& p, cudaStream_t s) {
    // query columns per item: what a sequence's rows need on average, within what tensor memory holds
    const int rows = (p.r.n_rows + p.q.n - 1) / p.q.n, need = rows * p.G;
    if (c.cfg.dtype == CB_BF16) {
        if (need <= 4) return launch_shape<bf16, HD, 4, 2, 3>(c, p, s);
        if (need <= 8) return launch_shape<bf16, HD, 8, 2, 3>(c, p, s);
        if (need <= 16) return launch_shape<bf16, HD, 16, 2, 3>(c, p, s);
        return launch_shape<bf16, HD, 32, 2, 3>(c, p, s);
    }
    return need <= 4 ? launch_shape<float, HD, 4, 6, 6>(c, p, s) : launch_shape<float, HD, 8, 6, 6>(c, p, s);
}

}  // namespace

size_t kv8_part_floats(int num_sms) {
    size_t most = 0;
    const size_t shapes[][2] = {{3, 8}, {2, 16}, {2, 32}};               // CTAs per SM, columns
    for (auto& s : shapes) most = s[0] * s[1] > most ? s[0] * s[1] : most;
    return most * num_sms * 2 * (128 + 2);
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
    p.kz = 2 * layer;
    p.box = c.cfg.page_size < TK ? c.cfg.page_size : TK;
    p.min_tiles = 2;
    p.part = c.part;
    p.arrived = c.arrived;
    p.scores = a.weights ? c.scores : nullptr;
    p.stats = c.stats;
    p.score_ld = (q.max_len + TK - 1) / TK * TK;
    if (r.n_rows > 0) {
        const cudaError_t e = c.cfg.head_dim == 128 ? launch_dim<128>(c, p, s) : launch_dim<64>(c, p, s);
        if (e != cudaSuccess) return e;
    }
    if (a.weights && q.max_len > 0)
        kv8_weights_kernel<<<dim3((q.max_len + 127) / 128, Hkv, q.n), 128, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace cb
