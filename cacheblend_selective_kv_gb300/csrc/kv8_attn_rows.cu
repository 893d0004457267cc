// Attention over the 8-bit paged K/V cache for many query rows per sequence (a query over a blended context, a prompt in
// pieces): bf16 queries, an item's 128 rows = 128 / G query rows x the G heads of their group in the lanes of tensor memory.
//
// With this many rows a tile of keys is used often enough to widen it once: eight warps turn the codes that TMA has brought
// into shared memory into fp16 (exact, without the block scales), in the swizzled layouts of the MMA operands, and
// S = Q K^T, O += P V run on kind::f16.  Against the e4m3 terms of kv8_attn.cu this costs a conversion per cached value and
// tile, and saves the terms of q and P for each of 128 rows and the maxima over keys in other threads (a row is one
// thread's).  Q is brought to fp16 by a power of two per row that puts its largest value at 2^14 .. 2^15: exact down to
// 2^-29 of that.  P is fp16: 11 bits, 2^-12 relative.  Block scales hold for 16 keys at least: K's multiplies the scores
// of a block together with the constants of the softmax, V's multiplies P.
//
// V's block scales differ, so P carries them: p_j = 2^(x_j - R) s_j with x the score in the exp2 domain, s_j the scale of
// key j's block and R a reference of the row no more than 2^8 below the largest x_j + log2 s_j so far.  It grows lazily (O
// is rescaled in tensor memory when it must), which keeps P within fp16.  A scale below 2^-100 counts as 2^-100 for R.
//
// The softmax sum takes 2^(x_j - X) in fp32.  X is R as long as R lies up to 30 below the row's largest score M, which it
// does for scales of 2^-30 to 1, and follows M otherwise: a key's weight in the sum has nothing to do with its V, and
// with R as its reference the weights of keys of small V would vanish beside a V that is 2^126 times larger, or all of
// them before a V of 2^100.  X is max(min(R, M), R - 60, M - 30): near enough to M for the sum, near enough to R for
// the factor 2^(R - X) between O and the sum.  It only grows, as R and M do.
//
// Each of the two halves of a tile's keys has its own R, X, sum and O (as the blend's attention kernel does, so that the
// warps of a row need not meet for every tile); they are joined at the end of an item, relative to X.
//
// Per tile and SM: 32 MMAs of 128 x 128 x 16 at about 99 cycles, 128 x 128 exponentials, 2 x 128 x HD conversions; about
// 3600 cycles a tile, bound by the softmax warps' chain (two warps a scheduler, 1.2 instructions a cycle) and not by the
// matrix unit.  2048 rows over 8K: 352 us, 36 % of the measured bf16 rate; the 64 rows of a query over 8K: 29.5 us, 45 us
// with weights (with four warps that widen: 371, 32 and 48).
#include <cstring>

#include "cb_kv8_attn.cuh"

namespace cb {

namespace {

constexpr int ROWS = 128;
constexpr int SOFT = 256, CONV = 256, THREADS = SOFT + CONV + 64;
constexpr int CONV_WARP = SOFT / 32, MMA_WARP = CONV_WARP + CONV / 32, TMA_WARP = MMA_WARP + 1;
constexpr int HK = 64;                   // keys of a half
constexpr int MARKS = 4;                 // items whose row scales and NaN marks are kept; tiles whose conversion is announced
constexpr int RING = 16;                 // tiles whose block scales are kept
constexpr int KT = 2, VT = 1;            // tiles of K and V codes
constexpr float GROW = 8.f;              // how far (log2) P may outgrow its reference
constexpr float SLACK = 38.f;            // how far (log2) a term of the sum may get above 1
constexpr float P_UP = 128.f;            // P is stored this much larger: its largest values are 2^7 .. 2^15 of fp16's 2^16

struct Todo {                            // an item that begins in a CTA and ends in another: its rows and pieces
    int row0, cols, g, pieces;
};

struct RowsShared {
    uint64_t kc_full[KT], kc_empty[KT], vc_full[VT], vc_empty[VT];          // codes
    uint64_t k_full[2], k_empty[2], v_full[2], pv_done[2], s_full[2], p_full[2];
    uint64_t rows_full[MARKS];           // an item's row scales are written
    uint64_t v_seen[MARKS];              // a tile's V is converted, its NaN marked
    uint64_t q_full, o_free, drain;
    ScaleRing<RING> ring;
    uint32_t tmem;
    int abort;
    Find find;
    int any_nan[MARKS];                  // an item's V held NaN that not all of its rows see
};

template <int HD> struct Rows {
    static constexpr int TILE = TK * HD * 2, CODES = TK * HD;    // a K or V tile, or Q, in fp16; a tile of codes
    static constexpr int OFF_K = TILE, OFF_V = 3 * TILE, OFF_KC = 5 * TILE, OFF_VC = OFF_KC + KT * CODES;
    static constexpr int OFF_X = OFF_VC + VT * CODES;
    // floats: row scales [MARKS][ROWS], (X, sum, R, -) [2][ROWS][4]; ints: nan_from [MARKS][HD]
    static constexpr int X_FLOATS = MARKS * ROWS + 8 * ROWS + MARKS * HD;
    static constexpr int OFF_C = OFF_X + X_FLOATS * 4;
    static constexpr int BYTES = OFF_C + (int)sizeof(RowsShared);
    static constexpr int PIECE = ROWS * (HD + 2);
    static_assert(BYTES <= 227 * 1024, "shared memory");
};

// a swizzled tile: halves of 64 elements (128 bytes) of the row, 128 rows each
__device__ __forceinline__ uint32_t wide_at(int row, int chunk) {           // 16-byte chunk of 8 elements
    return (chunk >> 3) * (TK * 128) + row * 128 + (((chunk ^ row) & 7) << 4);
}
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr) {               // MN-major, the next 64 columns TK * 128 on
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((TK * 128) >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma_f16_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tmem_st8_words(uint32_t addr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
    const __half2 t = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ uint32_t half2_word(const __half2& h) { return *reinterpret_cast<const uint32_t*>(&h); }

// Scores of a tile of keys: [TK / 4][columns], four keys each.  A thread has a row's scores, so that neighbouring threads
// write next to each other (a row's scores side by side had every store touch 32 sectors).
__device__ __forceinline__ float4* quads_of(const AttnArgs& p, const Seq& q, int g, int t) {
    return reinterpret_cast<float4*>(score_of(p, q, g, t, 0));
}

// NaN codes out of 16 codes of a V row that not all query rows see, and row j noted as the first to hold one in those dims
__device__ __noinline__ void take_nan(uint4& x, int j, int* marks, int* any) {
    uint32_t cw[4] = {x.x, x.y, x.z, x.w};
    for (int k = 0; k < 4; ++k) {
        const uint32_t bad = __vcmpeq4(cw[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        if (bad == 0) continue;
        cw[k] &= ~bad;
        for (int y = 0; y < 4; ++y)
            if (bad >> (8 * y) & 1) atomicMin(marks + 4 * k + y, j);
        *any = 1;
    }
    x = make_uint4(cw[0], cw[1], cw[2], cw[3]);
}

template <int HD, bool SCORES>
__global__ void __launch_bounds__(THREADS, 1) kv8_rows_kernel(const __grid_constant__ CUtensorMap map, const AttnArgs p) {
    using S = Rows<HD>;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint8_t* sQ = sm;
    uint8_t* sK = sm + S::OFF_K;                        // [2]
    uint8_t* sV = sm + S::OFF_V;                        // [2]
    float* row_scale = reinterpret_cast<float*>(sm + S::OFF_X);
    float* halves = row_scale + MARKS * ROWS;
    int* nan_marks = reinterpret_cast<int*>(halves + 8 * ROWS);
    RowsShared& c = *reinterpret_cast<RowsShared*>(sm + S::OFF_C);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned* status = p.q.status;
    volatile int* abort = &c.abort;
    if (ptx::smem_u32(sm) & 1023) {
        if (tid == 0) atomicOr(status, ST_WAIT_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_u32(&c.k_full[i]), CONV / 32);
            ptx::mbar_init(ptx::smem_u32(&c.k_empty[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&c.v_full[i]), CONV / 32);
            ptx::mbar_init(ptx::smem_u32(&c.pv_done[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&c.s_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&c.p_full[i]), SOFT / 32);
        }
        for (int i = 0; i < KT; ++i) {
            ptx::mbar_init(ptx::smem_u32(&c.kc_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&c.kc_empty[i]), CONV / 32);
        }
        for (int i = 0; i < VT; ++i) {
            ptx::mbar_init(ptx::smem_u32(&c.vc_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&c.vc_empty[i]), CONV / 32);
        }
        for (int i = 0; i < MARKS; ++i) {
            ptx::mbar_init(ptx::smem_u32(&c.rows_full[i]), CONV / 32);
            ptx::mbar_init(ptx::smem_u32(&c.v_seen[i]), CONV / 32);
            c.any_nan[i] = 0;
        }
        for (int i = 0; i < RING; ++i) ptx::mbar_init(ptx::smem_u32(&c.ring.full[i]), TK / p.box);
        ptx::mbar_init(ptx::smem_u32(&c.q_full), CONV / 32);
        ptx::mbar_init(ptx::smem_u32(&c.o_free), SOFT / 32);
        ptx::mbar_init(ptx::smem_u32(&c.drain), 1);
        c.abort = 0;
        ptx::fence_barrier_init();
        ptx::prefetch_tmap(&map);
    }
    if (warp == MMA_WARP) {
        ptx::tmem_alloc(ptx::smem_u32(&c.tmem), 512);
        ptx::tmem_relinquish();
    }
    grid_dep_launch();
    grid_dep_wait();
    Piece mine;
    Cursor cur;
    find_piece<THREADS>(p, c.find, mine, cur, [] { ptx::tc_fence_before(); }, [] { ptx::tc_fence_after(); });
    const int count = mine.count;
    const uint32_t tmem = c.tmem;                       // S and P: two buffers of 128 columns; O of each half at 256
    constexpr uint32_t O_COL = 256;

    if (warp >= CONV_WARP && warp < MMA_WARP) {
        // ------------------------------------------------------------------------------------ codes to fp16
        // Like the softmax warps, these run on to their last tile when a wait has given up.
        constexpr int LPR = HD / 16, RPW = 32 / LPR, NI = TK / (CONV / 32 * RPW);           // lanes per row, rows per warp and step, steps
        const int w = warp - CONV_WARP, t = tid - SOFT, e = lane % LPR, row0 = w * RPW + lane / LPR;
        const int box_shift = min(p.q.shift, 7);
        int item = -1;
        bool begins = true;
        for (int i = 0; i < count; ++i) {
            const int st = i & 1;
            const uint32_t par = ((i >> 1) & 1) ^ 1;
            const Seq q = cur.q;
            const int q0 = cur.qt * p.QT, cols = min(p.QT, q.n - q0) * p.G, pos0 = q.len - q.n + q0, tile = cur.t;
            if (begins) {
                ++item;
                const bf16* qbase = (const bf16*)p.a.q + (int64_t)(q.r0 + q0) * p.a.q_stride + (int64_t)cur.g * p.G * HD;
                constexpr int QL = HD / 8, QR = 32 / QL;         // lanes of a row (8 values each), rows of a warp
                // Once the products with the item before's Q are done; then the softmax is past tile i - 3, hence past the item
                // whose marks and row scales these were.  Q lands where it will stand and is converted in place, by the thread
                // that has asked for it (all of it under way at once; two rows ahead in registers cost an item 1.5 us more).
                if (i > 0) ptx::mbar_wait(ptx::smem_u32(&c.k_empty[(i - 1) & 1]), ((i - 1) >> 1) & 1, abort, status);
                const int r0 = w * QR + lane / QL;
#pragma unroll 1
                for (int r = r0; r < ROWS; r += CONV / 32 * QR) {
                    uint8_t* to = sQ + wide_at(r, lane % QL);
                    if (r < cols) cp_async16(ptx::smem_u32(to), qbase + (int64_t)div_g(p, r) * p.a.q_stride + mod_g(p, r) * HD + lane % QL * 8);
                    else *reinterpret_cast<uint4*>(to) = make_uint4(0, 0, 0, 0);
                }
                if (t < HD) nan_marks[(item % MARKS) * HD + t] = INT_MAX;
                if (t == 0) c.any_nan[item % MARKS] = 0;
                asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
                for (int r = r0; r < ROWS; r += CONV / 32 * QR) {
                    uint4* at = reinterpret_cast<uint4*>(sQ + wide_at(r, lane % QL));
                    const uint4 val = *at;
                    const uint32_t word[4] = {val.x, val.y, val.z, val.w};
                    float f[8], top = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        f[2 * k] = __uint_as_float(word[k] << 16);
                        f[2 * k + 1] = __uint_as_float(word[k] & 0xffff0000u);
                        top = fmaxf(top, fmaxf(kv8_mag(f[2 * k]), kv8_mag(f[2 * k + 1])));
                    }
#pragma unroll
                    for (int o = QL / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    // kv8_scale brings the largest value to 224 .. 448; 2^6 more is 2^14 .. 2^15 less a little (the softmax's
                    // scale gives its sign, and nothing when it is 0).  An infinity counts as NaN: it could give scores of -inf
                    // alone, which is how a row that sees nothing looks.
                    // (not below 2^-119, so that 1 / scale * 2^6 stays finite)
                    const float sc = top > 0.f ? fmaxf(kv8_scale(top), 1.5046328e-36f) : 0.f;
                    const float up = kv8_inverse(sc) * (p.a.scale < 0.f ? -64.f : p.a.scale > 0.f ? 64.f : 0.f);
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[k] = f16_pair(kv8_nan_inf(f[2 * k]) * up, kv8_nan_inf(f[2 * k + 1]) * up);
                    *at = make_uint4(o[0], o[1], o[2], o[3]);
                    if (lane % QL == 0) row_scale[(item % MARKS) * ROWS + r] = sc * (1.f / 64.f);
                }
                fence_async_smem();
                ptx::named_bar_sync(2, CONV);                    // also: the marks
                if (lane == 0) {
                    ptx::mbar_arrive(ptx::smem_u32(&c.q_full));
                    ptx::mbar_arrive(ptx::smem_u32(&c.rows_full[item % MARKS]));
                }
            }
            const auto widen = [&](uint8_t* to, int row, const uint4& x) {
                const uint32_t cw[4] = {x.x, x.y, x.z, x.w};
                uint32_t o[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    o[2 * k] = half2_word(kv8_half2(cw[k]));
                    o[2 * k + 1] = half2_word(kv8_half2(cw[k] >> 16));
                }
                *reinterpret_cast<uint4*>(to + wide_at(row, 2 * e)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(to + wide_at(row, 2 * e + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
            };
            // K: free once S of two tiles before is done (rows that are not loaded stay as they were: their scores are masked)
            ptx::mbar_wait(ptx::smem_u32(&c.kc_full[i % KT]), (i / KT) & 1, abort, status);
            ptx::mbar_wait(ptx::smem_u32(&c.k_empty[st]), par, abort, status);
#pragma unroll 1
            for (int n = 0; n < NI; ++n) {
                const int row = row0 + n * CONV / 32 * RPW;
                widen(sK + st * S::TILE, row, *reinterpret_cast<const uint4*>(sm + S::OFF_KC + (i % KT) * S::CODES + f8_at<HD>(row, e * 16)));
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(ptx::smem_u32(&c.k_full[st]));
                ptx::mbar_arrive(ptx::smem_u32(&c.kc_empty[i % KT]));
            }
            begins = false;
            if (i + 1 < count && ++cur.t == cur.nt) {
                cur.next_item(p);
                begins = true;
            }
            // V: zero where nothing is loaded or behind the sequence; a NaN that only later rows see is taken out and remembered
            ptx::mbar_wait(ptx::smem_u32(&c.ring.full[i % RING]), (i / RING) & 1, abort, status);
            ptx::mbar_wait(ptx::smem_u32(&c.vc_full[i % VT]), (i / VT) & 1, abort, status);
            ptx::mbar_wait(ptx::smem_u32(&c.pv_done[st]), par, abort, status);
            const float* loaded = c.ring.scale[i % RING][0];
            const bool plain = (tile + 1) * TK <= min(q.len, pos0 + 1) &&
                               !__any_sync(0xffffffffu, lane < (TK >> box_shift) && loaded[lane] < 0.f);
            const auto codes_of = [&](int row) {
                return *reinterpret_cast<const uint4*>(sm + S::OFF_VC + (i % VT) * S::CODES + f8_at<HD>(row, e * 16));
            };
            if (plain) {
#pragma unroll 1
                for (int n = 0; n < NI; ++n) widen(sV + st * S::TILE, row0 + n * CONV / 32 * RPW, codes_of(row0 + n * CONV / 32 * RPW));
            } else {
#pragma unroll 1
                for (int n = 0; n < NI; ++n) {
                    const int row = row0 + n * CONV / 32 * RPW, j = tile * TK + row;
                    uint4 x = codes_of(row);
                    if (j >= q.len || loaded[row >> box_shift] < 0.f) x = make_uint4(0, 0, 0, 0);
                    else if (j > pos0) take_nan(x, j, nan_marks + (item % MARKS) * HD + e * 16, &c.any_nan[item % MARKS]);
                    widen(sV + st * S::TILE, row, x);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(ptx::smem_u32(&c.v_full[st]));
                ptx::mbar_arrive(ptx::smem_u32(&c.vc_empty[i % VT]));
                ptx::mbar_arrive(ptx::smem_u32(&c.v_seen[i % MARKS]));
            }
        }
    } else if (warp == TMA_WARP) {
        // ------------------------------------------------------------------------------------ TMA
        // A scale slot is free again without a barrier of its own: K's codes of tile i - 1 waited for the conversion of tile
        // i - 1 - KT, which waited for S of two tiles before, which waited for P V of two before that.
        static_assert(RING - LOOK >= KT + 1 + 2 + 2, "scale ring");
        produce_tiles<HD, KT, VT>(p, map, cur, count, sm + S::OFF_KC, sm + S::OFF_VC, c.kc_full, c.kc_empty, c.vc_full, c.vc_empty, c.ring, abort);
    } else if (warp == MMA_WARP) {
        // ------------------------------------------------------------------------------------ MMA
        if (lane == 0) {
            constexpr uint32_t id_s = (1u << 4) | ((uint32_t)(TK >> 3) << 17) | (8u << 24);                  // fp16, 128 rows
            constexpr uint32_t id_o = (1u << 4) | (1u << 16) | ((uint32_t)(HD >> 3) << 17) | (8u << 24);     // B MN-major
            const uint64_t qd = ptx::sdesc_sw128(ptx::smem_u32(sQ));
            int left = 0, item = 0, items_o = 0;
            bool ok = true;
            const auto values = [&](int i, bool first) {         // O_h += P_h V_h of tile i
                const int b = i & 1;
                if (first) {                                     // the item before's O has been read
                    if (items_o > 0 && !ptx::mbar_wait(ptx::smem_u32(&c.o_free), (items_o - 1) & 1, abort, status)) return false;
                    ++items_o;
                }
                if (!ptx::mbar_wait(ptx::smem_u32(&c.v_full[b]), (i >> 1) & 1, abort, status) ||
                    !ptx::mbar_wait(ptx::smem_u32(&c.p_full[b]), (i >> 1) & 1, abort, status)) return false;
                ptx::tc_fence_after();
                const uint64_t vd = mn_desc(ptx::smem_u32(sV + b * S::TILE));
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int x = 0; x < HK / 16; ++x)
                        mma_f16_tmem_a(tmem + O_COL + h * HD, tmem + b * 128 + h * 64 + x * 8,
                                       vd + (uint64_t)((h * HK + x * 16) * 128 >> 4), id_o, !(first && x == 0));
                ptx::mma_commit(ptx::smem_u32(&c.pv_done[b]));
                return true;
            };
            bool first_before = false;
            for (int i = 0; i < count && ok; ++i) {
                bool first = false;
                if (left == 0) {
                    if (i > 0) cur.next_item(p);
                    left = cur.nt - cur.t;
                    if (!ptx::mbar_wait(ptx::smem_u32(&c.q_full), item & 1, abort, status)) break;
                    ++item;
                    first = true;
                }
                const int b = i & 1;
                if (!ptx::mbar_wait(ptx::smem_u32(&c.k_full[b]), (i >> 1) & 1, abort, status) ||
                    !ptx::mbar_wait(ptx::smem_u32(&c.pv_done[b]), ((i >> 1) & 1) ^ 1, abort, status)) break;
                ptx::tc_fence_after();
                const uint64_t kd = ptx::sdesc_sw128(ptx::smem_u32(sK + b * S::TILE));
#pragma unroll
                for (int x = 0; x < HD / 16; ++x) {
                    const uint64_t off = (uint64_t)(((x >> 2) * (TK * 128) + (x & 3) * 32) >> 4);
                    ptx::mma_bf16(tmem + b * 128, qd + off, kd + off, id_s, x > 0);
                }
                ptx::mma_commit(ptx::smem_u32(&c.s_full[b]));
                ptx::mma_commit(ptx::smem_u32(&c.k_empty[b]));
                if (i > 0) ok = values(i - 1, first_before);
                first_before = first;
                --left;
                if (ok && i == count - 1) ok = values(i, first);
            }
            ptx::mma_commit(ptx::smem_u32(&c.drain));
            int never = 0;
            ptx::mbar_wait(ptx::smem_u32(&c.drain), 0, &never, status);
        }
    } else {
        // ------------------------------------------------------------------------------------ softmax, output
        const int quarter = warp & 3, hf = warp >> 2, row = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const float to_exp2 = fabsf(p.a.scale) * 1.4426950408889634f;
        const int box_shift = min(p.q.shift, 7);
        Todo todo{0, 0, 0, 0};
        int item = 0;
        for (int i = 0; i < count; ++item) {
            const int first = cur.t, n_here = min(cur.nt - first, count - i), g = cur.g;
            const Seq q = cur.q;
            const int q0 = cur.qt * p.QT, cols = min(p.QT, q.n - q0) * p.G;
            const int pos0 = q.len - q.n + q0, pos = pos0 + div_g(p, row);       // positions of the item's first row and of this one
            const int64_t stat0 = ((int64_t)g * p.r.n_rows + q.r0 + q0) * p.G;
            float ref = -INFINITY, at = -INFINITY, most = -INFINITY;     // R, X and M
            float l = 0.f, up = 0.f, row_mul = 0.f;              // the sum of 2^(x - X); 2^(X - R) P_UP
            const auto set_at = [&] {
                at = fmaxf(fminf(ref, most), fmaxf(ref - 60.f, most - 30.f));
                up = at == ref ? P_UP : P_UP * exp2_fast(at - ref);
            };
            for (int t = first; t < first + n_here; ++t, ++i) {
                const int b = i & 1, j0 = t * TK + hf * HK;
                ptx::mbar_wait(ptx::smem_u32(&c.ring.full[i % RING]), (i / RING) & 1, abort, status);
                if (t == first) {
                    ptx::mbar_wait(ptx::smem_u32(&c.rows_full[item % MARKS]), (item / MARKS) & 1, abort, status);
                    row_mul = row_scale[(item % MARKS) * ROWS + row] * to_exp2;
                }
                ptx::mbar_wait(ptx::smem_u32(&c.s_full[b]), (i >> 1) & 1, abort, status);
                ptx::tc_fence_after();
                const uint32_t s_at = lanes + b * 128 + hf * HK;
                const float* scales = c.ring.scale[i % RING][0];
                // Blocks of 16 keys: what makes S scores in the exp2 domain (the scale of K's block with the row's and the
                // softmax's constants), V's scale and its logarithm.  Where the first is 0 S is too, and 1 serves: a key that is
                // not seen has S = -inf, which stays that way.
                const auto box_at = [&](int k) { return (hf * HK + k) >> box_shift; };
                const auto mul_at = [&](int k) {
                    const float ks = scales[box_at(k)];
                    return ks > 0.f && row_mul > 0.f ? fmaxf(ks * row_mul, 1.1754944e-38f) : 1.f;
                };
                const bool hole = fminf(fminf(scales[box_at(0)], scales[box_at(16)]), fminf(scales[box_at(32)], scales[box_at(48)])) < 0.f;
                // Away from the tile loop's usual path, which has to stay short (with everything unrolled in place, most cycles
                // went to waiting for instructions): -inf into S for keys that are not loaded or not seen
                if (hole || j0 + HK - 1 > pos0) {
#pragma unroll 1
                    for (int k = 0; k < HK; k += 16) {
                        float w[16];
                        ptx::tmem_ld16(s_at + k, w);
                        const int seen = scales[(hf * HK + k) >> box_shift] < 0.f ? 0 : pos - (j0 + k) + 1;
#pragma unroll
                        for (int y = 0; y < 16; ++y) w[y] = y < seen ? w[y] : -INFINITY;
                        ptx::tmem_st16(s_at + k, w);
                    }
                    ptx::tmem_wait_st();
                }
                // Both passes read S in steps of 16 keys, as loops: the fewer instructions the warps of the SM go through, the less
                // they wait for them, which is more than the second read and the steps' latency cost (2048 rows over 8K: one
                // pass unrolled over 64 keys 467 us, steps of 32 keys 382, of 16 371).
                float top = -INFINITY;                           // the largest of score + log2 of V's scale
#pragma unroll 1
                for (int k = 0; k < HK; k += 16) {
                    uint32_t x[16];
                    ptx::tmem_ld16_issue(s_at + k, x);
                    const float v = scales[8 + box_at(k)], mul = mul_at(k);
                    const float vl = v > 0.f ? fmaxf((float)((int)(__float_as_uint(v) >> 23) - 127), -100.f) : -100.f;
                    ptx::tmem_ld_wait16(x);
                    float m = __uint_as_float(x[0]);
#pragma unroll
                    for (int y = 1; y < 16; ++y) m = fmaxf(m, __uint_as_float(x[y]));
                    top = fmaxf(top, fmaf(m, mul, vl));
                    most = fmaxf(most, m * mul);
                    if (SCORES && row < cols) {
                        float4* score = quads_of(p, q, g, t) + (int64_t)((hf * HK + k) / 4) * (q.n * p.G) + q0 * p.G + row;
#pragma unroll
                        for (int y = 0; y < 16; y += 4, score += q.n * p.G)
                            *score = make_float4(__uint_as_float(x[y]) * mul, __uint_as_float(x[y + 1]) * mul, __uint_as_float(x[y + 2]) * mul,
                                                 __uint_as_float(x[y + 3]) * mul);
                    }
                }
                if (__any_sync(0xffffffffu, ref != -INFINITY && (top > ref + GROW || most > at + SLACK))) {
                    // O_h holds the tiles before: the whole warp rescales, each row by its own factor
                    {
                        ptx::mbar_wait(ptx::smem_u32(&c.pv_done[(i - 1) & 1]), ((i - 1) >> 1) & 1, abort, status);
                        ptx::tc_fence_after();
                        const float to = fmaxf(ref, top), f = ref == -INFINITY ? 1.f : exp2_fast(ref - to);
#pragma unroll 1
                        for (int k = 0; k < HD; k += 16) {
                            float o[16];
                            ptx::tmem_ld16(lanes + O_COL + hf * HD + k, o);
#pragma unroll
                            for (int y = 0; y < 16; ++y) o[y] *= f;
                            ptx::tmem_st16(lanes + O_COL + hf * HD + k, o);
                        }
                        ptx::tmem_wait_st();
                        if (ref != -INFINITY) {
                            const float was = at;
                            ref = to;
                            set_at();
                            l *= exp2_fast(was - at);
                        }
                    }
                }
                if (ref == -INFINITY) {                          // nothing summed yet
                    ref = top;
                    set_at();
                }
                const float neg = at == -INFINITY ? 0.f : -at;
                float sum = 0.f;
#pragma unroll 1
                for (int k = 0; k < HK; k += 16) {               // P over the S columns that have been read
                    uint32_t x[16], w[8];
                    ptx::tmem_ld16_issue(s_at + k, x);
                    // (held to finite numbers where the exponentials it meets have vanished)
                    const float m = mul_at(k), v = fminf(scales[8 + box_at(k)] * up, 3.402823466e38f);
                    ptx::tmem_ld_wait16(x);
#pragma unroll
                    for (int y = 0; y < 16; y += 2) {
                        const float e0 = exp2_fast(fmaf(__uint_as_float(x[y]), m, neg));
                        const float e1 = exp2_fast(fmaf(__uint_as_float(x[y + 1]), m, neg));
                        sum += e0 + e1;
                        w[y / 2] = f16_pair(e0 * v, e1 * v);
                    }
                    tmem_st8_words(s_at + k / 2, w);
                }
                l += sum;
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&c.p_full[b]));
            }
            ptx::mbar_wait(ptx::smem_u32(&c.v_seen[(i - 1) % MARKS]), ((i - 1) / MARKS) & 1, abort, status);
            ptx::mbar_wait(ptx::smem_u32(&c.pv_done[(i - 1) & 1]), ((i - 1) >> 1) & 1, abort, status);
            ptx::tc_fence_after();
            *reinterpret_cast<float4*>(halves + (hf * ROWS + row) * 4) = make_float4(at, l, ref, 0.f);
            ptx::named_bar_sync(3 + quarter, 64);                // the two warps of these rows
            const float4 h0 = *reinterpret_cast<const float4*>(halves + row * 4), h1 = *reinterpret_cast<const float4*>(halves + (ROWS + row) * 4);
            const float X = fmaxf(h0.x, h1.x);
            const auto power = [&](float x) { return x == -INFINITY ? 0.f : exp2_fast(x - X); };
            const float L = h0.y * power(h0.x) + h1.y * power(h1.x);
            const float f0 = power(h0.z), f1 = power(h1.z);      // of the halves' O
            const bool whole = first == 0 && n_here == cur.nt;
            const int u0 = first_cta(p, c.find, mine.per, first), n_pieces = piece_count(p, c.find, mine.per, first, n_here, cur.nt);
            const auto piece_at = [&](int u) { return p.part + (int64_t)((u0 + u) * 2 + (u == 0 ? 1 : 0)) * S::PIECE; };
            const auto out_at = [&](int r) {
                return (bf16*)p.a.out + (int64_t)(q.r0 + q0 + div_g(p, r)) * p.a.out_stride + (int64_t)(g * p.G + mod_g(p, r)) * HD;
            };
            const bool marked = c.any_nan[item % MARKS] != 0;
            const int* marks = nan_marks + (item % MARKS) * HD;
            const float inv = 1.f / L;
            // this thread's half of the row's dims
#pragma unroll 1
            for (int k = 0; k < HD / 2; k += 16) {
                const int d = hf * (HD / 2) + k;
                float a0[16], a1[16];
                ptx::tmem_ld16(lanes + O_COL + d, a0);
                ptx::tmem_ld16(lanes + O_COL + HD + d, a1);
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    // (an O that nothing was added to is not read: its factor is 0 and it may hold anything)
                    float o = (f0 != 0.f ? a0[y] * f0 : 0.f) + (f1 != 0.f ? a1[y] * f1 : 0.f);
                    o *= 1.f / P_UP;
                    if (marked && marks[d + y] <= pos) o = __int_as_float(0x7fc00000);
                    a0[y] = o;
                }
                if (row < cols) {
                    if (whole) {
                        uint32_t w[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) w[y] = L != 0.f ? bf16_pair(a0[2 * y] * inv, a0[2 * y + 1] * inv) : 0u;
                        uint4* o = reinterpret_cast<uint4*>(out_at(row) + d);
                        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        o[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    } else {
                        float4* o = reinterpret_cast<float4*>(piece_at(blockIdx.x - u0) + row * HD + d);
#pragma unroll
                        for (int y = 0; y < 4; ++y) o[y] = make_float4(a0[4 * y], a0[4 * y + 1], a0[4 * y + 2], a0[4 * y + 3]);
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&c.o_free));
            if (whole) {
                if (SCORES && hf == 0 && row < cols) p.stats[stat0 + row] = make_float2(X, inv);
                ptx::named_bar_sync(3 + quarter, 64);            // `halves` has been read
            } else {
                if (hf == 0 && row < cols)
                    *reinterpret_cast<float2*>(piece_at(blockIdx.x - u0) + ROWS * HD + 2 * row) = make_float2(X, L);
                // (the CTA in which the item begins says so to the joining kernel)
                if (first == 0 && tid == 0) todo = Todo{q.r0 + q0, cols, g, n_pieces};
                ptx::named_bar_sync(3 + quarter, 64);            // `halves` has been read
            }
            if (i < count) cur.next_item(p);
        }
        if (tid == 0) reinterpret_cast<Todo*>(p.todo)[blockIdx.x] = todo;
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// The items that span CTAs, a row per warp: block (u, y) has rows 8 y .. 8 y + 7 of the item that begins in CTA u.  A kernel
// of its own, because a piece is 128 rows: joined by the CTA that ends last, the 64 rows of a query over 8K took 15 us of
// one CTA's time, and with two rows per warp 1 us more than this way.
template <int HD>
__global__ void __launch_bounds__(256) kv8_join_kernel(const AttnArgs p) {
    __shared__ float4 buf[8][8 * 32];
    grid_dep_launch();
    grid_dep_wait();
    const Todo d = reinterpret_cast<const Todo*>(p.todo)[blockIdx.x];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, u0 = blockIdx.x, k = blockIdx.y * 8 + warp;
    if (d.pieces == 0 || k >= d.cols) return;
    const auto piece_at = [&](int u) { return p.part + (int64_t)((u0 + u) * 2 + (u == 0 ? 1 : 0)) * Rows<HD>::PIECE; };
    float m, l;
    const float4 a = join_pieces<HD, 8>(piece_at, d.pieces, k * HD, ROWS * HD + 2 * k, m, l, buf[warp]);
    bf16* out = (bf16*)p.a.out + (int64_t)(d.row0 + div_g(p, k)) * p.a.out_stride + (int64_t)(d.g * p.G + mod_g(p, k)) * HD;
    if (lane < HD / 4) store4(out + lane * 4, a, l);
    if (p.scores && lane == 0) p.stats[((int64_t)d.g * p.r.n_rows + d.row0) * p.G + k] = make_float2(m, 1.f / l);
}

// weights[s][g][j] = sum over the sequence's rows and the group's heads of exp2(score - max) / sum: four keys per warp, the
// columns over its lanes
__global__ void __launch_bounds__(256) kv8_rows_weights_kernel(const AttnArgs p) {
    grid_dep_launch();
    grid_dep_wait();
    const int at = blockIdx.x * 8 + (threadIdx.x >> 5), quad = at % (TK / 4), lane = threadIdx.x & 31, j = at * 4, g = blockIdx.y;
    const Seq q = seq_at(p, blockIdx.z);
    if (j >= q.len || *p.voided) return;
    const int seen = max(0, j - (q.len - q.n)) * p.G, cols = q.n * p.G;      // columns that see key j: [seen, cols)
    const float4* score = quads_of(p, q, g, at / (TK / 4)) + (int64_t)quad * cols;
    const float2* st = p.stats + ((int64_t)g * p.r.n_rows + q.r0) * p.G;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int k = seen + lane; k < cols; k += 32) {
        const float4 x = __ldcs(score + k);
        const float2 m = st[k];
        w[0] += x.x == -INFINITY ? 0.f : exp2_fast(x.x - m.x) * m.y;
        w[1] += x.y == -INFINITY ? 0.f : exp2_fast(x.y - m.x) * m.y;
        w[2] += x.z == -INFINITY ? 0.f : exp2_fast(x.z - m.x) * m.y;
        w[3] += x.w == -INFINITY ? 0.f : exp2_fast(x.w - m.x) * m.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int y = 0; y < 4; ++y) w[y] += __shfl_xor_sync(0xffffffffu, w[y], o);
    const float mine = lane == 0 ? w[0] : lane == 1 ? w[1] : lane == 2 ? w[2] : w[3];
    if (lane < 4 && j + lane < q.len) {
        float* dst = p.a.weights + ((int64_t)blockIdx.z * p.Hkv + g) * p.a.weights_ld + j + lane;
        *dst = p.a.add ? *dst + mine : mine;
    }
}

template <int HD, bool SCORES> cudaError_t launch_dim(const Kv8& c, AttnArgs& p, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = smem_limit_once(kv8_rows_kernel<HD, SCORES>, Rows<HD>::BYTES, done);
    if (e != cudaSuccess) return e;
    p.QT = ROWS / p.G;
    // 4096 rows over 4096 keys: 975 us when only tiles counted, 424 with 2 places; 256 with 4 and 5, 261 with 6 as the kernel
    // was then (252 now); 16 ragged sequences x 512 rows: 182, 185 and 193 us (184 now)
    p.ahead = 4;
    p.min_places = 1 + p.ahead;
    const int64_t items = ((int64_t)p.r.n_rows / p.QT + p.q.n) * p.Hkv;
    const int64_t tiles = items * ((p.q.max_len + TK - 1) / TK + 1);
    CUtensorMap map;
    memcpy(&map, c.map, sizeof map);
    const unsigned ctas = (unsigned)(tiles < c.num_sms ? tiles : c.num_sms);
    cudaError_t err = launch_ex(c.pdl, kv8_rows_kernel<HD, SCORES>, dim3(ctas), dim3(THREADS), Rows<HD>::BYTES, s, map, p);
    if (err == cudaSuccess) err = launch_ex(c.pdl, kv8_join_kernel<HD>, dim3(ctas, ROWS / 8), dim3(256), 0, s, p);
    if (err == cudaSuccess && SCORES)
        err = launch_ex(c.pdl, kv8_rows_weights_kernel, dim3((p.q.max_len + 31) / 32, p.Hkv, p.q.n), dim3(256), 0, s, p);
    return err;
}

}  // namespace

size_t kv8_rows_part_floats(int num_sms) { return (size_t)num_sms * 2 * Rows<128>::PIECE; }

cudaError_t launch_kv8_rows(const Kv8& c, const void* attn_args, cudaStream_t s) {
    AttnArgs p = *static_cast<const AttnArgs*>(attn_args);
    p.todo = c.todo;
    if (p.scores) return c.cfg.head_dim == 128 ? launch_dim<128, true>(c, p, s) : launch_dim<64, true>(c, p, s);
    return c.cfg.head_dim == 128 ? launch_dim<128, false>(c, p, s) : launch_dim<64, false>(c, p, s);
}

}  // namespace cb
