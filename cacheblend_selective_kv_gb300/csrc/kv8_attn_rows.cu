// Attention over the 8-bit paged K/V cache for many query rows per sequence (a query over a blended context, a prompt in
// pieces): bf16 queries, an item's 128 rows = 128 / G query rows x the G heads of their group in the lanes of tensor memory.
//
// With this many rows a tile of keys is used often enough to widen it once: warps 8-11 read the codes (page by page through
// the block table), write K as bf16 with its block scale multiplied in (exact: four significant bits times a power of two)
// and V as fp16 codes, in the swizzled layouts of the MMA operands, and S = Q K^T, O += P V run on kind::f16.  Against the
// e4m3 terms of kv8_attn.cu this costs a conversion per cached value and tile, and saves the terms of q and P for each of
// 128 rows, the shuffles of maxima over keys (a row is one thread's) and the products with the scales of K.  P is
// fp16: 11 bits, 2^-12 relative.
//
// V's block scales differ, so P carries them: p_j = 2^(x_j - R) s_j with x the score in the exp2 domain, s_j the scale of
// key j's block and R a reference of the row no more than 2^8 below the largest x_j + log2 s_j so far.  It grows lazily (O
// is rescaled in tensor memory when it must), which keeps P within fp16; the softmax sum takes 2^(x_j - R) in fp32.  A
// scale below 2^-100 counts as 2^-100 for R, so that no exponent overflows.
//
// Each of the two halves of a tile's keys has its own R, sum and O (as the blend's attention kernel does, so that the warps
// of a row need not meet for every tile); they are joined at the end of an item.  Per tile and SM: 32 MMAs of 128 x 128 x 16
// at about 99 cycles, 128 x 128 exponentials, 2 x 128 x HD conversions.
#include "cb_kv8_attn.cuh"

namespace cb {

namespace {

constexpr int ROWS = 128;
constexpr int SOFT = 256, CONV = 128, THREADS = SOFT + CONV + 32;
constexpr int CONV_WARP = SOFT / 32, MMA_WARP = CONV_WARP + CONV / 32;
constexpr int HK = 64;                   // keys of a half
constexpr int RING = 4;                  // tiles whose scales are kept; items whose NaN marks are
constexpr float GROW = 8.f;              // how far (log2) P may outgrow its reference
constexpr float P_UP = 128.f;            // P is stored this much larger: its largest values are 2^7 .. 2^15 of fp16's 2^16

struct RowsShared {
    uint64_t k_full[2], k_empty[2], v_full[2], pv_done[2], s_full[2], p_full[2], scale_full[RING], q_full, o_free, drain;
    uint32_t tmem;
    int abort;
    Find find;
    int last;
    int holes[RING];                     // a key of the tile is not loaded
    int any_nan[RING];                   // an item's V held NaN that not all of its rows see
};

template <int HD> struct Rows {
    static constexpr int TILE = TK * HD * 2;                     // a K or V tile, or Q, in 16-bit elements
    static constexpr int OFF_K = TILE, OFF_V = 3 * TILE;
    static constexpr int OFF_X = 5 * TILE;
    // floats: scale of V [RING][TK], its logarithm [RING][TK], (R, sum) [2][ROWS][2]; ints: nan_from [RING][HD]
    static constexpr int X_FLOATS = 2 * RING * TK + 4 * ROWS + RING * HD;
    static constexpr int OFF_C = OFF_X + X_FLOATS * 4;
    static constexpr int BYTES = OFF_C + (int)sizeof(RowsShared);
    static constexpr int PIECE = ROWS * (HD + 2);
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
__device__ __forceinline__ void tmem_st16_words(uint32_t addr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
          "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
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

template <int HD>
__global__ void __launch_bounds__(THREADS, 1) kv8_rows_kernel(const AttnArgs p, const uint8_t* __restrict__ kc,
                                                             const uint8_t* __restrict__ vc) {
    using S = Rows<HD>;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint8_t* sQ = sm;
    uint8_t* sK = sm + S::OFF_K;                        // [2]
    uint8_t* sV = sm + S::OFF_V;                        // [2]
    float* v_scale = reinterpret_cast<float*>(sm + S::OFF_X);
    float* v_log = v_scale + RING * TK;
    float* halves = v_log + RING * TK;
    int* nan_marks = reinterpret_cast<int*>(halves + 4 * ROWS);
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
        for (int i = 0; i < RING; ++i) {
            ptx::mbar_init(ptx::smem_u32(&c.scale_full[i]), CONV / 32);
            c.holes[i] = c.any_nan[i] = 0;
        }
        ptx::mbar_init(ptx::smem_u32(&c.q_full), CONV / 32);
        ptx::mbar_init(ptx::smem_u32(&c.o_free), SOFT / 32);
        ptx::mbar_init(ptx::smem_u32(&c.drain), 1);
        c.abort = 0;
        ptx::fence_barrier_init();
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
        // ------------------------------------------------------------------------------------ codes to operands
        // Like the softmax warps, these run on to their last tile when a wait has given up.  The codes of V are asked for
        // before K's are converted, the next tile's K before V's are.
        constexpr int LPR = HD / 16, RPW = 32 / LPR, NI = TK / (4 * RPW);           // lanes per row, rows per warp and step, steps
        const int w = warp - CONV_WARP, t = tid - SOFT, sub = lane / LPR, e = lane % LPR, P = 1 << p.q.shift;
        const auto row_of = [&](int n) { return (n * 4 + w) * RPW + sub; };
        int at[NI];                                     // this thread's rows among the layer's rows of all heads, or -1
        float ks[NI];
        float vs_key = 0.f;                             // V's scale of key t (-1: not loaded)
        uint4 k[NI], v[NI];
        const auto find_rows = [&](const Cursor& u) {
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                const int j = u.t * TK + row_of(n);
                const int pg = j < u.q.len ? kv8_page(p.q, u.s, j >> p.q.shift) : -1;
                at[n] = pg >= 0 ? (pg * p.Hkv + u.g) * P + (j & (P - 1)) : -1;
                ks[n] = pg >= 0 ? p.ks[(int64_t)pg * p.Hkv + u.g] : 0.f;
            }
            const int j = u.t * TK + t;
            const int pg = j < u.q.len ? kv8_page(p.q, u.s, j >> p.q.shift) : -1;
            vs_key = pg >= 0 ? p.vs[(int64_t)pg * p.Hkv + u.g] : -1.f;
        };
        const auto load = [&](const uint8_t* codes, uint4* x) {
#pragma unroll
            for (int n = 0; n < NI; ++n)
                x[n] = at[n] >= 0 ? *reinterpret_cast<const uint4*>(codes + (int64_t)at[n] * HD + e * 16) : make_uint4(0, 0, 0, 0);
        };
        if (count > 0) {
            find_rows(cur);
            load(kc, k);
        }
        int item = -1;
        bool begins = true;
        for (int i = 0; i < count; ++i) {
            const int st = i & 1;
            const uint32_t par = ((i >> 1) & 1) ^ 1;
            const Seq q = cur.q;
            const int q0 = cur.qt * p.QT, cols = min(p.QT, q.n - q0) * p.G, pos0 = q.len - q.n + q0, tile = cur.t;
            if (begins) {
                ++item;
                // Q once the products with the item before's are done; then the softmax is past tile i - 3, hence past the item
                // whose marks these were
                if (i > 0) ptx::mbar_wait(ptx::smem_u32(&c.k_empty[(i - 1) & 1]), ((i - 1) >> 1) & 1, abort, status);
                if (t < HD) nan_marks[(item % RING) * HD + t] = INT_MAX;
                if (t == 0) c.any_nan[item % RING] = 0;
                const bf16* qbase = (const bf16*)p.a.q + (int64_t)(q.r0 + q0) * p.a.q_stride + (int64_t)cur.g * p.G * HD;
                for (int x = t; x < ROWS * (HD / 8); x += CONV) {
                    const int row = x / (HD / 8), ch = x % (HD / 8);
                    uint4 val = make_uint4(0, 0, 0, 0);
                    if (row < cols)
                        val = *reinterpret_cast<const uint4*>(qbase + (int64_t)(row / p.G) * p.a.q_stride + (row % p.G) * HD + ch * 8);
                    *reinterpret_cast<uint4*>(sQ + wide_at(row, ch)) = val;
                }
                fence_async_smem();
                ptx::named_bar_sync(2, CONV);                    // also: the marks
                if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&c.q_full));
            }
            load(vc, v);
            float ks_now[NI];
            bool gone[NI];
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                ks_now[n] = ks[n];
                gone[n] = at[n] < 0;
            }
            const float vs_now = vs_key;
            // K: free once S of two tiles before is done, which also means that the softmax is past the tile four before
            ptx::mbar_wait(ptx::smem_u32(&c.k_empty[st]), par, abort, status);
            v_scale[(i % RING) * TK + t] = vs_now < 0.f ? 0.f : vs_now * P_UP;
            v_log[(i % RING) * TK + t] = vs_now < 0.f ? -INFINITY : fmaxf(log2f(vs_now), -100.f);
            const unsigned hole = __ballot_sync(0xffffffffu, vs_now < 0.f);
            if (t == 0) c.holes[i % RING] = 0;
            ptx::named_bar_sync(2, CONV);
            if (lane == 0) {
                if (hole) c.holes[i % RING] = 1;
                ptx::mbar_arrive(ptx::smem_u32(&c.scale_full[i % RING]));
            }
            uint8_t* dk = sK + st * S::TILE;
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                const uint32_t cw[4] = {k[n].x, k[n].y, k[n].z, k[n].w};
                uint32_t o[8];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float2 lo = kv8_value2(cw[x]), hi = kv8_value2(cw[x] >> 16);
                    o[2 * x] = bf16_pair(lo.x * ks_now[n], lo.y * ks_now[n]);
                    o[2 * x + 1] = bf16_pair(hi.x * ks_now[n], hi.y * ks_now[n]);
                }
                *reinterpret_cast<uint4*>(dk + wide_at(row_of(n), 2 * e)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(dk + wide_at(row_of(n), 2 * e + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&c.k_full[st]));
            // the next tile's rows and K
            begins = false;
            if (i + 1 < count) {
                if (++cur.t == cur.nt) {
                    cur.next_item(p);
                    begins = true;
                }
                find_rows(cur);
                load(kc, k);
            }
            // V: zero where nothing is loaded; a NaN that only later rows see is taken out and remembered
            ptx::mbar_wait(ptx::smem_u32(&c.pv_done[st]), par, abort, status);
            uint8_t* dv = sV + st * S::TILE;
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                uint32_t cw[4] = {v[n].x, v[n].y, v[n].z, v[n].w};
                const int j = tile * TK + row_of(n);
                if (gone[n]) {
                    cw[0] = cw[1] = cw[2] = cw[3] = 0;
                } else if (j > pos0) {
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t bad = __vcmpeq4(cw[x] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        if (bad == 0) continue;
                        cw[x] &= ~bad;
                        for (int y = 0; y < 4; ++y)
                            if (bad >> (8 * y) & 1) atomicMin(nan_marks + (item % RING) * HD + e * 16 + 4 * x + y, j);
                        c.any_nan[item % RING] = 1;
                    }
                }
                uint32_t o[8];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    o[2 * x] = half2_word(kv8_half2(cw[x]));
                    o[2 * x + 1] = half2_word(kv8_half2(cw[x] >> 16));
                }
                *reinterpret_cast<uint4*>(dv + wide_at(row_of(n), 2 * e)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(dv + wide_at(row_of(n), 2 * e + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&c.v_full[st]));
        }
    } else if (warp == MMA_WARP) {
        // ------------------------------------------------------------------------------------ MMA
        if (lane == 0) {
            constexpr uint32_t id_s = ptx::idesc_bf16(ROWS, TK);
            constexpr uint32_t id_o = (1u << 4) | (1u << 16) | ((uint32_t)(HD >> 3) << 17) | (8u << 24);     // f16, B MN-major
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
        const float to_exp2 = p.a.scale * 1.4426950408889634f;
        int item = 0;
        for (int i = 0; i < count; ++item) {
            const int first = cur.t, n_here = min(cur.nt - first, count - i), g = cur.g;
            const Seq q = cur.q;
            const int q0 = cur.qt * p.QT, cols = min(p.QT, q.n - q0) * p.G;
            const int pos0 = q.len - q.n + q0, pos = pos0 + row / p.G;       // positions of the item's first row and of this one
            const int64_t stat0 = ((int64_t)g * p.r.n_rows + q.r0 + q0) * p.G;
            float ref = -INFINITY, l = 0.f;                      // R and the sum of 2^(x - R)
            for (int t = first; t < first + n_here; ++t, ++i) {
                const int b = i & 1, j0 = t * TK + hf * HK;
                ptx::mbar_wait(ptx::smem_u32(&c.scale_full[i % RING]), (i / RING) & 1, abort, status);
                const float* vl = v_log + (i % RING) * TK + hf * HK;
                const float* vs = v_scale + (i % RING) * TK + hf * HK;
                const bool masked = c.holes[i % RING] != 0 || j0 + HK - 1 > pos0;
                ptx::mbar_wait(ptx::smem_u32(&c.s_full[b]), (i >> 1) & 1, abort, status);
                ptx::tc_fence_after();
                const uint32_t s_at = lanes + b * 128 + hf * HK;
                float x[HK];                                     // scores in the exp2 domain
#pragma unroll
                for (int k = 0; k < HK; k += 16) {
                    uint32_t w[16];
                    ptx::tmem_ld16_issue(s_at + k, w);
                    ptx::tmem_ld_wait16(w);
#pragma unroll
                    for (int y = 0; y < 16; ++y) x[k + y] = __uint_as_float(w[y]) * to_exp2;
                }
                if (masked) {
#pragma unroll
                    for (int k = 0; k < HK; ++k)
                        if (j0 + k > pos || vl[k] == -INFINITY) x[k] = -INFINITY;
                }
                if (p.scores && row < cols) {
                    float* score = p.scores + (stat0 + row) * p.score_ld + j0;
#pragma unroll
                    for (int k = 0; k < HK; k += 4) *reinterpret_cast<float4*>(score + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
                }
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < HK; k += 4) {
                    const float4 lg = *reinterpret_cast<const float4*>(vl + k);
                    top = fmaxf(top, fmaxf(fmaxf(x[k] + lg.x, x[k + 1] + lg.y), fmaxf(x[k + 2] + lg.z, x[k + 3] + lg.w)));
                }
                if (__any_sync(0xffffffffu, ref != -INFINITY && top > ref + GROW)) {
                    // O_h holds the tiles before: the whole warp rescales, each row by its own factor
                    {
                        ptx::mbar_wait(ptx::smem_u32(&c.pv_done[(i - 1) & 1]), ((i - 1) >> 1) & 1, abort, status);
                        ptx::tc_fence_after();
                        const float to = fmaxf(ref, top), f = ref == -INFINITY ? 1.f : exp2_fast(ref - to);
#pragma unroll
                        for (int k = 0; k < HD; k += 16) {
                            float o[16];
                            ptx::tmem_ld16(lanes + O_COL + hf * HD + k, o);
#pragma unroll
                            for (int y = 0; y < 16; ++y) o[y] *= f;
                            ptx::tmem_st16(lanes + O_COL + hf * HD + k, o);
                        }
                        ptx::tmem_wait_st();
                        l *= f;
                        if (ref != -INFINITY) ref = to;
                    }
                }
                if (ref == -INFINITY) ref = top;                 // nothing summed yet
                const float neg = ref == -INFINITY ? 0.f : -ref;
                float sum = 0.f;
#pragma unroll
                for (int h = 0; h < HK; h += 32) {               // P over the S columns that have been read
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const float4 sc = *reinterpret_cast<const float4*>(vs + h + k);
                        const float e0 = exp2_fast(x[h + k] + neg), e1 = exp2_fast(x[h + k + 1] + neg);
                        const float e2 = exp2_fast(x[h + k + 2] + neg), e3 = exp2_fast(x[h + k + 3] + neg);
                        sum += (e0 + e1) + (e2 + e3);
                        w[k / 2] = f16_pair(e0 * sc.x, e1 * sc.y);
                        w[k / 2 + 1] = f16_pair(e2 * sc.z, e3 * sc.w);
                    }
                    tmem_st16_words(s_at + h / 2, w);
                }
                l += sum;
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&c.p_full[b]));
            }
            ptx::mbar_wait(ptx::smem_u32(&c.pv_done[(i - 1) & 1]), ((i - 1) >> 1) & 1, abort, status);
            ptx::tc_fence_after();
            *reinterpret_cast<float2*>(halves + (hf * ROWS + row) * 2) = make_float2(ref, l);
            ptx::named_bar_sync(3 + quarter, 64);                // the two warps of these rows
            const float2 other = *reinterpret_cast<const float2*>(halves + ((hf ^ 1) * ROWS + row) * 2);
            const float M = fmaxf(ref, other.x);
            const float f_own = ref == -INFINITY ? 0.f : exp2_fast(ref - M), f_other = other.x == -INFINITY ? 0.f : exp2_fast(other.x - M);
            const float f0 = hf == 0 ? f_own : f_other, f1 = hf == 0 ? f_other : f_own;
            const float L = hf == 0 ? l * f_own + other.y * f_other : other.y * f_other + l * f_own;
            const bool whole = first == 0 && n_here == cur.nt;
            const long long begin = mine.t0 + (i - n_here) - first;          // the item's first tile in the list
            const int u0 = (int)(begin / mine.per), n_pieces = (int)((begin + cur.nt - 1) / mine.per) - u0 + 1;
            const auto piece_at = [&](int u) { return p.part + (int64_t)((u0 + u) * 2 + (u == 0 ? 1 : 0)) * S::PIECE; };
            const auto out_at = [&](int r) {
                return (bf16*)p.a.out + (int64_t)(q.r0 + q0 + r / p.G) * p.a.out_stride + (int64_t)(g * p.G + r % p.G) * HD;
            };
            const bool marked = c.any_nan[item % RING] != 0;
            const int* marks = nan_marks + (item % RING) * HD;
            const float inv = 1.f / L;
            // this thread's half of the row's dims
#pragma unroll
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
                        for (int y = 0; y < 8; ++y) w[y] = pos >= 0 ? bf16_pair(a0[2 * y] * inv, a0[2 * y + 1] * inv) : 0u;
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
                if (p.scores && hf == 0 && row < cols) p.stats[stat0 + row] = make_float2(M, inv);
                ptx::named_bar_sync(3 + quarter, 64);            // `halves` has been read
            } else {
                if (hf == 0 && row < cols)
                    *reinterpret_cast<float2*>(piece_at(blockIdx.x - u0) + ROWS * HD + 2 * row) = make_float2(M, L);
                ptx::named_bar_sync(1, SOFT);
                if (tid == 0) {
                    __threadfence();                             // the whole CTA's piece, ordered by the barrier
                    c.last = atomicAdd(p.arrived + u0, 1u) == (unsigned)n_pieces - 1;
                    if (c.last) atomicExch(p.arrived + u0, 0u);
                    __threadfence();
                }
                ptx::named_bar_sync(1, SOFT);
                if (c.last) {
                    for (int k = warp; k < cols; k += SOFT / 32) {
                        float m, sum;
                        const float4 a = join_pieces<HD>(piece_at, n_pieces, k * HD, ROWS * HD + 2 * k, m, sum);
                        if (lane < HD / 4) store4(out_at(k) + lane * 4, a, 1.f / sum, pos0 + k / p.G >= 0);
                        if (p.scores && lane == 0) p.stats[stat0 + k] = make_float2(m, 1.f / sum);
                    }
                    ptx::named_bar_sync(1, SOFT);                // `last` has been read
                }
            }
            if (i < count) cur.next_item(p);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <int HD> cudaError_t launch_dim(const Kv8& c, AttnArgs& p, const uint8_t* kc, const uint8_t* vc, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = smem_limit_once(kv8_rows_kernel<HD>, Rows<HD>::BYTES, done);
    if (e != cudaSuccess) return e;
    p.QT = ROWS / p.G;
    const int64_t items = ((int64_t)p.r.n_rows / p.QT + p.q.n) * p.Hkv;
    const int64_t tiles = items * ((p.q.max_len + TK - 1) / TK + 1);
    return launch_ex(c.pdl, kv8_rows_kernel<HD>, dim3((unsigned)(tiles < c.num_sms ? tiles : c.num_sms)), dim3(THREADS), Rows<HD>::BYTES, s,
                     p, kc, vc);
}

}  // namespace

size_t kv8_rows_part_floats(int num_sms) { return (size_t)num_sms * 2 * Rows<128>::PIECE; }

cudaError_t launch_kv8_rows(const Kv8& c, const void* attn_args, int layer, cudaStream_t s) {
    AttnArgs p = *static_cast<const AttnArgs*>(attn_args);
    const int64_t blocks = c.cfg.n_pages * c.cfg.n_kv_heads, bytes = (int64_t)c.cfg.head_dim << c.shift;
    const uint8_t* kc = c.codes + (int64_t)layer * 2 * blocks * bytes;
    const uint8_t* vc = kc + blocks * bytes;
    return c.cfg.head_dim == 128 ? launch_dim<128>(c, p, kc, vc, s) : launch_dim<64>(c, p, kc, vc, s);
}

}  // namespace cb
