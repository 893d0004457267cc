// Attention over the 8-bit paged K/V cache: which kernel a call takes, the weights its keys received, and what both kernels
// need of the host.
#include <cudaTypedefs.h>

#include <cmath>
#include <iterator>

#include "cb_kv8_few.cuh"

namespace cb {

namespace {

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

// Rows of sequences with a shared prefix: the sums over their own keys (BESIDE) and over the prefix (PREFIX, perhaps still in pieces),
// joined and divided.  Block (s, g, z) has columns of sequence s and KV head g, a warp each.
constexpr int JOINERS = 4, AT_ONCE = 16;
template <int HD, typename T>
__global__ void __launch_bounds__(32 * JOINERS) kv8_both_kernel(const AttnArgs p, const AttnArgs pre) {
    __shared__ float4 buf[JOINERS][AT_ONCE * 32];
    grid_dep_launch();
    grid_dep_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *p.opened = 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = blockIdx.y, cols = pre.piece_cols;
    const unsigned none = *p.voided | *pre.voided;
    const bool prefix = has_prefix(p, blockIdx.x);
    const Seq q = seq_at(p, blockIdx.x);
    if (none) return;
#pragma unroll 1
    for (int k = blockIdx.z * JOINERS + warp; k < q.n * p.G; k += gridDim.z * JOINERS) {
        const int row = q.r0 + k / p.G, head = g * p.G + k % p.G;      // (of a sequence: k may pass what div_g divides)
        const int64_t at = prefix_at(p, row, head);
        const float2 own_stat = p.side_stat[at];
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 own = lane < HD / 4 ? *reinterpret_cast<const float4*>(p.side_sum + at * HD + lane * 4) : zero;
        float2 before = make_float2(-INFINITY, 0.f);
        float4 sum = zero;
        if (prefix) {
            const int2 in = pre.pieces_of[at];
            const int u0 = in.x >> 7, r = in.x & 127;
            if (in.y > 0) {
                if (u0 < 0 || r >= cols || in.y > pre.piece_ctas - u0) continue;         // (offsets that have changed since)
                const auto piece_at = [&](int u) { return pre.part + (int64_t)((u0 + u) * 2 + (u == 0 ? 1 : 0)) * (cols * (HD + 2)); };
                sum = join_pieces<HD, AT_ONCE>(piece_at, in.y, r * HD, cols * HD + 2 * r, before.x, before.y, buf[warp]);
            } else {
                before = pre.side_stat[at];
                if (lane < HD / 4) sum = *reinterpret_cast<const float4*>(pre.side_sum + at * HD + lane * 4);
            }
        }
        const Merge merge(own_stat.x, own_stat.y, before);
        if (lane < HD / 4) store4((T*)p.a.out + (int64_t)row * p.a.out_stride + (int64_t)head * HD + lane * 4, merge(own, sum), merge.l);
    }
}
template <int HD, typename T> cudaError_t launch_both(const Kv8& c, const AttnArgs& own, const AttnArgs& pre, cudaStream_t s) {
    const int rows = (own.r.n_rows + own.q.n - 1) / own.q.n, z = (rows * own.G + JOINERS - 1) / JOINERS;
    return launch_ex(c.pdl, kv8_both_kernel<HD, T>, dim3(own.q.n, own.Hkv, z < 65535 ? z : 65535), dim3(32 * JOINERS), 0, s, own, pre);
}

}  // namespace

// scratch: two pieces for every CTA of the largest launch, and where calls may share a prefix of the largest that runs beside another (BESIDE)
template <typename S> constexpr size_t pieces() { return (size_t)S::CTAS * 2 * S::PIECE; }
static size_t few_part_floats(int num_sms) {
    const size_t sizes[] = {pieces<C4<128>>(), pieces<C4S<128>>(), pieces<C8<128>>(), pieces<C16<128>>(), pieces<C32<128>>(),
                            pieces<F4<128>>(), pieces<F8<128>>()};
    return *std::max_element(std::begin(sizes), std::end(sizes)) * num_sms;
}
static size_t most_part_floats(int num_sms) { return std::max(few_part_floats(num_sms), kv8_rows_part_floats(num_sms)); }
size_t kv8_part_floats(int num_sms, bool shared) { return most_part_floats(num_sms) + (shared ? few_part_floats(num_sms) : 0); }
static int most_ctas(int num_sms) { return 4 * num_sms; }
int kv8_most_ctas(int num_sms, bool shared) { return (shared ? 2 : 1) * most_ctas(num_sms); }

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
    AttnArgs p = attn_args(c, q, r, a, layer);
    p.voided = r.n_rows > 0 ? c.voided : nullptr;
    p.scores = a.weights && q.max_len > 0 ? c.scores : nullptr;      // (no keys: no weights to return)
    if (r.n_rows > 0) {
        if (many_rows(c, p)) return launch_kv8_rows(c, &p, PLAIN, s);      // sums its weights too
        const cudaError_t e = c.cfg.head_dim == 128 ? launch_few<128, PLAIN>(c, p, s) : launch_few<64, PLAIN>(c, p, s);
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

// What a launch over n sequences of `columns` columns each is made of: its items, the CTAs that an SM holds of it, and the time of one
// tile of 128 keys in all items, over all SMs, when the codes come from L2 (heads of 128; heads of 64 take as long).
struct Cost {
    double items, tile_ns;
    int ctas;
};
Cost cost_of(const Kv8& c, int n, int columns, bool short_items) {
    const bool wide = c.cfg.dtype == CB_F32;
    const int cols = wide ? (columns <= 4 ? 4 : 8) : columns <= 4 ? 4 : columns <= 8 ? 8 : columns <= 16 ? 16 : columns <= 32 ? 32 : 128;
    const double ns = wide ? (cols == 4 ? 3.3 : 4.3) : cols == 4 ? 2.7 : cols == 8 ? 3.5 : cols == 16 ? 5.5 : cols == 32 ? 9.5 : 10.0;
    const double items = (double)n * ((columns + cols - 1) / cols) * c.cfg.n_kv_heads;
    return Cost{items, items * ns, wide ? 2 : cols == 4 ? (short_items ? 4 : 3) : cols <= 16 ? 2 : 1};
}

cudaError_t launch_kv8_shared(const Kv8& c, const Kv8Prefix& pre, const Kv8Seqs& q, const Kv8Rows& r, const Kv8Attn& a, int layer,
                              cudaStream_t s) {
    AttnArgs p = attn_args(c, pre.q, r, a, layer);
    p.first = pre.first;
    p.per_group = pre.per_group;
    p.groups = pre.q.n;
    p.members = q.n;
    AttnArgs own = p;
    own.q = q;
    own.pre = pre.q;
    own.voided = c.voided;
    const bool many = many_rows(c, own);
    // One launch, each of whose sequences reads its prefix (from L2, once one has read it), or a launch over the prefixes with one over the
    // own keys beside it, on `beside` SMs: whichever is estimated to take less (us of both, 32 / 8 heads of 128: 64 sequences of 256 keys
    // on a prefix of 8192 95 and 33, on 2000 38 and 24; 32 of 64 on 2000 25.0 and 23.7; 16 of 300 on 1024 15.3 and 21; 8 of 300 on 16384 30 and
    // 26; 64 pairs of 300 on 600 46 and 89).  12 us are a launch of short items, 19 the launches over the prefixes and of the sums.  Beside
    // PREFIX an SM goes through its items one round of CTAs after another: items of a few tiles stay whole, so that rounds are whole
    // too, and each costs two tiles more where an SM has few CTAs (64 of 256 keys on 8192: 74, 48, 33, 33 and 38 us on 8, 16, 32, 40 and 64
    // SMs; 64 of 512 on 4 x 4096: 135, 82, 47, 39 and 39 on 8, 16, 32, 48 and 64).  A PREFIX of several CTAs to an SM leaves no SM to
    // the other launch, and both slow down (2 rows of 32 fp32 sequences on 8192: 94 us in one launch, 113 at best in two).  With many rows
    // per sequence the launches follow each other: 16 rows of 16 sequences of 300 on 4096 66 us in one, 62 in two.
    const int64_t pre_tiles = ((int64_t)pre.q.max_len + TK - 1) / TK, own_tiles = ((int64_t)q.max_len + TK - 1) / TK;
    const bool short_items = own_tiles <= 4;
    const Cost of_pre = cost_of(c, pre.q.n, (r.n_rows + pre.q.n - 1) / pre.q.n * p.G, false);
    const Cost of_own = cost_of(c, q.n, (r.n_rows + q.n - 1) / q.n * p.G, short_items);
    const double one = 12e3 + of_own.tile_ns * (double)(own_tiles + 1 + pre_tiles);
    double two = 12e3 + 17e3 + of_own.tile_ns * (double)(own_tiles + 1) + of_pre.tile_ns * (double)pre_tiles;
    int beside = 0;
    if (!many) {
        const double round_ns = of_own.tile_ns / of_own.items * of_own.ctas * c.num_sms * (double)(own_tiles + (of_own.ctas == 4 ? 0 : 2));
        for (int x = 8; x <= std::max(c.num_sms - 16, 8); x += 4) {
            double rounds = of_own.items / (x * of_own.ctas);
            if (short_items) rounds = std::ceil(rounds);
            double t = 19e3 + std::max(rounds * round_ns, of_pre.tile_ns * (double)pre_tiles * c.num_sms / (c.num_sms - x));
            if (of_pre.ctas > 1) t *= 1.3;
            if (beside == 0 || t < two) {
                beside = x;
                two = t;
            }
        }
    }
    const int64_t places = ((int64_t)r.n_rows + q.n) * p.Hkv * (pre_tiles + own_tiles + 9);
    if (one - two <= c.again_ns && places < 0x7fffffff)
        return many ? launch_kv8_rows(c, &own, JOINT, s) : launch_kv8_few_joint(c, &own, s);
    const int64_t heads = (int64_t)r.n_rows * p.Hq, sums = heads * c.cfg.head_dim;
    p.side_sum = pre.scratch;
    p.side_stat = reinterpret_cast<float2*>(pre.scratch + 2 * sums);
    p.voided = c.voided + 16;
    const bool rows = many_rows(c, p);
    if (rows) p.piece_cols = 128;                                // (the other kernel sets its own)
    if (!many) {
        p.sms = std::max(c.num_sms - beside, 2);
        p.piece_ctas = p.sms;
        own.sms = beside;
        own.part += most_part_floats(c.num_sms);
        own.arrived += most_ctas(c.num_sms);
        own.side_sum = p.side_sum + sums;
        own.side_stat = p.side_stat + heads;
        p.pieces_of = reinterpret_cast<int2*>(own.side_stat + heads);
        p.opened = own.opened = c.opened;
    }
    cudaError_t e = rows ? launch_kv8_rows(c, &p, PREFIX, s) : launch_kv8_few_prefix(c, &p, s);
    if (e != cudaSuccess) return e;
    if (many) {
        own.prefix_voided = p.voided;
        own.side_sum = p.side_sum;
        own.side_stat = p.side_stat;
        return launch_kv8_rows(c, &own, OWN, s);
    }
    e = launch_kv8_few_own(c, &own, s);
    const bool wide = c.cfg.head_dim == 128;
    if (e == cudaSuccess) {
        if (c.cfg.dtype == CB_F32) e = wide ? launch_both<128, float>(c, own, p, s) : launch_both<64, float>(c, own, p, s);
        else e = wide ? launch_both<128, bf16>(c, own, p, s) : launch_both<64, bf16>(c, own, p, s);
    }
    if (e != cudaSuccess) cudaMemsetAsync(c.opened, 0, sizeof(unsigned), s);      // what a later call must not take for its own
    return e;
}

}  // namespace cb
