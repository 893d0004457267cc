// Attention over the 8-bit paged K/V cache: which kernel a call takes, the weights its keys received, and what both kernels
// need of the host.
#include <cudaTypedefs.h>

#include <cstdlib>
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

}  // namespace

// scratch: two pieces for every CTA of the largest launch
template <typename S> constexpr size_t pieces() { return (size_t)S::CTAS * 2 * S::PIECE; }
size_t kv8_part_floats(int num_sms) {
    const size_t sizes[] = {pieces<C4<128>>(), pieces<C4S<128>>(), pieces<C8<128>>(), pieces<C16<128>>(), pieces<C32<128>>(),
                            pieces<F4<128>>(), pieces<F8<128>>()};
    return std::max(*std::max_element(std::begin(sizes), std::end(sizes)) * num_sms, kv8_rows_part_floats(num_sms));
}
int kv8_most_ctas(int num_sms) { return 4 * num_sms; }

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

// Time of one tile of 128 keys in all items of n sequences of `columns` columns each, over all SMs, when the codes come from L2
// (heads of 128; heads of 64 take as long).  A second launch costs 16 to 20 us: 8 sequences on 2048 keys 14.7 us in one launch,
// 32.4 in two; 64 on 2000 keys 36.7 and 38.4; 4 of 64 rows on 8192 keys 66 and 82.
double tiles_ns(const Kv8& c, int n, int columns) {
    const bool wide = c.cfg.dtype == CB_F32;
    const int per_item = wide ? (columns <= 4 ? 4 : 8) : columns <= 4 ? 4 : columns <= 8 ? 8 : columns <= 16 ? 16 : columns <= 32 ? 32 : 128;
    const double ns = wide ? (per_item == 4 ? 3.3 : 4.3) : per_item == 4 ? 2.7 : per_item == 8 ? 3.5 : per_item == 16 ? 5.5 : per_item == 32 ? 9.5 : 10.0;
    return (double)n * ((columns + per_item - 1) / per_item) * ns;
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
    {
        // One launch or two: the prefix read by each sequence (from L2, once one has read it) against a launch of its own.
        const int64_t pre_tiles = ((int64_t)pre.q.max_len + TK - 1) / TK, places = ((int64_t)r.n_rows + q.n) * p.Hkv * (pre_tiles + q.max_len / TK + 9);
        const double apart = tiles_ns(c, q.n, (r.n_rows + q.n - 1) / q.n * p.G) - tiles_ns(c, pre.q.n, (r.n_rows + pre.q.n - 1) / pre.q.n * p.G);
        const char* again = getenv("CB_SHARED_AGAIN");           // what reading it again may cost, ns
        if (apart * (double)(pre_tiles * p.Hkv) <= (again ? atof(again) : 17000.0) && places < 0x7fffffff)
            return many ? launch_kv8_rows(c, &own, JOINT, s) : launch_kv8_few_joint(c, &own, s);
    }
    p.prefix_sum = pre.scratch;
    p.prefix_stat = reinterpret_cast<float2*>(pre.scratch + (int64_t)r.n_rows * p.Hq * c.cfg.head_dim);
    p.voided = c.voided + 16;
    cudaError_t e = many_rows(c, p) ? launch_kv8_rows(c, &p, PREFIX, s) : launch_kv8_few_prefix(c, &p, s);
    if (e != cudaSuccess) return e;
    own.prefix_voided = p.voided;
    own.prefix_sum = p.prefix_sum;
    own.prefix_stat = p.prefix_stat;
    return many ? launch_kv8_rows(c, &own, OWN, s) : launch_kv8_few_own(c, &own, s);
}

}  // namespace cb
