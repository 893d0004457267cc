// Attention over the 8-bit paged K/V cache.  Query row i of a sequence's n sits at position len - n + i and sees
// keys 0 .. that position: out = softmax(q k * scale) v, the G query heads of a group sharing a KV head.  A row that
// sees nothing (its position is negative) gives 0.
//
// With weights, every key gets the sum of its softmax weights over the call's query rows and the group's heads.
//
// CUDA-core kernels: one CTA per (query row, KV head) streams 128 keys per step; the weights are computed by a second
// kernel, one CTA per 128 keys, from the rows' log-sum-exp.
#include "cb_kv8.cuh"

namespace cb {

namespace {

constexpr int KB = 128;   // keys per step (= threads)

struct AttnArgs {
    Kv8Seqs q;
    Kv8Rows r;
    Kv8Attn a;
    const uint8_t* kc;        // this layer's K and V codes [n_pages][Hkv][P][hd]
    const uint8_t* vc;
    const float* ks;          // [n_pages][Hkv]
    const float* vs;
    int Hq, Hkv, hd;
    float* lse;               // [n_q][Hq] (base e), or NULL
};

// sequence of query row i, or -1
__device__ __forceinline__ int seq_of(const Kv8Seqs& q, const Kv8Rows& r, int i) {
    if (!r.start) return i / r.each;
    int a = 0, z = q.n - 1;
    while (a < z) {
        const int m = (a + z + 1) >> 1;
        if (r.start[m] <= i) a = m; else z = m - 1;
    }
    return a;
}

template <typename T>
__global__ void __launch_bounds__(KB) kv8_attn_simt_kernel(const AttnArgs p) {
    extern __shared__ float sm[];
    const int i = blockIdx.x, g = blockIdx.y, G = p.Hq / p.Hkv, hd = p.hd, tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5, P = 1 << p.q.shift;
    float* qs = sm;                 // [G][hd]
    float* ps = qs + G * hd;        // [G][KB]
    float* vs = ps + G * KB;        // [KB][hd]
    float* mrun = vs + KB * hd;     // [G]
    float* lrun = mrun + G;
    float* alpha = lrun + G;
    const int s = seq_of(p.q, p.r, i);
    int r0, r1, len;
    if (!kv8_rows(p.q, p.r, s, r0, r1, len) || i < r0 || i >= r1) return;
    const int nk = len - (r1 - r0) + (i - r0) + 1;          // visible keys (<= 0: none)
    const T* qrow = (const T*)p.a.q + (int64_t)i * p.a.q_stride + (int64_t)g * G * hd;
    for (int t = tid; t < G * hd; t += KB) qs[t] = to_f(qrow[t]) * p.a.scale;
    if (tid < G) { mrun[tid] = -INFINITY; lrun[tid] = 0.f; }
    const int nslot = (G * hd + KB - 1) / KB;               // <= 8
    float acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    __syncthreads();
    for (int j0 = 0; j0 < nk; j0 += KB) {
        const int j = j0 + tid;
        int page = -1;
        if (j < nk) page = kv8_page(p.q, s, j >> p.q.shift);
        if (page >= 0) {
            const int64_t blk = (int64_t)page * p.Hkv + g;
            const uint16_t* kr = reinterpret_cast<const uint16_t*>(p.kc + (blk * P + (j & (P - 1))) * hd);
            const uint16_t* vr = reinterpret_cast<const uint16_t*>(p.vc + (blk * P + (j & (P - 1))) * hd);
            const float ksc = p.ks[blk], vsc = p.vs[blk];
            for (int gg = 0; gg < G; ++gg) {
                float a = 0.f;
                for (int d = 0; d < hd / 2; ++d) {
                    const float2 k2 = kv8_value2(kr[d]);
                    a = fmaf(qs[gg * hd + 2 * d], k2.x, fmaf(qs[gg * hd + 2 * d + 1], k2.y, a));
                }
                ps[gg * KB + tid] = a * ksc;
            }
            for (int d = 0; d < hd / 2; ++d) {
                const float2 v2 = kv8_value2(vr[d]);
                vs[tid * hd + 2 * d] = v2.x * vsc;
                vs[tid * hd + 2 * d + 1] = v2.y * vsc;
            }
        } else {
            for (int gg = 0; gg < G; ++gg) ps[gg * KB + tid] = -INFINITY;
            for (int d = 0; d < hd; ++d) vs[tid * hd + d] = 0.f;
        }
        __syncthreads();
        for (int gg = warp; gg < G; gg += KB / 32) {
            float mx = -INFINITY;
            for (int t = lane; t < KB; t += 32) mx = fmaxf(mx, ps[gg * KB + t]);
            mx = warp_max(mx);
            const float m_old = mrun[gg], m_new = fmaxf(m_old, mx);
            const float ref = m_new == -INFINITY ? 0.f : m_new;
            float sum = 0.f;
            for (int t = lane; t < KB; t += 32) {
                const float e = expf(ps[gg * KB + t] - ref);
                ps[gg * KB + t] = e;
                sum += e;
            }
            sum = warp_sum(sum);
            if (lane == 0) {
                const float a = m_old == -INFINITY ? 0.f : expf(m_old - m_new);
                alpha[gg] = a;
                lrun[gg] = lrun[gg] * a + sum;
                mrun[gg] = m_new;
            }
        }
        __syncthreads();
        for (int k = 0; k < nslot; ++k) {
            const int idx = tid + k * KB;
            if (idx >= G * hd) break;
            const int gg = idx / hd, d = idx % hd;
            float a = acc[k] * alpha[gg];
            for (int t = 0; t < KB; ++t) a = fmaf(ps[gg * KB + t], vs[t * hd + d], a);
            acc[k] = a;
        }
        __syncthreads();
    }
    T* orow = (T*)p.a.out + (int64_t)i * p.a.out_stride + (int64_t)g * G * hd;
    for (int k = 0; k < nslot; ++k) {
        const int idx = tid + k * KB;
        if (idx >= G * hd) break;
        orow[idx] = from_f<T>(nk > 0 ? acc[k] / lrun[idx / hd] : 0.f);
    }
    if (p.lse && tid < G) p.lse[(int64_t)i * p.Hq + g * G + tid] = mrun[tid] + logf(lrun[tid]);
}

template <typename T>
__global__ void __launch_bounds__(KB) kv8_weights_simt_kernel(const AttnArgs p) {
    extern __shared__ float qs[];   // [G][hd]
    const int j = blockIdx.x * KB + threadIdx.x, g = blockIdx.y, s = blockIdx.z;
    const int G = p.Hq / p.Hkv, hd = p.hd, P = 1 << p.q.shift;
    int r0, r1, len;
    if (!kv8_rows(p.q, p.r, s, r0, r1, len)) return;
    int page = -1;
    if (j < len) page = kv8_page(p.q, s, j >> p.q.shift);
    const int64_t blk = (int64_t)(page < 0 ? 0 : page) * p.Hkv + g;
    const uint16_t* kr = reinterpret_cast<const uint16_t*>(p.kc + (blk * P + (j & (P - 1))) * hd);
    const float ksc = page < 0 ? 0.f : p.ks[blk];
    float w = 0.f;
    for (int i = r0; i < r1; ++i) {
        const T* qrow = (const T*)p.a.q + (int64_t)i * p.a.q_stride + (int64_t)g * G * hd;
        __syncthreads();
        for (int t = threadIdx.x; t < G * hd; t += KB) qs[t] = to_f(qrow[t]) * p.a.scale;
        __syncthreads();
        if (page < 0 || j > len - (r1 - r0) + (i - r0)) continue;
        for (int gg = 0; gg < G; ++gg) {
            float a = 0.f;
            for (int d = 0; d < hd / 2; ++d) {
                const float2 k2 = kv8_value2(kr[d]);
                a = fmaf(qs[gg * hd + 2 * d], k2.x, fmaf(qs[gg * hd + 2 * d + 1], k2.y, a));
            }
            w += expf(a * ksc - p.lse[(int64_t)i * p.Hq + g * G + gg]);
        }
    }
    if (j < len) {
        float* dst = p.a.weights + ((int64_t)s * p.Hkv + g) * p.a.weights_ld + j;
        *dst = p.a.add ? *dst + w : w;
    }
}

template <typename T>
cudaError_t attention_typed(const AttnArgs& p, int n_q, cudaStream_t s) {
    const int G = p.Hq / p.Hkv;
    const size_t smem = sizeof(float) * ((size_t)G * p.hd + (size_t)G * KB + (size_t)KB * p.hd + 3 * G);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = smem_limit_once(kv8_attn_simt_kernel<T>, 96 * 1024, done);
    if (e != cudaSuccess) return e;
    if (n_q > 0) kv8_attn_simt_kernel<T><<<dim3(n_q, p.Hkv), KB, smem, s>>>(p);
    if (p.a.weights && p.q.max_len > 0)
        kv8_weights_simt_kernel<T><<<dim3((p.q.max_len + KB - 1) / KB, p.Hkv, p.q.n), KB, sizeof(float) * G * p.hd, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8_attention(const Kv8& c, const Kv8Seqs& q, const Kv8Rows& r, const Kv8Attn& a, int layer,
                                 cudaStream_t s) {
    const int Hkv = c.cfg.n_kv_heads, hd = c.cfg.head_dim;
    const int64_t blocks = c.cfg.n_pages * Hkv, k0 = (int64_t)layer * 2 * blocks, v0 = k0 + blocks;
    const int64_t bytes = (int64_t)hd << c.shift;
    AttnArgs p{q, r, a, c.codes + k0 * bytes, c.codes + v0 * bytes, c.scales + k0, c.scales + v0, c.cfg.n_heads, Hkv, hd,
               a.weights ? c.scores : nullptr};
    return c.cfg.dtype == CB_BF16 ? attention_typed<bf16>(p, r.n_rows, s) : attention_typed<float>(p, r.n_rows, s);
}

}  // namespace cb
