// 8-bit paged K/V cache: writing rows into it and reading them back.
//
// write: a block's scale is the smallest power of two s with max|x| <= 448 s, a row's code e4m3(x / s).  A block that
// already holds earlier rows of the sequence keeps max(old scale, new rows' scale); its old codes are rounded to
// the larger one when it grew.
// read: code * s, exact in bf16 and fp32.
//
// Both are bound by HBM: 2 or 4 bytes a value on one side, 1 on the other.  Work is split by block: TPB threads
// (32..256) hold one block's rows in registers as NP 16-byte vectors each, find the block's largest value with one
// reduction and store the codes, so every row is read once and a code block is written as one contiguous piece.
// 8256 rows x 32 layers of 8 heads of 128 (1.62 GB in all): written in 250 us (96 % of the measured copy rate), 8192 rows read
// back in 233 us (102 %).
#include "cb_kv8_block.cuh"

namespace cb {

namespace {

constexpr int THREADS = 256;
constexpr int VECTORS = 8;             // 16-byte vectors of a row per thread, where blocks are large enough

struct CacheArgs {
    Kv8Seqs q;
    Kv8Rows r;
    const void* src[2];
    int64_t layer_stride, row_stride;
    uint8_t* codes;
    float* scales;
    unsigned* also;           // a second status word, or NULL
    int per_seq, units;       // units = slots * Hkv
    int Hkv, hd, layer;
    int tpb_shift;            // log2 of the threads of a block's group
    int vpr_shift;            // log2 of the vectors of a row
};

// NP vectors per thread: vector t + i * tpb of the block, tpb / vpr rows apart
template <typename T, int NP>
__global__ void __launch_bounds__(THREADS) kv8_write_kernel(const CacheArgs a) {
    constexpr int VN = Vec<T>::N;
    grid_dep_launch();
    grid_dep_wait();
    __shared__ unsigned sm[THREADS / 32];
    kv8_check_offsets(a.q, a.r);
    const int tpb = 1 << a.tpb_shift, group = threadIdx.x >> a.tpb_shift, t = threadIdx.x & (tpb - 1);
    const int unit = blockIdx.x * (THREADS >> a.tpb_shift) + group;
    const int lk = blockIdx.y, kv = lk & 1, l = lk >> 1;
    const int P = 1 << a.q.shift;
    Block b{};
    const int slot = unit / a.Hkv, head = unit - slot * a.Hkv;
    const bool live = unit < a.units && kv8_block(a.q, a.r, a.per_seq, slot, a.also, b);
    const int row0 = t >> a.vpr_shift, rows = tpb >> a.vpr_shift, e = (t & ((1 << a.vpr_shift) - 1)) * VN;
    const int64_t blk = ((int64_t)((a.layer + l) * 2 + kv) * a.q.n_pages + b.page) * a.Hkv + head;
    uint4 x[NP];
    float was = 0.f;
    if (live) {
        const T* src = (const T*)a.src[kv] + l * a.layer_stride + (int64_t)head * a.hd + e +
                       (int64_t)(b.src_row - b.lo) * a.row_stride;
        if (b.lo > 0) was = a.scales[blk];             // earlier rows of the sequence stay in the block
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int row = row0 + i * rows;
            x[i] = row >= b.lo && row < b.hi ? __ldcs(reinterpret_cast<const uint4*>(src + row * a.row_stride)) : make_uint4(0, 0, 0, 0);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) x[i] = make_uint4(0, 0, 0, 0);
    }
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) m = Vec<T>::top(x[i], m);
    unsigned top = group_max(Vec<T>::joined(m), tpb, sm);
    const bool special = top >= Vec<T>::LAST;          // the finite maximum, infinities to NaN, what is storable of the rest
    if (__syncthreads_or(special)) {
        float f[VN], f_top = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            Vec<T>::get(x[i], f);
#pragma unroll
            for (int k = 0; k < VN; ++k) f_top = fmaxf(f_top, kv8_mag(f[k]));
        }
        f_top = __uint_as_float(group_max(__float_as_uint(f_top), tpb, sm));
        if (special) top = sizeof(T) == 2 ? __float_as_uint(f_top) >> 16 : __float_as_uint(f_top);
    }
    if (!live) return;                                 // no barrier of all threads below
    uint8_t* dst = a.codes + blk * P * a.hd;
    float sc = kv8_scale(Vec<T>::value(top));
    if (b.lo > 0) {
        if (was >= sc) {
            sc = was;
        } else if (was > 0.f) {                        // (codes of a block of zeros stay as they are)
            const Kv8Factor f = kv8_factor(was * kv8_inverse(sc));
            for (int i = t; i < b.lo * a.hd / 16; i += tpb) {
                uint4 c = reinterpret_cast<uint4*>(dst)[i];
                c.x = kv8_rescale4(c.x, f);
                c.y = kv8_rescale4(c.y, f);
                c.z = kv8_rescale4(c.z, f);
                c.w = kv8_rescale4(c.w, f);
                reinterpret_cast<uint4*>(dst)[i] = c;
            }
        }
    }
    const float inv = kv8_inverse(sc);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int row = row0 + i * rows;
        float f[VN];
        Vec<T>::get(x[i], f);
        if (special) {
#pragma unroll
            for (int k = 0; k < VN; ++k) f[k] = kv8_storable(f[k]);
        }
        uint32_t w[VN / 4];
#pragma unroll
        for (int k = 0; k < VN / 4; ++k)
            w[k] = kv8_code2(f[4 * k] * inv, f[4 * k + 1] * inv) | (kv8_code2(f[4 * k + 2] * inv, f[4 * k + 3] * inv) << 16);
        if (row < b.lo || row >= b.hi) continue;
        uint8_t* d = dst + row * a.hd + e;
        if (VN == 8) *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[VN / 4 - 1]);
        else *reinterpret_cast<uint32_t*>(d) = w[0];
    }
    if (b.lo > 0) {                                    // every thread of the group has read the old scale
        if (tpb > 32) asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpb) : "memory");
        else __syncwarp();
    }
    if (t == 0) a.scales[blk] = sc;
}

template <typename T> __device__ __forceinline__ uint4 pack_values(const float* f);
template <> __device__ __forceinline__ uint4 pack_values<bf16>(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ uint4 pack_values<float>(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// one vector of values (8 or 4 codes) per step, four steps loaded before the first is stored
template <typename T>
__global__ void __launch_bounds__(THREADS) kv8_read_kernel(const CacheArgs a) {
    constexpr int VN = Vec<T>::N, NB = 4;
    grid_dep_launch();
    grid_dep_wait();
    kv8_check_offsets(a.q, a.r);
    const int tpb = 1 << a.tpb_shift, group = threadIdx.x >> a.tpb_shift, t = threadIdx.x & (tpb - 1);
    const int unit = blockIdx.x * (THREADS >> a.tpb_shift) + group;
    const int lk = blockIdx.y, kv = lk & 1, l = lk >> 1;
    const int P = 1 << a.q.shift;
    Block b{};
    const int slot = unit / a.Hkv, head = unit - slot * a.Hkv;
    if (unit >= a.units || !kv8_block(a.q, a.r, a.per_seq, slot, a.also, b)) return;
    const int row0 = t >> a.vpr_shift, rows = tpb >> a.vpr_shift, e = (t & ((1 << a.vpr_shift) - 1)) * VN;
    const int64_t blk = ((int64_t)((a.layer + l) * 2 + kv) * a.q.n_pages + b.page) * a.Hkv + head;
    const uint8_t* src = a.codes + blk * P * a.hd + e;
    const float sc = a.scales[blk];
    T* dst = (T*)a.src[kv] + l * a.layer_stride + (int64_t)head * a.hd + e + (int64_t)(b.src_row - b.lo) * a.row_stride;
    for (int r0 = row0 + b.lo; r0 < b.hi; r0 += NB * rows) {
        uint32_t c[NB][VN / 4];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int row = r0 + i * rows;
            if (row >= b.hi) continue;
            if constexpr (VN == 8) {
                const uint2 u = __ldcs(reinterpret_cast<const uint2*>(src + row * a.hd));
                c[i][0] = u.x;
                c[i][1] = u.y;
            } else {
                c[i][0] = __ldcs(reinterpret_cast<const uint32_t*>(src + row * a.hd));
            }
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int row = r0 + i * rows;
            if (row >= b.hi) continue;
            float f[VN];
#pragma unroll
            for (int k = 0; k < VN / 4; ++k) {
                const float2 p = kv8_value2(c[i][k]), z = kv8_value2(c[i][k] >> 16);
                f[4 * k] = p.x * sc;
                f[4 * k + 1] = p.y * sc;
                f[4 * k + 2] = z.x * sc;
                f[4 * k + 3] = z.y * sc;
            }
            __stcs(reinterpret_cast<uint4*>(dst + row * a.row_stride), pack_values<T>(f));
        }
    }
}

CacheArgs cache_args(const Kv8& c, const Kv8Seqs& q, const Kv8Rows& r, const Kv8Io& io, int layer, int es) {
    CacheArgs a{};
    const Slots sl = kv8_slots(q, r);
    a.q = q;
    a.r = r;
    a.src[0] = io.k;
    a.src[1] = io.v;
    a.layer_stride = io.layer_stride;
    a.row_stride = io.row_stride;
    a.codes = c.codes;
    a.scales = c.scales;
    a.also = c.also;
    a.per_seq = sl.per_seq;
    a.Hkv = c.cfg.n_kv_heads;
    a.units = sl.total * a.Hkv;
    a.hd = c.cfg.head_dim;
    a.layer = layer;
    // Vectors of 16 bytes per thread: what a thread does once (finding its block) is spread over more of them, and
    // they are in flight together.  Eight (8K x 32 layers of the 8B shape written in
    // 250 us, four in 340).
    const int want = (1 << q.shift) * a.hd * es / (16 * VECTORS);
    a.tpb_shift = log2_of(want < 32 ? 32 : (want > THREADS ? THREADS : want));
    a.vpr_shift = log2_of(a.hd * es / 16);
    return a;
}

template <typename T>
cudaError_t write_typed(const CacheArgs& a, int n_layers, int np, bool pdl, cudaStream_t s) {
    const int groups = THREADS >> a.tpb_shift;
    const dim3 grid((a.units + groups - 1) / groups, 2 * n_layers);
    switch (np) {
        case 4: return launch_ex(pdl, kv8_write_kernel<T, 4>, grid, dim3(THREADS), 0, s, a);
        case 8: return launch_ex(pdl, kv8_write_kernel<T, 8>, grid, dim3(THREADS), 0, s, a);
        case 16: return launch_ex(pdl, kv8_write_kernel<T, 16>, grid, dim3(THREADS), 0, s, a);
        default:                                       // fp32 rows, head_dim 128, 256 rows per page
            if constexpr (sizeof(T) == 4) return launch_ex(pdl, kv8_write_kernel<T, 32>, grid, dim3(THREADS), 0, s, a);
            return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_kv8_write(const Kv8& c, const Kv8Seqs& q, const Kv8Rows& r, const Kv8Io& io, int layer, int n_layers,
                             cudaStream_t s) {
    const int es = io.bf16 ? 2 : 4;
    const CacheArgs a = cache_args(c, q, r, io, layer, es);
    if (a.units == 0 || n_layers == 0) return cudaSuccess;
    const int np = ((1 << q.shift) * a.hd * es / 16) >> a.tpb_shift;
    return io.bf16 ? write_typed<bf16>(a, n_layers, np, c.pdl, s) : write_typed<float>(a, n_layers, np, c.pdl, s);
}

cudaError_t launch_kv8_read(const Kv8& c, const Kv8Seqs& q, const Kv8Rows& r, const Kv8Io& io, int layer, int n_layers,
                            cudaStream_t s) {
    const CacheArgs a = cache_args(c, q, r, io, layer, io.bf16 ? 2 : 4);
    if (a.units == 0 || n_layers == 0) return cudaSuccess;
    const int groups = THREADS >> a.tpb_shift;
    const dim3 grid((a.units + groups - 1) / groups, 2 * n_layers);
    return io.bf16 ? launch_ex(c.pdl, kv8_read_kernel<bf16>, grid, dim3(THREADS), 0, s, a)
                   : launch_ex(c.pdl, kv8_read_kernel<float>, grid, dim3(THREADS), 0, s, a);
}

}  // namespace cb
