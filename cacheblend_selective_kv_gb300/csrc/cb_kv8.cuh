// 8-bit paged K/V cache: the parts its kernels share (block addressing, scales, e4m3 conversions).
//
// Pool: codes [L][2][n_pages][Hkv][P][hd] e4m3 bytes, scales [L][2][n_pages][Hkv] float.  A block (one page's rows
// of one KV head in one layer's K or V) is P * hd consecutive bytes, so a tile of an attention head is a few
// contiguous pieces whatever the number of heads.  A scale is a power of two (or 0 for a block of zeros): dividing
// by it and multiplying by it are exact in fp32, so the only rounding a value meets is the one to e4m3, and a
// code's value is exact in bf16.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "cb_common.cuh"

namespace cb {

// the cache handle (cb_kv8): the caller's buffers and the scratch of its calls
struct Kv8 {
    cb_kv8_config cfg;
    int device;
    int num_sms;
    int shift;               // log2(page_size)
    bool pdl;                // programmatic dependent launch
    uint8_t* codes;
    float* scales;
    unsigned* status;        // ST_* bits
    float* scores;           // weight_cells floats: attention calls that return weights
    float2* stats;           // their rows' (max, 1 / sum)
    float* part;             // attention: pieces of items that span CTAs
    int* todo;               // attention of many rows: items to be joined, four ints per CTA
    unsigned* arrived;       // attention: pieces finished, one count per CTA (0 between calls)
    unsigned* voided;        // attention: the last call's offsets decrease
    unsigned* opened;        // attention over a shared prefix: what its launches read is there (0 between calls)
    void* scratch;           // the allocation that holds the eight above
    unsigned* also;          // a blend's write and read: the model's status, which gets their bits too (else NULL)
    double again_ns;         // attention over a shared prefix in one launch: by how much it may be slower (CB_SHARED_AGAIN)
    alignas(64) unsigned char map[128];   // tensor map of the codes
};

// A batch of sequences as the kernels see it.
struct Kv8Seqs {
    int n;
    const int* table;        // [n][table_ld] page ids
    int table_ld;
    const int* lens;         // [n] rows in the cache, or NULL: max_len each
    int max_len;
    int64_t n_pages;
    int shift;
    unsigned* status;
};

// Rows that belong to the batch: sequence s owns rows start(s) .. start(s+1)-1 of an array of n_rows, and they are
// its last rows in the cache.
struct Kv8Rows {
    const int* start;        // [n + 1], or NULL: `each` rows per sequence
    int each;
    int n_rows;
};

__device__ __forceinline__ int kv8_len(const Kv8Seqs& q, int s) { return q.lens ? q.lens[s] : q.max_len; }

// rows [r0, r1) of sequence s; false (and a status bit) when the offsets or the length are out of range
__device__ __forceinline__ bool kv8_rows(const Kv8Seqs& q, const Kv8Rows& r, int s, int& r0, int& r1, int& len) {
    r0 = r.start ? r.start[s] : s * r.each;
    r1 = r.start ? r.start[s + 1] : r0 + r.each;
    len = kv8_len(q, s);
    if (r0 < 0 || r1 < r0 || r1 > r.n_rows || len < 0 || len > q.max_len) {
        atomicOr(q.status, ST_BAD_ROW);
        return false;
    }
    return true;
}

// page of block `blk` of sequence s, or -1 (and a status bit) for an id outside the pool
__device__ __forceinline__ int kv8_page(const Kv8Seqs& q, int s, int blk) {
    const int p = q.table[(int64_t)s * q.table_ld + blk];
    if (p < 0 || p >= q.n_pages) {
        atomicOr(q.status, ST_BAD_ROW);
        return -1;
    }
    return p;
}

// The smallest power of two sc with top <= 448 sc (0 for 0): 448 = 1.75 * 2^8.  Never below 2^-126, so that the
// scale and its reciprocal are normal numbers.
__device__ __forceinline__ float kv8_scale(float top) {
    if (!(top > 0.f)) return 0.f;
    const unsigned b = __float_as_uint(top);
    int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    if (e < 1) e = 1;
    return __uint_as_float((unsigned)e << 23);
}
// 1 / sc of a scale above (exact), 0 for 0
__device__ __forceinline__ float kv8_inverse(float sc) {
    return sc > 0.f ? __uint_as_float((254u << 23) - __float_as_uint(sc)) : 0.f;
}
// |x| for the block's largest value: infinities and NaN do not count
__device__ __forceinline__ float kv8_mag(float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;
}
// an infinity has no e4m3 code and is kept as NaN rather than as a large finite value
__device__ __forceinline__ float kv8_nan_inf(float x) { return fabsf(x) <= 3.402823466e38f ? x : __int_as_float(0x7fc00000); }
// A scale of 2^120 ends at the code 240, because 256 * 2^120 is not finite: finite values above 240 times it stand for that.
__device__ __forceinline__ float kv8_storable(float x) {
    const float m = 3.1901471e38f;                     // 240 * 2^120
    return fabsf(x) <= 3.402823466e38f ? fminf(fmaxf(x, -m), m) : __int_as_float(0x7fc00000);
}

__device__ __forceinline__ unsigned kv8_max_u16x2(unsigned a, unsigned b) {
    unsigned r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t kv8_code2(float a, float b) {           // codes of a (low byte) and b
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 kv8_value2(uint32_t c2) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c2 & 0xffffu), __NV_E4M3);
    return __half22float2(__half2(h));
}
__device__ __forceinline__ __half2 kv8_half2(uint32_t c2) {
    return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c2 & 0xffffu), __NV_E4M3));
}
// A power of two by which codes are multiplied, as two factors that fit in fp16 (2^-24 .. 2^9 each): a product that is
// neither 0 nor above 448 needs a factor within 2^-19 .. 2^18, and outside of that both give 0 or are never asked for.
struct Kv8Factor {
    __half2 a, b;
};
__device__ __forceinline__ Kv8Factor kv8_factor(float f) {
    const float a = fminf(fmaxf(f, 5.9604645e-8f), 512.f), b = f > 512.f ? fminf(f * (1.f / 512.f), 512.f) : 1.f;
    return Kv8Factor{__float2half2_rn(a), __float2half2_rn(b)};
}
// Four codes whose values are multiplied by it and rounded to e4m3 again.  An e4m3 value has four significant bits, so
// the products are exact in fp16 down to 2^-21, far below the 2^-10 under which e4m3 rounds to 0.
__device__ __forceinline__ uint32_t kv8_rescale4(uint32_t c4, const Kv8Factor& f) {
    const __half2 lo = __hmul2(__hmul2(kv8_half2(c4), f.a), f.b), hi = __hmul2(__hmul2(kv8_half2(c4 >> 16), f.a), f.b);
    return (uint32_t)__nv_cvt_halfraw2_to_fp8x2(__half2_raw(lo), __NV_SATFINITE, __NV_E4M3) |
           ((uint32_t)__nv_cvt_halfraw2_to_fp8x2(__half2_raw(hi), __NV_SATFINITE, __NV_E4M3) << 16);
}

// ------------------------------------------------------------------------------------------------
// launchers
// ------------------------------------------------------------------------------------------------
struct Kv8Io {                // contiguous K/V rows beside the cache
    void* k;
    void* v;
    int64_t layer_stride;     // elements between layers
    int64_t row_stride;       // elements between rows ([Hkv][hd] inside a row is contiguous)
    bool bf16;
};
cudaError_t launch_kv8_write(const Kv8& c, const Kv8Seqs& q, const Kv8Rows& r, const Kv8Io& io, int layer, int n_layers,
                             cudaStream_t s);
cudaError_t launch_kv8_read(const Kv8& c, const Kv8Seqs& q, const Kv8Rows& r, const Kv8Io& io, int layer, int n_layers,
                            cudaStream_t s);

struct Kv8Append {            // rows of a fused projection or of their own; [heads][hd] inside a row is contiguous
    const void* q;            // or NULL
    int64_t q_stride;
    void* out_q;
    int64_t out_q_stride;
    const void* k;
    const void* v;
    int64_t kv_stride;
    const int* positions;     // [n_rows] or NULL
    double theta;
};
cudaError_t launch_kv8_append(const Kv8& c, const Kv8Seqs& q, const Kv8Rows& r, const Kv8Append& p, int layer, cudaStream_t s);

struct Kv8Attn {
    const void* q;            // [n_q][Hq][hd]
    int64_t q_stride;         // elements between rows
    void* out;
    int64_t out_stride;
    float scale;
    float* weights;           // [n_seqs][Hkv][weights_ld] or NULL
    int weights_ld;
    bool add;                 // add to the weights instead of writing them
};
cudaError_t launch_kv8_attention(const Kv8& c, const Kv8Seqs& q, const Kv8Rows& r, const Kv8Attn& a, int layer,
                                 cudaStream_t s);

size_t kv8_part_floats(int num_sms, bool shared);
size_t kv8_rows_part_floats(int num_sms);
// many query rows per sequence (kv8_attn_rows.cu); attn_args: the AttnArgs of launch_kv8_attention, mode: what it computes
cudaError_t launch_kv8_rows(const Kv8& c, const void* attn_args, int mode, cudaStream_t s);

struct Kv8Prefix {            // prefixes that the batch's sequences share
    Kv8Seqs q;                // a group's prefix as a sequence
    const int* first;         // [groups + 1] first sequence of each group, or NULL: `per_group` each
    int per_group;
    float* scratch;           // n_q * n_heads * (2 * head_dim + 6) floats
};
cudaError_t launch_kv8_shared(const Kv8& c, const Kv8Prefix& pre, const Kv8Seqs& q, const Kv8Rows& r, const Kv8Attn& a, int layer,
                              cudaStream_t s);
cudaError_t launch_kv8_few_prefix(const Kv8& c, void* attn_args, cudaStream_t s);
cudaError_t launch_kv8_few_own(const Kv8& c, const void* attn_args, cudaStream_t s);
cudaError_t launch_kv8_few_joint(const Kv8& c, const void* attn_args, cudaStream_t s);
int kv8_most_ctas(int num_sms, bool shared);
bool kv8_make_map(const Kv8& c, void* out);

struct Kv8Evict {
    const int* dst_table;
    int dst_ld;
    const float* weights;     // [n_layers][n_seqs][Hkv][weights_ld]
    float* out_weights;
    int weights_ld;
    int keep, sink, recent;
    int* out_rows;            // [n_layers][n_seqs][Hkv][keep]
    int* out_lens;            // [n_seqs]
};
cudaError_t launch_kv8_evict(const Kv8& c, const Kv8Seqs& q, const Kv8Evict& e, int layer, int n_layers, cudaStream_t s);

}  // namespace cb

struct cb_kv8 : public cb::Kv8 {};
