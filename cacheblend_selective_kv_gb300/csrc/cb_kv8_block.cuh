// What writing, reading and appending rows of the 8-bit paged K/V cache share: the blocks that a call's rows touch, and
// 16-byte vectors of a row.
#pragma once
#include "cb_kv8.cuh"

namespace cb {

namespace {

// Which block a slot stands for.  With `each` rows per sequence, they touch at most per_seq blocks of it and the
// slots are s * per_seq ..; with ragged rows, n rows touch at most n / P + 2 blocks, so that start(s) / P + 2 s is a
// base that leaves every sequence room for its blocks.
struct Slots {
    int per_seq;              // > 0: equal rows
    int total;
};
Slots kv8_slots(const Kv8Seqs& q, const Kv8Rows& r) {
    const int P = 1 << q.shift;
    if (!r.start) {
        const int per = r.each > 0 ? (int)(((int64_t)r.each + P - 2) / P) + 1 : 0;
        return {per, per * q.n};
    }
    return {0, (r.n_rows >> q.shift) + 2 * q.n};
}

struct Block {
    int src_row;              // source row of logical row `first` of the sequence's new rows
    int lo, hi;               // rows of the block that belong to the call
    int page;
    int place;                // row lo's place in its sequence
};

__device__ __forceinline__ void kv8_bad_row(const Kv8Seqs& q, unsigned* also) {
    atomicOr(q.status, ST_BAD_ROW);
    if (also) atomicOr(also, ST_BAD_ROW);
}

// Offsets that decrease are recorded by the first CTA: the search below may pass them by.
__device__ __forceinline__ void kv8_check_offsets(const Kv8Seqs& q, const Kv8Rows& r) {
    if (!r.start || blockIdx.x > 0 || blockIdx.y > 0) return;
    for (int s = threadIdx.x; s < q.n; s += blockDim.x)
        if (r.start[s + 1] < r.start[s]) kv8_bad_row(q, nullptr);
}

// the block of slot u; false when the slot has none
__device__ __forceinline__ bool kv8_block(const Kv8Seqs& q, const Kv8Rows& r, int per_seq, int u, unsigned* also, Block& b) {
    int s, local;
    if (per_seq > 0) {
        s = u / per_seq;
        local = u - s * per_seq;
    } else {
        int a = 0, z = q.n - 1;                        // the last sequence whose base is at most u
        while (a < z) {
            const int m = (a + z + 1) >> 1;
            if ((r.start[m] >> q.shift) + 2 * m <= u) a = m; else z = m - 1;
        }
        s = a;
        local = u - ((r.start[s] >> q.shift) + 2 * s);
    }
    if (s >= q.n || local < 0) return false;
    int r0, r1, len;
    if (!kv8_rows(q, r, s, r0, r1, len)) {
        kv8_bad_row(q, also);
        return false;
    }
    const int n = r1 - r0;
    if (n == 0) return false;
    if (n > len) {
        if (len > 0) kv8_bad_row(q, also);             // (no length: a free place of the batch)
        return false;
    }
    const int P = 1 << q.shift, first = len - n;
    const int blk = (first >> q.shift) + local;
    if (blk > (len - 1) >> q.shift) return false;
    b.lo = max(first - blk * P, 0);
    b.hi = min(len - blk * P, P);
    b.place = blk * P + b.lo;
    b.src_row = r0 + b.place - first;                  // source row of block row lo
    b.page = kv8_page(q, s, blk);
    if (b.page < 0) kv8_bad_row(q, also);
    return b.page >= 0;
}

// maximum over the TPB threads of a group (TPB a power of two from 32 to 512)
__device__ __forceinline__ unsigned group_max(unsigned v, int tpb, unsigned* sm) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (tpb == 32) return v;
    const int warp = threadIdx.x >> 5, per = tpb >> 5, g0 = warp / per * per;
    if ((threadIdx.x & 31) == 0) sm[warp] = v;
    __syncthreads();
    v = sm[g0];
    for (int i = 1; i < per; ++i) v = max(v, sm[g0 + i]);
    return v;
}

// 16 bytes of a row.  Magnitudes compare as integers, so the largest is found on the packed words; the bits of an
// infinity or a NaN are above every finite number's, which is how a block that holds one is noticed, or a number from
// 248 * 2^120 on (LAST), which would round to a code whose value is not finite.
template <typename T> struct Vec;
template <> struct Vec<bf16> {
    static constexpr int N = 8;
    static constexpr unsigned LAST = 0x7f78u;
    __device__ static unsigned top(const uint4& u, unsigned m) {           // two running maxima in m
        m = kv8_max_u16x2(m, u.x & 0x7fff7fffu);
        m = kv8_max_u16x2(m, u.y & 0x7fff7fffu);
        m = kv8_max_u16x2(m, u.z & 0x7fff7fffu);
        return kv8_max_u16x2(m, u.w & 0x7fff7fffu);
    }
    __device__ static unsigned joined(unsigned m) { return max(m & 0xffffu, m >> 16); }
    __device__ static float value(unsigned bits) { return __uint_as_float(bits << 16); }
    __device__ static void get(const uint4& u, float* f) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <> struct Vec<float> {
    static constexpr int N = 4;
    static constexpr unsigned LAST = 0x7f780000u;
    __device__ static unsigned top(const uint4& u, unsigned m) {
        m = max(m, max(u.x & 0x7fffffffu, u.y & 0x7fffffffu));
        return max(m, max(u.z & 0x7fffffffu, u.w & 0x7fffffffu));
    }
    __device__ static unsigned joined(unsigned m) { return m; }
    __device__ static float value(unsigned bits) { return __uint_as_float(bits); }
    __device__ static void get(const uint4& u, float* f) {
        f[0] = __uint_as_float(u.x);
        f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z);
        f[3] = __uint_as_float(u.w);
    }
};

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

}  // namespace

}  // namespace cb
