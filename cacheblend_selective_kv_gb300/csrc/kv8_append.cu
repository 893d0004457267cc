// 8-bit paged K/V cache: appending rows whose q and k are rotated on the way (a decoding step, a prompt in pieces).
//
// Pair (2i, 2i + 1) of a head turns by the angle p theta^(-2i / hd) of its row's position p; k and v then go into their
// blocks as cb_kv8_write puts rows there, q goes to its output.  K meets one rounding, from the rotated fp32 value to its code.
//
// The angle.  The host gives every pair's float64 frequency as a 64-bit fraction of a turn, so that p times it modulo 2^64 is the phase
// of any int32 position, within 2^-33 turns: no reduction of a large angle in floating point.  Its upper 32 bits less the nearest quarter
// turn go to fp32, an angle within pi / 4, and from there the Taylor series of sine and cosine to x^9 and x^10; quarter turns exchange the
// two and change their signs.  (The special-function unit's sine and cosine, within 2^-20.5, made 8192 rows 34.0 us instead of 36.4, but
// moved codes at e4m3's borders.)
//
// Codes and scales are those of exact rotation.  Over all 2^32 phases the vector (cosine, sine) is off by at most 1.266e-7, to which the
// cut to 32 bits adds 1.5e-9 and the farthest positions 0.7e-9; the product and the sum are rounded by 2^-24 of the pair's length each.  A turned value is
// then off by less than 2.5e-7 of that length, and the length is at most the sum of the pair's two magnitudes.  Where the values less and
// plus that much do not have the same code (a pair of about 10 000), or the scales of maxima less and plus it differ, the pairs in question
// are turned again in 64 bits.  Left out are blocks with NaN, infinities or numbers from 248 * 2^120 on, and with none above 2^-100, whose
// codes are those of the fp32 values.
//
// Work, in one launch: the blocks that get rows of K, those of V, then q.  A block's rows stand in one group of 32 .. 512 threads,
// as 32 values per thread where there are that many, from the load to the largest value to the code; a decoding step's single
// rows are a warp each.  A thread of q has one vector of a row in several heads, which share its sines and cosines; the first
// four are under way while the row's sequence is looked up.
//
// 32 heads and 8 KV heads of 128, bf16: 8192 rows 38.6 us, 70 % of the measured copy rate (bound by HBM, and by the instructions of K
// and V, which alone take about half of it; in fp32 78.8 us, 66 %); one row of each of 64 sequences 4.3 us, one launch, of whose 33 thousand
// pairs some are nearly always turned again (3.1 us where none is).
#include <cmath>

#include "cb_kv8_block.cuh"

namespace cb {

namespace {

constexpr int MOST = 512;                // threads of a block's group, at most
constexpr int QB = 4;                    // heads of q that a thread has under way
// How far a turned value may be off, of the sum of its pair's magnitudes: 2.5e-7, and the rounding of value less and plus that.
constexpr float OFF = 3.2e-7f;

struct Turns {
    uint2 of[64];                        // pair i turns by (y 2^32 + x) / 2^64 per position
};

struct AppendArgs {
    Kv8Seqs q;
    Kv8Rows r;
    const void* src[2];                  // K, V rows
    int64_t kv_stride;
    const void* in_q;                    // or NULL
    void* out_q;
    int64_t q_stride, out_q_stride;
    const int* positions;                // [n_rows] or NULL: a row's place in its sequence
    uint8_t* codes;
    float* scales;
    int per_seq, units;                  // units = slots * Hkv
    int Hkv, Hq, hd, layer;
    int tpb_shift, vpr_shift;            // log2 of a group's threads, of a row's 16-byte vectors
    int kv_ctas;                         // CTAs of K, and of V; q's follow
    int q_heads, q_chunks;               // heads per thread of q, threads per row's vector
};

// the upper half of the phase of position p, in 2^-32 turns
__device__ __forceinline__ unsigned phase_of(int p, uint2 turn) {
    return __umulhi((unsigned)p, turn.x) + (unsigned)p * turn.y - (p < 0 ? turn.x : 0u);
}
// cosine and sine of a phase
__device__ __forceinline__ float2 cos_sin(unsigned phase) {
    const unsigned quarter = (phase + 0x20000000u) >> 30;
    const float x = (float)(int)(phase - (quarter << 30)) * 1.4629180792671596e-9f;      // 2 pi 2^-32
    const float z = x * x;
    float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f), c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
    s = fmaf(z, s, 8.3333333e-3f);
    c = fmaf(z, c, -1.3888889e-3f);
    s = fmaf(z, s, -1.6666667e-1f);
    c = fmaf(z, c, 4.1666667e-2f);
    s = fmaf(x * z, s, x);
    c = fmaf(z, c, -0.5f);
    c = fmaf(z, c, 1.f);
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}
// a vector's values turned by its pairs' angles at one position
template <typename T> struct Rotation {
    static constexpr int NP = Vec<T>::N / 2;
    float2 cs[NP];
    __device__ __forceinline__ void set(const uint2* turn, int position) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const unsigned phase = phase_of(position, turn[k]);
            cs[k] = cos_sin(phase);
        }
    }
    __device__ __forceinline__ void apply(float* f) const {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const float2 y = rotate_pair(f[2 * k], f[2 * k + 1], cs[k]);
            f[2 * k] = y.x;
            f[2 * k + 1] = y.y;
        }
    }
};

template <typename T> __device__ __forceinline__ uint4 pack(const float* f);
template <> __device__ __forceinline__ uint4 pack<bf16>(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ uint4 pack<float>(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// place of row `row` in its sequence; false where it is not written (as kv8_block decides for K and V)
__device__ __forceinline__ bool place_of(const Kv8Seqs& q, const Kv8Rows& r, int row, int& place) {
    int s = 0;
    if (r.start) {
        int z = q.n - 1;                               // the last sequence that begins at or before the row
        while (s < z) {
            const int m = (s + z + 1) >> 1;
            if (r.start[m] <= row) s = m; else z = m - 1;
        }
    } else {
        s = row / r.each;
    }
    int r0, r1, len;
    if (!kv8_rows(q, r, s, r0, r1, len) || row < r0 || row >= r1 || r1 - r0 > len) return false;
    place = len - (r1 - r0) + row - r0;
    return true;
}

// A pair turned in 64 bits, within 1e-13 of its length (and 2 pi 2^-64 for every position).
template <typename T> __device__ __noinline__ double2 exact_pair(const T* src, uint2 turn, int position) {
    const double x0 = (double)to_f(src[0]), x1 = (double)to_f(src[1]);
    const unsigned long long phase = (unsigned long long)(long long)position * (((unsigned long long)turn.y << 32) | turn.x);
    const unsigned long long quarter = (phase + (1ull << 61)) >> 62;
    const double x = (double)(long long)(phase - (quarter << 62)) * 3.40612158008655e-19, z = x * x;      // 2 pi 2^-64
    // the series of sine and cosine, to x^13 and x^14: off by at most 3e-14
    double s = fma(z, 1. / 6227020800, -1. / 39916800), c = fma(z, -1. / 87178291200, 1. / 479001600);
    s = fma(z, s, 1. / 362880);
    c = fma(z, c, -1. / 3628800);
    s = fma(z, s, -1. / 5040);
    c = fma(z, c, 1. / 40320);
    s = fma(z, s, 1. / 120);
    c = fma(z, c, -1. / 720);
    s = fma(z, s, -1. / 6);
    c = fma(z, c, 1. / 24);
    s = fma(x * z, s, x);
    c = fma(z, c, -0.5);
    c = fma(z, c, 1.);
    const double p = quarter & 1 ? s : c, q = quarter & 1 ? c : s;
    const double cosine = (quarter + 1) & 2 ? -p : p, sine = quarter & 2 ? -q : q;
    return make_double2(x0 * cosine - x1 * sine, x0 * sine + x1 * cosine);
}
// rounded to odd, so that the rounding to a code is the only one
__device__ __forceinline__ float to_odd(double y) {
    const float f = __double2float_rz(y);
    return (double)f == y ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// NV vectors per thread: vector t + i * tpb of the call's rows in the block, tpb / vpr rows apart.  KV: 0 for K, 1 for V (code of its own for
// each: 8192 rows 39.5 us a call, 40.8 with one for both)
template <typename T, int NV, int KV>
__device__ __forceinline__ void append_kv(const AppendArgs& a, const uint2* turns, int cta) {
    constexpr int VN = Vec<T>::N;
    __shared__ unsigned sm[MOST / 32];
    const int tpb = 1 << a.tpb_shift, group = threadIdx.x >> a.tpb_shift, t = threadIdx.x & (tpb - 1);
    const int unit = cta * ((int)blockDim.x >> a.tpb_shift) + group;
    const int P = 1 << a.q.shift;
    Block b{};
    const int slot = unit / a.Hkv, head = unit - slot * a.Hkv;
    const bool live = unit < a.units && kv8_block(a.q, a.r, a.per_seq, slot, nullptr, b);
    const int row0 = b.lo + (t >> a.vpr_shift), rows = tpb >> a.vpr_shift, e = (t & ((1 << a.vpr_shift) - 1)) * VN;
    const int64_t blk = ((int64_t)(a.layer * 2 + KV) * a.q.n_pages + b.page) * a.Hkv + head;
    float f[NV][VN];
    unsigned most = 0;                                 // the largest magnitude's bits, those of an infinity or a NaN among them
    float was = 0.f;
    if (live) {
        const T* src = (const T*)a.src[KV] + (int64_t)head * a.hd + e;
        if (b.lo > 0) was = a.scales[blk];             // earlier rows of the sequence stay in the block
        uint4 x[NV];
        int position[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int row = row0 + i * rows, from = b.src_row + row - b.lo;
            x[i] = make_uint4(0, 0, 0, 0);
            position[i] = 0;
            if (row >= b.hi) continue;
            x[i] = __ldcs(reinterpret_cast<const uint4*>(src + (int64_t)from * a.kv_stride));
            if (KV == 0) position[i] = a.positions ? a.positions[from] : b.place + row - b.lo;
        }
        uint2 turn[VN / 2];
#pragma unroll
        for (int k = 0; k < VN / 2; ++k) turn[k] = turns[e / 2 + k];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Vec<T>::get(x[i], f[i]);
            if (row0 + i * rows >= b.hi) continue;
            if (KV == 0) {
                Rotation<T> turned;
                turned.set(turn, position[i]);
                turned.apply(f[i]);
            }
#pragma unroll
            for (int k = 0; k < VN; ++k) most = max(most, __float_as_uint(f[i][k]) & 0x7fffffffu);
        }
    }
    most = group_max(most, tpb, sm);
    // pair `at` of this thread's (bits of a mask), turned in 64 bits
    const auto exact_at = [&](int at) {
        const int d = e + at % (VN / 2) * 2, from = b.src_row + row0 + at / (VN / 2) * rows - b.lo;
        return exact_pair((const T*)a.src[0] + (int64_t)head * a.hd + d + (int64_t)from * a.kv_stride, turns[d / 2],
                          a.positions ? a.positions[from] : b.place + from - b.src_row);
    };
    static_assert(NV * VN / 2 <= 32, "a bit for every pair");
    // infinities, NaN, and numbers that would round to a code whose value is not finite, are looked at one by one
    const bool special = most >= Vec<float>::LAST;
    // a maximum whose scale fp32 does not decide: all of its values are within 2^-21 of the largest
    float sc = kv8_scale(__uint_as_float(most));
    const auto scale_with = [&](float off) { return kv8_scale(__uint_as_float(most) * (1.f + off)); };
    const bool edge = KV == 0 && !special && scale_with(-0x1p-21f) != scale_with(0x1p-21f);
    if (__syncthreads_or(special || edge)) {
        unsigned found = 0;                            // special: the largest finite magnitude; edge: whether the larger scale is needed
        if (live && special) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
#pragma unroll
                for (int k = 0; k < VN; ++k) {
                    if (row0 + i * rows < b.hi) top = fmaxf(top, kv8_mag(f[i][k]));
                    f[i][k] = kv8_storable(f[i][k]);
                }
            }
            found = __float_as_uint(top);
        } else if (live && edge) {
            const float border = 448.f * scale_with(-0x1p-21f), from = border * (1.f - 0x1p-20f);
            unsigned left = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
#pragma unroll
                for (int k = 0; k < VN; k += 2)
                    if (row0 + i * rows < b.hi && fmaxf(fabsf(f[i][k]), fabsf(f[i][k + 1])) >= from) left |= 1u << (i * (VN / 2) + k / 2);
            }
#pragma unroll 1
            for (; left; left &= left - 1) {
                const double2 y = exact_at(__ffs(left) - 1);
                if (fmax(fabs(y.x), fabs(y.y)) > (double)border) found = 1;
            }
        }
        found = group_max(found, tpb, sm);
        if (special) sc = kv8_scale(__uint_as_float(found));
        else if (edge) sc = scale_with(found ? 0x1p-21f : -0x1p-21f);
    }
    if (!live) return;                                 // no barrier of all threads below
    uint8_t* dst = a.codes + blk * P * a.hd;
    if (b.lo > 0) {
        if (was >= sc) {
            sc = was;
        } else if (was > 0.f) {                        // (codes of a block of zeros stay as they are)
            const Kv8Factor by = kv8_factor(was * kv8_inverse(sc));
            for (int i = t; i < b.lo * a.hd / 16; i += tpb) {
                uint4 c = reinterpret_cast<uint4*>(dst)[i];
                c.x = kv8_rescale4(c.x, by);
                c.y = kv8_rescale4(c.y, by);
                c.z = kv8_rescale4(c.z, by);
                c.w = kv8_rescale4(c.w, by);
                reinterpret_cast<uint4*>(dst)[i] = c;
            }
        }
    }
    const float inv = kv8_inverse(sc), off = OFF * inv;
    unsigned near = 0;                                 // pairs with a value whose code fp32 does not decide
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int row = row0 + i * rows;
        if (row >= b.hi) continue;
        uint32_t w[VN / 2];
#pragma unroll
        for (int k = 0; k < VN / 2; ++k) {
            const float x = f[i][2 * k], y = f[i][2 * k + 1];
            if (KV == 0) {
                const float by = special ? 0.f : fmaf(fabsf(x), off, fabsf(y) * off);      // (one of the two may be NaN there; |x| + |y| may pass fp32)
                w[k] = kv8_code2(fmaf(x, inv, -by), fmaf(y, inv, -by));
                // (the sign of a 0 does not count: 0 turned may be -0; other codes of opposite signs are farther apart than twice `by`, at most 6e-4)
                if ((w[k] ^ kv8_code2(fmaf(x, inv, by), fmaf(y, inv, by))) & 0x7f7fu) near |= 1u << (i * (VN / 2) + k);
            } else {
                w[k] = kv8_code2(x * inv, y * inv);
            }
        }
        uint8_t* d = dst + row * a.hd + e;
        if constexpr (VN == 8) *reinterpret_cast<uint2*>(d) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        else *reinterpret_cast<uint32_t*>(d) = w[0] | w[1] << 16;
    }
#pragma unroll 1
    for (unsigned left = special ? 0u : near; left; left &= left - 1) {
        const int at = __ffs(left) - 1;
        const double2 y = exact_at(at);
        *reinterpret_cast<uint16_t*>(dst + (row0 + at / (VN / 2) * rows) * a.hd + e + at % (VN / 2) * 2) =
            (uint16_t)kv8_code2(to_odd(y.x * inv), to_odd(y.y * inv));
    }
    if (b.lo > 0) {                                    // every thread of the group has read the old scale
        if (tpb > 32) asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpb) : "memory");
        else __syncwarp();
    }
    if (t == 0) a.scales[blk] = sc;
}

template <typename T> __device__ __forceinline__ void append_q(const AppendArgs& a, const uint2* turns, int cta) {
    constexpr int VN = Vec<T>::N;
    const int64_t at = (int64_t)cta * blockDim.x + threadIdx.x, item = at >> a.vpr_shift;
    const int64_t row = item / a.q_chunks;
    if (row >= a.r.n_rows) return;
    const int chunk = (int)(item - row * a.q_chunks), e = ((int)at & ((1 << a.vpr_shift) - 1)) * VN;
    const T* src = (const T*)a.in_q + row * a.q_stride + e;
    const int h1 = min(a.Hq, (chunk + 1) * a.q_heads);
    int h0 = chunk * a.q_heads;
    uint4 x[QB];                                       // the first heads are under way while the row is looked up
#pragma unroll
    for (int i = 0; i < QB; ++i)
        if (h0 + i < h1) x[i] = __ldcs(reinterpret_cast<const uint4*>(src + (h0 + i) * a.hd));
    int place;
    if (!place_of(a.q, a.r, (int)row, place)) return;
    uint2 turn[VN / 2];
#pragma unroll
    for (int k = 0; k < VN / 2; ++k) turn[k] = turns[e / 2 + k];
    Rotation<T> turned;
    turned.set(turn, a.positions ? a.positions[row] : place);
    T* dst = (T*)a.out_q + row * a.out_q_stride + e;
    while (true) {
#pragma unroll
        for (int i = 0; i < QB; ++i) {
            if (h0 + i >= h1) continue;
            float f[VN];
            Vec<T>::get(x[i], f);
            turned.apply(f);
            __stcs(reinterpret_cast<uint4*>(dst + (h0 + i) * a.hd), pack<T>(f));
        }
        h0 += QB;
        if (h0 >= h1) return;
#pragma unroll
        for (int i = 0; i < QB; ++i)
            if (h0 + i < h1) x[i] = __ldcs(reinterpret_cast<const uint4*>(src + (h0 + i) * a.hd));
    }
}

// (four CTAs of 256 threads to an SM: 64 registers: 8192 rows 44.3 us a call with three)
template <typename T, int NV>
__global__ void __launch_bounds__(MOST, NV <= 4 ? 2 : 1) kv8_append_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ Turns turns) {
    __shared__ uint2 turn_of[64];                      // (a thread's own from the parameters would be one word at a time)
    grid_dep_launch();
    if (threadIdx.x < a.hd / 2) turn_of[threadIdx.x] = turns.of[threadIdx.x];
    grid_dep_wait();
    kv8_check_offsets(a.q, a.r);
    __syncthreads();
    const int cta = blockIdx.x;
    if (cta < a.kv_ctas) append_kv<T, NV, 0>(a, turn_of, cta);
    else if (cta < 2 * a.kv_ctas) append_kv<T, NV, 1>(a, turn_of, cta - a.kv_ctas);
    else append_q<T>(a, turn_of, cta - 2 * a.kv_ctas);
}

// the fractions of a turn, kept with the thread for the model's next call
const Turns& turns_of(double theta, int hd) {
    static thread_local Turns turns;
    static thread_local double of_theta = 0.0;
    static thread_local int of_hd = 0;
    if (of_theta != theta || of_hd != hd) {
        // A frequency M 2^e times 1 / (2 pi), which is (I1 2^64 + I0) 2^-128 (cut off), in integers: all 64 bits are right.
        constexpr unsigned long long I1 = 0x28be60db9391054aull, I0 = 0x7f09d5f47d4d3770ull;
        for (int i = 0; i < hd / 2; ++i) {
            int e;
            const unsigned long long M = (unsigned long long)std::ldexp(std::frexp(std::pow(theta, -2.0 * i / hd), &e), 53);
            const unsigned __int128 P = (unsigned __int128)M * I1 + ((unsigned __int128)M * I0 >> 64);
            const unsigned long long of = 53 - e < 128 ? (unsigned long long)(P >> (53 - e)) : 0ull;
            turns.of[i] = make_uint2((unsigned)of, (unsigned)(of >> 32));
        }
        of_theta = theta;
        of_hd = hd;
    }
    return turns;
}

template <typename T> cudaError_t append_typed(const AppendArgs& a, const Turns& turns, int nv, dim3 grid, dim3 block, bool pdl, cudaStream_t s) {
    switch (nv) {
        case 1: return launch_ex(pdl, kv8_append_kernel<T, 1>, grid, block, 0, s, a, turns);
        case 2: return launch_ex(pdl, kv8_append_kernel<T, 2>, grid, block, 0, s, a, turns);
        case 4: return launch_ex(pdl, kv8_append_kernel<T, 4>, grid, block, 0, s, a, turns);
        case 8: return launch_ex(pdl, kv8_append_kernel<T, 8>, grid, block, 0, s, a, turns);
        default:                                       // fp32 rows, head_dim 128, 256 rows per page
            if constexpr (sizeof(T) == 4) return launch_ex(pdl, kv8_append_kernel<T, 16>, grid, block, 0, s, a, turns);
            return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8& c, const Kv8Seqs& q, const Kv8Rows& r, const Kv8Append& p, int layer, cudaStream_t s) {
    const Slots sl = kv8_slots(q, r);
    const bool wide = c.cfg.dtype == CB_F32;
    const int es = wide ? 4 : 2, P = 1 << q.shift;
    AppendArgs a{};
    a.q = q;
    a.r = r;
    a.src[0] = p.k;
    a.src[1] = p.v;
    a.kv_stride = p.kv_stride;
    a.in_q = p.q;
    a.out_q = p.out_q;
    a.q_stride = p.q_stride;
    a.out_q_stride = p.out_q_stride;
    a.positions = p.positions;
    a.codes = c.codes;
    a.scales = c.scales;
    a.per_seq = sl.per_seq;
    a.Hkv = c.cfg.n_kv_heads;
    a.Hq = c.cfg.n_heads;
    a.units = sl.total * a.Hkv;
    a.hd = c.cfg.head_dim;
    a.layer = layer;
    a.vpr_shift = log2_of(a.hd * es / 16);
    // a group holds the rows that a call may have in a block
    const int most_rows = r.start ? r.n_rows : r.each, in_block = 1 << log2_of(most_rows < P ? most_rows : P);
    const int vectors = in_block << a.vpr_shift, per_thread = wide ? 8 : 4;
    int tpb = vectors / per_thread;
    tpb = tpb < 32 ? 32 : tpb > MOST ? MOST : tpb;
    a.tpb_shift = log2_of(tpb);
    const int nv = vectors < tpb ? 1 : vectors >> a.tpb_shift;
    const int threads = tpb < 256 ? 256 : tpb, groups = threads >> a.tpb_shift;
    a.kv_ctas = (a.units + groups - 1) / groups;
    int64_t q_ctas = 0;
    if (p.q) {
        // as many heads per thread as leave every SM two thousand threads, up to eight
        const int64_t vectors_of_q = ((int64_t)r.n_rows * a.Hq) << a.vpr_shift;
        const int64_t heads = vectors_of_q / ((int64_t)c.num_sms * 2048);
        a.q_heads = heads < 1 ? 1 : heads > 8 ? 8 : (int)heads;
        a.q_chunks = (a.Hq + a.q_heads - 1) / a.q_heads;
        q_ctas = ((((int64_t)r.n_rows * a.q_chunks) << a.vpr_shift) + threads - 1) / threads;
    }
    const dim3 grid((unsigned)(2 * (int64_t)a.kv_ctas + q_ctas));
    const Turns& turns = turns_of(p.theta, a.hd);
    return wide ? append_typed<float>(a, turns, nv, grid, dim3(threads), c.pdl, s) : append_typed<bf16>(a, turns, nv, grid, dim3(threads), c.pdl, s);
}

}  // namespace cb
