// fsdppack_train_device.h -- device helpers of the training operators:
// 8-element loads and stores of every dtype, the 8-bit checkpoint's encoding,
// wavefront sums.
#pragma once

#include <hip/hip_runtime.h>

#include "fsdppack_train.h"

namespace fsdppack {

typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));   // any element-aligned address:
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));   // global loads and stores need no more
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// fp32 -> bf16, round to nearest even (a NaN stays a quiet NaN).
__device__ __forceinline__ uint32_t to_bf16(float f)
{
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float scale_of(uint8_t s) { return __uint_as_float(static_cast<uint32_t>(s) << 23); }

// One 8-bit code's value before the scale.  INT8's -128 stands for "not finite".
template <int DT>
__device__ __forceinline__ void decode8(uint32_t lo, uint32_t hi, float scale, float *v)
{
    if constexpr (DT == FSDPPACK_E4M3) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w = h ? hi : lo;
            const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
            v[4 * h] = a.x * scale;
            v[4 * h + 1] = a.y * scale;
            v[4 * h + 2] = b.x * scale;
            v[4 * h + 3] = b.y * scale;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int8_t q = static_cast<int8_t>((i < 4 ? lo : hi) >> (8 * (i & 3)));
            v[i] = q == -128 ? __builtin_nanf("") : static_cast<float>(q) * scale;
        }
    }
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Eight elements as they lie in memory: what a load in flight holds.
template <int DT>
struct Raw8 {
    static constexpr int kSize = DT == FSDPPACK_FP32 ? 4 : DT == FSDPPACK_BF16 ? 2 : 1;
    uint32_t w[2 * kSize];
    uint32_t scale;                   // 8-bit formats
};

// Elements [col, col + 8) of a row; those at or past `cols` are 0.
// `row`: the row's first element; `scales`: the row's scale bytes.
template <int DT>
__device__ __forceinline__ Raw8<DT> read8(const void *row, const uint8_t *scales, int32_t col, int32_t cols)
{
    Raw8<DT> r = {};
    const int32_t n = cols - col;
    if constexpr (DT == FSDPPACK_BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(row) + col;
        if (n >= 8) {
            const u32x4u w = *reinterpret_cast<const u32x4u *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) r.w[i] = w[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) r.w[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
        }
    } else if constexpr (DT == FSDPPACK_FP32) {
        const uint32_t *p = static_cast<const uint32_t *>(row) + col;
        if (n >= 8) {
            const u32x4u a = *reinterpret_cast<const u32x4u *>(p), b = *reinterpret_cast<const u32x4u *>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r.w[i] = a[i];
                r.w[4 + i] = b[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) r.w[i] = i < n ? p[i] : 0;
        }
    } else {
        const uint8_t *p = static_cast<const uint8_t *>(row) + col;
        if (n >= 8) {
            const u32x2u w = *reinterpret_cast<const u32x2u *>(p);
            r.w[0] = w.x;
            r.w[1] = w.y;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) r.w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
        }
        r.scale = n > 0 ? scales[col / kGroup] : 0;
    }
    return r;
}

// Their values.
template <int DT>
__device__ __forceinline__ void value8(const Raw8<DT> &r, float *v)
{
    if constexpr (DT == FSDPPACK_BF16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (i & 1) ? bf16_hi(r.w[i >> 1]) : bf16_lo(r.w[i >> 1]);
    } else if constexpr (DT == FSDPPACK_FP32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
    } else {
        decode8<DT>(r.w[0], r.w[1], __uint_as_float(r.scale << 23), v);
    }
}

template <int DT>
__device__ __forceinline__ void load8(const void *row, const uint8_t *scales, int32_t col, int32_t cols, float *v)
{
    value8<DT>(read8<DT>(row, scales, col, cols), v);
}

// A store of 16 or 8 bytes at byte `at` from `base`, which is the same for the
// whole wavefront.  STREAM: past the caches (device scope, non-temporal), for
// results that L2 (8 x 4 MB) does not keep anyway, where lines left dirty are
// written back later and in a worse order: 8192 x 4096 norm 26.0 us against
// 29.4, checkpoint saved 17.4 against 20.2, read back 15.2 against 21.0.
constexpr int kStreamPolicy = 18;     // sc1 nt
template <typename V>
__device__ __forceinline__ void store_at(void *base, int32_t at, V v, bool stream)
{
    if (stream && (reinterpret_cast<uintptr_t>(base) & 15) == 0) {
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(base, 0, 0x7fffffff, 0x00020000);
        if constexpr (sizeof(V) == 16) __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, at, 0, kStreamPolicy);
        else __builtin_amdgcn_raw_buffer_store_b64(v, rsrc, at, 0, kStreamPolicy);
    } else if constexpr (sizeof(V) == 16) {
        *reinterpret_cast<u32x4u *>(static_cast<char *>(base) + at) = u32x4u{v.x, v.y, v.z, v.w};
    } else {
        *reinterpret_cast<u32x2u *>(static_cast<char *>(base) + at) = u32x2u{v.x, v.y};
    }
}

// load8 with the dtype known at run time (the same for the whole launch).
__device__ __forceinline__ void load8_dense(const void *row, int32_t dt, int32_t col, int32_t cols, float *v)
{
    if (dt == FSDPPACK_BF16) load8<FSDPPACK_BF16>(row, nullptr, col, cols, v);
    else load8<FSDPPACK_FP32>(row, nullptr, col, cols, v);
}

// Eight values rounded to the row's dtype; only columns below `cols` are written.
__device__ __forceinline__ void store8(void *row, int32_t dt, int32_t col, int32_t cols, const float *v, bool stream = false)
{
    const int32_t n = cols - col;
    if (dt == FSDPPACK_BF16) {
        uint16_t *p = static_cast<uint16_t *>(row) + col;
        if (n >= 8) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
            store_at(row, col * 2, w, stream);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = static_cast<uint16_t>(to_bf16(v[i]));
        }
    } else {
        float *p = static_cast<float *>(row) + col;
        if (n >= 8) {
            u32x4 w[2];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i >> 2][i & 3] = __float_as_uint(v[i]);
            store_at(row, col * 4, w[0], stream);
            store_at(row, col * 4 + 16, w[1], stream);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = v[i];
        }
    }
}

// The value of the lane that a DPP control names (every lane active).
template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

// Sum over the 64 lanes, the same bits in each (every step adds the two
// halves of a pair, which commutes).
__device__ __forceinline__ float wave_sum(float v)
{
    v += dpp<kDppXor1>(v);
    v += dpp<kDppXor2>(v);
    v += dpp<kDppHalfMirror>(v);
    v += dpp<kDppMirror>(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }

// The scale exponent of a group whose largest finite magnitude is `top`: the
// smallest e >= kMinExponent with top * 2^-e within the format's largest
// value, 1.75 * 2^8 (e4m3) or 127 = 1.984375 * 2^6 (int8).  Read off top's
// bits: exponent minus 8 (6), one more when the mantissa is past that of the limit.
template <int DT>
__device__ __forceinline__ int scale_exponent(float top)
{
    const uint32_t b = __float_as_uint(top);
    const int k = static_cast<int>(b >> 23) - 127;
    const int e = DT == FSDPPACK_E4M3 ? k - 8 + ((b & 0x7fffffu) > 0x600000u) : k - 6 + ((b & 0x7fffffu) > 0x7e0000u);
    return e < kMinExponent ? kMinExponent : e;
}

// The largest magnitude of eight values as fp32 bits: at or past kLastPlain
// when one of them is not finite (or so large that its code could round past
// the largest fp32 when read back).
constexpr uint32_t kLastPlain = 0x7f700000u;     // 1.875 * 2^127
__device__ __forceinline__ uint32_t top_bits8(const float *v)
{
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
        t = t > u ? t : u;
    }
    return t;
}

// The same over the finite ones only.
__device__ __forceinline__ float finite_top8(const float *v)
{
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = fmaxf(t, finite(v[i]) ? fabsf(v[i]) : 0.0f);
    return t;
}

// Eight values of a group with scale exponent e, as codes.  x * 2^-e is exact
// (or far below the smallest step), so this rounds once, to nearest even.
// PLAIN: every value is finite and below kLastPlain; otherwise NaN and
// infinity become the NaN code, and values that would round past the largest
// fp32 when read back (only within half a step of it) keep the code below.
template <int DT, bool PLAIN>
__device__ __forceinline__ void encode8(const float *x, int e, uint32_t &lo, uint32_t &hi)
{
    const float most = DT == FSDPPACK_E4M3 ? 0x1.Ep127f : 0x1.F8p127f;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = PLAIN ? x[i] : fminf(fmaxf(x[i], -most), most);
    uint32_t w[2];
    if constexpr (DT == FSDPPACK_E4M3) {
        // the hardware's scaled conversion: two values divided by 2^e and rounded
        typedef short s16x2 __attribute__((ext_vector_type(2)));
        const float scale = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s16x2 c = {0, 0};
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, v[4 * h], v[4 * h + 1], scale, false);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, v[4 * h + 2], v[4 * h + 3], scale, true);
            w[h] = __builtin_bit_cast(uint32_t, c);
        }
    } else {
        // x * 2^-e + 1.5 * 2^23 in one rounding: the integer is in the low byte
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(fmaf(v[i], inv, 0x1.8p23f));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t a = __builtin_amdgcn_perm(u[4 * h + 1], u[4 * h], 0x0c0c0400u), b = __builtin_amdgcn_perm(u[4 * h + 3], u[4 * h + 2], 0x0c0c0400u);
            w[h] = a | b << 16;
        }
    }
    if constexpr (!PLAIN) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!finite(x[i])) {
                const uint32_t at = 8 * (i & 3), code = DT == FSDPPACK_E4M3 ? 0x7fu : 0x80u;
                w[i >> 2] = (w[i >> 2] & ~(0xffu << at)) | code << at;
            }
    }
    lo = w[0];
    hi = w[1];
}

// Put columns [col, col + 8) of a row away.  Four neighbouring lanes hold one
// group of 32 columns (lane 4g holds its first eight); all four call this,
// with zeros past `cols`.
template <int DT>
__device__ __forceinline__ void save8_as(uint8_t *row, uint8_t *scales, int32_t col, int32_t cols, const float *v, bool stream)
{
    uint32_t bits = top_bits8(v);
    const uint32_t b1 = __float_as_uint(dpp<kDppXor1>(__uint_as_float(bits)));
    bits = bits > b1 ? bits : b1;
    const uint32_t b2 = __float_as_uint(dpp<kDppXor2>(__uint_as_float(bits)));
    bits = bits > b2 ? bits : b2;
    uint32_t lo, hi;
    int e;
    if (bits < kLastPlain) {
        e = scale_exponent<DT>(__uint_as_float(bits));
        encode8<DT, true>(v, e, lo, hi);
    } else {                              // all four lanes of the group
        float top = finite_top8(v);
        top = fmaxf(top, dpp<kDppXor1>(top));
        top = fmaxf(top, dpp<kDppXor2>(top));
        e = scale_exponent<DT>(top);
        encode8<DT, false>(v, e, lo, hi);
    }
    const int32_t n = cols - col;
    if (n >= 8) {
        store_at(row, col, u32x2{lo, hi}, stream);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) row[col + i] = static_cast<uint8_t>((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
    if (n > 0 && (col & (kGroup - 1)) == 0) scales[col / kGroup] = static_cast<uint8_t>(e + 127);
}

__device__ __forceinline__ void save8(const Mat &q, int64_t row, int32_t col, int32_t cols, const float *v, bool stream = false)
{
    uint8_t *p = static_cast<uint8_t *>(q.p) + row * q.ld;
    uint8_t *s = q.scales + row * ((cols + kGroup - 1) / kGroup);
    if (q.dt == FSDPPACK_E4M3) save8_as<FSDPPACK_E4M3>(p, s, col, cols, v, stream);
    else save8_as<FSDPPACK_INT8>(p, s, col, cols, v, stream);
}

__device__ __forceinline__ const void *row_of(const Mat &m, int64_t row)
{
    const int lg = m.dt == FSDPPACK_FP32 ? 2 : m.dt == FSDPPACK_BF16 ? 1 : 0;
    return static_cast<const char *>(m.p) + ((row * m.ld) << lg);
}
__device__ __forceinline__ void *row_of_out(const Mat &m, int64_t row) { return const_cast<void *>(row_of(m, row)); }

// The activation at g (see below).
__device__ __forceinline__ float activation_alone(int act, float g)
{
    if (act == FSDPPACK_SILU) return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g));
    const float g2 = fminf(g * g, 1e8f);
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-2.0f * 0.7978845608028654f * g * (1.0f + 0.044715f * g2)));
}

// The activation and its derivative at g.
//  SILU:      a = g s, a' = s (1 + g (1 - s)), s = 1 / (1 + e^-g)
//  GELU_TANH: a = g p, a' = p + 2 g p (1 - p) k (1 + 3 c g^2), p = 1 / (1 + e^-2v),
//             v = k (g + c g^3), the tanh form ((1 + tanh v) / 2 = p)
// e^-z overflows to infinity for z < -88: its reciprocal is then 0, the limit.
// The hardware's reciprocal is within one unit in fp32's last place.
__device__ __forceinline__ void activation(int act, float g, float &a, float &da)
{
    if (act == FSDPPACK_SILU) {
        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
        a = g * s;
        da = s * (1.0f + g * (1.0f - s));
    } else {
        const float k = 0.7978845608028654f, c = 0.044715f;
        const float g2 = fminf(g * g, 1e8f);     // past |g| = 1e4 p is 0 or 1 and the terms stay finite
        const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-2.0f * k * g * (1.0f + c * g2)));
        a = g * p;
        da = p + a * (1.0f - p) * (2.0f * k * (1.0f + 3.0f * c * g2));
    }
}

}  // namespace fsdppack
