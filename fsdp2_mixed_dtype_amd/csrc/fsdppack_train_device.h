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

// Elements [col, col + 8) of a row as fp32; those at or past `cols` are 0.
// `row`: the row's first element; `scales`: the row's scale bytes.
template <int DT>
__device__ __forceinline__ void load8(const void *row, const uint8_t *scales, int32_t col, int32_t cols, float *v)
{
    const int32_t n = cols - col;
    if constexpr (DT == FSDPPACK_BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(row) + col;
        if (n >= 8) {
            const u32x4u w = *reinterpret_cast<const u32x4u *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf16_lo(w[i]);
                v[2 * i + 1] = bf16_hi(w[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? bf16_lo(p[i]) : 0.0f;
        }
    } else if constexpr (DT == FSDPPACK_FP32) {
        const float *p = static_cast<const float *>(row) + col;
        if (n >= 8) {
            const f32x4u a = *reinterpret_cast<const f32x4u *>(p), b = *reinterpret_cast<const f32x4u *>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
        }
    } else {
        const uint8_t *p = static_cast<const uint8_t *>(row) + col;
        uint32_t lo = 0, hi = 0;
        float s = 0.0f;
        if (n >= 8) {
            const u32x2u w = *reinterpret_cast<const u32x2u *>(p);
            lo = w.x;
            hi = w.y;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) (i < 4 ? lo : hi) |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
        }
        if (n > 0) s = scale_of(scales[col / kGroup]);
        decode8<DT>(lo, hi, s, v);
    }
}

// load8 with the dtype known at run time (the same for the whole launch).
__device__ __forceinline__ void load8_dense(const void *row, int32_t dt, int32_t col, int32_t cols, float *v)
{
    if (dt == FSDPPACK_BF16) load8<FSDPPACK_BF16>(row, nullptr, col, cols, v);
    else load8<FSDPPACK_FP32>(row, nullptr, col, cols, v);
}

// Eight values rounded to the row's dtype; only columns below `cols` are written.
__device__ __forceinline__ void store8(void *row, int32_t dt, int32_t col, int32_t cols, const float *v)
{
    const int32_t n = cols - col;
    if (dt == FSDPPACK_BF16) {
        uint16_t *p = static_cast<uint16_t *>(row) + col;
        if (n >= 8) {
            u32x4u w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<u32x4u *>(p) = w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) p[i] = static_cast<uint16_t>(to_bf16(v[i]));
        }
    } else {
        float *p = static_cast<float *>(row) + col;
        if (n >= 8) {
            *reinterpret_cast<f32x4u *>(p) = f32x4u{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4u *>(p + 4) = f32x4u{v[4], v[5], v[6], v[7]};
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

// Eight values of a group with scale exponent e, as codes.  The product with
// 2^-e is exact (or far below the smallest step), so this rounds once, to
// nearest even.  Values that would round past the largest fp32 when read
// back (only within half a step of it) keep the largest code below instead.
template <int DT>
__device__ __forceinline__ void encode8(const float *v, int e, uint32_t &lo, uint32_t &hi)
{
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    const float most = DT == FSDPPACK_E4M3 ? 0x1.Ep127f : 0x1.F8p127f;
    uint32_t w[2] = {0, 0};
    if constexpr (DT == FSDPPACK_E4M3) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float s[4];
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = v[4 * h + i];
                bad |= finite(x) ? 0u : 0x7fu << (8 * i);
                s[i] = fminf(fmaxf(x, -most), most) * inv;
            }
            int c = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false);
            c = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], c, true);
            w[h] = static_cast<uint32_t>(c) | bad;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = v[i];
            const int c = finite(x) ? static_cast<int>(__builtin_rintf(fminf(fmaxf(x, -most), most) * inv)) : -128;
            w[i >> 2] |= (static_cast<uint32_t>(c) & 0xffu) << (8 * (i & 3));
        }
    }
    lo = w[0];
    hi = w[1];
}

__device__ __forceinline__ float top_of8(const float *v)
{
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = fmaxf(t, finite(v[i]) ? fabsf(v[i]) : 0.0f);
    return t;
}

// Put columns [col, col + 8) of a row away.  Four neighbouring lanes hold one
// group of 32 columns (lane 4g holds its first eight); all four call this,
// with zeros past `cols`.
template <int DT>
__device__ __forceinline__ void save8_as(uint8_t *row, uint8_t *scales, int32_t col, int32_t cols, const float *v)
{
    float top = top_of8(v);
    top = fmaxf(top, dpp<kDppXor1>(top));
    top = fmaxf(top, dpp<kDppXor2>(top));
    const int e = scale_exponent<DT>(top);
    uint32_t lo, hi;
    encode8<DT>(v, e, lo, hi);
    const int32_t n = cols - col;
    if (n >= 8) {
        *reinterpret_cast<u32x2u *>(row + col) = u32x2u{lo, hi};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) row[col + i] = static_cast<uint8_t>((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
    if (n > 0 && (col & (kGroup - 1)) == 0) scales[col / kGroup] = static_cast<uint8_t>(e + 127);
}

__device__ __forceinline__ void save8(const Mat &q, int64_t row, int32_t col, int32_t cols, const float *v)
{
    uint8_t *p = static_cast<uint8_t *>(q.p) + row * q.ld;
    uint8_t *s = q.scales + row * ((cols + kGroup - 1) / kGroup);
    if (q.dt == FSDPPACK_E4M3) save8_as<FSDPPACK_E4M3>(p, s, col, cols, v);
    else save8_as<FSDPPACK_INT8>(p, s, col, cols, v);
}

__device__ __forceinline__ const void *row_of(const Mat &m, int64_t row)
{
    const int lg = m.dt == FSDPPACK_FP32 ? 2 : m.dt == FSDPPACK_BF16 ? 1 : 0;
    return static_cast<const char *>(m.p) + ((row * m.ld) << lg);
}
__device__ __forceinline__ void *row_of_out(const Mat &m, int64_t row) { return const_cast<void *>(row_of(m, row)); }

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
