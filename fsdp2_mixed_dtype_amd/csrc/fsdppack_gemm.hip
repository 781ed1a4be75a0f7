// fsdppack_gemm.hip -- the training operators' matrix products on the matrix
// cores: the gated block's forward pass (both projections, the activation and
// the product in one kernel), its input gradient, and weight gradients from
// dense or 8-bit activations.
//
// All three are out[j, i] = sum_r A(i, r) B(j, r), with i the contiguous
// index of the output:
//   gated:  A = rows of W_gate and W_up   B = x              r = in features
//   dx:     A = columns of W (both)       B = dgate, dup     r = hidden features
//   dw:     A = columns of x              B = columns of dy  r = tokens
// An operand whose reduction index is contiguous in memory lies in LDS as
// rows of 64 reduction elements; one whose reduction index is strided keeps
// its memory order there (64 rows of the tile's width) and is turned by the
// transposing LDS read.
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <algorithm>

#include "fsdppack_train_device.h"

namespace fsdppack {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int BK = 64;               // reduction elements per step

template <int DT>
__device__ __forceinline__ u32x4 load_chunk(const Mat &m, int64_t row, int64_t col, int64_t cols)
{
    // 8 elements [col, col + 8) of a row as bf16 (exact), zeros past `cols`
    u32x4 o = {0, 0, 0, 0};
    if constexpr (DT == FSDPPACK_BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(m.p) + row * m.ld + col;
        if (col + 8 <= cols) {
            const u32x4u w = *reinterpret_cast<const u32x4u *>(p);
            o = u32x4{w.x, w.y, w.z, w.w};
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i < cols) o[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
        }
    } else {
        float v[8];
        load8<DT>(static_cast<const char *>(m.p) + row * m.ld, m.scales + row * ((cols + kGroup - 1) / kGroup),
                  static_cast<int32_t>(col), static_cast<int32_t>(cols), v);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    }
    return o;
}

// Where a chunk of 8 elements lies in a tile's LDS image (in elements).
//  reduction contiguous: [T][64], 8 chunks a row, chunk c at c ^ (row & 7)
//  reduction strided:    [64][T], T / 8 chunks a row, chunk c at c ^ 4 (row & 3)
template <bool TR, int T>
__device__ __forceinline__ int lds_at(int row, int chunk)
{
    if constexpr (TR) return row * T + ((chunk ^ ((row & 3) << 2)) << 3);
    else return row * BK + ((chunk ^ (row & 7)) << 3);
}

// The 8 reduction elements [16 s + 8 h, ...) of tile row / column `at + lane % 32`, h = lane / 32.
template <bool TR, int T>
__device__ __forceinline__ bf16x8 fragment(uint16_t *tile, int at, int s)
{
    const int lane = threadIdx.x & 63;
    if constexpr (TR) {
        // a group of 16 lanes reads 4 rows of 16 columns (lane: row lane / 4,
        // 4 columns) and gets them turned: lane = column, 4 rows
        const int g = lane >> 4, l = lane & 15;
        const int row = 16 * s + 8 * (g >> 1) + (l >> 2), col = at + 16 * (g & 1) + 4 * (l & 3);
        typedef bf16x4 __attribute__((address_space(3))) * lds4;
        const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4)(tile + lds_at<true, T>(row, col >> 3) + (col & 7)));
        const bf16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4)(tile + lds_at<true, T>(row + 4, col >> 3) + (col & 7)));
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        const int row = at + (lane & 31);
        return *reinterpret_cast<bf16x8 *>(tile + lds_at<false, T>(row, 2 * s + (lane >> 5)));
    }
}

// One 128 x 128 output tile per block of four wavefronts, 64 x 64 each.
constexpr int T = 128, kBlockThreads = 256, kChunks = T * BK / 8 / kBlockThreads;

template <GemmKind KIND, int ADT>
__global__ void __launch_bounds__(kBlockThreads) gemm_kernel(GemmArgs g)
{
    constexpr bool ATR = KIND != kGemmGated, BTR = KIND == kGemmDw;
    __shared__ __align__(16) uint16_t sa[2][T * BK], sb[2][T * BK];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int64_t b = blockIdx.x;
    const int ti = static_cast<int>(b % g.tiles_i);
    b /= g.tiles_i;
    const int tj = static_cast<int>(b % g.tiles_j);
    b /= g.tiles_j;
    const int split = static_cast<int>(b % g.splits), z = static_cast<int>(b / g.splits);
    // the gated product's tile holds 64 rows of W_gate and the same 64 of W_up
    const int64_t i0 = int64_t{ti} * (KIND == kGemmGated ? T / 2 : T), j0 = int64_t{tj} * T;
    const int64_t steps1 = (g.R + BK - 1) / BK, steps = steps1 * g.segs;
    const int64_t s0 = steps * split / g.splits, s1 = steps * (split + 1) / g.splits;

    u32x4 ra[kChunks], rb[kChunks];
    auto fetch = [&](int64_t step) {
        const int seg = step >= steps1;
        const int64_t r0 = (step - seg * steps1) * BK;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int u = tid + c * kBlockThreads;
            if constexpr (ATR) {
                const int64_t row = r0 + u / (T / 8), col = i0 + u % (T / 8) * 8;
                ra[c] = row < g.R && col < g.I ? load_chunk<ADT>(g.a[seg], row, col, g.I) : u32x4{0, 0, 0, 0};
            } else {
                const int t = u / 8;
                const int64_t row = i0 + (t & (T / 2 - 1)), col = r0 + u % 8 * 8;
                ra[c] = row < g.I && col < g.R ? load_chunk<ADT>(g.a[t / (T / 2)], row, col, g.R) : u32x4{0, 0, 0, 0};
            }
            const Mat &mb = g.b[KIND == kGemmDw ? z : seg];
            if constexpr (BTR) {
                const int64_t row = r0 + u / (T / 8), col = j0 + u % (T / 8) * 8;
                rb[c] = row < g.R && col < g.J ? load_chunk<FSDPPACK_BF16>(mb, row, col, g.J) : u32x4{0, 0, 0, 0};
            } else {
                const int64_t row = j0 + u / 8, col = r0 + u % 8 * 8;
                rb[c] = row < g.J && col < g.R ? load_chunk<FSDPPACK_BF16>(mb, row, col, g.R) : u32x4{0, 0, 0, 0};
            }
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int u = tid + c * kBlockThreads;
            constexpr int ca = ATR ? T / 8 : 8, cb = BTR ? T / 8 : 8;
            *reinterpret_cast<u32x4 *>(&sa[buf][lds_at<ATR, T>(u / ca, u % ca)]) = ra[c];
            *reinterpret_cast<u32x4 *>(&sb[buf][lds_at<BTR, T>(u / cb, u % cb)]) = rb[c];
        }
    };

    const int wi = wave & 1, wj = wave >> 1;
    // the wavefront's two 32-row pieces of A: of the gated product one of each matrix
    const int ia[2] = {KIND == kGemmGated ? wi * 32 : wi * 64, KIND == kGemmGated ? T / 2 + wi * 32 : wi * 64 + 32};
    f32x16 acc[2][2] = {};
    if (s0 < s1) {
        fetch(s0);
        put(0);
    }
    for (int64_t s = s0; s < s1; ++s) {
        const int buf = static_cast<int>(s - s0) & 1;
        __syncthreads();
        if (s + 1 < s1) fetch(s + 1);
#pragma unroll
        for (int k = 0; k < BK / 16; ++k) {
            bf16x8 fa[2], fb[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                fa[n] = fragment<ATR, T>(sa[buf], ia[n], k);
                fb[n] = fragment<BTR, T>(sb[buf], wj * 64 + 32 * n, k);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    acc[n][m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[n], fb[m], acc[n][m], 0, 0, 0);
        }
        if (s + 1 < s1) put(buf ^ 1);
    }

    // lane: output row j = lane % 32, output columns 8 q + 4 (lane / 32) + 0..3 for q < 4
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int64_t j = j0 + wj * 64 + 32 * m + (lane & 31);
        if constexpr (KIND == kGemmGated) {
            const int64_t i = i0 + wi * 32 + 4 * (lane >> 5);
            float gv[16], uv[16], hv[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                gv[e] = acc[0][m][e];
                uv[e] = acc[1][m][e];
                float act, dact;
                activation(g.act, gv[e], act, dact);
                hv[e] = act * uv[e];
            }
            const bool row_ok = j < g.J;
            auto dense = [&](const Mat &o, const float *v) {
                if (!row_ok) return;
                uint16_t *p = static_cast<uint16_t *>(o.p) + j * o.ld;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int64_t col = i + 8 * (e >> 2) + (e & 3);
                    if (col < g.I) p[col] = static_cast<uint16_t>(to_bf16(v[e]));
                }
            };
            // lanes l and l + 32 hold one scale group (32 columns of a row) between them
            auto keep = [&](const Mat &o, float *v) {
                if (o.p == nullptr) return;
                if (o.dt == FSDPPACK_BF16) return dense(o, v);
                float top = 0.0f;
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, finite(v[e]) ? fabsf(v[e]) : 0.0f);
                top = fmaxf(top, __shfl_xor(top, 32));
                const int ex = o.dt == FSDPPACK_E4M3 ? scale_exponent<FSDPPACK_E4M3>(top) : scale_exponent<FSDPPACK_INT8>(top);
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (o.dt == FSDPPACK_E4M3) encode8<FSDPPACK_E4M3>(v + 8 * q, ex, w[2 * q], w[2 * q + 1]);
                    else encode8<FSDPPACK_INT8>(v + 8 * q, ex, w[2 * q], w[2 * q + 1]);
                }
                if (!row_ok) return;
                uint8_t *p = static_cast<uint8_t *>(o.p) + j * o.ld;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int64_t col = i + 8 * (e >> 2) + (e & 3);
                    if (col < g.I) p[col] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
                }
                if (lane < 32 && i < g.I) o.scales[j * ((g.I + kGroup - 1) / kGroup) + i / kGroup] = static_cast<uint8_t>(ex + 127);
            };
            dense(g.out[0], hv);
            keep(g.gate, gv);
            keep(g.up, uv);
        } else {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int64_t i = i0 + ia[n] + 4 * (lane >> 5);
                if (j >= g.J) continue;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int64_t col = i + 8 * (e >> 2) + (e & 3);
                    if (col >= g.I) continue;
                    if (g.splits > 1)
                        g.partial[((int64_t{z} * g.splits + split) * g.J + j) * g.I + col] = acc[n][m][e];
                    else if (g.out[z].dt == FSDPPACK_BF16)
                        static_cast<uint16_t *>(g.out[z].p)[j * g.out[z].ld + col] = static_cast<uint16_t>(to_bf16(acc[n][m][e]));
                    else
                        static_cast<float *>(g.out[z].p)[j * g.out[z].ld + col] = acc[n][m][e];
                }
            }
        }
    }
}

// The splits' partial sums, in a fixed order, rounded once.
__global__ void __launch_bounds__(256) join_kernel(GemmArgs g)
{
    const int64_t n = g.J * g.I;
    for (int64_t t = int64_t{blockIdx.x} * 256 + threadIdx.x; t < n * g.outs; t += int64_t{gridDim.x} * 256) {
        const int64_t z = t / n, e = t - z * n, j = e / g.I, i = e - j * g.I;
        float sum = 0.0f;
        for (int s = 0; s < g.splits; ++s) sum += g.partial[(z * g.splits + s) * n + e];
        const Mat &o = g.out[z];
        if (o.dt == FSDPPACK_BF16) static_cast<uint16_t *>(o.p)[j * o.ld + i] = static_cast<uint16_t>(to_bf16(sum));
        else static_cast<float *>(o.p)[j * o.ld + i] = sum;
    }
}

}  // namespace

#define LAUNCH(kernel, grid, block, ...)                                                                       \
    hipExtLaunchKernelGGL(kernel, grid, block, 0, static_cast<hipStream_t>(stream), static_cast<hipEvent_t>(e0), \
                          static_cast<hipEvent_t>(e1), 0, __VA_ARGS__)

int gemm_splits(GemmKind kind, int64_t I, int64_t J, int64_t R, int outs)
{
    (void)kind; (void)I; (void)J; (void)R; (void)outs;
    return 1;
}

int launch_gemm(GemmKind kind, GemmArgs g, void *stream, void *e0, void *end, int *launches)
{
    const int ti = kind == kGemmGated ? T / 2 : T;
    g.tiles_i = static_cast<int32_t>((g.I + ti - 1) / ti);
    g.tiles_j = static_cast<int32_t>((g.J + T - 1) / T);
    void *e1 = g.splits > 1 ? nullptr : end;
    const dim3 grid(static_cast<uint32_t>(int64_t{g.tiles_i} * g.tiles_j * g.splits * g.outs)), block(kBlockThreads);
    if (kind == kGemmGated) LAUNCH((gemm_kernel<kGemmGated, FSDPPACK_BF16>), grid, block, g);
    else if (kind == kGemmDx) LAUNCH((gemm_kernel<kGemmDx, FSDPPACK_BF16>), grid, block, g);
    else if (g.a[0].dt == FSDPPACK_BF16) LAUNCH((gemm_kernel<kGemmDw, FSDPPACK_BF16>), grid, block, g);
    else if (g.a[0].dt == FSDPPACK_E4M3) LAUNCH((gemm_kernel<kGemmDw, FSDPPACK_E4M3>), grid, block, g);
    else LAUNCH((gemm_kernel<kGemmDw, FSDPPACK_INT8>), grid, block, g);
    *launches = 1;
    if (g.splits > 1) {
        e0 = nullptr;
        e1 = end;
        const int64_t n = g.J * g.I * g.outs;
        LAUNCH(join_kernel, dim3(static_cast<uint32_t>(std::min<int64_t>((n + 255) / 256, 1 << 16))), dim3(256), g);
        ++*launches;
    }
    return static_cast<int>(hipGetLastError());
}

}  // namespace fsdppack
