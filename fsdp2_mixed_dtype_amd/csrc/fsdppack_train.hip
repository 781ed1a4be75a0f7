// fsdppack_train.hip -- the training operators that are bound by memory: the
// norm's two passes, the 8-bit activation checkpoints, and the elementwise
// part of the gated block's backward pass.
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <algorithm>

#include "fsdppack_train_device.h"

namespace fsdppack {
namespace {

constexpr int kThreads = 256;

// Sum over the block's four wavefronts.
__device__ __forceinline__ float block_sum(float v, float *s)
{
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// One group of eight columns per thread and step; a row of ceil(cols / 32)
// groups of four such threads, so that a checkpoint's scale group never
// crosses a row's end.
template <int XT>
__global__ void __launch_bounds__(kThreads) save_kernel(Mat x, Mat q, int64_t rows, int32_t cols)
{
    const int32_t units = (cols + kGroup - 1) / kGroup * 4;
    for (int64_t t = int64_t{blockIdx.x} * kThreads + threadIdx.x; t < rows * units; t += int64_t{gridDim.x} * kThreads) {
        const int64_t r = t / units;
        const int32_t col = static_cast<int32_t>(t - r * units) * 8;
        float v[8];
        load8<XT>(row_of(x, r), nullptr, col, cols, v);
        save8(q, r, col, cols, v);
    }
}

template <int QT>
__global__ void __launch_bounds__(kThreads) load_kernel(Mat q, Mat out, int64_t rows, int32_t cols)
{
    const int32_t units = (cols + 7) / 8;
    for (int64_t t = int64_t{blockIdx.x} * kThreads + threadIdx.x; t < rows * units; t += int64_t{gridDim.x} * kThreads) {
        const int64_t r = t / units;
        const int32_t col = static_cast<int32_t>(t - r * units) * 8;
        float v[8];
        load8<QT>(row_of(q, r), q.scales + r * ((cols + kGroup - 1) / kGroup), col, cols, v);
        store8(row_of_out(out, r), out.dt, col, cols, v);
    }
}

__device__ __forceinline__ void load_weight(const void *w, int32_t dt, int32_t col, int32_t cols, float fallback, float *v)
{
    if (w == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fallback;
    } else {
        load8_dense(w, dt, col, cols, v);
    }
}

// One block per row; the row is read once for the mean, once for the spread
// and once for the result (all but the first from cache).
template <int XT>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(NormArgs a)
{
    __shared__ float s[4];
    const int32_t cols = a.cols;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const void *x = row_of(a.x, r);
        float v[8];
        float mean = 0.0f;
        if (!a.rms) {
            float sum = 0.0f;
            for (int32_t c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
                load8<XT>(x, nullptr, c, cols, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += v[i];
            }
            mean = block_sum(sum, s) / static_cast<float>(cols);
        }
        float sq = 0.0f;
        for (int32_t c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
            load8<XT>(x, nullptr, c, cols, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = c + i < cols ? v[i] - mean : 0.0f;
                sq += d * d;
            }
        }
        const float rstd = 1.0f / sqrtf(block_sum(sq, s) / static_cast<float>(cols) + a.eps);
        if (threadIdx.x == 0) {
            a.stats[2 * r] = mean;
            a.stats[2 * r + 1] = rstd;
        }
        // whole groups of four threads, so that a checkpoint's scale is found among them
        for (int32_t c = threadIdx.x * 8; c < (cols + kGroup - 1) / kGroup * kGroup; c += kThreads * 8) {
            float w[8], b[8], y[8];
            load8<XT>(x, nullptr, c, cols, v);
            load_weight(a.weight, a.wdt, c, cols, 1.0f, w);
            load_weight(a.bias, a.wdt, c, cols, 0.0f, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = c + i < cols ? (v[i] - mean) * rstd * w[i] + b[i] : 0.0f;
            store8(row_of_out(a.out, r), a.out.dt, c, cols, y);
            if (a.x_ckpt.p) save8(a.x_ckpt, r, c, cols, v);
            if (a.out_ckpt.p) save8(a.out_ckpt, r, c, cols, y);
        }
    }
}

// dx of a row: rstd * (w dy - c1 - xh c2), c1 and c2 the means of w dy and
// w dy xh over the row (c1 = 0 for the RMS norm).
template <int XT>
__global__ void __launch_bounds__(kThreads) norm_dx_kernel(NormBackArgs a)
{
    __shared__ float s[4];
    const int32_t cols = a.cols;
    const int32_t groups = (cols + kGroup - 1) / kGroup;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const void *x = row_of(a.x, r), *dy = row_of(a.dout, r);
        const uint8_t *sc = a.x.scales + r * groups;
        const float mean = a.stats[2 * r], rstd = a.stats[2 * r + 1];
        float v[8], d[8], w[8];
        float s1 = 0.0f, s2 = 0.0f;
        for (int32_t c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
            load8<XT>(x, sc, c, cols, v);
            load8_dense(dy, a.dout.dt, c, cols, d);
            load_weight(a.weight, a.wdt, c, cols, 1.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < cols) {
                    const float t = d[i] * w[i];
                    s1 += t;
                    s2 += t * ((v[i] - mean) * rstd);
                }
        }
        const float c2 = block_sum(s2, s) / static_cast<float>(cols);
        const float c1 = a.rms ? 0.0f : block_sum(s1, s) / static_cast<float>(cols);
        for (int32_t c = threadIdx.x * 8; c < cols; c += kThreads * 8) {
            load8<XT>(x, sc, c, cols, v);
            load8_dense(dy, a.dout.dt, c, cols, d);
            load_weight(a.weight, a.wdt, c, cols, 1.0f, w);
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = rstd * (d[i] * w[i] - c1 - (v[i] - mean) * rstd * c2);
            store8(row_of_out(a.dx, r), a.dx.dt, c, cols, o);
        }
    }
}

// Partial sums over a part of the rows of dy * xh and dy; thread = 8 columns.
template <int XT>
__global__ void __launch_bounds__(64) norm_dw_kernel(NormBackArgs a)
{
    const int32_t cols = a.cols, c = (blockIdx.x * 64 + threadIdx.x) * 8;
    if (c >= cols) return;
    const int32_t groups = (cols + kGroup - 1) / kGroup;
    float dw[8] = {}, db[8] = {};
    for (int64_t r = blockIdx.y; r < a.rows; r += a.parts) {
        float v[8], d[8];
        load8<XT>(row_of(a.x, r), a.x.scales + r * groups, c, cols, v);
        load8_dense(row_of(a.dout, r), a.dout.dt, c, cols, d);
        const float mean = a.stats[2 * r], rstd = a.stats[2 * r + 1];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dw[i] += d[i] * ((v[i] - mean) * rstd);
            db[i] += d[i];
        }
    }
    float *p = a.partial + int64_t{blockIdx.y} * 2 * cols;
    store8(p, FSDPPACK_FP32, c, cols, dw);
    store8(p + cols, FSDPPACK_FP32, c, cols, db);
}

// The parts' sums, in a fixed order: results do not depend on timing.
__global__ void __launch_bounds__(kThreads) norm_join_kernel(NormBackArgs a)
{
    const int64_t i = int64_t{blockIdx.x} * kThreads + threadIdx.x;
    if (i >= int64_t{2} * a.cols) return;
    void *dst = i < a.cols ? a.dweight : a.dbias;
    if (dst == nullptr) return;
    float sum = 0.0f;
    for (int32_t p = 0; p < a.parts; ++p) sum += a.partial[int64_t{p} * 2 * a.cols + i];
    const int64_t c = i < a.cols ? i : i - a.cols;
    if (a.gdt == FSDPPACK_BF16) static_cast<uint16_t *>(dst)[c] = static_cast<uint16_t>(to_bf16(sum));
    else static_cast<float *>(dst)[c] = sum;
}

// dg = dh u a'(g), du = dh a(g), and h = a(g) u where it is wanted again.
// They are rounded to bf16, the type in which the matrix products that follow
// read them.
__device__ __forceinline__ void load8_any(const Mat &m, int64_t r, int32_t c, int32_t cols, float *v)
{
    const uint8_t *sc = m.scales + r * ((cols + kGroup - 1) / kGroup);
    if (m.dt == FSDPPACK_BF16) load8<FSDPPACK_BF16>(row_of(m, r), nullptr, c, cols, v);
    else if (m.dt == FSDPPACK_E4M3) load8<FSDPPACK_E4M3>(row_of(m, r), sc, c, cols, v);
    else load8<FSDPPACK_INT8>(row_of(m, r), sc, c, cols, v);
}

__global__ void __launch_bounds__(kThreads) gate_backward_kernel(GateArgs a)
{
    const int32_t cols = a.cols, units = (cols + 7) / 8;
    for (int64_t t = int64_t{blockIdx.x} * kThreads + threadIdx.x; t < a.rows * units; t += int64_t{gridDim.x} * kThreads) {
        const int64_t r = t / units;
        const int32_t c = static_cast<int32_t>(t - r * units) * 8;
        float d[8], g[8], u[8], h[8];
        load8<FSDPPACK_BF16>(row_of(a.dout, r), nullptr, c, cols, d);
        load8_any(a.gate, r, c, cols, g);
        load8_any(a.up, r, c, cols, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float act, dact;
            activation(a.act, g[i], act, dact);
            h[i] = act * u[i];
            g[i] = d[i] * u[i] * dact;
            u[i] = d[i] * act;
        }
        store8(a.dgate + r * a.ldw, FSDPPACK_BF16, c, cols, g);
        store8(a.dup + r * a.ldw, FSDPPACK_BF16, c, cols, u);
        if (a.out.p) store8(row_of_out(a.out, r), FSDPPACK_BF16, c, cols, h);
    }
}

int blocks_for(int64_t work, int64_t per_block)
{
    return static_cast<int>(std::min<int64_t>((work + per_block - 1) / per_block, 1 << 16));
}

}  // namespace

#define LAUNCH(kernel, grid, block, ...)                                                                       \
    hipExtLaunchKernelGGL(kernel, grid, block, 0, static_cast<hipStream_t>(stream), static_cast<hipEvent_t>(e0), \
                          static_cast<hipEvent_t>(e1), 0, __VA_ARGS__)

int launch_checkpoint(const Mat &x, const Mat &q, int64_t rows, int64_t cols, bool save, void *stream, void *e0, void *e1)
{
    const int32_t c = static_cast<int32_t>(cols);
    const dim3 grid(blocks_for(rows * ((cols + kGroup - 1) / kGroup * 4), kThreads)), block(kThreads);
    if (save && x.dt == FSDPPACK_BF16) LAUNCH(save_kernel<FSDPPACK_BF16>, grid, block, x, q, rows, c);
    else if (save) LAUNCH(save_kernel<FSDPPACK_FP32>, grid, block, x, q, rows, c);
    else if (q.dt == FSDPPACK_E4M3) LAUNCH(load_kernel<FSDPPACK_E4M3>, grid, block, q, x, rows, c);
    else LAUNCH(load_kernel<FSDPPACK_INT8>, grid, block, q, x, rows, c);
    return static_cast<int>(hipGetLastError());
}

int launch_norm_forward(const NormArgs &a, void *stream, void *e0, void *e1)
{
    const dim3 grid(blocks_for(a.rows, 1)), block(kThreads);
    if (a.x.dt == FSDPPACK_BF16) LAUNCH(norm_forward_kernel<FSDPPACK_BF16>, grid, block, a);
    else LAUNCH(norm_forward_kernel<FSDPPACK_FP32>, grid, block, a);
    return static_cast<int>(hipGetLastError());
}

int norm_backward_parts(int64_t rows, int64_t cols)
{
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(rows, 512)));
}

int launch_norm_backward(const NormBackArgs &a, void *stream, void *e0, void *end, int *launches)
{
    const bool sums = a.dweight != nullptr || a.dbias != nullptr;
    void *e1 = sums ? nullptr : end;
    *launches = 0;
    if (a.rows > 0) {
        const dim3 grid(blocks_for(a.rows, 1)), block(kThreads);
        if (a.x.dt == FSDPPACK_BF16) LAUNCH(norm_dx_kernel<FSDPPACK_BF16>, grid, block, a);
        else if (a.x.dt == FSDPPACK_FP32) LAUNCH(norm_dx_kernel<FSDPPACK_FP32>, grid, block, a);
        else if (a.x.dt == FSDPPACK_E4M3) LAUNCH(norm_dx_kernel<FSDPPACK_E4M3>, grid, block, a);
        else LAUNCH(norm_dx_kernel<FSDPPACK_INT8>, grid, block, a);
        ++*launches;
        e0 = nullptr;
    }
    if (sums) {
        const dim3 grid((a.cols + 511) / 512, a.parts), block(64);
        if (a.x.dt == FSDPPACK_BF16) LAUNCH(norm_dw_kernel<FSDPPACK_BF16>, grid, block, a);
        else if (a.x.dt == FSDPPACK_FP32) LAUNCH(norm_dw_kernel<FSDPPACK_FP32>, grid, block, a);
        else if (a.x.dt == FSDPPACK_E4M3) LAUNCH(norm_dw_kernel<FSDPPACK_E4M3>, grid, block, a);
        else LAUNCH(norm_dw_kernel<FSDPPACK_INT8>, grid, block, a);
        e0 = nullptr;
        e1 = end;
        LAUNCH(norm_join_kernel, dim3((2 * a.cols + kThreads - 1) / kThreads), dim3(kThreads), a);
        *launches += 2;
    }
    return static_cast<int>(hipGetLastError());
}

int launch_gate_backward(const GateArgs &a, void *stream, void *e0, void *e1)
{
    const dim3 grid(blocks_for(a.rows * ((a.cols + 7) / 8), kThreads)), block(kThreads);
    LAUNCH(gate_backward_kernel, grid, block, a);
    return static_cast<int>(hipGetLastError());
}

}  // namespace fsdppack
