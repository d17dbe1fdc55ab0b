// norm.cu -- layer norm over the rows of an activation, forward and backward (include/nvfp4.h has
// the formulas).  Statistics and sums are fp32.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cmath>
#include <cstdint>

#include "device_common.cuh"
#include "host_common.h"

namespace nvfp4 {
namespace {

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ float round_to(float v, const float*) { return v; }
__device__ __forceinline__ float round_to(float v, const __nv_bfloat16*) {
    return __bfloat162float(__float2bfloat16_rn(v));
}

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < kThreads / 32; ++i) s += red[i];
    return s;
}

struct FwdParams {
    const void *x, *residual, *weight, *bias;
    void *y, *h;
    float *mean, *rstd;
    int64_t rows, cols, ldx, ldr, ldy, ldh;
    float eps;
};

template <typename X, typename Y, typename W>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(FwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float red[kThreads / 32];
    const W* w = static_cast<const W*>(p.weight);
    const W* b = static_cast<const W*>(p.bias);
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const X* x = static_cast<const X*>(p.x) + r * p.ldx;
        const X* res = p.residual ? static_cast<const X*>(p.residual) + r * p.ldr : nullptr;
        X* h = p.h ? static_cast<X*>(p.h) + r * p.ldh : nullptr;
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
            float v = load1(x + c);
            if (res) {
                v = round_to(v + load1(res + c), x);
                store1(h + c, v);
            }
            s += v;
        }
        const X* src = res ? h : x;
        const float mean = block_sum(s, red) / (float)p.cols;
        s = 0.0f;
        for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
            const float d = load1(src + c) - mean;
            s += d * d;
        }
        const float rstd = 1.0f / sqrtf(block_sum(s, red) / (float)p.cols + p.eps);
        Y* y = static_cast<Y*>(p.y) + r * p.ldy;
        for (int64_t c = threadIdx.x; c < p.cols; c += kThreads)
            store1(y + c, (load1(src + c) - mean) * rstd * load1(w + c) + (b ? load1(b + c) : 0.0f));
        if (threadIdx.x == 0) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
    }
}

struct BwdParams {
    const void *dy, *x, *weight, *dh;
    const float *mean, *rstd;
    void* dx;
    float *dweight, *dbias, *parts;
    int64_t rows, cols, lddy, ldx, lddh, lddx;
    int nparts;
};

// Column sums of one slice of rows: thread = column, slice = blockIdx.y.
template <typename X, typename Y>
__global__ void __launch_bounds__(kThreads) norm_bwd_cols_kernel(BwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t c = blockIdx.x * (int64_t)kThreads + threadIdx.x;
    if (c >= p.cols) return;
    const int64_t r0 = p.rows * blockIdx.y / p.nparts, r1 = p.rows * (blockIdx.y + 1) / p.nparts;
    float sw = 0.0f, sb = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const float dy = load1(static_cast<const Y*>(p.dy) + r * p.lddy + c);
        sw += dy * ((load1(static_cast<const X*>(p.x) + r * p.ldx + c) - p.mean[r]) * p.rstd[r]);
        sb += dy;
    }
    p.parts[(2 * (int64_t)blockIdx.y) * p.cols + c] = sw;
    p.parts[(2 * (int64_t)blockIdx.y + 1) * p.cols + c] = sb;
}

__global__ void __launch_bounds__(kThreads) norm_bwd_join_kernel(BwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t c = blockIdx.x * (int64_t)kThreads + threadIdx.x;
    if (c >= p.cols) return;
    float sw = 0.0f, sb = 0.0f;
    for (int i = 0; i < p.nparts; ++i) {
        sw += p.parts[(2 * (int64_t)i) * p.cols + c];
        sb += p.parts[(2 * (int64_t)i + 1) * p.cols + c];
    }
    p.dweight[c] = sw;
    if (p.dbias) p.dbias[c] = sb;
}

template <typename X, typename Y, typename W>
__global__ void __launch_bounds__(kThreads) norm_bwd_rows_kernel(BwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float red[kThreads / 32];
    const W* w = static_cast<const W*>(p.weight);
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const X* x = static_cast<const X*>(p.x) + r * p.ldx;
        const Y* dy = static_cast<const Y*>(p.dy) + r * p.lddy;
        const X* dh = p.dh ? static_cast<const X*>(p.dh) + r * p.lddh : nullptr;
        X* dx = static_cast<X*>(p.dx) + r * p.lddx;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
            const float g = load1(dy + c) * load1(w + c);
            s1 += g;
            s2 += g * ((load1(x + c) - mean) * rstd);
        }
        s1 = block_sum(s1, red) / (float)p.cols;
        s2 = block_sum(s2, red) / (float)p.cols;
        for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
            const float g = load1(dy + c) * load1(w + c), xhat = (load1(x + c) - mean) * rstd;
            store1(dx + c, rstd * (g - s1 - xhat * s2) + (dh ? load1(dh + c) : 0.0f));
        }
    }
}

constexpr int kMaxParts = 64;
int parts_for(int64_t rows) { return (int)std::max<int64_t>(1, std::min<int64_t>(kMaxParts, rows / 16)); }

template <typename T> struct Tag { using type = T; };

// f(X, Y, W) for the three element types.
template <typename F>
nvfp4_status with_types(int32_t x, int32_t y, int32_t w, F&& f) {
    auto on_w = [&](auto tx, auto ty) {
        return w == NVFP4_F32 ? f(tx, ty, Tag<float>{}) : f(tx, ty, Tag<__nv_bfloat16>{});
    };
    auto on_y = [&](auto tx) {
        return y == NVFP4_F32 ? on_w(tx, Tag<float>{}) : on_w(tx, Tag<__nv_bfloat16>{});
    };
    return x == NVFP4_F32 ? on_y(Tag<float>{}) : on_y(Tag<__nv_bfloat16>{});
}

bool known(int32_t t) { return t == NVFP4_F32 || t == NVFP4_BF16; }
bool aligned_to(const void* p, int32_t t) { return reinterpret_cast<uintptr_t>(p) % (t == NVFP4_F32 ? 4 : 2) == 0; }
nvfp4_status to_status(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_layer_norm_forward(const void* x, int32_t x_dtype, int64_t rows, int64_t cols,
                                                 int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                                                 const void* bias, int32_t w_dtype, float eps, void* y,
                                                 int32_t y_dtype, int64_t ldy, void* h, int64_t ldh, float* mean,
                                                 float* rstd, void* stream) {
    if (!known(x_dtype) || !known(y_dtype) || !known(w_dtype)) return NVFP4_ERR_INVALID_ARG;
    if (rows < 0 || cols < 1 || cols > (1ll << 30) || rows > (1ll << 40)) return NVFP4_ERR_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps) || (residual == nullptr) != (h == nullptr)) return NVFP4_ERR_INVALID_ARG;
    if (rows == 0) return NVFP4_OK;
    if (!x || !weight || !y || !mean || !rstd) return NVFP4_ERR_INVALID_ARG;
    if (ldx < cols || ldy < cols || (residual && (ldr < cols || ldh < cols))) return NVFP4_ERR_SHAPE;
    if (!aligned_to(x, x_dtype) || !aligned_to(residual, x_dtype) || !aligned_to(h, x_dtype) ||
        !aligned_to(weight, w_dtype) || !aligned_to(bias, w_dtype) || !aligned_to(y, y_dtype) ||
        !aligned_to(mean, NVFP4_F32) || !aligned_to(rstd, NVFP4_F32))
        return NVFP4_ERR_ALIGNMENT;
    FwdParams p{x, residual, weight, bias, y, h, mean, rstd, rows, cols, ldx, ldr, ldy, ldh, eps};
    const int grid = (int)std::min<int64_t>(rows, 1 << 20);
    return with_types(x_dtype, y_dtype, w_dtype, [&](auto tx, auto ty, auto tw) {
        return to_status(launch_pdl(
            norm_fwd_kernel<typename decltype(tx)::type, typename decltype(ty)::type, typename decltype(tw)::type>,
            dim3(grid), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), p));
    });
}

extern "C" size_t nvfp4_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1) return 0;
    return (size_t)parts_for(rows) * 2 * (size_t)cols * sizeof(float);
}

extern "C" nvfp4_status nvfp4_layer_norm_backward(const void* dy, int32_t y_dtype, int64_t lddy, const void* x,
                                                  int32_t x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                                                  const void* weight, int32_t w_dtype, const float* mean,
                                                  const float* rstd, const void* dh, int64_t lddh, void* dx,
                                                  int64_t lddx, float* dweight, float* dbias, void* workspace,
                                                  size_t workspace_bytes, void* stream) {
    if (!known(x_dtype) || !known(y_dtype) || !known(w_dtype)) return NVFP4_ERR_INVALID_ARG;
    if (rows < 0 || cols < 1 || cols > (1ll << 30) || rows > (1ll << 40)) return NVFP4_ERR_SHAPE;
    if (!dweight || (rows > 0 && (!dy || !x || !weight || !mean || !rstd || !dx))) return NVFP4_ERR_INVALID_ARG;
    if (rows > 0 && (lddy < cols || ldx < cols || lddx < cols || (dh && lddh < cols))) return NVFP4_ERR_SHAPE;
    if (!aligned_to(x, x_dtype) || !aligned_to(dh, x_dtype) || !aligned_to(dx, x_dtype) ||
        !aligned_to(weight, w_dtype) || !aligned_to(dy, y_dtype) || !aligned_to(mean, NVFP4_F32) ||
        !aligned_to(rstd, NVFP4_F32) || !aligned_to(dweight, NVFP4_F32) || !aligned_to(dbias, NVFP4_F32))
        return NVFP4_ERR_ALIGNMENT;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < nvfp4_layer_norm_backward_workspace_bytes(rows, cols))
        return NVFP4_ERR_WORKSPACE;
    BwdParams p{dy,   x,    weight, dh,   mean, rstd, dx,   dweight,        dbias, static_cast<float*>(workspace),
                rows, cols, lddy,   ldx,  lddh, lddx, parts_for(rows)};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned col_blocks = (unsigned)((cols + kThreads - 1) / kThreads);
    return with_types(x_dtype, y_dtype, w_dtype, [&](auto tx, auto ty, auto tw) {
        using X = typename decltype(tx)::type;
        using Y = typename decltype(ty)::type;
        using W = typename decltype(tw)::type;
        cudaError_t e = launch_pdl(norm_bwd_cols_kernel<X, Y>, dim3(col_blocks, p.nparts), dim3(kThreads), 0, s, p);
        if (e == cudaSuccess) e = launch_pdl(norm_bwd_join_kernel, dim3(col_blocks), dim3(kThreads), 0, s, p);
        if (e == cudaSuccess && rows > 0)
            e = launch_pdl(norm_bwd_rows_kernel<X, Y, W>, dim3((unsigned)std::min<int64_t>(rows, 1 << 20)),
                           dim3(kThreads), 0, s, p);
        return to_status(e);
    });
}
