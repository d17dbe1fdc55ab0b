// optimizer.cu -- AdamW over many tensors, with the two states in fp32 or in 8 bits (include/nvfp4.h
// has the formulas).  Every line of the update is one IEEE fp32 operation after another, so a result
// does not depend on how the compiler contracts it.
//
// 8-bit states: blocks of 128 elements with one fp32 scale and E4M3 codes, 2^-9 .. 448 below a
// block's largest value.  A step moves v by 1 - beta2 of its distance to g^2, less than half a code
// step (1/16 .. 1/8 of the value), so rounded to nearest it would stay where it is; rounded
// stochastically it follows in expectation, with a spread of about 0.018 / sqrt(1 - beta2) .. 0.036 /
// sqrt(1 - beta2) of the value (step^2 / 6 a step against a pull of 1 - beta2).  v's code is kept off
// zero: a denominator rounded to zero would blow the next step up.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cmath>
#include <cstdint>

#include "device_common.cuh"
#include "host_common.h"

namespace nvfp4 {
namespace {

constexpr int kBlock = 128;                    // elements with one scale

struct AdamwConsts {
    float b1, c1, b2, c2;                      // beta, 1 - beta
    float size, unbias, eps;                   // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    uint32_t step;
    const float* grad_scale;
    uint32_t* dev_status;
    PhiloxKey key;
};

struct AdamwTensor {
    void* param;
    const void* grad;
    void *m, *v;
    float *m_scale, *v_scale;
    int64_t n;
    float keep;                                // 1 - lr * weight_decay
    uint32_t id;
};

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ Philox4 words_of(const AdamwConsts& k, int64_t i, uint32_t stream) {
    return philox4x32_10((uint32_t)(i >> 2), (uint32_t)(i >> 34), stream, k.step, k.key);
}

// bf16 from fp32 bits: to nearest even, or up where the low half plus rand16 carries.
__device__ __forceinline__ float to_bf16(float v, bool sr, uint32_t rand16) {
    if (!sr) return __bfloat162float(__float2bfloat16_rn(v));
    uint32_t b = __float_as_uint(v);
    if ((b & 0x7F800000u) != 0x7F800000u) b += rand16;
    return __uint_as_float(b & 0xFFFF0000u);
}

// E4M3 code of x.  2^-120 x has the grid's exponents, subnormals included, as fp32's own: the code
// is the word's top bits, 20 bits below them deciding the rounding.
__device__ __forceinline__ uint32_t to_e4m3(float x, bool sr, uint32_t rand16) {
    const uint32_t sign = (__float_as_uint(x) >> 24) & 0x80u;
    const uint32_t b = __float_as_uint(__fmul_rn(fabsf(x), 0x1p-120f));
    const uint32_t up = sr ? rand16 << 4 : 0x7FFFFu + ((b >> 20) & 1u);
    return sign | min((b + up) >> 20, 126u);
}
__device__ __forceinline__ float from_e4m3(uint32_t code) {
    return __fmul_rn(__uint_as_float(((code & 0x80u) << 24) | ((code & 0x7Fu) << 20)), 0x1p120f);
}

__device__ __forceinline__ void update(const AdamwConsts& k, float g, float keep, float& p, float& m, float& v) {
    m = __fadd_rn(__fmul_rn(m, k.b1), __fmul_rn(g, k.c1));
    v = __fadd_rn(__fmul_rn(v, k.b2), __fmul_rn(__fmul_rn(g, g), k.c2));
    p = __fsub_rn(__fmul_rn(p, keep),
                  __fdiv_rn(__fmul_rn(m, k.size), __fadd_rn(__fmul_rn(__fsqrt_rn(v), k.unbias), k.eps)));
}

template <typename P>
__device__ __forceinline__ void store_param(const AdamwConsts& k, P* p, int64_t i, float v, bool sr, uint32_t id) {
    if constexpr (sizeof(P) == 4) p[i] = v;
    else {
        const uint32_t r = sr ? words_of(k, i, 2 * id + 1).w[i & 3] & 0xFFFFu : 0u;
        p[i] = __float2bfloat16_rn(to_bf16(v, sr, r));
    }
}

template <typename P, typename G>
__global__ void __launch_bounds__(256) adamw32_kernel(AdamwTensor t, AdamwConsts k, int sr) {
    pdl_launch_dependents();
    pdl_wait();
    const float gs = k.grad_scale ? *k.grad_scale : 1.0f;
    P* p = static_cast<P*>(t.param);
    float *m = static_cast<float*>(t.m), *v = static_cast<float*>(t.v);
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < t.n; i += gridDim.x * 256ll) {
        const float g = __fmul_rn(load1(static_cast<const G*>(t.grad) + i), gs);
        if (!isfinite(g)) set_status(k.dev_status, NVFP4_ERR_NONFINITE);
        float pv = load1(p + i), mv = m[i], vv = v[i];
        update(k, g, t.keep, pv, mv, vv);
        m[i] = mv;
        v[i] = vv;
        store_param(k, p, i, pv, sr, t.id);
    }
}

// max over a block's 128 threads, on the bits of non-negative values (NaN above all others).
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
    v = __reduce_max_sync(~0u, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return max(max(red[0], red[1]), max(red[2], red[3]));
}

__device__ __forceinline__ uint8_t encode(float x, uint32_t top_bits, float* scale, bool sr, uint32_t rand16,
                                          bool floor1) {
    const float top = __uint_as_float(top_bits);
    const float inv = top > 0.0f ? fminf(__fdiv_rn(448.0f, top), FLT_MAX) : 0.0f;
    if (threadIdx.x == 0) *scale = __fmul_rn(top, 1.0f / 448.0f);
    uint32_t c = to_e4m3(__fmul_rn(x, inv), sr, rand16);
    if (floor1 && x > 0.0f) c = max(c, 1u);
    return (uint8_t)c;
}

template <typename P, typename G>
__global__ void __launch_bounds__(kBlock) adamw8_kernel(AdamwTensor t, AdamwConsts k, int sr) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ uint32_t red[4];
    const float gs = k.grad_scale ? *k.grad_scale : 1.0f;
    P* p = static_cast<P*>(t.param);
    uint8_t *mc = static_cast<uint8_t*>(t.m), *vc = static_cast<uint8_t*>(t.v);
    const int64_t blocks = (t.n + kBlock - 1) / kBlock;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const int64_t i = b * kBlock + threadIdx.x;
        const bool in = i < t.n;
        float pv = 0.0f, mv = 0.0f, vv = 0.0f, g = 0.0f;
        if (in) {
            g = __fmul_rn(load1(static_cast<const G*>(t.grad) + i), gs);
            pv = load1(p + i);
            mv = __fmul_rn(from_e4m3(mc[i]), t.m_scale[b]);
            vv = __fmul_rn(from_e4m3(vc[i]), t.v_scale[b]);
        }
        if (!isfinite(g)) set_status(k.dev_status, NVFP4_ERR_NONFINITE);
        update(k, g, t.keep, pv, mv, vv);
        const uint32_t mt = block_max(__float_as_uint(fabsf(mv)), red);   // its barriers follow the scale reads
        const uint32_t vt = block_max(__float_as_uint(fabsf(vv)), red);
        const uint32_t w = sr ? words_of(k, i, 2 * t.id).w[i & 3] : 0u;
        const uint8_t cm = encode(mv, mt, t.m_scale + b, sr, w & 0xFFFFu, false);
        const uint8_t cv = encode(vv, vt, t.v_scale + b, sr, w >> 16, true);
        if (in) {
            mc[i] = cm;
            vc[i] = cv;
            store_param(k, p, i, pv, sr, t.id);
        }
    }
}

template <typename P, typename G>
cudaError_t launch_one(const AdamwTensor& t, const AdamwConsts& k, int bits, int sr, cudaStream_t s) {
    if (bits == 32) {
        const int grid = (int)std::min<int64_t>((t.n + 255) / 256, 152 * 32);
        return launch_pdl(adamw32_kernel<P, G>, dim3(grid), dim3(256), 0, s, t, k, sr);
    }
    const int grid = (int)std::min<int64_t>((t.n + kBlock - 1) / kBlock, 152 * 64);
    return launch_pdl(adamw8_kernel<P, G>, dim3(grid), dim3(kBlock), 0, s, t, k, sr);
}

bool known(int32_t t) { return t == NVFP4_F32 || t == NVFP4_BF16; }
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_adamw_step(const nvfp4_adamw_tensor* tensors, int32_t count,
                                         const nvfp4_adamw_params* hp, const float* grad_scale, uint32_t* dev_status,
                                         void* stream) {
    if (count < 0 || !hp || (count > 0 && !tensors)) return NVFP4_ERR_INVALID_ARG;
    if ((hp->bits != 32 && hp->bits != 8) || (hp->round != NVFP4_ROUND_RNE && hp->round != NVFP4_ROUND_SR) ||
        hp->step < 1 || hp->step > 0xFFFFFFFFll)
        return NVFP4_ERR_INVALID_ARG;
    if (!(hp->beta1 >= 0 && hp->beta1 < 1) || !(hp->beta2 >= 0 && hp->beta2 < 1) || !(hp->eps >= 0) ||
        !std::isfinite(hp->eps) || !std::isfinite(hp->lr))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned_to(grad_scale, 4)) return NVFP4_ERR_ALIGNMENT;
    for (int i = 0; i < count; ++i) {
        const nvfp4_adamw_tensor& t = tensors[i];
        if (t.n < 0 || t.n > (1ll << 40)) return NVFP4_ERR_SHAPE;
        if (!known(t.param_dtype) || !known(t.grad_dtype) || t.id < 0 || t.id >= (1ll << 30) ||
            !std::isfinite(t.weight_decay))
            return NVFP4_ERR_INVALID_ARG;
        if (t.n == 0 || !t.grad) continue;
        if (!t.param || !t.m || !t.v || (hp->bits == 8 && (!t.m_scale || !t.v_scale))) return NVFP4_ERR_INVALID_ARG;
        if (!aligned_to(t.param, t.param_dtype == NVFP4_F32 ? 4 : 2) ||
            !aligned_to(t.grad, t.grad_dtype == NVFP4_F32 ? 4 : 2) ||
            (hp->bits == 32 ? !aligned_to(t.m, 4) || !aligned_to(t.v, 4)
                            : !aligned_to(t.m_scale, 4) || !aligned_to(t.v_scale, 4)))
            return NVFP4_ERR_ALIGNMENT;
    }
    AdamwConsts k;
    k.b1 = (float)hp->beta1;
    k.c1 = (float)(1.0 - hp->beta1);
    k.b2 = (float)hp->beta2;
    k.c2 = (float)(1.0 - hp->beta2);
    k.size = (float)(hp->lr / (1.0 - std::pow(hp->beta1, (double)hp->step)));
    k.unbias = (float)(1.0 / std::sqrt(1.0 - std::pow(hp->beta2, (double)hp->step)));
    k.eps = (float)hp->eps;
    k.step = (uint32_t)hp->step;
    k.grad_scale = grad_scale;
    k.dev_status = dev_status;
    k.key = philox_key(hp->sr_seed);
    const int sr = hp->round == NVFP4_ROUND_SR;
    for (int i = 0; i < count; ++i) {
        const nvfp4_adamw_tensor& a = tensors[i];
        if (a.n == 0 || !a.grad) continue;
        const AdamwTensor t{a.param, a.grad, a.m, a.v, a.m_scale, a.v_scale, a.n,
                            (float)(1.0 - hp->lr * a.weight_decay), (uint32_t)a.id};
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        const bool pf = a.param_dtype == NVFP4_F32, gf = a.grad_dtype == NVFP4_F32;
        const cudaError_t e = pf ? (gf ? launch_one<float, float>(t, k, hp->bits, sr, s)
                                       : launch_one<float, __nv_bfloat16>(t, k, hp->bits, sr, s))
                                 : (gf ? launch_one<__nv_bfloat16, float>(t, k, hp->bits, sr, s)
                                       : launch_one<__nv_bfloat16, __nv_bfloat16>(t, k, hp->bits, sr, s));
        if (e != cudaSuccess) return NVFP4_ERR_CUDA;
    }
    return NVFP4_OK;
}
