// optimizer.cu -- AdamW over many tensors, with the two moments in fp32 or in 8 bits (include/nvfp4.h
// has the formulas).  Every line of the update is one IEEE fp32 operation after another, so a result
// does not depend on how the compiler contracts it.
//
// 8-bit states: blocks of 128 elements with one fp32 scale and E4M3 codes, 2^-9 .. 448 below a
// block's largest value.  A step moves v by 1 - beta2 of its distance to g^2, less than half a code
// step (1/16 .. 1/8 of the value), so rounded to nearest it would stay where it is; rounded
// stochastically it follows in expectation, with a spread of about 0.018 / sqrt(1 - beta2) .. 0.036 /
// sqrt(1 - beta2) of the value (step^2 / 6 a step against a pull of 1 - beta2).  v's code is kept off
// zero: a denominator rounded to zero would blow the next step up.
//
// One launch for many tensors: their descriptors are the kernel's parameter (no table to copy to the
// device), a block takes 2048 or 4096 neighbouring elements of one tensor and finds it by bisection.  Bound by
// memory: 26 bytes an element with fp32 parameters and states and bf16 gradients, 14.1 with 8-bit
// states.  A thread takes 8 neighbouring elements with 16-byte accesses, 16 threads an 8-bit state's
// block; tensors that do not lie on 16 bytes, and a tensor's last elements, go one by one.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cmath>
#include <cstdint>

#include "device_common.cuh"
#include "host_common.h"

namespace nvfp4 {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kBlock = 128;                    // elements with one scale
constexpr int kThreads = 256, kPer = 8;        // a thread's elements at a time
// Rounds of a CUDA block, their loads all issued first: 32-bit states bring enough bytes with one (272 M parameters: 998
// us, 1085 with two), 8-bit ones want two (751 us; 768 .. 825 with one).  Four blocks an SM for both (8-bit with
// three: 800 us).
template <int BITS> struct Slice {
    static constexpr int kRounds = BITS == 32 ? 1 : 2;
    static constexpr int kElements = kThreads * kPer * kRounds;
};
static_assert(Slice<8>::kElements % kBlock == 0 && kBlock == 16 * kPer, "an 8-bit block is 16 threads' elements");

struct AdamwConsts {
    float b1, c1, b2, c2;                      // beta, 1 - beta
    float size, unbias, eps;                   // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    uint32_t step;
    float one;                                 // 1, where the compiler must not know it
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
    uint32_t first_slice;
    uint32_t vec;                              // all of it on 16 bytes
};

// The descriptors of one launch: two sizes, so that few tensors do not carry a large parameter.
template <int MAX> struct Batch {
    AdamwTensor t[MAX];
    AdamwConsts k;
    int count;
};

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const bf16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ uint4 ld16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
template <int N> struct Raw;
template <> struct Raw<8> {                    // 8 bytes
    uint2 a;
    __device__ __forceinline__ void load(const void* p) {
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(a.x), "=r"(a.y) : "l"(p) : "memory");
    }
};
template <> struct Raw<16> {
    uint4 a;
    __device__ __forceinline__ void load(const void* p) { a = ld16(p); }
};
template <> struct Raw<32> {
    uint4 a, b;
    __device__ __forceinline__ void load(const void* p) {
        a = ld16(p);
        b = ld16(static_cast<const uint4*>(p) + 1);
    }
};
__device__ __forceinline__ void get8(const Raw<16>& r, float (&f)[8]) { Vec<uint16_t>::unpack(r.a, f); }      // bf16
__device__ __forceinline__ void get8(const Raw<32>& r, float (&f)[8]) {
    Vec<float>::unpack(r.a, f);
    Vec<float>::unpack(r.b, f + 4);
}
__device__ __forceinline__ void put8(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void put8(bf16* p, const float (&f)[8]) {       // values that bf16 holds
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __byte_perm(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]), 0x7632);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ Philox4 words_of(const AdamwConsts& k, int64_t i, uint32_t stream) {
    return philox4x32_10((uint32_t)(i >> 2), (uint32_t)(i >> 34), stream, k.step, k.key);
}

// The nearest-even or stochastic bf16 value (up where the low half plus rand16 carries).
template <bool SR> __device__ __forceinline__ float to_bf16(float v, uint32_t rand16) {
    if constexpr (!SR) return __bfloat162float(__float2bfloat16_rn(v));
    uint32_t b = __float_as_uint(v);
    if ((b & 0x7F800000u) != 0x7F800000u) b += rand16;
    return __uint_as_float(b & 0xFFFF0000u);
}

// Two fp32 operations at once.  The assembler contracts a packed product with a packed sum that follows it, both
// marked .rn or not (61660 of 262144 random pairs came out as fused ones), so a sum is written as a * 1 + b with a 1
// that it does not know.
__device__ __forceinline__ float2 mul2(float2 a, float b) { return __fmul2_rn(a, make_float2(b, b)); }
__device__ __forceinline__ float2 add2(const float one, float2 a, float2 b) { return __ffma2_rn(a, make_float2(one, one), b); }

// max of magnitudes; NaN wins
__device__ __forceinline__ float max_abs(float a, float b) {
    float r;
    asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %2;\n\tmax.NaN.f32 %0, %1, t;\n\t}" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Two E4M3 codes (the low 16 bits) as values.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
    uint32_t h;
    const uint16_t in = (uint16_t)codes;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(in));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// The E4M3 code of a magnitude x >= 0 in the top byte.  2^-120 x has the grid's exponents, subnormals
// included, as fp32's own: the code is the word's bits 20 .. 27, the 20 bits below them deciding the rounding.
// `scaled`: 2^-120 x; rand: 16 random bits at bits 4 .. 19.
template <bool SR> __device__ __forceinline__ uint32_t to_e4m3_top(float scaled, uint32_t rand, uint32_t least) {
    const uint32_t b = __float_as_uint(scaled) & 0x7FFFFFFFu;
    const uint32_t up = SR ? rand : 0x7FFFFu + ((b >> 20) & 1u);
    return max(min(b + up, (126u << 20) | 0xFFFFFu), least) << 4;
}
// The top bytes of four words, first in the lowest byte.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

__device__ __forceinline__ void update2(const AdamwConsts& k, float2 g, float keep, float2& p, float2& m, float2& v) {
    m = add2(k.one, mul2(m, k.b1), mul2(g, k.c1));
    v = add2(k.one, mul2(v, k.b2), mul2(__fmul2_rn(g, g), k.c2));
    const float2 num = mul2(m, k.size);
    const float2 den = add2(k.one, mul2(make_float2(__fsqrt_rn(v.x), __fsqrt_rn(v.y)), k.unbias), make_float2(k.eps, k.eps));
    const float2 q = make_float2(-__fdiv_rn(num.x, den.x), -__fdiv_rn(num.y, den.y));
    p = add2(k.one, mul2(p, keep), q);
}

__device__ __forceinline__ float inverse_of(float top) {
    return top > 0.0f ? fminf(__fdiv_rn(448.0f, top), FLT_MAX) : 0.0f;
}
// the largest over the 16 threads of a block; NaN wins
__device__ __forceinline__ float max16(float v) {
#pragma unroll
    for (int d = 8; d; d >>= 1) v = max_abs(v, __shfl_xor_sync(~0u, v, d));
    return v;
}

template <typename P, typename G, int BITS, bool SR, int MAX>
__global__ void __launch_bounds__(kThreads, 4) adamw_kernel(const __grid_constant__ Batch<MAX> batch) {
    pdl_launch_dependents();
    pdl_wait();
    // the tensor of this slice: the last that begins at or before it
    int lo = 0, hi = batch.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (batch.t[mid].first_slice <= blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const AdamwTensor& t = batch.t[lo];
    const AdamwConsts& k = batch.k;
    const float gs = k.grad_scale ? *k.grad_scale : 1.0f;
    P* param = static_cast<P*>(t.param);
    const G* grad = static_cast<const G*>(t.grad);
    constexpr int kRounds = Slice<BITS>::kRounds;
    constexpr int SB = BITS == 32 ? 32 : 8;                // bytes of eight elements of a state
    constexpr int PB = 8 * sizeof(P), GB = 8 * sizeof(G);
    const int64_t n = t.n;
    const float keep = t.keep;
    const int64_t base = (int64_t)(blockIdx.x - t.first_slice) * Slice<BITS>::kElements + threadIdx.x * kPer;
    uint8_t *mc = static_cast<uint8_t*>(t.m), *vc = static_cast<uint8_t*>(t.v);

    // all rounds' loads first
    Raw<PB> rp[kRounds];
    Raw<GB> rg[kRounds];
    Raw<SB> rm[kRounds], rv[kRounds];
    float sm[kRounds], sv[kRounds];
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
        const int64_t i = base + q * (kThreads * kPer);
        if (t.vec && i + kPer <= n) {
            rp[q].load(param + i);
            rg[q].load(grad + i);
            rm[q].load(mc + i * (SB / 8));
            rv[q].load(vc + i * (SB / 8));
        }
        if (BITS == 8) {
            sm[q] = i < n ? t.m_scale[i / kBlock] : 0.0f;
            sv[q] = i < n ? t.v_scale[i / kBlock] : 0.0f;
        }
    }
    float2 finite = make_float2(0.0f, 0.0f);               // sums 0 * g: NaN once a gradient is not finite
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
        const int64_t i = base + q * (kThreads * kPer);
        const bool full = t.vec && i + kPer <= n;
        float p[8] = {}, g[8] = {}, m[8] = {}, v[8] = {};
        uint32_t cm[2] = {}, cv[2] = {};
        if (full) {
            get8(rp[q], p);
            get8(rg[q], g);
            if constexpr (BITS == 32) {
                get8(rm[q], m);
                get8(rv[q], v);
            } else {
                cm[0] = rm[q].a.x; cm[1] = rm[q].a.y;
                cv[0] = rv[q].a.x; cv[1] = rv[q].a.y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (i + e < n) {
                    p[e] = load1(param + i + e);
                    g[e] = load1(grad + i + e);
                    if constexpr (BITS == 32) {
                        m[e] = static_cast<float*>(t.m)[i + e];
                        v[e] = static_cast<float*>(t.v)[i + e];
                    } else {
                        cm[e >> 2] |= (uint32_t)mc[i + e] << (8 * (e & 3));
                        cv[e >> 2] |= (uint32_t)vc[i + e] << (8 * (e & 3));
                    }
                }
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float2 p2 = make_float2(p[e], p[e + 1]), m2 = make_float2(m[e], m[e + 1]), v2 = make_float2(v[e], v[e + 1]);
            if constexpr (BITS == 8) {
                m2 = mul2(from_e4m3x2(cm[e >> 2] >> (8 * (e & 2))), sm[q]);
                v2 = mul2(from_e4m3x2(cv[e >> 2] >> (8 * (e & 2))), sv[q]);
            }
            const float2 g2 = mul2(make_float2(g[e], g[e + 1]), gs);
            finite = __ffma2_rn(g2, make_float2(0.0f, 0.0f), finite);
            update2(k, g2, keep, p2, m2, v2);
            p[e] = p2.x; p[e + 1] = p2.y;
            m[e] = m2.x; m[e + 1] = m2.y;
            v[e] = v2.x; v[e + 1] = v2.y;
        }
        // a bf16 parameter's random words, stream 1; words of elements 4 j .. 4 j + 3 from one call
        if constexpr (sizeof(P) == 2) {
            Philox4 w[2] = {};
            if constexpr (SR) {
                w[0] = words_of(k, i, 2 * t.id + 1);
                w[1] = words_of(k, i + 4, 2 * t.id + 1);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = to_bf16<SR>(p[e], w[e >> 2].w[e & 3] & 0xFFFFu);
        }
        if constexpr (BITS == 8) {
            // past the tensor's end everything is zero: it takes no part in the largest values
            float topm = 0.0f, topv = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                topm = max_abs(topm, m[e]);
                topv = max_abs(topv, v[e]);
            }
            topm = max16(topm);
            topv = max16(topv);
            if ((threadIdx.x & 15) == 0 && i < n) {
                t.m_scale[i / kBlock] = __fmul_rn(topm, 1.0f / 448.0f);
                t.v_scale[i / kBlock] = __fmul_rn(topv, 1.0f / 448.0f);
            }
            const float im = inverse_of(topm), iv = inverse_of(topv);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                Philox4 w = {};
                if constexpr (SR) w = words_of(k, i + 4 * h, 2 * t.id);
                uint32_t a[4], b[4];
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const int f = 4 * h + e;
                    const float2 x = mul2(mul2(make_float2(m[f], m[f + 1]), im), 0x1p-120f);
                    const float2 y = mul2(mul2(make_float2(v[f], v[f + 1]), iv), 0x1p-120f);
                    a[e] = to_e4m3_top<SR>(x.x, (w.w[e] << 4) & 0xFFFF0u, 0u);
                    a[e + 1] = to_e4m3_top<SR>(x.y, (w.w[e + 1] << 4) & 0xFFFF0u, 0u);
                    b[e] = to_e4m3_top<SR>(y.x, (w.w[e] >> 12) & 0xFFFF0u, v[f] > 0.0f ? 1u << 20 : 0u);
                    b[e + 1] = to_e4m3_top<SR>(y.y, (w.w[e + 1] >> 12) & 0xFFFF0u, v[f + 1] > 0.0f ? 1u << 20 : 0u);
                }
                const uint32_t sign = top_bytes(__float_as_uint(m[4 * h]), __float_as_uint(m[4 * h + 1]),
                                                __float_as_uint(m[4 * h + 2]), __float_as_uint(m[4 * h + 3]));
                cm[h] = top_bytes(a[0], a[1], a[2], a[3]) | (sign & 0x80808080u);
                cv[h] = top_bytes(b[0], b[1], b[2], b[3]);
            }
        }
        if (full) {
            put8(param + i, p);
            if constexpr (BITS == 32) {
                put8(static_cast<float*>(t.m) + i, m);
                put8(static_cast<float*>(t.v) + i, v);
            } else {
                *reinterpret_cast<uint2*>(mc + i) = make_uint2(cm[0], cm[1]);
                *reinterpret_cast<uint2*>(vc + i) = make_uint2(cv[0], cv[1]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (i + e < n) {
                    if constexpr (sizeof(P) == 4) param[i + e] = p[e];
                    else param[i + e] = __float2bfloat16_rn(p[e]);
                    if constexpr (BITS == 32) {
                        static_cast<float*>(t.m)[i + e] = m[e];
                        static_cast<float*>(t.v)[i + e] = v[e];
                    } else {
                        mc[i + e] = (uint8_t)(cm[e >> 2] >> (8 * (e & 3)));
                        vc[i + e] = (uint8_t)(cv[e >> 2] >> (8 * (e & 3)));
                    }
                }
        }
    }
    if (!(finite.x + finite.y == 0.0f)) set_status(k.dev_status, NVFP4_ERR_NONFINITE);
}

bool known(int32_t t) { return t == NVFP4_F32 || t == NVFP4_BF16; }
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

constexpr int kFew = 24, kMany = 400;
static_assert(sizeof(Batch<kMany>) <= 32764, "kernel parameters");

template <typename P, typename G, int MAX>
cudaError_t launch(const Batch<MAX>& b, int bits, bool sr, unsigned slices, cudaStream_t s) {
    auto kern = bits == 32 ? (sr && sizeof(P) == 2 ? adamw_kernel<P, G, 32, true, MAX> : adamw_kernel<P, G, 32, false, MAX>)
                           : (sr ? adamw_kernel<P, G, 8, true, MAX> : adamw_kernel<P, G, 8, false, MAX>);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(slices);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[1] = {const_cast<Batch<MAX>*>(&b)};         // by address: the batch is not copied on the way
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kern), args);
}

// The tensors of one pair of types, at most MAX a launch.
template <typename P, typename G, int MAX>
cudaError_t step_types(const nvfp4_adamw_tensor* ts, int count, const nvfp4_adamw_params& hp, const AdamwConsts& k,
                       int32_t pt, int32_t gt, cudaStream_t s) {
    Batch<MAX> b;
    b.k = k;
    b.count = 0;
    int64_t slices = 0;
    const int64_t slice = hp.bits == 32 ? Slice<32>::kElements : Slice<8>::kElements;
    cudaError_t e = cudaSuccess;
    auto flush = [&] {
        if (b.count && e == cudaSuccess) e = launch<P, G, MAX>(b, hp.bits, hp.round == NVFP4_ROUND_SR, (unsigned)slices, s);
        b.count = 0;
        slices = 0;
    };
    for (int i = 0; i < count; ++i) {
        const nvfp4_adamw_tensor& a = ts[i];
        if (a.n == 0 || !a.grad || a.param_dtype != pt || a.grad_dtype != gt) continue;
        const int64_t mine = (a.n + slice - 1) / slice;    // at most 2^29
        if (b.count == MAX || slices + mine > (1ll << 30)) flush();
        const size_t state = hp.bits == 32 ? 16 : 8;
        const bool vec = aligned16(a.param) && aligned16(a.grad) && aligned_to(a.m, state) && aligned_to(a.v, state);
        b.t[b.count++] = AdamwTensor{a.param, a.grad, a.m, a.v, a.m_scale, a.v_scale, a.n, (float)(1.0 - hp.lr * a.weight_decay),
                                     (uint32_t)a.id, (uint32_t)slices, vec};
        slices += mine;
    }
    flush();
    return e;
}

template <int MAX>
cudaError_t step_all(const nvfp4_adamw_tensor* ts, int count, const nvfp4_adamw_params& hp, const AdamwConsts& k,
                     const bool (&seen)[2][2], cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (seen[0][0]) e = step_types<float, float, MAX>(ts, count, hp, k, NVFP4_F32, NVFP4_F32, s);
    if (seen[0][1] && e == cudaSuccess) e = step_types<float, bf16, MAX>(ts, count, hp, k, NVFP4_F32, NVFP4_BF16, s);
    if (seen[1][0] && e == cudaSuccess) e = step_types<bf16, float, MAX>(ts, count, hp, k, NVFP4_BF16, NVFP4_F32, s);
    if (seen[1][1] && e == cudaSuccess) e = step_types<bf16, bf16, MAX>(ts, count, hp, k, NVFP4_BF16, NVFP4_BF16, s);
    return e;
}

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
    bool seen[2][2] = {};
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
        seen[t.param_dtype][t.grad_dtype] = true;
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
    k.one = 1.0f;
    k.grad_scale = grad_scale;
    k.dev_status = dev_status;
    k.key = philox_key(hp->sr_seed);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = count <= kFew ? step_all<kFew>(tensors, count, *hp, k, seen, s)
                                        : step_all<kMany>(tensors, count, *hp, k, seen, s);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
