// attention.cu -- attention over packed sequences, forward and backward (include/nvfp4.h has the
// formulas).  bf16 heads of at most 128 elements; sums and softmax statistics in fp32.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cmath>
#include <cstdint>

#include "device_common.cuh"
#include "host_common.h"

namespace nvfp4 {
namespace attn {

using bf16 = __nv_bfloat16;

struct Heads {
    bf16* p;
    int64_t ts, hs;
    __device__ __forceinline__ bf16* at(int64_t t, int h) const { return p + t * ts + h * hs; }
};

struct Params {
    Heads q, k, v, out, dout, dq, dk, dv;
    float* lse;
    float* delta;
    int64_t tq, tk;
    int heads, kv_heads, dim, causal, nseq;
    float scale;
    const int32_t *cu_q, *cu_k;
    uint32_t* dev_status;
};

// Bounds of sequence s among `total` tokens, forced into range whatever the offsets hold.
__device__ __forceinline__ void seq_bounds(const int32_t* cu, int s, int64_t total, int64_t& a, int64_t& b) {
    if (!cu) {
        a = 0;
        b = total;
        return;
    }
    a = min(max((int64_t)cu[s], (int64_t)0), total);
    b = min(max((int64_t)cu[s + 1], a), total);
}

// The sequence a token belongs to: the first whose end lies beyond it.
__device__ __forceinline__ int seq_of(const int32_t* cu, int nseq, int64_t t) {
    if (!cu) return 0;
    int lo = 0, hi = nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (cu[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__global__ void check_offsets_kernel(Params p) {
    pdl_launch_dependents();
    pdl_wait();
    for (int which = 0; which < 2; ++which) {
        const int32_t* cu = which ? p.cu_k : p.cu_q;
        const int64_t total = which ? p.tk : p.tq;
        for (int i = threadIdx.x; i < p.nseq; i += blockDim.x)
            if (cu[i] > cu[i + 1] || (i == 0 && cu[0] != 0) || (i == p.nseq - 1 && cu[p.nseq] != total))
                set_status(p.dev_status, NVFP4_ERR_INVALID_ARG);
    }
}

__device__ __forceinline__ void load_row(const bf16* p, int dim, float (&f)[4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = lane + 32 * j < dim ? __bfloat162float(p[lane + 32 * j]) : 0.0f;
}
__device__ __forceinline__ void store_row(bf16* p, int dim, const float (&f)[4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (lane + 32 * j < dim) p[lane + 32 * j] = __float2bfloat16_rn(f[j]);
}
__device__ __forceinline__ float dot(const float (&a)[4], const float (&b)[4]) {
    float s = a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    return s;
}

// Keys [k0, kend) that query t of its sequence sees.
__device__ __forceinline__ void keys_of(const Params& p, int64_t t, int64_t& k0, int64_t& kend) {
    const int s = seq_of(p.cu_q, p.nseq, t);
    int64_t q0, q1, k1;
    seq_bounds(p.cu_q, s, p.tq, q0, q1);
    seq_bounds(p.cu_k, s, p.tk, k0, k1);
    kend = p.causal ? max(k0, min(k1, k1 - (q1 - t) + 1)) : k1;
}

// One warp per query and head: the running maximum and sum of the softmax over the keys in turn.
__global__ void __launch_bounds__(256) fwd_kernel(Params p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = blockIdx.x * 8ll + (threadIdx.x >> 5);
    const int h = blockIdx.y, hk = h / (p.heads / p.kv_heads);
    if (t >= p.tq) return;
    int64_t k0, kend;
    keys_of(p, t, k0, kend);
    float q[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.0f;
    load_row(p.q.at(t, h), p.dim, q);
    for (int64_t j = k0; j < kend; ++j) {
        float k[4], v[4];
        load_row(p.k.at(j, hk), p.dim, k);
        load_row(p.v.at(j, hk), p.dim, v);
        const float z = dot(q, k) * p.scale, mn = fmaxf(m, z), ms = mn == -INFINITY ? 0.0f : mn;
        const float a = expf(m - ms), e = expf(z - ms);
        l = l * a + e;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = o[i] * a + e * v[i];
        m = mn;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= inv;
    store_row(p.out.at(t, h), p.dim, o);
    if ((threadIdx.x & 31) == 0) p.lse[h * p.tq + t] = m + logf(l);
}

// delta = sum(dout * out), and dq of one query and head per warp.
__global__ void __launch_bounds__(256) bwd_dq_kernel(Params p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = blockIdx.x * 8ll + (threadIdx.x >> 5);
    const int h = blockIdx.y, hk = h / (p.heads / p.kv_heads);
    if (t >= p.tq) return;
    int64_t k0, kend;
    keys_of(p, t, k0, kend);
    float q[4], o[4], d[4], dq[4] = {0, 0, 0, 0};
    load_row(p.q.at(t, h), p.dim, q);
    load_row(p.out.at(t, h), p.dim, o);
    load_row(p.dout.at(t, h), p.dim, d);
    const float delta = dot(o, d), lse = p.lse[h * p.tq + t];
    if ((threadIdx.x & 31) == 0) p.delta[h * p.tq + t] = delta;
    for (int64_t j = k0; j < kend; ++j) {
        float k[4], v[4];
        load_row(p.k.at(j, hk), p.dim, k);
        load_row(p.v.at(j, hk), p.dim, v);
        const float ds = expf(dot(q, k) * p.scale - lse) * (dot(d, v) - delta) * p.scale;
#pragma unroll
        for (int i = 0; i < 4; ++i) dq[i] += ds * k[i];
    }
    store_row(p.dq.at(t, h), p.dim, dq);
}

// dk and dv of one key and key head per warp, over the queries of the heads that share it.
__global__ void __launch_bounds__(256) bwd_dkv_kernel(Params p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t j = blockIdx.x * 8ll + (threadIdx.x >> 5);
    const int hk = blockIdx.y, share = p.heads / p.kv_heads;
    if (j >= p.tk) return;
    const int s = seq_of(p.cu_k, p.nseq, j);
    int64_t q0, q1, k0, k1;
    seq_bounds(p.cu_q, s, p.tq, q0, q1);
    seq_bounds(p.cu_k, s, p.tk, k0, k1);
    const int64_t first = p.causal ? max(q0, q1 - (k1 - j)) : q0;
    float k[4], v[4], dk[4] = {0, 0, 0, 0}, dv[4] = {0, 0, 0, 0};
    load_row(p.k.at(j, hk), p.dim, k);
    load_row(p.v.at(j, hk), p.dim, v);
    for (int h = hk * share; h < (hk + 1) * share; ++h)
        for (int64_t t = first; t < q1; ++t) {
            float q[4], d[4];
            load_row(p.q.at(t, h), p.dim, q);
            load_row(p.dout.at(t, h), p.dim, d);
            const float e = expf(dot(q, k) * p.scale - p.lse[h * p.tq + t]);
            const float ds = e * (dot(d, v) - p.delta[h * p.tq + t]) * p.scale;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dv[i] += e * d[i];
                dk[i] += ds * q[i];
            }
        }
    store_row(p.dk.at(j, hk), p.dim, dk);
    store_row(p.dv.at(j, hk), p.dim, dv);
}

nvfp4_status check_shape(const nvfp4_attention_shape* s) {
    if (!s) return NVFP4_ERR_INVALID_ARG;
    if (s->tq < 0 || s->tk < 0 || s->tq > (1ll << 30) || s->tk > (1ll << 30) || s->heads < 1 || s->kv_heads < 1 ||
        s->heads > 65535 || s->heads % s->kv_heads != 0 || s->dim < 8 || s->dim > 128 || s->dim % 8 != 0)
        return NVFP4_ERR_SHAPE;
    if (s->nseq < 1 || (!s->cu_q) != (!s->cu_k) || (!s->cu_q && s->nseq != 1) || !std::isfinite(s->scale))
        return NVFP4_ERR_INVALID_ARG;
    if (s->nseq > (1 << 24)) return NVFP4_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(s->cu_q) | reinterpret_cast<uintptr_t>(s->cu_k)) % 4) return NVFP4_ERR_ALIGNMENT;
    return NVFP4_OK;
}

// A tensor of `tokens` x `heads`; `data` may be null where there are no tokens.
nvfp4_status check_heads(const nvfp4_heads* h, int64_t tokens, int heads, int dim) {
    if (!h) return NVFP4_ERR_INVALID_ARG;
    if (tokens == 0) return NVFP4_OK;
    if (!h->data) return NVFP4_ERR_INVALID_ARG;
    if ((tokens > 1 && h->token_stride < dim) || (heads > 1 && h->head_stride < dim)) return NVFP4_ERR_SHAPE;
    if (!aligned16(h->data) || (tokens > 1 && h->token_stride % 8) || (heads > 1 && h->head_stride % 8))
        return NVFP4_ERR_ALIGNMENT;
    return NVFP4_OK;
}

Heads heads_of(const nvfp4_heads* h) { return Heads{static_cast<bf16*>(h->data), h->token_stride, h->head_stride}; }

Params params_of(const nvfp4_attention_shape* s, uint32_t* dev_status) {
    Params p = {};
    p.tq = s->tq;
    p.tk = s->tk;
    p.heads = s->heads;
    p.kv_heads = s->kv_heads;
    p.dim = s->dim;
    p.causal = s->causal != 0;
    p.nseq = s->nseq;
    p.scale = s->scale;
    p.cu_q = s->cu_q;
    p.cu_k = s->cu_k;
    p.dev_status = dev_status;
    return p;
}

}  // namespace attn
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_attention_forward(const nvfp4_attention_shape* shape, const nvfp4_heads* q,
                                                const nvfp4_heads* k, const nvfp4_heads* v, const nvfp4_heads* out,
                                                float* lse, uint32_t* dev_status, void* stream) {
    using namespace attn;
    nvfp4_status st = check_shape(shape);
    if (st == NVFP4_OK) st = check_heads(q, shape->tq, shape->heads, shape->dim);
    if (st == NVFP4_OK) st = check_heads(k, shape->tk, shape->kv_heads, shape->dim);
    if (st == NVFP4_OK) st = check_heads(v, shape->tk, shape->kv_heads, shape->dim);
    if (st == NVFP4_OK) st = check_heads(out, shape->tq, shape->heads, shape->dim);
    if (st != NVFP4_OK) return st;
    if (shape->tq == 0) return NVFP4_OK;
    if (!lse) return NVFP4_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(lse) % 4) return NVFP4_ERR_ALIGNMENT;
    Params p = params_of(shape, dev_status);
    p.q = heads_of(q);
    p.k = heads_of(k);
    p.v = heads_of(v);
    p.out = heads_of(out);
    p.lse = lse;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (p.cu_q) e = launch_pdl(check_offsets_kernel, dim3(1), dim3(256), 0, s, p);
    if (e == cudaSuccess)
        e = launch_pdl(fwd_kernel, dim3((unsigned)((p.tq + 7) / 8), p.heads), dim3(256), 0, s, p);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

extern "C" size_t nvfp4_attention_backward_workspace_bytes(const nvfp4_attention_shape* shape) {
    if (attn::check_shape(shape) != NVFP4_OK) return 0;
    return (size_t)shape->heads * (size_t)std::max<int64_t>(shape->tq, 4) * sizeof(float);
}

extern "C" nvfp4_status nvfp4_attention_backward(const nvfp4_attention_shape* shape, const nvfp4_heads* dout,
                                                 const nvfp4_heads* q, const nvfp4_heads* k, const nvfp4_heads* v,
                                                 const nvfp4_heads* out, const float* lse, const nvfp4_heads* dq,
                                                 const nvfp4_heads* dk, const nvfp4_heads* dv, void* workspace,
                                                 size_t workspace_bytes, uint32_t* dev_status, void* stream) {
    using namespace attn;
    nvfp4_status st = check_shape(shape);
    if (st != NVFP4_OK) return st;
    for (const nvfp4_heads* h : {dout, q, out, dq})
        if ((st = check_heads(h, shape->tq, shape->heads, shape->dim)) != NVFP4_OK) return st;
    for (const nvfp4_heads* h : {k, v, dk, dv})
        if ((st = check_heads(h, shape->tk, shape->kv_heads, shape->dim)) != NVFP4_OK) return st;
    if (shape->tq > 0 && !lse) return NVFP4_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(lse) % 4) return NVFP4_ERR_ALIGNMENT;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < nvfp4_attention_backward_workspace_bytes(shape))
        return NVFP4_ERR_WORKSPACE;
    Params p = params_of(shape, dev_status);
    p.q = heads_of(q);
    p.k = heads_of(k);
    p.v = heads_of(v);
    p.out = heads_of(out);
    p.dout = heads_of(dout);
    p.dq = heads_of(dq);
    p.dk = heads_of(dk);
    p.dv = heads_of(dv);
    p.lse = const_cast<float*>(lse);
    p.delta = static_cast<float*>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (p.cu_q) e = launch_pdl(check_offsets_kernel, dim3(1), dim3(256), 0, s, p);
    if (e == cudaSuccess && p.tq > 0)
        e = launch_pdl(bwd_dq_kernel, dim3((unsigned)((p.tq + 7) / 8), p.heads), dim3(256), 0, s, p);
    if (e == cudaSuccess && p.tk > 0)
        e = launch_pdl(bwd_dkv_kernel, dim3((unsigned)((p.tk + 7) / 8), p.kv_heads), dim3(256), 0, s, p);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
