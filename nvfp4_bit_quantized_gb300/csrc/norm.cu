// norm.cu -- layer norm over the rows of an activation, forward and backward (include/nvfp4.h has
// the formulas).  Statistics and sums are fp32.
//
// Both passes are bound by memory: x (and the residual) in and y (and h) out forward, dy, x (and dh)
// in and dx out backward, each once.  A row's values stay in registers between the loads, the
// statistics (mean first, then the squares about it) and the stores.  A thread holds NC chunks of E
// neighbouring elements: E = 8 with 16-byte accesses, E = 1 where a pointer, a pitch or the width does
// not allow them.
//   narrow rows: a group of G lanes takes a row, a warp 32 / G of them at a time;
//   others: a block takes a row, blocks stay for many rows, and each thread copies its own chunks of the next
//     rows to shared memory ahead (cp.async): the bytes in flight do not depend on how long a row's
//     two sums and their barriers take.  It waits for its own copies only;
//   rows too long for the registers go through the loops at the end, which read them again from the
//     caches.
//
// Backward, a block keeps the column sums of dy * xhat and dy for its columns in registers over all its
// rows and writes them once; a second kernel joins the blocks' parts in a fixed order (no atomics).
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cmath>
#include <cstdint>

#include "device_common.cuh"
#include "host_common.h"

namespace nvfp4 {
namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ float round_to(float v, const float*) { return v; }
__device__ __forceinline__ float round_to(float v, const bf16*) { return __bfloat162float(__float2bfloat16_rn(v)); }

// 16 bytes that are read once (they may be written in place later: not through the read-only path).
__device__ __forceinline__ uint4 ld16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// A chunk of E elements as it lies in memory.
template <typename T, int E> struct Chunk;
template <typename T> struct Chunk<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = load1(&v); }
    __device__ __forceinline__ static void put(T* p, const float (&f)[1]) { store1(p, f[0]); }
};
template <> struct Chunk<bf16, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const bf16* p) { v = ld16(p); }
    __device__ __forceinline__ void get(float (&f)[8]) const { Vec<uint16_t>::unpack(v, f); }
    __device__ __forceinline__ static void put(bf16* p, const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Chunk<float, 8> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = ld16(p);
        b = ld16(p + 4);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        Vec<float>::unpack(a, f);
        Vec<float>::unpack(b, f + 4);
    }
    __device__ __forceinline__ static void put(float* p, const float (&f)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// E elements of a weight or bias vector of either type, kept in the caches.
template <int E>
__device__ __forceinline__ void load_vec(const void* w, bool f32, int64_t at, float (&f)[E]) {
    if constexpr (E == 1) {
        f[0] = f32 ? __ldg(static_cast<const float*>(w) + at) : __bfloat162float(__ldg(static_cast<const bf16*>(w) + at));
    } else if (f32) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(w) + at);
        Vec<float>::unpack(__ldg(p), f);
        Vec<float>::unpack(__ldg(p + 1), f + 4);
    } else {
        Vec<uint16_t>::unpack(__ldg(reinterpret_cast<const uint4*>(static_cast<const bf16*>(w) + at)), f);
    }
}

// Elementwise on E values, two at a time (packed fp32) where there are pairs.
template <int E> __device__ __forceinline__ void vadd(float (&a)[E], const float (&b)[E]) {
    if constexpr (E == 1) a[0] += b[0];
    else
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 r = __fadd2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
            a[e] = r.x;
            a[e + 1] = r.y;
        }
}
template <int E> __device__ __forceinline__ void vadd(float (&a)[E], float b) {
    if constexpr (E == 1) a[0] += b;
    else
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 r = __fadd2_rn(make_float2(a[e], a[e + 1]), make_float2(b, b));
            a[e] = r.x;
            a[e + 1] = r.y;
        }
}
template <int E> __device__ __forceinline__ void vmul(float (&a)[E], const float (&b)[E]) {
    if constexpr (E == 1) a[0] *= b[0];
    else
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 r = __fmul2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
            a[e] = r.x;
            a[e + 1] = r.y;
        }
}
template <int E> __device__ __forceinline__ void vmul(float (&a)[E], float b) {
    if constexpr (E == 1) a[0] *= b;
    else
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 r = __fmul2_rn(make_float2(a[e], a[e + 1]), make_float2(b, b));
            a[e] = r.x;
            a[e + 1] = r.y;
        }
}
// a = b * c + d
template <int E>
__device__ __forceinline__ void vfma(float (&a)[E], const float (&b)[E], const float (&c)[E], const float (&d)[E]) {
    if constexpr (E == 1) a[0] = fmaf(b[0], c[0], d[0]);
    else
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 r = __ffma2_rn(make_float2(b[e], b[e + 1]), make_float2(c[e], c[e + 1]), make_float2(d[e], d[e + 1]));
            a[e] = r.x;
            a[e + 1] = r.y;
        }
}
template <int E> __device__ __forceinline__ void vfma(float (&a)[E], const float (&b)[E], float c, const float (&d)[E]) {
    if constexpr (E == 1) a[0] = fmaf(b[0], c, d[0]);
    else
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 r = __ffma2_rn(make_float2(b[e], b[e + 1]), make_float2(c, c), make_float2(d[e], d[e + 1]));
            a[e] = r.x;
            a[e + 1] = r.y;
        }
}
template <int E> __device__ __forceinline__ float vsum(const float (&a)[E]) {
    if constexpr (E == 1) return a[0];
    else {
        float2 s = make_float2(a[0], a[1]);
#pragma unroll
        for (int e = 2; e < E; e += 2) s = __fadd2_rn(s, make_float2(a[e], a[e + 1]));
        return s.x + s.y;
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    return v;
}

// The sum over a block's threads, through `red` (16 floats, 16-byte aligned; each call of a row its own).  At most 16 warps;
// `red` holds zeros for those that there are not.
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const float4* q = reinterpret_cast<const float4*>(red);
    const float4 a = q[0], b = q[1], c = q[2], d = q[3];
    return ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w)) + (((c.x + c.y) + (c.z + c.w)) + ((d.x + d.y) + (d.z + d.w)));
}

// One chunk's copy to this thread's own place in shared memory.
template <typename T, int E>
__device__ __forceinline__ void copy_chunk(Chunk<T, E>* dst, const T* src) {
    constexpr int kBytes = sizeof(T) * E;
    const uint32_t d = smem_addr(dst);
    if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes; i += 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                         :: "r"(d + i), "l"(reinterpret_cast<const char*>(src) + i) : "memory");
    } else if constexpr (kBytes == 4) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(d), "l"(src) : "memory");
    } else {
        dst->v = *src;                                     // two bytes: there is no such copy
    }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// The sum over the G (a power of two) neighbouring lanes of a group.
__device__ __forceinline__ float group_sum(float v, int G) {
    for (int d = G >> 1; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    return v;
}

struct FwdParams {
    const void *x, *residual, *weight, *bias;
    void *y, *h;
    float *mean, *rstd;
    int64_t rows, cols, ldx, ldr, ldy, ldh;
    float eps;
    int w_f32;
};

// One row's arithmetic after the loads: v (h, or x) in, y's values out; mean and rstd.  `here[i]`: whether the thread has
// chunk i (its v is 0 where not).  Sum: the sum over the row's threads.
template <int E, int NC, typename Sum>
__device__ __forceinline__ void norm_row(float (&v)[NC][E], const bool (&here)[NC], const float (&w)[NC][E],
                                         const float (&b)[NC][E], float inv_cols, float eps, float& mean, float& rstd,
                                         Sum&& sum) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) s += vsum(v[i]);
    mean = sum(s, 0) * inv_cols;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        float q[E] = {};
        vadd(v[i], -mean);
        vfma(q, v[i], v[i], q);
        s += here[i] ? vsum(q) : 0.0f;
    }
    rstd = rsqrtf(sum(s, 1) * inv_cols + eps);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        vmul(v[i], rstd);
        vfma(v[i], v[i], w[i], b[i]);
    }
}
template <typename X, int E>
__device__ __forceinline__ void add_residual(const Chunk<X, E>& c, float (&v)[E], X* h) {
    float a[E];
    c.get(a);
    vadd(v, a);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = round_to(v[e], static_cast<const X*>(nullptr));
    Chunk<X, E>::put(h, v);
}
// The thread's chunks of weight and bias (zeros without one, and where it has no chunk).
template <int E, int NC>
__device__ __forceinline__ void load_affine(const FwdParams& p, const bool (&here)[NC], int t, int width, float (&w)[NC][E],
                                            float (&b)[NC][E]) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
#pragma unroll
        for (int e = 0; e < E; ++e) w[i][e] = b[i][e] = 0.0f;
        if (here[i]) {
            load_vec<E>(p.weight, p.w_f32, (t + i * width) * E, w[i]);
            if (p.bias) load_vec<E>(p.bias, p.w_f32, (t + i * width) * E, b[i]);
        }
    }
}

// Groups of G lanes, U rows of a group at a time.
template <typename X, typename Y, int E, int NC, int U>
__global__ void __launch_bounds__(128, NC * E > 16 ? 3 : 4) norm_fwd_warp_kernel(FwdParams p, int G) {
    pdl_launch_dependents();
    pdl_wait();
    const int t = threadIdx.x & (G - 1), chunks = (int)(p.cols / E);
    const int64_t groups = gridDim.x * (int64_t)(128 / G);
    const float inv_cols = 1.0f / (float)p.cols;
    bool here[NC];
    float w[NC][E], b[NC][E];
#pragma unroll
    for (int i = 0; i < NC; ++i) here[i] = t + i * G < chunks;
    load_affine<E, NC>(p, here, t, G, w, b);
    // whole warps stay together (the sums are shuffles): the loop's bounds are the warp's first group's
    const int64_t mine = blockIdx.x * (int64_t)(128 / G) + threadIdx.x / G, lead = mine - (threadIdx.x & 31) / G;
    for (int64_t base = 0; lead + base < p.rows; base += U * groups) {
        Chunk<X, E> in[U][NC], add[U][NC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = mine + base + u * groups;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (r < p.rows && here[i]) {
                    in[u][i].load(static_cast<const X*>(p.x) + r * p.ldx + (t + i * G) * E);
                    if (p.residual) add[u][i].load(static_cast<const X*>(p.residual) + r * p.ldr + (t + i * G) * E);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = mine + base + u * groups;
            float v[NC][E] = {}, mean, rstd;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (r < p.rows && here[i]) {
                    in[u][i].get(v[i]);
                    if (p.residual) add_residual(add[u][i], v[i], static_cast<X*>(p.h) + r * p.ldh + (t + i * G) * E);
                }
            norm_row(v, here, w, b, inv_cols, p.eps, mean, rstd, [&](float s, int) { return group_sum(s, G); });
            if (r < p.rows) {
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (here[i]) Chunk<Y, E>::put(static_cast<Y*>(p.y) + r * p.ldy + (t + i * G) * E, v[i]);
                if (t == 0) {
                    p.mean[r] = mean;
                    p.rstd[r] = rstd;
                }
            }
        }
    }
}

// A block per row, S rows of copies: S - 1 ahead.  Shared memory: [S][x, residual][NC][threads] chunks.
template <typename X, typename Y, int E, int NC, int S, bool RES>
__global__ void __maxnreg__(96) norm_fwd_kernel(FwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ __align__(16) uint8_t norm_smem[];
    __shared__ __align__(16) float red[2][16];
    constexpr int A = RES ? 2 : 1;
    const int t = threadIdx.x, width = blockDim.x;
    Chunk<X, E>* ring = reinterpret_cast<Chunk<X, E>*>(norm_smem) + t;
    if (t < 32) red[t >> 4][t & 15] = 0.0f;
    __syncthreads();
    const float inv_cols = 1.0f / (float)p.cols;
    bool here[NC];
    float w[NC][E], b[NC][E];
#pragma unroll
    for (int i = 0; i < NC; ++i) here[i] = t + i * width < (int)(p.cols / E);
    load_affine<E, NC>(p, here, t, width, w, b);
    // this thread's first chunk of the row to fetch next, and of the row to store next
    const int64_t stride = gridDim.x, first = blockIdx.x;
    const X *x = static_cast<const X*>(p.x) + first * p.ldx + t * E, *res = static_cast<const X*>(p.residual) + first * p.ldr + t * E;
    X* h = static_cast<X*>(p.h) + first * p.ldh + t * E;
    Y* y = static_cast<Y*>(p.y) + first * p.ldy + t * E;
    const int64_t dx = stride * p.ldx, dres = stride * p.ldr, dh = stride * p.ldh, dy = stride * p.ldy;
    int64_t ahead = first;
    auto fetch = [&](int slot) {
        if (ahead < p.rows) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (here[i]) {
                    copy_chunk(ring + ((slot * A) * NC + i) * width, x + i * width * E);
                    if constexpr (RES) copy_chunk(ring + ((slot * A + 1) * NC + i) * width, res + i * width * E);
                }
        }
        copies_commit();
        ahead += stride;
        x += dx;
        if constexpr (RES) res += dres;
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fetch(k);
    int slot = 0;
    for (int64_t r = first; r < p.rows; r += stride) {
        fetch(slot == 0 ? S - 1 : slot - 1);
        copies_wait<S - 1>();
        float v[NC][E] = {}, mean, rstd;
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (here[i]) {
                ring[((slot * A) * NC + i) * width].get(v[i]);
                if constexpr (RES) add_residual(ring[((slot * A + 1) * NC + i) * width], v[i], h + i * width * E);
            }
        norm_row(v, here, w, b, inv_cols, p.eps, mean, rstd, [&](float s, int k) { return row_sum(s, red[k]); });
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (here[i]) Chunk<Y, E>::put(y + i * width * E, v[i]);
        if (t == 0) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
        y += dy;
        if constexpr (RES) h += dh;
        slot = slot + 1 == S ? 0 : slot + 1;
    }
}

struct BwdParams {
    const void *dy, *x, *weight, *dh;
    const float *mean, *rstd;
    void* dx;
    float *dweight, *dbias, *parts;
    int64_t rows, cols, lddy, ldx, lddh, lddx;
    int w_f32, nparts;
};

// One row of the backward pass after the loads: xhat = x and g = dy come in (0 where the thread has no chunk), dx
// without dh goes out in g, the column sums grow.  Sums: both over the row's threads.
template <int E, int NC, typename Sums>
__device__ __forceinline__ void grad_row(float (&xhat)[NC][E], float (&g)[NC][E], const float (&w)[NC][E],
                                         float (&sw)[NC][E], float (&sb)[NC][E], float mean, float rstd, float inv_cols,
                                         Sums&& sums) {
    float a[E] = {}, b[E] = {};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        vadd(xhat[i], -mean);
        vmul(xhat[i], rstd);
        vfma(sw[i], g[i], xhat[i], sw[i]);
        vadd(sb[i], g[i]);
        vmul(g[i], w[i]);
        vadd(a, g[i]);
        vfma(b, g[i], xhat[i], b);
    }
    float s1 = vsum(a), s2 = vsum(b);
    sums(s1, s2);
    s1 *= inv_cols;
    s2 *= inv_cols;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        vfma(g[i], xhat[i], -s2, g[i]);
        vadd(g[i], -s1);
        vmul(g[i], rstd);
    }
}

// Groups of G lanes, U rows of a group at a time.  Column sums of a block: parts[2 block] (dy xhat) and
// parts[2 block + 1] (dy), cols each.
template <typename X, typename Y, int E, int NC, int U>
__global__ void __launch_bounds__(128, 3) norm_bwd_warp_kernel(BwdParams p, int G) {
    pdl_launch_dependents();
    pdl_wait();
    const int t = threadIdx.x & (G - 1), chunks = (int)(p.cols / E);
    const int64_t groups = gridDim.x * (int64_t)(128 / G);
    const float inv_cols = 1.0f / (float)p.cols;
    float w[NC][E] = {}, sw[NC][E] = {}, sb[NC][E] = {};
#pragma unroll
    for (int i = 0; i < NC; ++i)
        if (t + i * G < chunks) load_vec<E>(p.weight, p.w_f32, (t + i * G) * E, w[i]);
    const int64_t mine = blockIdx.x * (int64_t)(128 / G) + threadIdx.x / G, lead = mine - (threadIdx.x & 31) / G;
    for (int64_t base = 0; lead + base < p.rows; base += U * groups) {
        Chunk<X, E> x[U][NC], dh[U][NC];
        Chunk<Y, E> dy[U][NC];
        float mean[U] = {}, rstd[U] = {};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = mine + base + u * groups;
            if (r < p.rows) {
                mean[u] = p.mean[r];
                rstd[u] = p.rstd[r];
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (t + i * G < chunks) {
                        x[u][i].load(static_cast<const X*>(p.x) + r * p.ldx + (t + i * G) * E);
                        dy[u][i].load(static_cast<const Y*>(p.dy) + r * p.lddy + (t + i * G) * E);
                        if (p.dh) dh[u][i].load(static_cast<const X*>(p.dh) + r * p.lddh + (t + i * G) * E);
                    }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = mine + base + u * groups;
            float xhat[NC][E] = {}, g[NC][E] = {};
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (r < p.rows && t + i * G < chunks) {
                    x[u][i].get(xhat[i]);
                    dy[u][i].get(g[i]);
                }
            grad_row(xhat, g, w, sw, sb, mean[u], rstd[u], inv_cols, [&](float& a, float& b) {
                a = group_sum(a, G);
                b = group_sum(b, G);
            });
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (r < p.rows && t + i * G < chunks) {
                    if (p.dh) {
                        float a[E];
                        dh[u][i].get(a);
#pragma unroll
                        for (int e = 0; e < E; ++e) g[i][e] += a[e];
                    }
                    Chunk<X, E>::put(static_cast<X*>(p.dx) + r * p.lddx + (t + i * G) * E, g[i]);
                }
        }
    }
    // the groups of a warp by shuffles, then the block's warps one after another, in order
    extern __shared__ __align__(16) uint8_t norm_smem[];
    float* sums = reinterpret_cast<float*>(norm_smem);     // 2 x cols
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e)
            for (int d = G; d < 32; d <<= 1) {
                sw[i][e] += __shfl_xor_sync(~0u, sw[i][e], d);
                sb[i][e] += __shfl_xor_sync(~0u, sb[i][e], d);
            }
    const int warp = threadIdx.x >> 5;
    for (int k = 0; k < 4; ++k) {
        if (warp == k && (threadIdx.x & 31) < G) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (t + i * G < chunks)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int c = (t + i * G) * E + e;
                        sums[c] = (k ? sums[c] : 0.0f) + sw[i][e];
                        sums[p.cols + c] = (k ? sums[p.cols + c] : 0.0f) + sb[i][e];
                    }
        }
        __syncthreads();
    }
    float* out = p.parts + 2 * (int64_t)blockIdx.x * p.cols;
    for (int c = threadIdx.x; c < 2 * (int)p.cols; c += 128) out[c] = sums[c];
}

// A block per row, S rows of copies.  Shared memory: [S][x, dy, dh][NC][threads] chunks.
template <typename X, typename Y, int E, int NC, int S, bool RES>
__global__ void __maxnreg__(96) norm_bwd_kernel(BwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ __align__(16) uint8_t norm_smem[];
    __shared__ __align__(16) float2 red[2][16];            // both sums of a row; two buffers take turns
    const int t = threadIdx.x, width = blockDim.x;
    if (t < 32) red[t >> 4][t & 15] = make_float2(0.0f, 0.0f);
    __syncthreads();
    const uint32_t xs = NC * width * sizeof(Chunk<X, E>), ys = NC * width * sizeof(Chunk<Y, E>);
    const uint32_t slot_bytes = xs + ys + (RES ? xs : 0);
    auto at_x = [&](uint32_t slot, int i) { return reinterpret_cast<Chunk<X, E>*>(norm_smem + slot) + i * width + t; };
    auto at_dy = [&](uint32_t slot, int i) { return reinterpret_cast<Chunk<Y, E>*>(norm_smem + slot + xs) + i * width + t; };
    auto at_dh = [&](uint32_t slot, int i) { return reinterpret_cast<Chunk<X, E>*>(norm_smem + slot + xs + ys) + i * width + t; };
    const float inv_cols = 1.0f / (float)p.cols;
    bool here[NC];
    float w[NC][E] = {}, sw[NC][E] = {}, sb[NC][E] = {};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        here[i] = t + i * width < (int)(p.cols / E);
        if (here[i]) load_vec<E>(p.weight, p.w_f32, (t + i * width) * E, w[i]);
    }
    const int64_t first = blockIdx.x, stride = gridDim.x;
    const X *x = static_cast<const X*>(p.x) + first * p.ldx + t * E, *dh = static_cast<const X*>(p.dh) + first * p.lddh + t * E;
    const Y* dy = static_cast<const Y*>(p.dy) + first * p.lddy + t * E;
    X* dx = static_cast<X*>(p.dx) + first * p.lddx + t * E;
    int64_t ahead = first;
    auto fetch = [&](uint32_t slot) {
        if (ahead < p.rows) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (here[i]) {
                    copy_chunk(at_x(slot, i), x + i * width * E);
                    copy_chunk(at_dy(slot, i), dy + i * width * E);
                    if constexpr (RES) copy_chunk(at_dh(slot, i), dh + i * width * E);
                }
        }
        copies_commit();
        ahead += stride;
        x += stride * p.ldx;
        dy += stride * p.lddy;
        if constexpr (RES) dh += stride * p.lddh;
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fetch(k * slot_bytes);
    float mean = 0.0f, rstd = 0.0f;
    if (first < p.rows) {
        mean = p.mean[first];
        rstd = p.rstd[first];
    }
    uint32_t slot = 0;
    int buf = 0;
    for (int64_t r = first; r < p.rows; r += stride, buf ^= 1) {
        fetch(slot == 0 ? (S - 1) * slot_bytes : slot - slot_bytes);
        copies_wait<S - 1>();
        const float m = mean, rs = rstd;
        if (r + stride < p.rows) {
            mean = p.mean[r + stride];
            rstd = p.rstd[r + stride];
        }
        float xhat[NC][E] = {}, g[NC][E] = {};
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (here[i]) {
                at_x(slot, i)->get(xhat[i]);
                at_dy(slot, i)->get(g[i]);
            }
        grad_row(xhat, g, w, sw, sb, m, rs, inv_cols, [&](float& a, float& b) {
            a = warp_sum(a);
            b = warp_sum(b);
            if ((t & 31) == 0) red[buf][t >> 5] = make_float2(a, b);
            __syncthreads();
            const float4* q = reinterpret_cast<const float4*>(red[buf]);
            float2 s[4] = {};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float4 v = q[k];
                s[k & 3] = __fadd2_rn(s[k & 3], __fadd2_rn(make_float2(v.x, v.y), make_float2(v.z, v.w)));
            }
            s[0] = __fadd2_rn(__fadd2_rn(s[0], s[1]), __fadd2_rn(s[2], s[3]));
            a = s[0].x;
            b = s[0].y;
        });
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (here[i]) {
                if constexpr (RES) {
                    float a[E];
                    at_dh(slot, i)->get(a);
                    vadd(g[i], a);
                }
                Chunk<X, E>::put(dx + i * width * E, g[i]);
            }
        dx += stride * p.lddx;
        slot = slot + slot_bytes == S * slot_bytes ? 0 : slot + slot_bytes;
    }
    float *pw = p.parts + 2 * (int64_t)blockIdx.x * p.cols + t * E, *pb = pw + p.cols;
#pragma unroll
    for (int i = 0; i < NC; ++i)
        if (here[i]) {
            Chunk<float, E>::put(pw + i * width * E, sw[i]);
            Chunk<float, E>::put(pb + i * width * E, sb[i]);
        }
}

// dweight and dbias from the parts: a block takes 32 of the 2 cols columns, its warps every eighth part.
__global__ void __launch_bounds__(256) norm_bwd_join_kernel(BwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = blockIdx.x * 32ll + lane;
    float s = 0.0f;
    if (c < 2 * p.cols) {
        // a part's two rows follow one another: column c of 2 cols
        const float* q = p.parts + c;
        int i = warp;
        for (; i + 24 < p.nparts; i += 32) {
            const float a = q[2 * (int64_t)i * p.cols], b = q[2 * (int64_t)(i + 8) * p.cols];
            const float d = q[2 * (int64_t)(i + 16) * p.cols], e = q[2 * (int64_t)(i + 24) * p.cols];
            s += (a + b) + (d + e);
        }
        for (; i < p.nparts; i += 8) s += q[2 * (int64_t)i * p.cols];
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < 2 * p.cols) {
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += red[k][lane];
        if (c < p.cols) p.dweight[c] = s;
        else if (p.dbias) p.dbias[c - p.cols] = s;
    }
}

// ---- rows too long for registers: a block per row, in loops over the row
constexpr int kLoopThreads = 512;

template <typename X, typename Y, int E>
__global__ void __launch_bounds__(kLoopThreads) norm_fwd_loop_kernel(FwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ __align__(16) float red[2][16];             // kLoopThreads has all 16 warps
    const float inv_cols = 1.0f / (float)p.cols;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const X* x = static_cast<const X*>(p.x) + r * p.ldx;
        const X* res = p.residual ? static_cast<const X*>(p.residual) + r * p.ldr : nullptr;
        X* h = p.h ? static_cast<X*>(p.h) + r * p.ldh : nullptr;
        const X* src = res ? h : x;
        Chunk<X, E> in;
        float v[E], a[E], s = 0.0f;
        for (int64_t c = threadIdx.x * E; c < p.cols; c += kLoopThreads * E) {
            in.load(x + c);
            in.get(v);
            if (res) {
                in.load(res + c);
                in.get(a);
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = round_to(v[e] + a[e], x);
                Chunk<X, E>::put(h + c, v);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) s += v[e];
        }
        const float mean = row_sum(s, red[0]) * inv_cols;
        s = 0.0f;
        for (int64_t c = threadIdx.x * E; c < p.cols; c += kLoopThreads * E) {
            in.load(src + c);
            in.get(v);
#pragma unroll
            for (int e = 0; e < E; ++e) s = fmaf(v[e] - mean, v[e] - mean, s);
        }
        const float rstd = rsqrtf(row_sum(s, red[1]) * inv_cols + p.eps);
        Y* y = static_cast<Y*>(p.y) + r * p.ldy;
        for (int64_t c = threadIdx.x * E; c < p.cols; c += kLoopThreads * E) {
            in.load(src + c);
            in.get(v);
            load_vec<E>(p.weight, p.w_f32, c, a);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = (v[e] - mean) * rstd * a[e];
            if (p.bias) {
                load_vec<E>(p.bias, p.w_f32, c, a);
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] += a[e];
            }
            Chunk<Y, E>::put(y + c, v);
        }
        if (threadIdx.x == 0) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
    }
}

// Column sums of one slice of rows: a thread takes a chunk of columns, blockIdx.y the slice.
template <typename X, typename Y, int E>
__global__ void __launch_bounds__(kLoopThreads) norm_bwd_cols_loop_kernel(BwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t c = (blockIdx.x * (int64_t)kLoopThreads + threadIdx.x) * E;
    if (c >= p.cols) return;
    const int64_t r0 = p.rows * blockIdx.y / p.nparts, r1 = p.rows * (blockIdx.y + 1) / p.nparts;
    float sw[E] = {}, sb[E] = {};
    for (int64_t r = r0; r < r1; ++r) {
        Chunk<Y, E> dy;
        Chunk<X, E> x;
        float g[E], v[E];
        dy.load(static_cast<const Y*>(p.dy) + r * p.lddy + c);
        x.load(static_cast<const X*>(p.x) + r * p.ldx + c);
        dy.get(g);
        x.get(v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            sw[e] = fmaf(g[e], (v[e] - p.mean[r]) * p.rstd[r], sw[e]);
            sb[e] += g[e];
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        p.parts[(2 * (int64_t)blockIdx.y) * p.cols + c + e] = sw[e];
        p.parts[(2 * (int64_t)blockIdx.y + 1) * p.cols + c + e] = sb[e];
    }
}

template <typename X, typename Y, int E>
__global__ void __launch_bounds__(kLoopThreads) norm_bwd_rows_loop_kernel(BwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ __align__(16) float red[2][16];             // kLoopThreads has all 16 warps
    const float inv_cols = 1.0f / (float)p.cols;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const X* x = static_cast<const X*>(p.x) + r * p.ldx;
        const Y* dy = static_cast<const Y*>(p.dy) + r * p.lddy;
        const X* dh = p.dh ? static_cast<const X*>(p.dh) + r * p.lddh : nullptr;
        X* dx = static_cast<X*>(p.dx) + r * p.lddx;
        const float mean = p.mean[r], rstd = p.rstd[r];
        Chunk<X, E> in;
        Chunk<Y, E> dyc;
        float s1 = 0.0f, s2 = 0.0f, w[E], g[E], v[E];
        for (int64_t c = threadIdx.x * E; c < p.cols; c += kLoopThreads * E) {
            in.load(x + c);
            dyc.load(dy + c);
            load_vec<E>(p.weight, p.w_f32, c, w);
            in.get(v);
            dyc.get(g);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s1 = fmaf(g[e], w[e], s1);
                s2 = fmaf(g[e] * w[e], (v[e] - mean) * rstd, s2);
            }
        }
        s1 = row_sum(s1, red[0]) * inv_cols;
        s2 = row_sum(s2, red[1]) * inv_cols;
        for (int64_t c = threadIdx.x * E; c < p.cols; c += kLoopThreads * E) {
            in.load(x + c);
            dyc.load(dy + c);
            load_vec<E>(p.weight, p.w_f32, c, w);
            in.get(v);
            dyc.get(g);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = rstd * (g[e] * w[e] - s1 - (v[e] - mean) * rstd * s2);
            if (dh) {
                in.load(dh + c);
                in.get(w);
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] += w[e];
            }
            Chunk<X, E>::put(dx + c, v);
        }
    }
}

// ---- host
template <typename T> struct Tag { using type = T; };
template <typename F>
nvfp4_status with_types(int32_t x, int32_t y, F&& f) {
    auto on_y = [&](auto tx) { return y == NVFP4_F32 ? f(tx, Tag<float>{}) : f(tx, Tag<bf16>{}); };
    return x == NVFP4_F32 ? on_y(Tag<float>{}) : on_y(Tag<bf16>{});
}

bool known(int32_t t) { return t == NVFP4_F32 || t == NVFP4_BF16; }
bool aligned_to(const void* p, int32_t t) { return reinterpret_cast<uintptr_t>(p) % (t == NVFP4_F32 ? 4 : 2) == 0; }
nvfp4_status to_status(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

// Rows (base and pitch in elements) that can be read 8 elements at a time.
bool rows16(const void* p, int64_t ld) { return !p || (aligned16(p) && ld % 8 == 0); }

constexpr int kBlock = 512;                    // the most threads of a row
constexpr int kNarrow = 128;                   // threads of a block of narrow rows
constexpr int kRingBytes = 100 * 1024;         // shared memory of a block's copies: two blocks on an SM

int sms() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? std::max(1, sm_count(dev)) : 1;
}
int block_threads(int64_t chunks, int nc) { return (int)((chunks + nc * 32 - 1) / (nc * 32)) * 32; }
// Lanes of a group: all the row's chunks at once where that is at most a warp, else a warp.
int group_lanes(int64_t chunks) {
    int g = 1;
    while (g < 32 && g < chunks) g *= 2;
    return g;
}
// Blocks of a persistent grid: as many as run at once, by registers (96 a thread) and shared memory.
int64_t resident_blocks(int threads, size_t smem) {
    return sms() * std::max<int64_t>(1, std::min<int64_t>(65536 / (96 * threads), 224 * 1024 / (smem + 1024)));
}
template <typename Kernel, typename P>
cudaError_t launch_ring(Kernel kern, int64_t grid, int threads, size_t smem, cudaStream_t s, const P& p) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    return e == cudaSuccess ? launch_pdl(kern, dim3((unsigned)grid), dim3(threads), smem, s, p) : e;
}

// How the backward pass cuts the rows.  Rows wider than its registers reach go through the loops.
struct BwdPlan {
    enum { kWarp, kBlock, kLoop } kind;
    int threads, stages, parts;
    size_t smem;
};
BwdPlan bwd_plan(int64_t rows, int64_t cols, bool vec, size_t row_elem_bytes) {
    const int64_t chunks = vec ? cols / 8 : cols;
    const int nc = vec ? 2 : 8;
    BwdPlan b = {};
    int64_t parts;
    if (chunks <= 32 * nc) {
        const int g = group_lanes(chunks);
        b.kind = BwdPlan::kWarp;
        b.threads = kNarrow;
        b.smem = 2 * (size_t)cols * sizeof(float);
        parts = std::min<int64_t>((rows + kNarrow / g - 1) / (kNarrow / g), sms() * 4ll);
    } else if (chunks <= kBlock * nc) {
        b.kind = BwdPlan::kBlock;
        b.threads = block_threads(chunks, nc);
        const size_t slot = (size_t)b.threads * nc * (vec ? 8 : 1) * row_elem_bytes;
        b.stages = 3 * slot <= kRingBytes ? 3 : 2;
        b.smem = b.stages * slot;
        parts = std::min<int64_t>(rows, resident_blocks(b.threads, b.smem));
    } else {
        b.kind = BwdPlan::kLoop;
        b.threads = kLoopThreads;
        parts = std::min<int64_t>(64, rows / 16);
    }
    b.parts = (int)std::max<int64_t>(1, parts);
    return b;
}

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
    const FwdParams p{x, residual, weight, bias, y, h, mean, rstd, rows, cols, ldx, ldr, ldy, ldh, eps, w_dtype == NVFP4_F32};
    const bool vec = cols % 8 == 0 && rows16(x, ldx) && rows16(residual, ldr) && rows16(h, ldh) && rows16(y, ldy) &&
                     aligned16(weight) && aligned16(bias);
    const int64_t chunks = vec ? cols / 8 : cols;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return with_types(x_dtype, y_dtype, [&](auto tx, auto ty) {
        using X = typename decltype(tx)::type;
        using Y = typename decltype(ty)::type;
        auto narrow = [&](auto kern) {
            const int g = group_lanes(chunks);
            const int64_t grid = std::min<int64_t>((rows + kNarrow / g - 1) / (kNarrow / g), sms() * 16ll);
            return to_status(launch_pdl(kern, dim3((unsigned)grid), dim3(kNarrow), 0, s, p, g));
        };
        auto wide = [&](auto plain4, auto plain2, auto res4, auto res2, int nc, int e) {
            const int threads = block_threads(chunks, nc);
            const size_t slot = (size_t)threads * nc * e * sizeof(X) * (residual ? 2 : 1);
            const int stages = 4 * slot <= kRingBytes ? 4 : 2;
            const int64_t grid = std::min<int64_t>(rows, resident_blocks(threads, stages * slot));
            return to_status(launch_ring(residual ? (stages == 4 ? res4 : res2) : (stages == 4 ? plain4 : plain2), grid, threads,
                                         stages * slot, s, p));
        };
        if (vec) {
            if (chunks <= 32) return narrow(norm_fwd_warp_kernel<X, Y, 8, 1, 4>);
            if (chunks <= 64) return narrow(norm_fwd_warp_kernel<X, Y, 8, 2, 2>);
            if (chunks <= 128) return narrow(norm_fwd_warp_kernel<X, Y, 8, 4, 1>);
            if (chunks <= kBlock * 2) return wide(norm_fwd_kernel<X, Y, 8, 2, 4, false>, norm_fwd_kernel<X, Y, 8, 2, 2, false>, norm_fwd_kernel<X, Y, 8, 2, 4, true>, norm_fwd_kernel<X, Y, 8, 2, 2, true>, 2, 8);
            // 16384 fp32 columns with a residual: two rows of copies do not fit
            if (chunks <= kBlock * 4 && 2 * cols * sizeof(X) * (residual ? 2 : 1) <= 216 * 1024)
                return wide(norm_fwd_kernel<X, Y, 8, 4, 4, false>, norm_fwd_kernel<X, Y, 8, 4, 2, false>, norm_fwd_kernel<X, Y, 8, 4, 4, true>, norm_fwd_kernel<X, Y, 8, 4, 2, true>, 4, 8);
            return to_status(launch_pdl(norm_fwd_loop_kernel<X, Y, 8>, dim3((unsigned)std::min<int64_t>(rows, 1 << 30)),
                                        dim3(kLoopThreads), 0, s, p));
        }
        if (chunks <= 32 * 8) return narrow(norm_fwd_warp_kernel<X, Y, 1, 8, 2>);
        if (chunks <= kBlock * 8) return wide(norm_fwd_kernel<X, Y, 1, 8, 4, false>, norm_fwd_kernel<X, Y, 1, 8, 2, false>, norm_fwd_kernel<X, Y, 1, 8, 4, true>, norm_fwd_kernel<X, Y, 1, 8, 2, true>, 8, 1);
        return to_status(launch_pdl(norm_fwd_loop_kernel<X, Y, 1>, dim3((unsigned)std::min<int64_t>(rows, 1 << 30)),
                                    dim3(kLoopThreads), 0, s, p));
    });
}

extern "C" size_t nvfp4_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1 || cols > (1ll << 30)) return 0;
    // whatever the types and the alignment turn out to be
    int parts = 0;
    for (size_t bytes = 4; bytes <= 12; bytes += 2)
        parts = std::max({parts, bwd_plan(rows, cols, false, bytes).parts, cols % 8 ? 0 : bwd_plan(rows, cols, true, bytes).parts});
    return (size_t)parts * 2 * (size_t)cols * sizeof(float);
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
    const bool vec = cols % 8 == 0 && rows16(x, ldx) && rows16(dy, lddy) && rows16(dh, lddh) && rows16(dx, lddx) &&
                     aligned16(weight);
    const size_t xb = x_dtype == NVFP4_F32 ? 4 : 2, yb = y_dtype == NVFP4_F32 ? 4 : 2;
    const BwdPlan plan = bwd_plan(rows, cols, vec, xb * (dh ? 2 : 1) + yb);
    const BwdParams p{dy,   x,    weight, dh,  mean, rstd, dx,   dweight, dbias, static_cast<float*>(workspace),
                      rows, cols, lddy,   ldx, lddh, lddx, w_dtype == NVFP4_F32, plan.parts};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return with_types(x_dtype, y_dtype, [&](auto tx, auto ty) {
        using X = typename decltype(tx)::type;
        using Y = typename decltype(ty)::type;
        cudaError_t e;
        const dim3 grid(plan.parts), block(plan.threads);
        if (plan.kind == BwdPlan::kWarp) {
            const int g = group_lanes(vec ? cols / 8 : cols);
            if (!vec) e = launch_pdl(norm_bwd_warp_kernel<X, Y, 1, 8, 1>, grid, block, plan.smem, s, p, g);
            else if (cols <= 256) e = launch_pdl(norm_bwd_warp_kernel<X, Y, 8, 1, 2>, grid, block, plan.smem, s, p, g);
            else e = launch_pdl(norm_bwd_warp_kernel<X, Y, 8, 2, 1>, grid, block, plan.smem, s, p, g);
        } else if (plan.kind == BwdPlan::kBlock) {
            auto wide = [&](auto plain3, auto plain2, auto res3, auto res2) {
                e = launch_ring(dh ? (plan.stages == 3 ? res3 : res2) : (plan.stages == 3 ? plain3 : plain2), plan.parts,
                                plan.threads, plan.smem, s, p);
            };
            if (vec) wide(norm_bwd_kernel<X, Y, 8, 2, 3, false>, norm_bwd_kernel<X, Y, 8, 2, 2, false>,
                          norm_bwd_kernel<X, Y, 8, 2, 3, true>, norm_bwd_kernel<X, Y, 8, 2, 2, true>);
            else wide(norm_bwd_kernel<X, Y, 1, 8, 3, false>, norm_bwd_kernel<X, Y, 1, 8, 2, false>,
                      norm_bwd_kernel<X, Y, 1, 8, 3, true>, norm_bwd_kernel<X, Y, 1, 8, 2, true>);
        } else {
            auto loops = [&](auto cols_kern, auto rows_kern, int per) {
                const dim3 cut((unsigned)((cols / per + kLoopThreads - 1) / kLoopThreads), plan.parts);
                e = launch_pdl(cols_kern, cut, block, 0, s, p);
                if (e == cudaSuccess && rows > 0)
                    e = launch_pdl(rows_kern, dim3((unsigned)std::min<int64_t>(rows, 1 << 30)), block, 0, s, p);
            };
            if (vec) loops(norm_bwd_cols_loop_kernel<X, Y, 8>, norm_bwd_rows_loop_kernel<X, Y, 8>, 8);
            else loops(norm_bwd_cols_loop_kernel<X, Y, 1>, norm_bwd_rows_loop_kernel<X, Y, 1>, 1);
        }
        if (e == cudaSuccess)
            e = launch_pdl(norm_bwd_join_kernel, dim3((unsigned)((2 * cols + 31) / 32)), dim3(256), 0, s, p);
        return to_status(e);
    });
}
