// norm.cu -- layer norm over the rows of an activation, forward and backward (include/nvfp4.h has
// the formulas).  Statistics and sums are fp32.
//
// Both passes are bound by memory: x (and the residual) in and y (and h) out forward, dy, x (and dh)
// in and dx out backward, each once up to the widths that registers hold.  A row's values stay there between the
// loads, the statistics (mean first, then the squares about it) and the stores.  A thread holds NC chunks of E
// neighbouring elements: E = 8 with 16-byte accesses, E = 1 where a pointer, a pitch or the width does
// not allow them.
//   narrow rows: a group of G lanes takes a row, a warp 32 / G of them at a time;
//   others: a block takes a row, blocks stay for many rows, and each thread copies its own chunks of the next
//     rows to shared memory ahead (cp.async): the bytes in flight do not depend on how long a row's
//     two sums and their barriers take.  It waits for its own copies only.  Single bf16 elements, too small for
//     such copies, are loaded and stored there one after another: 4099 x 5121 takes 71 us forward and 93 backward, fp32
//     rows of twice the bytes 46 and 81;
//   rows too long for the registers (forward past 16384 columns, backward and single elements past 8192) go through the
//     loops at the end, which read them two or three times, in part from the caches: 2048 x 20480 bf16 62 us
//     forward, 124 backward.
//
// Backward, a block keeps the column sums of dy * xhat and dy for its columns in registers over all its
// rows and writes them once; a second kernel joins the blocks' parts in a fixed order (no atomics).
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

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
    __device__ __forceinline__ void store(T* p) const { *p = v; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = load1(&v); }
    __device__ __forceinline__ void set(const float (&f)[1]) { store1(&v, f[0]); }
    __device__ __forceinline__ static void put(T* p, const float (&f)[1]) { store1(p, f[0]); }
};
template <> struct Chunk<bf16, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const bf16* p) { v = ld16(p); }
    __device__ __forceinline__ void store(bf16* p) const { *reinterpret_cast<uint4*>(p) = v; }
    __device__ __forceinline__ void get(float (&f)[8]) const { Vec<uint16_t>::unpack(v, f); }
    __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&b);
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        v = make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7]));
    }
    __device__ __forceinline__ static void put(bf16* p, const float (&f)[8]) {
        Chunk c;
        c.set(f);
        c.store(p);
    }
};
template <> struct Chunk<float, 8> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = ld16(p);
        b = ld16(p + 4);
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<uint4*>(p)[0] = a;
        reinterpret_cast<uint4*>(p)[1] = b;
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        Vec<float>::unpack(a, f);
        Vec<float>::unpack(b, f + 4);
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
    }
    __device__ __forceinline__ static void put(float* p, const float (&f)[8]) {
        Chunk c;
        c.set(f);
        c.store(p);
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

// The sums of N (a power of two) values over the threads of a block, in all of them; `red`: 32 N floats, of their own
// for consecutive calls.  A warp adds N values together: at each of the first steps a lane gives away half of those
// it still has, so that N values take 4 + N steps or so and not 5 N.
template <int N>
__device__ __forceinline__ float scatter_sum(float (&v)[N]) {
    const int lane = threadIdx.x & 31;
    int d = 16;
#pragma unroll
    for (int n = N / 2; n; n /= 2, d /= 2) {
        const bool up = lane & d;
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float give = up ? v[k] : v[k + n], keep = up ? v[k + n] : v[k];
            v[k] = keep + __shfl_xor_sync(~0u, give, d);
        }
    }
    float s = v[0];
    for (; d; d /= 2) s += __shfl_xor_sync(~0u, s, d);
    return s;                                              // value k in lanes 32 k / N ..
}
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* red) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const float s = scatter_sum(v);
    if ((lane & (32 / N - 1)) == 0) red[(threadIdx.x >> 5) * N + lane / (32 / N)] = s;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = lane < warps ? red[lane * N + k] : 0.0f;
    const float all = scatter_sum(v);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __shfl_sync(~0u, all, k * (32 / N));
}
__device__ __forceinline__ float row_sum(float v, float* red) {
    float a[1] = {v};
    block_sums(a, red);
    return a[0];
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
        dst->v = *src;                                     // two bytes: there is no such copy, the thread waits for the load
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

// The arithmetic of RB rows after the loads: v (h, or x) in, y's values out; mean and rstd.  `here[i]`: whether the thread
// has chunk i (its v is 0 where not).  Sums: RB sums over the rows' threads.
template <int E, int NC, int RB, typename Affine, typename Sums>
__device__ __forceinline__ void norm_rows(float (&v)[RB][NC][E], const bool (&here)[NC], Affine&& affine, float inv_cols,
                                          float eps, float (&mean)[RB], float (&rstd)[RB], Sums&& sums) {
#pragma unroll
    for (int k = 0; k < RB; ++k) {
        mean[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) mean[k] += vsum(v[k][i]);
    }
    sums(mean, 0);
#pragma unroll
    for (int k = 0; k < RB; ++k) {
        mean[k] *= inv_cols;
        rstd[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float q[E] = {};
            vadd(v[k][i], -mean[k]);
            vfma(q, v[k][i], v[k][i], q);
            rstd[k] += here[i] ? vsum(q) : 0.0f;
        }
    }
    float s[RB];
#pragma unroll
    for (int k = 0; k < RB; ++k) s[k] = rstd[k];
    sums(s, 1);
#pragma unroll
    for (int k = 0; k < RB; ++k) rstd[k] = rsqrtf(s[k] * inv_cols + eps);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        float w[E], b[E];
        affine(i, w, b);
#pragma unroll
        for (int k = 0; k < RB; ++k) {
            vmul(v[k][i], rstd[k]);
            vfma(v[k][i], v[k][i], w, b);
        }
    }
}
// h = v + the chunk, rounded to its type, stored and left in v.
template <typename X, int E>
__device__ __forceinline__ void add_residual(const Chunk<X, E>& c, float (&v)[E], X* h) {
    float a[E];
    c.get(a);
    vadd(v, a);
    Chunk<X, E> r;
    r.set(v);
    r.store(h);
    r.get(v);
}
// A chunk of weight and bias (zeros without one, and where the thread has no chunk).
template <int E>
__device__ __forceinline__ void load_affine(const FwdParams& p, bool here, int64_t at, float (&w)[E], float (&b)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = b[e] = 0.0f;
    if (here) {
        load_vec<E>(p.weight, p.w_f32, at, w);
        if (p.bias) load_vec<E>(p.bias, p.w_f32, at, b);
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
    for (int i = 0; i < NC; ++i) {
        here[i] = t + i * G < chunks;
        load_affine<E>(p, here[i], (t + i * G) * E, w[i], b[i]);
    }
    auto affine = [&](int i, float (&wi)[E], float (&bi)[E]) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            wi[e] = w[i][e];
            bi[e] = b[i][e];
        }
    };
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
            float v[1][NC][E] = {}, mean[1], rstd[1];
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (r < p.rows && here[i]) {
                    in[u][i].get(v[0][i]);
                    if (p.residual) add_residual(add[u][i], v[0][i], static_cast<X*>(p.h) + r * p.ldh + (t + i * G) * E);
                }
            norm_rows(v, here, affine, inv_cols, p.eps, mean, rstd, [&](float (&s)[1], int) { s[0] = group_sum(s[0], G); });
            if (r < p.rows) {
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (here[i]) Chunk<Y, E>::put(static_cast<Y*>(p.y) + r * p.ldy + (t + i * G) * E, v[0][i]);
                if (t == 0) {
                    p.mean[r] = mean[0];
                    p.rstd[r] = rstd[0];
                }
            }
        }
    }
}

// Registers of a thread of the wide kernels.  Two rows at a time with a residual, forward: 48, with weight and bias read
// for each batch, so that two blocks of 640 threads share an SM (8192 x 5120, fp32 x: 89 us, 101 us with 96 and one block).
// Without a residual, and backward with its column sums, 96 with weight and bias kept (bf16: 38 us, 42 us with 48).
// Blocks of more threads take one row at a time, with 64: there the forward kernel of two chunks a thread spills with a residual
// (8200 to 16384 columns: 48 to 128 bytes a thread; 2048 x 16384 bf16 50 us, 4.9 TB/s), the other block kernels
// at most 16 bytes, the narrow fp32 one of 264 to 512 columns 44.
constexpr int kFewRegs = 48, kRegs = 96, kManyThreadsRegs = 64;

// A block per RB rows, S such batches of copies: S - 1 ahead.  Shared memory: [S][RB][x, residual][NC][threads] chunks.
template <typename X, typename Y, int E, int NC, int RB, int S, bool RES>
__global__ void __maxnreg__(RB == 1 ? kManyThreadsRegs : RES ? kFewRegs : kRegs) norm_fwd_kernel(FwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ __align__(16) uint8_t norm_smem[];
    __shared__ float red[2][32 * RB];
    constexpr int A = RES ? 2 : 1;
    const int t = threadIdx.x, width = blockDim.x;
    Chunk<X, E>* ring = reinterpret_cast<Chunk<X, E>*>(norm_smem) + t;
    auto at = [&](int slot, int k, int a, int i) { return ring + (((slot * RB + k) * A + a) * NC + i) * width; };
    const float inv_cols = 1.0f / (float)p.cols;
    constexpr bool KEEP = !(RB == 2 && RES);               // weight and bias stay in registers
    bool here[NC];
    float wk[KEEP ? NC : 1][E], bk[KEEP ? NC : 1][E];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        here[i] = t + i * width < (int)(p.cols / E);
        if constexpr (KEEP) load_affine<E>(p, here[i], (t + i * width) * E, wk[i], bk[i]);
    }
    auto affine = [&](int i, float (&w)[E], float (&b)[E]) {
        if constexpr (KEEP) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                w[e] = wk[i][e];
                b[e] = bk[i][e];
            }
        } else {
            load_affine<E>(p, here[i], (t + i * width) * E, w, b);
        }
    };
    const int64_t stride = (int64_t)gridDim.x * RB, first = (int64_t)blockIdx.x * RB;
    // this thread's first chunk of the next batch to fetch, and of the next to store
    const X *x = static_cast<const X*>(p.x) + first * p.ldx + t * E, *res = static_cast<const X*>(p.residual) + first * p.ldr + t * E;
    X* h = static_cast<X*>(p.h) + first * p.ldh + t * E;
    Y* y = static_cast<Y*>(p.y) + first * p.ldy + t * E;
    const int64_t step_x = stride * p.ldx, step_res = stride * p.ldr, step_h = stride * p.ldh, step_y = stride * p.ldy;
    int64_t ahead = first;
    auto fetch = [&](int slot) {
#pragma unroll
        for (int k = 0; k < RB; ++k)
            if (ahead + k < p.rows) {
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (here[i]) {
                        copy_chunk(at(slot, k, 0, i), x + k * p.ldx + i * width * E);
                        if constexpr (RES) copy_chunk(at(slot, k, 1, i), res + k * p.ldr + i * width * E);
                    }
            }
        copies_commit();
        ahead += stride;
        x += step_x;
        if constexpr (RES) res += step_res;
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fetch(k);
    int slot = 0;
    for (int64_t r = first; r < p.rows; r += stride) {
        fetch(slot == 0 ? S - 1 : slot - 1);
        copies_wait<S - 1>();
        float v[RB][NC][E] = {}, mean[RB], rstd[RB];
#pragma unroll
        for (int k = 0; k < RB; ++k)
            if (r + k < p.rows)
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (here[i]) {
                        at(slot, k, 0, i)->get(v[k][i]);
                        if constexpr (RES) add_residual(*at(slot, k, 1, i), v[k][i], h + k * p.ldh + i * width * E);
                    }
        norm_rows(v, here, affine, inv_cols, p.eps, mean, rstd, [&](float (&s)[RB], int k) { block_sums(s, red[k]); });
#pragma unroll
        for (int k = 0; k < RB; ++k)
            if (r + k < p.rows) {
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (here[i]) Chunk<Y, E>::put(y + k * p.ldy + i * width * E, v[k][i]);
                if (t == 0) {
                    p.mean[r + k] = mean[k];
                    p.rstd[r + k] = rstd[k];
                }
            }
        y += step_y;
        if constexpr (RES) h += step_h;
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

// RB rows of the backward pass after the loads: xhat = x and g = dy come in (0 where the thread has no chunk or there is no
// row), dx without dh goes out in g, the column sums grow.  Sums: 2 RB sums over the rows' threads.
template <int E, int NC, int RB, typename Sums>
__device__ __forceinline__ void grad_rows(float (&xhat)[RB][NC][E], float (&g)[RB][NC][E], const float (&w)[NC][E],
                                          float (&sw)[NC][E], float (&sb)[NC][E], const float (&mean)[RB],
                                          const float (&rstd)[RB], float inv_cols, Sums&& sums) {
    float s[2 * RB];
#pragma unroll
    for (int k = 0; k < RB; ++k) {
        float a[E] = {}, b[E] = {};
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            vadd(xhat[k][i], -mean[k]);
            vmul(xhat[k][i], rstd[k]);
            vfma(sw[i], g[k][i], xhat[k][i], sw[i]);
            vadd(sb[i], g[k][i]);
            vmul(g[k][i], w[i]);
            vadd(a, g[k][i]);
            vfma(b, g[k][i], xhat[k][i], b);
        }
        s[2 * k] = vsum(a);
        s[2 * k + 1] = vsum(b);
    }
    sums(s);
#pragma unroll
    for (int k = 0; k < RB; ++k)
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            vfma(g[k][i], xhat[k][i], -s[2 * k + 1] * inv_cols, g[k][i]);
            vadd(g[k][i], -s[2 * k] * inv_cols);
            vmul(g[k][i], rstd[k]);
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
            float xhat[1][NC][E] = {}, g[1][NC][E] = {}, m[1] = {mean[u]}, rs[1] = {rstd[u]};
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (r < p.rows && t + i * G < chunks) {
                    x[u][i].get(xhat[0][i]);
                    dy[u][i].get(g[0][i]);
                }
            grad_rows(xhat, g, w, sw, sb, m, rs, inv_cols, [&](float (&s)[2]) {
                s[0] = group_sum(s[0], G);
                s[1] = group_sum(s[1], G);
            });
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (r < p.rows && t + i * G < chunks) {
                    if (p.dh) {
                        float a[E];
                        dh[u][i].get(a);
                        vadd(g[0][i], a);
                    }
                    Chunk<X, E>::put(static_cast<X*>(p.dx) + r * p.lddx + (t + i * G) * E, g[0][i]);
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

// A block per RB rows, S such batches of copies.  Shared memory: [S][RB][x, dy, dh][NC][threads] chunks.
template <typename X, typename Y, int E, int NC, int RB, int S, bool RES>
__global__ void __maxnreg__(RB == 1 ? kManyThreadsRegs : kRegs) norm_bwd_kernel(BwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ __align__(16) uint8_t norm_smem[];
    __shared__ float red[2][64 * RB];                      // two buffers take turns
    const int t = threadIdx.x, width = blockDim.x;
    const uint32_t xs = NC * width * sizeof(Chunk<X, E>), ys = NC * width * sizeof(Chunk<Y, E>);
    const uint32_t row_bytes = xs + ys + (RES ? xs : 0), slot_bytes = RB * row_bytes;
    auto at_x = [&](uint32_t row, int i) { return reinterpret_cast<Chunk<X, E>*>(norm_smem + row) + i * width + t; };
    auto at_dy = [&](uint32_t row, int i) { return reinterpret_cast<Chunk<Y, E>*>(norm_smem + row + xs) + i * width + t; };
    auto at_dh = [&](uint32_t row, int i) { return reinterpret_cast<Chunk<X, E>*>(norm_smem + row + xs + ys) + i * width + t; };
    const float inv_cols = 1.0f / (float)p.cols;
    bool here[NC];
    float w[NC][E] = {}, sw[NC][E] = {}, sb[NC][E] = {};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        here[i] = t + i * width < (int)(p.cols / E);
        if (here[i]) load_vec<E>(p.weight, p.w_f32, (t + i * width) * E, w[i]);
    }
    const int64_t first = (int64_t)blockIdx.x * RB, stride = (int64_t)gridDim.x * RB;
    const X *x = static_cast<const X*>(p.x) + first * p.ldx + t * E, *dh = static_cast<const X*>(p.dh) + first * p.lddh + t * E;
    const Y* dy = static_cast<const Y*>(p.dy) + first * p.lddy + t * E;
    X* dx = static_cast<X*>(p.dx) + first * p.lddx + t * E;
    const int64_t step_x = stride * p.ldx, step_dh = stride * p.lddh, step_dy = stride * p.lddy, step_dx = stride * p.lddx;
    int64_t ahead = first;
    auto fetch = [&](uint32_t slot) {
#pragma unroll
        for (int k = 0; k < RB; ++k)
            if (ahead + k < p.rows) {
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (here[i]) {
                        copy_chunk(at_x(slot + k * row_bytes, i), x + k * p.ldx + i * width * E);
                        copy_chunk(at_dy(slot + k * row_bytes, i), dy + k * p.lddy + i * width * E);
                        if constexpr (RES) copy_chunk(at_dh(slot + k * row_bytes, i), dh + k * p.lddh + i * width * E);
                    }
            }
        copies_commit();
        ahead += stride;
        x += step_x;
        dy += step_dy;
        if constexpr (RES) dh += step_dh;
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fetch(k * slot_bytes);
    float mean[RB] = {}, rstd[RB] = {};
    auto stats = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < RB; ++k)
            if (r + k < p.rows) {
                mean[k] = p.mean[r + k];
                rstd[k] = p.rstd[r + k];
            }
    };
    stats(first);
    uint32_t slot = 0;
    int buf = 0;
    for (int64_t r = first; r < p.rows; r += stride, buf ^= 1) {
        fetch(slot == 0 ? (S - 1) * slot_bytes : slot - slot_bytes);
        copies_wait<S - 1>();
        float m[RB], rs[RB], xhat[RB][NC][E] = {}, g[RB][NC][E] = {};
#pragma unroll
        for (int k = 0; k < RB; ++k) {
            m[k] = mean[k];
            rs[k] = rstd[k];
            if (r + k < p.rows)
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (here[i]) {
                        at_x(slot + k * row_bytes, i)->get(xhat[k][i]);
                        at_dy(slot + k * row_bytes, i)->get(g[k][i]);
                    }
        }
        stats(r + stride);
        grad_rows(xhat, g, w, sw, sb, m, rs, inv_cols, [&](float (&s)[2 * RB]) { block_sums(s, red[buf]); });
#pragma unroll
        for (int k = 0; k < RB; ++k)
            if (r + k < p.rows)
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (here[i]) {
                        if constexpr (RES) {
                            float a[E];
                            at_dh(slot + k * row_bytes, i)->get(a);
                            vadd(g[k][i], a);
                        }
                        Chunk<X, E>::put(dx + k * p.lddx + i * width * E, g[k][i]);
                    }
        dx += step_dx;
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

// dweight and dbias from the parts: a block takes 32 of the 2 cols columns (a part's two rows follow one another), its 16
// warps every sixteenth part, ten loads at a time.
constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads) norm_bwd_join_kernel(BwdParams p) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float red[16][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = blockIdx.x * 32ll + lane, part = 2 * p.cols;
    float s = 0.0f;
    if (c < part) {
        for (int i = warp; i < p.nparts; i += 160) {
            float v[10];
#pragma unroll
            for (int k = 0; k < 10; ++k) v[k] = i + 16 * k < p.nparts ? p.parts[(int64_t)(i + 16 * k) * part + c] : 0.0f;
#pragma unroll
            for (int k = 0; k < 10; ++k) s += v[k];
        }
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < part) {
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s += red[k][lane];
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
    __shared__ float red[2][32];
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
    int64_t r = r0;
    // Chunks of 16 bytes: four rows' loads before the first is used (whole backward pass, 300 x 12000 bf16: 27 -> 23 us, 2048 x
    // 16384: 107 -> 102).  Single elements the compiler's own unrolling serves better (3000 x 10001: 120 us, 174 with both
    // loops in batches of this kind).
    if constexpr (E == 8)
        for (; r < r1; r += 4) {
            Chunk<Y, E> dy[4];
            Chunk<X, E> x[4];
            float mean[4], rstd[4], g[E], v[E];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (r + u < r1) {
                    dy[u].load(static_cast<const Y*>(p.dy) + (r + u) * p.lddy + c);
                    x[u].load(static_cast<const X*>(p.x) + (r + u) * p.ldx + c);
                    mean[u] = p.mean[r + u];
                    rstd[u] = p.rstd[r + u];
                }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (r + u < r1) {
                    dy[u].get(g);
                    x[u].get(v);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        sw[e] = fmaf(g[e], (v[e] - mean[u]) * rstd[u], sw[e]);
                        sb[e] += g[e];
                    }
                }
        }
    for (; r < r1; ++r) {
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
    __shared__ float red[2][32];
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
template <int N> struct Int { static constexpr int value = N; };
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

constexpr int kNarrow = 128;                   // threads of a block of narrow rows
constexpr int kRingBytes = 200 * 1024;         // shared memory of an SM for copies
// The most threads that take two rows at a time, 5120 columns in chunks of 8 (96 registers each; the register file would hold 672
// threads).  8192 rows, with residual, forward / backward: 5120 columns 55 / 57 us (61 / 77 a row at a time); 6144, a row at a time,
// 64 / 79; 8192: 91 .. 94 / 94.
constexpr int kTwoRows = 640;

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
// A launch of a wide kernel: `rb` rows at a time where a block's registers allow it and there are rows enough to go
// round, `stages` batches of copies (as many as let the blocks that the registers allow run at once), the
// persistent grid.
struct WidePlan {
    int threads, rb, stages;
    size_t smem;
    int64_t grid;
};
WidePlan wide_plan(int64_t rows, int64_t chunks, int nc, size_t row_bytes_of_thread, int most_stages, int two_row_regs) {
    WidePlan w;
    w.threads = block_threads(chunks, nc);
    w.rb = nc == 1 && w.threads <= kTwoRows && rows > sms() && 4 * w.threads * row_bytes_of_thread <= 216 * 1024 ? 2 : 1;
    const int regs = w.rb == 2 ? two_row_regs : kManyThreadsRegs;
    const int64_t blocks = std::max(1, std::min(65536 / (regs * w.threads), 2048 / w.threads));
    const size_t slot = (size_t)w.threads * w.rb * row_bytes_of_thread;
    w.stages = most_stages * slot * blocks <= kRingBytes ? most_stages : 2;
    w.smem = w.stages * slot;
    w.grid = std::min<int64_t>((rows + w.rb - 1) / w.rb, sms() * std::max<int64_t>(1, std::min<int64_t>(blocks, 224 * 1024 / (w.smem + 2048))));
    return w;
}
// The shared memory that a kernel may take is an attribute of the kernel on a device, and one kernel serves many widths: it is
// raised once, to all that a block can have beside the kernel's own arrays, and never lowered, so that a call cannot take from
// a call of another thread what that is about to launch with.
template <auto kern, typename P>
cudaError_t launch_ring(int64_t grid, int threads, size_t smem, cudaStream_t s, const P& p) {
    static std::atomic<uint64_t> set{0};                   // the first 64 devices
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (e == cudaSuccess && !(set.load(std::memory_order_relaxed) & bit)) {
        cudaFuncAttributes fa;
        int most = 0;
        e = cudaFuncGetAttributes(&fa, kern);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)fa.sharedSizeBytes);
        if (e == cudaSuccess) set.fetch_or(bit, std::memory_order_relaxed);
    }
    return e == cudaSuccess ? launch_pdl(kern, dim3((unsigned)grid), dim3(threads), smem, s, p) : e;
}

// How the backward pass cuts the rows.  Rows wider than its registers reach go through the loops.
struct BwdPlan {
    enum { kWarp, kBlock, kLoop } kind;
    int parts;
    WidePlan w;
};
BwdPlan bwd_plan(int64_t rows, int64_t cols, bool vec, size_t row_elem_bytes) {
    const int64_t chunks = vec ? cols / 8 : cols;
    const int nc = vec ? 1 : chunks <= 4096 ? 4 : 8;
    BwdPlan b = {};
    int64_t parts;
    if (chunks <= (vec ? 64 : 256)) {
        const int g = group_lanes(chunks);
        b.kind = BwdPlan::kWarp;
        b.w.threads = kNarrow;
        b.w.smem = 2 * (size_t)cols * sizeof(float);
        parts = std::min<int64_t>((rows + kNarrow / g - 1) / (kNarrow / g), sms() * 4ll);
    } else if (chunks <= 1024 * nc) {
        b.kind = BwdPlan::kBlock;
        b.w = wide_plan(rows, chunks, nc, nc * (vec ? 8 : 1) * row_elem_bytes, 3, kRegs);
        b.w.grid = std::min<int64_t>(b.w.grid, 3 * sms());     // each block's part is written and read once more
        parts = b.w.grid;
    } else {
        b.kind = BwdPlan::kLoop;
        b.w.threads = kLoopThreads;
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
            const int64_t grid = std::min<int64_t>((rows + kNarrow / g - 1) / (kNarrow / g), sms() * 5ll);
            return to_status(launch_pdl(kern, dim3((unsigned)grid), dim3(kNarrow), 0, s, p, g));
        };
        // stages 4 or 2, with or without residual, for one shape of a thread's part
        auto wide = [&](auto e, auto nc, auto rb, const WidePlan& w) {
            constexpr int E = decltype(e)::value, NC = decltype(nc)::value, RB = decltype(rb)::value;
            auto run = [&](auto stages, auto res) {
                return to_status(launch_ring<norm_fwd_kernel<X, Y, E, NC, RB, decltype(stages)::value, decltype(res)::value>>(
                    w.grid, w.threads, w.smem, s, p));
            };
            if (residual) return w.stages == 4 ? run(Int<4>{}, std::true_type{}) : run(Int<2>{}, std::true_type{});
            return w.stages == 4 ? run(Int<4>{}, std::false_type{}) : run(Int<2>{}, std::false_type{});
        };
        const size_t elem = sizeof(X) * (residual ? 2 : 1);
        if (vec) {
            if (chunks <= 32) return narrow(norm_fwd_warp_kernel<X, Y, 8, 1, 4>);
            if (chunks <= 64) return narrow(norm_fwd_warp_kernel<X, Y, 8, 2, 2>);
            if (chunks <= 1024) {
                const WidePlan w = wide_plan(rows, chunks, 1, 8 * elem, 4, residual ? kFewRegs : kRegs);
                return w.rb == 2 ? wide(Int<8>{}, Int<1>{}, Int<2>{}, w) : wide(Int<8>{}, Int<1>{}, Int<1>{}, w);
            }
            // two rows of 16384 fp32 columns with a residual do not fit shared memory
            if (chunks <= 2048 && 2 * cols * elem <= 216 * 1024)
                return wide(Int<8>{}, Int<2>{}, Int<1>{}, wide_plan(rows, chunks, 2, 16 * elem, 4, residual ? kFewRegs : kRegs));
            return to_status(launch_pdl(norm_fwd_loop_kernel<X, Y, 8>, dim3((unsigned)std::min<int64_t>(rows, 1 << 30)),
                                        dim3(kLoopThreads), 0, s, p));
        }
        if (chunks <= 32 * 8) return narrow(norm_fwd_warp_kernel<X, Y, 1, 8, 2>);
        if (chunks <= 1024 * 8) return wide(Int<1>{}, Int<8>{}, Int<1>{}, wide_plan(rows, chunks, 8, 8 * elem, 4, residual ? kFewRegs : kRegs));
        return to_status(launch_pdl(norm_fwd_loop_kernel<X, Y, 1>, dim3((unsigned)std::min<int64_t>(rows, 1 << 30)),
                                    dim3(kLoopThreads), 0, s, p));
    });
}

extern "C" size_t nvfp4_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1 || cols > (1ll << 30)) return 0;
    // whatever the types and the alignment turn out to be
    int parts = 0;
    for (size_t bytes : {4, 6, 8, 10, 12})                 // of an element of x, dh (of x's type, if there is one) and dy
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
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {                                       // no kernel: they read the weight before they look for rows
        cudaError_t e = cudaMemsetAsync(dweight, 0, cols * sizeof(float), s);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, cols * sizeof(float), s);
        return to_status(e);
    }
    const bool vec = cols % 8 == 0 && rows16(x, ldx) && rows16(dy, lddy) && rows16(dh, lddh) && rows16(dx, lddx) &&
                     aligned16(weight);
    const size_t xb = x_dtype == NVFP4_F32 ? 4 : 2, yb = y_dtype == NVFP4_F32 ? 4 : 2;
    const BwdPlan plan = bwd_plan(rows, cols, vec, xb * (dh ? 2 : 1) + yb);
    const BwdParams p{dy,   x,    weight, dh,  mean, rstd, dx,   dweight, dbias, static_cast<float*>(workspace),
                      rows, cols, lddy,   ldx, lddh, lddx, w_dtype == NVFP4_F32, plan.parts};
    return with_types(x_dtype, y_dtype, [&](auto tx, auto ty) {
        using X = typename decltype(tx)::type;
        using Y = typename decltype(ty)::type;
        cudaError_t e;
        const dim3 grid(plan.parts), block(plan.w.threads);
        if (plan.kind == BwdPlan::kWarp) {
            const int g = group_lanes(vec ? cols / 8 : cols);
            if (!vec) e = launch_pdl(norm_bwd_warp_kernel<X, Y, 1, 8, 1>, grid, block, plan.w.smem, s, p, g);
            else if (cols <= 256) e = launch_pdl(norm_bwd_warp_kernel<X, Y, 8, 1, 2>, grid, block, plan.w.smem, s, p, g);
            else e = launch_pdl(norm_bwd_warp_kernel<X, Y, 8, 2, 1>, grid, block, plan.w.smem, s, p, g);
        } else if (plan.kind == BwdPlan::kBlock) {
            auto wide = [&](auto ee, auto nc, auto rb) {
                constexpr int E = decltype(ee)::value, NC = decltype(nc)::value, RB = decltype(rb)::value;
                auto run = [&](auto stages, auto res) {
                    return launch_ring<norm_bwd_kernel<X, Y, E, NC, RB, decltype(stages)::value, decltype(res)::value>>(
                        plan.parts, plan.w.threads, plan.w.smem, s, p);
                };
                if (dh) e = plan.w.stages == 3 ? run(Int<3>{}, std::true_type{}) : run(Int<2>{}, std::true_type{});
                else e = plan.w.stages == 3 ? run(Int<3>{}, std::false_type{}) : run(Int<2>{}, std::false_type{});
            };
            if (!vec && cols <= 4096) wide(Int<1>{}, Int<4>{}, Int<1>{});
            else if (!vec) wide(Int<1>{}, Int<8>{}, Int<1>{});
            else if (plan.w.rb == 2) wide(Int<8>{}, Int<1>{}, Int<2>{});
            else wide(Int<8>{}, Int<1>{}, Int<1>{});
        } else {
            auto loops = [&](auto cols_kern, auto rows_kern, int per) {
                const dim3 cut((unsigned)((cols / per + kLoopThreads - 1) / kLoopThreads), plan.parts);
                e = launch_pdl(cols_kern, cut, block, 0, s, p);
                if (e == cudaSuccess)
                    e = launch_pdl(rows_kern, dim3((unsigned)std::min<int64_t>(rows, 1 << 30)), block, 0, s, p);
            };
            if (vec) loops(norm_bwd_cols_loop_kernel<X, Y, 8>, norm_bwd_rows_loop_kernel<X, Y, 8>, 8);
            else loops(norm_bwd_cols_loop_kernel<X, Y, 1>, norm_bwd_rows_loop_kernel<X, Y, 1>, 1);
        }
        if (e == cudaSuccess)
            e = launch_pdl(norm_bwd_join_kernel, dim3((unsigned)((2 * cols + 31) / 32)), dim3(kJoinThreads), 0, s, p);
        return to_status(e);
    });
}
