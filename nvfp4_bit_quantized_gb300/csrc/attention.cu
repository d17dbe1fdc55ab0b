// attention.cu -- attention over packed sequences, forward and backward (include/nvfp4.h has the
// formulas), on the tcgen05 tensor cores: bf16 heads of at most 128 elements, fp32 accumulators in
// TMEM, fp32 softmax statistics and sums.
//
// Three kernels, one CTA per SM, each on a tile of rows that stays in shared memory while tiles of
// 128 rows of the other side stream past by TMA (HD = 64 or 128: the head size rounded up; the MMAs
// themselves run over the head size rounded up to 16):
//   fwd   256 queries of a head as two tiles; S = Q K^T, P = exp2(c S - m), O += P V;
//   dq    128 queries of a head;   S = Q K^T, dP = dO V^T, dS = P (dP - delta), dQ += dS K;
//   dkv   128 keys of a key head, over all query heads that read it;
//         S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q.
// fwd and dq stay on their SM for all their tiles and begin the next one while the last is stored.  Where there are too few
// tiles for the SMs, CTAs share a tile's steps and leave fp32 parts that a last kernel joins in order.
// P and dS go back to TMEM as bf16 and are the A operand of their product from there: the tensor cores want A of B's type, and
// the inputs are bf16.  Kept in fp32 they would need tf32 products, at half the rate and twice the TMEM, of operands converted
// from bf16.  What the rounding costs: against 64 bits the outputs are off by 0.00172 of their norm forward, 0.0029 backward (8192
// tokens, 40 / 8 heads of 128, causal); with P and dS in fp32 by 0.00168 and 0.0024.
// The streamed tile that was the K-major B operand of the first product is the MN-major B operand of the second, so
// each tile is loaded once.  The backward pass computes S and dP in both of its kernels (7 products
// instead of 5): in exchange dQ needs neither atomics (whose order would change the result from run
// to run) nor a pass of partial sums through memory.
//
// 8192 tokens, 40 / 8 heads of 128, causal: forward 399 .. 404 us, 1.70 .. 1.72 PFLOP/s of bf16; backward 1.25 .. 1.30 ms, 1.32 ..
// 1.37 PFLOP/s counting five products, 1.85 .. 1.92 counting the seven (in a CUDA graph; in a long row of passes at the clocks
// that the power limit leaves, 442 .. 452 us and 1.47 ms).  What bounds them there is the rate of the tensor
// cores under the power limit (cuBLAS sustains 1.71).  With short sequences (8192 tokens in 13 documents, 32 heads
// of 64: forward 78 .. 86 us, backward with 8 key heads 202) it is what a tile costs beside its steps: its loads, masks and stores,
// code that runs once a tile and is not in the instruction caches then.  So loops outside the steps are not unrolled (forward
// 90 us with them unrolled; the long case gains 2 % from it).
//
// Tiles that reach past their sequence: rows past the tensor's end arrive as zeros (TMA); rows
// of a neighbouring sequence are zeroed in shared memory before the MMAs read them where they are summed
// over (a zero probability times a neighbour's NaN would be NaN).
//
// Every wait is bounded (mbar_wait_bounded): on a timeout the kernel records NVFP4_ERR_TIMEOUT, every
// role leaves its loop, copies and MMAs in flight are waited for, TMEM is freed.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "device_common.cuh"
#include "host_common.h"
#include "tcgen05_bf16.cuh"

namespace nvfp4 {
namespace attn {

using bf16 = __nv_bfloat16;
using namespace tc;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Heads {
    bf16* p;
    int64_t ts, hs;
    __device__ __forceinline__ bf16* at(int64_t t, int h) const { return p + t * ts + h * hs; }
};

struct Params {
    Heads out, dout, dq, dk, dv;               // tensors reached by plain loads and stores
    float *lse, *delta;
    int64_t tq, tk;
    int heads, kv_heads, dim, causal, nseq;
    float scale;
    float c;                                   // |scale| log2(e), kept off zero; the MMAs negate A for scale < 0
    const int32_t *cu_q, *cu_k;
    uint32_t* dev_status;
    uint64_t timeout_ns;
    int work;                                  // tiles x heads x parts: what the CTAs go through
    int parts;                                 // CTAs that share a tile's steps
    float *part_sums, *part_lse;               // what they leave, parts > 1: [parts][..., tokens, heads, dim], [parts][heads, tq]
};

// One CTA's rows.  `first` .. first + rows - 1 are its tile's tokens of one sequence; the other
// side's sequence is `other` .. other + other_len - 1.  diag: row r of the tile faces other row
// r + diag on the causal diagonal.
struct Item {
    int valid;                                             // 0: nothing here; -1: no more work
    int part;                                              // of the tile's steps, where CTAs share them
    int head;
    int64_t first, other;
    int rows, other_len, diag;
};

// Whole warp: the last of nseq sequences whose slots begin, at cu[s] / tile + s, at or before `want`; 32 candidates at a time.
template <int tile>
__device__ __forceinline__ int search_slot(const int32_t* cu, int nseq, int64_t total, int64_t want) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = nseq;
    while (hi - lo > 1) {
        const int step = (int)(((int64_t)hi - lo + 31) / 32);
        const int64_t s = lo + (int64_t)lane * step;
        bool before = lane == 0;
        if (lane && s < hi) before = min(max((int64_t)cu[s], (int64_t)0), total) / tile + s <= want;
        lo += (31 - __clz(__ballot_sync(~0u, before))) * step;
        hi = (int)min((int64_t)hi, (int64_t)lo + step);
    }
    return lo;
}

// Whole warp: the tile and head that `work` stands for.  The longest tiles come first, as they are under a causal mask:
// a sequence's tiles are as long as the number of them up to them (of queries) or from them on (of keys).  That order runs
// through all sequences where there are at most 32, whose offsets a warp holds at once; more are taken one after another.
// Heads are fastest, so that CTAs that run together read the same K and V.
// Up to kCounted sequences' tiles are counted for each item; with more that would take longer than the tile, and the sequence is
// searched for, over slots of which some are empty and fall on the CTAs as they come (65536 tokens, 32 / 8 heads of 64,
// forward / backward: 48 equal documents 521 / 1645 us counted, 616 / 1568 searched for; 128: 387 / 1087 and 342 / 1050; 4096:
// 41700 / 58500 and 3600 / 6100).
constexpr int kCounted = 64;
template <int tile>
__device__ __forceinline__ void find_item(const Params& p, bool rows_are_q, int heads, int work, Item* out) {
    const int lane = threadIdx.x & 31, block = p.parts > 1 ? work / p.parts : work;
    const int32_t *cu = rows_are_q ? p.cu_q : p.cu_k, *cu_other = rows_are_q ? p.cu_k : p.cu_q;
    const int64_t total = rows_are_q ? p.tq : p.tk, total_other = rows_are_q ? p.tk : p.tq;
    // The lane's sequence of the present 32: its rows, the other side's, its tiles.  Offsets that break the rules are
    // forced into range and reported.
    int64_t a = 0, b = 0, oa = 0, ob = 0, tiles = 0;
    bool bad = false;
    auto bounds = [&](const int32_t* o, int s, int64_t all, int64_t& lo, int64_t& hi) {
        const int64_t x = o ? o[s] : 0, y = o ? o[s + 1] : all;
        bad |= x > y || (s == 0 && x != 0) || (s == p.nseq - 1 && y != all);
        lo = min(max(x, (int64_t)0), all);
        hi = min(max(y, lo), all);
    };
    auto load = [&](int s0) {
        const int s = s0 + lane;
        a = b = oa = ob = tiles = 0;
        if (s < p.nseq) {
            bounds(cu, s, total, a, b);
            bounds(cu_other, s, total_other, oa, ob);
            tiles = (int64_t)((uint64_t)(b - a + tile - 1) / tile);
        }
    };
    // n: tiles in all or, where they are not counted, the host's bound, of slots that are searched: sequence s has those from
    // cu[s] / tile + s on, and its tiles are the first of them (there is at most one slot more).
    const bool counted = p.nseq <= kCounted;
    int64_t n = 0;
    if (counted) {
#pragma unroll 1
        for (int s0 = 0; s0 < p.nseq; s0 += 32) {
            load(s0);
            int64_t sum = tiles;
#pragma unroll
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
            n += sum;
        }
    } else {
        n = total / tile + p.nseq;
        if ((int64_t)work * 32 < p.nseq) load(work * 32);  // the first items check everybody's offsets
    }
    if (bad && (work == 0 || !counted)) set_status(p.dev_status, NVFP4_ERR_INVALID_ARG);
    int64_t want = block / heads;
    if (want >= n) {
        if (lane == 0) out->valid = 0;
        return;
    }
    int64_t index = -1;                                    // of the tile in its sequence, in the lane that has that
    if (p.nseq <= 32) {
        // each sequence of at least c tiles has one of length c: bands of c with the same sequences, from the longest on
        const int mine = (int)tiles;
        int cur = __reduce_max_sync(~0u, mine), left = (int)want;
        while (cur > 0) {
            const uint32_t mask = __ballot_sync(~0u, mine >= cur);
            const int count = __popc(mask), next = __reduce_max_sync(~0u, mine < cur ? mine : 0);
            if (left < (cur - next) * count) {
                const int c = cur - left / count, rank = left % count;
                if (mine >= cur && __popc(mask & ((1u << lane) - 1u)) == rank) index = rows_are_q ? c - 1 : mine - c;
                break;
            }
            left -= (cur - next) * count;
            cur = next;
        }
    } else if (counted) {
        if (rows_are_q) want = n - 1 - want;
#pragma unroll 1
        for (int s0 = 0; s0 < p.nseq; s0 += 32) {
            load(s0);
            int64_t upto = tiles;                          // inclusive prefix
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t v = __shfl_up_sync(~0u, upto, d);
                if (lane >= d) upto += v;
            }
            if (want >= upto - tiles && want < upto) index = want - (upto - tiles);
            const int64_t all = __shfl_sync(~0u, upto, 31);
            if (want < all) break;
            want -= all;
        }
    } else {
        if (rows_are_q) want = n - 1 - want;
        const int s = search_slot<tile>(cu, p.nseq, total, want);
        bounds(cu, s, total, a, b);
        bounds(cu_other, s, total_other, oa, ob);
        if (lane == 0) {
            index = want - (a / tile + s);
            if (index * tile >= b - a) index = -1;         // an empty slot, or offsets that break the rules
            if (index < 0) out->valid = 0;
        }
    }
    if (index >= 0) {
        const int64_t t0 = index * tile;
        out->valid = 1;
        out->part = p.parts > 1 ? work - block * p.parts : 0;
        out->head = block % heads;
        out->first = a + t0;
        out->rows = (int)min((int64_t)tile, b - a - t0);
        out->other = oa;
        out->other_len = (int)(ob - oa);
        out->diag = (int)(t0 + (ob - oa) - (b - a));
    }
}

// Bounded waits, as mbar_wait_bounded, but timed by the SM's own clock: reading the global timer, as that one
// does after the first failed try, takes longer than most waits here last.  Two cycles a nanosecond:
// at the highest clock, 2.07 GHz, the limit, at lower clocks a multiple of it.  The lanes of a converged warp try, read the
// flag and the clock together and get one answer; `all` also tells the compiler so, and costs a vote (1 % of the backward
// pass where the softmax warps use it).
struct Wait {
    uint64_t timeout_ns;
    volatile uint32_t* abort;
    uint32_t* dev_status;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        const uint32_t a = smem_addr(bar);
        if (mbar_try_wait(a, parity & 1u)) return true;
        const int64_t t0 = clock64();
        for (uint32_t i = 1;; ++i) {
            if (mbar_try_wait(a, parity & 1u)) return true;
            if ((i & 63u) == 0) {
                if (*abort) return false;
                if ((uint64_t)(clock64() - t0) > 2 * timeout_ns) {
                    set_status(dev_status, NVFP4_ERR_TIMEOUT);
                    *abort = 1u;
                    return false;
                }
            }
        }
    }
    // whole warp; the same answer in all lanes, so that what follows is known not to diverge
    __device__ __forceinline__ bool all(uint64_t* bar, uint32_t parity) const {
        return __all_sync(~0u, (*this)(bar, parity));
    }
    // after an abort: still bounded, but not cut short by it
    __device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) const {
        mbar_wait_bounded(bar, parity & 1u, timeout_ns, nullptr, dev_status);
    }
};

// A slot of a ring of N and the parity of its barriers' present phase.
template <int N> struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// The tiles that a CTA goes through, found one ahead by a warp of their own and read by `readers` others, which copy them.
struct Queue {
    Item item[2];
    uint64_t full[2], empty[2];
    __device__ __forceinline__ void init(int readers) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], readers);
        }
    }
    // whole warp
    template <int tile> __device__ __forceinline__ void feed(const Params& p, bool rows_are_q, int heads, const Wait& wait) {
        Ring<2> r;
        const int grid = gridDim.x;
        for (int k = 0;; ++k) {
            // to and fro: the CTA with the longest tile of one round has the shortest of the next
            const int at = (k & 1) ? grid - 1 - (int)blockIdx.x : (int)blockIdx.x, work = k * grid + at;
            const bool more = work < p.work, last = (k + 1) * grid >= p.work;
            if (!wait.all(&empty[r.slot], r.phase ^ 1u)) break;
            if (more) find_item<tile>(p, rows_are_q, heads, work, &item[r.slot]);
            else if ((threadIdx.x & 31) == 0) item[r.slot].valid = -1;
            __syncwarp();
            if (!more && !last) continue;
            if (more && item[r.slot].valid == 0) continue;         // the host counts sequences' last tiles generously
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(&full[r.slot]);
            if (!more) break;
            r.next();
        }
    }
    // whole warp; false: no more, or aborted
    __device__ __forceinline__ bool next(Ring<2>& r, const Wait& wait, Item& out) {
        if (!wait.all(&full[r.slot], r.phase)) return false;
        out = item[r.slot];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[r.slot]);
        r.next();
        return out.valid > 0;
    }
};

// The two MMA warps issue their groups of MMAs in turns, first (w = 0) and second (w = 1) of each round: the tensor
// cores then work off one group after the other.  Groups issued at will run interleaved and end
// together, and nothing is left to run while the softmax warps work on what both produced.
struct Turns {
    uint64_t* bar;                                         // two barriers, one arrival each
    Wait wait;
    int w;
    __device__ __forceinline__ bool take(int round) const {
        return w ? wait.all(&bar[1], round) : round == 0 || wait.all(&bar[0], round - 1);
    }
    __device__ __forceinline__ void pass() const {
        if (elect_one()) mbar_arrive(&bar[w ^ 1]);
        __syncwarp();
    }
};

// One lane: a tile of 128 tokens from token t of head h, HD / 64 boxes.
template <int HD>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* tm, int64_t t, int h, uint64_t* bar) {
#pragma unroll
    for (int b = 0; b < HD / 64; ++b)
        tma_load_3d(smem_addr(dst + b * kBoxBytes), tm, b * 64, (int)t, h, smem_addr(bar));
}

// Whole warp: zeroes rows `valid` .. 127 of a tile that the async proxy reads next.
template <int HD>
__device__ __forceinline__ void zero_tail(uint8_t* tile, int valid) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int i = lane; i < (kRows - valid) * 8; i += 32)
#pragma unroll
        for (int b = 0; b < HD / 64; ++b)
            *reinterpret_cast<uint4*>(tile + b * kBoxBytes + valid * 128 + i * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
}

// Whole warp.  D[128, 128] = A B^T over `ksteps` times 16 elements of the head: both tiles K-major, given by their
// descriptors.
template <int HD>
__device__ __forceinline__ void mma_heads(uint32_t d, uint32_t a, uint32_t b, int ksteps, uint32_t idesc) {
    const uint32_t lead = elect_one();
#pragma unroll
    for (int k = 0; k < HD / 16; ++k) {
        const uint32_t off = (k >> 2) * (kBoxBytes >> 4) + (k & 3) * 2;
        if (k < ksteps) mma_ss(d, a + off, b + off, idesc, k != 0, lead);
    }
}
// Whole warp.  D[128, n] (+)= A B with A 128 x 128 bf16 in TMEM: K 0-63 at a0, 64-127 at a1; B a tile of 128 rows.
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a0, uint32_t a1, uint32_t b, uint32_t idesc,
                                         uint32_t accumulate) {
    const uint32_t lead = elect_one();
#pragma unroll
    for (int k = 0; k < 8; ++k)
        mma_ts(d, k < 4 ? a0 + k * 8 : a1 + (k - 4) * 8, b + k * (2048 >> 4), idesc, k ? 1u : accumulate, lead);
}

// Whole warp: 32 columns from `col` of 32 rows of `dim` bf16 values (a multiple of 8), a lane's row v * f; the first row is
// token t's, `rows` of them are stored.  Four lanes first exchange 16-byte pieces, so that they write 64 bytes of one
// row after the other: a row per lane, a store touches 32 lines.
__device__ __forceinline__ void store32(const Heads& to, int64_t t, int head, int rows, int col, int dim,
                                        const uint32_t (&v)[32], float f) {
    const int lane = threadIdx.x & 31, q = lane & 3;
    uint32_t w[4][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i >> 2][i & 3] = pack_bf16(__uint_as_float(v[2 * i]) * f, __uint_as_float(v[2 * i + 1]) * f);
#pragma unroll
    for (int n = 1; n <= 2; n *= 2)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (!(k & n))
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t got = __shfl_xor_sync(~0u, q & n ? w[k][e] : w[k | n][e], n);
                    if (q & n) w[k][e] = got;
                    else w[k | n][e] = got;
                }
    if (col + 8 * q < dim) {
        bf16* at = to.at(t + (lane & ~3), head) + col + 8 * q;
#pragma unroll
        for (int k = 0; k < 4; ++k, at += to.ts)
            if ((lane & ~3) + k < rows) *reinterpret_cast<uint4*>(at) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
    }
}
// The same in fp32, a row per lane: a part's.
__device__ __forceinline__ void store32(float* row, int col, int dim, const uint32_t (&v)[32], float f) {
#pragma unroll
    for (int i = 0; i < 32; i += 4)
        if (col + i < dim)
            *reinterpret_cast<float4*>(row + col + i) =
                make_float4(__uint_as_float(v[i]) * f, __uint_as_float(v[i + 1]) * f, __uint_as_float(v[i + 2]) * f,
                            __uint_as_float(v[i + 3]) * f);
}
__device__ __forceinline__ void store_zeros(float* row, int dim) {
#pragma unroll 1
    for (int i = 0; i < dim; i += 4) *reinterpret_cast<float4*>(row + i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
}
// This part's steps of `steps`.
struct Share {
    int first, count;
    __device__ __forceinline__ Share(const Params& p, int part, int steps) {
        first = 0;
        count = steps;
        if (p.parts > 1) {                                 // the divisions take longer than some tiles' steps
            // steps x parts is below 2^32 (parts_for).  With 64-bit divisions, whose code is long and in every role, the
            // backward pass of 8192 tokens in 13 documents takes 254 us, not 244.
            first = (int)((uint32_t)steps * (uint32_t)part / (uint32_t)p.parts);
            count = (int)((uint32_t)steps * (uint32_t)(part + 1) / (uint32_t)p.parts) - first;
        }
    }
};
__device__ __forceinline__ void store_zeros(bf16* row, int dim) {
#pragma unroll 1
    for (int i = 0; i < dim; i += 8) *reinterpret_cast<uint4*>(row + i) = make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
    return p + ((1024u - (smem_addr(p) & 1023u)) & 1023u);
}

// ---------------------------------------------------------------------------- forward
// Warps 0-3 and 4-7: the softmax of tile 0 and tile 1, a row per thread; warp 8: TMA; warps 9 and 10: the MMAs
// of tile 0 and of tile 1 (one warp cannot issue MMAs of 64 cycles fast enough beside the softmax
// warps); warp 11: the next tiles to work on.  While one tile's softmax runs, the tensor cores work on the
// other tile.  A CTA stays for all its tiles: the next ones' queries and keys are loaded, and their first
// scores computed, while the last ones' outputs are stored.  TMEM: S of tile t at 128 t.  HD = 128: P (bf16) in the
// first 64 columns of S, O of tile t at 256 + 128 t.  HD = 64, where the softmax takes longer than the MMAs:
// O at 256 + 64 t and P in columns of its own at 384 + 64 t, so that the next scores are computed as soon as
// the present ones have been read, and a softmax follows the other without a pause.  O is rescaled only when a row's maximum has
// grown by more than 2^8 since it was last taken: P stays below 2^8 and the final division by the
// sum cancels the choice.
// A softmax thread holds a row's 128 scores at once: registers move from the third warpgroup to its two.
constexpr int kFwdThreads = 384;
constexpr int kFwdRegs = 168, kFwdRegsSoftmax = 208, kFwdRegsOther = 88;    // at launch, after setmaxnreg
static_assert(2 * kFwdRegsSoftmax + kFwdRegsOther <= 3 * kFwdRegs, "register split within the launch's registers");
template <int HD> struct Fwd {
    static constexpr int TILE = kRows * HD * 2;
    static constexpr int STAGES = HD == 128 ? 4 : 8;
    static constexpr int SMEM = (2 + STAGES) * TILE + 1024;
    static constexpr bool OWN_P = HD == 64;                // P has columns of its own
};

// Rows and key tiles of an item's two query tiles: tile t takes the key tiles j0 .. j0 + n[t] - 1.
struct FwdPlan {
    int rows[2], n[2], j0, steps;
    __device__ __forceinline__ FwdPlan(const Params& p, const Item& item) {
        for (int t = 0; t < 2; ++t) {
            rows[t] = min(max(item.rows - kRows * t, 0), kRows);
            int keys = item.other_len;
            if (p.causal) keys = min(keys, max(0, kRows * t + rows[t] + item.diag));
            n[t] = rows[t] ? (keys + kRows - 1) / kRows : 0;
        }
        const Share mine(p, item.part, max(n[0], n[1]));
        j0 = uniform(mine.first);
        n[0] = uniform(max(0, min(n[0] - j0, mine.count)));
        n[1] = uniform(max(0, min(n[1] - j0, mine.count)));
        steps = max(n[0], n[1]);
    }
};

template <int HD>
__global__ void __launch_bounds__(kFwdThreads, 1)
fwd_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
           const __grid_constant__ CUtensorMap tmv, const Params p) {
    constexpr int TILE = Fwd<HD>::TILE, ST = Fwd<HD>::STAGES;
    constexpr bool OWN_P = Fwd<HD>::OWN_P;
    constexpr int O_COLS = OWN_P ? 64 : 128;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t q_full, q_empty, full[ST], empty[ST], s_full[2], s_read[2], p_ready[2], pv_done[2], o_empty[2],
        turn[2], mma_done[2];
    __shared__ uint32_t tmem_slot, abort_flag;
    __shared__ Queue queue;
    uint8_t* smem_q = align1024(raw);
    uint8_t* ring = smem_q + 2 * TILE;
    const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        mbar_init(&q_full, 1);
        mbar_init(&q_empty, 2);
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_ready[t], 4);
            mbar_init(&s_read[t], 4);
            mbar_init(&pv_done[t], 1);
            mbar_init(&o_empty[t], 4);
            mbar_init(&turn[t], 1);
            mbar_init(&mma_done[t], 1);
        }
        queue.init(11);
        abort_flag = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) tmem_alloc_all(&tmem_slot);
    pdl_wait();
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = uniform(tmem_slot);
    const Wait wait{p.timeout_ns, &abort_flag, p.dev_status};
    Ring<2> items;
    Item item;

    // inside the roles' own branches: code after a join is compiled for the smaller share
    if (warp >= 8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kFwdRegsOther));
      if (warp == 11) {
        queue.feed<2 * kRows>(p, true, p.heads, wait);
      } else if (warp == 8) {
        Ring<ST> r;
        uint32_t loads = 0, queries = 0;                   // tiles and query pairs loaded
        bool ok = true;
        while (ok && queue.next(items, wait, item)) {
            const FwdPlan plan(p, item);
            if (plan.steps == 0) continue;
            const int hk = item.head / (p.heads / p.kv_heads);
            if (lane == 0) {
                ok = wait(&q_empty, queries ^ 1u);
                if (ok) {
                    mbar_arrive_expect_tx(&q_full, TILE * (plan.rows[1] ? 2 : 1));
                    load_tile<HD>(smem_q, &tmq, item.first, item.head, &q_full);
                    if (plan.rows[1]) load_tile<HD>(smem_q + TILE, &tmq, item.first + kRows, item.head, &q_full);
                    ++queries;
                }
                for (int i = 0; ok && i < 2 * plan.steps; ++i) {       // K of step 0, V of step 0, K of step 1, ...
                    ok = wait(&empty[r.slot], r.phase ^ 1u);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&full[r.slot], TILE);
                    load_tile<HD>(ring + r.slot * TILE, (i & 1) ? &tmv : &tmk,
                                  item.other + (int64_t)(plan.j0 + (i >> 1)) * kRows, hk, &full[r.slot]);
                    ++loads;
                    r.next();
                }
            }
            ok = __all_sync(~0u, ok);
        }
        if (lane == 0 && abort_flag) {                     // the copies in flight land first
            if (queries) wait.drain(&q_full, (queries - 1) & 1u);
            for (uint32_t j = loads > ST ? loads - ST : 0; j < loads; ++j) wait.drain(&full[j % ST], (j / ST) & 1u);
        }
      } else if (warp == 9 || warp == 10) {
        const int t = warp - 9;
        const uint32_t idesc_s = idesc_bf16(kRows, false, p.scale < 0.0f);
        const uint32_t idesc_o = idesc_bf16((p.dim + 15) & ~15, true, false);
        const int ksteps = (p.dim + 15) / 16;
        const uint32_t desc_q = uniform(desc_k_major(smem_addr(smem_q + t * TILE)));
        const uint32_t desc_k = uniform(desc_k_major(smem_addr(ring))), desc_v = uniform(desc_mn_major(smem_addr(ring)));
        const uint32_t ts = uniform(tmem + 128 * t), to = uniform(tmem + 256 + O_COLS * t);
        const uint32_t tp = OWN_P ? uniform(tmem + 384 + 64 * t) : ts;
        const Turns turns{turn, wait, t};
        Ring<ST> rk, rv;                                   // the next K and the next V to arrive
        rv.next();
        uint32_t queries = 0, outputs = 0, step = 0;       // done so far: query pairs, outputs, steps of this tile
        int round = 0;
        bool ok = true;
        while (ok && queue.next(items, wait, item)) {
            const FwdPlan plan(p, item);
            if (plan.steps == 0) continue;
            const int len = uniform(item.other_len) - plan.j0 * kRows, nt = t ? plan.n[1] : plan.n[0];
            const bool neighbours = uniform((int)(item.other + item.other_len < p.tk)) != 0;
            // waits for a tile of step j; both warps zero its foreign rows
            auto tile = [&](const Ring<ST>& r, int j) {
                const int valid = len - j * kRows;
                if (!wait.all(&full[r.slot], r.phase)) return false;
                if (valid < kRows && neighbours) zero_tail<HD>(ring + r.slot * TILE, valid);
                return true;
            };
            auto two = [](Ring<ST>& r) {
                r.next();
                r.next();
            };
            if constexpr (OWN_P) {
                ok = wait.all(&q_full, queries) && tile(rk, 0) && (step == 0 || nt == 0 || wait.all(&s_read[t], step - 1));
                if (!ok) break;
                if (nt > 0) {
                    fence_after();
                    mma_heads<HD>(ts, desc_q, desc_k + rk.slot * (TILE >> 4), ksteps, idesc_s);
                    commit(&s_full[t], elect_one());
                }
                commit(&empty[rk.slot], elect_one());
                if (nt <= 1) commit(&q_empty, elect_one());
                two(rk);
                for (int j = 0; j < plan.steps; ++j) {
                    if (j + 1 < plan.steps) {
                        ok = tile(rk, j + 1) && (j + 1 >= nt || wait.all(&s_read[t], step));
                        if (!ok) break;
                        if (j + 1 < nt) {
                            fence_after();
                            mma_heads<HD>(ts, desc_q, desc_k + rk.slot * (TILE >> 4), ksteps, idesc_s);
                            commit(&s_full[t], elect_one());
                        }
                        commit(&empty[rk.slot], elect_one());
                        if (j + 2 == nt) commit(&q_empty, elect_one());
                        two(rk);
                    }
                    ok = tile(rv, j) && (j > 0 || nt == 0 || wait.all(&o_empty[t], outputs ^ 1u)) &&
                         (j >= nt || wait.all(&p_ready[t], step));
                    if (!ok) break;
                    if (j < nt) {
                        fence_after();
                        mma_rows(to, tp, tp + 32, desc_v + rv.slot * (TILE >> 4), idesc_o, j > 0);
                        commit(&pv_done[t], elect_one());
                        ++step;
                    }
                    commit(&empty[rv.slot], elect_one());
                    two(rv);
                }
            } else {
                ok = wait.all(&q_full, queries) && tile(rk, 0) && turns.take(round);
                if (!ok) break;
                if (nt > 0) {
                    mma_heads<HD>(ts, desc_q, desc_k + rk.slot * (TILE >> 4), ksteps, idesc_s);
                    commit(&s_full[t], elect_one());
                }
                turns.pass();
                ++round;
                commit(&empty[rk.slot], elect_one());
                if (nt <= 1) commit(&q_empty, elect_one());
                two(rk);
                for (int j = 0; j < plan.steps; ++j) {
                    // what comes last is waited for last: a wait costs time even where it is over
                    ok = tile(rv, j) && (j + 1 >= plan.steps || tile(rk, j + 1)) &&
                         (j > 0 || nt == 0 || wait.all(&o_empty[t], outputs ^ 1u)) && turns.take(round) &&
                         (j >= nt || wait.all(&p_ready[t], step));
                    if (!ok) break;
                    if (j < nt) {
                        fence_after();
                        mma_rows(to, tp, tp + 32, desc_v + rv.slot * (TILE >> 4), idesc_o, j > 0);
                        if (j + 1 == nt) commit(&pv_done[t], elect_one());
                        ++step;
                    }
                    if (j + 1 < nt) {
                        mma_heads<HD>(ts, desc_q, desc_k + rk.slot * (TILE >> 4), ksteps, idesc_s);
                        commit(&s_full[t], elect_one());
                    }
                    turns.pass();
                    ++round;
                    commit(&empty[rv.slot], elect_one());
                    two(rv);
                    if (j + 1 < plan.steps) {
                        commit(&empty[rk.slot], elect_one());
                        if (j + 2 == nt) commit(&q_empty, elect_one());    // the last scores that read the queries
                        two(rk);
                    }
                }
            }
            if (!ok) break;
            ++queries;
            outputs += nt > 0;
        }
        commit(&mma_done[t], elect_one());
        wait.drain(&mma_done[t], 0);
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kFwdRegsSoftmax));
        const int t = warp >> 2, r = (warp & 3) * 32 + lane, row = kRows * t + r;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + 128 * t + lanes, to = tmem + 256 + O_COLS * t + lanes;
        const uint32_t tp = OWN_P ? tmem + 384 + 64 * t + lanes : ts;
        const float2 c2 = make_float2(p.c, p.c);
        uint32_t step = 0, outputs = 0;
        bool ok = true;
        while (ok && queue.next(items, wait, item)) {
            const FwdPlan plan(p, item);
            const int nt = t ? plan.n[1] : plan.n[0], rows = t ? plan.rows[1] : plan.rows[0];
            // keys this row sees, and those that every row of the tile sees, from the first of this CTA's on
            const int len = item.other_len, first = plan.j0 * kRows;
            const int limit = (p.causal ? min(len, max(0, row + item.diag + 1)) : len) - first;
            const int common = (p.causal ? min(len, kRows * t + item.diag + 1) : len) - first;
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < nt; ++j, ++step) {
                ok = wait(&s_full[t], step);
                if (!ok) break;
                fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i) ld32(ts + 32 * i, s[i]);
                ld_wait();
#pragma unroll
                for (int i = 0; i < 4; ++i) fence32(s[i]);
                if constexpr (OWN_P) {                     // the next scores may come
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_read[t]);
                }
                if ((j + 1) * kRows > common) {
                    // most blocks of 32 columns are on one side of the mask for the whole warp
                    const int lim = limit - j * kRows, least = __reduce_min_sync(~0u, lim);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (least < 32 * i + 32)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (32 * i + e >= lim) s[i][e] = 0xFF800000u;
                }
                float mx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mx[i] = __uint_as_float(s[i][0]);
#pragma unroll
                    for (int e = 1; e < 32; ++e) mx[i] = fmaxf(mx[i], __uint_as_float(s[i][e]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.c;
                const bool grow = top > m + 8.0f;
                if (__any_sync(~0u, grow)) {
                    const float mn = grow ? top : m, f = grow ? ex2(m - mn) : 1.0f;
                    m = mn;
                    l *= f;
                    if (j > 0) {
                        if constexpr (OWN_P) {
                            ok = wait(&pv_done[t], step - 1);
                            if (!ok) break;
                            fence_after();
                        }
#pragma unroll 1
                        for (int i = 0; i < p.dim; i += 32) {
                            uint32_t o[32];
                            ld32(to + i, o);
                            ld_wait();
                            fence32(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            st32(to + i, o);
                        }
                    }
                }
                const float neg = m == -INFINITY ? 0.0f : -m;
                const float2 neg2 = make_float2(neg, neg);
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                uint32_t w[4][16];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 x = make_float2(__uint_as_float(s[i][2 * e]), __uint_as_float(s[i][2 * e + 1]));
                        x = __ffma2_rn(x, c2, neg2);
                        x = make_float2(ex2(x.x), ex2(x.y));
                        sum[e & 1] = __fadd2_rn(sum[e & 1], x);
                        w[i][e] = pack_bf16(x.x, x.y);
                    }
                    if constexpr (!OWN_P) st16(tp + 16 * i, w[i]);
                }
                if constexpr (OWN_P) {                     // the last P has to have been read
                    if (j > 0) {
                        ok = wait(&pv_done[t], step - 1);
                        if (!ok) break;
                        fence_after();
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) st16(tp + 16 * i, w[i]);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                st_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[t]);
            }
            if (ok && nt > 0) {
                ok = wait(&pv_done[t], OWN_P ? step - 1 : outputs);
                fence_after();
            }
            if (!ok) break;
            if (rows > 0) {                                // whole warps: the TMEM loads are collective
                const bool store = r < rows;
                const int64_t tok = item.first + (store ? row : 0), at = (int64_t)item.head * p.tq + tok;
                bf16* dst = p.out.at(tok, item.head);
                float* sum = p.part_sums + (((int64_t)item.part * p.tq + tok) * p.heads + item.head) * p.dim;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                if (nt == 0) {
                    if (store && p.parts == 1) store_zeros(dst, p.dim);
                    if (store && p.parts > 1) store_zeros(sum, p.dim);
                } else {
#pragma unroll 1
                    for (int i = 0; i < p.dim; i += 32) {
                        uint32_t o[32];
                        ld32(to + i, o);
                        ld_wait();
                        fence32(o);
                        if (p.parts == 1) store32(p.out, item.first + row - lane, item.head, rows - (r - lane), i, p.dim, o, inv);
                        if (store && p.parts > 1) store32(sum, i, p.dim, o, inv);
                    }
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&o_empty[t]);
                    ++outputs;
                }
                if (store)
                    (p.parts == 1 ? p.lse : p.part_lse + (int64_t)item.part * p.heads * p.tq)[at] =
                        l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 9) {
        fence_after();
        tmem_free_all(tmem);
    }
}

// ---------------------------------------------------------------------------- backward, dQ
// Warps 0-7: a row per thread, warps 0-3 the first 64 keys of a tile, warps 4-7 the last 64; warp 8: TMA; warp 9:
// the MMAs of S and dQ; warp 10: those of dP; warp 11: the next tiles to work on.  TMEM: S of even and odd steps at 0
// and 128 (dS takes S's place, in the columns its own warps have read), dP at 256, dQ at 384.  dQ of a step and S of the one
// after next are issued as soon as the step's dS is there, the next dP as soon as the present one has been read:
// the warps find both done.  (With dQ, S and dP issued in turns, each step waited for one round of the two
// MMA warps: 8192 tokens, 40 / 8 heads of 128, causal, whole backward pass 1350 us, 1296 without.)  The first
// kernel of the backward pass: it also leaves delta, computed while the last tile's dQ is still under way.
constexpr int kDqThreads = 384;
template <int HD> struct Dq {
    static constexpr int TILE = kRows * HD * 2;
    static constexpr int KS = HD == 128 ? 3 : 5, VS = HD == 128 ? 2 : 3;
    struct Ctl {
        uint64_t q_full, q_empty, k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], s_full[2], dp_full, dp_read, ds_ready[2], dq_full,
            dq_empty, delta_ready, mma_done[2];
        Queue queue;
        uint32_t tmem_slot, abort_flag;
        float delta[2][kRows];                             // of two items in turn
    };
    static constexpr int TILES = (2 + KS + VS) * TILE;     // Q, dO, the K's, the V's
    static constexpr int SMEM = TILES + (int)sizeof(Ctl);
    static_assert(SMEM <= 232448 && SMEM > 116 * 1024, "one CTA fits an SM (TMEM is taken whole)");
};

template <int HD>
__global__ void __launch_bounds__(kDqThreads, 1)
dq_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
          const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmdo, const Params p) {
    using Cfg = Dq<HD>;
    constexpr int TILE = Cfg::TILE, KS = Cfg::KS, VS = Cfg::VS;
    extern __shared__ __align__(1024) uint8_t tiles_smem[];
    uint8_t* smem_q = tiles_smem;
    uint8_t* smem_do = smem_q + TILE;
    uint8_t* ring_k = smem_do + TILE;
    uint8_t* ring_v = ring_k + KS * TILE;
    typename Cfg::Ctl& ctl = *reinterpret_cast<typename Cfg::Ctl*>(tiles_smem + Cfg::TILES);
    const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        mbar_init(&ctl.q_full, 1);
        mbar_init(&ctl.q_empty, 2);
        for (int i = 0; i < KS; ++i) {
            mbar_init(&ctl.k_full[i], 1);
            mbar_init(&ctl.k_empty[i], 1);
        }
        for (int i = 0; i < VS; ++i) {
            mbar_init(&ctl.v_full[i], 1);
            mbar_init(&ctl.v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.s_full[i], 1);
            mbar_init(&ctl.ds_ready[i], 8);
            mbar_init(&ctl.mma_done[i], 1);
        }
        mbar_init(&ctl.dp_full, 1);
        mbar_init(&ctl.dp_read, 8);
        mbar_init(&ctl.dq_full, 1);
        mbar_init(&ctl.dq_empty, 8);
        mbar_init(&ctl.delta_ready, 8);
        ctl.queue.init(11);
        ctl.abort_flag = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) tmem_alloc_all(&ctl.tmem_slot);
    pdl_wait();
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = uniform(ctl.tmem_slot);
    const Wait wait{p.timeout_ns, &ctl.abort_flag, p.dev_status};
    Ring<2> items;
    Item item;
    // an item's key tiles: j0 .. j0 + steps - 1
    auto share_of = [&](const Item& it) {
        const int keys = p.causal ? min(it.other_len, max(0, it.rows + it.diag)) : it.other_len;
        return Share(p, it.part, (keys + kRows - 1) / kRows);
    };

    if (warp == 11) {
        ctl.queue.template feed<kRows>(p, true, p.heads, wait);
    } else if (warp == 8) {
        Ring<KS> rk;
        Ring<VS> rv;
        uint32_t got_k = 0, got_v = 0, queries = 0;
        bool ok = true;
        while (ok && ctl.queue.next(items, wait, item)) {
            const Share mine = share_of(item);
            if (mine.count == 0) continue;
            const int hk = item.head / (p.heads / p.kv_heads);
            if (lane == 0) {
                ok = wait(&ctl.q_empty, queries ^ 1u);
                if (ok) {
                    mbar_arrive_expect_tx(&ctl.q_full, 2 * TILE);
                    load_tile<HD>(smem_q, &tmq, item.first, item.head, &ctl.q_full);
                    load_tile<HD>(smem_do, &tmdo, item.first, item.head, &ctl.q_full);
                    ++queries;
                }
                for (int j = 0; ok && j < mine.count; ++j) {
                    const int64_t tok = item.other + (int64_t)(mine.first + j) * kRows;
                    ok = wait(&ctl.k_empty[rk.slot], rk.phase ^ 1u);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&ctl.k_full[rk.slot], TILE);
                    load_tile<HD>(ring_k + rk.slot * TILE, &tmk, tok, hk, &ctl.k_full[rk.slot]);
                    ++got_k;
                    rk.next();
                    ok = wait(&ctl.v_empty[rv.slot], rv.phase ^ 1u);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&ctl.v_full[rv.slot], TILE);
                    load_tile<HD>(ring_v + rv.slot * TILE, &tmv, tok, hk, &ctl.v_full[rv.slot]);
                    ++got_v;
                    rv.next();
                }
            }
            ok = __all_sync(~0u, ok);
        }
        if (lane == 0 && ctl.abort_flag) {                 // the copies in flight land first
            if (queries) wait.drain(&ctl.q_full, (queries - 1) & 1u);
#pragma unroll 1
            for (uint32_t i = got_k > KS ? got_k - KS : 0; i < got_k; ++i) wait.drain(&ctl.k_full[i % KS], (i / KS) & 1u);
#pragma unroll 1
            for (uint32_t i = got_v > VS ? got_v - VS : 0; i < got_v; ++i) wait.drain(&ctl.v_full[i % VS], (i / VS) & 1u);
        }
    } else if (warp == 9) {
        const uint32_t idesc_s = idesc_bf16(kRows, false, p.scale < 0.0f);
        const uint32_t idesc_dq = idesc_bf16((p.dim + 15) & ~15, true, false);
        const int ksteps = (p.dim + 15) / 16;
        const uint32_t desc_q = uniform(desc_k_major(smem_addr(smem_q)));
        const uint32_t desc_k = uniform(desc_k_major(smem_addr(ring_k))), desc_kt = uniform(desc_mn_major(smem_addr(ring_k)));
        Ring<KS> rs, rq;                                   // the next K for S, and for dQ
        uint32_t queries = 0, gs = 0, gq = 0;              // items, and steps whose S and dQ have been issued
        bool ok = true;
        while (ok && ctl.queue.next(items, wait, item)) {
            const Share mine = share_of(item);
            const int steps = uniform(mine.count), len = uniform(item.other_len - mine.first * kRows);
            if (steps == 0) continue;
            const bool neighbours = uniform((int)(item.other + item.other_len < p.tk)) != 0;
            auto issue_s = [&](int j) {
                const int valid = len - j * kRows;
                if (!wait.all(&ctl.k_full[rs.slot], rs.phase)) return false;
                if (valid < kRows && neighbours) zero_tail<HD>(ring_k + rs.slot * TILE, valid);
                mma_heads<HD>(tmem + 128 * (gs & 1), desc_q, desc_k + rs.slot * (TILE >> 4), ksteps, idesc_s);
                commit(&ctl.s_full[gs & 1], elect_one());
                if (j + 1 == steps) commit(&ctl.q_empty, elect_one());
                rs.next();
                ++gs;
                return true;
            };
            ok = wait.all(&ctl.q_full, queries) && issue_s(0) && (steps < 2 || issue_s(1));
            for (int j = 0; ok && j < steps; ++j) {
                ok = (j > 0 || wait.all(&ctl.dq_empty, queries ^ 1u)) && wait.all(&ctl.ds_ready[gq & 1], gq >> 1);
                if (!ok) break;
                fence_after();
                const uint32_t ds = tmem + 128 * (gq & 1);
                mma_rows(tmem + 384, ds, ds + 64, desc_kt + rq.slot * (TILE >> 4), idesc_dq, j > 0);
                commit(&ctl.k_empty[rq.slot], elect_one());
                if (j + 1 == steps) commit(&ctl.dq_full, elect_one());
                rq.next();
                ++gq;
                if (j + 2 < steps) ok = issue_s(j + 2);
            }
            ++queries;
        }
        commit(&ctl.mma_done[0], elect_one());
        wait.drain(&ctl.mma_done[0], 0);
    } else if (warp == 10) {
        // V's rows past the sequence reach only columns of dP that are masked: no need to zero them
        const uint32_t idesc_dp = idesc_bf16(kRows, false, false);
        const int ksteps = (p.dim + 15) / 16;
        const uint32_t desc_do = uniform(desc_k_major(smem_addr(smem_do))), desc_v = uniform(desc_k_major(smem_addr(ring_v)));
        Ring<VS> rv;
        uint32_t queries = 0, g = 0;
        bool ok = true;
        while (ok && ctl.queue.next(items, wait, item)) {
            const int steps = uniform(share_of(item).count);
            if (steps == 0) continue;
            ok = wait.all(&ctl.q_full, queries);
            for (int j = 0; ok && j < steps; ++j) {
                ok = wait.all(&ctl.v_full[rv.slot], rv.phase) && (g == 0 || wait.all(&ctl.dp_read, g - 1));
                if (!ok) break;
                fence_after();
                mma_heads<HD>(tmem + 256, desc_do, desc_v + rv.slot * (TILE >> 4), ksteps, idesc_dp);
                commit(&ctl.dp_full, elect_one());
                commit(&ctl.v_empty[rv.slot], elect_one());
                if (j + 1 == steps) commit(&ctl.q_empty, elect_one());
                rv.next();
                ++g;
            }
            ++queries;
        }
        commit(&ctl.mma_done[1], elect_one());
        wait.drain(&ctl.mma_done[1], 0);
    } else {
        const int half = warp >> 2, row0 = (warp & 3) * 32, r = row0 + lane;
        const uint32_t lanes = (uint32_t)row0 << 16;
        const uint32_t tdp = tmem + 256 + 64 * half + lanes;
        const float2 c2 = make_float2(p.c, p.c);
        // delta = dout . out of row r; -lse log2(e).  A warp takes 16 rows, HD / 8 lanes each: read a row per lane, a load
        // touches 32 lines.
        float d = 0.0f, neg = 0.0f;
        uint32_t buf = 0;
        auto row_stats = [&](const Item& it) {
            constexpr int LANES = HD / 8, N = HD / 16;     // of a row; rows of a lane
            const int sub = lane / LANES, c = lane % LANES;
            uint4 o[N], g[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int row = 16 * warp + 16 / N * i + sub;
                o[i] = g[i] = make_uint4(0, 0, 0, 0);
                if (row < it.rows && 8 * c < p.dim) {
                    o[i] = *reinterpret_cast<const uint4*>(p.out.at(it.first + row, it.head) + 8 * c);
                    g[i] = *reinterpret_cast<const uint4*>(p.dout.at(it.first + row, it.head) + 8 * c);
                }
            }
            const bool in = r < it.rows;
            const int64_t at = (int64_t)it.head * p.tq + it.first + (in ? r : 0);
            const float lse = in ? p.lse[at] : 0.0f;
            float sum[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t x[4] = {o[i].x, o[i].y, o[i].z, o[i].w}, y[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
                sum[i] = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[i] += bf16_lo(x[e]) * bf16_lo(y[e]) + bf16_hi(x[e]) * bf16_hi(y[e]);
            }
            // N rows' sums over 2 N lanes: a lane keeps half of its rows in each round, row c / 2 at last
#pragma unroll
            for (int n = N / 2; n; n >>= 1) {
                const bool upper = c & (2 * n);
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float keep = upper ? sum[i + n] : sum[i], give = upper ? sum[i] : sum[i + n];
                    sum[i] = keep + __shfl_xor_sync(~0u, give, 2 * n);
                }
            }
            sum[0] += __shfl_xor_sync(~0u, sum[0], 1);
            if (!(c & 1)) ctl.delta[buf & 1][16 * warp + 16 / N * (c / 2) + sub] = sum[0];
            // all warps' rows: a barrier with a bounded wait; two buffers take turns
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.delta_ready);
            if (!wait.all(&ctl.delta_ready, buf)) return false;
            d = ctl.delta[buf & 1][r];
            ++buf;
            if (in && half == 0 && it.part == 0) p.delta[at] = d;
            neg = lse == -INFINITY ? -INFINITY : -lse * kLog2e;            // a row that sees no key: P = 0
            return true;
        };
        uint32_t queries = 0, g = 0;
        bool ok = ctl.queue.next(items, wait, item) && row_stats(item);
        while (ok) {
            const Share mine = share_of(item);
            const int steps = mine.count, first = mine.first * kRows;
            const bool in = r < item.rows;
            const int64_t tok = item.first + (in ? r : 0);
            const int limit = (p.causal ? min(item.other_len, max(0, r + item.diag + 1)) : item.other_len) - first;
            const int common = (p.causal ? min(item.other_len, item.diag + 1) : item.other_len) - first;
            const float2 neg2 = make_float2(neg, neg), delta2 = make_float2(-d, -d);
            for (int j = 0; j < steps; ++j, ++g) {
                const uint32_t ts = tmem + 128 * (g & 1) + 64 * half + lanes;
                ok = wait(&ctl.s_full[g & 1], g >> 1);
                if (!ok) break;
                fence_after();
                uint32_t s[2][32], u[2][32], w[32];
                ld32(ts, s[0]);
                ld32(ts + 32, s[1]);
                ld_wait();
                fence32(s[0]);
                fence32(s[1]);
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    float2 x = make_float2(__uint_as_float(s[i >> 5][i & 31]), __uint_as_float(s[i >> 5][(i & 31) + 1]));
                    x = __ffma2_rn(x, c2, neg2);
                    s[i >> 5][i & 31] = __float_as_uint(ex2(x.x));
                    s[i >> 5][(i & 31) + 1] = __float_as_uint(ex2(x.y));
                }
                ok = wait(&ctl.dp_full, g);
                if (!ok) break;
                fence_after();
                ld32(tdp, u[0]);
                ld32(tdp + 32, u[1]);
                ld_wait();
                fence32(u[0]);
                fence32(u[1]);
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.dp_read);
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    const float2 pr = make_float2(__uint_as_float(s[i >> 5][i & 31]), __uint_as_float(s[i >> 5][(i & 31) + 1]));
                    float2 x = make_float2(__uint_as_float(u[i >> 5][i & 31]), __uint_as_float(u[i >> 5][(i & 31) + 1]));
                    x = __fmul2_rn(pr, __fadd2_rn(x, delta2));
                    w[i >> 1] = pack_bf16(x.x, x.y);
                }
                if ((j + 1) * kRows > common) {            // masked pairs count for nothing, whatever they hold
                    const int lim = limit - j * kRows - 64 * half;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (2 * i >= lim) w[i] = 0u;
                        else if (2 * i + 1 >= lim) w[i] &= 0xFFFFu;
                    }
                }
                st32(ts, w);
                st_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.ds_ready[g & 1]);
            }
            if (!ok) break;
            // the next item's delta while this one's dQ is finished
            Item next;
            const bool more = ctl.queue.next(items, wait, next) && row_stats(next);
            bf16* dst = p.dq.at(tok, item.head);
            float* sum = p.part_sums + (((int64_t)item.part * p.tq + tok) * p.heads + item.head) * p.dim;
            if (steps == 0) {
                if (in && half == 0 && p.parts == 1) store_zeros(dst, p.dim);
                if (in && half == 0 && p.parts > 1) store_zeros(sum, p.dim);
            } else {
                ok = wait(&ctl.dq_full, queries);
                if (!ok) break;
                fence_after();
#pragma unroll 1
                for (int i = 64 * half; i < min(p.dim, 64 * half + 64); i += 32) {
                    uint32_t v[32];
                    ld32(tmem + 384 + i + lanes, v);
                    ld_wait();
                    fence32(v);
                    if (p.parts == 1) store32(p.dq, item.first + row0, item.head, item.rows - row0, i, p.dim, v, p.scale);
                    if (in && p.parts > 1) store32(sum, i, p.dim, v, p.scale);
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.dq_empty);
                ++queries;
            }
            item = next;
            ok = more;
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 9) {
        fence_after();
        tmem_free_all(tmem);
    }
}

// ---------------------------------------------------------------------------- backward, dK and dV
// Warps 0-7: a key per thread, warps 0-3 the first 64 queries of a tile, warps 4-7 the last 64; warp 8: TMA; warp 9:
// the MMAs of S and dV; warp 10: those of dP and dK; warp 11: lse and delta of the queries.  A step is one query tile of one of the heads that read the
// key head.  TMEM: S^T then P^T at 0, dP^T then dS^T at 128, dV at 256, dK at 384.  The tensor cores do dV of a
// step and S of the next while the warps compute dS, and dK and the next dP while they compute P.
constexpr int kDkvThreads = 384;
// Q is held from its first product to its last, a step and a half: with two slots a load had half a
// step's time and the MMAs waited for it (a third slot took 0.13 ms off 1.76 ms for the whole backward
// pass at 8192 tokens, 40 / 8 heads of 128, causal).
template <int HD> struct Dkv {
    static constexpr int TILE = kRows * HD * 2;
    static constexpr int QS = HD == 128 ? 3 : 4, DS = HD == 128 ? 2 : 4;
    struct Ctl {
        float stat[2][2][kRows];                           // per slot: -lse log2(e), -delta
        uint64_t kv_full, q_full[QS], q_empty[QS], do_full[DS], do_empty[DS], st_full[2], st_empty[2], s_full, dp_full,
            p_ready, ds_ready, turn[2], mma_done[2];
        Item item;
        uint32_t tmem_slot, abort_flag;
    };
    static constexpr int TILES = (2 + QS + DS) * TILE;     // K, V, the Q's, the dO's
    static constexpr int SMEM = TILES + (int)sizeof(Ctl);
    static_assert(SMEM <= 232448 && SMEM > 116 * 1024, "one CTA fits an SM (TMEM is taken whole)");
};

template <int HD>
__global__ void __launch_bounds__(kDkvThreads, 1)
dkv_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
           const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmdo, const Params p) {
    using Cfg = Dkv<HD>;
    constexpr int TILE = Cfg::TILE, QS = Cfg::QS, DS = Cfg::DS;
    extern __shared__ __align__(1024) uint8_t tiles_smem[];
    uint8_t* smem_k = tiles_smem;
    uint8_t* smem_v = smem_k + TILE;
    uint8_t* ring_q = smem_v + TILE;
    uint8_t* ring_do = ring_q + QS * TILE;
    typename Cfg::Ctl& ctl = *reinterpret_cast<typename Cfg::Ctl*>(tiles_smem + Cfg::TILES);
    const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        mbar_init(&ctl.kv_full, 1);
        for (int i = 0; i < QS; ++i) {
            mbar_init(&ctl.q_full[i], 1);
            mbar_init(&ctl.q_empty[i], 2);
        }
        for (int i = 0; i < DS; ++i) {
            mbar_init(&ctl.do_full[i], 1);
            mbar_init(&ctl.do_empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.st_full[i], 1);
            mbar_init(&ctl.st_empty[i], 8);
            mbar_init(&ctl.turn[i], 1);
            mbar_init(&ctl.mma_done[i], 1);
        }
        mbar_init(&ctl.s_full, 1);
        mbar_init(&ctl.dp_full, 1);
        mbar_init(&ctl.p_ready, 8);
        mbar_init(&ctl.ds_ready, 8);
        ctl.abort_flag = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) tmem_alloc_all(&ctl.tmem_slot);
    pdl_wait();
    if (warp == 8) find_item<kRows>(p, false, p.kv_heads, blockIdx.x, &ctl.item);
    fence_before();
    __syncthreads();
    fence_after();
    const Item& item = ctl.item;
    const uint32_t tmem = uniform(ctl.tmem_slot);
    const Wait wait{p.timeout_ns, &ctl.abort_flag, p.dev_status};
    const int share = p.heads / p.kv_heads;
    // With the causal mask key r of the tile is seen by the queries from r + diag on.
    int first_tile = 0, tiles = 0, steps = 0;
    if (item.valid) {
        if (p.causal) first_tile = max(0, item.diag) / kRows;
        tiles = max(0, (item.other_len + kRows - 1) / kRows - first_tile);
        steps = tiles * share;
    }
    const Share mine(p, item.part, steps);
    steps = uniform(mine.count);
    first_tile = uniform(first_tile);
    // the steps in order: the query tiles of the first head, of the second, ...
    struct Step {
        int head, tile, tiles;
        __device__ __forceinline__ void next() {
            if (++tile == tiles) {
                tile = 0;
                ++head;
            }
        }
    };
    const int ahead = mine.first > 0 ? mine.first / tiles : 0;
    const Step begin{uniform(item.head * share + ahead), uniform(mine.first - ahead * tiles), uniform(tiles)};
    auto row_of = [&](const Step& s) { return (first_tile + s.tile) * kRows; };

    if (warp == 8 && steps > 0) {
        if (lane == 0) {
            mbar_arrive_expect_tx(&ctl.kv_full, 2 * TILE);
            load_tile<HD>(smem_k, &tmk, item.first, item.head, &ctl.kv_full);
            load_tile<HD>(smem_v, &tmv, item.first, item.head, &ctl.kv_full);
            int got_q = 0, got_do = 0;
            Ring<QS> q;
            Ring<DS> d;
            Step s = begin;
            for (int i = 0; i < steps; ++i, s.next()) {
                if (!wait(&ctl.q_empty[q.slot], q.phase ^ 1u)) break;
                mbar_arrive_expect_tx(&ctl.q_full[q.slot], TILE);
                load_tile<HD>(ring_q + q.slot * TILE, &tmq, item.other + row_of(s), s.head, &ctl.q_full[q.slot]);
                got_q = i + 1;
                if (!wait(&ctl.do_empty[d.slot], d.phase ^ 1u)) break;
                mbar_arrive_expect_tx(&ctl.do_full[d.slot], TILE);
                load_tile<HD>(ring_do + d.slot * TILE, &tmdo, item.other + row_of(s), s.head, &ctl.do_full[d.slot]);
                got_do = i + 1;
                q.next();
                d.next();
            }
            if (got_do < steps) {                          // aborted: the copies in flight land first
                wait.drain(&ctl.kv_full, 0);
#pragma unroll 1
                for (int i = max(0, got_q - QS); i < got_q; ++i) wait.drain(&ctl.q_full[i % QS], i / QS);
#pragma unroll 1
                for (int i = max(0, got_do - DS); i < got_do; ++i) wait.drain(&ctl.do_full[i % DS], i / DS);
            }
        }
    } else if (warp == 11 && steps > 0) {
        // a step's values are fetched while the step before waits for its slot
        Ring<2> r;
        Step s = begin;
        float l[4], d[4];
        auto fetch = [&] {
            const int64_t at = (int64_t)s.head * p.tq + item.other;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int q = row_of(s) + lane + 32 * e;
                const bool in = q < item.other_len;
                l[e] = in ? p.lse[at + q] : -INFINITY;
                d[e] = in ? p.delta[at + q] : 0.0f;
            }
        };
        fetch();
        for (int i = 0; i < steps; ++i, r.next()) {
            if (!wait(&ctl.st_empty[r.slot], r.phase ^ 1u)) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ctl.stat[r.slot][0][lane + 32 * e] = l[e] == -INFINITY ? -INFINITY : -l[e] * kLog2e;   // such queries: P = 0
                ctl.stat[r.slot][1][lane + 32 * e] = -d[e];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.st_full[r.slot]);
            s.next();
            if (i + 1 < steps) fetch();
        }
    } else if ((warp == 9 || warp == 10) && steps > 0) {
        // The same loop for both, on other tiles: A = K or V once with the `in` tile (a first product into ts), then,
        // when the warps have put P or dS there, with the `out` tile (the sum at to).
        const uint32_t idesc_out = idesc_bf16((p.dim + 15) & ~15, true, false);
        const bool neighbours = item.other + item.other_len < p.tq;
        const int ksteps = (p.dim + 15) / 16, len = uniform(item.other_len);
        auto clean = [&](uint8_t* tile, const Step& s) {   // rows of a neighbouring sequence
            const int valid = len - row_of(s);
            if (valid < kRows && neighbours) zero_tail<HD>(tile, valid);
        };
        auto chain = [&](auto in, auto out, int w, uint32_t idesc_in, const uint8_t* a, uint8_t* ring_in, uint8_t* ring_out,
                         uint64_t* in_full, uint64_t* in_empty, uint64_t* out_full, uint64_t* out_empty, uint64_t* in_done,
                         uint64_t* ready) {
            const uint32_t desc_a = uniform(desc_k_major(smem_addr(a)));
            const uint32_t desc_in = uniform(desc_k_major(smem_addr(ring_in))), desc_out = uniform(desc_mn_major(smem_addr(ring_out)));
            const uint32_t ts = tmem + 128 * w, to = tmem + 256 + 128 * w;
            const Turns turns{ctl.turn, wait, w};
            Step si = begin, so = begin;
            auto tile_in = [&] {
                if (!wait.all(&in_full[in.slot], in.phase)) return false;
                clean(ring_in + in.slot * TILE, si);
                return true;
            };
            auto issue_in = [&] {
                mma_heads<HD>(ts, desc_a, desc_in + in.slot * (TILE >> 4), ksteps, idesc_in);
                commit(in_done, elect_one());
                turns.pass();
                commit(&in_empty[in.slot], elect_one());
                in.next();
                si.next();
            };
            // rounds: S 0, dP 0; dV 0 and S 1, dK 0 and dP 1; ...
            bool ok = wait.all(&ctl.kv_full, 0) && tile_in() && turns.take(0);
            if (ok) issue_in();
            for (int i = 0; ok && i < steps; ++i) {
                ok = wait.all(&out_full[out.slot], out.phase) && (i + 1 >= steps || tile_in());
                if (!ok) break;
                clean(ring_out + out.slot * TILE, so);
                ok = turns.take(i + 1) && wait.all(ready, i);
                if (!ok) break;
                fence_after();
                mma_rows(to, ts, ts + 64, desc_out + out.slot * (TILE >> 4), idesc_out, i > 0);
                commit(&out_empty[out.slot], elect_one());
                if (i + 1 < steps) issue_in();
                else turns.pass();
                out.next();
                so.next();
            }
            commit(&ctl.mma_done[w], elect_one());
            wait.drain(&ctl.mma_done[w], 0);
        };
        if (warp == 9)
            chain(Ring<QS>{}, Ring<DS>{}, 0, idesc_bf16(kRows, false, p.scale < 0.0f), smem_k, ring_q, ring_do, ctl.q_full,
                  ctl.q_empty, ctl.do_full, ctl.do_empty, &ctl.s_full, &ctl.p_ready);
        else
            chain(Ring<DS>{}, Ring<QS>{}, 1, idesc_bf16(kRows, false, false), smem_v, ring_do, ring_q, ctl.do_full,
                  ctl.do_empty, ctl.q_full, ctl.q_empty, &ctl.dp_full, &ctl.ds_ready);
    } else if (warp < 8 && item.valid) {
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + 64 * half + lanes, tdp = tmem + 128 + 64 * half + lanes;
        const float2 c2 = make_float2(p.c, p.c);
        bool ok = true;
        Ring<2> st;
        Step step = begin;
        for (int i = 0; i < steps; ++i, step.next(), st.next()) {
            ok = wait(&ctl.st_full[st.slot], st.phase);
            if (!ok) break;
            // read ahead of S: beside MMAs that take all of shared memory's bandwidth these loads are slow
            float4 lse4[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) lse4[e] = reinterpret_cast<const float4*>(&ctl.stat[st.slot][0][64 * half])[e];
            ok = wait(&ctl.s_full, i);
            if (!ok) break;
            fence_after();
            uint32_t s[2][32];
            ld32(ts, s[0]);
            ld32(ts + 32, s[1]);
            ld_wait();
            fence32(s[0]);
            fence32(s[1]);
            const float4* del4 = reinterpret_cast<const float4*>(&ctl.stat[st.slot][1][64 * half]);
            const int from = r + item.diag - row_of(step) - 64 * half;     // masked pairs: queries before r + diag
            auto probabilities = [&](auto masked) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        uint32_t* v = &s[h >> 1][(h & 1) * 16 + e];
                        const float4 n4 = lse4[h * 4 + (e >> 2)];
                        const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), c2, make_float2(n4.x, n4.y));
                        const float2 y = __ffma2_rn(make_float2(__uint_as_float(v[2]), __uint_as_float(v[3])), c2, make_float2(n4.z, n4.w));
                        float f[4] = {ex2(x.x), ex2(x.y), ex2(y.x), ex2(y.y)};
                        if constexpr (decltype(masked)::value)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (h * 16 + e + k < from) f[k] = 0.0f;
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = __float_as_uint(f[k]);
                        w[e >> 1] = pack_bf16(f[0], f[1]);
                        w[(e >> 1) + 1] = pack_bf16(f[2], f[3]);
                    }
                    st8(ts + 8 * h, w);
                }
            };
            if (p.causal && kRows - 1 + item.diag > row_of(step)) probabilities(std::true_type{});
            else probabilities(std::false_type{});
            st_wait();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.p_ready);
            ok = wait(&ctl.dp_full, i);
            if (!ok) break;
            fence_after();
            uint32_t g[2][32];
            ld32(tdp, g[0]);
            ld32(tdp + 32, g[1]);
            ld_wait();
            fence32(g[0]);
            fence32(g[1]);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const uint32_t *v = &s[h >> 1][(h & 1) * 16 + e], *u = &g[h >> 1][(h & 1) * 16 + e];
                    const float4 n4 = del4[h * 4 + (e >> 2)];
                    const float2 x = __fmul2_rn(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])),
                                                __fadd2_rn(make_float2(__uint_as_float(u[0]), __uint_as_float(u[1])), make_float2(n4.x, n4.y)));
                    const float2 y = __fmul2_rn(make_float2(__uint_as_float(v[2]), __uint_as_float(v[3])),
                                                __fadd2_rn(make_float2(__uint_as_float(u[2]), __uint_as_float(u[3])), make_float2(n4.z, n4.w)));
                    w[e >> 1] = pack_bf16(x.x, x.y);
                    w[(e >> 1) + 1] = pack_bf16(y.x, y.y);
                }
                st8(tdp + 8 * h, w);
            }
            st_wait();
            fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&ctl.ds_ready);
                mbar_arrive(&ctl.st_empty[st.slot]);
            }
        }
        const bool in = r < item.rows;
        const int64_t tok = item.first + (in ? r : 0);
        bf16* dst = half ? p.dk.at(tok, item.head) : p.dv.at(tok, item.head);
        // parts: [part][dV, dK][tk, kv_heads, dim]
        float* sum = p.part_sums + (((int64_t)(2 * item.part + half) * p.tk + tok) * p.kv_heads + item.head) * p.dim;
        if (steps == 0) {
            if (in && p.parts == 1) store_zeros(dst, p.dim);
            if (in && p.parts > 1) store_zeros(sum, p.dim);
        } else if (ok) {
            ok = wait(&ctl.mma_done[half], 0);
            fence_after();
            if (ok)
#pragma unroll 1
                for (int i = 0; i < p.dim; i += 32) {
                    uint32_t v[32];
                    ld32(tmem + 256 + 128 * half + i + lanes, v);
                    ld_wait();
                    fence32(v);
                    if (p.parts == 1)
                        store32(half ? p.dk : p.dv, item.first + r - lane, item.head, item.rows - (r - lane), i, p.dim, v,
                                half ? p.scale : 1.0f);
                    if (in && p.parts > 1) store32(sum, i, p.dim, v, half ? p.scale : 1.0f);
                }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 9) {
        fence_after();
        tmem_free_all(tmem);
    }
}

// ---------------------------------------------------------------------------- joins
// What the parts of a tile left, added in their order; a thread takes 8 elements of a token and head.  dK and dV: blockIdx.y
// says which.
constexpr int kJoinThreads = 256;

__device__ __forceinline__ void add8(float (&s)[8], const float* p, float f) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    s[0] += f * a.x; s[1] += f * a.y; s[2] += f * a.z; s[3] += f * a.w;
    s[4] += f * b.x; s[5] += f * b.y; s[6] += f * b.z; s[7] += f * b.w;
}
__device__ __forceinline__ void store8(bf16* dst, const float (&s)[8]) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]), pack_bf16(s[6], s[7]));
}

__global__ void __launch_bounds__(kJoinThreads) join_sums_kernel(const float* sums, int parts, int64_t part_stride, int64_t which_stride,
                                                                 int64_t tokens, int heads, int dim, Heads first, Heads second) {
    pdl_launch_dependents();
    pdl_wait();
    const int groups = dim / 8;
    const int64_t i = blockIdx.x * (int64_t)kJoinThreads + threadIdx.x;
    if (i >= tokens * heads * groups) return;
    const float* p = sums + blockIdx.y * which_stride + i * 8;
    float s[8] = {};
#pragma unroll 1
    for (int k = 0; k < parts; ++k) add8(s, p + k * part_stride, 1.0f);
    const int64_t th = i / groups;
    store8((blockIdx.y ? second : first).at(th / heads, (int)(th % heads)) + (i % groups) * 8, s);
}

// Forward: each part's output is that of its keys alone; their weights are exp(lse of the part - lse of all).
__global__ void __launch_bounds__(kJoinThreads) join_out_kernel(const Params p) {
    pdl_launch_dependents();
    pdl_wait();
    const int groups = p.dim / 8;
    const int64_t i = blockIdx.x * (int64_t)kJoinThreads + threadIdx.x, part_stride = p.tq * p.heads * p.dim;
    if (i >= p.tq * p.heads * groups) return;
    const int64_t th = i / groups, tok = th / p.heads;
    const int h = (int)(th % p.heads);
    const float* lse = p.part_lse + h * p.tq + tok;
    const int64_t lse_stride = p.heads * p.tq;
    float top = -INFINITY, total = 0.0f;
#pragma unroll 1
    for (int k = 0; k < p.parts; ++k) top = fmaxf(top, lse[k * lse_stride]);
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll 1
    for (int k = 0; k < p.parts; ++k) total += expf(lse[k * lse_stride] - ref);
    float s[8] = {};
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll 1
    for (int k = 0; k < p.parts; ++k) add8(s, p.part_sums + k * part_stride + i * 8, expf(lse[k * lse_stride] - ref) * inv);
    store8(p.out.at(tok, h) + (i % groups) * 8, s);
    if (i % groups == 0) p.lse[h * p.tq + tok] = total == 0.0f ? -INFINITY : ref + logf(total);
}

// ---------------------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// [heads, tokens, dim] with boxes of 128 tokens x 64 elements.  The stride of an axis of one element
// is never used; any valid one will do.
bool make_map(CUtensorMap* m, const nvfp4_heads* h, int64_t tokens, int heads, int dim) {
    auto fn = encode_fn();
    if (!fn) return false;
    if (tokens == 0) {
        std::memset(m, 0, sizeof(*m));
        return true;
    }
    cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)tokens, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)(tokens > 1 ? h->token_stride : dim) * 2,
                             (cuuint64_t)(heads > 1 ? h->head_stride : dim) * 2};
    cuuint32_t box[3] = {64, kRows, 1}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, h->data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A kernel's shared memory is an attribute of the kernel on a device: set once on each of the first 64.
template <auto kern, typename... Args>
cudaError_t launch(int smem, int threads, int64_t grid, cudaStream_t s, const Args&... args) {
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (e == cudaSuccess && !(set.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) set.fetch_or(bit, std::memory_order_relaxed);
    }
    return e == cudaSuccess ? launch_pdl(kern, dim3((unsigned)grid), dim3(threads), smem, s, args...) : e;
}

// The forward kernel's setmaxnreg.inc completes only if the launch holds the split's total: a build
// that allocated fewer registers a thread is never launched.
template <int HD> bool fwd_registers_fit() {
    static std::once_flag once;
    static bool fit = false;
    std::call_once(once, [] {
        cudaFuncAttributes fa;
        fit = cudaFuncGetAttributes(&fa, fwd_kernel<HD>) == cudaSuccess && fa.numRegs >= kFwdRegs;
    });
    return fit;
}

nvfp4_status check_shape(const nvfp4_attention_shape* s) {
    if (!s) return NVFP4_ERR_INVALID_ARG;
    if (s->tq < 0 || s->tk < 0 || s->tq > (1ll << 30) || s->tk > (1ll << 30) || s->heads < 1 || s->kv_heads < 1 ||
        s->heads > 65535 || s->heads % s->kv_heads != 0 || s->dim < 8 || s->dim > 128 || s->dim % 8 != 0)
        return NVFP4_ERR_SHAPE;
    if (s->nseq < 1 || (!s->cu_q) != (!s->cu_k) || (!s->cu_q && s->nseq != 1) || !std::isfinite(s->scale))
        return NVFP4_ERR_INVALID_ARG;
    // tiles x heads (parts only where they are few) are counted in 32 bits, by the grid and up to three grids past the last
    if ((std::max(s->tq, s->tk) / kRows + s->nseq) * s->heads > INT_MAX - (1 << 16)) return NVFP4_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(s->cu_q) | reinterpret_cast<uintptr_t>(s->cu_k)) % 4) return NVFP4_ERR_ALIGNMENT;
    return NVFP4_OK;
}

// A tensor of `tokens` x `heads`; `data` may be null where there are no tokens.
nvfp4_status check_heads(const nvfp4_heads* h, int64_t tokens, int heads, int dim) {
    if (!h) return NVFP4_ERR_INVALID_ARG;
    if (tokens == 0) return NVFP4_OK;
    if (!h->data) return NVFP4_ERR_INVALID_ARG;
    if ((tokens > 1 && h->token_stride < dim) || (heads > 1 && h->head_stride < dim)) return NVFP4_ERR_SHAPE;
    if (h->token_stride > (1ll << 38) || h->head_stride > (1ll << 38)) return NVFP4_ERR_SHAPE;
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
    p.c = std::max(std::fabs(s->scale) * kLog2e, 1e-30f);   // 0 would make -inf * 0 of a masked score
    p.cu_q = s->cu_q;
    p.cu_k = s->cu_k;
    p.dev_status = dev_status;
    p.timeout_ns = wait_timeout_ns();
    p.parts = 1;
    return p;
}

// CTAs for tiles of `tile` rows: at most one part tile more per sequence.
int64_t tiles_of(int64_t tokens, int nseq, int tile) {
    return nseq == 1 ? (tokens + tile - 1) / tile : tokens / tile + nseq;
}
int sms() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? std::max(1, sm_count(dev)) : 1;
}

// How many CTAs share a tile's steps.  Tiles of queries, forward and dQ: where fewer than half the SMs have one, as many
// as fill them.  Tiles of keys: each is a whole head group's work, so that few of them balance badly too; there the
// aim is three a SM.  A part costs a tile of fp32 sums written and read: a CTA keeps at least 4 steps, of keys' tiles with
// their two sums 8 (4096 tokens in 20 documents, 20 / 4 heads of 128, 10 steps a tile: backward 93 us, 111 in parts of 5).
// 64 queries over 7000 keys, 8 / 2 heads of 128: forward 70 -> 19 us; 8192 tokens, 8 / 1 heads: backward 715 -> 325 us (303
// with the later steps).
int parts_for(int64_t ctas, int64_t steps, int64_t most_steps, int64_t wanted, int least) {
    if (ctas < 1 || 2 * ctas > wanted) return 1;
    // a tile of one long sequence among short ones may have most_steps; Share multiplies by the parts in 32 bits
    return (int)std::max<int64_t>(1, std::min<int64_t>({wanted / ctas, steps / least, 64, UINT32_MAX / std::max<int64_t>(1, most_steps)}));
}
int64_t tile_steps(int64_t tokens, int nseq) { return (tokens / nseq + kRows - 1) / kRows; }
int parts_of_fwd(const nvfp4_attention_shape* s) {
    return parts_for(tiles_of(s->tq, s->nseq, 2 * kRows) * s->heads, tile_steps(s->tk, s->nseq), tile_steps(s->tk, 1), sms(), 4);
}
int parts_of_dq(const nvfp4_attention_shape* s) {
    return parts_for(tiles_of(s->tq, s->nseq, kRows) * s->heads, tile_steps(s->tk, s->nseq), tile_steps(s->tk, 1), sms(), 4);
}
int parts_of_dkv(const nvfp4_attention_shape* s) {
    const int64_t share = s->heads / s->kv_heads;
    return parts_for(tiles_of(s->tk, s->nseq, kRows) * s->kv_heads, tile_steps(s->tq, s->nseq) * share,
                     tile_steps(s->tq, 1) * share, 3 * sms(), 8);
}
size_t sums_bytes(int parts, int64_t tokens, int heads, int dim) {
    return parts > 1 ? (size_t)parts * tokens * heads * dim * sizeof(float) : 0;
}
size_t delta_bytes(const nvfp4_attention_shape* s) {       // a multiple of 16
    return ((size_t)s->heads * (size_t)s->tq * sizeof(float) + 15) / 16 * 16 + 16;
}
unsigned join_blocks(int64_t tokens, int heads, int dim) {
    return (unsigned)((tokens * heads * (dim / 8) + kJoinThreads - 1) / kJoinThreads);
}

}  // namespace attn
}  // namespace nvfp4

using namespace nvfp4;

namespace {
nvfp4_status forward_impl(const nvfp4_attention_shape* shape, const nvfp4_heads* q, const nvfp4_heads* k,
                          const nvfp4_heads* v, const nvfp4_heads* out, float* lse, void* workspace,
                          size_t workspace_bytes, uint32_t* dev_status, void* stream) {
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
    p.out = heads_of(out);
    p.lse = lse;
    if (workspace) {
        if (!aligned16(workspace) || workspace_bytes < nvfp4_attention_forward_workspace_bytes(shape)) return NVFP4_ERR_WORKSPACE;
        p.parts = parts_of_fwd(shape);
        p.part_sums = static_cast<float*>(workspace);
        p.part_lse = p.part_sums + sums_bytes(p.parts, p.tq, p.heads, p.dim) / sizeof(float);
    }
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, q, p.tq, p.heads, p.dim) || !make_map(&mk, k, p.tk, p.kv_heads, p.dim) ||
        !make_map(&mv, v, p.tk, p.kv_heads, p.dim))
        return NVFP4_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    p.work = (int)(tiles_of(p.tq, p.nseq, 2 * kRows) * p.heads * p.parts);
    const int64_t grid = std::min(p.work, sms());
    if (!(p.dim <= 64 ? fwd_registers_fit<64>() : fwd_registers_fit<128>())) return NVFP4_ERR_CUDA;
    cudaError_t e = p.dim <= 64 ? launch<fwd_kernel<64>>(Fwd<64>::SMEM, kFwdThreads, grid, s, mq, mk, mv, p)
                                : launch<fwd_kernel<128>>(Fwd<128>::SMEM, kFwdThreads, grid, s, mq, mk, mv, p);
    if (e == cudaSuccess && p.parts > 1)
        e = launch_pdl(join_out_kernel, dim3(join_blocks(p.tq, p.heads, p.dim)), dim3(kJoinThreads), 0, s, p);
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
}  // namespace

extern "C" nvfp4_status nvfp4_attention_forward(const nvfp4_attention_shape* shape, const nvfp4_heads* q,
                                                const nvfp4_heads* k, const nvfp4_heads* v, const nvfp4_heads* out,
                                                float* lse, uint32_t* dev_status, void* stream) {
    return forward_impl(shape, q, k, v, out, lse, nullptr, 0, dev_status, stream);
}

extern "C" size_t nvfp4_attention_forward_workspace_bytes(const nvfp4_attention_shape* shape) {
    using namespace attn;
    if (check_shape(shape) != NVFP4_OK) return 0;
    const int parts = parts_of_fwd(shape);
    return parts == 1 ? 16 : sums_bytes(parts, shape->tq, shape->heads, shape->dim) +
                                 (size_t)parts * shape->heads * shape->tq * sizeof(float);
}

extern "C" nvfp4_status nvfp4_attention_forward_ws(const nvfp4_attention_shape* shape, const nvfp4_heads* q,
                                                   const nvfp4_heads* k, const nvfp4_heads* v, const nvfp4_heads* out,
                                                   float* lse, void* workspace, size_t workspace_bytes,
                                                   uint32_t* dev_status, void* stream) {
    return forward_impl(shape, q, k, v, out, lse, workspace, workspace_bytes, dev_status, stream);
}

extern "C" size_t nvfp4_attention_backward_workspace_bytes(const nvfp4_attention_shape* shape) {
    using namespace attn;
    if (check_shape(shape) != NVFP4_OK) return 0;
    // delta, then the parts' sums of one kernel at a time
    return delta_bytes(shape) + std::max(sums_bytes(parts_of_dq(shape), shape->tq, shape->heads, shape->dim),
                                         2 * sums_bytes(parts_of_dkv(shape), shape->tk, shape->kv_heads, shape->dim));
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
    p.out = heads_of(out);
    p.dout = heads_of(dout);
    p.dq = heads_of(dq);
    p.dk = heads_of(dk);
    p.dv = heads_of(dv);
    p.lse = const_cast<float*>(lse);
    p.delta = static_cast<float*>(workspace);
    CUtensorMap mq, mk, mv, mdo;
    if (!make_map(&mq, q, p.tq, p.heads, p.dim) || !make_map(&mk, k, p.tk, p.kv_heads, p.dim) ||
        !make_map(&mv, v, p.tk, p.kv_heads, p.dim) || !make_map(&mdo, dout, p.tq, p.heads, p.dim))
        return NVFP4_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    p.part_sums = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + delta_bytes(shape));
    cudaError_t e = cudaSuccess;
    if (p.tq > 0) {
        p.parts = parts_of_dq(shape);
        p.work = (int)(tiles_of(p.tq, p.nseq, kRows) * p.heads * p.parts);
        const int64_t grid = std::min(p.work, sms());
        e = p.dim <= 64 ? launch<dq_kernel<64>>(Dq<64>::SMEM, kDqThreads, grid, s, mq, mk, mv, mdo, p)
                        : launch<dq_kernel<128>>(Dq<128>::SMEM, kDqThreads, grid, s, mq, mk, mv, mdo, p);
        if (e == cudaSuccess && p.parts > 1)
            e = launch_pdl(join_sums_kernel, dim3(join_blocks(p.tq, p.heads, p.dim)), dim3(kJoinThreads), 0, s, p.part_sums,
                           p.parts, p.tq * p.heads * p.dim, 0, p.tq, p.heads, p.dim, p.dq, p.dq);
    }
    if (e == cudaSuccess && p.tk > 0) {
        p.parts = parts_of_dkv(shape);
        const int64_t grid = tiles_of(p.tk, p.nseq, kRows) * p.kv_heads * p.parts, sums = p.tk * p.kv_heads * p.dim;
        e = p.dim <= 64 ? launch<dkv_kernel<64>>(Dkv<64>::SMEM, kDkvThreads, grid, s, mq, mk, mv, mdo, p)
                        : launch<dkv_kernel<128>>(Dkv<128>::SMEM, kDkvThreads, grid, s, mq, mk, mv, mdo, p);
        if (e == cudaSuccess && p.parts > 1)
            e = launch_pdl(join_sums_kernel, dim3(join_blocks(p.tk, p.kv_heads, p.dim), 2), dim3(kJoinThreads), 0, s,
                           p.part_sums, p.parts, 2 * sums, sums, p.tk, p.kv_heads, p.dim, p.dv, p.dk);
    }
    return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
