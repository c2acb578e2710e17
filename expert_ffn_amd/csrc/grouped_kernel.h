// The expert operation on grouped rows: grouping of any number of slots by expert,
// block quantisation, and the products grouped by expert, on gfx950.
//
// Rows.  The slots s = t*m + j of a pass of n tokens, sorted stably by expert, are its
// rows: row r holds slot slot_by_expert[r], and expert e owns rows offset[e] ..
// offset[e+1].  Rows from offset[N] on hold no slot (ids outside [0, N)).
//   gate/up  h_r = silu(W_gate[e] x_t) * (W_up[e] x_t)
//   down     O_s = W_down[e] h_r,   y_t = sum_j w_tj O_tj  in increasing j
//
// Both weight types are read in units of 128 bytes along the contraction: 64 bf16 or
// 128 e4m3 elements.  A lane's operands of a unit are two 16-byte chunks, kk = 0, 1, at
// byte 64 kk + 16 (lane / 16) of row lane % 16: two bf16 16x16x32 products, or one e4m3
// 16x16x128 product (any order of k that both operands share gives the same sum).  The
// weights are the product's first operand, so that lane l of the result holds four
// consecutive weight rows, 4 (l / 16) + i, of token l % 16.
//
// e4m3 operands carry a power of two for each block of 128 along the contraction (and
// 128 weight rows), as the byte k + 127 that the scaled matrix instruction takes for
// each row's 32 elements: all four get the block's.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "moe_expert.h"

namespace moe_g {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) unsigned int u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned int u32x2;
typedef __attribute__((ext_vector_type(8))) int i32x8;

constexpr int kUnit = 128;   // bytes of a contraction unit
constexpr int kBlk = 128;    // elements of a quantisation block
constexpr int kTile16 = 16;  // rows of a matrix operand

struct Args {
    const char* x;        // x [n][K] (gate/up, gathered) or h [S][K] (down, in row order)
    const uint8_t* xs;    // e4m3: scale bytes of x / h rows
    const char* w0;       // W_gate or W_down
    const char* w1;       // W_up
    const uint8_t* s0;    // e4m3: scale bytes of w0, w1  [N][ceil(R/128)][ceil(K/128)]
    const uint8_t* s1;
    const int32_t* offset;
    const int32_t* slot;
    char* out;            // gate/up: h [S][R]; down: O [S][R], rows in group order (thin tiles fp32, square ones fp16)
    int32_t* queue;       // square tiles: [8][kLine], tiles taken from each XCD's run, zero at the start
    uint8_t* outs;        // e4m3 gate/up: scale bytes of h; square down tiles: those of O [S][ceil(R/64)]
    int N, m, S, R, K;
    int tile0;            // thin tiles: the launch's first row tile
    int32_t* row_of;      // thin down tiles: null, or the row of each slot, to be written
};

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// One unit's product.  e4m3: the operands' scale bytes, sa's lowest and byte `sel` of sb
// (a constant once its loop is unrolled).
template <bool FP8>
__device__ __forceinline__ f32x4 mma_unit(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1, f32x4 c, int sa, int sb, int sel = 0) {
    if constexpr (FP8) {
        struct Pair {
            u32x4 lo, hi;
        };
        const i32x8 a = __builtin_bit_cast(i32x8, Pair{a0, a1}), b = __builtin_bit_cast(i32x8, Pair{b0, b1});
        switch (sel & 3) {
            case 0: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, sa, 0, sb);
            case 1: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, sa, 1, sb);
            case 2: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, sa, 2, sb);
            default: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, sa, 3, sb);
        }
    } else {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a0), __builtin_bit_cast(bf16x8_t, b0),
                                                    c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a1),
                                                       __builtin_bit_cast(bf16x8_t, b1), c, 0, 0, 0);
    }
}

// silu(z) = z / (1 + exp(-z)); exp(-z) overflows to infinity below z = -88: -0.
__device__ __forceinline__ float silu(float z) { return z * __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {  // to nearest even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2_t));
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ uint32_t f16_pair(float a, float b) {  // to nearest even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2_t));
}
__device__ __forceinline__ f32x2 f16_values(uint32_t v) {
    return __builtin_convertvector(__builtin_bit_cast(f16x2_t, v), f32x2);
}

// --- block quantisation ------------------------------------------------------------
// k = the smallest integer >= -127 with amax <= 448 * 2^k: 448 = 1.75 * 2^8, so for
// amax = f * 2^E with 1 <= f < 2, k = E - 8, plus one where f > 1.75.  A power of two
// keeps 448 * 2^k within a factor of two of amax, loses no precision (a product with
// it is exact) and is what the matrix instruction scales by at no cost; rounding to
// e4m3 then happens once, to nearest even.
__device__ __forceinline__ int block_exp(float amax) {
    const uint32_t b = __float_as_uint(amax);
    return max((int)(b >> 23) - 135 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0), -127);
}
// 2^k, -127 <= k <= 127
__device__ __forceinline__ float pow2(int k) {
    return k > -127 ? __uint_as_float((uint32_t)(k + 127) << 23) : __uint_as_float(0x400000u);
}
// |v|, 0 for what is not finite (which takes no part in a block's maximum)
__device__ __forceinline__ float mag(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
    return b < 0x7f800000u ? __uint_as_float(b) : 0.f;
}
// four codes of v * inv; an infinity or NaN gives the NaN code
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
    auto f = [&](float v) { return mag(v) == 0.f && v != 0.f ? __uint_as_float(0x7fc00000u) : v * inv; };
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(f(a), f(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f(c), f(d), p, true);
}

__device__ __forceinline__ uint32_t finite_codes4(f32x4 v, float inv) {
    const int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, p, true);
}

// Rows of bf16 (or float32) values to codes and scale bytes, in blocks of 128 along the row:
// sixteen lanes a block, eight values a lane (16 bytes of bf16), so that a block's maximum takes
// four exchanges and no shared memory; work group g of G.  Bound by memory: 16384 x 2048 in 22-24 us,
// 101 MB at 4.2-4.6 TB/s (a large copy here: 4.9).
template <bool F32>
__device__ __forceinline__ void quant_rows(const char* __restrict__ x, int64_t rows, int K, uint8_t* __restrict__ q,
                                           uint8_t* __restrict__ s, int64_t g, int64_t G) {
    const int KB = (K + kBlk - 1) / kBlk, per = blockDim.x / 16;
    const int64_t blocks = rows * KB;
    const int l = threadIdx.x & 15;
    for (int64_t b = g * per + threadIdx.x / 16; b < blocks; b += G * per) {
        const int64_t row = b / KB;
        const int kb = (int)(b - row * KB), c = kb * kBlk + l * 8;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
        if (c < K) {
            if (F32) {
                const f32x4* p = reinterpret_cast<const f32x4*>(x + (row * K + c) * 4);
                const f32x4 a = p[0], d = p[1];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = d[i];
            } else {
                const u32x4 a = *reinterpret_cast<const u32x4*>(x + (row * K + c) * 2);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(a[i]), v[2 * i + 1] = bf16_hi(a[i]);
            }
        }
        float am = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) am = fmaxf(am, mag(v[i]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor(am, o, 16));
        const int k = block_exp(am);
        const float inv = pow2(-k);
        if (c < K)
            *reinterpret_cast<u32x2*>(q + row * K + c) =
                u32x2{codes4(v[0], v[1], v[2], v[3], inv), codes4(v[4], v[5], v[6], v[7], inv)};
        if (l == 0) s[b] = (uint8_t)(k + 127);
    }
}

// `limit`: rows in use, where only the device knows (null: all)
template <bool F32>
__global__ __launch_bounds__(256) void k_quant_rows(const char* __restrict__ x, int64_t rows, int K,
                                                   const int32_t* __restrict__ limit, uint8_t* __restrict__ q,
                                                   uint8_t* __restrict__ s) {
    if (limit) rows = min(rows, (int64_t)max(*limit, 0));
    quant_rows<F32>(x, rows, K, q, s, blockIdx.x, gridDim.x);
}

// Codes and scale bytes of rows back to bf16: four bits of significand fit bf16's eight,
// so this is exact down to bf16's own least value.  16384 x 2048 in 17 us: 101 MB at 5.9 TB/s.
__global__ __launch_bounds__(256) void k_dequant_rows(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                     int64_t rows, int K, char* __restrict__ x) {
    const int KB = (K + kBlk - 1) / kBlk;
    const int64_t blocks = rows * KB;
    const int l = threadIdx.x & 15;
    for (int64_t b = (int64_t)blockIdx.x * 16 + threadIdx.x / 16; b < blocks; b += (int64_t)gridDim.x * 16) {
        const int64_t row = b / KB;
        const int c = (int)(b - row * KB) * kBlk + l * 8;
        if (c >= K) continue;
        const float f = pow2((int)s[b] - 127);
        const u32x2 v = *reinterpret_cast<const u32x2*>(q + row * K + c);
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], false);
            auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], true);
            o[2 * i] = bf16_pair(lo[0] * f, lo[1] * f);
            o[2 * i + 1] = bf16_pair(hi[0] * f, hi[1] * f);
        }
        *reinterpret_cast<u32x4*>(x + (row * K + c) * 2) = o;
    }
}

// One work group a block of 128 x 128 weights: thread t holds row t / 2's half t % 2, 64 values.
__global__ __launch_bounds__(256) void k_quant_weights(const char* __restrict__ w, int R, int K,
                                                      uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
    __shared__ float part[4];
    const int RB = (R + kBlk - 1) / kBlk, KB = (K + kBlk - 1) / kBlk;
    const int64_t b = blockIdx.x;
    const int kb = (int)(b % KB);
    const int rb = (int)(b / KB % RB);
    const int64_t e = b / KB / RB;
    const int tid = threadIdx.x, c = kb * kBlk + (tid & 15) * 8, r0 = rb * kBlk + tid / 16;
    u32x4 a[8];
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        a[i] = u32x4{0u, 0u, 0u, 0u};
        if (r < R && c < K) a[i] = *reinterpret_cast<const u32x4*>(w + ((e * R + r) * K + c) * 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) am = fmaxf(am, fmaxf(mag(bf16_lo(a[i][j])), mag(bf16_hi(a[i][j]))));
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor(am, o, 64));
    if ((tid & 63) == 0) part[tid >> 6] = am;
    __syncthreads();
    const int k = block_exp(fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])));
    const float inv = pow2(-k);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        if (r < R && c < K)
            *reinterpret_cast<u32x2*>(q + (e * R + r) * K + c) =
                u32x2{codes4(bf16_lo(a[i][0]), bf16_hi(a[i][0]), bf16_lo(a[i][1]), bf16_hi(a[i][1]), inv),
                      codes4(bf16_lo(a[i][2]), bf16_hi(a[i][2]), bf16_lo(a[i][3]), bf16_hi(a[i][3]), inv)};
    }
    if (tid == 0) s[b] = (uint8_t)(k + 127);
}

// --- grouping of any number of slots -------------------------------------------------
// A stable counting sort over G chunks of slots, one work group of 16 waves each, the
// waves on consecutive pieces of the chunk: first every chunk's histogram, then every
// chunk adds up the chunks before it and writes its slots behind them; one chunk needs
// one launch.  The rank of a slot among equal ids of its wave's 64 comes from one ballot
// for each bit of the id, so the order is that of the slots, whatever the timing.
//
// Latency is the time (a few loads, scans and barriers: 576 slots 5.4 us, 131072 slots 4.6 + 7.6 us,
// where the memory's share is 0.2 us), so a pass's other preparation rides along: work groups
// from G on quantise x, and the first clears the queues.  One chunk up to 8192 slots: of 576 slots two launches
// took 15.4 us with the host's share, one 9.8; beyond, one work group's loads take longer than a launch.
constexpr int kGThreads = 1024, kGWaves = kGThreads / 64;
constexpr int kGMaxChunks = 64, kGOne = 8192;  // slots of one chunk

__host__ __device__ __forceinline__ int64_t group_chunk(int64_t S) {
    const int64_t c = S <= kGOne ? S : (S + kGMaxChunks - 1) / kGMaxChunks;
    return (c + kGThreads - 1) / kGThreads * kGThreads;
}

struct Group {
    const int32_t* ids;
    int64_t S;
    int m, N, G;            // G chunks
    int32_t* hist;          // [G][N + 1], with more than one chunk
    int32_t *count, *offset, *sbe, *distinct, *u_err;
    int32_t* row_of;        // null, or the row of each slot
    int32_t* queues;        // null, or nq words to clear
    int nq;
    const char* x;          // null, or rows to quantise (n rows of d)
    uint8_t *xq, *xs;
    int n, d;
};

__device__ __forceinline__ bool group_quant(const Group& g) {
    if ((int)blockIdx.x < g.G) return false;
    quant_rows<false>(g.x, g.n, g.d, g.xq, g.xs, blockIdx.x - g.G, gridDim.x - g.G);
    return true;
}

// Whether slot s (its id valid) repeats an id of its token; eight loads at a time.
__device__ __forceinline__ bool group_repeat(const int32_t* __restrict__ ids, int64_t s, int m, int id) {
    const int j = (int)(s % m);
    bool again = false;
    for (int i0 = 1; i0 <= j; i0 += 8) {
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = ids[s - min(i0 + i, j)];
#pragma unroll
        for (int i = 0; i < 8; ++i) again |= v[i] == id;
    }
    return again;
}

__global__ __launch_bounds__(kGThreads) void k_group_hist(Group g) {
    __shared__ int cnt[MOE_MAX_EXPERTS];
    if (group_quant(g)) return;
    const int tid = threadIdx.x;
    const int64_t chunk = group_chunk(g.S), s0 = blockIdx.x * chunk;
    for (int e = tid; e < g.N; e += kGThreads) cnt[e] = 0;
    __syncthreads();
    int bad = 0;
    for (int64_t i = tid; i < chunk; i += kGThreads) {
        const int64_t s = s0 + i;
        if (s >= g.S) break;
        const int id = g.ids[s];
        if (id >= 0 && id < g.N) {
            atomicAdd(&cnt[id], 1);
            bad |= group_repeat(g.ids, s, g.m, id);
        } else {
            bad = 1;
        }
    }
    bad = __syncthreads_or(bad);
    int32_t* h = g.hist + (int64_t)blockIdx.x * (g.N + 1);
    for (int e = tid; e < g.N; e += kGThreads) h[e] = cnt[e];
    if (tid == 0) h[g.N] = bad;
}

// Exclusive sums over the work group of one value a thread; total to all.
__device__ __forceinline__ int group_scan(int v, int* part, int& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int s = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(s, o, 64);
        if (lane >= o) s += u;
    }
    if (lane == 63) part[wave] = s;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kGWaves; ++i) {
        before += i < wave ? part[i] : 0;
        all += part[i];
    }
    __syncthreads();
    total = all;
    return before + s - v;
}

__global__ __launch_bounds__(kGThreads) void k_group_scatter(Group g) {
    __shared__ int base[kGWaves * MOE_MAX_EXPERTS];  // [wave][N]: next place of the wave's slots
    __shared__ int sums[2][kGThreads];
    __shared__ int part[kGWaves];
    if (g.G == 1 && group_quant(g)) return;  // with more chunks the first launch has quantised
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, N = g.N;
    const int64_t chunk = group_chunk(g.S), s0 = blockIdx.x * chunk;
    const int64_t per = chunk / kGWaves, w0 = s0 + wave * per;  // per: a multiple of 64
    const bool first = blockIdx.x == 0;
    if (first)
        for (int i = tid; i < g.nq; i += kGThreads) g.queues[i] = 0;
    for (int i = tid; i < kGWaves * N; i += kGThreads) base[i] = 0;
    // Every chunk's counts of expert e: P threads an expert, each a part of the chunks,
    // with its loads in flight together.
    int bad = 0, lo = 0, hi = 0;
    const int P = kGThreads / N;  // >= 1
    const int pe = tid % N, pp = tid / N;
    if (g.G > 1 && pp < P) {
        for (int c0 = pp; c0 < g.G; c0 += 8 * P) {
            int v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = g.hist[(int64_t)min(c0 + i * P, g.G - 1) * (N + 1) + pe];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = c0 + i * P;
                if (c < g.G) {
                    hi += v[i];
                    lo += c < (int)blockIdx.x ? v[i] : 0;
                }
            }
        }
    }
    if (g.G > 1 && first && tid < g.G) bad = g.hist[(int64_t)tid * (N + 1) + N];
    sums[0][tid] = lo;
    sums[1][tid] = hi;
    __syncthreads();
    // this wave's own histogram
    for (int64_t i = lane; i < per; i += 64) {
        const int64_t s = w0 + i;
        if (s >= g.S) break;
        const int id = g.ids[s];
        const bool ok = id >= 0 && id < N;
        if (ok) atomicAdd(&base[wave * N + id], 1);
        if (g.G == 1) bad |= ok ? group_repeat(g.ids, s, g.m, id) : 1;
    }
    bad = __syncthreads_or(bad);
    // thread e: expert e's slots in the chunks before this one, and in all
    int before = 0, all = 0;
    if (tid < N) {
        if (g.G > 1) {
            for (int i = 0; i < P; ++i) {
                before += sums[0][i * N + tid];
                all += sums[1][i * N + tid];
            }
        } else {
#pragma unroll
            for (int w = 0; w < kGWaves; ++w) all += base[w * N + tid];
        }
    }
    int valid, U;
    const int start = group_scan(all, part, valid);
    const int dpos = group_scan(tid < N && all > 0, part, U);
    if (tid < N) {
        int c[kGWaves];
#pragma unroll
        for (int w = 0; w < kGWaves; ++w) c[w] = base[w * N + tid];
        int at = start + before;
#pragma unroll
        for (int w = 0; w < kGWaves; ++w) {
            base[w * N + tid] = at;
            at += c[w];
        }
        if (first) {
            g.count[tid] = all;
            g.offset[tid] = start;
            if (all > 0) g.distinct[dpos] = tid;
            if (tid >= U) g.distinct[tid] = -1;
        }
    }
    if (first && tid == 0) {
        g.offset[N] = valid;
        g.u_err[0] = U;
        g.u_err[1] = bad ? MOE_E_IDS : MOE_OK;
    }
    __syncthreads();
    for (int64_t i = lane; i < per; i += 64) {
        const int64_t s = w0 + i;
        const int id = s < g.S ? g.ids[s] : -1;
        const bool ok = id >= 0 && id < N;
        uint64_t same = __ballot(ok);
        for (int b = 0; (1 << b) < N; ++b) {
            const uint64_t v = __ballot((id >> b) & 1);
            same &= ((id >> b) & 1) ? v : ~v;
        }
        if (ok) {
            const uint64_t under = same & ((1ull << lane) - 1);
            const int at = base[wave * N + id];
            g.sbe[at + __popcll(under)] = (int)s;
            if (g.row_of) g.row_of[s] = at + __popcll(under);
            __builtin_amdgcn_wave_barrier();
            if (under == 0) base[wave * N + id] = at + __popcll(same);
        }
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // the places that no slot takes
    for (int64_t r = valid + (int64_t)blockIdx.x * kGThreads + tid; r < g.S; r += (int64_t)g.G * kGThreads) g.sbe[r] = -1;
}

// --- products ------------------------------------------------------------------------
// Tile t of the row tiles of `rows` rows, counted over the experts: its expert, first
// row and the end of the expert's rows.  Every wave finds it by itself: a lane adds the
// tiles of N / 64 consecutive experts, one scan over the lanes.  Offsets are kept within
// [0, S] whatever they hold.
struct TileAt {
    int e, r0, end;  // e < 0: past the last tile
};

__device__ __forceinline__ TileAt find_tile(const int32_t* __restrict__ offset, int N, int S, int rows, int t) {
    const int lane = threadIdx.x & 63, C = (N + 63) / 64;
    int sum = 0;
    for (int i = 0; i < C; ++i) {
        const int e = lane * C + i;
        if (e < N) {
            const int a = min(max(offset[e], 0), S), b = min(max(offset[e + 1], a), S);
            sum += (b - a + rows - 1) / rows;
        }
    }
    int s = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(s, o, 64);
        if (lane >= o) s += u;
    }
    const uint64_t past = __ballot(s > t);
    if (!past) return TileAt{-1, 0, 0};
    const int from = __ffsll((unsigned long long)past) - 1;
    int k = t - (__shfl(s, from, 64) - __shfl(sum, from, 64));
    for (int i = 0; i < C; ++i) {
        const int e = from * C + i;
        if (e >= N) break;
        const int a = min(max(uni(offset[e]), 0), S), b = min(max(uni(offset[e + 1]), a), S);
        const int c = (b - a + rows - 1) / rows;
        if (k < c) return TileAt{e, a + k * rows, b};
        k -= c;
    }
    return TileAt{-1, 0, 0};
}

// Thin tiles: 16 rows by 16 output columns (gate/up: of both matrices), the contraction
// split over the four waves, operands straight from memory.  For passes of few rows an
// expert, where the weights' bytes are the time: there is time for the e4m3 operands to
// be widened to bf16 (exact, their power of two with them), whose products and sums the
// matrix instruction rounds only to fp32, where its e4m3 form cuts small ones (see the
// note at k_tile).
//
// SPLIT: the four waves share a tile's contraction.  Without, for short contractions of many tiles,
// each has a tile of its own: 128 experts of 2048 x 768 at 2 rows, down, 85 -> 76 us in bf16 (12 units),
// 73 -> 37 in e4m3 (6 units; 201 MB at 5.5 TB/s), but 22 units in bf16 67 -> 70.  Few units of a wave's loads in
// flight leave registers for more waves: of 2 / 3 / 4 / 6 / 8 without SPLIT that e4m3 down took
// 36 / 37 / 40 / 43 / 51 us, one of 1408 columns 36 / 33 / 34 / 36 / 44; e4m3 gate/up with SPLIT at 1 / 2 / 3 / 4
// 72 / 70 / 76 / 79; bf16 differs by 1-3 %.
// Memory bounds them: gate/up and down of 32 tokens (skewed over 128 bf16 experts of 2048 x 768) 49 + 27 us;
// of one token on 8 e4m3 experts (25 + 13 MB in all) 9.4 + 6.9 us, where the latency of a launch and its first
// loads is most.  Quantising h inside e4m3 down tiles, which spares a launch, made each of
// them read 128 columns of fp32 h first: one token's pass 29 us for 24.
constexpr int kThinWaves = 4;
constexpr int kThinWhole = 16;  // most units of a contraction without SPLIT

// Two words of codes (eight values) to bf16, scaled.
__device__ __forceinline__ bf16x8_t widen(uint32_t lo, uint32_t hi, float f) {
    struct Eight {
        bf16x2_t v[4];
    };
    return __builtin_bit_cast(bf16x8_t, Eight{{__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, false),
                                               __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, true),
                                               __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, false),
                                               __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, true)}});
}

template <bool FP8, bool TILED, bool GU, bool SPLIT>
__global__ __launch_bounds__(64 * kThinWaves) void k_thin(Args a) {
    constexpr int ES = FP8 ? 1 : 2, NW = GU ? 2 : 1, AHEAD = !SPLIT ? 3 : GU ? 2 : 4;
    __shared__ f32x4 red[SPLIT ? kThinWaves : 1][NW][64];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int lr = lane & 15, q = lane >> 4;
    const int CB = (a.R + 15) / 16, CW = SPLIT ? CB : (CB + kThinWaves - 1) / kThinWaves;  // work groups a row tile
    const int tile = blockIdx.x / CW, cw = blockIdx.x - tile * CW;
    const int cb = SPLIT ? cw : cw * kThinWaves + wave;
    if (!SPLIT && cb >= CB) return;  // (no barrier without SPLIT)
    const TileAt t = find_tile(a.offset, a.N, a.S, kTile16, a.tile0 + tile);
    if (t.e < 0) return;
    const int KBy = a.K * ES, U = (KBy + kUnit - 1) / kUnit, KB = (a.K + kBlk - 1) / kBlk;
    const int row = min(t.r0 + lr, t.end - 1);
    if (!GU && a.row_of && cb == 0 && threadIdx.x < kTile16) a.row_of[min(max(a.slot[row], 0), a.S - 1)] = row;
    int64_t xrow = row;
    if (GU) xrow = min(max(a.slot[row], 0), a.S - 1) / a.m;
    const char* wp[2];
    const int wr = min(cb * 16 + lr, a.R - 1);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const char* w = (i ? a.w1 : a.w0) + (int64_t)t.e * a.R * KBy;
        wp[i] = TILED ? w + (int64_t)cb * 16 * KBy + lane * 16 : w + (int64_t)wr * KBy;
    }
    const int RB = (a.R + kBlk - 1) / kBlk;
    const int64_t sw = FP8 ? ((int64_t)t.e * RB + cb * 16 / kBlk) * KB : 0;
    f32x4 acc[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int STEP = SPLIT ? kThinWaves : 1;
    for (int u0 = SPLIT ? wave : 0; u0 < U; u0 += STEP * AHEAD) {
        u32x4 b[AHEAD][2], w[AHEAD][NW][2];
        int eb[AHEAD], ew[AHEAD][NW];
        // the weights first: they wait for nothing but the tile
#pragma unroll
        for (int p = 0; p < AHEAD; ++p) {
            const int u = u0 + p * STEP;
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                ew[p][i] = 0;
                if (FP8 && u < U) ew[p][i] = (i ? a.s1 : a.s0)[sw + u];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const int k = u * kUnit + kk * 64 + q * 16;
                    w[p][i][kk] = u < U && k < KBy ? *reinterpret_cast<const u32x4*>(
                                                         wp[i] + (TILED ? (int64_t)(2 * u + kk) * 1024 : (int64_t)k))
                                                   : u32x4{0u, 0u, 0u, 0u};
                }
            }
        }
#pragma unroll
        for (int p = 0; p < AHEAD; ++p) {
            const int u = u0 + p * STEP;
            eb[p] = 0;
            if (FP8 && u < U) eb[p] = a.xs[xrow * KB + u];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const int k = u * kUnit + kk * 64 + q * 16;
                b[p][kk] = u < U && k < KBy ? *reinterpret_cast<const u32x4*>(a.x + xrow * KBy + k)
                                            : u32x4{0u, 0u, 0u, 0u};
            }
        }
#pragma unroll
        for (int p = 0; p < AHEAD; ++p) {
            if constexpr (FP8) {
                const float fb = pow2(eb[p] - 127);
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int v = 0; v < 4; v += 2) {
                        const bf16x8_t x = widen(b[p][kk][v], b[p][kk][v + 1], fb);
#pragma unroll
                        for (int i = 0; i < NW; ++i)
                            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                widen(w[p][i][kk][v], w[p][i][kk][v + 1], pow2(ew[p][i] - 127)), x, acc[i], 0, 0, 0);
                    }
            } else {
#pragma unroll
                for (int i = 0; i < NW; ++i)
                    acc[i] = mma_unit<false>(w[p][i][0], w[p][i][1], b[p][0], b[p][1], acc[i], 0, 0);
            }
        }
    }
    f32x4 v[NW];
    if constexpr (SPLIT) {
#pragma unroll
        for (int i = 0; i < NW; ++i) red[wave][i][lane] = acc[i];
        __syncthreads();
        if (wave) return;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            v[i] = red[0][i][lane];
#pragma unroll
            for (int k = 1; k < kThinWaves; ++k) v[i] += red[k][i][lane];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NW; ++i) v[i] = acc[i];
    }
    const int c = cb * 16 + 4 * q;
    if (t.r0 + lr >= t.end || c >= a.R) return;
    if (GU) {
        float h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = silu(v[0][i]) * v[NW - 1][i];
        if (FP8)  // float32, quantised later: a block's maximum is over 128 columns
            *reinterpret_cast<f32x4*>(a.out + ((int64_t)row * a.R + c) * 4) = f32x4{h[0], h[1], h[2], h[3]};
        else
            *reinterpret_cast<u32x2*>(a.out + ((int64_t)row * a.R + c) * 2) =
                u32x2{bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3])};
    } else {  // float32: O is a partial sum of y
        *reinterpret_cast<f32x4*>(a.out + ((int64_t)row * a.R + c) * 4) = v[0];
    }
}

// Square tiles: up to 256 rows by 256 weight rows (gate/up: 128 of each matrix, so 128
// columns of h), eight waves as 2 x 4, each up to 128 rows by 64 weight rows in registers;
// a wave takes the 16-row blocks 2 i + wm, so a tile of few rows is shared by both wave
// rows.  One work group a compute unit runs its tiles as one stream of contraction units,
// so that a tile's first loads are on their way while the one before is finished.
//
// The two waves of a SIMD (wm = 0, 1) take turns: while one reads its operands of half a
// unit from shared memory, the other runs the products of its own.  A unit has four
// phases, a barrier after each: Ra (all weight rows and the first 128 rows), Ma (their
// products), Rb (the other 128), Mb; wm = 1 is one phase behind.  In Ma a block's place is free
// after its products, and a block of the other 128 rows is asked for at once (gate/up in e4m3 has
// no registers for that: in Rb).  Two units of each operand fit in shared memory.  A wave's eight
// loads of a unit go out as soon as what they overwrite has been read:
//     phase of unit v     loads                                       overwrites, last read
//     Ra                  last 128 rows of v + 1 (two)                of v - 1, in Ma / Rb (v - 1)
//     Rb, Mb              weight rows, first 128 rows of v + 2        of v, in Ra (v)
//                         (three each)
// (each read has ended before the barrier of Ra or Rb, and wm = 1 reads one phase later, before
// these).  They are waited for at the end of Mb (the last 128 rows of the next unit) and of Rb
// (the rest of it), one phase before wm = 0 reads them: the counts are of what was issued since.
// (Figures of 8-bit down in comparisons here and below are from when it handed its terms on in bf16, about
// 12 us less.)  With the last 128 rows read in Rb alone and loaded in Ma, gate/up of 4096 tokens (128 bf16 experts of
// 2048 x 768) took 298 us for 292, 8-bit down 133 for 128; with the first 128 rows also read a phase ahead
// (and so waited for a phase earlier) 313.
//
// What they reach, PFLOP/s: gate/up of one expert's 4096 rows of 2048 x 8192 in bf16 1.03 (a library
// product of that size 1.15), of 2048 rows of 4096 x 4096 1.19 (1.47); of 8 experts' 2048 rows each of
// 2048 x 4096 1.18, in e4m3 2.1.  128 experts of 2048 x 768 with 32768 skewed rows reach 0.75: 43 % of
// their tiles' rows are missing (a unit costs the same), each compute unit has 5 or 6 tiles, and a
// tile's change and results, 2 of its 32 units' time at this width, are not hidden.  Tiles of 128 rows
// instead: 366 us for 297, and 165 for 134 in 8-bit down.
//
// The e4m3 matrix instruction adds the products of 8 consecutive k after cutting each to
// multiples of 2^-13 of the power of two of the group's largest (measured: 2^16 + 2^2 in
// one group gives 2^16, across groups the sum; 16x16x32, 32x32x16 and 32x32x64 do the same).  That is 2^-9 of the
// step that quantising the operands has already taken (half of 2^-3); sums across groups, units and waves are
// fp32.  Without the cut the operands would have to be widened to bf16, whose products run at 1.3 PFLOP/s for 4.2
// (loops of the instruction alone): no faster than a bf16 layer.
constexpr int kTM = 256, kTN = 256, kTileThreads = 512;
constexpr int kStageA = kTM * kUnit, kStage = (kTM + kTN) * kUnit;
constexpr uint32_t kOOB = 0x80000000u;  // beyond every buffer: reads give zero
constexpr int kLine = 32;               // words a counter of its own cache line takes
constexpr int kQueue = 8 * kLine;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
// 1 KB of memory, 16 bytes a lane, to shared memory in lane order
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t vo, uint32_t so) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, (int)vo, (int)so, 0, 0);
}
// place of 16-byte chunk c of row r in shared memory's 128-byte rows: the 16 rows that a
// read instruction touches then fall on different banks
__device__ __forceinline__ int swz(int r, int c) { return r * kUnit + ((c ^ (r & 7)) << 4); }

template <int N>
__device__ __forceinline__ void wait_vm() {  // all but the last N loads of this wave are done
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | (N >> 4 << 14));
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void wait_lds() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xc07f);
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void block_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// O of square tiles: blocks of 64 columns of a row as fp16 times a power of two, which puts the block's
// largest into [2^14, 2^15).  `byte` is its exponent's byte in fp32, 14 at least so that 2^127 scales it.
__device__ __forceinline__ int term_byte(uint32_t largest) { return max((int)(largest >> 23), 14); }

// The largest of the four lanes l % 16 + 16 k.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    const u32x2 a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(a[0], a[1]);
    const u32x2 b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return max(b[0], b[1]);
}

struct Place {
    int e, r0, rows, ct;  // rows 0: no tile
};

// Every expert's row tiles and what they cost, one scan kept by the wave: lane l holds
// N / 64 experts.  A unit of a tile takes about the same time whatever its rows (the four
// phases' reads, loads and barriers; clocks / 100, measured): shares by 14 / 17 / 23 / 29 for up to
// 64 / 128 / 192 / 256 rows, nearer to the rows' own work, cost 8-bit down of 4096 tokens 142 us for 133
// and the 8-bit pass of 8191 tokens 531 for 510.
__device__ __forceinline__ int tile_cost(int rows) { return rows <= 64 ? 23 : rows <= 128 ? 26 : rows <= 192 ? 28 : 30; }

// offset, kept in shared memory: a load from memory would wait for every operand's before it
struct Groups {
    const int32_t* offset;
    int N, S;
};

struct Tiles {
    int sum, upto, cost, cost_upto;  // of this lane's experts; up to and with them
    int total, cost_total, C;

    struct Span {
        int lo, hi, tiles, cost;
    };
    __device__ __forceinline__ static Span span(const Groups& a, int lo, int hi) {
        lo = min(max(lo, 0), a.S);
        hi = min(max(hi, lo), a.S);
        const int n = hi - lo, rest = n & (kTM - 1);
        return Span{lo, hi, (n + kTM - 1) / kTM, n / kTM * tile_cost(kTM) + (rest ? tile_cost(rest) : 0)};
    }
    __device__ __forceinline__ static int scan(int v) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(v, o, 64);
            if (lane >= o) v += u;
        }
        return v;
    }
    __device__ __forceinline__ void count(const Groups& a) {
        const int lane = threadIdx.x & 63;
        C = (a.N + 63) / 64;
        sum = cost = 0;
        for (int i = 0; i < C; ++i) {
            const int e = lane * C + i;
            if (e < a.N) {
                const Span s = span(a, a.offset[e], a.offset[e + 1]);
                sum += s.tiles;
                cost += s.cost;
            }
        }
        upto = scan(sum);
        cost_upto = scan(cost);
        total = __builtin_amdgcn_readlane(upto, 63);
        cost_total = __builtin_amdgcn_readlane(cost_upto, 63);
    }

    // The tile (row tiles times CT) at cost x / 8 of all.
    __device__ __forceinline__ int bound(const Groups& a, int CT, int x) const {
        if (x >= 8) return total * CT;
        const int64_t target = (int64_t)cost_total * CT * x / 8;
        const uint64_t past = __ballot((int64_t)cost_upto * CT > target);
        if (!past) return total * CT;
        const int from = __ffsll((unsigned long long)past) - 1;
        int t = __builtin_amdgcn_readlane(upto, from) - __builtin_amdgcn_readlane(sum, from);
        int64_t left = target - (int64_t)(__builtin_amdgcn_readlane(cost_upto, from) - __builtin_amdgcn_readlane(cost, from)) * CT;
        for (int i = 0; i < C && from * C + i < a.N; ++i) {
            const int e = from * C + i;
            const Span s = span(a, uni(a.offset[e]), uni(a.offset[e + 1]));
            if (left < (int64_t)s.cost * CT) return t * CT + (int)(left * s.tiles / s.cost);
            left -= (int64_t)s.cost * CT;
            t += s.tiles;
        }
        return t * CT;
    }

    // Tile t of CT column tiles each: the column tiles of up to 8 row tiles are neighbours.
    __device__ __forceinline__ Place place(const Groups& a, int CT, int t) const {
        const uint64_t past = __ballot(upto * CT > t);
        if (t >= total * CT || !past) return Place{0, 0, 0, 0};
        const int from = __ffsll((unsigned long long)past) - 1;
        int k = t - (__builtin_amdgcn_readlane(upto, from) - __builtin_amdgcn_readlane(sum, from)) * CT;
        for (int i = 0; i < C && from * C + i < a.N; ++i) {
            const int e = from * C + i;
            const Span s = span(a, uni(a.offset[e]), uni(a.offset[e + 1]));
            if (k < s.tiles * CT) {
                const int sg = k < 8 * CT ? 0 : k / (8 * CT), in = min(8, s.tiles - 8 * sg);
                k -= sg * 8 * CT;
                // k / in: k < 8 * 512 and in <= 8, so 65536 / in + 1 for 1 / in is exact
                const int ct = k * ((int)(65536.f * __builtin_amdgcn_rcpf((float)in)) + 1) >> 16;
                const int r0 = s.lo + (8 * sg + k - ct * in) * kTM;
                return Place{e, r0, min(s.hi - r0, kTM), ct};
            }
            k -= s.tiles * CT;
        }
        return Place{0, 0, 0, 0};
    }
};

constexpr int kMaxKB = MOE_MAX_GROUP_WIDTH / kBlk;

struct TileLds {
    char stage[2][kStage];  // rows, then weight rows
    uint8_t xs[2][4][kTM];  // e4m3: scale bytes of four units' rows, [wm][row % 16][i]
    uint32_t red[4][kTM];   // e4m3 gate/up: |h| maxima (their bits) of a row's four column groups
    char turn[8][16 * 144]; // a wave's results on their way from columns to rows
    uint8_t ws[2][2][kMaxKB];  // e4m3: a tile's weight scale bytes: of both matrices, or of 128 rows each
    int after;              // the tile after the next
    int32_t token[kTM];     // gate/up: of the (next) tile's rows
    int32_t offset[MOE_MAX_EXPERTS + 1];
};

template <bool FP8, bool TILED, bool GU>
__global__ __launch_bounds__(kTileThreads) void k_tile(Args a) {
    constexpr int ES = FP8 ? 1 : 2;
    __shared__ TileLds lds;
    // The arguments that are needed now and then are loaded again each time: kept, they would
    // push others out of the scalar registers.
    auto arg = [] {
        auto k = (const __attribute__((address_space(4))) Args*)__builtin_amdgcn_kernarg_segment_ptr();
        asm volatile("" : "+s"(k));
        return k;
    };
    auto groups = [&] {
        const auto k = arg();
        return Groups{lds.offset, k->N, k->S};
    };
    constexpr int TC = GU ? kTN / 2 : kTN;  // weight rows of each matrix in a tile
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int lr = lane & 15, q = lane >> 4, wm = wave >> 2, wn = wave & 3;
    const int KBy = a.K * ES, U = (KBy + kUnit - 1) / kUnit, KB = (a.K + kBlk - 1) / kBlk;
    const int CT = (a.R + TC - 1) / TC, RB = (a.R + kBlk - 1) / kBlk;
    // Work groups b, b + 8, ... share an XCD and its L2: each XCD has a run of tiles of an
    // eighth of the cost, of which its work groups take two each and then whoever is free
    // the next (which tile runs where does not change its result).
    for (int e = tid; e <= a.N; e += kTileThreads) lds.offset[e] = a.offset[e];
    __syncthreads();
    Tiles tiles;
    tiles.count(groups());
    const int xcd = blockIdx.x & 7, mine = blockIdx.x >> 3, step = gridDim.x >> 3;
    const int run = uni(tiles.bound(groups(), CT, xcd)), run_end = uni(tiles.bound(groups(), CT, xcd + 1));
    auto take = [&](int k) {  // in scalar registers: buffer descriptors and loops go by it
        Place t{0, 0, 0, 0};
        if (k < run_end - run) t = tiles.place(groups(), CT, run + k);
        return Place{uni(t.e), uni(t.r0), uni(t.rows), uni(t.ct)};
    };
    int after = mine + step;  // the tile after this one

    // What a tile's loads go by: offsets are one value a lane (chunk of a row's unit, rows of
    // 8 or a whole 1 KB block) plus one the wave holds.  Rows and weight rows come in eights.
    // Beyond a tile's rows, and for no tile, loads give zeros.
    const uint32_t wbytes = (uint32_t)a.R * (uint32_t)KBy;
    const uint32_t ca = ((lane & 7) ^ (lane >> 3)) * 16;     // this lane's chunk of a row's unit
    const uint32_t v8 = (uint32_t)(lane >> 3) * KBy + ca;    // in eight consecutive rows
    const int rem = KBy - (U - 1) * kUnit;                   // bytes of the last unit
    const uint32_t cut = (int)ca >= rem ? kOOB : 0u;
    struct Weights {
        __amdgpu_buffer_rsrc_t r;
        int row, rows;  // first matrix row of the tile; rows of the matrix, 0 for no tile
    };
    struct Rows {
        __amdgpu_buffer_rsrc_t r;  // down: the tile's rows of h
        int rows;
    };
    const auto rx = rsrc(a.x, GU ? (uint32_t)(a.S / a.m) * (uint32_t)KBy : 0u);  // gate/up: all of x
    // slot / m: with ceil(2^32 / m) for 2^32 / m it is exact as slot * m < 2^32
    const int last_slot = a.S - 1;
    const uint32_t inv_m = a.m > 1 ? 0xffffffffu / (uint32_t)a.m + 1 : 0;
    auto token = [&](int slot) {
        const uint32_t v = (uint32_t)min(max(slot, 0), last_slot);
        return inv_m ? __umulhi(v, inv_m) : v;
    };
    auto rows_of = [&](const Place& t) {
        return Rows{GU ? rx : rsrc(arg()->x + (int64_t)t.r0 * KBy, (uint32_t)t.rows * (uint32_t)KBy), t.rows};
    };
    auto weights_of = [&](const Place& t) {
        Weights o;
        o.r = rsrc((GU && wm ? arg()->w1 : arg()->w0) + (int64_t)t.e * wbytes, wbytes);
        o.row = t.ct * TC;
        o.rows = t.rows ? a.R : 0;
        return o;
    };
    // load i of a wave's four row and four weight loads of unit u
    auto load_rows = [&](const Rows& w, const uint32_t (&gather)[4], int u, char* stage, int i) {
        const int in = i * 8 + wave;
        uint32_t vo = GU ? gather[i] : v8;
        if (u == U - 1) vo |= cut;
        to_lds(GU ? rx : w.r, stage + in * 1024, in * 8 < w.rows ? vo : kOOB, u * kUnit + (GU ? 0 : in * 8 * KBy));
    };
    auto load_weights = [&](const Weights& w, int u, char* stage, int i) {
        const int in = i * 8 + wave;
        // staged weight row -> matrix row: wave columns of 64, gate/up 32 of each matrix
        // (rows 8 in with wm = 1 are W_up's)
        const int st = in * 8, row = w.row + (GU ? (st >> 6) * 32 + (st & 31) : st);
        if (TILED) {  // blocks of 16 rows by 64 bytes
            const bool in_range = row < w.rows && u * kUnit + (in & 1) * 64 < KBy;
            to_lds(w.r, stage + kStageA + in * 1024, in_range ? (uint32_t)lane * 16 : kOOB,
                   (row & ~15) * KBy + (u * 2 + (in & 1)) * 1024);
        } else {
            const uint32_t vo = u == U - 1 ? v8 | cut : v8;
            to_lds(w.r, stage + kStageA + in * 1024, row < w.rows ? vo : kOOB, row * KBy + u * kUnit);
        }
    };

    Place p = take(mine);
    if (!p.rows) return;
    // Gate/up: offsets of the tokens of a lane's rows; e4m3: of this thread's row's scale bytes.
    uint32_t gather[4] = {0, 0, 0, 0}, xrow = 0;
    auto row_of = [&](const Place& t) { return t.r0 + min(tid & (kTM - 1), max(t.rows - 1, 0)); };
    auto ask = [&](const Place& t) { return arg()->slot[row_of(t)]; };  // the slot of this thread's row
    auto keep = [&](int slot) {
        if (tid < kTM) lds.token[tid] = (int)token(slot);
    };
    auto address = [&](int first, int end) {  // of loads first .. end
#pragma unroll
        for (int i = first; i < end; ++i)
            gather[i] = (uint32_t)lds.token[(i * 8 + wave) * 8 + (lane >> 3)] * KBy + ca;
    };
    auto row_address = [&](const Place& t) {
        if (FP8) xrow = (uint32_t)(GU ? lds.token[tid & (kTM - 1)] : min(row_of(t), last_slot)) * KB;
    };
    if (GU) {
        keep(ask(p));
        __syncthreads();
        address(0, 4);
    }
    row_address(p);
    // e4m3 scale bytes.  Weights: a tile's, of 128 rows of each matrix or of two 128 rows, at
    // once.  Rows: a thread a row, four units at a time, the word that ends with the array
    // where it has fewer left.
    const uint32_t xs_bytes = (uint32_t)(GU ? a.S / a.m : a.S) * KB;
    uint32_t nx = 0, nx_shift = 0;  // row scale bytes on their way to shared memory
    auto row_scales = [&](uint32_t row, int u) {
        const uint32_t o = row + u, o4 = min(o, xs_bytes - 4);  // KB >= 4: whole words exist
        __builtin_memcpy(&nx, a.xs + o4, 4);
        nx_shift = 8 * (o - o4);
    };
    auto weight_scale = [&](const Place& t, int i) {  // byte i of a tile's two rows of KB
        const int half = i >= KB, k = min(i - half * KB, KB - 1);
        const int rb = min(t.ct * TC + (GU ? 0 : half * kBlk), a.R - 1) / kBlk;
        const uint8_t *s0 = arg()->s0, *s1 = GU ? arg()->s1 : s0;  // both pointers, then a lane's choice
        return (half ? s1 : s0)[((int64_t)t.e * RB + rb) * KB + k];
    };
    auto keep_weight_scale = [&](int par, int i, uint8_t v) {
        if (i < 2 * KB) lds.ws[par][i >= KB][i >= KB ? i - KB : i] = v;
    };
    const int sxat = ((tid >> 4) & 1) * 128 + (tid & 15) * 8 + ((tid >> 5) & 7);
    auto keep_rows = [&](int par) {
        const uint32_t v = nx >> nx_shift;
#pragma unroll
        for (int i = 0; i < 4; ++i) lds.xs[par][i][sxat] = (uint8_t)(v >> (8 * i));
    };
    {
    const Rows xr = rows_of(p);
    const Weights wr = weights_of(p);
    if (FP8) {
        for (int i = tid; i < 2 * KB; i += kTileThreads) keep_weight_scale(0, i, weight_scale(p, i));
        if (!wm) {
            row_scales(xrow, 0);
            keep_rows(0);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) load_weights(wr, 0, lds.stage[0], i);
#pragma unroll
    for (int i = 0; i < 4; ++i) load_rows(xr, gather, 0, lds.stage[0], i);
#pragma unroll
    for (int i = 0; i < 4; ++i) load_weights(wr, 1, lds.stage[1], i);
    load_rows(xr, gather, 1, lds.stage[1], 0);
    load_rows(xr, gather, 1, lds.stage[1], 1);
    }
    wait_vm<6>();
    wait_lds();
    block_barrier();
    if (wm) block_barrier();

    // a wave's stores of a tile: the same number whatever its rows, those of no row are dropped by their bounds
    constexpr auto stores_of = [](int nb) { return GU ? (FP8 ? nb / 2 + 1 : nb) : 2 * nb + (nb + 3) / 4; };
    int par = 0;      // the stage of the unit at hand
    int before = 0;   // row blocks of a wave in the tile before, whose stores may still be on their way
    auto wait_past = [&](auto n, int nb) {
        constexpr int N = decltype(n)::value;
        if (nb == 0) wait_vm<N>();
        else if (nb == 2) wait_vm<N + stores_of(2)>();
        else if (nb == 4) wait_vm<N + stores_of(4)>();
        else if (nb == 6) wait_vm<N + stores_of(6)>();
        else wait_vm<N + stores_of(8)>();
    };
    int xpar = 0, spar = 0;  // where the scale bytes of the rows and weights at hand are
    auto tile = [&](auto nb) {
        constexpr int NB = decltype(nb)::value, H = NB < 4 ? NB : 4;  // row blocks of a wave; of Ra and Ma
        constexpr int EARLY = FP8 && GU ? 0 : 4;  // row blocks of the second half read in Ma
        Place pn{0, 0, 0, 0};  // the next tile
        int got = 0;
        int slot_n = 0;           // the next tile's, as asked for
        uint8_t wsn[2] = {0, 0};  // its weight scale bytes
        Rows xa = rows_of(p), xb = xa;  // the first and the last 128 rows
        Weights wr = weights_of(p);
        f32x4 acc[NB][4];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int u = 0; u < U; ++u) {
            char* here = lds.stage[par];
            char* there = lds.stage[par ^ 1];
            u32x4 b[4][2], x[H][2];
            uint32_t ex[2] = {0u, 0u};
            auto read_rows = [&](int i) {  // row block i, into its place among the H
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
                    x[i % H][kk] = *reinterpret_cast<const u32x4*>(here + swz((i * 2 + wm) * 16 + lr, kk * 4 + q));
            };
            int e0 = 0, e1 = 0;
            // the products of row blocks first .. end, `then(i)` after those of block i
            auto products = [&](auto first, auto end, auto then) {
                constexpr int F = decltype(first)::value, E = decltype(end)::value;
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int i = F; i < E; ++i) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = mma_unit<FP8>(b[j][0], b[j][1], x[i % H][0], x[i % H][1], acc[i][j],
                                                  GU && j >= 2 ? e1 : e0, (int)ex[i / 4], i);
                    __builtin_amdgcn_sched_barrier(0);
                    then(i);
                    __builtin_amdgcn_sched_barrier(0);
                }
                __builtin_amdgcn_s_setprio(0);
#pragma unroll
                for (int i = F; i < E; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(acc[i][j]));  // they stay in this phase
            };
            // Ra
            int ua = u + 1, ub = u + 2;  // past the last unit: the next tile's first
            if (ua >= U) {
                xb = rows_of(pn);
                if (GU) address(2, 4);
                ua = 0;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
                    b[j][kk] = *reinterpret_cast<const u32x4*>(
                        here + kStageA +
                        (TILED ? (wn * 4 + j) * 2048 + kk * 1024 + lane * 16 : swz(wn * 64 + j * 16 + lr, kk * 4 + q)));
#pragma unroll
            for (int i = 0; i < H; ++i) read_rows(i);
            load_rows(xb, gather, ua, there, 2);
            load_rows(xb, gather, ua, there, 3);
            if (FP8) {
                const u32x2 v = *reinterpret_cast<const u32x2*>(&lds.xs[xpar][u & 3][wm * 128 + lr * 8]);
                ex[0] = v[0];
                ex[1] = v[1];
                e0 = lds.ws[spar][GU ? 0 : wn >> 1][u];
                if (GU) e1 = lds.ws[spar][1][u];
            }
            wait_lds();
            block_barrier();
            // Ma
            products(std::integral_constant<int, 0>(), std::integral_constant<int, H>(), [&](int i) {
                if (i < EARLY && i + H < NB) read_rows(i + H);
            });
            block_barrier();
            // Rb
            if (u == 0) {
                pn = take(after);
                if (GU) slot_n = ask(pn);
                if (tid == 0) {
                    int at = xcd * kLine;
                    asm volatile("" : "+v"(at));  // a lane's address: a wave's would be waited for at once
                    got = atomicAdd(&arg()->queue[at], 1);
                }
                if (FP8) {
                    wsn[0] = weight_scale(pn, tid);
                    if (KB > kTileThreads / 2) wsn[1] = weight_scale(pn, tid + kTileThreads);
                }
            } else if (u == 1) {
                if (FP8) {
                    keep_weight_scale(spar ^ 1, tid, wsn[0]);
                    if (KB > kTileThreads / 2) keep_weight_scale(spar ^ 1, tid + kTileThreads, wsn[1]);
                }
                if (GU) keep(slot_n);
                if (tid == 0) lds.after = got + 2 * step;
            } else if (ub == U) {
                wr = weights_of(pn);
                xa = rows_of(pn);
                if (GU) address(0, 2);
                row_address(pn);
                after = uni(lds.after);
            }
            if (ub >= U) ub -= U;
#pragma unroll
            for (int i = H + EARLY; i < NB; ++i) read_rows(i);
            if (FP8) {
                // The next four units' row scales (or the next tile's first) are asked for two units
                // ahead and kept one ahead.
                const bool turn4 = u + 1 == U || ((u + 1) & 3) == 0, ask4 = u + 2 == U || (((u + 2) & 3) == 0 && u + 2 < U);
                if (turn4) {
                    if (!wm) keep_rows(xpar ^ 1);
                    xpar ^= 1;
                }
                if (ask4 && !wm) row_scales(xrow, ub);
            }
            load_weights(wr, ub, here, 0);
            load_weights(wr, ub, here, 1);
            load_rows(xa, gather, ub, here, 0);
            wait_lds();
            wait_past(std::integral_constant<int, 5>(), u == 0 ? before : 0);
            block_barrier();
            // Mb
            auto last = [&] {
                load_weights(wr, ub, here, 2);
                load_weights(wr, ub, here, 3);
                load_rows(xa, gather, ub, here, 1);
            };
            if (NB <= H) last();
            products(std::integral_constant<int, H>(), nb, [&](int i) {
                if (i == (H + NB - 1) / 2) last();
            });
            wait_vm<6>();
            block_barrier();
            par ^= 1;
        }
        // A lane holds columns 4 q .. + 4 of 16, of row lr of each block; turned in shared memory,
        // four or eight lanes store 64 or 128 bytes of a row.
        char* turn = lds.turn[wave];
        int el = lane;
        asm volatile("" : "+v"(el));  // addresses below are formed here, not kept through the products
        const int er = el & 15, eq = el >> 4;
        if constexpr (GU) {
            const auto ro = rsrc(arg()->out + (int64_t)p.r0 * a.R * ES, (uint32_t)p.rows * a.R * ES);
            const int c0 = p.ct * TC + wn * 32;  // this wave's 32 columns of h
            uint32_t m[NB];  // |h|'s largest bits: the order of the values, with what is not finite above
            bool odd = false;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                m[i] = 0;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float h = silu(acc[i][j][k]) * acc[i][j + 2][k];
                        acc[i][j][k] = h;
                        if (FP8) m[i] = max(m[i], __float_as_uint(h) & 0x7fffffffu);  // columns past R: 0
                    }
                odd |= m[i] >= 0x7f800000u;
            }
            if constexpr (FP8) {
                odd = __any(odd);
                if (odd) {  // rare: what is not finite takes no part
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        m[i] = 0;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int k = 0; k < 4; ++k) m[i] = max(m[i], __float_as_uint(mag(acc[i][j][k])));
                    }
                }
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    m[i] = max(m[i], (uint32_t)__shfl_xor((int)m[i], 16, 64));
                    m[i] = max(m[i], (uint32_t)__shfl_xor((int)m[i], 32, 64));
                    if (eq == 0) lds.red[wn][(i * 2 + wm) * 16 + er] = m[i];
                }
                wait_lds();
                block_barrier();
                auto exp_of = [&](int rr) {
                    return block_exp(__uint_as_float(
                        max(max(lds.red[0][rr], lds.red[1][rr]), max(lds.red[2][rr], lds.red[3][rr]))));
                };
                // codes, two blocks of rows at a time: 32 rows of 32 bytes
#pragma unroll
                for (int i = 0; i < NB; i += 2) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float inv = pow2(-exp_of(((i + k) * 2 + wm) * 16 + er));
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const f32x4 h = acc[i + k][j];
                            *reinterpret_cast<uint32_t*>(turn + (k * 16 + er) * 48 + j * 16 + 4 * eq) =
                                odd ? codes4(h[0], h[1], h[2], h[3], inv) : finite_codes4(h, inv);
                        }
                    }
                    const u32x4 v = *reinterpret_cast<const u32x4*>(turn + (el >> 1) * 48 + (el & 1) * 16);
                    const int rr = ((i + (el >> 5)) * 2 + wm) * 16 + ((el >> 1) & 15), c = c0 + (el & 1) * 16;
                    __builtin_amdgcn_raw_buffer_store_b128(v, ro, c < a.R ? (uint32_t)rr * a.R + c : kOOB, 0, 0);
                }
                // scale bytes: wave column wn those of two blocks
                const int i = wn * 2 + (el >> 4), rr = (i * 2 + wm) * 16 + er;
                const auto rso = rsrc(arg()->outs + (int64_t)p.r0 * CT, (uint32_t)p.rows * CT);
                __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(exp_of(rr & (kTM - 1)) + 127), rso,
                                                     el < 32 && i < NB ? rr * CT + p.ct : kOOB, 0, 0);
            } else {
#pragma unroll
                for (int i = 0; i < NB; ++i) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const f32x4 h = acc[i][j];
                        *reinterpret_cast<u32x2*>(turn + er * 80 + j * 32 + 8 * eq) =
                            u32x2{bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3])};
                    }
                    const u32x4 v = *reinterpret_cast<const u32x4*>(turn + (el >> 2) * 80 + (el & 3) * 16);
                    const int rr = (i * 2 + wm) * 16 + (el >> 2), c = c0 + (el & 3) * 8;
                    __builtin_amdgcn_raw_buffer_store_b128(v, ro, c < a.R ? ((uint32_t)rr * a.R + c) * 2 : kOOB, 0, 0);
                }
            }
        } else {
            const auto ro = rsrc(arg()->out + (int64_t)p.r0 * a.R * 2, (uint32_t)p.rows * a.R * 2);
            const int c0 = p.ct * TC + wn * 64;  // this wave's 64 columns, a block of O
            int byte[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                float v[4][4];  // read once from the accumulators
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        v[j][k] = acc[i][j][k];
                        asm volatile("" : "+v"(v[j][k]));
                        m = max(m, __float_as_uint(v[j][k]) & 0x7fffffffu);
                    }
                if (__any(m >= 0x7f800000u)) {  // rare: what is not finite takes no part
                    m = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int k = 0; k < 4; ++k) m = max(m, __float_as_uint(mag(v[j][k])));
                }
                byte[i] = term_byte(quad_max(m));
                const float inv = __uint_as_float((uint32_t)(268 - byte[i]) << 23);  // 2^(141 - byte)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float* o = v[j];
                    *reinterpret_cast<u32x2*>(turn + er * 144 + j * 32 + 8 * eq) =
                        u32x2{f16_pair(o[0] * inv, o[1] * inv), f16_pair(o[2] * inv, o[3] * inv)};
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int r = k * 8 + (el >> 3);
                    const u32x4 row = *reinterpret_cast<const u32x4*>(turn + r * 144 + (el & 7) * 16);
                    const int rr = (i * 2 + wm) * 16 + r, c = c0 + (el & 7) * 8;
                    __builtin_amdgcn_raw_buffer_store_b128(row, ro, c < a.R ? ((uint32_t)rr * a.R + c) * 2 : kOOB, 0, 0);
                }
            }
            // the bytes of four row blocks at a time, a lane a row
            const int OB = (a.R + 63) / 64, ob = p.ct * (TC / 64) + wn;
            const auto rso = rsrc(arg()->outs + (int64_t)p.r0 * OB, (uint32_t)p.rows * OB);
#pragma unroll
            for (int i = 0; i < NB; i += 4) {
                int v = byte[i];
#pragma unroll
                for (int k = 1; k < 4; ++k) v = i + k < NB && eq == k ? byte[min(i + k, NB - 1)] : v;
                const int rr = ((i + eq) * 2 + wm) * 16 + er;
                __builtin_amdgcn_raw_buffer_store_b8((uint8_t)v, rso, i + eq < NB && ob < OB ? (uint32_t)rr * OB + ob : kOOB,
                                                     0, 0);
            }
        }
        before = NB;
        spar ^= 1;
        return pn;
    };
    while (p.rows) {
        Place pn;
        if (p.rows <= 64) pn = tile(std::integral_constant<int, 2>());
        else if (p.rows <= 128) pn = tile(std::integral_constant<int, 4>());
        else if (p.rows <= 192) pn = tile(std::integral_constant<int, 6>());
        else pn = tile(std::integral_constant<int, 8>());
        // values of the wave, which the compiler no longer knows them to be where tiles of several heights meet
        p = Place{uni(pn.e), uni(pn.r0), uni(pn.rows), uni(pn.ct)};
        after = uni(after);
        par = uni(par);
        before = uni(before);
        xpar = uni(xpar);
        spar = uni(spar);
    }
    wait_vm<0>();  // the zeros of no tile are still on their way to shared memory
    if (!wm) block_barrier();
}

__global__ __launch_bounds__(kQueue) void k_zero_queue(int32_t* __restrict__ queue) { queue[threadIdx.x] = 0; }

// The row of each slot that has one; an empty queue.
__global__ __launch_bounds__(256) void k_row_of(const int32_t* __restrict__ slot, const int32_t* __restrict__ rows,
                                               int S, int32_t* __restrict__ row_of, int32_t* __restrict__ queue) {
    if (blockIdx.x == 0) queue[threadIdx.x] = 0;
    const int r = blockIdx.x * 256 + threadIdx.x;
    if (r < min(*rows, S)) row_of[min(max(slot[r], 0), S - 1)] = r;
}

// y_t = sum_j w_tj O_tj over the slots with a valid id, in increasing j, in fp32, rounded
// to bf16 once.  A wave takes 512 columns of a token (eight a lane); the lanes look up the
// token's slots together, so that the loads of O go out eight at a time: they are the time
// (4096 tokens of 8 x 2048 in 25 us: 151 MB at 6 TB/s).
//
// O, a partial sum of y, is fp32 from thin tiles, which costs them nothing that shows (passes of one token
// 26 us, of 32 tokens 91 us either way).  From square tiles fp32 would be 134 MB more each way for 4096 tokens of
// 8 x 2048, so there it is fp16 with a power of two for each 64 columns of a row (two bytes and 1/64 an element):
// 11 bits, three more than bf16, each term off by at most 2^-11 |w_j O_j| (half a step; and 2^-39 of its block's largest).
//                                            bf16   this   fp32
//     8-bit down of 4096 x 8 tokens, us        129    142    168
//     8-bit pass of 8191 x 8                   486    502    581
//     bf16 down of 2777 x 6                    159    165    180
//     wide bf16 pass of 2048 x 2              1602   1610   1625
// The error of y in that bf16 down is 0.0023 (norm) with bf16 terms and 0.0017 here, that of rounding y.
// (Long passes whose contraction is too short for square tiles pay for fp32: down of 4096 x 8 tokens of 16
// experts, 1024 x 176 in bf16, 128 -> 136 us, 1024 x 368 in e4m3 142 -> 153.)
// What is not finite is itself in fp16 and takes no part in a block's largest.
// info (may be null): U, ids status, MOE_OK.
template <bool F32>
__global__ __launch_bounds__(256) void k_combine(const char* __restrict__ O, const uint8_t* __restrict__ os,
                                                const int32_t* __restrict__ row_of,
                                                const int32_t* __restrict__ ids, const float* __restrict__ w, int64_t n,
                                                int m, int N, int d,
                                                int accumulate, char* __restrict__ y, const int32_t* __restrict__ u_err,
                                                int32_t* __restrict__ info) {
    const int lane = threadIdx.x & 63, CW = (d + 511) / 512, OB = (d + 63) / 64, last = (int)(n * m) - 1;
    if (info && blockIdx.x == 0 && threadIdx.x < 3) info[threadIdx.x] = threadIdx.x < 2 ? u_err[threadIdx.x] : MOE_OK;
    for (int64_t i = (int64_t)blockIdx.x * 4 + uni(threadIdx.x >> 6); i < n * CW; i += (int64_t)gridDim.x * 4) {
        const int64_t t = i / CW;
        const int c0 = (int)(i - t * CW) * 512, c = c0 + lane * 8;
        const bool in = c < d;
        float s[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] = 0.f;
        for (int j0 = 0; j0 < m; j0 += 64) {
            // this lane's slot: its row (-1: none) and weight
            int row = -1;
            float wj = 0.f;
            if (j0 + lane < m) {
                const int64_t slot = t * m + j0 + lane;
                const int id = ids[slot], r = min(max(row_of[slot], 0), last);
                wj = w[slot];
                row = id >= 0 && id < N ? r : -1;
            }
            uint64_t live = __ballot(row >= 0);
            while (live) {
                u32x4 o[8][F32 ? 2 : 1];
                float wt[8];
                int rows8 = 0;  // of lane 8 k + b: row k of the eight
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int l = live ? __ffsll((unsigned long long)live) - 1 : 64;
                    live &= live - 1;
#pragma unroll
                    for (auto& p : o[k]) p = u32x4{0u, 0u, 0u, 0u};
                    wt[k] = 0.f;
                    if (l < 64) {
                        const int64_t r = __builtin_amdgcn_readlane(row, l);
                        wt[k] = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(wj), l));
                        const u32x4* at = reinterpret_cast<const u32x4*>(O + (r * d + c) * (F32 ? 4 : 2));
                        if (in) o[k][0] = at[0];
                        if constexpr (F32) {
                            if (in) o[k][1] = at[1];
                        } else {
                            rows8 = lane >> 3 == k ? (int)r : rows8;
                        }
                    }
                }
                int byte = 0;
                if (!F32) byte = os[(int64_t)rows8 * OB + min((c0 >> 6) + (lane & 7), OB - 1)];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float f = F32 ? 1.f : pow2(__shfl(byte, k * 8 + (lane >> 3), 64) - 141);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        if constexpr (F32) {
                            s[v] += wt[k] * __uint_as_float(o[k][0][v]);
                            s[4 + v] += wt[k] * __uint_as_float(o[k][1][v]);
                        } else {
                            const f32x2 t2 = f16_values(o[k][0][v]);
                            s[2 * v] += wt[k] * (t2[0] * f);
                            s[2 * v + 1] += wt[k] * (t2[1] * f);
                        }
                    }
                }
            }
        }
        if (!in) continue;
        u32x4* p = reinterpret_cast<u32x4*>(y + (t * d + c) * 2);
        if (accumulate) {
            const u32x4 v = *p;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s[2 * k] += bf16_lo(v[k]);
                s[2 * k + 1] += bf16_hi(v[k]);
            }
        }
        *p = u32x4{bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3]), bf16_pair(s[4], s[5]), bf16_pair(s[6], s[7])};
    }
}

}  // namespace moe_g
