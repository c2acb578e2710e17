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
    char* out;            // gate/up: h [S][R]; down: O [S][R]
    uint8_t* outs;        // e4m3 gate/up: scale bytes of h
    int N, m, S, R, K;
};

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// One unit's product; sa, sb: the operands' scale bytes (e4m3).
template <bool FP8>
__device__ __forceinline__ f32x4 mma_unit(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1, f32x4 c, int sa, int sb) {
    if (FP8) {
        struct Pair {
            u32x4 lo, hi;
        };
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8, Pair{a0, a1}),
                                                                __builtin_bit_cast(i32x8, Pair{b0, b1}), c, 0, 0, 0, sa,
                                                                0, sb);
    }
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a0), __builtin_bit_cast(bf16x8_t, b0), c,
                                                0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a1), __builtin_bit_cast(bf16x8_t, b1),
                                                   c, 0, 0, 0);
}

// silu(z) = z / (1 + exp(-z)); exp(-z) overflows to infinity below z = -88: -0.
__device__ __forceinline__ float silu(float z) { return z / (1.f + __expf(-z)); }

__device__ __forceinline__ uint32_t bf16_bits(float v) {
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) { return bf16_bits(a) | (bf16_bits(b) << 16); }
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

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

// Rows of bf16 (or float32) values to codes and scale bytes, in blocks of 128 along the row:
// sixteen lanes a block, eight values a lane.
template <bool F32>
__global__ __launch_bounds__(256) void k_quant_rows(const char* __restrict__ x, int64_t rows, int K,
                                                   const int32_t* __restrict__ limit, uint8_t* __restrict__ q,
                                                   uint8_t* __restrict__ s) {
    const int KB = (K + kBlk - 1) / kBlk;
    if (limit) rows = min(rows, (int64_t)max(*limit, 0));
    const int64_t blocks = rows * KB;
    const int l = threadIdx.x & 15;
    for (int64_t b = (int64_t)blockIdx.x * 16 + threadIdx.x / 16; b < blocks; b += (int64_t)gridDim.x * 16) {
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

// Codes and scale bytes of rows back to bf16: four bits of significand fit bf16's eight,
// so this is exact down to bf16's own least value.
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
// chunk adds up the chunks before it and writes its slots behind them.  The rank of a
// slot among equal ids of its wave's 64 comes from one ballot for each bit of the id, so
// the order is that of the slots, whatever the timing.
constexpr int kGThreads = 1024, kGWaves = kGThreads / 64;
constexpr int kGMaxChunks = 64;

__host__ __device__ __forceinline__ int64_t group_chunk(int64_t S) {
    const int64_t c = (S + kGMaxChunks - 1) / kGMaxChunks;
    return (c + kGThreads - 1) / kGThreads * kGThreads;
}

// ids of this lane's slot, -1 outside [0, N) or past the end; sets bad for an invalid or
// repeated id
__device__ __forceinline__ int group_id(const int32_t* ids, int64_t s, int64_t S, int m, int N, bool& bad) {
    if (s >= S) return -1;
    const int id = ids[s];
    if (id < 0 || id >= N) {
        bad = true;
        return -1;
    }
    const int j = (int)(s % m);
    for (int i = 1; i <= j; ++i)
        if (ids[s - i] == id) bad = true;
    return id;
}

__global__ __launch_bounds__(kGThreads) void k_group_hist(const int32_t* __restrict__ ids, int64_t S, int m, int N,
                                                         int32_t* __restrict__ hist) {
    __shared__ int cnt[MOE_MAX_EXPERTS];
    __shared__ int flag;
    const int tid = threadIdx.x;
    const int64_t chunk = group_chunk(S), s0 = blockIdx.x * chunk;
    for (int e = tid; e < N; e += kGThreads) cnt[e] = 0;
    if (tid == 0) flag = 0;
    __syncthreads();
    bool bad = false;
    for (int64_t i = tid; i < chunk; i += kGThreads) {
        const int id = group_id(ids, s0 + i, S, m, N, bad);
        if (id >= 0) atomicAdd(&cnt[id], 1);
    }
    if (bad) atomicOr(&flag, 1);
    __syncthreads();
    int32_t* h = hist + (int64_t)blockIdx.x * (N + 1);
    for (int e = tid; e < N; e += kGThreads) h[e] = cnt[e];
    if (tid == 0) h[N] = flag;
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
    for (int i = 0; i < kGWaves; ++i) {
        before += i < wave ? part[i] : 0;
        all += part[i];
    }
    __syncthreads();
    total = all;
    return before + s - v;
}

__global__ __launch_bounds__(kGThreads) void k_group_scatter(const int32_t* __restrict__ ids, int64_t S, int m, int N,
                                                            const int32_t* __restrict__ hist, int32_t* __restrict__ count,
                                                            int32_t* __restrict__ offset, int32_t* __restrict__ sbe,
                                                            int32_t* __restrict__ distinct, int32_t* __restrict__ u_err) {
    __shared__ int base[kGWaves * MOE_MAX_EXPERTS];  // [wave][N]: next place of the wave's slots
    __shared__ int part[kGWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int G = gridDim.x, g = blockIdx.x;
    const int64_t chunk = group_chunk(S), s0 = g * chunk;
    const int64_t per = chunk / kGWaves;  // a multiple of 64
    for (int i = tid; i < kGWaves * N; i += kGThreads) base[i] = 0;
    __syncthreads();
    // this wave's own histogram
    for (int64_t i = lane; i < per; i += 64) {
        const int64_t s = s0 + wave * per + i;
        const int id = s < S ? ids[s] : -1;
        if (id >= 0 && id < N) atomicAdd(&base[wave * N + id], 1);
    }
    // thread e: expert e's slots in the chunks before this one, and in all
    int before = 0, all = 0, bad = 0;
    if (tid < N)
        for (int c = 0; c < G; ++c) {
            const int v = hist[(int64_t)c * (N + 1) + tid];
            before += c < g ? v : 0;
            all += v;
        }
    int valid;
    const int start = group_scan(all, part, valid);
    int U;
    const int dpos = group_scan(tid < N && all > 0, part, U);
    if (tid < N) {
        int at = start + before;
        for (int w = 0; w < kGWaves; ++w) {
            const int c = base[w * N + tid];
            base[w * N + tid] = at;
            at += c;
        }
        if (g == 0) {
            count[tid] = all;
            offset[tid] = start;
            if (all > 0) distinct[dpos] = tid;
            if (tid >= U) distinct[tid] = -1;
        }
    }
    if (g == 0) {
        if (tid < G) bad = hist[(int64_t)tid * (N + 1) + N];
        bad = __syncthreads_or(bad);
        if (tid == 0) {
            offset[N] = valid;
            u_err[0] = U;
            u_err[1] = bad ? MOE_E_IDS : MOE_OK;
        }
    }
    __syncthreads();
    for (int64_t i = lane; i < per; i += 64) {
        const int64_t s = s0 + wave * per + i;
        int id = s < S ? ids[s] : -1;
        const bool ok = id >= 0 && id < N;
        uint64_t same = __ballot(ok);
        for (int b = 0; (1 << b) < N; ++b) {
            const uint64_t v = __ballot((id >> b) & 1);
            same &= ((id >> b) & 1) ? v : ~v;
        }
        if (ok) {
            const uint64_t under = same & ((1ull << lane) - 1);
            const int at = base[wave * N + id];
            sbe[at + __popcll(under)] = (int)s;
            __builtin_amdgcn_wave_barrier();
            if (under == 0) base[wave * N + id] = at + __popcll(same);
        }
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // the places that no slot takes
    for (int64_t r = valid + (int64_t)g * kGThreads + tid; r < S; r += (int64_t)G * kGThreads) sbe[r] = -1;
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
// expert, where the weights' bytes are the time.
constexpr int kThinWaves = 4, kThinAhead = 4;  // units of a wave's loads in flight

template <bool FP8, bool TILED, bool GU>
__global__ __launch_bounds__(64 * kThinWaves) void k_thin(Args a) {
    constexpr int ES = FP8 ? 1 : 2, NW = GU ? 2 : 1;
    __shared__ f32x4 red[kThinWaves][NW][64];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int lr = lane & 15, q = lane >> 4;
    const int CB = (a.R + 15) / 16;
    const int tile = blockIdx.x / CB, cb = blockIdx.x - tile * CB;
    const TileAt t = find_tile(a.offset, a.N, a.S, kTile16, tile);
    if (t.e < 0) return;
    const int KBy = a.K * ES, U = (KBy + kUnit - 1) / kUnit, KB = (a.K + kBlk - 1) / kBlk;
    const int row = min(t.r0 + lr, t.end - 1);
    const int slot = min(max(a.slot[row], 0), a.S - 1);
    const int64_t xrow = GU ? slot / a.m : row;
    const char* xp = a.x + xrow * KBy;
    const char* wp[2];
    const int wr = min(cb * 16 + lr, a.R - 1);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const char* w = (i ? a.w1 : a.w0) + (int64_t)t.e * a.R * KBy;
        wp[i] = TILED ? w + (int64_t)cb * 16 * KBy + lane * 16 : w + (int64_t)wr * KBy;
    }
    const uint8_t* sx = FP8 ? a.xs + xrow * KB : nullptr;
    const int RB = (a.R + kBlk - 1) / kBlk;
    const int64_t sw = FP8 ? ((int64_t)t.e * RB + cb * 16 / kBlk) * KB : 0;
    f32x4 acc[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int u0 = wave; u0 < U; u0 += kThinWaves * kThinAhead) {
        u32x4 b[kThinAhead][2], w[kThinAhead][NW][2];
        int eb[kThinAhead], ew[kThinAhead][NW];
#pragma unroll
        for (int p = 0; p < kThinAhead; ++p) {
            const int u = u0 + p * kThinWaves;
            eb[p] = 0;
#pragma unroll
            for (int i = 0; i < NW; ++i) ew[p][i] = 0;
            if (FP8 && u < U) {
                eb[p] = sx[u];
                ew[p][0] = a.s0[sw + u];
                if (GU) ew[p][NW - 1] = a.s1[sw + u];
            }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const int k = u * kUnit + kk * 64 + q * 16;
                const bool ok = u < U && k < KBy;
                b[p][kk] = ok ? *reinterpret_cast<const u32x4*>(xp + k) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                for (int i = 0; i < NW; ++i)
                    w[p][i][kk] = ok ? *reinterpret_cast<const u32x4*>(
                                           wp[i] + (TILED ? (int64_t)(2 * u + kk) * 1024 : (int64_t)k))
                                     : u32x4{0u, 0u, 0u, 0u};
            }
        }
#pragma unroll
        for (int p = 0; p < kThinAhead; ++p)
#pragma unroll
            for (int i = 0; i < NW; ++i)
                acc[i] = mma_unit<FP8>(w[p][i][0], w[p][i][1], b[p][0], b[p][1], acc[i], ew[p][i], eb[p]);
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) red[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave) return;
    f32x4 v[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        v[i] = red[0][i][lane];
#pragma unroll
        for (int k = 1; k < kThinWaves; ++k) v[i] += red[k][i][lane];
    }
    const int c = cb * 16 + 4 * q;
    if (t.r0 + lr >= t.end || c >= a.R) return;
    if (GU) {
        float h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = silu(v[0][i]) * v[NW - 1][i];
        if (FP8)  // float32, quantised by a launch of its own: a block's maximum is over 128 columns
            *reinterpret_cast<f32x4*>(a.out + ((int64_t)row * a.R + c) * 4) = f32x4{h[0], h[1], h[2], h[3]};
        else
            *reinterpret_cast<u32x2*>(a.out + ((int64_t)row * a.R + c) * 2) =
                u32x2{bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3])};
    } else {
        *reinterpret_cast<u32x2*>(a.out + ((int64_t)slot * a.R + c) * 2) =
            u32x2{bf16_pair(v[0][0], v[0][1]), bf16_pair(v[0][2], v[0][3])};
    }
}

// Square tiles: up to 256 rows by 256 weight rows (gate/up: 128 of each matrix, so 128
// columns of h), eight waves as 2 x 4, each up to 128 rows by 64 weight rows in registers.
// Units of both operands go to shared memory two deep; a wave takes the 16-row blocks
// 2 i + wm, so a tile of few rows is shared by both wave rows.
constexpr int kTM = 256, kTN = 256, kTileThreads = 512;
constexpr int kStage = (kTM + kTN) * kUnit;
constexpr uint32_t kOOB = 0x80000000u;  // beyond every buffer: reads give zero

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
// 1 KB of memory, 16 bytes a lane, to shared memory in lane order
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t vo, uint32_t so) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, (int)vo, (int)so, 0, 0);
}
// place of 16-byte chunk c of row r in shared memory's 128-byte rows
__device__ __forceinline__ int swz(int r, int c) { return r * kUnit + ((c ^ (r & 7)) << 4); }

struct Place {
    int e, r0, rows, ct;
};

// Work group b's tile: expert, rows and column tile.  Work groups b, b + 8, ... share an
// XCD and its L2: each XCD takes a run of tiles, in which the column tiles of up to 8 row
// tiles are neighbours.
__device__ __forceinline__ Place find_place(const Args& a, int CT, int b) {
    const int lane = threadIdx.x & 63, C = (a.N + 63) / 64;
    int sum = 0;
    for (int i = 0; i < C; ++i) {
        const int e = lane * C + i;
        if (e < a.N) {
            const int lo = min(max(a.offset[e], 0), a.S), hi = min(max(a.offset[e + 1], lo), a.S);
            sum += (hi - lo + kTM - 1) / kTM;
        }
    }
    int s = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(s, o, 64);
        if (lane >= o) s += u;
    }
    const int total = __shfl(s, 63, 64) * CT;
    const int per = (total + 7) / 8;
    const int t = (b & 7) * per + (b >> 3);
    if ((b >> 3) >= per || t >= total) return Place{-1, 0, 0, 0};
    const uint64_t past = __ballot(s * CT > t);
    const int from = __ffsll((unsigned long long)past) - 1;
    int k = t - (__shfl(s, from, 64) - __shfl(sum, from, 64)) * CT;
    for (int i = 0; i < C; ++i) {
        const int e = from * C + i;
        if (e >= a.N) break;
        const int lo = min(max(uni(a.offset[e]), 0), a.S), hi = min(max(uni(a.offset[e + 1]), lo), a.S);
        const int rt = (hi - lo + kTM - 1) / kTM;
        if (k < rt * CT) {
            const int sg = k / (8 * CT), in = min(8, rt - 8 * sg);
            k -= sg * 8 * CT;
            const int r0 = lo + (8 * sg + k % in) * kTM;
            return Place{e, r0, min(hi - r0, kTM), k / in};
        }
        k -= rt * CT;
    }
    return Place{-1, 0, 0, 0};
}

struct TileLds {
    char stage[2][kStage];
    uint8_t xs[2][kTM];     // e4m3: scale bytes of a unit's rows, [wm][row % 16][i]
    float red[4][kTM];      // e4m3 gate/up: |h| maxima of a row's four column groups
};

template <bool FP8, bool TILED, bool GU>
__global__ __launch_bounds__(kTileThreads) void k_tile(Args a) {
    constexpr int ES = FP8 ? 1 : 2;
    __shared__ TileLds lds;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int lr = lane & 15, q = lane >> 4, wm = wave >> 2, wn = wave & 3;
    const int KBy = a.K * ES, U = (KBy + kUnit - 1) / kUnit, KB = (a.K + kBlk - 1) / kBlk;
    constexpr int TC = GU ? kTN / 2 : kTN;  // weight rows of each matrix in a tile
    const int CT = (a.R + TC - 1) / TC;
    const Place p = find_place(a, CT, blockIdx.x);
    if (p.e < 0) return;
    const int R16 = (p.rows + 15) / 16;
    // operands: rows of x through the slots (gate/up) or consecutive rows of h
    const auto rx = GU ? rsrc(a.x, (uint32_t)((int64_t)(a.S / a.m) * KBy))
                       : rsrc(a.x + (int64_t)p.r0 * KBy, (uint32_t)p.rows * KBy);
    const uint32_t wbytes = (uint32_t)((int64_t)a.R * KBy);
    const auto rw0 = rsrc(a.w0 + (int64_t)p.e * wbytes, wbytes);
    const auto rw1 = GU ? rsrc(a.w1 + (int64_t)p.e * wbytes, wbytes) : rw0;
    const int ca = ((lane & 7) ^ (lane >> 3)) * 16;  // byte of this lane's chunk in a row's unit
    uint32_t va[4], vb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int in = i * 8 + wave;
        int r = min(in * 8 + (lane >> 3), p.rows - 1);
        if (GU) r = min(max(a.slot[p.r0 + r], 0), a.S - 1) / a.m;
        va[i] = (uint32_t)r * KBy + ca;
        // staged weight row -> matrix row: wave columns wn of 64: gate/up 32 of each
        if (TILED) {
            const int blk = in >> 1;  // 16 rows
            const int row = p.ct * TC + (GU ? (blk >> 2) * 32 + (blk & 1) * 16 : blk * 16);
            vb[i] = row < a.R ? (uint32_t)row * KBy + (in & 1) * 1024 + lane * 16 : kOOB;
        } else {
            const int st = in * 8 + (lane >> 3);
            const int row = p.ct * TC + (GU ? (st >> 6) * 32 + (st & 31) : st);
            vb[i] = row < a.R ? (uint32_t)row * KBy + ca : kOOB;
        }
    }
    const uint8_t *sx = nullptr, *s0 = nullptr, *s1 = nullptr;
    if (FP8) {
        int64_t r = min(tid & (kTM - 1), p.rows - 1) + p.r0;
        if (GU) r = min(max(a.slot[r], 0), a.S - 1) / a.m;
        sx = a.xs + r * KB;
        const int RB = (a.R + kBlk - 1) / kBlk;
        const int64_t at = ((int64_t)p.e * RB + min(p.ct * TC + (GU ? 0 : wn * 64), a.R - 1) / kBlk) * KB;
        s0 = a.s0 + at;
        if (GU) s1 = a.s1 + at;
    }
    const int sxat = ((tid >> 4) & 1) * 128 + (tid & 15) * 8 + ((tid >> 5) & 7);
    auto stage = [&](int u) {
        char* A = lds.stage[u & 1];
        char* B = A + kTM * kUnit;
        const int left = KBy - u * kUnit;
        const bool tail = left < kUnit;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int in = i * 8 + wave;
            if (in < R16 * 2) to_lds(rx, A + in * 1024, tail && ca >= left ? kOOB : va[i], u * kUnit);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int in = i * 8 + wave;
            const bool up = GU && (TILED ? (in >> 2) & 1 : (in >> 2) & 1);
            const bool off = tail && (TILED ? (in & 1) * 64 >= left : ca >= left);
            to_lds(up ? rw1 : rw0, B + in * 1024, off ? kOOB : vb[i], u * (TILED ? 2048 : kUnit));
        }
    };

    auto run = [&](auto nb) {
        constexpr int NB = decltype(nb)::value;
        f32x4 acc[NB][4];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        int nx = 0, n0 = 0, n1 = 0;  // the next unit's scale bytes
        if (FP8) {
            nx = sx[0];
            n0 = s0[0];
            if (GU) n1 = s1[0];
        }
        stage(0);
        for (int u = 0; u < U; ++u) {
            int e0 = 0, e1 = 0;
            if (FP8) {
                if (tid < kTM) lds.xs[u & 1][sxat] = (uint8_t)nx;
                e0 = n0;
                e1 = n1;
            }
            __syncthreads();
            if (u + 1 < U) {
                stage(u + 1);
                if (FP8) {
                    nx = sx[u + 1];
                    n0 = s0[u + 1];
                    if (GU) n1 = s1[u + 1];
                }
            }
            const char* A = lds.stage[u & 1];
            const char* B = A + kTM * kUnit;
            u32x4 b[4][2];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
                    b[j][kk] = *reinterpret_cast<const u32x4*>(
                        B + (TILED ? (wn * 4 + j) * 2048 + kk * 1024 + lane * 16 : swz(wn * 64 + j * 16 + lr, kk * 4 + q)));
            uint32_t ex[2] = {0u, 0u};
            if (FP8) {
                const u32x2 v = *reinterpret_cast<const u32x2*>(&lds.xs[u & 1][wm * 128 + lr * 8]);
                ex[0] = v[0];
                ex[1] = v[1];
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                u32x4 x[2];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
                    x[kk] = *reinterpret_cast<const u32x4*>(A + swz((i * 2 + wm) * 16 + lr, kk * 4 + q));
                const int e = (int)(ex[i >> 2] >> (8 * (i & 3)));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = mma_unit<FP8>(b[j][0], b[j][1], x[0], x[1], acc[i][j], GU && j >= 2 ? e1 : e0, e);
            }
        }
        // a lane holds columns 4 q .. + 4 of 16, of row lr of each block
        if (GU) {
            float m[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                m[i] = 0.f;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float h = silu(acc[i][j][k]) * acc[i][j + 2][k];
                        acc[i][j][k] = h;
                        if (FP8) m[i] = fmaxf(m[i], p.ct * TC + wn * 32 + j * 16 + 4 * q + k < a.R ? mag(h) : 0.f);
                    }
            }
            if (FP8) {
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    m[i] = fmaxf(m[i], __shfl_xor(m[i], 16, 64));
                    m[i] = fmaxf(m[i], __shfl_xor(m[i], 32, 64));
                    if (q == 0) lds.red[wn][(i * 2 + wm) * 16 + lr] = m[i];
                }
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int rr = (i * 2 + wm) * 16 + lr;
                if (rr >= p.rows) continue;
                const int64_t row = p.r0 + rr;
                float inv = 1.f;
                if (FP8) {
                    const int k = block_exp(fmaxf(fmaxf(lds.red[0][rr], lds.red[1][rr]), fmaxf(lds.red[2][rr], lds.red[3][rr])));
                    inv = pow2(-k);
                    if (wn == 0 && q == 0) a.outs[row * CT + p.ct] = (uint8_t)(k + 127);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = p.ct * TC + wn * 32 + j * 16 + 4 * q;
                    const f32x4 h = acc[i][j];
                    if (c >= a.R) continue;
                    if (FP8)
                        *reinterpret_cast<uint32_t*>(a.out + row * a.R + c) = codes4(h[0], h[1], h[2], h[3], inv);
                    else
                        *reinterpret_cast<u32x2*>(a.out + (row * a.R + c) * 2) =
                            u32x2{bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3])};
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int rr = (i * 2 + wm) * 16 + lr;
                if (rr >= p.rows) continue;
                const int64_t slot = min(max(a.slot[p.r0 + rr], 0), a.S - 1);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = p.ct * TC + wn * 64 + j * 16 + 4 * q;
                    if (c < a.R)
                        *reinterpret_cast<u32x2*>(a.out + (slot * a.R + c) * 2) =
                            u32x2{bf16_pair(acc[i][j][0], acc[i][j][1]), bf16_pair(acc[i][j][2], acc[i][j][3])};
                }
            }
        }
    };
    const int nb = (R16 + 1) / 2;
    if (nb <= 1) run(std::integral_constant<int, 1>());
    else if (nb <= 2) run(std::integral_constant<int, 2>());
    else if (nb <= 4) run(std::integral_constant<int, 4>());
    else run(std::integral_constant<int, 8>());
}

// y_t = sum_j w_tj O_tj over the slots with a valid id, in increasing j, in fp32, rounded
// to bf16 once; eight columns a thread.  info (may be null): U, ids status, MOE_OK.
__global__ __launch_bounds__(256) void k_combine(const char* __restrict__ O, const int32_t* __restrict__ ids,
                                                const float* __restrict__ w, int64_t n, int m, int N, int d,
                                                int accumulate, char* __restrict__ y, const int32_t* __restrict__ u_err,
                                                int32_t* __restrict__ info) {
    const int D8 = d / 8;
    if (info && blockIdx.x == 0 && threadIdx.x < 3) info[threadIdx.x] = threadIdx.x < 2 ? u_err[threadIdx.x] : MOE_OK;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * D8; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / D8;
        const int c = (int)(i - t * D8) * 8;
        float s[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] = 0.f;
        for (int j = 0; j < m; ++j) {
            const int id = ids[t * m + j];
            if (id < 0 || id >= N) continue;
            const float wj = w[t * m + j];
            const u32x4 o = *reinterpret_cast<const u32x4*>(O + ((t * m + j) * d + c) * 2);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s[2 * k] += wj * bf16_lo(o[k]);
                s[2 * k + 1] += wj * bf16_hi(o[k]);
            }
        }
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
