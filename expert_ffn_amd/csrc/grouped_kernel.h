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
        *reinterpret_cast<f32x4*>(a.out + ((int64_t)slot * a.R + c) * 4) = v[0];
    }
}

// y_t = sum_j w_tj O_tj over the slots with a valid id, in increasing j, rounded to bf16
// once; four columns a thread.  info (may be null): U, ids status, MOE_OK.
__global__ __launch_bounds__(256) void k_combine(const float* __restrict__ O, const int32_t* __restrict__ ids,
                                                const float* __restrict__ w, int64_t n, int m, int N, int d,
                                                int accumulate, char* __restrict__ y, const int32_t* __restrict__ u_err,
                                                int32_t* __restrict__ info) {
    const int D4 = d / 4;
    if (info && blockIdx.x == 0 && threadIdx.x < 3) info[threadIdx.x] = threadIdx.x < 2 ? u_err[threadIdx.x] : MOE_OK;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * D4; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / D4;
        const int c = (int)(i - t * D4) * 4;
        f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < m; ++j) {
            const int id = ids[t * m + j];
            if (id < 0 || id >= N) continue;
            const float wj = w[t * m + j];
            const f32x4 o = *reinterpret_cast<const f32x4*>(O + (t * m + j) * d + c);
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] += wj * o[k];
        }
        u32x2* p = reinterpret_cast<u32x2*>(y + (t * d + c) * 2);
        if (accumulate) {
            const u32x2 v = *p;
            s += f32x4{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
        }
        *p = u32x2{bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3])};
    }
}

}  // namespace moe_g
