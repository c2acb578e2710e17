// Passes of up to 64 slots in 8-bit integers, in two launches: one decoded token, a short verification pass.
//
// The grouped pass takes five launches (grouping and x, gate/up, h, down, the tokens' sums), each with a
// latency of 2.5 us and more: one token on 8 of 128 experts of 2048 x 768 takes 24 us, of which the 38 MB of its
// codes are 8.  Here every work group groups the slots itself (a lane a slot, ten ballots) and quantises the rows
// that it needs, while its first weights are on their way; the tokens' sums are formed where the down products are:
// 14.7 us, 8.1-8.8 and 6.0-6.4, of which 5 are two launches.  The arithmetic is that of the grouped calls, bit for bit: sums of
// codes are whole numbers, so a contraction may be cut anywhere, and the rest is done in the same order.
#pragma once

#include "grouped_kernel.h"

namespace moe_g {

constexpr int kSmallSlots = 64;             // a lane a slot
constexpr int kSmallLds = 54 * 1024;        // bytes of codes in shared memory, at most (with the kernels' own 64 KB)
constexpr int kSmallDownThreads = 1024;

struct Small {
    const char* x;        // [n][d] bf16
    const int32_t* ids;   // [S]
    const float* rw;      // [S]
    const char *w0, *w1, *wd;
    const float *s0, *s1, *sd;
    char* h;              // [S][f] bf16, by slot
    char* y;              // [n][d] bf16
    int32_t* info;        // null, or U, ids status, MOE_OK
    int N, n, m, S, d, f;
    int accumulate;
};

// The slots of a pass, a lane each: the lanes of the same expert, and the row tiles of 16 slots, those of an
// expert at its first slot.
struct Slots {
    int id;          // this lane's, -1 where it is not valid
    uint64_t same;   // lanes with this id
    int tiles, at;   // tiles of the expert whose first slot this is (else 0), and those before
    int total;

    __device__ __forceinline__ Slots(const int32_t* __restrict__ ids, int S, int N) {
        const int lane = threadIdx.x & 63;
        const uint64_t below = (1ull << lane) - 1;
        const int v = lane < S ? ids[lane] : -1;
        const bool ok = v >= 0 && v < N;
        id = ok ? v : -1;
        same = __ballot(ok);
        for (int b = 0; (1 << b) < N; ++b) {
            const uint64_t set = __ballot((id >> b) & 1);
            same &= ((id >> b) & 1) ? set : ~set;
        }
        if (!ok) same = 0;
        const bool first = ok && !(same & below);
        tiles = first ? (__popcll(same) + kTile16 - 1) / kTile16 : 0;
        at = total = 0;
#pragma unroll
        for (int i = 1; i <= kSmallSlots / kTile16; ++i) {  // sums over the lanes, by those with i tiles or more
            const uint64_t have = __ballot(tiles >= i);
            at += __popcll(have & below);
            total += __popcll(have);
        }
    }

    struct Tile {
        int e, rows, slot;  // expert (-1: past the last), slots, and the slot of row lane % 16 (rows past the last: the last's)
    };
    __device__ __forceinline__ Tile tile(int t) const {
        const uint64_t who = __ballot(tiles > 0 && t >= at && t < at + tiles);
        if (!who) return Tile{-1, 0, 0};
        const int l = __ffsll((unsigned long long)who) - 1;
        uint64_t in = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(same >> 32), l) << 32) |
                      (uint32_t)__builtin_amdgcn_readlane((int)same, l);
        const int skip = (t - __builtin_amdgcn_readlane(at, l)) * kTile16;
        for (int i = 0; i < skip; ++i) in &= in - 1;
        const int rows = min(__popcll(in), kTile16), lr = threadIdx.x & 15;
        int slot = 0;
        for (int r = 0; r < rows; ++r, in &= in - 1)
            if (lr >= r) slot = __ffsll((unsigned long long)in) - 1;
        return Tile{__builtin_amdgcn_readlane(id, l), uni(rows), slot};
    }
};

// Codes of 16 bf16 values and more to shared memory: rows of K, `lanes` lanes a row (a power of two up to 64),
// row r read at from(r), its codes at lds + r * stride.  A row's values are held if they are at most 8 a lane and
// vector, four vectors; else they are read again.
template <typename From>
__device__ __forceinline__ void rows_to_lds(int rows, int K, int lanes, char* lds, int stride, float* scale, From from) {
    const int l = threadIdx.x & (lanes - 1), span = lanes * 8, V = (K + span - 1) / span;
    for (int r = threadIdx.x / lanes; r < rows; r += blockDim.x / lanes) {
        const char* x = from(r);
        u32x4 a[kRowVecs];
        uint32_t m = 0;
        auto load = [&](int v0) {
#pragma unroll
            for (int i = 0; i < kRowVecs; ++i) {
                const int c = (v0 + i) * span + l * 8;
                a[i] = c < K ? *reinterpret_cast<const u32x4*>(x + (int64_t)c * 2) : u32x4{0u, 0u, 0u, 0u};
            }
        };
        for (int v0 = 0; v0 < V; v0 += kRowVecs) {
            load(v0);
#pragma unroll
            for (int i = 0; i < kRowVecs; ++i) m = max(m, largest(a[i]));
        }
        for (int o = lanes / 2; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
        const RowScale s = row_scale(m);
        if (l == 0) scale[r] = scale_of(m);
        for (int v0 = 0; v0 < V; v0 += kRowVecs) {
            if (V > kRowVecs) load(v0);
#pragma unroll
            for (int i = 0; i < kRowVecs; ++i) {
                const int c = (v0 + i) * span + l * 8;
                if (c < K) *reinterpret_cast<u32x2*>(lds + r * stride + c) = codes8_i8(a[i], s);
            }
        }
    }
}

// Where the units of a matrix operand's 16 rows are: a lane's two chunks of unit u.
template <bool TILED>
struct Weight16 {
    const char* p;
    int K, q;
    __device__ __forceinline__ Weight16(const char* w, int e, int cb, int R, int K_) : K(K_) {
        const int lane = threadIdx.x & 63;
        q = lane >> 4;
        p = w + (int64_t)e * R * K + (TILED ? (int64_t)cb * 16 * K + lane * 16 : (int64_t)(cb * 16 + (lane & 15)) * K);
    }
    __device__ __forceinline__ void load(int u, bool ok, u32x4 (&w)[2]) const {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const int k = u * kUnit + kk * 64 + q * 16;
            w[kk] = ok && k < K ? *reinterpret_cast<const u32x4*>(p + (TILED ? (int64_t)(2 * u + kk) * 1024 : (int64_t)k))
                                : u32x4{0u, 0u, 0u, 0u};
        }
    }
};

// A row's codes of unit u; behind K zeros that are never read (the weights' chunk there is zero).
__device__ __forceinline__ void lds_unit(const char* row, int u, int q, int K, u32x4 (&b)[2]) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
        const int k = min(u * kUnit + kk * 64 + q * 16, K - 16);
        b[kk] = *reinterpret_cast<const u32x4*>(row + k);
    }
}

// Gate and up: a work group 16 columns of both matrices for one row tile, four waves sharing the contraction.
template <bool TILED>
__global__ __launch_bounds__(256) void k_small_gate_up(Small a) {
    extern __shared__ __align__(16) char codes[];  // [rows][d + 16]
    __shared__ i32x4 red[4][2][64];
    __shared__ float sx[kTile16];
    __shared__ int tok[kTile16];
    constexpr int AHEAD = 4;
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), lr = lane & 15, q = lane >> 4;
    const int CB = a.f / 16, t = blockIdx.x / CB, cb = blockIdx.x - t * CB;
    const Slots slots(a.ids, a.S, a.N);
    if (a.info && blockIdx.x == 0 && wave == 0) {
        const int first = lane / a.m * a.m;  // this token's slots before this one
        const uint64_t before = ((1ull << lane) - 1) & ~((1ull << (first & 63)) - 1);
        const uint64_t bad = __ballot(lane < a.S && (slots.id < 0 || (slots.same & before)));
        const uint64_t U = __ballot(slots.tiles > 0);
        if (lane == 0) {
            a.info[0] = __popcll(U);
            a.info[1] = bad ? MOE_E_IDS : MOE_OK;
            a.info[2] = MOE_OK;
        }
    }
    const auto tile = slots.tile(t);
    if (tile.e < 0) return;
    const int K = a.d, U = (K + kUnit - 1) / kUnit, stride = K + 16;
    const Weight16<TILED> wp[2] = {{a.w0, tile.e, cb, a.f, K}, {a.w1, tile.e, cb, a.f, K}};
    u32x4 w[AHEAD][2][2];
    auto load = [&](int u0) {
#pragma unroll
        for (int p = 0; p < AHEAD; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) wp[i].load(u0 + p * 4, u0 + p * 4 < U, w[p][i]);
    };
    load(wave);
    if (wave == 0 && lane < kTile16) tok[lane] = tile.slot / a.m;
    __syncthreads();
    rows_to_lds(tile.rows, K, 64, codes, stride, sx, [&](int r) { return a.x + (int64_t)uni(tok[r]) * K * 2; });
    __syncthreads();
    const char* row = codes + min(lr, tile.rows - 1) * stride;
    i32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    for (int u0 = wave; u0 < U; u0 += 4 * AHEAD) {
        if (u0 != wave) load(u0);
#pragma unroll
        for (int p = 0; p < AHEAD; ++p) {
            u32x4 b[2];
            lds_unit(row, u0 + p * 4, q, K, b);
#pragma unroll
            for (int i = 0; i < 2; ++i) acc[i] = mma_unit<kInt8>(w[p][i][0], w[p][i][1], b[0], b[1], acc[i], 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) red[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave || lr >= tile.rows) return;
    const int c = cb * 16 + 4 * q;
    f32x4 v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const i32x4 sum = red[0][i][lane] + red[1][i][lane] + red[2][i][lane] + red[3][i][lane];
        const float* sw = (i ? a.s1 : a.s0) + (int64_t)tile.e * a.f + c;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i][k] = (float)sum[k] * sw[k] * sx[lr];
    }
    float h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = silu(v[0][k]) * v[1][k];
    *reinterpret_cast<u32x2*>(a.h + ((int64_t)tile.slot * a.f + c) * 2) = u32x2{bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3])};
}

// Down: a work group of 16 waves takes 16 columns of all tiles, each cut into P parts of the contraction so that every
// wave has one; the parts meet in shared memory as whole numbers, whose sum no order changes.
template <bool TILED>
__global__ __launch_bounds__(kSmallDownThreads) void k_small_down(Small a) {
    extern __shared__ __align__(16) char codes[];  // [S][f + 16]
    __shared__ int sum[kSmallSlots][17];
    __shared__ float sh[kSmallSlots];
    constexpr int AHEAD = 3, W = kSmallDownThreads / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), lr = lane & 15, q = lane >> 4;
    const int cb = blockIdx.x, S = a.S, K = a.f, U = (K + kUnit - 1) / kUnit, stride = K + 16;
    const Slots slots(a.ids, S, a.N);
    const int T = slots.total, P = T > 0 ? min(max(W / T, 1), U) : 1, items = T * P;
    u32x4 w[AHEAD][2];
    int u = 0, end = 0;
    auto part_of = [&](int i) { return i - i / P * P; };
    auto begin = [&](int i) {
        u = part_of(i) * U / P;
        end = (part_of(i) + 1) * U / P;
    };
    auto load = [&](const Weight16<TILED>& wp) {
#pragma unroll
        for (int p = 0; p < AHEAD; ++p) wp.load(u + p, u + p < end, w[p]);
    };
    int item = wave;
    auto tile = slots.tile(item / P);
    if (item < items) {
        begin(item);
        load(Weight16<TILED>(a.wd, tile.e, cb, a.d, K));
    }
    // thread: slot tid / 16, column tid % 16
    const int s = tid >> 4, c = tid & 15;
    float sd = 0.f, rw = 0.f;
    bool live = false;
    if (s < S) {
        const int id = a.ids[s];
        live = id >= 0 && id < a.N;
        if (live) {
            sd = a.sd[(int64_t)id * a.d + cb * 16 + c];
            rw = a.rw[s];
        }
        sum[s][c] = 0;
    }
    int lanes = 64;
    while (lanes > 16 && S * lanes > kSmallDownThreads) lanes >>= 1;
    rows_to_lds(S, K, lanes, codes, stride, sh, [&](int r) { return a.h + (int64_t)r * K * 2; });
    __syncthreads();
    while (item < items) {
        const Weight16<TILED> wp(a.wd, tile.e, cb, a.d, K);
        const char* row = codes + tile.slot * stride;
        i32x4 acc = {0, 0, 0, 0};
        while (true) {
#pragma unroll
            for (int p = 0; p < AHEAD; ++p) {
                u32x4 b[2];
                lds_unit(row, u + p, q, K, b);
                acc = mma_unit<kInt8>(w[p][0], w[p][1], b[0], b[1], acc, 0, 0);
            }
            u += AHEAD;
            if (u >= end) break;
            load(wp);
        }
        if (lr < tile.rows) {
#pragma unroll
            for (int k = 0; k < 4; ++k) atomicAdd(&sum[tile.slot][4 * q + k], acc[k]);
        }
        item += W;
        if (item >= items) break;
        tile = slots.tile(item / P);
        begin(item);
        load(Weight16<TILED>(a.wd, tile.e, cb, a.d, K));
    }
    __syncthreads();
    // a slot's term w O, in fp32; in place of the sums
    float term = 0.f;
    if (live) term = (float)sum[s][c] * sd * sh[s];
    float* O = reinterpret_cast<float*>(&sum[0][0]);
    if (s < S) O[s * 17 + c] = term;
    float* wt = sh;  // the slots' weights, 0 for what is not valid, in place of the scales
    __syncthreads();
    if (s < S && c == 0) wt[s] = rw;
    __syncthreads();
    if (tid < a.n * 16) {  // thread: token s, column c
        float v = 0.f;
        for (int j = 0; j < a.m; ++j) v += wt[s * a.m + j] * O[(s * a.m + j) * 17 + c];
        uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + (int64_t)s * a.d + cb * 16 + c;
        if (a.accumulate) v += bf16_lo(*y);
        *y = (uint16_t)bf16_pair(v, v);
    }
}

}  // namespace moe_g
