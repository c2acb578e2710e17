// The router of a whole-layer pass in one launch: logits, selection and weights.
//
//   l_te = W_r[e] . x_t,   s_te = exp(l_te) / sum_e exp(l_te)  or  1 / (1 + exp(-l_te))
//   selected: the m largest s_te + b_e (without b: l_te, which orders them alike), equal ones: lower id
//   w_tj = scale * s_tj / (renorm ? sum over the selected : 1)
//
// One work group of 16 waves for 16 experts x 4 tokens x one of KS parts of the contraction; its waves split
// the part, so that at d = 2048 in bf16 each has one step: one round of loads.  The parts go to memory, and the work
// group that arrives last on a token tile adds them, in order, and selects: a wave a token, m rounds of a
// wave-wide maximum; or, of many experts a token, by rank (an expert's place is the number of those before it), all
// threads together.  How the contraction is cut depends on N, d and the type alone, so a token's routing does not
// depend on the pass that it is in.
//
// Latency is the time: one token on 128 experts of d = 2048 takes 6.3-7.0 us, of which logits and arrival are 4.5 (a launch,
// a round of loads, a store, an atomic); 32 tokens 7.6-9.0, with 16 tokens a work group, where four waves a SIMD select,
// 10.2.  The two launches of moe_router_topk are 7.3 for one token.  Half or a quarter of the parts: no difference for one
// token, 0.9 and 2.2 us more for 32.  Of 1 / 5 / 32 tokens, 8 experts each: 64 experts 6.4 / 6.6 / 7.0 us, 128 7.0 / 7.4 / 7.6,
// 256 7.6 / 8.4 / 11.8, 384 14.0 / 17.2 / 23.8, 1024 15.9 / 22.2 / 42.  Beyond 256 a lane holds 16 experts, and their parts
// of 8 in flight do not fit 128 registers: 32 of them go to the stack.
#pragma once

#include "expert_kernel.h"

namespace moe_k {

constexpr int kRouteWaves = 16, kRouteThreads = 64 * kRouteWaves;
constexpr int kRouteParts = 8;  // most parts of the contraction
// Tokens of a work group: a quarter of the matrix operand's columns, so that the waves that select have a SIMD each.
constexpr int kRouteTokens = 4;
// Selection by rank, not by rounds, of the m experts of each of nt tokens, NK places for experts a token.  A round is 0.07
// (64 places) to 0.17 us (256); by rank m costs nothing, but nt NK^2 comparisons are shared by the work group.  The launch by rank /
// by rounds in us, d = 2048 in bf16:
//              nt   m = 4        8            12           16           32           64
//     N =  64   1                6.1 / 6.5    6.3 / 6.6    6.1 / 7.0    6.1 / 8.6    6.1 / 11.8
//               4                6.9 / 6.6    6.8 / 6.9    7.0 / 7.4    6.6 / 9.0    7.0 / 12.3
//     N = 128   1   6.8 / 5.9    6.8 / 6.8    6.8 / 7.5    6.9 / 8.2    6.7 / 10.3   6.7 / 15.1
//               2   7.3 / 6.2    7.5 / 7.1    7.5 / 7.7    7.5 / 8.3    7.5 / 10.6   7.3 / 15.2
//               4   8.7 / 6.6    8.9 / 7.4    9.0 / 8.0    8.8 / 8.5    8.7 / 10.8   8.9 / 15.7
//     N = 256   1                8.9 / 7.4    9.1 / 8.3    9.1 / 8.9    9.1 / 11.5   9.2 / 17.0
//               2               11.5 / 8.0   11.5 / 8.6   11.6 / 9.5   11.3 / 11.7  11.2 / 17.0
//               4               16.3 / 8.3   16.2 / 8.8   16.2 / 9.6   16.3 / 12.2  16.0 / 17.3
// With more places by rounds alone (1024, one token, m = 8 / 64: by rank 49 / 49, by rounds 16 / 34).
constexpr int kRankPlaces = 256;
__device__ __forceinline__ bool by_rank(int nt, int NK, int m) {
    return NK <= kRankPlaces && m > max(8, 4 + nt * NK * NK / 5120);
}

struct RouteArgs {
    const char* wr;     // [N][d]
    const char* x;      // [n][d]
    const float* bias;  // [N] or null
    float* part;        // [KS][n][row of N, whole fours]
    int32_t* count;     // [token tiles][kLine], zero
    int32_t* ids;       // [n][m]
    float* w;
    int32_t N, n, m, d, KS;
    int32_t sigmoid, renorm;
    float scale;
};

// The order of the values as unsigned numbers, NaN (which is never selected) below all.
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);  // -0 as 0
    return v == v ? ((int)b < 0 ? ~b : b | 0x80000000u) : 0u;
}

__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float((int)k < 0 ? k & 0x7fffffffu : ~k); }

// The wave's largest, in every lane: rows of 16 by shifts, then across the rows.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define MOE_DPP_MAX(ctrl, rows) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, ctrl, rows, 0xf, false))
    MOE_DPP_MAX(0x111, 0xf);  // row_shr:1
    MOE_DPP_MAX(0x112, 0xf);
    MOE_DPP_MAX(0x114, 0xf);
    MOE_DPP_MAX(0x118, 0xf);
    MOE_DPP_MAX(0x142, 0xa);  // row_bcast:15
    MOE_DPP_MAX(0x143, 0xc);  // row_bcast:31
#undef MOE_DPP_MAX
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float wave_sum(float v) {  // a fixed tree, the same in every lane
#define MOE_DPP_ADD(ctrl, rows) \
    v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, rows, 0xf, true))
    MOE_DPP_ADD(0x111, 0xf);
    MOE_DPP_ADD(0x112, 0xf);
    MOE_DPP_ADD(0x114, 0xf);
    MOE_DPP_ADD(0x118, 0xf);
    MOE_DPP_ADD(0x142, 0xa);
    MOE_DPP_ADD(0x143, 0xc);
#undef MOE_DPP_ADD
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// Sigmoid times exp(-c), c <= 0, the same in every lane: with c the largest of the selected logits, or 0, the
// quotients of weights stay where all sigmoids are too small for fp32.
__device__ __forceinline__ float sigmoid_from(float l, float c) {
    const float t = expf(-fabsf(l));
    float up = t;
    if (c < 0.f) up = expf(l - c);
    return (l > 0.f ? 1.f : up) * __builtin_amdgcn_rcpf(1.f + t);
}

__host__ __device__ __forceinline__ uint32_t route_row(int N) { return (uint32_t)(N + 3) & ~3u; }

template <int V>
__device__ __forceinline__ void route_load(__amdgpu_buffer_rsrc_t r, uint32_t vo, uint32_t so, uint32_t* v) {
    if constexpr (V == 1) {
        v[0] = __builtin_amdgcn_raw_buffer_load_b32(r, vo, so, kSc1);
    } else if constexpr (V == 2) {
        const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, vo, so, kSc1));
        v[0] = w.x;
        v[1] = w.y;
    } else {
        const u32x4 w = bload2<kSc1>(r, vo, so);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = w[i];
    }
}

// CL: experts a lane holds, CL lane + j
template <bool BF16, int CL>
__global__ __launch_bounds__(kRouteThreads) void k_route(RouteArgs a) {
    using F = Fmt<BF16>;
    __shared__ f32x4 red[kRouteWaves][64];
    __shared__ int sel_e[kRouteTokens][MOE_MAX_SLOTS];
    __shared__ float sel_l[kRouteTokens][MOE_MAX_SLOTS];
    __shared__ int s_last;
    constexpr int NK = 64 * CL, kPairs = NK <= kRankPlaces ? kRouteTokens * NK : 4;
    __shared__ __align__(16) uint32_t s_key[kPairs];
    __shared__ float s_l[kPairs];
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int lr = lane & 15, q = lane >> 4;
    const int e0 = blockIdx.x * kTile, t0 = blockIdx.y * kRouteTokens, ks = blockIdx.z, KS = a.KS;
    const int nt = min(kRouteTokens, a.n - t0);  // tokens of this tile
    const int S = (a.d + F::kStep - 1) / F::kStep;
    const int kb = ks * S / KS, kl = (ks + 1) * S / KS - kb;  // this part's steps
    const int s0 = kb + wave * kl / kRouteWaves, s1 = kb + (wave + 1) * kl / kRouteWaves;
    const auto rw = rsrc(a.wr, (uint32_t)a.N * a.d * F::kEsize);
    const auto rx = rsrc(a.x, (uint32_t)a.n * a.d * F::kEsize);
    const uint32_t la = e0 + lr < a.N ? (uint32_t)(e0 + lr) * a.d * F::kEsize : kOOB;
    const uint32_t lb = lr < nt ? (uint32_t)(t0 + lr) * a.d * F::kEsize : kOOB;
    f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int kAhead = 4;
    for (int s = s0; s < s1; s += kAhead) {
        u32x4 wv[kAhead], xv[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int k = (s + j) * F::kStep + q * F::kPer;
            const bool ok = s + j < s1 && k < a.d;  // (d % 8 == 0: whole chunks)
            wv[j] = bload(rw, ok ? cat(la, (uint32_t)k * F::kEsize) : kOOB);
            xv[j] = bload(rx, ok ? cat(lb, (uint32_t)k * F::kEsize) : kOOB);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) acc = F::mma(wv[j], xv[j], acc);
    }
    red[wave][lane] = acc;
    __syncthreads();
    const uint32_t NP = route_row(a.N);
    const auto rp = rsrc(a.part, (uint32_t)KS * a.n * NP * 4);
    if (wave == 0) {
        f32x4 r[kRouteWaves];  // (read together)
#pragma unroll
        for (int w = 0; w < kRouteWaves; ++w) r[w] = red[w][lane];
        __builtin_amdgcn_sched_barrier(0);
        f32x4 v = r[0];
#pragma unroll
        for (int w = 1; w < kRouteWaves; ++w) v += r[w];
        // experts e0 + 4 q .. + 3 of token t0 + lr (past N: zeros)
        const uint32_t t = t0 + lr, e = e0 + 4 * q;
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rp,
                                               e < NP && lr < nt ? ((ks * a.n + t) * NP + e) * 4u : kOOB, 0, kSc1);
        stores_complete();
        if (lane == 0) {
            int32_t* count = a.count + kLine * blockIdx.y;
            s_last = atomicAdd(count, 1) == (int)(gridDim.x * gridDim.z) - 1;
            if (s_last) __hip_atomic_store(count, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // all have arrived
        }
    }
    __syncthreads();  // the loads (sc1) below go out after the last arrival was seen
    if (!s_last) return;
    const int t = t0 + wave;  // this wave's token
    const bool live = wave < nt;
    const bool rank = by_rank(nt, NK, a.m);
    if (!rank && !live) return;  // (by rounds there is no barrier)
    int* se = sel_e[live ? wave : 0];
    float* sl = sel_l[live ? wave : 0];
    float l[CL], top = -INFINITY, Z = 1.f;  // logits; the largest; sum of exp(l - top)
    uint32_t key[CL];
    if (live) {
        constexpr int V = CL < 4 ? CL : 4, W = CL / V;  // a lane's experts as W vectors
        uint32_t pv[kRouteParts][CL], bias[CL];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint32_t e = CL * lane + V * w, vo = e < NP ? (t * NP + e) * 4u : kOOB;
#pragma unroll
            for (int k = 0; k < kRouteParts; ++k)
                route_load<V>(rp, k < KS ? vo : kOOB, k * a.n * NP * 4u, &pv[k][V * w]);
        }
        const auto rb = rsrc(a.bias, a.bias ? a.N * 4u : 0u);
#pragma unroll
        for (int j = 0; j < CL; ++j) bias[j] = __builtin_amdgcn_raw_buffer_load_b32(rb, (CL * lane + j) * 4u, 0, 0);
#pragma unroll
        for (int j = 0; j < CL; ++j) {
            l[j] = __uint_as_float(pv[0][j]);
#pragma unroll
            for (int k = 1; k < kRouteParts; ++k) l[j] += __uint_as_float(pv[k][j]);  // (parts past KS: 0)
            key[j] = CL * lane + j < a.N ? order_of(l[j]) : 0u;
            if (key[j]) top = fmaxf(top, l[j]);
        }
        if (!a.sigmoid && (a.bias || !a.renorm)) {
            top = value_of(wave_max(order_of(top)));
            float z = 0.f;
#pragma unroll
            for (int j = 0; j < CL; ++j)
                if (key[j]) z += expf(l[j] - top);
            Z = wave_sum(z);
        }
        if (a.bias) {
#pragma unroll
            for (int j = 0; j < CL; ++j)
                if (key[j]) {
                    const float s = a.sigmoid ? sigmoid_from(l[j], 0.f) : expf(l[j] - top) / Z;
                    key[j] = order_of(s + __uint_as_float(bias[j]));
                }
        }
    }
    if (rank) {
        if (live) {
#pragma unroll
            for (int j = 0; j < CL; ++j) {
                s_key[wave * NK + CL * lane + j] = key[j];
                s_l[wave * NK + CL * lane + j] = l[j];
            }
            for (int j = lane; j < a.m; j += 64) se[j] = -1;
        }
        __syncthreads();
        // G threads an expert, each a part of the others; what is no expert has key 0, behind all
        int G = 1;
        while (G < 8 && 2 * G * nt * NK <= kRouteThreads) G *= 2;
        const int g = tid & (G - 1), part = NK / G;
        for (int i = tid / G; i < nt * NK; i += kRouteThreads / G) {
            const int u = i / NK, e = i & (NK - 1);
            const uint32_t mine = s_key[i];
            const u32x4* others = reinterpret_cast<const u32x4*>(&s_key[u * NK + g * part]);
            int before = 0;
#pragma unroll 4
            for (int k = 0; k < part / 4; ++k) {
                const u32x4 v = others[k];
                const int at = g * part + 4 * k;
#pragma unroll
                for (int c = 0; c < 4; ++c) before += v[c] + (at + c < e ? 1u : 0u) > mine;  // (no key is 2^32 - 1)
            }
            for (int o = G / 2; o > 0; o >>= 1) before += __shfl_xor(before, o, 64);
            if (g == 0 && mine && before < a.m) {
                sel_e[u][before] = e;
                sel_l[u][before] = s_l[i];
            }
        }
        __syncthreads();
        if (!live) return;
    } else {
        // rounds: the wave's largest key, of equal ones the lowest lane's (and a lane's first), which is the lowest
        // expert; the lanes keep 64 rounds' results, then hand them over
        for (int r0 = 0; r0 < a.m; r0 += 64) {
            int mine_e = -1;
            float mine_l = 0.f;
            const int rounds = min(64, a.m - r0);
            for (int r = 0; r < rounds; ++r) {
                uint32_t best = key[0];
                int bj = 0;
                float bl = l[0];
#pragma unroll
                for (int j = 1; j < CL; ++j) {
                    const bool more = key[j] > best;
                    best = more ? key[j] : best;
                    bj = more ? j : bj;
                    bl = more ? l[j] : bl;
                }
                const uint32_t most = wave_max(best);
                const int at = __ffsll((unsigned long long)__ballot(best == most)) - 1;
                const int j = __builtin_amdgcn_readlane(bj, at), e = most ? CL * at + j : -1;  // (0: nothing is left)
                const float v = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(bl), at));
                mine_e = lane == r ? e : mine_e;
                mine_l = lane == r ? v : mine_l;
#pragma unroll
                for (int i = 0; i < CL; ++i) key[i] = i == j && lane == at ? 0u : key[i];
            }
            if (lane < rounds) {
                se[r0 + lane] = mine_e;
                sl[r0 + lane] = mine_l;
            }
        }
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // weights: s_j over the sum of the selected, or over Z (with a bias the first selected need not be the largest)
    float c = -INFINITY;
    for (int j = lane; j < a.m; j += 64)
        if (se[j] >= 0) c = fmaxf(c, sl[j]);
    c = value_of(wave_max(order_of(c)));
    if (a.sigmoid) c = a.renorm ? fminf(c, 0.f) : 0.f;
    else if (!a.renorm) c = top;
    float z = 0.f;
    for (int j = lane; j < a.m; j += 64) {
        const float v = se[j] < 0 ? 0.f : a.sigmoid ? sigmoid_from(sl[j], c) : expf(sl[j] - c);
        sl[j] = v;  // (a lane's own places)
        z += v;
    }
    if (a.renorm) Z = wave_sum(z);
    const float f = a.scale / Z;
    for (int j = lane; j < a.m; j += 64) {
        a.ids[(size_t)t * a.m + j] = se[j];
        a.w[(size_t)t * a.m + j] = se[j] < 0 ? 0.f : sl[j] * f;
    }
}

}  // namespace moe_k
