// C ABI of the expert operation on grouped rows (include/moe_expert.h): argument checks,
// workspaces and launches of the kernels in grouped_kernel.h.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>

#include "grouped_kernel.h"
#include "moe_expert.h"

namespace {

using namespace moe_g;

constexpr size_t kAlign = 256;
constexpr int kCUs = 256;  // a work group of square tiles each
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
hipStream_t stream_of(void* s) { return reinterpret_cast<hipStream_t>(s); }
int launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_E_HIP; }
int64_t blocks_of(int64_t v) { return (v + kBlk - 1) / kBlk; }

int check_slots(int32_t n, int32_t m, int32_t N) {
    if (N < 1 || N > MOE_MAX_EXPERTS || m < 1 || m > N || m > MOE_MAX_SLOTS || n < 1 ||
        (int64_t)n * m > MOE_MAX_GROUP_SLOTS)
        return MOE_E_INVAL;
    return MOE_OK;
}

// The descriptor of a grouped product of `dtype` weights.
int check_desc(const moe_layer_desc* d, int32_t n, int32_t dtype) {
    if (!d) return MOE_E_INVAL;
    if (d->dtype != dtype) return MOE_E_DTYPE;
    const int per = dtype == MOE_FP8 ? 16 : 8;  // whole 16-byte pieces of a row
    if (d->d_model < per || d->d_ff < per || d->d_model % per || d->d_ff % per) return MOE_E_DTYPE;
    const int rc = check_slots(n, d->m, d->N);
    if (rc != MOE_OK) return rc;
    if (d->flags & ~(MOE_FLAG_ACCUMULATE | MOE_FLAG_TILED)) return MOE_E_INVAL;
    if (d->n_shared != 0) return MOE_E_INVAL;
    const int64_t es = dtype == MOE_FP8 ? 1 : 2;
    if ((d->flags & MOE_FLAG_TILED) && (d->d_model % (64 / es) || d->d_ff % (64 / es))) return MOE_E_INVAL;
    if (d->d_model > MOE_MAX_GROUP_WIDTH || d->d_ff > MOE_MAX_GROUP_WIDTH) return MOE_E_INVAL;
    return MOE_OK;
}

// Grouping workspace: [chunks][N + 1] counts
int group_chunks(int64_t S) { return (int)((S + group_chunk(S) - 1) / group_chunk(S)); }
size_t group_ws(int chunks, int N) { return align_up((size_t)chunks * (N + 1) * 4); }

int rows_grid(int64_t rows, int K) {  // sixteen blocks of 128 a work group
    return (int)std::min<int64_t>((rows * blocks_of(K) + 15) / 16, 16384);
}

void run_group(Group g, hipStream_t st) {
    g.G = group_chunks(g.S);
    // work groups of 1024 threads for the rows to quantise: 64 blocks of 128 at a time
    const int quant = g.x ? (int)std::min<int64_t>((g.n * blocks_of(g.d) + 63) / 64, 1024) : 0;
    if (g.G > 1) hipLaunchKernelGGL(k_group_hist, dim3(g.G + quant), dim3(kGThreads), 0, st, g);
    hipLaunchKernelGGL(k_group_scatter, dim3(g.G > 1 ? g.G : 1 + quant), dim3(kGThreads), 0, st, g);
}

// Square or thin tiles.  Thin ones take as long again with every 16 rows of an expert, square ones the
// same from few rows on.  At 8 / 16 / 24 rows of every expert, thin against square, us:
//     128 experts of 2048 x 768   gate/up bf16   138 / 148 / 202   135 / 134 / 135
//                                 gate/up e4m3    76 /  89 / 118    83 /  83 /  83
//                                 down bf16       83 /  96 / 129    88 /  93 /  98
//                                 down e4m3       48 /  56 /  77    60 /  62 /  66
//     8 experts of 4096 x 14336   down bf16      169 / 198 / 297   261 / 236 / 239
// (the last with fewer square tiles than compute units).  Routing is never that even, and an expert of
// 17 rows already takes two thin tiles: passes of the first layer at a mean of 7 / 9 / 11 / 13 rows, ids uniform,
// bf16 230 / 229 / 235 / 248 against 227 / 228 / 229 / 230, e4m3 129 / 134 / 139 / 148 against 144 / 146 / 147 / 148;
// with popularity falling as 1 / rank^1.1, bf16 147 / 173 / 191 / 213 against 146 / 160 / 159 / 165, e4m3
// 93 / 107 / 118 / 130 against 100 / 113 / 112 / 117.
// The mean counts padding, as only the device knows the groups.  4096 tokens of 8 slots of which 32 tokens are
// live, thin against square, whole passes of the first layer: bf16 296 / 214, e4m3 232 / 151 (a thin tile's work
// groups are launched for every row there could be).  900 of 1000 rows on one of the 128 experts: 179 / 166 and 103 / 107.
// Square tiles' loads run up to two units ahead into the next tile, which takes four
// units a tile, and have buffer offsets of 31 bits (x, or a matrix and the rows that its last
// tile has beyond it); thin tiles address all of memory.
bool square(const Args& a, bool fp8, bool gu) {
    const int64_t kby = (int64_t)a.K * (fp8 ? 1 : 2), most = (1ll << 31) - 4096;
    const int64_t tc = gu ? kTN / 2 : kTN, tiles = std::min(a.N, a.S) * ((a.R + tc - 1) / tc);
    return kby > 3 * kUnit && a.S >= (tiles >= 2 * kCUs ? (fp8 ? 12 : 8) : 16) * (int64_t)a.N && (a.R + kTN) * kby <= most &&
           (gu ? (int64_t)(a.S / a.m) * kby : kTM * kby) <= most;
}

Args shape_of(int N, int m, int n, int R, int K) {
    Args a{};
    a.N = N;
    a.m = m;
    a.S = n * m;
    a.R = R;
    a.K = K;
    return a;
}
bool square_gate_up(const moe_layer_desc* d, int n) {
    return square(shape_of(d->N, d->m, n, d->d_ff, d->d_model), d->dtype == MOE_FP8, true);
}
bool square_down(const moe_layer_desc* d, int n) {
    return square(shape_of(d->N, d->m, n, d->d_model, d->d_ff), d->dtype == MOE_FP8, false);
}

// Workspace of a whole pass, and of the products alone (which use the queue, row_of, hf, O and its bytes).
struct Space {
    size_t queue, hist, count, offset, sbe, row_of, distinct, u_err, xq, xs, h, hs, hf, o, os, total;
};

Space space_of(const moe_layer_desc* d, int32_t n) {
    const size_t S = (size_t)n * d->m;
    const bool fp8 = d->dtype == MOE_FP8;
    Space p;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t a = at;
        at += align_up(bytes);
        return a;
    };
    p.queue = take(2 * kQueue * 4);  // gate/up's, then down's
    // O: fp32 from thin tiles (of shapes that square tiles take, only below 16 rows an expert), fp16 from square ones
    size_t o = S * d->d_model * 4;
    if (square_down(d, n)) o = std::max(o / 2, (size_t)16 * d->N * d->d_model * 4);
    // gate/up's fp32 h (quantised before down begins), then O
    p.hf = p.o = take(std::max(o, fp8 ? S * d->d_ff * 4 : 0));
    p.os = take(S * ((d->d_model + 63) / 64));
    p.h = take(S * d->d_ff * (fp8 ? 1 : 2));
    p.hs = take(fp8 ? S * blocks_of(d->d_ff) : 0);
    p.xq = take(fp8 ? (size_t)n * d->d_model : 0);
    p.xs = take(fp8 ? (size_t)n * blocks_of(d->d_model) : 0);
    p.hist = take(group_ws(kGMaxChunks, d->N));  // (a longer pass may have fewer chunks)
    p.count = take((size_t)d->N * 4);
    p.offset = take((size_t)(d->N + 1) * 4);
    p.sbe = take(S * 4);
    p.row_of = take(S * 4);
    p.distinct = take((size_t)d->N * 4);
    p.u_err = take(8);
    p.total = at;
    return p;
}

// What a pass's grouping leaves for the products, where they run by themselves: an empty queue for
// square tiles, and the rows of the slots, which thin down tiles write themselves.
void before_gate_up(const moe_layer_desc* d, int n, int32_t* queue, hipStream_t st) {
    if (square_gate_up(d, n)) hipLaunchKernelGGL(k_zero_queue, dim3(1), dim3(kQueue), 0, st, queue);
}
void before_down(const moe_layer_desc* d, int n, const int32_t* sbe, const int32_t* offset, int32_t* row_of,
                 int32_t* queue, hipStream_t st) {
    static_assert(kQueue == 256, "");
    const int S = n * d->m;
    if (square_down(d, n))
        hipLaunchKernelGGL(k_row_of, dim3((S + 255) / 256), dim3(256), 0, st, sbe, offset + d->N, S, row_of, queue);
}

template <bool FP8, bool GU>
void launch_product(const Args& a, bool tiled, hipStream_t st) {
    if (square(a, FP8, GU)) {
        const int64_t tiles = (int64_t)a.S / kTM + std::min(a.N, a.S), tc = GU ? kTN / 2 : kTN;
        const int grid = (int)std::min<int64_t>(kCUs, (tiles * ((a.R + tc - 1) / tc) + 7) / 8 * 8);
        if (tiled)
            hipLaunchKernelGGL((k_tile<FP8, true, GU>), dim3(grid), dim3(kTileThreads), 0, st, a);
        else
            hipLaunchKernelGGL((k_tile<FP8, false, GU>), dim3(grid), dim3(kTileThreads), 0, st, a);
        return;
    }
    // A launch holds 2^32 threads at most: as many row tiles at once as keep below that.
    const int64_t cols = (a.R + 15) / 16, units = ((int64_t)a.K * (FP8 ? 1 : 2) + kUnit - 1) / kUnit;
    const int64_t tiles = (int64_t)a.S / kTile16 + std::min(a.N, a.S);  // most there can be
    auto launch = [&](auto split) {
        constexpr bool SPLIT = decltype(split)::value;
        const int64_t wide = SPLIT ? cols : (cols + kThinWaves - 1) / kThinWaves, most = (1 << 23) / wide;
        Args b = a;
        for (int64_t t = 0; t < tiles; t += most) {
            b.tile0 = (int)t;
            const int grid = (int)(std::min(most, tiles - t) * wide);
            if (tiled)
                hipLaunchKernelGGL((k_thin<FP8, true, GU, SPLIT>), dim3(grid), dim3(64 * kThinWaves), 0, st, b);
            else
                hipLaunchKernelGGL((k_thin<FP8, false, GU, SPLIT>), dim3(grid), dim3(64 * kThinWaves), 0, st, b);
        }
    };
    if constexpr (!GU) {
        if (units <= kThinWhole && tiles * cols >= 16 * kCUs)  // (one token's 1024 tiles: 1.5 us better split)
            return launch(std::false_type());
    }
    launch(std::true_type());
}

struct Weights {
    const void *w0, *w1;
    const uint8_t *s0, *s1;
};

template <bool FP8>
void run_gate_up(const moe_layer_desc* d, const Weights& w, const void* x, const uint8_t* xs, int32_t n,
                 const int32_t* offset, const int32_t* sbe, void* h, uint8_t* hs, void* hf, int32_t* queue,
                 hipStream_t st) {
    Args a = shape_of(d->N, d->m, n, d->d_ff, d->d_model);
    a.x = reinterpret_cast<const char*>(x);
    a.xs = xs;
    a.w0 = reinterpret_cast<const char*>(w.w0);
    a.w1 = reinterpret_cast<const char*>(w.w1);
    a.s0 = w.s0;
    a.s1 = w.s1;
    a.offset = offset;
    a.slot = sbe;
    a.out = reinterpret_cast<char*>(h);
    a.outs = hs;
    a.queue = queue;
    const bool by16 = FP8 && !square_gate_up(d, n);  // thin tiles leave h in fp32
    if (by16) a.out = reinterpret_cast<char*>(hf);
    launch_product<FP8, true>(a, d->flags & MOE_FLAG_TILED, st);
    if (by16)
        hipLaunchKernelGGL(k_quant_rows<true>, dim3(rows_grid(a.S, a.R)), dim3(256), 0, st,
                           reinterpret_cast<const char*>(hf), (int64_t)a.S, a.R, offset + d->N,
                           reinterpret_cast<uint8_t*>(h), hs);
}

template <bool FP8>
void run_down(const moe_layer_desc* d, const Weights& w, const void* h, const uint8_t* hs, const int32_t* ids,
              const float* rw, int32_t n, const int32_t* offset, const int32_t* sbe, int32_t* row_of, void* y,
              void* o, uint8_t* os, int32_t* queue, const int32_t* u_err, int32_t* info, hipStream_t st) {
    Args a = shape_of(d->N, d->m, n, d->d_model, d->d_ff);
    a.x = reinterpret_cast<const char*>(h);
    a.xs = hs;
    a.w0 = reinterpret_cast<const char*>(w.w0);
    a.s0 = w.s0;
    a.offset = offset;
    a.slot = sbe;
    a.out = reinterpret_cast<char*>(o);
    a.outs = os;
    a.queue = queue;
    if (!u_err) a.row_of = row_of;  // (a pass's grouping has left them)
    launch_product<FP8, false>(a, d->flags & MOE_FLAG_TILED, st);
    const int64_t work = (int64_t)n * ((d->d_model + 511) / 512);  // waves
    hipLaunchKernelGGL(square_down(d, n) ? k_combine<false> : k_combine<true>,
                       dim3((int)std::min<int64_t>((work + 3) / 4, 1 << 20)), dim3(256), 0, st,
                       reinterpret_cast<const char*>(o), os, row_of, ids, rw, (int64_t)n, d->m, d->N, d->d_model,
                       (d->flags & MOE_FLAG_ACCUMULATE) ? 1 : 0, reinterpret_cast<char*>(y), u_err, info);
}

template <bool FP8>
int run_pass(const moe_layer_desc* d, const Weights& gu, const Weights& dn, const void* x, const int32_t* ids,
             const float* w, int32_t n, void* y, int32_t* info, void* ws, hipStream_t st) {
    const Space p = space_of(d, n);
    char* b = reinterpret_cast<char*>(ws);
    auto i32 = [&](size_t at) { return reinterpret_cast<int32_t*>(b + at); };
    auto u8 = [&](size_t at) { return reinterpret_cast<uint8_t*>(b + at); };
    (void)hipGetLastError();
    Group g{};
    g.ids = ids;
    g.S = (int64_t)n * d->m;
    g.m = d->m;
    g.N = d->N;
    g.hist = i32(p.hist);
    g.count = i32(p.count);
    g.offset = i32(p.offset);
    g.sbe = i32(p.sbe);
    g.distinct = i32(p.distinct);
    g.u_err = i32(p.u_err);
    g.row_of = i32(p.row_of);
    g.queues = i32(p.queue);
    g.nq = 2 * kQueue;
    if (FP8) {
        g.x = reinterpret_cast<const char*>(x);
        g.xq = u8(p.xq);
        g.xs = u8(p.xs);
        g.n = n;
        g.d = d->d_model;
    }
    run_group(g, st);
    run_gate_up<FP8>(d, gu, FP8 ? static_cast<const void*>(b + p.xq) : x, u8(p.xs), n, i32(p.offset), i32(p.sbe),
                     b + p.h, u8(p.hs), b + p.hf, i32(p.queue), st);
    run_down<FP8>(d, dn, b + p.h, u8(p.hs), ids, w, n, i32(p.offset), i32(p.sbe), i32(p.row_of), y, b + p.o,
                  u8(p.os), i32(p.queue) + kQueue, i32(p.u_err), info, st);
    return launched();
}

int check_ws(const void* ws, size_t have, size_t need) {
    if (!ws || !aligned(ws, kAlign)) return MOE_E_INVAL;
    return have < need ? MOE_E_WORKSPACE : MOE_OK;
}

bool fp8_ok(const void* w, const uint8_t* s) { return w && aligned(w, 16) && s; }

}  // namespace

extern "C" {

size_t moe_group_workspace_bytes(int32_t n, int32_t m, int32_t N) {
    if (check_slots(n, m, N) != MOE_OK) return 0;
    return group_ws(kGMaxChunks, N);
}

int moe_group_slots(const int32_t* ids, int32_t n, int32_t m, int32_t N, int32_t* count, int32_t* offset,
                    int32_t* slot_by_expert, int32_t* distinct, int32_t* u_and_err, void* ws, size_t ws_bytes,
                    void* hip_stream) {
    if (!ids || !count || !offset || !slot_by_expert || !distinct || !u_and_err) return MOE_E_INVAL;
    int rc = check_slots(n, m, N);
    if (rc != MOE_OK) return rc;
    rc = check_ws(ws, ws_bytes, group_ws(group_chunks((int64_t)n * m), N));
    if (rc != MOE_OK) return rc;
    (void)hipGetLastError();
    Group g{};
    g.ids = ids;
    g.S = (int64_t)n * m;
    g.m = m;
    g.N = N;
    g.hist = reinterpret_cast<int32_t*>(ws);
    g.count = count;
    g.offset = offset;
    g.sbe = slot_by_expert;
    g.distinct = distinct;
    g.u_err = u_and_err;
    run_group(g, stream_of(hip_stream));
    return launched();
}

size_t moe_grouped_workspace_bytes(const moe_layer_desc* desc, int32_t n) {
    if (!desc || (desc->dtype != MOE_BF16 && desc->dtype != MOE_FP8)) return 0;
    if (check_desc(desc, n, desc->dtype) != MOE_OK) return 0;
    return space_of(desc, n).total;
}

int moe_grouped_square(const moe_layer_desc* desc, int32_t n, int32_t mat) {
    if (!desc || (mat != MOE_MAT_GATE_UP && mat != MOE_MAT_DOWN)) return MOE_E_INVAL;
    if (desc->dtype != MOE_BF16 && desc->dtype != MOE_FP8) return MOE_E_DTYPE;
    const int rc = check_desc(desc, n, desc->dtype);
    if (rc != MOE_OK) return rc;
    return mat == MOE_MAT_GATE_UP ? square_gate_up(desc, n) : square_down(desc, n);
}

int moe_grouped_gate_up(const moe_layer_desc* desc, const moe_layer_weights* weights, const void* x, int32_t n,
                        const int32_t* offset, const int32_t* slot_by_expert, void* h, void* ws, size_t ws_bytes,
                        void* hip_stream) {
    int rc = check_desc(desc, n, MOE_BF16);
    if (rc != MOE_OK) return rc;
    if (!weights || !weights->w_gate || !weights->w_up || !x || !offset || !slot_by_expert || !h) return MOE_E_INVAL;
    if (!aligned(weights->w_gate, 16) || !aligned(weights->w_up, 16) || !aligned(x, 16) || !aligned(h, 16))
        return MOE_E_INVAL;
    const Space p = space_of(desc, n);
    rc = check_ws(ws, ws_bytes, p.total);
    if (rc != MOE_OK) return rc;
    int32_t* queue = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(ws) + p.queue);
    (void)hipGetLastError();
    before_gate_up(desc, n, queue, stream_of(hip_stream));
    run_gate_up<false>(desc, Weights{weights->w_gate, weights->w_up, nullptr, nullptr}, x, nullptr, n, offset,
                       slot_by_expert, h, nullptr, nullptr, queue, stream_of(hip_stream));
    return launched();
}

int moe_grouped_gate_up_fp8(const moe_layer_desc* desc, const moe_fp8_weights* weights, const void* xq,
                            const uint8_t* x_scale, int32_t n, const int32_t* offset, const int32_t* slot_by_expert,
                            void* hq, uint8_t* h_scale, void* ws, size_t ws_bytes, void* hip_stream) {
    int rc = check_desc(desc, n, MOE_FP8);
    if (rc != MOE_OK) return rc;
    if (!weights || !fp8_ok(weights->w_gate, weights->s_gate) || !fp8_ok(weights->w_up, weights->s_up) ||
        !fp8_ok(xq, x_scale) || !fp8_ok(hq, h_scale) || !offset || !slot_by_expert)
        return MOE_E_INVAL;
    const Space p = space_of(desc, n);
    rc = check_ws(ws, ws_bytes, p.total);
    if (rc != MOE_OK) return rc;
    int32_t* queue = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(ws) + p.queue);
    (void)hipGetLastError();
    before_gate_up(desc, n, queue, stream_of(hip_stream));
    run_gate_up<true>(desc, Weights{weights->w_gate, weights->w_up, weights->s_gate, weights->s_up}, xq, x_scale, n,
                      offset, slot_by_expert, hq, h_scale, reinterpret_cast<char*>(ws) + p.hf, queue,
                      stream_of(hip_stream));
    return launched();
}

int moe_grouped_down(const moe_layer_desc* desc, const moe_layer_weights* weights, const void* h, const int32_t* ids,
                     const float* w, int32_t n, const int32_t* offset, const int32_t* slot_by_expert, void* y, void* ws,
                     size_t ws_bytes, void* hip_stream) {
    int rc = check_desc(desc, n, MOE_BF16);
    if (rc != MOE_OK) return rc;
    if (!weights || !weights->w_down || !h || !ids || !w || !offset || !slot_by_expert || !y) return MOE_E_INVAL;
    if (!aligned(weights->w_down, 16) || !aligned(h, 16) || !aligned(y, 16)) return MOE_E_INVAL;
    const Space p = space_of(desc, n);
    rc = check_ws(ws, ws_bytes, p.total);
    if (rc != MOE_OK) return rc;
    (void)hipGetLastError();
    char* b = reinterpret_cast<char*>(ws);
    int32_t* row_of = reinterpret_cast<int32_t*>(b + p.row_of);
    int32_t* queue = reinterpret_cast<int32_t*>(b + p.queue);
    before_down(desc, n, slot_by_expert, offset, row_of, queue, stream_of(hip_stream));
    run_down<false>(desc, Weights{weights->w_down, nullptr, nullptr, nullptr}, h, nullptr, ids, w, n, offset,
                    slot_by_expert, row_of, y, b + p.o, reinterpret_cast<uint8_t*>(b + p.os), queue, nullptr, nullptr,
                    stream_of(hip_stream));
    return launched();
}

int moe_grouped_down_fp8(const moe_layer_desc* desc, const moe_fp8_weights* weights, const void* hq,
                         const uint8_t* h_scale, const int32_t* ids, const float* w, int32_t n, const int32_t* offset,
                         const int32_t* slot_by_expert, void* y, void* ws, size_t ws_bytes, void* hip_stream) {
    int rc = check_desc(desc, n, MOE_FP8);
    if (rc != MOE_OK) return rc;
    if (!weights || !fp8_ok(weights->w_down, weights->s_down) || !fp8_ok(hq, h_scale) || !ids || !w || !offset ||
        !slot_by_expert || !y || !aligned(y, 16))
        return MOE_E_INVAL;
    const Space p = space_of(desc, n);
    rc = check_ws(ws, ws_bytes, p.total);
    if (rc != MOE_OK) return rc;
    (void)hipGetLastError();
    char* b = reinterpret_cast<char*>(ws);
    int32_t* row_of = reinterpret_cast<int32_t*>(b + p.row_of);
    int32_t* queue = reinterpret_cast<int32_t*>(b + p.queue);
    before_down(desc, n, slot_by_expert, offset, row_of, queue, stream_of(hip_stream));
    run_down<true>(desc, Weights{weights->w_down, nullptr, weights->s_down, nullptr}, hq, h_scale, ids, w, n, offset,
                   slot_by_expert, row_of, y, b + p.o, reinterpret_cast<uint8_t*>(b + p.os), queue, nullptr, nullptr,
                   stream_of(hip_stream));
    return launched();
}

int moe_expert_grouped(const moe_layer_desc* desc, const moe_layer_weights* weights, const void* x, const int32_t* ids,
                       const float* w, int32_t n, void* y, int32_t* info, void* ws, size_t ws_bytes,
                       void* hip_stream) {
    int rc = check_desc(desc, n, MOE_BF16);
    if (rc != MOE_OK) return rc;
    if (!weights || !weights->w_gate || !weights->w_up || !weights->w_down || !x || !ids || !w || !y)
        return MOE_E_INVAL;
    if (!aligned(weights->w_gate, 16) || !aligned(weights->w_up, 16) || !aligned(weights->w_down, 16) ||
        !aligned(x, 16) || !aligned(y, 16))
        return MOE_E_INVAL;
    rc = check_ws(ws, ws_bytes, space_of(desc, n).total);
    if (rc != MOE_OK) return rc;
    return run_pass<false>(desc, Weights{weights->w_gate, weights->w_up, nullptr, nullptr},
                           Weights{weights->w_down, nullptr, nullptr, nullptr}, x, ids, w, n, y, info, ws,
                           stream_of(hip_stream));
}

int moe_expert_grouped_fp8(const moe_layer_desc* desc, const moe_fp8_weights* weights, const void* x,
                           const int32_t* ids, const float* w, int32_t n, void* y, int32_t* info, void* ws,
                           size_t ws_bytes, void* hip_stream) {
    int rc = check_desc(desc, n, MOE_FP8);
    if (rc != MOE_OK) return rc;
    if (!weights || !fp8_ok(weights->w_gate, weights->s_gate) || !fp8_ok(weights->w_up, weights->s_up) ||
        !fp8_ok(weights->w_down, weights->s_down) || !x || !aligned(x, 16) || !ids || !w || !y || !aligned(y, 16))
        return MOE_E_INVAL;
    rc = check_ws(ws, ws_bytes, space_of(desc, n).total);
    if (rc != MOE_OK) return rc;
    return run_pass<true>(desc, Weights{weights->w_gate, weights->w_up, weights->s_gate, weights->s_up},
                          Weights{weights->w_down, nullptr, weights->s_down, nullptr}, x, ids, w, n, y, info, ws,
                          stream_of(hip_stream));
}

int moe_quant_rows(const void* x, int64_t rows, int32_t K, void* q, uint8_t* scale, void* hip_stream) {
    if (!x || !q || !scale || !aligned(x, 16) || !aligned(q, 16)) return MOE_E_INVAL;
    if (K < 16 || K % 16) return MOE_E_DTYPE;
    if (rows < 1 || rows > MOE_MAX_GROUP_SLOTS || K > MOE_MAX_GROUP_WIDTH) return MOE_E_INVAL;
    (void)hipGetLastError();
    hipLaunchKernelGGL(k_quant_rows<false>, dim3(rows_grid(rows, K)), dim3(256), 0, stream_of(hip_stream),
                       reinterpret_cast<const char*>(x), rows, K, static_cast<const int32_t*>(nullptr),
                       reinterpret_cast<uint8_t*>(q), scale);
    return launched();
}

int moe_dequant_rows(const void* q, const uint8_t* scale, int64_t rows, int32_t K, void* x, void* hip_stream) {
    if (!x || !q || !scale || !aligned(x, 16) || !aligned(q, 16)) return MOE_E_INVAL;
    if (K < 16 || K % 16) return MOE_E_DTYPE;
    if (rows < 1 || rows > MOE_MAX_GROUP_SLOTS || K > MOE_MAX_GROUP_WIDTH) return MOE_E_INVAL;
    (void)hipGetLastError();
    hipLaunchKernelGGL(k_dequant_rows, dim3(rows_grid(rows, K)), dim3(256), 0, stream_of(hip_stream),
                       reinterpret_cast<const uint8_t*>(q), scale, rows, K, reinterpret_cast<char*>(x));
    return launched();
}

int moe_quant_weights(const void* w, int32_t N, int32_t R, int32_t K, void* q, uint8_t* scale, void* hip_stream) {
    if (!w || !q || !scale || !aligned(w, 16) || !aligned(q, 16)) return MOE_E_INVAL;
    if (R < 16 || K < 16 || R % 16 || K % 16) return MOE_E_DTYPE;
    if (N < 1 || N > MOE_MAX_EXPERTS || R > MOE_MAX_GROUP_WIDTH || K > MOE_MAX_GROUP_WIDTH) return MOE_E_INVAL;
    const int64_t grid = (int64_t)N * blocks_of(R) * blocks_of(K);
    (void)hipGetLastError();
    hipLaunchKernelGGL(k_quant_weights, dim3((unsigned)grid), dim3(256), 0, stream_of(hip_stream),
                       reinterpret_cast<const char*>(w), R, K, reinterpret_cast<uint8_t*>(q), scale);
    return launched();
}

}  // extern "C"
