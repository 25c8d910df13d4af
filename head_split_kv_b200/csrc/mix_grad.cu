// mix_grad.cu -- the backward pass of the gated mix on the 5th-generation
// tensor cores (bf16, head_dim 128), and the preparation both backward paths
// share.
//
// Forward, per query head and row i: with scores s_ij (capped or not),
//   out = a A_c + (1 - a) A_s,  A_c / A_s softmax attention under the causal /
//   the Lambda mask, a the gate of the KV head.
// Backward, with P_c, P_s the two softmax matrices and dP_ij = dout_i . v_j:
//   D_c = dout_i . A_c,i    D_s = dout_i . A_s,i
//   W   = a P_c + (1 - a) P_s
//   E   = a P_c D_c + (1 - a) P_s D_s
//   dS  = (W dP - E) * (slope of the cap) * scale
//   dV  = W^T dout    dK = dS^T Q    dQ = dS K    da = sum (D_c - D_s),
// one pass for both attentions: P_s is nonzero in the tiles of the sink
// tokens and of the recent band only, so every other tile costs what causal
// attention costs.  P_c and P_s are recomputed from the scores and the rows'
// lse that the forward pass kept; a and 1 - a ride in the exponent:
// |a| P_c = 2^(s - (lse_c - log2 |a|)).
//
// mix_stats_kernel writes each row's {lse_c - log2|a|, D_c, lse_s - log2|1-a|,
// D_s} and its share of da; rows past the sequence get lse = +inf, so that
// their weights are 0 everywhere below.
//
// mix_grad_kernel, twice: with keys outer (dK, dV: a CTA owns 128 keys of one
// KV head and walks the 128-query tiles at or below the diagonal of every
// query head of the group) and with queries outer (dQ: 128 queries of one
// query head, walking the key tiles up to the diagonal).  So no partial sum
// leaves a CTA: no atomics, results do not depend on the order CTAs run in,
// and the heads of a group are summed in the accumulator.  The price is that
// S and dP are computed in both (7 products instead of 5).
//   outer tiles X0, X1 = K, V (or Q, dout), resident in shared memory;
//   inner tiles Y0, Y1 = Q, dout (or K, V), TMA into a 2-stage ring.
//   S = X0 Y0^T, dP = X1 Y1^T (lane = outer row), then W and dS rounded to
//   bf16 over the columns of S and dP they came from, and
//   ACC1 += W Y1 (dV), ACC2 += dS Y0 (dK or dQ) with A read from TMEM.
// TMEM: S | dP | ACC1 | ACC2, 128 columns each.  The MMA thread's order is
//   ACC1(j) S(j+1) | ACC2(j) dP(j+1) | ...
// so the element-wise warps turn dP(j) into dS(j) while the tensor core runs
// ACC1(j) and S(j+1), and S(j+1) into W(j+1) while it runs ACC2(j) and
// dP(j+1).  Roles (320 threads): warps 0-7 element-wise (warp w: lanes
// 32 (w % 4) .., columns 64 (w / 4) ..), warp 8 TMA, warp 9 MMA.
#include <cuda.h>

#include "cap.cuh"
#include "common.cuh"
#include "internal.h"
#include "mix_grad.cuh"
#include "tcgen05.cuh"

namespace duo {
namespace {

// ------------------------------------------------------------ row statistics

constexpr int kStatRows = 32;      // rows of a CTA, each with the G heads of one KV head
constexpr int kStatWarps = 8;

struct StatArgs {
    const void* dout;      // [B][N][Hq][d]
    const void* causal;    // A_c, [B][N][Hq][d]
    const void* streaming; // A_s
    const float* lse;      // [2][B][Hq][N]: causal, streaming
    const float* alpha;    // [Hkv]
    float* stats;          // [B][Hq][4][n_pad]
    float* part;           // [Hkv][B * chunks] shares of dalpha
    int N, n_pad, chunks;
};

template <typename T, int D>
__global__ void __launch_bounds__(kStatWarps * 32) mix_stats_kernel(const LayerArgs a, const StatArgs x) {
    constexpr int E = D / 32;      // elements a lane
    const int chunk = blockIdx.x, kv = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float al = x.alpha[kv];
    const float shift_c = -log2f(fabsf(al)), shift_s = -log2f(fabsf(1.f - al));   // +inf for a closed gate
    const size_t plane = (size_t)a.B * a.Hq * x.N;
    float share = 0.f;
    for (int it = warp; it < kStatRows * a.G; it += kStatWarps) {
        const int i = chunk * kStatRows + it / a.G, h = kv * a.G + it % a.G;
        if (i >= x.n_pad) break;
        float* st = x.stats + ((size_t)b * a.Hq + h) * 4 * x.n_pad + i;
        if (i >= x.N) {
            if (lane == 0) {
                st[0] = st[2 * (size_t)x.n_pad] = INFINITY;
                st[x.n_pad] = st[3 * (size_t)x.n_pad] = 0.f;
            }
            continue;
        }
        const size_t o = (((size_t)b * x.N + i) * a.Hq + h) * D + lane * E;
        float dc = 0.f, ds = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float g = Elem<T>::to_f32(static_cast<const T*>(x.dout)[o + e]);
            dc = fmaf(g, Elem<T>::to_f32(static_cast<const T*>(x.causal)[o + e]), dc);
            ds = fmaf(g, Elem<T>::to_f32(static_cast<const T*>(x.streaming)[o + e]), ds);
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) {
            dc += __shfl_xor_sync(0xffffffffu, dc, s);
            ds += __shfl_xor_sync(0xffffffffu, ds, s);
        }
        if (lane == 0) {
            const size_t r = ((size_t)b * a.Hq + h) * x.N + i;
            st[0] = x.lse[r] + shift_c;
            st[x.n_pad] = dc;
            st[2 * (size_t)x.n_pad] = x.lse[plane + r] + shift_s;
            st[3 * (size_t)x.n_pad] = ds;
            share += dc - ds;
        }
    }
    __shared__ float s_share[kStatWarps];
    if (lane == 0) s_share[warp] = share;
    __syncthreads();
    if (threadIdx.x == 0) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kStatWarps; ++w) sum += s_share[w];
        x.part[(size_t)kv * a.B * x.chunks + (size_t)b * x.chunks + chunk] = sum;
    }
}

// --------------------------------------------------------------- the kernel

constexpr int BM = 128;            // rows of an outer or inner tile
constexpr int HD = 128;
constexpr int kTmaWarp = 8, kMmaWarp = 9, kGradThreads = 320;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColP = 128, kColA1 = 256, kColA2 = 384;
constexpr uint32_t kTileBytes = BM * HD * 2;       // 32 KB: two 16 KB halves of d
constexpr uint32_t kHalfBytes = kTileBytes / 2;
constexpr uint32_t kStatBytes = 4 * BM * 4;        // a query tile's four rows of statistics
constexpr uint32_t kOffX = 0;                      // X0, X1
constexpr uint32_t kOffY = 2 * kTileBytes;         // stages of Y0, Y1
constexpr uint32_t kOffStat = kOffY + 4 * kTileBytes;
constexpr uint32_t kOffBar = kOffStat + 2 * kStatBytes;
constexpr uint32_t kOffHolder = kOffBar + 16 * 8;
constexpr uint32_t kGradSmem = kOffHolder + 16;
static_assert(kGradSmem + 1024 <= 232448, "one CTA per SM");

struct GradArgs {
    LayerArgs a;
    int N, n_tiles, n_pad;
    const float* stats;    // [B][Hq][4][n_pad]
    const float* alpha;
    void* d0;              // keys outer: dK; queries outer: dQ
    void* d1;              // keys outer: dV
    const float* part;     // [Hkv][n_part], keys outer: the shares of dalpha
    int n_part;
    float* dalpha;
    int32_t* status;
};

// A tile pair holds keys some query sees in the Lambda attention: sink tokens,
// or the recent band (the diagonal tile always does, so every tile that
// needs a mask is one of these).
__device__ __forceinline__ bool lambda_tile(const LayerArgs& a, int qt, int kt) {
    return kt * BM < a.sink || (qt - kt) * BM - (BM - 1) < a.recent;
}

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
    __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&h);
}

// A warp's 64 columns of a tile without Lambda keys.  First half: x[] dot
// products -> |a| P_c (packed bf16 to TMEM when `store`), x[] = |a| P_c times
// the cap's slope.
template <bool CAP, bool KEYS>
__device__ __forceinline__ void causal_weights(float (&x)[64], const LayerArgs& a, float sl, const float* s_lse, float lse,
                                               bool neg, uint32_t w_addr) {
    float big = 0.f;
    bool poly = false;
    if constexpr (CAP) {
#pragma unroll
        for (int c = 0; c < 64; c += 2) big = fmax3(big, fabsf(x[c]), fabsf(x[c + 1]));
        poly = __all_sync(0xffffffffu, big * a.cap.k <= 1.f);
        if (!poly) {
#pragma unroll
            for (int c = 0; c < 64; ++c) x[c] = tanh_sfu(x[c] * a.cap.k);
        }
    }
    uint32_t pk[32];
#pragma unroll
    for (int c4 = 0; c4 < 16; ++c4) {
        float4 l4 = KEYS ? reinterpret_cast<const float4*>(s_lse)[c4] : make_float4(lse, lse, lse, lse);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = 4 * c4 + 2 * h;
            float2 v = make_float2(x[c], x[c + 1]);
            const float2 nl = h ? make_float2(-l4.z, -l4.w) : make_float2(-l4.x, -l4.y);
            float2 slope;
            if constexpr (CAP) {
                if (poly) v = tanh_fma2(fmul2(v, make_float2(a.cap.k, a.cap.k)));
                slope = ffma2(make_float2(-v.x, -v.y), v, make_float2(1.f, 1.f));
                v = ffma2(v, make_float2(a.cap.c2, a.cap.c2), nl);
            } else {
                v = ffma2(v, make_float2(sl, sl), nl);
            }
            v = make_float2(sfu_exp2(v.x), sfu_exp2(v.y));
            if (neg) v = make_float2(-v.x, -v.y);
            if constexpr (KEYS) pk[c / 2] = pack_bf16(v.x, v.y);
            if constexpr (CAP) v = fmul2(v, slope);
            x[c] = v.x;
            x[c + 1] = v.y;
        }
    }
    if constexpr (KEYS) tmem_st32(w_addr, pk);
}

template <bool KEYS, bool CAP>
__global__ void __launch_bounds__(kGradThreads, 1)
    mix_grad_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDo,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const GradArgs p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const LayerArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((smem_u32(smem) & 1023u) != 0) {   // the swizzled layouts need 1024-byte alignment
        if (tid == 0) atomicOr(p.status, DUO_DEV_BAD_LENGTH);
        return;
    }
    const uint32_t sX = smem_u32(smem + kOffX), sY = smem_u32(smem + kOffY);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint64_t* x_full = bars + 0;
    uint64_t* y_full = bars + 1;    // [2]
    uint64_t* y_empty = bars + 3;   // [2]
    uint64_t* s_full = bars + 5;
    uint64_t* d_full = bars + 6;
    uint64_t* w_ready = bars + 7;   // W written (keys outer), S read
    uint64_t* g_ready = bars + 8;   // dS written
    uint64_t* done = bars + 9;
    uint32_t* holder = reinterpret_cast<uint32_t*>(smem + kOffHolder);

    // Work item, the longest first.  Keys outer: key tile ot of KV head `head`,
    // whose inner tiles are (query head of the group, query tile >= ot);
    // queries outer: query tile ot of query head `head`, key tiles 0 .. ot.
    const int heads = KEYS ? a.Hkv : a.Hq;
    const int ord = blockIdx.x / (a.B * heads), rest = blockIdx.x % (a.B * heads);
    const int head = rest % heads, b = rest / heads;
    const int ot = KEYS ? ord : p.n_tiles - 1 - ord;
    const int kv = KEYS ? head : head / a.G;
    const int per_head = p.n_tiles - ot;                   // keys outer: query tiles per query head
    const int n_in = KEYS ? a.G * per_head : ot + 1;
    auto inner_tile = [&](int j) { return KEYS ? ot + j % per_head : j; };
    auto inner_qhead = [&](int j) { return KEYS ? kv * a.G + j / per_head : head; };

    if (warp == kMmaWarp) tmem_alloc(holder, kTmemCols);
    if (tid == 0) {
        mbar_init(x_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&y_full[i], 1);
            mbar_init(&y_empty[i], KEYS ? 9 : 1);   // the MMAs' commit, and the warps that read the stage's statistics
        }
        mbar_init(s_full, 1);
        mbar_init(d_full, 1);
        mbar_init(w_ready, 8);
        mbar_init(g_ready, 8);
        mbar_init(done, 1);
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;

    if (warp == kTmaWarp) {
        if (lane == 0) {
            const CUtensorMap* mx0 = KEYS ? &tmK : &tmQ;
            const CUtensorMap* mx1 = KEYS ? &tmV : &tmDo;
            const CUtensorMap* my0 = KEYS ? &tmQ : &tmK;
            const CUtensorMap* my1 = KEYS ? &tmDo : &tmV;
            mbar_arrive_expect_tx(x_full, 2 * kTileBytes);
            for (int half = 0; half < 2; ++half) {
                tma_load_4d(sX + half * kHalfBytes, mx0, 64 * half, head, BM * ot, b, x_full);
                tma_load_4d(sX + kTileBytes + half * kHalfBytes, mx1, 64 * half, head, BM * ot, b, x_full);
            }
            for (int j = 0; j < n_in; ++j) {
                const int st = j & 1, it = inner_tile(j), ih = KEYS ? inner_qhead(j) : kv;
                if (j >= 2 && !mbar_wait(&y_empty[st], ((j >> 1) - 1) & 1, p.status)) break;
                mbar_arrive_expect_tx(&y_full[st], 2 * kTileBytes + (KEYS ? kStatBytes : 0u));
                const uint32_t y = sY + st * 2 * kTileBytes;
                for (int half = 0; half < 2; ++half) {
                    tma_load_4d(y + half * kHalfBytes, my0, 64 * half, ih, BM * it, b, &y_full[st]);
                    tma_load_4d(y + kTileBytes + half * kHalfBytes, my1, 64 * half, ih, BM * it, b, &y_full[st]);
                }
                if constexpr (KEYS) {
                    const float* src = p.stats + ((size_t)b * a.Hq + ih) * 4 * p.n_pad + BM * it;
                    for (int r = 0; r < 4; ++r)
                        bulk_g2s(smem + kOffStat + st * kStatBytes + r * BM * 4, src + (size_t)r * p.n_pad, BM * 4,
                                 &y_full[st]);
                }
            }
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            constexpr uint32_t idesc_kk = idesc_bf16(BM, BM, 0, 0);
            constexpr uint32_t idesc_mn = idesc_bf16(BM, HD, 0, 1);
            // D = X_w Y_w(j)^T over d
            auto issue_xy = [&](uint32_t col, int w, int j) {
                const uint32_t x = sX + w * kTileBytes, y = sY + ((j & 1) * 2 + w) * kTileBytes;
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t o = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
                    tc_mma(tmem + col, sw128_desc(x + o, 16, 1024), sw128_desc(y + o, 16, 1024), idesc_kk, kk > 0 ? 1u : 0u);
                }
            };
            // ACC += A (bf16 over the columns it came from) Y_w(j), over the inner rows
            auto issue_acc = [&](uint32_t col, uint32_t a_col, int w, int j) {
                const uint32_t y = sY + ((j & 1) * 2 + w) * kTileBytes;
#pragma unroll
                for (int kk = 0; kk < BM / 16; ++kk)
                    tc_mma_ta(tmem + col, tmem + a_col + 64 * (kk >> 2) + 8 * (kk & 3),
                              sw128_desc(y + kk * 2048, kHalfBytes, 1024), idesc_mn, (j > 0 || kk > 0) ? 1u : 0u);
            };
            bool ok = mbar_wait(x_full, 0, p.status) && mbar_wait(&y_full[0], 0, p.status);
            if (ok) {
                tc_fence_after();
                issue_xy(kColS, 0, 0);
                tc_commit(s_full);
                issue_xy(kColP, 1, 0);
                tc_commit(d_full);
            }
            for (int j = 0; j < n_in && ok; ++j) {
                const bool next = j + 1 < n_in;
                if (next) ok = mbar_wait(&y_full[(j + 1) & 1], ((j + 1) >> 1) & 1, p.status);
                ok = ok && mbar_wait(w_ready, j & 1, p.status);
                if (!ok) break;
                tc_fence_after();
                if constexpr (KEYS) issue_acc(kColA1, kColS, 1, j);
                if (next) {
                    issue_xy(kColS, 0, j + 1);
                    tc_commit(s_full);
                }
                ok = mbar_wait(g_ready, j & 1, p.status);
                if (!ok) break;
                tc_fence_after();
                issue_acc(kColA2, kColP, 0, j);
                tc_commit(&y_empty[j & 1]);
                if (next) {
                    issue_xy(kColP, 1, j + 1);
                    tc_commit(d_full);
                } else {
                    tc_commit(done);
                }
            }
        }
    } else {
        // ------------------------------------------------ element-wise warps
        const int wg = warp >> 2;                             // columns 64 wg ..
        const int row = 32 * (warp & 3) + lane;               // TMEM lane: outer row
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t s_addr = lane_addr + kColS + 64 * wg, d_addr = lane_addr + kColP + 64 * wg;
        const float sl = a.scale * kLog2e;
        const float al = p.alpha[kv];
        const bool neg_c = al < 0.f, neg_s = 1.f - al < 0.f;
        const int orow = BM * ot + row;                       // key (keys outer) or query
        float lse_c = 0.f, dc = 0.f, lse_s = 0.f, ds = 0.f;
        if constexpr (!KEYS) {
            const float* st = p.stats + ((size_t)b * a.Hq + head) * 4 * p.n_pad + orow;
            lse_c = st[0];
            dc = st[p.n_pad];
            lse_s = st[2 * (size_t)p.n_pad];
            ds = st[3 * (size_t)p.n_pad];
        }
        bool ok = true;
        for (int j = 0; j < n_in; ++j) {
            const int it = inner_tile(j);
            const float* stat = reinterpret_cast<const float*>(smem + kOffStat + (j & 1) * kStatBytes) + 64 * wg;
            // the statistics arrived with the tile that S(j) was computed from;
            // this wait makes the copy visible to this thread too
            if constexpr (KEYS) ok = ok && mbar_wait(&y_full[j & 1], (j >> 1) & 1, p.status);
            ok = __all_sync(0xffffffffu, ok && mbar_wait(s_full, j & 1, p.status));
            if (!ok) break;
            tc_fence_after();
            if (!lambda_tile(a, KEYS ? it : ot, KEYS ? ot : it)) {
                float x[64];
                tmem_ld64(s_addr, x);
                causal_weights<CAP, KEYS>(x, a, sl, stat, lse_c, neg_c, s_addr);
                if constexpr (KEYS) tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(w_ready);
                ok = __all_sync(0xffffffffu, mbar_wait(d_full, j & 1, p.status));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float d[32];
                    tmem_ld32(d_addr + 32 * h, d);
                    uint32_t pk[16];
#pragma unroll
                    for (int c4 = 0; c4 < 8; ++c4) {
                        const float4 q = KEYS ? reinterpret_cast<const float4*>(stat + BM)[8 * h + c4] : make_float4(dc, dc, dc, dc);
                        const int c = 4 * c4;
                        const float2 u = fmul2(make_float2(x[32 * h + c], x[32 * h + c + 1]),
                                               fadd2(make_float2(d[c], d[c + 1]), make_float2(-q.x, -q.y)));
                        const float2 v = fmul2(make_float2(x[32 * h + c + 2], x[32 * h + c + 3]),
                                               fadd2(make_float2(d[c + 2], d[c + 3]), make_float2(-q.z, -q.w)));
                        pk[2 * c4] = pack_bf16(u.x, u.y);
                        pk[2 * c4 + 1] = pack_bf16(v.x, v.y);
                    }
                    tmem_st16(d_addr + 16 * h, pk);
                }
            } else {
                // both attentions, and the masks: 16 columns at a time
                ok = __all_sync(0xffffffffu, mbar_wait(d_full, j & 1, p.status));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int ch = 0; ch < 4; ++ch) {
                    float x[16], d[16];
                    tmem_ld16(s_addr + 16 * ch, x);
                    tmem_ld16(d_addr + 16 * ch, d);
                    uint32_t pw[8], pg[8];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const int icol = BM * it + 64 * wg + 16 * ch + c;
                        const int query = KEYS ? icol : orow, key = KEYS ? orow : icol;
                        const float lc = KEYS ? stat[16 * ch + c] : lse_c, qc = KEYS ? stat[BM + 16 * ch + c] : dc;
                        const float ls = KEYS ? stat[2 * BM + 16 * ch + c] : lse_s, qs = KEYS ? stat[3 * BM + 16 * ch + c] : ds;
                        float slope = 1.f, s;
                        if constexpr (CAP) {
                            const float t = tanh_sfu(x[c] * a.cap.k);
                            slope = fmaf(-t, t, 1.f);
                            s = t * a.cap.c2;
                        } else {
                            s = x[c] * sl;
                        }
                        const bool causal = key <= query;
                        const bool lam = causal && (key < a.sink || query - key < a.recent);
                        float wc = causal ? sfu_exp2(s - lc) : 0.f;
                        float ws = lam ? sfu_exp2(s - ls) : 0.f;
                        wc = neg_c ? -wc : wc;
                        ws = neg_s ? -ws : ws;
                        const float w = wc + ws;
                        x[c] = w;
                        d[c] = slope * fmaf(w, d[c], -fmaf(wc, qc, ws * qs));
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        pw[c] = pack_bf16(x[2 * c], x[2 * c + 1]);
                        pg[c] = pack_bf16(d[2 * c], d[2 * c + 1]);
                    }
                    if constexpr (KEYS) tmem_st8(s_addr + 8 * ch, pw);
                    tmem_st8(d_addr + 8 * ch, pg);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(w_ready);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(g_ready);
                if constexpr (KEYS) mbar_arrive(&y_empty[j & 1]);   // done with the stage's statistics
            }
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait(done, 0, p.status));
        if (ok) {
            tc_fence_after();
            const int H = KEYS ? a.Hkv : a.Hq;
            const size_t off = (((size_t)b * p.N + orow) * H + head) * HD + 64 * wg;
            const bool live = orow < p.N && bounds_ok(b < a.B && head < H, p.status);
#pragma unroll
            for (int t = 0; t < (KEYS ? 2 : 1); ++t) {
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(t ? p.d1 : p.d0) + off;
                const float f = t ? 1.f : a.scale;            // dS held back the softmax scale
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[32];
                    tmem_ld32(lane_addr + (t ? kColA1 : kColA2) + 64 * wg + 32 * h, v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v8[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v8[i] = v[8 * e + i] * f;
                        if (live) store_row<__nv_bfloat16, 8>(o + 32 * h + 8 * e, v8);
                    }
                }
            }
        }
        // one warp per KV head adds up the shares of dalpha, in their order
        if (KEYS && ot == 0 && b == 0 && warp == 0) sum_shares(p.part + (size_t)kv * p.n_part, p.n_part, &p.dalpha[kv], lane);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <bool KEYS, bool CAP>
cudaError_t launch_grad(const CUtensorMap (&m)[4], const GradArgs& p, cudaStream_t s) {
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = smem_limit_once(mix_grad_kernel<KEYS, CAP>, (int)kGradSmem, configured);
    if (e != cudaSuccess) return e;
    const long grid = (long)p.a.B * (KEYS ? p.a.Hkv : p.a.Hq) * p.n_tiles;
    if (grid > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    mix_grad_kernel<KEYS, CAP><<<(unsigned)grid, kGradThreads, kGradSmem, s>>>(m[0], m[1], m[2], m[3], p);
    return cudaGetLastError();
}

}  // namespace

MixGradPlan mix_grad_plan(const LayerArgs& a, int N) {
    MixGradPlan pl{};
    pl.n_pad = (N + BM - 1) / BM * BM;
    pl.chunks = (pl.n_pad + kStatRows - 1) / kStatRows;
    const size_t stats = (size_t)a.B * a.Hq * 4 * pl.n_pad * sizeof(float);
    pl.part_offset = (stats + 255) / 256 * 256;
    pl.bytes = pl.part_offset + ((size_t)a.Hkv * a.B * pl.chunks * sizeof(float) + 255) / 256 * 256;
    return pl;
}

cudaError_t launch_mix_stats(const LayerArgs& a, const MixGradArgs& g, int N, cudaStream_t s) {
    const MixGradPlan pl = mix_grad_plan(a, N);
    if (a.B > 65535) return cudaErrorInvalidConfiguration;
    const StatArgs x{g.dout, g.causal, g.streaming, g.lse, g.alpha, g.stats, g.part, N, pl.n_pad, pl.chunks};
    const dim3 grid((unsigned)pl.chunks, (unsigned)a.Hkv, (unsigned)a.B);
    constexpr int th = kStatWarps * 32;
    if (a.dtype == DUO_BF16) {
        if (a.D == 128) mix_stats_kernel<__nv_bfloat16, 128><<<grid, th, 0, s>>>(a, x);
        else mix_stats_kernel<__nv_bfloat16, 64><<<grid, th, 0, s>>>(a, x);
    } else {
        if (a.D == 128) mix_stats_kernel<float, 128><<<grid, th, 0, s>>>(a, x);
        else mix_stats_kernel<float, 64><<<grid, th, 0, s>>>(a, x);
    }
    return cudaGetLastError();
}

cudaError_t launch_mix_grad_tc(const LayerArgs& a, const MixGradArgs& g, int N, cudaStream_t s) {
    const MixGradPlan pl = mix_grad_plan(a, N);
    CUtensorMap m[4];
    const void* base[4] = {g.q, g.dout, g.k, g.v};
    for (int i = 0; i < 4; ++i) {
        const uint64_t H = i < 2 ? a.Hq : a.Hkv, row = HD * 2;
        const uint64_t d[4] = {HD, H, (uint64_t)N, (uint64_t)a.B};
        const uint64_t st[3] = {row, row * H, row * H * N};
        const uint32_t bx[4] = {64, 1, BM, 1};
        if (!encode_tmap_bf16(&m[i], base[i], 4, d, st, bx)) return cudaErrorInvalidValue;
    }
    GradArgs p{a, N, pl.n_pad / BM, pl.n_pad, g.stats, g.alpha, g.dk, g.dv, g.part, a.B * pl.chunks, g.dalpha, g.status};
    cudaError_t e = a.cap.on ? launch_grad<true, true>(m, p, s) : launch_grad<true, false>(m, p, s);
    if (e != cudaSuccess) return e;
    p.d0 = g.dq;
    p.d1 = nullptr;
    return a.cap.on ? launch_grad<false, true>(m, p, s) : launch_grad<false, false>(m, p, s);
}

}  // namespace duo
