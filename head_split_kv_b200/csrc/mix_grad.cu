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
// One row of statistics serves both attentions.  P_c and P_s of a row are the
// same exponentials over different sums, so for a key that both see
//   W = 2^(s - lse*)  with  2^-lse* = a 2^-lse_c + (1 - a) 2^-lse_s,
//   dS ~ W (dP - D*)  with  D* the mean of D_c and D_s under those two shares,
// and a tile with sink or recent keys costs a choice between two (lse, D)
// pairs, not a second exponential.  (A gate outside [0, 1] makes the shares
// differ in sign; those heads take both exponentials there.)
//
// mix_stats_kernel computes D_c and D_s as sums of P dP in fp32 over the same
// tiles, and corrects the log-sums by the sum of P: dout . A from the stored
// bf16 attention would carry the roundings of P and of A, which where a row's
// softmax is peaked are as large as dP - D itself (dq and dk were 3.4 times as
// far from fp64 as their rounding).  It writes each row's {lse_c - log2 a, D_c,
// lse*, D*} and its share of da; rows past the sequence get lse = +inf, so that
// their weights are 0 below.
//
// mix_grad_kernel, twice: with keys outer (dK, dV: a CTA owns 128 keys of one
// KV head and walks the 128-query tiles at or below the diagonal of every
// query head of the group) and with queries outer (dQ: 128 queries of one
// query head, walking the key tiles up to the diagonal).  Where the first key
// tile alone would outlast an SM's share, the two CTAs of a cluster halve a
// tile's queries and each adds the other's part of one accumulator through
// shared memory (share_key_tiles).  So no partial sum goes through global
// memory: no atomics, results do not depend on the order CTAs run in, and the
// heads of a group are summed in the accumulator.  The price is that S and dP
// are computed in every launch (9 products instead of 5).
//   outer tiles X0, X1 = K, V (or Q, dout), resident in shared memory;
//   inner tiles Y0, Y1 = Q, dout (or K, V), TMA into a 2-stage ring.
//   S = X0 Y0^T, dP = X1 Y1^T (lane = outer row), then W and dS, rounded to
//   bf16, share the columns of dP, and
//   ACC1 += W Y1 (dV), ACC2 += dS Y0 (dK or dQ) with A read from TMEM.
// TMEM: S | dP | ACC1 | ACC2, 128 columns each; without ACC1 (statistics, dQ) a
// second S takes its place, and for the statistics a second dP that of ACC2.
// (Sequences of one tile add dS's rounding remainder as a third operand; keep_rest.)
// S is free as soon as the element-wise warps have loaded it, so S(j + 1) is
// there when they have finished tile j, and
//   ACC1(j) ACC2(j) dP(j + 1)
// run while they turn S(j + 1) into weights.  (With W over S's columns, S(j + 1)
// had to wait for ACC1(j), and the warps for it: dK and dV 355 -> 323 us.)
// Roles (576 threads): warps 0-15 element-wise (warp w: lanes 32 (w % 4) ..,
// columns 32 (w / 4) ..), warp 16 TMA, warp 17 MMA.  Sixteen warps at 96
// registers (an SM sub-partition holds five warps) against eight at 168: the
// element-wise work is a chain of dependent operations, and with two warps
// to a sub-partition it issued on 29-39 % of cycles.
#include <cuda.h>

#include "cap.cuh"
#include "common.cuh"
#include "internal.h"
#include "mix_grad.cuh"
#include "tcgen05.cuh"

namespace duo {
namespace {

// --------------------------------------------------------------- the kernel

constexpr int BM = 128;            // rows of an outer or inner tile
constexpr int HD = 128;
constexpr int kElemWarps = 16, kCols = 32;          // columns of an element-wise warp
constexpr int kChunk = 16;                          // of them taken from TMEM at a time
constexpr int kTmaWarp = 16, kMmaWarp = 17, kGradThreads = 576;
constexpr int kRegThreads = 640;                   // five warps to a sub-partition: 96 registers
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColP = 128, kColA1 = 256, kColA2 = 384;   // second S at kColA1, second dP at kColA2
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
    float* stats;          // [B][Hq][4][n_pad]: -(lse_c - log2 a), -D_c, -lse*, -D*
    const float* lse;      // [2][B][Hq][N] of the forward pass
    const float* alpha;
    void* d0;              // keys outer: dK; queries outer: dQ
    void* d1;              // keys outer: dV
    float* part;           // [Hkv][B][n_tiles][G], the shares of dalpha
    float* dalpha;
    int32_t* status;
    TanhPoly poly;         // tanh(k x)
};

// What a launch computes: the rows' statistics, dK and dV (keys outer; with
// pairs of CTAs that share a key tile), or dQ.
enum { STATS = 0, KEYS = 1, QUERIES = 2, KEY_PAIRS = 3 };
enum { NO_CAP = 0, CAPPED = 1, CAP_FAR = 2 };   // CapArgs::on, ::far
__host__ __device__ constexpr bool keys_outer(int mode) { return mode == KEYS || mode == KEY_PAIRS; }

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
    __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&h);
}

// Every thread of the cluster's CTAs, what they wrote to shared memory visible after it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\t"
        "barrier.cluster.wait.acquire.aligned;" ::
            : "memory");
}
// The address of this CTA's shared-memory location in CTA `rank` of the cluster, and a store there.
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_peer(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Bits lo .. hi (inclusive, clipped to 0 .. 31).
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, 31);
    return lo > hi ? 0u : (~0u >> (31 - hi)) & (~0u << lo);
}

// Which of a thread's 32 columns its row sees under the two masks.  Rows are
// keys and columns queries, or the other way round.
struct Seen {
    uint32_t causal, lam;
};
__device__ __forceinline__ Seen seen_columns(const LayerArgs& a, bool keys_outer, int row, int col0) {
    if (keys_outer) {
        const uint32_t c = bit_range(row - col0, 31);
        return {c, row < a.sink ? c : bit_range(row - col0, row + a.recent - 1 - col0)};
    }
    const uint32_t c = bit_range(0, row - col0);
    return {c, c & (bit_range(0, a.sink - 1 - col0) | bit_range(row - a.recent + 1 - col0, 31))};
}

// Where a thread finds the (-lse, -D) pairs of its columns: one pair of pairs
// in registers when its row is the query, four rows of shared memory (one
// entry per column) when its columns are.
struct RowStats {
    float lse_c, dc, lse_l, dl;
    const float* cols;
};
template <bool COLS>
__device__ __forceinline__ float4 stat4(const RowStats& r, int which, int c4) {
    if constexpr (COLS) return reinterpret_cast<const float4*>(r.cols + which * BM)[c4];
    const float v = which == 0 ? r.lse_c : which == 1 ? r.dc : which == 2 ? r.lse_l : r.dl;
    return make_float4(v, v, v, v);
}

__device__ __forceinline__ float4 choose4(uint32_t bits, int shift, const float4& yes, const float4& no) {
    return make_float4((bits >> shift) & 1u ? yes.x : no.x, (bits >> (shift + 1)) & 1u ? yes.y : no.y,
                       (bits >> (shift + 2)) & 1u ? yes.z : no.z, (bits >> (shift + 3)) & 1u ? yes.w : no.w);
}

// A pair's scores plus `add`, and t, their tanh (CAP); POLY: the dot products
// are within the polynomial's range (never under a far cap, whose kernels are
// instantiations of their own: one for both took 1.5 % more).
template <int CAP, bool POLY>
__device__ __forceinline__ float2 capped2(float2 x, const CapArgs& cap, const TanhPoly& tp, float2 add, float2& t) {
    if constexpr (POLY) {
        t = poly_fma2(x, tp);
        return ffma2(t, tp.c2, add);
    }
    // the score rounded as the forward pass rounded it: whatever its size, it
    // does not lie far above the row's log-sum
    constexpr bool far = CAP == CAP_FAR;
    const Capped a = cap_sfu<far>(x.x, cap.sl, cap.k, cap.c2), b = cap_sfu<far>(x.y, cap.sl, cap.k, cap.c2);
    t = make_float2(a.t, b.t);
    return fadd2(make_float2(a.s, b.s), add);
}

// A warp's 32 columns: x[] dot products -> W, or with a cap -W times
// its slope (t^2 - 1 is one instruction; the sign goes into the last multiply);
// pk[] = W packed as bf16 when COLS (keys outer).  MASKED: some
// column is not seen, or is seen by both attentions.  One loop from the dot
// product to the packed W, so that the FMA, SFU and ALU work of neighbouring
// pairs interleaves (in separate loops the pipes took turns: their shares of
// the time added up to 96 %).
template <int CAP, bool COLS, bool MASKED, bool POLY>
__device__ __forceinline__ void weights_loop(float* x, const LayerArgs& a, float sl, const TanhPoly& tp, const RowStats& r,
                                             const Seen& seen, int col0, uint32_t* pk) {
#pragma unroll
    for (int c4 = 0; c4 < kChunk / 4; ++c4) {
        const int q4 = col0 / 4 + c4;
        float4 l4 = stat4<COLS>(r, 0, q4);
        if constexpr (MASKED) {
            l4 = choose4(seen.lam, 4 * q4, stat4<COLS>(r, 2, q4), l4);
            l4 = choose4(seen.causal, 4 * q4, l4, make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = 4 * c4 + 2 * h;
            float2 v = make_float2(x[c], x[c + 1]);
            const float2 nl = h ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y);
            float2 slope;
            if constexpr (CAP != NO_CAP) {
                float2 t;
                v = capped2<CAP, POLY>(v, a.cap, tp, nl, t);
                slope = ffma2(t, t, tp.minus1);
            } else {
                v = ffma2(v, make_float2(sl, sl), nl);
            }
            v = make_float2(sfu_exp2(v.x), sfu_exp2(v.y));
            if constexpr (COLS) pk[c / 2] = pack_bf16(v.x, v.y);
            if constexpr (CAP != NO_CAP) v = fmul2(v, slope);
            x[c] = v.x;
            x[c + 1] = v.y;
        }
    }
}
template <int CAP, bool COLS, bool MASKED>
__device__ __forceinline__ void weights(float (&x)[kCols], uint32_t (&pk)[kCols / 2], const LayerArgs& a, float sl,
                                        const TanhPoly& tp, const RowStats& r, const Seen& seen) {
#pragma unroll
    for (int ch = 0; ch < kCols / kChunk; ++ch) {
        float* y = x + kChunk * ch;
        if (CAP == NO_CAP || (CAP == CAPPED && __all_sync(0xffffffffu, largest<kChunk>(y) <= tp.x_max)))
            weights_loop<CAP, COLS, MASKED, true>(y, a, sl, tp, r, seen, kChunk * ch, pk + kChunk / 2 * ch);
        else
            weights_loop<CAP, COLS, MASKED, false>(y, a, sl, tp, r, seen, kChunk * ch, pk + kChunk / 2 * ch);
    }
}

// What the rounding of a packed pair took off it, packed as bf16.
__device__ __forceinline__ uint32_t pack_rest(uint32_t hi, float x, float y) {
    return pack_bf16(x - bf16_lo(hi), y - bf16_hi(hi));
}

// x[] and pk[] as weights left them, TMEM dP -> of every 16 columns of dP's the
// first 8 hold W (COLS) and the last 8 dS (with a cap: -dS), packed as bf16.
// REST: what dS lost in its rounding goes where S was (COLS), or the first 8.
template <bool COLS, bool MASKED, bool REST>
__device__ __forceinline__ void score_grads(const float (&x)[kCols], const uint32_t (&pk)[kCols / 2], const RowStats& r,
                                            const Seen& seen, uint32_t s_addr, uint32_t d_addr) {
#pragma unroll
    for (int ch = 0; ch < kCols / kChunk; ++ch) {
        float d[kChunk];
        tmem_ld16(d_addr + kChunk * ch, d);
        uint32_t o[kChunk], rest[kChunk / 2];
#pragma unroll
        for (int c4 = 0; c4 < kChunk / 4; ++c4) {
            const int q4 = kChunk / 4 * ch + c4;
            float4 q = stat4<COLS>(r, 1, q4);
            if constexpr (MASKED) q = choose4(seen.lam, 4 * q4, stat4<COLS>(r, 3, q4), q);
            const float* w = x + 4 * q4;
            const int c = 4 * c4;
            const float2 u = fmul2(make_float2(w[0], w[1]), fadd2(make_float2(d[c], d[c + 1]), make_float2(q.x, q.y)));
            const float2 v = fmul2(make_float2(w[2], w[3]), fadd2(make_float2(d[c + 2], d[c + 3]), make_float2(q.z, q.w)));
            o[kChunk / 2 + 2 * c4] = pack_bf16(u.x, u.y);
            o[kChunk / 2 + 2 * c4 + 1] = pack_bf16(v.x, v.y);
            if constexpr (REST) {
                rest[2 * c4] = pack_rest(o[kChunk / 2 + 2 * c4], u.x, u.y);
                rest[2 * c4 + 1] = pack_rest(o[kChunk / 2 + 2 * c4 + 1], v.x, v.y);
            }
            if constexpr (COLS) {
                o[2 * c4] = pk[2 * q4];
                o[2 * c4 + 1] = pk[2 * q4 + 1];
            }
        }
        if constexpr (REST) tmem_st8((COLS ? s_addr : d_addr) + kChunk * ch, rest);
        if constexpr (COLS) {
            tmem_st16(d_addr + kChunk * ch, o);
        } else {
            uint32_t g[kChunk / 2];
#pragma unroll
            for (int c = 0; c < kChunk / 2; ++c) g[c] = o[kChunk / 2 + c];
            tmem_st8(d_addr + kChunk * ch + kChunk / 2, g);
        }
    }
}

// A tile with keys that both attentions see, for a gate outside [0, 1]: the
// shares a P_c and (1 - a) P_s differ in sign and are formed one by one (the
// statistics hold lse_s - log2 |1 - a| and D_s), 16 columns at a time.  For a
// negative a everything a CTA accumulates is negated, so that |a| P_c is W in
// the other tiles; here its share is positive and the other one negative,
// whichever of the two signs is the odd one.
template <int CAP, bool COLS, bool REST>
__device__ __forceinline__ void signed_shares(const LayerArgs& a, float sl, const RowStats& r, Seen seen,
                                              uint32_t s_addr, uint32_t d_addr) {
#pragma unroll 1
    for (int ch = 0; ch < kCols / 16; ++ch) {
        float x[16], d[16];
        tmem_ld16(s_addr + 16 * ch, x);
        tmem_ld16(d_addr + 16 * ch, d);
        uint32_t pw[8], pg[8], rest[8];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            const float* st = r.cols + 16 * ch + c;
            const float lc = COLS ? st[0] : r.lse_c, qc = COLS ? st[BM] : r.dc;
            const float ls = COLS ? st[2 * BM] : r.lse_l, qs = COLS ? st[3 * BM] : r.dl;
            float slope = 1.f, s;
            if constexpr (CAP != NO_CAP) {
                const Capped cs = cap_sfu<CAP == CAP_FAR>(x[c], sl, a.cap.k, a.cap.c2);
                slope = fmaf(cs.t, cs.t, -1.f);
                s = cs.s;
            } else {
                s = x[c] * sl;
            }
            const float wc = (seen.causal >> c) & 1u ? sfu_exp2(s + lc) : 0.f;
            const float ws = (seen.lam >> c) & 1u ? sfu_exp2(s + ls) : 0.f;
            x[c] = wc - ws;
            d[c] = slope * fmaf(x[c], d[c], fmaf(wc, qc, -ws * qs));
        }
        seen.causal >>= 16;
        seen.lam >>= 16;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            pw[c] = pack_bf16(x[2 * c], x[2 * c + 1]);
            pg[c] = pack_bf16(d[2 * c], d[2 * c + 1]);
            if constexpr (REST) rest[c] = pack_rest(pg[c], d[2 * c], d[2 * c + 1]);
        }
        if constexpr (REST) tmem_st8((COLS ? s_addr : d_addr) + 16 * ch, rest);
        if constexpr (COLS) tmem_st8(d_addr + 16 * ch, pw);
        tmem_st8(d_addr + 16 * ch + 8, pg);
    }
}

// The sums of P and P dP of a thread's 32 columns under each mask.
struct RowSums {
    float lc, dc, ls, ds;
};
template <int CAP, bool MASKED, bool POLY>
__device__ __forceinline__ void sums_loop(RowSums& sum, const float (&x)[kCols], const LayerArgs& a, float sl, const TanhPoly& tp,
                                          float nlse_c, float nlse_s, const Seen& seen, uint32_t d_addr) {
    const float f = CAP == NO_CAP ? sl : POLY ? a.cap.c2 : 1.f;   // t below times f is the score
    float2 lc = make_float2(0.f, 0.f), dc = lc;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float d[16];
        tmem_ld16(d_addr + 16 * h, d);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const int c = 16 * h + i;
            float2 t = make_float2(x[c], x[c + 1]);
            if constexpr (CAP != NO_CAP) {
                constexpr bool far = CAP == CAP_FAR;
                t = POLY ? poly_fma2(t, tp) : make_float2(score_log2<true, far>(t.x, sl, a.cap), score_log2<true, far>(t.y, sl, a.cap));
            }
            float2 v = ffma2(t, make_float2(f, f), make_float2(nlse_c, nlse_c));
            if constexpr (MASKED) {
                // both attentions: the score once more, relative to lse_s
                const float p0 = (seen.lam >> c) & 1u ? sfu_exp2(fmaf(t.x, f, nlse_s)) : 0.f;
                const float p1 = (seen.lam >> (c + 1)) & 1u ? sfu_exp2(fmaf(t.y, f, nlse_s)) : 0.f;
                sum.ls += p0 + p1;
                sum.ds = fmaf(p0, d[i], fmaf(p1, d[i + 1], sum.ds));
                v.x = (seen.causal >> c) & 1u ? v.x : -INFINITY;
                v.y = (seen.causal >> (c + 1)) & 1u ? v.y : -INFINITY;
            }
            v = make_float2(sfu_exp2(v.x), sfu_exp2(v.y));
            lc = fadd2(lc, v);
            dc = ffma2(v, make_float2(d[i], d[i + 1]), dc);
        }
    }
    sum.lc += lc.x + lc.y;
    sum.dc += dc.x + dc.y;
}
template <int CAP, bool MASKED>
__device__ __forceinline__ void add_sums(RowSums& sum, const LayerArgs& a, float sl, const TanhPoly& tp, float nlse_c, float nlse_s,
                                         const Seen& seen, uint32_t s_addr, uint32_t d_addr) {
    float x[kCols];
    tmem_ld32(s_addr, x);
    if (CAP == NO_CAP || (CAP == CAPPED && __all_sync(0xffffffffu, largest<kCols>(x) <= tp.x_max)))
        sums_loop<CAP, MASKED, true>(sum, x, a, sl, tp, nlse_c, nlse_s, seen, d_addr);
    else
        sums_loop<CAP, MASKED, false>(sum, x, a, sl, tp, nlse_c, nlse_s, seen, d_addr);
}

// TMEM columns of S(j) and dP(j).
template <int MODE>
__device__ __forceinline__ uint32_t s_col(int j) { return !keys_outer(MODE) && (j & 1) ? kColA1 : kColS; }
template <int MODE>
__device__ __forceinline__ uint32_t d_col(int j) { return MODE == STATS && (j & 1) ? kColA2 : kColP; }

template <int MODE, int CAP, bool REST>
__global__ void __launch_bounds__(kRegThreads, 1)
    mix_grad_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDo,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const GradArgs p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr bool kKeys = keys_outer(MODE), kStats = MODE == STATS, kPairs = MODE == KEY_PAIRS;
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
    uint64_t* s_full = bars + 5;    // [2], by the tile's parity, as the next three
    uint64_t* d_full = bars + 7;
    uint64_t* w_ready = bars + 9;   // S read (statistics: dP too)
    uint64_t* g_ready = bars + 11;  // W and dS written
    uint64_t* done = bars + 13;
    uint32_t* holder = reinterpret_cast<uint32_t*>(smem + kOffHolder);

    // Work item, the longest first.  Keys outer: key tile ot of KV head `head`,
    // whose inner tiles are (query head of the group, query tile >= ot);
    // queries outer: query tile ot of query head `head`, key tiles 0 .. ot.
    // Pairs: a cluster of two CTAs takes an item, half of its inner tiles each.
    const int heads = kKeys ? a.Hkv : a.Hq;
    const int item = kPairs ? blockIdx.x >> 1 : blockIdx.x, part = kPairs ? blockIdx.x & 1 : 0;
    const int ord = item / (a.B * heads), rest = item % (a.B * heads);
    const int head = rest % heads, b = rest / heads;
    const int ot = kKeys ? ord : p.n_tiles - 1 - ord;
    const int kv = kKeys ? head : head / a.G;
    const int per_head = p.n_tiles - ot;                   // keys outer: query tiles per query head
    const int n_all = kKeys ? a.G * per_head : ot + 1;
    const int j_first = part * ((n_all + 1) / 2);          // this CTA's: j_first .. j_first + n_in - 1, none if n_all is 1
    const int n_in = !kPairs ? n_all : part ? n_all / 2 : (n_all + 1) / 2;
    auto inner_tile = [&](int j) { return kKeys ? ot + (j_first + j) % per_head : j; };
    auto inner_qhead = [&](int j) { return kKeys ? kv * a.G + (j_first + j) / per_head : head; };

    if (warp == kMmaWarp) tmem_alloc(holder, kTmemCols);
    if (tid == 0) {
        mbar_init(x_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&y_full[i], 1);
            // the MMAs' commit, and the warps that read the stage's statistics
            mbar_init(&y_empty[i], kKeys ? 1 + kElemWarps : 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&d_full[i], 1);
            mbar_init(&w_ready[i], kElemWarps);
            mbar_init(&g_ready[i], kElemWarps);
        }
        mbar_init(done, 1);
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;

    bool ok = n_in > 0;   // element-wise warps: the accumulators are complete
    if (warp == kTmaWarp) {
        if (lane == 0 && n_in > 0) {
            const CUtensorMap* mx0 = kKeys ? &tmK : &tmQ;
            const CUtensorMap* mx1 = kKeys ? &tmV : &tmDo;
            const CUtensorMap* my0 = kKeys ? &tmQ : &tmK;
            const CUtensorMap* my1 = kKeys ? &tmDo : &tmV;
            mbar_arrive_expect_tx(x_full, 2 * kTileBytes);
            for (int half = 0; half < 2; ++half) {
                tma_load_4d(sX + half * kHalfBytes, mx0, 64 * half, head, BM * ot, b, x_full);
                tma_load_4d(sX + kTileBytes + half * kHalfBytes, mx1, 64 * half, head, BM * ot, b, x_full);
            }
            for (int j = 0; j < n_in; ++j) {
                const int st = j & 1, it = inner_tile(j), ih = kKeys ? inner_qhead(j) : kv;
                if (j >= 2 && !mbar_wait(&y_empty[st], ((j >> 1) - 1) & 1, p.status)) break;
                mbar_arrive_expect_tx(&y_full[st], 2 * kTileBytes + (kKeys ? kStatBytes : 0u));
                const uint32_t y = sY + st * 2 * kTileBytes;
                for (int half = 0; half < 2; ++half) {
                    tma_load_4d(y + half * kHalfBytes, my0, 64 * half, ih, BM * it, b, &y_full[st]);
                    tma_load_4d(y + kTileBytes + half * kHalfBytes, my1, 64 * half, ih, BM * it, b, &y_full[st]);
                }
                if constexpr (kKeys) {
                    const float* src = p.stats + ((size_t)b * a.Hq + ih) * 4 * p.n_pad + BM * it;
                    for (int r = 0; r < 4; ++r)
                        bulk_g2s(smem + kOffStat + st * kStatBytes + r * BM * 4, src + (size_t)r * p.n_pad, BM * 4,
                                 &y_full[st]);
                }
            }
        }
    } else if (warp == kMmaWarp) {
        {
            // the whole warp waits, one lane issues (every call of the
            // lambdas below is under elect_one)
            constexpr uint32_t idesc_kk = idesc_bf16(BM, BM, 0, 0);
            constexpr uint32_t idesc_mn = idesc_bf16(BM, HD, 0, 1);
            // D = X_w Y_w(j)^T over d
            auto issue_xy = [&](uint32_t col, int w, int j) {
                const uint64_t x = sw128_desc(sX + w * kTileBytes, 16, 1024);
                const uint64_t y = sw128_desc(sY + ((j & 1) * 2 + w) * kTileBytes, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t o = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
                    tc_mma(tmem + col, x + o, y + o, idesc_kk, kk > 0 ? 1u : 0u);
                }
            };
            // ACC += A (W, dS or its rest, 8 of every 16 columns of dP's or S's) Y_w(j), over the inner rows
            auto issue_acc = [&](uint32_t col, uint32_t a_col, int w, int j, bool first = true) {
                const uint64_t y = sw128_desc(sY + ((j & 1) * 2 + w) * kTileBytes, kHalfBytes, 1024);
#pragma unroll
                for (int kk = 0; kk < BM / 16; ++kk)
                    tc_mma_ta(tmem + col, tmem + a_col + kChunk * kk, y + kk * (2048 >> 4), idesc_mn,
                              (!first || j > 0 || kk > 0) ? 1u : 0u);
            };
            auto wait_tile = [&](int j) { return mbar_wait(&y_full[j & 1], (j >> 1) & 1, p.status); };
            auto issue_s = [&](int j) {
                issue_xy(s_col<MODE>(j), 0, j);
                tc_commit(&s_full[j & 1]);
            };
            auto issue_d = [&](int j) {
                issue_xy(d_col<MODE>(j), 1, j);
                tc_commit(&d_full[j & 1]);
            };
            ok = ok && mbar_wait(x_full, 0, p.status) && wait_tile(0);
            if (ok) {
                tc_fence_after();
                if (elect_one()) {
                    issue_s(0);
                    issue_d(0);
                    if (kStats) tc_commit(&y_empty[0]);
                }
            }
            if (!kKeys && n_in > 1 && ok) {
                ok = wait_tile(1);
                if (ok) {
                    tc_fence_after();
                    if (elect_one()) {
                        issue_s(1);
                        if (kStats) {
                            issue_d(1);
                            tc_commit(&y_empty[1]);
                        }
                    }
                }
            }
            for (int j = 0; j < n_in && ok; ++j) {
                const int ph = (j >> 1) & 1;
                if constexpr (kStats) {
                    // both slots run ahead: tile j + 2 once tile j is read
                    ok = mbar_wait(&w_ready[j & 1], ph, p.status);
                    if (ok && j + 2 < n_in) {
                        ok = wait_tile(j + 2);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            issue_s(j + 2);
                            issue_d(j + 2);
                            tc_commit(&y_empty[j & 1]);
                        }
                    }
                } else {
                    const bool next = j + 1 < n_in;
                    if (kKeys && next && !REST) {
                        // S(j) is in registers: its columns take S(j + 1)
                        ok = wait_tile(j + 1) && mbar_wait(&w_ready[j & 1], ph, p.status);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) issue_s(j + 1);
                    }
                    ok = mbar_wait(&g_ready[j & 1], ph, p.status);
                    if (REST && kKeys && next) ok = ok && wait_tile(j + 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        if (kKeys) issue_acc(kColA1, kColP, 1, j);
                        issue_acc(kColA2, kColP + kChunk / 2, 0, j);
                        if (REST) issue_acc(kColA2, kKeys ? kColS : kColP, 0, j, false);
                        tc_commit(&y_empty[j & 1]);
                        if (REST && kKeys && next) issue_s(j + 1);   // S's columns held the rest until here
                        if (next) issue_d(j + 1);
                    }
                    if (!kKeys && j + 2 < n_in) {
                        // one S ahead: its slot was read before dS(j) was written
                        ok = mbar_wait(&w_ready[j & 1], ph, p.status) && wait_tile(j + 2);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) issue_s(j + 2);
                    }
                }
            }
            if (ok && elect_one()) tc_commit(done);
        }
        __syncwarp();
    } else if (warp < kElemWarps) {
        // ------------------------------------------------ element-wise warps
        const int wg = warp >> 2;                             // columns 32 wg ..
        const int row = 32 * (warp & 3) + lane;               // TMEM lane: outer row
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const float sl = a.scale * kLog2e;
        const float al = p.alpha[kv];
        const bool neg_c = al < 0.f, neg_s = 1.f - al < 0.f;
        const TanhPoly& tp = p.poly;
        const int orow = BM * ot + row;                       // key (keys outer) or query
        RowStats rs{0.f, 0.f, 0.f, 0.f, nullptr};
        RowSums sum{0.f, 0.f, 0.f, 0.f};
        // statistics: both masks show the query the same keys, so the two attentions
        // are one: the same log-sum and D, and no share of dalpha but 0
        const bool one_attention = orow < a.sink + a.recent;
        if constexpr (kStats) {
            const bool live = orow < p.N;
            const size_t r = ((size_t)b * a.Hq + head) * p.N + (live ? orow : 0);
            rs.lse_c = live ? -p.lse[r] : -INFINITY;
            rs.lse_l = live ? -p.lse[(one_attention ? 0 : (size_t)a.B * a.Hq * p.N) + r] : -INFINITY;
        } else if constexpr (!kKeys) {
            const float* st = p.stats + ((size_t)b * a.Hq + head) * 4 * p.n_pad + orow;
            rs = {st[0], st[p.n_pad], st[2 * (size_t)p.n_pad], st[3 * (size_t)p.n_pad], nullptr};
        }
        int it = inner_tile(0) - 1;                           // inner_tile(j), step by step
        for (int j = 0; j < n_in; ++j) {
            it = it + 1 < p.n_tiles || !kKeys ? it + 1 : ot;
            const int ph = (j >> 1) & 1;
            const uint32_t s_addr = lane_addr + s_col<MODE>(j) + kCols * wg, d_addr = lane_addr + d_col<MODE>(j) + kCols * wg;
            if constexpr (kKeys) {
                rs.cols = reinterpret_cast<const float*>(smem + kOffStat + (j & 1) * kStatBytes) + kCols * wg;
                // the statistics arrived with the tile that S(j) was computed from;
                // this wait makes the copy visible to this thread too
                ok = ok && mbar_wait(&y_full[j & 1], ph, p.status);
            }
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&s_full[j & 1], ph, p.status));
            if (!ok) break;
            tc_fence_after();
            // every pair of the warp's part is seen by the causal attention only?
            const int r0 = BM * ot + 32 * (warp & 3), c0 = BM * it + kCols * wg;
            const int key0 = kKeys ? r0 : c0, key1 = kKeys ? r0 + 31 : c0 + kCols - 1, query0 = kKeys ? c0 : r0;
            const bool plain = key0 >= a.sink && query0 - key1 >= a.recent;   // recent >= 1: below the diagonal too
            Seen seen{};
            if (!plain) seen = seen_columns(a, kKeys, orow, c0);
            if constexpr (kStats) {
                ok = __all_sync(0xffffffffu, mbar_wait(&d_full[j & 1], ph, p.status));
                if (!ok) break;
                tc_fence_after();
                if (plain)
                    add_sums<CAP, false>(sum, a, sl, tp, rs.lse_c, rs.lse_l, seen, s_addr, d_addr);
                else
                    add_sums<CAP, true>(sum, a, sl, tp, rs.lse_c, rs.lse_l, seen, s_addr, d_addr);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&w_ready[j & 1]);
                continue;
            } else if (plain || !(neg_c || neg_s)) {
                float x[kCols];
                uint32_t pk[kCols / 2];
                tmem_ld32(s_addr, x);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&w_ready[j & 1]);
                if (plain)
                    weights<CAP, kKeys, false>(x, pk, a, sl, tp, rs, seen);
                else
                    weights<CAP, kKeys, true>(x, pk, a, sl, tp, rs, seen);
                ok = __all_sync(0xffffffffu, mbar_wait(&d_full[j & 1], ph, p.status));
                if (!ok) break;
                tc_fence_after();
                if (plain)
                    score_grads<kKeys, false, REST>(x, pk, rs, seen, s_addr, d_addr);
                else
                    score_grads<kKeys, true, REST>(x, pk, rs, seen, s_addr, d_addr);
            } else {
                ok = __all_sync(0xffffffffu, mbar_wait(&d_full[j & 1], ph, p.status));
                if (!ok) break;
                tc_fence_after();
                signed_shares<CAP, kKeys, REST>(a, sl, rs, seen, s_addr, d_addr);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&w_ready[j & 1]);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&g_ready[j & 1]);
                if constexpr (kKeys) mbar_arrive(&y_empty[j & 1]);   // done with the stage's statistics
            }
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait(done, 0, p.status));
        if constexpr (kStats) {
            // join the four quarters of each row, then the row's statistics
            float4* quarter = reinterpret_cast<float4*>(smem + kOffY);   // [3][128]; every tile has been read
            float* share = reinterpret_cast<float*>(quarter + 3 * BM);   // [4] of the warps
            if (wg > 0) quarter[(wg - 1) * BM + row] = make_float4(sum.lc, sum.dc, sum.ls, sum.ds);
            asm volatile("bar.sync 1, 512;" ::: "memory");
            if (wg == 0) {
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const float4 t = quarter[k * BM + row];
                    o = make_float4(o.x + t.x, o.y + t.y, o.z + t.z, o.w + t.w);
                }
                const float lc = sum.lc + o.x, ls = one_attention ? lc : sum.ls + o.z;
                const bool live = ok && orow < p.N && lc > 0.f && ls > 0.f;
                const float dc = live ? (sum.dc + o.y) / lc : 0.f;
                const float ds = !live ? 0.f : one_attention ? dc : (sum.ds + o.w) / ls;
                const float lse_c = live ? log2f(lc) - rs.lse_c - log2f(fabsf(al)) : INFINITY;       // +inf: a closed gate
                const float lse_s = live ? log2f(ls) - rs.lse_l - log2f(fabsf(1.f - al)) : INFINITY;
                float lse_l = lse_s, dl = ds;
                if (!(neg_c || neg_s) && live) {
                    // 2^-lse* = 2^-lse_c + 2^-lse_s, the two shares' weights
                    const float lo = fminf(lse_c, lse_s);
                    const float wc = exp2f(lo - lse_c), ws = exp2f(lo - lse_s);
                    lse_l = lo - log2f(wc + ws);
                    dl = (wc * dc + ws * ds) / (wc + ws);
                }
                float* st = p.stats + ((size_t)b * a.Hq + head) * 4 * p.n_pad + orow;
                if (bounds_ok(orow < p.n_pad, p.status)) {
                    st[0] = -lse_c;
                    st[p.n_pad] = -dc;
                    st[2 * (size_t)p.n_pad] = -lse_l;
                    st[3 * (size_t)p.n_pad] = -dl;
                }
                float d = dc - ds;
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
                if (lane == 0) share[warp] = d;
                asm volatile("bar.sync 2, 128;" ::: "memory");
                if (tid == 0)
                    p.part[(((size_t)kv * a.B + b) * p.n_tiles + ot) * a.G + head % a.G] =
                        (share[0] + share[1]) + (share[2] + share[3]);
            }
        }
        // one warp per KV head adds up the shares of dalpha, in their order
        if (kKeys && ot == 0 && b == 0 && part == 0 && warp == 0) {
            const int n = a.B * p.n_tiles * a.G;
            sum_shares(p.part + (size_t)kv * n, n, &p.dalpha[kv], lane);
        }
    }
    if constexpr (!kStats) {
        // Pairs: each CTA hands one accumulator to the other, over the tiles that are
        // done with (64 KB, [column][row]), and stores the sum of the other
        // accumulator: the first dK, the second dV.
        const int wg = warp >> 2, row = 32 * (warp & 3) + lane;
        const bool elem = warp < kElemWarps;
        const uint32_t acc = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kCols * wg;
        const uint32_t slot = (uint32_t)((kCols * wg * BM + row) * 4);
        auto take = [&](uint32_t col, float (&v)[kCols]) {
            if (ok) {
                tc_fence_after();
                tmem_ld32(acc + col, v);
            } else {
#pragma unroll
                for (int i = 0; i < kCols; ++i) v[i] = 0.f;
            }
        };
        float v[kCols];
        if constexpr (kPairs) {
            __syncwarp();
            cluster_sync();
            if (elem) {
                take(part ? kColA2 : kColA1, v);
                const uint32_t to = peer_smem(sY, part ^ 1) + slot;
#pragma unroll
                for (int i = 0; i < kCols; ++i) st_peer(to + i * BM * 4, v[i]);
            }
            __syncwarp();
            cluster_sync();
        }
        if (elem) {
            const int orow = BM * ot + row;
            const bool live = orow < p.N && (kPairs || ok) && bounds_ok(b < a.B && head < heads, p.status);
            const size_t off = (((size_t)b * p.N + orow) * heads + head) * HD + kCols * wg;
            const float sign = p.alpha[kv] < 0.f ? -1.f : 1.f;   // a negative gate's sums are negated
#pragma unroll
            for (int t = kPairs ? part : 0; t < (kPairs ? part + 1 : kKeys ? 2 : 1); ++t) {
                take(t ? kColA1 : kColA2, v);
                if constexpr (kPairs) {
                    const float* peer = reinterpret_cast<const float*>(smem + kOffY + slot);
#pragma unroll
                    for (int i = 0; i < kCols; ++i) v[i] += peer[i * BM];
                }
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(t ? p.d1 : p.d0) + off;
                const float f = (t ? 1.f : CAP != NO_CAP ? -a.scale : a.scale) * sign;   // dS held back the softmax scale
#pragma unroll
                for (int e = 0; e < kCols / 8; ++e) {
                    float v8[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v8[i] = v[8 * e + i] * f;
                    if (live) store_row<__nv_bfloat16, 8>(o + 8 * e, v8);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int MODE, int CAP, bool REST>
cudaError_t launch_cap(const CUtensorMap (&m)[4], const GradArgs& p, cudaStream_t s) {
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = smem_limit_once(mix_grad_kernel<MODE, CAP, REST>, (int)kGradSmem, configured);
    if (e != cudaSuccess) return e;
    const long grid = (long)p.a.B * (keys_outer(MODE) ? p.a.Hkv : p.a.Hq) * p.n_tiles * (MODE == KEY_PAIRS ? 2 : 1);
    if (grid > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kGradThreads);
    cfg.dynamicSmemBytes = kGradSmem;
    cfg.stream = s;
    cudaLaunchAttribute cluster{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = MODE == KEY_PAIRS ? 2 : 1;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cfg.attrs = &cluster;
    cfg.numAttrs = MODE == KEY_PAIRS ? 1 : 0;
    const cudaError_t launched = cudaLaunchKernelEx(&cfg, mix_grad_kernel<MODE, CAP, REST>, m[0], m[1], m[2], m[3], p);
    return launched != cudaSuccess ? launched : cudaGetLastError();
}

template <int MODE, bool REST>
cudaError_t launch_grad(const CUtensorMap (&m)[4], const GradArgs& p, cudaStream_t s) {
    const CapArgs& cap = p.a.cap;
    return !cap.on    ? launch_cap<MODE, NO_CAP, REST>(m, p, s)
           : !cap.far ? launch_cap<MODE, CAPPED, REST>(m, p, s)
                      : launch_cap<MODE, CAP_FAR, REST>(m, p, s);
}

// Two CTAs to a key tile where the first, seen by every query of its group,
// would take one CTA longer than an SM's share of all tiles: a whole step of
// 4,096 tokens and 32 + 8 heads 900 -> 879 us, of 1,000 tokens 169 -> 140; with
// 32 + 32 heads at 4,096, below the rule, pairs lose (923 -> 1,004: the pair's
// exchange and its second load of K and V).
bool share_key_tiles(const LayerArgs& a, int n_tiles) {
    const long all = (long)a.B * a.Hkv * n_tiles * (n_tiles + 1) / 2;   // in tiles of one query head, as the next
    return a.G * n_tiles > 1 && (long)n_tiles * sm_count() > all;       // (one inner tile is not halved)
}

// dS as two bf16 operands, its value and what the rounding took off, where a
// sequence is one tile: with few keys a row's gradient is a term or two, whose
// rounding shows (dq and dk of up to 128 tokens were 1.2 to 1.7 times as far from
// fp64 as their own rounding, and now are 1.00 times), and the step is mostly
// launch latency: 43 to 55 us, 2 to 6 more with 4 or 8 query heads to a KV head,
// none with one.  Over many tiles it would cost a product of nine, and S(j + 1)
// its place beside dP(j) (the rest of dK's dS waits in S's columns).
bool keep_rest(int n_tiles) { return n_tiles == 1; }

}  // namespace

MixGradPlan mix_grad_plan(const LayerArgs& a, int N) {
    MixGradPlan pl{};
    pl.n_tiles = (N + BM - 1) / BM;
    pl.n_pad = pl.n_tiles * BM;
    const size_t stats = (size_t)a.B * a.Hq * 4 * pl.n_pad * sizeof(float);
    pl.part_offset = (stats + 255) / 256 * 256;
    // a share per query head and 128 rows (here), or per KV head and 32 rows (tiled_attn.cu)
    const size_t shares = (size_t)a.B * pl.n_tiles * (a.Hq > 4 * a.Hkv ? a.Hq : 4 * a.Hkv);
    pl.bytes = pl.part_offset + (shares * sizeof(float) + 255) / 256 * 256;
    return pl;
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
    GradArgs p{a, N, pl.n_tiles, pl.n_pad, g.stats, g.lse, g.alpha, nullptr, nullptr, g.part, g.dalpha, g.status, tanh_poly(a.cap, 1.f)};
    cudaError_t e = launch_grad<STATS, false>(m, p, s);
    if (e != cudaSuccess) return e;
    p.d0 = g.dk;
    p.d1 = g.dv;
    const bool rest = keep_rest(pl.n_tiles);
    if (share_key_tiles(a, pl.n_tiles))
        e = rest ? launch_grad<KEY_PAIRS, true>(m, p, s) : launch_grad<KEY_PAIRS, false>(m, p, s);
    else
        e = rest ? launch_grad<KEYS, true>(m, p, s) : launch_grad<KEYS, false>(m, p, s);
    if (e != cudaSuccess) return e;
    p.d0 = g.dq;
    p.d1 = nullptr;
    return rest ? launch_grad<QUERIES, true>(m, p, s) : launch_grad<QUERIES, false>(m, p, s);
}

}  // namespace duo
