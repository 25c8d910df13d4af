// prefill_capped.cu -- the tensor-core attention of prefill_tc.cu for scores
// capped by a tanh, where the cap bounds them: the capped pre-fill and the
// gated mix's training forward pass.
//
// A capped score lies in [-cap, cap], so the softmax needs no running maximum:
// with x the dot product, p = 2^(c2 tanh(k x)) lies in [2^-c2, 2^c2], which for
// caps up to 60 (c2 <= 87) stays inside fp32 -- and bf16, whose exponent is the
// same -- with room for the row sum of 2^40 keys.  p is then a function of one
// score alone.  No row statistic stands between the scores and the
// exponentials, O is never rescaled, the columns of a row may be split over
// several threads that never talk until the end, and the splits of a key range
// merge by addition.  (Larger caps, and caches of 8- or 4-bit codes, whose fp16
// p needs the maximum, take prefill_tc.cu.)
//
// O = P V is the one sum whose range depends on more than the cap: with scores
// near +cap, values past 2^40 or so could overflow it, and in a row whose every
// score lies near -cap small values would fall below fp32's normal range.  So a
// CTA looks at its rows as it stores them, and where a result is not finite (a
// split's, to be added to others: past 2^100), or a row sum is below 2^-32 and O
// below 2^-90 (where products lost to the flush could count), it walks its tiles
// once more (second_pass) with p = 2^(score - log2(2 l)), l the row's own sum, which is
// always in range: those weights add up to 1/2, whatever the scores.  Scores
// and values of a model never ask for it; that it can be asked for costs the
// pre-fill of a 4,096-token chunk 0.9 % of its time.
//
// Work and masks as in prefill_tc.cu (prefill_sched.cuh), but a CTA owns one
// 128-row query tile: S then has three buffers in TMEM (S0 | S1 | S2 | O, 128
// columns each), the tensor core runs up to three Q K^T ahead, and a warp's
// exponentials wait for no MMA.  (With two query tiles to a CTA and one S
// each, a warp spent 1,850 of 4,650 cycles of a tile pair waiting for P V and
// the next Q K^T; the price, K and V read once per 128 queries instead of
// 256, is L2 traffic, 6 TB/s.)
// Roles (608 threads): warps 0-15 the exponentials, in two groups of eight
// that take alternate key tiles (warp w of a group: lanes 32 (w % 4) .., columns
// 64 (w / 4) ..), warp 16 TMA (K and V three tiles deep), warps 17 and 18 the
// MMAs of Q K^T and of P V: one issuing warp's waits and instructions took
// 1,850 cycles a tile, two run side by side.
// Each warp takes 32 columns at a time from TMEM: tanh on the FMA pipe, the
// exponential on the SFU, p packed as bf16 over the columns it came from.  The
// polynomial's range (cap.cuh) is checked after the fact by a vote over the
// largest x^2; a part outside takes its scores from TMEM again and tanh on the
// SFU.  The row sum adds the rounded p, so that an output is a convex
// combination of V rows.
// The gated mix (MIX) computes both attentions at once: p is the same under
// both masks, so a tile with sink or recent keys writes p twice, once for the
// causal mask and once for the Lambda mask, side by side in the columns of its
// scores, and P V runs once into each of two accumulators (S0 | S1 | Os | Oc;
// two S tiles in flight).  A separate pass over the Lambda tiles took 70 us of
// 253 for 4,096 tokens and 32 heads.
#include <cuda.h>

#include "cap.cuh"
#include "common.cuh"
#include "internal.h"
#include "prefill_sched.cuh"
#include "tcgen05.cuh"

namespace duo {
namespace {

constexpr int kExpWarps = 16, kTmaWarp = 16, kQkWarp = 17, kPvWarp = 18, kThreads = 608;
constexpr int kRegThreads = 640;                   // five warps to a sub-partition: 96 registers
constexpr int kStages = 3;                         // K and V tiles in shared memory
template <bool MIX>
__device__ __forceinline__ constexpr int s_slots() { return MIX ? 2 : 3; }   // S tiles in TMEM
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 384, kColOs = 256;      // Os: the Lambda attention (MIX)
constexpr uint32_t kTileBytes = BN * HD * 2;       // 32 KB per Q, K or V tile (two 16 KB halves of d)
constexpr uint32_t kHalfBytes = kTileBytes / 2;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + kTileBytes;
constexpr uint32_t kOffV = kOffK + kStages * kTileBytes;
constexpr uint32_t kOffSum = kOffV + kStages * kTileBytes;   // [4][128] partial row sums
constexpr uint32_t kOffBar = kOffSum + 4 * BM * 4;
constexpr uint32_t kOffHolder = kOffBar + 24 * 8;  // TMEM base, last split, a row asks for a second pass, a wait ran out
constexpr uint32_t kSmemBytes = kOffHolder + 16;
constexpr uint32_t kOffSums2 = kOffK;              // a second pass's (l, l of the Lambda attention) by row
constexpr float kMaxO = 0x1p100f, kMinSum = 0x1p-32f, kMinO = 0x1p-90f;   // of a first pass: a split's |O|; a row's sum with its |O|
static_assert(kSmemBytes <= 232448, "one CTA per SM");

// The key tiles of query tile mt (chunk rows 128 mt ..), as make_sched lists
// them for a pair; tile_at and visible_columns take the result.
__device__ __forceinline__ Sched make_sched_single(const TcArgs& p, bool retrieval, int c0, int mt) {
    const LayerArgs& a = p.a;
    Sched s;
    s.retrieval = retrieval;
    s.chunk = !retrieval && a.stream_chunk;
    s.c0 = c0;
    s.m = mt;
    const int hi = min(mt, (p.C + BN - 1) / BN - 1);      // the diagonal's tile
    s.n_prior = retrieval ? (c0 + BN - 1) / BN : 0;
    s.n_ring = !retrieval && min(c0, a.W) > 0 ? 1 : 0;
    s.lo = 0;
    s.sink_tile = 0;
    if (!retrieval && !s.chunk) {
        s.lo = max(0, BM * mt - a.recent + 1) / BN;       // first key of the band
        s.sink_tile = (c0 < a.sink && s.lo > 0) ? 1 : 0;  // the chunk's own sink tokens (sink <= 128)
    }
    s.n = s.n_prior + s.n_ring + s.sink_tile + (hi - s.lo + 1);
    s.n0 = s.n;
    return s;
}
// Tiles first .. last - 1 of the list need no mask: all but the tile that
// starts before position 0, the ring and the diagonal's (Lambda mode: none).
__device__ __forceinline__ void unmasked_tiles(const Sched& s, int& first, int& last) {
    first = s.retrieval ? (s.c0 % BN != 0 ? 1 : 0) : s.n_ring;
    last = s.retrieval || s.chunk ? s.n - 1 : 0;
}

// 32 columns of a row: dot products x -> p, packed as bf16 in pk; returns the
// sum of the rounded p.  POLY: tanh by its polynomial, `big` raised to the
// largest x^2; else on the SFU.  One loop from the dot product to the packed
// p, so that the FMA, SFU and ALU work of neighbouring pairs interleaves.
// LAM: the sum in .y and the packed pairs in pk[16 ..] are those of the columns
// in `lam` (a subset of vis).
template <bool MASKED, bool LAM, bool POLY>
__device__ __forceinline__ float2 exp_loop(const float (&x)[32], uint32_t (&pk)[LAM ? 32 : 16], const CapArgs& cap,
                                           const TanhPoly& tp, uint32_t vis, uint32_t lam, float& big) {
    float2 sum = make_float2(0.f, 0.f), sum_l = sum;
    big = 0.f;
#pragma unroll
    for (int c2 = 0; c2 < 16; ++c2) {
        float2 v = make_float2(x[2 * c2], x[2 * c2 + 1]);
        if constexpr (POLY) {
            const float2 u = fmul2(v, v);
            big = fmax3(big, u.x, u.y);
            v = poly_fma2(v, u, tp);
        } else {
            v = make_float2(score_log2<true, false>(v.x, cap.sl, cap), score_log2<true, false>(v.y, cap.sl, cap));
        }
        float2 e = make_float2(sfu_exp2(v.x), sfu_exp2(v.y));
        if constexpr (MASKED) {
            e.x = (vis >> (2 * c2)) & 1u ? e.x : 0.f;
            e.y = (vis >> (2 * c2 + 1)) & 1u ? e.y : 0.f;
        }
        __nv_bfloat162 h = __floats2bfloat162_rn(e.x, e.y);
        pk[c2] = *reinterpret_cast<uint32_t*>(&h);
        sum = fadd2(sum, make_float2(bf16_lo(pk[c2]), bf16_hi(pk[c2])));
        if constexpr (LAM) {
            pk[16 + c2] = ((lam >> (2 * c2)) & 1u ? pk[c2] & 0xffffu : 0u) |
                          ((lam >> (2 * c2 + 1)) & 1u ? pk[c2] & 0xffff0000u : 0u);
            sum_l = fadd2(sum_l, make_float2(bf16_lo(pk[16 + c2]), bf16_hi(pk[16 + c2])));
        }
    }
    return make_float2(sum.x + sum.y, sum_l.x + sum_l.y);
}

// 64 columns of a row: dot products at s_addr -> p over the first half of every
// 32, and (LAM) p under the Lambda mask over the second half; the row's sums
// are added to l.
template <bool MASKED, bool LAM>
__device__ __forceinline__ void exp_columns(float2& l, uint32_t s_addr, const CapArgs& cap, const TanhPoly& tp,
                                            uint64_t vis, uint64_t lam) {
#pragma unroll 1
    for (int ch = 0; ch < 2; ++ch) {
        float x[32], big;
        tmem_ld32(s_addr + 32 * ch, x);
        uint32_t pk[LAM ? 32 : 16];
        float2 t = exp_loop<MASKED, LAM, true>(x, pk, cap, tp, (uint32_t)vis, (uint32_t)lam, big);
        if (!__all_sync(0xffffffffu, big <= tp.x2_max)) {
            tmem_ld32(s_addr + 32 * ch, x);
            t = exp_loop<MASKED, LAM, false>(x, pk, cap, tp, (uint32_t)vis, (uint32_t)lam, big);
        }
        l = fadd2(l, t);
        vis >>= 32;
        lam >>= 32;
        if constexpr (LAM)
            tmem_st32(s_addr + 32 * ch, pk);
        else
            tmem_st16(s_addr + 32 * ch, pk);
    }
}

// MIX (whole sequences, no cache: tile j holds keys 128 j ..): does query tile
// mt see keys of tile j in the Lambda attention?
__device__ __forceinline__ bool lambda_tile(const LayerArgs& a, int mt, int j) {
    return j * BN < a.sink || (mt - j) * BM - (BN - 1) < a.recent;
}

__device__ __forceinline__ uint64_t half_bits(const uint32_t (&v)[4], int half) {
    return half ? ((uint64_t)v[3] << 32 | v[2]) : ((uint64_t)v[1] << 32 | v[0]);
}

// A CTA's work item, ordered as in prefill_tc.cu: (sequence, KV head) outermost,
// then the split, then the query tile (heaviest first) and the query head.
struct Work {
    Sched sc;
    bool retrieval;
    int unit, split, ns_use;           // of the pair of query tiles: records and tickets are laid out by pairs
    int mt, b, slot, q_idx, kv_idx;
    int j0, j1;                        // tiles of the schedule; none: nothing to do
};
__device__ __forceinline__ Work work_item(const TcArgs& p) {
    const LayerArgs& a = p.a;
    Work w;
    w.retrieval = (int)blockIdx.x < 2 * p.n_ret_ctas;
    const int n_mt = 2 * p.n_mpairs;                  // the last may lie past the chunk
    w.unit = w.split = 0;
    int g, hs;
    if (w.retrieval) {
        const int per_group = n_mt * a.G;
        const int r = (int)blockIdx.x;
        const int inner = r % per_group;
        w.split = (r / per_group) % p.ns;
        const int bh = r / (per_group * p.ns);
        g = inner % a.G;
        w.mt = n_mt - 1 - inner / a.G;
        hs = bh % a.R;
        w.b = bh / a.R;
        w.unit = (bh * p.n_mpairs + w.mt / 2) * a.G + g;
    } else {
        int idx = (int)blockIdx.x - 2 * p.n_ret_ctas;
        const int per_m = a.B * a.S * a.G;
        w.mt = n_mt - 1 - idx / per_m;
        idx %= per_m;
        g = idx % a.G;
        hs = (idx / a.G) % a.S;
        w.b = idx / (a.G * a.S);
    }
    w.slot = w.retrieval ? hs : a.R + hs;
    w.q_idx = a.q_head0[w.slot] + g;
    w.kv_idx = a.kv_head[w.slot];
    int c0 = p.seq_len ? p.seq_len[w.b] : 0;          // no lengths: whole sequences, no cache
    if (c0 < 0) c0 = 0;
    if (w.retrieval && c0 > a.capacity) {
        if (threadIdx.x == 0 && w.mt == 0 && p.status) atomicOr(p.status, DUO_DEV_BAD_LENGTH);
        c0 = a.capacity;
    }
    w.ns_use = 1;
    w.j0 = w.j1 = 0;
    if (BM * w.mt >= p.C) return w;
    w.sc = make_sched_single(p, w.retrieval, c0, w.mt);
    w.j1 = w.sc.n;
    if (w.retrieval && p.ns > 1) {
        w.ns_use = min(p.ns, max(1, w.sc.n / kMinSplitTiles));
        w.j0 = min(w.split, w.ns_use) * w.sc.n / w.ns_use;
        w.j1 = min(w.split + 1, w.ns_use) * w.sc.n / w.ns_use;
    }
    return w;
}

// ------------------------------------------------------------------- roles
//
// A CTA's tiles in its passes: number jj = base .. base + nl - 1, base a multiple
// of nl, so that a second pass goes on where the first left the rings and the
// barriers' phases.

enum {   // barriers
    kKFull = 0, kKEmpty = 3, kVFull = 6, kVEmpty = 9,   // [kStages]
    kSFull = 12, kPFull = 15, kSFree = 18,              // [kSlots]
    kQFull = 21, kODone = 22                            // kODone: once a pass
};
struct Cta {
    Sched sc;
    int j0, nl;                        // tiles j0 .. j0 + nl - 1 of the schedule
    int mt, b, kv_idx, cache_z, ring_z;
    uint32_t sQ, sK, sV, tmem;
    uint64_t* bars;
};
__device__ __forceinline__ Cta make_cta(const LayerArgs& a, const Work& w, uint8_t* smem) {
    return {w.sc, w.j0, w.j1 - w.j0, w.mt, w.b, w.kv_idx, w.b * a.R + w.slot, w.b * a.S + (w.slot - a.R),
            smem_u32(smem + kOffQ), smem_u32(smem + kOffK), smem_u32(smem + kOffV),
            *reinterpret_cast<uint32_t*>(smem + kOffHolder), reinterpret_cast<uint64_t*>(smem + kOffBar)};
}
struct KvMaps {
    const CUtensorMap *kc, *vc, *kx, *vx, *kr, *vr;
};

// One thread: K and V tiles, three deep.
__device__ __forceinline__ void load_tiles(const Cta& c, const KvMaps& m, int base, int32_t* status) {
    bool ok = true;
    for (int jj = base; jj < base + c.nl && ok; ++jj) {
        const Tile t = tile_at(c.sc, c.j0 + jj - base);
        const int st = jj % kStages, use = jj / kStages;
        for (int kv = 0; kv < 2 && ok; ++kv) {
            uint64_t* full = c.bars + (kv ? kVFull : kKFull) + st;
            if (use > 0) ok = mbar_wait(c.bars + (kv ? kVEmpty : kKEmpty) + st, (use - 1) & 1, status);
            if (!ok) break;
            mbar_arrive_expect_tx(full, kTileBytes);
            const uint32_t dst = (kv ? c.sV : c.sK) + st * kTileBytes;
            for (int half = 0; half < 2; ++half)
                for (int rh = 0; rh < BN / kBox; ++rh) {
                    const uint32_t d2 = dst + half * kHalfBytes + rh * kBox * 128;
                    const int x = 64 * half, row = t.row + kBox * rh;
                    if (t.src == SRC_CACHE)
                        tma_load_3d(d2, kv ? m.vc : m.kc, x, row, c.cache_z, full);
                    else if (t.src == SRC_CHUNK)
                        tma_load_4d(d2, kv ? m.vx : m.kx, x, c.kv_idx, row, c.b, full);
                    else
                        tma_load_3d(d2, kv ? m.vr : m.kr, x, row, c.ring_z, full);
                }
        }
    }
}

// One warp: S(j) = Q K(j)^T; the whole warp waits, one lane issues.
template <int kSlots>
__device__ __forceinline__ void issue_qk(const Cta& c, int base, int32_t* status) {
    constexpr uint32_t idesc_qk = idesc_bf16(BM, BN, 0, 0);
    bool ok = mbar_wait(c.bars + kQFull, 0, status);
    for (int jj = base; jj < base + c.nl && ok; ++jj) {
        const int st = jj % kStages, sl = jj % kSlots, use = jj / kSlots;
        // the slot holds P(jj - kSlots) until its P V is done
        if (use > 0) ok = mbar_wait(c.bars + kSFree + sl, (use - 1) & 1, status);
        ok = ok && mbar_wait(c.bars + kKFull + st, (jj / kStages) & 1, status);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
            const uint64_t qd = sw128_desc(c.sQ, 16, 1024), kd = sw128_desc(c.sK + st * kTileBytes, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
                const uint32_t o = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
                tc_mma(c.tmem + 128 * sl, qd + o, kd + o, idesc_qk, kk > 0 ? 1u : 0u);
            }
            tc_commit(c.bars + kSFull + sl);
            tc_commit(c.bars + kKEmpty + st);
        }
    }
    __syncwarp();
}

// One warp: O += P(j) V(j), P from TMEM: 16 packed columns at the start of every 32 of S.
template <bool MIX, int kSlots>
__device__ __forceinline__ void issue_pv(const Cta& c, const LayerArgs& a, int base, int32_t* status) {
    constexpr uint32_t idesc_pv = idesc_bf16(BM, HD, 0, 1);
    bool ok = true, first_lam = true;
    for (int jj = base; jj < base + c.nl && ok; ++jj) {
        const int st = jj % kStages, sl = jj % kSlots;
        ok = mbar_wait(c.bars + kVFull + st, (jj / kStages) & 1, status) &&
             mbar_wait(c.bars + kPFull + sl, (jj / kSlots) & 1, status);
        if (!ok) break;
        tc_fence_after();
        const bool lam = MIX && lambda_tile(a, c.mt, jj - base);
        if (elect_one()) {
            const uint64_t vd = sw128_desc(c.sV + st * kTileBytes, kHalfBytes, 1024);
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
                tc_mma_ta(c.tmem + kColO, c.tmem + 128 * sl + 32 * (kk >> 1) + 8 * (kk & 1), vd + kk * (2048 >> 4), idesc_pv,
                          (jj > base || kk > 0) ? 1u : 0u);
            if (lam) {
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                    tc_mma_ta(c.tmem + kColOs, c.tmem + 128 * sl + 32 * (kk >> 1) + 16 + 8 * (kk & 1), vd + kk * (2048 >> 4),
                              idesc_pv, (!first_lam || kk > 0) ? 1u : 0u);
            }
            tc_commit(c.bars + kVEmpty + st);
            tc_commit(c.bars + kSFree + sl);
            if (jj == base + c.nl - 1) tc_commit(c.bars + kODone);
        }
        if (lam) first_lam = false;
    }
    __syncwarp();
}

// The largest size among 32 values; NaN if one is NaN.
__device__ __forceinline__ float largest_nan(const float (&o)[32]) {
    auto max_nan = [](float a, float b, float c) {
        float d;
        asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
        return d;
    };
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; i += 2) m[(i >> 1) & 3] = max_nan(m[(i >> 1) & 3], o[i], o[i + 1]);
    return max_nan(max_nan(m[0], m[1], m[2]), m[3], 0.f);
}

// The end of a pass for a thread of the exponential warps, one row and 32
// columns (`quarter`) each: the row's sums l_row and l_lam from the shares l,
// the stores, and in the first pass whether its results are in range.  bias,
// bias_l: log2 by which the pass lowered the row's p.
template <int EPI>
__device__ __forceinline__ void store_rows(const TcArgs& p, const Work& w, const Cta& c, uint8_t* smem, int row, int quarter, float2 l,
                                           float bias, float bias_l, bool ok, int pass) {
    constexpr bool MIX = EPI == EPI_MIX_KEEP;
    const LayerArgs& a = p.a;
    uint32_t* holder = reinterpret_cast<uint32_t*>(smem + kOffHolder);
    const int tid = threadIdx.x, crow = BM * w.mt + row, b = w.b, mt = w.mt, q_idx = w.q_idx, kv_idx = w.kv_idx;
    const int unit = w.unit, split = w.split, ns_use = w.ns_use;
    const uint32_t lane_base = c.tmem + ((uint32_t)(row & ~31) << 16);
    // the row's sum over both groups and column halves; each thread then
    // stores 32 columns of its row
    float* sums = reinterpret_cast<float*>(smem + kOffSum);
    auto row_total = [&](float part) {
        sums[quarter * BM + row] = part;
        asm volatile("bar.sync 1, 512;" ::: "memory");
        return (sums[row] + sums[BM + row]) + (sums[2 * BM + row] + sums[3 * BM + row]);
    };
    const float l_row = row_total(l.x);
    float l_lam = 0.f;
    if constexpr (MIX) {
        asm volatile("bar.sync 1, 512;" ::: "memory");    // everyone has read the first totals
        l_lam = row_total(l.y);
    }
    if (pass == 0 && quarter == 0)   // where a second pass finds them: over tiles that are done with
        reinterpret_cast<float2*>(smem + kOffSums2)[row] = make_float2(l_row, l_lam);
    const size_t off = (((size_t)b * p.C + crow) * a.Hq + q_idx) * HD + 32 * quarter;
    const bool out_ok = bounds_ok(b < a.B && q_idx >= 0 && q_idx < a.Hq, p.status);
    const bool live = crow < p.C && out_ok;
    ok = __all_sync(0xffffffffu, ok && mbar_wait(c.bars + kODone, pass, p.status));
    float o[32];
    // the first pass: do this row's results, in o (divided by the sums, or a
    // split's), ask for a second one?
    auto judge = [&](float limit, bool divided) {
        if (pass != 0 || !live || !ok) return;
        const float m = largest_nan(o);
        auto lost = [&](float l) { return l > 0.f && l < kMinSum && m * (divided ? l : 1.f) < kMinO; };
        if (!(m <= limit) || lost(l_row) || (MIX && lost(l_lam))) holder[2] = 1u;
    };
    if (ok) {
        tc_fence_after();
        tmem_ld32(lane_base + kColO + 32 * quarter, o);
    } else {
        holder[3] = 1u;
    }
    __nv_bfloat16* op = static_cast<__nv_bfloat16*>(p.out) + off;
    if (!out_ok) {
        // debug build: the check failed, nothing is written
    } else if (MIX || ns_use == 1) {
        if (ok) {
            const float inv = l_row > 0.f ? 1.f / l_row : 0.f;
            if constexpr (MIX) {
                // both attentions into the mix, and both log-sums kept
                const float al = p.epi.alpha[kv_idx];
                const float fc = al * inv, fs = l_lam > 0.f ? (1.f - al) / l_lam : 0.f;
                if (quarter == 0 && live) {
                    const size_t r = ((size_t)b * a.Hq + q_idx) * p.C + crow;
                    p.epi.lse[r] = bias + log2f(l_row);
                    p.epi.lse[(size_t)a.B * a.Hq * p.C + r] = bias_l + log2f(l_lam);
                }
                float os[32];
                tmem_ld32(lane_base + kColOs + 32 * quarter, os);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = fmaf(fs, os[e], fc * o[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= inv;
            }
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
                float v8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v8[e] = o[8 * q4 + e];
                if (live) store_row<__nv_bfloat16, 8>(op + 8 * q4, v8);
            }
            judge(3.4028235e38f, true);
        }
    } else if (bounds_ok(unit < p.n_units && split < p.ns, p.status)) {
        // this split's record of the query tile (the maximum is the bias), then a
        // ticket per query tile (half a word of the pair's); the CTA that arrives
        // last merges (no CTA ever waits)
        judge(kMaxO, false);
        const int qi = mt & 1;
        float* rec = p.part + (((size_t)unit * p.ns + split) * 2 + qi) * kPartFloats;
        if (quarter == 0) {
            rec[row] = ok ? bias : -INFINITY;
            rec[BM + row] = ok ? l_row : 0.f;
        }
#pragma unroll
        for (int g4 = 0; g4 < 8; ++g4)
            reinterpret_cast<float4*>(rec + 2 * BM)[(8 * quarter + g4) * BM + row] =
                ok ? make_float4(o[4 * g4], o[4 * g4 + 1], o[4 * g4 + 2], o[4 * g4 + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
        __threadfence();
        asm volatile("bar.sync 1, 512;" ::: "memory");
        if (pass == 0 && holder[2] != 0u && holder[3] == 0u) return;   // the record is written again
        if (tid == 0) {
            const uint32_t seen = atomicAdd(&p.ticket[unit], 1u << (16 * qi)) >> (16 * qi);
            holder[1] = (seen & 0xffffu) == (uint32_t)ns_use - 1 ? 1u : 0u;
        }
        asm volatile("bar.sync 1, 512;" ::: "memory");
        if (holder[1] && quarter == 0) {
            __threadfence();
            merge_split_records(p.part + (size_t)unit * p.ns * 2 * kPartFloats + (size_t)qi * kPartFloats, ns_use, row,
                                crow < p.C, op, 2);
        }
    }
}

// The second pass, by all of the CTA's warps: its rows again, with every row's
// exponents lowered by the log2 of twice its sum (l_row; of the Lambda attention
// l_lam).  It works its item out again: nothing is held for it through the first
// pass (that, and a call instead of code in place, took 1.8 % of the time).
template <int EPI>
__device__ __forceinline__ void second_pass(const KvMaps m, const TcArgs& p) {
    constexpr bool MIX = EPI == EPI_MIX_KEEP;
    constexpr int kSlots = s_slots<MIX>();
    extern __shared__ __align__(1024) uint8_t smem[];
    const LayerArgs& a = p.a;
    const Work w = work_item(p);
    const Cta c = make_cta(a, w, smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, base = c.nl;
    const float2 sums = reinterpret_cast<const float2*>(smem + kOffSums2)[32 * (warp & 3) + lane];
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();                                  // the sums are read: the tiles may come
    if (warp == kTmaWarp) {
        if (lane == 0) load_tiles(c, m, base, p.status);
        __syncwarp();
    } else if (warp == kQkWarp) {
        issue_qk<kSlots>(c, base, p.status);
    } else if (warp == kPvWarp) {
        issue_pv<MIX, kSlots>(c, a, base, p.status);
    } else if (warp < kExpWarps) {
        const int group = warp >> 3, half = (warp >> 2) & 1, quarter = warp >> 2;
        const int row = 32 * (warp & 3) + lane, crow = BM * c.mt + row;
        const uint32_t lane_base = c.tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const float bias = sums.x > 0.f ? log2f(sums.x) + 1.f : 0.f, bias_l = sums.y > 0.f ? log2f(sums.y) + 1.f : 0.f;
        Sched lam_sc = c.sc;
        lam_sc.retrieval = false;
        float2 l = make_float2(0.f, 0.f);
        bool ok = true;
        for (int jj = base + ((base ^ group) & 1); jj < base + c.nl; jj += 2) {
            const int sl = jj % kSlots;
            ok = __all_sync(0xffffffffu, mbar_wait(c.bars + kSFull + sl, (jj / kSlots) & 1, p.status));
            if (!ok) break;
            tc_fence_after();
            const Tile t = tile_at(c.sc, c.j0 + jj - base);
            const bool lam = MIX && lambda_tile(a, c.mt, jj - base);
            uint32_t vis[4] = {0u, 0u, 0u, 0u}, seen_l[4] = {0u, 0u, 0u, 0u};
            visible_columns(a, c.sc, t, c.sc.c0 + crow, vis);
            if (lam) visible_columns(a, lam_sc, t, c.sc.c0 + crow, seen_l);
            const uint32_t s_addr = lane_base + 128 * sl + 64 * half;
#pragma unroll 1
            for (int ch = 0; ch < 2; ++ch) {
                const uint32_t v = half ? (ch ? vis[3] : vis[2]) : (ch ? vis[1] : vis[0]);
                const uint32_t vl = half ? (ch ? seen_l[3] : seen_l[2]) : (ch ? seen_l[1] : seen_l[0]);
                float x[32];
                tmem_ld32(s_addr + 32 * ch, x);
                uint32_t pk[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float e[2], f[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float s = score_log2<true, false>(x[2 * i + h], a.cap.sl, a.cap);
                        e[h] = (v >> (2 * i + h)) & 1u ? sfu_exp2(s - bias) : 0.f;
                        f[h] = (vl >> (2 * i + h)) & 1u ? sfu_exp2(s - bias_l) : 0.f;
                    }
                    __nv_bfloat162 pe = __floats2bfloat162_rn(e[0], e[1]), pf = __floats2bfloat162_rn(f[0], f[1]);
                    pk[i] = *reinterpret_cast<uint32_t*>(&pe);
                    pk[16 + i] = *reinterpret_cast<uint32_t*>(&pf);
                    l.x += bf16_lo(pk[i]) + bf16_hi(pk[i]);
                    l.y += bf16_lo(pk[16 + i]) + bf16_hi(pk[16 + i]);
                }
                tmem_st32(s_addr + 32 * ch, pk);   // the second half is read in Lambda tiles only
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bars + kPFull + sl);
        }
        store_rows<EPI>(p, w, c, smem, row, quarter, l, bias, bias_l, ok, 1);
    }
}

// EPI: EPI_STORE (store, or key-range split records) or EPI_MIX_KEEP (both
// attentions, mixed; every KV head in the retrieval block).
template <int EPI>
__global__ void __launch_bounds__(kRegThreads, 1)
    prefill_capped_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKc,
                          const __grid_constant__ CUtensorMap tmVc, const __grid_constant__ CUtensorMap tmKx,
                          const __grid_constant__ CUtensorMap tmVx, const __grid_constant__ CUtensorMap tmKr,
                          const __grid_constant__ CUtensorMap tmVr, const TcArgs p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr bool MIX = EPI == EPI_MIX_KEEP;
    constexpr int kSlots = s_slots<MIX>();
    const LayerArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((smem_u32(smem) & 1023u) != 0) {   // the swizzled layouts need 1024-byte alignment
        if (tid == 0 && p.status) atomicOr(p.status, DUO_DEV_BAD_LENGTH);
        return;
    }
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint32_t* holder = reinterpret_cast<uint32_t*>(smem + kOffHolder);

    const Work w = work_item(p);
    if (w.j0 >= w.j1) return;
    const Sched& sc = w.sc;
    const int mt = w.mt, c0 = sc.c0, j0 = w.j0, nl = w.j1 - w.j0;   // nl tiles, at least one

    if (warp == kQkWarp) tmem_alloc(holder, kTmemCols);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bars + kKFull + i, 1);
            mbar_init(bars + kKEmpty + i, 1);
            mbar_init(bars + kVFull + i, 1);
            mbar_init(bars + kVEmpty + i, 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(bars + kSFull + i, 1);
            mbar_init(bars + kPFull + i, kExpWarps / 2);
            mbar_init(bars + kSFree + i, 1);
        }
        mbar_init(bars + kQFull, 1);
        mbar_init(bars + kODone, 1);
        holder[2] = holder[3] = 0u;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;
    const Cta cta = make_cta(a, w, smem);

    if (warp == kTmaWarp) {
        if (lane == 0) {
            mbar_arrive_expect_tx(bars + kQFull, kTileBytes);
            for (int half = 0; half < 2; ++half)
                tma_load_4d(cta.sQ + half * kHalfBytes, &tmQ, 64 * half, w.q_idx, BM * mt, w.b, bars + kQFull);
            load_tiles(cta, KvMaps{&tmKc, &tmVc, &tmKx, &tmVx, &tmKr, &tmVr}, 0, p.status);
        }
        __syncwarp();
    } else if (warp == kQkWarp) {
        issue_qk<kSlots>(cta, 0, p.status);
    } else if (warp == kPvWarp) {
        issue_pv<MIX, kSlots>(cta, a, 0, p.status);
    } else if (warp < kExpWarps) {
        const int group = warp >> 3, half = (warp >> 2) & 1;  // key tiles j % 2 == group; column half
        const int row = 32 * (warp & 3) + lane;               // TMEM lane
        const int crow = BM * mt + row;                       // chunk row
        const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        float2 l = make_float2(0.f, 0.f);                     // row sums: causal (or the head's mask), Lambda (MIX)
        bool ok = true;
        int plain_first, plain_last;
        unmasked_tiles(sc, plain_first, plain_last);
        Sched lam_sc = sc;                                    // the same tiles under the Lambda mask
        lam_sc.retrieval = false;
        for (int j = group; j < nl; j += 2) {
            const int sl = j % kSlots;
            ok = __all_sync(0xffffffffu, mbar_wait(bars + kSFull + sl, (j / kSlots) & 1, p.status));
            if (!ok) break;
            tc_fence_after();
            const uint32_t s_addr = lane_base + 128 * sl + 64 * half;
            if (MIX && lambda_tile(a, mt, j)) {
                const Tile t = tile_at(sc, j);
                uint32_t vis[4] = {0u, 0u, 0u, 0u}, lam[4] = {0u, 0u, 0u, 0u};
                visible_columns(a, sc, t, crow, vis);
                visible_columns(a, lam_sc, t, crow, lam);
                exp_columns<true, true>(l, s_addr, a.cap, p.poly, half_bits(vis, half), half_bits(lam, half));
            } else if (j0 + j >= plain_first && j0 + j < plain_last) {
                exp_columns<false, false>(l, s_addr, a.cap, p.poly, 0u, 0u);
            } else if (!MIX) {
                uint32_t vis[4] = {0u, 0u, 0u, 0u};           // the tile's keys this row sees, a bit per column
                visible_columns(a, sc, tile_at(sc, j0 + j), c0 + crow, vis);
                exp_columns<true, false>(l, s_addr, a.cap, p.poly, half_bits(vis, half), 0u);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + kPFull + sl);
        }
        store_rows<EPI>(p, w, cta, smem, row, warp >> 2, l, 0.f, 0.f, ok, 0);
    }
    tc_fence_before();
    __syncthreads();
    if (__builtin_expect(holder[2] != 0u && holder[3] == 0u, 0)) {
        tc_fence_after();
        second_pass<EPI>(KvMaps{&tmKc, &tmVc, &tmKx, &tmVx, &tmKr, &tmVr}, p);
        tc_fence_before();
        __syncthreads();
    }
    if (warp == kQkWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int EPI>
cudaError_t launch_variant(const TcMaps& m, const TcArgs& p, unsigned grid, cudaStream_t s) {
    if (grid > 0x3fffffffu) return cudaErrorInvalidConfiguration;
    grid *= 2;   // a CTA per query tile, not per pair
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = smem_limit_once(prefill_capped_kernel<EPI>, (int)kSmemBytes, configured);
    if (e != cudaSuccess) return e;
    prefill_capped_kernel<EPI><<<grid, kThreads, kSmemBytes, s>>>(m.q, m.kc, m.vc, m.kx, m.vx, m.kr, m.vr, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_capped(const TcMaps& m, const TcArgs& p, int mode, unsigned grid, cudaStream_t s) {
    if (mode == EPI_STORE) return launch_variant<EPI_STORE>(m, p, grid, s);
    if (mode == EPI_MIX_KEEP) return launch_variant<EPI_MIX_KEEP>(m, p, grid, s);
    return cudaErrorInvalidValue;
}

}  // namespace duo
