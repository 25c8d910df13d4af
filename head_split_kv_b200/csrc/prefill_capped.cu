// prefill_capped.cu -- the tensor-core attention of prefill_tc.cu for scores
// capped by a tanh, where the cap bounds them: the capped pre-fill and the
// gated mix's training forward pass.
//
// A capped score lies in [-cap, cap], so the softmax needs no running maximum:
// with x the dot product, p = 2^(c2 tanh(k x)) lies in [2^-c2, 2^c2], which for
// caps up to 60 (c2 <= 87) stays inside fp32 -- and bf16, whose exponent is the
// same -- with room for the sums: 2^87 a key, 2^20 keys, values up to 2^20.  p
// is then a function of one score alone.  No row statistic stands between
// the scores and the exponentials, O is never rescaled, the columns of a row
// may be split over several threads that never talk until the end, and the
// splits of a key range merge by addition.  (Larger caps, and caches of 8- or
// 4-bit codes, whose fp16 p needs the maximum, take prefill_tc.cu.)
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
constexpr uint32_t kOffHolder = kOffBar + 24 * 8;
constexpr uint32_t kSmemBytes = kOffHolder + 16;
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
            v = make_float2(cap.c2 * tanh_sfu(v.x * cap.k), cap.c2 * tanh_sfu(v.y * cap.k));
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
    const uint32_t sQ = smem_u32(smem + kOffQ), sK = smem_u32(smem + kOffK), sV = smem_u32(smem + kOffV);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint64_t* k_full = bars + 0;    // [kStages]
    uint64_t* k_empty = bars + 3;   // [kStages]
    uint64_t* v_full = bars + 6;    // [kStages]
    uint64_t* v_empty = bars + 9;   // [kStages]
    uint64_t* s_full = bars + 12;   // [kSlots], as the next two
    uint64_t* p_full = bars + 15;
    uint64_t* s_free = bars + 18;
    uint64_t* q_full = bars + 21;
    uint64_t* o_done = bars + 22;
    uint32_t* holder = reinterpret_cast<uint32_t*>(smem + kOffHolder);

    // the work item, ordered as in prefill_tc.cu: (sequence, KV head)
    // outermost, then the split, then the query tile (heaviest first) and
    // the query head
    const bool retrieval = (int)blockIdx.x < 2 * p.n_ret_ctas;
    const int n_mt = 2 * p.n_mpairs;                  // the last may lie past the chunk
    int unit = 0, split = 0, mt, g, hs, b;
    if (retrieval) {
        const int per_group = n_mt * a.G;
        const int r = (int)blockIdx.x;
        const int inner = r % per_group;
        split = (r / per_group) % p.ns;
        const int bh = r / (per_group * p.ns);
        g = inner % a.G;
        mt = n_mt - 1 - inner / a.G;
        hs = bh % a.R;
        b = bh / a.R;
        unit = (bh * p.n_mpairs + mt / 2) * a.G + g;  // of the pair: records and tickets are laid out by pairs
    } else {
        int idx = (int)blockIdx.x - 2 * p.n_ret_ctas;
        const int per_m = a.B * a.S * a.G;
        mt = n_mt - 1 - idx / per_m;
        idx %= per_m;
        g = idx % a.G;
        hs = (idx / a.G) % a.S;
        b = idx / (a.G * a.S);
    }
    const int slot = retrieval ? hs : a.R + hs;
    const int q_idx = a.q_head0[slot] + g, kv_idx = a.kv_head[slot];
    int c0 = p.seq_len ? p.seq_len[b] : 0;            // no lengths: whole sequences, no cache
    if (c0 < 0) c0 = 0;
    if (retrieval && c0 > a.capacity) {
        if (tid == 0 && mt == 0 && p.status) atomicOr(p.status, DUO_DEV_BAD_LENGTH);
        c0 = a.capacity;
    }
    if (BM * mt >= p.C) return;
    const Sched sc = make_sched_single(p, retrieval, c0, mt);
    int ns_use = 1, j0 = 0, j1 = sc.n;
    if (retrieval && p.ns > 1) {
        ns_use = min(p.ns, max(1, sc.n / kMinSplitTiles));
        if (split >= ns_use) return;
        j0 = split * sc.n / ns_use;
        j1 = (split + 1) * sc.n / ns_use;
    }
    const int nl = j1 - j0;                           // tiles of this CTA, at least one

    if (warp == kQkWarp) tmem_alloc(holder, kTmemCols);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], kExpWarps / 2);
            mbar_init(&s_free[i], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(o_done, 1);
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;

    if (warp == kTmaWarp) {
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, kTileBytes);
            for (int half = 0; half < 2; ++half)
                tma_load_4d(sQ + half * kHalfBytes, &tmQ, 64 * half, q_idx, BM * mt, b, q_full);
            const int cache_z = b * a.R + slot, ring_z = b * a.S + (slot - a.R);
            bool ok = true;
            for (int j = 0; j < nl && ok; ++j) {
                const Tile t = tile_at(sc, j0 + j);
                const int st = j % kStages, use = j / kStages;
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    uint64_t* full = kv ? &v_full[st] : &k_full[st];
                    if (use > 0) ok = mbar_wait(kv ? &v_empty[st] : &k_empty[st], (use - 1) & 1, p.status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(full, kTileBytes);
                    const uint32_t dst = (kv ? sV : sK) + st * kTileBytes;
                    for (int half = 0; half < 2; ++half)
                        for (int rh = 0; rh < BN / kBox; ++rh) {
                            const uint32_t d2 = dst + half * kHalfBytes + rh * kBox * 128;
                            const int x = 64 * half, row = t.row + kBox * rh;
                            if (t.src == SRC_CACHE)
                                tma_load_3d(d2, kv ? &tmVc : &tmKc, x, row, cache_z, full);
                            else if (t.src == SRC_CHUNK)
                                tma_load_4d(d2, kv ? &tmVx : &tmKx, x, kv_idx, row, b, full);
                            else
                                tma_load_3d(d2, kv ? &tmVr : &tmKr, x, row, ring_z, full);
                        }
                }
            }
        }
    } else if (warp == kQkWarp) {
        // S(j) = Q K(j)^T; the whole warp waits, one lane issues
        constexpr uint32_t idesc_qk = idesc_bf16(BM, BN, 0, 0);
        bool ok = mbar_wait(q_full, 0, p.status);
        for (int j = 0; j < nl && ok; ++j) {
            const int st = j % kStages, sl = j % kSlots, use = j / kSlots;
            // the slot holds P(j - kSlots) until its P V is done
            if (use > 0) ok = mbar_wait(&s_free[sl], (use - 1) & 1, p.status);
            ok = ok && mbar_wait(&k_full[st], (j / kStages) & 1, p.status);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t qd = sw128_desc(sQ, 16, 1024), kd = sw128_desc(sK + st * kTileBytes, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t o = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
                    tc_mma(tmem + 128 * sl, qd + o, kd + o, idesc_qk, kk > 0 ? 1u : 0u);
                }
                tc_commit(&s_full[sl]);
                tc_commit(&k_empty[st]);
            }
        }
        __syncwarp();
    } else if (warp == kPvWarp) {
        // O += P(j) V(j), P from TMEM: 16 packed columns at the start of every 32 of S
        constexpr uint32_t idesc_pv = idesc_bf16(BM, HD, 0, 1);
        bool ok = true, first_lam = true;
        for (int j = 0; j < nl && ok; ++j) {
            const int st = j % kStages, sl = j % kSlots;
            ok = mbar_wait(&v_full[st], (j / kStages) & 1, p.status) && mbar_wait(&p_full[sl], (j / kSlots) & 1, p.status);
            if (!ok) break;
            tc_fence_after();
            const bool lam = MIX && lambda_tile(a, mt, j);
            if (elect_one()) {
                const uint64_t vd = sw128_desc(sV + st * kTileBytes, kHalfBytes, 1024);
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                    tc_mma_ta(tmem + kColO, tmem + 128 * sl + 32 * (kk >> 1) + 8 * (kk & 1), vd + kk * (2048 >> 4), idesc_pv,
                              (j > 0 || kk > 0) ? 1u : 0u);
                if (lam) {
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        tc_mma_ta(tmem + kColOs, tmem + 128 * sl + 32 * (kk >> 1) + 16 + 8 * (kk & 1), vd + kk * (2048 >> 4),
                                  idesc_pv, (!first_lam || kk > 0) ? 1u : 0u);
                }
                tc_commit(&v_empty[st]);
                tc_commit(&s_free[sl]);
                if (j == nl - 1) tc_commit(o_done);
            }
            if (lam) first_lam = false;
        }
        __syncwarp();
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
            ok = __all_sync(0xffffffffu, mbar_wait(&s_full[sl], (j / kSlots) & 1, p.status));
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
            if (lane == 0) mbar_arrive(&p_full[sl]);
        }
        // the row's sum over both groups and column halves; each thread then
        // stores 32 columns of its row
        float* sums = reinterpret_cast<float*>(smem + kOffSum);
        const int quarter = warp >> 2;
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
        const size_t off = (((size_t)b * p.C + crow) * a.Hq + q_idx) * HD + 32 * quarter;
        const bool out_ok = bounds_ok(b < a.B && q_idx >= 0 && q_idx < a.Hq, p.status);
        const bool live = crow < p.C && out_ok;
        ok = __all_sync(0xffffffffu, ok && mbar_wait(o_done, 0, p.status));
        float o[32];
        if (ok) {
            tc_fence_after();
            tmem_ld32(lane_base + kColO + 32 * quarter, o);
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
                        p.epi.lse[r] = log2f(l_row);
                        p.epi.lse[(size_t)a.B * a.Hq * p.C + r] = log2f(l_lam);
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
            }
        } else if (bounds_ok(unit < p.n_units && split < p.ns, p.status)) {
            // this split's record of the query tile (the maximum is 0 for every
            // row), then a ticket per query tile (half a word of the pair's);
            // the CTA that arrives last merges (no CTA ever waits)
            const int qi = mt & 1;
            float* rec = p.part + (((size_t)unit * p.ns + split) * 2 + qi) * kPartFloats;
            if (quarter == 0) {
                rec[row] = ok ? 0.f : -INFINITY;
                rec[BM + row] = ok ? l_row : 0.f;
            }
#pragma unroll
            for (int g4 = 0; g4 < 8; ++g4)
                reinterpret_cast<float4*>(rec + 2 * BM)[(8 * quarter + g4) * BM + row] =
                    ok ? make_float4(o[4 * g4], o[4 * g4 + 1], o[4 * g4 + 2], o[4 * g4 + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
            __threadfence();
            asm volatile("bar.sync 1, 512;" ::: "memory");
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
    tc_fence_before();
    __syncthreads();
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
