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
// Work, schedule of key tiles and masks: prefill_sched.cuh, as prefill_tc.cu:
// a CTA owns two 128-row query tiles that share every 128-key tile;
// TMEM S0 | S1 | O0 | O1, 128 columns each; the MMA thread's order is
//   QK0(0) QK1(0) | PV0(0) QK0(1) PV1(0) QK1(1) | ...
// Roles (576 threads): warps 0-15 the exponentials (warp w: query tile w / 8,
// lanes 32 (w % 4) .., columns 64 ((w / 4) % 2) ..), warp 16 TMA, warp 17 MMA.
// Each takes 32 columns at a time from TMEM: tanh on the FMA pipe when the
// warp's |k x| are all within its polynomial's range (cap.cuh), one
// exponential pair in kFmaExpEvery on the FMA pipe too, the others on the SFU;
// p packed as bf16 goes over the columns it came from.  The row sum adds
// the rounded p, so that an output is a convex combination of V rows.
// Bound: SFU, FMA pipe and tensor pipe alike, about 1,000 cycles each per
// 128 x 128 tile.
#include <cuda.h>

#include "cap.cuh"
#include "common.cuh"
#include "internal.h"
#include "prefill_sched.cuh"
#include "tcgen05.cuh"

namespace duo {
namespace {

constexpr int kExpWarps = 16, kTmaWarp = 16, kMmaWarp = 17, kThreads = 576;
constexpr int kRegThreads = 640;                   // five warps to a sub-partition: 96 registers
constexpr int kFmaExpEvery = 4;
constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ constexpr uint32_t col_s(int i) { return 128u * (uint32_t)i; }
__device__ __forceinline__ constexpr uint32_t col_o(int i) { return 256u + 128u * (uint32_t)i; }
constexpr uint32_t kQBytes = BM * HD * 2;          // 32 KB per query tile (two 16 KB halves of d)
constexpr uint32_t kTileBytes = BN * HD * 2;       // 32 KB per K or V tile (two 16 KB halves of d)
constexpr uint32_t kHalfBytes = kTileBytes / 2;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + 2 * kQBytes;
constexpr uint32_t kOffV = kOffK + 2 * kTileBytes;
constexpr uint32_t kOffSum = kOffV + 2 * kTileBytes;   // [2][2][128] row sums of the column halves
constexpr uint32_t kOffBar = kOffSum + 4 * BM * 4;
constexpr uint32_t kOffHolder = kOffBar + 16 * 8;
constexpr uint32_t kSmemBytes = kOffHolder + 16;
static_assert(kSmemBytes + 1024 <= 232448, "one CTA per SM");

// 2^x for a pair, |x| <= 90, on the FMA pipe: as exp2_fma2 of prefill_tc.cu
// (range reduction to [-0.5, 0.5], a cubic fitted to 7.5e-5), without its
// clamp: the exponent cannot leave the normal range.
__device__ __forceinline__ float2 exp2_fma_bounded2(float2 x) {
    constexpr float kShift = 12582912.f;  // 1.5 * 2^23
    constexpr float c0 = 0.9999280571937561f, c1 = 0.6932610273361206f, c2 = 0.24261116981506348f,
                    c3 = 0.055171627551317215f;
    const float2 t = fadd2(x, make_float2(kShift, kShift));
    const float2 n = fadd2(t, make_float2(-kShift, -kShift));
    const float2 f = ffma2(n, make_float2(-1.f, -1.f), x);
    float2 q = ffma2(make_float2(c3, c3), f, make_float2(c2, c2));
    q = ffma2(q, f, make_float2(c1, c1));
    q = ffma2(q, f, make_float2(c0, c0));
    return make_float2(__uint_as_float(__float_as_uint(q.x) + (__float_as_uint(t.x) << 23)),
                       __uint_as_float(__float_as_uint(q.y) + (__float_as_uint(t.y) << 23)));
}

// 32 columns of a row: dot products x -> p, packed as bf16 in pk; returns the
// sum of the rounded p.  POLY: every |k x| is within the polynomial's range.
// One loop from the dot product to the packed p, so that the FMA, SFU and ALU
// work of neighbouring pairs interleaves.
template <bool MASKED, bool POLY>
__device__ __forceinline__ float exp_loop(const float (&x)[32], uint32_t (&pk)[16], const CapArgs& cap, const TanhPoly& tp,
                                          uint32_t vis) {
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int c2 = 0; c2 < 16; ++c2) {
        float2 v = make_float2(x[2 * c2], x[2 * c2 + 1]);
        v = POLY ? poly_fma2(v, tp) : make_float2(cap.c2 * tanh_sfu(v.x * cap.k), cap.c2 * tanh_sfu(v.y * cap.k));
        float2 e = c2 % kFmaExpEvery == kFmaExpEvery - 1 ? exp2_fma_bounded2(v) : make_float2(sfu_exp2(v.x), sfu_exp2(v.y));
        if constexpr (MASKED) {
            e.x = (vis >> (2 * c2)) & 1u ? e.x : 0.f;
            e.y = (vis >> (2 * c2 + 1)) & 1u ? e.y : 0.f;
        }
        __nv_bfloat162 h = __floats2bfloat162_rn(e.x, e.y);
        pk[c2] = *reinterpret_cast<uint32_t*>(&h);
        sum[c2 & 1] = fadd2(sum[c2 & 1], make_float2(bf16_lo(pk[c2]), bf16_hi(pk[c2])));
    }
    return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// 32 columns of a row: dot products at s_addr -> p over the first 16 of them.
template <bool MASKED>
__device__ __forceinline__ float exp_columns(uint32_t s_addr, const CapArgs& cap, const TanhPoly& tp, uint32_t vis) {
    float x[32];
    tmem_ld32(s_addr, x);
    uint32_t pk[16];
    const float l = __all_sync(0xffffffffu, largest(x) * cap.k <= kTanhRange) ? exp_loop<MASKED, true>(x, pk, cap, tp, vis)
                                                                             : exp_loop<MASKED, false>(x, pk, cap, tp, vis);
    tmem_st16(s_addr, pk);
    return l;
}

// EPI: EPI_STORE (store, or key-range split records), EPI_KEEP, EPI_MIX_KEEP
// (internal.h).
template <int EPI>
__global__ void __launch_bounds__(kRegThreads, 1)
    prefill_capped_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKc,
                          const __grid_constant__ CUtensorMap tmVc, const __grid_constant__ CUtensorMap tmKx,
                          const __grid_constant__ CUtensorMap tmVx, const __grid_constant__ CUtensorMap tmKr,
                          const __grid_constant__ CUtensorMap tmVr, const TcArgs p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const LayerArgs& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((smem_u32(smem) & 1023u) != 0) {   // the swizzled layouts need 1024-byte alignment
        if (tid == 0 && p.status) atomicOr(p.status, DUO_DEV_BAD_LENGTH);
        return;
    }
    const uint32_t sQ = smem_u32(smem + kOffQ), sK = smem_u32(smem + kOffK), sV = smem_u32(smem + kOffV);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint64_t* q_full = bars + 0;
    uint64_t* k_full = bars + 1;    // [2]
    uint64_t* k_empty = bars + 3;   // [2]
    uint64_t* v_full = bars + 5;    // [2]
    uint64_t* v_empty = bars + 7;   // [2]
    uint64_t* s_full = bars + 9;    // [2]: per query tile
    uint64_t* p_full = bars + 11;   // [2]: per query tile
    uint64_t* o_done = bars + 13;   // [2]: per query tile, once
    uint32_t* holder = reinterpret_cast<uint32_t*>(smem + kOffHolder);

    // the work item: as prefill_tc.cu, (sequence, KV head) outermost, then the
    // split, then the query-tile pair (heaviest first) and the query head
    const bool retrieval = (int)blockIdx.x < p.n_ret_ctas;
    int unit = 0, split = 0, m, g, hs, b;
    if (retrieval) {
        const int per_group = p.n_mpairs * a.G;
        const int r = (int)blockIdx.x;
        const int inner = r % per_group;
        split = (r / per_group) % p.ns;
        const int bh = r / (per_group * p.ns);
        g = inner % a.G;
        m = p.n_mpairs - 1 - inner / a.G;
        hs = bh % a.R;
        b = bh / a.R;
        unit = (bh * p.n_mpairs + m) * a.G + g;
    } else {
        int idx = (int)blockIdx.x - p.n_ret_ctas;
        const int per_m = a.B * a.S * a.G;
        m = p.n_mpairs - 1 - idx / per_m;
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
        if (tid == 0 && m == p.n_mpairs - 1 && p.status) atomicOr(p.status, DUO_DEV_BAD_LENGTH);
        c0 = a.capacity;
    }
    const Sched sc = make_sched(p, retrieval, c0, m);
    int ns_use = 1, j0 = 0, j1 = sc.n;
    if (retrieval && p.ns > 1) {
        ns_use = min(p.ns, max(1, sc.n / kMinSplitTiles));
        if (split >= ns_use) return;
        j0 = split * sc.n / ns_use;
        j1 = (split + 1) * sc.n / ns_use;
    }
    const int nl = j1 - j0;                           // tiles of this CTA for Q1
    const int nl0 = max(0, min(j1, sc.n0) - j0);      // ... and for Q0

    if (warp == kMmaWarp) tmem_alloc(holder, kTmemCols);
    if (tid == 0) {
        mbar_init(q_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], kExpWarps / 2);
            mbar_init(&o_done[i], 1);
        }
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;

    if (warp == kTmaWarp) {
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, 2 * kQBytes);
            for (int qi = 0; qi < 2; ++qi)
                for (int half = 0; half < 2; ++half)
                    tma_load_4d(sQ + qi * kQBytes + half * (kQBytes / 2), &tmQ, 64 * half, q_idx, BM * (2 * m + qi), b,
                                q_full);
            const int cache_z = b * a.R + slot, ring_z = b * a.S + (slot - a.R);
            bool ok = true;
            for (int j = 0; j < nl && ok; ++j) {
                const Tile t = tile_at(sc, j0 + j);
                const int st = j & 1;
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    uint64_t* full = kv ? &v_full[st] : &k_full[st];
                    if (j >= 2) ok = mbar_wait(kv ? &v_empty[st] : &k_empty[st], ((j >> 1) - 1) & 1, p.status);
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
    } else if (warp == kMmaWarp) {
        // the whole warp, one lane issuing
        const uint32_t lead = lane == 0 ? 1u : 0u;
        constexpr uint32_t idesc_qk = idesc_bf16(BM, BN, 0, 0);
        constexpr uint32_t idesc_pv = idesc_bf16(BM, HD, 0, 1);
        const uint32_t q_lo = sw128_lo(sQ, 16), k_lo = sw128_lo(sK, 16), v_lo = sw128_lo(sV, kHalfBytes);
        auto issue_qk = [&](int qi, int j) {
            const uint32_t q = q_lo + qi * (kQBytes >> 4), k = k_lo + (j & 1) * (kTileBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
                const uint32_t o = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
                tc_mma_lead(lead, tmem + col_s(qi), q + o, k + o, idesc_qk, kk > 0 ? 1u : 0u);
            }
            tc_commit_lead(lead, &s_full[qi]);
        };
        // P from TMEM: 16 packed columns at the start of every 32 of S
        auto issue_pv = [&](int qi, int j) {
            const uint32_t v = v_lo + (j & 1) * (kTileBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
                tc_mma_ta_lead(lead, tmem + col_o(qi), tmem + col_s(qi) + 32 * (kk >> 1) + 8 * (kk & 1),
                               v + kk * (2048 >> 4), idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
        };
        bool ok = mbar_wait(q_full, 0, p.status) && mbar_wait(&k_full[0], 0, p.status);
        if (ok) {
            tc_fence_after();
            if (nl0 > 0) issue_qk(0, 0);
            issue_qk(1, 0);
            tc_commit_lead(lead, &k_empty[0]);
        }
        for (int j = 0; j < nl && ok; ++j) {
            const bool next = j + 1 < nl;
            if (next) ok = mbar_wait(&k_full[(j + 1) & 1], ((j + 1) >> 1) & 1, p.status);
            ok = ok && mbar_wait(&v_full[j & 1], (j >> 1) & 1, p.status);
            if (j < nl0) {
                ok = ok && mbar_wait(&p_full[0], j & 1, p.status);
                if (!ok) break;
                tc_fence_after();
                issue_pv(0, j);
                if (j == nl0 - 1) tc_commit_lead(lead, &o_done[0]);
                if (j + 1 < nl0) issue_qk(0, j + 1);
            }
            ok = ok && mbar_wait(&p_full[1], j & 1, p.status);
            if (!ok) break;
            tc_fence_after();
            issue_pv(1, j);
            tc_commit_lead(lead, &v_empty[j & 1]);
            if (!next) tc_commit_lead(lead, &o_done[1]);
            if (next) {
                issue_qk(1, j + 1);
                tc_commit_lead(lead, &k_empty[(j + 1) & 1]);
            }
        }
        __syncwarp();
    } else if (warp < kExpWarps) {
        const int qi = warp >> 3, half = (warp >> 2) & 1;     // query tile and column half
        const int row = 32 * (warp & 3) + lane;               // TMEM lane
        const int crow = BM * (2 * m + qi) + row;             // chunk row
        const int n_me = qi ? nl : nl0;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const TanhPoly tp = tanh_poly(a.cap.k, a.cap.c2);
        float l_sum = 0.f;
        bool ok = true;
        for (int j = 0; j < n_me; ++j) {
            ok = __all_sync(0xffffffffu, mbar_wait(&s_full[qi], j & 1, p.status));
            if (!ok) break;
            tc_fence_after();
            const Tile t = tile_at(sc, j0 + j);
            const uint32_t s_addr = lane_base + col_s(qi) + 64 * half;
            if (needs_mask(sc, t, qi)) {
                uint32_t vis[4] = {0u, 0u, 0u, 0u};           // the tile's keys this row sees, a bit per column
                visible_columns(a, sc, t, c0 + crow, vis);
                l_sum += exp_columns<true>(s_addr, a.cap, tp, half ? vis[2] : vis[0]);
                l_sum += exp_columns<true>(s_addr + 32, a.cap, tp, half ? vis[3] : vis[1]);
            } else {
                l_sum += exp_columns<false>(s_addr, a.cap, tp, 0u);
                l_sum += exp_columns<false>(s_addr + 32, a.cap, tp, 0u);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[qi]);
        }
        // the row's sum over both column halves
        float* sums = reinterpret_cast<float*>(smem + kOffSum) + qi * 2 * BM;
        sums[half * BM + row] = l_sum;
        asm volatile("bar.sync %0, 256;" ::"r"(1 + qi) : "memory");
        const float l_row = sums[row] + sums[BM + row];
        // this thread's output: 64 columns of its row
        const size_t off = (((size_t)b * p.C + crow) * a.Hq + q_idx) * HD + 64 * half;
        const bool out_ok = bounds_ok(b < a.B && q_idx >= 0 && q_idx < a.Hq, p.status);
        const bool live = crow < p.C && out_ok;
        uint4 pre[8];   // EPI_MIX_KEEP: the streaming attention of these columns, loaded before the wait below
        if constexpr (EPI == EPI_MIX_KEEP) {
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.epi.streaming) + off);
#pragma unroll
            for (int i = 0; i < 8; ++i) pre[i] = live ? src[i] : make_uint4(0u, 0u, 0u, 0u);
        }
        if (ok && n_me >= 1) ok = __all_sync(0xffffffffu, mbar_wait(&o_done[qi], 0, p.status));
        const bool have = ok && n_me >= 1;                    // warp-uniform
        if (have) tc_fence_after();
        const uint32_t o_addr = lane_base + col_o(qi) + 64 * half;
        __nv_bfloat16* op = static_cast<__nv_bfloat16*>(p.out) + off;
        if (!out_ok) {
            // debug build: the check failed, nothing is written
        } else if (EPI != EPI_STORE || ns_use == 1) {
            if (have) {
                const float inv = l_row > 0.f ? 1.f / l_row : 0.f;
                const float al = EPI == EPI_MIX_KEEP ? p.epi.alpha[kv_idx] : 0.f;
                if (EPI != EPI_STORE && half == 0 && live)
                    p.epi.lse[((size_t)b * a.Hq + q_idx) * p.C + crow] = log2f(l_row);
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    float o[32];
                    tmem_ld32(o_addr + 32 * ch, o);
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                        float v8[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v8[e] = o[8 * q4 + e] * inv;
                        if constexpr (EPI == EPI_MIX_KEEP) {
                            const uint4 u = pre[4 * ch + q4];
                            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                v8[2 * e] = al * v8[2 * e] + (1.f - al) * bf16_lo(w[e]);
                                v8[2 * e + 1] = al * v8[2 * e + 1] + (1.f - al) * bf16_hi(w[e]);
                            }
                        }
                        if (live) store_row<__nv_bfloat16, 8>(op + 32 * ch + 8 * q4, v8);
                    }
                }
            }
        } else if (bounds_ok(unit < p.n_units && split < p.ns, p.status)) {
            // this split's record of the query tile (the maximum is 0 for every
            // row that has keys), then a ticket per unit; the CTA that arrives
            // last merges (no CTA ever waits)
            float* rec = p.part + (((size_t)unit * p.ns + split) * 2 + qi) * kPartFloats;
            if (half == 0) {
                rec[row] = have ? 0.f : -INFINITY;
                rec[BM + row] = have ? l_row : 0.f;
            }
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
                float o[32];
                if (have) {
                    tmem_ld32(o_addr + 32 * ch, o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
#pragma unroll
                for (int g4 = 0; g4 < 8; ++g4)
                    reinterpret_cast<float4*>(rec + 2 * BM)[(16 * half + 8 * ch + g4) * BM + row] =
                        make_float4(o[4 * g4], o[4 * g4 + 1], o[4 * g4 + 2], o[4 * g4 + 3]);
            }
            __threadfence();
            asm volatile("bar.sync 3, 512;" ::: "memory");
            if (tid == 0) holder[1] = (atomicAdd(&p.ticket[unit], 1u) == (unsigned)ns_use - 1) ? 1u : 0u;
            asm volatile("bar.sync 3, 512;" ::: "memory");
            if (holder[1] && half == 0) {
                __threadfence();
                merge_split_records(p.part + (size_t)unit * p.ns * 2 * kPartFloats + (size_t)qi * kPartFloats, ns_use, row,
                                    crow < p.C, op, 4 + qi);
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

template <int EPI>
cudaError_t launch_variant(const TcMaps& m, const TcArgs& p, unsigned grid, cudaStream_t s) {
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = smem_limit_once(prefill_capped_kernel<EPI>, (int)kSmemBytes, configured);
    if (e != cudaSuccess) return e;
    prefill_capped_kernel<EPI><<<grid, kThreads, kSmemBytes, s>>>(m.q, m.kc, m.vc, m.kx, m.vx, m.kr, m.vr, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_capped(const TcMaps& m, const TcArgs& p, int mode, unsigned grid, cudaStream_t s) {
    switch (mode) {
        case EPI_STORE: return launch_variant<EPI_STORE>(m, p, grid, s);
        case EPI_KEEP: return launch_variant<EPI_KEEP>(m, p, grid, s);
        case EPI_MIX_KEEP: return launch_variant<EPI_MIX_KEEP>(m, p, grid, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace duo
