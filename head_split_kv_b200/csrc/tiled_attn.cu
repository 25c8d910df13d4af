// tiled_attn.cu -- attention on the CUDA cores in 64 x 64 tiles, for what the
// tensor-core kernels do not take: the capped pre-fill in fp32 and with
// head_dim 64, and the gated mix's training forward and backward passes in
// those and over windows wider than a tile.
// All arithmetic is fp32 (CUDA's exp2f and tanhf).
//
// Threads as 16 x 16 or 8 x 16; every product is a register tile of RI x 4
// scores (or RI rows x D / 16 columns) per thread, in tiles of 64 outer rows
// or 32 (twice the CTAs, for grids that would leave SMs idle).
// Operands lie in shared memory as fp32 rows padded by four floats, so that 16
// threads reading 16 rows use all banks.  A thread's rows are RI ty .., the
// same for scores and accumulators, so a row's softmax state stays in the 16
// threads of one half-warp (shuffles, no shared memory); its score columns are
// tx + 16 j.  Probabilities pass between the products through shared memory,
// transposed.  The next tile's rows are loaded into registers while the
// current one is computed (rows of 512 bytes, fp32 with d 128, would take too
// many and are not).
// Bound by shared-memory reads (a 32 x 64 x 64 product took 2,800 cycles for
// 1,024 of FMAs, with 6 16-byte reads to 32 FMAs a thread) and, for short
// sequences, by the longest CTA.  The training kernels at d 64 take 8 x 16
// threads, which read less (8 to 64) and leave room for three CTAs to an SM: a
// step of 509 tokens 211 -> 197 us, one of 2,048 and 32 + 8 heads 2.99 -> 2.70
// ms.  In small grids a CTA has much of an SM to itself, where one such group
// hides too little latency: two groups take alternate inner tiles, each with
// its own sums (or running softmax), and merge at the end: that step 197 -> 142
// us; a pre-fill of 2 x 333 rows behind 900 tokens 106 us with 16 x 16 threads
// on one tile, 131 with 8 x 16, 92 with two groups.
#include <type_traits>

#include "cap.cuh"
#include "common.cuh"
#include "internal.h"
#include "mix_grad.cuh"

namespace duo {
namespace {

constexpr int TT = 64;              // rows of an inner tile
// Threads that share an inner tile: 16 x 16; 8 x 16 for the training kernels
// at d 64, and in CTAs of 32 rows (small grids), which have two such groups.
template <int D, bool TRAIN, int OT>
__host__ __device__ constexpr int tiled_threads() { return D == 64 && (TRAIN || OT == 32) ? 128 : 256; }
template <int D, int OT>
__host__ __device__ constexpr int tiled_groups() { return D == 64 && OT == 32 ? 2 : 1; }
template <int GROUPS, int TH>
__device__ __forceinline__ void group_sync(int group) {
    if constexpr (GROUPS == 1)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(TH) : "memory");
}

template <int D>
__host__ __device__ constexpr int row_stride() { return D + 4; }
template <int D>
__host__ __device__ constexpr size_t tile_floats(int rows) { return (size_t)rows * row_stride<D>(); }
template <int OT>
__host__ __device__ constexpr int p_stride() { return OT + 4; }   // of the transposed probabilities

// ROWS rows of D elements on their way from global memory to shared memory as
// fp32: fetch (rows where src(r) is NULL are zero), then store.
template <typename T, int D, int ROWS, int TH>
struct Rows {
    static constexpr int N = 16 / (int)sizeof(T), PPR = D / N;   // elements of a 16-byte piece, pieces per row
    static constexpr int kPer = ROWS * PPR / TH;
    uint4 w[kPer];
    template <typename F>
    __device__ __forceinline__ void fetch(int tid, F src) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = tid + k * TH;
            const T* p = src(i / PPR);
            w[k] = p ? reinterpret_cast<const uint4*>(p)[i % PPR] : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    __device__ __forceinline__ void store(int tid, float* dst) const {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = tid + k * TH, r = i / PPR, c = i % PPR * N;
            float v[N];
            load_row_f32<T, N>(reinterpret_cast<const T*>(&w[k]), v);
#pragma unroll
            for (int e = 0; e < N; e += 4)
                *reinterpret_cast<float4*>(dst + r * row_stride<D>() + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
    }
};
template <typename T, int D>
__host__ __device__ constexpr bool prefetches() { return D * sizeof(T) < 512; }

// s[i][j] = X row (RI ty + i) . Y row (tx + 16 j)
template <int D, int RI>
__device__ __forceinline__ void tile_dot(const float* x, const float* y, int tx, int ty, float (&s)[RI][4]) {
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int e = 0; e < D; e += 4) {
        float4 a[RI], b[4];
#pragma unroll
        for (int i = 0; i < RI; ++i) a[i] = *reinterpret_cast<const float4*>(x + (RI * ty + i) * row_stride<D>() + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(y + (tx + 16 * j) * row_stride<D>() + e);
#pragma unroll
        for (int i = 0; i < RI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, s[i][j]))));
    }
}

// acc[i][:] += sum over the tile's 64 inner rows k of pt[k][RI ty + i] * y[k][columns 4 tx + 64 j ..]
template <int D, int RI, int PS>
__device__ __forceinline__ void tile_acc(const float* pt, const float* y, int tx, int ty, float (&acc)[RI][D / 16]) {
#pragma unroll 4
    for (int k = 0; k < TT; ++k) {
        __align__(16) float pr[RI];
        if constexpr (RI % 4 == 0) {
#pragma unroll
            for (int i = 0; i < RI; i += 4)
                *reinterpret_cast<float4*>(pr + i) = *reinterpret_cast<const float4*>(pt + k * PS + RI * ty + i);
        } else {
#pragma unroll
            for (int i = 0; i < RI; i += 2)
                *reinterpret_cast<float2*>(pr + i) = *reinterpret_cast<const float2*>(pt + k * PS + RI * ty + i);
        }
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            const float4 v = *reinterpret_cast<const float4*>(y + k * row_stride<D>() + 4 * tx + 64 * j);
#pragma unroll
            for (int i = 0; i < RI; ++i) {
                acc[i][4 * j] = fmaf(pr[i], v.x, acc[i][4 * j]);
                acc[i][4 * j + 1] = fmaf(pr[i], v.y, acc[i][4 * j + 1]);
                acc[i][4 * j + 2] = fmaf(pr[i], v.z, acc[i][4 * j + 2]);
                acc[i][4 * j + 3] = fmaf(pr[i], v.w, acc[i][4 * j + 3]);
            }
        }
    }
}

// pt[tx + 16 j][RI ty ..] = p[..][j]
template <int RI, int PS>
__device__ __forceinline__ void put_transposed(float* pt, const float (&p)[RI][4], int tx, int ty) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < RI; i += 2)
            *reinterpret_cast<float2*>(pt + (tx + 16 * j) * PS + RI * ty + i) = make_float2(p[i][j], p[i + 1][j]);
}

// Over the 16 threads that hold a row's columns.
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One online-softmax step of a row group: x (log2-domain scores, -inf where
// unseen) becomes p; m, l and acc are brought to the new maximum.
template <int RI, int W>
__device__ __forceinline__ void softmax_step(float (&x)[RI][4], float (&m)[RI], float (&l)[RI], float (&acc)[RI][W]) {
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        const float mn = fmaxf(m[i], row_max(fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3]))));
        const float corr = exp2f(m[i] - mn);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[i][j] = exp2f(x[i][j] - mn);           // mn is at least kNegBig, so -inf gives 0
            sum += x[i][j];
        }
        l[i] = l[i] * corr + sum;                     // this thread's columns; summed over the row at the end
        m[i] = mn;
#pragma unroll
        for (int e = 0; e < W; ++e) acc[i][e] *= corr;
    }
}

// ------------------------------------------------------------------ forward

struct TiledArgs {
    const void* q;         // [B][N][Hq][D]
    const void* k;         // [B][N][Hkv][D]: the chunk (pre-fill) or the sequence (mix)
    const void* v;
    int N;
    void* out;
    const float* alpha;    // mix: [Hkv]
    float* causal;         // mix: A_c and A_s, [B][N][Hq][D]
    float* streaming;
    float* lse;            // mix: [2][B][Hq][N]
};

// What a group has to itself: K, V, P (two of them for the mix), positions.
template <int D, bool MIX, int OT>
__host__ __device__ constexpr size_t group_floats() {
    return 2 * tile_floats<D>(TT) + (MIX ? 2 : 1) * (size_t)TT * p_stride<OT>() + TT;
}
template <int D, bool MIX, int OT>
constexpr size_t forward_smem() {
    return tile_floats<D>(OT) * sizeof(float) + tiled_groups<D, OT>() * group_floats<D, MIX, OT>() * sizeof(float);
}

template <typename T, int D, bool MIX, bool CAP, int OT>
__global__ void __launch_bounds__(tiled_threads<D, MIX, OT>() * tiled_groups<D, OT>())
    tiled_forward_kernel(const LayerArgs a, const CacheArgs c, const TiledArgs s) {
    extern __shared__ __align__(16) float sm[];
    constexpr int TH = tiled_threads<D, MIX, OT>(), GROUPS = tiled_groups<D, OT>();
    constexpr int RI = 16 * OT / TH, PS = p_stride<OT>();   // OT query rows a CTA
    const int tid = threadIdx.x % TH, group = threadIdx.x / TH;
    float* sQ = sm;
    float* sK = sQ + tile_floats<D>(OT) + group * group_floats<D, MIX, OT>();
    float* sV = sK + tile_floats<D>(TT);
    float* sP = sV + tile_floats<D>(TT);
    float* sP2 = sP + TT * PS;                        // mix only
    int* sPos = reinterpret_cast<int*>(sP + (MIX ? 2 : 1) * TT * PS);
    const int tx = tid & 15, ty = tid >> 4;
    const int tiles = (s.N + OT - 1) / OT, heads = a.B * a.Hq;
    // MIX: tile t of every head before the next shorter one (a step of 509 tokens
    // 233 -> 211 us); a pre-fill chunk's tiles are about as long as one another,
    // and a head's tiles side by side keep its keys in L2 (106 us; 119 the other way)
    const int t = MIX ? blockIdx.x / heads : blockIdx.x % tiles, bh = MIX ? blockIdx.x % heads : blockIdx.x / tiles;
    const int b = bh / a.Hq, hq = bh % a.Hq, slot = hq / a.G, g = hq % a.G;
    const int q_idx = a.q_head0[slot] + g, kv_idx = a.kv_head[slot];
    if (!bounds_ok(b < a.B && q_idx >= 0 && q_idx < a.Hq && kv_idx >= 0 && kv_idx < a.Hkv, c.status)) return;
    const int r0 = (tiles - 1 - t) * OT;               // the longest rows first
    const int N = s.N;
    const bool retrieval = MIX || slot < a.R;
    int c0 = 0;
    if constexpr (!MIX) {
        c0 = c.seq_len[b];
        if (c0 < 0 || (retrieval && c0 > a.capacity)) {
            if (threadIdx.x == 0) atomicOr(c.status, DUO_DEV_BAD_LENGTH);
            c0 = c0 < 0 ? 0 : a.capacity;
        }
    }
    if (group == 0) {
        Rows<T, D, OT, TH> q;
        q.fetch(tid, [&](int r) -> const T* {
            return r0 + r < N ? static_cast<const T*>(s.q) + (((size_t)b * N + r0 + r) * a.Hq + q_idx) * D : nullptr;
        });
        q.store(tid, sQ);
    }
    if constexpr (GROUPS > 1) __syncthreads();
    constexpr int W = D / 16;
    float o[RI][W], o2[MIX ? RI : 1][W], m[RI], l[RI], m2[RI], l2[RI];
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        m[i] = m2[i] = kNegBig;
        l[i] = l2[i] = 0.f;
#pragma unroll
        for (int e = 0; e < W; ++e) o[i][e] = 0.f;
    }
    if constexpr (MIX) {
#pragma unroll
        for (int i = 0; i < RI; ++i)
#pragma unroll
            for (int e = 0; e < W; ++e) o2[i][e] = 0.f;
    }
    const float sl = a.scale * kLog2e;
    const int last = min(N, r0 + OT);                 // chunk rows some query of this tile sees
    // key segments: 0 = prior keys from the caches, 1 and 2 = chunk rows
    int begin[3] = {0, 0, 0}, end[3] = {0, last, 0};
    if constexpr (!MIX) {
        end[0] = retrieval ? c0 : a.W;
        if (!retrieval && !a.stream_chunk) {
            end[1] = max(0, min(last, a.sink - c0));  // the chunk's own sink tokens, then the recent band
            begin[2] = max(end[1], r0 - a.recent + 1);
            end[2] = last;
        }
    }
    // the tiles in their order: the first, and the one after (seg, k0)
    int seg = -1, k0 = 0;
    auto step = [&](int& sg, int& k) {
        if (sg >= 0 && k + TT < end[sg]) {
            k += TT;
            return true;
        }
        while (++sg < 3)
            if (begin[sg] < end[sg]) {
                k = begin[sg];
                return true;
            }
        return false;
    };
    Rows<T, D, TT, TH> nk_, nv_;
    auto fetch = [&](int sg, int k) {
        const int n = min(TT, end[sg] - k);
        auto row = [&](int r, const void* full, const void* ring, const void* chunk) -> const T* {
            if (r >= n) return nullptr;
            const int kr = k + r;
            if (MIX || sg > 0) return static_cast<const T*>(chunk) + (((size_t)b * N + kr) * a.Hkv + kv_idx) * D;
            if (retrieval) return static_cast<const T*>(full) + (((size_t)b * a.R + slot) * a.capacity + kr) * D;
            const int pos = c.ring_pos[(size_t)b * a.W + kr];
            if (pos < 0 || pos >= c0) return nullptr;
            return static_cast<const T*>(ring) + (((size_t)b * a.S + (slot - a.R)) * a.W + kr) * D;
        };
        nk_.fetch(tid, [&](int r) { return row(r, c.k_full, c.k_ring, s.k); });
        nv_.fetch(tid, [&](int r) { return row(r, c.v_full, c.v_ring, s.v); });
    };
    // a group's tiles: every one, or every second
    auto step_group = [&](int& sg, int& k) {
        bool there = step(sg, k);
        if (GROUPS > 1 && there) there = step(sg, k);
        return there;
    };
    bool more = step(seg, k0);
    if (group == 1 && more) more = step(seg, k0);
    if (prefetches<T, D>() && more) fetch(seg, k0);
    while (more) {
        const int nk = min(TT, end[seg] - k0);
        group_sync<GROUPS, TH>(group);
        if (!prefetches<T, D>()) fetch(seg, k0);
        nk_.store(tid, sK);
        nv_.store(tid, sV);
        if (tid < TT) {
            const int r = tid;
            int pos = -1;
            if (r < nk) {
                pos = MIX || seg > 0 ? c0 + k0 + r : retrieval ? k0 + r : c.ring_pos[(size_t)b * a.W + k0 + r];
                if (!MIX && seg == 0 && pos >= c0) pos = -1;   // only tokens before the chunk come from the caches
            }
            sPos[r] = pos;
        }
        group_sync<GROUPS, TH>(group);
        int seg1 = seg, k1 = k0;
        more = step_group(seg1, k1);
        if (prefetches<T, D>() && more) fetch(seg1, k1);
        float x[RI][4], x2[RI][4];
        tile_dot<D, RI>(sQ, sK, tx, ty, x);
        // the tile's keys are before the band of every row: no Lambda state (mix)
        const bool lam_tile = MIX && (k0 < a.sink || r0 - (k0 + TT - 1) < a.recent);
        auto scores = [&](auto far) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int pos = sPos[tx + 16 * j];
#pragma unroll
                for (int i = 0; i < RI; ++i) {
                    const int P = c0 + r0 + RI * ty + i;
                    const bool causal = pos >= 0 && pos <= P;
                    const bool lam = causal && (pos < a.sink || (!MIX && a.stream_chunk ? pos >= c0 - a.recent
                                                                                       : P - pos < a.recent));
                    float sc = x[i][j];
                    if constexpr (CAP)
                        sc = cap_exact<decltype(far)::value>(sc, sl, a.cap).s;
                    else
                        sc *= sl;
                    x[i][j] = (MIX || retrieval ? causal : lam) ? sc : -INFINITY;
                    x2[i][j] = lam ? sc : -INFINITY;
                }
            }
        };
        if (CAP && a.cap.far)
            scores(std::true_type{});
        else
            scores(std::false_type{});
        softmax_step<RI, W>(x, m, l, o);
        put_transposed<RI, PS>(sP, x, tx, ty);
        if constexpr (MIX) {
            if (lam_tile) {
                softmax_step<RI, W>(x2, m2, l2, o2);
                put_transposed<RI, PS>(sP2, x2, tx, ty);
            }
        }
        group_sync<GROUPS, TH>(group);
        tile_acc<D, RI, PS>(sP, sV, tx, ty, o);
        if constexpr (MIX) {
            if (lam_tile) tile_acc<D, RI, PS>(sP2, sV, tx, ty, o2);
        }
        seg = seg1;
        k0 = k1;
    }
    if constexpr (GROUPS > 1) {
        // the second group's (m, l, o) through its K and V tiles, merged by the first
        constexpr int kState = RI * (W + 2);
        static_assert((MIX ? 2 : 1) * kState * TH <= 2 * tile_floats<D>(TT), "the tiles hold a group's state");
        float* rec = sQ + tile_floats<D>(OT) + group_floats<D, MIX, OT>() + tid;
        auto put = [&](float* r, const float (&ms)[RI], const float (&ls)[RI], const float (&acc)[RI][W]) {
#pragma unroll
            for (int i = 0; i < RI; ++i) {
                r[(i * (W + 2)) * TH] = ms[i];
                r[(i * (W + 2) + 1) * TH] = ls[i];
#pragma unroll
                for (int e = 0; e < W; ++e) r[(i * (W + 2) + 2 + e) * TH] = acc[i][e];
            }
        };
        auto merge = [&](const float* r, float (&ms)[RI], float (&ls)[RI], float (&acc)[RI][W]) {
#pragma unroll
            for (int i = 0; i < RI; ++i) {
                const float m1 = r[(i * (W + 2)) * TH], mn = fmaxf(ms[i], m1);
                const float w0 = exp2f(ms[i] - mn), w1 = exp2f(m1 - mn);
                ms[i] = mn;
                ls[i] = ls[i] * w0 + r[(i * (W + 2) + 1) * TH] * w1;
#pragma unroll
                for (int e = 0; e < W; ++e) acc[i][e] = acc[i][e] * w0 + r[(i * (W + 2) + 2 + e) * TH] * w1;
            }
        };
        if (group == 1) {
            group_sync<GROUPS, TH>(group);
            put(rec, m, l, o);
            if constexpr (MIX) put(rec + kState * TH, m2, l2, o2);
        }
        __syncthreads();
        if (group == 1) return;
        merge(rec, m, l, o);
        if constexpr (MIX) merge(rec + kState * TH, m2, l2, o2);
    }
    const float al = MIX ? s.alpha[kv_idx] : 0.f;
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        const float ls = row_sum(l[i]), inv = ls > 0.f ? 1.f / ls : 0.f;
        const float ls2 = MIX ? row_sum(l2[i]) : 0.f, inv2 = ls2 > 0.f ? 1.f / ls2 : 0.f;
        const int r = r0 + RI * ty + i;
        if (r >= N) continue;
        const size_t off = (((size_t)b * N + r) * a.Hq + q_idx) * D + 4 * tx;
        if (MIX && tx == 0) {
            const size_t at = ((size_t)b * a.Hq + q_idx) * N + r;
            s.lse[at] = m[i] + log2f(ls);
            s.lse[(size_t)a.B * a.Hq * N + at] = m2[i] + log2f(ls2);
        }
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            float v[4], v2[4], mix[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = o[i][4 * j + e] * inv;
                if constexpr (MIX) {
                    v2[e] = o2[i][4 * j + e] * inv2;
                    mix[e] = al * v[e] + (1.f - al) * v2[e];
                }
            }
            T* out = static_cast<T*>(s.out) + off + 64 * j;
            if constexpr (MIX) {
                store_row<T, 4>(out, mix);
                store_row<float, 4>(s.causal + off + 64 * j, v);
                store_row<float, 4>(s.streaming + off + 64 * j, v2);
            } else {
                store_row<T, 4>(out, v);
            }
        }
    }
}

// ----------------------------------------------------------------- backward
//
// The scheme of mix_grad.cu: keys outer for dK and dV, queries outer for dQ.
// The forward pass kept both attentions in fp32, so D_c and D_s are plain dot
// products here, and both shares of a key are formed one by one (the
// statistics are {lse_c - log2 |a|, D_c, lse_s - log2 |1 - a|, D_s}).

constexpr int kStatRows = 32;      // rows of a CTA, each with the G heads of one KV head
constexpr int kStatWarps = 8;

struct StatArgs {
    const void* dout;      // [B][N][Hq][D]
    const float* causal;   // A_c, [B][N][Hq][D]
    const float* streaming;
    const float* lse;      // [2][B][Hq][N]: causal, Lambda
    const float* alpha;    // [Hkv]
    float* stats;          // [B][Hq][4][n_pad]
    float* part;           // [Hkv][B][chunks] shares of dalpha
    int N, n_pad;
};

template <typename T, int D>
__global__ void __launch_bounds__(kStatWarps * 32) tiled_stats_kernel(const LayerArgs a, const StatArgs x) {
    constexpr int E = D / 32;      // elements a lane
    const int chunks = x.n_pad / kStatRows, chunk = blockIdx.x % chunks, b = blockIdx.x / chunks, kv = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float al = x.alpha[kv];
    const float shift_c = -log2f(fabsf(al)), shift_s = -log2f(fabsf(1.f - al));   // +inf for a closed gate
    const size_t plane = (size_t)a.B * a.Hq * x.N;
    float share = 0.f;
    for (int it = warp; it < kStatRows * a.G; it += kStatWarps) {
        const int i = chunk * kStatRows + it / a.G, h = kv * a.G + it % a.G;
        float* st = x.stats + ((size_t)b * a.Hq + h) * 4 * x.n_pad + i;   // n_pad is whole chunks
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
            dc = fmaf(g, x.causal[o + e], dc);
            ds = fmaf(g, x.streaming[o + e], ds);
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
        x.part[((size_t)kv * a.B + b) * chunks + chunk] = sum;
    }
}

struct TiledGradArgs {
    const void* q;
    const void* dout;
    const void* k;
    const void* v;
    const float* stats;    // [B][Hq][4][n_pad]
    const float* alpha;
    void* d0;              // dK or dQ
    void* d1;              // dV
    const float* part;
    int n_part;
    float* dalpha;
    int32_t* status;
    int N, n_pad;
};

// What a group has to itself: Y0, Y1, the queries' statistics, dS (and W).
template <int D, bool KEYS, int OT>
__host__ __device__ constexpr size_t grad_group_floats() {
    return 2 * tile_floats<D>(TT) + (KEYS ? 2 : 1) * (size_t)TT * p_stride<OT>() + 4 * TT;
}
template <int D, bool KEYS, int OT>
constexpr size_t grad_smem() {
    return (2 * tile_floats<D>(OT) + tiled_groups<D, OT>() * grad_group_floats<D, KEYS, OT>()) * sizeof(float);
}

template <typename T, int D, bool KEYS, bool CAP, int OT>
__global__ void __launch_bounds__(tiled_threads<D, true, OT>() * tiled_groups<D, OT>())
    tiled_grad_kernel(const LayerArgs a, const TiledGradArgs p) {
    extern __shared__ __align__(16) float sm[];
    constexpr int TH = tiled_threads<D, true, OT>(), GROUPS = tiled_groups<D, OT>();
    constexpr int RI = 16 * OT / TH, PS = p_stride<OT>();   // OT outer rows a CTA
    const int tid = threadIdx.x % TH, group = threadIdx.x / TH;
    float* sX0 = sm;
    float* sX1 = sX0 + tile_floats<D>(OT);
    float* sY0 = sX1 + tile_floats<D>(OT) + group * grad_group_floats<D, KEYS, OT>();
    float* sY1 = sY0 + tile_floats<D>(TT);
    float* sStat = sY1 + tile_floats<D>(TT);          // [4][TT] of the tile's queries
    float* sG = sStat + 4 * TT;                       // dS, transposed
    float* sW = sG + TT * PS;                         // W, transposed (keys outer)
    const int tx = tid & 15, ty = tid >> 4;
    const int heads = KEYS ? a.Hkv : a.Hq, N = p.N, tiles = (N + OT - 1) / OT;
    const int t = blockIdx.x / (a.B * heads), bh = blockIdx.x % (a.B * heads), b = bh / heads, head = bh % heads;
    const int kv = KEYS ? head : head / a.G;
    const int ot = KEYS ? t : tiles - 1 - t;                         // the longest of every head first
    const int o0 = ot * OT, n_it = (N + TT - 1) / TT;                // first outer row; inner tiles of the sequence
    auto rows = [&](const void* base, int H, int h, int first) {
        return [=](int r) -> const T* {
            const int i = first + r;
            return i < N ? static_cast<const T*>(base) + (((size_t)b * N + i) * H + h) * D : nullptr;
        };
    };
    auto load_stats = [&](int qh, int first, int n) {
        if (tid < n) {
#pragma unroll
            for (int r = 0; r < 4; ++r) sStat[r * TT + tid] = p.stats[(((size_t)b * a.Hq + qh) * 4 + r) * p.n_pad + first + tid];
        }
    };
    if (!KEYS) load_stats(head, o0, OT);
    if (group == 0) {
        Rows<T, D, OT, TH> x0, x1;
        x0.fetch(tid, KEYS ? rows(p.k, a.Hkv, kv, o0) : rows(p.q, a.Hq, head, o0));
        x1.fetch(tid, KEYS ? rows(p.v, a.Hkv, kv, o0) : rows(p.dout, a.Hq, head, o0));
        x0.store(tid, sX0);
        x1.store(tid, sX1);
    }
    if constexpr (GROUPS > 1) __syncthreads();
    constexpr int W = D / 16;
    float a0[RI][W], a1[KEYS ? RI : 1][W];
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int e = 0; e < W; ++e) {
            a0[i][e] = 0.f;
            if constexpr (KEYS) a1[i][e] = 0.f;
        }
    const float al = p.alpha[kv], sl = a.scale * kLog2e;
    const float sgn_c = al < 0.f ? -1.f : 1.f, sgn_s = 1.f - al < 0.f ? -1.f : 1.f;
    // keys outer: the query tiles from the one that holds row o0 on, of every
    // query head; queries outer: the key tiles up to the diagonal
    const int it0 = KEYS ? o0 / TT : 0, per_head = KEYS ? n_it - it0 : (min(o0 + OT, N) - 1) / TT + 1;
    const int n_in = KEYS ? a.G * per_head : per_head;
    Rows<T, D, TT, TH> y0, y1;
    auto fetch = [&](int j) {
        const int first = (it0 + j % per_head) * TT, qh = kv * a.G + j / per_head;
        y0.fetch(tid, KEYS ? rows(p.q, a.Hq, qh, first) : rows(p.k, a.Hkv, kv, first));
        y1.fetch(tid, KEYS ? rows(p.dout, a.Hq, qh, first) : rows(p.v, a.Hkv, kv, first));
    };
    if (prefetches<T, D>() && group < n_in) fetch(group);
    for (int j0 = group; j0 < n_in; j0 += GROUPS) {
        const int it = it0 + j0 % per_head, qh = KEYS ? kv * a.G + j0 / per_head : head;
        group_sync<GROUPS, TH>(group);
        if (!prefetches<T, D>()) fetch(j0);
        y0.store(tid, sY0);
        y1.store(tid, sY1);
        if (KEYS) load_stats(qh, it * TT, TT);
        group_sync<GROUPS, TH>(group);
        if (prefetches<T, D>() && j0 + GROUPS < n_in) fetch(j0 + GROUPS);
        float x[RI][4], d[RI][4];
        tile_dot<D, RI>(sX0, sY0, tx, ty, x);
        tile_dot<D, RI>(sX1, sY1, tx, ty, d);
        const int i0 = it * TT;                                       // first inner row
        const int query0 = KEYS ? i0 : o0, key0 = KEYS ? o0 : i0, n_keys = KEYS ? OT : TT;
        const bool lam_tile = key0 < a.sink || query0 - (key0 + n_keys - 1) < a.recent;
        auto weights_and_grads = [&](auto far) {
#pragma unroll
            for (int i = 0; i < RI; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int orow = RI * ty + i, icol = tx + 16 * j;
                    const int qr = KEYS ? icol : orow;                    // the query's row in its tile
                    const int query = query0 + qr, key = key0 + (KEYS ? orow : icol);
                    float slope = 1.f, s;
                    if constexpr (CAP) {
                        const Capped c = cap_exact<decltype(far)::value>(x[i][j], sl, a.cap);
                        slope = fmaf(-c.t, c.t, 1.f);
                        s = c.s;
                    } else {
                        s = x[i][j] * sl;
                    }
                    const bool causal = key <= query;
                    const float wc = causal ? sgn_c * exp2f(s - sStat[qr]) : 0.f;
                    float ws = 0.f;
                    if (lam_tile && causal && (key < a.sink || query - key < a.recent))
                        ws = sgn_s * exp2f(s - sStat[2 * TT + qr]);
                    x[i][j] = wc + ws;
                    d[i][j] = slope * (wc * (d[i][j] - sStat[TT + qr]) + ws * (d[i][j] - sStat[3 * TT + qr]));
                }
            }
        };
        if (CAP && a.cap.far)
            weights_and_grads(std::true_type{});
        else
            weights_and_grads(std::false_type{});
        put_transposed<RI, PS>(sG, d, tx, ty);
        if constexpr (KEYS) put_transposed<RI, PS>(sW, x, tx, ty);
        group_sync<GROUPS, TH>(group);
        tile_acc<D, RI, PS>(sG, sY0, tx, ty, a0);
        if constexpr (KEYS) tile_acc<D, RI, PS>(sW, sY1, tx, ty, a1);
    }
    bool stores = true;
    if constexpr (GROUPS > 1) {
        // the second group's sums through its Y0 tile
        static_assert((KEYS ? 2 : 1) * RI * W * TH <= tile_floats<D>(TT), "a tile holds a group's sums");
        float* rec = sX1 + tile_floats<D>(OT) + grad_group_floats<D, KEYS, OT>() + tid;
        stores = group == 0;
        if (!stores) group_sync<GROUPS, TH>(group);
#pragma unroll
        for (int k = 0; k < RI * W; ++k)
            if (!stores) {
                rec[k * TH] = a0[k / W][k % W];
                if constexpr (KEYS) rec[(RI * W + k) * TH] = a1[k / W][k % W];
            }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < RI * W; ++k)
            if (stores) {
                a0[k / W][k % W] += rec[k * TH];
                if constexpr (KEYS) a1[k / W][k % W] += rec[(RI * W + k) * TH];
            }
    }
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        const int r = o0 + RI * ty + i;
        if (!stores || r >= N || !bounds_ok(b < a.B && head < heads, p.status)) continue;
        const size_t off = (((size_t)b * N + r) * heads + head) * D + 4 * tx;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = a0[i][4 * j + e] * a.scale;
            store_row<T, 4>(static_cast<T*>(p.d0) + off + 64 * j, v);
            if constexpr (KEYS) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = a1[i][4 * j + e];
                store_row<T, 4>(static_cast<T*>(p.d1) + off + 64 * j, v);
            }
        }
    }
    if (KEYS && ot == 0 && b == 0 && threadIdx.x < 32)
        sum_shares(p.part + (size_t)kv * p.n_part, p.n_part, &p.dalpha[kv], threadIdx.x);
}

// 64 outer rows a CTA where that still gives every SM two CTAs, else 32: at
// 509 tokens and 16 heads (128 CTAs of 64 rows) a step took 231 us with 64 rows
// and 209 with 32, both with one group of 16 x 16 threads; at 2,048 tokens the
// two differed by less than the noise.
bool few_ctas(const LayerArgs& a, int N, int heads) {
    return (long)a.B * heads * ((N + 63) / 64) < 2L * sm_count();
}

template <typename T, int D, bool MIX, bool CAP, int OT>
cudaError_t launch_forward_rows(const LayerArgs& a, const CacheArgs& c, const TiledArgs& s, cudaStream_t st) {
    constexpr size_t smem = forward_smem<D, MIX, OT>();
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = smem_limit_once(tiled_forward_kernel<T, D, MIX, CAP, OT>, (int)smem, configured);
    if (e != cudaSuccess) return e;
    const long ctas = (long)a.B * a.Hq * ((s.N + OT - 1L) / OT);
    if (ctas > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    tiled_forward_kernel<T, D, MIX, CAP, OT><<<(unsigned)ctas, tiled_threads<D, MIX, OT>() * tiled_groups<D, OT>(), smem, st>>>(a, c, s);
    return cudaGetLastError();
}
template <typename T, int D, bool MIX, bool CAP>
cudaError_t launch_forward(const LayerArgs& a, const CacheArgs& c, const TiledArgs& s, cudaStream_t st) {
    return few_ctas(a, s.N, a.Hq) ? launch_forward_rows<T, D, MIX, CAP, 32>(a, c, s, st)
                                  : launch_forward_rows<T, D, MIX, CAP, 64>(a, c, s, st);
}

template <typename T, int D, bool KEYS, bool CAP, int OT>
cudaError_t launch_grad_rows(const LayerArgs& a, const TiledGradArgs& p, cudaStream_t st) {
    constexpr size_t smem = grad_smem<D, KEYS, OT>();
    static std::atomic<unsigned long long> configured{0};
    const cudaError_t e = smem_limit_once(tiled_grad_kernel<T, D, KEYS, CAP, OT>, (int)smem, configured);
    if (e != cudaSuccess) return e;
    const long ctas = (long)a.B * (KEYS ? a.Hkv : a.Hq) * ((p.N + OT - 1L) / OT);
    if (ctas > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    tiled_grad_kernel<T, D, KEYS, CAP, OT><<<(unsigned)ctas, tiled_threads<D, true, OT>() * tiled_groups<D, OT>(), smem, st>>>(a, p);
    return cudaGetLastError();
}
template <typename T, int D, bool KEYS, bool CAP>
cudaError_t launch_grad(const LayerArgs& a, const TiledGradArgs& p, cudaStream_t st) {
    return few_ctas(a, p.N, KEYS ? a.Hkv : a.Hq) ? launch_grad_rows<T, D, KEYS, CAP, 32>(a, p, st)
                                                 : launch_grad_rows<T, D, KEYS, CAP, 64>(a, p, st);
}

template <typename T, int D>
cudaError_t launch_grads(const LayerArgs& a, TiledGradArgs p, const StatArgs& x, void* dq, cudaStream_t st) {
    const long chunks = (long)a.B * (x.n_pad / kStatRows);
    if (chunks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)chunks, (unsigned)a.Hkv);
    tiled_stats_kernel<T, D><<<grid, kStatWarps * 32, 0, st>>>(a, x);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = a.cap.on ? launch_grad<T, D, true, true>(a, p, st) : launch_grad<T, D, true, false>(a, p, st);
    if (e != cudaSuccess) return e;
    p.d0 = dq;
    p.d1 = nullptr;
    return a.cap.on ? launch_grad<T, D, false, true>(a, p, st) : launch_grad<T, D, false, false>(a, p, st);
}

}  // namespace

cudaError_t launch_tiled_prefill(const LayerArgs& a, const CacheArgs& c, const void* q, const void* k, const void* v,
                                 int C, void* out, cudaStream_t st) {
    if (!a.cap.on) return cudaErrorInvalidConfiguration;
    const TiledArgs s{q, k, v, C, out, nullptr, nullptr, nullptr, nullptr};
    if (a.dtype == DUO_BF16)   // with d 128 a layer the tensor cores take, or one that is refused
        return a.D == 64 ? launch_forward<__nv_bfloat16, 64, false, true>(a, c, s, st) : cudaErrorInvalidConfiguration;
    if (a.D == 128) return launch_forward<float, 128, false, true>(a, c, s, st);
    return launch_forward<float, 64, false, true>(a, c, s, st);
}

cudaError_t launch_tiled_mix(const LayerArgs& a, const float* alpha, const void* q, const void* k, const void* v, int N,
                             void* out, float* causal, float* streaming, float* lse, int32_t* status, cudaStream_t st) {
    const TiledArgs s{q, k, v, N, out, alpha, causal, streaming, lse};
    CacheArgs c{};
    c.status = status;
    auto run = [&](auto t, auto d) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value;
        return a.cap.on ? launch_forward<T, D, true, true>(a, c, s, st) : launch_forward<T, D, true, false>(a, c, s, st);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (a.dtype == DUO_BF16) return a.D == 128 ? run(__nv_bfloat16{}, D128{}) : run(__nv_bfloat16{}, D64{});
    return a.D == 128 ? run(float{}, D128{}) : run(float{}, D64{});
}

cudaError_t launch_tiled_mix_grad(const LayerArgs& a, const MixGradArgs& g, int N, cudaStream_t st) {
    const MixGradPlan pl = mix_grad_plan(a, N);
    const StatArgs x{g.dout, g.causal, g.streaming, g.lse, g.alpha, g.stats, g.part, N, pl.n_pad};
    const TiledGradArgs p{g.q, g.dout, g.k, g.v, g.stats, g.alpha, g.dk, g.dv, g.part, a.B * (pl.n_pad / kStatRows),
                          g.dalpha, g.status, N, pl.n_pad};
    if (a.dtype == DUO_BF16) {
        if (a.D == 128) return launch_grads<__nv_bfloat16, 128>(a, p, x, g.dq, st);
        return launch_grads<__nv_bfloat16, 64>(a, p, x, g.dq, st);
    }
    if (a.D == 128) return launch_grads<float, 128>(a, p, x, g.dq, st);
    return launch_grads<float, 64>(a, p, x, g.dq, st);
}

}  // namespace duo
