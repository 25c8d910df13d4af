// prefill_sched.cuh -- what the two tensor-core attention kernels share: the
// work description, the schedule of key tiles, the masks as column bits, and
// the merge of key-range splits.
#pragma once

#include <cuda.h>

#include "cap.cuh"
#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace duo {

constexpr int BM = 128;            // query rows per tile (prefill_tc.cu: two tiles to a CTA; prefill_capped.cu: one)
constexpr int BN = 128;            // keys per K/V tile
constexpr int HD = 128;            // head dim
constexpr int kBox = 64;           // rows per TMA box (tiles are loaded as 2 x 2 boxes)

constexpr int kMaxRing = 128;      // sink + recent held by one tile
constexpr int kMaxSplit = 8;       // key-range splits per retrieval unit
constexpr int kMinSplitTiles = 48; // no split shorter than 48 key tiles (6,144 keys)
// One query tile's partial record of one split: the lazily raised row maxima
// (log2 domain), the row sums, then O unnormalised as [32 column groups][128
// rows][4], so that a warp's 32 rows write one 512-byte run per group.
constexpr int kPartFloats = 2 * BM + BM * HD;

enum { SRC_CACHE = 0, SRC_CHUNK = 1, SRC_RING = 2 };

struct TcArgs {
    LayerArgs a;
    int C;                 // chunk length
    int n_mpairs;          // ceil(C / 256): pairs of query tiles
    int n_units;           // retrieval units B * R * G * n_mpairs
    int ns;                // CTAs per retrieval unit (key-range splits; 1 = none)
    int n_ret_ctas;        // n_units * ns
    float* part;           // [n_units][ns][2][kPartFloats] partial records (ns > 1)
    uint32_t* ticket;      // [n_units] arrivals; the last split merges them
    EpiArgs epi;           // gated-mix epilogues (EPI_MIX, EPI_DOT)
    TanhPoly poly;         // capped scores: c2 tanh(k x)
    const int32_t* seq_len;
    int32_t* status;
    void* out;
};

// ------------------------------------------------------------ tile schedule
//
// Tiles are listed in visiting order; tile j is described by tile_at(j).
struct Sched {
    bool retrieval;
    bool chunk;      // streaming head in whole-chunk mode: ring, then the chunk causally
    int c0;          // chunk start position (cached tokens before the chunk)
    int m;           // query-tile pair: chunk rows 256m .. 256m+255
    int n;           // tiles visited by Q1
    int n0;          // tiles visited by Q0 (n or n - 1)
    int n_prior;     // retrieval: tiles from the full cache
    int n_ring;      // streaming: ring tiles (0 or 1)
    int sink_tile;   // streaming: 1 if the chunk's tile 0 is listed before the band
    int lo;          // first chunk tile of the band (streaming) / 0 (retrieval)
};

struct Tile {
    int src, row, pos0;
};

__device__ __forceinline__ Sched make_sched(const TcArgs& p, bool retrieval, int c0, int m) {
    const LayerArgs& a = p.a;
    Sched s;
    s.retrieval = retrieval;
    s.c0 = c0;
    s.m = m;
    const int n_ct = (p.C + BN - 1) / BN;                 // chunk tiles that hold keys
    const int hi = min(2 * m + 1, n_ct - 1);              // last chunk tile (Q1's diagonal)
    s.chunk = !retrieval && a.stream_chunk;
    if (retrieval) {
        s.n_prior = (c0 + BN - 1) / BN;
        s.n_ring = 0;
        s.sink_tile = 0;
        s.lo = 0;
        s.n = s.n_prior + hi + 1;
    } else if (s.chunk) {
        s.n_prior = 0;
        s.n_ring = min(c0, a.W) > 0 ? 1 : 0;
        s.sink_tile = 0;
        s.lo = 0;
        s.n = s.n_ring + hi + 1;
    } else {
        s.n_prior = 0;
        s.n_ring = min(c0, a.W) > 0 ? 1 : 0;
        s.lo = max(0, 2 * BM * m - a.recent + 1) / BN;    // first key of Q0's band
        s.sink_tile = (c0 < a.sink && s.lo > 0) ? 1 : 0;  // the chunk's own sink tokens (sink <= 128)
        s.n = s.n_ring + s.sink_tile + (hi - s.lo + 1);
    }
    // Q0's rows end at 256m + 127: the tile 2m + 1, when listed, lies wholly
    // above its diagonal and is the last one
    s.n0 = (hi == 2 * m + 1) ? s.n - 1 : s.n;
    return s;
}

__device__ __forceinline__ Tile tile_at(const Sched& s, int j) {
    Tile t;
    if (s.retrieval) {
        if (j < s.n_prior) {
            t.src = SRC_CACHE;
            t.row = s.c0 - BN * (s.n_prior - j);
            t.pos0 = t.row;
        } else {
            const int u = j - s.n_prior;
            t.src = SRC_CHUNK;
            t.row = BN * u;
            t.pos0 = s.c0 + BN * u;
        }
    } else if (j < s.n_ring) {
        t.src = SRC_RING;
        t.row = 0;
        t.pos0 = 0;
    } else {
        const int k = j - s.n_ring;
        const int u = (s.sink_tile && k == 0) ? 0 : s.lo + k - s.sink_tile;
        t.src = SRC_CHUNK;
        t.row = BN * u;
        t.pos0 = s.c0 + BN * u;
    }
    return t;
}

// Whether query tile `qi` needs the mask on tile j: every Lambda-mode
// streaming tile and ring tile, the retrieval tile that starts before
// position 0, and the chunk tiles that reach past the query tile's first row.
__device__ __forceinline__ bool needs_mask(const Sched& s, const Tile& t, int qi) {
    if (!s.retrieval && !s.chunk) return true;
    if (t.src == SRC_RING) return true;
    if (t.src == SRC_CACHE) return t.row < 0;
    return t.row + BN - 1 > BM * (2 * s.m + qi);
}

// ------------------------------------------------------------------ masks
//
// A row's visible keys in one 128-key tile, set as bits (column c = bit c % 32
// of word c / 32), so that masking costs a bit test per score.  The ranges
// follow from the key positions of the tile:
//   cache / chunk tile, keys pos0 + c: causal (retrieval head, whole-chunk
//     streaming head) c <= P - pos0 and pos0 + c >= 0; Lambda streaming head
//     additionally pos0 + c < sink or pos0 + c > P - recent;
//   ring tile, the streaming cache as it stood at the chunk start c0: slot s
//     < min(c0, sink) holds sink s; the recent slots hold positions
//     max(sink, c0 - recent) .. c0 - 1, position p in slot
//     sink + (p - sink) % recent.  Whole-chunk mode sees all of them, Lambda
//     mode the positions above P - recent.

// columns lo .. hi (inclusive, clipped to the tile)
__device__ __forceinline__ void set_columns(uint32_t (&m)[4], int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, BN - 1);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int a = max(lo - 32 * w, 0), b = min(hi - 32 * w, 31);
        if (a <= b) m[w] |= (0xffffffffu >> (31 - b)) & (0xffffffffu << a);
    }
}

__device__ __forceinline__ void visible_columns(const LayerArgs& a, const Sched& sc, const Tile& t, int P,
                                                uint32_t (&m)[4]) {
    if (t.src != SRC_RING) {
        const int last = P - t.pos0;                      // causal: columns 0 .. last
        if (sc.retrieval || sc.chunk) {
            set_columns(m, -t.pos0, last);
        } else {
            set_columns(m, 0, min(last, a.sink - 1 - t.pos0));
            set_columns(m, P - a.recent + 1 - t.pos0, last);
        }
        return;
    }
    const int c0 = sc.c0;
    set_columns(m, 0, min(c0, a.sink) - 1);               // the sinks
    int lo = max(a.sink, c0 - a.recent);                  // oldest recent position held
    if (!sc.chunk) lo = max(lo, P - a.recent + 1);
    const int len = c0 - lo;                              // positions lo .. c0 - 1
    if (len <= 0) return;
    const int start = (lo - a.sink) % a.recent;           // slot of lo, relative to the recent block
    set_columns(m, a.sink + start, a.sink + min(start + len, a.recent) - 1);
    if (start + len > a.recent) set_columns(m, a.sink, a.sink + start + len - a.recent - 1);
}

struct TcMaps {
    CUtensorMap q, kc, vc, kx, vx, kr, vr, sc;
};

// prefill_capped.cu: EPI_STORE, and EPI_MIX_KEEP with both attentions in the
// one launch (epi.streaming is not read).
cudaError_t launch_prefill_capped(const TcMaps& m, const TcArgs& p, int mode, unsigned grid, cudaStream_t s);

// ------------------------------------------------------------------ split merge
//
// The split that arrives last merges the ns_use records of one query tile,
// row by row (thread = row): the splits' maxima and sums give each record's
// weight, and the weighted sum of the unnormalised O rows over the total
// weight is the row's output.  Not inlined, so that its registers do not
// count against the softmax loop's: the kernel runs at the 168 a thread
// that ten warps leave (an SM sub-partition holds three of them in its 16K
// registers).
static __device__ __noinline__ void merge_split_records(const float* base, int ns_use, int row, bool store,
                                                 __nv_bfloat16* op, int bar_id) {
    constexpr size_t kSplitStride = 2 * (size_t)kPartFloats;
    float w[kMaxSplit];
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int sp = 0; sp < kMaxSplit; ++sp)
        if (sp < ns_use) M = fmaxf(M, __ldcg(base + sp * kSplitStride + row));
#pragma unroll
    for (int sp = 0; sp < kMaxSplit; ++sp) {
        w[sp] = 0.f;
        if (sp < ns_use) {
            const float ms = __ldcg(base + sp * kSplitStride + row);
            w[sp] = ms == -INFINITY ? 0.f : exp2f(ms - M);
            L += w[sp] * __ldcg(base + sp * kSplitStride + BM + row);
        }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll 1
    for (int g8 = 0; g8 < HD / 8; ++g8) {
        float v8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int sp = 0; sp < kMaxSplit; ++sp) {
            if (sp < ns_use) {
                const float4* o4 = reinterpret_cast<const float4*>(base + sp * kSplitStride + 2 * BM);
                const float4 x0 = __ldcg(o4 + (2 * g8) * BM + row);
                const float4 x1 = __ldcg(o4 + (2 * g8 + 1) * BM + row);
                v8[0] += w[sp] * x0.x; v8[1] += w[sp] * x0.y; v8[2] += w[sp] * x0.z; v8[3] += w[sp] * x0.w;
                v8[4] += w[sp] * x1.x; v8[5] += w[sp] * x1.y; v8[6] += w[sp] * x1.z; v8[7] += w[sp] * x1.w;
            }
        }
        if (store) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v8[e] *= inv;
            store_row<__nv_bfloat16, 8>(op + 8 * g8, v8);
        }
    }
    // The records are dead once the warpgroup has read them (only this, the
    // last split of the unit, reads them; every writer took its ticket after
    // a fence): drop their lines from L2 without writing them back, so the
    // splits cost L2 traffic, not DRAM writes.  A record is 520 whole
    // 128-byte lines at a 128-byte-aligned offset of the workspace.
    static_assert(kPartFloats * sizeof(float) % 128 == 0, "records are whole L2 lines");
    constexpr int kLines = (int)(kPartFloats * sizeof(float) / 128);
    asm volatile("bar.sync %0, 128;" ::"r"(bar_id) : "memory");
    for (int sp = 0; sp < ns_use; ++sp)
        for (int ln = row; ln < kLines; ln += BM)
            asm volatile("discard.global.L2 [%0], 128;" ::"l"(base + sp * kSplitStride + (size_t)ln * 32) : "memory");
}

}  // namespace duo
