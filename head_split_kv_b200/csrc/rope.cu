// rope.cu -- duo_rope_qk and duo_append_kv_rope: the rotary position embedding
// of queries and keys, alone and on the way into the two caches.
//
// Channel pair i of a row at position p turns by the angle p * inv_freq[i]:
//   (a, b) -> factor * (a cos - b sin, b cos + a sin),
// and the gradient of that map is the same rotation by the negative angle.
// With several axes (time, height, width) pair i takes the position of the
// axis whose section it lies in.
//
// Angles: p * inv_freq reaches 1e6 rad and more, where an fp32 product has
// lost the fraction of a turn that matters, so the product and its reduction
// to half a turn are fp64; the sine and cosine of the reduced angle are fp32,
// with the part of the reduced angle below its fp32 value added to first
// order.  A token's pairs are the same for all of its heads: a CTA takes one
// token and a range of head rows and evaluates each pair's angle once, into
// shared memory.  Each thread first loads the row pieces it will rotate, so
// that the reads of HBM run under the trigonometry.
//
// A head row is cut into units of two 16-byte pieces.  Where the pairs are
// (i, i + rot/2) a unit takes the two pieces whose elements pair up, so both
// results come from registers (and in-place calls need no care); where the
// pairs are neighbours each piece is its own.  Rotations whose half is not a
// whole number of pieces take one pair a unit (element accesses).
//
// Bound: HBM for long chunks (each row read once and written once), launch
// and load latency for a decode step's rows.
#include "common.cuh"
#include "internal.h"
#include "kvq4.cuh"
#include "kvq8.cuh"

namespace duo {
namespace {

constexpr int kRopeThreads = 256;   // most threads of a CTA
constexpr int kAhead = 2;           // units a thread loads before the angles are ready
constexpr int kMaxPairs = 64;       // head_dim / 2

struct RopeKernelArgs {
    RopeArgs r;
    const void* q;
    const void* k;
    const void* v;      // append only
    void* q_out;
    void* k_out;        // rope_qk only
    int T;
    int n_q, n_k, n_v;  // head rows per token of each tensor (0: not given)
    int rows_per_cta;
};

// cos and sin (times factor) of the token's pairs, by the CTA's first threads.
__device__ __forceinline__ void token_angles(const RopeArgs& r, int b, int t, int T, int B, int p_cache,
                                             float2* cs) {
    const int n_pairs = r.rot_dim >> 1;
    for (int i = threadIdx.x; i < n_pairs; i += blockDim.x) {
        const int axis = (i >= r.section_end[0]) + (i >= r.section_end[1]);
        const int p = r.pos ? r.pos[((size_t)axis * B + b) * T + t] : p_cache;
        constexpr double kInvTwoPi = 0.15915494309189533577;
        const double turns = (double)p * ((double)r.inv_freq[i] * kInvTwoPi);
        const double half = 2.0 * (turns - rint(turns));           // half turns in [-1, 1]
        const float hi = (float)half;
        const float lo = (float)(half - (double)hi) * 3.14159265f;  // radians below hi's last bit
        float s, c;
        sincospif(hi, &s, &c);
        const float c2 = fmaf(-s, lo, c);
        const float s2 = fmaf(c, lo, s);
        cs[i] = make_float2(c2 * r.factor, (r.inverse ? -s2 : s2) * r.factor);
    }
}

__device__ __forceinline__ void rotate(float& a, float& b, float2 cs) {
    const float x = a, y = b;
    a = fmaf(x, cs.x, -y * cs.y);
    b = fmaf(y, cs.x, x * cs.y);
}

// One 16-byte piece as fp32 values and back (rounded once).
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void unpack(const uint4& w, float (&o)[8]) {
        o[0] = bf16_lo(w.x); o[1] = bf16_hi(w.x); o[2] = bf16_lo(w.y); o[3] = bf16_hi(w.y);
        o[4] = bf16_lo(w.z); o[5] = bf16_hi(w.z); o[6] = bf16_lo(w.w); o[7] = bf16_hi(w.w);
    }
    __device__ static __forceinline__ uint4 pack(const float (&v)[8]) {
        uint4 w;
        store_row<__nv_bfloat16, 8>(reinterpret_cast<__nv_bfloat16*>(&w), v);
        return w;
    }
};
template <>
struct Piece<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void unpack(const uint4& w, float (&o)[4]) {
        o[0] = __uint_as_float(w.x); o[1] = __uint_as_float(w.y); o[2] = __uint_as_float(w.z); o[3] = __uint_as_float(w.w);
    }
    __device__ static __forceinline__ uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};

// The two pieces of unit u of a row.
struct UnitAt {
    int p0, p1;      // piece indices
    int pair0;       // first pair index of piece 0's elements when they pair with piece 1's; else -1
};
template <typename T>
__device__ __forceinline__ UnitAt unit_at(const RopeArgs& r, bool turned, int u) {
    const int np = (r.rot_dim >> 1) / Piece<T>::N;   // pieces of half a rotation (halves layout)
    if (turned && r.layout == DUO_ROPE_HALVES) {
        if (u < np) return {u, u + np, u * Piece<T>::N};
        return {2 * u, 2 * u + 1, -1};               // 2 np + 2 (u - np)
    }
    return {2 * u, 2 * u + 1, -1};
}

template <typename T>
__device__ __forceinline__ void turn_unit(const RopeArgs& r, const UnitAt& at, const float2* cs, uint4& w0, uint4& w1) {
    constexpr int N = Piece<T>::N;
    if (r.layout == DUO_ROPE_HALVES) {
        if (at.pair0 < 0) return;
        float a[N], b[N];
        Piece<T>::unpack(w0, a);
        Piece<T>::unpack(w1, b);
#pragma unroll
        for (int i = 0; i < N; ++i) rotate(a[i], b[i], cs[at.pair0 + i]);
        w0 = Piece<T>::pack(a);
        w1 = Piece<T>::pack(b);
    } else {
        const int n_pairs = r.rot_dim >> 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint4& w = h ? w1 : w0;
            const int pr = (h ? at.p1 : at.p0) * (N / 2);
            if (pr >= n_pairs) continue;
            float x[N];
            Piece<T>::unpack(w, x);
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (pr + i < n_pairs) rotate(x[2 * i], x[2 * i + 1], cs[pr + i]);
            w = Piece<T>::pack(x);
        }
    }
}

// Where a head row goes: NULL when it is not stored.
struct RowTarget {
    const void* src;
    void* dst;
    bool turned;
};

// Head row `row` of token (b, t): rows 0 .. n_q - 1 are q's, then k's, then
// v's.  For an append the cache row of k and v follows from the position
// p = L + t; status bits are set by the thread that asks with `report`.
template <typename T, bool APPEND>
__device__ __forceinline__ RowTarget row_target(const LayerArgs& a, const CacheArgs& c, const RopeKernelArgs& x,
                                                int b, int t, int row, int L, bool report) {
    const size_t bt = (size_t)b * x.T + t;
    const int D = a.D;
    if (row < x.n_q) {
        const size_t o = (bt * x.n_q + row) * D;
        return {static_cast<const T*>(x.q) + o, static_cast<T*>(x.q_out) + o, true};
    }
    const int kv = row - x.n_q >= x.n_k;              // 0: K, 1: V
    const int h = row - x.n_q - (kv ? x.n_k : 0);
    if constexpr (!APPEND) {
        const size_t o = (bt * x.n_k + h) * D;
        return {static_cast<const T*>(x.k) + o, static_cast<T*>(x.k_out) + o, true};
    } else {
        RowTarget none{nullptr, nullptr, false};
        const T* src = static_cast<const T*>(kv ? x.v : x.k) + (bt * a.Hkv + h) * D;
        const int slot = a.slot_of[h];
        if (!bounds_ok(slot >= 0 && slot < a.R + a.S, c.status)) return none;
        const int p = L + t;
        if (slot < a.R) {
            if (p < 0 || p >= a.capacity) {
                if (report) atomicOr(c.status, DUO_DEV_FULL_CACHE_OVERFLOW);
                return none;
            }
            size_t dst_row;
            if (a.page_size == 0) {
                dst_row = ((size_t)b * a.R + slot) * a.capacity + p;
            } else {
                const int pg = c.page_table[(size_t)b * a.max_pages + p / a.page_size];
                if (pg < 0 || pg >= a.n_pages) {
                    if (report) atomicOr(c.status, DUO_DEV_BAD_PAGE);
                    return none;
                }
                dst_row = ((size_t)pg * a.R + slot) * a.page_size + p % a.page_size;
            }
            return {src, static_cast<T*>(kv ? c.v_full : c.k_full) + dst_row * D, !kv};
        }
        if (p < 0) {
            if (report) atomicOr(c.status, DUO_DEV_BAD_LENGTH);
            return none;
        }
        if (p >= a.sink && t < x.T - a.recent) return none;   // does not survive this append
        const int rs = ring_slot(p, a.sink, a.recent);
        if (!bounds_ok(rs >= 0 && rs < a.W, c.status)) return none;
        if (report && !kv && slot == a.R) c.ring_pos[(size_t)b * a.W + rs] = p;
        const size_t dst_row = ((size_t)b * a.S + (slot - a.R)) * a.W + rs;
        return {src, static_cast<T*>(kv ? c.v_ring : c.k_ring) + dst_row * D, !kv};
    }
}

// The last CTA of the grid advances the lengths: every CTA read them before
// its ticket (acquire-release, so the reads come before and the new lengths
// after).
__device__ __forceinline__ void advance_lengths(const LayerArgs& a, const CacheArgs& c, int T) {
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned n = gridDim.x * gridDim.y;
        uint32_t old;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(&c.counters[0]) : "memory");
        if (old == n - 1) {
            for (int b = 0; b < a.B; ++b) c.seq_len[b] += T;
            c.counters[0] = 0u;
        }
    }
}

// VEC: units of two 16-byte pieces; else one pair (or two elements) a unit.
template <typename T, bool APPEND, bool VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const LayerArgs a, const CacheArgs c,
                                                            const RopeKernelArgs x) {
    __shared__ float2 cs[kMaxPairs];
    const int bt = blockIdx.x;
    const int b = bt / x.T, t = bt - b * x.T;
    const int n_rows = x.n_q + x.n_k + x.n_v;
    const int row0 = blockIdx.y * x.rows_per_cta;
    const int rows = min(x.rows_per_cta, n_rows - row0);
    const int L = c.seq_len ? c.seq_len[b] : 0;
    if constexpr (VEC) {
        const int upr = a.D / (2 * Piece<T>::N);       // units per row
        const int units = rows * upr;
        for (int u0 = threadIdx.x; u0 - (int)threadIdx.x < units; u0 += kAhead * blockDim.x) {
            RowTarget tg[kAhead];
            UnitAt at[kAhead];
            uint4 w[kAhead][2];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int u = u0 + i * blockDim.x;
                tg[i] = {nullptr, nullptr, false};
                if (u < units) {
                    const int row = u / upr, k = u - row * upr;
                    tg[i] = row_target<T, APPEND>(a, c, x, b, t, row0 + row, L, k == 0);
                    at[i] = unit_at<T>(x.r, tg[i].turned, k);
                    if (tg[i].src) {
                        w[i][0] = static_cast<const uint4*>(tg[i].src)[at[i].p0];
                        w[i][1] = static_cast<const uint4*>(tg[i].src)[at[i].p1];
                    }
                }
            }
            if (u0 == (int)threadIdx.x) {              // the first pass: the angles, under those loads
                token_angles(x.r, b, t, x.T, a.B, L + t, cs);
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (!tg[i].src) continue;
                if (tg[i].turned) turn_unit<T>(x.r, at[i], cs, w[i][0], w[i][1]);
                static_cast<uint4*>(tg[i].dst)[at[i].p0] = w[i][0];
                static_cast<uint4*>(tg[i].dst)[at[i].p1] = w[i][1];
            }
        }
    } else {
        token_angles(x.r, b, t, x.T, a.B, L + t, cs);
        __syncthreads();
        const int upr = a.D / 2, half = x.r.rot_dim >> 1;
        for (int u = threadIdx.x; u < rows * upr; u += blockDim.x) {
            const int row = u / upr, k = u - row * upr;
            const RowTarget tg = row_target<T, APPEND>(a, c, x, b, t, row0 + row, L, k == 0);
            if (!tg.src) continue;
            const bool turn = tg.turned && k < half;
            const int e0 = turn ? k : 2 * k, e1 = turn ? k + half : 2 * k + 1;   // halves layout
            const T* s = static_cast<const T*>(tg.src);
            float v0 = Elem<T>::to_f32(s[e0]), v1 = Elem<T>::to_f32(s[e1]);
            if (turn) rotate(v0, v1, cs[k]);
            static_cast<T*>(tg.dst)[e0] = Elem<T>::from_f32(v0);
            static_cast<T*>(tg.dst)[e1] = Elem<T>::from_f32(v1);
        }
    }
    if constexpr (APPEND) advance_lengths(a, c, x.T);
}

// 8- and 4-bit full caches (bf16, head_dim 128): one warp a head row, four
// consecutive elements a lane, as the plain quantizing append.  The rotated
// row is rounded to bf16 before it is quantized, so that the codes are those
// of a rotation followed by an append.
template <int BITS>
__global__ void __launch_bounds__(kRopeThreads) rope_append_q_kernel(const LayerArgs a, const CacheArgs c,
                                                                     const RopeKernelArgs x) {
    using T = __nv_bfloat16;
    __shared__ float2 cs[kMaxPairs];
    const int bt = blockIdx.x;
    const int b = bt / x.T, t = bt - b * x.T;
    const int n_rows = x.n_q + x.n_k + x.n_v;
    const int row0 = blockIdx.y * x.rows_per_cta;
    const int rows = min(x.rows_per_cta, n_rows - row0);
    const int L = c.seq_len[b];
    const int lane = threadIdx.x & 31;
    token_angles(x.r, b, t, x.T, a.B, L + t, cs);
    __syncthreads();
    const int half = x.r.rot_dim >> 1;
    for (int row = threadIdx.x >> 5; row < rows; row += blockDim.x >> 5) {
        const int rr = row0 + row;
        const T* src;
        T* dst = nullptr;
        int slot = -1, kv = 0;
        const int p = L + t;
        if (rr < x.n_q) {
            const size_t o = ((size_t)bt * x.n_q + rr) * 128;
            src = static_cast<const T*>(x.q) + o;
            dst = static_cast<T*>(x.q_out) + o;
        } else {
            kv = rr - x.n_q >= x.n_k;
            const int h = rr - x.n_q - (kv ? x.n_k : 0);
            src = static_cast<const T*>(kv ? x.v : x.k) + ((size_t)bt * a.Hkv + h) * 128;
            slot = a.slot_of[h];
            if (slot < a.R) {
                if (p < 0 || p >= a.capacity) {
                    if (lane == 0) atomicOr(c.status, DUO_DEV_FULL_CACHE_OVERFLOW);
                    continue;
                }
            } else {
                const RowTarget tg = row_target<T, true>(a, c, x, b, t, rr, L, lane == 0);
                if (!tg.dst) continue;
                dst = static_cast<T*>(tg.dst);
            }
        }
        const uint2 w = reinterpret_cast<const uint2*>(src)[lane];
        float e[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
        if (!kv) {
            if (x.r.layout == DUO_ROPE_PAIRS) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (2 * lane + i < half) rotate(e[2 * i], e[2 * i + 1], cs[2 * lane + i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int f = 4 * lane + i;
                    if (f < 2 * half) {
                        const int k = f < half ? f : f - half;
                        float lo = f < half ? e[i] : __bfloat162float(src[k]);
                        float hi = f < half ? __bfloat162float(src[k + half]) : e[i];
                        rotate(lo, hi, cs[k]);
                        e[i] = f < half ? lo : hi;
                    }
                }
            }
        }
        __syncwarp();   // every lane has read its partners before an in-place row is written
        uint2 o;
        store_row<T, 4>(reinterpret_cast<T*>(&o), e);
        if (dst) {
            reinterpret_cast<uint2*>(dst)[lane] = o;
            continue;
        }
        const float xv[4] = {bf16_lo(o.x), bf16_hi(o.x), bf16_lo(o.y), bf16_hi(o.y)};
        float scale;
        if constexpr (BITS == 8) {
            const uint32_t codes = q8_quantize(xv, scale);
            q8_store_row(a, c, kv, b, slot, p, codes, scale, lane);
        } else {
            int codes[4];
            q4_quantize(xv, codes, scale);
            q4_store_row(a, c, kv, b, slot, p, codes, scale, lane);
        }
    }
    advance_lengths(a, c, x.T);
}

// Head rows a CTA takes: as many as its threads hold in kAhead units each,
// fewer when the tokens alone do not fill the SMs (a decode step).
int rows_per_cta(int tokens, int n_rows, int units_per_row, int* threads) {
    int rows = kAhead * kRopeThreads / units_per_row;
    if (rows > n_rows) rows = n_rows;
    const int fill = 2 * sm_count();
    while (rows > 8 && (long)tokens * ((n_rows + rows - 1) / rows) < fill) rows = (rows + 1) / 2;
    // even shares
    const int parts = (n_rows + rows - 1) / rows;
    rows = (n_rows + parts - 1) / parts;
    int th = (rows * units_per_row + kAhead - 1) / kAhead;
    th = (th + 31) / 32 * 32;
    if (th < 64) th = 64;
    if (th > kRopeThreads) th = kRopeThreads;
    *threads = th;
    return rows;
}

template <typename T, bool APPEND>
cudaError_t launch_t(const LayerArgs& a, const CacheArgs& c, RopeKernelArgs x, cudaStream_t s) {
    const int n_rows = x.n_q + x.n_k + x.n_v;
    const long tokens = (long)a.B * x.T;
    if (tokens > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    constexpr int N = Piece<T>::N;
    const bool vec = x.r.layout == DUO_ROPE_PAIRS || (x.r.rot_dim / 2) % N == 0;
    int threads;
    x.rows_per_cta = rows_per_cta((int)tokens, n_rows, a.D / (2 * N), &threads);
    const dim3 grid((unsigned)tokens, (unsigned)((n_rows + x.rows_per_cta - 1) / x.rows_per_cta));
    if (vec)
        rope_kernel<T, APPEND, true><<<grid, threads, 0, s>>>(a, c, x);
    else
        rope_kernel<T, APPEND, false><<<grid, threads, 0, s>>>(a, c, x);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const LayerArgs& a, const int32_t* seq_len, const RopeArgs& r, const void* q, const void* k,
                        void* q_out, void* k_out, int T, cudaStream_t s) {
    CacheArgs c{};
    c.seq_len = const_cast<int32_t*>(seq_len);
    RopeKernelArgs x{r, q, k, nullptr, q_out, k_out, T, q ? a.Hq : 0, k ? a.Hkv : 0, 0, 0};
    return a.dtype == DUO_BF16 ? launch_t<__nv_bfloat16, false>(a, c, x, s) : launch_t<float, false>(a, c, x, s);
}

cudaError_t launch_append_rope(const LayerArgs& a, const CacheArgs& c, const RopeArgs& r, const void* q,
                               const void* k_new, const void* v_new, void* q_out, int T, cudaStream_t s) {
    RopeKernelArgs x{r, q, k_new, v_new, q_out, nullptr, T, q ? a.Hq : 0, a.Hkv, a.Hkv, 0};
    if (a.kv_bits) {
        const int n_rows = x.n_q + 2 * a.Hkv;
        const long tokens = (long)a.B * T;
        if (tokens > 0x7fffffffL) return cudaErrorInvalidConfiguration;
        int threads;
        x.rows_per_cta = rows_per_cta((int)tokens, n_rows, 8, &threads);
        const dim3 grid((unsigned)tokens, (unsigned)((n_rows + x.rows_per_cta - 1) / x.rows_per_cta));
        if (a.kv_bits == 8)
            rope_append_q_kernel<8><<<grid, kRopeThreads, 0, s>>>(a, c, x);
        else
            rope_append_q_kernel<4><<<grid, kRopeThreads, 0, s>>>(a, c, x);
        return cudaGetLastError();
    }
    return a.dtype == DUO_BF16 ? launch_t<__nv_bfloat16, true>(a, c, x, s) : launch_t<float, true>(a, c, x, s);
}

}  // namespace duo
