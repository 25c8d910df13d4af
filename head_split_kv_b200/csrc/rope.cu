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
// token's head rows (or a range of them) and evaluates each pair's angle once,
// into shared memory.  Each thread first loads the row pieces it will rotate --
// their addresses need no length -- so that the reads of HBM run under the
// trigonometry and the look-up of the lengths and pages.  A thread has the same
// place in all of its rows, so it takes its cosines and sines from shared
// memory once.  (A 4,096-token prompt of 32 + 8 heads takes 20 us, 16 when its
// rows are still in L2.  When it took 18 there, a grid of resident CTAs that
// walks the tokens, loading one ahead, took 23 at 80 registers, and two or four
// tokens to a CTA the same as one.)
//
// A head row is cut into units of two 16-byte pieces.  Where the pairs are
// (i, i + rot/2) a unit takes the two pieces whose elements pair up, so both
// results come from registers (and in-place calls need no care); where the
// pairs are neighbours each piece is its own.  Rotations whose pairs do not
// fill whole units take one pair a unit (element accesses).
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
constexpr int kAhead = 2;           // rows a thread loads before it stores the first
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

// cos and sin (times factor) of the pairs of token (b, t), by the CTA's threads.
__device__ __forceinline__ void token_angles(const RopeArgs& r, const int32_t* seq_len, int b, int t, int T, int B,
                                             float* cos_t, float* sin_t) {
    const int n_pairs = r.rot_dim >> 1;
    for (int i = threadIdx.x; i < n_pairs; i += blockDim.x) {
        const int axis = (i >= r.section_end[0]) + (i >= r.section_end[1]);
        const int p = r.pos ? r.pos[((size_t)axis * B + b) * T + t] : (seq_len ? seq_len[b] : 0) + t;
        constexpr double kInvTwoPi = 0.15915494309189533577;
        const double turns = (double)p * ((double)r.inv_freq[i] * kInvTwoPi);
        const double half = 2.0 * (turns - rint(turns));           // half turns in [-1, 1]
        const float hi = (float)half;
        const float lo = (float)(half - (double)hi) * 3.14159265f;  // radians below hi's last bit
        float s, c;
        sincospif(hi, &s, &c);
        const float c2 = fmaf(-s, lo, c);
        const float s2 = fmaf(c, lo, s);
        cos_t[i] = c2 * r.factor;
        sin_t[i] = (r.inverse ? -s2 : s2) * r.factor;
    }
}

__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
    const float x = a, y = b;
    a = fmaf(x, c, -y * s);
    b = fmaf(y, c, x * s);
}
// One 16-byte piece as fp32 pairs and back (rounded once).
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void unpack(const uint4& w, float2 (&o)[4]) {
        o[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
        o[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
        o[2] = make_float2(bf16_lo(w.z), bf16_hi(w.z));
        o[3] = make_float2(bf16_lo(w.w), bf16_hi(w.w));
    }
    __device__ static __forceinline__ uint4 pack(const float2 (&v)[4]) {
        const float f[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
        uint4 w;
        store_row<__nv_bfloat16, 8>(reinterpret_cast<__nv_bfloat16*>(&w), f);
        return w;
    }
};
template <>
struct Piece<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void unpack(const uint4& w, float2 (&o)[2]) {
        o[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
        o[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    __device__ static __forceinline__ uint4 pack(const float2 (&v)[2]) {
        return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
    }
};

// The two pieces of unit u of a row.
template <typename T>
__device__ __forceinline__ void unit_pieces(const RopeArgs& r, bool turned, int u, int& p0, int& p1) {
    const int np = (r.rot_dim >> 1) / Piece<T>::N;    // pieces of half a rotation (halves layout)
    const bool split = turned && r.layout == DUO_ROPE_HALVES && u < np;
    p0 = split ? u : 2 * u;                           // from 2 np on, pieces in order
    p1 = split ? u + np : 2 * u + 1;
}

// Unit u of a row turned by its N pairs' cosines and sines (halves: pair i is
// element i of both pieces; neighbours: piece 0 holds the first N / 2 pairs).
template <typename T>
__device__ __forceinline__ void turn_unit(const RopeArgs& r, const float2 (&c)[Piece<T>::N / 2],
                                          const float2 (&s)[Piece<T>::N / 2], uint4& w0, uint4& w1) {
    constexpr int N = Piece<T>::N;
    float2 a[N / 2], b[N / 2];
    Piece<T>::unpack(w0, a);
    Piece<T>::unpack(w1, b);
    if (r.layout == DUO_ROPE_HALVES) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 x = a[i], y = b[i];
            const float2 ys = fmul2(y, s[i]);
            a[i] = ffma2(x, c[i], make_float2(-ys.x, -ys.y));
            b[i] = ffma2(y, c[i], fmul2(x, s[i]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            rotate(a[2 * i].x, a[2 * i].y, c[i].x, s[i].x);
            rotate(a[2 * i + 1].x, a[2 * i + 1].y, c[i].y, s[i].y);
            rotate(b[2 * i].x, b[2 * i].y, c[N / 4 + i].x, s[N / 4 + i].x);
            rotate(b[2 * i + 1].x, b[2 * i + 1].y, c[N / 4 + i].y, s[N / 4 + i].y);
        }
    }
    w0 = Piece<T>::pack(a);
    w1 = Piece<T>::pack(b);
}

// Head row `row` of token bt: rows 0 .. n_q - 1 are q's, then k's, then v's.
// Where it comes from (NULL: an append of later tokens evicts it; L is the
// sequence's length, or 0 while that is on its way: a negative one, which is
// reported, evicts fewer rows) ...
template <typename T, bool APPEND>
__device__ __forceinline__ const T* row_src(const LayerArgs& a, const RopeKernelArgs& x, size_t bt, int t, int row, int L,
                                            bool& turned) {
    turned = row < x.n_q + x.n_k;
    if (row < x.n_q) return static_cast<const T*>(x.q) + (bt * x.n_q + row) * a.D;
    const int kv = row - x.n_q >= x.n_k, h = row - x.n_q - (kv ? x.n_k : 0);
    if (APPEND && a.slot_of[h] >= a.R && t + min(L, 0) >= a.sink && t < x.T - a.recent) return nullptr;
    return static_cast<const T*>(kv ? x.v : x.k) + (bt * x.n_k + h) * a.D;
}

// ... and where it goes (NULL: not stored).  For an append the cache row of k
// and v follows from the position p = L + t; status bits are set, and the ring
// position is written, by the thread that asks with `report`.
template <typename T, bool APPEND>
__device__ __forceinline__ T* row_dst(const LayerArgs& a, const CacheArgs& c, const RopeKernelArgs& x, size_t bt, int b,
                                      int t, int row, int L, bool report) {
    if (row < x.n_q) return static_cast<T*>(x.q_out) + (bt * x.n_q + row) * a.D;
    const int kv = row - x.n_q >= x.n_k;              // 0: K, 1: V
    const int h = row - x.n_q - (kv ? x.n_k : 0);
    if constexpr (!APPEND) {
        return static_cast<T*>(x.k_out) + (bt * x.n_k + h) * a.D;
    } else {
        const int slot = a.slot_of[h];
        if (!bounds_ok(slot >= 0 && slot < a.R + a.S, c.status)) return nullptr;
        const int p = L + t;
        if (slot < a.R) {
            if (p < 0 || p >= a.capacity) {
                if (report) atomicOr(c.status, DUO_DEV_FULL_CACHE_OVERFLOW);
                return nullptr;
            }
            size_t dst_row;
            if (a.page_size == 0) {
                dst_row = ((size_t)b * a.R + slot) * a.capacity + p;
            } else {
                const int pg = c.page_table[(size_t)b * a.max_pages + p / a.page_size];
                if (pg < 0 || pg >= a.n_pages) {
                    if (report) atomicOr(c.status, DUO_DEV_BAD_PAGE);
                    return nullptr;
                }
                dst_row = ((size_t)pg * a.R + slot) * a.page_size + p % a.page_size;
            }
            return static_cast<T*>(kv ? c.v_full : c.k_full) + dst_row * a.D;
        }
        if (p < 0) {
            if (report) atomicOr(c.status, DUO_DEV_BAD_LENGTH);
            return nullptr;
        }
        if (p >= a.sink && t < x.T - a.recent) return nullptr;   // does not survive this append
        const int rs = ring_slot(p, a.sink, a.recent);
        if (!bounds_ok(rs >= 0 && rs < a.W, c.status)) return nullptr;
        if (report && !kv && slot == a.R) c.ring_pos[(size_t)b * a.W + rs] = p;
        return static_cast<T*>(kv ? c.v_ring : c.k_ring) + (((size_t)b * a.S + (slot - a.R)) * a.W + rs) * a.D;
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

// Rows row0 .. row1 - 1 of a token, one pair (or two elements) at a time.
// skipped: only those that a length of 0 would have evicted.
template <typename T, int D, bool APPEND>
__device__ __forceinline__ void turn_pairs(const LayerArgs& a, const CacheArgs& c, const RopeKernelArgs& x, size_t bt, int b,
                                           int t, int row0, int row1, int L, bool skipped, const float* cos_t,
                                           const float* sin_t) {
    const int half = x.r.rot_dim >> 1;
    for (int u = threadIdx.x; u < (row1 - row0) * (D / 2); u += blockDim.x) {
        const int row = row0 + u / (D / 2), k = u % (D / 2);
        bool turned;
        if (skipped && row_src<T, APPEND>(a, x, bt, t, row, 0, turned)) continue;
        const T* src = row_src<T, APPEND>(a, x, bt, t, row, L, turned);
        T* dst = src ? row_dst<T, APPEND>(a, c, x, bt, b, t, row, L, k == 0) : nullptr;
        if (!dst) continue;
        const bool is_pair = turned && k < half;
        const bool apart = is_pair && x.r.layout == DUO_ROPE_HALVES;
        const int e0 = apart ? k : 2 * k, e1 = apart ? k + half : 2 * k + 1;
        float v0 = Elem<T>::to_f32(src[e0]), v1 = Elem<T>::to_f32(src[e1]);
        if (is_pair) rotate(v0, v1, cos_t[k], sin_t[k]);
        dst[e0] = Elem<T>::from_f32(v0);
        dst[e1] = Elem<T>::from_f32(v1);
    }
}

// VEC: units of two 16-byte pieces, thread (unit, row) walking the rows; else
// one pair (or two elements) a unit.
template <typename T, int D, bool APPEND, bool VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const LayerArgs a, const CacheArgs c,
                                                            const RopeKernelArgs x) {
    __shared__ __align__(16) float cos_t[kMaxPairs], sin_t[kMaxPairs];
    const int bt = blockIdx.x, b = bt / x.T, t = bt - b * x.T;
    const int row0 = blockIdx.y * x.rows_per_cta;
    const int row1 = min(row0 + x.rows_per_cta, x.n_q + x.n_k + x.n_v);
    const int half = x.r.rot_dim >> 1;
    if constexpr (VEC) {
        constexpr int N = Piece<T>::N, kUnits = D / (2 * N);   // units of a row
        const int k = threadIdx.x % kUnits, step = blockDim.x / kUnits;
        const bool turns = k * N < half;               // whole units turn or pass
        float2 cc[N / 2], ss[N / 2];
        int L = 0;
        bool ready = false;
        // every thread of the CTA makes the first pass, for its barrier
        for (int r = row0 + (int)threadIdx.x / kUnits; r < row1 || !ready; r += kAhead * step) {
            const T* src[kAhead];
            bool turned[kAhead];
            int p0[kAhead], p1[kAhead];
            uint4 w[kAhead][2];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int row = r + i * step;
                src[i] = row < row1 ? row_src<T, APPEND>(a, x, bt, t, row, 0, turned[i]) : nullptr;
                if (!src[i]) continue;
                unit_pieces<T>(x.r, turned[i], k, p0[i], p1[i]);
                w[i][0] = reinterpret_cast<const uint4*>(src[i])[p0[i]];
                w[i][1] = reinterpret_cast<const uint4*>(src[i])[p1[i]];
            }
            if (!ready) {                              // the angles, under those loads
                ready = true;
                if (APPEND) L = c.seq_len[b];
                token_angles(x.r, c.seq_len, b, t, x.T, a.B, cos_t, sin_t);
                __syncthreads();
#pragma unroll
                for (int i = 0; i < N / 2; ++i) {
                    const int pr = k * N + 2 * i;
                    cc[i] = turns ? *reinterpret_cast<const float2*>(cos_t + pr) : make_float2(1.f, 1.f);
                    ss[i] = turns ? *reinterpret_cast<const float2*>(sin_t + pr) : make_float2(0.f, 0.f);
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (!src[i]) continue;
                T* dst = row_dst<T, APPEND>(a, c, x, bt, b, t, r + i * step, L, k == 0);
                if (!dst) continue;
                if (turned[i] && turns) turn_unit<T>(x.r, cc, ss, w[i][0], w[i][1]);
                reinterpret_cast<uint4*>(dst)[p0[i]] = w[i][0];
                reinterpret_cast<uint4*>(dst)[p1[i]] = w[i][1];
            }
        }
        if (APPEND && L < 0) turn_pairs<T, D, APPEND>(a, c, x, bt, b, t, row0, row1, L, true, cos_t, sin_t);
    } else {
        const int L = APPEND ? c.seq_len[b] : 0;
        token_angles(x.r, c.seq_len, b, t, x.T, a.B, cos_t, sin_t);
        __syncthreads();
        turn_pairs<T, D, APPEND>(a, c, x, bt, b, t, row0, row1, L, false, cos_t, sin_t);
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
    __shared__ float cos_t[kMaxPairs], sin_t[kMaxPairs];
    const int bt = blockIdx.x;
    const int b = bt / x.T, t = bt - b * x.T;
    const int n_rows = x.n_q + x.n_k + x.n_v;
    const int row0 = blockIdx.y * x.rows_per_cta;
    const int rows = min(x.rows_per_cta, n_rows - row0);
    const int L = c.seq_len[b];
    const int lane = threadIdx.x & 31;
    token_angles(x.r, c.seq_len, b, t, x.T, a.B, cos_t, sin_t);
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
                dst = row_dst<T, true>(a, c, x, bt, b, t, rr, L, lane == 0);
                if (!dst) continue;
            }
        }
        const uint2 w = reinterpret_cast<const uint2*>(src)[lane];
        float e[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
        if (!kv) {
            if (x.r.layout == DUO_ROPE_PAIRS) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (2 * lane + i < half) rotate(e[2 * i], e[2 * i + 1], cos_t[2 * lane + i], sin_t[2 * lane + i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int f = 4 * lane + i;
                    if (f < 2 * half) {
                        const int k = f < half ? f : f - half;
                        float lo = f < half ? e[i] : __bfloat162float(src[k]);
                        float hi = f < half ? __bfloat162float(src[k + half]) : e[i];
                        rotate(lo, hi, cos_t[k], sin_t[k]);
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

template <typename T, int D, bool APPEND>
cudaError_t launch_t(const LayerArgs& a, const CacheArgs& c, RopeKernelArgs x, cudaStream_t s) {
    const int n_rows = x.n_q + x.n_k + x.n_v;
    const long tokens = (long)a.B * x.T;
    if (tokens > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    constexpr int N = Piece<T>::N, kUnits = D / (2 * N);
    const bool vec = (x.r.rot_dim / 2) % N == 0;
    // a CTA's rows: as many as its threads hold in kAhead units each, fewer
    // when the tokens alone do not fill the SMs (a decode step)
    const int room = kAhead * kRopeThreads / kUnits;
    int rows = room < n_rows ? room : n_rows;
    while (rows > 8 && tokens * ((n_rows + rows - 1) / rows) < 2L * sm_count()) rows = (rows + 1) / 2;
    const int parts = (n_rows + rows - 1) / rows;
    x.rows_per_cta = (n_rows + parts - 1) / parts;    // even shares
    int threads = (x.rows_per_cta * kUnits + kAhead - 1) / kAhead;
    threads = (threads + 31) / 32 * 32;               // whole units of a row: kUnits divides 32
    if (threads < 64) threads = 64;
    const dim3 grid((unsigned)tokens, (unsigned)parts);
    if (vec)
        rope_kernel<T, D, APPEND, true><<<grid, threads, 0, s>>>(a, c, x);
    else
        rope_kernel<T, D, APPEND, false><<<grid, threads, 0, s>>>(a, c, x);
    return cudaGetLastError();
}

template <bool APPEND>
cudaError_t launch(const LayerArgs& a, const CacheArgs& c, const RopeKernelArgs& x, cudaStream_t s) {
    if (a.dtype == DUO_BF16)
        return a.D == 128 ? launch_t<__nv_bfloat16, 128, APPEND>(a, c, x, s) : launch_t<__nv_bfloat16, 64, APPEND>(a, c, x, s);
    return a.D == 128 ? launch_t<float, 128, APPEND>(a, c, x, s) : launch_t<float, 64, APPEND>(a, c, x, s);
}

}  // namespace

cudaError_t launch_rope(const LayerArgs& a, const int32_t* seq_len, const RopeArgs& r, const void* q, const void* k,
                        void* q_out, void* k_out, int T, cudaStream_t s) {
    CacheArgs c{};
    c.seq_len = const_cast<int32_t*>(seq_len);
    return launch<false>(a, c, RopeKernelArgs{r, q, k, nullptr, q_out, k_out, T, q ? a.Hq : 0, k ? a.Hkv : 0, 0, 0}, s);
}

cudaError_t launch_append_rope(const LayerArgs& a, const CacheArgs& c, const RopeArgs& r, const void* q,
                               const void* k_new, const void* v_new, void* q_out, int T, cudaStream_t s) {
    RopeKernelArgs x{r, q, k_new, v_new, q_out, nullptr, T, q ? a.Hq : 0, a.Hkv, a.Hkv, 0};
    if (a.kv_bits) {
        const int n_rows = x.n_q + 2 * a.Hkv;
        const long tokens = (long)a.B * T;
        if (tokens > 0x7fffffffL) return cudaErrorInvalidConfiguration;
        // one warp a row, a token's rows spread over CTAs until the SMs are filled
        x.rows_per_cta = n_rows;
        while (x.rows_per_cta > 8 && tokens * ((n_rows + x.rows_per_cta - 1) / x.rows_per_cta) < 2L * sm_count())
            x.rows_per_cta = (x.rows_per_cta + 1) / 2;
        const dim3 grid((unsigned)tokens, (unsigned)((n_rows + x.rows_per_cta - 1) / x.rows_per_cta));
        if (a.kv_bits == 8)
            rope_append_q_kernel<8><<<grid, kRopeThreads, 0, s>>>(a, c, x);
        else
            rope_append_q_kernel<4><<<grid, kRopeThreads, 0, s>>>(a, c, x);
        return cudaGetLastError();
    }
    return launch<true>(a, c, x, s);
}

}  // namespace duo
