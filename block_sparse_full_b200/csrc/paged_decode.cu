// Attention of single query tokens over a paged key/value cache
// (ssa_paged_decode), and over a prefix that a batch shares followed by each
// sequence's own pages (ssa_prefix_decode).
//
// Each key and value is used by the G = Hq / Hkv query heads of its group
// only, so the call is bound by reading the cache once.  The work is the list
// of (sequence, head, row tile of 16 query rows, tile of keys) units, in that
// order, keys fastest; every CTA takes an equal stretch of the list, whatever
// the lengths are (they are read on the device, so a captured launch follows
// them).  A row tile's end counts as one unit more, about what starting and
// joining it costs, so that CTAs with many short sequences get fewer of them
// (64 sequences of up to 1024 tokens, 32/8 heads: 44 us without, 36 with).  Few row
// tiles of few keys have a cluster each instead, see cluster_of.  Walking its stretch a CTA keeps a running maximum, sum and output
// (float32) per row and writes them down as a partial result where a
// (sequence, head, row tile) is split between CTAs; a second kernel joins the
// partials of each row:  h = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
// Which CTAs hold a row's partials follows from the lengths alone, so nothing
// is counted or cleared, and the order of the sums is fixed.  Every share of a row
// counts, also one whose maximum is -inf: its sum may be NaN (the maximum ignores
// NaN scores), or 0 where every score is -inf, and then the row's output is NaN as
// by the formula, however the row was split.
//
// Keys and values come in by 16-byte asynchronous copies through a ring of
// shared-memory stages (3 x 32 KB per CTA and two CTAs per SM keep the
// bandwidth-delay product in flight); rows that are not seen are zero-filled,
// so that nothing left behind in a page reaches the products.  bf16: one warp
// takes 16 keys of a tile, S = Q K^T and O += P V on mma.sync m16n8k16 (a
// tile of 16 query rows cannot fill a larger tensor tile; the prefix of a batch
// of more rows goes to the 128-row kernel of window_fwd_tc.cu); P is rounded to bf16,
// by at most 2^-8 of each weight, to be an operand beside the bf16 values (h against 64
// bits: a relative 0.0020 to 0.0024, its own rounding alone 0.0016).  float32:
// CUDA cores, a warp takes 8 keys.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "device_util.cuh"
#include "ssa_internal.h"

namespace ssa {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kRows = 16;  // query rows of a unit
constexpr int kStages = 3;
constexpr int kFew = 2;  // units that a CTA takes at least: with one, the join of so many partials costs more
                         // (4096 tokens behind 8 sequences: 14.6 us, 14.1 with two, 15 with three)
constexpr float kLn2 = 0.693147180559945309f;

__device__ unsigned int g_paged_status;

template <typename T>
struct Tile {
    static constexpr int keys = sizeof(T) == 2 ? 64 : 32;
};

// One pass over pages: nseq sequences of R query rows per key/value head each
// (row r of sequence b is batch entry b + r / G, head h*G + r % G).
struct Pass {
    const int32_t *table, *lens;  // lens NULL: fixed_len everywhere
    int nseq, R, RT, width, cap, fixed_len, window, sinks;
    int C;         // CTAs
    bool direct;   // rows held by one CTA go to the output, else to its own slot
    int one;       // CTAs of a cluster that takes a row tile, 0: the list of units
    float* part;   // slots [2C + nseq*Hkv*RT] x 16 rows x (D outputs, then m, l)
};

struct DecodeArgs {
    const void *k_pages, *v_pages;
    View q, h;
    float* lse;
    int B, Hq, Hkv, G, page_shift, n_pages;
    long long page_stride;
    float scale_log2;
};

// The tiles of keys that a query sees: [0, ns) and [w0t, end), or one stretch.
struct Seen {
    int len, w0, ns, w0t, nt;
};
__device__ __forceinline__ Seen seen_tiles(const Pass& p, int len, int tk) {
    Seen s;
    s.len = len;
    s.w0 = p.window > 0 && len > p.window ? len - p.window : 0;
    const int send = min(p.sinks, s.w0);
    s.ns = (send + tk - 1) / tk;
    s.w0t = s.w0 / tk;
    s.w0t = max(s.w0t, s.ns);
    s.nt = s.ns + (len + tk - 1) / tk - s.w0t;
    return s;
}
__device__ __forceinline__ int tile_key(const Seen& s, int t, int tk) {
    return (t < s.ns ? t : s.w0t + t - s.ns) * tk;
}
__device__ __forceinline__ bool is_seen(const Seen& s, int sinks, int key) {
    return key < s.len && (key >= s.w0 || key < sinks);
}

__device__ __forceinline__ int seq_len(const Pass& p, int b) {
    if (!p.lens) return p.fixed_len;
    const int n = p.lens[b];
    if (n < 0 || n > p.cap) {
        atomicOr(&g_paged_status, 1u);
        return n < 0 ? 0 : p.cap;
    }
    return n;
}

// Units of a row tile of nt key tiles: those, and one for its end.
__device__ __forceinline__ int units_of(int nt) { return nt > 0 ? nt + 1 : 0; }

// Warp-wide: units of a row tile of each of the sequences before `upto`.
__device__ __forceinline__ long long units_before(const Pass& p, int upto, int tk) {
    long long n = 0;
    for (int b0 = 0; b0 < upto; b0 += 32) {
        const int b = b0 + (int)(threadIdx.x & 31);
        int x = b < upto ? units_of(seen_tiles(p, seq_len(p, b), tk).nt) : 0;
        x = __reduce_add_sync(0xffffffffu, x);
        n += x;
    }
    return n;
}

// CTAs that take part: each has a unit
__device__ __forceinline__ int used_ctas(long long total, int C) {
    const long long n = (total + kFew - 1) / kFew;
    return n < C ? (int)n : C;
}
// first unit of CTA c's stretch, and the CTA whose stretch holds unit u
__device__ __forceinline__ long long stretch(long long total, int C, int c) { return total * c / C; }
__device__ __forceinline__ int cta_of(long long total, int C, long long u) {
    return (int)(((u + 1) * C - 1) / total);  // the largest c with total * c / C <= u
}
// slot of the partial that CTA c holds of the units [u0, u1)
__device__ __forceinline__ size_t slot_of(long long total, int C, int c, long long u0) {
    return 2 * (size_t)c + (stretch(total, C, c) < u0 ? 1 : 0);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t s_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ void put4(float* dst, float4 v, float f) {
    *reinterpret_cast<float4*>(dst) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ void put4(__nv_bfloat16* dst, float4 v, float f) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2(v.x * f, v.y * f), pack2(v.z * f, v.w * f));
}

// A place in the list of units.
struct Cursor {
    long long u;  // unit
    int b, hr, t; // sequence, head and row tile, key tile
    Seen s;
};

// Rows of a unit and their products, by type.  Every warp holds the 16 (or
// fewer) rows against its own keys.
template <typename T, int D, int RG>
struct Rows;

// bf16: fragments of mma.sync m16n8k16 (RG is 16)
template <int D, int RG>
struct Rows<__nv_bfloat16, D, RG> {
    uint32_t q[D / 16][4];
    float o[D / 8][4];
    float m[2], l[2];  // rows lane / 4 and lane / 4 + 8; l is this thread's share

    // the queries of a unit's rows (not needed by maxima() and add(): the loads of
    // the next rows run while the last ones are joined)
    static constexpr bool kEarly = true;
    __device__ __forceinline__ void queries(const DecodeArgs& a, const Pass& p, int b, int h, int r0, float*) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = r0 + (lane >> 2) + 8 * i;
            const __nv_bfloat16* src = nullptr;
            if (r < p.R)
                src = static_cast<const __nv_bfloat16*>(a.q.data) + (size_t)(b + r / a.G) * a.q.sb +
                      (size_t)(h * a.G + r % a.G) * a.q.sh;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    q[k][i + 2 * x] =
                        src ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8 * x + 2 * (lane & 3)) : 0u;
        }
    }
    __device__ __forceinline__ void reset() {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    }

    __device__ __forceinline__ void tile(uint32_t kt, uint32_t vt, int key0, const Seen& s, int sinks,
                                         float scale_log2, const float*) {
        constexpr uint32_t pitch = D * 2;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int mi = lane >> 3, mr = lane & 7;
        float c[2][4] = {};
        {
            const int row = warp * 16 + (mi >> 1) * 8 + mr;
            const uint32_t base = kt + row * pitch;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t f[4];
                ldsm4(base + (((2 * k + (mi & 1)) ^ (row & 7)) << 4), f);
                mma16816(c[0], q[k], f[0], f[1]);
                mma16816(c[1], q[k], f[2], f[3]);
            }
        }
        const int kb = key0 + warp * 16;
        float mx[2] = {-INFINITY, -INFINITY};
        const bool whole = kb + 16 <= s.len && (kb >= s.w0 || kb + 16 <= sinks);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = kb + 8 * n + 2 * (lane & 3) + (e & 1);
                c[n][e] = whole || is_seen(s, sinks, key) ? c[n][e] * scale_log2 : -INFINITY;
                mx[e >> 1] = fmaxf(mx[e >> 1], c[n][e]);
            }
        bool up = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            up = up || mx[i] > m[i];
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float mn = fmaxf(m[i], mx[i]);
                const float al = m[i] == mn ? 1.f : ex2f(m[i] - mn);  // m may be -inf
                m[i] = mn;
                l[i] *= al;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) o[n][2 * i] *= al, o[n][2 * i + 1] *= al;
            }
        }
        const float mz[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                c[n][e] = ex2f(c[n][e] - mz[e >> 1]);
                l[e >> 1] += c[n][e];  // the sum takes the weights before they are rounded to bf16
            }
        const uint32_t pa[4] = {pack2(c[0][0], c[0][1]), pack2(c[0][2], c[0][3]), pack2(c[1][0], c[1][1]),
                                pack2(c[1][2], c[1][3])};
        {
            const int row = warp * 16 + (mi & 1) * 8 + mr;
            const uint32_t base = vt + row * pitch;
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                uint32_t f[4];
                ldsm4t(base + (((2 * n + (mi >> 1)) ^ (row & 7)) << 4), f);
                mma16816(o[2 * n], pa, f[0], f[1]);
                mma16816(o[2 * n + 1], pa, f[2], f[3]);
            }
        }
    }

    // this warp's maxima of its rows -> ml[row]; then its share is added to sum
    __device__ __forceinline__ void maxima(float* dst) const {
        const int lane = threadIdx.x & 31;
        if ((lane & 3) == 0) dst[lane >> 2] = m[0], dst[(lane >> 2) + 8] = m[1];
    }
    // this warp's share of the rows, scaled to the common maximum: stored, or added to what is there
    __device__ __forceinline__ void add(float* sum, float* lsum, const float* top, bool first, int nr) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (lane >> 2) + 8 * i;
            float ls = l[i];
            ls += __shfl_xor_sync(0xffffffffu, ls, 1);
            ls += __shfl_xor_sync(0xffffffffu, ls, 2);
            if (r >= nr) continue;
            const float w = m[i] == -INFINITY ? 0.f : ex2f(m[i] - top[r]);
            if ((lane & 3) == 0) lsum[r] = (first ? 0.f : lsum[r]) + w * ls;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                float2* p = reinterpret_cast<float2*>(sum + r * D + 8 * n + 2 * (lane & 3));
                float2 v = first ? make_float2(0.f, 0.f) : *p;
                v.x += w * o[n][2 * i];
                v.y += w * o[n][2 * i + 1];
                *p = v;
            }
        }
    }
};

// float32: lane = (key of 8, quarter of D) for the scores, 4 columns for the sums
template <int D, int RG>
struct Rows<float, D, RG> {
    float o[RG][4];
    float m[RG], l[RG];
    static constexpr int kCol = D / 4;  // lanes that hold the columns (32, or 16 twice)

    static constexpr bool kEarly = false;
    __device__ __forceinline__ void queries(const DecodeArgs& a, const Pass& p, int b, int h, int r0, float* qs) {
        __syncthreads();  // the unit before has done with qs
        for (int x = threadIdx.x; x < RG * D / 4; x += kThreads) {
            const int r = r0 + x / (D / 4), c = 4 * (x % (D / 4));
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < p.R)
                v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q.data) +
                                                     (size_t)(b + r / a.G) * a.q.sb +
                                                     (size_t)(h * a.G + r % a.G) * a.q.sh + c);
            *reinterpret_cast<float4*>(qs + (x / (D / 4)) * D + c) = v;
        }
        __syncthreads();
    }
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            m[g] = -INFINITY, l[g] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[g][e] = 0.f;
        }
    }

    __device__ __forceinline__ void tile(uint32_t kt, uint32_t vt, int key0, const Seen& s, int sinks,
                                         float scale_log2, const float* qs) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int row = warp * 8 + (lane & 7);
        const float* kr = reinterpret_cast<const float*>(__cvta_shared_to_generic(kt)) + row * D;
        const float* vr = reinterpret_cast<const float*>(__cvta_shared_to_generic(vt));
        float x[RG];
#pragma unroll
        for (int g = 0; g < RG; ++g) x[g] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const int c = (lane >> 3) + 4 * j;
            const float4 k4 = *reinterpret_cast<const float4*>(kr + 4 * (c ^ (row & 7)));
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                const float4 q4 = *reinterpret_cast<const float4*>(qs + g * D + 4 * c);
                x[g] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, x[g]))));
            }
        }
        const bool vis = is_seen(s, sinks, key0 + row);
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            x[g] += __shfl_xor_sync(0xffffffffu, x[g], 8);
            x[g] += __shfl_xor_sync(0xffffffffu, x[g], 16);
            x[g] = vis ? x[g] * scale_log2 : -INFINITY;
            float mx = x[g];
#pragma unroll
            for (int sh = 1; sh < 8; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
            if (mx > m[g]) {  // the same in every lane
                const float al = ex2f(m[g] - mx);
                m[g] = mx;
                l[g] *= al;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[g][e] *= al;
            }
            x[g] = ex2f(x[g] - (m[g] == -INFINITY ? 0.f : m[g]));
            if (lane < 8) l[g] += x[g];
        }
        const int cc = lane & (kCol - 1);
#pragma unroll
        for (int j = 0; j < 8 * kCol / 32; ++j) {
            const int key = kCol == 32 ? j : 2 * j + (lane >> 4);
            const int vrow = warp * 8 + key;
            const float4 v4 = *reinterpret_cast<const float4*>(vr + vrow * D + 4 * (cc ^ (vrow & 7)));
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                const float w = __shfl_sync(0xffffffffu, x[g], key);
                o[g][0] = fmaf(w, v4.x, o[g][0]);
                o[g][1] = fmaf(w, v4.y, o[g][1]);
                o[g][2] = fmaf(w, v4.z, o[g][2]);
                o[g][3] = fmaf(w, v4.w, o[g][3]);
            }
        }
    }

    __device__ __forceinline__ void maxima(float* dst) const {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int g = 0; g < RG; ++g) dst[g] = m[g];
    }
    // this warp's share of the rows, scaled to the common maximum: stored, or added to what is there
    __device__ __forceinline__ void add(float* sum, float* lsum, const float* top, bool first, int nr) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            float ls = l[g];
#pragma unroll
            for (int sh = 1; sh < 8; sh <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, sh);
            if constexpr (kCol == 16)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[g][e] += __shfl_xor_sync(0xffffffffu, o[g][e], 16);
            if (g >= nr) continue;
            const float w = m[g] == -INFINITY ? 0.f : ex2f(m[g] - top[g]);
            if (lane == 0) lsum[g] = (first ? 0.f : lsum[g]) + w * ls;
            if (lane < kCol) {
                float4* p = reinterpret_cast<float4*>(sum + g * D + 4 * lane);
                float4 v = first ? make_float4(0.f, 0.f, 0.f, 0.f) : *p;
                v.x += w * o[g][0], v.y += w * o[g][1], v.z += w * o[g][2], v.w += w * o[g][3];
                *p = v;
            }
        }
    }
};

template <typename T, int D>
constexpr size_t ring_bytes() {
    return (size_t)kStages * 2 * Tile<T>::keys * D * sizeof(T);
}
template <typename T, int D>
constexpr size_t decode_smem() {
    // ring, joined sums [16][D], queries [16][D] (float32 only), maxima [4][16], sums [16], top [16]
    return ring_bytes<T, D>() + kRows * D * 4 * (sizeof(T) == 4 ? 2 : 1) + (kWarps + 2) * kRows * 4;
}

// kOne: a cluster of CTAs takes one row tile, each CTA an equal stretch of its key
// tiles, and joins their shares through distributed shared memory.
template <typename T, int D, int RG, bool kOne>
__global__ void __launch_bounds__(kThreads, 2)
decode_kernel(const DecodeArgs a, const Pass p) {
    constexpr int TK = Tile<T>::keys;
    constexpr int CH = D * (int)sizeof(T) / 16;       // 16-byte chunks of a row
    constexpr int RPP = kThreads / CH;                // rows per pass of the CTA
    constexpr uint32_t TB = TK * D * sizeof(T);       // bytes of a K or V tile
    extern __shared__ __align__(128) uint8_t smem[];
    float* sum = reinterpret_cast<float*>(smem + ring_bytes<T, D>());
    float* qs = sum + kRows * D;
    float* maxs = sum + kRows * D * (sizeof(T) == 4 ? 2 : 1);  // [warp][row]
    float* lsum = maxs + kWarps * kRows;
    float* top = lsum + kRows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int HR = a.Hkv * p.RT;

    Cursor ld;
    long long ubeg, uend;
    bool none = false;  // kOne: the sequence is empty
    if constexpr (kOne) {
        const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
        const int cs = cluster.num_blocks(), rank = cluster.block_rank(), x = (int)blockIdx.x / cs;
        ld.b = x / HR, ld.hr = x % HR;
        ld.s = seen_tiles(p, seq_len(p, ld.b), TK);
        ubeg = ld.s.nt * rank / cs, uend = ld.s.nt * (rank + 1) / cs;
        ld.u = ubeg, ld.t = (int)ubeg;
        none = ld.s.nt == 0;
        if (ubeg == uend) {  // no tile: a share of zeros
            for (int e = threadIdx.x; e < kRows * D; e += kThreads) sum[e] = 0.f;
            if (threadIdx.x < kRows) top[threadIdx.x] = -INFINITY, lsum[threadIdx.x] = 0.f;
        }
    } else {
        launch_dependents();  // every CTA is on its SM: the next kernel's may come in beside them
        const long long total = units_before(p, p.nseq, TK) * HR;
        const int C = used_ctas(total, p.C);
        if ((int)blockIdx.x >= C) {
            wait_for_previous();
            return;
        }
        ubeg = stretch(total, C, blockIdx.x), uend = stretch(total, C, blockIdx.x + 1);
        // the place of unit ubeg: the sequence by a warp-wide scan
        long long before = 0;
        int found = -1;
        for (int b0 = 0; found < 0; b0 += 32) {
            const int b = b0 + lane;
            const int n = b < p.nseq ? units_of(seen_tiles(p, seq_len(p, b), TK).nt) : 0;
            long long inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const uint32_t in = __ballot_sync(0xffffffffu, (before + inc) * HR > ubeg);
            if (in) {
                found = b0 + __ffs(in) - 1;
                before += __shfl_sync(0xffffffffu, inc - n, __ffs(in) - 1);
            } else {
                before += __shfl_sync(0xffffffffu, inc, 31);
                if (b0 + 32 >= p.nseq) {  // cannot be: ubeg < total
                    wait_for_previous();
                    return;
                }
            }
        }
        ld.b = found;
        ld.s = seen_tiles(p, seq_len(p, found), TK);
        const long long r = ubeg - before * HR;
        ld.u = ubeg;
        ld.hr = (int)(r / (ld.s.nt + 1));
        ld.t = (int)(r % (ld.s.nt + 1));
    }
    // the next key tile (a row tile's last unit is none)
    auto advance = [&](Cursor& c) {
        ++c.u;
        if (++c.t < c.s.nt) return;
        if (c.t == c.s.nt) ++c.u;
        c.t = 0;
        if (++c.hr < HR) return;
        c.hr = 0;
        do {
            if (++c.b >= p.nseq) return;  // past the last unit
            c.s = seen_tiles(p, seq_len(p, c.b), TK);
        } while (c.s.nt == 0);
    };
    if constexpr (!kOne) {
        if (ld.t == ld.s.nt) advance(ld);
        if (ld.u >= uend) {  // nothing but an end
            wait_for_previous();
            return;
        }
    }
    Cursor cu = ld;
    // The page numbers of a tile: lane g holds that of its g-th 16 keys (a page
    // holds whole groups of 16), read one unit before the copies need it.
    auto page_of = [&](const Cursor& c) -> int {
        int pg = 0;
        if (lane < TK / 16) {
            const int k0 = tile_key(c.s, c.t, TK) + 16 * lane;
            const bool any = k0 < c.s.len && (k0 + 16 > c.s.w0 || k0 < p.sinks);
            if (any) pg = p.table[(size_t)c.b * p.width + (k0 >> a.page_shift)];
            if (pg < 0 || pg >= a.n_pages) {
                atomicOr(&g_paged_status, 2u);
                pg = 0;
            }
        }
        return pg;
    };
    const int crow = threadIdx.x / CH, ccol = threadIdx.x % CH;
    const uint32_t ring = s_u32(smem);
    const int pmask = (1 << a.page_shift) - 1;
    auto copy = [&](const Cursor& c, int stage, int pg) {
        const int k0 = tile_key(c.s, c.t, TK), hd = c.hr / p.RT;
        const uint32_t dk = ring + stage * 2 * TB;
#pragma unroll
        for (int i = 0; i < TK / RPP; ++i) {
            const int row = crow + i * RPP, key = k0 + row;
            const int pid = __shfl_sync(0xffffffffu, pg, row >> 4);
            const bool ok = is_seen(c.s, p.sinks, key);
            const size_t off = (size_t)pid * a.page_stride +
                               ((size_t)hd * (pmask + 1) + (key & pmask)) * D + ccol * (16 / sizeof(T));
            const uint32_t so = row * (D * (uint32_t)sizeof(T)) + ((ccol ^ (row & 7)) << 4);
            cp_async16(dk + so, static_cast<const T*>(a.k_pages) + off, ok);
            cp_async16(dk + TB + so, static_cast<const T*>(a.v_pages) + off, ok);
        }
    };

    int pg = ld.u < uend ? page_of(ld) : 0;
    auto copy_next = [&](int st) {
        if (ld.u < uend) {
            copy(ld, st, pg);
            advance(ld);
            if (ld.u < uend) pg = page_of(ld);
        }
        cp_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) copy_next(i);
    Rows<T, D, RG> rows;
    int stage = 0;
    int t0 = 0;  // first key tile of the current row tile here
    bool fresh = true, early = false;
    while (cu.u < uend) {
        if (fresh) {
            if (!early) rows.queries(a, p, cu.b, cu.hr / p.RT, (cu.hr % p.RT) * kRows, qs);
            rows.reset();
            t0 = cu.t;
            fresh = false;
        }
        cp_wait<kStages - 2>();
        __syncthreads();  // the tile is there for all, and the stage before is free
        copy_next(stage == 0 ? kStages - 1 : stage - 1);
        const uint32_t kt = ring + stage * 2 * TB;
        rows.tile(kt, kt + TB, tile_key(cu.s, cu.t, TK), cu.s, p.sinks, a.scale_log2, qs);
        stage = stage + 1 == kStages ? 0 : stage + 1;

        const bool last = cu.t + 1 == cu.s.nt;
        Cursor nx = cu;
        advance(nx);
        if (last || nx.u >= uend) {
            // join the warps' shares, in warp order
            early = decltype(rows)::kEarly && nx.u < uend;
            if (early) rows.queries(a, p, nx.b, nx.hr / p.RT, (nx.hr % p.RT) * kRows, qs);
            const int r0 = (cu.hr % p.RT) * kRows, nr = min(kRows, p.R - r0);
            rows.maxima(maxs + warp * kRows);
            __syncthreads();
            if (threadIdx.x < kRows) {
                float t = maxs[threadIdx.x];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) t = fmaxf(t, maxs[w * kRows + threadIdx.x]);
                top[threadIdx.x] = t;
            }
            __syncthreads();
            // up to four rows: every warp has room for its own share, else one after the other
            const bool apart = nr <= kRows / kWarps;
            if (apart) {
                rows.add(sum + warp * 4 * D, lsum + warp * 4, top, true, nr);
                __syncthreads();
            } else {
#pragma unroll 1
                for (int w = 0; w < kWarps; ++w) {
                    if (w == warp) rows.add(sum, lsum, top, w == 0, nr);
                    __syncthreads();
                }
            }
            auto out4 = [&](int x) -> float4 {  // 4 outputs of a row, x = their place in [row][D / 4]
                float4 v = reinterpret_cast<const float4*>(sum)[x];
                if (apart)
#pragma unroll
                    for (int w = 1; w < kWarps; ++w) {
                        const float4 y = reinterpret_cast<const float4*>(sum + w * 4 * D)[x];
                        v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
                    }
                return v;
            };
            auto sum_of = [&](int r) -> float {
                return apart ? (lsum[r] + lsum[4 + r]) + (lsum[8 + r] + lsum[12 + r]) : lsum[r];
            };
            const bool whole = last && t0 == 0;
            const int hd = cu.hr / p.RT;
            if constexpr (kOne) {  // for the other CTAs: the sums at their first place
                for (int x = threadIdx.x; x < nr * D / 4; x += kThreads) reinterpret_cast<float4*>(sum)[x] = out4(x);
                if ((int)threadIdx.x < nr) lsum[threadIdx.x] = sum_of(threadIdx.x);
                break;
            }
            if (whole && p.direct) {
                for (int x = threadIdx.x; x < nr * D / 4; x += kThreads) {
                    const int r = x / (D / 4), c = 4 * (x % (D / 4));
                    const float4 v = out4(x);
                    const float inv = 1.f / sum_of(r);
                    T* dst = static_cast<T*>(a.h.data) + (size_t)(cu.b + (r0 + r) / a.G) * a.h.sb +
                             (size_t)(hd * a.G + (r0 + r) % a.G) * a.h.sh + c;
                    put4(dst, v, inv);
                }
                if ((int)threadIdx.x < nr) {
                    const int r = r0 + threadIdx.x;
                    a.lse[(size_t)(cu.b + r / a.G) * a.Hq + hd * a.G + r % a.G] =
                        (top[threadIdx.x] + log2f(sum_of(threadIdx.x))) * kLn2;
                }
            } else {
                const size_t slot = whole ? 2 * (size_t)p.C + (size_t)cu.b * HR + cu.hr
                                          : 2 * (size_t)blockIdx.x + (cu.u - cu.t > ubeg ? 1 : 0);
                float* dst = p.part + slot * kRows * (D + 2);
                for (int x = threadIdx.x; x < nr * D / 4; x += kThreads)
                    reinterpret_cast<float4*>(dst)[x] = out4(x);
                if ((int)threadIdx.x < nr)
                    *reinterpret_cast<float2*>(dst + kRows * D + 2 * threadIdx.x) =
                        make_float2(top[threadIdx.x], sum_of(threadIdx.x));
            }
            fresh = true;
            __syncthreads();  // sum, top and lsum are free again
        }
        cu = nx;
    }
    cp_wait<0>();
    if constexpr (kOne) {
        const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
        const int cs = cluster.num_blocks(), rank = cluster.block_rank(), x = (int)blockIdx.x / cs;
        const int b = x / HR, hd = x % HR / p.RT, r0 = x % HR % p.RT * kRows, nr = min(kRows, p.R - r0);
        cluster.sync();
        // four outputs to a thread, the shares in the order of the ranks
        for (int e = rank * kThreads + threadIdx.x; e < nr * D / 4; e += cs * kThreads) {
            const int r = e / (D / 4), c = 4 * (e % (D / 4)), head = hd * a.G + r0 + r;
            float M = -INFINITY, L = 0.f;
            for (int k = 0; k < cs; ++k) M = fmaxf(M, cluster.map_shared_rank(top, k)[r]);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < cs; ++k) {
                const float m = cluster.map_shared_rank(top, k)[r];
                const float w = m == -INFINITY ? 0.f : ex2f(m - M);
                const float4 y = reinterpret_cast<const float4*>(cluster.map_shared_rank(sum, k))[e];
                L = fmaf(w, cluster.map_shared_rank(lsum, k)[r], L);
                v.x = fmaf(w, y.x, v.x), v.y = fmaf(w, y.y, v.y), v.z = fmaf(w, y.z, v.z), v.w = fmaf(w, y.w, v.w);
            }
            const float inv = none ? 0.f : 1.f / L;
            put4(static_cast<T*>(a.h.data) + (size_t)b * a.h.sb + (size_t)head * a.h.sh + c, v, inv);
            if (c == 0) a.lse[(size_t)b * a.Hq + head] = none ? -INFINITY : (M + log2f(L)) * kLn2;
        }
        cluster.sync();  // the shares stay until every CTA has read them
        return;
    }
    // The pass over a shared prefix may still be running beside this one; the join
    // waits for this kernel only, so this kernel ends after it.
    wait_for_previous();
}

// Where the partials of a row lie: n slots, one from every CTA c0 .. c0 + n - 1,
// or the row's own slot.
struct Parts {
    int c0, n;
    size_t first, rest;  // slot of the first; the i-th one after it is rest + 2 i
};
__device__ __forceinline__ Parts parts_of(const Pass& p, long long total, long long u0, long long u1, size_t own) {
    Parts r;
    const int C = used_ctas(total, p.C);
    r.c0 = cta_of(total, C, u0);
    r.n = cta_of(total, C, u1 - 1) - r.c0 + 1;
    r.first = r.n == 1 ? own : slot_of(total, C, r.c0, u0);
    r.rest = 2 * (size_t)r.c0;
    return r;
}

// The partials that a row of the tensor-core pass over the prefix left: one of
// every split, 128 rows (nb batch entries) to a slot.  splits = 0: none.
struct PrefixTc {
    const float* part;
    int splits, ntq, nb;
};

// Joins the partials of the rows of one sequence and head.  pre: the pass over
// the shared prefix (nseq = 0: none), or ptc.  Few rows leave several of the eight
// warps to each, all eight where a row has a block of its own: they take its
// partials in turn and are joined in order (one sequence of 65536 tokens, 74
// partials to each of 16 rows: 41 us with two warps to a row, 32 with eight; 64 sequences behind a
// prefix of 32768: 87 us, 101 with a block to each of their 2048 rows).
constexpr int kJoinWarps = 8, kJoinBlocks = 592;  // warps of a block; blocks up to which each row has its own

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
join_kernel(const DecodeArgs a, const Pass p, const Pass pre, const PrefixTc ptc) {
    constexpr int TK = Tile<T>::keys, E = D / 32;  // outputs per lane
    constexpr size_t kSlot = (size_t)kRows * (D + 2);
    __shared__ float2 ml_of[kJoinWarps];
    __shared__ float o_of[kJoinWarps][D];
    const int b = blockIdx.y, h = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int HR = a.Hkv * p.RT;
    const bool alone = gridDim.z > 1;  // a block to a row
    const int per = alone ? 8 : a.G >= 5 ? 1 : a.G >= 3 ? 2 : a.G == 2 ? 4 : 8;  // warps of a row
    const int sub = warp % per;
    // the lengths were there before the passes began: the lists are laid out while they still run
    const Seen s = seen_tiles(p, seq_len(p, b), TK);
    const long long before = units_before(p, b, TK);
    const long long total = units_before(p, p.nseq, TK) * HR;
    for (int g0 = blockIdx.z; g0 < (alone ? (int)blockIdx.z + 1 : a.G); g0 += kJoinWarps / per) {
        const int g = min(g0 + warp / per, a.G - 1);
        const bool row = g0 + warp / per < a.G;
        // own partials: a first one, then every `step` floats; then the prefix's likewise
        const float *own0 = nullptr, *own1 = nullptr, *pre0 = nullptr, *pre1 = nullptr;
        int n_own = 0, n_pre = 0, pr = 0, prows = kRows;
        size_t pstep = 2 * kSlot;
        const int rt = g / kRows, r = g % kRows;
        if (s.nt > 0) {
            const long long u0 = before * HR + (long long)(h * p.RT + rt) * (s.nt + 1);
            const Parts x = parts_of(p, total, u0, u0 + s.nt, 2 * (size_t)p.C + (size_t)b * HR + h * p.RT + rt);
            n_own = x.n;
            own0 = p.part + x.first * kSlot;
            own1 = p.part + x.rest * kSlot;
        }
        if (pre.nseq > 0) {
            const int prow = b * a.G + g, hr = h * pre.RT + prow / kRows;
            const Seen ps = seen_tiles(pre, pre.fixed_len, TK);
            const long long ptotal = (long long)(ps.nt + 1) * a.Hkv * pre.RT;
            pr = prow % kRows;
            const Parts x = parts_of(pre, ptotal, (long long)hr * (ps.nt + 1), (long long)hr * (ps.nt + 1) + ps.nt,
                                     2 * (size_t)pre.C + hr);
            n_pre = x.n;
            pre0 = pre.part + x.first * kSlot;
            pre1 = pre.part + x.rest * kSlot;
        } else if (ptc.splits > 0) {
            prows = 128;
            pr = (b % ptc.nb) * a.G + g;
            n_pre = ptc.splits;
            pstep = (size_t)128 * (D + 2);
            pre0 = pre1 = ptc.part + (size_t)(h * ptc.ntq + b / ptc.nb) * ptc.splits * pstep;
        }
        const bool written = n_pre == 0 && n_own == 1;  // by the pass itself
        const int np = row && !written ? n_own + n_pre : 0;
        auto part = [&](int i) -> const float* {
            if (i < n_own) return i == 0 ? own0 : own1 + i * (2 * kSlot);
            i -= n_own;
            return i == 0 ? pre0 : pre1 + i * pstep;
        };
        wait_for_previous();
        // this warp's partials sub, sub + per, ..: 32 at a time, a lane holding one's (maximum, sum)
        float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        const int mine = (np - sub + per - 1) / per;
        for (int i0 = 0; i0 < mine; i0 += 32) {
            const int m = min(32, mine - i0);
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < m) {
                const int i = sub + (i0 + lane) * per;
                ml = *reinterpret_cast<const float2*>(part(i) + (i < n_own ? kRows * D + 2 * r : prows * D + 2 * pr));
            }
            const float up = fmaxf(M, warp_max(ml.x));
            const float al = M == up ? 1.f : ex2f(M - up);  // both may be -inf
            const float w = ml.x == -INFINITY ? 0.f : ex2f(ml.x - up);
            M = up;
            L = L * al + warp_sum(w * ml.y);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= al;
#pragma unroll 8
            for (int k = 0; k < m; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, k);
                const int i = sub + (i0 + k) * per;
                const float* src = part(i) + (i < n_own ? r : pr) * D + E * lane;
                float x[E];
                if constexpr (E == 4) *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(src);
                else *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(src);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(wk, x[e], acc[e]);
            }
        }
        if (per > 1) {
            __syncthreads();
            if (lane == 0) ml_of[warp] = make_float2(M, L);
#pragma unroll
            for (int e = 0; e < E; ++e) o_of[warp][E * lane + e] = acc[e];
            __syncthreads();
            if (sub == 0) {
                float up = M;
                for (int k = 1; k < per; ++k) up = fmaxf(up, ml_of[warp + k].x);
                const float al = M == -INFINITY ? 0.f : ex2f(M - up);
                L *= al;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] *= al;
                for (int k = 1; k < per; ++k) {
                    const float2 ml = ml_of[warp + k];
                    const float w = ml.x == -INFINITY ? 0.f : ex2f(ml.x - up);
                    L = fmaf(w, ml.y, L);
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = fmaf(w, o_of[warp + k][E * lane + e], acc[e]);
                }
                M = up;
            }
        }
        if (!row || written || sub != 0) continue;
        const bool none = np == 0;  // no key at all
        const float inv = none ? 0.f : 1.f / L;
        T* dst = static_cast<T*>(a.h.data) + (size_t)b * a.h.sb + (size_t)(h * a.G + g) * a.h.sh + E * lane;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int e = 0; e < E; e += 2)
                *reinterpret_cast<uint32_t*>(dst + e) = pack2(acc[e] * inv, acc[e + 1] * inv);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) dst[e] = acc[e] * inv;
        }
        if (lane == 0)
            a.lse[(size_t)b * a.Hq + h * a.G + g] = none ? -INFINITY : (M + log2f(L)) * kLn2;
    }
}

constexpr int kCtas = 296;  // two CTAs on each of 148 SMs
// Row tiles of few keys are a cluster's each, if the GPU holds all clusters at once:
// one launch, no partials in memory.  Eight CTAs a cluster with up to four key tiles
// each, or as many as keep the total at 256, then with up to 16 (at 288 CTAs in
// clusters of eight not all are placed at once: 17 us instead of 11).  16/4 heads of
// 128, window 1024: one sequence 8.6 us, 9.1 by the list of units (and a launch more
// for the host); 32 sequences 17.8 and 21.8; 8, window 4000: 18.2 and 20.3; one,
// window 3000 (6 tiles a CTA): 11.8 and 9.9, so left to the list.
constexpr int kOneCtas = 256;  // CTAs of all clusters at most

template <typename T, int D, int RG>
int launch_pass(const DecodeArgs& a, const Pass& p, bool beside, cudaStream_t s) {
    const int st = opt_in_max_smem<decode_kernel<T, D, RG, false>>("decode_kernel");
    if (st != SSA_OK) return st;
    if (beside)
        return launch_beside("decode_kernel", decode_kernel<T, D, RG, false>, dim3((unsigned)p.C), kThreads,
                             decode_smem<T, D>(), s, a, p);
    decode_kernel<T, D, RG, false><<<p.C, kThreads, decode_smem<T, D>(), s>>>(a, p);
    return check_launch("decode_kernel");
}
// One launch: a cluster to a row tile.
template <typename T, int D, int RG>
int launch_one(const DecodeArgs& a, const Pass& p, cudaStream_t s) {
    const int st = opt_in_max_smem<decode_kernel<T, D, RG, true>>("decode_kernel<cluster>");
    if (st != SSA_OK) return st;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(p.one * p.nseq * a.Hkv * p.RT));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = decode_smem<T, D>();
    c.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)p.one;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&c, decode_kernel<T, D, RG, true>, a, p);
    if (e != cudaSuccess) return fail(SSA_ERR_CUDA, "decode_kernel<cluster>: %s", cudaGetErrorString(e));
    return check_launch("decode_kernel<cluster>");
}
template <typename T, int D>
int run_pass(const DecodeArgs& a, const Pass& p, bool beside, cudaStream_t s) {
    if constexpr (sizeof(T) == 4)  // few rows: fewer registers and products per key
        if (p.R <= 4) return launch_pass<T, D, 4>(a, p, beside, s);
    return launch_pass<T, D, kRows>(a, p, beside, s);
}

template <typename T, int D>
int run(const DecodeArgs& a, const Pass& own, const Pass& pre, const PrefixTc& ptc, cudaStream_t s) {
    int st = SSA_OK;
    if (own.one) {
        if constexpr (sizeof(T) == 4)
            if (own.R <= 4) return launch_one<T, D, 4>(a, own, s);
        return launch_one<T, D, kRows>(a, own, s);
    }
    if (pre.nseq) st = run_pass<T, D>(a, pre, false, s);
    // the sequences' own pages do not wait for the prefix (the kernel ends after it, though)
    if (st == SSA_OK) st = run_pass<T, D>(a, own, pre.nseq || ptc.splits, s);
    if (st != SSA_OK) return st;
    // few sequences leave many partials to a row: a block to each row, as far as that takes about four to an SM
    const unsigned rows = (long long)a.B * a.Hq <= kJoinBlocks ? (unsigned)a.G : 1u;
    return launch_beside("join_kernel", join_kernel<T, D>, dim3((unsigned)a.Hkv, (unsigned)a.B, rows), 32 * kJoinWarps, 0,
                         s, a, own, pre, ptc);
}

int tile_keys(const ssa_cache_params_t& p) { return p.dtype == SSA_BF16 ? 64 : 32; }
int row_tiles(long long R) { return (int)((R + kRows - 1) / kRows); }
// CTAs of a pass: no more than the units that its longest sequences could have
int pass_ctas(long long nseq, long long Hkv, long long RT, long long max_keys, int tk) {
    const long long u = nseq * Hkv * RT * ((max_keys + tk - 1) / tk + 2);
    return (int)(u < kCtas ? u : kCtas);
}
size_t pass_bytes(int C, long long segments, int D) {
    return align_up((2 * (size_t)C + (size_t)segments) * kRows * (D + 2) * sizeof(float), 256);
}
long long seen_most(const ssa_cache_params_t& p) {
    const long long cap = (long long)p.max_pages * p.page;
    const long long w = p.window > 0 ? (long long)p.window + p.sinks + 2 * 64 : cap;
    return w < cap ? w : cap;
}

int cluster_of(const ssa_cache_params_t& p, int RT) {
    const long long tiles = (seen_most(p) + tile_keys(p) - 1) / tile_keys(p), rows = (long long)p.B * p.Hkv * RT;
    for (int cs = 8; cs > 1; cs /= 2)
        if (rows * cs <= kOneCtas) return tiles <= cs * (rows * cs > kOneCtas / 2 ? 16 : 4) ? cs : 0;
    return 0;
}

}  // namespace

size_t paged_decode_workspace(const ssa_cache_params_t& p, int prefix_len) {
    const int G = p.Hq / p.Hkv, RT = row_tiles(G), tk = tile_keys(p);
    // (without a prefix a row tile that one CTA holds is written to the output)
    size_t n = pass_bytes(pass_ctas(p.B, p.Hkv, RT, seen_most(p), tk), prefix_len > 0 ? (long long)p.B * p.Hkv * RT : 0, p.D);
    if (prefix_len > 0 && prefix_tc_supported(p)) {
        n += align_up(prefix_tc_plan(p, prefix_len).bytes, 256);
    } else if (prefix_len > 0) {
        const int PT = row_tiles((long long)p.B * G);
        n += pass_bytes(pass_ctas(1, p.Hkv, PT, prefix_len, tk), (long long)p.Hkv * PT, p.D);
    }
    return n;
}

int launch_paged_decode(const ssa_cache_params_t& p, const View& q, const void* k_pages, const void* v_pages,
                        const int32_t* prefix_pages, int prefix_len, const int32_t* table,
                        const int32_t* lens, const View& h, float* lse, void* ws, cudaStream_t s) {
    const int G = p.Hq / p.Hkv, tk = tile_keys(p);
    DecodeArgs a{};
    a.k_pages = k_pages, a.v_pages = v_pages, a.q = q, a.h = h, a.lse = lse;
    a.B = p.B, a.Hq = p.Hq, a.Hkv = p.Hkv, a.G = G;
    a.page_shift = __builtin_ctz((unsigned)p.page);
    a.n_pages = p.n_pages, a.page_stride = p.page_stride;
    a.scale_log2 = p.sm_scale * 1.4426950408889634f;
    Pass own{}, pre{};
    own.table = table, own.lens = lens, own.nseq = p.B, own.R = G, own.RT = row_tiles(G);
    own.width = p.max_pages, own.cap = p.max_pages * p.page, own.window = p.window;
    own.sinks = p.window > 0 ? p.sinks : 0;
    own.C = pass_ctas(p.B, p.Hkv, own.RT, seen_most(p), tk);
    own.direct = prefix_len == 0;
    own.one = prefix_len == 0 ? cluster_of(p, own.RT) : 0;
    own.part = static_cast<float*>(ws);
    PrefixTc ptc{};
    void* pre_ws = static_cast<char*>(ws) + pass_bytes(own.C, (long long)p.B * p.Hkv * own.RT, p.D);
    if (prefix_len > 0 && prefix_tc_supported(p)) {
        const PrefixPlan plan = prefix_tc_plan(p, prefix_len);
        ptc.part = static_cast<const float*>(pre_ws);
        ptc.splits = plan.splits, ptc.ntq = plan.ntq, ptc.nb = plan.nb;
        const int st = launch_prefix_tc(p, q, k_pages, v_pages, prefix_pages, prefix_len, pre_ws, s);
        if (st != SSA_OK) return st;
    } else if (prefix_len > 0) {
        pre.table = prefix_pages, pre.nseq = 1, pre.R = p.B * G, pre.RT = row_tiles((long long)p.B * G);
        pre.width = 0, pre.cap = pre.fixed_len = prefix_len;
        pre.C = pass_ctas(1, p.Hkv, pre.RT, prefix_len, tk);
        pre.part = static_cast<float*>(pre_ws);
    }
    if (p.dtype == SSA_BF16)
        return p.D == 64 ? run<__nv_bfloat16, 64>(a, own, pre, ptc, s) : run<__nv_bfloat16, 128>(a, own, pre, ptc, s);
    return p.D == 64 ? run<float, 64>(a, own, pre, ptc, s) : run<float, 128>(a, own, pre, ptc, s);
}

int paged_take_status() {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_paged_status, sizeof v);
    if (e != cudaSuccess) return fail(SSA_ERR_CUDA, "status read: %s", cudaGetErrorString(e));
    if (v != 0) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_paged_status, &zero, sizeof zero);
        return fail(SSA_ERR_INVALID_ARG, "paged decode: a %s was out of range", v & 2u ? "page number" : "length");
    }
    return SSA_OK;
}

}  // namespace ssa
