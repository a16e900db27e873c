// Sliding-window attention with sinks over whole sequences, CUDA-core path
// (float32, or SSA_FLAG_FORCE_SIMT): forward, and the gradients.
//
//   x_ts = sm_scale q_t . k_s over s <= t with s > t - window or s < sinks,
//   p_ts = e^(x_ts - lse_t), h_t = sum_s p_ts v_s;
//   dp_ts = dh_t . v_s, delta_t = dh_t . h_t, ds_ts = p_ts (dp_ts - delta_t) sm_scale,
//   dq_t = sum_s ds_ts k_s, dk_s = sum_t ds_ts q_t, dv_s = sum_t p_ts dh_t.
//
// float32 products run on the FMA pipe, fed from shared memory, whose reads bound
// these kernels: 64 x 64 tiles with rows of D + 4 floats (no bank conflicts), 8 x 4
// scores to a thread.  Only the tiles that the window and the sinks reach
// are visited.  The gradients take two kernels, one per query tile for dq and one
// over key tiles for dk and dv, which run beside one another (each forms delta from
// dh and h itself: 73 us against 93 one after the other with 4 x 4 scores and a
// kernel for delta, for two sequences of 777 tokens, 4/2 heads of 64, window 128,
// 4 sinks, forward included).  A key tile's list of (query head of the group, query
// tile) is one CTA's, or, where there are too few key tiles to fill the SMs and
// for tiles that hold sinks (every later query sees them), is cut into
// stretches whose parts window_parts_kernel sums in order (without: 332 us).
// Clusters of CTAs share a query tile of dq as they do in the forward.  The longest
// tiles start first (4000 tokens, 2/1 heads of 128, all keys, forward: 247 us, 368 in
// ascending order; the FMA pipe is then about 70 % busy; packed f32x2 products measured the same).
#include <cooperative_groups.h>

#include "device_util.cuh"
#include "ssa_internal.h"

namespace ssa {
namespace {

constexpr int BT = 64;  // tokens of a tile
constexpr int kThreads = 256;
constexpr int PP = BT + 4;  // row of a score tile in shared memory
constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.4426950408889634f;

__device__ unsigned int g_window_status;

struct WinArgs {
    View q, k, v, h, dh, dq, dk, dv;
    float* lse;
    const int32_t* lens;
    int B, Hq, Hkv, G, T, window, sinks;
    int nsink, cuts, sink_cuts;  // key tiles with sinks; stretches of a tile's list without and with them
    float* part;                 // [B * Hkv][slots][dk, dv][64][D]
    float sm_scale;
};

// Slots of a head: a tile with one stretch has none.
__host__ __device__ __forceinline__ int first_slot(const WinArgs& a, int tile) {
    const int s = a.sink_cuts > 1 ? a.sink_cuts : 0, c = a.cuts > 1 ? a.cuts : 0;
    return tile < a.nsink ? tile * s : a.nsink * s + (tile - a.nsink) * c;
}

__device__ __forceinline__ int seq_len(const WinArgs& a, int b) {
    if (!a.lens) return a.T;
    const int n = a.lens[b];
    if (n < 0 || n > a.T) {
        atomicOr(&g_window_status, 1u);
        return n < 0 ? 0 : a.T;
    }
    return n;
}
__device__ __forceinline__ bool sees(const WinArgs& a, int t, int s) {
    return s <= t && (t - s < a.window || s < a.sinks);
}
template <typename T>
__device__ __forceinline__ T* at(const View& v, int b, int h, int t) {
    return static_cast<T*>(v.data) + (size_t)b * v.sb + (size_t)h * v.sh + (size_t)t * v.st;
}

// 4 consecutive elements as float32
__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void st4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void st4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
__device__ __forceinline__ void axpy(float w, float4 v, float4& o) {
    o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y), o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
}

// Key tiles of the queries t0 .. tl: [0, ns) with sinks only, then [w0, w0 + nw).
struct KeyTiles {
    int ns, w0, n;
    __device__ KeyTiles(const WinArgs& a, int t0, int tl) {
        const int lo = max(0, t0 - (a.window - 1));
        ns = (min(a.sinks, lo) + BT - 1) / BT;
        w0 = max(lo / BT, ns);
        n = ns + tl / BT + 1 - w0;
    }
    __device__ int tile(int j) const { return j < ns ? j : w0 + j - ns; }
};

template <int D>
constexpr size_t tile_floats() { return (size_t)BT * (D + 4); }

// Forward: groups of 128 threads walk the key tiles in turn, each with its own
// buffers, running maximum, sum and output, and are joined at the end in group
// order.  A thread holds 8 rows x 4 keys of the scores and 8 x D / 16 outputs (8 x 8
// scores in groups of 64 threads: 100 tokens, D = 64: 17.7 us instead of 12.8).
// Key and value tiles are on their way while the other is in use.  Where the
// query tiles do not fill the SMs a cluster of CTAs shares one, tile by tile,
// and reads the others' shares through distributed shared memory (1000 tokens, 2
// heads of 64, window 256: 32 us with one CTA to a query tile, 17 with four).
template <int D>
struct Fwd {
    static constexpr int kGroup = 128, kGroups = D == 64 ? 4 : 2;  // threads of a group; groups
    static constexpr int TX = kGroup / 8, KT = BT / TX;            // key columns of threads; keys of a thread
    static constexpr int NC = D / (4 * TX);                        // outputs of a thread in a row, four each
    static constexpr size_t kFloats = 2 * (size_t)BT * (D + 4) + BT * PP;  // K, V, P of a group
    static constexpr size_t smem = (BT * (D + 4) + kGroups * kFloats) * sizeof(float);
};

// Rows t0 .. of one head -> shared memory, by the n threads of a group; rows from
// len on are zero.  float32 is copied asynchronously, bf16 converted on the way.
template <typename T, int D>
__device__ __forceinline__ void stage(float* dst, const View& v, int b, int h, int t0, int len, int tid, int n) {
    constexpr int kAll = BT * D / 4;
    if constexpr (sizeof(T) == 4) {
        for (int e = tid; e < kAll; e += n) {
            const int r = e / (D / 4), c = 4 * (e % (D / 4));
            const bool in = t0 + r < len;
            const T* src = at<const T>(v, b, h, in ? t0 + r : 0) + c;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             static_cast<uint32_t>(__cvta_generic_to_shared(dst + r * (D + 4) + c))),
                         "l"(src), "r"(in ? 16 : 0)
                         : "memory");
        }
    } else {
#pragma unroll 8
        for (int e = tid; e < kAll; e += n) {
            const int r = e / (D / 4), c = 4 * (e % (D / 4));
            *reinterpret_cast<float4*>(dst + r * (D + 4) + c) =
                t0 + r < len ? ld4(at<const T>(v, b, h, t0 + r) + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <typename T, int D>
__global__ void __launch_bounds__(Fwd<D>::kGroup* Fwd<D>::kGroups, 1)
window_fwd_simt_kernel(const WinArgs a) {
    using F = Fwd<D>;
    constexpr int TX = F::TX, KT = F::KT, G = F::kGroups;
    extern __shared__ __align__(16) float sm[];
    const int group = threadIdx.x / F::kGroup, tid = threadIdx.x % F::kGroup;
    float *Q = sm, *K = Q + BT * (D + 4) + group * F::kFloats, *V = K + BT * (D + 4), *P = V + BT * (D + 4);
    auto sync = [group] { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(F::kGroup) : "memory"); };
    auto wait1 = [] { asm volatile("cp.async.wait_group 1;" ::: "memory"); };
    const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int cs = cluster.num_blocks(), rank = cluster.block_rank();
    // (the last tiles of all heads first: without a window they have the most keys)
    const int x = blockIdx.x / cs, hq = x % a.Hq, b = x / a.Hq % a.B, hk = hq / a.G;
    const int t0 = ((a.T + BT - 1) / BT - 1 - x / (a.Hq * a.B)) * BT;
    const int first = rank + cs * group, step = cs * G;  // this group's key tiles: CTAs first
    const int tx = tid % TX, ty = tid / TX;  // rows ty + 8 i, keys tx + TX j
    const int len = seq_len(a, b);
    float4 o[8][F::NC];
    float m[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < F::NC; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (t0 < len) {
        const float sl2 = a.sm_scale * kLog2e;
        const KeyTiles kt(a, t0, min(t0 + BT, len) - 1);
        stage<T, D>(Q, a.q, b, hq, t0, len, threadIdx.x, F::kGroup * G);
        if (first < kt.n) {
            stage<T, D>(K, a.k, b, hk, kt.tile(first) * BT, len, tid, F::kGroup);
            stage<T, D>(V, a.v, b, hk, kt.tile(first) * BT, len, tid, F::kGroup);
        }
        // the queries are the oldest copies of every thread: there once the keys are
        if (first < kt.n) wait1();
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        for (int j = first; j < kt.n; j += step) {
            const int s0 = kt.tile(j) * BT;
            wait1();
            sync();  // the keys are there
            float s[8][KT];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int x = 0; x < KT; ++x) s[i][x] = 0.f;
#pragma unroll 2
            for (int d = 0; d < D; d += 4) {
                float4 q[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] = ld4(Q + (ty + 8 * i) * (D + 4) + d);
#pragma unroll
                for (int x = 0; x < KT; ++x) {
                    const float4 k = ld4(K + (tx + TX * x) * (D + 4) + d);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[i][x] = dot4(q[i], k, s[i][x]);
                }
            }
            sync();  // the keys are used up
            if (j + step < kt.n) stage<T, D>(K, a.k, b, hk, kt.tile(j + step) * BT, len, tid, F::kGroup);
            else asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = t0 + ty + 8 * i;
                float mx = -INFINITY;
#pragma unroll
                for (int x = 0; x < KT; ++x) {
                    s[i][x] = sees(a, t, s0 + tx + TX * x) ? s[i][x] * sl2 : -INFINITY;
                    mx = fmaxf(mx, s[i][x]);
                }
#pragma unroll
                for (int sh = 1; sh < TX; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
                const float mn = fmaxf(m[i], mx), mz = mn == -INFINITY ? 0.f : mn;
                const float al = exp2f(m[i] - mz);
                m[i] = mn;
                l[i] *= al;
#pragma unroll
                for (int c = 0; c < F::NC; ++c) o[i][c].x *= al, o[i][c].y *= al, o[i][c].z *= al, o[i][c].w *= al;
#pragma unroll
                for (int x = 0; x < KT; ++x) {
                    const float p = exp2f(s[i][x] - mz);
                    l[i] += p;
                    P[(ty + 8 * i) * PP + tx + TX * x] = p;
                }
            }
            wait1();
            sync();  // weights and values are there
#pragma unroll 2
            for (int n = 0; n < BT; n += 4) {
                float4 w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = ld4(P + (ty + 8 * i) * PP + n);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int c = 0; c < F::NC; ++c) {
                        const float4 v = ld4(V + (n + k) * (D + 4) + 4 * tx + 4 * TX * c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) axpy((&w[i].x)[k], v, o[i][c]);
                    }
            }
            sync();  // and used up
            if (j + step < kt.n) stage<T, D>(V, a.v, b, hk, kt.tile(j + step) * BT, len, tid, F::kGroup);
            else asm volatile("cp.async.commit_group;" ::: "memory");
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int sh = 1; sh < TX; sh <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], sh);
    // every group's share goes over its own tiles
    sync();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int c = 0; c < F::NC; ++c) *reinterpret_cast<float4*>(K + (ty + 8 * i) * (D + 4) + 4 * tx + 4 * TX * c) = o[i][c];
        if (tx == 0) P[2 * (ty + 8 * i)] = m[i], P[2 * (ty + 8 * i) + 1] = l[i];
    }
    if (cs > 1) cluster.sync();
    else __syncthreads();
    // and the threads of all CTAs join them, four outputs each
    constexpr int kAll = F::kGroup * G;
    for (int e = rank * kAll + threadIdx.x; e < BT * D / 4; e += cs * kAll) {
        const int r = e / (D / 4), c = 4 * (e % (D / 4)), t = t0 + r;
        if (t >= a.T) continue;
        float mx = -INFINITY, L = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < len) {
            for (int g = 0; g < G; ++g)
                for (int k = 0; k < cs; ++k) {
                    const float* own = sm + BT * (D + 4) + g * F::kFloats;
                    const float* base = k == rank ? own : cluster.map_shared_rank(own, k);
                    const float2 ml = *reinterpret_cast<const float2*>(base + 2 * BT * (D + 4) + 2 * r);
                    if (ml.x == -INFINITY && ml.y == 0.f) continue;  // nothing seen (a sum of NaN counts)
                    const float mn = fmaxf(mx, ml.x), w0 = exp2f(mx - mn), w1 = exp2f(ml.x - mn);
                    mx = mn;
                    L = fmaf(L, w0, w1 * ml.y);
                    x.x *= w0, x.y *= w0, x.z *= w0, x.w *= w0;
                    axpy(w1, ld4(base + r * (D + 4) + c), x);
                }
            const float inv = 1.f / L;
            x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
        }
        st4(at<T>(a.h, b, hq, t) + c, x);
        if (c == 0) a.lse[((size_t)b * a.Hq + hq) * a.T + t] = t < len ? (mx + log2f(L)) * kLn2 : -INFINITY;
    }
    if (cs > 1) cluster.sync();  // the shares stay until every CTA has read them
}

// Gradients: two groups of 128 threads.  The first forms q k^T and from it p, the
// second dh v^T and, once p is in shared memory, ds.  A thread holds 8 x 4 scores
// (rows row_of(ty, i): its warp's other half lies 4 rows on, in other banks;
// keys tx + 16 x) and 8 x D / 16 outputs: 12 reads of 16 bytes to 128 FMAs, where
// 4 x 4 scores take 16.
constexpr int kHalf = kThreads / 2;

__device__ __forceinline__ int row_of(int ty, int i) { return 16 * (ty >> 1) + 4 * (ty & 1) + (i & 3) + 8 * (i >> 2); }

// Rows t0 .. t0 + 63 of one head -> shared memory; rows from len on are zero,
// whatever is stored there.
template <typename T, int D>
__device__ __forceinline__ void load_tile(const View& v, int b, int h, int t0, int len, float* dst) {
    constexpr int L = D / 4, N = BT * L / kThreads;
    float4 x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = threadIdx.x + i * kThreads, r = e / L, c = 4 * (e % L);
        x[i] = t0 + r < len ? ld4(at<const T>(v, b, h, t0 + r) + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = threadIdx.x + i * kThreads, r = e / L, c = 4 * (e % L);
        *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = x[i];
    }
}

// A tile of q and dh, and of its rows' values: -lse log2 e and delta = dh . h.
template <typename T, int D>
__device__ __forceinline__ void load_queries(const WinArgs& a, int b, int hq, int t0, int len, float* Q, float* dO,
                                             float* row) {
    constexpr int L = D / 4, N = BT * L / kThreads;
    float4 x[N], y[N], z[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = threadIdx.x + i * kThreads, r = e / L, c = 4 * (e % L);
        x[i] = y[i] = z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t0 + r < len) {
            x[i] = ld4(at<const T>(a.q, b, hq, t0 + r) + c);
            y[i] = ld4(at<const T>(a.dh, b, hq, t0 + r) + c);
            z[i] = ld4(at<const T>(a.h, b, hq, t0 + r) + c);
        }
    }
    const int t = t0 + (int)threadIdx.x;
    if (threadIdx.x < BT) row[threadIdx.x] = t < len ? -kLog2e * a.lse[((size_t)b * a.Hq + hq) * a.T + t] : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = threadIdx.x + i * kThreads, r = e / L, c = 4 * (e % L);
        *reinterpret_cast<float4*>(Q + r * (D + 4) + c) = x[i];
        *reinterpret_cast<float4*>(dO + r * (D + 4) + c) = y[i];
        float d = dot4(y[i], z[i], 0.f);
#pragma unroll
        for (int sh = 1; sh < L; sh <<= 1) d += __shfl_xor_sync(0xffffffffu, d, sh);
        if (c == 0) row[BT + r] = d;
    }
}

// s[i][x] = row row_of(ty, i) of A . row tx + 16 x of B
template <int D>
__device__ __forceinline__ void scores(const float* A, const float* Bm, int ty, int tx, float (&s)[8][4]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[i][x] = 0.f;
#pragma unroll 2
    for (int d = 0; d < D; d += 4) {
        float4 q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = ld4(A + row_of(ty, i) * (D + 4) + d);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float4 k = ld4(Bm + (tx + 16 * x) * (D + 4) + d);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i][x] = dot4(q[i], k, s[i][x]);
        }
    }
}

// The first group's p, and from them the second's ds, at the same places of P and dS
// (which may be one array: a thread overwrites what it alone has read).
__device__ __forceinline__ void put_p(const WinArgs& a, const float* row, int t0, int s0, int len, int ty, int tx,
                                      const float (&s)[8][4], float* P) {
    const float sl2 = a.sm_scale * kLog2e;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = row_of(ty, i), t = t0 + r;
        const float nl = row[r];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            P[r * PP + tx + 16 * x] =
                t < len && sees(a, t, s0 + tx + 16 * x) ? exp2f(fmaf(s[i][x], sl2, nl)) : 0.f;
    }
}
__device__ __forceinline__ void put_ds(const WinArgs& a, const float* row, int ty, int tx, const float (&dp)[8][4],
                                       const float* P, float* dS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = row_of(ty, i);
        const float de = row[BT + r];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int e = r * PP + tx + 16 * x;
            dS[e] = P[e] * (dp[i][x] - de) * a.sm_scale;
        }
    }
}

template <int D>
using Out = float4[8][D / 64];
template <int D>
__device__ __forceinline__ void clear(Out<D>& o) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// o[i][c] += sum over n0 <= n < n0 + 32 of W[row_of(ty, i)][n] X[n][4 tx + 64 c ..]
template <int D>
__device__ __forceinline__ void gather(const float* W, const float* X, int n0, int ty, int tx, Out<D>& o) {
#pragma unroll 2
    for (int n = n0; n < n0 + BT / 2; n += 4) {
        float4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = ld4(W + row_of(ty, i) * PP + n);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const float4 x = ld4(X + (n + m) * (D + 4) + 4 * tx + 64 * c);
#pragma unroll
                for (int i = 0; i < 8; ++i) axpy((&w[i].x)[m], x, o[i][c]);
            }
    }
}
// o[i][c] += sum_n W[n][8 ty + i] X[n][4 tx + 64 c ..]
template <int D>
__device__ __forceinline__ void scatter(const float* W, const float* X, int ty, int tx, Out<D>& o) {
#pragma unroll 8
    for (int n = 0; n < BT; ++n) {
        const float4 w0 = ld4(W + n * PP + 8 * ty), w1 = ld4(W + n * PP + 8 * ty + 4);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const float4 x = ld4(X + n * (D + 4) + 4 * tx + 64 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                axpy((&w0.x)[i], x, o[i][c]);
                axpy((&w1.x)[i], x, o[4 + i][c]);
            }
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1)
window_dq_simt_kernel(const WinArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr size_t N = tile_floats<D>();
    float *Q = sm, *dO = Q + N, *K = dO + N, *V = K + N, *P = V + N, *row = P + BT * PP;
    // (a cluster shares a query tile as in the forward)
    const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int cs = cluster.num_blocks(), rank = cluster.block_rank();
    // (the last tiles of all heads first: without a window they have the most keys)
    const int x = blockIdx.x / cs, hq = x % a.Hq, b = x / a.Hq % a.B, hk = hq / a.G;
    const int t0 = ((a.T + BT - 1) / BT - 1 - x / (a.Hq * a.B)) * BT;
    const int group = threadIdx.x / kHalf, tx = threadIdx.x & 15, ty = (threadIdx.x % kHalf) >> 4;
    const int len = seq_len(a, b);
    launch_dependents();
    Out<D> o;
    clear<D>(o);
    if (t0 < len) {
        const KeyTiles kt(a, t0, min(t0 + BT, len) - 1);
        load_queries<T, D>(a, b, hq, t0, len, Q, dO, row);
        for (int j = rank; j < kt.n; j += cs) {
            const int s0 = kt.tile(j) * BT;
            __syncthreads();
            load_tile<T, D>(a.k, b, hk, s0, len, K);
            load_tile<T, D>(a.v, b, hk, s0, len, V);
            __syncthreads();
            float s[8][4];
            scores<D>(group ? dO : Q, group ? V : K, ty, tx, s);
            if (group == 0) put_p(a, row, t0, s0, len, ty, tx, s, P);
            __syncthreads();
            if (group == 1) put_ds(a, row, ty, tx, s, P, P);
            __syncthreads();
            gather<D>(P, K, group * (BT / 2), ty, tx, o);  // each group half of the keys
        }
    }
    // the groups' sums, then the CTAs' in the order of the ranks, the rows of a tile
    // spread over the CTAs
    __syncthreads();
    float* mine = group ? dO : Q;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            *reinterpret_cast<float4*>(mine + row_of(ty, i) * (D + 4) + 4 * tx + 64 * c) = o[i][c];
    if (cs > 1) cluster.sync();
    else __syncthreads();
    for (int e = rank * kThreads + threadIdx.x; e < BT * D / 4; e += cs * kThreads) {
        const int r = e / (D / 4), c = 4 * (e % (D / 4));
        if (t0 + r >= a.T) continue;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < cs; ++k) {
            const float* base = k == rank ? Q : cluster.map_shared_rank(Q, k);
            axpy(1.f, ld4(base + r * (D + 4) + c), x);
            axpy(1.f, ld4(base + N + r * (D + 4) + c), x);
        }
        st4(at<T>(a.dq, b, hq, t0 + r) + c, x);
    }
    if (cs > 1) cluster.sync();  // the shares stay until every CTA has read them
}

// Launched beside the kernel for dq, which it does not depend on: only the last
// CTA waits for that one, so that this kernel's end is both kernels'.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1)
window_dkdv_simt_kernel(const WinArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr size_t N = tile_floats<D>();
    float *Q = sm, *dO = Q + N, *K = dO + N, *V = K + N, *P = V + N, *dS = P + BT * PP, *row = dS + BT * PP;
    // item -> (tile, stretch): the tiles with sinks first, of all heads, then the first tiles, which
    // without a window have the longest lists
    const int hk = blockIdx.x % a.Hkv, b = blockIdx.x / a.Hkv % a.B, item = blockIdx.x / (a.Hkv * a.B);
    const int nsc = a.nsink * a.sink_cuts;
    const bool sink = item < nsc;
    const int cuts = sink ? a.sink_cuts : a.cuts, x0 = sink ? item : item - nsc;
    const int tile = (sink ? 0 : a.nsink) + x0 / cuts, cut = x0 % cuts, s0 = tile * BT;
    const int group = threadIdx.x / kHalf, tx = threadIdx.x & 15, ty = (threadIdx.x % kHalf) >> 4;
    const int len = seq_len(a, b);
    launch_dependents();
    Out<D> o;  // dv in the first group, dk in the second
    clear<D>(o);
    if (s0 < len) {
        load_tile<T, D>(a.k, b, hk, s0, len, K);
        load_tile<T, D>(a.v, b, hk, s0, len, V);
        // the last query that sees a key of the tile (a sink: the last of all)
        const int tl = s0 < a.sinks ? len - 1 : (int)min((long long)len - 1, (long long)s0 + BT - 1 + a.window - 1);
        const int per = tl / BT - tile + 1;  // query tiles of a head
        const long long all = (long long)a.G * per;
        const int i1 = (int)(all * (cut + 1) / cuts);
        for (int i = (int)(all * cut / cuts); i < i1; ++i) {
            const int hq = hk * a.G + i / per, t0 = s0 + i % per * BT;
            __syncthreads();
            load_queries<T, D>(a, b, hq, t0, len, Q, dO, row);
            __syncthreads();
            float s[8][4];
            scores<D>(group ? dO : Q, group ? V : K, ty, tx, s);
            if (group == 0) put_p(a, row, t0, s0, len, ty, tx, s, P);
            __syncthreads();
            if (group == 1) {
                put_ds(a, row, ty, tx, s, P, dS);
                asm volatile("bar.sync 1, %0;" ::"n"(kHalf) : "memory");
            }
            scatter<D>(group ? dS : P, group ? Q : dO, ty, tx, o);
        }
    }
    float* slot = nullptr;
    if (cuts > 1) {
        const int nt = (a.T + BT - 1) / BT;
        slot = a.part + ((size_t)(b * a.Hkv + hk) * first_slot(a, nt) + first_slot(a, tile) + cut) * 2 * BT * D;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 8 * ty + i;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            if (slot) st4(slot + ((group ? 0 : BT) + r) * D + 4 * tx + 64 * c, o[i][c]);
            else if (s0 + r < a.T) st4(at<T>(group ? a.dk : a.dv, b, hk, s0 + r) + 4 * tx + 64 * c, o[i][c]);
        }
    }
    if (blockIdx.x == gridDim.x - 1) wait_for_previous();
}

// dk and dv of the tiles whose lists are in stretches: their parts in order
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
window_parts_kernel(const WinArgs a) {
    wait_for_previous();
    constexpr int kBlocks = 2 * BT * D / 4 / kThreads;  // of a tile
    const int tile = blockIdx.x / kBlocks, hk = blockIdx.y, b = blockIdx.z, nt = (a.T + BT - 1) / BT;
    const int cuts = tile < a.nsink ? a.sink_cuts : a.cuts;
    if (cuts == 1) return;
    const float* src = a.part + ((size_t)(b * a.Hkv + hk) * first_slot(a, nt) + first_slot(a, tile)) * 2 * BT * D;
    const int x = (int)(blockIdx.x % kBlocks) * kThreads + threadIdx.x;
    const int w = x / (BT * D / 4), r = x / (D / 4) % BT, c = 4 * (x % (D / 4));
    if (tile * BT + r >= a.T) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < cuts; ++i) {
        const float4 v = ld4(src + (size_t)i * 2 * BT * D + 4 * x);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    st4(at<T>(w ? a.dv : a.dk, b, hk, tile * BT + r) + c, s);
}

WinArgs args(const ssa_window_params_t& p, const View& q, const View& k, const View& v, const int32_t* lens,
             const View& h, float* lse) {
    WinArgs a{};
    a.q = q, a.k = k, a.v = v, a.h = h, a.lse = lse, a.lens = lens;
    a.B = p.B, a.Hq = p.Hq, a.Hkv = p.Hkv, a.G = p.Hq / p.Hkv, a.T = p.T;
    a.window = p.window > 0 && p.window < p.T ? p.window : p.T;  // a window of T tokens leaves none behind
    a.sinks = a.window < p.T ? (p.sinks < p.T ? p.sinks : p.T) : 0;
    a.sm_scale = p.sm_scale;
    // stretches: about three CTAs for each of 148 SMs; those of a tile with sinks about as long as the others
    const int nt = (p.T + BT - 1) / BT;
    const long long tiles = (long long)p.B * p.Hkv * nt, per = ((long long)BT - 1 + a.window - 1) / BT + 1;
    const long long list = a.G * (per < nt ? per : nt);
    long long cuts = (444 + tiles - 1) / tiles;
    cuts = cuts < list ? cuts : list;
    a.cuts = (int)cuts;
    a.nsink = (a.sinks + BT - 1) / BT;
    const long long longest = (long long)a.G * nt, usual = (list + cuts - 1) / cuts;
    const long long sc = (longest + usual - 1) / usual;
    a.sink_cuts = a.nsink ? (int)(sc < 64 ? sc : 64) : 1;
    return a;
}

size_t part_bytes(const WinArgs& a, int D) {
    return (size_t)a.B * a.Hkv * first_slot(a, (a.T + BT - 1) / BT) * 2 * BT * D * sizeof(float);
}

// CTAs that share a query tile: as long as each has an SM and a key tile.  With
// all keys the late tiles are the longest: three CTAs to an SM even out (4000
// tokens, 2 heads of 64: 137 us, 264 with one), if each has four key tiles of the
// longest (1000 tokens, D = 128: 39 us, 54 with two).
int cluster_of(const WinArgs& a) {
    const long long tiles = (a.T + BT - 1) / BT, ctas = tiles * a.Hq * a.B;
    const long long keys = (a.window + BT - 1) / BT + 1 + (a.sinks + BT - 1) / BT;
    const bool all = 2 * (long long)a.window > a.T;
    for (int cs = 8; cs > 1; cs /= 2) {
        const bool fits = cs * ctas <= 148 ? cs <= keys : all && cs * ctas <= 444 && 4 * cs <= keys;
        if (fits && cs <= tiles) return cs;
    }
    return 1;
}
template <typename K>
int launch_clusters(const char* what, K* kernel, const WinArgs& a, int threads, size_t smem, cudaStream_t s) {
    const int cs = cluster_of(a);
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)((a.T + BT - 1) / BT) * cs * a.Hq * a.B);
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&c, kernel, a);
    if (e != cudaSuccess) return fail(SSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return check_launch(what);
}

template <typename T, int D>
int fwd(const WinArgs& a, cudaStream_t s) {
    static_assert(Fwd<D>::smem <= kMaxSmemPerCta, "shared memory");
    const int st = opt_in_max_smem<window_fwd_simt_kernel<T, D>>("window_fwd_simt_kernel");
    if (st != SSA_OK) return st;
    return launch_clusters("window_fwd_simt_kernel", window_fwd_simt_kernel<T, D>, a, Fwd<D>::kGroup * Fwd<D>::kGroups,
                           Fwd<D>::smem, s);
}

template <typename T, int D>
int bwd(const WinArgs& a, cudaStream_t s) {
    constexpr size_t smem_q = (4 * tile_floats<D>() + BT * PP + 2 * BT) * sizeof(float);
    constexpr size_t smem_k = smem_q + BT * PP * sizeof(float);
    static_assert(smem_k <= kMaxSmemPerCta, "shared memory");
    int st = opt_in_max_smem<window_dq_simt_kernel<T, D>>("window_dq_simt_kernel");
    if (st == SSA_OK) st = opt_in_max_smem<window_dkdv_simt_kernel<T, D>>("window_dkdv_simt_kernel");
    if (st == SSA_OK) st = launch_clusters("window_dq_simt_kernel", window_dq_simt_kernel<T, D>, a, kThreads, smem_q, s);
    const unsigned nt = (unsigned)((a.T + BT - 1) / BT), Hkv = (unsigned)a.Hkv, B = (unsigned)a.B;
    const unsigned items = (unsigned)(a.nsink * a.sink_cuts + ((int)nt - a.nsink) * a.cuts);
    if (st == SSA_OK)
        st = launch_beside("window_dkdv_simt_kernel", window_dkdv_simt_kernel<T, D>, dim3(items * Hkv * B), kThreads, smem_k,
                           s, a);
    if (st == SSA_OK && (a.cuts > 1 || a.sink_cuts > 1))
        st = launch_beside("window_parts_kernel", window_parts_kernel<T, D>,
                           dim3((a.cuts > 1 ? nt : (unsigned)a.nsink) * (2 * BT * D / 4 / kThreads), Hkv, B), kThreads, 0, s,
                           a);
    return st;
}

}  // namespace

int launch_window_fwd_simt(const ssa_window_params_t& p, const View& q, const View& k, const View& v,
                           const int32_t* lens, const View& h, float* lse, cudaStream_t s) {
    const WinArgs a = args(p, q, k, v, lens, h, lse);
    if (p.dtype == SSA_BF16) return p.D == 64 ? fwd<__nv_bfloat16, 64>(a, s) : fwd<__nv_bfloat16, 128>(a, s);
    return p.D == 64 ? fwd<float, 64>(a, s) : fwd<float, 128>(a, s);
}

size_t window_bwd_simt_workspace(const ssa_window_params_t& p) {
    return align_up(part_bytes(args(p, View{}, View{}, View{}, nullptr, View{}, nullptr), p.D), 256);
}

int launch_window_bwd_simt(const ssa_window_params_t& p, const View& q, const View& k, const View& v,
                           const int32_t* lens, const View& h, const float* lse, const View& dh,
                           const View& dq, const View& dk, const View& dv, void* ws, cudaStream_t s) {
    WinArgs a = args(p, q, k, v, lens, h, const_cast<float*>(lse));
    a.dh = dh, a.dq = dq, a.dk = dk, a.dv = dv, a.part = static_cast<float*>(ws);
    if (p.dtype == SSA_BF16) return p.D == 64 ? bwd<__nv_bfloat16, 64>(a, s) : bwd<__nv_bfloat16, 128>(a, s);
    return p.D == 64 ? bwd<float, 64>(a, s) : bwd<float, 128>(a, s);
}

int window_take_status() {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_window_status, sizeof v);
    if (e != cudaSuccess) return fail(SSA_ERR_CUDA, "status read: %s", cudaGetErrorString(e));
    if (v != 0) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_window_status, &zero, sizeof zero);
        return fail(SSA_ERR_INVALID_ARG, "window attention: a length was out of range");
    }
    return SSA_OK;
}

}  // namespace ssa
