// Appending new tokens to a paged key/value cache, with the rotation of keys
// and queries to their positions on the way (ssa_cache_append).
//
// Pair (a, b) of a head at position p turns by the angle p * f_i:
//   a' = a cos - b sin,  b' = a sin + b cos.
// The angle is formed in float64 and reduced to half turns there, because a
// float32 product p * f_i is off by p * 2^-24 radians (0.004 at p = 65536);
// the reduced angle, the sines and the products are float32 and each output
// element is rounded once.  (The reduced angle, at most pi, is rounded by at most
// 2^-24 of itself: float32 outputs are off by a relative 3.7e-8 root mean square
// against 64 bits, 2.9e-8 with sines of the unrounded angle, which would cost the
// float64 units' latency in a call that is one chain of latencies.)
//
// The call only moves data: a token's rows are read and written once.  One CTA
// per token: its rotary angles are computed once, by one thread per pair, and
// shared by all heads through shared memory, while every thread's first
// 16-byte vectors are already on their way.  (Four tokens to a CTA, and two or
// four accesses in flight per thread, cost more in resident threads than they
// gave: 86 to 143 us for 16384 tokens.)  Vectors of 16 bytes need
// rot_dim / 2 (pairs a half apart) or rot_dim (neighbours) to be whole
// vectors; other rotary sizes take the element-wise instance.
#include "device_util.cuh"
#include "ssa_internal.h"

namespace ssa {
namespace {

__device__ unsigned int g_append_status;

struct AppendArgs {
    View k, v, q, q_out, k_out;  // data NULL: absent (q, q_out, k_out)
    void *k_pages, *v_pages;
    const int32_t *table, *lens, *q_start;
    int32_t* new_lens;
    const double* inv_freq;
    int N, B, Hq, Hkv, D, page, page_shift, n_pages, max_pages, half, pos_offset;
    long long page_stride;
    bool step;  // one token per sequence: the token's CTA writes its new length
};

// tokens of sequence b in this call
__device__ __forceinline__ long long new_tokens(const AppendArgs& a, int b) {
    if (!a.q_start) return a.N / a.B;
    const long long s0 = max(0, a.q_start[b]), s1 = min(a.N, a.q_start[b + 1]);
    return s1 > s0 ? s1 - s0 : 0;
}
__device__ __forceinline__ int grown(const AppendArgs& a, int b, int len) {
    const long long cap = (long long)a.max_pages * a.page;
    const long long n = max(0, len) + new_tokens(a, b);
    return (int)(n < cap ? n : cap);
}

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
    T x[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> ldv(const T* p) {
    return *reinterpret_cast<const Vec<T, VEC>*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void stv(T* p, const Vec<T, VEC>& v) {
    *reinterpret_cast<Vec<T, VEC>*>(p) = v;
}

// VEC: elements per access of the turned rows (16 bytes, or 1 / 2).
template <typename T, int VEC, bool kInter, int kThreads>
__global__ void __launch_bounds__(kThreads)
append_kernel(const AppendArgs a) {
    constexpr int VMAX = 16 / (int)sizeof(T);
    __shared__ float2 cs[64];  // (cos, sin) of the token's pairs
    const int i = blockIdx.x;
    if (i == a.N) {  // the extra CTA: new lengths (new_lens and lens are distinct here)
        for (int b = threadIdx.x; b < a.B; b += kThreads) a.new_lens[b] = grown(a, b, a.lens[b]);
        return;
    }
    // the token's sequence, slot and cache row
    int b = -1;
    long long first = 0;
    if (!a.q_start) {
        const int n = a.N / a.B;
        b = i / n;
        first = (long long)b * n;
    } else {
        // the last sequence that starts at i or before, 32 of them at a time (every
        // warp for itself; a search by halves would wait for a load at each step)
        const int lane = threadIdx.x & 31;
        for (int b0 = 0; b0 <= a.B; b0 += 32) {
            const int s = b0 + lane <= a.B ? a.q_start[b0 + lane] : 0x7fffffff;
            const unsigned le = __ballot_sync(0xffffffffu, s <= i);
            if (le) {
                b = b0 + 31 - __clz(le);
                first = __shfl_sync(0xffffffffu, s, 31 - __clz(le));
            }
            if (le != 0xffffffffu) break;
        }
        if (b == a.B) b = -1;  // behind the last one
    }
    long long slot = -1;
    size_t row = 0;  // element offset of head 0's row in the pools
    bool cached = false;
    if (b >= 0) {
        const int len = a.lens[b];
        slot = (long long)max(0, len) + (i - first);
        bool bad = len < 0 || slot >= (long long)a.max_pages * a.page;
        if (!bad) {
            const int pg = a.table[(size_t)b * a.max_pages + (slot >> a.page_shift)];
            bad = pg < 0 || pg >= a.n_pages;
            row = (size_t)(bad ? 0 : pg) * a.page_stride + (size_t)(slot & (a.page - 1)) * a.D;
        }
        cached = !bad;
        if (bad && threadIdx.x == 0) atomicOr(&g_append_status, 1u);
        if (a.step && a.new_lens) {
            __syncthreads();  // new_lens may be lens: every thread has read its length
            if (threadIdx.x == 0) a.new_lens[b] = grown(a, b, len);
        }
    }

    // units: one access of q, then k (a pair of accesses where pairs are a half
    // apart), then v (16 bytes)
    const int rot = 2 * a.half;
    const int uh = kInter ? a.D / VEC : (a.half + a.D - rot) / VEC;  // per turned head
    const int nq = a.q.data ? a.Hq * uh : 0, nk = a.Hkv * uh, nv = a.Hkv * (a.D / VMAX);
    const int total = nq + nk + nv;

    Vec<T, VEC> x, y;
    Vec<T, VMAX> z;
    auto place = [&](int u, int& h, int& c, bool& pair) {  // head, first element
        h = u / uh;
        c = (u - h * uh) * VEC;
        pair = !kInter && c < a.half;
        if (!kInter && !pair) c += a.half;  // past the turned part
    };
    auto load = [&](int u) {
        if (u >= nq + nk) {
            const int w = u - nq - nk, per = a.D / VMAX, h = w / per;
            z = ldv<T, VMAX>(static_cast<const T*>(a.v.data) + (size_t)i * a.v.st + (size_t)h * a.v.sh +
                             (w - h * per) * VMAX);
            return;
        }
        int h, c;
        bool pair;
        place(u < nq ? u : u - nq, h, c, pair);
        const View& s = u < nq ? a.q : a.k;
        const T* p = static_cast<const T*>(s.data) + (size_t)i * s.st + (size_t)h * s.sh + c;
        x = ldv<T, VEC>(p);
        if (pair) y = ldv<T, VEC>(p + a.half);
    };
    auto finish = [&](int u) {
        if (u >= nq + nk) {
            if (!cached) return;
            const int w = u - nq - nk, per = a.D / VMAX, h = w / per;
            stv<T, VMAX>(static_cast<T*>(a.v_pages) + row + (size_t)h * a.page * a.D + (w - h * per) * VMAX, z);
            return;
        }
        int h, c;
        bool pair;
        place(u < nq ? u : u - nq, h, c, pair);
        if (b >= 0) {
            if constexpr (kInter) {
                if constexpr (VEC > 1) {
                    if (c < rot) {
#pragma unroll
                        for (int e = 0; e < VEC; e += 2) {
                            const float2 t = cs[(c + e) >> 1];
                            const float p = to_f32(x.x[e]), r = to_f32(x.x[e + 1]);
                            x.x[e] = from_f32<T>(p * t.x - r * t.y);
                            x.x[e + 1] = from_f32<T>(p * t.y + r * t.x);
                        }
                    }
                }
            } else if (pair) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float2 t = cs[c + e];
                    const float p = to_f32(x.x[e]), r = to_f32(y.x[e]);
                    x.x[e] = from_f32<T>(p * t.x - r * t.y);
                    y.x[e] = from_f32<T>(p * t.y + r * t.x);
                }
            }
        }
        const View& o = u < nq ? a.q_out : a.k_out;
        if (o.data) {
            T* p = static_cast<T*>(o.data) + (size_t)i * o.st + (size_t)h * o.sh + c;
            stv<T, VEC>(p, x);
            if (pair) stv<T, VEC>(p + a.half, y);
        }
        if (u >= nq && cached) {
            T* p = static_cast<T*>(a.k_pages) + row + (size_t)h * a.page * a.D + c;
            stv<T, VEC>(p, x);
            if (pair) stv<T, VEC>(p + a.half, y);
        }
    };

    int u = threadIdx.x;
    if (u < total) load(u);  // in flight while the angles are formed
    if (b >= 0 && (int)threadIdx.x < a.half) {
        const double turns = (double)(a.pos_offset + slot) * a.inv_freq[threadIdx.x] * 0.31830988618379067154;  // in units of pi
        float s, c;
        sincospif((float)(turns - 2.0 * rint(0.5 * turns)), &s, &c);
        cs[threadIdx.x] = make_float2(c, s);
    }
    __syncthreads();
    if (u < total) finish(u);
    for (u += kThreads; u < total; u += kThreads) {
        load(u);
        finish(u);
    }
}

__global__ void lens_kernel(const AppendArgs a) {
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) a.new_lens[b] = grown(a, b, a.lens[b]);
}

template <typename T, int kThreads>
void launch(const AppendArgs& a, bool inter, unsigned grid, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    if (inter) {
        if (2 * a.half % V == 0) append_kernel<T, V, true, kThreads><<<grid, kThreads, 0, s>>>(a);
        else append_kernel<T, 2, true, kThreads><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (a.half % V == 0) append_kernel<T, V, false, kThreads><<<grid, kThreads, 0, s>>>(a);
        else append_kernel<T, 1, false, kThreads><<<grid, kThreads, 0, s>>>(a);
    }
}

// Tokens up to which a CTA has 256 threads and not 128: few tokens leave SMs
// idle, and the wider CTA is done sooner (8 tokens of 16/4 heads of 128, bf16: 3.3 us
// against 3.7); many are held up by the barrier behind the look-ups, which
// couples fewer warps in a small CTA (16384 tokens of 32/8 heads 91 against 74 us,
// 81 % of the measured copy bandwidth).  256 against 128 threads, us, SM clock 1965 MHz:
//     tokens           64    256    512    768   1024   2048
//     32/8 heads      4.1    4.8    5.6    6.7    9.0   14.4
//                     4.8    5.3    6.2    6.9    7.1   13.7
//     8/2 heads       3.5    3.7    3.8           5.9
//                     3.5    3.7    3.8           4.2
constexpr int kFewTokens = 512;

}  // namespace

int launch_cache_append(const ssa_cache_params_t& p, int n, const View& k, const View& v, const View& q,
                        void* k_pages, void* v_pages, const int32_t* table, const int32_t* lens,
                        int32_t* new_lens, const int32_t* q_start, const double* inv_freq, int rot,
                        int interleaved, int pos_offset, const View& q_out, const View& k_out,
                        cudaStream_t s) {
    AppendArgs a{};
    a.k = k, a.v = v, a.q = q, a.q_out = q_out, a.k_out = k_out;
    a.k_pages = k_pages, a.v_pages = v_pages;
    a.table = table, a.lens = lens, a.q_start = q_start, a.new_lens = new_lens, a.inv_freq = inv_freq;
    a.N = n, a.B = p.B, a.Hq = p.Hq, a.Hkv = p.Hkv, a.D = p.D, a.page = p.page;
    a.page_shift = __builtin_ctz((unsigned)p.page);
    a.n_pages = p.n_pages, a.max_pages = p.max_pages, a.half = rot / 2, a.pos_offset = pos_offset;
    a.page_stride = p.page_stride;
    a.step = !q_start && n == p.B;
    // Who writes the new lengths: with one token per sequence the token's own CTA;
    // with distinct arrays one CTA more; in place (several CTAs still read the
    // old lengths) a launch of its own after the first.
    const bool extra = new_lens && !a.step && new_lens != lens;
    const unsigned grid = (unsigned)n + (extra ? 1u : 0u);
    if (grid) {
        const bool inter = interleaved != 0, few = n <= kFewTokens;
        if (p.dtype == SSA_BF16)
            few ? launch<__nv_bfloat16, 256>(a, inter, grid, s) : launch<__nv_bfloat16, 128>(a, inter, grid, s);
        else
            few ? launch<float, 256>(a, inter, grid, s) : launch<float, 128>(a, inter, grid, s);
        const int st = check_launch("append_kernel");
        if (st != SSA_OK) return st;
    }
    if (new_lens && !a.step && !extra) {
        lens_kernel<<<1, 256, 0, s>>>(a);
        return check_launch("lens_kernel");
    }
    return SSA_OK;
}

int append_take_status() {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_append_status, sizeof v);
    if (e != cudaSuccess) return fail(SSA_ERR_CUDA, "status read: %s", cudaGetErrorString(e));
    if (v != 0) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_append_status, &zero, sizeof zero);
        return fail(SSA_ERR_INVALID_ARG, "cache append: a length, slot or page number was out of range");
    }
    return SSA_OK;
}

}  // namespace ssa
