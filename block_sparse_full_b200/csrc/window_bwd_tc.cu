// Gradients of sliding-window attention with sinks on the sm_100a tensor cores
// (bf16 in, float32 accumulate; ssa_window_bwd).
//
//   P = 2^(S sm_scale log2 e - lse log2 e), S = Q K^T
//   dV = P^T dO,  dS = P (dO V^T - delta),  delta = rowsum(dO h)
//   dQ = sm_scale dS K,  dK = sm_scale dS^T Q
//
// Four launches (five with sinks that the window leaves behind):
//   window_rows_kernel   -lse log2 e and -delta of every row, padded to whole
//                        tiles: one pass over dO and h, bound by reading them
//   window_dq_kernel     a CTA per query tile of 128 walks the key tiles of 64:
//                        three products per tile (where rows see few keys it walks
//                        them twice, first for delta)
//   window_dkdv_kernel   a CTA per key tile of 128 and key/value head walks the
//                        query tiles of 128 that see it, for each query head of
//                        its group in turn: four products per tile
//   window_sink_kernel   sums the parts of the first key tile (below)
// S and dP are formed in both kernels: seven products instead of five, but every sum
// has one owner and a fixed order, without atomics, and without a dS of T x
// window elements in memory: writing and reading that costs more than forming
// it again (at T = 4096, window 1024, 128 heads 2.4 GB, 0.37 ms, against two
// products of 0.1 ms each).
//
// dK/dV: S^T = K Q^T, dP^T = V dO^T (M = 128 keys, N = 128 queries), dK and dV take
// all 512 TMEM columns (D = 128), so one CTA fills the SM and its four products
// are ordered so that each runs beside a part of the softmax that does not
// need it:
//     tensor cores   dK_i-1   dP_i    | dV_i     S_i+1    | dK_i ...
//     softmax        P_i = 2^(S_i ..) | dS_i = P_i (dP_i ..) | P_i+1 ...
// P^T and dS^T go back to TMEM as bf16 (over the scores) and are the A
// operands, Q and dO tiles (used K-major for the scores) the MN-major B
// operands.  Sixteen softmax warps, four threads per key with 32 queries each.
// Bound by the chain S -> P -> dV, next S: the tensor cores are busy 45 % of the
// time (610 us at T = 4096, window 1024, 32/8 heads, batch 4).  Tiles of 64 queries
// in two TMEM buffers, two groups of warps in turn, overlap more but read K and V
// from shared memory twice as often (612 us); P^T in shared memory, which frees S
// earlier, adds 64 KB of such traffic to a tile and was 12 % slower.
// A 128-key tile that holds sinks is seen by every later query; the queries
// past the window's reach are split into stretches of about a CTA's usual
// work, whose float32 parts are summed in order by window_sink_kernel.
//
// dQ: 256 TMEM columns (S 64, dP 64, dQ 128) and 112 KB, so two CTAs share the SM
// and take turns on the tensor cores.  dS goes over dP, so that the next S is
// formed as soon as the softmax has read the last, and the exponentials do not
// wait for dP (573 us -> 436 us at the same shape).
//
// P and dS are rounded to bf16, each value by at most 2^-8 of itself, because they
// are operands of products with the bf16 rows of Q, K and dO; sums, the row values and
// dS before that rounding are float32.  Against 64 bits dq, dk and dv are off by a
// relative 0.0024 (root mean square), where their own rounding alone is 0.0016.
//
// Rows and keys behind a sequence's length may be NaN: weights are selected, not
// multiplied, to zero, and such rows of a tile are cleared in shared memory
// before they are an operand along the summed axis.
#include <cooperative_groups.h>
#include <cuda.h>

#include "device_util.cuh"
#include "ssa_internal.h"
#include "tc_util.cuh"
#include "tmap.h"

namespace ssa {
namespace {

using namespace tc;

constexpr int BM = 128;  // rows of a CTA's tile
constexpr int BN = 64;   // rows of a tile that it walks
constexpr int kThreads = 320, kSoftmax = 256;
constexpr int kThreadsK = 640, kSoftmaxK = 512;  // dK/dV: four warps of roles, sixteen softmax warps
constexpr uint32_t BOX_M = BM * 128, BOX_N = BN * 128;  // boxes of 64 columns
constexpr uint32_t TILE_M = 2 * BOX_M, TILE_N = 2 * BOX_N;
constexpr float kLog2e = 1.4426950408889634f;

__device__ unsigned int g_bwd_status[2];  // dQ, dK/dV: bit 0: a wait expired, bit 1: misaligned shared memory
__device__ unsigned int g_bwd_range;   // a length was out of range

struct BwdArgs {
    const int32_t* lens;
    const float* nlse;    // [B, Hq, Tp]: -lse log2 e
    const float* ndelta;  // [B, Hq, Tp]: -delta
    float* part;          // per head, with sinks out of reach: [dK, dV][128][D], then splits x [dK, dV][sinks][D]
    bool sweep;           // every query tile of dQ sweeps the keys for delta first
    int B, Hq, Hkv, G, T, Tp, window, sinks, nt;  // nt: tiles of 128
    int splits;           // stretches of queries past the reach of key tile 0
    int cluster;          // CTAs that share a key tile's list
    float scale, scale_log2;
    unsigned long long timeout_ns;
};

// Floats before part i (0: the queries in reach) of head bh.
__host__ __device__ __forceinline__ size_t part_offset(const BwdArgs& a, int bh, int i, int D) {
    const size_t head = 2 * (size_t)D * (BM + (size_t)a.splits * a.sinks);
    return bh * head + (i > 0 ? 2 * (size_t)D * (BM + (size_t)(i - 1) * a.sinks) : 0);
}

__device__ __forceinline__ int seq_len(const BwdArgs& a, int b) {
    if (!a.lens) return a.T;
    const int n = a.lens[b];
    if (n < 0 || n > a.T) {
        if (threadIdx.x == 0) atomicOr(&g_bwd_range, 1u);
        return n < 0 ? 0 : a.T;
    }
    return n;
}

__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer() - t0 > kDrainLimitNs) return false;
    return true;
}
// Untiled copy of `bytes` (a multiple of 16) from global memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 TMEM columns of a row, times mul, as bf16 columns [col, col + 32) of a
// staged [128 rows x 64] x 2 tile (128-byte swizzle)
__device__ __forceinline__ void stage32(uint32_t taddr, float mul, bool some, uint8_t* tile, int col0, int r) {
    uint32_t u[32];
    tmem_ld32(taddr, u);
    tmem_wait_ld();
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = some ? pack_bf16(__uint_as_float(u[8 * v + 2 * e]) * mul, __uint_as_float(u[8 * v + 2 * e + 1]) * mul)
                        : 0u;
        const int col = col0 + 8 * v;
        const uint32_t chunk = (uint32_t)((col & 63) >> 3) ^ (uint32_t)(r & 7);
        *reinterpret_cast<uint4*>(tile + (col >> 6) * BOX_M + r * 128 + chunk * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ---------------------------------------------------------------- rows

template <int D>
__global__ void __launch_bounds__(256)
window_rows_kernel(const View h, const View dh, const float* lse, float* nlse, float* ndelta, const BwdArgs a) {
    constexpr int L = D / 8;  // lanes of a row, 16 bytes each
    launch_dependents();
    const int t = blockIdx.x * (256 / L) + (int)threadIdx.x / L, c = 8 * ((int)threadIdx.x % L);
    const int hq = blockIdx.y, b = blockIdx.z;
    if (t >= a.Tp) return;  // (Tp is a multiple of the rows of a block: whole blocks)
    const bool row = t < seq_len(a, b);
    float s = 0.f;
    if (row && !a.sweep) {
        const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(h.data) + (size_t)b * h.sb +
                                                        (size_t)hq * h.sh + (size_t)t * h.st + c);
        const uint4 y = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(dh.data) + (size_t)b * dh.sb +
                                                        (size_t)hq * dh.sh + (size_t)t * dh.st + c);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s = fmaf(__uint_as_float(xs[i] << 16), __uint_as_float(ys[i] << 16), s);
            s = fmaf(__uint_as_float(xs[i] & 0xffff0000u), __uint_as_float(ys[i] & 0xffff0000u), s);
        }
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (c == 0) {
        const size_t i = ((size_t)b * a.Hq + hq) * a.Tp + t;
        nlse[i] = row ? -kLog2e * lse[((size_t)b * a.Hq + hq) * a.T + t] : 0.f;
        ndelta[i] = -s;
    }
}

// ---------------------------------------------------------------- dK, dV

// Two slots of 128 queries each for Q (with the row values) and dO.
constexpr uint32_t K_OFF_K = 0, K_OFF_V = TILE_M, K_OFF_Q = 2 * TILE_M, K_OFF_DO = 4 * TILE_M;
constexpr uint32_t K_OFF_ROW = 6 * TILE_M, ROWS = 2 * BM * 4;  // nlse, ndelta of a Q tile's queries
constexpr uint32_t K_OFF_BAR = K_OFF_ROW + 2 * ROWS;
enum : int { KB_KV, KB_QFULL, KB_QEMPTY = KB_QFULL + 2, KB_OFULL = KB_QEMPTY + 2, KB_OEMPTY = KB_OFULL + 2,
             KB_SREADY = KB_OEMPTY + 2, KB_DPREADY, KB_PREADY, KB_DSREADY, KB_DRAIN, KB_COUNT };
constexpr uint32_t K_OFF_MISC = K_OFF_BAR + KB_COUNT * 8;
constexpr uint32_t K_SMEM = K_OFF_MISC + 16 + 1024;
static_assert(K_SMEM <= kMaxSmemPerCta, "shared memory");
constexpr uint32_t TK_S = 0, TK_DP = 128, TK_DK = 256, TK_DV = 384;

// kShared: a cluster of CTAs shares a key tile's list.
template <int D, bool kShared>
__global__ void __launch_bounds__(kThreadsK, 1)
window_dkdv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                   const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_dk, const __grid_constant__ CUtensorMap tm_dv,
                   const View dk, const View dv, const BwdArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + K_OFF_MISC + 4);
    unsigned int* status = &g_bwd_status[1];
    const uint64_t lim = a.timeout_ns;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto BAR = [&](int i) { return base + K_OFF_BAR + 8u * (uint32_t)i; };

    // ---- the key tile and the flattened list [i0, i1) of (query head of the group, query tile)
    const int BH = a.B * a.Hkv;
    const int cs = kShared ? a.cluster : 1, rank = (int)blockIdx.x % cs, x0 = (int)blockIdx.x / cs;
    const int item = x0 / BH, bh = x0 % BH;  // early tiles first: the longest without a window
    const int b = bh / a.Hkv, hk = bh % a.Hkv;
    const int J = item < a.nt ? item : 0;
    const int k0 = J * BM;
    const int len = seq_len(a, b);
    const int last = (len - 1) / BM;  // last query tile (len 0: none, below)
    const int reach = (int)min((long long)last, ((long long)k0 + BM - 1 + a.window - 1) / BM);
    int q_first = J, q_count, i0 = 0, i1;
    if (item < a.nt) {
        q_count = k0 < len ? reach - q_first + 1 : 0;
        i1 = a.G * q_count;
    } else {
        q_first = reach + 1;
        q_count = len > 0 ? last - reach : 0;
        const long long n = (long long)a.G * q_count;
        const int sp = item - a.nt;
        i0 = (int)(n * sp / a.splits);
        i1 = (int)(n * (sp + 1) / a.splits);
    }
    if constexpr (kShared) {  // the cluster's CTAs take a stretch each
        const int all = i1 - i0;
        i1 = i0 + (int)((long long)all * (rank + 1) / cs);
        i0 += (int)((long long)all * rank / cs);
    }
    const int n = i1 - i0;
    auto head_of = [&](int i) { return hk * a.G + (i0 + i) / q_count; };
    auto query_of = [&](int i) { return (q_first + (i0 + i) % q_count) * BM; };
    const bool parts = a.splits > 0 && J == 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < KB_COUNT; ++i)
            mbar_init(BAR(i), i == KB_PREADY || i == KB_DSREADY ? kSoftmaxK : i == KB_SREADY && lim == kLostScoresNs ? 2 : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(base + K_OFF_MISC, 512);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    launch_dependents();
    const uint32_t tmem = *reinterpret_cast<uint32_t*>(gbase + K_OFF_MISC);
    const unsigned FULL = 0xffffffffu;
    auto wait = [&](int bar, uint32_t ph) -> bool {
        return __all_sync(FULL, mbar_wait(BAR(bar), ph & 1, abort_flag, status, lim));
    };

    // Loads the tiles of one ring (with Q the row values too); the copies in flight
    // land before the CTA ends, also where a wait gave up.
    auto ring = [&](int full, int empty, const CUtensorMap* tm, uint32_t off, bool rows) {
        int issued = 0;
        for (int i = 0; i < n; ++i) {
            const int s = i & 1;
            if (i >= 2 && !wait(empty + s, (i >> 1) + 1)) break;
            const int hq = head_of(i), q0 = query_of(i);
            if (elect_one()) {
                const uint32_t bar = BAR(full + s), dst = base + off + s * TILE_M;
                mbar_expect_tx(bar, BM * D * 2 + (rows ? ROWS : 0));
#pragma unroll
                for (int x = 0; x < D / 64; ++x) tma_load_4d(dst + x * BOX_M, tm, bar, 64 * x, q0, hq, b);
                if (rows) {
                    const size_t row = ((size_t)b * a.Hq + hq) * a.Tp + q0;
                    bulk_load(base + K_OFF_ROW + s * ROWS, a.nlse + row, BM * 4, bar);
                    bulk_load(base + K_OFF_ROW + s * ROWS + BM * 4, a.ndelta + row, BM * 4, bar);
                }
            }
            __syncwarp();
            issued = i + 1;
        }
        for (int i = max(0, issued - 2); i < issued; ++i) wait_drain(BAR(full + (i & 1)), (i >> 1) & 1);
    };

    if (warp == 0) {
        // ------------------------------------------------ K, V and the ring of Q
        if (n > 0 && elect_one()) {
            prefetch_tmap(&tm_q);
            mbar_expect_tx(BAR(KB_KV), 2 * BM * D * 2);
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
                tma_load_4d(base + K_OFF_K + x * BOX_M, &tm_k, BAR(KB_KV), 64 * x, k0, hk, b);
                tma_load_4d(base + K_OFF_V + x * BOX_M, &tm_v, BAR(KB_KV), 64 * x, k0, hk, b);
            }
        }
        __syncwarp();
        wait_for_previous();  // the row values are the kernels' before this one; K and V may come sooner
        ring(KB_QFULL, KB_QEMPTY, &tm_q, K_OFF_Q, true);
        if (n > 0) wait_drain(BAR(KB_KV), 0);
    } else if (warp == 2) {
        // ------------------------------------------------ the ring of dO
        ring(KB_OFULL, KB_OEMPTY, &tm_do, K_OFF_DO, false);
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BM, false), idesc_g = idesc_bf16_f32(BM, D, true);
        const uint64_t kdesc = smem_desc_sw128(base + K_OFF_K, 16, 1024), vdesc = smem_desc_sw128(base + K_OFF_V, 16, 1024);
        // Q and dO tiles, K-major for the scores and MN-major for the gradients
        const uint64_t qdesc = smem_desc_sw128(base + K_OFF_Q, 16, 1024), odesc = smem_desc_sw128(base + K_OFF_DO, 16, 1024);
        const uint64_t qmdesc = smem_desc_sw128(base + K_OFF_Q, BOX_M, 1024), omdesc = smem_desc_sw128(base + K_OFF_DO, BOX_M, 1024);
        auto product = [&](uint32_t d, uint64_t ad, uint64_t bd) {  // 128 keys x 128 queries over D
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t o = (kk >> 2) * BOX_M + (kk & 3) * 32;
                mma_ss(d, desc_add(ad, o), desc_add(bd, o), idesc_s, kk > 0 ? 1u : 0u);
            }
        };
        auto gradient = [&](uint32_t d, uint32_t w, uint64_t bd, int i) {  // 128 keys x D over 128 queries
#pragma unroll
            for (int kk = 0; kk < BM / 16; ++kk)  // the quarters' weights lie 32 columns apart
                mma_ts(d, w + 32 * (kk >> 1) + 8 * (kk & 1), desc_add(bd, kk * 2048), idesc_g, i > 0 || kk > 0 ? 1u : 0u);
        };
        auto scores = [&](int i) -> bool {  // S^T, behind the product that reads P from its columns
            if (!wait(KB_QFULL + (i & 1), i >> 1)) return false;
            fence_after_sync();
            if (elect_one()) {
                product(tmem + TK_S, kdesc, desc_add(qdesc, (i & 1) * TILE_M));
                mma_commit(BAR(KB_SREADY));
            }
            __syncwarp();
            return true;
        };
        auto values = [&](int i) -> bool {  // dP^T, behind the product that reads dS from its columns
            if (!wait(KB_OFULL + (i & 1), i >> 1)) return false;
            fence_after_sync();
            if (elect_one()) {
                product(tmem + TK_DP, vdesc, desc_add(odesc, (i & 1) * TILE_M));
                mma_commit(BAR(KB_DPREADY));
            }
            __syncwarp();
            return true;
        };
        bool ok = n == 0 || (wait(KB_KV, 0) && scores(0) && values(0));
        for (int i = 0; ok && i < n; ++i) {
            ok = wait(KB_PREADY, i);
            if (!ok) break;
            fence_after_sync();
            if (elect_one()) {
                gradient(tmem + TK_DV, tmem + TK_S, desc_add(omdesc, (i & 1) * TILE_M), i);
                mma_commit(BAR(KB_OEMPTY + (i & 1)));
            }
            __syncwarp();
            if (i + 1 < n) ok = scores(i + 1);
            ok = ok && wait(KB_DSREADY, i);
            if (!ok) break;
            fence_after_sync();
            if (elect_one()) {
                gradient(tmem + TK_DK, tmem + TK_DP, desc_add(qmdesc, (i & 1) * TILE_M), i);
                mma_commit(BAR(KB_QEMPTY + (i & 1)));
            }
            __syncwarp();
            if (i + 1 < n) ok = values(i + 1);
        }
        if (elect_one()) mma_commit(BAR(KB_DRAIN));
        __syncwarp();
        wait_drain(BAR(KB_DRAIN), 0);
    } else if (warp >= 4) {
        // ------------------------------------------------ weights, four threads per key
        const int q4 = warp & 3, part = (warp - 4) >> 2;  // the warp's TMEM lanes; its quarter of the queries
        const int r = q4 * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
        const int key = k0 + r, c0 = 32 * part;
        const float sl2 = a.scale_log2;
        // the last query that sees the key
        const int seen = key < a.sinks ? len - 1 : (int)min((long long)len - 1, (long long)key + a.window - 1);
        const f32x2 sl = mk2(sl2, sl2);
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int q0 = query_of(i);
            ok = wait(KB_SREADY, i) && wait(KB_QFULL + (i & 1), i >> 1);
            if (!ok) break;
            fence_after_sync();
            if (a.lens && q0 + BM > len) {
                // queries behind the end: cleared before they are summed over
                ok = wait(KB_OFULL + (i & 1), i >> 1);
                if (!ok) break;
                const int x = (int)threadIdx.x - 128, row = x & 127, box = (x >> 7) & 1;
                if (q0 + row >= len && box < D / 64) {
                    uint8_t* tile = gbase + (x >> 8 ? K_OFF_DO : K_OFF_Q) + (i & 1) * TILE_M;
                    uint4* p = reinterpret_cast<uint4*>(tile + box * BOX_M + row * 128);
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[e] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async();
                __syncwarp();
            }
            const uint32_t ts = trow + TK_S + c0, td = trow + TK_DP + c0;
            uint32_t u[32];
            tmem_ld32(ts, u);
            tmem_wait_ld();
            const float4* nl = reinterpret_cast<const float4*>(gbase + K_OFF_ROW + (i & 1) * ROWS) + c0 / 4;
            // the queries of this quarter that see the key
            const bool masked = q0 < k0 + BM - 1 || q0 + BM - 1 - k0 >= a.window || q0 + BM > len;
            const uint32_t bits = masked ? bit_range(key - q0 - c0, seen - q0 - c0) : 0xffffffffu;
            float p[32];
            uint32_t pk[16];
            if (__any_sync(FULL, bits != 0)) {
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    const float4 w = nl[c / 4];
                    un2(fma2(mk2(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), sl, mk2(w.x, w.y)), p[c], p[c + 1]);
                    un2(fma2(mk2(__uint_as_float(u[c + 2]), __uint_as_float(u[c + 3])), sl, mk2(w.z, w.w)), p[c + 2], p[c + 3]);
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) p[c] = ex2(p[c]);
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!(bits >> c & 1u)) p[c] = 0.f;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 32; ++c) p[c] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < 16; ++c) pk[c] = pack_bf16(p[2 * c], p[2 * c + 1]);
            tmem_st<16>(ts, pk);
            tmem_wait_st();
            fence_before_sync();
            mbar_arrive(BAR(KB_PREADY));
            ok = wait(KB_DPREADY, i);
            if (!ok) break;
            fence_after_sync();
            tmem_ld32(td, u);
            tmem_wait_ld();
            const float4* nd = nl + BM / 4;
            const bool tail = a.lens && (q0 + BM > len || k0 + BM > len);
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
                const float4 w = nd[c / 4];
                const f32x2 d0 = add2(mk2(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), mk2(w.x, w.y));
                const f32x2 d1 = add2(mk2(__uint_as_float(u[c + 2]), __uint_as_float(u[c + 3])), mk2(w.z, w.w));
                float e0, e1, e2, e3;
                un2(mul2(d0, mk2(p[c], p[c + 1])), e0, e1);
                un2(mul2(d1, mk2(p[c + 2], p[c + 3])), e2, e3);
                if (tail) {  // selected: dP of rows behind the end may be NaN (elsewhere a masked P of 0 does it)
                    if (!(bits >> c & 1u)) e0 = 0.f;
                    if (!(bits >> (c + 1) & 1u)) e1 = 0.f;
                    if (!(bits >> (c + 2) & 1u)) e2 = 0.f;
                    if (!(bits >> (c + 3) & 1u)) e3 = 0.f;
                }
                pk[c / 2] = pack_bf16(e0, e1);
                pk[c / 2 + 1] = pack_bf16(e2, e3);
            }
            tmem_st<16>(td, pk);
            tmem_wait_st();
            fence_before_sync();
            mbar_arrive(BAR(KB_DSREADY));
        }
        if (ok) ok = wait(KB_DRAIN, 0);
        ok = bar_and(ok && !*abort_flag, 1, kSoftmaxK);
        fence_after_sync();
        if (kShared) {  // the shares, float32, over the tiles: [dK, dV][row][D], 16-byte pieces swizzled by row
            if (ok) {
#pragma unroll 1
                for (int x = 0; x < D / 64; ++x) {
                    const int w = part >> 1, col = (D / 2) * (part & 1) + 32 * x;
                    uint32_t u[32];
                    tmem_ld32(trow + (w ? TK_DV : TK_DK) + col, u);
                    tmem_wait_ld();
                    uint4* dst = reinterpret_cast<uint4*>(gbase) + (w * BM + r) * (D / 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[(col / 4 + e) ^ (r & 7)] = n > 0 ? make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3])
                                                             : make_uint4(0u, 0u, 0u, 0u);
                }
            }
        } else if (ok && parts) {
            const int rows = item < a.nt ? BM : a.sinks;  // (far queries see the sinks alone)
            float* slot = a.part + part_offset(a, bh, item < a.nt ? 0 : 1 + item - a.nt, D);
#pragma unroll 1
            for (int x = 0; x < D / 64; ++x) {  // two parts for dK, two for dV
                const int w = part >> 1, col = (D / 2) * (part & 1) + 32 * x;
                uint32_t u[32];
                tmem_ld32(trow + (w ? TK_DV : TK_DK) + col, u);
                tmem_wait_ld();
                float4* dst = reinterpret_cast<float4*>(slot + ((size_t)w * rows + r) * D + col);
#pragma unroll
                for (int e = 0; e < 8 && r < rows; ++e)
                    dst[e] = n > 0 ? make_float4(__uint_as_float(u[4 * e]), __uint_as_float(u[4 * e + 1]),
                                                 __uint_as_float(u[4 * e + 2]), __uint_as_float(u[4 * e + 3]))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        } else if (!parts) {
            if (ok) {
#pragma unroll 1
                for (int x = 0; x < D / 64; ++x) {  // K and V are used up
                    const int w = part >> 1, col = (D / 2) * (part & 1) + 32 * x;
                    stage32(trow + (w ? TK_DV : TK_DK) + col, w ? 1.f : a.scale, n > 0, gbase + (w ? K_OFF_V : K_OFF_K),
                            col, r);
                }
            }
            fence_async();
            bar_sync(1, kSoftmaxK);
            if (warp == 4 && lane == 0 && ok) {
#pragma unroll
                for (int x = 0; x < D / 64; ++x) {
                    tma_store_4d(&tm_dk, base + K_OFF_K + x * BOX_M, 64 * x, k0, hk, b);
                    tma_store_4d(&tm_dv, base + K_OFF_V + x * BOX_M, 64 * x, k0, hk, b);
                }
                bulk_commit_group();
                bulk_wait_group_read0();
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
    if constexpr (kShared) {  // the shares are summed in the order of the ranks, the rows spread over the CTAs
        __syncwarp();
        const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
        cluster.sync();
        constexpr int kAll = 2 * BM * D / 4;
        float* slot = a.part + part_offset(a, bh, item < a.nt ? 0 : 1 + item - a.nt, D);
        const int rows = !parts ? min(BM, a.T - k0) : item < a.nt ? BM : a.sinks;
        constexpr int kBatch = 4;  // reads in flight
        const int e1 = (rank + 1) * kAll / cs;
        for (int e0 = rank * kAll / cs + (int)threadIdx.x; e0 < e1; e0 += kBatch * kThreadsK) {
            float4 s[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < cs; ++k) {
                const float4* share = reinterpret_cast<const float4*>(cluster.map_shared_rank(gbase, k));
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int e = e0 + i * kThreadsK, r = e / (D / 4) % BM, c = e % (D / 4);
                    if (e >= e1) continue;
                    const float4 v = share[e - c + (c ^ (r & 7))];
                    s[i].x += v.x, s[i].y += v.y, s[i].z += v.z, s[i].w += v.w;
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int e = e0 + i * kThreadsK, w = e / (BM * D / 4), r = e / (D / 4) % BM, c = e % (D / 4);
                if (e >= e1 || r >= rows) continue;
                if (parts) {
                    *reinterpret_cast<float4*>(slot + ((size_t)w * rows + r) * D + 4 * c) = s[i];
                } else {
                    const View& o = w ? dv : dk;
                    const float m = w ? 1.f : a.scale;
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(o.data) + (size_t)b * o.sb + (size_t)hk * o.sh +
                                              (size_t)(k0 + r) * o.st + 4 * c) =
                        make_uint2(pack_bf16(s[i].x * m, s[i].y * m), pack_bf16(s[i].z * m, s[i].w * m));
                }
            }
        }
        cluster.sync();  // the shares stay until every CTA has read them
    }
}

// dk and dv of the first key tile: its parts in order
template <int D>
__global__ void __launch_bounds__(256)
window_sink_kernel(const View dk, const View dv, const BwdArgs a) {
    wait_for_previous();
    const int x = blockIdx.y * 256 + threadIdx.x, r = x / (D / 4), c = 4 * (x % (D / 4));
    const int w = blockIdx.x & 1, bh = blockIdx.x >> 1, b = bh / a.Hkv, hk = bh % a.Hkv;
    if (r >= min(BM, a.T)) return;
    float4 s = *reinterpret_cast<const float4*>(a.part + part_offset(a, bh, 0, D) + ((size_t)w * BM + r) * D + c);
    if (r < a.sinks) {
        const float* src = a.part + part_offset(a, bh, 1, D) + ((size_t)w * a.sinks + r) * D + c;
#pragma unroll 4
        for (int i = 0; i < a.splits; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(src + (size_t)i * 2 * a.sinks * D);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
    }
    const float m = w ? 1.f : a.scale;
    const View& o = w ? dv : dk;
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(o.data) + (size_t)b * o.sb + (size_t)hk * o.sh +
                              (size_t)r * o.st + c) = make_uint2(pack_bf16(s.x * m, s.y * m), pack_bf16(s.z * m, s.w * m));
}

// ---------------------------------------------------------------- dQ

constexpr uint32_t Q_OFF_Q = 0, Q_OFF_DO = TILE_M, Q_OFF_K = 2 * TILE_M, Q_OFF_V = Q_OFF_K + 2 * TILE_N;
constexpr uint32_t Q_OFF_BAR = Q_OFF_V + TILE_N;
enum : int { QB_Q, QB_KFULL, QB_KEMPTY = QB_KFULL + 2, QB_VFULL = QB_KEMPTY + 2, QB_VEMPTY, QB_SREADY, QB_DPREADY, QB_SFREE, QB_DSREADY, QB_DRAIN, QB_COUNT };
constexpr uint32_t Q_OFF_MISC = Q_OFF_BAR + QB_COUNT * 8;
constexpr uint32_t Q_OFF_SUM = Q_OFF_MISC + 16;  // [row] float
constexpr uint32_t Q_SMEM = Q_OFF_SUM + BM * 4;
// two CTAs and their 1 KB of system memory each in the SM's 228 KB: no room to
// round the base up, it is 1024-byte aligned by declaration (and checked)
static_assert(2 * (Q_SMEM + 1024) <= 233472, "two CTAs per SM");
constexpr uint32_t TQ_S = 0, TQ_DP = 64, TQ_DQ = 128;

// Where rows see few keys the tiles are walked twice, first for delta_t = sum_s
// P_ts dP_ts, which replaces the one from dh . h (for the dK/dV kernel after this one
// too): h was rounded to bf16, and with few keys it is so large that the error
// counts beside the rounding of dS.  (Relative errors of dq and dk against 64 bits
// at T = 150, window 140: 0.0028 from h, 0.0024 from the sweep; with 1024 keys 0.0024
// from h.)  The sweep adds two products to the three of a tile.
constexpr int kSweepWindow = 128;  // windows up to so many keys, and
constexpr int kSweepTokens = 512;  // the first tokens of a sequence

struct None {};
// kShared: a cluster of CTAs shares a query tile, each takes a stretch of its key
// tiles (a tile that is swept for delta, of few keys, is the first CTA's).  Out:
// the view of dq then, None for the unshared kernel (with the view among its
// arguments it measured 474 us, 440 without).
template <int D, bool kShared, typename Out>
__global__ void __launch_bounds__(kThreads, 2)
window_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                 const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ CUtensorMap tm_k16, const __grid_constant__ CUtensorMap tm_v16,
                 const __grid_constant__ CUtensorMap tm_dq, const BwdArgs a, const Out dq) {
    extern __shared__ __align__(1024) uint8_t smem_q[];
    uint8_t* gbase = smem_q;
    const uint32_t base = smem_u32(smem_q);
    if (base & 1023u) {  // not reached: the tiles' swizzle needs the alignment
        if (threadIdx.x == 0) atomicOr(&g_bwd_status[0], 2u);
        return;
    }
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + Q_OFF_MISC + 4);
    unsigned int* status = &g_bwd_status[0];
    const uint64_t lim = a.timeout_ns;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto BAR = [&](int i) { return base + Q_OFF_BAR + 8u * (uint32_t)i; };

    const int BH = a.B * a.Hq;
    const int cs = kShared ? (int)(gridDim.x / (unsigned)(BH * a.nt)) : 1, rank = kShared ? (int)blockIdx.x % cs : 0;
    const unsigned x0 = kShared ? blockIdx.x / cs : blockIdx.x;
    const int I = a.nt - 1 - (int)(x0 / BH), bh = (int)(x0 % BH);
    const int b = bh / a.Hq, hq = bh % a.Hq, hk = hq / a.G;
    const int t0 = I * BM, len = seq_len(a, b);
    int ns = 0, w0 = 0, nt = 0;  // as in the forward: tiles of sinks alone, then those the window reaches
    if (t0 < len) {
        const int lo = max(0, t0 - (a.window - 1));
        w0 = lo / BN;
        ns = min((a.sinks + BN - 1) / BN, w0);
        nt = ns + (min(t0 + BM, len) - 1) / BN + 1 - w0;
    }
    int j0 = 0;  // first tile of a cluster's stretch
    if constexpr (kShared) {
        if (a.sweep || t0 < kSweepTokens) {
            nt = rank > 0 ? 0 : nt;
        } else {  // tiles j0 .. of the list, counted from 0 again
            const int all = nt;
            j0 = all * rank / cs;
            nt = all * (rank + 1) / cs - j0;
            if (j0 >= ns) w0 += j0 - ns, ns = j0 = 0;
            else ns = min(ns - j0, nt);
        }
    }
    const int once = a.sweep || t0 < kSweepTokens ? nt : 0;  // tiles of the first sweep
    nt += once;
    auto tile_of = [&](int j) { return j >= once ? j - once : j; };
    auto tile_key = [&](int j) {
        const int x = tile_of(j);
        return (x < ns ? (kShared ? j0 : 0) + x : w0 + x - ns) * BN;
    };
    auto tile_keys = [&](int j) {
        const int x = tile_of(j);
        return x < ns ? min(BN, (a.sinks - ((kShared ? j0 : 0) + x) * BN + 15) & ~15) : BN;
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < QB_COUNT; ++i)
            mbar_init(BAR(i), i == QB_DSREADY || i == QB_SFREE ? kSoftmax : i == QB_SREADY && lim == kLostScoresNs ? 2 : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(base + Q_OFF_MISC, 256);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    launch_dependents();
    const uint32_t tmem = *reinterpret_cast<uint32_t*>(gbase + Q_OFF_MISC);
    const unsigned FULL = 0xffffffffu;
    auto wait = [&](int bar, uint32_t ph) -> bool {
        return __all_sync(FULL, mbar_wait(BAR(bar), ph & 1, abort_flag, status, lim));
    };

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (nt > 0 && elect_one()) {
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            mbar_expect_tx(BAR(QB_Q), 2 * BM * D * 2);
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
                tma_load_4d(base + Q_OFF_Q + x * BOX_M, &tm_q, BAR(QB_Q), 64 * x, t0, hq, b);
                tma_load_4d(base + Q_OFF_DO + x * BOX_M, &tm_do, BAR(QB_Q), 64 * x, t0, hq, b);
            }
        }
        __syncwarp();
        auto load = [&](const CUtensorMap* tm, const CUtensorMap* tm16, uint32_t bar, uint32_t dst, int j) {
            const int s0 = tile_key(j), keys = tile_keys(j);
            if (elect_one()) {
                mbar_expect_tx(bar, (uint32_t)keys * D * 2);
                if (keys < BN) {
                    for (int r = 0; r < keys; r += 16)
#pragma unroll
                        for (int x = 0; x < D / 64; ++x) tma_load_4d(dst + x * BOX_N + r * 128, tm16, bar, 64 * x, s0 + r, hk, b);
                } else {
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) tma_load_4d(dst + x * BOX_N, tm, bar, 64 * x, s0, hk, b);
                }
            }
            __syncwarp();
        };
        int nk = 0, nv = 0;
        for (int j = 0; j < nt; ++j) {
            if (j > 1 && !wait(QB_KEMPTY + (j & 1), (j >> 1) + 1)) break;
            load(&tm_k, &tm_k16, BAR(QB_KFULL + (j & 1)), base + Q_OFF_K + (j & 1) * TILE_N, j);
            nk = j + 1;
            if (j > 0 && !wait(QB_VEMPTY, j - 1)) break;
            load(&tm_v, &tm_v16, BAR(QB_VFULL), base + Q_OFF_V, j);
            nv = j + 1;
        }
        if (nt > 0) wait_drain(BAR(QB_Q), 0);
        for (int j = max(0, nk - 2); j < nk; ++j) wait_drain(BAR(QB_KFULL + (j & 1)), (j >> 1) & 1);
        if (nv > 0) wait_drain(BAR(QB_VFULL), (nv - 1) & 1);
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        constexpr uint32_t idesc_g = idesc_bf16_f32(BM, D, true);
        const uint64_t qdesc = smem_desc_sw128(base + Q_OFF_Q, 16, 1024), odesc = smem_desc_sw128(base + Q_OFF_DO, 16, 1024);
        const uint64_t kdesc = smem_desc_sw128(base + Q_OFF_K, 16, 1024), vdesc = smem_desc_sw128(base + Q_OFF_V, 16, 1024);
        const uint64_t kmdesc = smem_desc_sw128(base + Q_OFF_K, BOX_N, 1024);  // MN-major
        auto product = [&](uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc) {  // 128 x keys over D
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t m = (kk >> 2) * BOX_M + (kk & 3) * 32, o = (kk >> 2) * BOX_N + (kk & 3) * 32;
                mma_ss(d, desc_add(ad, m), desc_add(bd, o), idesc, kk > 0 ? 1u : 0u);
            }
        };
        auto scores = [&](int j) -> bool {  // S = Q K_j^T
            if (!wait(QB_KFULL + (j & 1), j >> 1)) return false;
            fence_after_sync();
            if (elect_one()) {
                product(tmem + TQ_S, qdesc, desc_add(kdesc, (j & 1) * TILE_N), idesc_bf16_f32(BM, tile_keys(j), false));
                mma_commit(BAR(QB_SREADY));
            }
            __syncwarp();
            return true;
        };
        auto values = [&](int j) -> bool {  // dP = dO V_j^T, behind the product that reads dS from its columns
            if (!wait(QB_VFULL, j)) return false;
            fence_after_sync();
            if (elect_one()) {
                product(tmem + TQ_DP, odesc, vdesc, idesc_bf16_f32(BM, tile_keys(j), false));
                mma_commit(BAR(QB_DPREADY));
                mma_commit(BAR(QB_VEMPTY));
            }
            __syncwarp();
            return true;
        };
        bool ok = nt == 0 || (wait(QB_Q, 0) && scores(0) && values(0));
        for (int j = 0; ok && j < nt; ++j) {
            if (j + 1 < nt) {  // the scores have been read: the next ones while dS is formed
                ok = wait(QB_SFREE, j) && scores(j + 1);
                if (!ok) break;
            }
            ok = wait(QB_DSREADY, j);
            if (!ok) break;
            fence_after_sync();
            const uint64_t kd = desc_add(kmdesc, (j & 1) * TILE_N);
            const int steps = tile_keys(j) / 16;
            if (elect_one()) {
                for (int kk = 0; kk < steps && j >= once; ++kk)
                    mma_ts(tmem + TQ_DQ, tmem + TQ_DP + 32 * (kk >> 1) + 8 * (kk & 1), desc_add(kd, kk * 2048), idesc_g,
                           j > once || kk > 0 ? 1u : 0u);
                mma_commit(BAR(QB_KEMPTY + (j & 1)));
            }
            __syncwarp();
            if (j + 1 < nt) ok = values(j + 1);
        }
        if (elect_one()) mma_commit(BAR(QB_DRAIN));
        __syncwarp();
        wait_drain(BAR(QB_DRAIN), 0);
    } else {
        // ------------------------------------------------ weights, two threads per query
        const int q4 = warp & 3, half = (warp - 2) >> 2;
        const int r = q4 * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
        const int t = t0 + r, c0 = 32 * half;
        const size_t row = ((size_t)b * a.Hq + hq) * a.Tp + t;  // (rows are padded to whole tiles)
        wait_for_previous();  // (the products start without the row values)
        const float nl = a.nlse[row], nd = once > 0 ? 0.f : a.ndelta[row];
        const f32x2 sl = mk2(a.scale_log2, a.scale_log2), nl2 = mk2(nl, nl);
        f32x2 nd2 = mk2(nd, nd);
        float delta = 0.f;  // sum of P dP over this half of the first sweep
        float* sums = reinterpret_cast<float*>(gbase + Q_OFF_SUM);
        bool ok = true, voted = false;
        for (int j = 0; j < nt; ++j) {
            if (j == once && once > 0) {  // the halves of delta, in order; the second sweep takes it, and dK/dV
                if (half == 1) sums[r] = delta;
                if (!bar_and(true, 1, kSoftmax)) {  // a warp has given up: this was the vote below
                    ok = false, voted = true;
                    break;
                }
                if (half == 0) sums[r] += delta;
                bar_sync(1, kSoftmax);
                const float d = -sums[r];
                nd2 = mk2(d, d);
                if (half == 0) const_cast<float*>(a.ndelta)[row] = d;
            }
            const int s0 = tile_key(j), keys = tile_keys(j);
            ok = wait(QB_SREADY, j);
            if (!ok) break;
            fence_after_sync();
            if (a.lens && s0 + BN > len) {
                // keys behind the end: cleared before they are summed over
                const int x = (int)threadIdx.x - 64, kr = x & 63, box = x >> 6;
                if (s0 + kr >= len && box < D / 64) {
                    uint4* p = reinterpret_cast<uint4*>(gbase + Q_OFF_K + (j & 1) * TILE_N + box * BOX_N + kr * 128);
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[e] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async();
                __syncwarp();
            }
            uint32_t u[32];
            if (c0 < keys) {
                tmem_ld32(trow + TQ_S + c0, u);
                tmem_wait_ld();
            }
            fence_before_sync();
            mbar_arrive(BAR(QB_SFREE));
            if (c0 < keys) {
                const uint32_t td = trow + TQ_DP + c0;
                // keys of this half that the row sees: the window's, or a sink
                const bool masked = s0 + BN - 1 > t0 || t0 + BM > len || s0 <= t0 + BM - 1 - a.window;
                uint32_t bits = 0xffffffffu;
                if (masked) {
                    const int hi = t < len ? t - s0 - c0 : -1;
                    bits = bit_range(t - a.window + 1 - s0 - c0, hi) | bit_range(0, min(a.sinks - s0 - c0 - 1, hi));
                }
                float p[32];
#pragma unroll
                for (int c = 0; c < 32; c += 2)
                    un2(fma2(mk2(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), sl, nl2), p[c], p[c + 1]);
#pragma unroll
                for (int c = 0; c < 32; ++c) p[c] = ex2(p[c]);
                ok = wait(QB_DPREADY, j);
                if (!ok) break;
                fence_after_sync();
                tmem_ld32(td, u);
                tmem_wait_ld();
                uint32_t pk[16];
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    float e0, e1;
                    un2(mul2(add2(mk2(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), nd2), mk2(p[c], p[c + 1])), e0, e1);
                    if (masked) {
                        if (!(bits >> c & 1u)) e0 = 0.f;
                        if (!(bits >> (c + 1) & 1u)) e1 = 0.f;
                    }
                    if (j < once) delta += e0 + e1;
                    pk[c / 2] = pack_bf16(e0, e1);
                }
                if (j >= once) {
                    tmem_st<16>(td, pk);
                    tmem_wait_st();
                }
            } else {
                // nothing of the tile is here, but an arrival before the barrier's
                // phase has begun would count for the tile before
                ok = wait(QB_DPREADY, j);
                if (!ok) break;
            }
            fence_before_sync();
            mbar_arrive(BAR(QB_DSREADY));
        }
        if (ok) ok = wait(QB_DRAIN, 0);
        if (!voted) ok = bar_and(ok && !*abort_flag, 1, kSoftmax);
        fence_after_sync();
        if constexpr (kShared) {  // the share over the tiles, float32: [row][D], 16-byte pieces swizzled by row
#pragma unroll 1
            for (int x = 0; ok && x < D / 64; ++x) {
                const int col = (D / 2) * half + 32 * x;
                uint32_t u[32];
                tmem_ld32(trow + TQ_DQ + col, u);
                tmem_wait_ld();
                uint4* dst = reinterpret_cast<uint4*>(gbase) + r * (D / 4);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dst[(col / 4 + e) ^ (r & 7)] = nt > 0 && t < len
                                                       ? make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3])
                                                       : make_uint4(0u, 0u, 0u, 0u);
            }
        } else if (ok) {
#pragma unroll 1
            for (int x = 0; x < D / 64; ++x) {  // the queries are used up
                const int col = (D / 2) * half + 32 * x;
                stage32(trow + TQ_DQ + col, a.scale, nt > 0 && t < len, gbase + Q_OFF_Q, col, r);
            }
        }
        if constexpr (!kShared) {
            fence_async();
            bar_sync(1, kSoftmax);
            if (warp == 2 && lane == 0 && ok) {
#pragma unroll
                for (int x = 0; x < D / 64; ++x) tma_store_4d(&tm_dq, base + Q_OFF_Q + x * BOX_M, 64 * x, t0, hq, b);
                bulk_commit_group();
                bulk_wait_group_read0();
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_dealloc(tmem, 256);
    }
    if constexpr (kShared) {  // the shares are summed in the order of the ranks, the rows spread over the CTAs
        static_assert(BM * D * 4 <= Q_OFF_BAR, "shares");
        __syncwarp();
        const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
        cluster.sync();
        constexpr int kAll = BM * D / 4, kBatch = 4;  // reads in flight
        const int e1 = (rank + 1) * kAll / cs;
        for (int e0 = rank * kAll / cs + (int)threadIdx.x; e0 < e1; e0 += kBatch * kThreads) {
            float4 s[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < cs; ++k) {
                const float4* share = reinterpret_cast<const float4*>(cluster.map_shared_rank(gbase, k));
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int e = e0 + i * kThreads, r = e / (D / 4), c = e % (D / 4);
                    if (e >= e1) continue;
                    const float4 v = share[e - c + (c ^ (r & 7))];
                    s[i].x += v.x, s[i].y += v.y, s[i].z += v.z, s[i].w += v.w;
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int e = e0 + i * kThreads, t = t0 + e / (D / 4), c = e % (D / 4);
                if (e < e1 && t < a.T)
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(dq.data) + (size_t)b * dq.sb +
                                              (size_t)hq * dq.sh + (size_t)t * dq.st + 4 * c) =
                        make_uint2(pack_bf16(s[i].x * a.scale, s[i].y * a.scale),
                                   pack_bf16(s[i].z * a.scale, s[i].w * a.scale));
            }
        }
        cluster.sync();  // the shares stay until every CTA has read them
    }
}

// Shape of a call: padded rows, reach and stretches of the first key tile.
constexpr int kClusterCtas = 148;
struct Plan {
    int window, sinks, nt, Tp, splits, cluster, cluster_q;
    size_t rows, bytes;
};
Plan plan_of(const ssa_window_params_t& p) {
    Plan x{};
    x.window = p.window > 0 && p.window < p.T ? p.window : p.T;
    x.sinks = x.window < p.T ? (p.sinks < p.T ? p.sinks : p.T) : 0;
    x.nt = (p.T + BM - 1) / BM;
    x.Tp = x.nt * BM;
    const long long last = (p.T - 1) / BM, reach = ((long long)BM - 1 + x.window - 1) / BM;
    if (x.sinks > 0 && last > reach) {
        // a stretch of queries as long as a key tile's usual list, 16 tiles at least, 64 stretches at most
        const long long usual = reach + 1 > 16 ? reach + 1 : 16, far = last - reach;
        const long long n = (far + usual - 1) / usual;
        x.splits = (int)(n < 64 ? n : 64);
    }
    // Few key tiles: clusters share their lists, as far as every CTA has an SM and two query tiles
    // (8/1 heads of 128, 1000 tokens, all keys, both directions: 171 -> 66 us; 4096 tokens, window
    // 1024: 246 -> 129 us).
    const long long items = (long long)p.B * p.Hkv * (x.nt + x.splits), list = p.Hq / p.Hkv * (reach < last ? reach + 1 : last + 1);
    x.cluster = 1;
    while (x.cluster < 8 && 2 * x.cluster * items <= kClusterCtas && 4 * x.cluster <= list) x.cluster *= 2;
    // Few query tiles likewise, of 32 key tiles at least, as in the forward (one head of 128, 8192
    // tokens, all keys, both directions: 280 -> 179 us).
    const long long ctas = (long long)p.B * p.Hq * x.nt, most = 2 * (long long)x.window > p.T ? 2 * kClusterCtas : kClusterCtas;
    long long keys = ((long long)x.window + BN - 2) / BN + 1 + (x.sinks + BN - 1) / BN;
    keys = keys < 2 * x.nt ? keys : 2 * x.nt;
    x.cluster_q = 1;
    while (keys >= 32 && x.cluster_q < 8 && 2 * x.cluster_q * ctas <= most && 8 * x.cluster_q <= keys) x.cluster_q *= 2;
    x.rows = align_up((size_t)p.B * p.Hq * x.Tp * sizeof(float), 256);
    x.bytes = 2 * x.rows;
    if (x.splits)
        x.bytes += align_up((size_t)p.B * p.Hkv * 2 * p.D * (BM + (size_t)x.splits * x.sinks) * sizeof(float), 256);
    return x;
}

template <int D>
int run(const ssa_window_params_t& p, const View& q, const View& k, const View& v, const View& h, const float* lse,
        const View& dh, const View& dq, const View& dk, const View& dv, BwdArgs a, int cluster_q, cudaStream_t s) {
    const bool shared = a.cluster > 1;
    int st = shared ? opt_in_max_smem<window_dkdv_kernel<D, true>>("window_dkdv_kernel")
                    : opt_in_max_smem<window_dkdv_kernel<D, false>>("window_dkdv_kernel");
    const bool shared_q = cluster_q > 1;
    if (st == SSA_OK)
        st = shared_q ? opt_in_max_smem<window_dq_kernel<D, true, View>>("window_dq_kernel")
                      : opt_in_max_smem<window_dq_kernel<D, false, None>>("window_dq_kernel");
    CUtensorMap k128, v128, mdk, mdv, q128, do128, k64, v64, k16, v16, mdq;
    struct { CUtensorMap* m; const View* x; int H, rows; } maps[] = {
        {&k128, &k, p.Hkv, BM}, {&v128, &v, p.Hkv, BM},
        {&mdk, &dk, p.Hkv, BM}, {&mdv, &dv, p.Hkv, BM}, {&q128, &q, p.Hq, BM}, {&do128, &dh, p.Hq, BM},
        {&k64, &k, p.Hkv, BN}, {&v64, &v, p.Hkv, BN}, {&k16, &k, p.Hkv, 16}, {&v16, &v, p.Hkv, 16},
        {&mdq, &dq, p.Hq, BM}};
    for (const auto& m : maps)
        if (st == SSA_OK) st = make_view_map(m.m, *m.x, D, p.T, m.H, p.B, m.rows);
    if (st != SSA_OK) return st;
    // Each kernel may begin while the one before runs out: it waits for that one only
    // where it needs its results (and so completes after it).
    constexpr int rows = 256 / (D / 8);
    window_rows_kernel<D><<<dim3((unsigned)(a.Tp / rows), (unsigned)p.Hq, (unsigned)p.B), 256, 0, s>>>(
        h, dh, lse, const_cast<float*>(a.nlse), const_cast<float*>(a.ndelta), a);
    st = check_launch("window_rows_kernel");
    if (st == SSA_OK)
        st = shared_q ? launch_beside_clusters("window_dq_kernel", window_dq_kernel<D, true, View>,
                                               dim3((unsigned)p.B * p.Hq * a.nt * cluster_q), (unsigned)cluster_q,
                                               kThreads, Q_SMEM, s, q128, do128, k64, v64, k16, v16, mdq, a, dq)
                      : launch_beside("window_dq_kernel", window_dq_kernel<D, false, None>, dim3((unsigned)p.B * p.Hq * a.nt),
                                      kThreads, Q_SMEM, s, q128, do128, k64, v64, k16, v16, mdq, a, None{});
    if (st == SSA_OK)
        st = launch_beside_clusters("window_dkdv_kernel", shared ? window_dkdv_kernel<D, true> : window_dkdv_kernel<D, false>,
                                    dim3((unsigned)p.B * p.Hkv * (a.nt + a.splits) * a.cluster), (unsigned)a.cluster,
                                    kThreadsK, K_SMEM, s, q128, do128, k128, v128, mdk, mdv, dk, dv, a);
    if (st == SSA_OK && a.splits)
        st = launch_beside("window_sink_kernel", window_sink_kernel<D>,
                           dim3(2u * p.B * p.Hkv, (unsigned)(BM * D / 4 / 256)), 256, 0, s, dk, dv, a);
    return st;
}

}  // namespace

bool window_bwd_tc_supported(const ssa_window_params_t& p) {
    return window_tc_supported(p) && (long long)p.B * p.Hq * ((p.T + BM - 1) / BM + 64) <= 0x7fffffffll;
}

size_t window_bwd_tc_workspace(const ssa_window_params_t& p) { return plan_of(p).bytes; }

int launch_window_bwd_tc(const ssa_window_params_t& p, const View& q, const View& k, const View& v,
                         const int32_t* lens, const View& h, const float* lse, const View& dh, const View& dq,
                         const View& dk, const View& dv, void* ws, cudaStream_t s) {
    const Plan x = plan_of(p);
    BwdArgs a{};
    a.lens = lens;
    a.nlse = static_cast<float*>(ws);
    a.ndelta = reinterpret_cast<float*>(static_cast<char*>(ws) + x.rows);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + 2 * x.rows);
    a.B = p.B, a.Hq = p.Hq, a.Hkv = p.Hkv, a.G = p.Hq / p.Hkv, a.T = p.T, a.Tp = x.Tp;
    a.window = x.window, a.sinks = x.sinks, a.nt = x.nt, a.splits = x.splits, a.cluster = x.cluster;
    a.sweep = x.window <= kSweepWindow;
    a.scale = p.sm_scale, a.scale_log2 = p.sm_scale * kLog2e;
    a.timeout_ns = wait_limit_ns();
    return p.D == 64 ? run<64>(p, q, k, v, h, lse, dh, dq, dk, dv, a, x.cluster_q, s)
                     : run<128>(p, q, k, v, h, lse, dh, dq, dk, dv, a, x.cluster_q, s);
}

int window_bwd_take_status() {
    unsigned int v[2] = {0, 0}, w = 0;
    cudaError_t e = cudaMemcpyFromSymbol(v, g_bwd_status, sizeof v);
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&w, g_bwd_range, sizeof w);
    if (e != cudaSuccess) return fail(SSA_ERR_CUDA, "status read: %s", cudaGetErrorString(e));
    const unsigned int zero[2] = {0, 0};
    if (v[0] | v[1]) cudaMemcpyToSymbol(g_bwd_status, zero, sizeof zero);
    if (w) cudaMemcpyToSymbol(g_bwd_range, zero, sizeof w);
    if ((v[0] | v[1]) & 1u)
        return fail(SSA_ERR_TIMEOUT, "%s%s%s: a bounded mbarrier wait expired", v[0] & 1u ? "window_dq_kernel" : "",
                    v[0] & v[1] & 1u ? " and " : "", v[1] & 1u ? "window_dkdv_kernel" : "");
    if (w) return fail(SSA_ERR_INVALID_ARG, "window attention: a length was out of range");
    if (v[0]) return fail(SSA_ERR_CUDA, "window_dq_kernel: shared memory is not aligned");
    return SSA_OK;
}

}  // namespace ssa
