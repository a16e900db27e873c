// Attention of a tile of 128 query rows on the sm_100a tensor cores (bf16 in,
// float32 accumulate): the forward of sliding-window attention with sinks
// (ssa_window_fwd), and the pass of a batch over its shared prefix in a paged
// cache (the first half of ssa_prefix_decode).
//
//   S = Q K_j^T, P = 2^(S sm_scale log2 e - m), l += rowsum P, O += P V_j
// over the key tiles j of 128 that some row of the tile sees.
//
// CTA = one query tile of one head, 288 threads, two CTAs on an SM:
//   warp 0      TMEM owner; issues the copies (Q once, then K_j and V_j, one
//               buffer each: K_j+1 is on its way while the weights of tile j
//               are formed, V_j+1 while those of tile j+1 are) and the MMAs.
//               One warp for both, so that two CTAs leave 112 registers for a
//               thread and a row's 64 scores stay in them.
//   warps 1..8  softmax, two threads per row with 64 keys of the tile each:
//               they read their scores from TMEM into registers, form P there
//               and write it back as bf16 over the scores.  (One thread per row
//               took 1.6 times as long per tile: four warps cannot hide each
//               other's latencies.)  The two warps of a row agree on its
//               running maximum by a vote, and exchange it only when it moves.
// TMEM: 256 of the 512 columns, S/P in [0, 128), O in [128, 128 + D); shared
// memory: 3 x 32 KB.  Within a CTA the products and the softmax of a tile
// follow one another; the two CTAs of an SM take turns, so the tensor cores
// work on one tile while the other's weights are formed.  (One CTA of two query
// tiles would need its roles to hand over more often for the same overlap, and
// with a window the work of a CTA is short: two CTAs also hide each other's
// first loads and last stores.)
//
// A row's running maximum is raised, and O rescaled, only when a tile exceeds
// it by more than 2^8; the sums are taken against the same maximum, so the
// result does not change.  Off the masked tiles three eighths of the weights
// come from a polynomial on the FMA pipe (2.7e-6), because the 16 exponentials
// per clock of an SM's special-function units would take as long as both
// products together.
//
// Sinks that the window has left behind are a key tile of their own, of
// 16-row steps: loads, products and weights cover ceil(sinks / 16) steps only.
//
// Keys and values behind a sequence's length may be NaN: their scores are
// replaced, and the value rows of the tile that holds the end are cleared in
// shared memory before the product (0 times NaN would spread).
//
// Every mbarrier wait is bounded; on expiry the kernel records
// SSA_ERR_TIMEOUT, the other roles stop, MMAs and copies in flight land, and
// TMEM is released.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "ssa_internal.h"
#include "tc_util.cuh"
#include "tmap.h"

namespace ssa {
namespace {

using namespace tc;

constexpr int BM = 128, BN = 128;
constexpr int kThreads = 288;
constexpr int kSoftmax = 256;
constexpr uint32_t HALF_BYTES = 128 * 128;  // [128 rows x 64 columns] bf16 box
constexpr uint32_t TILE_BYTES = 2 * HALF_BYTES;
constexpr uint32_t OFF_Q = 0, OFF_K = TILE_BYTES, OFF_V = 2 * TILE_BYTES, OFF_BAR = 3 * TILE_BYTES;
enum : int { B_QFULL, B_KFULL, B_VFULL, B_VEMPTY, B_SREADY, B_PREADY, B_DRAIN, B_COUNT };
constexpr uint32_t OFF_MISC = OFF_BAR + B_COUNT * 8;  // [0] tmem base, [1] abort flag
constexpr uint32_t OFF_XCH = OFF_MISC + 16;  // [parity][half][row] float: maxima, at the end sums
constexpr uint32_t SMEM_BYTES = OFF_XCH + 512 * 4 + 1024;  // slack for 1024-byte alignment
constexpr uint32_t TM_S = 0, TM_O = 128, kTmemCols = 256;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kLn2 = 0.693147180559945309f;

__device__ unsigned int g_attn_tc_status;   // bit 0: a wait expired
__device__ unsigned int g_attn_tc_range;    // a length (1) or page number (2) was out of range

struct AttnArgs {
    const int32_t* lens;  // window: lengths or NULL
    const int32_t* pages; // prefix: its pages
    float* lse;           // window
    float* part;          // prefix: partials, see prefix_slot
    int H;                // heads of the grid: query heads (window), key/value heads (prefix)
    int B, G, T, window, sinks;
    int ntq;              // query tiles of a sequence (window), row tiles of a head (prefix)
    int splits, page, n_pages, nb;  // prefix: CTAs per row tile, tokens of a page, batch entries of a row tile
    float scale_log2;
    unsigned long long timeout_ns;
};

__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer() - t0 > kDrainLimitNs) return false;
    return true;
}

// kPrefix: rows are (batch entry, query head of the group), keys the pages of
// the prefix, all of them seen; the CTA takes one stretch of the key tiles and
// writes a partial result.
template <int D, bool kPrefix>
__global__ void __launch_bounds__(kThreads, 2)
attn_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k16,
               const __grid_constant__ CUtensorMap tm_v16, const __grid_constant__ CUtensorMap tm_h,
               const AttnArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + OFF_MISC + 4);
    unsigned int* status = &g_attn_tc_status;
    const uint64_t lim = a.timeout_ns;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto BAR = [&](int i) { return base + OFF_BAR + 8u * (uint32_t)i; };

    // ---- the CTA's rows and key tiles
    int b = 0, h, t0 = 0, len, I;  // I: query tile / row tile
    int ns = 0, w0, nt;            // tiles: ns sink tiles (0 or 1), then w0 .. w0 + nt - ns - 1
    int split = 0;
    if constexpr (kPrefix) {
        split = (int)(blockIdx.x % a.splits);
        const int x = (int)(blockIdx.x / a.splits);
        I = x % a.ntq;
        h = x / a.ntq;
        len = a.T;
        const int n = (len + BN - 1) / BN;
        w0 = (int)((long long)n * split / a.splits);
        nt = (int)((long long)n * (split + 1) / a.splits) - w0;
    } else {
        const int BH = a.B * a.H;
        I = a.ntq - 1 - (int)(blockIdx.x / BH);  // late tiles first: without a window they are the longest
        const int bh = (int)(blockIdx.x % BH);
        b = bh / a.H;
        h = bh % a.H;
        t0 = I * BM;
        len = a.T;
        if (a.lens) {
            len = a.lens[b];
            if (len < 0 || len > a.T) {
                if (threadIdx.x == 0) atomicOr(&g_attn_tc_range, 1u);
                len = len < 0 ? 0 : a.T;
            }
        }
        if (t0 >= len) {
            nt = w0 = 0;
        } else {
            const int lo = max(0, t0 - (a.window - 1));
            w0 = lo / BN;
            ns = w0 > 0 && a.sinks > 0 ? 1 : 0;  // sinks fit into one tile; in reach of the window: no tile of their own
            nt = ns + I + 1 - w0;
        }
    }
    const int hk = kPrefix ? h : h / a.G;
    const int sink_rows = (a.sinks + 15) & ~15;  // keys that a sink tile loads and multiplies
    auto tile_key = [&](int j) { return (j < ns ? 0 : w0 + j - ns) * BN; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) mbar_init(BAR(i), i == B_PREADY ? kSoftmax : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(base + OFF_MISC, kTmemCols);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<uint32_t*>(gbase + OFF_MISC);
    const unsigned FULL = 0xffffffffu;

    if (warp == 0) {
        // ------------------------------------------------ copies and MMAs
        if (elect_one() && nt > 0) {
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            const int rows = kPrefix ? a.nb * a.G : BM;
            mbar_expect_tx(BAR(B_QFULL), (uint32_t)rows * D * 2);
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
                if constexpr (kPrefix) tma_load_4d(base + OFF_Q + x * HALF_BYTES, &tm_q, BAR(B_QFULL), 64 * x, 0, h, I * a.nb);
                else tma_load_4d(base + OFF_Q + x * HALF_BYTES, &tm_q, BAR(B_QFULL), 64 * x, t0, h, b);
            }
        }
        __syncwarp();
        // one K or V tile: whole boxes, the sinks' 16-row steps, or a box per page
        auto load = [&](bool is_k, int j) {
            const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
            const uint32_t bar = BAR(is_k ? B_KFULL : B_VFULL), dst = base + (is_k ? OFF_K : OFF_V);
            const int s0 = tile_key(j);
            if constexpr (kPrefix) {
                const int np = min(BN / a.page, (len - s0 + a.page - 1) / a.page);
                int pg = 0;
                if (lane < np) {
                    pg = a.pages[s0 / a.page + lane];
                    if (pg < 0 || pg >= a.n_pages) {
                        atomicOr(&g_attn_tc_range, 2u);
                        pg = 0;
                    }
                }
                if (lane == 0) mbar_expect_tx(bar, (uint32_t)(np * a.page) * D * 2);
                __syncwarp();
                if (lane < np) {
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        tma_load_4d(dst + x * HALF_BYTES + lane * a.page * 128, tm, bar, 64 * x, 0, hk, pg);
                }
            } else if (j < ns) {
                if (elect_one()) {
                    mbar_expect_tx(bar, (uint32_t)sink_rows * D * 2);
                    for (int r = 0; r < sink_rows; r += 16)
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tma_load_4d(dst + x * HALF_BYTES + r * 128, is_k ? &tm_k16 : &tm_v16, bar, 64 * x, r, hk, b);
                }
            } else if (elect_one()) {
                mbar_expect_tx(bar, BN * D * 2);
#pragma unroll
                for (int x = 0; x < D / 64; ++x) tma_load_4d(dst + x * HALF_BYTES, tm, bar, 64 * x, s0, hk, b);
            }
            __syncwarp();
        };
        auto wait = [&](int bar, uint32_t ph) -> bool {
            return __all_sync(FULL, mbar_wait(BAR(bar), ph, abort_flag, status, lim));
        };
        const uint64_t qdesc = smem_desc_sw128(base + OFF_Q, 16, 1024);          // K-major
        const uint64_t kdesc = smem_desc_sw128(base + OFF_K, 16, 1024);          // K-major
        const uint64_t vdesc = smem_desc_sw128(base + OFF_V, HALF_BYTES, 1024);  // MN-major
        constexpr uint32_t idesc_pv = idesc_bf16_f32(BM, D, true);
        auto tile_keys = [&](int j) { return j < ns ? sink_rows : BN; };
        auto scores = [&](int j) {  // S = Q K_j^T
            const uint32_t idesc_qk = idesc_bf16_f32(BM, tile_keys(j), false);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * HALF_BYTES + (kk & 3) * 32;
                    mma_ss(tmem + TM_S, desc_add(qdesc, off), desc_add(kdesc, off), idesc_qk, kk > 0 ? 1u : 0u);
                }
                mma_commit(BAR(B_SREADY));
            }
            __syncwarp();
        };
        int nk = 0, nv = 0;  // tiles whose copies have been issued
        if (nt > 0) {
            load(true, 0);
            load(false, 0);
            nk = nv = 1;
        }
        bool ok = nt == 0 || (wait(B_QFULL, 0) && wait(B_KFULL, 0));
        if (ok && nt > 0) {
            fence_after_sync();
            scores(0);
        }
        for (int j = 0; ok && j < nt; ++j) {
            const uint32_t ph = j & 1;
            if (j + 1 < nt) {  // K is free once the scores are there
                ok = wait(B_SREADY, ph);
                if (!ok) break;
                load(true, j + 1);
                nk = j + 2;
            }
            ok = wait(B_PREADY, ph) && wait(B_VFULL, ph);
            if (!ok) break;
            fence_after_sync();
            const int steps = tile_keys(j) / 16;
            if (elect_one()) {
                for (int kk = 0; kk < steps; ++kk)
                    mma_ts(tmem + TM_O, tmem + TM_S + 64 * (kk >> 2) + 8 * (kk & 3), desc_add(vdesc, kk * 2048), idesc_pv,
                           j > 0 || kk > 0 ? 1u : 0u);
                mma_commit(BAR(B_VEMPTY));
            }
            __syncwarp();
            if (j + 1 < nt) {
                ok = wait(B_KFULL, ph ^ 1);
                if (!ok) break;
                fence_after_sync();
                scores(j + 1);  // in order behind the product that reads P from the same columns
                ok = wait(B_VEMPTY, ph);
                if (!ok) break;
                load(false, j + 1);
                nv = j + 2;
            }
        }
        if (elect_one()) mma_commit(BAR(B_DRAIN));
        __syncwarp();
        wait_drain(BAR(B_DRAIN), 0);
        // copies in flight land before the CTA ends, also where a wait gave up
        if (nt > 0) wait_drain(BAR(B_QFULL), 0);
        if (nk > 0) wait_drain(BAR(B_KFULL), (nk - 1) & 1);
        if (nv > 0) wait_drain(BAR(B_VFULL), (nv - 1) & 1);
    } else {
        // ------------------------------------------------ softmax, two threads per row
        const int q4 = warp & 3, half = (warp - 1) >> 2;  // the warp's TMEM lanes; its half of the keys
        const int r = q4 * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
        const uint32_t sb = trow + TM_S + 64 * half;       // 64 scores; P over the first 32 of these columns
        const uint32_t ob = trow + TM_O + (D / 2) * half;  // the thread's share of O
        const int c0 = 64 * half;
        float* xch = reinterpret_cast<float*>(gbase + OFF_XCH);
        const int t = t0 + r;
        const float sl2 = a.scale_log2;
        float m2 = -INFINITY, l = 0.f;
        bool ok = true;
        // or-vote of the two warps that hold the same rows
        auto pair_vote = [q4](bool flag) -> bool {
            uint32_t out;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.u32 q, %1, 0;\n\t"
                "bar.red.or.pred p, %2, 64, q;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(out)
                : "r"((uint32_t)flag), "r"(2 + q4)
                : "memory");
            return out != 0;
        };
        // The running maximum (log2 units) after scores up to mx in this half, and
        // O rescaled where it moved.  False: a wait gave up in either warp.
        auto raise = [&](float mx, int j, bool got) -> bool {
            const bool moved = j == 0 || mx * sl2 > m2 + kRescaleThreshold;
            if (!pair_vote(moved || !got)) return true;
            float* xm = xch + (j & 1) * 256;
            xm[half * 128 + r] = mx;
            if (pair_vote(!got)) return false;
            const float mn = fmaxf(mx, xm[(1 - half) * 128 + r]) * sl2;
            if (j == 0) {
                m2 = mn;
                return true;
            }
            const bool need = mn > m2 + kRescaleThreshold;
            if (__any_sync(FULL, need)) {  // O is complete: its last product came before these scores
                const float up = need ? mn : m2;
                const float al = up == m2 ? 1.f : ex2(m2 - up);  // m2 may be -inf
                m2 = up;
                l *= al;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {  // (16 at a time: the scores stay in registers)
                    uint32_t o[16];
                    tmem_ld<16>(ob + 16 * c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
                    tmem_st<16>(ob + 16 * c, o);
                }
            }
            return true;
        };
        for (int j = 0; j < nt; ++j) {
            const int s0 = tile_key(j) + c0;  // the first of the thread's keys
            bool got = __all_sync(FULL, mbar_wait(BAR(B_SREADY), j & 1, abort_flag, status, lim));
            fence_after_sync();
            // rows that end in this tile: nothing stored behind the end may reach the product
            const int end = len - s0;
            if (end + c0 < BN && (kPrefix || a.lens)) {
                got = got && __all_sync(FULL, mbar_wait(BAR(B_VFULL), j & 1, abort_flag, status, lim));
                if (got && r >= end + c0 && half < D / 64) {
                    uint4* p = reinterpret_cast<uint4*>(gbase + OFF_V + half * HALF_BYTES + r * 128);
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i] = make_uint4(0u, 0u, 0u, 0u);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            if (j < ns) {
                // the sinks on their own: every row is past all of them
                const int cols = min(64, sink_rows - c0);
                float mx = -INFINITY;
                for (int c1 = 0; c1 < cols; c1 += 16) {
                    uint32_t u[16];
                    tmem_ld<16>(sb + c1, u);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (c0 + c1 + c < a.sinks) mx = fmaxf(mx, __uint_as_float(u[c]));
                }
                ok = raise(mx, j, got);
                if (!ok) break;
                for (int c1 = 0; c1 < cols; c1 += 16) {
                    uint32_t u[16], pk[8];
                    tmem_ld<16>(sb + c1, u);
                    tmem_wait_ld();
                    float p[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        p[c] = c0 + c1 + c < a.sinks ? ex2(fmaf(__uint_as_float(u[c]), sl2, -m2)) : 0.f;
                        l += p[c];
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c) pk[c] = pack_bf16(p[2 * c], p[2 * c + 1]);
                    // P of columns c1 .. lies over scores c1 / 2 .., which have been read
                    tmem_st<8>(sb + c1 / 2, pk);
                }
            } else {
                float s[64];
                {
                    uint32_t u0[32], u1[32];
                    tmem_ld32(sb, u0);
                    tmem_ld32(sb + 32, u1);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; ++c) s[c] = __uint_as_float(u0[c]), s[32 + c] = __uint_as_float(u1[c]);
                }
                // keys of this half that the row sees: lo <= c <= hi, or a sink c <= sh
                bool masked;
                if constexpr (kPrefix) {
                    masked = end < 64;
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (c >= end) s[c] = -INFINITY;
                    }
                } else {
                    masked = s0 + 63 > t0 || end < 64 || s0 <= t0 + BM - 1 - a.window;
                    if (masked) {
                        const int hi = min(t, len - 1) - s0, lo = max(t - a.window + 1 - s0, 0);
                        const unsigned span = hi >= lo ? (unsigned)(hi - lo) : 0u;
                        const int off = hi >= lo ? lo : 64;  // an empty range lies past the half
                        const int sh = min(a.sinks - s0 - 1, hi);
                        if (a.sinks <= s0) {
#pragma unroll
                            for (int c = 0; c < 64; ++c)
                                if ((unsigned)(c - off) > span) s[c] = -INFINITY;
                        } else {
#pragma unroll
                            for (int c = 0; c < 64; ++c)
                                if ((unsigned)(c - off) > span && c > sh) s[c] = -INFINITY;
                        }
                    }
                }
                float mx4[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mx4[k] = fmaxf(s[k], s[4 + k]);
#pragma unroll
                    for (int c = 8; c < 64; c += 8) mx4[k] = max3(mx4[k], s[c + k], s[c + 4 + k]);
                }
                ok = raise(max3(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3])), j, got);
                if (!ok) break;
                const float neg = m2 == -INFINITY ? 0.f : -m2;  // a row that has seen nothing: 2^-inf = 0
                const f32x2 sl = mk2(sl2, sl2), nm = mk2(neg, neg);
                f32x2 acc[4] = {mk2(0.f, 0.f), mk2(0.f, 0.f), mk2(0.f, 0.f), mk2(0.f, 0.f)};
                auto weights = [&](auto poly) {
#pragma unroll
                    for (int c1 = 0; c1 < 32; c1 += 8) {
                        uint32_t pk[8];
#pragma unroll
                        for (int i = c1; i < c1 + 8; ++i) {
                            const f32x2 x2 = fma2(mk2(s[2 * i], s[2 * i + 1]), sl, nm);
                            float p0, p1;
                            if (decltype(poly)::value && ((i & 7) == 1 || (i & 7) == 4 || (i & 7) == 6)) {
                                un2(exp2_poly4_2(x2), p0, p1);
                            } else {
                                float x0, x1;
                                un2(x2, x0, x1);
                                p0 = ex2(x0);
                                p1 = ex2(x1);
                            }
                            acc[i & 3] = add2(acc[i & 3], mk2(p0, p1));
                            pk[i - c1] = pack_bf16(p0, p1);
                        }
                        tmem_st<8>(sb + c1, pk);
                    }
                };
                if (masked) weights(std::false_type{});
                else weights(std::true_type{});
                float x0, x1, y0, y1;
                un2(add2(acc[0], acc[1]), x0, x1);
                un2(add2(acc[2], acc[3]), y0, y1);
                l += (x0 + x1) + (y0 + y1);
            }
            tmem_wait_st();
            fence_before_sync();
            mbar_arrive(BAR(B_PREADY));
        }
        if (ok) ok = __all_sync(FULL, mbar_wait(BAR(B_DRAIN), 0, abort_flag, status, lim));
        // the two halves' sums (the maxima of the last two tiles may still be read: a barrier first)
        ok = bar_and(ok && !*abort_flag, 1, kSoftmax);
        xch[half * 128 + r] = l;
        bar_sync(1, kSoftmax);
        l += xch[(1 - half) * 128 + r];
        fence_after_sync();
        if constexpr (kPrefix) {
            // unnormalised outputs, then the maximum and the sum, in float32
            const int row_b = I * a.nb + r / a.G;
            if (ok) {
                const bool row = r < a.nb * a.G && row_b < a.B;
                float* slot = a.part + ((size_t)(h * a.ntq + I) * a.splits + split) * BM * (D + 2);
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t u[32];
                    tmem_ld32(ob + 32 * c, u);
                    tmem_wait_ld();
                    if (row)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            reinterpret_cast<uint4*>(slot + (size_t)r * D + (D / 2) * half + 32 * c)[i] =
                                make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
                }
                if (row && half == 0) *reinterpret_cast<float2*>(slot + BM * D + 2 * r) = make_float2(m2, l);
            }
        } else {
            const bool row = t < len;
            const float inv = row ? 1.f / l : 0.f;
            uint8_t* tile = gbase + OFF_Q + (uint32_t)r * 128;  // the queries are used up
            if (ok) {
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t u[32];
                    if (nt > 0) tmem_ld32(ob + 32 * c, u);
                    tmem_wait_ld();
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = row ? pack_bf16(__uint_as_float(u[8 * v + 2 * e]) * inv,
                                                   __uint_as_float(u[8 * v + 2 * e + 1]) * inv)
                                       : 0u;
                        const int col = (D / 2) * half + 32 * c + 8 * v;
                        const uint32_t chunk = (uint32_t)((col & 63) >> 3) ^ (uint32_t)(r & 7);
                        *reinterpret_cast<uint4*>(tile + (col >> 6) * HALF_BYTES + chunk * 16) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                if (half == 0 && t < a.T)
                    a.lse[((size_t)b * a.H + h) * a.T + t] = row ? (m2 + log2f(l)) * kLn2 : -INFINITY;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            bar_sync(1, kSoftmax);
            if (warp == 1 && lane == 0 && ok) {
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    tma_store_4d(&tm_h, base + OFF_Q + x * HALF_BYTES, 64 * x, t0, h, b);
                bulk_commit_group();
                bulk_wait_group_read0();
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, bool kPrefix>
int launch(const CUtensorMap (&m)[6], const AttnArgs& a, long long grid, cudaStream_t s) {
    const char* name = kPrefix ? "attn_tc_kernel<prefix>" : "attn_tc_kernel<window>";
    const int st = opt_in_max_smem<attn_tc_kernel<D, kPrefix>>(name);
    if (st != SSA_OK) return st;
    attn_tc_kernel<D, kPrefix><<<(unsigned)grid, kThreads, SMEM_BYTES, s>>>(m[0], m[1], m[2], m[3], m[4], m[5], a);
    return check_launch(name);
}

}  // namespace

int make_map4(CUtensorMap* m, void* ptr, const unsigned long long (&dims)[4], const long long (&strides)[3],
              const unsigned (&box)[4]) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    if (!fn) return fail(SSA_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    cuuint64_t d[4], st[3];
    cuuint32_t bx[4], es[4] = {1, 1, 1, 1};
    for (int i = 0; i < 4; ++i) d[i] = dims[i], bx[i] = box[i];
    for (int i = 0; i < 3; ++i) st[i] = (cuuint64_t)strides[i] * 2;
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, ptr, d, st, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(SSA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return SSA_OK;
}

int make_view_map(CUtensorMap* m, const View& v, int D, int T, int H, int B, int rows) {
    return make_map4(m, v.data, {(unsigned long long)D, (unsigned long long)T, (unsigned long long)H, (unsigned long long)B},
                     {v.st, v.sh, v.sb}, {64, (unsigned)rows, 1, 1});
}

bool window_tc_supported(const ssa_window_params_t& p) {
    return p.dtype == SSA_BF16 && !(p.flags & SSA_FLAG_FORCE_SIMT) &&
           (long long)p.B * p.Hq * ((p.T + BM - 1) / BM) <= 0x7fffffffll;
}

int launch_window_fwd_tc(const ssa_window_params_t& p, const View& q, const View& k, const View& v,
                         const int32_t* lens, const View& h, float* lse, cudaStream_t s) {
    CUtensorMap m[6];
    int st = make_view_map(&m[0], q, p.D, p.T, p.Hq, p.B, BM);
    if (st == SSA_OK) st = make_view_map(&m[1], k, p.D, p.T, p.Hkv, p.B, BN);
    if (st == SSA_OK) st = make_view_map(&m[2], v, p.D, p.T, p.Hkv, p.B, BN);
    if (st == SSA_OK) st = make_view_map(&m[3], k, p.D, p.T, p.Hkv, p.B, 16);
    if (st == SSA_OK) st = make_view_map(&m[4], v, p.D, p.T, p.Hkv, p.B, 16);
    if (st == SSA_OK) st = make_view_map(&m[5], h, p.D, p.T, p.Hq, p.B, BM);
    if (st != SSA_OK) return st;
    AttnArgs a{};
    a.lens = lens, a.lse = lse, a.H = p.Hq, a.B = p.B, a.G = p.Hq / p.Hkv, a.T = p.T;
    a.window = p.window > 0 && p.window < p.T ? p.window : p.T;
    a.sinks = a.window < p.T ? p.sinks : 0;
    a.ntq = (p.T + BM - 1) / BM;
    a.scale_log2 = p.sm_scale * 1.4426950408889634f;
    a.timeout_ns = wait_limit_ns();
    const long long grid = (long long)p.B * p.Hq * a.ntq;
    return p.D == 64 ? launch<64, false>(m, a, grid, s) : launch<128, false>(m, a, grid, s);
}

int attn_tc_take_status() {
    unsigned int v = 0, w = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_tc_status, sizeof v);
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&w, g_attn_tc_range, sizeof w);
    if (e != cudaSuccess) return fail(SSA_ERR_CUDA, "status read: %s", cudaGetErrorString(e));
    const unsigned int zero = 0;
    if (v) {
        cudaMemcpyToSymbol(g_attn_tc_status, &zero, sizeof zero);
        return fail(SSA_ERR_TIMEOUT, "attn_tc_kernel: a bounded mbarrier wait expired");
    }
    if (w) {
        cudaMemcpyToSymbol(g_attn_tc_range, &zero, sizeof zero);
        return fail(SSA_ERR_INVALID_ARG, "attention: a %s was out of range", w & 2u ? "page number" : "length");
    }
    return SSA_OK;
}

}  // namespace ssa
