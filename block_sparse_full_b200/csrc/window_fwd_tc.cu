// Attention of a tile of 128 query rows on the sm_100a tensor cores (bf16 in,
// float32 accumulate): the forward of sliding-window attention with sinks
// (ssa_window_fwd), and the pass of a batch over its shared prefix in a paged
// cache (the first half of ssa_prefix_decode).
//
//   S = Q K_j^T, P = 2^(S sm_scale log2 e - m), l += rowsum P, O += P V_j
// over the key tiles j of 64 that some row of the tile sees.
//
// CTA = one query tile of one head, 192 threads, two CTAs on an SM:
//   warp 0      TMA producer: Q once, then K_j into a ring of three and V_j into
//               one of two
//   warp 1      TMEM owner and MMA issuer (one thread)
//   warps 2..5  softmax, a thread per row: it reads its 64 scores from TMEM
//               into registers, forms P there and writes it back as bf16 over
//               the scores.
// TMEM: 256 of the 512 columns: S/P in two buffers of 64, O in [128, 128 + D);
// shared memory: 112 KB.  The scores of tile j+1 are formed while the weights
// of tile j are, and the product with V_j while those of tile j+1 are, so a
// CTA's softmax does not wait for its products; the second CTA of the SM fills
// the softmax's own latencies, the first loads and the last stores.  Tiles are
// 64 keys wide because two buffers of 128 beside O would leave TMEM for one
// CTA only; a score product 64 wide re-reads Q from shared memory at 3/4 of
// the tensor rate, which costs less than it gains: with one buffer of 128 keys
// (products and softmax of a CTA taking turns) T = 65536, 8 heads, window 2048
// took 578 us.
//
// A row's running maximum is raised, and O rescaled, only when a tile exceeds
// it by more than 2^8; the sums are taken against the same maximum, so the
// result does not change.  All weights come from the special-function units; a
// polynomial on the FMA pipe for a part of them measured slower at every share
// from an eighth to a half (the softmax is bound by latency and issue slots).
//
// P is rounded to bf16 because both operands of a product have one 16-bit type and V
// is bf16; each weight is then off by at most 2^-8 of itself, independently of the
// others.  l takes the weights before that rounding, in float32.  Against 64 bits h
// is off by a relative 0.0024 (root mean square), where its own rounding alone is 0.0016.
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
#include <cooperative_groups.h>
#include <cuda.h>

#include "ssa_internal.h"
#include "device_util.cuh"
#include "tc_util.cuh"
#include "tmap.h"

namespace ssa {
namespace {

using namespace tc;

constexpr int BM = 128, BN = 64;
constexpr int kThreads = 192;
constexpr uint32_t Q_BOX = BM * 128;  // [128 rows x 64 columns] bf16 box
constexpr uint32_t KV_BOX = BN * 128; // [64 rows x 64 columns]
constexpr uint32_t KV_BYTES = 2 * KV_BOX;
constexpr int kK = 3;  // slots of K; V, the scores and their barriers have two
constexpr uint32_t OFF_Q = 0, OFF_K = 2 * Q_BOX, OFF_V = OFF_K + kK * KV_BYTES, OFF_BAR = OFF_V + 2 * KV_BYTES;
enum : int {  // one of Q, kK of K, two of the others: tile j uses number j % 2
    B_QFULL, B_KFULL, B_KEMPTY = B_KFULL + kK, B_VFULL = B_KEMPTY + kK, B_VEMPTY = B_VFULL + 2, B_SREADY = B_VEMPTY + 2,
    B_PREADY = B_SREADY + 2, B_DRAIN = B_PREADY + 2, B_COUNT
};
constexpr uint32_t OFF_MISC = OFF_BAR + B_COUNT * 8;  // [0] tmem base, [1] abort flag
// two CTAs and their 1 KB of system memory each in the SM's 228 KB: no room to
// round the base up, it is 1024-byte aligned by declaration (and checked)
constexpr uint32_t SMEM_BYTES = OFF_MISC + 16;
static_assert(2 * (SMEM_BYTES + 1024) <= 233472, "two CTAs per SM");
constexpr int kSharedCtas = 296, kSharedTiles = 4;  // CTAs of clusters at most, key tiles of each at least
constexpr int kPrefixCtas = 296, kPrefixTiles = 2;  // CTAs of a pass over a prefix, at least so many key tiles each
constexpr uint32_t TM_S = 0, TM_O = 128, kTmemCols = 256;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kLn2 = 0.693147180559945309f;

__device__ unsigned int g_attn_tc_status;   // bit 0: a wait expired, bit 1: misaligned shared memory
__device__ unsigned int g_attn_tc_range;    // a length (1) or page number (2) was out of range

struct AttnArgs {
    const int32_t* lens;  // window: lengths or NULL
    const int32_t* pages; // prefix: its pages
    float* lse;           // window
    float* part;          // prefix: partials, see prefix_slot
    int H;                // heads of the grid: query heads (window), key/value heads (prefix)
    int B, G, T, window, sinks;
    int ntq;              // query tiles of a sequence (window), row tiles of a head (prefix)
    View h;               // window, where a cluster shares a query tile
    int cluster;          // its CTAs
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
// writes a partial result.  kShared: a cluster of CTAs shares a query tile, each
// takes a stretch of its key tiles.
template <int D, bool kPrefix, bool kShared>
__global__ void __launch_bounds__(kThreads, 2)
attn_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k16,
               const __grid_constant__ CUtensorMap tm_v16, const __grid_constant__ CUtensorMap tm_h,
               const AttnArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_tiles[];
    uint8_t* gbase = smem_tiles;
    const uint32_t base = smem_u32(smem_tiles);
    if (base & 1023u) {  // not reached: the tiles' swizzle needs the alignment
        if (threadIdx.x == 0) atomicOr(&g_attn_tc_status, 2u);
        return;
    }
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + OFF_MISC + 4);
    unsigned int* status = &g_attn_tc_status;
    const uint64_t lim = a.timeout_ns;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto BAR = [&](int i) { return base + OFF_BAR + 8u * (uint32_t)i; };

    // ---- the CTA's rows and key tiles
    int b = 0, h, t0 = 0, len, I;  // I: query tile / row tile
    int ns = 0, w0, nt;            // tiles: ns sink tiles (0 to 2), then w0 .. w0 + nt - ns - 1
    int split = 0;
    int j0 = 0;                    // first tile of a cluster's stretch
    const int cs = kShared ? a.cluster : 1, rank = (int)blockIdx.x % cs;
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
        const int x = (int)blockIdx.x / cs;
        I = a.ntq - 1 - x / BH;  // late tiles first: without a window they are the longest
        const int bh = x % BH;
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
            ns = min((a.sinks + BN - 1) / BN, w0);  // tiles of sinks that every row's window has left behind
            nt = ns + (min(t0 + BM, len) - 1) / BN + 1 - w0;
        }
        if constexpr (kShared) {  // tiles j0 .. of the list, counted from 0 again
            const int all = nt;
            j0 = all * rank / cs;
            nt = all * (rank + 1) / cs - j0;
            if (j0 >= ns) w0 += j0 - ns, ns = j0 = 0;
            else ns = min(ns - j0, nt);
        }
    }
    const int hk = kPrefix ? h : h / a.G;
    // bytes between the 64-column parts of a K or V row and between groups of eight
    // rows: a view's tile is two boxes of 64 rows, a page's rows come in one box
    constexpr uint32_t kCols = kPrefix ? 1024 : KV_BOX, kEight = kPrefix ? 16 * D : 1024;
    auto tile_key = [&](int j) { return (j < ns ? j0 + j : w0 + j - ns) * BN; };
    // keys that tile j loads and multiplies: of a sink tile whole steps of 16
    auto tile_keys = [&](int j) { return j < ns ? min(BN, (a.sinks - (j0 + j) * BN + 15) & ~15) : BN; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i)
            mbar_init(BAR(i), i >= B_PREADY && i < B_DRAIN ? 128 : i == B_SREADY && lim == kLostScoresNs ? 2 : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(base + OFF_MISC, kTmemCols);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if constexpr (kPrefix) ssa::launch_dependents();
    const uint32_t tmem = *reinterpret_cast<uint32_t*>(gbase + OFF_MISC);
    const unsigned FULL = 0xffffffffu;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (elect_one() && nt > 0) {
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            const int rows = kPrefix ? a.nb * a.G : BM;
            mbar_expect_tx(BAR(B_QFULL), (uint32_t)rows * D * 2);
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
                if constexpr (kPrefix) tma_load_4d(base + OFF_Q + x * Q_BOX, &tm_q, BAR(B_QFULL), 64 * x, 0, h, I * a.nb);
                else tma_load_4d(base + OFF_Q + x * Q_BOX, &tm_q, BAR(B_QFULL), 64 * x, t0, h, b);
            }
        }
        __syncwarp();
        // the pages of tile j, one to a lane
        auto page_of = [&](int j) -> int {
            int pg = 0;
            if constexpr (kPrefix) {
                const int s0 = tile_key(j), step = min(BN, a.page);
                if (j < nt && lane < BN / step && s0 + lane * step < len) pg = a.pages[(s0 + lane * step) / a.page];
            }
            return pg;
        };
        // one K or V tile: whole boxes, the sinks' 16-row steps, or a box per page
        auto load = [&](bool is_k, int j, int pg) {
            const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
            const uint32_t bar = BAR(is_k ? B_KFULL + j % kK : B_VFULL + (j & 1));
            const uint32_t dst = base + (is_k ? OFF_K + j % kK * KV_BYTES : OFF_V + (j & 1) * KV_BYTES);
            const int s0 = tile_key(j), keys = tile_keys(j);
            if constexpr (kPrefix) {
                const int step = min(BN, a.page);  // rows of a box
                const int np = min(BN / step, (len - s0 + step - 1) / step);
                if (lane < np && (pg < 0 || pg >= a.n_pages)) {
                    atomicOr(&g_attn_tc_range, 2u);
                    pg = 0;
                }
                if (lane == 0) mbar_expect_tx(bar, (uint32_t)(np * step) * D * 2);
                __syncwarp();
                if (lane < np)
                    tma_load_5d(dst + lane * step * 2 * D, tm, bar, 0, 0, 0, (hk * a.page + s0 % a.page) / 8, pg);
            } else if (elect_one()) {
                mbar_expect_tx(bar, (uint32_t)keys * D * 2);
                if (keys < BN) {
                    for (int r = 0; r < keys; r += 16)
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tma_load_4d(dst + x * KV_BOX + r * 128, is_k ? &tm_k16 : &tm_v16, bar, 64 * x, s0 + r, hk, b);
                } else {
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) tma_load_4d(dst + x * KV_BOX, tm, bar, 64 * x, s0, hk, b);
                }
            }
            __syncwarp();
        };
        // K runs kK tiles ahead of V: behind V_j in line, K_j+1 would be asked for only
        // one tile before its scores are due
        int nk = 0, nv = 0, pg[kK + 1];
#pragma unroll
        for (int i = 0; i <= kK; ++i) pg[i] = page_of(i);
#pragma unroll
        for (int i = 0; i < kK; ++i)
            if (i < nt) {
                load(true, i, pg[i]);
                nk = i + 1;
            }
        for (int j = 0; j < nt; ++j) {
            if (j > 1 && !__all_sync(FULL, mbar_wait(BAR(B_VEMPTY + (j & 1)), ((j >> 1) + 1) & 1, abort_flag, status, lim))) break;
            load(false, j, pg[0]);
            nv = j + 1;
            const int jk = j + kK;
            if (jk < nt) {
                if (!__all_sync(FULL, mbar_wait(BAR(B_KEMPTY + jk % kK), (jk / kK + 1) & 1, abort_flag, status, lim))) break;
                load(true, jk, pg[kK]);
                nk = jk + 1;
            }
#pragma unroll
            for (int i = 0; i < kK; ++i) pg[i] = pg[i + 1];
            pg[kK] = page_of(jk + 1);  // (not looked at before it is used: nothing waits for it here)
        }
        // copies in flight land before the CTA ends, also where a wait gave up
        if (nt > 0) wait_drain(BAR(B_QFULL), 0);
        for (int j = max(0, nk - kK); j < nk; ++j) wait_drain(BAR(B_KFULL + j % kK), (j / kK) & 1);
        for (int j = max(0, nv - 2); j < nv; ++j) wait_drain(BAR(B_VFULL + (j & 1)), (j >> 1) & 1);
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        const uint64_t qdesc = smem_desc_sw128(base + OFF_Q, 16, 1024);      // K-major
        const uint64_t kdesc = smem_desc_sw128(base + OFF_K, 16, kEight);    // K-major
        const uint64_t vdesc = smem_desc_sw128(base + OFF_V, kCols, kEight); // MN-major
        constexpr uint32_t idesc_pv = idesc_bf16_f32(BM, D, true);
        auto wait = [&](int bar, int j) -> bool {
            return __all_sync(FULL, mbar_wait(BAR(bar + (j & 1)), (j >> 1) & 1, abort_flag, status, lim));
        };
        auto scores = [&](int j) -> bool {  // S = Q K_j^T, behind the product that reads P from the same columns
            if (!__all_sync(FULL, mbar_wait(BAR(B_KFULL + j % kK), (j / kK) & 1, abort_flag, status, lim))) return false;
            fence_after_sync();
            const uint32_t idesc_qk = idesc_bf16_f32(BM, tile_keys(j), false);
            const uint64_t kd = desc_add(kdesc, j % kK * KV_BYTES);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(tmem + TM_S + BN * (j & 1), desc_add(qdesc, (kk >> 2) * Q_BOX + (kk & 3) * 32),
                           desc_add(kd, (kk >> 2) * kCols + (kk & 3) * 32), idesc_qk, kk > 0 ? 1u : 0u);
                mma_commit(BAR(B_SREADY + (j & 1)));
                mma_commit(BAR(B_KEMPTY + j % kK));
            }
            __syncwarp();
            return true;
        };
        bool ok = nt == 0 || __all_sync(FULL, mbar_wait(BAR(B_QFULL), 0, abort_flag, status, lim));
        for (int j = 0; ok && j < min(nt, 2); ++j) ok = scores(j);
        for (int j = 0; ok && j < nt; ++j) {
            ok = wait(B_PREADY, j) && wait(B_VFULL, j);
            if (!ok) break;
            fence_after_sync();
            const uint64_t vd = desc_add(vdesc, (j & 1) * KV_BYTES);
            const uint32_t p = tmem + TM_S + BN * (j & 1);
            const int steps = tile_keys(j) / 16;
            if (elect_one()) {
                for (int kk = 0; kk < steps; ++kk)
                    mma_ts(tmem + TM_O, p + 8 * kk, desc_add(vd, kk * 2 * kEight), idesc_pv, j > 0 || kk > 0 ? 1u : 0u);
                mma_commit(BAR(B_VEMPTY + (j & 1)));
            }
            __syncwarp();
            if (j + 2 < nt) ok = scores(j + 2);
        }
        if (elect_one()) mma_commit(BAR(B_DRAIN));
        __syncwarp();
        wait_drain(BAR(B_DRAIN), 0);
    } else {
        // ------------------------------------------------ softmax, a thread per row
        const int q4 = warp & 3;  // the warp's quarter of the TMEM lanes
        const int r = q4 * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
        const int t = t0 + r;
        const float sl2 = a.scale_log2;
        float m2 = -INFINITY, l = 0.f;
        bool ok = true;
        // the running maximum (log2 units) after scores up to mx, and O rescaled where it moved
        auto raise = [&](float mx, int j) {
            const float mn = mx * sl2;
            if (j == 0) {
                m2 = mn;
                return;
            }
            const bool need = mn > m2 + kRescaleThreshold;
            // the last product must have landed in O (if that wait gives up so does the next one)
            if (__any_sync(FULL, need) &&
                __all_sync(FULL, mbar_wait(BAR(B_VEMPTY + ((j - 1) & 1)), ((j - 1) >> 1) & 1, abort_flag, status, lim))) {
                fence_after_sync();
                const float up = need ? mn : m2;
                const float al = up == m2 ? 1.f : ex2(m2 - up);  // m2 may be -inf
                m2 = up;
                l *= al;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(trow + TM_O + 32 * c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
                    tmem_st32(trow + TM_O + 32 * c, o);
                }
            }
        };
        auto wait = [&](int bar, int j) -> bool {
            return __all_sync(FULL, mbar_wait(BAR(bar + (j & 1)), (j >> 1) & 1, abort_flag, status, lim));
        };
        for (int j = 0; j < nt; ++j) {
            const int s0 = tile_key(j);
            const uint32_t sb = trow + TM_S + BN * (j & 1);
            ok = wait(B_SREADY, j);
            if (!ok) break;
            fence_after_sync();
            // rows that end in this tile: nothing stored behind the end may reach the product
            const int end = len - s0;
            if (end < BN && (kPrefix || a.lens)) {
                ok = wait(B_VFULL, j);
                if (!ok) break;
                const int vr = r & (BN - 1), box = r / BN;  // 128 threads: 64 rows of two boxes
                if (vr >= end && box < D / 64) {
                    uint4* p = reinterpret_cast<uint4*>(gbase + OFF_V + (j & 1) * KV_BYTES + box * kCols + vr / 8 * kEight +
                                                        vr % 8 * 128);
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i] = make_uint4(0u, 0u, 0u, 0u);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
            if (j < ns) {
                // the sinks on their own: every row is past all of them
                const int keys = tile_keys(j);
                float mx = -INFINITY;
                for (int c0 = 0; c0 < keys; c0 += 16) {
                    uint32_t u[16];
                    tmem_ld<16>(sb + c0, u);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (s0 + c0 + c < a.sinks) mx = fmaxf(mx, __uint_as_float(u[c]));
                }
                raise(mx, j);
                for (int c0 = 0; c0 < keys; c0 += 16) {
                    uint32_t u[16], pk[8];
                    tmem_ld<16>(sb + c0, u);
                    tmem_wait_ld();
                    float p[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        p[c] = s0 + c0 + c < a.sinks ? ex2(fmaf(__uint_as_float(u[c]), sl2, -m2)) : 0.f;
                        l += p[c];
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c) pk[c] = pack_bf16(p[2 * c], p[2 * c + 1]);
                    // P of columns c0 .. lies over scores c0 / 2 .., which have been read
                    tmem_st<8>(sb + c0 / 2, pk);
                }
            } else {
                float s[BN];
                {
                    uint32_t u0[32], u1[32];
                    tmem_ld32(sb, u0);
                    tmem_ld32(sb + 32, u1);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; ++c) s[c] = __uint_as_float(u0[c]), s[32 + c] = __uint_as_float(u1[c]);
                }
                // keys of this tile that the row sees: the window's, or a sink
                if (kPrefix ? end < BN : s0 + BN - 1 > t0 || end < BN || s0 <= t0 + BM - 1 - a.window) {
#pragma unroll
                    for (int c0 = 0; c0 < BN; c0 += 32) {
                        uint32_t bits;
                        if constexpr (kPrefix) {
                            bits = bit_range(0, end - 1 - c0);
                        } else {
                            const int hi = min(t, len - 1) - s0 - c0;
                            bits = bit_range(t - a.window + 1 - s0 - c0, hi) | bit_range(0, min(a.sinks - s0 - c0 - 1, hi));
                        }
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!(bits >> c & 1u)) s[c0 + c] = -INFINITY;
                    }
                }
                float mx4[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mx4[k] = fmaxf(s[k], s[4 + k]);
#pragma unroll
                    for (int c = 8; c < BN; c += 8) mx4[k] = max3(mx4[k], s[c + k], s[c + 4 + k]);
                }
                raise(max3(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3])), j);
                const float neg = m2 == -INFINITY ? 0.f : -m2;  // a row that has seen nothing: 2^-inf = 0
                const f32x2 sl = mk2(sl2, sl2), nm = mk2(neg, neg);
                f32x2 acc[4] = {mk2(0.f, 0.f), mk2(0.f, 0.f), mk2(0.f, 0.f), mk2(0.f, 0.f)};
#pragma unroll
                for (int cc = 0; cc < BN / 32; ++cc) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int c = 32 * cc + 2 * i;
                        float x0, x1;
                        un2(fma2(mk2(s[c], s[c + 1]), sl, nm), x0, x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        acc[i & 3] = add2(acc[i & 3], mk2(p0, p1));
                        pk[i] = pack_bf16(p0, p1);
                    }
                    tmem_st<16>(sb + 16 * cc, pk);
                }
                float x0, x1, y0, y1;
                un2(add2(acc[0], acc[1]), x0, x1);
                un2(add2(acc[2], acc[3]), y0, y1);
                l += (x0 + x1) + (y0 + y1);
            }
            tmem_wait_st();
            fence_before_sync();
            mbar_arrive(BAR(B_PREADY + (j & 1)));
        }
        if (ok) ok = __all_sync(FULL, mbar_wait(BAR(B_DRAIN), 0, abort_flag, status, lim));
        ok = bar_and(ok && !*abort_flag, 1, 128);
        fence_after_sync();
        if constexpr (kPrefix) {
            // unnormalised outputs, then the maximum and the sum, in float32
            // (TMEM is read by whole warps, rows that do not exist among them)
            const bool row = r < a.nb * a.G && I * a.nb + r / a.G < a.B;
            if (ok) {
                float* slot = a.part + ((size_t)(h * a.ntq + I) * a.splits + split) * BM * (D + 2);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t u[32];
                    tmem_ld32(trow + TM_O + 32 * c, u);
                    tmem_wait_ld();
                    if (row)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            reinterpret_cast<uint4*>(slot + (size_t)r * D + 32 * c)[i] =
                                make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
                    __syncwarp();
                }
                if (row) *reinterpret_cast<float2*>(slot + BM * D + 2 * r) = make_float2(m2, l);
            }
        } else if constexpr (kShared) {
            // the share over the tiles, float32: [row][D], 16-byte pieces swizzled by row; then [row] (m, l)
#pragma unroll 1
            for (int c = 0; ok && c < D / 32; ++c) {
                uint32_t u[32];
                tmem_ld32(trow + TM_O + 32 * c, u);
                tmem_wait_ld();
                uint4* dst = reinterpret_cast<uint4*>(gbase) + r * (D / 4);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dst[(8 * c + e) ^ (r & 7)] = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
            }
            reinterpret_cast<float2*>(gbase + BM * D * 4)[r] = make_float2(m2, l);  // (no tile: -inf, 0)
        } else {
            const bool row = t < len;
            const float inv = row ? 1.f / l : 0.f;
            uint8_t* tile = gbase + OFF_Q;  // the queries are used up
            const uint32_t rowoff = (uint32_t)r * 128;
            if (ok) {
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t u[32];
                    if (nt > 0) tmem_ld32(trow + TM_O + 32 * c, u);
                    tmem_wait_ld();
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = row ? pack_bf16(__uint_as_float(u[8 * v + 2 * e]) * inv,
                                                   __uint_as_float(u[8 * v + 2 * e + 1]) * inv)
                                       : 0u;
                        const uint32_t chunk = (uint32_t)(((32 * c & 63) >> 3) + v) ^ (uint32_t)(r & 7);
                        *reinterpret_cast<uint4*>(tile + (c >> 1) * Q_BOX + rowoff + chunk * 16) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                if (t < a.T) a.lse[((size_t)b * a.H + h) * a.T + t] = row ? (m2 + log2f(l)) * kLn2 : -INFINITY;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            bar_sync(1, 128);
            if (warp == 2 && lane == 0 && ok) {
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    tma_store_4d(&tm_h, base + OFF_Q + x * Q_BOX, 64 * x, t0, h, b);
                bulk_commit_group();
                bulk_wait_group_read0();
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
    if constexpr (kShared) {  // the shares are joined in the order of the ranks, the rows spread over the CTAs
        static_assert(BM * D * 4 + BM * 8 <= OFF_BAR, "shares");
        __syncwarp();
        const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
        cluster.sync();
        const int rows = BM / cs, r0 = rank * rows;  // this CTA's
        float* weight = reinterpret_cast<float*>(gbase + OFF_V);  // [share][row], 1 / the sum among it
        if ((int)threadIdx.x < rows) {
            const int r = r0 + threadIdx.x, t = t0 + r;
            float2 ml[8];
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                ml[k] = make_float2(-INFINITY, 0.f);
                if (k < cs) ml[k] = reinterpret_cast<const float2*>(cluster.map_shared_rank(gbase, k) + BM * D * 4)[r];
                M = fmaxf(M, ml[k].x);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                ml[k].x = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - M);
                L = fmaf(ml[k].x, ml[k].y, L);
            }
            const float inv = t < len ? 1.f / L : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < cs) weight[k * BM + r] = t < len ? ml[k].x * inv : 0.f;
            if (t < a.T) a.lse[((size_t)b * a.H + h) * a.T + t] = t < len ? (M + log2f(L)) * kLn2 : -INFINITY;
        }
        __syncthreads();
        constexpr int kBatch = 4;  // reads in flight
        for (int e0 = threadIdx.x; e0 < rows * D / 4; e0 += kBatch * kThreads) {
            float4 o[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < cs; ++k) {
                const float4* share = reinterpret_cast<const float4*>(cluster.map_shared_rank(gbase, k));
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int e = e0 + i * kThreads, r = r0 + e / (D / 4), c = e % (D / 4);
                    if (e >= rows * D / 4) continue;
                    const float w = weight[k * BM + r];
                    const float4 v = share[r * (D / 4) + (c ^ (r & 7))];
                    if (w == 0.f) continue;  // (a share without a tile holds anything)
                    o[i].x = fmaf(w, v.x, o[i].x), o[i].y = fmaf(w, v.y, o[i].y);
                    o[i].z = fmaf(w, v.z, o[i].z), o[i].w = fmaf(w, v.w, o[i].w);
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int e = e0 + i * kThreads, t = t0 + r0 + e / (D / 4), c = e % (D / 4);
                if (e < rows * D / 4 && t < a.T)
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.h.data) + (size_t)b * a.h.sb +
                                              (size_t)h * a.h.sh + (size_t)t * a.h.st + 4 * c) =
                        make_uint2(pack_bf16(o[i].x, o[i].y), pack_bf16(o[i].z, o[i].w));
            }
        }
        cluster.sync();  // the shares stay until every CTA has read them
    }
}

template <int D, bool kPrefix, bool kShared>
int launch(const CUtensorMap (&m)[6], const AttnArgs& a, long long grid, cudaStream_t s) {
    const char* name = kPrefix ? "attn_tc_kernel<prefix>" : "attn_tc_kernel<window>";
    const int st = opt_in_max_smem<attn_tc_kernel<D, kPrefix, kShared>>(name);
    if (st != SSA_OK) return st;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)grid);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = SMEM_BYTES;
    c.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)a.cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = kShared ? 1 : 0;
    const cudaError_t e =
        cudaLaunchKernelEx(&c, attn_tc_kernel<D, kPrefix, kShared>, m[0], m[1], m[2], m[3], m[4], m[5], a);
    if (e != cudaSuccess) return fail(SSA_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
    return check_launch(name);
}

// Few query tiles: clusters share their key tiles, as far as every CTA has an SM, or
// half of one where all keys are seen and the late tiles are the longest, and four
// tiles; lists of 16 tiles at least (one head of 128: 8192 tokens, all keys 98 -> 38
// us; 4000 tokens, window 1024 19 -> 15; 512 tokens of 8 heads 11 us, 13 shared).
int cluster_of(const AttnArgs& a) {
    const long long ctas = (long long)a.B * a.H * a.ntq, all = (a.T + BN - 1) / BN;
    const long long reach = ((long long)a.window + BM - 2) / BN + 1 + (a.sinks + BN - 1) / BN;
    const long long list = reach < all ? reach : all;
    const long long most = 2 * (long long)a.window > a.T ? kSharedCtas : kSharedCtas / 2;
    int cs = 1;
    while (cs < 8 && 2 * cs * ctas <= most && 2 * kSharedTiles * cs <= list) cs *= 2;
    return list < 4 * kSharedTiles ? 1 : cs;
}

}  // namespace

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
    a.h = h, a.cluster = cluster_of(a);
    if (a.cluster > 1)
        return p.D == 64 ? launch<64, false, true>(m, a, grid * a.cluster, s) : launch<128, false, true>(m, a, grid * a.cluster, s);
    return p.D == 64 ? launch<64, false, false>(m, a, grid, s) : launch<128, false, false>(m, a, grid, s);
}

// One row tile reads the prefix once; up to 16 rows a head the kernel for single
// tokens does the same with less work per key.
bool prefix_tc_supported(const ssa_cache_params_t& p) {
    const int G = p.Hq / p.Hkv;
    return p.dtype == SSA_BF16 && G <= BM && (long long)p.B * G > 16;
}

PrefixPlan prefix_tc_plan(const ssa_cache_params_t& p, int prefix_len) {
    PrefixPlan x{};
    const int G = p.Hq / p.Hkv, tiles = (prefix_len + BN - 1) / BN;
    x.nb = BM / G;
    x.ntq = (p.B + x.nb - 1) / x.nb;
    const long long rows = (long long)p.Hkv * x.ntq;
    long long n = kPrefixCtas / rows;  // one round of CTAs
    if (n > tiles / kPrefixTiles) n = tiles / kPrefixTiles;
    x.splits = n < 1 ? 1 : (int)n;
    x.bytes = (size_t)rows * x.splits * BM * (p.D + 2) * sizeof(float);
    return x;
}

int launch_prefix_tc(const ssa_cache_params_t& p, const View& q, const void* k_pages, const void* v_pages,
                     const int32_t* prefix_pages, int prefix_len, void* ws, cudaStream_t s) {
    const PrefixPlan x = prefix_tc_plan(p, prefix_len);
    const int G = p.Hq / p.Hkv;
    using U = unsigned long long;
    CUtensorMap m[6];
    const U qdims[4] = {(U)p.D, (U)G, (U)p.Hkv, (U)p.B};
    const long long qstrides[3] = {q.sh, q.sh * G, q.sb};
    const unsigned qbox[4] = {64, (unsigned)G, 1, (unsigned)x.nb};
    int st = make_map(&m[0], q.data, 4, qdims, qstrides, qbox);
    const U dims[5] = {64, 8, (U)p.D / 64, (U)p.Hkv * p.page / 8, (U)p.n_pages};
    const long long strides[4] = {p.D, 64, 8ll * p.D, p.page_stride};
    const unsigned box[5] = {64, 8, (unsigned)p.D / 64, (unsigned)(p.page < BN ? p.page : BN) / 8, 1};
    if (st == SSA_OK) st = make_map(&m[1], const_cast<void*>(k_pages), 5, dims, strides, box);
    if (st == SSA_OK) st = make_map(&m[2], const_cast<void*>(v_pages), 5, dims, strides, box);
    if (st != SSA_OK) return st;
    m[3] = m[1], m[4] = m[2], m[5] = m[0];  // not used by this pass
    AttnArgs a{};
    a.pages = prefix_pages, a.part = static_cast<float*>(ws);
    a.H = p.Hkv, a.B = p.B, a.G = G, a.T = prefix_len;
    a.ntq = x.ntq, a.splits = x.splits, a.page = p.page, a.n_pages = p.n_pages, a.nb = x.nb;
    a.scale_log2 = p.sm_scale * 1.4426950408889634f;
    a.timeout_ns = wait_limit_ns();
    const long long grid = (long long)p.Hkv * x.ntq * x.splits;
    if (grid > 0x7fffffffll) return fail(SSA_ERR_UNSUPPORTED, "prefix_decode: too many row tiles");
    return p.D == 64 ? launch<64, true, false>(m, a, grid, s) : launch<128, true, false>(m, a, grid, s);
}

int attn_tc_take_status() {
    unsigned int v = 0, w = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_tc_status, sizeof v);
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&w, g_attn_tc_range, sizeof w);
    if (e != cudaSuccess) return fail(SSA_ERR_CUDA, "status read: %s", cudaGetErrorString(e));
    const unsigned int zero = 0;
    if (v) cudaMemcpyToSymbol(g_attn_tc_status, &zero, sizeof zero);
    if (w) cudaMemcpyToSymbol(g_attn_tc_range, &zero, sizeof zero);
    if (v & 1u) return fail(SSA_ERR_TIMEOUT, "attn_tc_kernel: a bounded mbarrier wait expired");
    if (w) return fail(SSA_ERR_INVALID_ARG, "attention: a %s was out of range", w & 2u ? "page number" : "length");
    if (v) return fail(SSA_ERR_CUDA, "attn_tc_kernel: shared memory is not aligned");
    return SSA_OK;
}

}  // namespace ssa
