// y = W q(x) on the block-scaled tensor cores, and the gated block
// h = act(Wg q(x) + g_add) (Wu q(x) + u_add), for many tokens.
//
// Mathematics: both operands are microscaled (dbf_mx.cuh), so a product of
// two blocks of 32 is 2^(sa + sb) times a sum of 32 products of E2M1 codes:
// tcgen05.mma kind::mxf4 computes it with fp32 accumulators from packed codes
// and scale bytes as they lie in memory. A pre-pass quantises x (one pass
// over x); one persistent launch does the rest.
//
// Tile: a CTA pair (cta_group::2) owns 512 weight rows x w tokens as two
// accumulators of 256 x w: two row blocks of W, or 256 rows of Wg and the same
// rows of Wu, so the gated block finds g and u of one element in one place. At
// four times the bf16 rate the operands' way into the SM bounds the tile, not
// the MMA: 512 x 224 takes 50 KB per 896 cycles of MMA and SM; a double-buffered
// 256 x 224 would take 32 KB per 448.
//   warp 0      TMA: per stage of 256 columns, 2 x 128 rows of codes (128-byte
//               swizzle), w/2 token rows, and their scale tiles;
//   warp 1      tensor memory; in CTA 0 one elected thread issues eight MMAs a stage;
//   warps 2..5  bring the stage's scales into tensor memory, each into its own
//               32 lanes, through registers. tcgen05.cp would do it too, but
//               runs in the MMAs' own queue: at about 70 cycles a copy, eight
//               of them a stage took a fifth of the time of an 8192^3 product
//               (316 us, and 249 us without them);
//   warps 6..13 epilogue.
// The token width w is chosen per call (a multiple of 16 up to 224, what 512
// tensor-memory columns hold beside two buffers of 32 of scales) so that the
// tiles fill whole waves of pairs; narrower tiles, whose stages take less time
// than scales need to get there, have up to four buffers. 8192^3 takes 219 us
// in short graphs: 31 of the pre-pass, 156 of the products and 26 of epilogues
// (255 us call after call, at the clocks of the power cap). Every wait is bounded;
// on expiry the status word is set.
#include <algorithm>
#include <atomic>

#include "dbf_mx_layer.cuh"
#include "dbf_tc.cuh"

namespace dbf {
namespace {

using namespace mx;
using namespace tc;

constexpr int kMaxStages = 10, kMaxSfBufs = 4;
constexpr int kMaxW = 224;
constexpr int kScaleWarps = 4, kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kScaleWarps + kEpiWarps);
constexpr uint32_t kABytes = 128 * 128;            // 128 rows x 256 codes
constexpr uint32_t kSfBytes = 1024;                // scales of 128 rows x 256 codes
constexpr int kMaxSmem = 227 * 1024;
// A stage: the codes of 'accs' blocks of 128 weight rows and of this CTA's half
// of the tokens, then the scales of both (of all the tokens). From the last MMA
// on a stage to the next one's data it takes about 2.2 us, so a ring of n
// stages gives one every 2.2 / n us at best: as many as fit.
__host__ __device__ constexpr uint32_t b_at(int accs) { return accs * kABytes; }
__host__ __device__ constexpr uint32_t sf_at(int accs, int w) { return accs * kABytes + w / 2 * 128; }
__host__ __device__ constexpr uint32_t stage_bytes(int accs, int w) { return sf_at(accs, w) + (accs + (w > 128 ? 2 : 1)) * kSfBytes; }
// tensor-memory columns: accs w per set of accumulators, then buffers of
// scales: 8 per weight block (4 per K half), 16 kept for them, then 4 per K half
// and 128 tokens
__host__ __device__ constexpr uint32_t sf_cols(int w) { return w > 128 ? 32u : 24u; }
constexpr uint32_t kTmemCols = 512;

struct Smem {
    uint64_t full[kMaxStages], sf_full[kMaxStages], empty[kMaxStages], sf_ready[kMaxSfBufs], acc_full[2], acc_empty[2], drain, exit_bar;
    uint32_t tmem_base;
    int abort;
};

struct Args {
    int nk;         // stages of 256 columns
    int w;          // tokens per tile
    int accs;       // accumulators of a set: 2, or 1 (plain, where tiles are few)
    int ring;       // stages in shared memory
    int sf_bufs;    // scale buffers, 2 to kMaxSfBufs
    int bufs;       // 2: two sets of accumulators, so that an epilogue overlaps the next tile's products
    int n_p;        // row tiles
    int tiles;
    int row_step;   // weight rows of a tile: 256 accs plain, 256 gated
    int row_off;    // rows from the first accumulator's to the second's: 256 plain, 0 gated
    Epilogue ep;
    int32_t *status;
};

__device__ __forceinline__ void load_chunk(uint32_t at, int, float (&col)[1][8]) { tmem_ld8(at, col); }
__device__ __forceinline__ void load_chunk(uint32_t at, int w, float (&col)[2][8]) { tmem_ld8(at, at + w, col); }
__device__ __forceinline__ void load_chunk(uint32_t at, int, float (&col)[1][16]) { tmem_ld16(at, col); }
__device__ __forceinline__ void load_chunk(uint32_t at, int w, float (&col)[2][16]) { tmem_ld16(at, at + w, col); }

// Which set of accumulators a tile uses, and the phase of its barriers.
struct Turn {
    uint32_t buf = 0, phase = 0;
    __device__ __forceinline__ void next(int bufs)
    {
        if (++buf == static_cast<uint32_t>(bufs)) buf = 0, phase ^= 1u;
    }
};

// A tile's addends into L2 while its products are computed: w tokens x 128
// columns (two lines of 128 bytes a row) of both, over the epilogue's warps.
__device__ __forceinline__ void prefetch_addends(const Epilogue &e, int64_t t0, int w, int n0, int warp)
{
    for (int i = warp * 32 + (threadIdx.x & 31); i < 4 * w; i += kEpiWarps * 32) {
        const int64_t t = t0 + (i >> 2);
        const int c = n0 + (i & 1) * 64;
        if (t < e.T && c < e.N) {
            const uint16_t *p = static_cast<const uint16_t *>(i & 2 ? e.u_add : e.g_add) + t * e.N + c;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
        }
    }
}

// A warp's share of a gated tile: 16 tokens of both accumulators at a time,
// every second 16 from j0. The next 16 tokens' addends are asked for as soon as
// these have left their registers, the first before the products are there.
// False when the wait for them gave up.
template <bool kAdd, bool kSave, int kAct, class Ready>
__device__ __forceinline__ bool gated_tile(const Args &g, float *own, uint32_t lanes, int64_t t, int n, int j0, Ready ready)
{
    uint4 x[2][2];
    gated_reads<kAdd>(g.ep, t + j0, n, j0 < g.w, x);
    if (!ready()) return false;
#pragma unroll 1
    for (int j = j0; j < g.w; j += 32) {
        float v[2][16], r[2][16];
        load_chunk(lanes + j, g.w, v);
        gated_turn<kAdd>(own, v, x, r);
        gated_reads<kAdd>(g.ep, t + j + 32, n, j + 32 < g.w, x);
        gated_finish<kSave, kAct>(g.ep, t + j, n, r);
    }
    return true;
}
template <int kAct, class Ready>
__device__ __forceinline__ bool gated_tile(const Args &g, float *own, uint32_t lanes, int64_t t, int n, int j0, Ready ready)
{
    const bool add = g.ep.g_add != nullptr, save = g.ep.g8 != nullptr;
    return add ? (save ? gated_tile<true, true, kAct>(g, own, lanes, t, n, j0, ready)
                       : gated_tile<true, false, kAct>(g, own, lanes, t, n, j0, ready))
               : gated_tile<false, true, kAct>(g, own, lanes, t, n, j0, ready);
}
// The same where the finish is simple, or rows are no whole vectors.
template <int kMats, int kAct>
__device__ __forceinline__ void column_tile(const Args &g, float *own, uint32_t lanes, int64_t t, int n, int j0, int step, bool simple)
{
    if (simple) {
        for (int j = j0; j < g.w; j += step) {
            float v[kMats][16];
            load_chunk(lanes + j, g.w, v);
            simple_finish<kMats, kAct>(g.ep, reinterpret_cast<uint32_t *>(own), t + j, n, v, threadIdx.x & 31);
        }
        return;
    }
    for (int j = j0; j < g.w; j += step) {
        float v[kMats][16];
        load_chunk(lanes + j, g.w, v);
        column_finish<kMats, kAct>(g.ep, own, t + j, n, v);
    }
}

template <bool kGated>
__global__ void __launch_bounds__(kThreads, 1) mx_gemm_kernel(
    const __grid_constant__ CUtensorMap mA0, const __grid_constant__ CUtensorMap mA1, const __grid_constant__ CUtensorMap mS0,
    const __grid_constant__ CUtensorMap mS1, const __grid_constant__ CUtensorMap mB, const __grid_constant__ CUtensorMap mSB,
    const __grid_constant__ Args g)
{
    constexpr int kMats = kGated ? 2 : 1;
    extern __shared__ uint8_t raw[];
    uint8_t *stage0 = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const int accs = kGated ? 2 : g.accs, stages = g.ring;
    const uint32_t stage_size = stage_bytes(accs, g.w), off_b = b_at(accs), off_sf = sf_at(accs, g.w);
    float *turn = reinterpret_cast<float *>(stage0 + stages * stage_size);
    Smem *sh = reinterpret_cast<Smem *>(turn + kEpiWarps * kMats * kTurnFloats);
    const int warp = warp_number(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int unit = blockIdx.x >> 1, units = gridDim.x >> 1;
    volatile int *abort = &sh->abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            bar_init(&sh->full[i], 1);
            bar_init(&sh->sf_full[i], 1);
            bar_init(&sh->empty[i], 1);
        }
        for (int i = 0; i < kMaxSfBufs; ++i) bar_init(&sh->sf_ready[i], 2 * kScaleWarps);
        for (int i = 0; i < 2; ++i) {
            bar_init(&sh->acc_full[i], 1);
            bar_init(&sh->acc_empty[i], 2 * kEpiWarps);
        }
        bar_init(&sh->drain, 1);
        bar_init(&sh->exit_bar, 1);
        sh->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<2>(&sh->tmem_base, kTmemCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers exist before either is reached from the other
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh->tmem_base, 0);
    // the pre-pass before this launch has waited for all earlier work, so
    // weights may be read at once; x's codes, and y, only after it is done
    griddep_launch();

    if (warp == 0) {
        const int half_w = g.w / 2, nrt = g.w > 128 ? 2 : 1;
        const uint32_t bytes = 2 * off_sf, sf_bytes = stage_size - off_sf;
        int s = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true, waited = false;
        for (int tile = unit; tile < g.tiles && ok; tile += units) {
            const int p = tile % g.n_p, c = tile / g.n_p;
            const int row0 = p * g.row_step + static_cast<int>(rank) * 128, row1 = row0 + g.row_off;
            const int tok = c * g.w + static_cast<int>(rank) * half_w;
            for (int ks = 0; ks < g.nk; ++ks) {
                ok = warp_wait(&sh->empty[s], ph ^ 1u, abort);
                if (!ok) break;
                uint8_t *st = stage0 + s * stage_size, *sf = st + off_sf;
                const bool one = elect_one();
                if (one) {
                    if (rank == 0) bar_expect_tx(&sh->full[s], bytes);
                    bar_expect_tx(&sh->sf_full[s], sf_bytes);   // the scales are counted by each CTA for itself
                    tma_2d_pair(st, &mA0, ks * 128, row0, &sh->full[s]);
                    tma_3d(sf, &mS0, 0, ks * 2, row0 >> 7, &sh->sf_full[s]);
                    if (accs == 2) {
                        tma_2d_pair(st + kABytes, &mA1, ks * 128, row1, &sh->full[s]);
                        tma_3d(sf + kSfBytes, &mS1, 0, ks * 2, row1 >> 7, &sh->sf_full[s]);
                    }
                }
                __syncwarp();
                if (!waited) {
                    griddep_wait();
                    waited = true;
                }
                if (one) {
                    tma_2d_pair(st + off_b, &mB, ks * 128, tok, &sh->full[s]);
                    tma_3d(sf + accs * kSfBytes, &mSB, 0, ks * 2, c * nrt, &sh->sf_full[s]);
                }
                __syncwarp();
                ++issued;
                if (++s == stages) s = 0, ph ^= 1u;
            }
        }
        // after a wait gave up, the loads in flight are still waited for
        // (CTA 0's barriers count both CTAs' bytes)
        if (*abort)
            for (int i = issued > stages ? issued - stages : 0; i < issued; ++i) {
                drain_wait(&sh->sf_full[i % stages], static_cast<uint32_t>(i / stages) & 1u);
                if (rank == 0) drain_wait(&sh->full[i % stages], static_cast<uint32_t>(i / stages) & 1u);
            }
    } else if (warp == 1) {
        if (rank == 0) {
            int s = 0;
            uint32_t ph = 0;
            Turn acc, sf_turn;
            const uint32_t sf0 = tmem + accs * g.w * g.bufs, b_half = g.w > 128 ? 8 : 4;
            bool ok = true;
            const uint32_t id0 = mxf4_idesc(256, g.w, 0), id2 = mxf4_idesc(256, g.w, 2);
            for (int tile = unit; tile < g.tiles && ok; tile += units, acc.next(g.bufs)) {
                ok = warp_wait(&sh->acc_empty[acc.buf], acc.phase ^ 1u, abort);
                if (!ok) break;
                const uint32_t d = tmem + acc.buf * accs * g.w;
                for (int ks = 0; ks < g.nk; ++ks, sf_turn.next(g.sf_bufs)) {
                    ok = warp_wait(&sh->full[s], ph, abort) && warp_wait(&sh->sf_ready[sf_turn.buf], sf_turn.phase, abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t st = smem_u32(stage0) + s * stage_size, sf = sf0 + sf_turn.buf * sf_cols(g.w);
                    const uint64_t a0 = sw128_desc(st), a1 = sw128_desc(st + kABytes), b = sw128_desc(st + off_b);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint32_t id = kk & 1 ? id2 : id0, more = ks > 0 || kk > 0 ? 1u : 0u;
                            const uint32_t sb = sf + 16 + b_half * (kk >> 1);
                            mma_mxf4<2>(d, a0 + 2 * kk, b + 2 * kk, id, sf + 4 * (kk >> 1), sb, more);
                            if (accs == 2) mma_mxf4<2>(d + g.w, a1 + 2 * kk, b + 2 * kk, id, sf + 8 + 4 * (kk >> 1), sb, more);
                        }
                        commit_pair_both(&sh->empty[s]);
                    }
                    __syncwarp();
                    if (++s == stages) s = 0, ph ^= 1u;
                }
                if (!ok) break;
                if (elect_one()) commit_pair_both(&sh->acc_full[acc.buf]);
                __syncwarp();
            }
            if (*abort) {
                if (elect_one()) commit_pair_own(&sh->drain);
                __syncwarp();
                drain_wait(&sh->drain, 0);
            }
        }
    } else if (warp < 2 + kScaleWarps) {
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const int64_t total = static_cast<int64_t>((g.tiles - 1 - unit) / units + 1) * g.nk;   // stages of this pair
        int s = 0;
        uint32_t ph = 0;
        Turn buf;
        for (int64_t k = 0; k < total; ++k, buf.next(g.sf_bufs)) {
            // the buffer is free once the MMAs of stage k - sf_bufs are done
            const int64_t before = k - g.sf_bufs;
            if (before >= 0 && !bar_wait(&sh->empty[before % stages], static_cast<uint32_t>(before / stages) & 1u, abort)) break;
            if (!bar_wait(&sh->sf_full[s], ph, abort)) break;
            tc_fence_after();
            const uint4 *sf = reinterpret_cast<const uint4 *>(stage0 + s * stage_size + off_sf) + lane;
            // 512 bytes hold 128 rows x 4 blocks, a lane's 16 the rows lane, lane + 32, ...
            const uint32_t to = lanes + accs * g.w * g.bufs + buf.buf * sf_cols(g.w);
            const uint4 *sb = sf + accs * 64;
            if (accs == 2)
                tmem_st16(to, sf[0], sf[32], sf[64], sf[96]);
            else
                tmem_st8(to, sf[0], sf[32]);
            if (g.w > 128)
                tmem_st16(to + 16, sb[0], sb[64], sb[32], sb[96]);
            else
                tmem_st8(to + 16, sb[0], sb[32]);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_leader(&sh->sf_ready[buf.buf]);
            if (++s == stages) s = 0, ph ^= 1u;
        }
    } else {
        griddep_wait();   // y (and the addends) belong to earlier work until then
        const int quarter = warp & 3, half = (warp - 2 - kScaleWarps) >> 2;
        const bool two = !kGated && accs == 2;
        const uint32_t lanes0 = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + (two ? half * g.w : 0);
        float *own = turn + (warp - 2 - kScaleWarps) * kMats * kTurnFloats;
        // two plain accumulators: each of a lane quarter's two warps takes one;
        // else they take turns by 8 (16) tokens
        const int j_first = two ? 0 : half * 8, j_step = two ? 8 : 16;
        const bool simple = epilogue_is_simple(g.ep), bf16 = epilogue_is_bf16(g.ep), silu = g.ep.act == DBF_GATE_SILU;
        Turn acc;
        for (int tile = unit; tile < g.tiles; tile += units, acc.next(g.bufs)) {
            const uint32_t lanes = lanes0 + acc.buf * accs * g.w;
            uint64_t *full = &sh->acc_full[acc.buf], *empty = &sh->acc_empty[acc.buf];
            const int p = tile % g.n_p, c = tile / g.n_p;
            const int n = p * g.row_step + (two ? half * g.row_off : 0) + static_cast<int>(rank) * 128 + quarter * 32 +
                          (lane & 3) * 8;
            const int64_t t = static_cast<int64_t>(c) * g.w + (lane >> 2);
            if (simple || !epilogue_vec(g.ep)) {
                if (g.ep.g_add && g.ep.u_add && g.ep.add_dt == DBF_BF16)
                    prefetch_addends(g.ep, t - (lane >> 2), g.w, n - (lane & 3) * 8 - quarter * 32, warp - 2 - kScaleWarps);
                if (!bar_wait(full, acc.phase, abort)) break;
                tc_fence_after();
                const int64_t t0 = t - (lane >> 2);
                const int n0 = n - (lane & 3) * 8;
                if (!kGated || silu)
                    column_tile<kMats, DBF_GATE_SILU>(g, own, lanes, t0, n0, 2 * j_first, 2 * j_step, simple);
                else
                    column_tile<kMats, DBF_GATE_GELU>(g, own, lanes, t0, n0, 2 * j_first, 2 * j_step, simple);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive_leader(empty);
                continue;
            }
            if constexpr (kGated) {
                if (bf16) {
                    if (g.ep.g_add) prefetch_addends(g.ep, t - (lane >> 2), g.w, n - (lane & 3) * 8 - quarter * 32, warp - 2 - kScaleWarps);
                    auto ready = [&] {
                        const bool ok = bar_wait(full, acc.phase, abort);
                        tc_fence_after();
                        return ok;
                    };
                    const int64_t t16 = t - (lane >> 2) + (lane >> 1);
                    const int n16 = n - (lane & 3) * 8 + (lane & 1) * 8;
                    const bool ok = silu ? gated_tile<DBF_GATE_SILU>(g, own, lanes, t16, n16, half * 16, ready)
                                         : gated_tile<DBF_GATE_GELU>(g, own, lanes, t16, n16, half * 16, ready);
                    if (!ok) break;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive_leader(empty);
                    continue;
                }
            }
            // what a chunk reads is asked for a chunk ahead, the first before the products are there
            Raw8 x[2][kMats];
            epilogue_reads<kGated>(g.ep, t + j_first, n, t + j_first < g.ep.T, x[0]);
            if (!bar_wait(full, acc.phase, abort)) break;
            tc_fence_after();
            for (int j0 = j_first; j0 < g.w; j0 += 2 * j_step) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int j = j0 + i * j_step, next = j + j_step;
                    if (j >= g.w) break;
                    epilogue_reads<kGated>(g.ep, t + next, n, next < g.w && t + next < g.ep.T, x[i ^ 1]);
                    float col[kMats][8], row[kMats][8];
                    load_chunk(lanes + j, g.w, col);
                    turn8<kMats>(own, col, row, lane);
                    epilogue_finish<kGated>(g.ep, t + j, n, t + j < g.ep.T, x[i], row);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_leader(empty);
        }
    }

    tc_fence_before();
    __syncthreads();
    // neither CTA ends while the other may still reach its shared memory
    if (threadIdx.x == 0) {
        bar_arrive_rank(&sh->exit_bar, rank ^ 1u);
        drain_wait(&sh->exit_bar, 0);
        if (sh->abort && g.status) atomicExch(g.status, static_cast<int32_t>(DBF_ERR_TIMEOUT));
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free<2>(tmem, kTmemCols);
    }
}

// Pre-pass: x to codes and scales in the workspace. The scales of the tokens
// of one tile start a new 128-row scale tile, since a tile of w tokens is no
// multiple of 128 (x_scale_row).
template <dbf_dtype DT, bool kVec>
__global__ void __launch_bounds__(256) quantize_x_kernel(const void *__restrict__ x, int64_t T, int64_t M, int w, int pad,
                                                         uint8_t *__restrict__ codes, uint8_t *__restrict__ scales)
{
    griddep_wait();   // the workspace may still be read by the call before
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kCols = lane_cols<DT>();
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * kCols;
    const int64_t nb = blocks(M), pitch = nb * 16, tiles = scale_tiles(M);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 32 + warp;
    const int left = static_cast<int>(T - row < 32 ? T - row : 32);   // row + 8 i exists where 8 i < left
    Raw8 in[4][kCols / 8];
#pragma unroll
    for (int i = 0; i < 4; ++i) load_cols<DT, kVec, kCols>(x, (row + 8 * i) * M, 8 * i < left ? c : M, M, T * M, in[i]);
    uint8_t *out = codes + row * pitch + c / 2;
#pragma unroll
    for (int i = 0; i < 4; ++i, out += 8 * pitch) {
        const int r = static_cast<int>(row) + 8 * i;
        uint32_t byte, q[kCols / 8];
        quantize_e2m1<DT, kCols>(in[i], byte, q);
        const uint32_t word = tile_scales<kCols>(byte, lane);
        if (8 * i >= left) continue;
        if (c < nb * kBlock) store_words(out, q);
        if (lane % (128 / kCols) == 0 && (c >> 7) < tiles)
            *reinterpret_cast<uint32_t *>(scales + scale_at(x_scale_row(r, w, pad), c >> 5, tiles)) = word;
    }
    // Only now: the product's CTAs would take the registers of this kernel's
    // (one of its CTAs beside a product's on an SM against four alone). They
    // then start with all earlier work done.
    griddep_launch();
}

// CTA pairs that can be resident at once (the query is slow next to a launch:
// kept per device).
template <bool kGated>
int resident_pairs(cudaLaunchConfig_t cfg)
{
    static std::atomic<int> known[kMaxDevices];
    int dev = 0;
    const bool keep = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices;
    int pairs = keep ? known[dev].load(std::memory_order_relaxed) : 0;
    if (pairs == 0) {
        pairs = std::max(1, device_sms() / 2);
        cfg.gridDim = dim3(2 * pairs);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, mx_gemm_kernel<kGated>, &cfg) == cudaSuccess && n > 0) pairs = std::min(n, pairs);
        (void)cudaGetLastError();
        if (keep) known[dev].store(pairs, std::memory_order_relaxed);
    }
    return pairs;
}

// What an epilogue costs per token of a tile, in cycles: plain bf16 rows, the
// gate, addends, 8-bit copies (from 6 waves of 4096 -> 11008 at 2048 tokens).
enum Kind { kPlain, kGate, kGateAdd, kGateSave, kKinds };
constexpr double kEpilogueCycles[kKinds] = {25, 29, 75, 78};   // plain: of two accumulators

Kind kind_of(const Product &c)
{
    if (c.mats == 1) return kPlain;
    return c.ep.g8 ? kGateSave : c.ep.g_add || c.ep.u_add ? kGateAdd : kGate;
}

struct Plan {
    int w, bufs, accs, ring, pad;   // pad: scale rows of a tile
};
int fixed_smem(int mats) { return 1024 + kEpiWarps * mats * kTurnFloats * 4 + static_cast<int>(sizeof(Smem)); }

// Tokens per tile, one or two sets of accumulators, and for a plain product one
// or two accumulators in a set. Cost of the last pair to finish, in cycles:
// waves of tiles, each nk stages and an epilogue, which two sets hide behind the
// next tile's stages. A stage takes its MMAs (2 w cycles an accumulator), its
// operands' way from L2 (about 45 bytes a cycle and SM, 38 beside a running
// epilogue) or its share of the ring's round trip, whichever is longest. Wide
// tiles pay least for their weights' way there: two sets win only where the
// epilogue is long against K (2048 x 8192 at 4096 tokens with addends: 112 us on
// one set, 102 us on two; 4096 x 11008 at 2048 tokens: 109 us and 121 us), one
// accumulator only where tiles are fewer than pairs.
Plan plan(int64_t M, int64_t N, int64_t T, int mats, Kind kind, int sms)
{
    const int64_t nk = (M + 255) / 256, pairs = std::max(1, sms / 2);
    Plan p = {};
    double least = -1;
    for (int accs = mats; accs <= 2; ++accs)
        for (int bufs = 1; bufs <= 2; ++bufs)
            for (int w = 16; w <= kMaxW; w += 16) {
                if (accs * w * bufs > 2 * kMaxW) break;
                const int64_t rows = mats == 2 ? 256 : 256 * accs;
                const int64_t waves = ((N + rows - 1) / rows * ((T + w - 1) / w) + pairs - 1) / pairs;
                const double bytes = stage_bytes(accs, w);
                const int ring = std::min<int>(kMaxStages, (kMaxSmem - fixed_smem(mats)) / stage_bytes(accs, w));
                const double stage = std::max({2.0 * accs * w, bytes / (bufs == 1 ? 45 : 38), 4000.0 / ring});
                const double products = nk * stage, epilogue = 800 + kEpilogueCycles[kind] * w * accs / 2;
                const double cost = bufs == 1 ? waves * (products + epilogue)
                                              : (waves - 1) * std::max(products, epilogue) + products + epilogue;
                if (least < 0 || cost < least) least = cost, p.w = w, p.bufs = bufs, p.accs = accs, p.ring = ring;
                if (w >= T) break;
            }
    p.pad = p.w > 128 ? 256 : 128;
    return p;
}

bool code_map(CUtensorMap *m, const uint8_t *codes, int64_t k, int64_t rows, int box_rows)
{
    const uint64_t dims[2] = {static_cast<uint64_t>(code_pitch(k)), static_cast<uint64_t>(rows)};
    const uint64_t strides[1] = {static_cast<uint64_t>(code_pitch(k))};
    const uint32_t box[2] = {128, static_cast<uint32_t>(box_rows)};
    return tc_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, box, true);
}

bool scale_map(CUtensorMap *m, const uint8_t *scales, int64_t k, int64_t row_tiles, int box_tiles)
{
    const uint64_t tiles = static_cast<uint64_t>(scale_tiles(k));
    const uint64_t dims[3] = {128, tiles, static_cast<uint64_t>(row_tiles)};
    const uint64_t strides[2] = {512, tiles * 512};
    const uint32_t box[3] = {128, 2, static_cast<uint32_t>(box_tiles)};
    return tc_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, scales, dims, strides, box, false);
}

}  // namespace

bool tc_map(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const uint64_t *dims,
            const uint64_t *strides, const uint32_t *box, bool swizzle128)
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    if (!fn) return false;
    cuuint64_t d[3] = {}, s[2] = {};
    cuuint32_t b[3] = {}, one[3] = {1, 1, 1};
    for (int i = 0; i < rank; ++i) d[i] = dims[i], b[i] = box[i];
    for (int i = 0; i + 1 < rank; ++i) s[i] = strides[i];
    return fn(map, type, static_cast<cuuint32_t>(rank), const_cast<void *>(base), d, s, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

void mx_gemm_cut(const Product &c, int sms, int64_t (&cut)[8])
{
    const Plan pl = plan(c.M, c.N, c.T, c.mats, kind_of(c), sms);
    const int64_t rows = c.mats == 2 ? 256 : 256 * pl.accs;
    const int64_t of[8] = {DBF_MX4_MANY_TOKENS, pl.w, pl.accs, pl.bufs, pl.ring, (c.M + 255) / 256,
                           (c.N + rows - 1) / rows * ((c.T + pl.w - 1) / pl.w), x_scale_row(static_cast<int>(c.T - 1), pl.w, pl.pad)};
    std::copy(of, of + 8, cut);
}

cudaError_t mx_quantize_x(const Product &c, int w, int pad, uint8_t *codes, uint8_t *scales, cudaStream_t s)
{
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const bool vec = c.M % 8 == 0;   // x is 16-byte aligned
    const int cols = 32 * (c.xd == DBF_BF16 ? lane_cols<DBF_BF16>() : lane_cols<DBF_F32>());
    cfg.gridDim = dim3(static_cast<unsigned>((c.T + 31) / 32), static_cast<unsigned>((c.M + cols - 1) / cols));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const auto kernel = c.xd == DBF_F32 ? (vec ? quantize_x_kernel<DBF_F32, true> : quantize_x_kernel<DBF_F32, false>)
                                        : (vec ? quantize_x_kernel<DBF_BF16, true> : quantize_x_kernel<DBF_BF16, false>);
    return cudaLaunchKernelEx(&cfg, kernel, c.x, c.T, c.M, w, pad, codes, scales);
}

cudaError_t mx_gemm(const Product &c, cudaStream_t s)
{
    const Plan pl = plan(c.M, c.N, c.T, c.mats, kind_of(c), device_sms());
    uint8_t *codes = static_cast<uint8_t *>(c.ws) + x_codes_at(), *scales = static_cast<uint8_t *>(c.ws) + x_scales_at(c.M, c.T);

    CUtensorMap a[2], sa[2], b, sb;
    const bool gated = c.mats == 2;
    for (int m = 0; m < c.mats; ++m)
        if (!code_map(&a[m], c.codes[m], c.M, c.N, 128) || !scale_map(&sa[m], c.scales[m], c.M, (c.N + 127) / 128, 1))
            return cudaErrorInvalidValue;
    if (!gated) a[1] = a[0], sa[1] = sa[0];
    if (!code_map(&b, codes, c.M, c.T, pl.w / 2) ||
        !scale_map(&sb, scales, c.M, (c.T + pl.w - 1) / pl.w * (pl.pad / 128), pl.pad / 128))
        return cudaErrorInvalidValue;

    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;

    cudaError_t e = mx_quantize_x(c, pl.w, pl.pad, codes, scales, s);
    if (e != cudaSuccess) return e;

    const auto kernel = gated ? mx_gemm_kernel<true> : mx_gemm_kernel<false>;
    // the largest a launch may ask for, so that no second CTA shares the SM: each allocates all of its tensor memory
    const int smem = kMaxSmem;
    e = allow_smem(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    Args g = {};
    g.nk = static_cast<int>((c.M + 255) / 256);
    g.w = pl.w;
    g.bufs = pl.bufs;
    g.accs = pl.accs;
    g.ring = pl.ring;
    g.sf_bufs = std::min<int>({kMaxSfBufs, pl.ring, static_cast<int>((kTmemCols - pl.accs * pl.w * pl.bufs) / sf_cols(pl.w))});
    g.row_step = gated ? 256 : 256 * pl.accs;
    g.row_off = gated ? 0 : 256;
    g.n_p = static_cast<int>((c.N + g.row_step - 1) / g.row_step);
    g.tiles = static_cast<int>(g.n_p * ((c.T + pl.w - 1) / pl.w));
    g.ep = c.ep;
    g.status = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(c.ws) + kWsStatusOffset);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr + 1;
    cfg.numAttrs = 1;
    const int pairs = std::min(gated ? resident_pairs<true>(cfg) : resident_pairs<false>(cfg), g.tiles);
    cfg.gridDim = dim3(2 * pairs);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a[0], a[1], sa[0], sa[1], b, sb, g);
}

}  // namespace dbf
