// y = W q(x) and the gated block for few tokens.
//
// With few tokens every weight is used a handful of times, so the codes and
// scales must stream from device memory at its full rate (17 bytes per 32
// weights); the block-scaled MMA (dbf_mx_gemm.cu has the mathematics) with
// the weights as its 128 rows and the tokens, padded to 16, as its columns
// keeps the arithmetic far below that. A cluster of S CTAs shares one block of
// 128 weight rows (of both weights in the gated block), each taking 1/S of
// the columns, so that 148 SMs have loads in flight also for small layers:
//   warp 0      TMA ring of weight stages (256 columns), started before the
//               kernel in front has ended where the caller allows it;
//   warps 2..9  meanwhile quantise the CTA's columns of x into shared memory
//               in the MMA's layout. Each cluster does it again, which up to
//               kInline pieces of 256 columns is cheaper than a launch that does it once;
//               beyond, a pre-pass leaves x's codes and scales in the workspace
//               and warp 0 loads them;
//   warp 1      one thread copies scales and issues the MMAs.
// The partial sums then meet in shared memory: each CTA adds the S partials of
// its share of (token, 32 rows) over distributed shared memory in CTA order,
// so results do not depend on timing, and finishes them.
#include <algorithm>

#include "dbf_mx_layer.cuh"
#include "dbf_tc.cuh"

namespace dbf {
namespace {

using namespace mx;
using namespace tc;

constexpr int kMaxRing = 8;
constexpr int kMaxColumns = 32;   // tokens of a call times its weights: beyond, dbf_mx_gemm.cu is as fast or faster
                                  // (4096 -> 11008 at 64 tokens 14.9 us here, 11.6 us there; at 16 10.3 us and 10.8 us)
constexpr int kInline = 48;       // rows of 256 columns of x up to which a CTA quantises its part itself
constexpr int kSplit = 4;          // parts of the columns (2048 x 2048 at one token: 4.9 us in 4, 5.7 us in 8); 8 where x does not fit otherwise
constexpr int kWorkers = 8;
constexpr int kThreads = 32 * (2 + kWorkers);
constexpr uint32_t kABytes = 128 * 128, kSfBytes = 1024;

struct Smem {
    uint64_t full[kMaxRing], empty[kMaxRing], x_ready, done;
    uint32_t tmem_base;
    int abort;
};

struct Args {
    int nk;      // stages of 256 columns, all CTAs of a cluster together
    int w;       // columns of the MMA: T rounded up to 16
    int ring;    // weight stages in shared memory
    int nks;     // most stages of one CTA
    int T;
    int64_t M;
    const void *x;
    dbf_dtype xd;
    int vec;
    int pre;     // x's codes and scales are in the workspace (mX, mXS)
    int early;   // weights may be read before earlier work is done
    uint32_t tmem_cols;
    Epilogue ep;
    int32_t *status;
};

template <bool kGated>
__global__ void __launch_bounds__(kThreads) mx_decode_kernel(
    const __grid_constant__ CUtensorMap mA0, const __grid_constant__ CUtensorMap mA1, const __grid_constant__ CUtensorMap mS0,
    const __grid_constant__ CUtensorMap mS1, const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mXS,
    const __grid_constant__ Args g)
{
    constexpr int kMats = kGated ? 2 : 1;
    constexpr uint32_t kStage = kMats * (kABytes + kSfBytes);
    extern __shared__ uint8_t raw[];
    uint8_t *ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint8_t *xq = ring + g.ring * kStage;   // per stage: w rows of 128 bytes, then 1 KB of scales
    const uint32_t x_stage = g.w * 128 + 1024;
    Smem *sh = reinterpret_cast<Smem *>(xq + g.nks * x_stage);
    float *part = reinterpret_cast<float *>(ring);   // [mat][token][128 rows], once the ring is done with
    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int S = gridDim.x, rank = blockIdx.x;
    const int row0 = blockIdx.y * 128;
    const int k0 = g.nk * rank / S, nks = g.nk * (rank + 1) / S - k0;
    volatile int *abort = &sh->abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < g.ring; ++i) {
            bar_init(&sh->full[i], 1);
            bar_init(&sh->empty[i], 1);
        }
        bar_init(&sh->x_ready, g.pre ? 1 : kWorkers);
        bar_init(&sh->done, 1);
        sh->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<1>(&sh->tmem_base, g.tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh->tmem_base, 0);
    const uint32_t sf_col = kMats * g.w;   // scales: 8 columns per weight, then 8 of x

    if (warp == 0) {
        if (!g.early) griddep_wait();
        const int first = min(nks, g.ring) - 1;
        int i = 0;
        for (; i < nks; ++i) {
            if (g.pre && i == first) {   // after the first weights, before a wait for a free stage
                griddep_wait();
                if (elect_one()) {
                    bar_expect_tx(&sh->x_ready, nks * x_stage);
                    for (int k = 0; k < nks; ++k) {
                        tma_2d(xq + k * x_stage, &mX, (k0 + k) * 128, 0, &sh->x_ready);
                        tma_3d(xq + k * x_stage + g.w * 128, &mXS, 0, (k0 + k) * 2, 0, &sh->x_ready);
                    }
                }
                __syncwarp();
            }
            const int s = i % g.ring;
            if (!warp_wait(&sh->empty[s], (static_cast<uint32_t>(i / g.ring) & 1u) ^ 1u, abort)) break;
            uint8_t *st = ring + s * kStage;
            if (elect_one()) {
                bar_expect_tx(&sh->full[s], kStage);
                tma_2d(st, &mA0, (k0 + i) * 128, row0, &sh->full[s]);
                if (kGated) tma_2d(st + kABytes, &mA1, (k0 + i) * 128, row0, &sh->full[s]);
                tma_3d(st + kMats * kABytes, &mS0, 0, (k0 + i) * 2, blockIdx.y, &sh->full[s]);
                if (kGated) tma_3d(st + kMats * kABytes + kSfBytes, &mS1, 0, (k0 + i) * 2, blockIdx.y, &sh->full[s]);
            }
            __syncwarp();
        }
        if (*abort && g.pre && i >= first) drain_wait(&sh->x_ready, 0);
        if (*abort)
            for (int j = i > g.ring ? i - g.ring : 0; j < i; ++j)
                drain_wait(&sh->full[j % g.ring], static_cast<uint32_t>(j / g.ring) & 1u);
    } else if (warp == 1) {
        const uint32_t id0 = mxf4_idesc(128, g.w, 0), id2 = mxf4_idesc(128, g.w, 2);
        bool ok = warp_wait(&sh->x_ready, 0, abort);
        for (int i = 0; i < nks && ok; ++i) {
            const int s = i % g.ring;
            ok = warp_wait(&sh->full[s], static_cast<uint32_t>(i / g.ring) & 1u, abort);
            if (!ok) break;
            tc_fence_after();
            const uint32_t st = smem_u32(ring) + s * kStage, sf = st + kMats * kABytes;
            const uint32_t xs = smem_u32(xq) + i * x_stage;
            const uint64_t b = sw128_desc(xs);
            if (elect_one()) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    scale_copy(tmem + sf_col + 4 * c, scale_desc(sf + c * 512));
                    if (kGated) scale_copy(tmem + sf_col + 8 + 4 * c, scale_desc(sf + kSfBytes + c * 512));
                    scale_copy(tmem + sf_col + 8 * kMats + 4 * c, scale_desc(xs + g.w * 128 + c * 512));
                }
#pragma unroll
                for (int m = 0; m < kMats; ++m) {
                    const uint64_t a = sw128_desc(st + m * kABytes);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_mxf4<1>(tmem + m * g.w, a + 2 * kk, b + 2 * kk, kk & 1 ? id2 : id0,
                                    tmem + sf_col + 8 * m + 4 * (kk >> 1), tmem + sf_col + 8 * kMats + 4 * (kk >> 1),
                                    i > 0 || kk > 0 ? 1u : 0u);
                }
                commit_own(&sh->empty[s]);
            }
            __syncwarp();
        }
        if (elect_one()) commit_own(&sh->done);
        __syncwarp();
        drain_wait(&sh->done, 0);
    } else {
        const int worker = warp - 2;
        griddep_wait();     // x, y and the addends belong to earlier work until then
        griddep_launch();   // what follows may be set up: all earlier work is done
        for (int u0 = worker; u0 < g.T * nks && !g.pre; u0 += 4 * kWorkers) {
            Raw8 in[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int u = u0 + i * kWorkers;
                const int t = u / nks, ks = u - t * nks;
                const int64_t c = static_cast<int64_t>(k0 + ks) * 256 + lane * 8;
                in[i] = load_raw8(g.x, g.xd, t * g.M, u < g.T * nks ? c : g.M, g.M, g.vec);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int u = u0 + i * kWorkers;
                if (u >= g.T * nks) break;
                const int t = u / nks, ks = u - t * nks;
                uint32_t byte, q[1];
                const Raw8 r[1] = {in[i]};
                if (g.xd == DBF_BF16 && g.vec)
                    quantize_e2m1<DBF_BF16, 8>(r, byte, q);
                else   // fp32 values, loaded as they are or one by one
                    quantize_e2m1<DBF_F32, 8>(r, byte, q);
                const uint32_t word = tile_scales<8>(byte, lane);
                uint8_t *xs = xq + ks * x_stage;
                *reinterpret_cast<uint32_t *>(xs + t * 128 + (((lane >> 2) ^ (t & 7)) << 4) + (lane & 3) * 4) = q[0];
                if ((lane & 15) == 0)
                    *reinterpret_cast<uint32_t *>(xs + g.w * 128 + (lane >> 4) * 512 + (t & 31) * 16 + (t >> 5) * 4) = word;
            }
        }
        fence_proxy_async();   // the MMA reads what these stores wrote
        __syncwarp();
        if (lane == 0 && !g.pre) bar_arrive(&sh->x_ready);
        if (bar_wait(&sh->done, 0, abort)) {
            tc_fence_after();
            const int quarter = warp & 3, half = worker >> 2;
            for (int col = half * 16; col < kMats * g.w; col += 32) {
                float v[1][16];
                tmem_ld16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + col, v);
#pragma unroll
                for (int j = 0; j < 16; ++j) part[(col + j) * 128 + quarter * 32 + lane] = v[0][j];
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    if (warp >= 2) {
        const uint32_t base = smem_u32(part);
        // a unit is 8 tokens x 32 rows, a lane eight rows of one token
        for (int u = rank + S * (warp - 2); u < (g.T + 7) / 8 * 4; u += S * kWorkers) {
            const int t = (u >> 2) * 8 + (lane >> 2), r = (u & 3) * 32 + (lane & 3) * 8;
            Raw8 x[kMats];
            epilogue_reads<kGated>(g.ep, t, row0 + r, t < g.T, x);
            float sum[kMats][8];
#pragma unroll
            for (int m = 0; m < kMats; ++m) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[m][i] = 0.0f;
                const uint32_t at = base + ((m * g.w + t) * 128 + r) * 4;
                for (int s = 0; s < S; ++s) {
                    const float4 a = ld_cluster_f32x4(at, s), b = ld_cluster_f32x4(at + 16, s);
                    sum[m][0] += a.x, sum[m][1] += a.y, sum[m][2] += a.z, sum[m][3] += a.w;
                    sum[m][4] += b.x, sum[m][5] += b.y, sum[m][6] += b.z, sum[m][7] += b.w;
                }
            }
            epilogue_finish<kGated>(g.ep, t, row0 + r, t < g.T, x, sum);
        }
    }
    __syncwarp();
    cluster_sync();   // no CTA ends while another still reads its partial sums
    if (threadIdx.x == 0 && sh->abort && g.status) atomicExch(g.status, static_cast<int32_t>(DBF_ERR_TIMEOUT));
    if (warp == 1) {
        tc_fence_after();
        tmem_free<1>(tmem, g.tmem_cols);
    }
}

struct Shape {
    int w, split, ring, nks, pre, tmem_cols;
    size_t smem;
};

// Split of the columns, ring depth and CTAs to an SM; false when the CTA's
// columns of x do not fit in shared memory.
bool shape(int64_t M, int64_t N, int64_t T, int mats, int64_t sms, Shape &p)
{
    if (T > kMaxColumns / mats) return false;
    const int64_t nk = (M + 255) / 256, row_blocks = (N + 127) / 128;
    if (row_blocks > 65535) return false;
    p.w = static_cast<int>((T + 15) / 16 * 16);
    const int64_t stage = mats * int64_t{kABytes + kSfBytes}, x_stage = p.w * 128 + 1024, partials = int64_t{mats} * p.w * 512;
    const int64_t fixed = 1024 + sizeof(Smem);
    for (int per_sm = 2; per_sm >= 1; --per_sm) {
        const int64_t room = (per_sm == 2 ? 113 : 227) * 1024 - fixed;
        int64_t split = std::max<int64_t>(1, std::min<int64_t>({kSplit, nk, per_sm * sms / row_blocks}));
        // one CTA to an SM where that occupies four fifths of them and a CTA's
        // weights are all in flight at once (4096 x 4096 at one token: 6.2 us split
        // in 4, 7.0 us in 8; 8192 x 8192, whose CTAs would take 16 stages: 13.0 us
        // at one to an SM, 10.2 us at two)
        const int64_t one = sms / row_blocks;
        if (one >= 1 && one <= kSplit && one * row_blocks * 5 >= sms * 4 && (nk + one - 1) / one <= kMaxRing) split = std::min(one, nk);
        for (; split <= std::min<int64_t>(8, nk); ++split) {
            p.split = static_cast<int>(split);
            p.nks = static_cast<int>((nk + split - 1) / split);
            const int64_t x_bytes = p.nks * x_stage, fit = (room - x_bytes) / stage;
            if (fit < 2) continue;
            int64_t ring = std::min<int64_t>({fit, kMaxRing, std::max(2, p.nks)});
            while (ring < fit && ring * stage + x_bytes < partials) ++ring;   // the partial sums take this place
            if (ring * stage + x_bytes < partials) continue;
            p.ring = static_cast<int>(ring);
            // Shared memory in proportion to tensor memory: whatever CTAs share an SM,
            // of this or another of these kernels, their columns are always there, so
            // that no CTA waits for them while another of its cluster waits at the
            // exchange. (The other kernels with tensor memory take 192 KB at least:
            // what is left beside them holds no CTA of this one, two stages and more.)
            const int cols = mats * p.w + 8 * mats + 8;
            p.tmem_cols = 32;
            while (p.tmem_cols < cols) p.tmem_cols *= 2;
            p.smem = static_cast<size_t>(std::max<int64_t>(fixed + x_bytes + ring * stage, 227 * 1024 / 512 * p.tmem_cols));
            p.pre = T * p.nks > kInline ? 1 : 0;
            return true;
        }
    }
    return false;
}

}  // namespace

bool mx_decode_fits(int64_t M, int64_t N, int64_t T, int mats)
{
    Shape p;
    return shape(M, N, T, mats, device_sms(), p);
}

bool mx_decode_cut(const Product &c, int sms, int64_t (&cut)[8])
{
    Shape p;
    if (!shape(c.M, c.N, c.T, c.mats, sms, p)) return false;
    const int64_t of[8] = {DBF_MX4_FEW_TOKENS, p.w, p.split, p.pre, p.ring, p.nks, (c.N + 127) / 128, c.T - 1};
    std::copy(of, of + 8, cut);
    return true;
}

cudaError_t mx_decode(const Product &c, cudaStream_t s)
{
    Shape p;
    if (!shape(c.M, c.N, c.T, c.mats, device_sms(), p)) return cudaErrorInvalidValue;
    const bool gated = c.mats == 2;
    CUtensorMap a[2], sa[2];
    for (int m = 0; m < 2; ++m) {
        const uint64_t dims[2] = {static_cast<uint64_t>(code_pitch(c.M)), static_cast<uint64_t>(c.N)};
        const uint64_t strides[1] = {dims[0]};
        const uint32_t box[2] = {128, 128};
        const uint64_t tiles = static_cast<uint64_t>(scale_tiles(c.M));
        const uint64_t sdims[3] = {128, tiles, static_cast<uint64_t>((c.N + 127) / 128)};
        const uint64_t sstrides[2] = {512, tiles * 512};
        const uint32_t sbox[3] = {128, 2, 1};
        if (m > 0 && !gated) {
            a[m] = a[0], sa[m] = sa[0];
            break;
        }
        if (!tc_map(&a[m], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, c.codes[m], dims, strides, box, true) ||
            !tc_map(&sa[m], CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, c.scales[m], sdims, sstrides, sbox, false))
            return cudaErrorInvalidValue;
    }
    CUtensorMap xm = a[0], xs = sa[0];
    uint8_t *codes = static_cast<uint8_t *>(c.ws) + x_codes_at(), *scales = static_cast<uint8_t *>(c.ws) + x_scales_at(c.M, c.T);
    if (p.pre) {
        const uint64_t dims[2] = {static_cast<uint64_t>(code_pitch(c.M)), static_cast<uint64_t>(c.T)};
        const uint32_t box[2] = {128, static_cast<uint32_t>(p.w)};
        const uint64_t tiles = static_cast<uint64_t>(scale_tiles(c.M));
        const uint64_t sdims[3] = {128, tiles, 1};
        const uint64_t sstrides[2] = {512, tiles * 512};
        const uint32_t sbox[3] = {128, 2, 1};
        if (!tc_map(&xm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, dims, box, true) ||
            !tc_map(&xs, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, scales, sdims, sstrides, sbox, false))
            return cudaErrorInvalidValue;
        const cudaError_t e = mx_quantize_x(c, p.w, 128, codes, scales, s);
        if (e != cudaSuccess) return e;
    }
    Args g = {};
    g.pre = p.pre;
    g.nk = static_cast<int>((c.M + 255) / 256);
    g.w = p.w;
    g.ring = p.ring;
    g.nks = p.nks;
    g.T = static_cast<int>(c.T);
    g.M = c.M;
    g.x = c.x;
    g.xd = c.xd;
    g.vec = c.M % 8 == 0;   // x is 16-byte aligned
    g.early = p.pre || (c.flags & DBF_WEIGHTS_STATIC) ? 1 : 0;
    g.tmem_cols = static_cast<uint32_t>(p.tmem_cols);
    g.ep = c.ep;
    g.status = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(c.ws) + kWsStatusOffset);

    const auto kernel = gated ? mx_decode_kernel<true> : mx_decode_kernel<false>;
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), static_cast<int>(p.smem), true);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.split), static_cast<unsigned>((c.N + 127) / 128));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a[0], a[1], sa[0], sa[1], xm, xs, g);
}

}  // namespace dbf
