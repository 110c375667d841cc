// Gradients through the 4-bit layer and its gated block.
//
//   dx = [acc] dx + dy W            (the product's gradient for q(x); the
//                                    rounding of x is passed straight through)
//   du = dh act(g), dg = dh u act'(g), dx = [acc] dx + dg Wg + du Wu
//
// with g and u as the 8-bit checkpoints hold them. The scales of W run along
// the columns, which are now the rows of the product and not its contraction,
// so the block-scaled MMA cannot take them: the codes are expanded on chip to
// bf16, exactly (E2M1 times a power of two has two significant bits), and the
// product runs at the bf16 rate with fp32 accumulators. bf16 gradients are
// operands as they are; fp32 ones are cut into three bf16 pieces of eight bits
// (v = p0 + p1 + p2 exactly), three times the products, whatever dx's type: what
// two pieces leave of a value, 2^-16 of it, is not small beside a dx whose terms
// cancel. The smallest pieces of all weights are summed first: the tensor cores
// truncate their fp32 sums, and a small piece's terms added to the large ones' sum
// are cut off at its last place, each time towards zero (4096 -> 11008 at 2048
// tokens, normal data: dx off by 4.7e-5 with the smallest last, 6.3e-7 so; a
// plain fp32 product by 1.8e-6).
//
// A CTA pair owns 256 columns of W x w <= 512 tokens of dx, over 256 tokens as
// two accumulators (an expanded stage feeds two MMAs a step), contraction over
// the rows of W in stages of 64:
//   warp 0       TMA: w / 2 token rows of the gradient, 64 columns each;
//   warps 2..17  expansion, two groups taking turns by stages: a thread takes
//                32 codes of one row of W (16 bytes and a scale, loaded four
//                stages ahead) and writes them as 64
//                bytes of a 128-byte-swizzled tile whose rows are rows of W:
//                the A operand in its M-major form, so nothing is transposed;
//                a warp's lanes hold 32 different rows, whose swizzled chunks
//                lie in different banks;
//   warp 1       one thread of CTA 0 issues the MMAs (M = 256, N up to 256, K = 16);
//   warps 18..25 epilogue.
// Where the tiles are fewer than the pairs, the contraction is cut into parts
// whose fp32 sums a second launch adds in order.
#include <algorithm>
#include <atomic>

#include "dbf_mx_layer.cuh"
#include "dbf_tc.cuh"

namespace dbf {
namespace {

using namespace mx;
using namespace tc;

constexpr int kMaxStages = 10;
constexpr int kGroups = 2, kExpand = 8, kEpiWarps = 8;   // groups of kExpand warps, taking turns by stages
constexpr int kThreads = 32 * (2 + kGroups * kExpand + kEpiWarps);
constexpr int kAhead = 2;                           // a group's stages that its loads run ahead
constexpr int kRowsK = 64;                          // rows of W per stage
constexpr uint32_t kABytes = 128 * kRowsK * 2;
// A stage is this CTA's half of W's columns and w / 2 token rows; as many as fit.
__host__ __device__ constexpr uint32_t stage_bytes(int w) { return kABytes + w / 2 * kRowsK * 2; }
constexpr int kMaxSmem = 227 * 1024;
constexpr uint32_t kTmemCols = 512;

struct Smem {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full, acc_empty, drain, exit_bar;
    uint32_t tmem_base;
    int abort;
};

struct Args {
    const uint8_t *codes[2], *scales[2];
    int64_t pitch;       // bytes of a row of codes
    int64_t sf_tiles;    // scale tiles of a row tile
    int nb;              // blocks of a row of W
    int N;               // rows of W (contraction)
    int nn;              // stages of one product: ceil(N / 64)
    int mats, planes;    // products summed: weights, pieces of the gradient
    int64_t plane_rows;  // rows from one piece to the next in the gradient's map
    int w;               // tokens per tile
    int ring;            // stages in shared memory
    int halves;          // accumulators: 1 up to 256 tokens, else 2
    int n_p, n_c;        // tiles along the columns of W and along the tokens
    int splits;          // parts of the contraction; over 1, each writes fp32 sums [T][M] of its own
    int tiles;           // n_p * n_c * splits
    float *partial;
    int early;           // W may be read before earlier work is done
    Epilogue ep;
    int32_t *status;
};

// kind::f16 on bf16 operands, A M-major ("transposed"), B K-major
__device__ __forceinline__ uint32_t bf16_idesc(int n)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | 1u << 15 | static_cast<uint32_t>(n >> 3) << 17 | static_cast<uint32_t>(256 >> 4) << 24;
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Codes i and i + 4 of a word of eight as bf16 bit patterns: sign to bit 15, the
// three magnitude bits to the lowest exponent bits and the highest mantissa
// bit. That pattern is the code's value times 2^-126 (0.5 becomes a bf16
// subnormal), so one multiplication by 2^(126 + s) gives value * 2^s. Codes four
// apart lie 16 bits apart, so two shifts serve both; a group of eight columns
// thus comes out in the order 0 4 1 5 2 6 3 7, which column_slot() undoes where
// dx leaves tensor memory.
template <int i>
__device__ __forceinline__ uint32_t bf16_pattern(uint32_t w)
{
    const uint32_t mag = i < 2 ? w << (6 - 4 * i) : w >> (4 * i - 6);
    return (mag & 0x01C001C0u) | ((w << (12 - 4 * i)) & 0x80008000u);
}
__device__ __forceinline__ int column_slot(int lane) { return (lane & 24) | (lane & 1) << 2 | (lane & 7) >> 1; }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The products that are summed, small pieces first, the weights in turn.
__device__ __forceinline__ int weight_of(const Args &g, int seg) { return g.mats == 2 ? seg & 1 : 0; }
__device__ __forceinline__ int piece_of(const Args &g, int seg) { return g.planes - 1 - (g.mats == 2 ? seg >> 1 : seg); }

// Tiles (256 columns of W x w tokens, a part of the contraction) in column
// order, so that pairs that run together share the gradient's rows.
struct Tile {
    int p, c, s, k0, k1;   // column and token tile, part, its stages [k0, k1)
};
__device__ __forceinline__ Tile tile_of(const Args &g, int tile, int nk)
{
    Tile t;
    t.p = tile % g.n_p;
    const int rest = tile / g.n_p;
    t.c = rest % g.n_c;
    t.s = rest / g.n_c;
    t.k0 = static_cast<int>(static_cast<int64_t>(nk) * t.s / g.splits);
    t.k1 = static_cast<int>(static_cast<int64_t>(nk) * (t.s + 1) / g.splits);
    return t;
}

__global__ void __launch_bounds__(kThreads, 1) mx_back_kernel(const __grid_constant__ CUtensorMap mB0,
                                                              const __grid_constant__ CUtensorMap mB1,
                                                              const __grid_constant__ Args g)
{
    extern __shared__ uint8_t raw[];
    uint8_t *stage0 = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const int stages = g.ring;
    const uint32_t stage_size = stage_bytes(g.w);
    float *turn = reinterpret_cast<float *>(stage0 + stages * stage_size);
    Smem *sh = reinterpret_cast<Smem *>(turn + kEpiWarps * kTurnFloats);
    const int warp = warp_number(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int unit = blockIdx.x >> 1, units = gridDim.x >> 1;
    const int nseg = g.mats * g.planes, nk = nseg * g.nn;
    volatile int *abort = &sh->abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            bar_init(&sh->full[i], 1 + 2 * kExpand);
            bar_init(&sh->empty[i], 1);
        }
        bar_init(&sh->acc_full, 1);
        bar_init(&sh->acc_empty, 2 * kEpiWarps);
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

    if (warp == 0) {
        griddep_wait();   // the gradient belongs to earlier work until then
        const int rows = g.w / g.halves / 2;   // of this CTA, per accumulator
        int s = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int tile = unit; tile < g.tiles && ok; tile += units) {
            const Tile c = tile_of(g, tile, nk);
            const int tok = c.c * g.w + static_cast<int>(rank) * rows;
            int seg = c.k0 / g.nn, i = c.k0 - seg * g.nn;
            for (int k = c.k0; k < c.k1; ++k) {
                ok = warp_wait(&sh->empty[s], ph ^ 1u, abort);
                if (!ok) break;
                const CUtensorMap *map = weight_of(g, seg) ? &mB1 : &mB0;
                const int row = tok + static_cast<int>(piece_of(g, seg) * g.plane_rows);
                uint8_t *st = stage0 + s * stage_size + kABytes;
                if (elect_one()) {
                    if (rank == 0) bar_expect_tx(&sh->full[s], g.w * kRowsK * 2);
                    tma_2d_pair(st, map, i * kRowsK, row, &sh->full[s]);
                    if (g.halves == 2) tma_2d_pair(st + rows * kRowsK * 2, map, i * kRowsK, row + 2 * rows, &sh->full[s]);
                }
                __syncwarp();
                ++issued;
                if (++s == stages) s = 0, ph ^= 1u;
                if (++i == g.nn) i = 0, ++seg;
            }
        }
        if (*abort && rank == 0)
            for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
                drain_wait(&sh->full[i % stages], static_cast<uint32_t>(i / stages) & 1u);
    } else if (warp == 1) {
        if (rank == 0) {
            int s = 0;
            uint32_t ph = 0, acc_ph = 0;
            bool ok = true;
            const uint32_t id = bf16_idesc(g.w / g.halves), second = g.w / 4 * kRowsK * 2;
            for (int tile = unit; tile < g.tiles && ok; tile += units) {
                const Tile c = tile_of(g, tile, nk);
                ok = warp_wait(&sh->acc_empty, acc_ph ^ 1u, abort);
                if (!ok) break;
                for (int k = c.k0; k < c.k1; ++k) {
                    ok = warp_wait(&sh->full[s], ph, abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t st = smem_u32(stage0) + s * stage_size;
                    // A: 64 columns of W to a 128-byte row; groups of 8 rows 1 KB apart, the second
                    // 64 columns 8 KB on
                    const uint64_t a = sw128_desc(st, 1024, 8192), b0 = sw128_desc(st + kABytes), b1 = sw128_desc(st + kABytes + second);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint32_t acc = k > c.k0 || kk > 0 ? 1u : 0u;
                            mma_bf16_pair(tmem, a + kk * (2048 >> 4), b0 + 2 * kk, id, acc);
                            if (g.halves == 2) mma_bf16_pair(tmem + 256, a + kk * (2048 >> 4), b1 + 2 * kk, id, acc);
                        }
                        commit_pair_both(&sh->empty[s]);
                    }
                    __syncwarp();
                    if (++s == stages) s = 0, ph ^= 1u;
                }
                if (!ok) break;
                if (elect_one()) commit_pair_both(&sh->acc_full);
                __syncwarp();
                acc_ph ^= 1u;
            }
            if (*abort) {
                if (elect_one()) commit_pair_own(&sh->drain);
                __syncwarp();
                drain_wait(&sh->drain, 0);
            }
        }
    } else if (warp < 2 + kGroups * kExpand) {
        if (!g.early) griddep_wait();
        const int group = (warp - 2) / kExpand, e = (warp - 2) % kExpand;
        const int q = e >> 1, r = (e & 1) * 32 + lane;   // block of 32 columns, row of the stage
        uint32_t to[4];   // where the four 16-byte pieces of the row go
#pragma unroll
        for (int j = 0; j < 4; ++j) to[j] = smem_u32(stage0) + (q >> 1) * 8192 + r * 128 + ((((q & 1) * 4 + j) ^ (r & 7)) << 4);
        // A cursor over (tile, product, stage) runs kAhead of the group's stages
        // ahead of the expansion; its loads land in slots with fixed names, so that
        // nothing waits for a load before the stage that uses it. Its pointers move
        // by 128 rows, the scales' to the next tile of them; 'steps' counts down to
        // the next product or tile.
        static_assert(kGroups * kRowsK == 128, "a group's step is a row tile of scales");
        const uint8_t *code_at = nullptr, *scale_from = nullptr;
        const int64_t code_step = kGroups * kRowsK * g.pitch, scale_step = g.sf_tiles * 512;
        int tile = unit, steps = 0, left = 0;   // left: rows of W from this thread's on
        Tile c = tile_of(g, unit, nk);
        int k = c.k0 + group;
        auto place = [&] {
            while (k >= c.k1 && tile < g.tiles) {
                k -= c.k1;
                tile += units;
                c = tile_of(g, tile < g.tiles ? tile : unit, nk);
                k += c.k0;
            }
            const int at = min(k, nk - 1), seg = at / g.nn, m = weight_of(g, seg), i = at - seg * g.nn, n = i * kRowsK + r;
            const int block = c.p * 8 + static_cast<int>(rank) * 4 + q;
            steps = (min(g.nn - i, c.k1 - at) + kGroups - 1) / kGroups;
            k += steps * kGroups;
            // columns past the last stay zero (rows of dx that are not stored)
            left = tile < g.tiles && block < g.nb ? g.N - n : 0;
            code_at = g.codes[m] + n * g.pitch + block * 16;
            scale_from = g.scales[m] + scale_at(n, block, g.sf_tiles);
        };
        auto load = [&](uint4 &codes, uint32_t &scale) {
            if (steps <= 0) place();
            codes = make_uint4(0u, 0u, 0u, 0u);
            scale = 0;
            if (left > 0) {   // rows past the last stay zero (they meet zeros of the gradient)
                codes = *reinterpret_cast<const uint4 *>(code_at);
                scale = *scale_from;
            }
            --steps;
            left -= kGroups * kRowsK;
            code_at += code_step;
            scale_from += scale_step;
        };
        uint4 codes[kAhead];
        uint32_t scale[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) load(codes[a], scale[a]);
        int64_t total = 0;   // stages of this pair
        for (int t = unit; t < g.tiles; t += units) {
            const Tile c = tile_of(g, t, nk);
            total += c.k1 - c.k0;
        }
        int s = group;                                     // the ring is longer than the groups are many
        uint32_t ph = 0, at = group * stage_size;          // at: the stage's place in the ring
        bool ok = true;
        for (total -= group; total > 0 && ok; total -= kAhead * kGroups) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (a * kGroups >= total) break;
                // exponent field of 2^(126 + s); what passes 254 is a second factor
                const uint32_t field = scale[a] + 126u;
                const uint32_t f1 = scale[a] == 255u ? 0x7FC0u : (field > 254u ? 254u : field) << 7;
                const uint32_t f1x2 = f1 | f1 << 16;
                const uint32_t words[4] = {codes[a].x, codes[a].y, codes[a].z, codes[a].w};
                uint32_t v[16];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[4 * j] = mul_bf16x2(bf16_pattern<0>(words[j]), f1x2);
                    v[4 * j + 1] = mul_bf16x2(bf16_pattern<1>(words[j]), f1x2);
                    v[4 * j + 2] = mul_bf16x2(bf16_pattern<2>(words[j]), f1x2);
                    v[4 * j + 3] = mul_bf16x2(bf16_pattern<3>(words[j]), f1x2);
                }
                if (field > 254u && scale[a] != 255u) {
                    const uint32_t f2 = (127u + field - 254u) << 7, f2x2 = f2 | f2 << 16;
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = mul_bf16x2(v[j], f2x2);
                }
                load(codes[a], scale[a]);
                ok = bar_wait(&sh->empty[s], ph ^ 1u, abort);
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to[j] + at), "r"(v[4 * j]), "r"(v[4 * j + 1]),
                                 "r"(v[4 * j + 2]), "r"(v[4 * j + 3])
                                 : "memory");
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) bar_arrive_leader(&sh->full[s]);
                s += kGroups, at += kGroups * stage_size;
                if (s >= stages) s -= stages, at -= stages * stage_size, ph ^= 1u;
            }
        }
    } else {
        griddep_wait();
        griddep_launch();   // all earlier work is done
        const int quarter = warp & 3, half = (warp - 2 - kGroups * kExpand) >> 2, slot = column_slot(lane);
        float *own = turn + (warp - 2 - kGroups * kExpand) * kTurnFloats;
        // two accumulators: each of a lane quarter's two warps takes one; one: they
        // take turns by 8 (16) tokens
        const bool two = g.halves == 2;
        const int wide = g.w / g.halves, first = two ? half * wide : 0;
        const int j_first = two ? 0 : half * 8, j_step = two ? 8 : 16;
        const uint32_t from = tmem + (two ? half * 256 : 0) + (static_cast<uint32_t>(quarter * 32) << 16);
        uint32_t acc_ph = 0;
        for (int tile = unit; tile < g.tiles; tile += units) {
            const Tile c = tile_of(g, tile, nk);
            const int64_t t = static_cast<int64_t>(c.c) * g.w + first + (lane >> 2);
            const int n = c.p * 256 + static_cast<int>(rank) * 128 + quarter * 32 + (lane & 3) * 8;
            Epilogue ep = g.ep;
            if (g.splits > 1) {
                ep.y = g.partial + c.s * g.ep.T * g.ep.N;
                ep.yd = DBF_F32;
                ep.accumulate = 0;
            }
            if (epilogue_is_simple(ep)) {
                if (!bar_wait(&sh->acc_full, acc_ph, abort)) break;
                acc_ph ^= 1u;
                tc_fence_after();
                for (int j = 2 * j_first; j < wide; j += 2 * j_step) {
                    float v[1][16];
                    tmem_ld16(from + j, v);
                    simple_finish<1>(ep, reinterpret_cast<uint32_t *>(own), t - (lane >> 2) + j, n - (lane & 3) * 8, v, slot);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive_leader(&sh->acc_empty);
                continue;
            }
            Raw8 x[2][1];   // what a chunk of 8 tokens reads is asked for a chunk ahead
            epilogue_reads<false>(ep, t + j_first, n, t + j_first < ep.T, x[0]);
            if (!bar_wait(&sh->acc_full, acc_ph, abort)) break;
            acc_ph ^= 1u;
            tc_fence_after();
            for (int j0 = j_first; j0 < wide; j0 += 2 * j_step) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int j = j0 + i * j_step, next = j + j_step;
                    if (j >= wide) break;
                    epilogue_reads<false>(ep, t + next, n, next < wide && t + next < ep.T, x[i ^ 1]);
                    float col[1][8], row[1][8];
                    tmem_ld8(from + j, col);
                    turn8<1>(own, col, row, slot);
                    epilogue_finish<false>(ep, t + j, n, t + j < ep.T, x[i], row);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_leader(&sh->acc_empty);
        }
    }

    __syncwarp();
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

// fp32 to three bf16 pieces by truncation: p0 the upper half of the word, then
// the same of what is left (each difference is exact); the last has at most
// eight bits left. A NaN or an infinity stays whole in p0.
__device__ __forceinline__ void split3(float v, uint16_t (&p)[3])
{
    const uint32_t b = __float_as_uint(v);
    if ((b & 0x7F800000u) == 0x7F800000u) {
        p[0] = static_cast<uint16_t>((b >> 16) | ((b & 0x7FFFFFu) ? 0x40u : 0u));
        p[1] = p[2] = 0;
        return;
    }
    p[0] = static_cast<uint16_t>(b >> 16);
    const float r1 = v - __uint_as_float(b & 0xFFFF0000u);
    p[1] = static_cast<uint16_t>(__float_as_uint(r1) >> 16);
    const float r2 = r1 - __uint_as_float(__float_as_uint(r1) & 0xFFFF0000u);
    p[2] = static_cast<uint16_t>(__float_as_uint(r2) >> 16);
}

// Eight gradient values to the product's operand planes [planes][T][ld].
__device__ __forceinline__ void store_planes(uint16_t *op, int64_t ld, int64_t plane, int64_t t, int64_t c, int planes,
                                             const float (&v)[8])
{
    uint16_t p[8][3];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (planes == 3)
            split3(v[i], p[i]);
        else
            p[i][0] = static_cast<uint16_t>(__float_as_uint(v[i]) >> 16);   // a bf16 value already
    }
    for (int k = 0; k < planes; ++k) {
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = static_cast<uint32_t>(k == 0 ? p[2 * i][0] : k == 1 ? p[2 * i][1] : p[2 * i][2]) |
                   static_cast<uint32_t>(k == 0 ? p[2 * i + 1][0] : k == 1 ? p[2 * i + 1][1] : p[2 * i + 1][2]) << 16;
        *reinterpret_cast<uint4 *>(op + k * plane + t * ld + c) = make_uint4(q[0], q[1], q[2], q[3]);
    }
}

// dy to operand planes where it cannot be an operand itself (fp32, or rows
// that are no multiple of 16 bytes).
__global__ void __launch_bounds__(256) planes_kernel(const void *__restrict__ dy, dbf_dtype dt, int64_t T, int64_t N, bool vec,
                                                     uint16_t *__restrict__ op, int64_t ld, int planes)
{
    griddep_wait();
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + (threadIdx.x & 31)) * 8;
    if (c >= ld) return;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); t < T; t += static_cast<int64_t>(gridDim.x) * 8) {
        float v[8];
        const Raw8 in = vec             ? load_raw8(dy, DBF_F32, t * N, c, N, true)   // bf16 rows of whole vectors are operands
                        : dt == DBF_F32 ? load_shifted8<DBF_F32>(dy, t * N, c, N, T * N)
                                        : load_shifted8<DBF_BF16>(dy, t * N, c, N, T * N);
        raw8_values(in, dt, v);
        store_planes(op, ld, T * ld, t, c, planes, v);
    }
    griddep_launch();   // at the end: the product's CTAs would take this kernel's registers
}

// dg and du of 32 tokens x 256 columns from dh and the 8-bit g and u, and their
// operand planes (kOperands: fp32, or rows that cannot be operands themselves).
struct GateArgs {
    const uint8_t *g8, *gs, *u8, *us;
    const void *dh;
    void *dg, *du;
    uint16_t *op_g, *op_u;
    int64_t T, N, pitch8, ld;
    int planes;
};

template <dbf_dtype DT, bool kVec, bool kOperands, int kAct>
__global__ void __launch_bounds__(256, kOperands ? 2 : 3) gate_back_kernel(const __grid_constant__ GateArgs a)
{
    __shared__ uint8_t sc[2][8][32];
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 32, row = r0 + warp;
    const int64_t c = static_cast<int64_t>(blockIdx.y) * 256 + lane * 8;
    const int64_t b = static_cast<int64_t>(blockIdx.y) * 8 + warp;
    const bool has = b < blocks(a.N) && r0 + lane < a.T;
    sc[0][warp][lane] = has ? a.gs[b * a.T + r0 + lane] : 0;
    sc[1][warp][lane] = has ? a.us[b * a.T + r0 + lane] : 0;
    const int left = static_cast<int>(a.T - row < 32 ? a.T - row : 32);   // row + 8 i exists where 8 i < left
    // all reads of the lane's four tokens before the first is used
    uint2 wg[4], wu[4];
    Raw8 in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool on = 8 * i < left && c < a.pitch8;
        const int64_t at = (row + 8 * i) * a.pitch8 + c;
        wg[i] = on ? *reinterpret_cast<const uint2 *>(a.g8 + at) : make_uint2(0u, 0u);
        wu[i] = on ? *reinterpret_cast<const uint2 *>(a.u8 + at) : make_uint2(0u, 0u);
        in[i] = kVec ? load_raw8(a.dh, DT, (row + 8 * i) * a.N, on ? c : a.N, a.N, true)
                     : load_shifted8<DT>(a.dh, (row + 8 * i) * a.N, on ? c : a.N, a.N, a.T * a.N);
    }
    __syncthreads();
    if (!kVec || c < a.pitch8) {   // store_shifted8 is the whole warp's
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (8 * i >= left) break;
            const int64_t t = row + 8 * i;
            float dh[8], g[8], u[8];
            raw8_values(in[i], DT, dh);
            const float sg = scale_value(sc[0][lane >> 2][8 * i + warp]), su = scale_value(sc[1][lane >> 2][8 * i + warp]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float p[4], q[4];
                from_e4m3x4(h ? wg[i].y : wg[i].x, p);
                from_e4m3x4(h ? wu[i].y : wu[i].x, q);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float value;
                    const float slope = gate_slope<DT == DBF_F32>(kAct, p[j] * sg, value);
                    g[4 * h + j] = dh[4 * h + j] * (q[j] * su) * slope;
                    u[4 * h + j] = dh[4 * h + j] * value;
                }
            }
            if (kVec) {
                store8(a.dg, DT, t * a.N, c, a.N, true, g);
                store8(a.du, DT, t * a.N, c, a.N, true, u);
            } else {
                store_shifted8<DT>(a.dg, t * a.N, c, a.N, g);
                store_shifted8<DT>(a.du, t * a.N, c, a.N, u);
            }
            if (kOperands && c < a.ld) {
                // columns past the last are not read: the maps end at column N
#pragma unroll
                for (int j = 0; j < 8 && DT == DBF_BF16; ++j) {
                    g[j] = __bfloat162float(__float2bfloat16_rn(g[j]));
                    u[j] = __bfloat162float(__float2bfloat16_rn(u[j]));
                }
                store_planes(a.op_g, a.ld, a.T * a.ld, t, c, a.planes, g);
                store_planes(a.op_u, a.ld, a.T * a.ld, t, c, a.planes, u);
            }
        }
    }
    griddep_launch();   // at the end: the product's CTAs would take this kernel's registers
}

template <dbf_dtype DT, bool kVec>
auto gate_back(bool operands, int act)
{
    constexpr bool kCan = DT == DBF_F32 || !kVec;   // bf16 rows of whole vectors are operands themselves
    if (act == DBF_GATE_SILU)
        return operands ? gate_back_kernel<DT, kVec, kCan, DBF_GATE_SILU> : gate_back_kernel<DT, kVec, false, DBF_GATE_SILU>;
    return operands ? gate_back_kernel<DT, kVec, kCan, DBF_GATE_GELU> : gate_back_kernel<DT, kVec, false, DBF_GATE_GELU>;
}

// dx = [acc] dx + the parts' sums, in order.
__global__ void __launch_bounds__(256) join_kernel(const float *__restrict__ partial, int splits, const __grid_constant__ Epilogue e)
{
    griddep_wait();
    griddep_launch();
    const int64_t N = e.N, plane = e.T * N;
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + (threadIdx.x & 31)) * 8;
    const bool vec = epilogue_vec(e);
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); t < e.T; t += static_cast<int64_t>(gridDim.x) * 8) {
        if (!vec) {   // single values: neighbouring lanes take neighbouring ones
            for (int i = 0; i < 8; ++i) {
                const int64_t at = static_cast<int64_t>(blockIdx.y) * 256 + i * 32 + (threadIdx.x & 31);
                if (at >= N) break;
                const float v = e.accumulate ? load_act(e.y, e.yd, t * N + at) : 0.0f;
                float sum = 0.0f;
                for (int s = 0; s < splits; ++s) sum += partial[s * plane + t * N + at];
                store_act(e.y, e.yd, t * N + at, sum + v);
            }
            continue;
        }
        Raw8 x[1];
        epilogue_reads<false>(e, t, static_cast<int>(c), c < N, x);
        float v[1][8] = {};
        for (int s = 0; s < splits; ++s) {
            const Raw8 r = load_raw8(partial + s * plane, DBF_F32, t * N, c, N, true);
            add_raw8(r, DBF_F32, true, v[0]);
        }
        epilogue_finish<false>(e, t, static_cast<int>(c), c < N, x, v);
    }
}

// CTA pairs that can be resident at once (kept per device)
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
        if (cudaOccupancyMaxActiveClusters(&n, mx_back_kernel, &cfg) == cudaSuccess && n > 0) pairs = std::min(n, pairs);
        (void)cudaGetLastError();
        if (keep) known[dev].store(pairs, std::memory_order_relaxed);
    }
    return pairs;
}

// Tokens per tile (a multiple of 16, over 256 of 32, up to 512) and parts of the contraction.
// Cost of the last pair to finish, in cycles: waves of tiles, each so many
// stages, a stage taking its MMAs (2 w and the hand-over) or the expansion of W
// (the same at every width), and an epilogue; a second launch for the parts,
// whose sums are written and read once more. 4096 -> 11008: 256 tokens 32 us in
// four parts of one tile, 46 us in one; 2048 x 2048 at 600 tokens 15.8 us in
// tiles of 96, 16.9 us in three parts of tiles of 208.
constexpr int64_t kMaxSplits = 16;
struct Plan {
    int w, splits;
};
Plan plan(int64_t M, int64_t T, int64_t nk, int sms)
{
    const int64_t n_p = (M + 255) / 256, pairs = std::max(1, sms / 2);
    Plan best = {16, 1};
    double least = -1;
    for (int w = 16; w <= 512; w += w < 256 ? 16 : 32) {
        const int64_t tiles = n_p * ((T + w - 1) / w);
        for (int splits = 1; splits <= kMaxSplits && splits <= nk; ++splits) {
            if (splits > 1 && tiles * splits > pairs) break;
            const double waves = static_cast<double>((tiles * splits + pairs - 1) / pairs);
            const double stages = static_cast<double>((nk + splits - 1) / splits);
            const double join = splits > 1 ? 4000.0 + 800.0 * splits + 8.0 * T * M * (splits + 1) / 3500.0 : 0.0;   // a launch, and bytes at 3.5 KB a cycle
            const double cost = waves * (stages * std::max(2.0 * w + 120, 560.0) + 3000 + 12.0 * w) + join;
            if (least < 0 || cost < least) least = cost, best = {w, splits};
        }
        if (w >= T) break;
    }
    return best;
}
// pieces of a gradient's values
int pieces(dbf_dtype d) { return d == DBF_F32 ? 3 : 1; }
int64_t stages(int64_t N, int mats, int planes) { return (N + kRowsK - 1) / kRowsK * mats * planes; }

int ring_of(int w)
{
    const int fixed = 1024 + kEpiWarps * kTurnFloats * 4 + static_cast<int>(sizeof(Smem));
    return std::min<int>(kMaxStages, (kMaxSmem - fixed) / stage_bytes(w));
}

int64_t operand_ld(int64_t N) { return (N + 7) / 8 * 8; }
bool direct_operand(int64_t N, dbf_dtype d) { return d == DBF_BF16 && N % 8 == 0; }
size_t plane_bytes(int64_t N, int64_t T, dbf_dtype d)
{
    return align_up(static_cast<size_t>(T * operand_ld(N)) * 2 * pieces(d), 256);
}

struct PdlAttr {
    cudaLaunchAttribute attr[2];
    PdlAttr()
    {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 2;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    }
};

// a warp a row of eight-column lanes
dim3 row_grid(int64_t T, int64_t cols)
{
    return dim3(static_cast<unsigned>(std::min<int64_t>((T + 7) / 8, 1 << 20)), static_cast<unsigned>((cols + 255) / 256));
}

// dx from the operands (one map per weight)
cudaError_t product(const Gradient &c, const void *const *operand, int64_t ld, int planes, bool pre, size_t partial_at, cudaStream_t s)
{
    const int mats = c.codes[1] ? 2 : 1;
    const Plan pl = plan(c.M, c.T, stages(c.N, mats, planes), device_sms());
    const int w = pl.w, halves = w > 256 ? 2 : 1;
    CUtensorMap map[2];
    for (int m = 0; m < 2; ++m) {
        const uint64_t dims[2] = {static_cast<uint64_t>(c.N), static_cast<uint64_t>(c.T * planes)};
        const uint64_t strides[1] = {static_cast<uint64_t>(ld) * 2};
        const uint32_t box[2] = {kRowsK, static_cast<uint32_t>(w / halves / 2)};
        if (!tc_map(&map[m], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, operand[m < mats ? m : 0], dims, strides, box, true))
            return cudaErrorInvalidValue;
    }
    Args g = {};
    for (int m = 0; m < 2; ++m) g.codes[m] = c.codes[m], g.scales[m] = c.scales[m];
    g.pitch = code_pitch(c.M);
    g.sf_tiles = scale_tiles(c.M);
    g.nb = static_cast<int>(blocks(c.M));
    g.N = static_cast<int>(c.N);
    g.nn = static_cast<int>((c.N + kRowsK - 1) / kRowsK);
    g.mats = mats;
    g.planes = planes;
    g.plane_rows = c.T;
    g.w = w;
    g.halves = halves;
    g.n_p = static_cast<int>((c.M + 255) / 256);
    g.n_c = static_cast<int>((c.T + w - 1) / w);
    g.splits = pl.splits;
    g.tiles = g.n_p * g.n_c * g.splits;
    g.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(c.ws) + partial_at);
    g.early = pre || (c.flags & DBF_WEIGHTS_STATIC) ? 1 : 0;
    g.ep.y = c.dx, g.ep.yd = c.dxd, g.ep.accumulate = c.flags & DBF_ACCUMULATE ? 1 : 0;
    g.ep.N = static_cast<int32_t>(c.M), g.ep.T = c.T;
    g.status = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(c.ws) + kWsStatusOffset);

    g.ring = ring_of(w);
    // the largest a launch may ask for, so that no second CTA shares the SM: each allocates all of its tensor memory
    const int smem = kMaxSmem;
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(mx_back_kernel), smem);
    if (e != cudaSuccess) return e;
    PdlAttr attr;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr.attr + 1;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(2 * std::min(resident_pairs(cfg), g.tiles));
    cfg.attrs = attr.attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, mx_back_kernel, map[0], map[1], g);
    if (e != cudaSuccess || pl.splits == 1) return e;
    cudaLaunchConfig_t join = {};
    join.gridDim = row_grid(c.T, c.M);
    join.blockDim = dim3(256);
    join.stream = s;
    join.attrs = attr.attr;
    join.numAttrs = 1;
    return cudaLaunchKernelEx(&join, join_kernel, static_cast<const float *>(g.partial), pl.splits, g.ep);
}

}  // namespace

size_t mx_back_workspace_bytes(int64_t M, int64_t N, int64_t T, dbf_dtype d, int mats)
{
    // parts of the contraction times tokens: at most 16 T, and no more tiles (of
    // 512 tokens at most) than pairs. It grows with T.
    const int64_t n_p = (M + 255) / 256, pairs = std::max(1, device_sms() / 2);
    const size_t partial = static_cast<size_t>(std::min(kMaxSplits * T, pairs * 512 / n_p)) * static_cast<size_t>(M) * 4;
    return kWsHeaderBytes + (direct_operand(N, d) ? 0 : mats * plane_bytes(N, T, d)) + partial;
}

void mx_back_cut(const Gradient &c, int mats, int sms, int64_t (&cut)[8])
{
    const int64_t nk = stages(c.N, mats, pieces(c.dyd));
    const Plan pl = plan(c.M, c.T, nk, sms);
    const int64_t of[8] = {DBF_MX4_GRADIENT, pl.w, pl.w > 256 ? 2 : 1, pl.splits, ring_of(pl.w), nk,
                           (c.M + 255) / 256 * ((c.T + pl.w - 1) / pl.w) * pl.splits, 0};
    std::copy(of, of + 8, cut);
}

cudaError_t mx_backward(const Gradient &c, cudaStream_t s)
{
    const void *operand[2] = {c.dy, nullptr};
    const int planes = pieces(c.dyd);
    if (direct_operand(c.N, c.dyd)) return product(c, operand, c.N, 1, false, kWsHeaderBytes, s);
    uint16_t *op = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(c.ws) + kWsHeaderBytes);
    const int64_t ld = operand_ld(c.N);
    PdlAttr attr;
    cudaLaunchConfig_t pre = {};
    pre.gridDim = row_grid(c.T, ld);
    pre.blockDim = dim3(256);
    pre.stream = s;
    pre.attrs = attr.attr;
    pre.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&pre, planes_kernel, c.dy, c.dyd, c.T, c.N, c.N % 8 == 0, op, ld, planes);
    if (e != cudaSuccess) return e;
    operand[0] = op;
    return product(c, operand, ld, planes, true, kWsHeaderBytes + plane_bytes(c.N, c.T, c.dyd), s);
}

cudaError_t mx_gated_backward(const Gradient &c, int act, const dbf_act8 &sg, const dbf_act8 &su, void *dg, void *du, cudaStream_t s)
{
    const bool want = c.dx != nullptr, direct = direct_operand(c.N, c.dyd);
    GateArgs a = {};
    a.g8 = sg.codes, a.gs = sg.scales, a.u8 = su.codes, a.us = su.scales;
    a.dh = c.dy, a.dg = dg, a.du = du;
    a.T = c.T, a.N = c.N, a.pitch8 = blocks(c.N) * kBlock, a.ld = operand_ld(c.N);
    a.planes = pieces(c.dyd);
    const void *operand[2] = {dg, du};
    if (want && !direct) {
        a.op_g = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(c.ws) + kWsHeaderBytes);
        a.op_u = reinterpret_cast<uint16_t *>(reinterpret_cast<uint8_t *>(a.op_g) + plane_bytes(c.N, c.T, c.dyd));
        operand[0] = a.op_g, operand[1] = a.op_u;
    }
    PdlAttr attr;
    cudaLaunchConfig_t pre = {};
    pre.gridDim = dim3(static_cast<unsigned>((c.T + 31) / 32), static_cast<unsigned>((c.N + 255) / 256));
    pre.blockDim = dim3(256);
    pre.stream = s;
    pre.attrs = attr.attr;
    pre.numAttrs = 1;
    const bool vec = c.N % 8 == 0, op = a.op_g != nullptr;
    const auto kernel = c.dyd == DBF_F32 ? (vec ? gate_back<DBF_F32, true>(op, act) : gate_back<DBF_F32, false>(op, act))
                                         : (vec ? gate_back<DBF_BF16, true>(op, act) : gate_back<DBF_BF16, false>(op, act));
    const cudaError_t e = cudaLaunchKernelEx(&pre, kernel, a);
    if (e != cudaSuccess || !want) return e;
    return product(c, operand, direct ? c.N : a.ld, direct ? 1 : a.planes, true,
                   kWsHeaderBytes + (direct ? 0 : 2 * plane_bytes(c.N, c.T, c.dyd)), s);
}

}  // namespace dbf
