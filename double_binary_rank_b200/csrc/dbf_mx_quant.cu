// Microscaled formats: a matrix to 4-bit codes and scales and back, an
// activation to 8-bit codes and scales and back (dbf_mx.cuh has the formats).
//
// Each kernel reads every input and writes every output once and computes
// little, so device memory should bound it. A warp takes 256 columns (a lane
// eight of them, four lanes a block) of four rows, whose loads are all in flight
// before the first is used; the quantisers of 16-bit types 512, a lane sixteen.
// The four rows of a 4-bit warp are 32 apart: their scales are neighbours in the
// tiled layout, so a warp writes them as 16-byte vectors. The 8-bit scales lie block by block ([block][row]),
// the order in which the gated block's epilogue produces them; a CTA gathers
// them for 32 rows in shared memory and writes 32 bytes at a time.
#include <type_traits>

#include "dbf_mx.cuh"

namespace dbf {
namespace {

using namespace mx;

constexpr int kRowsPerWarp = 4;
constexpr int kWarps = 8;
constexpr int kSegment = 256;   // columns of a warp

// kVec: rows are whole aligned vectors of eight values. Integer instructions are
// what the quantisers run into first (11008 x 4096 bf16, 17.4 us for the bytes:
// 30 us with eight values to a lane, run-time types and a conversion each; 25 us
// with packed comparisons and compile-time types, the ALU pipe 82 % busy; 20.3 us
// with sixteen values to a lane, 19.5 us with comparisons that take the
// magnitudes themselves).
template <dbf_dtype DT, bool kVec>
__global__ void __launch_bounds__(32 * kWarps) quantize4_kernel(const void *__restrict__ src, int64_t rows, int64_t k,
                                                                uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                                int32_t *status)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // four CTAs along x cover one tile of 128 rows, each kWarps rows of all
    // four groups of 32
    const int64_t tile = blockIdx.x / (32 / kWarps);
    const int r32 = static_cast<int>(blockIdx.x % (32 / kWarps)) * kWarps + warp;
    constexpr int kCols = lane_cols<DT>();
    const int64_t row = tile * 128 + r32, c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * kCols;
    const int64_t nb = blocks(k), pitch = nb * 16, tiles = scale_tiles(k);
    const int left = static_cast<int>(rows - row < 128 ? rows - row : 128);   // row + 32 g exists where 32 g < left
    Raw8 x[kRowsPerWarp][kCols / 8];
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g)
        load_cols<DT, kVec, kCols>(src, (row + 32 * g) * k, 32 * g < left ? c : k, k, rows * k, x[g]);
    uint32_t words[kRowsPerWarp];
    bool bad = false;
    uint8_t *out = codes + row * pitch + c / 2;
    const bool in = c < nb * kBlock;
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g, out += 32 * pitch) {
        uint32_t byte, w[kCols / 8];
        quantize_e2m1<DT, kCols>(x[g], byte, w);
        bad |= byte == 255u;
        if (in && 32 * g < left) store_words(out, w);
        words[g] = tile_scales<kCols>(byte, lane);
    }
    const int64_t ct = c >> 7;   // scale tile of these lanes; blocks and rows past the end hold scale 0
    if (lane % (128 / kCols) == 0 && ct < tiles)
        *reinterpret_cast<uint4 *>(scales + (tile * tiles + ct) * 512 + r32 * 16) =
            make_uint4(words[0], words[1], words[2], words[3]);
    if (status && bad) atomicExch(status, static_cast<int32_t>(DBF_ERR_INVALID_ARG));
}

template <dbf_dtype DT, bool kVec>
__global__ void __launch_bounds__(32 * kWarps) dequantize4_kernel(const uint8_t *__restrict__ codes,
                                                                  const uint8_t *__restrict__ scales, int64_t rows, int64_t k,
                                                                  void *__restrict__ dst)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tile = blockIdx.x / (32 / kWarps);
    const int r32 = static_cast<int>(blockIdx.x % (32 / kWarps)) * kWarps + warp;
    const int64_t row = tile * 128 + r32, c = static_cast<int64_t>(blockIdx.y) * kSegment + lane * 8;
    if (kVec && c >= k) return;
    const int64_t pitch = code_pitch(k), tiles = scale_tiles(k);
    const int left = static_cast<int>(rows - row < 128 ? rows - row : 128);
    // the scales of the four rows and four blocks of this half-warp: 16 bytes
    const bool in_row = kVec || c < k;
    const uint4 s4 = in_row ? *reinterpret_cast<const uint4 *>(scales + (tile * tiles + (c >> 7)) * 512 + r32 * 16) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t sw[4] = {s4.x, s4.y, s4.z, s4.w};
    const uint8_t *in = codes + row * pitch + c / 2;
    uint32_t w[kRowsPerWarp];
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g, in += 32 * pitch) w[g] = in_row && 32 * g < left ? *reinterpret_cast<const uint32_t *>(in) : 0u;
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g) {
        if (32 * g >= left) break;
        const float s = scale_value((sw[g] >> (lane * 2 & 24)) & 255u);
        float v[8];
        from_e2m1x8(w[g], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= s;
        if (kVec)
            store8(dst, DT, (row + 32 * g) * k, c, k, true, v);
        else
            store_shifted8<DT>(dst, (row + 32 * g) * k, c, k, v);
    }
}

template <dbf_dtype DT, bool kVec>
__global__ void __launch_bounds__(32 * kWarps) act8_save_kernel(const void *__restrict__ src, int64_t rows, int64_t k,
                                                                uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                                int32_t *status)
{
    constexpr int kCols = lane_cols<DT>();
    __shared__ uint8_t gather[kCols][32];   // kCols blocks: a warp's columns
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 32, row = r0 + warp;
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * kCols;
    const int64_t nb = blocks(k), pitch = nb * kBlock;
    const int left = static_cast<int>(rows - row < 32 ? rows - row : 32);   // row + 8 g exists where 8 g < left
    Raw8 x[kRowsPerWarp][kCols / 8];
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g)
        load_cols<DT, kVec, kCols>(src, (row + kWarps * g) * k, kWarps * g < left ? c : k, k, rows * k, x[g]);
    bool bad = false;
    uint8_t *out = codes + row * pitch + c;
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g, out += kWarps * pitch) {
        uint32_t byte, w[kCols / 4];
        quantize_e4m3<DT, kCols>(x[g], byte, w);
        bad |= byte == 255u;
        if (kWarps * g < left && c < pitch) store_words(out, w);
        if (lane % (32 / kCols) == 0) gather[lane * kCols / 32][g * kWarps + warp] = static_cast<uint8_t>(byte);
    }
    __syncthreads();
    // a warp writes a block's scales of the CTA's 32 rows
#pragma unroll
    for (int i = 0; i < kCols / kWarps; ++i) {
        const int64_t b = static_cast<int64_t>(blockIdx.y) * kCols + i * kWarps + warp;
        if (b < nb && r0 + lane < rows) scales[b * rows + r0 + lane] = gather[i * kWarps + warp][lane];
    }
    if (status && bad) atomicExch(status, static_cast<int32_t>(DBF_ERR_INVALID_ARG));
}

template <dbf_dtype DT, bool kVec>
__global__ void __launch_bounds__(32 * kWarps) act8_load_kernel(const uint8_t *__restrict__ codes,
                                                                const uint8_t *__restrict__ scales, int64_t rows, int64_t k,
                                                                void *__restrict__ dst)
{
    __shared__ uint8_t gather[kSegment / kBlock][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 32, row = r0 + warp;
    const int64_t c = static_cast<int64_t>(blockIdx.y) * kSegment + lane * 8;
    const int64_t nb = blocks(k), pitch = nb * kBlock;
    const int left = static_cast<int>(rows - row < 32 ? rows - row : 32);
    uint2 w[kRowsPerWarp];
    const uint8_t *in = codes + row * pitch + c;
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g, in += kWarps * pitch)
        w[g] = kWarps * g < left && c < pitch ? *reinterpret_cast<const uint2 *>(in) : make_uint2(0u, 0u);
    const int64_t b = static_cast<int64_t>(blockIdx.y) * (kSegment / kBlock) + warp;
    gather[warp][lane] = b < nb && r0 + lane < rows ? scales[b * rows + r0 + lane] : 0;
    __syncthreads();
    if (kVec && c >= k) return;
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g) {
        if (kWarps * g >= left) break;
        const float s = scale_value(gather[lane >> 2][g * kWarps + warp]);
        float lo[4], hi[4];
        from_e4m3x4(w[g].x, lo);
        from_e4m3x4(w[g].y, hi);
        const float v[8] = {lo[0] * s, lo[1] * s, lo[2] * s, lo[3] * s, hi[0] * s, hi[1] * s, hi[2] * s, hi[3] * s};
        if (kVec)
            store8(dst, DT, (row + kWarps * g) * k, c, k, true, v);
        else
            store_shifted8<DT>(dst, (row + kWarps * g) * k, c, k, v);
    }
}

// cols: columns of a warp
dim3 grid4(int64_t rows, int64_t k, int cols)
{
    return dim3(static_cast<unsigned>((rows + 127) / 128 * (32 / kWarps)), static_cast<unsigned>((k + cols - 1) / cols));
}
dim3 grid8(int64_t rows, int64_t k, int cols)
{
    return dim3(static_cast<unsigned>((rows + 31) / 32), static_cast<unsigned>((k + cols - 1) / cols));
}

template <class F>
void by_type(dbf_dtype dt, bool vec, F f)
{
    using F32 = std::integral_constant<dbf_dtype, DBF_F32>;
    using BF16 = std::integral_constant<dbf_dtype, DBF_BF16>;
    using F16 = std::integral_constant<dbf_dtype, DBF_F16>;
    if (dt == DBF_F32)
        vec ? f(F32{}, std::true_type{}) : f(F32{}, std::false_type{});
    else if (dt == DBF_BF16)
        vec ? f(BF16{}, std::true_type{}) : f(BF16{}, std::false_type{});
    else
        vec ? f(F16{}, std::true_type{}) : f(F16{}, std::false_type{});
}

bool vectors(const void *p, int64_t k) { return k % 8 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

// gridDim limits: x 2^31 - 1, y 65535
bool mx_size_ok(int64_t rows, int64_t k)
{
    return rows > 0 && k > 0 && rows <= (int64_t{1} << 31) && k <= int64_t{65535} * kSegment;
}

cudaError_t launch_quantize4(const void *src, dbf_dtype dt, int64_t rows, int64_t k, uint8_t *codes, uint8_t *scales,
                             int32_t *status, cudaStream_t s)
{
    by_type(dt, vectors(src, k), [&](auto type, auto vec) {
        quantize4_kernel<decltype(type)::value, decltype(vec)::value>
            <<<grid4(rows, k, 32 * lane_cols<decltype(type)::value>()), 32 * kWarps, 0, s>>>(src, rows, k, codes, scales, status);
    });
    return cudaGetLastError();
}

cudaError_t launch_dequantize4(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t k, void *dst,
                               dbf_dtype dt, cudaStream_t s)
{
    const dim3 g = grid4(rows, k, kSegment);
    by_type(dt, vectors(dst, k), [&](auto type, auto vec) {
        dequantize4_kernel<decltype(type)::value, decltype(vec)::value><<<g, 32 * kWarps, 0, s>>>(codes, scales, rows, k, dst);
    });
    return cudaGetLastError();
}

cudaError_t launch_act8_save(const void *src, dbf_dtype dt, int64_t rows, int64_t k, uint8_t *codes, uint8_t *scales,
                             int32_t *status, cudaStream_t s)
{
    by_type(dt, vectors(src, k), [&](auto type, auto vec) {
        act8_save_kernel<decltype(type)::value, decltype(vec)::value>
            <<<grid8(rows, k, 32 * lane_cols<decltype(type)::value>()), 32 * kWarps, 0, s>>>(src, rows, k, codes, scales, status);
    });
    return cudaGetLastError();
}

cudaError_t launch_act8_load(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t k, void *dst,
                             dbf_dtype dt, cudaStream_t s)
{
    const dim3 g = grid8(rows, k, kSegment);
    by_type(dt, vectors(dst, k), [&](auto type, auto vec) {
        act8_load_kernel<decltype(type)::value, decltype(vec)::value><<<g, 32 * kWarps, 0, s>>>(codes, scales, rows, k, dst);
    });
    return cudaGetLastError();
}

}  // namespace dbf
