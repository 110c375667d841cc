// Microscaled formats: a matrix to 4-bit codes and scales and back, an
// activation to 8-bit codes and scales and back (dbf_mx.cuh has the formats).
//
// Each kernel reads every input and writes every output once and computes
// little, so device memory bounds it. A warp takes 256 columns (a lane eight
// of them: one 16-byte load of 16-bit values; four lanes a block, whose
// largest magnitude two shuffles find) of four rows, whose loads are all in
// flight before the first is used. The four rows of a 4-bit warp are 32
// apart: their scales are neighbours in the tiled layout, so a warp writes
// them as 16-byte vectors. The 8-bit scales lie block by block ([block][row]),
// the order in which the gated block's epilogue produces them; a CTA gathers
// them for 32 rows in shared memory and writes 32 bytes at a time.
#include "dbf_mx.cuh"

namespace dbf {
namespace {

using namespace mx;

constexpr int kRowsPerWarp = 4;
constexpr int kWarps = 8;
constexpr int kSegment = 256;   // columns of a warp

template <dbf_dtype DT>
__global__ void __launch_bounds__(32 * kWarps) quantize4_kernel(const void *__restrict__ src, int64_t rows, int64_t k, bool vec,
                                 uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, int32_t *status)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // four CTAs along x cover one tile of 128 rows, each kWarps rows of all
    // four groups of 32
    const int64_t tile = blockIdx.x / (32 / kWarps);
    const int r32 = static_cast<int>(blockIdx.x % (32 / kWarps)) * kWarps + warp;
    const int64_t c = static_cast<int64_t>(blockIdx.y) * kSegment + lane * 8;
    const int64_t nb = blocks(k), pitch = nb * 16, tiles = scale_tiles(k);
    float v[kRowsPerWarp][8];
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g) {
        const int64_t r = tile * 128 + g * 32 + r32;
        load8(src, DT, r * k, r < rows ? c : k, k, vec, v[g]);
    }
    uint32_t words[kRowsPerWarp];
    bool bad = false;
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g) {
        const int64_t r = tile * 128 + g * 32 + r32;
        uint32_t byte;
        const uint32_t w = quantize8_e2m1(v[g], byte);
        bad |= byte == 255u;
        if (r < rows && c < nb * kBlock) *reinterpret_cast<uint32_t *>(codes + r * pitch + c / 2) = w;
        words[g] = half_warp_scales(byte, lane);
    }
    const int64_t ct = (c >> 7);   // scale tile of this half-warp; blocks and rows past the end hold scale 0
    if ((lane & 15) == 0 && ct < tiles)
        *reinterpret_cast<uint4 *>(scales + (tile * tiles + ct) * 512 + r32 * 16) =
            make_uint4(words[0], words[1], words[2], words[3]);
    if (status && bad) atomicExch(status, static_cast<int32_t>(DBF_ERR_INVALID_ARG));
}

template <dbf_dtype DT>
__global__ void __launch_bounds__(32 * kWarps) dequantize4_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                   int64_t rows, int64_t k, bool vec, void *__restrict__ dst)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tile = blockIdx.x / (32 / kWarps);
    const int r32 = static_cast<int>(blockIdx.x % (32 / kWarps)) * kWarps + warp;
    const int64_t c = static_cast<int64_t>(blockIdx.y) * kSegment + lane * 8;
    if (c >= k) return;
    const int64_t pitch = code_pitch(k), tiles = scale_tiles(k);
    // the scales of the four rows and four blocks of this half-warp: 16 bytes
    const uint4 s4 = *reinterpret_cast<const uint4 *>(scales + (tile * tiles + (c >> 7)) * 512 + r32 * 16);
    const uint32_t sw[4] = {s4.x, s4.y, s4.z, s4.w};
    uint32_t w[kRowsPerWarp];
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g) {
        const int64_t r = tile * 128 + g * 32 + r32;
        w[g] = r < rows ? *reinterpret_cast<const uint32_t *>(codes + r * pitch + c / 2) : 0u;
    }
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g) {
        const int64_t r = tile * 128 + g * 32 + r32;
        if (r >= rows) break;
        const float s = scale_value((sw[g] >> (8 * ((lane >> 2) & 3))) & 255u);
        float v[8];
        from_e2m1x8(w[g], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= s;
        store8(dst, DT, r * k, c, k, vec, v);
    }
}

template <dbf_dtype DT>
__global__ void __launch_bounds__(32 * kWarps) act8_save_kernel(const void *__restrict__ src, int64_t rows, int64_t k, bool vec,
                                 uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, int32_t *status)
{
    __shared__ uint8_t gather[kSegment / kBlock][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 32;
    const int64_t c = static_cast<int64_t>(blockIdx.y) * kSegment + lane * 8;
    const int64_t nb = blocks(k), pitch = nb * kBlock;
    float v[kRowsPerWarp][8];
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g) {
        const int64_t r = r0 + g * kWarps + warp;
        load8(src, DT, r * k, r < rows ? c : k, k, vec, v[g]);
    }
    bool bad = false;
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g) {
        const int64_t r = r0 + g * kWarps + warp;
        const uint32_t byte = scale_byte8(block_amax(amax_bits8(v[g])));
        const float inv = inv_scale(byte);
        bad |= byte == 255u;
        uint2 w;
        w.x = e4m3x4(v[g][0] * inv, v[g][1] * inv, v[g][2] * inv, v[g][3] * inv);
        w.y = e4m3x4(v[g][4] * inv, v[g][5] * inv, v[g][6] * inv, v[g][7] * inv);
        if (byte == 255u) w = make_uint2(0u, 0u);
        if (r < rows && c < pitch) *reinterpret_cast<uint2 *>(codes + r * pitch + c) = w;
        if ((lane & 3) == 0) gather[lane >> 2][g * kWarps + warp] = static_cast<uint8_t>(byte);
    }
    __syncthreads();
    // a warp writes one block's scales of the CTA's 32 rows
    const int64_t b = static_cast<int64_t>(blockIdx.y) * (kSegment / kBlock) + warp;
    if (b < nb && r0 + lane < rows) scales[b * rows + r0 + lane] = gather[warp][lane];
    if (status && bad) atomicExch(status, static_cast<int32_t>(DBF_ERR_INVALID_ARG));
}

template <dbf_dtype DT>
__global__ void __launch_bounds__(32 * kWarps) act8_load_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                 int64_t rows, int64_t k, bool vec, void *__restrict__ dst)
{
    __shared__ uint8_t gather[kSegment / kBlock][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 32;
    const int64_t c = static_cast<int64_t>(blockIdx.y) * kSegment + lane * 8;
    const int64_t nb = blocks(k), pitch = nb * kBlock;
    uint2 w[kRowsPerWarp];
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g) {
        const int64_t r = r0 + g * kWarps + warp;
        w[g] = r < rows && c < pitch ? *reinterpret_cast<const uint2 *>(codes + r * pitch + c) : make_uint2(0u, 0u);
    }
    const int64_t b = static_cast<int64_t>(blockIdx.y) * (kSegment / kBlock) + warp;
    gather[warp][lane] = b < nb && r0 + lane < rows ? scales[b * rows + r0 + lane] : 0;
    __syncthreads();
    if (c >= k) return;
#pragma unroll
    for (int g = 0; g < kRowsPerWarp; ++g) {
        const int64_t r = r0 + g * kWarps + warp;
        if (r >= rows) break;
        const float s = scale_value(gather[lane >> 2][g * kWarps + warp]);
        float lo[4], hi[4];
        from_e4m3x4(w[g].x, lo);
        from_e4m3x4(w[g].y, hi);
        const float v[8] = {lo[0] * s, lo[1] * s, lo[2] * s, lo[3] * s, hi[0] * s, hi[1] * s, hi[2] * s, hi[3] * s};
        store8(dst, DT, r * k, c, k, vec, v);
    }
}

dim3 grid4(int64_t rows, int64_t k)
{
    return dim3(static_cast<unsigned>((rows + 127) / 128 * (32 / kWarps)), static_cast<unsigned>((k + kSegment - 1) / kSegment));
}
dim3 grid8(int64_t rows, int64_t k)
{
    return dim3(static_cast<unsigned>((rows + 31) / 32), static_cast<unsigned>((k + kSegment - 1) / kSegment));
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
    const bool vec = vectors(src, k);
    const dim3 g = grid4(rows, k);
    if (dt == DBF_F32)
        quantize4_kernel<DBF_F32><<<g, 32 * kWarps, 0, s>>>(src, rows, k, vec, codes, scales, status);
    else if (dt == DBF_BF16)
        quantize4_kernel<DBF_BF16><<<g, 32 * kWarps, 0, s>>>(src, rows, k, vec, codes, scales, status);
    else
        quantize4_kernel<DBF_F16><<<g, 32 * kWarps, 0, s>>>(src, rows, k, vec, codes, scales, status);
    return cudaGetLastError();
}

cudaError_t launch_dequantize4(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t k, void *dst,
                               dbf_dtype dt, cudaStream_t s)
{
    const bool vec = vectors(dst, k);
    const dim3 g = grid4(rows, k);
    if (dt == DBF_F32)
        dequantize4_kernel<DBF_F32><<<g, 32 * kWarps, 0, s>>>(codes, scales, rows, k, vec, dst);
    else if (dt == DBF_BF16)
        dequantize4_kernel<DBF_BF16><<<g, 32 * kWarps, 0, s>>>(codes, scales, rows, k, vec, dst);
    else
        dequantize4_kernel<DBF_F16><<<g, 32 * kWarps, 0, s>>>(codes, scales, rows, k, vec, dst);
    return cudaGetLastError();
}

cudaError_t launch_act8_save(const void *src, dbf_dtype dt, int64_t rows, int64_t k, uint8_t *codes, uint8_t *scales,
                             int32_t *status, cudaStream_t s)
{
    const bool vec = vectors(src, k);
    const dim3 g = grid8(rows, k);
    if (dt == DBF_F32)
        act8_save_kernel<DBF_F32><<<g, 32 * kWarps, 0, s>>>(src, rows, k, vec, codes, scales, status);
    else if (dt == DBF_BF16)
        act8_save_kernel<DBF_BF16><<<g, 32 * kWarps, 0, s>>>(src, rows, k, vec, codes, scales, status);
    else
        act8_save_kernel<DBF_F16><<<g, 32 * kWarps, 0, s>>>(src, rows, k, vec, codes, scales, status);
    return cudaGetLastError();
}

cudaError_t launch_act8_load(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t k, void *dst,
                             dbf_dtype dt, cudaStream_t s)
{
    const bool vec = vectors(dst, k);
    const dim3 g = grid8(rows, k);
    if (dt == DBF_F32)
        act8_load_kernel<DBF_F32><<<g, 32 * kWarps, 0, s>>>(codes, scales, rows, k, vec, dst);
    else if (dt == DBF_BF16)
        act8_load_kernel<DBF_BF16><<<g, 32 * kWarps, 0, s>>>(codes, scales, rows, k, vec, dst);
    else
        act8_load_kernel<DBF_F16><<<g, 32 * kWarps, 0, s>>>(codes, scales, rows, k, vec, dst);
    return cudaGetLastError();
}

}  // namespace dbf
