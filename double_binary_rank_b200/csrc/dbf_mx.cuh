// Microscaled formats shared by the 4-bit base layer and the 8-bit
// activations: block scales, conversions, layouts.
//
// A row is cut into blocks of 32 columns. Each block holds one scale 2^s,
// stored as the byte s + 127 (E8M0; 255 is NaN and marks a block that held a
// NaN or an infinity), and 32 codes of the block's values divided by 2^s:
//   4 bits, E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives;
//       s = floor(log2 amax) - 2, so amax / 2^s lies in [4, 8) and what is
//       above 6 saturates;
//   8 bits, E4M3: up to 448; s the smallest with amax <= 448 * 2^s, so
//       nothing saturates.
// Both s are clamped to [-127, 127]. Dividing by a power of two is exact, so
// the one rounding is that to the code (nearest, ties to even).
#pragma once

#include "dbf_internal.cuh"

namespace dbf {
namespace mx {

constexpr int kBlock = 32;

__host__ __device__ inline int64_t blocks(int64_t k) { return (k + kBlock - 1) / kBlock; }
// bytes of one row of 4-bit codes: whole blocks, 16 bytes each
__host__ __device__ inline int64_t code_pitch(int64_t k) { return blocks(k) * 16; }
// 4-bit scales lie in tiles of 128 rows x 4 blocks (512 bytes), tiles of one
// row tile side by side: the order in which tcgen05.cp brings them into
// tensor memory, so a tile of them is one contiguous copy.
__host__ __device__ inline int64_t scale_tiles(int64_t k) { return (blocks(k) + 3) / 4; }
__host__ __device__ inline int64_t scale_at(int64_t row, int64_t block, int64_t tiles)
{
    return ((row >> 7) * tiles + (block >> 2)) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4 + (block & 3);
}

// Largest finite magnitude's bits in, scale byte out; NaN and infinity give 255.
__device__ __forceinline__ uint32_t scale_byte4(uint32_t amax_bits)
{
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
__device__ __forceinline__ uint32_t scale_byte8(uint32_t amax_bits)
{
    const uint32_t e = amax_bits >> 23;
    if (e == 255u) return 255u;
    const uint32_t up = (amax_bits & 0x7FFFFFu) > 0x600000u ? 1u : 0u;   // above 1.75 * 2^e = 448 * 2^(e - 8)
    return e + up > 8u ? e + up - 8u : 0u;
}
// 2^-s of a scale byte below 254, exact (255 gives 0: the block's codes are 0)
__device__ __forceinline__ float inv_scale(uint32_t b) { return b == 255u ? 0.0f : __uint_as_float((254u - b) << 23); }
// 2^s; NaN for 255
__device__ __forceinline__ float scale_value(uint32_t b)
{
    return __uint_as_float(b == 255u ? 0x7FC00000u : (b ? b << 23 : 0x00400000u));
}

// Eight values to eight E2M1 codes, v[0] in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight E2M1 codes to their values (exact in fp16, then fp32).
__device__ __forceinline__ void from_e2m1x8(uint32_t w, float (&v)[8])
{
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(lo) : "f"(a), "f"(b));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(hi) : "f"(c), "f"(d));
    return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}

__device__ __forceinline__ void from_e4m3x4(uint32_t w, float (&v)[4])
{
    uint32_t h[2];
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[0]) : "h"(static_cast<uint16_t>(w & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[1]) : "h"(static_cast<uint16_t>(w >> 16)));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// Eight values to columns c .. c + 7 of a row, those at or past k left out; c is
// a multiple of 8. vec: every row starts 16-byte aligned and k is a multiple of
// 8, so the eight are one or two aligned vectors; else fp32 or bf16.
__device__ __forceinline__ void store8(void *dst, dbf_dtype dt, int64_t row_start, int64_t c, int64_t k, bool vec,
                                       const float (&v)[8])
{
    if (c >= k) return;
    const int64_t at = row_start + c;
    if (vec) {
        if (dt == DBF_F32) {
            float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(dst) + at);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (dt == DBF_BF16) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    q[i] = *reinterpret_cast<const uint32_t *>(&b);
                } else {
                    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                    q[i] = *reinterpret_cast<const uint32_t *>(&h);
                }
            }
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(dst) + at) = make_uint4(q[0], q[1], q[2], q[3]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (c + i >= k) break;
        store_act(dst, dt, at + i, v[i]);
    }
}

// Eight values as loaded, so that the load can be issued long before its
// conversion: 16-bit types in 'lo', fp32 (and what is loaded without 'vec') in
// both. vec and columns past k as in store8; those read as zero.
struct Raw8 {
    uint4 lo, hi;
};
__device__ __forceinline__ Raw8 load_raw8(const void *src, dbf_dtype dt, int64_t row_start, int64_t c, int64_t k, bool vec)
{
    Raw8 r;
    r.lo = r.hi = make_uint4(0u, 0u, 0u, 0u);
    if (c >= k) return r;
    const int64_t at = row_start + c;
    if (vec) {
        if (dt == DBF_F32) {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(src) + at);
            r.lo = p[0], r.hi = p[1];
        } else {
            r.lo = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + at);
        }
        return r;
    }
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < k ? load_act(src, dt, at + i) : 0.0f;
    r.lo = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    r.hi = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    return r;
}
// The values of what was loaded as vectors
__device__ __forceinline__ void raw8_values(const Raw8 &r, dbf_dtype dt, float (&v)[8])
{
    const uint32_t a[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
    if (dt == DBF_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(a[i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (dt == DBF_BF16) {
            v[2 * i] = __uint_as_float(a[i] << 16);
            v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&a[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}
// v += the eight values (bf16 or fp32)
__device__ __forceinline__ void add_raw8(const Raw8 &r, dbf_dtype dt, bool vec, float (&v)[8])
{
    const uint32_t a[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
    if (dt == DBF_F32 || !vec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += __uint_as_float(a[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] += __uint_as_float(a[i] << 16);
            v[2 * i + 1] += __uint_as_float(a[i] & 0xFFFF0000u);
        }
    }
}

// fp32 bits of the largest magnitude; a NaN among them gives a NaN (as
// integers NaN > infinity > finite, so the comparisons across lanes keep it)
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t amax_bits8(const float (&v)[8])
{
    const float a = max_nan(max_nan(fabsf(v[0]), fabsf(v[1])), max_nan(fabsf(v[2]), fabsf(v[3])));
    const float b = max_nan(max_nan(fabsf(v[4]), fabsf(v[5])), max_nan(fabsf(v[6]), fabsf(v[7])));
    return __float_as_uint(max_nan(a, b)) & 0x7FFFFFFFu;
}

// The four lanes that hold one block agree on its largest magnitude.
__device__ __forceinline__ uint32_t block_amax(uint32_t m)
{
    const uint32_t a = __shfl_xor_sync(0xFFFFFFFFu, m, 1);
    m = a > m ? a : m;
    const uint32_t b = __shfl_xor_sync(0xFFFFFFFFu, m, 2);
    return b > m ? b : m;
}

// How many values of one row a lane takes: sixteen of a 16-bit type, else eight.
// The quantisers run out of integer instructions before anything else, and with
// sixteen the block's scale and its exchange between lanes cost half as many per
// value.
template <dbf_dtype DT>
constexpr int lane_cols() { return DT != DBF_F32 ? 16 : 8; }

// Words first .. first + kOut - 1 of w, 'first' 0 to 3 at run time.
template <int kIn, int kOut>
__device__ __forceinline__ void pick_words(uint32_t (&w)[kIn], uint32_t first, uint32_t (&out)[kOut])
{
    static_assert(kIn >= kOut + 3, "enough words");
#pragma unroll
    for (int i = 0; i < kOut + 1; ++i) w[i] = first & 2u ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < kOut; ++i) out[i] = first & 1u ? w[i + 1] : w[i];
}

// load_raw8 in the form of 'vec' where rows start anywhere: the aligned vectors
// around the eight values, shifted. Single values (each instruction over all
// lanes' vectors again) only where a vector would leave the tensor, which ends
// at element 'total'. A 5003 x 6895 bf16 matrix to 4 bits and back took 130 us in
// single values, 68 us so (31 us with rows of whole vectors).
template <dbf_dtype DT>
__device__ __forceinline__ Raw8 load_shifted8(const void *src, int64_t row_start, int64_t c, int64_t k, int64_t total)
{
    constexpr int kSize = DT == DBF_F32 ? 4 : 2, kVecs = DT == DBF_F32 ? 3 : 2, kWords = 2 * kSize;
    Raw8 r;
    r.lo = r.hi = make_uint4(0u, 0u, 0u, 0u);
    if (c >= k) return r;
    const uintptr_t base = reinterpret_cast<uintptr_t>(src), at = base + static_cast<uintptr_t>(row_start + c) * kSize;
    const uint32_t off = static_cast<uint32_t>(at & 15u);
    const uintptr_t from = at - off;
    const int vecs = off ? kVecs : kVecs - 1;
    uint32_t out[8] = {};
    if (from >= base && from + 16u * vecs <= base + static_cast<uintptr_t>(total) * kSize) {
        uint32_t w[kWords + 4];   // one more than the eight values take
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const uint4 q = i < vecs ? reinterpret_cast<const uint4 *>(from)[i] : make_uint4(0u, 0u, 0u, 0u);
            w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
        }
        if constexpr (kSize == 4) {
            pick_words(w, off >> 2, out);
        } else {
            uint32_t p[5];
            pick_words(w, off >> 2, p);
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = __funnelshift_r(p[i], p[i + 1], (off & 2u) * 8u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c + i >= k) break;
            if constexpr (kSize == 4)
                out[i] = reinterpret_cast<const uint32_t *>(at)[i];
            else
                out[i >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(at)[i]) << (i & 1) * 16;
        }
    }
    if (c + 8 > k) {   // the next row's values
        const int left = static_cast<int>(k - c);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i >= left) {
                if constexpr (kSize == 4)
                    out[i] = 0u;
                else
                    out[i >> 1] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
            }
    }
    r.lo = make_uint4(out[0], out[1], out[2], out[3]);
    r.hi = make_uint4(out[4], out[5], out[6], out[7]);
    return r;
}

// The reverse, a whole warp's call: lane i has columns c = c0 + 8 i of a row that
// starts anywhere. Each lane stores the aligned vectors that begin in its
// neighbour's columns and end in its own; single values only at both ends.
template <dbf_dtype DT>
__device__ __forceinline__ void store_shifted8(void *dst, int64_t row_start, int64_t c, int64_t k, const float (&v)[8])
{
    constexpr int kSize = DT == DBF_F32 ? 4 : 2, kWords = 2 * kSize;
    const int lane = threadIdx.x & 31;
    uint32_t own[kWords], out[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        if (DT == DBF_F32) {
            own[i] = __float_as_uint(v[i]);
        } else if (DT == DBF_BF16) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            own[i] = *reinterpret_cast<const uint32_t *>(&p);
        } else {
            const __half2 p = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            own[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
    }
    const uintptr_t at = reinterpret_cast<uintptr_t>(dst) + static_cast<uintptr_t>(row_start + c) * kSize;
    const uint32_t off = static_cast<uint32_t>(at & 15u);   // the same in all lanes
    const int shift = static_cast<int>(off) / kSize;        // columns of the neighbour in front
    if constexpr (kSize == 4) {
        uint32_t w[11];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[3 + i] = own[i];
#pragma unroll
        for (int i = 0; i < 3; ++i) w[i] = __shfl_up_sync(0xFFFFFFFFu, own[5 + i], 1);
        pick_words(w, 3u - (off >> 2), out);
    } else {
        uint32_t w[8], p[5];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 + i] = own[i], w[i] = __shfl_up_sync(0xFFFFFFFFu, own[i], 1);
        const uint32_t first = 16u - off;   // byte; 16: nothing of the neighbour's
        pick_words(w, first >> 2 & 3u, p);
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = off ? __funnelshift_r(p[i], p[i + 1], (first & 2u) * 8u) : own[i];
    }
    auto one = [&](const uint32_t (&w)[kWords], int i, int64_t column) {
        const uintptr_t to = reinterpret_cast<uintptr_t>(dst) + static_cast<uintptr_t>(row_start + column) * kSize;
        if constexpr (kSize == 4)
            *reinterpret_cast<uint32_t *>(to) = w[i];
        else
            *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(w[i >> 1] >> (i & 1) * 16);
    };
    const int64_t from = c - shift;
    const int low = lane == 0 ? shift : 0;
    if (low == 0 && from + 8 <= k) {
        uint4 *to = reinterpret_cast<uint4 *>(at - off);
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) to[i] = make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i >= low && from + i < k) one(out, i, from + i);
    }
    if (lane == 31) {
#pragma unroll
        for (int i = 1; i < 8; ++i)
            if (i >= 8 - shift && c + i < k) one(own, i, c + i);
    }
}

// Columns c .. c + kCols - 1 of a row as loaded. kVec: rows are whole aligned
// vectors of eight values.
template <dbf_dtype DT, bool kVec, int kCols>
__device__ __forceinline__ void load_cols(const void *src, int64_t row_start, int64_t c, int64_t k, int64_t total, Raw8 (&r)[kCols / 8])
{
#pragma unroll
    for (int i = 0; i < kCols / 8; ++i)
        r[i] = kVec ? load_raw8(src, DT, row_start, c + 8 * i, k, true) : load_shifted8<DT>(src, row_start, c + 8 * i, k, total);
}

// Larger magnitudes of two pairs of 16-bit values, in all but the sign bits; NaN
// wins.
template <dbf_dtype DT>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if (DT == DBF_BF16)
        asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// fp32 bits of the largest magnitude of the block that this lane and its
// neighbours (32 / kCols lanes) hold.
template <dbf_dtype DT, int kCols>
__device__ __forceinline__ uint32_t block_amax_bits(const Raw8 (&r)[kCols / 8])
{
    if (DT == DBF_F32) {
        float v[8];
        raw8_values(r[0], DBF_F32, v);
        return block_amax(amax_bits8(v));
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kCols / 8; ++i) {
        const uint32_t a = max_abs2<DT>(max_abs2<DT>(r[i].lo.x, r[i].lo.y), max_abs2<DT>(r[i].lo.z, r[i].lo.w));
        m = i ? max_abs2<DT>(m, a) : a;
    }
#pragma unroll
    for (int d = 1; d < 32 / kCols; d *= 2) m = max_abs2<DT>(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    m &= 0x7FFF7FFFu;
    const uint32_t hi = m >> 16, lo = m & 0xFFFFu;   // as integers, NaN > infinity > finite
    const uint32_t top = hi > lo ? hi : lo;
    return DT == DBF_BF16 ? top << 16 : __float_as_uint(h2f(static_cast<uint16_t>(top)));
}

// Eight values times 2^-s of a scale byte, exact (bf16 in pairs: results below
// its normal range round to the code 0 in any case).
template <dbf_dtype DT>
__device__ __forceinline__ void scaled_values(const Raw8 &r, uint32_t byte, float (&v)[8])
{
    if (DT == DBF_BF16) {
        const uint32_t f = byte == 255u ? 0u : (254u - byte) << 7, f2 = f | f << 16;
        const uint32_t a[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t p;
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p) : "r"(a[i]), "r"(f2));
            v[2 * i] = __uint_as_float(p << 16);
            v[2 * i + 1] = __uint_as_float(p & 0xFFFF0000u);
        }
        return;
    }
    const float inv = inv_scale(byte);
    raw8_values(r, DT, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= inv;
}

// A lane's values to codes (eight to a word, or four); its neighbours hold the
// rest of the block. Sets the block's scale byte.
template <dbf_dtype DT, int kCols>
__device__ __forceinline__ void quantize_e2m1(const Raw8 (&r)[kCols / 8], uint32_t &byte, uint32_t (&w)[kCols / 8])
{
    byte = scale_byte4(block_amax_bits<DT, kCols>(r));
#pragma unroll
    for (int i = 0; i < kCols / 8; ++i) {
        float v[8];
        scaled_values<DT>(r[i], byte, v);
        w[i] = byte == 255u ? 0u : e2m1x8(v);
    }
}
template <dbf_dtype DT, int kCols>
__device__ __forceinline__ void quantize_e4m3(const Raw8 (&r)[kCols / 8], uint32_t &byte, uint32_t (&w)[kCols / 4])
{
    byte = scale_byte8(block_amax_bits<DT, kCols>(r));
#pragma unroll
    for (int i = 0; i < kCols / 8; ++i) {
        float v[8];
        scaled_values<DT>(r[i], byte, v);
        w[2 * i] = byte == 255u ? 0u : e4m3x4(v[0], v[1], v[2], v[3]);
        w[2 * i + 1] = byte == 255u ? 0u : e4m3x4(v[4], v[5], v[6], v[7]);
    }
}

// kWords neighbouring words, aligned
template <int kWords>
__device__ __forceinline__ void store_words(uint8_t *p, const uint32_t (&w)[kWords])
{
    if constexpr (kWords == 1)
        *reinterpret_cast<uint32_t *>(p) = w[0];
    else if constexpr (kWords == 2)
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The scale bytes of the four blocks of 128 columns as one word, the same in
// every one of the 128 / kCols lanes that hold them.
template <int kCols>
__device__ __forceinline__ uint32_t tile_scales(uint32_t byte, int lane)
{
    constexpr int kLanes = 32 / kCols;
    uint32_t w = byte << (lane / kLanes * 8 & 24);
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, kLanes);
    return w | __shfl_xor_sync(0xFFFFFFFFu, w, 2 * kLanes);
}

}  // namespace mx
}  // namespace dbf
