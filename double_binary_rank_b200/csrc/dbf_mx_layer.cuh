// What the 4-bit layer's product kernels share: their epilogue (plain and
// gated) and the host-side description of a call.
#pragma once

#include "dbf_mx.cuh"

namespace dbf {
namespace mx {

constexpr int kMaxDevices = 64;

// Outputs of one product call. Plain: y = [acc] y + W q(x). Gated: g and u
// are the two products plus the optional addends, y = act(g) u, and g and u
// are kept in 8 bits where g8 is set.
struct Epilogue {
    void *y;
    dbf_dtype yd;
    int accumulate;
    int act;
    const void *g_add, *u_add;   // T x N, add_dt; null: none
    dbf_dtype add_dt;
    uint8_t *g8, *gs, *u8, *us;   // 8-bit codes [T][pitch8] and scales [ceil(N/32)][T]; null: not kept
    int64_t pitch8;
    int32_t N;
    int64_t T;
};

// act(g) and its derivative. SiLU: g s with s = 1 / (1 + e^-g), derivative
// s (1 + g (1 - s)). GELU in its tanh form: with z = c (g + 0.044715 g^3) and
// c = sqrt(2 / pi), g / 2 (1 + tanh z) = g s with s = 1 / (1 + e^-2z),
// derivative s + g s (1 - s) 2 c (1 + 3 * 0.044715 g^2). e^-g overflows to
// infinity and its reciprocal is 0, as the limit is.
// The reciprocal is off by a unit of fp32 (2^-23 of it) at most; below 2^-126 it
// is 0. kExact, for results that stay fp32: expf, off by two units. Results that
// are rounded to bf16 (2^-8 of a value) take __expf, off by 2 + 1.173 |z| units of
// e^-z, at most 2^-16 where s is not 0: with expf for them too the plain gate took
// 85.6 us, 80.3 us so (2 x (4096 -> 11008) at 2048 tokens); fp32 results 89 us
// either way. A division instead of the reciprocal took fp32 results to 130 us.
constexpr float kGelu2c = 1.5957691216057308f, kGeluCube = 0.044715f;
template <bool kExact>
__device__ __forceinline__ float sigmoid(float g)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + (kExact ? expf(-g) : __expf(-g))));
    return r;
}
template <bool kExact>
__device__ __forceinline__ float gate_value(int act, float g)
{
    return g * sigmoid<kExact>(act == DBF_GATE_SILU ? g : kGelu2c * (g + kGeluCube * g * g * g));
}
template <bool kExact>
__device__ __forceinline__ float gate_slope(int act, float g, float &value)
{
    if (act == DBF_GATE_SILU) {
        const float s = sigmoid<kExact>(g);
        value = g * s;
        return s * (1.0f + g * (1.0f - s));
    }
    const float s = sigmoid<kExact>(kGelu2c * (g + kGeluCube * g * g * g));
    const float d = s * (1.0f - s);
    value = g * s;
    return d == 0.0f ? s : s + g * d * kGelu2c * (1.0f + 3.0f * kGeluCube * g * g);   // d == 0: g * g may be infinite
}

// ---- epilogue. A lane finishes eight consecutive columns c .. c + 7 of one
// token (four neighbouring lanes hold a block of 32, for the 8-bit format);
// what it reads (y when accumulating, the addends) it asks for early with
// epilogue_reads(). Every lane of the warp calls these; 'on' says whether the
// lane's token exists.
__device__ __forceinline__ bool epilogue_vec(const Epilogue &e) { return (e.N & 7) == 0; }

template <bool kGated>
__device__ __forceinline__ void epilogue_reads(const Epilogue &e, int64_t t, int c, bool on, Raw8 (&x)[kGated ? 2 : 1])
{
    const int64_t N = e.N;
    if constexpr (kGated) {
        x[0] = load_raw8(e.g_add, e.add_dt, t * N, on && e.g_add ? c : N, N, epilogue_vec(e));
        x[1] = load_raw8(e.u_add, e.add_dt, t * N, on && e.u_add ? c : N, N, epilogue_vec(e));
    } else {
        x[0] = load_raw8(e.y, e.yd, t * N, on && e.accumulate ? c : N, N, epilogue_vec(e));
    }
}

// One block of the 8-bit format from the four lanes that hold it; lanes past
// the last column hold zeros.
__device__ __forceinline__ void keep8(uint8_t *codes, uint8_t *scales, int64_t pitch, int64_t T, int64_t t, int c, bool on,
                                      const float (&v)[8])
{
    const uint32_t byte = scale_byte8(block_amax(amax_bits8(v)));
    const float inv = inv_scale(byte);
    uint2 w;
    w.x = e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    w.y = e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    if (byte == 255u) w = make_uint2(0u, 0u);
    if (!on || c >= pitch) return;
    *reinterpret_cast<uint2 *>(codes + t * pitch + c) = w;
    if ((c & 31) == 0) scales[static_cast<int64_t>(c / kBlock) * T + t] = static_cast<uint8_t>(byte);
}

template <bool kGated>
__device__ __forceinline__ void epilogue_finish(const Epilogue &e, int64_t t, int c, bool on, const Raw8 (&x)[kGated ? 2 : 1],
                                                float (&v)[kGated ? 2 : 1][8])
{
    const int64_t N = e.N;
    const bool vec = epilogue_vec(e);
    if constexpr (!kGated) {
        if (e.accumulate) add_raw8(x[0], e.yd, vec, v[0]);
    } else {
        float(&g)[8] = v[0];
        float(&u)[8] = v[1];
        if (e.g_add) add_raw8(x[0], e.add_dt, vec, g);
        if (e.u_add) add_raw8(x[1], e.add_dt, vec, u);
        if (e.g8) {
            if (c + 8 > N) {   // columns past the last may hold anything, a NaN too
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i >= N) g[i] = u[i] = 0.0f;
            }
            keep8(e.g8, e.gs, e.pitch8, e.T, t, c, on, g);
            keep8(e.u8, e.us, e.pitch8, e.T, t, c, on, u);
        }
        if (e.yd == DBF_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = gate_value<true>(e.act, g[i]) * u[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = gate_value<false>(e.act, g[i]) * u[i];
        }
    }
    if (on) store8(e.y, e.yd, t * N, c, N, vec, v[0]);
}

// Tensor memory holds a column of W's rows per lane and a token per register;
// the epilogue wants eight columns of one token per lane. A warp turns 8
// tokens x 32 columns in its own shared memory: rows of 36 floats, so that the
// 16-byte reads of eight lanes (two tokens, four groups of columns) hit
// different banks.
constexpr int kTurnFloats = 8 * 36;   // per accumulator

// slot: which of the 32 columns the lane holds.
template <int kMats>
__device__ __forceinline__ void turn8(float *own, const float (&col)[kMats][8], float (&row)[kMats][8], int slot)
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j) own[m * kTurnFloats + j * 36 + slot] = col[m][j];
    __syncwarp();
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
        const float4 *p = reinterpret_cast<const float4 *>(own + m * kTurnFloats + (lane >> 2) * 36 + (lane & 3) * 8);
        const float4 a = p[0], b = p[1];
        row[m][0] = a.x, row[m][1] = a.y, row[m][2] = a.z, row[m][3] = a.w;
        row[m][4] = b.x, row[m][5] = b.y, row[m][6] = b.z, row[m][7] = b.w;
    }
}

// The epilogue where nothing but the products is read: 16 tokens at once are
// finished as they come, a column of 16 tokens per lane. fp32, and rows that are no
// whole 16-byte vectors, are stored so (a warp's lanes are 128 or 64 bytes of a
// row); other bf16 is turned as pairs of tokens in one word: a third of the
// instructions of the general one, whose issue bounds the prefill kernel's
// epilogue.
__device__ __forceinline__ bool epilogue_is_simple(const Epilogue &e)
{
    return !e.accumulate && !e.g_add && !e.u_add && !e.g8;
}
// A lane's column of 16 tokens of a T x N matrix as loaded (all loads before the
// first use), added to v, and stored from it. n: the column.
__device__ __forceinline__ void read_column(const void *src, dbf_dtype dt, const Epilogue &e, int64_t t0, int n, uint32_t (&a)[16])
{
    const int left = n < e.N && src ? static_cast<int>(e.T - t0 < 16 ? e.T - t0 : 16) : 0;
    const int64_t at = t0 * e.N + n, step = e.N;
    if (dt == DBF_F32) {
        const uint32_t *p = static_cast<const uint32_t *>(src) + at;
#pragma unroll
        for (int j = 0; j < 16; ++j) a[j] = j < left ? p[j * step] : 0u;
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(src) + at;
#pragma unroll
        for (int j = 0; j < 16; ++j) a[j] = j < left ? p[j * step] : 0u;
    }
}
__device__ __forceinline__ void add_column(const uint32_t (&a)[16], dbf_dtype dt, float (&v)[16])
{
    const int shift = dt == DBF_F32 ? 0 : 16;
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] += __uint_as_float(a[j] << shift);
}
template <int kMats, int kAct>
__device__ __forceinline__ void store_column(const Epilogue &e, int64_t t0, int n, const float (&v)[kMats][16])
{
    const int left = n < e.N ? static_cast<int>(e.T - t0 < 16 ? e.T - t0 : 16) : 0;
    const int64_t at = t0 * e.N + n, step = e.N;
    if (e.yd == DBF_F32) {
        float *p = static_cast<float *>(e.y) + at;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float y = kMats == 2 ? gate_value<true>(kAct, v[0][j]) * v[kMats - 1][j] : v[0][j];
            if (j < left) p[j * step] = y;
        }
    } else {
        __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(e.y) + at;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float y = kMats == 2 ? gate_value<false>(kAct, v[0][j]) * v[kMats - 1][j] : v[0][j];
            if (j < left) p[j * step] = __float2bfloat16_rn(y);
        }
    }
}
// n0: the warp's first column; own: kTurnFloats words; slot: which column the
// lane holds
template <int kMats, int kAct = DBF_GATE_SILU>
__device__ __forceinline__ void simple_finish(const Epilogue &e, uint32_t *own, int64_t t0, int n0, const float (&v)[kMats][16],
                                              int slot)
{
    const int lane = threadIdx.x & 31;
    if (e.yd == DBF_F32 || !epilogue_vec(e)) {
        store_column<kMats, kAct>(e, t0, n0 + slot, v);
        return;
    }
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        float a = v[0][2 * p], b = v[0][2 * p + 1];
        if (kMats == 2) {
            a = gate_value<false>(kAct, a) * v[kMats - 1][2 * p];
            b = gate_value<false>(kAct, b) * v[kMats - 1][2 * p + 1];
        }
        const __nv_bfloat162 w = __floats2bfloat162_rn(a, b);
        own[p * 36 + slot] = *reinterpret_cast<const uint32_t *>(&w);
    }
    __syncwarp();
    const int p = lane >> 2, c = n0 + (lane & 3) * 8;
    const uint4 a = *reinterpret_cast<const uint4 *>(own + p * 36 + (lane & 3) * 8);
    const uint4 b = *reinterpret_cast<const uint4 *>(own + p * 36 + (lane & 3) * 8 + 4);
    if (c >= e.N) return;
    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(e.y) + (t0 + 2 * p) * e.N + c;
    if (t0 + 2 * p < e.T)
        *reinterpret_cast<uint4 *>(y) = make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                                                   __byte_perm(b.x, b.y, 0x5410), __byte_perm(b.z, b.w, 0x5410));
    if (t0 + 2 * p + 1 < e.T)
        *reinterpret_cast<uint4 *>(y + e.N) = make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                                                         __byte_perm(b.x, b.y, 0x7632), __byte_perm(b.z, b.w, 0x7632));
}

// The same rows for the gated block with bf16 addends and 8-bit copies of g and
// u, 16 tokens at once, a lane sixteen columns of one token: two lanes hold a
// block, so its scale is found once for sixteen values. They are columns 8 s ..
// 8 s + 7 and 16 more than these, s the lane's parity, so that the two lanes'
// 16-byte accesses meet in whole 32-byte sectors.
__device__ __forceinline__ bool epilogue_is_bf16(const Epilogue &e)
{
    return epilogue_vec(e) && e.yd == DBF_BF16 && !e.g_add == !e.u_add && (!e.g_add || e.add_dt == DBF_BF16);
}
// t: the lane's token; c: its first column (rows hold whole vectors of eight)
template <bool kAdd>
__device__ __forceinline__ void gated_reads(const Epilogue &e, int64_t t, int c, bool on, uint4 (&x)[2][2])
{
    if constexpr (kAdd) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool in = on && t < e.T && c + 16 * i < e.N;
            const int64_t at = t * e.N + c + 16 * i;
            x[0][i] = in ? *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(e.g_add) + at) : make_uint4(0u, 0u, 0u, 0u);
            x[1][i] = in ? *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(e.u_add) + at) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
}
// 16 tokens x 32 columns, a column per lane, to 16 columns of token lane / 2;
// those of an even lane are put in front
__device__ __forceinline__ void turn16(float *own, const float (&col)[16], float (&row)[16])
{
    const int lane = threadIdx.x & 31, slot = (lane & 7) | (lane & 8) << 1 | (lane & 16) >> 1;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 16; ++j) own[j * 36 + slot] = col[j];
    __syncwarp();
    const float4 *p = reinterpret_cast<const float4 *>(own + (lane >> 1) * 36 + (lane & 1) * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 a = p[j];
        row[4 * j] = a.x, row[4 * j + 1] = a.y, row[4 * j + 2] = a.z, row[4 * j + 3] = a.w;
    }
}
__device__ __forceinline__ void keep8(uint8_t *codes, uint8_t *scales, int64_t pitch, int64_t T, int64_t t, int c, bool on,
                                      const float (&v)[16])
{
    float m = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) m = max_nan(m, fabsf(v[i]));
    uint32_t bits = __float_as_uint(m) & 0x7FFFFFFFu;
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, bits, 1);
    bits = other > bits ? other : bits;
    const uint32_t byte = scale_byte8(bits);
    const float inv = inv_scale(byte);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = e4m3x4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
        if (byte == 255u) w[i] = 0u;
    }
    // the lanes swap halves: sixteen neighbouring codes each
    const bool odd = (threadIdx.x & 1) != 0;
    const uint32_t a = __shfl_xor_sync(0xFFFFFFFFu, odd ? w[0] : w[2], 1), b = __shfl_xor_sync(0xFFFFFFFFu, odd ? w[1] : w[3], 1);
    const uint4 all = odd ? make_uint4(a, b, w[2], w[3]) : make_uint4(w[0], w[1], a, b);
    if (!on || (c & ~31) >= pitch) return;
    *reinterpret_cast<uint4 *>(codes + t * pitch + (c & ~31) + (odd ? 16 : 0)) = all;
    if (!odd) scales[static_cast<int64_t>(c / kBlock) * T + t] = static_cast<uint8_t>(byte);
}
// The lane's columns of both products, turned, plus what was read for them.
template <bool kAdd>
__device__ __forceinline__ void gated_turn(float *own, const float (&v)[2][16], const uint4 (&x)[2][2], float (&r)[2][16])
{
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        turn16(own, v[m], r[m]);
        if (kAdd) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t a[4] = {x[m][i].x, x[m][i].y, x[m][i].z, x[m][i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    r[m][8 * i + 2 * j] += __uint_as_float(a[j] << 16);
                    r[m][8 * i + 2 * j + 1] += __uint_as_float(a[j] & 0xFFFF0000u);
                }
            }
        }
    }
}
template <bool kSave, int kAct>
__device__ __forceinline__ void gated_finish(const Epilogue &e, int64_t t, int c, float (&r)[2][16])
{
    const bool on = t < e.T;
    if (kSave) {
        if (c + 24 > e.N) {   // rows past the last may have given anything, a NaN too
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c + j + (j & 8) >= e.N) r[0][j] = r[1][j] = 0.0f;
        }
        keep8(e.g8, e.gs, e.pitch8, e.T, t, c, on, r[0]);
        keep8(e.u8, e.us, e.pitch8, e.T, t, c, on, r[1]);
    }
    if (!on) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = gate_value<false>(kAct, r[0][8 * i + j]) * r[1][8 * i + j];
        store8(e.y, DBF_BF16, t * e.N, c + 16 * i, e.N, true, h);
    }
}

// Rows that are no whole 16-byte vectors, where more is read or kept: everything
// but the 8-bit copies, whose rows are, stays a column to a lane. Eight values to a
// lane would be as many accesses of single values, each over eight rows instead of
// one (2 x (209 -> 10325) at 3484 tokens with addends: 521 us, 160 us so).
template <int kMats, int kAct>
__device__ __forceinline__ void column_finish(const Epilogue &e, float *own, int64_t t0, int n0, float (&v)[kMats][16])
{
    const int lane = threadIdx.x & 31, n = n0 + lane;
    if (kMats == 2) {
        if (e.g_add || e.u_add) {
            uint32_t a[2][16];
            read_column(e.g_add, e.add_dt, e, t0, n, a[0]);
            read_column(e.u_add, e.add_dt, e, t0, n, a[1]);
            add_column(a[0], e.add_dt, v[0]);
            add_column(a[1], e.add_dt, v[kMats - 1]);
        }
        if (e.g8) {
#pragma unroll
            for (int m = 0; m < kMats; ++m) {
                float r[16];
                if (n >= e.N) {   // rows past the last may have given anything, a NaN too
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[m][j] = 0.0f;
                }
                turn16(own, v[m], r);
                const int64_t t = t0 + (lane >> 1);
                keep8(m ? e.u8 : e.g8, m ? e.us : e.gs, e.pitch8, e.T, t, n0 + (lane & 1) * 8, t < e.T, r);
            }
        }
    } else if (e.accumulate) {
        uint32_t a[16];
        read_column(e.y, e.yd, e, t0, n, a);
        add_column(a, e.yd, v[0]);
    }
    store_column<kMats, kAct>(e, t0, n, v);
}

// The workspace of a product: x's codes, and its scales in whole tiles of 128
// rows, one at most per 16 tokens however the tokens are cut into tiles. It
// grows with T, so one made for the largest T serves every call.
inline size_t x_codes_at() { return kWsHeaderBytes; }
inline size_t x_scales_at(int64_t M, int64_t T) { return align_up(x_codes_at() + static_cast<size_t>(T * code_pitch(M)), 256); }
inline size_t product_workspace_bytes(int64_t M, int64_t T)
{
    return x_scales_at(M, T) + static_cast<size_t>((T + 15) / 16 * scale_tiles(M) * 512);
}

// The scale row of token t: each tile of w tokens starts a new one of 128 (pad:
// the scale rows of a tile). The row passes 2^31 where t does not (w < pad).
__host__ __device__ inline int64_t x_scale_row(int t, int w, int pad) { return static_cast<int64_t>(t / w) * pad + t % w; }

// One call: a weight (plain) or two of one shape (gated), and its tokens.
struct Product {
    int64_t M, N, T;
    int mats;                              // 1 plain, 2 gated
    const uint8_t *codes[2], *scales[2];   // as dbf_mx4_layer
    const void *x;
    dbf_dtype xd;
    Epilogue ep;
    int flags;
    void *ws;
};

// A backward call: dx = [acc] dx + dy W, or with two weights + the second's.
struct Gradient {
    int64_t M, N, T;
    const uint8_t *codes[2], *scales[2];   // codes[1] null: one weight
    const void *dy;                        // gated: dh
    dbf_dtype dyd;
    void *dx;
    dbf_dtype dxd;
    int flags;
    void *ws;
};

}  // namespace mx
}  // namespace dbf
