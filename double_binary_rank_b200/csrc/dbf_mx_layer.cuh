// What the 4-bit layer's product kernels share: their epilogue (plain and
// gated) and the host-side description of a call.
#pragma once

#include "dbf_mx.cuh"

namespace dbf {
namespace mx {

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
// infinity and its reciprocal is 0, as the limit is; both approximations are
// off by an ulp or two of fp32.
constexpr float kGelu2c = 1.5957691216057308f, kGeluCube = 0.044715f;
__device__ __forceinline__ float sigmoid(float g)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-g)));
    return r;
}
__device__ __forceinline__ float gate_value(int act, float g)
{
    return g * sigmoid(act == DBF_GATE_SILU ? g : kGelu2c * (g + kGeluCube * g * g * g));
}
__device__ __forceinline__ float gate_slope(int act, float g, float &value)
{
    if (act == DBF_GATE_SILU) {
        const float s = sigmoid(g);
        value = g * s;
        return s * (1.0f + g * (1.0f - s));
    }
    const float s = sigmoid(kGelu2c * (g + kGeluCube * g * g * g));
    const float d = s * (1.0f - s);
    value = g * s;
    return d == 0.0f ? s : s + g * d * kGelu2c * (1.0f + 3.0f * kGeluCube * g * g);   // d == 0: g * g may be infinite
}

// The epilogues below take, in each lane, one column n (32 consecutive columns
// a warp, the first a multiple of 32) of kTok consecutive tokens from t0, of
// which 'count' exist. Every lane of the warp calls them. All reads are issued
// before the first result is formed, and no lane's control flow differs up to
// its stores.
template <int kTok>
__device__ __forceinline__ void add_columns(const void *p, dbf_dtype dt, int64_t N, int64_t t0, int count, int n, float (&v)[kTok])
{
    float a[kTok];
#pragma unroll
    for (int j = 0; j < kTok; ++j) a[j] = n < N && j < count ? load_act(p, dt, (t0 + j) * N + n) : 0.0f;
#pragma unroll
    for (int j = 0; j < kTok; ++j) v[j] += a[j];
}

// bf16 rows of even length: neighbouring lanes swap one of two tokens, so that
// a lane stores two columns of one token as one word (half the store
// instructions).
template <int kTok>
__device__ __forceinline__ void store_columns(void *p, dbf_dtype dt, int64_t N, int64_t t0, int count, int n, const float (&v)[kTok])
{
    const bool in = n < N;
    if (dt == DBF_F32) {
        float *y = static_cast<float *>(p) + t0 * N + n;
#pragma unroll
        for (int j = 0; j < kTok; ++j)
            if (in && j < count) y[j * N] = v[j];
        return;
    }
    if (kTok % 2 == 0 && (N & 1) == 0) {
        const int odd = threadIdx.x & 1;
        // token j + odd, columns n - odd and n - odd + 1
        uint32_t *y = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p) + (t0 + odd) * N + (n - odd));
#pragma unroll
        for (int j = 0; j < kTok; j += 2) {
            const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[j] : v[j + 1], 1);
            const __nv_bfloat162 w = odd ? __floats2bfloat162_rn(got, v[j + 1]) : __floats2bfloat162_rn(v[j], got);
            if (in && j + odd < count) y[j * (N / 2)] = *reinterpret_cast<const uint32_t *>(&w);
        }
        return;
    }
    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p) + t0 * N + n;
#pragma unroll
    for (int j = 0; j < kTok; ++j)
        if (in && j < count) y[j * N] = __float2bfloat16_rn(v[j]);
}

// Keep the warp's 32 columns, a block of the 8-bit format, of each token; the
// warp finds the largest magnitude together (as an integer: NaN above
// infinity above all else). Columns at or past N hold 0.
template <int kTok>
__device__ __forceinline__ void keep8(uint8_t *codes, uint8_t *scales, int64_t pitch, int64_t T, int64_t t0, int count, int n,
                                      const float (&v)[kTok])
{
    static_assert(kTok <= 32, "lane j stores token j's scale");
    const int lane = threadIdx.x & 31;
    if (n - lane >= pitch) return;   // the warp's block does not exist
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
        const uint32_t byte = scale_byte8(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[j]) & 0x7FFFFFFFu));
        const uint32_t w = byte == 255u ? 0u : e4m3x4(v[j] * inv_scale(byte), 0.0f, 0.0f, 0.0f);
        if (j < count) codes[(t0 + j) * pitch + n] = static_cast<uint8_t>(w);
        if (lane == j) mine = byte;
    }
    if (lane < count && lane < kTok) scales[static_cast<int64_t>(n / kBlock) * T + t0 + lane] = static_cast<uint8_t>(mine);
}

template <int kTok>
__device__ __forceinline__ void finish_plain(const Epilogue &e, int64_t t0, int count, int n, float (&v)[kTok])
{
    if (e.accumulate) add_columns(e.y, e.yd, e.N, t0, count, n, v);
    store_columns(e.y, e.yd, e.N, t0, count, n, v);
}
template <int kTok>
__device__ __forceinline__ void finish_gated(const Epilogue &e, int64_t t0, int count, int n, float (&g)[kTok], float (&u)[kTok])
{
    if (e.g_add) add_columns(e.g_add, e.add_dt, e.N, t0, count, n, g);
    if (e.u_add) add_columns(e.u_add, e.add_dt, e.N, t0, count, n, u);
    if (e.g8) {
        if (n >= e.N) {
#pragma unroll
            for (int j = 0; j < kTok; ++j) g[j] = u[j] = 0.0f;
        }
        keep8(e.g8, e.gs, e.pitch8, e.T, t0, count, n, g);
        keep8(e.u8, e.us, e.pitch8, e.T, t0, count, n, u);
    }
#pragma unroll
    for (int j = 0; j < kTok; ++j) g[j] = gate_value(e.act, g[j]) * u[j];
    store_columns(e.y, e.yd, e.N, t0, count, n, g);
}

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
