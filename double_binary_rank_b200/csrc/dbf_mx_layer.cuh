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

// One value per lane: 32 consecutive columns n of token t (a block of the
// 8-bit format), so the warp finds the block's scale and keeps the codes.
// Every lane calls it; columns at or past N hold 0.
__device__ __forceinline__ void keep8(uint8_t *codes, uint8_t *scales, int64_t pitch, int64_t T, int64_t t, int n, float v)
{
    const uint32_t byte = scale_byte8(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu));
    const uint32_t w = byte == 255u ? 0u : e4m3x4(v * inv_scale(byte), 0.0f, 0.0f, 0.0f);
    if (n < pitch) codes[t * pitch + n] = static_cast<uint8_t>(w);
    if ((threadIdx.x & 31) == 0 && n < pitch) scales[static_cast<int64_t>(n / kBlock) * T + t] = static_cast<uint8_t>(byte);
}

// Epilogue of one token t and, in each lane, one column n (32 consecutive
// columns a warp, the first a multiple of 32). Every lane calls it.
__device__ __forceinline__ void finish_plain(const Epilogue &e, int64_t t, int n, float v)
{
    if (n >= e.N) return;
    const int64_t at = t * e.N + n;
    if (e.accumulate) v += load_act(e.y, e.yd, at);
    store_act(e.y, e.yd, at, v);
}
__device__ __forceinline__ void finish_gated(const Epilogue &e, int64_t t, int n, float g, float u)
{
    const bool in = n < e.N;
    const int64_t at = t * e.N + n;
    if (in && e.g_add) g += load_act(e.g_add, e.add_dt, at);
    if (in && e.u_add) u += load_act(e.u_add, e.add_dt, at);
    if (e.g8) {   // the same in every lane
        keep8(e.g8, e.gs, e.pitch8, e.T, t, n, in ? g : 0.0f);
        keep8(e.u8, e.us, e.pitch8, e.T, t, n, in ? u : 0.0f);
    }
    if (in) store_act(e.y, e.yd, at, gate_value(e.act, g) * u);
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

}  // namespace mx
}  // namespace dbf
