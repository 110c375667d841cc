// Host entry points of the 4-bit base layer, its gated block and the 8-bit
// activations: argument checks (no launch on a failed check) and path choice.
#include <algorithm>

#include "dbf_mx_layer.cuh"

namespace {

using namespace dbf;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
dbf_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DBF_OK : DBF_ERR_CUDA; }
bool act_dtype_ok(dbf_dtype d) { return d == DBF_F32 || d == DBF_BF16; }
bool float_dtype_ok(dbf_dtype d) { return d == DBF_F32 || d == DBF_BF16 || d == DBF_F16; }
uintptr_t size_of(dbf_dtype d) { return d == DBF_F32 ? 4 : 2; }

dbf_status check_matrix(const void *values, dbf_dtype d, const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t k,
                        const int32_t *status)
{
    if (rows <= 0 || k <= 0 || !values || !codes || !scales || !float_dtype_ok(d)) return DBF_ERR_INVALID_ARG;
    if (!mx_size_ok(rows, k)) return DBF_ERR_UNSUPPORTED;
    if (!aligned(values, size_of(d)) || !aligned(codes, 16) || !aligned(scales, 16) || (status && !aligned(status, 4)))
        return DBF_ERR_ALIGNMENT;
    return DBF_OK;
}

bool layer_shape_ok(const dbf_mx4_layer *L) { return L && L->M > 0 && L->N > 0; }
// tiles of at least 16 tokens and 256 rows are counted in 32 bits, and rows
// past the last one of a tile still have 32-bit numbers
constexpr int64_t kMost = (int64_t{1} << 31) - 4096;
bool tokens_ok(const dbf_mx4_layer *L, int64_t T)
{
    return T >= 0 && T < kMost && L->N < kMost && (int64_t{L->N} + 255) / 256 * ((T + 15) / 16) < (int64_t{1} << 31) &&
           mx_size_ok(L->N, L->M);
}

// the gradient's rows, three pieces of each, are counted in 32 bits; its
// columns, rows of W, are 65535 * 256 at most
bool gradient_ok(const dbf_mx4_layer *L, int64_t T)
{
    return T >= 0 && 3 * T < kMost && (int64_t{L->M} + 255) / 256 * ((T + 31) / 32) < (int64_t{1} << 31) &&
           mx_size_ok(L->N, L->M) && L->N <= 65535 * 256;
}

dbf_status check_layer(const dbf_mx4_layer *L)
{
    if (!L->codes || !L->scales) return DBF_ERR_INVALID_ARG;
    return aligned(L->codes, 16) && aligned(L->scales, 16) ? DBF_OK : DBF_ERR_ALIGNMENT;
}

size_t product_workspace(const dbf_mx4_layer *L, int64_t T)
{
    return layer_shape_ok(L) && tokens_ok(L, T) ? mx::product_workspace_bytes(L->M, T) : 0;
}

// Whether two T x cols matrices share memory: tiles of an output are written while
// other tiles' inputs are still read.
struct Span {
    const void *p;
    int64_t bytes;
};
Span span(const void *p, dbf_dtype d, int64_t T, int64_t cols) { return {p, T * cols * static_cast<int64_t>(size_of(d))}; }
bool meet(const Span &a, const Span &b)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}
// Whether one of the first 'outs' of them shares memory with any other
template <size_t n>
bool any_meet(const Span (&s)[n], size_t outs)
{
    for (size_t i = 0; i < outs; ++i)
        for (size_t j = i + 1; j < n; ++j)
            if (meet(s[i], s[j])) return true;
    return false;
}

dbf_status run(const mx::Product &c, size_t need, size_t ws_bytes, cudaStream_t s)
{
    if (!c.ws || ws_bytes < need) return DBF_ERR_WORKSPACE;
    if (!aligned(c.ws, 256)) return DBF_ERR_ALIGNMENT;
    const Span x = span(c.x, c.xd, c.T, c.M), y = span(c.ep.y, c.ep.yd, c.T, c.N);
    const int64_t codes = c.T * c.ep.pitch8, scales = c.T * mx::blocks(c.N);
    const Span all[] = {y, {c.ep.g8, codes}, {c.ep.gs, scales}, {c.ep.u8, codes}, {c.ep.us, scales}, x};
    if (any_meet(all, 5)) return DBF_ERR_INVALID_ARG;
    return from_cuda(mx_decode_fits(c.M, c.N, c.T, c.mats) ? mx_decode(c, s) : mx_gemm(c, s));
}

bool same_shape(const dbf_mx4_layer *a, const dbf_mx4_layer *b)
{
    return layer_shape_ok(a) && layer_shape_ok(b) && a->M == b->M && a->N == b->N;
}

}  // namespace

extern "C" {

size_t dbf_mx4_code_bytes(int64_t rows, int64_t k)
{
    return rows > 0 && k > 0 ? static_cast<size_t>(rows * mx::code_pitch(k)) : 0;
}

size_t dbf_mx4_scale_bytes(int64_t rows, int64_t k)
{
    return rows > 0 && k > 0 ? static_cast<size_t>((rows + 127) / 128 * mx::scale_tiles(k) * 512) : 0;
}

dbf_status dbf_mx4_quantize(const void *src, dbf_dtype src_dtype, int64_t rows, int64_t k, uint8_t *codes, size_t codes_bytes,
                            uint8_t *scales, size_t scales_bytes, int32_t *status_dev, void *stream)
{
    const dbf_status st = check_matrix(src, src_dtype, codes, scales, rows, k, status_dev);
    if (st != DBF_OK) return st;
    if (codes_bytes < dbf_mx4_code_bytes(rows, k) || scales_bytes < dbf_mx4_scale_bytes(rows, k)) return DBF_ERR_INVALID_ARG;
    return from_cuda(launch_quantize4(src, src_dtype, rows, k, codes, scales, status_dev, static_cast<cudaStream_t>(stream)));
}

dbf_status dbf_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t k, void *dst,
                              dbf_dtype dst_dtype, void *stream)
{
    const dbf_status st = check_matrix(dst, dst_dtype, codes, scales, rows, k, nullptr);
    if (st != DBF_OK) return st;
    return from_cuda(launch_dequantize4(codes, scales, rows, k, dst, dst_dtype, static_cast<cudaStream_t>(stream)));
}

size_t dbf_act8_code_bytes(int64_t rows, int64_t cols)
{
    return rows > 0 && cols > 0 ? static_cast<size_t>(rows * mx::blocks(cols) * mx::kBlock) : 0;
}

size_t dbf_act8_scale_bytes(int64_t rows, int64_t cols)
{
    return rows > 0 && cols > 0 ? static_cast<size_t>(rows * mx::blocks(cols)) : 0;
}

dbf_status dbf_act8_save(const void *src, dbf_dtype src_dtype, int64_t rows, int64_t cols, const dbf_act8 *dst,
                         int32_t *status_dev, void *stream)
{
    if (!dst) return DBF_ERR_INVALID_ARG;
    if (rows == 0 && cols > 0) return DBF_OK;
    const dbf_status st = check_matrix(src, src_dtype, dst->codes, dst->scales, rows, cols, status_dev);
    if (st != DBF_OK) return st;
    return from_cuda(
        launch_act8_save(src, src_dtype, rows, cols, dst->codes, dst->scales, status_dev, static_cast<cudaStream_t>(stream)));
}

dbf_status dbf_act8_load(const dbf_act8 *src, int64_t rows, int64_t cols, void *dst, dbf_dtype dst_dtype, void *stream)
{
    if (!src) return DBF_ERR_INVALID_ARG;
    if (rows == 0 && cols > 0) return DBF_OK;
    const dbf_status st = check_matrix(dst, dst_dtype, src->codes, src->scales, rows, cols, nullptr);
    if (st != DBF_OK) return st;
    return from_cuda(launch_act8_load(src->codes, src->scales, rows, cols, dst, dst_dtype, static_cast<cudaStream_t>(stream)));
}

size_t dbf_mx4_workspace_bytes(const dbf_mx4_layer *L, int64_t T) { return product_workspace(L, T); }

dbf_status dbf_mx4_forward(const dbf_mx4_layer *L, const void *x, dbf_dtype x_dtype, void *y, dbf_dtype y_dtype, int64_t T,
                           int flags, void *ws, size_t ws_bytes, void *stream)
{
    if (!layer_shape_ok(L) || T < 0 || !act_dtype_ok(x_dtype) || !act_dtype_ok(y_dtype) ||
        (flags & ~(DBF_ACCUMULATE | DBF_WEIGHTS_STATIC)))
        return DBF_ERR_INVALID_ARG;
    if (!tokens_ok(L, T)) return DBF_ERR_UNSUPPORTED;
    if (T == 0) return DBF_OK;
    if (!x || !y) return DBF_ERR_INVALID_ARG;
    const dbf_status st = check_layer(L);
    if (st != DBF_OK) return st;
    if (!aligned(x, 16) || !aligned(y, 16)) return DBF_ERR_ALIGNMENT;
    mx::Product c = {};
    c.M = L->M, c.N = L->N, c.T = T, c.mats = 1;
    c.codes[0] = L->codes, c.scales[0] = L->scales;
    c.x = x, c.xd = x_dtype;
    c.ep.y = y, c.ep.yd = y_dtype, c.ep.accumulate = flags & DBF_ACCUMULATE ? 1 : 0;
    c.ep.N = L->N, c.ep.T = T;
    c.flags = flags, c.ws = ws;
    return run(c, product_workspace(L, T), ws_bytes, static_cast<cudaStream_t>(stream));
}

size_t dbf_mx4_gated_workspace_bytes(const dbf_mx4_layer *gate, const dbf_mx4_layer *up, int64_t T)
{
    return same_shape(gate, up) ? product_workspace(gate, T) : 0;
}

dbf_status dbf_mx4_gated_forward(const dbf_mx4_layer *gate, const dbf_mx4_layer *up, dbf_gate act, const void *x,
                                 dbf_dtype x_dtype, const void *g_add, const void *u_add, dbf_dtype add_dtype, void *h,
                                 dbf_dtype h_dtype, const dbf_act8 *save_g, const dbf_act8 *save_u, int64_t T, int flags,
                                 void *ws, size_t ws_bytes, void *stream)
{
    if (!same_shape(gate, up) || T < 0 || (act != DBF_GATE_SILU && act != DBF_GATE_GELU) || !act_dtype_ok(x_dtype) ||
        !act_dtype_ok(h_dtype) || ((g_add || u_add) && !act_dtype_ok(add_dtype)) || !save_g != !save_u ||
        (flags & ~DBF_WEIGHTS_STATIC))
        return DBF_ERR_INVALID_ARG;
    if (!tokens_ok(gate, T)) return DBF_ERR_UNSUPPORTED;
    if (T == 0) return DBF_OK;
    if (!x || !h || (save_g && (!save_g->codes || !save_g->scales || !save_u->codes || !save_u->scales)))
        return DBF_ERR_INVALID_ARG;
    dbf_status st = check_layer(gate);
    if (st == DBF_OK) st = check_layer(up);
    if (st != DBF_OK) return st;
    if (!aligned(x, 16) || !aligned(h, 16) || !aligned(g_add, 16) || !aligned(u_add, 16) ||
        (save_g && (!aligned(save_g->codes, 16) || !aligned(save_g->scales, 16) || !aligned(save_u->codes, 16) ||
                    !aligned(save_u->scales, 16))))
        return DBF_ERR_ALIGNMENT;
    mx::Product c = {};
    c.M = gate->M, c.N = gate->N, c.T = T, c.mats = 2;
    c.codes[0] = gate->codes, c.scales[0] = gate->scales;
    c.codes[1] = up->codes, c.scales[1] = up->scales;
    c.x = x, c.xd = x_dtype;
    c.ep.y = h, c.ep.yd = h_dtype, c.ep.act = act;
    c.ep.g_add = g_add, c.ep.u_add = u_add, c.ep.add_dt = add_dtype;
    if (save_g) {
        c.ep.g8 = save_g->codes, c.ep.gs = save_g->scales;
        c.ep.u8 = save_u->codes, c.ep.us = save_u->scales;
    }
    c.ep.pitch8 = mx::blocks(gate->N) * mx::kBlock;
    c.ep.N = gate->N, c.ep.T = T;
    c.flags = flags, c.ws = ws;
    return run(c, product_workspace(gate, T), ws_bytes, static_cast<cudaStream_t>(stream));
}

size_t dbf_mx4_backward_workspace_bytes(const dbf_mx4_layer *L, int64_t T, dbf_dtype dy_dtype)
{
    if (!layer_shape_ok(L) || !gradient_ok(L, T) || !act_dtype_ok(dy_dtype)) return 0;
    return mx_back_workspace_bytes(L->M, L->N, T, dy_dtype, 1);
}

dbf_status dbf_mx4_backward(const dbf_mx4_layer *L, const void *dy, dbf_dtype dy_dtype, void *dx, dbf_dtype dx_dtype, int64_t T,
                            int flags, void *ws, size_t ws_bytes, void *stream)
{
    if (!layer_shape_ok(L) || T < 0 || !act_dtype_ok(dy_dtype) || !act_dtype_ok(dx_dtype) ||
        (flags & ~(DBF_ACCUMULATE | DBF_WEIGHTS_STATIC)))
        return DBF_ERR_INVALID_ARG;
    if (!gradient_ok(L, T)) return DBF_ERR_UNSUPPORTED;
    if (T == 0) return DBF_OK;
    if (!dy || !dx) return DBF_ERR_INVALID_ARG;
    const dbf_status st = check_layer(L);
    if (st != DBF_OK) return st;
    if (!aligned(dy, 16) || !aligned(dx, 16)) return DBF_ERR_ALIGNMENT;
    if (!ws || ws_bytes < mx_back_workspace_bytes(L->M, L->N, T, dy_dtype, 1)) return DBF_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return DBF_ERR_ALIGNMENT;
    if (meet(span(dy, dy_dtype, T, L->N), span(dx, dx_dtype, T, L->M))) return DBF_ERR_INVALID_ARG;
    mx::Gradient c = {};
    c.M = L->M, c.N = L->N, c.T = T;
    c.codes[0] = L->codes, c.scales[0] = L->scales;
    c.dy = dy, c.dyd = dy_dtype, c.dx = dx, c.dxd = dx_dtype;
    c.flags = flags, c.ws = ws;
    return from_cuda(mx_backward(c, static_cast<cudaStream_t>(stream)));
}

size_t dbf_mx4_gated_backward_workspace_bytes(const dbf_mx4_layer *gate, const dbf_mx4_layer *up, int64_t T, dbf_dtype dh_dtype)
{
    if (!same_shape(gate, up) || !gradient_ok(gate, T) || !act_dtype_ok(dh_dtype)) return 0;
    return mx_back_workspace_bytes(gate->M, gate->N, T, dh_dtype, 2);
}

dbf_status dbf_mx4_gated_backward(const dbf_mx4_layer *gate, const dbf_mx4_layer *up, dbf_gate act, const dbf_act8 *saved_g,
                                  const dbf_act8 *saved_u, const void *dh, dbf_dtype dh_dtype, void *dg, void *du, void *dx,
                                  dbf_dtype dx_dtype, int64_t T, int flags, void *ws, size_t ws_bytes, void *stream)
{
    if (!same_shape(gate, up) || T < 0 || (act != DBF_GATE_SILU && act != DBF_GATE_GELU) || !act_dtype_ok(dh_dtype) ||
        (dx && !act_dtype_ok(dx_dtype)) || (flags & ~(DBF_ACCUMULATE | DBF_WEIGHTS_STATIC)))
        return DBF_ERR_INVALID_ARG;
    if (!gradient_ok(gate, T)) return DBF_ERR_UNSUPPORTED;
    if (T == 0) return DBF_OK;
    if (!saved_g || !saved_u || !saved_g->codes || !saved_g->scales || !saved_u->codes || !saved_u->scales || !dh || !dg || !du)
        return DBF_ERR_INVALID_ARG;
    if (!aligned(saved_g->codes, 16) || !aligned(saved_g->scales, 16) || !aligned(saved_u->codes, 16) ||
        !aligned(saved_u->scales, 16) || !aligned(dh, 16) || !aligned(dg, 16) || !aligned(du, 16) || !aligned(dx, 16))
        return DBF_ERR_ALIGNMENT;
    mx::Gradient c = {};
    c.M = gate->M, c.N = gate->N, c.T = T;
    c.dy = dh, c.dyd = dh_dtype, c.dx = dx, c.dxd = dx_dtype;
    c.flags = flags;
    if (dx) {
        dbf_status st = check_layer(gate);
        if (st == DBF_OK) st = check_layer(up);
        if (st != DBF_OK) return st;
        if (!ws || ws_bytes < mx_back_workspace_bytes(gate->M, gate->N, T, dh_dtype, 2)) return DBF_ERR_WORKSPACE;
        if (!aligned(ws, 256)) return DBF_ERR_ALIGNMENT;
        c.codes[0] = gate->codes, c.scales[0] = gate->scales;
        c.codes[1] = up->codes, c.scales[1] = up->scales;
        c.ws = ws;
    }
    // dx may lie over dh: the launch that reads dh ends before one writes dx
    const Span g = span(dg, dh_dtype, T, gate->N), u = span(du, dh_dtype, T, gate->N);
    const Span by_gate[] = {g, u, span(dh, dh_dtype, T, gate->N)}, by_product[] = {g, u, span(dx, dx_dtype, T, gate->M)};
    if (any_meet(by_gate, 2) || any_meet(by_product, 2)) return DBF_ERR_INVALID_ARG;
    return from_cuda(mx_gated_backward(c, act, *saved_g, *saved_u, dg, du, static_cast<cudaStream_t>(stream)));
}

dbf_status dbf_debug_mx4_cut(dbf_mx4_call call, int32_t M, int32_t N, int64_t T, dbf_dtype dy_dtype, int32_t sms, int64_t *cut)
{
    dbf_mx4_layer L = {};
    L.M = M, L.N = N;
    const bool back = call == DBF_MX4_BACKWARD || call == DBF_MX4_GATED_BACKWARD;
    if (call < DBF_MX4_FORWARD || call > DBF_MX4_GATED_BACKWARD || !layer_shape_ok(&L) || T < 1 || sms < 1 || !cut ||
        (back && !act_dtype_ok(dy_dtype)))
        return DBF_ERR_INVALID_ARG;
    if (back ? !gradient_ok(&L, T) : !tokens_ok(&L, T)) return DBF_ERR_UNSUPPORTED;
    int64_t of[8];
    if (back) {
        mx::Gradient c = {};
        c.M = M, c.N = N, c.T = T, c.dyd = dy_dtype;
        mx_back_cut(c, call == DBF_MX4_GATED_BACKWARD ? 2 : 1, sms, of);
    } else {
        // only whether there are addends and copies is looked at
        uint8_t there = 0;
        mx::Product c = {};
        c.M = M, c.N = N, c.T = T, c.mats = call == DBF_MX4_FORWARD ? 1 : 2;
        c.ep.g_add = c.ep.u_add = call == DBF_MX4_GATED_ADD ? &there : nullptr;
        c.ep.g8 = call == DBF_MX4_GATED_SAVE ? &there : nullptr;
        if (!mx_decode_cut(c, sms, of)) mx_gemm_cut(c, sms, of);
    }
    std::copy(of, of + 8, cut);
    return DBF_OK;
}

}  // extern "C"
