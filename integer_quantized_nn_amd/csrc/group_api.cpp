// group_api.cpp -- the extern "C" entry points for codes with group scales: validation
// and dispatch to group_quant.hip, w4.hip and wgrad.hip.  Contracts are in include/iqnn.h.
#include <hip/hip_runtime.h>

#include "iqnn.h"
#include "iqnn_internal.h"

using namespace iqnn;

namespace {

constexpr int64_t kMaxCols = (int64_t)1 << 30, kMaxRows = (int64_t)1 << 40, kMaxElems = (int64_t)1 << 46;

bool ftype_ok(int32_t t) { return t == F_F32 || t == F_F16 || t == F_BF16; }
int64_t fsize(int32_t t) { return t == F_F32 ? 4 : 2; }
bool four_bit(int32_t t) { return t == T_INT4 || t == T_UINT4; }
bool asym(int32_t t) { return t == T_UINT8 || t == T_UINT4; }
bool group_ok(int32_t g) { return g == 0 || g == 32 || g == 64 || g == 128; }
int64_t groups_of(int64_t cols, int32_t g) { return g ? (cols + g - 1) / g : 1; }
// units of 8 elements per row, the last group's missing ones included
int32_t units_of(int64_t cols, int32_t g) { return (int32_t)(g ? groups_of(cols, g) * (g / 8) : (cols + 7) / 8); }
bool aligned(const void* p, int64_t a) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(a - 1)) == 0; }
bool rows_vec(const void* p, int64_t ld, int32_t t) { return aligned(p, 16) && ld * fsize(t) % 16 == 0; }

// rows x cols of a floating-point tensor with row stride ld, and its group.
iqnn_status check_view(const char* op, int32_t type, int64_t rows, int64_t cols, int64_t ld, int64_t width,
                       int32_t group) {
    if (!ftype_ok(type)) return fail(IQNN_ERR_INVALID_ARG, "%s: type %d is not a floating-point type", op, type);
    if (rows < 0 || cols <= 0)
        return fail(IQNN_ERR_INVALID_ARG, "%s: bad sizes (rows=%lld cols=%lld)", op, (long long)rows, (long long)cols);
    if (!group_ok(group)) return fail(IQNN_ERR_INVALID_ARG, "%s: group %d is not 0, 32, 64 or 128", op, group);
    if (cols > kMaxCols || rows > kMaxRows)
        return fail(IQNN_ERR_UNSUPPORTED, "%s: more than 2^30 columns or 2^40 rows", op);
    if (ld < width)
        return fail(IQNN_ERR_INVALID_ARG, "%s: row stride %lld below the row's %lld elements", op, (long long)ld,
                    (long long)width);
    if (rows > 0 && ld > kMaxElems / rows) return fail(IQNN_ERR_UNSUPPORTED, "%s: more than 2^46 elements", op);
    return IQNN_OK;
}

iqnn_status launched(const char* op, hipError_t e) {
    if (e == hipErrorInvalidValue) return fail(IQNN_ERR_UNSUPPORTED, "%s: more blocks than a launch can hold", op);
    if (e != hipSuccess) return fail(IQNN_ERR_HIP, "%s launch failed: %s", op, hipGetErrorString(e));
    return ok();
}

bool is_act(int32_t a) { return a >= A_RELU && a <= A_SILU; }

iqnn_status check_w4(const iqnn_w4_desc* d) {
    if (!d) return fail(IQNN_ERR_INVALID_ARG, "null descriptor");
    if (d->n <= 0 || d->k <= 0) return fail(IQNN_ERR_INVALID_ARG, "w4: sizes must be positive");
    if (d->n > kMaxCols || d->k > kMaxCols || d->n > kMaxElems / d->k)
        return fail(IQNN_ERR_UNSUPPORTED, "w4: n or k above 2^30, or n * k above 2^46");
    if (d->k % 2) return fail(IQNN_ERR_INVALID_ARG, "w4: 4-bit weights need an even k");
    if (!four_bit(d->w_type)) return fail(IQNN_ERR_INVALID_ARG, "w4: weight type %d is not INT4 or UINT4", d->w_type);
    if (!ftype_ok(d->x_type)) return fail(IQNN_ERR_INVALID_ARG, "w4: type %d is not a floating-point type", d->x_type);
    if (!group_ok(d->group)) return fail(IQNN_ERR_INVALID_ARG, "w4: group %d is not 0, 32, 64 or 128", d->group);
    return IQNN_OK;
}

iqnn_status check_wgrad(const iqnn_ckpt_wgrad_desc* d) {
    if (!d) return fail(IQNN_ERR_INVALID_ARG, "null descriptor");
    if (d->m < 0 || d->n <= 0 || d->k <= 0) return fail(IQNN_ERR_INVALID_ARG, "ckpt_wgrad: bad sizes");
    if (d->n > kMaxCols || d->k > kMaxCols || d->m > kMaxRows || d->n > kMaxElems / d->k ||
        (d->m > 0 && (d->n > kMaxElems / d->m || d->k > kMaxElems / d->m)))
        return fail(IQNN_ERR_UNSUPPORTED, "ckpt_wgrad: sizes above 2^30 (m 2^40) or tensors above 2^46 elements");
    if (!ftype_ok(d->dy_type)) return fail(IQNN_ERR_INVALID_ARG, "ckpt_wgrad: dy_type %d is not a floating-point type", d->dy_type);
    if (d->dw_type != d->dy_type && d->dw_type != F_F32)
        return fail(IQNN_ERR_INVALID_ARG, "ckpt_wgrad: dw_type %d is neither dy_type nor FLOAT32", d->dw_type);
    if (!group_ok(d->group)) return fail(IQNN_ERR_INVALID_ARG, "ckpt_wgrad: group %d is not 0, 32, 64 or 128", d->group);
    const WgradPlan w = wgrad_plan(d->m, d->n, d->k, d->dw_type == F_F32);
    if (w.n_tiles * w.k_tiles * w.splits > kWgradMaxBlocks)
        return fail(IQNN_ERR_UNSUPPORTED, "ckpt_wgrad: more blocks than a launch can hold");
    return IQNN_OK;
}

}  // namespace

extern "C" {

iqnn_status iqnn_quantize_groups(const void* x_dev, int32_t x_type, int64_t rows, int64_t cols, int64_t ldx,
                                 int32_t group, void* q_dev, int32_t qtype, float* scale_dev, int32_t* zp_dev,
                                 void* stream) {
    const char* op = "quantize_groups";
    const iqnn_status s = check_view(op, x_type, rows, cols, ldx, cols, group);
    if (s != IQNN_OK) return s;
    if (qtype < T_INT8 || qtype > T_UINT4) return fail(IQNN_ERR_INVALID_ARG, "%s: type %d is not a code type", op, qtype);
    if (four_bit(qtype) && cols % 2) return fail(IQNN_ERR_INVALID_ARG, "%s: 4-bit codes need an even cols", op);
    if (rows == 0) return ok();
    if (!x_dev || !q_dev || !scale_dev || (asym(qtype) && !zp_dev)) return fail(IQNN_ERR_INVALID_ARG, "%s: null pointer", op);
    if (!aligned(x_dev, fsize(x_type)) || !aligned(scale_dev, 4) || (asym(qtype) && !aligned(zp_dev, 4)))
        return fail(IQNN_ERR_ALIGNMENT, "%s: misaligned pointer", op);
    const bool vec = cols % 8 == 0 && rows_vec(x_dev, ldx, x_type) && aligned(q_dev, 8);
    const GroupQuantParams p{x_dev, static_cast<uint8_t*>(q_dev), scale_dev, zp_dev, rows, cols, ldx,
                             groups_of(cols, group), group, units_of(cols, group), x_type, qtype, vec};
    return launched(op, launch_quantize_groups(p, static_cast<hipStream_t>(stream)));
}

iqnn_status iqnn_dequantize_groups(const void* q_dev, int32_t qtype, int64_t rows, int64_t cols, int32_t group,
                                   const float* scale_dev, const int32_t* zp_dev, void* x_dev, int32_t x_type,
                                   int64_t ldx, void* stream) {
    const char* op = "dequantize_groups";
    const iqnn_status s = check_view(op, x_type, rows, cols, ldx, cols, group);
    if (s != IQNN_OK) return s;
    if (qtype < T_INT8 || qtype > T_UINT4) return fail(IQNN_ERR_INVALID_ARG, "%s: type %d is not a code type", op, qtype);
    if (four_bit(qtype) && cols % 2) return fail(IQNN_ERR_INVALID_ARG, "%s: 4-bit codes need an even cols", op);
    if (rows == 0) return ok();
    if (!x_dev || !q_dev || !scale_dev || (asym(qtype) && !zp_dev)) return fail(IQNN_ERR_INVALID_ARG, "%s: null pointer", op);
    if (!aligned(x_dev, fsize(x_type)) || !aligned(scale_dev, 4) || (asym(qtype) && !aligned(zp_dev, 4)))
        return fail(IQNN_ERR_ALIGNMENT, "%s: misaligned pointer", op);
    const bool vec = cols % 8 == 0 && rows_vec(x_dev, ldx, x_type) && aligned(q_dev, 8);
    const GroupDequantParams p{static_cast<const uint8_t*>(q_dev), x_dev, scale_dev, zp_dev, rows, cols, ldx,
                               groups_of(cols, group), group, units_of(cols, group), x_type, qtype, vec};
    return launched(op, launch_dequantize_groups(p, static_cast<hipStream_t>(stream)));
}

size_t iqnn_w4_packed_size(const iqnn_w4_desc* desc) {
    if (check_w4(desc) != IQNN_OK) return 0;
    ok();
    return (size_t)w4_geom(desc->n, desc->k, desc->group, desc->w_type == T_UINT4).bytes;
}

iqnn_status iqnn_w4_prepack(const iqnn_w4_desc* desc, const void* q_dev, const float* scale_dev,
                            const int32_t* zp_dev, void* packed_dev, size_t packed_bytes, void* stream) {
    const iqnn_status s = check_w4(desc);
    if (s != IQNN_OK) return s;
    const bool zp = desc->w_type == T_UINT4;
    const W4Geom g = w4_geom(desc->n, desc->k, desc->group, zp);
    if (!q_dev || !scale_dev || !packed_dev || (zp && !zp_dev)) return fail(IQNN_ERR_INVALID_ARG, "w4_prepack: null pointer");
    if (packed_bytes < (size_t)g.bytes)
        return fail(IQNN_ERR_INVALID_ARG, "w4_prepack: packed buffer of %zu bytes, %lld needed", packed_bytes, (long long)g.bytes);
    if (!aligned(packed_dev, 256) || !aligned(scale_dev, 4) || (zp && !aligned(zp_dev, 4)))
        return fail(IQNN_ERR_ALIGNMENT, "w4_prepack: misaligned pointer");
    const W4PrepackParams p{static_cast<const uint8_t*>(q_dev), scale_dev, zp ? zp_dev : nullptr,
                            static_cast<uint8_t*>(packed_dev), g, desc->n, desc->k, desc->group, desc->x_type};
    return launched("w4_prepack", launch_w4_prepack(p, static_cast<hipStream_t>(stream)));
}

iqnn_status iqnn_w4_fwd(const iqnn_w4_desc* desc, int64_t m, const void* x_dev, int64_t ldx, const void* packed_dev,
                        const void* bias_dev, void* y_dev, int64_t ldy, void* stream) {
    iqnn_status s = check_w4(desc);
    if (s != IQNN_OK) return s;
    s = check_view("w4_fwd x", desc->x_type, m, desc->k, ldx, desc->k, desc->group);
    if (s != IQNN_OK) return s;
    s = check_view("w4_fwd y", desc->x_type, m, desc->n, ldy, desc->n, desc->group);
    if (s != IQNN_OK) return s;
    if (m == 0) return ok();
    if (!x_dev || !packed_dev || !y_dev) return fail(IQNN_ERR_INVALID_ARG, "w4_fwd: null pointer");
    const int64_t e = fsize(desc->x_type);
    if (!aligned(x_dev, e) || !aligned(y_dev, e) || !aligned(packed_dev, 256) || (bias_dev && !aligned(bias_dev, e)))
        return fail(IQNN_ERR_ALIGNMENT, "w4_fwd: misaligned pointer");
    const bool zp = desc->w_type == T_UINT4;
    const W4Params p{x_dev, static_cast<const uint8_t*>(packed_dev), bias_dev, y_dev,
                     w4_geom(desc->n, desc->k, desc->group, zp), m, desc->n, desc->k, ldx, ldy,
                     desc->k % 8 == 0 && rows_vec(x_dev, ldx, desc->x_type)};
    return launched("w4_fwd", launch_w4(p, desc->x_type, zp, static_cast<hipStream_t>(stream)));
}

iqnn_status iqnn_w4_kernel(const iqnn_w4_desc* desc, int64_t m, int aligned_x, int32_t kernel[4]) {
    const iqnn_status s = check_w4(desc);
    if (s != IQNN_OK) return s;
    if (m <= 0 || !kernel) return fail(IQNN_ERR_INVALID_ARG, "w4_kernel: m must be positive, kernel not null");
    const W4Choice c = w4_choice(m, desc->n, w4_geom(desc->n, desc->k, desc->group, false).gpb, desc->x_type == F_F32,
                                 aligned_x && desc->k % 8 == 0);
    kernel[0] = c.tile;
    kernel[1] = c.rows;
    kernel[2] = c.nt;
    kernel[3] = c.sets;
    return ok();
}

iqnn_status iqnn_ckpt_act_fwd(const void* x_dev, int32_t x_type, int64_t rows, int64_t cols, int64_t ldx,
                              int32_t act, int gated, int32_t group, void* y_dev, int64_t ldy, void* q_dev,
                              float* scale_dev, void* stream) {
    const char* op = "ckpt_act_fwd";
    iqnn_status s = check_view(op, x_type, rows, cols, ldx, gated ? 2 * cols : cols, group);
    if (s != IQNN_OK) return s;
    s = check_view(op, x_type, rows, cols, ldy, cols, group);
    if (s != IQNN_OK) return s;
    if (!is_act(act)) return fail(IQNN_ERR_INVALID_ARG, "%s: unknown activation %d", op, act);
    if (rows == 0) return ok();
    if (!x_dev || !y_dev || !q_dev != !scale_dev) return fail(IQNN_ERR_INVALID_ARG, "%s: null pointer", op);
    if (!aligned(x_dev, fsize(x_type)) || !aligned(y_dev, fsize(x_type)) || !aligned(scale_dev, 4))
        return fail(IQNN_ERR_ALIGNMENT, "%s: misaligned pointer", op);
    const bool vec = cols % 8 == 0 && rows_vec(x_dev, ldx, x_type) && rows_vec(y_dev, ldy, x_type) && aligned(q_dev, 8);
    const ActParams p{x_dev, y_dev, static_cast<uint8_t*>(q_dev), scale_dev, rows, cols, ldx, ldy,
                      groups_of(cols, group), group, units_of(cols, group), x_type, act, gated != 0, vec};
    return launched(op, launch_act_fwd(p, static_cast<hipStream_t>(stream)));
}

iqnn_status iqnn_ckpt_act_bwd(const void* dy_dev, int32_t dy_type, int64_t rows, int64_t cols, int64_t lddy,
                              int32_t act, int gated, int32_t group, const void* q_dev, const float* scale_dev,
                              void* dx_dev, int64_t lddx, void* stream) {
    const char* op = "ckpt_act_bwd";
    iqnn_status s = check_view(op, dy_type, rows, cols, lddy, cols, group);
    if (s != IQNN_OK) return s;
    s = check_view(op, dy_type, rows, cols, lddx, gated ? 2 * cols : cols, group);
    if (s != IQNN_OK) return s;
    if (!is_act(act)) return fail(IQNN_ERR_INVALID_ARG, "%s: unknown activation %d", op, act);
    if (rows == 0) return ok();
    if (!dy_dev || !dx_dev || !q_dev || !scale_dev) return fail(IQNN_ERR_INVALID_ARG, "%s: null pointer", op);
    if (!aligned(dy_dev, fsize(dy_type)) || !aligned(dx_dev, fsize(dy_type)) || !aligned(scale_dev, 4))
        return fail(IQNN_ERR_ALIGNMENT, "%s: misaligned pointer", op);
    const bool vec = cols % 8 == 0 && rows_vec(dy_dev, lddy, dy_type) && rows_vec(dx_dev, lddx, dy_type) && aligned(q_dev, 8);
    // the kernel only reads the codes and scales
    const ActParams p{dy_dev, dx_dev, static_cast<uint8_t*>(const_cast<void*>(q_dev)), const_cast<float*>(scale_dev),
                      rows, cols, lddy, lddx, groups_of(cols, group), group, units_of(cols, group), dy_type, act,
                      gated != 0, vec};
    return launched(op, launch_act_bwd(p, static_cast<hipStream_t>(stream)));
}

size_t iqnn_ckpt_wgrad_workspace(const iqnn_ckpt_wgrad_desc* desc) {
    if (check_wgrad(desc) != IQNN_OK) return 0;
    ok();
    return (size_t)wgrad_plan(desc->m, desc->n, desc->k, desc->dw_type == F_F32).workspace;
}

iqnn_status iqnn_ckpt_wgrad(const iqnn_ckpt_wgrad_desc* desc, const void* dy_dev, int64_t lddy, const void* q_dev,
                            const float* scale_dev, void* dw_dev, void* db_dev, void* workspace_dev,
                            size_t workspace_bytes, void* stream) {
    iqnn_status s = check_wgrad(desc);
    if (s != IQNN_OK) return s;
    s = check_view("ckpt_wgrad", desc->dy_type, desc->m, desc->n, lddy, desc->n, desc->group);
    if (s != IQNN_OK) return s;
    const WgradPlan w = wgrad_plan(desc->m, desc->n, desc->k, desc->dw_type == F_F32);
    if (!dw_dev || (desc->m > 0 && (!dy_dev || !q_dev || !scale_dev)) || (w.workspace && !workspace_dev))
        return fail(IQNN_ERR_INVALID_ARG, "ckpt_wgrad: null pointer");
    if (workspace_bytes < (size_t)w.workspace)
        return fail(IQNN_ERR_INVALID_ARG, "ckpt_wgrad: workspace of %zu bytes, %lld needed", workspace_bytes,
                    (long long)w.workspace);
    if (!aligned(dy_dev, fsize(desc->dy_type)) || !aligned(scale_dev, 4) || !aligned(dw_dev, fsize(desc->dw_type)) ||
        !aligned(db_dev, fsize(desc->dw_type)) || (w.workspace && !aligned(workspace_dev, 16)))
        return fail(IQNN_ERR_ALIGNMENT, "ckpt_wgrad: misaligned pointer");
    const bool vec = desc->n % 8 == 0 && desc->k % 8 == 0 && rows_vec(dy_dev, lddy, desc->dy_type) && aligned(q_dev, 8);
    const bool ring = vec && desc->m > 0 && desc->k % 16 == 0 && aligned(q_dev, 16);   // 16-byte units of codes
    const WgradParams p{dy_dev, static_cast<const uint8_t*>(q_dev), scale_dev, dw_dev, db_dev,
                        static_cast<float*>(workspace_dev), desc->m, desc->n, desc->k, lddy,
                        groups_of(desc->k, desc->group), w.tile, w.n_tiles, w.k_tiles, w.splits, w.rows_per_split,
                        desc->group, vec, ring};
    return launched("ckpt_wgrad", launch_wgrad(p, desc->dy_type, desc->dw_type == F_F32, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
