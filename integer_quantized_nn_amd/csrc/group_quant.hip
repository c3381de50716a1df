// group_quant.hip -- quantization with parameters found on the device, one scale per
// group of consecutive elements of a row, its inverse, and an activation function whose
// input is kept as such 8-bit codes for the backward pass.
//
//   S = max|x| / Q_MAX, Z = 0                          (INT8, INT4)
//   S = (max(x,0) - min(x,0)) / (Q_MAX - Q_MIN), Z = clip(Q_MIN - rne(min(x,0) / S))   (UINT8, UINT4)
//   q = clip(rne(x / S) + Z),  x^ = (q - Z) * S
// with every step one binary32 operation, as iqnn_choose_qparams and iqnn_quantize.
//
// All kernels are HBM-bound streams.  A thread owns 8 consecutive elements of a row, so
// a 32 / 64 / 128-element group is 4 / 8 / 16 neighbouring lanes and its range is a
// butterfly of DPP moves inside a 16-lane row: x is read once and no LDS is used.  With
// one scale per row (group 0) a wave or a block walks the row twice; the second walk
// hits the caches.
//
// A group that holds a NaN or an infinity gets scale NaN (and codes and zero point 0),
// so it restores to NaN: a bad activation stays visible in the gradients.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <type_traits>

#include "float_types.h"
#include "iqnn_internal.h"

#pragma clang fp contract(off)

namespace iqnn {
namespace {

// ---- range of a group ---------------------------------------------------------------

// The range of |x| is kept as integers: for non-negative floats the order of the bits
// is the order of the values, and infinities and NaN lie above every finite value, so
// one integer maximum both finds the range and reports a non-finite element.
struct Range {
    uint32_t amax;
    float lo, hi;   // min(x, 0), max(x, 0); only kept for unsigned codes
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

template <bool ASYM>
__device__ __forceinline__ void take(Range& r, uint32_t amax, float lo, float hi) {
    r.amax = r.amax > amax ? r.amax : amax;
    if (ASYM) { r.lo = fminf(r.lo, lo); r.hi = fmaxf(r.hi, hi); }
}

template <int CTRL, bool ASYM>
__device__ __forceinline__ void merge_dpp(Range& r) {
    const uint32_t a = dpp<CTRL>(r.amax);
    float lo = 0, hi = 0;
    if (ASYM) { lo = as_f32(dpp<CTRL>(as_u32(r.lo))); hi = as_f32(dpp<CTRL>(as_u32(r.hi))); }
    take<ASYM>(r, a, lo, hi);
}

template <bool ASYM>
__device__ __forceinline__ Range range_of(const float v[8]) {
    Range r{0, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) take<ASYM>(r, as_u32(v[j]) & 0x7FFFFFFFu, v[j], v[j]);
    return r;
}

// Over `lanes` (4, 8 or 16, uniform) neighbouring lanes: quad_perm pairs and swaps,
// then the mirrored half row and row, which hold the other quad and the other half.
template <bool ASYM>
__device__ __forceinline__ void merge_lanes(Range& r, int lanes) {
    merge_dpp<0xB1, ASYM>(r);    // quad_perm [1,0,3,2]
    merge_dpp<0x4E, ASYM>(r);    // quad_perm [2,3,0,1]
    if (lanes >= 8) merge_dpp<0x141, ASYM>(r);    // row_half_mirror
    if (lanes >= 16) merge_dpp<0x140, ASYM>(r);   // row_mirror
}

template <bool ASYM>
__device__ __forceinline__ void merge_wave(Range& r) {
    merge_lanes<ASYM>(r, 16);
#pragma unroll
    for (int d = 16; d < 64; d <<= 1) {
        const uint32_t a = __shfl_xor(r.amax, d);
        float lo = 0, hi = 0;
        if (ASYM) { lo = __shfl_xor(r.lo, d); hi = __shfl_xor(r.hi, d); }
        take<ASYM>(r, a, lo, hi);
    }
}

// ---- parameters and codes -----------------------------------------------------------

struct QParams {
    float s, inv;
    int32_t z;
    bool ok, exact_div;
};

template <bool ASYM, bool FOUR>
__device__ __forceinline__ QParams params_of(const Range& r) {
    constexpr int lo = ASYM ? 0 : (FOUR ? -8 : -128), hi = ASYM ? (FOUR ? 15 : 255) : (FOUR ? 7 : 127);
    QParams p;
    p.z = 0;
    const float width = ASYM ? r.hi - r.lo : as_f32(r.amax);
    p.ok = r.amax < 0x7F800000u && as_u32(width) < 0x7F800000u;
    float s = width / (ASYM ? (float)(hi - lo) : (float)hi);
    if (!(s >= 1.17549435e-38f)) s = 1.0f;
    if (ASYM && p.ok) {
        const int32_t t = (int32_t)__builtin_rintf(r.lo / s);
        p.z = lo - t < lo ? lo : (lo - t > hi ? hi : lo - t);
    }
    p.s = p.ok ? s : as_f32(0x7FC00000u);
    p.inv = 1.0f / s;
    p.exact_div = s < 0x1p-90f;
    return p;
}

// x / S correctly rounded, without a division: with r = RN(1/S), one residual step brings
// x * r within an ulp of x / S and a second one rounds it correctly (Markstein's theorem;
// the residuals are exact while nothing underflows, hence the plain division for tiny S).
__device__ __forceinline__ float quotient(float x, const QParams& p) {
    float q = x * p.inv;
    q = __builtin_fmaf(__builtin_fmaf(-q, p.s, x), p.inv, q);
    return __builtin_fmaf(__builtin_fmaf(-q, p.s, x), p.inv, q);
}

// Eight codes, packed.  Adding 1.5 * 2^23 rounds a quotient to the nearest even integer and
// leaves its two's complement in the low bits.  Symmetric quotients need no clip: |x| / S is
// at most Q_MAX (1 + 2^-23), which rounds to Q_MAX.
template <bool ASYM, bool FOUR>
__device__ __forceinline__ uint2 codes_of(const float v[8], const QParams& p) {
    constexpr int lo = ASYM ? 0 : (FOUR ? -8 : -128), hi = ASYM ? (FOUR ? 15 : 255) : (FOUR ? 7 : 127);
    float q[8];
    if (p.exact_div) {
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = v[j] / p.s;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = quotient(v[j], p);
    }
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (ASYM) {
            const float t = fminf(fmaxf(__builtin_rintf(q[j]), (float)(lo - p.z)), (float)(hi - p.z));
            c[j] = (uint32_t)((int32_t)t + p.z);
        } else {
            c[j] = as_u32(q[j] + 12582912.0f);
        }
    }
    uint32_t w[2] = {0, 0};
    if (FOUR) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[0] |= (c[j] & 0xFu) << (4 * j);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[h] = __builtin_amdgcn_perm(c[4 * h + 1], c[4 * h], 0x0C0C0400u) |
                   __builtin_amdgcn_perm(c[4 * h + 3], c[4 * h + 2], 0x04000C0Cu);
    }
    return p.ok ? make_uint2(w[0], w[1]) : make_uint2(0, 0);
}

// Eight codes of one row chunk to memory: VEC writes 8 (4) aligned bytes.
template <bool FOUR, bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* base, int64_t e, int n, uint2 w) {
    if (FOUR) {
        if (VEC) *reinterpret_cast<uint32_t*>(base + e / 2) = w.x;
        else if (n == 8) __builtin_memcpy(base + e / 2, &w.x, 4);
        else
            for (int j = 0; j < n / 2; ++j) base[e / 2 + j] = (uint8_t)(w.x >> (8 * j));
    } else {
        if (VEC) *reinterpret_cast<uint2*>(base + e) = w;
        else store_bytes(base + e, n, w);
    }
}

template <bool VEC, typename T>
__device__ __forceinline__ void load_chunk(const T* p, int n, float v[8]) {
    if (VEC) load8(p, v);
    else load_n(p, n, v);
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_chunk(T* p, int n, const float v[8]) {
    if (VEC) store8(p, v);
    else store_n(p, n, v);
}

// Position of a thread in the [rows][units] grid of 8-element units (rows of
// p.units_per_row units, the last group's missing ones included).
struct Unit {
    int64_t row;
    int32_t u;
    bool in;
};
__device__ __forceinline__ Unit unit_of(int64_t rows, int32_t per_row) {
    const int64_t t = block_id() * 256 + threadIdx.x;
    Unit r;
    if (rows * per_row < ((int64_t)1 << 31)) {
        r.row = (uint32_t)t / (uint32_t)per_row;
        r.u = (int32_t)((uint32_t)t - (uint32_t)r.row * (uint32_t)per_row);
    } else {
        r.row = t / per_row;
        r.u = (int32_t)(t - r.row * per_row);
    }
    r.in = r.row < rows;
    return r;
}

// ---- quantize / dequantize ----------------------------------------------------------

template <typename T, bool ASYM, bool FOUR, bool VEC>
__global__ __launch_bounds__(256) void quantize_groups_kernel(const GroupQuantParams p) {
    const Unit t = unit_of(p.rows, p.units_per_row);
    const int64_t c0 = (int64_t)t.u * 8;
    const bool in = t.in && c0 < p.cols;
    const int n = !in ? 0 : (p.cols - c0 < 8 ? (int)(p.cols - c0) : 8);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (in) load_chunk<VEC>(static_cast<const T*>(p.x) + t.row * p.ldx + c0, n, v);
    const int lanes = p.group / 8;
    Range r = range_of<ASYM>(v);
    merge_lanes<ASYM>(r, lanes);
    if (!in) return;
    const QParams qp = params_of<ASYM, FOUR>(r);
    store_codes<FOUR, VEC>(p.q, t.row * p.cols + c0, n, codes_of<ASYM, FOUR>(v, qp));
    if (t.u % lanes == 0) {
        const int64_t g = t.row * p.groups + t.u / lanes;
        p.scale[g] = qp.s;
        if (ASYM) p.zp[g] = qp.z;
    }
}

// One scale per row: WAVES waves of a block share a row (1: a row per wave).
template <int WAVES, bool ASYM>
__device__ __forceinline__ void merge_row(Range& r) {
    merge_wave<ASYM>(r);
    if (WAVES > 1) {
        __shared__ uint32_t part[3][WAVES];
        const int w = threadIdx.x / 64;
        __syncthreads();
        if (threadIdx.x % 64 == 0) { part[0][w] = r.amax; part[1][w] = as_u32(r.lo); part[2][w] = as_u32(r.hi); }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WAVES; ++i) take<ASYM>(r, part[0][i], as_f32(part[1][i]), as_f32(part[2][i]));
    }
}

template <typename T, bool ASYM, bool FOUR, bool VEC, int WAVES>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const GroupQuantParams p) {
    constexpr int kStep = WAVES * 64 * 8;
    const int64_t row = block_id() * (4 / WAVES) + threadIdx.x / (64 * WAVES);
    if (row >= p.rows) return;   // whole waves; with WAVES = 4 the whole block
    const int64_t t0 = (int64_t)(threadIdx.x % (64 * WAVES)) * 8;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    Range r{0, 0.0f, 0.0f};
    for (int64_t c = t0; c < p.cols; c += kStep) {
        float v[8];
        load_chunk<VEC>(x + c, p.cols - c < 8 ? (int)(p.cols - c) : 8, v);
        const Range s = range_of<ASYM>(v);
        take<ASYM>(r, s.amax, s.lo, s.hi);
    }
    merge_row<WAVES, ASYM>(r);
    const QParams qp = params_of<ASYM, FOUR>(r);
    for (int64_t c = t0; c < p.cols; c += kStep) {
        const int n = p.cols - c < 8 ? (int)(p.cols - c) : 8;
        float v[8];
        load_chunk<VEC>(x + c, n, v);
        store_codes<FOUR, VEC>(p.q, row * p.cols + c, n, codes_of<ASYM, FOUR>(v, qp));
    }
    if (t0 == 0) {
        p.scale[row] = qp.s;
        if (ASYM) p.zp[row] = qp.z;
    }
}

// Codes of one 8-element chunk as q - Z.
template <bool ASYM, bool FOUR, bool VEC>
__device__ __forceinline__ void load_codes(const uint8_t* base, int64_t e, int n, int32_t z, float v[8]) {
    uint32_t w[2] = {0, 0};
    if (FOUR) {
        if (VEC) w[0] = *reinterpret_cast<const uint32_t*>(base + e / 2);
        else if (n == 8) __builtin_memcpy(w, base + e / 2, 4);
        else
            for (int j = 0; j < n / 2; ++j) w[0] |= (uint32_t)base[e / 2 + j] << (8 * j);
    } else {
        const uint2 a = VEC ? *reinterpret_cast<const uint2*>(base + e) : load_bytes(base + e, n);
        w[0] = a.x;
        w[1] = a.y;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        int32_t q;
        if (FOUR) q = ASYM ? (int32_t)((w[0] >> (4 * j)) & 0xF) : ((int32_t)(w[0] << (28 - 4 * j)) >> 28);
        else q = ASYM ? (int32_t)((w[j >> 2] >> (8 * (j & 3))) & 0xFF)
                      : (int32_t)(int8_t)(w[j >> 2] >> (8 * (j & 3)));
        v[j] = (float)(q - z);
    }
}

template <typename T, bool ASYM, bool FOUR, bool VEC>
__global__ __launch_bounds__(256) void dequantize_groups_kernel(const GroupDequantParams p) {
    const Unit t = unit_of(p.rows, p.units_per_row);
    const int64_t c0 = (int64_t)t.u * 8;
    if (!t.in || c0 >= p.cols) return;
    const int n = p.cols - c0 < 8 ? (int)(p.cols - c0) : 8;
    const int64_t g = t.row * p.groups + (p.group ? t.u / (p.group / 8) : 0);
    const float s = p.scale[g];
    float v[8];
    load_codes<ASYM, FOUR, VEC>(p.q, t.row * p.cols + c0, n, ASYM ? p.zp[g] : 0, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * s;
    store_chunk<VEC>(static_cast<T*>(p.x) + t.row * p.ldx + c0, n, v);
}

// ---- activation with an 8-bit checkpoint of its input -------------------------------

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhC = 0.79788456080286536f;   // sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;

// T: the element type of the result.  float results take the accurate library functions;
// 16-bit ones take the hardware exp and reciprocal (about 2^-22), far below their half
// step of 2^-12 (f16) and 2^-9 (bf16).
template <typename T>
struct Acc { static constexpr bool value = false; };
template <>
struct Acc<float> { static constexpr bool value = true; };

template <typename T>
__device__ __forceinline__ float exp_of(float x) {
    if constexpr (Acc<T>::value) return expf(x);
    else return __builtin_amdgcn_exp2f(x * 1.4426950408889634f);
}
template <typename T>
__device__ __forceinline__ float sigmoid(float x) {
    if constexpr (Acc<T>::value) return 1.0f / (1.0f + expf(-x));
    else return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f));
}

// The normal distribution function and its density (times 1; see kInvSqrt2Pi).  For 16-bit
// results e = exp(-x^2 / 2) serves both: the tail is e * erfcx(|x| / sqrt 2) / 2, with the
// scaled erfc as a polynomial in t = 1 / (1 + 0.44 z), a least-squares fit reweighted to
// a relative error below 5.2e-6 on z in [0, 12]; beyond it e underflows.
template <typename T>
__device__ __forceinline__ float normal_cdf(float x, float* e) {
    *e = exp_of<T>(-0.5f * x * x);
    if constexpr (Acc<T>::value) {
        return 0.5f * erfcf(-x * kSqrtHalf);
    } else {
        const float ax = __builtin_fabsf(x);
        const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(ax, 0.44f * kSqrtHalf, 1.0f));
        float c = -0.14616722f;
        c = __builtin_fmaf(c, t, 0.35084396f);
        c = __builtin_fmaf(c, t, 0.04050405f);
        c = __builtin_fmaf(c, t, 0.26371356f);
        c = __builtin_fmaf(c, t, 0.24253621f);
        c = __builtin_fmaf(c, t, 0.24856425f);
        const float tail = 0.5f * *e * (c * t);
        return x > 0.0f ? 1.0f - tail : tail;
    }
}

// act(x) and act'(x).  GELU_TANH as x * sigmoid(2u), u = c (x + a x^3), which is
// 0.5 x (1 + tanh u) without the cancellation for negative x.
template <typename T>
__device__ __forceinline__ float act_value(int32_t act, float x) {
    float e;
    switch (act) {
    case A_RELU: return x > 0.0f ? x : (x == x ? 0.0f : x);
    case A_GELU: return x * normal_cdf<T>(x, &e);
    case A_GELU_TANH: return x * sigmoid<T>(2.0f * kTanhC * x * (1.0f + kTanhA * x * x));
    default: return x * sigmoid<T>(x);
    }
}

template <typename T>
__device__ __forceinline__ float act_slope(int32_t act, float x) {
    switch (act) {
    case A_RELU: return x == x ? (x > 0.0f ? 1.0f : 0.0f) : x;
    case A_GELU: {
        float e;
        const float cdf = normal_cdf<T>(x, &e);
        return cdf + x * kInvSqrt2Pi * e;
    }
    case A_GELU_TANH: {
        // beyond |x| = 30 the slope is 0 or 1; the clamp keeps 0 * inf out
        const float y = fminf(fmaxf(x, -30.0f), 30.0f);
        const float y2 = y * y;
        const float u2 = 2.0f * kTanhC * y * (1.0f + kTanhA * y2);
        const float sg = sigmoid<T>(u2);
        const float d = sg + y * 2.0f * sg * sigmoid<T>(-u2) * kTanhC * (1.0f + 3.0f * kTanhA * y2);
        return x == x ? d : x;
    }
    default: {
        const float sg = sigmoid<T>(x);
        return sg * (1.0f + x * sigmoid<T>(-x));
    }
    }
}

template <typename T, bool GATED, bool VEC>
__device__ __forceinline__ void act_chunk(const ActParams& p, int64_t row, int64_t c0, int n, const float a[8],
                                          const float b[8]) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = act_value<T>(p.act, a[j]);
        if (GATED) y[j] = y[j] * b[j];
    }
    store_chunk<VEC>(static_cast<T*>(p.y) + row * p.ldy + c0, n, y);
}

template <typename T, bool GATED, bool VEC>
__global__ __launch_bounds__(256) void act_fwd_groups_kernel(const ActParams p) {
    const Unit t = unit_of(p.rows, p.units_per_row);
    const int64_t c0 = (int64_t)t.u * 8;
    const bool in = t.in && c0 < p.cols;
    const int n = !in ? 0 : (p.cols - c0 < 8 ? (int)(p.cols - c0) : 8);
    float a[8] = {0, 0, 0, 0, 0, 0, 0, 0}, b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const T* x = static_cast<const T*>(p.x) + t.row * p.ldx + c0;
    if (in) {
        load_chunk<VEC>(x, n, a);
        if (GATED) load_chunk<VEC>(x + p.cols, n, b);
    }
    const int lanes = p.group / 8;
    Range ra = range_of<false>(a), rb = range_of<false>(b);
    merge_lanes<false>(ra, lanes);
    if (GATED) merge_lanes<false>(rb, lanes);
    if (!in) return;
    act_chunk<T, GATED, VEC>(p, t.row, c0, n, a, b);
    if (!p.q) return;   // y alone
    const int64_t halves = GATED ? 2 : 1;
    int64_t e = t.row * p.cols * halves + c0;
    int64_t g = t.row * p.groups * halves + t.u / lanes;
    const QParams qa = params_of<false, false>(ra);
    store_codes<false, VEC>(p.q, e, n, codes_of<false, false>(a, qa));
    if (t.u % lanes == 0) p.scale[g] = qa.s;
    if (GATED) {
        e += p.cols;
        g += p.groups;
        const QParams qb = params_of<false, false>(rb);
        store_codes<false, VEC>(p.q, e, n, codes_of<false, false>(b, qb));
        if (t.u % lanes == 0) p.scale[g] = qb.s;
    }
}

template <typename T, bool GATED, bool VEC, int WAVES>
__global__ __launch_bounds__(256) void act_fwd_rows_kernel(const ActParams p) {
    constexpr int kStep = WAVES * 64 * 8;
    const int64_t row = block_id() * (4 / WAVES) + threadIdx.x / (64 * WAVES);
    if (row >= p.rows) return;   // whole waves; with WAVES = 4 the whole block
    const int64_t t0 = (int64_t)(threadIdx.x % (64 * WAVES)) * 8;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    constexpr int64_t halves = GATED ? 2 : 1;
    Range r[halves];
#pragma unroll
    for (int h = 0; h < halves; ++h) r[h] = Range{0, 0.0f, 0.0f};
    for (int64_t c = t0; c < p.cols; c += kStep) {
        const int n = p.cols - c < 8 ? (int)(p.cols - c) : 8;
#pragma unroll
        for (int h = 0; h < halves; ++h) {
            float v[8];
            load_chunk<VEC>(x + h * p.cols + c, n, v);
            take<false>(r[h], range_of<false>(v).amax, 0, 0);
        }
    }
    QParams qp[halves];
#pragma unroll
    for (int h = 0; h < halves; ++h) {
        merge_row<WAVES, false>(r[h]);
        qp[h] = params_of<false, false>(r[h]);
        if (t0 == 0) p.scale[row * halves + h] = qp[h].s;
    }
    for (int64_t c = t0; c < p.cols; c += kStep) {
        const int n = p.cols - c < 8 ? (int)(p.cols - c) : 8;
        float v[2][8];
#pragma unroll
        for (int h = 0; h < halves; ++h) {
            load_chunk<VEC>(x + h * p.cols + c, n, v[h]);
            store_codes<false, VEC>(p.q, (row * halves + h) * p.cols + c, n, codes_of<false, false>(v[h], qp[h]));
        }
        act_chunk<T, GATED, VEC>(p, row, c, n, v[0], v[halves - 1]);
    }
}

template <typename T, bool GATED, bool VEC>
__global__ __launch_bounds__(256) void act_bwd_kernel(const ActParams p) {
    const Unit t = unit_of(p.rows, p.units_per_row);
    const int64_t c0 = (int64_t)t.u * 8;
    if (!t.in || c0 >= p.cols) return;
    const int n = p.cols - c0 < 8 ? (int)(p.cols - c0) : 8;
    const int64_t halves = GATED ? 2 : 1;
    const int64_t g = t.row * p.groups * halves + (p.group ? t.u / (p.group / 8) : 0);
    const int64_t e = t.row * p.cols * halves + c0;
    float dy[8], a[8], b[8], d[8];
    load_chunk<VEC>(static_cast<const T*>(p.x) + t.row * p.ldx + c0, n, dy);
    load_codes<false, false, VEC>(p.q, e, n, 0, a);
    const float sa = p.scale[g];
    T* dx = static_cast<T*>(p.y) + t.row * p.ldy + c0;
    if (GATED) {
        load_codes<false, false, VEC>(p.q, e + p.cols, n, 0, b);
        const float sb = p.scale[g + p.groups];
        float du[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = a[j] * sa;
            d[j] = dy[j] * (b[j] * sb) * act_slope<T>(p.act, x);
            du[j] = dy[j] * act_value<T>(p.act, x);
        }
        store_chunk<VEC>(dx + p.cols, n, du);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = dy[j] * act_slope<T>(p.act, a[j] * sa);
    }
    store_chunk<VEC>(dx, n, d);
}

// ---- launch -------------------------------------------------------------------------

// A row of more elements than this is shared by the four waves of a block.
constexpr int64_t kWaveRow = 4 * 64 * 8;

template <typename F>
hipError_t with_type(int32_t t, F f) {
    switch (t) {
    case F_F32: return f((float*)nullptr);
    case F_F16: return f((_Float16*)nullptr);
    default: return f((__bf16*)nullptr);
    }
}
template <typename F>
hipError_t with_bool(bool b, F f) {
    return b ? f(std::true_type()) : f(std::false_type());
}

hipError_t blocks_of(int64_t threads, dim3* g) { return grid_of((threads + 255) / 256, 256, g); }

}  // namespace

hipError_t launch_quantize_groups(const GroupQuantParams& p, hipStream_t stream) {
    if (p.rows == 0) return hipSuccess;
    const bool asym = p.qtype == T_UINT8 || p.qtype == T_UINT4, four = p.qtype == T_INT4 || p.qtype == T_UINT4;
    return with_type(p.x_type, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        return with_bool(asym, [&](auto A) { return with_bool(four, [&](auto F) { return with_bool(p.vec, [&](auto V) {
            constexpr bool a = decltype(A)::value, f = decltype(F)::value, v = decltype(V)::value;
            dim3 g;
            if (p.group) {
                const hipError_t e = blocks_of(p.rows * p.units_per_row, &g);
                if (e != hipSuccess) return e;
                quantize_groups_kernel<T, a, f, v><<<g, 256, 0, stream>>>(p);
            } else if (p.cols <= kWaveRow) {
                const hipError_t e = blocks_of(p.rows * 64, &g);
                if (e != hipSuccess) return e;
                quantize_rows_kernel<T, a, f, v, 1><<<g, 256, 0, stream>>>(p);
            } else {
                const hipError_t e = blocks_of(p.rows * 256, &g);
                if (e != hipSuccess) return e;
                quantize_rows_kernel<T, a, f, v, 4><<<g, 256, 0, stream>>>(p);
            }
            return hipGetLastError();
        }); }); });
    });
}

hipError_t launch_dequantize_groups(const GroupDequantParams& p, hipStream_t stream) {
    if (p.rows == 0) return hipSuccess;
    const bool asym = p.qtype == T_UINT8 || p.qtype == T_UINT4, four = p.qtype == T_INT4 || p.qtype == T_UINT4;
    dim3 g;
    const hipError_t e = blocks_of(p.rows * p.units_per_row, &g);
    if (e != hipSuccess) return e;
    return with_type(p.x_type, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        return with_bool(asym, [&](auto A) { return with_bool(four, [&](auto F) { return with_bool(p.vec, [&](auto V) {
            dequantize_groups_kernel<T, decltype(A)::value, decltype(F)::value, decltype(V)::value>
                <<<g, 256, 0, stream>>>(p);
            return hipGetLastError();
        }); }); });
    });
}

hipError_t launch_act_fwd(const ActParams& p, hipStream_t stream) {
    if (p.rows == 0) return hipSuccess;
    return with_type(p.x_type, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        return with_bool(p.gated, [&](auto G) { return with_bool(p.vec, [&](auto V) {
            constexpr bool gt = decltype(G)::value, v = decltype(V)::value;
            dim3 g;
            if (p.group || !p.q) {   // without codes no group matters
                const hipError_t e = blocks_of(p.rows * p.units_per_row, &g);
                if (e != hipSuccess) return e;
                act_fwd_groups_kernel<T, gt, v><<<g, 256, 0, stream>>>(p);
            } else if (p.cols <= kWaveRow) {
                const hipError_t e = blocks_of(p.rows * 64, &g);
                if (e != hipSuccess) return e;
                act_fwd_rows_kernel<T, gt, v, 1><<<g, 256, 0, stream>>>(p);
            } else {
                const hipError_t e = blocks_of(p.rows * 256, &g);
                if (e != hipSuccess) return e;
                act_fwd_rows_kernel<T, gt, v, 4><<<g, 256, 0, stream>>>(p);
            }
            return hipGetLastError();
        }); });
    });
}

hipError_t launch_act_bwd(const ActParams& p, hipStream_t stream) {
    if (p.rows == 0) return hipSuccess;
    dim3 g;
    const hipError_t e = blocks_of(p.rows * p.units_per_row, &g);
    if (e != hipSuccess) return e;
    return with_type(p.x_type, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        return with_bool(p.gated, [&](auto G) { return with_bool(p.vec, [&](auto V) {
            act_bwd_kernel<T, decltype(G)::value, decltype(V)::value><<<g, 256, 0, stream>>>(p);
            return hipGetLastError();
        }); });
    });
}

}  // namespace iqnn
