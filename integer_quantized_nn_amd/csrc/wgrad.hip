// wgrad.hip -- weight and bias gradient of a linear layer y = x W^T + b whose input is
// kept as 8-bit codes with a scale per group:
//
//   x^[m][k] = q[m][k] * s[m][k / group]
//   dW[n][k] = sum_m dY[m][n] x^[m][k],   db[n] = sum_m dY[m][n]
//
// The contraction runs over the rows of both operands, so both MFMA operands come out of
// LDS transposed (ds_read_b64_tr_b16: 16 lanes read a 4 x 16 block by rows and receive it
// by columns).  The codes are restored on the way into LDS, once per block.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>
#include <type_traits>

#include "float_types.h"
#include "iqnn_internal.h"

#pragma clang fp contract(off)

namespace iqnn {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// How the operands reach the 16-bit matrix cores.
//   HALF   bf16 or f16 gradients of bf16 or f16 dY: dY as it is, x^ rounded once to its
//          type -- the activation as it was before it was saved, up to the code's own
//          half step (2^-8 of the group's maximum; the rounding is 2^-9 or 2^-12 of x^).
//          12608 x 4096 x 1024 bf16 lies 0.0022 from 64-bit sums (relative, root mean square),
//          0.0017 of it the result's own rounding.  A second piece of x^ would double the
//          products of a kernel whose products alone take half its time.
//   SPLIT  f32 gradients: both operands as exact sums of bf16 pieces of 8 significand
//          bits (dY 1, 2 or 3 of them, x^ 3); products of pieces i + j < 3 are kept.  Where
//          that leaves any out, pieces are rounded to nearest: piece 1 is at most 2^-8 of the
//          value and piece 2 2^-17, so what is left out lies below 1.01 * 2^-24 of the product,
//          of either sign.  (Cut off towards zero it reaches 2^-21, always of the product's
//          sign; 4096 x 2048 x 2048 f32, group 32: 286 us so, 298 us to nearest.)
//   FOLD   f32 gradients where a tile's columns share one scale per row: the codes alone
//          are exact in one piece, and three pieces of dY * s, rounded to binary32 first,
//          need three products instead of five (f16) or six (f32).
// Accumulation is binary32 in all.
template <typename T, bool SPLIT, bool FOLD = false>
struct Mode {
    static constexpr int pa = !SPLIT ? 1 : (FOLD || sizeof(T) == 4 ? 3 : (std::is_same<T, _Float16>::value ? 2 : 1));
    static constexpr int pb = SPLIT && !FOLD ? 3 : 1;
    static constexpr bool f16 = !SPLIT && std::is_same<T, _Float16>::value;
    static constexpr bool nearest = pa > 1 && pb > 1;   // some products of pieces are left out
};

template <bool F16>
__device__ __forceinline__ f32x4 mma(uint4 a, uint4 b, f32x4 c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// P bf16 pieces of eight floats whose sum they are (of an infinity, NaN: a non-finite operand
// makes its sums non-finite).  Each is the upper half of what is left, or with NEAREST, but for
// the last, what is left rounded; there the first is kept from rounding up to infinity.
template <int P, bool NEAREST>
__device__ __forceinline__ void split8(float v[8], uint4 o[P]) {
    constexpr float kMax = 0x1.FEp127f;   // bf16's largest
#pragma unroll
    for (int i = 0; i < P; ++i) {
        uint32_t w[4];
        if (NEAREST && i + 1 < P) {
            bf16x8 a;
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = (__bf16)(i == 0 ? __builtin_amdgcn_fmed3f(v[j], -kMax, kMax) : v[j]);
            o[i] = __builtin_bit_cast(uint4, a);
            w[0] = o[i].x; w[1] = o[i].y; w[2] = o[i].z; w[3] = o[i].w;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = v[2 * j] - as_f32(w[j] << 16);
                v[2 * j + 1] = v[2 * j + 1] - as_f32(w[j] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = __builtin_amdgcn_perm(as_u32(v[2 * j + 1]), as_u32(v[2 * j]), 0x07060302u);
            o[i] = make_uint4(w[0], w[1], w[2], w[3]);
            if (i + 1 < P) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = v[j] - as_f32(as_u32(v[j]) & 0xFFFF0000u);
            }
        }
    }
}

__device__ __forceinline__ uint4 to_bf16(const float v[8]) {
    bf16x8 a;
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = (__bf16)v[j];
    return __builtin_bit_cast(uint4, a);
}
__device__ __forceinline__ uint4 to_f16(const float v[8]) {
    f16x8 a;
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = half_of(v[j]);
    return __builtin_bit_cast(uint4, a);
}

// LDS image of an operand tile: 32 rows of C 16-bit elements, C = 64 or 128.  A transposed
// read touches eight rows r = 0..3 and 8..11 (or 4..7 and 12..15, 16 higher) at one 32-byte
// column unit per half wave; the unit's index is XORed with a different value on each of
// them (C = 64: on each of those in the same half of the banks), so the half wave covers all
// 64 banks.
template <int C>
__device__ __forceinline__ int lds_off(int r, int c) {   // byte offset of element (r, c), c % 4 == 0
    static_assert(C == 64 || C == 128, "columns");
    const int u = (c >> 4) ^ (C == 128 ? (r & 3) | ((r >> 1) & 4) : ((r >> 1) & 1) | ((r >> 2) & 2));
    return r * C * 2 + (u << 5) + (c & 15) * 2;
}

template <int C>
__device__ __forceinline__ uint4 frag_at(const uint8_t* t, int c0, int lane) {
    const int i = lane & 15, g = lane >> 4;
    typedef __attribute__((address_space(3))) s16x4* lp;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(t + lds_off<C>(8 * g + (i >> 2), c0 + 4 * (i & 3))));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(t + lds_off<C>(8 * g + 4 + (i >> 2), c0 + 4 * (i & 3))));
    const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
    return make_uint4(x.x, x.y, y.x, y.y);
}

constexpr int kStepM = 32;   // contraction rows per LDS stage: one MFMA step

// A block computes a BN x BK tile of dW over the rows of one split.  KS sets of 2 x 2 waves
// take every KS-th stage each, with LDS buffers of their own, and add up at the end: one
// set alone leaves a SIMD idle while its wave loads, restores and waits.
template <typename T, bool SPLIT, bool FOLD, int BN, int BK, int KS, bool VEC>
__global__ __launch_bounds__(256 * KS, KS) void wgrad_kernel(const WgradParams p) {
    typedef Mode<T, SPLIT, FOLD> Md;
    constexpr int PA = Md::pa, PB = Md::pb;
    constexpr int NI = BN / 32, KI = BK / 32;                 // 16-wide tiles per wave
    constexpr int CA = kStepM * BN / 8 / 256, CB = kStepM * BK / 8 / 256;   // 8-element chunks per thread
    constexpr int RA = 256 / (BN / 8), RB = 256 / (BK / 8);   // rows between a thread's chunks
    constexpr int kBuf = (PA * BN + PB * BK) * kStepM * 2;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[KS][2][kBuf];
    const int ks = KS == 1 ? 0 : threadIdx.x >> 8, tid = threadIdx.x & 255, lane = tid & 63, wave = tid >> 6;
    const int wn = (wave >> 1) * (BN / 2), wk = (wave & 1) * (BK / 2);

    const int64_t tiles = p.n_tiles * p.k_tiles;
    const int64_t id = block_id(), split = id / tiles, tile = id - split * tiles;
    if (split >= p.splits) return;   // a block that fills up a row of blocks
    const int64_t n0 = (tile / p.k_tiles) * BN, k0 = (tile % p.k_tiles) * BK;
    const int64_t m_lo = split * p.rows_per_split;
    const int64_t m_hi = m_lo + p.rows_per_split < p.m ? m_lo + p.rows_per_split : p.m;
    const bool bias = p.db != nullptr && tile % p.k_tiles == 0;

    const int ca = (tid % (BN / 8)) * 8, ra = tid / (BN / 8);
    const int cb = (tid % (BK / 8)) * 8, rb = tid / (BK / 8);
    const int na = p.n - (n0 + ca) < 8 ? (p.n - (n0 + ca) < 0 ? 0 : (int)(p.n - (n0 + ca))) : 8;
    const int nb = p.k - (k0 + cb) < 8 ? (p.k - (k0 + cb) < 0 ? 0 : (int)(p.k - (k0 + cb))) : 8;
    // Loads without branches, so that a stage's are all in flight at once.  Columns past the
    // end read column 0 (their results are not stored).  Rows past the end read the last row
    // with scale 0: what they add is 0, or NaN where that row makes the sum non-finite anyway.
    const bool ina = na == 8 || (!VEC && na > 0), inb = nb == 8 || (!VEC && nb > 0);
    const T* dy = static_cast<const T*>(p.dy) + (ina ? n0 + ca : 0);
    const uint8_t* qp = p.q + (inb ? k0 + cb : 0);
    const float* sp = p.scale + (p.group ? (FOLD || !inb ? k0 : k0 + cb) / p.group : 0);

    uint4 va[CA][sizeof(T) == 4 ? 2 : 1];
    uint2 vb[CB];
    float vs[FOLD ? CA : CB];
    const auto load = [&](int64_t m) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < CA; ++c) {
            const int64_t r = m + ra + c * RA;
            const T* src = dy + (r < m_hi ? r : m_hi - 1) * p.lddy;
            if (VEC) {
#pragma unroll
                for (int h = 0; h < (int)(sizeof(T) / 2); ++h)
                    va[c][h * (sizeof(T) == 4)] = reinterpret_cast<const uint4*>(src)[h * (sizeof(T) == 4)];
            } else {
                Pack8<T> e;
                if (na == 8) {
                    __builtin_memcpy(&e, src, sizeof e);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) e.e[j] = j < na ? src[j] : (T)0.0f;
                }
                __builtin_memcpy(va[c], &e, sizeof e);
            }
            if (FOLD) vs[FOLD ? c : 0] = sp[(r < m_hi ? r : m_hi - 1) * p.groups];
        }
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            const int64_t r = m + rb + c * RB, rc = r < m_hi ? r : m_hi - 1;
            if (!FOLD) vs[c] = sp[rc * p.groups];
            vb[c] = VEC ? *reinterpret_cast<const uint2*>(qp + rc * p.k) : load_bytes(qp + rc * p.k, nb);
        }
    };
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const auto stage = [&](int64_t m, uint8_t* buf) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < CA; ++c) {
            uint8_t* dst = buf + lds_off<BN>(ra + c * RA, ca);
            float v[8];
            if (SPLIT || bias) load8(reinterpret_cast<const T*>(va[c]), v);
            if (bias && m + ra + c * RA < m_hi) {
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += v[j];
            }
            if constexpr (SPLIT) {
                if (FOLD) {
                    const float sc = m + ra + c * RA < m_hi ? vs[FOLD ? c : 0] : 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = v[j] * sc;
                }
                uint4 o[PA];
                split8<PA, Md::nearest>(v, o);
#pragma unroll
                for (int i = 0; i < PA; ++i) *reinterpret_cast<uint4*>(dst + i * BN * kStepM * 2) = o[i];
            } else {
                *reinterpret_cast<uint4*>(dst) = va[c][0];
            }
        }
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            uint8_t* dst = buf + PA * BN * kStepM * 2 + lds_off<BK>(rb + c * RB, cb);
            float v[8];
            const float sc = FOLD ? 1.0f : (m + rb + c * RB < m_hi ? vs[FOLD ? 0 : c] : 0.0f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = (float)(int8_t)((j < 4 ? vb[c].x : vb[c].y) >> (8 * (j & 3)));
                if (!FOLD) v[j] = v[j] * sc;
            }
            if constexpr (SPLIT && !FOLD) {
                uint4 o[PB];
                split8<PB, Md::nearest>(v, o);
#pragma unroll
                for (int i = 0; i < PB; ++i) *reinterpret_cast<uint4*>(dst + i * BK * kStepM * 2) = o[i];
            } else {
                *reinterpret_cast<uint4*>(dst) = Md::f16 ? to_f16(v) : to_bf16(v);
            }
        }
    };

    f32x4 acc[NI][KI];
#pragma unroll
    for (int a = 0; a < NI; ++a)
#pragma unroll
        for (int b = 0; b < KI; ++b) acc[a][b] = f32x4{0, 0, 0, 0};

    const int64_t m_own = m_lo + ks * kStepM;
    if (m_own < m_hi) load(m_own);
    int cur = 0;
    for (int64_t mm = m_lo; mm < m_hi; mm += KS * kStepM) {
        const int64_t m = mm + ks * kStepM;
        const bool in = m < m_hi;
        if (in) {
            stage(m, lds[ks][cur]);
            if (m + KS * kStepM < m_hi) load(m + KS * kStepM);
        }
        __syncthreads();   // one barrier per stage: buffer cur is written again two stages on
        if (in) {
            const uint8_t* A = lds[ks][cur];
            const uint8_t* Bt = A + PA * BN * kStepM * 2;
#pragma unroll
            for (int j = 0; j < PB; ++j) {
                uint4 fb[KI];
#pragma unroll
                for (int b = 0; b < KI; ++b) fb[b] = frag_at<BK>(Bt + j * BK * kStepM * 2, wk + 16 * b, lane);
#pragma unroll
                for (int i = 0; i < PA; ++i) {
                    if (SPLIT && i + j >= 3) continue;
#pragma unroll
                    for (int a = 0; a < NI; ++a) {
                        const uint4 fa = frag_at<BN>(A + i * BN * kStepM * 2, wn + 16 * a, lane);
#pragma unroll
                        for (int b = 0; b < KI; ++b) acc[a][b] = mma<Md::f16>(fa, fb[b], acc[a][b]);
                    }
                }
            }
        }
        cur ^= 1;
    }

    if constexpr (KS > 1) {
        // the first set adds the others' sums, in order, a row of 16-wide tiles at a time
        f32x4* red = reinterpret_cast<f32x4*>(&lds[0][0][0]);   // [KS - 1][KI][256]
        static_assert((KS - 1) * KI * 4096 <= KS * 2 * kBuf, "LDS");
#pragma unroll
        for (int a = 0; a < NI; ++a) {
            __syncthreads();
            if (ks > 0) {
#pragma unroll
                for (int b = 0; b < KI; ++b) red[((ks - 1) * KI + b) * 256 + tid] = acc[a][b];
            }
            __syncthreads();
            if (ks == 0) {
#pragma unroll
                for (int o = 0; o < KS - 1; ++o)
#pragma unroll
                    for (int b = 0; b < KI; ++b) acc[a][b] = acc[a][b] + red[(o * KI + b) * 256 + tid];
            }
        }
    }
    // lane l of an accumulator holds rows 4 (l / 16) + r, column l % 16
    const bool whole = p.splits == 1;
    float* part = whole ? nullptr : p.part + split * p.n * p.k;
    if (ks == 0) {
#pragma unroll
        for (int a = 0; a < NI; ++a)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t n = n0 + wn + 16 * a + 4 * (lane >> 4) + r;
                if (n >= p.n) continue;
#pragma unroll
                for (int b = 0; b < KI; ++b) {
                    const int64_t k = k0 + wk + 16 * b + (lane & 15);
                    if (k >= p.k) continue;
                    if (!whole) part[n * p.k + k] = acc[a][b][r];
                    else if (SPLIT) static_cast<float*>(p.dw)[n * p.k + k] = acc[a][b][r];
                    else static_cast<T*>(p.dw)[n * p.k + k] = (T)acc[a][b][r];
                }
            }
    }
    if (bias) {
        float* red = reinterpret_cast<float*>(&lds[0][0][0]);   // [KS * RA][BN]
        static_assert(KS * RA * BN * 4 <= KS * 2 * kBuf, "LDS");
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) red[(ks * RA + ra) * BN + ca + j] = sum[j];
        __syncthreads();
        const int c = (int)threadIdx.x;
        if (c < BN && n0 + c < p.n) {
            float v = 0.0f;
            for (int r = 0; r < KS * RA; ++r) v += red[r * BN + c];
            if (!whole) p.part[p.splits * p.n * p.k + split * p.n + n0 + c] = v;
            else if (SPLIT) static_cast<float*>(p.db)[n0 + c] = v;
            else static_cast<T*>(p.db)[n0 + c] = (T)v;
        }
    }
}

// Position of a block among the output tiles: consecutive blocks go to the eight XCDs in
// turn, so each XCD takes a run of tiles, four across k and as many down n as it has; they
// share their rows of dY and of the codes in its L2.
struct Place {
    int64_t split, n_tile, k_tile;
};
__device__ __forceinline__ Place place_of(const WgradParams& p) {
    const uint32_t G = gridDim.x, q8 = G / 8, r8 = G % 8, xcd = blockIdx.x % 8;
    const int64_t at = (int64_t)(xcd < r8 ? xcd * (q8 + 1) : r8 * (q8 + 1) + (xcd - r8) * q8) + blockIdx.x / 8;
    const int64_t tiles = p.n_tiles * p.k_tiles;
    Place r;
    r.split = at / tiles;
    const int64_t t = at - r.split * tiles, band = t / (4 * p.n_tiles), in = t - band * 4 * p.n_tiles;
    const int64_t wide = p.k_tiles - band * 4 < 4 ? p.k_tiles - band * 4 : 4;
    r.n_tile = in / wide;
    r.k_tile = band * 4 + in % wide;
    return r;
}

// Loads from memory straight into LDS: lane i's 16 (4) bytes land at lds + 16 i (4 i); lds is
// wave-uniform.  m0 and the load sit in one statement so that nothing comes between them.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p);
}
__device__ __forceinline__ void load_lds16(uint8_t* lds, const void* src) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds_address(lds)), "v"(src)
                 : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(uint8_t* lds, const void* src) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds_address(lds)), "v"(src)
                 : "memory", "m0");
}

// 16-bit dY whose rows, like the codes', are whole 16-byte units.  dY, codes and scales all
// go from memory to LDS without registers.  For 16-bit results a stage multiplies what is in
// registers, reads the next one's operands and restores the codes of the one after that into
// the other of two buffers of x^; one barrier a stage, loads four stages ahead.  (f32 results:
// one buffer of x^, two barriers, loads two stages ahead.)  KS sets of 2 x 2 waves take every
// KS-th stage each, with LDS of their own, and add up at the end.
//
// What bounds it: 12608 x 4096 x 1024 bf16 takes 149 us, and copies of the kernel with a part
// left out of its stages take 117 us without reading and restoring the codes, 117 without the
// direct loads (132 without dY's, 138 without the codes' and scales'), 132 without the operand
// reads, 70 with products and barriers alone.  The parts overlap, so these do not add up.
//
// The waits are counted here: the compiler would empty the queue before every transposed
// read, and before every use of a code that came through a register (12608 x 4096 x 1024 bf16
// so: 180 us, 164 us with the first counted waits).  Each stage requests the same four loads
// per wave, also behind the last row, which is read again; so a batch has landed when at most
// the two later ones are outstanding.
//
// The bias gradient rides on dY's fragments: a product with rows of ones.  Its eight 16-wide
// column tiles are shared out among the waves and the blocks of a row of tiles, for a wave
// that does more than the others holds all of them up.
template <typename T, bool SPLIT, int KS, bool BIAS>
__global__ __launch_bounds__(256 * KS, 2) void wgrad_ring_kernel(const WgradParams p) {
    typedef Mode<T, SPLIT> Md;
    static_assert(Md::pa == 1 && (!SPLIT || KS == 1), "dY as it is");
    constexpr bool F16 = Md::f16;
    constexpr int PB = Md::pb, NB = SPLIT ? 3 : 4, XB = SPLIT ? 1 : 2;   // pieces of x^; buffers
    constexpr int BN = 128, BK = 128, NI = 4, KI = 4;
    constexpr int kY = BN * kStepM * 2, kQ = BK * kStepM, kS = 32 * kStepM, kX = PB * BK * kStepM * 2;
    // [buffer][set]: rows of dY (lds_off), of codes (128 bytes) and of scales (8 slots)
    __shared__ __attribute__((aligned(1024))) uint8_t yb[NB * KS * kY];
    __shared__ __attribute__((aligned(1024))) uint8_t qb[NB * KS * kQ];
    __shared__ __attribute__((aligned(1024))) uint8_t sb[NB * KS * kS];
    __shared__ __attribute__((aligned(1024))) uint8_t xb[XB * KS * kX];
    const int ks = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    const int tid = threadIdx.x & 255, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = (wave >> 1) * (BN / 2), wk = (wave & 1) * (BK / 2);
    const Place at = place_of(p);
    const int64_t n0 = at.n_tile * BN, k0 = at.k_tile * BK;
    const int64_t m_lo = at.split * p.rows_per_split;
    const int64_t m_hi = m_lo + p.rows_per_split < p.m ? m_lo + p.rows_per_split : p.m;

    // Columns past the end read column 0 (their results are not stored).  Rows past the end
    // read the last row and count as scale 0: what they add is 0, or NaN where that row makes
    // the sum non-finite anyway.
    // dY: lane l of a wave fills 16-byte unit l % 16 of rows 4 wave + l / 16 and 16 higher, and
    // fetches the unit that lds_off puts there (its XOR is the same 16 rows up)
    const int ry = 4 * wave + (lane >> 4);
    const int uy = (((lane & 15) >> 1) ^ ((ry & 3) | ((ry >> 1) & 4))) * 2 + (lane & 1);
    const T* const dy = static_cast<const T*>(p.dy) + (n0 + uy * 8 < p.n ? n0 + uy * 8 : 0);
    // codes and scales: lane l fills unit and slot l % 8 of row 8 wave + l / 8
    const int rq = 8 * wave + (lane >> 3);
    const uint8_t* const qp = p.q + (k0 + (lane & 7) * 16 < p.k ? k0 + (lane & 7) * 16 : 0);
    int64_t gi = p.group ? k0 / p.group + (lane & 7) : 0;
    const float* const sp = p.scale + (gi < p.groups ? gi : p.groups - 1);
    // A whole stage's addresses are one add each to offsets kept per lane; only the last rows
    // need the clamp and its products.
    const int64_t oy0 = ry * p.lddy, oy1 = (ry + 16) * p.lddy, oq = rq * p.k, os = rq * p.groups;
    constexpr int64_t step = KS * kStepM;
    // load i of the four of a batch: dY of the stage at row m, buffer u (0, 1), codes and
    // scales of the stage after it (2, 3)
    const auto request = [&](int64_t m, int u, int i) __attribute__((always_inline)) {
        if (i < 2) {
            const T* y = dy + m * p.lddy + (i ? oy1 : oy0);
            const int64_t r = m + ry + 16 * i;
            if (m + kStepM > m_hi) y = dy + (r < m_hi ? r : m_hi - 1) * p.lddy;
            load_lds16(yb + (u % NB * KS + ks) * kY + (wave * 4 + 16 * i) * BN * 2, y);
            return;
        }
        m += step;
        const int64_t r = m + rq < m_hi ? m + rq : m_hi - 1;
        if (i == 2) {
            const uint8_t* q = qp + m * p.k + oq;
            if (m + kStepM > m_hi) q = qp + r * p.k;
            load_lds16(qb + ((u + 1) % NB * KS + ks) * kQ + wave * 1024, q);
        } else {
            const float* c = sp + m * p.groups + os;
            if (m + kStepM > m_hi) c = sp + r * p.groups;
            load_lds4(sb + ((u + 1) % NB * KS + ks) * kS + wave * 256, c);
        }
    };

    f32x4 acc[NI][KI];
    f32x4 sum[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};   // of tiles (t, t + 1); every row of the product alike
#pragma unroll
    for (int a = 0; a < NI; ++a)
#pragma unroll
        for (int b = 0; b < KI; ++b) acc[a][b] = f32x4{0, 0, 0, 0};
    // the wave's column tiles whose bias it sums: the even ones or the odd ones of its half,
    // of each the blocks' k_tiles-th
    uint32_t mine = 0;
    const uint32_t one2 = F16 ? 0x3C003C00u : 0x3F803F80u;
    if constexpr (BIAS) {
        for (int t = wave & 1; t < NI; t += 2)
            if ((wn / 16 + t) % p.k_tiles == at.k_tile) mine |= 1u << t;
    }

    const auto rows_left = [&](int64_t m) { return (int)(m_hi - m < kStepM ? m_hi - m : kStepM); };   // below 1: none
    // the codes of the stage at row m, in buffer u, into x^'s buffer u % 2: thread t takes
    // unit t % 16 of 8 codes of rows t / 16 and 16 higher
    const int rx = tid >> 4, cx = (tid & 15) * 8, slot = p.group ? cx / p.group : 0;
    uint2 code[2];
    float rs[2];
    const auto read_codes = [&](int64_t m, int u) __attribute__((always_inline)) {
        const int left = rows_left(m);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = rx + 16 * h;
            code[h] = *reinterpret_cast<const uint2*>(qb + (u % NB * KS + ks) * kQ + r * 128 + cx);
            const float v = *reinterpret_cast<const float*>(sb + (u % NB * KS + ks) * kS + (r * 8 + slot) * 4);
            rs[h] = r < left ? v : 0.0f;
        }
    };
    const auto restore = [&](int u, int h) __attribute__((always_inline)) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (float)(int8_t)((j < 4 ? code[h].x : code[h].y) >> (8 * (j & 3))) * rs[h];
        uint8_t* dst = xb + (u % XB * KS + ks) * kX + lds_off<BK>(rx + 16 * h, cx);
        if constexpr (SPLIT) {
            uint4 o[PB];
            split8<PB, Md::nearest>(v, o);
#pragma unroll
            for (int i = 0; i < PB; ++i) *reinterpret_cast<uint4*>(dst + i * BK * kStepM * 2) = o[i];
        } else {
            *reinterpret_cast<uint4*>(dst) = F16 ? to_f16(v) : to_bf16(v);
        }
    };
    const auto add_bias = [&](int64_t m, const uint4 f[NI]) __attribute__((always_inline)) {
        if constexpr (BIAS) {
            if (mine) {
                uint4 o = make_uint4(one2, one2, one2, one2);
                if (m + kStepM > m_hi) {   // 0 for the rows past the end
                    const int rows = rows_left(m) - 8 * (lane >> 4);
                    o.x &= (0 < rows ? 0xFFFFu : 0u) | (1 < rows ? 0xFFFF0000u : 0u);
                    o.y &= (2 < rows ? 0xFFFFu : 0u) | (3 < rows ? 0xFFFF0000u : 0u);
                    o.z &= (4 < rows ? 0xFFFFu : 0u) | (5 < rows ? 0xFFFF0000u : 0u);
                    o.w &= (6 < rows ? 0xFFFFu : 0u) | (7 < rows ? 0xFFFF0000u : 0u);
                }
#pragma unroll
                for (int t = 0; t < NI; ++t)
                    if (mine >> t & 1) sum[t >> 1] = mma<F16>(o, f[t], sum[t >> 1]);
            }
        }
    };
    if constexpr (SPLIT) {
        // Three products to each of the other kind: x^ has one buffer, so that two blocks find
        // room on a CU and fill each other's waits, and two barriers a stage.
        request(m_lo - kStepM, 2, 2);
        request(m_lo - kStepM, 2, 3);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) request(m_lo + u * kStepM, u, i);
        asm volatile("s_waitcnt vmcnt(8)\n\ts_barrier" ::: "memory");   // the first codes
        read_codes(m_lo, 0);
        restore(0, 0);
        restore(0, 1);
        int u = 0;
        for (int64_t m = m_lo; m < m_hi; m += kStepM) {
            // this stage's operands and the next one's codes are in LDS; what was read a stage
            // ago is free
            asm volatile("s_waitcnt vmcnt(4) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            uint4 fa[NI], fb[PB][KI];
#pragma unroll
            for (int t = 0; t < NI; ++t) fa[t] = frag_at<BN>(yb + u * kY, wn + 16 * t, lane);
#pragma unroll
            for (int j = 0; j < PB; ++j)
#pragma unroll
                for (int t = 0; t < KI; ++t) fb[j][t] = frag_at<BK>(xb + j * BK * kStepM * 2, wk + 16 * t, lane);
            read_codes(m + kStepM, u + 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) request(m + 2 * kStepM, u + 2, i);
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // x^ is read
            restore(0, 0);
            restore(0, 1);
#pragma unroll
            for (int j = 0; j < PB; ++j)
#pragma unroll
                for (int t = 0; t < NI; ++t)
#pragma unroll
                    for (int b = 0; b < KI; ++b) acc[t][b] = mma<F16>(fa[t], fb[j][b], acc[t][b]);
#pragma unroll
            for (int i = 0; i < 48; ++i) {   // one product, then some of the restoring
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
            }
            add_bias(m, fa);
            u = u == 2 ? 0 : u + 1;
        }
    } else {
        uint4 fa[2][NI], fb[2][KI];   // operands of this stage and the next
        const auto read = [&](int u, int t, uint4 a[NI], uint4 b[KI]) __attribute__((always_inline)) {
            a[t] = frag_at<BN>(yb + (u % NB * KS + ks) * kY, wn + 16 * t, lane);
            b[t] = frag_at<BK>(xb + (u % XB * KS + ks) * kX, wk + 16 * t, lane);
        };
        const auto stage = [&](int64_t m, auto at_buffer) __attribute__((always_inline)) {
            constexpr int u = decltype(at_buffer)::value, c = u & 1;
            // this wave's operands of this stage are in registers, its part of the next stage's and
            // of the codes after those in LDS; behind the barrier that holds for all, and what was
            // read a stage ago is free
            asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            read_codes(m + 2 * step, u + 2);
            // In four parts, each a quarter of the products and, in their shadow, one load (eight
            // waves that issue all their loads at once wait for each other), the reads of a quarter
            // of the next operands and a share of the restoring.
#pragma unroll
            for (int t = 0; t < NI; ++t) {
#pragma unroll
                for (int b = 0; b < KI; ++b) acc[t][b] = mma<F16>(fa[c][t], fb[c][b], acc[t][b]);
                read(u + 1, t, fa[c ^ 1], fb[c ^ 1]);
                request(m + 4 * step, u + 4, t);
                if (t < 2) restore(u + 2, t);
                __builtin_amdgcn_sched_barrier(0);
            }
            add_bias(m, fa[c]);
        };
        const int64_t own = (int64_t)ks * kStepM, m_own = m_lo + own;
        // batches of stages -1 (the first codes), 0, 1 and 2
#pragma unroll
        for (int u = -1; u < 3; ++u)
#pragma unroll
            for (int i = u < 0 ? 2 : 0; i < 4; ++i) request(m_own + u * step, u, i);
        asm volatile("s_waitcnt vmcnt(8)\n\ts_barrier" ::: "memory");   // all but the last two
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            read_codes(m_own + u * step, u);
            restore(u, 0);
            restore(u, 1);
        }
        __syncthreads();
        // batch 3, whose codes take the place of the first
#pragma unroll
        for (int i = 0; i < 4; ++i) request(m_own + 3 * step, 3, i);
#pragma unroll
        for (int t = 0; t < NI; ++t) read(0, t, fa[0], fb[0]);
        // whole rounds of the four buffers, then the rest; a stage that only some sets have rows
        // for is run by all
        int64_t m = m_lo;
        for (; m + 3 * step < m_hi; m += 4 * step) {
            stage(m + own, std::integral_constant<int, 0>());
            stage(m + step + own, std::integral_constant<int, 1>());
            stage(m + 2 * step + own, std::integral_constant<int, 2>());
            stage(m + 3 * step + own, std::integral_constant<int, 3>());
        }
        if (m < m_hi) stage(m + own, std::integral_constant<int, 0>());
        if (m + step < m_hi) stage(m + step + own, std::integral_constant<int, 1>());
        if (m + 2 * step < m_hi) stage(m + 2 * step + own, std::integral_constant<int, 2>());
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing lands in LDS from here on

    if constexpr (KS > 1) {
        // the first set adds the others' sums, in order, a row of 16-wide tiles at a time
        f32x4* red = reinterpret_cast<f32x4*>(xb);   // [KS - 1][KI][256]
        static_assert((KS - 1) * KI * 4096 <= KS * XB * kX && NI == 4, "LDS");
#pragma unroll
        for (int a = 0; a < NI + BIAS; ++a) {
            __syncthreads();
            if (ks > 0) {
                if (a == NI) red[(ks - 1) * 256 + tid] = f32x4{sum[0][0], sum[1][0], 0, 0};
                else
#pragma unroll
                    for (int b = 0; b < KI; ++b) red[((ks - 1) * KI + b) * 256 + tid] = acc[a % NI][b];
            }
            __syncthreads();
            if (ks == 0) {
#pragma unroll
                for (int o = 0; o < KS - 1; ++o) {
                    if (a == NI) {
                        const f32x4 v = red[o * 256 + tid];
#pragma unroll
                        for (int t = 0; t < 2; ++t) sum[t][0] += v[t];
                    } else {
#pragma unroll
                        for (int b = 0; b < KI; ++b) acc[a % NI][b] = acc[a % NI][b] + red[(o * KI + b) * 256 + tid];
                    }
                }
            }
        }
        if (ks > 0) return;
    }
    // lane l of an accumulator holds rows 4 (l / 16) + r, column l % 16
    const bool whole = p.splits == 1;
    float* part = whole ? nullptr : p.part + at.split * p.n * p.k;
#pragma unroll
    for (int a = 0; a < NI; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t n = n0 + wn + 16 * a + 4 * (lane >> 4) + r;
            if (n >= p.n) continue;
#pragma unroll
            for (int b = 0; b < KI; ++b) {
                const int64_t k = k0 + wk + 16 * b + (lane & 15);
                if (k >= p.k) continue;
                if (!whole) part[n * p.k + k] = acc[a][b][r];
                else if (SPLIT) static_cast<float*>(p.dw)[n * p.k + k] = acc[a][b][r];
                else static_cast<T*>(p.dw)[n * p.k + k] = (T)acc[a][b][r];
            }
        }
    if constexpr (BIAS) {
#pragma unroll
        for (int t = 0; t < NI; ++t) {
            const float v = sum[t >> 1][0];
            const int64_t n = n0 + wn + 16 * t + (lane & 15);
            if ((mine >> t & 1) == 0 || lane >= 16 || n >= p.n) continue;
            if (!whole) p.part[p.splits * p.n * p.k + at.split * p.n + n] = v;
            else if (SPLIT) static_cast<float*>(p.db)[n] = v;
            else static_cast<T*>(p.db)[n] = (T)v;
        }
    }
}

// Sums the splits' partial results in order: dW, then (one past it) db.
template <typename O>
__global__ __launch_bounds__(256) void wgrad_join_kernel(const WgradParams p) {
    const int64_t total = p.n * p.k;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e < total) {
        float v = 0.0f;
        for (int64_t s = 0; s < p.splits; ++s) v += p.part[s * total + e];
        static_cast<O*>(p.dw)[e] = (O)v;
    } else if (p.db != nullptr && e - total < p.n) {
        const int64_t c = e - total;
        float v = 0.0f;
        for (int64_t s = 0; s < p.splits; ++s) v += p.part[p.splits * total + s * p.n + c];
        static_cast<O*>(p.db)[c] = (O)v;
    }
}

template <typename T, bool SPLIT>
hipError_t launch_mode(const WgradParams& p, hipStream_t stream) {
    const int64_t blocks = p.n_tiles * p.k_tiles * p.splits;
    if (blocks > kWgradMaxBlocks) return hipErrorInvalidValue;
    const auto go = [&](auto fold, auto tile, auto sets) {
        constexpr bool F = decltype(fold)::value;
        constexpr int TILE = decltype(tile)::value, KS = decltype(sets)::value;
        dim3 g;
        grid_of(blocks, 256 * KS, &g);
        if (p.vec) wgrad_kernel<T, SPLIT, F, TILE, TILE, KS, true><<<g, 256 * KS, 0, stream>>>(p);
        else wgrad_kernel<T, SPLIT, F, TILE, TILE, KS, false><<<g, 256 * KS, 0, stream>>>(p);
    };
    const bool fold = p.group == 0 || p.group % p.tile == 0;   // one scale per row and tile
    const std::true_type yes;
    const std::false_type no;
    typedef std::integral_constant<int, 1> i1;
    typedef std::integral_constant<int, 2> i2;
    typedef std::integral_constant<int, 4> i4;
    // as many sets of waves as LDS holds buffers for (64-wide tiles), or as keep two blocks on
    // a CU (128)
    typedef std::integral_constant<int, 64> t64;
    typedef std::integral_constant<int, 128> t128;
    if constexpr (Mode<T, SPLIT>::pa == 1) {   // dY in one piece
        const auto ring = [&](auto sets) {
            constexpr int KS = decltype(sets)::value;
            const dim3 g((unsigned)blocks);
            if (p.db) wgrad_ring_kernel<T, SPLIT, KS, true><<<g, 256 * KS, 0, stream>>>(p);
            else wgrad_ring_kernel<T, SPLIT, KS, false><<<g, 256 * KS, 0, stream>>>(p);
        };
        if (p.tile == 64) {
            go(no, t64(), i4());
        } else if (!p.ring) {
            if constexpr (SPLIT) go(no, t128(), i1());
            else go(no, t128(), i2());
        } else if constexpr (SPLIT) {
            ring(i1());
        } else {
            // Two blocks on a CU overlap better than two sets of waves behind one barrier
            // (4096^3 bf16: 186 us against 199 us), if there is a second block for each CU
            // (12608 x 4096 x 1024, 256 blocks: 198 us against 149 us).
            if (blocks > 256) ring(i1());
            else ring(i2());
        }
    } else {
        if (p.tile == 64 && fold) go(yes, t64(), i4());
        else if (p.tile == 64) go(no, t64(), i2());
        else if (fold) go(yes, t128(), i1());
        else go(no, t128(), i1());
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t outs = p.n * p.k + (p.db ? p.n : 0);
    const dim3 gj((unsigned)((outs + 255) / 256));
    if (SPLIT) wgrad_join_kernel<float><<<gj, 256, 0, stream>>>(p);
    else wgrad_join_kernel<T><<<gj, 256, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

WgradPlan wgrad_plan(int64_t m, int64_t n, int64_t k, bool f32_out) {
    WgradPlan w;
    const int64_t steps = (m + kStepM - 1) / kStepM;
    const auto tiles_of = [&](int64_t t) { return ((n + t - 1) / t) * ((k + t - 1) / t); };
    // The rows are split so that the 256 CUs are filled about twice, but no split is shorter
    // than 8 stages.  Where that leaves CUs idle, tiles of 64 x 64.
    w.tile = tiles_of(128) * std::max<int64_t>(1, steps / 8) < 256 ? 64 : 128;
    w.n_tiles = (n + w.tile - 1) / w.tile;
    w.k_tiles = (k + w.tile - 1) / w.tile;
    const int64_t tiles = w.n_tiles * w.k_tiles;
    // (float results run two blocks on a CU: 256 tiles of 12608 x 4096 x 1024 bf16 take 402 us
    // unsplit, 316 us split; 16-bit ones, one block of two sets of waves)
    int64_t s = tiles >= (f32_out ? 512 : 256) ? 1 : 512 / tiles;
    if (s > steps / 8) s = steps / 8;
    if (s < 1) s = 1;
    const int64_t per = (steps + s - 1) / s;
    w.rows_per_split = (per ? per : 1) * kStepM;
    w.splits = m ? (m + w.rows_per_split - 1) / w.rows_per_split : 1;
    w.workspace = w.splits == 1 ? 0 : w.splits * (n * k + n) * 4;
    return w;
}

hipError_t launch_wgrad(const WgradParams& p, int32_t dy_type, bool f32_out, hipStream_t stream) {
    switch (dy_type) {
    case F_F32: return launch_mode<float, true>(p, stream);
    case F_F16: return f32_out ? launch_mode<_Float16, true>(p, stream) : launch_mode<_Float16, false>(p, stream);
    default: return f32_out ? launch_mode<__bf16, true>(p, stream) : launch_mode<__bf16, false>(p, stream);
    }
}

}  // namespace iqnn
