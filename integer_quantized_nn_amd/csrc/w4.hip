// w4.hip -- y = x W^T + b with 4-bit weights W = (q - z) * s, one scale (and zero point)
// per group of 32, 64 or 128 consecutive K positions of an output row, or per row.
//
// y[m][n] = sum_g s[n][g] * (sum_{k in g} x[m][k] (q[n][k] - z[n][g])) + b[n]
//
// The weights stay integers on the matrix cores: a 4-bit difference is exact in bf16 and
// in f16, products and the sum over a group are accumulated in binary32 by
// v_mfma_f32_16x16x32, and the group's scale multiplies that sum in binary32.  Nothing
// but the final result is rounded below 32 bits.  f32 activations run as three bf16
// pieces of 8 significand bits each (an exact split), so their products are exact too.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <type_traits>

#include "float_types.h"
#include "iqnn_internal.h"

#pragma clang fp contract(off)

namespace iqnn {

// Packed weights: blocks of 16 output rows x 128 K, block (t, b) of rows 16t.. and K
// 128b.. at (t * kb + b).  A block's codes are 1 KB: lane l = 16 g + i of a wave reads 16
// bytes, row 16t + i, its 32-bit word j holding K 128b + 32j + 8g + 0..7, which is that
// lane's B operand of the 16x16x32 MFMA of step j.
W4Geom w4_geom(int64_t n, int64_t k, int32_t group, bool zp) {
    W4Geom g;
    g.nt = (n + 15) / 16;
    g.kb = (k + 127) / 128;
    g.gpb = group ? 128 / group : 0;
    const int64_t scales = g.nt * 16 * (group ? g.kb * g.gpb : 1);
    g.s_off = g.nt * g.kb * 1024;
    g.z_off = g.s_off + (scales * 4 + 255) / 256 * 256;
    g.bytes = g.z_off + (zp ? (scales + 255) / 256 * 256 : 0);
    return g;
}

W4Choice w4_choice(int64_t m, int64_t n, int32_t gpb, bool f32, bool vec) {
    // Up to 16 rows: one 16-row tile of weights per block, unless there are so many that
    // every CU has three; then four share each block's x where x is what costs (16 x 8192 x
    // 28672 bf16: 36 us against 61 us; 16 x 4096 x 4096: 9.0 us against 6.9 us).
    const bool wide = vec && (n + 15) / 16 >= 768;
    if (m <= 4) {
        if (!f32) return {false, 4, 1, 4};
        return wide ? W4Choice{false, 4, 4, 1} : W4Choice{false, 4, 1, 2};
    }
    if (m <= 16) {
        const int32_t rows = m <= 8 ? 8 : 16;
        return wide ? W4Choice{false, rows, 4, 1} : W4Choice{false, rows, 1, 2};
    }
    // Tiles of 16 rows x 64 nt with sets of waves, by their measured time at K = 4096 per
    // round of blocks that fill the 256 CUs (bf16, group 128): the fewest rounds of a tile
    // that keeps its waves busy.
    const auto rounds = [&](int64_t bm, int64_t bn, int64_t per_round) {
        const int64_t blocks = ((m + bm - 1) / bm) * ((n + bn - 1) / bn);
        return (blocks + per_round - 1) / per_round;
    };
    if (f32)   // three pieces of x: LDS holds 64 rows at most
        return rounds(32, 64, 256) * 21 <= rounds(64, 128, 256) * 55 ? W4Choice{true, 2, 1, 2} : W4Choice{true, 4, 2, 1};
    if (!vec)
        return rounds(64, 64, 256) * 17 <= rounds(64, 128, 256) * 27 ? W4Choice{true, 4, 1, 2} : W4Choice{true, 4, 2, 2};
    // the last one's sums of shorter groups do not fit beside its totals in 256 registers
    const int tiles = gpb <= 1 ? 5 : 4;
    const int64_t us[5] = {rounds(32, 64, 256) * 12, rounds(64, 64, 256) * 17, rounds(64, 128, 256) * 27,
                           rounds(128, 128, 256) * 41, rounds(128, 128, 512) * 74};
    const W4Choice of[5] = {{true, 2, 1, 4}, {true, 4, 1, 4}, {true, 4, 2, 2}, {true, 8, 2, 2}, {true, 8, 2, 1}};
    int best = 0;
    for (int i = 1; i < tiles; ++i)
        if (us[i] < us[best]) best = i;
    return of[best];
}

namespace {

// Which K position (0..7 of a word) nibble i holds.  bf16 and f32 activations: v_cvt_off_f32_i4
// with a byte select converts the low nibbles of bytes 0..3, then the high ones.  f16:
// (w >> 4i) & 0x000F000F holds nibbles i and i + 4, a pair of consecutive elements.
__device__ __forceinline__ int k_of_nibble(bool f16, int i) { return f16 ? (i < 4 ? 2 * i : 2 * (i - 4) + 1) : (i & 1) * 4 + (i >> 1); }

// One 16 x 128 block of weights at a time: thread t reads the eight codes t % 16 of row t / 16
// (64 contiguous bytes a row), puts them in order and leaves them in LDS for a contiguous
// store.
__global__ __launch_bounds__(256) void w4_prepack_kernel(const W4PrepackParams p) {
    __shared__ uint32_t words[256];
    const W4Geom& g = p.g;
    const bool f16 = p.x_type == F_F16;
    const int64_t groups = p.group ? (p.k + p.group - 1) / p.group : 1;
    const int i = threadIdx.x >> 4, c = threadIdx.x & 15;   // K 8c = 32 j + 8 g of the block
    for (int64_t blk = blockIdx.x; blk < g.nt * g.kb; blk += gridDim.x) {
        const int64_t t = blk / g.kb, b = blk - t * g.kb;
        const int64_t n = t * 16 + i, k0 = b * 128 + 8 * c;
        uint32_t w = p.zp ? 0x88888888u : 0;   // padding is the weight 0: its group's zero point, 8 where there is none
        if (n < p.n && k0 + 8 <= p.k) {
            __builtin_memcpy(&w, p.q + (n * p.k + k0) / 2, 4);
        } else if (n < p.n) {
            for (int e = 0; e < 8; ++e) {
                const int64_t k = k0 + e, gi = p.group ? k / p.group : 0;
                uint32_t code;
                if (k < p.k) code = (uint32_t)p.q[(n * p.k + k) >> 1] >> (4 * (k & 1));
                else if (p.zp && gi < groups) code = (uint32_t)p.zp[n * groups + gi];
                else continue;
                w = (w & ~(0xFu << (4 * e))) | ((code & 0xFu) << (4 * e));
            }
        }
        // f16 holds offset codes, the others two's complement
        if (f16 != (p.zp != nullptr)) w ^= 0x88888888u;
        uint32_t out = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) out |= (w >> (4 * (f16 ? k_of_nibble(true, e) : k_of_nibble(false, e))) & 0xFu) << (4 * e);
        __syncthreads();   // the words of the block before are stored
        words[(16 * (c & 3) + i) * 4 + (c >> 2)] = out;
        __syncthreads();
        reinterpret_cast<uint32_t*>(p.packed)[blk * 256 + threadIdx.x] = words[threadIdx.x];
    }
    const int64_t per = g.gpb ? g.gpb : 1, nb = g.gpb ? g.kb : 1;
    float* sp = reinterpret_cast<float*>(p.packed + g.s_off);
    uint8_t* zo = p.packed + g.z_off;
    const int64_t ns = g.nt * nb * 16 * per;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < ns; e += (int64_t)gridDim.x * 256) {
        const int64_t c = e % per, i = (e / per) & 15, b = (e / (per * 16)) % nb, t = e / (per * 16 * nb);
        const int64_t n = t * 16 + i, gi = b * per + c;
        const bool in = n < p.n && gi < groups;
        // bf16 and f32 weights are held as (q - z) / 16
        sp[e] = in ? p.scale[n * groups + gi] * (f16 ? 1.0f : 16.0f) : 0.0f;
        if (p.zp) zo[e] = in ? (uint8_t)(p.zp[n * groups + gi] & 0xF) : 8;
    }
}

// ---- operands -----------------------------------------------------------------------

template <typename T>
struct Traits {   // bf16
    typedef bf16x8 frag;
    static constexpr int pieces = 1;
};
template <>
struct Traits<_Float16> {
    typedef f16x8 frag;
    static constexpr int pieces = 1;
};
template <>
struct Traits<float> {
    typedef bf16x8 frag;
    static constexpr int pieces = 3;
};

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// The zero point of a lane's row in the form weights_of subtracts: z / 16 - 1 / 2 as a
// float, or (16 + z, 16 + z) as an f16 pair.
template <typename T>
__device__ __forceinline__ uint32_t zero_of(uint32_t z) {
    if constexpr (std::is_same<T, _Float16>::value) return 0x4C004C00u + z * 0x00400040u;
    else return as_u32((float)((int)z - 8) * 0.0625f);
}

// Eight weights of one packed word.  f16: the nibble is ORed into the top mantissa bits
// of 16.0 (16 + u, exact) and 16 + z is subtracted, exact.  bf16: the signed nibble is
// converted to a float of sixteenths, whose upper half is its bf16.
template <typename T, bool ASYM>
__device__ __forceinline__ typename Traits<T>::frag weights_of(uint32_t w, uint32_t zero) {
    uint32_t o[4];
    if constexpr (std::is_same<T, _Float16>::value) {
        const uint32_t m[4] = {w << 6, w << 2, w >> 2, w >> 6};
        const f16x2 z = __builtin_bit_cast(f16x2, ASYM ? zero : 0x4E004E00u);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (m[j] & 0x03C003C0u) | 0x4C004C00u) - z);
    } else {
        float f[8];
        uint32_t h = w >> 4;
        asm("" : "+v"(h));   // one shift for four byte selects
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = __builtin_amdgcn_cvt_off_f32_i4((int)((w >> (8 * j)) & 0xFF));
            f[4 + j] = __builtin_amdgcn_cvt_off_f32_i4((int)((h >> (8 * j)) & 0xFF));
        }
        if (ASYM) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f[j] - as_f32(zero);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = __builtin_amdgcn_perm(as_u32(f[2 * j + 1]), as_u32(f[2 * j]), 0x07060302u);
    }
    return __builtin_bit_cast(typename Traits<T>::frag, make_uint4(o[0], o[1], o[2], o[3]));
}

// Eight activations x[row][k0 .. k0+8) as MFMA operands; K and beyond read as 0.  VEC:
// rows start 16-byte aligned and K % 8 == 0, so the eight are all in or all out.
template <bool VEC, typename T>
__device__ __forceinline__ void x_frags(const T* row, int64_t k0, int64_t k, typename Traits<T>::frag a[1]) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (VEC) {
        if (k0 < k) v = *reinterpret_cast<const uint4*>(row + k0);
        a[0] = __builtin_bit_cast(typename Traits<T>::frag, v);
    } else {
        if (k0 + 8 <= k) {
            __builtin_memcpy(&v, row + k0, 16);
        } else {
            Pack8<T> e;
#pragma unroll
            for (int j = 0; j < 8; ++j) e.e[j] = k0 + j < k ? row[k0 + j] : (T)0.0f;
            __builtin_memcpy(&v, &e, 16);
        }
        a[0] = __builtin_bit_cast(typename Traits<T>::frag, v);
    }
}

// f32: three bf16 pieces, each the truncated upper half of what is left (of an infinity,
// NaN: a non-finite x makes its row of y non-finite).
template <bool VEC>
__device__ __forceinline__ void x_frags(const float* row, int64_t k0, int64_t k, bf16x8 a[3]) {
    float v[8];
    if (VEC) {
        if (k0 < k) load8(row + k0, v);
        else
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    } else {
        load_n(row + k0, k - k0 < 8 ? (k - k0 < 0 ? 0 : (int)(k - k0)) : 8, v);
    }
    uint32_t o[3][4];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = __builtin_amdgcn_perm(as_u32(v[2 * j + 1]), as_u32(v[2 * j]), 0x07060302u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] - as_f32(as_u32(v[j]) & 0xFFFF0000u);
        a[i] = __builtin_bit_cast(bf16x8, make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]));
    }
}

// One of a quad's four operands in all four lanes (ML 4), or one of each pair's two in both
// (ML 8), by DPP quad_perm; the operand itself otherwise.
template <int ML, typename F>
__device__ __forceinline__ F spread(F v, int j) {
    if constexpr (ML == 16) return v;
    uint4 u = __builtin_bit_cast(uint4, v);
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
    constexpr int k4[4] = {0x00, 0x55, 0xAA, 0xFF}, k8[2] = {0xA0, 0xF5};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int x = (int)w[c];
        if (ML == 4)
            w[c] = (uint32_t)(j == 0   ? __builtin_amdgcn_mov_dpp(x, k4[0], 0xF, 0xF, true)
                              : j == 1 ? __builtin_amdgcn_mov_dpp(x, k4[1], 0xF, 0xF, true)
                              : j == 2 ? __builtin_amdgcn_mov_dpp(x, k4[2], 0xF, 0xF, true)
                                       : __builtin_amdgcn_mov_dpp(x, k4[3], 0xF, 0xF, true));
        else
            w[c] = (uint32_t)((j & 1) == 0 ? __builtin_amdgcn_mov_dpp(x, k8[0], 0xF, 0xF, true)
                                           : __builtin_amdgcn_mov_dpp(x, k8[1], 0xF, 0xF, true));
    }
    return __builtin_bit_cast(F, make_uint4(w[0], w[1], w[2], w[3]));
}

// ---- few rows: a block owns 16 * NT output rows, its W waves split K -----------------

// The kernel is bound by reading the codes: a wave has the codes of U blocks of K in flight
// and reads each block's 1 KB in one instruction.
//
// Up to ML rows of x (4, 8 or 16).  Row m stands in rows C m .. C m + C - 1 of the MFMA's
// operand, C = 16 / ML, and lane i loads step i % C of every C steps of row i / C: one load
// brings C steps, which spread() hands to the C lanes of the row one by one.  With ML 4 a
// 128-K block of x is one instruction instead of four, and the kernel no longer waits for
// its x (1 x 8192 x 28672, f16 with zero points: 39.4 us with ML 16, 28.5 us with ML 4).
//
// GPB: scales per 128-K block and row (0: one per row, applied at the end).
//
// More blocks than a launch holds along x (2^32 threads) stand in rows of kFewRow.  (A row's
// length from gridDim would be one more load to wait for: 1 x 4096 x 4096 3.7 us, so 3.6 us.)
template <int W>
constexpr int64_t kFewRow = 0xFFFFFFFFll / (W * 64);
template <typename T, bool ASYM, int GPB, int ML, int NT, int W, int U, bool VEC>
__global__ __launch_bounds__(W * 64) void w4_few_kernel(const W4Params p) {
    typedef typename Traits<T>::frag frag;
    constexpr int P = Traits<T>::pieces, S = GPB ? GPB : 1;
    constexpr int C = 16 / ML, X = 4 / C, R = 4 / C;   // loads of x per block; accumulator registers of distinct rows
    __shared__ float red[W][NT][R * 64];
    const int l = threadIdx.x & 63, wave = threadIdx.x >> 6, i = l & 15, g = l >> 4;
    const int64_t t0 = (blockIdx.y * kFewRow<W> + blockIdx.x) * NT;
    if (t0 >= p.g.nt) return;
    const uint4* codes[NT];
    const float* sc[NT];
    const uint8_t* zc[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int64_t t = t0 + nt < p.g.nt ? t0 + nt : p.g.nt - 1;
        codes[nt] = reinterpret_cast<const uint4*>(p.packed) + t * p.g.kb * 64 + l;
        sc[nt] = reinterpret_cast<const float*>(p.packed + p.g.s_off) + (t * (GPB ? p.g.kb : 1) * 16 + i) * S;
        zc[nt] = p.packed + p.g.z_off + (t * (GPB ? p.g.kb : 1) * 16 + i) * S;
    }
    // rows past the last repeat it; their results are not stored
    const int64_t mi = i / C;
    const T* row = static_cast<const T*>(p.x) + (mi < p.m ? mi : p.m - 1) * p.ldx;
    f32x4 acc[NT];
    float tot[NT][R];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        acc[nt] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < R; ++r) tot[nt][r] = 0.0f;
    }
    for (int64_t b0 = wave; b0 < p.g.kb; b0 += U * W) {
        uint4 cw[U][NT];
        frag xa[U][X][P];
        float s[U][NT][S];
        uint32_t z[U][NT][S];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t b = b0 + u * W < p.g.kb ? b0 + u * W : b0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                cw[u][nt] = codes[nt][b * 64];
#pragma unroll
                for (int c = 0; c < S; ++c) {
                    if (GPB) s[u][nt][c] = sc[nt][b * 16 * S + c];
                    z[u][nt][c] = ASYM ? zc[nt][(GPB ? b * 16 * S : 0) + c] : 0;
                }
            }
#pragma unroll
            for (int x = 0; x < X; ++x) x_frags<VEC>(row, b * 128 + 32 * (C * x + i % C) + 8 * g, p.k, xa[u][x]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t b = b0 + u * W;
            if (b >= p.g.kb) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                constexpr int per = GPB ? 4 / GPB : 4;   // MFMA steps per group
                frag a[P];
#pragma unroll
                for (int q = 0; q < P; ++q) a[q] = spread<ML>(xa[u][j / C][q], j % C);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint32_t w = j == 0 ? cw[u][nt].x : (j == 1 ? cw[u][nt].y : (j == 2 ? cw[u][nt].z : cw[u][nt].w));
                    const frag wf = weights_of<T, ASYM>(w, ASYM ? zero_of<T>(z[u][nt][j / per]) : 0);
#pragma unroll
                    for (int q = 0; q < P; ++q) acc[nt] = mfma(a[q], wf, acc[nt]);
                    if (GPB && (j + 1) % per == 0) {
#pragma unroll
                        for (int r = 0; r < R; ++r) tot[nt][r] = __builtin_fmaf(s[u][nt][j / per], acc[nt][r * C], tot[nt][r]);
                        acc[nt] = f32x4{0, 0, 0, 0};
                    }
                }
            }
        }
    }
    // lane l of an accumulator holds operand rows 4g + r, column i: rows R g + r of x
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < R; ++r) red[wave][nt][(R * g + r) * 16 + i] = GPB ? tot[nt][r] : acc[nt][r * C];
    __syncthreads();
    for (int e = threadIdx.x; e < NT * R * 64; e += W * 64) {
        const int nt = e / (R * 64), m = (e / 16) % ML;
        const int64_t n = (t0 + nt) * 16 + (e & 15);
        if (m >= p.m || n >= p.n) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += red[w][nt][e % (R * 64)];
        if (!GPB) v = v * reinterpret_cast<const float*>(p.packed + p.g.s_off)[n];
        if (p.bias) v = v + (float)static_cast<const T*>(p.bias)[n];
        static_cast<T*>(p.y)[m * p.ldy + n] = (T)v;
    }
}

// ---- many rows: 16 * MT rows of x in LDS, shared by four waves of 16 * NT output rows ---

// A stage is one 128-K block of x in one of two LDS buffers; each wave reads its weights'
// codes straight from memory as MFMA operands, unpacks them once per stage and uses them
// for all MT row tiles, whose fragments are read one tile ahead.  16-byte unit c of LDS row
// r sits at c ^ (r & 15), so a fragment read (16 rows, 4 units) meets every bank equally.
//
// A stage is a chain -- unpack, read, multiply, scale -- that one wave per SIMD cannot
// overlap with itself.  Where there are too few tiles for two blocks per CU, KS sets of four
// waves take every KS-th stage each, with buffers of their own, and add up at the end.
//
// DMA (16-bit x in whole vectors): x goes from memory to LDS without registers.  The two
// buffers are separate arrays and the loop runs in pairs of stages, so that the compiler
// can tell the loads into one from the reads of the other.  K past the end rereads the
// row's last unit: the weights there are 0.
template <typename T, bool ASYM, int GPB, int MT, int NT, int KS, bool VEC>
__global__ __launch_bounds__(256 * KS, KS == 1 ? 2 : KS) void w4_tile_kernel(const W4Params p) {
    typedef typename Traits<T>::frag frag;
    typedef __attribute__((address_space(1))) const void* gptr;
    typedef __attribute__((address_space(3))) void* lptr;
    constexpr int P = Traits<T>::pieces, S = GPB ? GPB : 1;
    constexpr int kPlane = MT * 16 * 256;   // bytes of one piece of the stage
    constexpr bool DMA = VEC && sizeof(T) == 2;
    __shared__ __attribute__((aligned(1024))) uint8_t lds0[KS * P * kPlane];
    __shared__ __attribute__((aligned(1024))) uint8_t lds1[KS * P * kPlane];
    const int ks = KS == 1 ? 0 : threadIdx.x >> 8, tid = threadIdx.x & 255;
    const int l = tid & 63, wave = tid >> 6, i = l & 15, g = l >> 4;
    // consecutive blocks go to the eight XCDs in turn: each XCD takes a run of tiles that
    // share their weights
    const int64_t mblk = (p.m + 16 * MT - 1) / (16 * MT);
    const uint32_t G = gridDim.x * gridDim.y, q8 = G / 8, r8 = G % 8, id = (uint32_t)block_id(), xcd = id % 8;
    const int64_t tile = (int64_t)(xcd < r8 ? xcd * (q8 + 1) : r8 * (q8 + 1) + (xcd - r8) * q8) + id / 8;
    const int64_t m0 = (tile % mblk) * 16 * MT, t0 = (tile / mblk) * 4 * NT + wave * NT;

    const uint4* codes[NT];
    const float* sc[NT];
    const uint8_t* zc[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int64_t t = t0 + nt < p.g.nt ? t0 + nt : p.g.nt - 1;
        codes[nt] = reinterpret_cast<const uint4*>(p.packed) + t * p.g.kb * 64 + l;
        sc[nt] = reinterpret_cast<const float*>(p.packed + p.g.s_off) + (t * (GPB ? p.g.kb : 1) * 16 + i) * S;
        zc[nt] = p.packed + p.g.z_off + (t * (GPB ? p.g.kb : 1) * 16 + i) * S;
    }
    // thread tid stages unit tid % 16 of LDS rows 16 t + tid / 16.  DMA puts lane l's 16 bytes
    // at unit l % 16 of its row, so the lane fetches the unit that belongs there.
    const int sr = tid >> 4, su = DMA ? (tid & 15) ^ sr : tid & 15;
    const T* rows[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t r = m0 + t * 16 + sr;   // rows past the last repeat it; their results are not stored
        rows[t] = static_cast<const T*>(p.x) + (r < p.m ? r : p.m - 1) * p.ldx;
    }
    frag st[DMA ? 1 : MT][P];
    uint4 cw[NT];
    float s[NT][S];
    uint32_t z[NT][S];
    const auto request = [&](int64_t b, uint8_t* buf) __attribute__((always_inline)) {
        if constexpr (DMA) {
            int64_t k0 = b * 128 + 8 * su;
            k0 = k0 < p.k ? k0 : p.k - 8;
#pragma unroll
            for (int t = 0; t < MT; ++t)
                __builtin_amdgcn_global_load_lds((gptr)(rows[t] + k0), (lptr)(buf + t * 4096 + wave * 1024), 16, 0, 0);
        } else {
#pragma unroll
            for (int t = 0; t < MT; ++t) x_frags<VEC>(rows[t], b * 128 + 8 * su, p.k, st[t]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            cw[nt] = codes[nt][b * 64];
#pragma unroll
            for (int c = 0; c < S; ++c) {
                if (GPB) s[nt][c] = sc[nt][b * 16 * S + c];
                z[nt][c] = ASYM ? zc[nt][(GPB ? b * 16 * S : 0) + c] : 0;
            }
        }
    };
    f32x4 tot[MT][NT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) tot[t][nt] = f32x4{0, 0, 0, 0};

    uint8_t* const mine0 = lds0 + ks * P * kPlane;
    uint8_t* const mine1 = lds1 + ks * P * kPlane;
    if (ks < p.g.kb) request(ks, mine0);
    // x of stage b is on its way to buf (DMA) or in st, its codes in cw
    const auto stage = [&](int64_t b, uint8_t* buf, uint8_t* next) __attribute__((always_inline)) {
        const bool in = b < p.g.kb;
        frag wf[NT][4];
        float sv[NT][S];
        if (in) {
            if constexpr (!DMA) {
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int q = 0; q < P; ++q)
                        *reinterpret_cast<frag*>(buf + q * kPlane + t * 4096 + sr * 256 + ((su ^ sr) << 4)) = st[t][q];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint32_t w[4] = {cw[nt].x, cw[nt].y, cw[nt].z, cw[nt].w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    wf[nt][j] = weights_of<T, ASYM>(w[j], ASYM ? zero_of<T>(z[nt][GPB ? j * GPB / 4 : 0]) : 0);
#pragma unroll
                for (int c = 0; c < S; ++c) sv[nt][c] = GPB ? s[nt][c] : 0.0f;
            }
        }
        // this wave's direct loads have landed (nothing later is in flight yet); behind the
        // barrier buf is complete, and next, last read a stage ago, may be filled again
        if constexpr (DMA) __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
        __syncthreads();
        if (!in) return;
        if (b + KS < p.g.kb) request(b + KS, next);
        frag af[2][4][P];
        const auto read = [&](int t, frag a[4][P]) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int q = 0; q < P; ++q)
                    a[j][q] = *reinterpret_cast<const frag*>(buf + q * kPlane + t * 4096 + i * 256 + (((4 * j + g) ^ i) << 4));
        };
        read(0, af[0]);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if (t + 1 < MT) read(t + 1, af[(t + 1) & 1]);
            __builtin_amdgcn_sched_barrier(0);   // else the reads sink to just before their use
            f32x4 acc[NT];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                constexpr int per = GPB ? 4 / GPB : 4;   // MFMA steps per group
                if (j % per == 0) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) acc[nt] = GPB ? f32x4{0, 0, 0, 0} : tot[t][nt];
                }
#pragma unroll
                for (int q = 0; q < P; ++q)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) acc[nt] = mfma(af[t & 1][j][q], wf[nt][j], acc[nt]);
                if ((j + 1) % per == 0) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            tot[t][nt][r] = GPB ? __builtin_fmaf(sv[nt][j / per], acc[nt][r], tot[t][nt][r]) : acc[nt][r];
                }
            }
        }
    };
    for (int64_t b = 0; b < p.g.kb; b += 2 * KS) {
        stage(b + ks, mine0, mine1);
        if (b + KS < p.g.kb) stage(b + KS + ks, mine1, mine0);
    }
    if constexpr (KS > 1) {
        // the first set adds the others' sums, in order, one column tile at a time
        f32x4* red = reinterpret_cast<f32x4*>(lds0);   // [KS - 1][MT][256]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            __syncthreads();
            if (ks > 0) {
#pragma unroll
                for (int t = 0; t < MT; ++t) red[((ks - 1) * MT + t) * 256 + tid] = tot[t][nt];
            }
            __syncthreads();
            if (ks == 0) {
#pragma unroll
                for (int o = 0; o < KS - 1; ++o)
#pragma unroll
                    for (int t = 0; t < MT; ++t) tot[t][nt] = tot[t][nt] + red[(o * MT + t) * 256 + tid];
            }
        }
        if (ks > 0) return;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int64_t n = (t0 + nt) * 16 + i;
        if (n >= p.n) continue;
        const float row_scale = GPB ? 1.0f : sc[nt][0];
        const float bias = p.bias ? (float)static_cast<const T*>(p.bias)[n] : 0.0f;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t m = m0 + t * 16 + 4 * g + r;
                if (m < p.m) static_cast<T*>(p.y)[m * p.ldy + n] = (T)(tot[t][nt][r] * row_scale + bias);
            }
    }
}

template <typename T, bool ASYM, int GPB, bool VEC>
hipError_t launch_rows(const W4Params& p, hipStream_t stream) {
    const auto few = [&](auto ml, auto nt, auto w, auto u) {
        constexpr int ML = decltype(ml)::value, NT = decltype(nt)::value, W = decltype(w)::value, U = decltype(u)::value;
        const int64_t blocks = (p.g.nt + NT - 1) / NT, rows = (blocks + kFewRow<W> - 1) / kFewRow<W>;
        const dim3 grid((unsigned)(rows == 1 ? blocks : kFewRow<W>), (unsigned)rows);
        w4_few_kernel<T, ASYM, GPB, ML, NT, W, U, VEC><<<grid, W * 64, 0, stream>>>(p);
        return hipGetLastError();
    };
    const auto tile = [&](auto mt, auto nt, auto ks) {
        constexpr int MT = decltype(mt)::value, NT = decltype(nt)::value, KS = decltype(ks)::value;
        dim3 grid;
        const hipError_t e = grid_of(((p.m + 16 * MT - 1) / (16 * MT)) * ((p.g.nt + 4 * NT - 1) / (4 * NT)), 256 * KS, &grid);
        if (e != hipSuccess) return e;
        w4_tile_kernel<T, ASYM, GPB, MT, NT, KS, VEC><<<grid, 256 * KS, 0, stream>>>(p);
        return hipGetLastError();
    };
    typedef std::integral_constant<int, 1> i1;
    typedef std::integral_constant<int, 2> i2;
    typedef std::integral_constant<int, 4> i4;
    typedef std::integral_constant<int, 8> i8;
    typedef std::integral_constant<int, 16> i16;
    constexpr bool F32 = std::is_same<T, float>::value;
    const W4Choice c = w4_choice(p.m, p.n, GPB, F32, VEC);
    if (!c.tile) {
        if (c.rows == 4) {
            if constexpr (!F32) return few(i4(), i1(), i8(), i4());
            else if (c.nt == 1) return few(i4(), i1(), i8(), i2());
            else if constexpr (VEC) return few(i4(), i4(), i8(), i1());
        } else if (c.rows == 8) {
            if (c.nt == 1) return few(i8(), i1(), i8(), i2());
            else if constexpr (VEC) return few(i8(), i4(), i8(), i1());
        } else {
            if (c.nt == 1) return few(i16(), i1(), i8(), i2());
            else if constexpr (VEC) return few(i16(), i4(), i8(), i1());
        }
    } else if constexpr (F32) {
        return c.rows == 2 ? tile(i2(), i1(), i2()) : tile(i4(), i2(), i1());
    } else if constexpr (!VEC) {
        return c.nt == 1 ? tile(i4(), i1(), i2()) : tile(i4(), i2(), i2());
    } else {
        if (c.rows == 2) return tile(i2(), i1(), i4());
        if (c.rows == 4) return c.nt == 1 ? tile(i4(), i1(), i4()) : tile(i4(), i2(), i2());
        if constexpr (GPB <= 1) {
            if (c.sets == 1) return tile(i8(), i2(), i1());
        }
        return tile(i8(), i2(), i2());
    }
    return hipErrorInvalidValue;   // no such form of w4_choice
}

template <typename T, bool ASYM>
hipError_t launch_typed(const W4Params& p, hipStream_t stream) {
    const auto go = [&](auto gpb) {
        constexpr int GPB = decltype(gpb)::value;
        return p.vec ? launch_rows<T, ASYM, GPB, true>(p, stream) : launch_rows<T, ASYM, GPB, false>(p, stream);
    };
    switch (p.g.gpb) {
    case 0: return go(std::integral_constant<int, 0>());
    case 1: return go(std::integral_constant<int, 1>());
    case 2: return go(std::integral_constant<int, 2>());
    default: return go(std::integral_constant<int, 4>());
    }
}

}  // namespace

hipError_t launch_w4_prepack(const W4PrepackParams& p, hipStream_t stream) {
    const int64_t blocks = p.g.nt * p.g.kb;
    w4_prepack_kernel<<<dim3((unsigned)(blocks < 65536 ? blocks : 65536)), 256, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_w4(const W4Params& p, int32_t x_type, bool asym, hipStream_t stream) {
    switch (x_type) {
    case F_F32: return asym ? launch_typed<float, true>(p, stream) : launch_typed<float, false>(p, stream);
    case F_F16: return asym ? launch_typed<_Float16, true>(p, stream) : launch_typed<_Float16, false>(p, stream);
    default: return asym ? launch_typed<__bf16, true>(p, stream) : launch_typed<__bf16, false>(p, stream);
    }
}

}  // namespace iqnn
