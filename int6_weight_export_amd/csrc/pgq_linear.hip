// pgq_linear.hip -- the quantized linear layer (gfx950): Y = act(X What^T + b) + R and its gradient.
//
// What[n][k] = bf16(fp32(code[n][k] * s_n)), the STE forward's weight ("SubSixteen v2" card, PR #69,
// section Other).  Three products:
//     Z [m][n] = sum_k X[m][k]  What[n][k]          (forward)
//     dX[m][k] = sum_n dZ[m][n] What[n][k]          dZ = dY * act'(Z)
//     dW[n][k] = sum_m dZ[m][n] X[m][k]
// Products of two bf16 values are exact in fp32; every sum is held in fp32.
//
// dZ is a binary32 value, the matrix cores take bf16: it enters the products as the sum of one to three bf16 parts,
// as many as keep what is lost of it far below the outputs' own rounding (dz_parts), each part a product of its
// own on the same sums.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "pgq_desc.h"
#include "pgq_linear.h"
#include "pgq_train.h"
#include "../../include/pgq.h"

namespace pgq {
namespace {

#define GLB __attribute__((address_space(1)))

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

enum Product { P_FWD, P_DX, P_DW };

// One part of a value, and what is left of it for the next: 8 bits cut off (so that the rest keeps the value's sign
// and nothing overflows), the last part rounded to nearest.  Where the value ends before its last part the rest
// goes on as 2^-40 of the value: a part of 0 would make NaN of an infinite weight or input, one of the other sign
// would take its infinity away.  (Below 2^-93 that underflows, and an infinity there may still become NaN.)
__device__ __forceinline__ uint16_t next_part(float value, float& rest, bool last)
{
    const uint32_t bits = __builtin_bit_cast(uint32_t, rest);
    const uint16_t part = last || rest != rest ? f32_to_bf16(rest) : (uint16_t)(bits >> 16);
    rest = fabsf(value) < INFINITY ? rest - bf16_to_f32(part) : value;
    if (rest == 0.0f) rest = value * 0x1p-40f;
    return part;
}
__device__ __forceinline__ uint16_t part_of(float value, int part, int parts)
{
    float rest = value;
    uint16_t h = 0;
    for (int i = 0; i <= part; ++i) h = next_part(value, rest, i + 1 == parts);
    return h;
}

// dZ in fp32 (m, n)
__device__ __forceinline__ float dz_at(const pgq_linear_bwd& b, int64_t m, int64_t n)
{
    const float g = load_any(b.dy, b.dy_dtype, m * b.lddy + n);
    return b.act == PGQ_ACT_NONE ? g : g * act_slope(b.act, b.slope, bf16_to_f32(b.z[m * b.ldz + n]));
}

// One 64 x 64 tile of a product per workgroup of four wavefronts, 32 x 32 each: element loads through
// registers into LDS, any shape and stride.
constexpr int kGT = 64, kGK = 32, kGPad = kGK + 8;

template <int P>
__global__ void __launch_bounds__(256) pgq_linear_tile_kernel(pgq_linear_fwd f, pgq_linear_bwd b, int32_t parts)
{
    __shared__ __align__(16) uint16_t As[kGT][kGPad];
    __shared__ __align__(16) uint16_t Bs[kGT][kGPad];
    const int64_t I = P == P_FWD ? f.M : P == P_DX ? b.M : b.N;
    const int64_t J = P == P_FWD ? f.N : b.K;
    const int64_t L = P == P_FWD ? f.K : P == P_DX ? b.N : b.M;
    const int64_t gx = (J + kGT - 1) / kGT;
    const int64_t i0 = (int64_t)blockIdx.x / gx * kGT, j0 = (int64_t)blockIdx.x % gx * kGT;
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wi = (wave >> 1) * 32, wj = (wave & 1) * 32;
    auto what = [&](const int8_t* codes, int64_t ldc, const uint16_t* scales, int64_t n, int64_t k) {
        return f32_to_bf16((float)codes[n * ldc + k] * f16_to_f32(scales[n]));
    };
    auto load_a = [&](int64_t i, int64_t l, int part) -> uint16_t {
        if (i >= I || l >= L) return 0;
        if (P == P_FWD) return f.x[i * f.ldx + l];
        return part_of(P == P_DX ? dz_at(b, i, l) : dz_at(b, l, i), part, parts);
    };
    auto load_b = [&](int64_t j, int64_t l) -> uint16_t {
        if (j >= J || l >= L) return 0;
        if (P == P_FWD) return what(f.codes, f.ldc, f.scales, j, l);
        return P == P_DX ? what(b.codes, b.ldc, b.scales, l, j) : b.x[l * b.ldx + j];
    };
    f32x16 acc = {};
    for (int64_t l0 = 0, part = 0; l0 < L; part + 1 < parts ? ++part : (part = 0, l0 += kGK)) {
        __syncthreads();
        for (int e = tid; e < kGT * kGK; e += 256) {
            // the thread order follows the contiguous index of each operand
            const int r = P == P_DW ? e % kGT : e / kGK, l = P == P_DW ? e / kGT : e % kGK;
            As[r][l] = load_a(i0 + r, l0 + l, (int)part);
        }
        for (int e = tid; e < kGT * kGK; e += 256) {
            const int r = P == P_FWD ? e / kGK : e % kGT, l = P == P_FWD ? e % kGK : e / kGT;
            Bs[r][l] = load_b(j0 + r, l0 + l);
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kGK; kk += 16) {
            const int ko = kk + 8 * (lane >> 5);
            const bf16x8 a = *reinterpret_cast<const bf16x8*>(&As[wi + (lane & 31)][ko]);
            const bf16x8 w = *reinterpret_cast<const bf16x8*>(&Bs[wj + (lane & 31)][ko]);
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, w, acc, 0, 0, 0);
        }
    }
    const int64_t j = j0 + wj + (lane & 31);
    if (j >= J) return;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int64_t i = i0 + wi + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        if (i >= I) continue;
        if (P == P_FWD) {
            const float z = f.bias ? acc[r] + load_any(f.bias, f.bias_dtype, j) : acc[r];
            if (f.z) f.z[i * f.ldz + j] = f32_to_bf16(z);
            float y = act_value(f.act, f.slope, z);
            if (f.residual) y += load_any(f.residual, f.residual_dtype, i * f.ldr + j);
            store_any(f.y, f.y_dtype, i * f.ldy + j, y);
        } else if (P == P_DX) {
            store_any(b.dx, b.dx_dtype, i * b.lddx + j, acc[r]);
        } else {
            const bool keep = !b.mask || ((b.mask[i * ((b.K + 7) / 8) + j / 8] >> (j % 8)) & 1);
            store_any(b.dw, b.dw_dtype, i * b.lddw + j, keep ? acc[r] : 0.0f);
        }
    }
}

// the same for values that this call reads once
__device__ __forceinline__ u32x4 load16_once(const void* p)
{
    typedef u32x4 any_u32x4 __attribute__((aligned(2)));
    return __builtin_nontemporal_load((const GLB any_u32x4*)p);
}
__device__ __forceinline__ uint64_t load8(const void* p)
{
    uint64_t v;
    __builtin_memcpy(&v, p, 8);
    return v;
}
__device__ __forceinline__ uint32_t pk_bf16(float a, float b) { return (uint32_t)f32_to_bf16(a) | ((uint32_t)f32_to_bf16(b) << 16); }

// ---- operands laid out for the matrix products --------------------------------------------------------
// One launch prepares everything the products of a call read: dZ (and the partial sums of db), What as bf16
// rows (forward) or transposed (dX), and a copy of X with 16-byte aligned rows where X has none.  Rows are
// padded to 8 elements with zeros, their strides to whole cache lines.  What is formed once here instead of in every tile: it is small beside X
// and Y, and its conversion from codes cost the matrix kernel about a sixth of its time.
constexpr int kDzCols = 256;                   // columns of a dZ unit
constexpr int kFlat = 256;                     // granules (8 elements) of a flat unit, one a thread

struct Prep {
    pgq_linear_bwd b;            // the sources (codes, scales, x and their strides also in forward)
    uint16_t* dz;                // M x (parts x Np), row stride ldn, or NULL: only the partial sums
    int32_t parts;               // of dZ
    float* dbias_part;           // ceil(M / dz_rows) x N, or NULL
    int32_t dz_rows;             // rows of a dZ unit
    uint16_t* what;              // N x Kp, row stride ldk
    uint16_t* what_t;            // K x Np, row stride ldt
    uint16_t* xc;                // M x Kp, row stride ldk
    int64_t Kp, Np, ldk, ldn, ldt;
    int64_t n_dz, n_what, n_what_t, n_x;      // units of each kind, in this order
};

// two bf16 of a word as fp32
__device__ __forceinline__ void unpack2(uint32_t w, float* f)
{
    f[0] = __builtin_bit_cast(float, w << 16);
    f[1] = __builtin_bit_cast(float, w & 0xFFFF0000u);
}

// 16 bytes holding E consecutive values of a row from column n on, with zeros past column N: past the edge the
// row's last 16 bytes are loaded and shifted down; rows shorter than that go element by element.
template <int E, typename T>
__device__ __forceinline__ u32x4 load_cols(const T* row, int64_t n, int64_t N)
{
    if (n + E <= N) return load16_once(row + n);
    u32x4 v = {};
    if (n >= N) return v;
    if (N >= E) {
        const int bits = (int)(n + E - N) * (128 / E);         // 1 .. E - 1 values
        uint64_t w[2];
        v = load16(row + N - E);
        __builtin_memcpy(w, &v, 16);
        w[0] = bits < 64 ? (w[0] >> bits) | (w[1] << (64 - bits)) : w[1] >> (bits - 64);
        w[1] = bits < 64 ? w[1] >> bits : 0;
        __builtin_memcpy(&v, w, 16);
        return v;
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (n + e < N) {
            const uint32_t x = E == 8 ? (uint32_t)(uint16_t)row[n + e] : (uint32_t)row[n + e];
            if (E == 8) v[e / 2] |= x << (16 * (e % 2));
            else v[e] = x;
        }
    return v;
}

// A thread takes 8 columns of every eighth row of the unit, the loads of kHold rows issued together (rows past M
// repeat the last one and are not used).  Short loops: a small call runs this code cold, and straight-line
// code for all eight rows cost 20 us of instruction fetch.
template <bool F32, bool ACT>
__device__ __forceinline__ void prep_dz(const Prep& p, int64_t unit, float* sums)
{
    constexpr int kHold = 2;
    const pgq_linear_bwd& b = p.b;
    const int64_t cu = (p.Np + kDzCols - 1) / kDzCols;
    const int64_t rb = unit / cu, n = unit % cu * kDzCols + ((int)threadIdx.x & 31) * 8;
    const int phase = (int)threadIdx.x >> 5;
    float t[8] = {};
    if (n < p.Np) {
#pragma unroll 1
        for (int k0 = 0; k0 < p.dz_rows / 8; k0 += kHold) {
            u32x4 v[kHold][F32 ? 2 : 1], zv[kHold];
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
                const int64_t m = min(rb * p.dz_rows + phase + 8 * (k0 + k), b.M - 1);
                if constexpr (F32) {
                    const uint32_t* row = (const uint32_t*)b.dy + m * b.lddy;
                    v[k][0] = load_cols<4>(row, n, b.N);
                    v[k][1] = load_cols<4>(row, n + 4, b.N);
                } else {
                    v[k][0] = load_cols<8>((const uint16_t*)b.dy + m * b.lddy, n, b.N);
                }
                if constexpr (ACT) zv[k] = load_cols<8>(b.z + m * b.ldz, n, b.N);
            }
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
                const int64_t m = rb * p.dz_rows + phase + 8 * (k0 + k);
                float d[8];
                if constexpr (F32) {
                    const f32x4 lo = __builtin_bit_cast(f32x4, v[k][0]), hi = __builtin_bit_cast(f32x4, v[k][1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) { d[e] = lo[e]; d[4 + e] = hi[e]; }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) unpack2(v[k][0][e], d + 2 * e);
                }
                if constexpr (ACT) {                          // (in the padding dY is 0 and the slope of Z = 0 finite)
                    float z[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) unpack2(zv[k][e], z + 2 * e);
                    if (b.act == PGQ_ACT_SILU) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) d[e] *= act_slope(PGQ_ACT_SILU, 0.0f, z[e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float g = act_slope(PGQ_ACT_RELU, b.slope, z[e]);
                            d[e] *= b.act == PGQ_ACT_RELU ? g : 2.0f * z[e] * g * g;
                        }
                    }
                }
                if (m < b.M) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) t[e] += d[e];
                    if (p.dz && p.parts == 1) {
                        *(GLB u32x4*)(p.dz + m * p.ldn + n) = u32x4{pk_bf16(d[0], d[1]), pk_bf16(d[2], d[3]), pk_bf16(d[4], d[5]), pk_bf16(d[6], d[7])};
                    } else if (p.dz) {
                        float rest[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) rest[e] = d[e];
#pragma unroll 1
                        for (int part = 0; part < p.parts; ++part) {
                            uint32_t h[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) h[e] = next_part(d[e], rest[e], part + 1 == p.parts);
                            *(GLB u32x4*)(p.dz + m * p.ldn + part * p.Np + n) = u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
                        }
                    }
                }
            }
        }
    }
    if (!p.dbias_part) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[phase * kDzCols + ((int)threadIdx.x & 31) * 8 + e] = t[e];
    __syncthreads();
    const int64_t c = unit % cu * kDzCols + threadIdx.x;
    if (c < b.N) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) v += sums[k * kDzCols + threadIdx.x];
        p.dbias_part[rb * b.N + c] = v;
    }
}

__device__ __forceinline__ void prep_what_t(const Prep& p, int64_t unit, uint16_t* t)
{
    constexpr int kPitch = 64 + 8;
    const pgq_linear_bwd& b = p.b;
    const int64_t nu = (p.Np + 63) / 64;
    const int64_t n0 = unit % nu * 64, k0 = unit / nu * 64;
    const int tid = (int)threadIdx.x;
    {
        const int64_t n = n0 + (tid >> 2), k = k0 + (tid & 3) * 16;
        int8_t q[16] = {};
        float s = 0.0f;
        if (n < b.N) {
            s = f16_to_f32(b.scales[n]);
            if (k + 16 <= b.K) {
                const u32x4 v = load16(b.codes + n * b.ldc + k);
                __builtin_memcpy(q, &v, 16);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) q[e] = b.codes[n * b.ldc + min(k + e, b.K - 1)];      // columns past K are not stored
            }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) t[((tid & 3) * 16 + e) * kPitch + (tid >> 2)] = n < b.N ? f32_to_bf16((float)q[e] * s) : (uint16_t)0;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int r = (tid >> 3) + 32 * c, g = tid & 7;
        const int64_t k = k0 + r, n = n0 + 8 * g;
        if (k < b.K && n < p.Np) *(GLB u32x4*)(p.what_t + k * p.ldt + n) = *reinterpret_cast<const u32x4*>(t + r * kPitch + 8 * g);
    }
}

__global__ void __launch_bounds__(256) pgq_linear_prep_kernel(Prep p)
{
    __shared__ __align__(16) float lds[8 * kDzCols];
    __shared__ __align__(16) uint16_t tr[64 * 72];
    int64_t unit = blockIdx.x;
    if (unit < p.n_dz) {
        const bool act = p.b.act != PGQ_ACT_NONE;
        if (p.b.dy_dtype == PGQ_F32) return act ? prep_dz<true, true>(p, unit, lds) : prep_dz<true, false>(p, unit, lds);
        return act ? prep_dz<false, true>(p, unit, lds) : prep_dz<false, false>(p, unit, lds);
    }
    unit -= p.n_dz;
    if (unit < p.n_what_t) return prep_what_t(p, unit, tr);
    unit -= p.n_what_t;
    const bool what = unit < p.n_what;
    if (!what) unit -= p.n_what;
    const pgq_linear_bwd& b = p.b;
    const int64_t g = p.Kp / 8, rows = what ? b.N : b.M;
    const int64_t i = unit * kFlat + threadIdx.x;
    if (i >= rows * g) return;
    int64_t r, k;
    if (rows * g <= 0xFFFFFFFFll) {                       // (a 64-bit division costs as much as the rest)
        r = (uint32_t)i / (uint32_t)g;
        k = ((uint32_t)i - (uint32_t)r * (uint32_t)g) * 8;
    } else {
        r = i / g;
        k = i % g * 8;
    }
    u32x4 o;
    if (what) {
        const float s = f16_to_f32(b.scales[r]);
        const int8_t* src = b.codes + r * b.ldc + k;
        int8_t q[8] = {};
        if (k + 8 <= b.K) {
            const uint64_t v = load8(src);
            __builtin_memcpy(q, &v, 8);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int8_t v = src[min((int64_t)e, b.K - 1 - k)];
                q[e] = k + e < b.K ? v : (int8_t)0;
            }
        }
        // padding is 0 whatever the scale is
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pk_bf16(k + 2 * e < b.K ? (float)q[2 * e] * s : 0.0f, k + 2 * e + 1 < b.K ? (float)q[2 * e + 1] * s : 0.0f);
        *(GLB u32x4*)(p.what + r * p.ldk + k) = o;
    } else {
        o = load_cols<8>(b.x + r * b.ldx, k, b.K);
        *(GLB u32x4*)(p.xc + r * p.ldk + k) = o;
    }
}

// ---- few tokens -----------------------------------------------------------------------------------
// Up to 64 tokens: the codes are the traffic (N K bytes), each read once.  A workgroup takes 16 weight rows;
// its eight wavefronts take 64-wide blocks of K in turn, so that a wavefront's loads cover 64 contiguous
// codes of each row, and their sums are joined through LDS.  v_mfma_f32_16x16x32_bf16 with the weights as A
// (row lane % 16, k = 8 (lane / 16) .. + 7) and the tokens as B (column lane % 16): lane quarter q supplies
// k = 16 q + 8 t .. + 7 of a block in instruction t, so that a lane's 16 codes are one load.  Lanes past M
// or N repeat the last row, whose sums they do not store.
//
// A compute unit takes 0.3 us (one token) to 1.9 us (64) for eight blocks, so few weight rows with long K are cut
// into parts of K: their sums go to scratch and a second launch adds them in order (16 x 256 x 8192 13.2 -> 8.4 us,
// 19 x 224 x 6176 with rows at odd addresses 29 -> 10).
constexpr int kSkinnyMost = 64;
constexpr int kSkinnyWaves = 8;

struct Parts {
    float* sums;                 // n > 1: n x M x N
    int64_t blocks;              // 64-wide blocks of K in a part
    int32_t n;
};

__device__ __forceinline__ void finish(const pgq_linear_fwd& f, int64_t m, int64_t n, float z)
{
    if (f.bias) z += load_any(f.bias, f.bias_dtype, n);
    if (f.z) f.z[m * f.ldz + n] = f32_to_bf16(z);
    float y = act_value(f.act, f.slope, z);
    if (f.residual) y += load_any(f.residual, f.residual_dtype, m * f.ldr + n);
    store_any(f.y, f.y_dtype, m * f.ldy + n, y);
}

template <int MB>
__global__ void __launch_bounds__(64 * kSkinnyWaves) pgq_linear_skinny_kernel(pgq_linear_fwd f, Parts parts)
{
    __shared__ f32x4 sums[kSkinnyWaves][MB][64];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int r = lane & 15, q = lane >> 4;
    const uint32_t part = blockIdx.x % (uint32_t)parts.n;
    const int64_t n0 = (int64_t)(blockIdx.x / (uint32_t)parts.n) * 16;
    const int64_t n = min(n0 + r, f.N - 1);
    const int8_t* crow = f.codes + n * f.ldc + 16 * q;
    const uint16_t* xrow[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) xrow[i] = f.x + min((int64_t)(16 * i + r), f.M - 1) * f.ldx + 16 * q;
    const float s = f.K > 0 ? f16_to_f32(f.scales[n]) : 0.0f;
    f32x4 acc[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[i] = f32x4{};
    auto multiply = [&](u32x4 c, const u32x4 (*x)[2], int left = 16) __attribute__((always_inline)) {
        float v[16];                                      // code * s exactly (at most 7 + 11 significant bits)
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[4 * w + e] = (float)(int8_t)(c[w] >> (8 * e)) * s;
                if (4 * w + e >= left) v[4 * w + e] = 0.0f;        // (0 * s is NaN for an infinite s)
            }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const u32x4 a = {pk_bf16(v[8 * t], v[8 * t + 1]), pk_bf16(v[8 * t + 2], v[8 * t + 3]),
                             pk_bf16(v[8 * t + 4], v[8 * t + 5]), pk_bf16(v[8 * t + 6], v[8 * t + 7])};
#pragma unroll
            for (int i = 0; i < MB; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, x[i][t]), acc[i], 0, 0, 0);
        }
    };
    const bool last = part + 1 == (uint32_t)parts.n;
    const int64_t full = last ? f.K / 64 : (part + 1) * parts.blocks;       // one past this part's whole blocks
    constexpr int U = MB == 1 ? 8 : MB == 2 ? 4 : 2;      // blocks whose loads are in flight together
    int64_t kb = part * parts.blocks + wave;
    for (; kb + (int64_t)(U - 1) * kSkinnyWaves < full; kb += (int64_t)U * kSkinnyWaves) {
        u32x4 c[U], x[U][MB][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = (kb + (int64_t)u * kSkinnyWaves) * 64;
            c[u] = load16(crow + k);
#pragma unroll
            for (int i = 0; i < MB; ++i) { x[u][i][0] = load16(xrow[i] + k); x[u][i][1] = load16(xrow[i] + k + 8); }
        }
        __builtin_amdgcn_sched_barrier(0);                // every load is issued before the first use
#pragma unroll
        for (int u = 0; u < U; ++u) multiply(c[u], x[u]);
    }
    for (; kb < full; kb += kSkinnyWaves) {
        const int64_t k = kb * 64;
        u32x4 x[MB][2];
        const u32x4 c = load16(crow + k);
#pragma unroll
        for (int i = 0; i < MB; ++i) { x[i][0] = load16(xrow[i] + k); x[i][1] = load16(xrow[i] + k + 8); }
        multiply(c, x);
    }
    if (last && f.K % 64 && kb == full) {                 // the last block, element by element past K
        const int64_t k = full * 64;
        const int left = (int)max((int64_t)0, min((int64_t)16, f.K - k - 16 * q));
        union { u32x4 v; uint8_t b[16]; } c = {};
        union { u32x4 v[2]; uint16_t h[16]; } x[MB] = {};
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (e < left) {
                c.b[e] = (uint8_t)crow[k + e];
#pragma unroll
                for (int i = 0; i < MB; ++i) x[i].h[e] = xrow[i][k + e];
            }
        u32x4 xv[MB][2];
#pragma unroll
        for (int i = 0; i < MB; ++i) { xv[i][0] = x[i].v[0]; xv[i][1] = x[i].v[1]; }
        multiply(c.v, xv, left);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) sums[wave][i][lane] = acc[i];
    __syncthreads();
    // accumulator element e of lane l: weight row 4 (l / 16) + e, token l % 16
    for (int u = (int)threadIdx.x; u < 64 * MB * 4; u += 64 * kSkinnyWaves) {
        const int e = u & 3, l = (u >> 2) & 63, i = u >> 8;
        const int64_t m = 16 * i + (l & 15), nn = n0 + 4 * (l >> 4) + e;
        if (m >= f.M || nn >= f.N) continue;
        float z = sums[0][i][l][e];
#pragma unroll
        for (int w = 1; w < kSkinnyWaves; ++w) z += sums[w][i][l][e];
        if (parts.n > 1) parts.sums[(part * f.M + m) * f.N + nn] = z;
        else finish(f, m, nn, z);
    }
}

__global__ void __launch_bounds__(256) pgq_linear_join_kernel(pgq_linear_fwd f, Parts parts)
{
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, mn = f.M * f.N;
    if (at >= mn) return;
    const GLB float* src = (const GLB float*)parts.sums + at;
    float z = src[0];
#pragma unroll 8
    for (int i = 1; i < parts.n; ++i) z += src[i * mn];
    finish(f, at / f.N, at % f.N, z);
}

pgq_status check_fwd(const pgq_linear_fwd* p)
{
    if (!p) return PGQ_ERR_NULL;
    const int64_t M = p->M, N = p->N, K = p->K;
    if (M < 0 || N < 0 || K < 0 || M > kMaxSize || N > kMaxSize || K > kMaxSize) return PGQ_ERR_SHAPE;
    if (p->ldx < K || p->ldc < K || p->ldy < N || (p->residual && p->ldr < N) || (p->z && p->ldz < N)) return PGQ_ERR_SHAPE;
    if (!float_type(p->y_dtype) || (p->bias && !float_type(p->bias_dtype)) ||
        (p->residual && !float_type(p->residual_dtype)))
        return PGQ_ERR_DTYPE;
    if (!act_ok(p->act, p->slope) || p->reserved != 0) return PGQ_ERR_PARAM;
    if (M == 0 || N == 0) return PGQ_OK;
    if (!p->y || (K > 0 && (!p->x || !p->codes || !p->scales))) return PGQ_ERR_NULL;
    if (!is_aligned(p->y, float_size(p->y_dtype)) || (p->x && !is_aligned(p->x, 2)) ||
        (p->scales && !is_aligned(p->scales, 2)) || (p->z && !is_aligned(p->z, 2)) ||
        (p->bias && !is_aligned(p->bias, float_size(p->bias_dtype))) ||
        (p->residual && !is_aligned(p->residual, float_size(p->residual_dtype))))
        return PGQ_ERR_ALIGN;
    const int64_t ye = (int64_t)float_size(p->y_dtype), re = (int64_t)float_size(p->residual_dtype);
    const bool in_place = p->residual == p->y && p->ldr == p->ldy && p->residual_dtype == p->y_dtype;
    const Span spans[] = {{p->y, M, N * ye, p->ldy * ye},
                          {p->z, M, N * 2, p->ldz * 2},
                          {p->x, M, K * 2, p->ldx * 2},
                          {p->codes, N, K, p->ldc},
                          {p->scales, K > 0, N * 2, N * 2},
                          {p->bias, 1, N * (int64_t)float_size(p->bias_dtype), N * 4},
                          {in_place ? nullptr : p->residual, M, N * re, p->ldr * re}};
    return any_clash(spans, 2, 7) ? PGQ_ERR_PARAM : PGQ_OK;
}

pgq_status check_bwd(const pgq_linear_bwd* p)
{
    if (!p) return PGQ_ERR_NULL;
    const int64_t M = p->M, N = p->N, K = p->K;
    if (M < 0 || N < 0 || K < 0 || M > kMaxSize || N > kMaxSize || K > kMaxSize) return PGQ_ERR_SHAPE;
    if (!act_ok(p->act, p->slope) || p->reserved != 0) return PGQ_ERR_PARAM;
    const bool act = p->act != PGQ_ACT_NONE;
    if (p->lddy < N || (act && p->ldz < N) || (p->dw && (p->ldx < K || p->lddw < K)) ||
        (p->dx && (p->ldc < K || p->lddx < K)))
        return PGQ_ERR_SHAPE;
    if (!float_type(p->dy_dtype) || (p->dx && !float_type(p->dx_dtype)) || (p->dw && !float_type(p->dw_dtype)))
        return PGQ_ERR_DTYPE;
    if (M > 0 && N > 0 && (p->dx || p->dw || p->dbias)) {
        if (!p->dy || (act && !p->z)) return PGQ_ERR_NULL;
        if (K > 0 && ((p->dw && !p->x) || (p->dx && (!p->codes || !p->scales)))) return PGQ_ERR_NULL;
    }
    if ((p->dy && !is_aligned(p->dy, float_size(p->dy_dtype))) || (act && p->z && !is_aligned(p->z, 2)) ||
        (p->dw && p->x && !is_aligned(p->x, 2)) || (p->dx && p->scales && !is_aligned(p->scales, 2)) ||
        (p->dx && !is_aligned(p->dx, float_size(p->dx_dtype))) || (p->dw && !is_aligned(p->dw, float_size(p->dw_dtype))) ||
        (p->dbias && !is_aligned(p->dbias, 4)))
        return PGQ_ERR_ALIGN;
    const int64_t ge = (int64_t)float_size(p->dy_dtype), xe = (int64_t)float_size(p->dx_dtype), we = (int64_t)float_size(p->dw_dtype);
    const Span spans[] = {{p->dx, M, K * xe, p->lddx * xe},
                          {p->dw, N, K * we, p->lddw * we},
                          {p->dbias, 1, N * 4, N * 4},
                          {p->dy, M, N * ge, p->lddy * ge},
                          {act ? p->z : nullptr, M, N * 2, p->ldz * 2},
                          {p->dw ? p->x : nullptr, M, K * 2, p->ldx * 2},
                          {p->dx ? p->codes : nullptr, N, K, p->ldc},
                          {p->dx ? p->scales : nullptr, 1, N * 2, N * 2},
                          {p->dw ? p->mask : nullptr, N, (K + 7) / 8, (K + 7) / 8}};
    return any_clash(spans, 3, 9) ? PGQ_ERR_PARAM : PGQ_OK;
}

int64_t tiles_of(int64_t I, int64_t J) { return ((I + kGT - 1) / kGT) * ((J + kGT - 1) / kGT); }
int64_t up8(int64_t x) { return (x + 7) / 8 * 8; }
// Row stride of a laid-out operand: whole 128-byte lines, so that a stage's 128 bytes of a row are one line, not
// two (16384 x 1584 x 528 50.1 -> 48.2 us, 4899 x 947 x 4656 114 -> 107); short rows stay dense.
int64_t pitch(int64_t x) { return x >= 256 ? (x + 63) / 64 * 64 : up8(x); }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Contractions and rows this long go through the 64 x 64 element-load kernel: the matrix kernels address
// a tile's rows with 32-bit byte offsets.
constexpr int64_t kLong = (int64_t)1 << 21;
// bf16 rows the matrix kernels can load where they lie
bool direct(const void* p, int64_t ld, int64_t cols)
{
    return cols % 8 == 0 && ld % 8 == 0 && ld < kLong && is_aligned(p, 16);
}

// How a forward call runs, and where its scratch goes.
struct FwdPlan {
    bool skinny, tile;           // few tokens; the element-load kernel; else the matrix kernels
    bool copy_x;
    MmNt nt;                     // sizes, tile and parts
    Parts parts;                 // of the few-token kernel
    size_t what, xc, part, bytes;
};
// The few-token kernel's parts and estimated microseconds: eight blocks a time (above), a tile's reads of X and the codes
// unaligned three times that; 5.5 for the second launch.  Parts for at most two workgroups a compute unit.
double skinny_plan(const pgq_linear_fwd& p, Parts& parts)
{
    const int64_t tiles = (p.N + 15) / 16, blocks = (p.K + 63) / 64;
    double block = p.M <= 16 ? 0.3 + 0.02 * (double)p.M : p.M <= 32 ? 0.75 : 1.9;
    if (p.M > 1 && (p.ldx % 8 || p.ldc % 16 || !is_aligned(p.x, 16) || !is_aligned(p.codes, 16))) block *= 3.0;
    double best = 0;
    for (int64_t n = 1; n <= 64; n *= 2) {
        const int64_t per = (blocks + n - 1) / n;
        if (n > 1 && (tiles * n > 512 || per < kSkinnyWaves || (n - 1) * per >= blocks)) break;
        const double rounds = std::max(1.0, (double)(tiles * n) / 256.0);
        const double t = 3.0 + (double)((per + kSkinnyWaves - 1) / kSkinnyWaves) * block * rounds + (n > 1 ? 5.5 : 0.0);
        if (best == 0 || t < best) {
            best = t;
            parts.n = (int32_t)n;
            parts.blocks = per;
        }
    }
    return best;
}
FwdPlan plan_fwd(const pgq_linear_fwd& p)
{
    FwdPlan q;
    memset(&q, 0, sizeof(q));
    if (p.M == 0 || p.N == 0) return q;
    auto few = [&] {
        q.skinny = true;
        q.copy_x = false;
        q.bytes = q.parts.n > 1 ? up256((size_t)q.parts.n * p.M * p.N * 4) : 0;
        return q;
    };
    const double skinny = p.M <= kSkinnyMost ? skinny_plan(p, q.parts) : 0.0;
    if (p.M <= 16 || (p.M <= kSkinnyMost && (p.K >= kLong || p.K == 0))) return few();
    q.tile = p.K >= kLong || p.K == 0;
    if (q.tile) return q;
    q.copy_x = !direct(p.x, p.ldx, p.K);
    q.nt.I = p.M;
    q.nt.J = p.N;
    q.nt.L = up8(p.K);
    q.nt.parts = 1;
    double mm = mm_nt_plan(q.nt, p.K % 16 == 0 && p.ldc % 16 == 0 && p.ldc < kLong && is_aligned(p.codes, 16),
                           (double)float_size(p.y_dtype) + (p.z ? 2.0 : 0.0) + (p.residual ? (double)float_size(p.residual_dtype) : 0.0));
    if (p.M <= kSkinnyMost) {
        // 17 to 64 tokens: the few-token kernel reads all of X again for every 16 weight rows (at 64 x 4096 x 4096 19.7
        // us against 13.6 for the tiles, at 64 x 1584 x 528 5.9 against 8.4)
        if (q.copy_x || !q.nt.from_codes) mm += 5.0;
        if (skinny <= mm) return few();
    }
    if (!q.nt.from_codes) q.bytes = up256((size_t)p.N * pitch(p.K) * 2);
    q.xc = q.bytes;
    if (q.copy_x) q.bytes += up256((size_t)p.M * pitch(p.K) * 2);
    q.part = q.bytes;
    q.bytes += up256(mm_nt_partial_bytes(q.nt));
    return q;
}

struct BwdPlan {
    bool dx, dw, db;             // what there is to compute
    bool tile;                   // by the element-load kernel
    int32_t parts, parts_dx, parts_dw;       // bf16 values that stand for a dZ: in scratch, in each product
    int64_t Np, ldn, ldt;        // columns of a part, row strides of dZ and of the transposed weights
    bool dz, copy_x;             // dZ and X go through scratch
    MmNt nt;                     // dX, dW: sizes, tiles and parts
    MmTt tt;
    int both;                    // dX and dW: their pair of tiles in one launch
    int32_t dz_rows;
    int64_t blocks;              // row blocks of dZ units (and of the db partial sums)
    size_t o_dz, o_db, o_what_t, o_x, o_part, o_part_dx, bytes;
};
// The bf16 parts of dZ that a product with outputs of this type takes.  One is dZ where nothing multiplies a bf16
// dY but 0 or powers of two; two are where a bf16 Z does (8 and 8 bits).  Otherwise two leave 2^-14 of dZ, a 64th of a
// bf16 output's own rounding (one left 2^-8, and bf16 gradients 0.0024 off where their own rounding is 0.0017), and
// three leave nothing: 24 bits.
int32_t dz_parts(const pgq_linear_bwd& p, int32_t out_dtype)
{
    uint32_t slope;
    memcpy(&slope, &p.slope, 4);
    if (p.dy_dtype == PGQ_BF16) {
        if (p.act == PGQ_ACT_NONE) return 1;
        if (p.act != PGQ_ACT_SILU && (slope & 0x7FFFFFu) == 0) return p.act == PGQ_ACT_RELU ? 1 : 2;
    }
    return out_dtype == PGQ_F32 ? 3 : 2;
}
BwdPlan plan_bwd(const pgq_linear_bwd& p)
{
    BwdPlan q;
    memset(&q, 0, sizeof(q));
    q.dx = p.dx && p.M > 0 && p.K > 0;
    q.dw = p.dw && p.N > 0 && p.K > 0;
    q.db = p.dbias && p.N > 0;
    q.parts_dx = q.dx ? dz_parts(p, p.dx_dtype) : 1;
    q.parts_dw = q.dw ? dz_parts(p, p.dw_dtype) : 1;
    q.parts = std::max(q.parts_dx, q.parts_dw);
    // several parts of a row of dZ lie one behind the other, each padded with zeros to whole stages
    q.Np = q.parts > 1 ? (p.N + 63) / 64 * 64 : up8(p.N);
    q.ldn = q.parts > 1 ? q.parts * q.Np : pitch(p.N);
    q.ldt = q.parts > 1 ? q.Np : pitch(p.N);
    q.tile = q.ldn >= kLong || p.K >= kLong;
    auto take = [&](size_t n) { const size_t at = q.bytes; q.bytes += up256(n); return at; };
    // long units for few partial sums, short ones where there are not enough of them to fill the machine
    q.dz_rows = p.M * p.N >= (int64_t)4 << 20 ? 64 : 16;
    q.blocks = (p.M + q.dz_rows - 1) / q.dz_rows;
    if (q.db) q.o_db = take((size_t)q.blocks * p.N * 4);
    if (q.tile || p.N == 0 || p.M == 0) return q;
    if (q.dx || q.dw) {
        q.dz = p.act != PGQ_ACT_NONE || p.dy_dtype != PGQ_BF16 || !direct(p.dy, p.lddy, p.N);    // (else one part)
        if (q.dz) q.o_dz = take((size_t)p.M * q.ldn * 2);
    }
    if (q.dx) {
        q.o_what_t = take((size_t)p.K * q.ldt * 2);
        q.nt.I = p.M;
        q.nt.J = p.K;
        q.nt.L = q.Np;
        q.nt.parts = q.parts_dx;
    }
    if (q.dw) {
        q.copy_x = !direct(p.x, p.ldx, p.K);
        if (q.copy_x) q.o_x = take((size_t)p.M * pitch(p.K) * 2);
        q.tt.I = p.N;
        q.tt.J = p.K;
        q.tt.L = p.M;
        q.tt.parts = q.parts_dw;
        q.tt.part_cols = q.Np;
    }
    if (q.dx && q.dw) q.both = mm_both_plan(q.nt, q.tt, (double)float_size(p.dx_dtype));
    else if (q.dx) mm_nt_plan(q.nt, false, (double)float_size(p.dx_dtype));
    else if (q.dw) mm_tt_plan(q.tt);
    if (q.dx) q.o_part_dx = take(mm_nt_partial_bytes(q.nt));
    if (q.dw) q.o_part = take(mm_tt_partial_bytes(q.tt));
    return q;
}

// Workgroups of the preparation, the element-load kernel and the few-token kernel
int64_t flat_units(int64_t rows, int64_t cols) { return (rows * (up8(cols) / 8) + kFlat - 1) / kFlat; }
int64_t dz_units(const pgq_linear_bwd& p, const BwdPlan& q) { return q.dz || q.db ? q.blocks * ((q.Np + kDzCols - 1) / kDzCols) : 0; }
int64_t what_t_units(const pgq_linear_bwd& p) { return ((p.N + 63) / 64) * ((p.K + 63) / 64); }
int64_t skinny_grid(const pgq_linear_fwd& p, const Parts& parts) { return (p.N + 15) / 16 * parts.n; }
int64_t join_grid(const pgq_linear_fwd& p) { return (p.M * p.N + 255) / 256; }
int64_t prep_units(const pgq_linear_fwd& p, const FwdPlan& q)
{
    return (q.nt.from_codes ? 0 : flat_units(p.N, p.K)) + (q.copy_x ? flat_units(p.M, p.K) : 0);
}
int64_t prep_units(const pgq_linear_bwd& p, const BwdPlan& q)
{
    const bool mm = !q.tile && p.M > 0 && p.N > 0;
    return dz_units(p, q) + (mm && q.dx ? what_t_units(p) : 0) + (mm && q.copy_x ? flat_units(p.M, p.K) : 0);
}
// Every launch of the call is within the runtime's limits.
bool launches_fit(const pgq_linear_fwd& p, const FwdPlan& q)
{
    if (p.M == 0 || p.N == 0) return true;
    if (q.skinny) return grid_fits(skinny_grid(p, q.parts), 64 * kSkinnyWaves) && (q.parts.n == 1 || grid_fits(join_grid(p), 256));
    if (q.tile) return grid_fits(tiles_of(p.M, p.N), 256);
    return grid_fits(prep_units(p, q), 256) && mm_nt_fits(q.nt);
}
bool launches_fit(const pgq_linear_bwd& p, const BwdPlan& q)
{
    const bool mm = !q.tile && p.M > 0 && p.N > 0;
    if (!grid_fits(prep_units(p, q), 256)) return false;
    if (mm && q.dx && q.dw) return mm_both_fits(q.nt, q.tt, q.db ? p.N : 0);
    if (q.db && !mm_dbias_fits(p.N)) return false;
    if (!mm) return (!q.dx || grid_fits(tiles_of(p.M, p.K), 256)) && (!q.dw || grid_fits(tiles_of(p.N, p.K), 256));
    return (!q.dx || mm_nt_fits(q.nt)) && (!q.dw || mm_tt_fits(q.tt));
}

bool rows16(const void* p, int32_t dtype, int64_t ld) { return is_aligned(p, 16) && ld % (16 / (int64_t)float_size(dtype)) == 0; }

}  // namespace
}  // namespace pgq

using namespace pgq;

extern "C" {

pgq_status pgq_linear_forward_workspace(const pgq_linear_fwd* p, size_t* workspace_bytes)
{
    if (!workspace_bytes) return PGQ_ERR_NULL;
    const pgq_status st = check_fwd(p);
    if (st != PGQ_OK) return st;
    const FwdPlan q = plan_fwd(*p);
    if (!launches_fit(*p, q)) return PGQ_ERR_SHAPE;
    *workspace_bytes = q.bytes;
    return PGQ_OK;
}

pgq_status pgq_linear_backward_workspace(const pgq_linear_bwd* p, size_t* workspace_bytes)
{
    if (!workspace_bytes) return PGQ_ERR_NULL;
    const pgq_status st = check_bwd(p);
    if (st != PGQ_OK) return st;
    const BwdPlan q = plan_bwd(*p);
    if (!launches_fit(*p, q)) return PGQ_ERR_SHAPE;
    *workspace_bytes = q.bytes;
    return PGQ_OK;
}

pgq_status pgq_linear_forward_plan(const pgq_linear_fwd* p, pgq_linear_plan* out)
{
    if (!out) return PGQ_ERR_NULL;
    const pgq_status st = check_fwd(p);
    if (st != PGQ_OK) return st;
    const FwdPlan q = plan_fwd(*p);
    if (!launches_fit(*p, q)) return PGQ_ERR_SHAPE;
    memset(out, 0, sizeof(*out));
    if (p->M == 0 || p->N == 0) return PGQ_OK;
    out->path = q.skinny ? PGQ_LINEAR_FEW : q.tile ? PGQ_LINEAR_ELEMENTS : PGQ_LINEAR_TILES;
    out->parts = q.skinny ? q.parts.n : 1;
    if (out->path == PGQ_LINEAR_TILES) {
        mm_nt_tile(q.nt, &out->tile_rows, &out->tile_cols);
        out->parts = q.nt.splits;
        out->from_codes = q.nt.from_codes;
        out->copies_x = q.copy_x;
    }
    return PGQ_OK;
}

pgq_status pgq_linear_backward_plan(const pgq_linear_bwd* p, pgq_linear_plan* out)
{
    if (!out) return PGQ_ERR_NULL;
    const pgq_status st = check_bwd(p);
    if (st != PGQ_OK) return st;
    const BwdPlan q = plan_bwd(*p);
    if (!launches_fit(*p, q)) return PGQ_ERR_SHAPE;
    memset(out, 0, sizeof(*out));
    if (!q.dx && !q.dw) return PGQ_OK;
    out->path = q.tile || p->M == 0 || p->N == 0 ? PGQ_LINEAR_ELEMENTS : PGQ_LINEAR_TILES;
    out->dz_dx = q.dx ? q.parts_dx : 0;
    out->dz_dw = q.dw ? q.parts_dw : 0;
    if (out->path != PGQ_LINEAR_TILES) return PGQ_OK;
    if (q.dx) {
        mm_nt_tile(q.nt, &out->tile_rows, &out->tile_cols);
        out->parts = q.nt.splits;
    }
    if (q.dw) {
        mm_tt_tile(q.tt, &out->dw_rows, &out->dw_cols);
        out->dw_parts = q.tt.splits;
    }
    out->copies_x = q.copy_x;
    out->joint = q.dx && q.dw;
    return PGQ_OK;
}

pgq_status pgq_linear_forward(const pgq_linear_fwd* p, void* workspace, size_t workspace_bytes, void* stream)
{
    const pgq_status st = check_fwd(p);
    if (st != PGQ_OK || p->M == 0 || p->N == 0) return st;
    const FwdPlan q = plan_fwd(*p);
    if (!launches_fit(*p, q)) return PGQ_ERR_SHAPE;
    if (q.bytes && (!workspace || workspace_bytes < q.bytes)) return PGQ_ERR_WORKSPACE;
    if (q.bytes && !is_aligned(workspace, 256)) return PGQ_ERR_ALIGN;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    pgq_linear_fwd f = *p;
    pgq_linear_bwd b;
    memset(&b, 0, sizeof(b));
    if (q.skinny) {
        Parts parts = q.parts;
        parts.sums = reinterpret_cast<float*>(ws);
        Launches l(parts.n > 1 ? 2 : 1, stream);
        void* args[] = {&f, &parts};
        const void* k = f.M <= 16   ? reinterpret_cast<const void*>(&pgq_linear_skinny_kernel<1>)
                        : f.M <= 32 ? reinterpret_cast<const void*>(&pgq_linear_skinny_kernel<2>)
                                    : reinterpret_cast<const void*>(&pgq_linear_skinny_kernel<4>);
        l.go(k, skinny_grid(f, parts), 64 * kSkinnyWaves, args);
        if (parts.n > 1) l.go(reinterpret_cast<const void*>(&pgq_linear_join_kernel), join_grid(f), 256, args);
        return l.done();
    }
    if (q.tile) {
        Launches l(1, stream);
        int32_t parts = 1;
        void* args[] = {&f, &b, &parts};
        l.go(reinterpret_cast<const void*>(&pgq_linear_tile_kernel<P_FWD>), tiles_of(f.M, f.N), 256, args);
        return l.done();
    }
    const bool reduce = q.nt.splits > 1;
    const bool prep = !q.nt.from_codes || q.copy_x;
    Launches l(1 + prep + reduce, stream);
    Prep pr;
    memset(&pr, 0, sizeof(pr));
    pr.b.M = f.M;
    pr.b.N = f.N;
    pr.b.K = f.K;
    pr.b.codes = f.codes;
    pr.b.ldc = f.ldc;
    pr.b.scales = f.scales;
    pr.b.x = f.x;
    pr.b.ldx = f.ldx;
    pr.Kp = up8(f.K);
    pr.ldk = pitch(f.K);
    if (!q.nt.from_codes) {
        pr.what = reinterpret_cast<uint16_t*>(ws + q.what);
        pr.n_what = flat_units(f.N, f.K);
    }
    if (q.copy_x) {
        pr.xc = reinterpret_cast<uint16_t*>(ws + q.xc);
        pr.n_x = flat_units(f.M, f.K);
    }
    void* args[] = {&pr};
    if (prep) l.go(reinterpret_cast<const void*>(&pgq_linear_prep_kernel), pr.n_what + pr.n_x, 256, args);
    MmNt mm = q.nt;
    mm.a = q.copy_x ? pr.xc : f.x;
    mm.lda = q.copy_x ? pr.ldk : f.ldx;
    mm.b = pr.what;
    mm.codes = f.codes;
    mm.scales = f.scales;
    mm.ldb = q.nt.from_codes ? f.ldc : pr.ldk;
    mm.partial = reinterpret_cast<float*>(ws + q.part);
    mm.e.bias = f.bias;
    mm.e.residual = f.residual;
    mm.e.z = f.z;
    mm.e.y = f.y;
    mm.e.ldr = f.ldr;
    mm.e.ldz = f.ldz;
    mm.e.ldy = f.ldy;
    mm.e.bias_dtype = f.bias_dtype;
    mm.e.residual_dtype = f.residual_dtype;
    mm.e.y_dtype = f.y_dtype;
    mm.e.act = f.act;
    mm.e.slope = f.slope;
    mm.e.vec = rows16(f.y, f.y_dtype, f.ldy) && (!f.z || rows16(f.z, PGQ_BF16, f.ldz)) &&
               (!f.residual || rows16(f.residual, f.residual_dtype, f.ldr));
    if (l.next()) l.e = launch_mm_nt(mm, stream);
    if (reduce && l.next()) l.e = launch_mm_nt_reduce(mm, stream);
    return l.done();
}

pgq_status pgq_linear_backward(const pgq_linear_bwd* p, void* workspace, size_t workspace_bytes, void* stream)
{
    const pgq_status st = check_bwd(p);
    if (st != PGQ_OK) return st;
    const BwdPlan q = plan_bwd(*p);
    if (!q.dx && !q.dw && !q.db) return PGQ_OK;
    if (!launches_fit(*p, q)) return PGQ_ERR_SHAPE;
    if (q.bytes && (!workspace || workspace_bytes < q.bytes)) return PGQ_ERR_WORKSPACE;
    if (q.bytes && !is_aligned(workspace, 256)) return PGQ_ERR_ALIGN;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    pgq_linear_bwd b = *p;
    // an empty sum (N = 0 for dX, M = 0 for dW) is written by the element-load kernel
    const bool mm = !q.tile && b.M > 0 && b.N > 0;
    Prep pr;
    memset(&pr, 0, sizeof(pr));
    pr.b = b;
    pr.Kp = up8(b.K);
    pr.Np = q.Np;
    pr.ldk = pitch(b.K);
    pr.ldn = q.ldn;
    pr.ldt = q.ldt;
    pr.parts = q.parts;
    pr.dz = q.dz ? reinterpret_cast<uint16_t*>(ws + q.o_dz) : nullptr;
    pr.dz_rows = q.dz_rows;
    pr.dbias_part = q.db ? reinterpret_cast<float*>(ws + q.o_db) : nullptr;
    pr.n_dz = dz_units(b, q);
    if (mm && q.dx) {
        pr.what_t = reinterpret_cast<uint16_t*>(ws + q.o_what_t);
        pr.n_what_t = what_t_units(b);
    }
    if (mm && q.copy_x) {
        pr.xc = reinterpret_cast<uint16_t*>(ws + q.o_x);
        pr.n_x = flat_units(b.M, b.K);
    }
    const int64_t units = pr.n_dz + pr.n_what_t + pr.n_x;
    const bool reduce = mm && q.dw && q.tt.splits > 1, reduce_dx = mm && q.dx && q.nt.splits > 1;
    const bool both = mm && q.dx && q.dw;
    Launches l((units > 0) + (both ? 1 : q.dx + q.dw + q.db) + reduce + reduce_dx, stream);
    void* pargs[] = {&pr};
    if (units > 0) l.go(reinterpret_cast<const void*>(&pgq_linear_prep_kernel), units, 256, pargs);
    const Dbias db = {pr.dbias_part, q.blocks, b.N, q.db ? b.dbias : nullptr};
    if (q.db && !both && l.next()) l.e = launch_mm_dbias(db, stream);
    if (!mm) {
        pgq_linear_fwd f;
        memset(&f, 0, sizeof(f));
        int32_t pdx = q.parts_dx, pdw = q.parts_dw;
        void *xargs[] = {&f, &b, &pdx}, *wargs[] = {&f, &b, &pdw};
        if (q.dx) l.go(reinterpret_cast<const void*>(&pgq_linear_tile_kernel<P_DX>), tiles_of(b.M, b.K), 256, xargs);
        if (q.dw) l.go(reinterpret_cast<const void*>(&pgq_linear_tile_kernel<P_DW>), tiles_of(b.N, b.K), 256, wargs);
        return l.done();
    }
    MmNt x = q.nt;
    MmTt w = q.tt;
    x.a = w.a = q.dz ? pr.dz : static_cast<const uint16_t*>(b.dy);
    x.lda = w.lda = q.dz ? pr.ldn : b.lddy;
    x.b = pr.what_t;
    x.ldb = pr.ldt;
    x.partial = reinterpret_cast<float*>(ws + q.o_part_dx);
    x.e.y = b.dx;
    x.e.ldy = b.lddx;
    x.e.y_dtype = b.dx_dtype;
    x.e.vec = rows16(b.dx, b.dx_dtype, b.lddx);
    w.b = q.copy_x ? pr.xc : b.x;
    w.ldb = q.copy_x ? pr.ldk : b.ldx;
    w.c = b.dw;
    w.ldc = b.lddw;
    w.c_dtype = b.dw_dtype;
    w.mask = b.mask;
    w.partial = reinterpret_cast<float*>(ws + q.o_part);
    if (both && l.next()) l.e = launch_mm_both(q.both, x, w, db, stream);
    if (q.dx && !both && l.next()) l.e = launch_mm_nt(x, stream);
    if (q.dw && !both && l.next()) l.e = launch_mm_tt(w, stream);
    if (reduce_dx && l.next()) l.e = launch_mm_nt_reduce(x, stream);
    if (reduce && l.next()) l.e = launch_mm_tt_reduce(w, stream);
    return l.done();
}

}  // extern "C"
