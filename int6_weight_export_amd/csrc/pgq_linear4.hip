// pgq_linear4.hip -- the linear layer over 4-bit weights with group scales, for few tokens (gfx950):
// Y = act(X W^T + b) + R, W[n][k] = code[n][k] * s[n][k / group].
//
// The codes are the traffic: N K / 2 bytes, each read once.  A workgroup takes 16 weight rows and its wavefronts
// blocks of 128 columns in turn; v_mfma_f32_16x16x32_bf16 multiplies 16 tokens (A) with the 16 rows (B).  Codes are
// whole numbers, which bf16 holds, and products with bf16 tokens are exact in fp32: the matrix cores sum x * code over
// a group and one multiply-add per sum brings in the group's scale, so no weight is ever rounded and a weight costs no
// multiplication of its own.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "pgq_linear.h"
#include "pgq_train.h"
#include "../../include/pgq.h"

namespace pgq {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves4 = 8;
constexpr int kMost = 64;                         // tokens of a workgroup
constexpr int kBlockK = 128;                      // columns of a block: 64 bytes of a row's codes

// Eight codes as bf16.  A byte 0000 0mmm (sign in its top bit) is, read as e4m3, the number m * 2^-9: below 2^-6 such
// numbers are equally spaced, so the conversion from fp8 with a scale of 2^9 makes the whole number.  Ten instructions.
__device__ __forceinline__ bf16x8 decode8(uint32_t w)
{
    const uint32_t lo = (w & 0x07070707u) | ((w << 4) & 0x80808080u), hi = ((w >> 4) & 0x07070707u) | (w & 0x80808080u);
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A lane's load is 32 consecutive codes of its row: word d of lane quarter q holds columns 32 q + 8 d .. + 7 of the
// block.  For groups of 128 word d is multiplied as it lies, so instruction d sums columns 32 q + 8 d of every q.  For 64
// the halves of the wavefront trade words, so that instructions 0 and 1 stay within columns 0 .. 63; for 32 the
// quarters do too, and instruction d takes columns 32 d .. 32 d + 31.
template <int G>
__device__ __forceinline__ void trade(u32x4& w)
{
    if (G <= 64) {
        const u32x2 a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false), b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
        w = u32x4{a[0], b[0], a[1], b[1]};
    }
    if (G == 32) {
        const u32x2 a = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false), b = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
        w = u32x4{a[0], a[1], b[0], b[1]};
    }
}
// first of the eight columns that lane quarter q supplies to instruction d
template <int G>
__device__ __forceinline__ int column(int d, int q)
{
    if (G == 128) return 32 * q + 8 * d;
    if (G == 64) return 64 * (d >> 1) + 32 * (q & 1) + 16 * (q >> 1) + 8 * (d & 1);
    return 32 * d + 8 * q;
}

// 16 bytes of a row from byte `at` on, zeros past its last one: past the edge the row's last 16 bytes shifted down
__device__ __forceinline__ u32x4 load16_edge(const void* row, int64_t at, int64_t bytes)
{
    const uint8_t* p = static_cast<const uint8_t*>(row);
    unsigned __int128 v = 0;
    if (at >= bytes) return u32x4{};
    if (bytes >= 16) {
        const int over = (int)max((int64_t)0, at + 16 - bytes);
        __builtin_memcpy(&v, p + at - over, 16);
        v >>= 8 * over;
    } else {
#pragma unroll 1
        for (int64_t e = bytes - 1; e >= at; --e) v = v << 8 | p[e];
    }
    return __builtin_bit_cast(u32x4, v);
}

__device__ __forceinline__ void finish(const pgq_linear4_fwd& f, int64_t m, int64_t n, float z)
{
    if (f.bias) z += load_any(f.bias, f.bias_dtype, n);
    float y = act_value(f.act, f.slope, z);
    if (f.residual) y += load_any(f.residual, f.residual_dtype, m * f.ldr + n);
    store_any(f.y, f.y_dtype, m * f.ldy + n, y);
}

// T: tiles of 16 tokens.  Lane l: token l % 16 of A, weight row l % 16 of B, columns by the quarter l / 16.  Lanes past
// M or N repeat the last row, whose sums they do not store.
template <int T, int G>
__global__ void __launch_bounds__(64 * kWaves4) pgq_linear4_kernel(pgq_linear4_fwd f, int32_t token_blocks)
{
    __shared__ f32x4 sums[kWaves4][T][64];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int r = lane & 15, q = lane >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x % (uint32_t)token_blocks) * kMost;
    const int64_t n0 = (int64_t)(blockIdx.x / (uint32_t)token_blocks) * 16;
    const int64_t n = min(n0 + r, f.N - 1);
    const uint8_t* crow = f.codes + n * f.ldc;
    const uint16_t* srow = f.scales + n * f.lds;
    const uint16_t* xrow[T];
#pragma unroll
    for (int t = 0; t < T; ++t) xrow[t] = f.x + min(m0 + 16 * t + r, f.M - 1) * f.ldx;
    f32x4 acc[T];
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t] = f32x4{};
    constexpr int GB = kBlockK / G;               // groups of a block
    auto multiply = [&](u32x4 c, const u32x4 (*x)[4], const float* s) __attribute__((always_inline)) {
        trade<G>(c);
#pragma unroll
        for (int g = 0; g < GB; ++g) {
            f32x4 p[T];
#pragma unroll
            for (int t = 0; t < T; ++t) p[t] = f32x4{};
#pragma unroll
            for (int d = g * (4 / GB); d < (g + 1) * (4 / GB); ++d) {
                const bf16x8 w = decode8(c[d]);
#pragma unroll
                for (int t = 0; t < T; ++t) p[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[t][d]), w, p[t], 0, 0, 0);
            }
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][e] = __builtin_fmaf(p[t][e], s[g], acc[t][e]);
        }
    };
    const int64_t full = f.K / kBlockK;
#pragma unroll 1
    for (int64_t b = wave; b < full; b += kWaves4) {
        const u32x4 c = load16(crow + 64 * b + 16 * q);
        u32x4 x[T][4];
        float s[GB];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int d = 0; d < 4; ++d) x[t][d] = load16(xrow[t] + kBlockK * b + column<G>(d, q));
#pragma unroll
        for (int g = 0; g < GB; ++g) s[g] = f16_to_f32(srow[GB * b + g]);
        multiply(c, x, s);
    }
    if (f.K % kBlockK && wave == (int)(full % kWaves4)) {          // the last block: nothing past K is read, X is 0 there
        const int64_t k0 = full * kBlockK;
        const int left = (int)(f.K - k0);
        const u32x4 c = load16_edge(crow, 64 * full + 16 * q, (f.K + 7) / 8 * 4);
        u32x4 x[T][4];
        float s[GB];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int d = 0; d < 4; ++d) x[t][d] = load16_edge(xrow[t], 2 * (k0 + column<G>(d, q)), 2 * f.K);
#pragma unroll
        for (int g = 0; g < GB; ++g) s[g] = g * G < left ? f16_to_f32(srow[GB * full + g]) : 0.0f;
        multiply(c, x, s);
    }
#pragma unroll
    for (int t = 0; t < T; ++t) sums[wave][t][lane] = acc[t];
    __syncthreads();
    // accumulator element e of lane l: token 4 (l / 16) + e, weight row l % 16
    for (int u = (int)threadIdx.x; u < 64 * T * 4; u += 64 * kWaves4) {
        const int l = u & 63, e = (u >> 6) & 3, t = u >> 8;
        const int64_t m = m0 + 16 * t + 4 * (l >> 4) + e, nn = n0 + (l & 15);
        if (m >= f.M || nn >= f.N) continue;
        float z = sums[0][t][l][e];
#pragma unroll
        for (int w = 1; w < kWaves4; ++w) z += sums[w][t][l][e];
        finish(f, m, nn, z);
    }
}

pgq_status check(const pgq_linear4_fwd* p)
{
    if (!p) return PGQ_ERR_NULL;
    const int64_t M = p->M, N = p->N, K = p->K;
    if (M < 0 || N < 0 || K < 0 || M > kMaxSize || N > kMaxSize || K > kMaxSize) return PGQ_ERR_SHAPE;
    if (p->group != 32 && p->group != 64 && p->group != 128) return PGQ_ERR_PARAM;
    const int64_t bytes = (K + 7) / 8 * 4, groups = (K + p->group - 1) / p->group;
    if (p->ldx < K || p->ldc < bytes || p->lds < groups || p->ldy < N || (p->residual && p->ldr < N)) return PGQ_ERR_SHAPE;
    if (!float_type(p->y_dtype) || (p->bias && !float_type(p->bias_dtype)) || (p->residual && !float_type(p->residual_dtype)))
        return PGQ_ERR_DTYPE;
    if (!act_ok(p->act, p->slope)) return PGQ_ERR_PARAM;
    if (M == 0 || N == 0) return PGQ_OK;
    if (!p->y || (K > 0 && (!p->x || !p->codes || !p->scales))) return PGQ_ERR_NULL;
    if (!is_aligned(p->y, float_size(p->y_dtype)) || (p->x && !is_aligned(p->x, 2)) || (p->scales && !is_aligned(p->scales, 2)) ||
        (p->bias && !is_aligned(p->bias, float_size(p->bias_dtype))) ||
        (p->residual && !is_aligned(p->residual, float_size(p->residual_dtype))))
        return PGQ_ERR_ALIGN;
    const int64_t ye = (int64_t)float_size(p->y_dtype), re = (int64_t)float_size(p->residual_dtype);
    const bool in_place = p->residual == p->y && p->ldr == p->ldy && p->residual_dtype == p->y_dtype;
    const Span spans[] = {{p->y, M, N * ye, p->ldy * ye},
                          {p->x, M, K * 2, p->ldx * 2},
                          {p->codes, N, bytes, p->ldc},
                          {p->scales, N, groups * 2, p->lds * 2},
                          {p->bias, 1, N * (int64_t)float_size(p->bias_dtype), N * 4},
                          {in_place ? nullptr : p->residual, M, N * re, p->ldr * re}};
    return any_clash(spans, 1, 6) ? PGQ_ERR_PARAM : PGQ_OK;
}
int64_t token_blocks(const pgq_linear4_fwd& p) { return (p.M + kMost - 1) / kMost; }
int64_t grid_of(const pgq_linear4_fwd& p) { return (p.N + 15) / 16 * token_blocks(p); }
bool launches_fit(const pgq_linear4_fwd& p) { return grid_fits(grid_of(p), 64 * kWaves4); }

template <int T>
const void* kernel(int32_t group)
{
    return group == 32   ? reinterpret_cast<const void*>(&pgq_linear4_kernel<T, 32>)
           : group == 64 ? reinterpret_cast<const void*>(&pgq_linear4_kernel<T, 64>)
                         : reinterpret_cast<const void*>(&pgq_linear4_kernel<T, 128>);
}

}  // namespace
}  // namespace pgq

using namespace pgq;

extern "C" {

pgq_status pgq_linear4_forward_workspace(const pgq_linear4_fwd* p, size_t* workspace_bytes)
{
    if (!workspace_bytes) return PGQ_ERR_NULL;
    const pgq_status st = check(p);
    if (st != PGQ_OK) return st;
    if (!launches_fit(*p)) return PGQ_ERR_SHAPE;
    *workspace_bytes = 0;
    return PGQ_OK;
}

pgq_status pgq_linear4_forward(const pgq_linear4_fwd* p, void* workspace, size_t workspace_bytes, void* stream)
{
    const pgq_status st = check(p);
    if (st != PGQ_OK || p->M == 0 || p->N == 0) return st;
    if (!launches_fit(*p)) return PGQ_ERR_SHAPE;
    pgq_linear4_fwd f = *p;
    int32_t tb = (int32_t)token_blocks(f);
    void* args[] = {&f, &tb};
    Launches l(1, stream);
    l.go(f.M <= 16 ? kernel<1>(f.group) : f.M <= 32 ? kernel<2>(f.group) : kernel<4>(f.group), grid_of(f), 64 * kWaves4, args);
    return l.done();
}

}  // extern "C"
