// pgq_linear.hip -- the quantized linear layer (gfx950): Y = act(X What^T + b) + R and its gradient.
//
// What[n][k] = bf16(fp32(code[n][k] * s_n)), the STE forward's weight ("SubSixteen v2" card, PR #69,
// section Other).  Three products:
//     Z [m][n] = sum_k X[m][k]  What[n][k]          (forward)
//     dX[m][k] = sum_n dZ[m][n] What[n][k]          dZ = bf16(dY * act'(Z))
//     dW[n][k] = sum_m dZ[m][n] X[m][k]
// Products of two bf16 values are exact in fp32; every sum is held in fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "pgq_desc.h"
#include "pgq_train.h"
#include "../../include/pgq.h"

namespace pgq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float f16_to_f32(uint16_t h) { return (float)__builtin_bit_cast(_Float16, h); }
__device__ __forceinline__ float bf16_to_f32(uint16_t h) { return __builtin_bit_cast(float, (uint32_t)h << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

__device__ __forceinline__ float load_any(const void* p, int32_t dtype, int64_t i)
{
    return dtype == PGQ_F32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int32_t dtype, int64_t i, float v)
{
    if (dtype == PGQ_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
}

__device__ __forceinline__ float act_value(int32_t act, float slope, float z)
{
    if (act == PGQ_ACT_NONE) return z;
    if (act == PGQ_ACT_SILU) return z / (1.0f + expf(-z));
    const float r = z > 0.0f ? z : z * slope;
    return act == PGQ_ACT_RELU ? r : r * r;
}
__device__ __forceinline__ float act_slope(int32_t act, float slope, float z)
{
    if (act == PGQ_ACT_NONE) return 1.0f;
    if (act == PGQ_ACT_SILU) {
        const float s = 1.0f / (1.0f + expf(-z));
        return s * (1.0f + z * (1.0f - s));
    }
    const float d = z > 0.0f ? 1.0f : slope;
    return act == PGQ_ACT_RELU ? d : 2.0f * z * d * d;
}

enum Product { P_FWD, P_DX, P_DW };

// dZ in fp32 (m, n), rounded to bf16 where it enters a product
__device__ __forceinline__ float dz_at(const pgq_linear_bwd& b, int64_t m, int64_t n)
{
    const float g = load_any(b.dy, b.dy_dtype, m * b.lddy + n);
    return b.act == PGQ_ACT_NONE ? g : g * act_slope(b.act, b.slope, bf16_to_f32(b.z[m * b.ldz + n]));
}

// One 64 x 64 tile of a product per workgroup of four wavefronts, 32 x 32 each: element loads through
// registers into LDS, any shape and stride.
constexpr int kGT = 64, kGK = 32, kGPad = kGK + 8;

template <int P>
__global__ void __launch_bounds__(256) pgq_linear_tile_kernel(pgq_linear_fwd f, pgq_linear_bwd b)
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
    auto load_a = [&](int64_t i, int64_t l) -> uint16_t {
        if (i >= I || l >= L) return 0;
        if (P == P_FWD) return f.x[i * f.ldx + l];
        return P == P_DX ? f32_to_bf16(dz_at(b, i, l)) : f32_to_bf16(dz_at(b, l, i));
    };
    auto load_b = [&](int64_t j, int64_t l) -> uint16_t {
        if (j >= J || l >= L) return 0;
        if (P == P_FWD) return what(f.codes, f.ldc, f.scales, j, l);
        return P == P_DX ? what(b.codes, b.ldc, b.scales, l, j) : b.x[l * b.ldx + j];
    };
    f32x16 acc = {};
    for (int64_t l0 = 0; l0 < L; l0 += kGK) {
        __syncthreads();
        for (int e = tid; e < kGT * kGK; e += 256) {
            // the thread order follows the contiguous index of each operand
            const int r = P == P_DW ? e % kGT : e / kGK, l = P == P_DW ? e / kGT : e % kGK;
            As[r][l] = load_a(i0 + r, l0 + l);
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

// db[n] = sum over m of the unrounded dZ: 64 columns per workgroup, four row phases joined in LDS
__global__ void __launch_bounds__(256) pgq_linear_dbias_kernel(pgq_linear_bwd b)
{
    __shared__ float part[4][64];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int64_t n = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (n < b.N)
        for (int64_t m = wave; m < b.M; m += 4) s += dz_at(b, m, n);
    part[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && n < b.N) b.dbias[n] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
}

constexpr int64_t kMaxSize = ((int64_t)1 << 31) - 1;

bool float_type(int32_t dt) { return dt == PGQ_F32 || dt == PGQ_BF16; }
size_t float_size(int32_t dt) { return dt == PGQ_F32 ? 4 : 2; }
bool act_ok(int32_t act, float slope)
{
    if (act == PGQ_ACT_NONE || act == PGQ_ACT_SILU) return true;
    return (act == PGQ_ACT_RELU || act == PGQ_ACT_RELU2) && slope - slope == 0.0f;
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
    // the residual may be y itself; any other reading of memory that the call writes is refused
    if (p->residual == p->y && (p->ldr != p->ldy || p->residual_dtype != p->y_dtype)) return PGQ_ERR_PARAM;
    return PGQ_OK;
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
    return PGQ_OK;
}

int64_t tiles_of(int64_t I, int64_t J) { return ((I + kGT - 1) / kGT) * ((J + kGT - 1) / kGT); }

}  // namespace
}  // namespace pgq

using namespace pgq;

extern "C" {

pgq_status pgq_linear_forward_workspace(const pgq_linear_fwd* p, size_t* workspace_bytes)
{
    if (!workspace_bytes) return PGQ_ERR_NULL;
    const pgq_status st = check_fwd(p);
    if (st == PGQ_OK) *workspace_bytes = 0;
    return st;
}

pgq_status pgq_linear_backward_workspace(const pgq_linear_bwd* p, size_t* workspace_bytes)
{
    if (!workspace_bytes) return PGQ_ERR_NULL;
    const pgq_status st = check_bwd(p);
    if (st == PGQ_OK) *workspace_bytes = 0;
    return st;
}

pgq_status pgq_linear_forward(const pgq_linear_fwd* p, void* workspace, size_t workspace_bytes, void* stream)
{
    (void)workspace;
    (void)workspace_bytes;
    pgq_status st = check_fwd(p);
    if (st != PGQ_OK || p->M == 0 || p->N == 0) return st;
    const int64_t tiles = tiles_of(p->M, p->N);
    if (tiles > kMaxSize) return PGQ_ERR_SHAPE;
    pgq_linear_fwd f = *p;
    pgq_linear_bwd b;
    memset(&b, 0, sizeof(b));
    void* args[] = {&f, &b};
    const hipError_t e = launch_plain(reinterpret_cast<const void*>(&pgq_linear_tile_kernel<P_FWD>), dim3((unsigned)tiles),
                                      dim3(256), args, stream);
    return e != hipSuccess ? (pgq_status)note_hip_error(e) : PGQ_OK;
}

pgq_status pgq_linear_backward(const pgq_linear_bwd* p, void* workspace, size_t workspace_bytes, void* stream)
{
    (void)workspace;
    (void)workspace_bytes;
    pgq_status st = check_bwd(p);
    if (st != PGQ_OK) return st;
    pgq_linear_fwd f;
    memset(&f, 0, sizeof(f));
    pgq_linear_bwd b = *p;
    void* args[] = {&f, &b};
    const bool dx = p->dx && p->M > 0 && p->K > 0, dw = p->dw && p->N > 0 && p->K > 0, db = p->dbias && p->N > 0;
    if ((dx && tiles_of(p->M, p->K) > kMaxSize) || (dw && tiles_of(p->N, p->K) > kMaxSize)) return PGQ_ERR_SHAPE;
    void *ev_start = nullptr, *ev_stop = nullptr;
    take_timing_events(&ev_start, &ev_stop);
    int left = (dx ? 1 : 0) + (dw ? 1 : 0) + (db ? 1 : 0);
    auto go = [&](const void* fn, int64_t grid) {
        set_timing_events(ev_start, --left == 0 ? ev_stop : nullptr);
        ev_start = nullptr;
        const hipError_t e = launch_plain(fn, dim3((unsigned)grid), dim3(256), args, stream);
        return e;
    };
    hipError_t e = hipSuccess;
    void* bargs[] = {&b};
    if (db) {
        set_timing_events(ev_start, --left == 0 ? ev_stop : nullptr);
        ev_start = nullptr;
        e = launch_plain(reinterpret_cast<const void*>(&pgq_linear_dbias_kernel), dim3((unsigned)((p->N + 63) / 64)),
                         dim3(256), bargs, stream);
    }
    if (e == hipSuccess && dx) e = go(reinterpret_cast<const void*>(&pgq_linear_tile_kernel<P_DX>), tiles_of(p->M, p->K));
    if (e == hipSuccess && dw) e = go(reinterpret_cast<const void*>(&pgq_linear_tile_kernel<P_DW>), tiles_of(p->N, p->K));
    return e != hipSuccess ? (pgq_status)note_hip_error(e) : PGQ_OK;
}

}  // extern "C"
