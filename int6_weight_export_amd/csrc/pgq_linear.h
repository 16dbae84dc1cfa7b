// pgq_linear.h -- the matrix products behind the linear layer (pgq_linear_mm.hip), as its host layer
// (pgq_linear.hip) calls them.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pgq_desc.h"
#include "pgq_train.h"
#include "../../include/pgq.h"

namespace pgq {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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
// 16 (8) bytes at any alignment: one load, the hardware takes unaligned global addresses
__device__ __forceinline__ u32x4 load16(const void* p)
{
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

// 1 / (1 + e^-z), for z <= 0 as e^z / (1 + e^z): the exponential, within 2 units of the last place, does not overflow,
// and the reciprocal, within 1, is of a number between 1 and 2 (of one past 2^126 it would be 0: the instruction
// gives no subnormals, and z = -88 lost its value of -5e-37)
__device__ __forceinline__ float sigmoid(float z)
{
    const float a = expf(-fabsf(z));
    return (z > 0.0f ? 1.0f : a) * __builtin_amdgcn_rcpf(1.0f + a);
}

__device__ __forceinline__ float act_value(int32_t act, float slope, float z)
{
    if (act == PGQ_ACT_NONE) return z;
    if (act == PGQ_ACT_SILU) return z * sigmoid(z);
    const float r = z > 0.0f ? z : z * slope;
    return act == PGQ_ACT_RELU ? r : r * r;
}
__device__ __forceinline__ float act_slope(int32_t act, float slope, float z)
{
    if (act == PGQ_ACT_NONE) return 1.0f;
    if (act == PGQ_ACT_SILU) {
        const float s = sigmoid(z);
        return s * (1.0f + z * (1.0f - s));
    }
    const float d = z > 0.0f ? 1.0f : slope;
    return act == PGQ_ACT_RELU ? d : 2.0f * z * d * d;
}

// What a product does with its sums on the way out: v = act(sum + bias) + residual, Z stored on the side.
struct Epilogue {
    const void* bias;            // per column
    const void* residual;        // I x J
    uint16_t* z;                 // I x J bf16
    void* y;                     // I x J
    int64_t ldr, ldz, ldy;
    int32_t bias_dtype, residual_dtype, y_dtype, act;
    float slope;
    int32_t vec;                 // rows of y, z and residual take 16-byte accesses of 8 (bf16) or 4 (fp32) columns
};

// Y[i][j] = epilogue(sum_l A[i][l] B[j][l]): 16-byte aligned rows, row strides below 2^22 elements.  B in bf16 and
// L a multiple of 8, or B as int8 codes with a scale per row (bf16(code * s)) and L a multiple of 16.  With parts > 1
// an element of A is the sum of that many bf16 values L columns apart, L a multiple of 64 and B in bf16.
struct MmNt {
    const uint16_t* a;
    const uint16_t* b;
    const int8_t* codes;         // in place of b where from_codes
    const uint16_t* scales;
    int64_t lda, ldb, I, J, L;
    int32_t parts;
    int32_t kind, splits;        // tile, and pieces the contraction is cut into (mm_nt_plan)
    int32_t from_codes;
    int64_t chunk;               // l per piece, those of one part after the other's, a multiple of 64
    float* partial;              // splits > 1: mm_nt_partial_bytes() of scratch
    Epilogue e;
};
// kind, splits, chunk, from_codes from I, J, L, whether codes will do and the bytes in and out for each element
// of Y; returns the estimated microseconds
double mm_nt_plan(MmNt& p, bool codes_ok, double out_bytes);
size_t mm_nt_partial_bytes(const MmNt& p);
void mm_nt_tile(const MmNt& p, int32_t* rows, int32_t* cols);
bool mm_nt_fits(const MmNt& p);          // its launches are within the runtime's limits
hipError_t launch_mm_nt(const MmNt& p, void* stream);
// splits > 1: the sums of the parts, in their order, through the epilogue
hipError_t launch_mm_nt_reduce(const MmNt& p, void* stream);

// C[i][j] = sum_l sum_p A[l][p part_cols + i] B[l][j], p below parts: bf16 operands, 16-byte aligned rows of at least I and J elements rounded
// up to 8, row strides below 2^23.  C goes out as dw_dtype, zero where the mask bit of (i, j) is 0.
struct MmTt {
    const uint16_t* a;
    const uint16_t* b;
    int64_t lda, ldb, I, J, L;
    void* c;
    int64_t ldc;
    int32_t c_dtype;
    int32_t parts;               // bf16 values whose sum stands for an element of A, part_cols columns apart
    int64_t part_cols;
    int32_t kind, splits;        // tile, and pieces the sum is cut into (mm_tt_plan)
    int64_t chunk;               // stages (64 l of one part) per piece
    const uint8_t* mask;         // NULL or I x ceil(J / 8) bytes
    float* partial;              // splits > 1: mm_tt_partial_bytes() of scratch
};
void mm_tt_plan(MmTt& p);        // kind, splits and chunk from I, J, L and parts
size_t mm_tt_partial_bytes(const MmTt& p);
void mm_tt_tile(const MmTt& p, int32_t* rows, int32_t* cols);
bool mm_tt_fits(const MmTt& p);
hipError_t launch_mm_tt(const MmTt& p, void* stream);
// splits > 1: the sum of the parts, in their order
hipError_t launch_mm_tt_reduce(const MmTt& p, void* stream);

// db[n] = sum of part[i][n] over the row blocks i.
struct Dbias {
    const float* part;
    int64_t blocks, N;
    float* out;                  // NULL: nothing to do
};
bool mm_dbias_fits(int64_t N);
hipError_t launch_mm_dbias(const Dbias& d, void* stream);
// dX, dW and db in one launch: the pair of tiles, with kind, splits and chunk of both products.
int mm_both_plan(MmNt& x, MmTt& w, double out_bytes);
bool mm_both_fits(const MmNt& x, const MmTt& w, int64_t db_cols);
hipError_t launch_mm_both(int both, const MmNt& x, const MmTt& w, const Dbias& d, void* stream);

}  // namespace pgq
