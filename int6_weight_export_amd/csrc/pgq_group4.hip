// pgq_group4.hip -- 4-bit codes with a scale for every 32, 64 or 128 columns of a row: quantizer and decode (gfx950).
//
// A lane takes V consecutive columns of a row -- eight of 16-bit values, four where 32-bit ones are read or written, so that a
// wavefront's accesses of 16 bytes a lane lie side by side -- and group / V neighbouring lanes a group: its maximum is two to five
// exchanges between lanes, nothing goes through LDS, and two lanes of four columns put a block of codes together.  The
// arithmetic is the row quantizer's with Q = 7 (pgq.h), every step an IEEE binary32 operation.  Both kernels are streams:
// what bounds them is the memory traffic of the weights and values, which are read and written past the caches.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pgq_linear.h"
#include "pgq_train.h"
#include "../../include/pgq.h"

namespace pgq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kRuns = 2;                          // blocks of lanes that a quantizing workgroup loads together

struct Groups {
    const void* w;               // quantize: rows x cols of w_dtype
    uint8_t* codes;
    uint16_t* scales;
    void* out;                   // dq, or the decoded values; NULL: none
    uint32_t* status;
    int64_t rows, cols, ld, ldc, lds, ldo;
    int64_t slots;               // lanes of a row: whole groups (quantize), whole blocks of eight columns (decode)
    int32_t group, w_dtype, out_dtype;
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 any_u32x4 __attribute__((aligned(2)));
typedef u32x2 any_u32x2 __attribute__((aligned(2)));
#define GLB __attribute__((address_space(1)))

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xF, 0xF, false);
}
// maximum over LANES neighbouring lanes, in every one of them
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t x)
{
    x = max(x, dpp<0xB1>(x));                     // quad_perm: lane ^ 1
    x = max(x, dpp<0x4E>(x));                     // quad_perm: lane ^ 2
    if (LANES >= 8) x = max(x, dpp<0x141>(x));    // row_half_mirror
    if (LANES >= 16) x = max(x, dpp<0x140>(x));   // row_mirror
    if (LANES >= 32) {                            // rows of 16 lanes 0 and 1, 2 and 3
        const u32x2 y = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        x = max(y[0], y[1]);
    }
    return x;
}

// row and first column of a lane
template <int V>
__device__ __forceinline__ void place(const Groups& a, int64_t i, int64_t& r, int64_t& k)
{
    if (a.rows * a.slots <= 0xFFFFFFFFll) {       // (a 64-bit division costs as much as the rest)
        r = (uint32_t)i / (uint32_t)a.slots;
        k = ((uint32_t)i - (uint32_t)r * (uint32_t)a.slots) * V;
    } else {
        r = i / a.slots;
        k = i % a.slots * V;
    }
}

// V columns of a row of weights, zeros past the last
template <int V>
__device__ __forceinline__ void load_weights(const Groups& a, int64_t r, int64_t k, float* x)
{
    if (V == 4 && a.w_dtype == PGQ_F32) {
        const float* p = static_cast<const float*>(a.w) + r * a.ld + k;
        if (k + 4 <= a.cols) {
            const f32x4 v = __builtin_bit_cast(f32x4, __builtin_nontemporal_load((const GLB any_u32x4*)p));
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = v[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = k + e < a.cols ? p[e] : 0.0f;
        }
        return;
    }
    const uint16_t* p = static_cast<const uint16_t*>(a.w) + r * a.ld + k;
    uint32_t v[V / 2] = {};
    if (k + V <= a.cols) {
        if constexpr (V == 8) {
            const u32x4 t = __builtin_nontemporal_load((const GLB any_u32x4*)p);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = t[e];
        } else {
            const u32x2 t = __builtin_nontemporal_load((const GLB any_u32x2*)p);
            v[0] = t[0];
            v[1] = t[1];
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (k + e < a.cols) v[e / 2] |= (uint32_t)p[e] << (16 * (e % 2));
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const uint16_t h = (uint16_t)(v[e / 2] >> (16 * (e % 2)));
        x[e] = a.w_dtype == PGQ_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
    }
}

// V values to columns k .. of a row, those past the last left out
template <int V>
__device__ __forceinline__ void store_values(const Groups& a, int64_t r, int64_t k, const float* x)
{
    const bool whole = k + V <= a.cols;
    if (V == 4 && a.out_dtype == PGQ_F32) {
        float* p = static_cast<float*>(a.out) + r * a.ldo + k;
        if (whole) {
            __builtin_nontemporal_store(__builtin_bit_cast(u32x4, f32x4{x[0], x[1], x[2], x[3]}), (GLB any_u32x4*)p);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (k + e < a.cols) p[e] = x[e];
        }
        return;
    }
    uint16_t* p = static_cast<uint16_t*>(a.out) + r * a.ldo + k;
    uint32_t h[V];
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = f32_to_bf16(x[e]);
    if (whole) {
        if constexpr (V == 8) __builtin_nontemporal_store(u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16}, (GLB any_u32x4*)p);
        else __builtin_nontemporal_store(u32x2{h[0] | h[1] << 16, h[2] | h[3] << 16}, (GLB any_u32x2*)p);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (k + e < a.cols) p[e] = (uint16_t)h[e];
    }
}

template <int V, int G>
__global__ void __launch_bounds__(kThreads) pgq_quantize_groups_kernel(Groups a)
{
    constexpr int LANES = G / V;
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kRuns) + threadIdx.x, slots = a.rows * a.slots;
    int64_t r[kRuns], k[kRuns];
    float x[kRuns][V];
#pragma unroll
    for (int u = 0; u < kRuns; ++u) {             // all loads first (past the last slot the last row's first is read, and not stored)
        const int64_t i = first + u * kThreads;
        place<V>(a, i < slots ? i : slots - a.slots, r[u], k[u]);
        load_weights<V>(a, r[u], k[u], x[u]);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < kRuns; ++u) {
        const bool live = first + u * kThreads < slots;      // (a row's slots are whole groups, so a group is live or not)
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) top = max(top, __builtin_bit_cast(uint32_t, x[u][e]) & 0x7FFFFFFFu);
        top = group_max<LANES>(top);
        const float clip = __builtin_bit_cast(float, top);
        uint16_t sh = __builtin_bit_cast(uint16_t, (_Float16)(clip / 7.0f));
        if (sh == 0) sh = 0x3C00;
        const float s = f16_to_f32(sh), inv = 1.0f / s;
        uint32_t bits = 0;
        if (top >= 0x7F800000u) bits = PGQ_DEV_NONFINITE;
        else if (sh == 0x7C00) bits = PGQ_DEV_SCALE_OVF;
        if (live && bits && a.status) atomicOr(a.status, bits);
        // rint(x / s): y is within 2^-15 of the quotient, so the two round alike unless y is that close to a half; there
        // the correctly rounded quotient decides, which is a half exactly when x / s is.
        float c[V];
        bool tie = false;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float y = x[u][e] * inv;
            c[e] = rintf(y);
            tie |= fabsf(y - c[e]) > 0.5f - 0x1p-12f;
        }
        if (tie) {
#pragma unroll
            for (int e = 0; e < V; ++e) c[e] = rintf(x[u][e] / s);
        }
        uint32_t word = 0;
        float v[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            c[e] = __builtin_amdgcn_fmed3f(c[e], -7.0f, 7.0f) + 0.0f;          // (a zero code is +0)
            const uint32_t sign = __builtin_bit_cast(uint32_t, c[e]) >> 28 & 8u;
            word |= ((uint32_t)fabsf(c[e]) | sign) << (8 * (e & 3) + 4 * (e >> 2));
            v[e] = c[e] * s;
        }
        if (V == 4) {                             // columns 0 .. 3 of a block in an even lane, 4 .. 7 in the odd one after it
            word <<= 4 * (threadIdx.x & 1);
            word |= dpp<0xB1>(word);
        }
        if (!live) continue;
        if (k[u] < a.cols && (V == 8 || (k[u] & 4) == 0)) __builtin_memcpy(a.codes + r[u] * a.ldc + k[u] / 2, &word, 4);
        if ((threadIdx.x & (LANES - 1)) == 0) a.scales[r[u] * a.lds + (uint32_t)k[u] / G] = sh;
        if (a.out && k[u] < a.cols) store_values<V>(a, r[u], k[u], v);
    }
}

template <int V>
__global__ void __launch_bounds__(kThreads) pgq_dequant_groups_kernel(Groups a)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= a.rows * a.slots) return;
    int64_t r, k;
    place<V>(a, i, r, k);
    uint32_t word;
    __builtin_memcpy(&word, a.codes + r * a.ldc + (k / 8) * 4, 4);
    if (V == 4) word >>= k & 4;
    const float s = f16_to_f32(a.scales[r * a.lds + (uint32_t)k / (uint32_t)a.group]);
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const uint32_t nib = word >> (8 * (e & 3) + 4 * (e >> 2));
        const float m = (float)(nib & 7u);
        v[e] = ((nib & 8u) && m != 0.0f ? -m : m) * s;        // (a zero code is +0)
    }
    store_values<V>(a, r, k, v);
}

int64_t up8(int64_t x) { return (x + 7) / 8 * 8; }

// sizes, strides and types that both calls take
pgq_status check(const void* codes, int64_t ldc, const uint16_t* scales, int64_t lds, int64_t rows, int64_t cols, int32_t group,
                 const void* out, int32_t out_dtype, int64_t ldo)
{
    if (rows < 0 || cols < 0 || rows > kMaxSize || cols > kMaxSize) return PGQ_ERR_SHAPE;
    if (group != 32 && group != 64 && group != 128) return PGQ_ERR_PARAM;
    if (ldc < up8(cols) / 2 || lds < (cols + group - 1) / group || (out && ldo < cols)) return PGQ_ERR_SHAPE;
    if (out && !float_type(out_dtype)) return PGQ_ERR_DTYPE;
    if (rows == 0 || cols == 0) return PGQ_OK;
    if (!codes || !scales) return PGQ_ERR_NULL;
    if (!is_aligned(scales, 2) || (out && !is_aligned(out, float_size(out_dtype)))) return PGQ_ERR_ALIGN;
    return PGQ_OK;
}
template <int V>
const void* quantize_kernel(int32_t group)
{
    return group == 32   ? reinterpret_cast<const void*>(&pgq_quantize_groups_kernel<V, 32>)
           : group == 64 ? reinterpret_cast<const void*>(&pgq_quantize_groups_kernel<V, 64>)
                         : reinterpret_cast<const void*>(&pgq_quantize_groups_kernel<V, 128>);
}
int64_t grid_of(const Groups& a, int runs) { return (a.rows * a.slots + kThreads * runs - 1) / (kThreads * runs); }

}  // namespace
}  // namespace pgq

using namespace pgq;

extern "C" {

pgq_status pgq_quantize_groups(const void* w, int32_t w_dtype, int64_t rows, int64_t cols, int64_t ld, int32_t group, uint8_t* codes,
                               int64_t ldc, uint16_t* scales, int64_t lds, void* dq, int32_t dq_dtype, int64_t ldq,
                               uint32_t* dev_status, void* stream)
{
    const pgq_status st = check(codes, ldc, scales, lds, rows, cols, group, dq, dq_dtype, ldq);
    if (st != PGQ_OK) return st;
    if (w_dtype != PGQ_F32 && w_dtype != PGQ_BF16 && w_dtype != PGQ_F16) return PGQ_ERR_DTYPE;
    if (ld < cols) return PGQ_ERR_SHAPE;
    if (rows == 0 || cols == 0) return PGQ_OK;
    if (!w) return PGQ_ERR_NULL;
    const int64_t we = w_dtype == PGQ_F32 ? 4 : 2, de = (int64_t)float_size(dq_dtype), groups = (cols + group - 1) / group;
    if (!is_aligned(w, (size_t)we)) return PGQ_ERR_ALIGN;
    const Span spans[] = {{codes, rows, up8(cols) / 2, ldc}, {scales, rows, groups * 2, lds * 2}, {dq, rows, cols * de, ldq * de},
                          {w, rows, cols * we, ld * we}};
    if (any_clash(spans, 3, 4)) return PGQ_ERR_PARAM;
    const int v = w_dtype == PGQ_F32 || (dq && dq_dtype == PGQ_F32) ? 4 : 8;
    Groups a = {w, codes, scales, dq, dev_status, rows, cols, ld, ldc, lds, ldq, groups * (group / v), group, w_dtype, dq_dtype};
    if (!grid_fits(grid_of(a, kRuns), kThreads)) return PGQ_ERR_SHAPE;
    Launches l(1, stream);
    void* args[] = {&a};
    const void* fn = v == 4 ? quantize_kernel<4>(group) : quantize_kernel<8>(group);
    l.go(fn, grid_of(a, kRuns), kThreads, args);
    return l.done();
}

pgq_status pgq_dequant_groups(const uint8_t* codes, int64_t ldc, const uint16_t* scales, int64_t lds, int64_t rows, int64_t cols,
                              int32_t group, void* out, int32_t out_dtype, int64_t ldo, void* stream)
{
    pgq_status st = check(codes, ldc, scales, lds, rows, cols, group, out, out_dtype, ldo);
    if (st != PGQ_OK || rows == 0 || cols == 0) return st;
    if (!out) return PGQ_ERR_NULL;
    const int64_t oe = (int64_t)float_size(out_dtype), groups = (cols + group - 1) / group;
    const Span spans[] = {{out, rows, cols * oe, ldo * oe}, {codes, rows, up8(cols) / 2, ldc}, {scales, rows, groups * 2, lds * 2}};
    if (any_clash(spans, 1, 3)) return PGQ_ERR_PARAM;
    const int v = out_dtype == PGQ_F32 ? 4 : 8;
    Groups a = {nullptr, const_cast<uint8_t*>(codes), const_cast<uint16_t*>(scales), out, nullptr, rows, cols, 0, ldc, lds, ldo,
                up8(cols) / v, group, 0, out_dtype};
    if (!grid_fits(grid_of(a, 1), kThreads)) return PGQ_ERR_SHAPE;
    Launches l(1, stream);
    void* args[] = {&a};
    l.go(v == 4 ? reinterpret_cast<const void*>(&pgq_dequant_groups_kernel<4>) : reinterpret_cast<const void*>(&pgq_dequant_groups_kernel<8>), grid_of(a, 1), kThreads, args);
    return l.done();
}

}  // extern "C"
