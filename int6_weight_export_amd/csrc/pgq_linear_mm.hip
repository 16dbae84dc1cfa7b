// pgq_linear_mm.hip -- the matrix products of the linear layer on the matrix cores (gfx950).
//
// Operands are bf16 in memory; v_mfma_f32_32x32x16_bf16 accumulates in fp32.  Operand layout of the
// instruction (checked on the device): lane l supplies row l % 32 of A (and column l % 32 of B) with 8
// consecutive l, lanes 32..63 the next 8; accumulator register j of lane l is row 8 (j / 4) + 4 (l / 32) +
// j % 4, column l % 32.
//
// Sizes with a measurement are I x J x L: rows of A, rows (columns, for dW) of B, contraction.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pgq_desc.h"
#include "pgq_linear.h"

namespace pgq {
namespace {

#define GLB __attribute__((address_space(1)))

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int kTK = 64;                        // contraction per stage
constexpr uint32_t kOOB = 0x80000000u;         // a buffer offset past every range: the load returns 0

// every wave's LDS reads are complete, then the workgroup barrier (the asm keeps the compiler from
// moving memory operations across it)
template <int N>        // all but the N youngest loads of this wave have arrived, its LDS reads are complete; then the barrier
__device__ __forceinline__ void wait_barrier() { asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory"); }
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// 16 bytes a lane from buffer offset voff + soff to LDS, the wave's 1 KB in lane order from `to` on
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t voff, int soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)to, 16, voff, soff, 0, 0);
}

__device__ __forceinline__ uint32_t pk_bf16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));   // round to nearest even
}

// Workgroup -> tile.  Workgroups are dealt to the 8 XCDs round robin and each XCD has its own L2, so
// each XCD takes a contiguous eighth of the tiles; within it tiles go down kBand tile rows before the
// next column, so that the ~32 tiles an XCD works on at a time share kBand row panels of A and 32 / kBand
// column panels of B.
constexpr uint32_t kBand = 4;
__device__ __forceinline__ void tile_at(uint32_t tile, uint32_t gi, uint32_t gj, uint32_t& ti, uint32_t& tj)
{
    const uint32_t band = tile / (kBand * gj), in = tile % (kBand * gj);
    const uint32_t rows = min(kBand, gi - band * kBand);
    ti = band * kBand + in % rows;
    tj = in / rows;
}
__device__ __forceinline__ void tile_of(uint32_t wid, uint32_t total, uint32_t gi, uint32_t gj, uint32_t& ti, uint32_t& tj, uint32_t& part)
{
    const uint32_t xcd = wid % 8u, per = total / 8u, rem = total % 8u;
    const uint32_t t = (xcd < rem ? xcd * (per + 1u) : rem * (per + 1u) + (xcd - rem) * per) + wid / 8u;
    part = t / (gi * gj);
    tile_at(t % (gi * gj), gi, gj, ti, tj);
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// V values as bf16, one store
template <int V>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float* o)
{
    if constexpr (V == 8)
        *(GLB u32x4*)p = u32x4{pk_bf16(o[0], o[1]), pk_bf16(o[2], o[3]), pk_bf16(o[4], o[5]), pk_bf16(o[6], o[7])};
    else
        *(GLB u32x2*)p = u32x2{pk_bf16(o[0], o[1]), pk_bf16(o[2], o[3])};
}

// The epilogue of one lane, which holds V consecutive columns of several rows.  The columns are the same
// for every row, so the bias is loaded once; the residuals of G rows are loaded together.
template <int V, typename YT>
struct Out {
    const Epilogue& e;
    int64_t col, J;
    bool vec;
    float bias[V];
    __device__ __forceinline__ Out(const Epilogue& e_, int64_t col_, int64_t J_) : e(e_), col(col_), J(J_)
    {
        vec = e.vec && col + V <= J;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            bias[i] = 0.0f;
            if (e.bias && col + i < J)
                bias[i] = e.bias_dtype == PGQ_F32 ? ((const GLB float*)e.bias)[col + i] : bf16_to_f32(((const GLB uint16_t*)e.bias)[col + i]);
        }
    }
    // G rows, `step` apart, of which those below I are stored; v: their sums
    template <int G>
    __device__ __forceinline__ void rows(int64_t row, int step, int64_t I, float (*v)[V]) const
    {
        if (!vec) {
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (row + g * step < I) edge(row + g * step, v[g]);
            return;
        }
        float r[G][V];
        if (e.residual) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int64_t at = min(row + g * step, I - 1) * e.ldr + col;
                if (e.residual_dtype == PGQ_F32) {
                    const GLB f32x4* pr = (const GLB f32x4*)((const float*)e.residual + at);
#pragma unroll
                    for (int q = 0; q < V / 4; ++q) {
                        const f32x4 x = pr[q];
#pragma unroll
                        for (int i = 0; i < 4; ++i) r[g][4 * q + i] = x[i];
                    }
                } else {
                    uint32_t x[V / 2];
                    if constexpr (V == 8) {
                        const u32x4 y = *(const GLB u32x4*)((const uint16_t*)e.residual + at);
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] = y[i];
                    } else {
                        const u32x2 y = *(const GLB u32x2*)((const uint16_t*)e.residual + at);
                        x[0] = y[0];
                        x[1] = y[1];
                    }
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        r[g][2 * i] = __builtin_bit_cast(float, x[i] << 16);
                        r[g][2 * i + 1] = __builtin_bit_cast(float, x[i] & 0xFFFF0000u);
                    }
                }
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < V; ++i) v[g][i] += bias[i];
        if (e.z) {
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (row + g * step < I) store_bf16<V>(e.z + (row + g * step) * e.ldz + col, v[g]);
        }
        if (e.act == PGQ_ACT_SILU) {
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < V; ++i) v[g][i] = act_value(PGQ_ACT_SILU, 0.0f, v[g][i]);
        } else if (e.act != PGQ_ACT_NONE) {
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float x = act_value(PGQ_ACT_RELU, e.slope, v[g][i]);
                    v[g][i] = e.act == PGQ_ACT_RELU ? x : x * x;
                }
        }
        if (e.residual) {
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < V; ++i) v[g][i] += r[g][i];
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (row + g * step < I) {
                const int64_t at = (row + g * step) * e.ldy + col;
                if constexpr (sizeof(YT) == 4)
                    *(GLB f32x4*)((float*)e.y + at) = f32x4{v[g][0], v[g][1], v[g][2], v[g][3]};
                else
                    store_bf16<V>((uint16_t*)e.y + at, v[g]);
            }
    }
    // a row element by element: the last columns, and rows without 16-byte alignment
    __device__ __forceinline__ void edge(int64_t row, const float* v) const
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t c = col + i;
            if (c >= J) continue;
            float x = v[i] + bias[i];
            if (e.z) ((GLB uint16_t*)e.z)[row * e.ldz + c] = f32_to_bf16(x);
            x = act_value(e.act, e.slope, x);
            if (e.residual)
                x += e.residual_dtype == PGQ_F32 ? ((const GLB float*)e.residual)[row * e.ldr + c]
                                                 : bf16_to_f32(((const GLB uint16_t*)e.residual)[row * e.ldr + c]);
            if constexpr (sizeof(YT) == 4) ((GLB float*)e.y)[row * e.ldy + c] = x;
            else ((GLB uint16_t*)e.y)[row * e.ldy + c] = f32_to_bf16(x);
        }
    }
};

// ---- A rows times B rows ----------------------------------------------------------------------------
// A workgroup of WR x WC wavefronts computes a tile of 32 IB WR x 32 JB WC, each wavefront IB x JB blocks
// of 32 x 32.  Each 64-wide stage of both operands goes from global memory straight into LDS (buffer
// loads with the LDS destination), double-buffered, so the next stage's loads are in flight while the
// matrix cores work on this one; a lane past I, J or L gets zeros from the buffer range check.  Where the LDS has room
// A, which comes from memory, is three stages deep and B, which stays in the caches, two (16384 x 528 x 1584 with an
// fp32 residual 60 -> 55 us for the call, 8192 x 8192 x 4096 483 -> 465).
//
// LDS slots are 16-byte granules, 8 to a row; granule g of row r sits in slot g ^ swz(r), so that the
// rows a fragment read touches spread over distinct banks in every group of 8 and of 16 lanes.
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// Q: B is the weights' int8 codes (4 granules to a row, in slot g ^ swz4(r)), which each wavefront turns into bf16
// in registers right before it multiplies: for few tile rows, where laying What out first costs more.
__device__ __forceinline__ int swz4(int r) { return (((r >> 1) & 1) ^ ((r >> 3) & 1)) | (((r >> 2) & 1) << 1); }

// 16 codes -> two fragments of bf16(code * s): the product is exact (at most 7 + 11 significant bits)
__device__ __forceinline__ void codes_to_bf16(u32x4 q, float s, bf16x8& lo, bf16x8& hi)
{
    u32x4 a, c;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)(int8_t)(q[w] >> (8 * e)) * s;
        u32x4& to = w < 2 ? a : c;
        to[2 * (w & 1)] = pk_bf16(v[0], v[1]);
        to[2 * (w & 1) + 1] = pk_bf16(v[2], v[3]);
    }
    lo = __builtin_bit_cast(bf16x8, a);
    hi = __builtin_bit_cast(bf16x8, c);
}

// In the large tiles the R LDS reads of a half stage go between the M matrix instructions of the half before it: a
// wavefront issues in order, and reads issued in one piece kept it from multiplying while the LDS worked them off
// (16384 x 528 x 6336 155 -> 144 us, 8192 x 8448 x 4096 554 -> 535; the small tiles, bound by latency, lose
// 1 us to the longer code and go without).
template <int IB, int JB>
constexpr bool kSpread = IB * JB >= 6;
template <int R, int M>
__device__ __forceinline__ void spread()
{
    static_assert(R <= 2 * M, "at most two reads to an instruction");
#pragma unroll
    for (int m = 0; m < M; ++m) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                          // a matrix instruction
        const int reads = R * (m + 1) / M - R * m / M;
        if (reads == 1) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);          // then LDS reads
        if (reads == 2) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
}

__host__ __device__ inline int64_t nt_stages(const MmNt& p) { return (p.L + kTK - 1) / kTK * p.parts; }

constexpr int kWayOut = 64 + 4;                // floats of a row on its way out, at most

template <int WR, int WC, int IB, int JB, bool Q, int NB, int NA>
constexpr int nt_lds()
{
    constexpr int stages = (NA * 32 * IB * WR * 8 + NB * 32 * JB * WC * (Q ? 4 : 8)) * 16;
    constexpr int out = WR * WC * 32 * kWayOut * 4;
    return stages > out ? stages : out;
}

// A wavefront's way out of NJ of its blocks of 32 columns, from block J0 on: row i0.., column j0.. of Y.
template <int IB, int JB, int J0, int NJ, typename YT>
__device__ __forceinline__ void way_out(const MmNt& p, const f32x16 (&acc)[IB][JB], float* tl, int64_t i0, int64_t j0, int lane)
{
    constexpr int V = sizeof(YT) == 4 ? 4 : 8;
    constexpr int EP = 32 * NJ + 4;                           // row pitch in LDS, floats
    static_assert(EP <= kWayOut, "the scratch of a wavefront");
    constexpr int LPR = 32 * NJ / V;                          // lanes per row
    constexpr int STEP = 64 / LPR;                            // rows a wavefront covers at once
    constexpr int G = sizeof(YT) == 4 && STEP <= 8 ? 4 : 2;   // and a lane takes G of those at a time (more spill)
    static_assert(64 % LPR == 0 && 32 % (STEP * G) == 0, "whole groups");
    const int h = lane >> 5, r32 = lane & 31;
    const Out<V, YT> out(p.e, j0 + 32 * J0 + lane % LPR * V, p.J);
#pragma unroll
    for (int i = 0; i < IB; ++i) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) tl[(8 * (r >> 2) + 4 * h + (r & 3)) * EP + 32 * j + r32] = acc[i][J0 + j][r];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
        for (int q = 0; q < 32; q += STEP * G) {
            const int rr = q + lane / LPR;
            float v[G][V];
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int u = 0; u < V / 4; ++u) {
                    const f32x4 x = *reinterpret_cast<const f32x4*>(tl + (rr + g * STEP) * EP + lane % LPR * V + 4 * u);
#pragma unroll
                    for (int w = 0; w < 4; ++w) v[g][4 * u + w] = x[w];
                }
            const int64_t row = i0 + 32 * i + rr;
            if (row < p.I && out.col < p.J) out.template rows<G>(row, STEP, p.I, v);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

template <int WR, int WC, int IB, int JB, bool Q, int NB, int NA, typename YT>
__device__ __forceinline__ void nt_body(const MmNt& p, uint32_t wid, uint32_t total, uint8_t* lds)
{
    constexpr int T = 64 * WR * WC, TI = 32 * IB * WR, TJ = 32 * JB * WC;
    constexpr int BG = Q ? 4 : 8;                            // granules per row of B
    constexpr int AI = TI * 8 / T, BI = TJ * BG / T;         // load instructions per thread per stage
    constexpr int AS = TI * kTK * 2, BS = TJ * BG * 16;      // bytes per stage
    static_assert(TI * 8 % T == 0 && TJ * BG % T == 0, "whole load instructions");
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t gi = (uint32_t)((p.I + TI - 1) / TI), gj = (uint32_t)((p.J + TJ - 1) / TJ);
    uint32_t ti, tj, part;
    tile_of(wid, total, gi, gj, ti, tj, part);
    const int64_t i0 = (int64_t)ti * TI, j0 = (int64_t)tj * TJ;
    const int64_t l0 = (int64_t)part * p.chunk, len = min(p.chunk, p.parts * p.L - l0);      // this piece of the contraction
    const int irows = (int)min((int64_t)TI, p.I - i0), jrows = (int)min((int64_t)TJ, p.J - j0);
    const __amdgpu_buffer_rsrc_t ar = __builtin_amdgcn_make_buffer_rsrc((void*)(p.a + i0 * p.lda + l0), 0, (int)(((int64_t)(irows - 1) * p.lda + len) * 2), 0x00020000);
    const __amdgpu_buffer_rsrc_t br =
        Q ? __builtin_amdgcn_make_buffer_rsrc((void*)(p.codes + j0 * p.ldb + l0), 0, (int)((int64_t)(jrows - 1) * p.ldb + len), 0x00020000)
          : __builtin_amdgcn_make_buffer_rsrc((void*)(p.b + j0 * p.ldb), 0, (int)(((int64_t)(jrows - 1) * p.ldb + p.L) * 2), 0x00020000);
    // load slot of instruction c: row c T / 8 + tid / 8, slot tid % 8 (its granule is the same for every c)
    const int r0 = tid >> 3, g0 = (tid & 7) ^ swz(r0);
    const int br0 = tid / BG, bg0 = Q ? (tid & 3) ^ swz4(br0) : g0;
    // byte offsets of this thread's loads within a stage; rows past the edge are out of range for good
    uint32_t ao[AI], bo[BI];
#pragma unroll
    for (int c = 0; c < AI; ++c)
        ao[c] = r0 + c * (T / 8) < irows ? (uint32_t)((r0 + c * (T / 8)) * p.lda + 8 * g0) * 2u : kOOB;
#pragma unroll
    for (int c = 0; c < BI; ++c)
        bo[c] = br0 + c * (T / BG) < jrows ? (uint32_t)((br0 + c * (T / BG)) * p.ldb + (Q ? 16 * bg0 : 8 * bg0)) * (Q ? 1u : 2u) : kOOB;
    const int nst = (int)((len + kTK - 1) / kTK);
    const int nfull = (int)(len / kTK);
    // A part's columns start those of B again: their byte offset for the stage that is issued next
    const int b_end = p.parts > 1 ? (int)p.L * 2 : 0x7FFFFFFF;
    int b_off = (int)(l0 >= 2 * p.L ? l0 - 2 * p.L : l0 >= p.L ? l0 - p.L : l0) * 2;      // (at most three parts)
    // A whole stage costs a load instruction and its scalar offset each (address arithmetic in the vector unit
    // would run while no wavefront multiplies: the barrier has just lined them up); the last, partial stage
    // masks the granules past the contraction's end.
    auto issue_a = [&](int st) __attribute__((always_inline)) {
        uint8_t* la = lds + (st % NA) * AS;
        const uint32_t off = st < nfull || st * kTK + 8 * g0 < (int)len ? 0u : kOOB;
        if (st < nfull) {
#pragma unroll
            for (int c = 0; c < AI; ++c) load_lds(ar, la + (c * T + wave * 64) * 16, ao[c], st * (kTK * 2));
        } else {
#pragma unroll
            for (int c = 0; c < AI; ++c) load_lds(ar, la + (c * T + wave * 64) * 16, ao[c] | off, st * (kTK * 2));
        }
    };
    auto issue_b = [&](int st) __attribute__((always_inline)) {
        uint8_t* lb = lds + NA * AS + (st % NB) * BS;
        const int kb = Q ? st * kTK : b_off;
        const uint32_t off = st < nfull || st * kTK + (Q ? 16 : 8) * bg0 < (int)len ? 0u : kOOB;
        if (st < nfull) {
#pragma unroll
            for (int c = 0; c < BI; ++c) load_lds(br, lb + (c * T + wave * 64) * 16, bo[c], kb);
        } else {
#pragma unroll
            for (int c = 0; c < BI; ++c) load_lds(br, lb + (c * T + wave * 64) * 16, bo[c] | off, kb);
        }
        if constexpr (!Q) {
            b_off += kTK * 2;
            b_off = b_off == b_end ? 0 : b_off;
        }
    };
    const int wi = (wave / WC) * (32 * IB), wj = (wave % WC) * (32 * JB);
    const int r32 = lane & 31, h = lane >> 5;
    float sc[Q ? JB : 1];                                    // the scales of this lane's weight rows
    if constexpr (Q) {
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            const int64_t n = j0 + wj + 32 * j + r32;
            sc[j] = n < p.J ? f16_to_f32(((const GLB uint16_t*)p.scales)[n]) : 0.0f;
        }
    }
    f32x16 acc[IB][JB];
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j) acc[i][j] = f32x16{};
    // Fragments of one 32-wide half of a stage: lane half h supplies l = 16 h + 8 t .. + 7 in instruction t,
    // so that its 16 l are contiguous in LDS.
    struct Frag {
        bf16x8 a[IB][2], b[JB][Q ? 1 : 2];
    } f0, f1;
    auto fetch = [&](Frag& f, int st, int kb) __attribute__((always_inline)) {
        const uint8_t* la = lds + (st % NA) * AS;
        const uint8_t* lb = lds + NA * AS + (st % NB) * BS;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int i = 0; i < IB; ++i) {
                const int r = wi + 32 * i + r32;
                f.a[i][t] = *reinterpret_cast<const bf16x8*>(la + (r * 8 + ((4 * kb + 2 * h + t) ^ swz(r))) * 16);
            }
            if constexpr (!Q) {
#pragma unroll
                for (int j = 0; j < JB; ++j) {
                    const int r = wj + 32 * j + r32;
                    f.b[j][t] = *reinterpret_cast<const bf16x8*>(lb + (r * 8 + ((4 * kb + 2 * h + t) ^ swz(r))) * 16);
                }
            }
        }
        if constexpr (Q) {
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                const int r = wj + 32 * j + r32;
                f.b[j][0] = *reinterpret_cast<const bf16x8*>(lb + (r * 4 + ((2 * kb + h) ^ swz4(r))) * 16);
            }
        }
    };
    auto multiply = [&](const Frag& f, int l) __attribute__((always_inline)) {
        bf16x8 b[JB][2];
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            if constexpr (Q) {                               // past the end 0 * 0, whatever the scale is
                codes_to_bf16(__builtin_bit_cast(u32x4, f.b[j][0]), l + 16 * h < (int)len ? sc[j] : 0.0f, b[j][0], b[j][1]);
            } else {
                b[j][0] = f.b[j][0];
                b[j][1] = f.b[j][1];
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < IB; ++i)
#pragma unroll
                for (int j = 0; j < JB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i][t], b[j][t], acc[i][j], 0, 0, 0);
    };
    // Two sets of fragments: while the matrix cores work on one half stage, the next half is read from LDS.
    // The barrier sits between the halves: there every wave has read all of stage st, so the loads of B's stage
    // st + NB and A's stage st + NA may overwrite it, and those of st + 1 have arrived (younger ones may still be out:
    // loads are counted in the order B(st + NB), A(st + NA)).
    constexpr int NL = AI + BI, EL = (NA - NB) * AI;
    if (nst > 0) {
#pragma unroll
        for (int s = 0; s < NA; ++s)
            if (s < nst) {
                if (s < NB) issue_b(s);
                issue_a(s);
            }
        if (nst >= NA) wait_barrier<(NB - 1) * NL + EL>();
        else wait_barrier<0>();
        fetch(f0, 0, 0);
    }
    int st = 0;
    if constexpr (kSpread<IB, JB>) {
        for (; st + 1 < nst; ++st) {                          // all but the last stage
            fetch(f1, st, 1);
            multiply(f0, st * kTK);
            spread<2 * (IB + JB), 2 * IB * JB>();
            if (st + NA - 1 < nst) wait_barrier<(NB - 2) * NL + EL>();
            else wait_barrier<0>();
            if (st + NB < nst) issue_b(st + NB);
            if (st + NA < nst) issue_a(st + NA);
            fetch(f0, st + 1, 0);
            multiply(f1, st * kTK + 32);
            spread<2 * (IB + JB), 2 * IB * JB>();
        }
    }
    for (; st < nst; ++st) {
        fetch(f1, st, 1);
        multiply(f0, st * kTK);
        if (st + NA - 1 < nst) wait_barrier<(NB - 2) * NL + EL>();
        else wait_barrier<0>();
        if (st + NB < nst) issue_b(st + NB);
        if (st + NA < nst) issue_a(st + NA);
        if (st + 1 < nst) fetch(f0, st + 1, 0);
        if (st * kTK + 32 < (int)len) multiply(f1, st * kTK + 32);
    }
    if (p.splits > 1) {                                       // the part's sums as they lie in the registers
        f32x4* part_out = reinterpret_cast<f32x4*>(p.partial) +
                          (((size_t)part * (gi * gj) + ti * gj + tj) * (WR * WC) + wave) * (IB * JB * 4 * 64) + lane;
#pragma unroll
        for (int i = 0; i < IB; ++i)
#pragma unroll
            for (int j = 0; j < JB; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    part_out[((i * JB + j) * 4 + q) * 64] = f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        return;
    }
    // out through LDS, 32 rows at a time, so that a lane holds consecutive columns
    float* tl = reinterpret_cast<float*>(lds) + wave * (32 * kWayOut);
    lds_barrier();
    way_out<IB, JB, 0, JB == 3 ? 2 : JB, YT>(p, acc, tl, i0 + wi, j0 + wj, lane);
    if constexpr (JB == 3) way_out<IB, JB, 2, 1, YT>(p, acc, tl, i0 + wi, j0 + wj, lane);
}

template <int WR, int WC, int IB, int JB, bool Q, int NB, int NA, typename YT>
__global__ void __launch_bounds__(64 * WR * WC) __attribute__((amdgpu_waves_per_eu(2)))
pgq_mm_nt_kernel(MmNt p)
{
    __shared__ __align__(16) uint8_t lds[nt_lds<WR, WC, IB, JB, Q, NB, NA>()];
    nt_body<WR, WC, IB, JB, Q, NB, NA, YT>(p, blockIdx.x, gridDim.x, lds);
}

// the sums of the parts, in their order, through the epilogue: one wavefront takes 8 rows of 32 columns
template <int WR, int WC, int IB, int JB>
__global__ void __launch_bounds__(256) pgq_mm_nt_reduce_kernel(MmNt p)
{
    constexpr int TI = 32 * IB * WR, TJ = 32 * JB * WC;
    const uint32_t gi = (uint32_t)((p.I + TI - 1) / TI), gj = (uint32_t)((p.J + TJ - 1) / TJ), tiles = gi * gj;
    const uint32_t unit = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t tile = unit / (WR * WC * IB * JB * 4), u = unit % (WR * WC * IB * JB * 4);
    if (tile >= tiles) return;
    const uint32_t wave = u / (IB * JB * 4), ij = u / 4 % (IB * JB), q = u % 4;
    const int64_t i = (int64_t)(tile / gj) * TI + (wave / WC) * (32 * IB) + 32 * (ij / JB) + 8 * q + 4 * (lane >> 5);
    const int64_t j = (int64_t)(tile % gj) * TJ + (wave % WC) * (32 * JB) + 32 * (ij % JB) + (lane & 31);
    if (i >= p.I || j >= p.J) return;
    const GLB f32x4* src = (const GLB f32x4*)p.partial + (size_t)unit * 64 + lane;
    const size_t step = (size_t)tiles * (WR * WC * IB * JB * 4 * 64);
    f32x4 v = *src;
#pragma unroll 8
    for (int s = 1; s < p.splits; ++s) {                      // (loads of several parts in flight together)
        src += step;
        const f32x4 x = *src;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += x[e];
    }
    const Epilogue& e = p.e;
    const float bias = !e.bias ? 0.0f : e.bias_dtype == PGQ_F32 ? ((const GLB float*)e.bias)[j] : bf16_to_f32(((const GLB uint16_t*)e.bias)[j]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t row = i + k;
        if (row >= p.I) break;
        float x = v[k] + bias;
        if (e.z) ((GLB uint16_t*)e.z)[row * e.ldz + j] = f32_to_bf16(x);
        x = act_value(e.act, e.slope, x);
        if (e.residual)
            x += e.residual_dtype == PGQ_F32 ? ((const GLB float*)e.residual)[row * e.ldr + j]
                                             : bf16_to_f32(((const GLB uint16_t*)e.residual)[row * e.ldr + j]);
        if (e.y_dtype == PGQ_F32) ((GLB float*)e.y)[row * e.ldy + j] = x;
        else ((GLB uint16_t*)e.y)[row * e.ldy + j] = f32_to_bf16(x);
    }
}

// The tiles a product can be cut into.  stage: microseconds of one 64-wide stage of a workgroup that has its
// compute unit alone; busy: a stage's share of a compute unit that several keep busy; per_cu: how many fit; start:
// the launch, the first loads and the last stores.  Fitted to the clock over the sizes at mm_nt_plan.
struct NtKind {
    int ti, tj, threads, per_cu;
    double stage, busy, start;
    const void *f32, *bf16, *reduce;
    bool codes;                                   // B as codes
};
template <int WR, int WC, int IB, int JB, bool Q, int NB, int NA = NB>
NtKind nt_kind(int per_cu, double stage, double busy, double start = 4.0)
{
    return {32 * IB * WR, 32 * JB * WC, 64 * WR * WC, per_cu, stage, busy, start,
            reinterpret_cast<const void*>(&pgq_mm_nt_kernel<WR, WC, IB, JB, Q, NB, NA, float>),
            reinterpret_cast<const void*>(&pgq_mm_nt_kernel<WR, WC, IB, JB, Q, NB, NA, uint16_t>),
            reinterpret_cast<const void*>(&pgq_mm_nt_reduce_kernel<WR, WC, IB, JB>), Q};
}
// (256 x 192 beside 256 x 256 for outputs that end shortly behind a multiple of 256; whole calls, inputs from memory:
// 16384 x 528 x 1584 with an fp32 residual takes 59 us with it against 64, with bf16 Y alone 46 against 51;
// 16384 x 1584 x 528 65 against 50)
const NtKind kNt[] = {nt_kind<2, 4, 4, 2, false, 2, 3>(1, 1.70, 1.60), nt_kind<2, 2, 2, 2, false, 2, 3>(2, 0.50, 0.55), nt_kind<2, 2, 2, 1, false, 3>(2, 0.50, 0.36),
                      nt_kind<2, 2, 1, 1, false, 4>(2, 0.33, 0.24), nt_kind<1, 4, 4, 1, true, 3>(2, 0.50, 0.62, 6.0),
                      nt_kind<1, 4, 2, 1, true, 4>(2, 0.55, 0.40), nt_kind<4, 2, 2, 3, false, 2, 3>(1, 1.35, 1.35)};
int64_t nt_tiles(const NtKind& k, int64_t I, int64_t J) { return ((I + k.ti - 1) / k.ti) * ((J + k.tj - 1) / k.tj); }

// ---- A columns times B columns ----------------------------------------------------------------------
// The contraction runs down the rows of both operands (dW sums over tokens).  A stage is 64 rows of TI and
// TJ columns, loaded straight into LDS as they lie in memory; ds_read_b64_tr_b16 transposes on the way to the
// registers: the 16 lanes of a group read four rows of 16 columns (lane i the columns 4 (i % 4) .. + 3 of row
// i / 4) and lane i receives column i of the four rows (checked on the device).
//
// A group's four rows are one row pitch apart, a multiple of 128 bytes, so their 32-byte pieces would share
// banks: granule g (16 bytes) of row r sits in slot g ^ turn(r), which moves the four rows 64 bytes apart.
template <int COLS>
__device__ __forceinline__ int turn(int r)
{
    return COLS % 128 == 0 ? 4 * (r & 3) : 4 * ((r >> 1) & 1);      // pitch 0 or 128 modulo 256 bytes
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

__device__ __forceinline__ bool mask_bit(const uint8_t* mask, int64_t J, int64_t i, int64_t j)
{
    return !mask || ((((const GLB uint8_t*)mask)[i * ((J + 7) / 8) + (j >> 3)] >> (j & 7)) & 1);
}
// rows i .. i + 3 of column j
__device__ __forceinline__ void put4(const MmTt& p, int64_t i, int64_t j, f32x4 v)
{
    if (j >= p.J) return;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (i + e < p.I) {
            const float x = mask_bit(p.mask, p.J, i + e, j) ? v[e] : 0.0f;
            if (p.c_dtype == PGQ_F32) ((GLB float*)p.c)[(i + e) * p.ldc + j] = x;
            else ((GLB uint16_t*)p.c)[(i + e) * p.ldc + j] = f32_to_bf16(x);
        }
}

__host__ __device__ inline int64_t tt_stages(const MmTt& p) { return (p.L + 63) / 64 * p.parts; }

template <int WR, int WC, int IB, int JB>
constexpr int tt_lds() { return 2 * 64 * 2 * (32 * IB * WR + 32 * JB * WC); }

template <int WR, int WC, int IB, int JB>
__device__ __forceinline__ void tt_body(const MmTt& p, uint32_t wid, uint32_t total, uint8_t* lds)
{
    constexpr int T = 64 * WR * WC, TI = 32 * IB * WR, TJ = 32 * JB * WC;
    constexpr int AG = TI / 8, BG = TJ / 8;                  // granules per row
    constexpr int AI = 64 * AG / T, BI = 64 * BG / T;        // load instructions per thread per stage
    constexpr int AS = 64 * TI * 2, BS = 64 * TJ * 2;
    static_assert(64 * AG % T == 0 && 64 * BG % T == 0, "whole load instructions");
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t gi = (uint32_t)((p.I + TI - 1) / TI), gj = (uint32_t)((p.J + TJ - 1) / TJ), tiles = gi * gj;
    uint32_t ti, tj, part;       // the tiles of one part read the same rows: they share an XCD
    tile_of(wid, total, gi, gj, ti, tj, part);
    const uint32_t tile = ti * gj + tj;
    const int64_t i0 = (int64_t)ti * TI, j0 = (int64_t)tj * TJ;
    // this piece's stages: 64 rows of each part of A in turn, with the same rows of B (the second read of them is served
    // by the cache)
    const int64_t first = (int64_t)part * p.chunk;
    const int nst = (int)min(p.chunk, tt_stages(p) - first);
    const uint32_t block = (uint32_t)first / (uint32_t)p.parts;
    int64_t row = (int64_t)block * 64;           // of the stage that is issued next, and its part
    int which = (int)((uint32_t)first - block * (uint32_t)p.parts);
    const int ig = (int)min((int64_t)AG, (p.I - i0 + 7) / 8), jg = (int)min((int64_t)BG, (p.J - j0 + 7) / 8);
    uint32_t ao[AI], bo[BI];     // byte offsets of this thread's loads within a stage; columns past the edge are out of range
#pragma unroll
    for (int c = 0; c < AI; ++c) {
        const int s = c * T + tid, r = s / AG, g = (s % AG) ^ turn<TI>(r);
        ao[c] = g < ig ? (uint32_t)r * (uint32_t)p.lda * 2u + 16u * g : kOOB;
    }
#pragma unroll
    for (int c = 0; c < BI; ++c) {
        const int s = c * T + tid, r = s / BG, g = (s % BG) ^ turn<TJ>(r);
        bo[c] = g < jg ? (uint32_t)r * (uint32_t)p.ldb * 2u + 16u * g : kOOB;
    }
    auto issue = [&](int st) __attribute__((always_inline)) {
        uint8_t* la = lds + (st & 1) * (AS + BS);
        uint8_t* lb = la + AS;
        const int rows = (int)min((int64_t)64, p.L - row);
        // ranges over this stage's rows: the last one ends with its last used granule, rows past it are out of range
        const __amdgpu_buffer_rsrc_t ar = __builtin_amdgcn_make_buffer_rsrc((void*)(p.a + row * p.lda + which * p.part_cols + i0), 0, (int)((rows - 1) * p.lda * 2 + 16 * ig), 0x00020000);
        const __amdgpu_buffer_rsrc_t br = __builtin_amdgcn_make_buffer_rsrc((void*)(p.b + row * p.ldb + j0), 0, (int)((rows - 1) * p.ldb * 2 + 16 * jg), 0x00020000);
#pragma unroll
        for (int c = 0; c < AI; ++c)
            load_lds(ar, la + (c * T + wave * 64) * 16, ao[c], 0);
#pragma unroll
        for (int c = 0; c < BI; ++c)
            load_lds(br, lb + (c * T + wave * 64) * 16, bo[c], 0);
        if (++which == p.parts) {
            which = 0;
            row += 64;
        }
    };
    const int wi = (wave / WC) * (32 * IB), wj = (wave % WC) * (32 * JB);
    const int h = lane >> 5, r32 = lane & 31;
    f32x16 acc[IB][JB];
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j) acc[i][j] = f32x16{};
    struct Frag {
        bf16x8 a[IB][2], b[JB][2];
    } f0, f1;
    // half stage kb: lane half h supplies l = 32 kb + 16 t + 8 h .. + 7 in instruction t, four at a read
    const int rl = 8 * h + ((lane >> 2) & 3);                          // row in the half stage, t = 0, first read
    const int gc = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);          // granule in a block's 32 columns
    auto read8 = [&](const uint8_t* base, int pitch) __attribute__((always_inline)) -> bf16x8 {
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)base);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(base + 4 * pitch));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto fetch = [&](Frag& f, int st, int kb) __attribute__((always_inline)) {
        const uint8_t* la = lds + (st & 1) * (AS + BS) + (32 * kb + rl) * (2 * TI) + (lane & 1) * 8;
        const uint8_t* lb = lds + (st & 1) * (AS + BS) + AS + (32 * kb + rl) * (2 * TJ) + (lane & 1) * 8;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int i = 0; i < IB; ++i)
                f.a[i][t] = read8(la + 16 * t * (2 * TI) + ((((wi + 32 * i) >> 3) + gc) ^ turn<TI>(rl)) * 16, 2 * TI);
#pragma unroll
            for (int j = 0; j < JB; ++j)
                f.b[j][t] = read8(lb + 16 * t * (2 * TJ) + ((((wj + 32 * j) >> 3) + gc) ^ turn<TJ>(rl)) * 16, 2 * TJ);
        }
    };
    auto multiply = [&](const Frag& f) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < IB; ++i)
#pragma unroll
                for (int j = 0; j < JB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i][t], f.b[j][t], acc[i][j], 0, 0, 0);
    };
    if (nst > 0) {
        issue(0);
        wait_barrier<0>();
        if (nst > 1) issue(1);
        fetch(f0, 0, 0);
    }
    int st = 0;
    if constexpr (kSpread<IB, JB>) {
        // past the edge: only this wavefront's share of the loads (1584 x 528 x 16384 in one part, with its dX: 96 -> 91 us;
        // 1584 rows of dW leave three quarters of the last tile row empty)
        if (i0 + wi >= p.I || j0 + wj >= p.J) {
            for (; st < nst; ++st) {
                wait_barrier<0>();
                if (st + 2 < nst) issue(st + 2);
            }
            return;
        }
        for (; st + 1 < nst; ++st) {                          // all but the last stage
            fetch(f1, st, 1);
            multiply(f0);
            spread<4 * (IB + JB), 2 * IB * JB>();
            wait_barrier<0>();
            if (st + 2 < nst) issue(st + 2);
            fetch(f0, st + 1, 0);
            multiply(f1);
            spread<4 * (IB + JB), 2 * IB * JB>();
        }
    }
    for (; st < nst; ++st) {
        fetch(f1, st, 1);
        multiply(f0);
        wait_barrier<0>();
        if (st + 2 < nst) issue(st + 2);
        if (st + 1 < nst) fetch(f0, st + 1, 0);
        multiply(f1);
    }
    // one part: to C; several: the parts' sums as they lie in the registers, 16 bytes a lane
    f32x4* out = reinterpret_cast<f32x4*>(p.partial) + (((size_t)part * tiles + tile) * (WR * WC) + wave) * (IB * JB * 4 * 64) + lane;
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                if (p.splits > 1) {
                    if (i0 + wi + 32 * i < p.I && j0 + wj + 32 * j < p.J) out[((i * JB + j) * 4 + q) * 64] = v;
                } else {
                    put4(p, i0 + wi + 32 * i + 8 * q + 4 * h, j0 + wj + 32 * j + r32, v);
                }
            }
}

template <int WR, int WC, int IB, int JB>
__global__ void __launch_bounds__(64 * WR * WC) __attribute__((amdgpu_waves_per_eu(2)))
pgq_mm_tt_kernel(MmTt p)
{
    __shared__ __align__(16) uint8_t lds[tt_lds<WR, WC, IB, JB>()];
    tt_body<WR, WC, IB, JB>(p, blockIdx.x, gridDim.x, lds);
}

// db[n]: the row blocks' partial sums for 64 columns, sixteen phases of blocks joined in order, by any number of
// wavefronts (the order of the additions does not depend on it)
__device__ __forceinline__ void dbias_body(const Dbias& p, uint32_t unit, uint8_t* lds)
{
    float(*sums)[64] = reinterpret_cast<float(*)[64]>(lds);
    const int lane = (int)threadIdx.x & 63, waves = (int)blockDim.x >> 6;
    const int64_t n = (int64_t)unit * 64 + lane;
    for (int phase = (int)threadIdx.x >> 6; phase < 16; phase += waves) {
        float s = 0.0f;
        if (n < p.N) {
#pragma unroll 8
            for (int64_t i = phase; i < p.blocks; i += 16) s += ((const GLB float*)p.part)[i * p.N + n];
        }
        sums[phase][lane] = s;
    }
    __syncthreads();
    if (threadIdx.x < 64 && n < p.N) {
        float v = sums[0][lane];
#pragma unroll
        for (int i = 1; i < 16; ++i) v += sums[i][lane];
        p.out[n] = v;
    }
}
__global__ void __launch_bounds__(1024) pgq_mm_dbias_kernel(Dbias p)
{
    __shared__ __align__(16) uint8_t lds[16 * 64 * 4];
    dbias_body(p, blockIdx.x, lds);
}

// A whole backward pass after its operands are laid out: the tiles of dX, those of dW and the sums of db are
// independent, so one launch holds them all and the second product fills the compute units that the first
// leaves idle in its last round.
template <int A0, int A1, int A2, int A3, int NB, int NA, int B0, int B1, int B2, int B3, typename YT>
__global__ void __launch_bounds__(64 * A0 * A1) __attribute__((amdgpu_waves_per_eu(2)))
pgq_mm_both_kernel(MmNt x, MmTt w, Dbias d, uint32_t nx, uint32_t nw)
{
    static_assert(A0 * A1 == B0 * B1, "one block size");
    constexpr int LX = nt_lds<A0, A1, A2, A3, false, NB, NA>(), LW = tt_lds<B0, B1, B2, B3>();
    __shared__ __align__(16) uint8_t lds[LX > LW ? LX : LW];
    if (blockIdx.x < nx) nt_body<A0, A1, A2, A3, false, NB, NA, YT>(x, blockIdx.x, nx, lds);
    else if (blockIdx.x < nx + nw) tt_body<B0, B1, B2, B3>(w, blockIdx.x - nx, nw, lds);
    else dbias_body(d, blockIdx.x - nx - nw, lds);
}

template <int WR, int WC, int IB, int JB>
__global__ void __launch_bounds__(256) pgq_mm_tt_reduce_kernel(MmTt p)
{
    constexpr int TI = 32 * IB * WR, TJ = 32 * JB * WC;
    const uint32_t gi = (uint32_t)((p.I + TI - 1) / TI), gj = (uint32_t)((p.J + TJ - 1) / TJ), tiles = gi * gj;
    const uint32_t unit = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;      // one wave: 8 rows of 32 columns
    const uint32_t tile = unit / (WR * WC * IB * JB * 4), u = unit % (WR * WC * IB * JB * 4);
    if (tile >= tiles) return;
    const uint32_t wave = u / (IB * JB * 4), ij = u / 4 % (IB * JB), q = u % 4;
    const int64_t i = (int64_t)(tile / gj) * TI + (wave / WC) * (32 * IB) + 32 * (ij / JB);
    const int64_t j = (int64_t)(tile % gj) * TJ + (wave % WC) * (32 * JB) + 32 * (ij % JB);
    if (i >= p.I || j >= p.J) return;
    const GLB f32x4* src = (const GLB f32x4*)p.partial + (size_t)unit * 64 + lane;
    const size_t step = (size_t)tiles * (WR * WC * IB * JB * 4 * 64);
    f32x4 v = *src;
#pragma unroll 8
    for (int s = 1; s < p.splits; ++s) {                      // (loads of several parts in flight together)
        src += step;
        const f32x4 x = *src;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += x[e];
    }
    put4(p, i + 8 * q + 4 * (lane >> 5), j + (lane & 31), v);
}

// The tiles a product can be cut into.  stage: microseconds of one 64-row stage with every slot busy (what the
// choice below weighs; measured at 4096 x 4096 x 8192 and 1584 x 528 x 16384).
struct TtKind {
    int ti, tj, threads, slots;                   // slots: workgroups that run at once
    double stage;
    const void *kernel, *reduce;
};
template <int WR, int WC, int IB, int JB>
TtKind tt_kind(int slots, double stage)
{
    return {32 * IB * WR, 32 * JB * WC, 64 * WR * WC, slots, stage,
            reinterpret_cast<const void*>(&pgq_mm_tt_kernel<WR, WC, IB, JB>),
            reinterpret_cast<const void*>(&pgq_mm_tt_reduce_kernel<WR, WC, IB, JB>)};
}
const TtKind kTt[] = {tt_kind<4, 2, 2, 4>(256, 1.9), tt_kind<4, 2, 2, 3>(256, 1.5), tt_kind<2, 2, 2, 2>(512, 1.1),
                      tt_kind<2, 2, 1, 1>(768, 0.8)};
int64_t tt_tiles(const TtKind& k, int64_t I, int64_t J) { return ((I + k.ti - 1) / k.ti) * ((J + k.tj - 1) / k.tj); }

}  // namespace

// Microseconds that workgroups of `per` stages each take: whole rounds over the places, then the rest.  A rest of at most
// one workgroup a compute unit runs at the lone workgroup's pace, more at a pace between the two; a tile that has
// its unit to itself runs a stage faster the fewer units are at work: the model goes straight from `busy` with all of
// them to 0.8 of it with none.  Measured, as the difference of 128 and 32 stages: 256 x 256 1.74 us with all, 1.28 with
// half and 1.22 with a quarter, where the model has 1.60, 1.44 and 1.36; 256 x 192 1.39, 1.03 and 1.00 (1.35, 1.22, 1.15).
static double rounds_of_stages(const NtKind& kind, int64_t wgs, double per)
{
    const int64_t places = 256 * kind.per_cu, full = wgs / places, rest = wgs % places;
    if (kind.per_cu == 1) {
        const double last = kind.busy * (0.8 + 0.2 * (double)rest / 256.0);
        return (double)full * (per * kind.busy + 2.0) + (rest ? per * last + 2.0 : 0.0) + 2.0;
    }
    const double both = kind.busy * (double)kind.per_cu;
    const double last = rest <= 256 ? kind.stage : kind.stage + (both - kind.stage) * (double)(rest - 256) / (double)(places - 256);
    return (double)full * per * both + (rest ? per * last : 0.0) + kind.start;
}

// The tile and the number of parts with the least estimated time: the stages, the trip of the outputs (5.3 MB a
// microsecond: the stores of a tile hardly overlap its stages) and, for parts, their sums' trip and a launch.  Every tile
// timed against the choice at 31 sizes from 96 x 1584 x 528 to 8192 x 8192 x 1024 (X from memory): the tile chosen is
// within 7% of the best at 30 of them; at 4899 x 947 x 4656, whose rows of X straddle cache lines, it is 26% off.
double mm_nt_plan(MmNt& p, bool codes_ok, double out_bytes)
{
    double best = 0;
    // laying What out: codes in, bf16 out, and a launch
    const double layout = codes_ok ? 4.0 + (double)p.J * (double)p.L * 3.0 / 4e6 : 0.0;
    const double out = (double)p.I * (double)p.J * out_bytes / 5.3e6;
    const int64_t stages = std::max<int64_t>(1, nt_stages(p));
    for (int k = 0; k < (int)(sizeof(kNt) / sizeof(kNt[0])); ++k) {
        const NtKind& kind = kNt[k];
        if (kind.codes && !codes_ok) continue;
        const int64_t tiles = nt_tiles(kind, p.I, p.J);
        for (int64_t s = 1; s <= 16; s *= 2) {
            const int64_t per = (stages + s - 1) / s, parts = (stages + per - 1) / per;
            if (s > 1 && (parts != s || per < 4 || tiles * parts > 512)) break;
            const int64_t wgs = tiles * parts;
            double t = out + rounds_of_stages(kind, wgs, (double)per);
            if (parts > 1) t += 4.0 + (double)wgs * kind.ti * kind.tj * 8.0 / 5e6;
            if (!kind.codes) t += layout;
            if (best == 0 || t < best) {
                best = t;
                p.kind = k;
                p.from_codes = kind.codes;
                p.splits = (int32_t)parts;
                p.chunk = per * 64;
            }
        }
    }
    return best;
}

size_t mm_nt_partial_bytes(const MmNt& p)
{
    const NtKind& k = kNt[p.kind];
    return p.splits > 1 ? (size_t)p.splits * (size_t)nt_tiles(k, p.I, p.J) * k.ti * k.tj * 4 : 0;
}

void mm_nt_tile(const MmNt& p, int32_t* rows, int32_t* cols)
{
    *rows = kNt[p.kind].ti;
    *cols = kNt[p.kind].tj;
}
void mm_tt_tile(const MmTt& p, int32_t* rows, int32_t* cols)
{
    *rows = kTt[p.kind].ti;
    *cols = kTt[p.kind].tj;
}
static int64_t nt_grid(const MmNt& p) { return nt_tiles(kNt[p.kind], p.I, p.J) * p.splits; }
static int64_t nt_reduce_grid(const MmNt& p)
{
    const NtKind& k = kNt[p.kind];
    return p.splits > 1 ? nt_tiles(k, p.I, p.J) * (k.ti * k.tj / 256) / 4 : 0;
}
bool mm_nt_fits(const MmNt& p) { return grid_fits(nt_grid(p), kNt[p.kind].threads) && grid_fits(nt_reduce_grid(p), 256); }

hipError_t launch_mm_nt(const MmNt& p, void* stream)
{
    const NtKind& k = kNt[p.kind];
    const int64_t grid = nt_grid(p);
    MmNt copy = p;
    void* args[] = {&copy};
    return launch_grid(p.e.y_dtype == PGQ_F32 ? k.f32 : k.bf16, grid, k.threads, args, stream);
}

hipError_t launch_mm_nt_reduce(const MmNt& p, void* stream)
{
    const NtKind& k = kNt[p.kind];
    const int64_t grid = nt_reduce_grid(p);
    MmNt copy = p;
    void* args[] = {&copy};
    return launch_grid(k.reduce, grid, 256, args, stream);
}

// The tile and the number of parts with the least estimated time: stages of a part times the rounds its
// workgroups take, plus the trip of the parts' sums and a launch.
constexpr int kParts[] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16, 20, 24, 32, 48, 64};
void mm_tt_plan(MmTt& p)
{
    double best = 0;
    const int64_t stages = std::max<int64_t>(1, tt_stages(p));
    for (int k = 0; k < (int)(sizeof(kTt) / sizeof(kTt[0])); ++k) {
        const TtKind& kind = kTt[k];
        const int64_t tiles = tt_tiles(kind, p.I, p.J);
        for (const int s : kParts) {
            const int64_t per = (stages + s - 1) / s, parts = (stages + per - 1) / per;
            if (s > 1 && (parts != s || tiles * parts > 4 * kind.slots)) continue;
            const int64_t rounds = (tiles * parts + kind.slots - 1) / kind.slots;
            double t = (double)rounds * ((double)per * kind.stage + 4.0);
            if (parts > 1) t += 4.0 + (double)(tiles * parts) * kind.ti * kind.tj * 5.5 / 6e6;
            if (best == 0 || t < best) {
                best = t;
                p.kind = k;
                p.splits = (int32_t)parts;
                p.chunk = per;
            }
        }
    }
}

// The pairs of tiles that dX and dW run with in one launch.
struct BothKind {
    int nt, tt;                                   // places in kNt, kTt
    int per_cu;
    double nt_stage, tt_stage;                    // microseconds of a stage when every unit is busy, times per_cu
    const void *f32, *bf16;
};
template <int A0, int A1, int A2, int A3, int NB, int NA, int B0, int B1, int B2, int B3>
BothKind both_kind(int nt, int tt, int per_cu, double nt_stage, double tt_stage)
{
    return {nt, tt, per_cu, nt_stage, tt_stage,
            reinterpret_cast<const void*>(&pgq_mm_both_kernel<A0, A1, A2, A3, NB, NA, B0, B1, B2, B3, float>),
            reinterpret_cast<const void*>(&pgq_mm_both_kernel<A0, A1, A2, A3, NB, NA, B0, B1, B2, B3, uint16_t>)};
}
const BothKind kBoth[] = {both_kind<2, 4, 4, 2, 2, 3, 4, 2, 2, 4>(0, 0, 1, 1.75, 1.9), both_kind<2, 4, 4, 2, 2, 3, 4, 2, 2, 3>(0, 1, 1, 1.75, 1.5),
                          both_kind<2, 2, 2, 2, 2, 3, 2, 2, 2, 2>(1, 2, 2, 1.4, 1.1), both_kind<2, 2, 1, 1, 4, 4, 2, 2, 1, 1>(3, 3, 2, 0.45, 0.5),
                          both_kind<4, 2, 2, 3, 2, 3, 4, 2, 2, 3>(6, 1, 1, 1.40, 1.5)};

// When `first` workgroups of one_first microseconds and then `second` of one_second each, taken in that order by
// `slots` places, are done: the places free after the first kind's last whole round start at t0, the others at
// t1; the answer is a multiple of one_second after one of these.
double two_kinds_done(int64_t slots, int64_t first, double one_first, int64_t second, double one_second)
{
    const int64_t rem = first % slots;
    const double t0 = (double)(first / slots) * one_first, t1 = t0 + (rem ? one_first : 0.0);
    for (int64_t k = 0;; ++k) {
        const double ta = t0 + (double)k * one_second;                    // k workgroups on each early place
        const int64_t late = ta > t1 ? (int64_t)((ta - t1) / one_second) : 0;
        if ((slots - rem) * k + rem * late >= second) return std::max(ta, t1);
        const double tb = t1 + (double)(late + 1) * one_second;           // one more on each late place first
        const int64_t early = (int64_t)((tb - t0) / one_second);
        if (tb < ta + one_second && (slots - rem) * early + rem * (late + 1) >= second) return tb;
    }
}

// The pair and the parts with the least estimated time: both kinds of workgroup over the places, the way out of
// dX, the trip of the parts' sums (written beside the other work, read back at 6 MB a microsecond), a launch for
// parts.
int mm_both_plan(MmNt& x, MmTt& w, double out_bytes)
{
    double best = 0;
    int chosen = 0;
    const int64_t sx = std::max<int64_t>(1, nt_stages(x)), sw = std::max<int64_t>(1, tt_stages(w));
    const double out = (double)x.I * (double)x.J * out_bytes / 5.3e6;
    for (int k = 0; k < (int)(sizeof(kBoth) / sizeof(kBoth[0])); ++k) {
        const BothKind& b = kBoth[k];
        const NtKind& nk = kNt[b.nt];
        const TtKind& tk = kTt[b.tt];
        const int64_t tx = nt_tiles(nk, x.I, x.J), tw = tt_tiles(tk, w.I, w.J), slots = 256 * b.per_cu;
        for (int64_t s = 1; s <= 16; s *= 2) {
            const int64_t perx = (sx + s - 1) / s, partx = (sx + perx - 1) / perx;
            if (s > 1 && (partx != s || perx < 4 || tx * partx > 2 * slots)) break;
            const double one_x = (double)perx * b.nt_stage + 3.0;
            for (const int s2 : kParts) {
                const int64_t perw = (sw + s2 - 1) / s2, partw = (sw + perw - 1) / perw;
                if (s2 > 1 && (partw != s2 || tw * partw > 4 * slots)) continue;
                const double one_w = (double)perw * b.tt_stage + 3.0;
                double t = two_kinds_done(slots, tx * partx, one_x, tw * partw, one_w) + out;
                if (partx > 1) t += 4.0 + (double)(tx * partx) * nk.ti * nk.tj * 5.5 / 6e6;
                if (partw > 1) t += 4.0 + (double)(tw * partw) * tk.ti * tk.tj * 5.5 / 6e6;
                if (best == 0 || t < best) {
                    best = t;
                    chosen = k;
                    x.splits = (int32_t)partx;
                    x.chunk = perx * 64;
                    w.splits = (int32_t)partw;
                    w.chunk = perw;
                }
            }
        }
    }
    x.kind = kBoth[chosen].nt;
    x.from_codes = 0;
    w.kind = kBoth[chosen].tt;
    return chosen;
}

static int64_t tt_grid(const MmTt& p) { return tt_tiles(kTt[p.kind], p.I, p.J) * p.splits; }
static int64_t tt_reduce_grid(const MmTt& p)               // a wavefront: 8 rows of 32 columns
{
    const TtKind& k = kTt[p.kind];
    return p.splits > 1 ? tt_tiles(k, p.I, p.J) * (k.ti * k.tj / 256) / 4 : 0;
}
static int64_t dbias_grid(int64_t N) { return (N + 63) / 64; }
bool mm_tt_fits(const MmTt& p) { return grid_fits(tt_grid(p), kTt[p.kind].threads) && grid_fits(tt_reduce_grid(p), 256); }
bool mm_dbias_fits(int64_t N) { return grid_fits(dbias_grid(N), 1024); }
bool mm_both_fits(const MmNt& x, const MmTt& w, int64_t db_cols)
{
    return grid_fits(nt_grid(x) + tt_grid(w) + dbias_grid(db_cols), kNt[x.kind].threads) && grid_fits(nt_reduce_grid(x), 256) &&
           grid_fits(tt_reduce_grid(w), 256);
}

hipError_t launch_mm_both(int both, const MmNt& x, const MmTt& w, const Dbias& d, void* stream)
{
    const BothKind& b = kBoth[both];
    const int64_t nx = nt_grid(x), nw = tt_grid(w);
    const int64_t grid = nx + nw + (d.out ? dbias_grid(d.N) : 0);
    MmNt cx = x;
    MmTt cw = w;
    Dbias cd = d;
    uint32_t ux = (uint32_t)nx, uw = (uint32_t)nw;
    void* args[] = {&cx, &cw, &cd, &ux, &uw};
    return launch_grid(x.e.y_dtype == PGQ_F32 ? b.f32 : b.bf16, grid, kNt[x.kind].threads, args, stream);
}

hipError_t launch_mm_dbias(const Dbias& d, void* stream)
{
    Dbias copy = d;
    void* args[] = {&copy};
    return launch_grid(reinterpret_cast<const void*>(&pgq_mm_dbias_kernel), dbias_grid(d.N), 1024, args, stream);
}

size_t mm_tt_partial_bytes(const MmTt& p)
{
    const TtKind& k = kTt[p.kind];
    return p.splits > 1 ? (size_t)p.splits * (size_t)tt_tiles(k, p.I, p.J) * k.ti * k.tj * 4 : 0;
}

hipError_t launch_mm_tt(const MmTt& p, void* stream)
{
    const TtKind& k = kTt[p.kind];
    const int64_t grid = tt_grid(p);
    MmTt copy = p;
    void* args[] = {&copy};
    return launch_grid(k.kernel, grid, k.threads, args, stream);
}

hipError_t launch_mm_tt_reduce(const MmTt& p, void* stream)
{
    const TtKind& k = kTt[p.kind];
    const int64_t grid = tt_reduce_grid(p);
    MmTt copy = p;
    void* args[] = {&copy};
    return launch_grid(k.reduce, grid, 256, args, stream);
}

}  // namespace pgq
