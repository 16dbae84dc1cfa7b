// pgq_gradnorm.hip -- the global norm of many gradient tensors and clipping to it (gfx950).
//
// norm = |c| sqrt(sum g^2); factor = min(1, max_norm / norm).  One launch for every 128 tensors reads each once: a
// workgroup takes a tile of one tensor, squares and adds in 64 bits (an fp64 multiply-add goes at the rate of
// an fp32 one here, no square overflows, and the sum of 2^36 squares is still good to 2^-52 or so of itself for
// each addition), and writes one partial sum.  The last launch's workgroup that finishes last adds the partial sums, always in
// the same order, and writes norm and factor: no launch of its own for that, and no atomic whose order the result depends on.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <utility>

#include "pgq_linear.h"
#include "pgq_train.h"
#include "../../include/pgq.h"

namespace pgq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kArgTensors = 128;                  // tensors in the kernel arguments of a launch
// Elements of the smallest tile.  Lists of less than 16 M elements have fewer tiles than would fill the machine, which costs little: calls
// of 0.1, 1, 2 and 4 M fp32 elements take 5.0, 5.1, 5.8 and 7.3 us, of which 5 are any call's (smaller tiles have not been measured).
constexpr int64_t kTile = 16384;
// Tiles grow until about so many are left, 4 workgroups a compute unit (30.7 M bf16 a call 13.3 us, with 2048 15.0, with 512 14.0).
constexpr int64_t kTilesWanted = 1024;
// Counts of finished workgroups.  One counter takes an increment every 13 ns, which for 1900 workgroups is longer than the
// reading (30.7 M bf16: 32 us), so large grids count in kCounters groups and then the groups.  Each counter has a cache
// line, and a memory channel, of its own.
constexpr uint32_t kCounters = 16;
constexpr uint32_t kOneCounter = 256;             // workgroups that a single counter is enough for: one step less at the end
constexpr int kCounterBytes = 256;
constexpr size_t kCountersBytes = (size_t)kCounterBytes * (kCounters + 1);
constexpr int64_t kMaxNumel = (int64_t)1 << 40;

struct Tensors {
    const void* p[kArgTensors];
    int64_t numel[kArgTensors];
    uint32_t end[kArgTensors];                    // one past the last tile of each, from this launch's first
    uint8_t dtype[kArgTensors];
};

struct NormArgs {
    uint8_t* counters;
    double* part;
    float* result;
    uint32_t* status;
    const float* scale_dev;
    float scale, max_norm;
    int64_t tile;                                 // elements
    uint32_t first, total;                        // this launch's first partial sum, partial sums in all
    int32_t last;                                 // 1: no launch of this call comes after this one
};

// One more workgroup of the grid is done: true in the one that is last.  Counters wrap to 0 for the next call.
__device__ __forceinline__ bool is_last(uint8_t* counters)
{
    auto count = [&](uint32_t i, uint32_t most) { return atomicInc(reinterpret_cast<uint32_t*>(counters + i * kCounterBytes), most - 1) == most - 1; };
    const uint32_t grid = gridDim.x;
    if (grid <= kOneCounter) return count(0, grid);
    const uint32_t g = blockIdx.x % kCounters;
    return count(1 + g, (grid - g + kCounters - 1) / kCounters) && count(0, kCounters);
}

// the tensor of a tile: the number of tensors that end at or before it (unused entries end past every tile; without any tensor, the
// one workgroup of the launch finds entry 0, of no elements)
__device__ __forceinline__ int tensor_of(const Tensors& t, uint32_t tile)
{
    const int lane = (int)threadIdx.x & 63;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kArgTensors; i += 64) n += __popcll(__ballot(t.end[i + lane] <= tile));
    return n;
}

// 16 bytes of T as fp32 values
template <typename T>
__device__ __forceinline__ void unpack(u32x4 v, float* f);
struct Bf16 { uint16_t b; };
struct F16 { uint16_t b; };
template <>
__device__ __forceinline__ void unpack<float>(u32x4 v, float* f)
{
    const f32x4 x = __builtin_bit_cast(f32x4, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = x[e];
}
template <>
__device__ __forceinline__ void unpack<Bf16>(u32x4 v, float* f)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __builtin_bit_cast(float, v[e] << 16);
        f[2 * e + 1] = __builtin_bit_cast(float, v[e] & 0xFFFF0000u);
    }
}
template <>
__device__ __forceinline__ void unpack<F16>(u32x4 v, float* f)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = f16_to_f32((uint16_t)v[e]);
        f[2 * e + 1] = f16_to_f32((uint16_t)(v[e] >> 16));
    }
}
__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(Bf16 x) { return bf16_to_f32(x.b); }
__device__ __forceinline__ float value(F16 x) { return f16_to_f32(x.b); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(Bf16* p, float v) { p->b = f32_to_bf16(v); }
__device__ __forceinline__ void put(F16* p, float v) { p->b = __builtin_bit_cast(uint16_t, (_Float16)v); }

template <typename T>
__device__ __forceinline__ double sum_squares(const T* p, int64_t count)
{
    constexpr int V = 16 / sizeof(T), U = 4;      // elements of a load, loads in flight
    constexpr int64_t kStep = (int64_t)kThreads * V;
    double s[U] = {};
    auto add = [&](u32x4 v, double& a) __attribute__((always_inline)) {
        float f[V];
        unpack<T>(v, f);
#pragma unroll
        for (int e = 0; e < V; ++e) a = __builtin_fma((double)f[e], (double)f[e], a);
    };
    int64_t i = (int64_t)threadIdx.x * V;
    for (; i + (U - 1) * kStep + V <= count; i += U * kStep) {
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = load16(p + i + u * kStep);
#pragma unroll
        for (int u = 0; u < U; ++u) add(v[u], s[u]);
    }
    for (; i + V <= count; i += kStep) add(load16(p + i), s[0]);
    for (; i < count; ++i) {                      // (only the thread whose 16 bytes reach past the end)
        const double x = (double)value(p[i]);
        s[1] = __builtin_fma(x, x, s[1]);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// the sum over the workgroup, in thread 0
__device__ __forceinline__ double block_sum(double x, double* lds)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_down(x, d);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// norm and factor from the sum of squares; returns the factor
__device__ __forceinline__ float put_result(const NormArgs& a, double r)
{
    const double c = (double)(a.scale_dev ? *a.scale_dev : a.scale);
    const double norm = fabs(c) * sqrt(r);
    const float nf = (float)norm;
    const bool finite = nf < INFINITY;
    const float factor = !finite ? NAN : norm > (double)a.max_norm ? (float)((double)a.max_norm / norm) : 1.0f;
    a.result[0] = nf;
    a.result[1] = factor;
    if (!finite && a.status) atomicOr(a.status, PGQ_DEV_NONFINITE);
    return factor;
}

__global__ void __launch_bounds__(kThreads) pgq_grad_norm_kernel(NormArgs a, Tensors t)
{
    __shared__ double lds[2][kThreads / 64];
    __shared__ bool last;
    double s;
    const int ti = __builtin_amdgcn_readfirstlane(tensor_of(t, blockIdx.x));
    const int64_t base = (int64_t)(blockIdx.x - (ti > 0 ? t.end[ti - 1] : 0u)) * a.tile;
    const int64_t count = min(a.tile, t.numel[ti] - base);
    const int32_t dtype = t.dtype[ti];
    if (dtype == PGQ_F32) s = sum_squares(static_cast<const float*>(t.p[ti]) + base, count);
    else if (dtype == PGQ_BF16) s = sum_squares(static_cast<const Bf16*>(t.p[ti]) + base, count);
    else s = sum_squares(static_cast<const F16*>(t.p[ti]) + base, count);
    s = block_sum(s, lds[0]);
    if (threadIdx.x == 0) {
        __hip_atomic_store(a.part + a.first + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (a.last) {
            // The partial sums are stored and loaded past the caches that other compute units do not see (agent scope), so
            // the store's end is all there is to wait for; a fence would write the whole L2 back, once a workgroup
            // (61 MB of bf16: 100 us with it).
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            last = is_last(a.counters);
        }
    }
    if (!a.last) return;
    __syncthreads();
    if (!last) return;
    double r = 0.0;
#pragma unroll 8
    for (uint32_t i = threadIdx.x; i < a.total; i += kThreads) r += __hip_atomic_load(a.part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    r = block_sum(r, lds[1]);
    if (threadIdx.x != 0) return;
    put_result(a, r);
}

template <typename T>
__device__ __forceinline__ void scale_all(T* p, int64_t count, float factor)
{
    constexpr int V = 16 / sizeof(T), U = 4;
    constexpr int64_t kStep = (int64_t)kThreads * V;
    auto times = [&](u32x4 v) __attribute__((always_inline)) {
        float f[V];
        unpack<T>(v, f);
        T o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) put(o + e, f[e] * factor);
        __builtin_memcpy(&v, o, 16);
        return v;
    };
    int64_t i = (int64_t)threadIdx.x * V;
    for (; i + (U - 1) * kStep + V <= count; i += U * kStep) {
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = load16(p + i + u * kStep);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const u32x4 o = times(v[u]);
            __builtin_memcpy(p + i + u * kStep, &o, 16);
        }
    }
    for (; i + V <= count; i += kStep) {
        const u32x4 o = times(load16(p + i));
        __builtin_memcpy(p + i, &o, 16);
    }
    for (; i < count; ++i) put(p + i, value(p[i]) * factor);
}

__global__ void __launch_bounds__(kThreads) pgq_grad_scale_kernel(NormArgs a, Tensors t)
{
    const float factor = a.result[1];
    if (!(factor < 1.0f)) return;                 // 1, or NaN
    // the tiles last read come first: they are still in the caches
    const uint32_t tile = gridDim.x - 1 - blockIdx.x;
    const int ti = __builtin_amdgcn_readfirstlane(tensor_of(t, tile));
    const int64_t base = (int64_t)(tile - (ti > 0 ? t.end[ti - 1] : 0u)) * a.tile;
    const int64_t count = min(a.tile, t.numel[ti] - base);
    const int32_t dtype = t.dtype[ti];
    void* p = const_cast<void*>(t.p[ti]);
    if (dtype == PGQ_F32) scale_all(static_cast<float*>(p) + base, count, factor);
    else if (dtype == PGQ_BF16) scale_all(static_cast<Bf16*>(p) + base, count, factor);
    else scale_all(static_cast<F16*>(p) + base, count, factor);
}

// Clipping of a few small tensors in one launch: one workgroup, which keeps what it has read (16-byte pieces, kSmallPieces a
// thread) until the factor is known.  What bounds it is latency, of the piece's tensor, its load, the sum and the store, then what one
// compute unit can load; two launches against this one: 18 x 512 bf16 12.2 and 5.2 us, 45 x 257 fp32 12.6 and 7.3, 60 x 1000 bf16
// 12.9 and 9.4, 32768 fp32 (all the pieces there are) 9.7 and 8.0.
constexpr int kSmallThreads = 1024, kSmallPieces = 8;
constexpr int64_t kSmallMost = (int64_t)kSmallThreads * kSmallPieces;

template <typename T>
__device__ __forceinline__ double piece_squares(u32x4 v)
{
    constexpr int V = 16 / sizeof(T);
    float f[V];
    unpack<T>(v, f);
    double s = 0.0;
#pragma unroll
    for (int e = 0; e < V; ++e) s = __builtin_fma((double)f[e], (double)f[e], s);
    return s;
}
template <typename T>
__device__ __forceinline__ u32x4 piece_times(u32x4 v, float factor)
{
    constexpr int V = 16 / sizeof(T);
    float f[V];
    unpack<T>(v, f);
    T o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) put(o + e, f[e] * factor);
    __builtin_memcpy(&v, o, 16);
    return v;
}

// (t.end: one past the last piece of each tensor; a.total: pieces in all)
__global__ void __launch_bounds__(kSmallThreads) pgq_grad_clip_small_kernel(NormArgs a, Tensors t)
{
    __shared__ uint32_t end[kArgTensors];
    __shared__ double sums[kSmallThreads / 64];
    __shared__ float factor;
    const uint32_t tid = threadIdx.x;
    if (tid < kArgTensors) end[tid] = t.end[tid];
    __syncthreads();
    uint8_t* p[kSmallPieces];
    u32x4 v[kSmallPieces];
    int32_t bytes[kSmallPieces], dtype[kSmallPieces];
#pragma unroll
    for (int u = 0; u < kSmallPieces; ++u) {
        const uint32_t piece = tid + u * kSmallThreads;
        v[u] = u32x4{};
        bytes[u] = 0;
        dtype[u] = PGQ_F32;
        p[u] = nullptr;
        if (piece >= a.total) continue;
        uint32_t ti = 0;                          // tensors that end at or before the piece
#pragma unroll
        for (uint32_t d = kArgTensors / 2; d > 0; d /= 2)
            if (end[ti + d - 1] <= piece) ti += d;
        const uint32_t first = ti > 0 ? end[ti - 1] : 0u;
        dtype[u] = t.dtype[ti];
        const int64_t at = (int64_t)(piece - first) * 16, size = t.numel[ti] * (dtype[u] == PGQ_F32 ? 4 : 2);
        p[u] = static_cast<uint8_t*>(const_cast<void*>(t.p[ti])) + at;
        bytes[u] = (int32_t)min(size - at, (int64_t)16);
    }
#pragma unroll
    for (int u = 0; u < kSmallPieces; ++u) {
        if (bytes[u] == 16) v[u] = load16(p[u]);
        else
            for (int e = 0; e < bytes[u]; e += 2) {
                const uint32_t h = *reinterpret_cast<const uint16_t*>(p[u] + e);
                v[u][e >> 2] |= h << (8 * (e & 2));
            }
    }
    double s = 0.0;
#pragma unroll
    for (int u = 0; u < kSmallPieces; ++u)
        s += dtype[u] == PGQ_F32 ? piece_squares<float>(v[u]) : dtype[u] == PGQ_BF16 ? piece_squares<Bf16>(v[u]) : piece_squares<F16>(v[u]);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_down(s, d);
    if ((tid & 63) == 0) sums[tid >> 6] = s;
    __syncthreads();
    if (tid == 0) {
        double r = 0.0;
#pragma unroll
        for (int i = 0; i < kSmallThreads / 64; ++i) r += sums[i];
        factor = put_result(a, r);
    }
    __syncthreads();
    const float f = factor;
    if (!(f < 1.0f)) return;                      // 1, or NaN
#pragma unroll
    for (int u = 0; u < kSmallPieces; ++u) {
        const u32x4 o = dtype[u] == PGQ_F32 ? piece_times<float>(v[u], f) : dtype[u] == PGQ_BF16 ? piece_times<Bf16>(v[u], f) : piece_times<F16>(v[u], f);
        if (bytes[u] == 16) __builtin_memcpy(p[u], &o, 16);
        else
            for (int e = 0; e < bytes[u]; e += 2) *reinterpret_cast<uint16_t*>(p[u] + e) = (uint16_t)(o[e >> 2] >> (8 * (e & 2)));
    }
}

// Elements of a tile, and the number of tiles of all tensors.
pgq_status plan(const int64_t* numel, int32_t n, int64_t* tile, int64_t* total)
{
    if (n < 0) return PGQ_ERR_SHAPE;
    if (n > 0 && !numel) return PGQ_ERR_NULL;
    int64_t filled = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (numel[i] < 0 || numel[i] > kMaxNumel) return PGQ_ERR_SHAPE;
        filled += numel[i] > 0;
    }
    for (*tile = kTile;; *tile *= 2) {
        *total = 0;
        for (int32_t i = 0; i < n; ++i) *total += (numel[i] + *tile - 1) / *tile;
        if (*total <= kTilesWanted + filled) break;
    }
    if (!grid_fits(*total, kThreads)) return PGQ_ERR_SHAPE;
    return PGQ_OK;
}
size_t workspace_size(int64_t total) { return kCountersBytes + ((size_t)std::max<int64_t>(total, 1) * 8 + 63) / 64 * 64; }

size_t size_of(int32_t dtype) { return dtype == PGQ_F32 ? 4 : 2; }

pgq_status check(const void* const* grad, const int64_t* numel, const int32_t* dtype, int32_t n, float max_norm, const float* result,
                 const void* workspace, size_t workspace_bytes, int64_t* tile, int64_t* total)
{
    const pgq_status st = plan(numel, n, tile, total);
    if (st != PGQ_OK) return st;
    if (!result || (n > 0 && (!grad || !dtype))) return PGQ_ERR_NULL;
    if (!(max_norm >= 0.0f)) return PGQ_ERR_PARAM;
    if (!is_aligned(result, 4)) return PGQ_ERR_ALIGN;
    for (int32_t i = 0; i < n; ++i) {
        if (dtype[i] != PGQ_F32 && dtype[i] != PGQ_BF16 && dtype[i] != PGQ_F16) return PGQ_ERR_DTYPE;
        if (numel[i] == 0) continue;
        if (!grad[i]) return PGQ_ERR_NULL;
        if (!is_aligned(grad[i], size_of(dtype[i]))) return PGQ_ERR_ALIGN;
    }
    if (!workspace || workspace_bytes < workspace_size(*total)) return PGQ_ERR_WORKSPACE;
    return is_aligned(workspace, 64) ? PGQ_OK : PGQ_ERR_ALIGN;
}

// One launch of fn for every kArgTensors tensors that hold anything; at least one where `always`.
pgq_status run(const void* fn, Launches& l, NormArgs a, const void* const* grad, const int64_t* numel, const int32_t* dtype, int32_t n,
               bool always)
{
    int32_t i = 0;
    uint32_t done = 0;
    do {
        Tensors t;
        memset(&t, 0, sizeof(t));
        memset(t.end, 0xFF, sizeof(t.end));
        uint32_t grid = 0;
        int k = 0;
        for (; k < kArgTensors && i < n; ++i) {
            if (numel[i] == 0) continue;
            t.p[k] = grad[i];
            t.numel[k] = numel[i];
            t.dtype[k] = (uint8_t)dtype[i];
            grid += (uint32_t)((numel[i] + a.tile - 1) / a.tile);
            t.end[k++] = grid;
        }
        while (i < n && numel[i] == 0) ++i;
        a.first = done;
        a.last = i == n;
        done += grid;
        if (grid == 0 && !always) break;
        void* args[] = {&a, &t};
        l.go(fn, std::max(grid, 1u), kThreads, args);
    } while (i < n);
    return l.done();
}

int launches_of(const int64_t* numel, int32_t n)
{
    int64_t filled = 0;
    for (int32_t i = 0; i < n; ++i) filled += numel[i] > 0;
    return (int)((filled + kArgTensors - 1) / kArgTensors);
}

// 16-byte pieces of all tensors (more than kSmallMost: some number past it)
int64_t pieces_of(const int64_t* numel, const int32_t* dtype, int32_t n)
{
    int64_t pieces = 0;
    for (int32_t i = 0; i < n && pieces <= kSmallMost; ++i) pieces += (numel[i] * (int64_t)size_of(dtype[i]) + 15) / 16;
    return pieces;
}
pgq_status run_small(Launches& l, NormArgs a, void* const* grad, const int64_t* numel, const int32_t* dtype, int32_t n)
{
    Tensors t;
    memset(&t, 0, sizeof(t));
    memset(t.end, 0xFF, sizeof(t.end));
    uint32_t end = 0;
    int k = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (numel[i] == 0) continue;
        t.p[k] = grad[i];
        t.numel[k] = numel[i];
        t.dtype[k] = (uint8_t)dtype[i];
        end += (uint32_t)((numel[i] * (int64_t)size_of(dtype[i]) + 15) / 16);
        t.end[k++] = end;
    }
    void* args[] = {&a, &t};
    l.go(reinterpret_cast<const void*>(&pgq_grad_clip_small_kernel), 1, kSmallThreads, args);
    return l.done();
}

NormArgs args_of(float scale, const float* scale_dev, float max_norm, float* result, void* workspace, uint32_t* status, int64_t tile, int64_t total)
{
    NormArgs a;
    memset(&a, 0, sizeof(a));
    a.counters = static_cast<uint8_t*>(workspace);
    a.part = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + kCountersBytes);
    a.result = result;
    a.status = status;
    a.scale_dev = scale_dev;
    a.scale = scale;
    a.max_norm = max_norm;
    a.tile = tile;
    a.total = (uint32_t)std::max<int64_t>(total, 1);
    return a;
}

}  // namespace
}  // namespace pgq

using namespace pgq;

extern "C" {

pgq_status pgq_grad_norm_workspace(const int64_t* numel, int32_t n, size_t* workspace_bytes)
{
    if (!workspace_bytes) return PGQ_ERR_NULL;
    int64_t tile, total;
    const pgq_status st = plan(numel, n, &tile, &total);
    if (st != PGQ_OK) return st;
    *workspace_bytes = workspace_size(total);
    return PGQ_OK;
}

pgq_status pgq_grad_norm(const void* const* grad, const int64_t* numel, const int32_t* dtype, int32_t n, float grad_scale,
                         const float* grad_scale_dev, float max_norm, float* result, void* workspace, size_t workspace_bytes,
                         uint32_t* dev_status, void* stream)
{
    int64_t tile, total;
    const pgq_status st = check(grad, numel, dtype, n, max_norm, result, workspace, workspace_bytes, &tile, &total);
    if (st != PGQ_OK) return st;
    if (!grad_scale_dev && !(grad_scale - grad_scale == 0.0f)) return PGQ_ERR_PARAM;
    if (grad_scale_dev && !is_aligned(grad_scale_dev, 4)) return PGQ_ERR_ALIGN;
    Launches l(std::max(launches_of(numel, n), 1), stream);
    return run(reinterpret_cast<const void*>(&pgq_grad_norm_kernel), l,
               args_of(grad_scale, grad_scale_dev, max_norm, result, workspace, dev_status, tile, total), grad, numel, dtype, n, true);
}

pgq_status pgq_grad_clip(void* const* grad, const int64_t* numel, const int32_t* dtype, int32_t n, float max_norm, float* result,
                         void* workspace, size_t workspace_bytes, uint32_t* dev_status, void* stream)
{
    int64_t tile, total;
    pgq_status st = check(grad, numel, dtype, n, max_norm, result, workspace, workspace_bytes, &tile, &total);
    if (st != PGQ_OK) return st;
    // a tensor that two entries share would be multiplied twice, or by two workgroups at once
    typedef std::pair<uintptr_t, uintptr_t> Range;
    Range few[256];
    Range* ranges = n <= 256 ? few : new (std::nothrow) Range[(size_t)n];
    if (!ranges) return (pgq_status)note_hip_error(hipErrorOutOfMemory);
    int32_t k = 0;
    for (int32_t i = 0; i < n; ++i)
        if (numel[i] > 0) ranges[k++] = Range((uintptr_t)grad[i], (uintptr_t)grad[i] + (uintptr_t)numel[i] * size_of(dtype[i]));
    std::sort(ranges, ranges + k);
    for (int32_t i = 1; i < k && st == PGQ_OK; ++i)
        if (ranges[i].first < ranges[i - 1].second) st = PGQ_ERR_PARAM;
    if (ranges != few) delete[] ranges;
    if (st != PGQ_OK) return st;
    const int per = launches_of(numel, n);
    NormArgs a = args_of(1.0f, nullptr, max_norm, result, workspace, dev_status, tile, total);
    const int64_t pieces = per <= 1 ? pieces_of(numel, dtype, n) : kSmallMost + 1;
    if (pieces <= kSmallMost) {
        a.total = (uint32_t)pieces;
        Launches l(1, stream);
        return run_small(l, a, grad, numel, dtype, n);
    }
    Launches l(std::max(per, 1) + per, stream);
    st = run(reinterpret_cast<const void*>(&pgq_grad_norm_kernel), l, a, grad, numel, dtype, n, true);
    if (st != PGQ_OK) return st;
    return run(reinterpret_cast<const void*>(&pgq_grad_scale_kernel), l, a, grad, numel, dtype, n, false);
}

}  // extern "C"
