// pgq_train.h -- host helpers shared by the entry points outside pgq_api.hip (the linear layers, the
// optimizer step, the gradient norm, 4-bit weights).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pgq_desc.h"
#include "../../include/pgq.h"

namespace pgq {

// PGQ_ERR_HIP, after keeping e as the calling thread's latest HIP error (pgq_last_error).
int32_t note_hip_error(hipError_t e);
// 64-bit hash of n bytes, chained through h (descriptor table checksums).
uint64_t hash_bytes(const void* data, size_t n, uint64_t h);

inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxSize = ((int64_t)1 << 31) - 1;

inline bool float_type(int32_t dt) { return dt == PGQ_F32 || dt == PGQ_BF16; }
inline size_t float_size(int32_t dt) { return dt == PGQ_F32 ? 4 : 2; }
inline bool act_ok(int32_t act, float slope)
{
    if (act == PGQ_ACT_NONE || act == PGQ_ACT_SILU) return true;
    return (act == PGQ_ACT_RELU || act == PGQ_ACT_RELU2) && slope - slope == 0.0f;
}

// The bytes of a matrix argument.  clash: two of them share a byte, or might: rows of different strides in
// one range of memory are not told apart.
struct Span {
    const void* at;
    int64_t rows, width, ld;             // width and row stride in bytes
};
inline bool clash(const Span& a, const Span& b)
{
    if (!a.at || !b.at || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const uintptr_t a0 = (uintptr_t)a.at, b0 = (uintptr_t)b.at;
    const uintptr_t a1 = a0 + (uintptr_t)(a.rows - 1) * (uintptr_t)a.ld + (uintptr_t)a.width;
    const uintptr_t b1 = b0 + (uintptr_t)(b.rows - 1) * (uintptr_t)b.ld + (uintptr_t)b.width;
    if (a1 <= b0 || b1 <= a0) return false;
    if (a.ld != b.ld) return true;
    const int64_t d = (int64_t)(b0 - a0) % a.ld, at = d < 0 ? d + a.ld : d;       // columns of one buffer
    return at < a.width || at + b.width > a.ld;
}
// one of the outputs (the first n_out spans) shares memory with another span
inline bool any_clash(const Span* s, int n_out, int n)
{
    for (int i = 0; i < n_out; ++i)
        for (int j = i + 1; j < n; ++j)
            if (clash(s[i], s[j])) return true;
    return false;
}

// The runtime's limits: 2^31 - 1 workgroups, 2^32 - 1 threads.  A call one of whose launches would pass them is
// refused before the first.
inline bool grid_fits(int64_t grid, int block) { return grid <= 0x7FFFFFFF && grid * block <= 0xFFFFFFFFll; }
// One launch of a linear grid; a refused one leaves no timing events for the thread's next call.
inline hipError_t launch_grid(const void* fn, int64_t grid, int block, void** args, void* stream)
{
    if (!grid_fits(grid, block)) {
        void *start, *stop;
        take_timing_events(&start, &stop);
        return hipErrorInvalidValue;
    }
    return launch_plain(fn, dim3((unsigned)grid), dim3((unsigned)block), args, stream);
}

// The launches of one call: the first takes a pending start event, the last the stop event.
struct Launches {
    void *start = nullptr, *stop = nullptr, *stream;
    int left;
    hipError_t e = hipSuccess;
    Launches(int n, void* s) : stream(s), left(n) { take_timing_events(&start, &stop); }
    bool next()
    {
        if (e != hipSuccess) return false;
        set_timing_events(start, --left == 0 ? stop : nullptr);
        start = nullptr;
        return true;
    }
    void go(const void* fn, int64_t grid, int block, void** args)
    {
        if (!next()) return;
        e = launch_grid(fn, grid, block, args, stream);
    }
    pgq_status done() const { return e == hipSuccess ? PGQ_OK : (pgq_status)note_hip_error(e); }
};

}  // namespace pgq
