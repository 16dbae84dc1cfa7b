// pgq_adamw.hip -- one AdamW step over many tensors (gfx950), states in binary32 or in 8 bits.
//
// A workgroup handles one tile: kTile consecutive elements of one tensor.  Lane l of a wavefront takes
// the four elements 4 l .. 4 l + 3 of each 256-element group, so fp32 streams move in 16-byte and codes in
// 4-byte accesses, and a block of 64 elements that shares a state scale is 16 neighbouring lanes: its
// maximum is four DPP steps inside a row of 16.  The arithmetic is the one pgq.h spells out, operation by
// operation (no contraction), so a step gives the same bits on every path and run.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <new>

#include "pgq_desc.h"
#include "pgq_train.h"
#include "../../include/pgq.h"

namespace pgq {
namespace {

#define GLB __attribute__((address_space(1)))

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kGroups = 4;                        // 4-element groups per lane in a tile
constexpr int kTile = kThreads * 4 * kGroups;     // elements
constexpr int kArgPtrs = 256;                     // pointers carried in the kernel arguments of a launch
constexpr uint64_t kAdamMagic = 0x5047514144414d31ull;

struct alignas(16) AdDesc {
    void* w;
    uint16_t* copy;
    void* m;
    void* v;
    uint8_t* m_scale;
    uint8_t* v_scale;
    int64_t numel;
    uint32_t first_tile;
    uint32_t id;                                  // place in the caller's list
    float lr_scale, weight_decay;
    uint8_t w_bf16, vec, pad0[2];                 // vec: weights, copy and states are aligned to 4-element accesses
    uint32_t pad1;
};

struct Ptrs {
    const void* p[kArgPtrs];
    uint8_t dtype[kArgPtrs];                      // step: the gradients' types
};

struct AdArgs {
    const TableHeader* hdr;
    const AdDesc* table;
    const uint32_t* tile_desc;
    uint64_t checksum;
    uint32_t* status;
    const pgq_adamw_hyper* h_dev;
    pgq_adamw_hyper h;
    uint32_t first_tile;                          // tiles before this launch's
    uint32_t first_desc;                          // tensors before its pointers
};

// Constants of a step have ib1, ib2 >= 1; zeros (never written) would make every weight 0 / 0 and clear the states.
__host__ __device__ inline bool is_step(const pgq_adamw_hyper& h) { return h.ib1 > 0.0f && h.ib2 > 0.0f; }

__device__ __forceinline__ float bf16_to_f32(uint16_t h) { return __builtin_bit_cast(float, (uint32_t)h << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

__device__ __forceinline__ uint32_t mix(uint32_t x)
{
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x ^ (x >> 16);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xF, 0xF, false);
}
// maximum over the 16 lanes of a row, in every lane of it
__device__ __forceinline__ uint32_t max16(uint32_t x)
{
    x = max(x, dpp<0xB1>(x));                     // quad_perm: lane ^ 1
    x = max(x, dpp<0x4E>(x));                     // quad_perm: lane ^ 2
    x = max(x, dpp<0x141>(x));                    // row_half_mirror
    return max(x, dpp<0x140>(x));                 // row_mirror
}

// |value| bits of a magnitude code with MANT mantissa bits under scale byte b
template <int MANT>
__device__ __forceinline__ float decode(uint32_t c, uint32_t b)
{
    return ldexpf(__builtin_bit_cast(float, c << (23 - MANT)), (int)b - 7);
}
// magnitude code of |x| (bits ax), stochastic with 16 random bits u
template <int MANT>
__device__ __forceinline__ uint32_t encode(uint32_t ax, uint32_t b, uint32_t u)
{
    const float y = ldexpf(__builtin_bit_cast(float, ax), 7 - (int)b);
    return (__builtin_bit_cast(uint32_t, y) + (u << (7 - MANT))) >> (23 - MANT);
}
__device__ __forceinline__ uint32_t scale_byte(uint32_t block_max_bits)
{
    const int e = (int)(block_max_bits >> 23) - 7;
    return (uint32_t)max(e, 0);
}

// kinds of stream a launch holds: fp32 weights with fp32 or bf16 gradients in every tensor, or any mix
enum Streams { S_F32 = 0, S_BF16G = 1, S_ANY = 2 };

// Four elements of a lane as they lie in memory: fp32 streams in four words, 16-bit ones in two, codes in one.
struct Raw {
    u32x4 w, g, m, v;
    uint32_t mb, rb;                              // 8 bits: scale bytes
};

__device__ __forceinline__ u32x4 load4(const void* p, int64_t i, bool wide)
{
    if (wide) return __builtin_nontemporal_load((const GLB u32x4*)((const uint32_t*)p + i));
    const u32x2 q = __builtin_nontemporal_load((const GLB u32x2*)((const uint16_t*)p + i));
    return u32x4{q[0], q[1], 0, 0};
}
// the same element by element, zeros past `live`
__device__ __forceinline__ u32x4 load4_edge(const void* p, int64_t i, bool wide, int live)
{
    u32x4 r = {};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < live) {
            if (wide) r[e] = ((const uint32_t*)p)[i + e];
            else r[e / 2] |= (uint32_t)((const uint16_t*)p)[i + e] << (16 * (e % 2));
        }
    return r;
}
__device__ __forceinline__ uint32_t load_codes_edge(const void* p, int64_t i, int live)
{
    uint32_t r = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < live) r |= (uint32_t)((const uint8_t*)p)[i + e] << (8 * e);
    return r;
}
// element e of four loaded values of a type
__device__ __forceinline__ float value(const u32x4& r, int e, int32_t dtype)
{
    if (dtype == PGQ_F32) {
        const uint32_t x = r[e];
        return __builtin_bit_cast(float, x);
    }
    const uint16_t h = (uint16_t)(r[e / 2] >> (16 * (e % 2)));
    return dtype == PGQ_BF16 ? bf16_to_f32(h) : (float)__builtin_bit_cast(_Float16, h);
}
__device__ __forceinline__ u32x2 pack_bf16(const float* w)
{
    return u32x2{(uint32_t)f32_to_bf16(w[0]) | ((uint32_t)f32_to_bf16(w[1]) << 16), (uint32_t)f32_to_bf16(w[2]) | ((uint32_t)f32_to_bf16(w[3]) << 16)};
}

template <int BITS, int S>
__global__ void __launch_bounds__(kThreads) pgq_adamw_kernel(AdArgs a, Ptrs grads)
{
    if (a.hdr->magic != kAdamMagic || a.hdr->checksum != a.checksum) {
        if (blockIdx.x == 0 && threadIdx.x == 0 && a.status) atomicOr(a.status, PGQ_DEV_STALE_TABLE);
        return;
    }
    const uint32_t tile = a.first_tile + blockIdx.x;
    const uint32_t di = a.tile_desc[tile];
    const AdDesc d = a.table[di];
    const void* grad = grads.p[di - a.first_desc];
    const pgq_adamw_hyper h = a.h_dev ? *a.h_dev : a.h;
    if (!is_step(h)) {
        if (blockIdx.x == 0 && threadIdx.x == 0 && a.status) atomicOr(a.status, PGQ_DEV_NO_HYPER);
        return;
    }
    const float lr = d.lr_scale * h.lr;
    const float step = lr * h.ib1;
    const float keep = 1.0f - lr * d.weight_decay;
    const uint32_t tseed = mix(0x9E3779B1u * (d.id + 1u) + h.seed);
    const int32_t wt = S == S_ANY && d.w_bf16 ? PGQ_BF16 : PGQ_F32;
    const int32_t gt = S == S_F32 ? PGQ_F32 : S == S_BF16G ? PGQ_BF16 : (int32_t)grads.dtype[di - a.first_desc];
    const int64_t base = (int64_t)(tile - d.first_tile) * kTile;
    const int lane4 = ((int)threadIdx.x & 63) * 4, wave = (int)threadIdx.x >> 6;
    const int64_t first = base + wave * (kGroups * 256) + lane4;
    const bool vec = d.vec && base + kTile <= d.numel && (S != S_ANY || ((uintptr_t)grad & (gt == PGQ_F32 ? 15 : 7)) == 0);
    bool bad = false;

    // one group of 256 elements: from the loaded values to the stores
    auto update = [&](int64_t i0, const Raw& q, int live, bool whole) __attribute__((always_inline)) {
        float w[4], m[4], v[4], r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = value(q.w, e, wt);
            const float g = value(q.g, e, gt);
            if (BITS == 8) {
                const uint32_t c = (q.m[0] >> (8 * e)) & 0xFFu;
                const float x = decode<3>(c & 0x7Fu, q.mb);
                m[e] = (c & 0x80u) ? -x : x;
                r[e] = decode<4>((q.v[0] >> (8 * e)) & 0xFFu, q.rb);
                v[e] = r[e] * r[e];
            } else {
                m[e] = value(q.m, e, PGQ_F32);
                v[e] = value(q.v, e, PGQ_F32);
            }
            const float gs = h.grad_scale * g;
            const float m1 = m[e] * h.beta1 + gs * h.c1;
            const float v1 = v[e] * h.beta2 + (gs * gs) * h.c2;
            const float root = sqrtf(v1);
            const float w1 = w[e] * keep - (m1 / (root * h.ib2 + h.eps)) * step;
            const bool ok = fabsf(m1) < INFINITY && v1 < INFINITY;
            bad |= !ok && e < live;
            w[e] = ok ? w1 : w[e];
            m[e] = ok ? m1 : m[e];
            if (BITS == 8) r[e] = ok ? root : r[e];
            else v[e] = ok ? v1 : v[e];
        }
        if (whole) {
            if (wt == PGQ_BF16) {
                *(GLB u32x2*)((uint16_t*)d.w + i0) = pack_bf16(w);
            } else {
                __builtin_nontemporal_store(f32x4{w[0], w[1], w[2], w[3]}, (GLB f32x4*)((float*)d.w + i0));
                if (d.copy) *(GLB u32x2*)(d.copy + i0) = pack_bf16(w);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < live) {
                    if (wt == PGQ_BF16) ((uint16_t*)d.w)[i0 + e] = f32_to_bf16(w[e]);
                    else ((float*)d.w)[i0 + e] = w[e];
                    if (d.copy) d.copy[i0 + e] = f32_to_bf16(w[e]);
                }
        }
        if (BITS == 8) {
            uint32_t tm = 0, tr = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < live) {
                    tm = max(tm, __builtin_bit_cast(uint32_t, m[e]) & 0x7FFFFFFFu);
                    tr = max(tr, __builtin_bit_cast(uint32_t, r[e]));
                }
            const uint32_t bm = scale_byte(max16(tm)), br = scale_byte(max16(tr));
            uint32_t mc = 0, rc = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t u = mix(tseed ^ (uint32_t)(i0 + e));
                const uint32_t mbits = __builtin_bit_cast(uint32_t, m[e]);
                mc |= (encode<3>(mbits & 0x7FFFFFFFu, bm, u >> 16) | (mbits >> 31 << 7)) << (8 * e);
                uint32_t c = encode<4>(__builtin_bit_cast(uint32_t, r[e]), br, u & 0xFFFFu);
                c = r[e] > 0.0f && c == 0 ? 1u : c;
                rc |= c << (8 * e);
            }
            if (whole) {
                *(GLB uint32_t*)((uint8_t*)d.m + i0) = mc;
                *(GLB uint32_t*)((uint8_t*)d.v + i0) = rc;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < live) {
                        ((uint8_t*)d.m)[i0 + e] = (uint8_t)(mc >> (8 * e));
                        ((uint8_t*)d.v)[i0 + e] = (uint8_t)(rc >> (8 * e));
                    }
            }
            if ((lane4 & 63) == 0 && live > 0) {
                d.m_scale[i0 >> 6] = (uint8_t)bm;
                d.v_scale[i0 >> 6] = (uint8_t)br;
            }
        } else if (whole) {
            __builtin_nontemporal_store(f32x4{m[0], m[1], m[2], m[3]}, (GLB f32x4*)((float*)d.m + i0));
            __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, (GLB f32x4*)((float*)d.v + i0));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < live) { ((float*)d.m)[i0 + e] = m[e]; ((float*)d.v)[i0 + e] = v[e]; }
        }
    };

    if (vec) {
        // every load of the tile first, so that a lane has kGroups groups of all streams in flight
        Raw q[kGroups];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int64_t i0 = first + k * 256;
            q[k].w = load4(d.w, i0, wt == PGQ_F32);
            q[k].g = load4(grad, i0, gt == PGQ_F32);
            if (BITS == 8) {
                q[k].m[0] = __builtin_nontemporal_load((const GLB uint32_t*)((const uint8_t*)d.m + i0));
                q[k].v[0] = __builtin_nontemporal_load((const GLB uint32_t*)((const uint8_t*)d.v + i0));
                q[k].mb = ((const GLB uint8_t*)d.m_scale)[i0 >> 6];
                q[k].rb = ((const GLB uint8_t*)d.v_scale)[i0 >> 6];
            } else {
                q[k].m = load4(d.m, i0, true);
                q[k].v = load4(d.v, i0, true);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) update(first + k * 256, q[k], 4, true);
    } else {
#pragma unroll 1
        for (int k = 0; k < kGroups; ++k) {
            const int64_t i0 = first + k * 256;
            const int live = (int)min((int64_t)4, max((int64_t)0, d.numel - i0));
            Raw q;
            q.w = load4_edge(d.w, i0, wt == PGQ_F32, live);
            q.g = load4_edge(grad, i0, gt == PGQ_F32, live);
            q.mb = q.rb = 0;
            if (BITS == 8) {
                q.m[0] = load_codes_edge(d.m, i0, live);
                q.v[0] = load_codes_edge(d.v, i0, live);
                if (live > 0) {
                    q.mb = d.m_scale[i0 >> 6];
                    q.rb = d.v_scale[i0 >> 6];
                }
            } else {
                q.m = load4_edge(d.m, i0, true, live);
                q.v = load4_edge(d.v, i0, true, live);
            }
            update(i0, q, live, false);
        }
    }
    if (a.status && __ballot(bad) != 0 && ((int)threadIdx.x & 63) == 0) atomicOr(a.status, PGQ_DEV_NONFINITE);
}

// the values of 8-bit states as bf16: pointers p[2 i] = m_out, p[2 i + 1] = r_out of tensor i
__global__ void __launch_bounds__(kThreads) pgq_adamw_decode_kernel(AdArgs a, Ptrs outs)
{
    if (a.hdr->magic != kAdamMagic || a.hdr->checksum != a.checksum) {
        if (blockIdx.x == 0 && threadIdx.x == 0 && a.status) atomicOr(a.status, PGQ_DEV_STALE_TABLE);
        return;
    }
    const uint32_t tile = a.first_tile + blockIdx.x;
    const uint32_t di = a.tile_desc[tile];
    const AdDesc d = a.table[di];
    uint16_t* mo = (uint16_t*)outs.p[2 * (di - a.first_desc)];
    uint16_t* ro = (uint16_t*)outs.p[2 * (di - a.first_desc) + 1];
    const int64_t base = (int64_t)(tile - d.first_tile) * kTile;
    const bool vec = base + kTile <= d.numel && (((uintptr_t)mo | (uintptr_t)ro) & 7) == 0 && (((uintptr_t)d.m | (uintptr_t)d.v) & 3) == 0;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        const int64_t i0 = base + ((int)threadIdx.x >> 6) * (kGroups * 256) + k * 256 + ((int)threadIdx.x & 63) * 4;
        const int live = (int)min((int64_t)4, max((int64_t)0, d.numel - i0));
        if (live == 0) continue;
        const uint32_t mb = d.m_scale[i0 >> 6], rb = d.v_scale[i0 >> 6];
        uint32_t mc = 0, rc = 0;
        if (vec) {
            mc = *(const GLB uint32_t*)((const uint8_t*)d.m + i0);
            rc = *(const GLB uint32_t*)((const uint8_t*)d.v + i0);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < live) {
                    mc |= (uint32_t)((const uint8_t*)d.m)[i0 + e] << (8 * e);
                    rc |= (uint32_t)((const uint8_t*)d.v)[i0 + e] << (8 * e);
                }
        }
        u16x4 qm, qr;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t c = (mc >> (8 * e)) & 0xFFu;
            const float x = decode<3>(c & 0x7Fu, mb);
            qm[e] = f32_to_bf16((c & 0x80u) ? -x : x);
            qr[e] = f32_to_bf16(decode<4>((rc >> (8 * e)) & 0xFFu, rb));
        }
        if (vec) {
            __builtin_nontemporal_store(qm, (GLB u16x4*)(mo + i0));
            __builtin_nontemporal_store(qr, (GLB u16x4*)(ro + i0));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < live) { mo[i0 + e] = qm[e]; ro[i0 + e] = qr[e]; }
        }
    }
}

constexpr int64_t kMaxNumel = (int64_t)1 << 40;

pgq_status check_tensors(const pgq_adamw_tensor* t, int32_t n, int32_t bits, uint64_t* tiles)
{
    if (n < 0) return PGQ_ERR_SHAPE;
    if (bits != 32 && bits != 8) return PGQ_ERR_PARAM;
    *tiles = 0;
    if (n > 0 && !t) return PGQ_ERR_NULL;
    for (int32_t i = 0; i < n; ++i) {
        const pgq_adamw_tensor& x = t[i];
        if (x.numel < 0 || x.numel > kMaxNumel) return PGQ_ERR_SHAPE;
        if (x.w_dtype != PGQ_F32 && x.w_dtype != PGQ_BF16) return PGQ_ERR_DTYPE;
        if (x.g_dtype != PGQ_F32 && x.g_dtype != PGQ_BF16 && x.g_dtype != PGQ_F16) return PGQ_ERR_DTYPE;
        if (x.copy && x.w_dtype != PGQ_F32) return PGQ_ERR_DTYPE;
        if (!(x.lr_scale - x.lr_scale == 0.0f) || !(x.weight_decay - x.weight_decay == 0.0f)) return PGQ_ERR_PARAM;
        *tiles += (uint64_t)((x.numel + kTile - 1) / kTile);
        if (*tiles * kThreads > 0xFFFFFFFFull) return PGQ_ERR_SHAPE;       // a launch's limit: 2^32 - 1 threads
        if (x.numel == 0) continue;
        if (!x.w || !x.m || !x.v || (bits == 8 && (!x.m_scale || !x.v_scale))) return PGQ_ERR_NULL;
        if (!is_aligned(x.w, x.w_dtype == PGQ_F32 ? 4 : 2) || (x.copy && !is_aligned(x.copy, 2)) ||
            (bits == 32 && (!is_aligned(x.m, 4) || !is_aligned(x.v, 4))))
            return PGQ_ERR_ALIGN;
    }
    return PGQ_OK;
}

size_t up64(size_t x) { return (x + 63) / 64 * 64; }
size_t desc_off() { return up64(sizeof(TableHeader)); }
size_t tdesc_off(int32_t n) { return desc_off() + up64((size_t)n * sizeof(AdDesc)); }
size_t table_size(int32_t n, uint64_t tiles) { return tdesc_off(n) + up64(tiles * sizeof(uint32_t)); }

AdDesc desc_of(const pgq_adamw_tensor& x, int32_t bits, uint32_t first_tile, uint32_t id)
{
    AdDesc d;
    memset(&d, 0, sizeof(d));
    d.w = x.w;
    d.copy = x.copy;
    d.m = x.m;
    d.v = x.v;
    d.m_scale = bits == 8 ? x.m_scale : nullptr;
    d.v_scale = bits == 8 ? x.v_scale : nullptr;
    d.numel = x.numel;
    d.first_tile = first_tile;
    d.id = id;
    d.lr_scale = x.lr_scale;
    d.weight_decay = x.weight_decay;
    d.w_bf16 = x.w_dtype == PGQ_BF16;
    const size_t s = bits == 8 ? 4 : 16;
    d.vec = is_aligned(x.w, x.w_dtype == PGQ_F32 ? 16 : 8) && (!x.copy || is_aligned(x.copy, 8)) && is_aligned(x.m, s) &&
            is_aligned(x.v, s);
    return d;
}

// The checksum of the table these tensors make (and, when buf is given, the table itself).
uint64_t build_table(const pgq_adamw_tensor* t, int32_t n, int32_t bits, uint64_t tiles, uint8_t* buf)
{
    uint64_t sum = 0x452821E638D01377ull ^ (uint64_t)bits;
    uint32_t first = 0;
    for (int32_t i = 0; i < n; ++i) {
        const AdDesc d = desc_of(t[i], bits, first, (uint32_t)i);
        sum = hash_bytes(&d, sizeof(d), sum);
        const uint32_t next = first + (uint32_t)((t[i].numel + kTile - 1) / kTile);
        if (buf) {
            memcpy(buf + desc_off() + (size_t)i * sizeof(AdDesc), &d, sizeof(d));
            uint32_t* td = reinterpret_cast<uint32_t*>(buf + tdesc_off(n));
            for (uint32_t k = first; k < next; ++k) td[k] = (uint32_t)i;
        }
        first = next;
    }
    if (buf) {
        TableHeader* h = reinterpret_cast<TableHeader*>(buf);
        h->magic = kAdamMagic;
        h->checksum = sum;
        h->n_desc = (uint32_t)n;
        h->n_tiles = (uint32_t)tiles;
    }
    return sum;
}

// Table upload (unless resident) and launches over runs of tensors whose pointers fit the kernel
// arguments: per pointers a tensor, fn the kernel.
pgq_status run(const pgq_adamw_tensor* t, int32_t n, int32_t bits, uint64_t tiles, const void* fn, int per,
               const void* const* p0, const void* const* p1, const pgq_adamw_hyper* h, const pgq_adamw_hyper* h_dev,
               void* workspace, size_t workspace_bytes, uint32_t flags, uint32_t* dev_status, void* stream)
{
    if (!workspace || workspace_bytes < table_size(n, tiles)) return PGQ_ERR_WORKSPACE;
    if (!is_aligned(workspace, 64)) return PGQ_ERR_ALIGN;
    if (h && !is_step(*h)) return PGQ_ERR_PARAM;
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint64_t sum;
    if (flags & PGQ_TABLE_RESIDENT) {
        sum = build_table(t, n, bits, tiles, nullptr);
    } else {
        hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
        hipError_t e = hipStreamIsCapturing(s, &cap);
        if (e != hipSuccess) return (pgq_status)note_hip_error(e);
        if (cap != hipStreamCaptureStatusNone) return PGQ_ERR_PARAM;
        const size_t bytes = table_size(n, tiles);
        uint8_t* buf = new (std::nothrow) uint8_t[bytes];
        if (!buf) return (pgq_status)note_hip_error(hipErrorOutOfMemory);
        memset(buf, 0, bytes);
        sum = build_table(t, n, bits, tiles, buf);
        // a pageable source is staged by the runtime before this call returns
        e = hipMemcpyAsync(workspace, buf, bytes, hipMemcpyHostToDevice, s);
        delete[] buf;
        if (e != hipSuccess) return (pgq_status)note_hip_error(e);
    }
    const uint8_t* base = static_cast<const uint8_t*>(workspace);
    AdArgs a;
    memset(&a, 0, sizeof(a));
    a.hdr = reinterpret_cast<const TableHeader*>(base);
    a.table = reinterpret_cast<const AdDesc*>(base + desc_off());
    a.tile_desc = reinterpret_cast<const uint32_t*>(base + tdesc_off(n));
    a.checksum = sum;
    a.status = dev_status;
    a.h_dev = h_dev;
    if (h) a.h = *h;
    void *ev_start = nullptr, *ev_stop = nullptr;
    take_timing_events(&ev_start, &ev_stop);
    uint32_t first = 0;
    for (int32_t i = 0; i < n;) {
        Ptrs p;
        memset(&p, 0, sizeof(p));
        a.first_tile = first;
        a.first_desc = (uint32_t)i;
        int32_t k = 0;
        for (; k < kArgPtrs / per && i < n; ++k, ++i) {
            p.p[per * k] = p0[i];
            if (per == 2) p.p[2 * k + 1] = p1[i];
            else p.dtype[k] = (uint8_t)t[i].g_dtype;
            first += (uint32_t)((t[i].numel + kTile - 1) / kTile);
        }
        const uint32_t grid = first - a.first_tile;
        if (grid == 0) continue;
        set_timing_events(ev_start, first == tiles ? ev_stop : nullptr);
        ev_start = nullptr;
        void* args[] = {&a, &p};
        const hipError_t e = launch_plain(fn, dim3(grid), dim3(kThreads), args, stream);
        if (e != hipSuccess) return (pgq_status)note_hip_error(e);
    }
    return PGQ_OK;
}

template <int BITS>
const void* step_kernel(int s)
{
    return s == S_F32 ? reinterpret_cast<const void*>(&pgq_adamw_kernel<BITS, S_F32>)
           : s == S_BF16G ? reinterpret_cast<const void*>(&pgq_adamw_kernel<BITS, S_BF16G>)
                          : reinterpret_cast<const void*>(&pgq_adamw_kernel<BITS, S_ANY>);
}

}  // namespace
}  // namespace pgq

using namespace pgq;

extern "C" {

pgq_status pgq_adamw_hyper_at(double lr, double beta1, double beta2, double eps, int64_t step, float grad_scale,
                              uint32_t seed, pgq_adamw_hyper* out)
{
    if (!out) return PGQ_ERR_NULL;
    if (!(lr >= 0 && (float)lr < INFINITY) || !(eps >= 0 && (float)eps < INFINITY) || !(beta1 >= 0 && beta1 < 1) ||
        !(beta2 >= 0 && beta2 < 1) || step < 1)
        return PGQ_ERR_PARAM;
    memset(out, 0, sizeof(*out));
    out->lr = (float)lr;
    out->beta1 = (float)beta1;
    out->c1 = (float)(1 - beta1);
    out->beta2 = (float)beta2;
    out->c2 = (float)(1 - beta2);
    out->ib1 = (float)(1 / (1 - pow(beta1, (double)step)));
    out->ib2 = (float)(1 / sqrt(1 - pow(beta2, (double)step)));
    out->eps = (float)eps;
    out->grad_scale = grad_scale;
    out->seed = seed;
    return PGQ_OK;
}

pgq_status pgq_adamw_workspace(const pgq_adamw_tensor* t, int32_t n, size_t* workspace_bytes)
{
    if (!workspace_bytes) return PGQ_ERR_NULL;
    if (n < 0) return PGQ_ERR_SHAPE;
    if (n > 0 && !t) return PGQ_ERR_NULL;
    uint64_t tiles = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (t[i].numel < 0 || t[i].numel > kMaxNumel) return PGQ_ERR_SHAPE;
        tiles += (uint64_t)((t[i].numel + kTile - 1) / kTile);
        if (tiles * kThreads > 0xFFFFFFFFull) return PGQ_ERR_SHAPE;
    }
    *workspace_bytes = table_size(n, tiles);
    return PGQ_OK;
}

pgq_status pgq_adamw_step(const pgq_adamw_tensor* t, int32_t n, int32_t state_bits, const void* const* grad,
                          const pgq_adamw_hyper* h, const pgq_adamw_hyper* h_dev, void* workspace,
                          size_t workspace_bytes, uint32_t flags, uint32_t* dev_status, void* stream)
{
    uint64_t tiles = 0;
    const pgq_status st = check_tensors(t, n, state_bits, &tiles);
    if (st != PGQ_OK) return st;
    if (!h && !h_dev) return PGQ_ERR_NULL;
    if (n > 0 && !grad) return PGQ_ERR_NULL;
    if (h_dev && !is_aligned(h_dev, 4)) return PGQ_ERR_ALIGN;
    bool bf16_w = false, f32_g = true, bf16_g = true, grads_vec = true;
    for (int32_t i = 0; i < n; ++i) {
        if (t[i].numel == 0) continue;
        const size_t es = t[i].g_dtype == PGQ_F32 ? 4 : 2;
        if (!grad[i]) return PGQ_ERR_NULL;
        if (!is_aligned(grad[i], es)) return PGQ_ERR_ALIGN;
        grads_vec = grads_vec && is_aligned(grad[i], 4 * es);
        bf16_w = bf16_w || t[i].w_dtype == PGQ_BF16;
        f32_g = f32_g && t[i].g_dtype == PGQ_F32;
        bf16_g = bf16_g && t[i].g_dtype == PGQ_BF16;
    }
    if (tiles == 0) return PGQ_OK;
    // (gradients that are not aligned to four elements are handled by the element path of the mixed kernel)
    const int s = bf16_w || !grads_vec ? S_ANY : f32_g ? S_F32 : bf16_g ? S_BF16G : S_ANY;
    return run(t, n, state_bits, tiles, state_bits == 8 ? step_kernel<8>(s) : step_kernel<32>(s), 1, grad, nullptr,
               h_dev ? nullptr : h, h_dev, workspace, workspace_bytes, flags, dev_status, stream);
}

pgq_status pgq_adamw_decode(const pgq_adamw_tensor* t, int32_t n, uint16_t* const* m_out, uint16_t* const* r_out,
                            void* workspace, size_t workspace_bytes, uint32_t flags, uint32_t* dev_status, void* stream)
{
    uint64_t tiles = 0;
    const pgq_status st = check_tensors(t, n, 8, &tiles);
    if (st != PGQ_OK) return st;
    if (n > 0 && (!m_out || !r_out)) return PGQ_ERR_NULL;
    for (int32_t i = 0; i < n; ++i) {
        if (t[i].numel == 0) continue;
        if (!m_out[i] || !r_out[i]) return PGQ_ERR_NULL;
        if (!is_aligned(m_out[i], 2) || !is_aligned(r_out[i], 2)) return PGQ_ERR_ALIGN;
    }
    if (tiles == 0) return PGQ_OK;
    return run(t, n, 8, tiles, reinterpret_cast<const void*>(&pgq_adamw_decode_kernel), 2,
               reinterpret_cast<const void* const*>(m_out), reinterpret_cast<const void* const*>(r_out), nullptr, nullptr,
               workspace, workspace_bytes, flags, dev_status, stream);
}

}  // extern "C"
