// pgq_linear4.hip -- the linear layer over 4-bit weights with group scales, for few tokens (gfx950):
// Y = act(X W^T + b) + R, W[n][k] = code[n][k] * s[n][k / group].
//
// The codes are the traffic: N K / 2 bytes, each read once.  Codes are whole numbers, which bf16 holds, and their products
// with bf16 tokens are exact in fp32: x * code is summed over a group and one multiply-add per sum brings in the group's
// scale, so no weight is ever rounded and a weight costs no multiplication of its own.  Three kernels:
//   stream   1 and 2 tokens: a wavefront along K, tokens in its registers, rows streaming by (8192 -> 28672, one token: 22 us,
//            5.5 TB/s)
//   rows     small layers: 16 R weight rows a workgroup, K spread over its wavefronts, sums joined through LDS
//   shared   the rest: 64 R rows a workgroup, the tokens of a block of K shared through LDS (8192 -> 28672, 16 tokens: 30 us)
// The last two multiply on the matrix cores, v_mfma_f32_16x16x32_bf16 with 16 tokens as A and 16 weight rows as B, so that a lane
// has the sums of one weight row and needs one scale.
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
constexpr int kBlockK = 256;                      // columns of a block: 128 bytes of a row's codes, a cache line
constexpr int kHalfK = 128;                       // of which an instruction's load takes half

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
// A load of 64 bytes of each of 16 rows costs a compute unit's load path a quarter where four neighbouring lanes take a row (row l / 4,
// piece l % 4 of it); the matrix instructions want row l % 16, piece l / 16.  16 bytes a lane on their way from one to the other.
__device__ __forceinline__ u32x4 from_quads(u32x4 v, int lane)
{
    const int from = 4 * (4 * (lane & 15) + (lane >> 4));
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v[e]);
    return v;
}

// 16 bytes at any address, past the caches: for whole rows in one go (8192 -> 28672 25.7 -> 22.2 us).  The tiles' loads, 64 bytes
// of a row each, lose by it: the other half of the line is gone when its turn comes (64 tokens 71 -> 82 us).
__device__ __forceinline__ u32x4 load16_once(const void* p)
{
    typedef u32x4 any_u32x4 __attribute__((aligned(1)));
    return __builtin_nontemporal_load((const __attribute__((address_space(1))) any_u32x4*)p);
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

// ---- rows ---------------------------------------------------------------------------------------------
// How the work is cut: K in `parts` pieces of `blocks` blocks, one for each of as many workgroups.
struct Cut {
    float* sums;                 // parts > 1: parts x M x N
    int64_t blocks;
    int32_t token_blocks, parts;
};

// T: tiles of 16 tokens, R: of 16 weight rows.  Lane l: token l % 16 of A, weight row l % 16 of B, columns by the quarter
// l / 16.  Lanes past N repeat the last row, whose sums they do not store.  Loads are by quads, and a word of codes of every piece is
// one instruction's (the order of groups of 32), so that a load of X serves one instruction too.
//
// What bounds it is the compute unit's load path: besides the codes every workgroup reads all of X (16 tokens by 4096: 131 KB beside
// 32 KB of codes for R = 1).  By quads 16 x 4096 x 4096 goes from 7.6 to 6.5 us, 32 x 4096 x 4096 from 11.1 to 8.8, 16 x 8192 x 8192
// with R = 1 from 21.6 to 15.8 (four tokens 5.7 -> 6.1: few of their lanes load at all).  R = 2 halves X (8192 -> 8192, 16 tokens:
// 14.2).  Scales come 16 bytes of a row at a time, not a few for each block (one token 8192 -> 28672 38 -> 33 us).
template <int T, int R, int G>
__global__ void __launch_bounds__(64 * kWaves4) pgq_linear4_rows_kernel(pgq_linear4_fwd f, Cut cut)
{
    __shared__ f32x4 sums[kWaves4][R * T][64];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int r = lane & 15, quad = lane >> 2, piece = lane & 3;
    const uint32_t tb = blockIdx.x % (uint32_t)cut.token_blocks, rest = blockIdx.x / (uint32_t)cut.token_blocks;
    const uint32_t part = rest % (uint32_t)cut.parts;
    const int64_t m0 = (int64_t)tb * kMost, n0 = (int64_t)(rest / (uint32_t)cut.parts) * (16 * R);
    const uint8_t* crow[R];
    const uint16_t *srow[R], *xrow[T];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        crow[j] = f.codes + min(n0 + 16 * j + quad, f.N - 1) * f.ldc + 16 * piece;
        srow[j] = f.scales + min(n0 + 16 * j + r, f.N - 1) * f.lds;
    }
#pragma unroll
    for (int t = 0; t < T; ++t) xrow[t] = f.x + min(m0 + 16 * t + quad, f.M - 1) * f.ldx + 8 * piece;
    f32x4 acc[R][T];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[j][t] = f32x4{};
    bool live[T];                                 // lanes past M load nothing of X: their rows of the products go nowhere
#pragma unroll
    for (int t = 0; t < T; ++t) live[t] = m0 + 16 * t + quad < f.M;
    constexpr int GH = kHalfK / G;                // groups of half a block
    constexpr int SB = 8 / (2 * GH);              // blocks whose scales are loaded together, 16 bytes of a row
    const int64_t scale_bytes = 2 * ((f.K + G - 1) / G);
    // products of half a block: sc holds the scales of its groups in its lowest halves
    auto multiply = [&](u32x4 c, const u32x4 (*x)[4], uint64_t sc, f32x4* a) __attribute__((always_inline)) {
        c = from_quads(c, lane);
        trade<32>(c);
#pragma unroll
        for (int g = 0; g < GH; ++g) {
            f32x4 p[T];
#pragma unroll
            for (int t = 0; t < T; ++t) p[t] = f32x4{};
#pragma unroll
            for (int d = g * (4 / GH); d < (g + 1) * (4 / GH); ++d) {
                const bf16x8 w = decode8(c[d]);
#pragma unroll
                for (int t = 0; t < T; ++t) p[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[t][d]), w, p[t], 0, 0, 0);
            }
            const float s = f16_to_f32((uint16_t)(sc >> (16 * g)));
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) a[t][e] = __builtin_fmaf(p[t][e], s, a[t][e]);
        }
    };
    // the lowest GH scales of `half` of a block whose scales are the lowest of s
    auto scales_of = [&](const u32x4& s, int half) __attribute__((always_inline)) -> uint64_t {
        if (GH == 1) return half ? s[0] >> 16 : s[0];
        if (GH == 2) return half ? s[1] : s[0];
        return half ? (uint64_t)s[3] << 32 | s[2] : (uint64_t)s[1] << 32 | s[0];
    };
    struct Codes { u32x4 c[R][2]; };
    auto load_codes = [&](int64_t b, Codes& h) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            h.c[j][0] = load16(crow[j] + kBlockK / 2 * b);
            h.c[j][1] = load16(crow[j] + kBlockK / 2 * b + kHalfK / 2);
        }
    };
    auto load_scales = [&](int64_t b, u32x4* s) __attribute__((always_inline)) {
        const int64_t at = 4 * GH * b;
        if (at + 16 <= scale_bytes) {
#pragma unroll
            for (int j = 0; j < R; ++j) s[j] = load16((const uint8_t*)srow[j] + at);
        } else {
#pragma unroll
            for (int j = 0; j < R; ++j) s[j] = load16_edge(srow[j], at, scale_bytes);
        }
    };
    // This wavefront's blocks: an equal run of its part's, so that the scales of a run are neighbours.  Codes of the next block
    // are in flight while one is multiplied; X of a block is loaded before them, since loads complete in order and waiting for X
    // must not be waiting for those.
    const int64_t whole = f.K / kBlockK, blocks = (f.K + kBlockK - 1) / kBlockK;
    const int64_t part_end = min(blocks, (int64_t)(part + 1) * cut.blocks);
    const int64_t run = (cut.blocks + kWaves4 - 1) / kWaves4;
    int64_t b = (int64_t)part * cut.blocks + wave * run;
    const int64_t end = min(part_end, b + run), mine = min(whole, end);
    if (b < mine) {
        Codes h, next;
        u32x4 s[R];
        load_scales(b, s);
        load_codes(b, h);
        int held = SB;                            // blocks whose scales are in s
        auto block = [&](bool more) __attribute__((always_inline)) {
            u32x4 x[2][T][4];
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int t = 0; t < T; ++t) {
#pragma unroll
                    for (int d = 0; d < 4; ++d) x[half][t][d] = u32x4{};
                    if (live[t]) {
#pragma unroll
                        for (int d = 0; d < 4; ++d) x[half][t][d] = load16(xrow[t] + kBlockK * b + kHalfK * half + 32 * d);
                    }
                }
            u32x4 sn[R];
            const bool refill = more && held == 1;
            if (refill) load_scales(b + 1, sn);
            __builtin_amdgcn_sched_barrier(0);
            if (more) load_codes(b + 1, next);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int t = 0; t < T; ++t)
#pragma unroll
                    for (int d = 0; d < 4; ++d) x[half][t][d] = from_quads(x[half][t][d], lane);
#pragma unroll
                for (int j = 0; j < R; ++j) multiply(h.c[j][half], x[half], scales_of(s[j], half), acc[j]);
            }
            if (!more) return;
            h = next;
            if (refill) {
#pragma unroll
                for (int j = 0; j < R; ++j) s[j] = sn[j];
                held = SB;
            } else {
#pragma unroll
                for (int j = 0; j < R; ++j) s[j] = GH == 1 ? u32x4{s[j][1], s[j][2], s[j][3], 0} : u32x4{s[j][2], s[j][3], 0, 0};
                --held;
            }
        };
#pragma unroll 1
        for (; b + 1 < mine; ++b) block(true);
        block(false);
        ++b;
    }
    if (b < end) {                                // the last block of all: nothing past K is read, X is 0 there
        const int64_t row = (f.K + 7) / 8 * 4;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            const int64_t k0 = kBlockK * whole + kHalfK * half;
            if (k0 >= f.K) break;
            u32x4 x[T][4];
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int d = 0; d < 4; ++d) x[t][d] = from_quads(load16_edge(xrow[t] - 8 * piece, 2 * (k0 + 32 * d + 8 * piece), 2 * f.K), lane);
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const u32x4 c = load16_edge(crow[j] - 16 * piece, k0 / 2 + 16 * piece, row);
                const u32x4 s = load16_edge(srow[j], 2 * (k0 / G), scale_bytes);
                multiply(c, x, (uint64_t)s[1] << 32 | s[0], acc[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int t = 0; t < T; ++t) sums[wave][j * T + t][lane] = acc[j][t];
    __syncthreads();
    // accumulator element e of lane l: token 4 (l / 16) + e, weight row l % 16
#pragma unroll 1
    for (int u = (int)threadIdx.x; u < R * T * 256; u += 64 * kWaves4) {
        const int l = u & 63, e = (u >> 6) & 3, i = u >> 8;
        const int64_t m = m0 + 16 * (i % T) + 4 * (l >> 4) + e, n = n0 + 16 * (i / T) + (l & 15);
        if (m >= f.M || n >= f.N) continue;
        float z = sums[0][i][l][e];
#pragma unroll
        for (int w = 1; w < kWaves4; ++w) z += sums[w][i][l][e];
        if (cut.parts > 1) cut.sums[((int64_t)part * f.M + m) * f.N + n] = z;
        else finish(f, m, n, z);
    }
}

// the parts' sums, in their order, through the epilogue
__global__ void __launch_bounds__(256) pgq_linear4_join_kernel(pgq_linear4_fwd f, Cut cut)
{
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, mn = f.M * f.N;
    if (at >= mn) return;
    float z = cut.sums[at];
#pragma unroll 4
    for (int i = 1; i < cut.parts; ++i) z += cut.sums[at + i * mn];
    finish(f, at / f.N, at % f.N, z);
}

// ---- shared ---------------------------------------------------------------------------------------------
// Four wavefronts of a workgroup take 16 R weight rows each and share the tokens of a block of 256 columns through LDS; the other
// four do the same for the second half of the part's blocks, and the sums of the two halves are added at the end.  One barrier a
// block; the next block's operands are loaded into registers meanwhile.
//
// What bounds it first is again how many cache lines a compute unit takes in (8192 -> 28672, 32 tokens, R = 2): tokens, codes and
// scales a million each when a step of K loads its own scales, and 44 us; with scales 64 bytes of a row at a time 37.  Blocks of 128
// columns leave half of each line of codes for later: 53.  For 64 tokens the loads of operands come first too, then the products: 60 us
// with all of them, 41 without those of codes, 48 without those of tokens, 35 without both; without decoding 57, without the LDS reads 56
// (then by steps to 55).  A compute unit holds one workgroup there, two wavefronts a SIMD: the tokens take 128 of its 160 KB of LDS, and
// two workgroups would need both halves of that and at most 128 registers (R = 1: 157 to 172, R = 2: 235 to 256).  Codes two and three
// blocks ahead: no faster.
constexpr int kSharedWaves = 4, kSharedHalves = 2;
constexpr int kSubs = kBlockK / kHalfK;

template <int T, int R, int G>
__global__ void __launch_bounds__(64 * kSharedWaves * kSharedHalves) pgq_linear4_shared_kernel(pgq_linear4_fwd f, Cut cut)
{
    __shared__ __align__(16) uint8_t lds[kSharedHalves][2][kSubs * 16 * T * 256];
    const int tid = (int)threadIdx.x & 255, lane = tid & 63, wave = tid >> 6;
    const int mine = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 8);            // half
    const int r = lane & 15, q = lane >> 4;
    // Codes by quads (8192 -> 28672, R = 1: 16 tokens 31.8 -> 29.7 us, 32 41.6 -> 38.8), but with larger tiles the registers and the
    // way through LDS cost more than that (32 tokens, R = 2: 36.4 -> 37.5; 64: 54 -> 58).
    constexpr bool kQuads = T * R <= 2;
    const int code_row = kQuads ? lane >> 2 : r, code_piece = kQuads ? lane & 3 : q;
    const uint32_t tb = blockIdx.x % (uint32_t)cut.token_blocks, rest = blockIdx.x / (uint32_t)cut.token_blocks;
    const uint32_t part = rest % (uint32_t)cut.parts;
    const int64_t m0 = (int64_t)tb * kMost, n0 = ((int64_t)(rest / (uint32_t)cut.parts) * kSharedWaves + wave) * (16 * R);
    const uint8_t* crow[R];
    const uint16_t* srow[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        crow[j] = f.codes + min(n0 + 16 * j + code_row, f.N - 1) * f.ldc + 16 * code_piece;
        srow[j] = f.scales + min(n0 + 16 * j + r, f.N - 1) * f.lds;
    }
    // Thread: piece tid % 16 (8 columns) of each half block of T token rows, into LDS rows of 256 bytes.  The piece that quarter q
    // supplies to instruction d lies at place (4 d + q) ^ (row % 16): a 16-byte LDS read is done for lanes 0-3, 12-15 and 20-27 of a
    // half wavefront together (then for the others), and those are 16 different places.
    const int piece = tid & 15;
    int place = piece;
    if (G == 128) place = 4 * (piece & 3) + (piece >> 2);
    if (G == 64) place = 8 * (piece >> 3) + 4 * (piece & 1) + 2 * ((piece >> 1) & 1) + ((piece >> 2) & 1);
    const uint16_t* xrow[T];
    uint32_t to[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int m = (tid >> 4) + 16 * t;
        xrow[t] = f.x + min(m0 + m, f.M - 1) * f.ldx + 8 * piece;
        to[t] = m * 256 + (place ^ (m & 15)) * 16;
    }
    constexpr int GH = kHalfK / G;
    const int64_t row_bytes = (f.K + 7) / 8 * 4, scale_bytes = 2 * ((f.K + G - 1) / G);
    const int64_t whole = f.K / kBlockK, blocks = (f.K + kBlockK - 1) / kBlockK;
    const int64_t b0 = (int64_t)part * cut.blocks, end = min(blocks, b0 + cut.blocks);
    struct Tokens { u32x4 x[kSubs][T]; };
    struct Codes { u32x4 c[R][kSubs]; };
    auto load_x = [&](int64_t b, Tokens& h) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int u = 0; u < kSubs; ++u) h.x[u][t] = load16(xrow[t] + kBlockK * b + kHalfK * u);
    };
    auto load_codes = [&](int64_t b, Codes& h) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int u = 0; u < kSubs; ++u) h.c[j][u] = load16(crow[j] + kBlockK / 2 * b + kHalfK / 2 * u);
    };
    auto put_x = [&](int i, const Tokens& h) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < kSubs; ++u)
#pragma unroll
            for (int t = 0; t < T; ++t) *reinterpret_cast<u32x4*>(&lds[mine][i & 1][u * 16 * T * 256 + to[t]]) = h.x[u][t];
    };
    // Scales: 64 bytes of a row, 16 in each quarter of the wavefront, for the kRun blocks from a multiple of kRun on.
    constexpr int SB = kSubs * GH / 2, SW = GH > 1 ? GH / 2 : 1, kRun = 16 / SB;       // words of a block, of half of one; blocks of a load
    u32x4 held[R];
    auto load_scales = [&](int64_t run, u32x4* s) __attribute__((always_inline)) {
        if (64 * run + 64 <= scale_bytes) {
#pragma unroll
            for (int j = 0; j < R; ++j) s[j] = load16((const uint8_t*)srow[j] + 64 * run + 16 * q);
        } else {
#pragma unroll
            for (int j = 0; j < R; ++j) s[j] = load16_edge(srow[j], 64 * run + 16 * q, scale_bytes);
        }
    };
    f32x4 acc[R][T];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[j][t] = f32x4{};
    // products of block b, whose tokens lie in buffer i
    auto multiply = [&](int i, int b, const Codes& h) __attribute__((always_inline)) {
        const int word = SB * b & 15, from = 4 * (16 * (word >> 2) + r);
#pragma unroll
        for (int u = 0; u < kSubs; ++u) {
            uint32_t sc[R][SW];
#pragma unroll
            for (int j = 0; j < R; ++j)
#pragma unroll
                for (int i = 0; i < SW; ++i) {
                    const int e = u * GH / 2 + i;              // of the block's words
                    const uint32_t lo = SB == 4 ? held[j][e] : SB == 2 ? held[j][e] : word & 1 ? held[j][1] : held[j][0];
                    const uint32_t hi = SB == 4 ? held[j][e] : SB == 2 ? held[j][2 + e] : word & 1 ? held[j][3] : held[j][2];
                    sc[j][i] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)(word & 2 ? hi : lo));
                }
            u32x4 c[R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                c[j] = h.c[j][u];
                if (kQuads) c[j] = from_quads(c[j], lane);
                trade<G>(c[j]);
            }
#pragma unroll
            for (int g = 0; g < GH; ++g) {
                f32x4 p[R][T];
#pragma unroll
                for (int j = 0; j < R; ++j)
#pragma unroll
                    for (int t = 0; t < T; ++t) p[j][t] = f32x4{};
#pragma unroll
                for (int d = g * (4 / GH); d < (g + 1) * (4 / GH); ++d) {
                    bf16x8 x[T];
#pragma unroll
                    for (int t = 0; t < T; ++t)
                        x[t] = *reinterpret_cast<const bf16x8*>(&lds[mine][i & 1][u * 16 * T * 256 + (16 * t + r) * 256 + ((4 * d + q) ^ r) * 16]);
#pragma unroll
                    for (int j = 0; j < R; ++j) {
                        const bf16x8 w = decode8(c[j][d]);
#pragma unroll
                        for (int t = 0; t < T; ++t) p[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[t], w, p[j][t], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    const int i = u * GH % 2 + g;
                    const float s = f16_to_f32((uint16_t)(sc[j][i / 2] >> (16 * (i & 1))));
#pragma unroll
                    for (int t = 0; t < T; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j][t][e] = __builtin_fmaf(p[j][t][e], s, acc[j][t][e]);
                }
            }
        }
    };
    // Whole blocks: the first half takes as many as the second or one more; both take as many turns, for the barriers' sake.
    const int64_t last = min(end, whole);
    const int n = (int)max((int64_t)0, last - b0), turns = (n + 1) / 2, own = mine ? n - turns : turns;
    if (n > 0) {
        const int64_t first = b0 + (mine ? turns : 0);
        auto at = [&](int i) __attribute__((always_inline)) { return min(first + i, last - 1); };      // (loads past the last repeat it)
        Codes ring[2];
        Tokens x;
        u32x4 next[R];
        int64_t run = -1;
        load_scales(at(0) / kRun, next);
        load_x(at(0), x);
        load_codes(at(0), ring[0]);
        put_x(0, x);
#pragma unroll 1
        for (int b = 0; b < turns; b += 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                __syncthreads();
                const int64_t now = at(b + i);
                if (now / kRun != run) {
                    run = now / kRun;
#pragma unroll
                    for (int j = 0; j < R; ++j) held[j] = next[j];
                    if ((run + 1) * kRun < last) load_scales(run + 1, next);
                }
                load_x(at(b + i + 1), x);
                load_codes(at(b + i + 1), ring[1 - i]);
                __builtin_amdgcn_sched_barrier(0);
                if (b + i < own) multiply(b + i, (int)now, ring[i]);
                if (b + i + 1 >= turns) break;
                put_x(b + i + 1, x);
            }
        }
    }
    if (last < end) {                             // the last block, by the first half: nothing past K is read, X is 0 there
        Codes h;
        Tokens x;
        if (mine == 0) {
#pragma unroll
            for (int u = 0; u < kSubs; ++u) {
#pragma unroll
                for (int t = 0; t < T; ++t) x.x[u][t] = load16_edge(xrow[t] - 8 * piece, 2 * (kBlockK * last + kHalfK * u + 8 * piece), 2 * f.K);
#pragma unroll
                for (int j = 0; j < R; ++j) h.c[j][u] = load16_edge(crow[j] - 16 * code_piece, kBlockK / 2 * last + kHalfK / 2 * u + 16 * code_piece, row_bytes);
            }
            load_scales(last / kRun, held);
            put_x(turns, x);                      // (the buffer that the turn before the last one used)
        }
        __syncthreads();
        if (mine == 0) multiply(turns, (int)last, h);
    }
    __syncthreads();
    f32x4(*sums)[kSharedWaves][R * T][64] = reinterpret_cast<f32x4(*)[kSharedWaves][R * T][64]>(&lds[0][0][0]);
    static_assert(sizeof(f32x4) * kSharedHalves * kSharedWaves * R * T * 64 <= sizeof(lds), "sums fit in the tokens' place");
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int t = 0; t < T; ++t) sums[mine][wave][j * T + t][lane] = acc[j][t];
    __syncthreads();
    // accumulator element e of lane l: token 4 (l / 16) + e, weight row l % 16; each half finishes every other one
#pragma unroll 1
    for (int u = lane + 64 * mine; u < R * T * 256; u += 128) {
        const int e = (u >> 6) & 3, i = u >> 8;
        const int64_t m = m0 + 16 * (i % T) + 4 * q + e, nn = n0 + 16 * (i / T) + r;
        if (m >= f.M || nn >= f.N) continue;
        const float z = sums[0][wave][i][lane][e] + sums[1][wave][i][lane][e];
        if (cut.parts > 1) cut.sums[((int64_t)part * f.M + m) * f.N + nn] = z;
        else finish(f, m, nn, z);
    }
}

// ---- stream ---------------------------------------------------------------------------------------------
// A wavefront lies along K: lane l holds 32 columns of each slab of 2048, whose tokens stay in its registers while rows go by,
// 16 bytes of codes and one scale a lane, row and slab; v_dot2_f32_bf16 multiplies (two additions of fp32 each).  Nothing is shared
// before a row's 64 partial sums are added, so the codes of the next 8 KB of rows are always in flight, and a row is read in one go:
// 4096 -> 4096 4.1 us of which 2.5 are any kernel's, 8192 -> 8192 9.0, 8192 -> 28672 22.2, 4096 -> 128256 49 (5.6 TB/s), 8192 -> 262144
// 171 (6.5, as fast as anything here reads).  With
// three and four tokens the multiplications take over (8192 -> 28672: 42 and 50 us, the shared kernel 27).
constexpr int kStreamWaves = 4;
constexpr int kSlab = 2048;

struct Stream {
    int32_t rows;                // of a wavefront, or of the `split` that share them
    int32_t split;               // wavefronts of a workgroup that share rows, each with its slabs of K
};

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float x)
{
    return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, ROWS, 0xF, false));
}
// the sum over the wavefront, in lane 63
__device__ __forceinline__ float wave_sum(float x)
{
    x = dpp_add<0xB1, 0xF>(x);                    // quad_perm: lane ^ 1
    x = dpp_add<0x4E, 0xF>(x);                    // quad_perm: lane ^ 2
    x = dpp_add<0x141, 0xF>(x);                   // row_half_mirror
    x = dpp_add<0x140, 0xF>(x);                   // row_mirror: every lane of a row of 16 has its sum
    x = dpp_add<0x142, 0xA>(x);                   // row_bcast 15 to rows 1 and 3
    return dpp_add<0x143, 0xC>(x);                // row_bcast 31 to rows 2 and 3
}

// S: slabs of a wavefront, M: tokens.  25 <= K <= 2048 S split, for two tokens a multiple of 32.
template <int S, int M>
__global__ void __launch_bounds__(64 * kStreamWaves) pgq_linear4_stream_kernel(pgq_linear4_fwd f, Stream a)
{
    constexpr int RG = 8 / S;       // rows loaded together: 8 KB
    __shared__ float part[kStreamWaves][M][64];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int piece = wave % a.split;
    const int64_t w = (int64_t)blockIdx.x * (kStreamWaves / a.split) + wave / a.split;
    const int64_t first = min(f.N, w * a.rows), last = min(f.N, first + a.rows);
    const int shift = 31 - __builtin_clz((unsigned)f.group);
    uint32_t x[M][S][16];
    uint32_t code_at[S], scale_at[S];
    // `past`: K is not whole lanes (one token only).  The lane that reaches past the row takes its last 32 columns, with token values of 0
    // where they are another lane's.  Lanes wholly past K: token values of 0, any codes and scale of the row.
    auto load_x = [&](bool past) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int64_t k = ((int64_t)piece * S + s) * kSlab + 32 * lane;
            const int64_t at = past ? min(k, (f.K + 7) / 8 * 8 - 32) : k;
            const bool in = k < f.K;
            code_at[s] = in ? (uint32_t)(at / 2) : 0u;
            scale_at[s] = in ? (uint32_t)(k >> shift) : 0u;
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u32x4 v = {};
                    if (past && i == 3 && in && at + 32 > f.K) v = load16_edge(f.x, 2 * (at + 24), 2 * f.K);
                    else if (past ? in && at + 8 * i >= k : in) v = load16(f.x + m * f.ldx + at + 8 * i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[m][s][4 * i + e] = v[e];
                }
        }
    };
    if (M == 1 && f.K % 32 != 0) load_x(true);
    else load_x(false);
    struct Rows { u32x4 c[RG][S]; uint16_t s[RG][S]; };
    auto load = [&](int64_t n, Rows& h) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < RG; ++j) {
            const int64_t row = min(n + j, f.N - 1);      // (rows past the last are not stored)
            const uint8_t* c = f.codes + row * f.ldc;
            const uint16_t* sc = f.scales + row * f.lds;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                h.c[j][s] = load16_once(c + code_at[s]);
                h.s[j][s] = sc[scale_at[s]];
            }
        }
    };
    float sum[M];                                         // lane i: of row first + i
#pragma unroll
    for (int m = 0; m < M; ++m) sum[m] = 0.0f;
    auto multiply = [&](int64_t n, const Rows& h) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < RG; ++j) {
            float acc[M];
#pragma unroll
            for (int m = 0; m < M; ++m) acc[m] = 0.0f;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float p[M];
#pragma unroll
                for (int m = 0; m < M; ++m) p[m] = 0.0f;
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const u32x4 v = __builtin_bit_cast(u32x4, decode8(h.c[j][s][d]));
#pragma unroll
                    for (int m = 0; m < M; ++m)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t ve = v[e];
                            p[m] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, ve), __builtin_bit_cast(bf16x2, x[m][s][4 * d + e]), p[m], false);
                        }
                }
#pragma unroll
                for (int m = 0; m < M; ++m) acc[m] = __builtin_fmaf(p[m], f16_to_f32(h.s[j][s]), acc[m]);
            }
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int total = __builtin_amdgcn_readlane(__builtin_bit_cast(int, wave_sum(acc[m])), 63);
                sum[m] = lane == (int)(n - first) + j ? __builtin_bit_cast(float, total) : sum[m];
            }
        }
    };
    if (first < last) {
        Rows h, next;
        load(first, h);
        int64_t n = first;
#pragma unroll 1
        for (; n + RG < last; n += RG) {
            load(n + RG, next);
            __builtin_amdgcn_sched_barrier(0);
            multiply(n, h);
            h = next;
        }
        multiply(n, h);
    }
    if (a.split > 1) {
#pragma unroll
        for (int m = 0; m < M; ++m) part[wave][m][lane] = sum[m];
        __syncthreads();
        if (piece != 0) return;
#pragma unroll
        for (int m = 0; m < M; ++m)
            for (int i = 1; i < a.split; ++i) sum[m] += part[wave + i][m][lane];
    }
    if (first + lane >= last) return;
#pragma unroll
    for (int m = 0; m < M; ++m) finish(f, m, first + lane, sum[m]);
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
int token_tiles(const pgq_linear4_fwd& p) { return p.M <= 16 ? 1 : p.M <= 32 ? 2 : 4; }

// ---- how a call runs ----------------------------------------------------------------------------------
enum Path { P_STREAM, P_ROWS, P_SHARED };
struct Plan {
    int path;
    int rows;                    // R, or the slabs of a streaming wavefront
    Stream stream;
    Cut cut;
    size_t bytes;
};

// Streaming needs the 16 bytes of codes that a lane loads and at most four slabs (two tokens: two) a wavefront, sixteen (eight) a workgroup.  With three or
// four slabs one wavefront a SIMD takes an equal share of the rows (8192 -> 28672, 1024 and 8192 wavefronts: 22.2 and 25.8 us, 14336
// -> 4096 9.0 and 10.4); with fewer, every load of rows has a wavefront of its own (4096 -> 14336 8.9 and 8.6, 2048 -> 16384 6.5
// and 5.5).  K that is not whole lanes of 32 columns: for one token (4100 -> 4100 5.9, the tiles 7.5; 8200 -> 28672 29 and 35).
bool stream_plan(const pgq_linear4_fwd& p, Plan& q)
{
    const int64_t slabs = (p.K + kSlab - 1) / kSlab, most = p.M == 1 ? 4 : 2;
    if (p.M > 2 || p.K < 25 || (p.M > 1 && p.K % 32 != 0) || slabs > most * kStreamWaves) return false;
    q.path = P_STREAM;
    q.stream.split = slabs <= most ? 1 : slabs <= 2 * most ? 2 : 4;
    q.rows = (int)((slabs + q.stream.split - 1) / q.stream.split);
    const int64_t group = 8 / q.rows, waves = (q.rows >= 3 ? 1024 : 8192) / q.stream.split, per = (p.N + waves - 1) / waves;
    q.stream.rows = (int32_t)std::min<int64_t>(64, (per + group - 1) / group * group);
    return true;
}

// One way to cut a call for the kernels of 16-row tiles, and its estimated microseconds past the launch: turns of the kernel's K
// loop times their measured length and rounds of workgroups, what comes before and after the loop, and the second launch with the
// traffic of the parts' sums (at 5 TB/s, written and read).  A turn is longer where the machine is full (`busy`).  Of the shared
// kernel's larger tiles a compute unit holds one workgroup.
double tile_cost(const pgq_linear4_fwd& p, int path, int rows, int64_t parts, Cut& cut)
{
    const int t = token_tiles(p);
    const int64_t blocks = (p.K + kBlockK - 1) / kBlockK;
    const int64_t together = path == P_ROWS ? kWaves4 : kSharedHalves;        // blocks a workgroup takes at a time
    const int64_t tile = 16 * rows * (path == P_ROWS ? 1 : kSharedWaves);
    const int64_t grid = (p.N + tile - 1) / tile * token_blocks(p) * parts, per = (blocks + parts - 1) / parts;
    if (parts > 1 && (per < together || (parts - 1) * per >= blocks || grid > 512)) return -1.0;
    cut.parts = (int32_t)parts;
    cut.blocks = per;
    const bool one = path == P_SHARED && (t == 4 || rows == 2);
    const double full = (double)grid / 256.0, busy = std::min(1.0, full);
    const double rounds = one ? (double)((grid + 255) / 256) : std::max(1.0, full);
    double turn, rest = 0.0;
    if (path == P_ROWS) {
        turn = t == 1 ? 1.0 + (0.4 + 0.02 * (double)p.M) * busy + (0.5 + 0.6 * busy) * (rows - 1) : t == 2 ? 1.0 + 1.5 * busy : 1.6 + 3.4 * busy;
        rest = 0.6;
    } else if (rows == 1) {
        turn = t == 1 ? 0.6 + 0.4 * busy : t == 2 ? 0.9 + 0.4 * busy : 1.3 + 0.75 * busy;
        rest = t == 4 ? 3.0 : 1.5;
    } else {
        turn = t == 1 ? 1.2 + 0.35 * busy : t == 2 ? 1.95 : 3.0;
        rest = t == 4 ? 4.0 : 2.5;
    }
    const double join = parts > 1 ? 4.0 + (double)parts * (double)p.M * (double)p.N * 8.0 / 5e6 : 0.0;
    return (double)((per + together - 1) / together) * turn * rounds + rest + join;
}

// Streaming for one or two tokens; the cheapest way through the kernels of 16-row tiles for more: K spread over a workgroup where the
// layer is small, the tokens shared through LDS where X would be read too often.  Measured on one MI355X in us, each at its best rows
// and parts:
//   tokens x K x N        rows    shared        tokens x K x N         rows    shared
//   4 x 4096 x 4096        6.1     10.0         4 x 8192 x 28672       40.7     27.1
//   16 x 4096 x 4096       6.5      9.5         16 x 4096 x 14336      15.7     11.2
//   16 x 8192 x 8192      11.8     15.8         16 x 8192 x 28672      44       29
//   32 x 4096 x 4096       8.8     11.7         32 x 8192 x 28672      79       37
//   32 x 1024 x 1024       4.1      6.0         32 x 8192 x 8192       24.9     18.6
//   64 x 528 x 1584        5.4      8.7         64 x 2048 x 2048        7.5     12.0
//   64 x 4096 x 4096      13.7     14.6         64 x 8192 x 8192       40       26
// The choice was within 8% of the best of all that were tried at all but a few of 96 sizes.
Plan plan(const pgq_linear4_fwd& p)
{
    Plan q;
    memset(&q, 0, sizeof(q));
    if (stream_plan(p, q)) return q;
    const int t = token_tiles(p);
    double best = -1.0;
    for (int path = P_ROWS; path <= P_SHARED; ++path)
        for (int rows = 1; rows <= (path == P_ROWS && t > 1 ? 1 : 2); ++rows)
            for (int64_t parts = 1; parts <= 16; parts *= 2) {
                Cut cut = {};
                const double us = tile_cost(p, path, rows, parts, cut);
                if (us < 0) break;
                if (best >= 0 && us >= best) continue;
                best = us;
                q.path = path;
                q.rows = rows;
                q.cut = cut;
            }
    q.cut.token_blocks = (int32_t)token_blocks(p);
    q.bytes = q.cut.parts > 1 ? ((size_t)q.cut.parts * p.M * p.N * 4 + 255) / 256 * 256 : 0;
    return q;
}
int64_t stream_grid(const pgq_linear4_fwd& p, const Plan& q)
{
    const int64_t rows = (int64_t)q.stream.rows * (kStreamWaves / q.stream.split);
    return (p.N + rows - 1) / rows;
}
int64_t grid_of(const pgq_linear4_fwd& p, const Plan& q)
{
    if (q.path == P_STREAM) return stream_grid(p, q);
    const int64_t rows = 16 * q.rows * (q.path == P_SHARED ? kSharedWaves : 1);
    return (p.N + rows - 1) / rows * q.cut.token_blocks * q.cut.parts;
}
int block_of(const Plan& q) { return 64 * (q.path == P_STREAM ? kStreamWaves : q.path == P_SHARED ? kSharedWaves * kSharedHalves : kWaves4); }
int64_t join_grid(const pgq_linear4_fwd& p) { return (p.M * p.N + 255) / 256; }
bool launches_fit(const pgq_linear4_fwd& p, const Plan& q)
{
    return grid_fits(grid_of(p, q), block_of(q)) && (q.cut.parts <= 1 || grid_fits(join_grid(p), 256));
}

const void* stream_kernel(int slabs, int m)
{
    if (m == 2) return slabs == 1 ? reinterpret_cast<const void*>(&pgq_linear4_stream_kernel<1, 2>) : reinterpret_cast<const void*>(&pgq_linear4_stream_kernel<2, 2>);
    return slabs == 1   ? reinterpret_cast<const void*>(&pgq_linear4_stream_kernel<1, 1>)
           : slabs == 2 ? reinterpret_cast<const void*>(&pgq_linear4_stream_kernel<2, 1>)
           : slabs == 3 ? reinterpret_cast<const void*>(&pgq_linear4_stream_kernel<3, 1>)
                        : reinterpret_cast<const void*>(&pgq_linear4_stream_kernel<4, 1>);
}
template <int T, int R>
const void* rows_kernel(int32_t group)
{
    return group == 32   ? reinterpret_cast<const void*>(&pgq_linear4_rows_kernel<T, R, 32>)
           : group == 64 ? reinterpret_cast<const void*>(&pgq_linear4_rows_kernel<T, R, 64>)
                         : reinterpret_cast<const void*>(&pgq_linear4_rows_kernel<T, R, 128>);
}
template <int T, int R>
const void* shared_kernel(int32_t group)
{
    return group == 32   ? reinterpret_cast<const void*>(&pgq_linear4_shared_kernel<T, R, 32>)
           : group == 64 ? reinterpret_cast<const void*>(&pgq_linear4_shared_kernel<T, R, 64>)
                         : reinterpret_cast<const void*>(&pgq_linear4_shared_kernel<T, R, 128>);
}
const void* kernel_of(const pgq_linear4_fwd& p, const Plan& q)
{
    const int t = token_tiles(p), g = p.group;
    if (q.path == P_STREAM) return stream_kernel(q.rows, (int)p.M);
    if (q.path == P_ROWS) {
        if (t > 1) return t == 2 ? rows_kernel<2, 1>(g) : rows_kernel<4, 1>(g);
        return q.rows == 1 ? rows_kernel<1, 1>(g) : rows_kernel<1, 2>(g);
    }
    if (t == 1) return q.rows == 1 ? shared_kernel<1, 1>(g) : shared_kernel<1, 2>(g);
    if (t == 2) return q.rows == 1 ? shared_kernel<2, 1>(g) : shared_kernel<2, 2>(g);
    return q.rows == 1 ? shared_kernel<4, 1>(g) : shared_kernel<4, 2>(g);
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
    const Plan q = plan(*p);
    if (!launches_fit(*p, q)) return PGQ_ERR_SHAPE;
    *workspace_bytes = q.bytes;
    return PGQ_OK;
}

pgq_status pgq_linear4_forward(const pgq_linear4_fwd* p, void* workspace, size_t workspace_bytes, void* stream)
{
    const pgq_status st = check(p);
    if (st != PGQ_OK || p->M == 0 || p->N == 0) return st;
    Plan q = plan(*p);
    if (!launches_fit(*p, q)) return PGQ_ERR_SHAPE;
    if (q.bytes && (!workspace || workspace_bytes < q.bytes)) return PGQ_ERR_WORKSPACE;
    if (q.bytes && !is_aligned(workspace, 256)) return PGQ_ERR_ALIGN;
    pgq_linear4_fwd f = *p;
    q.cut.sums = static_cast<float*>(workspace);
    void *sargs[] = {&f, &q.stream}, *args[] = {&f, &q.cut};
    Launches l(q.cut.parts > 1 ? 2 : 1, stream);
    l.go(kernel_of(f, q), grid_of(f, q), block_of(q), q.path == P_STREAM ? sargs : args);
    if (q.cut.parts > 1) l.go(reinterpret_cast<const void*>(&pgq_linear4_join_kernel), join_grid(f), 256, args);
    return l.done();
}

}  // extern "C"
