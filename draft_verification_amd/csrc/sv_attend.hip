// Attention of the rows of drafted blocks over the paged cache
// (spec_verify_attend in include/spec_verify.h, which states the formulas).

#include <float.h>
#include <math.h>

#include <algorithm>

#include "spec_verify.h"
#include "sv_attend_plan.h"
#include "sv_cache.h"
#include "sv_host.h"

using sv::cache_status;
using sv::cache_uniform;
using sv::DeviceGuard;
using sv::kAttendTokens;
using sv::kAttendWaves;
using sv::launch_kernel;
using sv::Sequence;

namespace {

constexpr int kThreads = 64 * kAttendWaves;

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct Attend {
    sv::Cache c;
    sv::Rows r;
    int b0, B;                  // sequences of the launch
    int kv_heads, group, dim;   // group: heads to a key-value head
    const unsigned short* q;
    long long qb, qr, qh;
    unsigned short* out;
    long long ob, orow, oh;
    float* lse;
    const char* keys;
    const char* values;
    long long page_stride, head_stride; // bytes
    unsigned token_stride;
    const float* kscale;
    const float* vscale;
    float scale;
    int window, max_len;
    int blocks, splits, span;
    float* parts;               // [B][kv_heads][blocks][splits]: sums of a workgroup, then its (reference, sum) pairs
    int* status;
};

// 16 bytes of a wavefront's part of LDS, written and read by this wavefront only:
// LDS operations of one wavefront stay in order, so the compiler alone has to be
// held back.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The tokens that a sequence's rows see, and how they are split.
struct Reach {
    int low, end; // low: a multiple of the tile
    int splits;
};

__device__ __forceinline__ Reach reach_of(const Attend& q, const Sequence& s)
{
    Reach r;
    r.end = s.start + s.count;
    r.low = 0;
    if (q.window && s.start + 1 > q.window) r.low = (s.start + 1 - q.window) / kAttendTokens * kAttendTokens;
    r.splits = (r.end - r.low + q.span - 1) / q.span;
    return r;
}

// The sequence, with those marked bad that are longer than the caller said.
__device__ __forceinline__ Sequence sequence_within(const Attend& q, int b)
{
    Sequence s = sv::sequence_of(q.c, q.r, b);
    if (s.count > 0 && s.start + s.count > q.max_len) s.count = -1;
    return s;
}

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ unsigned pack_bf16(float a, float b)
{
    const bf16x2 p = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(unsigned, p);
}

// Two codes of e4m3 as two bf16 (exact: 3 bits of fraction, exponents from -9 to 8).
template <bool HIGH>
__device__ __forceinline__ unsigned widen_e4m3(unsigned codes)
{
    return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, HIGH));
}

// Whether one of two bf16 is infinite or NaN.
__device__ __forceinline__ bool special2(unsigned w)
{
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

__device__ __forceinline__ unsigned without_special(unsigned w)
{
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

// Attention of one block of rows over one split of a sequence's length.
//
// The scores of a tile of 16 tokens and 16 rows are K Q^T, so that a lane holds one
// row's scores of four tokens in each of two tiles; rounded, these are in place as
// the right operand of out^T = V^T P^T, whose left operand LDS reads transposed.  A
// row's maximum is not followed at every step: its reference stays as long as no
// score lies more than 8 (in log2) above it, which keeps the weights below 2^8 and
// spares the sums' rescaling.
//
// The four wavefronts take every fourth tile of 32 tokens, each through its own part
// of LDS and with registers one tile ahead, without a barrier until the end, where
// their sums are joined.
template <int DIM, bool E4M3, int TILES>
__global__ __launch_bounds__(kThreads, DIM == 64 && TILES == 1 ? 4 : (DIM == 128 && TILES <= 3) || DIM == 64 ? 2 : 1) void sv_attend_kernel(Attend q)
{
    constexpr int kUnit = E4M3 ? 16 : 8;           // values of 16 bytes of the cache
    constexpr int kLanes = DIM / kUnit;            // lanes that read a token's row
    constexpr int kPer = 64 / kLanes;              // tokens of a load
    constexpr int kLoads = kAttendTokens / kPer;   // loads of a tile, of keys and of values each
    constexpr int kChunks = DIM / 8;               // 16 bytes of bf16
    constexpr int kSteps = DIM / 32;               // products of a score
    constexpr int kOut = DIM / 16;                 // tiles of a row of outputs
    constexpr int kTileBytes = kAttendTokens * DIM * 2;
    constexpr bool kQueryLds = TILES > 2;
    constexpr int kMergeRow = DIM + 4;             // floats of a row where the sums meet
    constexpr int kStage = kAttendWaves * kTileBytes;
    constexpr int kMerge = kAttendWaves * 16 * kMergeRow * 4;
    __shared__ __attribute__((aligned(16))) char stage[kStage > kMerge ? kStage : kMerge];
    __shared__ u32x4 query[kQueryLds ? TILES * kSteps * 64 : 1];
    __shared__ int place[TILES * 16];              // position of each row
    __shared__ float refs[kAttendWaves][TILES * 16], sums[kAttendWaves][TILES * 16];

    const int lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // consecutive workgroups go round the eight dies; the row blocks that read the same
    // tokens follow each other on one
    unsigned id = blockIdx.x;
    int block = 0;
    if (q.blocks > 1) {
        const unsigned die = id % 8, turn = id / 8;
        block = (int)(turn % q.blocks);
        id = turn / q.blocks * 8 + die;
    }
    const unsigned per = (unsigned)q.kv_heads * q.B;
    const int split = (int)(id / per);
    if (split >= q.splits) return;
    const unsigned in_split = id % per;
    const int b = q.b0 + (int)(in_split / q.kv_heads), head = (int)(in_split % q.kv_heads);

    const Sequence s = sequence_within(q, b);
    if (s.count <= 0) {
        if (s.count < 0 && threadIdx.x == 0) cache_status(q.status, SV_STATUS_BAD_INPUT);
        return;
    }
    const Reach reach = reach_of(q, s);
    if (split >= reach.splits) return;
    const int row0 = block * TILES * 16;           // first row (of a row and a head) of the workgroup
    const int rows = s.count * q.group - row0;     // and how many there are
    if (rows <= 0) return;
    const int first = reach.low + split * q.span, last = min(first + q.span, reach.end);

    // the queries, negative for a negative scale, as right operands; rows past the last
    // are those of the last
    float scale = q.scale * 1.44269504088896340736f;
    if (E4M3 && q.kscale) scale *= cache_uniform(q.kscale + head);
    const unsigned flip = scale < 0 ? 0x80008000u : 0u;
    scale = fabsf(scale);
    const float room = 8.0f / scale;               // how far a score may lie above its reference
    const bool followed = room < FLT_MAX;          // (a scale of about zero: the reference is 0)
    auto query_at = [&](int tile, int step) {
        const int m = min(tile * 16 + n16, rows - 1) + row0;
        const int r = m / q.group, h = head * q.group + m % q.group;
        const unsigned short* from = q.q + (q.r.roff ? (s.first + r) * q.qr : b * q.qb + r * q.qr) + h * q.qh;
        const int d = step * 32 + g * 8;
        u32x4 x = {0, 0, 0, 0};
        if (d < q.dim) x = *(const u32x4_any*)(from + d);
        return x ^ flip;
    };
    u32x4 qreg[kQueryLds ? 1 : TILES][kQueryLds ? 1 : kSteps];
    if constexpr (kQueryLds) {
        for (int i = wave; i < TILES * kSteps; i += kAttendWaves) query[i * 64 + lane] = query_at(i / kSteps, i % kSteps);
    } else {
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
            for (int k = 0; k < kSteps; ++k) qreg[i][k] = query_at(i, k);
    }
    for (int i = threadIdx.x; i < TILES * 16; i += kThreads) place[i] = s.start + (min(i, rows - 1) + row0) / q.group;

    // the wavefront's own LDS, for keys and then for values: a token's row of 16-byte chunks,
    // their order changed from token to token so that a column of them lies in different banks
    char* const own = stage + wave * kTileBytes;
    auto key_at = [](int t, int chunk) { return t * DIM * 2 + ((chunk ^ ((DIM == 64 ? t >> 1 : t) & (kChunks < 16 ? 7 : 15))) * 16); };
    auto value_at = [](int t, int half) { return t * DIM * 2 + ((half ^ ((DIM == 64 ? t >> 1 : t) & (kOut < 8 ? 3 : 7))) * 32); };

    const int in_load = lane / kLanes, unit = lane % kLanes;
    const bool lane_in = unit * kUnit < q.dim;
    const long long in_page = head * q.head_stride + (lane_in ? unit * 16 : 0);
    const int* table = q.c.table + (long long)s.slot * q.c.max_pages;
    const int mask = (1 << q.c.shift) - 1;

    // the pages of a tile's tokens, a token to each of 32 lanes; those past the end are the last
    auto pages_of = [&](int t0) { return table[min(t0 + (lane & 31), reach.end - 1) >> q.c.shift]; };
    u32x4 kr[kLoads], vr[kLoads];
    auto is_bad = [&](int page) { return page < 0 || page >= q.c.n_pages; };
    auto load = [&](u32x4 (&x)[kLoads], const char* from, int t0, int page) { // of a bad page's tokens, the first page's
        if (is_bad(page)) page = 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int t = i * kPer + in_load;
            x[i] = *(const u32x4*)(from + in_page + __shfl(page, t) * q.page_stride + (unsigned)(min(t0 + t, reach.end - 1) & mask) * (unsigned long long)q.token_stride);
        }
    };
    auto widen = [](u32x4 x, int k) -> u32x4 { // eight values of a load as bf16
        if constexpr (!E4M3) return x;
        else return u32x4{widen_e4m3<false>(x[2 * k]), widen_e4m3<true>(x[2 * k]), widen_e4m3<false>(x[2 * k + 1]), widen_e4m3<true>(x[2 * k + 1])};
    };

    f32x4 acc[TILES][kOut] = {};
    float ref[TILES], top[TILES], sum[TILES]; // ref: a score; top = ref * scale
#pragma unroll
    for (int i = 0; i < TILES; ++i) ref[i] = followed ? -FLT_MAX : 0.0f, top[i] = followed ? -FLT_MAX : 0.0f, sum[i] = 0.0f;

    const int stride = kAttendTokens * kAttendWaves;
    int t0 = first + wave * kAttendTokens;
    int page = 0, next_page = 0; // of a token of the tile in hand and of the next
    if (t0 < last) {
        page = pages_of(t0);
        load(kr, q.keys, t0, page);
        load(vr, q.values, t0, page);
        next_page = pages_of(t0 + stride);
    }
    __syncthreads(); // queries and places
    for (; t0 < last; t0 += stride) {
        const bool more = t0 + stride < last;
        const unsigned gone = (unsigned)__ballot(is_bad(page)); // tokens whose page is bad
        if (gone && lane == 0) cache_status(q.status, SV_STATUS_BAD_INPUT);
        // some row does not see some token
        const bool mixed = t0 + kAttendTokens - 1 > s.start || gone || (q.window && t0 <= s.start + s.count - 1 - q.window);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (int k = 0; k < kUnit / 8; ++k)
                *(u32x4*)(own + key_at(i * kPer + in_load, unit * (kUnit / 8) + k)) = lane_in ? widen(kr[i], k) : u32x4{0, 0, 0, 0};
        if (more) load(kr, q.keys, t0 + stride, next_page);
        wave_sync();
        bf16x8 k[2][kSteps];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < kSteps; ++e) k[u][e] = *(const bf16x8*)(own + key_at(u * 16 + n16, e * 4 + g));
        u32x4 p[TILES];
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            f32x4 x[2] = {};
#pragma unroll
            for (int e = 0; e < kSteps; ++e) {
                bf16x8 y;
                if constexpr (kQueryLds) y = __builtin_bit_cast(bf16x8, query[(i * kSteps + e) * 64 + lane]);
                else y = __builtin_bit_cast(bf16x8, qreg[i][e]);
#pragma unroll
                for (int u = 0; u < 2; ++u) x[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[u][e], y, x[u], 0, 0, 0);
            }
            unsigned hidden = 0; // bit u * 4 + j
            if (mixed) {
                const int at = place[i * 16 + n16], low = q.window ? at - q.window : -1;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int in = u * 16 + g * 4 + j, t = t0 + in;
                        if (t > at || t <= low || (gone >> in & 1)) {
                            hidden |= 1u << (u * 4 + j);
                            x[u][j] = -FLT_MAX;
                        }
                    }
            }
            if (followed) {
                float most = fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])), fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3])));
                if (__ballot(most > ref[i] + room)) {
                    most = fmaxf(most, __shfl_xor(most, 16));
                    most = fmaxf(most, __shfl_xor(most, 32));
                    most = fmaxf(most, ref[i]);
                    if (most > ref[i]) {
                        const float now = most * scale, factor = exp2_of(top[i] - now);
                        ref[i] = most;
                        top[i] = now;
                        sum[i] *= factor;
#pragma unroll
                        for (int e = 0; e < kOut; ++e) acc[i][e] *= factor;
                    }
                }
            }
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = exp2_of(fmaf(x[j / 4][j % 4], scale, -top[i]));
            if (mixed) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (hidden >> j & 1) w[j] = 0.0f;
            }
            sum[i] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
            // rounded to bf16, as the matrix cores take them: half a step of 2^-8 each, as the
            // outputs' own rounding is
            p[i] = u32x4{pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]), pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7])};
        }
        wave_sync(); // the keys are read
        bool odd = false; // infinities or NaN among the values of a mixed tile
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (int k = 0; k < kUnit / 8; ++k) {
                const int chunk = unit * (kUnit / 8) + k;
                u32x4 v = lane_in ? widen(vr[i], k) : u32x4{0, 0, 0, 0};
                if (mixed) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) odd |= special2(v[j]), v[j] = without_special(v[j]);
                }
                *(u32x4*)(own + value_at(i * kPer + in_load, chunk / 2) + chunk % 2 * 16) = v;
            }
        if (more) load(vr, q.values, t0 + stride, next_page);
        wave_sync();
#pragma unroll
        for (int e = 0; e < kOut; ++e) {
            // values of four tokens of each half, a column to each lane
            s16x4 v[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = u * 16 + g * 4 + n16 / 4;
                v[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(own + value_at(t, e) + n16 % 4 * 8));
            }
            const u32x2 lo = __builtin_bit_cast(u32x2, v[0]), hi = __builtin_bit_cast(u32x2, v[1]);
            const bf16x8 a = __builtin_bit_cast(bf16x8, u32x4{lo[0], lo[1], hi[0], hi[1]});
#pragma unroll
            for (int i = 0; i < TILES; ++i) acc[i][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, p[i]), acc[i][e], 0, 0, 0);
        }
        if (mixed && __ballot(odd)) {
            // Values that are infinite or NaN were taken as zero, since a weight of zero does not
            // hide them from rows that do not see their token.  They are added one by one.
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                wave_sync();
                ((u32x4*)own)[lane] = p[i];
                wave_sync();
                const int at = place[i * 16 + n16], low = q.window ? at - q.window : -1;
                for (int in = 0; in < kAttendTokens && t0 + in < reach.end; ++in) {
                    const int t = t0 + in;
                    if (gone >> in & 1) continue;
                    const unsigned short* const all = (const unsigned short*)own;
                    const float w = __uint_as_float((unsigned)all[(in % 16 / 4 * 16 + n16) * 8 + in / 16 * 4 + in % 4] << 16);
                    const bool sees = t <= at && t > low;
                    const char* from = q.values + head * q.head_stride + table[t >> q.c.shift] * q.page_stride + (unsigned)(t & mask) * (unsigned long long)q.token_stride;
#pragma unroll
                    for (int e = 0; e < kOut; ++e) {
                        const int d = e * 16 + g * 4;
                        if (!sees || d >= q.dim) continue;
                        unsigned x[2];
                        if constexpr (E4M3) {
                            const unsigned codes = *(const unsigned*)(from + d);
                            x[0] = widen_e4m3<false>(codes), x[1] = widen_e4m3<true>(codes);
                        } else {
                            const u32x2 raw = *(const u32x2*)(from + 2 * d);
                            x[0] = raw[0], x[1] = raw[1];
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const unsigned bits = j % 2 ? x[j / 2] & 0xffff0000u : x[j / 2] << 16;
                            if ((bits & 0x7f800000u) == 0x7f800000u) acc[i][e][j] += w * __uint_as_float(bits);
                        }
                    }
                }
            }
        }
        wave_sync(); // the values are read
        page = next_page;
        if (more) next_page = pages_of(t0 + 2 * stride);
    }

    // the four wavefronts' sums, a tile of rows at a time
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
        sum[i] += __shfl_xor(sum[i], 16);
        sum[i] += __shfl_xor(sum[i], 32);
        if (g == 0) refs[wave][i * 16 + n16] = top[i], sums[wave][i * 16 + n16] = sum[i];
    }
    float* const meet = (float*)stage;
    const float vscale = E4M3 && q.vscale ? cache_uniform(q.vscale + head) : 1.0f;
    const bool whole = reach.splits == 1;
    float* const parts = q.parts + (((long long)(b * (long long)q.kv_heads + head) * q.blocks + block) * q.splits + split) * (TILES * 16 * (DIM + 2));
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
        if (i * 16 >= rows) break;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kOut; ++e) *(f32x4*)(meet + (wave * 16 + n16) * kMergeRow + e * 16 + g * 4) = acc[i][e];
        __syncthreads();
        const int r = threadIdx.x / 16, m = i * 16 + r;
        float most = refs[0][m];
#pragma unroll
        for (int w = 1; w < kAttendWaves; ++w) most = fmaxf(most, refs[w][m]);
        float factor[kAttendWaves], all = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttendWaves; ++w) {
            factor[w] = exp2_of(refs[w][m] - most);
            all += factor[w] * sums[w][m];
        }
        if (m >= rows) continue;
        const int full = m + row0, row = full / q.group, h = head * q.group + full % q.group;
        const float by = whole ? (all == 0.0f ? 0.0f : vscale / all) : 1.0f;
        const long long line = q.r.roff ? s.first + row : (long long)b * q.r.rows + row;
#pragma unroll
        for (int e = 0; e < DIM / 64; ++e) {
            const int d = e * 64 + threadIdx.x % 16 * 4;
            f32x4 x = {};
#pragma unroll
            for (int w = 0; w < kAttendWaves; ++w) x += factor[w] * *(const f32x4*)(meet + (w * 16 + r) * kMergeRow + d);
            if (!whole) {
                *(f32x4*)(parts + m * DIM + d) = x;
            } else if (d < q.dim) {
                unsigned short* to = q.out + (q.r.roff ? line * q.orow : b * q.ob + row * q.orow) + h * q.oh + d;
                *(u32x2_any*)to = u32x2{pack_bf16(x[0] * by, x[1] * by), pack_bf16(x[2] * by, x[3] * by)};
            }
        }
        if (threadIdx.x % 16 == 0) {
            if (!whole) {
                parts[TILES * 16 * DIM + 2 * m] = most;
                parts[TILES * 16 * DIM + 2 * m + 1] = all;
            } else if (q.lse) {
                q.lse[line * (q.kv_heads * q.group) + h] = all == 0.0f ? -INFINITY : (most + __builtin_amdgcn_logf(all)) * 0.69314718055994530942f;
            }
        }
    }
}

// Joins the splits of a row: a quarter of a wavefront to each row and head.
template <int DIM>
__global__ __launch_bounds__(kThreads) void sv_attend_join_kernel(Attend q, int tiles, int scaled)
{
    const int b = q.b0 + blockIdx.y;
    const Sequence s = sequence_within(q, b);
    if (s.count <= 0) return;
    const Reach reach = reach_of(q, s);
    if (reach.splits <= 1) return;
    const int at = blockIdx.x * 16 + threadIdx.x / 16; // row of the sequence, over all heads
    const int heads = q.kv_heads * q.group;
    if (at >= s.count * heads) return;
    const int head = at / (s.count * q.group), full = at % (s.count * q.group);
    const int block = full / (tiles * 16), m = full % (tiles * 16);
    const int row = full / q.group, h = head * q.group + full % q.group;
    const long long size = (long long)tiles * 16 * (DIM + 2);
    const float* parts = q.parts + (((long long)b * q.kv_heads + head) * q.blocks + block) * q.splits * size;
    const float* pairs = parts + (long long)tiles * 16 * DIM + 2 * m;
    float most = -INFINITY;
    for (int i = 0; i < reach.splits; ++i) most = fmaxf(most, pairs[i * size]);
    float all = 0.0f;
    constexpr int kEach = DIM / 64;
    f32x4 x[kEach] = {};
    for (int i = 0; i < reach.splits; ++i) {
        const float factor = exp2_of(pairs[i * size] - most);
        all += factor * pairs[i * size + 1];
#pragma unroll
        for (int e = 0; e < kEach; ++e) x[e] += factor * *(const f32x4*)(parts + i * size + m * DIM + e * 64 + threadIdx.x % 16 * 4);
    }
    const float by = all == 0.0f ? 0.0f : (scaled ? q.vscale[head] : 1.0f) / all;
    const long long line = q.r.roff ? s.first + row : (long long)b * q.r.rows + row;
    unsigned short* to = q.out + (q.r.roff ? line * q.orow : b * q.ob + row * q.orow) + h * q.oh;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int d = e * 64 + threadIdx.x % 16 * 4;
        if (d < q.dim) *(u32x2_any*)(to + d) = u32x2{pack_bf16(x[e][0] * by, x[e][1] * by), pack_bf16(x[e][2] * by, x[e][3] * by)};
    }
    if (q.lse && threadIdx.x % 16 == 0)
        q.lse[line * heads + h] = all == 0.0f ? -INFINITY : (most + __builtin_amdgcn_logf(all)) * 0.69314718055994530942f;
}

__global__ void sv_attend_status_kernel(int* status) { *status = 0; }

int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// Tokens that a sequence's rows may see, by what the call says.
long long most_seen(const spec_verify_attend_args* a)
{
    long long len = a->max_len ? a->max_len : (long long)a->cache.max_pages * a->cache.page_size;
    // with a window: its tokens, those before the first row's last one in its tile, and the other rows'
    if (a->window) len = std::min(len, (long long)a->window + a->rows + kAttendTokens);
    return len;
}

sv::AttendPlan plan_of(const spec_verify_attend_args* a)
{
    return sv::attend_plan(a->B, a->kv.kv_heads, padded_dim(a->kv.head_dim), (long long)a->rows * (a->heads / a->kv.kv_heads), most_seen(a));
}

template <int DIM, bool E4M3, int TILES>
hipError_t launch_attend(const Attend& q, hipStream_t s)
{
    constexpr int kMost = 0x7fffffff / kThreads; // workgroups of a launch, and more than enough
    const unsigned join = (unsigned)(((long long)q.r.rows * q.kv_heads * q.group + 15) / 16);
    const long long per = std::max<long long>((long long)q.kv_heads * q.blocks * q.splits, join);
    const int step = (int)std::max(1ll, std::min<long long>(65535, (kMost - 8 * q.blocks) / per));
    hipError_t e = hipSuccess;
    Attend a = q;
    for (a.b0 = 0; a.b0 < q.B && e == hipSuccess; a.b0 += step) {
        a.B = std::min(q.B - a.b0, step);
        long long groups = (long long)a.B * q.kv_heads * q.splits;
        if (q.blocks > 1) groups = (groups + 7) / 8 * 8 * q.blocks;
        e = launch_kernel(sv_attend_kernel<DIM, E4M3, TILES>, dim3((unsigned)groups), dim3(kThreads), 0, s, nullptr, nullptr, a);
        if (q.splits == 1) continue;
        const dim3 grid(join, (unsigned)a.B);
        if (e == hipSuccess)
            e = launch_kernel(sv_attend_join_kernel<DIM>, grid, dim3(kThreads), 0, s, nullptr, nullptr, a, TILES, (int)(E4M3 && q.vscale));
    }
    return e;
}

template <int DIM, bool E4M3>
hipError_t launch_tiles(const Attend& q, int tiles, hipStream_t s)
{
    switch (tiles) {
    case 1: return launch_attend<DIM, E4M3, 1>(q, s);
    case 2: return launch_attend<DIM, E4M3, 2>(q, s);
    case 3: return launch_attend<DIM, E4M3, 3>(q, s);
    }
    if constexpr (DIM == 256) return launch_attend<DIM, E4M3, 4>(q, s);
    else return tiles == 5 ? launch_attend<DIM, E4M3, 5>(q, s) : launch_attend<DIM, E4M3, 9>(q, s);
}

template <bool E4M3>
hipError_t launch_dim(const Attend& q, int tiles, hipStream_t s)
{
    switch (padded_dim(q.dim)) {
    case 64: return launch_tiles<64, E4M3>(q, tiles, s);
    case 128: return launch_tiles<128, E4M3>(q, tiles, s);
    default: return launch_tiles<256, E4M3>(q, tiles, s);
    }
}

// All that does not look at the buffers of the rows and the workspace.
int check_sizes(const spec_verify_config* cfg, const spec_verify_attend_args* a)
{
    int rc = sv::check_config(cfg);
    if (rc != SV_OK) return rc;
    if (!a) return SV_EINVAL;
    const spec_verify_kv& k = a->kv;
    if (k.type != SV_KV_BF16 && k.type != SV_KV_E4M3) return SV_EUNSUPPORTED;
    if (k.kv_heads < 1 || k.head_dim < 1 || a->heads < 1 || a->heads % k.kv_heads) return SV_EINVAL;
    if (k.kv_heads > 1024 || k.head_dim > SV_MAX_HEAD_DIM || k.head_dim % 16 || a->heads / k.kv_heads > 64) return SV_EUNSUPPORTED;
    const spec_verify_cache& c = a->cache;
    if (c.max_pages < 1 || c.page_size < 1 || (long long)c.max_pages * c.page_size > SV_MAX_CACHE_TOKENS) return SV_EINVAL;
    if (a->B < 0 || a->B > cfg->max_batch || a->rows < 1 || a->row0 < 0 || (long long)a->row0 + a->rows > cfg->max_draft + 1) return SV_EINVAL;
    if (a->window < 0 || a->max_len < 0 || a->max_len > SV_MAX_CACHE_TOKENS) return SV_EINVAL;
    return SV_OK;
}

} // namespace

extern "C" {

int64_t spec_verify_attend_workspace_bytes(const spec_verify_config* cfg, const spec_verify_attend_args* a)
{
    const int rc = check_sizes(cfg, a);
    if (rc != SV_OK) return rc;
    if (a->B == 0) return 0;
    const sv::AttendPlan p = plan_of(a);
    if (p.splits == 1) return 0;
    return (int64_t)a->B * a->kv.kv_heads * p.blocks * p.splits * p.tiles * 16 * (padded_dim(a->kv.head_dim) + 2) * 4;
}

int spec_verify_attend_check(const spec_verify_config* cfg, const spec_verify_attend_args* a)
{
    int rc = check_sizes(cfg, a);
    if (rc == SV_OK) rc = sv::check_cache(a->cache, false);
    if (rc == SV_OK) rc = sv::check_kv(a->kv);
    if (rc == SV_OK) rc = sv::check_rows(cfg, a->B, a->cache, a->slots, a->last_row, a->row_offsets);
    if (rc != SV_OK) return rc;
    if (!(fabsf(a->scale) <= FLT_MAX)) return SV_EINVAL;
    if (a->kv.token_stride > (1 << 28)) return SV_EUNSUPPORTED;
    if (a->B == 0) return SV_OK;
    if (!a->queries || !a->outputs) return SV_EINVAL;
    const int dim = a->kv.head_dim;
    if (a->query_row_stride < dim || a->query_head_stride < dim || a->output_row_stride < dim || a->output_head_stride < dim) return SV_EINVAL;
    if (!a->row_offsets && (a->query_batch_stride < 0 || a->output_batch_stride < 0)) return SV_EINVAL;
    const int64_t bytes = spec_verify_attend_workspace_bytes(cfg, a);
    if (bytes > 0 && (!a->workspace || (uintptr_t)a->workspace % 16 || a->workspace_bytes < bytes)) return SV_EINVAL;
    return SV_OK;
}

int spec_verify_attend(spec_verify_t* h, const spec_verify_attend_args* a, void* hip_stream)
{
    if (!h) return SV_EINVAL;
    const spec_verify_config* cfg = sv::handle_config(h);
    const int rc = spec_verify_attend_check(cfg, a);
    if (rc != SV_OK) return rc;
    DeviceGuard guard(cfg->device);
    hipStream_t s = (hipStream_t)hip_stream;
    hipError_t e = hipSuccess;
    if (a->device_status) e = launch_kernel(sv_attend_status_kernel, dim3(1), dim3(1), 0, s, nullptr, nullptr, a->device_status);
    if (e != hipSuccess) return SV_EDEVICE;
    if (a->B == 0) return SV_OK;
    const bool e4m3 = a->kv.type == SV_KV_E4M3;
    const int es = e4m3 ? 1 : 2;
    const sv::AttendPlan p = plan_of(a);
    Attend q;
    q.c = sv::cache_of(a->cache);
    q.r = sv::Rows{a->rows, a->row0, a->slots, a->last_row, (const long long*)a->row_offsets};
    q.b0 = 0;
    q.B = a->B;
    q.kv_heads = a->kv.kv_heads;
    q.group = a->heads / a->kv.kv_heads;
    q.dim = a->kv.head_dim;
    q.q = (const unsigned short*)a->queries;
    q.qb = a->query_batch_stride, q.qr = a->query_row_stride, q.qh = a->query_head_stride;
    q.out = (unsigned short*)a->outputs;
    q.ob = a->output_batch_stride, q.orow = a->output_row_stride, q.oh = a->output_head_stride;
    q.lse = a->lse;
    q.keys = (const char*)a->kv.keys;
    q.values = (const char*)a->kv.values;
    q.page_stride = a->kv.page_stride * es;
    q.head_stride = a->kv.head_stride * es;
    q.token_stride = (unsigned)(a->kv.token_stride * es);
    q.kscale = a->kv.key_scales;
    q.vscale = a->kv.value_scales;
    q.scale = a->scale;
    q.window = a->window;
    q.max_len = a->max_len ? a->max_len : a->cache.max_pages * a->cache.page_size;
    q.blocks = p.blocks;
    q.splits = p.splits;
    q.span = p.span;
    q.parts = (float*)a->workspace;
    q.status = a->device_status;
    e = e4m3 ? launch_dim<true>(q, p.tiles, s) : launch_dim<false>(q, p.tiles, s);
    return e == hipSuccess ? SV_OK : SV_EDEVICE;
}

} // extern "C"
