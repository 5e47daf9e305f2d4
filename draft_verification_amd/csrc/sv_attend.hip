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
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// A barrier for LDS alone: loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
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

// Whether one of eight bf16 is infinite or NaN.
__device__ __forceinline__ bool special4(u32x4 w)
{
    bool is = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) is |= ((w[j] & 0x7f80u) == 0x7f80u) | ((w[j] & 0x7f800000u) == 0x7f800000u);
    return is;
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
// score lies more than 16 (in log2) above it, which keeps the weights below 2^16 and
// spares the sums' rescaling (bf16 holds such weights as well as those below 1).
//
// SHARED = false, for few rows: the four wavefronts take every fourth tile of 32 tokens,
// each through its own part of LDS and with registers one tile ahead, without a barrier
// until the end, where their sums are joined.
// SHARED = true, for many rows: each wavefront has rows of its own and they share a tile
// of 64 tokens (32 of more than 128 columns) in LDS, so that no sums are held twice.
template <int DIM, bool E4M3, int TILES, bool SHARED>
__global__ __launch_bounds__(kThreads, SHARED ? 2 : DIM == 64 && TILES == 1 ? 4 : DIM < 256 ? 2 : 1) void sv_attend_kernel(Attend q)
{
    constexpr int kUnit = E4M3 ? 16 : 8;           // values of 16 bytes of the cache
    constexpr int kLanes = DIM / kUnit;            // lanes that read a token's row
    constexpr int kTile = SHARED && DIM < 256 ? 2 * kAttendTokens : kAttendTokens; // tokens in LDS at a time
    constexpr int kPer = (SHARED ? kThreads : 64) / kLanes; // tokens of a round of loads
    constexpr int kLoads = kTile / kPer;           // rounds of a tile, of keys and of values each
    constexpr int kSteps = DIM / 32;               // products of a score
    constexpr int kOut = DIM / 16;                 // tiles of a row of outputs
    constexpr int kTeams = SHARED ? kAttendWaves : 1; // wavefronts with rows of their own
    constexpr int kRows = TILES * 16 * kTeams;     // of the workgroup
    constexpr int kTileBytes = kTile * DIM * 2;
    constexpr bool kTwo = SHARED;                  // keys and values in LDS of their own
    // tiles whose queries stay in registers; the others' are in LDS
    constexpr int kQueryRegs = SHARED ? (DIM == 128 && TILES == 3 ? 1 : TILES) : TILES == 1 ? 1 : 0;
    constexpr int kQueryLds = TILES - kQueryRegs;
    constexpr int kMergeRow = DIM + 4;             // floats of a row where the sums meet
    constexpr int kStage = SHARED ? 2 * kTileBytes : kAttendWaves * kTileBytes;
    constexpr int kMerge = SHARED ? 0 : kAttendWaves * 16 * kMergeRow * 4;
    constexpr int kStride = SHARED ? kTile : kTile * kAttendWaves;
    __shared__ __attribute__((aligned(16))) char stage[kStage > kMerge ? kStage : kMerge];
    __shared__ u32x4 query[kQueryLds ? kQueryLds * kTeams * kSteps * 64 : 1];
    __shared__ int place[kRows];                   // position of each row
    __shared__ unsigned noted[kRows * kOut];       // infinities beside the sums: bit 2i of column i, bit 2i + 1 the negative one; both: NaN
    __shared__ float refs[kAttendWaves][SHARED ? 1 : kRows], sums[kAttendWaves][SHARED ? 1 : kRows];

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
    const int row0 = block * kRows;                // first row (of a row and a head) of the workgroup
    const int rows = s.count * q.group - row0;     // and how many there are
    if (rows <= 0) return;
    const int first = reach.low + split * q.span, last = min(first + q.span, reach.end);
    // tiles of the wavefront's rows (SHARED: every fourth), and how many there are
    auto tile_of = [&](int i) { return SHARED ? i * kAttendWaves + wave : i; };
    const int tiles = ((rows + 15) / 16 - (SHARED ? wave : 0) + kTeams - 1) / kTeams;

    // the queries, negative for a negative scale, as right operands; rows past the last
    // are those of the last
    float scale = q.scale * 1.44269504088896340736f;
    if (E4M3 && q.kscale) scale *= cache_uniform(q.kscale + head);
    const unsigned flip = scale < 0 ? 0x80008000u : 0u;
    scale = fabsf(scale);
    const float room = 16.0f / scale;              // how far a score may lie above its reference
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
    u32x4 qreg[kQueryRegs ? kQueryRegs : 1][kSteps];
#pragma unroll
    for (int i = 0; i < kQueryRegs; ++i)
#pragma unroll
        for (int k = 0; k < kSteps; ++k) qreg[i][k] = query_at(tile_of(i), k);
    for (int i = wave; i < kQueryLds * kTeams * kSteps; i += kAttendWaves)
        query[i * 64 + lane] = query_at(kQueryRegs * kTeams + i / kSteps, i % kSteps);
    for (int i = threadIdx.x; i < kRows * kOut; i += kThreads) noted[i] = 0;
    for (int i = threadIdx.x; i < kRows; i += kThreads) place[i] = s.start + (min(i, rows - 1) + row0) / q.group;

    // keys and values in LDS: a token's row of 16-byte chunks, their order changed from token
    // to token so that a column of them, or a pair of columns, lies in different banks
    char* const kt = stage + (SHARED ? 0 : wave * kTileBytes);
    char* const vt = kTwo ? kt + kTileBytes : kt;
    auto at = [](int t, int chunk) { return t * DIM * 2 + ((chunk ^ ((DIM == 64 ? t >> 1 : t) & (DIM < 128 ? 7 : 15))) * 16); };
    auto sync = [&] {
        if constexpr (SHARED) lds_barrier();
        else wave_sync();
    };

    const int* table = q.c.table + (long long)s.slot * q.c.max_pages;
    const int mask = (1 << q.c.shift) - 1;
    // which of a tile's tokens this lane loads in round 0, and which 16 bytes
    const int loader = SHARED ? threadIdx.x : lane;
    const bool lane_in = loader % kLanes * kUnit < q.dim;
    if (q.dim < DIM) { // columns past the head's size stay zero
        for (int i = threadIdx.x; i < kStage / 16; i += kThreads) ((u32x4*)stage)[i] = u32x4{0, 0, 0, 0};
        __syncthreads();
    }
    const char* const keys = q.keys + head * q.head_stride;
    const char* const values = q.values + head * q.head_stride;
    const unsigned in_row = lane_in ? loader % kLanes * 16 : 0;
    // a wavefront's load is 64 / kLanes tokens in a row, in one page if that has as many places
    const bool wide = (1 << q.c.shift) >= 64 / kLanes;
    const unsigned in_group = lane / kLanes * q.token_stride + in_row;

    // the pages of a tile's tokens, a token to a lane; those past the end are the last
    auto pages_of = [&](int t0) { return table[min(t0 + (lane & (kTile - 1)), reach.end - 1) >> q.c.shift]; };
    u32x4 kr[kLoads], vr[kLoads];
    auto is_bad = [&](int page) { return page < 0 || page >= q.c.n_pages; };
    auto load = [&](u32x4 (&x)[kLoads], const char* from, int t0, int page) { // of a bad page's tokens, the first page's
        if (is_bad(page)) page = 0;
        if (wide) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int t = i * kPer + (SHARED ? wave * (64 / kLanes) : 0);
                const char* group = from + __builtin_amdgcn_readlane(page, t) * q.page_stride + (long long)((t0 + t) & mask) * q.token_stride;
                x[i] = *(const u32x4*)(group + in_group);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int t = i * kPer + loader / kLanes;
                x[i] = *(const u32x4*)(from + __shfl(page, t) * q.page_stride + (unsigned)((t0 + t) & mask) * (unsigned long long)q.token_stride + in_row);
            }
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

    int t0 = first + (SHARED ? 0 : wave * kTile);
    int page = 0, next_page = 0; // of a token of the tile in hand and of the next
    if (t0 < last) {
        page = pages_of(t0);
        load(kr, keys, t0, page);
        load(vr, values, t0, page);
        next_page = pages_of(t0 + kStride);
    }
    __syncthreads(); // queries and places
    for (; t0 < last; t0 += kStride) {
        const bool more = t0 + kStride < last;
        // with many sums to hold, places in LDS are worked out anew rather than kept
        int lane_ = lane;
        if constexpr (TILES > 1) asm volatile("" : "+v"(lane_));
        const int n16 = lane_ & 15, g = lane_ >> 4;
        const int loader = SHARED ? wave * 64 + lane_ : lane_, in_load = loader / kLanes, unit = loader % kLanes;
        const unsigned long long gone = __ballot(is_bad(page)); // tokens whose page is bad
        if (gone && lane == 0) cache_status(q.status, SV_STATUS_BAD_INPUT);
        // some row does not see some token
        const bool mixed = t0 + kTile - 1 > s.start || gone || (q.window && t0 <= s.start + s.count - 1 - q.window);
        bool odd = false; // whether a value of a mixed tile is infinite or NaN
        auto store_keys = [&] {
            if (lane_in)
#pragma unroll
                for (int i = 0; i < kLoads; ++i)
#pragma unroll
                    for (int k = 0; k < kUnit / 8; ++k)
                        *(u32x4*)(kt + at(i * kPer + in_load, unit * (kUnit / 8) + k)) = widen(kr[i], k);
            if (more) load(kr, keys, t0 + kStride, next_page);
        };
        auto store_values = [&] {
            if (lane_in)
#pragma unroll
                for (int i = 0; i < kLoads; ++i)
#pragma unroll
                    for (int k = 0; k < kUnit / 8; ++k) {
                        const u32x4 v = widen(vr[i], k);
                        if (mixed) odd |= special4(v);
                        *(u32x4*)(vt + at(i * kPer + in_load, unit * (kUnit / 8) + k)) = v;
                    }
            if (more) load(vr, values, t0 + kStride, next_page);
        };
        // A weight of zero does not hide an infinity or a NaN from rows that do not see its
        // token.  Such values are noted for the rows that do, and taken as zero.
        auto take_out = [&] {
            if constexpr (SHARED) odd = __syncthreads_or(odd);
            else odd = __ballot(odd) != 0;
            if (!odd) return;
            for (int in = SHARED ? wave : 0; in < kTile && t0 + in < reach.end; in += SHARED ? kAttendWaves : 1) {
                const int t = t0 + in;
                if (gone >> in & 1) continue;
                for (int d = lane; d < q.dim; d += 64) {
                    const unsigned x = *(const unsigned short*)(vt + at(in, d / 8) + d % 8 * 2);
                    if ((x & 0x7f80u) != 0x7f80u) continue;
                    const unsigned kind = (x & 0x7fu ? 3u : x & 0x8000u ? 2u : 1u) << (d % 16 * 2);
                    for (int m = 0; m < rows && m < kRows; ++m)
                        if (t <= place[m] && (!q.window || t > place[m] - q.window)) atomicOr(&noted[m * kOut + d / 16], kind);
                }
            }
            sync();
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
#pragma unroll
                for (int k = 0; k < kUnit / 8; ++k) {
                    const int chunk = unit * (kUnit / 8) + k;
                    u32x4* const here = (u32x4*)(vt + at(i * kPer + in_load, chunk));
                    u32x4 v = *here;
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = without_special(v[j]);
                    *here = v;
                }
            sync();
        };
        store_keys();
        if constexpr (kTwo) store_values();
        sync();
        if (kTwo && mixed) take_out();
#pragma unroll
        for (int part = 0; part < kTile / kAttendTokens; ++part) { // 32 tokens at a time
            if (part && t0 + part * kAttendTokens >= last) break;
            const int in_tile = part * kAttendTokens;
            bf16x8 k[2][kSteps];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < kSteps; ++e) k[u][e] = *(const bf16x8*)(kt + at(in_tile + u * 16 + n16, e * 4 + g));
            u32x4 p[TILES] = {};
#pragma unroll
            for (int i = 0; i < TILES; ++i) {
                if (SHARED && i >= tiles) break;
                f32x4 x[2] = {};
#pragma unroll
                for (int e = 0; e < kSteps; ++e) {
                    const bf16x8 y = __builtin_bit_cast(bf16x8, i < kQueryRegs ? qreg[i < kQueryRegs ? i : 0][e]
                                                                               : query[((tile_of(i) - kQueryRegs * kTeams) * kSteps + e) * 64 + lane_]);
#pragma unroll
                    for (int u = 0; u < 2; ++u) x[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[u][e], y, x[u], 0, 0, 0);
                }
                unsigned hidden = 0; // bit u * 4 + j
                if (mixed) {
                    const int here = place[tile_of(i) * 16 + n16], low = q.window ? here - q.window : -1;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int in = in_tile + u * 16 + g * 4 + j, t = t0 + in;
                            if (t > here || t <= low || (gone >> in & 1)) {
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
                        // (every lane takes part: sums that only some lanes change would be held twice)
                        const float now = most > ref[i] ? most * scale : top[i], factor = exp2_of(top[i] - now);
                        ref[i] = most;
                        top[i] = now;
                        sum[i] *= factor;
#pragma unroll
                        for (int e = 0; e < kOut; ++e) acc[i][e] *= factor;
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
                if constexpr (TILES > 1) __builtin_amdgcn_sched_barrier(0); // one tile after the other, or their scores pile up and spill
            }
            if constexpr (!kTwo) {
                sync(); // the keys are read
                store_values();
                sync();
                if (mixed) take_out();
            }
#pragma unroll
            for (int e = 0; e < kOut; ++e) {
                // values of four tokens of each half, a column to each lane: tokens u * 16 + g * 4 + j
                s16x4 v[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = in_tile + u * 16 + g * 4 + n16 / 4;
                    v[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(vt + at(t, 2 * e + n16 % 4 / 2) + n16 % 2 * 8));
                }
                const u32x2 lo = __builtin_bit_cast(u32x2, v[0]), hi = __builtin_bit_cast(u32x2, v[1]);
                const bf16x8 a = __builtin_bit_cast(bf16x8, u32x4{lo[0], lo[1], hi[0], hi[1]});
#pragma unroll
                for (int i = 0; i < TILES; ++i)
                    acc[i][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, p[i]), acc[i][e], 0, 0, 0);
            }
        }
        sync(); // the tile is read
        page = next_page;
        if (more) next_page = pages_of(t0 + 2 * kStride);
    }

    const float vscale = E4M3 && q.vscale ? cache_uniform(q.vscale + head) : 1.0f;
    const bool whole = reach.splits == 1;
    float* const parts = q.parts + (((long long)b * q.kv_heads + head) * q.blocks + block) * ((long long)q.splits * (kRows * (DIM + 2)))
                       + (long long)split * (kRows * (DIM + 2));
    // stores four columns of row m of the workgroup, with what was noted for them
    auto put = [&](int m, int d, f32x4 x, float all) {
        const unsigned also = noted[m * kOut + d / 16] >> (d % 16 * 2) & 0xffu;
        if (also) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (also >> 2 * j & 1) x[j] += INFINITY;
                if (also >> 2 * j & 2) x[j] -= INFINITY;
            }
        }
        if (!whole) {
            *(f32x4*)(parts + m * DIM + d) = x;
        } else if (d < q.dim) {
            const int row = (m + row0) / q.group, h = head * q.group + (m + row0) % q.group;
            const float by = all == 0.0f ? 0.0f : vscale / all;
            unsigned short* to = q.out + (q.r.roff ? (s.first + row) * q.orow : b * q.ob + row * q.orow) + h * q.oh + d;
            *(u32x2_any*)to = u32x2{pack_bf16(x[0] * by, x[1] * by), pack_bf16(x[2] * by, x[3] * by)};
        }
    };
    auto put_sum = [&](int m, float most, float all) {
        if (!whole) {
            parts[kRows * DIM + 2 * m] = most;
            parts[kRows * DIM + 2 * m + 1] = all;
        } else if (q.lse) {
            const int row = (m + row0) / q.group, h = head * q.group + (m + row0) % q.group;
            const long long line = q.r.roff ? s.first + row : (long long)b * q.r.rows + row;
            q.lse[line * (q.kv_heads * q.group) + h] = all == 0.0f ? -INFINITY : (most + __builtin_amdgcn_logf(all)) * 0.69314718055994530942f;
        }
    };
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
        sum[i] += __shfl_xor(sum[i], 16);
        sum[i] += __shfl_xor(sum[i], 32);
    }
    if constexpr (SHARED) {
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            const int m = tile_of(i) * 16 + n16;
            if (m >= rows) continue;
#pragma unroll
            for (int e = 0; e < kOut; ++e) put(m, e * 16 + g * 4, acc[i][e], sum[i]);
            if (g == 0) put_sum(m, top[i], sum[i]);
        }
    } else {
        // the four wavefronts' sums, a tile of rows at a time
        float* const meet = (float*)stage;
        if (g == 0) {
#pragma unroll
            for (int i = 0; i < TILES; ++i) refs[wave][i * 16 + n16] = top[i], sums[wave][i * 16 + n16] = sum[i];
        }
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
#pragma unroll
            for (int e = 0; e < DIM / 64; ++e) {
                const int d = e * 64 + threadIdx.x % 16 * 4;
                f32x4 x = {};
#pragma unroll
                for (int w = 0; w < kAttendWaves; ++w) x += factor[w] * *(const f32x4*)(meet + (w * 16 + r) * kMergeRow + d);
                put(m, d, x, all);
            }
            if (threadIdx.x % 16 == 0) put_sum(m, most, all);
        }
    }
}

// Joins the splits of a row and head: DIM / 4 lanes hold its columns, `parts` such
// groups take every parts-th split and meet in LDS.
template <int DIM>
__global__ __launch_bounds__(kThreads) void sv_attend_join_kernel(Attend q, int rows, int parts)
{
    constexpr int kLanes = DIM / 4;
    __shared__ f32x4 meet[kThreads];
    __shared__ float refs[kThreads / kLanes], sums[kThreads / kLanes];
    const int b = q.b0 + blockIdx.y;
    const Sequence s = sequence_within(q, b);
    if (s.count <= 0) return;
    const Reach reach = reach_of(q, s);
    if (reach.splits <= 1) return;
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes, part = group % parts;
    const int heads = q.kv_heads * q.group, total = s.count * heads;
    const int each = kThreads / kLanes / parts; // rows of a workgroup
    if ((int)blockIdx.x * each >= total) return;
    const int at = min((int)blockIdx.x * each + group / parts, total - 1); // row of the sequence, over all heads
    const int head = at / (s.count * q.group), full = at % (s.count * q.group);
    const int block = full / rows, m = full % rows;
    const long long size = (long long)rows * (DIM + 2);
    const float* from = q.parts + (((long long)b * q.kv_heads + head) * q.blocks + block) * q.splits * size;
    const float* pairs = from + rows * DIM + 2 * m;
    float most = -FLT_MAX, all = 0.0f;
#pragma unroll 4
    for (int i = part; i < reach.splits; i += parts) most = fmaxf(most, pairs[i * size]);
    f32x4 x = {};
#pragma unroll 4
    for (int i = part; i < reach.splits; i += parts) {
        const float factor = exp2_of(pairs[i * size] - most);
        all += factor * pairs[i * size + 1];
        x += factor * *(const f32x4*)(from + i * size + m * DIM + lane * 4);
    }
    if (parts > 1) {
        meet[threadIdx.x] = x;
        if (lane == 0) refs[group] = most, sums[group] = all;
        __syncthreads();
        const int first = group - part;
        for (int i = 0; i < parts; ++i) most = fmaxf(most, refs[first + i]);
        x = f32x4{};
        all = 0.0f;
        for (int i = 0; i < parts; ++i) {
            const float factor = exp2_of(refs[first + i] - most);
            all += factor * sums[first + i];
            x += factor * meet[(first + i) * kLanes + lane];
        }
        if (part) return;
    }
    if ((int)blockIdx.x * each + group / parts >= total) return;
    const int row = full / q.group, h = head * q.group + full % q.group, d = lane * 4;
    const float by = all == 0.0f ? 0.0f : (q.vscale ? q.vscale[head] : 1.0f) / all;
    const long long line = q.r.roff ? s.first + row : (long long)b * q.r.rows + row;
    unsigned short* to = q.out + (q.r.roff ? line * q.orow : b * q.ob + row * q.orow) + h * q.oh + d;
    if (d < q.dim) *(u32x2_any*)to = u32x2{pack_bf16(x[0] * by, x[1] * by), pack_bf16(x[2] * by, x[3] * by)};
    if (q.lse && lane == 0) q.lse[line * heads + h] = all == 0.0f ? -INFINITY : (most + __builtin_amdgcn_logf(all)) * 0.69314718055994530942f;
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

template <int DIM, bool E4M3, int TILES, bool SHARED>
hipError_t launch_attend(const Attend& q, hipStream_t s)
{
    constexpr int kMost = 0x7fffffff / kThreads; // workgroups of a launch, and more than enough
    int parts = 1; // groups that join a row: half as many as it has splits
    while (parts * 2 <= kThreads / (DIM / 4) && parts * 2 < q.splits) parts *= 2;
    const int each = kThreads / (DIM / 4) / parts;
    const unsigned join = (unsigned)(((long long)q.r.rows * q.kv_heads * q.group + each - 1) / each);
    const long long per = std::max<long long>((long long)q.kv_heads * q.blocks * q.splits, join);
    const int step = (int)std::max(1ll, std::min<long long>(65535, (kMost - 8 * q.blocks) / per));
    hipError_t e = hipSuccess;
    Attend a = q;
    for (a.b0 = 0; a.b0 < q.B && e == hipSuccess; a.b0 += step) {
        a.B = std::min(q.B - a.b0, step);
        long long groups = (long long)a.B * q.kv_heads * q.splits;
        if (q.blocks > 1) groups = (groups + 7) / 8 * 8 * q.blocks;
        e = launch_kernel(sv_attend_kernel<DIM, E4M3, TILES, SHARED>, dim3((unsigned)groups), dim3(kThreads), 0, s, nullptr, nullptr, a);
        if (q.splits == 1 || e != hipSuccess) continue;
        e = launch_kernel(sv_attend_join_kernel<DIM>, dim3(join, (unsigned)a.B), dim3(kThreads), 0, s, nullptr, nullptr, a,
                          TILES * 16 * (SHARED ? kAttendWaves : 1), parts);
    }
    return e;
}

template <int DIM, bool E4M3>
hipError_t launch_tiles(const Attend& q, const sv::AttendPlan& p, hipStream_t s)
{
    if (!p.shared) {
        if constexpr (DIM < 256)
            if (p.tiles == 2) return launch_attend<DIM, E4M3, 2, false>(q, s);
        return launch_attend<DIM, E4M3, 1, false>(q, s);
    }
    if constexpr (DIM < 256) {
        if (p.tiles == 3) return launch_attend<DIM, E4M3, 3, true>(q, s);
        if (p.tiles == 2) return launch_attend<DIM, E4M3, 2, true>(q, s);
    }
    return launch_attend<DIM, E4M3, 1, true>(q, s);
}

template <bool E4M3>
hipError_t launch_dim(const Attend& q, const sv::AttendPlan& p, hipStream_t s)
{
    switch (padded_dim(q.dim)) {
    case 64: return launch_tiles<64, E4M3>(q, p, s);
    case 128: return launch_tiles<128, E4M3>(q, p, s);
    default: return launch_tiles<256, E4M3>(q, p, s);
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
    return (int64_t)a->B * a->kv.kv_heads * p.blocks * p.splits * p.rows * (padded_dim(a->kv.head_dim) + 2) * 4;
}

int spec_verify_attend_check(const spec_verify_config* cfg, const spec_verify_attend_args* a)
{
    int rc = check_sizes(cfg, a);
    if (rc == SV_OK) rc = sv::check_cache(a->cache, false);
    if (rc == SV_OK) rc = sv::check_kv(a->kv);
    if (rc == SV_OK) rc = sv::check_rows(cfg, a->B, a->cache, a->slots, a->last_row, a->row_offsets);
    if (rc != SV_OK) return rc;
    if (!(fabsf(a->scale) <= FLT_MAX)) return SV_EINVAL;
    if (a->kv.token_stride > (1 << 26)) return SV_EUNSUPPORTED; // 16 tokens of 2 bytes within 32 bits
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
    q.kscale = e4m3 ? a->kv.key_scales : nullptr;
    q.vscale = e4m3 ? a->kv.value_scales : nullptr;
    q.scale = a->scale;
    q.window = a->window;
    q.max_len = a->max_len ? a->max_len : a->cache.max_pages * a->cache.page_size;
    q.blocks = p.blocks;
    q.splits = p.splits;
    q.span = p.span;
    q.parts = (float*)a->workspace;
    q.status = a->device_status;
    e = e4m3 ? launch_dim<true>(q, p, s) : launch_dim<false>(q, p, s);
    return e == hipSuccess ? SV_OK : SV_EDEVICE;
}

} // extern "C"
