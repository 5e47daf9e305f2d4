// Attention of the rows of drafted blocks over the paged cache
// (spec_verify_attend in include/spec_verify.h, which states the formulas).

#include <float.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "spec_verify.h"
#include "sv_attend_plan.h"
#include "sv_cache.h"
#include "sv_host.h"

using sv::cache_status;
using sv::cache_uniform;
using sv::DeviceGuard;
using sv::kAttendBatch;
using sv::kAttendTokens;
using sv::kAttendUnit;
using sv::kAttendWaves;
using sv::launch_kernel;
using sv::lds_barrier;
using sv::Sequence;

namespace {

constexpr int kThreads = 64 * kAttendWaves;

constexpr float kRoom = 16.0f; // how far (in log2) a score may lie above its row's reference

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// A sequence that is cut, at the first share that does not begin it: its place in the launch
// (none: -1), the shares that have some of it, its rows, and whether the first of these
// shares has another sequence's piece in front.
struct Cut {
    int in, first, last, count;
    int second, unused;
    long long row;
};

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
    int blocks, shares, begin;
    struct Cut* cuts;           // [shares]: what the join of each has to know; null: no sequence is cut
    float* parts;               // [shares][kv_heads][blocks][2]: sums of a workgroup, then its (reference, sum) pairs
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

// The tokens that a sequence's rows see.
struct Reach {
    int low, end; // low: a multiple of the tile
};

__device__ __forceinline__ Reach reach_of(const Attend& q, const Sequence& s)
{
    Reach r;
    r.end = s.start + s.count;
    r.low = 0;
    if (q.window && s.start + 1 > q.window) r.low = (s.start + 1 - q.window) / kAttendTokens * kAttendTokens;
    return r;
}

// The sequence, with those marked bad that are longer than the caller said.
template <bool UNIFORM = true>
__device__ __forceinline__ Sequence sequence_within(const Attend& q, int b)
{
    Sequence s = sv::sequence_of<UNIFORM>(q.c, q.r, b);
    if (s.count > 0 && s.start + s.count > q.max_len) s.count = -1;
    return s;
}

// All sequences' units of tokens, one after the other, are cut into equal shares.  A
// sequence counts `begin` units more than it has, in front.  These are the units
// from .. to - 1 of a sequence that ends at `end`, after one that ends at `base`, in a
// share from lo to hi - 1 (from >= to: none).
struct Piece {
    int from, to;
};

__device__ __forceinline__ Piece piece_of(int begin, int base, int end, int lo, int hi)
{
    return Piece{max(0, max(lo, base) - base - begin), max(0, min(hi, end) - base - begin)};
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

// The kernel's arguments, in memory: the compiler does not know that they are the same at
// every call.
__device__ __forceinline__ const Attend* fresh_args()
{
    typedef const __attribute__((address_space(4))) char* Kernarg;
    Kernarg p = (Kernarg)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return (const Attend*)p;
}

// Attention of a block of rows over a share of the sequences' tokens.
//
// The scores of a tile of 16 tokens and 16 rows are K Q^T, so that a lane holds one
// row's scores of four tokens in each of two tiles; rounded, these are in place as
// the right operand of out^T = V^T P^T, whose left operand LDS reads transposed.  A
// row's maximum is not followed at every step: its reference stays as long as no
// score lies more than 16 (in log2) above it, which keeps the weights below 2^16 and
// spares the sums' rescaling (bf16 holds such weights as well as those below 1).  That
// is 519 us for the 596 of following it on 256 blocks of 17 rows.
//
// SHARED = false, for few rows: the four wavefronts take every fourth tile of 32 tokens,
// each through its own part of LDS and with registers one tile ahead, without a barrier
// until the end, where their sums are joined.
// SHARED = true, for many rows: each wavefront has rows of its own and they share a tile
// of 64 tokens (32 of more than 128 columns) in LDS, so that no sums are held twice.
//
// Bound by HBM where there are few rows, and by the 9 us that a launch's first sums take
// (arguments, slots, lengths, pages, keys, values, one after the other): one request of
// 131000 tokens 5.0 TB/s in 107 us, a token each of 64 requests, 282 MB, 4.0 TB/s in 70 (a
// large copy reaches 4.9, read and write).  With more rows, by both HBM and what a tile
// costs in matrix, vector and LDS instructions, which only partly overlap: 9 rows of 64
// requests, 292 MB in e4m3, 87 us; 17 rows of 256 requests, 1.9 GB and 242 GFLOP, 522 us.
// Spilled to scratch, read and written once a piece: 19 vector registers of <128, bf16, 3, rows
// split> (two of them read in the loop over tiles), 8 of <128, e4m3, 3, tokens split>, 18 of
// <256, e4m3, 1, tokens split>.
//
// Sequences are cut into equal shares rather than each into as many pieces: with lengths
// that differ the longest one no longer decides (the 64 requests' tokens 82 us for 90).
template <int DIM, bool E4M3, int TILES, bool SHARED>
__global__ __launch_bounds__(kThreads, sv::attend_at_once(DIM, E4M3, TILES, SHARED)) void sv_attend_kernel(Attend args)
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
    // Keys and values take turns in registers, each half a tile ahead, rather than both being one
    // tile ahead: a drafting step of bf16 71 us for 79.  In e4m3, whose loads are half as many,
    // the other way: a verify batch 99 us for 107.
    constexpr bool kHalves = !SHARED && !E4M3;
    // tiles whose queries stay in registers; the others' are in LDS
    constexpr int kQueryRegs = SHARED ? (DIM == 128 && TILES == 3 ? 1 : TILES) : TILES == 1 ? 1 : 0;
    constexpr int kQueryLds = TILES - kQueryRegs;
    constexpr int kMergeRow = DIM + 4;             // floats of a row where the sums meet
    constexpr int kStage = SHARED ? 2 * kTileBytes : kAttendWaves * kTileBytes;
    constexpr int kMerge = kAttendWaves * 16 * kMergeRow * 4;
    constexpr int kStride = SHARED ? kTile : kTile * kAttendWaves;
    __shared__ __attribute__((aligned(16))) char stage[kStage > kMerge ? kStage : kMerge];
    __shared__ u32x4 query[kQueryLds ? kQueryLds * kTeams * kSteps * 64 : 1];
    __shared__ int place[kRows];                   // position of each row
    __shared__ unsigned noted[kRows * kOut];       // infinities beside the sums: bit 2i of column i, bit 2i + 1 the negative one; both: NaN
    __shared__ float refs[kAttendWaves][16], sums[kAttendWaves][16];
    __shared__ int ends[kAttendBatch];
    __shared__ Sequence known[kAttendBatch];
    static_assert(kAttendBatch == kThreads, "a thread to each sequence");

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Consecutive workgroups go round the eight dies.  What reads the same tokens, or tokens
    // beside each other (row blocks, and key-value heads in one page), follows on one die.
    unsigned id = blockIdx.x / 8;
    const int block = (int)(id % args.blocks);
    id /= args.blocks;
    const int head = (int)(id % args.kv_heads);
    const int share = (int)(id / args.kv_heads * 8 + blockIdx.x % 8);
    if (share >= args.shares) return;

    // what each sequence has, and where its units end; a thread to each
    {
        int sum = 0;
        if ((int)threadIdx.x < args.B) {
            const Sequence s = sequence_within<false>(args, args.b0 + threadIdx.x);
            if (s.count < 0 && blockIdx.x == 0) cache_status(args.status, SV_STATUS_BAD_INPUT);
            if (s.count > 0) {
                const Reach reach = reach_of(args, s);
                sum = (reach.end - reach.low + kAttendUnit - 1) / kAttendUnit + args.begin;
            }
            known[threadIdx.x] = s;
        }
        int upto = sum;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int y = __shfl_up(upto, d);
            if (lane >= d) upto += y;
        }
        if (lane == 63) place[wave] = upto;
        lds_barrier();
        for (int w = 0; w < wave; ++w) upto += place[w];
        ends[threadIdx.x] = upto;
        lds_barrier();
    }
    const int total = ends[args.B - 1], width = (total + args.shares - 1) / args.shares;
    const int lo = share * width, hi = min(total, lo + width);
    int next = 0; // the first sequence that ends behind lo
    for (int n = args.B; n > 0;) {
        const int half = n / 2;
        if (ends[next + half] <= lo) next += half + 1, n -= half + 1;
        else n = half;
    }
    if (args.cuts && head == 0 && block == 0 && threadIdx.x == 0) {
        Cut cut = {-1};
        if (next < args.B) {
            const int base = next ? ends[next - 1] : 0, first = (base + args.begin) / width, last = (ends[next] - 1) / width;
            if (share == first + 1 && share <= last) cut = {next, first, last, known[next].count, base > first * width, 0, known[next].first};
        }
        args.cuts[share] = cut;
    }
    for (; next < args.B; ++next) {
    // What a piece needs is worked out anew for it: kept from piece to piece, it would take
    // the registers that the sums need.
    const Attend& q = *fresh_args();
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int n16 = lane & 15, g = lane >> 4;
    const int base = next ? __builtin_amdgcn_readfirstlane(ends[next - 1]) : 0, end = __builtin_amdgcn_readfirstlane(ends[next]);
    if (base >= hi) break;
    const Piece piece = piece_of(q.begin, base, end, lo, hi);
    if (piece.from >= piece.to) continue;
    const int b = q.b0 + next;
    Sequence s;
    s.slot = __builtin_amdgcn_readfirstlane(known[next].slot);
    s.count = __builtin_amdgcn_readfirstlane(known[next].count);
    s.start = __builtin_amdgcn_readfirstlane(known[next].start);
    s.first = known[next].first;
    const Reach reach = reach_of(q, s);
    const int row0 = block * kRows;                // first row (of a row and a head) of the workgroup
    const int rows = s.count * q.group - row0;     // and how many there are
    if (rows <= 0) continue;
    const int first = reach.low + piece.from * kAttendUnit, last = min(reach.low + piece.to * kAttendUnit, reach.end);
    lds_barrier(); // the piece before has left LDS
    // Tiles of rows.  SHARED: each wavefront has every fourth tile of as many as go round; one
    // tile that is left over is taken by all four in turn, 32 tokens each, two by two wavefronts
    // each, three by one each, as their last tile.  What is taken in turn is summed at the end.
    const int all_tiles = min(TILES * kTeams, (rows + 15) / 16);
    const int full = all_tiles / kTeams, left = all_tiles % kTeams;
    const int takers = left == 1 ? 4 : left == 2 ? 2 : 1;     // of a tile that is left over
    auto tile_of = [&](int i) { return SHARED ? (left && i == TILES - 1 ? full * kTeams + wave / takers : i * kTeams + wave) : i; };

    // the queries, negative for a negative scale, as right operands; rows past the last
    // are those of the last
    float scale = q.scale * 1.44269504088896340736f;
    if (E4M3 && q.kscale) scale *= cache_uniform(q.kscale + head);
    const unsigned flip = scale < 0 ? 0x80008000u : 0u;
    scale = fabsf(scale);
    // m / group, exactly: m + 0.5 lies at least 1 / 128 from a multiple, and m below 2^15
    const float by_group = 1.0f / q.group;
    auto row_of = [&](int m) { return (int)((m + 0.5f) * by_group); };
    for (int i = threadIdx.x; i < kRows * kOut; i += kThreads) noted[i] = 0;
    for (int i = threadIdx.x; i < kRows; i += kThreads) place[i] = s.start + row_of(min(i, rows - 1) + row0);

    // keys and values in LDS: a token's row of 16-byte chunks, their order changed from token
    // to token so that a column of 16 of them, and a pair of columns of 8, lie in different banks
    char* const kt = stage + (SHARED ? 0 : wave * kTileBytes);
    char* const vt = kTwo ? kt + kTileBytes : kt;
    auto turn_of = [](int t) { return ((DIM == 64 ? (t >> 1 & 3) * 2 : (t & 7) * 2) + (t >> 3 & 1)) * 16; };
    auto at = [&](int t, int chunk) { return t * DIM * 2 + ((chunk * 16) ^ turn_of(t)); };
    // the same for a place that is known (token t, bits of a chunk) away from a lane's own
    auto off = [&](int base, int t, int chunk) { return t * DIM * 2 + (base ^ (chunk * 16 ^ turn_of(t))); };
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
        lds_barrier();
    }
    const char* const keys = q.keys + head * q.head_stride;
    const char* const values = q.values + head * q.head_stride;
    // a lane's own places in LDS: where it writes, its first key and its first value
    const int write_at0 = at(loader / kLanes, loader % kLanes * (kUnit / 8));
    const int key_at0 = at(n16, g), value_at0 = at(g * 4 + n16 / 4, n16 % 4 / 2) + n16 % 2 * 8;
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
    float top[TILES], sum[TILES]; // top: a row's reference, a scaled score
#pragma unroll
    for (int i = 0; i < TILES; ++i) top[i] = -FLT_MAX, sum[i] = 0.0f;

    // What is asked for from memory comes behind all that other workgroups of the compute unit
    // have asked for: as few steps as can be.  First the pages of two tiles and the queries, ...
    int t0 = first + (SHARED ? 0 : wave * kTile);
    int page = pages_of(t0), next_page = pages_of(t0 + kStride); // of a token of the tile in hand and of the next
    auto query_at = [&](int tile, int step) {
        const int m = min(tile * 16 + n16, rows - 1) + row0;
        const int r = row_of(m), h = head * q.group + m - r * q.group;
        const unsigned short* from = q.q + (q.r.roff ? (s.first + r) * q.qr : b * q.qb + r * q.qr) + h * q.qh;
        const int d = step * 32 + g * 8;
        u32x4 x = {0, 0, 0, 0};
        if (d < q.dim) x = *(const u32x4_any*)(from + d);
        return x;
    };
    u32x4 qreg[kQueryRegs ? kQueryRegs : 1][kSteps];
#pragma unroll
    for (int i = 0; i < kQueryRegs; ++i)
#pragma unroll
        for (int k = 0; k < kSteps; ++k) qreg[i][k] = query_at(tile_of(i), k);
    // (a wavefront's own where rows are split, and else a share of all)
    constexpr int kQueryEach = SHARED ? kQueryLds * kSteps : (kQueryLds * kSteps + kAttendWaves - 1) / kAttendWaves;
    u32x4 qlds[kQueryEach ? kQueryEach : 1];
#pragma unroll
    for (int i = 0; i < kQueryEach; ++i) {
        const int k = SHARED ? i : min(i * kAttendWaves + wave, kQueryLds * kSteps - 1);
        qlds[i] = query_at(tile_of(kQueryRegs + k / kSteps), k % kSteps);
    }
    // ... then keys and values
    __builtin_amdgcn_sched_barrier(0);
    if (t0 < last) {
        load(kr, keys, t0, page);
        if constexpr (!kHalves) load(vr, values, t0, page);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kQueryRegs; ++i)
#pragma unroll
        for (int k = 0; k < kSteps; ++k) qreg[i][k] ^= flip;
#pragma unroll
    for (int i = 0; i < kQueryEach; ++i) {
        const int k = SHARED ? i * kTeams + wave : min(i * kAttendWaves + wave, kQueryLds * kSteps - 1);
        query[k * 64 + lane] = qlds[i] ^ flip;
    }
    lds_barrier(); // queries and places
    for (; t0 < last; t0 += kStride) {
        const bool more = t0 + kStride < last;
        // with many sums to hold, places in LDS are worked out anew rather than kept
        int key_at = key_at0, value_at = value_at0, write_at = write_at0;
        if constexpr (TILES > 1 || DIM == 256) asm volatile("" : "+v"(key_at), "+v"(value_at), "+v"(write_at));
        // asked for ahead of the next tile's keys and values, so that it is there when they are
        const int far_page = pages_of(t0 + 2 * kStride);
        __builtin_amdgcn_sched_barrier(0);
        const unsigned long long gone = __ballot(is_bad(page)); // tokens whose page is bad
        // (those in front of every row's window, in the first tile, may be)
        if (gone && is_bad(page) && (!q.window || t0 + (lane & (kTile - 1)) > s.start - q.window)) cache_status(q.status, SV_STATUS_BAD_INPUT);
        // some row does not see some token
        const bool mixed = t0 + kTile - 1 > s.start || gone || (q.window && t0 <= s.start + s.count - 1 - q.window);
        bool odd = false; // whether a value of a mixed tile is infinite or NaN
        auto store_keys = [&] {
            if (lane_in)
#pragma unroll
                for (int i = 0; i < kLoads; ++i)
#pragma unroll
                    for (int k = 0; k < kUnit / 8; ++k)
                        *(u32x4*)(kt + off(write_at, i * kPer, k)) = widen(kr[i], k);
            if constexpr (kHalves) load(vr, values, t0, page);
            else if (more) load(kr, keys, t0 + kStride, next_page);
        };
        auto store_values = [&] {
            if (lane_in)
#pragma unroll
                for (int i = 0; i < kLoads; ++i)
#pragma unroll
                    for (int k = 0; k < kUnit / 8; ++k) {
                        const u32x4 v = widen(vr[i], k);
                        if (mixed) odd |= special4(v);
                        *(u32x4*)(vt + off(write_at, i * kPer, k)) = v;
                    }
            if (more) {
                if constexpr (kHalves) load(kr, keys, t0 + kStride, next_page);
                else load(vr, values, t0 + kStride, next_page);
            }
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
                    u32x4* const here = (u32x4*)(vt + off(write_at, i * kPer, k));
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
            // whether these tokens count for the wavefront's last tile
            const bool last_too = left ? wave < left * takers && (t0 - first + in_tile) / kAttendTokens % takers == wave % takers : full == TILES;
            // scores, weights and sums of tiles from .. to - 1
            auto pass = [&](auto from, auto to) {
                f32x4 x[to - from][2] = {};
#pragma unroll
                for (int e = 0; e < kSteps; ++e) {
                    bf16x8 k[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) k[u] = *(const bf16x8*)(kt + off(key_at, in_tile + u * 16, e * 4));
#pragma unroll
                    for (int i = from; i < to; ++i) {
                        const bf16x8 y = __builtin_bit_cast(bf16x8, i < kQueryRegs ? qreg[i < kQueryRegs ? i : 0][e]
                                                                                   : query[(((i - kQueryRegs) * kSteps + e) * kTeams + (SHARED ? wave : 0)) * 64 + lane]);
#pragma unroll
                        for (int u = 0; u < 2; ++u) x[i - from][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[u], y, x[i - from][u], 0, 0, 0);
                    }
                }
                if constexpr (!SHARED) {
                    sync(); // the keys are read
                    store_values();
                    sync();
                    if (mixed) take_out();
                }
                // values of four tokens of each half, a column to each lane: tokens u * 16 + g * 4 + j
                auto value = [&](int e) {
                    s16x4 half[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        half[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(vt + off(value_at, in_tile + u * 16, 2 * e)));
                    const u32x2 lo = __builtin_bit_cast(u32x2, half[0]), hi = __builtin_bit_cast(u32x2, half[1]);
                    return __builtin_bit_cast(bf16x8, u32x4{lo[0], lo[1], hi[0], hi[1]});
                };
                bf16x8 p[to - from] = {};
#pragma unroll
                for (int i = from; i < to; ++i) {
                    if (i < TILES - 1 && i >= full) continue;
                    const f32x4* const y = x[i - from];
                    // w: how far the scores lie above the reference; those that are not seen at -infinity
                    float w[8], most;
                    auto above = [&] {
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] = fmaf(y[j / 4][j % 4], scale, -top[i]);
                        if (mixed) {
                            const int here = place[tile_of(i) * 16 + n16], low = q.window ? here - q.window : -1;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int in = in_tile + j / 4 * 16 + g * 4 + j % 4, t = t0 + in;
                                if ((t > here) | (t <= low) | (int)(gone >> in & 1)) w[j] = -INFINITY;
                            }
                        }
                        most = fmaxf(fmaxf(fmaxf(fmaxf(w[0], w[1]), w[2]), fmaxf(fmaxf(w[3], w[4]), w[5])), fmaxf(w[6], w[7]));
                    };
                    above();
                    if (__ballot(most > kRoom)) {
                        // (a row's own scores alone move its reference: what other rows see of a token
                        // that it does not see is not to change its last bits)
                        float high = fmaxf(most, __shfl_xor(most, 16));
                        high = fmaxf(high, __shfl_xor(high, 32));
                        most = -FLT_MAX;
#pragma unroll
                        for (int j = 0; j < 8; ++j) most = fmaxf(most, w[j] == -INFINITY ? -FLT_MAX : y[j / 4][j % 4] * scale);
                        most = fmaxf(most, __shfl_xor(most, 16));
                        most = fmaxf(most, __shfl_xor(most, 32));
                        most = high > kRoom ? fmaxf(most, top[i]) : top[i];
                        // (every lane takes part: sums that only some lanes change would be held twice)
                        const float factor = exp2_of(top[i] - most);
                        top[i] = most;
                        sum[i] *= factor;
#pragma unroll
                        for (int e = 0; e < kOut; ++e) acc[i][e] *= factor;
                        above();
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = exp2_of(w[j]);
                    sum[i] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
                    // rounded to bf16, as the matrix cores take them: half a step of 2^-8 each, as the
                    // outputs' own rounding is (both together are 0.0023 from 64 bits, in the root of the mean
                    // square relative to the outputs', the latter alone 0.0017; 0.0019 if the reference were the
                    // row's maximum, whose weight of 1 is exact)
                    p[i - from] = __builtin_bit_cast(bf16x8, u32x4{pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]), pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7])});
                }
                // out^T += V^T P^T
#pragma unroll
                for (int e = 0; e < kOut; ++e) {
                    const bf16x8 a = value(e);
#pragma unroll
                    for (int i = from; i < to; ++i) acc[i][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, p[i - from], acc[i][e], 0, 0, 0);
                }
            };
            constexpr std::integral_constant<int, 0> kFirst;
            constexpr std::integral_constant<int, TILES - 1> kLast;
            constexpr std::integral_constant<int, TILES> kEnd;
            if constexpr (SHARED) {
                if constexpr (TILES > 1) {
                    if (full) pass(kFirst, kLast);
                }
                // (left out where another wavefront takes it: weights of zero would make NaN of an infinity)
                if (last_too) pass(kLast, kEnd);
            } else {
                pass(kFirst, kEnd);
            }
        }
        sync(); // the tile is read
        page = next_page;
        next_page = far_page;
    }

    const float vscale = E4M3 && q.vscale ? cache_uniform(q.vscale + head) : 1.0f;
    const bool whole = piece.from == 0 && last == reach.end;
    float* const parts = q.parts + ((((long long)share * q.kv_heads + head) * q.blocks + block) * 2 + (base > lo)) * (kRows * (DIM + 2));
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
            const int row = row_of(m + row0), h = head * q.group + m + row0 - row * q.group;
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
            const int row = row_of(m + row0), h = head * q.group + m + row0 - row * q.group;
            const long long line = q.r.roff ? s.first + row : (long long)b * q.r.rows + row;
            q.lse[line * (q.kv_heads * q.group) + h] = all == 0.0f ? -INFINITY : (most + __builtin_amdgcn_logf(all)) * 0.69314718055994530942f;
        }
    };
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
        sum[i] += __shfl_xor(sum[i], 16);
        sum[i] += __shfl_xor(sum[i], 32);
    }
    // Where wavefronts have sums of the same rows, they meet in LDS: `takers` of them, from
    // wavefront `from` on, brought the same tile of the rows.
    float* const meet = (float*)stage;
    auto join = [&](int tile, int from, int takers) {
        const int r = threadIdx.x / 16, m = tile * 16 + r;
        float most = -FLT_MAX, all = 0.0f, factor[kAttendWaves];
#pragma unroll
        for (int w = 0; w < kAttendWaves; ++w)
            if (w < takers) most = fmaxf(most, refs[from + w][r]);
#pragma unroll
        for (int w = 0; w < kAttendWaves; ++w) {
            factor[w] = w < takers ? exp2_of(refs[from + w][r] - most) : 0.0f;
            if (w < takers) all += factor[w] * sums[from + w][r];
        }
        if (m >= rows) return;
#pragma unroll
        for (int e = 0; e < DIM / 64; ++e) {
            const int d = e * 64 + threadIdx.x % 16 * 4;
            f32x4 x = {};
#pragma unroll
            for (int w = 0; w < kAttendWaves; ++w)
                if (w < takers) x += factor[w] * *(const f32x4*)(meet + ((from + w) * 16 + r) * kMergeRow + d);
            put(m, d, x, all);
        }
        if (threadIdx.x % 16 == 0) put_sum(m, most, all);
    };
    // puts tile i of every wavefront there
    auto bring = [&](int i) {
        lds_barrier();
#pragma unroll
        for (int e = 0; e < kOut; ++e) *(f32x4*)(meet + (wave * 16 + n16) * kMergeRow + e * 16 + g * 4) = acc[i][e];
        if (g == 0) refs[wave][n16] = top[i], sums[wave][n16] = sum[i];
        lds_barrier();
    };
    if constexpr (SHARED) {
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            const int m = tile_of(i) * 16 + n16;
            if (i >= full || m >= rows) continue;
#pragma unroll
            for (int e = 0; e < kOut; ++e) put(m, e * 16 + g * 4, acc[i][e], sum[i]);
            if (g == 0) put_sum(m, top[i], sum[i]);
        }
        if (left) {
            bring(TILES - 1);
            for (int k = 0; k < left; ++k) join(full * kTeams + k, k * takers, takers);
        }
    } else {
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            if (i * 16 >= rows) break;
            bring(i);
            join(i, 0, kAttendWaves);
        }
    }
    }
}

// Joins the pieces of a row and head: DIM / 4 lanes hold its columns, `parts` such
// groups take every parts-th piece and meet in LDS.  There is a column of workgroups for
// each share but the first; it does the sequence that is cut there first.
// Bound by its chain of loads (what is cut, sums), kept short by asking for kAhead pieces at
// once: 4 us alone, 7 behind 64 requests of 9 rows, 18 (for 27 with a loop for the
// references and one for the sums) behind 256 of 17.
template <int DIM>
__global__ __launch_bounds__(kThreads) void sv_attend_join_kernel(Attend q, int rows, int parts)
{
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    constexpr int kLanes = DIM / 4, kAhead = 4;
    __shared__ f32x4 meet[kThreads];
    __shared__ float refs[kThreads / kLanes], sums[kThreads / kLanes];
    const i32x4* const from_cut = (const i32x4*)(q.cuts + blockIdx.y + 1);
    const i32x4 cut = cache_uniform(from_cut), more = cache_uniform(from_cut + 1);
    if (cut[0] < 0) return;
    const int b = q.b0 + cut[0], first = cut[1], last = cut[2], count = cut[3];
    const long long row0 = (long long)((unsigned long long)(unsigned)more[3] << 32 | (unsigned)more[2]);
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes, part = group % parts;
    const int heads = q.kv_heads * q.group, total = count * heads;
    const int each = kThreads / kLanes / parts; // rows of a workgroup
    if ((int)blockIdx.x * each >= total) return;
    const int at = min((int)blockIdx.x * each + group / parts, total - 1); // row of the sequence, over all heads
    const int head = at / (count * q.group), full = at % (count * q.group);
    const int block = full / rows, m = full % rows;
    const long long size = (long long)rows * (DIM + 2), step = size * 2 * q.blocks * q.kv_heads;
    const float* from = q.parts + ((long long)head * q.blocks + block) * 2 * size;
    float most = -FLT_MAX, all = 0.0f;
    f32x4 x = {};
    for (int i = first + part; i <= last; i += parts * kAhead) {
        float ref[kAhead], sum[kAhead];
        f32x4 y[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int n = i + k * parts;
            ref[k] = -FLT_MAX, sum[k] = 0.0f, y[k] = f32x4{};
            if (n > last) continue;
            const float* of = from + n * step + (n == first && more[0] ? size : 0);
            ref[k] = of[rows * DIM + 2 * m];
            sum[k] = of[rows * DIM + 2 * m + 1];
            y[k] = *(const f32x4*)(of + m * DIM + lane * 4);
        }
        float top = most;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) top = fmaxf(top, ref[k]);
        const float old = exp2_of(most - top);
        all *= old;
        x *= old;
        most = top;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const float factor = exp2_of(ref[k] - top);
            all += factor * sum[k];
            x += factor * y[k];
        }
    }
    if (parts > 1) {
        meet[threadIdx.x] = x;
        if (lane == 0) refs[group] = most, sums[group] = all;
        __syncthreads();
        const int group0 = group - part;
        for (int i = 0; i < parts; ++i) most = fmaxf(most, refs[group0 + i]);
        x = f32x4{};
        all = 0.0f;
        for (int i = 0; i < parts; ++i) {
            const float factor = exp2_of(refs[group0 + i] - most);
            all += factor * sums[group0 + i];
            x += factor * meet[(group0 + i) * kLanes + lane];
        }
        if (part) return;
    }
    if ((int)blockIdx.x * each + group / parts >= total) return;
    const int row = full / q.group, h = head * q.group + full % q.group, d = lane * 4;
    const float by = all == 0.0f ? 0.0f : (q.vscale ? q.vscale[head] : 1.0f) / all;
    const long long line = q.r.roff ? row0 + row : (long long)b * q.r.rows + row;
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
    return sv::attend_plan(a->B, a->kv.kv_heads, padded_dim(a->kv.head_dim), a->kv.type == SV_KV_E4M3, (long long)a->rows * (a->heads / a->kv.kv_heads), most_seen(a));
}

template <int DIM, bool E4M3, int TILES, bool SHARED>
hipError_t launch_attend(const Attend& q, int batch, hipStream_t s)
{
    const long long groups = (long long)(q.shares + 7) / 8 * 8 * q.kv_heads * q.blocks;
    // groups that join a row: half as many as a sequence has pieces if all have as many
    int parts = 1;
    while (parts * 2 <= kThreads / (DIM / 4) && parts * 2 < q.shares / std::min(q.B, batch)) parts *= 2;
    const int each = kThreads / (DIM / 4) / parts;
    const dim3 join((unsigned)(((long long)q.r.rows * q.kv_heads * q.group + each - 1) / each), (unsigned)(q.shares - 1));
    hipError_t e = hipSuccess;
    Attend a = q;
    for (a.b0 = 0; a.b0 < q.B && e == hipSuccess; a.b0 += batch) {
        a.B = std::min(q.B - a.b0, batch);
        e = launch_kernel(sv_attend_kernel<DIM, E4M3, TILES, SHARED>, dim3((unsigned)groups), dim3(kThreads), 0, s, nullptr, nullptr, a);
        if (!q.cuts || e != hipSuccess) continue;
        e = launch_kernel(sv_attend_join_kernel<DIM>, join, dim3(kThreads), 0, s, nullptr, nullptr, a, TILES * 16 * (SHARED ? kAttendWaves : 1), parts);
    }
    return e;
}

template <int DIM, bool E4M3>
hipError_t launch_tiles(const Attend& q, const sv::AttendPlan& p, hipStream_t s)
{
    constexpr int kSplit = DIM > 128 ? 1 : DIM / 64 + E4M3; // most tiles where tokens are split
    if (!p.shared) {
        if constexpr (kSplit >= 3) if (p.tiles == 3) return launch_attend<DIM, E4M3, 3, false>(q, p.batch, s);
        if constexpr (kSplit >= 2) if (p.tiles == 2) return launch_attend<DIM, E4M3, 2, false>(q, p.batch, s);
        return launch_attend<DIM, E4M3, 1, false>(q, p.batch, s);
    }
    if constexpr (DIM < 256) {
        if (p.tiles == 3) return launch_attend<DIM, E4M3, 3, true>(q, p.batch, s);
        if (p.tiles == 2) return launch_attend<DIM, E4M3, 2, true>(q, p.batch, s);
    }
    return launch_attend<DIM, E4M3, 1, true>(q, p.batch, s);
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

// Whether a sequence may be too long for one unit.
bool may_split(const spec_verify_attend_args* a) { return most_seen(a) > kAttendUnit; }

// Workspace for the pieces of sequences that are split; behind it, where they are cut.
int64_t parts_bytes(const spec_verify_attend_args* a, const sv::AttendPlan& p)
{
    return (int64_t)p.shares * a->kv.kv_heads * p.blocks * 2 * p.rows * (padded_dim(a->kv.head_dim) + 2) * 4;
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
    if ((long long)a->rows * a->heads > 1 << 23) return SV_EUNSUPPORTED; // the join's work-items stay within 32 bits
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
    if (!may_split(a)) return 0;
    return parts_bytes(a, p) + (int64_t)p.shares * sizeof(Cut);
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
    q.shares = p.shares;
    q.begin = p.begin;
    q.parts = (float*)a->workspace;
    q.cuts = may_split(a) ? (Cut*)((char*)a->workspace + parts_bytes(a, p)) : nullptr;
    q.status = a->device_status;
    e = e4m3 ? launch_dim<true>(q, p, s) : launch_dim<false>(q, p, s);
    return e == hipSuccess ? SV_OK : SV_EDEVICE;
}

} // extern "C"
