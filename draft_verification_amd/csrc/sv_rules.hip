// Rules on logits around verification, and the token history they read
// (spec_verify_process and spec_verify_history in include/spec_verify.h, which
// states the formulas).

#include <math.h>

#include <algorithm>

#include "spec_verify.h"
#include "sv_host.h"

using sv::DeviceGuard;
using sv::launch_kernel;

namespace {

constexpr int kThreads = 256; // 4 wavefronts of 64

struct Rules {
    int B, rows, row0, V, words;
    const void* in;
    long long ibs, irs;
    void* out;
    long long obs, ors;
    const long long* roff;
    const int* vlen;
    const int* draft;
    long long dstride;
    const int* counts;
    const unsigned* seen;
    int n_slots;
    const int* slots;
    const float* rep;
    const float* freq;
    const float* pres;
    const int* boff;
    const int* btok;
    const float* bval;
    int n_biases;
    const unsigned* masks;
    long long mstride;
    int n_masks;
    const int* midx;
    int* live;
    int* status;
    int b0;    // first sequence of the launch
    int chunk; // rows of a workgroup
};

__device__ __forceinline__ void bad_input(int* status)
{
    if (status) __hip_atomic_fetch_or(status, SV_STATUS_BAD_INPUT, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A value that every lane reads alike and no kernel of the call writes, through
// the scalar cache.
template <typename T>
__device__ __forceinline__ T uniform(const T* p)
{
    return *(const __attribute__((address_space(4))) T*)(uintptr_t)p;
}

// First row and number of rows that the call processes of sequence b; a
// negative count marks a bad one.
__device__ __forceinline__ int rows_of(const Rules& q, int b, long long& first)
{
    if (q.roff) {
        first = uniform(q.roff + b);
        const long long end = uniform(q.roff + b + 1);
        return first < 0 || end < first || end - first > q.rows ? -1 : (int)(end - first);
    }
    first = 0;
    if (!q.vlen) return q.rows;
    const int L = uniform(q.vlen + b);
    if (L < 0) return -1;
    return L < q.row0 ? 0 : (L - q.row0 < q.rows ? L - q.row0 + 1 : q.rows);
}

// Start values of the outputs that the workgroups of the call add to: the
// status word, and the live counts (0 for a row that has a mask, else -1).
__global__ __launch_bounds__(kThreads) void sv_rules_start_kernel(Rules q)
{
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i == 0 && q.status) *q.status = 0;
    if (!q.live || i >= (long long)q.B * q.rows) return;
    int live = -1;
    if (q.masks && q.midx[i] != -1) {
        const int b = (int)(i / q.rows), r = (int)(i % q.rows);
        if (q.roff) {
            const long long first = q.roff[b], end = q.roff[b + 1];
            if (first >= 0 && end >= first && end - first <= q.rows && r < end - first) live = 0;
        } else if (!q.vlen || q.row0 + r <= q.vlen[b]) {
            live = 0;
        }
    }
    q.live[i] = live;
}

__global__ void sv_status_clear_kernel(int* status) { *status = 0; }

// Logits in memory, PT of them to a lane (16 bytes).  The vector types ask for
// the element's alignment only: rows of odd lengths start anywhere.
template <int DT>
struct Vec;

template <>
struct Vec<SV_BF16> {
    typedef unsigned short elem;
    typedef unsigned short raw __attribute__((ext_vector_type(8), aligned(2)));
    static constexpr int PT = 8;
    static __device__ float get(elem x) { return __uint_as_float((unsigned)x << 16); }
    static __device__ elem put(float x) { return __builtin_bit_cast(elem, (__bf16)x); }
    static __device__ elem none() { return 0xff80; } // -infinity

    // -infinity where the bit is 0, two tokens at a time.
    static __device__ __forceinline__ void mask(raw& x, unsigned bits)
    {
        typedef unsigned pairs __attribute__((ext_vector_type(4)));
        pairs p = __builtin_bit_cast(pairs, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned lo = (unsigned)__builtin_amdgcn_sbfe((int)bits, 2 * i, 1), hi = (unsigned)__builtin_amdgcn_sbfe((int)bits, 2 * i + 1, 1);
            const unsigned keep = (lo & 0xffffu) | (hi & 0xffff0000u);
            p[i] = (p[i] & keep) | (0xff80ff80u & ~keep);
        }
        x = __builtin_bit_cast(raw, p);
    }

    // Whether a token is infinite or NaN.
    static __device__ __forceinline__ bool special(const raw& x)
    {
        typedef unsigned short two __attribute__((ext_vector_type(2)));
        typedef unsigned pairs __attribute__((ext_vector_type(4)));
        const pairs p = __builtin_bit_cast(pairs, x) & 0x7fff7fffu;
        two m = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned one = p[i];
            m = __builtin_elementwise_max(m, __builtin_bit_cast(two, one));
        }
        return m[0] >= 0x7f80 || m[1] >= 0x7f80;
    }
};

// The sum of a value over a wavefront's lanes.
__device__ __forceinline__ int wave_total(int v)
{
#define SV_ADD(ctrl, rows) v += __builtin_amdgcn_update_dpp(0, v, ctrl, rows, 0xf, false)
    SV_ADD(0x111, 0xf); // row shifts by 1, 2, 4, 8
    SV_ADD(0x112, 0xf);
    SV_ADD(0x114, 0xf);
    SV_ADD(0x118, 0xf);
    SV_ADD(0x142, 0xa); // row 0's and 2's last lane to the next row
    SV_ADD(0x143, 0xc); // the first half's last lane to the second
#undef SV_ADD
    return __builtin_amdgcn_readlane(v, 63);
}

template <>
struct Vec<SV_F32> {
    typedef float elem;
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
    static constexpr int PT = 4;
    static __device__ float get(elem x) { return x; }
    static __device__ elem put(float x) { return x; }
    static __device__ elem none() { return -INFINITY; }
    static __device__ __forceinline__ void mask(raw& x, unsigned bits)
    {
#pragma unroll
        for (int k = 0; k < PT; ++k) x[k] = bits >> k & 1 ? x[k] : -INFINITY;
    }
    static __device__ __forceinline__ bool special(const raw& x)
    {
        bool any = false;
#pragma unroll
        for (int k = 0; k < PT; ++k) any |= !(fabsf(x[k]) < INFINITY);
        return any;
    }
};

// A lane's PT bits of a bit row, from token v0 (a multiple of PT).
template <int PT>
__device__ __forceinline__ unsigned bits_at(const unsigned* row, int v0)
{
    const unsigned byte = ((const unsigned char*)row)[v0 >> 3];
    return PT == 8 ? byte : (byte >> (v0 & 4)) & 15u;
}

// A lane's PT logits; past the row's end they read as -infinity.  Stores are
// non-temporal, and loads too where the rows are copied (4352 rows of 129280
// bf16: 450 us, with other loads 465, with neither 474); in place the loaded
// lines are written in part, and stay for that (1360 masked rows of 50264: 42
// us, with non-temporal loads 61).
template <int DT, bool INPLACE>
__device__ __forceinline__ typename Vec<DT>::raw load_logits(const typename Vec<DT>::elem* p, int v0, int V)
{
    typedef Vec<DT> X;
    if (v0 + X::PT <= V) return INPLACE ? *(const typename X::raw*)p : __builtin_nontemporal_load((const typename X::raw*)p);
    typename X::raw x;
#pragma unroll
    for (int k = 0; k < X::PT; ++k) x[k] = v0 + k < V ? p[k] : X::none();
    return x;
}

template <int DT>
__device__ __forceinline__ void store_logits(typename Vec<DT>::elem* p, typename Vec<DT>::raw x, int v0, int V)
{
    typedef Vec<DT> X;
    if (v0 + X::PT <= V) {
        __builtin_nontemporal_store(x, (typename X::raw*)p);
        return;
    }
#pragma unroll
    for (int k = 0; k < X::PT; ++k)
        if (v0 + k < V) p[k] = x[k];
}

// Orders a wavefront's LDS accesses among its own lanes (they execute in
// order; this keeps the compiler to it).
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// One workgroup per (sequence, chunk of its rows, block of 256 PT tokens); each
// of its wavefronts works alone on SPAN = 64 PT consecutive tokens, a lane on
// PT of them, whose seen and mask bits are one byte or half a byte.
//
// A history marks a few percent of the vocabulary.  So a row is a plain copy,
// bound by HBM, and the marked tokens are listed: the wavefront keeps the list
// of its tokens that any row of the chunk touches, with their counts and
// biases, in LDS, passes the row's 1 KB through LDS, and lane p changes the
// p-th listed token there.  (Every lane computing its own PT tokens instead
// costs 20 vector instructions a token, about what the chip can issue in the
// time HBM takes: 737 us at B = 256, 17 rows, V = 129280 bf16 where this takes
// 450, 5.0 TB/s.)  The next row adds one drafted token to the counts.  kAhead
// rows are in flight, and the first are asked for before the rules are read.
constexpr int kAhead = 2;

template <int DT>
struct Listed {
    static constexpr int SPAN = 64 * Vec<DT>::PT;
    typename Vec<DT>::elem row[SPAN]; // the row's logits
    int cnt[SPAN];                    // 1 + count of a seen token, 0 for one not seen (yet)
    float bias[SPAN];
    unsigned short at[SPAN];          // the touched tokens, ascending
};

// Element i of an array that may not be given.  The load is unconditional, so
// that several of them are under way together.
struct Given {
    const char* any = (const char*)__builtin_amdgcn_kernarg_segment_ptr();
    template <typename T>
    __device__ __forceinline__ T operator()(const T* p, long long i, T otherwise) const
    {
        const T v = uniform(p ? p + i : (const T*)any);
        return p ? v : otherwise;
    }
};

// What the wavefronts of a workgroup have left alive of its rows.
struct Tally {
    int live[64]; // of row r0 + i
    int done;     // wavefronts that have added theirs
};

// RULES: a history, drafted tokens or biases are given; without them only masks
// are applied, and neither the lists nor their LDS are there.
template <int DT, bool INPLACE, bool RULES>
__device__ __forceinline__ void process_block(const Rules& q, Listed<DT>& s, Tally& t)
{
    typedef Vec<DT> X;
    typedef typename X::elem elem;
    typedef typename X::raw raw;
    constexpr int PT = X::PT;
    constexpr int SPAN = 64 * PT; // tokens of a wavefront
    constexpr unsigned ALL = (1u << PT) - 1;
    const int blk = blockIdx.x, r0 = blockIdx.y * q.chunk, b = q.b0 + blockIdx.z;
    const int lane = threadIdx.x & 63;
    const int w0 = (blk * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * SPAN; // the wavefront's first token
    const int v0 = w0 + lane * PT;
    if (w0 >= q.V) return;
    const bool inside = v0 < q.V;
    const bool teller = w0 == 0;         // the wavefront that reports what the sequence brings
    const bool tells = teller && lane == 0;

    // What the sequence brings, asked for all at once (an array that is not
    // given reads the kernel's arguments, and its value is not used): a call of
    // one row takes as long as its chain of dependent loads.
    const Given give;
    long long first;
    const int n = rows_of(q, b, first);
    const int given_slot = RULES ? give(q.slots, b, b) : -1;
    float rep = 1.0f, freq = 0.0f, pres = 0.0f; // without history or drafted tokens only looked at for their range
    if (RULES || teller) rep = give(q.rep, b, 1.0f), freq = give(q.freq, b, 0.0f), pres = give(q.pres, b, 0.0f);
    int e0 = RULES ? give(q.boff, b, 0) : 0, e1 = RULES ? give(q.boff, b + 1, 0) : 0;
    const int far = min(q.chunk, q.rows - r0); // rows of the chunk, if the sequence has them all
    int my_mask = -1, my_draft = -1, draft0 = -1;
    if (q.masks && lane < far) my_mask = q.midx[(long long)b * q.rows + r0 + lane];
    const int* draft = q.draft + b * q.dstride;
    if (RULES && q.draft && lane + 1 < far) my_draft = draft[q.row0 + r0 + lane]; // between row lane and the next
    if (RULES && q.draft && lane < q.row0 + r0 + far - 1) draft0 = draft[lane];

    if (tells && r0 == 0 && n < 0) bad_input(q.status);
    if (r0 >= n) return;
    const int r1 = min(r0 + q.chunk, n); // at most 64 rows: a lane's share of what each row brings
    if (r0 + lane >= r1) my_mask = -1;
    if (r0 + lane + 1 >= r1) my_draft = -1;
    int slot = q.counts ? given_slot : -1;
    const bool slot_ok = slot >= -1 && slot < q.n_slots;
    const bool rep_ok = rep >= 0x1p-126f && rep < INFINITY, freq_ok = fabsf(freq) < INFINITY, pres_ok = fabsf(pres) < INFINITY;
    const bool bias_ok = e0 >= 0 && e0 <= e1 && e1 <= q.n_biases;
    if (tells && !((slot_ok || !q.counts) && rep_ok && freq_ok && pres_ok && (bias_ok || !q.boff))) bad_input(q.status);
    if (teller && q.masks && (my_mask < -1 || my_mask >= q.n_masks)) bad_input(q.status);
    if (!slot_ok) slot = -1;
    if (!rep_ok) rep = 1.0f;
    if (!freq_ok) freq = 0.0f;
    if (!pres_ok) pres = 0.0f;
    if (!bias_ok) e0 = e1 = 0;

    const elem* src = (const elem*)q.in + (q.roff ? (first + r0) * q.irs : b * q.ibs + r0 * q.irs) + v0;
    elem* dst = (elem*)q.out + (q.roff ? (first + r0) * q.ors : b * q.obs + r0 * q.ors) + w0;

    // rows in flight: slot u holds row r0 + u, then r0 + u + kAhead, ...; its
    // mask bits are asked for one turn of the slots earlier than its logits
    raw x[kAhead];
    unsigned allow[kAhead], allow_next[kAhead];
    auto fetch = [&](int i, raw& xr) {
        if (r0 + i < r1 && inside) xr = load_logits<DT, INPLACE>(src + i * q.irs, v0, q.V);
    };
    unsigned mine = 0; // the lane's touched tokens
    if (slot >= 0 && inside) mine = bits_at<PT>(q.seen + (long long)slot * q.words, v0);
    int bias_tok = -1;
    float bias_val = 0.0f;
    if (lane < e1 - e0) { // (e0 + lane may be past 2^31 - 1)
        bias_tok = q.btok[e0 + lane];
        bias_val = q.bval[e0 + lane];
    }
    auto mask_of = [&](int i) { return __builtin_amdgcn_readlane(my_mask, i); }; // of row r0 + i, i < 64
    auto fetch_mask = [&](int i, unsigned& al) {
        al = ALL;
        if (r0 + i >= r1) return;
        const int m = mask_of(i);
        if (m == -1) return;
        al = 0; // of an index out of range
        if (m >= 0 && m < q.n_masks && inside) al = bits_at<PT>(q.masks + m * q.mstride, v0);
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch_mask(u, allow[u]);
    if (!INPLACE) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) fetch(u, x[u]);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch_mask(u + kAhead, allow_next[u]);

    const int j0 = RULES && q.draft ? q.row0 + r0 : 0, j1 = RULES && q.draft ? q.row0 + r1 - 1 : 0;
    auto add_draft = [&](int y) { // counts token w0 + y once more
        if (lane == 0) {
            const int c = s.cnt[y];
            s.cnt[y] = c ? c + 1 : 2;
        }
    };
    int listed = 0; // tokens that any row of the chunk touches
    if (RULES && (slot >= 0 || j1 > 0 || e0 < e1)) {
        // history
        if (v0 + PT > q.V) mine &= inside ? (1u << (q.V - v0)) - 1 : 0u;
        {
            typedef int four __attribute__((ext_vector_type(4), aligned(4)));
            const int* c = q.counts + (long long)slot * q.V + v0;
            four count[PT / 4] = {};
            if (mine && v0 + PT <= q.V) {
#pragma unroll
                for (int k = 0; k < PT / 4; ++k) count[k] = ((const four*)c)[k];
            } else if (mine) {
#pragma unroll
                for (int k = 0; k < PT; ++k)
                    if (mine >> k & 1) count[k / 4][k % 4] = c[k];
            }
#pragma unroll
            for (int k = 0; k < PT; ++k) {
                s.cnt[lane * PT + k] = mine >> k & 1 ? 1 + count[k / 4][k % 4] : 0;
                s.bias[lane * PT + k] = 0.0f;
            }
        }
        wave_sync();
        // drafted tokens, 64 ids at a time, those of the wavefront's span one by
        // one: the first j0 precede the chunk's first row, the others a later one
        for (int i0 = 0; i0 < j1; i0 += 64) {
            const int i = i0 + lane;
            const int x = i0 == 0 ? draft0 : i < j1 ? draft[i] : -1;
            const bool fine = (unsigned)x < (unsigned)q.V;
            if (teller && i < j1 && !fine) bad_input(q.status);
            unsigned long long hit = __ballot(i < j1 && fine && (unsigned)(x - w0) < (unsigned)SPAN);
            while (hit) {
                const int src = __builtin_ctzll(hit);
                hit &= hit - 1;
                const int y = __builtin_amdgcn_readlane(x, src) - w0;
                if (y / PT == lane) mine |= 1u << (y % PT);
                if (i0 + src < j0) add_draft(y);
            }
        }
        // biases, likewise, added in the list's order
        for (int left = e1 - e0; left > 0; left -= 64) {
            const int x = bias_tok;
            const float val = bias_val;
            if (lane < left - 64) {
                bias_tok = q.btok[e1 - left + 64 + lane];
                bias_val = q.bval[e1 - left + 64 + lane];
            }
            const bool fine = (unsigned)x < (unsigned)q.V;
            if (teller && lane < left && !fine) bad_input(q.status);
            unsigned long long hit = __ballot(lane < left && fine && (unsigned)(x - w0) < (unsigned)SPAN);
            while (hit) {
                const int src = __builtin_ctzll(hit);
                hit &= hit - 1;
                const int y = __builtin_amdgcn_readlane(x, src) - w0;
                const float add = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(val), src));
                if (y / PT == lane) mine |= 1u << (y % PT);
                if (lane == 0) s.bias[y] += add;
            }
        }
        // the list, in the order of the lanes
        int at = 0;
#pragma unroll
        for (int k = 0; k < PT; ++k) {
            const unsigned long long has = __ballot(mine >> k & 1);
            listed += __popcll(has);
            at += __builtin_amdgcn_mbcnt_hi((unsigned)(has >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)has, 0));
        }
        for (unsigned m = mine; m; m &= m - 1) s.at[at++] = (unsigned short)(lane * PT + __builtin_ctz(m));
        wave_sync();
    }

    const float inv = 1.0f / rep;
    auto apply = [&](float l, int y) { // the rules for token w0 + y
        const int c = s.cnt[y];
        // l / rep: the product with 1 / rep, corrected by its remainder (a division
        // in full: 464 us for the 456 of 4352 rows of 129280 bf16)
        const float d = l * inv;
        const float e = fmaf(fmaf(-d, rep, l), inv, d);
        if (c) l = l > 0.0f ? (d < INFINITY ? e : d) : l * rep;
        l -= fmaf(freq, (float)(c - 1 + !c), c > 1 ? pres : 0.0f);
        return l + s.bias[y];
    };
    // in place, an unmasked row's touched tokens are changed one by one, and a
    // masked row's logits are read and written where they matter
    auto fetch_where = [&](int i, raw& xr, unsigned al) {
        if (!INPLACE) fetch(i, xr);
        else if (r0 + i < r1 && mask_of(i) != -1 && al && (q.live || mine || al != ALL)) fetch(i, xr);
    };
    if (INPLACE) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) fetch_where(u, x[u], allow[u]);
    }
    int my_live = 0; // of row r0 + lane
    for (int ia = 0; r0 + ia < r1; ia += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = ia + u;
            if (r0 + i >= r1) break;
            const bool masked = mask_of(i) != -1;
            elem* out = dst + i * q.ors;
            if (listed && i > 0) { // the drafted token between the last row and this one
                const int y = __builtin_amdgcn_readlane(my_draft, i - 1) - w0;
                if ((unsigned)y < (unsigned)SPAN && w0 + y < q.V) {
                    add_draft(y);
                    wave_sync();
                }
            }
            if (INPLACE && !masked) {
                for (int p = lane; p < listed; p += 64) {
                    const int y = s.at[p];
                    out[y] = X::put(apply(X::get(out[y]), y));
                }
            } else {
                if (listed) {
                    *(raw*)&s.row[lane * PT] = x[u];
                    wave_sync();
                    for (int p = lane; p < listed; p += 64) {
                        const int y = s.at[p];
                        s.row[y] = X::put(apply(X::get(s.row[y]), y));
                    }
                    wave_sync();
                    x[u] = *(const raw*)&s.row[lane * PT];
                    wave_sync();
                }
                if (masked) {
                    if (!__any(allow[u])) { // a grammar often leaves nothing of a span
#pragma unroll
                        for (int k = 0; k < PT; ++k) x[u][k] = X::none();
                    } else {
                        // live: the allowed tokens, if none of the row's is infinite or NaN
                        const bool plain = q.live && !__any(allow[u] && X::special(x[u]));
                        X::mask(x[u], allow[u]);
                        if (q.live) {
                            int n = __popc(allow[u]);
                            if (!plain || w0 + SPAN > q.V) { // tokens past the row's end are -infinity here
                                n = 0;
#pragma unroll
                                for (int k = 0; k < PT; ++k) n += X::get(x[u][k]) > -INFINITY;
                            }
                            n = wave_total(n);
                            if (lane == i) my_live = n;
                        }
                    }
                }
                if (inside && (!INPLACE || mine || allow[u] != ALL)) store_logits<DT>(out + lane * PT, x[u], v0, q.V);
            }
            allow[u] = allow_next[u];
            fetch_where(i + kAhead, x[u], allow[u]);
            fetch_mask(i + 2 * kAhead, allow_next[u]);
        }
    }
    // The counts of the workgroup's wavefronts are joined in LDS and its last
    // wavefront adds them to the output: one atomic instruction for all rows.
    // (One for each row and wavefront: 42 us instead of 28 for 400 masked
    // rows of 50257 tokens, most of it spent on their few cache lines.)
    if (q.live && q.masks) {
        if (my_live) __hip_atomic_fetch_add(&t.live[lane], my_live, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        int done = 0;
        if (lane == 0) done = __hip_atomic_fetch_add(&t.done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        done = __builtin_amdgcn_readfirstlane(done);
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
        const int waves = min(kThreads / 64, (q.V - blk * (kThreads / 64) * SPAN + SPAN - 1) / SPAN);
        if (done == waves - 1) {
            const int live = t.live[lane];
            if (live)
                __hip_atomic_fetch_add(q.live + (long long)b * q.rows + r0 + lane, live, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
}

// Eight wavefronts to a SIMD (six with bf16's lists, whose LDS allows no more):
// 1605 MB of fp32 rows, up to 5 to a sequence, take 298 us, with six 335; 4352
// fp32 rows, 17 to a sequence, 815 and 787.  (Asked for as seven: for eight, scalar
// registers spill, 308 us.)  One block to a workgroup: a loop over
// blocks keeps so much in scalar registers that they spill (the masks of 500
// rows of 50257 took 19.9 us with it, 17.9 without).
template <int DT, bool INPLACE, bool RULES>
__global__ __launch_bounds__(kThreads, 7) void sv_process_kernel(Rules q)
{
    __shared__ __align__(16) Listed<DT> lists[RULES ? kThreads / 64 : 1];
    __shared__ Tally tally;
    if (threadIdx.x < 64) tally.live[threadIdx.x] = 0;
    if (threadIdx.x == 0) tally.done = 0;
    __syncthreads();
    process_block<DT, INPLACE, RULES>(q, lists[RULES ? threadIdx.x >> 6 : 0], tally);
}

// ---------------------------------------------------------------- history

struct Hist {
    int B, V, words, most, kind, n_slots;
    const int* tok;
    long long stride;
    const long long* off;
    long long n_tokens;
    const int* len;
    const int* slots;
    const int* reset;
    int* counts;
    unsigned* seen;
    int* status;
    int per; // workgroups per sequence
};

// Slot, first token and number of tokens of sequence b; slot -1: skipped.
__device__ __forceinline__ int hist_seq(const Hist& q, int b, long long& first, int& n, bool tell)
{
    const int slot = q.slots ? q.slots[b] : b;
    long long m = q.most;
    first = b * q.stride;
    bool bad = slot < -1 || slot >= q.n_slots;
    if (q.off) {
        first = q.off[b];
        const long long end = q.off[b + 1];
        m = end - first;
        bad = bad || first < 0 || end > q.n_tokens;
    } else if (q.len) {
        m = q.len[b];
    }
    bad = bad || m < 0 || m > q.most;
    if (bad && tell) bad_input(q.status);
    n = bad ? 0 : (int)m;
    return bad ? -1 : slot;
}

// Clears a slot's counts from v0 to V, thread t of `threads` (non-temporal: 256
// slots of 129280 in 40 us with the rest of their call, 48 with other stores).
__device__ __forceinline__ void zero_counts(int* c, int v0, int V, int t, int threads)
{
    typedef int four __attribute__((ext_vector_type(4), aligned(4)));
    const four zero = {0, 0, 0, 0};
    for (int v = v0 + t * 4; v < V; v += threads * 4) {
        if (v + 4 <= V) __builtin_nontemporal_store(zero, (four*)(c + v));
        else
            for (int k = v; k < V; ++k) c[k] = 0;
    }
}

__global__ __launch_bounds__(kThreads) void sv_history_clear_kernel(Hist q)
{
    const int b = blockIdx.x / q.per, part = blockIdx.x % q.per;
    long long first;
    int n;
    const int slot = hist_seq(q, b, first, n, false);
    if (slot < 0 || !q.reset[b]) return;
    zero_counts(q.counts + (long long)slot * q.V, 0, q.V, part * kThreads + threadIdx.x, q.per * kThreads);
    unsigned* s = q.seen + (long long)slot * q.words;
    for (int v = part * kThreads + threadIdx.x; v < q.words; v += q.per * kThreads) s[v] = 0;
}

// A token of sequence b's list, or -1 (padding, or an id that is reported and
// left out).
__device__ __forceinline__ int token_at(const Hist& q, long long i)
{
    const int v = q.tok[i];
    if ((unsigned)v < (unsigned)q.V) return v;
    if (v != -1) bad_input(q.status);
    return -1;
}

// One token to a thread, with an atomic on its word of the seen bits and one on
// its count.  Bound by those atomics, about 17 to a ns over the whole chip.
__global__ __launch_bounds__(kThreads) void sv_history_add_kernel(Hist q)
{
    const int b = blockIdx.x / q.per, part = blockIdx.x % q.per;
    long long first;
    int n;
    const int slot = hist_seq(q, b, first, n, part == 0 && threadIdx.x == 0);
    if (slot < 0) return;
    int* c = q.counts + (long long)slot * q.V;
    unsigned* s = q.seen + (long long)slot * q.words;
    for (int i = part * kThreads + threadIdx.x; i < n; i += q.per * kThreads) {
        const int v = token_at(q, first + i);
        if (v < 0) continue;
        __hip_atomic_fetch_or(s + (v >> 5), 1u << (v & 31), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (q.kind == SV_HISTORY_OUTPUT) __hip_atomic_fetch_add(c + v, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// Long lists: a workgroup gathers the seen bits of its part of a list in LDS and
// adds them to the slot's word by word, where consecutive lanes meet
// consecutive words.  A range of kBitWords words at a time (all of them up to
// a vocabulary of 524288).
constexpr int kBitThreads = 1024;
constexpr int kBitWords = 16384;

__global__ __launch_bounds__(kBitThreads) void sv_history_bits_kernel(Hist q)
{
    extern __shared__ unsigned bits[];
    const int b = blockIdx.x / q.per, part = blockIdx.x % q.per;
    long long first;
    int n;
    const int slot = hist_seq(q, b, first, n, part == 0 && threadIdx.x == 0);
    if (slot < 0) return;
    int* c = q.counts + (long long)slot * q.V;
    unsigned* s = q.seen + (long long)slot * q.words;
    const int share = (n + q.per - 1) / q.per, i0 = part * share, i1 = min(n, i0 + share);
    if (i0 >= i1) return;
    for (int w0 = 0; w0 < q.words; w0 += kBitWords) {
        const int words = min(kBitWords, q.words - w0);
        for (int w = threadIdx.x; w < words; w += kBitThreads) bits[w] = 0;
        __syncthreads();
        for (int i = i0 + threadIdx.x; i < i1; i += kBitThreads) {
            const int v = token_at(q, first + i), w = (v >> 5) - w0;
            if (v < 0 || (unsigned)w >= (unsigned)words) continue;
            __hip_atomic_fetch_or(bits + w, 1u << (v & 31), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            if (q.kind == SV_HISTORY_OUTPUT) __hip_atomic_fetch_add(c + v, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        for (int w = threadIdx.x; w < words; w += kBitThreads)
            if (bits[w]) __hip_atomic_fetch_or(s + w0 + w, bits[w], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
    }
}

// A call with resets, in one launch: kResetParts workgroups per sequence, each with a
// part of the slot's tokens to itself, for which it reads the whole list.  Of
// several sequences that name one slot the first takes the tokens of all, so
// that every reset comes before every token and nothing but this workgroup
// touches the part: the counts need atomics of its own scope only, the seen bits
// none.  Bound by the writes of the cleared counts.
// It saves a launch, about 2 us, but its workgroups are large, each looks through
// the slots of the call, and each reads a list alone.  us in one launch, and as a
// clear and an addition, lists of 500 ids:
//   sequences           16         128         256         512
//   slots of 4000      4.0  6.8   7.4  7.5  11.6 10.7  19.7 17.6   (2048: 52 and 18)
//   slots of 129280    6.6  6.9  17.5 18.9  31.6 35.4  60.0 67.9
// and 4 lists of up to 32768 11.6 and 12.3, of up to 131072 27 and 12.  Many
// sequences on one slot leave its four workgroups all their lists: 256 of 500 ids
// take 191 us and 30, of 8192 1134 and 100.  The host does not see the slots.
constexpr int kResetBatch = 256;
constexpr int kResetTokens = 32768;
// One slot of 129280 and a list of 900 take the kernel 4.8 us in four parts, 8.1
// in one, 4.2 in sixteen; calls that reset 256 such slots, lists of up to 500,
// 29.8, 31.1 and 33.9.
constexpr int kResetParts = 4;
static_assert((SV_MAX_VOCAB / 32 + kResetParts - 1) / kResetParts <= kBitWords, "a part's bits are gathered in one go");

__global__ __launch_bounds__(kBitThreads) void sv_history_reset_kernel(Hist q)
{
    extern __shared__ unsigned bits[];
    __shared__ int lower, others, clear;
    const int b = blockIdx.x / q.per, part = blockIdx.x % q.per;
    long long first;
    int n;
    const int slot = hist_seq(q, b, first, n, part == 0 && threadIdx.x == 0);
    const int share_words = (q.words + q.per - 1) / q.per; // of a part
    const int begin = part * share_words, end = min(q.words, begin + share_words);
    if (slot < 0 || begin >= end) return;
    if (threadIdx.x == 0) {
        lower = others = 0;
        clear = q.reset[b] != 0;
    }
    __syncthreads();
    if (q.slots) // without them, no two sequences share one
        for (int o = threadIdx.x; o < q.B; o += kBitThreads) {
            if (o == b || q.slots[o] != slot) continue;
            long long f;
            int m;
            if (hist_seq(q, o, f, m, false) < 0) continue;
            if (o < b) lower = 1;
            else others = 1;
            if (q.reset[o]) clear = 1;
        }
    __syncthreads();
    if (lower) return;
    const bool share = others, anew = clear;
    int* c = q.counts + (long long)slot * q.V;
    unsigned* s = q.seen + (long long)slot * q.words;
    if (anew) {
        zero_counts(c, begin * 32, min(q.V, end * 32), threadIdx.x, kBitThreads);
        if (q.kind == SV_HISTORY_OUTPUT) {
            __builtin_amdgcn_s_waitcnt(0x0f70); // vmcnt 0: the zeros are in the L2, where the counts are added to
            __syncthreads();
        }
    }
    const int words = end - begin;
    for (int w = threadIdx.x; w < words; w += kBitThreads) bits[w] = 0;
    __syncthreads();
    for (int o = b; o < (share ? q.B : b + 1); ++o) {
        if (o > b && (q.slots[o] != slot || hist_seq(q, o, first, n, false) < 0)) continue;
        for (int i = threadIdx.x; i < n; i += kBitThreads) {
            const int v = token_at(q, first + i), w = (v >> 5) - begin;
            if (v < 0 || (unsigned)w >= (unsigned)words) continue;
            __hip_atomic_fetch_or(bits + w, 1u << (v & 31), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            if (q.kind == SV_HISTORY_OUTPUT) __hip_atomic_fetch_add(c + v, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
    }
    __syncthreads();
    for (int w = threadIdx.x; w < words; w += kBitThreads) {
        if (anew) s[begin + w] = bits[w];
        else if (bits[w]) s[begin + w] |= bits[w];
    }
}

// ---------------------------------------------------------------- host

int words_of(int V) { return (V + 31) / 32; }

template <int DT, bool INPLACE>
hipError_t launch_process(Rules q, hipStream_t s)
{
    const int span = kThreads * Vec<DT>::PT, nblk = (q.V + span - 1) / span;
    // A workgroup takes all rows of its sequence, so that the rules are read once,
    // unless that leaves fewer workgroups than fill the chip (8 to each of 256
    // compute units): then as many chunks of the rows as do (4 sequences of 17 rows
    // of 129280 bf16: 16.3 us, by sequence 33.0, by row 22.0; with 1024 or 4096
    // workgroups wanted 16.7 and 17.4).  A chunk has at most 64 rows, one to a lane.
    const long long by_seq = (long long)q.B * nblk;
    int nchunk = (int)std::min((long long)q.rows, (2048 + by_seq - 1) / by_seq);
    q.chunk = std::min(64, (q.rows + nchunk - 1) / nchunk);
    nchunk = (q.rows + q.chunk - 1) / q.chunk;
    // launches within 2^32 work-items and 65535 workgroups along z
    const int most = (int)std::min(65535ll, 0xffffffffll / kThreads / ((long long)nblk * nchunk));
    for (q.b0 = 0; q.b0 < q.B; q.b0 += most) {
        const dim3 grid(nblk, nchunk, std::min(most, q.B - q.b0)), block(kThreads);
        const hipError_t e = q.counts || q.draft || q.boff
            ? launch_kernel(sv_process_kernel<DT, INPLACE, true>, grid, block, 0, s, nullptr, nullptr, q)
            : launch_kernel(sv_process_kernel<DT, INPLACE, false>, grid, block, 0, s, nullptr, nullptr, q);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

} // namespace

extern "C" {

int spec_verify_process_check(const spec_verify_config* cfg, const spec_verify_process_args* a)
{
    int rc = sv::check_config(cfg);
    if (rc != SV_OK) return rc;
    if (!a) return SV_EINVAL;
    if (a->B < 0 || a->B > cfg->max_batch || a->rows < 1 || a->row0 < 0) return SV_EINVAL;
    if ((long long)a->row0 + a->rows > (long long)cfg->max_draft + 1) return SV_EINVAL;
    if (a->B == 0) return SV_OK;
    const int V = cfg->vocab;
    if (!a->logits_in || !a->logits_out || a->in_row_stride < V || a->out_row_stride < V) return SV_EINVAL;
    const bool packed = a->row_offsets != nullptr;
    if (packed && a->verify_len) return SV_EINVAL;
    if (!packed) {
        if (a->in_batch_stride < 0 || a->out_batch_stride < 0) return SV_EINVAL;
        // no two output rows overlap, whichever of the two strides is the outer one
        const long long by_b = a->out_batch_stride, by_r = a->out_row_stride;
        const bool b_outer = by_b >= (long long)(a->rows - 1) * by_r + V;
        const bool r_outer = by_b >= V && by_r >= (long long)(a->B - 1) * by_b + V;
        if (a->B > 1 && !b_outer && !r_outer) return SV_EINVAL;
    }
    if (a->logits_in == a->logits_out) {
        if (a->in_row_stride != a->out_row_stride) return SV_EINVAL;
        if (!packed && a->in_batch_stride != a->out_batch_stride) return SV_EINVAL;
    }
    if (a->draft_tokens && a->draft_stride < (long long)a->row0 + a->rows - 1) return SV_EINVAL;
    if (!a->history_counts != !a->history_seen) return SV_EINVAL;
    if (a->history_counts && (a->n_slots < 1 || (!a->slots && a->n_slots < a->B))) return SV_EINVAL;
    if (a->bias_offsets && (a->n_biases < 0 || (a->n_biases && (!a->bias_tokens || !a->bias_values)))) return SV_EINVAL;
    if (a->masks && (!a->mask_index || a->n_masks < 1 || a->mask_stride < words_of(V))) return SV_EINVAL;
    return SV_OK;
}

int spec_verify_process(spec_verify_t* h, const spec_verify_process_args* a, void* hip_stream)
{
    if (!h) return SV_EINVAL;
    const spec_verify_config* cfg = sv::handle_config(h);
    int rc = spec_verify_process_check(cfg, a);
    if (rc != SV_OK) return rc;
    if (a->B == 0) return SV_OK;
    DeviceGuard guard(cfg->device);
    hipStream_t s = (hipStream_t)hip_stream;
    Rules q;
    q.B = a->B;
    q.rows = a->rows;
    q.row0 = a->row0;
    q.V = cfg->vocab;
    q.words = words_of(q.V);
    q.in = a->logits_in;
    q.ibs = a->in_batch_stride;
    q.irs = a->in_row_stride;
    q.out = a->logits_out;
    q.obs = a->out_batch_stride;
    q.ors = a->out_row_stride;
    q.roff = (const long long*)a->row_offsets;
    q.vlen = a->verify_len;
    q.draft = a->draft_tokens;
    q.dstride = a->draft_stride;
    q.counts = a->history_counts;
    q.seen = a->history_seen;
    q.n_slots = a->n_slots;
    q.slots = a->slots;
    q.rep = a->repetition;
    q.freq = a->frequency;
    q.pres = a->presence;
    q.boff = a->bias_offsets;
    q.btok = a->bias_tokens;
    q.bval = a->bias_values;
    q.n_biases = a->n_biases;
    q.masks = a->masks;
    q.mstride = a->mask_stride;
    q.n_masks = a->n_masks;
    q.midx = a->mask_index;
    q.live = a->live_tokens;
    q.status = a->device_status;
    q.b0 = q.chunk = 0;
    hipError_t e = hipSuccess;
    if (q.live || q.status) {
        const long long rows = q.live ? (long long)q.B * q.rows : 1;
        e = launch_kernel(sv_rules_start_kernel, dim3((unsigned)((rows + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
                          nullptr, nullptr, q);
    }
    if (e == hipSuccess) {
        const bool same = q.in == q.out;
        if (cfg->dtype == SV_BF16) e = same ? launch_process<SV_BF16, true>(q, s) : launch_process<SV_BF16, false>(q, s);
        else e = same ? launch_process<SV_F32, true>(q, s) : launch_process<SV_F32, false>(q, s);
    }
    return e == hipSuccess ? SV_OK : SV_EDEVICE;
}

int spec_verify_history_check(const spec_verify_config* cfg, const spec_verify_history_args* a)
{
    int rc = sv::check_config(cfg);
    if (rc != SV_OK) return rc;
    if (!a) return SV_EINVAL;
    if (a->B < 0 || a->B > cfg->max_batch || a->max_tokens < 0) return SV_EINVAL;
    if (a->kind != SV_HISTORY_PROMPT && a->kind != SV_HISTORY_OUTPUT) return SV_EINVAL;
    if (a->B == 0) return SV_OK;
    if (!a->counts || !a->seen || a->n_slots < 1 || (!a->slots && a->n_slots < a->B)) return SV_EINVAL;
    if (a->max_tokens && !a->tokens) return SV_EINVAL;
    if (a->max_tokens > SV_MAX_HISTORY_TOKENS) return SV_EUNSUPPORTED;
    if (a->token_offsets) {
        if (a->lengths || a->n_tokens < 0) return SV_EINVAL;
    } else if (a->token_stride < a->max_tokens) {
        return SV_EINVAL;
    }
    return SV_OK;
}

int spec_verify_history(spec_verify_t* h, const spec_verify_history_args* a, void* hip_stream)
{
    if (!h) return SV_EINVAL;
    const spec_verify_config* cfg = sv::handle_config(h);
    int rc = spec_verify_history_check(cfg, a);
    if (rc != SV_OK) return rc;
    if (a->B == 0) return SV_OK;
    DeviceGuard guard(cfg->device);
    hipStream_t s = (hipStream_t)hip_stream;
    Hist q;
    q.B = a->B;
    q.V = cfg->vocab;
    q.words = words_of(q.V);
    q.most = a->max_tokens;
    q.kind = a->kind;
    q.n_slots = a->n_slots;
    q.tok = a->tokens;
    q.stride = a->token_stride;
    q.off = (const long long*)a->token_offsets;
    q.n_tokens = a->n_tokens;
    q.len = a->lengths;
    q.slots = a->slots;
    q.reset = a->reset;
    q.counts = a->counts;
    q.seen = a->seen;
    q.status = a->device_status;
    q.per = 1;
    hipError_t e = hipSuccess;
    if (q.status) e = launch_kernel(sv_status_clear_kernel, dim3(1), dim3(1), 0, s, nullptr, nullptr, q.status);
    // workgroups per sequence: enough for the work, within 2^32 work-items in all
    const long long cap = std::max(1ll, 0xffffffffll / kThreads / q.B);
    auto parts = [&](long long items) {
        return (int)std::min(cap, std::max(1ll, (items + kThreads - 1) / kThreads));
    };
    const size_t lds = sizeof(unsigned) * std::min(kBitWords, q.words);
    if (e == hipSuccess && q.reset && q.B <= kResetBatch && q.most <= kResetTokens) {
        q.per = kResetParts;
        const size_t part = sizeof(unsigned) * ((q.words + q.per - 1) / q.per);
        e = launch_kernel(sv_history_reset_kernel, dim3((unsigned)(q.B * q.per)), dim3(kBitThreads), (uint32_t)part,
                          s, nullptr, nullptr, q);
        return e == hipSuccess ? SV_OK : SV_EDEVICE;
    }
    if (e == hipSuccess && q.reset) {
        q.per = std::min(64, parts(q.V / 4 + 1));
        e = launch_kernel(sv_history_clear_kernel, dim3((unsigned)((long long)q.B * q.per)), dim3(kThreads), 0, s, nullptr,
                          nullptr, q);
    }
    // The bits in LDS cost a workgroup about 5 us whatever the list, so they are for
    // long lists, and where the atomics would take longer than that: 256 lists of
    // up to 8192 tokens take 8 us with them and 95 without.
    if (e == hipSuccess && q.most >= 512 && (long long)q.B * q.most >= 32768) {
        q.per = (int)std::min(cap / 4, std::min(64ll, (q.most + 8191ll) / 8192));
        e = launch_kernel(sv_history_bits_kernel, dim3((unsigned)((long long)q.B * q.per)), dim3(kBitThreads), (uint32_t)lds, s,
                          nullptr, nullptr, q);
    } else if (e == hipSuccess) {
        q.per = std::min(64, parts(q.most));
        e = launch_kernel(sv_history_add_kernel, dim3((unsigned)((long long)q.B * q.per)), dim3(kThreads), 0, s, nullptr,
                          nullptr, q);
    }
    return e == hipSuccess ? SV_OK : SV_EDEVICE;
}

} // extern "C"
