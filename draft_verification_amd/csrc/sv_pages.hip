// The pages of the target's cache: which slot holds which (spec_verify_pages),
// copies of them (spec_verify_pages_copy), and the keys and values of new rows
// (spec_verify_append).  include/spec_verify.h states what each does.

#include <algorithm>

#include "spec_verify.h"
#include "sv_cache.h"
#include "sv_host.h"

using sv::cache_status;
using sv::cache_uniform;
using sv::Cache;
using sv::DeviceGuard;
using sv::launch_kernel;
using sv::lds_barrier;
using sv::Sequence;

namespace {

constexpr int kThreads = 256;
constexpr int kPlan = 1024;        // threads of the one workgroup that gives pages out
constexpr int kHash = 8192;        // twice SV_MAX_PAGE_BATCH

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

struct Pages {
    Cache c;
    int B, kind;
    const int* slots;
    const int* from;
    int rows;
    const int* last;
    int* granted;
    int2* copies;
    int max_copies;
    int* status;
};

__global__ void sv_cache_status_kernel(int* status) { *status = 0; }

// Where the cache has pages for a length.
__device__ __forceinline__ long long pages_for(const Cache& c, long long tokens)
{
    return (tokens + (1 << c.shift) - 1) >> c.shift;
}

__device__ __forceinline__ int held_pages(const Cache& c, int slot)
{
    const int n = c.counts[slot];
    return n < 0 || n > c.max_pages ? -1 : n;
}

// Rows that RESERVE and COMMIT count for sequence b, or -1.
__device__ __forceinline__ int counted_rows(const Pages& q, int b)
{
    if (!q.last) return q.rows;
    const int last = q.last[b];
    return last < -1 ? -1 : last < q.rows ? last + 1 : q.rows;
}

// Exclusive sum over the workgroup's threads; total gets the whole sum.  part:
// an entry for each wavefront.
__device__ __forceinline__ int block_before(int x, int* part, int& total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int sum = x;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(sum, d);
        if (lane >= d) sum += y;
    }
    lds_barrier(); // the last use of part
    if (lane == 63) part[wave] = sum;
    lds_barrier();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kPlan / 64; ++w) {
        if (w < wave) before += part[w];
        total += part[w];
    }
    return before + sum - x;
}

__device__ __forceinline__ unsigned hash_of(int slot) { return ((unsigned)slot * 2654435761u) >> (32 - 13); }

// Place of a slot in the table, or -1.
__device__ __forceinline__ int hash_find(const int* key, int slot)
{
    for (unsigned h = hash_of(slot);; h = (h + 1) % kHash) {
        if (key[h] == slot) return (int)h;
        if (key[h] < 0) return -1;
    }
}

// Free pages of a word of the bitmap (bits behind the last page do not count).
__device__ __forceinline__ unsigned free_word(const Cache& c, int w)
{
    const int pages = c.n_pages - w * 32;
    const unsigned x = pages > 0 ? c.free[w] : 0u;
    return pages >= 32 ? x : pages > 0 ? x & ((1u << pages) - 1) : 0u;
}

// RESERVE, and the new pages of FORK: one workgroup, since every page that is given
// depends on all that are given before.  It counts what each sequence needs, sums that
// up, and walks the bitmap of free pages, 32768 of them at a time, whose free ones it
// lists in LDS, up to the last one needed.  Bound by the steps that wait for one
// another (slots, their numbers, the bitmap, the stores: 8 us for 16 sequences of 125
// pages), and with many pages by what one compute unit stores.  So many pages are given in
// two launches: in the first a workgroup for every 32768 pages writes the tables and the
// references, each having summed up for itself (GIVE_TABLES), and the second does the rest
// (GIVE_STATE): 256 prompts of 1000 pages, with what their slots held given back first and
// both launches, 56 us for 104.
enum { GIVE_ALL, GIVE_TABLES, GIVE_STATE };

template <int PART>
__global__ __launch_bounds__(kPlan) void sv_pages_give_kernel(Pages q)
{
    constexpr int kEach = SV_MAX_PAGE_BATCH / kPlan; // most sequences of a thread
    constexpr int kCount = 8;                        // words of a thread at a time where they are only counted
    __shared__ int key[kHash];             // slots that the call names, by hash
    __shared__ unsigned twice[kHash / 32]; // named again
    __shared__ int upto[SV_MAX_PAGE_BATCH]; // pages needed up to and with each sequence
    __shared__ int slots[SV_MAX_PAGE_BATCH];
    __shared__ int place[SV_MAX_PAGE_BATCH]; // RESERVE: pages that it has; FORK: the page to copy
    __shared__ unsigned short list[kPlan * 32];
    __shared__ int part[kPlan / 64];
    __shared__ int said;
    const Cache& c = q.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const bool fork = q.kind == SV_PAGES_FORK;
    const int words = (c.n_pages + 31) / 32;
    const int each = (q.B + kPlan - 1) / kPlan, b0 = tid * each; // sequences of a thread, one after the other

    for (int i = tid; i < kHash; i += kPlan) key[i] = -1;
    for (int i = tid; i < kHash / 32; i += kPlan) twice[i] = 0;
    if (tid == 0) said = 0;
    lds_barrier();
    for (int i = 0; i < each; ++i) {
        const int b = b0 + i;
        if (b >= q.B) break;
        const int slot = q.slots ? q.slots[b] : b;
        slots[b] = slot;
        if (slot < 0 || slot >= c.n_slots) continue;
        for (unsigned h = hash_of(slot);; h = (h + 1) % kHash) {
            const int was = atomicCAS(&key[h], -1, slot);
            if (was == slot) atomicOr(&twice[h / 32], 1u << (h % 32));
            if (was == -1 || was == slot) break;
        }
    }
    lds_barrier();
    if (fork) { // a slot that is filled here is no source
        for (int i = 0; i < each; ++i) {
            const int b = b0 + i;
            if (b >= q.B) break;
            const int from = q.from[b];
            const int h = from >= 0 && slots[b] != -1 ? hash_find(key, from) : -1;
            if (h >= 0) atomicOr(&twice[h / 32], 1u << (h % 32));
        }
        lds_barrier();
    }

    // what each sequence needs: -1 nothing is to be done, -2 it is bad
    auto need_of = [&](int b) -> int {
        const int slot = slots[b];
        if (slot == -1) return -1;
        if (slot < 0 || slot >= c.n_slots) return -2;
        const int h = hash_find(key, slot);
        const int held = held_pages(c, slot), len = c.lengths[slot];
        place[b] = held;
        if (twice[h / 32] >> (h % 32) & 1) return -2;
        if (held < 0 || len < 0) return -2;
        if (fork) {
            const int from = q.from[b];
            if (held != 0 || len != 0 || from < 0 || from >= c.n_slots || hash_find(key, from) >= 0) return -2;
            const int n = c.lengths[from], pages = held_pages(c, from);
            if (n < 0 || pages < 0 || pages_for(c, n) > pages) return -2;
            if (!(n & ((1 << c.shift) - 1))) return 0;
            const int last = c.table[(long long)from * c.max_pages + (n >> c.shift)];
            place[b] = last;
            return last < 0 || last >= c.n_pages ? -2 : 1;
        }
        const int n = counted_rows(q, b);
        if (n < 0) return -2;
        const long long pages = pages_for(c, (long long)len + n);
        return pages > c.max_pages ? -2 : pages > held ? (int)pages - held : 0;
    };
    // sums stop at one page more than there are, which is too much already
    const int most = c.n_pages + 1;
    int need[kEach], mine = 0, total = 0, bits = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        need[i] = i < each && b0 + i < q.B ? need_of(b0 + i) : -1;
        if (need[i] == -2) bits |= SV_STATUS_BAD_INPUT;
        mine = min(mine + min(max(need[i], 0), most), most);
    }
    {
        int sum = mine;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int y = __shfl_up(sum, d);
            if (lane >= d) sum = min(sum + y, most);
        }
        if (lane == 63) part[wave] = sum;
        lds_barrier();
        int before = 0;
#pragma unroll
        for (int w = 0; w < kPlan / 64; ++w) {
            if (w < wave) before = min(before + part[w], most);
            total = min(total + part[w], most);
        }
        int run = __shfl_up(sum, 1);
        run = min(before + (lane ? run : 0), most);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (i >= each || b0 + i >= q.B) break;
            run = min(run + min(max(need[i], 0), most), most);
            upto[b0 + i] = run;
        }
        lds_barrier();
    }
    // how many pages are free, up to what is needed, and before the workgroup's own
    const int own = PART == GIVE_TABLES ? (int)blockIdx.x * kPlan : 0;
    int have = 0, base = 0;
    for (int w0 = 0; w0 < words && have < total; w0 += kPlan * kCount) {
        int n = 0, found, before = 0;
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int w = w0 + i * kPlan + tid, k = __popc(w < words ? free_word(c, w) : 0u);
            n += k;
            if (PART == GIVE_TABLES && w < own) before += k;
        }
        (void)block_before(n, part, found);
        have += found;
        if constexpr (PART == GIVE_TABLES) {
            (void)block_before(before, part, found);
            base += found;
        }
    }
    // all of the sequences whose sums stay below that; the sums do not fall
    int given = 0;
    {
        int lo = 0, hi = q.B; // first sequence that gets nothing
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (upto[mid] <= have) lo = mid + 1;
            else hi = mid;
        }
        given = lo ? upto[lo - 1] : 0;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int b = b0 + i;
        if (PART == GIVE_TABLES || i >= each || b >= q.B) break;
        const bool ok = need[i] == 0 || (need[i] > 0 && upto[b] <= have);
        if (q.granted) q.granted[b] = ok;
        if (need[i] > 0 && !ok) bits |= SV_STATUS_NO_PAGES;
        if (fork && !(need[i] > 0 && ok)) q.copies[b] = make_int2(-1, -1);
        if (!fork && need[i] > 0 && ok) c.counts[slots[b]] = place[b] + need[i];
    }
    // the pages: the k-th free one to the sequence whose sums enclose k
    unsigned ahead = own + tid < words ? free_word(c, own + tid) : 0u;
    for (int w0 = own; w0 < words && base < given && (PART != GIVE_TABLES || w0 == own); w0 += kPlan) {
        unsigned x = ahead;
        ahead = w0 + kPlan + tid < words ? free_word(c, w0 + kPlan + tid) : 0u;
        int found;
        int at = block_before(__popc(x), part, found);
        const int here = min(found, given - base);
        unsigned taken = 0;
        if (PART == GIVE_STATE && at + __popc(x) <= here) taken = x, x = 0;
        for (; x && at < here; x &= x - 1, ++at) {
            if constexpr (PART != GIVE_STATE) list[at] = (unsigned short)(tid * 32 + __ffs(x) - 1);
            taken |= x & -x;
        }
        if (PART != GIVE_TABLES && taken) c.free[w0 + tid] &= ~taken;
        if constexpr (PART == GIVE_STATE) {
            base += found;
            continue;
        }
        lds_barrier();
        int lo = 0, hi = q.B; // first sequence that ends behind base
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (upto[mid] <= base) lo = mid + 1;
            else hi = mid;
        }
        for (int b = lo + wave; b < q.B; b += kPlan / 64) {
            const int first = b ? upto[b - 1] : 0, end = min(upto[b], base + here);
            if (first >= base + here) break;
            if (first == upto[b]) continue;
            int* const to = c.table + (long long)slots[b] * c.max_pages + place[b] - first;
            for (int k = max(first, base) + lane; k < end; k += 64) {
                const int page = w0 * 32 + list[k - base];
                c.refs[page] = 1;
                if (fork) q.copies[b] = make_int2(place[b], page);
                else to[k] = page;
            }
        }
        base += found;
        lds_barrier();
    }
    if (PART != GIVE_TABLES && q.status) {
        if (bits) atomicOr(&said, bits);
        lds_barrier();
        if (tid == 0) *q.status = said;
    }
}

// FORK, second part: a workgroup fills one slot's table.  The new page is known by
// then; a full page gets one reference more.  Bound by its chain of loads.
__global__ __launch_bounds__(kThreads) void sv_pages_share_kernel(Pages q)
{
    const int b = blockIdx.x;
    if (!q.granted[b]) return;
    const Cache& c = q.c;
    const int slot = q.slots ? q.slots[b] : b, from = q.from[b], len = c.lengths[from];
    const long long to_row = (long long)slot * c.max_pages, from_row = (long long)from * c.max_pages;
    const int full = len >> c.shift;
    for (int i = threadIdx.x; i < full; i += kThreads) {
        int page = c.table[from_row + i];
        if (page < 0 || page >= c.n_pages) {
            cache_status(q.status, SV_STATUS_BAD_INPUT);
            page = -1;
        } else {
            atomicAdd(&c.refs[page], 1);
        }
        c.table[to_row + i] = page;
    }
    if (threadIdx.x == 0) {
        const bool part = len & ((1 << c.shift) - 1);
        if (part) c.table[to_row + full] = q.copies[b].y;
        c.counts[slot] = full + part;
        c.lengths[slot] = len;
    }
}

// COMMIT and RELEASE: a workgroup gives back one slot's pages past those it keeps, four
// to a thread at a time.  Bound by the steps that wait for one another: the slot, its
// numbers, its pages, their references.
__global__ __launch_bounds__(kThreads) void sv_pages_back_kernel(Pages q)
{
    constexpr int kEach = 4;
    const int b = blockIdx.x;
    const Cache& c = q.c;
    const int slot = q.slots ? cache_uniform(q.slots + b) : b;
    if (slot == -1) return;
    bool bad = slot < 0 || slot >= c.n_slots;
    const int held = bad ? -1 : held_pages(c, slot), len = bad ? -1 : c.lengths[slot];
    if (q.slots)
        for (int i = threadIdx.x; i < q.B; i += kThreads) bad |= i != b && q.slots[i] == slot;
    long long length = 0, keep = 0;
    if (q.kind == SV_PAGES_COMMIT) {
        const int n = counted_rows(q, b);
        length = (long long)len + n;
        keep = pages_for(c, length);
        bad |= n < 0 || len < 0 || keep > held;
    }
    bad |= held < 0;
    if (__syncthreads_or(bad)) { // (every thread has read what is changed below)
        if (threadIdx.x == 0) cache_status(q.status, SV_STATUS_BAD_INPUT);
        return;
    }
    if (threadIdx.x == 0) {
        c.lengths[slot] = (int)length;
        c.counts[slot] = (int)keep;
    }
    int* const row = c.table + (long long)slot * c.max_pages;
    for (int i0 = (int)keep + threadIdx.x; i0 < held; i0 += kThreads * kEach) {
        int page[kEach], refs[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = i0 + k * kThreads;
            page[k] = i < held ? row[i] : -1;
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const bool there = page[k] >= 0 && page[k] < c.n_pages;
            refs[k] = there ? atomicSub(&c.refs[page[k]], 1) : 0;
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = i0 + k * kThreads;
            if (i >= held) break;
            row[i] = -1;
            if (refs[k] == 1) {
                atomicOr(&c.free[page[k] / 32], 1u << (page[k] % 32));
            } else if (refs[k] < 1) { // nothing that these calls leave
                if (page[k] >= 0 && page[k] < c.n_pages) atomicAdd(&c.refs[page[k]], 1);
                cache_status(q.status, SV_STATUS_BAD_INPUT);
            }
        }
    }
}

__global__ __launch_bounds__(kThreads) void sv_pages_clear_kernel(Cache c)
{
    const long long step = (long long)gridDim.x * kThreads, first = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long entries = (long long)c.n_slots * c.max_pages;
    for (long long i = first; i < entries; i += step) c.table[i] = -1;
    for (long long i = first; i < c.n_slots; i += step) c.lengths[i] = c.counts[i] = 0;
    for (long long i = first; i < c.n_pages; i += step) c.refs[i] = 0;
    for (long long i = first; i < (c.n_pages + 31) / 32; i += step) {
        const int pages = c.n_pages - (int)i * 32;
        c.free[i] = pages >= 32 ? ~0u : (1u << pages) - 1;
    }
}

// COMPACT, first part: one workgroup pairs the highest pages with the lowest free
// places.  A page that moves leaves ~(its new place) in page_refs, by which the
// tables are then changed.  Bound by the steps that wait for one another.
__global__ __launch_bounds__(kPlan) void sv_pages_pair_kernel(Pages q)
{
    constexpr int kEach = 4;
    __shared__ int part[kPlan / 64];
    const Cache& c = q.c;
    const int tid = threadIdx.x;
    const int words = (c.n_pages + 31) / 32;
    int free = 0, total, holes;
    for (int w = tid; w < words; w += kPlan) free += __popc(free_word(c, w));
    (void)block_before(free, part, total);
    const int live = c.n_pages - total;
    // bits of a word below the number of pages in use
    auto below = [&](int w) { const int n = live - w * 32; return n >= 32 ? ~0u : n > 0 ? (1u << n) - 1 : 0u; };
    free = 0;
    for (int w = tid; w < words; w += kPlan) free += __popc(free_word(c, w) & below(w));
    (void)block_before(free, part, holes);
    const int moves = min(holes, q.max_copies);
    // upwards: the lowest free places are taken
    for (int w0 = 0, done = 0; done < moves; w0 += kPlan) {
        const int w = w0 + tid;
        unsigned x = w < words ? free_word(c, w) & below(w) : 0u, used = 0;
        int found;
        int at = done + block_before(__popc(x), part, found);
        for (; x && at < moves; x &= x - 1, ++at) {
            q.copies[at].y = w * 32 + __ffs(x) - 1;
            used |= x & -x;
        }
        if (used) c.free[w] &= ~used;
        done += found;
    }
    // the word that page `live` lies in is changed both ways, by two threads: what one has
    // stored the other has to read (block_before's barriers are for LDS alone)
    __syncthreads();
    // downwards: the highest pages leave theirs
    for (int w0 = words - 1, done = 0; done < moves; w0 -= kPlan) {
        const int w = w0 - tid;
        unsigned x = 0, used = 0;
        if (w >= 0) {
            const int pages = c.n_pages - w * 32;
            x = ~free_word(c, w) & ~below(w);
            if (pages < 32) x &= (1u << pages) - 1;
        }
        int found;
        int at = done + block_before(__popc(x), part, found);
        for (; x && at < moves; ++at) {
            const int bit = 31 - __clz((int)x);
            q.copies[at].x = w * 32 + bit;
            x ^= 1u << bit;
            used |= 1u << bit;
        }
        if (used) c.free[w] |= used;
        done += found;
    }
    __syncthreads();
    for (int i0 = tid; i0 < q.max_copies; i0 += kPlan * kEach) {
        int2 pair[kEach];
        int refs[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = i0 + k * kPlan;
            pair[k] = i < moves ? q.copies[i] : make_int2(-1, -1);
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) refs[k] = pair[k].x >= 0 ? c.refs[pair[k].x] : 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = i0 + k * kPlan;
            if (i >= q.max_copies) break;
            if (pair[k].x >= 0) {
                c.refs[pair[k].y] = refs[k];
                c.refs[pair[k].x] = ~pair[k].y;
            } else {
                q.copies[i] = pair[k];
            }
        }
    }
    if (tid == 0 && q.status) *q.status = 0;
}

// Second part: the tables take the new places.  A workgroup to a slot.
__global__ __launch_bounds__(kThreads) void sv_pages_rename_kernel(Cache c)
{
    for (long long slot = blockIdx.x; slot < c.n_slots; slot += gridDim.x) {
        const int held = min(c.counts[slot], c.max_pages);
        for (int i = threadIdx.x; i < held; i += kThreads) {
            const int page = c.table[slot * c.max_pages + i];
            if (page < 0 || page >= c.n_pages) continue;
            const int to = ~c.refs[page];
            if (to >= 0 && to < c.n_pages) c.table[slot * c.max_pages + i] = to;
        }
    }
}

// Third part: what a page that moved left in page_refs goes.
__global__ __launch_bounds__(kThreads) void sv_pages_left_kernel(Pages q)
{
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < q.max_copies; i += (long long)gridDim.x * kThreads) {
        const int from = q.copies[i].x;
        if (from >= 0) q.c.refs[from] = 0;
    }
}

struct Copy {
    const int2* copies;
    int n_pages;
    unsigned n_pools;
    char* pools;
    long long pool_stride, page_stride;
    int units;                // of 16 bytes in a page
    unsigned parts;           // workgroups of a page
    long long total;          // workgroups' worth of work
    int* status;
};

constexpr int kCopyUnits = 4; // of 16 bytes for a thread

// A piece of 16 KB of one page in one pool at a time.  Bound by HBM; neither side is
// read again soon, so that both pass the caches by: 437 MB in 88 us (4.9 TB/s).
__global__ __launch_bounds__(kThreads) void sv_pages_copy_kernel(Copy q)
{
    for (long long job = blockIdx.x; job < q.total; job += gridDim.x) {
        const unsigned piece = (unsigned)(job % q.parts);
        const long long rest = job / q.parts;
        const unsigned pool = (unsigned)(rest % q.n_pools);
        const int2 pair = q.copies[rest / q.n_pools];
        if (pair.x == -1 || pair.y == -1) continue;
        if (pair.x < 0 || pair.x >= q.n_pages || pair.y < 0 || pair.y >= q.n_pages) {
            if (threadIdx.x == 0) cache_status(q.status, SV_STATUS_BAD_INPUT);
            continue;
        }
        char* base = q.pools + pool * q.pool_stride;
        const u32x4* from = (const u32x4*)(base + pair.x * q.page_stride);
        u32x4* to = (u32x4*)(base + pair.y * q.page_stride);
        const int first = piece * (kThreads * kCopyUnits) + threadIdx.x;
        u32x4 x[kCopyUnits];
#pragma unroll
        for (int i = 0; i < kCopyUnits; ++i)
            if (first + i * kThreads < q.units) x[i] = __builtin_nontemporal_load(from + first + i * kThreads);
#pragma unroll
        for (int i = 0; i < kCopyUnits; ++i)
            if (first + i * kThreads < q.units) __builtin_nontemporal_store(x[i], to + first + i * kThreads);
    }
}

struct Append {
    Cache c;
    sv::Rows r;
    int b0;
    int kv_heads, per_head; // units of a thread in a head's row
    const unsigned short* k;
    const unsigned short* v;
    long long bs, rs, hs;
    char* keys;
    char* values;
    long long page_stride, head_stride, token_stride; // bytes
    const float* kscale;
    const float* vscale;
    int* status;
};

// Four values to e4m3, the first lowest.  v_cvt_pk_fp8_f32 rounds to nearest, ties
// to even; what is beyond the largest value is brought to it first (a NaN stays).
__device__ __forceinline__ unsigned to_e4m3(float a, float b, float c, float d)
{
    auto lim = [](float x) { return x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x; };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(lim(a), lim(b), 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(lim(c), lim(d), w, true);
}

// A thread takes 16 bytes of the cache: 8 values of bf16, or 16 of e4m3.  Bound by
// HBM, 36 MB of 4352 rows in 7.9 us (4.5 TB/s with the launch) and 302 MB of prompts
// to e4m3 in 62 to 67 (4.5 to 4.9 TB/s); e4m3 divides (fp32, correctly rounded) beside its loads.
template <bool E4M3>
__global__ __launch_bounds__(kThreads) void sv_append_kernel(Append q)
{
    constexpr int kUnit = E4M3 ? 16 : 8;
    const int b = q.b0 + blockIdx.y;
    const Sequence s = sequence_of(q.c, q.r, b);
    if (s.count < 0 && blockIdx.x == 0 && threadIdx.x == 0) cache_status(q.status, SV_STATUS_BAD_INPUT);
    if (s.count <= 0) return;
    const int* table = q.c.table + (long long)s.slot * q.c.max_pages;
    const int mask = (1 << q.c.shift) - 1;
    const unsigned per_row = (unsigned)q.kv_heads * q.per_head;
    const unsigned total = (unsigned)s.count * per_row; // checked on the host to fit
    for (unsigned i = blockIdx.x * kThreads + threadIdx.x; i < total; i += gridDim.x * kThreads) {
        const unsigned row = i / per_row, in_row = i - row * per_row;
        const unsigned head = in_row / q.per_head, unit = in_row - head * q.per_head;
        const int t = s.start + (int)row;
        const int page = table[t >> q.c.shift];
        if (page < 0 || page >= q.c.n_pages) {
            cache_status(q.status, SV_STATUS_BAD_INPUT);
            continue;
        }
        const long long from = (q.r.roff ? (s.first + row) * q.rs : b * q.bs + row * q.rs) + head * q.hs + unit * kUnit;
        const long long to = page * q.page_stride + head * q.head_stride + (t & mask) * q.token_stride + unit * 16;
        if constexpr (!E4M3) {
            const u32x4 x = *(const u32x4_any*)(q.k + from), y = *(const u32x4_any*)(q.v + from);
            *(u32x4*)(q.keys + to) = x;
            *(u32x4*)(q.values + to) = y;
        } else {
            auto convert = [](u32x4 lo, u32x4 hi, float scale) {
                auto two = [&](unsigned w, unsigned w2) {
                    return to_e4m3(__uint_as_float(w << 16) / scale, __uint_as_float(w & 0xffff0000u) / scale,
                                   __uint_as_float(w2 << 16) / scale, __uint_as_float(w2 & 0xffff0000u) / scale);
                };
                return u32x4{two(lo[0], lo[1]), two(lo[2], lo[3]), two(hi[0], hi[1]), two(hi[2], hi[3])};
            };
            const u32x4 x0 = *(const u32x4_any*)(q.k + from), x1 = *(const u32x4_any*)(q.k + from + 8);
            const u32x4 y0 = *(const u32x4_any*)(q.v + from), y1 = *(const u32x4_any*)(q.v + from + 8);
            *(u32x4*)(q.keys + to) = convert(x0, x1, q.kscale ? q.kscale[head] : 1.0f);
            *(u32x4*)(q.values + to) = convert(y0, y1, q.vscale ? q.vscale[head] : 1.0f);
        }
    }
}

int status_of(hipError_t e) { return e == hipSuccess ? SV_OK : SV_EDEVICE; }

hipError_t clear_status(int* status, hipStream_t s)
{
    if (!status) return hipSuccess;
    return launch_kernel(sv_cache_status_kernel, dim3(1), dim3(1), 0, s, nullptr, nullptr, status);
}

} // namespace

extern "C" {

int spec_verify_pages_check(const spec_verify_config* cfg, const spec_verify_pages_args* a)
{
    int rc = sv::check_config(cfg);
    if (rc != SV_OK) return rc;
    if (!a) return SV_EINVAL;
    if (a->kind < SV_PAGES_CLEAR || a->kind > SV_PAGES_COMPACT) return SV_EUNSUPPORTED;
    rc = sv::check_cache(a->cache, true);
    if (rc != SV_OK || a->kind == SV_PAGES_CLEAR) return rc;
    if (a->kind == SV_PAGES_COMPACT) {
        if (a->max_copies < 0 || a->max_copies > SV_MAX_PAGES || (a->max_copies && !a->copies)) return SV_EINVAL;
        return (uintptr_t)a->copies % 8 ? SV_EINVAL : SV_OK;
    }
    rc = sv::check_rows(cfg, a->B, a->cache, a->slots, nullptr, nullptr);
    if (rc != SV_OK) return rc;
    if (a->B > SV_MAX_PAGE_BATCH) return SV_EUNSUPPORTED;
    if (a->B == 0) return SV_OK;
    if ((a->kind == SV_PAGES_RESERVE || a->kind == SV_PAGES_COMMIT) && (a->rows < 0 || a->rows > SV_MAX_CACHE_TOKENS)) return SV_EINVAL;
    if (a->kind == SV_PAGES_FORK && (!a->granted || !a->from_slots || !a->copies || a->max_copies < a->B)) return SV_EINVAL;
    if (a->kind == SV_PAGES_FORK && (uintptr_t)a->copies % 8) return SV_EINVAL;
    return SV_OK;
}

int spec_verify_pages(spec_verify_t* h, const spec_verify_pages_args* a, void* hip_stream)
{
    if (!h) return SV_EINVAL;
    const spec_verify_config* cfg = sv::handle_config(h);
    const int rc = spec_verify_pages_check(cfg, a);
    if (rc != SV_OK) return rc;
    DeviceGuard guard(cfg->device);
    hipStream_t s = (hipStream_t)hip_stream;
    Pages q;
    q.c = sv::cache_of(a->cache);
    q.B = a->B;
    q.kind = a->kind;
    q.slots = a->slots;
    q.from = a->from_slots;
    q.rows = a->rows;
    q.last = a->last_row;
    q.granted = a->granted;
    q.copies = (int2*)a->copies;
    q.max_copies = a->max_copies;
    q.status = a->device_status;
    hipError_t e = hipSuccess;
    auto launch = [&](auto kernel, long long groups, int threads, auto what) {
        if (e == hipSuccess) e = launch_kernel(kernel, dim3((unsigned)groups), dim3(threads), 0, s, nullptr, nullptr, what);
    };
    if (a->kind == SV_PAGES_CLEAR) {
        const long long most = std::max((long long)q.c.n_slots * q.c.max_pages, (long long)q.c.n_pages);
        e = clear_status(q.status, s);
        launch(sv_pages_clear_kernel, std::min((most + kThreads - 1) / kThreads, 4096ll), kThreads, q.c);
    } else if (a->kind == SV_PAGES_COMPACT) {
        launch(sv_pages_pair_kernel, 1, kPlan, q);
        launch(sv_pages_rename_kernel, std::min(q.c.n_slots, 1 << 16), kThreads, q.c);
        if (q.max_copies) launch(sv_pages_left_kernel, std::min((q.max_copies + kThreads - 1) / kThreads, 1024), kThreads, q);
    } else if (a->B == 0) {
        e = clear_status(q.status, s);
    } else if (a->kind == SV_PAGES_COMMIT || a->kind == SV_PAGES_RELEASE) {
        e = clear_status(q.status, s);
        launch(sv_pages_back_kernel, q.B, kThreads, q);
    } else {
        // us of a release and a reservation for 256 sequences of 512 in a pool of 600000 pages, in
        // one launch and in two: 75 pages each 30 and 39, 150 each 36 and 41, 560 each 72 and 50
        const long long may = q.kind == SV_PAGES_RESERVE ? (long long)q.B * ((q.rows >> q.c.shift) + 1) : 0;
        if (may > 65536) {
            launch(sv_pages_give_kernel<GIVE_TABLES>, (q.c.n_pages + 32 * kPlan - 1) / (32 * kPlan), kPlan, q);
            launch(sv_pages_give_kernel<GIVE_STATE>, 1, kPlan, q);
        } else {
            launch(sv_pages_give_kernel<GIVE_ALL>, 1, kPlan, q);
        }
        if (a->kind == SV_PAGES_FORK) launch(sv_pages_share_kernel, q.B, kThreads, q);
    }
    return status_of(e);
}

int spec_verify_pages_copy_check(const spec_verify_config* cfg, const spec_verify_pages_copy_args* a)
{
    int rc = sv::check_config(cfg);
    if (rc != SV_OK) return rc;
    if (!a) return SV_EINVAL;
    if (a->n_copies < 0 || a->n_copies > SV_MAX_PAGES || a->n_pages < 1 || a->n_pages > SV_MAX_PAGES) return SV_EINVAL;
    if (a->n_pools < 1 || a->n_pools > 65535) return SV_EINVAL;
    if (a->page_bytes < 16 || a->page_bytes % 16 || a->page_stride < a->page_bytes || a->page_stride % 16) return SV_EINVAL;
    if (a->page_bytes > (1 << 30) || a->page_stride > (1ll << 40)) return SV_EUNSUPPORTED;
    // (n_pages * page_stride might not fit 63 bits)
    if (a->n_pools > 1 && (a->pool_stride % 16 || a->pool_stride / a->n_pages < a->page_stride)) return SV_EINVAL;
    if (a->n_pools > 1 && a->pool_stride > (1ll << 46)) return SV_EUNSUPPORTED;
    if (a->n_copies && (!a->copies || !a->pools || (uintptr_t)a->pools % 16 || (uintptr_t)a->copies % 8)) return SV_EINVAL;
    return SV_OK;
}

int spec_verify_pages_copy(spec_verify_t* h, const spec_verify_pages_copy_args* a, void* hip_stream)
{
    if (!h) return SV_EINVAL;
    const spec_verify_config* cfg = sv::handle_config(h);
    const int rc = spec_verify_pages_copy_check(cfg, a);
    if (rc != SV_OK) return rc;
    DeviceGuard guard(cfg->device);
    hipStream_t s = (hipStream_t)hip_stream;
    Copy q;
    q.copies = (const int2*)a->copies;
    q.n_pages = a->n_pages;
    q.n_pools = (unsigned)a->n_pools;
    q.pools = (char*)a->pools;
    q.pool_stride = a->n_pools > 1 ? a->pool_stride : 0;
    q.page_stride = a->page_stride;
    q.units = (int)(a->page_bytes / 16);
    q.parts = (unsigned)((q.units + kThreads * kCopyUnits - 1) / (kThreads * kCopyUnits));
    q.total = (long long)a->n_copies * a->n_pools * q.parts;
    q.status = a->device_status;
    hipError_t e = clear_status(q.status, s);
    if (e == hipSuccess && q.total)
        e = launch_kernel(sv_pages_copy_kernel, dim3((unsigned)std::min(q.total, 1ll << 16)), dim3(kThreads), 0, s, nullptr, nullptr, q);
    return status_of(e);
}

int spec_verify_append_check(const spec_verify_config* cfg, const spec_verify_append_args* a)
{
    int rc = sv::check_config(cfg);
    if (rc != SV_OK) return rc;
    if (!a) return SV_EINVAL;
    rc = sv::check_cache(a->cache, false);
    if (rc == SV_OK) rc = sv::check_kv(a->kv);
    if (rc == SV_OK) rc = sv::check_rows(cfg, a->B, a->cache, a->slots, a->last_row, a->row_offsets);
    if (rc != SV_OK) return rc;
    if (a->rows < 1 || a->rows > SV_MAX_PAGE_ROWS || a->row0 < 0 || a->row0 > SV_MAX_PAGE_ROWS) return SV_EINVAL;
    // (a sequence's units are counted in 32 bits)
    if ((long long)a->rows * a->kv.kv_heads * (a->kv.head_dim / 8) > 0x7fffffffll) return SV_EUNSUPPORTED;
    if (a->B == 0) return SV_OK;
    if (!a->keys || !a->values) return SV_EINVAL;
    if (a->row_stride < a->kv.head_dim || a->head_stride < a->kv.head_dim || (!a->row_offsets && a->batch_stride < 0)) return SV_EINVAL;
    return SV_OK;
}

int spec_verify_append(spec_verify_t* h, const spec_verify_append_args* a, void* hip_stream)
{
    if (!h) return SV_EINVAL;
    const spec_verify_config* cfg = sv::handle_config(h);
    const int rc = spec_verify_append_check(cfg, a);
    if (rc != SV_OK) return rc;
    DeviceGuard guard(cfg->device);
    hipStream_t s = (hipStream_t)hip_stream;
    const bool e4m3 = a->kv.type == SV_KV_E4M3;
    const int es = e4m3 ? 1 : 2, unit = 16 / es;
    Append q;
    q.c = sv::cache_of(a->cache);
    q.r = sv::Rows{a->rows, a->row0, a->slots, a->last_row, (const long long*)a->row_offsets};
    q.kv_heads = a->kv.kv_heads;
    q.per_head = a->kv.head_dim / unit;
    q.k = (const unsigned short*)a->keys;
    q.v = (const unsigned short*)a->values;
    q.bs = a->batch_stride;
    q.rs = a->row_stride;
    q.hs = a->head_stride;
    q.keys = (char*)a->kv.keys;
    q.values = (char*)a->kv.values;
    q.page_stride = a->kv.page_stride * es;
    q.head_stride = a->kv.head_stride * es;
    q.token_stride = a->kv.token_stride * es;
    q.kscale = a->kv.key_scales;
    q.vscale = a->kv.value_scales;
    q.status = a->device_status;
    hipError_t e = clear_status(q.status, s);
    const long long units = (long long)a->rows * q.kv_heads * q.per_head;
    const unsigned groups = (unsigned)std::min((units + kThreads - 1) / kThreads, 1024ll);
    constexpr int kMostB = 8192; // groups * B * 256 stays within 2^32 - 1
    for (q.b0 = 0; q.b0 < a->B && e == hipSuccess; q.b0 += kMostB) {
        const dim3 grid(groups, (unsigned)std::min(a->B - q.b0, kMostB));
        e = e4m3 ? launch_kernel(sv_append_kernel<true>, grid, dim3(kThreads), 0, s, nullptr, nullptr, q)
                 : launch_kernel(sv_append_kernel<false>, grid, dim3(kThreads), 0, s, nullptr, nullptr, q);
    }
    return status_of(e);
}

} // extern "C"
