// The target's cache as its kernels take it: which rows a sequence has, where
// its tokens lie, and the host checks that its entry points share.
#ifndef SV_CACHE_H
#define SV_CACHE_H

#include <hip/hip_runtime.h>

#include "spec_verify.h"

namespace sv {

struct Cache {
    int n_slots, n_pages, max_pages;
    int shift; // log2 of the page size
    int* table;
    int* lengths;
    int* counts;
    int* refs;
    unsigned* free;
};

struct Rows {
    int rows, row0;
    const int* slots;
    const int* last_row;
    const long long* roff;
};

__device__ __forceinline__ void cache_status(int* status, int bits)
{
    if (status) __hip_atomic_fetch_or(status, bits, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A barrier for LDS alone: what is under way from and to memory stays so.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A value that every lane reads alike and nothing writes while the kernel runs, through
// the scalar cache.
template <typename T>
__device__ __forceinline__ T cache_uniform(const T* p)
{
    return *(const __attribute__((address_space(4))) T*)(uintptr_t)p;
}

// What the call does for a sequence: its slot, its rows (count; first of a packed
// batch) and the position of row 0.  A bad sequence has -1 rows.
struct Sequence {
    int slot, count, start;
    long long first;
};

// (UNIFORM: every lane asks for the same b)
template <bool UNIFORM = true>
__device__ __forceinline__ Sequence sequence_of(const Cache& c, const Rows& q, int b)
{
    auto get = [](const auto* p) {
        if constexpr (UNIFORM) return cache_uniform(p);
        else return *p;
    };
    Sequence s;
    s.slot = q.slots ? get(q.slots + b) : b;
    s.count = -1;
    s.start = 0;
    s.first = 0;
    if (s.slot == -1) {
        s.count = 0;
        return s;
    }
    if (s.slot < 0 || s.slot >= c.n_slots) return s;
    int n = q.rows;
    if (q.roff) {
        s.first = get(q.roff + b);
        const long long end = get(q.roff + b + 1);
        if (s.first < 0 || end < s.first || end - s.first > q.rows) return s;
        n = (int)(end - s.first);
    } else if (q.last_row) {
        const int last = get(q.last_row + b);
        if (last < -1) return s;
        if (last < n) n = last + 1;
    }
    if (n == 0) { // nothing is looked at
        s.count = 0;
        return s;
    }
    const int len = get(c.lengths + s.slot);
    const int held = c.counts ? min(get(c.counts + s.slot), c.max_pages) : c.max_pages;
    if (len < 0 || (long long)len + q.row0 + n > ((long long)held << c.shift)) return s;
    s.start = len + q.row0;
    s.count = n;
    return s;
}

// Host: the device's view of a cache; and its checks (full: the arrays that only
// spec_verify_pages uses are wanted too).
inline Cache cache_of(const spec_verify_cache& a)
{
    return Cache{a.n_slots, a.n_pages, a.max_pages, __builtin_ctz((unsigned)a.page_size),
                 a.page_table, a.lengths, a.page_counts, a.page_refs, a.free_pages};
}

inline int check_cache(const spec_verify_cache& c, bool full)
{
    if (c.n_slots < 1 || c.n_pages < 1 || c.page_size < 1 || c.max_pages < 1) return SV_EINVAL;
    if (c.n_slots > SV_MAX_BATCH || c.n_pages > SV_MAX_PAGES || c.page_size > SV_MAX_PAGE_SIZE) return SV_EUNSUPPORTED;
    if (c.page_size & (c.page_size - 1)) return SV_EUNSUPPORTED;
    if ((long long)c.max_pages * c.page_size > SV_MAX_CACHE_TOKENS) return SV_EUNSUPPORTED;
    if (!c.page_table || !c.lengths) return SV_EINVAL;
    if (full && (!c.page_counts || !c.page_refs || !c.free_pages)) return SV_EINVAL;
    return SV_OK;
}

inline int check_kv(const spec_verify_kv& k)
{
    if (k.type != SV_KV_BF16 && k.type != SV_KV_E4M3) return SV_EUNSUPPORTED;
    if (k.kv_heads < 1 || k.head_dim < 1) return SV_EINVAL;
    if (k.kv_heads > 1024 || k.head_dim > SV_MAX_HEAD_DIM || k.head_dim % 16) return SV_EUNSUPPORTED;
    if (!k.keys || !k.values || (uintptr_t)k.keys % 16 || (uintptr_t)k.values % 16) return SV_EINVAL;
    const int unit = k.type == SV_KV_BF16 ? 8 : 16; // elements of 16 bytes
    for (const int64_t s : {k.page_stride, k.head_stride, k.token_stride})
        if (s < k.head_dim || s % unit || s > (1ll << 40)) return SV_EINVAL;
    return SV_OK;
}

inline int check_rows(const spec_verify_config* cfg, int32_t B, const spec_verify_cache& c, const int32_t* slots,
                      const int32_t* last_row, const int64_t* row_offsets)
{
    if (B < 0 || B > cfg->max_batch) return SV_EINVAL;
    if (!slots && c.n_slots < B) return SV_EINVAL;
    if (last_row && row_offsets) return SV_EINVAL;
    return SV_OK;
}

} // namespace sv

#endif // SV_CACHE_H
