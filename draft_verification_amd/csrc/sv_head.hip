// Output head with 4-bit weights (spec_verify_head in include/spec_verify.h).
//
// y[m][v] = sum_k x[m][k] W[v][k] as a matrix-core product with the vocabulary
// as the rows of the tile and the hidden rows as its 16 columns: the weights
// are widened to bf16 in registers, where each is exact, so the only rounding
// before the result's is that of the fp32 sums.

#include <math.h>

#include <algorithm>

#include "spec_verify.h"
#include "sv_host.h"

using sv::DeviceGuard;
using sv::launch_kernel;

namespace {

constexpr int kThreads = 256;
constexpr int kStrip = 64;   // vocabulary rows of a strip: 4 matrix-core tiles of 16
constexpr int kStep = 128;   // values of k of a step: 4 products of 32

// Packed weights.  A block of 4 KB is one strip over one step; the blocks of a
// strip follow each other.  In it, tile t's 1 KB holds lane l's 16 bytes at
// l * 16, so that a wavefront's load is contiguous.  Lane l = (r, g) with r =
// l % 16 and g = l / 16 is row r of the tile, and word w of its 16 bytes are
// the 8 values of k that it feeds to product w:
//   FP4:  k = 128 step + 32 g + 8 w ..  (a lane's 32 values share one scale)
//   INT4: k = 128 step + 32 w + 8 g ..  (a product's 32 values share one scale)
// Row r of tile t is vocabulary row 64 strip + 16 (r / 4) + 4 t + r % 4: the
// product leaves a lane with rows 4 g .. 4 g + 3 of each tile, which makes them
// 16 consecutive tokens.
// After all blocks, the scales: FP4, per block and lane the four tiles' scale
// bytes; INT4, per block and group of the step 64 bf16 in vocabulary order.
// Rows past V and values past the hidden size are zero.
struct Layout {
    int V, H, group;
    int steps;            // steps of a strip
    long long strips;
    int groups;           // INT4: groups of a step
    long long scale_at;   // byte offset of the scales
    long long bytes;
};

Layout layout_of(int V, int H, int format, int group)
{
    Layout y;
    y.V = V;
    y.H = H;
    y.group = group;
    y.steps = (H + kStep - 1) / kStep;
    y.strips = (V + kStrip - 1) / kStrip;
    y.groups = kStep / group;
    y.scale_at = y.strips * y.steps * 4096;
    y.bytes = y.scale_at + y.strips * y.steps * (format == SV_W4_FP4 ? 256 : (long long)y.groups * 128);
    return y;
}

__device__ __forceinline__ int vocab_row(int t, int r) { return 16 * (r >> 2) + 4 * t + (r & 3); }

struct Pack {
    Layout y;
    const unsigned char* w;
    long long ws;
    const unsigned char* s8;
    const unsigned short* s16;
    long long ss;
    unsigned* packed;
};

// One thread per 16 bytes of weights (a lane of a tile), and per lane its scales.
template <int FMT>
__global__ __launch_bounds__(kThreads) void sv_head_pack_kernel(Pack q)
{
    const long long n = q.y.strips * q.y.steps * 256; // 16-byte pieces
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kThreads) {
        const int lane = (int)(i & 63), t = (int)(i >> 6 & 3);
        const long long block = i >> 8;
        const int step = (int)(block % q.y.steps);
        const long long strip = block / q.y.steps;
        const int r = lane & 15, g = lane >> 4;
        const long long v = strip * kStrip + vocab_row(t, r);
        const bool row = v < q.y.V;
        for (int w = 0; w < 4; ++w) {
            const int k0 = step * kStep + (FMT == SV_W4_FP4 ? 32 * g + 8 * w : 32 * w + 8 * g);
            unsigned word = FMT == SV_W4_FP4 ? 0u : 0x88888888u;
            if (row && k0 < q.y.H) {
                const unsigned char* src = q.w + v * q.ws + k0 / 2;
                word = src[0] | (unsigned)src[1] << 8 | (unsigned)src[2] << 16 | (unsigned)src[3] << 24;
                if (FMT == SV_W4_INT4) {
                    // halves of value pairs apart: nibble p is value 2p, nibble p + 4 value 2p + 1
                    unsigned e = 0;
                    for (int p = 0; p < 4; ++p)
                        e |= (word >> (8 * p) & 15) << (4 * p) | (word >> (8 * p + 4) & 15) << (4 * p + 16);
                    word = e;
                }
            }
            q.packed[i * 4 + w] = word;
        }
        if (FMT == SV_W4_FP4) {
            if (t == 0) {
                unsigned word = 0;
                for (int u = 0; u < 4; ++u) {
                    const long long vu = strip * kStrip + vocab_row(u, r);
                    const int grp = step * 4 + g;
                    const unsigned s = vu < q.y.V && grp * 32 < q.y.H ? q.s8[vu * q.ss + grp] : 127u;
                    word |= s << (8 * u);
                }
                q.packed[q.y.scale_at / 4 + block * 64 + lane] = word;
            }
        } else if (t < q.y.groups) {
            const long long vl = strip * kStrip + lane;
            const int grp = step * q.y.groups + t;
            const unsigned short s = vl < q.y.V && grp * q.y.group < q.y.H ? q.s16[vl * q.ss + grp] : (unsigned short)0;
            ((unsigned short*)q.packed)[q.y.scale_at / 2 + (block * q.y.groups + t) * 64 + lane] = s;
        }
    }
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// 8 weights of a word as bf16, exactly.  FP4: times their scale.
__device__ __forceinline__ bf16x8 widen_fp4(unsigned w, float scale)
{
    union { bf16x2 p[4]; bf16x8 v; } u;
    u.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
    u.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    u.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
    u.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    return u.v;
}

// INT4: code + 16, whose bf16 has the code in the top four bits of its
// fraction: a shift, a mask and the exponent of 16 make two of them at once.
__device__ __forceinline__ bf16x8 widen_int4(unsigned w)
{
    union { unsigned u[4]; bf16x8 v; } u;
    u.u[0] = (w << 3 & 0x00780078u) | 0x41804180u;
    u.u[1] = (w >> 1 & 0x00780078u) | 0x41804180u;
    u.u[2] = (w >> 5 & 0x00780078u) | 0x41804180u;
    u.u[3] = (w >> 9 & 0x00780078u) | 0x41804180u;
    return u.v;
}

struct Head {
    Layout y;
    const unsigned char* packed;
    int M;
    const unsigned short* x;
    long long xs;
    void* out;
    long long os;
    long long nwg; // workgroups of four strips in a row block
};

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__bf16* p, float v) { *p = (__bf16)v; }

// One wavefront per strip and 16 rows.
template <int FMT, int GROUPS, typename OUT>
__global__ __launch_bounds__(kThreads) void sv_head_kernel(Head q)
{
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const long long strip = (long long)(blockIdx.x % q.nwg) * 4 + (threadIdx.x >> 6);
    if (strip >= q.y.strips) return;
    const int m = (int)(blockIdx.x / q.nwg) * 16 + c;
    const unsigned short* x = q.x + (long long)m * q.xs;
    f32x4 acc[4] = {};
    bf16x8 ones;
#pragma unroll
    for (int k = 0; k < 8; ++k) ones[k] = (__bf16)1.0f;

    for (int step = 0; step < q.y.steps; ++step) {
        const long long block = strip * q.y.steps + step;
        u32x4 w[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = *(const u32x4*)(q.packed + (block * 4 + t) * 1024 + lane * 16);
        bf16x8 b[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int k = step * kStep + (FMT == SV_W4_FP4 ? 32 * g + 8 * p : 32 * p + 8 * g);
            u32x4 raw = {0, 0, 0, 0};
            if (m < q.M && k < q.y.H) raw = *(const u32x4_any*)(x + k);
            b[p] = __builtin_bit_cast(bf16x8, raw);
        }
        if constexpr (FMT == SV_W4_FP4) {
            const unsigned sc = *(const unsigned*)(q.packed + q.y.scale_at + (block * 64 + lane) * 4);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const unsigned e = sc >> (8 * t) & 255u;
                const float s = __uint_as_float(e ? e << 23 : 0x00400000u);
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_fp4(w[t][p], s), b[p], acc[t], 0, 0, 0);
            }
        } else {
            constexpr int P = 4 / GROUPS; // products of a group
#pragma unroll
            for (int u = 0; u < GROUPS; ++u) {
                const unsigned char* sp = q.packed + q.y.scale_at + ((block * GROUPS + u) * 64 + 16 * g) * 2;
                const u32x4 s0 = *(const u32x4*)sp, s1 = *(const u32x4*)(sp + 16);
                f32x4 sum = {}; // of x over the group, in every row
#pragma unroll
                for (int p = u * P; p < u * P + P; ++p)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, b[p], sum, 0, 0, 0);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    f32x4 d = {};
#pragma unroll
                    for (int p = u * P; p < u * P + P; ++p)
                        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_int4(w[t][p]), b[p], d, 0, 0, 0);
                    const unsigned lo = t < 2 ? s0[t * 2] : s1[t * 2 - 4], hi = t < 2 ? s0[t * 2 + 1] : s1[t * 2 - 3];
                    const float s[4] = {__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u),
                                        __uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)};
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[t][i] += s[i] * (d[i] - 24.0f * sum[i]);
                }
            }
        }
    }
    if (m >= q.M) return;
    OUT* out = (OUT*)q.out + (long long)m * q.os;
    const long long v0 = strip * kStrip + 16 * g;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (v0 + 4 * t + i < q.y.V) put(out + v0 + 4 * t + i, acc[t][i]);
}

int check_weights(int32_t hidden, int32_t format, int32_t group)
{
    if (format != SV_W4_FP4 && format != SV_W4_INT4) return SV_EUNSUPPORTED;
    if (format == SV_W4_FP4 ? group != 32 : group != 32 && group != 64 && group != 128) return SV_EUNSUPPORTED;
    if (hidden < 1 || hidden > SV_MAX_HIDDEN || hidden % group) return SV_EINVAL;
    return SV_OK;
}

template <int FMT, int GROUPS>
hipError_t launch_head(Head q, bool bf16, hipStream_t s)
{
    q.nwg = (q.y.strips + 3) / 4;
    // launches of at most 2^32 - 1 work-items
    const int most = (int)std::min(0xffffffffll / kThreads / q.nwg, 1ll << 24) * 16;
    hipError_t e = hipSuccess;
    for (int left = q.M; left > 0 && e == hipSuccess; left -= most) {
        q.M = std::min(left, most);
        const dim3 grid((unsigned)(q.nwg * ((q.M + 15) / 16)));
        if (bf16) e = launch_kernel(sv_head_kernel<FMT, GROUPS, __bf16>, grid, dim3(kThreads), 0, s, nullptr, nullptr, q);
        else e = launch_kernel(sv_head_kernel<FMT, GROUPS, float>, grid, dim3(kThreads), 0, s, nullptr, nullptr, q);
        q.x += (long long)most * q.xs;
        q.out = (char*)q.out + (long long)most * q.os * (bf16 ? 2 : 4);
    }
    return e;
}

} // namespace

extern "C" {

int64_t spec_verify_head_packed_bytes(const spec_verify_config* cfg, int32_t hidden, int32_t format, int32_t group)
{
    int rc = sv::check_config(cfg);
    if (rc == SV_OK) rc = check_weights(hidden, format, group);
    if (rc != SV_OK) return rc;
    return layout_of(cfg->vocab, hidden, format, group).bytes;
}

int spec_verify_head_pack_check(const spec_verify_config* cfg, const spec_verify_head_pack_args* a)
{
    int rc = sv::check_config(cfg);
    if (rc != SV_OK) return rc;
    if (!a) return SV_EINVAL;
    rc = check_weights(a->hidden, a->format, a->group);
    if (rc != SV_OK) return rc;
    if (!a->weights || !a->scales || !a->packed || (uintptr_t)a->packed % 16) return SV_EINVAL;
    if (a->weight_stride < a->hidden / 2 || a->scale_stride < a->hidden / a->group) return SV_EINVAL;
    return SV_OK;
}

int spec_verify_head_pack(spec_verify_t* h, const spec_verify_head_pack_args* a, void* hip_stream)
{
    if (!h) return SV_EINVAL;
    const spec_verify_config* cfg = sv::handle_config(h);
    int rc = spec_verify_head_pack_check(cfg, a);
    if (rc != SV_OK) return rc;
    DeviceGuard guard(cfg->device);
    Pack q;
    q.y = layout_of(cfg->vocab, a->hidden, a->format, a->group);
    q.w = (const unsigned char*)a->weights;
    q.ws = a->weight_stride;
    q.s8 = (const unsigned char*)a->scales;
    q.s16 = (const unsigned short*)a->scales;
    q.ss = a->scale_stride;
    q.packed = (unsigned*)a->packed;
    const dim3 grid((unsigned)std::min(q.y.strips * q.y.steps, 1ll << 20));
    hipStream_t s = (hipStream_t)hip_stream;
    hipError_t e = a->format == SV_W4_FP4
        ? launch_kernel(sv_head_pack_kernel<SV_W4_FP4>, grid, dim3(kThreads), 0, s, nullptr, nullptr, q)
        : launch_kernel(sv_head_pack_kernel<SV_W4_INT4>, grid, dim3(kThreads), 0, s, nullptr, nullptr, q);
    return e == hipSuccess ? SV_OK : SV_EDEVICE;
}

int spec_verify_head_check(const spec_verify_config* cfg, const spec_verify_head_args* a)
{
    int rc = sv::check_config(cfg);
    if (rc != SV_OK) return rc;
    if (!a) return SV_EINVAL;
    rc = check_weights(a->hidden, a->format, a->group);
    if (rc != SV_OK) return rc;
    if (a->rows < 0 || a->rows > (long long)cfg->max_batch * (cfg->max_draft + 1)) return SV_EINVAL;
    if (a->rows == 0) return SV_OK;
    if (!a->packed || (uintptr_t)a->packed % 16 || !a->hidden_states || !a->logits) return SV_EINVAL;
    if (a->hidden_stride < a->hidden || a->logits_stride < cfg->vocab) return SV_EINVAL;
    return SV_OK;
}

int spec_verify_head(spec_verify_t* h, const spec_verify_head_args* a, void* hip_stream)
{
    if (!h) return SV_EINVAL;
    const spec_verify_config* cfg = sv::handle_config(h);
    int rc = spec_verify_head_check(cfg, a);
    if (rc != SV_OK) return rc;
    if (a->rows == 0) return SV_OK;
    DeviceGuard guard(cfg->device);
    hipStream_t s = (hipStream_t)hip_stream;
    Head q;
    q.y = layout_of(cfg->vocab, a->hidden, a->format, a->group);
    q.packed = (const unsigned char*)a->packed;
    q.M = a->rows;
    q.x = (const unsigned short*)a->hidden_states;
    q.xs = a->hidden_stride;
    q.out = a->logits;
    q.os = a->logits_stride;
    q.nwg = 0;
    const bool bf16 = cfg->dtype == SV_BF16;
    hipError_t e;
    if (a->format == SV_W4_FP4) e = launch_head<SV_W4_FP4, 4>(q, bf16, s);
    else if (a->group == 32) e = launch_head<SV_W4_INT4, 4>(q, bf16, s);
    else if (a->group == 64) e = launch_head<SV_W4_INT4, 2>(q, bf16, s);
    else e = launch_head<SV_W4_INT4, 1>(q, bf16, s);
    return e == hipSuccess ? SV_OK : SV_EDEVICE;
}

} // extern "C"
