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
// the 8 values k = 128 step + 32 w + 8 g .. that it feeds to product w.  (So a
// product's 32 values share one scale, and the hidden values of a product are
// 64 contiguous bytes of each row.)
// Row r of tile t is vocabulary row 64 strip + 16 (r / 4) + 4 t + r % 4: the
// product leaves a lane with rows 4 g .. 4 g + 3 of each tile, which makes them
// 16 consecutive tokens.
// After all blocks, the scales: FP4, per block and row r the words of the four
// tiles, byte w the scale of product w; INT4, per block and group of the step
// 64 bf16 in vocabulary order.
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
            const int k0 = step * kStep + 32 * w + 8 * g;
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
            if (g == 0) {
                unsigned word = 0;
                for (int w = 0; w < 4; ++w) {
                    const int grp = step * 4 + w;
                    const unsigned s = row && grp * 32 < q.y.H ? q.s8[v * q.ss + grp] : 127u;
                    word |= s << (8 * w);
                }
                q.packed[q.y.scale_at / 4 + block * 64 + r * 4 + t] = word;
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

// Scale byte p of a word as the exponent of a float, which is all that the
// conversion reads of it (255: NaN).
__device__ __forceinline__ float fp4_scale(unsigned word, int p)
{
    return __uint_as_float((p == 3 ? word >> 1 : word << (23 - 8 * p)) & 0x7f800000u);
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

// acc += the INT4 scales of tile t's four rows (in the tile pair's 16 bytes) * d
__device__ __forceinline__ void add_scaled(f32x4& acc, f32x4 d, u32x4 s, int t)
{
    const unsigned lo = s[t % 2 * 2], hi = s[t % 2 * 2 + 1];
    acc[0] = fmaf(__uint_as_float(lo << 16), d[0], acc[0]);
    acc[1] = fmaf(__uint_as_float(lo & 0xffff0000u), d[1], acc[1]);
    acc[2] = fmaf(__uint_as_float(hi << 16), d[2], acc[2]);
    acc[3] = fmaf(__uint_as_float(hi & 0xffff0000u), d[3], acc[3]);
}

struct Head {
    Layout y;
    const unsigned char* packed;
    int M;
    const unsigned short* x;
    long long xs;
    void* out;
    long long os;
    unsigned nstrip; // strips, as the grid counts them
    unsigned nblock; // row blocks
};

__device__ __forceinline__ void put4(float* p, f32x4 v, int n)
{
    typedef float any __attribute__((ext_vector_type(4), aligned(4)));
    if (n >= 4) *(any*)p = v;
    else
        for (int i = 0; i < n; ++i) p[i] = v[i];
}

__device__ __forceinline__ void put4(__bf16* p, f32x4 v, int n)
{
    typedef __bf16 any __attribute__((ext_vector_type(4), aligned(2)));
    if (n >= 4) *(any*)p = __builtin_convertvector(v, any);
    else
        for (int i = 0; i < n; ++i) p[i] = (__bf16)v[i];
}

// One lane's part of a step: its weights of the four tiles, the scales, and 32
// hidden values of one row.
template <int FMT, int GROUPS>
struct Part {
    u32x4 w[4];
    u32x4 x[4];
    u32x4 s[FMT == SV_W4_INT4 ? 2 * GROUPS : 1];

    __device__ __forceinline__ void load(const Head& q, long long block, int step, int lane, const unsigned short* x, bool row)
    {
        const int g = lane >> 4;
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = __builtin_nontemporal_load((const u32x4*)(q.packed + block * 4096 + t * 1024 + lane * 16));
        if constexpr (FMT == SV_W4_FP4) {
            s[0] = __builtin_nontemporal_load((const u32x4*)(q.packed + q.y.scale_at + block * 256 + (lane & 15) * 16));
        } else {
            const unsigned char* sp = q.packed + q.y.scale_at + block * (GROUPS * 128) + g * 32;
#pragma unroll
            for (int u = 0; u < GROUPS; ++u) {
                s[2 * u] = *(const u32x4*)(sp + u * 128);
                s[2 * u + 1] = *(const u32x4*)(sp + u * 128 + 16);
            }
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int k = step * kStep + 32 * p + 8 * g;
            this->x[p] = u32x4{0, 0, 0, 0};
            if (row && k < q.y.H) this->x[p] = *(const u32x4_any*)(x + k);
        }
    }

    __device__ __forceinline__ void add(f32x4* acc) const
    {
        if constexpr (FMT == SV_W4_FP4) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_fp4(w[t][p], fp4_scale(s[0][t], p)), __builtin_bit_cast(bf16x8, x[p]), acc[t], 0, 0, 0);
        } else {
            constexpr int P = 4 / GROUPS; // products of a group
            bf16x8 ones;
#pragma unroll
            for (int k = 0; k < 8; ++k) ones[k] = (__bf16)1.0f;
#pragma unroll
            for (int u = 0; u < GROUPS; ++u) {
                f32x4 sum = {}; // of x over the group, in every row
#pragma unroll
                for (int p = u * P; p < u * P + P; ++p)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, __builtin_bit_cast(bf16x8, x[p]), sum, 0, 0, 0);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    f32x4 d = sum * -24.0f;
#pragma unroll
                    for (int p = u * P; p < u * P + P; ++p)
                        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_int4(w[t][p]), __builtin_bit_cast(bf16x8, x[p]), d, 0, 0, 0);
                    add_scaled(acc[t], d, s[2 * u + t / 2], t);
                }
            }
        }
    }
};

// Up to 16 rows: one workgroup of WK wavefronts per strip, which take its steps
// in turn (so that the workgroup reads WK blocks, one after the other in
// memory, at a time), each with the next step's loads under way, and join
// their sums in LDS.  Bound by the weights' HBM bytes.
template <int FMT, int GROUPS, int WK, typename OUT>
__global__ __launch_bounds__(64 * WK) void sv_head_rows_kernel(Head q)
{
    __shared__ f32x4 part[WK][4][64];
    const int lane = threadIdx.x & 63, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long long strip = blockIdx.x % q.nstrip;
    const int m = (int)(blockIdx.x / q.nstrip) * 16 + c;
    const unsigned short* x = q.x + (long long)m * q.xs;
    const bool row = m < q.M;
    f32x4 acc[4] = {};

    const long long first = strip * q.y.steps;
    Part<FMT, GROUPS> a, b;
    int step = wave;
    if (step < q.y.steps) a.load(q, first + step, step, lane, x, row);
    while (step < q.y.steps) {
        if (step + WK < q.y.steps) b.load(q, first + step + WK, step + WK, lane, x, row);
        a.add(acc);
        step += WK;
        if (step >= q.y.steps) break;
        if (step + WK < q.y.steps) a.load(q, first + step + WK, step + WK, lane, x, row);
        b.add(acc);
        step += WK;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    if (wave >= 4) return;
    f32x4 sum = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < WK; ++w) sum += part[w][wave][lane];
    const long long v = strip * kStrip + 16 * (lane >> 4) + 4 * wave;
    if (row && v < q.y.V) put4((OUT*)q.out + (long long)m * q.os + v, sum, (int)(q.y.V - v));
}

// Workgroup barrier for LDS alone: global loads stay in flight across it.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The sum of 8 bf16 values.
__device__ __forceinline__ float sum8(u32x4 x)
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s += __uint_as_float(x[i] << 16) + __uint_as_float(x[i] & 0xffff0000u);
    return s;
}

// More rows: a workgroup computes 256 vocabulary rows, a strip to each of its
// four wavefronts, for 16 MT hidden rows, which they share through LDS.  Each
// step's hidden values are staged one step ahead, in the order in which the
// products take them (a wavefront stages product p = its number of every tile,
// so that both its LDS writes and all reads are contiguous); the weights go
// straight to the registers of the wavefront that needs them.
template <int FMT, int GROUPS, int MT, typename OUT>
__global__ __launch_bounds__(256, 2) void sv_head_tile_kernel(Head q)
{
    __shared__ u32x4 xt[2][MT][4][64];
    __shared__ float xsum[2][MT][4][16]; // INT4: -24 times the sum of a product's hidden values
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Workgroups go round the eight dies: the row blocks of one strip group
    // follow each other on one die, whose L2 then holds its weights.
    const unsigned die = blockIdx.x % 8, turn = blockIdx.x / 8;
    const unsigned group = turn / q.nblock * 8 + die;
    if (group * 4ll >= q.y.strips) return;
    const int m0 = (int)(turn % q.nblock) * (16 * MT);
    const int tiles = min(MT, (q.M - m0 + 15) / 16);
    const long long strip = min(group * 4ll + wave, q.y.strips - 1); // past the last: computed, not stored
    const long long first = strip * q.y.steps;

    u32x4 xr[MT];
    auto load_x = [&](int step) {
        const int k = step * kStep + 32 * wave + 8 * g;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = m0 + 16 * mt + c;
            xr[mt] = u32x4{0, 0, 0, 0};
            if (m < q.M && k < q.y.H) xr[mt] = *(const u32x4_any*)(q.x + (long long)m * q.xs + k);
        }
    };
    auto stage_x = [&](int buf) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            xt[buf][mt][wave][lane] = xr[mt];
            if constexpr (FMT == SV_W4_INT4) {
                float s = sum8(xr[mt]);
                s += __shfl_xor(s, 16);
                s += __shfl_xor(s, 32);
                if (g == 0) xsum[buf][mt][wave][c] = -24.0f * s;
            }
        }
    };
    u32x4 w[4], s[FMT == SV_W4_INT4 ? 2 * GROUPS : 1];
    auto load_w = [&](int step) {
        const long long block = first + step;
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = *(const u32x4*)(q.packed + block * 4096 + t * 1024 + lane * 16);
        if constexpr (FMT == SV_W4_FP4) {
            s[0] = *(const u32x4*)(q.packed + q.y.scale_at + block * 256 + c * 16);
        } else {
            const unsigned char* sp = q.packed + q.y.scale_at + block * (GROUPS * 128) + g * 32;
#pragma unroll
            for (int u = 0; u < GROUPS; ++u) {
                s[2 * u] = *(const u32x4*)(sp + u * 128);
                s[2 * u + 1] = *(const u32x4*)(sp + u * 128 + 16);
            }
        }
    };

    f32x4 acc[MT][4] = {};
    load_x(0);
    load_w(0);
    stage_x(0);
    if (q.y.steps > 1) load_x(1);
    for (int step = 0; step < q.y.steps; ++step) {
        const int buf = step & 1;
        u32x4 wn[4], sn[FMT == SV_W4_INT4 ? 2 * GROUPS : 1];
#pragma unroll
        for (int t = 0; t < 4; ++t) wn[t] = w[t];
#pragma unroll
        for (int u = 0; u < (FMT == SV_W4_INT4 ? 2 * GROUPS : 1); ++u) sn[u] = s[u];
        lds_barrier();
        if (step + 1 < q.y.steps) {
            load_w(step + 1);
            stage_x(buf ^ 1);
            if (step + 2 < q.y.steps) load_x(step + 2);
        }
        constexpr int P = 4 / GROUPS; // products of a group (INT4)
        f32x4 d[FMT == SV_W4_INT4 ? MT : 1][4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            bf16x8 a[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                a[t] = FMT == SV_W4_FP4 ? widen_fp4(wn[t][p], fp4_scale(sn[0][t], p)) : widen_int4(wn[t][p]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (mt >= tiles) continue;
                const bf16x8 b = __builtin_bit_cast(bf16x8, xt[buf][mt][p][lane]);
                if constexpr (FMT == SV_W4_FP4) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) acc[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t], b, acc[mt][t], 0, 0, 0);
                } else {
                    if (p % P == 0) {
                        float z = xsum[buf][mt][p][c];
#pragma unroll
                        for (int o = 1; o < P; ++o) z += xsum[buf][mt][p + o][c];
#pragma unroll
                        for (int t = 0; t < 4; ++t) d[mt][t] = f32x4{z, z, z, z};
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) d[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t], b, d[mt][t], 0, 0, 0);
                    if (p % P == P - 1) {
#pragma unroll
                        for (int t = 0; t < 4; ++t) add_scaled(acc[mt][t], d[mt][t], sn[2 * (p / P) + t / 2], t);
                    }
                }
            }
        }
    }
    if (group * 4ll + wave >= q.y.strips) return;
    const long long v = strip * kStrip + 16 * g;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int m = m0 + 16 * mt + c;
        if (m >= q.M) continue;
        OUT* out = (OUT*)q.out + (long long)m * q.os + v;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (v + 4 * t < q.y.V) put4(out + 4 * t, acc[mt][t], (int)(q.y.V - v - 4 * t));
    }
}

int check_weights(int32_t hidden, int32_t format, int32_t group)
{
    if (format != SV_W4_FP4 && format != SV_W4_INT4) return SV_EUNSUPPORTED;
    if (format == SV_W4_FP4 ? group != 32 : group != 32 && group != 64 && group != 128) return SV_EUNSUPPORTED;
    if (hidden < 1 || hidden > SV_MAX_HIDDEN || hidden % group) return SV_EINVAL;
    return SV_OK;
}

template <int FMT, int GROUPS, int WK>
hipError_t launch_rows(Head q, bool bf16, hipStream_t s)
{
    q.nstrip = (unsigned)q.y.strips;
    // launches of at most 2^32 - 1 work-items
    const int most = (int)std::min(0xffffffffll / (64 * WK) / q.nstrip, 1ll << 24) * 16;
    hipError_t e = hipSuccess;
    for (int left = q.M; left > 0 && e == hipSuccess; left -= most) {
        q.M = std::min(left, most);
        const dim3 grid(q.nstrip * (unsigned)((q.M + 15) / 16));
        if (bf16) e = launch_kernel(sv_head_rows_kernel<FMT, GROUPS, WK, __bf16>, grid, dim3(64 * WK), 0, s, nullptr, nullptr, q);
        else e = launch_kernel(sv_head_rows_kernel<FMT, GROUPS, WK, float>, grid, dim3(64 * WK), 0, s, nullptr, nullptr, q);
        q.x += (long long)most * q.xs;
        q.out = (char*)q.out + (long long)most * q.os * (bf16 ? 2 : 4);
    }
    return e;
}

template <int FMT, int GROUPS, int MT>
hipError_t launch_tile(Head q, bool bf16, hipStream_t s)
{
    const long long groups = ((q.y.strips + 3) / 4 + 7) / 8 * 8;
    const int most = (int)std::min(0xffffffffll / 256 / groups, 1ll << 22) * (16 * MT);
    hipError_t e = hipSuccess;
    for (int left = q.M; left > 0 && e == hipSuccess; left -= most) {
        q.M = std::min(left, most);
        q.nblock = (unsigned)((q.M + 16 * MT - 1) / (16 * MT));
        const dim3 grid((unsigned)(groups * q.nblock));
        if (bf16) e = launch_kernel(sv_head_tile_kernel<FMT, GROUPS, MT, __bf16>, grid, dim3(256), 0, s, nullptr, nullptr, q);
        else e = launch_kernel(sv_head_tile_kernel<FMT, GROUPS, MT, float>, grid, dim3(256), 0, s, nullptr, nullptr, q);
        q.x += (long long)most * q.xs;
        q.out = (char*)q.out + (long long)most * q.os * (bf16 ? 2 : 4);
    }
    return e;
}

template <int FMT, int GROUPS>
hipError_t launch_head(const Head& q, bool bf16, hipStream_t s)
{
    if (q.M <= 16) return launch_rows<FMT, GROUPS, 4>(q, bf16, s);
    if (q.M <= 32) return launch_tile<FMT, GROUPS, 2>(q, bf16, s);
    return launch_tile<FMT, GROUPS, 4>(q, bf16, s);
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
    q.nstrip = q.nblock = 0;
    const bool bf16 = cfg->dtype == SV_BF16;
    hipError_t e;
    if (a->format == SV_W4_FP4) e = launch_head<SV_W4_FP4, 4>(q, bf16, s);
    else if (a->group == 32) e = launch_head<SV_W4_INT4, 4>(q, bf16, s);
    else if (a->group == 64) e = launch_head<SV_W4_INT4, 2>(q, bf16, s);
    else e = launch_head<SV_W4_INT4, 1>(q, bf16, s);
    return e == hipSuccess ? SV_OK : SV_EDEVICE;
}

} // extern "C"
