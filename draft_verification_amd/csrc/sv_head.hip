// Output head with 4-bit weights (spec_verify_head in include/spec_verify.h).
//
// y[m][v] = sum_k x[m][k] W[v][k] as a matrix-core product with the vocabulary
// as the rows of the tile and the hidden rows as its 16 columns: the weights
// are widened to bf16 in registers, where each is exact, so the only rounding
// before the result's is that of the fp32 sums.

#include <math.h>

#include <algorithm>

#include "spec_verify.h"
#include "sv_head_choice.h"
#include "sv_host.h"

using sv::DeviceGuard;
using sv::launch_kernel;

namespace {

constexpr int kThreads = 256;
constexpr int kStrip = sv::kHeadStrip; // vocabulary rows of a strip: 4 matrix-core tiles of 16
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
            if (FMT == SV_W4_INT4) word = word << 3 | word >> 29; // pair 0 where widening wants it
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
// conversion reads of it (0: 2^-127, 255: NaN).
__device__ __forceinline__ float fp4_scale(unsigned word, int p)
{
    return __uint_as_float((p == 3 ? word >> 1 : word << (23 - 8 * p)) & 0x7f800000u);
}

// INT4: code + 16, whose bf16 has the code in the top four bits of its
// fraction.  A word holds pair p of its eight codes at bits 3 + 4 p and 19 + 4 p
// (round the end), so a shift, none for pair 0, and one and-or make two of them.
// The and-or takes no literal and one scalar operand, so its constants are held
// in a scalar and a vector register.
struct Int4Bits {
    unsigned mask, expo;
    __device__ __forceinline__ Int4Bits() : mask(0x00780078u), expo(0x41804180u)
    {
        asm("" : "+s"(mask));
        asm("" : "+v"(expo));
    }
    __device__ __forceinline__ bf16x8 widen(unsigned w) const
    {
        union { unsigned u[4]; bf16x8 v; } u;
        u.u[0] = (w & mask) | expo;
        u.u[1] = (w >> 4 & mask) | expo;
        u.u[2] = (w >> 8 & mask) | expo;
        u.u[3] = ((w >> 12 | w << 20) & mask) | expo;
        return u.v;
    }
};

__device__ __forceinline__ void add_scaled(f32x4& acc, f32x4 d, f32x4 s)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(s[i], d[i], acc[i]);
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

// Orders a wavefront's LDS accesses among its own lanes (they execute in
// order; this keeps the compiler to it).
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Workgroup barrier for LDS alone: global loads stay in flight across it.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Hidden values of a 16-row tile in LDS.  Sixteen lanes read a row's 128
// values of a step (256 contiguous bytes: consecutive lanes in other rows would
// cost the address unit four times as much), lane n the chunk n of 8 of them,
// which lane (row, g = n % 4) of product n / 4 takes.  A chunk's 16 slots are
// turned by its number, so that writes and reads meet all banks.
__device__ __forceinline__ int x_slot(int chunk, int row) { return chunk * 16 + (row ^ chunk); }

// INT4: -24 times the sum of a product's 32 values of a row, in the lanes that
// hold its four chunks.
__device__ __forceinline__ float x_offset(u32x4 x)
{
    const bf16x2 ones = {(__bf16)1.0f, (__bf16)1.0f};
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned two = x[i]; // (a vector's element itself does not cast: the compiler takes element 0)
        s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, two), ones, s, false);
    }
    s += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(s), 0xb1, 0xf, 0xf, true)); // lane ^ 1
    s += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(s), 0x4e, 0xf, 0xf, true)); // lane ^ 2
    return -24.0f * s;
}

// Few rows, or few vocabulary rows: one workgroup of kRowWaves wavefronts per
// strip and 16 hidden rows.  The wavefronts take the strip's steps in turn, so
// that the workgroup reads kRowWaves blocks, one after the other in memory, at
// a time, and join their sums at the end.  Bound by the weights' HBM bytes: 6.9
// TB/s at one row, V = 129280, H = 7168, FP4 (72 us in a long run of calls, 76 in
// the first hundred after a pause).  Eight wavefronts with
// one step's loads each beat four with two steps' (the registers of the second
// leave fewer wavefronts) by 1 to 15%.  INT4's scales go through LDS, since a
// lane needs those of 16 rows (as loads from memory, they cost the address unit
// more than the weights: 65 us instead of 55 for one row at V = 129280, H =
// 4096, group 32).
constexpr int kRowWaves = 8;

template <int FMT, int GROUPS, typename OUT>
__global__ __launch_bounds__(64 * kRowWaves) void sv_head_rows_kernel(Head q)
{
    typedef unsigned short sraw __attribute__((ext_vector_type(GROUPS)));
    typedef float sfloat __attribute__((ext_vector_type(GROUPS)));
    __shared__ f32x4 part[kRowWaves][4][64]; // a wavefront's own until the sums are joined
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long long strip = blockIdx.x % q.nstrip;
    const int m = (int)(blockIdx.x / q.nstrip) * 16 + c;
    const unsigned short* row = q.x + (long long)m * q.xs;
    const bool there = m < q.M;
    const Int4Bits bits;
    bf16x8 ones;
#pragma unroll
    for (int k = 0; k < 8; ++k) ones[k] = (__bf16)1.0f;
    f32x4 acc[4] = {};

    for (int step = wave; step < q.y.steps; step += kRowWaves) {
        const long long block = strip * q.y.steps + step;
        u32x4 w[4], x[4], s4;
        sraw s2;
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = __builtin_nontemporal_load((const u32x4*)(q.packed + block * 4096 + t * 1024 + lane * 16));
        if constexpr (FMT == SV_W4_FP4) s4 = __builtin_nontemporal_load((const u32x4*)(q.packed + q.y.scale_at + block * 256 + c * 16));
        else s2 = __builtin_nontemporal_load((const sraw*)(q.packed + q.y.scale_at + block * (GROUPS * 128)) + lane);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int k = step * kStep + 32 * p + 8 * g;
            x[p] = u32x4{0, 0, 0, 0};
            if (there && k < q.y.H) x[p] = *(const u32x4_any*)(row + k);
        }
        if constexpr (FMT == SV_W4_FP4) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_fp4(w[t][p], fp4_scale(s4[t], p)), __builtin_bit_cast(bf16x8, x[p]), acc[t], 0, 0, 0);
        } else {
            sfloat f;
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) f[i] = __uint_as_float((unsigned)s2[i] << 16);
            f32x4* scales = part[wave][0]; // of the step's groups, in vocabulary order
            wave_sync();
            ((sfloat*)scales)[lane] = f;
            wave_sync();
            constexpr int P = 4 / GROUPS; // products of a group
#pragma unroll
            for (int u = 0; u < GROUPS; ++u) {
                f32x4 sum = {}; // of x over the group, in every row
#pragma unroll
                for (int p = u * P; p < u * P + P; ++p)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, __builtin_bit_cast(bf16x8, x[p]), sum, 0, 0, 0);
                sum *= -24.0f;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    f32x4 d = sum;
#pragma unroll
                    for (int p = u * P; p < u * P + P; ++p)
                        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bits.widen(w[t][p]), __builtin_bit_cast(bf16x8, x[p]), d, 0, 0, 0);
                    add_scaled(acc[t], d, scales[u * 16 + g * 4 + t]);
                }
            }
        }
    }
    wave_sync();
#pragma unroll
    for (int t = 0; t < 4; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    if (wave >= 4) return;
    f32x4 sum = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) sum += part[w][wave][lane];
    const long long v = strip * kStrip + 16 * g + 4 * wave;
    if (there && v < q.y.V) put4((OUT*)q.out + (long long)m * q.os + v, sum, (int)min(4ll, q.y.V - v));
}

// More rows: a workgroup computes 256 vocabulary rows, a strip to each of its
// four wavefronts, for 16 MT hidden rows, which they share through LDS.  The
// hidden values are staged one step ahead and asked for one step before that;
// the weights go straight to the registers of the wavefront that needs them,
// two steps ahead, and are widened between the products, where the vector unit
// has time.  ONCE: there is one row block, and the weights are read once.  Bound by
// the matrix rate (559 rows, V = 129280, H = 4096: FP4 498 us, 1190 TFLOP/s), for
// INT4 by that and the vector instructions that widen and scale (group 128 587 us,
// 64 649, 32 765), and with few rows by the weights' HBM bytes (64 rows FP4 73 us).
template <int FMT, int GROUPS, int MT, bool ONCE, typename OUT>
__global__ __launch_bounds__(256, 2) void sv_head_tile_kernel(Head q)
{
    typedef unsigned short sraw __attribute__((ext_vector_type(GROUPS)));
    typedef float sfloat __attribute__((ext_vector_type(GROUPS)));
    __shared__ u32x4 xt[2][MT][256];
    __shared__ f32x4 offset[2][FMT == SV_W4_INT4 ? 16 * MT : 1];              // of a row's four products
    __shared__ f32x4 scales[FMT == SV_W4_INT4 ? 4 : 1][GROUPS * 16]; // of the wavefront's groups, in vocabulary order
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Workgroups go round the eight dies: the row blocks of one strip group
    // follow each other on one die, whose L2 then holds its weights.
    const unsigned die = blockIdx.x % 8, turn = blockIdx.x / 8;
    const unsigned group = turn / q.nblock * 8 + die;
    if (group * 4ll >= q.y.strips) return;
    const int m0 = (int)(turn % q.nblock) * (16 * MT);
    const long long strip = min(group * 4ll + wave, q.y.strips - 1); // past the last: computed, not stored
    const int steps = q.y.steps;
    const unsigned char* wp = q.packed + strip * steps * 4096;
    const unsigned char* sp = q.packed + q.y.scale_at + strip * steps * (FMT == SV_W4_FP4 ? 256 : GROUPS * 128);
    const Int4Bits bits;

    // staging: chunk n of row r0 of every tile.  Rows past the last are read
    // from the last (and not stored), values past the hidden size from the last
    // values (which meet weights or scales of zero).
    const int n = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    const unsigned short* row[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) row[mt] = q.x + (long long)min(m0 + r0 + 16 * mt, q.M - 1) * q.xs;
    u32x4 xr[MT], w[2][4], s4[2];
    sraw s2[2];
    auto load_x = [&](int step) {
        const unsigned k = (unsigned)min(step * kStep + 8 * n, q.y.H - 8);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) xr[mt] = *(const u32x4_any*)(row[mt] + k);
    };
    auto stage_x = [&](int buf) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            xt[buf][mt][x_slot(n, r0)] = xr[mt];
            if constexpr (FMT == SV_W4_INT4) {
                const float z = x_offset(xr[mt]);
                if ((n & 3) == 0) ((float*)&offset[buf][16 * mt + r0])[n >> 2] = z;
            }
        }
    };
    auto load_w = [&](int step, int j) { // past the end: the last step again, not used
        const long long at = min(step, steps - 1);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const u32x4* from = (const u32x4*)(wp + at * 4096 + t * 1024 + lane * 16);
            // (16 rows at V = 129280, H = 7168: 77 us, with other loads 86; 64 rows at V =
            // 16000, H = 4096 in four blocks: 19 us, with other loads 16)
            w[j][t] = ONCE ? __builtin_nontemporal_load(from) : *from;
        }
        if constexpr (FMT == SV_W4_FP4) s4[j] = *(const u32x4*)(sp + at * 256 + c * 16);
        else s2[j] = ((const sraw*)(sp + at * (GROUPS * 128)))[lane];
    };
    f32x4 acc[MT][4] = {};
    auto take = [&](int step, int j) { // step's products; j = step % 2
        if constexpr (FMT == SV_W4_INT4) {
            sfloat f;
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) f[i] = __uint_as_float((unsigned)s2[j][i] << 16);
            ((sfloat*)scales[wave])[lane] = f;
        }
        lds_barrier();
        stage_x(j ^ 1);
        load_x(step + 2);
        __builtin_amdgcn_sched_barrier(0); // the loads stay ahead of the products
        auto hidden = [&](int mt, int p) { return __builtin_bit_cast(bf16x8, xt[j][mt][x_slot(4 * p + g, c)]); };
        if constexpr (FMT == SV_W4_FP4) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                bf16x8 a[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) a[t] = widen_fp4(w[j][t][p], fp4_scale(s4[j][t], p));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const bf16x8 b = hidden(mt, p);
#pragma unroll
                    for (int t = 0; t < 4; ++t) acc[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t], b, acc[mt][t], 0, 0, 0);
                }
            }
        } else if constexpr (GROUPS == 1) {
            f32x4 d[MT][4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                bf16x8 a[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) a[t] = bits.widen(w[j][t][p]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const bf16x8 b = hidden(mt, p);
                    if (p == 0) {
                        const f32x4 z4 = offset[j][16 * mt + c];
                        const float z = (z4[0] + z4[1]) + (z4[2] + z4[3]);
#pragma unroll
                        for (int t = 0; t < 4; ++t) d[mt][t] = f32x4{z, z, z, z};
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) d[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t], b, d[mt][t], 0, 0, 0);
                }
            }
            f32x4 s[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) s[t] = scales[wave][g * 4 + t];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int t = 0; t < 4; ++t) add_scaled(acc[mt][t], d[mt][t], s[t]);
        } else {
            constexpr int P = 4 / GROUPS; // products of a group
#pragma unroll
            for (int u = 0; u < GROUPS; ++u) {
                bf16x8 a[P][4];
                f32x4 s[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        unsigned word = w[j][t][u * P + p];
                        asm volatile("" : "+v"(word));
                        a[p][t] = bits.widen(word);
                    }
                    s[t] = scales[wave][u * 16 + g * 4 + t];
                }
                f32x4 d[2][4]; // a tile of rows is multiplied while the one before is scaled
                auto scale_tile = [&](int mt) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        add_scaled(acc[mt][t], d[mt & 1][t], s[t]);
                        asm("" : "+v"(acc[mt][t])); // one tile after the other, or their sums pile up and spill
                    }
                };
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const f32x4 z4 = offset[j][16 * mt + c];
                    const float z = GROUPS == 4 ? z4[u] : z4[2 * u & 3] + z4[(2 * u + 1) & 3];
#pragma unroll
                    for (int t = 0; t < 4; ++t) d[mt & 1][t] = f32x4{z, z, z, z};
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const bf16x8 b = hidden(mt, u * P + p);
#pragma unroll
                        for (int t = 0; t < 4; ++t) d[mt & 1][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p][t], b, d[mt & 1][t], 0, 0, 0);
                    }
                    if (mt > 0) scale_tile(mt - 1);
                }
                scale_tile(MT - 1);
            }
        }
        load_w(step + 2, j);
        __builtin_amdgcn_sched_barrier(0);
    };

    load_x(0);
    load_w(0, 0);
    load_w(1, 1);
    stage_x(0);
    load_x(1);
    int step = 0;
    for (; step + 2 <= steps; step += 2) {
        take(step, 0);
        take(step + 1, 1);
    }
    if (step < steps) take(step, 0);

    if (group * 4ll + wave >= q.y.strips) return;
    const long long v = strip * kStrip + 16 * g;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int m = m0 + 16 * mt + c;
        if (m >= q.M) continue;
        OUT* out = (OUT*)q.out + (long long)m * q.os + v;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (v + 4 * t < q.y.V) put4(out + 4 * t, acc[mt][t], (int)min(4ll, q.y.V - v - 4 * t));
    }
}

int check_weights(int32_t hidden, int32_t format, int32_t group)
{
    if (format != SV_W4_FP4 && format != SV_W4_INT4) return SV_EUNSUPPORTED;
    if (format == SV_W4_FP4 ? group != 32 : group != 32 && group != 64 && group != 128) return SV_EUNSUPPORTED;
    if (hidden < 1 || hidden > SV_MAX_HIDDEN || hidden % group) return SV_EINVAL;
    return SV_OK;
}

// Launches of at most 2^32 - 1 work-items: `per` workgroups of `threads` for
// each block of `rows` hidden rows.
template <typename Launch>
hipError_t in_launches(Head q, long long per, int threads, int rows, int es, Launch launch)
{
    const int most = (int)std::min(0xffffffffll / threads / per, (long long)(1 << 30) / rows) * rows;
    for (int left = q.M; left > 0; left -= most) {
        q.M = std::min(left, most);
        q.nblock = (unsigned)((q.M + rows - 1) / rows);
        const hipError_t e = launch(q, dim3((unsigned)(per * q.nblock)), dim3(threads));
        if (e != hipSuccess) return e;
        q.x += (long long)most * q.xs;
        q.out = (char*)q.out + (long long)most * q.os * es;
    }
    return hipSuccess;
}

template <int FMT, int GROUPS, typename OUT>
hipError_t launch_rows(Head q, hipStream_t s)
{
    q.nstrip = (unsigned)q.y.strips;
    return in_launches(q, q.y.strips, 64 * kRowWaves, 16, sizeof(OUT), [&](const Head& a, dim3 grid, dim3 block) {
        return launch_kernel(sv_head_rows_kernel<FMT, GROUPS, OUT>, grid, block, 0, s, nullptr, nullptr, a);
    });
}

template <int FMT, int GROUPS, int MT, typename OUT>
hipError_t launch_tile(const Head& q, hipStream_t s)
{
    return in_launches(q, ((q.y.strips + 3) / 4 + 7) / 8 * 8, 256, 16 * MT, sizeof(OUT), [&](const Head& a, dim3 grid, dim3 block) {
        if (sv::head_tile_once(16 * MT, a.nblock))
            return launch_kernel(sv_head_tile_kernel<FMT, GROUPS, MT, sv::head_tile_once(16 * MT, 1), OUT>, grid, block, 0, s, nullptr,
                                 nullptr, a);
        return launch_kernel(sv_head_tile_kernel<FMT, GROUPS, MT, false, OUT>, grid, block, 0, s, nullptr, nullptr, a);
    });
}

template <int FMT, int GROUPS, typename OUT>
hipError_t launch_head(const Head& q, hipStream_t s)
{
    switch (sv::head_tile_rows(q.M, q.y.V, FMT == SV_W4_FP4, kStep / GROUPS)) {
    case 16: return launch_tile<FMT, GROUPS, 1, OUT>(q, s);
    case 32: return launch_tile<FMT, GROUPS, 2, OUT>(q, s);
    case 64: return launch_tile<FMT, GROUPS, 4, OUT>(q, s);
    default: return launch_rows<FMT, GROUPS, OUT>(q, s);
    }
}

template <typename OUT>
hipError_t launch_format(const Head& q, int format, int group, hipStream_t s)
{
    if (format == SV_W4_FP4) return launch_head<SV_W4_FP4, 4, OUT>(q, s);
    if (group == 32) return launch_head<SV_W4_INT4, 4, OUT>(q, s);
    if (group == 64) return launch_head<SV_W4_INT4, 2, OUT>(q, s);
    return launch_head<SV_W4_INT4, 1, OUT>(q, s);
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
    const hipError_t e = cfg->dtype == SV_BF16 ? launch_format<__bf16>(q, a->format, a->group, s)
                                               : launch_format<float>(q, a->format, a->group, s);
    return e == hipSuccess ? SV_OK : SV_EDEVICE;
}

} // extern "C"
