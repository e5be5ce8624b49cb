// grouped_kernel.h -- y = x W^T + bias for a few rows of x and 4-bit weights with one
// scale (and zero point) for every 32, 64 or 128 input channels of a row:
//
//   y[m][n] = sum_g s[n][g] (sum_{k in g} u[n][k] x[m][k] - z[n][g] sum_{k in g} x[m][k]) + bias[n]
//
// u in [0, 15] are the codes as stored (two's complement codes q are read as
// u = q + 8 with z = 8).  Both inner sums run on the 16-bit matrix cores with
// binary32 sums; the second one is the product with a matrix of ones, so it
// comes out in the lanes that need it.  A code becomes a bf16 or f16 value
// without rounding: the byte u is the FP8 e4m3 value u / 512 (denormals and
// the first binade are one arithmetic progression), which one conversion
// instruction widens two at a time, times 512.
//
// The codes are read as they are interchanged, N x packed-K.
//
// Few rows are bound by memory: 1 x 4096 -> 12288 reads 26 MB in 7.9 us (3.3
// TB/s, a kernel that only reads them 5.9 us), 1 x 1024 -> 1024 takes 2.4 us where
// an empty kernel takes 1.9.  With more rows every compute unit reads all of x
// and widens its share of the codes, some 60 vector instructions for each 16 x
// 128 of them beside 8 or 16 matrix instructions: 32 x 16384 -> 16384 takes 44
// us (143 MB, 3.2 TB/s), 34 with its codes in the cache and 26 for reading alone,
// and 16 x 4128 -> 9001 with groups of 32 takes 13.3 us: 4.3 for launch, first
// loads and the joining of the waves, then 1.6 to 1.8 for each block of a wave
// (10.8 with rows of 4096, which begin with a line of memory and give a wave four
// blocks instead of five).  Of those nine, the some 1200 vector instructions a
// wave, two waves a SIMD at some 4.6 cycles each, are about half and its 66 matrix
// instructions one; the rest is waiting for a block's way through shared memory,
// which the fences around `multiply` leave in the open.
//
// Few outputs and long rows leave units idle: a workgroup for every 16 outputs
// (8 for few rows of x), and only its own waves share K.  4096 -> 1024 takes 4.0,
// 4.5, 5.1 and 7.2 us for 1, 8, 16 and 32 rows of x, 14336 -> 1024 7.3, 10.4, 12.6
// and 18.8, and hardly less for 256 outputs; reading the codes alone would take 2
// to 3 us.
#pragma once
#include "block_ops.h"

namespace convrot {
namespace grouped {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename D>
struct Mat;
template <>
struct Mat<__bf16> {
    typedef __bf16 Frag __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    template <bool HI>
    static __device__ __forceinline__ uint32_t widen(uint32_t v)
    {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.f, HI));
    }
};
template <>
struct Mat<_Float16> {
    typedef _Float16 Frag __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    template <bool HI>
    static __device__ __forceinline__ uint32_t widen(uint32_t v)
    {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 512.f, HI));
    }
};

struct GroupedParams {
    const void *x, *scales, *bias;
    const uint8_t *codes, *zeros;
    void* y;
    int M, N, K, groups, rows;   // rows: outputs a workgroup
};

// Eight codes of one word: the even ones lie in the low nibbles of its bytes,
// the odd ones in the high nibbles.  IN_ORDER: k0 k1 .. k7, for two more
// instructions a word; otherwise k0 k2 k4 k6 k1 k3 k5 k7, and x has to be so too.
template <typename D, bool IN_ORDER>
__device__ __forceinline__ typename Mat<D>::Frag widen8(uint32_t w)
{
    uint32_t a = w & 0x0F0F0F0Fu, b = (w >> 4) & 0x0F0F0F0Fu;
    if constexpr (IN_ORDER) {
        const uint32_t even = a, odd = b;
        a = __builtin_amdgcn_perm(odd, even, 0x05010400u);
        b = __builtin_amdgcn_perm(odd, even, 0x07030602u);
    }
    const u32x4 v = {Mat<D>::template widen<false>(a), Mat<D>::template widen<true>(a),
                     Mat<D>::template widen<false>(b), Mat<D>::template widen<true>(b)};
    return __builtin_bit_cast(typename Mat<D>::Frag, v);
}

// Eight consecutive values of x in that second order.
__device__ __forceinline__ u32x4 reorder8(u32x4 x)
{
    return u32x4{__builtin_amdgcn_perm(x[1], x[0], 0x05040100u), __builtin_amdgcn_perm(x[3], x[2], 0x05040100u),
                 __builtin_amdgcn_perm(x[1], x[0], 0x07060302u), __builtin_amdgcn_perm(x[3], x[2], 0x07060302u)};
}

// 4 x 4 transpose of (lane quarter, word): word j of quarter q becomes what
// word q of quarter j was.  A group of 32 channels then lies in one word of
// all four quarters, that is in one matrix instruction.
__device__ __forceinline__ u32x4 transpose4(u32x4 w)
{
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{c[0], c[1], d[0], d[1]};
}

template <int BYTES>
struct UintOf;
template <> struct UintOf<1> { typedef uint8_t type; };
template <> struct UintOf<2> { typedef uint16_t type; };
template <> struct UintOf<4> { typedef uint32_t type; };
template <> struct UintOf<8> { typedef uint64_t type; };

// The value that lane `from / 4` holds.
__device__ __forceinline__ uint32_t fetch(int from, uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v);
}

// A workgroup of W waves makes p.rows outputs, at most 16 NT, for up to 16 MT
// rows of x.  Its waves share the 128-K blocks, a run of consecutive ones each,
// and add their parts in a fixed order at the end.
//
// In a matrix tile lane (r, q) = (lane % 16, lane / 16) owns row r and the
// channels of quarter q.  Loads that way would touch a line of memory for every
// lane (and a load costs the lines it touches: 157 against 85 us for 32 x 16384
// -> 16384), so neighbouring lanes load neighbouring pieces of a row -- of the
// codes lane / 8 is the row and lane % 8 the 16-byte piece of two blocks, a
// whole line, of x lane / 16 and lane % 16 -- and a wave passes them on through
// its own part of shared memory.  Scales and zero points come for four blocks at
// a time, lane % 4 the block.  Two blocks of codes are on their way while two
// are multiplied, of x two blocks or one: more in flight costs registers and
// time (four blocks of codes: 32 x 16384 -> 16384 49 against 44 us, 16 x 4096 ->
// 16384 12.9 against 12.0).
//
// Row m of x sits at row 4 (m % 4) + m / 4 of its matrix tile, so that the
// first E of the four sums a lane holds are the ones in use for M <= 4 E.
//
// LINES: every row of the codes is whole lines of memory, which are then loaded
// with the hint that they are used once (1 x 4096 -> 12288 8.6 -> 8.0 us, 32 x
// 16384 -> 16384 47.4 -> 44.9); where rows begin inside a line, two loads want it
// (16 x 4128 -> 9001 14.2 -> 15.2).
// OCC: the waves of a SIMD that the registers have to leave room for.
template <typename D, int GROUP, bool ZEROS, bool LINES, int MT, int E, int NT, int W, int OCC>
__global__ __launch_bounds__(W * 64, OCC) void grouped_kernel(GroupedParams p)
{
    typedef typename Mat<D>::Frag Frag;
    constexpr int kPer = 128 / GROUP;                // groups a block
    constexpr int kSteps = GROUP / 32;               // matrix instructions a group
    constexpr int kWords = (kPer + 1) / 2;           // words of a block's scales
    constexpr bool kTurn = GROUP != 128;             // step j holds k = 32 j + 8 q, without it k = 32 q + 8 j
    constexpr int kXLoads = E * MT;                  // four rows of x a load
    constexpr int PX = E == 1 ? 2 : 1;               // blocks of x loaded ahead
    constexpr uint32_t kNowhere = 0x80000000u;       // an offset behind any buffer, whatever row is added
    constexpr bool kInOrder = kXLoads > 2 * NT;      // which of x and the codes is cheaper to reorder
    typedef typename UintOf<kPer * 2>::type Scales __attribute__((aligned(2)));
    typedef typename UintOf<kPer>::type Zeros __attribute__((aligned(1)));

    union Shared {
        u32x4 part[W][(kXLoads + 2 * NT) * 64];   // a wave's block of x and two of codes, 16-byte pieces
        float parts[W][MT * NT * E][64];
    };
    __shared__ Shared shared;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int r = lane % 16, q = lane / 16;
    const int n0 = (int)blockIdx.x * p.rows, n_end = min(n0 + p.rows, p.N);
    const int m_own = 4 * (r % 4 % E) + r / 4;   // row of x at row r of a matrix tile

    // Blocks of 128 K, the last one filled up with zeros (a row shorter than one
    // comes at the end).  A wave's run begins with a line where rows do; where they
    // do not, runs are as even as they can be (16 x 4224 -> 9001 in groups of 32:
    // 12.5 us, with even numbers of blocks 14.0; 1 x 5120 -> 8192: 7.7 and 7.1).
    const int blocks = p.K < 128 ? 0 : (p.K + 127) / 128, least = blocks / W, more = blocks % W;
    const int most = least + (more > 0), run = most < 4 ? most : (most + 1) / 2 * 2;
    const int first = LINES ? wave * run : wave * least + min(wave, more);
    const int end = LINES ? min(first + run, blocks) : first + least + (wave < more);
    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};

    // one block, every operand with its owner
    const auto multiply = [&](const u32x4 (&w)[NT], const u32x4 (&x)[MT][4], const uint32_t (&s)[NT][kWords],
                              const uint32_t (&z)[NT]) {
        // sums of x, negated and times the constant zero point
        Frag offset;
#pragma unroll
        for (int i = 0; i < 8; ++i) offset[i] = (D)(ZEROS ? -1.f : -8.f);
        Frag xf[MT][4];
        f32x4 sum[MT][kPer];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int j = 0; j < 4; ++j) xf[mt][j] = __builtin_bit_cast(Frag, x[mt][j]);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                sum[mt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = i * kSteps; j < (i + 1) * kSteps; ++j) sum[mt][i] = Mat<D>::mma(xf[mt][j], offset, sum[mt][i]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            u32x4 v = w[nt];
            if constexpr (kTurn) v = transpose4(v);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                f32x4 part[MT];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) part[mt] = ZEROS ? f32x4{0.f, 0.f, 0.f, 0.f} : sum[mt][i];
#pragma unroll
                for (int j = i * kSteps; j < (i + 1) * kSteps; ++j) {
                    const Frag wf = widen8<D, kInOrder>(ZEROS ? v[j] : v[j] ^ 0x88888888u);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) part[mt] = Mat<D>::mma(xf[mt][j], wf, part[mt]);
                }
                const float scale = (float)__builtin_bit_cast(D, (uint16_t)(s[nt][i / 2] >> (16 * (i % 2))));
                const float zero = ZEROS ? (float)((z[nt] >> (8 * i)) & 0xFFu) : 0.f;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        acc[mt][nt][e] = fmaf(scale, ZEROS ? fmaf(zero, sum[mt][i][e], part[mt][e]) : part[mt][e], acc[mt][nt][e]);
            }
            // The sums are made here and not where the loop ends, which would keep every part until then.
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) asm volatile("" : "+v"(acc[mt][nt]));
        }
    };

    if (first < end) {
        // Rows behind the last one, and what is nowhere, read as zeros; their outputs are computed and not stored.
        const auto codes = __builtin_amdgcn_make_buffer_rsrc((void*)(p.codes + (int64_t)n0 * (p.K / 2)), 0,
                                                             (n_end - n0) * (p.K / 2), 0x20000);
        const auto rows = __builtin_amdgcn_make_buffer_rsrc((void*)p.x, 0, 2 * p.M * p.K, 0x20000);
        const uint16_t* const scales = (const uint16_t*)p.scales + (int64_t)n0 * p.groups;
        const uint8_t* const zeros = p.zeros + (int64_t)n0 * p.groups;
        const int half = lane % 8 / 4;   // which of the two blocks
        const uint32_t w_at = (uint32_t)(lane / 8) * (uint32_t)(p.K / 2) + 16 * (lane % 4);
        const uint32_t x_at = (uint32_t)(lane / 16) * (uint32_t)(2 * p.K) + 16 * (lane % 16);
        uint32_t s_at[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s_at[nt] = (uint32_t)min(16 * nt + lane / 4, n_end - 1 - n0) * (uint32_t)p.groups;
        u32x4 w[2 * NT], x[PX][kXLoads];
        uint32_t s[NT][kWords], z[NT];
        // With 32 rows an offset is worked out for each load: kept, those of all
        // of them take registers that are not there.
        const auto load_w = [&](int b) {   // blocks b and b + 1
            const uint32_t of = (uint32_t)min(b + half, end - 1) * 64u;
            const uint32_t at = LINES || of + 16 * (lane % 4) < (uint32_t)(p.K / 2) ? w_at + of : kNowhere;
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i) {
                uint32_t row = (uint32_t)(8 * i) * (uint32_t)(p.K / 2);
                if constexpr (MT > 1) asm volatile("" : "+s"(row));
                w[i] = __builtin_amdgcn_raw_buffer_load_b128(codes, at + row, 0, LINES ? 2 : 0);
            }
        };
        const auto load_x = [&](u32x4 (&to)[kXLoads], int b) {
            const uint32_t at = LINES || b * 128 + 8 * (lane % 16) < p.K ? x_at : kNowhere;
#pragma unroll
            for (int i = 0; i < kXLoads; ++i) {
                uint32_t row = (uint32_t)(4 * i) * (uint32_t)(2 * p.K) + (uint32_t)b * 256u;
                if constexpr (MT > 1) asm volatile("" : "+s"(row));
                to[i] = __builtin_amdgcn_raw_buffer_load_b128(rows, at + row, 0, 0);
            }
        };
        const auto load_s = [&](uint32_t (&to)[NT][kWords], uint32_t (&to_z)[NT], int b) {
            // of the row's last groups where a block has fewer of its own
            uint32_t at = (uint32_t)min(b + lane % 4, blocks - 1) * kPer;
            if constexpr (!LINES) at = min(at, (uint32_t)(p.groups - kPer));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const auto v = *(const Scales*)((const uint8_t*)scales + 2 * (s_at[nt] + at));
                to[nt][0] = (uint32_t)v;
                if constexpr (kPer == 4) to[nt][1] = (uint32_t)(v >> 32);
                if constexpr (ZEROS) to_z[nt] = *(const Zeros*)(zeros + (s_at[nt] + at));
            }
        };
        // The wave's own part of shared memory, whose accesses happen in order.
        // Piece c of row m of x lies at 16 m + (c ^ m), piece c of row r of a
        // block's codes at 4 r + (c ^ r / 4), in the second block with the rows
        // swapped in pairs: the 16 lanes that read one piece of 16 rows, and the
        // 8 that write a line, meet different places.
        u32x4* const part_x = shared.part[wave];
        u32x4* const part_w = part_x + kXLoads * 64;
        const auto take_x = [&](u32x4 (&to)[MT][4], const u32x4 (&from)[kXLoads]) {
#pragma unroll
            for (int i = 0; i < kXLoads; ++i) {
                const int m = 4 * i + lane / 16;
                part_x[16 * m + ((lane % 16) ^ (m % 16))] = kInOrder ? from[i] : reorder8(from[i]);
            }
            wave_exchange();
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) to[mt][i] = part_x[16 * (16 * mt + m_own) + ((kTurn ? 4 * i + q : 4 * q + i) ^ m_own)];
            wave_exchange();
        };
        const auto put_w = [&]() {
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i) {
                const int row = 8 * (i % 2) + lane / 8;
                part_w[64 * NT * half + 64 * (i / 2) + 4 * (row ^ half) + (lane % 4 ^ row / 4)] = w[i];
            }
            wave_exchange();
        };
        const auto take_w = [&](u32x4 (&to)[NT], int h) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) to[nt] = part_w[64 * NT * h + 64 * nt + 4 * (r ^ h) + (q ^ r / 4)];
            wave_exchange();
        };
        const auto take_s = [&](uint32_t (&so)[NT][kWords], uint32_t (&zo)[NT], int j) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < kWords; ++i) so[nt][i] = fetch(4 * (4 * r + j), s[nt][i]);
                zo[nt] = ZEROS ? fetch(4 * (4 * r + j), z[nt]) : 0;
            }
        };
        // Loads return in order, so what is used first is asked for first: x of a
        // block before its codes.
        load_s(s, z, first);
        load_x(x[0], first);
        load_w(first);
        if constexpr (PX > 1) load_x(x[1], min(first + 1, end - 1));
        u32x4 xo[MT][4];
        int b = first;
        for (; b + 4 < end; b += 4) {
            uint32_t next_s[NT][kWords], next_z[NT];
            load_s(next_s, next_z, b + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32x4 wo[NT];
                uint32_t so[NT][kWords], zo[NT];
                take_x(xo, x[j % PX]);
                load_x(x[j % PX], min(b + j + PX, end - 1));
                take_s(so, zo, j);
                if (j % 2 == 0) {
                    put_w();
                    load_w(b + j + 2);
                }
                take_w(wo, j % 2);
                __builtin_amdgcn_sched_barrier(0);
                multiply(wo, xo, so, zo);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < kWords; ++i) s[nt][i] = next_s[nt][i];
                if constexpr (ZEROS) z[nt] = next_z[nt];
            }
        }
        if (!LINES && kPer > 1 && end == blocks && lane % 4 == blocks - 1 - b) {
            const int before = blocks * kPer - p.groups;   // groups in front of the last block's own
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint64_t v = s[nt][0];
                if constexpr (kPer == 4) v |= (uint64_t)s[nt][1] << 32;
                v >>= 16 * before;
                s[nt][0] = (uint32_t)v;
                if constexpr (kPer == 4) s[nt][1] = (uint32_t)(v >> 32);
                if constexpr (ZEROS) z[nt] >>= 8 * before;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (b + j < end) {
                u32x4 wo[NT];
                uint32_t so[NT][kWords], zo[NT];
                take_x(xo, x[j % PX]);
                if (j + PX < 4) load_x(x[j % PX], min(b + j + PX, end - 1));
                take_s(so, zo, j);
                if (j % 2 == 0) put_w();
                if (j == 0) load_w(b + 2);
                take_w(wo, j % 2);
                __builtin_amdgcn_sched_barrier(0);
                multiply(wo, xo, so, zo);
                __builtin_amdgcn_sched_barrier(0);
            }
    }
    if (!LINES && kPer > 1 && wave == W - 1 && p.K < 128) {   // a row shorter than a block: zeros behind it
        u32x4 w[NT], x[MT][4];
        uint32_t s[NT][kWords] = {}, z[NT] = {};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int64_t n = min(n0 + 16 * nt + r, n_end - 1);
            w[nt] = u32x4{0u, 0u, 0u, 0u};
            if (32 * q < p.K) w[nt] = *(const u32x4*)(p.codes + n * (p.K / 2) + 16 * q);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i < p.groups) {
                    const int64_t g = n * p.groups + i;
                    s[nt][i / 2] |= (uint32_t)((const uint16_t*)p.scales)[g] << (16 * (i % 2));
                    if constexpr (ZEROS) z[nt] |= (uint32_t)p.zeros[g] << (8 * i);
                }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = 16 * mt + m_own;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = kTurn ? 32 * j + 8 * q : 32 * q + 8 * j;
                x[mt][j] = u32x4{0u, 0u, 0u, 0u};
                if (k < p.K) x[mt][j] = *(const u32x4*)((const uint16_t*)p.x + (int64_t)min(m, p.M - 1) * p.K + k);
                if constexpr (!kInOrder) x[mt][j] = reorder8(x[mt][j]);
            }
        }
        multiply(w, x, s, z);
    }
    __syncthreads();   // x is done with
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < E; ++e) shared.parts[wave][(mt * NT + nt) * E + e][lane] = acc[mt][nt][e];
    __syncthreads();
    for (int i = threadIdx.x; i < MT * NT * E * 64; i += W * 64) {
        const int slot = i / 64, l = i % 64, mt = slot / (E * NT), nt = slot / E % NT, e = slot % E;
        const int m = 16 * mt + 4 * e + l / 16, n = n0 + 16 * nt + l % 16;
        if (m >= p.M || n >= n_end) continue;
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) v += shared.parts[k][slot][l];
        if (p.bias) v += (float)((const D*)p.bias)[n];
        ((D*)p.y)[(int64_t)m * p.N + n] = (D)v;
    }
}

template <typename D, int GROUP, bool ZEROS, int MT, int E, int NT, int W, int OCC>
void launch_one(GroupedParams p, hipStream_t s)
{
    const dim3 grid((p.N + p.rows - 1) / p.rows), block(W * 64);
    if (p.K % 256 == 0 && (uintptr_t)p.codes % 128 == 0)
        hipLaunchKernelGGL((grouped_kernel<D, GROUP, ZEROS, true, MT, E, NT, W, OCC>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((grouped_kernel<D, GROUP, ZEROS, false, MT, E, NT, W, OCC>), grid, block, 0, s, p);
}

// Which variant, by M and N (times in a graph, us):
// M <= 4: x is small, so one tile a workgroup and many workgroups; four waves
//   from N > 8192 on (1 x 4096 -> 12288: 7.8, with eight 10.0; 4096 -> 4096: 5.9,
//   with eight 5.3); a long row of few outputs gets half-filled tiles, to have a
//   workgroup for every unit (4 x 12288 -> 2048: 7.7, with whole ones 8.0).
// M > 4: every workgroup reads all of x, so it takes as many outputs as one
//   round (or several equal ones) over the units allows, up to 64 (16 x 4096 ->
//   16384: 11.9 with 64 outputs, 14.0 with 32, 15.1 with 16), with eight waves:
//   two a SIMD cover some of each other's waits (32 x 16384 -> 16384: 42.8, with four
//   46.4; 32 x 4096 -> 16384 in groups of 32: 17.4 (with zero points 19.3), with
//   four 22.9, although eight have to keep 10 (24 to 29) registers in memory).
template <typename D, int GROUP, bool ZEROS>
void launch_zeros(GroupedParams p, hipStream_t s)
{
    if (p.M <= 4) {
        p.rows = p.N <= 2048 && p.K >= 8192 ? 8 : 16;
        if (p.N > 8192) launch_one<D, GROUP, ZEROS, 1, 1, 1, 4, 4>(p, s);
        else launch_one<D, GROUP, ZEROS, 1, 1, 1, 8, 4>(p, s);
        return;
    }
    const int rounds = (p.N + 64 * kUnits - 1) / (64 * kUnits);
    p.rows = (p.N + rounds * kUnits - 1) / (rounds * kUnits);
    if (p.rows < 16) p.rows = 16;
    const int tiles = (p.rows + 15) / 16;
    if (p.M <= 8) {
        if (tiles == 1) launch_one<D, GROUP, ZEROS, 1, 2, 1, 8, 4>(p, s);
        else if (tiles == 2) launch_one<D, GROUP, ZEROS, 1, 2, 2, 8, 2>(p, s);
        else if (tiles == 3) launch_one<D, GROUP, ZEROS, 1, 2, 3, 8, 2>(p, s);
        else launch_one<D, GROUP, ZEROS, 1, 2, 4, 8, 2>(p, s);
    } else if (p.M <= 16) {
        if (tiles == 1) launch_one<D, GROUP, ZEROS, 1, 4, 1, 8, 2>(p, s);
        else if (tiles == 2) launch_one<D, GROUP, ZEROS, 1, 4, 2, 8, 2>(p, s);
        else if (tiles == 3) launch_one<D, GROUP, ZEROS, 1, 4, 3, 8, 2>(p, s);
        else launch_one<D, GROUP, ZEROS, 1, 4, 4, 8, 2>(p, s);
    } else {
        if (tiles == 1) launch_one<D, GROUP, ZEROS, 2, 4, 1, 8, 2>(p, s);
        else if (tiles == 2) launch_one<D, GROUP, ZEROS, 2, 4, 2, 8, 2>(p, s);
        else if (tiles == 3) launch_one<D, GROUP, ZEROS, 2, 4, 3, 8, 2>(p, s);
        else launch_one<D, GROUP, ZEROS, 2, 4, 4, 8, 2>(p, s);
    }
}

template <typename D, int GROUP>
void launch_group(const GroupedParams& p, hipStream_t s)
{
    p.zeros ? launch_zeros<D, GROUP, true>(p, s) : launch_zeros<D, GROUP, false>(p, s);
}

template <typename D>
void launch_type(const GroupedParams& p, int group, hipStream_t s)
{
    if (group == 32) launch_group<D, 32>(p, s);
    else if (group == 64) launch_group<D, 64>(p, s);
    else launch_group<D, 128>(p, s);
}

}  // namespace grouped
}  // namespace convrot
