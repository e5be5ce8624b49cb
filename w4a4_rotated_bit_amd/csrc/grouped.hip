// grouped.hip -- y = x W^T + bias for a few rows of x and 4-bit weights with one
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
// The codes are read as they are interchanged, N x packed-K: lane (r, q) of a
// wave loads the 16 bytes of row r that hold k = 128 b + 32 q .. + 31.
#include "block_ops.h"

namespace convrot {

namespace {

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
    int M, N, K, groups, blocks;   // blocks: 128-K blocks, the last one perhaps in part
};

// Eight codes of one word in the order k0 k2 k4 k6 k1 k3 k5 k7.
template <typename D>
__device__ __forceinline__ typename Mat<D>::Frag widen8(uint32_t w)
{
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
    const u32x4 v = {Mat<D>::template widen<false>(lo), Mat<D>::template widen<true>(lo),
                     Mat<D>::template widen<false>(hi), Mat<D>::template widen<true>(hi)};
    return __builtin_bit_cast(typename Mat<D>::Frag, v);
}

// Eight consecutive values of x in the same order.
template <typename D>
__device__ __forceinline__ typename Mat<D>::Frag reorder8(u32x4 x)
{
    const u32x4 v = {__builtin_amdgcn_perm(x[1], x[0], 0x05040100u), __builtin_amdgcn_perm(x[3], x[2], 0x05040100u),
                     __builtin_amdgcn_perm(x[1], x[0], 0x07060302u), __builtin_amdgcn_perm(x[3], x[2], 0x07060302u)};
    return __builtin_bit_cast(typename Mat<D>::Frag, v);
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

// A workgroup of W waves makes 16 NT outputs for up to 16 MT rows; its waves
// share the 128-K blocks, UB consecutive ones at a time, and add their parts
// in a fixed order at the end.
template <typename D, int GROUP, int MT, int NT, int W, int UB>
__global__ __launch_bounds__(W * 64) void grouped_kernel(GroupedParams p)
{
    constexpr int kPer = 128 / GROUP;   // groups a block
    typedef typename Mat<D>::Frag Frag;
    __shared__ float parts[W][MT * NT * 4][64];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, r = lane % 16, q = lane / 16;
    const int n0 = (int)blockIdx.x * 16 * NT;

    const uint8_t* codes[NT];
    int64_t group0[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int64_t n = min(n0 + 16 * nt + r, p.N - 1);   // outputs past N are computed and not stored
        codes[nt] = p.codes + n * (p.K / 2) + 16 * q;
        group0[nt] = n * p.groups;
    }
    const uint16_t* x[MT];
    bool row_in[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        row_in[mt] = 16 * mt + r < p.M;
        x[mt] = (const uint16_t*)p.x + (int64_t)(row_in[mt] ? 16 * mt + r : 0) * p.K;
    }
    Frag ones;
#pragma unroll
    for (int i = 0; i < 8; ++i) ones[i] = (D)1.f;
    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};

    const uint32_t flip = p.zeros ? 0u : 0x88888888u;
    for (int b0 = wave * UB; b0 < p.blocks; b0 += W * UB) {
        u32x4 w[UB][NT], xv[UB][MT][4];
        float s[UB][NT][kPer], z[UB][NT][kPer];
#pragma unroll
        for (int ub = 0; ub < UB; ++ub) {
            const int kb = (b0 + ub) * 128;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                w[ub][nt] = u32x4{0u, 0u, 0u, 0u};
                if (kb + 32 * q < p.K) w[ub][nt] = *(const u32x4*)(codes[nt] + kb / 2);
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    s[ub][nt][i] = 0.f;
                    z[ub][nt][i] = 8.f;
                    const int g = (b0 + ub) * kPer + i;
                    if (g < p.groups) {
                        s[ub][nt][i] = (float)((const D*)p.scales)[group0[nt] + g];
                        if (p.zeros) z[ub][nt][i] = (float)p.zeros[group0[nt] + g];
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = kb + (GROUP == 128 ? 32 * q + 8 * j : 32 * j + 8 * q);
                    xv[ub][mt][j] = u32x4{0u, 0u, 0u, 0u};
                    if (row_in[mt] && k < p.K) xv[ub][mt][j] = *(const u32x4*)(x[mt] + k);
                }
        }
#pragma unroll
        for (int ub = 0; ub < UB; ++ub) {
            Frag xf[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j) xf[mt][j] = reorder8<D>(xv[ub][mt][j]);
            f32x4 sum[MT][kPer];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    sum[mt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = i * (4 / kPer); j < (i + 1) * (4 / kPer); ++j)
                        sum[mt][i] = Mat<D>::mma(xf[mt][j], ones, sum[mt][i]);
                }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                u32x4 v = w[ub][nt];
                if constexpr (GROUP != 128) v = transpose4(v);
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    f32x4 part[MT];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) part[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = i * (4 / kPer); j < (i + 1) * (4 / kPer); ++j) {
                        const Frag wf = widen8<D>(v[j] ^ flip);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) part[mt] = Mat<D>::mma(xf[mt][j], wf, part[mt]);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[mt][nt][e] = fmaf(s[ub][nt][i], fmaf(-z[ub][nt][i], sum[mt][i][e], part[mt][e]),
                                                  acc[mt][nt][e]);
                }
            }
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) parts[wave][(mt * NT + nt) * 4 + e][lane] = acc[mt][nt][e];
    __syncthreads();
    for (int i = threadIdx.x; i < MT * NT * 256; i += W * 64) {
        const int slot = i / 64, l = i % 64, mt = slot / (4 * NT), nt = slot / 4 % NT, e = slot % 4;
        const int m = 16 * mt + 4 * (l / 16) + e, n = n0 + 16 * nt + l % 16;
        if (m >= p.M || n >= p.N) continue;
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) v += parts[k][slot][l];
        if (p.bias) v += (float)((const D*)p.bias)[n];
        ((D*)p.y)[(int64_t)m * p.N + n] = (D)v;
    }
}

template <typename D, int GROUP, int MT>
void launch_rows(const GroupedParams& p, hipStream_t s)
{
    hipLaunchKernelGGL((grouped_kernel<D, GROUP, MT, 1, 8, 2>), dim3((p.N + 15) / 16), dim3(512), 0, s, p);
}

template <typename D>
void launch_type(const GroupedParams& p, int group, hipStream_t s)
{
    const bool two = p.M > 16;
    if (group == 32) two ? launch_rows<D, 32, 2>(p, s) : launch_rows<D, 32, 1>(p, s);
    else if (group == 64) two ? launch_rows<D, 64, 2>(p, s) : launch_rows<D, 64, 1>(p, s);
    else two ? launch_rows<D, 128, 2>(p, s) : launch_rows<D, 128, 1>(p, s);
}

// Codes, scales and zero points of a weight.  Two channels a lane, GROUP / 2
// lanes a group.  The scale is rounded to its storage type first, and the
// codes are those of the rounded scale.
template <typename D, int GROUP>
__device__ __forceinline__ void quantize_row(const D* W, int bytes, uint8_t* codes, D* scales, uint8_t* zeros)
{
    constexpr int L = GROUP / 2;
    const int i = (int)blockIdx.x * 256 + threadIdx.x;   // one packed byte
    const bool in = i < bytes;                           // a whole number of groups
    float a = 0.f, b = 0.f;
    if (in) {
        a = (float)W[2 * i];
        b = (float)W[2 * i + 1];
    }
    float lo = 0.f, hi = 0.f;
    bool bad = !(fabsf(a) < INFINITY) || !(fabsf(b) < INFINITY);
    if (zeros) {
        lo = fminf(fminf(a, b), 0.f);
        hi = fmaxf(fmaxf(a, b), 0.f);
    } else {
        hi = fmaxf(fabsf(a), fabsf(b));
    }
#pragma unroll
    for (int d = 1; d < L; d *= 2) {
        lo = fminf(lo, __shfl_xor(lo, d, 64));
        hi = fmaxf(hi, __shfl_xor(hi, d, 64));
        const int other = __shfl_xor((int)bad, d, 64);
        bad = bad || other;
    }
    const float s = bad ? NAN : (float)(D)(zeros ? (hi - lo) / 15.f : hi / 7.f);
    const bool usable = s > 0.f && s < INFINITY;
    int z = 0, qa = 0, qb = 0;
    if (usable) {
        qa = (int)rintf(fminf(fmaxf(a / s, -32.f), 32.f));
        qb = (int)rintf(fminf(fmaxf(b / s, -32.f), 32.f));
        if (zeros) {
            z = min(15, (int)rintf(fminf(-lo / s, 15.f)));
            qa = min(15, max(0, qa + z));
            qb = min(15, max(0, qb + z));
        } else {
            qa = min(7, max(-7, qa));
            qb = min(7, max(-7, qb));
        }
    }
    if (!in) return;
    codes[i] = (uint8_t)((qa & 15) | (qb & 15) << 4);
    if (i % L == 0) {
        scales[i / L] = (D)s;
        if (zeros) zeros[i / L] = (uint8_t)z;
    }
}

template <typename D, int GROUP>
__global__ __launch_bounds__(256) void quantize_grouped_kernel(const D* W, int N, int K, uint8_t* codes, D* scales,
                                                               uint8_t* zeros)
{
    const int groups = K / GROUP;
    for (int64_t n = blockIdx.y; n < N; n += gridDim.y)
        quantize_row<D, GROUP>(W + n * K, K / 2, codes + n * (K / 2), scales + n * groups,
                               zeros ? zeros + n * groups : nullptr);
}

template <typename D>
void quantize_type(const D* W, int N, int K, int group, uint8_t* codes, D* scales, uint8_t* zeros, hipStream_t s)
{
    const dim3 grid((K / 2 + 255) / 256, N < 65535 ? N : 65535), block(256);
    if (group == 32)
        hipLaunchKernelGGL((quantize_grouped_kernel<D, 32>), grid, block, 0, s, W, N, K, codes, scales, zeros);
    else if (group == 64)
        hipLaunchKernelGGL((quantize_grouped_kernel<D, 64>), grid, block, 0, s, W, N, K, codes, scales, zeros);
    else
        hipLaunchKernelGGL((quantize_grouped_kernel<D, 128>), grid, block, 0, s, W, N, K, codes, scales, zeros);
}

}  // namespace

void launch_linear_grouped(const convrot_grouped_args& a, hipStream_t s)
{
    GroupedParams p{};
    p.x = a.x_dev;
    p.codes = (const uint8_t*)a.codes_dev;
    p.scales = a.scales_dev;
    p.zeros = (const uint8_t*)a.zeros_dev;
    p.bias = a.bias_dev;
    p.y = a.y_dev;
    p.M = (int)a.M;
    p.N = (int)a.N;
    p.K = (int)a.K;
    p.groups = (int)(a.K / a.group);
    p.blocks = (int)((a.K + 127) / 128);
    if (a.dtype == CONVROT_BF16)
        launch_type<__bf16>(p, a.group, s);
    else
        launch_type<_Float16>(p, a.group, s);
}

void launch_quantize_grouped(const void* W, int64_t N, int64_t K, int group, int dtype, uint8_t* codes, void* scales,
                             uint8_t* zeros, hipStream_t s)
{
    if (dtype == CONVROT_BF16)
        quantize_type<__bf16>((const __bf16*)W, (int)N, (int)K, group, codes, (__bf16*)scales, zeros, s);
    else
        quantize_type<_Float16>((const _Float16*)W, (int)N, (int)K, group, codes, (_Float16*)scales, zeros, s);
}

}  // namespace convrot
