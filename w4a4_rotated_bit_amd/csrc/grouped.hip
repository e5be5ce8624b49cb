// grouped.hip -- the group-scaled 4-bit linear's launch, and the quantizer that
// makes such weights.
#include "grouped_kernel.h"

namespace convrot {

void launch_grouped_bf16(const grouped::GroupedParams& p, int group, hipStream_t s);
void launch_grouped_f16(const grouped::GroupedParams& p, int group, hipStream_t s);

namespace {

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
    const float span = hi - lo, step = span < INFINITY ? span / 15.f : hi / 15.f - lo / 15.f;   // of finite bf16: up to 2^129
    const float s = bad ? NAN : (float)(D)(zeros ? step : hi / 7.f);
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
    grouped::GroupedParams p{};
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
    if (a.dtype == CONVROT_BF16)
        launch_grouped_bf16(p, a.group, s);
    else
        launch_grouped_f16(p, a.group, s);
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
