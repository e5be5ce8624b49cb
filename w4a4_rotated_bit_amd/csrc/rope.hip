// rope.hip -- rotary positions over several axes for the query and key heads.
//
// Pair i of a head is turned by the angle positions[axis_i] * freq_i:
//   (u, v) -> (u cos - v sin, u sin + v cos),
// u and v being elements 2i, 2i + 1 (interleaved) or i, i + pairs (halves);
// elements from 2 pairs on pass through.  In front of it, where asked for, the
// head's RMS norm: x / sqrt(mean(x^2) + eps) * weight.
//
// The angle is formed in binary64 as turns (frequencies come divided by 2 pi)
// and only its fraction of a turn goes on to binary32 sine and cosine: a
// position of a million keeps the accuracy of the first ones.  Every token's
// angles are computed once by its workgroup and shared by all its heads.
#include "block_ops.h"

namespace convrot {

namespace {

constexpr int kThreads = 256;

struct Heads {
    const void* in;
    void* out;
    const void* weight;
    int64_t in_batch, in_token, in_head, out_batch, out_token, out_head;
    int heads;
};

struct RopeParams {
    Heads t[kMaxRopeTensors];
    const void* pos;
    int64_t pos_batch, pos_token;
    int count, tokens, dim, pairs, pos_dtype, norm;
    float eps, inv_dim;
    RopePlan plan;
};

// cos and sin of pair i at the position of (batch b, token t)
__device__ __forceinline__ float2 turn(const RopeParams& p, int64_t b, int64_t t, int i)
{
    const int64_t at = b * p.pos_batch + t * p.pos_token + p.plan.axis[i];
    const double place = p.pos_dtype == CONVROT_F32 ? (double)((const float*)p.pos)[at]
                                                    : (double)((const int32_t*)p.pos)[at];
    double turns = place * p.plan.turns[i];
    turns -= rint(turns);
    float2 cs;
    sincospif(2.f * (float)turns, &cs.y, &cs.x);
    return cs;
}

// Heads of V-element chunks, V elements being 16 bytes and the rotated part
// whole chunks (of both halves): L lanes a head, lane c holds chunk c.
template <typename D, int L, bool HALVES>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeParams p, int tile)
{
    constexpr int V = 16 / sizeof(D);
    typedef typename VecOf<D, V>::type Chunk;
    extern __shared__ float2 cs[];   // [tile][pairs]
    const int64_t b = blockIdx.y;
    const int t0 = (int)blockIdx.x * tile, nt = min(tile, p.tokens - t0);
    for (int i = threadIdx.x; i < nt * p.pairs; i += kThreads) {
        const int t = i / p.pairs;
        cs[i] = turn(p, b, t0 + t, i - t * p.pairs);
    }
    __syncthreads();

    const int c = threadIdx.x % L, chunks = p.dim / V;
    const bool in = c < chunks;
    const int half = p.pairs / V;            // HALVES: chunks of one half
    const bool rotated = c * V < 2 * p.pairs;
    const bool second = HALVES && c >= half;
    for (int k = 0; k < p.count; ++k) {
        const Heads& h = p.t[k];
        float w[V];
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = 1.f;
        if (h.weight && in) load_f32<D, V>((const D*)h.weight + c * V, w);
        const int items = nt * h.heads;
        for (int item = threadIdx.x / L; item < items; item += kThreads / L) {
            const int t = item / h.heads, head = item - t * h.heads;
            float x[V];
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = 0.f;
            if (in)
                load_f32<D, V>((const D*)h.in + b * h.in_batch + (t0 + t) * h.in_token + head * h.in_head + c * V, x);
            if (p.norm) {
                float q = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) q = fmaf(x[i], x[i], q);
                const float rstd = 1.f / sqrtf(lane_sum<L>(q) * p.inv_dim + p.eps);
#pragma unroll
                for (int i = 0; i < V; ++i) x[i] = x[i] * rstd * w[i];
            }
            float y[V];
            if constexpr (HALVES) {
                const int other = (threadIdx.x & ~(L - 1)) + (second ? c - half : c + half);
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] = __shfl(x[i], other, 64);
            }
            if (!in) continue;
            if (rotated) {
                const float2* a = cs + t * p.pairs;
                if constexpr (HALVES) {
                    a += (second ? c - half : c) * V;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float s = second ? a[i].y : -a[i].y;
                        x[i] = fmaf(x[i], a[i].x, y[i] * s);
                    }
                } else {
                    a += c * (V / 2);
#pragma unroll
                    for (int i = 0; i < V; i += 2) {
                        const float u = x[i], v = x[i + 1];
                        x[i] = fmaf(u, a[i / 2].x, -(v * a[i / 2].y));
                        x[i + 1] = fmaf(u, a[i / 2].y, v * a[i / 2].x);
                    }
                }
            }
            store_f32<D, V>((D*)h.out + b * h.out_batch + (t0 + t) * h.out_token + head * h.out_head + c * V, x);
        }
    }
}

// Any head size, rotated width, alignment and stride: one wave a head, lane l
// holding elements l, l + 64, ...  All loads of a head come before its first
// store, so the output may be the input.
template <typename D>
__global__ __launch_bounds__(kThreads) void rope_any_kernel(RopeParams p, int tile, int halves)
{
    constexpr int kEach = kMaxHeadDim / 64;
    extern __shared__ float2 cs[];
    const int64_t b = blockIdx.y;
    const int t0 = (int)blockIdx.x * tile, nt = min(tile, p.tokens - t0);
    for (int i = threadIdx.x; i < nt * p.pairs; i += kThreads) {
        const int t = i / p.pairs;
        cs[i] = turn(p, b, t0 + t, i - t * p.pairs);
    }
    __syncthreads();
    const int lane = threadIdx.x % 64;
    for (int k = 0; k < p.count; ++k) {
        const Heads& h = p.t[k];
        const int items = nt * h.heads;
        for (int item = threadIdx.x / 64; item < items; item += kThreads / 64) {
            const int t = item / h.heads, head = item - t * h.heads;
            const D* x = (const D*)h.in + b * h.in_batch + (t0 + t) * h.in_token + head * h.in_head;
            float u[kEach], v[kEach];   // an element and the other one of its pair
            float q = 0.f;
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const int e = lane + 64 * j;
                u[j] = v[j] = 0.f;
                if (e >= p.dim) continue;
                u[j] = (float)x[e];
                const int o = halves ? (e < p.pairs ? e + p.pairs : e - p.pairs) : e ^ 1;
                if (e < 2 * p.pairs) v[j] = (float)x[o];
                q = fmaf(u[j], u[j], q);
                if (h.weight) {
                    u[j] *= (float)((const D*)h.weight)[e];
                    if (e < 2 * p.pairs) v[j] *= (float)((const D*)h.weight)[o];
                }
            }
            const float rstd = p.norm ? 1.f / sqrtf(lane_sum<64>(q) * p.inv_dim + p.eps) : 1.f;
            D* out = (D*)h.out + b * h.out_batch + (t0 + t) * h.out_token + head * h.out_head;
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const int e = lane + 64 * j;
                if (e >= p.dim) continue;
                float r = u[j] * rstd;
                if (e < 2 * p.pairs) {
                    const bool second = halves ? e >= p.pairs : e & 1;
                    const float2 a = cs[t * p.pairs + (halves ? (second ? e - p.pairs : e) : e / 2)];
                    r = fmaf(r, a.x, v[j] * rstd * (second ? a.y : -a.y));
                }
                out[e] = (D)r;
            }
        }
    }
}

bool wide_ok(const convrot_heads& h, int64_t batch, int V)
{
    const bool strides = h.in_token_stride % V == 0 && h.in_head_stride % V == 0 && h.out_token_stride % V == 0 &&
                         h.out_head_stride % V == 0 &&
                         (batch == 1 || (h.in_batch_stride % V == 0 && h.out_batch_stride % V == 0));
    return strides && (uintptr_t)h.in_dev % 16 == 0 && (uintptr_t)h.out_dev % 16 == 0 &&
           (uintptr_t)h.weight_dev % 16 == 0;
}

template <typename D, int L>
void launch_lanes(const RopeParams& p, int tile, bool halves, dim3 grid, size_t lds, hipStream_t s)
{
    if (halves)
        hipLaunchKernelGGL((rope_kernel<D, L, true>), grid, dim3(kThreads), lds, s, p, tile);
    else
        hipLaunchKernelGGL((rope_kernel<D, L, false>), grid, dim3(kThreads), lds, s, p, tile);
}

template <typename D>
void launch_type(const convrot_rope_args& a, const RopeParams& p, hipStream_t s)
{
    constexpr int V = 16 / sizeof(D);
    const bool halves = a.layout == CONVROT_ROPE_HALVES;
    const int tile = 4;
    const dim3 grid((p.tokens + tile - 1) / tile, (unsigned)a.batch);
    const size_t lds = sizeof(float2) * tile * p.pairs;
    bool wide = p.dim % V == 0 && (halves ? p.pairs % V == 0 : 2 * p.pairs % V == 0);
    for (int k = 0; k < a.count; ++k) wide = wide && wide_ok(a.heads[k], a.batch, V);
    if (!wide) {
        hipLaunchKernelGGL((rope_any_kernel<D>), grid, dim3(kThreads), lds, s, p, tile, halves ? 1 : 0);
        return;
    }
    const int chunks = p.dim / V;
    if (chunks <= 4) launch_lanes<D, 4>(p, tile, halves, grid, lds, s);
    else if (chunks <= 8) launch_lanes<D, 8>(p, tile, halves, grid, lds, s);
    else if (chunks <= 16) launch_lanes<D, 16>(p, tile, halves, grid, lds, s);
    else if (chunks <= 32) launch_lanes<D, 32>(p, tile, halves, grid, lds, s);
    else launch_lanes<D, 64>(p, tile, halves, grid, lds, s);
}

}  // namespace

void launch_rope(const convrot_rope_args& a, const RopePlan& plan, hipStream_t s)
{
    RopeParams p{};
    for (int k = 0; k < a.count; ++k) {
        const convrot_heads& h = a.heads[k];
        p.t[k] = {h.in_dev, h.out_dev, h.weight_dev, h.in_batch_stride, h.in_token_stride, h.in_head_stride,
                  h.out_batch_stride, h.out_token_stride, h.out_head_stride, (int)h.heads};
    }
    p.pos = a.pos_dev;
    p.pos_batch = a.pos_batch_stride;
    p.pos_token = a.pos_token_stride;
    p.count = a.count;
    p.tokens = (int)a.tokens;
    p.dim = a.head_dim;
    p.pairs = a.pairs;
    p.pos_dtype = a.pos_dtype;
    p.norm = a.norm;
    p.eps = a.eps;
    p.inv_dim = 1.f / (float)a.head_dim;
    p.plan = plan;
    if (a.dtype == CONVROT_BF16)
        launch_type<__bf16>(a, p, s);
    else if (a.dtype == CONVROT_F16)
        launch_type<_Float16>(a, p, s);
    else
        launch_type<float>(a, p, s);
}

}  // namespace convrot
