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
constexpr int kRopeEach = 4;   // heads a group of lanes

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
    int tile, parts, slots;   // tokens a workgroup, workgroups a token, heads a workgroup and token
    uint32_t per_slot;        // 65536 / slots, rounded up
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

enum Exchange { PAIRS, CHUNKS, ELEMENTS };   // how a lane gets the other elements of its pairs

// Even heads of at least one 16-byte chunk.  L lanes a head, lane c holding
// chunk c (the last one ends where the head ends, and may share elements with
// the one before it; both write the same values).  A workgroup takes `tile`
// tokens, or some of the heads of one, at most kEach heads a lane group: it asks
// for all of them first, then works out the angles while they arrive.
//   PAIRS:    interleaved pairs, within the chunk
//   CHUNKS:   halves of whole chunks: the pairs' other elements are one lane's
//   ELEMENTS: halves of any size: through shared memory
// Lanes of a head are in one wave, whose loads all precede its stores: the
// output may be the input.
template <typename D, int L, Exchange EX>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeParams p)
{
    constexpr int V = 16 / sizeof(D), kGroups = kThreads / L, kEach = kRopeEach;
    typedef typename VecOf<D, V>::type Chunk;
    typedef uint32_t Words __attribute__((ext_vector_type(4)));
    extern __shared__ __attribute__((aligned(16))) float shared[];
    float2* const cs = (float2*)shared;                                // [tile][pairs]
    float* const weights = shared + 2 * p.tile * p.pairs;              // [tensor][dim] where there are any
    D* const rows = (D*)(weights + (p.norm ? p.count * p.dim : 0));    // ELEMENTS: [group][dim]
    const int64_t b = blockIdx.y;
    const int part = (int)blockIdx.z % p.parts;                        // of a token's heads
    const int t0 = (int)(blockIdx.z / p.parts * gridDim.x + blockIdx.x) * p.tile, nt = min(p.tile, p.tokens - t0);
    const int group = threadIdx.x / L, c = threadIdx.x % L;
    if (nt <= 0) return;
    const int slots = p.slots, items = nt * slots;                     // heads a token here, heads here

    const bool in = c * V < p.dim;
    const int at = min(c * V, p.dim - V), skip = c * V - at;
    int tensor[kEach], token[kEach], head[kEach];
    Chunk x[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int item = group + u * kGroups;
        token[u] = (int)((uint32_t)item * p.per_slot >> 16);           // item / slots
        head[u] = item - token[u] * slots + part * slots;
        tensor[u] = head[u] >= p.t[0].heads;
        if (tensor[u]) head[u] -= p.t[0].heads;
        if (item >= items || (tensor[u] && (p.count < 2 || head[u] >= p.t[1].heads))) token[u] = -1;
        if (token[u] >= 0 && in) {
            const Heads& h = p.t[tensor[u]];
            x[u] = load_chunk<D, V>((const D*)h.in + b * h.in_batch + (t0 + token[u]) * h.in_token +
                                    head[u] * h.in_head + at);
        }
    }
    for (int i = threadIdx.x; i < nt * p.pairs; i += kThreads) {
        const int t = i / p.pairs;
        cs[i] = turn(p, b, t0 + t, i - t * p.pairs);
    }
    if (p.norm)
        for (int i = threadIdx.x; i < p.count * p.dim; i += kThreads) {
            const D* w = (const D*)p.t[i >= p.dim].weight;
            weights[i] = w ? (float)w[i >= p.dim ? i - p.dim : i] : 1.f;
        }
    __syncthreads();

#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        if (token[u] < 0) continue;   // the same for the lanes of a head
        float v[V], rstd = 1.f;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = in ? (float)x[u][i] : 0.f;
        if (p.norm) {
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) q = i >= skip ? fmaf(v[i], v[i], q) : q;
            rstd = 1.f / sqrtf(lane_sum<L>(q) * p.inv_dim + p.eps);
        }
        const float* const w = weights + tensor[u] * p.dim;
        const float2* const a = cs + token[u] * p.pairs;
        float o[V];   // the other elements
        const int half = p.pairs / V;
        const bool second = c >= half;
        if constexpr (EX == CHUNKS) {
            Words raw = __builtin_bit_cast(Words, x[u]);
            const int from = 4 * ((threadIdx.x & ~(L - 1) & 63) + (second ? c - half : c + half));
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)raw[i]);
            const Chunk other = __builtin_bit_cast(Chunk, raw);
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = (float)other[i];
        }
        if constexpr (EX == ELEMENTS) {
            D* const row = rows + group * p.dim;
            if (in) store_chunk<D, V>(row + at, x[u]);
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = at + i;
                o[i] = in && e < 2 * p.pairs ? (float)row[e < p.pairs ? e + p.pairs : e - p.pairs] : 0.f;
            }
            __builtin_amdgcn_wave_barrier();
        }
        if (!in) continue;
        if (p.norm)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[i] = v[i] * rstd * w[at + i];
                if constexpr (EX == CHUNKS)
                    if (at < 2 * p.pairs) o[i] = o[i] * rstd * w[(second ? at - p.pairs : at + p.pairs) + i];
                if constexpr (EX == ELEMENTS) {
                    const int e = at + i;
                    if (e < 2 * p.pairs) o[i] = o[i] * rstd * w[e < p.pairs ? e + p.pairs : e - p.pairs];
                }
            }
        Chunk y;
        if constexpr (EX == PAIRS) {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                float r0 = v[i], r1 = v[i + 1];
                if (at + i < 2 * p.pairs) {
                    const float2 t = a[(at + i) / 2];
                    r0 = fmaf(v[i], t.x, -(v[i + 1] * t.y));
                    r1 = fmaf(v[i], t.y, v[i + 1] * t.x);
                }
                y[i] = (D)r0;
                y[i + 1] = (D)r1;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = at + i;
                float r = v[i];
                if (EX == CHUNKS ? at < 2 * p.pairs : e < 2 * p.pairs) {
                    const bool two = EX == CHUNKS ? second : e >= p.pairs;
                    const float2 t = a[two ? e - p.pairs : e];
                    r = fmaf(v[i], t.x, o[i] * (two ? t.y : -t.y));
                }
                y[i] = (D)r;
            }
        }
        const Heads& h = p.t[tensor[u]];
        store_chunk<D, V>((D*)h.out + b * h.out_batch + (t0 + token[u]) * h.out_token + head[u] * h.out_head + at, y);
    }
}

// Heads of an odd size or shorter than a chunk: one wave a head, lane l holding
// elements l, l + 64, ...  All loads of a head come before its first
// store, so the output may be the input.
template <typename D>
__global__ __launch_bounds__(kThreads) void rope_any_kernel(RopeParams p, int halves)
{
    constexpr int kEach = kMaxHeadDim / 64;
    extern __shared__ float2 cs[];
    const int64_t b = blockIdx.y;
    const int t0 = (int)blockIdx.x * p.tile, nt = min(p.tile, p.tokens - t0);
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

template <typename D, int L>
void launch_lanes(RopeParams p, bool halves, int batch, hipStream_t s)
{
    constexpr int V = 16 / sizeof(D), kHeads = kThreads / L * kRopeEach;   // heads a workgroup
    const int heads = p.t[0].heads + (p.count > 1 ? p.t[1].heads : 0);
    p.parts = (heads + kHeads - 1) / kHeads;
    p.slots = (heads + p.parts - 1) / p.parts;
    p.tile = p.parts > 1 ? 1 : kHeads / heads;
    // fewer tokens a workgroup while there are units without one
    while (p.tile > 1 && (int64_t)((p.tokens + p.tile - 1) / p.tile) * batch < 2 * kUnits) p.tile = (p.tile + 1) / 2;
    p.per_slot = (65536 + p.slots - 1) / p.slots;
    // a grid dimension holds fewer than 2^32 threads
    const unsigned tiles = (p.tokens + p.tile - 1) / p.tile, gx = tiles < (1u << 20) ? tiles : 1u << 20;
    const dim3 grid(gx, batch, (tiles + gx - 1) / gx * p.parts);
    const bool chunks = halves && p.dim % V == 0 && p.pairs % V == 0;
    const size_t lds = sizeof(float2) * p.tile * p.pairs + (p.norm ? sizeof(float) * p.count * p.dim : 0) +
                       (halves && !chunks ? sizeof(D) * (kThreads / L) * p.dim : 0);
    if (!halves)
        hipLaunchKernelGGL((rope_kernel<D, L, PAIRS>), grid, dim3(kThreads), lds, s, p);
    else if (chunks)
        hipLaunchKernelGGL((rope_kernel<D, L, CHUNKS>), grid, dim3(kThreads), lds, s, p);
    else
        hipLaunchKernelGGL((rope_kernel<D, L, ELEMENTS>), grid, dim3(kThreads), lds, s, p);
}

template <typename D>
void launch_type(RopeParams p, bool halves, int batch, hipStream_t s)
{
    constexpr int V = 16 / sizeof(D);
    if (p.dim < V || p.dim % 2 != 0) {
        p.tile = 4;
        hipLaunchKernelGGL((rope_any_kernel<D>), dim3((p.tokens + p.tile - 1) / p.tile, batch), dim3(kThreads),
                           sizeof(float2) * p.tile * p.pairs, s, p, halves ? 1 : 0);
        return;
    }
    const int chunks = (p.dim + V - 1) / V;
    if (chunks <= 4) launch_lanes<D, 4>(p, halves, batch, s);
    else if (chunks <= 8) launch_lanes<D, 8>(p, halves, batch, s);
    else if (chunks <= 16) launch_lanes<D, 16>(p, halves, batch, s);
    else if (chunks <= 32) launch_lanes<D, 32>(p, halves, batch, s);
    else launch_lanes<D, 64>(p, halves, batch, s);
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
    const bool halves = a.layout == CONVROT_ROPE_HALVES;
    if (a.dtype == CONVROT_BF16)
        launch_type<__bf16>(p, halves, (int)a.batch, s);
    else if (a.dtype == CONVROT_F16)
        launch_type<_Float16>(p, halves, (int)a.batch, s);
    else
        launch_type<float>(p, halves, (int)a.batch, s);
}

}  // namespace convrot
