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
// position of a million keeps the accuracy of the first ones.  A wave works out
// its token's angles once for all the heads it takes, up to 32 of 128 bf16.
//
// Bound by memory where there are many tokens: 32768 tokens of 16 + 16 heads of
// 128 bf16 with norms, heads first, move 537 MB in 96 us (5.6 TB/s; a copy of
// 256 MB reaches 5.5).  1536 such tokens (25 MB) take 6.6 us (3.8 TB/s): the chip
// holds every wave at once, so what a wave waits for -- its position, its heads,
// sincos, the norm -- adds up instead of hiding behind other waves.  Heads are
// loaded and stored with the hint that they are used once (without it 104 and
// 9.6 us); the stores not where lanes are idle, which end inside lines (3 x 333
// tokens of 72 6.5 against 6.2 us).  One token of each of four sequences takes
// 3.0 us where an empty kernel takes 1.9; those tokens of 72, whose halves end
// inside a chunk, 6.1 us.
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
    int tile;   // rope_any_kernel: tokens a workgroup
    float eps, inv_dim;
    RopePlan plan;
};

// Position of (batch b, token t) on the axis of pair i.
__device__ __forceinline__ double place_of(const RopeParams& p, int64_t b, int64_t t, int i)
{
    const int64_t at = b * p.pos_batch + t * p.pos_token + p.plan.axis[i];
    return p.pos_dtype == CONVROT_F32 ? (double)((const float*)p.pos)[at] : (double)((const int32_t*)p.pos)[at];
}

// cos and sin of the angle of `turns` turns.
__device__ __forceinline__ float2 turned_by(double turns)
{
    turns -= rint(turns);
    float2 cs;
    sincospif(2.f * (float)turns, &cs.y, &cs.x);
    return cs;
}

enum Exchange { PAIRS, CHUNKS, ELEMENTS };   // how a lane gets the other elements of its pairs

// Even heads of at least one 16-byte chunk.  L lanes a head, lane c holding
// chunk c (the last one ends where the head ends, and may share elements with
// the one before it; both write the same values), so a wave holds 64 / L heads:
// one item.  A wave takes IW items of one token: it asks for all of them, works
// out the token's angles while they arrive, one or two a lane, and passes those
// on through its own part of shared memory; nothing waits for another wave.
//   PAIRS:    interleaved pairs, within the chunk
//   CHUNKS:   halves of whole chunks: the pairs' other elements are one lane's
//   ELEMENTS: halves of any size: through shared memory
// WHOLE: a head is L chunks, none of them shared.
// All loads of an item precede its stores: the output may be the input.
template <typename D, int L, Exchange EX, int IW, bool WHOLE>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeParams p)
{
    constexpr int V = 16 / sizeof(D), kHeads = 64 / L;
    typedef typename VecOf<D, V>::type Chunk;
    typedef uint32_t Words __attribute__((ext_vector_type(4)));
    __shared__ float2 angles[kThreads / 64][kMaxRopePairs];
    __shared__ __attribute__((aligned(16))) D rows[EX == ELEMENTS ? kThreads / 64 : 1][EX == ELEMENTS ? 64 * V : 1];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int64_t b = blockIdx.y, t = (int64_t)blockIdx.x * (kThreads / 64) + wave;
    if (t >= p.tokens) return;
    const int g = lane / L, c = lane % L;
    const bool in = WHOLE || c * V < p.dim;
    const int at = WHOLE ? c * V : min(c * V, p.dim - V), skip = c * V - at;
    const int items0 = (p.t[0].heads + kHeads - 1) / kHeads;
    const int items = items0 + (p.count > 1 ? (p.t[1].heads + kHeads - 1) / kHeads : 0);
    const int first = (int)blockIdx.z * IW;

    // Loads return in order: the positions are asked for before the heads, so
    // that the angles need not wait for those.
    constexpr int kPairs = kMaxRopePairs / 64;
    double turns[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
        if (lane + 64 * j < p.pairs) turns[j] = p.plan.turns[lane + 64 * j] * place_of(p, b, t, lane + 64 * j);

    // lane offsets within an item; everything else about it is the same for the wave
    const int64_t in0 = g * p.t[0].in_head + at, in1 = g * p.t[1].in_head + at;
    Chunk x[IW];
    bool has[IW];
#pragma unroll
    for (int u = 0; u < IW; ++u) {
        const bool second = first + u >= items0;
        const int head = (first + u - (second ? items0 : 0)) * kHeads;
        has[u] = first + u < items && in && head + g < (second ? p.t[1].heads : p.t[0].heads);
        const D* const base = second ? (const D*)p.t[1].in + b * p.t[1].in_batch + t * p.t[1].in_token + head * p.t[1].in_head
                                     : (const D*)p.t[0].in + b * p.t[0].in_batch + t * p.t[0].in_token + head * p.t[0].in_head;
        x[u] = Chunk{};
        if (has[u]) x[u] = load_once<D, V>(base + (second ? in1 : in0));
    }
    constexpr int kKinds = IW == 1 ? 1 : kMaxRopeTensors;   // tensors a wave may meet
    Chunk weight[kKinds];
#pragma unroll
    for (int k = 0; k < kKinds; ++k) {
        const D* const w = (const D*)(k == 1 || (IW == 1 && first >= items0) ? p.t[1].weight : p.t[0].weight);
#pragma unroll
        for (int i = 0; i < V; ++i) weight[k][i] = (D)1.f;
        if (w && in) weight[k] = load_chunk<D, V>(w + at);
    }
    float2* const cs = angles[wave];
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
        if (lane + 64 * j < p.pairs) cs[lane + 64 * j] = turned_by(turns[j]);
    wave_exchange();

    // the lane's part of the angles, the other lane of its pairs, and its weights there
    const int half = p.pairs / V;
    const bool upper = c >= half;   // CHUNKS: of the second half
    constexpr int kAngles = EX == PAIRS ? V / 2 : V;
    float2 a[kAngles];
    bool turned[kAngles];
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {
        const int e = EX == PAIRS ? at / 2 + i : at + i;   // of the pairs, of the elements
        turned[i] = EX == PAIRS ? e < p.pairs : e < 2 * p.pairs;
        a[i] = make_float2(1.f, 0.f);
        if (turned[i]) a[i] = cs[EX == PAIRS || e < p.pairs ? e : e - p.pairs];
        if (EX != PAIRS && e < p.pairs) a[i].y = -a[i].y;
    }
    const int other = 4 * ((lane & ~(L - 1)) + (upper ? c - half : c + half));
    const auto exchanged = [&](Chunk v) {
        if constexpr (EX == CHUNKS) {
            Words w = __builtin_bit_cast(Words, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t from = w[i];
                w[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(other, (int)from);
            }
            return __builtin_bit_cast(Chunk, w);
        } else {
            D* const row = rows[wave] + g * p.dim;
            if (in) store_chunk<D, V>(row + at, v);
            wave_exchange();
            Chunk o;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = at + i;
                o[i] = row[in && e < 2 * p.pairs ? (e < p.pairs ? e + p.pairs : e - p.pairs) : 0];
            }
            wave_exchange();
            return o;
        }
    };
    Chunk other_weight[kKinds];
    if (EX != PAIRS && p.norm)
#pragma unroll
        for (int k = 0; k < kKinds; ++k) other_weight[k] = exchanged(weight[k]);

    const int64_t out0 = g * p.t[0].out_head + at, out1 = g * p.t[1].out_head + at;
#pragma unroll
    for (int u = 0; u < IW; ++u) {
        const bool second = first + u >= items0;
        const int head = (first + u - (second ? items0 : 0)) * kHeads;
        float v[V], o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (float)x[u][i];
        if constexpr (EX != PAIRS) {
            const Chunk other_x = exchanged(x[u]);
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = (float)other_x[i];
        }
        if (p.norm) {
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) q = i >= skip ? fmaf(v[i], v[i], q) : q;
            const float rstd = rsqrtf(lane_sum<L>(q) * p.inv_dim + p.eps);
            const Chunk w = second ? weight[kKinds - 1] : weight[0];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] *= rstd * (float)w[i];
            if constexpr (EX != PAIRS) {
                const Chunk ow = second ? other_weight[kKinds - 1] : other_weight[0];
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] *= rstd * (float)ow[i];
            }
        }
        Chunk y;
        if constexpr (EX == PAIRS) {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const float2 t = a[i / 2];
                const float r0 = fmaf(v[i], t.x, -(v[i + 1] * t.y)), r1 = fmaf(v[i], t.y, v[i + 1] * t.x);
                y[i] = (D)(turned[i / 2] ? r0 : v[i]);
                y[i + 1] = (D)(turned[i / 2] ? r1 : v[i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = (D)(turned[i] ? fmaf(v[i], a[i].x, o[i] * a[i].y) : v[i]);
        }
        D* const base = second ? (D*)p.t[1].out + b * p.t[1].out_batch + t * p.t[1].out_token + head * p.t[1].out_head
                               : (D*)p.t[0].out + b * p.t[0].out_batch + t * p.t[0].out_token + head * p.t[0].out_head;
        D* const to = base + (second ? out1 : out0);
        if (has[u]) WHOLE ? store_once<D, V>(to, y) : store_chunk<D, V>(to, y);
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
        cs[i] = turned_by(place_of(p, b, t0 + t, i - t * p.pairs) * p.plan.turns[i - t * p.pairs]);
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

template <typename D, int L, Exchange EX, bool WHOLE>
void launch_items(const RopeParams& p, int batch, hipStream_t s)
{
    constexpr int kHeads = 64 / L, kWaves = kThreads / 64;
    const int items = (p.t[0].heads + kHeads - 1) / kHeads + (p.count > 1 ? (p.t[1].heads + kHeads - 1) / kHeads : 0);
    const int64_t all = (int64_t)p.tokens * batch * items;
    // Items a wave takes, one, four or eight: more of them share the token's
    // angles, fewer spread few tokens over more waves (one token of each of four
    // sequences 3.0, 3.7, 4.6 us; 1536 tokens of 32 heads 8.9, 6.6, 7.5; 32768 of
    // them 141 with one, 96 with eight).
    const auto grid = [&](int each) { return dim3((p.tokens + kWaves - 1) / kWaves, batch, (items + each - 1) / each); };
    if (all >= 64 * kUnits && items > 4)
        hipLaunchKernelGGL((rope_kernel<D, L, EX, 8, WHOLE>), grid(8), dim3(kThreads), 0, s, p);
    else if (all >= 16 * kUnits && items > 1)
        hipLaunchKernelGGL((rope_kernel<D, L, EX, 4, WHOLE>), grid(4), dim3(kThreads), 0, s, p);
    else
        hipLaunchKernelGGL((rope_kernel<D, L, EX, 1, WHOLE>), grid(1), dim3(kThreads), 0, s, p);
}

template <typename D, int L>
void launch_lanes(const RopeParams& p, bool halves, int batch, hipStream_t s)
{
    constexpr int V = 16 / sizeof(D);
    const bool whole = p.dim == L * V, chunks = p.dim % V == 0 && p.pairs % V == 0;
    if (halves && !chunks) launch_items<D, L, ELEMENTS, false>(p, batch, s);
    else if (halves) whole ? launch_items<D, L, CHUNKS, true>(p, batch, s) : launch_items<D, L, CHUNKS, false>(p, batch, s);
    else whole ? launch_items<D, L, PAIRS, true>(p, batch, s) : launch_items<D, L, PAIRS, false>(p, batch, s);
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
