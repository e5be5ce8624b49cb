// norm.hip -- the residual update of a transformer sub-block with the norms on
// both sides of it:
//
//   z = P(y)                       P: nothing, LayerNorm or RMS norm, times post_weight
//   r = a x + gate * z
//   h = N(r) weight (1 + scale) + shift
//
// One row is held in the registers of T threads from its first load to its
// last store, so each of x, y, r and h crosses memory once; the statistics are
// sums of binary32 in registers, and N works on r as it is before its rounding
// to the storage type.  LayerNorm's mean is found twice: a first one, off by the
// roundings of a sum of the row's full size, is taken away from the row, and the
// mean of what is left, found in the same pass as its squares, is taken out of
// both.  Its roundings are those of the deviations, so a mean far from zero costs
// nothing (in rows of one value, 1000, the first mean alone left up to 0.06 in h).
//
// Bound by memory: 32768 rows of 4096 bf16 with both norms, every vector and
// both outputs move 1.07 GB in 194 us (5.5 TB/s; a copy of that size reaches
// 5.0 TB/s, one of 256 MB 5.5), 1536 rows 50 MB in 10.3 us (4.9 TB/s).  Rows are
// loaded and stored with the hint that they are used once, without it 204 and
// 12.5 us (16384 rows of 2048, whose 268 MB the last cache all but holds, 48.4
// with it and 44.8 without); not where a chunk does not divide the width, whose
// chunks share lines (999 rows of 1035: 6.8 us with and without).  Short inputs
// are bound by latency: one row of 4096 takes 2.4 us where an empty kernel takes
// 1.9, and 999 rows of 1035 f16, two norms, 6.8 us: four exchanges across the
// workgroup one after the other, and chunks that cross lines of memory.
//
// One row a workgroup, and nothing else kept from row to row: workgroups that
// went on to further rows, with the vectors in registers, held fewer rows in
// flight (250 against 215 us for the 32768 rows, before that hint).
#include "block_ops.h"

namespace convrot {

namespace {

struct NormParams {
    const void *x, *y, *gate, *scale, *shift, *weight, *post_weight;
    void *r, *h;
    int64_t x_stride, y_stride, r_stride, h_stride, gate_stride, scale_stride, shift_stride;
    int rows, rows_per_vec, width;
    int norm, post_norm;
    float a, eps, inv_width;
    bool in_place;   // r or h is x or y
};

// Sums of C values over the T threads of a row; every exchange of a kernel has
// slots of its own, so one barrier is enough.
template <int T, int C>
__device__ __forceinline__ void row_sums(float (&v)[C], float* slot)
{
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = lane_sum<64>(v[c]);
    if constexpr (T > 64) {
        const int wave = threadIdx.x / 64;
        if (threadIdx.x % 64 == 0) {
#pragma unroll
            for (int c = 0; c < C; ++c) slot[C * wave + c] = v[c];
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; ++c) {
            v[c] = 0.f;
#pragma unroll
            for (int w = 0; w < T / 64; ++w) v[c] += slot[C * w + c];
        }
    }
}

// D: type of the rows, E: of the vectors.  T threads a row, NV chunks of V
// elements a thread.  EARLY: the vectors are loaded with the row, before its
// sums, instead of where they are needed.
//
// TAIL: V does not divide the width.  The last chunk then ends where the row
// ends and begins inside the chunk before it; the elements both have are left
// out of its sums, and stored twice with the same value.
template <typename D, typename E, int T, int V, int NV, bool TAIL, bool EARLY>
__global__ __launch_bounds__(T < 256 ? 256 : T) void residual_norm_kernel(NormParams p)
{
    constexpr int kRows = T < 256 ? 256 / T : 1;   // rows at a time
    static_assert(T == 64 || kRows == 1, "several rows share a workgroup only where a row is one wave");
    typedef typename VecOf<D, V>::type Chunk;
    typedef typename VecOf<E, V>::type Vector;
    constexpr int kSlots = T > 64 ? 3 * (T / 64) : 0;   // of one norm: a sum, then a pair
    __shared__ float slots[T > 64 ? 2 * kSlots : 1];
    const int t = threadIdx.x % T;
    const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kRows + threadIdx.x / T;

    int at[NV], skip[NV];   // a chunk's first element, and how many of its elements the chunk before it has
    bool in[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        at[j] = (j * T + t) * V;
        in[j] = at[j] < p.width;
        skip[j] = 0;
        if (TAIL && at[j] + V > p.width) {
            skip[j] = in[j] ? at[j] + V - p.width : V;
            at[j] = p.width - V;
        }
    }
    const auto load_vector = [&](Vector (&to)[NV], const void* from) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (in[j]) to[j] = load_chunk<E, V>((const E*)from + at[j]);
    };
    // f(j, i) for every element
    const auto all = [&](auto&& f) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) f(j, i);
    };
    // v -> (v - mean) rstd, with the sums of the row in `slots`
    const auto normalise = [&](float (&v)[NV][V], int kind, float* slots) {
        const auto own = [&](int j, int i) { return in[j] && (!TAIL || i >= skip[j]) ? v[j][i] : 0.f; };
        if (kind == CONVROT_NORM_LAYER) {
            float first[1] = {0.f}, rest[2] = {0.f, 0.f};
            all([&](int j, int i) { first[0] += own(j, i); });
            row_sums<T>(first, slots);
            float mean = first[0] * p.inv_width;
            asm volatile("" : "+v"(mean));   // rounded, for every element: some subtractions would take the product in
            all([&](int j, int i) { v[j][i] -= mean; });
            all([&](int j, int i) {
                const float d = own(j, i);
                rest[0] += d;
                rest[1] = fmaf(d, d, rest[1]);
            });
            row_sums<T>(rest, slots + T / 64);
            const float left = rest[0] * p.inv_width;
            const float var = fmaxf(fmaf(-left, left, rest[1] * p.inv_width), 0.f);
            const float rstd = 1.f / sqrtf(var + p.eps);
            all([&](int j, int i) { v[j][i] = fmaf(v[j][i], rstd, -left * rstd); });
        } else {
            float q[1] = {0.f};
            all([&](int j, int i) { q[0] = fmaf(own(j, i), own(j, i), q[0]); });
            row_sums<T>(q, slots);
            const float rstd = 1.f / sqrtf(q[0] * p.inv_width + p.eps);
            all([&](int j, int i) { v[j][i] *= rstd; });
        }
    };

    if (row >= p.rows) return;   // whole waves; a workgroup with barriers has one row
    Vector gate[NV], scale[NV], shift[NV], weight[NV], post_weight[NV];
    const D* const xp = (const D*)p.x + row * p.x_stride;
    const D* const yp = (const D*)p.y + row * p.y_stride;
    const auto load = [](const D* p) { return TAIL ? load_chunk<D, V>(p) : load_once<D, V>(p); };
    Chunk x[NV], y[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (in[j]) x[j] = load(xp + at[j]);
    if (p.y) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (in[j]) y[j] = load(yp + at[j]);
    }
    const int64_t vec = row / p.rows_per_vec;
    const E* const gate_p = (const E*)p.gate + vec * p.gate_stride;
    const E* const scale_p = (const E*)p.scale + vec * p.scale_stride;
    const E* const shift_p = (const E*)p.shift + vec * p.shift_stride;
    if (EARLY) {
        if (p.post_weight) load_vector(post_weight, p.post_weight);
        if (p.weight) load_vector(weight, p.weight);
        if (p.gate) load_vector(gate, gate_p);
        if (p.scale) load_vector(scale, scale_p);
        if (p.shift) load_vector(shift, shift_p);
    }
    if (TAIL && T > 64 && p.in_place) {   // every wave has read what the last chunk shares before it is written
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    }
    float r[NV][V];
    all([&](int j, int i) { r[j][i] = p.a * (float)x[j][i]; });
    if (p.y) {
        float z[NV][V];
        all([&](int j, int i) { z[j][i] = (float)y[j][i]; });
        if (p.post_norm != CONVROT_NORM_NONE) {
            normalise(z, p.post_norm, slots);
            if (p.post_weight) {
                if (!EARLY) load_vector(post_weight, p.post_weight);
                all([&](int j, int i) { z[j][i] *= (float)post_weight[j][i]; });
            }
        }
        if (p.gate) {
            if (!EARLY) load_vector(gate, gate_p);
            all([&](int j, int i) { r[j][i] = fmaf((float)gate[j][i], z[j][i], r[j][i]); });
        } else {
            all([&](int j, int i) { r[j][i] += z[j][i]; });
        }
    }
    const auto store = [&](D* to) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            Chunk c;
#pragma unroll
            for (int i = 0; i < V; ++i) c[i] = (D)r[j][i];
            if (in[j]) TAIL ? store_chunk<D, V>(to + at[j], c) : store_once<D, V>(to + at[j], c);
        }
    };
    if (p.r) store((D*)p.r + row * p.r_stride);
    if (!p.h) return;
    if (p.norm != CONVROT_NORM_NONE) normalise(r, p.norm, slots + kSlots);
    if (p.weight) {
        if (!EARLY) load_vector(weight, p.weight);
        all([&](int j, int i) { r[j][i] *= (float)weight[j][i]; });
    }
    if (p.scale) {
        if (!EARLY) load_vector(scale, scale_p);
        all([&](int j, int i) { r[j][i] = fmaf(r[j][i], (float)scale[j][i], r[j][i]); });
    }
    if (p.shift) {
        if (!EARLY) load_vector(shift, shift_p);
        all([&](int j, int i) { r[j][i] += (float)shift[j][i]; });
    }
    store((D*)p.h + row * p.h_stride);
}

template <typename D, typename E, int T, int V, int NV, bool TAIL>
void launch_one(const NormParams& p, hipStream_t s)
{
    constexpr int kThreads = T < 256 ? 256 : T, kRows = kThreads / T;
    // a grid dimension holds fewer than 2^32 threads
    const unsigned blocks = (p.rows + kRows - 1) / kRows, gx = blocks < (1u << 20) ? blocks : 1u << 20;
    // Registers for the vectors too only where that leaves as many rows
    // resident: 16384 rows of 2048 48.4 us with, 49.4 without, 1536 of 4096 (two
    // chunks a thread) 12.6 with, 10.3 without.
    hipLaunchKernelGGL((residual_norm_kernel<D, E, T, V, NV, TAIL, (NV == 1)>), dim3(gx, (blocks + gx - 1) / gx),
                       dim3(kThreads), 0, s, p);
}

template <typename D, typename E, bool TAIL>
void launch_width(const NormParams& p, hipStream_t s)
{
    constexpr int V = 16 / sizeof(D);
    const int chunks = (p.width + V - 1) / V;
    // A row of up to 128 chunks is one wave's and needs no barrier; from there on
    // a thread of a workgroup has one chunk (999 rows of 130 chunks: 6.8 us, one
    // wave with three chunks a lane 6.95), or two, which holds more rows in
    // flight (1536 rows of 512 chunks: 10.3 us, with one chunk a thread 12.9),
    // unless there are fewer rows than units (one row of 512 chunks: 2.4 us with
    // one chunk a thread, 2.6 with two).
    if (chunks <= 64) launch_one<D, E, 64, V, 1, TAIL>(p, s);
    else if (chunks <= 128) launch_one<D, E, 64, V, 2, TAIL>(p, s);
    else if (chunks <= 256) launch_one<D, E, 256, V, 1, TAIL>(p, s);
    else if (chunks <= 512 && p.rows <= kUnits) launch_one<D, E, 512, V, 1, TAIL>(p, s);
    else if (chunks <= 512) launch_one<D, E, 256, V, 2, TAIL>(p, s);
    else if (chunks <= 1024) launch_one<D, E, 512, V, 2, TAIL>(p, s);
    else if (chunks <= 2048) launch_one<D, E, 1024, V, 2, TAIL>(p, s);
    else if constexpr (V == 4) launch_one<D, E, 1024, V, 4, TAIL>(p, s);
}

template <typename D, typename E>
void launch_types(const NormParams& p, hipStream_t s)
{
    constexpr int V = 16 / sizeof(D);
    if (p.width < V) launch_one<D, E, 64, 1, 1, false>(p, s);   // shorter than a chunk
    else if (p.width % V == 0) launch_width<D, E, false>(p, s);
    else launch_width<D, E, true>(p, s);
}

}  // namespace

void launch_residual_norm(const convrot_residual_norm_args& a, hipStream_t s)
{
    NormParams p{};
    p.x = a.x_dev;
    p.y = a.y_dev;
    p.gate = a.gate_dev;
    p.scale = a.scale_dev;
    p.shift = a.shift_dev;
    p.weight = a.weight_dev;
    p.post_weight = a.post_weight_dev;
    p.r = a.r_dev;
    p.h = a.h_dev;
    p.x_stride = a.x_stride;
    p.y_stride = a.y_stride;
    p.r_stride = a.r_stride;
    p.h_stride = a.h_stride;
    p.gate_stride = a.gate_stride;
    p.scale_stride = a.scale_stride;
    p.shift_stride = a.shift_stride;
    p.rows = (int)a.rows;
    p.rows_per_vec = (int)(a.rows_per_vec < a.rows ? a.rows_per_vec : a.rows);
    p.width = (int)a.width;
    p.norm = a.norm;
    p.post_norm = a.y_dev ? a.post_norm : CONVROT_NORM_NONE;
    p.a = a.residual_scale;
    p.eps = a.eps;
    p.inv_width = 1.f / (float)a.width;
    p.in_place = a.r_dev == a.x_dev || a.h_dev == a.x_dev || (a.y_dev && (a.r_dev == a.y_dev || a.h_dev == a.y_dev));
    const bool f32v = a.vec_dtype == CONVROT_F32;
    if (a.dtype == CONVROT_BF16)
        f32v ? launch_types<__bf16, float>(p, s) : launch_types<__bf16, __bf16>(p, s);
    else if (a.dtype == CONVROT_F16)
        f32v ? launch_types<_Float16, float>(p, s) : launch_types<_Float16, _Float16>(p, s);
    else
        launch_types<float, float>(p, s);
}

}  // namespace convrot
