// norm.hip -- the residual update of a transformer sub-block with the norms on
// both sides of it:
//
//   z = P(y)                       P: nothing, LayerNorm or RMS norm, times post_weight
//   r = a x + gate * z
//   h = N(r) weight (1 + scale) + shift
//
// One row is held in the registers of T threads from its first load to its
// last store, so each of x, y, r and h crosses memory once; the statistics are
// sums of binary32 in registers (LayerNorm: the mean first, then the squared
// deviations, so that a large mean costs nothing), and N works on r as it is
// before its rounding to the storage type.
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
};

// Sum over the T threads of a row.  `slot` alternates between calls, so that
// one barrier a call is enough: a thread writes a slot again only after a
// barrier that every thread reached after reading it.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* slot)
{
    v = lane_sum<64>(v);
    if constexpr (T > 64) {
        const int wave = threadIdx.x / 64;
        if (threadIdx.x % 64 == 0) slot[wave] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < T / 64; ++w) v += slot[w];
    }
    return v;
}

// Row statistics of v: the factor and offset of v -> (v - mean) / sqrt(var + eps).
template <int T, int V, int NV>
__device__ __forceinline__ void row_stats(const float (&v)[NV][V], const bool (&in)[NV], int kind, float inv_width,
                                          float eps, float* slots, float& mean, float& rstd)
{
    mean = 0.f;
    if (kind == CONVROT_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) s += v[j][i];   // zero outside the row
        mean = row_sum<T>(s, slots) * inv_width;
    }
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (in[j])
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = v[j][i] - mean;
                q = fmaf(d, d, q);
            }
    rstd = 1.f / sqrtf(row_sum<T>(q, slots + T / 64) * inv_width + eps);
}

// T threads a row, NV chunks of V elements a thread.
template <typename D, typename E, int T, int V, int NV>
__global__ __launch_bounds__(T < 256 ? 256 : T) void residual_norm_kernel(NormParams p)
{
    constexpr int kRows = T < 256 ? 256 / T : 1;   // rows a workgroup
    static_assert(T == 64 || kRows == 1, "several rows share a workgroup only where a row is one wave");
    __shared__ float slots[T > 64 ? 4 * (T / 64) : 1];
    const int t = threadIdx.x % T;
    const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kRows + threadIdx.x / T;
    if (row >= p.rows) return;   // whole waves; a workgroup with barriers has one row
    const int64_t vec = row / p.rows_per_vec;

    int at[NV];
    bool in[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        at[j] = (j * T + t) * V;
        in[j] = at[j] < p.width;
    }
    const D* x = (const D*)p.x + row * p.x_stride;
    float r[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) r[j][i] = 0.f;
        if (in[j]) load_f32<D, V>(x + at[j], r[j]);
    }
    if (p.y) {
        const D* y = (const D*)p.y + row * p.y_stride;
        float z[NV][V];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < V; ++i) z[j][i] = 0.f;
            if (in[j]) load_f32<D, V>(y + at[j], z[j]);
        }
        if (p.post_norm != CONVROT_NORM_NONE) {
            float mean, rstd;
            row_stats<T, V, NV>(z, in, p.post_norm, p.inv_width, p.eps, slots, mean, rstd);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float w[V];
#pragma unroll
                for (int i = 0; i < V; ++i) w[i] = 1.f;
                if (p.post_weight && in[j]) load_f32<E, V>((const E*)p.post_weight + at[j], w);
#pragma unroll
                for (int i = 0; i < V; ++i) z[j][i] = (z[j][i] - mean) * rstd * w[i];
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float g[V];
#pragma unroll
            for (int i = 0; i < V; ++i) g[i] = 1.f;
            if (p.gate && in[j]) load_f32<E, V>((const E*)p.gate + vec * p.gate_stride + at[j], g);
#pragma unroll
            for (int i = 0; i < V; ++i) r[j][i] = fmaf(g[i], z[j][i], p.a * r[j][i]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) r[j][i] *= p.a;
    }
    if (p.r) {
        D* out = (D*)p.r + row * p.r_stride;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (in[j]) store_f32<D, V>(out + at[j], r[j]);
    }
    if (!p.h) return;

    if (p.norm != CONVROT_NORM_NONE) {
        // elements outside the row have to stay out of the sums
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (!in[j])
#pragma unroll
                for (int i = 0; i < V; ++i) r[j][i] = 0.f;
        float mean, rstd;
        row_stats<T, V, NV>(r, in, p.norm, p.inv_width, p.eps, slots + (T > 64 ? 2 * (T / 64) : 0), mean, rstd);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) r[j][i] = (r[j][i] - mean) * rstd;
    }
    D* out = (D*)p.h + row * p.h_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (!in[j]) continue;
        float v[V];
        if (p.weight) {
            load_f32<E, V>((const E*)p.weight + at[j], v);
#pragma unroll
            for (int i = 0; i < V; ++i) r[j][i] *= v[i];
        }
        if (p.scale) {
            load_f32<E, V>((const E*)p.scale + vec * p.scale_stride + at[j], v);
#pragma unroll
            for (int i = 0; i < V; ++i) r[j][i] = fmaf(r[j][i], v[i], r[j][i]);
        }
        if (p.shift) {
            load_f32<E, V>((const E*)p.shift + vec * p.shift_stride + at[j], v);
#pragma unroll
            for (int i = 0; i < V; ++i) r[j][i] += v[i];
        }
        store_f32<D, V>(out + at[j], r[j]);
    }
}

template <typename D, typename E, int T, int V, int NV>
void launch_one(const NormParams& p, hipStream_t s)
{
    constexpr int kRows = T < 256 ? 256 / T : 1;
    // a grid dimension holds fewer than 2^32 threads
    const unsigned blocks = (p.rows + kRows - 1) / kRows, gx = blocks < (1u << 20) ? blocks : 1u << 20;
    hipLaunchKernelGGL((residual_norm_kernel<D, E, T, V, NV>), dim3(gx, (blocks + gx - 1) / gx),
                       dim3(T < 256 ? 256 : T), 0, s, p);
}

template <typename D, typename E, int V>
void launch_width(const NormParams& p, hipStream_t s)
{
    const int chunks = (p.width + V - 1) / V;
    if (chunks <= 64) return launch_one<D, E, 64, V, 1>(p, s);
    if (chunks <= 256) return launch_one<D, E, 256, V, 1>(p, s);
    if (chunks <= 512) return launch_one<D, E, 256, V, 2>(p, s);
    if (chunks <= 1024) return launch_one<D, E, 256, V, 4>(p, s);
    if (chunks <= 2048) return launch_one<D, E, 1024, V, 2>(p, s);
    if (chunks <= 4096) return launch_one<D, E, 1024, V, 4>(p, s);
    if constexpr (V == 1) launch_one<D, E, 1024, V, 16>(p, s);   // up to 16384 scalars
}

bool vec_ok(const void* p, int64_t stride, int bytes, int V)
{
    return !p || ((uintptr_t)p % (V * bytes < 16 ? V * bytes : 16) == 0 && stride % V == 0);
}

template <typename D, typename E>
void launch_types(const convrot_residual_norm_args& a, const NormParams& p, hipStream_t s)
{
    constexpr int V = 16 / sizeof(D);
    const int db = sizeof(D), eb = sizeof(E);
    const bool wide = a.width % V == 0 && vec_ok(a.x_dev, a.x_stride, db, V) && vec_ok(a.y_dev, a.y_stride, db, V) &&
                      vec_ok(a.r_dev, a.r_stride, db, V) && vec_ok(a.h_dev, a.h_stride, db, V) &&
                      vec_ok(a.gate_dev, a.gate_stride, eb, V) && vec_ok(a.scale_dev, a.scale_stride, eb, V) &&
                      vec_ok(a.shift_dev, a.shift_stride, eb, V) && vec_ok(a.weight_dev, 0, eb, V) &&
                      vec_ok(a.post_weight_dev, 0, eb, V);
    if (wide)
        launch_width<D, E, V>(p, s);
    else
        launch_width<D, E, 1>(p, s);
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
    p.rows_per_vec = (int)a.rows_per_vec;
    p.width = (int)a.width;
    p.norm = a.norm;
    p.post_norm = a.y_dev ? a.post_norm : CONVROT_NORM_NONE;
    p.a = a.residual_scale;
    p.eps = a.eps;
    p.inv_width = 1.f / (float)a.width;
    const bool f32v = a.vec_dtype == CONVROT_F32;
    if (a.dtype == CONVROT_BF16)
        f32v ? launch_types<__bf16, float>(a, p, s) : launch_types<__bf16, __bf16>(a, p, s);
    else if (a.dtype == CONVROT_F16)
        f32v ? launch_types<_Float16, float>(a, p, s) : launch_types<_Float16, _Float16>(a, p, s);
    else
        launch_types<float, float>(a, p, s);
}

}  // namespace convrot
