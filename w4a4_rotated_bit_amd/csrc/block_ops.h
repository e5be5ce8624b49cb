// block_ops.h -- launch interface and shared pieces of the operators around a
// rotated linear: the residual update with its norms, the rotary positions and
// the product with group-scaled 4-bit weights.
#pragma once
#include <stdint.h>

#include "../../include/convrot.h"

namespace convrot {

constexpr int64_t kMaxNormWidth = 16384;   // one row is held in the registers of one workgroup
constexpr int kMaxHeadDim = 256;
constexpr int kMaxRopePairs = kMaxHeadDim / 2;
constexpr int kMaxRopeAxes = 8;
constexpr int kMaxRopeTensors = 2;
constexpr int64_t kMaxHeads = 65535;
constexpr int64_t kMaxGroupedK = 65536;
constexpr int kMaxGroupedM = 32;

inline int elem_bytes(int dtype) { return dtype == CONVROT_F32 ? 4 : 2; }

// Frequencies of a rotation, in turns for a position of one (radians / 2 pi),
// and the axis each pair follows.  Passed by value in the kernel arguments.
struct RopePlan {
    double turns[kMaxRopePairs];
    uint8_t axis[kMaxRopePairs];
};

}  // namespace convrot

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>

namespace convrot {

void launch_residual_norm(const convrot_residual_norm_args& a, hipStream_t s);
void launch_rope(const convrot_rope_args& a, const RopePlan& plan, hipStream_t s);
void launch_linear_grouped(const convrot_grouped_args& a, hipStream_t s);
void launch_quantize_grouped(const void* W, int64_t N, int64_t K, int group, int dtype, uint8_t* codes, void* scales,
                             uint8_t* zeros, hipStream_t s);

// ---- device helpers ---------------------------------------------------------

template <typename T, int N>
struct VecOf {
    typedef T type __attribute__((ext_vector_type(N)));
};
template <typename T>
struct VecOf<T, 1> {
    typedef T type;
};

// N consecutive elements at p, as one load (p aligned to the vector) widened to binary32.
template <typename T, int N>
__device__ __forceinline__ void load_f32(const T* p, float (&v)[N])
{
    if constexpr (N == 1) {
        v[0] = (float)*p;
    } else if constexpr (sizeof(T) * N > 16) {
        constexpr int H = N / 2;
        typedef typename VecOf<T, H>::type V;
        const V a = *(const V*)p, b = *(const V*)(p + H);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            v[i] = (float)a[i];
            v[H + i] = (float)b[i];
        }
    } else {
        typedef typename VecOf<T, N>::type V;
        const V a = *(const V*)p;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = (float)a[i];
    }
}

// The same values rounded to T (nearest even) and stored.
template <typename T, int N>
__device__ __forceinline__ void store_f32(T* p, const float (&v)[N])
{
    if constexpr (N == 1) {
        *p = (T)v[0];
    } else {
        typedef typename VecOf<T, N>::type V;
        V a;
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] = (T)v[i];
        *(V*)p = a;
    }
}

// Sum over the W lanes of an aligned group (W a power of two, at most 64).
template <int W>
__device__ __forceinline__ float lane_sum(float v)
{
#pragma unroll
    for (int d = 1; d < W; d *= 2) v += __shfl_xor(v, d, 64);
    return v;
}

}  // namespace convrot
#endif
