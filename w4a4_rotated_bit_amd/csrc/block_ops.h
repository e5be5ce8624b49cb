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

constexpr int kUnits = 256;   // compute units of an MI355X

// ---- device helpers ---------------------------------------------------------

template <typename T, int N>
struct VecOf {
    typedef T type __attribute__((ext_vector_type(N)));
};

// V consecutive elements, in one access whatever their alignment.
template <typename T, int V>
__device__ __forceinline__ typename VecOf<T, V>::type load_chunk(const T* p)
{
    typedef typename VecOf<T, V>::type Any __attribute__((aligned(sizeof(T))));
    return *(const Any*)p;
}
template <typename T, int V>
__device__ __forceinline__ void store_chunk(T* p, typename VecOf<T, V>::type v)
{
    typedef typename VecOf<T, V>::type Any __attribute__((aligned(sizeof(T))));
    *(Any*)p = v;
}
// The same with the hint that the data is used once: lines that are read or
// written whole need not stay in the caches near the units.
template <typename T, int V>
__device__ __forceinline__ typename VecOf<T, V>::type load_once(const T* p)
{
    typedef typename VecOf<T, V>::type Any __attribute__((aligned(sizeof(T))));
    return __builtin_nontemporal_load((const Any*)p);
}
template <typename T, int V>
__device__ __forceinline__ void store_once(T* p, typename VecOf<T, V>::type v)
{
    typedef typename VecOf<T, V>::type Any __attribute__((aligned(sizeof(T))));
    __builtin_nontemporal_store((Any)v, (Any*)p);
}

// Where lanes of a wave pass values on through shared memory: what they wrote
// before it is what they read after it, and no write behind it comes before a
// read in front of it.  A wave's accesses to shared memory happen in their
// order, so this is no instruction, only the order that the compiler has to keep.
__device__ __forceinline__ void wave_exchange()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// v of another lane of the same 16, by a lane permutation of the vector unit
// (a shuffle through shared memory takes some ten times as long).
template <int CTRL>
__device__ __forceinline__ float lane_perm(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// Sum over the W lanes of an aligned group (W a power of two, at most 64), the
// same bits in all of them.
template <int W>
__device__ __forceinline__ float lane_sum(float v)
{
    if constexpr (W >= 2) v += lane_perm<0xB1>(v);    // neighbour
    if constexpr (W >= 4) v += lane_perm<0x4E>(v);    // other pair of four
    if constexpr (W >= 8) v += lane_perm<0x141>(v);   // other four of eight, mirrored
    if constexpr (W >= 16) v += lane_perm<0x140>(v);  // other eight of sixteen, mirrored
    // rows of 16 lanes, then halves of 32, swapped between v and a copy of it (in
    // a register of its own: swapped with itself a register stays as it is)
    if constexpr (W >= 32) {
        int i = __builtin_bit_cast(int, v), copy = i;
        asm volatile("" : "+v"(copy));
        const auto r = __builtin_amdgcn_permlane16_swap(i, copy, false, false);
        const uint32_t a = r[0], b = r[1];
        v = __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
    }
    if constexpr (W >= 64) {
        int i = __builtin_bit_cast(int, v), copy = i;
        asm volatile("" : "+v"(copy));
        const auto r = __builtin_amdgcn_permlane32_swap(i, copy, false, false);
        const uint32_t a = r[0], b = r[1];
        v = __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
    }
    return v;
}

}  // namespace convrot
#endif
