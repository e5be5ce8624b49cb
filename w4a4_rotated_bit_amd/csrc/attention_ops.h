// attention_ops.h -- plans, launch interface and shared pieces of attention and
// of the paged cache that it reads.
#pragma once
#include <stdint.h>

#include <algorithm>

#include "../../include/convrot.h"
#include "block_ops.h"

namespace convrot {

constexpr int kMaxHeadWidth = 256;          // channels of a head
constexpr int kMaxPageSize = 65536;
constexpr int64_t kMaxBatch = 65535;
constexpr int64_t kMaxPlaces = (int64_t)1 << 30;   // of one sequence in a cache
constexpr int64_t kMaxTokenStride = ((int64_t)1 << 24) - 1;   // 64 rows stay within 32-bit byte offsets
constexpr int64_t kMaxCacheTokenStride = (int64_t)1 << 27;   // bytes: 16 rows stay within 32-bit offsets
constexpr int64_t kMaxThreads = 0xffffffff;   // of one launch
constexpr int kBlock = 32;                  // channels that share a scale
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

inline bool cache_quantized(int kind) { return kind == CONVROT_CACHE_E4M3 || kind == CONVROT_CACHE_E2M1; }
// bytes of a row of `dim` values
inline int64_t cache_row_bytes(int kind, int dim)
{
    return kind == CONVROT_CACHE_E4M3 ? dim : kind == CONVROT_CACHE_E2M1 ? dim / 2 : 2 * dim;
}
// channels that the kernels compute with
inline int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// ---- one token over the pages ----
constexpr int kPagedHeads = 16;    // query heads of a key head that one workgroup takes (columns of a matrix product)
constexpr int kPagedTile = 32;     // keys of a wave's step
constexpr int kPagedUnit = 128;    // keys that work is shared out by
constexpr int kPagedWaves = 4;     // of a workgroup that has a share
constexpr int kPagedWavesAlone = 8;     // of one that has a whole sequence
// Most keys of such a sequence, by the width of the page table: the lengths are known on
// the GPU alone.  250 bf16 keys of 8 heads of 128 take 7.6 us alone and 10.2 in shares that
// a second launch joins, as they do in a wider table (128 such sequences 32 and 37); 500
// keys 10.6 alone and 10.8 (64 and 57).
constexpr int64_t kPagedAlone = 384;
// With as many sequences and columns the chip is full without shares, and tables may be
// longer (and four waves a workgroup do, which work on longer parts): 256 sequences of 1 to
// 2000 e2m1 keys of 8 heads 106 us and 140 in shares, 128 of 1000 bf16 keys 92 and 99, 4096
// of 512 e2m1 keys of 2 heads 208 and 326; where one of 2000 keys stands among 255 of 100,
// 42 and 34.
constexpr int64_t kPagedMany = 1024;
constexpr int64_t kPagedAloneMany = 2048;
constexpr int kPagedShares = 512;  // most workgroups that share the units: two on each compute unit

struct PagedPlan {
    int columns;      // key heads times groups of query heads: each walks a sequence's keys by itself
    int workgroups;   // that share all units out evenly; 0: one workgroup a sequence and column
    int64_t slot;     // floats of one partial result
    int64_t bytes() const { return 2 * (int64_t)workgroups * slot * 4; }
};

inline PagedPlan paged_plan(const convrot_attention_paged_args& a)
{
    PagedPlan p{};
    const int group = a.q_heads / a.cache.heads;
    p.columns = a.cache.heads * ((group + kPagedHeads - 1) / kPagedHeads);
    p.slot = kPagedHeads * (padded_dim(a.cache.head_dim) + 2);
    const int64_t capacity = a.table_width * a.cache.page_size;
    if (capacity <= (a.batch * p.columns < kPagedMany ? kPagedAlone : kPagedAloneMany)) return p;
    const int64_t units = a.batch * p.columns * ((capacity + kPagedUnit - 1) / kPagedUnit);
    p.workgroups = (int)std::min<int64_t>(units, kPagedShares);
    return p;
}

// ---- whole prompts ----
constexpr int kPromptRows = 128;   // queries of a workgroup: four waves of 32
constexpr int kPromptKeys = 64;    // keys of a step
constexpr int kPromptSplits = 64;  // most workgroups that share a tile's keys: a lane each when they are joined

struct PromptPlan {
    int64_t tiles;    // most tiles of kPromptRows queries that the sequences can have
    int splits;       // workgroups that share the keys of a tile
    int64_t rows;     // rows of partial results: splits * batch entries * q_tokens * q_heads
    int64_t bytes(int head_dim) const { return splits > 1 ? rows * (head_dim + 2) * 4 : 0; }
};

// Whether rows of keys and values can be copied in pieces of 16 bytes, with the end of
// the last one as the only bound.
inline bool prompt_direct(const convrot_attention_args& a)
{
    const uint64_t bits = (uint64_t)a.k_dev | (uint64_t)a.v_dev |
                          2 * (uint64_t)(a.k_batch_stride | a.k_token_stride | a.k_head_stride | a.v_batch_stride |
                                         a.v_token_stride | a.v_head_stride);
    return bits % 16 == 0 && a.k_token_stride >= a.head_dim && a.v_token_stride >= a.head_dim;
}

inline PromptPlan prompt_plan(const convrot_attention_args& a)
{
    PromptPlan p{};
    const bool packed = a.q_starts_dev != nullptr;
    // packed: sum of ceil(len / 128) over the sequences, for any lengths
    p.tiles = packed ? (a.q_tokens + (kPromptRows - 1) * std::min(a.batch, a.q_tokens)) / kPromptRows
                     : a.batch * ((a.q_tokens + kPromptRows - 1) / kPromptRows);
    // Few queries against many keys: the keys of a tile go to several workgroups, as many as
    // fill the chip (two on each compute unit) and as it pays: a step of 64 keys takes 1.4 us,
    // or 2 us where two workgroups share a unit (measured with heads of 128, taken for all),
    // a second launch 6 us, and partial results are written and read at some 4 TB/s.  (233
    // queries of 9 heads of 72 against 13243 keys: 27 us in 19 parts, 240 us in one; 1024
    // causal queries of 32 heads of 128: 41 us in two parts, 24 us in one.)  A tile's steps
    // are counted without a mask, and of packed sequences, whose lengths are known on the GPU
    // alone, by their mean, 256 keys a part at least: where one is far longer than the others
    // it gets too few parts (one query each for 64 sequences of 4 heads, one with 100000 keys
    // and 63 with 100: 2 parts and 920 us; the long one alone 57).
    const int64_t groups = std::max<int64_t>(p.tiles * a.q_heads, 1);
    const double steps = (double)a.k_tokens / (packed ? std::max<int64_t>(a.batch, 1) : 1) / kPromptKeys;
    const double part = (double)(packed ? 1 : a.batch) * a.q_tokens * a.q_heads * a.head_dim * 8 / 4e6;
    double best = 1e300;
    p.splits = 1;
    for (int s = 1; s == 1 || (s <= kPromptSplits && groups * s <= 512 && 4 * s <= steps); ++s) {
        const double us = steps / s * (groups * s > 256 ? 2.0 : 1.4) + (s > 1 ? 6 + part * s : 0);
        if (us < best) {
            best = us;
            p.splits = s;
        }
    }
    p.rows = p.splits * (packed ? 1 : a.batch) * a.q_tokens * a.q_heads;
    return p;
}

}  // namespace convrot

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>

namespace convrot {

void launch_cache(const convrot_cache_args& a, bool write, hipStream_t s);
void launch_attention_paged(const convrot_attention_paged_args& a, const PagedPlan& plan, float* partial, hipStream_t s);
void launch_attention(const convrot_attention_args& a, const PromptPlan& plan, float* partial, hipStream_t s);
template <typename T>
void launch_paged_typed(const convrot_attention_paged_args& a, const PagedPlan& plan, float* partial, hipStream_t s);
template <typename T>
void launch_prompt_typed(const convrot_attention_args& a, const PromptPlan& plan, float* partial, hipStream_t s);

// ---- device helpers ---------------------------------------------------------

typedef float F4 __attribute__((ext_vector_type(4)));
typedef float F16v __attribute__((ext_vector_type(16)));
typedef uint32_t U4 __attribute__((ext_vector_type(4)));
typedef uint32_t U2 __attribute__((ext_vector_type(2)));

constexpr float kInf = __builtin_inff();

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Two values to a register of two T, rounded to nearest.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    typedef T T2 __attribute__((ext_vector_type(2)));
    typedef float F2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(F2{a, b}, T2));
}

// Weights of a softmax are 2^(s - m), s a score times log2(e) and m a reference that is
// kLift below the largest score when it is set, and is set again when a score exceeds it
// by more than kRoom.  They are rounded to T before they multiply values.  bf16 has
// binary32's exponents, so that is half a step of each, and seldom moving the reference
// is all that counts.  f16 rounds what lies below 2^-14 to multiples of 2^-24: with the
// largest weight between 2^11 and 2^15 (of 65504) that is half a step at most for weights
// of 2^-25 times the largest one or more, and 2^-36 times the largest for those below,
// so that 2^24 of them lose half a step of an f16 output.  Without a lift 32768 keys 17
// below another one of no value were 44% off.
template <typename T>
struct Reference;
template <>
struct Reference<__bf16> {
    static constexpr float kLift = 0.f, kRoom = 8.f;
};
template <>
struct Reference<_Float16> {
    static constexpr float kLift = 11.f, kRoom = 15.f;
};
// From here on binary32 holds every second whole number at most.  The lift would be
// rounded there to as much as leaves f16's range, and nothing needs it: weights that are
// neither 0 nor 1 are 2^-2 or less and few.
constexpr float kCoarse = 0x1p24f;
// The reference for a largest score.
template <typename T>
__device__ __forceinline__ float reference(float most)
{
    if constexpr (Reference<T>::kLift == 0.f) return most;
    return fabsf(most) < kCoarse ? most - Reference<T>::kLift : most;
}
// Whether a score leaves the room of its reference.  The difference of neighbouring numbers
// is exact, where a sum of the reference and its room is rounded by up to half a step: to
// bf16, which bears more than 2^8 too, that is all the same.
template <typename T>
__device__ __forceinline__ bool leaves_room(float most, float m)
{
    if constexpr (Reference<T>::kLift == 0.f) return most > m + Reference<T>::kRoom;
    return most - m > Reference<T>::kRoom;
}
// The natural logarithm of a sum of weights.
template <typename T>
__device__ __forceinline__ float log_sum(float m, float sum)
{
    constexpr float kUnit = Reference<T>::kLift == 0.f ? 1.f : 1.f / 2048;    // 2^-kLift
    static_assert(Reference<T>::kLift == 0.f || Reference<T>::kLift == 11.f, "");
    return sum == 0.f ? -kInf : (m + Reference<T>::kLift + __log2f(sum * kUnit)) * kLn2;
}

// The scale 2^(s - 127) of a block as the conversions take it: they read the
// exponent field alone, 0 as 2^-127 and 255 as NaN.
__device__ __forceinline__ float block_scale(uint32_t s) { return __builtin_bit_cast(float, s << 23); }

// Eight consecutive values of a quantized row to four registers of two T: exact
// in bf16 (four significant bits at most), rounded to nearest in f16 where small.
template <typename T>
struct Unpack;
template <>
struct Unpack<__bf16> {
    static __device__ __forceinline__ U4 e2m1(uint32_t c, float s)
    {
        return U4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3))};
    }
    static __device__ __forceinline__ U4 e4m3(uint32_t lo, uint32_t hi, float s)
    {
        return U4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true))};
    }
};
template <>
struct Unpack<_Float16> {
    static __device__ __forceinline__ U4 e2m1(uint32_t c, float s)
    {
        return U4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 0)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 1)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 2)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 3))};
    }
    static __device__ __forceinline__ U4 e4m3(uint32_t lo, uint32_t hi, float s)
    {
        return U4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, s, false)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, s, true)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, s, false)),
                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, s, true))};
    }
};

// v of the lane whose number differs by 32 (HALF) or by 16, beside this lane's
// own: {v of lanes with that bit clear, v of lanes with it set}.
struct Pair {
    uint32_t low, high;
};
__device__ __forceinline__ Pair across32(uint32_t v)
{
    uint32_t copy = v;
    asm volatile("" : "+v"(copy));   // a register of its own: swapped with itself it stays as it is
    const auto r = __builtin_amdgcn_permlane32_swap(v, copy, false, false);
    return Pair{(uint32_t)r[0], (uint32_t)r[1]};
}
__device__ __forceinline__ Pair across16(uint32_t v)
{
    uint32_t copy = v;
    asm volatile("" : "+v"(copy));
    const auto r = __builtin_amdgcn_permlane16_swap(v, copy, false, false);
    return Pair{(uint32_t)r[0], (uint32_t)r[1]};
}
__device__ __forceinline__ float max32(float v)
{
    const Pair p = across32(__builtin_bit_cast(uint32_t, v));
    return fmaxf(__builtin_bit_cast(float, p.low), __builtin_bit_cast(float, p.high));
}
__device__ __forceinline__ float sum32(float v)
{
    const Pair p = across32(__builtin_bit_cast(uint32_t, v));
    return __builtin_bit_cast(float, p.low) + __builtin_bit_cast(float, p.high);
}
// over the four lanes that share lane % 16
__device__ __forceinline__ float max4(float v)
{
    const Pair p = across16(__builtin_bit_cast(uint32_t, v));
    return max32(fmaxf(__builtin_bit_cast(float, p.low), __builtin_bit_cast(float, p.high)));
}
__device__ __forceinline__ float sum4(float v)
{
    const Pair p = across16(__builtin_bit_cast(uint32_t, v));
    return sum32(__builtin_bit_cast(float, p.low) + __builtin_bit_cast(float, p.high));
}

template <int CTRL>
__device__ __forceinline__ int lane_perm(int v)
{
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true);
}
// sum over the wave, in all lanes
__device__ __forceinline__ int wave_sum(int v)
{
    v += lane_perm<0xB1>(v);     // neighbour, other pair of four, other four of eight, other eight of sixteen
    v += lane_perm<0x4E>(v);
    v += lane_perm<0x141>(v);
    v += lane_perm<0x140>(v);
    const Pair a = across16((uint32_t)v);
    const Pair b = across32(a.low + a.high);
    return (int)(b.low + b.high);
}
// inclusive sum over the lanes up to this one
__device__ __forceinline__ int wave_scan(int v)
{
    const int lane = __lane_id();
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int up = __shfl_up(v, d);
        if (lane >= d) v += up;
    }
    return v;
}

}  // namespace convrot
#endif
