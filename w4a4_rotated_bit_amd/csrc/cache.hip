// cache.hip -- rows of keys and values into a paged cache and out of it.
//
// A block of 32 channels is four neighbouring lanes' (16 bytes each): they find its
// largest magnitude by two lane permutations, as a whole number, so that NaN and
// infinities count as the largest, and its exponent gives the scale without a
// logarithm.  The conversion instructions round to nearest, ties to even, and divide or
// multiply by the scale exactly; e2m1 saturates by itself, e4m3 is cut to its range
// before.  No result depends on another block, and no sum is formed.
//
// Bound by memory; few tokens by its latency, three loads one after the other: the slot, the
// key's row, and the value's behind the key's stores.  A workgroup takes consecutive tokens of one head: what a prompt's
// tokens leave in a page, and are read from, lies side by side there (64 bytes a row
// of 128 e2m1 values), while the tokens' rows are whole lines.  These are loaded and
// stored with the hint that they are used once (78 -> 63 us for both directions of
// the sizes below).  32768 tokens of 8 heads of 128, e2m1: 35 us to write (170 MB, 4.9
// TB/s), 26 to 28 us to read back (6 TB/s: the codes are still in the last cache); one token
// 2.7 us each, a launch.
#include <hip/hip_runtime.h>

#include "attention_ops.h"

namespace convrot {
namespace {

typedef short S2 __attribute__((ext_vector_type(2)));

struct CacheRows {
    char* rows;
    uint8_t* scales;
    int64_t page, head, token, scale_page, scale_head, scale_token;   // strides in bytes
};

struct CacheParams {
    CacheRows kept[2];        // keys, values
    uint16_t* dense[2];
    int64_t token[2], head[2];   // strides of dense, elements
    const void* slots;
    int64_t tokens, places;
    int shift, chunks, wide;     // log2 of the page size, chunks of 8 values a row, 64-bit slots
};

// Eight values to the codes of a block that four neighbouring lanes share; s:
// the block's scale byte.
template <typename T>
__device__ __forceinline__ uint32_t block_exponent(const float (&x)[8], int top)
{
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __builtin_bit_cast(uint32_t, x[i]) & 0x7fffffffu);
    // as whole numbers, NaN above infinity above every finite magnitude
    most = max(most, (uint32_t)__builtin_amdgcn_mov_dpp((int)most, 0xB1, 0xF, 0xF, true));
    most = max(most, (uint32_t)__builtin_amdgcn_mov_dpp((int)most, 0x4E, 0xF, 0xF, true));
    const int e = (int)(most >> 23);
    return e == 255 ? 255u : (uint32_t)max(e - top, 0);
}

__device__ __forceinline__ uint32_t to_e2m1(const float (&x)[8], float s)
{
    uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0], x[1], s, 0);   // saturates
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], s, 3);
}
__device__ __forceinline__ U2 to_e4m3(float (&x)[8], uint32_t byte)
{
    const float s = block_scale(byte);
    // 448 times the scale, which is 1.75 times a normal number also for the smallest
    // scale: the conversion makes NaN of what lies beyond
    const float most = 1.75f * block_scale(byte + 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __builtin_amdgcn_fmed3f(x[i], -most, most);
    S2 lo{0, 0}, hi{0, 0};
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, x[0], x[1], s, false);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, x[2], x[3], s, true);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, x[4], x[5], s, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, x[6], x[7], s, true);
    return U2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}

template <int KIND, typename T, bool WRITE>
__global__ __launch_bounds__(256) void cache_kernel(CacheParams p)
{
    const int per = 256 / p.chunks;   // tokens of a workgroup
    const int i = threadIdx.x / p.chunks, c = threadIdx.x % p.chunks;
    const int64_t token = (int64_t)blockIdx.x * per + i;
    if (i >= per || token >= p.tokens) return;   // whole rows, so that the lanes of a block stay together
    const int head = blockIdx.y;
    const int64_t slot = p.wide ? ((const int64_t*)p.slots)[token] : (int64_t)((const int*)p.slots)[token];
    const bool inside = slot >= 0 && slot < p.places;
    if (WRITE && !inside) return;
    const int64_t page = slot >> p.shift, place = slot & (((int64_t)1 << p.shift) - 1);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const CacheRows& r = p.kept[k];
        uint16_t* dense = p.dense[k] + token * p.token[k] + head * p.head[k] + c * 8;
        char* row = r.rows + page * r.page + head * r.head + place * r.token;
        uint8_t* scale = nullptr;
        if constexpr (KIND >= CONVROT_CACHE_E4M3)
            scale = r.scales + page * r.scale_page + head * r.scale_head + place * r.scale_token + c / 4;
        if constexpr (WRITE) {
            const auto v = load_once<uint16_t, 8>(dense);
            if constexpr (KIND < CONVROT_CACHE_E4M3) {
                *(U4*)(row + c * 16) = __builtin_bit_cast(U4, v);
            } else {
                typedef T T8 __attribute__((ext_vector_type(8)));
                const T8 t = __builtin_bit_cast(T8, v);
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = (float)t[j];
                const uint32_t s = block_exponent<T>(x, KIND == CONVROT_CACHE_E4M3 ? 8 : 2);
                if constexpr (KIND == CONVROT_CACHE_E4M3)
                    *(U2*)(row + c * 8) = to_e4m3(x, s);
                else
                    *(uint32_t*)(row + c * 4) = to_e2m1(x, block_scale(s));
                if (c % 4 == 0) *scale = (uint8_t)s;
            }
        } else {
            U4 v{0, 0, 0, 0};
            if (inside) {
                if constexpr (KIND < CONVROT_CACHE_E4M3) {
                    v = *(const U4*)(row + c * 16);
                } else {
                    const float s = block_scale(*scale);
                    if constexpr (KIND == CONVROT_CACHE_E4M3) {
                        const U2 codes = *(const U2*)(row + c * 8);
                        v = Unpack<T>::e4m3(codes[0], codes[1], s);
                    } else {
                        v = Unpack<T>::e2m1(*(const uint32_t*)(row + c * 4), s);
                    }
                }
            }
            typedef uint16_t H8 __attribute__((ext_vector_type(8)));
            store_once<uint16_t, 8>(dense, __builtin_bit_cast(H8, v));
        }
    }
}

template <bool WRITE>
void launch(const convrot_cache_args& a, hipStream_t s)
{
    CacheParams p{};
    const convrot_cache_rows* rows[2] = {&a.cache.k, &a.cache.v};
    for (int k = 0; k < 2; ++k)
        p.kept[k] = CacheRows{(char*)rows[k]->rows_dev,       rows[k]->scales_dev,       rows[k]->page_stride,
                              rows[k]->head_stride,           rows[k]->token_stride,     rows[k]->scale_page_stride,
                              rows[k]->scale_head_stride,     rows[k]->scale_token_stride};
    p.dense[0] = (uint16_t*)a.k_dev;
    p.dense[1] = (uint16_t*)a.v_dev;
    p.token[0] = a.k_token_stride;
    p.token[1] = a.v_token_stride;
    p.head[0] = a.k_head_stride;
    p.head[1] = a.v_head_stride;
    p.slots = a.slots_dev;
    p.tokens = a.tokens;
    p.places = a.cache.pages * a.cache.page_size;
    p.shift = __builtin_ctz(a.cache.page_size);
    p.chunks = a.cache.head_dim / 8;
    p.wide = a.slots_dtype == CONVROT_I64;
    const int per = 256 / p.chunks;
    const dim3 grid((unsigned)((a.tokens + per - 1) / per), (unsigned)a.cache.heads);
    const bool bf16 = a.dtype == CONVROT_BF16;
    if (a.cache.kind == CONVROT_CACHE_E4M3)
        bf16 ? cache_kernel<CONVROT_CACHE_E4M3, __bf16, WRITE><<<grid, 256, 0, s>>>(p)
             : cache_kernel<CONVROT_CACHE_E4M3, _Float16, WRITE><<<grid, 256, 0, s>>>(p);
    else if (a.cache.kind == CONVROT_CACHE_E2M1)
        bf16 ? cache_kernel<CONVROT_CACHE_E2M1, __bf16, WRITE><<<grid, 256, 0, s>>>(p)
             : cache_kernel<CONVROT_CACHE_E2M1, _Float16, WRITE><<<grid, 256, 0, s>>>(p);
    else
        cache_kernel<CONVROT_BF16, uint16_t, WRITE><<<grid, 256, 0, s>>>(p);
}

}  // namespace

void launch_cache(const convrot_cache_args& a, bool write, hipStream_t s)
{
    write ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace convrot
