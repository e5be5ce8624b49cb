// prompt_kernel.h -- attention over whole prompts.  Included by one source for
// each type of the heads.
//
// A workgroup of four waves takes 128 queries of a head, 32 a wave, and walks
// the keys 64 at a time.  Both products are computed transposed: S^T = K Q^T
// leaves a lane with 32 scores of one query, so the softmax's maximum and sum
// need one exchange between the wave's halves, and rounded they are, where they
// lie, the second operand of O^T = V^T P^T: its inner index runs over the keys in
// the order in which the lane holds them.  The first operand's values are read
// from shared memory with the transposing load, four keys of a channel at a
// time, in that same order.
//
// Keys and values lie in shared memory as they do in memory, rows of channels,
// in two stages: the next 64 are copied straight there (no registers involved)
// while these are used.  The 16-byte pieces of a row are permuted by an exclusive
// or with the row's number, so that neither the rows' reads nor the transposing
// ones meet in a bank.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "attention_ops.h"

namespace convrot {
namespace {

template <typename T>
struct Mfma32;
template <>
struct Mfma32<__bf16> {
    typedef __bf16 Frag __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ F16v run(U4 a, U4 b, F16v c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(Frag, a), __builtin_bit_cast(Frag, b), c, 0, 0, 0);
    }
};
template <>
struct Mfma32<_Float16> {
    typedef _Float16 Frag __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ F16v run(U4 a, U4 b, F16v c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(Frag, a), __builtin_bit_cast(Frag, b), c, 0, 0, 0);
    }
};

struct PromptParams {
    convrot_attention_args a;
    float* partial;      // outputs [splits][rows][head_dim], then maximum and sum [splits][rows][2]
    int64_t tiles, rows;
    int splits, group, direct;   // heads a key head; whether rows can be copied 16 bytes at a time
    float scale;         // times log2(e)
};

// A sequence, and the tile of its queries that a workgroup takes.
struct Prompt {
    int b, tile;
    int64_t q0, k0;      // first query and key row
    int nq, nk;
};

__device__ __forceinline__ int starts_at(const int* starts, int64_t b, int64_t rows)
{
    return min(max(starts[b], 0), (int)rows);
}
__device__ __forceinline__ int tiles_of(const PromptParams& p, int64_t b)
{
    if (b >= p.a.batch) return 0;
    const int n = starts_at(p.a.q_starts_dev, b + 1, p.a.q_tokens) - starts_at(p.a.q_starts_dev, b, p.a.q_tokens);
    return (max(n, 0) + kPromptRows - 1) / kPromptRows;
}
// Tiles whose number within their sequence is `level` or more.
__device__ __forceinline__ int tiles_from(const PromptParams& p, int level)
{
    const int lane = __lane_id();
    int sum = 0;
    for (int64_t b = 0; b < p.a.batch; b += 64) sum += wave_sum(max(tiles_of(p, b + lane) - level, 0));
    return sum;
}

// Tile t of all sequences', those with the highest numbers first: under a
// causal mask they have the most keys, and what starts last should be short.
__device__ __forceinline__ bool find_prompt(const PromptParams& p, int64_t t, Prompt& x)
{
    if (!p.a.q_starts_dev) {
        const int per = (int)((p.a.q_tokens + kPromptRows - 1) / kPromptRows);
        x.b = (int)(t % p.a.batch);
        x.tile = per - 1 - (int)(t / p.a.batch);
        x.q0 = x.k0 = 0;
        x.nq = (int)p.a.q_tokens;
        x.nk = (int)p.a.k_tokens;
        return true;
    }
    const int lane = __lane_id();
    if (t >= tiles_from(p, 0)) return false;
    int low = 0, high = (int)((p.a.q_tokens + kPromptRows - 1) / kPromptRows);   // tiles_from(low) > t >= tiles_from(high)
    int above = 0;
    while (high - low > 1) {
        const int mid = (low + high) / 2, n = tiles_from(p, mid);
        if (n > t) low = mid;
        else high = mid, above = n;
    }
    // the (t - above)-th of the sequences that have tile `low`
    int rank = (int)(t - above);
    for (int64_t b = 0;; b += 64) {
        const bool has = tiles_of(p, b + lane) > low;
        const uint64_t mask = __ballot(has);
        const int n = __popcll(mask);
        if (rank < n) {
            const int before = __popcll(mask & (((uint64_t)1 << lane) - 1));
            const uint64_t here = __ballot(has && before == rank);
            x.b = (int)b + __builtin_ctzll(here);
            break;
        }
        rank -= n;
    }
    x.tile = low;
    x.q0 = starts_at(p.a.q_starts_dev, x.b, p.a.q_tokens);
    x.nq = max(starts_at(p.a.q_starts_dev, x.b + 1, p.a.q_tokens) - (int)x.q0, 0);
    x.k0 = starts_at(p.a.k_starts_dev, x.b, p.a.k_tokens);
    x.nk = max(starts_at(p.a.k_starts_dev, x.b + 1, p.a.k_tokens) - (int)x.k0, 0);
    return true;
}

// 16 bytes a lane from base + offset to shared memory at `to` + 16 lane; an
// offset of kBeyond gives zeros.  Nothing is returned, and the wait is
// the caller's (copies_done).
constexpr uint32_t kBeyond = 0x80000000u;
__device__ __forceinline__ void copy16(U4 rows, uint32_t offset, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(offset), "s"(rows), "s"(to)
                 : "memory", "m0");
}
// Every copy of this wave has landed, every read of shared memory returned; then all waves meet.
__device__ __forceinline__ void copies_done()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
__device__ __forceinline__ U4 descriptor(const char* base)
{
    const uint64_t at = (uint64_t)base;
    U4 d;
    d[0] = __builtin_amdgcn_readfirstlane((uint32_t)at);
    d[1] = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32) & 0xffffu);
    d[2] = kBeyond;
    d[3] = 0x20000;
    return d;
}

template <typename T, int DIM>
__global__ __launch_bounds__(256, DIM > 128 ? 1 : 2) void prompt_kernel(PromptParams p)
{
    constexpr int KEYS = kPromptKeys, ROW = 2 * DIM, PIECES = DIM / 8;   // bytes and 16-byte pieces of a row
    constexpr int STAGE = KEYS * ROW, COPIES = KEYS * PIECES / 256, STEPS = DIM / 16, TILES = DIM / 32;
    __shared__ __attribute__((aligned(16))) char shared[2][2][STAGE];    // stage; keys, values
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int col = lane % 32, half = lane / 32;
    const int dim = p.a.head_dim;

    // Workgroups go to the eight dies in turn: a die takes query heads that share
    // keys, where the heads divide evenly, and finds those keys in its cache.
    const int64_t id = blockIdx.x / p.splits;
    const int split = blockIdx.x % p.splits;
    int head;
    int64_t t;
    if (p.a.q_heads % 8 == 0 && p.splits == 1) {
        const int each = p.a.q_heads / 8;
        head = (int)(id % 8) * each + (int)(id / 8 % each);
        t = id / 8 / each;
    } else {
        head = (int)(id % p.a.q_heads);
        t = id / p.a.q_heads;
    }
    Prompt x;
    if (!find_prompt(p, t, x)) return;
    const int b = __builtin_amdgcn_readfirstlane(x.b), nq = __builtin_amdgcn_readfirstlane(x.nq), nk = __builtin_amdgcn_readfirstlane(x.nk);
    const int first_row = __builtin_amdgcn_readfirstlane(x.tile) * kPromptRows;
    const int row = first_row + wave * 32 + col;        // this lane's query
    const int64_t kb = p.a.q_starts_dev ? 0 : b;        // batch entries lie apart unless packed
    const T* q_row = (const T*)p.a.q_dev + kb * p.a.q_batch_stride + (x.q0 + min(row, nq - 1)) * p.a.q_token_stride + head * p.a.q_head_stride;
    const char* k_base = (const char*)p.a.k_dev + 2 * (kb * p.a.k_batch_stride + x.k0 * p.a.k_token_stride + head / p.group * p.a.k_head_stride);
    const char* v_base = (const char*)p.a.v_dev + 2 * (kb * p.a.v_batch_stride + x.k0 * p.a.v_token_stride + head / p.group * p.a.v_head_stride);

    // keys that the rows see: row i those up to i + nk - nq under a causal mask
    const int shift = nk - nq;
    const int last_row = min(first_row + kPromptRows, nq) - 1;
    const int most = p.a.causal ? min(max(last_row + shift + 1, 0), nk) : nk;            // that any row sees
    const int least = p.a.causal ? min(max(first_row + shift + 1, 0), nk) : nk;          // that every row sees
    const int steps = (most + KEYS - 1) / KEYS;
    const int begin = (int)((int64_t)steps * split / p.splits), end = (int)((int64_t)steps * (split + 1) / p.splits);
    const int open = least / KEYS;                      // steps without a mask
    const int limit = p.a.causal ? min(row + shift, nk - 1) : nk - 1;    // this lane's last key

    // The scale's sign goes to the queries (exactly), and a scale of 0 makes them
    // zeros: scores grow with the products.
    const float scale = p.scale == 0.f ? 1.f : fabsf(p.scale);
    const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
    U4 q[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int c = i * 16 + half * 8;
        q[i] = c < dim && p.scale != 0.f ? __builtin_bit_cast(U4, load_chunk<uint16_t, 8>((const uint16_t*)q_row + c)) ^ flip : U4{0, 0, 0, 0};
    }

    // copies: piece s of a stage holds piece (s % PIECES) ^ (row's permutation) of row s / PIECES
    const auto permuted = [](int r) { return DIM == 64 ? (r >> 1) & 7 : r & 15; };       // keys
    const auto permuted_v = [](int r) { return DIM == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2; };
    uint32_t from_k[COPIES], from_v[COPIES];
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int s = (wave * COPIES + i) * 64 + lane, r = s / PIECES, pc = s % PIECES;
        const int ck = pc ^ permuted(r), cv = pc ^ permuted_v(r);
        from_k[i] = 8 * ck < dim ? (uint32_t)(2 * r * (int)p.a.k_token_stride + 16 * ck) : kBeyond;
        from_v[i] = 8 * cv < dim ? (uint32_t)(2 * r * (int)p.a.v_token_stride + 16 * cv) : kBeyond;
    }
    // the 64 rows of step j to shared memory; rows behind the last key as zeros
    const auto issue = [&](const char* rows_at, int64_t stride, const uint32_t (&from)[COPIES], int j, char* to) {
        const int rows = nk - j * KEYS;
        const char* at = rows_at + 2 * (int64_t)(j * KEYS) * stride;
        if (p.direct) {
            const U4 d = descriptor(at);
            const uint32_t dest = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)to + wave * COPIES * 1024;
            if (rows >= KEYS) {
#pragma unroll
                for (int i = 0; i < COPIES; ++i) copy16(d, from[i], dest + i * 1024);
            } else {
#pragma unroll
                for (int i = 0; i < COPIES; ++i)
                    copy16(d, ((wave * COPIES + i) * 64 + lane) / PIECES < rows ? from[i] : kBeyond, dest + i * 1024);
            }
        } else {     // rows that do not begin with a multiple of 16 bytes
#pragma unroll
            for (int i = 0; i < COPIES; ++i) {
                const bool in = ((wave * COPIES + i) * 64 + lane) / PIECES < rows;
                U4 a{0, 0, 0, 0};
                if (in && from[i] != kBeyond) a = __builtin_bit_cast(U4, load_chunk<uint16_t, 8>((const uint16_t*)(at + from[i])));
                *(U4*)(to + (wave * COPIES + i) * 1024 + 16 * lane) = a;
            }
        }
    };
    const auto issue_keys = [&](int j, int stage) { issue(k_base, p.a.k_token_stride, from_k, j, shared[stage][0]); };
    const auto issue_values = [&](int j, int stage) { issue(v_base, p.a.v_token_stride, from_v, j, shared[stage][1]); };
    // four keys (16 n + 4 half ..) of channel 32 c + lane % 32, and the four 8 behind them
    const auto values = [&](const char* vs, int n, int c) {
        typedef short S4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) S4 Shared4;
        U4 v;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 16 * n + 8 * h + 4 * half + lane / 4 % 4;
            const int piece = (c * 4 + lane / 16 % 2 * 2 + lane % 4 / 2) ^ permuted_v(r);
            const U2 u = __builtin_bit_cast(U2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Shared4*)(vs + r * ROW + piece * 16 + lane % 2 * 8)));
            v[2 * h] = u[0];
            v[2 * h + 1] = u[1];
        }
        return v;
    };

    float m = -kInf, sum = 0.f;
    F16v o[TILES];
    // Scores of step j: this lane's query against keys 32 kt + 8 (i / 4) + 4 half + i % 4.
    struct Scores {
        F16v s[2];
    };
    const auto product = [&](Scores& x, const char* ks, int i, int kt) {
        const int r = kt * 32 + col;
        x.s[kt] = Mfma32<T>::run(*(const U4*)(ks + r * ROW + ((2 * i + half) ^ permuted(r)) * 16), q[i], x.s[kt]);
    };
    const auto hide = [&](Scores& x, int j) {
        const int mine = limit - j * KEYS - 4 * half;    // this lane's last key, from the step's first of its half
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (kt * 32 + 8 * (i / 4) + i % 4 > mine) x.s[kt][i] = -kInf;
    };
    // The running maximum moves when one of these scores exceeds it by 2^8.
    const auto raise = [&](float top) {
        if (__ballot(top > m + 8.f)) {
            const float next = fmaxf(m, max32(top));
            const float f = next == -kInf ? 0.f : exp2_fast(m - next);
            sum *= f;
#pragma unroll
            for (int i = 0; i < TILES; ++i) o[i] *= f;
            m = next;
        }
    };
    const auto highest = [&](const Scores& x) {
        float top = fmaxf(x.s[0][0], x.s[1][0]);
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(fmaxf(top, x.s[0][i]), x.s[1][i]);
        return top * scale;
    };
    const auto weigh = [&](Scores& x, int e, float from) {
        x.s[e / 16][e % 16] = exp2_fast(__builtin_fmaf(x.s[e / 16][e % 16], scale, -from));
        sum += x.s[e / 16][e % 16];
    };
    // weights rounded to T: at most half a step of each, as the outputs are
    const auto weights = [&](const Scores& x, int n) {
        const F16v& s = x.s[n / 2];
        const int e = n % 2 * 8;
        return U4{pack2<T>(s[e], s[e + 1]), pack2<T>(s[e + 2], s[e + 3]), pack2<T>(s[e + 4], s[e + 5]), pack2<T>(s[e + 6], s[e + 7])};
    };
    constexpr int kLast = 0, kOpen = 1, kMasked = 2;

    // Step j's weights and outputs, between them the scores of step j + 1 (next:
    // whether there is one, and whether its keys are masked).
    Scores cur;
    float top;
    const auto step = [&](int j, auto next) {
        const int stage = (j - begin) & 1;
        copies_done();       // keys of step j + 1, values of step j; nobody reads the other stages any more
        if (j + 2 < end) issue_keys(j + 2, stage);
        if (j + 1 < end) issue_values(j + 1, stage ^ 1);
        raise(top);
        const float from = m == -kInf ? 0.f : m;
        const char *ks = shared[stage ^ 1][0], *vs = shared[stage][1];
        Scores y{};
        constexpr int EACH = 32 / (2 * STEPS) ? 32 / (2 * STEPS) : 1;
#pragma unroll
        for (int i = 0; i < 2 * STEPS; ++i) {
            if constexpr (next.value != kLast) product(y, ks, i / 2, i % 2);
#pragma unroll
            for (int e = i * EACH; e < (i + 1) * EACH && e < 32; ++e) weigh(cur, e, from);
        }
        U4 w[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) w[n] = weights(cur, n);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int c = 0; c < TILES; ++c) o[c] = Mfma32<T>::run(values(vs, n, c), w[n], o[c]);
        if constexpr (next.value == kMasked) hide(y, j + 1);
        if constexpr (next.value != kLast) {
            cur = y;
            top = highest(cur);
        }
    };
    if (begin < end) {
#pragma unroll
        for (int i = 0; i < TILES; ++i) o[i] = F16v{};
        issue_keys(begin, 0);
        issue_values(begin, 0);
        if (begin + 1 < end) issue_keys(begin + 1, 1);
        copies_done();
        cur = Scores{};
#pragma unroll
        for (int i = 0; i < 2 * STEPS; ++i) product(cur, shared[0][0], i / 2, i % 2);
        if (begin >= open) hide(cur, begin);
        top = highest(cur);
        int j = begin;
        for (; j + 1 < min(end, open); ++j) step(j, std::integral_constant<int, kOpen>{});
        for (; j + 1 < end; ++j) step(j, std::integral_constant<int, kMasked>{});
        step(j, std::integral_constant<int, kLast>{});
    } else {
#pragma unroll
        for (int i = 0; i < TILES; ++i) o[i] = F16v{};
    }

    // Weights of 0 times a masked value that is no number leave no number behind:
    // then the rows are computed once more, step by step, with values that are no
    // numbers left out of the products, and counted for the queries that see them:
    // 1 for an infinity, 128 for a negative one, 16384 for a NaN, each at most 64 times.
    if (p.a.causal && open < end && begin < end) {
        float check = 0.f;
#pragma unroll
        for (int c = 0; c < TILES; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) check += o[c][e] * 0.f;
        if (__syncthreads_or(!(check == 0.f))) {
            constexpr uint16_t one = __builtin_bit_cast(uint16_t, (T)1.f), many = __builtin_bit_cast(uint16_t, (T)128.f),
                               most16 = __builtin_bit_cast(uint16_t, (T)16384.f), top16 = __builtin_bit_cast(uint16_t, (T)kInf);
            m = -kInf;
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < TILES; ++i) o[i] = F16v{};
            for (int j = begin; j < end; ++j) {
                issue_keys(j, 0);
                issue_values(j, 0);
                copies_done();
                cur = Scores{};
#pragma unroll
                for (int i = 0; i < 2 * STEPS; ++i) product(cur, shared[0][0], i / 2, i % 2);
                hide(cur, j);
                raise(highest(cur));
                const float from = m == -kInf ? 0.f : m;
#pragma unroll
                for (int e = 0; e < 32; ++e) weigh(cur, e, from);
                const int mine = limit - j * KEYS - 4 * half;
                const char* vs = shared[0][1];
#pragma unroll
                for (int c = 0; c < TILES; ++c) {
                    F16v count{};
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        typedef uint16_t H8 __attribute__((ext_vector_type(8)));
                        H8 v = __builtin_bit_cast(H8, values(vs, n, c)), bad, seen;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint16_t bits = v[e] & 0x7fff;
                            bad[e] = bits < top16 ? 0 : bits > top16 ? most16 : v[e] >> 15 ? many : one;
                            if (bits >= top16) v[e] = 0;
                            seen[e] = 16 * n + 8 * (e / 4) + e % 4 <= mine ? one : 0;
                        }
                        o[c] = Mfma32<T>::run(__builtin_bit_cast(U4, v), weights(cur, n), o[c]);
                        count = Mfma32<T>::run(__builtin_bit_cast(U4, bad), __builtin_bit_cast(U4, seen), count);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int k = (int)count[e];
                        if (k % 128) o[c][e] += kInf;
                        if (k / 128 % 128) o[c][e] -= kInf;
                        if (k / 16384) o[c][e] = __builtin_nanf("");
                    }
                }
                __syncthreads();     // the next step's rows come to the same place
            }
        }
    }

    sum = sum32(sum);
    if (row >= nq) return;
    const int64_t out_row = x.q0 + row;
    if (p.splits > 1) {
        const int64_t r = split * p.rows + ((kb * p.a.q_tokens + out_row) * p.a.q_heads + head);
        float* to = p.partial + r * dim;
#pragma unroll
        for (int c = 0; c < TILES; ++c)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const int ch = c * 32 + 2 * e + 4 * half;
                if (ch < dim) *(F4*)(to + ch) = F4{o[c][e], o[c][e + 1], o[c][e + 2], o[c][e + 3]};
            }
        if (half == 0) {
            float* stats = p.partial + p.splits * p.rows * dim + 2 * r;
            stats[0] = m;
            stats[1] = sum;
        }
        return;
    }
    const float r = sum == 0.f ? 0.f : 1.f / sum;   // no key: zeros; NaN stays
    uint16_t* out = (uint16_t*)p.a.o_dev + kb * p.a.o_batch_stride + out_row * p.a.o_token_stride + head * p.a.o_head_stride;
#pragma unroll
    for (int c = 0; c < TILES; ++c)
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
            // four channels here and four in the other half: a half gives one group away and gets eight in a row
            U2 a{pack2<T>(o[c][e] * r, o[c][e + 1] * r), pack2<T>(o[c][e + 2] * r, o[c][e + 3] * r)};
            U2 d{pack2<T>(o[c][e + 4] * r, o[c][e + 5] * r), pack2<T>(o[c][e + 6] * r, o[c][e + 7] * r)};
            U4 all;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const auto sw = __builtin_amdgcn_permlane32_swap(a[k], d[k], false, false);
                all[k] = sw[0];
                all[2 + k] = sw[1];
            }
            const int ch = c * 32 + 2 * e + 8 * half;
            typedef uint16_t H8 __attribute__((ext_vector_type(8)));
            if (ch < dim) store_chunk<uint16_t, 8>(out + ch, __builtin_bit_cast(H8, all));
        }
    if (half == 0 && p.a.lse_dev)
        p.a.lse_dev[(kb * p.a.q_tokens + out_row) * p.a.q_heads + head] = sum == 0.f ? -kInf : (m + __log2f(sum)) * kLn2;
}

// The partial results of each row and head, joined: a wave a row of a head.
template <typename T>
__global__ __launch_bounds__(256) void prompt_join_kernel(PromptParams p)
{
    const int64_t r = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    if (r >= p.rows) return;
    const int64_t row = r / p.a.q_heads;
    const int head = (int)(r % p.a.q_heads), lane = threadIdx.x % 64, dim = p.a.head_dim;
    int64_t b = 0, at = row;
    if (p.a.q_starts_dev) {   // rows of no sequence stay as they are
        if (row < starts_at(p.a.q_starts_dev, 0, p.a.q_tokens) || row >= starts_at(p.a.q_starts_dev, p.a.batch, p.a.q_tokens)) return;
    } else {
        b = row / p.a.q_tokens;
        at = row % p.a.q_tokens;
    }
    const float* stats = p.partial + p.splits * p.rows * dim + 2 * r;
    float most = -kInf, total = 0.f;
    for (int i = 0; i < p.splits; ++i) most = fmaxf(most, stats[2 * i * p.rows]);
    F4 out{0, 0, 0, 0};
    const int c = 4 * lane;
    for (int i = 0; i < p.splits; ++i) {
        const float m = stats[2 * i * p.rows], f = m == -kInf ? 0.f : exp2_fast(m - most);
        total += stats[2 * i * p.rows + 1] * f;
        if (c < dim) out += *(const F4*)(p.partial + (i * p.rows + r) * dim + c) * f;
    }
    const float s = total == 0.f ? 0.f : 1.f / total;
    typedef uint16_t H4 __attribute__((ext_vector_type(4)));
    if (c < dim)
        store_chunk<uint16_t, 4>((uint16_t*)p.a.o_dev + b * p.a.o_batch_stride + at * p.a.o_token_stride + head * p.a.o_head_stride + c,
                                 __builtin_bit_cast(H4, U2{pack2<T>(out[0] * s, out[1] * s), pack2<T>(out[2] * s, out[3] * s)}));
    if (lane == 0 && p.a.lse_dev) p.a.lse_dev[r] = total == 0.f ? -kInf : (most + __log2f(total)) * kLn2;
}

template <typename T>
void launch_prompt_dim(const PromptParams& p, unsigned grid, hipStream_t s)
{
    switch (padded_dim(p.a.head_dim)) {
    case 64: prompt_kernel<T, 64><<<grid, 256, 0, s>>>(p); break;
    case 128: prompt_kernel<T, 128><<<grid, 256, 0, s>>>(p); break;
    default: prompt_kernel<T, 256><<<grid, 256, 0, s>>>(p); break;
    }
}

}  // namespace

template <typename T>
void launch_prompt_typed(const convrot_attention_args& a, const PromptPlan& plan, float* partial, hipStream_t s)
{
    PromptParams p{};
    p.a = a;
    p.partial = partial;
    p.tiles = plan.tiles;
    p.splits = plan.splits;
    p.rows = plan.rows / plan.splits;
    p.group = a.q_heads / a.k_heads;
    const uint64_t bits = (uint64_t)a.k_dev | (uint64_t)a.v_dev | 2 * (uint64_t)(a.k_batch_stride | a.k_token_stride | a.k_head_stride |
                                                                                  a.v_batch_stride | a.v_token_stride | a.v_head_stride);
    p.direct = bits % 16 == 0;
    p.scale = a.scale * kLog2e;
    launch_prompt_dim<T>(p, (unsigned)(plan.tiles * a.q_heads * plan.splits), s);
    if (plan.splits > 1) prompt_join_kernel<T><<<(unsigned)((p.rows + 3) / 4), 256, 0, s>>>(p);
}

}  // namespace convrot
