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
//
// Bound by the matrix cores and, just behind them, the vector unit (an fma, an
// exponential and a sum for each pair of a query and a key, and half a conversion): a
// step's products and the vector instructions of the step before are written
// side by side, and two workgroups share a compute unit.  16384 causal tokens of 32 + 8
// heads of 128: 1.87 to 1.93 ms, 1.14 to 1.18 PFLOP/s, where a bf16 matrix product of
// torch reaches 1.15 (8192) to 1.37 (16384) on such values.  Counted over launches one
// after the other, the matrix cores are busy for 70% of the cycles and the vector unit for
// 60%, at a clock that falls to 1.6 GHz.  Eight waves and 256
// queries a workgroup: 1.91 against 1.90 ms; 64 queries a wave, to read each operand
// once for two products, spills registers (4.0 ms).
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
    float* partial;      // outputs [splits][rows][head_dim], then reference and sum [splits][rows][2]
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

// Tile t of all sequences'.  Up to 64 sequences, the tiles with the highest numbers
// come first: under a causal mask they have the most keys, and what starts last
// should be short.  More sequences follow one another.
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
    if (p.a.batch <= 64) {
        const int n = tiles_of(p, lane);
        const auto from = [&](int level) { return wave_sum(max(n - level, 0)); };   // tiles numbered `level` or more
        if (t >= from(0)) return false;
        int low = 0, high = (int)((p.a.q_tokens + kPromptRows - 1) / kPromptRows), above = 0;     // from(low) > t >= from(high) = above
        while (high - low > 1) {
            const int mid = (low + high) / 2, count = from(mid);
            if (count > t) low = mid;
            else high = mid, above = count;
        }
        // the (t - above)-th of the sequences that have a tile `low`
        const bool has = n > low;
        const int before = __popcll(__ballot(has) & (((uint64_t)1 << lane) - 1));
        x.b = __builtin_ctzll(__ballot(has && before == (int)t - above));
        x.tile = low;
    } else {
        int64_t b = 0;
        int rank = (int)t;
        for (;; b += 64) {
            if (b >= p.a.batch) return false;
            const int n = tiles_of(p, b + lane), sum = wave_scan(n), all = __builtin_amdgcn_readlane(sum, 63);
            if (rank < all) {
                const int l = __builtin_ctzll(__ballot(sum > rank));
                x.b = (int)b + l;
                x.tile = __builtin_amdgcn_readlane(sum, l) - 1 - rank;
                break;
            }
            rank -= all;
        }
    }
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
// Every copy of this wave has landed, every access to shared memory is done; then all waves meet.
__device__ __forceinline__ void copies_done()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
// Of `bytes` bytes from base; what lies behind them reads as zeros.
__device__ __forceinline__ U4 descriptor(const char* base, uint32_t bytes)
{
    const uint64_t at = (uint64_t)base;
    U4 d;
    d[0] = __builtin_amdgcn_readfirstlane((uint32_t)at);
    d[1] = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32) & 0xffffu);
    d[2] = __builtin_amdgcn_readfirstlane(bytes);
    d[3] = 0x20000;
    return d;
}

// WIDTH: channels computed with, those of a head and zeros behind them.  DIRECT: keys and values are copied straight to shared
// memory; otherwise (rows that do not begin with a multiple of 16 bytes, or overlap) by
// way of registers.
template <typename T, int WIDTH, bool DIRECT>
__global__ __launch_bounds__(256, WIDTH > 128 ? 1 : 2) void prompt_kernel(PromptParams p)
{
    constexpr int DIM = WIDTH <= 64 ? 64 : WIDTH <= 128 ? 128 : 256;     // of a row in shared memory: the permutations need a power of two
    constexpr int KEYS = kPromptKeys, ROW = 2 * DIM, PIECES = DIM / 8;   // bytes and 16-byte pieces of a row
    constexpr int STAGE = KEYS * ROW, COPIES = KEYS * PIECES / 256, STEPS = WIDTH / 16, TILES = WIDTH / 32;
    __shared__ __attribute__((aligned(16))) char shared[2][2][STAGE];    // keys, values; stages
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
    if (first_row >= nq) return;     // starts written while they are read
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

    // The scale's sign goes to the queries (exactly), and a scale of 0 is multiplied into
    // them: scores grow with the products.
    const float scale = p.scale == 0.f ? 1.f : fabsf(p.scale);
    const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
    U4 q[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int c = i * 16 + half * 8;
        q[i] = c < dim ? __builtin_bit_cast(U4, load_chunk<uint16_t, 8>((const uint16_t*)q_row + c)) ^ flip : U4{0, 0, 0, 0};
        if (p.scale == 0.f) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                typedef T T2 __attribute__((ext_vector_type(2)));
                const uint32_t word = q[i][k];
                const T2 pair = __builtin_bit_cast(T2, word);
                q[i][k] = pack2<T>((float)pair[0] * 0.f, (float)pair[1] * 0.f);
            }
        }
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
    // The 64 rows of a step to a stage of shared memory, rows behind the last key as
    // zeros, in COPIES pieces a wave.
    struct Source {
        U4 rows;
        uint32_t to;
    };
    const auto source = [&](const char* rows_at, int64_t stride, int j, const char* to) {
        const int rows = min(max(nk - j * KEYS, 0), KEYS);
        return Source{descriptor(rows_at + 2 * (int64_t)(j * KEYS) * stride, (uint32_t)(2 * rows * (int)stride)),
                      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)to + wave * COPIES * 1024};
    };
    const auto by_registers = [&](const char* rows_at, int64_t stride, const uint32_t (&from)[COPIES], int j, char* to) {
        const int rows = nk - j * KEYS;
        const char* at = rows_at + 2 * (int64_t)(j * KEYS) * stride;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const bool in = ((wave * COPIES + i) * 64 + lane) / PIECES < rows;
            U4 a{0, 0, 0, 0};
            if (in && from[i] != kBeyond) a = __builtin_bit_cast(U4, load_chunk<uint16_t, 8>((const uint16_t*)(at + from[i])));
            *(U4*)(to + (wave * COPIES + i) * 1024 + 16 * lane) = a;
        }
    };
    const auto keys_from = [&](int j, int stage) { return source(k_base, p.a.k_token_stride, j, shared[0][stage]); };
    const auto values_from = [&](int j, int stage) { return source(v_base, p.a.v_token_stride, j, shared[1][stage]); };
    const auto issue_keys = [&](int j, int stage) {
        if constexpr (DIRECT) {
            const Source s = keys_from(j, stage);
#pragma unroll
            for (int i = 0; i < COPIES; ++i) copy16(s.rows, from_k[i], s.to + i * 1024);
        } else {
            by_registers(k_base, p.a.k_token_stride, from_k, j, shared[0][stage]);
        }
    };
    const auto issue_values = [&](int j, int stage) {
        if constexpr (DIRECT) {
            const Source s = values_from(j, stage);
#pragma unroll
            for (int i = 0; i < COPIES; ++i) copy16(s.rows, from_v[i], s.to + i * 1024);
        } else {
            by_registers(v_base, p.a.v_token_stride, from_v, j, shared[1][stage]);
        }
    };
    // Shared memory by address: the pieces' permutation is an exclusive or of bits that
    // the rest of an address leaves clear, so a step's address is one of the lane's own.
    typedef __attribute__((address_space(3))) const U4 Piece;
    typedef short S4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) S4 Quarter;
    const uint32_t key_at = col * ROW + ((half ^ permuted(col)) << 4);
    const int v_row = 4 * half + lane / 4 % 4;
    const uint32_t value_at = v_row * ROW + (((lane / 16 % 2 * 2 + lane % 4 / 2) ^ permuted_v(v_row)) << 4) + lane % 2 * 8;
    // channels 16 i + 8 half .. of key 32 kt + lane % 32
    const auto key = [&](uint32_t keys, int i, int kt) { return *(Piece*)((keys ^ (i * 32)) + kt * 32 * ROW); };
    // channel 32 c + lane % 32 of keys 16 n + 4 half .. and of the four 8 behind them
    const auto value = [&](uint32_t vals, int n, int c) {
        const uint32_t at = (vals ^ (c * 64)) + n * 16 * ROW;
        const U2 x = __builtin_bit_cast(U2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Quarter*)at));
        const U2 y = __builtin_bit_cast(U2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Quarter*)(at + 8 * ROW)));
        return U4{x[0], x[1], y[0], y[1]};
    };
    const auto keys_of = [&](int stage) { return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)shared[0][stage] + key_at; };
    const auto values_of = [&](int stage) { return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)shared[1][stage] + value_at; };

    float m = -kInf, sum = 0.f;
    F16v o[TILES];
    // Scores of step j: this lane's query against keys 32 kt + 8 (i / 4) + 4 half + i % 4.
    struct Scores {
        F16v s[2];
    };
    const auto product = [&](Scores& x, uint32_t keys) {
#pragma unroll
        for (int i = 0; i < 2 * STEPS; ++i) x.s[i % 2] = Mfma32<T>::run(key(keys, i / 2, i % 2), q[i / 2], x.s[i % 2]);
    };
    const auto hide = [&](Scores& x, int j) {
        const int mine = limit - j * KEYS - 4 * half;    // this lane's last key, from the step's first of its half
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (kt * 32 + 8 * (i / 4) + i % 4 > mine) x.s[kt][i] = -kInf;
    };
    // The reference of the weights moves when one of these scores leaves its room.
    const auto raise = [&](float top) {
        if (__ballot(leaves_room<T>(top, m))) {
            const float next = fmaxf(m, reference<T>(max32(top)));
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
    // the careful pass's weights: of the rounded score that the reference was taken from
    const auto weigh = [&](Scores& x, int e, float from) {
#pragma clang fp contract(off)
        const float s = x.s[e / 16][e % 16] * scale;
        x.s[e / 16][e % 16] = exp2_fast(s - from);
        sum += x.s[e / 16][e % 16];
    };
    // weights rounded to T, as the outputs are (Reference)
    const auto weights = [&](const Scores& x, int n) {
        const F16v& s = x.s[n / 2];
        const int e = n % 2 * 8;
        return U4{pack2<T>(s[e], s[e + 1]), pack2<T>(s[e + 2], s[e + 3]), pack2<T>(s[e + 4], s[e + 5]), pack2<T>(s[e + 6], s[e + 7])};
    };
    constexpr int kLast = 0, kOpen = 1, kMasked = 2;

    // Step j's weights and outputs, between them the scores of step j + 1 (next:
    // whether there is one, and whether its keys are masked) and the copies of the steps
    // behind it (beyond the last one: zeros).  The order is written out, a matrix product a
    // slot: behind it come the vector instructions that fill its time, the shared memory
    // read of the product four slots on, and now and then a copy: issued one after the
    // other they would hold the wave up.
    float top;
    const auto step = [&](int j, auto next, Scores& cur, Scores& out) {
        const int stage = (j - begin) & 1;
        // keys of step j + 1 and values of step j are there, and nobody reads the stages of the ones before
        copies_done();
        if constexpr (!DIRECT && next.value != kLast) {
            issue_keys(j + 2, stage);
            issue_values(j + 1, stage ^ 1);
        }
        const Source next_keys = keys_from(j + 2, stage), next_values = values_from(j + 1, stage ^ 1);
        raise(top);
        const float from = m == -kInf ? 0.f : m;
        const uint32_t keys = keys_of(stage ^ 1), vals = values_of(stage);
        constexpr int RING = 4, SCORES = 2 * STEPS, OUTS = 4 * TILES;
        // weights worked out by the end of slot i: those of the first outputs' keys among the
        // scores, the others just ahead of theirs
        constexpr int EARLY = 20;
        U4 ring[RING], w[4];
        float sums[2] = {0.f, 0.f};
        // An element's three instructions, slots apart so that none waits for the one before
        // it.  Its exponential belongs to slot 1 + e (SCORES - 2) / EARLY, or behind the first
        // EARLY ones to SCORES + (e - EARLY) (OUTS / 2) / (32 - EARLY); `upto` elements come
        // before a slot.
        const auto upto = [&](int slot) {
            const int early = ((slot - 1) * EARLY + SCORES - 3) / (SCORES - 2), late = ((slot - SCORES) * (32 - EARLY) + OUTS / 2 - 1) / (OUTS / 2);
            return (slot < 1 ? 0 : early < EARLY ? early : EARLY) + (slot <= SCORES ? 0 : late < 32 - EARLY ? late : 32 - EARLY);
        };
        const auto weigh_in = [&](int slot) {
#pragma unroll
            for (int e = upto(slot + 1); e < upto(slot + 2); ++e) cur.s[e / 16][e % 16] = __builtin_fmaf(cur.s[e / 16][e % 16], scale, -from);
#pragma unroll
            for (int e = upto(slot); e < upto(slot + 1); ++e) cur.s[e / 16][e % 16] = exp2_fast(cur.s[e / 16][e % 16]);
#pragma unroll
            for (int e = upto(slot - 1); e < upto(slot); ++e) sums[e % 2] += cur.s[e / 16][e % 16];
        };
        const auto read = [&](int i) {     // what slot i multiplies
            if (i < SCORES) return key(keys, i / 2, i % 2);
            return value(vals, (i - SCORES) / TILES, (i - SCORES) % TILES);
        };
        constexpr int FIRST = next.value == kLast ? SCORES : 0;
        if constexpr (next.value != kLast) out = Scores{};
#pragma unroll
        for (int i = 0; i < RING; ++i) ring[i] = read(FIRST + i);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (next.value == kLast) {
#pragma unroll
            for (int i = 0; i < SCORES; ++i) weigh_in(i);
            w[0] = weights(cur, 0);
            w[1] = weights(cur, 1);
        } else {
#pragma unroll
            for (int i = 0; i < SCORES; ++i) {
                out.s[i % 2] = Mfma32<T>::run(ring[i % RING], q[i / 2], out.s[i % 2]);
                ring[i % RING] = read(i + RING);
                if constexpr (DIRECT) {
#pragma unroll
                    for (int k = i * 2 * COPIES / SCORES; k < (i + 1) * 2 * COPIES / SCORES; ++k) {
                        if (k < COPIES) copy16(next_keys.rows, from_k[k % COPIES], next_keys.to + k % COPIES * 1024);
                        else copy16(next_values.rows, from_v[k % COPIES], next_values.to + k % COPIES * 1024);
                    }
                }
                weigh_in(i);
                if (i == SCORES - 2) w[0] = weights(cur, 0);
                if (i == SCORES - 1) w[1] = weights(cur, 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (next.value == kMasked) hide(out, j + 1);
        }
        float high[2] = {-kInf, -kInf};
#pragma unroll
        for (int i = 0; i < OUTS; ++i) {
            const int n = i / TILES, c = i % TILES;
            o[c] = Mfma32<T>::run(ring[i % RING], w[n], o[c]);
            if (i + RING < OUTS) ring[i % RING] = read(SCORES + i + RING);
            // the rest of the weights in the first half, the next scores' maximum in the second
            weigh_in(SCORES + i);
            if (i == OUTS / 2 - TILES / 2 - 1) w[2] = weights(cur, 2);
            if (i == OUTS / 2 - 1) w[3] = weights(cur, 3);
            if (next.value != kLast && i >= OUTS / 2) {
#pragma unroll
                for (int e = (i - OUTS / 2) * 32 / OUTS; e < (i + 1 - OUTS / 2) * 32 / OUTS; ++e) high[e % 2] = fmaxf(fmaxf(high[e % 2], out.s[0][e]), out.s[1][e]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        sum += sums[0] + sums[1];
        if constexpr (next.value != kLast) top = fmaxf(high[0], high[1]) * scale;
    };
#pragma unroll
    for (int i = 0; i < TILES; ++i) o[i] = F16v{};
    if (begin < end) {
        Scores cur{}, out;
        issue_keys(begin, 0);
        issue_values(begin, 0);
        issue_keys(begin + 1, 1);
        copies_done();
        product(cur, keys_of(0));
        if (begin >= open) hide(cur, begin);
        top = highest(cur);
        int j = begin;
        for (; j + 2 < min(end, open); j += 2) {
            step(j, std::integral_constant<int, kOpen>{}, cur, out);
            step(j + 1, std::integral_constant<int, kOpen>{}, out, cur);
        }
        for (; j + 1 < min(end, open); ++j) {
            step(j, std::integral_constant<int, kOpen>{}, cur, out);
            cur = out;
        }
        for (; j + 1 < end; ++j) {
            step(j, std::integral_constant<int, kMasked>{}, cur, out);
            cur = out;
        }
        step(j, std::integral_constant<int, kLast>{}, cur, out);
    }

    // The careful pass.  Weights of 0 times a masked value that is no number leave no number
    // behind; and the exponent's fma takes the exact score, where the reference is a rounded
    // one: beyond kCoarse that leaves more than half between them, and weights that overflow
    // or vanish.  In either case the rows are computed once more, step by step, from rounded
    // scores, with values that are no numbers left out of the products, and counted for the
    // queries that see them: 1 for an infinity, 128 for a negative one, 16384 for a NaN, each
    // at most 64 times.
    if (begin < end) {
        bool again = fabsf(m) >= kCoarse && m != -kInf;
        if (p.a.causal && open < end) {
            float check = 0.f;
#pragma unroll
            for (int c = 0; c < TILES; ++c)
#pragma unroll
                for (int e = 0; e < 16; ++e) check += o[c][e] * 0.f;
            again |= !(check == 0.f);
        }
        if (__syncthreads_or(again)) {
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
                Scores cur{};
                product(cur, keys_of(0));
                hide(cur, j);
                raise(highest(cur));
                const float from = m == -kInf ? 0.f : m;
#pragma unroll
                for (int e = 0; e < 32; ++e) weigh(cur, e, from);
                const int mine = limit - j * KEYS - 4 * half;
#pragma unroll
                for (int c = 0; c < TILES; ++c) {
                    F16v count{};
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        typedef uint16_t H8 __attribute__((ext_vector_type(8)));
                        H8 v = __builtin_bit_cast(H8, value(values_of(0), n, c)), bad, seen;
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
        p.a.lse_dev[(kb * p.a.q_tokens + out_row) * p.a.q_heads + head] = log_sum<T>(m, sum);
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
    // a lane a part: its reference, sum, and what it counts for
    const float* stats = p.partial + p.splits * p.rows * dim + 2 * (lane * p.rows + r);
    const float m = lane < p.splits ? stats[0] : -kInf, l = lane < p.splits ? stats[1] : 0.f;
    float most = m;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
    const float f = m == -kInf ? 0.f : exp2_fast(m - most);
    const float total = lane_sum<64>(l * f);
    const float s = total == 0.f ? 0.f : 1.f / total;
    // four channels a lane; lanes left over share the parts, in up to four groups
    const int per = dim / 4, groups = min(64 / per, 4), g = lane / per, c = lane % per * 4;
    F4 out{0, 0, 0, 0};
    const float* from = p.partial + r * dim + c;
    for (int i = 0; i < p.splits; i += 4 * groups) {     // loads of four parts in flight
        F4 v[4];
        float w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int part = i + k * groups + g;
            const bool on = g < groups && part < p.splits;
            w[k] = __shfl(f, min(part, 63));
            v[k] = on ? *(const F4*)(from + part * p.rows * dim) : F4{0, 0, 0, 0};
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) out += v[k] * w[k];
    }
    F4 sum = out;
    for (int k = 1; k < groups; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] += __shfl(out[j], lane + k * per);
    typedef uint16_t H4 __attribute__((ext_vector_type(4)));
    if (lane < per)
        store_chunk<uint16_t, 4>((uint16_t*)p.a.o_dev + b * p.a.o_batch_stride + at * p.a.o_token_stride + head * p.a.o_head_stride + c,
                                 __builtin_bit_cast(H4, U2{pack2<T>(sum[0] * s, sum[1] * s), pack2<T>(sum[2] * s, sum[3] * s)}));
    if (lane == 0 && p.a.lse_dev) p.a.lse_dev[r] = log_sum<T>(most, total);
}

template <typename T, int WIDTH>
void launch_prompt_width(const PromptParams& p, unsigned grid, hipStream_t s)
{
    p.direct ? prompt_kernel<T, WIDTH, true><<<grid, 256, 0, s>>>(p) : prompt_kernel<T, WIDTH, false><<<grid, 256, 0, s>>>(p);
}
template <typename T>
void launch_prompt_dim(const PromptParams& p, unsigned grid, hipStream_t s)
{
    const int width = (p.a.head_dim + 31) / 32;
    if (width <= 2) launch_prompt_width<T, 64>(p, grid, s);
    else if (width == 3) launch_prompt_width<T, 96>(p, grid, s);
    else if (width == 4) launch_prompt_width<T, 128>(p, grid, s);
    else if (width <= 6) launch_prompt_width<T, 192>(p, grid, s);
    else launch_prompt_width<T, 256>(p, grid, s);
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
    p.direct = prompt_direct(a);
    p.scale = a.scale * kLog2e;
    launch_prompt_dim<T>(p, (unsigned)(plan.tiles * a.q_heads * plan.splits), s);
    if (plan.splits > 1) prompt_join_kernel<T><<<(unsigned)((p.rows + 3) / 4), 256, 0, s>>>(p);
}

}  // namespace convrot
