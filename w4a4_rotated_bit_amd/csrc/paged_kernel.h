// paged_kernel.h -- attention of one new token of each sequence over the pages
// of its keys and values.  Included by one source for each type of the heads.
//
// Up to 16 query heads of a key head are the columns of both matrix products,
// transposed so that nothing moves between lanes: S^T = K Q^T leaves a lane with
// the scores of one head and eight keys, and those, rounded, are the lane's own
// part of the second operand of O^T = V^T P^T.  A wave takes 32 keys a step.
// Keys come as the first operand straight from memory (a lane a row); values,
// which that operand wants by channel, are loaded by row, eight channels of
// eight keys a lane, and transposed within the lane's registers.  No value
// crosses shared memory before the waves' results are joined.
// The running maximum of a head only moves when a score exceeds it by 2^8
// (a factor that binary32 sums and 16-bit weights of the softmax bear), so most
// steps rescale nothing.
//
// Work is shared out in units of 128 keys, over all sequences and key heads in
// one line that the workgroups cut into equal parts: the lengths are known on
// the GPU alone.  A workgroup's part may end inside a sequence; such ends go to
// the workspace as partial results (maximum, sum, unscaled outputs) and a second
// launch joins them.
#pragma once
#include <hip/hip_runtime.h>

#include "attention_ops.h"

namespace convrot {
namespace {

template <typename T>
struct Mfma16;
template <>
struct Mfma16<__bf16> {
    typedef __bf16 Frag __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ F4 run(U4 a, U4 b, F4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(Frag, a), __builtin_bit_cast(Frag, b), c, 0, 0, 0);
    }
};
template <>
struct Mfma16<_Float16> {
    typedef _Float16 Frag __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ F4 run(U4 a, U4 b, F4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(Frag, a), __builtin_bit_cast(Frag, b), c, 0, 0, 0);
    }
};

struct PagedParams {
    convrot_attention_paged_args a;
    float* partial;
    int64_t slot;
    int columns, workgroups, groups, group, shift, capacity;   // groups: of 16 heads a key head; group: heads a key head
    float scale;   // times log2(e)
};

// Where a sequence lies among the units.
struct Place {
    int b, units;       // sequence and its units
    int64_t before;     // units (a column) of the sequences before it
};

__device__ __forceinline__ int length_of(const PagedParams& p, int b)
{
    return min(max(p.a.lengths_dev[b], 0), p.capacity);
}
__device__ __forceinline__ int units_of(int length) { return (length + kPagedUnit - 1) / kPagedUnit; }

__device__ __forceinline__ int64_t all_units(const PagedParams& p)
{
    const int lane = __lane_id();
    int64_t sum = 0;
    for (int b = 0; b < p.a.batch; b += 64) sum += wave_sum(b + lane < p.a.batch ? units_of(length_of(p, b + lane)) : 0);
    return sum;
}

// The sequence that holds unit `at` of the line in which each unit counts `columns` times.
__device__ __forceinline__ Place find_unit(const PagedParams& p, int64_t at)
{
    const int lane = __lane_id();
    int64_t before = 0;
    for (int b = 0;; b += 64) {
        const int n = b + lane < p.a.batch ? units_of(length_of(p, b + lane)) : 0;
        const int sum = wave_scan(n);
        const uint64_t past = __ballot((before + sum) * p.columns > at);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int units = __builtin_amdgcn_readlane(n, l);
            return Place{b + l, units, before + __builtin_amdgcn_readlane(sum, l) - units};
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
}

// Every workgroup that shares has a unit: what lies between the first and the
// last one of a sequence has all written their part.
__device__ __forceinline__ int sharing(const PagedParams& p, int64_t units) { return (int)min((int64_t)p.workgroups, units); }
__device__ __forceinline__ int64_t share_begin(int64_t units, int workgroups, int w) { return units * w / workgroups; }
__device__ __forceinline__ int share_of(int64_t units, int workgroups, int64_t u)
{
    return (int)(((u + 1) * workgroups - 1) / units);
}

// The raw bytes of 32 keys or values, as a lane holds them.
// DIM: padded width, 64, 128 or 256.
template <int KIND, int DIM>
struct Shape {
    static constexpr int STEPS = DIM / 32;                  // matrix products over the channels of 16 keys
    static constexpr int LANE = DIM / 4;                    // channels of a key that a quantized lane holds
    static constexpr bool QUANT = KIND >= CONVROT_CACHE_E4M3;
    static constexpr int K_BYTES = KIND == CONVROT_CACHE_E4M3 ? LANE : KIND == CONVROT_CACHE_E2M1 ? LANE / 2 : 2 * LANE;
    static constexpr int K_WORDS = K_BYTES / 4;
    static constexpr int K_SCALES = QUANT ? (LANE + kBlock - 1) / kBlock : 1;
    static constexpr int WIDE = DIM == 64 ? 4 : 8;          // channels of a value that a lane loads at once
    static constexpr int SETS = DIM / (16 * WIDE);          // such loads a row
    static constexpr int V_BYTES = KIND == CONVROT_CACHE_E4M3 ? WIDE : KIND == CONVROT_CACHE_E2M1 ? WIDE / 2 : 2 * WIDE;
    static constexpr int V_WORDS = (V_BYTES + 3) / 4;
};

template <int KIND, int DIM>
struct Tile {
    using S = Shape<KIND, DIM>;
    uint32_t k[2][S::K_WORDS];
    uint32_t v[8][S::SETS][S::V_WORDS];
    uint8_t ks[2][S::K_SCALES], vs[8][S::SETS];
};

struct Lookup {
    int k[2], v[2];   // pages of this lane's keys (two of 16) and of its two quads of values
};

template <typename T, int KIND, int DIM>
struct Walker {
    using S = Shape<KIND, DIM>;
    const PagedParams& p;
    const int* table;         // of the sequence
    int length, head, lane, col, quad;
    // offsets inside a row of this lane's bytes
    int dim;

    __device__ __forceinline__ Lookup lookup(int t) const
    {
        Lookup l;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l.k[h] = table[min(t * kPagedTile + 16 * h + col, length - 1) >> p.shift];
            l.v[h] = table[min(t * kPagedTile + 16 * h + 4 * quad, length - 1) >> p.shift];
        }
        return l;
    }
    __device__ __forceinline__ bool good(int page) const { return (uint32_t)page < (uint32_t)p.a.cache.pages; }

    __device__ __forceinline__ void load(Tile<KIND, DIM>& x, int t, const Lookup& l) const
    {
        const convrot_cache_rows &kr = p.a.cache.k, &vr = p.a.cache.v;
        const int mask = (1 << p.shift) - 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t page = good(l.k[h]) ? l.k[h] : 0;
            const int place = min(t * kPagedTile + 16 * h + col, length - 1) & mask;
            const char* row = (const char*)kr.rows_dev + page * kr.page_stride + head * kr.head_stride + place * kr.token_stride;
            if constexpr (!S::QUANT) {
#pragma unroll
                for (int i = 0; i < S::STEPS; ++i) {
                    const int c = i * 32 + quad * 8;
                    const U4 r = *(const U4*)(row + (c < dim ? 2 * c : 0));   // beyond the head: its first channels, times 0
#pragma unroll
                    for (int j = 0; j < 4; ++j) x.k[h][4 * i + j] = r[j];
                }
            } else {
                const uint8_t* scales = kr.scales_dev + page * kr.scale_page_stride + head * kr.scale_head_stride + place * kr.scale_token_stride;
                // whole blocks: a lane's bytes lie inside the head or beyond it, 16 (8) bytes at a time
                constexpr int PART = S::K_BYTES < 16 ? S::K_BYTES : 16;
                constexpr int VALUES = KIND == CONVROT_CACHE_E4M3 ? PART : 2 * PART;
#pragma unroll
                for (int i = 0; i < S::K_BYTES / PART; ++i) {
                    const int c = quad * S::LANE + i * VALUES;
                    const char* at = row + (c < dim ? (KIND == CONVROT_CACHE_E4M3 ? c : c / 2) : 0);
                    if constexpr (PART == 16) {
                        const U4 r = *(const U4*)at;
#pragma unroll
                        for (int j = 0; j < 4; ++j) x.k[h][4 * i + j] = r[j];
                    } else {
                        const U2 r = *(const U2*)at;
                        x.k[h][0] = r[0];
                        x.k[h][1] = r[1];
                    }
                }
#pragma unroll
                for (int i = 0; i < S::K_SCALES; ++i) {
                    const int c = quad * S::LANE + i * kBlock;
                    x.ks[h][i] = scales[c < dim ? c / kBlock : 0];
                }
            }
            const int64_t vpage = good(l.v[h]) ? l.v[h] : 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int vplace = min(t * kPagedTile + 16 * h + 4 * quad + j, length - 1) & mask;
                const char* vrow = (const char*)vr.rows_dev + vpage * vr.page_stride + head * vr.head_stride + vplace * vr.token_stride;
#pragma unroll
                for (int set = 0; set < S::SETS; ++set) {
                    const int c0 = (set * 16 + col) * S::WIDE;
                    const int c = c0 < dim ? c0 : 0;   // beyond the head: outputs that nobody reads
                    uint32_t(&d)[S::V_WORDS] = x.v[4 * h + j][set];
                    if constexpr (S::V_BYTES == 16) {
                        const U4 r = *(const U4*)(vrow + 2 * c);
                        d[0] = r[0], d[1] = r[1], d[2] = r[2], d[3] = r[3];
                    } else if constexpr (S::V_BYTES == 8) {
                        const U2 r = *(const U2*)(vrow + c * S::V_BYTES / S::WIDE);
                        d[0] = r[0], d[1] = r[1];
                    } else if constexpr (S::V_BYTES == 4) {
                        d[0] = *(const uint32_t*)(vrow + c * S::V_BYTES / S::WIDE);
                    } else {
                        d[0] = *(const uint16_t*)(vrow + c / 2);
                    }
                    if constexpr (S::QUANT)
                        x.vs[4 * h + j][set] = vr.scales_dev[vpage * vr.scale_page_stride + head * vr.scale_head_stride +
                                                             vplace * vr.scale_token_stride + c / kBlock];
                }
            }
        }
    }

    // eight channels of a key as the operand of step i
    __device__ __forceinline__ U4 key(const Tile<KIND, DIM>& x, int h, int i) const
    {
        if constexpr (!S::QUANT) {
            return U4{x.k[h][4 * i], x.k[h][4 * i + 1], x.k[h][4 * i + 2], x.k[h][4 * i + 3]};
        } else {
            const float s = block_scale(x.ks[h][i * 8 / kBlock]);
            if constexpr (KIND == CONVROT_CACHE_E4M3) return Unpack<T>::e4m3(x.k[h][2 * i], x.k[h][2 * i + 1], s);
            else return Unpack<T>::e2m1(x.k[h][i], s);
        }
    }
    // the channels of step i that this lane's queries have to match
    __device__ __forceinline__ int channel(int i) const { return S::QUANT ? quad * S::LANE + i * 8 : i * 32 + quad * 8; }

    // one value's channels as registers of two
    __device__ __forceinline__ U4 value(const Tile<KIND, DIM>& x, int j, int set) const
    {
        const uint32_t(&d)[S::V_WORDS] = x.v[j][set];
        if constexpr (!S::QUANT) {
            if constexpr (S::WIDE == 8) return U4{d[0], d[1], d[2], d[3]};
            else return U4{d[0], d[1], 0, 0};
        } else {
            const float s = block_scale(x.vs[j][set]);
            if constexpr (KIND == CONVROT_CACHE_E4M3) return Unpack<T>::e4m3(d[0], S::WIDE == 8 ? d[S::V_WORDS - 1] : 0u, s);
            else return Unpack<T>::e2m1(d[0], s);
        }
    }
};

template <typename T, int KIND, int DIM>
__global__ __launch_bounds__(64 * kPagedWaves, 2) void paged_kernel(PagedParams p)
{
    using S = Shape<KIND, DIM>;
    constexpr int NW = kPagedWaves, PITCH = DIM + 4, TILES = S::SETS * S::WIDE;
    __shared__ float stats[NW][kPagedHeads][2];
    __shared__ __attribute__((aligned(16))) float outs[NW][kPagedHeads][PITCH];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int col = lane % 16, quad = lane / 16;
    const int dim = p.a.cache.head_dim;

    int64_t u = 0, last = 0;
    Place at{};
    int column, first;
    if (p.workgroups) {
        const int64_t units = all_units(p) * p.columns;
        const int shares = sharing(p, units);
        if ((int)blockIdx.x >= shares) return;
        u = share_begin(units, shares, blockIdx.x);
        last = share_begin(units, shares, blockIdx.x + 1);
        at = find_unit(p, u);
        const int64_t rest = u - at.before * p.columns;
        column = (int)(rest / at.units);
        first = (int)(rest % at.units);
    } else {
        at.b = blockIdx.x / p.columns;
        column = blockIdx.x % p.columns;
        at.units = units_of(length_of(p, at.b));
        first = 0;
        last = at.units;
    }
    const int64_t start = u;

    for (;;) {
        const int take = (int)min((int64_t)(at.units - first), last - u);
        const int length = length_of(p, at.b);
        const int head = column / p.groups, part = column % p.groups;
        const int heads = min(p.group - part * kPagedHeads, kPagedHeads);       // columns in use
        const int q_head = head * p.group + part * kPagedHeads;                 // the first of them
        const Walker<T, KIND, DIM> walk{p, p.a.page_table_dev + at.b * p.a.table_stride, length, head, lane, col, quad, dim};

        U4 q[S::STEPS];
        {
            const T* row = (const T*)p.a.q_dev + at.b * p.a.q_batch_stride + (q_head + min(col, heads - 1)) * p.a.q_head_stride;
#pragma unroll
            for (int i = 0; i < S::STEPS; ++i) {
                const int c = walk.channel(i);
                q[i] = col < heads && c < dim ? __builtin_bit_cast(U4, load_chunk<uint16_t, 8>((const uint16_t*)row + c)) : U4{0, 0, 0, 0};
            }
        }
        float m = -kInf, sum = 0.f;
        F4 o[TILES];
#pragma unroll
        for (int i = 0; i < TILES; ++i) o[i] = F4{0, 0, 0, 0};

        const auto step = [&](const Tile<KIND, DIM>& x, int t, const Lookup& l) {
            float s[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                F4 acc{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < S::STEPS; ++i) acc = Mfma16<T>::run(walk.key(x, h, i), q[i], acc);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[4 * h + j] = acc[j] * p.scale;
            }
            // keys behind the last one, or on a page that is none: not seen, and their values not multiplied
            bool seen[8];
            bool all = true;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                seen[j] = t * kPagedTile + (j & 4) * 4 + quad * 4 + (j & 3) < length && walk.good(l.v[j / 4]);
                all &= seen[j];
            }
            const bool partial = __ballot(!all) != 0;
            if (partial) {
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = seen[j] ? s[j] : -kInf;
            }
            float most = s[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) most = fmaxf(most, s[j]);
            if (__ballot(most > m + 8.f)) {
                const float next = fmaxf(m, max4(most));
                const float f = next == -kInf ? 0.f : exp2_fast(m - next);
                sum *= f;
#pragma unroll
                for (int i = 0; i < TILES; ++i) o[i] *= f;
                m = next;
            }
            const float base = m == -kInf ? 0.f : m;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[j] = exp2_fast(s[j] - base);
                sum += s[j];
            }
            // weights rounded to T: at most half a step of each, as the outputs are
            const U4 w{pack2<T>(s[0], s[1]), pack2<T>(s[2], s[3]), pack2<T>(s[4], s[5]), pack2<T>(s[6], s[7])};
#pragma unroll
            for (int set = 0; set < S::SETS; ++set) {
                U4 v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[j] = walk.value(x, j, set);
                    if (partial && !seen[j]) v[j] = U4{0, 0, 0, 0};
                }
#pragma unroll
                for (int c = 0; c < S::WIDE; ++c) {
                    const uint32_t sel = c % 2 ? 0x07060302u : 0x05040100u;
                    U4 a;
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[j] = __builtin_amdgcn_perm(v[2 * j + 1][c / 2], v[2 * j][c / 2], sel);
                    o[set * S::WIDE + c] = Mfma16<T>::run(a, w, o[set * S::WIDE + c]);
                }
            }
        };

        // A step's rows are asked for one step ahead, the pages they lie on two.
        int t = first * NW + wave;
        const int end = min((first + take) * NW, (length + kPagedTile - 1) / kPagedTile);
        if (t < end) {
            Tile<KIND, DIM> x, y;
            Lookup lx = walk.lookup(t), ly = walk.lookup(t + NW);
            walk.load(x, t, lx);
            for (;;) {
                Lookup next = walk.lookup(t + 2 * NW);
                if (t + NW < end) walk.load(y, t + NW, ly);
                step(x, t, lx);
                t += NW;
                if (t >= end) break;
                lx = next;
                next = walk.lookup(t + 2 * NW);
                if (t + NW < end) walk.load(x, t + NW, lx);
                step(y, t, ly);
                t += NW;
                if (t >= end) break;
                ly = next;
            }
        }

        // join the waves
        sum = sum4(sum);
        if (quad == 0) {
            stats[wave][col][0] = m;
            stats[wave][col][1] = sum;
        }
#pragma unroll
        for (int set = 0; set < S::SETS; ++set)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int c = 0; c < S::WIDE; c += 4) {
                    const int i = set * S::WIDE + c;
                    *(F4*)&outs[wave][col][(set * 16 + quad * 4 + j) * S::WIDE + c] = F4{o[i][j], o[i + 1][j], o[i + 2][j], o[i + 3][j]};
                }
        __syncthreads();
        const bool whole = take == at.units;
        float* slot = p.partial + (2 * (int64_t)blockIdx.x + (u == start ? 0 : 1)) * p.slot;
        for (int i = threadIdx.x; i < heads * (dim / 4); i += 64 * NW) {
            const int h = i / (dim / 4), c = i % (dim / 4) * 4;
            float most = stats[0][h][0];
#pragma unroll
            for (int w = 1; w < NW; ++w) most = fmaxf(most, stats[w][h][0]);
            F4 out{0, 0, 0, 0};
            float total = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = stats[w][h][0] == -kInf ? 0.f : exp2_fast(stats[w][h][0] - most);
                total += stats[w][h][1] * f;
                out += *(const F4*)&outs[w][h][c] * f;
            }
            if (whole) {
                // a sum of 0 has no key; NaN stays
                const float r = total == 0.f ? 0.f : 1.f / total;
                U2 packed{pack2<T>(out[0] * r, out[1] * r), pack2<T>(out[2] * r, out[3] * r)};
                typedef uint16_t H4 __attribute__((ext_vector_type(4)));
                store_chunk<uint16_t, 4>((uint16_t*)p.a.o_dev + at.b * p.a.o_batch_stride + (q_head + h) * p.a.o_head_stride + c,
                                         __builtin_bit_cast(H4, packed));
                if (c == 0 && p.a.lse_dev)
                    p.a.lse_dev[(int64_t)at.b * p.a.q_heads + q_head + h] = total == 0.f ? -kInf : (most + __log2f(total)) * kLn2;
            } else {
                *(F4*)(slot + 2 * kPagedHeads + h * DIM + c) = out;
                if (c == 0) {
                    slot[2 * h] = most;
                    slot[2 * h + 1] = total;
                }
            }
        }
        u += take;
        if (u >= last) return;
        __syncthreads();   // the next part writes the shared arrays again
        first = 0;
        if (++column == p.columns) {
            column = 0;
            do at.units = units_of(length_of(p, ++at.b));
            while (at.units == 0);
        }
    }
}

// The partial results of each sequence and column, joined; sequences without a
// key get zeros.
template <typename T>
__global__ __launch_bounds__(256) void paged_join_kernel(PagedParams p, int pitch)
{
    __shared__ float factors[kPagedHeads][kPagedShares + 1], scales[kPagedHeads];
    __shared__ F4 sums[256];
    const int b = blockIdx.x / p.columns, column = blockIdx.x % p.columns;
    const int head = column / p.groups, part = column % p.groups;
    const int heads = min(p.group - part * kPagedHeads, kPagedHeads), q_head = head * p.group + part * kPagedHeads;
    const int dim = p.a.cache.head_dim, lane = __lane_id(), wave = threadIdx.x / 64;
    const int mine = units_of(length_of(p, b));
    int w0 = 0, count = 0, shares = 0;
    int64_t units = 0, u0 = 0;
    if (mine > 0) {
        int64_t before = 0;
        for (int c = 0; c < p.a.batch; c += 64) {
            const int n = c + lane < p.a.batch ? units_of(length_of(p, c + lane)) : 0;
            units += wave_sum(n);
            before += wave_sum(c + lane < b ? n : 0);
        }
        units *= p.columns;
        shares = sharing(p, units);
        u0 = before * p.columns + (int64_t)column * mine;
        w0 = share_of(units, shares, u0);
        count = share_of(units, shares, u0 + mine - 1) - w0 + 1;
        if (count == 1) return;   // one workgroup had all of it, and wrote the outputs
    }
    // the first part is its workgroup's first one if that workgroup begins here
    const bool begins = count > 0 && share_begin(units, shares, w0) == u0;
    const auto slot = [&](int i) { return p.partial + (2 * (int64_t)(w0 + i) + (i == 0 && !begins ? 1 : 0)) * p.slot; };
    // a wave a head: what each part counts for
    for (int h = wave; h < heads; h += 4) {
        float most = -kInf, total = 0.f;
        for (int i = lane; i < count; i += 64) most = fmaxf(most, slot(i)[2 * h]);
#pragma unroll
        for (int d = 1; d < 64; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
        for (int i = lane; i < count; i += 64) {
            const float m = slot(i)[2 * h], f = m == -kInf ? 0.f : exp2_fast(m - most);
            factors[h][i] = f;
            total += slot(i)[2 * h + 1] * f;
        }
        total = lane_sum<64>(total);
        if (lane == 0) {
            scales[h] = total == 0.f ? 0.f : 1.f / total;
            if (p.a.lse_dev) p.a.lse_dev[(int64_t)b * p.a.q_heads + q_head + h] = total == 0.f ? -kInf : (most + __log2f(total)) * kLn2;
        }
    }
    __syncthreads();
    // four channels a thread; threads left over share the parts
    const int items = heads * (dim / 4), groups = max(256 / items, 1);
    for (int i0 = 0; i0 < items; i0 += 256) {
        const int item = i0 + (int)threadIdx.x % min(items, 256), g = groups > 1 ? threadIdx.x / items : 0;
        const int h = item / (dim / 4), c = item % (dim / 4) * 4;
        const bool on = item < items && g < groups;
        F4 out{0, 0, 0, 0};
        if (on) {
            int i = g;
            for (; i + 3 * groups < count; i += 4 * groups) {     // loads of four parts in flight
                F4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = *(const F4*)(slot(i + k * groups) + 2 * kPagedHeads + h * pitch + c);
#pragma unroll
                for (int k = 0; k < 4; ++k) out += v[k] * factors[h][i + k * groups];
            }
            for (; i < count; i += groups) out += *(const F4*)(slot(i) + 2 * kPagedHeads + h * pitch + c) * factors[h][i];
        }
        if (groups > 1) {
            sums[threadIdx.x] = out;
            __syncthreads();
            if (on && g == 0)
                for (int k = 1; k < groups; ++k) out += sums[k * items + item];
        }
        if (on && g == 0) {
            const float r = scales[h];
            typedef uint16_t H4 __attribute__((ext_vector_type(4)));
            store_chunk<uint16_t, 4>((uint16_t*)p.a.o_dev + b * p.a.o_batch_stride + (q_head + h) * p.a.o_head_stride + c,
                                     __builtin_bit_cast(H4, U2{pack2<T>(out[0] * r, out[1] * r), pack2<T>(out[2] * r, out[3] * r)}));
        }
    }
}

template <typename T, int KIND>
void launch_paged_kind(const PagedParams& p, unsigned grid, hipStream_t s)
{
    switch (padded_dim(p.a.cache.head_dim)) {
    case 64: paged_kernel<T, KIND, 64><<<grid, 64 * kPagedWaves, 0, s>>>(p); break;
    case 128: paged_kernel<T, KIND, 128><<<grid, 64 * kPagedWaves, 0, s>>>(p); break;
    default: paged_kernel<T, KIND, 256><<<grid, 64 * kPagedWaves, 0, s>>>(p); break;
    }
}

}  // namespace

template <typename T>
void launch_paged_typed(const convrot_attention_paged_args& a, const PagedPlan& plan, float* partial, hipStream_t s)
{
    PagedParams p{};
    p.a = a;
    p.partial = partial;
    p.slot = plan.slot;
    p.columns = plan.columns;
    p.workgroups = plan.workgroups;
    p.group = a.q_heads / a.cache.heads;
    p.groups = (p.group + kPagedHeads - 1) / kPagedHeads;
    p.shift = __builtin_ctz(a.cache.page_size);
    p.capacity = (int)(a.table_width * a.cache.page_size);
    p.scale = a.scale * kLog2e;
    const unsigned pairs = (unsigned)(a.batch * plan.columns);
    const unsigned grid = plan.workgroups ? (unsigned)plan.workgroups : pairs;
    switch (a.cache.kind) {
    case CONVROT_CACHE_E4M3: launch_paged_kind<T, CONVROT_CACHE_E4M3>(p, grid, s); break;
    case CONVROT_CACHE_E2M1: launch_paged_kind<T, CONVROT_CACHE_E2M1>(p, grid, s); break;
    default: launch_paged_kind<T, CONVROT_BF16>(p, grid, s); break;
    }
    if (plan.workgroups) paged_join_kernel<T><<<pairs, 256, 0, s>>>(p, padded_dim(a.cache.head_dim));
}

}  // namespace convrot
