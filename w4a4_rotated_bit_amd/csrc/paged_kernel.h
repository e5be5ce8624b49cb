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
// The reference of a head's weights only moves when a score exceeds it by so much that
// 16-bit weights ask for it (Reference), so most steps rescale nothing.
//
// Rows of 16 bits are bound by their bytes: one to three steps' rows are under way while
// one is computed.  Quantized rows have half or a quarter of the bytes and the same
// instructions.  A lane's place among a step's rows never changes, but pages, and rows
// within them, are addressed by 64-bit scalar arithmetic: a step of 32 e2m1 keys takes
// some 215 scalar instructions (102 scalars do not fit and are kept in lanes of vector
// registers) and 270 vector ones, which the SIMDs issue for 40% of the time, with two waves
// each.  Rows copied to shared memory instead, without registers, were slower (eight
// sequences of 28 to 32 thousand e2m1 keys 131 against 76 us): every copy's addresses are
// the wave's work again.
// Eight sequences of 16384 keys of 8 heads of 128, 32 query heads: bf16 95 us (5.7
// TB/s), e4m3 67 us (4.1), e2m1 47 us (3.0); eight of 28 to 32 thousand keys in e2m1 78
// us, the first kernel 66 of it alone (4.2 TB/s) and the join 5.
//
// Work is shared out in units of 128 keys, over all sequences and key heads in
// one line that the workgroups cut into equal parts: the lengths are known on
// the GPU alone.  A workgroup's part may end inside a sequence; such ends go to
// the workspace as partial results (reference, sum, unscaled outputs) and a second
// launch joins them (5 us).  No atomics: the same bits on every run.
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

__device__ __forceinline__ int length_of(const PagedParams& p, int64_t b)
{
    const int n = p.a.lengths_dev[min(b, p.a.batch - 1)];    // read by every lane, so that many are under way
    return b < p.a.batch ? min(max(n, 0), p.capacity) : 0;
}
__device__ __forceinline__ int units_of(int length) { return (length + kPagedUnit - 1) / kPagedUnit; }
// The lanes' sequences of four times 64 from b on: at most 2^23 units each.
struct Quad {
    int n[4];
    __device__ __forceinline__ Quad(const PagedParams& p, int64_t b)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) n[i] = units_of(length_of(p, b + 64 * i + __lane_id()));
    }
    __device__ __forceinline__ uint32_t sum() const { return (uint32_t)wave_sum(n[0] + n[1] + n[2] + n[3]); }
};

// The first 64 sequences' units are in the lanes of `mine`: most calls have no more,
// and read the lengths once.
__device__ __forceinline__ int64_t all_units(const PagedParams& p, int mine)
{
    int64_t sum = wave_sum(mine);
    for (int64_t b = 64; b < p.a.batch; b += 256) sum += Quad(p, b).sum();
    return sum;
}

// The sequence that holds unit `at` of the line in which each unit counts `columns` times
// (none, with no units, only where lengths are written while they are read).
__device__ __forceinline__ Place find_unit(const PagedParams& p, int mine, int64_t at)
{
    int64_t before = 0;
    Place found{};
    const auto search = [&](int n, int64_t b) {
        const int sum = wave_scan(n);
        const uint64_t past = __ballot((before + sum) * p.columns > at);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int units = __builtin_amdgcn_readlane(n, l);
            found = Place{(int)b + l, units, before + __builtin_amdgcn_readlane(sum, l) - units};
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
        return false;
    };
    if (search(mine, 0)) return found;
    for (int64_t b = 64; b < p.a.batch; b += 256) {
        const Quad q(p, b);
        const uint32_t sum = q.sum();
        if ((before + sum) * p.columns <= at) {
            before += sum;
            continue;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (search(q.n[i], b + 64 * i)) return found;
    }
    return found;
}

// Every workgroup that shares has a unit: what lies between the first and the
// last one of a sequence has all written their part.
__device__ __forceinline__ int sharing(const PagedParams& p, int64_t units) { return (int)min((int64_t)p.workgroups, units); }
__device__ __forceinline__ int64_t share_begin(int64_t units, int workgroups, int w) { return units * w / workgroups; }
__device__ __forceinline__ int share_of(int64_t units, int workgroups, int64_t u)
{
    return (int)(((u + 1) * workgroups - 1) / units);
}

// Rows of 16-bit values are read with the hint that they are used once (in whole
// lines: eight sequences of 16384 keys of 128 channels 104 -> 95 us); quantized ones,
// whose loads take parts of a line, without (of 256 channels 125 against 154 us).
template <bool ONCE, typename V>
__device__ __forceinline__ V read_row(const char* at)
{
    if constexpr (ONCE) return __builtin_nontemporal_load((const V*)at);
    else return *(const V*)at;
}

// The raw bytes of 32 keys and values, as a lane holds them.
// DIM: padded width, 64, 128 or 256.
template <int KIND, int DIM>
struct Shape {
    static constexpr int STEPS = DIM / 32;                  // matrix products over the channels of 16 keys
    static constexpr int LANE = DIM / 4;                    // channels of a key that a quantized lane holds
    static constexpr bool QUANT = KIND >= CONVROT_CACHE_E4M3;
    static constexpr int BITS = KIND == CONVROT_CACHE_E4M3 ? 8 : KIND == CONVROT_CACHE_E2M1 ? 4 : 16;
    static constexpr int K_WORDS = LANE * BITS / 32;
    static constexpr int K_SCALES = QUANT ? (LANE + kBlock - 1) / kBlock : 1;
    static constexpr int WIDE = DIM == 64 ? 4 : 8;          // channels of a value that a lane loads at once
    static constexpr int SETS = DIM / (16 * WIDE);          // such loads a row
    static constexpr int V_BYTES = WIDE * BITS / 8;
    static constexpr int V_WORDS = (V_BYTES + 3) / 4;
    static constexpr int REGISTERS = 2 * K_WORDS + 8 * SETS * V_WORDS + (QUANT ? 2 * K_SCALES + 8 * SETS : 0);
    static constexpr int HELD = REGISTERS <= 32 ? 4 : REGISTERS <= 48 ? 3 : 2;   // steps in registers, the current one among them
};

template <int KIND, int DIM>
struct Tile {
    using S = Shape<KIND, DIM>;
    uint32_t k[2][S::K_WORDS];
    uint32_t v[8][S::SETS][S::V_WORDS];
    uint32_t ks[2][S::K_SCALES], vs[8][S::SETS];
};

// NW: waves of a workgroup.
template <typename T, int KIND, int DIM, int NW>
__global__ __launch_bounds__(64 * NW, DIM > 128 ? 1 : 2) void paged_kernel(PagedParams p)
{
    using S = Shape<KIND, DIM>;
    constexpr int PITCH = DIM + 4, TILES = S::SETS * S::WIDE;
    __shared__ float stats[NW][kPagedHeads][2];
    __shared__ __attribute__((aligned(16))) float outs[NW][kPagedHeads][PITCH];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int col = lane % 16, quad = lane / 16;
    const int dim = p.a.cache.head_dim;

    int64_t u = 0, last = 0;
    Place at{};
    int column, first;
    if (p.workgroups) {
        const int mine = units_of(length_of(p, lane));
        const int64_t units = all_units(p, mine) * p.columns;
        const int shares = sharing(p, units);
        if ((int)blockIdx.x >= shares) return;
        u = share_begin(units, shares, blockIdx.x);
        last = share_begin(units, shares, blockIdx.x + 1);
        at = find_unit(p, mine, u);
        if (at.units == 0) return;
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

    // Offsets of this lane's bytes from the first of 16 rows: row `col` of the keys, rows
    // 4 quad .. of the values.  What lies beyond the head is not read: its first bytes
    // stand for it, times a query's zeros, or for outputs that nobody reads.
    // (Infinities among them would leave no number: 16-bit values are cleared, and `inside`
    // makes a block's scale the smallest.)
    const convrot_cache_rows &kr = p.a.cache.k, &vr = p.a.cache.v;
    constexpr int K_PART = S::K_WORDS * 4 < 16 ? S::K_WORDS * 4 : 16;   // bytes of a load, all inside the head or beyond it
    constexpr int K_LOADS = S::K_WORDS * 4 / K_PART;
    uint32_t k_off[K_LOADS], v_off[S::SETS], ks_off[S::K_SCALES], vs_off[S::SETS];
    const auto key_channel = [&](int i) {    // first channel of load i of a key
        return S::QUANT ? quad * S::LANE + i * K_PART * 8 / S::BITS : i * 32 + quad * 8;
    };
#pragma unroll
    for (int i = 0; i < K_LOADS; ++i)
        k_off[i] = col * (uint32_t)kr.token_stride + (key_channel(i) < dim ? key_channel(i) * S::BITS / 8 : 0);
#pragma unroll
    for (int set = 0; set < S::SETS; ++set) {
        const int c = (set * 16 + col) * S::WIDE;
        v_off[set] = 4 * quad * (uint32_t)vr.token_stride + (c < dim ? c * S::BITS / 8 : 0);
        vs_off[set] = 4 * quad * (uint32_t)vr.scale_token_stride + (c < dim ? c / kBlock : 0);
    }
#pragma unroll
    for (int i = 0; i < S::K_SCALES; ++i) {
        const int c = quad * S::LANE + i * kBlock;
        ks_off[i] = col * (uint32_t)kr.scale_token_stride + (c < dim ? c / kBlock : 0);
    }

    uint32_t inside[(S::LANE + kBlock - 1) / kBlock];
#pragma unroll
    for (int i = 0; i < (S::LANE + kBlock - 1) / kBlock; ++i) inside[i] = quad * S::LANE + i * kBlock < dim ? ~0u : 0u;

    for (;;) {
        const int b = __builtin_amdgcn_readfirstlane(at.b), units = __builtin_amdgcn_readfirstlane(at.units);
        first = __builtin_amdgcn_readfirstlane(first);
        column = __builtin_amdgcn_readfirstlane(column);
        const int take = (int)min((int64_t)(units - first), last - u);
        const int length = __builtin_amdgcn_readfirstlane(length_of(p, b));
        const int head = column / p.groups, part = column % p.groups;
        const int heads = min(p.group - part * kPagedHeads, kPagedHeads);       // columns in use
        const int q_head = head * p.group + part * kPagedHeads;                 // the first of them
        typedef __attribute__((address_space(4))) const int Constant;           // scalar loads
        Constant* table = (Constant*)(p.a.page_table_dev + b * p.a.table_stride);
        const char* keys = (const char*)kr.rows_dev + head * kr.head_stride;
        const char* vals = (const char*)vr.rows_dev + head * vr.head_stride;
        const uint8_t* key_scales = kr.scales_dev + head * kr.scale_head_stride;
        const uint8_t* val_scales = vr.scales_dev + head * vr.scale_head_stride;
        // this wave's steps: t0, t0 + NW, ... below end; those of the whole share when it has none
        const int end = __builtin_amdgcn_readfirstlane(min((first + take) * (kPagedUnit / kPagedTile), (length + kPagedTile - 1) / kPagedTile));
        const int t0 = first * (kPagedUnit / kPagedTile) + wave;

        // The pages of a step's four groups of eight keys (a page has eight places at least);
        // behind the last key its page.
        struct Pages {
            int page[4];
        };
        const auto pages_of = [&](int t) {
            Pages x;
#pragma unroll
            for (int i = 0; i < 4; ++i) x.page[i] = table[min(min(t, end - 1) * kPagedTile + 8 * i, length - 1) >> p.shift];
            return x;
        };
        const auto good = [&](int page) { return (uint32_t)page < (uint32_t)p.a.cache.pages; };

        U4 q[S::STEPS];
        {
            const T* row = (const T*)p.a.q_dev + b * p.a.q_batch_stride + (q_head + min(col, heads - 1)) * p.a.q_head_stride;
#pragma unroll
            for (int i = 0; i < S::STEPS; ++i) {
                const int c = S::QUANT ? quad * S::LANE + i * 8 : i * 32 + quad * 8;
                q[i] = col < heads && c < dim ? __builtin_bit_cast(U4, load_chunk<uint16_t, 8>((const uint16_t*)row + c)) : U4{0, 0, 0, 0};
            }
        }

        const auto load = [&](Tile<KIND, DIM>& x, int t, const Pages& pages) {
            t = min(t, end - 1);    // behind the last step: it again, so that the loads under way are always as many
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // 16 keys, or twice 8 on pages of 8: their first rows
                const auto first_of = [&](int g, const char* base, int64_t page_stride, int64_t token_stride) {
                    const int page = pages.page[2 * h + g];
                    return base + (good(page) ? page : 0) * page_stride + ((t * kPagedTile + 16 * h + 8 * g) & ((1 << p.shift) - 1)) * token_stride;
                };
                const auto rows = [&](const char* base, int64_t page_stride, int64_t token_stride, int second) {
                    const char* low = first_of(0, base, page_stride, token_stride);
                    if (p.shift > 3) return low;
                    // offsets count from the first of the 16 rows
                    return second ? first_of(1, base, page_stride, token_stride) - 8 * token_stride : low;
                };
                const char* k_rows = rows(keys, kr.page_stride, kr.token_stride, col / 8);
                const char* v_rows = rows(vals, vr.page_stride, vr.token_stride, quad / 2);
#pragma unroll
                for (int i = 0; i < K_LOADS; ++i) {
                    if constexpr (K_PART == 16) {
                        const U4 r = read_row<!S::QUANT, U4>(k_rows + k_off[i]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) x.k[h][4 * i + j] = r[j];
                    } else {
                        const U2 r = read_row<!S::QUANT, U2>(k_rows + k_off[i]);
                        x.k[h][0] = r[0];
                        x.k[h][1] = r[1];
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int set = 0; set < S::SETS; ++set) {
                        const char* at_v = v_rows + j * vr.token_stride + v_off[set];
                        uint32_t(&d)[S::V_WORDS] = x.v[4 * h + j][set];
                        if constexpr (S::V_BYTES == 16) {
                            const U4 r = read_row<!S::QUANT, U4>(at_v);
                            d[0] = r[0], d[1] = r[1], d[2] = r[2], d[3] = r[3];
                        } else if constexpr (S::V_BYTES == 8) {
                            const U2 r = read_row<!S::QUANT, U2>(at_v);
                            d[0] = r[0], d[1] = r[1];
                        } else if constexpr (S::V_BYTES == 4) {
                            d[0] = *(const uint32_t*)at_v;
                        } else {
                            d[0] = *(const uint16_t*)at_v;
                        }
                    }
                if constexpr (S::QUANT) {
                    const char* ks_rows = rows((const char*)key_scales, kr.scale_page_stride, kr.scale_token_stride, col / 8);
                    const char* vs_rows = rows((const char*)val_scales, vr.scale_page_stride, vr.scale_token_stride, quad / 2);
#pragma unroll
                    for (int i = 0; i < S::K_SCALES; ++i) x.ks[h][i] = *(const uint8_t*)(ks_rows + ks_off[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int set = 0; set < S::SETS; ++set)
                            x.vs[4 * h + j][set] = *(const uint8_t*)(vs_rows + j * vr.scale_token_stride + vs_off[set]);
                }
            }
        };

        float m = -kInf, sum = 0.f;
        F4 o[TILES];
#pragma unroll
        for (int i = 0; i < TILES; ++i) o[i] = F4{0, 0, 0, 0};

        const auto step = [&](Tile<KIND, DIM>& x, int t, const Pages& pages) {
            float s[8];
            if constexpr (!S::QUANT) {
                if (__builtin_expect(dim < DIM, 0)) {
#pragma unroll
                    for (int i = 0; i < S::K_WORDS; ++i)
                        if (i / 4 * 32 + quad * 8 >= dim) x.k[0][i] = x.k[1][i] = 0;
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                F4 acc{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < S::STEPS; ++i) {
                    U4 a;
                    const uint32_t in = inside[i * 8 / kBlock];
                    if constexpr (!S::QUANT) a = U4{x.k[h][4 * i], x.k[h][4 * i + 1], x.k[h][4 * i + 2], x.k[h][4 * i + 3]};
                    else if constexpr (KIND == CONVROT_CACHE_E4M3) a = Unpack<T>::e4m3(x.k[h][2 * i], x.k[h][2 * i + 1], block_scale(x.ks[h][i * 8 / kBlock] & in));
                    else a = Unpack<T>::e2m1(x.k[h][i], block_scale(x.ks[h][i * 8 / kBlock] & in));
                    acc = Mfma16<T>::run(a, q[i], acc);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) s[4 * h + j] = acc[j] * p.scale;
            }
            bool whole = (t + 1) * kPagedTile <= length;
#pragma unroll
            for (int i = 0; i < 4; ++i) whole &= good(pages.page[i]);
            if (!whole) {
                // keys behind the last one, or on a page that is none: not seen, and their values zeros
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int page = quad < 2 ? pages.page[j / 4 * 2] : pages.page[j / 4 * 2 + 1];
                    if (good(page) && t * kPagedTile + (j & 4) * 4 + quad * 4 + (j & 3) < length) continue;
                    s[j] = -kInf;
#pragma unroll
                    for (int set = 0; set < S::SETS; ++set) {
                        x.vs[j][set] = 0;
#pragma unroll
                        for (int k = 0; k < S::V_WORDS; ++k) x.v[j][set][k] = 0;
                    }
                }
            }
            float most = s[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) most = fmaxf(most, s[j]);
            if (__ballot(leaves_room<T>(most, m))) {
                const float next = fmaxf(m, reference<T>(max4(most)));
                const float f = next == -kInf ? 0.f : exp2_fast(m - next);
                sum *= f;
#pragma unroll
                for (int i = 0; i < TILES; ++i) o[i] *= f;
                m = next;
            }
            const float base = m == -kInf ? 0.f : m;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma clang fp contract(off)     // the score is the rounded one that the reference was taken from
                s[j] = exp2_fast(s[j] - base);
                sum += s[j];
            }
            // weights rounded to T, as the outputs are (Reference)
            const U4 w{pack2<T>(s[0], s[1]), pack2<T>(s[2], s[3]), pack2<T>(s[4], s[5]), pack2<T>(s[6], s[7])};
#pragma unroll
            for (int set = 0; set < S::SETS; ++set) {
                U4 v[8];     // a value's channels as registers of two
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t(&d)[S::V_WORDS] = x.v[j][set];
                    if constexpr (!S::QUANT) {
                        v[j] = U4{d[0], d[1], S::WIDE == 8 ? d[S::V_WORDS - 2] : 0u, S::WIDE == 8 ? d[S::V_WORDS - 1] : 0u};
                    } else {
                        const float scale = block_scale(x.vs[j][set]);
                        if constexpr (KIND == CONVROT_CACHE_E4M3) v[j] = Unpack<T>::e4m3(d[0], S::WIDE == 8 ? d[S::V_WORDS - 1] : 0u, scale);
                        else v[j] = Unpack<T>::e2m1(d[0], scale);
                    }
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

        // Steps in registers in turn; a step's pages are asked for before its rows.
        if (t0 + NW >= end) {
            if (t0 < end) {     // one step: nothing to ask for ahead
                Tile<KIND, DIM> x;
                const Pages pages = pages_of(t0);
                load(x, t0, pages);
                step(x, t0, pages);
            }
        } else {
            constexpr int HELD = S::HELD;
            Tile<KIND, DIM> x[HELD];
            Pages pages[HELD];
#pragma unroll
            for (int i = 0; i < HELD; ++i) pages[i] = pages_of(t0 + i * NW);
#pragma unroll
            for (int i = 0; i + 1 < HELD; ++i) load(x[i], t0 + i * NW, pages[i]);
            for (int t = t0; t < end;) {
#pragma unroll
                for (int i = 0; i < HELD; ++i) {
                    constexpr int LAST = HELD - 1;
                    load(x[(i + LAST) % HELD], t + LAST * NW, pages[(i + LAST) % HELD]);
                    step(x[i], t, pages[i]);
                    pages[i] = pages_of(t + HELD * NW);
                    t += NW;
                    if (t >= end) break;
                }
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
        const bool whole = take == units;
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
                store_chunk<uint16_t, 4>((uint16_t*)p.a.o_dev + b * p.a.o_batch_stride + (q_head + h) * p.a.o_head_stride + c,
                                         __builtin_bit_cast(H4, packed));
                if (c == 0 && p.a.lse_dev)
                    p.a.lse_dev[(int64_t)b * p.a.q_heads + q_head + h] = log_sum<T>(most, total);
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
            do {
                if (++at.b >= p.a.batch) return;
                at.units = units_of(length_of(p, at.b));
            } while (at.units == 0);
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
    const int here = units_of(length_of(p, lane));
    const int mine = b < 64 ? __builtin_amdgcn_readlane(here, b) : units_of(length_of(p, b));
    int w0 = 0, count = 0, shares = 0;
    int64_t units = 0, u0 = 0;
    if (mine > 0) {
        int64_t before = wave_sum(lane < b ? here : 0);
        units = wave_sum(here);
        for (int64_t c = 64; c < p.a.batch; c += 256) {
            Quad q(p, c);
            units += q.sum();
#pragma unroll
            for (int i = 0; i < 4; ++i) q.n[i] = c + 64 * i + lane < b ? q.n[i] : 0;
            before += q.sum();
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
    // four channels a thread; threads left over share the parts.  The first four parts
    // are asked for here, the others where they are summed.
    const int items = heads * (dim / 4), groups = max(256 / items, 1);
    const int first = (int)threadIdx.x % min(items, 256), g = groups > 1 ? threadIdx.x / items : 0;
    F4 early[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        early[k] = g + k * groups < count && g < groups ? *(const F4*)(slot(g + k * groups) + 2 * kPagedHeads + first / (dim / 4) * pitch + first % (dim / 4) * 4) : F4{0, 0, 0, 0};
    // a wave a head: what each part counts for
    for (int h = wave; h < heads; h += 4) {
        const float m0 = lane < count ? slot(lane)[2 * h] : -kInf, l0 = lane < count ? slot(lane)[2 * h + 1] : 0.f;
        float most = m0;
        for (int i = lane + 64; i < count; i += 64) most = fmaxf(most, slot(i)[2 * h]);
#pragma unroll
        for (int d = 1; d < 64; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
        const float f0 = m0 == -kInf ? 0.f : exp2_fast(m0 - most);
        factors[h][lane] = f0;
        float total = l0 * f0;
        for (int i = lane + 64; i < count; i += 64) {
            const float m = slot(i)[2 * h], f = m == -kInf ? 0.f : exp2_fast(m - most);
            factors[h][i] = f;
            total += slot(i)[2 * h + 1] * f;
        }
        total = lane_sum<64>(total);
        if (lane == 0) {
            scales[h] = total == 0.f ? 0.f : 1.f / total;
            if (p.a.lse_dev) p.a.lse_dev[(int64_t)b * p.a.q_heads + q_head + h] = log_sum<T>(most, total);
        }
    }
    __syncthreads();
    for (int i0 = 0; i0 < items; i0 += 256) {
        const int item = i0 + first, h = item / (dim / 4), c = item % (dim / 4) * 4;
        const bool on = item < items && g < groups;
        F4 out{0, 0, 0, 0};
        if (on) {
            int i = g;
            if (i0 == 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (g + k * groups < count) out += early[k] * factors[h][g + k * groups];
                i += 4 * groups;
            }
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

template <typename T, int KIND, int DIM>
void launch_paged_dim(const PagedParams& p, unsigned grid, hipStream_t s)
{
    constexpr int ALONE = DIM > 128 ? kPagedWaves : kPagedWavesAlone;    // registers for 256 channels leave one wave a SIMD
    if (p.workgroups || grid >= kPagedMany) paged_kernel<T, KIND, DIM, kPagedWaves><<<grid, 64 * kPagedWaves, 0, s>>>(p);
    else paged_kernel<T, KIND, DIM, ALONE><<<grid, 64 * ALONE, 0, s>>>(p);
}
template <typename T, int KIND>
void launch_paged_kind(const PagedParams& p, unsigned grid, hipStream_t s)
{
    switch (padded_dim(p.a.cache.head_dim)) {
    case 64: launch_paged_dim<T, KIND, 64>(p, grid, s); break;
    case 128: launch_paged_dim<T, KIND, 128>(p, grid, s); break;
    default: launch_paged_dim<T, KIND, 256>(p, grid, s); break;
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
