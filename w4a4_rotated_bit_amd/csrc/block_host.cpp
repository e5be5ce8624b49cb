// block_host.cpp -- argument checks of the operators around a rotated linear.
// Pure C++: nothing here calls the HIP runtime.
#include <math.h>
#include <stdlib.h>

#include <algorithm>

#include "../../include/convrot.h"
#include "block_ops.h"
#include "internal.h"
#include "overlap.h"

using namespace convrot;

namespace {

bool known_type(int dtype) { return dtype == CONVROT_BF16 || dtype == CONVROT_F16 || dtype == CONVROT_F32; }
bool known_norm(int norm) { return norm == CONVROT_NORM_NONE || norm == CONVROT_NORM_LAYER || norm == CONVROT_NORM_RMS; }

}  // namespace

extern "C" {

int convrot_validate_residual_norm(const convrot_residual_norm_args* args)
{
    if (!args) return CONVROT_EINVAL;
    const convrot_residual_norm_args& a = *args;
    if (!known_type(a.dtype) || (a.vec_dtype != a.dtype && a.vec_dtype != CONVROT_F32)) return CONVROT_EINVAL;
    if (!within(a.rows, 0, kMaxRows) || !within(a.width, 1, kMaxNormWidth)) return CONVROT_EINVAL;
    if (!known_norm(a.norm) || !known_norm(a.post_norm)) return CONVROT_EINVAL;
    if (!(a.eps >= 0.f) || a.rows_per_vec < 1) return CONVROT_EINVAL;
    const int64_t vectors = a.rows > 0 ? (a.rows - 1) / a.rows_per_vec + 1 : 0;
    for (int64_t s : {a.x_stride, a.y_stride, a.r_stride, a.h_stride})
        if (!reaches(a.rows, s)) return CONVROT_EINVAL;
    for (int64_t s : {a.gate_stride, a.scale_stride, a.shift_stride})
        if (!reaches(vectors, s)) return CONVROT_EINVAL;
    if (a.rows == 0) return CONVROT_OK;   // empty buffers may be NULL
    if (!a.y_dev && (a.gate_dev || a.post_norm != CONVROT_NORM_NONE)) return CONVROT_EINVAL;
    if (a.post_weight_dev && a.post_norm == CONVROT_NORM_NONE) return CONVROT_EINVAL;
    if (!a.r_dev && !a.h_dev) return CONVROT_EINVAL;
    if (!a.h_dev && (a.weight_dev || a.scale_dev || a.shift_dev)) return CONVROT_EINVAL;
    if (!a.x_dev) return CONVROT_EINVAL;
    const int e = elem_bytes(a.dtype), v = elem_bytes(a.vec_dtype);
    for (const void* p : {a.x_dev, a.y_dev, (const void*)a.r_dev, (const void*)a.h_dev})
        if (!aligned(p, e)) return CONVROT_EINVAL;
    for (const void* p : {a.gate_dev, a.scale_dev, a.shift_dev, a.weight_dev, a.post_weight_dev})
        if (!aligned(p, v)) return CONVROT_EINVAL;
    const auto block = [&](const void* p, int64_t stride) {
        Block b(p, a.width, e);
        b.add(a.rows, stride, e);
        return b;
    };
    const Block x = block(a.x_dev, a.x_stride), y = block(a.y_dev, a.y_stride);
    const Block r = block(a.r_dev, a.r_stride), h = block(a.h_dev, a.h_stride);
    for (const Block& out : {r, h}) {
        if (!out.at) continue;
        if (!out.injective()) return CONVROT_EINVAL;
        if (!out.same(x) && !apart(x, out)) return CONVROT_EINVAL;
        if (y.at && !out.same(y) && !apart(y, out)) return CONVROT_EINVAL;
    }
    if (r.at && h.at && !apart(r, h)) return CONVROT_EINVAL;
    const struct {
        const void* at;
        int64_t stride, count;
    } vecs[] = {{a.gate_dev, a.gate_stride, vectors}, {a.scale_dev, a.scale_stride, vectors},
                {a.shift_dev, a.shift_stride, vectors}, {a.weight_dev, 0, 1}, {a.post_weight_dev, 0, 1}};
    for (const auto& g : vecs) {
        if (!g.at) continue;
        Block b(g.at, a.width, v);
        b.add(g.count, g.stride, v);
        if ((r.at && !apart(b, r)) || (h.at && !apart(b, h))) return CONVROT_EINVAL;
    }
    return CONVROT_OK;
}

int convrot_validate_rope(const convrot_rope_args* args)
{
    if (!args) return CONVROT_EINVAL;
    const convrot_rope_args& a = *args;
    if (!known_type(a.dtype) || !within(a.count, 1, kMaxRopeTensors)) return CONVROT_EINVAL;
    if (!within(a.batch, 0, 65535) || !within(a.tokens, 0, kMaxRows)) return CONVROT_EINVAL;
    if (!within(a.head_dim, 1, kMaxHeadDim) || !within(a.pairs, 1, a.head_dim / 2)) return CONVROT_EINVAL;
    if (!within(a.axes, 1, kMaxRopeAxes) || !a.freq_host || !a.axis_host) return CONVROT_EINVAL;
    for (int i = 0; i < a.pairs; ++i)
        if (!isfinite(a.freq_host[i]) || !within(a.axis_host[i], 0, a.axes - 1)) return CONVROT_EINVAL;
    if (a.layout != CONVROT_ROPE_INTERLEAVED && a.layout != CONVROT_ROPE_HALVES) return CONVROT_EINVAL;
    if (a.norm != CONVROT_NORM_NONE && a.norm != CONVROT_NORM_RMS) return CONVROT_EINVAL;
    if (!(a.eps >= 0.f) || (a.pos_dtype != CONVROT_I32 && a.pos_dtype != CONVROT_F32)) return CONVROT_EINVAL;
    if (!reaches(a.batch, a.pos_batch_stride) || !reaches(a.tokens, a.pos_token_stride)) return CONVROT_EINVAL;
    const bool empty = a.batch == 0 || a.tokens == 0;
    if (!empty && (!a.pos_dev || !aligned(a.pos_dev, 4))) return CONVROT_EINVAL;
    const int e = elem_bytes(a.dtype);
    for (int k = 0; k < a.count; ++k) {
        const convrot_heads& h = a.heads[k];
        if (!within(h.heads, 1, kMaxHeads)) return CONVROT_EINVAL;
        if (!reaches(a.batch, h.in_batch_stride) || !reaches(a.batch, h.out_batch_stride)) return CONVROT_EINVAL;
        if (!reaches(a.tokens, h.in_token_stride) || !reaches(a.tokens, h.out_token_stride)) return CONVROT_EINVAL;
        if (!reaches(h.heads, h.in_head_stride) || !reaches(h.heads, h.out_head_stride)) return CONVROT_EINVAL;
        if (h.weight_dev && a.norm == CONVROT_NORM_NONE) return CONVROT_EINVAL;
        if (empty) continue;
        if (!h.in_dev || !h.out_dev) return CONVROT_EINVAL;
        if (!aligned(h.in_dev, e) || !aligned(h.out_dev, e) || !aligned(h.weight_dev, e)) return CONVROT_EINVAL;
    }
    if (empty) return CONVROT_OK;
    const auto block = [&](const convrot_heads& h, bool out) {
        Block b(out ? h.out_dev : h.in_dev, a.head_dim, e);
        b.add(a.batch, out ? h.out_batch_stride : h.in_batch_stride, e);
        b.add(a.tokens, out ? h.out_token_stride : h.in_token_stride, e);
        b.add(h.heads, out ? h.out_head_stride : h.in_head_stride, e);
        return b;
    };
    Block places(a.pos_dev, a.axes, 4);
    places.add(a.batch, a.pos_batch_stride, 4);
    places.add(a.tokens, a.pos_token_stride, 4);
    for (int k = 0; k < a.count; ++k) {
        const Block out = block(a.heads[k], true);
        if (!out.injective() || !apart(places, out)) return CONVROT_EINVAL;
        for (int j = 0; j < a.count; ++j) {
            const Block in = block(a.heads[j], false);
            if (!(j == k && out.same(in)) && !apart(in, out)) return CONVROT_EINVAL;
            if (j < k && !apart(block(a.heads[j], true), out)) return CONVROT_EINVAL;
            if (a.heads[j].weight_dev && !apart(Block(a.heads[j].weight_dev, a.head_dim, e), out)) return CONVROT_EINVAL;
        }
    }
    return CONVROT_OK;
}

int convrot_validate_linear_grouped(const convrot_grouped_args* args)
{
    if (!args) return CONVROT_EINVAL;
    const convrot_grouped_args& a = *args;
    if (a.dtype != CONVROT_BF16 && a.dtype != CONVROT_F16) return CONVROT_EINVAL;
    if (a.group != 32 && a.group != 64 && a.group != 128) return CONVROT_EINVAL;
    if (!within(a.M, 0, kMaxGroupedM) || !within(a.N, 0, kMaxRows)) return CONVROT_EINVAL;
    if (!within(a.K, a.group, kMaxGroupedK) || a.K % a.group != 0) return CONVROT_EINVAL;
    if (a.M == 0 || a.N == 0) return CONVROT_OK;
    if (!a.x_dev || !a.codes_dev || !a.scales_dev || !a.y_dev) return CONVROT_EINVAL;
    if (!aligned(a.x_dev, 16) || !aligned(a.codes_dev, 16)) return CONVROT_EINVAL;
    if (!aligned(a.scales_dev, 2) || !aligned(a.bias_dev, 2) || !aligned(a.y_dev, 2)) return CONVROT_EINVAL;
    const Block y(a.y_dev, a.M * a.N, 2);
    const int64_t groups = a.N * (a.K / a.group);
    for (const Block& in : {Block(a.x_dev, a.M * a.K, 2), Block(a.codes_dev, a.N * (a.K / 2), 1), Block(a.scales_dev, groups, 2)})
        if (!apart(in, y)) return CONVROT_EINVAL;
    if (a.zeros_dev && !apart(Block(a.zeros_dev, groups, 1), y)) return CONVROT_EINVAL;
    if (a.bias_dev && !apart(Block(a.bias_dev, a.N, 2), y)) return CONVROT_EINVAL;
    return CONVROT_OK;
}

int convrot_validate_quantize_weight_grouped(const void* W, int64_t N, int64_t K, int group, int dtype,
                                             const uint8_t* codes, const void* scales, const uint8_t* zeros)
{
    if (dtype != CONVROT_BF16 && dtype != CONVROT_F16) return CONVROT_EINVAL;
    if (group != 32 && group != 64 && group != 128) return CONVROT_EINVAL;
    if (!within(N, 0, kMaxRows) || !within(K, group, kMaxGroupedK) || K % group != 0) return CONVROT_EINVAL;
    if (N == 0) return CONVROT_OK;
    if (!W || !codes || !scales || !aligned(W, 2) || !aligned(scales, 2)) return CONVROT_EINVAL;
    const int64_t groups = N * (K / group);
    const Block all[] = {Block(W, N * K, 2), Block(codes, N * (K / 2), 1), Block(scales, groups, 2), Block(zeros, groups, 1)};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (all[i].at && !apart(all[i], all[j])) return CONVROT_EINVAL;
    return CONVROT_OK;
}

}  // extern "C"
