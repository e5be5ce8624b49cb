// overlap.h -- host checks shared by the operators around a rotated linear:
// whether strided blocks of elements share memory, and how far strides reach.
#pragma once
#include <stdint.h>

namespace convrot {

inline bool within(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

// A strided block of elements: `inner` dense ones, repeated over up to three
// dimensions, the largest stride first.  Dimensions of one element are left out.
struct Block {
    const char* at;
    int64_t bytes;   // of the dense run
    int dims = 0;
    int64_t size[3], stride[3];   // strides in bytes

    Block(const void* p, int64_t inner, int elem) : at((const char*)p), bytes(inner * elem) {}
    void add(int64_t n, int64_t s, int elem)
    {
        if (n <= 1) return;
        int i = dims++;
        for (; i > 0 && stride[i - 1] < s * elem; --i) {
            size[i] = size[i - 1];
            stride[i] = stride[i - 1];
        }
        size[i] = n;
        stride[i] = s * elem;
    }
    int64_t extent(int from = 0) const
    {
        int64_t e = bytes;
        for (int i = from; i < dims; ++i) e += (size[i] - 1) * stride[i];
        return e;
    }
    // no element is reached twice
    bool injective() const
    {
        for (int i = 0; i < dims; ++i)
            if (stride[i] < extent(i + 1)) return false;
        return true;
    }
    bool same(const Block& b) const
    {
        if (at != b.at || bytes != b.bytes || dims != b.dims) return false;
        for (int i = 0; i < dims; ++i)
            if (size[i] != b.size[i] || stride[i] != b.stride[i]) return false;
        return true;
    }
};

// Whether b, starting d bytes behind a, shares no byte with a (dimensions from
// `level` on).  Ranges that cross are told apart as long as both step by the
// same stride; otherwise they count as shared.
inline bool apart(const Block& a, const Block& b, int64_t d, int level)
{
    if (d >= a.extent(level) || -d >= b.extent(level)) return true;
    if (level >= a.dims || level >= b.dims || a.stride[level] != b.stride[level] || a.stride[level] == 0) return false;
    const int64_t s = a.stride[level];
    if (a.extent(level + 1) > s || b.extent(level + 1) > s) return false;
    const int64_t rest = ((d % s) + s) % s;
    return apart(a, b, rest, level + 1) && apart(a, b, rest - s, level + 1);
}
inline bool apart(const Block& a, const Block& b) { return apart(a, b, (int64_t)((intptr_t)b.at - (intptr_t)a.at), 0); }

// largest stride taken, and largest offset that a dimension may reach, in
// elements: keeps every offset far inside 64 bits
constexpr int64_t kMaxStride = (int64_t)1 << 40, kMaxReach = (int64_t)1 << 56;
inline bool reaches(int64_t n, int64_t stride)
{
    return within(stride, 0, kMaxStride) && (n <= 1 || stride <= kMaxReach / (n - 1));
}

}  // namespace convrot
