// overlap.cuh - whether two buffers of a call share memory (host side).
#pragma once
#include <cstdint>

namespace moe {

// A buffer: n pieces of `bytes` bytes, `step` bytes apart (a dense one is one piece).
struct Extent {
    uintptr_t at;
    int64_t bytes, step, n;

    Extent(const void *p, int64_t bytes_) : Extent(p, bytes_, bytes_, 1) {}
    Extent(const void *p, int64_t bytes_, int64_t step_, int64_t n_)
        : at(reinterpret_cast<uintptr_t>(p)), bytes(bytes_), step(step_), n(n_)
    {
        if (step == bytes) {
            bytes *= n;
            n = 1;
        }
    }
    bool none() const { return at == 0 || bytes <= 0 || n <= 0; }
    uintptr_t end() const { return at + static_cast<uintptr_t>((n - 1) * step + bytes); }
};

// Exact: a piece that lies between two pieces of the other buffer shares nothing with it.
// Only buffers that lie in one another's range are compared piece by piece.
inline bool overlap(const Extent &a, const Extent &b)
{
    if (a.none() || b.none() || a.at >= b.end() || b.at >= a.end()) return false;
    const Extent &few = a.n <= b.n ? a : b, &many = a.n <= b.n ? b : a;
    for (int64_t i = 0; i < few.n; ++i) {
        const uintptr_t from = few.at + static_cast<uintptr_t>(i * few.step), behind = from + static_cast<uintptr_t>(few.bytes);
        // the first piece of the other that ends behind `from`
        const uintptr_t first_end = many.at + static_cast<uintptr_t>(many.bytes);
        const int64_t j = from < first_end ? 0 : static_cast<int64_t>((from - first_end) / static_cast<uintptr_t>(many.step)) + 1;
        if (j < many.n && many.at + static_cast<uintptr_t>(j * many.step) < behind) return true;
    }
    return false;
}

}  // namespace moe
