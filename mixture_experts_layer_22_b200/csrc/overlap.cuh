// overlap.cuh - whether two buffers of a call share memory (host side).
#pragma once
#include <cstdint>

namespace moe {

// A buffer: n pieces of `bytes` bytes, `step` bytes apart (a dense one is one piece), up to
// `end`.  One that is NULL or empty ends at 0 and so shares nothing.
struct Extent {
    uintptr_t at, end;
    int64_t bytes, step, n;

    Extent(const void *p, int64_t bytes_) : Extent(p, bytes_, bytes_, 1) {}
    Extent(const void *p, int64_t bytes_, int64_t step_, int64_t n_)
        : at(reinterpret_cast<uintptr_t>(p)), end(0), bytes(bytes_), step(step_), n(n_)
    {
        if (at != 0 && bytes > 0 && n > 0) end = at + static_cast<uintptr_t>((n - 1) * step + bytes);
    }
};

// Piece by piece, exactly: a piece that lies between two pieces of the other buffer shares
// nothing with it.  With one step for both (K and V pages that alternate, millions of
// them) piece i of a and piece j of b are apart by what j - i says.
inline bool pieces_overlap(const Extent &a, const Extent &b)
{
    if (a.step == b.step && a.n > 1 && b.n > 1) {
        // the least d = j - i with which b's piece ends behind the start of a's
        const int64_t diff = static_cast<int64_t>(a.at - b.at), x = diff - b.bytes;
        int64_t d = x / a.step - (x % a.step < 0 ? 1 : 0) + 1;
        if (d < 1 - a.n) d = 1 - a.n;
        return d < b.n && d * a.step < diff + a.bytes;
    }
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

// Nearly always two comparisons: a call has some fifty pairs of buffers.
inline bool overlap(const Extent &a, const Extent &b) { return a.at < b.end && b.at < a.end && pieces_overlap(a, b); }

}  // namespace moe
