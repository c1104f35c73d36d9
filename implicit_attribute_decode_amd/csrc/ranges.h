// Whether memory that a call writes shares a byte with anything else that it
// reads or writes (host only).  Blocks of one launch run in no order, so such
// a call would have no defined result.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <memory>
#include <new>
#include <numeric>

namespace ia {

// `rows` rows of `width` bytes, `pitch` >= width bytes apart.
struct Rows {
    uintptr_t at;
    uint64_t rows, width, pitch;
    bool written;

    uintptr_t end() const { return at + (rows - 1) * pitch + width; }
};

// Rows of `cols` elements of `es` bytes, `ld` elements apart (0 repeats one row).
inline Rows rows_of(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t es, bool written) {
    if (!p || rows <= 0 || cols <= 0) return Rows{0, 0, 0, 0, written};
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const uint64_t width = (uint64_t)cols * es, pitch = (uint64_t)ld * es;
    if (rows == 1 || ld == 0) return Rows{at, 1, width, width, written};
    if (ld == cols) return Rows{at, 1, width * (uint64_t)rows, width * (uint64_t)rows, written};
    return Rows{at, (uint64_t)rows, width, pitch, written};
}
inline Rows bytes_of(const void* p, size_t bytes, bool written) { return rows_of(p, 1, (int64_t)bytes, 0, 1, written); }

// The rows k0 .. k1 of a that share a byte with [lo, hi); false if none does
// (rows are in order, so these are consecutive).
inline bool rows_in(const Rows& a, uintptr_t lo, uintptr_t hi, uint64_t& k0, uint64_t& k1) {
    if (hi <= a.at) return false;
    k0 = lo < a.at + a.width ? 0 : (lo - a.at - a.width) / a.pitch + 1;  // the first that ends after lo
    k1 = std::min((hi - 1 - a.at) / a.pitch, a.rows - 1);                // the last that starts before hi
    return k0 <= k1;
}

// a and b share a byte.  Row by row of a within b's extent; where that is long,
// one period of the rows' places between b's rows (all rows but the first and the
// last lie wholly within the extent, where only that place counts) and the last.
inline bool share(const Rows& a, const Rows& b) {
    if (a.rows == 0 || b.rows == 0) return false;
    uint64_t a0, a1, b0, b1, x, y;
    if (!rows_in(a, b.at, b.end(), a0, a1) || !rows_in(b, a.at, a.end(), b0, b1)) return false;
    const uint64_t g = std::gcd(a.pitch, b.pitch);
    if (std::min(a1 - a0, b.pitch / g) > std::min(b1 - b0, a.pitch / g)) return share(b, a);
    const auto meets = [&](uint64_t k) {
        const uintptr_t at = a.at + k * a.pitch;
        return rows_in(b, at, at + a.width, x, y);
    };
    for (uint64_t k = a0, stop = std::min(a1, a0 + b.pitch / g); k <= stop; ++k)
        if (meets(k)) return true;
    return meets(a1);
}

// Some written range shares a byte with another range (few ranges: every pair).
inline bool clash(const Rows* r, int n) {
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < i; ++j)
            if ((r[i].written || r[j].written) && share(r[i], r[j])) return true;
    return false;
}

// The same for many ranges, filled in runs that are mostly in order of address:
// a sweep over the starts.
class Ranges {
public:
    // Room for n ranges; false without memory.
    bool reserve(size_t n) {
        items_.reset(new (std::nothrow) Rows[n]);
        open_.reset(new (std::nothrow) uint32_t[n]);
        return items_ && open_;
    }
    void add(const Rows& r) {
        if (r.rows > 0) items_[count_++] = r;
    }
    // Ends a run of add()s.
    void run_done() {
        const auto before = [](const Rows& a, const Rows& b) { return a.at < b.at; };
        Rows* const first = items_.get();
        if (!std::is_sorted(first + done_, first + count_, before)) std::sort(first + done_, first + count_, before);
        if (done_ > 0 && done_ < count_ && before(first[done_], first[done_ - 1]))
            std::inplace_merge(first, first + done_, first + count_, before);
        done_ = count_;
    }
    bool clash() {
        size_t open = 0;
        for (size_t i = 0; i < count_; ++i) {
            const Rows& r = items_[i];
            size_t kept = 0;
            for (size_t k = 0; k < open; ++k) {
                const Rows& o = items_[open_[k]];
                if (o.end() <= r.at) continue;
                if ((o.written || r.written) && share(o, r)) return true;
                open_[kept++] = open_[k];
            }
            open_[kept++] = (uint32_t)i;
            open = kept;
        }
        return false;
    }

private:
    std::unique_ptr<Rows[]> items_;
    std::unique_ptr<uint32_t[]> open_;
    size_t count_ = 0, done_ = 0;
};

}  // namespace ia
