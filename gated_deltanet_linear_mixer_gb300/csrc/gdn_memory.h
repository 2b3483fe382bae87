// Whether two arguments of a call share memory (host side).
#pragma once

#include <stdint.h>

namespace gdn {

// Memory of rows [tokens, heads] of `width` bytes, strides in bytes; a contiguous array is one row.
struct Memory {
    long long base, token_stride, head_stride, tokens, heads, width;
    static Memory rows(const void* p, long long tokens, long long heads, long long token_stride, long long head_stride, long long channels,
                       long long bytes) {
        Memory m{static_cast<long long>(reinterpret_cast<uintptr_t>(p)), tokens > 1 ? token_stride : 0,
                 heads > 1 ? head_stride : 0, tokens, heads, bytes * channels};
        // no rows, or strides that no memory is large enough for
        if (tokens < 1 || heads < 1 || m.token_stride >= 1ll << 56 || m.head_stride >= 1ll << 56) m.width = 0;
        m.token_stride *= m.width ? bytes : 0;
        m.head_stride *= m.width ? bytes : 0;
        return m;
    }
    static Memory array(const void* p, long long bytes) { return rows(p, 1, 1, 0, 0, bytes, 1); }
    // The same bytes as fewer and longer rows, where rows lie side by side.
    Memory joined() const {
        Memory m = *this;
        for (int i = 0; i < 2; ++i) {
            if (m.heads > 1 && m.head_stride == m.width) m.width *= m.heads, m.heads = 1, m.head_stride = 0;
            if (m.tokens > 1 && m.token_stride == m.width) m.width *= m.tokens, m.tokens = 1, m.token_stride = 0;
        }
        return m;
    }
    bool end(long long* at) const {  // false where that is no address
        long long t, h;
        return !__builtin_mul_overflow(tokens - 1, token_stride, &t) && !__builtin_mul_overflow(heads - 1, head_stride, &h) &&
               !__builtin_add_overflow(base + width, t, at) && !__builtin_add_overflow(*at, h, at);
    }
};
// Whether lo < d step < hi for a d of first .. last.
inline bool step_between(long long first, long long last, long long step, long long lo, long long hi) {
    if (step == 0) return lo < 0 && 0 < hi;
    const long long above = lo / step - (lo % step < 0 ? 1 : 0) + 1;  // floor(lo / step) + 1
    const long long d = above > first ? above : first;
    return d <= last && d * step < hi;
}
// Whether two of them share bytes.  Rows whose token strides differ, where their extents overlap, are not
// told apart (false).
inline bool meet(const Memory& a, const Memory& b) {
    long long end_a, end_b;
    if (!a.end(&end_a) || !b.end(&end_b) || a.base >= end_b || b.base >= end_a || a.width == 0 || b.width == 0) return false;
    if (a.tokens > 1 && b.tokens > 1 && a.token_stride != b.token_stride) return false;
    const long long step = a.tokens > 1 ? a.token_stride : b.token_stride;
    // row (d tokens, heads) of a from row 0 of b on: at x + d step, and from -a.width to b.width they meet
    auto at = [&](long long x) { return step_between(1 - b.tokens, a.tokens - 1, step, -a.width - x, b.width - x); };
    const long long x = a.base - b.base;
    if (a.head_stride == b.head_stride || a.heads == 1 || b.heads == 1) {
        const long long hs = a.heads > 1 ? a.head_stride : b.head_stride;
        for (long long h = 1 - b.heads; h < a.heads; ++h)
            if (at(x + h * hs)) return true;
        return false;
    }
    for (long long h = 0; h < a.heads; ++h)
        for (long long k = 0; k < b.heads; ++k)
            if (at(x + h * a.head_stride - k * b.head_stride)) return true;
    return false;
}
inline bool same(const Memory& a, const Memory& b) {
    return a.base == b.base && a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}

}  // namespace gdn
