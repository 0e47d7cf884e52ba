// wsm_deal.cuh -- how paged attention deals its work out (wsm_cache.cu): plain functions, which compile for the host
// too, where they are tested.  Not part of the public C ABI.
//
// The groups of kGroup tokens of all (sequence, key-value head, query tile) items lie end to end in a line, each item
// with a fixed cost before its groups; every warp takes an equal consecutive range of the line.
#pragma once

#if defined(__CUDACC__)
#define WSM_HD __host__ __device__ __forceinline__
#else
#define WSM_HD inline
#endif

namespace wsm {

constexpr int kGroup = 16;          // tokens a warp takes at a time (the MMA's k)
constexpr int kMinShare = 4;        // least length of a warp's range: no more than the shortest item's
constexpr int kSnapGroups = 8;      // items of up to this many groups (128 tokens) are never cut
// What beginning and ending an item costs a warp, in groups: counted when the work is dealt out, so that a warp
// with many short sequences does not finish last.
constexpr int kItemCost = 3;

// The tokens a sequence attends to, [first, len), and its groups: kGroup-aligned from first down.
struct Span {
    int first, len, base, groups;
};
WSM_HD Span span_of(int max_tokens, int window, int len) {
    Span s;
    s.len = len < 0 ? 0 : len > max_tokens ? max_tokens : len;
    s.first = window > 0 && s.len > window ? s.len - window : 0;
    s.base = s.first & ~(kGroup - 1);
    s.groups = (s.len - s.base + kGroup - 1) / kGroup;  // 0 for an empty sequence
    return s;
}

// The work in a line: sequence b's items follow one another, each kItemCost + groups long, so b begins at
// (prefix[b] + kItemCost * b) * hq with prefix the groups before b and hq the items of a sequence.  (At most
// 2^31 - 1 in all: checked by the host.)
WSM_HD int line_of(const int *prefix, int hq, int b) { return (prefix[b] + kItemCost * b) * hq; }

// Length of a warp's range.  (Rounded up without a sum: the line may be 2^31 - 1 long.)
WSM_HD int share_of(int total, int workers) {
    const int per = total / workers + (total % workers != 0 ? 1 : 0);
    return per < kMinShare ? kMinShare : per;
}

// The sequence at place `pos` of the line.
WSM_HD int seq_of(const int *prefix, int batch, int hq, int pos) {
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (line_of(prefix, hq, mid + 1) > pos) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Where range w begins: sequence, item and group.  A range that would begin within an item's fixed cost, or
// within a short item, begins with the item.
struct Place {
    int b, item, g;
};
WSM_HD Place place_of(const int *prefix, int batch, int hq, int total, int per, int w) {
    Place r;
    const long long pos = (long long)w * per;
    if (pos >= total) {
        r.b = batch;
        r.item = r.g = 0;
        return r;
    }
    r.b = seq_of(prefix, batch, hq, (int)pos);
    const int n = prefix[r.b + 1] - prefix[r.b], off = (int)pos - line_of(prefix, hq, r.b);
    r.item = off / (n + kItemCost);
    const int into = off - r.item * (n + kItemCost) - kItemCost;
    r.g = n <= kSnapGroups || into < 0 ? 0 : into;
    return r;
}
// Groups before a place.
WSM_HD int groups_before(const int *prefix, int hq, const Place &r, int batch) {
    if (r.b >= batch) return prefix[batch] * hq;
    return prefix[r.b] * hq + r.item * (prefix[r.b + 1] - prefix[r.b]) + r.g;
}

// Where range w leaves its partial of the item at place `at` of the line.  First slot: the range begins in this item;
// second: the item begins in the range.  (A range holds parts of one item of either kind at most.)
WSM_HD int slot_of(int w, int per, int at) { return w * 2 + ((long long)w * per >= at ? 0 : 1); }

// The ranges that hold an item of n groups, more than kSnapGroups, at place `at`: group g lies kItemCost + g past it.
struct Ranges {
    int first, last;
};
WSM_HD Ranges ranges_of(int at, int n, int per) { return Ranges{(at + kItemCost) / per, (at + kItemCost + n - 1) / per}; }

}  // namespace wsm
