// Which slots a query row sees: shared by the kernels that attend with many
// tokens at once.
#pragma once

#include <stdint.h>

#include "gemv_decode.h"
#include "gemv_device.cuh"

namespace mbg {
namespace span {

// One sequence's new tokens, or (prefix) the whole batch's tokens over the
// slots that they share, which are looked up in the table's first row.
struct Seq {
    int b;       // row of the page table
    int q0, m;   // its tokens [q0, q0 + m)
    int n;       // its slots; prefix: the shared ones
};

// Clamps what lies out of range; `report`: says so (one thread).
__device__ __forceinline__ Seq seq_of(const SpanArgs &a, int b, bool report)
{
    Seq s;
    s.b = b;
    bool bad = false;
    if (a.prefix) {
        const int p = __ldg(a.prefix);
        s.q0 = 0;
        s.m = a.tokens;
        s.n = min(max(p, 0), static_cast<int>(a.kv.capacity));
        bad = s.n != p;
    } else {
        const int s0 = __ldg(a.starts + b), s1 = __ldg(a.starts + b + 1), n = __ldg(a.lengths + b);
        bad = s0 < 0 || s1 < s0 || s1 > a.tokens;
        s.q0 = bad ? 0 : s0;
        s.m = bad ? 0 : s1 - s0;
        s.n = min(max(n, 0), static_cast<int>(a.kv.capacity));
        bad = bad || s.n != n || s.m > s.n;  // tokens without a slot see nothing
    }
    if (bad && report) report_error(a.err, DEVERR_BAD_INDEX);
    return s;
}

// Starts that do not ascend: a sequence that begins below the start of one before
// it, the largest of which is `top`, has no tokens, so that no two sequences have
// the same.
__device__ __forceinline__ Seq seq_behind(const SpanArgs &a, int b, int &top)
{
    Seq s = seq_of(a, b, false);
    const int from = __ldg(a.starts + b);
    if (from < top) s.q0 = s.m = 0;
    top = max(top, from);
    return s;
}

// Token i of a sequence sees the slots t with lo <= t < hi or t < min(sinks,
// hi).
struct Seen {
    int lo, hi;
};

__device__ __forceinline__ Seen seen_by(const SpanArgs &a, const Seq &s, int i)
{
    Seen r;
    // its length with itself; prefix: what its sequence has in all
    int n = s.n - s.m + i + 1;
    if (a.prefix) n = min(__ldg(a.lengths + i), static_cast<int>(a.kv.capacity));
    n = max(n, 0);
    r.hi = min(n, s.n);
    r.lo = a.window > 0 && n > a.window ? n - a.window : 0;
    return r;
}

}  // namespace span
}  // namespace mbg
