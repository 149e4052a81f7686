// The table of pieces of many tensors (zero_build_pieces): host code only, no
// device calls.

#include <stdint.h>

#include <algorithm>
#include <new>
#include <utility>
#include <vector>

#include "zero_internal.h"

namespace {

typedef std::pair<uintptr_t, uintptr_t> Range;   // [first, second)

int64_t dtype_bytes(int dt)
{
    return dt == ZERO_BF16 || dt == ZERO_FP16 ? 2 : (dt == ZERO_FP32 ? 4 : 0);
}

// Elements by which an address is past a 16-byte boundary.
int64_t past_boundary(const void *p, int64_t bytes) { return (int64_t)((uintptr_t)p & 15u) / bytes; }

// Pieces of a tensor of n elements whose first is shorter by `past`.
int64_t pieces_of(int64_t n, int64_t past, int64_t max_piece)
{
    return n == 0 ? 1 : (n + past + max_piece - 1) / max_piece;
}

// Does any of `ranges` (sorted by start, disjoint) meet r?
bool meets(const std::vector<Range> &ranges, const Range &r)
{
    auto it = std::upper_bound(ranges.begin(), ranges.end(), r.first,
                               [](uintptr_t x, const Range &q) { return x < q.second; });
    return it != ranges.end() && it->first < r.second;
}

// A place may be exactly its own tensor; otherwise it meets no tensor and no
// other place.
int check_places(const void *const *src, const int *src_dt, void *const *dst, const int *dst_dt,
                 const int64_t *numels, int n)
{
    std::vector<Range> in, out;
    for (int t = 0; t < n; ++t) {
        if (numels[t] == 0)
            continue;
        const uintptr_t s = (uintptr_t)src[t], d = (uintptr_t)(dst ? dst[t] : src[t]);
        const int ddt = dst ? dst_dt[t] : src_dt[t];
        const uintptr_t sb = (uintptr_t)(numels[t] * dtype_bytes(src_dt[t]));
        const uintptr_t db = (uintptr_t)(numels[t] * dtype_bytes(ddt));
        if (s > UINTPTR_MAX - sb || d > UINTPTR_MAX - db)
            return ZERO_ERR_INVALID;
        out.emplace_back(d, d + db);
        if (s != d || ddt != src_dt[t])
            in.emplace_back(s, s + sb);
    }
    std::sort(out.begin(), out.end());
    for (size_t i = 1; i < out.size(); ++i)
        if (out[i].first < out[i - 1].second)
            return ZERO_ERR_ALIAS;
    // tensors in place are among the places, checked above; the others, which
    // may overlap one another, must meet no place at all
    for (const Range &r : in)
        if (meets(out, r))
            return ZERO_ERR_ALIAS;
    return ZERO_OK;
}

}  // namespace

extern "C" {

int zero_build_pieces(const void *const *src, const int *src_dt, void *const *dst,
                      const int *dst_dt, const int64_t *numels, int n_tensors, int64_t max_piece,
                      zero_piece *out, int64_t cap, int64_t *n_out)
{
    if (n_tensors < 0 || (n_tensors > 0 && (!src || !src_dt || !numels)) || !dst != !dst_dt)
        return ZERO_ERR_INVALID;
    if (max_piece <= 0 || max_piece % 64 != 0 || max_piece > (int64_t(1) << 24))
        return ZERO_ERR_INVALID;
    if (out && cap < 0)
        return ZERO_ERR_INVALID;
    int64_t total = 0;
    for (int t = 0; t < n_tensors; ++t) {
        if (numels[t] < 0 || numels[t] > ZERO_MAX_LEN - total ||
            (numels[t] > 0 && (!src[t] || (dst && !dst[t]))))
            return ZERO_ERR_INVALID;
        total += numels[t];
    }
    for (int t = 0; t < n_tensors; ++t) {
        // an unknown type has no size to divide by; it is refused below
        const int64_t sb = dtype_bytes(src_dt[t]), db = dst ? dtype_bytes(dst_dt[t]) : sb;
        if (numels[t] > 0 && ((sb && (uintptr_t)src[t] % (uintptr_t)sb) ||
                              (dst && db && (uintptr_t)dst[t] % (uintptr_t)db)))
            return ZERO_ERR_MISALIGNED;
    }
    for (int t = 0; t < n_tensors; ++t)
        if (!dtype_bytes(src_dt[t]) || (dst && !dtype_bytes(dst_dt[t])))
            return ZERO_ERR_UNSUPPORTED;
    // pieces in all, before the table itself: a tensor's first piece is shorter
    // by the elements its place is past a 16-byte boundary
    int64_t pieces_all = 0;
    for (int t = 0; t < n_tensors; ++t) {
        const int64_t db = dtype_bytes(dst ? dst_dt[t] : src_dt[t]);
        pieces_all += pieces_of(numels[t], past_boundary(dst ? dst[t] : src[t], db), max_piece);
    }
    if (pieces_all > ZERO_MAX_PIECES)
        return ZERO_ERR_INVALID;
    try {
        const int rc = check_places(src, src_dt, dst, dst_dt, numels, n_tensors);
        if (rc)
            return rc;
    } catch (const std::bad_alloc &) {
        return ZERO_ERR_CAPACITY;
    }

    int64_t count = 0;
    for (int t = 0; t < n_tensors; ++t) {
        const int ddt = dst ? dst_dt[t] : src_dt[t];
        const int64_t sb = dtype_bytes(src_dt[t]), db = dtype_bytes(ddt);
        char *d = (char *)(dst ? dst[t] : (void *)src[t]);
        const int64_t past = past_boundary(d, db);
        const int64_t pieces = pieces_of(numels[t], past, max_piece);
        int64_t at = 0;
        for (int64_t p = 0; p < pieces; ++p, ++count) {
            int64_t end = (p + 1) * max_piece - past;
            if (end > numels[t])
                end = numels[t];
            if (out && count < cap) {
                zero_piece &c = out[count];
                c.src = (const char *)src[t] + at * sb;
                c.dst = d + at * db;
                c.len = (int32_t)(end - at);
                c.tensor_id = t;
                c.tensor_pieces = p == 0 ? (int32_t)pieces : 0;
                c.src_dt = (int16_t)src_dt[t];
                c.dst_dt = (int16_t)ddt;
            }
            at = end;
        }
    }
    if (n_out)
        *n_out = count;
    if (out && count > cap)
        return ZERO_ERR_CAPACITY;
    return ZERO_OK;
}

}  // extern "C"
