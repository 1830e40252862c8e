// Host-side checks shared by the entry points of the decode and serving steps.
#pragma once

#include <stdint.h>

#include <cmath>

#include "cache_layout.h"
#include "tq_internal.h"

namespace {

constexpr int64_t MAX_TOKENS = int64_t(1) << 20;
constexpr int64_t MAX_BATCH = 65535;
constexpr int64_t MAX_HEADS = 1024;
constexpr int64_t MAX_SLOTS = int64_t(1) << 31;
// Positions of one sequence: key numbers plus a few steps stay below 2^31.
constexpr int64_t MAX_POSITIONS = int64_t(1) << 30;
constexpr int64_t MAX_PAGES = int64_t(1) << 26;
constexpr int64_t MAX_STRIDE = int64_t(1) << 40;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int launch_status(hipError_t e) { return e == hipSuccess ? TQ_OK : TQ_E_LAUNCH; }
bool valid_dtype(int t) { return t == TQ_F32 || t == TQ_BF16 || t == TQ_F16; }
uintptr_t size_of(int dtype) { return dtype == TQ_F32 ? 4 : 2; }
bool within(int64_t x, int64_t lo, int64_t hi) { return x >= lo && x <= hi; }

bool valid_strides(int64_t ts, int64_t hs)
{
    return within(ts, 0, MAX_STRIDE) && within(hs, 0, MAX_STRIDE);
}

// An output's rows must be apart: heads inside a token, or tokens inside a head.
bool apart(int64_t ts, int64_t hs, int64_t tokens, int64_t heads, int64_t D)
{
    if (!valid_strides(ts, hs))
        return false;
    if (heads == 0)
        return true;
    const bool one_head = heads == 1, one_token = tokens <= 1;
    if (one_head && one_token)
        return true;
    if (one_head)
        return ts >= D;
    if (one_token)
        return hs >= D;
    return (hs >= D && ts >= (heads - 1) * hs + D) || (ts >= D && hs >= (tokens - 1) * ts + D);
}

bool valid_cache(int64_t n_pages, int64_t page_size, int64_t kv_heads, int64_t D)
{
    return tq::cache_dim_ok(D) && tq::cache_page_ok(page_size) && within(kv_heads, 1, MAX_HEADS) &&
           within(n_pages, 1, MAX_PAGES) && n_pages * page_size < MAX_SLOTS;
}

// Whether bytes [a, a + na) and [b, b + nb) meet.
bool overlap(const void *a, int64_t na, const void *b, int64_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// An array of `rows` rows of n bytes, `stride` bytes apart (0: one for all).
struct Span {
    const void *p;
    int64_t stride, n, rows;
};

// Whether rows of the two have a byte in common; rows that lie between each other's
// (columns of one buffer) do not.
bool meet(const Span &a, const Span &b)
{
    if (a.rows < 1 || b.rows < 1 ||
        !overlap(a.p, (a.rows - 1) * a.stride + a.n, b.p, (b.rows - 1) * b.stride + b.n))
        return false;
    const int64_t d = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p);
    // Row j of b and a row at place `at` of a meet if at - b.n < d + j * b.stride < at
    // + a.n; the first j from `least` on that passes the lower end
    auto any = [&](int64_t at, int64_t least, int64_t rows) {
        const int64_t below = at - b.n - d;
        int64_t j = least;
        if (b.stride && below >= j * b.stride)
            j += (below - j * b.stride) / b.stride + 1;
        const int64_t place = d + j * b.stride;
        return j < rows && place > at - b.n && place < at + a.n;
    };
    if (a.stride == b.stride)                    // j: b's row less a's
        return any(0, 1 - a.rows, b.rows);
    for (int64_t i = 0; i < a.rows; i++)
        if (any(i * a.stride, 0, b.rows))
            return true;
    return false;
}

// The scratch region of a workspace of `bytes` bytes, or a status.
int scratch_of(void *workspace, size_t bytes, size_t need, uint32_t **counters, void **scratch)
{
    *counters = nullptr;
    *scratch = nullptr;
    if (need == 0)
        return TQ_OK;
    if (!workspace)
        return TQ_E_NULL;
    if (!aligned(workspace, 256))
        return TQ_E_ALIGN;
    if (bytes < need)
        return TQ_E_SHAPE;
    *counters = (uint32_t *)workspace;
    *scratch = (uint8_t *)workspace + TQ_NOALLOC_SCRATCH_BYTES;
    return TQ_OK;
}

}  // namespace
