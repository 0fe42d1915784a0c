// What the heads' kernels share: rows of a ragged batch, their places in a paged
// cache, and the values that its codes stand for.
#pragma once

#include "dq_stream.h"

namespace dq {

// A ragged batch's sequences (dq_seqs) and the cache's pages (dq_kv), as kernels see them.
struct Pages {
    const int* first;
    const int* length;
    const int* table;
    int seqs, ld, pages;
    int shift;              // tokens to a page: 1 << shift
    int heads;
};

// Where a row's token lies: its place t in its sequence (NOWHERE: a row of no
// sequence), and its page (-1: no token in the cache).
constexpr int NOWHERE = INT32_MIN;
struct Place {
    int t, page;
};

// The sequences' starts, ends and lengths, as a wave looks them up: up to 63 of
// them lie in its lanes after one round of loads; of more the lanes hold every
// step-th start.
struct Starts {
    int first, length, step;
};
__device__ __forceinline__ Starts starts_of(const Pages& p) {
    const int lane = threadIdx.x & 63, step = (p.seqs + 63) / 64, i = min(lane * step, p.seqs);
    return {p.first[i], p.length[min(i, p.seqs - 1)], step};
}

// A sequence: its rows [f0, f1) and its length; f0 > f1 - 1 for none.
struct Sequence {
    int b, f0, f1, length;
};
// The last sequence b with at(first[b], b) <= x, by the lanes (x is the wave's).
template <class At>
__device__ __forceinline__ Sequence sequence_of(const Pages& p, const Starts& s, long long x, At at) {
    const int lane = threadIdx.x & 63;
    int b = __popcll(__ballot(lane * s.step < p.seqs && at(s.first, lane * s.step) <= x)) - 1;
    if (b < 0) return {0, 0, 0, 0};
    if (s.step == 1 && p.seqs < 64)
        return {b, __builtin_amdgcn_readlane(s.first, b), __builtin_amdgcn_readlane(s.first, b + 1), __builtin_amdgcn_readlane(s.length, b)};
    b *= s.step;
    int n = min(s.step, p.seqs - b);                // the answer is one of b .. b + n - 1
    while (n > 1) {
        const int h = n >> 1;
        if (at(p.first[b + h], b + h) <= x) b += h, n -= h;
        else n = h;
    }
    return {b, p.first[b], p.first[b + 1], p.length[b]};
}

// Page `i` of sequence b, or -1 where the table has none or names none of the cache's.
__device__ __forceinline__ int page_of(const Pages& p, int b, int i) {
    if ((uint32_t)i >= (uint32_t)p.ld) return -1;
    const int page = p.table[(size_t)b * p.ld + i];
    return (uint32_t)page < (uint32_t)p.pages ? page : -1;
}

// The place of a wave's lanes' rows: `row` of its first lane, and one more for each `tpr` lanes.
__device__ __forceinline__ Place place_of(const Pages& p, const Starts& s, long long row, int tpr) {
    const int lane = threadIdx.x & 63;
    int b = 0, t = NOWHERE;
    for (int i = 0; i < 64; i += tpr, ++row) {      // (once where a row takes the wave)
        const Sequence q = sequence_of(p, s, row, [](int f, int) { return (long long)f; });
        const int at = row >= q.f0 && row < q.f1 ? (int)max((long long)q.length - q.f1 + row, -(1ll << 30)) : NOWHERE;
        const bool mine = lane >= i;
        b = mine ? q.b : b;
        t = mine ? at : t;
    }
    return {t, t < 0 ? -1 : page_of(p, b, t >> p.shift)};
}

// The cache's row of one token of one head.
__device__ __forceinline__ long long token_row(const Pages& p, Place at, int head) {
    return (((long long)at.page * p.heads + head) << p.shift) + (at.t & ((1 << p.shift) - 1));
}

// A scale code as the converters take it: 2^(e - 127), NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t e) { return __uint_as_float(e == 255 ? 0x7fc00000u : max(e << 23, 0x00400000u)); }

// The fp32 values of 8 codes (two words of E4M3, one of E2M1) under one scale code.
template <int BITS>
__device__ __forceinline__ void decode8_f32(const uint32_t* code, uint32_t e, float* v) {
    const float scale = scale_of(e);
    if constexpr (BITS == 8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(code[i], scale, false);
            const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(code[i], scale, true);
            v[4 * i] = a[0], v[4 * i + 1] = a[1], v[4 * i + 2] = b[0], v[4 * i + 3] = b[1];
        }
    } else {
        const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[0], scale, 0);
        const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[0], scale, 1);
        const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[0], scale, 2);
        const v2f d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[0], scale, 3);
        v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
    }
}

// Checks of a caller's cache and batch (heads.hip), and their sizes.
dq_status check_kv(const dq_kv* kv);
dq_status check_seqs(const dq_seqs* s);
int64_t kv_code_bytes(const dq_kv* kv);
int64_t kv_scale_bytes(const dq_kv* kv);
Pages pages_of(const dq_kv* kv, const dq_seqs* s);

}  // namespace dq
