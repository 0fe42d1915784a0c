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

// The sequence that holds `row`: the last b with first[b] <= row, -1 if none.
// All 64 lanes take part, each with a row of its own (`one`: the same row in the
// whole wave); up to 64 sequences cost one load.
__device__ __forceinline__ int sequence_of(const int* first, int seqs, long long row, bool one) {
    const int lane = threadIdx.x & 63, step = (seqs + 63) >> 6;
    const int f = lane * step < seqs ? first[lane * step] : INT32_MAX;
    int b;
    if (one) {
        b = __popcll(__ballot(f <= row)) - 1;
    } else {
        b = -1;
#pragma unroll
        for (int s = 32; s > 0; s >>= 1)
            if (__shfl(f, b + s, 64) <= row) b += s;
        if (b < 63 && __shfl(f, b + 1, 64) <= row) ++b;
    }
    if (b < 0 || step == 1) return b;
    int lo = b * step, n = min(step, seqs - lo);    // the answer is one of lo .. lo + n - 1
    while (n > 1) {
        const int h = n >> 1;
        if (first[lo + h] <= row) lo += h, n -= h;
        else n = h;
    }
    return lo;
}

// Page `i` of sequence b, or -1 where the table has none or names none of the cache's.
__device__ __forceinline__ int page_of(const Pages& p, int b, int i) {
    if ((uint32_t)i >= (uint32_t)p.ld) return -1;
    const int page = p.table[(size_t)b * p.ld + i];
    return (uint32_t)page < (uint32_t)p.pages ? page : -1;
}

__device__ __forceinline__ Place place_of(const Pages& p, long long row, bool one) {
    const int b = sequence_of(p.first, p.seqs, row, one);
    if (b < 0) return {NOWHERE, -1};
    const long long f1 = p.first[b + 1], len = p.length[b];
    if (row >= f1) return {NOWHERE, -1};
    const int t = (int)max(len - f1 + row, -(1ll << 30));
    return {t, t < 0 ? -1 : page_of(p, b, t >> p.shift)};
}

// The cache's row of one token of one head.
__device__ __forceinline__ long long token_row(const Pages& p, Place at, int head) {
    return (((long long)at.page * p.heads + head) << p.shift) + (at.t & ((1 << p.shift) - 1));
}

typedef float v2f __attribute__((ext_vector_type(2)));

// A scale code as the converters take it: 2^(e - 127), NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t e) { return __uint_as_float(e == 255 ? 0x7fc00000u : max(e << 23, 0x00400000u)); }

// The fp32 values of 16 codes under one scale code.
template <int BITS>
__device__ __forceinline__ void decode16(const uint32_t* code, uint32_t e, float* v) {
    const float scale = scale_of(e);
#pragma unroll
    for (int i = 0; i < (BITS == 8 ? 4 : 2); ++i) {
        if constexpr (BITS == 8) {
            const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(code[i], scale, false);
            const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(code[i], scale, true);
            v[4 * i] = a[0], v[4 * i + 1] = a[1], v[4 * i + 2] = b[0], v[4 * i + 3] = b[1];
        } else {
            const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[i], scale, 0);
            const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[i], scale, 1);
            const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[i], scale, 2);
            const v2f d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[i], scale, 3);
            v[8 * i] = a[0], v[8 * i + 1] = a[1], v[8 * i + 2] = b[0], v[8 * i + 3] = b[1];
            v[8 * i + 4] = c[0], v[8 * i + 5] = c[1], v[8 * i + 6] = d[0], v[8 * i + 7] = d[1];
        }
    }
}

// Checks of a caller's cache and batch (heads.hip), and their sizes.
dq_status check_kv(const dq_kv* kv);
dq_status check_seqs(const dq_seqs* s);
int64_t kv_code_bytes(const dq_kv* kv);
int64_t kv_scale_bytes(const dq_kv* kv);
Pages pages_of(const dq_kv* kv, const dq_seqs* s);

}  // namespace dq
