// dq_attn_rows: attention of a few query rows over a cache of MX-FP8 or MX-FP4
// keys and values.
//
//   s_t = scale (q k_t), capped where asked;  y = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m)
//
// One pass over the cache with the running maximum m, the weights' sum and the
// weighted sum of the values, all fp32, rescaled when m grows.
//
// The rows of a sequence that share a key head (its query heads, times its rows)
// are the 16 columns of a matrix instruction, RB such blocks to a workgroup, so
// each key and value is read and decoded once for all of them.  A wave takes 32
// tokens at a time:
//   S^T [tokens][rows] = K Q^T: a lane decodes a run of its token's channels
//     straight from global memory into the instruction's operand (channels may
//     take any order that both operands share);
//   O^T [channels][rows] += V^T P^T: S^T's accumulators are P^T's operand as they
//     lie (the order of tokens is again free); V goes through the wave's own part
//     of LDS as bf16 and comes back transposed.
// The four waves of a workgroup take blocks of tokens in turn, without a
// barrier, and join at the end; a long cache is split over workgroups while the
// batch leaves the card room for that (launch_attn), and a second launch joins
// their sums in order.
//
// What bounds it (8 key heads of 128 channels, 40 query heads): HBM where the cache
// is long (64 sequences of 132 to 8192 tokens 119 us, 4.8 TB/s; one of 131072 and
// one of 81006 in 4 bits 55 us, 4.2, the kernel alone 51); where it is short,
// launch, a chain of loads (the batch, the pages, the tokens) and the join's launch
// (1 x 4097 12.4 us: 8.8 and 4.1 in the two kernels; 1 x 128, without a join, 6.1);
// from 16 rows that share a key head on the decoding and the weights' vector
// instructions (4 x 1024 rows over 8192 tokens 291 us, 472 TFLOP/s).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>
#include <type_traits>

#include "dq.h"
#include "dq_heads.h"

struct dq_attn {
    int device = 0;
    float* sums = nullptr;     // [unit][row block][16][D] sums, then [unit][row block][16][4] statistics, then tiles
};

namespace dq {
namespace {

// Parts of tiles (a tile: up to 16 RB rows that share a key head; a part: some of
// the tokens they see) that may meet in the workspace, and blocks of 16 rows to one.
constexpr int MAX_SLOTS = 2048, MAX_RB = 2;
constexpr size_t SUM_FLOATS = size_t(MAX_SLOTS) * MAX_RB * 16 * 128, STAT_FLOATS = size_t(MAX_SLOTS) * MAX_RB * 16 * 4;
// A tile in parts: how many (0 or 1: nothing to join), its rows, its sequence's
// first row and the rows before it, and the first part's slot.
struct TileInfo {
    int used, rows, f0, r0, slot, pad[3];
};
// In blocks of 32 tokens: what a tile costs beside them where a workgroup takes
// parts of several (its start and end take as long; 64 ragged sequences 116 us with
// 3, 4 and 8), the least that a workgroup takes (8: 1 x 8192 12.8 us, with 4 14.4,
// with 12 13.9; 1 x 1024 11.6, 10.4 and 12.9), and the widest page table whose tiles
// are taken whole, without a join.  The host does not know the lengths, so the
// table's width stands for them: 1 x 512 in a table of 512 10.1 us against 11.5 in two
// parts, 16 x 768 12.8 against 14.5 (1 x 768 12.6 against 11.6); of 1024 15.4 against
// 11.6.  1 x 128 takes 6.1 us in a table of up to 768 tokens, 8.3 in a wider one.
constexpr int TILE_COST = 4, LEAST_SHARE = 8, MOST_WHOLE = 24;
constexpr float LOG2E = 1.44269504088896340736f;

struct AttnArgs {
    const void* q;
    void* y;
    long long ldq, ldy;
    const uint8_t* codes[2];
    const uint8_t* scales[2];
    Pages pages;
    const int* prefix;
    int N, G;               // query rows; query heads to a key head
    int shares;             // workgroups that share a key head's tokens (0: one to a tile)
    int most;               // tiles of a key head at most
    int join;               // workgroups that join 16 rows of a tile
    long long block, window;
    float scale;            // of q k, for powers of 2; 1 with a cap
    float cap, cap_in;      // the cap (0: none), and scale / cap
    float* sums;
    float* stats;
    TileInfo* tiles;        // [key head][tile]
};

typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

// Maximum and sum over the four lanes that hold one row.
__device__ __forceinline__ float max_rows(float v) {
    const uint32_t w = __float_as_uint(v);
    const v2w a = __builtin_bit_cast(v2w, __builtin_amdgcn_permlane16_swap(w, w, false, false));
    const float m = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const uint32_t x = __float_as_uint(m);
    const v2w b = __builtin_bit_cast(v2w, __builtin_amdgcn_permlane32_swap(x, x, false, false));
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_rows(float v) {
    const uint32_t w = __float_as_uint(v);
    const v2w a = __builtin_bit_cast(v2w, __builtin_amdgcn_permlane16_swap(w, w, false, false));
    const uint32_t x = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
    const v2w b = __builtin_bit_cast(v2w, __builtin_amdgcn_permlane32_swap(x, x, false, false));
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
typedef const __attribute__((address_space(4))) int* Scalars;   // (nothing that the kernel writes)

__device__ __forceinline__ float power(float x) { return __builtin_amdgcn_exp2f(x); }
// What a sum is worth by a larger maximum.  Never 0, which would turn a sum that is infinite to NaN: below fp32's range its
// smallest number (a selection of infinite sums instead, here and in both joins, costs 1 row over 4097 tokens 6 %, 4 x 1024 rows 2 %).
__device__ __forceinline__ float worth(float from, float to) { return fmaxf(power(from - to), 0x1p-149f); }

// tanh: (1 - t) / (1 + t) with t = e^-2|x|, and its series where that cancels.
__device__ __forceinline__ float tanh_of(float x) {
    const float a = fabsf(x), t = power(-2.0f * LOG2E * a), x2 = x * x;
    const float far = copysignf((1.0f - t) * __builtin_amdgcn_rcpf(1.0f + t), x);
    const float near = x * (1.0f + x2 * (-0.33333333f + x2 * (0.13333333f + x2 * (-0.053968254f + x2 * 0.021869489f))));
    return a < 0.3f ? near : far;
}

// 8 codes (two words of E4M3, one of E2M1) as bf16, exactly.
template <int BITS>
__device__ __forceinline__ v8bf decode8(const uint32_t* w, float scale) {
    v2b p[4];
    if constexpr (BITS == 8) {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], scale, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], scale, true);
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 0);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 1);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 2);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 3);
    }
    return v8bf{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// An address that is the same in the whole wave, in scalar registers.
typedef const __attribute__((address_space(1))) uint8_t* Bytes;
__device__ __forceinline__ Bytes scalar(const uint8_t* p) {
    const uint64_t v = (uint64_t)(uintptr_t)p;
    return (Bytes)(uintptr_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                              (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}
template <int N>
__device__ __forceinline__ void load_words(Bytes p, uint32_t* w) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const v4w v = *(const __attribute__((address_space(1))) v4w*)(p + 4 * i);
            w[i] = v[0], w[i + 1] = v[1], w[i + 2] = v[2], w[i + 3] = v[3];
        }
    } else {
        const v2w v = *(const __attribute__((address_space(1))) v2w*)p;
        w[0] = v[0], w[1] = v[1];
    }
}

// Of a word's scale codes those so large (246 or more) that a value may pass bf16's range, or NaN: by their highest bits.
__device__ __forceinline__ uint32_t large_scales(uint32_t w) {
    return ((w & 0x7f7f7f7fu) + 0x0a0a0a0au) & w & 0x80808080u;   // (carries into the sign's place, which it has)
}

// One wave's 32 tokens, as they are held in the cache.
template <int BITS, int D>
struct Tokens {
    static constexpr int KW = D / 4 * BITS / 32;    // words of codes a lane holds of a key (D / 4 channels)
    static constexpr int VP = D / 32;               // 16-channel pieces of values a lane holds
    static constexpr int VW = 16 * BITS / 32;
    uint32_t k[2][KW], v[VP][VW];
    uint32_t ks[2], vs[VP];

    // Whether one of the lane's values may be infinite, or has a NaN scale.
    __device__ __forceinline__ bool large() const {
        uint32_t large = 0;
#pragma unroll
        for (int i = 0; i < VP; ++i) large |= large_scales(vs[i]);
        return large != 0;
    }
    // Whether one has a NaN code.
    __device__ __forceinline__ bool nan_code() const {
        uint32_t nan = 0;
        if constexpr (BITS == 8) {
#pragma unroll
            for (int i = 0; i < VP; ++i)
#pragma unroll
                for (int j = 0; j < VW; ++j) nan |= (v[i][j] & 0x7f7f7f7fu) + 0x01010101u;   // (0x7f: carries into the sign's place)
        }
        return (nan & 0x80808080u) != 0;
    }
};
// Of 8 bf16 values those that are not finite put to zero ...
__device__ __forceinline__ v8bf finite(v8bf v) {
    v4w w = __builtin_bit_cast(v4w, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] &= ~(((((w[i] & 0x7f807f80u) + 0x00800080u) >> 15) & 0x00010001u) * 0xffffu);   // (a full exponent carries into the sign's place)
    return __builtin_bit_cast(v8bf, w);
}
// ... or put to what counts them, and zero for the rest: 1 for +infinity, 64 for -infinity, 65 for NaN (of 32 tokens: sums are exact, and
// each of the first two is below 64 times).
__device__ __forceinline__ v8bf counted(v8bf v) {
    v4w w = __builtin_bit_cast(v4w, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = (((w[i] & 0x7f807f80u) + 0x00800080u) >> 15) & 0x00010001u;
        const uint32_t nan = (((w[i] & 0x7fff7fffu) + 0x007f007fu) >> 15) & 0x00010001u, sign = w[i] >> 15;
        w[i] = nan * 0x4282u | (c & ~nan & sign) * 0x4280u | (c & ~nan & ~sign) * 0x3f80u;
    }
    return __builtin_bit_cast(v8bf, w);
}

// Four channels of a row: the weighted values over the weights' sum, or zero where no token was seen.
__device__ __forceinline__ void store4(float* y, v4f o, float sum, bool any) {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = any ? o[e] / sum : 0.0f;
    *(v4f*)y = o;
}
__device__ __forceinline__ void store4(uint16_t* y, v4f o, float sum, bool any) {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = any ? o[e] / sum : 0.0f;
    const v2b a{(__bf16)o[0], (__bf16)o[1]}, b{(__bf16)o[2], (__bf16)o[3]};
    *(v2w*)y = v2w{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
}

// Tokens that a sequence's row of the page table reaches.
__device__ __forceinline__ long long reach(const Pages& p) { return min((long long)p.ld << p.shift, (1ll << 31) - 64); }

// The inclusive sum over the wave's lanes, in order.
template <class V>
__device__ __forceinline__ V scan(V v) {
    const auto moved = [](V x, auto ctrl, auto rows) {
        constexpr int C = decltype(ctrl)::value, R = decltype(rows)::value;
        return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), C, R, 0xF, true));
    };
    using std::integral_constant;
    const integral_constant<int, 0xF> all{};
    v += moved(v, integral_constant<int, 0x111>{}, all);   // 1, 2, 4 and 8 lanes down in each row of 16
    v += moved(v, integral_constant<int, 0x112>{}, all);
    v += moved(v, integral_constant<int, 0x114>{}, all);
    v += moved(v, integral_constant<int, 0x118>{}, all);
    v += moved(v, integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});   // a row's last lane to the next row, in every other row
    v += moved(v, integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});   // the first half's last lane to the second half
    return v;
}

// One workgroup's work for one tile: blocks c0 .. c1 - 1 of the tokens that tile
// `tile` of sequence b sees.
struct Work {
    int b, f0, f1, length, tile, c0, c1;
    int parts, slot, number;  // of the tile: its parts; this one's slot; its number
    bool head;                // its first part
};
// Up to 64 sequences: a lane holds one.  Their tiles stand in a row, each as long
// as the blocks of tokens that it sees at most, and a workgroup takes an equal
// stretch of the row, a share.  Where the card holds a workgroup for each part, a
// tile's length is rounded up to whole shares, so that no workgroup meets two
// tiles (16 sequences of 1024 tokens 15.1 us against 16.7, 8 12.2 against 14.1, one of
// 8192 12.8 against 17.7).  Otherwise TILE_COST is added to it, and a workgroup takes
// a part of a long tile or several short ones, whatever the lengths (64 sequences of
// 132 to 8192 tokens 116 us; in three parts to each tile, when this was chosen, 144
// against 111).
struct Batch64 {
    int f0, f1, length, tiles;
    int cost, upto, tiles_upto;     // of one tile; of this sequence's and earlier tiles together
    int parts;                      // of a tile, where they are whole shares
};
template <int TR>
__device__ __forceinline__ Batch64 batch_of(const AttnArgs& a) {
    const Pages& p = a.pages;
    const int lane = threadIdx.x & 63, i = min(lane, p.seqs - 1);
    const int first = p.first[i], next = p.first[i + 1], len = p.length[i], keep = a.prefix ? a.prefix[i] : 0;
    Batch64 x;
    x.f0 = min(max(first, 0), a.N), x.f1 = min(max(next, x.f0), a.N), x.length = max(len, 0);
    x.tiles = lane < p.seqs ? ((x.f1 - x.f0) * a.G + TR - 1) / TR : 0;
    const long long L = min((long long)x.length, reach(p));
    long long tokens = L;                                  // that a tile's rows see, or a few more
    if (a.block && a.window) tokens = min(L, min(L, a.window + a.block + TR) + min((long long)max(keep, 0), L) + 64);
    x.cost = max((int)((tokens + 31) / 32) + (a.window ? 1 : 0), 1);   // (a tile that sees nothing is answered, too)
    x.tiles_upto = scan(x.tiles);
    x.upto = 0;
    x.parts = 0;
    return x;
}
__device__ __forceinline__ Batch64 of_lane(const Batch64& x, int b) {
    const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, b); };
    return {of(x.f0), of(x.f1), of(x.length), of(x.tiles), of(x.cost), of(x.upto), of(x.tiles_upto), 0};
}
// One tile to a workgroup: the u-th; tile -1 past the last.  (Of more than 64
// sequences, b's are numbered from floor(first[b] G / TR) + b on, which leaves
// each as many as it needs.)
template <int TR>
__device__ __forceinline__ Work whole_tile(const AttnArgs& a, int u) {
    const Pages& p = a.pages;
    const auto one = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    if (p.seqs <= 64) {
        const Batch64 x = batch_of<TR>(a);
        const int b = (int)__popcll(__ballot(x.tiles_upto <= u));
        if (b > 63) return {0, 0, 0, 0, -1, 0, 0, 1, 0, 0, true};
        const Batch64 y = of_lane(x, b);
        return {b, y.f0, y.f1, y.length, u - y.tiles_upto + y.tiles, 0, INT32_MAX, 1, 0, 0, true};
    }
    const auto base_of = [&](int first, int i) { return min(max(first, 0), a.N) * a.G / TR + i; };
    const Sequence q = sequence_of(p, starts_of(p), u, [&](int f, int i) { return (long long)base_of(f, i); });
    const int f0 = min(max(q.f0, 0), a.N), f1 = min(max(q.f1, f0), a.N);
    return {one(q.b), one(f0), one(f1), one(max(q.length, 0)), one(u - base_of(q.f0, q.b)), 0, INT32_MAX, 1, 0, 0, true};
}

// Waves to a SIMD that the registers are kept for (one more spills the sums).
constexpr int waves_of(bool f32, int D, int RB) { return RB == 1 ? (f32 ? (D == 64 ? 3 : 2) : D == 64 ? 4 : 3) : f32 && D == 128 ? 1 : 2; }

template <class T, int BITS, int D, int RB>
__global__ __launch_bounds__(256, waves_of(sizeof(T) == 4, D, RB)) void k_attn(AttnArgs a) {
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int QP = F32 ? 3 : 1, PP = F32 ? 3 : 2;      // bf16 parts of q and of the weights
    constexpr int TR = 16 * RB, CB = D / 16, NJ = D / 32;  // rows of a tile; blocks of 16 channels; steps of 32 channels
    constexpr int LPR = D / 16;                            // lanes to a token's values, 16 channels each
    using Tok = Tokens<BITS, D>;
    __shared__ __attribute__((aligned(16))) uint8_t lds[4][64 * D];   // a wave's V [32][D] bf16, then its sums [16][D] fp32
    __shared__ float stat[4][3][TR];
    __shared__ Batch64 batch[64];
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int u = blockIdx.x, head = blockIdx.y;
    // (what is the same in the whole wave is kept in scalar registers)
    const auto one = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    // (the arguments' cache lines, all at once)
    asm volatile("" ::"s"(a.q), "s"(a.scales[1]), "s"(a.prefix), "s"(a.tiles));
    Work work;
    int pos = 0, end = 0, share = 0;                       // of the row of tiles: what is left to this workgroup
    int lead = TILE_COST;                                  // of a tile's length, before its first block
    if (a.shares) {
        Batch64 x = batch_of<TR>(a);
        const int tiles = __builtin_amdgcn_readlane(x.tiles_upto, 63);
        // (more tiles than there can be: first_dev is not ascending, and nothing is done)
        const bool fit = tiles <= a.most;
        if (u >= (fit ? tiles : 0) && u < a.most && tid == 0) a.tiles[(size_t)head * a.most + u].used = 0;   // (no tile of that number)
        if (!fit) return;
        const auto last = [](int v) { return __builtin_amdgcn_readlane(v, 63); };
        // whole shares: the least, or a few sizes from an equal division on
        share = LEAST_SHARE;
        int parts = (x.cost + LEAST_SHARE - 1) / LEAST_SHARE;
        x.upto = scan(x.tiles * parts);
        if (last(x.upto) > a.shares) {
            const int sum = last(scan(x.tiles * x.cost));
            share = one((int)(((uint32_t)sum + a.shares - 1) / (uint32_t)a.shares));
#pragma unroll 1
            for (int i = 0;; ++i, share += 4) {
                parts = (int)(((uint32_t)x.cost + share - 1) / (uint32_t)share);
                x.upto = scan(x.tiles * parts);
                if (i == 4 || last(x.upto) <= a.shares) break;
            }
        }
        if (last(x.upto) <= a.shares) {
            x.cost = parts * share, x.upto *= share, lead = 0;
        } else {
            x.cost += TILE_COST, x.upto = scan(x.tiles * x.cost);
            share = one((int)(((uint32_t)last(x.upto) + a.shares - 1) / (uint32_t)a.shares));
        }
        const int total = last(x.upto);
        x.parts = parts;
        batch[tid & 63] = x;                                   // (every wave the same)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        pos = (int)min((long long)u * share, (long long)total), end = min(total, pos + share);
    } else {
        work = whole_tile<TR>(a, u);
    }
    for (;;) {
        int lane = tid & 63;
        asm volatile("" : "+v"(lane));                         // (what goes by the lane is formed for each tile, not kept over all of them)
        const int r16 = lane & 15, g = lane >> 4;
        if (a.shares) {
            if (pos >= end) return;
            const int b = (int)__popcll(__ballot(batch[lane].upto <= pos));
            const Batch64 x = batch[b];
            const int tiles = one(x.tiles), cost = one(x.cost), begin = one(x.upto) - tiles * cost, tile = tiles > 1 ? (pos - begin) / cost : 0;
            const int first = begin + tile * cost, from = pos - first, to = min(cost, from + end - pos), number = one(x.tiles_upto) - tiles + tile;
            pos += to - from;
            work = {b, one(x.f0), one(x.f1), one(x.length), tile, max(from - lead, 0), max(to - lead, 0), 0, u + number, number, false};
            if (work.c0 >= work.c1) continue;                  // (the part that stands for the tile's cost)
            if (!lead) {
                work.parts = one(x.parts), work.head = from == 0;
            } else {
                const int head_of = (first + lead) / share;    // the workgroup of its first block
                work.parts = (first + cost - 1) / share - head_of + 1;
                work.head = u == head_of;
            }
        }
        const int b = one(work.b), f0 = one(work.f0), f1 = one(work.f1), length = one(work.length);
        const int L = (int)min((long long)length, reach(a.pages));
        const int rows = (f1 - f0) * a.G, r0 = one(work.tile) * TR;
        if (r0 < 0 || r0 >= rows) return;                      // (no such tile; of shares there is none)
        const int pf = a.block && a.prefix ? min(max(((Scalars)(uintptr_t)a.prefix)[b], 0), L) : 0;
        const int used = one(work.parts);
        if (a.shares && work.head && tid == 0)
            a.tiles[(size_t)head * a.most + work.number] = TileInfo{used, min(rows - r0, TR), f0, r0, work.slot, {0, 0, 0}};

        // ---- what each row sees: [lo, hi) and [0, pf)
        const int t0 = length - (f1 - f0);                     // the first row's place
        const auto sees = [&](int r, int* lo, int* hi) {       // r: packed row
            *lo = 0, *hi = L;
            if (!a.block) return;
            const int t = t0 + (int)((uint32_t)r / (uint32_t)a.G);
            // the end of the row's block (0 before the first token)
            const long long e = t < 0 ? 0 : a.block == 1 ? t + 1ll : (long long)((uint32_t)t / (uint32_t)a.block + 1) * a.block;
            *hi = (int)min(e, (long long)L);
            if (a.window) *lo = (int)min(max(e - a.window, 0ll), (long long)L);
        };
        int lo0, hi0, lo1, hi1;                                // of the tile's first and last row
        sees(r0, &lo0, &hi0);
        sees(min(rows, r0 + TR) - 1, &lo1, &hi1);
        lo0 = one(lo0), hi0 = one(hi0), lo1 = one(lo1), hi1 = one(hi1);
        // blocks of 32 tokens that some row sees: [0, na) and [b0, b0 + nb)
        int na = (pf + 31) >> 5, b0 = lo0 >> 5, nb = hi1 > lo0 ? ((hi1 + 31) >> 5) - b0 : 0;
        if (na >= b0) nb = max(b0 + nb, na), b0 = 0, na = 0;
        const int blocks = na + nb;
        const int c_end = min(blocks, one(work.c1));

        // ---- the cache
        const auto token0 = [&](int c) { return (c < na ? c : c - na + b0) << 5; };
        // Pages of a block's two halves, as the table has them (places past its end:
        // its last entry; a block past the part's last: the last's), and those that
        // are the cache's, or -1.  Scalar loads: a wave's wait for them does not wait for the cache's.
        struct Two {
            int p[2];
        };
        const Scalars table = (Scalars)(uintptr_t)(a.pages.table + (size_t)b * a.pages.ld);
        const auto near = [&](int c) { return max(min(c, c_end - 1), 0); };
        const auto entries = [&](int c) {
            const int t = token0(near(c));
            return Two{{table[min(t >> a.pages.shift, a.pages.ld - 1)], table[min((t + 16) >> a.pages.shift, a.pages.ld - 1)]}};
        };
        const auto pages_at = [&](int c, Two e) {
            const int t = token0(near(c));
            return Two{{t < L && (uint32_t)e.p[0] < (uint32_t)a.pages.pages ? e.p[0] : -1,
                        t + 16 < L && (uint32_t)e.p[1] < (uint32_t)a.pages.pages ? e.p[1] : -1}};
        };
        const int mask = (1 << a.pages.shift) - 1;
        // A load's address is a block's, which is scalar, and an offset that is the
        // lane's.  Scale codes come as the aligned word that holds a row's (with D 64 two rows').
        constexpr int RC = D * BITS / 8, RS = D / 32;          // bytes of a row's codes and scale codes
        const auto scale_in = [](uint32_t word, int row, int group) {
            return scale_of(word >> (8 * (D == 128 ? group : 2 * (row & 1) + group)) & 0xff);
        };
        const uint32_t key_at = r16 * RC + g * (Tok::KW * 4), key_scale_at = r16 * RS & ~3;
        const uint32_t value_at = lane / LPR * RC + lane % LPR * (Tok::VW * 4), value_scale_at = lane / LPR * RS & ~3;
        Tok x;
        const auto row_of = [&](int c, Two pg, int h) {        // the cache's row of a half's first token (in page 0 where there is none)
            return (((long long)max(pg.p[h], 0) * a.pages.heads + head) << a.pages.shift) + ((token0(near(c)) + 16 * h) & mask);
        };
        const auto load_keys = [&](int c, Two pg) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const long long row = row_of(c, pg, h);
                load_words<Tok::KW>(scalar(a.codes[0] + row * RC) + key_at, x.k[h]);
                x.ks[h] = *(const __attribute__((address_space(1))) uint32_t*)(scalar(a.scales[0] + row * RS) + key_scale_at);
            }
        };
        const auto load_values = [&](int c, Two pg) {
#pragma unroll
            for (int i = 0; i < Tok::VP; ++i) {                // piece i: token (64 / LPR) i + lane / LPR
                const long long row = row_of(c, pg, (64 / LPR) * i < 16 ? 0 : 1) + (64 / LPR) * i % 16;
                load_words<Tok::VW>(scalar(a.codes[1] + row * RC) + value_at, x.v[i]);
                x.vs[i] = *(const __attribute__((address_space(1))) uint32_t*)(scalar(a.scales[1] + row * RS) + value_scale_at);
            }
        };

        v4f acc[RB][CB];
        float m[RB], l[RB];
        uint32_t seen = 0;                                     // row blocks whose row (of this lane) saw a token
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            m[i] = -INFINITY, l[i] = 0.0f;
#pragma unroll
            for (int c = 0; c < CB; ++c) acc[i][c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }

        // V [32][D] bf16: 32 bytes (16 channels) of a token at slot c16 ^ its own, so
        // that the transposing reads' 8 rows of 32 bytes meet 64 banks
        uint8_t* const mine = lds[w];                          // (64 D bytes: the slots' exclusive or stays inside)
        const auto place_v = [&](int tok, int c16) {
            const int s = D == 128 ? tok & 7 : (tok >> 1) & 3;
            return tok * (2 * D) + ((c16 ^ s) << 5);
        };
        const auto place_values = [&](auto change) {
#pragma unroll
            for (int i = 0; i < Tok::VP; ++i) {
                const int tok = (64 / LPR) * i + lane / LPR, c16 = lane % LPR;
                const float scale = scale_in(x.vs[i], tok, c16 / 2);
                uint4* to = (uint4*)(mine + place_v(tok, c16));
                to[0] = __builtin_bit_cast(uint4, change(decode8<BITS>(x.v[i], scale)));
                to[1] = __builtin_bit_cast(uint4, change(decode8<BITS>(x.v[i] + BITS / 4, scale)));
            }
        };
        const auto read_v = [&](int cb) {                      // V^T: channels 16 cb + lane % 16, tokens 4 g .. and 16 + 4 g ..
            const int tok = 4 * g + (r16 >> 2), in = (r16 & 3) * 8;
            const uint8_t* from = mine + ((place_v(tok, 0) + in) ^ (cb << 5));
            const v4s p = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)from);
            const v4s q = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(from + 32 * D));   // (16 tokens on)
            typedef short v8s __attribute__((ext_vector_type(8)));
            return __builtin_bit_cast(v8bf, v8s{p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3]});
        };

        const int c_first = one(work.c0) + w;
        Two pg = pages_at(c_first, entries(c_first)), later = entries(c_first + 4);
        load_keys(c_first, pg);
        load_values(c_first, pg);

        // ---- q as the second operand: lane (row, g), channels (D / 4) g + 8 j ..
        v8bf q[RB][QP][NJ];
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const uint32_t r = min(r0 + 16 * i + r16, rows - 1), n = r / (uint32_t)a.G;
            const T* p = (const T*)a.q + (long long)(f0 + n) * a.ldq + (head * a.G + (int)(r - n * a.G)) * D + (D / 4) * g;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                if constexpr (F32) {
                    float v[8];
                    Stream<float>::load(p + 8 * j, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const __bf16 h = (__bf16)v[e];
                        const float rest = v[e] - (float)h;
                        const __bf16 m = (__bf16)rest;
                        q[i][0][j][e] = h;
                        q[i][1][j][e] = m;
                        q[i][2][j][e] = (__bf16)(rest - (float)m);
                    }
                    // (an infinite value has no rest)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if ((__float_as_uint(v[e]) & 0x7f800000u) == 0x7f800000u || fabsf((float)q[i][0][j][e]) > 3.4e38f) {
                            q[i][1][j][e] = (__bf16)0.0f;
                            q[i][2][j][e] = (__bf16)0.0f;
                        }
                } else {
                    q[i][0][j] = __builtin_bit_cast(v8bf, get16(p + 8 * j));
                }
            }
        }

        int lo[RB], hi[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) sees(min(r0 + 16 * i + r16, rows - 1), &lo[i], &hi[i]);

        for (int c = c_first; c < c_end;) {
            // (The next block's keys are loaded as soon as this one's are used, its
            // values too: no registers for two blocks.  Past the last block the last
            // is loaded again: with a branch there the waits, which count loads,
            // would have to assume that there were none.)
            const Two here = pg;
            pg = pages_at(c + 4, later);
            later = entries(c + 8);
            const int t = token0(c);
            // ---- scores
            v4f s[RB][2];
            const auto score = [&](auto rest) {                // (rest: of a key what q's lower parts meet)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float scale = scale_in(x.ks[h], r16, D / 4 * g / 32);
#pragma unroll
                    for (int i = 0; i < RB; ++i) s[i][h] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const v8bf k = decode8<BITS>(x.k[h] + j * (BITS / 4), scale);
#pragma unroll
                        for (int i = 0; i < RB; ++i)
#pragma unroll
                            for (int p = QP - 1; p >= 0; --p)
                                s[i][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p ? rest(k) : k, q[i][p][j], s[i][h], 0, 0, 0);
                    }
                }
            };
            score([](v8bf k) { return k; });
            // (An infinite key's product is infinite by the sign of q's first part; the others may be 0 or of the other
            // sign.  Once more, since that is rare: fp32 rows take up to 7 % longer with a choice ahead, 2 % with this.)
            if (F32 && __builtin_expect(__ballot((large_scales(x.ks[0]) | large_scales(x.ks[1])) != 0) != 0, 0))
                score([](v8bf k) { return finite(k); });
            load_keys(c + 4, pg);
            // ---- values into LDS
            const bool all = here.p[0] >= 0 && here.p[1] >= 0 && ((t >= lo1 && t + 32 <= hi0) || t + 32 <= pf);   // every row sees every token
            // (in the product a value that is not finite would reach rows that do not see it, times 0, and an infinite
            // one turn to NaN by a weight's part that is 0 or negative)
            const bool odd = __ballot(x.large()) != 0 || (!all && __ballot(x.nan_code()) != 0);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (!odd) place_values([](v8bf v) { return v; });
            else place_values([](v8bf v) { return finite(v); });
            load_values(c + 4, pg);
            // ---- weights
            v8bf pw[RB][PP];
            uint32_t vis[RB];
            float grown[RB];                                   // what the sums so far are worth by the new maximum
            const auto weigh = [&](auto masked) {
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    float e[8];
                    vis[i] = 0xff;
                    if constexpr (decltype(masked)::value) {
                        vis[i] = 0;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int tok = t + 16 * (j >> 2) + 4 * g + (j & 3);
                            const bool on = ((tok >= lo[i] && tok < hi[i]) || tok < pf) && here.p[j >> 2] >= 0;
                            vis[i] |= on ? 1u << j : 0u;
                        }
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 8; ++j) e[j] = s[i][j >> 2][j & 3];
                    if (a.cap > 0.0f) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) e[j] = a.cap * LOG2E * tanh_of(e[j] * a.cap_in);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if constexpr (decltype(masked)::value) e[j] = vis[i] >> j & 1 ? e[j] : -INFINITY;
                        top = fmaxf(top, e[j]);
                    }
                    if (vis[i]) seen |= 1u << i;
                    top = max_rows(top) * a.scale;             // (1 with a cap)
                    const float mn = fmaxf(m[i], top);
                    grown[i] = mn == m[i] ? 1.0f : worth(m[i], mn);   // (also where both are infinite, whose sums are NaN by the weights)
                    m[i] = mn;
                    l[i] *= grown[i];
                    const float at = m[i] == -INFINITY ? 0.0f : m[i];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float p = power(__builtin_fmaf(e[j], a.scale, -at));
                        l[i] += p;
                        // The weight in bf16 parts, exact but for 2^-16 of it where y is bf16 (one part alone is off by 2^-8, as much
                        // as y's own rounding where the values' signs differ), and for 2^-24 where it is fp32.  A second part
                        // costs 1 row over 4097 tokens 2 %, 64 sequences 1 %, 4 x 1024 rows 11 %; a third 2 to 9 % of fp32 rows.
                        float rest = p;
#pragma unroll
                        for (int n = 0; n < PP; ++n) {
                            const __bf16 part = (__bf16)rest;
                            pw[i][n][j] = part;
                            rest -= (float)part;
                        }
                    }
                }
            };
            if (all) weigh(std::false_type{});
            else weigh(std::true_type{});
#pragma unroll
            for (int i = 0; i < RB; ++i)
                if (__ballot(grown[i] != 1.0f)) {
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) acc[i][cb] *= grown[i];
                }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            // ---- O^T += V^T P^T
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) {
                const v8bf v = read_v(cb);
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int p = PP - 1; p >= 0; --p) acc[i][cb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, pw[i][p], acc[i][cb], 0, 0, 0);
            }
            if (odd) {
                // the rows that do see a value that is not finite: counted as ones times ones, whatever its weight
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                load_values(c, here);
                place_values([](v8bf v) { return counted(v); });
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    v8bf on;
#pragma unroll
                    for (int j = 0; j < 8; ++j) on[j] = (__bf16)(vis[i] >> j & 1 ? 1.0f : 0.0f);
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) {
                        const v4f n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(read_v(cb), on, v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = (int)n[e];
                            acc[i][cb][e] += k & 63 ? INFINITY : 0.0f;
                            acc[i][cb][e] -= k >> 6 ? INFINITY : 0.0f;
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                load_values(c + 4, pg);
            }
            c += 4;
        }

        // ---- the four waves' sums, a block of rows at a time: thread (row, its D / 16 channels)
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const float sum = sum_rows(l[i]);
            const uint64_t s = __ballot(seen >> i & 1);
            const bool any = ((s | s >> 16 | s >> 32 | s >> 48) >> r16) & 1;
            if (g == 0) {
                stat[w][0][16 * i + r16] = m[i];
                stat[w][1][16 * i + r16] = sum;
                stat[w][2][16 * i + r16] = any ? 1.0f : 0.0f;
            }
        }
        constexpr int CT = D / 16, Q4 = CT / 4;                // channels of a thread, in pieces of 4
        const int row = tid >> 4, ch = (tid & 15) * CT;
        const size_t unit = ((size_t)head * (a.shares + a.most) + work.slot) * RB;
        const auto finish = [&](int i, const v4f* o, float sum, bool any) {
            const uint32_t r = r0 + 16 * i + row, n = r / (uint32_t)a.G;
            if ((int)r >= rows) return;
            T* y = (T*)a.y + (long long)(f0 + n) * a.ldy + (head * a.G + (int)(r - n * a.G)) * D + ch;
#pragma unroll
            for (int p = 0; p < Q4; ++p) store4(y + 4 * p, o[p], sum, any);
        };
        // (16-byte piece c of a row lies at c ^ row, so the lanes' stores and loads meet all banks)
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            __syncthreads();
            v4f* o = (v4f*)mine;
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) o[r16 * (D / 4) + ((4 * cb + g) ^ r16)] = acc[i][cb];
            __syncthreads();
            float top = -INFINITY, sum = 0.0f, any = 0.0f;
#pragma unroll
            for (int p = 0; p < 4; ++p) top = fmaxf(top, stat[p][0][16 * i + row]);
            v4f out[Q4];
#pragma unroll
            for (int p = 0; p < Q4; ++p) out[p] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float mp = stat[p][0][16 * i + row], f = mp == -INFINITY ? 1.0f : worth(mp, top);
                sum += f * stat[p][1][16 * i + row];
                any = fmaxf(any, stat[p][2][16 * i + row]);
                const v4f* from = (const v4f*)lds[p] + row * (D / 4);
#pragma unroll
                for (int j = 0; j < Q4; ++j) out[j] += f * from[((ch >> 2) + j) ^ row];
            }
            if (used == 1) {
                finish(i, out, sum, any > 0.0f);
            } else {
                if (r0 + 16 * i + row >= rows) continue;
#pragma unroll
                for (int j = 0; j < Q4; ++j) *(v4f*)(a.sums + ((unit + i) * 16 + row) * D + ch + 4 * j) = out[j];
                if ((tid & 15) == 0) *(v4f*)(a.stats + ((unit + i) * 16 + row) * 4) = v4f{top, sum, any, 0.0f};
            }
        }
        if (!a.shares) return;
        __syncthreads();                                       // (the sums in LDS are read)
    }
}

// The sums of a tile's parts: a wave to a row, 16 bytes of a part to a lane, so
// 256 / D parts to a load, and U loads on their way at once.
template <class T, int D, int RB>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
    constexpr int LP = D / 4, PL = 64 / LP, U = 8;         // lanes to a part, parts to a load
    const int lane = threadIdx.x & 63, head = blockIdx.y;
    const int by = a.join * RB, first = (int)(blockIdx.x % by) * (16 / a.join);   // of the tile's rows
    const TileInfo info = a.tiles[(size_t)head * a.most + blockIdx.x / by];
    if (info.used < 2) return;
    for (int row = first + (threadIdx.x >> 6); row < min(info.rows, first + 16 / a.join); row += 4) {
        const size_t unit = ((size_t)head * (a.shares + a.most) + info.slot) * RB + (row >> 4), step = RB;
        const auto at = [&](int p) { return (unit + p * step) * 16 + (row & 15); };
        // 64 parts at a time, a lane holding one's statistics, with the maximum and the sums so far rescaled
        float top = -INFINITY, sum = 0.0f, any = 0.0f;
        v4f out{0.0f, 0.0f, 0.0f, 0.0f};
        const int sub = lane / LP, ch = 4 * (lane % LP);
        for (int p64 = 0; p64 < info.used; p64 += 64) {
            const int n = min(info.used - p64, 64);
            v4f from[U];
            const auto fetch = [&](int p0) {
#pragma unroll
                for (int u = 0; u < U; ++u) from[u] = *(const v4f*)(a.sums + at(p64 + min(p0 + u * PL + sub, n - 1)) * D + ch);
            };
            const v4f st = *(const v4f*)(a.stats + at(p64 + min(lane, n - 1)) * 4);
            fetch(0);
            float m = st[0];
#pragma unroll
            for (int s = 1; s < 64; s *= 2) m = fmaxf(m, __shfl_xor(m, s, 64));
            m = fmaxf(m, top);
            const float old = m == -INFINITY ? 1.0f : worth(top, m);
            const float f = lane >= n ? 0.0f : st[0] == -INFINITY ? 1.0f : worth(st[0], m);
            top = m;
            float more = lane < n ? f * st[1] : 0.0f;
#pragma unroll
            for (int s = 1; s < 64; s *= 2) more += __shfl_xor(more, s, 64);
            sum = sum * old + more;
            any = fmaxf(any, __ballot(st[2] > 0.0f) ? 1.0f : 0.0f);
            out *= old;
            for (int p0 = 0; p0 < n; p0 += U * PL) {
                if (p0) fetch(p0);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int p = p0 + u * PL + sub;
                    const float wt = __shfl(f, p & 63, 64);
#pragma unroll
                    for (int e = 0; e < 4; ++e) out[e] = p < n ? out[e] + wt * from[u][e] : out[e];
                }
            }
        }
#pragma unroll
        for (int s = LP; s < 64; s *= 2)
#pragma unroll
            for (int e = 0; e < 4; ++e) out[e] += __shfl_xor(out[e], s, 64);
        if (lane >= LP) continue;
        const uint32_t r = info.r0 + row, n = r / (uint32_t)a.G;
        store4((T*)a.y + (long long)(info.f0 + n) * a.ldy + (head * a.G + (int)(r - n * a.G)) * D + ch, out, sum, any > 0.0f);
    }
}

template <class T, int BITS, int D, int RB>
hipError_t launch_attn(AttnArgs a, int kv_heads, hipStream_t st) {
    const long long tiles = ((long long)a.N * a.G) / (16 * RB) + a.pages.seqs;   // at most, of one key head
    const long long blocks = (((long long)a.pages.ld << a.pages.shift) + 31) / 32;
    // as many workgroups as the card holds at once, if the tiles do not make them by themselves.  If they do, each is one
    // workgroup's whatever its length, so a sequence much longer than the others sets the time (8 key heads: one of 131072
    // tokens beside 63 of 500 80 us, beside 80 1280; 80 of 500 alone 21)
    const long long full = 256 * waves_of(sizeof(T) == 4, D, RB) / kv_heads;
    if (a.pages.seqs > 64 && tiles < full) {
        // 64 sequences at a time, one launch or two for each (one key head: 500 sequences of 100 tokens 52 us; 800, which
        // fill the card and are one launch, 15)
        hipError_t e = hipSuccess;
        for (int i = 0; i < a.pages.seqs && e == hipSuccess; i += 64) {
            AttnArgs some = a;
            some.pages.first += i, some.pages.length += i, some.pages.table += (size_t)i * a.pages.ld;
            if (a.prefix) some.prefix += i;
            some.pages.seqs = std::min(64, a.pages.seqs - i);
            e = launch_attn<T, BITS, D, RB>(some, kv_heads, st);
        }
        return e;
    }
    a.most = (int)tiles;
    const bool fits = (full + tiles) * kv_heads <= MAX_SLOTS && tiles * (blocks + 16) < 1ll << 30;
    a.shares = a.pages.seqs <= 64 && blocks > MOST_WHOLE && tiles < full && fits ? (int)full : 0;
    const hipError_t e = launch(k_attn<T, BITS, D, RB>, dim3((unsigned)(a.shares ? a.shares : tiles), kv_heads), 256u, st, a);
    if (e != hipSuccess || !a.shares) return e;
    // (a wave to a row while that makes no more workgroups than the card holds at once: 1 x 4096 12.9 -> 11.7 us; else
    // four rows to a wave: 64 sequences 118 -> 116)
    a.join = tiles * kv_heads * RB <= 512 ? 4 : 1;
    return launch(k_attn_join<T, D, RB>, dim3((unsigned)tiles * RB * a.join, kv_heads), 256u, st, a);
}

template <class T, int BITS, int D>
hipError_t launch_attn(const AttnArgs& a, int kv_heads, hipStream_t st) {
    const long long rows = ((long long)a.N * a.G + a.pages.seqs - 1) / a.pages.seqs;   // of a sequence, in the mean
    // (4 sequences of 8192 tokens: 16 rows 23.5 us in one block of rows, 24.7 with room for two; 32 rows 26.1 in two
    // at once against 32.8, 256 rows 93 against 171)
    if (rows <= 16) return launch_attn<T, BITS, D, 1>(a, kv_heads, st);
    return launch_attn<T, BITS, D, 2>(a, kv_heads, st);
}

void free_attn(dq_attn* a) {
    if (!a) return;
    DeviceGuard dg(a->device);
    (void)hipFree(a->sums);
    delete a;
}

}  // namespace
}  // namespace dq

using namespace dq;

extern "C" {

dq_status dq_attn_create(int32_t device, dq_attn** out) {
    set_error("");
    if (!out) return fail(DQ_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    const dq_status st = known_device(device);
    if (st != DQ_OK) return st;
    DeviceGuard dg(device);
    if (!dg.ok) return fail(DQ_ERR_DEVICE, "hipSetDevice failed");
    auto* a = new (std::nothrow) dq_attn();
    if (!a) return fail(DQ_ERR_OUT_OF_MEMORY, "host allocation failed");
    std::unique_ptr<dq_attn, void (*)(dq_attn*)> guard(a, free_attn);
    a->device = device;
    hipError_t e;
    if ((e = hipMalloc((void**)&a->sums, (SUM_FLOATS + STAT_FLOATS) * 4 + MAX_SLOTS * sizeof(TileInfo))) != hipSuccess) {
        a->sums = nullptr;
        return hip_fail(e, "hipMalloc workspace");
    }
    *out = guard.release();
    return DQ_OK;
}

void dq_attn_destroy(dq_attn* a) { free_attn(a); }

dq_status dq_attn_rows(const dq_kv* kv, const dq_seqs* seqs, int64_t N, const void* q_dev, int64_t ldq, dq_dtype dt,
                       int32_t q_heads, const dq_attn_ops* ops, dq_attn* a, void* y_dev, int64_t ldy, int32_t device,
                       void* stream) {
    set_error("");
    dq_status st = check_kv(kv);
    if (st != DQ_OK || (st = check_seqs(seqs)) != DQ_OK) return st;
    const int D = kv->head_dim;
    if (D != 64 && D != 128) return fail(DQ_ERR_SHAPE, "attention takes a head_dim of 64 or 128");
    if (dt != DQ_F32 && dt != DQ_BF16) return fail(DQ_ERR_INVALID_ARG, "unknown dtype");
    if (N < 0 || N > 1 << 24) return fail(DQ_ERR_SHAPE, "N must be in [0, 2^24]");   // (a launch takes fewer than 2^32 threads)
    if (q_heads < 1 || q_heads % kv->heads != 0 || (int64_t)q_heads * D > 32768)
        return fail(DQ_ERR_SHAPE, "q_heads must be a multiple of the cache's heads with q_heads * head_dim <= 32768");
    if (N * (q_heads / kv->heads) > 1 << 27) return fail(DQ_ERR_SHAPE, "N * q_heads / heads must be at most 2^27");
    if (!ops || !a) return fail(DQ_ERR_INVALID_ARG, "ops or workspace is NULL");
    const double most = 4294967296.0;                      // 2^32: the factors of the scores stay in fp32's range
    if (!(ops->scale >= 1.0 / most) || !(ops->scale <= most)) return fail(DQ_ERR_INVALID_ARG, "scale must be in [2^-32, 2^32]");
    if (ops->cap != 0.0 && !(ops->cap >= 1.0 / most && ops->cap <= most)) return fail(DQ_ERR_INVALID_ARG, "cap must be 0 or in [2^-32, 2^32]");
    if (ops->block < 0 || ops->block >= int64_t(1) << 31 || ops->window < 0 || ops->window >= int64_t(1) << 31)
        return fail(DQ_ERR_SHAPE, "block and window must be in [0, 2^31)");
    if (ops->block == 0 && ops->window != 0) return fail(DQ_ERR_INVALID_ARG, "a window needs a block of 1 or more");
    if ((uintptr_t)ops->prefix_dev % 4 != 0) return fail(DQ_ERR_INVALID_ARG, "prefix_dev must be 4-byte aligned");
    if (a->device != device) return fail(DQ_ERR_INVALID_ARG, "the workspace is on another device");
    if (N == 0) return DQ_OK;
    if (!q_dev || !y_dev) return fail(DQ_ERR_INVALID_ARG, "q_dev or y_dev is NULL");
    if (((uintptr_t)q_dev | (uintptr_t)y_dev) % 16 != 0) return fail(DQ_ERR_INVALID_ARG, "q_dev and y_dev must be 16-byte aligned");
    const int64_t esz = dt == DQ_BF16 ? 2 : 4, C = (int64_t)q_heads * D;
    for (const int64_t ld : {ldq, ldy})
        if (ld < C || ld > (int64_t(1) << 40) / N || ld * esz % 16 != 0)
            return fail(DQ_ERR_SHAPE, "the row strides must be at least the row's width and a multiple of 16 bytes");
    const Span y{y_dev, N, ldy * esz, C * esz};
    const int64_t cb = kv_code_bytes(kv), sb = kv_scale_bytes(kv);
    const struct {
        Span s;
        const char* name;
    } in[] = {{{q_dev, N, ldq * esz, C * esz}, "q_dev"}, {{kv->k_codes, 1, cb, cb}, "k_codes"}, {{kv->k_scales, 1, sb, sb}, "k_scales"},
              {{kv->v_codes, 1, cb, cb}, "v_codes"}, {{kv->v_scales, 1, sb, sb}, "v_scales"},
              {{seqs->first_dev, 1, 4 * (seqs->seqs + 1), 4 * (seqs->seqs + 1)}, "first_dev"},
              {{seqs->length_dev, 1, 4 * seqs->seqs, 4 * seqs->seqs}, "length_dev"},
              {{seqs->pages_dev, 1, 4 * seqs->seqs * seqs->pages_ld, 4 * seqs->seqs * seqs->pages_ld}, "pages_dev"},
              {{ops->prefix_dev, 1, 4 * seqs->seqs, 4 * seqs->seqs}, "prefix_dev"}};
    for (const auto& i : in)
        if (overlap(y, i.s)) return fail(DQ_ERR_INVALID_ARG, std::string("y_dev overlaps ") + i.name);
    DeviceGuard dg(device);
    if (!dg.ok) return fail(DQ_ERR_DEVICE, "hipSetDevice failed");
    AttnArgs k{};
    k.q = q_dev, k.y = y_dev;
    k.ldq = ldq, k.ldy = ldy;
    k.codes[0] = kv->k_codes, k.codes[1] = kv->v_codes;
    k.scales[0] = kv->k_scales, k.scales[1] = kv->v_scales;
    k.pages = pages_of(kv, seqs);
    k.prefix = ops->prefix_dev;
    k.N = (int)N, k.G = q_heads / kv->heads;
    k.block = ops->block, k.window = ops->window;
    k.cap = (float)ops->cap;
    k.cap_in = ops->cap != 0.0 ? (float)(ops->scale / ops->cap) : 0.0f;
    k.scale = ops->cap != 0.0 ? 1.0f : (float)(ops->scale * 1.4426950408889634);
    k.sums = a->sums, k.stats = a->sums + SUM_FLOATS;
    k.tiles = (TileInfo*)(k.stats + STAT_FLOATS);
    const auto go = [&](auto bits, auto dim) {
        constexpr int B = decltype(bits)::value, W = decltype(dim)::value;
        return dt == DQ_BF16 ? launch_attn<uint16_t, B, W>(k, kv->heads, (hipStream_t)stream)
                             : launch_attn<float, B, W>(k, kv->heads, (hipStream_t)stream);
    };
    const auto by_dim = [&](auto bits) {
        return D == 64 ? go(bits, std::integral_constant<int, 64>{}) : go(bits, std::integral_constant<int, 128>{});
    };
    const hipError_t e = kv->bits == 8 ? by_dim(std::integral_constant<int, 8>{}) : by_dim(std::integral_constant<int, 4>{});
    return e == hipSuccess ? DQ_OK : hip_fail(e, "attention launch");
}

}  // extern "C"
