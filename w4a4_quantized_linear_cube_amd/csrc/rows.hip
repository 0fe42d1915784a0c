// Products of a few token rows with a prepared 4-bit weight, and the loading
// of a weight that is already coded.
//
//   y[n][j] = sum_c x[n][c] Q4(R)[j][c] + sum_q U[n][q] L2[q][j],   U = x L1
//
// x is bf16, fp32 or MX-FP8; nothing is quantized on the way: Q4(R) decodes to
// bf16 exactly (2 significant bits and a power of two), an MX-FP8 value is a
// bf16 value (4 significant bits), and an fp32 value is the sum of three bf16
// values (8 bits each), so every product is exact in the bf16 matrix
// instruction and the sums are fp32.  (The scaled FP8 x FP4 instruction would
// not need the decoding, but keeps only about 13 bits of its products' sum.)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <memory>
#include <new>
#include <string>
#include <type_traits>

#include "dq.h"
#include "dq_device.h"
#include "dq_internal.h"

namespace dq {

constexpr int CUS = 256, MAX_ROWS = 4096;

// How the general form splits N rows of a weight: tiles of 64 rb channels and
// 16 tb rows, K slices of `per` steps.
struct SplitPlan {
    int tb, rb, groups, tiles, slices, per;
    int64_t units() const { return (int64_t)groups * tiles; }
    int64_t sum_floats() const { return slices > 1 ? units() * slices * 4 * rb * tb * 256 : 0; }
};

// `parts` of a row: three for fp32 rows, whose larger operands leave LDS for
// 16 rows at a time.  Figures below are us of bf16 rows, rank 32.
//  - rb: 256 channels to a tile (rb 4) halve what is read again of x and L1, which
//    pays for several groups of rows where the tiles fill a quarter of the chip.
//    128 / 256: 64 rows 5120 -> 10240 18.2 / 16.3, 13824 -> 8192 27.0 / 24.4, 5120 ->
//    13824 19.3 / 19.4; but 5120 -> 5120 12.1 / 13.6 and, with few K steps,
//    1536 -> 10240 8.7 / 10.9.
//  - slices: a CU's time goes by the K steps of its slice, three more to every
//    chunk of four begun, and each slice costs the workgroup that joins them the
//    time of 1.6 steps (1.0 where a step is longer: three parts, more low ranks).
//    Slices of 4 / 8 / 12 / 20 steps: 16 rows 8960 -> 1536 10.5 / 9.1 / 9.3 / 10.8,
//    24 rows 5120 -> 5120 14.2 / 10.4 / 10.6 / 12.6, 64 rows 1536 -> 1536
//    7.2 of 4 and 8.0 of 12.  Not more workgroups than CUs, or than two to a CU
//    where two fit, in fp32 (64 rows 5120 -> 5120: 480 of 14 steps 21.2, 160 of 40
//    25.3; in bf16 64 rows 1536 -> 8960: 420 of 4 steps 14.4, 140 of 12 9.0).
// Over 58 shapes the choice is within 0.4 % of the best slice length on average,
// 5.5 % at worst (24 fp32 rows 13824 -> 5120: 3 slices 27.1, 6 slices 25.7).
static SplitPlan plan_split(int64_t N, int64_t Co, int nks, int rp, int parts) {
    SplitPlan p;
    p.tb = N <= 16 || parts > 1 ? 1 : 2;
    p.groups = (int)((N + 16 * p.tb - 1) / (16 * p.tb));
    p.rb = p.groups > 1 && parts == 1 && (Co + 255) / 256 * p.groups >= 64 && nks >= 24 ? 4 : 2;
    p.tiles = (int)((Co + 64 * p.rb - 1) / (64 * p.rb));
    const int most = parts == 3 && rp <= 32 ? 2 * CUS : CUS;
    double least = 0.0;
    for (int s = 1; s == 1 || (s <= nks / 2 && p.units() * s <= most); ++s) {
        const int per = (nks + s - 1) / s, slices = (nks + per - 1) / per;
        const int64_t rounds = (p.units() * slices + CUS - 1) / CUS;
        const double cost = (double)rounds * (per + 3 * ((per + 3) / 4)) + (parts == 1 && rp <= 32 ? 1.6 : 1.0) * slices;
        if (s == 1 || cost < least) {
            least = cost;
            p.per = per;
            p.slices = slices;
        }
    }
    return p;
}

}  // namespace dq

// Workspace of the few-row products: where workgroups that share a tile meet.
struct dq_rows {
    int device = 0;
    int64_t max_rows = 0, Ci = 0, Co = 0, Kp = 0;
    int rp = 0;
    float* sums = nullptr;     // the K slices' sums of every tile
    int* arrivals = nullptr;   // slices of a tile that have ended (0 between launches)
    dq::SplitPlan plans[2][dq::MAX_ROWS / 16];   // of 1 .. 16, 17 .. 32, .. rows, for one part a row and for three
};

namespace dq {
namespace {

constexpr int X_BF16 = 0, X_F32 = 1, X_MX8 = 2;

struct RowsArgs {
    const void* x;                        // rows (bf16, fp32) or E4M3 codes
    const uint8_t* xs;                    // E8M0 codes of MX-FP8 rows
    long long ldx;
    int N, Ci, nks, Co, rank, rp, y_bf16, y_wide, tiles, slices, per;
    const uint8_t *rq, *rs;
    const uint4* l1p;
    const uint16_t* l2t;
    float* sums;
    int* arrivals;
    void* y;
    long long ldy;
};

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// 8 consecutive channels of a row as they are loaded.
template <int XK> struct Piece { uint4 d; };
template <> struct Piece<X_F32> { uint4 d, hi; };
template <> struct Piece<X_MX8> { uint2 d; int e; };

// Channels ch .. of row n, zeros past N and Ci or where !live.  The load is
// made in any case, from the nearest place that exists: a number of loads in
// flight that does not depend on the lane lets the waits count them.
template <int XK>
__device__ __forceinline__ Piece<XK> load_piece(const RowsArgs& a, int n, int ch, bool live = true) {
    Piece<XK> v;
    live = live && n < a.N && ch < a.Ci;
    const long long row = min(n, a.N - 1);
    ch = min(ch, a.Ci - 8);
    if constexpr (XK == X_BF16) {
        v.d = *(const uint4*)((const uint16_t*)a.x + row * a.ldx + ch);
    } else if constexpr (XK == X_F32) {
        const uint4* p = (const uint4*)((const float*)a.x + row * a.ldx + ch);
        v.d = p[0];
        v.hi = p[1];
        v.hi = live ? v.hi : make_uint4(0u, 0u, 0u, 0u);
    } else {
        v.d = *(const uint2*)((const uint8_t*)a.x + row * a.Ci + ch);
        v.e = a.xs[row * (a.Ci >> 5) + (ch >> 5)];
        v.e = live ? v.e : 0;
    }
    v.d = live ? v.d : decltype(v.d){};
    return v;
}

// fp32 values as the sum of three bf16 values: the leading 8 bits, then those
// of what is left, twice.  The differences are exact, so the parts sum to the
// value (bits below 2^-133 apart).  What is left of an infinity is made zero; of
// a NaN it is NaN.
__device__ __forceinline__ void split3(const float* v, uint4* out) {
    uint32_t w[3][4];
    const auto upper = [](uint32_t hi, uint32_t lo) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); };   // two leading halves
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t b[3][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float f = v[2 * j + k];
            b[0][k] = __float_as_uint(f);
            float left = f - __uint_as_float(b[0][k] & 0xffff0000u);
            left = __builtin_fabsf(f) == __builtin_inff() ? 0.0f : left;
            b[1][k] = __float_as_uint(left);
            b[2][k] = __float_as_uint(left - __uint_as_float(b[1][k] & 0xffff0000u));
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) w[p][j] = upper(b[p][1], b[p][0]);
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) out[p] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}

// ... and as bf16 operand pieces: one, or three parts of fp32 values.
template <int XK>
__device__ __forceinline__ void operand(const Piece<XK>& v, uint4* out) {
    if constexpr (XK == X_BF16) {
        out[0] = v.d;
    } else if constexpr (XK == X_F32) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = __uint_as_float(word(v.d, i));
            f[4 + i] = __uint_as_float(word(v.hi, i));
        }
        split3(f, out);
    } else {
        // (4 significant bits times a power of two: exact in bf16; scale code 255 makes the group NaN)
        const float s = pow2f(v.e - 127);
        const uint32_t lo = v.e == 255 ? 0x7f7f7f7fu : v.d.x, hi = v.e == 255 ? 0x7f7f7f7fu : v.d.y;
        out[0] = make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false)),
                            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true)),
                            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false)),
                            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true)));
    }
}

// The weight of one row and 32 channels as four bf16 operands; exact (2
// significant bits and a power of two).
__device__ __forceinline__ v8bf weight8(uint32_t codes, float scale) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    const v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return v8bf{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

__device__ __forceinline__ v4f mfma(v8bf w, uint4 x, v4f acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(v8bf, x), acc, 0, 0, 0);
}

// U as a matrix operand.  Its 16 x 16 blocks (ranks by rows) come out of the
// matrix instruction with ranks 4 g .. + 3 of row n in lane 16 g + n; as an
// operand, lane l needs ranks 8 (l / 16) .. + 7 of row l % 16, which two lanes
// 16 apart hold, the first of them in place u_place(l) of two blocks' 128.
// Ranks past the last are zeros whatever x holds (an infinite channel makes
// its product with a padding column NaN); `left` ranks remain from the lane's first.
__device__ __forceinline__ int u_place(int lane) {
    const int q = lane >> 4;
    return (q >> 1) * 64 + 32 * (q & 1) + (lane & 15);
}
__device__ __forceinline__ void split_u(v4f u0, v4f u1, int left, uint4* part) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[j] = j < left ? u0[j] : 0.0f;
        f[4 + j] = 4 + j < left ? u1[j] : 0.0f;
    }
    split3(f, part);
}

// acc += U L2 for the 32 low ranks from `at` on and output channels row + l % 16.
__device__ __forceinline__ uint4 load_l2(const RowsArgs& a, int at, int row, int lane) {
    return *(const uint4*)(a.l2t + (long long)(row + (lane & 15)) * a.rp + at + 8 * (lane >> 4));
}
__device__ __forceinline__ v4f low_rank(uint4 l2, const uint4* u, v4f acc) {
#pragma unroll
    for (int p = 0; p < 3; ++p) acc = mfma(__builtin_bit_cast(v8bf, l2), u[p], acc);
    return acc;
}

// The weight stream of 16 RB output channels from row on.  Lane l reads channel
// chunk l / 16 (32 channels, 16 bytes of codes and one scale) of row l % 16 in
// each K step: 1 KB of codes in a row of the step-major layout.
template <int RB>
struct Stream {
    const uint8_t *rq, *rs;
    int so[RB];
    __device__ __forceinline__ Stream(const RowsArgs& a, int row, int lane) {
        const int q = lane >> 4, r0 = (row & 255) + (lane & 15);
        const size_t block = (size_t)(row >> 8) * a.nks;
        rq = a.rq + block * 16384 + r0 * 64 + ((q ^ swz4(r0)) << 4);
        rs = a.rs + block * 1024;
#pragma unroll
        for (int i = 0; i < RB; ++i) so[i] = (int)toff_scale(r0 + 16 * i, q);
    }
    __device__ __forceinline__ void fetch(int ks, uint4* c, int* e) const {
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            c[i] = *(const uint4*)(rq + (size_t)ks * 16384 + i * 1024);
            e[i] = rs[(size_t)ks * 1024 + so[i]];
        }
    }
};

// The outputs of a lane: channels j .. j + 3 of row n.
__device__ __forceinline__ void store_y(const RowsArgs& a, int n, int j, v4f y) {
    if (n >= a.N || j >= a.Co) return;
    typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
    if (a.y_bf16) {
        __bf16* p = (__bf16*)a.y + n * a.ldy + j;
        const v4bf b = {(__bf16)y[0], (__bf16)y[1], (__bf16)y[2], (__bf16)y[3]};
        if (a.y_wide && j + 4 <= a.Co) *(v4bf*)p = b;
        else
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (j + i < a.Co) p[i] = b[i];
    } else {
        float* p = (float*)a.y + n * a.ldy + j;
        if (a.y_wide && j + 4 <= a.Co) *(v4f*)p = y;
        else
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (j + i < a.Co) p[i] = y[i];
    }
}

// Few row parts and few channels (N16 rows, one part each or three): a wave
// takes the rows' channels of its own K steps straight from x, G steps at a
// time, and lays them out as operands in its own LDS rows (17 pieces apart, so
// that neither the writes by row nor the reads by piece meet in a bank).  The
// W waves of a workgroup share out the K steps of 16 RB output channels and
// their partial sums are added in wave order.  With LR (groups of 32 low
// ranks, 1 or 2) every workgroup forms U as well: L1 is read again by each, from L2.
// D steps are in flight.
// Bound by the weight's bytes for many channels (2 fp32 rows 5120 -> 30720, rank
// 0: 83.8 MB in 16.1 us, 5.2 TB/s; one MX-FP8 row 5120 -> 13824, rank 32: 38.9 MB
// in 9.5 us, 4.1 TB/s, of which U takes 1.6), and for few by the launch and one
// chain of loads, products and a sum (1 row 1536 -> 1536 4.1 us, 3.2 without U).
// Forming U in a launch of its own instead costs 2.8 to 3.1 us.
template <int XK, int N16, int LR, int RB, int W, int D>
__global__ __launch_bounds__(64 * W) void k_rows_direct(RowsArgs a) {
    constexpr int P = XK == X_F32 ? 3 : 1, G = N16 * P > 16 ? 1 : 16 / (N16 * P), NI = (G * N16 + 3) / 4, SUMS = RB + 2 * LR;
    constexpr int STAGED = G * P * N16 * 17, SLOTS = STAGED > 64 * SUMS ? STAGED : 64 * SUMS;
    __shared__ uint4 lds[W][SLOTS];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    // workgroups go to the 8 XCDs in turn; an XCD takes neighbouring tiles,
    // which share the 128-row blocks of the scale layout in its L2
    const int tile = (int)(blockIdx.x & 7) * (gridDim.x >> 3) + (int)(blockIdx.x >> 3);
    if (tile >= a.tiles) return;
    const int row0 = tile * 16 * RB;
    const int per = (a.nks + W - 1) / W, k0 = w * per, k1 = min(a.nks, k0 + per);
    v4f acc[SUMS];                                     // RB blocks of output channels, then two of low ranks
#pragma unroll
    for (int i = 0; i < SUMS; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    // pieces of G steps: lane l takes piece l % 16 of source rows l / 16, + 4, ..
    Piece<XK> px[NI];
    auto load_x = [&](int ks) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int R = 4 * i + (lane >> 4), g = R / N16;
            px[i] = load_piece<XK>(a, R % N16, 128 * (ks + g) + 8 * (lane & 15), g < G && ks + g < k1);
        }
    };
    uint4* xs = lds[w];
    auto stage_x = [&]() {
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int R = 4 * i + (lane >> 4), g = R / N16, n = R % N16;
            uint4 part[P];
            operand<XK>(px[i], part);
#pragma unroll
            for (int p = 0; p < P; ++p)
                if (g < G) xs[((g * P + p) * N16 + n) * 17 + (lane & 15)] = part[p];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    const Stream<RB> weight(a, row0, lane);
    uint4 c[D][RB], l1[D][LR ? 8 * LR : 1];
    int e[D][RB];
    auto fetch = [&](int d, int ks) {
        weight.fetch(ks, c[d], e[d]);
        if constexpr (LR) {
#pragma unroll
            for (int f = 0; f < 8 * LR; ++f) l1[d][f] = a.l1p[((long long)ks * (8 * LR) + f) * 64 + lane];
        }
    };
    if (k0 < k1) load_x(k0);
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (k0 + d < k1) fetch(d, k0 + d);
    uint4 l2[LR ? LR : 1];
#pragma unroll
    for (int r = 0; r < LR; ++r) l2[r] = load_l2(a, 32 * r, row0 + 16 * (w % RB), lane);
    const int rd = (lane & (N16 - 1)) * 17 + 4 * (lane >> 4);
    int staged = G;                                    // steps used of the staged ones
    for (int ks = k0; ks < k1; ks += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (ks + d >= k1) break;
            if (staged == G) {
                stage_x();
                if (ks + d + G < k1) load_x(ks + d + G);
                staged = 0;
            }
            const int at = staged++ * P * N16 * 17 + rd;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                uint4 x[P];
#pragma unroll
                for (int p = 0; p < P; ++p) x[p] = xs[at + p * N16 * 17 + f];
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    const v8bf wv = weight8(word(c[d][i], f), pow2f(e[d][i] - 127));
#pragma unroll
                    for (int p = 0; p < P; ++p) acc[i] = mfma(wv, x[p], acc[i]);
                }
                if constexpr (LR) {
#pragma unroll
                    for (int i = 0; i < 2 * LR; ++i)
#pragma unroll
                        for (int p = 0; p < P; ++p) acc[RB + i] = mfma(__builtin_bit_cast(v8bf, l1[d][4 * i + f]), x[p], acc[RB + i]);
                }
            }
            if (ks + d + D < k1) fetch(d, ks + d + D);
        }
    }
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < SUMS; ++i) ((v4f*)lds[w])[i * 64 + lane] = acc[i];
    __syncthreads();
    if (w >= RB) return;
    const int row = row0 + 16 * w;
    v4f y = ((const v4f*)lds[0])[w * 64 + lane];
#pragma unroll
    for (int i = 1; i < W; ++i) y += ((const v4f*)lds[i])[w * 64 + lane];
#pragma unroll
    for (int r = 0; r < LR; ++r) {
        const int from = (RB + 2 * r) * 64 + u_place(lane);
        v4f u0 = {0.0f, 0.0f, 0.0f, 0.0f}, u1 = u0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            u0 += ((const v4f*)lds[i])[from];
            u1 += ((const v4f*)lds[i])[from + 16];
        }
        uint4 part[3];
        split_u(u0, u1, a.rank - 32 * r - 8 * (lane >> 4), part);
        y = low_rank(l2[r], part, y);
    }
    if ((lane & 15) < N16) store_y(a, lane & 15, row + 4 * (lane >> 4), y);
}

// Sums that workgroups of one launch hand to each other: stores and loads with
// the agent scope's cache bit (sc1, 16 in the buffer instructions' last
// operand) go to and come from where every XCD's caches meet, so no cache
// needs writing back or invalidating (fences that do that, one a wave, cost
// 30 to 100 us here).
typedef unsigned v4u __attribute__((ext_vector_type(4)));
__device__ __forceinline__ __amdgpu_buffer_rsrc_t shared_sums(float* p, size_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(p, (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ void hand_over(__amdgpu_buffer_rsrc_t r, int at, v4f v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v), r, at * 16, 0, 16);
}
__device__ __forceinline__ v4f take_over(__amdgpu_buffer_rsrc_t r, int at) {
    return __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(r, at * 16, 0, 16));
}

// The general form: a workgroup owns 64 RB output channels of 16 TB rows over
// one slice of the K steps, in chunks of CH steps whose operands all its waves
// share in LDS.  Wave w takes 16 RB channels (w % 4) of every other step (w / 4).
// The slice's U is formed too (wave w: step w % 4 of a chunk, 16 of each 32
// low ranks, w / 4) and applied to the slice's sums, both being linear in x, so
// L1 is read once a tile and step.  The slices' sums meet in the workspace:
// whichever workgroup of a tile ends last adds them up in slice order, so
// nothing waits and a result does not depend on the order of arrival.
// The operands of the next chunk are laid out in LDS while one is used, so a
// chunk has one barrier (0.39 -> 0.29 us a K step of 24 rows; where that leaves
// no room for a second workgroup or its registers, in fp32 and with 256 channels,
// it costs more than it gives and there is one place).
// A K step of 128 x 32 operands takes a CU 0.29 us, whether 12 workgroups run
// or 240.  In timing copies of the form with one place (0.39 us) it was 0.15 less
// without laying out x, 0.10 without reading the operands from LDS, 0.07 without
// loading L1, 0.05 without loading x.  Before and after the loop come the launch and the first loads,
// 2.2 us, and the chain of low-rank product, hand-over, arrival and joining, 3 us:
// 64 MX-FP8 rows 5120 -> 5120 11.8 us, 16 bf16 rows 13824 -> 5120 12.8 us (39.4 MB,
// 3.1 TB/s), 37 rows 2080 -> 4999 9.2 us.
// LP: groups of 32 low ranks (1, also for rank 0, or 4, whose next group's L1
// loads while one is used: 64 rows 5120 -> 5120 rank 128 21.6 -> 18.6 us).
template <int XK, int TB, int LP, int RB>
__global__ __launch_bounds__(512, XK == X_F32 && LP == 1 ? 4 : 2) void k_rows_split(RowsArgs a) {
    constexpr int P = XK == X_F32 ? 3 : 1, CH = 4, J = CH / 2, NP = CH * TB / 2, BLK = 16 * 17;
    constexpr int HB = RB / 2, OUT = 8 * TB * HB * 64; // blocks of channels a wave finishes; 16-byte places of the tile's sums
    constexpr int ALL = OUT + LP * 8 * TB * 64;        // ... with U's shares, where the operands were
    constexpr bool TWO = P == 1 && RB == 2;                       // the next chunk's operands are laid out beside the one in use
    constexpr int X = CH * P * TB * BLK, ROOM = TWO ? 2 * X : X;
    __shared__ uint4 lds[ROOM > ALL ? ROOM : ALL];
    __shared__ int arrived;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    // (a row of workgroups is a multiple of 8, so the groups of rows that read the
    // same weight are on the same XCD and its L2: 64 rows 5120 -> 13824 21.2 -> 19.3 us)
    const int tile = (int)blockIdx.x % a.tiles, slice = (int)blockIdx.x / a.tiles;
    if (slice >= a.slices) return;
    const int n0 = (int)blockIdx.y * 16 * TB, wk = w >> 2, row0 = tile * 64 * RB + 16 * RB * (w & 3);
    const int row = row0 + 16 * HB * wk;               // the 16 HB channels this wave finishes
    const int k0 = slice * a.per, k1 = min(a.nks, k0 + a.per), passes = a.rp >> 5, ug = w % CH;
    v4f acc[TB][RB], u[LP][TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
#pragma unroll
        for (int i = 0; i < RB; ++i) acc[t][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int r = 0; r < LP; ++r) u[r][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // thread t takes piece t % 16 of rows t / 16, + 32, .. of a chunk (16 TB rows a step)
    Piece<XK> px[NP];
    auto load_x = [&](int ks) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int R = 32 * i + (tid >> 4);
            px[i] = load_piece<XK>(a, n0 + R % (16 * TB), 128 * (ks + R / (16 * TB)) + 8 * (tid & 15));
        }
    };
    auto stage_x = [&](int to) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int R = 32 * i + (tid >> 4), g = R / (16 * TB), n = R % (16 * TB);
            uint4 part[P];
            operand<XK>(px[i], part);
#pragma unroll
            for (int p = 0; p < P; ++p) lds[to + ((g * P + p) * TB * 16 + n) * 17 + (tid & 15)] = part[p];
        }
    };
    const Stream<RB> weight(a, row0, lane);
    uint4 c[J][RB], l1[LP > 1 ? 2 : 1][4], l2[LP][HB];  // (of one group of 32 low ranks in use, and the next)
    int e[J][RB];
    auto load_u = [&](int ks, int r) {                 // (places past the slice: its last step again, not used)
        const uint4* p = a.l1p + ((long long)min(ks + ug, k1 - 1) * (a.rp >> 4) + 2 * r + wk) * 256 + lane;
#pragma unroll
        for (int f = 0; f < 4; ++f) l1[r & 1][f] = p[f * 64];
    };
    const int own = (lane & 15) * 17 + 4 * (lane >> 4);
    int at = 0;                                        // place of the chunk in use
    auto chunk = [&](int ks, auto next, auto after) {
        constexpr bool MORE = decltype(next)::value, AFTER = decltype(after)::value;   // another chunk follows, another two
        const int rd = at + own;
        if constexpr (!TWO) {
            stage_x(0);
            __syncthreads();
            if constexpr (MORE) load_x(ks + CH);
        }
        auto form_u = [&](int r) {
#pragma unroll
            for (int f = 0; f < 4; ++f)
#pragma unroll
                for (int t = 0; t < TB; ++t)
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        u[r][t] = mfma(__builtin_bit_cast(v8bf, l1[r & 1][f]), lds[((ug * P + p) * TB + t) * BLK + rd + f], u[r][t]);
        };
        if (passes && (MORE || ks + ug < k1)) {
#pragma unroll
            for (int r = 0; r < LP; ++r) {
                if (r && r >= passes) break;
                if (r + 1 < LP && r + 1 < passes) load_u(ks, r + 1);
                form_u(r);
            }
        }
        if constexpr (MORE)
            if (passes) load_u(ks + CH, 0);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int g = 2 * j + wk;
            if (!MORE && ks + g >= k1) break;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                v8bf wv[RB];
#pragma unroll
                for (int i = 0; i < RB; ++i) wv[i] = weight8(word(c[j][i], f), pow2f(e[j][i] - 127));
#pragma unroll
                for (int t = 0; t < TB; ++t)
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const uint4 x = lds[((g * P + p) * TB + t) * BLK + rd + f];
#pragma unroll
                        for (int i = 0; i < RB; ++i) acc[t][i] = mfma(wv[i], x, acc[t][i]);
                    }
            }
            if constexpr (MORE) weight.fetch(min(ks + CH + g, k1 - 1), c[j], e[j]);
            if constexpr (TWO && MORE)
                if (j == 0) {
                    stage_x(X - at);
                    if constexpr (AFTER) load_x(ks + 2 * CH);
                }
        }
        __syncthreads();                               // (the operands are read, the next ones laid out)
        if constexpr (TWO) at = X - at;
    };
    auto load_l2s = [&](int r) {
#pragma unroll
        for (int i = 0; i < HB; ++i) l2[r][i] = load_l2(a, 32 * r, row + 16 * i, lane);
    };
    load_x(k0);
    if (passes) {
        load_u(k0, 0);
        load_l2s(0);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) weight.fetch(min(k0 + 2 * j + wk, k1 - 1), c[j], e[j]);
    if constexpr (TWO) {
        stage_x(0);
        if (k0 + CH < k1) load_x(k0 + CH);
        __syncthreads();
    }
    const std::true_type yes;
    const std::false_type no;
    int ks = k0;
    for (; ks + 2 * CH < k1; ks += CH) chunk(ks, yes, yes);
    if (ks + CH < k1) {
        chunk(ks, yes, no);
        ks += CH;
    }
    chunk(ks, no, no);
    // each wave finishes one half of its channels: the other half goes to its
    // partner (w ^ 4) through LDS, and its share of U to every wave
    v4f *part = (v4f*)lds, *us = part + OUT;
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int i = 0; i < HB; ++i) part[((w * TB + t) * HB + i) * 64 + lane] = wk ? acc[t][i] : acc[t][HB + i];
#pragma unroll
    for (int r = 0; r < LP; ++r) {
        if (r && r >= passes) break;
        if (r) load_l2s(r);
#pragma unroll
        for (int t = 0; t < TB; ++t) us[((r * 8 + w) * TB + t) * 64 + lane] = u[r][t];
    }
    __syncthreads();
    v4f y[TB][HB];
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            const v4f other = part[(((w ^ 4) * TB + t) * HB + i) * 64 + lane];
            y[t][i] = wk ? other + acc[t][HB + i] : acc[t][i] + other;
        }
    // rank block b of 32 lies with the waves 4 b .. 4 b + 3, a share of the steps each
    const int from = u_place(lane), base = 4 * (from >> 6) * TB * 64 + (from & 63);
#pragma unroll
    for (int r = 0; r < LP; ++r) {
        if (r ? r >= passes : !passes) break;
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            v4f u0 = {0.0f, 0.0f, 0.0f, 0.0f}, u1 = u0;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                u0 += us[base + ((r * 8 + i) * TB + t) * 64];
                u1 += us[base + ((r * 8 + i) * TB + t) * 64 + 16];
            }
            uint4 up[3];
            split_u(u0, u1, a.rank - 32 * r - 8 * (lane >> 4), up);
#pragma unroll
            for (int i = 0; i < HB; ++i) y[t][i] = low_rank(l2[r][i], up, y[t][i]);
        }
    }
    if (a.slices > 1) {
        const long long unit = (long long)blockIdx.y * a.tiles + tile;
        const int mine = w * TB * HB * 64 + lane;
        const __amdgpu_buffer_rsrc_t sums = shared_sums(a.sums + unit * a.slices * OUT * 4, (size_t)a.slices * OUT * 16);
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int i = 0; i < HB; ++i) hand_over(sums, slice * OUT + mine + (t * HB + i) * 64, y[t][i]);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (every wave's sums have arrived before the workgroup says so)
        __syncthreads();
        if (tid == 0) arrived = __hip_atomic_fetch_add(a.arrivals + unit, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (arrived != a.slices - 1) return;
        for (int s = 0; s < a.slices; s += 4) {        // (4 slices' loads in flight)
            v4f v[4][TB * HB];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (s + k < a.slices)
#pragma unroll
                    for (int i = 0; i < TB * HB; ++i) v[k][i] = take_over(sums, (s + k) * OUT + mine + i * 64);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (s + k < a.slices)
#pragma unroll
                    for (int i = 0; i < TB * HB; ++i) y[i / HB][i % HB] = s + k ? y[i / HB][i % HB] + v[k][i] : v[k][i];
        }
        if (tid == 0) a.arrivals[unit] = 0;            // (for the next launch)
    }
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int i = 0; i < HB; ++i) store_y(a, n0 + 16 * t + (lane & 15), row + 16 * i + 4 * (lane >> 4), y[t][i]);
}

template <int XK, int N16, int LR, int RB, int W, int D>
hipError_t launch_direct(RowsArgs a, hipStream_t st) {
    a.tiles = (a.Co + 16 * RB - 1) / (16 * RB);
    return launch(k_rows_direct<XK, N16, LR, RB, W, D>, dim3((unsigned)round_up(a.tiles, 8)), 64 * W, st, a);
}

template <int XK, int TB, int RB>
hipError_t launch_split(RowsArgs a, const SplitPlan& p, hipStream_t st) {
    a.tiles = p.tiles;
    a.slices = p.slices;
    a.per = p.per;
    const dim3 grid((unsigned)round_up(p.tiles * p.slices, 8), (unsigned)p.groups);
    return launch(a.rp <= 32 ? k_rows_split<XK, TB, 1, RB> : k_rows_split<XK, TB, 4, RB>, grid, 512, st, a);
}

// Measured at bf16 rows, rank 32 unless said otherwise (us, a captured run of calls):
//  - Direct or split.  The direct form needs no meeting of workgroups, but each
//    of its workgroups reads all of L1 and x, so it pays up to a number of K
//    steps that depends on what it reads.  Direct / split: one row 1536 -> 1536
//    4.1 / 5.6, 5120 -> 5120 8.2 / 8.4, 5120 -> 13824 10.0 / 11.8, 8960 -> 5120
//    11.5 / 9.8; 8 rows 2080 -> 4999 5.9 / 7.1, 5120 -> 5120 9.1 / 8.7.  Without
//    low ranks: 16 rows 5120 -> 5120 6.8 / 8.2, 10240 -> 5120 10.0 / 10.9, 13824 ->
//    5120 12.3 / 12.0; 8 rows 16384 -> 5120 10.8 / 12.7; 4 rows 5120 -> 10240 8.0 /
//    9.4, 13824 -> 10240 16.5 / 15.8.  Rank
//    64: one row 928 -> 3265 5.3 / 6.3, 16 rows 1536 -> 1536 6.3 / 6.6, 2080 -> 4999
//    8.5 / 8.5, one row 2976 -> 1536 7.4 / 7.2; rank 128: 1536 -> 1536 8.3 / 7.5.
//    fp32 rows have three parts, and 5 to 16 of them: 16 rows 928 -> 3265 5.6 / 7.5,
//    1536 -> 1536 7.2 / 7.2; without low ranks 2080 -> 4999 7.6 / 8.0, 2976 -> 1536
//    7.4 / 7.2.
//  - 64 output channels to a workgroup halve the readings of L1 and x, but leave
//    CUs idle for few channels.  32 / 64 channels: one row 5120 -> 5120 8.2 / 9.0,
//    1536 -> 8960 6.3 / 5.4, 5120 -> 13824 13.2 / 10.0.
//  - Two K steps in flight help where U and more rows do not need the registers.
//    One / two: rank 0 5120 -> 5120 4 rows 6.4 / 5.8, but 5120 -> 13824 16 rows
//    9.3 / 9.8; with U one row 5120 -> 13824 10.0 / 11.3.
//  - 16 waves to a workgroup instead of 8 help where neither U nor 64 channels
//    take the registers and LDS of two: rank 0 8 rows 8960 -> 5120 9.4 / 7.5, one row
//    5120 -> 5120 5.2 / 5.4; but 8 rows 5120 -> 13824 8.9 / 9.2, and with U one
//    row 1536 -> 1536 4.1 / 4.6, 5120 -> 5120 8.3 / 8.7.
template <int XK>
hipError_t launch_rows_product(const RowsArgs& a, const SplitPlan& p, hipStream_t st) {
    constexpr int P = XK == X_F32 ? 3 : 1;
    int most;                                              // K steps the direct form takes
    if (P > 1 && a.N > 4) most = a.rp ? 8 : 17;
    else if (a.rp) most = a.rp > 32 ? 14 : a.N == 1 ? 48 : 24;
    else most = a.Co >= 8192 ? 60 : a.N <= 8 ? 128 : 100;
    const bool direct = a.N <= 16 && a.rp <= 64 && a.nks <= most;
    if (direct) {
        const auto go = [&](auto lr, auto rb) {
            constexpr int LR = decltype(lr)::value, RB = decltype(rb)::value, D = LR || P == 3 ? 1 : 2, W = LR || RB == 4 ? 8 : 16;
            if (a.N == 1) return launch_direct<XK, 1, LR, RB, W, D>(a, st);
            if (a.N <= 4) return launch_direct<XK, 4, LR, RB, W, D>(a, st);
            return launch_direct<XK, 16, LR, RB, P == 1 ? W : 8, 1>(a, st);
        };
        const std::integral_constant<int, 0> none;
        const std::integral_constant<int, 1> one;
        const std::integral_constant<int, 2> two;
        const std::integral_constant<int, 4> four;
        if (a.Co >= 8192) return a.rp > 32 ? go(two, four) : a.rp ? go(one, four) : go(none, four);
        return a.rp > 32 ? go(two, two) : a.rp ? go(one, two) : go(none, two);
    }
    if constexpr (P == 1) {
        if (p.tb == 2) return p.rb == 2 ? launch_split<XK, 2, 2>(a, p, st) : launch_split<XK, 2, 4>(a, p, st);
    }
    return launch_split<XK, 1, 2>(a, p, st);
}

// Canonical codes [Co][Ci / 2] and scale codes [Co][Ci / 32] to the step-major layout.
__global__ __launch_bounds__(256) void k_import(const uint8_t* codes, const uint8_t* scales, long long Co, int groups,
                                                int nks, uint8_t* rq, uint8_t* rs) {
    for (long long id = (long long)blockIdx.x * 256 + threadIdx.x; id < Co * groups; id += (long long)gridDim.x * 256) {
        const long long j = id / groups;
        const int G = (int)(id % groups);
        *(uint4*)(rq + off_fp4(j, G, nks)) = ((const uint4*)codes)[id];
        rs[off_scale(j, G, nks)] = scales[id];
    }
}

template <class T>
hipError_t zalloc(T** p, size_t count, size_t* total) {
    *p = nullptr;
    if (count == 0) return hipSuccess;
    hipError_t e = hipMalloc((void**)p, count * sizeof(T));
    if (e != hipSuccess) {
        *p = nullptr;
        return e;
    }
    *total += count * sizeof(T);
    return hipMemset(*p, 0, count * sizeof(T));
}

void free_rows(dq_rows* a) {
    if (!a) return;
    DeviceGuard dg(a->device);
    (void)hipFree(a->sums);
    (void)hipFree(a->arrivals);
    delete a;
}

dq_status check_rows(const dq_weights* w, const dq_rows* a, int64_t N, const void* y_dev, dq_dtype ydt, int64_t ldy) {
    if (!w) return fail(DQ_ERR_INVALID_ARG, "weights handle is NULL");
    if (!a) return fail(DQ_ERR_INVALID_ARG, "workspace handle is NULL");
    if (w->wfmt != 4) return fail(DQ_ERR_INVALID_ARG, "a 6-bit weight takes the 6-bit entry points");
    if (a->Ci != w->Ci || a->Co != w->Co || a->rp != w->rp || a->device != w->device)
        return fail(DQ_ERR_INVALID_ARG, "workspace was created for a different weight");
    if (ydt != DQ_F32 && ydt != DQ_BF16) return fail(DQ_ERR_INVALID_ARG, "unknown output dtype");
    if (N < 0 || N > a->max_rows) return fail(DQ_ERR_SHAPE, "N must be in [0, max_rows] of the workspace");
    if (N == 0) return DQ_OK;
    if (!y_dev) return fail(DQ_ERR_INVALID_ARG, "y_dev is NULL");
    if ((uintptr_t)y_dev % (ydt == DQ_BF16 ? 2 : 4) != 0) return fail(DQ_ERR_INVALID_ARG, "y_dev must be aligned to its type");
    if (ldy < w->Co || ldy > (int64_t(1) << 40) / N) return fail(DQ_ERR_SHAPE, "the row stride of y must be at least Co");
    return DQ_OK;
}

RowsArgs rows_args(const dq_weights* w, dq_rows* a, int64_t N, void* y, dq_dtype ydt, int64_t ldy) {
    RowsArgs r{};
    r.N = (int)N;
    r.Ci = (int)w->Ci;
    r.nks = (int)(w->Kp / 128);
    r.Co = (int)w->Co;
    r.rank = (int)w->rank;
    r.rp = w->rp;
    r.rq = w->rq;
    r.rs = w->rs;
    r.l1p = (const uint4*)w->l1p;
    r.l2t = w->l2t;
    r.sums = a->sums;
    r.arrivals = a->arrivals;
    r.y = y;
    r.ldy = ldy;
    r.y_bf16 = ydt == DQ_BF16;
    const int four = ydt == DQ_BF16 ? 8 : 16;       // bytes of a lane's four outputs
    r.y_wide = (uintptr_t)y % four == 0 && (N == 1 || ldy % 4 == 0);
    return r;
}

}  // namespace
}  // namespace dq

using namespace dq;

extern "C" {

dq_status dq_import_weights(const uint8_t* rcodes_host, const uint8_t* rscales_host, int64_t Ci, int64_t Co, int32_t rank,
                            const uint16_t* l1_host, const uint16_t* l2_host, int32_t device, dq_weights** out) {
    set_error("");
    if (!out) return fail(DQ_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (!rcodes_host || !rscales_host) return fail(DQ_ERR_INVALID_ARG, "codes or scales are NULL");
    if (Ci < 32 || Ci % 32 != 0) return fail(DQ_ERR_SHAPE, "Ci must be a positive multiple of 32");
    if (Co < 1) return fail(DQ_ERR_SHAPE, "Co must be >= 1");
    if (Ci > (1 << 24) || Co > (1 << 24)) return fail(DQ_ERR_SHAPE, "Ci and Co must be <= 2^24");
    if (rank < 0 || rank > std::min<int64_t>(std::min(Ci, Co), 128))
        return fail(DQ_ERR_INVALID_ARG, "rank must be in [0, min(Ci, Co, 128)]");
    if (rank > 0 && (!l1_host || !l2_host)) return fail(DQ_ERR_INVALID_ARG, "factors are NULL");
    const int64_t groups = Ci / 32;
    uint8_t top = 0;
    for (int64_t i = 0; i < Co * groups; ++i) top = std::max(top, rscales_host[i]);
    if (top == 255) return fail(DQ_ERR_INVALID_ARG, "a scale code is 255 (not a number)");
    if (top >= 253)                                // (4 2^126 and 2 2^127 are the first that bf16 cannot hold: codes 6 and 4)
        for (int64_t i = 0; i < Co * groups; ++i)
            for (int k = 0; rscales_host[i] >= 253 && k < 32; ++k)
                if ((rcodes_host[i * 16 + k / 2] >> (k % 2 * 4) & 7) >= (rscales_host[i] == 253 ? 6 : 4))
                    return fail(DQ_ERR_INVALID_ARG, "a weight reaches 2^128: output " + std::to_string(i / groups) + ", channel " +
                                                        std::to_string(i % groups * 32 + k));
    dq_status st = known_device(device);
    if (st != DQ_OK) return st;
    DeviceGuard dg(device);
    if (!dg.ok) return fail(DQ_ERR_DEVICE, "hipSetDevice failed");
    auto* w = new (std::nothrow) dq_weights();
    if (!w) return fail(DQ_ERR_OUT_OF_MEMORY, "host allocation failed");
    std::unique_ptr<dq_weights, void (*)(dq_weights*)> guard(w, dq_weights_destroy);
    w->device = device;
    w->Ci = Ci;
    w->Co = Co;
    w->rank = rank;
    w->rp = (int)round_up(rank, RPAD);
    w->Kp = round_up(Ci, KPAD);
    w->Cop = round_up(Co, NPAD);
    struct Buf {                                   // freed on every way out
        uint8_t* p = nullptr;
        ~Buf() { (void)hipFree(p); }
    } cd, sd;
    size_t scratch = 0;
    hipError_t e;
    if ((e = zalloc(&w->rq, (size_t)(w->Cop * w->Kp / 2), &w->bytes)) != hipSuccess ||
        (e = zalloc(&w->rs, (size_t)(w->Cop * w->Kp / 32), &w->bytes)) != hipSuccess ||
        (e = zalloc(&cd.p, (size_t)(Co * Ci / 2), &scratch)) != hipSuccess ||
        (e = zalloc(&sd.p, (size_t)(Co * groups), &scratch)) != hipSuccess)
        return hip_fail(e, "hipMalloc weight");
    if ((e = hipMemcpy(cd.p, rcodes_host, (size_t)(Co * Ci / 2), hipMemcpyHostToDevice)) != hipSuccess ||
        (e = hipMemcpy(sd.p, rscales_host, (size_t)(Co * groups), hipMemcpyHostToDevice)) != hipSuccess)
        return hip_fail(e, "copy weight");
    k_import<<<(unsigned)std::min<int64_t>((Co * groups + 255) / 256, 1 << 16), 256, 0, nullptr>>>(
        cd.p, sd.p, (long long)Co, (int)groups, (int)(w->Kp / 128), w->rq, w->rs);
    if ((e = hipGetLastError()) != hipSuccess) return hip_fail(e, "import kernel");
    if ((st = upload_factors(w, l1_host, l2_host)) != DQ_OK) return st;
    if ((e = hipDeviceSynchronize()) != hipSuccess) return hip_fail(e, "weight import");
    *out = guard.release();
    return DQ_OK;
}

dq_status dq_rows_create(const dq_weights* w, int64_t max_rows, dq_rows** out) {
    set_error("");
    if (!out) return fail(DQ_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (!w) return fail(DQ_ERR_INVALID_ARG, "weights handle is NULL");
    if (w->wfmt != 4) return fail(DQ_ERR_INVALID_ARG, "a 6-bit weight takes the 6-bit entry points");
    if (max_rows < 1 || max_rows > MAX_ROWS) return fail(DQ_ERR_SHAPE, "max_rows must be in [1, 4096]");
    if (w->Ci > 65536) return fail(DQ_ERR_SHAPE, "Ci must be <= 65536 for few-row products");
    DeviceGuard dg(w->device);
    if (!dg.ok) return fail(DQ_ERR_DEVICE, "hipSetDevice failed");
    auto* a = new (std::nothrow) dq_rows();
    if (!a) return fail(DQ_ERR_OUT_OF_MEMORY, "host allocation failed");
    std::unique_ptr<dq_rows, void (*)(dq_rows*)> guard(a, free_rows);
    a->device = w->device;
    a->max_rows = max_rows;
    a->Ci = w->Ci;
    a->Co = w->Co;
    a->Kp = w->Kp;
    a->rp = w->rp;
    size_t bytes = 0;
    int64_t floats = 0, units = 0;                      // the largest need of any row count up to max_rows
    for (int64_t n = 16; n < max_rows + 16; n += 16)
        for (const int parts : {1, 3}) {
            const SplitPlan p = plan_split(n, w->Co, (int)(w->Kp / 128), w->rp, parts);
            floats = std::max(floats, p.sum_floats());
            units = std::max(units, p.units());
            a->plans[parts > 1][n / 16 - 1] = p;
        }
    hipError_t e;
    if ((e = zalloc(&a->sums, (size_t)floats, &bytes)) != hipSuccess ||
        (e = zalloc(&a->arrivals, (size_t)units, &bytes)) != hipSuccess)
        return hip_fail(e, "hipMalloc workspace");
    if ((e = hipDeviceSynchronize()) != hipSuccess) return hip_fail(e, "workspace init");
    *out = guard.release();
    return DQ_OK;
}

void dq_rows_destroy(dq_rows* a) { free_rows(a); }

dq_status dq_linear_rows(const dq_weights* w, const void* x_dev, dq_dtype dt, int64_t ldx, int64_t N, dq_rows* a,
                         void* y_dev, dq_dtype ydt, int64_t ldy, void* stream) {
    set_error("");
    const dq_status st = check_rows(w, a, N, y_dev, ydt, ldy);
    if (st != DQ_OK) return st;
    if (dt != DQ_F32 && dt != DQ_BF16) return fail(DQ_ERR_INVALID_ARG, "unknown dtype");
    if (N == 0) return DQ_OK;
    if (!x_dev) return fail(DQ_ERR_INVALID_ARG, "x_dev is NULL");
    if ((uintptr_t)x_dev % 16 != 0) return fail(DQ_ERR_INVALID_ARG, "x_dev must be 16-byte aligned");
    if (ldx < w->Ci || ldx > (int64_t(1) << 40) / N || ldx * (dt == DQ_BF16 ? 2 : 4) % 16 != 0)
        return fail(DQ_ERR_SHAPE, "the row stride of x must be at least Ci and a multiple of 16 bytes");
    const int64_t xs = dt == DQ_BF16 ? 2 : 4, ys = ydt == DQ_BF16 ? 2 : 4;
    if (overlap({x_dev, N, ldx * xs, w->Ci * xs}, {y_dev, N, ldy * ys, w->Co * ys})) return fail(DQ_ERR_INVALID_ARG, "y_dev overlaps x_dev");
    DeviceGuard dg(a->device);
    if (!dg.ok) return fail(DQ_ERR_DEVICE, "hipSetDevice failed");
    RowsArgs r = rows_args(w, a, N, y_dev, ydt, ldy);
    r.x = x_dev;
    r.ldx = ldx;
    const SplitPlan& p = a->plans[dt == DQ_F32][(N - 1) / 16];
    const hipError_t e = dt == DQ_BF16 ? launch_rows_product<X_BF16>(r, p, (hipStream_t)stream)
                                       : launch_rows_product<X_F32>(r, p, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "product launch");
    return DQ_OK;
}

dq_status dq_linear_rows8(const dq_weights* w, const uint8_t* codes_dev, const uint8_t* scales_dev, int64_t N, dq_rows* a,
                          void* y_dev, dq_dtype ydt, int64_t ldy, void* stream) {
    set_error("");
    const dq_status st = check_rows(w, a, N, y_dev, ydt, ldy);
    if (st != DQ_OK) return st;
    if (N == 0) return DQ_OK;
    if (!codes_dev || !scales_dev) return fail(DQ_ERR_INVALID_ARG, "codes_dev or scales_dev is NULL");
    if ((uintptr_t)codes_dev % 8 != 0) return fail(DQ_ERR_INVALID_ARG, "codes_dev must be 8-byte aligned");
    const int64_t ys = ydt == DQ_BF16 ? 2 : 4;
    const Span y{y_dev, N, ldy * ys, w->Co * ys};
    if (overlap({codes_dev, N, w->Ci, w->Ci}, y) || overlap({scales_dev, N, w->Ci / 32, w->Ci / 32}, y))
        return fail(DQ_ERR_INVALID_ARG, "y_dev overlaps the codes or scales");
    DeviceGuard dg(a->device);
    if (!dg.ok) return fail(DQ_ERR_DEVICE, "hipSetDevice failed");
    RowsArgs r = rows_args(w, a, N, y_dev, ydt, ldy);
    r.x = codes_dev;
    r.xs = scales_dev;
    const hipError_t e = launch_rows_product<X_MX8>(r, a->plans[0][(N - 1) / 16], (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "product launch");
    return DQ_OK;
}

}  // extern "C"
