// dq_rmsnorm8: residual addition, root-mean-square norm and MX-FP8 encoding
// of token rows in one pass.
//
//   h = x + r, rounded to the stream's type;  s = sum_c h_c^2 in fp64
//   f = fl32(1 / sqrt(s / C + eps)), formed in fp64 and rounded once
//   v_c = fl32(fl32(h_c f) g_c);  MX-FP8 of v per 32 (or 64) channels
//
// The sum of squares is kept in fp64, in an order that goes by C alone: 8
// channels one by one, and such chunks pairwise by the bits of their place,
// lowest first.  So a row's results do not depend on the rows beside it,
// whichever form they take.  Every later step is one fp32 rounding per element.
// Another order moves the sum by some 2^-54 of it, and f by one unit in its
// last place where it lies that near to a border of two fp32 values: about one
// row in 10^9.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "dq.h"
#include "dq_device.h"
#include "dq_internal.h"
#include "dq_stream.h"

namespace dq {
namespace {

constexpr int MAX_NORM_C = 32768;

struct NormArgs {
    const void* x;
    const void* r;      // residual or null
    const void* g;      // gain or null (ones)
    void* h;            // x + r, or null
    void* y;            // v in the stream's type, or null
    uint8_t* codes;     // or null
    uint8_t* scales;
    long long first, N, ldx, ldr, ldh, ldy;   // first: row of the launch's first block
    int C, wide;        // wide: one scale for 64 channels
    int g_bf16;
    double eps;
};

__device__ __forceinline__ void load_gain(const NormArgs& a, int c, float* g) {
    if (!a.g) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = 1.0f;
    } else if (a.g_bf16) {
        Stream<uint16_t>::load((const uint16_t*)a.g + 8 * c, g);
    } else {
        Stream<float>::load((const float*)a.g + 8 * c, g);
    }
}

// The wave's sums of CH values, value i in lane i: from the first two steps on
// a lane carries on with one value (its place's lowest bits), which takes half
// the additions that each value by itself would (1024 x 5120 with plain values
// 9.4 -> 9.2 us).  Lanes from 4 on hold sums in other orders.
template <int CH>
__device__ __forceinline__ double sum_wave(const double* q, int t) {
    if constexpr (CH == 1) return sum_lanes<64>(q[0]);
    const bool odd = t & 1, upper = t & 2;
    double v = (odd ? q[1 % CH] : q[0]) + moved<0xB1>(odd ? q[0] : q[1 % CH]);
    if constexpr (CH > 2) {
        const double q3 = CH > 3 ? q[3 % CH] : 0.0;
        const double u = (odd ? q3 : q[2 % CH]) + moved<0xB1>(odd ? q[2 % CH] : q3);
        v = (upper ? u : v) + moved<0x4E>(upper ? v : u);
    } else {
        v += moved<0x4E>(v);
    }
    v += moved<0x12C>(v);                              // row rotated: the lane 4 places on
    v += moved<0x128>(v);                              // ... 8 places on
    return add_half(add_row(v));
}

// A row is held in registers by TPR threads, CH chunks of 8 channels each
// (chunk i of thread t: channels 8 (i TPR + t) ..), so it is read once; a
// group of 32 channels is 4 neighbouring lanes' chunk.
// Many rows are bound by HBM: 75600 x 5120 bf16 moves 2.72 GB in 464 us, 5.9
// TB/s (a copy of 1 GiB reaches 4.8), 32760 x 1536 fp32 44 us, 5.7 TB/s.  One
// row is bound by its chain of two loads, the sum across 16 waves and the
// stores: 1 x 5120 2.7 us, where an empty kernel takes 2.3.
template <class T, int TPR, int CH, bool NT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm8(NormArgs a) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    constexpr int WPR = TPR / 64;                   // waves to a row (0: several rows to a wave)
    const int t = threadIdx.x % TPR;
    const long long row = a.first + (long long)blockIdx.x * RPB + threadIdx.x / TPR;
    const bool live = row < a.N;
    const int nch = a.C >> 3;
    float h[CH][8];
    double q[CH];                                   // sums of squares of the chunks
#pragma unroll
    for (int i = 0; i < CH; ++i) q[i] = 0.0;
    if (live) {
        const T* xp = (const T*)a.x + row * a.ldx;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = i * TPR + t;
            if (c < nch) {
                Stream<T>::load(xp + 8 * c, h[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
            }
        }
        if (a.r) {
            const T* rp = (const T*)a.r + row * a.ldr;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = i * TPR + t;
                if (c < nch) {
                    float r[8];
                    Stream<T>::load(rp + 8 * c, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[i][j] = Stream<T>::round(h[i][j] + r[j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) q[i] = __builtin_fma((double)h[i][j], (double)h[i][j], q[i]);
    }
    double s;
    if constexpr (WPR > 1) {                        // (block of 64 chunks i WPR + w)
        static_assert(RPB == 1 && CH * WPR <= 64);
        __shared__ double part[CH * WPR];
        s = sum_wave<CH>(q, t);
        if ((t & 63) < CH) part[(t & 63) * WPR + (t >> 6)] = s;
        __syncthreads();
        s = (t & 63) < CH * WPR ? part[t & 63] : 0.0;
        s = first_lane(sum_lanes<(CH * WPR > 32 ? 64 : CH * WPR > 16 ? 32 : CH * WPR > 8 ? 16 : 8)>(s));
    } else if constexpr (CH > 1) {
        s = sum_wave<CH>(q, t);
        s = first_lane(sum_lanes<4>((t & 3) < CH ? s : 0.0));
    } else {
        s = sum_lanes<(TPR < 64 ? TPR : 64)>(q[0]);
    }
    if (!live) return;
    const float f = (float)(1.0 / sqrt(s / (double)a.C + a.eps));
    if (a.h) {
        T* hp = (T*)a.h + row * a.ldh;
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (i * TPR + t < nch) Stream<T>::template store<NT>(hp + 8 * (i * TPR + t), h[i]);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * TPR + t;
        if (c >= nch) continue;                     // (whole groups: C % 32 == 0, or % 64 with wide scales)
        float g[8], v[8];
        load_gain(a, c, g);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = (h[i][j] * f) * g[j];
            top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);   // (magnitudes order like their bits)
        }
        if (a.y) Stream<T>::template store<NT>((T*)a.y + row * a.ldy + 8 * c, v);
        if (!a.codes) continue;
        uint32_t bad = 0;                           // infinite or NaN elements: the NaN code, not part of the scale
        if (top >= 0x7f800000u) {
            top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t m = __float_as_uint(v[j]) & 0x7fffffffu;
                if (m >= 0x7f800000u) {
                    bad |= 1u << j;
                    v[j] = 0.0f;
                } else {
                    top = max(top, m);
                }
            }
        }
        top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
        if (a.wide) top = max(top, (uint32_t)__shfl_xor((int)top, 4, 64));
        const int e = mx_exp_fp8(__uint_as_float(top));
        v2w d = encode8(v, pow2f(e));
        if (bad) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (bad >> j & 1) d[0] |= 0x7fu << (8 * j);
                if (bad >> (j + 4) & 1) d[1] |= 0x7fu << (8 * j);
            }
        }
        put<NT>(a.codes + row * a.C + 8 * c, d);
        if ((t & 3) == 0) a.scales[row * (a.C >> 5) + (c >> 2)] = (uint8_t)(e + 127);
    }
}

// C / 8 chunks over TPR threads: MIN to MAX each.  A launch takes fewer than
// 2^32 threads, so more rows than that are several launches.
template <class T, int TPR, int MIN, int MAX, bool NT>
hipError_t launch_norm(NormArgs a, hipStream_t st) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1, THREADS = TPR < 256 ? 256 : TPR;
    constexpr long long MOST = (1ll << 31) / THREADS;
    const int ch = (a.C / 8 + TPR - 1) / TPR;
    const auto go = [&](unsigned grid) {
        if constexpr (MIN <= 1 && MAX > 1) if (ch == 1) return launch(k_rmsnorm8<T, TPR, 1, NT>, grid, THREADS, st, a);
        if constexpr (MIN <= 2 && MAX > 2) if (ch == 2) return launch(k_rmsnorm8<T, TPR, 2, NT>, grid, THREADS, st, a);
        if constexpr (MIN <= 3 && MAX > 3) if (ch == 3) return launch(k_rmsnorm8<T, TPR, 3, NT>, grid, THREADS, st, a);
        return launch(k_rmsnorm8<T, TPR, MAX, NT>, grid, THREADS, st, a);
    };
    hipError_t e = hipSuccess;
    for (; a.first < a.N && e == hipSuccess; a.first += MOST * RPB) e = go((unsigned)std::min(MOST, (a.N - a.first + RPB - 1) / RPB));
    return e;
}

// Rows of up to 64 chunks: one to a wave, or several, with as many lanes to a
// row as it has chunks.  In bf16 with a residual, by 256 threads a row for few
// rows and 64 for many / by these: 4096 x 128 5.6 / 3.0 us, 16384 x 64 14.9 / 3.3,
// 524288 x 128 221 / 81, 1024 x 512 3.3 / 3.0; 65536 x 512 43.9 / 43.0.
template <class T, bool NT>
hipError_t launch_short(const NormArgs& a, hipStream_t st) {
    if (a.C <= 64) return launch_norm<T, 8, 1, 1, NT>(a, st);
    if (a.C <= 128) return launch_norm<T, 16, 1, 1, NT>(a, st);
    if (a.C <= 256) return launch_norm<T, 32, 1, 1, NT>(a, st);
    return launch_norm<T, 64, 1, 1, NT>(a, st);
}

// Few longer rows are bound by their own latency, so a row gets as many threads as it
// has chunks; many by HBM, so a thread holds up to four chunks, and the
// outputs bypass the caches.  Measured in bf16 with a residual, few / many form:
//   1 x 5120 3.1 / 4.4 us; 64 x 1536 2.9 / 4.7 us; 256 x 5120 with plain values
//   4.5 / 5.3 us; 1024 x 5120 the same 11.1 / 9.2 us; 4096 x 1536 10.6 / 9.3 us.
// Bypassing stores on 75600 x 5120: 480 -> 466 us (5.8 TB/s); bypassing loads
// as well gain another 2 % there, but lose 12 % where the rows are still in the
// memory-side cache (32760 x 1536 fp32: 44 -> 49 us), so they stay plain.
// Threads to a long row: 20000 x 13824 takes 358 us with 512, 368 us with 256.
template <class T>
hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
    const bool few = a.N * a.C <= (3ll << 20);
    if (a.C <= 512) return few ? launch_short<T, false>(a, st) : launch_short<T, true>(a, st);
    if (few) return a.C <= 2048 ? launch_norm<T, 256, 1, 1, false>(a, st) : launch_norm<T, 1024, 1, 4, false>(a, st);
    if (a.C <= 2048) return launch_norm<T, 64, 2, 4, true>(a, st);
    if (a.C <= 8192) return launch_norm<T, 256, 2, 4, true>(a, st);
    if (a.C <= 16384) return launch_norm<T, 512, 3, 4, true>(a, st);
    return launch_norm<T, 1024, 3, 4, true>(a, st);
}

}  // namespace

}  // namespace dq

using namespace dq;

extern "C" dq_status dq_rmsnorm8(const void* x_dev, int64_t ldx, const void* res_dev, int64_t ldr, dq_dtype dt,
                                 const void* gain_dev, dq_dtype gain_dt, double eps, int64_t N, int64_t C, int32_t group,
                                 void* h_dev, int64_t ldh, uint8_t* codes_dev, uint8_t* scales_dev, void* y_dev,
                                 int64_t ldy, int32_t device, void* stream) {
    set_error("");
    if (dt != DQ_F32 && dt != DQ_BF16) return fail(DQ_ERR_INVALID_ARG, "unknown dtype");
    if (gain_dev && gain_dt != DQ_F32 && gain_dt != DQ_BF16) return fail(DQ_ERR_INVALID_ARG, "unknown gain dtype");
    if (group != 32 && group != 64) return fail(DQ_ERR_INVALID_ARG, "group must be 32 or 64");
    if (!(eps > 0.0) || !std::isfinite(eps) || eps < 1e-60) return fail(DQ_ERR_INVALID_ARG, "eps must be finite and at least 1e-60");
    if (C < 32 || C % 32 != 0 || C > MAX_NORM_C) return fail(DQ_ERR_SHAPE, "C must be a multiple of 32 in [32, 32768]");
    if (C % group != 0) return fail(DQ_ERR_SHAPE, "group must divide C");
    if (N < 0 || N > (int64_t(1) << 31) - 256) return fail(DQ_ERR_SHAPE, "N must be in [0, 2^31 - 256]");
    if ((codes_dev == nullptr) != (scales_dev == nullptr)) return fail(DQ_ERR_INVALID_ARG, "codes and scales come together");
    if (N == 0) return DQ_OK;
    if (!x_dev) return fail(DQ_ERR_INVALID_ARG, "x_dev is NULL");
    if (!codes_dev && !y_dev) return fail(DQ_ERR_INVALID_ARG, "no output: give codes and scales, or y");
    if (h_dev && !res_dev) return fail(DQ_ERR_INVALID_ARG, "h_dev without a residual");
    const int64_t esz = dt == DQ_BF16 ? 2 : 4, lim = int64_t(1) << 40;
    const struct { const void* p; int64_t ld; const char* name; } rows[] = {
        {x_dev, ldx, "x_dev"}, {res_dev, ldr, "res_dev"}, {h_dev, ldh, "h_dev"}, {y_dev, ldy, "y_dev"}};
    for (const auto& b : rows) {
        if (!b.p) continue;
        if ((uintptr_t)b.p % 16 != 0) return fail(DQ_ERR_INVALID_ARG, std::string(b.name) + " must be 16-byte aligned");
        if (b.ld < C || b.ld > lim / N || b.ld * esz % 16 != 0)
            return fail(DQ_ERR_SHAPE, std::string(b.name) + ": the row stride must be at least C and a multiple of 16 bytes");
    }
    if ((uintptr_t)gain_dev % 16 != 0) return fail(DQ_ERR_INVALID_ARG, "gain_dev must be 16-byte aligned");
    if ((uintptr_t)codes_dev % 8 != 0) return fail(DQ_ERR_INVALID_ARG, "codes_dev must be 8-byte aligned");
    // (a thread reads its elements of x and the residual before it writes the
    // same elements, so h or y may be one of them; nothing else may share memory)
    const struct { Span s; const char* name; } all[] = {
        {{x_dev, N, ldx * esz, C * esz}, "x_dev"}, {{res_dev, N, ldr * esz, C * esz}, "res_dev"},
        {{gain_dev, 1, C * 4, C * (gain_dt == DQ_BF16 ? 2 : 4)}, "gain_dev"},
        {{h_dev, N, ldh * esz, C * esz}, "h_dev"}, {{y_dev, N, ldy * esz, C * esz}, "y_dev"},
        {{codes_dev, N, C, C}, "codes_dev"}, {{scales_dev, N, C / 32, C / 32}, "scales_dev"}};
    for (int o = 3; o < 7; ++o)
        for (int i = 0; i < o; ++i) {
            const bool in_place = o < 5 && i < 2 && all[o].s.p == all[i].s.p && all[o].s.pitch == all[i].s.pitch;
            if (!in_place && overlap(all[o].s, all[i].s))
                return fail(DQ_ERR_INVALID_ARG, std::string(all[o].name) + " overlaps " + all[i].name);
        }
    const dq_status st = known_device(device);
    if (st != DQ_OK) return st;
    DeviceGuard dg(device);
    if (!dg.ok) return fail(DQ_ERR_DEVICE, "hipSetDevice failed");
    const NormArgs a{x_dev, res_dev, gain_dev, h_dev, y_dev, codes_dev, scales_dev, 0, (long long)N, (long long)ldx,
                     (long long)ldr, (long long)ldh, (long long)ldy, (int)C, group == 64, gain_dt == DQ_BF16, eps};
    const hipError_t e = dt == DQ_BF16 ? launch_norm<uint16_t>(a, (hipStream_t)stream) : launch_norm<float>(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "norm launch");
    return DQ_OK;
}
