// dq_norm_rope, dq_kv_write, dq_kv_read, dq_rope_table: the heads of queries,
// keys and values between their projection and attention.
//
//   f = fl32(1 / sqrt(sum x_c^2 / C + eps)), over a head or the whole row (fp64)
//   v_c = fl32(fl32(x_c f) g_c)
//   a' = fl32(fl32(a c) - fl32(b s)), b' = fl32(fl32(a s) + fl32(b c))
// then one rounding to the output's type, or MX codes of 32 channels in the
// cache's pages.  Every step is one fp32 operation and the sums' order goes by C
// alone, so codes and values are defined to the bit.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "dq.h"
#include "dq_heads.h"
#include "dq_stream.h"

namespace dq {
namespace {

constexpr int64_t MAX_ROWS = (int64_t(1) << 31) - 256;
constexpr int MAX_C = 32768, MAX_PAIRS = 128;

enum Kind { TO_BF16, TO_F32, TO_FP8, TO_FP4 };

// One of q, k, v: rows of nch chunks of 8 channels.
struct Part {
    const void* x;
    long long ld;
    const void* g;          // gain or null (ones)
    void* y;                // rows (TO_BF16, TO_F32), or the cache's codes
    long long ldy;
    uint8_t* scales;
    int nch, segs;          // blocks to a row
    int kind, norm, turn;
};

struct Turn {
    const float* table[3];
    int count[3], positions[3];
    int pairs, axes, interleaved;
    const int* pos;         // [N][axes] or null
};

struct HeadsArgs {
    Part part[3];
    Turn turn;
    Pages pages;            // (pages.first null: no cache)
    long long N, first;     // first: row of the launch's first block
    double eps;
    int lph;                // lanes (chunks) to a head
    int tpr;                // threads to a row, a power of two
    int g_bf16;
};

// Sums over groups of n neighbouring lanes (n a power of two, 4 to 64), pairwise by the lanes' bits, lowest first.
__device__ __forceinline__ double sum_group(double v, int n) {
    v += moved<0xB1>(v);
    v += moved<0x4E>(v);
    if (n > 4) v += moved<0x141>(v);
    if (n > 8) v += moved<0x140>(v);
    if (n > 16) v = add_row(v);
    if (n > 32) v = add_half(v);
    return v;
}

__device__ __forceinline__ float factor_of(double mean, double eps) { return (float)(1.0 / sqrt(mean + eps)); }

// A kernel's argument as a value of its own: the compiler would else turn a
// choice between two arguments into a load from the chosen one's address.
__device__ __forceinline__ int fixed(int v) { return __builtin_amdgcn_readfirstlane(v); }
typedef const __attribute__((address_space(1))) float* Table;
__device__ __forceinline__ Table fixed(const float* p) {
    const uint64_t v = (uint64_t)(uintptr_t)p;
    return (Table)(uintptr_t)((uint64_t)(uint32_t)fixed((int)(v >> 32)) << 32 | (uint32_t)fixed((int)v));
}

// The coefficients of one lane's 8 channels at one row: out = v c + partner s,
// for channels of `on`.
struct Coef {
    float c[8], s[8];
    uint32_t on;            // channels that are rotated
};
// (cos, sin) of COUNT pairs from j0 on, all loads issued before any is used
// (pairs past the last: the last's).
template <int COUNT>
__device__ __forceinline__ void pairs_from(const Turn& r, const int (&at)[3], int j0, float2 (&cs)[COUNT]) {
    typedef const __attribute__((address_space(1))) v2f* From;
    const float nan = __builtin_nanf("");
    const int n0 = fixed(r.count[0]), n1 = fixed(r.count[1]), e0 = n0, e1 = n0 + n1, last = fixed(r.pairs) - 1;
    const bool in0 = (uint32_t)at[0] < (uint32_t)r.positions[0];
    // (each axis' row from where pair 0 would be, at position 0 where its own is outside)
    const Table w0 = fixed(r.table[0]) + 2 * ((size_t)(in0 ? (uint32_t)at[0] : 0u) * n0);
    v2f got[COUNT];
    if (r.axes == 1) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) got[i] = *(From)(w0 + 2 * min(j0 + i, last));
#pragma unroll
        for (int i = 0; i < COUNT; ++i) cs[i] = in0 ? make_float2(got[i][0], got[i][1]) : make_float2(nan, nan);
        return;
    }
    const bool in1 = (uint32_t)at[1] < (uint32_t)r.positions[1], in2 = (uint32_t)at[2] < (uint32_t)r.positions[2];
    const Table w1 = fixed(r.table[1]) + 2 * ((long long)((size_t)(in1 ? (uint32_t)at[1] : 0u) * n1) - e0);
    const Table w2 = fixed(r.table[2]) + 2 * ((long long)((size_t)(in2 ? (uint32_t)at[2] : 0u) * fixed(r.count[2])) - e1);
    bool in[COUNT];
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        const int j = min(j0 + i, last);
        const bool a1 = j >= e0, a2 = j >= e1;
        got[i] = *(From)((a2 ? w2 : a1 ? w1 : w0) + 2 * j);
        in[i] = a2 ? in2 : a1 ? in1 : in0;
    }
#pragma unroll
    for (int i = 0; i < COUNT; ++i) cs[i] = in[i] ? make_float2(got[i][0], got[i][1]) : make_float2(nan, nan);
}
__device__ __forceinline__ Coef coefficients(const Turn& r, const int (&at)[3], int lane) {
    Coef k;
    const int turned = 2 * r.pairs - 8 * lane;      // of the lane's channels, if pairs are side by side
    if (r.interleaved) {
        float2 cs[4];
        pairs_from<4>(r, at, 4 * lane, cs);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            k.c[2 * i] = k.c[2 * i + 1] = cs[i].x;
            k.s[2 * i] = -cs[i].y;
            k.s[2 * i + 1] = cs[i].y;
        }
        k.on = turned >= 8 ? 0xffu : turned <= 0 ? 0u : (1u << turned) - 1;
    } else {
        float2 cs[8];
        const bool second = 8 * lane >= r.pairs;
        pairs_from<8>(r, at, 8 * lane - (second ? r.pairs : 0), cs);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            k.c[i] = cs[i].x;
            k.s[i] = second ? cs[i].y : -cs[i].y;
        }
        k.on = turned > 0 ? 0xffu : 0u;
    }
    return k;
}

// MX codes of the lane's 8 values in its group of 4 lanes (32 channels): FP8 in
// d[0..1], FP4 in d[0]; returns the scale code.
template <bool FP4>
__device__ __forceinline__ uint32_t encode_group(float* v, v2w& d) {
    uint32_t top = 0, bad = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
    if (top >= 0x7f800000u) {                       // infinite or NaN: not part of the scale
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
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xF, 0xF, true));
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xF, 0xF, true));
    if constexpr (FP4) {
        const int e = mx_exp_fp4(__uint_as_float(top));
        const float scale = pow2f(e);
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
        d = v2w{w, 0u};
        bad |= (uint32_t)__builtin_amdgcn_mov_dpp((int)bad, 0xB1, 0xF, 0xF, true);
        bad |= (uint32_t)__builtin_amdgcn_mov_dpp((int)bad, 0x4E, 0xF, 0xF, true);
        return bad ? 255u : (uint32_t)(e + 127);
    } else {
        const int e = mx_exp_fp8(__uint_as_float(top));
        d = encode8(v, pow2f(e));
        if (bad) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (bad >> j & 1) d[0] |= 0x7fu << (8 * j);
                if (bad >> (j + 4) & 1) d[1] |= 0x7fu << (8 * j);
            }
        }
        return (uint32_t)(e + 127);
    }
}

__device__ __forceinline__ void load_gains(const HeadsArgs& a, const Part& p, int lane, int c, float* g) {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 1.0f;
    if (!p.g) return;
    const int at = 8 * (p.norm == DQ_NORM_HEAD ? lane : min(c, p.nch - 1));
    if (a.g_bf16) Stream<uint16_t>::load((const uint16_t*)p.g + at, g);
    else Stream<float>::load((const float*)p.g + at, g);
}

// What bounds it: HBM where there are many rows (32760 x 12 heads 45.5 us a call among others, 4.4 TB/s, the kernel
// by itself 47 to 53; 75600 x 40 fp32 heads 394, 5.9 TB/s);
// launch and a chain of three loads where there are few (1 x 40 heads 3.5 us).
// A row's part is held in registers by tpr threads (of several blocks, where no
// sum crosses them), CH chunks of 8 channels each, chunk i of thread t: i tpr + t.
// tpr is a multiple of the lanes to a head, so a thread's chunks are at one place
// of their heads and share the rotation's coefficients.
// Loads come in rounds without a branch between them (rows and chunks past the
// end read the last one): the row's values, gains and sequences, then its
// coefficients and page.
template <class T, int CH>
__global__ __launch_bounds__(1024) void k_heads(HeadsArgs a) {
    __shared__ double sums[64];                     // [row of the block][block of 64 chunks]
    // (the arguments' cache lines, all at once)
    asm volatile("" ::"s"(a.part[0].nch), "s"(a.part[1].ldy), "s"(a.part[2].g), "s"(a.part[2].turn), "s"(a.turn.table[1]), "s"(a.pages.first),
                 "s"(a.N), "s"(a.g_bf16));
    int seg = blockIdx.y, pi = 0;
    if (seg >= a.part[0].segs) {
        seg -= a.part[0].segs, pi = 1;
        if (seg >= a.part[1].segs) seg -= a.part[1].segs, pi = 2;
    }
    const Part& p = a.part[pi];
    const int tpr = a.tpr, shift = __builtin_ctz(tpr), t = threadIdx.x & (tpr - 1), sub = threadIdx.x >> shift;
    const long long row0 = a.first + (long long)blockIdx.x * (blockDim.x >> shift), row = row0 + sub, near = min(row, a.N - 1);
    const bool live = row < a.N;
    const int c0 = seg * tpr * CH + t, lane = t & (a.lph - 1);
    typename Stream<T>::Raw raw[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) raw[i] = Stream<T>::raw((const T*)p.x + near * p.ld + 8 * min(c0 + i * tpr, p.nch - 1));
    float gain[8];          // (of a thread's one chunk)
    if constexpr (CH == 1) load_gains(a, p, lane, c0, gain);
    int pos[3] = {(int)near, 0, 0};
    if (p.turn && a.turn.pos) {
#pragma unroll
        for (int i = 0; i < 3; ++i) pos[i] = a.turn.pos[near * a.turn.axes + min(i, a.turn.axes - 1)];
    }
    Place at{-1, -1};
    if (a.pages.first) {
        const Starts starts = starts_of(a.pages);
        at = place_of(a.pages, starts, row0 + ((threadIdx.x & ~63u) >> shift), tpr);
        if (!a.turn.pos) pos[0] = at.t;
    }
    Coef k{};
    if (p.turn) k = coefficients(a.turn, pos, lane);
    float v[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) Stream<T>::values(raw[i], v[i]);
    if (p.norm != DQ_NORM_NONE) {
        double q[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            q[i] = 0.0;
            if (c0 + i * tpr < p.nch) {
#pragma unroll
                for (int j = 0; j < 8; ++j) q[i] = __builtin_fma((double)v[i][j], (double)v[i][j], q[i]);
            }
        }
        float f[CH];
        if (p.norm == DQ_NORM_HEAD) {
            // (a head has a power of two of channels: its mean by an exact product.)  All
            // of a head's lanes hold its sum, so each forms the factor of one of
            // the thread's CH heads and they are exchanged: a square root
            // and a division in fp64 take as long as the rest
            const double share = 1.0 / (double)(8 * a.lph);
#pragma unroll
            for (int i = 0; i < CH; ++i) q[i] = sum_group(q[i], a.lph) * share;
            if (CH == 1 || a.lph < CH) {
#pragma unroll
                for (int i = 0; i < CH; ++i) f[i] = factor_of(q[i], a.eps);
            } else {
                double mine = q[0];
#pragma unroll
                for (int i = 1; i < CH; ++i) mine = lane == i ? q[i] : mine;
                const float g = factor_of(mine, a.eps);
#pragma unroll
                for (int i = 0; i < CH; ++i) f[i] = __shfl(g, (int)(threadIdx.x & 63) - lane + i, 64);
            }
        } else {
            // blocks of 64 chunks by their lanes, then the blocks by their number's bits
            double s;
            if (CH == 1 && tpr <= 64) {
                s = sum_group(q[0], tpr);
            } else {
                const int waves = tpr >> 6;         // (tpr >= 64 where a row takes more than one chunk a thread)
                double* mine = sums + sub * (CH * waves);
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const double b = sum_group(q[i], 64);
                    if ((t & 63) == 0) mine[i * waves + (t >> 6)] = b;
                }
                __syncthreads();
                s = sum_group((t & 63) < CH * waves ? mine[t & 63] : 0.0, 64);
            }
            const float g = factor_of(s / (double)(8 * p.nch), a.eps);
#pragma unroll
            for (int i = 0; i < CH; ++i) f[i] = g;
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if constexpr (CH > 1) load_gains(a, p, lane, c0 + i * tpr, gain);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = (v[i][j] * f[i]) * gain[j];
        }
    }
    if (p.turn) {
        const int half = a.turn.pairs >> 3;         // lanes between partners
        const int other = (int)((threadIdx.x & 63) - lane) + (lane < half ? lane + half : lane < 2 * half ? lane - half : lane);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = a.turn.interleaved ? v[i][j ^ 1] : __shfl(v[i][j], other, 64);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float r = v[i][j] * k.c[j] + o[j] * k.s[j];
                v[i][j] = k.on >> j & 1 ? r : v[i][j];
            }
        }
    }
    if (!live) return;
    if (p.kind <= TO_F32) {
        if (a.pages.first && at.t == NOWHERE) return;   // a row of no sequence
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = c0 + i * tpr;
            if (c >= p.nch) continue;
            if (p.kind == TO_BF16) {
                uint16_t* y = (uint16_t*)p.y + row * p.ldy + 8 * c;
                Stream<uint16_t>::template store<false>(y, v[i]);
            } else {
                float* y = (float*)p.y + row * p.ldy + 8 * c;
                Stream<float>::template store<false>(y, v[i]);
            }
        }
        return;
    }
    if (at.page < 0) return;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = c0 + i * tpr;
        if (c >= p.nch) continue;                   // (whole heads, so whole groups)
        const long long tok = token_row(a.pages, at, c / a.lph);
        v2w d;
        uint32_t e;
        if (p.kind == TO_FP8) {
            e = encode_group<false>(v[i], d);
            *(v2w*)((uint8_t*)p.y + (tok * a.lph + lane) * 8) = d;
        } else {
            e = encode_group<true>(v[i], d);
            *(uint32_t*)((uint8_t*)p.y + (tok * a.lph + lane) * 4) = d[0];
        }
        if ((lane & 3) == 0) p.scales[tok * (a.lph >> 2) + (lane >> 2)] = (uint8_t)e;
    }
}

// ---- reading back ----
struct ReadArgs {
    const uint8_t* codes[2];
    const uint8_t* scales[2];
    void* y[2];
    long long ldy[2];
    Pages pages;
    long long N, first;
    int lph;                // lanes (chunks of 8 channels) to a head
    int nch, tpr, segs;     // chunks to a row; threads and workgroups to one
    int part0;              // 1: only values are read
};

// A thread decodes U chunks of 8 channels, tpr apart, of a row's keys and values
// (P: 2, or 1 of one of them), so one look at the page table serves 2 U loads, and
// a wave writes whole 128-byte lines of bf16: 32760 x 12 heads from HBM 57.6 us
// (5.3 TB/s).  With 16 channels to a thread, whose two stores leave every line
// half written, 72; with U 1, 63.5.
template <class T, int BITS, int P, int U>
__global__ __launch_bounds__(256) void k_read(ReadArgs a) {
    const int tpr = a.tpr, shift = __builtin_ctz(tpr), t = threadIdx.x & (tpr - 1);
    const long long row = a.first + (long long)blockIdx.x * (256 >> shift) + (threadIdx.x >> shift);
    const Place at = place_of(a.pages, starts_of(a.pages), row - ((threadIdx.x & 63) >> shift), tpr);
    if (row >= a.N || at.t == NOWHERE) return;
    constexpr int W = BITS == 8 ? 2 : 1;            // words of codes
    const int lane = t & (a.lph - 1), c0 = (int)blockIdx.y * tpr * U + t;
    uint32_t code[U][P][2] = {}, e[U][P] = {};
    if (at.page >= 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long tok = token_row(a.pages, at, min(c0 + u * tpr, a.nch - 1) / a.lph);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const uint32_t* p = (const uint32_t*)a.codes[a.part0 + i] + (tok * a.lph + lane) * W;
                if constexpr (BITS == 8) {
                    const v2w v = *((const v2w*)p);
                    code[u][i][0] = v[0], code[u][i][1] = v[1];
                } else {
                    code[u][i][0] = *p;
                }
                e[u][i] = a.scales[a.part0 + i][tok * (a.lph >> 2) + (lane >> 2)];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = c0 + u * tpr;
        if (c >= a.nch) continue;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float v[8];
            decode8_f32<BITS>(code[u][i], e[u][i], v);
            Stream<T>::template store<true>((T*)a.y[a.part0 + i] + row * a.ldy[a.part0 + i] + 8 * c, v);
        }
    }
}

struct TableArgs {
    double freq[MAX_PAIRS];
    float* table;
    long long total;
    int pairs;
};
__global__ __launch_bounds__(256) void k_table(TableArgs a) {
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < a.total; i += gridDim.x * 256ll) {
        const long long p = i / a.pairs;
        const double x = (double)p * a.freq[i - p * a.pairs];
        ((float2*)a.table)[i] = make_float2((float)cos(x), (float)sin(x));
    }
}

// ---- launches ----
int pow2_at_least(int n, int least) {
    int p = least;
    while (p < n) p *= 2;
    return p;
}

// Threads to a row of nch chunks (a power of two from `least` on) and chunks to a
// thread (up to 5; one, where a row takes less than a wave) that leave the fewest
// lanes idle; of equal ones the fewest threads.
void share_row(int nch, int least, int* tpr, int* ch) {
    int best = 1 << 30;
    for (int t = least; t <= 1024; t *= 2) {
        const int c = (nch + t - 1) / t;
        if (c > 5 || (c > 1 && t < 64)) continue;
        if (c * t < best) best = c * t, *tpr = t, *ch = c;
    }
}

template <class T>
hipError_t launch_heads(HeadsArgs a, int parts, hipStream_t st) {
    int nch = 0, row_norm = 0, ch = 1;
    for (int i = 0; i < parts; ++i) {
        nch = std::max(nch, a.part[i].nch);
        row_norm |= a.part[i].norm == DQ_NORM_ROW;
    }
    // Few chunks: one to a thread, for the shortest chain (of 5120 channels 1 row 2.9
    // us against 3.9, 200 rows 3.2 against 4.5); more: as share_row has it (800
    // rows, norm of the row 5.9 us against 7.9 with one to a thread).  All parts go
    // by the widest, so narrow keys leave most of their threads' chunks idle: 4096 rows
    // of 40 query and 8 key heads 42 us (their bytes 23), of 8 and 8 16 (9).
    const bool few = a.N * nch <= (1 << 17);
    if (few) {
        a.tpr = std::min(pow2_at_least(nch, a.lph), row_norm ? 1024 : 256);
        ch = row_norm ? (nch + a.tpr - 1) / a.tpr : 1;
    } else {
        share_row(nch, a.lph, &a.tpr, &ch);
    }
    int segs = 0;
    for (int i = 0; i < 3; ++i) {
        Part& p = a.part[i];
        p.segs = i >= parts ? 0 : (p.nch + a.tpr * ch - 1) / (a.tpr * ch);   // (1 with a norm of the row)
        segs += p.segs;
    }
    const int threads = std::max(256, a.tpr), rows = threads / a.tpr;
    const long long most = (1ll << 31) / threads;
    hipError_t e = hipSuccess;
    for (; a.first < a.N && e == hipSuccess; a.first += most * rows) {
        const dim3 grid((unsigned)std::min(most, (a.N - a.first + rows - 1) / rows), segs);
        switch (ch) {
            case 1: e = launch(k_heads<T, 1>, grid, threads, st, a); break;
            case 2: e = launch(k_heads<T, 2>, grid, threads, st, a); break;
            case 3: e = launch(k_heads<T, 3>, grid, threads, st, a); break;
            case 4: e = launch(k_heads<T, 4>, grid, threads, st, a); break;
            default: e = launch(k_heads<T, 5>, grid, threads, st, a); break;
        }
    }
    return e;
}

template <class T, int BITS, int P>
hipError_t launch_read(ReadArgs a, hipStream_t st) {
    // chunks to a thread and threads to a row that leave the fewest idle, of equal
    // ones the most (540 rows of 8 x 64 channels take as long with one chunk to a thread)
    int best = 1 << 30, per = 1;
    for (int u = 1; u <= 4; ++u)
        for (int t = u == 1 ? a.lph : 64; t <= 256; t *= 2) {
            const int n = (a.nch + t * u - 1) / (t * u);
            if (n * t * u <= best && (n == 1 || t >= 64)) best = n * t * u, a.tpr = t, a.segs = n, per = u;
        }
    const int rows = 256 / a.tpr;
    const long long most = (1ll << 31) / 256;
    hipError_t e = hipSuccess;
    const auto kernel = per == 1 ? k_read<T, BITS, P, 1> : per == 2 ? k_read<T, BITS, P, 2> :
                        per == 3 ? k_read<T, BITS, P, 3> : k_read<T, BITS, P, 4>;
    for (; a.first < a.N && e == hipSuccess; a.first += most * rows)
        e = launch(kernel, dim3((unsigned)std::min(most, (a.N - a.first + rows - 1) / rows), a.segs), 256u, st, a);
    return e;
}

// ---- checks ----
bool head_dim_ok(int d) { return d == 32 || d == 64 || d == 128 || d == 256; }

dq_status check_ops(const dq_head_ops* ops, int head_dim, Turn* t) {
    *t = Turn{};
    if (!ops) return fail(DQ_ERR_INVALID_ARG, "ops is NULL");
    if (ops->norm != DQ_NORM_NONE && ops->norm != DQ_NORM_HEAD && ops->norm != DQ_NORM_ROW) return fail(DQ_ERR_INVALID_ARG, "unknown norm");
    if (ops->norm != DQ_NORM_NONE) {
        if (ops->gain_dt != DQ_F32 && ops->gain_dt != DQ_BF16) return fail(DQ_ERR_INVALID_ARG, "unknown gain dtype");
        if (!std::isfinite(ops->eps) || !(ops->eps >= 1e-60)) return fail(DQ_ERR_INVALID_ARG, "eps must be finite and at least 1e-60");
    }
    const dq_rope* r = ops->rope;
    if (!r) return DQ_OK;
    if (r->axes < 1 || r->axes > 3) return fail(DQ_ERR_INVALID_ARG, "axes must be 1 to 3");
    if (r->interleaved != 0 && r->interleaved != 1) return fail(DQ_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    if (!ops->pos_dev && r->axes != 1) return fail(DQ_ERR_INVALID_ARG, "pos_dev may be NULL for one axis only");
    if ((uintptr_t)ops->pos_dev % 4 != 0) return fail(DQ_ERR_INVALID_ARG, "pos_dev must be 4-byte aligned");
    int64_t pairs = 0;
    for (int i = 0; i < 3; ++i) {
        if (i >= r->axes) {                         // (never chosen, but its address is formed)
            t->table[i] = t->table[0];
            t->positions[i] = 1;
            continue;
        }
        if (r->pairs[i] < 1 || r->pairs[i] > MAX_PAIRS) return fail(DQ_ERR_SHAPE, "an axis has 1 to 128 pairs");
        if (r->positions[i] < 1 || r->positions[i] >= int64_t(1) << 31) return fail(DQ_ERR_SHAPE, "positions must be in [1, 2^31)");
        if (!r->table_dev[i]) return fail(DQ_ERR_INVALID_ARG, "table_dev is NULL");
        if ((uintptr_t)r->table_dev[i] % 8 != 0) return fail(DQ_ERR_INVALID_ARG, "table_dev must be 8-byte aligned");
        pairs += r->pairs[i];
        t->table[i] = r->table_dev[i];
        t->count[i] = r->pairs[i];
        t->positions[i] = (int)r->positions[i];
    }
    if (2 * pairs > head_dim) return fail(DQ_ERR_SHAPE, "more pairs than half the head's channels");
    if (!r->interleaved && pairs % 8 != 0) return fail(DQ_ERR_SHAPE, "pairs of two halves must come in multiples of 8");
    t->pairs = (int)pairs;
    t->axes = r->axes;
    t->interleaved = r->interleaved;
    t->pos = ops->pos_dev;
    return DQ_OK;
}

struct RowsOf {                     // a caller's rows
    const void* p;
    int64_t ld, C;
    dq_dtype dt;
    const char* name;
    int64_t esz() const { return dt == DQ_BF16 ? 2 : 4; }
    Span span(int64_t N) const { return {p, N, ld * esz(), C * esz()}; }
};
dq_status check_row_array(const RowsOf& r, int64_t N) {
    if (r.dt != DQ_F32 && r.dt != DQ_BF16) return fail(DQ_ERR_INVALID_ARG, std::string("unknown dtype of ") + r.name);
    if (!r.p) return fail(DQ_ERR_INVALID_ARG, std::string(r.name) + " is NULL");
    if ((uintptr_t)r.p % 16 != 0) return fail(DQ_ERR_INVALID_ARG, std::string(r.name) + " must be 16-byte aligned");
    if (r.ld < r.C || r.ld > (int64_t(1) << 40) / N || r.ld * r.esz() % 16 != 0)
        return fail(DQ_ERR_SHAPE, std::string(r.name) + ": the row stride must be at least the row's width and a multiple of 16 bytes");
    return DQ_OK;
}
bool in_place(const RowsOf& a, const RowsOf& b) { return a.p == b.p && a.ld == b.ld && a.dt == b.dt; }

// Whether any of the outputs o meets one of the inputs i or another output.
struct Named {
    Span s;
    const char* name;
};
template <int O, int I>
const char* meets(const Named (&out)[O], const Named (&in)[I], std::string* with) {
    for (int o = 0; o < O; ++o) {
        for (int i = 0; i < I; ++i)
            if (overlap(out[o].s, in[i].s)) return *with = in[i].name, out[o].name;
        for (int i = 0; i < o; ++i)
            if (overlap(out[o].s, out[i].s)) return *with = out[i].name, out[o].name;
    }
    return nullptr;
}

Named flat(const void* p, int64_t bytes, const char* name) { return {{p, 1, bytes, bytes}, name}; }

Part part_of(const RowsOf& x, const void* gain, void* y, int64_t ldy, int kind, uint8_t* scales, int norm, bool turn) {
    return Part{x.p, (long long)x.ld, gain, y, (long long)ldy, scales, (int)(x.C / 8), 0, kind, norm, turn};
}

}  // namespace

dq_status check_kv(const dq_kv* kv) {
    if (!kv) return fail(DQ_ERR_INVALID_ARG, "kv is NULL");
    if (kv->bits != 8 && kv->bits != 4) return fail(DQ_ERR_INVALID_ARG, "bits must be 8 or 4");
    if (!head_dim_ok(kv->head_dim)) return fail(DQ_ERR_SHAPE, "head_dim must be 32, 64, 128 or 256");
    if (kv->heads < 1 || (int64_t)kv->heads * kv->head_dim > MAX_C) return fail(DQ_ERR_SHAPE, "heads * head_dim must be in [32, 32768]");
    if (kv->page_tokens < 16 || kv->page_tokens > 65536 || (kv->page_tokens & (kv->page_tokens - 1)))
        return fail(DQ_ERR_SHAPE, "page_tokens must be a power of two in [16, 65536]");
    if (kv->pages < 1 || kv->pages >= int64_t(1) << 31) return fail(DQ_ERR_SHAPE, "pages must be in [1, 2^31)");
    if (kv->pages > (int64_t(1) << 44) / ((int64_t)kv->heads * kv->page_tokens * kv->head_dim))
        return fail(DQ_ERR_SHAPE, "the cache is larger than 2^44 values");
    if (!kv->k_codes || !kv->k_scales || !kv->v_codes || !kv->v_scales) return fail(DQ_ERR_INVALID_ARG, "a cache array is NULL");
    if (((uintptr_t)kv->k_codes | (uintptr_t)kv->v_codes) % 16 != 0) return fail(DQ_ERR_INVALID_ARG, "the cache's codes must be 16-byte aligned");
    if (((uintptr_t)kv->k_scales | (uintptr_t)kv->v_scales) % 4 != 0) return fail(DQ_ERR_INVALID_ARG, "the cache's scales must be 4-byte aligned");
    return DQ_OK;
}

dq_status check_seqs(const dq_seqs* s) {
    if (!s) return fail(DQ_ERR_INVALID_ARG, "seqs is NULL");
    if (s->seqs < 1 || s->seqs > int64_t(1) << 20) return fail(DQ_ERR_SHAPE, "seqs must be in [1, 2^20]");
    if (s->pages_ld < 1 || s->pages_ld >= int64_t(1) << 31) return fail(DQ_ERR_SHAPE, "pages_ld must be in [1, 2^31)");
    if (!s->first_dev || !s->length_dev || !s->pages_dev) return fail(DQ_ERR_INVALID_ARG, "an array of the batch is NULL");
    if (((uintptr_t)s->first_dev | (uintptr_t)s->length_dev | (uintptr_t)s->pages_dev) % 4 != 0)
        return fail(DQ_ERR_INVALID_ARG, "the batch's arrays must be 4-byte aligned");
    return DQ_OK;
}

int64_t kv_code_bytes(const dq_kv* kv) { return kv->pages * kv->heads * kv->page_tokens * (kv->head_dim * kv->bits / 8); }
int64_t kv_scale_bytes(const dq_kv* kv) { return kv->pages * kv->heads * kv->page_tokens * (kv->head_dim / 32); }

Pages pages_of(const dq_kv* kv, const dq_seqs* s) {
    return Pages{s->first_dev, s->length_dev, s->pages_dev, (int)s->seqs, (int)s->pages_ld, (int)kv->pages,
                 __builtin_ctz((unsigned)kv->page_tokens), kv->heads};
}

}  // namespace dq

using namespace dq;

extern "C" {

dq_status dq_rope_table(const double* freq_host, int32_t pairs, int64_t positions, float* table_dev, int32_t device, void* stream) {
    set_error("");
    if (!freq_host || !table_dev) return fail(DQ_ERR_INVALID_ARG, "freq_host or table_dev is NULL");
    if (pairs < 1 || pairs > MAX_PAIRS) return fail(DQ_ERR_SHAPE, "an axis has 1 to 128 pairs");
    if (positions < 1 || positions >= int64_t(1) << 31) return fail(DQ_ERR_SHAPE, "positions must be in [1, 2^31)");
    if ((uintptr_t)table_dev % 8 != 0) return fail(DQ_ERR_INVALID_ARG, "table_dev must be 8-byte aligned");
    TableArgs a{};
    for (int i = 0; i < pairs; ++i) {
        if (!std::isfinite(freq_host[i])) return fail(DQ_ERR_INVALID_ARG, "a frequency is not finite");
        a.freq[i] = freq_host[i];
    }
    const dq_status st = known_device(device);
    if (st != DQ_OK) return st;
    DeviceGuard dg(device);
    if (!dg.ok) return fail(DQ_ERR_DEVICE, "hipSetDevice failed");
    a.table = table_dev;
    a.total = (long long)positions * pairs;
    a.pairs = pairs;
    const hipError_t e = launch(k_table, dim3((unsigned)std::min<long long>((a.total + 255) / 256, 65536)), 256u, (hipStream_t)stream, a);
    return e == hipSuccess ? DQ_OK : hip_fail(e, "table launch");
}

dq_status dq_norm_rope(const void* x_dev, int64_t ldx, dq_dtype dt, int64_t N, int32_t heads, int32_t head_dim,
                       const void* gain_dev, const dq_head_ops* ops, void* y_dev, int64_t ldy, dq_dtype ydt, int32_t device,
                       void* stream) {
    set_error("");
    if (!head_dim_ok(head_dim)) return fail(DQ_ERR_SHAPE, "head_dim must be 32, 64, 128 or 256");
    if (heads < 1 || (int64_t)heads * head_dim > MAX_C) return fail(DQ_ERR_SHAPE, "heads * head_dim must be in [32, 32768]");
    if (N < 0 || N > MAX_ROWS) return fail(DQ_ERR_SHAPE, "N must be in [0, 2^31 - 256]");
    HeadsArgs a{};
    dq_status st = check_ops(ops, head_dim, &a.turn);
    if (st != DQ_OK) return st;
    if (N == 0) return DQ_OK;
    const int64_t C = (int64_t)heads * head_dim;
    const RowsOf x{x_dev, ldx, C, dt, "x_dev"}, y{y_dev, ldy, C, ydt, "y_dev"};
    for (const RowsOf& r : {x, y})
        if ((st = check_row_array(r, N)) != DQ_OK) return st;
    const void* gain = ops->norm == DQ_NORM_NONE ? nullptr : gain_dev;
    if ((uintptr_t)gain % 16 != 0) return fail(DQ_ERR_INVALID_ARG, "gain_dev must be 16-byte aligned");
    const int64_t gains = ops->norm == DQ_NORM_HEAD ? head_dim : C;
    std::string with;
    const Named out[] = {{y.span(N), "y_dev"}};
    const Named in[] = {{in_place(x, y) ? Span{} : x.span(N), "x_dev"}, flat(gain, gains * (ops->gain_dt == DQ_BF16 ? 2 : 4), "gain_dev"),
                        flat(a.turn.pos, N * 4 * a.turn.axes, "pos_dev"),
                        flat(a.turn.table[0], 8ll * a.turn.positions[0] * a.turn.count[0], "table_dev"),
                        flat(a.turn.table[1], 8ll * a.turn.positions[1] * a.turn.count[1], "table_dev"),
                        flat(a.turn.table[2], 8ll * a.turn.positions[2] * a.turn.count[2], "table_dev")};
    if (const char* o = meets(out, in, &with)) return fail(DQ_ERR_INVALID_ARG, std::string(o) + " overlaps " + with);
    if ((st = known_device(device)) != DQ_OK) return st;
    DeviceGuard dg(device);
    if (!dg.ok) return fail(DQ_ERR_DEVICE, "hipSetDevice failed");
    a.part[0] = part_of(x, gain, y_dev, ldy, ydt == DQ_BF16 ? TO_BF16 : TO_F32, nullptr, ops->norm, a.turn.pairs > 0);
    a.N = N;
    a.eps = ops->eps;
    a.lph = head_dim / 8;
    a.g_bf16 = ops->gain_dt == DQ_BF16;
    const hipError_t e = dt == DQ_BF16 ? launch_heads<uint16_t>(a, 1, (hipStream_t)stream) : launch_heads<float>(a, 1, (hipStream_t)stream);
    return e == hipSuccess ? DQ_OK : hip_fail(e, "heads launch");
}

dq_status dq_kv_write(const dq_kv* kv, const dq_seqs* seqs, int64_t N, dq_dtype dt, const void* k_dev, int64_t ldk,
                      const void* v_dev, int64_t ldv, const void* gain_k_dev, const void* q_dev, int64_t ldq, int32_t q_heads,
                      const void* gain_q_dev, void* y_dev, int64_t ldy, dq_dtype ydt, const dq_head_ops* ops, int32_t device,
                      void* stream) {
    set_error("");
    dq_status st = check_kv(kv);
    if (st != DQ_OK || (st = check_seqs(seqs)) != DQ_OK) return st;
    const int D = kv->head_dim;
    if (N < 0 || N > MAX_ROWS) return fail(DQ_ERR_SHAPE, "N must be in [0, 2^31 - 256]");
    HeadsArgs a{};
    if ((st = check_ops(ops, D, &a.turn)) != DQ_OK) return st;
    if ((q_dev == nullptr) != (y_dev == nullptr)) return fail(DQ_ERR_INVALID_ARG, "q_dev and y_dev come together");
    if (q_dev && (q_heads < 1 || (int64_t)q_heads * D > MAX_C)) return fail(DQ_ERR_SHAPE, "q_heads * head_dim must be in [32, 32768]");
    if (N == 0) return DQ_OK;
    const int64_t C = (int64_t)kv->heads * D, Cq = (int64_t)q_heads * D;
    const RowsOf k{k_dev, ldk, C, dt, "k_dev"}, v{v_dev, ldv, C, dt, "v_dev"}, q{q_dev, ldq, Cq, dt, "q_dev"}, y{y_dev, ldy, Cq, ydt, "y_dev"};
    for (const RowsOf& r : {k, v})
        if ((st = check_row_array(r, N)) != DQ_OK) return st;
    for (const RowsOf& r : {q, y})
        if (q_dev && (st = check_row_array(r, N)) != DQ_OK) return st;
    const bool normed = ops->norm != DQ_NORM_NONE;
    const void *gk = normed ? gain_k_dev : nullptr, *gq = normed && q_dev ? gain_q_dev : nullptr;
    if (((uintptr_t)gk | (uintptr_t)gq) % 16 != 0) return fail(DQ_ERR_INVALID_ARG, "gains must be 16-byte aligned");
    const int64_t gsz = ops->gain_dt == DQ_BF16 ? 2 : 4;
    const int64_t cb = kv_code_bytes(kv), sb = kv_scale_bytes(kv);
    std::string with;
    const Named out[] = {flat(kv->k_codes, cb, "k_codes"), flat(kv->k_scales, sb, "k_scales"), flat(kv->v_codes, cb, "v_codes"),
                         flat(kv->v_scales, sb, "v_scales"), {y.span(N), "y_dev"}};
    const Named in[] = {{k.span(N), "k_dev"}, {v.span(N), "v_dev"}, {in_place(q, y) ? Span{} : q.span(N), "q_dev"},
                        flat(gk, (ops->norm == DQ_NORM_HEAD ? D : C) * gsz, "gain_k_dev"),
                        flat(gq, (ops->norm == DQ_NORM_HEAD ? D : Cq) * gsz, "gain_q_dev"),
                        flat(a.turn.pos, N * 4 * a.turn.axes, "pos_dev"),
                        flat(a.turn.table[0], 8ll * a.turn.positions[0] * a.turn.count[0], "table_dev"),
                        flat(a.turn.table[1], 8ll * a.turn.positions[1] * a.turn.count[1], "table_dev"),
                        flat(a.turn.table[2], 8ll * a.turn.positions[2] * a.turn.count[2], "table_dev"),
                        flat(seqs->first_dev, 4 * (seqs->seqs + 1), "first_dev"), flat(seqs->length_dev, 4 * seqs->seqs, "length_dev"),
                        flat(seqs->pages_dev, 4 * seqs->seqs * seqs->pages_ld, "pages_dev")};
    if (const char* o = meets(out, in, &with)) return fail(DQ_ERR_INVALID_ARG, std::string(o) + " overlaps " + with);
    if ((st = known_device(device)) != DQ_OK) return st;
    DeviceGuard dg(device);
    if (!dg.ok) return fail(DQ_ERR_DEVICE, "hipSetDevice failed");
    const int kind = kv->bits == 8 ? TO_FP8 : TO_FP4;
    int parts = 0;
    a.part[parts++] = part_of(k, gk, kv->k_codes, 0, kind, kv->k_scales, ops->norm, a.turn.pairs > 0);
    a.part[parts++] = part_of(v, nullptr, kv->v_codes, 0, kind, kv->v_scales, DQ_NORM_NONE, false);
    if (q_dev) a.part[parts++] = part_of(q, gq, y_dev, ldy, ydt == DQ_BF16 ? TO_BF16 : TO_F32, nullptr, ops->norm, a.turn.pairs > 0);
    a.pages = pages_of(kv, seqs);
    a.N = N;
    a.eps = ops->eps;
    a.lph = D / 8;
    a.g_bf16 = ops->gain_dt == DQ_BF16;
    const hipError_t e = dt == DQ_BF16 ? launch_heads<uint16_t>(a, parts, (hipStream_t)stream)
                                       : launch_heads<float>(a, parts, (hipStream_t)stream);
    return e == hipSuccess ? DQ_OK : hip_fail(e, "cache write launch");
}

dq_status dq_kv_read(const dq_kv* kv, const dq_seqs* seqs, int64_t N, void* k_dev, int64_t ldk, void* v_dev, int64_t ldv,
                     dq_dtype dt, int32_t device, void* stream) {
    set_error("");
    dq_status st = check_kv(kv);
    if (st != DQ_OK || (st = check_seqs(seqs)) != DQ_OK) return st;
    if (N < 0 || N > MAX_ROWS) return fail(DQ_ERR_SHAPE, "N must be in [0, 2^31 - 256]");
    if (dt != DQ_F32 && dt != DQ_BF16) return fail(DQ_ERR_INVALID_ARG, "unknown dtype");
    if (N == 0) return DQ_OK;
    if (!k_dev && !v_dev) return fail(DQ_ERR_INVALID_ARG, "no output: give k_dev or v_dev");
    const int64_t C = (int64_t)kv->heads * kv->head_dim;
    const RowsOf k{k_dev, ldk, C, dt, "k_dev"}, v{v_dev, ldv, C, dt, "v_dev"};
    for (const RowsOf& r : {k, v})
        if (r.p && (st = check_row_array(r, N)) != DQ_OK) return st;
    const int64_t cb = kv_code_bytes(kv), sb = kv_scale_bytes(kv);
    std::string with;
    const Named out[] = {{k.span(N), "k_dev"}, {v.span(N), "v_dev"}};
    const Named in[] = {flat(kv->k_codes, cb, "k_codes"), flat(kv->k_scales, sb, "k_scales"), flat(kv->v_codes, cb, "v_codes"),
                        flat(kv->v_scales, sb, "v_scales"), flat(seqs->first_dev, 4 * (seqs->seqs + 1), "first_dev"),
                        flat(seqs->length_dev, 4 * seqs->seqs, "length_dev"), flat(seqs->pages_dev, 4 * seqs->seqs * seqs->pages_ld, "pages_dev")};
    if (const char* o = meets(out, in, &with)) return fail(DQ_ERR_INVALID_ARG, std::string(o) + " overlaps " + with);
    if ((st = known_device(device)) != DQ_OK) return st;
    DeviceGuard dg(device);
    if (!dg.ok) return fail(DQ_ERR_DEVICE, "hipSetDevice failed");
    ReadArgs a{};
    a.codes[0] = kv->k_codes, a.codes[1] = kv->v_codes;
    a.scales[0] = kv->k_scales, a.scales[1] = kv->v_scales;
    a.y[0] = k_dev, a.y[1] = v_dev;
    a.ldy[0] = ldk, a.ldy[1] = ldv;
    a.pages = pages_of(kv, seqs);
    a.N = N;
    a.lph = kv->head_dim / 8;
    a.nch = (int)(C / 8);
    a.part0 = k_dev ? 0 : 1;
    const int parts = k_dev && v_dev ? 2 : 1;
    const auto go = [&](auto bits) {
        constexpr int B = decltype(bits)::value;
        if (parts == 2) return dt == DQ_BF16 ? launch_read<uint16_t, B, 2>(a, (hipStream_t)stream) : launch_read<float, B, 2>(a, (hipStream_t)stream);
        return dt == DQ_BF16 ? launch_read<uint16_t, B, 1>(a, (hipStream_t)stream) : launch_read<float, B, 1>(a, (hipStream_t)stream);
    };
    const hipError_t e = kv->bits == 8 ? go(std::integral_constant<int, 8>{}) : go(std::integral_constant<int, 4>{});
    return e == hipSuccess ? DQ_OK : hip_fail(e, "cache read launch");
}

}  // extern "C"
