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

#include <cstring>
#include <memory>
#include <new>

#include "dq.h"
#include "dq_device.h"
#include "dq_internal.h"

// Workspace of the few-row products: the rows as bf16 matrix operands, and U.
struct dq_rows {
    int device = 0, cus = 256;
    int64_t max_rows = 0, Ci = 0, Co = 0, Kp = 0;
    int rp = 0;
    uint16_t* xp = nullptr;    // operand pieces of 16 rows: [row / 16][Kp / 128][part][4][64 lanes][8]
    float* u = nullptr;        // [round_up(max_rows, 64)][rp]
};

namespace dq {
namespace {

constexpr int WAVES = 8;                  // waves of a workgroup, one share of the K steps each
constexpr int X_BF16 = 0, X_F32 = 1, X_MX8 = 2;

struct RowsArgs {
    const void* x;                        // rows (bf16, fp32) or E4M3 codes
    const uint8_t* xs;                    // E8M0 codes of MX-FP8 rows
    long long ldx;
    int N, Ci, nks, Kp, Co, rp, tiles;
    const uint8_t *rq, *rs;
    const uint16_t *l1t, *l2t;
    uint16_t* xp;
    float* u;
    void* y;
    long long ldy;
};

// 8 consecutive channels of row n as bf16 operand pieces (zeros past N and Ci).
template <int XK>
__device__ __forceinline__ void operand8(const RowsArgs& a, int n, int ch, uint4* out) {
    constexpr int P = XK == X_F32 ? 3 : 1;
#pragma unroll
    for (int p = 0; p < P; ++p) out[p] = make_uint4(0u, 0u, 0u, 0u);
    if (n >= a.N || ch >= a.Ci) return;
    if constexpr (XK == X_BF16) {
        out[0] = *(const uint4*)((const uint16_t*)a.x + n * a.ldx + ch);
    } else {
        float v[8];
        if constexpr (XK == X_F32) {
            const float4* p = (const float4*)((const float*)a.x + n * a.ldx + ch);
            const float4 lo = p[0], hi = p[1];
            v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
            v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
        } else {
            const uint2 d = *(const uint2*)((const uint8_t*)a.x + (long long)n * a.Ci + ch);
            const int e = a.xs[(long long)n * (a.Ci >> 5) + (ch >> 5)];
            const float s = e == 255 ? __uint_as_float(0x7fc00000u) : pow2f(e - 127);
            typedef float v2f __attribute__((ext_vector_type(2)));
            const v2f f0 = __builtin_amdgcn_cvt_pk_f32_fp8(d.x, false), f1 = __builtin_amdgcn_cvt_pk_f32_fp8(d.x, true);
            const v2f f2 = __builtin_amdgcn_cvt_pk_f32_fp8(d.y, false), f3 = __builtin_amdgcn_cvt_pk_f32_fp8(d.y, true);
            v[0] = f0[0] * s; v[1] = f0[1] * s; v[2] = f1[0] * s; v[3] = f1[1] * s;
            v[4] = f2[0] * s; v[5] = f2[1] * s; v[6] = f3[0] * s; v[7] = f3[1] * s;
        }
        // the leading 8 bits, then those of what is left: differences are
        // exact, so the parts sum to the value (a NaN or infinity is its first
        // part alone)
        uint32_t w[P][4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float left = v[j];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                uint32_t b = __float_as_uint(left) >> 16;
                if (p == 0 && (__float_as_uint(left) & 0x7fffffffu) > 0x7f800000u) b = 0x7fc0u;
                left = p == 0 && (b & 0x7f80u) == 0x7f80u ? 0.0f : left - __uint_as_float(b << 16);
                w[p][j >> 1] = j & 1 ? w[p][j >> 1] | (b << 16) : b;
            }
        }
#pragma unroll
        for (int p = 0; p < P; ++p) out[p] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
    }
}

// First kernel: workgroups [0, nu) form U for one block of 16 rows and 16 low
// ranks each; the others lay the rows out as matrix operands.  Piece f of K
// step ks holds, for lane l, channels 128 ks + 32 (l / 16) + 8 f .. + 7 of row
// l % 16: the lane quarter l / 16 walks one 32-channel group, as the weight's
// 16-byte code chunks do.
template <int XK>
__global__ __launch_bounds__(512) void k_rows_operands(RowsArgs a, int nu) {
    constexpr int P = XK == X_F32 ? 3 : 1;
    const int tid = threadIdx.x, lane = tid & 63;
    if ((int)blockIdx.x >= nu) {
        const long long id = (long long)(blockIdx.x - nu) * 512 + tid;      // (tb, ks, f, lane)
        const long long step = id >> 8;
        const int f = (int)(id >> 6) & 3;
        const int tb = (int)(step / a.nks), ks = (int)(step % a.nks);
        if (16 * tb >= a.N) return;
        uint4 part[P];
        operand8<XK>(a, 16 * tb + (lane & 15), 128 * ks + 32 * (lane >> 4) + 8 * f, part);
#pragma unroll
        for (int p = 0; p < P; ++p) ((uint4*)a.xp)[((step * P + p) * 4 + f) * 64 + lane] = part[p];
        return;
    }
    __shared__ float red[WAVES][256];
    const int rb = a.rp >> 4, tb = blockIdx.x / rb, q0 = blockIdx.x % rb * 16, w = tid >> 6;
    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int ks = w; ks < a.nks; ks += WAVES) {
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            const int ch = 128 * ks + 32 * (lane >> 4) + 8 * f;
            const uint4 l1 = *(const uint4*)(a.l1t + (long long)(q0 + (lane & 15)) * a.Kp + ch);
            uint4 part[P];
            operand8<XK>(a, 16 * tb + (lane & 15), ch, part);
#pragma unroll
            for (int p = 0; p < P; ++p)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, l1), __builtin_bit_cast(v8bf, part[p]),
                                                              acc, 0, 0, 0);
        }
    }
    *(v4f*)&red[w][4 * lane] = acc;
    __syncthreads();
    if (tid < 256) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) s += red[i][tid];
        const int n = 16 * tb + ((tid >> 2) & 15), q = q0 + 4 * (tid >> 6) + (tid & 3);
        a.u[(long long)n * a.rp + q] = s;
    }
}

// Second kernel: a workgroup owns 16 RB output channels of 16 TB rows; its
// waves share out the K steps and their partial tiles are summed in wave
// order, so a result does not depend on how the work was scheduled.
template <int RB, int TB, int P, class YT>
__global__ __launch_bounds__(64 * WAVES) void k_rows(RowsArgs a) {
    __shared__ float red[WAVES][RB * TB * 256];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    // workgroups go to the 8 XCDs in turn; an XCD takes neighbouring tiles,
    // which share the 128-row blocks of the scale layout in its L2
    const int tile = (int)(blockIdx.x & 7) * (gridDim.x >> 3) + (int)(blockIdx.x >> 3);
    if (tile >= a.tiles) return;
    const int row0 = tile * 16 * RB, q = lane >> 4, r0 = (row0 & 255) + (lane & 15);
    const int n0 = blockIdx.y * 16 * TB;
    const size_t block = (size_t)(row0 >> 8) * a.nks;
    const uint8_t* rq = a.rq + block * 16384 + r0 * 64 + ((q ^ swz4(r0)) << 4);
    const uint8_t* rs = a.rs + block * 1024;
    int so[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) so[i] = (int)toff_scale(r0 + 16 * i, q);
    const uint4* xp = (const uint4*)a.xp + (size_t)(n0 >> 4) * a.nks * P * 256 + lane;
    const int per = (a.nks + WAVES - 1) / WAVES, k0 = w * per, k1 = min(a.nks, k0 + per);
    v4f acc[RB][TB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int t = 0; t < TB; ++t) acc[i][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int U = RB == 1 ? 4 : 2;
    for (int ks = k0; ks < k1; ks += U) {
        uint4 c[U][RB];
        int e[U][RB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = min(ks + u, k1 - 1);
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                c[u][i] = *(const uint4*)(rq + (size_t)k * 16384 + i * 1024);
                e[u][i] = rs[(size_t)k * 1024 + so[i]];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (ks + u >= k1) break;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                v8bf wv[RB];
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    const float s = pow2f(e[u][i] - 127);
                    const uint32_t d = f == 0 ? c[u][i].x : f == 1 ? c[u][i].y : f == 2 ? c[u][i].z : c[u][i].w;
                    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
                    const v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 0);
                    const v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 1);
                    const v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 2);
                    const v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 3);
                    wv[i] = v8bf{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
                }
#pragma unroll
                for (int t = 0; t < TB; ++t)
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        // (row blocks past N, read by the last group, lie in the workspace; their results are not stored)
                        const v8bf xv = __builtin_bit_cast(v8bf, xp[(((size_t)t * a.nks + ks + u) * P + p) * 256 + f * 64]);
#pragma unroll
                        for (int i = 0; i < RB; ++i)
                            acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[i], xv, acc[i][t], 0, 0, 0);
                    }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int t = 0; t < TB; ++t) *(v4f*)&red[w][((i * TB + t) * 64 + lane) * 4] = acc[i][t];
    __syncthreads();
    for (int o = tid; o < RB * TB * 256; o += 64 * WAVES) {
        const int l = (o >> 2) & 63, unit = o >> 8;
        const int n = n0 + unit % TB * 16 + (l & 15), j = row0 + unit / TB * 16 + 4 * (l >> 4) + (o & 3);
        if (n >= a.N || j >= a.Co) continue;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) s += red[i][o];
        if (a.rp) {
            const float* u = a.u + (long long)n * a.rp;
            const uint16_t* l2 = a.l2t + (long long)j * a.rp;
            float lr = 0.0f;
            for (int i = 0; i < a.rp; i += 8) {
                float b[8];
                const uint4 d = *(const uint4*)(l2 + i);
                const uint32_t wd[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    b[2 * k] = __uint_as_float(wd[k] << 16);
                    b[2 * k + 1] = __uint_as_float(wd[k] & 0xffff0000u);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) lr = __builtin_fmaf(u[i + k], b[k], lr);
            }
            s += lr;
        }
        if constexpr (sizeof(YT) == 2) ((__bf16*)a.y)[n * a.ldy + j] = (__bf16)s;
        else ((float*)a.y)[n * a.ldy + j] = s;
    }
}

template <int RB, int TB, int P>
void launch_tiles(RowsArgs a, int y_bf16, hipStream_t st) {
    a.tiles = (a.Co + 16 * RB - 1) / (16 * RB);
    const dim3 grid((unsigned)round_up(a.tiles, 8), (unsigned)((a.N + 16 * TB - 1) / (16 * TB)));
    if (y_bf16) k_rows<RB, TB, P, uint16_t><<<grid, 64 * WAVES, 0, st>>>(a);
    else k_rows<RB, TB, P, float><<<grid, 64 * WAVES, 0, st>>>(a);
}

template <int XK>
hipError_t launch_rows_product(const RowsArgs& a, int y_bf16, hipStream_t st) {
    constexpr int P = XK == X_F32 ? 3 : 1;
    const int tbs = (a.N + 15) / 16, nu = tbs * (a.rp / 16);
    const long long pieces = (long long)tbs * a.nks * 256;
    k_rows_operands<XK><<<(unsigned)(nu + (pieces + 511) / 512), 512, 0, st>>>(a, nu);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (tbs == 1) {
        if (a.Co >= 16 * 1024) launch_tiles<2, 1, P>(a, y_bf16, st);
        else launch_tiles<1, 1, P>(a, y_bf16, st);
    } else if (tbs == 2) {
        launch_tiles<2, 2, P>(a, y_bf16, st);
    } else {
        launch_tiles<2, 4, P>(a, y_bf16, st);
    }
    return hipGetLastError();
}

// Canonical codes [Co][Ci / 2] and scale codes [Co][Ci / 32] to the step-major layout.
__global__ __launch_bounds__(256) void k_import(const uint8_t* codes, const uint8_t* scales, long long Co, int groups,
                                                int nks, uint8_t* rq, uint8_t* rs) {
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    if (id >= Co * groups) return;
    const long long j = id / groups;
    const int G = (int)(id % groups);
    *(uint4*)(rq + off_fp4(j, G, nks)) = ((const uint4*)codes)[id];
    rs[off_scale(j, G, nks)] = scales[id];
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
    (void)hipFree(a->xp);
    (void)hipFree(a->u);
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

RowsArgs rows_args(const dq_weights* w, dq_rows* a, int64_t N, void* y, int64_t ldy) {
    RowsArgs r{};
    r.N = (int)N;
    r.Ci = (int)w->Ci;
    r.nks = (int)(w->Kp / 128);
    r.Kp = (int)w->Kp;
    r.Co = (int)w->Co;
    r.rp = w->rp;
    r.rq = w->rq;
    r.rs = w->rs;
    r.l1t = w->l1t;
    r.l2t = w->l2t;
    r.xp = a->xp;
    r.u = a->u;
    r.y = y;
    r.ldy = ldy;
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
    if (std::memchr(rscales_host, 255, (size_t)(Co * groups)))
        return fail(DQ_ERR_INVALID_ARG, "a scale code is 255 (not a number)");
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
    k_import<<<(unsigned)((Co * groups + 255) / 256), 256, 0, nullptr>>>(cd.p, sd.p, (long long)Co, (int)groups,
                                                                        (int)(w->Kp / 128), w->rq, w->rs);
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
    if (max_rows < 1 || max_rows > 4096) return fail(DQ_ERR_SHAPE, "max_rows must be in [1, 4096]");
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
    // (three parts for fp32 rows; whole groups of 64 rows, which the widest tile reads)
    const int64_t rows = round_up(max_rows, max_rows <= 16 ? 16 : max_rows <= 32 ? 32 : 64);
    hipError_t e;
    if ((e = zalloc(&a->xp, (size_t)(rows * w->Kp * 3), &bytes)) != hipSuccess ||
        (e = zalloc(&a->u, (size_t)(rows * w->rp), &bytes)) != hipSuccess)
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
    DeviceGuard dg(a->device);
    if (!dg.ok) return fail(DQ_ERR_DEVICE, "hipSetDevice failed");
    RowsArgs r = rows_args(w, a, N, y_dev, ldy);
    r.x = x_dev;
    r.ldx = ldx;
    const hipError_t e = dt == DQ_BF16 ? launch_rows_product<X_BF16>(r, ydt == DQ_BF16, (hipStream_t)stream)
                                       : launch_rows_product<X_F32>(r, ydt == DQ_BF16, (hipStream_t)stream);
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
    DeviceGuard dg(a->device);
    if (!dg.ok) return fail(DQ_ERR_DEVICE, "hipSetDevice failed");
    RowsArgs r = rows_args(w, a, N, y_dev, ldy);
    r.x = codes_dev;
    r.xs = scales_dev;
    const hipError_t e = launch_rows_product<X_MX8>(r, ydt == DQ_BF16, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "product launch");
    return DQ_OK;
}

}  // extern "C"
