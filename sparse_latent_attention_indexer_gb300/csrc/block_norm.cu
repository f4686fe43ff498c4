// The norms on both sides of a block, fused with its gate and its residual:
//
//   h' = skip h + scale act(g) norm_post(u)        y = norm_pre(h')
//
// h is the residual stream, u what the block gave, g its gate; norm: none, RMS with gain,
// layer with gain and bias ("DeepSeek-V3.2-Exp - Block input" page, RMSNorm excerpt,
// float32 compute; nnterp deepseek_v32 printout).  y comes from h' before h' is rounded, so
// the stream's type costs the next block nothing.
//
// Bound by HBM (8192 rows of 7168 in bf16: 74 us, 0.94 of the measured copy rate; normed twice and gated 98, 0.88; in rows
// off 16 bytes by latency, 8192 of 7167 in bf16: 123, 0.56): every value is read once and written once.  A row lies in the registers of
// one CTA (of one warp up to 1024 values) between its loads, which are all issued first, and
// its stores; a thread stores where it has loaded, so h' may be h and y may be u.  A norm is one sum over the row (two for layer:
// the mean, then the squares of what is left, so that a large mean costs no digits).
#include <algorithm>

#include "dsa_common.cuh"

namespace dsa {
namespace {

struct NormParams {
    const void *h, *u, *gate;
    void *ho, *y;
    const float *post_gain, *post_bias, *pre_gain, *pre_bias;
    int64_t ld_h, ld_u, ld_g, ld_ho, ld_y, rows;
    int D, post, pre, gate_act;
    int base;             // FLAT: which of four values the first row starts with
    bool gate_row;        // FLAT: one gate for all rows, at an offset of its own
    float skip, scale, eps;
};

constexpr int MAX_D = 16384;

// W values (8, 4 or 1) as they are stored.
template <typename T, int W> struct Raw { T v[W]; };
template <typename T> struct Raw<T, 8> { uint4 q[sizeof(T) / 2]; };
template <> struct Raw<float, 4> { uint4 q; };
template <> struct Raw<__nv_bfloat16, 4> { uint2 q; };

template <typename T>
__device__ __forceinline__ void fetch(const T *p, Raw<T, 1> &r) { r.v[0] = *p; }
template <typename T>
__device__ __forceinline__ void fetch(const T *p, Raw<T, 8> &r) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)  // read once: the gains keep their place in L1
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.q[i].x), "=r"(r.q[i].y), "=r"(r.q[i].z), "=r"(r.q[i].w)
                     : "l"((const uint4 *)p + i));
}
__device__ __forceinline__ void fetch(const float *p, Raw<float, 4> &r) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.q.x), "=r"(r.q.y), "=r"(r.q.z), "=r"(r.q.w)
                 : "l"(p));
}
__device__ __forceinline__ void fetch(const __nv_bfloat16 *p, Raw<__nv_bfloat16, 4> &r) {
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.q.x), "=r"(r.q.y) : "l"(p));
}
__device__ __forceinline__ void unpack(const Raw<float, 4> &r, float (&v)[4]) {
    v[0] = __uint_as_float(r.q.x); v[1] = __uint_as_float(r.q.y);
    v[2] = __uint_as_float(r.q.z); v[3] = __uint_as_float(r.q.w);
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 4> &r, float (&v)[4]) {
    v[0] = __uint_as_float(r.q.x << 16); v[1] = __uint_as_float(r.q.x & 0xffff0000u);
    v[2] = __uint_as_float(r.q.y << 16); v[3] = __uint_as_float(r.q.y & 0xffff0000u);
}
template <typename T>
__device__ __forceinline__ void unpack(const Raw<T, 1> &r, float (&v)[1]) { v[0] = to_f32(r.v[0]); }
__device__ __forceinline__ void unpack(const Raw<float, 8> &r, float (&v)[8]) {
    const uint32_t w[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w, r.q[1].x, r.q[1].y, r.q[1].z, r.q[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 8> &r, float (&v)[8]) {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <typename T>
__device__ __forceinline__ void put(T *p, const float (&v)[1]) { *p = from_f32<T>(v[0]); }
__device__ __forceinline__ void put(float *p, const float (&v)[8]) {
    ((float4 *)p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    ((float4 *)p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void put(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *(const uint32_t *)&t;
    }
    *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put(float *p, const float (&v)[4]) { *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void put(__nv_bfloat16 *p, const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *(uint2 *)p = make_uint2(*(const uint32_t *)&a, *(const uint32_t *)&b);
}
// Values d .. d + 3 of a vector of D that may start anywhere: the two groups of four that they lie in, of which only one that
// holds a value of the vector is loaded, shifted (by the same in every thread of the row).
__device__ __forceinline__ void load_shifted(const float *p, int d, int D, float (&v)[4]) {
    const int s = (int)((uintptr_t)(p + d) / 4 & 3);
    float w[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = d - s + 4 * i;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (at > -4 && at < D && (i == 0 || s != 0)) a = __ldg((const float4 *)(p + at));
        w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
    }
#pragma unroll
    for (int e = 0; e < 6; ++e) w[e] = s & 2 ? w[e + 2] : w[e];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = s & 1 ? w[e + 1] : w[e];
}
__device__ __forceinline__ void load_shifted(const __nv_bfloat16 *p, int d, int D, float (&v)[4]) {
    const int s = (int)((uintptr_t)(p + d) / 2 & 3);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = d - s + 4 * i;
        uint2 a = make_uint2(0, 0);
        if (at > -4 && at < D && (i == 0 || s != 0)) a = __ldg((const uint2 *)(p + at));
        w[2 * i] = a.x; w[2 * i + 1] = a.y;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e) w[e] = s & 2 ? w[e + 1] : w[e];
    Raw<__nv_bfloat16, 4> r;
    r.q = make_uint2(__funnelshift_r(w[0], w[1], (s & 1) * 16), __funnelshift_r(w[1], w[2], (s & 1) * 16));
    unpack(r, v);
}
template <int W>
__device__ __forceinline__ void load_gain(const float *p, int d, int D, float (&v)[W]) {
    p += W == 4 ? 0 : d;
    if constexpr (W == 4) {
        load_shifted(p, d, D, v);
    } else if constexpr (W == 8) {
        const float4 a = __ldg((const float4 *)p), b = __ldg((const float4 *)p + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        v[0] = __ldg(p);
    }
}

// Where nothing is stored in more than bf16 (2^-8), the quick exponential's 2^-16 and better do; an fp32 h' or y has all digits of
// expf.  The quotient is good to 2 units in the last place.
template <bool FP32>
__device__ __forceinline__ float sigmoid(float v) {
    return __fdividef(1.0f, 1.0f + (FP32 ? expf(-v) : __expf(-v)));
}

// Sum over the row's threads, the same in each.  `part` takes a value a warp and is used by no other sum.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float *part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (WARP) return v;
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Whether value e of the vector from d on is the row's: vectors of four may hold some before or behind it.
template <int W>
__device__ __forceinline__ bool in_row(int d, int e, int D) {
    return W == 4 ? (unsigned)(d + e) < (unsigned)D : d < D;
}

// Norms the row's values in place; part: two sums' worth of warps.
template <int W, int N, bool WARP>
__device__ __forceinline__ void norm_row(float (&v)[N][W], int kind, const float *gain, const float *bias, int D, float inv_D,
                                         float eps, int first, int step, float *part) {
    if (kind == DSA_NORM_NONE) return;
    if (kind == DSA_NORM_LAYER) {
        float mu = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < W; ++e) mu += v[j][e];  // zeros behind D
        mu = row_sum<WARP>(mu, part) * inv_D;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < W; ++e) v[j][e] -= in_row<W>(first + j * step, e, D) ? mu : 0.0f;
    }
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < W; ++e) q = fmaf(v[j][e], v[j][e], q);
    const float inv = rsqrtf(fmaf(row_sum<WARP>(q, part + 32), inv_D, eps));
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int d = first + j * step;
        if (d >= D) continue;
        float g[W];
#pragma unroll
        for (int e = 0; e < W; ++e) v[j][e] *= inv;
        if (gain) {
            load_gain<W>(gain, d, D, g);
#pragma unroll
            for (int e = 0; e < W; ++e) v[j][e] *= g[e];
        }
        if (bias && kind == DSA_NORM_LAYER) {
            load_gain<W>(bias, d, D, g);
#pragma unroll
            for (int e = 0; e < W; ++e) v[j][e] += g[e];
        }
    }
}

template <int W, typename T>
__device__ __forceinline__ void put_row(T *p, const float (&v)[W], int d, int D) {
    if (W != 4 || (d >= 0 && d + W <= D)) {
        if (d < D) put(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (in_row<W>(d, e, D)) p[e] = from_f32<T>(v[e]);
    }
}

// Vectors of W values; N of them a thread, `step` values apart.  WARP: a warp takes a row.  AHEAD: a CTA takes one row after
// the other, and the next row's loads are issued once this row's values are unpacked, so they travel while it is summed and
// stored (8192 rows of 7168 in bf16: 82 -> 74 us, normed and gated 115 -> 98).
// W = 4 (FLAT): rows off 16 bytes that start on the same place of four in all tensors, as rows of odd width do.  A vector is
// four values on 16 bytes (8 of bf16), so that a row's first and last may hold values of its neighbours, which count as
// nothing and are left as they are.
template <typename TH, typename TX, int W, int N, int THREADS, bool WARP, bool AHEAD>
__global__ void __launch_bounds__(THREADS) block_norm_kernel(const __grid_constant__ NormParams P) {
    __shared__ float parts[2][4 * 32];  // of the row and the next: a warp may be a row ahead
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
    constexpr bool FLAT = W == 4;
    const int step = (WARP ? 32 : (int)blockDim.x) * W;
    const auto first_of = [&](int64_t row) { return t * W - (FLAT ? (int)(P.base + row * P.ld_h & 3) : 0); };
    const float inv_D = 1.0f / (float)P.D;
    const int64_t by = WARP ? (int64_t)gridDim.x * (THREADS / 32) : (int64_t)gridDim.x;
    int64_t r = WARP ? (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    Raw<TH, W> rh[N];
    Raw<TX, W> ru[N], rg[N];
    const auto load = [&](int64_t row) {
        const int first = first_of(row);
        const TH *h = (const TH *)P.h + row * P.ld_h + first;
        const TX *u = (const TX *)P.u + row * P.ld_u + first, *g = (const TX *)P.gate + row * P.ld_g + first;
        if (P.u) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                ru[j] = Raw<TX, W>{};
                if (first + j * step < P.D) fetch(u + j * step, ru[j]);
            }
            if (P.gate && !(FLAT && P.gate_row))
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    rg[j] = Raw<TX, W>{};
                    if (first + j * step < P.D) fetch(g + j * step, rg[j]);
                }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            rh[j] = Raw<TH, W>{};
            if (first + j * step < P.D) fetch(h + j * step, rh[j]);
        }
    };
    pdl_wait();
    if (AHEAD && r < P.rows) load(r);
    for (int odd = 0; r < P.rows; r += by, odd ^= 1) {
        float *part = parts[odd];
        float v[N][W];
        const int first = first_of(r);
        const auto only_row = [&](float (&a)[W], int d) {
            if (FLAT && (d < 0 || d + W > P.D))
#pragma unroll
                for (int e = 0; e < W; ++e) a[e] = in_row<W>(d, e, P.D) ? a[e] : 0.0f;
        };
        if (!AHEAD) load(r);
        if (P.u) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                unpack(ru[j], v[j]);
                only_row(v[j], first + j * step);
            }
            norm_row<W, N, WARP>(v, P.post, P.post_gain, P.post_bias, P.D, inv_D, P.eps, first, step, part);
            if (P.gate)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    float a[W];
                    if constexpr (FLAT) {
                        if (P.gate_row) load_shifted((const TX *)P.gate, first + j * step, P.D, a);
                        else unpack(rg[j], a);
                    } else {
                        unpack(rg[j], a);
                    }
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        if (P.gate_act != DSA_ACT_NONE) {
                            const float s = sigmoid<sizeof(TH) == 4 || sizeof(TX) == 4>(a[e]);
                            a[e] = P.gate_act == DSA_ACT_SILU ? a[e] * s : s;
                        }
                        v[j][e] *= a[e];
                    }
                }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float a[W];
                unpack(rh[j], a);
#pragma unroll
                for (int e = 0; e < W; ++e) v[j][e] = fmaf(P.scale, v[j][e], P.skip * a[e]);
                only_row(v[j], first + j * step);  // gains and gates beside the row may be anything
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                unpack(rh[j], v[j]);
                only_row(v[j], first + j * step);
#pragma unroll
                for (int e = 0; e < W; ++e) v[j][e] *= P.skip;
            }
        }
        if (AHEAD && r + by < P.rows) load(r + by);
        else pdl_trigger();
        if (P.ho) {
            TH *o = (TH *)P.ho + r * P.ld_ho + first;
#pragma unroll
            for (int j = 0; j < N; ++j)
                put_row<W>(o + j * step, v[j], first + j * step, P.D);
        }
        if (P.y) {
            norm_row<W, N, WARP>(v, P.pre, P.pre_gain, P.pre_bias, P.D, inv_D, P.eps, first, step, part + 64);
            TX *y = (TX *)P.y + r * P.ld_y + first;
#pragma unroll
            for (int j = 0; j < N; ++j)
                put_row<W>(y + j * step, v[j], first + j * step, P.D);
        }
        if (!AHEAD) break;
    }
}

template <typename TH, typename TX, int W, int N, int THREADS, bool WARP, bool AHEAD>
cudaError_t go(const NormParams &P, cudaStream_t s) {
    const int vecs = (P.D + (W == 4 ? 3 : 0) + W - 1) / W, t = WARP ? THREADS : ((vecs + N - 1) / N + 31) / 32 * 32;
    const int64_t grid = WARP ? (P.rows + THREADS / 32 - 1) / (THREADS / 32) : P.rows;
    // with loads ahead, as many CTAs as the SMs hold threads, each with rows to walk
    const int64_t most = AHEAD ? (int64_t)device_sm_count() * std::max(1, std::min(2048 / t, 32)) : 0x7fffffff;
    if (!AHEAD && grid > most) return cudaErrorInvalidConfiguration;
    return launch_pdl(block_norm_kernel<TH, TX, W, N, THREADS, WARP, AHEAD>, dim3((unsigned)std::min(grid, most)), dim3(t), 0, s, P);
}

template <typename TH, typename TX>
cudaError_t launch(const NormParams &P, bool vec, bool flat, cudaStream_t s) {
    // 8192 rows of 7167 in bf16, four values at a time or one: 123 us and 278 (with loads ahead 119, but 199 instead of 143 where
    // h is fp32); 3001 of 2049 16 and 23; 16384 of 201 10 and 11
    if (flat && P.D <= 253) return go<TH, TX, 4, 2, 128, true, false>(P, s);
    if (flat && P.D <= 509) return go<TH, TX, 4, 4, 128, true, false>(P, s);
    if (flat && P.D <= 4093) return go<TH, TX, 4, 2, 512, false, false>(P, s);
    if (flat && P.D <= 16381) return go<TH, TX, 4, 4, 1024, false, false>(P, s);
    if (!vec) {
        if (P.D <= 256) return go<TH, TX, 1, 8, 128, true, false>(P, s);
        if (P.D <= 4096) return go<TH, TX, 1, 8, 512, false, false>(P, s);
        return go<TH, TX, 1, 16, 1024, false, false>(P, s);
    }
    if (P.D <= 256) return go<TH, TX, 8, 1, 128, true, true>(P, s);
    if (P.D <= 512) return go<TH, TX, 8, 2, 128, true, true>(P, s);
    // few rows: as many threads a row as there are vectors (64 rows of 7168: 2.8 us, with two vectors a thread 3.9)
    if (P.D <= 8192 && P.rows <= device_sm_count()) return go<TH, TX, 8, 1, 1024, false, false>(P, s);
    // loads ahead of fp32 take registers that more threads would use, as long as two CTAs' worth of them fit: 8192 rows of 5120 in
    // fp32 alone 145 us with and 122 without, of 6144 gated 197 and 204; in an fp32 stream of bf16 blocks 4096 71 and 66, 7168
    // 114 and 128 (all bf16: 79 and 99)
    if (P.D <= (sizeof(TH) + sizeof(TX) > 4 ? 5120 : 0)) return go<TH, TX, 8, 2, 1024, false, false>(P, s);
    if (P.D <= 8192) return go<TH, TX, 8, 2, 512, false, true>(P, s);
    // 4096 rows of 16384: all bf16 95 us and with four vectors a thread 104; mixed 157 and 148; all fp32 with loads ahead 319
    // and without 235
    if (sizeof(TH) + sizeof(TX) == 8) return go<TH, TX, 8, 2, 1024, false, false>(P, s);
    if (sizeof(TH) + sizeof(TX) == 4) return go<TH, TX, 8, 2, 1024, false, true>(P, s);
    return go<TH, TX, 8, 4, 512, false, true>(P, s);
}

inline size_t esz(int dtype) { return dtype == DSA_F32 ? 4 : 2; }

int check_norm(const dsa_norm &n) {
    if (n.kind != DSA_NORM_NONE && n.kind != DSA_NORM_RMS && n.kind != DSA_NORM_LAYER) return DSA_ERR_UNSUPPORTED;
    return (uintptr_t)n.gain % 4 || (uintptr_t)n.bias % 4 ? DSA_ERR_INVALID_ARG : DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_block_norm(const dsa_block_norm_args *a, void *stream) {
    reset_trace();
    if (!a || a->rows < 0 || a->D < 1 || !(a->eps >= 0.0f)) return DSA_ERR_INVALID_ARG;
    if ((a->h_dtype != DSA_F32 && a->h_dtype != DSA_BF16) || (a->x_dtype != DSA_F32 && a->x_dtype != DSA_BF16) || a->D > MAX_D)
        return DSA_ERR_UNSUPPORTED;
    int rc = check_norm(a->post);
    if (!rc) rc = check_norm(a->pre);
    if (rc) return rc;
    if (a->gate_act != DSA_ACT_NONE && a->gate_act != DSA_ACT_SIGMOID && a->gate_act != DSA_ACT_SILU) return DSA_ERR_UNSUPPORTED;
    if (a->rows == 0) return DSA_OK;  // empty tensors have no addresses
    if (!a->u && (a->gate || a->post.kind != DSA_NORM_NONE)) return DSA_ERR_INVALID_ARG;
    if (!a->h_out && !a->y) return DSA_ERR_INVALID_ARG;
    if (!a->h) return DSA_ERR_INVALID_ARG;
    const size_t eh = esz(a->h_dtype), ex = esz(a->x_dtype);
    struct { const void *p; int64_t ld; size_t e; bool out; } t[5] = {
        {a->h, a->ld_h, eh, false}, {a->u, a->ld_u, ex, false}, {a->gate, a->ld_gate, ex, false}, {a->h_out, a->ld_ho, eh, true}, {a->y, a->ld_y, ex, true}};
    bool vec = a->D % 8 == 0, flat = true;
    const int base = (int)((uintptr_t)a->h / eh & 3);
    const bool gate_row = a->gate && (a->rows == 1 || a->ld_gate == 0);
    for (const auto &x : t) {
        if (!x.p) continue;
        if ((uintptr_t)x.p % x.e) return DSA_ERR_INVALID_ARG;
        if (x.out && a->rows > 1 && x.ld < a->D) return DSA_ERR_INVALID_ARG;  // rows of an output that overlap
        if (!(gate_row && &x == &t[2]))  // by its place: u may lie at the same address
            flat = flat && (int)((uintptr_t)x.p / x.e & 3) == base && (a->rows == 1 || ((x.ld - a->ld_h) & 3) == 0);
        vec = vec && (uintptr_t)x.p % 16 == 0 && (a->rows <= 1 || x.ld * (int64_t)x.e % 16 == 0);
    }
    if (a->h_out == a->h && a->h_out && a->rows > 1 && a->ld_ho != a->ld_h) return DSA_ERR_INVALID_ARG;
    if (a->y && a->y == a->u && a->rows > 1 && a->ld_y != a->ld_u) return DSA_ERR_INVALID_ARG;
    if (a->y && (a->y == a->h || a->y == a->gate || a->y == a->h_out)) return DSA_ERR_INVALID_ARG;
    if (a->h_out && (a->h_out == a->u || a->h_out == a->gate)) return DSA_ERR_INVALID_ARG;
    for (const float *g : {a->post.gain, a->post.bias, a->pre.gain, a->pre.bias}) vec = vec && (uintptr_t)g % 16 == 0;
    NormParams P;
    P.h = a->h;
    P.u = a->u;
    P.gate = a->gate;
    P.ho = a->h_out;
    P.y = a->y;
    P.post_gain = a->post.gain;
    P.post_bias = a->post.bias;
    P.pre_gain = a->pre.gain;
    P.pre_bias = a->pre.bias;
    P.ld_h = a->ld_h;
    P.ld_u = a->ld_u;
    P.ld_g = a->ld_gate;
    P.ld_ho = a->ld_ho;
    P.ld_y = a->ld_y;
    P.rows = a->rows;
    P.D = a->D;
    P.base = base;
    P.gate_row = gate_row;
    P.post = a->post.kind;
    P.pre = a->pre.kind;
    P.gate_act = a->gate_act;
    P.skip = a->skip;
    P.scale = a->scale;
    P.eps = a->eps;
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (a->h_dtype == DSA_F32)
        e = a->x_dtype == DSA_F32 ? launch<float, float>(P, vec, !vec && flat, s) : launch<float, __nv_bfloat16>(P, vec, !vec && flat, s);
    else
        e = a->x_dtype == DSA_F32 ? launch<__nv_bfloat16, float>(P, vec, !vec && flat, s) : launch<__nv_bfloat16, __nv_bfloat16>(P, vec, !vec && flat, s);
    if (e != cudaSuccess) return fail_cuda(e);
    note_launch(DSA_KERNEL_BLOCK_NORM);
    return DSA_OK;
}
