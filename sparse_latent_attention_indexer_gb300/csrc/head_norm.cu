// Norm of every query and key head and the rotation of its rotary dims to the
// row's position, in one pass over the heads.
//
//   y = norm(x) (none, RMS with gain, layer with gain and bias; "DeepSeek-V3.2-Exp
//   - Block input" page, RMSNorm excerpt, float32 compute; nnterp deepseek_v32
//   printout, LayerNorm with gain and bias), then pair i of the d_r rotary dims
//   (a, b) -> (a cos - b sin, a sin + b cos) ("Attention input" page, mla-kv excerpt,
//   apply_rotary_emb).
//
// Bound by HBM: a head is read once and written once and a handful of operations
// are done per value.  A CTA takes heads of one row (query token), so the row's angles
// and the gains and biases are fetched once, into shared memory.  Eight lanes take a head
// (sixteen above 256 dims), one to four vectors of eight values each, so a norm costs
// three shuffles; the next heads are on their way while these are turned and stored:
// 4096 rows of 129 heads of 192 in bf16 take 74 us, 5504 of 65 heads of 128 in fp32 66 us
// (0.81 of the measured copy rate; one warp a head took 165 and 92).
// A pair of the "pairs" order lies in one vector; in the "halves" order its other value is
// 1, 2 or 4 lanes (8: one vector) away (rotary parts of 16, 32, 64 or 128 at a multiple of
// that).  Every load of a head comes before its first store, so y may be x.  Other widths
// and rows off 16 bytes go value by value, one warp a head.
#include <algorithm>

#include "dsa_common.cuh"

namespace dsa {
namespace {

struct Half {  // the heads of q or of k
    const void *x;
    void *y, *pe;
    const float *gain, *bias;
    int64_t ld_x, hd_x, ld_y, hd_y, ld_pe, hd_pe;
    int n, norm;
};
struct HeadParams {
    SeqTab st;
    Half t[2];
    const float *cos, *sin;
    const int32_t *pos;
    int64_t rows;       // (query rows) * (heads of q + heads of k)
    int per_cta;        // warps' items that a CTA of the vector path takes
    int D, d_r, at;     // at: first rotary dim
    int halves, n_pos, wide;  // wide: every row starts on 32 bytes
    float eps, inv_D;
};
static_assert(sizeof(HeadParams) + 256 <= 32764, "launch parameters");

constexpr int MAX_D = 512;

// Position of row r (-1: no rotation).
__device__ __forceinline__ int position(const HeadParams &P, int r) {
    if (P.d_r == 0) return -1;
    if (!P.pos) return row_info(P.st, r).p;
    const int p = __ldg(P.pos + r);
    return (unsigned)p < (unsigned)P.n_pos ? p : -1;
}

// Eight values as they are stored.
template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> { uint4 a; };
template <> struct Vec8<float> { uint4 a, b; };
__device__ __forceinline__ void fetch(const __nv_bfloat16 *p, Vec8<__nv_bfloat16> &v, bool) { v.a = *(const uint4 *)p; }
__device__ __forceinline__ void fetch(const float *p, Vec8<float> &v, bool wide) {
    if (wide) {
        load32(p, v.a, v.b);
        return;
    }
    v.a = ((const uint4 *)p)[0];
    v.b = ((const uint4 *)p)[1];
}
__device__ __forceinline__ void unpack(const Vec8<__nv_bfloat16> &s, float (&v)[8]) {
    const uint32_t w[4] = {s.a.x, s.a.y, s.a.z, s.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const Vec8<float> &s, float (&v)[8]) {
    const uint32_t w[8] = {s.a.x, s.a.y, s.a.z, s.a.w, s.b.x, s.b.y, s.b.z, s.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}
template <int N>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[N], bool) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *(const uint32_t *)&t;
    }
    if constexpr (N == 8) *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
    else *(uint2 *)p = make_uint2(w[0], w[1]);
}
template <int N>
__device__ __forceinline__ void store(float *p, const float (&v)[N], bool wide) {
    uint4 w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        w[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                          __float_as_uint(v[4 * i + 3]));
    if (N == 8 && wide) {
        store32(p, w[0], w[N / 4 - 1]);
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) ((uint4 *)p)[i] = w[i];
    }
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Where value d of a row of MAX values lies in shared memory, and the eight from d on: the first four and the last four of
// each eight have a plane of their own, so that neighbouring lanes read neighbouring 16 bytes.
template <int MAX>
__device__ __forceinline__ int slot(int d) { return (d >> 2 & 1) * (MAX / 2) + (d >> 3) * 4 + (d & 3); }
template <int MAX>
__device__ __forceinline__ void lds8(const float *row, int d, float (&v)[8]) {
    const float4 a = *(const float4 *)(row + d / 2), b = *(const float4 *)(row + MAX / 2 + d / 2);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

constexpr int CTA = 128;

// LANES of a head, each with VPT vectors of 8 values (D <= 8 * LANES * VPT).
template <typename TX, typename TY, int LANES, int VPT, bool HALVES>
__global__ void __launch_bounds__(CTA, VPT * sizeof(Vec8<TX>) <= 32 ? 9 : VPT * sizeof(Vec8<TX>) <= 64 ? 7 : 4) head_norm_kernel(const __grid_constant__ HeadParams P) {
    __shared__ __align__(16) float turn[2][MAX_D / 2];  // cos, sin of the row's position
    __shared__ __align__(16) float aff[2][2 * MAX_D];   // q's and k's gains and biases
    constexpr int PACK = 32 / LANES, WARPS = CTA / 32;  // heads of a warp
    const int half = P.d_r / 2, lane = threadIdx.x & 31, sub = lane & (LANES - 1), mine = lane / LANES;
    const int rq = (P.t[0].n + PACK - 1) / PACK, all = rq + (P.t[1].n + PACK - 1) / PACK;  // warps' items
    const int end = min(all, (int)(blockIdx.y + 1) * P.per_cta);
    const int r = blockIdx.x;
    int it = blockIdx.y * P.per_cta + (threadIdx.x >> 5);
    Vec8<TX> raw[VPT];
    const auto load = [&](int item) {
        const Half &t = P.t[item >= rq];
        const int h = (item >= rq ? item - rq : item) * PACK + mine;
        const TX *x = (const TX *)t.x + r * t.ld_x + h * t.hd_x + sub * 8;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            raw[j] = Vec8<TX>{};
            if (h < t.n && (j * LANES + sub) * 8 < P.D) fetch(x + j * LANES * 8, raw[j], P.wide);
        }
    };
    if (it < end) load(it);
    const int p = position(P, r);
    if (p >= 0)
        for (int i = threadIdx.x; i < half; i += CTA) {
            const int at = HALVES ? slot<MAX_D / 2>(i) : i;
            turn[0][at] = __ldg(P.cos + (int64_t)p * half + i);
            turn[1][at] = __ldg(P.sin + (int64_t)p * half + i);
        }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const Half &t = P.t[i];
        for (int d = threadIdx.x; d < P.D; d += CTA) {
            if (t.gain) aff[i][slot<MAX_D>(d)] = __ldg(t.gain + d);
            if (t.bias) aff[i][MAX_D + slot<MAX_D>(d)] = __ldg(t.bias + d);
        }
    }
    __syncthreads();
    for (; it < end; it += WARPS) {  // every lane of a warp stays for the shuffles
        const int which = it >= rq;
        const Half &t = P.t[which];
        const int h = (which ? it - rq : it) * PACK + mine;
        const bool live = h < t.n;
        float v[VPT][8];
#pragma unroll
        for (int j = 0; j < VPT; ++j) unpack(raw[j], v[j]);  // zeros behind D
        if (t.norm != DSA_NORM_NONE) {
            float mu = 0.0f, s = 0.0f;
            if (t.norm == DSA_NORM_LAYER) {
#pragma unroll
                for (int j = 0; j < VPT; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) mu += v[j][e];
                mu = group_sum<LANES>(mu) * P.inv_D;
#pragma unroll
                for (int j = 0; j < VPT; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[j][e] -= (j * LANES + sub) * 8 < P.D ? mu : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(v[j][e], v[j][e], s);
            const float inv = rsqrtf(fmaf(group_sum<LANES>(s), P.inv_D, P.eps));
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int d = (j * LANES + sub) * 8;
                float g[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] *= inv;
                if (t.gain && d < P.D) {
                    lds8<MAX_D>(aff[which], d, g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[j][e] *= g[e];
                }
                if (t.bias && t.norm == DSA_NORM_LAYER && d < P.D) {
                    lds8<MAX_D>(aff[which] + MAX_D, d, g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[j][e] += g[e];
                }
            }
        }
        TY *y = (TY *)t.y + r * t.ld_y + h * t.hd_y;
        TY *pe = t.pe ? (TY *)t.pe + r * t.ld_pe + h * t.hd_pe : y + P.at;
        __syncwarp();  // every lane has its values, so y may be x: the next heads are others
        if (it + WARPS < end) load(it + WARPS);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int d = (j * LANES + sub) * 8, k = d - P.at;  // dim, and dim within the rotary part
            const bool rot = k >= 0 && k < P.d_r;
            if constexpr (HALVES) {
                // do the lanes' vectors j hold rotary dims?  (the same for the whole warp)
                if (p >= 0 && j * LANES * 8 < P.at + P.d_r && (j + 1) * LANES * 8 > P.at) {
                    const bool second = rot && k >= half;
                    float o[8], c[8], sn[8];
                    if (half < LANES * 8) {  // the pairs' other values lie half / 8 lanes away
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = __shfl_xor_sync(0xffffffffu, v[j][e], half / 8);
                    } else {  // or in the next or last vector (half == 8 * LANES): both are turned at the first
                        if (j + 1 < VPT && !second && rot) {
                            lds8<MAX_D / 2>(turn[0], k, c);
                            lds8<MAX_D / 2>(turn[1], k, sn);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float a = v[j][e], b = v[(j + 1) % VPT][e];
                                v[j][e] = a * c[e] - b * sn[e];
                                v[(j + 1) % VPT][e] = b * c[e] + a * sn[e];
                            }
                        }
                    }
                    if (half < LANES * 8 && rot) {
                        lds8<MAX_D / 2>(turn[0], second ? k - half : k, c);
                        lds8<MAX_D / 2>(turn[1], second ? k - half : k, sn);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] * c[e] + (second ? o[e] : -o[e]) * sn[e];
                    }
                }
            }
            if (!live || d >= P.D) continue;
            if (!rot) {
                // with an output of their own for the rotary dims, the others close up
                store<8>(y + (t.pe && k >= 0 ? d - P.d_r : d), v[j], P.wide);
            } else if (HALVES) {
                store<8>(pe + k, v[j], P.wide);
            } else {
                float4 c = make_float4(1.0f, 1.0f, 1.0f, 1.0f), sn = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (p >= 0) {
                    c = *(const float4 *)(turn[0] + k / 2);
                    sn = *(const float4 *)(turn[1] + k / 2);
                }
                const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
                float a[4], b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    a[e] = v[j][2 * e] * cc[e] - v[j][2 * e + 1] * ss[e];
                    b[e] = v[j][2 * e] * ss[e] + v[j][2 * e + 1] * cc[e];
                }
                store<4>(pe + k / 2, a, P.wide);
                store<4>(pe + half + k / 2, b, P.wide);
            }
        }
    }
}

// Any width: one warp a head, the normed row passes through shared memory.
template <typename TX, typename TY>
__global__ void __launch_bounds__(256) head_norm_any_kernel(const __grid_constant__ HeadParams P) {
    __shared__ float rows[8][MAX_D];
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= P.rows) return;
    float *v = rows[threadIdx.x >> 5];
    const int all = P.t[0].n + P.t[1].n, r = (int)(i / all), at = (int)(i - (int64_t)r * all);
    const Half &t = P.t[at >= P.t[0].n];
    const int h = at >= P.t[0].n ? at - P.t[0].n : at, p = position(P, r);
    const TX *x = (const TX *)t.x + r * t.ld_x + h * t.hd_x;
    float s = 0.0f;
    for (int d = lane; d < P.D; d += 32) {
        v[d] = to_f32(x[d]);
        s += v[d];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mean = t.norm == DSA_NORM_LAYER ? s / (float)P.D : 0.0f;
    float q = 0.0f;
    for (int d = lane; d < P.D; d += 32) q = fmaf(v[d] - mean, v[d] - mean, q);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
    const float inv = rsqrtf(q / (float)P.D + P.eps);
    if (t.norm != DSA_NORM_NONE)
        for (int d = lane; d < P.D; d += 32) {
            float z = (v[d] - mean) * inv;
            if (t.gain) z *= t.gain[d];
            if (t.bias && t.norm == DSA_NORM_LAYER) z += t.bias[d];
            v[d] = z;
        }
    __syncwarp();  // the row is read and normed: y may be x
    TY *y = (TY *)t.y + r * t.ld_y + h * t.hd_y;
    TY *pe = t.pe ? (TY *)t.pe + r * t.ld_pe + h * t.hd_pe : y + P.at;
    const int half = P.d_r / 2, rot_end = P.at + P.d_r;
    for (int d = lane; d < P.D; d += 32)
        if (d < P.at || d >= rot_end) y[t.pe && d >= rot_end ? d - P.d_r : d] = from_f32<TY>(v[d]);
    for (int k = lane; k < half; k += 32) {
        const int ia = P.at + (P.halves ? k : 2 * k), ib = P.at + (P.halves ? half + k : 2 * k + 1);
        const float a = v[ia], b = v[ib];
        float c = 1.0f, sn = 0.0f;
        if (p >= 0) {
            c = __ldg(P.cos + (int64_t)p * half + k);
            sn = __ldg(P.sin + (int64_t)p * half + k);
        }
        pe[k] = from_f32<TY>(a * c - b * sn);
        pe[half + k] = from_f32<TY>(a * sn + b * c);
    }
}

inline size_t esz(int dtype) { return dtype == DSA_F32 ? 4 : 2; }
inline bool on(const void *p, int64_t a, int64_t b, int dtype, size_t n) {
    return (uintptr_t)p % n == 0 && a * esz(dtype) % n == 0 && b * esz(dtype) % n == 0;
}

template <typename TX, typename TY, int LANES, int VPT>
cudaError_t launch_vec(HeadParams &P, cudaStream_t s) {
    // Few rows: a row's heads are spread over CTAs, so that about four of them come on every SM; many rows: one CTA takes
    // them all and fetches the angles and gains once.  An item is the heads that a warp takes at once.  Rows of 129 heads of 192,
    // spread over nine CTAs and taken by one: 16 rows 3.5 and 9.9 us, 128 6.0 and 10.0 (five, as here, 5.2), 608 15.8 and 12.7.
    constexpr int PACK = 32 / LANES, WARPS = CTA / 32;
    const int items = (P.t[0].n + PACK - 1) / PACK + (P.t[1].n + PACK - 1) / PACK, rounds = (items + WARPS - 1) / WARPS;
    const int n = (int)(P.rows / (P.t[0].n + P.t[1].n));
    const int parts = std::max(1, std::min({rounds, (4 * device_sm_count() + n - 1) / n, 65535}));
    P.per_cta = (rounds + parts - 1) / parts * WARPS;
    const dim3 grid(n, (items + P.per_cta - 1) / P.per_cta);
    if (P.halves) head_norm_kernel<TX, TY, LANES, VPT, true><<<grid, CTA, 0, s>>>(P);
    else head_norm_kernel<TX, TY, LANES, VPT, false><<<grid, CTA, 0, s>>>(P);
    return cudaGetLastError();
}

template <typename TX, typename TY>
cudaError_t launch_heads(HeadParams &P, bool vec, cudaStream_t s) {
    if (!vec) {
        const int64_t grid = (P.rows + 7) / 8;
        if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
        head_norm_any_kernel<TX, TY><<<(unsigned)grid, 256, 0, s>>>(P);
        return cudaGetLastError();
    }
    if (P.D <= 64) return launch_vec<TX, TY, 8, 1>(P, s);
    if (P.D <= 128) return launch_vec<TX, TY, 8, 2>(P, s);
    if (P.D <= 192) return launch_vec<TX, TY, 8, 3>(P, s);
    if (P.D <= 256) return launch_vec<TX, TY, 8, 4>(P, s);
    return launch_vec<TX, TY, 16, 4>(P, s);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_head_norm_rope(const dsa_heads *q, const dsa_heads *k, int x_dtype, int y_dtype, int D, int d_r,
                                  int rope_first, int rope, float eps, const float *rope_cos, const float *rope_sin,
                                  int n_pos, const int32_t *pos, const dsa_seqs *seqs, void *stream) {
    reset_trace();
    Batch bt;
    int rc = build_batch(seqs, bt);
    if (rc) return rc;
    if (D < 1 || d_r < 0 || d_r > D || d_r % 2 || n_pos < 0 || !(eps >= 0.0f)) return DSA_ERR_INVALID_ARG;
    if (D > MAX_D) return DSA_ERR_UNSUPPORTED;
    if ((x_dtype != DSA_F32 && x_dtype != DSA_BF16) || (y_dtype != DSA_F32 && y_dtype != DSA_BF16) ||
        (rope != DSA_ROPE_PAIRS && rope != DSA_ROPE_HALVES))
        return DSA_ERR_UNSUPPORTED;
    static thread_local HeadParams P;
    bool vec = D % 8 == 0 && d_r % 16 == 0, wide = true;
    const dsa_heads *in[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
        Half &t = P.t[i];
        t = Half{};
        if (!in[i] || in[i]->n_heads == 0) continue;
        const dsa_heads &h = *in[i];
        if (h.n_heads < 0) return DSA_ERR_INVALID_ARG;
        if (h.norm != DSA_NORM_NONE && h.norm != DSA_NORM_RMS && h.norm != DSA_NORM_LAYER) return DSA_ERR_UNSUPPORTED;
        const bool own_y = !h.y_pe || d_r < D;  // some dims go to y
        if (h.y_pe && d_r == 0) return DSA_ERR_INVALID_ARG;
        if (bt.total_q > 0 && (!h.x || (own_y && !h.y))) return DSA_ERR_INVALID_ARG;
        if ((uintptr_t)h.x % esz(x_dtype) || (uintptr_t)h.y % esz(y_dtype) || (uintptr_t)h.y_pe % esz(y_dtype) ||
            (uintptr_t)h.gain % 4 || (uintptr_t)h.bias % 4)
            return DSA_ERR_INVALID_ARG;
        if (h.y == h.x && h.x &&
            (x_dtype != y_dtype || h.y_pe || h.ld_x != h.ld_y || (h.n_heads > 1 && h.hd_x != h.hd_y)))
            return DSA_ERR_INVALID_ARG;
        t.x = h.x;
        t.y = h.y;
        t.pe = h.y_pe;
        t.gain = h.gain;
        t.bias = h.bias;
        t.ld_x = h.ld_x;
        t.hd_x = h.hd_x;
        t.ld_y = h.ld_y;
        t.hd_y = h.hd_y;
        t.ld_pe = h.ld_pe;
        t.hd_pe = h.hd_pe;
        t.n = h.n_heads;
        t.norm = h.norm;
        wide = wide && on(h.x, h.ld_x, h.hd_x, x_dtype, 32) && on(h.y, h.ld_y, h.hd_y, y_dtype, 32) &&
               (!h.y_pe || on(h.y_pe, h.ld_pe, h.hd_pe, y_dtype, 32));
        vec = vec && on(h.x, h.ld_x, h.hd_x, x_dtype, 16) && on(h.y, h.ld_y, h.hd_y, y_dtype, 16) &&
              (!h.y_pe || on(h.y_pe, h.ld_pe, h.hd_pe, y_dtype, 16)) && (uintptr_t)h.gain % 16 == 0 &&
              (uintptr_t)h.bias % 16 == 0;
    }
    // heads and rows are counted in 32 bits, up to a few warps past the last one
    if ((int64_t)P.t[0].n + P.t[1].n >= (int64_t(1) << 31) - 1024 || bt.total_q >= 0x7fffffff - 1024) return DSA_ERR_UNSUPPORTED;
    P.rows = (int64_t)bt.total_q * ((int64_t)P.t[0].n + P.t[1].n);
    if (P.rows == 0) return DSA_OK;
    if (d_r > 0) {
        if (!rope_cos || !rope_sin || (uintptr_t)rope_cos % 4 || (uintptr_t)rope_sin % 4 || (uintptr_t)pos % 4)
            return DSA_ERR_INVALID_ARG;
        if (!pos)
            for (int b = 0; b < bt.st.B; ++b) {
                const int Tb = bt.st.q_off[b + 1] - bt.st.q_off[b];
                if (Tb > 0 && bt.st.start_pos[b] + Tb > n_pos) return DSA_ERR_INVALID_ARG;
            }
        vec = vec && (uintptr_t)rope_cos % 16 == 0 && (uintptr_t)rope_sin % 16 == 0;
    }
    P.st = bt.st;
    P.cos = rope_cos;
    P.sin = rope_sin;
    P.pos = pos;
    P.D = D;
    P.d_r = d_r;
    P.at = rope_first ? 0 : D - d_r;
    P.halves = rope == DSA_ROPE_HALVES;
    if (P.halves && d_r > 0)  // the other value of a pair is 1, 2, 4 or 8 lanes or one vector away
        vec = vec && (d_r == 16 || d_r == 32 || d_r == 64 || d_r == 128) && P.at % d_r == 0;
    P.n_pos = n_pos;
    P.wide = wide;
    P.eps = eps;
    P.inv_D = 1.0f / (float)D;
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (x_dtype == DSA_F32)
        e = y_dtype == DSA_F32 ? launch_heads<float, float>(P, vec, s) : launch_heads<float, __nv_bfloat16>(P, vec, s);
    else
        e = y_dtype == DSA_F32 ? launch_heads<__nv_bfloat16, float>(P, vec, s)
                               : launch_heads<__nv_bfloat16, __nv_bfloat16>(P, vec, s);
    if (e != cudaSuccess) return fail_cuda(e);
    note_launch(DSA_KERNEL_HEAD_NORM);
    return DSA_OK;
}
