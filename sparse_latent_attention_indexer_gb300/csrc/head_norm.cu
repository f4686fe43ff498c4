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
// are done per value.  Eight lanes take a head, 16-byte vectors round robin (a
// head of 192 bf16 values is three vectors a lane), so a norm costs three
// shuffles, and neighbouring heads of a row share the angles through L1.  A pair
// of the "pairs" order lies in one vector; in the "halves" order the other half's
// vector is read too (from L1) rather than passed between lanes, because which
// lane holds it depends on D and d_r.  Every load of a row comes before its first
// store, so y may be x.  Widths that are no multiple of 8 (d_r: of 16) and rows off
// 16 bytes go value by value, one warp a head.
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
    int D, d_r, at;     // at: first rotary dim
    int halves, n_pos;
    float eps;
};
static_assert(sizeof(HeadParams) + 256 <= 32764, "launch parameters");

constexpr int LANES = 8;    // lanes of a head (vector path)
constexpr int MAX_D = 512;

struct Item {
    const Half *t;
    int h, r, p;  // head, query row, position (-1: no rotation)
};
__device__ __forceinline__ Item item_of(const HeadParams &P, int64_t i) {
    const int all = P.t[0].n + P.t[1].n;
    Item m;
    m.r = (int)(i / all);
    m.h = (int)(i - (int64_t)m.r * all);
    m.t = &P.t[0];
    if (m.h >= P.t[0].n) {
        m.h -= P.t[0].n;
        m.t = &P.t[1];
    }
    if (P.d_r == 0) {
        m.p = -1;
    } else if (P.pos) {
        m.p = __ldg(P.pos + m.r);
        if ((unsigned)m.p >= (unsigned)P.n_pos) m.p = -1;
    } else {
        m.p = row_info(P.st, m.r).p;
    }
    return m;
}

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 a = *(const uint4 *)p;
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = ((const float4 *)p)[0], b = ((const float4 *)p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <int N>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[N]) {
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
__device__ __forceinline__ void store(float *p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) ((float4 *)p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// (x - mean) * inv * gain + bias of 8 values at dim d (mean 0, inv 1, gain 1, bias 0 where the norm has none).
__device__ __forceinline__ void norm8(float (&v)[8], const Half &t, int d, float mean, float inv) {
    if (t.norm == DSA_NORM_NONE) return;
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (v[i] - mean) * inv;
    if (t.gain) {
        load8(t.gain + d, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= g[i];
    }
    if (t.bias && t.norm == DSA_NORM_LAYER) {
        load8(t.bias + d, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += g[i];
    }
}

// VPT: vectors of 8 values a lane holds (D <= 64 * VPT).
template <typename TX, typename TY, int VPT>
__global__ void __launch_bounds__(256) head_norm_kernel(const __grid_constant__ HeadParams P) {
    const int sub = threadIdx.x & (LANES - 1);
    const int64_t i = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
    const bool live = i < P.rows;  // idle groups stay for the shuffles
    const Item m = item_of(P, live ? i : 0);
    const Half &t = *m.t;
    const TX *x = (const TX *)t.x + m.r * t.ld_x + m.h * t.hd_x;
    const int half = P.d_r / 2, rot_end = P.at + P.d_r;
    float v[VPT][8], o[VPT][8];  // o: the other half's values of a rotary vector ("halves" order)
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int d = (j * LANES + sub) * 8;
        if (d < P.D) {
            load8(x + d, v[j]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = 0.0f;
        }
        if (P.halves && m.p >= 0 && d >= P.at && d < rot_end) load8(x + (d < P.at + half ? d + half : d - half), o[j]);
    }
    float mean = 0.0f, inv = 1.0f;
    if (t.norm == DSA_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) s += v[j][e];
        mean = s;
    }
    mean = group_sum(mean) / (float)P.D;  // every lane of the warp shuffles, whatever its head's norm
    {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float c = (j * LANES + sub) * 8 < P.D ? v[j][e] - mean : 0.0f;
                s = fmaf(c, c, s);
            }
        s = group_sum(s);
        if (t.norm != DSA_NORM_NONE) inv = rsqrtf(s / (float)P.D + P.eps);
    }
    __syncwarp();  // every lane has read its values: y may be x
    if (!live) return;
    TY *y = (TY *)t.y + m.r * t.ld_y + m.h * t.hd_y;
    TY *pe = t.pe ? (TY *)t.pe + m.r * t.ld_pe + m.h * t.hd_pe : y + P.at;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int d = (j * LANES + sub) * 8;
        if (d >= P.D) continue;
        norm8(v[j], t, d, mean, inv);
        if (d < P.at || d >= rot_end) {
            // with an output of their own for the rotary dims, the others close up
            store<8>(y + (t.pe && d >= rot_end ? d - P.d_r : d), v[j]);
            continue;
        }
        const int k = d - P.at;  // dim within the rotary part
        if (m.p < 0 && P.halves) {
            store<8>(pe + k, v[j]);
        } else if (P.halves) {
            const bool second = k >= half;
            norm8(o[j], t, second ? d - half : d + half, mean, inv);
            float c[8], s[8];
            load8(P.cos + (int64_t)m.p * half + (second ? k - half : k), c);
            load8(P.sin + (int64_t)m.p * half + (second ? k - half : k), s);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = second ? o[j][e] * s[e] + v[j][e] * c[e] : v[j][e] * c[e] - o[j][e] * s[e];
            store<8>(pe + k, v[j]);
        } else {
            float4 c = make_float4(1.0f, 1.0f, 1.0f, 1.0f), s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (m.p >= 0) {
                c = __ldg((const float4 *)(P.cos + (int64_t)m.p * half + k / 2));
                s = __ldg((const float4 *)(P.sin + (int64_t)m.p * half + k / 2));
            }
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
            float a[4], b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = v[j][2 * e] * cc[e] - v[j][2 * e + 1] * ss[e];
                b[e] = v[j][2 * e] * ss[e] + v[j][2 * e + 1] * cc[e];
            }
            store<4>(pe + k / 2, a);
            store<4>(pe + half + k / 2, b);
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
    const Item m = item_of(P, i);
    const Half &t = *m.t;
    const TX *x = (const TX *)t.x + m.r * t.ld_x + m.h * t.hd_x;
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
    TY *y = (TY *)t.y + m.r * t.ld_y + m.h * t.hd_y;
    TY *pe = t.pe ? (TY *)t.pe + m.r * t.ld_pe + m.h * t.hd_pe : y + P.at;
    const int half = P.d_r / 2, rot_end = P.at + P.d_r;
    for (int d = lane; d < P.D; d += 32)
        if (d < P.at || d >= rot_end) y[t.pe && d >= rot_end ? d - P.d_r : d] = from_f32<TY>(v[d]);
    for (int k = lane; k < half; k += 32) {
        const int ia = P.at + (P.halves ? k : 2 * k), ib = P.at + (P.halves ? half + k : 2 * k + 1);
        const float a = v[ia], b = v[ib];
        float c = 1.0f, sn = 0.0f;
        if (m.p >= 0) {
            c = __ldg(P.cos + (int64_t)m.p * half + k);
            sn = __ldg(P.sin + (int64_t)m.p * half + k);
        }
        pe[k] = from_f32<TY>(a * c - b * sn);
        pe[half + k] = from_f32<TY>(a * sn + b * c);
    }
}

inline size_t esz(int dtype) { return dtype == DSA_F32 ? 4 : 2; }
inline bool on(const void *p, int64_t a, int64_t b, int dtype, size_t n) {
    return (uintptr_t)p % n == 0 && a * esz(dtype) % n == 0 && b * esz(dtype) % n == 0;
}

template <typename TX, typename TY>
cudaError_t launch_heads(const HeadParams &P, bool vec, cudaStream_t s) {
    const int64_t per = vec ? 256 / LANES : 8;
    const int64_t grid = (P.rows + per - 1) / per;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (!vec) head_norm_any_kernel<TX, TY><<<(unsigned)grid, 256, 0, s>>>(P);
    else if (P.D <= 64) head_norm_kernel<TX, TY, 1><<<(unsigned)grid, 256, 0, s>>>(P);
    else if (P.D <= 128) head_norm_kernel<TX, TY, 2><<<(unsigned)grid, 256, 0, s>>>(P);
    else if (P.D <= 192) head_norm_kernel<TX, TY, 3><<<(unsigned)grid, 256, 0, s>>>(P);
    else if (P.D <= 256) head_norm_kernel<TX, TY, 4><<<(unsigned)grid, 256, 0, s>>>(P);
    else head_norm_kernel<TX, TY, 8><<<(unsigned)grid, 256, 0, s>>>(P);
    return cudaGetLastError();
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
    bool vec = D % 8 == 0 && d_r % 16 == 0;
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
        vec = vec && on(h.x, h.ld_x, h.hd_x, x_dtype, 16) && on(h.y, h.ld_y, h.hd_y, y_dtype, 16) &&
              (!h.y_pe || on(h.y_pe, h.ld_pe, h.hd_pe, y_dtype, 16)) && (uintptr_t)h.gain % 16 == 0 &&
              (uintptr_t)h.bias % 16 == 0;
    }
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
    P.n_pos = n_pos;
    P.eps = eps;
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (x_dtype == DSA_F32)
        e = y_dtype == DSA_F32 ? launch_heads<float, float>(P, vec, s) : launch_heads<float, __nv_bfloat16>(P, vec, s);
    else
        e = y_dtype == DSA_F32 ? launch_heads<__nv_bfloat16, float>(P, vec, s)
                               : launch_heads<__nv_bfloat16, __nv_bfloat16>(P, vec, s);
    note_launch(DSA_KERNEL_HEAD_NORM);
    return e == cudaSuccess ? DSA_OK : fail_cuda(e);
}
