// Attention of a tree of drafted tokens over the latent cache, in absorbed form:
// the entry point, and the generic CUDA-core kernel.
//
//   q~[r,h]   = q_nope[r,h] W_UK[h]
//   z[r,h,s]  = scale (q~[r,h] . c[s] + q_pe[r,h] . k_pe[s])   for the tokens s that row r sees
//   out[r,h]  = (sum_s softmax_s(z) c[s]) W_UV[h]
// (DeepSeek-V3.2-Exp atlas page, MoE transformer block: k^C = c^KV W_UK, v = c^KV
// W_UV, K_i = [K^C_i; k^R], with the causal mask M replaced by the tree's: every
// token before the tree, and the nodes whose bit the row's mask sets.)
//
// The generic kernel holds every shape and type: one CTA is one row and eight
// heads (a warp each), 32 tokens at a time in shared memory as fp32.  It runs
// far from any limit of the machine (each CTA reads the row's whole context);
// the shapes of the released model take the tensor-core kernel instead.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "dsa_common.cuh"

namespace dsa {
namespace {

constexpr int HG = 8;             // heads per CTA (one warp each)
constexpr int KC = 32;            // tokens per step
constexpr int MAX_PER_LANE = 32;  // d_c <= 1024

struct TreeSimt {
    SeqTab st;
    PageTab pt;
    int64_t ld_kv, ld_pe;
    const uint64_t *mask;
    int words;
    int H, d_r, d_c;
    float scale;
};
static_assert(sizeof(TreeSimt) + 256 <= 32764, "launch parameters");

__device__ __forceinline__ float latent(const float *kv, const float *, int64_t row, int64_t ld, int c, int) {
    return kv[row * ld + c];
}
__device__ __forceinline__ float latent(const __nv_bfloat16 *kv, const float *, int64_t row, int64_t ld, int c, int) {
    return to_f32(kv[row * ld + c]);
}
__device__ __forceinline__ float latent(const uint8_t *kv, const float *scale, int64_t row, int64_t ld, int c, int d_c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)kv[row * ld + c], __NV_E4M3);
    return __half2float(*(const __half *)&h) * scale[row * (d_c / 128) + c / 128];
}

template <typename T, typename TC>
__global__ void __launch_bounds__(HG * 32) tree_simt_kernel(const float *__restrict__ qt, const T *__restrict__ q_pe,
                                                            const TC *__restrict__ kv,
                                                            const float *__restrict__ kv_scale,
                                                            const T *__restrict__ kpe,
                                                            const __grid_constant__ TreeSimt P,
                                                            float *__restrict__ olat, float *__restrict__ lse) {
    extern __shared__ float smem[];
    __shared__ int rows[KC];
    const int r = blockIdx.x;
    const int h0 = blockIdx.y * HG;
    const RowInfo ri = row_info(P.st, r);
    const int first = ri.p - ri.t;                                  // tokens before the tree
    const int T_b = P.st.q_off[ri.b + 1] - P.st.q_off[ri.b];
    const int n = first + (P.mask ? T_b : ri.t + 1);                // tokens that the row may see
    const int W = P.d_c + P.d_r, WP = W + 1;
    float *qs = smem;          // [HG][W]
    float *cs = qs + HG * W;   // [KC][WP]
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int h = h0 + wid;
    for (int i = threadIdx.x; i < HG * W; i += blockDim.x) {
        const int hh = i / W, c = i - hh * W;
        float v = 0.0f;
        if (h0 + hh < P.H) {
            const int64_t rh = (int64_t)r * P.H + h0 + hh;
            v = c < P.d_c ? qt[rh * P.d_c + c] : to_f32(q_pe[rh * P.d_r + (c - P.d_c)]);
        }
        qs[i] = v;
    }
    float o[MAX_PER_LANE];
#pragma unroll
    for (int i = 0; i < MAX_PER_LANE; ++i) o[i] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    for (int s0 = 0; s0 < n; s0 += KC) {
        __syncthreads();
        if (threadIdx.x < KC) {
            const int s = s0 + threadIdx.x, j = s - first;
            bool see = s < n;
            if (see && P.mask && j >= 0) see = (__ldg(P.mask + (int64_t)r * P.words + (j >> 6)) >> (j & 63)) & 1;
            rows[threadIdx.x] = see ? (int)cache_row(P.pt, ri.b, ri.kbase, s) : -1;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < KC * W; i += blockDim.x) {
            const int jj = i / W, c = i - jj * W;
            const int64_t row = rows[jj];
            float v = 0.0f;
            if (row >= 0)
                v = c < P.d_c ? latent(kv, kv_scale, row, P.ld_kv, c, P.d_c) : to_f32(kpe[row * P.ld_pe + (c - P.d_c)]);
            cs[jj * WP + c] = v;
        }
        __syncthreads();
        if (h >= P.H) continue;
        float z = -INFINITY;
        if (rows[lane] >= 0) {
            float dot = 0.0f;
            const float *q = qs + wid * W, *c = cs + lane * WP;
            for (int d = 0; d < W; ++d) dot = fmaf(q[d], c[d], dot);
            z = dot * P.scale;
        }
        float zmax = z;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) zmax = fmaxf(zmax, __shfl_xor_sync(0xffffffffu, zmax, off));
        const float m_new = fmaxf(m, zmax);
        if (m_new == -INFINITY && !__any_sync(0xffffffffu, z != z)) continue;  // nothing seen yet
        const float corr = expf(m - m_new);
        const float p = (z == -INFINITY) ? 0.0f : expf(z - m_new);
        float psum = p;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) psum += __shfl_xor_sync(0xffffffffu, psum, off);
        l = l * corr + psum;
        m = m_new;
#pragma unroll
        for (int i = 0; i < MAX_PER_LANE; ++i) o[i] *= corr;
        for (int jj = 0; jj < KC; ++jj) {
            const float pj = __shfl_sync(0xffffffffu, p, jj);
            if (pj == 0.0f) continue;
            const float *c = cs + jj * WP;
#pragma unroll
            for (int i = 0; i < MAX_PER_LANE; ++i) {
                const int d = lane + 32 * i;
                if (d < P.d_c) o[i] = fmaf(pj, c[d], o[i]);
            }
        }
    }
    if (h >= P.H) return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a NaN that the row sees stays one
    const int64_t rh = (int64_t)r * P.H + h;
#pragma unroll
    for (int i = 0; i < MAX_PER_LANE; ++i) {
        const int d = lane + 32 * i;
        if (d < P.d_c) olat[rh * P.d_c + d] = o[i] * inv;
    }
    if (lse && lane == 0) lse[rh] = l == 0.0f ? -INFINITY : m + logf(l);
}

template <typename T, typename TC>
cudaError_t tree_simt_typed(const TreeSimt &P, const float *qt, const void *q_pe, const dsa_latent_cache *c, int N,
                            float *olat, float *lse, cudaStream_t s) {
    const int W = P.d_c + P.d_r;
    const size_t smem = ((size_t)HG * W + (size_t)KC * (W + 1)) * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(tree_simt_kernel<T, TC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    tree_simt_kernel<T, TC><<<dim3(N, (P.H + HG - 1) / HG), HG * 32, smem, s>>>(
        qt, (const T *)q_pe, (const TC *)c->kv, c->kv_scale, (const T *)c->k_pe, P, olat, lse);
    return cudaGetLastError();
}

cudaError_t launch_tree_simt(const float *qt, const void *q_pe, int dtype, const dsa_latent_cache *c,
                             const uint64_t *mask, int words, const Batch &bt, const PageTab &pt, int H, int d_r,
                             int d_c, float scale, float *olat, float *lse, cudaStream_t s) {
    static thread_local TreeSimt P;
    P.st = bt.st;
    P.pt = pt;
    P.ld_kv = c->ld_kv;
    P.ld_pe = c->ld_pe;
    P.mask = mask;
    P.words = words;
    P.H = H;
    P.d_r = d_r;
    P.d_c = d_c;
    P.scale = scale;
    const int N = bt.total_q;
    cudaError_t e;
    if (dtype == DSA_F32) e = tree_simt_typed<float, float>(P, qt, q_pe, c, N, olat, lse, s);
    else if (c->dtype == DSA_E4M3) e = tree_simt_typed<__nv_bfloat16, uint8_t>(P, qt, q_pe, c, N, olat, lse, s);
    else e = tree_simt_typed<__nv_bfloat16, __nv_bfloat16>(P, qt, q_pe, c, N, olat, lse, s);
    if (e == cudaSuccess) note_launch(DSA_KERNEL_TREE_SIMT);
    return e;
}

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }
inline bool on16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Scratch of a call: q~ and the latent context [N, H, d_c] (bf16 for the tensor-core kernel, fp32 for the
// generic one), and the partial contexts of split rows.
struct TreeWs {
    bool tc;
    size_t olat, part, total;
};
TreeWs tree_ws(int dtype, int H, int d_n, int d_r, int d_c, int d_v, const Batch &bt) {
    TreeWs w;
    w.tc = !force_generic() && tree_tc_supported(dtype, H, d_n, d_r, d_c, d_v);
    const size_t per = align256((size_t)bt.total_q * H * d_c * (w.tc ? 2 : 4));
    w.olat = per;
    w.part = 2 * per;
    w.total = w.part + (w.tc ? tree_tc_partial_bytes(H, bt) : 0);
    return w;
}

int check_tree_shape(int dtype, int H, int d_n, int d_r, int d_c, int d_v) {
    return check_mla_shape(dtype, H, d_n, d_r, d_c, d_v, 1);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

size_t dsa_tree_mla_workspace_size(int dtype, int H, int d_n, int d_r, int d_c, int d_v, const dsa_seqs *seqs) {
    Batch bt;
    if (check_tree_shape(dtype, H, d_n, d_r, d_c, d_v) || build_batch(seqs, bt)) return 0;
    return tree_ws(dtype, H, d_n, d_r, d_c, d_v, bt).total;
}

int dsa_tree_mla_fwd(const void *q_nope, const void *q_pe, int dtype, const dsa_latent_cache *cache, const void *W_UK,
                     const void *W_UV, int H, int d_n, int d_r, int d_c, int d_v, const uint64_t *tree_mask,
                     int mask_words, const dsa_seqs *seqs, const dsa_pages *pages, float softmax_scale, void *out,
                     float *lse, void *workspace, size_t ws_bytes, void *stream) {
    reset_trace();
    Batch bt;
    PageTab pt;
    int rc = check_tree_shape(dtype, H, d_n, d_r, d_c, d_v);
    if (rc || (rc = check_latent_cache(cache, d_c, d_r)) || (rc = build_batch(seqs, bt)) ||
        (rc = check_pages(pages, cache, bt, false, pt)))
        return rc;
    if (dtype == DSA_F32 ? cache->dtype != DSA_F32 : cache->dtype == DSA_F32) return DSA_ERR_UNSUPPORTED;
    if (!std::isfinite(softmax_scale * 1.4426950408889634f)) return DSA_ERR_INVALID_ARG;  // in powers of two, too
    if ((int64_t)bt.total_q * H >= (int64_t(1) << 31) - 256) return DSA_ERR_UNSUPPORTED;
    for (int b = 0; b < bt.st.B; ++b)  // tiles end past the last token
        if (bt.st.start_pos[b] > 0x7fffffff - 256 - (bt.st.q_off[b + 1] - bt.st.q_off[b])) return DSA_ERR_UNSUPPORTED;
    if (bt.total_q == 0) return DSA_OK;
    if (!q_nope || (d_r > 0 && !q_pe) || !W_UK || !W_UV || !out) return DSA_ERR_INVALID_ARG;
    if (!on16(q_nope) || !on16(q_pe) || !on16(W_UK) || !on16(W_UV) || !on16(out) || (uintptr_t)lse % 4 ||
        !on16(cache->kv_scale))
        return DSA_ERR_INVALID_ARG;
    if (tree_mask) {
        if (mask_words < 1 || (uintptr_t)tree_mask % 8) return DSA_ERR_INVALID_ARG;
        for (int b = 0; b < bt.st.B; ++b)
            if (bt.st.q_off[b + 1] - bt.st.q_off[b] > (int64_t)64 * mask_words) return DSA_ERR_INVALID_ARG;
    }
    const TreeWs L = tree_ws(dtype, H, d_n, d_r, d_c, d_v, bt);
    if (!workspace || (uintptr_t)workspace % 256 || ws_bytes < L.total) return DSA_ERR_WORKSPACE;
    const cudaStream_t s = (cudaStream_t)stream;
    char *ws = (char *)workspace;
    const int N = bt.total_q;
    cudaError_t e;
    if (L.tc) {
        void *qt = ws, *olat = ws + L.olat;
        e = launch_absorb_q_tc(q_nope, W_UK, qt, N, H, s);
        if (e != cudaSuccess) return fail_cuda(e);
        e = launch_tree_tc(qt, q_pe, cache, tree_mask, mask_words, bt, pt, H, softmax_scale, olat, lse, ws + L.part, s);
        if (e != cudaSuccess) return fail_cuda(e);
        e = launch_absorb_v_tc(olat, W_UV, out, N, H, s);
        return e == cudaSuccess ? DSA_OK : fail_cuda(e);
    }
    float *qt = (float *)ws, *olat = (float *)(ws + L.olat);
    e = launch_absorb_simt(q_nope, dtype, (int64_t)H * d_n, W_UK, dtype, qt, DSA_F32, (int64_t)H * d_c, N, H,
                                       d_n, d_c, s);
    if (e != cudaSuccess) return fail_cuda(e);
    e = launch_tree_simt(qt, q_pe, dtype, cache, tree_mask, mask_words, bt, pt, H, d_r, d_c, softmax_scale, olat, lse, s);
    if (e != cudaSuccess) return fail_cuda(e);
    e = launch_absorb_simt(olat, DSA_F32, (int64_t)H * d_c, W_UV, dtype, out, dtype, (int64_t)H * d_v, N, H, d_c, d_v, s);
    return e == cudaSuccess ? DSA_OK : fail_cuda(e);
}

}  // extern "C"
