// Writing the latent cache by token position (quantising on the way) and
// reading it back.
//
//   write: token t of sequence b -> row of position start_pos[b] + t:
//          bf16 / fp32 rows as they are, or per 128 values e4m3 codes
//          rne(x 2^-e) and the scale 2^e, e the smallest integer with
//          amax <= 448 * 2^e (config_671B_v3.2.json excerpt, "DeepSeek-V3.2-Exp
//          - Block input" page: dtype fp8, scale_fmt ue8m0);
//   read:  code * scale, by position.
//
// Both only move bytes (1152 or 2304 in and 656 out per token, or back), so each is one
// pass and HBM bounds them: 98,638 fp32 tokens into an FP8 cache take 50 us, 116,400
// tokens of one into bf16 36 us (0.87 and 0.86 of the measured copy rate).  A warp takes
// four tokens where there are enough of them to fill the GPU, else one: the lanes look the
// tokens' rows up side by side, and loads run ahead of the arithmetic (a read has all four
// tokens in flight, a write the next one; with one token a warp they take 75 and 57 us).
// A lane takes 16 consecutive values: eight lanes make a 128-block, whose maximum is three
// shuffles away, and the codes leave as one 16-byte store a lane.  Rows that do not start
// on 16 bytes, or whose width is no multiple of 16, go value by value.
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "dsa_common.cuh"

namespace dsa {
namespace {

struct MoveParams {
    SeqTab st;
    PageTab pt;
    int n;              // tokens
    int d_c, d_r;
    int64_t ld_c, ld_x;     // dense rows
    int64_t ld_kv, ld_pe;   // cache rows
    int wide;               // every row but e4m3 codes starts on 32 bytes
};
static_assert(sizeof(MoveParams) + 256 <= 32764, "launch parameters");

constexpr int PER = 16;  // values of a lane

// 16 values as they are stored.
template <typename T> struct Raw16;
template <> struct Raw16<__nv_bfloat16> { uint4 w[2]; };
template <> struct Raw16<float> { uint4 w[4]; };
template <> struct Raw16<uint8_t> { uint4 w[1]; };
template <typename T>
__device__ __forceinline__ void fetch(const T *p, Raw16<T> &v, bool wide) {
    if constexpr (sizeof(v) >= 32) {
        if (wide) {
#pragma unroll
            for (int i = 0; i < (int)(sizeof(v) / 32); ++i) load32((const uint4 *)p + 2 * i, v.w[2 * i], v.w[2 * i + 1]);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < (int)(sizeof(v) / 16); ++i) v.w[i] = __ldg((const uint4 *)p + i);
}
__device__ __forceinline__ void unpack(const Raw16<__nv_bfloat16> &s, float (&v)[PER]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {s.w[i].x, s.w[i].y, s.w[i].z, s.w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ void unpack(const Raw16<float> &s, float (&v)[PER]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[4 * i] = __uint_as_float(s.w[i].x);
        v[4 * i + 1] = __uint_as_float(s.w[i].y);
        v[4 * i + 2] = __uint_as_float(s.w[i].z);
        v[4 * i + 3] = __uint_as_float(s.w[i].w);
    }
}
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float (&v)[PER], bool wide) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *(const uint32_t *)&t;
    }
    const uint4 a = make_uint4(w[0], w[1], w[2], w[3]), b = make_uint4(w[4], w[5], w[6], w[7]);
    if (wide) {
        store32(p, a, b);
    } else {
        ((uint4 *)p)[0] = a;
        ((uint4 *)p)[1] = b;
    }
}
__device__ __forceinline__ void store16(float *p, const float (&v)[PER], bool wide) {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                          __float_as_uint(v[4 * i + 3]));
    if (wide) {
        store32(p, w[0], w[1]);
        store32(p + 8, w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) ((uint4 *)p)[i] = w[i];
    }
}

// 16 e4m3 codes -> values times the block's scale.
__device__ __forceinline__ void decode16(const uint4 &c, float sc, float (&v)[PER]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((w[i >> 1] >> (16 * (i & 1))) & 0xffffu),
                                                         __NV_E4M3);
        const float2 f = __half22float2(*(const __half2 *)&h);
        v[2 * i] = f.x * sc;
        v[2 * i + 1] = f.y * sc;
    }
}

// TC: uint8_t = e4m3 codes, else the value type of the cache; rotary keys of an e4m3 cache are bf16.
template <typename TC> struct PeOf { using T = TC; };
template <> struct PeOf<uint8_t> { using T = __nv_bfloat16; };

// The rows of d values of NT tokens from r0 on, between the dense side and the cache (own: lane n's is token n's cache row,
// -1: none).  VEC: rows start on 16 bytes and d is a multiple of 16; the rows' pieces of 16 values lie one after another
// over the lanes, and the first 32 (all of the rotary dims' at 64 values a row) are fetched by ahead().
template <typename TI, typename TO, bool VEC, int NT, bool READ>
struct Rows {
    const TI *src;
    TO *dst;
    int64_t ld_src, ld_dst, own;
    int r0, d;
    bool wide;
    Raw16<TI> w;

    // piece i, for all lanes together
    __device__ __forceinline__ bool piece(int i, const TI *&s, TO *&t) const {
        const int per = d / PER, n = i / per, at = (i - n * per) * PER;
        const int64_t row = __shfl_sync(0xffffffffu, own, min(n, 31));
        s = src + (READ ? row : (int64_t)(r0 + n)) * ld_src + at;
        t = dst + (READ ? (int64_t)(r0 + n) : row) * ld_dst + at;
        return n < NT && row >= 0;
    }
    __device__ __forceinline__ void ahead(int lane) {
        const TI *s;
        TO *t;
        if constexpr (VEC)
            if (piece(lane, s, t)) fetch(s, w, wide);
    }
    __device__ __forceinline__ void move(int lane) {
        if constexpr (VEC) {
            for (int i0 = 0; i0 < NT * (d / PER); i0 += 32) {
                const TI *s;
                TO *t;
                if (!piece(i0 + lane, s, t)) continue;
                if (i0) fetch(s, w, wide);
                float v[PER];
                unpack(w, v);
                store16(t, v, wide);
            }
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int64_t row = __shfl_sync(0xffffffffu, own, n);
                if (row < 0) continue;
                const TI *s = src + (READ ? row : (int64_t)(r0 + n)) * ld_src;
                TO *t = dst + (READ ? (int64_t)(r0 + n) : row) * ld_dst;
                for (int i = lane; i < d; i += 32) t[i] = from_f32<TO>(to_f32(s[i]));
            }
        }
    }
};

// 2^e, -127 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(e > -127 ? (uint32_t)(e + 127) << 23 : 0x00400000u); }

// The block's e4m3 codes of 16 values a lane (eight lanes a block), and its exponent.
__device__ __forceinline__ uint4 encode16(const float (&v)[PER], int &e) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // ue8m0_exponent() from the bits: amax = 1.f * 2^(E - 127) <= 448 * 2^e = 1.75 * 2^(8 + e)
    const uint32_t bits = __float_as_uint(amax);
    e = amax > 0.0f ? max(-127, (int)(bits >> 23) - 135 + ((bits & 0x7fffffu) > 0x600000u)) : 0;
    const float inv = pow2(-e);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * inv, v[4 * i + 1] * inv), __NV_SATFINITE,
                                                     __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv), __NV_SATFINITE,
                                                     __NV_E4M3);
        w[i] = lo | hi << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename TX, typename TC, bool VEC, bool VEC_PE, int NT>
__global__ void __launch_bounds__(256, 4) cache_write_kernel(const __grid_constant__ MoveParams P,
                                                             const TX *__restrict__ c_kv, const TX *__restrict__ k_pe,
                                                             TC *__restrict__ kv, float *__restrict__ kv_scale,
                                                             typename PeOf<TC>::T *__restrict__ pe) {
    const int lane = threadIdx.x & 31;
    const int r0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * NT;
    if (r0 >= P.n) return;
    int64_t own = -1;  // cache rows: lane n looks up token n's
    if (lane < NT && r0 + lane < P.n) {
        const RowInfo ri = row_info(P.st, r0 + lane);
        own = cache_row(P.pt, ri.b, ri.kbase, ri.p);
    }
    Rows<TX, typename PeOf<TC>::T, VEC_PE, NT, false> rot = {k_pe, pe, P.ld_x, P.ld_pe, own, r0, P.d_r, (bool)P.wide};
    if (P.d_r) rot.ahead(lane);
    if constexpr (sizeof(TC) == 1) {
        // four blocks a pass, eight lanes each; the next token's values are on their way while a token's are encoded
        const int nb = P.d_c / 128, left = min(NT, P.n - r0);
        for (int g0 = 0; g0 < nb; g0 += 4) {
            const int g = g0 + (lane >> 3), j = g * 128 + (lane & 7) * PER;
            const TX *x = c_kv + (int64_t)r0 * P.ld_c + j;
            Raw16<TX> w = {};
            if (VEC && g < nb) fetch(x, w, P.wide);
            for (int n = 0; n < left; ++n, x += P.ld_c) {
                float v[PER];
                if constexpr (VEC) {
                    unpack(w, v);
                    if (n + 1 < left && g < nb) fetch(x + P.ld_c, w, P.wide);
                } else {
#pragma unroll
                    for (int i = 0; i < PER; ++i) v[i] = g < nb ? to_f32(x[i]) : 0.0f;
                }
                int e;
                const uint4 c = encode16(v, e);
                const int64_t row = __shfl_sync(0xffffffffu, own, n);
                if (row >= 0 && g < nb) {
                    *(uint4 *)(kv + row * P.ld_kv + j) = c;
                    if ((lane & 7) == 0) kv_scale[row * nb + g] = pow2(e);
                }
            }
        }
    } else {
        Rows<TX, TC, VEC, NT, false> lat = {c_kv, kv, P.ld_c, P.ld_kv, own, r0, P.d_c, (bool)P.wide};
        lat.ahead(lane);
        lat.move(lane);
    }
    if (P.d_r) rot.move(lane);
}

template <typename TC, typename TO, bool VEC, bool VEC_PE, int NT>
__global__ void __launch_bounds__(256) cache_read_kernel(const __grid_constant__ MoveParams P,
                                                         const int32_t *__restrict__ pos, const TC *__restrict__ kv,
                                                         const float *__restrict__ kv_scale,
                                                         const typename PeOf<TC>::T *__restrict__ pe,
                                                         TO *__restrict__ c_kv, TO *__restrict__ k_pe) {
    const int lane = threadIdx.x & 31;
    const int r0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * NT;
    if (r0 >= P.n) return;
    int64_t row[NT], own = -1;  // cache rows: lane n looks up token n's
    if (lane < NT && r0 + lane < P.n) {
        const RowInfo ri = row_info(P.st, r0 + lane);
        const int p = pos ? __ldg(pos + r0 + lane) : ri.p;
        if ((unsigned)p < (unsigned)ri.S) own = cache_row(P.pt, ri.b, ri.kbase, p);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) row[n] = __shfl_sync(0xffffffffu, own, n);
    Rows<typename PeOf<TC>::T, TO, VEC_PE, NT, true> rot = {pe, k_pe, P.ld_pe, P.ld_x, own, r0, P.d_r, (bool)P.wide};
#pragma unroll
    for (int n = 0; n < NT; ++n)
        if (row[n] < 0 && r0 + n < P.n) {  // no such token
            for (int i = lane; i < P.d_c; i += 32) c_kv[(int64_t)(r0 + n) * P.ld_c + i] = from_f32<TO>(0.0f);
            for (int i = lane; i < P.d_r; i += 32) k_pe[(int64_t)(r0 + n) * P.ld_x + i] = from_f32<TO>(0.0f);
        }
    if (P.d_r) rot.ahead(lane);
    if constexpr (sizeof(TC) == 1) {
        const int nb = P.d_c / 128;
        for (int j = lane * PER; j < P.d_c; j += 32 * PER) {
            Raw16<TC> c[NT];
            float sc[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (row[n] >= 0) {
                    fetch(kv + row[n] * P.ld_kv + j, c[n], false);
                    sc[n] = __ldg(kv_scale + row[n] * nb + j / 128);
                }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (row[n] < 0) continue;
                float v[PER];
                decode16(c[n].w[0], sc[n], v);
                TO *t = c_kv + (int64_t)(r0 + n) * P.ld_c + j;
                if constexpr (VEC) {
                    store16(t, v, P.wide);
                } else {
#pragma unroll
                    for (int i = 0; i < PER; ++i) t[i] = from_f32<TO>(v[i]);
                }
            }
        }
    } else {
        Rows<TC, TO, VEC, NT, true> lat = {kv, c_kv, P.ld_kv, P.ld_c, own, r0, P.d_c, (bool)P.wide};
        lat.ahead(lane);
        lat.move(lane);
    }
    if (P.d_r) rot.move(lane);
}

inline bool on16(const void *p) { return ((uintptr_t)p & 15) == 0; }
inline size_t esz(int dtype) { return dtype == DSA_F32 ? 4 : (dtype == DSA_BF16 ? 2 : 1); }
// Whether rows of d values at p with stride ld take the 16-value path (the cache's rows always start on
// 16 bytes).
inline bool vec_rows(const void *p, int64_t ld, int dtype, int d) {
    return on16(p) && ld * esz(dtype) % 16 == 0 && d % PER == 0;
}

template <typename F>
auto by_bools(bool a, bool b, F f) {
    if (a) return b ? f(std::true_type(), std::true_type()) : f(std::true_type(), std::false_type());
    return b ? f(std::false_type(), std::true_type()) : f(std::false_type(), std::false_type());
}

// Four tokens a warp once that still leaves two warps for each of an SM's four schedulers (4864 tokens); else one.  A write of
// bf16 tokens into an FP8 cache, four and one a warp: 512 tokens 3.2 and 2.6 us, 4096 3.5 and 3.5, 16,384 5.7 and 8.3; a read
// 3.1 and 2.6, 3.2 and 3.5, 5.9 and 7.6.
inline bool many(const MoveParams &P, int nt) { return P.n >= (int64_t)nt * 8 * device_sm_count(); }

template <typename TX, typename TC>
cudaError_t launch_write(const MoveParams &P, const void *c_kv, const void *k_pe, const dsa_latent_cache *c, bool vec,
                         bool vec_pe, cudaStream_t s) {
    by_bools(vec, vec_pe, [&](auto v, auto vp) {
        const auto go = [&](auto kern, int nt) {
            kern<<<(P.n + 8 * nt - 1) / (8 * nt), 256, 0, s>>>(P, (const TX *)c_kv, (const TX *)k_pe, (TC *)c->kv, c->kv_scale,
                                                               (typename PeOf<TC>::T *)c->k_pe);
        };
        if (many(P, 4)) go(cache_write_kernel<TX, TC, decltype(v)::value, decltype(vp)::value, 4>, 4);
        else go(cache_write_kernel<TX, TC, decltype(v)::value, decltype(vp)::value, 1>, 1);
    });
    return cudaGetLastError();
}
template <typename TC, typename TO>
cudaError_t launch_read(const MoveParams &P, const int32_t *pos, const dsa_latent_cache *c, void *c_kv, void *k_pe,
                        bool vec, bool vec_pe, cudaStream_t s) {
    by_bools(vec, vec_pe, [&](auto v, auto vp) {
        const auto go = [&](auto kern, int nt) {
            kern<<<(P.n + 8 * nt - 1) / (8 * nt), 256, 0, s>>>(P, pos, (const TC *)c->kv, c->kv_scale,
                                                               (const typename PeOf<TC>::T *)c->k_pe, (TO *)c_kv, (TO *)k_pe);
        };
        if (many(P, 4)) go(cache_read_kernel<TC, TO, decltype(v)::value, decltype(vp)::value, 4>, 4);
        else go(cache_read_kernel<TC, TO, decltype(v)::value, decltype(vp)::value, 1>, 1);
    });
    return cudaGetLastError();
}

// What a write and a read check alike; fills P.
int check_move(int dense_dtype, int d_c, int d_r, const dsa_latent_cache *cache, const dsa_seqs *seqs,
               const dsa_pages *pages, bool whole, const void *c_kv, int64_t ld_c, const void *k_pe, int64_t ld_x,
               MoveParams &P) {
    if (dense_dtype != DSA_F32 && dense_dtype != DSA_BF16) return DSA_ERR_UNSUPPORTED;
    int rc = check_latent_cache(cache, d_c, d_r);
    if (rc) return rc;
    Batch bt;
    if ((rc = build_batch(seqs, bt))) return rc;
    if ((rc = check_pages(pages, cache, bt, whole, P.pt))) return rc;
    if (ld_c < d_c || (d_r > 0 && ld_x < d_r)) return DSA_ERR_INVALID_ARG;
    if (bt.total_q >= 0x7fffffff - 1024) return DSA_ERR_UNSUPPORTED;  // rows are counted in 32 bits, up to a few warps past the last one
    P.st = bt.st;
    P.n = bt.total_q;
    if (P.n == 0) return DSA_OK;
    if (!c_kv || (d_r > 0 && !k_pe)) return DSA_ERR_INVALID_ARG;
    const size_t a = esz(dense_dtype);
    if ((uintptr_t)c_kv % a || (uintptr_t)k_pe % a) return DSA_ERR_INVALID_ARG;
    P.d_c = d_c;
    P.d_r = d_r;
    P.ld_c = ld_c;
    P.ld_x = ld_x;
    P.ld_kv = cache->ld_kv;
    P.ld_pe = cache->ld_pe;
    const bool codes = cache->dtype == DSA_E4M3;
    const auto on32 = [](const void *p, int64_t ld, size_t size) { return (uintptr_t)p % 32 == 0 && ld * size % 32 == 0; };
    P.wide = on32(c_kv, ld_c, a) && (codes || on32(cache->kv, cache->ld_kv, esz(cache->dtype))) &&
             (d_r == 0 || (on32(k_pe, ld_x, a) && on32(cache->k_pe, cache->ld_pe, codes ? 2 : esz(cache->dtype))));
    return DSA_OK;
}

}  // namespace

int check_latent_cache(const dsa_latent_cache *c, int d_c, int d_r) {
    if (!c || d_c < 1 || d_r < 0) return DSA_ERR_INVALID_ARG;
    if (c->dtype != DSA_F32 && c->dtype != DSA_BF16 && c->dtype != DSA_E4M3) return DSA_ERR_UNSUPPORTED;
    if (d_c > 1024 || d_r > 128 || (c->dtype == DSA_E4M3 && d_c % 128)) return DSA_ERR_UNSUPPORTED;
    const int pe_dtype = c->dtype == DSA_E4M3 ? DSA_BF16 : c->dtype;
    if (!c->kv || c->ld_kv < d_c || c->ld_kv * esz(c->dtype) % 16 || !on16(c->kv)) return DSA_ERR_INVALID_ARG;
    if (d_r > 0 && (!c->k_pe || c->ld_pe < d_r || c->ld_pe * esz(pe_dtype) % 16 || !on16(c->k_pe)))
        return DSA_ERR_INVALID_ARG;
    if (c->dtype == DSA_E4M3 && (!c->kv_scale || (uintptr_t)c->kv_scale % 4)) return DSA_ERR_INVALID_ARG;
    if (c->rows < 0 || c->rows >= (int64_t(1) << 31) - 64) return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

int check_pages(const dsa_pages *pages, const dsa_latent_cache *c, const Batch &bt, bool whole, PageTab &pt) {
    pt = PageTab{nullptr, 0, 1, 0};
    if (!pages) return bt.total_k <= c->rows ? DSA_OK : DSA_ERR_INVALID_ARG;
    if (pages->page_size < 16 || pages->page_size % 16 || pages->n_pages < 0 || pages->width < 0 ||
        pages->ld_table < pages->width)
        return DSA_ERR_INVALID_ARG;
    if ((int64_t)pages->n_pages * pages->page_size > c->rows) return DSA_ERR_INVALID_ARG;
    int64_t most = 0;
    for (int b = 0; b < bt.st.B; ++b) {
        const int64_t T = bt.st.q_off[b + 1] - bt.st.q_off[b];
        if (T > 0) most = std::max<int64_t>(most, whole ? bt.st.k_len[b] : bt.st.start_pos[b] + T);
    }
    if (most > pages->width * pages->page_size) return DSA_ERR_INVALID_ARG;
    if (most > 0 && (!pages->block_table || (uintptr_t)pages->block_table % 4)) return DSA_ERR_INVALID_ARG;
    pt = PageTab{pages->block_table, pages->ld_table, pages->page_size, pages->n_pages};
    return DSA_OK;
}

}  // namespace dsa

using namespace dsa;

extern "C" {

int dsa_latent_cache_write(const void *c_kv, int64_t ld_c, const void *k_pe, int64_t ld_x, int x_dtype, int d_c, int d_r,
                           const dsa_latent_cache *cache, const dsa_seqs *seqs, const dsa_pages *pages, void *stream) {
    reset_trace();
    static thread_local MoveParams P;  // 16 KB: keep it off the host stack
    const int rc = check_move(x_dtype, d_c, d_r, cache, seqs, pages, false, c_kv, ld_c, k_pe, ld_x, P);
    if (rc || P.n == 0) return rc;
    const bool vec = vec_rows(c_kv, ld_c, x_dtype, d_c), vec_pe = vec_rows(k_pe, ld_x, x_dtype, d_r);
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    auto go = [&](auto x) {
        using TX = decltype(x);
        if (cache->dtype == DSA_E4M3) return launch_write<TX, uint8_t>(P, c_kv, k_pe, cache, vec, vec_pe, s);
        if (cache->dtype == DSA_BF16) return launch_write<TX, __nv_bfloat16>(P, c_kv, k_pe, cache, vec, vec_pe, s);
        return launch_write<TX, float>(P, c_kv, k_pe, cache, vec, vec_pe, s);
    };
    e = x_dtype == DSA_F32 ? go(float()) : go(__nv_bfloat16());
    if (e != cudaSuccess) return fail_cuda(e);
    note_launch(DSA_KERNEL_CACHE_WRITE);
    return DSA_OK;
}

int dsa_latent_cache_read(const dsa_latent_cache *cache, int d_c, int d_r, const dsa_seqs *seqs, const dsa_pages *pages,
                          const int32_t *pos, void *c_kv, int64_t ld_c, void *k_pe, int64_t ld_x, int out_dtype,
                          void *stream) {
    reset_trace();
    static thread_local MoveParams P;
    const int rc = check_move(out_dtype, d_c, d_r, cache, seqs, pages, pos != nullptr, c_kv, ld_c, k_pe, ld_x, P);
    if (rc || P.n == 0) return rc;
    if ((uintptr_t)pos % 4) return DSA_ERR_INVALID_ARG;
    const bool vec = vec_rows(c_kv, ld_c, out_dtype, d_c), vec_pe = vec_rows(k_pe, ld_x, out_dtype, d_r);
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    auto go = [&](auto o) {
        using TO = decltype(o);
        if (cache->dtype == DSA_E4M3) return launch_read<uint8_t, TO>(P, pos, cache, c_kv, k_pe, vec, vec_pe, s);
        if (cache->dtype == DSA_BF16) return launch_read<__nv_bfloat16, TO>(P, pos, cache, c_kv, k_pe, vec, vec_pe, s);
        return launch_read<float, TO>(P, pos, cache, c_kv, k_pe, vec, vec_pe, s);
    };
    e = out_dtype == DSA_F32 ? go(float()) : go(__nv_bfloat16());
    if (e != cudaSuccess) return fail_cuda(e);
    note_launch(DSA_KERNEL_CACHE_READ);
    return DSA_OK;
}

}  // extern "C"
