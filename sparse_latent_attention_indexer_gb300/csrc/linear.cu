// A linear layer with its epilogue, y = act(x W^T + bias) + residual, on tcgen05 tensor cores.
//
// A tile is 128 features (rows of W: the MMA's M) times up to 256 tokens (rows of x: its N), so
// a decode step of few tokens wastes none of the tensor cores' rows on padding and streams W
// with MMAs of N = 16: y^T = W x^T.  Per tile:
//   * warp 0 (one thread) streams 64-wide K slabs of W (128 rows) and of x by TMA, 128-byte
//     swizzled, through a ring that takes what shared memory there is (4 stages at 256 tokens,
//     12 at 16: 200 KB in flight per SM keep HBM busy);
//   * warp 1 (one thread) issues the MMAs into one of two fp32 accumulators in tensor memory;
//   * warps 4..11 read the accumulator back, a thread a feature: bias and activation need one
//     register, then the values turn through shared memory so that a warp stores 128 features
//     of a token at once, with the residual added on the way.
// Many tiles: a persistent grid, the epilogue of a tile beside the MMAs of the next.  Few tiles
// (SPLIT): a cluster of up to 8 CTAs shares a tile's K, each leaves its partial tile in its
// shared memory, and every CTA adds a share of it over the cluster in the order of the ranks, so
// the same call gives the same bits; no workspace, no second launch.
//
// The tensor cores cut off what does not fit a running sum of 24 bits, step by step: over 448 steps
// of 16 products (K = 7168) an fp32 result was off by 7.9e-6 of the whole, ten times what fp32
// arithmetic loses.  Where y is fp32 (EXACT) the epilogue takes the sum over after every 8 slabs
// (32 steps) and adds these parts to nearest in its registers.
//
// fp32 layers run on the same kernel: a value is the sum of three bf16 terms of 8 bits each, and
// of the nine products of terms the six above 2^-24 of the whole are added, smallest first.
// Rows that do not start on 16 bytes are laid out anew first (linear_layout_kernel).
#include "tc_common.cuh"

namespace dsa {

__device__ int g_linear_error = 0;

namespace {

constexpr int BF = 128, MAX_BT = 256;             // features, tokens of a tile
constexpr int W_SLAB = BF * 128;                  // 16 KB: 128 rows x 64 bf16
constexpr int MAX_STAGES = 12;
constexpr int NUM_THREADS = 384;                  // 0 TMA, 1 MMA, 2 TMEM owner, 3 idle, 4-11 epilogue
constexpr int EPI_WARP0 = 4, EPI_THREADS = 256;
constexpr int TURN = 2 * 32 * BF * 4;             // 32 tokens x 128 features in fp32 for each half of the epilogue
constexpr int SMEM_MAX = 232448;
constexpr int MAX_EXACT = 128;                     // tokens of a tile whose sums are exact
constexpr int CHAIN = 8;                          // slabs of an exact sum's parts
constexpr int GROUP_T = 8;                        // token tiles that share a panel of W in L2

struct Epilogue {
    const float *bias;
    const void *res;
    void *y;
    int64_t ld_r, ld_y;
    int act, f32, vec;    // f32: type of y and res; vec: four values at once are aligned
};
struct LinearParams {
    Epilogue e;
    int M, N;
    int bt, tt, tiles;    // tokens of a tile, token tiles, tiles
    int slabs, total;     // slabs of K; of all products of planes
    int plane;            // columns from one plane to the next; 0: one plane
    int stages, stage_bytes;
    int share;            // CTAs that share a tile's K (SPLIT)
    int chain;            // slabs that are added up in tensor memory (all, or CHAIN with EXACT)
    long long wait_limit;
};

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case DSA_ACT_RELU: return v < 0.0f ? 0.0f : v;  // a NaN stays
        case DSA_ACT_SILU: return v / (1.0f + expf(-v));
        case DSA_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678f));
        case DSA_ACT_GELU_TANH: return 0.5f * v * (1.0f + tanhf(0.79788456f * fmaf(0.044715f * v * v, v, v)));
        default: return v;
    }
}

// Four features from f on of a token, as they lie in res and y.
__device__ __forceinline__ void residual4(const Epilogue &E, int64_t row, int f, float (&r)[4]) {
    if (E.f32) {
        const float4 a = *(const float4 *)((const float *)E.res + row * E.ld_r + f);
        r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
    } else {
        const uint2 a = *(const uint2 *)((const __nv_bfloat16 *)E.res + row * E.ld_r + f);
        r[0] = __uint_as_float(a.x << 16); r[1] = __uint_as_float(a.x & 0xffff0000u);
        r[2] = __uint_as_float(a.y << 16); r[3] = __uint_as_float(a.y & 0xffff0000u);
    }
}
__device__ __forceinline__ void store4(const Epilogue &E, int64_t row, int f, const float (&v)[4]) {
    if (E.f32) {
        *(float4 *)((float *)E.y + row * E.ld_y + f) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *(uint2 *)((__nv_bfloat16 *)E.y + row * E.ld_y + f) = make_uint2(*(const uint32_t *)&a, *(const uint32_t *)&b);
    }
}
// One value: act and bias are done, the residual is not.
__device__ __forceinline__ void store1(const Epilogue &E, int64_t row, int f, float v) {
    if (E.f32) {
        if (E.res) v += ((const float *)E.res)[row * E.ld_r + f];
        ((float *)E.y)[row * E.ld_y + f] = v;
    } else {
        if (E.res) v += to_f32(((const __nv_bfloat16 *)E.res)[row * E.ld_r + f]);
        ((__nv_bfloat16 *)E.y)[row * E.ld_y + f] = from_f32<__nv_bfloat16>(v);
    }
}

__device__ __forceinline__ void bar(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool epi_and(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, 1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"((uint32_t)EPI_THREADS)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ float4 peer4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void tile_of(const LinearParams &P, int u, int &m0, int &f0) {
    const int ft = (P.N + BF - 1) / BF, per_group = GROUP_T * ft;
    const int grp = u / per_group, r = u - grp * per_group;
    const int gt = min(GROUP_T, P.tt - grp * GROUP_T);
    m0 = (grp * GROUP_T + r % gt) * P.bt;
    f0 = (r / gt) * BF;
}

// The planes of W and x whose product slab i belongs to, smallest products first, and its column.
__device__ __forceinline__ void slab_at(const LinearParams &P, int i, int &xw, int &xx) {
    if (P.plane == 0) {
        xw = xx = i * 64;
        return;
    }
    const int q = i / P.slabs, k = (i - q * P.slabs) * 64;
    xw = ((0x001102 >> (4 * q)) & 15) * P.plane + k;  // (2, 0) (0, 2) (1, 1) (1, 0) (0, 1) (0, 0), a digit each
    xx = ((0x010120 >> (4 * q)) & 15) * P.plane + k;
}

template <bool SPLIT, bool EXACT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                  const __grid_constant__ LinearParams P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);  // [stages][W slab | x slab]
    float *turn = (float *)(ring + P.stages * P.stage_bytes);                      // [2][32][BF] (not SPLIT)
    __shared__ __align__(8) uint64_t full[MAX_STAGES], empty[MAX_STAGES], tfull[2], tempty[2], mmadone;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word, never;
    volatile int *abort_flag = &abort_word, *nv = &never;
    int *err = &g_linear_error;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = SPLIT ? (int)tc::cluster_rank() : 0, share = SPLIT ? P.share : 1;
    const int who = (int)blockIdx.x / share, step = (int)gridDim.x / share;
    const int mine = P.tiles > who ? (P.tiles - who + step - 1) / step : 0;  // SPLIT: 1
    const int s0 = SPLIT ? (int)((int64_t)P.total * rank / share) : 0;
    const int s1 = SPLIT ? (int)((int64_t)P.total * (rank + 1) / share) : P.total;

    if (threadIdx.x == 0) {
        for (int i = 0; i < P.stages; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&tfull[i], 1);
            tc::mbar_init(&tempty[i], EPI_THREADS / 32);
        }
        tc::mbar_init(&mmadone, 1);
        abort_word = 0;
        never = 0;
        tc::fence_mbar_init();
    }
    if (warp == 2) {
        tc::tmem_alloc(&tmem_slot, 2 * MAX_BT);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();  // the set-up above overlapped the previous kernel; global memory only from here

    if (warp == 0 && lane == 0) {
        // ---------------- TMA producer ----------------
        tc::prefetch_tmap(&tm_w);
        tc::prefetch_tmap(&tm_x);
        int it = 0, st = 0, round = 0;
        bool ok = true;
        for (int i = 0; ok && i < mine; ++i) {
            int m0, f0;
            tile_of(P, who + i * step, m0, f0);
            for (int ks = s0; ks < s1; ++ks, ++it) {
                if (!(ok = tc::mbar_wait(&empty[st], (round & 1) ^ 1, abort_flag, err, 61, P.wait_limit))) break;
                uint8_t *sw = ring + st * P.stage_bytes;
                int xw, xx;
                slab_at(P, ks, xw, xx);
                tc::mbar_arrive_expect_tx(&full[st], P.stage_bytes);
                tc::tma_load_2d(sw, &tm_w, &full[st], xw, f0);
                tc::tma_load_2d(sw + W_SLAB, &tm_x, &full[st], xx, m0);
                if (++st == P.stages) st = 0, ++round;
            }
        }
        // Drain: nothing may still be landing in shared memory when the CTA goes on.
        for (int j = max(0, it - P.stages); j < it; ++j)
            tc::mbar_wait(&full[j % P.stages], (j / P.stages) & 1, nv, err, 62);
    } else if (warp == 1 && lane == 0) {
        // ---------------- MMA issuer ----------------
        const uint32_t idesc = tc::instr_desc(tc::kFmtBF16, tc::kFmtBF16, BF, P.bt, 0, 0);
        int st = 0, round = 0, issued = 0, n = 0;
        bool ok = true;
        for (int i = 0; ok && i < mine; ++i) {
            for (int k0 = s0; ok && k0 < s1; k0 += P.chain, ++n) {
                const int acc = n & 1, k1 = min(s1, k0 + P.chain);
                if (!(ok = tc::mbar_wait(&tempty[acc], ((n >> 1) & 1) ^ 1, abort_flag, err, 63, P.wait_limit))) break;
                const uint32_t d = tmem + acc * MAX_BT;
                for (int ks = k0; ks < k1; ++ks) {
                    if (!(ok = tc::mbar_wait(&full[st], round & 1, abort_flag, err, 64, P.wait_limit))) break;
                    tc::tc_fence_after();
                    const uint32_t a0 = tc::smem_u32(ring + st * P.stage_bytes), b0 = a0 + W_SLAB;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc::mma_f16(d, tc::smem_desc(a0 + kk * 32, 16, 1024), tc::smem_desc(b0 + kk * 32, 16, 1024), idesc,
                                    ks != k0 || kk != 0);
                    tc::mma_commit(&empty[st]);
                    ++issued;
                    if (++st == P.stages) st = 0, ++round;
                }
                if (ok) tc::mma_commit(&tfull[acc]);
            }
        }
        // No MMA may still be running when the tensor memory is released.
        if (issued > 0) {
            tc::mma_commit(&mmadone);
            tc::mbar_wait(&mmadone, 0, nv, err, 65);
        }
    } else if (warp >= EPI_WARP0) {
        // ---------------- epilogue ----------------
        // Warp (q, g): TMEM lanes (features) 32q .. 32q + 31, every other chunk of 32 tokens.
        const int q = warp & 3, g = (warp - EPI_WARP0) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        float *part = (float *)ring;           // SPLIT: [tokens][BF], once every load of the ring has landed and been used
        float *mine_turn = turn + g * 32 * BF;
        int n = 0;
        for (int i = 0; i < mine; ++i) {
            int m0, f0;
            tile_of(P, who + i * step, m0, f0);
            const int tokens = min(P.bt, P.M - m0);
            const int f = f0 + q * 32 + lane, f4 = f0 + lane * 4;
            const float b = !SPLIT && P.e.bias && f < P.N ? __ldg(P.e.bias + f) : 0.0f;
            const bool ahead = !SPLIT && !EXACT && P.e.res && P.e.vec && f4 < P.N;  // EXACT has no registers to spare
            const auto put = [&](int c, float (&v)[32]) {  // tokens c .. c + 31 of this thread's feature
                if (SPLIT) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j < tokens) part[(c + j) * BF + q * 32 + lane] = v[j];
                    return;
                }
                const int64_t row0 = m0 + c + q * 8;  // the eight tokens that this warp stores
                float r[8][4];
                if (ahead)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (row0 + j < P.M) residual4(P.e, row0 + j, f4, r[j]);
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = activate(v[j] + b, P.e.act);
                bar(2 + g, EPI_THREADS / 2);  // the last chunk has been read
#pragma unroll
                for (int j = 0; j < 32; ++j) mine_turn[j * BF + q * 32 + lane] = v[j];
                bar(2 + g, EPI_THREADS / 2);
                const int left = min(8, tokens - c - q * 8);
                if (P.e.vec) {
                    if (f4 < P.N)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < left) {
                                const float4 a = *(const float4 *)(mine_turn + (q * 8 + j) * BF + lane * 4);
                                float o[4] = {a.x, a.y, a.z, a.w};
                                if (EXACT && P.e.res) residual4(P.e, row0 + j, f4, r[j]);
                                if (P.e.res)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) o[e] += r[j][e];
                                store4(P.e, row0 + j, f4, o);
                            }
                } else {
                    for (int j = 0; j < left; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (f0 + e * 32 + lane < P.N)
                                store1(P.e, row0 + j, f0 + e * 32 + lane, mine_turn[(q * 8 + j) * BF + e * 32 + lane]);
                }
            };
            bool ok = true;
            if (EXACT) {
                float sum[MAX_EXACT / 64][32];
#pragma unroll
                for (int j = 0; j < MAX_EXACT / 64; ++j)
#pragma unroll
                    for (int e = 0; e < 32; ++e) sum[j][e] = 0.0f;
                for (int k0 = s0; k0 < s1; k0 += P.chain, ++n) {
                    ok = epi_and(tc::mbar_wait(&tfull[n & 1], (n >> 1) & 1, abort_flag, err, 66, P.wait_limit));
                    if (!ok) break;
                    tc::tc_fence_after();
#pragma unroll
                    for (int j = 0; j < MAX_EXACT / 64; ++j)
                        if (j * 64 + g * 32 < tokens) {
                            float v[32];
                            tc::tmem_ld32(lanes + (n & 1) * MAX_BT + j * 64 + g * 32, v);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) sum[j][e] += v[e];
                        }
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&tempty[n & 1]);
                }
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < MAX_EXACT / 64; ++j)
                    if (j * 64 + g * 32 < tokens) put(j * 64 + g * 32, sum[j]);
            } else {
                ok = epi_and(tc::mbar_wait(&tfull[n & 1], (n >> 1) & 1, abort_flag, err, 66, P.wait_limit));
                if (!ok) break;
                tc::tc_fence_after();
                for (int c = g * 32; c < tokens; c += 64) {
                    float v[32];
                    tc::tmem_ld32(lanes + (n & 1) * MAX_BT + c, v);
                    tc::tmem_ld_wait();
                    put(c, v);
                }
                // every column of this accumulator has been read
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&tempty[n & 1]);
                ++n;
            }
        }
    }
    __syncthreads();
    if (SPLIT) {
        tc::cluster_sync();  // every CTA's partial tile is in its shared memory
        int m0, f0;
        tile_of(P, who, m0, f0);
        const int units = min(P.bt, P.M - m0) * (BF / 4);
        const uint32_t part = tc::smem_u32(ring);
        for (int u = rank * NUM_THREADS + (int)threadIdx.x; u < units; u += share * NUM_THREADS) {
            const int t = u / (BF / 4), f = f0 + (u % (BF / 4)) * 4;
            if (f >= P.N) continue;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, r[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            const int64_t row = m0 + t;
            if (P.e.res && P.e.vec) residual4(P.e, row, f, r);
            for (int k = 0; k < share; ++k) {
                const float4 a = peer4(tc::map_peer(part + u * 16, k));
                v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (f + e < P.N) v[e] = activate(v[e] + (P.e.bias ? __ldg(P.e.bias + f + e) : 0.0f), P.e.act);
            if (P.e.vec) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += r[e];
                store4(P.e, row, f, v);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (f + e < P.N) store1(P.e, row, f + e, v[e]);
            }
        }
        __syncwarp();
        tc::cluster_sync();  // nobody leaves while its partial tile is read
    }
    if (warp == 2) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 2 * MAX_BT);
    }
}

// ---------------------------------------------------------------------------
// Rows laid out for the TMA: bf16 rows copied to rows on 16 bytes; fp32 rows as three planes of
// bf16 terms, each the nearest to what the terms before it leave (a term that would round to
// infinity is the largest number instead; infinities and NaN stay in the first plane).
// ---------------------------------------------------------------------------
template <bool F32>
__global__ void __launch_bounds__(256) linear_layout_kernel(const void *src, int64_t ld, __nv_bfloat16 *dst, int64_t rows, int K,
                                                             int cols, int64_t ld_dst) {
    pdl_wait();
    const int per = cols / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= rows * per) return;
    const int64_t r = i / per;
    const int k = (int)(i - r * per) * 8;
    __nv_bfloat16 *d = dst + r * ld_dst + k;
    if (F32) {
        __nv_bfloat16 t[3][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = k + e < K ? ((const float *)src)[r * ld + k + e] : 0.0f;
            const bool finite = fabsf(v) < INFINITY;
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                float h = __bfloat162float(__float2bfloat16_rn(v));
                if (finite && !(fabsf(h) < INFINITY)) h = copysignf(3.38953139e38f, v);
                t[p][e] = __float2bfloat16_rn(h);
                v = finite ? v - h : 0.0f;
            }
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) *(uint4 *)(d + (int64_t)p * cols) = *(const uint4 *)t[p];
    } else {
        __align__(16) uint16_t t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = k + e < K ? ((const uint16_t *)src)[r * ld + k + e] : (uint16_t)0;
        *(uint4 *)d = *(const uint4 *)t;
    }
}

// ---------------------------------------------------------------------------
// Few tokens whose rows the TMA does not take (off 16 bytes, fp32): a second pass over W to lay it
// out would cost twice what the product does, so a warp takes four features and every token,
// and reads W once, value by value.  SPLIT: the CTA's eight warps share K.
// ---------------------------------------------------------------------------
constexpr int FEW = 16;

template <typename T, int MT, bool SPLIT>
__global__ void __launch_bounds__(256) linear_few_kernel(const T *x, int64_t ld_x, const T *W, int64_t ld_w, int M, int N, int K,
                                                         const __grid_constant__ Epilogue E) {
    __shared__ float sums[8][4 * MT];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int f0 = SPLIT ? (int)blockIdx.x * 4 : ((int)blockIdx.x * 8 + warp) * 4;
    const int per = SPLIT ? ((K + 7) / 8 + 31) / 32 * 32 : K;
    const int k0 = SPLIT ? warp * per : 0, k1 = min(K, k0 + per);
    float acc[4][MT];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[a][m] = 0.0f;
    const T *w[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) w[a] = W + (int64_t)min(f0 + a, N - 1) * ld_w;
#pragma unroll 4
    for (int k = k0 + lane; k < k1; k += 32) {
        float wv[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) wv[a] = to_f32(w[a][k]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float xv = m < M ? to_f32(x[m * ld_x + k]) : 0.0f;
#pragma unroll
            for (int a = 0; a < 4; ++a) acc[a][m] = fmaf(wv[a], xv, acc[a][m]);
        }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float v = acc[a][m];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) sums[warp][m * 4 + a] = v;
        }
    __syncthreads();
    const int count = SPLIT ? 4 * MT : 8 * 4 * MT;
    for (int i = threadIdx.x; i < count; i += 256) {
        const int wi = i / (4 * MT), at = i % (4 * MT), m = at / 4;
        const int f = SPLIT ? f0 + at % 4 : ((int)blockIdx.x * 8 + wi) * 4 + at % 4;
        if (m >= M || f >= N) continue;
        float v = sums[wi][at];
        if (SPLIT)
#pragma unroll
            for (int j = 1; j < 8; ++j) v += sums[j][at];
        store1(E, m, f, activate(v + (E.bias ? E.bias[f] : 0.0f), E.act));
    }
}

template <typename T, int MT>
cudaError_t launch_few(const T *x, int64_t ld_x, const T *W, int64_t ld_w, int M, int N, int K, const Epilogue &E,
                       cudaStream_t s) {
    // 32 features a CTA once that gives every SM a CTA
    const bool split = N < 32 * device_sm_count();
    return split ? launch_pdl(linear_few_kernel<T, MT, true>, dim3((N + 3) / 4), dim3(256), 0, s, x, ld_x, W, ld_w, M, N, K, E)
                 : launch_pdl(linear_few_kernel<T, MT, false>, dim3((N + 31) / 32), dim3(256), 0, s, x, ld_x, W, ld_w, M, N, K, E);
}
template <typename T>
cudaError_t launch_few(const void *x, int64_t ld_x, const void *W, int64_t ld_w, int M, int N, int K, const Epilogue &E,
                       cudaStream_t s) {
    if (M <= 1) return launch_few<T, 1>((const T *)x, ld_x, (const T *)W, ld_w, M, N, K, E, s);
    if (M <= 4) return launch_few<T, 4>((const T *)x, ld_x, (const T *)W, ld_w, M, N, K, E, s);
    return launch_few<T, FEW>((const T *)x, ld_x, (const T *)W, ld_w, M, N, K, E, s);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
inline int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
// Rows that the TMA takes as they are (strides of 0 or below the row's length are laid out).
inline bool on16(const void *p, int64_t ld, int rows, int K) {
    return (uintptr_t)p % 16 == 0 && (rows <= 1 || (ld % 8 == 0 && ld >= K && ld < (int64_t(1) << 38)));
}

// How a call goes: which operands are laid out anew, and how many features of W at once.
struct Plan {
    bool few, lay_x, lay_w;
    int planes, chunk;
    int64_t cols, ld;      // columns of a plane, row of the layout
    size_t x_bytes, w_bytes;
};
Plan plan(const void *x, int64_t ld_x, const void *W, int64_t ld_w, int dtype, int M, int N, int K) {
    Plan p{};
    p.planes = dtype == DSA_F32 ? 3 : 1;
    p.lay_x = dtype == DSA_F32 || !on16(x, ld_x, M, K);
    p.lay_w = dtype == DSA_F32 || !on16(W, ld_w, N, K);
    p.few = p.lay_w && M <= FEW;
    p.cols = up(K, p.planes == 3 ? 64 : 8);
    p.ld = p.cols * p.planes;
    p.chunk = N;
    if (p.lay_w)  // as many features as stay in L2 between the two kernels, but enough to fill the SMs
        p.chunk = (int)std::min<int64_t>(N, std::max<int64_t>(2048, (64 << 20) / (p.ld * 2) / BF * BF));
    if (!p.few) {
        p.x_bytes = p.lay_x ? up((int64_t)M * p.ld * 2, 256) : 0;
        p.w_bytes = p.lay_w ? up((int64_t)p.chunk * p.ld * 2, 256) : 0;
    }
    return p;
}

cudaError_t lay_out(const void *src, int64_t ld, int dtype, int64_t rows, int K, const Plan &p, void *dst, cudaStream_t s) {
    const int64_t n = (rows * (p.cols / 8) + 255) / 256;
    if (n > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const cudaError_t e =
        dtype == DSA_F32
            ? launch_pdl(linear_layout_kernel<true>, dim3((unsigned)n), dim3(256), 0, s, src, ld, (__nv_bfloat16 *)dst, rows, K, (int)p.cols, p.ld)
            : launch_pdl(linear_layout_kernel<false>, dim3((unsigned)n), dim3(256), 0, s, src, ld, (__nv_bfloat16 *)dst, rows, K, (int)p.cols, p.ld);
    if (e == cudaSuccess) note_launch(DSA_KERNEL_LINEAR_LAYOUT);
    return e;
}

cudaError_t launch_tiles(const void *x, int64_t ld_x, const void *W, int64_t ld_w, int K, int plane, LinearParams &P,
                         cudaStream_t s) {
    const int sms = device_sm_count();
    P.slabs = (K + 63) / 64;
    P.total = plane ? 6 * P.slabs : P.slabs;
    const bool exact = P.e.f32 && P.total > CHAIN;
    P.chain = exact ? CHAIN : P.total;
    const int most = exact ? MAX_EXACT : MAX_BT;
    P.tt = (P.M + most - 1) / most;
    P.bt = (int)up((P.M + P.tt - 1) / P.tt, 16);
    P.tt = (P.M + P.bt - 1) / P.bt;
    const int64_t tiles = (int64_t)P.tt * ((P.N + BF - 1) / BF);
    if (tiles > 0x3fffffff) return cudaErrorInvalidConfiguration;
    P.tiles = (int)tiles;
    P.plane = plane;
    P.stage_bytes = W_SLAB + P.bt * 128;
    P.wait_limit = wait_limit_cycles();
    P.share = 1;
    while (P.share < 8 && tiles * P.share * 2 <= sms && P.total >= P.share * 2 * 4) P.share *= 2;
    const bool split = P.share > 1;
    P.stages = std::min(MAX_STAGES, (SMEM_MAX - 2048 - (split ? 0 : TURN)) / P.stage_bytes);
    const int smem = 1024 + P.stages * P.stage_bytes + (split ? 0 : TURN);
    CUtensorMap tw, tx;
    const uint64_t wide = plane ? 3 * (uint64_t)plane : (uint64_t)K;
    {
        const uint64_t dims[2] = {wide, (uint64_t)P.N}, strides[1] = {(uint64_t)ld_w * 2};
        const uint32_t box[2] = {64, BF};
        if (!make_tmap(&tw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, W, dims, strides, box)) return cudaErrorInvalidValue;
    }
    {
        const uint64_t dims[2] = {wide, (uint64_t)P.M}, strides[1] = {(uint64_t)ld_x * 2};
        const uint32_t box[2] = {64, (uint32_t)P.bt};
        if (!make_tmap(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, dims, strides, box)) return cudaErrorInvalidValue;
    }
    auto *kernel = split ? exact ? linear_kernel<true, true> : linear_kernel<true, false>
                         : exact ? linear_kernel<false, true> : linear_kernel<false, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX - 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split ? P.tiles * P.share : std::min(P.tiles, sms));
    cfg.blockDim = dim3(NUM_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)P.share, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = split ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, tw, tx, P);
    if (e == cudaSuccess) note_launch(DSA_KERNEL_LINEAR);
    return e;
}

int check_linear(const void *x, int64_t ld_x, const void *W, int64_t ld_w, int dtype, int M, int N, int K) {
    if (M < 0 || N < 1 || K < 1) return DSA_ERR_INVALID_ARG;
    if (dtype != DSA_F32 && dtype != DSA_BF16) return DSA_ERR_UNSUPPORTED;
    if (M >= 0x7fffffff - 1024 || N >= 0x7fffffff - 1024 || K >= 0x7fffffff - 1024) return DSA_ERR_UNSUPPORTED;
    // a plane's columns are counted in 32 bits, and a row of the tensor map in 40
    if (dtype == DSA_F32 && K >= 0x7fffffff / 6 - 64) return DSA_ERR_UNSUPPORTED;
    const size_t e = dtype == DSA_F32 ? 4 : 2;
    if ((uintptr_t)x % e || (uintptr_t)W % e) return DSA_ERR_INVALID_ARG;
    if ((M > 1 && ld_x < 0) || (N > 1 && ld_w < 0)) return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

}  // namespace

int linear_read_error(int *site) {
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_linear_error, sizeof(int));
    if (e != cudaSuccess) return fail_cuda(e);
    if (v) {
        e = cudaMemcpyToSymbol(g_linear_error, &zero, sizeof(int));
        if (e != cudaSuccess) return fail_cuda(e);
        if (site) *site = v;
        return DSA_ERR_TIMEOUT;
    }
    return DSA_OK;
}

}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_linear_workspace_size(const void *x, int64_t ld_x, const void *W, int64_t ld_w, int dtype, int M, int N,
                                            int K) {
    if (check_linear(x, ld_x, W, ld_w, dtype, M, N, K) || M == 0) return 0;
    const Plan p = plan(x, ld_x, W, ld_w, dtype, M, N, K);
    return p.x_bytes + p.w_bytes;
}

extern "C" int dsa_linear(const void *x, int64_t ld_x, const void *W, int64_t ld_w, int dtype, int M, int N, int K,
                          const float *bias, int act, const void *residual, int64_t ld_r, void *y, int64_t ld_y,
                          int y_dtype, void *workspace, size_t ws_bytes, void *stream) {
    reset_trace();
    int rc = check_linear(x, ld_x, W, ld_w, dtype, M, N, K);
    if (rc) return rc;
    if (y_dtype != DSA_F32 && y_dtype != DSA_BF16) return DSA_ERR_UNSUPPORTED;
    if (act < DSA_ACT_NONE || act > DSA_ACT_GELU_TANH) return DSA_ERR_UNSUPPORTED;
    const size_t ey = y_dtype == DSA_F32 ? 4 : 2;
    if ((uintptr_t)y % ey || (uintptr_t)residual % ey || (uintptr_t)bias % 4) return DSA_ERR_INVALID_ARG;
    if (M == 0) return DSA_OK;
    if (!x || !W || !y || y == x || y == W) return DSA_ERR_INVALID_ARG;
    if (M > 1 && ld_y < N) return DSA_ERR_INVALID_ARG;  // rows of y that overlap
    if (residual == y && M > 1 && ld_r != ld_y) return DSA_ERR_INVALID_ARG;
    const Plan p = plan(x, ld_x, W, ld_w, dtype, M, N, K);
    if (p.x_bytes + p.w_bytes > 0 &&
        (!workspace || (uintptr_t)workspace % 256 || ws_bytes < p.x_bytes + p.w_bytes))
        return DSA_ERR_WORKSPACE;
    const cudaStream_t s = (cudaStream_t)stream;
    Epilogue E;
    E.bias = bias;
    E.res = residual;
    E.y = y;
    E.ld_r = ld_r;
    E.ld_y = ld_y;
    E.act = act;
    E.f32 = y_dtype == DSA_F32;
    const size_t four = 4 * ey;
    E.vec = N % 4 == 0 && (uintptr_t)y % four == 0 && (M <= 1 || ld_y % 4 == 0) &&
            (!residual || ((uintptr_t)residual % four == 0 && (M <= 1 || ld_r % 4 == 0)));
    cudaError_t e;
    if (p.few) {
        e = dtype == DSA_F32 ? launch_few<float>(x, ld_x, W, ld_w, M, N, K, E, s)
                             : launch_few<__nv_bfloat16>(x, ld_x, W, ld_w, M, N, K, E, s);
        if (e != cudaSuccess) return fail_cuda(e);
        note_launch(DSA_KERNEL_LINEAR_SIMT);
        return DSA_OK;
    }
    const int64_t rows_x = M > 1 ? ld_x : up(K, 8), rows_w = N > 1 ? ld_w : up(K, 8);
    if (p.lay_x) {
        e = lay_out(x, ld_x, dtype, M, K, p, workspace, s);
        if (e != cudaSuccess) return fail_cuda(e);
    }
    const void *xs = p.lay_x ? workspace : x;
    for (int n0 = 0; n0 < N; n0 += p.chunk) {
        const int n = std::min(p.chunk, N - n0);
        const void *ws = W;
        if (p.lay_w) {
            ws = (char *)workspace + p.x_bytes;
            const char *from = (const char *)W + (int64_t)n0 * ld_w * (dtype == DSA_F32 ? 4 : 2);
            e = lay_out(from, ld_w, dtype, n, K, p, (void *)ws, s);
            if (e != cudaSuccess) return fail_cuda(e);
        }
        LinearParams P{};
        P.e = E;
        if (bias) P.e.bias = bias + n0;
        P.e.y = (char *)y + n0 * ey;
        if (residual) P.e.res = (const char *)residual + n0 * ey;
        P.M = M;
        P.N = n;
        e = launch_tiles(xs, p.lay_x ? p.ld : rows_x, ws, p.lay_w ? p.ld : rows_w, K, p.planes == 3 ? (int)p.cols : 0, P, s);
        if (e != cudaSuccess) return fail_cuda(e);
    }
    return DSA_OK;
}
