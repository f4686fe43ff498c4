// A linear layer with its epilogue, y = act(x W^T + bias) + residual, on tcgen05 tensor cores.
//
// A tile is 128 features (rows of W: the MMA's M) times up to 256 tokens (rows of x: its N), so
// a decode step of few tokens wastes none of the tensor cores' rows on padding and streams W
// with MMAs of N = 16: y^T = W x^T.  Per tile:
//   * warp 0 streams 64-wide K slabs of W (128 rows) and of x by TMA, 128-byte
//     swizzled, through a ring that takes what shared memory there is (4 stages at 256 tokens,
//     12 at 16: 200 KB in flight per SM keep HBM busy);
//   * warp 1 issues the MMAs into one of two fp32 accumulators in tensor memory;
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
// (32 steps; fp32 layers: 4) and adds these parts to nearest in its registers: 4.7e-7 of the whole (fp32 layers 2.4e-7) at any K.
// A sum of one part is as it was cut off: over K = 512 in bf16 4.7e-7, where fp32 arithmetic loses 1.6e-7.
//
// fp32 layers run on the same kernel: a value is the sum of three bf16 terms of 8 bits each (planes),
// and of the nine products of terms the six above 2^-24 of the whole are added.  A stage holds
// all planes of a slab, x's one behind the other, so that W's plane p meets x's planes 0 .. 2 - p in
// one MMA of as many times the tokens: W is read three times instead of six (1000 tokens, 2048
// to 5000: 189 -> 122 us).  Products of one order share an accumulator; the three are added last.
// Rows that do not start on 16 bytes, and fp32 ones, are laid out anew first (linear_layout_kernel);
// of a large fp32 W and few tokens, or of little work, the epilogue's warps make the planes themselves
// (RAW), bound by shared memory, which a slab passes three times (17 tokens, 7168 to 7168: 134 -> 73 us).
//
// Bound by HBM with few tokens (17 tokens, 7168 to 131,072, fp32 out: 267 to 272 us, 1.02 of the measured copy
// rate; 64 tokens, 16384 to 7168: 43 us, 0.81, the rest being the start and the end of a tile), by shared memory with
// many (4096 tokens, 16384 to 7168: 535 us by itself, 1.80 PFLOP/s or 0.94 of the measured peak, and 593 to 609 call after call, when
// power limits it: a slab is written once and read by the MMAs once, 96 KB in 730 cycles of which the MMAs need 512).
#include <atomic>
#include <type_traits>

#include "tc_common.cuh"

namespace dsa {

__device__ int g_linear_error = 0;

namespace {

constexpr int BF = 128, MAX_BT = 256;             // features, tokens of a tile
// Where a tile's operands come from: bf16 rows by TMA; planes of fp32 rows by TMA; fp32 rows, by the epilogue's warps.
enum { ROWS, PLANES, RAW };
constexpr int planes_of(int src) { return src == ROWS ? 1 : 3; }
// Tokens of a tile: the MMA's N is that or, with planes, three times that; less where exact sums take registers or rows on
// their way shared memory.
constexpr int max_bt(bool exact, int src) { return src == RAW ? 64 : src == PLANES ? 80 : exact ? 128 : MAX_BT; }
constexpr int W_SLAB = BF * 128;                  // 16 KB: 128 rows x 64 bf16
constexpr int MAX_STAGES = 12;
constexpr int NUM_THREADS = 384;                  // 0 TMA, 1 MMA, 2 TMEM owner, 3 idle, 4-11 epilogue
constexpr int EPI_WARP0 = 4, EPI_THREADS = 256;
constexpr int TURN = 2 * 32 * BF * 4;             // 32 tokens x 128 features in fp32 for each half of the epilogue
constexpr int SMEM_MAX = 232448;
constexpr int chain_of(int planes) { return planes == 3 ? 4 : 8; }  // slabs of an exact sum's parts
constexpr int MAX_SHARE = 8;                      // CTAs that share a tile's K
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
    int total, K;         // slabs (64 columns) of K
    const void *w, *x;    // RAW: the operands and their row strides
    int64_t ld_w, ld_x;
    int deep, raw_bytes;  // RAW: slabs that are on their way, bytes of one
    int stages, stage_bytes;
    int share;            // CTAs that share a tile's K (SPLIT)
    int acc_cols, tmem_cols;  // columns from one accumulator to the next; of tensor memory
    int chain;            // slabs that are added up in tensor memory (all, or with EXACT a part)
    long long wait_limit;
};

template <int ACT>
__device__ __forceinline__ float activation(float v) {
    if (ACT == DSA_ACT_RELU) return v < 0.0f ? 0.0f : v;  // a NaN stays
    // the quotient to 2 units in the last place, 0 where it is next to nothing: with full division 777 tokens, 2048 to 5000, took
    // 32 us instead of 20
    if (ACT == DSA_ACT_SILU) return __fdividef(v, 1.0f + expf(-v));
    if (ACT == DSA_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678f));
    if (ACT == DSA_ACT_GELU_TANH) return 0.5f * v * (1.0f + tanhf(0.79788456f * fmaf(0.044715f * v * v, v, v)));
    return v;
}
template <int ACT, int N>
__device__ __forceinline__ void activation(float (&v)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = activation<ACT>(v[j]);
}
// One branch for all values: a branch for each made so much code that a tile's end waited 7 us for it.
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
    switch (act) {
        case DSA_ACT_RELU: return activation<DSA_ACT_RELU>(v);
        case DSA_ACT_SILU: return activation<DSA_ACT_SILU>(v);
        case DSA_ACT_GELU: return activation<DSA_ACT_GELU>(v);
        case DSA_ACT_GELU_TANH: return activation<DSA_ACT_GELU_TANH>(v);
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
// One value.
__device__ __forceinline__ float residual1(const Epilogue &E, int64_t row, int f) {
    return E.f32 ? ((const float *)E.res)[row * E.ld_r + f] : to_f32(((const __nv_bfloat16 *)E.res)[row * E.ld_r + f]);
}
__device__ __forceinline__ void store1(const Epilogue &E, int64_t row, int f, float v) {
    if (E.f32) ((float *)E.y)[row * E.ld_y + f] = v;
    else ((__nv_bfloat16 *)E.y)[row * E.ld_y + f] = from_f32<__nv_bfloat16>(v);
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

// The producer and the MMA issuer are whole warps in convergence, of which one lane issues: what they hand to an instruction
// then stays in uniform registers.  From a single lane's branch a slab took them 510 and 570 cycles.
__device__ __forceinline__ void expect_if(uint32_t issue, uint64_t *bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(tc::smem_u32(bar)),
        "r"(bytes), "r"(issue)
        : "memory");
}
template <int SRC>  // all planes of the rows at once
__device__ __forceinline__ void load_if(uint32_t issue, void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y) {
    if constexpr (planes_of(SRC) == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
            "[%2];\n\t}" ::"r"(tc::smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(x), "r"(y), "r"(issue)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
            "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
            "[%2];\n\t}" ::"r"(tc::smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(x), "r"(y), "r"(0), "r"(issue)
            : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t issue, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc::smem_u32(bar)),
        "r"(issue)
        : "memory");
}
// mbar_wait for a warp in convergence: every lane has the same answer.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *err, int site,
                                          long long limit = tc::kWaitLimitCycles) {
    const uint32_t a = tc::smem_u32(bar);
    if (__all_sync(0xffffffffu, tc::mbar_try_wait(a, parity))) return true;
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, tc::mbar_try_wait(a, parity))) {
        if (__any_sync(0xffffffffu, *abort_flag)) return false;
        if (__any_sync(0xffffffffu, clock64() - t0 > limit)) {
            atomicCAS(err, 0, site);
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}

// The epilogue's wait for an accumulator.  A limit that is set is polled for: the hardware's own patience is longer than a part of
// a sum takes, so that no limit would run out.
__device__ __forceinline__ bool wait_sum(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *err, int site, long long limit) {
    if (limit >= tc::kWaitLimitCycles) return tc::mbar_wait(bar, parity, abort_flag, err, site);
    const long long t0 = clock64();
    while (!tc::mbar_test(bar, parity)) {
        if (*abort_flag) return false;
        if (clock64() - t0 > limit) {
            atomicCAS(err, 0, site);
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void tile_of(const LinearParams &P, int u, int &m0, int &f0) {
    const int ft = (P.N + BF - 1) / BF, per_group = GROUP_T * ft;
    const int grp = u / per_group, r = u - grp * per_group;
    const int gt = min(GROUP_T, P.tt - grp * GROUP_T);
    m0 = (grp * GROUP_T + r % gt) * P.bt;
    f0 = (r / gt) * BF;
}

// Eight fp32 values as three planes of bf16 terms, each the nearest to what the terms before it leave (above the largest bf16
// number that and what is left; infinities and NaN in the first plane alone).
constexpr float BF16_MAX = 3.38953139e38f;
__device__ __forceinline__ void split_eight(const float (&v)[8], uint32_t (&o)[3][4]) {
    bool large = false;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float a = v[e], b = v[e + 1];
        large |= !(fabsf(a) <= BF16_MAX) || !(fabsf(b) <= BF16_MAX);
#pragma unroll
        for (int t = 0; t < 3; ++t) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            o[t][e / 2] = *(const uint32_t *)&h;
            a -= __uint_as_float(o[t][e / 2] << 16);
            b -= __uint_as_float(o[t][e / 2] & 0xffff0000u);
        }
    }
    if (large) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float a = v[e];
            if (fabsf(a) <= BF16_MAX) continue;
            const bool finite = fabsf(a) < INFINITY;
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                const float h = t == 0 && finite ? copysignf(BF16_MAX, a) : __bfloat162float(__float2bfloat16_rn(a));
                const uint32_t bits = __float_as_uint(h) >> 16;
                o[t][e / 2] = e & 1 ? (o[t][e / 2] & 0xffffu) | bits << 16 : (o[t][e / 2] & 0xffff0000u) | bits;
                a = finite ? a - h : 0.0f;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// RAW: a warp copies four rows of a slab at a time to shared memory, as they are, and turns them into planes in the MMAs'
// layout a slab or more later: eight lanes a row, eight values each.  Copied are the whole 16 bytes (chunks) that values
// of the row lie in; each holds one, so it lies in memory that is there.
// ---------------------------------------------------------------------------
constexpr int RAW_ROW = 256;
// Where chunk c of a row lies: chunks 0..7, 8..15, the even and the odd ones each pass all banks once.
__device__ __forceinline__ int chunk_at(int c) { return (c ^ ((c >> 3) & 1)) * 16; }
__device__ __forceinline__ void copy16_if(bool there, uint32_t dst, const char *src) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst), "l"(src),
                 "r"((int)there)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// A lane's two chunks of a row's slab; bytes: from the slab's start to the row's end.
__device__ __forceinline__ void copy_row(uint32_t dst, const char *from, int part8, int bytes) {
#pragma unroll
    for (int i = 0; i < 2; ++i) copy16_if((i * 8 + part8) * 16 < bytes, dst + chunk_at(i * 8 + part8), from + i * 128);
}
// To dst, and the further planes `plane` bytes on; left: values to the row's end.
template <bool TAIL>
__device__ __forceinline__ void store_eight(const uint4 &a, const uint4 &b, int left, uint8_t *dst, int plane) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = TAIL && e >= left ? 0.0f : __uint_as_float(w[e]);
    uint32_t o[3][4];
    split_eight(v, o);
#pragma unroll
    for (int t = 0; t < 3; ++t) *(uint4 *)(dst + t * plane) = make_uint4(o[t][0], o[t][1], o[t][2], o[t][3]);
}

template <bool SPLIT, bool EXACT, int SRC>
__global__ void __launch_bounds__(NUM_THREADS, SPLIT && !EXACT && SRC == ROWS ? 2 : 1)
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

    // One slab's loads, by the lane of `issue`.
    const auto load = [&](uint32_t issue, int st, int ks, int m0, int f0) {
        uint8_t *sw = ring + st * P.stage_bytes;
        expect_if(issue, &full[st], P.stage_bytes);
        load_if<SRC>(issue, sw, &tm_w, &full[st], ks * 64, f0);
        load_if<SRC>(issue, sw + planes_of(SRC) * W_SLAB, &tm_x, &full[st], ks * 64, m0);
    };
    // The producer's first loads go out before the CTA has met, while warp 2 waits for tensor memory.
    const int ahead_slabs = SRC != RAW && mine > 0 ? min(s1 - s0, P.stages) : 0;
    if (warp == 0) {
        int m0, f0;
        tile_of(P, who, m0, f0);
        const uint32_t issue = tc::elect_one();
        if (lane == 0) {
            if (SRC != RAW) {
                tc::prefetch_tmap(&tm_w);
                tc::prefetch_tmap(&tm_x);
            }
            for (int i = 0; i < P.stages; ++i) {
                tc::mbar_init(&full[i], SRC == RAW ? EPI_THREADS / 32 : 1);
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
        __syncwarp();
        pdl_wait();  // the set-up above overlapped the previous kernel; global memory only from here
        for (int j = 0; j < ahead_slabs; ++j) load(issue, j, s0 + j, m0, f0);
    } else if (warp == 2) {
        tc::tmem_alloc(&tmem_slot, P.tmem_cols);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    if (warp != 0) pdl_wait();

    if (SRC != RAW && warp == 0) {
        // ---------------- TMA producer ----------------
        const uint32_t issue = tc::elect_one();
        int it = ahead_slabs, st = ahead_slabs == P.stages ? 0 : ahead_slabs, round = ahead_slabs == P.stages ? 1 : 0;
        bool ok = true;
        for (int i = 0; ok && i < mine; ++i) {
            int m0, f0;
            tile_of(P, who + i * step, m0, f0);
            for (int ks = i > 0 ? s0 : s0 + ahead_slabs; ks < s1; ++ks, ++it) {
                if (!(ok = wait_warp(&empty[st], (round & 1) ^ 1, abort_flag, err, 61, P.wait_limit))) break;
                load(issue, st, ks, m0, f0);
                if (++st == P.stages) st = 0, ++round;
            }
        }
        // Drain: nothing may still be landing in shared memory when the CTA goes on.
        for (int j = max(0, it - P.stages); j < it; ++j) wait_warp(&full[j % P.stages], (j / P.stages) & 1, nv, err, 62);
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        const uint32_t issue = tc::elect_one();
        const uint32_t idesc = tc::instr_desc(tc::kFmtBF16, tc::kFmtBF16, BF, planes_of(SRC) * P.bt, 0, 0);
        const uint32_t idesc2 = tc::instr_desc(tc::kFmtBF16, tc::kFmtBF16, BF, 2 * P.bt, 0, 0);
        const uint32_t idesc1 = tc::instr_desc(tc::kFmtBF16, tc::kFmtBF16, BF, P.bt, 0, 0);
        const uint64_t first = tc::smem_desc(tc::smem_u32(ring), 16, 1024);
        int st = 0, round = 0, issued = 0, n = 0;
        bool ok = true;
        for (int i = 0; ok && i < mine; ++i) {
            for (int k0 = s0; ok && k0 < s1; k0 += P.chain, ++n) {
                const int acc = n & 1, k1 = min(s1, k0 + P.chain);
                if (!(ok = wait_warp(&tempty[acc], ((n >> 1) & 1) ^ 1, abort_flag, err, 63, P.wait_limit))) break;
                const uint32_t d = tmem + acc * P.acc_cols;
                for (int ks = k0; ks < k1; ++ks) {
                    if (!(ok = wait_warp(&full[st], round & 1, abort_flag, err, 64, P.wait_limit))) break;
                    tc::tc_fence_after();
                    // addresses in a descriptor count 16 bytes and stay below its 14 bits
                    const uint64_t wd = first + (uint32_t)(st * P.stage_bytes / 16), xd = wd + planes_of(SRC) * W_SLAB / 16;
                    if (planes_of(SRC) == 1) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc::mma_f16_if(issue, d, wd + kk * 2, xd + kk * 2, idesc, ks != k0 || kk != 0);
                    } else {
                        // W's plane p times x's planes 0 .. 2 - p, which lie one behind the other: one MMA of as many times the
                        // tokens, into the accumulators of the orders p .. 2
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                            for (int p = 0; p < planes_of(SRC); ++p)
                                tc::mma_f16_if(issue, d + p * P.bt, wd + p * (W_SLAB / 16) + kk * 2, xd + kk * 2,
                                               p == 0 ? idesc : p == 1 ? idesc2 : idesc1, ks != k0 || kk != 0 || p != 0);
                    }
                    commit_if(issue, &empty[st]);
                    ++issued;
                    if (++st == P.stages) st = 0, ++round;
                }
                if (ok) commit_if(issue, &tfull[acc]);
            }
        }
        // No MMA may still be running when the tensor memory is released.
        if (issued > 0) {
            commit_if(issue, &mmadone);
            wait_warp(&mmadone, 0, nv, err, 65);
        }
    } else if (warp >= EPI_WARP0) {
        // ---------------- epilogue ----------------
        // Warp (q, g): TMEM lanes (features) 32q .. 32q + 31, every other chunk of 32 tokens.
        const int q = warp & 3, g = (warp - EPI_WARP0) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        float *part = (float *)ring;           // SPLIT: [tokens][BF], once every load of the ring has landed and been used
        float *mine_turn = turn + g * 32 * BF;
        int n = 0, st = 0, round = 0;
        for (int i = 0; i < mine; ++i) {
            int m0, f0;
            tile_of(P, who + i * step, m0, f0);
            const int tokens = min(P.bt, P.M - m0);
            const int f = f0 + q * 32 + lane, f4 = f0 + lane * 4;
            const float b = !SPLIT && P.e.bias && f < P.N ? __ldg(P.e.bias + f) : 0.0f;
            const bool ahead = !SPLIT && !EXACT && P.e.res;  // EXACT has no registers to spare
            const auto residuals = [&](int64_t row, float (&r)[4]) {  // of a token, as this lane stores it
                if (P.e.vec) {
                    if (f4 < P.N) residual4(P.e, row, f4, r);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (f0 + e * 32 + lane < P.N) r[e] = residual1(P.e, row, f0 + e * 32 + lane);
                }
            };
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
                        if (row0 + j < P.M) residuals(row0 + j, r[j]);
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] += b;
                activate(v, P.e.act);
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
                } else if (!P.e.res) {
                    for (int j = 0; j < left; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (f0 + e * 32 + lane < P.N)
                                store1(P.e, row0 + j, f0 + e * 32 + lane, mine_turn[(q * 8 + j) * BF + e * 32 + lane]);
                } else {
                    // residuals before the first store, which no load passes: one after the other took 4096 tokens, 2048 to 7166,
                    // 328 us instead of 183, and 7966, 810 to 26446, bf16 with residual and y in fp32, 2799 instead of 700 to 725
#pragma unroll
                    for (int h = 0; h < 8; h += 4) {
                        if (EXACT)
#pragma unroll
                            for (int j = h; j < h + 4; ++j)
                                if (j < left) residuals(row0 + j, r[j]);
#pragma unroll
                        for (int j = h; j < h + 4; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (j < left && f0 + e * 32 + lane < P.N)
                                    store1(P.e, row0 + j, f0 + e * 32 + lane, mine_turn[(q * 8 + j) * BF + e * 32 + lane] + r[j][e]);
                    }
                }
            };
            const auto read = [&](int c, float (&v)[32]) {  // tokens c .. c + 31 of the accumulator
                const uint32_t at = lanes + (n & 1) * P.acc_cols + c;
                if constexpr (planes_of(SRC) == 1) {
                    tc::tmem_ld32(at, v);
                    tc::tmem_ld_wait();
                } else {
                    float u[32];
                    tc::tmem_ld32(at + 2 * P.bt, u);
                    tc::tmem_ld32(at + P.bt, v);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) u[e] += v[e];
                    tc::tmem_ld32(at, v);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] += u[e];
                }
            };
            constexpr int SUMS = EXACT ? (max_bt(EXACT, SRC) + 63) / 64 : 1;
            float sum[SUMS][32];
            // EXACT: takes the next part over from tensor memory, where all warps are sound.
            const auto drain = [&](bool sound) -> bool {
                if (!epi_and(sound && wait_sum(&tfull[n & 1], (n >> 1) & 1, abort_flag, err, 66, P.wait_limit))) return false;
                tc::tc_fence_after();
#pragma unroll
                for (int j = 0; j < SUMS; ++j)
                    if (j * 64 + g * 32 < tokens) {
                        float v[32];
                        read(j * 64 + g * 32, v);
#pragma unroll
                        for (int e = 0; e < 32; ++e) sum[j][e] += v[e];
                    }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&tempty[n & 1]);
                ++n;
                return true;
            };
            if (EXACT) {
#pragma unroll
                for (int j = 0; j < SUMS; ++j)
#pragma unroll
                    for (int e = 0; e < 32; ++e) sum[j][e] = 0.0f;
            }
            int parts = (s1 - s0 + P.chain - 1) / P.chain;  // yet to be taken over
            bool ok = true;
            if constexpr (SRC == RAW) {
                // Rows r0, r0 + 32 and so on.  Rows behind the last one are its, or one 32 rows before: what they give is
                // stored nowhere.
                constexpr int XS = (max_bt(EXACT, SRC) + 31) / 32;
                const int r0 = (warp - EPI_WARP0) * 4 + (lane >> 3), part8 = lane & 7;  // row of the first 32, eighth of a slab
                const int fw = min(f0 + r0, P.N - 1), mx = m0 + min(r0, tokens - 1);
                const int last_w = (P.N - 1 - fw) / 32, last_x = (m0 + tokens - 1 - mx) / 32;
                const char *pw[4], *px[XS];  // this lane's first chunk of each row, in the next slab to copy
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    pw[j] = (const char *)P.w + ((fw + min(j, last_w) * 32) * P.ld_w + (int64_t)s0 * 64) * 4 + part8 * 16;
#pragma unroll
                for (int j = 0; j < XS; ++j)
                    px[j] = (const char *)P.x + ((mx + min(j, last_x) * 32) * P.ld_x + (int64_t)s0 * 64) * 4 + part8 * 16;
                uint8_t *raw = ring + P.stages * P.stage_bytes + (SPLIT ? 0 : TURN) + r0 * RAW_ROW;
                const auto fetch = [&](int ks, int slot) {
                    const uint32_t to = tc::smem_u32(raw) + slot * P.raw_bytes;
                    const int bytes = ks < s1 ? min(P.K - ks * 64, 64) * 4 : 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        copy_row(to + j * 32 * RAW_ROW, pw[j], part8, bytes);
                        pw[j] += 256;
                    }
#pragma unroll
                    for (int j = 0; j < XS; ++j)
                        if (r0 + j * 32 < P.bt) {
                            copy_row(to + (j + 4) * 32 * RAW_ROW, px[j], part8, bytes);
                            px[j] += 256;
                        }
                    copies_commit();
                };
                for (int d = 0; d < P.deep; ++d) fetch(s0 + d, d);
                int slot = 0;
                uint4 w[4][2], x[XS][2];
                const auto store = [&](auto tail, uint8_t *to, int left) {
                    constexpr bool TAIL = decltype(tail)::value;
#pragma unroll
                    for (int j = 0; j < 4; ++j) store_eight<TAIL>(w[j][0], w[j][1], left, to + j * 4096, W_SLAB);
                    to += 3 * W_SLAB;
#pragma unroll
                    for (int j = 0; j < XS; ++j)
                        if (r0 + j * 32 < P.bt) store_eight<TAIL>(x[j][0], x[j][1], left, to + j * 4096, P.bt * 128);
                };
                const auto take = [&](uint4 (&c)[2], const uint8_t *row) {
                    c[0] = *(const uint4 *)(row + chunk_at(part8 * 2));
                    c[1] = *(const uint4 *)(row + chunk_at(part8 * 2 + 1));
                };
                // A warp whose wait ran out goes on to where all of them meet.
                for (int ks = s0; ks < s1; ++ks) {
                    if (ok) {
                        if (P.deep == 1) copies_wait<0>();
                        else if (P.deep == 2) copies_wait<1>();
                        else copies_wait<2>();
                        __syncwarp();
                        const uint8_t *rows = raw + slot * P.raw_bytes;
#pragma unroll
                        for (int j = 0; j < 4; ++j) take(w[j], rows + j * 32 * RAW_ROW);
#pragma unroll
                        for (int j = 0; j < XS; ++j)
                            if (r0 + j * 32 < P.bt) take(x[j], rows + (j + 4) * 32 * RAW_ROW);
                        __syncwarp();
                        fetch(ks + P.deep, slot);
                        if (++slot == P.deep) slot = 0;
                        ok = wait_warp(&empty[st], (round & 1) ^ 1, abort_flag, err, 61, P.wait_limit);
                    }
                    if (ok) {
                        uint8_t *to = ring + st * P.stage_bytes + ((part8 ^ (r0 & 7)) << 4) + r0 * 128;  // the 128-byte swizzle
                        if (ks * 64 + 64 <= P.K) store(std::false_type{}, to, 64);
                        else store(std::true_type{}, to, P.K - ks * 64 - part8 * 8);
                        tc::fence_proxy_async_smem();  // the MMAs read what these threads wrote
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&full[st]);
                        if (++st == P.stages) st = 0, ++round;
                    }
                    // the part before the one that this slab ends: its products are done or nearly so
                    if (EXACT && (ks + 1 - s0) % P.chain == 0 && ks + 1 - s0 > P.chain) {
                        if (!(ok = drain(ok))) break;
                        --parts;
                    }
                }
                copies_wait<0>();
            }
            if (EXACT) {
                for (bool agreed = true; agreed && parts > 0; --parts) agreed = ok = drain(ok);
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < SUMS; ++j)
                    if (j * 64 + g * 32 < tokens) put(j * 64 + g * 32, sum[j]);
            } else {
                ok = epi_and(ok && wait_sum(&tfull[n & 1], (n >> 1) & 1, abort_flag, err, 66, P.wait_limit));
                if (!ok) break;
                tc::tc_fence_after();
                for (int c = g * 32; c < tokens; c += 64) {
                    float v[32];
                    read(c, v);
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
        int m0, f0;
        tile_of(P, who, m0, f0);
        tc::cluster_sync();  // every CTA's partial tile is in its shared memory
        const int units = min(P.bt, P.M - m0) * (BF / 4);
        const uint32_t part = tc::smem_u32(ring);
        // four features of a token at a time; the next one's parts are on their way while these are stored
        const auto fetch = [&](int u, float4 (&a)[MAX_SHARE]) {
#pragma unroll
            for (int k = 0; k < MAX_SHARE; ++k)
                if (k < share && u < units) a[k] = peer4(tc::map_peer(part + u * 16, k));
        };
        const int by = share * NUM_THREADS;
        float4 next[MAX_SHARE];
        int u = rank * NUM_THREADS + (int)threadIdx.x;
        fetch(u, next);
        for (; u < units; u += by) {
            const int f = f0 + (u % (BF / 4)) * 4;
            const int64_t row = m0 + u / (BF / 4);
            const bool live = f < P.N;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, r[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (live && P.e.res) {
                if (P.e.vec) residual4(P.e, row, f, r);
                else
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (f + e < P.N) r[e] = residual1(P.e, row, f + e);
            }
#pragma unroll
            for (int k = 0; k < MAX_SHARE; ++k)
                if (k < share) {
                    v[0] += next[k].x; v[1] += next[k].y; v[2] += next[k].z; v[3] += next[k].w;
                }
            fetch(u + by, next);
            if (!live) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (f + e < P.N) v[e] += P.e.bias ? __ldg(P.e.bias + f + e) : 0.0f;
            activate(v, P.e.act);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += r[e];
            if (P.e.vec) {
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
        tc::tmem_dealloc(tmem, P.tmem_cols);
    }
}

// ---------------------------------------------------------------------------
// Rows laid out for the TMA: bf16 rows copied to rows on 16 bytes; fp32 rows as three planes.
// ---------------------------------------------------------------------------
struct Layout {
    const void *src[2];       // x and W (rows 0: neither)
    __nv_bfloat16 *dst[2];
    int64_t ld[2], ld_dst;
    int rows[2], K, cols;     // cols: of a plane, K up to a multiple of 8 or 64
};

// A warp takes CHUNKS times 256 values of a row, a lane eight of each; all loads before the first use.
template <bool F32>
__global__ void __launch_bounds__(256) linear_layout_kernel(const __grid_constant__ Layout L) {
    constexpr int CHUNKS = F32 ? 1 : 4;
    pdl_wait();
    const int lane = threadIdx.x & 31, parts = (L.cols + CHUNKS * 256 - 1) / (CHUNKS * 256);
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    int64_t r = i / parts;
    const int k0 = (int)(i - r * parts) * (CHUNKS * 256) + lane * 8;
    const int which = r >= L.rows[0];
    if (which) r -= L.rows[0];
    if (r >= L.rows[which]) return;  // the whole warp
    __nv_bfloat16 *d = L.dst[which] + r * L.ld_dst + k0;
    if constexpr (F32) {
        if (k0 >= L.cols) return;
        const float *s = (const float *)L.src[which] + r * L.ld[which] + k0;
        float v[8];
        if (k0 + 8 <= L.K && (uintptr_t)s % 16 == 0) {
            const float4 a = *(const float4 *)s, b = *((const float4 *)s + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = k0 + e < L.K ? s[e] : 0.0f;
        }
        uint32_t o[3][4];
        split_eight(v, o);
#pragma unroll
        for (int p = 0; p < 3; ++p) *(uint4 *)(d + (int64_t)p * L.cols) = make_uint4(o[p][0], o[p][1], o[p][2], o[p][3]);
    } else {
        // The whole 16 bytes, one or two, that the lane's eight values lie in.  Each holds a value of the row, so it lies in
        // memory that is there.
        const uintptr_t at = (uintptr_t)((const uint16_t *)L.src[which] + r * L.ld[which] + k0);
        const int off = (int)(at & 15);  // the same in every lane
        uint4 a[CHUNKS], b[CHUNKS];
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const uintptr_t from = at - off + c * 512;
            const int64_t bytes = off + 2 * (int64_t)(L.K - k0 - c * 256);  // to the row's end
            a[c] = b[c] = make_uint4(0, 0, 0, 0);
            if (bytes > off) a[c] = *(const uint4 *)from;
            if (off && bytes > max(off, 16)) b[c] = *(const uint4 *)(from + 16);
        }
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const int k = k0 + c * 256;
            if (k >= L.cols) break;
            uint32_t w[8] = {a[c].x, a[c].y, a[c].z, a[c].w, b[c].x, b[c].y, b[c].z, b[c].w};
#pragma unroll
            for (int e = 0; e < 6; ++e) w[e] = off & 8 ? w[e + 2] : w[e];
#pragma unroll
            for (int e = 0; e < 5; ++e) w[e] = off & 4 ? w[e + 1] : w[e];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = __funnelshift_r(w[e], w[e + 1], (off & 2) * 8);
            if (k + 8 > L.K)
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // nothing behind the row's end
                    if (k + 2 * e >= L.K) w[e] = 0;
                    else if (k + 2 * e + 1 >= L.K) w[e] &= 0xffffu;
                }
            *(uint4 *)(d + c * 256) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ---------------------------------------------------------------------------
// Few tokens whose rows the TMA does not take (off 16 bytes, fp32): a pass over W to lay it out would cost several times what
// the product does, so a warp takes four features and up to 16 tokens (more: more CTAs, W from L2) and reads W as it is, V values at once.  SPLIT: the CTA's eight warps share K.  Bound by HBM for a token or two, then by the FMA pipes.
// ---------------------------------------------------------------------------
constexpr int FEW = 16;

template <typename T, int V>
__device__ __forceinline__ void read(const T *p, bool in, float (&v)[V]) {
    if constexpr (V == 4) {
        const float4 a = in ? *(const float4 *)p : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else {
        v[0] = in ? to_f32(*p) : 0.0f;
    }
}

template <typename T, int MT, int V, bool SPLIT>
__global__ void __launch_bounds__(256) linear_few_kernel(const T *x, int64_t ld_x, const T *W, int64_t ld_w, int M, int N, int K,
                                                         const __grid_constant__ Epilogue E) {
    constexpr int AHEAD = MT == 1 ? 8 / V : MT == 4 ? 4 / V : 2 / V + 1;  // loads of a feature in flight
    __shared__ float sums[8][4 * MT];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int f0 = SPLIT ? (int)blockIdx.x * 4 : ((int)blockIdx.x * 8 + warp) * 4, m0 = (int)blockIdx.y * MT;
    const int per = SPLIT ? ((K + 7) / 8 + 32 * V - 1) / (32 * V) * (32 * V) : K;
    const int k0 = min((int64_t)K, SPLIT ? (int64_t)warp * per : 0), k1 = (int)min((int64_t)K, (int64_t)k0 + per);
    float acc[4][MT];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[a][m] = 0.0f;
    const T *w[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) w[a] = W + (int64_t)min(f0 + a, N - 1) * ld_w;
    for (int k = k0 + lane * V; k < k1; k += 32 * V * AHEAD) {
        float wv[AHEAD][4][V];
#pragma unroll
        for (int h = 0; h < AHEAD; ++h)
#pragma unroll
            for (int a = 0; a < 4; ++a) read<T, V>(w[a] + k + h * 32 * V, k + h * 32 * V < k1, wv[h][a]);
#pragma unroll
        for (int h = 0; h < AHEAD; ++h)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float xv[V];
                read<T, V>(x + (int64_t)(m0 + m) * ld_x + k + h * 32 * V, m0 + m < M && k + h * 32 * V < k1, xv);
#pragma unroll
                for (int a = 0; a < 4; ++a)
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[a][m] = fmaf(wv[h][a][e], xv[e], acc[a][m]);
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
        const int wi = i / (4 * MT), at = i % (4 * MT), m = m0 + at / 4;
        const int f = SPLIT ? f0 + at % 4 : ((int)blockIdx.x * 8 + wi) * 4 + at % 4;
        if (m >= M || f >= N) continue;
        float v = sums[wi][at];
        if (SPLIT)
#pragma unroll
            for (int j = 1; j < 8; ++j) v += sums[j][at];
        float o[1] = {v + (E.bias ? E.bias[f] : 0.0f)};
        activate(o, E.act);
        if (E.res) o[0] += residual1(E, m, f);
        store1(E, m, f, o[0]);
    }
}

template <typename T, int MT, int V>
cudaError_t launch_few(const T *x, int64_t ld_x, const T *W, int64_t ld_w, int M, int N, int K, const Epilogue &E,
                       cudaStream_t s) {
    // 32 features a CTA once that gives every SM two
    const int groups = (M + MT - 1) / MT;
    const bool split = (int64_t)N * groups < 64 * device_sm_count();
    return split ? launch_pdl(linear_few_kernel<T, MT, V, true>, dim3((N + 3) / 4, groups), dim3(256), 0, s, x, ld_x, W, ld_w, M, N, K, E)
                 : launch_pdl(linear_few_kernel<T, MT, V, false>, dim3((N + 31) / 32, groups), dim3(256), 0, s, x, ld_x, W, ld_w, M, N, K, E);
}
template <typename T, int V>
cudaError_t launch_few(const void *x, int64_t ld_x, const void *W, int64_t ld_w, int M, int N, int K, const Epilogue &E,
                       cudaStream_t s) {
    if (M <= 1) return launch_few<T, 1, V>((const T *)x, ld_x, (const T *)W, ld_w, M, N, K, E, s);
    if (M <= 4) return launch_few<T, 4, V>((const T *)x, ld_x, (const T *)W, ld_w, M, N, K, E, s);
    return launch_few<T, FEW, V>((const T *)x, ld_x, (const T *)W, ld_w, M, N, K, E, s);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
inline int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
// bf16 rows that the TMA takes as they are (strides of 0 or below the row's length are laid out).
inline bool on16(const void *p, int64_t ld, int rows, int K) {
    return (uintptr_t)p % 16 == 0 && (rows <= 1 || (ld % 8 == 0 && ld >= K && ld < (int64_t(1) << 38)));
}

// How a call goes: which operands are laid out anew, and how many features of W at once.
struct Plan {
    bool few, lay_x, lay_w;
    int src, chunk;
    int64_t cols, ld;      // columns of a plane, row of the layout
    size_t x_bytes, w_bytes;
};
Plan plan(const void *x, int64_t ld_x, const void *W, int64_t ld_w, int dtype, int M, int N, int K) {
    Plan p{};
    const bool f32 = dtype == DSA_F32, x16 = !f32 && on16(x, ld_x, M, K), w16 = !f32 && on16(W, ld_w, N, K);
    // 7168 to 7168, this way and laid out: fp32 4 tokens 38 us and 135, 16 tokens 131 and 137 (1024 to 8192: 47 and 20);
    // bf16 off 16 bytes 1 token 26, 16 tokens 169 and 70.  Little work is worth no second launch: 8 tokens, 4096 to 1024 in
    // fp32, 15.2 and 15.4; 64, 1536 to 260, 8.3 and 10.1; 100, 256 to 256, 8.2 and 6.3; 30 tokens, 511 to 300 in bf16, 4.6
    // and 6.3; 100 of them 9.4 and 6.3
    p.few = !w16 && (M <= 4 || (M <= 64 && (double)M * N * K <= (f32 ? 3.5e7 : 6e6)));
    p.chunk = N;
    if (p.few) return p;
    p.src = f32 ? PLANES : ROWS;
    // RAW: of a large W, read once: 64 tokens, 7168 to 7168, 81 us and laid out 141 (17 tokens 73 and 134); 4096 to 2048 22 and 23,
    // 4096 to 1024 19 and 17, 16384 to 512 45 and 32; 80 tokens, two tiles, 138 and 140.  Of little work, for one launch and no
    // workspace, which are 8 us of the host's time (a call of 500 tokens, 1536 to 260, 25 -> 17 us), although the GPU takes longer,
    // which is what counts in a graph: 500 tokens, 1536 to 260, 15 and 12 us; 128, 2048 to 1024, 17 and 14; but 64, 7168 to
    // 256, 22 and 15
    const bool large = M <= max_bt(true, RAW) && N >= 2048 && (int64_t)N * K >= 1 << 23;
    const bool little = K <= 4096 && (double)M * N * K <= 3e8;
    if (f32 && (large || little) && (uintptr_t)x % 16 == 0 && (uintptr_t)W % 16 == 0 && (M <= 1 || ld_x % 4 == 0) &&
        (N <= 1 || ld_w % 4 == 0)) {
        p.src = RAW;
        return p;
    }
    p.lay_x = !x16;
    p.lay_w = !w16;
    p.cols = up(K, f32 ? 64 : 8);
    p.ld = p.cols * planes_of(p.src);
    if (p.lay_w) {  // as many features as stay in L2 between the two kernels, but enough to fill the SMs
        const int64_t most = std::max<int64_t>(2048, (64 << 20) / (p.ld * 2) / BF * BF), parts = (N + most - 1) / most;
        p.chunk = (int)std::min<int64_t>(N, up((N + parts - 1) / parts, BF));
    }
    p.x_bytes = p.lay_x ? up((int64_t)M * p.ld * 2, 256) : 0;
    p.w_bytes = p.lay_w ? up((int64_t)p.chunk * p.ld * 2, 256) : 0;
    return p;
}

cudaError_t lay_out(Layout &L, int dtype, const Plan &p, int K, cudaStream_t s) {
    L.K = K;
    L.cols = (int)p.cols;
    L.ld_dst = p.ld;
    const int of = dtype == DSA_F32 ? 256 : 1024;  // values of a row that a warp takes
    const int64_t n = (((int64_t)L.rows[0] + L.rows[1]) * ((p.cols + of - 1) / of) + 7) / 8;
    if (n == 0) return cudaSuccess;
    if (n > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const cudaError_t e = dtype == DSA_F32 ? launch_pdl(linear_layout_kernel<true>, dim3((unsigned)n), dim3(256), 0, s, L)
                                           : launch_pdl(linear_layout_kernel<false>, dim3((unsigned)n), dim3(256), 0, s, L);
    if (e == cudaSuccess) note_launch(DSA_KERNEL_LINEAR_LAYOUT);
    return e;
}

// How the product is cut: tokens of a tile, CTAs that share a tile's K, CTAs that an SM holds.  The one of least time by
// what bounds a slab (64 columns of K), in SM cycles, each measured:
//   * shared memory: the slab is written once and read by the MMAs (W once, x once), 128 bytes a cycle (256 tokens: 730
//     cycles, of which the MMAs need 512); of planes W three times and x's six, 1488 cycles for 80 tokens;
//   * 350 cycles to hand a slab on and for 16 KB of W from HBM to one SM;
//   * HBM, 3550 bytes a cycle for all, which W passes once;
// and what a CTA needs besides: 5000 cycles until its first slab is there and its last result stored, more for the
// cluster to meet and add.  64 tokens, 16384 to 7168, take 44 us with two CTAs a tile and 51 with one; 300 tokens, 7168 to
// 2112, 16 us with four and 31 with one; 777 tokens, 2048 to 5001, 20 us in tiles of 112 and 31 in tiles of 208
// (280 tiles and 160 for 152 SMs); 512 tokens, 16384 to 7168, 99 us in 112 tiles of 256 and 119 with two CTAs a tile.
struct Cut {
    int bt, share, per_sm;
};
using Kernel = void (*)(CUtensorMap, CUtensorMap, LinearParams);
template <int SRC>
Kernel kernel_for(bool split, bool exact) {
    return split ? exact ? linear_kernel<true, true, SRC> : linear_kernel<true, false, SRC>
                 : exact ? linear_kernel<false, true, SRC> : linear_kernel<false, false, SRC>;
}
Kernel kernel_for(int src, bool split, bool exact) {
    return src == RAW ? kernel_for<RAW>(split, exact) : src == PLANES ? kernel_for<PLANES>(split, exact) : kernel_for<ROWS>(split, exact);
}

// Clusters of `share` CTAs that the device holds at once (they lie within one group of SMs each).
int clusters_at_once(int share, int per_sm, bool exact) {
    static std::atomic<int> known[2][3][MAX_SHARE + 1];  // per kind: the same answer whoever asks first
    std::atomic<int> &k = known[exact][per_sm][share];
    int n = k.load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(share);
        cfg.blockDim = dim3(NUM_THREADS);
        cfg.dynamicSmemBytes = SMEM_MAX / per_sm - 2048;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {(unsigned)share, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const Kernel kernel = kernel_for<ROWS>(true, exact);
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX - 1024) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
            (void)cudaGetLastError();
            n = std::max(1, device_sm_count() * per_sm / (2 * share));
        }
        k.store(n, std::memory_order_relaxed);
    }
    return n;
}

Cut cut(int M, int N, int total, bool exact, int src, int sms) {
    const int most = max_bt(exact, src), least_tt = (M + most - 1) / most;
    const int64_t ft = ((int64_t)N + BF - 1) / BF;
    Cut best{MAX_BT, 1, 1};
    double least = 1e30;
    for (int tt = least_tt; tt < least_tt + 8; ++tt) {
        const int bt = (int)up(((int64_t)M + tt - 1) / tt, 16);
        const int64_t tiles = (M + bt - 1) / bt * ft;
        const double smem = src == ROWS ? 2 * (W_SLAB + 128.0 * bt) / 128 : src == PLANES ? 768 + 9.0 * bt : 1600 + 16.0 * bt;
        const double hbm = (double)ft * total * W_SLAB * (src == ROWS ? 1 : src == PLANES ? 3 : 2) / 3550;
        for (int share = 1; share <= MAX_SHARE && (share == 1 || total >= (src == PLANES ? 2 : 4) * share); ++share)
            for (int per_sm = 1; per_sm <= (share > 1 && !exact && src == ROWS && bt <= 128 ? 2 : 1); ++per_sm) {
                const int64_t room = share == 1 ? sms : clusters_at_once(share, per_sm, exact), rounds = (tiles + room - 1) / room;
                const double slabs = (total + share - 1) / share, side = tiles * share > sms ? per_sm : 1;
                const double work = slabs * std::max(smem * side, 350.0);
                const double fix = share == 1 ? 5000 + 14.0 * bt : 8000 + 60.0 * bt;
                // one CTA a tile: the end of a tile is beside the next one's product (RAW: behind its own)
                const double tile = src == RAW ? work + 14.0 * bt : std::max(work, 14.0 * bt);
                const double t = std::max(hbm + fix, share == 1 ? rounds * tile + fix : rounds * (work + fix));
                if (t < least * 0.98) {
                    least = t;
                    best = {bt, share, per_sm};
                }
            }
        if (bt == 16) break;
    }
    return best;
}

cudaError_t launch_tiles(const void *x, int64_t ld_x, const void *W, int64_t ld_w, int K, int64_t cols, int src, LinearParams &P,
                         cudaStream_t s) {
    const int sms = device_sm_count(), planes = planes_of(src);
    P.total = (K + 63) / 64;
    const bool exact = P.e.f32 && P.total > chain_of(planes);
    P.chain = exact ? chain_of(planes) : P.total;
    P.K = K;
    P.x = x;
    P.w = W;
    P.ld_x = ld_x;
    P.ld_w = ld_w;
    const Cut c = cut(P.M, P.N, P.total, exact, src, sms);
    P.bt = c.bt;
    P.share = c.share;
    P.tt = (P.M + P.bt - 1) / P.bt;
    const int64_t tiles = (int64_t)P.tt * (((int64_t)P.N + BF - 1) / BF);
    if (tiles > 0x7fffffff / 8) return cudaErrorInvalidConfiguration;
    P.tiles = (int)tiles;
    P.stage_bytes = planes * (W_SLAB + P.bt * 128);
    P.wait_limit = wait_limit_cycles();
    const bool split = P.share > 1;
    P.acc_cols = 32;
    while (P.acc_cols < (planes - 1) * P.bt + up(P.bt, 32)) P.acc_cols *= 2;
    if (!split) P.acc_cols = MAX_BT;
    P.tmem_cols = split && !exact ? P.acc_cols : 2 * P.acc_cols;
    const int turn = split ? 0 : TURN, room = SMEM_MAX / c.per_sm - 2048 - turn;
    if (src == RAW) {  // two slabs for the MMAs, up to three on their way, then more for the MMAs
        P.raw_bytes = (BF + P.bt) * RAW_ROW;
        P.deep = std::min(3, (room - 2 * P.stage_bytes) / P.raw_bytes);
    }
    P.stages = std::min(MAX_STAGES, (room - P.deep * P.raw_bytes) / P.stage_bytes);
    const int smem = 1024 + P.stages * P.stage_bytes + turn + P.deep * P.raw_bytes;
    CUtensorMap tw{}, tx{};
    if (src != RAW) {
        const int rank = src == ROWS ? 2 : 3;
        const uint64_t wide = src == ROWS ? K : cols;
        const uint64_t dims_w[3] = {wide, (uint64_t)P.N, 3}, strides_w[2] = {(uint64_t)ld_w * 2, (uint64_t)cols * 2};
        const uint64_t dims_x[3] = {wide, (uint64_t)P.M, 3}, strides_x[2] = {(uint64_t)ld_x * 2, (uint64_t)cols * 2};
        const uint32_t box_w[3] = {64, BF, 3}, box_x[3] = {64, (uint32_t)P.bt, 3};
        if (!make_tmap(&tw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, W, dims_w, strides_w, box_w) ||
            !make_tmap(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, x, dims_x, strides_x, box_x))
            return cudaErrorInvalidValue;
    }
    const Kernel kernel = kernel_for(src, split, exact);
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
        const bool four_in = K % 4 == 0 && (uintptr_t)x % 16 == 0 && (uintptr_t)W % 16 == 0 && (M <= 1 || ld_x % 4 == 0) &&
                             (N <= 1 || ld_w % 4 == 0);
        e = dtype != DSA_F32 ? launch_few<__nv_bfloat16, 1>(x, ld_x, W, ld_w, M, N, K, E, s)
            : four_in        ? launch_few<float, 4>(x, ld_x, W, ld_w, M, N, K, E, s)
                             : launch_few<float, 1>(x, ld_x, W, ld_w, M, N, K, E, s);
        if (e != cudaSuccess) return fail_cuda(e);
        note_launch(DSA_KERNEL_LINEAR_SIMT);
        return DSA_OK;
    }
    const int64_t rows_x = M > 1 ? ld_x : up(K, 8), rows_w = N > 1 ? ld_w : up(K, 8);
    const void *xs = p.lay_x ? workspace : x;
    for (int64_t n0 = 0; n0 < N; n0 += p.chunk) {  // (the sum behind the last part may pass 32 bits)
        const int n = (int)std::min<int64_t>(p.chunk, N - n0);
        const void *ws = W;
        Layout L{};
        if (p.lay_x && n0 == 0) {
            L.src[0] = x;
            L.ld[0] = ld_x;
            L.rows[0] = M;
            L.dst[0] = (__nv_bfloat16 *)workspace;
        }
        if (p.lay_w) {
            ws = (char *)workspace + p.x_bytes;
            L.src[1] = (const char *)W + n0 * ld_w * (dtype == DSA_F32 ? 4 : 2);
            L.ld[1] = ld_w;
            L.rows[1] = n;
            L.dst[1] = (__nv_bfloat16 *)ws;
        }
        if (p.lay_x || p.lay_w) {
            e = lay_out(L, dtype, p, K, s);
            if (e != cudaSuccess) return fail_cuda(e);
        }
        LinearParams P{};
        P.e = E;
        if (bias) P.e.bias = bias + n0;
        P.e.y = (char *)y + n0 * ey;
        if (residual) P.e.res = (const char *)residual + n0 * ey;
        P.M = M;
        P.N = n;
        e = launch_tiles(xs, p.lay_x ? p.ld : rows_x, ws, p.lay_w ? p.ld : rows_w, K, p.cols, p.src, P, s);
        if (e != cudaSuccess) return fail_cuda(e);
    }
    return DSA_OK;
}
