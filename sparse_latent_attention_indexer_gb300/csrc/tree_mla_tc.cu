// Attention of a tree of drafted tokens over the latent cache on tcgen05 tensor
// cores (bf16 queries, 512 latent + 64 rotary values per token, any head count).
//
//   z[i,s]   = scale (q~[i] . c[s] + q_pe[i] . k_pe[s])   rows i = (node, head), tokens s that the node sees
//   o_lat[i] = sum_s softmax_s(z[i,s]) c[s]
// (DeepSeek-V3.2-Exp atlas page, MoE transformer block: Q = [Q^C; Q^R], K_i =
// [K^C_i; k^R], v = c^KV W_UV, with W_UK folded into q~ and W_UV applied afterwards;
// the mask is the tree's.)
//
// Work unit: 128 rows of one sequence (nodes x heads are rows of one matrix: every
// head reads the same latent) times a range of its tokens.  The context of
// 128 x 512 fp32 values would fill an SM's tensor memory, so two CTAs on two
// SMs share a unit by columns: CTA c owns latent columns 256c.. and rotary columns
// 32c.. of every row and token.  A tile is 64 tokens.
//   * Each CTA multiplies its columns: a partial score tile (q~ slice resident in
//     tensor memory as the A operand, so QK^T reads only the tokens from shared
//     memory).  Of each 32 rows CTA c finishes 16c .. 16c+15: the other CTA sends it
//     its partial scores of those rows (fp32, 16 KB, from registers), it adds its own,
//     runs the softmax and sends the probabilities (bf16, 8 KB) back, which both
//     need for PV.  Nothing is computed twice, and a row's maximum and sum live in
//     one place.  The halves cross in fp32: a rounding would be relative to the half,
//     and what all tokens of a half share cancels in the softmax only if it is exact.
//   * Twelve softmax warps in three groups that take the tiles in turn; tensor-memory
//     lanes are rows, so each of a group's four warps finishes 16 rows of its quarter
//     and sends the other 16, and all four quarters of the SM share the exponentials.
//   * Lazy rescaling: a row's reference maximum is a whole number (of powers of two) and
//     moves only when a tile exceeds it by more than 8; the factor travels with the
//     probabilities, and both CTAs rescale their half of the context.  A group works
//     with the reference that it knows and corrects by a power of two (exact) if the
//     tile before has moved it.
//   * bf16 tokens arrive by TMA (two copies a tile where 64 lie together) in two stages
//     as K and once more, from L2, in two as V, so that no operand waits for a softmax;
//     of an e4m3 cache codes, rotary keys and scales arrive so, and eight more warps
//     spread the codes (exact in bf16) into three stages that serve K and V.
//   * A token that some row does not see may hold anything, and 0 x NaN is NaN: in the V
//     of tiles with hidden tokens Inf and NaN become 0 (two warps of their own: by the
//     loader itself 25 short trees took 1.13 ms instead of 0.69).  Scores of hidden tokens
//     are replaced after the MMA.
// Roundings: q~, the probabilities and the context to bf16, as operands of the next product (as
// in the sparse attention); scores, maxima, sums and the context's accumulation in fp32.
// Bound by shared memory: a bf16 tile moves 219 KB through it (92 MMA operands, 68 tokens by
// TMA, 59 partial scores and probabilities), 1711 cycles at 128 bytes a cycle of the 2000 that
// it takes (its MMAs take 1088; trees of 32 nodes over up to 12K tokens run at 1150 TFLOP/s; with
// the halves rounded to fp16 1810 and 1270).  An e4m3 tile takes 2790, of which 226 KB through
// shared memory are 1766 (32 x 64K decode at 874 TFLOP/s); what the rest waits for has not been
// measured.  A unit's start and end take 12 us: 11 bf16 tiles, 9 e4m3 ones (76 units of 4 to 36).
//
// Waits are bounded; a timeout records its site in the device error word and
// both CTAs drain and exit.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "tc_common.cuh"

namespace dsa {

__device__ int g_tree_tc_error = 0;

namespace {

constexpr int ROWS = 128;               // rows of a unit (MMA M)
constexpr int HR = 64;                  // rows that a CTA finishes
constexpr int DC = 512, DR = 64;
constexpr int TK = 64;                  // tokens of a tile
constexpr int SLAB = TK * 128;          // 64 tokens x 64 columns, 128-byte swizzle: 8 KB
constexpr int ROPE = TK * 64;           // 64 tokens x 32 rotary columns, 64-byte swizzle: 4 KB
constexpr int STAGE = 4 * SLAB + ROPE;  // a CTA's columns of a tile
// bf16 caches: two stages of K, free after QK^T, and two of V (the latents again), loaded when PV comes near: no operand
// waits in shared memory for a softmax.
constexpr int VSTAGE = 4 * SLAB;
// e4m3 caches: three stages that serve K and V, and two of raw codes, rotary keys and scales.
constexpr int NSTAGE = 3;
constexpr int RAW_LD = 256, RAW_SCALE = TK * RAW_LD + ROPE, RAW = RAW_SCALE + TK * 16;
constexpr int KV_BYTES = std::max(2 * STAGE + 2 * VSTAGE, NSTAGE * STAGE + 2 * RAW);
constexpr int P_BYTES = ROWS * TK * 2;  // probabilities of all rows
constexpr int X_BYTES = HR * TK * 4;    // fp32 partial scores of half of the rows
constexpr int Q_BOX = ROWS * 128;       // 128 rows x 64 columns of q~ (staged in the exchange buffers)
constexpr int QR_BYTES = ROWS * 64;     // rotary slice of the queries, 64-byte swizzle
constexpr int NB = 6;                   // barriers of a kind: tile t uses number t % 6, which belongs to one group and one buffer
constexpr uint32_t COL_S = 0, COL_Q = 128, COL_O = 256;
constexpr uint32_t IDESC_QK = tc::instr_desc(tc::kFmtBF16, tc::kFmtBF16, ROWS, TK, 0, 0);
constexpr uint32_t IDESC_PV = tc::instr_desc(tc::kFmtBF16, tc::kFmtBF16, ROWS, 256, 0, 1);
constexpr float RESCALE_LOG2 = 8.0f;
constexpr float LN2 = 0.69314718055994530942f;
constexpr long long kAbortQuietCycles = 1LL << 18;
constexpr int kMaxSplits = 76;          // of a sequence
// warp 0: TMA (Q, bf16 K); 1: QK^T; 2: tensor memory, PV; 3: TMA (bf16 V); from 4 on the softmax groups of four
// (warp % 4 = lane quarter); of an e4m3 cache eight more load, of a bf16 cache two more look V tiles over
constexpr int G = 3;                    // softmax groups
constexpr int SOFT = 4 * G;
constexpr int FIRST_LOAD = 4 + SOFT;
constexpr int LOADERS = 8, SCRUBBERS = 2;

struct Bars {
    // one arrival
    uint64_t q_stage, peer_ready, qk_done, o_done, kv_empty[4], raw[2], mask_full[NB], hand[4][NB], s_full[NB];
    uint64_t x_full[NB], p_in[NB];    // the other CTA's partial scores are here; its probabilities are
    // a group's four warps
    uint64_t s_empty[NB], x_free[NB]; // they (x_free: the other CTA's) have read the scores
    uint64_t p_full[NB];              // all probabilities are here, and the context is ready for them
    // two
    uint64_t p_free[NB];              // the PV products of both CTAs are done
    // as start() says
    uint64_t kv_full[4], raw_free[2], q_ready;
    static constexpr int ONE = 10 + 8 * NB, FOUR = ONE + 3 * NB, TWO = FOUR + NB, ALL = TWO + 7;

    __device__ __forceinline__ void start(bool kv8, int lane) {
        for (int i = lane; i < ALL; i += 32)
            tc::mbar_init(&q_stage + i, i < ONE ? 1 : i < FOUR ? 4 : i < TWO ? 2 : i == ALL - 1 ? SOFT : kv8 ? LOADERS : 1);
    }
};
static_assert(sizeof(Bars) == 8 * (Bars::TWO + 7), "every barrier is set up");
struct Misc {
    float m_pub[G][HR];           // reference maximum that a group used, for the next tile's group
    float alpha_out[2][HR], alpha_in[2][HR];  // context factors of a tile, of this CTA's rows and of the other's
    float inv[ROWS];                  // 1 / row sum
    uint64_t live[NB];                // tokens of a tile whose page exists
    Bars bar;
    uint32_t tmem_slot;
    int abort_flag, never;
};
struct RowSums {                      // in the exchange buffers, at the end
    float sum[G][HR], ref[G][HR];     // a group's share of the row sum and its reference
};
constexpr int SMEM = 1024 + KV_BYTES + 2 * P_BYTES + 2 * X_BYTES + QR_BYTES + (int)sizeof(Misc);
static_assert(SMEM <= 232448, "shared memory per CTA");
static_assert(4 * Q_BOX <= 2 * P_BYTES + 2 * X_BYTES, "the q~ slice is staged in the exchange buffers");
// The epilogue stages a CTA's 256 columns, rows 16 bytes apart from a power of two, in the token stages.
constexpr int OUT_LD_F32 = 256 * 4 + 16, OUT_LD_BF16 = 256 * 2 + 16;
static_assert(ROWS * OUT_LD_F32 <= KV_BYTES, "staged context");

// A sequence's units.
struct SeqUnits {
    int unit0;       // first unit
    int q0, T;       // first query row, nodes
    int first;       // tokens before the tree
    int at;          // contiguous caches: its first cache row; paged ones: its row of the table
    int splits;      // ranges of its tokens
    int part0;       // first partial context of a split sequence
};
struct TreeParams {
    PageTab pt;
    const uint64_t *mask;
    int words, H;
    int oob;                     // a cache row past the last one
    int n_seq;
    // softmax_scale log2(e) = +-scale_log2 2^k with scale_log2 in [1/2, 1): the queries carry +-2^k (exact), so that the
    // largest product is the largest score, and products stay in fp32's range where scores do.
    float scale_log2;
    uint32_t q_factor;           // +-2^k, twice in bf16
    long long wait_limit;
    SeqUnits s[DSA_MAX_SEQS];    // in the order of the units (the longest first)
};
static_assert(sizeof(TreeParams) + 4 * 128 + 128 <= 32764, "launch parameters");

// Two bf16 values a word: bits 15 and 31 say which are Inf or NaN (an exponent of ones carries into the sign's place).
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
    return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
// Inf and NaN become 0.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
    return w;
}

// Four e4m3 codes -> four bf16 values times 2^-120 (exact: sign, exponent and mantissa move to bf16's fields, whose
// exponent bias is 120 larger; subnormal codes become bf16 subnormals).  A code's low nibble is the upper half of the
// value's low byte, its sign and the three bits behind make the high byte.
__device__ __forceinline__ void spread4(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    const uint32_t low = (codes << 4) & 0xf0f0f0f0u, high = ((codes >> 4) & 0x07070707u) | (codes & 0x80808080u);
    lo = __byte_perm(low, high, 0x5140);
    hi = __byte_perm(low, high, 0x7362);
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmul2(*(const __nv_bfloat162 *)&a, *(const __nv_bfloat162 *)&b);
    return *(const uint32_t *)&r;
}

// 16 codes x 2^120 scale -> 16 bf16 (two 16-byte chunks).
__device__ __forceinline__ void dequant16(const uint4 &c, uint32_t up, uint4 (&o)[2]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        spread4(w[i], r[2 * i], r[2 * i + 1]);
        r[2 * i] = mul2(r[2 * i], up);
        r[2 * i + 1] = mul2(r[2 * i + 1], up);
    }
    o[0] = make_uint4(r[0], r[1], r[2], r[3]);
    o[1] = make_uint4(r[4], r[5], r[6], r[7]);
}
__device__ __forceinline__ uint32_t bf16_pair(float x) {
    const __nv_bfloat162 v = __float2bfloat162_rn(x);
    return *(const uint32_t *)&v;
}
// 2^d of a whole number d (0 below the normal range).
__device__ __forceinline__ float pow2(float d) {
    const int e = (int)fmaxf(d, -127.0f) + 127;
    return e > 0 ? __int_as_float(min(e, 254) << 23) : 0.0f;
}

// COUNT threads arrive at barrier ID; returns the AND of `v` over them.
template <int ID, int COUNT>
__device__ __forceinline__ bool bar_and(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, %2, %3, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "n"(ID), "n"(COUNT)
        : "memory");
    return r != 0;
}

// O[rows of this warp] *= alpha (tcgen05.ld/st are warp-wide: rows that stay take a factor of 1).
__device__ __forceinline__ void rescale_rows(uint32_t lanes, float alpha) {
    tc::tc_fence_after();
#pragma unroll 1
    for (int cc = 0; cc < 8; ++cc) {
        float o[32];
        uint32_t ob[32];
        tc::tmem_ld32(lanes + COL_O + cc * 32, o);
        tc::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) ob[j] = __float_as_uint(o[j] * alpha);
        tc::tmem_st32(lanes + COL_O + cc * 32, ob);
    }
    tc::tmem_st_wait();
    tc::tc_fence_before();
}

// 16 lanes x 64 fp32 columns: thread i gets of rows i / 4 (v[4j], v[4j + 1]) and i / 4 + 8 (v[4j + 2], v[4j + 3]) the
// columns 8j + 2 (i % 4) and the next.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// Four 8 x 8 tiles of 16-bit values in that layout -> shared memory rows (lane i: row i % 8 of tile i / 8).
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

template <bool KV8>
struct Cfg {
    static constexpr int THREADS = 32 * (FIRST_LOAD + (KV8 ? LOADERS : SCRUBBERS));
};

template <bool KV8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<KV8>::THREADS, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                   const __grid_constant__ CUtensorMap tm_pe, const __grid_constant__ CUtensorMap tm_sc, int run,
                   const __nv_bfloat16 *__restrict__ qpe, const __grid_constant__ TreeParams P,
                   __nv_bfloat16 *__restrict__ olat, float *__restrict__ lse, float *__restrict__ opart,
                   float *__restrict__ lpart) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *KV = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *Pb = KV + KV_BYTES;   // [t % 2] probabilities: rows x 64 tokens, 128-byte swizzle
    uint8_t *X = Pb + 2 * P_BYTES;       // [t % 2] the other CTA's partial scores of this CTA's rows
    uint8_t *QR = X + 2 * X_BYTES;       // rotary slice of the queries
    Misc *ms = (Misc *)(QR + QR_BYTES);
    Bars *bar = &ms->bar;
    volatile int *abort_flag = (volatile int *)&ms->abort_flag, *nv = (volatile int *)&ms->never;
    int *err = &g_tree_tc_error;

    const unsigned FULL = 0xffffffffu;
    const int warp = __shfl_sync(FULL, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank(), peer = rank ^ 1u;

    if (warp == 0) {
        bar->start(KV8, lane);
        if (lane == 0) {
            *abort_flag = 0;
            ms->never = 0;
        }
        tc::fence_mbar_init();
        __syncwarp();
    }
    if (warp == 2) {
        tc::tmem_alloc(&ms->tmem_slot, 512);
        tc::tmem_relinquish();
    }

    // ---- the unit: rows row0 .. of a sequence, tiles t0 .. t0 + n - 1 of its tokens ----
    const int u = (int)(blockIdx.x >> 1);
    int lo = 0, hi = P.n_seq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P.s[mid].unit0 <= u) lo = mid; else hi = mid - 1;
    }
    const SeqUnits &me = P.s[lo];
    const int T = me.T, first = me.first, at = me.at;
    const int nt = (int)(((int64_t)T * P.H + ROWS - 1) / ROWS);
    const int splits = me.splits;
    const int rem = u - me.unit0, split = rem / nt, rt = nt - 1 - (rem - split * nt);
    const int seq_rows = T * P.H;                                  // rows of the sequence
    const int64_t seq_row0 = (int64_t)me.q0 * P.H;
    const int lrow = rt * ROWS;                                    // first row of the unit within the sequence
    const int node_lo = lrow / P.H, node_hi = min(T - 1, (lrow + ROWS - 1) / P.H);
    const int tokens = first + (P.mask ? T : node_hi + 1);         // tokens that some row may see
    const int safe = first + (P.mask ? 0 : node_lo + 1);           // tokens before this one are seen by every row
    const int tiles = (first + T + TK - 1) / TK;
    const int per = (tiles + splits - 1) / splits;
    const int t0 = split * per;
    const int n = max(0, min((tokens + TK - 1) / TK, t0 + per) - t0);

    pdl_wait();  // the set-up so far overlapped the previous kernel; global memory only from here
    if (threadIdx.x == 0 && n > 0) {  // the q~ slice, on its way before the CTAs have met (staged in the exchange buffers)
        tc::mbar_arrive_expect_tx(&bar->q_stage, 4 * Q_BOX);
        for (int j = 0; j < 4; ++j)
            tc::tma_load_2d(Pb + j * Q_BOX, &tm_q, &bar->q_stage, rank * 256 + j * 64, (int)(seq_row0 + lrow));
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    // The CTAs meet: a warp that reaches into the other one first waits until that one's barriers exist; the others pass
    // here again when their work is done.
    const bool reaches = warp >= 4 && warp < FIRST_LOAD;
    tc::cluster_arrive_relaxed();
    const uint32_t tmem = __shfl_sync(FULL, ms->tmem_slot, 0);

    // Cache row of token s, or -1 (behind the last token, or on no page).
    const auto row_of = [&](int s) -> int64_t { return s < tokens ? cache_row(P.pt, at, at, s) : -1; };
    // Rows of a tile's four runs of 16 tokens, a run a lane: its cache row, -1 behind the last token, or the row past
    // the cache (read as zeros) where there is no page.
    const auto runs_of = [&](int t) {
        const int s = (t0 + t) * TK + (lane & 3) * 16;
        const int64_t r = row_of(s);
        return t >= n || s >= tokens ? -1 : r >= 0 ? (int)r : P.oob;
    };
    // Publishes which of tile t's tokens have a page (one warp).
    const auto put_mask = [&](int t, int rows) {
        if (!P.pt.table) return;
        const unsigned have = __ballot_sync(FULL, rows >= 0 && rows != P.oob);
        if (lane == 0) {
            uint64_t m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (have >> i & 1) m |= 0xffffull << 16 * i;
            ms->live[t % NB] = m;
            tc::mbar_arrive(&bar->mask_full[t % NB]);
        }
    };

    if (warp == 0 && n > 0) {
        // ---------------- TMA: K of a bf16 cache, or raw codes ----------------
        // Lane's copy: latents of run k (bf16: all four slabs at once where 64 tokens lie together), or rotary columns.
        const int runs = TK / run, per_run = KV8 || runs == 1 ? 1 : 4, nlat = per_run * runs;
        const bool lat = lane < nlat;
        const int k = lat ? lane / per_run : lane - nlat, j = lat ? lane % per_run : 0;
        int rows = runs_of(0);
        for (int t = 0; t < n; ++t) {
            const int st = t & 1;
            if (!__all_sync(FULL, tc::mbar_wait(KV8 ? &bar->raw_free[st] : &bar->kv_empty[st], ((t >> 1) & 1) ^ 1, abort_flag,
                                                err, 101, P.wait_limit)))
                break;
            put_mask(t, rows);
            uint64_t *full = KV8 ? &bar->raw[st] : &bar->kv_full[st];
            // of runs behind the last token nothing is read
            const int row = __shfl_sync(FULL, rows, (k * (run / 16)) & 3);
            const bool go = (lat || k < runs) && row >= 0;
            const int n_lat = __popc(__ballot_sync(FULL, go && lat)), n_pe = __popc(__ballot_sync(FULL, go && !lat));
            if (lane == 0)
                tc::mbar_arrive_expect_tx(full, (uint32_t)(run * (n_lat * (KV8 ? RAW_LD + 16 : 512 / per_run) + n_pe * 64)));
            __syncwarp();
            uint8_t *dst = KV8 ? KV + NSTAGE * STAGE + st * RAW : KV + st * STAGE;
            if (go && lat) {
                if (KV8) {
                    tc::tma_load_2d(dst + k * run * RAW_LD, &tm_kv, full, rank * 256, row);
                    tc::tma_load_2d(dst + RAW_SCALE + k * run * 16, &tm_sc, full, 0, row);
                } else tc::tma_load_3d(dst + j * SLAB + k * run * 128, &tm_kv, full, 0, row, rank * 4 + j);
            } else if (go) {
                tc::tma_load_2d(dst + (KV8 ? TK * RAW_LD : 4 * SLAB) + k * run * 64, &tm_pe, full, rank * 32, row);
            }
            rows = runs_of(t + 1);
        }
    } else if (warp == 1 && n > 0) {
        // ---------------- QK^T issuer: tile t into score buffer t % 2 once its tokens are here ----------------
        // (PV comes from another warp: an issue blocks while the tensor pipe is busy.)
        const uint32_t issue = tc::elect_one();
        const uint32_t kv0 = __shfl_sync(FULL, tc::smem_u32(KV), 0), qr0 = __shfl_sync(FULL, tc::smem_u32(QR), 0);
        const uint64_t kd = tc::smem_desc(kv0, 16, 1024);
        const uint64_t rd = tc::smem_desc(kv0 + 4 * SLAB, 16, 512, tc::kSwizzle64B);
        const uint64_t qd = tc::smem_desc(qr0, 16, 512, tc::kSwizzle64B);
        bool ok = __all_sync(FULL, tc::mbar_wait(&bar->q_ready, 0, abort_flag, err, 102, P.wait_limit));
        for (int t = 0; ok && t < n; ++t) {
            const int st = KV8 ? t % NSTAGE : t & 1;
            if (t >= 2) ok = tc::mbar_wait(&bar->s_empty[(t - 2) % NB], ((t - 2) / NB) & 1, abort_flag, err, 103, P.wait_limit);
            ok = tc::mbar_wait(&bar->kv_full[st], (KV8 ? t / NSTAGE : t >> 1) & 1, abort_flag, err, 104, P.wait_limit) && ok;
            if (!(ok = __all_sync(FULL, ok))) break;
            tc::tc_fence_after();
            const uint32_t d = tmem + COL_S + (t & 1) * TK;
            const uint64_t off = (uint64_t)(uint32_t)(st * (STAGE / 16));
#pragma unroll
            for (int i = 0; i < 16; ++i)
                tc::mma_f16_ts_if(issue, d, tmem + COL_Q + i * 8, kd + off + ((i >> 2) * SLAB + (i & 3) * 32) / 16, IDESC_QK,
                                  i != 0);
#pragma unroll
            for (int i = 0; i < 2; ++i) tc::mma_f16_if(issue, d, qd + i * 2, rd + off + i * 2, IDESC_QK, 1);
            if (issue) {
                tc::mma_commit(&bar->s_full[t % NB]);
                if (!KV8) tc::mma_commit(&bar->kv_empty[st]);
            }
            __syncwarp();
        }
        // No MMA of this warp may still be running when the tensor memory is released.
        if (issue) tc::mma_commit(&bar->qk_done);
        tc::mbar_wait(&bar->qk_done, 0, nv, err, 105);
    } else if (warp == 2 && n > 0) {
        // ---------------- PV issuer: frees the stage and the probabilities (which both CTAs hold) ----------------
        const uint32_t issue = tc::elect_one();
        const uint32_t kv0 = __shfl_sync(FULL, tc::smem_u32(KV), 0), p0 = __shfl_sync(FULL, tc::smem_u32(Pb), 0);
        const uint64_t pd = tc::smem_desc(p0, 16, 1024), vd = tc::smem_desc(kv0 + (KV8 ? 0 : 2 * STAGE), SLAB, 1024);
        for (int t = 0; t < n; ++t) {
            bool ok = KV8 || tc::mbar_wait(&bar->kv_full[2 + (t & 1)], (t >> 1) & 1, abort_flag, err, 109, P.wait_limit);
            ok = tc::mbar_wait(&bar->p_full[t % NB], (t / NB) & 1, abort_flag, err, 106, P.wait_limit) && ok;
            if (!__all_sync(FULL, ok)) break;
            tc::tc_fence_after();
            const int st = KV8 ? t % NSTAGE : t & 1;
            const uint64_t a0 = pd + (uint64_t)(uint32_t)((t & 1) * (P_BYTES / 16));
            const uint64_t b0 = vd + (uint64_t)(uint32_t)(st * ((KV8 ? STAGE : VSTAGE) / 16));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                tc::mma_f16_if(issue, tmem + COL_O, a0 + kk * 2, b0 + kk * (16 * 128 / 16), IDESC_PV, (t | kk) != 0);
            if (issue) {
                tc::mma_commit(&bar->kv_empty[KV8 ? st : 2 + st]);
                tc::mma_commit_multicast(&bar->p_free[t % NB], 3);
            }
            __syncwarp();
        }
        if (issue) tc::mma_commit(&bar->o_done);
        tc::mbar_wait(&bar->o_done, 0, nv, err, 107);
        tc::mbar_wait(&bar->q_stage, 0, nv, err, 108);  // after an abort nobody else may have waited for it
    } else if (!KV8 && warp == 3 && n > 0) {
        // ---------------- TMA: V of a bf16 cache ----------------
        const int runs = TK / run, copies = runs == 1 ? 1 : 4 * runs;
        const int k = runs == 1 ? 0 : lane >> 2, j = runs == 1 ? 0 : lane & 3;
        int rows = runs_of(0);
        for (int t = 0; t < n; ++t) {
            const int st = t & 1;
            if (!__all_sync(FULL, tc::mbar_wait(&bar->kv_empty[2 + st], ((t >> 1) & 1) ^ 1, abort_flag, err, 110, P.wait_limit))) break;
            const int row = __shfl_sync(FULL, rows, (k * (run / 16)) & 3);
            const bool go = lane < copies && row >= 0;
            const int some = __popc(__ballot_sync(FULL, go));
            uint64_t *full = (t0 + t + 1) * TK > safe ? &bar->raw[st] : &bar->kv_full[2 + st];
            if (lane == 0) tc::mbar_arrive_expect_tx(full, (uint32_t)(run * some * (runs == 1 ? 512 : 128)));
            __syncwarp();
            if (go)
                tc::tma_load_3d(KV + 2 * STAGE + st * VSTAGE + j * SLAB + k * run * 128, &tm_kv, full, 0, row, rank * 4 + j);
            rows = runs_of(t + 1);
        }
    } else if (!KV8 && warp >= FIRST_LOAD && n > 0) {
        // ---------------- V tiles with hidden tokens, which are the last ones: Inf and NaN become 0 ----------------
        const int behind = max(0, safe / TK - t0);  // tiles before them
        for (int t = behind; t < n; ++t) {
            const int st = t & 1;
            const bool ok = tc::mbar_wait(&bar->raw[st], ((t - behind) >> 1) & 1, abort_flag, err, 125, P.wait_limit);
            if (!bar_and<3, 32 * SCRUBBERS>(ok)) break;
            // 16 tokens a step, half of the slabs a warp, from the first hidden token's on
            uint8_t *half = KV + 2 * STAGE + st * VSTAGE + (warp - FIRST_LOAD) * 2 * SLAB;
#pragma unroll 1
            for (int at = (max(0, safe - (t0 + t) * TK) & ~15) * 128 + lane * 16; at < SLAB; at += 2048) {
                uint4 v[8];
                uint32_t bad = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = *(const uint4 *)(half + (i >> 2) * SLAB + at + (i & 3) * 512);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    bad |= not_finite2(v[i].x) | not_finite2(v[i].y) | not_finite2(v[i].z) | not_finite2(v[i].w);
                if (bad)
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        uint4 *p = (uint4 *)(half + (i >> 2) * SLAB + at + (i & 3) * 512);
                        *p = make_uint4(finite2(p->x), finite2(p->y), finite2(p->z), finite2(p->w));
                    }
            }
            tc::fence_proxy_async_smem();  // read by the MMAs (async proxy)
            bar_and<3, 32 * SCRUBBERS>(true);
            if (warp == FIRST_LOAD && lane == 0) tc::mbar_arrive(&bar->kv_full[2 + st]);
        }
    } else if (KV8 && warp >= FIRST_LOAD && n > 0) {
        // ---------------- loading warps (e4m3) ----------------
        // Warp w: eight tokens of the tile.  A pass takes four tokens' 128 codes of one block: 16 codes a lane, eight lanes a
        // token's 128, which are one row of 128 bytes where they landed and two slabs' 64 columns where they go; the lanes of
        // the second slab store their second half first, so that eight lanes hit the eight chunks of the swizzled rows.  (Eight
        // unrolled passes with the codes in registers, loaded a tile ahead, were slower: that loop and the softmax evict one
        // another from the instruction cache.)
        const int w = warp - FIRST_LOAD, slab = lane >> 2 & 1, chunk = (lane & 3) * 2, sub = lane >> 3;
        for (int t = 0; t < n; ++t) {
            const int st = t % NSTAGE;
            if (!__all_sync(FULL, tc::mbar_wait(&bar->raw[t & 1], (t >> 1) & 1, abort_flag, err, 109, P.wait_limit))) break;
            // Everything into registers, so that the raw codes' place is free and no load is left when the stage is.
            const uint8_t *raw = KV + NSTAGE * STAGE + (t & 1) * RAW;
            const uint8_t *from = raw + (w * 8 + sub) * RAW_LD + slab * 64 + (lane & 3) * 16;
            const int at = w * 512 + lane * 16;
            uint4 c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = *(const uint4 *)(from + (i >> 1) * 4 * RAW_LD + (i & 1) * 128);
            const uint4 rot = *(const uint4 *)(raw + TK * RAW_LD + at);
            // scale of token lane / 2 % 8, block lane % 2
            const float sc = *(const float *)(raw + RAW_SCALE + (w * 8 + (lane >> 1 & 7)) * 16 + (rank * 2 + (lane & 1)) * 4);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar->raw_free[t & 1]);
            if (!__all_sync(FULL, tc::mbar_wait(&bar->kv_empty[st], ((t / NSTAGE) & 1) ^ 1, abort_flag, err, 110, P.wait_limit))) break;
            uint8_t *stage = KV + st * STAGE;
            // 2^120 scale is one factor while it stays in bf16's range; scales above 128 go in two.  A hidden token's scale
            // may be anything (the codes themselves become finite numbers, whatever they are): where there may be such
            // tokens, products that are not finite become 0.
            const bool hidden = (t0 + t + 1) * TK > safe;
            uint8_t *to = stage + slab * SLAB + (w * 8 + sub) * 128;
            const auto pass = [&](int i, const uint4 &c, float up, auto more) {
                const int tok = (i >> 1) * 4 + sub, x = tok & 7;
                uint4 o[2];
                dequant16(slab ? make_uint4(c.z, c.w, c.x, c.y) : c, bf16_pair(__shfl_sync(FULL, up, tok * 2 + (i & 1))), o);
                if constexpr (decltype(more)::value) {
                    const uint32_t f = bf16_pair(__shfl_sync(FULL, sc, tok * 2 + (i & 1)));
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        o[e] = make_uint4(mul2(o[e].x, f), mul2(o[e].y, f), mul2(o[e].z, f), mul2(o[e].w, f));
                    if (hidden)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            o[e] = make_uint4(finite2(o[e].x), finite2(o[e].y), finite2(o[e].z), finite2(o[e].w));
                }
                uint8_t *dst = to + (i & 1) * 2 * SLAB + (i >> 1) * 512;
                *(uint4 *)(dst + (((chunk + slab) ^ x) << 4)) = o[0];
                *(uint4 *)(dst + (((chunk + 1 - slab) ^ x) << 4)) = o[1];
            };
            if (__all_sync(FULL, fabsf(sc) <= 128.0f)) {  // (a scale that nobody sees may be negative, or NaN)
#pragma unroll
                for (int i = 0; i < 4; ++i) pass(i, c[i], 0x1p120f * sc, std::false_type());
            } else {
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    pass(i, c[0], 0x1p120f, std::true_type());
                    c[0] = c[1];
                    c[1] = c[2];
                    c[2] = c[3];
                }
            }
            // the rotary columns as they are (both sides in the same 64-byte swizzle)
            *(uint4 *)(stage + 4 * SLAB + at) = rot;
            tc::fence_proxy_async_smem();  // read by the MMAs (async proxy)
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar->kv_full[st]);
        }
    } else if (warp >= 4 && warp < FIRST_LOAD) {
        // ---------------- softmax groups: group g takes tiles g, g + G, .. ----------------
        // Of its lane quarter's 32 rows a warp finishes 16 and sends the partial scores of the other 16.
        const int q = warp & 3, g = (warp >> 2) - 1;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        const uint32_t own_lanes = lanes + (rank * 16u << 16), other_lanes = lanes + (peer * 16u << 16);
        const float sl2 = P.scale_log2;
        bool ok = true;
        if (n > 0) {
            // The q~ slice moves to tensor memory (A operand of QK^T): four slabs of 32 packed columns, two each of the first
            // groups; the last one puts the rotary slice of the queries into shared memory.
            const int h = q * 32 + lane;
            const uint32_t f = P.q_factor;
            uint4 rq[4];
            if (g == G - 1) {
                const int64_t row = seq_row0 + lrow + h;
                const bool there = lrow + h < seq_rows;
                const uint4 *src = (const uint4 *)(qpe + row * DR + rank * 32);
#pragma unroll
                for (int e = 0; e < 4; ++e) rq[e] = there ? __ldg(src + e) : make_uint4(0, 0, 0, 0);
            }
            ok = __all_sync(FULL, tc::mbar_wait(&bar->q_stage, 0, abort_flag, err, 111, P.wait_limit));
#pragma unroll 1
            for (int js = g * 2; ok && g < 2 && js < g * 2 + 2; ++js) {
                const uint8_t *srow = Pb + js * Q_BOX + h * 128;
                uint32_t qv[32];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint4 t4 = *(const uint4 *)(srow + ((e ^ (h & 7)) << 4));
                    qv[4 * e] = mul2(t4.x, f);
                    qv[4 * e + 1] = mul2(t4.y, f);
                    qv[4 * e + 2] = mul2(t4.z, f);
                    qv[4 * e + 3] = mul2(t4.w, f);
                }
                tc::tmem_st32(lanes + COL_Q + js * 32, qv);
            }
            tc::tmem_st_wait();
            if (g == G - 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *(uint4 *)(QR + h * 64 + ((e ^ ((h >> 1) & 3)) << 4)) =
                        make_uint4(mul2(rq[e].x, f), mul2(rq[e].y, f), mul2(rq[e].z, f), mul2(rq[e].w, f));
                tc::fence_proxy_async_smem();  // read by the rotary MMAs (async proxy)
            }
            tc::tc_fence_before();
            // Every warp has read its part of the staging: the buffers may carry scores, here and from the other CTA.
            ok = bar_and<1, 32 * SOFT>(ok);
            if (lane == 0) tc::mbar_arrive(&bar->q_ready);
            tc::cluster_wait();
            if (threadIdx.x == 4 * 32) tc::mbar_arrive_remote(tc::map_peer(tc::smem_u32(&bar->peer_ready), peer));
            ok = ok && __all_sync(FULL, tc::mbar_wait(&bar->peer_ready, 0, abort_flag, err, 112, P.wait_limit));
        } else {
            tc::cluster_wait();
        }
        // A lane's waits only note a failure; the warp stops together at the end of the tile.
        const auto wait = [&](uint64_t *bars, int t, int site) {
            ok = tc::mbar_wait(&bars[t % NB], (t / NB) & 1, abort_flag, err, site, P.wait_limit) && ok;
        };
        // This thread's two rows (eight apart) and columns 8j + 2 (lane % 4) and the next of each eight.
        const int ra = q * 16 + (lane >> 2), c0 = 2 * (lane & 3);   // ra: among the CTA's 64 rows
        const int la = lrow + q * 32 + (int)rank * 16 + (lane >> 2);  // row within the sequence; may be past its end
        float ref_a = -INFINITY, ref_b = -INFINITY;                 // this group's references
        float sum_a = 0.0f, sum_b = 0.0f;                           // its share of the row sums, of this thread's columns
        // Which of tile t's 64 tokens row li sees, from this thread's first column on.
        const auto sees = [&](int t, int li) {
            const int rel = (t0 + t) * TK - first;  // node number of the tile's first token (negative: before the tree)
            const int node = li < seq_rows ? li / P.H : 0;
            uint64_t see = ~0ull;
            if (!P.mask) {
                const int left = node + 1 - rel;
                see = left >= 64 ? ~0ull : left <= 0 ? 0ull : (1ull << left) - 1;
            } else if (rel + 64 > 0) {
                const uint64_t *bits = P.mask + (int64_t)(me.q0 + node) * P.words;
                const int w = rel >> 6, sh = rel & 63;
                const uint64_t w0 = w < 0 ? ~0ull : w < P.words ? __ldg(bits + w) : 0ull;
                const uint64_t w1 = w + 1 < P.words ? __ldg(bits + w + 1) : 0ull;
                see = sh ? (w0 >> sh) | (w1 << (64 - sh)) : w0;
                const int left = T - rel;
                if (left < 64) see &= left <= 0 ? 0ull : (1ull << left) - 1;
            }
            return see;
        };
        const uint32_t p_row = (uint32_t)(q * 32 + rank * 16 + (lane & 15));  // the row this lane addresses in stmatrix
#pragma unroll 1
        for (int t = g; ok && t < n; t += G) {
            const int buf = t & 1;
            uint8_t *Xw = X + buf * X_BYTES + q * 4096 + lane * 16, *Pt = Pb + buf * P_BYTES;
            if (lane == 0 && q == 0) {
                tc::mbar_arrive_expect_tx(&bar->x_full[t % NB], X_BYTES);
                tc::mbar_arrive_expect_tx(&bar->p_in[t % NB], P_BYTES / 2 + HR * 4);
            }
            uint64_t see_a = ~0ull, see_b = ~0ull;
            if ((t0 + t + 1) * TK > safe) {
                see_a = sees(t, la);
                see_b = sees(t, la + 8);
            }
            if (P.pt.table) {
                wait(bar->mask_full, t, 113);
                const uint64_t m = ms->live[t % NB];
                see_a &= m;
                see_b &= m;
            }
            // --- the other CTA's rows: partial scores in this layout (the receiving thread has the same); the buffer there
            // is free once the other CTA has read tile t-2 ---
            if (t >= 2) wait(bar->x_free, t - 2, 114);
            wait(bar->s_full, t, 115);
            __syncwarp();
            tc::tc_fence_after();
            float v[32];
            {
                tmem_ld_16x64(other_lanes + COL_S + buf * TK, v);
                tc::tmem_ld_wait();
                const uint32_t to = tc::map_peer(tc::smem_u32(Xw), peer);
                const uint32_t there = tc::map_peer(tc::smem_u32(&bar->x_full[t % NB]), peer);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    tc::st_async16(to + i * 512, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], there);
            }
            // --- this CTA's rows: its own half and the other one's ---
            tmem_ld_16x64(own_lanes + COL_S + buf * TK, v);
            tc::tmem_ld_wait();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar->s_empty[t % NB]);
            wait(bar->x_full, t, 116);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 x = *(const float4 *)(Xw + i * 512);
                v[4 * i] += x.x;
                v[4 * i + 1] += x.y;
                v[4 * i + 2] += x.z;
                v[4 * i + 3] += x.w;
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_remote(tc::map_peer(tc::smem_u32(&bar->x_free[t % NB]), peer));
            if (!__all_sync(FULL, (see_a & see_b) == ~0ull)) {
                const uint64_t sa = see_a >> c0, sb = see_b >> c0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (!(sa >> (8 * j) & 1)) v[4 * j] = -INFINITY;
                    if (!(sa >> (8 * j + 1) & 1)) v[4 * j + 1] = -INFINITY;
                    if (!(sb >> (8 * j) & 1)) v[4 * j + 2] = -INFINITY;
                    if (!(sb >> (8 * j + 1) & 1)) v[4 * j + 3] = -INFINITY;
                }
            }
            float ma = fmaxf(v[0], v[1]), mb = fmaxf(v[2], v[3]);
#pragma unroll
            for (int j = 1; j < 8; ++j) {
                ma = tc::max3(ma, v[4 * j], v[4 * j + 1]);
                mb = tc::max3(mb, v[4 * j + 2], v[4 * j + 3]);
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                ma = fmaxf(ma, __shfl_xor_sync(FULL, ma, o));
                mb = fmaxf(mb, __shfl_xor_sync(FULL, mb, o));
            }
            ma *= sl2;
            mb *= sl2;
            // --- A row's reference (a whole number, in log2 units) moves up when a tile exceeds it by more than 8.  The one
            // that tile t-1 used comes from another group; rather than wait for it the probabilities are taken against this
            // group's last one, and corrected by a power of two in the rare case that it has moved. ---
            const auto moved = [&](float m, float from) {
                return m != -INFINITY && !(m <= from + RESCALE_LOG2) ? ceilf(m) : from;
            };
            float prev_a = ref_a, prev_b = ref_b;
            const bool ahead = __all_sync(FULL, ref_a != -INFINITY && ref_b != -INFINITY);
            const auto handed = [&]() {
                wait(bar->hand[q], t - 1, 117);
                prev_a = ms->m_pub[(t + G - 1) % G][ra];
                prev_b = ms->m_pub[(t + G - 1) % G][ra + 8];
            };
            if (!ahead && t > 0) handed();
            const float used_a = moved(ma, prev_a), used_b = moved(mb, prev_b);
            // --- probabilities, rounded to bf16 for the PV product; the row sums take the rounded ones ---
            const float neg_a = used_a == -INFINITY ? 0.0f : -used_a, neg_b = used_b == -INFINITY ? 0.0f : -used_b;
            uint32_t pk[16];
            float sa = 0.0f, sb = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const __nv_bfloat162 a = __floats2bfloat162_rn(tc::ex2_approx(fmaf(v[4 * j], sl2, neg_a)),
                                                               tc::ex2_approx(fmaf(v[4 * j + 1], sl2, neg_a)));
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(tc::ex2_approx(fmaf(v[4 * j + 2], sl2, neg_b)),
                                                                tc::ex2_approx(fmaf(v[4 * j + 3], sl2, neg_b)));
                pk[2 * j] = *(const uint32_t *)&a;
                pk[2 * j + 1] = *(const uint32_t *)&b2;
                sa = tc::add_bf16_f32((uint16_t)(pk[2 * j] & 0xffffu), sa);
                sb = tc::add_bf16_f32((uint16_t)(pk[2 * j + 1] & 0xffffu), sb);
                sa = tc::add_bf16_f32((uint16_t)(pk[2 * j] >> 16), sa);
                sb = tc::add_bf16_f32((uint16_t)(pk[2 * j + 1] >> 16), sb);
            }
            float now_a = used_a, now_b = used_b;
            if (ahead) {
                handed();
                now_a = moved(ma, prev_a);
                now_b = moved(mb, prev_b);
                if (__any_sync(FULL, now_a != used_a || now_b != used_b)) {
                    const float fa = pow2(used_a - now_a), fb = pow2(used_b - now_b);
                    const uint32_t fa2 = bf16_pair(fa), fb2 = bf16_pair(fb);
                    sa *= fa;
                    sb *= fb;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        pk[2 * j] = mul2(pk[2 * j], fa2);
                        pk[2 * j + 1] = mul2(pk[2 * j + 1], fb2);
                    }
                }
            }
            if (t + 1 < n) {
                if (c0 == 0) {
                    ms->m_pub[g][ra] = now_a;
                    ms->m_pub[g][ra + 8] = now_b;
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar->hand[q][t % NB]);
            }
            float alpha_a = 1.0f, alpha_b = 1.0f;  // what the context is multiplied by before PV(t)
            if (__any_sync(FULL, now_a != prev_a || now_b != prev_b || now_a != ref_a || now_b != ref_b)) {
                if (prev_a != -INFINITY) alpha_a = pow2(prev_a - now_a);
                if (prev_b != -INFINITY) alpha_b = pow2(prev_b - now_b);
                if (ref_a != -INFINITY) sum_a *= pow2(ref_a - now_a);
                if (ref_b != -INFINITY) sum_b *= pow2(ref_b - now_b);
                ref_a = now_a;
                ref_b = now_b;
            }
            sum_a += sa;
            sum_b += sb;
            // --- P(t), here and to the other CTA, into the buffer that both PV(t-2) are done with ---
            if (t >= 2) wait(bar->p_free, t - 2, 118);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                stmatrix4(tc::smem_u32(Pt) + p_row * 128 + (((j + (lane >> 4)) ^ (lane & 7)) << 4), pk[2 * j], pk[2 * j + 1],
                          pk[2 * j + 2], pk[2 * j + 3]);
            if (c0 == 0) {
                ms->alpha_out[buf][ra] = alpha_a;
                ms->alpha_out[buf][ra + 8] = alpha_b;
            }
            tc::fence_proxy_async_smem();  // read by the PV product and by the copies (async proxy)
            __syncwarp();
            if (lane == 0) {
                const uint32_t in = tc::map_peer(tc::smem_u32(&bar->p_in[t % NB]), peer);
                uint8_t *rows16 = Pt + (q * 32 + rank * 16) * 128;
                tc::bulk_copy_to_peer(tc::map_peer(tc::smem_u32(rows16), peer), rows16, 2048, in);
                tc::bulk_copy_to_peer(tc::map_peer(tc::smem_u32(&ms->alpha_in[buf][q * 16]), peer), &ms->alpha_out[buf][q * 16],
                                      64, in);
            }
            // --- the other CTA's rows have come back: the context moves after PV(t-1) and before PV(t) ---
            wait(bar->p_in, t, 119);
            __syncwarp();
            const float alpha = ((uint32_t)lane >> 4) == rank ? ms->alpha_out[buf][q * 16 + (lane & 15)]
                                                              : ms->alpha_in[buf][q * 16 + (lane & 15)];
            if (__any_sync(FULL, alpha != 1.0f)) {
                wait(bar->p_free, t - 1, 120);
                __syncwarp();
                rescale_rows(lanes, alpha);
            }
            ok = __all_sync(FULL, ok);
            if (lane == 0) tc::mbar_arrive(&bar->p_full[t % NB]);
        }
        // The PV products of the group's last tile are done in both CTAs: copies from here have been read, and the commits
        // that arrive here have arrived.
        if (ok && g < n) wait(bar->p_free, (n - 1 - g) / G * G + g, 121);
        __syncwarp();
        // ---------------- row sums, to both CTAs ----------------
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            sum_a += __shfl_xor_sync(FULL, sum_a, o);
            sum_b += __shfl_xor_sync(FULL, sum_b, o);
        }
        bar_and<1, 32 * SOFT>(ok);
        RowSums *rs = (RowSums *)X;
        if (c0 == 0) {
            rs->sum[g][ra] = sum_a;
            rs->sum[g][ra + 8] = sum_b;
            rs->ref[g][ra] = ref_a;
            rs->ref[g][ra + 8] = ref_b;
        }
        bar_and<1, 32 * SOFT>(ok);
        if (g == 0 && lane < 16) {
            const int r = q * 16 + lane, h = q * 32 + (int)rank * 16 + lane;
            float m = rs->ref[0][r], sum = 0.0f;
#pragma unroll
            for (int i = 1; i < G; ++i) m = fmaxf(m, rs->ref[i][r]);
#pragma unroll
            for (int i = 0; i < G; ++i)
                sum += rs->sum[i][r] * (rs->ref[i][r] == -INFINITY ? 1.0f : pow2(rs->ref[i][r] - m));  // (no reference: 0, or NaN)
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // a NaN that the row sees stays one
            ms->inv[h] = inv;
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(tc::map_peer(tc::smem_u32(&ms->inv[h]), peer)), "f"(inv)
                         : "memory");
            if (lrow + h < seq_rows) {
                const float row_lse = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * LN2;
                if (splits > 1) lpart[((int64_t)me.part0 + rem) * ROWS + h] = row_lse;
                else if (lse) lse[seq_row0 + lrow + h] = row_lse;
            }
        }
    }
    __syncwarp();
    if (!reaches) tc::cluster_wait();
    __syncthreads();
    if (*abort_flag) {
        // Copies that nobody waits for any more land within microseconds.
        const long long c0 = clock64();
        while (clock64() - c0 < kAbortQuietCycles) {
        }
    }
    tc::cluster_sync();  // both CTAs have every row's sum, and send each other nothing more
    if (warp < 16) {  // four warps a lane quarter
        // ---------------- epilogue: normalise, stage rows in the token stages, write whole rows ----------------
        const int q = warp & 3, g = warp >> 2, h = q * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        const float inv = ms->inv[h];
        const bool have = n > 0 && !*abort_flag, whole = splits == 1;
        tc::tc_fence_after();
        const int ld = whole ? OUT_LD_BF16 : OUT_LD_F32;
        uint8_t *srow = KV + h * ld;
#pragma unroll 1
        for (int cc = g * 2; cc < g * 2 + 2; ++cc) {
            float o[32];
            tc::tmem_ld32(lanes + COL_O + cc * 32, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = have && inv != 0.0f ? o[j] * inv : 0.0f;
            if (whole) {
                uint4 *d = (uint4 *)(srow + cc * 64);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 t2 = __floats2bfloat162_rn(o[8 * e + 2 * i], o[8 * e + 2 * i + 1]);
                        w[i] = *(const uint32_t *)&t2;
                    }
                    d[e] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else {
                float4 *d = (float4 *)(srow + cc * 128);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
        }
        bar_and<2, 512>(true);
        const int64_t part = whole ? 0 : (int64_t)me.part0 + rem;
        uint4 *dst = whole ? (uint4 *)(olat + (seq_row0 + lrow) * DC + rank * 256)
                           : (uint4 *)(opart + part * ROWS * DC + rank * 256);
        const int ld_dst = whole ? DC / 8 : DC / 4, two = whole ? 0 : 1;  // 16-byte words of a row; log2 of a lane's
        const int words = min(ROWS, seq_rows - lrow) << two;
#pragma unroll 1
        for (int i0 = warp; i0 < words; i0 += 64) {  // four loads ahead of four stores
            uint4 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + e * 16, row = i >> two, c = (i & two) * 32 + lane;
                if (i < words) v[e] = *((const uint4 *)(KV + row * ld) + c);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + e * 16, row = i >> two, c = (i & two) * 32 + lane;
                if (i < words) dst[(int64_t)row * ld_dst + c] = v[e];
            }
        }
        tc::tc_fence_before();
    }
    __syncthreads();
    if (warp == 2) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// Joins the normalised partial contexts of the split sequences: lse = log sum exp(lse_s), o = sum exp(lse_s -
// lse) o_s.  One warp per (row, quarter of the columns).
struct JoinParams {
    SeqTab st;
    int splits[DSA_MAX_SEQS];
    int part0[DSA_MAX_SEQS];
    int H;
    int64_t rows;
};
static_assert(sizeof(JoinParams) + 128 <= 32764, "launch parameters");
// AHEAD loads in flight a warp: eight where sequences are cut into 12 ranges or more, two where not (more warps fit).  Of one
// token and 128 heads each over 4000 or 8000 tokens, with two and with eight, us a call on the GPU: 25 sequences in 3 ranges
// 64.0 and 66.4, 15 in 5 52.3 and 53.5, 9 in 8 39.6 and 40.5, 7 in 11 50.0 and 50.2, 6 in 12 47.2 and 46.8, 4 in 18 37.0 and
// 35.9, one in 63 35.9 and 31.1.
template <int AHEAD>
__global__ void __launch_bounds__(256) tree_join_kernel(const __grid_constant__ JoinParams P,
                                                        const float *__restrict__ opart,
                                                        const float *__restrict__ lpart,
                                                        __nv_bfloat16 *__restrict__ olat, float *__restrict__ lse) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t rh = w >> 2;
    const int quarter = (int)(w & 3);
    if (rh >= P.rows) return;
    const int b = seq_of_row(P.st, (int)(rh / P.H));
    const int splits = P.splits[b];
    if (splits == 1) return;
    const int nt = (int)(((int64_t)(P.st.q_off[b + 1] - P.st.q_off[b]) * P.H + ROWS - 1) / ROWS);
    const int lr = (int)(rh - (int64_t)P.st.q_off[b] * P.H), rt = lr / ROWS;
    const int64_t p0 = P.part0[b] + (nt - 1 - rt);  // partial of split 0; split s: + s * nt
    const int i = lr - rt * ROWS;
    // lane s has splits s, s + 32, ..: their weights
    static_assert(kMaxSplits <= 96, "three splits a lane");
    float l[3], mxl = -INFINITY;
    bool bad = false;  // a NaN that the row sees
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int s = k * 32 + lane;
        l[k] = s < splits ? lpart[(p0 + (int64_t)s * nt) * ROWS + i] : -INFINITY;
        bad = bad || l[k] != l[k];
        mxl = fmaxf(mxl, l[k]);
    }
    bad = __any_sync(0xffffffffu, bad);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mxl = fmaxf(mxl, __shfl_xor_sync(0xffffffffu, mxl, o));
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
    if (mxl != -INFINITY) {
        const float *x = opart + (p0 * ROWS + i) * DC + quarter * 128 + lane * 4;
        const int64_t step = (int64_t)nt * ROWS * DC;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const float w = expf(l[k] - mxl);  // 0 behind the last split
            const int left = splits - k * 32;
#pragma unroll 1
            for (int s = 0; s < min(32, left); s += AHEAD, x += AHEAD * step) {
                float4 v[AHEAD];
#pragma unroll
                for (int e = 0; e < AHEAD; ++e)
                    v[e] = s + e < left ? __ldg((const float4 *)(x + e * step)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int e = 0; e < AHEAD; ++e) {
                    const float ws = __shfl_sync(0xffffffffu, w, s + e);
                    sum += ws;
                    acc.x = fmaf(ws, v[e].x, acc.x);
                    acc.y = fmaf(ws, v[e].y, acc.y);
                    acc.z = fmaf(ws, v[e].z, acc.z);
                    acc.w = fmaf(ws, v[e].w, acc.w);
                }
            }
        }
    }
    const float inv = bad ? NAN : sum > 0.0f ? 1.0f / sum : 0.0f;
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), c = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *((uint2 *)(olat + rh * DC + quarter * 128) + lane) = make_uint2(*(const uint32_t *)&a, *(const uint32_t *)&c);
    if (lse && quarter == 0 && lane == 0) lse[rh] = bad ? NAN : sum > 0.0f ? mxl + logf(sum) : -INFINITY;
}

// How the work is cut: every sequence's tokens in `splits` ranges of at most `chunk` tiles.
struct Plan {
    int splits[DSA_MAX_SEQS];
    int64_t units = 0, parts = 0;
};
struct Shape {
    int64_t nt;
    int tiles;
};
Shape shape_of(const Batch &bt, int H, int b) {
    const int64_t T = bt.st.q_off[b + 1] - bt.st.q_off[b];
    return Shape{(T * H + ROWS - 1) / ROWS, (int)(((int64_t)bt.st.start_pos[b] + T + TK - 1) / TK)};
}
// One pair of SMs works on a unit at a time, so units come in waves of half the SMs (76 on a GB300).  A unit costs its tiles and about
// kUnitCost tiles to start and end.  Of the chunk sizes that fill one, two, .. waves the cheapest is
// taken; no split at all competes with them, and saves the join: kJoinCost tiles, and kJoinSplit a split.
// (On the GPU alone, with 128 heads: one token over 1000 cached whole 36.0 us, in ranges of 2 tiles 27.1; 4 nodes of each
// of 8 sequences over 300 whole 26.2, in ranges of 4 32.9; 2 nodes of each of 12 over 3600 whole 77.7, of 19 tiles 53.9, of 12
// 69.6.)  kUnitCost is the plan's own and less than what a unit's start and end take alone (9 to 11 tiles): these choices
// come out alike with 6 and with 10.
constexpr int kUnitCost = 6, kMinChunk = 2, kMaxWaves = 4;
constexpr double kJoinCost = 4.5, kJoinSplit = 0.08;
int split_of(const Shape &s, int chunk) { return std::min(kMaxSplits, (s.tiles + chunk - 1) / chunk); }
void make_plan(const Batch &bt, int H, Plan &plan) {
    const int B = bt.st.B, pairs = std::max(1, device_sm_count() / 2);
    static thread_local Shape sh[DSA_MAX_SEQS];
    int longest = 1;
    int64_t work = 0, rows = 0;
    for (int b = 0; b < B; ++b) {
        sh[b] = shape_of(bt, H, b);
        if (!sh[b].nt) continue;
        longest = std::max(longest, sh[b].tiles);
        work += sh[b].nt * sh[b].tiles;
        rows += sh[b].nt;
    }
    const auto units = [&](int chunk) {
        int64_t n = 0;
        for (int b = 0; b < B; ++b) n += sh[b].nt * split_of(sh[b], chunk);
        return n;
    };
    int best = longest;
    // many waves: the average load and half of the longest unit; few: whole waves of the longest unit
    const auto cost = [&](int64_t n, int chunk) {
        const int64_t waves = (n + pairs - 1) / pairs;
        if (waves > kMaxWaves) return (double)(work + n * kUnitCost) / pairs + 0.5 * (chunk + kUnitCost);
        return (double)waves * (chunk + kUnitCost);
    };
    double least = cost(rows, longest);
    for (int w = 1; w <= kMaxWaves && rows <= (int64_t)w * pairs; ++w) {
        int lo = kMinChunk, hi = longest;  // the smallest chunk whose units fit w waves
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (units(mid) <= (int64_t)w * pairs) hi = mid; else lo = mid + 1;
        }
        const double c = cost(units(lo), lo) + kJoinCost + kJoinSplit * split_of(Shape{1, longest}, lo);
        if (c < least) {
            least = c;
            best = lo;
        }
    }
    plan.units = plan.parts = 0;
    for (int b = 0; b < B; ++b) {
        plan.splits[b] = sh[b].nt ? split_of(sh[b], best) : 0;
        plan.units += sh[b].nt * plan.splits[b];
        if (plan.splits[b] > 1) plan.parts += sh[b].nt * plan.splits[b];
    }
}

size_t part_bytes(const Plan &p) { return (size_t)p.parts * ROWS * DC * sizeof(float); }

}  // namespace

bool tree_tc_supported(int dtype, int H, int d_n, int d_r, int d_c, int d_v) {
    return dtype == DSA_BF16 && d_n == 128 && d_r == DR && d_c == DC && d_v == 128 && H >= 1;
}

size_t tree_tc_partial_bytes(int H, const Batch &bt) {
    static thread_local Plan plan;
    make_plan(bt, H, plan);
    return plan.parts ? (part_bytes(plan) + (size_t)plan.parts * ROWS * sizeof(float) + 255) / 256 * 256 : 0;
}

cudaError_t launch_tree_tc(const void *qt, const void *qpe, const dsa_latent_cache *c, const uint64_t *mask, int words,
                           const Batch &bt, const PageTab &pt, int H, float scale, void *olat, float *lse,
                           void *part_ws, cudaStream_t s) {
    static thread_local Plan plan;
    static thread_local TreeParams P;
    static thread_local JoinParams J;
    static thread_local int order[DSA_MAX_SEQS], per[DSA_MAX_SEQS];
    make_plan(bt, H, plan);
    const int B = bt.st.B, N = bt.total_q;
    int n = 0;
    for (int b = 0; b < B; ++b) {
        if (!plan.splits[b]) continue;
        order[n++] = b;
        per[b] = (shape_of(bt, H, b).tiles + plan.splits[b] - 1) / plan.splits[b];
    }
    std::sort(order, order + n, [&](int x, int y) { return per[x] != per[y] ? per[x] > per[y] : x < y; });  // (a stable sort would allocate)
    P.n_seq = n;
    int64_t unit = 0, part = 0;
    for (int i = 0; i < n; ++i) {
        const int b = order[i];
        const int64_t u = shape_of(bt, H, b).nt * plan.splits[b];
        P.s[i] = SeqUnits{(int)unit, bt.st.q_off[b], bt.st.q_off[b + 1] - bt.st.q_off[b], bt.st.start_pos[b],
                          pt.table ? b : bt.st.k_base[b], plan.splits[b], (int)part};
        J.part0[b] = (int)part;
        unit += u;
        if (plan.splits[b] > 1) part += u;
    }
    P.pt = pt;
    P.mask = mask;
    P.words = words;
    P.H = H;
    int k;
    P.scale_log2 = std::frexp(std::fabs(scale == 0.0f ? 1e-30f : scale * 1.4426950408889634f), &k);  // 0: every score counts alike
    const int kc = std::max(-120, std::min(120, k));
    P.scale_log2 = std::ldexp(P.scale_log2, k - kc);
    P.q_factor = 0x10001u * ((uint32_t)(kc + 127) << 7 | (scale < 0.0f ? 0x8000u : 0u));
    P.wait_limit = wait_limit_cycles();
    const uint64_t rows = (uint64_t)std::max<int64_t>(c->rows, 1);
    P.oob = (int)rows;
    const bool kv8 = c->dtype == DSA_E4M3;
    // Tokens that lie together: a whole tile (contiguous caches, pages of 64), or less.
    const int run = !pt.table || pt.page % TK == 0 ? TK : pt.page % 32 == 0 ? 32 : 16;
    CUtensorMap tq, tkv, tpe, tsc;
    {
        const uint64_t dims[2] = {DC, (uint64_t)N * H}, strides[1] = {DC * 2};
        const uint32_t box[2] = {64, ROWS};
        if (!make_tmap(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, qt, dims, strides, box)) return cudaErrorInvalidValue;
    }
    {
        const uint64_t pdims[2] = {DR, rows}, pstrides[1] = {(uint64_t)c->ld_pe * 2};
        const uint32_t pbox[2] = {32, (uint32_t)run};  // half of the rotary columns
        if (!make_tmap(&tpe, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c->k_pe, pdims, pstrides, pbox, CU_TENSOR_MAP_SWIZZLE_64B))
            return cudaErrorInvalidValue;
    }
    if (kv8) {
        const uint64_t dims[2] = {DC, rows}, strides[1] = {(uint64_t)c->ld_kv};
        const uint32_t box[2] = {RAW_LD, (uint32_t)run};
        const uint64_t sdims[2] = {DC / 128, rows}, sstrides[1] = {DC / 128 * 4};
        const uint32_t sbox[2] = {DC / 128, (uint32_t)run};
        if (!make_tmap(&tkv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, c->kv, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE) ||
            !make_tmap(&tsc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, c->kv_scale, sdims, sstrides, sbox,
                       CU_TENSOR_MAP_SWIZZLE_NONE))
            return cudaErrorInvalidValue;
    } else {
        // latents as slabs of 64 columns: (column, row, slab)
        const uint64_t dims[3] = {64, rows, DC / 64}, strides[2] = {(uint64_t)c->ld_kv * 2, 128};
        const uint32_t box[3] = {64, (uint32_t)run, run == TK ? 4u : 1u};
        if (!make_tmap(&tkv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, c->kv, dims, strides, box)) return cudaErrorInvalidValue;
        tsc = tkv;  // not used
    }
    float *opart = (float *)part_ws, *lpart = (float *)((char *)part_ws + part_bytes(plan));
    auto kern = kv8 ? tree_tc_kernel<true> : tree_tc_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)(2 * unit)), dim3(kv8 ? Cfg<true>::THREADS : Cfg<false>::THREADS), SMEM, s, tq, tkv, tpe, tsc, run,
                   (const __nv_bfloat16 *)qpe, P,
                   (__nv_bfloat16 *)olat, lse, opart, lpart);
    if (e != cudaSuccess) return e;
    note_launch(DSA_KERNEL_TREE_TC);
    if (!plan.parts) return cudaSuccess;
    J.st = bt.st;
    int most = 0;
    for (int b = 0; b < B; ++b) most = std::max(most, J.splits[b] = plan.splits[b]);
    J.H = H;
    J.rows = (int64_t)N * H;
    e = launch_pdl(most >= 12 ? tree_join_kernel<8> : tree_join_kernel<2>, dim3((unsigned)((J.rows * 4 + 7) / 8)), dim3(256), 0, s, J, (const float *)opart,
                   (const float *)lpart, (__nv_bfloat16 *)olat, lse);
    if (e != cudaSuccess) return e;
    note_launch(DSA_KERNEL_TREE_COMBINE);
    return cudaSuccess;
}

int tree_tc_read_error(int *site) {
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_tree_tc_error, sizeof(int));
    if (e != cudaSuccess) return fail_cuda(e);
    if (v) {
        e = cudaMemcpyToSymbol(g_tree_tc_error, &zero, sizeof(int));
        if (e != cudaSuccess) return fail_cuda(e);
        if (site) *site = v;
        return DSA_ERR_TIMEOUT;
    }
    return DSA_OK;
}

}  // namespace dsa
