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
//     memory).  CTA c finishes rows 64c .. 64c+63: the other CTA sends it its partial
//     scores of those rows (fp16, 8 KB), it adds its own in
//     fp32, runs the softmax and sends the probabilities (bf16, 8 KB) back, which both
//     need for PV.  Nothing is computed twice, and a row's maximum and sum live in
//     one place.
//   * Eight softmax warps in two groups that take alternate tiles.  Tensor-memory
//     lanes are rows, so in each group two warps finish the CTA's own rows (a thread
//     a row) and two send the other rows' partial scores and then watch for the
//     probabilities that come back.
//   * Lazy rescaling: a row's reference maximum moves only when a tile exceeds it by
//     more than 2^8; the factor travels with the probabilities, and both CTAs rescale
//     their half of the context.
//   * bf16 caches arrive by TMA (two copies a tile where 64 tokens lie together); of e4m3
//     caches four warps keep the next tile's codes in registers, dequantise (exact in
//     bf16) and store them swizzled.
//   * A token that some row does not see may hold anything, and 0 x NaN is NaN: tiles
//     with hidden tokens are loaded through registers, where Inf and NaN become 0.
//     Scores of hidden tokens are replaced after the MMA.
// Bound by shared memory and by the length of a tile's chain (score, exchange, softmax,
// exchange) over four stages of tokens: per tile a CTA's MMAs take 1088 cycles and its
// shared-memory traffic (MMA operands 92 KB, copies 37, scores and probabilities 64) 1.5K.
//
// Waits are bounded; a timeout records its site in the device error word and
// both CTAs drain and exit.
#include <algorithm>

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
constexpr int NSTAGE = 4;
constexpr int P_BYTES = ROWS * TK * 2;  // probabilities of all rows
constexpr int X_BYTES = HR * TK * 2;    // fp16 partial scores of half of the rows
constexpr int Q_BOX = ROWS * 128;       // 128 rows x 64 columns of q~ (staged in the exchange buffers)
constexpr int QR_BYTES = ROWS * 64;     // rotary slice of the queries, 64-byte swizzle
constexpr int NB = 6;                   // barriers of a kind: tile t uses number t % 6, which belongs to one softmax group and one
                                        // buffer whether there are two groups or three
constexpr uint32_t COL_S = 0, COL_Q = 128, COL_O = 256;
constexpr uint32_t IDESC_QK = tc::instr_desc(tc::kFmtBF16, tc::kFmtBF16, ROWS, TK, 0, 0);
constexpr uint32_t IDESC_PV = tc::instr_desc(tc::kFmtBF16, tc::kFmtBF16, ROWS, 256, 0, 1);
constexpr float RESCALE_LOG2 = 8.0f;
constexpr float LN2 = 0.69314718055994530942f;
constexpr long long kAbortQuietCycles = 1LL << 18;
constexpr int PAIRS = 76;               // 152 SMs
// warp 0: TMA; 1: QK^T; 2: tensor memory, PV; 3: bf16 tiles with hidden tokens; from 4 on the softmax groups of four
// (warp % 4 = lane quarter): three, or for e4m3 two, and 12-15 load
constexpr int THREADS = 512;
constexpr int MAX_G = 3;

struct Bars {
    uint64_t q_stage, q_ready, peer_ready, kv_full[NSTAGE], kv_empty[NSTAGE], raw[NSTAGE], s_full[NB], s_empty[NB];
    uint64_t x_full[NB], x_free[NB];  // the other CTA's partial scores are here; it has read ours
    uint64_t p_in[NB], p_full[NB];    // the other CTA's probabilities are here; all are, and the context is ready for them
    uint64_t p_free[NB];              // the PV products of both CTAs are done
    uint64_t hand[2][NB], mask_full[NB], qk_done, o_done;
};
struct Misc {
    float m_pub[MAX_G][HR];           // reference maximum that a group used, for the next tile's group
    float alpha_out[2][HR], alpha_in[2][HR];  // context factors of a tile, of this CTA's rows and of the other's
    float sum[MAX_G][HR], ref[MAX_G][HR];     // a group's share of the row sum and its reference
    float inv[ROWS];                  // 1 / row sum
    uint64_t live[NB];                // tokens of a tile whose page exists
    Bars bar;
    uint32_t tmem_slot;
    int abort_flag, never;
};
constexpr int SMEM = 1024 + NSTAGE * STAGE + 2 * P_BYTES + 4 * X_BYTES + QR_BYTES + (int)sizeof(Misc);
static_assert(SMEM <= 232448, "shared memory per CTA");
static_assert(4 * Q_BOX <= 2 * P_BYTES + 4 * X_BYTES, "the q~ slice is staged in the exchange buffers");
// The epilogue stages a CTA's 256 columns, rows 16 bytes apart from a power of two, in the token stages.
constexpr int OUT_LD_F32 = 256 * 4 + 16, OUT_LD_BF16 = 256 * 2 + 16;
static_assert(ROWS * OUT_LD_F32 <= NSTAGE * STAGE, "staged context");

// Sequences in the order of the units (the longest units first).
struct TreeParams {
    int n_seq;
    int q0[DSA_MAX_SEQS];        // first query row
    int T[DSA_MAX_SEQS];         // nodes
    int kbase[DSA_MAX_SEQS];     // first cache row (contiguous caches)
    int first[DSA_MAX_SEQS];     // tokens before the tree
    int seq[DSA_MAX_SEQS];       // the caller's sequence number
    int unit0[DSA_MAX_SEQS + 1]; // first unit
    int part0[DSA_MAX_SEQS];     // first partial context of a split sequence
    PageTab pt;
    const uint64_t *mask;
    int words, H;
    int oob;                     // a cache row past the last one
    int64_t ld_kv, ld_pe;
    float scale_log2;
    long long wait_limit;
};
static_assert(sizeof(TreeParams) + 3 * 128 + 128 <= 32764, "launch parameters");

// One 16-bit pair per word: bf16 Inf and NaN become 0.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
    return w;
}

// Four e4m3 codes -> four bf16 values times 2^120 (exact: the code's exponent and mantissa move to bf16's
// field, whose bias is 120 larger; subnormal codes become bf16 subnormals).
__device__ __forceinline__ void spread4(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    const uint32_t a = __byte_perm(codes, 0, 0x1404), b = __byte_perm(codes, 0, 0x3424);  // codes in the high bytes
    lo = (a & 0x80008000u) | ((a >> 4) & 0x07f007f0u);
    hi = (b & 0x80008000u) | ((b >> 4) & 0x07f007f0u);
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

// Maximum of 64 values as a tree (depth 4).
__device__ __forceinline__ float max64(const float (&v)[64]) {
    float a[22], b[8];
#pragma unroll
    for (int i = 0; i < 21; ++i) a[i] = tc::max3(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
    a[21] = v[63];
#pragma unroll
    for (int i = 0; i < 7; ++i) b[i] = tc::max3(a[3 * i], a[3 * i + 1], a[3 * i + 2]);
    b[7] = a[21];
    return tc::max3(tc::max3(b[0], b[1], b[2]), tc::max3(b[3], b[4], b[5]), fmaxf(b[6], b[7]));
}

template <bool KV8>
struct Cfg {
    static constexpr int G = KV8 ? 2 : 3;  // softmax groups
};

template <bool KV8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                   const __grid_constant__ CUtensorMap tm_pe, int run, const void *__restrict__ kv,
                   const float *__restrict__ kv_scale, const __nv_bfloat16 *__restrict__ kpe,
                   const __nv_bfloat16 *__restrict__ qpe, const __grid_constant__ TreeParams P,
                   __nv_bfloat16 *__restrict__ olat, float *__restrict__ lse, float *__restrict__ opart,
                   float *__restrict__ lpart) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *KV = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    constexpr int G = Cfg<KV8>::G, SOFT = 4 * G;
    uint8_t *Pb = KV + NSTAGE * STAGE;   // [t % 2] probabilities: rows x 64 tokens, 128-byte swizzle
    uint8_t *X = Pb + 2 * P_BYTES;       // [t % 2] the other CTA's partial scores of this CTA's rows
    uint8_t *Y = X + 2 * X_BYTES;        // [t % 2] this CTA's partial scores of the other's rows, sent from here
    uint8_t *QR = Y + 2 * X_BYTES;       // rotary slice of the queries
    Misc *ms = (Misc *)(QR + QR_BYTES);
    Bars *bar = &ms->bar;
    volatile int *abort_flag = (volatile int *)&ms->abort_flag, *nv = (volatile int *)&ms->never;
    int *err = &g_tree_tc_error;

    const unsigned FULL = 0xffffffffu;
    const int warp = __shfl_sync(FULL, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank(), peer = rank ^ 1u;

    // ---- the unit: rows row0 .. of a sequence, tiles t0 .. t0 + n - 1 of its tokens ----
    const int u = (int)(blockIdx.x >> 1);
    int lo = 0, hi = P.n_seq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P.unit0[mid] <= u) lo = mid; else hi = mid - 1;
    }
    const int T = P.T[lo], first = P.first[lo], b = P.seq[lo], kbase = P.kbase[lo];
    const int nt = (int)(((int64_t)T * P.H + ROWS - 1) / ROWS);
    const int splits = (P.unit0[lo + 1] - P.unit0[lo]) / nt;
    const int rem = u - P.unit0[lo], split = rem / nt, rt = nt - 1 - (rem - split * nt);
    const int seq_rows = T * P.H;                                  // rows of the sequence
    const int64_t seq_row0 = (int64_t)P.q0[lo] * P.H;
    const int lrow = rt * ROWS;                                    // first row of the unit within the sequence
    const int node_lo = lrow / P.H, node_hi = min(T - 1, (lrow + ROWS - 1) / P.H);
    const int tokens = first + (P.mask ? T : node_hi + 1);         // tokens that some row may see
    const int safe = first + (P.mask ? 0 : node_lo + 1);           // tokens before this one are seen by every row
    const int tiles = (first + T + TK - 1) / TK;
    const int per = (tiles + splits - 1) / splits;
    const int t0 = split * per;
    const int n = max(0, min((tokens + TK - 1) / TK, t0 + per) - t0);

    if (threadIdx.x == 0) {
        tc::mbar_init(&bar->q_stage, 1);
        tc::mbar_init(&bar->q_ready, SOFT);
        tc::mbar_init(&bar->peer_ready, 1);
        for (int i = 0; i < NSTAGE; ++i) {
            tc::mbar_init(&bar->kv_full[i], KV8 ? 4 : 1);
            tc::mbar_init(&bar->kv_empty[i], 1);
            tc::mbar_init(&bar->raw[i], 1);
        }
        for (int i = 0; i < NB; ++i) {
            tc::mbar_init(&bar->s_full[i], 1);
            tc::mbar_init(&bar->s_empty[i], 4);  // the group's warps have read the scores
            tc::mbar_init(&bar->x_full[i], 1);   // armed here with what the other CTA sends
            tc::mbar_init(&bar->x_free[i], 2);   // its two finishing warps
            tc::mbar_init(&bar->p_in[i], 1);
            tc::mbar_init(&bar->p_full[i], 4);
            tc::mbar_init(&bar->p_free[i], 2);
            tc::mbar_init(&bar->hand[0][i], 1);
            tc::mbar_init(&bar->hand[1][i], 1);
            tc::mbar_init(&bar->mask_full[i], 1);
        }
        tc::mbar_init(&bar->qk_done, 1);
        tc::mbar_init(&bar->o_done, 1);
        *abort_flag = 0;
        ms->never = 0;
        tc::fence_mbar_init();
    }
    if (warp == 2) {
        tc::tmem_alloc(&ms->tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    tc::cluster_sync();  // both CTAs' barriers exist before any remote arrive
    const uint32_t tmem = __shfl_sync(FULL, ms->tmem_slot, 0);
    pdl_wait();  // the set-up above overlapped the previous kernel; global memory only from here

    // Cache row of token s, or -1 (behind the last token, or on no page).
    const auto row_of = [&](int s) -> int64_t { return s < tokens ? cache_row(P.pt, b, kbase, s) : -1; };
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
        // ---------------- TMA: the q~ slice (staged in the exchange buffers), then a bf16 cache's tiles ----------------
        if (lane == 0) {
            tc::mbar_arrive_expect_tx(&bar->q_stage, 4 * Q_BOX);
            for (int j = 0; j < 4; ++j)
                tc::tma_load_2d(Pb + j * Q_BOX, &tm_q, &bar->q_stage, rank * 256 + j * 64, (int)(seq_row0 + lrow));
        }
        __syncwarp();
        if constexpr (!KV8) {
            // Lane's copy: latents of run k (all four slabs at once where 64 tokens lie together), or rotary columns.
            const int runs = TK / run, nlat = runs == 1 ? 1 : 4 * runs;
            const bool lat = lane < nlat;
            const int k = lat ? (runs == 1 ? 0 : lane >> 2) : lane - nlat, j = lat && runs > 1 ? lane & 3 : 0;
            int rows = runs_of(0);
            bool ok = true;
            for (int t = 0; ok && t < n; ++t) {
                const int st = t % NSTAGE;
                ok = __all_sync(FULL, tc::mbar_wait(&bar->kv_empty[st], ((t / NSTAGE) & 1) ^ 1, abort_flag, err, 101, P.wait_limit));
                if (!ok) break;
                put_mask(t, rows);
                // Tiles with hidden tokens pass through warp 3; of runs behind the last token nothing is read.
                uint64_t *full = (t0 + t + 1) * TK > safe ? &bar->raw[st] : &bar->kv_full[st];
                const int row = __shfl_sync(FULL, rows, (k * (run / 16)) & 3);
                const bool go = (lat || k < runs) && row >= 0;
                const int n_lat = __popc(__ballot_sync(FULL, go && lat)), n_pe = __popc(__ballot_sync(FULL, go && !lat));
                if (lane == 0)
                    tc::mbar_arrive_expect_tx(full, (uint32_t)(run * (n_lat * (runs == 1 ? 512 : 128) + n_pe * 64)));
                __syncwarp();
                uint8_t *dst = KV + st * STAGE;
                if (go && lat) tc::tma_load_3d(dst + j * SLAB + k * run * 128, &tm_kv, full, 0, row, rank * 4 + j);
                else if (go) tc::tma_load_2d(dst + 4 * SLAB + k * run * 64, &tm_pe, full, rank * 32, row);
                rows = runs_of(t + 1);
            }
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
            const int st = t % NSTAGE;
            if (t >= 2) ok = tc::mbar_wait(&bar->s_empty[(t - 2) % NB], ((t - 2) / NB) & 1, abort_flag, err, 103, P.wait_limit);
            ok = tc::mbar_wait(&bar->kv_full[st], (t / NSTAGE) & 1, abort_flag, err, 104, P.wait_limit) && ok;
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
            if (issue) tc::mma_commit(&bar->s_full[t % NB]);
            __syncwarp();
        }
        // No MMA of this warp may still be running when the tensor memory is released.
        if (issue) tc::mma_commit(&bar->qk_done);
        tc::mbar_wait(&bar->qk_done, 0, nv, err, 105);
    } else if (warp == 2 && n > 0) {
        // ---------------- PV issuer: frees the stage and the probabilities (which both CTAs hold) ----------------
        const uint32_t issue = tc::elect_one();
        const uint32_t kv0 = __shfl_sync(FULL, tc::smem_u32(KV), 0), p0 = __shfl_sync(FULL, tc::smem_u32(Pb), 0);
        const uint64_t pd = tc::smem_desc(p0, 16, 1024), vd = tc::smem_desc(kv0, SLAB, 1024);
        for (int t = 0; t < n; ++t) {
            if (!__all_sync(FULL, tc::mbar_wait(&bar->p_full[t % NB], (t / NB) & 1, abort_flag, err, 106, P.wait_limit))) break;
            tc::tc_fence_after();
            const int st = t % NSTAGE;
            const uint64_t a0 = pd + (uint64_t)(uint32_t)((t & 1) * (P_BYTES / 16));
            const uint64_t b0 = vd + (uint64_t)(uint32_t)(st * (STAGE / 16));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                tc::mma_f16_if(issue, tmem + COL_O, a0 + kk * 2, b0 + kk * (16 * 128 / 16), IDESC_PV, (t | kk) != 0);
            if (issue) {
                tc::mma_commit(&bar->kv_empty[st]);
                tc::mma_commit_multicast(&bar->p_free[t % NB], 3);
            }
            __syncwarp();
        }
        if (issue) tc::mma_commit(&bar->o_done);
        tc::mbar_wait(&bar->o_done, 0, nv, err, 107);
        tc::mbar_wait(&bar->q_stage, 0, nv, err, 108);  // after an abort nobody else may have waited for it
    } else if (!KV8 && warp == 3 && n > 0) {
        // ---------------- bf16 tiles with hidden tokens: Inf and NaN of the latents (V) become 0 ----------------
        for (int t = max(0, safe / TK - t0); t < n; ++t) {
            const int st = t % NSTAGE;
            // the stage's first such tile is number t % NSTAGE + a multiple: every phase of `raw` is this warp's
            const int use = (t - max(0, safe / TK - t0)) / NSTAGE;
            if (!__all_sync(FULL, tc::mbar_wait(&bar->raw[st], use & 1, abort_flag, err, 110, P.wait_limit))) break;
            uint4 *p = (uint4 *)(KV + st * STAGE) + lane;
#pragma unroll 8
            for (int i = 0; i < 4 * SLAB / 512; ++i) {
                const uint4 v = p[i * 32];
                const uint4 f = make_uint4(finite2(v.x), finite2(v.y), finite2(v.z), finite2(v.w));
                if ((v.x ^ f.x) | (v.y ^ f.y) | (v.z ^ f.z) | (v.w ^ f.w)) p[i * 32] = f;
            }
            tc::fence_proxy_async_smem();  // read by the MMAs (async proxy)
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar->kv_full[st]);
        }
    } else if (KV8 && warp >= 12 && n > 0) {
        // ---------------- loading warps (e4m3) ----------------
        // Warp w brings 16 tokens, which lie together: one look at the block table a tile.
        const int w = warp - 12;
        int64_t row = -1;   // of its first token
        int count = 0;      // tokens that exist
        const auto locate = [&](int t) {
            const int s = (t0 + t) * TK + w * 16;
            row = row_of(s);
            count = row >= 0 ? min(16, tokens - s) : 0;
        };
        // Rotary columns: eight tokens x four 16-byte chunks an instruction.
        uint4 rp[2];
        const auto get_rope = [&]() {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int tok = e * 8 + (lane >> 2);
                rp[e] = tok < count ? __ldg((const uint4 *)(kpe + (row + tok) * P.ld_pe + rank * 32) + (lane & 3))
                                    : make_uint4(0, 0, 0, 0);
            }
        };
        const auto put_rope = [&](uint8_t *stage) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int tok = w * 16 + e * 8 + (lane >> 2);
                *(uint4 *)(stage + 4 * SLAB + tok * 64 + (((lane & 3) ^ ((tok >> 1) & 3)) << 4)) = rp[e];
            }
        };
        bool ok = true;
        {
            // Pass i: tokens 4 (i / 2) .., block i % 2 of the CTA's two; a token's 128 codes are eight lanes' 16 bytes.
            // The next tile's codes wait in registers.
            const uint8_t *codes = (const uint8_t *)kv + rank * 256 + (lane & 7) * 16;
            uint4 c[8];
            float sc = 0.0f;   // scale of token lane / 2, block lane % 2
            int runs = 0;
            const auto fetch = [&](int t) {
                locate(t);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int tok = (i >> 1) * 4 + (lane >> 3);
                    c[i] = tok < count ? __ldg((const uint4 *)(codes + (row + tok) * P.ld_kv + (i & 1) * 128))
                                       : make_uint4(0, 0, 0, 0);
                }
                sc = (lane >> 1) < count ? __ldg(kv_scale + (row + (lane >> 1)) * (DC / 128) + rank * 2 + (lane & 1)) : 0.0f;
                get_rope();
                if (w == 0) runs = runs_of(t);
            };
            const int slab = (lane >> 2) & 1, chunk = (lane & 3) * 2;
            fetch(0);
            for (int t = 0; t < n; ++t) {
                const int st = t % NSTAGE;
                ok = __all_sync(FULL, tc::mbar_wait(&bar->kv_empty[st], ((t / NSTAGE) & 1) ^ 1, abort_flag, err, 109, P.wait_limit));
                if (!ok) break;
                if (w == 0) put_mask(t, runs);
                uint8_t *stage = KV + st * STAGE;
                // A hidden token's scale may be anything: past what a finite product allows it counts as 0 (the codes
                // themselves become finite numbers, whatever they are).
                if ((t0 + t + 1) * TK > safe && !(fabsf(sc) <= 0x1p118f)) sc = 0.0f;
                // 2^120 scale is one factor while it stays in bf16's range
                const bool big = __any_sync(FULL, sc > 128.0f);
                const float up = big ? 0x1p120f : 0x1p120f * sc;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int tok = (i >> 1) * 4 + (lane >> 3);
                    const float f = __shfl_sync(FULL, up, tok * 2 + (i & 1));
                    uint4 o[2];
                    dequant16(c[i], bf16_pair(f), o);
                    uint8_t *dst = stage + ((i & 1) * 2 + slab) * SLAB + (w * 16 + tok) * 128;
                    const int x = (w * 16 + tok) & 7;
                    // the two slabs' lanes store their chunks in opposite order: eight lanes cover all banks
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *(uint4 *)(dst + (((chunk + (e ^ slab)) ^ x) << 4)) = (e ^ slab) ? o[1] : o[0];
                }
                if (big) {  // the second factor, over the stored values
#pragma unroll 1
                    for (int i = 0; i < 16; ++i) {
                        const int tok = i, lane_slab = lane >> 3;
                        const float f = __shfl_sync(FULL, sc, tok * 2 + (lane_slab >> 1));
                        uint4 *p = (uint4 *)(stage + lane_slab * SLAB + (w * 16 + tok) * 128 + (lane & 7) * 16);
                        __syncwarp();
                        uint4 v = *p;
                        const uint32_t m = bf16_pair(f);
                        *p = make_uint4(mul2(v.x, m), mul2(v.y, m), mul2(v.z, m), mul2(v.w, m));
                    }
                }
                put_rope(stage);
                tc::fence_proxy_async_smem();  // read by the MMAs (async proxy)
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar->kv_full[st]);
                if (t + 1 < n) fetch(t + 1);
            }
        }
    } else if (warp >= 4 && warp < 4 + SOFT) {
        // ---------------- softmax groups: group g takes tiles g, g + G, ..; thread = row h ----------------
        const int q = warp & 3, g = (warp >> 2) - 1, h = q * 32 + lane;
        const bool own = (uint32_t)(q >> 1) == rank;      // rows that this CTA finishes
        const int r = h & 63;                             // row within its half
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        bool ok = true;
        if (n > 0) {
            // The q~ slice moves to tensor memory (A operand of QK^T): four slabs of 32 packed columns, two each of the first
            // groups; the last one puts the rotary slice of the queries into shared memory.
            uint4 rq[4];
            if (g == G - 1) {
                const int64_t row = seq_row0 + lrow + h;
                const bool there = lrow + h < seq_rows;
                const uint4 *src = (const uint4 *)(qpe + row * DR + rank * 32);
#pragma unroll
                for (int e = 0; e < 4; ++e) rq[e] = there ? __ldg(src + e) : make_uint4(0, 0, 0, 0);
            }
            ok = __all_sync(FULL, tc::mbar_wait(&bar->q_stage, 0, abort_flag, err, 111, P.wait_limit));
            for (int js = g * 2; ok && g < 2 && js < g * 2 + 2; ++js) {
                const uint8_t *srow = Pb + js * Q_BOX + h * 128;
                uint32_t qv[32];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint4 t4 = *(const uint4 *)(srow + ((e ^ (h & 7)) << 4));
                    qv[4 * e] = t4.x;
                    qv[4 * e + 1] = t4.y;
                    qv[4 * e + 2] = t4.z;
                    qv[4 * e + 3] = t4.w;
                }
                tc::tmem_st32(lanes + COL_Q + js * 32, qv);
            }
            tc::tmem_st_wait();
            if (g == G - 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) *(uint4 *)(QR + h * 64 + ((e ^ ((h >> 1) & 3)) << 4)) = rq[e];
                tc::fence_proxy_async_smem();  // read by the rotary MMAs (async proxy)
            }
            tc::tc_fence_before();
            // Every warp has read its part of the staging: the buffers may carry scores, here and from the other CTA.
            ok = bar_and<1, 32 * SOFT>(ok);
            if (lane == 0) tc::mbar_arrive(&bar->q_ready);
            if (threadIdx.x == 4 * 32) tc::mbar_arrive_remote(tc::map_peer(tc::smem_u32(&bar->peer_ready), peer));
            ok = ok && __all_sync(FULL, tc::mbar_wait(&bar->peer_ready, 0, abort_flag, err, 112, P.wait_limit));
        }
        const float sl2 = fabsf(P.scale_log2);            // not 0
        const bool negative = P.scale_log2 < 0.0f;
        const auto sw = [&](uint8_t *rowp, int c) { return rowp + ((c ^ (h & 7)) << 4); };
        // this warp's scores of tile t
        const auto load_scores = [&](int t, float (&v)[64]) {
            tc::tc_fence_after();
            float a[32], c[32];
            tc::tmem_ld32(lanes + COL_S + (t & 1) * TK, a);
            tc::tmem_ld32(lanes + COL_S + (t & 1) * TK + 32, c);
            tc::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                v[j] = a[j];
                v[32 + j] = c[j];
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar->s_empty[t % NB]);
            if (negative) {
#pragma unroll
                for (int j = 0; j < 64; ++j) v[j] = -v[j];
            }
        };
        // A lane's waits only note a failure; the warp stops together at the end of the tile.
        const auto wait = [&](uint64_t *bars, int t, int site) {
            ok = tc::mbar_wait(&bars[t % NB], (t / NB) & 1, abort_flag, err, site, P.wait_limit) && ok;
        };
        if (own) {
            const int li = lrow + h;                      // row within the sequence
            const bool mine = li < seq_rows;              // else a row of the next sequence, or none
            const int node = mine ? li / P.H : 0;
            const uint64_t *bits = P.mask ? P.mask + (int64_t)(P.q0[lo] + node) * P.words : nullptr;
            float m_g = -INFINITY, l_g = 0.0f;            // this group's reference and its share of the row sum
            for (int t = g; ok && t < n; t += G) {
                uint8_t *Xb = X + (t & 1) * X_BYTES, *Pt = Pb + (t & 1) * P_BYTES;
                if (lane == 0 && !(q & 1)) tc::mbar_arrive_expect_tx(&bar->x_full[t % NB], X_BYTES);
                // --- which of the 64 tokens the row sees ---
                uint64_t see = ~0ull;
                if ((t0 + t + 1) * TK > safe) {
                    const int rel = (t0 + t) * TK - first;  // node number of the first token (negative: before the tree)
                    if (!bits) {
                        const int left = node + 1 - rel;
                        see = left >= 64 ? ~0ull : left <= 0 ? 0ull : (1ull << left) - 1;
                    } else if (rel + 64 > 0) {
                        const int w = rel >> 6, sh = rel & 63;
                        const uint64_t w0 = w < 0 ? ~0ull : w < P.words ? __ldg(bits + w) : 0ull;
                        const uint64_t w1 = w + 1 < P.words ? __ldg(bits + w + 1) : 0ull;
                        see = sh ? (w0 >> sh) | (w1 << (64 - sh)) : w0;
                        const int left = T - rel;
                        if (left < 64) see &= left <= 0 ? 0ull : (1ull << left) - 1;
                    }
                }
                if (P.pt.table) {
                    wait(bar->mask_full, t, 113);
                    see &= ms->live[t % NB];
                }
                wait(bar->s_full, t, 114);
                __syncwarp();
                float v[64];
                load_scores(t, v);
                // --- + the other CTA's half ---
                wait(bar->x_full, t, 115);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint4 x = *(const uint4 *)sw(Xb + r * 128, c);
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[8 * c + 2 * e] = tc::add_f16_f32((uint16_t)(xs[e] & 0xffffu), v[8 * c + 2 * e]);
                        v[8 * c + 2 * e + 1] = tc::add_f16_f32((uint16_t)(xs[e] >> 16), v[8 * c + 2 * e + 1]);
                    }
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_remote(tc::map_peer(tc::smem_u32(&bar->x_free[t % NB]), peer));
                if (!__all_sync(FULL, see == ~0ull)) {
                    const uint32_t s0 = (uint32_t)see, s1 = (uint32_t)(see >> 32);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (!(s0 >> j & 1)) v[j] = -INFINITY;
                        if (!(s1 >> j & 1)) v[32 + j] = -INFINITY;
                    }
                }
                const float mt = max64(v) * sl2;
                // --- The row's reference (a whole number, in log2 units) moves up when a tile exceeds it by more than 8.  The
                // one that tile t-1 used comes from the other group; rather than wait for it the probabilities are taken
                // against this group's last one, and corrected by a power of two in the rare case that it has moved. ---
                const auto moved = [&](float from) {
                    return mt != -INFINITY && !(mt <= from + RESCALE_LOG2) ? ceilf(mt) : from;
                };
                float m_prev = m_g, m_used;
                const bool ahead = __all_sync(FULL, m_g != -INFINITY);
                const auto handed = [&]() {
                    wait(bar->hand[q & 1], t - 1, 116);
                    m_prev = ms->m_pub[(t + G - 1) % G][r];
                };
                if (!ahead && t > 0) handed();
                m_used = moved(m_prev);
                // --- probabilities, rounded to bf16 for the PV product; the row sum takes the rounded ones ---
                const float neg = m_used == -INFINITY ? 0.0f : -m_used;
                uint32_t pk[32];
                float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float p0 = tc::ex2_approx(fmaf(v[2 * j], sl2, neg)), p1 = tc::ex2_approx(fmaf(v[2 * j + 1], sl2, neg));
                    const __nv_bfloat162 t2 = __floats2bfloat162_rn(p0, p1);
                    pk[j] = *(const uint32_t *)&t2;
                    sum0 = tc::add_bf16_f32((uint16_t)(pk[j] & 0xffffu), sum0);
                    sum1 = tc::add_bf16_f32((uint16_t)(pk[j] >> 16), sum1);
                }
                float sum = sum0 + sum1, m_now = m_used;
                if (ahead) {
                    handed();
                    m_now = moved(m_prev);
                    if (__any_sync(FULL, m_now != m_used)) {
                        const float f = pow2(m_used - m_now);
                        const uint32_t f2 = bf16_pair(f);
                        sum *= f;
#pragma unroll
                        for (int j = 0; j < 32; ++j) pk[j] = mul2(pk[j], f2);
                    }
                }
                if (t + 1 < n) {
                    ms->m_pub[g][r] = m_now;
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar->hand[q & 1][t % NB]);
                }
                float alpha = 1.0f;
                if (__any_sync(FULL, m_now != m_prev || m_now != m_g)) {
                    if (m_prev != -INFINITY) alpha = pow2(m_prev - m_now);
                    if (m_g != -INFINITY) l_g *= pow2(m_g - m_now);
                    m_g = m_now;
                }
                l_g += sum;
                // --- the buffer that P(t) goes to is free once both PV(t-2) are done ---
                if (t >= 2) wait(bar->p_free, t - 2, 117);
                // --- the context moves after PV(t-1) and before PV(t) ---
                if (__any_sync(FULL, alpha != 1.0f)) {
                    wait(bar->p_free, t - 1, 118);
                    __syncwarp();
                    rescale_rows(lanes, alpha);
                }
                // --- P(t), here and to the other CTA ---
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    *(uint4 *)sw(Pt + h * 128, c) = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                ms->alpha_out[t & 1][r] = alpha;
                tc::fence_proxy_async_smem();  // read by the PV product and by the copies (async proxy)
                ok = __all_sync(FULL, ok);
                if (lane == 0) {
                    const uint32_t in = tc::map_peer(tc::smem_u32(&bar->p_in[t % NB]), peer);
                    uint8_t *rows32 = Pt + q * 32 * 128;
                    tc::bulk_copy_to_peer(tc::map_peer(tc::smem_u32(rows32), peer), rows32, 32 * 128, in);
                    tc::bulk_copy_to_peer(tc::map_peer(tc::smem_u32(&ms->alpha_in[t & 1][(q & 1) * 32]), peer),
                                          &ms->alpha_out[t & 1][(q & 1) * 32], 32 * 4, in);
                    tc::mbar_arrive(&bar->p_full[t % NB]);
                }
            }
            // The PV products of the group's last tile are done in both CTAs: copies from here have been read, and the
            // commits that arrive here have arrived.
            if (ok && g < n) wait(bar->p_free, (n - 1 - g) / G * G + g, 119);
            ms->sum[g][r] = l_g;
            ms->ref[g][r] = m_g;
        } else {
            // The probabilities of these rows and their context factors, when they come back: tile t is ready for PV here.
            const auto take = [&](int t) {
                const float alpha = ms->alpha_in[t & 1][r];
                if (__any_sync(FULL, alpha != 1.0f)) {
                    wait(bar->p_free, t - 1, 120);
                    __syncwarp();
                    rescale_rows(lanes, alpha);
                }
                ok = __all_sync(FULL, ok);
                if (lane == 0) tc::mbar_arrive(&bar->p_full[t % NB]);
            };
            bool owed = false;  // the previous tile's probabilities have not been taken yet
            for (int t = g; ok && t < n; t += G) {
                uint8_t *Yb = Y + (t & 1) * X_BYTES;
                if (lane == 0 && !(q & 1)) tc::mbar_arrive_expect_tx(&bar->p_in[t % NB], X_BYTES + HR * 4);
                // Whichever is first: this tile's scores, or the previous one's probabilities.
                if (owed) {
                    const long long c0 = clock64();
                    while (!__all_sync(FULL, tc::mbar_test(&bar->s_full[t % NB], (t / NB) & 1))) {
                        if (__all_sync(FULL, tc::mbar_test(&bar->p_in[(t - G) % NB], ((t - G) / NB) & 1))) {
                            take(t - G);
                            owed = false;
                            break;
                        }
                        // the wait below reports it
                        if (__any_sync(FULL, *abort_flag || clock64() - c0 > P.wait_limit)) break;
                    }
                }
                // the other CTA has read tile t - 2 from its buffer, and so from the one here
                if (t >= 2) wait(bar->x_free, t - 2, 121);
                wait(bar->s_full, t, 122);
                __syncwarp();
                float v[64];
                load_scores(t, v);
                uint32_t w[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) w[j] = tc::f16x2_satfinite(v[2 * j], v[2 * j + 1]);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    *(uint4 *)sw(Yb + r * 128, c) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                tc::fence_proxy_async_smem();  // read by the copy (async proxy)
                __syncwarp();
                if (lane == 0)
                    tc::bulk_copy_to_peer(tc::map_peer(tc::smem_u32(X + (t & 1) * X_BYTES + (q & 1) * 32 * 128), peer),
                                          Yb + (q & 1) * 32 * 128, 32 * 128,
                                          tc::map_peer(tc::smem_u32(&bar->x_full[t % NB]), peer));
                if (owed) {
                    wait(bar->p_in, t - G, 123);
                    take(t - G);
                }
                ok = __all_sync(FULL, ok);
                owed = true;
            }
            if (ok && owed) {
                const int t = (n - 1 - g) / G * G + g;  // the group's last tile
                wait(bar->p_in, t, 124);
                take(t);
            }
        }
        // ---------------- row sums: the finishing warps' results, to both CTAs ----------------
        bar_and<1, 32 * SOFT>(ok);
        if (own && g == 0) {
            float m = ms->ref[0][r], sum = 0.0f;
#pragma unroll
            for (int i = 1; i < G; ++i) m = fmaxf(m, ms->ref[i][r]);
#pragma unroll
            for (int i = 0; i < G; ++i)
                if (ms->ref[i][r] != -INFINITY) sum += ms->sum[i][r] * pow2(ms->ref[i][r] - m);
            const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
            ms->inv[h] = inv;
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(tc::map_peer(tc::smem_u32(&ms->inv[h]), peer)), "f"(inv)
                         : "memory");
            if (lrow + h < seq_rows) {
                const float row_lse = sum > 0.0f ? (m + log2f(sum)) * LN2 : -INFINITY;
                if (splits > 1) lpart[((int64_t)P.part0[lo] + rem) * ROWS + h] = row_lse;
                else if (lse) lse[seq_row0 + lrow + h] = row_lse;
            }
        }
    }
    __syncthreads();
    if (*abort_flag) {
        // Copies that nobody waits for any more land within microseconds.
        const long long c0 = clock64();
        while (clock64() - c0 < kAbortQuietCycles) {
        }
    }
    tc::cluster_sync();  // both CTAs have every row's sum, and send each other nothing more
    if (warp >= 4 && warp < 12) {  // two warps a lane quarter
        // ---------------- epilogue: normalise, stage rows in the token stages, write whole rows ----------------
        const int q = warp & 3, g = (warp >> 2) - 1, h = q * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        const float inv = ms->inv[h];
        const bool have = n > 0 && !*abort_flag, whole = splits == 1;
        tc::tc_fence_after();
        const int ld = whole ? OUT_LD_BF16 : OUT_LD_F32;
        uint8_t *srow = KV + h * ld;
#pragma unroll 1
        for (int cc = g * 4; cc < g * 4 + 4; ++cc) {
            float o[32];
            tc::tmem_ld32(lanes + COL_O + cc * 32, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = have && inv > 0.0f ? o[j] * inv : 0.0f;
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
        bar_and<2, 256>(true);
        const int64_t part = whole ? 0 : (int64_t)P.part0[lo] + rem;
        const int rows = min(ROWS, seq_rows - lrow);
        for (int i = warp - 4; i < rows; i += 8) {
            const uint4 *src = (const uint4 *)(KV + i * ld);
            uint4 *dst = whole ? (uint4 *)(olat + (seq_row0 + lrow + i) * DC + rank * 256)
                               : (uint4 *)(opart + (part * ROWS + i) * DC + rank * 256);
            for (int c = lane; c < (whole ? 32 : 64); c += 32) dst[c] = src[c];
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
    float mxl = -INFINITY;
    for (int s = lane; s < splits; s += 32) mxl = fmaxf(mxl, lpart[(p0 + (int64_t)s * nt) * ROWS + i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mxl = fmaxf(mxl, __shfl_xor_sync(0xffffffffu, mxl, o));
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
    if (mxl != -INFINITY) {
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
            const int64_t p = (p0 + (int64_t)s * nt) * ROWS + i;
            const float wgt = expf(lpart[p] - mxl);
            const float4 x = *((const float4 *)(opart + p * DC + quarter * 128) + lane);
            sum += wgt;
            acc.x = fmaf(wgt, x.x, acc.x);
            acc.y = fmaf(wgt, x.y, acc.y);
            acc.z = fmaf(wgt, x.z, acc.z);
            acc.w = fmaf(wgt, x.w, acc.w);
        }
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), c = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *((uint2 *)(olat + rh * DC + quarter * 128) + lane) = make_uint2(*(const uint32_t *)&a, *(const uint32_t *)&c);
    if (lse && quarter == 0 && lane == 0) lse[rh] = sum > 0.0f ? mxl + logf(sum) : -INFINITY;
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
// One pair of SMs works on a unit at a time, so units come in waves of 76.  A unit costs its tiles and about
// kUnitCost tiles to start and end.  Of the chunk sizes that fill one, two, .. waves the cheapest is
// taken; no split at all competes with them.
constexpr int kUnitCost = 6, kMinChunk = 4, kMaxWaves = 4, kMaxSplits = 76;
int split_of(const Shape &s, int chunk) { return std::min(kMaxSplits, (s.tiles + chunk - 1) / chunk); }
void make_plan(const Batch &bt, int H, Plan &plan) {
    const int B = bt.st.B;
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
        const int64_t waves = (n + PAIRS - 1) / PAIRS;
        if (waves > kMaxWaves) return (double)(work + n * kUnitCost) / PAIRS + 0.5 * (chunk + kUnitCost);
        return (double)waves * (chunk + kUnitCost);
    };
    double least = cost(rows, longest);
    for (int w = 1; w <= kMaxWaves && rows <= (int64_t)w * PAIRS; ++w) {
        int lo = kMinChunk, hi = longest;  // the smallest chunk whose units fit w waves
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (units(mid) <= (int64_t)w * PAIRS) hi = mid; else lo = mid + 1;
        }
        const double c = cost(units(lo), lo);
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
    std::stable_sort(order, order + n, [&](int x, int y) { return per[x] > per[y]; });
    P.n_seq = n;
    int64_t unit = 0, part = 0;
    for (int i = 0; i < n; ++i) {
        const int b = order[i];
        const int64_t u = shape_of(bt, H, b).nt * plan.splits[b];
        P.q0[i] = bt.st.q_off[b];
        P.T[i] = bt.st.q_off[b + 1] - bt.st.q_off[b];
        P.kbase[i] = bt.st.k_base[b];
        P.first[i] = bt.st.start_pos[b];
        P.seq[i] = b;
        P.unit0[i] = (int)unit;
        P.part0[i] = (int)part;
        J.part0[b] = (int)part;
        unit += u;
        if (plan.splits[b] > 1) part += u;
    }
    P.unit0[n] = (int)unit;
    P.pt = pt;
    P.mask = mask;
    P.words = words;
    P.H = H;
    P.ld_kv = c->ld_kv;
    P.ld_pe = c->ld_pe;
    P.scale_log2 = scale == 0.0f ? 1e-30f : scale * 1.4426950408889634f;  // 0: so small that every score counts alike
    P.wait_limit = wait_limit_cycles();
    const uint64_t rows = (uint64_t)std::max<int64_t>(c->rows, 1);
    P.oob = (int)rows;
    const bool kv8 = c->dtype == DSA_E4M3;
    // Tokens that lie together: a whole tile (contiguous caches, pages of 64), or less.
    const int run = !pt.table || pt.page % TK == 0 ? TK : pt.page % 32 == 0 ? 32 : 16;
    CUtensorMap tq, tkv, tpe;
    {
        const uint64_t dims[2] = {DC, (uint64_t)N * H}, strides[1] = {DC * 2};
        const uint32_t box[2] = {64, ROWS};
        if (!make_tmap(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, qt, dims, strides, box)) return cudaErrorInvalidValue;
    }
    tkv = tpe = tq;  // e4m3: not used
    if (!kv8) {
        // latents as slabs of 64 columns (column, row, slab); rotary keys in halves of 32 columns
        const uint64_t dims[3] = {64, rows, DC / 64}, strides[2] = {(uint64_t)c->ld_kv * 2, 128};
        const uint32_t box[3] = {64, (uint32_t)run, run == TK ? 4u : 1u};
        const uint64_t pdims[2] = {DR, rows}, pstrides[1] = {(uint64_t)c->ld_pe * 2};
        const uint32_t pbox[2] = {32, (uint32_t)run};
        if (!make_tmap(&tkv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, c->kv, dims, strides, box) ||
            !make_tmap(&tpe, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c->k_pe, pdims, pstrides, pbox, CU_TENSOR_MAP_SWIZZLE_64B))
            return cudaErrorInvalidValue;
    }
    float *opart = (float *)part_ws, *lpart = (float *)((char *)part_ws + part_bytes(plan));
    auto kern = kv8 ? tree_tc_kernel<true> : tree_tc_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)(2 * unit)), dim3(THREADS), SMEM, s, tq, tkv, tpe, run, (const void *)c->kv,
                   (const float *)c->kv_scale, (const __nv_bfloat16 *)c->k_pe, (const __nv_bfloat16 *)qpe, P,
                   (__nv_bfloat16 *)olat, lse, opart, lpart);
    if (e != cudaSuccess) return e;
    note_launch(DSA_KERNEL_TREE_TC);
    if (!plan.parts) return cudaSuccess;
    J.st = bt.st;
    for (int b = 0; b < B; ++b) J.splits[b] = plan.splits[b];
    J.H = H;
    J.rows = (int64_t)N * H;
    e = launch_pdl(tree_join_kernel, dim3((unsigned)((J.rows * 4 + 7) / 8)), dim3(256), 0, s, J, (const float *)opart,
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
