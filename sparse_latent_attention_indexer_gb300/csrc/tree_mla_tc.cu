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
// head reads the same latent) times a range of its tokens, on a pair of SMs.
// The context of 128 x 512 fp32 values would fill one SM's tensor memory, so
// the pair runs every MMA together (cta_group::2, M = 128): CTA c holds rows
// 64c .. 64c+63 and leaves half of its tensor memory to three score buffers.  A row
// then lives in one SM: its softmax needs nothing from the other one.
//   * QK^T (N = 128 tokens): CTA c brings the 64 tokens 64c.. of the tile, all 576
//     columns, in 64-column slabs.
//   * PV (N = 256 columns, twice): CTA c brings columns 256c.. of all 128 tokens, in
//     chunks of 32 tokens.
//   The quarter of the tile that a CTA needs in both forms is loaded twice: L2
//   delivers 73 B/clk/SM (measured), the copy costs 16 of the 45 that the kernel
//   takes, and in exchange slabs and chunks pass through one ring of 16 KB slots in
//   the order the MMAs use them, so no operand waits in shared memory for a softmax.
//   * The MMA thread issues QK^T two tiles ahead of PV, which hides a whole
//     softmax; P (bf16) goes through two shared-memory buffers.
//   * Softmax: four warps, lane l of the tensor memory is row l % 64 and tokens
//     64 (l / 64) ..; the two halves of a row meet once per tile for its maximum.  The
//     running maximum moves (and the context is rescaled) only when a tile exceeds
//     it by more than 2^8.
//   * bf16 caches arrive by TMA; e4m3 caches are read by eight warps that hold a whole
//     tile of codes in registers, dequantise (exact in bf16) and store it swizzled.
//   * A token that some row does not see may hold anything, and 0 x NaN is NaN: the
//     V chunks of tiles with hidden tokens are loaded through registers, where
//     Inf and NaN become 0.  Scores of hidden tokens are replaced after the MMA.
// Bound by shared memory: per 128 tokens a CTA's MMAs read 240 KB (A again for every 64
// columns), copies write 139 KB and P 16 KB, 3.1K cycles at 128 B/clk against 2.2K
// of MMA.
//
// Waits are bounded; a timeout records its site in the device error word and
// both CTAs drain and exit.
#include <algorithm>

#include "tc_common.cuh"

namespace dsa {

__device__ int g_tree_tc_error = 0;

namespace {

constexpr int ROWS = 128;               // rows of a unit (MMA M, 64 per CTA)
constexpr int HR = 64;                  // rows of a CTA
constexpr int DC = 512, DR = 64;
constexpr int TK = 128;                 // tokens of a tile
constexpr int SLAB = HR * 128;          // 64 rows or tokens x 64 columns, 128-byte swizzle: 8 KB
constexpr int NQ = (DC + DR) / 64;      // slabs of a row
constexpr int SLOT = 16384;             // two K slabs, the rotary slab (half a slot), or 32 tokens x 256 columns of V
constexpr int K_SLOTS = 5, V_SLOTS = 4; // slots of a tile
constexpr int VCH = TK / V_SLOTS;       // tokens of a V chunk
constexpr int VSLAB = VCH * 128;        // 64 columns of a V chunk
constexpr int NSLOT = 7;
constexpr int P_BYTES = HR * TK * 2;
constexpr int AHEAD = 2;                // tiles that QK^T runs ahead of PV
constexpr int NS = AHEAD + 1;           // score buffers
constexpr int NMASK = 8;
constexpr uint32_t COL_O = 0, COL_S = 256;
constexpr uint32_t IDESC_QK = tc::instr_desc(tc::kFmtBF16, tc::kFmtBF16, ROWS, TK, 0, 0);
constexpr uint32_t IDESC_PV = tc::instr_desc(tc::kFmtBF16, tc::kFmtBF16, ROWS, 256, 0, 1);
constexpr float RESCALE_LOG2 = 8.0f;
constexpr float LN2 = 0.69314718055994530942f;
constexpr long long kAbortQuietCycles = 1LL << 18;
constexpr int PAIRS = 76;               // 152 SMs

struct Bars {
    uint64_t q_full, full[NSLOT], empty[NSLOT], go[NSLOT], s_full[NS], s_empty[NS], p_full[2], p_empty[2], mask_full[NMASK], o_done,
        drain;
};
constexpr int MISC = 2 * 128 * 4 + NMASK * 16 + (int)sizeof(Bars) + 16;
constexpr int SMEM = 1024 + NQ * SLAB + 2 * P_BYTES + NSLOT * SLOT + MISC;
static_assert(SMEM <= 232448, "shared memory per CTA");
// The epilogue stages 64 rows of the context, 16 bytes apart from a power of two, where P and the ring were.
constexpr int OUT_LD_F32 = DC * 4 + 16, OUT_LD_BF16 = DC * 2 + 16;
static_assert(HR * OUT_LD_F32 <= 2 * P_BYTES + NSLOT * SLOT, "staged context");

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
    int64_t ld_kv;
    float scale_log2;
    long long wait_limit;
};
static_assert(sizeof(TreeParams) + 5 * 128 + 128 <= 32764, "launch parameters");

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

// 16 codes x scale -> 16 bf16 (two 16-byte chunks).  `up` is 2^120 * scale / `rest`, a bf16 pair each: the scale
// goes in one factor unless 2^120 times it leaves bf16's range.
struct Scale2 {
    uint32_t up, rest;
    bool two;
};
__device__ __forceinline__ Scale2 scale2(float s) {
    Scale2 r;
    r.two = !(s <= 128.0f);  // Inf and NaN included
    const float up = r.two ? 0x1p120f : 0x1p120f * s;
    const __nv_bfloat162 u = __float2bfloat162_rn(up), v = __float2bfloat162_rn(s);
    r.up = *(const uint32_t *)&u;
    r.rest = *(const uint32_t *)&v;
    return r;
}
template <bool SCRUB>
__device__ __forceinline__ void dequant16(const uint4 &c, const Scale2 &s, uint4 (&o)[2]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        spread4(w[i], r[2 * i], r[2 * i + 1]);
        r[2 * i] = mul2(r[2 * i], s.up);
        r[2 * i + 1] = mul2(r[2 * i + 1], s.up);
    }
    if (s.two) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = mul2(r[i], s.rest);
    }
    if (SCRUB) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = finite2(r[i]);
    }
    o[0] = make_uint4(r[0], r[1], r[2], r[3]);
    o[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

// Four warps (1: softmax, 2: loading) arrive at barrier ID; returns the AND of `v` over them.
template <int ID>
__device__ __forceinline__ bool bar_and(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, %2, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "n"(ID)
        : "memory");
    return r != 0;
}

// Position of a tile's first slot in the unit's sequence of slots: step s brings K(s), then V(s - AHEAD).
__device__ __forceinline__ int k_pos(int t) { return K_SLOTS * t + V_SLOTS * max(0, t - AHEAD); }
__device__ __forceinline__ int v_pos(int t, int n) { return K_SLOTS * min(t + AHEAD + 1, n) + V_SLOTS * t; }

template <bool KV8>
struct Cfg {
    static constexpr int NLOAD = KV8 ? 8 : 4;  // loading warps
    static constexpr int ARRIVE = KV8 ? 8 : 1; // arrivals of a CTA on a full slot
    static constexpr int THREADS = 32 * (6 + NLOAD);
};

template <bool KV8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<KV8>::THREADS, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qpe,
                   const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_pe, int run,
                   const void *__restrict__ kv, const float *__restrict__ kv_scale,
                   const __grid_constant__ TreeParams P, __nv_bfloat16 *__restrict__ olat, float *__restrict__ lse,
                   float *__restrict__ opart, float *__restrict__ lpart) {
    constexpr int ARRIVE = Cfg<KV8>::ARRIVE;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *Q = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *Pb = Q + NQ * SLAB;
    uint8_t *Ring = Pb + 2 * P_BYTES;
    float *mx = (float *)(Ring + NSLOT * SLOT);              // [2][128] tile maxima, then row sums
    uint64_t *live = (uint64_t *)(mx + 256);                 // [NMASK][2] tokens whose page exists
    Bars *bar = (Bars *)(live + 2 * NMASK);
    uint32_t *tmem_slot = (uint32_t *)(bar + 1);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    __shared__ int never;
    volatile int *nv = (volatile int *)&never;
    int *err = &g_tree_tc_error;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();

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
        tc::mbar_init(&bar->q_full, 2);
        for (int i = 0; i < NSLOT; ++i) {
            tc::mbar_init(&bar->full[i], 2 * ARRIVE);
            tc::mbar_init(&bar->empty[i], 1);
            tc::mbar_init(&bar->go[i], 1);
        }
        for (int i = 0; i < NS; ++i) {
            tc::mbar_init(&bar->s_full[i], 1);
            tc::mbar_init(&bar->s_empty[i], 8);       // the softmax warps of both CTAs
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bar->p_full[i], 8);
            tc::mbar_init(&bar->p_empty[i], 1);
        }
        for (int i = 0; i < NMASK; ++i) tc::mbar_init(&bar->mask_full[i], 1);
        tc::mbar_init(&bar->o_done, 1);
        tc::mbar_init(&bar->drain, 1);
        *abort_flag = 0;
        never = 0;
        tc::fence_mbar_init();
    }
    if (warp == 5) {
        tc::tmem_alloc_pair(tmem_slot, 512);
        tc::tmem_relinquish_pair();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    tc::cluster_sync();  // both CTAs' barriers exist before any remote arrive
    const uint32_t tmem = *tmem_slot;
    pdl_wait();  // the set-up above overlapped the previous kernel; global memory only from here

    const auto leader = [&](uint64_t *p) { return tc::map_peer(tc::smem_u32(p), 0); };
    // Cache row of token s, or -1 (behind the last token, or on no page).
    const auto row_of = [&](int s) -> int64_t { return s < tokens ? cache_row(P.pt, b, kbase, s) : -1; };

    // ---- one warp's work: TMA copies of the cache ----
    // Rows of a tile's eight runs of 16 tokens, a run a lane: its cache row, -1 behind the last token, or the row past
    // the cache (read as zeros) where there is no page.
    const auto runs_of = [&](int t) {
        const int s = (t0 + t) * TK + (lane & 7) * 16;
        const int64_t r = row_of(s);
        return t >= n || s >= tokens ? -1 : r >= 0 ? (int)r : P.oob;
    };
    // `ntok` tokens from run r0 on, `parts` slabs of 64 columns from column slab x0 on.  A copy takes `run` tokens;
    // where that is all of them it takes all slabs at once.
    const auto slot_copy = [&](int pos, const CUtensorMap *map, int parts, int slab_bytes, int ntok, int rows, int r0,
                               int x0) {
        const int st = pos % NSLOT;
        const uint32_t fb = leader(&bar->full[st]), dst = tc::smem_u32(Ring + st * SLOT);
        const int each = min(run, ntok), at_once = run >= ntok ? parts : 1;
        const int copies = (ntok / each) * (parts / at_once);
        const int k = lane / (parts / at_once), j = lane - k * (parts / at_once);  // this lane's copy: tokens, slab
        const int row = __shfl_sync(0xffffffffu, rows, (r0 + k * (each / 16)) & 7);
        const bool go = lane < copies && row >= 0;
        const int some = __popc(__ballot_sync(0xffffffffu, go));
        if (lane == 0) tc::mbar_arrive_expect_tx_remote(fb, (uint32_t)(some * each * at_once * 128));
        __syncwarp();
        if (go) tc::tma_load_3d_pair(dst + j * slab_bytes + k * each * 128, map, fb, 0, row, x0 + j);
    };
    // Publishes which of tile t's tokens have a page.
    const auto put_mask = [&](int t, int rows) {
        if (!P.pt.table) return;
        const unsigned have = __ballot_sync(0xffffffffu, rows >= 0 && rows != P.oob);
        if (lane < 2) {
            uint64_t m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (have >> (4 * lane + i) & 1) m |= 0xffffull << 16 * i;
            live[2 * (t % NMASK) + lane] = m;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar->mask_full[t % NMASK]);
    };

    if (warp == 4 && n > 0) {
        // ---------------- producer: Q; of a bf16 cache K and V ----------------
        if (lane == 0) {
            const uint32_t qb = leader(&bar->q_full);
            tc::mbar_arrive_expect_tx_remote(qb, NQ * SLAB);
            const int y = (int)(seq_row0 + lrow + rank * HR);
            for (int j = 0; j < DC / 64; ++j) tc::tma_load_2d_pair(tc::smem_u32(Q + j * SLAB), &tm_q, qb, j * 64, y);
            tc::tma_load_2d_pair(tc::smem_u32(Q + (NQ - 1) * SLAB), &tm_qpe, qb, 0, y);
        }
        __syncwarp();
        // Who waits for slots waits for every one in turn: a barrier's phase can be told from its neighbours only.  So the
        // producer also waits for the slots that the loading warps fill, and hands them on.
        const auto slot_wait = [&](int pos) {
            return __all_sync(0xffffffffu, tc::mbar_wait(&bar->empty[pos % NSLOT], ((pos / NSLOT) & 1) ^ 1, abort_flag,
                                                         err, 101, P.wait_limit));
        };
        bool ok = true;
        int rows[AHEAD + 2];  // of tiles s - AHEAD .. s + 1
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) rows[i] = -1;
        rows[AHEAD] = runs_of(0);
        for (int s = 0; !KV8 && ok && s < n + AHEAD; ++s) {
            rows[AHEAD + 1] = runs_of(s + 1);
            if (s < n) {
                put_mask(s, rows[AHEAD]);
                for (int j = 0; ok && j < K_SLOTS; ++j) {
                    if (!(ok = slot_wait(k_pos(s) + j))) break;
                    if (j < K_SLOTS - 1) slot_copy(k_pos(s) + j, &tm_k, 2, SLAB, HR, rows[AHEAD], rank * 4, 2 * j);
                    else slot_copy(k_pos(s) + j, &tm_pe, 1, SLAB, HR, rows[AHEAD], rank * 4, 0);
                }
            }
            if (s >= AHEAD) {
                const int t = s - AHEAD;
                const bool pass = (t0 + t + 1) * TK > safe;  // tiles with hidden tokens: the loading warps
                for (int j = 0; ok && j < V_SLOTS; ++j) {
                    const int pos = v_pos(t, n) + j;
                    if (!(ok = slot_wait(pos))) break;
                    if (!pass) slot_copy(pos, &tm_v, 4, VSLAB, VCH, rows[0], 2 * j, rank * 4);
                    else if (lane == 0) tc::mbar_arrive(&bar->go[pos % NSLOT]);
                }
            }
#pragma unroll
            for (int i = 0; i <= AHEAD; ++i) rows[i] = rows[i + 1];
        }
    } else if (warp == 5 && rank == 0 && lane == 0 && n > 0) {
        // ---------------- MMA issuer (of the pair) ----------------
        // Descriptors are a base plus (bytes >> 4): the issuing thread has little time between MMAs.
        const uint64_t qd = tc::smem_desc(tc::smem_u32(Q), 16, 1024), pd = tc::smem_desc(tc::smem_u32(Pb), 16, 1024);
        const uint64_t kd = tc::smem_desc(tc::smem_u32(Ring), 16, 1024), vd = tc::smem_desc(tc::smem_u32(Ring), VSLAB, 1024);
        const uint16_t both = 3;
        bool ok = tc::mbar_wait(&bar->q_full, 0, abort_flag, err, 102, P.wait_limit);
        int st = 0;
        uint32_t ring_ph = 0;
        const auto slot_ready = [&]() {
            const bool r = tc::mbar_wait(&bar->full[st], ring_ph, abort_flag, err, 103, P.wait_limit);
            tc::tc_fence_after();
            return r;
        };
        const auto slot_used = [&]() {
            tc::mma_commit_pair(&bar->empty[st], both);
            if (++st == NSLOT) {
                st = 0;
                ring_ph ^= 1;
            }
        };
        for (int s = 0; ok && s < n + AHEAD; ++s) {
            if (s < n) {
                const int sb = s % NS;
                if (s >= NS && !(ok = tc::mbar_wait(&bar->s_empty[sb], ((s / NS) - 1) & 1, abort_flag, err, 104, P.wait_limit))) break;
                const uint32_t d = tmem + COL_S + sb * (TK / 2);
#pragma unroll
                for (int j = 0; j < K_SLOTS; ++j) {
                    if (!(ok = slot_ready())) break;
                    const uint64_t b0 = kd + (uint64_t)(uint32_t)(st * (SLOT / 16));
#pragma unroll
                    for (int i = 0; i < (j < K_SLOTS - 1 ? 8 : 4); ++i)  // slab i / 4, 16 columns each
                        tc::mma_f16_pair(d, qd + ((2 * j + (i >> 2)) * SLAB + (i & 3) * 32) / 16,
                                         b0 + ((i >> 2) * SLAB + (i & 3) * 32) / 16, IDESC_QK, (j | i) != 0);
                    slot_used();
                }
                if (!ok) break;
                tc::mma_commit_pair(&bar->s_full[sb], both);
            }
            if (s >= AHEAD) {
                const int t = s - AHEAD, pb = t & 1;
                if (!(ok = tc::mbar_wait(&bar->p_full[pb], (t >> 1) & 1, abort_flag, err, 105, P.wait_limit))) break;
                tc::tc_fence_after();
                const uint64_t a0 = pd + (uint64_t)(uint32_t)(pb * (P_BYTES / 16));
#pragma unroll
                for (int j = 0; j < V_SLOTS; ++j) {
                    if (!(ok = slot_ready())) break;
                    const uint64_t b0 = vd + (uint64_t)(uint32_t)(st * (SLOT / 16));
#pragma unroll
                    for (int i = 0; i < 2 * (VCH / 16); ++i) {  // 16 tokens i / 2, columns of half i % 2
                        const int key = j * VCH + (i >> 1) * 16;
                        tc::mma_f16_pair(tmem + COL_O + (i & 1) * 128, a0 + ((key >> 6) * SLAB + (key & 63) * 2) / 16,
                                         b0 + ((i & 1) * 2 * VSLAB + (i >> 1) * 16 * 128) / 16, IDESC_PV,
                                         (t | j | (i >> 1)) != 0);
                    }
                    slot_used();
                }
                if (!ok) break;
                tc::mma_commit_pair(&bar->p_empty[pb], both);
            }
        }
        // No MMA may still be running when the tensor memory is released, whatever stopped the loop.
        if (ok) tc::mma_commit_pair(&bar->o_done, both);
        tc::mma_commit_pair(&bar->drain, 1);
        tc::mbar_wait(&bar->drain, 0, nv, err, 106);
    } else if (warp >= 6 && n > 0) {
        // ---------------- loading warps ----------------
        const int tid = threadIdx.x - 6 * 32;
        bool ok = true;
        uint32_t turn = 0;  // bf16: phase of every slot's `go`
        const auto slot_free = [&](int pos) {
            const int st = pos % NSLOT;
            const uint32_t ph = KV8 ? ((pos / NSLOT) & 1) ^ 1 : (turn >> st) & 1u;
            turn ^= 1u << st;
            return ok = __all_sync(0xffffffffu, tc::mbar_wait(KV8 ? &bar->empty[st] : &bar->go[st], ph, abort_flag, err, 107,
                                                              P.wait_limit));
        };
        if constexpr (KV8) {
            // Thread (K): 32 columns of one of the CTA's 64 tokens; (V): 32 of its columns of one of the chunk's
            // 32 tokens.  Codes are loaded a whole tile before they are needed.
            const uint8_t *codes = (const uint8_t *)kv;
            const int k_tok = tid >> 2, k_col = (tid & 3) * 32, v_tok = tid >> 3, v_col = (tid & 7) * 32;
            uint4 kc[K_SLOTS - 1][2], vc[V_SLOTS][2];
            float ks[K_SLOTS - 1], vs[V_SLOTS];
            const auto slot_done = [&](int pos) {
                tc::fence_proxy_async_smem();  // read by the MMAs (async proxy)
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_remote(leader(&bar->full[pos % NSLOT]));
            };
            const auto fetch = [&](uint4 (&c)[2], float &sc, int64_t row, int col) {
                c[0] = c[1] = make_uint4(0, 0, 0, 0);
                sc = 0.0f;
                if (row >= 0) {
                    const uint4 *p = (const uint4 *)(codes + row * P.ld_kv + col);
                    c[0] = __ldg(p);
                    c[1] = __ldg(p + 1);
                    sc = __ldg(kv_scale + row * (DC / 128) + (col >> 7));
                }
            };
            const auto put = [&](const uint4 (&c)[2], float sc, uint8_t *dst, int tok, int col, bool scrub) {
                // columns col .. col + 31 of a slab's 64: chunks c0 .. c0 + 3 of the token's 128-byte row
                const Scale2 s2 = scale2(sc);
                const int c0 = (col & 63) >> 3;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint4 o[2];
                    if (scrub) dequant16<true>(c[i], s2, o); else dequant16<false>(c[i], s2, o);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *(uint4 *)(dst + tok * 128 + (((c0 + 2 * i + e) ^ (tok & 7)) << 4)) = o[e];
                }
            };
            // All loads of a tile's K (or V) together: the wait for one batch must not include a younger load's.
            const auto fetch_k = [&](int t) {
                const int64_t row = row_of((t0 + t) * TK + rank * HR + k_tok);
#pragma unroll
                for (int j = 0; j < K_SLOTS - 1; ++j) fetch(kc[j], ks[j], row, j * 128 + k_col);
            };
            const auto fetch_v = [&](int t) {
#pragma unroll
                for (int j = 0; j < V_SLOTS; ++j)
                    fetch(vc[j], vs[j], row_of((t0 + t) * TK + j * VCH + v_tok), rank * 256 + v_col);
            };
            fetch_k(0);
            for (int s = 0; ok && s < n + AHEAD; ++s) {
                if (s < n) {
#pragma unroll
                    for (int j = 0; j < K_SLOTS - 1; ++j) {
                        const int pos = k_pos(s) + j;
                        if (!slot_free(pos)) break;
                        put(kc[j], ks[j], Ring + (pos % NSLOT) * SLOT + (k_col >> 6) * SLAB, k_tok, k_col, false);
                        slot_done(pos);
                    }
                    // the rotary slab is bf16: one of the warps copies it
                    if (ok && slot_free(k_pos(s) + K_SLOTS - 1)) {
                        const int pos = k_pos(s) + K_SLOTS - 1;
                        if (warp == 6) {
                            const int rows = runs_of(s);
                            put_mask(s, rows);
                            slot_copy(pos, &tm_pe, 1, SLAB, HR, rows, rank * 4, 0);
                        } else if (lane == 0) {
                            tc::mbar_arrive_remote(leader(&bar->full[pos % NSLOT]));
                        }
                    }
                    if (s + 1 < n) fetch_k(s + 1);
                }
                if (s == AHEAD - 1) fetch_v(0);
                if (ok && s >= AHEAD) {
                    const int t = s - AHEAD;
                    const bool scrub = (t0 + t + 1) * TK > safe;
#pragma unroll
                    for (int j = 0; j < V_SLOTS; ++j) {
                        const int pos = v_pos(t, n) + j;
                        if (!slot_free(pos)) break;
                        put(vc[j], vs[j], Ring + (pos % NSLOT) * SLOT + (v_col >> 6) * VSLAB, v_tok, v_col, scrub);
                        slot_done(pos);
                    }
                    if (t + 1 < n) fetch_v(t + 1);
                }
            }
        } else {
            // V chunks of the tiles with hidden tokens: thread = one token, 64 of the CTA's columns.
            const __nv_bfloat16 *lat = (const __nv_bfloat16 *)kv;
            const int tok = tid >> 2, q = tid & 3;
            const int t_first = max(0, (safe / TK) - t0);  // the first tile that ends behind `safe`
            for (int t = t_first; ok && t < n; ++t)
                for (int j = 0; j < V_SLOTS; ++j) {
                    const int pos = v_pos(t, n) + j;
                    const int64_t row = row_of((t0 + t) * TK + j * VCH + tok);
                    uint4 w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[e] = row >= 0 ? __ldg((const uint4 *)(lat + row * P.ld_kv + rank * 256 + q * 64) + e)
                                        : make_uint4(0, 0, 0, 0);
                    // a warp whose wait gave up comes to the barrier all the same, and they stop together
                    if (slot_free(pos)) {
                        uint8_t *dst = Ring + (pos % NSLOT) * SLOT + q * VSLAB + tok * 128;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *(uint4 *)(dst + ((e ^ (tok & 7)) << 4)) =
                                make_uint4(finite2(w[e].x), finite2(w[e].y), finite2(w[e].z), finite2(w[e].w));
                        tc::fence_proxy_async_smem();  // read by the MMAs (async proxy)
                    }
                    if (!(ok = bar_and<2>(ok))) break;
                    if (tid == 0) tc::mbar_arrive_remote(leader(&bar->full[pos % NSLOT]));
                }
        }
    } else if (warp < 4) {
        // ---------------- softmax: thread = row r of the CTA's 64, tokens 64 hh .. of the tile's 128 ----------------
        const unsigned FULL = 0xffffffffu;
        const int r = threadIdx.x & 63, hh = threadIdx.x >> 6;
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const int li = lrow + (int)rank * HR + r;      // row within the sequence
        const bool mine = li < seq_rows;               // else a row of the next sequence, or none
        const int node = mine ? li / P.H : 0;
        const uint64_t *bits = P.mask ? P.mask + (int64_t)(P.q0[lo] + node) * P.words : nullptr;
        const float sl2 = fabsf(P.scale_log2);         // not 0
        const bool negative = P.scale_log2 < 0.0f;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int t = 0; t < n; ++t) {
            const int sb = t % NS;
            const int kb = (t0 + t) * TK + hh * 64;    // this thread's first token
            // --- which of its 64 tokens the row sees ---
            uint64_t see = ~0ull;
            if ((t0 + t + 1) * TK > safe) {
                const int rel = kb - first;            // node number of the first token (negative: before the tree)
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
                if (!mine) see &= 1;                   // any row will do that is computed and not stored
            }
            // A warp whose wait gave up goes on to the barrier below, where all four warps stop together.
            if (P.pt.table) {
                ok = ok && tc::mbar_wait(&bar->mask_full[t % NMASK], (t / NMASK) & 1, abort_flag, err, 108, P.wait_limit);
                see &= live[2 * (t % NMASK) + hh];
            }
            ok = ok && tc::mbar_wait(&bar->s_full[sb], (t / NS) & 1, abort_flag, err, 109, P.wait_limit);
            ok = __all_sync(FULL, ok);
            tc::tc_fence_after();
            float v[64];
            {
                float a[32], c[32];
                tc::tmem_ld32(lanes + COL_S + sb * (TK / 2), a);
                tc::tmem_ld32(lanes + COL_S + sb * (TK / 2) + 32, c);
                tc::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    v[j] = a[j];
                    v[32 + j] = c[j];
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_remote(leader(&bar->s_empty[sb]));
            if (negative) {
#pragma unroll
                for (int j = 0; j < 64; ++j) v[j] = -v[j];
            }
            if (!__all_sync(FULL, see == ~0ull)) {
                const uint32_t s0 = (uint32_t)see, s1 = (uint32_t)(see >> 32);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (!(s0 >> j & 1)) v[j] = -INFINITY;
                    if (!(s1 >> j & 1)) v[32 + j] = -INFINITY;
                }
            }
            // --- the row's maximum: a tree over the 64 values, then the other half's ---
            float mt;
            {
                float a[22], b8[8];
#pragma unroll
                for (int i = 0; i < 21; ++i) a[i] = tc::max3(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
                a[21] = v[63];
#pragma unroll
                for (int i = 0; i < 7; ++i) b8[i] = tc::max3(a[3 * i], a[3 * i + 1], a[3 * i + 2]);
                b8[7] = a[21];
                mt = tc::max3(tc::max3(b8[0], b8[1], b8[2]), tc::max3(b8[3], b8[4], b8[5]), fmaxf(b8[6], b8[7]));
            }
            float *ex = mx + (t & 1) * 128;
            ex[threadIdx.x] = mt;
            if (!(ok = bar_and<1>(ok))) break;
            mt = fmaxf(mt, ex[threadIdx.x ^ 64]) * sl2;
            float m_new = m;
            bool rescale = false;
            if (mt != -INFINITY) {
                if (m == -INFINITY) {
                    m_new = mt;
                } else if (mt > m + RESCALE_LOG2) {
                    m_new = mt;
                    rescale = true;
                }
            }
            if (__any_sync(FULL, rescale)) {
                // after PV(t-1), before PV(t); tcgen05.ld/st are warp-wide: rows that stay take a factor of 1
                const float alpha = rescale ? tc::ex2_approx(m - m_new) : 1.0f;
                l *= alpha;
                ok = __all_sync(FULL, tc::mbar_wait(&bar->p_empty[(t - 1) & 1], ((t - 1) >> 1) & 1, abort_flag, err,
                                                            110, P.wait_limit));
                if (!ok) continue;
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
            m = m_new;
            // --- probabilities, rounded to bf16 for the PV product; the row sum takes the rounded ones ---
            const float neg = m == -INFINITY ? 0.0f : -m;
            uint32_t pk[32];
            float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float p0 = tc::ex2_approx(fmaf(v[2 * j], sl2, neg));
                const float p1 = tc::ex2_approx(fmaf(v[2 * j + 1], sl2, neg));
                const __nv_bfloat162 t2 = __floats2bfloat162_rn(p0, p1);
                pk[j] = *(const uint32_t *)&t2;
                sum0 = tc::add_bf16_f32((uint16_t)(pk[j] & 0xffffu), sum0);
                sum1 = tc::add_bf16_f32((uint16_t)(pk[j] >> 16), sum1);
            }
            l += sum0 + sum1;
            if (t >= 2) {
                ok = __all_sync(FULL, tc::mbar_wait(&bar->p_empty[t & 1], ((t >> 1) - 1) & 1, abort_flag, err, 111,
                                                            P.wait_limit));
                if (!ok) continue;
            }
            uint8_t *prow = Pb + (t & 1) * P_BYTES + hh * SLAB + r * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                *(uint4 *)(prow + ((c ^ (r & 7)) << 4)) = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
            tc::fence_proxy_async_smem();  // read by the PV product (async proxy)
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_remote(leader(&bar->p_full[t & 1]));
        }
        // ---------------- epilogue: normalise, stage rows in shared memory, write whole rows ----------------
        const bool have = __all_sync(FULL, n > 0 && ok && tc::mbar_wait(&bar->o_done, 0, abort_flag, err, 112, P.wait_limit));
        asm volatile("bar.sync 1, 128;" ::: "memory");
        mx[threadIdx.x] = l;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const float sum = have ? l + mx[threadIdx.x ^ 64] : 0.0f;
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        const float row_lse = sum > 0.0f ? (m + log2f(sum)) * LN2 : -INFINITY;
        if (have) tc::tc_fence_after();
        const bool whole = splits == 1;
        const int ld = whole ? OUT_LD_BF16 : OUT_LD_F32;
        uint8_t *srow = Pb + r * ld + hh * 256 * (whole ? 2 : 4);
#pragma unroll 1
        for (int cc = 0; cc < 8; ++cc) {
            float o[32];
            if (have) {
                tc::tmem_ld32(lanes + COL_O + cc * 32, o);
                tc::tmem_ld_wait();
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = have && sum > 0.0f ? o[j] * inv : 0.0f;
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
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const int64_t part = splits == 1 ? 0 : (int64_t)P.part0[lo] + rem;
        const int rows = min(HR, seq_rows - lrow - (int)rank * HR);  // of this CTA; may be <= 0
        for (int i = warp; i < rows; i += 4) {
            const uint4 *src = (const uint4 *)(Pb + i * ld);
            uint4 *dst = whole ? (uint4 *)(olat + (seq_row0 + lrow + rank * HR + i) * DC)
                               : (uint4 *)(opart + (part * ROWS + rank * HR + i) * DC);
            for (int c = lane; c < (whole ? DC / 8 : DC / 4); c += 32) dst[c] = src[c];
        }
        if (hh == 0 && mine) {
            if (!whole) lpart[part * ROWS + rank * HR + r] = row_lse;
            else if (lse) lse[seq_row0 + li] = row_lse;
        }
    }
    __syncthreads();
    if (*abort_flag) {
        // copies that nobody waits for any more land within microseconds
        const long long c0 = clock64();
        while (clock64() - c0 < kAbortQuietCycles) {
        }
    }
    tc::cluster_sync();  // the other CTA's MMAs, copies and arrivals are done with this CTA's memory
    if (warp == 5) {
        tc::tc_fence_after();
        tc::tmem_dealloc_pair(tmem, 512);
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
constexpr int kUnitCost = 3, kMinChunk = 2, kMaxWaves = 4, kMaxSplits = 76;
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
    P.scale_log2 = scale == 0.0f ? 1e-30f : scale * 1.4426950408889634f;  // 0: so small that every score counts alike
    P.wait_limit = wait_limit_cycles();
    const uint64_t rows = (uint64_t)std::max<int64_t>(c->rows, 1);
    P.oob = (int)rows;
    const bool kv8 = c->dtype == DSA_E4M3;
    // Tokens that lie together: all of a K slot's 64 (contiguous caches, pages of 64), or fewer.
    const int run = !pt.table || pt.page % 64 == 0 ? 64 : pt.page % 32 == 0 ? 32 : 16;
    CUtensorMap tq, tqpe, tk, tv, tpe;
    const auto map2 = [](CUtensorMap *m, const void *base, int cols, uint64_t n_rows) {
        const uint64_t dims[2] = {(uint64_t)cols, n_rows}, strides[1] = {(uint64_t)cols * 2};
        const uint32_t bx[2] = {64, HR};
        return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, bx);
    };
    // Cache rows as slabs of 64 columns: (column, row, slab).
    const auto map3 = [&](CUtensorMap *m, const void *base, int cols, int64_t ld, int box_rows, int box_slabs) {
        const uint64_t dims[3] = {64, rows, (uint64_t)cols / 64}, strides[2] = {(uint64_t)ld * 2, 128};
        const uint32_t bx[3] = {64, (uint32_t)box_rows, (uint32_t)box_slabs};
        return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, bx);
    };
    if (!map2(&tq, qt, DC, (uint64_t)N * H) || !map2(&tqpe, qpe, DR, (uint64_t)N * H) ||
        !map3(&tpe, c->k_pe, DR, c->ld_pe, run, 1))
        return cudaErrorInvalidValue;
    if (kv8) tk = tv = tpe;  // not used
    else if (!map3(&tk, c->kv, DC, c->ld_kv, run, run == HR ? 2 : 1) ||
             !map3(&tv, c->kv, DC, c->ld_kv, std::min(run, VCH), run >= VCH ? 4 : 1))
        return cudaErrorInvalidValue;
    float *opart = (float *)part_ws, *lpart = (float *)((char *)part_ws + part_bytes(plan));
    auto kern = kv8 ? tree_tc_kernel<true> : tree_tc_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)(2 * unit)), dim3(kv8 ? Cfg<true>::THREADS : Cfg<false>::THREADS), SMEM, s, tq,
                   tqpe, tk, tv, tpe, run, (const void *)c->kv, (const float *)c->kv_scale, P, (__nv_bfloat16 *)olat, lse,
                   opart, lpart);
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
