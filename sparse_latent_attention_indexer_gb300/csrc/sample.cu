// The next token of a row of logits: temperature, top-k, top-p, min-p and the draw, from a given
// random number.
//
// Every rule keeps a run from the start of one order, falling logit and rising index, so a row's
// kept set is one bound in that order, and min-p a bound on the weight.  An order of 50-bit
// numbers stands for it: c = ~(logit as an ordered integer) << 18 | index, lower is better.
//
// Which token is drawn hangs on comparisons of sums of up to 262,144 weights, so sums are exact:
// a weight 2^-y, y = (max - l) log2(e) / T, is a whole number of steps of 2^-45, worked out from
// pairs of fp32 values (fp64 units are few on this GPU: 2 results a cycle an SM against 128).
// Integer sums do not depend on their order, which lets threads, CTAs and atomics add as they come.
//
// A cluster of up to 8 CTAs keeps a row in shared memory, so HBM is read once.  Bounds are found
// by histograms of 512 bins (counts, or weights): first over the weight's logarithm, which spreads
// logits evenly, then over c between the least and the greatest value left in the bin, until one
// token is left; ties end in the index, so they need no rule of their own.  Every CTA adds up all
// CTAs' histograms and takes the same decision.
#include <algorithm>

#include "dsa_common.cuh"
#include "tc_common.cuh"

namespace dsa {
namespace {

typedef unsigned long long u64;

constexpr int THREADS = 512, WARPS = THREADS / 32, BINS = THREADS;
constexpr int MAX_V = 1 << 18, INDEX_BITS = 18;
constexpr int MAX_SHARE = 8;
constexpr int FEW = 2 * THREADS, LIST = 128;  // candidates that one CTA finishes; that a warp lists
constexpr u64 NONE = ~0ull, ONE = 1ull << 45;
constexpr float LN2_H = 0.693147182464599609375f, LN2_L = -1.90465429995776765e-9f;  // ln 2 as a pair

struct SampleParams {
    const void *logits;
    int64_t ld;
    int V, slice, share;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *token, *kept;
    float *logprob;
};

// 2^(-j/512) as pairs of fp32 values, from the nine roots of two that make up an exponent of nine bits.
struct Roots {
    float hi[512], lo[512];
};
constexpr Roots make_roots() {
    constexpr double root[9] = {0.9986471128909701735881, 0.9972960560854701262576, 0.9945994234836331756524, 0.9892280131939754841291, 0.9785720620877001345091, 0.9576032806985736469363, 0.9170040432046712317435, 0.8408964152537145430311, 0.7071067811865475244008};
    Roots r{};
    for (int j = 0; j < 512; ++j) {
        double v = 1.0;
        for (int b = 0; b < 9; ++b)
            if (j >> b & 1) v *= root[b];
        r.hi[j] = (float)v;
        r.lo[j] = (float)(v - (double)r.hi[j]);
    }
    return r;
}
__device__ const Roots kRoots = make_roots();

struct alignas(16) Shared {
    u64 hist[2][BINS];           // finish_few: the sorted candidates
    u64 few[FEW];                // candidates of all CTAs, in the cluster's first
    u64 list[WARPS][LIST];       // a warp's candidates, by index
    float2 root[512];
    u64 warp_sum[WARPS], warp_two[WARPS];
    u64 best, low, high, sum;    // what the other CTAs read
    int count;
    u64 pick_base;               // of the bin that holds the bound
    int pick_bin;
    float ch, cl, yh, yl;        // log2(e) / T, -log2(min_p)
};

__device__ __forceinline__ u64 peer_u64(const u64 *p, int rank) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(tc::map_peer(tc::smem_u32(p), rank)) : "memory");
    return v;
}
// Into the cluster's first CTA.
__device__ __forceinline__ void push_u64(const u64 *p, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(tc::map_peer(tc::smem_u32(p), 0)), "l"(v) : "memory");
}
__device__ __forceinline__ int peer_int(const int *p, int rank) {
    int v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(tc::map_peer(tc::smem_u32(p), rank)) : "memory");
    return v;
}

// Every thread of the cluster, with what they have written to shared memory.
__device__ __forceinline__ void meet() {
    __syncwarp();
    tc::cluster_sync();
}

__device__ __forceinline__ u64 order_of(float l, int index) { return (u64)~ordered_key(l) << INDEX_BITS | (unsigned)index; }
__device__ __forceinline__ float logit_of(u64 c) {
    const uint32_t k = ~(uint32_t)(c >> INDEX_BITS);
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// y = (top - l) log2(e) / T as a pair; false where the weight is below 2^-45 and counts as nothing.
__device__ __forceinline__ bool exponent(float top, float l, float ch, float cl, float &yh, float &yl) {
    const float d = __fsub_rn(top, l), b = __fsub_rn(d, top);  // the exact difference is d + e
    const float e = __fsub_rn(__fsub_rn(top, __fsub_rn(d, b)), __fadd_rn(l, b));
    yh = __fmul_rn(d, ch);
    if (!(d < INFINITY) || !(yh < 46.0f)) return false;
    yl = fmaf(d, cl, fmaf(e, ch, fmaf(d, ch, -yh)));
    return true;
}
// 2^-y in steps of 2^-45, y = yh + yl in [0, 46].  With k = round(512 yh), k = 512 n + j, and what is left, r (exact)
// and yl, 2^-y = 2^-n 2^-(j/512) (1 - p + p^2/2 - p^3/6), p = (r + yl) ln 2 < 2^-10.5; every term is kept to 2^-44 or better:
// the two large ones as integers on a grid of 2^-24 and 2^-32, the rest, below 2^-21, on one of 2^-43.
__device__ __forceinline__ u64 weight(float yh, float yl, const float2 *root) {
    const float magic = 12582912.0f;  // 1.5 2^23: adding it rounds to a whole number
    const float kf = fmaf(yh, 512.0f, magic);
    const int k = __float_as_int(kf) - __float_as_int(magic);
    const float r = fmaf(__fsub_rn(kf, magic), -1.0f / 512.0f, yh);
    const float2 t = root[k & 511];
    const float rh = __fadd_rn(r, yl), rb = __fsub_rn(rh, r);
    const float rl = __fadd_rn(__fsub_rn(r, __fsub_rn(rh, rb)), __fsub_rn(yl, rb));  // r + yl = rh + rl
    const float ph = __fmul_rn(rh, LN2_H);
    const float pl = fmaf(rl, LN2_H, fmaf(rh, LN2_L, fmaf(rh, LN2_H, -ph)));
    const float p = ph + pl;
    const float q = p * p * fmaf(p, -1.0f / 6.0f, 0.5f);
    const float a = __fmul_rn(t.x, ph);               // the first-order term, a + b
    const float b = fmaf(t.x, ph, -a);
    float s = fmaf(t.x, q - pl, -b);
    s = __fadd_rn(s, fmaf(-t.y, ph, t.y));            // the root's second half
    const float ma = 1.5f / 512.0f;                   // ulp 2^-32
    const float ra = __fadd_rn(a, ma);
    const int ia = __float_as_int(ra) - __float_as_int(ma);
    s = __fsub_rn(s, __fsub_rn(a, __fsub_rn(ra, ma)));
    const float ms = 1.5f / 1048576.0f;               // ulp 2^-43
    const int is = __float_as_int(__fadd_rn(s, ms)) - __float_as_int(ms);
    const int ih = __float_as_int(t.x) - 0x3e800000;  // t.x 2^24, t.x in (1/2, 1]
    const long long w = ((long long)ih << 19) - ((long long)ia << 11) + is;  // in steps of 2^-43
    const int n = k >> 9;
    // to the nearest step: many small weights that are all cut off would shift the sum
    return n <= 2 ? (u64)w << (2 - n) : ((u64)w + (1ull << (n - 3))) >> (n - 2);
}

// floor(f w), or the next whole number where it is not whole: f in [0, 1), w < 2^63.
__device__ __forceinline__ u64 part_of(float f, u64 w, bool ceil) {
    const uint32_t bits = __float_as_uint(f);
    const int e = 150 - (int)(bits >> 23);            // f = m 2^-e
    if (!(f > 0.0f)) return 0;
    if ((bits >> 23) == 0) return ceil ? 1 : 0;       // below 2^-126
    const u64 m = (bits & 0x7fffffu) | 0x800000u, lo = m * w, hi = __umul64hi(m, w);
    u64 v, rest;
    if (e < 64) {                                     // e >= 24, hi < 2^23
        v = hi << (64 - e) | lo >> e;
        rest = lo & ((1ull << e) - 1);
    } else {
        v = e - 64 < 64 ? hi >> (e - 64) : 0;
        rest = lo | (e - 64 < 64 ? hi & ((1ull << (e - 64)) - 1) : hi);
    }
    return v + (ceil && rest ? 1 : 0);
}

__device__ __forceinline__ u64 warp_min(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 a = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += a;
    }
    return v;
}

struct Row {
    const float *l;        // the CTA's logits
    int first, n;          // index of the first, how many
    int rank, share;
    float top, ch, cl, bins;  // bins: level-1 bins per unit of logit
};

// Bin of the first level: falls with the logit, the same for equal ones.
__device__ __forceinline__ int first_bin(const Row &R, float l) {
    const float x = (R.top - l) * R.bins;
    return x >= (float)(BINS - 1) ? BINS - 1 : (int)x;
}

// A bin of a histogram: its number, what lies before it, and the whole.
struct Pick {
    int bin;
    u64 base, all;
};

// Adds the cluster's histograms up and finds the bin in which the sum from `base` on reaches the target: `want`, or with
// SHARE the share p of the whole.  Every thread of every CTA gets the same answer; no such bin (bin -1): all <= want.
template <bool SHARE>
__device__ Pick pick_bin(const Row &R, Shared &S, const u64 *hist, u64 base, u64 want, float p) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    meet();
    u64 mine = 0;
    for (int r = 0; r < R.share; ++r) mine += peer_u64(&hist[tid], r);
    u64 sum = warp_scan(mine, lane);
    if (lane == 31) S.warp_sum[warp] = sum;
    if (tid == 0) S.pick_bin = -1;
    __syncthreads();
    u64 before = base, all = 0;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += S.warp_sum[w];
        all += S.warp_sum[w];
    }
    sum += before;
    const u64 target = SHARE ? max(part_of(p, all, true), 1ull) : want;
    if (sum >= target && sum - mine < target) {
        S.pick_bin = tid;
        S.pick_base = sum - mine;
    }
    __syncthreads();
    return {S.pick_bin, S.pick_base, all};
}

// First level: counts or weights of the tokens with c <= bound.
template <bool WEIGHT>
__device__ Pick first_level(const Row &R, Shared &S, u64 bound, u64 want, float p, int &turn) {
    u64 *hist = S.hist[turn];
    turn ^= 1;  // the other CTAs may still read this one after the next level's meeting; the one after clears it
    hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < R.n; i += THREADS) {
        const float l = R.l[i];
        if (!(l > -INFINITY) || (bound != NONE && order_of(l, R.first + i) > bound)) continue;
        if (WEIGHT) {
            float yh, yl;
            if (!exponent(R.top, l, R.ch, R.cl, yh, yl)) continue;
            const u64 w = weight(yh, yl, S.root);
            if (w) atomicAdd(&hist[first_bin(R, l)], w);
        } else {
            atomicAdd((unsigned *)&hist[first_bin(R, l)], 1u);
        }
    }
    return pick_bin<WEIGHT>(R, S, hist, 0, want, p);
}

// From the first level's bin on to one token: the last of the shortest run whose count (or weight) reaches the target.
template <bool WEIGHT>
__device__ u64 refine(const Row &R, Shared &S, u64 bound, Pick at, u64 target, int &turn) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    u64 low = 0, high = NONE;
    int shift = -1;  // -1: `at` is the first level's bin
    for (;;) {
        // the least and the greatest c of the bin
        u64 lo = NONE, hi = NONE;  // hi: of ~c
        for (int i = tid; i < R.n; i += THREADS) {
            const float l = R.l[i];
            if (!(l > -INFINITY)) continue;
            if (shift < 0 && first_bin(R, l) != at.bin) continue;
            const u64 c = order_of(l, R.first + i);
            if (c > bound || c < low || c > high) continue;
            if (shift >= 0 && (int)((c - low) >> shift) != at.bin) continue;
            lo = min(lo, c);
            hi = min(hi, ~c);
        }
        lo = warp_min(lo);
        hi = warp_min(hi);
        __syncthreads();
        if (lane == 0) {
            S.warp_sum[warp] = lo;
            S.warp_two[warp] = hi;
        }
        __syncthreads();
        if (warp == 0) {
            lo = warp_min(lane < WARPS ? S.warp_sum[lane] : NONE);
            hi = warp_min(lane < WARPS ? S.warp_two[lane] : NONE);
            if (lane == 0) {
                S.low = lo;
                S.high = hi;
            }
        }
        meet();
        low = high = NONE;
        for (int r = 0; r < R.share; ++r) {
            low = min(low, peer_u64(&S.low, r));
            high = min(high, peer_u64(&S.high, r));
        }
        high = ~high;
        if (low >= high) return low;
        shift = max(0, 64 - __clzll((long long)(high - low)) - 9);
        u64 *hist = S.hist[turn];
        turn ^= 1;
        hist[tid] = 0;
        __syncthreads();
        for (int i = tid; i < R.n; i += THREADS) {
            const float l = R.l[i];
            if (!(l > -INFINITY)) continue;
            const u64 c = order_of(l, R.first + i);
            if (c > bound || c < low || c > high) continue;
            if (WEIGHT) {
                float yh, yl;
                if (!exponent(R.top, l, R.ch, R.cl, yh, yl)) continue;
                const u64 w = weight(yh, yl, S.root);
                if (w) atomicAdd(&hist[(c - low) >> shift], w);
            } else {
                atomicAdd((unsigned *)&hist[(c - low) >> shift], 1u);
            }
        }
        at = pick_bin<false>(R, S, hist, at.base, target, 0.0f);
    }
}

// Sum of v over the threads before this one and itself, and over all.
__device__ __forceinline__ u64 block_scan(Shared &S, u64 v, u64 &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_scan(v, lane);
    __syncthreads();
    if (lane == 31) S.warp_sum[warp] = v;
    __syncthreads();
    u64 before = 0;
    all = 0;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += S.warp_sum[w];
        all += S.warp_sum[w];
    }
    return before + v;
}

__device__ __forceinline__ void write_token(const SampleParams &P, int64_t row, int token, float yh, float yl, u64 all, int kept) {
    P.token[row] = token;
    // both terms are of one sign: nothing cancels
    if (P.logprob) P.logprob[row] = -(fmaf(yh, LN2_H, yl * LN2_H) + log1pf((float)(all - ONE) * (1.0f / (float)ONE)));
    if (P.kept) P.kept[row] = kept;
}

// The end of a row whose kept tokens are among n <= FEW candidates, which lie in S.few by index: one CTA sorts them,
// cuts the run by each rule and draws.  all: what every token weighs, where there is no top-k.
__device__ void finish_few(const SampleParams &P, const Row &R, Shared &S, int64_t row, int n, int k, float p, float m, u64 all) {
    const int tid = threadIdx.x;
    u64 *sorted = S.hist[0];
    int size = 32;
    while (size < n) size *= 2;
    for (int i = tid; i < size; i += THREADS) sorted[i] = i < n ? S.few[i] : NONE;
    for (int len = 2; len <= size; len *= 2)
        for (int d = len / 2; d > 0; d /= 2) {
            __syncthreads();
            if (tid < size / 2) {
                const int i = 2 * tid - (tid & (d - 1)), j = i + d;
                const u64 a = sorted[i], b = sorted[j];
                if ((a > b) == ((i & len) == 0)) {
                    sorted[i] = b;
                    sorted[j] = a;
                }
            }
        }
    if (tid == 0) S.count = 0x7fffffff;
    __syncthreads();
    const int run = k > 0 ? min(k, n) : n;
    // two neighbours a thread
    u64 w[2] = {0, 0};
    bool under[2] = {false, false};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * tid + e;
        if (i >= run) continue;
        float yh, yl;
        const bool some = exponent(R.top, logit_of(sorted[i]), R.ch, R.cl, yh, yl);
        if (some) w[e] = weight(yh, yl, S.root);
        under[e] = m > 0.0f && i > 0 && !(some ? (yh - S.yh) + (yl - S.yl) <= 0.0f : yh <= S.yh);
    }
    u64 total, cum = block_scan(S, w[0] + w[1], total);
    if (k <= 0) total = all;
    const u64 target = p < 1.0f ? max(part_of(p, total, true), 1ull) : NONE;
    int keep = run;
    if (under[1]) keep = min(keep, 2 * tid + 1);
    if (under[0]) keep = min(keep, 2 * tid);
    if (cum >= target) keep = min(keep, 2 * tid + 2);
    if (cum - w[1] >= target) keep = min(keep, 2 * tid + 1);
    if (keep < run) atomicMin(&S.count, keep);
    __syncthreads();
    keep = min(run, S.count);
    const u64 bound = sorted[keep - 1];
    float yh[2], yl[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * tid + e;
        w[e] = 0;
        yh[e] = yl[e] = 0.0f;
        if (i < n && S.few[i] <= bound && exponent(R.top, logit_of(S.few[i]), R.ch, R.cl, yh[e], yl[e])) w[e] = weight(yh[e], yl[e], S.root);
    }
    cum = block_scan(S, w[0] + w[1], total);
    float u = __ldg(P.u + row);
    u = u > 0.0f ? fminf(u, 0.99999994f) : 0.0f;
    const u64 at = part_of(u, total, false);
    if (cum > at && cum - w[0] - w[1] <= at) {
        const int e = cum - w[1] > at ? 0 : 1;
        write_token(P, row, (int)(S.few[2 * tid + e] & (MAX_V - 1)), yh[e], yl[e], total, keep);
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS, 2) sample_kernel(const __grid_constant__ SampleParams P) {
    extern __shared__ __align__(16) uint8_t dynamic[];
    Shared &S = *(Shared *)dynamic;
    float *logits = (float *)(dynamic + sizeof(Shared));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)tc::cluster_rank();
    const int64_t row = blockIdx.x / P.share;
    Row R;
    R.l = logits;
    R.rank = rank;
    R.share = P.share;
    R.first = min(P.V, rank * P.slice);
    R.n = min(P.V, R.first + P.slice) - R.first;

    const float T_ = P.temperature ? __ldg(P.temperature + row) : 1.0f;
    const bool greedy = !((double)T_ >= 1e-5);
    const float p = P.top_p ? __ldg(P.top_p + row) : 1.0f, m = P.min_p ? __ldg(P.min_p + row) : 0.0f;
    const int k = greedy ? 1 : P.top_k ? __ldg(P.top_k + row) : 0;
    if (tid == THREADS - 1 && !greedy) {
        const double c = 1.4426950408889634074 / (double)T_;
        S.ch = (float)c;
        S.cl = (float)(c - (double)S.ch);
        const double y = m > 0.0f ? -log2((double)m) : 0.0;
        S.yh = (float)y;
        S.yl = (float)(y - (double)S.yh);
    }
    for (int j = tid; j < 512; j += THREADS) S.root[j] = make_float2(kRoots.hi[j], kRoots.lo[j]);

    // ---------------- the row, and the first of the order ----------------
    const T *src = (const T *)P.logits + row * P.ld + R.first;
    u64 best = NONE;
#pragma unroll 8
    for (int i = tid; i < R.n; i += THREADS) {
        float l = to_f32(src[i]);
        if (!(l > -INFINITY)) l = -INFINITY;  // NaN too
        else best = min(best, order_of(l, R.first + i));
        logits[i] = l;
    }
    best = warp_min(best);
    if (lane == 0) S.warp_sum[warp] = best;
    __syncthreads();
    if (warp == 0) {
        best = warp_min(lane < WARPS ? S.warp_sum[lane] : NONE);
        if (lane == 0) S.best = best;
    }
    meet();
    best = NONE;
    for (int r = 0; r < P.share; ++r) best = min(best, peer_u64(&S.best, r));

    const bool none = best == NONE, one = !none && k == 1;
    if (none || one) {  // the same in every thread of the cluster
        if (rank == 0 && tid == 0) {
            P.token[row] = none ? -1 : (int)(best & (MAX_V - 1));
            if (P.logprob) P.logprob[row] = none ? -INFINITY : 0.0f;
            if (P.kept) P.kept[row] = none ? 0 : 1;
        }
        meet();  // nobody leaves while the others read
        return;
    }
    R.top = logit_of(best);
    R.ch = S.ch;
    R.cl = S.cl;
    R.bins = 16.0f / T_;  // bins a sixteenth of a nat wide
    if (R.top == INFINITY) {  // the infinite ones alone, as equals
        for (int i = tid; i < R.n; i += THREADS) logits[i] = logits[i] == INFINITY ? 0.0f : -INFINITY;
        R.top = 0.0f;
        best = order_of(0.0f, (int)(best & (MAX_V - 1)));
        __syncthreads();
    }

    const int per = ((R.n + WARPS - 1) / WARPS + 31) / 32 * 32;  // a warp's tokens follow one another
    const int w0 = min(R.n, warp * per), w1 = min(R.n, w0 + per);

    // ---------------- the bound ----------------
    // One pass finds the bin in which the run ends (top-k's, else top-p's, else min-p's own); the tokens up to
    // that bin are candidates, and few of them are finished by one CTA.
    u64 bound = NONE;
    int turn = 0;
    const bool by_k = k > 0 && k < P.V, by_p = p < 1.0f, by_m = m > 0.0f;
    Pick at{-1, 0, 0};
    if (by_k) at = first_level<false>(R, S, NONE, (u64)k, 0.0f, turn);
    else if (by_p) at = first_level<true>(R, S, NONE, 0, p, turn);
    else if (by_m) at.bin = min(BINS - 1, (int)fminf(16.0f * LN2_H * S.yh + 2.0f, (float)(BINS - 1)));
    if (by_k && at.all <= (u64)k) at.bin = -1;  // fewer tokens than that: no bound
    const bool cut = at.bin >= 0;
    if (cut) {
        int n = 0;
        for (int i0 = w0; i0 < w1; i0 += 32) {
            const float l = i0 + lane < w1 ? logits[i0 + lane] : -INFINITY;
            const bool in = l > -INFINITY && first_bin(R, l) <= at.bin;
            const unsigned hit = __ballot_sync(0xffffffffu, in);
            const int to = n + __popc(hit & ((1u << lane) - 1));
            if (in && to < LIST) S.list[warp][to] = order_of(l, R.first + i0 + lane);
            n += __popc(hit);
        }
        if (lane == 0) S.warp_two[warp] = (u64)n;
        __syncthreads();
        int before = 0, mine = 0;
        bool over = false;
        for (int w = 0; w < WARPS; ++w) {
            const int c = (int)S.warp_two[w];
            if (w < warp) before += c;
            mine += c;
            over |= c > LIST;
        }
        if (tid == 0) S.count = over ? FEW + 1 : mine;
        meet();
        int total = 0;
        for (int r = 0; r < P.share; ++r) {
            const int c = peer_int(&S.count, r);
            if (r < rank) before += c;
            total = min(FEW + 1, total + c);
        }
        if (total <= FEW) {
            for (int i = lane; i < n; i += 32) push_u64(&S.few[before + i], S.list[warp][i]);
            meet();
            if (rank == 0) finish_few(P, R, S, row, total, by_k ? k : 0, p, m, at.all);
            return;
        }
    }
    if (by_k && cut) bound = refine<false>(R, S, NONE, at, (u64)k, turn);
    if (by_p) {
        if (by_k) at = first_level<true>(R, S, bound, 0, p, turn);
        bound = refine<true>(R, S, bound, at, max(part_of(p, at.all, true), 1ull), turn);
    }

    // ---------------- the draw ----------------
    const bool floor_on = m > 0.0f;
    const float fh = S.yh, fl = S.yl;
    // weight of a kept token; kept: whether it is
    const auto take = [&](int i, bool &kept, float &yh, float &yl) -> u64 {
        const float l = logits[i];
        kept = false;
        yh = yl = 0.0f;
        if (!(l > -INFINITY)) return 0;
        const u64 c = order_of(l, R.first + i);
        if (c > bound) return 0;
        const bool some = exponent(R.top, l, R.ch, R.cl, yh, yl);
        if (floor_on && c != best && !(some ? (yh - fh) + (yl - fl) <= 0.0f : yh <= fh)) return 0;
        kept = true;
        return some ? weight(yh, yl, S.root) : 0;
    };
    u64 sum = 0;
    int count = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
        bool kept;
        float yh, yl;
        sum += take(i, kept, yh, yl);
        count += kept;
    }
    sum = warp_sum(sum);
    count = __reduce_add_sync(0xffffffffu, count);
    __syncthreads();  // the last search's warp_sum has been read
    if (lane == 0) {
        S.warp_sum[warp] = sum;
        S.warp_two[warp] = (u64)count;
    }
    __syncthreads();
    if (tid == 0) {
        u64 all = 0;
        int n = 0;
        for (int w = 0; w < WARPS; ++w) {
            all += S.warp_sum[w];
            n += (int)S.warp_two[w];
        }
        S.sum = all;
        S.count = n;
    }
    meet();
    u64 all = 0, before = 0;
    int kept_all = 0;
    for (int r = 0; r < P.share; ++r) {
        const u64 v = peer_u64(&S.sum, r);
        if (r < rank) before += v;
        all += v;
        kept_all += peer_int(&S.count, r);
    }
    float u = __ldg(P.u + row);
    u = u > 0.0f ? fminf(u, 0.99999994f) : 0.0f;
    const u64 goal = part_of(u, all, false);
    for (int w = 0; w < warp; ++w) before += S.warp_sum[w];
    if (before <= goal && goal < before + S.warp_sum[warp]) {  // the token is this warp's
        for (int i0 = w0; i0 < w1; i0 += 32) {
            bool kept = false;
            float yh = 0.0f, yl = 0.0f;
            const u64 w = i0 + lane < w1 ? take(i0 + lane, kept, yh, yl) : 0;
            const u64 upto = before + warp_scan(w, lane);
            const unsigned hit = __ballot_sync(0xffffffffu, upto > goal);
            if (hit) {
                if (lane == __ffs(hit) - 1) write_token(P, row, R.first + i0 + lane, yh, yl, all, kept_all);
                break;
            }
            before = __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    meet();  // nobody leaves while the others read
}

template <typename T>
cudaError_t launch(const SampleParams &P, int R, cudaStream_t s) {
    auto *kernel = sample_kernel<T>;
    const int smem = (int)sizeof(Shared) + P.slice * 4;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared) + MAX_V / MAX_SHARE * 4);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)R * P.share);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)P.share, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_sample(const void *logits, int64_t ld, int dtype, int R, int V, const float *u, const float *temperature,
                          const int32_t *top_k, const float *top_p, const float *min_p, int32_t *token, float *logprob,
                          int32_t *kept, void *stream) {
    reset_trace();
    if (R < 0 || V < 1) return DSA_ERR_INVALID_ARG;
    if ((dtype != DSA_F32 && dtype != DSA_BF16) || V > MAX_V || R > 0x7fffffff / MAX_SHARE) return DSA_ERR_UNSUPPORTED;
    if ((uintptr_t)logits % (dtype == DSA_F32 ? 4 : 2) || ((uintptr_t)u | (uintptr_t)temperature | (uintptr_t)top_k |
                                                           (uintptr_t)top_p | (uintptr_t)min_p | (uintptr_t)token |
                                                           (uintptr_t)logprob | (uintptr_t)kept) % 4)
        return DSA_ERR_INVALID_ARG;
    if (R == 0) return DSA_OK;
    if (!logits || !u || !token || (R > 1 && ld < 0)) return DSA_ERR_INVALID_ARG;
    SampleParams P;
    P.logits = logits;
    P.ld = R > 1 ? ld : 0;
    P.V = V;
    P.share = 1;
    while (P.share < MAX_SHARE && V > P.share * 4096) P.share *= 2;
    P.slice = ((V + P.share - 1) / P.share + 31) / 32 * 32;
    P.u = u;
    P.temperature = temperature;
    P.top_k = top_k;
    P.top_p = top_p;
    P.min_p = min_p;
    P.token = token;
    P.logprob = logprob;
    P.kept = kept;
    const cudaError_t e = dtype == DSA_F32 ? launch<float>(P, R, (cudaStream_t)stream) : launch<__nv_bfloat16>(P, R, (cudaStream_t)stream);
    if (e != cudaSuccess) return fail_cuda(e);
    note_launch(DSA_KERNEL_SAMPLE);
    return DSA_OK;
}
