// The next token of a row of logits: temperature, top-k, top-p, min-p and the draw, from a given
// random number.
//
// Every rule keeps a run from the start of one order, falling logit and rising index, so a row's
// kept set is one bound in that order.  Whole numbers of 50 bits stand for it:
// c = ~(logit as an ordered integer) << 18 | index, lower is better.
//
// Which token is drawn hangs on comparisons of sums of up to 262,144 weights, so sums are exact:
// a weight 2^-y, y = (max - l) log2(e) / T, is a whole number of steps of 2^-45, worked out from
// pairs of fp32 values (fp64 units are few on this GPU: 2 results a cycle an SM against 128).
// Integer sums do not depend on their order, which lets threads and CTAs add as they come.
//
// A cluster of up to 8 CTAs shares a row, and keeps it in shared memory (one bulk copy each) or
// finds it in L2 again, so HBM is read once.  What follows the maximum is to find few candidates
// among many tokens:
//   * top-k: the k-th largest of the threads' own maxima (a histogram of one value a thread) is
//     not above the k-th largest logit, so the tokens from there on hold the run;
//   * min-p: the tokens down to that weight;
//   * top-p: a histogram of approximate weights in bins of 1/32 of a nat, whose sums are good to
//     2^-13, finds the bin or two in which the run ends; a pass over exact weights gives the sum
//     before them and the whole.
// Up to 2048 candidates are sorted by one CTA, which cuts the run (and draws, where the candidates
// are all there is to draw from).  More of them, as many equal logits or a top_p near 1 give, go
// another way: histograms, of counts or exact weights, over ever narrower ranges of c until one
// token is left; ties end in the index, so they need no rule of their own.
//
// Bound by latency for a row (131,072 logits in fp32, replayed in a graph: highest logit 5.5 us, top-k 50 11.5, top-k 1000 19,
// top-p 0.95 32, no rule 16, of which reading takes 2: meetings of the cluster, barriers, code that runs once), by latency and
// instructions for many (256 rows: highest logit 43 us, top-k 50 59, top-k 1000 119, top-p 0.95 277, no rule 152; HBM 20).  An
// exact weight takes some 75 instructions, the rest of a pass 20.
// A row's code runs once, between other kernels from cold caches: it is kept short (loops over CTAs and steps of sorting are not
// unrolled, the end has one place), which took one row (settings drawn), among other kernels, from 28 to 18 us.
#include <algorithm>

#include "dsa_common.cuh"
#include "tc_common.cuh"

namespace dsa {

__device__ int g_sample_error = 0;

namespace {

typedef unsigned long long u64;

constexpr int THREADS = 512, WARPS = THREADS / 32, BINS = 2 * THREADS;
constexpr int MAX_V = 1 << 18, INDEX_BITS = 18;
constexpr int MAX_SHARE = 8;
constexpr int FEW = 4 * THREADS, LIST = 96;  // candidates that one CTA finishes; that a warp lists
constexpr float PER_NAT = 32.0f;              // bins
constexpr u64 NONE = ~0ull, ONE = 1ull << 45;
constexpr float LN2_H = 0.693147182464599609375f, LN2_L = -1.90465429995776765e-9f;  // ln 2 as a pair
constexpr float LOG2E = 1.44269504f;

struct SampleParams {
    const void *logits;
    int64_t ld;
    int V, slice, share;
    int order;             // rows that are put in order, the slow ones first (0: as they come)
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *token, *kept;
    float *logprob;
    long long wait_limit;
};

// 2^(-j/512) as pairs of fp32 values, from the nine roots of two that make up an exponent of nine bits.
struct Roots {
    float2 at[512];
};
constexpr Roots make_roots() {
    constexpr double root[9] = {0.9986471128909701735881, 0.9972960560854701262576, 0.9945994234836331756524, 0.9892280131939754841291, 0.9785720620877001345091, 0.9576032806985736469363, 0.9170040432046712317435, 0.8408964152537145430311, 0.7071067811865475244008};
    Roots r{};
    for (int j = 0; j < 512; ++j) {
        double v = 1.0;
        for (int b = 0; b < 9; ++b)
            if (j >> b & 1) v *= root[b];
        r.at[j].x = (float)v;
        r.at[j].y = (float)(v - (double)r.at[j].x);
    }
    return r;
}
__device__ const Roots kRoots = make_roots();

struct alignas(16) Shared {
    union {
        u64 hist[2][BINS];       // exact sums or counts
        unsigned rough[BINS];    // approximate ones
        u64 sorted[FEW];         // finish_few
    };
    u64 few[FEW];                // candidates of all CTAs, in the cluster's first
    u64 list[WARPS][LIST];       // a warp's candidates, by index
    float2 root[512];
    u64 warp_sum[WARPS], warp_two[WARPS];
    // What the other CTAs and this one have found, by rank.  A CTA may push while another still reads what the last meeting
    // brought, so what follows within one meeting has a place of its own.
    u64 in[2][MAX_SHARE], in_draw[MAX_SHARE], bound;
    int in_alone[MAX_SHARE], in_count[MAX_SHARE], in_kept[MAX_SHARE], in_first[MAX_SHARE];
    float in_top[MAX_SHARE];
    int first, picked;
    u64 pick_base;               // of the bin that holds the bound
    int pick_bin, pick_to;
    float ch, cl, yh, yl;        // log2(e) / T, -log2(min_p)
    uint64_t arrived;
    int abort_word, never;
};

// Every thread of the cluster, with what they have written to shared memory; and the same in two halves.
__device__ __forceinline__ void meet_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void meet_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void meet() {
    meet_arrive();
    meet_wait();
}
// Remote stores are sent and forgotten (meet() makes them seen), a remote load is waited for: what every CTA needs is
// pushed, and a histogram's loads are issued together.
__device__ __forceinline__ void push(const u64 *p, int rank, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(tc::map_peer(tc::smem_u32(p), rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void push(const int *p, int rank, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(tc::map_peer(tc::smem_u32(p), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void push(const float *p, int rank, float v) { push((const int *)p, rank, __float_as_int(v)); }
__device__ __forceinline__ void peer2(const u64 *p, int rank, u64 &a, u64 &b) {
    asm volatile("ld.shared::cluster.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(tc::map_peer(tc::smem_u32(p), rank)) : "memory");
}
__device__ __forceinline__ void peer2(const unsigned *p, int rank, unsigned &a, unsigned &b) {
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(tc::map_peer(tc::smem_u32(p), rank)) : "memory");
}
// This thread's two bins of all CTAs, added up as A.
template <typename A, typename T>
__device__ __forceinline__ void merge(const T *hist, int share, A &one, A &two) {
    T a[MAX_SHARE], b[MAX_SHARE];
#pragma unroll
    for (int r = 0; r < MAX_SHARE; ++r) {
        a[r] = b[r] = 0;
        if (r < share) peer2(hist + 2 * threadIdx.x, r, a[r], b[r]);
    }
    one = two = 0;
#pragma unroll
    for (int r = 0; r < MAX_SHARE; ++r) {
        one += (A)a[r];
        two += (A)b[r];
    }
}

__device__ __forceinline__ u64 order_of(float l, int index) { return (u64)~ordered_key(l) << INDEX_BITS | (unsigned)index; }
__device__ __forceinline__ float logit_of(u64 c) {
    const uint32_t k = ~(uint32_t)(c >> INDEX_BITS);
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// y = (top - l) log2(e) / T as a pair; false where the weight is below 2^-46 and counts as nothing.
__device__ __forceinline__ bool exponent(float top, float l, float ch, float cl, float &yh, float &yl) {
    const float d = __fsub_rn(top, l), b = __fsub_rn(d, top);  // the exact difference is d + e
    const float e = __fsub_rn(__fsub_rn(top, __fsub_rn(d, b)), __fadd_rn(l, b));
    yh = __fmul_rn(d, ch);
    yl = fmaf(d, cl, fmaf(e, ch, fmaf(d, ch, -yh)));
    return d < INFINITY && yh < 46.0f;
}
// Whether 2^-y is at least min_p, 2^-f (above fp32's range y is infinite, or not a number).
__device__ __forceinline__ bool passes(float yh, float yl, float fh, float fl) { return (yh - fh) + (yl - fl) <= 0.0f; }
// 2^-y in steps of 2^-45, y = yh + yl in [0, 46].  With k = round(512 yh), k = 512 n + j, and what is left, r (exact)
// and yl, 2^-y = 2^-n 2^-(j/512) (1 - p + p^2/2 - p^3/6), p = (r + yl) ln 2 < 2^-10.5; every term is kept to 2^-41 or
// better: the two large ones as integers on grids of 2^-24 and 2^-32, the rest, below 2^-18, on one of 2^-40.
__device__ __forceinline__ u64 weight(float yh, float yl, const float2 *root) {
    const float magic = 12582912.0f;  // 1.5 2^23: adding it rounds to a whole number
    const float kf = fmaf(yh, 512.0f, magic);
    const int k = __float_as_int(kf) - __float_as_int(magic);
    const float r = fmaf(__fsub_rn(kf, magic), -1.0f / 512.0f, yh);
    const float2 t = root[k & 511];
    const float ph = __fmul_rn(r, LN2_H);
    const float pl = fmaf(yl, LN2_H, fmaf(r, LN2_L, fmaf(r, LN2_H, -ph)));
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
    const float ms = 1.5f / 131072.0f;                // ulp 2^-40
    const int is = __float_as_int(__fadd_rn(s, ms)) - __float_as_int(ms);
    const int ih = __float_as_int(t.x) - 0x3e800000;  // t.x 2^24, t.x in (1/2, 1]
    const u64 w = (u64)((long long)ih * 65536 + (is - ia * 256)) << 5;
    // to the nearest step: many small weights that are all cut off would shift the sum
    return ((w << 1 >> (k >> 9)) + 1) >> 1;
}
// The weight of any logit, -inf and NaN among them.
__device__ __forceinline__ u64 weight_of(float top, float l, float ch, float cl, const float2 *root) {
    float yh, yl;
    const bool some = exponent(top, l, ch, cl, yh, yl);
    const u64 w = weight(some ? yh : 0.0f, some ? yl : 0.0f, root);
    return some ? w : 0;
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

// A CTA's part of a row, in shared memory or (not CACHED) where it lies.
template <typename T_, bool CACHED>
struct Row {
    typedef T_ T;
    const T *raw;          // the logits, as they come
    bool infinite;         // not CACHED: +inf counts as 0, all else as nothing
    int first, n;          // index of the first, how many
    int rank, share;
    float top, ch, cl, bins;  // bins: bins per unit of logit

    __device__ __forceinline__ float at(int i) const {
        const float l = to_f32(raw[i]);
        return CACHED || !infinite ? l : l == INFINITY ? 0.0f : -INFINITY;
    }
    // Bins fall with the logit; equal logits have equal ones.  A token is in bin b or before: x < b + 1.  The last bin takes all that
    // is further down, a mask of the type's lowest number too, whose product is infinite like that of -inf, which is no token.
    __device__ __forceinline__ float x(float l) const { return (top - l) * bins; }
    __device__ __forceinline__ int bin(float l) const { return (int)fminf(x(l), (float)(BINS - 1)); }
};

// Sum of v over the threads up to this one, and over all.
__device__ __forceinline__ u64 block_scan(Shared &S, u64 v, u64 &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_scan(v, lane);
    __syncthreads();
    if (lane == 31) S.warp_sum[warp] = v;
    __syncthreads();
    const u64 upto = warp_scan(lane < WARPS ? S.warp_sum[lane] : 0, lane);
    const u64 before = __shfl_sync(0xffffffffu, upto, max(0, warp - 1));
    all = __shfl_sync(0xffffffffu, upto, 31);
    return (warp > 0 ? before : 0) + v;
}

// A bin of a histogram: its number, what lies before it, and the whole.
struct Pick {
    int bin;
    u64 base, all;
};

// Adds the cluster's histograms up and finds the bin in which the sum from `base` on reaches the target: `want`, or with
// SHARE the share p of the whole.  Every thread of every CTA gets the same answer; no such bin (bin -1): all < want.
template <bool SHARE>
__device__ Pick pick_bin(int share, Shared &S, const u64 *hist, u64 base, u64 want, float p) {
    const int tid = threadIdx.x;
    meet();
    u64 one, two;
    merge(hist, share, one, two);
    if (tid == 0) S.pick_bin = -1;
    u64 all;
    const u64 sum = base + block_scan(S, one + two, all);
    const u64 target = SHARE ? max(part_of(p, all, true), 1ull) : want;
    if (sum >= target && sum - one - two < target) {
        const bool second = sum - two < target;
        S.pick_bin = 2 * tid + second;
        S.pick_base = second ? sum - two : sum - two - one;
    }
    __syncthreads();
    return {S.pick_bin, S.pick_base, all};
}

// Counts or weights of the tokens with c <= bound over the whole range.
template <bool WEIGHT, typename Part>
__device__ Pick first_level(const Part &R, Shared &S, u64 bound, u64 want, float p, int &turn) {
    u64 *hist = S.hist[turn];
    turn ^= 1;  // the other CTAs may still read this one until the next level's meeting; the level after clears it
    __syncthreads();
    for (int b = threadIdx.x; b < BINS; b += THREADS) hist[b] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < R.n; i += THREADS) {
        const float l = R.at(i);
        if (!(l > -INFINITY) || (bound != NONE && order_of(l, R.first + i) > bound)) continue;
        if (WEIGHT) {
            const u64 w = weight_of(R.top, l, R.ch, R.cl, S.root);
            if (w) atomicAdd(&hist[R.bin(l)], w);
        } else {
            atomicAdd((unsigned *)&hist[R.bin(l)], 1u);
        }
    }
    return pick_bin<WEIGHT>(R.share, S, hist, 0, want, p);
}

// From the first level's bin on to one token: the last of the shortest run whose count (or weight) reaches the target.
template <bool WEIGHT, typename Part>
__device__ u64 refine(const Part &R, Shared &S, u64 bound, Pick at, u64 target, int &turn) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    u64 low = 0, high = NONE;
    int shift = -1;  // -1: `at` is the first level's bin
    for (;;) {
        // the least and the greatest c of the bin
        u64 lo = NONE, hi = NONE;  // hi: of ~c
        for (int i = tid; i < R.n; i += THREADS) {
            const float l = R.at(i);
            if (!(l > -INFINITY)) continue;
            if (shift < 0 && R.bin(l) != at.bin) continue;
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
            if (lane < R.share) {
                push(&S.in[0][R.rank], lane, lo);
                push(&S.in[1][R.rank], lane, hi);
            }
        }
        meet();
        low = high = NONE;
#pragma unroll 1
        for (int r = 0; r < R.share; ++r) {
            low = min(low, S.in[0][r]);
            high = min(high, S.in[1][r]);
        }
        high = ~high;
        if (low >= high) return low;
        shift = max(0, 64 - __clzll((long long)(high - low)) - 10);  // (high - low) >> shift < BINS
        u64 *hist = S.hist[turn];
        turn ^= 1;
        for (int b = tid; b < BINS; b += THREADS) hist[b] = 0;
        __syncthreads();
        for (int i = tid; i < R.n; i += THREADS) {
            const float l = R.at(i);
            if (!(l > -INFINITY)) continue;
            const u64 c = order_of(l, R.first + i);
            if (c > bound || c < low || c > high) continue;
            if (WEIGHT) {
                const u64 w = weight_of(R.top, l, R.ch, R.cl, S.root);
                if (w) atomicAdd(&hist[(c - low) >> shift], w);
            } else {
                atomicAdd((unsigned *)&hist[(c - low) >> shift], 1u);
            }
        }
        at = pick_bin<false>(R.share, S, hist, at.base, target, 0.0f);
    }
}

__device__ __forceinline__ float random_of(const SampleParams &P, int64_t row) {
    const float u = __ldg(P.u + row);
    return u > 0.0f ? fminf(u, 0.99999994f) : 0.0f;
}
__device__ __forceinline__ void write_token(const SampleParams &P, int64_t row, int token, float yh, float yl, u64 all, int kept) {
    P.token[row] = token;
    // both terms are of one sign: nothing cancels
    if (P.logprob) P.logprob[row] = -(fmaf(yh, LN2_H, yl * LN2_H) + log1pf((float)(all - ONE) * (1.0f / (float)ONE)));
    if (P.kept) P.kept[row] = kept;
}

// How many tokens the CTA's warps have listed (above FEW: more than a list holds, or more than `most`), and how many of them
// come before this warp's.
__device__ __forceinline__ int count_listed(Shared &S, int listed, int most, int &before) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) S.warp_two[warp] = (u64)listed;
    __syncthreads();
    const int c = lane < WARPS ? (int)S.warp_two[lane] : 0;
    const bool over = __any_sync(0xffffffffu, c > LIST);
    before = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
    const int all = __reduce_add_sync(0xffffffffu, c);
    __syncthreads();
    return over || all > most ? FEW + 1 : all;
}

// Candidate i < n of the cluster, by index: they lie in S.few, rank r's S.in_alone[r] from region r on (0: one after another).
__device__ __forceinline__ u64 candidate(const Shared &S, int i, int n, int region, int share) {
    if (i >= n) return NONE;
    if (region == 0) return S.few[i];
    int r = 0;
#pragma unroll 1
    while (r < share - 1 && i >= S.in_alone[r]) i -= S.in_alone[r++];
    return S.few[r * region + i];
}

// The thread's share of the candidates (E neighbours, by index) becomes that of the candidates in order, best first, NONE
// behind them: one value a thread turns in registers as long as its partner is in its warp, more go through shared memory.
template <int E>
__device__ void sort_few(Shared &S, u64 (&c)[E], int n) {
    const int tid = threadIdx.x;
    int size = 32;
#pragma unroll 1
    while (size < n) size *= 2;
    if constexpr (E == 1) {
        if (tid < size) {
#pragma unroll 1
            for (int len = 2; len <= size; len *= 2)
#pragma unroll 1
                for (int d = len / 2; d > 0; d /= 2) {
                    u64 other;
                    if (d >= 32) {
                        asm volatile("bar.sync 1, %0;" ::"r"(size) : "memory");
                        S.sorted[tid] = c[0];
                        asm volatile("bar.sync 1, %0;" ::"r"(size) : "memory");
                        other = S.sorted[tid ^ d];
                    } else {
                        other = __shfl_xor_sync(0xffffffffu, c[0], d);
                    }
                    const bool low = ((tid & d) == 0) == ((tid & len) == 0);  // this thread keeps the smaller one
                    if (low ? other < c[0] : other > c[0]) c[0] = other;
                }
        }
    } else {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) S.sorted[E * tid + e] = c[e];
#pragma unroll 1
        for (int len = 2; len <= size; len *= 2)
#pragma unroll 1
            for (int d = len / 2; d > 0; d /= 2) {
                __syncthreads();
                for (int t = tid; t < size / 2; t += THREADS) {
                    const int i = 2 * t - (t & (d - 1)), j = i + d;
                    const u64 a = S.sorted[i], b = S.sorted[j];
                    if ((a > b) == ((i & len) == 0)) {
                        S.sorted[i] = b;
                        S.sorted[j] = a;
                    }
                }
            }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) c[e] = S.sorted[E * tid + e];
    }
}

// Among one CTA's candidates (E a thread, at most `bound`): the last token of the shortest run whose count (or weight w) reaches
// the target, which all of them together have to reach.  A histogram finds its bin, the bin's few tokens are sorted; many in one
// bin: all are.
template <int E, bool WEIGHT, typename Part>
__device__ u64 select_few(const Part &R, Shared &S, const u64 (&c)[E], const u64 (&w)[E], u64 bound, int n, u64 target) {
    const int tid = threadIdx.x;
    u64 *hist = S.hist[0], *some = &S.list[0][0], all;
    __syncthreads();
    for (int b = tid; b < BINS; b += THREADS) hist[b] = 0;
    if (tid == 0) S.picked = 0;
    __syncthreads();
    int bin[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        bin[e] = c[e] <= bound && c[e] != NONE ? R.bin(logit_of(c[e])) : -1;
        if (bin[e] >= 0) atomicAdd(&hist[bin[e]], WEIGHT ? w[e] : 1ull);
    }
    __syncthreads();
    const u64 one = hist[2 * tid], two = hist[2 * tid + 1], sum = block_scan(S, one + two, all);
    if (sum >= target && sum - one - two < target) {
        const bool second = sum - two < target;
        S.pick_bin = 2 * tid + second;
        S.pick_base = second ? sum - two : sum - two - one;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (bin[e] == S.pick_bin) {
            const int at = atomicAdd(&S.picked, 1);
            if (at < WARPS * LIST) some[at] = c[e];
        }
    __syncthreads();
    const int m = S.picked;
    u64 base = S.pick_base;
    const auto last = [&](auto &v, auto &of) {  // sorted values and their weights, base before them
        u64 mine = 0;
#pragma unroll
        for (const u64 &x : of) mine += x;
        u64 cum = base + block_scan(S, mine, all) - mine;
        int e = 0;
#pragma unroll
        for (const u64 &x : of) {
            if (cum < target && cum + x >= target) S.bound = v[e];
            cum += x;
            ++e;
        }
        __syncthreads();
    };
    const auto worth = [&](u64 x) { return x > bound || x == NONE ? 0ull : WEIGHT ? weight_of(R.top, logit_of(x), R.ch, R.cl, S.root) : 1ull; };
    if (m <= THREADS) {
        u64 v[1] = {tid < m ? some[tid] : NONE};
        sort_few<1>(S, v, m);
        u64 of[1] = {worth(v[0])};
        last(v, of);
    } else {
        u64 v[E], of[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = c[e];
        sort_few<E>(S, v, n);
        base = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) of[e] = worth(v[e]);
        last(v, of);
    }
    return S.bound;
}

// The end of a row whose kept tokens are among n <= E * THREADS candidates: one CTA cuts the run by each rule and draws.
// all: what every token weighs, where there is no top-k.  E = 1 sorts them, E = 4 looks for the bounds (top-k 1000 of
// 131,072: 28 us sorted, 18 so).
template <int E, typename Part>
__device__ void finish_few(const SampleParams &P, const Part &R, Shared &S, int64_t row, int n, int region, int k, float p, float m,
                           u64 all) {
    const int first = E * threadIdx.x;
    u64 by_index[E], w[E], mine = 0, total = all, bound = NONE;
    float yh[E], yl[E];
#pragma unroll
    for (int e = 0; e < E; ++e) by_index[e] = candidate(S, first + e, n, region, R.share);
    if constexpr (E == 1) {
        u64 sorted[1] = {by_index[0]};
        sort_few<1>(S, sorted, n);
        const int run = k > 0 ? min(k, n) : n;
        if (first == run - 1) S.bound = sorted[0];
        if (p < 1.0f) {
            mine = first < run ? weight_of(R.top, logit_of(sorted[0]), R.ch, R.cl, S.root) : 0;
            u64 sum, cum = block_scan(S, mine, sum);
            if (k > 0) total = sum;
            const u64 target = max(part_of(p, total, true), 1ull);
            if (cum >= target && cum - mine < target) S.bound = sorted[0];
        }
        __syncthreads();
        bound = S.bound;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        yh[e] = yl[e] = 0.0f;
        // what weighs nothing keeps its exponent, which a min-p below 2^-46 may let pass
        const bool some = by_index[e] != NONE && exponent(R.top, logit_of(by_index[e]), R.ch, R.cl, yh[e], yl[e]);
        w[e] = weight(some ? yh[e] : 0.0f, some ? yl[e] : 0.0f, S.root);
        if (!some) w[e] = 0;
    }
    if constexpr (E > 1) {
        if (k > 0 && k < n) bound = select_few<E, false>(R, S, by_index, w, NONE, n, (u64)k);
        if (p < 1.0f) {
            u64 here;
            mine = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) mine += by_index[e] <= bound ? w[e] : 0;
            block_scan(S, mine, here);
            if (k > 0) total = here;
            const u64 target = max(part_of(p, total, true), 1ull);
            // candidates by min-p may weigh less than that share of all tokens: then the run has them all and more
            if (here >= target) bound = select_few<E, true>(R, S, by_index, w, bound, n, target);
        }
    }
    int kept = 0;
    mine = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        // min-p after the others: a token that it drops counts towards their sums
        const bool in = by_index[e] <= bound && by_index[e] != NONE && (!(m > 0.0f) || passes(yh[e], yl[e], S.yh, S.yl));
        if (!in) w[e] = 0;
        kept += in;
        mine += w[e];
    }
    u64 kept_all, cum = block_scan(S, mine, total) - mine;
    block_scan(S, (u64)kept, kept_all);
    const u64 goal = part_of(random_of(P, row), total, false);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (cum <= goal && cum + w[e] > goal) write_token(P, row, (int)(by_index[e] & (MAX_V - 1)), yh[e], yl[e], total, (int)kept_all);
        cum += w[e];
    }
}

// The last token of a run by top-p that ends among n candidates: `before` is what the tokens before them weigh.
template <int E, typename Part>
__device__ void bound_few(const Part &R, Shared &S, int n, u64 before, u64 target) {
    u64 c[E], w[E], mine = 0, sum;
#pragma unroll
    for (int e = 0; e < E; ++e) c[e] = candidate(S, E * threadIdx.x + e, n, 0, R.share);
    sort_few<E>(S, c, n);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        w[e] = c[e] != NONE ? weight_of(R.top, logit_of(c[e]), R.ch, R.cl, S.root) : 0;
        mine += w[e];
    }
    u64 cum = before + block_scan(S, mine, sum) - mine;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (cum < target && cum + w[e] >= target)
#pragma unroll 1
            for (int r = 0; r < R.share; ++r) push(&S.bound, r, c[e]);
        cum += w[e];
    }
}

// The CTA's logits into shared memory, element i at raw[i]: whole 16 bytes by one bulk copy, what lies before and after
// them by itself.
template <typename T>
__device__ T *fetch_slice(Shared &S, uint8_t *room, const T *src, int n, bool &coming) {
    const int off = (int)((uintptr_t)src & 15);
    T *raw = (T *)(room + off);
    const int head = min(n, (16 - off) % 16 / (int)sizeof(T)), body = (n - head) * (int)sizeof(T) / 16 * 16;
    const int tail = head + body / (int)sizeof(T);
    coming = body > 0;
    if (threadIdx.x == 0) {
        tc::mbar_init(&S.arrived, 1);
        S.abort_word = S.never = 0;
        tc::fence_mbar_init();
        if (body) {
            tc::mbar_arrive_expect_tx(&S.arrived, body);
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             tc::smem_u32(raw + head)),
                         "l"(src + head), "r"(body), "r"(tc::smem_u32(&S.arrived))
                         : "memory");
        }
    }
    if (threadIdx.x >= 32) {
        const int i = threadIdx.x - 32;
        if (i < head) raw[i] = src[i];
        if (i < n - tail) raw[tail + i] = src[tail + i];
    }
    return raw;
}

// Waits for the CTA's bulk copy.  The phase is polled, not waited for by the hardware, whose patience is longer than a copy takes:
// so a limit that is set counts.
__device__ __forceinline__ bool wait_copy(Shared &S, volatile int *abort_flag, int site, long long limit) {
    if (tc::mbar_test(&S.arrived, 0)) return true;
    const long long t0 = clock64();
    while (!tc::mbar_test(&S.arrived, 0)) {
        if (*abort_flag) return false;
        if (clock64() - t0 > limit) {
            atomicCAS(&g_sample_error, 0, site);
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}

// This thread's maximum over its share of a CTA's logits, 16 bytes at a time: 64 KB of the CTA are on their way at once.
__device__ __forceinline__ float max_in(const uint4 &q, float m, const float *) {
    return fmaxf(fmaxf(fmaxf(m, __uint_as_float(q.x)), fmaxf(__uint_as_float(q.y), __uint_as_float(q.z))), __uint_as_float(q.w));
}
__device__ __forceinline__ float max_in(const uint4 &q, float m, const __nv_bfloat16 *) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)));
    return m;
}
template <typename T>
__device__ __forceinline__ float max_of(const T *src, int n) {
    const int off = (int)((uintptr_t)src & 15), each = 16 / (int)sizeof(T), head = min(n, (16 - off) % 16 / (int)sizeof(T));
    const int body = (n - head) / each, tail = head + body * each;
    const uint4 *p = (const uint4 *)(src + head);
    float m = -INFINITY;
    if ((int)threadIdx.x < head) m = fmaxf(m, to_f32(src[threadIdx.x]));
    if ((int)threadIdx.x < n - tail) m = fmaxf(m, to_f32(src[tail + threadIdx.x]));
#pragma unroll 8
    for (int i = threadIdx.x; i < body; i += THREADS) m = max_in(__ldg(p + i), m, (const T *)nullptr);
    return m;
}

// What a row's settings ask for.
struct Settings {
    float T, p, m;
    int k;                 // 1: the first token alone, as without a temperature, a share, or where no other token weighs enough
    bool by_k, by_p, by_m;
};
__device__ __forceinline__ Settings settings_of(const SampleParams &P, int64_t row) {
    Settings s;
    s.T = P.temperature ? __ldg(P.temperature + row) : 1.0f;
    s.p = P.top_p ? __ldg(P.top_p + row) : 1.0f;
    s.m = P.min_p ? __ldg(P.min_p + row) : 0.0f;
    s.k = P.top_k ? __ldg(P.top_k + row) : 0;
    if (!((double)s.T >= 1e-5) || s.p <= 0.0f || s.m > 1.0f) s.k = 1;
    s.by_k = s.k > 0 && s.k < P.V;
    s.by_p = s.p < 1.0f;
    s.by_m = s.m > 0.0f;
    return s;
}
// The i-th row where those come first that weigh every token (top-p without top-k): a slow row that starts last would be what
// a batch waits for (256 rows with settings of every kind: 121 -> 108 us).
__device__ __forceinline__ int slow_first(const SampleParams &P, Shared &S, int i) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = threadIdx.x;  // order <= THREADS rows
    bool slow = false;
    if (row < P.order) {
        const Settings s = settings_of(P, row);
        slow = !s.by_k && s.k != 1 && s.by_p;
    }
    const unsigned in = __ballot_sync(0xffffffffu, row < P.order), hit = __ballot_sync(0xffffffffu, slow);
    if (lane == 0) {
        S.warp_sum[warp] = __popc(hit);
        S.warp_two[warp] = __popc(in & ~hit);
    }
    __syncthreads();
    const int a = lane < WARPS ? (int)S.warp_sum[lane] : 0, b = lane < WARPS ? (int)S.warp_two[lane] : 0;
    const int slow_all = __reduce_add_sync(0xffffffffu, a);
    const int slow_before = __reduce_add_sync(0xffffffffu, lane < warp ? a : 0), fast_before = __reduce_add_sync(0xffffffffu, lane < warp ? b : 0);
    const unsigned below = (1u << lane) - 1;
    const int at = slow ? slow_before + __popc(hit & below) : slow_all + fast_before + __popc(in & ~hit & below);
    if (row < P.order && at == i) S.first = row;
    __syncthreads();
    i = S.first;
    __syncthreads();
    return i;
}

template <typename T, bool CACHED>
__global__ void __launch_bounds__(THREADS, 2) sample_kernel(const __grid_constant__ SampleParams P) {
    extern __shared__ __align__(16) uint8_t dynamic[];
    Shared &S = *(Shared *)dynamic;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)tc::cluster_rank();
    pdl_wait();
    const int64_t row = P.order ? slow_first(P, S, (int)(blockIdx.x / P.share)) : (int64_t)(blockIdx.x / P.share);
    Row<T, CACHED> R;
    R.rank = rank;
    R.share = P.share;
    R.first = min(P.V, rank * P.slice);
    R.n = min(P.V, R.first + P.slice) - R.first;
    meet_arrive();  // waited for before anything is pushed: the other CTAs have started
    bool coming = false;
    const T *src = (const T *)P.logits + row * P.ld + R.first;
    T *raw = nullptr;
    if constexpr (CACHED) R.raw = raw = fetch_slice(S, dynamic + sizeof(Shared), src, R.n, coming);
    else R.raw = src;
    R.infinite = false;

    const Settings set = settings_of(P, row);
    const float T_ = set.T, p = set.p, m = set.m;
    const int k = set.k;
    const bool by_k = set.by_k, by_p = set.by_p, by_m = set.by_m;
    if (tid == THREADS - 1 && k != 1) {
        const double c = 1.4426950408889634074 / (double)T_;
        S.ch = (float)c;
        S.cl = (float)(c - (double)S.ch);
        const double y = by_m ? -log2((double)m) : 0.0;
        S.yh = (float)y;
        S.yl = (float)(y - (double)S.yh);
    }
    for (int j = tid; j < 512; j += THREADS) S.root[j] = kRoots.at[j];
    if (tid == 0) S.first = MAX_V;
    __syncthreads();
    if (coming) wait_copy(S, &S.abort_word, 71, P.wait_limit);
    const int per = ((R.n + WARPS - 1) / WARPS + 31) / 32 * 32;  // a warp's tokens follow one another
    const int w0 = min(R.n, warp * per), w1 = min(R.n, w0 + per);
    R.bins = PER_NAT / T_;

    // ---------------- the maximum ----------------
    float mine = -INFINITY;  // of this thread's tokens; a NaN counts as nothing
    if constexpr (CACHED) {
#pragma unroll 8
        for (int i = tid; i < R.n; i += THREADS) mine = fmaxf(mine, R.at(i));
    } else {
        mine = max_of(src, R.n);
    }
    {
        const u64 w = warp_min((u64)~ordered_key(mine));
        if (lane == 0) S.warp_sum[warp] = w;
        __syncthreads();
        const u64 b = warp_min(lane < WARPS ? S.warp_sum[lane] : NONE);
        R.top = logit_of(b << INDEX_BITS);  // the CTA's
    }
    const float own_top = R.top;
    // A wait that ran out (the barrier above has shown it to every thread): the CTA's maximum is no number, which tells the cluster
    // when it meets; until then what lies in shared memory is taken as it is.
    bool lost = false;
    if constexpr (CACHED)
        if (*(volatile int *)&S.abort_word) R.top = NAN;

    // The tokens of the bins up to `to` (no more than `most` of them, or the answer is above FEW), in S.list by warp; and where
    // this warp's go among them.
    const auto list_up_to = [&](int to, int most, int &listed, int &before) -> int {
        listed = 0;
        // up to the last bin lie all tokens: -l < INFINITY
        const bool last = to == BINS - 1;
        const float top = last ? 0.0f : R.top, bins = last ? 1.0f : R.bins, xt = last ? INFINITY : (float)to + 1.0f;
#pragma unroll 1
        for (int i0 = w0; i0 < w1; i0 += 256) {
            float l[8];
            unsigned hit[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) l[e] = i0 + e * 32 + lane < w1 ? R.at(i0 + e * 32 + lane) : -INFINITY;
#pragma unroll
            for (int e = 0; e < 8; ++e) hit[e] = __ballot_sync(0xffffffffu, (top - l[e]) * bins < xt);  // false for -inf and NaN
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (hit[e] == 0) continue;
                const int at = listed + __popc(hit[e] & ((1u << lane) - 1));
                if ((hit[e] >> lane & 1) && at < LIST) S.list[warp][at] = order_of(l[e], R.first + i0 + e * 32 + lane);
                listed += __popc(hit[e]);
            }
        }
        return count_listed(S, listed, most, before);
    };
    // The bin up to which at least `want` of the threads' maxima lie (the last one, if there are not so many), from their
    // histogram over one CTA or all.
    const auto pick_maxima = [&](u64 one_, u64 two, u64 want) -> int {
        u64 all;
        const u64 sum = block_scan(S, one_ + two, all);
        if (tid == 0) S.pick_bin = BINS - 1;
        __syncthreads();
        if (sum >= want && sum - one_ - two < want) S.pick_bin = 2 * tid + (sum - two < want);
        __syncthreads();
        return S.pick_bin;
    };
    const auto maxima = [&]() {
        for (int b = tid; b < BINS; b += THREADS) S.rough[b] = 0;
        __syncthreads();
        if (mine > -INFINITY) atomicAdd(&S.rough[R.bin(mine)], 1u);
    };

    // ---------------- a CTA's own candidates ----------------
    // A token of the row's first k is one of its CTA's first k, and one near the row's maximum is nearer to its CTA's: with
    // a small k, or min-p alone, the CTAs list what they have and meet once.
    const int region = FEW / P.share;
    int n_few = -1, regions = 0;  // candidates of a row whose kept tokens are among them, and where they lie
    u64 all_few = 0;
    const bool alone = k != 1 && ((by_k && k <= min(region * 2 / 3, THREADS / 2)) || (by_m && !by_k && !by_p));
    if (alone) {
        int to, listed = 0, before = 0, count = FEW + 1;
        if (R.top < INFINITY) {
            if (by_k) {
                maxima();
                __syncthreads();
                to = pick_maxima(S.rough[2 * tid], S.rough[2 * tid + 1], (u64)k);
            } else {
                to = (int)fminf(PER_NAT * LN2_H * S.yh + 2.0f, (float)(BINS - 1));  // rounding moves a token by less than a bin
            }
            count = list_up_to(to, region, listed, before);
        }
        meet_wait();
        if (tid < P.share) {
            push(&S.in_top[rank], tid, R.top);
            push(&S.in_alone[rank], tid, count);
        }
        if (count <= region)
#pragma unroll 1
            for (int i = lane; i < listed; i += 32) push(&S.few[rank * region + before + i], 0, S.list[warp][i]);
        meet();
        int total = 0;
#pragma unroll 1
        for (int r = 0; r < P.share; ++r) {
            lost |= isnan(S.in_top[r]);
            R.top = fmaxf(R.top, S.in_top[r]);
            total = max(total, S.in_alone[r]);
        }
        if (total <= region && R.top > -INFINITY && !lost) {
            if (rank != 0) return;
            n_few = 0;
#pragma unroll 1
            for (int r = 0; r < P.share; ++r) n_few += S.in_alone[r];
            regions = region;
        }
    } else {
        meet_wait();
        if (tid < P.share) push(&S.in_top[rank], tid, R.top);
        meet();
#pragma unroll 1
        for (int r = 0; r < P.share; ++r) {
            lost |= isnan(S.in_top[r]);
            R.top = fmaxf(R.top, S.in_top[r]);
        }
    }
    if (CACHED && lost) {  // the same in every thread of the cluster: the row has no token
        if (coming) wait_copy(S, &S.never, 72, tc::kWaitLimitCycles);  // nothing may still be landing when the CTA leaves
        if (rank == 0 && tid == 0) {
            P.token[row] = -1;
            if (P.logprob) P.logprob[row] = -INFINITY;
            if (P.kept) P.kept[row] = 0;
        }
        return;
    }

    if (n_few < 0) {
        // ---------------- the first token, or none ----------------
        if (R.top == -INFINITY || k == 1) {  // the same in every thread of the cluster
            // CACHED: a thread's maximum is over the tokens that it looks through here; else the CTA's is known, not the thread's
            if (R.top > -INFINITY && (CACHED ? mine : own_top) == R.top) {
#pragma unroll 8
                for (int i = tid; i < R.n; i += THREADS)
                    if (R.at(i) == R.top) atomicMin(&S.first, R.first + i);
            }
            __syncthreads();
            if (tid == 0) push(&S.in_first[rank], 0, S.first);
            meet();
            if (rank == 0 && tid == 0) {
                const bool none = R.top == -INFINITY;
                int first = MAX_V;
#pragma unroll 1
                for (int r = 0; r < P.share; ++r) first = min(first, S.in_first[r]);
                P.token[row] = none ? -1 : first;
                if (P.logprob) P.logprob[row] = none ? -INFINITY : 0.0f;
                if (P.kept) P.kept[row] = none ? 0 : 1;
            }
            return;
        }
        R.ch = S.ch;
        R.cl = S.cl;
        if (R.top == INFINITY) {  // the infinite ones alone, as equals
            __syncthreads();
            if constexpr (CACHED)
                for (int i = tid; i < R.n; i += THREADS) raw[i] = from_f32<T>(R.at(i) == INFINITY ? 0.0f : -INFINITY);
            else R.infinite = true;
            mine = mine == INFINITY ? 0.0f : -INFINITY;
            R.top = 0.0f;
            __syncthreads();
        }

        // ---------------- where the run ends ----------------
        u64 bound = NONE;
        int turn = 0;
        // bins: the tokens before `from` are kept for certain, those behind `to` are not
        int from = 0, to = BINS;
        if (by_k) {
            // as many of the threads' maxima as tokens are wanted lie in the bins up to `to`: so do as many tokens
            maxima();
            meet();
            u64 one_, two;
            merge(S.rough, P.share, one_, two);
            to = pick_maxima(one_, two, (u64)k);
        } else if (by_m) {
            to = (int)fminf(PER_NAT * LN2_H * S.yh + 2.0f, (float)(BINS - 1));  // rounding moves a token by less than a bin
        } else if (by_p) {
            // The weight of a bin is that of its start times a sum of factors in (e^(-1/32), 1], counted in
            // steps that let all of the CTA's tokens lie in one bin.
            const float steps = P.slice < 65536 ? 65536.0f : 8192.0f;
            for (int b = tid; b < BINS; b += THREADS) S.rough[b] = 0;
            __syncthreads();
#pragma unroll 4
            for (int i = tid; i < R.n; i += THREADS) {
                const float l = R.at(i), x = R.x(l);
                if (!(l > -INFINITY) || x >= (float)(BINS - 1)) continue;
                const int b = (int)x;
                atomicAdd(&S.rough[b], (unsigned)fmaf(steps, tc::ex2_approx(((float)b - x) * (LOG2E / PER_NAT)), 0.5f));
            }
            meet();
            float one_, two;
            merge(S.rough, P.share, one_, two);
            one_ *= tc::ex2_approx((float)(2 * tid) * (-LOG2E / PER_NAT));
            two *= tc::ex2_approx((float)(2 * tid + 1) * (-LOG2E / PER_NAT));
            float sum = one_ + two;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float a = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += a;
            }
            __syncthreads();
            if (lane == 31) S.warp_sum[warp] = (u64)__float_as_uint(sum);
            if (tid == 0) S.pick_bin = S.pick_to = BINS - 1;
            __syncthreads();
            float before = 0.0f, all = 0.0f;
#pragma unroll 1
            for (int w = 0; w < WARPS; ++w) {
                const float a = __uint_as_float((unsigned)S.warp_sum[w]);
                if (w < warp) before += a;
                all += a;
            }
            sum += before;
            // Sums are off by less than 2^-15 of themselves, x and the bins' starts (arguments near 46 in 24 bits) by 2^-17, and by
            // half a step a factor; the tokens 32 nats down, left out, weigh less than 2^-28 in all.
            const float slack = 1.0f / 16384.0f + 1.0f / steps, least = p * all * (1.0f - slack), most = p * all * (1.0f + slack);
            if (sum >= least) atomicMin(&S.pick_bin, sum - two >= least ? 2 * tid : 2 * tid + 1);
            if (sum >= most) atomicMin(&S.pick_to, sum - two >= most ? 2 * tid : 2 * tid + 1);
            __syncthreads();
            from = S.pick_bin;
            to = S.pick_to;
        }

        // ---------------- candidates, and exact sums ----------------
        // w_all: what the warp's tokens weigh (top-p needs it of all, a draw from all of them too); w_sure: of those before `from`
        u64 w_all = 0, w_sure = 0;
        int sure = 0, listed = 0;
        bool by_few = false;
        const bool weigh = !by_k && (by_p || !by_m), list = to < BINS;
        if (weigh) {
            // a token beyond the last bin's finite products weighs nothing: no run by top-p ends there
            const float xf = (float)from, xt = to >= BINS - 1 ? INFINITY : (float)to + 1.0f;
#pragma unroll 1
            for (int i0 = w0; i0 < w1; i0 += 128) {
                float l[4];
                u64 w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) l[e] = i0 + e * 32 + lane < w1 ? R.at(i0 + e * 32 + lane) : -INFINITY;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = weight_of(R.top, l[e], R.ch, R.cl, S.root);
                if (!list) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w_all += w[e];
                        sure += l[e] > -INFINITY;
                    }
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = R.x(l[e]);  // -inf and NaN are in no bin
                    w_all += w[e];
                    if (x < xf) {
                        w_sure += w[e];
                        ++sure;
                    }
                    const unsigned hit = __ballot_sync(0xffffffffu, x >= xf && x < xt);
                    if (hit == 0) continue;
                    const int at = listed + __popc(hit & ((1u << lane) - 1));
                    if ((hit >> lane & 1) && at < LIST) S.list[warp][at] = order_of(l[e], R.first + i0 + e * 32 + lane);
                    listed += __popc(hit);
                }
            }
        }
        u64 all = 0, sure_all = 0;  // of the cluster
        if (list) {
            const u64 a = warp_sum(w_all), b = warp_sum(w_sure);
            int before, count = weigh ? count_listed(S, listed, FEW, before) : list_up_to(to, FEW, listed, before);
            if (lane == 0) {
                S.warp_sum[warp] = a;
                S.warp_two[warp] = b;
            }
            __syncthreads();
            if (warp == 0) {
                const u64 x = warp_sum(lane < WARPS ? S.warp_sum[lane] : 0), y = warp_sum(lane < WARPS ? S.warp_two[lane] : 0);
                if (lane < P.share) {
                    push(&S.in[0][rank], lane, x);
                    push(&S.in[1][rank], lane, y);
                    push(&S.in_count[rank], lane, count);
                }
            }
            meet();
            int total = 0;
#pragma unroll 1
            for (int r = 0; r < P.share; ++r) {
                const int c = S.in_count[r];
                if (r < rank) before += c;
                total += c;
                all += S.in[0][r];
                sure_all += S.in[1][r];
            }
            if (total <= FEW) {
#pragma unroll 1
                for (int i = lane; i < listed; i += 32) push(&S.few[before + i], 0, S.list[warp][i]);
                meet();
                if (from == 0) {  // there is nothing but the candidates
                    if (rank != 0) return;
                    n_few = total;
                    all_few = all;
                    goto few;
                }
                if (rank == 0) {  // top-p alone: the run ends among the candidates
                    const u64 target = part_of(p, all, true);
                    if (total <= THREADS) bound_few<1>(R, S, total, sure_all, target);
                    else bound_few<4>(R, S, total, sure_all, target);
                }
                meet();
                bound = S.bound;
                u64 w = 0;
#pragma unroll 1
                for (int i = lane; i < listed; i += 32)
                    if (S.list[warp][i] <= bound) {
                        w += weight_of(R.top, logit_of(S.list[warp][i]), R.ch, R.cl, S.root);
                        ++sure;
                    }
                w_all = w_sure + w;  // what the warp's kept tokens weigh
                by_few = true;
            }
        }
        if (list && !by_few) {  // many candidates
            if (by_k) {
                const Pick at = first_level<false>(R, S, NONE, (u64)k, 0.0f, turn);
                if (at.all > (u64)k) bound = refine<false>(R, S, NONE, at, (u64)k, turn);
            }
            if (by_p) {
                const Pick at = first_level<true>(R, S, bound, 0, p, turn);
                bound = refine<true>(R, S, bound, at, max(part_of(p, at.all, true), 1ull), turn);
            }
        }

        // ---------------- the draw ----------------
        const float fh = S.yh, fl = S.yl;
        // weight of a token, if it is kept
        const auto take = [&](int i, bool &kept, float &yh, float &yl) -> u64 {
            const float l = R.at(i);
            kept = l > -INFINITY && (bound == NONE || order_of(l, R.first + i) <= bound);
            const bool some = exponent(R.top, l, R.ch, R.cl, yh, yl);
            if (by_m && !passes(yh, yl, fh, fl)) kept = false;
            return kept && some ? weight(yh, yl, S.root) : 0;
        };
        if (list && !by_few) {
            w_all = 0;
            sure = 0;
            for (int i = w0 + lane; i < w1; i += 32) {
                bool kept;
                float yh, yl;
                w_all += take(i, kept, yh, yl);
                sure += kept;
            }
        }
        const u64 sum = warp_sum(w_all);
        const int count = __reduce_add_sync(0xffffffffu, sure);
        __syncthreads();
        if (lane == 0) {
            S.warp_sum[warp] = sum;
            S.warp_two[warp] = (u64)count;
        }
        __syncthreads();
        if (warp == 0) {
            const u64 x = warp_sum(lane < WARPS ? S.warp_sum[lane] : 0), n = warp_sum(lane < WARPS ? S.warp_two[lane] : 0);
            if (lane < P.share) {
                push(&S.in_draw[rank], lane, x);
                push(&S.in_kept[rank], lane, (int)n);
            }
        }
        meet();
        u64 whole = 0, before = 0;
        int kept_all = 0;
#pragma unroll 1
        for (int r = 0; r < P.share; ++r) {
            if (r < rank) before += S.in_draw[r];
            whole += S.in_draw[r];
            kept_all += S.in_kept[r];
        }
        const u64 goal = part_of(random_of(P, row), whole, false);
#pragma unroll 1
        for (int w = 0; w < warp; ++w) before += S.warp_sum[w];
        if (before <= goal && goal < before + S.warp_sum[warp]) {  // the token is this warp's
#pragma unroll 1
            for (int i0 = w0; i0 < w1; i0 += 32) {
                bool kept = false;
                float yh = 0.0f, yl = 0.0f;
                const u64 w = i0 + lane < w1 ? take(i0 + lane, kept, yh, yl) : 0;
                const u64 upto = before + warp_scan(w, lane);
                const unsigned hit = __ballot_sync(0xffffffffu, upto > goal);
                if (hit) {
                    if (lane == __ffs(hit) - 1) write_token(P, row, R.first + i0 + lane, yh, yl, whole, kept_all);
                    break;
                }
                before = __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        return;
    }
few:
    R.ch = S.ch;
    R.cl = S.cl;
    if (n_few <= THREADS) finish_few<1>(P, R, S, row, n_few, regions, by_k ? k : 0, p, m, all_few);
    else finish_few<4>(P, R, S, row, n_few, regions, by_k ? k : 0, p, m, all_few);
}

template <typename T, bool CACHED>
cudaError_t launch(const SampleParams &P, int R, cudaStream_t s) {
    auto *kernel = sample_kernel<T, CACHED>;
    const int most = (int)sizeof(Shared) + MAX_V / MAX_SHARE * (int)sizeof(T) + 16;
    const int smem = (int)sizeof(Shared) + (CACHED ? P.slice * (int)sizeof(T) + 16 : 0);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)R * P.share);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)P.share, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, P);
}

}  // namespace

int sample_read_error(int *site) {
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_sample_error, sizeof(int));
    if (e != cudaSuccess) return fail_cuda(e);
    if (v) {
        e = cudaMemcpyToSymbol(g_sample_error, &zero, sizeof(int));
        if (e != cudaSuccess) return fail_cuda(e);
        if (site) *site = v;
        return DSA_ERR_TIMEOUT;
    }
    return DSA_OK;
}

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
    // CTAs a row, and whether they keep their part of it.  A row takes some 20,000 cycles and 0.8 for a token of a CTA, one with
    // top-p alone 25,000 and 2.7; without its part in shared memory (from L2) a fifth more for a token, but two CTAs
    // an SM at any length.  What comes after the first rows that the SMs hold takes the average, the last rows may be slow ones.
    // 256 rows of 131,072, top-k 50: fp32 80 us with eight CTAs that keep theirs, 58 with four from L2; bf16 79 and 48 (four
    // that keep theirs); 67 masked rows of 50,001 in bf16 38 us with eight a row, 30 as chosen.
    const int item = dtype == DSA_F32 ? 4 : 2, sms = device_sm_count();
    double least = 1e30;
    bool cached = true;
    for (int share = 1; share <= MAX_SHARE; share *= 2)
        for (int keep = 1; keep >= 0; --keep) {
            const int slice = ((V + share - 1) / share + 31) / 32 * 32;
            if (keep && slice > MAX_V / MAX_SHARE) continue;
            const int per_sm = !keep || (int)sizeof(Shared) + slice * item + 16 <= 113 * 1024 ? 2 : 1;
            const double more = std::max(0.0, (double)R * share / (sms * per_sm) - 1), token = keep ? slice : 1.2 * slice;
            const double t = more * (20000 + 0.8 * token) + 25000 + 2.7 * token;
            if (t < least) {
                least = t;
                P.share = share;
                P.slice = slice;
                cached = keep;
            }
        }
    P.order = top_p && R <= THREADS && (int64_t)R * P.share > 2 * sms ? R : 0;
    P.u = u;
    P.temperature = temperature;
    P.top_k = top_k;
    P.top_p = top_p;
    P.min_p = min_p;
    P.token = token;
    P.logprob = logprob;
    P.kept = kept;
    P.wait_limit = wait_limit_cycles();
    const cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == DSA_F32 ? cached ? launch<float, true>(P, R, s) : launch<float, false>(P, R, s)
                          : cached ? launch<__nv_bfloat16, true>(P, R, s) : launch<__nv_bfloat16, false>(P, R, s);
    if (e != cudaSuccess) return fail_cuda(e);
    note_launch(DSA_KERNEL_SAMPLE);
    return DSA_OK;
}
