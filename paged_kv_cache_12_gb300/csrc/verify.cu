// Verification of drafted tokens against the target's probabilities, and the
// draw of the token that follows the ones that stand.
//
// A draft d with draft probability q(d) stands with probability
// min(1, p(d) / q(d)): when u q(d) < p(d) for a given u in [0, 1).  After the
// first one that fails the next token is drawn from the normalised
// max(p - q, 0), so that tokens come out distributed as p (the rejection step
// of speculative sampling; the drafts themselves are the pages' speculative
// tokens, "PagedAttention de vLLM : comment la gestion de la VRAM soutient
// l'inference des grands modeles", deepsonar.com.cn, section 2.5).
//
// Of the n + 1 rows of a sequence only the one after the last standing draft is
// read whole, with the draft's row beside it: the kernel is bound by HBM on a
// batch and by latency on a few sequences.  A cluster of eight CTAs, or of fewer
// where the batch fills the GPU's CTA slots, takes a sequence.  Every CTA finds
// the number of standing drafts (a warp, one draft a lane); the row's elements
// are summed in slices, one a warp of the cluster; one warp collects the totals
// through distributed shared memory and finds the slice in which the running sum
// passes the drawn height.  A short slice is searched by the warp that summed it;
// a long one is read again by the first CTA in eight parts, and the part that
// passes by a warp.
//
// Sums: a draw is decided where a running sum over up to a hundred thousand
// terms passes u * total, so sums are carried as an unevaluated pair of floats
// (Knuth's two-sum, exact error terms) and compared as such.  64-bit sums cost
// more than the reads: this GPU's 64-bit rate is two a clock and SM (512 totals
// of a row scanned in 64 bits by one warp took 14,000 clocks, eight partial sums
// compared in 64 bits by eight warps 4,000).
//
// One GB300: 100 sequences of 131,072 tokens in fp32, 27.5 us (3.5 TB/s of reads
// between the dependent steps: drafts, slices, collection, the slice again, the
// part); 4 sequences of 32,003 tokens, 8 us,
// the call included.

#include <climits>
#include <mutex>
#include <type_traits>

#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int VMAX_CTAS = 8;                   // CTAs of a sequence's cluster, at most
constexpr int VTHREADS = 256;
constexpr int VWARPS = VTHREADS / 32;
constexpr int VWIDE = 16;                      // warps of a CTA where few trees have the GPU
constexpr int VRESIDENT = 4;                   // CTAs an SM holds (64 registers a thread)
constexpr int VCHUNK = 128;                    // elements a warp reads at once, four a lane
constexpr int VBATCH = 4;                      // chunks on their way at once
constexpr int VSLICES = 64;                    // of a row, at most: two a lane of the collecting warp
static_assert(VMAX_CTAS * VWARPS == VSLICES, "two slices a lane");

struct VerifyArgs {
    int32_t *accepted, *tokens;
    const void *target, *draft;
    const int32_t *draft_tokens, *draft_start;
    const float *uniform, *sample;
    int num_seqs, num_drafts, max_drafts, vocab;
    long long target_stride, draft_stride;
};

__device__ __forceinline__ float prob(float x) { return x; }
__device__ __forceinline__ float prob(__half x) { return __half2float(x); }
__device__ __forceinline__ float prob(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
struct alignas(4 * sizeof(T)) Quad {
    T v[4];
};

// hi + lo, a sum carried in two floats.
struct Sum2 {
    float hi = 0.f, lo = 0.f;
    // adds s + e exactly in the high part's rounding error
    __device__ __forceinline__ void add(float s, float e) {
        const float t = __fadd_rn(hi, s);
        const float b = __fsub_rn(t, hi);
        const float r = __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(s, b));
        hi = t;
        lo = __fadd_rn(lo, __fadd_rn(r, e));
    }
    __device__ __forceinline__ void add(const Sum2 &x) { add(x.hi, x.lo); }
    __device__ __forceinline__ float value() const { return hi + lo; }
    // this > x: the high parts' difference is exact where they are near
    __device__ __forceinline__ bool over(const Sum2 &x) const {
        return __fadd_rn(__fsub_rn(hi, x.hi), __fsub_rn(lo, x.lo)) > 0.f;
    }
    __device__ __forceinline__ Sum2 times(float u) const {   // exact to twice a float's precision
        const float h = __fmul_rn(u, hi);
        return Sum2{h, __fmaf_rn(u, lo, __fmaf_rn(u, hi, -h))};
    }
    __device__ __forceinline__ Sum2 scaled(float f) const { return Sum2{hi * f, lo * f}; }   // f a power of two
    __device__ __forceinline__ bool any() const { return hi > 0.f; }   // sums of weights >= 0
};

// Two sums side by side, each hi + lo in two floats (Sum2 on pairs: seven
// instructions for two terms).
struct Sum2Pair {
    uint64_t hi = 0, lo = 0;
    __device__ __forceinline__ void add(uint64_t s) {
        const uint64_t minus = pair_of(-1.f, -1.f);
        const uint64_t t = pair_add(hi, s), b = pair_fma(hi, minus, t);
        const uint64_t r = pair_add(pair_fma(pair_fma(b, minus, t), minus, hi), pair_fma(b, minus, s));
        hi = t;
        lo = pair_add(lo, r);
    }
    // the same for 0 <= s <= hi in four (Dekker's form: there t - hi is exact)
    __device__ __forceinline__ void add_below(uint64_t s) {
        const uint64_t minus = pair_of(-1.f, -1.f), t = pair_add(hi, s);
        lo = pair_add(lo, pair_fma(pair_fma(hi, minus, t), minus, s));
        hi = t;
    }
    __device__ __forceinline__ float least() const {
        float h0, h1;
        pair_parts(hi, h0, h1);
        return fminf(h0, h1);
    }
    __device__ __forceinline__ Sum2 sum() const {
        float h0, h1, l0, l1;
        pair_parts(hi, h0, h1);
        pair_parts(lo, l0, l1);
        Sum2 x{h0, l0};
        x.add(h1, l1);
        return x;
    }
};

// The sum over the warp's lanes, the same in every lane.
__device__ __forceinline__ Sum2 warp_sum(Sum2 x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        x.add(__shfl_xor_sync(0xffffffffu, x.hi, d), __shfl_xor_sync(0xffffffffu, x.lo, d));
    return Sum2{__shfl_sync(0xffffffffu, x.hi, 0), __shfl_sync(0xffffffffu, x.lo, 0)};
}

// The sum over this lane and the ones before it.
__device__ __forceinline__ Sum2 warp_scan(Sum2 x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const float h = __shfl_up_sync(0xffffffffu, x.hi, d), l = __shfl_up_sync(0xffffffffu, x.lo, d);
        if (lane >= d) x.add(h, l);
    }
    return x;
}

// The weight max(p - q, 0) as its rounded value and rounding error; NaN is 0.
__device__ __forceinline__ void weight(float p, float q, float &s, float &e) {
    s = __fsub_rn(p, q);
    const float b = __fsub_rn(s, p);
    e = __fsub_rn(__fsub_rn(p, __fsub_rn(s, b)), __fadd_rn(q, b));
    if (!(s > 0.f)) s = e = 0.f;
}

// A row's weights: p, less q where a draft's row stands beside it, none for
// the token `out` (-1: all count).
template <typename T>
struct Weights {
    const T *p, *q;
    int out;
    bool quads;   // both rows may be read four elements at a time
    __device__ __forceinline__ Weights(const T *p_, const T *q_, int out_) : p(p_), q(q_), out(out_) {
        quads = ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & (4 * sizeof(T) - 1)) == 0;
    }
    __device__ __forceinline__ void at(int v, float pv, float qv, float &s, float &e) const {
        weight(pv, qv, s, e);
        if (v == out) s = e = 0.f;
    }
};

// Four elements a lane of the chunk at `base` (elements from `end` on are 0).
template <typename T>
__device__ __forceinline__ void load_chunk(const Weights<T> &w, int base, int end, float (&p)[4], float (&q)[4]) {
    const int lane = threadIdx.x & 31;
    if (w.quads && base + VCHUNK <= end) {
        const Quad<T> a = *reinterpret_cast<const Quad<T> *>(w.p + base + 4 * lane);
        Quad<T> b{};
        if (w.q) b = *reinterpret_cast<const Quad<T> *>(w.q + base + 4 * lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = prob(a.v[k]), q[k] = w.q ? prob(b.v[k]) : 0.f;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int v = base + 4 * lane + k;
            p[k] = v < end ? prob(w.p[v]) : 0.f;
            q[k] = w.q && v < end ? prob(w.q[v]) : 0.f;
        }
    }
}

// Sum of the weights [lo, hi), lo a multiple of four, by a warp: the same in every lane.
template <typename T>
__device__ __forceinline__ Sum2 range_sum(const Weights<T> &w, int lo, int hi) {
    const int lane = threadIdx.x & 31;
    Sum2 acc;
    for (int base = lo; base < hi; base += VBATCH * VCHUNK) {
        float p[VBATCH][4], q[VBATCH][4];
#pragma unroll
        for (int u = 0; u < VBATCH; ++u) load_chunk(w, min(hi, base + u * VCHUNK), hi, p[u], q[u]);
#pragma unroll
        for (int u = 0; u < VBATCH; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float s, e;
                w.at(base + u * VCHUNK + 4 * lane + i, p[u][i], q[u][i], s, e);
                acc.add(s, e);
            }
    }
    return warp_sum(acc);
}

// The height u * total that a running sum has to pass.  Sums are compared with it
// at `up` times their value: a small total's are raised, because a float's steps end
// at 2^-149 and the low part of u * total would be lost there.
struct Height {
    Sum2 at;
    float up = 1.f;
    Height() = default;
    __device__ __forceinline__ Height(const Sum2 &total, float u) {
        up = total.hi < 0x1p-60f ? 0x1p60f : 1.f;
        at = total.scaled(up).times(u);
    }
    __device__ __forceinline__ bool passed_by(const Sum2 &run) const { return run.scaled(up).over(at); }
};

// The smallest v in [lo, hi) of positive weight whose running sum, from
// `before` on, passes `height`; where rounding lets none pass, the last of
// positive weight.  One warp, in element order: four consecutive elements a lane.
template <typename T>
__device__ int find_in_range(const Weights<T> &w, int lo, int hi, Sum2 before, const Height height) {
    const int lane = threadIdx.x & 31;
    int last = -1;
    for (int base = lo; base < hi; base += VCHUNK) {
        float p[4], q[4], s[4], e[4];
        load_chunk(w, base, hi, p, q);
        Sum2 mine;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w.at(base + 4 * lane + k, p[k], q[k], s[k], e[k]);
            mine.add(s[k], e[k]);
            if (s[k] > 0.f) last = base + 4 * lane + k;
        }
        const Sum2 upto = warp_scan(mine);
        Sum2 run = upto;   // the running sum before this lane's elements
        run.add(-mine.hi, -mine.lo);
        run.add(before);
        int v = INT_MAX;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            run.add(s[k], e[k]);
            if (v == INT_MAX && s[k] > 0.f && height.passed_by(run)) v = base + 4 * lane + k;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, d));
        if (v != INT_MAX) return v;
        before.add(__shfl_sync(0xffffffffu, upto.hi, 31), __shfl_sync(0xffffffffu, upto.lo, 31));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, d));
    return last;
}

// What a cluster's CTAs, of W warps each, share while they draw a token.
template <int W>
struct Draw {
    Sum2 totals[W];   // this CTA's slices; then, in the leader, the parts of one
    Sum2 before;           // the leader's: the sum before the slice that passes
    Height height;
    int slice;             // the leader's: that slice; -1: no token; -2: no weight at all
};

// The first of the leader's parts (in sh.totals) at whose end the running sum, from `run`
// on, passes the height, else the last of any weight; `before`: the sum before it.
template <int W>
__device__ __forceinline__ int passing_part(const Draw<W> &sh, Sum2 run, Sum2 &before) {
    int at = -1;
    bool passed = false;
    for (int k = 0; k < W; ++k) {
        const Sum2 x = sh.totals[k];
        Sum2 after = run;
        after.add(x);
        if (!passed && x.any()) {
            at = k;
            before = run;
            passed = sh.height.passed_by(after);
        }
        run = after;
    }
    return at;
}

// The sum of a row's own weights [lo, hi), lo a multiple of eight, by a thread.
template <typename T>
__device__ __forceinline__ Sum2 piece_sum(const Weights<T> &w, int lo, int hi) {
    Sum2Pair acc;
#pragma unroll 4
    for (int base = lo; base < hi; base += 8) {
        float p[8];
        if (w.quads && base + 8 <= hi) {
            const Quad<T> a = *reinterpret_cast<const Quad<T> *>(w.p + base);
            const Quad<T> b = *reinterpret_cast<const Quad<T> *>(w.p + base + 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = prob(a.v[k]), p[4 + k] = prob(b.v[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) p[k] = base + k < hi ? prob(w.p[base + k]) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; k += 2) acc.add(pair_of(fmaxf(p[k], 0.f), fmaxf(p[k + 1], 0.f)));
    }
    return acc.sum();
}

// The element of a slice [lo, hi) of a row's own weights at which the running sum, `run`
// before the slice, passes sh.height; by a CTA, a consecutive piece a thread.  (In parts
// until one was as short as a warp's chunk: three reads one after another, and 64
// sequences of 131072 tokens in bf16 took 54.8 us where this takes 45.8.)
constexpr int VPIECE = 128;   // elements of a thread's piece, at most
template <typename T, int W, class Publish>
__device__ __forceinline__ void find_in_slice(Draw<W> &sh, Publish publish, const Weights<T> &w, int lo, int hi, Sum2 run) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int piece = ((hi - lo + 32 * W - 1) / (32 * W) + 7) / 8 * 8;
    const int plo = min(hi, lo + (int)threadIdx.x * piece), phi = min(hi, plo + piece);
    const Sum2 mine = piece_sum(w, plo, phi);
    const Sum2 upto = warp_scan(mine);
    if (lane == 31) sh.totals[warp] = upto;
    __syncthreads();
    // Of the sums x of one part a lane, x_upto being their running sum: the first at whose
    // end that sum passes, from `run` on, else the last of any weight; run becomes the sum
    // before it.
    auto first_passing = [&](const Sum2 &x, Sum2 x_upto) {
        x_upto.add(run);
        const unsigned any = __ballot_sync(0xffffffffu, x.any());
        const unsigned over = __ballot_sync(0xffffffffu, x.any() && sh.height.passed_by(x_upto));
        const int l = over ? __ffs((int)over) - 1 : 31 - __clz((int)any);
        x_upto.add(-x.hi, -x.lo);
        run = Sum2{__shfl_sync(0xffffffffu, x_upto.hi, l & 31), __shfl_sync(0xffffffffu, x_upto.lo, l & 31)};
        return l;   // -1: no weight at all
    };
    // eight parts one after another, sixteen a lane each (64 x 32 nodes of 131,072 tokens in
    // bf16 41.4 us, with a lane each 42.3; 4 x 16 of 32,003 in fp32 9.7 and 9.2)
    int at;
    if constexpr (W <= 8) {
        const Sum2 start = run;
        at = passing_part(sh, start, run);
    } else {
        const Sum2 part = lane < W ? sh.totals[lane] : Sum2();
        at = first_passing(part, warp_scan(part));
    }
    if (warp != at) return;
    const int l = first_passing(mine, upto);
    publish(find_in_range(w, __shfl_sync(0xffffffffu, plo, l), __shfl_sync(0xffffffffu, phi, l), run, sh.height));
}

// Draws a token by the weights w: the smallest whose running sum passes u times
// the total.  `ctas` CTAs of the cluster from rank `leader` on do it (`has`: for a row;
// the same CTAs may have none), all CTAs of the cluster take part in its meetings.  One
// warp calls publish with the token after the first of them (none does where there is no
// token).  Returns the slice in which it lies, -1 where there is none, or `empty` where
// the weights sum to zero.  OWN: the weights are a row's own, nobody needs that answer, and
// a slice may be long (where few CTAs have a row).
template <typename T, bool OWN, int W, class Range, class Publish>
__device__ __forceinline__ int draw_token(cg::cluster_group &cluster, int leader, int ctas, Draw<W> &sh,
                                          const Weights<T> &w, int vocab, bool has, const float *u, int empty,
                                          Range range, Publish publish) {
    const int rank = (int)cluster.block_rank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slices = ctas * W;   // at most VSLICES
    const int len = ((vocab + slices - 1) / slices + VCHUNK - 1) / VCHUNK * VCHUNK;   // of a slice
    const int own = (rank - leader) * W + warp;
    const long long from = (long long)own * len;
    const int lo = (int)min((long long)vocab, from), hi = has ? (int)min((long long)vocab, from + len) : lo;
    const Sum2 mine = range(w, lo, hi);
    if (lane == 0) sh.totals[warp] = mine;
    cluster.sync();
    if (rank == leader && warp == 0) {   // lane l: slices 2 l and 2 l + 1
        Sum2 x0, x1;
        if (2 * lane < slices) {
            const Sum2 *src = cluster.map_shared_rank(sh.totals, leader + 2 * lane / W) + 2 * lane % W;
            x0 = src[0];
            x1 = src[1];
        }
        Sum2 both = x0;
        both.add(x1);
        const Sum2 upto = warp_scan(both);
        const Sum2 all{__shfl_sync(0xffffffffu, upto.hi, 31), __shfl_sync(0xffffffffu, upto.lo, 31)};
        const float total = all.value();   // the same in all lanes
        int slice = total == 0.f ? empty : -1;
        if (total > 0.f && isfinite(total)) {
            const Height height(all, *u);
            Sum2 run = upto;   // before the lane's slices
            run.add(-both.hi, -both.lo);
            Sum2 run1 = run;
            run1.add(x0);
            // the first slice whose running sum passes, else the last of any weight
            const int g = x0.any() && height.passed_by(run1)   ? 2 * lane
                          : x1.any() && height.passed_by(upto) ? 2 * lane + 1
                                                               : INT_MAX;
            int first = g, last = x1.any() ? 2 * lane + 1 : x0.any() ? 2 * lane : -1;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                first = min(first, __shfl_xor_sync(0xffffffffu, first, d));
                last = max(last, __shfl_xor_sync(0xffffffffu, last, d));
            }
            slice = first != INT_MAX ? first : last;
            if (slice >> 1 == lane) {
                sh.before = slice & 1 ? run1 : run;
                sh.height = height;
            }
        }
        if (lane == 0) sh.slice = slice;
    }
    const bool is_short = !OWN && len <= VBATCH * VCHUNK;
    if (OWN) {   // the leader goes on alone
        if (rank != leader) return -1;
        __syncthreads();
    } else {
        cluster.sync();   // the leader has read every CTA's totals and decided
    }
    const int slice = *cluster.map_shared_rank(&sh.slice, leader);
    if (is_short) {   // short slices: the warp that summed it finds the element
        if (slice == own)
            publish(find_in_range(w, lo, hi, *cluster.map_shared_rank(&sh.before, leader),
                                  *cluster.map_shared_rank(&sh.height, leader)));
    } else if (rank == leader && slice >= 0) {   // the slice again, in parts (OWN: while it is long)
        int first = slice * len, n = len;
        Sum2 before = sh.before;
        for (;;) {
            if (OWN && n <= 32 * W * VPIECE) {
                find_in_slice(sh, publish, w, first, min(vocab, first + n), before);
                break;
            }
            const int part = ((n + W - 1) / W + VCHUNK - 1) / VCHUNK * VCHUNK;
            const int plo = min(vocab, min(first + n, first + warp * part));
            const int phi = min(vocab, min(first + n, plo + part));
            const Sum2 mine = range(w, plo, phi);
            if (lane == 0) sh.totals[warp] = mine;
            __syncthreads();
            const Sum2 run = before;
            const int at = passing_part(sh, run, before);
            if (!OWN || at < 0) {
                if (warp == at) publish(find_in_range(w, plo, phi, before, sh.height));
                break;
            }
            n = min(part, n - at * part);
            first += at * part;
            __syncthreads();   // the totals have been read
        }
    }
    return slice;
}

template <typename T, int VCTAS>
__global__ void __cluster_dims__(VCTAS, 1, 1) __launch_bounds__(VTHREADS, VRESIDENT) verify_kernel(const VerifyArgs a) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    const int seq = blockIdx.x / VCTAS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ Draw<VWARPS> draw;
    __shared__ int s_next;
    __shared__ int s_kept, s_n, s_d0;
    grid_release();
    grid_wait();

    if (warp == 0) {
        const int d0 = a.draft_start[seq], d1 = a.draft_start[seq + 1];
        const int n = d1 - d0;
        bool ok = d0 >= 0 && d1 >= d0 && d1 <= a.num_drafts && n <= a.max_drafts && (seq > 0 || d0 == 0) &&
                  (seq < a.num_seqs - 1 || d1 == a.num_drafts);
        int kept = 0;
        for (int base = 0; ok && base < n; base += 32) {
            const int j = base + lane;
            bool in_range = true, stands = j < n;
            if (j < n) {
                const int d = a.draft_tokens[d0 + j];
                in_range = d >= 0 && d < a.vocab;
                if (in_range) {
                    const float p = prob(static_cast<const T *>(a.target)[(long long)(d0 + seq + j) * a.target_stride + d]);
                    const float q =
                        a.draft ? prob(static_cast<const T *>(a.draft)[(long long)(d0 + j) * a.draft_stride + d]) : 1.f;
                    stands = (double)a.uniform[d0 + j] * (double)q < (double)p;   // 24 + 24 bits: exact
                }
            }
            const unsigned fails = __ballot_sync(0xffffffffu, !(stands && in_range));
            const unsigned off = __ballot_sync(0xffffffffu, !in_range);
            const int first = fails ? __ffs((int)fails) - 1 : 32;
            kept = base + first;
            if (first < 32) {
                if (off >> first & 1u) ok = false;   // a token outside the vocabulary decides
                break;
            }
        }
        if (lane == 0) {
            s_kept = ok ? min(kept, n) : -1;
            s_n = n;
            s_d0 = d0;
        }
    }
    __syncthreads();
    const int kept = s_kept, n = s_n, d0 = s_d0;
    int32_t *out = a.tokens + (long long)seq * (a.max_drafts + 1);
    if (rank == 0 && threadIdx.x == 0) s_next = -1;   // (others write it after the cluster's first meeting)
    if (kept >= 0) {   // the same in every CTA of the cluster
        const bool failed = kept < n;
        const T *p = static_cast<const T *>(a.target) + (long long)(d0 + seq + kept) * a.target_stride;
        const T *q = failed && a.draft ? static_cast<const T *>(a.draft) + (long long)(d0 + kept) * a.draft_stride : nullptr;
        Weights<T> w(p, q, failed && !a.draft ? a.draft_tokens[d0 + kept] : -1);
        for (int attempt = 0; attempt < 2; ++attempt) {
            const int slice =
                draw_token<T, false>(cluster, 0, VCTAS, draw, w, a.vocab, true, a.sample + seq,
                                     attempt == 0 && failed ? -2 : -1,
                                     [](const Weights<T> &x, int lo, int hi) { return range_sum(x, lo, hi); },
                                     [&](int v) { if (lane == 0) *cluster.map_shared_rank(&s_next, 0) = v; });
            if (slice != -2) break;
            w = Weights<T>(p, nullptr, -1);   // q covers p: draw from p itself
            cluster.sync();   // every CTA has read the decision
        }
        cluster.sync();   // the token is there, and rank 0's shared memory outlives its readers
    }
    if (rank == 0 && warp == 0) {
        for (int j = lane; j <= a.max_drafts; j += 32)
            out[j] = kept < 0 ? -1 : j < kept ? a.draft_tokens[d0 + j] : j == kept ? s_next : -1;
        if (lane == 0) a.accepted[seq] = kept;
    }
}

// ------------------------------------------------------------------ trees

struct TreeVerifyArgs {
    int32_t *accepted, *tokens, *path;
    const void *target;
    const int32_t *node_tokens, *parents, *tree_start;
    const float *uniform;
    int num_seqs, num_nodes, max_depth, vocab;
    long long target_stride;
};

// Eight 16-bit elements of a row as weights (what is negative or NaN becomes zero),
// their largest, and their sum added to one that is no less than any of them.
template <typename T>
struct Weights8 {
    static __device__ __forceinline__ void clamp(uint4 &v) {
        v.x = not_below_zero(v.x), v.y = not_below_zero(v.y), v.z = not_below_zero(v.z), v.w = not_below_zero(v.w);
    }
    static __device__ __forceinline__ uint32_t largest(uint32_t m, uint4 v) {
        return __vmaxu2(__vmaxu2(__vmaxu2(m, v.x), __vmaxu2(v.y, v.z)), v.w);
    }
    static __device__ __forceinline__ float value(uint32_t m) {
        float a, b;
        pair_parts(two(m), a, b);
        return fmaxf(a, b);
    }
    static __device__ __forceinline__ void add(Sum2Pair &acc, uint4 v) {
        acc.add_below(two(v.x));
        acc.add_below(two(v.y));
        acc.add_below(two(v.z));
        acc.add_below(two(v.w));
    }

private:
    static __device__ __forceinline__ uint32_t not_below_zero(uint32_t w) {
        uint32_t r;
        if constexpr (std::is_same<T, __half>::value)
            asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0));
        else
            asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0));
        return r;
    }
    static __device__ __forceinline__ uint64_t two(uint32_t w) {
        if constexpr (std::is_same<T, __half>::value) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
            return pair_of(f.x, f.y);
        } else {
            return pair_of(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        }
    }
};

// range_sum of a row's own weights, with more bytes on their way: 16 at a time
// from the first 16-byte boundary on, whatever the row's alignment.  Eight loads and
// one sum are what 64 registers hold (64 sequences of 131072 tokens in bf16, mean of
// eight draws, 54.5 us at first: with two and four sums 56 and 65, four loads 77; through
// shared memory cells with two sums 57).
//
// The additions are a quarter of the time (plain fp32 sums: 46 us -> 35).  Of 16-bit
// elements the largest of a lane's 64 costs half an instruction each, and a sum that is no
// less than it needs four instructions for two terms instead of seven: so a sum that is
// less is first lifted by that largest, which the end takes off again (46 -> 41; the lifts
// at most double the sum, so the error stays a few steps of its second float).  Of fp32
// elements the maxima cost what they save.
constexpr int VLOADS = 8;
template <typename T>
__device__ __forceinline__ Sum2 row_sum(const T *p, int lo, int hi) {
    constexpr int E = 16 / sizeof(T);
    const int lane = threadIdx.x & 31;
    const int skip = (int)((16 - (reinterpret_cast<uintptr_t>(p + lo) & 15u)) & 15u) / (int)sizeof(T);
    const int head = min(hi, lo + skip), nvec = (hi - head) / E, tail = head + nvec * E;
    const uint4 *v = reinterpret_cast<const uint4 *>(p + head);
    Sum2Pair acc;
    Sum2 lift;   // what both sums of acc hold beside the weights
    if (lane < head - lo) acc.add(pair_of(fmaxf(prob(p[lo + lane]), 0.f), 0.f));
    if (lane < hi - tail) acc.add(pair_of(fmaxf(prob(p[tail + lane]), 0.f), 0.f));
    for (int i0 = 0; i0 < nvec; i0 += 32 * VLOADS) {
        uint4 x[VLOADS];
#pragma unroll
        for (int k = 0; k < VLOADS; ++k) {
            const int i = i0 + 32 * k + lane;
            x[k] = i < nvec ? v[i] : make_uint4(0, 0, 0, 0);
        }
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int k = 0; k < VLOADS; ++k) {
                acc.add(pair_of(fmaxf(__uint_as_float(x[k].x), 0.f), fmaxf(__uint_as_float(x[k].y), 0.f)));
                acc.add(pair_of(fmaxf(__uint_as_float(x[k].z), 0.f), fmaxf(__uint_as_float(x[k].w), 0.f)));
            }
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < VLOADS; ++k) {
                Weights8<T>::clamp(x[k]);
                m = Weights8<T>::largest(m, x[k]);
            }
            const float top = Weights8<T>::value(m);
            if (top > acc.least()) {
                acc.add(pair_of(top, top));
                lift.add(top, 0.f);
            }
#pragma unroll
            for (int k = 0; k < VLOADS; ++k) Weights8<T>::add(acc, x[k]);
        }
    }
    Sum2 sum = acc.sum();
    sum.add(-lift.hi, -lift.lo);
    sum.add(-lift.hi, -lift.lo);
    return warp_sum(sum);
}

// A path through a sequence's tree, by a cluster.  One level after another would
// cost a row's read and the meetings for each; so the cluster's CTAs draw the
// tokens of several nodes at a time, the present one's and those of descendants
// that it may lead to, in groups of as many CTAs each, and then walk as far as
// those tokens go.  `rows`: nodes of the first such wave; later ones take one a CTA,
// however long the rows.  That suits drafts that usually stand, where most sequences reach
// a third or fourth wave: 64 x 32 nodes of 131,072 tokens in bf16 with 1.7 drafts standing
// on average 42 us, with 5.3 of them 87; with `rows` nodes in every wave 39 and 97 (in fp32
// 63 and 135 against 57 and 163).
//
// One GB300: 64 sequences of 32 nodes and 131,072 tokens in bf16 41 us (mean of eight
// draws, on the device; one level after another 139), two or three waves, of whose first the
// 67 MB of sums take about half; 4 sequences of 16 nodes and 32,003 tokens in fp32 9.2 us.
template <typename T, int VCTAS, int W>
__global__ void __cluster_dims__(VCTAS, 1, 1) __launch_bounds__(32 * W, VRESIDENT * VWARPS / W)
    verify_tree_kernel(const TreeVerifyArgs a, int rows) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    const int seq = blockIdx.x / VCTAS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ Draw<W> draw;
    // the groups' tokens, written into every CTA; by the wave's parity (a CTA may still read
    // one wave's while the next is drawn)
    __shared__ int s_next[2][VCTAS];
    __shared__ int s_nodes[VCTAS], s_count;
    __shared__ int s_node, s_level;
    __shared__ int32_t s_parents[PA_TREE_MAX_NODES], s_tokens[PA_TREE_MAX_NODES];   // of the tree's first nodes
    grid_release();
    grid_wait();
    const int n0 = a.tree_start[seq], n1 = a.tree_start[seq + 1];
    const bool ok = n0 >= 0 && n1 > n0 && n1 <= a.num_nodes && (seq > 0 || n0 == 0) &&
                    (seq < a.num_seqs - 1 || n1 == a.num_nodes);
    const int n = n1 - n0;
    auto parent = [&](int j) { return j < PA_TREE_MAX_NODES ? s_parents[j] : a.parents[n0 + j]; };
    auto drafted = [&](int j) { return j < PA_TREE_MAX_NODES ? s_tokens[j] : a.node_tokens[n0 + j]; };
    for (int j = threadIdx.x; ok && j < min(n, PA_TREE_MAX_NODES); j += 32 * W) {
        s_parents[j] = a.parents[n0 + j];
        s_tokens[j] = a.node_tokens[n0 + j];
    }
    __syncthreads();
    int32_t *tokens = a.tokens + (long long)seq * (a.max_depth + 1);
    int32_t *path = a.path + (long long)seq * (a.max_depth + 1);
    // everything here is the same in every CTA of the cluster
    int level = 0, node = ok ? 0 : -1;
    for (int wave = 0; node >= 0; ++wave) {
        const int most = wave ? VCTAS : rows;
        if (warp == 0) {
            // The present node and the first of its descendants, in the order of their
            // numbers, among the 1024 nodes behind it: lane k holds those of the k-th 32.
            unsigned words = 0;
            int count = 1;
            for (int k = 0; k < 32 && count < most && node + 1 + 32 * k < n; ++k) {
                const int j = node + 1 + 32 * k + lane;
                const int up = j < n ? parent(j) - (node + 1) : -2;   // the parent, so counted; -1: the present node
                const unsigned word = __shfl_sync(0xffffffffu, words, up >> 5 & 31);
                bool in = up == -1 || (up >= 0 && up < 32 * k && (word >> (up & 31) & 1u));
                unsigned set = __ballot_sync(0xffffffffu, in);
                for (;;) {   // and those whose parent is one of these 32
                    const int own = up - 32 * k;
                    in = in || (own >= 0 && own < 32 && (set >> (own & 31) & 1u));
                    const unsigned more = __ballot_sync(0xffffffffu, in);
                    if (more == set) break;
                    set = more;
                }
                const int place = count + __popc(set & ((1u << lane) - 1u));
                if (in && place < most) s_nodes[place] = j;
                count = min(most, count + __popc(set));
                if (lane == k) words = set;
            }
            if (lane == 0) {
                s_nodes[0] = node;
                s_count = count;
            }
        }
        int *next = s_next[wave & 1];
        if (threadIdx.x < VCTAS) next[threadIdx.x] = -1;
        __syncthreads();
        int groups = 1;
        while (groups < s_count) groups *= 2;
        const int ctas = min(VSLICES / W, VCTAS / groups), group = rank / ctas, leader = group * ctas;
        const bool has = group < s_count;   // a group without a node has no row either
        const int who = has ? s_nodes[group] : node;
        const T *p = static_cast<const T *>(a.target) + (long long)(n0 + who) * a.target_stride;
        draw_token<T, true>(cluster, leader, ctas, draw, Weights<T>(p, nullptr, -1), a.vocab, has,
                            a.uniform + n0 + who, -1,
                            [](const Weights<T> &x, int lo, int hi) { return row_sum(x.p, lo, hi); },
                            [&](int v) { if (lane < VCTAS) *cluster.map_shared_rank(&next[group], lane) = v; });
        cluster.sync();   // the tokens are there
        if (warp == 0) {
            const int count = s_count;
            const int token = lane < count ? next[lane] : -1;
            const int number = lane < count ? s_nodes[lane] : -1;
            int at = 0, cur = node, lv = level, go = -1;
            for (;;) {   // node cur, the at-th of the wave
                const int v = __shfl_sync(0xffffffffu, token, at);
                if (rank == 0 && lane == 0) {
                    tokens[lv] = v;
                    path[lv] = cur;
                }
                int child = -1;
                for (int base = cur + 1; v >= 0 && lv < a.max_depth && base < n; base += 32) {
                    const int j = base + lane;
                    const unsigned has = __ballot_sync(0xffffffffu, j < n && parent(j) == cur && drafted(j) == v);
                    if (has) {
                        child = base + __ffs((int)has) - 1;
                        break;
                    }
                }
                if (child < 0) break;
                cur = child;
                ++lv;
                const unsigned here = __ballot_sync(0xffffffffu, number == child);
                if (!here) {
                    go = child;   // drawn in the next wave
                    break;
                }
                at = __ffs((int)here) - 1;
            }
            if (lane == 0) {
                s_node = go;
                s_level = lv;
            }
        }
        __syncthreads();
        node = s_node;
        level = s_level;
    }
    if (rank == 0) {
        for (int j = (ok ? level + 1 : 0) + (int)threadIdx.x; j <= a.max_depth; j += 32 * W) tokens[j] = path[j] = -1;
        if (threadIdx.x == 0) a.accepted[seq] = ok ? level : -1;
    }
    // (nothing reaches into another CTA's shared memory after the last meeting)
}

// The largest cluster with which all sequences' CTAs are resident at once (100
// sequences of 131072 tokens: clusters of 8, in two rounds, 34 us; 4 sequences of
// 32003: 9 us with 8).
template <typename T>
int launch_verify(const VerifyArgs &a, cudaStream_t st) {
    const long long slots = (long long)num_sms() * VRESIDENT;
    const unsigned b = (unsigned)a.num_seqs;
    if (b * 8LL <= slots)
        return launch_early(verify_kernel<T, 8>, dim3(b * 8), VTHREADS, 0, st, a);
    if (b * 4LL <= slots) return launch_early(verify_kernel<T, 4>, dim3(b * 4), VTHREADS, 0, st, a);
    if (b * 2LL <= slots) return launch_early(verify_kernel<T, 2>, dim3(b * 2), VTHREADS, 0, st, a);
    return launch_early(verify_kernel<T, 1>, dim3(b), VTHREADS, 0, st, a);
}

// Whether the kernel can run in clusters of sixteen CTAs, above the portable size.
template <typename T, int W>
bool wide_cluster() {
    const auto kernel = verify_tree_kernel<T, 16, W>;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 16, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(32 * W);
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    const bool ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n >= 1;
    if (!ok) cudaGetLastError();
    return ok;
}

// The same for both forms of the current device, asked once.
template <typename T>
bool wide_clusters() {
    static std::mutex mu;
    static int known[64] = {};   // 1: yes, 2: no
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return false;
    std::lock_guard<std::mutex> lock(mu);
    if (!known[dev]) known[dev] = wide_cluster<T, VWARPS>() && wide_cluster<T, VWIDE>() ? 1 : 2;
    return known[dev] == 1;
}

// The same rule for the cluster, up to sixteen CTAs where a tree has more than eight
// nodes on average, and of twice the warps where such clusters leave half of the SMs
// idle: rows in L2, mean of eight draws, with eight CTAs / sixteen / of sixteen warps:
// 4 x 16 nodes of 32,003 tokens in fp32 13.2 / 9.9 / 9.2 us, 2 x 64 of 131,072 in fp32
// 22.4 / 18.8 / 16.5, 8 x 12 of 32,003 in fp32 13.1 / 11.3 / 11.4.
// The first wave takes as many nodes a sequence (a power of two, at most a CTA each) as
// keep its reads within VWAVE_BYTES, and no more than a tree has on average (with 32, 64 and
// 128 MB, means of six draws: 64 x 32 nodes of 131,072 tokens in bf16 44, 42 and 46 us, in
// fp32 61, 63 and 63; 38 x 32 in bf16 35, 30 and 32; 100 x 16 of 32,003 in fp32 32, 30 and
// 30; 128 x 24 of 65,536 in bf16 39, 40 and 40).
constexpr long long VWAVE_BYTES = 64LL << 20;
template <typename T>
int launch_verify_tree(const TreeVerifyArgs &a, cudaStream_t st) {
    const long long slots = (long long)num_sms() * VRESIDENT;
    const unsigned b = (unsigned)a.num_seqs;
    int ctas = b * 8LL <= slots ? 8 : b * 4LL <= slots ? 4 : b * 2LL <= slots ? 2 : 1;
    int warps = VWARPS;
    if (b * 16LL <= slots && a.num_nodes > 8LL * a.num_seqs && wide_clusters<T>()) {
        ctas = 16;
        if (b * 16LL <= num_sms() / 2) warps = VWIDE;
    }
    const long long row = (long long)a.num_seqs * a.vocab * (long long)sizeof(T);
    int rows = 1;
    while (rows < ctas && 2 * rows * row <= VWAVE_BYTES && (long long)rows * a.num_seqs < a.num_nodes) rows *= 2;
    if (warps == VWIDE) return launch_early(verify_tree_kernel<T, 16, VWIDE>, dim3(b * 16), 32 * VWIDE, 0, st, a, rows);
    if (ctas == 16) return launch_early(verify_tree_kernel<T, 16, VWARPS>, dim3(b * 16), VTHREADS, 0, st, a, rows);
    if (ctas == 8) return launch_early(verify_tree_kernel<T, 8, VWARPS>, dim3(b * 8), VTHREADS, 0, st, a, rows);
    if (ctas == 4) return launch_early(verify_tree_kernel<T, 4, VWARPS>, dim3(b * 4), VTHREADS, 0, st, a, rows);
    if (ctas == 2) return launch_early(verify_tree_kernel<T, 2, VWARPS>, dim3(b * 2), VTHREADS, 0, st, a, rows);
    return launch_early(verify_tree_kernel<T, 1, VWARPS>, dim3(b), VTHREADS, 0, st, a, rows);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_verify_drafts(int32_t *accepted, int32_t *tokens, const void *target_probs, const void *draft_probs,
                                const int32_t *draft_tokens, const int32_t *draft_start, const float *uniform,
                                const float *sample_uniform, int num_seqs, int num_drafts, int max_drafts,
                                int vocab_size, int64_t target_stride, int64_t draft_stride, int probs_dtype,
                                void *stream) {
    if (num_seqs < 0 || num_drafts < 0 || max_drafts < 0 || vocab_size <= 0 || target_stride < vocab_size ||
        (draft_probs && draft_stride < vocab_size) || (num_seqs == 0 && num_drafts > 0))
        return PA_ERR_INVALID_ARG;
    if (probs_dtype != PA_PROBS_F32 && probs_dtype != PA_PROBS_F16 && probs_dtype != PA_PROBS_BF16)
        return PA_ERR_INVALID_ARG;
    // rows, drafts and a sequence's tokens are counted in 32 bits
    if (num_seqs > (1 << 24) || vocab_size > (1 << 30) || num_drafts > (1 << 30) || max_drafts > (1 << 30))
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!accepted || !tokens || !target_probs || !draft_start || !sample_uniform ||
        (num_drafts > 0 && (!draft_tokens || !uniform)))
        return PA_ERR_INVALID_ARG;
    const uintptr_t mis = reinterpret_cast<uintptr_t>(target_probs) | reinterpret_cast<uintptr_t>(draft_probs);
    if (mis & (probs_dtype == PA_PROBS_F32 ? 3u : 1u)) return PA_ERR_INVALID_ARG;
    VerifyArgs a{accepted, tokens, target_probs, draft_probs, draft_tokens, draft_start, uniform, sample_uniform,
                 num_seqs, num_drafts, max_drafts, vocab_size, target_stride, draft_stride};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug_validate())
        if (const int e = validate_starts(draft_start, num_seqs, num_drafts, true, st)) return e;
    if (probs_dtype == PA_PROBS_F16) return launch_verify<__half>(a, st);
    if (probs_dtype == PA_PROBS_BF16) return launch_verify<__nv_bfloat16>(a, st);
    return launch_verify<float>(a, st);
}

extern "C" int pa_verify_tree(int32_t *accepted, int32_t *tokens, int32_t *path, const void *target_probs,
                              const int32_t *node_tokens, const int32_t *parents, const int32_t *tree_start,
                              const float *uniform, int num_seqs, int num_nodes, int max_depth, int vocab_size,
                              int64_t target_stride, int probs_dtype, void *stream) {
    if (num_seqs < 0 || num_nodes < 0 || max_depth < 0 || vocab_size <= 0 || target_stride < vocab_size ||
        (num_seqs == 0 && num_nodes > 0))
        return PA_ERR_INVALID_ARG;
    if (probs_dtype != PA_PROBS_F32 && probs_dtype != PA_PROBS_F16 && probs_dtype != PA_PROBS_BF16)
        return PA_ERR_INVALID_ARG;
    // nodes and a path's tokens are counted in 32 bits
    if (num_seqs > (1 << 24) || vocab_size > (1 << 30) || num_nodes > (1 << 30) || max_depth > (1 << 30))
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!accepted || !tokens || !path || !tree_start ||
        (num_nodes > 0 && (!target_probs || !node_tokens || !parents || !uniform)))
        return PA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(target_probs) & (probs_dtype == PA_PROBS_F32 ? 3u : 1u)) return PA_ERR_INVALID_ARG;
    const TreeVerifyArgs a{accepted, tokens, path, target_probs, node_tokens, parents, tree_start, uniform, num_seqs,
                           num_nodes, max_depth, vocab_size, target_stride};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug_validate())
        if (const int e = validate_starts(tree_start, num_seqs, num_nodes, true, st)) return e;
    if (probs_dtype == PA_PROBS_F16) return launch_verify_tree<__half>(a, st);
    if (probs_dtype == PA_PROBS_BF16) return launch_verify_tree<__nv_bfloat16>(a, st);
    return launch_verify_tree<float>(a, st);
}
