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

#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int VMAX_CTAS = 8;                   // CTAs of a sequence's cluster, at most
constexpr int VTHREADS = 256;
constexpr int VWARPS = VTHREADS / 32;
constexpr int VRESIDENT = 4;                   // CTAs an SM holds (64 registers a thread)
constexpr int VCHUNK = 128;                    // elements a warp reads at once, four a lane
constexpr int VBATCH = 4;                      // chunks on their way at once
static_assert(VMAX_CTAS * VWARPS == 64, "at most two slices a lane of the collecting warp");

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

template <typename T, int VCTAS>
__global__ void __cluster_dims__(VCTAS, 1, 1) __launch_bounds__(VTHREADS, VRESIDENT) verify_kernel(const VerifyArgs a) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    const int seq = blockIdx.x / VCTAS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ Sum2 totals[VWARPS];   // this CTA's slices; then, in rank 0, the parts of one
    __shared__ Sum2 s_before;         // rank 0: the sum before the slice that passes
    __shared__ Height s_height;
    __shared__ int s_slice;           // rank 0: that slice; -1: no token; -2: draw from p itself
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
        constexpr int VSLICES = VCTAS * VWARPS;
        const int len = ((a.vocab + VSLICES - 1) / VSLICES + VCHUNK - 1) / VCHUNK * VCHUNK;   // of a slice
        for (int attempt = 0; attempt < 2; ++attempt) {
            const long long from = (long long)(rank * VWARPS + warp) * len;
            const int lo = (int)min((long long)a.vocab, from), hi = (int)min((long long)a.vocab, from + len);
            const Sum2 mine = range_sum(w, lo, hi);
            if (lane == 0) totals[warp] = mine;
            cluster.sync();
            if (rank == 0 && warp == 0) {   // lane l: slices 2 l and 2 l + 1
                Sum2 x0, x1;
                if (2 * lane < VSLICES) {
                    const Sum2 *src = cluster.map_shared_rank(totals, 2 * lane / VWARPS) + 2 * lane % VWARPS;
                    x0 = src[0];
                    x1 = src[1];
                }
                Sum2 both = x0;
                both.add(x1);
                const Sum2 upto = warp_scan(both);
                const Sum2 all{__shfl_sync(0xffffffffu, upto.hi, 31), __shfl_sync(0xffffffffu, upto.lo, 31)};
                const float total = all.value();   // the same in all lanes
                int slice = attempt == 0 && failed && total == 0.f ? -2 : -1;
                if (total > 0.f && isfinite(total)) {
                    const Height height(all, a.sample[seq]);
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
                        s_before = slice & 1 ? run1 : run;
                        s_height = height;
                    }
                }
                if (lane == 0) s_slice = slice;
            }
            cluster.sync();   // rank 0 has read every CTA's totals and decided
            const int slice = *cluster.map_shared_rank(&s_slice, 0);
            if (len <= VBATCH * VCHUNK) {   // short slices: the warp that summed it finds the element
                if (slice == rank * VWARPS + warp) {
                    const int v = find_in_range(w, lo, hi, *cluster.map_shared_rank(&s_before, 0),
                                                *cluster.map_shared_rank(&s_height, 0));
                    if (lane == 0) *cluster.map_shared_rank(&s_next, 0) = v;
                }
            } else if (rank == 0 && slice >= 0) {   // the slice again, in parts
                const int first = slice * len, part = (len / VCHUNK + VWARPS - 1) / VWARPS * VCHUNK;
                const int plo = min(a.vocab, min(first + len, first + warp * part));
                const int phi = min(a.vocab, min(first + len, plo + part));
                const Sum2 mine = range_sum(w, plo, phi);
                if (lane == 0) totals[warp] = mine;
                __syncthreads();
                Sum2 run = s_before, before = run;
                int at = -1;       // the first part that passes, else the last of any weight
                bool passed = false;
                for (int k = 0; k < VWARPS; ++k) {
                    const Sum2 x = totals[k];
                    Sum2 after = run;
                    after.add(x);
                    if (!passed && x.any()) {
                        at = k;
                        before = run;
                        passed = s_height.passed_by(after);
                    }
                    run = after;
                }
                if (warp == at) {
                    const int v = find_in_range(w, plo, phi, before, s_height);
                    if (lane == 0) s_next = v;
                }
            }
            if (slice != -2) break;
            w = Weights<T>(p, nullptr, -1);
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
    if (num_seqs > (1 << 24) || vocab_size > (1 << 30)) return PA_ERR_UNSUPPORTED;
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
