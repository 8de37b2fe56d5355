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
// batch and by latency on a few sequences.  A cluster of eight CTAs takes a
// sequence.  Every CTA finds the number of standing drafts (a warp, one draft a
// lane), then the row's elements are summed in 512 groups, dealt to the
// cluster's 64 warps in turn; the totals are exchanged through distributed
// shared memory, and one warp reads the group again in which the running sum
// passes the drawn height.
//
// Sums: a draw is decided where a running sum over up to a hundred thousand
// terms passes u * total, so sums are carried as an unevaluated pair of floats
// (Knuth's two-sum, exact error terms), and joined in 64 bits over groups.  In
// 64 bits throughout the adds alone would take longer than the reads: this
// GPU's 64-bit rate is two per clock and SM.

#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int VCTAS = 8;                       // CTAs of a sequence's cluster
constexpr int VTHREADS = 256;
constexpr int VWARPS = VTHREADS / 32;
constexpr int VPER = 8;                        // groups per warp
constexpr int VGROUPS = VCTAS * VWARPS * VPER; // groups of a row
constexpr int VCHUNK = 128;                    // elements a warp reads at once, four a lane

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
    __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

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
    __device__ __forceinline__ void at(int v, float pv, float qv, float &s, float &e) const {
        weight(pv, qv, s, e);
        if (v == out) s = e = 0.f;
    }
};

// Sum of the warp's group [lo, hi): four elements a lane and step.  Every
// element belongs to one lane; the sum's order is fixed.
template <typename T, bool QUADS>
__device__ __forceinline__ Sum2 group_sum(const Weights<T> &w, int lo, int hi) {
    const int lane = threadIdx.x & 31;
    Sum2 acc;
    for (int base = lo; base < hi; base += VCHUNK) {
        float p[4], q[4];
        int v[4];
        if (QUADS && base + VCHUNK <= hi) {
            const int at = base + 4 * lane;
            const Quad<T> a = *reinterpret_cast<const Quad<T> *>(w.p + at);
            Quad<T> b{};
            if (w.q) b = *reinterpret_cast<const Quad<T> *>(w.q + at);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = at + k, p[k] = prob(a.v[k]), q[k] = w.q ? prob(b.v[k]) : 0.f;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = base + 32 * k + lane;
                p[k] = v[k] < hi ? prob(w.p[v[k]]) : 0.f;
                q[k] = w.q && v[k] < hi ? prob(w.q[v[k]]) : 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float s, e;
            w.at(v[k], p[k], q[k], s, e);
            acc.add(s, e);
        }
    }
    return acc;
}

// The smallest v in [lo, hi) whose running sum, from `before` on, passes
// `height`; -1 if none does (rounding at the end of a group).  One warp, in
// element order: four consecutive elements a lane.
template <typename T>
__device__ int find_in_group(const Weights<T> &w, int lo, int hi, double before, double height) {
    const int lane = threadIdx.x & 31;
    for (int base = lo; base < hi; base += VCHUNK) {
        float s[4], e[4];
        double mine = 0.0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int v = base + 4 * lane + k;
            s[k] = e[k] = 0.f;
            if (v < hi) w.at(v, prob(w.p[v]), w.q ? prob(w.q[v]) : 0.f, s[k], e[k]);
            mine += (double)s[k] + (double)e[k];
        }
        double upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, mine > 0.0 && before + upto > height);
        if (hit) {
            const int src = __ffs((int)hit) - 1;
            double run = before + (upto - mine);
            int v = -1, last = -1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                run += (double)s[k] + (double)e[k];
                if (s[k] > 0.f) last = base + 4 * lane + k;
                if (v < 0 && s[k] > 0.f && run > height) v = base + 4 * lane + k;
            }
            if (v < 0) v = last;   // the lane's sum passed in another rounding
            return __shfl_sync(0xffffffffu, v, src);
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return -1;
}

// The last v in [lo, hi) of positive weight, -1 if none.  One warp.
template <typename T>
__device__ int last_in_group(const Weights<T> &w, int lo, int hi) {
    int last = -1;
    for (int v = lo + (int)(threadIdx.x & 31); v < hi; v += 32) {
        float s, e;
        w.at(v, prob(w.p[v]), w.q ? prob(w.q[v]) : 0.f, s, e);
        if (s > 0.f) last = v;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, d));
    return last;
}

template <typename T>
__global__ void __cluster_dims__(VCTAS, 1, 1) __launch_bounds__(VTHREADS) verify_kernel(const VerifyArgs a) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    const int seq = blockIdx.x / VCTAS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ double totals[VWARPS * VPER];   // this CTA's groups: [turn][warp]
    __shared__ double part[VGROUPS], sums[VGROUPS];   // the row's groups in order: totals, running sums
    __shared__ double warp_sum[VWARPS];
    __shared__ int s_kept, s_n, s_d0;

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
    int next = -1;
    if (kept >= 0) {   // the same in every CTA of the cluster
        const bool failed = kept < n;
        Weights<T> w;
        w.p = static_cast<const T *>(a.target) + (long long)(d0 + seq + kept) * a.target_stride;
        w.q = failed && a.draft ? static_cast<const T *>(a.draft) + (long long)(d0 + kept) * a.draft_stride : nullptr;
        w.out = failed && !a.draft ? a.draft_tokens[d0 + kept] : -1;
        const int len = ((a.vocab + VGROUPS - 1) / VGROUPS + VCHUNK - 1) / VCHUNK * VCHUNK;   // of a group
        const int used = (a.vocab + len - 1) / len;
        for (int attempt = 0; attempt < 2; ++attempt) {
            const bool quads = ((reinterpret_cast<uintptr_t>(w.p) | (w.q ? reinterpret_cast<uintptr_t>(w.q) : 0)) &
                                (4 * sizeof(T) - 1)) == 0;
#pragma unroll 1
            for (int k = 0; k < VPER; ++k) {
                const int g = (k * VCTAS + rank) * VWARPS + warp;
                const long long lo = (long long)g * len;
                Sum2 acc;
                if (g < used) {
                    const int hi = (int)min((long long)a.vocab, lo + len);
                    acc = quads ? group_sum<T, true>(w, (int)lo, hi) : group_sum<T, false>(w, (int)lo, hi);
                }
                double x = acc.value();
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                if (lane == 0) totals[k * VWARPS + warp] = x;
            }
            cluster.sync();
            // running sums over all groups, the same in every CTA: two a thread
            double x[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int g = 2 * threadIdx.x + k;
                const double *src = cluster.map_shared_rank(totals, (g / VWARPS) % VCTAS);
                part[g] = x[k] = src[g / (VWARPS * VCTAS) * VWARPS + g % VWARPS];
            }
            double upto = x[0] + x[1];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += y;
            }
            if (lane == 31) warp_sum[warp] = upto;
            __syncthreads();
            double before = 0.0;
            for (int k = 0; k < warp; ++k) before += warp_sum[k];
            sums[2 * threadIdx.x] = before + (upto - x[1]);
            sums[2 * threadIdx.x + 1] = before + upto;
            __syncthreads();
            const double total = sums[VGROUPS - 1];
            const bool none = !(total > 0.0);
            cluster.sync();   // no CTA leaves, or sums again, while another reads its totals
            if (none && attempt == 0 && failed && total == 0.0) {   // nothing is left of p: draw from p itself
                w.q = nullptr;
                w.out = -1;
                continue;
            }
            if (rank == 0 && warp == 0 && !none && isfinite(total)) {
                const double height = (double)a.sample[seq] * total;
                // the first group whose running sum passes, else the last with any weight
                int first = VGROUPS, last = 0;
                for (int g = lane; g < VGROUPS; g += 32) {
                    if (part[g] > 0.0) {
                        last = g;
                        if (sums[g] > height && first == VGROUPS) first = g;
                    }
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) {
                    first = min(first, __shfl_xor_sync(0xffffffffu, first, d));
                    last = max(last, __shfl_xor_sync(0xffffffffu, last, d));
                }
                const int g = first < VGROUPS ? first : last;
                const int lo = g * len, hi = min(a.vocab, lo + len);
                next = first < VGROUPS ? find_in_group<T>(w, lo, hi, g ? sums[g - 1] : 0.0, height) : -1;
                if (next < 0) next = last_in_group<T>(w, lo, hi);
            }
            break;
        }
    }
    if (rank == 0 && warp == 0) {
        for (int j = lane; j <= a.max_drafts; j += 32)
            out[j] = kept < 0 ? -1 : j < kept ? a.draft_tokens[d0 + j] : j == kept ? next : -1;
        if (lane == 0) a.accepted[seq] = kept;
    }
}

template <typename T>
int launch_verify(const VerifyArgs &a, cudaStream_t st) {
    verify_kernel<T><<<(unsigned)a.num_seqs * VCTAS, VTHREADS, 0, st>>>(a);
    return cuda_status(cudaGetLastError());
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
    if (probs_dtype == PA_PROBS_F16) return launch_verify<__half>(a, st);
    if (probs_dtype == PA_PROBS_BF16) return launch_verify<__nv_bfloat16>(a, st);
    return launch_verify<float>(a, st);
}
