// Attention of trees of drafted tokens over the paged cache: a node sees the
// context before the tree, itself and its ancestors.
//
// A warp takes one query row (a node's head) and walks the positions that it
// sees, with a running maximum and sum.

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>
#include <vector>

#include "decode_common.cuh"

namespace pa {
namespace {

struct TreeArgs {
    uint16_t *out;
    const uint16_t *query;
    const void *k_cache, *v_cache;
    const int32_t *block_tables, *context_lens, *query_start, *parents;
    WsHeader *hdr;
    int num_seqs, num_query_tokens, Hq, Hkv, G, bs, mbps, max_ctx;
    long long num_blocks;
    float scale_log2, v_scale;
};

template <int KV>
__device__ __forceinline__ float element(const void *cache, long long at) {
    if constexpr (KV == PA_KV_F16) return __half2float(static_cast<const __half *>(cache)[at]);
    if constexpr (KV == PA_KV_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(cache)[at]);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t *>(cache)[at], __NV_E4M3);
    return __half2float(__half(h));
}

constexpr int TS_WARPS = 8;

template <int KV, int D>
__global__ void __launch_bounds__(32 * TS_WARPS) tree_simple_kernel(const TreeArgs a) {
    constexpr int E = D / 32;
    __shared__ uint32_t sees[TS_WARPS][PA_TREE_MAX_NODES / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_release();
    grid_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->error = PA_OK;
    bool ok = a.query_start[0] == 0 && a.query_start[a.num_seqs] == a.num_query_tokens;
    for (int i = threadIdx.x; i < a.num_seqs; i += blockDim.x) ok = ok && a.query_start[i] <= a.query_start[i + 1];
    ok = __syncthreads_and(ok);
    const long long row = blockIdx.x * (long long)TS_WARPS + warp;
    if (row >= (long long)a.num_query_tokens * a.Hq) return;
    const int tok = (int)(row / a.Hq), h = (int)(row - (long long)tok * a.Hq), g = h / a.G;
    float o[E], q[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f, q[e] = 0.f;
    bool bad = !ok;
    if (ok) {
        int lo = 0, hi = a.num_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.query_start[mid] <= tok) lo = mid; else hi = mid;
        }
        const int q0 = a.query_start[lo], T = a.query_start[lo + 1] - q0, L = a.context_lens[lo];
        bad = L < 0 || L > a.max_ctx || L > (long long)a.mbps * a.bs || T > L || T > PA_TREE_MAX_NODES;
        if (!bad) {
            if (lane < PA_TREE_MAX_NODES / 32) sees[warp][lane] = 0;
            __syncwarp();
            if (lane == 0)
                for (int n = tok - q0; n >= 0;) {
                    sees[warp][n >> 5] |= 1u << (n & 31);
                    const int p = a.parents[q0 + n];
                    if (p < -1 || p >= n) {
                        bad = true;
                        break;
                    }
                    n = p;
                }
            __syncwarp();
            bad = __any_sync(0xffffffffu, bad);
#pragma unroll
            for (int e = 0; e < E; ++e) q[e] = element<KV == PA_KV_BF16 ? PA_KV_BF16 : PA_KV_F16>(a.query, row * D + lane * E + e);
            for (int t = 0; !bad && t < L; ++t) {
                const long long blk = a.block_tables[(long long)lo * a.mbps + t / a.bs];
                if (blk < 0 || blk >= a.num_blocks) {
                    bad = true;
                    break;
                }
                const int n = t - (L - T);
                if (n >= 0 && !(sees[warp][n >> 5] >> (n & 31) & 1u)) continue;
                const long long at = ((blk * a.Hkv + g) * a.bs + t % a.bs) * D + lane * E;
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) s = fmaf(q[e], element<KV>(a.k_cache, at + e), s);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                s *= a.scale_log2;
                const float nm = fmaxf(m, s), mu = nm == -INFINITY ? 0.f : nm, old = exp2f(m - mu), p = exp2f(s - mu);
                m = nm;
                l = l * old + p;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = o[e] * old + p * element<KV>(a.v_cache, at + e);
            }
        }
    }
    const float inv = bad ? __int_as_float(0x7fc00000) : a.v_scale / l;
#pragma unroll
    for (int e = 0; e < E; ++e) a.out[row * D + lane * E + e] = out_bits<KV>(o[e] * inv);
}

template <int KV, int D>
int launch_tree(const TreeArgs &a, cudaStream_t st) {
    const long long rows = (long long)a.num_query_tokens * a.Hq;
    return launch_early(tree_simple_kernel<KV, D>, dim3((unsigned)((rows + TS_WARPS - 1) / TS_WARPS)), 32 * TS_WARPS, 0, st,
                        a);
}

// PA_DEBUG_VALIDATE: lengths, row offsets, block ids and parents.
int validate_tree(const TreeArgs &a, cudaStream_t st) try {
    if (const int e = validate_starts(a.query_start, a.num_seqs, a.num_query_tokens, true, st)) return e;
    const size_t n = (size_t)a.num_seqs;
    std::vector<int32_t> lens(n), qs(n + 1), parents((size_t)a.num_query_tokens);
    std::vector<int64_t> last(n);
    if (const int e = copy_to_host(lens.data(), a.context_lens, 4 * n, st)) return e;
    if (const int e = copy_to_host(qs.data(), a.query_start, 4 * (n + 1), st)) return e;
    if (const int e = copy_to_host(parents.data(), a.parents, 4 * parents.size(), st)) return e;
    for (size_t i = 0; i < n; ++i) {
        const int T = qs[i + 1] - qs[i];
        if (lens[i] < 0 || lens[i] > a.max_ctx || T > lens[i] || T > PA_TREE_MAX_NODES) return PA_ERR_INVALID_ARG;
        for (int j = 0; j < T; ++j)
            if (parents[(size_t)(qs[i] + j)] < -1 || parents[(size_t)(qs[i] + j)] >= j) return PA_ERR_INVALID_ARG;
        last[i] = lens[i];
    }
    return validate_tables(a.block_tables, last.data(), a.num_seqs, a.mbps, a.bs, a.num_blocks, st);
} catch (...) {   // no host memory for the check
    return PA_ERR_STATE;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_attention_tree_workspace_size(int num_seqs, int num_query_tokens, int num_heads, int num_kv_heads,
                                                   int head_dim, int max_context_len) {
    if (num_seqs < 0 || num_query_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        num_heads % num_kv_heads != 0 || head_dim <= 0 || max_context_len < 0)
        return 0;
    return 256;
}

extern "C" int pa_attention_tree(void *out, const void *query, const void *k_cache, const void *v_cache,
                                 const int32_t *block_tables, const int32_t *context_lens, const int32_t *query_start,
                                 const int32_t *parents, int num_seqs, int num_query_tokens, int num_heads,
                                 int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                                 int max_blocks_per_seq, int max_context_len, float scale, int kv_dtype, float k_scale,
                                 float v_scale, void *workspace, size_t workspace_bytes, void *stream) {
    if (num_seqs < 0 || num_query_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        num_heads % num_kv_heads != 0 || max_context_len < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
        !std::isfinite(scale) || !(scale > 0.f))
        return PA_ERR_INVALID_ARG;
    const int G = num_heads / num_kv_heads;
    const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
    if (!fp8 && kv_dtype != PA_KV_F16 && kv_dtype != PA_KV_BF16) return PA_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || (block_size != 8 && block_size != 16 && block_size != 32) || G > 16)
        return PA_ERR_UNSUPPORTED;
    if (fp8) {
        if (!std::isfinite(k_scale) || !(k_scale > 0.f) || !std::isfinite(v_scale) || !(v_scale > 0.f))
            return PA_ERR_INVALID_ARG;
        if (head_dim != 128) return PA_ERR_UNSUPPORTED;
    }
    if (num_query_tokens == 0) return PA_OK;
    if (num_seqs == 0) return PA_ERR_INVALID_ARG;
    if (!out || !query || !k_cache || !v_cache || !block_tables || !context_lens || !query_start || !parents)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache))
        return PA_ERR_INVALID_ARG;
    if ((long long)num_blocks * num_kv_heads * block_size >= (1LL << 31) ||
        (long long)num_query_tokens * num_heads >= (1LL << 31))
        return PA_ERR_UNSUPPORTED;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < pa_attention_tree_workspace_size(num_seqs, num_query_tokens, num_heads, num_kv_heads,
                                                           head_dim, max_context_len))
        return PA_ERR_WORKSPACE;
    TreeArgs a{};
    a.out = static_cast<uint16_t *>(out);
    a.query = static_cast<const uint16_t *>(query);
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.parents = parents;
    a.hdr = static_cast<WsHeader *>(workspace);
    a.num_seqs = num_seqs;
    a.num_query_tokens = num_query_tokens;
    a.Hq = num_heads;
    a.Hkv = num_kv_heads;
    a.G = G;
    a.bs = block_size;
    a.mbps = max_blocks_per_seq;
    a.max_ctx = max_context_len;
    a.num_blocks = num_blocks;
    a.scale_log2 = scale * (fp8 ? k_scale : 1.f) * 1.4426950408889634f;
    a.v_scale = fp8 ? v_scale : 1.f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug_validate())
        if (const int e = validate_tree(a, st)) return e;
    if (fp8) return launch_tree<PA_KV_FP8_E4M3, 128>(a, st);
    if (kv_dtype == PA_KV_BF16)
        return head_dim == 128 ? launch_tree<PA_KV_BF16, 128>(a, st) : launch_tree<PA_KV_BF16, 64>(a, st);
    return head_dim == 128 ? launch_tree<PA_KV_F16, 128>(a, st) : launch_tree<PA_KV_F16, 64>(a, st);
}
