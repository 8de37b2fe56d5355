// Attention over the latent cache in the absorbed form.
#include <cmath>

#include "decode_common.cuh"
#include "latent.h"

namespace pa {
namespace {

struct LatentArgs {
    uint16_t *out;
    const uint16_t *query;
    const uint8_t *cache;
    const int32_t *block_tables, *context_lens, *query_start;
    WsHeader *hdr;
    int num_seqs, num_query_tokens, H, bs, mbps, max_context_len;
    long long num_blocks;
    float scale_log2;
};

template <int KV>
__device__ __forceinline__ float to_float(uint16_t b) {
    if constexpr (KV == PA_KV_F16)
        return __half2float(__ushort_as_half(b));
    else
        return __uint_as_float((uint32_t)b << 16);
}
template <int KV>
__device__ __forceinline__ uint16_t to_bits(float x) {
    if constexpr (KV == PA_KV_F16)
        return __half_as_ushort(__float2half_rn(x));
    else
        return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// One CTA per query row, a token per warp and step.
template <int KV>
__global__ void __launch_bounds__(256) latent_simple_kernel(const LatentArgs a) {
    const int h = blockIdx.x % a.H, qt = blockIdx.x / a.H;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->error = 0;
    __shared__ float sm[8], sl[8], so[8][LC];
    int seq = qt, L = 0, vis = 0;
    bool bad = false;
    if (a.query_start) {
        bool order = a.query_start[0] == 0 && a.query_start[a.num_seqs] == a.num_query_tokens;
        for (int i = threadIdx.x; i < a.num_seqs; i += blockDim.x)
            if (a.query_start[i] > a.query_start[i + 1]) order = false;
        bad = !__syncthreads_and(order);
        int lo = 0, hi = a.num_seqs;
        while (!bad && hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.query_start[mid] <= qt) lo = mid; else hi = mid;
        }
        seq = lo;
    }
    if (!bad) {
        L = a.context_lens[seq];
        const int q0 = a.query_start ? a.query_start[seq] : qt, T = a.query_start ? a.query_start[seq + 1] - q0 : 1;
        bad = L < 0 || L > a.max_context_len || (long long)L > (long long)a.mbps * a.bs ||
              (a.query_start && T > L);
        vis = L - T + (qt - q0) + 1;
        if (!a.query_start) vis = L;
    }
    const uint16_t *qr = a.query + (long long)blockIdx.x * LROW;
    float q[18], o[16], m = -INFINITY, l = 0.f;
    for (int k = 0; k < 18; ++k) q[k] = to_float<KV>(qr[32 * k + lane]);
    for (int k = 0; k < 16; ++k) o[k] = 0.f;
    for (int t = warp; !bad && t < vis; t += 8) {
        const long long blk = a.block_tables[(long long)seq * a.mbps + t / a.bs];
        float x[18];
        if (blk < 0 || blk >= a.num_blocks) {
            for (int k = 0; k < 18; ++k) x[k] = __int_as_float(0x7fc00000);
        } else {
            const long long slot = blk * a.bs + t % a.bs;
            if constexpr (KV == PA_KV_FP8_E4M3) {
                const uint8_t *row = a.cache + slot * LROW8;
                for (int k = 0; k < 16; ++k) {
                    const uint32_t c = row[32 * k + lane];
                    const float s = *reinterpret_cast<const float *>(row + L8_SCALE + 4 * (k / 4));
                    x[k] = __uint_as_float(latent_codes_to_bf16(c, s).x << 16);
                }
                for (int k = 0; k < 2; ++k)
                    x[16 + k] = to_float<KV>(*reinterpret_cast<const uint16_t *>(row + L8_ROPE + 2 * (32 * k + lane)));
            } else {
                const uint16_t *row = reinterpret_cast<const uint16_t *>(a.cache) + slot * LROW;
                for (int k = 0; k < 18; ++k) x[k] = to_float<KV>(row[32 * k + lane]);
            }
        }
        float s = 0.f;
        for (int k = 0; k < 18; ++k) s = fmaf(q[k], x[k], s);
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale_log2;
        const float nm = fmaxf(m, s), al = fast_exp2(m - nm), p = s != s ? s : fast_exp2(s - nm);
        l = l * al + p;
        for (int k = 0; k < 16; ++k) o[k] = o[k] * al + p * x[k];
        m = nm;
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
    for (int k = 0; k < 16; ++k) so[warp][32 * k + lane] = o[k];
    __syncthreads();
    float M = -INFINITY, den = 0.f;
    for (int w = 0; w < 8; ++w) M = fmaxf(M, sm[w]);
    for (int w = 0; w < 8; ++w)
        if (sl[w] != 0.f) den += sl[w] * fast_exp2(sm[w] - M);
    for (int d = threadIdx.x; d < LC; d += 256) {
        float v = 0.f;
        for (int w = 0; w < 8; ++w)
            if (sl[w] != 0.f) v += so[w][d] * fast_exp2(sm[w] - M);
        v = bad ? __int_as_float(0x7fc00000) : vis <= 0 ? 0.f : v / den;
        a.out[(long long)blockIdx.x * LC + d] = to_bits<KV>(v);
    }
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_latent_attention_workspace_size(int num_seqs, int num_query_tokens, int num_heads,
                                                     int max_context_len) {
    if (num_seqs < 0 || num_query_tokens < 0 || num_heads <= 0 || num_heads > 128 || max_context_len < 0) return 0;
    return 4096;
}

extern "C" int pa_latent_attention(void *out, const void *query, const void *cache, const int32_t *block_tables,
                                   const int32_t *context_lens, const int32_t *query_start, int num_seqs,
                                   int num_query_tokens, int num_heads, int block_size, int64_t num_blocks,
                                   int max_blocks_per_seq, int max_context_len, float scale, int kv_dtype,
                                   void *workspace, size_t workspace_bytes, void *stream) {
    if (num_seqs < 0 || num_query_tokens < 0 || num_heads <= 0 || max_context_len < 0 || max_blocks_per_seq <= 0 ||
        num_blocks <= 0 || block_size <= 0 || !std::isfinite(scale) || !(scale > 0.f) ||
        latent_row_bytes(kv_dtype) == 0 || (num_seqs == 0 && num_query_tokens > 0) ||
        (!query_start && num_query_tokens != num_seqs))
        return PA_ERR_INVALID_ARG;
    if (!latent_block_size_ok(block_size) || num_heads > 128 || num_blocks > (1LL << 31) / block_size)
        return PA_ERR_UNSUPPORTED;
    if (num_query_tokens == 0) return PA_OK;
    if (!out || !query || !cache || !block_tables || !context_lens || !aligned16(out) || !aligned16(query) ||
        !aligned16(cache))
        return PA_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < pa_latent_attention_workspace_size(num_seqs, num_query_tokens, num_heads, max_context_len))
        return PA_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    LatentArgs a{static_cast<uint16_t *>(out), static_cast<const uint16_t *>(query),
                 static_cast<const uint8_t *>(cache), block_tables, context_lens, query_start,
                 static_cast<WsHeader *>(workspace), num_seqs, num_query_tokens, num_heads, block_size,
                 max_blocks_per_seq, max_context_len, num_blocks, scale * 1.4426950408889634f};
    const unsigned grid = (unsigned)num_query_tokens * num_heads;
    if (kv_dtype == PA_KV_F16) latent_simple_kernel<PA_KV_F16><<<grid, 256, 0, st>>>(a);
    else if (kv_dtype == PA_KV_BF16) latent_simple_kernel<PA_KV_BF16><<<grid, 256, 0, st>>>(a);
    else latent_simple_kernel<PA_KV_FP8_E4M3><<<grid, 256, 0, st>>>(a);
    return cuda_status(cudaGetLastError());
}
