// Attention in the expanded form.
#include <cmath>

#include "decode_common.cuh"
#include "latent.h"

namespace pa {
namespace {

constexpr int EN = 128, ER = PA_LATENT_ROPE_DIM, EQ = EN + ER, EV = 128;

struct ExpandedArgs {
    uint16_t *out;
    const uint16_t *query, *k_nope, *k_rope, *value;
    const int32_t *query_start, *kv_start;
    WsHeader *hdr;
    int num_seqs, num_query_tokens, num_kv_tokens, H;
    long long kt, kh, rt, vt, vh;
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

template <int KV>
__global__ void __launch_bounds__(256) expanded_simple_kernel(const ExpandedArgs a) {
    const int h = blockIdx.x % a.H, qt = blockIdx.x / a.H;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->error = 0;
    __shared__ float sm[8], sl[8], so[8][EV];
    bool order = a.query_start[0] == 0 && a.query_start[a.num_seqs] == a.num_query_tokens && a.kv_start[0] == 0 &&
                 a.kv_start[a.num_seqs] == a.num_kv_tokens;
    for (int i = threadIdx.x; i < a.num_seqs; i += blockDim.x)
        if (a.query_start[i] > a.query_start[i + 1] || a.kv_start[i] > a.kv_start[i + 1]) order = false;
    bool bad = !__syncthreads_and(order);
    int lo = 0, hi = a.num_seqs;
    while (!bad && hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.query_start[mid] <= qt) lo = mid; else hi = mid;
    }
    int vis = 0;
    long long k0 = 0;
    if (!bad) {
        const int T = a.query_start[lo + 1] - a.query_start[lo];
        const int L = a.kv_start[lo + 1] - a.kv_start[lo];
        k0 = a.kv_start[lo];
        bad = T > L;
        vis = L - T + (qt - a.query_start[lo]) + 1;
    }
    const uint16_t *qr = a.query + (long long)blockIdx.x * EQ;
    float q[6], o[4], m = -INFINITY, l = 0.f;
    for (int k = 0; k < 6; ++k) q[k] = to_float<KV>(qr[32 * k + lane]);
    for (int k = 0; k < 4; ++k) o[k] = 0.f;
    for (int t = warp; !bad && t < vis; t += 8) {
        const uint16_t *kn = a.k_nope + (k0 + t) * a.kt + h * a.kh, *kr = a.k_rope + (k0 + t) * a.rt;
        const uint16_t *vr = a.value + (k0 + t) * a.vt + h * a.vh;
        float s = 0.f;
        for (int k = 0; k < 4; ++k) s = fmaf(q[k], to_float<KV>(kn[32 * k + lane]), s);
        for (int k = 0; k < 2; ++k) s = fmaf(q[4 + k], to_float<KV>(kr[32 * k + lane]), s);
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale_log2;
        const float nm = fmaxf(m, s), al = fast_exp2(m - nm), p = s != s ? s : fast_exp2(s - nm);
        l = l * al + p;
        for (int k = 0; k < 4; ++k) o[k] = o[k] * al + p * to_float<KV>(vr[32 * k + lane]);
        m = nm;
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
    for (int k = 0; k < 4; ++k) so[warp][32 * k + lane] = o[k];
    __syncthreads();
    float M = -INFINITY, den = 0.f;
    for (int w = 0; w < 8; ++w) M = fmaxf(M, sm[w]);
    for (int w = 0; w < 8; ++w)
        if (sl[w] != 0.f) den += sl[w] * fast_exp2(sm[w] - M);
    for (int d = threadIdx.x; d < EV; d += 256) {
        float v = 0.f;
        for (int w = 0; w < 8; ++w)
            if (sl[w] != 0.f) v += so[w][d] * fast_exp2(sm[w] - M);
        a.out[(long long)blockIdx.x * EV + d] = to_bits<KV>(bad ? __int_as_float(0x7fc00000) : v / den);
    }
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_latent_attention_expanded_workspace_size(int num_seqs, int num_query_tokens, int num_heads) {
    if (num_seqs < 0 || num_query_tokens < 0 || num_heads <= 0) return 0;
    return 4096;
}

extern "C" int pa_latent_attention_expanded(void *out, const void *query, const void *k_nope, const void *k_rope,
                                            const void *value, const int32_t *query_start, const int32_t *kv_start,
                                            int num_seqs, int num_query_tokens, int num_kv_tokens, int num_heads,
                                            int64_t k_token_stride, int64_t k_head_stride, int64_t rope_stride,
                                            int64_t v_token_stride, int64_t v_head_stride, float scale, int dtype,
                                            void *workspace, size_t workspace_bytes, void *stream) {
    if (num_seqs < 0 || num_query_tokens < 0 || num_kv_tokens < 0 || num_heads <= 0 || !std::isfinite(scale) ||
        !(scale > 0.f) || (dtype != PA_KV_F16 && dtype != PA_KV_BF16) || (num_seqs == 0 && num_query_tokens > 0) ||
        k_head_stride < EN || v_head_stride < EV || rope_stride < ER || k_token_stride < EN || v_token_stride < EV ||
        (k_token_stride | k_head_stride | rope_stride | v_token_stride | v_head_stride) % 8 != 0)
        return PA_ERR_INVALID_ARG;
    if (num_query_tokens == 0) return PA_OK;
    if (!out || !query || !query_start || !kv_start || !aligned16(out) || !aligned16(query) ||
        (num_kv_tokens > 0 && (!k_nope || !k_rope || !value)) || !aligned16(k_nope) || !aligned16(k_rope) ||
        !aligned16(value))
        return PA_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < pa_latent_attention_expanded_workspace_size(num_seqs, num_query_tokens, num_heads))
        return PA_ERR_WORKSPACE;
    ExpandedArgs a{static_cast<uint16_t *>(out), static_cast<const uint16_t *>(query),
                   static_cast<const uint16_t *>(k_nope), static_cast<const uint16_t *>(k_rope),
                   static_cast<const uint16_t *>(value), query_start, kv_start, static_cast<WsHeader *>(workspace),
                   num_seqs, num_query_tokens, num_kv_tokens, num_heads, k_token_stride, k_head_stride, rope_stride,
                   v_token_stride, v_head_stride, scale * 1.4426950408889634f};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)num_query_tokens * num_heads;
    if (dtype == PA_KV_F16) expanded_simple_kernel<PA_KV_F16><<<grid, 256, 0, st>>>(a);
    else expanded_simple_kernel<PA_KV_BF16><<<grid, 256, 0, st>>>(a);
    return cuda_status(cudaGetLastError());
}
