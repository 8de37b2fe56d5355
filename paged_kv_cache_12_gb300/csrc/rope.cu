// KV write with the position rotation applied on the way: keys turned and
// scattered into their slots, values beside them, queries turned into query_out.
//
// A rotation by angle a takes the pair (x, y) to (x cos a - y sin a,
// y cos a + x sin a).  The angle of a pair is a position (an integer, one for each
// axis) times a frequency.  A position of a million times a frequency of one has
// lost the turn's fraction in 32 bits, so the angle is taken in turns in 64 bits
// (position * inv_freq / 2 pi), reduced to its fraction exactly, and its sine and
// cosine computed in 32.  All heads of a token share its angles: a CTA computes
// them once a token, in shared memory.
//
// Sources: the new token goes into the free slot of the sequence's current block
// ("PagedAttention : comment optimiser la memoire GPU lors de l'inference des
// LLM", deeplearn.tn, section "Un exemple concret d'allocation"); the pages do not
// say how a key gets its position.

#include <algorithm>
#include <cmath>

#include "common.cuh"

namespace pa {
namespace {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_MAX_DIM = 512;   // rotary elements of a head: a thread per pair
static_assert(ROPE_MAX_DIM / 2 <= ROPE_THREADS, "a thread per pair");

struct RopeArgs {
    uint16_t *query_out;
    const uint16_t *query, *key, *value;
    const int32_t *positions;
    const float *inv_freq;
    const int32_t *pair_axis;
    const int64_t *slot_mapping;
    void *k_cache, *v_cache;
    int num_tokens, hq, hk, d, rope_dim, num_axes, interleaved, block_size;
    long long query_stride, query_out_stride, key_stride, value_stride, num_slots;
    float kinv, vinv;
};

template <int KV>
__device__ __forceinline__ float2 floats_of(uint32_t pair) {
    if constexpr (KV == PA_KV_BF16)
        return make_float2(__uint_as_float(pair << 16), __uint_as_float(pair & 0xffff0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2 *>(&pair));
}
template <int KV>
__device__ __forceinline__ uint32_t bits_of(float lo, float hi) {
    if constexpr (KV == PA_KV_BF16)
        return pack_bf162(lo, hi);
    else
        return pack_half2(lo, hi);
}

template <int KV>
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = floats_of<KV>(w[k]);
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
    }
}
template <int KV>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(bits_of<KV>(x[0], x[1]), bits_of<KV>(x[2], x[3]), bits_of<KV>(x[4], x[5]),
                      bits_of<KV>(x[6], x[7]));
}
// Eight floats -> eight E4M3 codes of fl32(x * inv), as kv_write_fp8_kernel makes them.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        c[k] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
            make_float2(__fmul_rn(x[2 * k], inv), __fmul_rn(x[2 * k + 1], inv)), __NV_SATFINITE, __NV_E4M3));
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Eight elements at element offset `at` of a cache.
template <int KV>
__device__ __forceinline__ void store_cache(void *cache, long long at, const float (&x)[8], float inv) {
    if constexpr (KV == PA_KV_FP8_E4M3)
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(cache) + at) = codes8(x, inv);
    else
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(cache) + at) = pack8<KV>(x);
}

// A CTA takes every gridDim-th token.  A thread's piece of work is eight
// elements of a head, or, where a pair's halves lie rope_dim / 2 apart, eight
// and their eight partners.
template <int KV>
__global__ void __launch_bounds__(ROPE_THREADS) rope_write_kernel(const RopeArgs a) {
    __shared__ float2 turn[ROPE_MAX_DIM / 2];   // cosine and sine of every pair
    const int pairs = a.rope_dim / 2, tid = threadIdx.x;
    const int turned = a.interleaved ? a.rope_dim / 8 : a.rope_dim / 16;   // pieces of a head that turn
    const int pieces = turned + (a.d - a.rope_dim) / 8;                    // of a query or key head
    const int vecs = a.d / 8;                                              // of a value head
    const int n_turn = (a.hq + a.hk) * pieces, n_all = n_turn + a.hk * vecs;
    grid_release();
    grid_wait();
    double per_turn = 0.0;   // this thread's pair: turns for each step of its axis
    int axis = 0;
    if (tid < pairs) {
        per_turn = (double)a.inv_freq[tid] * 0.15915494309189535;   // 1 / (2 pi)
        if (a.pair_axis) axis = a.pair_axis[tid];
    }
    for (int t = blockIdx.x; t < a.num_tokens; t += gridDim.x) {
        const long long slot = a.slot_mapping[t];
        if (slot < 0 || slot >= a.num_slots) continue;   // padding (the whole CTA)
        __syncthreads();   // the last token's angles have been used
        if (tid < pairs) {
            float2 cs = make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
            if (axis >= 0 && axis < a.num_axes) {
                const double x = per_turn * (double)a.positions[(long long)axis * a.num_tokens + t];
                sincospif(2.f * (float)(x - rint(x)), &cs.y, &cs.x);
            }
            turn[tid] = cs;
        }
        __syncthreads();
        const long long blk = slot / a.block_size, off = slot - blk * a.block_size;
        for (int i = tid; i < n_all; i += ROPE_THREADS) {
            if (i >= n_turn) {   // a value's piece
                const int h = (i - n_turn) / vecs, v = (i - n_turn) - h * vecs;
                const uint4 raw = *reinterpret_cast<const uint4 *>(a.value + (long long)t * a.value_stride +
                                                                   (long long)h * a.d + 8 * v);
                const long long at = ((blk * a.hk + h) * a.block_size + off) * a.d + 8 * v;
                if constexpr (KV == PA_KV_FP8_E4M3) {
                    float x[8];
                    unpack8<KV>(raw, x);
                    store_cache<KV>(a.v_cache, at, x, a.vinv);
                } else {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.v_cache) + at) = raw;
                }
                continue;
            }
            const int head = i / pieces, p = i - head * pieces;
            const bool is_key = head >= a.hq;
            const int h = is_key ? head - a.hq : head;
            const uint16_t *src = is_key ? a.key + (long long)t * a.key_stride + (long long)h * a.d
                                         : a.query + (long long)t * a.query_stride + (long long)h * a.d;
            // first element of the piece, and of its partner's
            const int e = p < turned ? 8 * p : a.rope_dim + 8 * (p - turned);
            const bool two = p < turned && !a.interleaved;
            float x[8], y[8];
            unpack8<KV>(*reinterpret_cast<const uint4 *>(src + e), x);
            if (two) {
                unpack8<KV>(*reinterpret_cast<const uint4 *>(src + e + pairs), y);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 cs = turn[e + k];
                    const float u = x[k], w = y[k];
                    x[k] = fmaf(u, cs.x, -(w * cs.y));
                    y[k] = fmaf(w, cs.x, u * cs.y);
                }
            } else if (p < turned) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 cs = turn[e / 2 + k];
                    const float u = x[2 * k], w = x[2 * k + 1];
                    x[2 * k] = fmaf(u, cs.x, -(w * cs.y));
                    x[2 * k + 1] = fmaf(w, cs.x, u * cs.y);
                }
            }
            if (is_key) {
                const long long at = ((blk * a.hk + h) * a.block_size + off) * a.d + e;
                store_cache<KV>(a.k_cache, at, x, a.kinv);
                if (two) store_cache<KV>(a.k_cache, at + pairs, y, a.kinv);
            } else {
                uint16_t *dst = a.query_out + (long long)t * a.query_out_stride + (long long)h * a.d + e;
                *reinterpret_cast<uint4 *>(dst) = pack8<KV>(x);
                if (two) *reinterpret_cast<uint4 *>(dst + pairs) = pack8<KV>(y);
            }
        }
    }
}

template <int KV>
int launch_rope(const RopeArgs &a, cudaStream_t st) {
    const int ctas = std::min(a.num_tokens, 8 * num_sms());
    return launch_early(rope_write_kernel<KV>, dim3((unsigned)ctas), ROPE_THREADS, 0, st, a);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_kv_write_rope(void *query_out, const void *query, const void *key, const void *value,
                                const int32_t *positions, const float *inv_freq, const int32_t *pair_axis,
                                const int64_t *slot_mapping, void *k_cache, void *v_cache, int num_tokens,
                                int num_heads, int num_kv_heads, int head_dim, int rope_dim, int num_axes,
                                int interleaved, int64_t query_stride, int64_t query_out_stride, int64_t key_stride,
                                int64_t value_stride, int block_size, int64_t num_blocks, int kv_dtype, float k_scale,
                                float v_scale, void *stream) {
    if (num_tokens < 0 || num_heads < 0 || num_kv_heads <= 0 || head_dim <= 0 || head_dim % 8 != 0 || rope_dim <= 0 ||
        rope_dim % 16 != 0 || rope_dim > head_dim || num_axes < 1 || num_axes > PA_ROPE_MAX_AXES || block_size <= 0 ||
        num_blocks <= 0 || (kv_dtype != PA_KV_F16 && kv_dtype != PA_KV_BF16 && kv_dtype != PA_KV_FP8_E4M3))
        return PA_ERR_INVALID_ARG;
    if (kv_dtype == PA_KV_FP8_E4M3 &&
        (!std::isfinite(k_scale) || !(k_scale > 0.f) || !std::isfinite(v_scale) || !(v_scale > 0.f)))
        return PA_ERR_INVALID_ARG;
    // a token's pieces of work are counted in 32 bits
    if (rope_dim > ROPE_MAX_DIM || (long long)(num_heads + 2LL * num_kv_heads) * head_dim >= (1LL << 30))
        return PA_ERR_UNSUPPORTED;
    const long long q_row = (long long)num_heads * head_dim, k_row = (long long)num_kv_heads * head_dim;
    if (query_stride < q_row || query_out_stride < q_row || key_stride < k_row || value_stride < k_row ||
        (query_stride | query_out_stride | key_stride | value_stride) % 8 != 0)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !positions || !inv_freq || !slot_mapping || !k_cache || !v_cache ||
        (num_heads > 0 && (!query || !query_out)) || (query && query == query_out && query_stride != query_out_stride))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(query) ||
        !aligned16(query_out))
        return PA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    RopeArgs a{};
    a.query_out = static_cast<uint16_t *>(query_out);
    a.query = static_cast<const uint16_t *>(query);
    a.key = static_cast<const uint16_t *>(key);
    a.value = static_cast<const uint16_t *>(value);
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.pair_axis = pair_axis;
    a.slot_mapping = slot_mapping;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.num_tokens = num_tokens;
    a.hq = num_heads;
    a.hk = num_kv_heads;
    a.d = head_dim;
    a.rope_dim = rope_dim;
    a.num_axes = num_axes;
    a.interleaved = interleaved != 0;
    a.block_size = block_size;
    a.query_stride = query_stride;
    a.query_out_stride = query_out_stride;
    a.key_stride = key_stride;
    a.value_stride = value_stride;
    a.num_slots = (long long)num_blocks * block_size;
    if (kv_dtype == PA_KV_FP8_E4M3) {   // IEEE float divisions, once
        a.kinv = 1.0f / k_scale;
        a.vinv = 1.0f / v_scale;
    }
    if (debug_validate())
        if (const int e = validate_slots(slot_mapping, num_tokens, a.num_slots, st)) return e;
    if (kv_dtype == PA_KV_F16) return launch_rope<PA_KV_F16>(a, st);
    if (kv_dtype == PA_KV_BF16) return launch_rope<PA_KV_BF16>(a, st);
    return launch_rope<PA_KV_FP8_E4M3>(a, st);
}
