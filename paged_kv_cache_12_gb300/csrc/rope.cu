// KV write with the position rotation applied on the way: keys turned and
// scattered into their slots, values beside them, queries turned into query_out.
//
// A rotation by angle a takes the pair (x, y) to (x cos a - y sin a,
// y cos a + x sin a).  The angle of a pair is a position (an integer, one for each
// axis) times a frequency.  A position of a million times a frequency of one has
// lost most of the turn's fraction in 32 bits, so the fraction is found with whole
// numbers of 64 bits, and its sine and cosine in 32.  All heads of a token share its
// angles: they are computed once a token, in shared memory.
//
// Bound by HBM, and on a step's few tokens by the launch.  One GB300: 16,384 tokens of
// 32 query and 8 kv heads of 128 into an E4M3 cache 60 us (5.7 TB/s of reads and
// writes, 0.86 of a copy's rate), 5,003 tokens of 32 and 32 heads with three axes into
// an fp16 cache 40 us (5.7 TB/s), 100 tokens of 64 and 8 heads 4.2 us.
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

constexpr int ROPE_THREADS = 128;
// Steps of a thread on their way and CTAs of an SM.  The chunk and the video tokens
// above: 4 and 8 60 and 41 us, 3 and 8 60 and 41, 4 and 10 69 and 45, 8 and 6 65 and 48;
// CTAs of 64 threads 6 and 12 59 and 50, 4 and 16 66 and 44.  With the loads held in
// registers the best was 75 and 50.
constexpr int ROPE_DEPTH = 4;
constexpr int ROPE_RESIDENT = 8;
constexpr int ROPE_MAX_DIM = 512;   // rotary elements of a head
constexpr int ROPE_MAX_HEAD = 8 * ROPE_THREADS;   // elements of a head: a thread a piece

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

// Where a token's key and value go: its block's first row and its offset in the
// block as an element offset of kv head 0, or -1 for padding.
__device__ __forceinline__ long long cache_row(const RopeArgs &a, long long slot) {
    if (slot < 0 || slot >= a.num_slots) return -1;
    long long blk, off;
    if (slot >> 32) {
        blk = slot / a.block_size;
        off = slot - blk * a.block_size;
    } else {
        const uint32_t q = (uint32_t)slot / (uint32_t)a.block_size;
        blk = q;
        off = (uint32_t)slot - q * (uint32_t)a.block_size;
    }
    return (blk * a.hk * a.block_size + off) * a.d;
}

__device__ __forceinline__ void cell_load(uint4 *cell, const uint16_t *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(cell)), "l"(src) : "memory");
}

// A pair's frequency: the fraction of a turn that a step of its axis makes, in
// units of 2^-64 turns, so that the fraction after any number of steps is the low
// 64 bits of a product (off by the roundings of the frequency in turns, 2^-53 of it,
// times the steps).  axis: -1 where it is out of range or the frequency is not
// finite.
struct Frequency {
    unsigned long long step;
    int axis;
    bool back;   // a negative frequency
};
__device__ __forceinline__ Frequency frequency(const RopeArgs &a, int pair) {
    Frequency f;
    const double turns = (double)a.inv_freq[pair] * 0.15915494309189535;   // 1 / (2 pi)
    const double size = fabs(turns);
    f.axis = a.pair_axis ? a.pair_axis[pair] : 0;
    if (f.axis >= a.num_axes || !(size < 1e300)) f.axis = -1;
    f.back = turns < 0.0;
    f.step = f.axis < 0 ? 0ull : (unsigned long long)((size - floor(size)) * 18446744073709551616.0);
    return f;
}
__device__ __forceinline__ float2 cosine_sine(const Frequency &f, int position) {
    if (f.axis < 0) return make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
    const unsigned long long turns = f.step * (unsigned long long)(long long)position;
    float2 cs;
    sincospif((float)(int)(turns >> 32) * 0x1p-31f, &cs.y, &cs.x);   // in half turns, from -1 to 1
    if (f.back) cs.y = -cs.y;
    return cs;
}

// A CTA takes every gridDim-th token, and a thread a piece of a head of its own --
// eight elements, and their eight partners where a pair's halves lie rope_dim / 2
// apart -- in every head that is its turn: so it reads its pairs' cosines and sines
// once a token.  A thread's pieces of one token after another are one sequence of
// steps (query heads, key heads, values), whose loads it has on their way ROPE_DEPTH
// steps ahead, in shared memory cells that no other thread touches: the only thing
// that the threads wait for one another for is the next token's angles.
template <int KV, bool INTERLEAVED>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_RESIDENT) rope_write_kernel(const RopeArgs a) {
    constexpr int PER = INTERLEAVED ? 4 : 8;            // pairs of a piece that turns
    constexpr int CELLS = INTERLEAVED ? 1 : 2;          // 16-byte cells of a step
    __shared__ uint4 cells[ROPE_DEPTH * CELLS][ROPE_THREADS];
    __shared__ float2 turn[2][ROPE_MAX_DIM / 2];        // cosine and sine of a token's pairs, by the token's parity
    const int pairs = a.rope_dim / 2, tid = threadIdx.x;
    const int turned = pairs / PER;                     // pieces of a head that turn
    const int pieces = turned + (a.d - a.rope_dim) / 8; // of a query or key head
    const int vecs = a.d / 8;                           // of a value head
    // heads at a time, and this thread's head and piece among them
    const int heads = ROPE_THREADS / pieces, h0 = tid / pieces, p = tid - h0 * pieces;
    const int vheads = ROPE_THREADS / vecs, vh0 = tid / vecs, v = tid - vh0 * vecs;
    const bool some = h0 < heads, vsome = vh0 < vheads;
    const bool turns = p < turned, two = turns && !INTERLEAVED;
    const int e = turns ? 8 * p : a.rope_dim + 8 * (p - turned);   // the piece's first element
    const int nq = (a.hq + heads - 1) / heads, nk = (a.hk + heads - 1) / heads, nv = (a.hk + vheads - 1) / vheads;
    const int steps = nq + nk + nv;                     // of a token
    const long long head_rows = (long long)a.block_size * a.d;
    const int stride = gridDim.x;
    grid_release();
    grid_wait();
    Frequency f0{};
    if (tid < pairs) f0 = frequency(a, tid);
    auto position = [&](const Frequency &f, int t) {
        return f.axis < 0 ? 0 : a.positions[(long long)f.axis * a.num_tokens + t];
    };
    auto angles = [&](int t, int place, int pos0) {     // of token t; pos0: this thread's first pair's position
        if (tid < pairs) turn[place][tid] = cosine_sine(f0, pos0);
        for (int i = tid + ROPE_THREADS; i < pairs; i += ROPE_THREADS) {   // (rotary parts above 2 ROPE_THREADS)
            const Frequency f = frequency(a, i);
            turn[place][i] = cosine_sine(f, position(f, t));
        }
    };
    // the loads: a cursor ROPE_DEPTH - 1 steps ahead of the work
    int lt = blockIdx.x, lu = 0, lc = 0;                // its token, step and cell
    int64_t lslot = a.slot_mapping[lt], lnext = lt + stride < a.num_tokens ? a.slot_mapping[lt + stride] : -1;
    auto load = [&]() {
        if (lt < a.num_tokens) {
            if (lslot >= 0 && lslot < a.num_slots) {    // (padding is not read)
                const uint16_t *src;
                bool mine, pair = two;
                if (lu < nq) {
                    const int h = h0 + lu * heads;
                    mine = some && h < a.hq;
                    src = a.query + (long long)lt * a.query_stride + h * a.d + e;
                } else if (lu < nq + nk) {
                    const int h = h0 + (lu - nq) * heads;
                    mine = some && h < a.hk;
                    src = a.key + (long long)lt * a.key_stride + h * a.d + e;
                } else {
                    const int h = vh0 + (lu - nq - nk) * vheads;
                    mine = vsome && h < a.hk;
                    src = a.value + (long long)lt * a.value_stride + h * a.d + 8 * v;
                    pair = false;
                }
                if (mine) {
                    cell_load(&cells[lc * CELLS][tid], src);
                    if (CELLS == 2 && pair) cell_load(&cells[lc * CELLS + CELLS - 1][tid], src + pairs);
                }
            }
            if (++lu == steps) {
                lu = 0;
                lt += stride;
                lslot = lnext;
                lnext = lt + stride < a.num_tokens ? a.slot_mapping[lt + stride] : -1;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        lc = (lc + 1) % ROPE_DEPTH;
    };
#pragma unroll 1
    for (int i = 0; i < ROPE_DEPTH - 1; ++i) load();
    const int t00 = blockIdx.x;
    angles(t00, 0, tid < pairs ? position(f0, t00) : 0);
    int pos = tid < pairs && t00 + stride < a.num_tokens ? position(f0, t00 + stride) : 0;   // of the next token
    int64_t slot = a.slot_mapping[t00];
    int c = 0, place = 0;
    __syncthreads();
    for (int t = t00; t < a.num_tokens; t += stride, place ^= 1) {
        const long long row = cache_row(a, slot);
        if (t + stride < a.num_tokens) {
            angles(t + stride, place ^ 1, pos);
            slot = a.slot_mapping[t + stride];
            if (tid < pairs && t + 2LL * stride < a.num_tokens) pos = position(f0, t + 2 * stride);
        }
        float2 cs[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) cs[k] = turns ? turn[place][PER * p + k] : make_float2(1.f, 0.f);
#pragma unroll 1
        for (int u = 0; u < steps; ++u, c = (c + 1) % ROPE_DEPTH) {
            load();
            asm volatile("cp.async.wait_group %0;" ::"n"(ROPE_DEPTH - 1) : "memory");
            if (row < 0) continue;
            if (u >= nq + nk) {   // a value's piece
                const int h = vh0 + (u - nq - nk) * vheads;
                if (!vsome || h >= a.hk) continue;
                const uint4 raw = cells[c * CELLS][tid];
                const long long at = row + h * head_rows + 8 * v;
                if constexpr (KV == PA_KV_FP8_E4M3) {
                    float x[8];
                    unpack8<KV>(raw, x);
                    store_cache<KV>(a.v_cache, at, x, a.vinv);
                } else {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.v_cache) + at) = raw;
                }
                continue;
            }
            const int h = h0 + (u < nq ? u : u - nq) * heads;
            if (!some || h >= (u < nq ? a.hq : a.hk)) continue;
            float x[8], y[8];
            unpack8<KV>(cells[c * CELLS][tid], x);
            if (INTERLEAVED) {
                if (turns)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 r = cs[k];
                        const float m = x[2 * k], w = x[2 * k + 1];
                        x[2 * k] = fmaf(m, r.x, -(w * r.y));
                        x[2 * k + 1] = fmaf(w, r.x, m * r.y);
                    }
            } else if (two) {
                unpack8<KV>(cells[c * CELLS + CELLS - 1][tid], y);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 r = cs[k % PER];
                    const float m = x[k], w = y[k];
                    x[k] = fmaf(m, r.x, -(w * r.y));
                    y[k] = fmaf(w, r.x, m * r.y);
                }
            }
            if (u < nq) {
                uint16_t *to = a.query_out + (long long)t * a.query_out_stride + h * a.d + e;
                *reinterpret_cast<uint4 *>(to) = pack8<KV>(x);
                if (two) *reinterpret_cast<uint4 *>(to + pairs) = pack8<KV>(y);
            } else {
                const long long at = row + h * head_rows + e;
                store_cache<KV>(a.k_cache, at, x, a.kinv);
                if (two) store_cache<KV>(a.k_cache, at + pairs, y, a.kinv);
            }
        }
        __syncthreads();   // the next token's angles are there, and this one's have been read
    }
}

// PA_DEBUG_VALIDATE: every pair's axis is one of the positions'.
int validate_axes(const int32_t *pair_axis, int pairs, int num_axes, cudaStream_t st) {
    int32_t axis[ROPE_MAX_DIM / 2];
    if (!pair_axis) return 0;
    if (const int e = copy_to_host(axis, pair_axis, sizeof(int32_t) * (size_t)pairs, st)) return e;
    for (int i = 0; i < pairs; ++i)
        if (axis[i] < 0 || axis[i] >= num_axes) return PA_ERR_INVALID_ARG;
    return 0;
}

template <int KV>
int launch_rope(const RopeArgs &a, cudaStream_t st) {
    const dim3 ctas((unsigned)std::min(a.num_tokens, ROPE_RESIDENT * num_sms()));
    return a.interleaved ? launch_early(rope_write_kernel<KV, true>, ctas, ROPE_THREADS, 0, st, a)
                         : launch_early(rope_write_kernel<KV, false>, ctas, ROPE_THREADS, 0, st, a);
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
    // tokens, and a token's elements, are counted in 32 bits
    if (num_tokens > (1 << 30) || rope_dim > ROPE_MAX_DIM || head_dim > ROPE_MAX_HEAD || (long long)(num_heads + 2LL * num_kv_heads) * head_dim >= (1LL << 30))
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
    if (debug_validate()) {
        if (const int e = validate_slots(slot_mapping, num_tokens, a.num_slots, st)) return e;
        if (const int e = validate_axes(pair_axis, rope_dim / 2, num_axes, st)) return e;
    }
    if (kv_dtype == PA_KV_F16) return launch_rope<PA_KV_F16>(a, st);
    if (kv_dtype == PA_KV_BF16) return launch_rope<PA_KV_BF16>(a, st);
    return launch_rope<PA_KV_FP8_E4M3>(a, st);
}
