// The latent cache's row formats, shared by its data movement (latent.cu) and
// the attention kernels that read it (latent_attn.cu).
#pragma once

#include "common.cuh"

namespace pa {

constexpr int LC = PA_LATENT_DIM;               // latent elements of a row
constexpr int LR = PA_LATENT_ROPE_DIM;          // rotary elements of a row
constexpr int LROW = PA_LATENT_ROW;             // elements of a row
constexpr int LROW8 = PA_LATENT_ROW_FP8_BYTES;  // bytes of a quantised row
constexpr int L8_ROPE = LC;                     // byte offset of its rotary elements
constexpr int L8_SCALE = LC + 2 * LR;           // and of its four scales
constexpr int LGROUP = 128;                     // latent elements that share a scale
static_assert(LROW == LC + LR && L8_SCALE + 4 * (LC / LGROUP) == LROW8, "latent row formats");

inline bool latent_block_size_ok(int bs) { return bs == 8 || bs == 16 || bs == 32 || bs == 64; }

// Bytes of a cached row, 0 for an unknown element type.
inline int latent_row_bytes(int kv) {
    return kv == PA_KV_F16 || kv == PA_KV_BF16 ? 2 * LROW : kv == PA_KV_FP8_E4M3 ? LROW8 : 0;
}

// E4M3 codes times a power of two as bf16 (exact: a code has four significant
// bits and the scale none), by bits: a code's exponent and mantissa, moved to
// the low end of a bf16's, are the value times 2^-120 (a subnormal code becomes a
// subnormal bf16), and a product with 2^120 times the scale is exact.
// Conversion instructions (E4M3 to fp16 to float to bf16) take three times as
// long.  Two cases need the long way: NaN codes (latent_codes_nan finds them), and
// scales above 2^7, where 2^120 times the scale is no bf16 (latent_scale_special).
__device__ __forceinline__ uint32_t bf162_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Four codes (lowest byte first) at 2^-120 of their values.
__device__ __forceinline__ uint2 latent_codes_low(uint32_t codes) {
    const uint32_t w0 = __byte_perm(codes, 0, 0x1404), w1 = __byte_perm(codes, 0, 0x3424);
    return make_uint2(((w0 >> 4) & 0x07f007f0u) | (w0 & 0x80008000u),
                      ((w1 >> 4) & 0x07f007f0u) | (w1 & 0x80008000u));
}
// 2^120 times the scale, twice (scales up to 2^7).
__device__ __forceinline__ uint32_t latent_scale_up(float scale) {
    return __byte_perm(__float_as_uint(scale * 0x1p120f), 0, 0x3232);
}
__device__ __forceinline__ uint2 latent_codes_fast(uint32_t codes, uint32_t scale_up) {
    const uint2 r = latent_codes_low(codes);
    return make_uint2(bf162_mul(r.x, scale_up), bf162_mul(r.y, scale_up));
}
// Nonzero if one of eight codes is NaN (all exponent and mantissa bits set).
__device__ __forceinline__ uint32_t latent_codes_nan(uint2 codes) {
    return (((codes.x & 0x7f7f7f7fu) + 0x01010101u) | ((codes.y & 0x7f7f7f7fu) + 0x01010101u)) & 0x80808080u;
}
__device__ __forceinline__ bool latent_scale_special(float scale) { return !(scale <= 128.f); }
// Any codes and scale.
__device__ __forceinline__ uint2 latent_codes_to_bf16(uint32_t codes, float scale) {
    uint2 r = latent_codes_low(codes);
    const uint32_t s2 = __byte_perm(__float_as_uint(scale), 0, 0x3232);
    r.x = bf162_mul(bf162_mul(r.x, 0x7b807b80u), s2);   // 2^120, then the scale
    r.y = bf162_mul(bf162_mul(r.y, 0x7b807b80u), s2);
    if ((codes & 0x7fu) == 0x7fu) r.x = (r.x & 0xffff0000u) | 0x7fc0u;
    if ((codes >> 8 & 0x7fu) == 0x7fu) r.x = (r.x & 0xffffu) | 0x7fc00000u;
    if ((codes >> 16 & 0x7fu) == 0x7fu) r.y = (r.y & 0xffff0000u) | 0x7fc0u;
    if ((codes >> 24 & 0x7fu) == 0x7fu) r.y = (r.y & 0xffffu) | 0x7fc00000u;
    return r;
}

// Whether one of eight 16-bit values is not finite (all exponent bits set), and a
// pair with what is not finite made zero.
template <int KV>
__device__ __forceinline__ bool not_finite(uint4 v) {
    constexpr uint32_t E = KV == PA_KV_F16 ? 0x7c007c00u : 0x7f807f80u, ONE = KV == PA_KV_F16 ? 0x04000400u : 0x00800080u;
    return (((v.x & E) + ONE) | ((v.y & E) + ONE) | ((v.z & E) + ONE) | ((v.w & E) + ONE)) & 0x80008000u;
}
template <int KV>
__device__ __forceinline__ uint32_t finite_part(uint32_t v) {
    constexpr uint32_t E = KV == PA_KV_F16 ? 0x7c00u : 0x7f80u;
    return ((v & E) == E ? 0u : v & 0xffffu) | ((v >> 16 & E) == E ? 0u : v & 0xffff0000u);
}

}  // namespace pa
