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

// Four E4M3 codes times a power of two, as two pairs of bf16 (exact: a code
// has four significant bits and the scale none).  By bits: a code's exponent and
// mantissa, moved to the low end of a bf16's, are the value times 2^-120 (a
// subnormal code becomes a subnormal bf16); two exact products undo that and
// scale.  Conversion instructions (E4M3 to fp16 to float to bf16) would take
// three times as long: 3100 cycles for a tile of 48 x 512 codes by eight warps.
__device__ __forceinline__ uint32_t bf162_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint2 latent_codes_to_bf16(uint32_t codes, float scale) {
    const uint32_t s2 = (__float_as_uint(scale) >> 16) * 0x10001u;   // a power of two, or NaN, twice
    const uint32_t w0 = __byte_perm(codes, 0, 0x1404), w1 = __byte_perm(codes, 0, 0x3424);
    constexpr uint32_t UP = 0x7b807b80u;   // 2^120, twice
    uint2 r = make_uint2(((w0 >> 4) & 0x07f007f0u) | (w0 & 0x80008000u),
                         ((w1 >> 4) & 0x07f007f0u) | (w1 & 0x80008000u));
    r.x = bf162_mul(bf162_mul(r.x, UP), s2);
    r.y = bf162_mul(bf162_mul(r.y, UP), s2);
    if (((codes & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) {   // a NaN code (all exponent and mantissa bits)
        if ((codes & 0x7fu) == 0x7fu) r.x = (r.x & 0xffff0000u) | 0x7fc0u;
        if ((codes >> 8 & 0x7fu) == 0x7fu) r.x = (r.x & 0xffffu) | 0x7fc00000u;
        if ((codes >> 16 & 0x7fu) == 0x7fu) r.y = (r.y & 0xffff0000u) | 0x7fc0u;
        if ((codes >> 24 & 0x7fu) == 0x7fu) r.y = (r.y & 0xffffu) | 0x7fc00000u;
    }
    return r;
}

}  // namespace pa
