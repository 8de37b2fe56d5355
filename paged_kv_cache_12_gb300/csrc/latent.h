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
// has four significant bits and the scale none).
__device__ __forceinline__ uint2 latent_codes_to_bf16(uint32_t codes, float scale) {
    const uint32_t lo = e4m3x2_lo_to_f16x2(codes), hi = e4m3x2_hi_to_f16x2(codes);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return make_uint2(pack_bf162(a.x * scale, a.y * scale), pack_bf162(b.x * scale, b.y * scale));
}

}  // namespace pa
