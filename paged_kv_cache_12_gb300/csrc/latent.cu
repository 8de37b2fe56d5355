// Data movement of the latent cache: the write of new tokens' rows (copied, or
// quantised to E4M3 codes with a scale per 128 elements), the read back of
// rows through block tables, and the block copy.
//
// Every row is moved in 16-byte vectors and every index read from the device
// is range-checked before it is used as an address.  All three are bound by
// HBM on large calls and by the launch on a decode step's few rows (one GB300:
// 65,536 rows to E4M3 in 19.1 us, 5.85 TB/s of reads and writes; 100 rows in 6.1 us,
// nearly all of it the call).
//
// Sources: the new token goes into the free slot of the sequence's current
// block ("PagedAttention : comment optimiser la memoire GPU lors de
// l'inference des LLM", deeplearn.tn, section "Un exemple concret
// d'allocation"); tokens are found through the block table ("PagedAttention de
// vLLM : comment la gestion de la VRAM soutient l'inference des grands
// modeles", deepsonar.com.cn, section 2.2), which does not depend on what a
// slot holds.

#include <algorithm>
#include <vector>

#include "latent.h"

namespace pa {
namespace {

constexpr int VROW = LROW / 8;   // 16-byte vectors of a 16-bit row
constexpr int VLAT = LC / 8;     // of them latent

// Rows of 16-bit elements, one thread per 16-byte vector.
__global__ void __launch_bounds__(256) latent_write_kernel(const uint4 *latent, const uint4 *rope,
                                                           const int64_t *slot_mapping, uint4 *cache, int num_tokens,
                                                           long long latent_vecs, long long rope_vecs,
                                                           long long num_slots) {
    const long long total = (long long)num_tokens * VROW;
    grid_release();
    grid_wait();
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
         i += (long long)gridDim.x * blockDim.x) {
        const long long t = i / VROW;
        const int v = (int)(i - t * VROW);
        const uint4 x = v < VLAT ? latent[t * latent_vecs + v] : rope[t * rope_vecs + (v - VLAT)];
        const long long slot = slot_mapping[t];
        if (slot >= 0 && slot < num_slots) cache[slot * VROW + v] = x;
    }
}

// The larger of m and a bf16 pair's magnitudes; fmaxf drops a NaN.
__device__ __forceinline__ float max_magnitude(float m, uint32_t pair) {
    return fmaxf(fmaxf(m, fabsf(__uint_as_float(pair << 16))), fabsf(__uint_as_float(pair & 0xffff0000u)));
}

// The smallest e in [-100, 119] with a <= 448 * 2^e, 448 = 1.75 * 2^8: from
// the exponent and mantissa of a = m * 2^k, e = k - 8 if m <= 1.75, else k - 7
// (an infinity, k = 128, ends at the upper bound).
__device__ __forceinline__ int scale_exponent(float a) {
    const uint32_t u = __float_as_uint(a);
    const int k = (int)(u >> 23) - 127;   // subnormals end at the lower bound too
    return max(-100, min(119, k - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0)));
}

// Eight bf16 elements times 2^-e (exact in fp32) to eight E4M3 codes.
__device__ __forceinline__ uint2 quantise_bf16x8(uint4 x, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 y = make_float2(__uint_as_float(w[k] << 16) * inv, __uint_as_float(w[k] & 0xffff0000u) * inv);
        c[k] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3));
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Quantised rows, one warp per token: lane l holds elements 8 l .. 8 l + 7
// (groups 0 and 1, sixteen lanes each) and 256 + 8 l .. (groups 2 and 3).
__global__ void __launch_bounds__(256) latent_write_fp8_kernel(const uint4 *latent, const uint4 *rope,
                                                               const int64_t *slot_mapping, uint8_t *cache,
                                                               int num_tokens,
                                                               long long latent_vecs, long long rope_vecs,
                                                               long long num_slots) {
    const int lane = threadIdx.x & 31;
    const int step = (int)(gridDim.x * (blockDim.x >> 5));
    grid_release();
    grid_wait();
    for (long long t = blockIdx.x * (long long)(blockDim.x >> 5) + (threadIdx.x >> 5); t < num_tokens; t += step) {
        const uint4 x = latent[t * latent_vecs + lane], y = latent[t * latent_vecs + 32 + lane];
        uint4 r = make_uint4(0, 0, 0, 0);
        if (lane < 8) r = rope[t * rope_vecs + lane];
        const long long slot = slot_mapping[t];
        float mx = max_magnitude(max_magnitude(max_magnitude(max_magnitude(0.f, x.x), x.y), x.z), x.w);
        float my = max_magnitude(max_magnitude(max_magnitude(max_magnitude(0.f, y.x), y.y), y.z), y.w);
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) {   // over the sixteen lanes of a group
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, d));
        }
        const int ex = scale_exponent(mx), ey = scale_exponent(my);
        if (slot < 0 || slot >= num_slots) continue;   // the whole warp
        uint8_t *row = cache + slot * LROW8;
        *reinterpret_cast<uint2 *>(row + 8 * lane) = quantise_bf16x8(x, __uint_as_float((uint32_t)(127 - ex) << 23));
        *reinterpret_cast<uint2 *>(row + 256 + 8 * lane) =
            quantise_bf16x8(y, __uint_as_float((uint32_t)(127 - ey) << 23));
        if (lane < 8) *reinterpret_cast<uint4 *>(row + L8_ROPE + 16 * lane) = r;
        if ((lane & 15) == 0) {
            float *scale = reinterpret_cast<float *>(row + L8_SCALE);
            scale[lane >> 4] = __uint_as_float((uint32_t)(127 + ex) << 23);
            scale[2 + (lane >> 4)] = __uint_as_float((uint32_t)(127 + ey) << 23);
        }
    }
}

// Read back: a CTA takes READ_ROWS consecutive rows of out, a thread a column of
// 16 bytes in each.  The CTA checks the order of row_start (and keeps it in shared
// memory when it fits), one thread per row finds its sequence by binary search
// and its slot through the block table (a slot below 0 marks a NaN row), then all
// threads move vectors, a load per row on its way at once.  Small CTAs, because
// each spends two thirds of its time on those dependent steps: 115,000 quantised
// rows of a ragged batch took 37 us with 8 rows by 72 threads, 38 with 16 by 288,
// 42 with 32 by 288 and 48 with 64 by 288 (34 launched early); the bytes alone take
// 28.5.
constexpr int READ_ROWS = 8, READ_THREADS = VROW;
constexpr int READ_STARTS = 1024;

template <bool F8>
__global__ void __launch_bounds__(READ_THREADS) latent_read_kernel(
    uint4 *out, const uint8_t *cache, const int32_t *block_tables, const int32_t *row_start,
    const int32_t *first_token, int num_seqs, int num_rows,
    long long out_vecs, int block_size, long long num_blocks, int mbps, uint32_t nan_pair) {
    __shared__ long long slots[READ_ROWS];
    __shared__ int starts[READ_STARTS + 1];
    const int base = blockIdx.x * READ_ROWS;
    const bool kept = num_seqs <= READ_STARTS;
    bool ok = true;
    grid_release();
    grid_wait();
    for (int i = threadIdx.x; i <= num_seqs; i += blockDim.x) {
        const int b = row_start[i], a = i ? row_start[i - 1] : 0;
        if (b < a || b > num_rows || (i == 0 && b != 0)) ok = false;
        if (kept) starts[i] = b;
    }
    ok = __syncthreads_and(ok);
    const int end = ok ? min(num_rows, kept ? starts[num_seqs] : row_start[num_seqs]) : num_rows;
    if (threadIdx.x < READ_ROWS) {
        const int row = base + threadIdx.x;
        const int *from = kept ? starts : row_start;
        long long slot = -1;
        if (ok && row < end) {
            int lo = 0, hi = num_seqs;   // the last i with row_start[i] <= row
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (from[mid] <= row) lo = mid; else hi = mid;
            }
            const long long t = (long long)row - from[lo] + (first_token ? first_token[lo] : 0);
            if (t >= 0 && t < (long long)mbps * block_size) {
                const long long blk = block_tables[(long long)lo * mbps + t / block_size];
                if (blk >= 0 && blk < num_blocks) slot = blk * block_size + t % block_size;
            }
        }
        slots[threadIdx.x] = slot;
    }
    __syncthreads();
    const int v = threadIdx.x;
    const int left = end - base;   // rows of this CTA
    if constexpr (F8) {
        if (v < VLAT) {
            uint2 c[READ_ROWS];
            float s[READ_ROWS];
#pragma unroll
            for (int k = 0; k < READ_ROWS; ++k) {
                const long long slot = slots[k];
                c[k] = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);   // NaN codes
                s[k] = 1.f;
                if (slot >= 0) {
                    const uint8_t *row = cache + slot * LROW8;
                    c[k] = *reinterpret_cast<const uint2 *>(row + 8 * v);
                    s[k] = *reinterpret_cast<const float *>(row + L8_SCALE + 4 * (v / (LGROUP / 8)));
                }
            }
#pragma unroll
            for (int k = 0; k < READ_ROWS; ++k) {
                const uint32_t up = latent_scale_up(s[k]);
                uint2 a = latent_codes_fast(c[k].x, up), b = latent_codes_fast(c[k].y, up);
                if (latent_codes_nan(c[k]) || latent_scale_special(s[k])) {
                    a = latent_codes_to_bf16(c[k].x, s[k]);
                    b = latent_codes_to_bf16(c[k].y, s[k]);
                }
                if (k < left) out[(long long)(base + k) * out_vecs + v] = make_uint4(a.x, a.y, b.x, b.y);
            }
            return;
        }
    }
    uint4 x[READ_ROWS];
#pragma unroll
    for (int k = 0; k < READ_ROWS; ++k) {
        const long long slot = slots[k];
        x[k] = make_uint4(nan_pair, nan_pair, nan_pair, nan_pair);
        if (slot >= 0)
            x[k] = F8 ? *reinterpret_cast<const uint4 *>(cache + slot * LROW8 + L8_ROPE + 16 * (v - VLAT))
                      : *reinterpret_cast<const uint4 *>(cache + slot * (2 * LROW) + 16 * v);
    }
#pragma unroll
    for (int k = 0; k < READ_ROWS; ++k) {
        if (k < left) out[(long long)(base + k) * out_vecs + v] = x[k];
    }
}

// blockIdx.y = pair; the block's vectors are strided over blockIdx.x.
__global__ void latent_copy_kernel(uint4 *__restrict__ cache, const int64_t *__restrict__ pairs,
                                   long long vecs_per_block, long long num_blocks) {
    const long long src = pairs[2 * (long long)blockIdx.y];
    const long long dst = pairs[2 * (long long)blockIdx.y + 1];
    if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) return;
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < vecs_per_block;
         i += (long long)gridDim.x * blockDim.x)
        cache[dst * vecs_per_block + i] = cache[src * vecs_per_block + i];
}

// PA_DEBUG_VALIDATE of a read: the rows' order, and a block in range for every
// token read (the tables' entries before a sequence's last token count too).
int validate_read(const int32_t *block_tables, const int32_t *row_start, const int32_t *first_token, int num_seqs,
                  int num_rows, int block_size, long long num_blocks, int mbps, cudaStream_t st) try {
    if (const int e = validate_starts(row_start, num_seqs, num_rows, false, st)) return e;
    std::vector<int32_t> start((size_t)num_seqs + 1), first((size_t)num_seqs);
    std::vector<int64_t> last((size_t)num_seqs);
    if (const int e = copy_to_host(start.data(), row_start, sizeof(int32_t) * start.size(), st)) return e;
    if (first_token)
        if (const int e = copy_to_host(first.data(), first_token, sizeof(int32_t) * first.size(), st)) return e;
    for (int i = 0; i < num_seqs; ++i) {
        const int n = start[(size_t)i + 1] - start[(size_t)i];
        if (n > 0 && first[(size_t)i] < 0) return PA_ERR_INVALID_ARG;
        last[(size_t)i] = n > 0 ? (int64_t)first[(size_t)i] + n : 0;
    }
    return validate_tables(block_tables, last.data(), num_seqs, mbps, block_size, num_blocks, st);
} catch (...) {   // no host memory for the check
    return PA_ERR_STATE;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_latent_write(const uint16_t *latent, const uint16_t *rope, const int64_t *slot_mapping, void *cache,
                               int num_tokens, int64_t latent_stride, int64_t rope_stride, int block_size,
                               int64_t num_blocks, int kv_dtype, void *stream) {
    if (num_tokens < 0 || num_blocks <= 0 || block_size <= 0 || latent_row_bytes(kv_dtype) == 0)
        return PA_ERR_INVALID_ARG;
    if (!latent_block_size_ok(block_size)) return PA_ERR_UNSUPPORTED;
    if (latent_stride < LC || latent_stride % 8 != 0 || rope_stride < LR || rope_stride % 8 != 0)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!latent || !rope || !slot_mapping || !cache || !aligned16(latent) || !aligned16(rope) || !aligned16(cache))
        return PA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const long long num_slots = (long long)num_blocks * block_size;
    if (debug_validate())
        if (const int e = validate_slots(slot_mapping, num_tokens, num_slots, st)) return e;
    const uint4 *c = reinterpret_cast<const uint4 *>(latent), *r = reinterpret_cast<const uint4 *>(rope);
    const long long cap = (long long)num_sms() * 16;
    if (kv_dtype == PA_KV_FP8_E4M3) {
        const long long blocks = std::min(((long long)num_tokens + 7) / 8, cap);
        return launch_early(latent_write_fp8_kernel, dim3((unsigned)blocks), 256, 0, st, c, r, slot_mapping,
                            static_cast<uint8_t *>(cache), num_tokens, (long long)latent_stride / 8,
                            (long long)rope_stride / 8, num_slots);
    }
    const long long blocks = std::min(((long long)num_tokens * VROW + 255) / 256, cap);
    return launch_early(latent_write_kernel, dim3((unsigned)blocks), 256, 0, st, c, r, slot_mapping,
                        static_cast<uint4 *>(cache), num_tokens, (long long)latent_stride / 8,
                        (long long)rope_stride / 8, num_slots);
}

extern "C" int pa_latent_block_copy(void *cache, const int64_t *pairs, int num_pairs, int block_size,
                                    int64_t num_blocks, int kv_dtype, void *stream) {
    const int row = latent_row_bytes(kv_dtype);
    if (num_pairs < 0 || block_size <= 0 || num_blocks <= 0 || row == 0) return PA_ERR_INVALID_ARG;
    if (!latent_block_size_ok(block_size)) return PA_ERR_UNSUPPORTED;
    if (num_pairs == 0) return PA_OK;
    if (!cache || !pairs || !aligned16(cache)) return PA_ERR_INVALID_ARG;
    if (num_pairs > 65535) return PA_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug_validate())
        if (const int e = validate_pairs(pairs, num_pairs, num_blocks, st)) return e;
    const long long vecs = (long long)row * block_size / 16;
    const dim3 grid((unsigned)std::min((vecs + 255) / 256, 64LL), (unsigned)num_pairs);
    latent_copy_kernel<<<grid, 256, 0, st>>>(static_cast<uint4 *>(cache), pairs, vecs, num_blocks);
    return cuda_status(cudaGetLastError());
}

extern "C" int pa_latent_read(uint16_t *out, const void *cache, const int32_t *block_tables, const int32_t *row_start,
                              const int32_t *first_token, int num_seqs, int num_rows, int64_t out_stride,
                              int block_size, int64_t num_blocks, int max_blocks_per_seq, int kv_dtype,
                              void *stream) {
    if (num_seqs < 0 || num_rows < 0 || (num_seqs == 0 && num_rows > 0) || out_stride < LROW || out_stride % 8 != 0 ||
        block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || latent_row_bytes(kv_dtype) == 0)
        return PA_ERR_INVALID_ARG;
    if (!latent_block_size_ok(block_size) || num_rows > (1 << 30)) return PA_ERR_UNSUPPORTED;
    if (num_rows == 0) return PA_OK;
    if (!out || !cache || !block_tables || !row_start || !aligned16(out) || !aligned16(cache))
        return PA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug_validate())
        if (const int e = validate_read(block_tables, row_start, first_token, num_seqs, num_rows, block_size, num_blocks,
                                        max_blocks_per_seq, st))
            return e;
    const unsigned grid = ((unsigned)num_rows + READ_ROWS - 1) / READ_ROWS;
    uint4 *o = reinterpret_cast<uint4 *>(out);
    const uint8_t *c = static_cast<const uint8_t *>(cache);
    const uint32_t nan_pair = kv_dtype == PA_KV_F16 ? 0x7e007e00u : 0x7fc07fc0u;
    return launch_early(kv_dtype == PA_KV_FP8_E4M3 ? latent_read_kernel<true> : latent_read_kernel<false>, dim3(grid),
                        READ_THREADS, 0, st, o, c, block_tables, row_start, first_token, num_seqs, num_rows,
                        (long long)out_stride / 8, block_size, (long long)num_blocks, max_blocks_per_seq, nan_pair);
}
