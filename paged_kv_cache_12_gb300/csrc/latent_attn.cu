// Attention over the latent cache in the absorbed form.
#include <algorithm>
#include <cmath>

#include "decode_common.cuh"
#include "latent.h"
#include "umma.cuh"
#include "work_axis.cuh"

namespace pa {
namespace {

constexpr int LT_ROWS = 64;   // query rows of a row tile (new token x head, token-major)
constexpr int LT_TOK = 64;    // tokens of a KV tile

struct LatentArgs {
    uint16_t *out;
    const uint16_t *query;
    const uint8_t *cache;
    const int32_t *block_tables, *context_lens, *query_start;
    WsHeader *hdr;
    int num_seqs, num_query_tokens, H, bs, mbps, max_context_len;
    long long num_blocks;
    float scale_log2;
    long long wait_limit;
    // workspace
    int *status;            // [AXIS_MAX_CTAS] nonzero: the CTA gave up waiting
    long long *unit_base;   // [num_seqs + 1]
    float2 *ml;             // [2 AXIS_MAX_CTAS][LT_ROWS] maximum (log2 units) and sum of a partial row
    float *o;               // [2 AXIS_MAX_CTAS][LT_ROWS][LC] its unnormalised output

    // ---- the work axis
    static constexpr int COST = 1;
    struct Seq {
        int L, T, q0;   // context, new tokens, first query token
        int tiles;      // KV tiles of the context (0: nothing to compute)
        int rts;        // row tiles
        bool valid;     // rows are computed (or zero, for an empty context)
    };
    __device__ __forceinline__ Seq seq_work(int i) const {
        Seq w;
        w.L = __ldg(context_lens + i);
        w.q0 = query_start ? __ldg(query_start + i) : i;
        w.T = query_start ? __ldg(query_start + i + 1) - w.q0 : 1;
        w.valid = w.L >= 0 && w.L <= max_context_len && (long long)w.L <= (long long)mbps * bs &&
                  !(query_start && w.T > w.L);
        w.tiles = w.valid && w.T > 0 ? (w.L + LT_TOK - 1) / LT_TOK : 0;
        w.rts = w.tiles ? (int)(((long long)w.T * H + LT_ROWS - 1) / LT_ROWS) : 0;
        return w;
    }
    // Every row tile counts the whole context's KV tiles (a chunk's earlier
    // rows see fewer, which matters only for long chunks; those belong to the
    // expanded form).
    __device__ __forceinline__ long long start(const Seq &w, int r) const { return (long long)r * (w.tiles + COST); }
    // KV tiles that row tile r sees: up to its last row's own position.
    __device__ __forceinline__ int row_tiles(const Seq &w, int r) const {
        const long long last = min((long long)w.T * H, (long long)(r + 1) * LT_ROWS) - 1;
        return (w.L - w.T + (int)(last / H) + 1 + LT_TOK - 1) / LT_TOK;
    }
    __device__ __forceinline__ bool starts_ok() const {
        return !query_start || offsets_ok(query_start, num_seqs, num_query_tokens);
    }
    // rows of row tile r, and its first row in the query
    __device__ __forceinline__ int rows(const Seq &w, int r) const {
        return (int)min((long long)LT_ROWS, (long long)w.T * H - (long long)r * LT_ROWS);
    }
    __device__ __forceinline__ long long first_row(const Seq &w, int r) const {
        return (long long)w.q0 * H + (long long)r * LT_ROWS;
    }
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

// ------------------------------------------------------------------ 16-bit kernel

constexpr int LT_THREADS = 256;
constexpr int LT_GROUP = 9 * 1024;            // 8 rows of 576 elements: nine 128-byte-swizzled blocks of 64 columns
constexpr int LT_STAGES = 2;
constexpr int LT_STAGE = LT_TOK / 8 * LT_GROUP;
constexpr int LT_OFF_Q = 0;
constexpr int LT_OFF_KV = LT_ROWS / 8 * LT_GROUP;
constexpr int LT_OFF_P = LT_OFF_KV + LT_STAGES * LT_STAGE;
constexpr int LT_OFF_CTRL = LT_OFF_P + LT_ROWS * LT_TOK * 2;
constexpr int LT_CTRL = 1024;
constexpr int LT_SMEM = LT_OFF_CTRL + LT_CTRL + 1024;   // + alignment slack
static_assert(LT_SMEM <= 227 * 1024, "shared memory of one CTA");
constexpr int LT_TMEM = 512;                  // columns: O (256), S0, S1 (64 each)
constexpr int LT_S = 256;
constexpr uint32_t LT_HI = 16u << 16;         // lanes 16 .. 31 of each quarter: output dims 256 .. 511
constexpr int LT_BAD_SLOTS = 16;

struct LtCtrl {
    uint64_t kvfull[2], kvempty[2], sfull[2], sfree[2], pfull, pvdone, qfull, qempty, done;
    uint32_t tmem;
    int abort;
    int bad[LT_BAD_SLOTS];   // 1 + the number of a piece that met a block id out of range
    Plan plan;
    long long warp_sums[LT_THREADS / 32];
};
static_assert(sizeof(LtCtrl) <= LT_CTRL, "control block");

template <int KV>
__global__ void __launch_bounds__(LT_THREADS, 1) latent_kernel(const __grid_constant__ CUtensorMap tmkv,
                                                              const __grid_constant__ CUtensorMap tmq,
                                                              const LatentArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    LtCtrl &c = *reinterpret_cast<LtCtrl *>(smem + LT_OFF_CTRL);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    constexpr bool BF16 = KV != PA_KV_F16;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&c.kvfull[s]), 1);
            mbar_init(smem_u32(&c.kvempty[s]), 1);
            mbar_init(smem_u32(&c.sfull[s]), 1);
            mbar_init(smem_u32(&c.sfree[s]), 128);
        }
        mbar_init(smem_u32(&c.pfull), 128);
        mbar_init(smem_u32(&c.pvdone), 1);
        mbar_init(smem_u32(&c.qfull), 1);
        mbar_init(smem_u32(&c.qempty), 2);
        mbar_init(smem_u32(&c.done), 3);
        c.abort = 0;
        for (int k = 0; k < LT_BAD_SLOTS; ++k) c.bad[k] = 0;
        fence_mbar_init();
    }
    make_plan(a, &c.plan, c.warp_sums);
    const Plan plan = c.plan;
    volatile int *abort_flag = &c.abort;
    if (plan.u0 < plan.u1) {   // the whole CTA has work, or none of it
        if (warp == 0) {
            tmem_alloc(smem_u32(&c.tmem), LT_TMEM);
            tmem_relinquish();
        }
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
        const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&c.tmem);
        Walk<LatentArgs> p(a, plan);
        if (warp == 0) {
            // ---- producer: lane j < 8 copies tokens 8 j .. 8 j + 7 of a tile, lanes 8 .. 15 the query rows
            const uint64_t first = policy_evict_first(), keep = policy_evict_normal();
            int cnt = 0, pieces = 0;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                const bool got = !*abort_flag && mbar_wait_bounded(smem_u32(bar), parity, a.wait_limit);
                ok = __all_sync(0xffffffffu, got);
                if (!ok) *abort_flag = 1;
                return ok;
            };
            while (ok && p.next()) {
                const int32_t *row = a.block_tables + (long long)p.seq * a.mbps;
                if (!wait(&c.qempty, (uint32_t)((pieces & 1) ^ 1))) break;
                if (lane == 0) mbar_arrive_expect_tx(smem_u32(&c.qfull), LT_ROWS / 8 * LT_GROUP);
                __syncwarp();
                if (lane >= 8 && lane < 16)
                    tma_load_3d(base + LT_OFF_Q + (lane - 8) * LT_GROUP, &tmq, 0, (int)(a.first_row(p.w, p.r) + 8 * (lane - 8)),
                                0, smem_u32(&c.qfull), keep);
                ++pieces;
                for (int t = p.t0; t < p.t1; ++t) {
                    const int tok = t * LT_TOK + 8 * lane;
                    const bool mine = lane < LT_TOK / 8 && tok < p.w.L;
                    const int32_t blk = mine ? __ldg(row + tok / a.bs) : 0;
                    const int st = cnt & 1;
                    if (!wait(&c.kvempty[st], (uint32_t)(((cnt >> 1) & 1) ^ 1))) break;
                    const unsigned boxes = __ballot_sync(0xffffffffu, mine);
                    const bool bad = __any_sync(0xffffffffu, mine && (blk < 0 || blk >= a.num_blocks));
                    if (lane == 0) {
                        if (bad) *reinterpret_cast<volatile int *>(&c.bad[p.local % LT_BAD_SLOTS]) = p.local + 1;
                        mbar_arrive_expect_tx(smem_u32(&c.kvfull[st]), bad ? 0u : (uint32_t)(__popc(boxes) * LT_GROUP));
                    }
                    __syncwarp();
                    if (!bad && mine)
                        tma_load_3d(base + LT_OFF_KV + st * LT_STAGE + lane * LT_GROUP, &tmkv, 0,
                                    (int)((long long)blk * a.bs) + tok % a.bs, 0, smem_u32(&c.kvfull[st]), first);
                    __syncwarp();
                    ++cnt;
                }
            }
            // the last copies into every buffer have landed before the CTA leaves
            for (int s = 0; s < 2; ++s)
                if (cnt > s)
                    mbar_wait_bounded(smem_u32(&c.kvfull[s]), (uint32_t)(((cnt - 1 - s) / 2) & 1), WAIT_LIMIT);
            if (pieces) mbar_wait_bounded(smem_u32(&c.qfull), (uint32_t)((pieces - 1) & 1), WAIT_LIMIT);
        } else if (warp < 4) {
            // ---- MMA issuers, one thread each: warps 1 and 2 the S products of even and odd KV tiles, warp 3 P V
            if (lane == 0) {
                bool ok = true;
                auto wait = [&](uint64_t *bar, uint32_t parity) {
                    ok = !*abort_flag && mbar_wait_bounded(smem_u32(bar), parity, a.wait_limit);
                    if (!ok) *abort_flag = 1;
                    return ok;
                };
                int n = 0, pieces = 0;   // KV tiles and pieces so far
                if (warp < 3) {
                    const int e = warp - 1;
                    constexpr uint32_t ID = idesc_f16(LT_ROWS, LT_TOK, BF16, false);
                    const uint64_t dq = sw128_desc(base + LT_OFF_Q, 16, LT_GROUP);
                    const uint64_t dk = sw128_desc(base + LT_OFF_KV + e * LT_STAGE, 16, LT_GROUP);
                    const uint32_t d = tmem + LT_S + 64 * e;
                    while (ok && p.next()) {
                        if (!wait(&c.qfull, (uint32_t)(pieces & 1))) break;
                        ++pieces;
                        for (int t = p.t0; t < p.t1; ++t, ++n) {
                            if ((n & 1) != e) continue;
                            if (!wait(&c.sfree[e], (uint32_t)(((n >> 1) & 1) ^ 1))) break;
                            if (!wait(&c.kvfull[e], (uint32_t)((n >> 1) & 1))) break;
                            tc_fence_after_sync();
#pragma unroll
                            for (int k = 0; k < LROW / 16; ++k) {
                                const uint64_t off = (uint64_t)(((k >> 2) * 1024 + (k & 3) * 32) >> 4);
                                umma_f16(d, dq + off, dk + off, ID, k > 0 ? 1u : 0u);
                            }
                            umma_commit(smem_u32(&c.sfull[e]));
                        }
                        if (ok) umma_commit(smem_u32(&c.qempty));   // after this issuer's last product of the piece
                    }
                } else {
                    constexpr uint32_t ID = idesc_f16(LT_ROWS, LC / 2, BF16, true);
                    const uint64_t dp = sw128_desc(base + LT_OFF_P, 16, 1024);
                    const uint64_t dv0 = sw128_desc(base + LT_OFF_KV, 1024, LT_GROUP);
                    while (ok && p.next()) {
                        for (int t = p.t0; t < p.t1; ++t, ++n) {
                            const int st = n & 1;
                            if (!wait(&c.kvfull[st], (uint32_t)((n >> 1) & 1))) break;
                            if (!wait(&c.pfull, (uint32_t)(n & 1))) break;
                            tc_fence_after_sync();
                            const uint64_t dv = dv0 + (uint64_t)(st * (LT_STAGE >> 4));
#pragma unroll
                            for (int k = 0; k < LT_TOK / 16; ++k) {
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    umma_f16(tmem + (h ? LT_HI : 0u), dp + (uint64_t)((k * 32) >> 4),
                                             dv + (uint64_t)((k * 2 * LT_GROUP + h * 4096) >> 4), ID,
                                             t > p.t0 || k > 0 ? 1u : 0u);
                            }
                            umma_commit(smem_u32(&c.pvdone));
                            umma_commit(smem_u32(&c.kvempty[st]));
                        }
                    }
                }
                // every product issued has completed before tensor memory is freed
                umma_commit(smem_u32(&c.done));
                mbar_wait_bounded(smem_u32(&c.done), 0, WAIT_LIMIT);
            }
            __syncwarp();
        } else {
            // ---- softmax: row 16 (warp - 4) + (lane & 15); lanes 0 .. 15 take tokens 0 .. 31 of a tile and
            // output dims 0 .. 255, lanes 16 .. 31 the others
            const int q = warp - 4, half = lane >> 4, m = 16 * q + (lane & 15), tid = threadIdx.x - 128;
            const uint32_t trow = tmem + ((uint32_t)(32 * q) << 16);
            uint8_t *prow = smem + LT_OFF_P + m * 128;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                const bool got = !*abort_flag && mbar_wait_bounded(smem_u32(bar), parity, a.wait_limit);
                ok = __all_sync(0xffffffffu, got);
                if (!ok) *abort_flag = 1;
                return ok;
            };
            int n = 0;
            while (ok && p.next()) {
                const int rows = a.rows(p.w, p.r);
                const bool live = 16 * q < rows;      // some row of this warp exists
                const bool mine = m < rows;
                const int vis = mine ? p.w.L - p.w.T + (int)(((long long)p.r * LT_ROWS + m) / a.H) + 1 : p.w.L;
                float mrun = -INFINITY, l = 0.f;
                for (int t = p.t0; t < p.t1 && ok; ++t, ++n) {
                    const int st = n & 1, t0 = t * LT_TOK;
                    if (!wait(&c.sfull[st], (uint32_t)((n >> 1) & 1))) break;
                    tc_fence_after_sync();
                    uint32_t pw[16];
                    float alpha = 1.f;
                    bool grew = false;
                    if (live) {
                        uint32_t sr[32];
                        tmem_ld_half32(trow + LT_S + 64 * st, sr);
                        tmem_wait_ld();
                        tc_fence_before_sync();
                        float s[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) s[k] = __uint_as_float(sr[k]);
                        const int first = t0 + 32 * half;
                        if (first + 32 > vis) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) s[k] = first + k < vis ? s[k] : -INFINITY;
                        }
                        float mp[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                        for (int k = 4; k < 32; ++k) mp[k & 3] = fmaxf(mp[k & 3], s[k]);
                        float mx = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16)) * a.scale_log2;
                        const bool grow = mx > mrun + RESCALE_THRESHOLD;
                        grew = __any_sync(0xffffffffu, grow);
                        if (grew) {
                            const float nm = grow ? mx : mrun;
                            alpha = grow ? fast_exp2(mrun - nm) : 1.f;
                            l *= alpha;
                            mrun = nm;
                        }
                        const float mu = mrun == -INFINITY ? 0.f : mrun;   // a row that has seen nothing yet
                        float lp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float x = fast_exp2(fmaf(s[2 * k], a.scale_log2, -mu));
                            const float y = fast_exp2(fmaf(s[2 * k + 1], a.scale_log2, -mu));
                            lp[k & 1] += x;
                            lp[2 + (k & 1)] += y;
                            pw[k] = pack_p<KV>(x, y);
                        }
                        l += (lp[0] + lp[1]) + (lp[2] + lp[3]);
                    }
                    mbar_arrive(smem_u32(&c.sfree[st]));
                    // P is free, and O up to date, once the previous product is done
                    if (n > 0 && !wait(&c.pvdone, (uint32_t)((n - 1) & 1))) break;
                    if (live) {
                        if (grew && t > p.t0) {
                            tc_fence_after_sync();
#pragma unroll 1
                            for (int k = 0; k < 8; ++k) {
                                uint32_t o[32];
                                tmem_ld32(trow + 32 * k, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                                tmem_st32(trow + 32 * k, o);
                            }
                            tmem_wait_st();
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<uint4 *>(prow + (((4 * half + k) ^ (m & 7)) << 4)) =
                                make_uint4(pw[4 * k], pw[4 * k + 1], pw[4 * k + 2], pw[4 * k + 3]);
                    }
                    if (t0 + LT_TOK > p.w.L) {
                        // the context's last tile: rows past it hold anything, and P is 0 there
                        uint8_t *kv = smem + LT_OFF_KV + st * LT_STAGE;
                        for (int k = tid + (p.w.L - t0) * 64; k < LT_TOK * 64; k += 128) {
                            const int r = k >> 6, cc = k & 63;
                            *reinterpret_cast<uint4 *>(kv + (r >> 3) * LT_GROUP + (cc >> 3) * 1024 + (r & 7) * 128 +
                                                       (cc & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_proxy_async_smem();
                    tc_fence_before_sync();
                    mbar_arrive(smem_u32(&c.pfull));
                }
                if (!ok) break;
                // ---- the piece's rows: finished, or a partial row
                if (!wait(&c.pvdone, (uint32_t)((n - 1) & 1))) break;
                tc_fence_after_sync();
                if (live) {
                    l += __shfl_xor_sync(0xffffffffu, l, 16);
                    const bool bad = *reinterpret_cast<volatile int *>(&c.bad[p.local % LT_BAD_SLOTS]) == p.local + 1;
                    if (bad) l = __int_as_float(0x7fc00000);
                    const bool whole = p.whole();
                    const float inv = 1.f / l;
                    uint16_t *orow = a.out + (a.first_row(p.w, p.r) + m) * LC + 256 * half;
                    float *part = a.o + ((long long)p.slot() * LT_ROWS + m) * LC + 256 * half;
                    if (!whole && mine && half == 0) a.ml[p.slot() * LT_ROWS + m] = make_float2(mrun, l);
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) {
                        uint32_t o[32];
                        tmem_ld32(trow + 32 * k, o);
                        tmem_wait_ld();
                        if (mine && whole) {
#pragma unroll
                            for (int j = 0; j < 32; j += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    w[i] = (uint32_t)out_bits<KV>(__uint_as_float(o[j + 2 * i]) * inv) |
                                           ((uint32_t)out_bits<KV>(__uint_as_float(o[j + 2 * i + 1]) * inv) << 16);
                                *reinterpret_cast<uint4 *>(orow + 32 * k + j) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        } else if (mine) {
#pragma unroll
                            for (int j = 0; j < 32; j += 4)
                                *reinterpret_cast<uint4 *>(part + 32 * k + j) =
                                    make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                        }
                        __syncwarp();   // the next load is the whole warp's
                    }
                }
                tc_fence_before_sync();
            }
        }
        tc_fence_before_sync();
        __syncthreads();
        if (warp == 0) {
            tc_fence_after_sync();
            tmem_dealloc(tmem, LT_TMEM);
        }
    }
    if (threadIdx.x == 0) a.status[blockIdx.x] = c.abort;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------ merge

// One CTA per query row: rows of a cut row tile from their pieces' partial rows,
// zeros for an empty context, NaN for an invalid one (and for every row when a
// CTA of the first kernel gave up).  Four groups of 128 threads take every
// fourth piece, four output dims a thread.
template <int KV>
__global__ void __launch_bounds__(512) latent_merge_kernel(const LatentArgs a, int ctas) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float4 so[3][128];
    __shared__ float sl[3];
    const long long row = blockIdx.x;
    const int qt = (int)(row / a.H);
    int failed = 0;
    for (int i = threadIdx.x; i < ctas; i += blockDim.x) failed |= a.status[i];
    failed = __syncthreads_or(failed);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->error = failed ? PA_ERR_TIMEOUT : PA_OK;
    const long long total = a.unit_base[a.num_seqs];
    uint16_t *orow = a.out + row * LC;
    const int seq = a.query_start && total >= 0 ? sequence_of(a.query_start, a.num_seqs, qt) : qt;
    LatentArgs::Seq w{};
    if (total >= 0) w = a.seq_work(seq);
    if (failed || total < 0 || !w.valid || w.tiles == 0) {
        const uint16_t x = !failed && total >= 0 && w.valid ? 0 : out_bits<KV>(__int_as_float(0x7fc00000));
        for (int d = threadIdx.x; d < LC; d += blockDim.x) orow[d] = x;
        return;
    }
    const long long idx = row - (long long)w.q0 * a.H;
    const int r = (int)(idx / LT_ROWS), m = (int)(idx % LT_ROWS);
    const Pieces pc(a.unit_base[seq] + a.start(w, r), a.row_tiles(w, r), LatentArgs::COST, total, ctas);
    if (pc.k0 == pc.k1) return;   // finished by one CTA
    const int g = threadIdx.x >> 7, d = threadIdx.x & 127;
    float M = -INFINITY;
#pragma unroll 8
    for (int k = pc.k0; k <= pc.k1; ++k) M = fmaxf(M, a.ml[pc.slot(k) * LT_ROWS + m].x);
    const float mu = M == -INFINITY ? 0.f : M;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int k = pc.k0 + g; k <= pc.k1; k += 4) {
        const int slot = pc.slot(k);
        const float2 ml = a.ml[slot * LT_ROWS + m];
        const float4 o = *reinterpret_cast<const float4 *>(a.o + ((long long)slot * LT_ROWS + m) * LC + 4 * d);
        const float wt = fast_exp2(ml.x - mu);
        l = fmaf(ml.y, wt, l);
        acc.x = fmaf(o.x, wt, acc.x);
        acc.y = fmaf(o.y, wt, acc.y);
        acc.z = fmaf(o.z, wt, acc.z);
        acc.w = fmaf(o.w, wt, acc.w);
    }
    if (g) {
        so[g - 1][d] = acc;
        if (d == 0) sl[g - 1] = l;
    }
    __syncthreads();
    if (g == 0) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const float4 x = so[k][d];
            acc.x += x.x;
            acc.y += x.y;
            acc.z += x.z;
            acc.w += x.w;
            l += sl[k];
        }
        const float inv = 1.f / l;
        uint2 v;
        v.x = (uint32_t)out_bits<KV>(acc.x * inv) | ((uint32_t)out_bits<KV>(acc.y * inv) << 16);
        v.y = (uint32_t)out_bits<KV>(acc.z * inv) | ((uint32_t)out_bits<KV>(acc.w * inv) << 16);
        *reinterpret_cast<uint2 *>(orow + 4 * d) = v;
    }
}

// ------------------------------------------------------------------ launch

struct LtLayout {
    size_t status, unit_base, ml, o, total;
};

LtLayout lt_layout(int num_seqs) {
    LtLayout l;
    size_t at = 256;   // header
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at = (at + bytes + 255) / 256 * 256;
        return p;
    };
    l.status = take(sizeof(int) * AXIS_MAX_CTAS);
    l.unit_base = take(sizeof(long long) * ((size_t)num_seqs + 1));
    l.ml = take(sizeof(float2) * 2 * AXIS_MAX_CTAS * LT_ROWS);
    l.o = take(sizeof(float) * 2 * AXIS_MAX_CTAS * LT_ROWS * LC);
    l.total = at;
    return l;
}

// 3-D view of rows of 576 16-bit elements: 64-column blocks x rows x nine
// blocks, boxes of 8 rows over all blocks (nine 1024-byte swizzled atoms).
bool row_map(CUtensorMap *map, const void *base, long long rows, int kv) {
    auto enc = tma_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {64, (cuuint64_t)rows, LROW / 64};
    cuuint64_t strides[2] = {2 * LROW, 128};
    cuuint32_t box[3] = {64, 8, LROW / 64};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, kv == PA_KV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
               const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared-memory limits are set per device, on its first call.
template <int KV>
cudaError_t lt_setup() {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    if (const cudaError_t e = cudaGetDevice(&dev)) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64 && done[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(latent_kernel<KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, LT_SMEM);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
    return e;
}

template <int KV>
int launch_merge(const LatentArgs &a, int ctas, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.num_query_tokens * a.H));
    cfg.blockDim = dim3(512);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;   // launched while the first kernel drains
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, latent_merge_kernel<KV>, a, ctas));
}

template <int KV>
int launch_latent(const LatentArgs &a, cudaStream_t st) {
    if (lt_setup<KV>() != cudaSuccess) return PA_ERR_CUDA;
    CUtensorMap tmkv, tmq;
    if (!row_map(&tmkv, a.cache, a.num_blocks * a.bs, KV) ||
        !row_map(&tmq, a.query, (long long)a.num_query_tokens * a.H, KV))
        return PA_ERR_CUDA;
    const int ctas = std::min(num_sms(), AXIS_MAX_CTAS);
    latent_kernel<KV><<<ctas, LT_THREADS, LT_SMEM, st>>>(tmkv, tmq, a);
    if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
    return launch_merge<KV>(a, ctas, st);
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
    return lt_layout(num_seqs).total;
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
    if ((long long)num_query_tokens * num_heads >= (1LL << 31)) return PA_ERR_UNSUPPORTED;
    if (num_query_tokens == 0) return PA_OK;
    if (!out || !query || !cache || !block_tables || !context_lens || !aligned16(out) || !aligned16(query) ||
        !aligned16(cache))
        return PA_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < pa_latent_attention_workspace_size(num_seqs, num_query_tokens, num_heads, max_context_len))
        return PA_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const LtLayout lay = lt_layout(num_seqs);
    LatentArgs a{};
    a.out = static_cast<uint16_t *>(out);
    a.query = static_cast<const uint16_t *>(query);
    a.cache = static_cast<const uint8_t *>(cache);
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.hdr = reinterpret_cast<WsHeader *>(ws);
    a.num_seqs = num_seqs;
    a.num_query_tokens = num_query_tokens;
    a.H = num_heads;
    a.bs = block_size;
    a.mbps = max_blocks_per_seq;
    a.max_context_len = max_context_len;
    a.num_blocks = num_blocks;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.wait_limit = pipeline_wait_limit();
    a.status = reinterpret_cast<int *>(ws + lay.status);
    a.unit_base = reinterpret_cast<long long *>(ws + lay.unit_base);
    a.ml = reinterpret_cast<float2 *>(ws + lay.ml);
    a.o = reinterpret_cast<float *>(ws + lay.o);
    if (kv_dtype == PA_KV_F16) return launch_latent<PA_KV_F16>(a, st);
    if (kv_dtype == PA_KV_BF16) return launch_latent<PA_KV_BF16>(a, st);
    const unsigned grid = (unsigned)num_query_tokens * num_heads;
    latent_simple_kernel<PA_KV_FP8_E4M3><<<grid, 256, 0, st>>>(a);
    return cuda_status(cudaGetLastError());
}
