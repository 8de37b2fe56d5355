// Attention in the expanded form: every head's keys and values have been
// computed from the latents, contiguous and ragged (no block table), keys of
// 128 + 64 elements whose last 64 all heads share.
//
// A row tile is 256 consecutive new tokens of one sequence and one head, in two
// halves of 128 rows that share every key and value block the CTA loads.  Its
// causal KV tiles are a stretch of the work axis (work_axis.cuh), cut into
// equal ranges over the CTAs, so that a chunk of few heads or a ragged batch
// leaves no CTA idle in a last round (2048 new tokens of 32 heads are 256 row
// tiles for 152 CTAs: whole tiles would take two rounds where 1.7 do).
//
// Warps: 0 loads, 1 and 3 idle, 2 issues the MMAs, 4-7 and 8-11 run the softmax
// of the two halves, one row per thread.  Tensor memory: S0, S1, O0, O1 (128
// columns each); P is written over the first 64 columns of its S.  Shared
// memory: both halves' queries (96 KB) and a ring of eight 16 KB blocks (128
// tokens x 64 elements), which the three blocks of a key tile and the two of a
// value tile pass through in the order in which the MMAs take them: 128 KB hold
// 1.6 KV tiles, where whole tiles would leave room for one and a half stages.
// MMA order: PV0(n), S0(n + 1), PV1(n), S1(n + 1): while one half's softmax works
// on its S, the other half's products run.  The MMAs of one thread complete in
// issue order, so when S_x(n) is complete so is PV_x(n - 1).
//
// Probabilities are rounded to the 16-bit type because the second product's operands
// have one type (l takes them unrounded): against 64 bits the whole is off by 0.0023
// normwise in bf16 and 0.00025 in fp16, 32-bit arithmetic rounded once by 0.0017 and
// 0.0002.
//
// What bounds it (one GB300): 2048 new of 12,000 tokens, 32 heads, bf16: 360 us,
// 1278 TFLOP/s, tensor pipe 58 % busy.  The S products read their queries from
// shared memory (107 clocks for M 128, N 128, K 16; 64 from tensor memory, which S,
// P and O of two halves fill), and the keys and values, read by eight row tiles a
// head, come 3.8 times from HBM.  A 600-token prompt of 16 heads takes 24 us, a
// chain of the plan, the loads, one to three KV tiles, partial rows and the merge.

#include <algorithm>
#include <climits>
#include <cmath>

#include "decode_common.cuh"
#include "latent.h"
#include "umma.cuh"
#include "work_axis.cuh"

namespace pa {
namespace {

constexpr int EN = 128, ER = PA_LATENT_ROPE_DIM, EQ = EN + ER, EV = 128;
constexpr int EX_HALF = 128;               // rows of a half
constexpr int EX_ROWS = 2 * EX_HALF;       // rows of a row tile
constexpr int EX_TOK = 128;                // tokens of a KV tile
constexpr int EX_PAST = 2;                 // teams of two from a past of this many times the new tokens on

struct ExpandedArgs {
    uint16_t *out;
    const int32_t *query_start, *kv_start;
    WsHeader *hdr;
    int num_seqs, num_query_tokens, num_kv_tokens, H;
    float scale_log2;
    long long wait_limit;
    // workspace
    int *status;            // [AXIS_MAX_CTAS] nonzero: the CTA gave up waiting
    Cut *cuts;              // [AXIS_MAX_CTAS]
    float2 *ml;             // [2 AXIS_MAX_CTAS][EX_ROWS] maximum (log2 units) and sum of a partial row
    float4 *o;              // [2 AXIS_MAX_CTAS][EX_ROWS * EV / 4] its unnormalised output (see partial_at)

    // ---- the work axis: row tile r of a sequence is tile r % tiles_per_head of head r / tiles_per_head
    static constexpr int COST = 4;   // 600 tokens, 16 heads: 27.6 us with 1, 26.6 with 4, 27.9 with 6
    struct Seq {
        int L, T, q0, k0;
        int per_head;   // row tiles of a head
        int rts;
        bool valid;
    };
    __device__ __forceinline__ Seq seq_work(int i) const {
        Seq w;
        w.q0 = query_start[i];
        w.T = query_start[i + 1] - w.q0;
        w.k0 = kv_start[i];
        w.L = kv_start[i + 1] - w.k0;
        w.valid = w.T <= w.L;
        w.per_head = w.valid ? (w.T + EX_ROWS - 1) / EX_ROWS : 0;
        w.rts = w.per_head * H;
        return w;
    }
    // Row tile i of a head, but the last, sees ceil(past / 128) + 2 (i + 1) KV
    // tiles; a team's two count as the later one.
    __device__ __forceinline__ long long start(const Seq &w, int j, int team) const {
        const int per = w.per_head / team;
        if (per == 0) return 0;
        const long long past = (w.L - w.T + EX_TOK - 1) / EX_TOK;
        auto before = [&](long long i) { return i * (COST + past) + team * i * (i + 1); };
        const int h = j / per, i = j - h * per;
        return h * (before(per - 1) + COST + (w.L + EX_TOK - 1) / EX_TOK) + before(i);
    }
    __device__ __forceinline__ int row_tile_at(const Seq &w, long long u, int team) const {
        const int per = w.per_head / team;   // (of a sequence with work)
        const int h = (int)quick_div(u, start(w, per, team));
        int r = h * per, hi = r + per;
        while (hi - r > 1) {
            const int mid = (r + hi) >> 1;
            if (start(w, mid, team) <= u) r = mid; else hi = mid;
        }
        return r;
    }
    // In teams where a sequence's past is long against its new tokens, so that
    // the two row tiles' KV ranges are nearly the same (2048 of 12000 tokens, 32
    // heads: 358 us in teams, 378 without).
    __device__ __forceinline__ bool in_teams(const Seq &w) const {
        return w.per_head % 2 == 0 && (w.per_head == 0 || w.L - w.T >= EX_PAST * w.T);
    }
    // KV tiles of the first `rows` new tokens.
    __device__ __forceinline__ int tiles_of(const Seq &w, int rows) const {
        return (w.L - w.T + rows + EX_TOK - 1) / EX_TOK;
    }
    __device__ __forceinline__ int row_tiles(const Seq &w, int r) const {
        return tiles_of(w, min(w.T, (r % w.per_head + 1) * EX_ROWS));
    }
    __device__ __forceinline__ int cut_rows(const Seq &w, int r) const {
        return min(EX_ROWS, w.T - r % w.per_head * EX_ROWS);
    }
    __device__ __forceinline__ long long first_row(const Seq &w, int r) const {   // later rows: H apart
        return (long long)(w.q0 + r % w.per_head * EX_ROWS) * H + r / w.per_head;
    }
    __device__ __forceinline__ int first_tiles(const Seq &w, int r) const {   // the first half's, of two
        return tiles_of(w, min(w.T, r % w.per_head * EX_ROWS + EX_HALF));
    }
    __device__ __forceinline__ bool seq_ok(int i) const {
        return query_start[i] <= query_start[i + 1] && kv_start[i] <= kv_start[i + 1];
    }
    __device__ __forceinline__ bool ends_ok() const {
        return *query_start == 0 && query_start[num_seqs] == num_query_tokens && *kv_start == 0 &&
               kv_start[num_seqs] == num_kv_tokens;
    }
};

// Where the softmax keeps four dims (32 k + 4 j ..) of a row, in float4: a store
// of a warp's 32 rows (rows 32 q .. of the row tile's 256) is one run of 512 bytes.
__device__ __forceinline__ long long partial_at(int slot, int q, int k, int j, int lane) {
    return (((long long)slot * 8 + q) * 4 + k) * 8 * 32 + j * 32 + lane;
}

// The halves of a piece: half 0 the later rows, which see the longer range,
// half 1 the earlier ones (no tiles if the row tile has at most 128 rows, or if
// the piece lies past what they see).
struct Half {
    int row0;     // first new token
    int ntiles;   // KV tiles that its rows see
    int n;        // KV tiles of the piece that it takes, from the piece's first on
};

__device__ __forceinline__ Half half_of(const ExpandedArgs &a, const Walk<ExpandedArgs> &p, int x) {
    const int first = p.r % p.w.per_head * EX_ROWS;
    const bool both = p.w.T - first > EX_HALF;
    Half h;
    h.row0 = first + (both && x == 0 ? EX_HALF : 0);
    h.ntiles = x == 0 ? p.ntiles : both ? a.tiles_of(p.w, first + EX_HALF) : 0;
    h.n = max(0, min(p.t1, h.ntiles) - p.t0);
    return h;
}

constexpr int EX_THREADS = 12 * 32;
constexpr int EX_BLOCK = EX_TOK * 128;               // 128 rows x 64 elements, 128-byte swizzle
constexpr int EX_RING = 8;
constexpr int EX_Q = 3 * EX_BLOCK;                   // one half's queries
constexpr int EX_OFF_RING = 2 * EX_Q;
constexpr int EX_OFF_CTRL = EX_OFF_RING + EX_RING * EX_BLOCK;
constexpr int EX_CTRL = 1024;
constexpr int EX_SMEM = EX_OFF_CTRL + EX_CTRL + 1024;   // + alignment slack
static_assert(EX_SMEM <= 227 * 1024, "shared memory of one CTA");
constexpr int EX_TMEM = 512, EX_O = 256;             // S0, S1 at columns 0 and 128; O0, O1 at 256 and 384
constexpr int EX_REGS_LAUNCH = 168;                  // per thread at launch: 65536 / 384, rounded down to 8
constexpr int EX_REGS_LOW = 104;                     // warpgroup 0
constexpr int EX_REGS_HIGH = 200;                    // the softmax warpgroups
static_assert(128 * EX_REGS_LOW + 256 * EX_REGS_HIGH <= EX_THREADS * EX_REGS_LAUNCH,
              "register split within the launch's pool");

constexpr uint32_t EX_LAST = 0x7fffffffu;

struct ExCtrl {
    uint64_t full[EX_RING], empty[EX_RING], qfull[2], qempty[2], sfull[2], pfull[2], pvdone[2], done;
    uint32_t tmem;
    int abort;
    Plan plan;
    long long warp_sums[EX_THREADS / 32];
    // For each half, by the number of a piece among those that it takes: 1 + that
    // number in the high word, and in the low one how far below the largest position
    // the piece's first non-finite value of a new token is.  Half 0 writes both
    // halves' records before it hands over a P.  Two of each are enough: half 0 has
    // the first S of the half's piece k + 2 only after the MMA thread has had every P
    // of that half's piece k + 1, and so after all its warps have read piece k's.
    unsigned long long poison[2][2];
};
static_assert(sizeof(ExCtrl) <= EX_CTRL, "control block");

// One lane: queries and ring blocks in the order the MMAs take them.
__device__ void ex_load(uint8_t *smem, ExCtrl &c, const ExpandedArgs &a, Walk<ExpandedArgs> &p, const CUtensorMap *tmq,
                        const CUtensorMap *tmk, const CUtensorMap *tmr, const CUtensorMap *tmv) {
    const uint32_t base = smem_u32(smem);
    const uint64_t keep = policy_evict_normal();
    volatile int *abort_flag = &c.abort;
    int cnt = 0, qc[2] = {0, 0};
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        ok = ok && !*abort_flag && mbar_wait_bounded(smem_u32(bar), parity, a.wait_limit);
        if (!ok) *abort_flag = 1;
        return ok;
    };
    // a free ring slot's address and barrier
    auto slot = [&](uint32_t &bar) {
        const int s = cnt % EX_RING;
        if (!wait(&c.empty[s], (uint32_t)(((cnt / EX_RING) & 1) ^ 1))) return 0u;
        bar = smem_u32(&c.full[s]);
        mbar_arrive_expect_tx(bar, EX_BLOCK);
        ++cnt;
        return base + EX_OFF_RING + s * EX_BLOCK;
    };
    while (ok && p.next()) {
        const int head = p.r / p.w.per_head;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const Half h = half_of(a, p, x);
            if (h.n == 0) continue;
            if (!wait(&c.qempty[x], (uint32_t)((qc[x] & 1) ^ 1))) break;
            const uint32_t bar = smem_u32(&c.qfull[x]);
            mbar_arrive_expect_tx(bar, EX_Q);
            for (int b = 0; b < 3; ++b)
                tma_load_3d(base + x * EX_Q + b * EX_BLOCK, tmq, 64 * b, head, p.w.q0 + h.row0, bar, keep);
            ++qc[x];
        }
        for (int t = p.t0; ok && t < p.t1; ++t) {
            const int y = p.w.k0 + t * EX_TOK;
            uint32_t bar, dst;
            for (int b = 0; ok && b < 2; ++b)
                if ((dst = slot(bar))) tma_load_3d(dst, tmk, 64 * b, head, y, bar, keep);
            if (ok && (dst = slot(bar))) tma_load_2d(dst, tmr, 0, y, bar, keep);
            for (int b = 0; ok && b < 2; ++b)
                if ((dst = slot(bar))) tma_load_3d(dst, tmv, 64 * b, head, y, bar, keep);
        }
    }
    // the last copies into every buffer have landed before the CTA leaves
    for (int s = 0; s < EX_RING; ++s)
        if (cnt > s)
            mbar_wait_bounded(smem_u32(&c.full[s]), (uint32_t)(((cnt - 1 - s) / EX_RING) & 1), WAIT_LIMIT);
    for (int x = 0; x < 2; ++x)
        if (qc[x]) mbar_wait_bounded(smem_u32(&c.qfull[x]), (uint32_t)((qc[x] - 1) & 1), WAIT_LIMIT);
}

// One lane: the MMAs.
template <int KV>
__device__ void ex_mma(uint8_t *smem, ExCtrl &c, const ExpandedArgs &a, Walk<ExpandedArgs> &p, uint32_t tmem) {
    const uint32_t base = smem_u32(smem);
    constexpr uint32_t ID_S = idesc_f16(EX_HALF, EX_TOK, KV == PA_KV_BF16, false);
    constexpr uint32_t ID_O = idesc_f16(EX_HALF, EV, KV == PA_KV_BF16, true);
    constexpr uint32_t ID_O64 = idesc_f16(EX_HALF, EV / 2, KV == PA_KV_BF16, true);
    const uint64_t dq0 = sw128_desc(base, 16, 1024);
    const uint64_t dk0 = sw128_desc(base + EX_OFF_RING, 16, 1024);
    const uint64_t dv0 = sw128_desc(base + EX_OFF_RING, EX_BLOCK, 1024);
    volatile int *abort_flag = &c.abort;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        ok = ok && !*abort_flag && mbar_wait_bounded(smem_u32(bar), parity, a.wait_limit);
        if (!ok) *abort_flag = 1;
        return ok;
    };
    int cnt = 0, qc[2] = {0, 0}, pc[2] = {0, 0};   // ring blocks released; queries and P tiles taken
    auto ring_wait = [&](int k) { return wait(&c.full[k % EX_RING], (uint32_t)((k / EX_RING) & 1)); };
    // S_x = Q_x K^T, the key tile in ring blocks cnt .. cnt + 2 (waited for by half 0)
    auto issue_s = [&](int x, int at, bool load) {
        for (int b = 0; b < 3; ++b) {
            if (load) {
                if (!ring_wait(at + b)) return;
                tc_fence_after_sync();
            }
            const uint64_t dk = dk0 + (uint64_t)((at + b) % EX_RING * (EX_BLOCK >> 4));
            const uint64_t dq = dq0 + (uint64_t)((x * EX_Q + b * EX_BLOCK) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                umma_f16(tmem + x * EX_TOK, dq + 2 * k, dk + 2 * k, ID_S, b > 0 || k > 0 ? 1u : 0u);
        }
        umma_commit(smem_u32(&c.sfull[x]));
    };
    // O_x += P_x V, the value tile in ring blocks at and at + 1 (64 dims each), P_x
    // over S_x: one product of N 128, or, where the ring wraps between the two
    // (every eighth tile), two of N 64
    auto issue_pv = [&](int x, int at, int n) {
        const int b0 = at % EX_RING;
        const uint64_t dv = dv0 + (uint64_t)(b0 * (EX_BLOCK >> 4));
        const uint32_t o = tmem + EX_O + x * EV, pt = tmem + x * EX_TOK;
        if (b0 + 1 < EX_RING) {
#pragma unroll
            for (int k = 0; k < EX_TOK / 16; ++k)   // 16 tokens: P columns 8 k .. 8 k + 7, V rows 16 k ..
                umma_f16_ts(o, pt + 8 * k, dv + (uint64_t)((k * 16 * 128) >> 4), ID_O, n > 0 || k > 0 ? 1u : 0u);
        } else {
#pragma unroll
            for (int k = 0; k < EX_TOK / 16; ++k) {
                umma_f16_ts(o, pt + 8 * k, dv + (uint64_t)((k * 16 * 128) >> 4), ID_O64, n > 0 || k > 0 ? 1u : 0u);
                umma_f16_ts(o + 64, pt + 8 * k, dv0 + (uint64_t)((k * 16 * 128) >> 4), ID_O64,
                            n > 0 || k > 0 ? 1u : 0u);
            }
        }
        umma_commit(smem_u32(&c.pvdone[x]));
    };
    while (ok && p.next()) {
        const int n0 = half_of(a, p, 0).n, n1 = half_of(a, p, 1).n;
        if (!wait(&c.qfull[0], (uint32_t)(qc[0]++ & 1))) break;
        if (n1 > 0 && !wait(&c.qfull[1], (uint32_t)(qc[1]++ & 1))) break;
        issue_s(0, cnt, true);
        if (!ok) break;
        if (n1 > 0) issue_s(1, cnt, false);
        for (int b = 0; b < 3; ++b) umma_commit(smem_u32(&c.empty[(cnt + b) % EX_RING]));
        cnt += 3;
        for (int n = 0; n < n0; ++n) {   // ring: V(n), then K(n + 1)
            if (n + 1 == n0) umma_commit(smem_u32(&c.qempty[0]));
            if (n + 1 == n1) umma_commit(smem_u32(&c.qempty[1]));
            const bool more0 = n + 1 < n0, more1 = n + 1 < n1;
            if (!wait(&c.pfull[0], (uint32_t)(pc[0]++ & 1)) || !ring_wait(cnt) || !ring_wait(cnt + 1)) break;
            tc_fence_after_sync();
            issue_pv(0, cnt, n);
            if (more0) issue_s(0, cnt + 2, true);
            if (!ok) break;
            if (n < n1) {
                if (!wait(&c.pfull[1], (uint32_t)(pc[1]++ & 1))) break;
                tc_fence_after_sync();
                issue_pv(1, cnt, n);
                if (more1) issue_s(1, cnt + 2, false);
            }
            const int used = more0 ? 5 : 2;
            for (int b = 0; b < used; ++b) umma_commit(smem_u32(&c.empty[(cnt + b) % EX_RING]));
            cnt += used;
        }
    }
    // every product issued has completed before tensor memory is freed
    umma_commit(smem_u32(&c.done));
    mbar_wait_bounded(smem_u32(&c.done), 0, WAIT_LIMIT);
}

// One warpgroup: the softmax of half x, a row per thread.
template <int KV>
__device__ void ex_softmax(uint8_t *smem, ExCtrl &c, const ExpandedArgs &a, Walk<ExpandedArgs> &p, uint32_t tmem, int x) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, m = quarter * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t scol = (uint32_t)(x * EX_TOK), ocol = (uint32_t)(EX_O + x * EV);
    const float sl2 = a.scale_log2;
    volatile int *abort_flag = &c.abort;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        const bool got = ok && !*abort_flag && mbar_wait_bounded(smem_u32(bar), parity, a.wait_limit);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) *abort_flag = 1;
        return ok;
    };
    int sc = 0, cnt = 0;   // S_x and P_x so far; ring blocks before this piece
    int both = -1;         // number of the last piece that both halves take
    while (ok && p.next()) {
        const Half h = half_of(a, p, x);
        const int blocks = 5 * (p.t1 - p.t0);
        if (h.n == 0) {
            cnt += blocks;
            continue;
        }
        const bool shared = x == 1 || half_of(a, p, 1).n > 0;
        if (shared) ++both;
        const int tok = h.row0 + m;
        const bool mine = tok < p.w.T;
        const int vis = mine ? p.w.L - p.w.T + tok + 1 : p.w.L;   // positions this row sees
        // what the row tile's first row sees
        const int first_vis = p.w.L - p.w.T + p.r % p.w.per_head * EX_ROWS + 1;
        float mrun = -INFINITY, l = 0.f;
        for (int n = 0; n < h.n && ok; ++n) {
            if (!wait(&c.sfull[x], (uint32_t)(sc & 1))) break;
            // (done when S is; every phase is seen, so that the one waited for last is not taken for another)
            if (n > 0 && !wait(&c.pvdone[x], (uint32_t)((sc - 1) & 1))) break;
            tc_fence_after_sync();
            float s[EX_TOK];
#pragma unroll
            for (int q = 0; q < EX_TOK / 32; ++q) {
                uint32_t r[32];
                tmem_ld32(trow + scol + 32 * q, r);
#pragma unroll
                for (int k = 0; k < 32; ++k) s[32 * q + k] = __uint_as_float(r[k]);
            }
            tmem_wait_ld();
            const int t0 = (p.t0 + n) * EX_TOK;
            if (t0 + EX_TOK > vis) {
#pragma unroll
                for (int k = 0; k < EX_TOK; ++k) s[k] = t0 + k < vis ? s[k] : -INFINITY;
            }
            float mp[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int k = 4; k + 8 <= EX_TOK; k += 8)
#pragma unroll
                for (int j = 0; j < 4; ++j) mp[j] = max3(mp[j], s[k + 2 * j], s[k + 2 * j + 1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) mp[j] = fmaxf(mp[j], s[EX_TOK - 4 + j]);
            const float mx = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])) * sl2;
            // decided per row, done warp-wide (tensor-memory accesses are the
            // whole warp's); rows that do not grow scale by exactly 1
            const bool grow = mx > mrun + RESCALE_THRESHOLD;
            if (__any_sync(0xffffffffu, grow)) {
                const float nm = grow ? mx : mrun;
                const float alpha = grow ? fast_exp2(mrun - nm) : 1.f;
                if (n > 0) {   // PV_x(n - 1) is complete: S_x(n) was committed after it
#pragma unroll 1
                    for (int q = 0; q < EV / 32; ++q) {
                        uint32_t o[32];
                        tmem_ld32(trow + ocol + 32 * q, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                        tmem_st32(trow + ocol + 32 * q, o);
                    }
                    tmem_wait_st();
                }
                l *= alpha;
                mrun = nm;
            }
            // Value rows that some row of the row tile does not see, where P is 0 and
            // a product with an infinity or a NaN would not be: those past the
            // sequence (the next one's, or nothing) are zeroed, and so is what is not
            // finite among the new tokens' (the rows that see it become NaN below).
            // Half 0 does it for both: it runs every KV tile, and PV1(n) is issued
            // after P0(n).
            bool changed = false;
            if (x == 0 && t0 + EX_TOK > first_vis) {
                const int at = cnt + 5 * n + 3;   // the value tile's ring blocks
                int bad = INT_MAX;
#pragma unroll 1
                for (int b = 0; b < 2; ++b) {
                    if (!wait(&c.full[(at + b) % EX_RING], (uint32_t)(((at + b) / EX_RING) & 1))) break;
                    uint4 *blk = reinterpret_cast<uint4 *>(smem + EX_OFF_RING + (at + b) % EX_RING * EX_BLOCK);
                    // this thread's chunks m, m + 128, ..: row m / 8 + 16 i
                    const int lo = max(0, first_vis - t0), hi = p.w.L - t0;
                    bool any = false;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = m / 8 + 16 * i;
                        if (r >= hi)
                            blk[m + EX_HALF * i] = make_uint4(0, 0, 0, 0);
                        else if (r >= lo)
                            any |= not_finite<KV>(blk[m + EX_HALF * i]);
                    }
                    if (any) {
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) {
                            const int r = m / 8 + 16 * i;
                            uint4 &v = blk[m + EX_HALF * i];
                            if (r >= lo && r < hi && not_finite<KV>(v)) {
                                v = make_uint4(finite_part<KV>(v.x), finite_part<KV>(v.y), finite_part<KV>(v.z),
                                               finite_part<KV>(v.w));
                                bad = min(bad, t0 + r);
                            }
                        }
                    }
                }
                if (!ok) break;
                if (bad != INT_MAX) {
                    const uint32_t below = EX_LAST - (uint32_t)bad;
                    atomicMax(&c.poison[0][p.local & 1], (unsigned long long)(p.local + 1) << 32 | below);
                    if (shared) atomicMax(&c.poison[1][both & 1], (unsigned long long)(both + 1) << 32 | below);
                }
                changed = true;
            }
            const float mu = mrun == -INFINITY ? 0.f : mrun;   // a row that has seen nothing yet
            const uint64_t sl2x2 = pair_of(sl2, sl2), negm = pair_of(-mu, -mu);
            uint64_t lp[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) lp[j] = 0;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t r[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    float e0, e1;
                    pair_parts(pair_fma(pair_of(s[64 * q + 2 * k], s[64 * q + 2 * k + 1]), sl2x2, negm), e0, e1);
                    e0 = fast_exp2(e0);
                    e1 = fast_exp2(e1);
                    lp[k & 3] = pair_add(lp[k & 3], pair_of(e0, e1));
                    r[k] = pack_p<KV>(e0, e1);
                }
                tmem_st32(trow + scol + 32 * q, r);
            }
            float l0, l1;
            pair_parts(pair_add(pair_add(lp[0], lp[1]), pair_add(lp[2], lp[3])), l0, l1);
            l += l0 + l1;
            tmem_wait_st();
            if (changed) fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();   // one arrival a warp: 32 atomics on one word hold up the shared-memory pipe
            if (lane == 0) mbar_arrive(smem_u32(&c.pfull[x]));
            ++sc;
        }
        if (!ok || !wait(&c.pvdone[x], (uint32_t)((sc - 1) & 1))) break;
        tc_fence_after_sync();
        // ---- the piece's rows: finished, or a partial row
        const int piece = x == 0 ? p.local : both;   // (half 0 takes every piece)
        const unsigned long long poison = *reinterpret_cast<volatile unsigned long long *>(&c.poison[x][piece & 1]);
        if ((int)(poison >> 32) == piece + 1 && vis > (int)(EX_LAST - (uint32_t)poison)) l = __int_as_float(0x7fc00000);
        const bool whole = p.t0 == 0 && p.t1 >= h.ntiles;
        const int slot_row = p.slot() * EX_ROWS + h.row0 % EX_ROWS + m;
        if (!whole && mine) a.ml[slot_row] = make_float2(mrun, l);
        const float inv = 1.f / l;
        uint16_t *orow = a.out + ((long long)(p.w.q0 + tok) * a.H + p.r / p.w.per_head) * EV;
        const int part_q = h.row0 % EX_ROWS / 32 + quarter;
#pragma unroll 1
        for (int q = 0; q < EV / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(trow + ocol + 32 * q, o);
            tmem_wait_ld();
            if (mine && whole) {
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = (uint32_t)out_bits<KV>(__uint_as_float(o[k + 2 * i]) * inv) |
                               ((uint32_t)out_bits<KV>(__uint_as_float(o[k + 2 * i + 1]) * inv) << 16);
                    *reinterpret_cast<uint4 *>(orow + 32 * q + k) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else if (mine) {
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                    *reinterpret_cast<uint4 *>(a.o + partial_at(p.slot(), part_q, q, k / 4, lane)) =
                        make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            }
            __syncwarp();   // the next load is the whole warp's
        }
        tc_fence_before_sync();
        cnt += blocks;
    }
}

template <int KV>
__global__ void __launch_bounds__(EX_THREADS, 1)
    expanded_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmr, const __grid_constant__ CUtensorMap tmv,
                    const ExpandedArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    ExCtrl &c = *reinterpret_cast<ExCtrl *>(smem + EX_OFF_CTRL);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < EX_RING; ++s) {
            mbar_init(smem_u32(&c.full[s]), 1);
            mbar_init(smem_u32(&c.empty[s]), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&c.qfull[x]), 1);
            mbar_init(smem_u32(&c.qempty[x]), 1);
            mbar_init(smem_u32(&c.sfull[x]), 1);
            mbar_init(smem_u32(&c.pfull[x]), EX_HALF / 32);
            mbar_init(smem_u32(&c.pvdone[x]), 1);
        }
        mbar_init(smem_u32(&c.done), 1);
        c.abort = 0;
        fence_mbar_init();
        tma_prefetch_map(&tmq);
        tma_prefetch_map(&tmk);
        tma_prefetch_map(&tmr);
        tma_prefetch_map(&tmv);
    } else if (threadIdx.x >= 32 && threadIdx.x < 36) {
        c.poison[(threadIdx.x >> 1) & 1][threadIdx.x & 1] = 0;
    }
    grid_wait();
    if (warp == 2) {   // (not before: an earlier kernel may still need its own)
        tmem_alloc(smem_u32(&c.tmem), EX_TMEM);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    make_plan(a, &c.plan, c.warp_sums);
    tc_fence_after_sync();
    const Plan plan = c.plan;
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&c.tmem);
    grid_release();   // the merge's CTAs may come as this kernel's leave (they wait for all of them)
    fill_idle_rows<EV / 8>(a, plan, a.out, (long long)a.num_query_tokens * a.H,
                           KV == PA_KV_F16 ? 0x7e007e00u : 0x7fc07fc0u);
    if (plan.u0 < plan.u1) {   // the whole CTA has work, or none of it
        Walk<ExpandedArgs> p(a, plan);
        if (warp >= 4) {
            regs_increase<EX_REGS_HIGH>();
            ex_softmax<KV>(smem, c, a, p, tmem, (warp - 4) >> 2);
        } else {
            regs_decrease<EX_REGS_LOW>();
            if (warp == 0) {
                if (elect_one()) ex_load(smem, c, a, p, &tmq, &tmk, &tmr, &tmv);
            } else if (warp == 2) {
                if (elect_one()) ex_mma<KV>(smem, c, a, p, tmem);
            }
            __syncwarp();
        }
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
    }
    if (warp == 2) tmem_dealloc(tmem, EX_TMEM);
    if (threadIdx.x == 0) a.status[blockIdx.x] = c.abort;
}

// Rows of the cut row tiles from their pieces' partial rows: blockIdx.x is the
// CTA whose range begins in the row tile; a warp takes 32 rows and eight of their
// dims, in the order in which the softmax left them.  When a CTA of the first
// kernel gave up, every row becomes NaN.
constexpr int EM_WARPS = 8, EM_UNITS = EV / 8;   // warps of 32 rows
static_assert(32 * EM_WARPS >= AXIS_MAX_CTAS, "a thread per CTA's status");

template <int KV>
__global__ void __launch_bounds__(32 * EM_WARPS) expanded_merge_kernel(const ExpandedArgs a, int ctas) {
    grid_release();
    grid_wait();
    const int cta = blockIdx.x, lane = threadIdx.x & 31;
    const int gave_up = threadIdx.x < ctas ? a.status[threadIdx.x] : 0;
    const Cut cut = a.cuts[cta];
    const int unit = blockIdx.y * EM_WARPS + (threadIdx.x >> 5), q = unit / EM_UNITS;
    if (32 * (blockIdx.y * EM_WARPS / EM_UNITS) >= cut.rows && (cta || blockIdx.y)) return;   // the whole block
    const bool failed = __syncthreads_or(gave_up);
    if (cta == 0 && blockIdx.y == 0) {
        if (threadIdx.x == 0) a.hdr->error = failed ? PA_ERR_TIMEOUT : PA_OK;
        if (failed) fill_rows(a.out, 0, (long long)a.num_query_tokens * a.H * (EV / 8), KV == PA_KV_F16 ? 0x7e007e00u : 0x7fc07fc0u);
    }
    const int m = 32 * q + lane, k4 = unit % EM_UNITS >> 2, j = 2 * (unit & 3);
    if (failed || m >= cut.rows) return;
    const int pieces = m < EX_HALF ? cut.pieces1 : cut.pieces;
    if (pieces == 1) return;   // this half was finished by one CTA
    float acc[8], l;
    join_pieces(
        pieces, [&](int i) { return a.ml[piece_slot(cut, cta, i) * EX_ROWS + m]; },
        [&](int i) { return a.o[partial_at(piece_slot(cut, cta, i), q, k4, j, lane)]; },
        [&](int i) { return a.o[partial_at(piece_slot(cut, cta, i), q, k4, j + 1, lane)]; }, acc, l);
    const float inv = 1.f / l;
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = (uint32_t)out_bits<KV>(acc[2 * i] * inv) | ((uint32_t)out_bits<KV>(acc[2 * i + 1] * inv) << 16);
    *reinterpret_cast<uint4 *>(a.out + (cut.row0 + (long long)m * a.H) * EV + 32 * k4 + 4 * j) =
        make_uint4(v[0], v[1], v[2], v[3]);
}

// ------------------------------------------------------------------ launch

struct ExLayout {
    size_t status, cuts, ml, o, total;
};

ExLayout ex_layout() {
    ExLayout l;
    size_t at = 256;   // header
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at = (at + bytes + 255) / 256 * 256;
        return p;
    };
    l.status = take(sizeof(int) * AXIS_MAX_CTAS);
    l.cuts = take(sizeof(Cut) * AXIS_MAX_CTAS);
    l.ml = take(sizeof(float2) * 2 * AXIS_MAX_CTAS * EX_ROWS);
    l.o = take(sizeof(float) * 2 * AXIS_MAX_CTAS * EX_ROWS * EV);
    l.total = at;
    return l;
}

// [rows][heads][width] 16-bit elements with the given strides, boxes of 64
// elements of one head over 128 rows; heads = 0: [rows][width].
bool heads_map(CUtensorMap *map, const void *base, int width, int heads, long long rows, long long head_stride,
               long long row_stride, int dtype) {
    auto enc = tma_encoder();
    if (!enc) return false;
    const int rank = heads ? 3 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)(heads ? heads : rows), (cuuint64_t)rows};
    cuuint64_t strides[2] = {2 * (cuuint64_t)(heads ? head_stride : row_stride), 2 * (cuuint64_t)row_stride};
    cuuint32_t box[3] = {64, heads ? 1u : (cuuint32_t)EX_TOK, EX_TOK};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, dtype == PA_KV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
               (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared-memory limits are set per device, on its first call; the kernel runs
// only if it was built with the registers that its split assumes (with another
// count the softmax warpgroups' increase could wait forever).
template <int KV>
int ex_setup() {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64 && done[dev]) return PA_OK;
    cudaFuncAttributes fa;
    if (cudaFuncSetAttribute(expanded_kernel<KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, EX_SMEM) !=
            cudaSuccess ||
        cudaFuncGetAttributes(&fa, expanded_kernel<KV>) != cudaSuccess)
        return PA_ERR_CUDA;
    if (fa.numRegs != EX_REGS_LAUNCH) return PA_ERR_UNSUPPORTED;
    if (dev < 64) done[dev] = true;
    return PA_OK;
}

template <int KV>
int launch_expanded(const ExpandedArgs &a, const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmr,
                    const CUtensorMap &tmv, cudaStream_t st) {
    if (const int e = ex_setup<KV>()) return e;
    const int ctas = std::min(num_sms(), AXIS_MAX_CTAS);
    if (const int e = launch_early(expanded_kernel<KV>, dim3((unsigned)ctas), EX_THREADS, EX_SMEM, st, tmq, tmk, tmr, tmv, a))
        return e;
    const dim3 grid((unsigned)ctas, (unsigned)((std::min(EX_ROWS, a.num_query_tokens) + 31) / 32 * EM_UNITS / EM_WARPS));
    return launch_early(expanded_merge_kernel<KV>, grid, 32 * EM_WARPS, 0, st, a, ctas);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_latent_attention_expanded_workspace_size(int num_seqs, int num_query_tokens, int num_heads) {
    if (num_seqs < 0 || num_query_tokens < 0 || num_heads <= 0) return 0;
    return ex_layout().total;
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
    if ((long long)num_query_tokens * num_heads >= (1LL << 31)) return PA_ERR_UNSUPPORTED;
    if (num_query_tokens == 0) return PA_OK;
    if (!out || !query || !query_start || !kv_start || !aligned16(out) || !aligned16(query) ||
        (num_kv_tokens > 0 && (!k_nope || !k_rope || !value)) || !aligned16(k_nope) || !aligned16(k_rope) ||
        !aligned16(value))
        return PA_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < pa_latent_attention_expanded_workspace_size(num_seqs, num_query_tokens, num_heads))
        return PA_ERR_WORKSPACE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug_validate()) {
        if (const int e = validate_starts(query_start, num_seqs, num_query_tokens, true, st)) return e;
        if (const int e = validate_starts(kv_start, num_seqs, num_kv_tokens, true, st)) return e;
    }
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const ExLayout lay = ex_layout();
    ExpandedArgs a{};
    a.out = static_cast<uint16_t *>(out);
    a.query_start = query_start;
    a.kv_start = kv_start;
    a.hdr = reinterpret_cast<WsHeader *>(ws);
    a.num_seqs = num_seqs;
    a.num_query_tokens = num_query_tokens;
    a.num_kv_tokens = num_kv_tokens;
    a.H = num_heads;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.wait_limit = pipeline_wait_limit();
    a.status = reinterpret_cast<int *>(ws + lay.status);
    a.cuts = reinterpret_cast<Cut *>(ws + lay.cuts);
    a.ml = reinterpret_cast<float2 *>(ws + lay.ml);
    a.o = reinterpret_cast<float4 *>(ws + lay.o);
    // without keys no row tile has work and no copy is made: any base will do
    const bool none = num_kv_tokens == 0;
    const long long nk = none ? 1 : num_kv_tokens;
    CUtensorMap tmq, tmk, tmr, tmv;
    if (!heads_map(&tmq, query, EQ, num_heads, num_query_tokens, EQ, (long long)EQ * num_heads, dtype) ||
        !heads_map(&tmk, none ? query : k_nope, EN, num_heads, nk, k_head_stride, k_token_stride, dtype) ||
        !heads_map(&tmr, none ? query : k_rope, ER, 0, nk, 0, rope_stride, dtype) ||
        !heads_map(&tmv, none ? query : value, EV, num_heads, nk, v_head_stride, v_token_stride, dtype))
        return PA_ERR_CUDA;
    return dtype == PA_KV_F16 ? launch_expanded<PA_KV_F16>(a, tmq, tmk, tmr, tmv, st)
                              : launch_expanded<PA_KV_BF16>(a, tmq, tmk, tmr, tmv, st);
}
