// Attention over the latent cache in the absorbed form: with the map from a
// latent to a head's key multiplied into the query, all heads of a token attend
// to the same rows c_t of 576 elements,
//   s_t = scale <q, c_t>,  out = sum_t softmax(s)_t c_t[0 .. 511],
// the running maximum m and sum l of 2^(s_t scale log2 e - m) carried in fp32 (m
// follows the maximum only when that grows by more than 2^8, which keeps the
// probabilities, rounded to the 16-bit type for the second product, below 2^8),
// and pieces of a context joined by M = max m, sum of 2^(m - M) (l, o).
//
// Why the probabilities are rounded: the tensor cores take both operands of P C in
// one type, and C lies in shared memory in the cache's.  The sum l takes them
// unrounded.  Half a step of each probability, at random, comes to about what
// rounding the output does: against 64 bits the whole is off by 0.0019 to 0.0021
// normwise in bf16 and 0.00026 in fp16, where 32-bit arithmetic rounded once at the
// end is off by 0.0016 to 0.0017 and 0.00021.
//
// A row tile is 64 query rows (new token x head) of a sequence.  Each KV tile of 64
// tokens is read once into shared memory and serves both products: S = Q C^T
// (M 64, N 64, K 576) and O += P C (M 64, N 2 x 256, K 64).  Why 64 rows: O of 512
// dims in fp32 is 512 columns at M = 128, all of tensor memory; at M = 64 an
// accumulator uses 16 of each quarter's 32 lanes, so dims 0 .. 255 and 256 .. 511
// share 256 columns and S has room.  One CTA per SM; warps: 0 loads, 1 and 2 issue
// S of even and odd KV tiles, 3 issues P C, 4-7 run the softmax (two threads a row),
// 8-15 turn E4M3 rows into bf16.  Shared memory: the query rows (72 KB), two KV
// stages (72 KB each; 54 KB of 48 tokens over a quantised cache, beside a staging
// ring of 31 KB), P (8 KB).
//
// What bounds it (one GB300, 1.9 GHz): 16 heads, 100 x 8192 bf16 tokens: 157 us,
// the kernel 153 at 6.2 TB/s of HBM reads, tensor pipe 62 % busy.  128 heads are
// two row tiles a token, 96 contexts of 64 .. 32768 fp16 tokens: 195 us, a latency
// chain: a stage goes through load, S (36 products of 38 clocks), softmax and P C
// (8 of 155) in 5500 clocks, and two stages are all that fits beside the queries;
// halving both products takes 158.  Products of M 64 run at half the tensor
// cores' rate.  E4M3, 16 heads x 4 new tokens, 100 contexts of 1024 .. 8192: 111 us,
// 3600 clocks a tile, in which no unit is busy half of the time (ALU 44 %, HBM 30 %).
// Halving both products leaves it as it is, and without conversion and stores 96
// us remain.  By elimination most of it is the way of the rows to the converting
// warps (ids, copy, hand-over and hand-back of a slot) through a staging ring that
// holds just one tile, with rows fetched into L2 only as their batch begins; its
// steps are not measured one by one.  The E4M3 cache saves memory here, not time:
// the same contexts in bf16 take 88 us; one new token 103 and 78, at 128 heads 197
// and 140, where each of a token's row tiles converts the rows again.
#include <algorithm>
#include <cmath>

#include "decode_common.cuh"
#include "latent.h"
#include "umma.cuh"
#include "work_axis.cuh"

namespace pa {
namespace {

constexpr int LT_ROWS = 64;   // query rows of a row tile (new token x head, token-major)

// TOK: tokens of a KV tile.
template <int TOK>
struct LatentArgs {
    uint16_t *out;
    const uint16_t *query;
    const uint8_t *cache;
    const int32_t *block_tables, *context_lens, *query_start;
    WsHeader *hdr;
    int num_seqs, num_query_tokens, H, bs_log2, mbps, max_context_len;
    long long num_blocks;
    float scale_log2;
    long long wait_limit;
    // workspace
    int *status;            // [AXIS_MAX_CTAS] nonzero: the CTA gave up waiting
    Cut *cuts;              // [AXIS_MAX_CTAS]
    float2 *ml;             // [2 AXIS_MAX_CTAS][LT_ROWS] maximum (log2 units) and sum of a partial row
    float4 *o;              // [2 AXIS_MAX_CTAS][LT_ROWS * LC / 4] its unnormalised output (see partial_at)

    // ---- the work axis
    static constexpr int COST = 2;   // 128 heads: 214 us with 1, 209 with 2, 212 with 3, 217 with 6
    struct Seq {
        int L, T, q0;   // context, new tokens, first query token
        int tiles;      // KV tiles of the context (0: nothing to compute)
        int rts;        // row tiles
        bool valid;     // rows are computed (or zero, for an empty context)
    };
    __device__ __forceinline__ Seq seq_work(int i) const {
        Seq w;
        w.L = context_lens[i];
        w.q0 = query_start ? query_start[i] : i;
        w.T = query_start ? query_start[i + 1] - w.q0 : 1;
        w.valid = w.L >= 0 && w.L <= max_context_len && (long long)w.L <= (long long)mbps << bs_log2 &&
                  !(query_start && w.T > w.L);
        w.tiles = w.valid && w.T > 0 ? w.L / TOK + (w.L % TOK != 0) : 0;
        w.rts = w.tiles ? (int)(((long long)w.T * H + LT_ROWS - 1) / LT_ROWS) : 0;
        return w;
    }
    // Every row tile counts the whole context's KV tiles (a chunk's earlier
    // rows see fewer, which matters only for long chunks; those belong to the
    // expanded form).
    __device__ __forceinline__ long long start(const Seq &w, int j, int) const { return (long long)j * (w.tiles + COST); }
    __device__ __forceinline__ int row_tile_at(const Seq &w, long long u, int) const {
        return (int)quick_div(u, w.tiles + COST);
    }
    __device__ __forceinline__ bool in_teams(const Seq &w) const { return w.rts % 2 == 0; }
    // KV tiles that row tile r sees: up to its last row's own position.
    __device__ __forceinline__ int row_tiles(const Seq &w, int r) const {
        const uint32_t last = min((uint32_t)w.T * H, ((uint32_t)r + 1) * LT_ROWS) - 1;
        return (w.L - w.T + (int)(last / (uint32_t)H)) / TOK + 1;
    }
    __device__ __forceinline__ bool seq_ok(int i) const {
        return !query_start || query_start[i] <= query_start[i + 1];
    }
    __device__ __forceinline__ bool ends_ok() const {
        return !query_start || (*query_start == 0 && query_start[num_seqs] == num_query_tokens);
    }
    // A token's entry in its block table, and its offset in the block (a block
    // size is a power of two).
    __device__ __forceinline__ int entry_of(int tok) const { return tok >> bs_log2; }
    __device__ __forceinline__ int offset_of(int tok) const { return tok & ((1 << bs_log2) - 1); }
    // rows of row tile r, and its first row in the query
    __device__ __forceinline__ int cut_rows(const Seq &w, int r) const { return rows(w, r); }
    __device__ __forceinline__ int first_tiles(const Seq &w, int r) const { return row_tiles(w, r); }
    __device__ __forceinline__ int rows(const Seq &w, int r) const {
        return (int)min((long long)LT_ROWS, (long long)w.T * H - (long long)r * LT_ROWS);
    }
    __device__ __forceinline__ long long first_row(const Seq &w, int r) const {
        return (long long)w.q0 * H + (long long)r * LT_ROWS;
    }
};

template <int KV>
__device__ __forceinline__ uint16_t to_bits(float x) {
    if constexpr (KV == PA_KV_F16)
        return __half_as_ushort(__float2half_rn(x));
    else
        return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// Where a softmax thread keeps four dims (32 k + 4 j ..) of its row's half, in
// float4: a store of the warp's lanes (16 rows x 2 halves) is one run of 512 bytes.
__device__ __forceinline__ long long partial_at(int slot, int quarter, int k, int j, int lane) {
    return (((long long)slot * 4 + quarter) * 8 + k) * 8 * 32 + j * 32 + lane;
}

// ------------------------------------------------------------------ the kernel

constexpr int LT_GROUP = 9 * 1024;            // 8 rows of 576 elements: nine 128-byte-swizzled blocks of 64 columns
constexpr int LT_Q = LT_ROWS / 8 * LT_GROUP;
constexpr int LT_P = LT_ROWS * 128;
constexpr int LT_CTRL = 1024;
constexpr int LT_TMEM = 512;                  // columns: O (256), S0, S1 (64 each)
constexpr int LT_S = 256;
constexpr uint32_t LT_HI = 16u << 16;         // lanes 16 .. 31 of each quarter: output dims 256 .. 511
// Pieces whose flags are kept.  The producer has a piece's queries copied only after
// all S of the piece before, and an S waits until the softmax has read the one two
// tiles earlier: it is at most three pieces ahead of the softmax.
constexpr int LT_BAD_SLOTS = 16;
constexpr uint32_t LT_LAST = 0x7fffffffu;
constexpr int L8_WARPS = 8;                   // converting warps
constexpr int L8_STEP = 16;                   // tokens of a staging slot of quantised rows: two groups of eight
constexpr int L8_GROUP = 8 * LROW8;           // bytes of a group, consecutive in its block
constexpr int L8_SLOTS = 3;

// What differs between a 16-bit and an E4M3 cache.
template <int KV>
struct Lt {
    static constexpr bool F8 = KV == PA_KV_FP8_E4M3;
    static constexpr int TOK = F8 ? 48 : 64;   // tokens of a KV tile
    // a stage is freed in parts, as the products with the values pass them
    static constexpr int PARTS = F8 ? 3 : 2, PART_TOK = TOK / PARTS;
    static constexpr int THREADS = F8 ? 256 + 32 * L8_WARPS : 256;
    static constexpr int STAGE = TOK / 8 * LT_GROUP;
    static constexpr int OFF_KV = LT_Q;
    static constexpr int OFF_P = OFF_KV + 2 * STAGE;
    static constexpr int OFF_8 = OFF_P + LT_P;
    static constexpr int OFF_CTRL = OFF_8 + (F8 ? L8_SLOTS * 2 * L8_GROUP : 0);
    static constexpr int SMEM = OFF_CTRL + LT_CTRL + 1024;   // + alignment slack
    static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
    using Args = LatentArgs<TOK>;
};

struct LtCtrl {
    uint64_t kvfull[2], kvempty[2][3], sfull[2], sfree[2], pfull, pvdone, qfull, qempty, done;
    uint64_t full8[L8_SLOTS], empty8[L8_SLOTS];
    uint32_t tmem;
    int abort;
    int bad[LT_BAD_SLOTS];   // 1 + the number of a piece that met a block id out of range
    // by a piece's number: 1 + that number in the high word, and in the low one
    // how far below the largest position its first non-finite new token is
    unsigned long long poison[LT_BAD_SLOTS];
    Plan plan;
    long long warp_sums[16];
};
static_assert(sizeof(LtCtrl) <= LT_CTRL, "control block");

// Tensor maps: rows of a 16-bit cache (a quantised one is copied as it lies),
// rows of the query.
struct LtMaps {
    CUtensorMap kv, q;
};

// A role's bounded wait, the outcome shared by the warp (or one lane's own).  A
// barrier that is ready costs one test; the flag of a role that gave up is looked
// at only before waiting.
struct Waiter {
    volatile int *abort_flag;
    long long limit;
    bool ok = true;
    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
        return mbar_try_wait(bar, parity) || (!*abort_flag && mbar_wait_bounded(bar, parity, limit));
    }
    __device__ __forceinline__ bool warp(const uint64_t &bar, int parity) {
        ok = __all_sync(0xffffffffu, ok && wait(smem_u32(&bar), (uint32_t)(parity & 1)));
        if (!ok) *abort_flag = 1;
        return ok;
    }
    __device__ __forceinline__ bool lane(const uint64_t &bar, int parity) {
        ok = ok && wait(smem_u32(&bar), (uint32_t)(parity & 1));
        if (!ok) *abort_flag = 1;
        return ok;
    }
};

// One arrival for a warp, after all its lanes' accesses (an arrival per thread
// is 32 atomics on one word, and they hold up the shared-memory pipe).
__device__ __forceinline__ void arrive_warp(uint64_t &bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bar));
}

// The producer warp of a 16-bit cache: lane j copies tokens 8 j .. 8 j + 7 of a
// tile, lanes 8 .. 15 the query rows.  The next tile's rows are fetched into L2
// while both stages are full: 100 x 8192 tokens 167 -> 164 us, 128 heads 237 -> 229
// us; two, three or four tiles ahead gain less and less.
template <int KV>
__device__ void lt_load(uint8_t *smem, LtCtrl &c, const typename Lt<KV>::Args &a, Walk<typename Lt<KV>::Args> &p,
                        const LtMaps &maps) {
    using L = Lt<KV>;
    const int lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    const uint64_t first = policy_evict_first(), keep = policy_evict_normal();
    Waiter w{&c.abort, a.wait_limit};
    int cnt = 0, pieces = 0;
    while (w.ok && p.next()) {
        const int32_t *row = a.block_tables + (long long)p.seq * a.mbps;
        auto id_of = [&](int tok) { return lane < L::TOK / 8 && tok < p.w.L ? row[a.entry_of(tok)] : 0; };
        const int32_t first_id = id_of(p.t0 * L::TOK + 8 * lane);   // on its way with the queries
        if (!w.warp(c.qempty, pieces + 1)) break;
        if (lane == 0) mbar_arrive_expect_tx(smem_u32(&c.qfull), LT_Q);
        __syncwarp();
        if (lane >= 8 && lane < 16)
            tma_load_3d(base + (lane - 8) * LT_GROUP, &maps.q, 0, (int)a.first_row(p.w, p.r) + 8 * (lane - 8), 0,
                        smem_u32(&c.qfull), keep);
        ++pieces;
        for (int t = p.t0; t < p.t1; ++t, ++cnt) {
            const int tok = t * L::TOK + 8 * lane, st = cnt & 1;
            const bool mine = lane < L::TOK / 8 && tok < p.w.L;
            const int32_t blk = t == p.t0 ? first_id : id_of(tok);
            // lanes 8 .. 15: a group of the next tile, to be fetched into L2
            const int ntok = tok + L::TOK - 64;
            const bool ahead = lane >= 8 && lane < 16 && t + 1 < p.t1 && ntok < p.w.L;
            const int32_t nblk = ahead ? row[a.entry_of(ntok)] : -1;
            const bool bad = __any_sync(0xffffffffu, mine && (blk < 0 || blk >= a.num_blocks));
            // (a group past the context is a box outside the cache, which reads as zeros)
            const unsigned boxes = __ballot_sync(0xffffffffu, lane < L::TOK / 8 && !bad);
            const int from = mine ? (blk << a.bs_log2) + a.offset_of(tok) : -8;
            if (bad && lane == 0) *reinterpret_cast<volatile int *>(&c.bad[p.local % LT_BAD_SLOTS]) = p.local + 1;
            int sent = 0;   // parts
#pragma unroll
            for (int part = 0; part < L::PARTS; ++part) {
                constexpr int N = L::PART_TOK / 8;   // groups of a part
                if (!w.warp(c.kvempty[st][part], (cnt >> 1) + 1)) break;
                ++sent;
                if (lane == 0)
                    mbar_arrive_expect_tx(smem_u32(&c.kvfull[st]),
                                          (uint32_t)(__popc(boxes >> (part * N) & ((1u << N) - 1)) * LT_GROUP));
                __syncwarp();
                if (lane / N == part && (boxes >> lane & 1u))
                    tma_load_3d(base + L::OFF_KV + st * L::STAGE + lane * LT_GROUP, &maps.kv, 0, from, 0,
                                smem_u32(&c.kvfull[st]), first);
            }
            if (!w.ok) {
                // parts on their way count as a use of the stage below: the others arrive
                // without copies, so that its phase ends when these have landed
                if (sent) {
                    if (lane == 0)
                        for (int part = sent; part < L::PARTS; ++part) mbar_arrive(smem_u32(&c.kvfull[st]));
                    ++cnt;
                }
                break;
            }
            if (nblk >= 0 && nblk < a.num_blocks)
                tma_prefetch_3d(&maps.kv, 0, (nblk << a.bs_log2) + a.offset_of(ntok), 0);
            __syncwarp();
        }
    }
    // the last copies into every buffer have landed before the CTA leaves
    for (int s = 0; s < 2; ++s)
        if (cnt > s) mbar_wait_bounded(smem_u32(&c.kvfull[s]), (uint32_t)(((cnt - 1 - s) / 2) & 1), WAIT_LIMIT);
    if (pieces) mbar_wait_bounded(smem_u32(&c.qfull), (uint32_t)((pieces - 1) & 1), WAIT_LIMIT);
}

// The producer warp of a quantised cache: steps of 16 tokens (two groups of
// eight rows, 5248 bytes each, consecutive in their block) into the staging ring.
// The ring holds only a tile, so the time from a freed slot to its next rows
// counts: block ids are loaded 32 groups at a time, a batch early, and a batch's
// rows are fetched into L2 when its ids are first used.  (Ids loaded per step
// kept the warp waiting for 1500 clocks a step, whether by lane or queued in a
// thread's registers, since moving a register waits for its load: 123 to 140 us
// for four new tokens of 100 sequences.)
template <int KV>
__device__ void lt_load8(uint8_t *smem, LtCtrl &c, const typename Lt<KV>::Args &a, Walk<typename Lt<KV>::Args> &p,
                         const LtMaps &maps) {
    using L = Lt<KV>;
    const int lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    const uint64_t keep = policy_evict_normal();
    Waiter w{&c.abort, a.wait_limit};
    int steps = 0, pieces = 0;
    while (w.ok && p.next()) {
        const int32_t *row = a.block_tables + (long long)p.seq * a.mbps;
        const int g0 = p.t0 * (L::TOK / 8), groups = (p.t1 - p.t0) * (L::TOK / 8);   // of the piece
        const int with = min(groups, p.w.L / 8 + (p.w.L % 8 != 0) - g0);               // those with tokens
        auto ids = [&](int g) { return g + lane < with ? row[a.entry_of(8 * (g0 + g + lane))] : 0; };
        // lane j's group of a batch: its rows in the cache, null if its id is out of range or it has no tokens
        auto rows_of = [&](int32_t id, int g) {
            const bool in = g < with && id >= 0 && id < a.num_blocks;
            return in ? a.cache + (((long long)id << a.bs_log2) + a.offset_of(8 * (g0 + g))) * LROW8 : nullptr;
        };
        int32_t next_ids = ids(0);
        if (!w.warp(c.qempty, pieces + 1)) break;
        if (lane == 0) mbar_arrive_expect_tx(smem_u32(&c.qfull), LT_Q);
        __syncwarp();
        if (lane < 8)
            tma_load_3d(base + lane * LT_GROUP, &maps.q, 0, (int)a.first_row(p.w, p.r) + 8 * lane, 0,
                        smem_u32(&c.qfull), keep);
        ++pieces;
        const uint8_t *mine = nullptr;
        for (int g = 0; g < groups; g += 2, ++steps) {
            if ((g & 31) == 0) {   // the next batch
                mine = rows_of(next_ids, g + lane);
                if (__any_sync(0xffffffffu, !mine && g + lane < with) && lane == 0)
                    *reinterpret_cast<volatile int *>(&c.bad[p.local % LT_BAD_SLOTS]) = p.local + 1;
                next_ids = ids(g + 32);
                if (mine) bulk_prefetch(mine, L8_GROUP);
            }
            const int s = steps % L8_SLOTS, j = lane - (g & 31);   // lanes of the step's groups: j = 0, 1
            if (!w.warp(c.empty8[s], steps / L8_SLOTS + 1)) break;
            const unsigned there = __ballot_sync(0xffffffffu, (j == 0 || j == 1) && mine);
            if (lane == 0) mbar_arrive_expect_tx(smem_u32(&c.full8[s]), (uint32_t)(__popc(there) * L8_GROUP));
            __syncwarp();
            if (there >> lane & 1u)
                bulk_load(base + L::OFF_8 + (2 * s + j) * L8_GROUP, mine, L8_GROUP, smem_u32(&c.full8[s]));
            __syncwarp();
        }
    }
    // the last copies into every buffer have landed before the CTA leaves
    for (int s = 0; s < L8_SLOTS; ++s)
        if (steps > s)
            mbar_wait_bounded(smem_u32(&c.full8[s]), (uint32_t)(((steps - 1 - s) / L8_SLOTS) & 1), WAIT_LIMIT);
    if (pieces) mbar_wait_bounded(smem_u32(&c.qfull), (uint32_t)((pieces - 1) & 1), WAIT_LIMIT);
}

// A converting warp of a quantised cache: row cw of both groups of every step,
// codes times their group's scale as bf16 and the rotary elements, in the layout
// a 16-bit copy would have written.  Lane l turns the codes 16 l .. 16 l + 15 into
// two 16-byte chunks; lanes of odd 64-element blocks store their second chunk
// first, so that eight lanes of a store cover all banks.  Rows past the context
// become zeros (their probabilities are 0).  Other shapes were slower (a step of
// four new tokens of 100 sequences, 123 us here): sixteen warps of a row each, 141;
// twelve of four rows of one step, 152; rows loaded from global memory into
// registers instead of staged, 130 (the loads in flight held up the stores behind
// them); and, against 110 later, two sets of eight warps that take turns, 115, the
// next step's loads before a step's stores, 114.
template <int KV>
__device__ void lt_convert(uint8_t *smem, LtCtrl &c, const typename Lt<KV>::Args &a, Walk<typename Lt<KV>::Args> &p) {
    using L = Lt<KV>;
    const int lane = threadIdx.x & 31, cw = (threadIdx.x >> 5) - 8;
    const bool odd = (lane >> 2) & 1;
    // chunks 2 (l % 4) and 2 (l % 4) + 1 of block l / 4, in the order of their stores; rotary elements 2 l, 2 l + 1
    const int at0 = (lane >> 2) * 1024 + cw * 128 + (((2 * (lane & 3) + odd) ^ cw) << 4);
    const int at1 = (lane >> 2) * 1024 + cw * 128 + (((2 * (lane & 3) + 1 - odd) ^ cw) << 4);
    const int atr = 8192 + cw * 128 + (((lane >> 2) ^ cw) << 4) + (lane & 3) * 4;
    Waiter w{&c.abort, a.wait_limit};
    int cnt = 0, steps = 0;
    while (w.ok && p.next()) {
        for (int t = p.t0; t < p.t1; ++t, ++cnt) {
            const int st = cnt & 1, left = p.w.L - t * L::TOK;   // tokens from the tile's first on
            uint8_t *stage = smem + L::OFF_KV + st * L::STAGE;
            for (int k = 0; k < L::TOK / L8_STEP; ++k, ++steps) {
                const int s = steps % L8_SLOTS;
                if (!w.warp(c.full8[s], steps / L8_SLOTS)) break;
                const uint8_t *src = smem + L::OFF_8 + 2 * s * L8_GROUP + cw * LROW8;
                uint4 v[2];
                float sc[2];
                uint32_t rope[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    v[i] = *reinterpret_cast<const uint4 *>(src + i * L8_GROUP + 16 * lane);
                    sc[i] = *reinterpret_cast<const float *>(src + i * L8_GROUP + L8_SCALE + 4 * (lane >> 3));
                    rope[i] = *reinterpret_cast<const uint32_t *>(src + i * L8_GROUP + L8_ROPE + 4 * lane);
                }
                uint2 x[2][4];
                uint32_t special = left < (k + 1) * L8_STEP;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t up = latent_scale_up(sc[i]);
                    x[i][0] = latent_codes_fast(v[i].x, up), x[i][1] = latent_codes_fast(v[i].y, up);
                    x[i][2] = latent_codes_fast(v[i].z, up), x[i][3] = latent_codes_fast(v[i].w, up);
                    special |= latent_codes_nan(make_uint2(v[i].x, v[i].y)) | latent_codes_nan(make_uint2(v[i].z, v[i].w)) |
                               (uint32_t)latent_scale_special(sc[i]);
                }
                if (__any_sync(0xffffffffu, special)) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        x[i][0] = latent_codes_to_bf16(v[i].x, sc[i]), x[i][1] = latent_codes_to_bf16(v[i].y, sc[i]);
                        x[i][2] = latent_codes_to_bf16(v[i].z, sc[i]), x[i][3] = latent_codes_to_bf16(v[i].w, sc[i]);
                        if (k * L8_STEP + 8 * i + cw >= left)
                            x[i][0] = x[i][1] = x[i][2] = x[i][3] = make_uint2(0, 0);
                    }
                }
                arrive_warp(c.empty8[s]);   // after every lane's loads (the vote orders no memory)
                if (!w.warp(c.kvempty[st][k], (cnt >> 1) + 1)) break;
                uint8_t *dst = stage + 2 * k * LT_GROUP;
#pragma unroll
                for (int i = 0; i < 2; ++i, dst += LT_GROUP) {
                    const int f = odd ? 2 : 0;
                    const uint2 a0 = f ? x[i][2] : x[i][0], b0 = f ? x[i][3] : x[i][1];
                    const uint2 a1 = f ? x[i][0] : x[i][2], b1 = f ? x[i][1] : x[i][3];
                    *reinterpret_cast<uint4 *>(dst + at0) = make_uint4(a0.x, a0.y, b0.x, b0.y);
                    *reinterpret_cast<uint4 *>(dst + at1) = make_uint4(a1.x, a1.y, b1.x, b1.y);
                    *reinterpret_cast<uint32_t *>(dst + atr) = rope[i];
                }
            }
            if (!w.ok) break;
            fence_proxy_async_smem();   // the rows, for the tensor cores
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c.kvfull[st]));
        }
    }
}

// MMA issuers, one lane each: warps 1 and 2 the S products of even and odd KV
// tiles, warp 3 the products with the values.
template <int KV>
__device__ void lt_mma(uint8_t *smem, LtCtrl &c, const typename Lt<KV>::Args &a, Walk<typename Lt<KV>::Args> &p,
                       uint32_t tmem, int warp) {
    using L = Lt<KV>;
    constexpr bool BF16 = KV != PA_KV_F16;
    const uint32_t base = smem_u32(smem);
    Waiter w{&c.abort, a.wait_limit};
    int n = 0, pieces = 0;   // KV tiles and pieces so far
    if (warp < 3) {
        const int e = warp - 1;
        constexpr uint32_t ID = idesc_f16(LT_ROWS, L::TOK, BF16, false);
        const uint64_t dq = sw128_desc(base, 16, LT_GROUP);
        const uint64_t dk = sw128_desc(base + L::OFF_KV + e * L::STAGE, 16, LT_GROUP);
        const uint32_t d = tmem + LT_S + 64 * e;
        while (w.ok && p.next()) {
            if (!w.lane(c.qfull, pieces)) break;
            ++pieces;
            for (int t = p.t0; t < p.t1; ++t, ++n) {
                if ((n & 1) != e) continue;
                if (!w.lane(c.sfree[e], (n >> 1) + 1) || !w.lane(c.kvfull[e], n >> 1)) break;
                tc_fence_after_sync();
#pragma unroll
                for (int k = 0; k < LROW / 16; ++k) {
                    const uint64_t off = (uint64_t)(((k >> 2) * 1024 + (k & 3) * 32) >> 4);
                    umma_f16(d, dq + off, dk + off, ID, k > 0 ? 1u : 0u);
                }
                umma_commit(smem_u32(&c.sfull[e]));
            }
            if (w.ok) umma_commit(smem_u32(&c.qempty));   // after this issuer's last product of the piece
        }
    } else {
        constexpr uint32_t ID = idesc_f16(LT_ROWS, LC / 2, BF16, true);
        const uint64_t dp = sw128_desc(base + L::OFF_P, 16, 1024);
        const uint64_t dv0 = sw128_desc(base + L::OFF_KV, 1024, LT_GROUP);
        while (w.ok && p.next()) {
            for (int t = p.t0; t < p.t1; ++t, ++n) {
                const int st = n & 1;
                if (!w.lane(c.kvfull[st], n >> 1) || !w.lane(c.pfull, n)) break;
                tc_fence_after_sync();
                const uint64_t dv = dv0 + (uint64_t)(st * (L::STAGE >> 4));
#pragma unroll
                for (int k = 0; k < L::TOK / 16; ++k) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        umma_f16(tmem + (h ? LT_HI : 0u), dp + (uint64_t)((k * 32) >> 4),
                                 dv + (uint64_t)((k * 2 * LT_GROUP + h * 4096) >> 4), ID, t > p.t0 || k > 0 ? 1u : 0u);
                    if ((k + 1) % (L::PART_TOK / 16) == 0)
                        umma_commit(smem_u32(&c.kvempty[st][k / (L::PART_TOK / 16)]));
                }
                umma_commit(smem_u32(&c.pvdone));
            }
        }
    }
    // every product issued has completed before tensor memory is freed
    umma_commit(smem_u32(&c.done));
    mbar_wait_bounded(smem_u32(&c.done), 0, WAIT_LIMIT);
}

// The softmax warps (4 .. 7): row 16 (warp - 4) + (lane & 15); lanes 0 .. 15
// take the first half of a tile's tokens and output dims 0 .. 255, lanes 16 ..
// 31 the others.
template <int KV>
__device__ void lt_softmax(uint8_t *smem, LtCtrl &c, const typename Lt<KV>::Args &a, Walk<typename Lt<KV>::Args> &p,
                           uint32_t tmem) {
    using L = Lt<KV>;
    constexpr int HT = L::TOK / 2;   // tokens of a tile per thread
    const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3;
    const int half = lane >> 4, m = 16 * q + (lane & 15), tid = threadIdx.x & 127;
    const uint32_t trow = tmem + ((uint32_t)(32 * q) << 16);
    uint8_t *prow = smem + L::OFF_P + m * 128;
    Waiter w{&c.abort, a.wait_limit};
    int n = 0;
    while (w.ok && p.next()) {
        const int rows = a.rows(p.w, p.r);
        const bool live = 16 * q < rows;   // some row of this warp exists
        const bool mine = m < rows;
        const int vis = mine ? p.w.L - p.w.T + (int)(((uint32_t)p.r * LT_ROWS + m) / (uint32_t)a.H) + 1 : p.w.L;
        // what the row tile's first row sees
        const int first_vis = p.w.L - p.w.T + (int)((uint32_t)p.r * LT_ROWS / (uint32_t)a.H) + 1;
        float mrun = -INFINITY, l = 0.f;
        for (int t = p.t0; t < p.t1; ++t, ++n) {
            const int st = n & 1, t0 = t * L::TOK;
            if (!w.warp(c.sfull[st], n >> 1)) break;
            tc_fence_after_sync();
            uint32_t pw[HT / 2];
            float alpha = 1.f;
            bool grew = false;
            if (live) {
                float s[HT];
                tmem_ld_halves(trow + LT_S + 64 * st, s);
                tmem_wait_ld();
                tc_fence_before_sync();
                const int seen = vis - t0 - HT * half;   // of this thread's tokens (the tile may end past the last int)
                if (seen < HT) {
#pragma unroll
                    for (int k = 0; k < HT; ++k) s[k] = k < seen ? s[k] : -INFINITY;
                }
                float mp[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int k = 4; k < HT; ++k) mp[k & 3] = fmaxf(mp[k & 3], s[k]);
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
                for (int k = 0; k < HT / 2; ++k) {
                    const float x = fast_exp2(fmaf(s[2 * k], a.scale_log2, -mu));
                    const float y = fast_exp2(fmaf(s[2 * k + 1], a.scale_log2, -mu));
                    lp[k & 1] += x;
                    lp[2 + (k & 1)] += y;
                    pw[k] = pack_p<KV == PA_KV_F16 ? PA_KV_F16 : PA_KV_BF16>(x, y);
                }
                l += (lp[0] + lp[1]) + (lp[2] + lp[3]);
            }
            arrive_warp(c.sfree[st]);
            // P is free, and O up to date, once the previous product is done
            if (n > 0 && !w.warp(c.pvdone, n - 1)) break;
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
                for (int k = 0; k < HT / 8; ++k)
                    *reinterpret_cast<uint4 *>(prow + (((HT / 8 * half + k) ^ (m & 7)) << 4)) =
                        make_uint4(pw[4 * k], pw[4 * k + 1], pw[4 * k + 2], pw[4 * k + 3]);
            }
            // Rows that some query row does not see, where P is 0 and a product with
            // an infinity or a NaN would not be: those past the context in its last
            // group of eight are zeroed (a quantised tile's and those of later groups
            // already are), and so is what is not finite among the new tokens' (the
            // rows that see it become NaN below).
            if (first_vis - t0 < L::TOK) {
                if (!w.warp(c.kvfull[st], n >> 1)) break;   // (long past: it makes the rows this warp's to read)
                uint8_t *kv = smem + L::OFF_KV + st * L::STAGE;
                const int left = min(L::TOK, p.w.L - t0), end = L::F8 ? left : (left + 7) & ~7;
                for (int k = tid + max(0, first_vis - t0) * 64; k < end * 64; k += 128) {
                    const int r = k >> 6, cc = k & 63;
                    uint4 *at = reinterpret_cast<uint4 *>(kv + (r >> 3) * LT_GROUP + (cc >> 3) * 1024 + (r & 7) * 128 +
                                                          (cc & 7) * 16);
                    if (r >= left) {
                        *at = make_uint4(0, 0, 0, 0);
                    } else if (const uint4 v = *at; not_finite<KV>(v)) {
                        *at = make_uint4(finite_part<KV>(v.x), finite_part<KV>(v.y), finite_part<KV>(v.z),
                                         finite_part<KV>(v.w));
                        atomicMax(&c.poison[p.local % LT_BAD_SLOTS],
                                  (unsigned long long)(p.local + 1) << 32 | (LT_LAST - (uint32_t)(t0 + r)));
                    }
                }
            }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            arrive_warp(c.pfull);
        }
        // ---- the piece's rows: finished, or a partial row
        if (!w.ok || !w.warp(c.pvdone, n - 1)) break;
        tc_fence_after_sync();
        if (live) {
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const bool bad = *reinterpret_cast<volatile int *>(&c.bad[p.local % LT_BAD_SLOTS]) == p.local + 1;
            const unsigned long long poison =
                *reinterpret_cast<volatile unsigned long long *>(&c.poison[p.local % LT_BAD_SLOTS]);
            const bool poisoned = (int)(poison >> 32) == p.local + 1 && vis > (int)(LT_LAST - (uint32_t)poison);
            if (bad || poisoned) l = __int_as_float(0x7fc00000);
            const bool whole = p.whole();
            const float inv = 1.f / l;
            uint16_t *orow = a.out + (a.first_row(p.w, p.r) + m) * LC + 256 * half;
            if (!whole && mine && half == 0) a.ml[p.slot() * LT_ROWS + m] = make_float2(mrun, l);
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
                uint32_t o[32];
                tmem_ld32(trow + 32 * k, o);
                tmem_wait_ld();
                if (mine && whole) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        uint32_t x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[i] = (uint32_t)to_bits<KV>(__uint_as_float(o[j + 2 * i]) * inv) |
                                   ((uint32_t)to_bits<KV>(__uint_as_float(o[j + 2 * i + 1]) * inv) << 16);
                        *reinterpret_cast<uint4 *>(orow + 32 * k + j) = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                } else if (mine) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<uint4 *>(a.o + partial_at(p.slot(), q, k, j / 4, lane)) =
                            make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
                __syncwarp();   // the next load is the whole warp's
            }
        }
        tc_fence_before_sync();
    }
}

template <int KV>
__global__ void __launch_bounds__(Lt<KV>::THREADS, 1)
    latent_kernel(const __grid_constant__ LtMaps maps, const typename Lt<KV>::Args a) {
    using L = Lt<KV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    LtCtrl &c = *reinterpret_cast<LtCtrl *>(smem + L::OFF_CTRL);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&c.kvfull[s]), L::F8 ? L8_WARPS : L::PARTS);
            for (int part = 0; part < 3; ++part) mbar_init(smem_u32(&c.kvempty[s][part]), 1);
            mbar_init(smem_u32(&c.sfull[s]), 1);
            mbar_init(smem_u32(&c.sfree[s]), 4);
        }
        for (int s = 0; s < L8_SLOTS; ++s) {
            mbar_init(smem_u32(&c.full8[s]), 1);
            mbar_init(smem_u32(&c.empty8[s]), L8_WARPS);
        }
        mbar_init(smem_u32(&c.pfull), 4);
        mbar_init(smem_u32(&c.pvdone), 1);
        mbar_init(smem_u32(&c.qfull), 1);
        mbar_init(smem_u32(&c.qempty), 2);
        mbar_init(smem_u32(&c.done), 3);
        c.abort = 0;
        fence_mbar_init();
        tma_prefetch_map(&maps.q);
        if (!L::F8) tma_prefetch_map(&maps.kv);
    } else if (threadIdx.x >= 32 && threadIdx.x < 32 + LT_BAD_SLOTS) {
        c.bad[threadIdx.x - 32] = 0;
        c.poison[threadIdx.x - 32] = 0;
    }
    grid_wait();
    if (warp == 3) {   // (not before: an earlier kernel may still need its own)
        tmem_alloc(smem_u32(&c.tmem), LT_TMEM);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    make_plan(a, &c.plan, c.warp_sums);
    tc_fence_after_sync();
    const Plan plan = c.plan;
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&c.tmem);
    grid_release();   // the merge's CTAs may come as this kernel's leave (they wait for all of them)
    fill_idle_rows<LC / 8>(a, plan, a.out, (long long)a.num_query_tokens * a.H,
                           KV == PA_KV_F16 ? 0x7e007e00u : 0x7fc07fc0u);
    if (plan.u0 < plan.u1) {   // the whole CTA has work, or none of it
        Walk<typename L::Args> p(a, plan);
        if (warp == 0) {
            if constexpr (L::F8)
                lt_load8<KV>(smem, c, a, p, maps);
            else
                lt_load<KV>(smem, c, a, p, maps);
        } else if (warp < 4) {
            if (elect_one()) lt_mma<KV>(smem, c, a, p, tmem, warp);
            __syncwarp();
        } else if (warp < 8) {
            lt_softmax<KV>(smem, c, a, p, tmem);
        } else {
            if constexpr (L::F8) lt_convert<KV>(smem, c, a, p);
        }
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
    }
    if (warp == 3) tmem_dealloc(tmem, LT_TMEM);
    if (threadIdx.x == 0) a.status[blockIdx.x] = c.abort;
}

// ------------------------------------------------------------------ merge

// Rows of the cut row tiles from their pieces' partial rows.  blockIdx.x is the
// CTA whose range begins in the row tile; a warp takes a quarter of its rows (16,
// two lanes each) and eight of a half's 256 dims, in the order in which the
// softmax warps left them.  When a CTA of the first kernel gave up, every row
// becomes NaN.
constexpr int MG_WARPS = 8, MG_BLOCKS = 4 * 32 / MG_WARPS;
static_assert(32 * MG_WARPS >= AXIS_MAX_CTAS, "a thread per CTA's status");

template <int KV>
__global__ void __launch_bounds__(32 * MG_WARPS) latent_merge_kernel(const typename Lt<KV>::Args a, int ctas) {
    grid_release();
    grid_wait();
    const int cta = blockIdx.x, lane = threadIdx.x & 31;
    const int gave_up = threadIdx.x < ctas ? a.status[threadIdx.x] : 0;
    const Cut cut = a.cuts[cta];
    const int unit = blockIdx.y * MG_WARPS + (threadIdx.x >> 5), quarter = unit >> 5;
    if (16 * (blockIdx.y * MG_WARPS >> 5) >= cut.rows && (cta || blockIdx.y)) return;   // the whole block
    const bool failed = __syncthreads_or(gave_up);
    if (cta == 0 && blockIdx.y == 0) {
        if (threadIdx.x == 0) a.hdr->error = failed ? PA_ERR_TIMEOUT : PA_OK;
        if (failed) fill_rows(a.out, 0, (long long)a.num_query_tokens * a.H * (LC / 8), KV == PA_KV_F16 ? 0x7e007e00u : 0x7fc07fc0u);
    }
    const int m = 16 * quarter + (lane & 15), k8 = (unit & 31) >> 2, j = 2 * (unit & 3);
    if (failed || m >= cut.rows) return;
    float acc[8], l;
    join_pieces(
        cut.pieces, [&](int i) { return a.ml[piece_slot(cut, cta, i) * LT_ROWS + m]; },
        [&](int i) { return a.o[partial_at(piece_slot(cut, cta, i), quarter, k8, j, lane)]; },
        [&](int i) { return a.o[partial_at(piece_slot(cut, cta, i), quarter, k8, j + 1, lane)]; }, acc, l);
    const float inv = 1.f / l;
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = (uint32_t)to_bits<KV>(acc[2 * i] * inv) | ((uint32_t)to_bits<KV>(acc[2 * i + 1] * inv) << 16);
    *reinterpret_cast<uint4 *>(a.out + (cut.row0 + m) * LC + 256 * (lane >> 4) + 32 * k8 + 4 * j) =
        make_uint4(v[0], v[1], v[2], v[3]);
}

// ------------------------------------------------------------------ launch

struct LtLayout {
    size_t status, cuts, ml, o, total;
};

LtLayout lt_layout() {
    LtLayout l;
    size_t at = 256;   // header
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at = (at + bytes + 255) / 256 * 256;
        return p;
    };
    l.status = take(sizeof(int) * AXIS_MAX_CTAS);
    l.cuts = take(sizeof(Cut) * AXIS_MAX_CTAS);
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
    const cudaError_t e = cudaFuncSetAttribute(latent_kernel<KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lt<KV>::SMEM);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
    return e;
}

template <int KV>
int launch_latent(const typename Lt<KV>::Args &a, cudaStream_t st) {
    if (lt_setup<KV>() != cudaSuccess) return PA_ERR_CUDA;
    LtMaps maps{};
    const bool ok = row_map(&maps.q, a.query, (long long)a.num_query_tokens * a.H, KV) &&
                    (Lt<KV>::F8 || row_map(&maps.kv, a.cache, a.num_blocks << a.bs_log2, KV));
    if (!ok) return PA_ERR_CUDA;
    const int ctas = std::min(num_sms(), AXIS_MAX_CTAS);
    if (const int e = launch_early(latent_kernel<KV>, dim3((unsigned)ctas), Lt<KV>::THREADS, Lt<KV>::SMEM, st, maps, a))
        return e;
    return launch_early(latent_merge_kernel<KV>, dim3((unsigned)ctas, MG_BLOCKS), 32 * MG_WARPS, 0, st, a, ctas);
}

// Arguments of the kernels for a call.
template <int KV>
int run_latent(void *out, const void *query, const void *cache, const int32_t *block_tables,
               const int32_t *context_lens, const int32_t *query_start, int num_seqs, int num_query_tokens,
               int num_heads, int block_size, int64_t num_blocks, int max_blocks_per_seq, int max_context_len,
               float scale, uint8_t *ws, cudaStream_t st) {
    const LtLayout lay = lt_layout();
    typename Lt<KV>::Args a{};
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
    a.bs_log2 = block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : 6;
    a.mbps = max_blocks_per_seq;
    a.max_context_len = max_context_len;
    a.num_blocks = num_blocks;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.wait_limit = pipeline_wait_limit();
    a.status = reinterpret_cast<int *>(ws + lay.status);
    a.cuts = reinterpret_cast<Cut *>(ws + lay.cuts);
    a.ml = reinterpret_cast<float2 *>(ws + lay.ml);
    a.o = reinterpret_cast<float4 *>(ws + lay.o);
    return launch_latent<KV>(a, st);
}

// PA_DEBUG_VALIDATE of a call: lengths, row offsets and the blocks of every token.
int validate_latent(const int32_t *block_tables, const int32_t *context_lens, const int32_t *query_start, int num_seqs,
                    int num_query_tokens, int block_size, long long num_blocks, int mbps, int max_context_len,
                    cudaStream_t st) try {
    std::vector<int32_t> lens((size_t)num_seqs), start((size_t)num_seqs + 1);
    if (const int e = copy_to_host(lens.data(), context_lens, sizeof(int32_t) * lens.size(), st)) return e;
    if (query_start) {
        if (const int e = validate_starts(query_start, num_seqs, num_query_tokens, true, st)) return e;
        if (const int e = copy_to_host(start.data(), query_start, sizeof(int32_t) * start.size(), st)) return e;
    }
    std::vector<int64_t> last((size_t)num_seqs);
    for (int i = 0; i < num_seqs; ++i) {
        const int len = lens[(size_t)i];
        if (len > max_context_len || (query_start && start[(size_t)i + 1] - start[(size_t)i] > len))
            return PA_ERR_INVALID_ARG;
        last[(size_t)i] = len;
    }
    return validate_tables(block_tables, last.data(), num_seqs, mbps, block_size, num_blocks, st);
} catch (...) {   // no host memory for the check
    return PA_ERR_STATE;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_latent_attention_workspace_size(int num_seqs, int num_query_tokens, int num_heads,
                                                     int max_context_len) {
    if (num_seqs < 0 || num_query_tokens < 0 || num_heads <= 0 || num_heads > 128 || max_context_len < 0) return 0;
    return lt_layout().total;
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
    if (debug_validate())
        if (const int e = validate_latent(block_tables, context_lens, query_start, num_seqs, num_query_tokens, block_size,
                                          num_blocks, max_blocks_per_seq, max_context_len, st))
            return e;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const auto run = kv_dtype == PA_KV_F16    ? run_latent<PA_KV_F16>
                     : kv_dtype == PA_KV_BF16 ? run_latent<PA_KV_BF16>
                                              : run_latent<PA_KV_FP8_E4M3>;
    return run(out, query, cache, block_tables, context_lens, query_start, num_seqs, num_query_tokens, num_heads,
               block_size, num_blocks, max_blocks_per_seq, max_context_len, scale, ws, st);
}
