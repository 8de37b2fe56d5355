// Attention of trees of drafted tokens over the paged cache: a node sees the
// context before the tree, itself and its ancestors.
//
// The query rows of a sequence and kv head are its T nodes times the G heads of
// the group, node by node.  A row tile is up to 256 of them (128 over an FP8
// cache) and sees every KV tile of 128 tokens up to the context's end: only the
// tiles that the tree's own positions reach are masked.  So a KV tile crosses HBM
// once for all nodes of a usual tree.  The row tiles make the work axis
// (work_axis.cuh), cut into equal ranges over the CTAs: one sequence with a long
// context occupies the GPU as well as a batch.
//
// Warps: 0 loads keys and 3 values (TMA boxes of a block's rows, the gather being
// the row coordinate), 1 the queries, 2 issues the MMAs, 4-7 and 8-11 run the
// softmax, a row per thread; over an FP8 cache 12-15 turn the staged codes into
// 16-bit tiles.  Tensor memory: S0, S1 (128 columns each), O0, O1; P is written over
// its S.
//
// A row tile of more than 128 rows is two halves, each with its own S, O and
// softmax warps, that share every tile the CTA loads (PV0(n), S0(n + 1), PV1(n),
// S1(n + 1): one half's products run while the other's softmax works).  With 128
// rows or fewer S0 and S1 are two buffers: S(n + 1) is computed while the softmax
// works on S(n), each of the two warpgroups on 64 of its columns with a maximum, a
// sum and an O of its own, joined at the end.  (A warpgroup each second tile instead:
// the same rate over 16-bit caches, 214 us against 193 on the mix over an FP8 cache.)
//
// What a node sees of a masked tile is found by walking its chain of parents: a
// set of 128 bits.  Values that some row does not see are made finite before the
// product (0 times an infinity is none), and rows that do see one become NaN.
//
// Probabilities are rounded to the 16-bit type because the second product's operands
// have one type; the sums take them unrounded.
//
// What bounds it (one GB300).  16 nodes x 64 heads over 100 x 8192 tokens, bf16: HBM,
// 500 to 517 us, 6.6 TB/s or more (a copy's rate).  25 nodes x 32 heads over 64 contexts
// of 512 .. 16384 tokens, E4M3: 185 us, 3.3 TB/s; the shared memory's pipe: on 32 x 8192
// tokens it is busy for 2070 of a KV tile's 2360 clocks, 1049 of loads and stores (256 read
// codes and 512 store 16-bit tiles; 142 are bank conflicts), 768 of the products' operands,
// 256 of the codes' copies (by their bytes; the others counted).  64 nodes x 64 heads over
// 4 x 32768 tokens, fp16: 216 to 229 us, 1200 to 1270 TFLOP/s; the chain of a half, S with
// its queries from shared memory 856 clocks, softmax 1900, PV 550 and the hand-overs between
// them; the same over E4M3, whose KV tiles come and are turned once per 128 rows, 264 us.
// head_dim 64: 16 nodes x 64 heads over 100 x 8192 tokens, bf16, 286 us, 6.0 TB/s; the wide
// trees 172 us (the softmax's chain is the same for half the products).
// The kernel spills: 208 bytes of stores and 296 of loads (16-bit, head_dim 128; 180 and 256
// with 64; E4M3 128 and 164), in the run 28 loads and 7 stores of a warp a KV tile of the
// wide trees, 11 and 2 over E4M3.
// One sequence of 600 tokens and 8 nodes: 12.5 us, latency (of 100 tokens 10.8).

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>
#include <vector>

#include "decode_common.cuh"
#include "latent.h"
#include "umma.cuh"
#include "work_axis.cuh"

namespace pa {
namespace {

constexpr int TR_HALF = 128;      // rows of a half
constexpr int TR_TOK = 128;       // tokens of a KV tile
constexpr int TR_MAX_ROWS = 256;
constexpr int TR_SOFTMAX_WARPS = 8;

struct TreeArgs {
    uint16_t *out;
    const uint16_t *query;
    const int32_t *block_tables, *context_lens, *query_start, *parents;
    WsHeader *hdr;
    int num_seqs, num_query_tokens, H, Hkv, G, bs, mbps, max_ctx;
    int tile_toks;          // nodes of a row tile
    int ginv;               // 65536 / G + 1: m / G = m * ginv >> 16 for a row m of a tile
    int tinv;               // 2^20 / tile_toks + 1: n / tile_toks = n * tinv >> 20 for n < 2 PA_TREE_MAX_NODES
    long long num_blocks;
    float scale_log2, v_scale;
    long long wait_limit;
    // workspace
    int *status;            // [AXIS_MAX_CTAS] nonzero: the CTA gave up waiting
    Cut *cuts;              // [AXIS_MAX_CTAS]
    float2 *ml;             // [2 AXIS_MAX_CTAS][rows] maximum (log2 units) and sum of a partial row
    float4 *o;              // [2 AXIS_MAX_CTAS][rows * D / 4] its unnormalised output (see partial_at)

    // ---- the work axis: row tile r of a sequence is tile r % per_head of kv head r / per_head
    // With 4 / 8 / 12 / 16, us: 25 nodes x 32 heads over 64 x 512 .. 16384 tokens, E4M3 192 / 185 /
    // 190 / 200, bf16 216 / 201 / 193 / 199, 16 nodes at head_dim 64 116 / 118 / 123 / 130; 16 nodes
    // over 64 x 100 .. 1000, bf16 46 / 46 / 48 / 48; 64 nodes x 64 heads over 24 x 512 .. 8192, bf16
    // 206 / 204 / 186 / 193.  One number for all: 8 is within 9% of the best everywhere.
    static constexpr int COST = 8;
    struct Seq {
        int L, T, q0;
        int per_head;   // row tiles of a kv head
        int rts, ntiles;
        bool valid;
    };
    __device__ __forceinline__ Seq seq_work(int i) const {
        Seq w;
        w.L = context_lens[i];
        w.q0 = query_start[i];
        w.T = query_start[i + 1] - w.q0;
        w.valid = w.L >= 0 && w.L <= max_ctx && w.L <= (long long)mbps * bs && w.T <= w.L && w.T <= PA_TREE_MAX_NODES;
        w.per_head = w.valid ? (w.T + tile_toks - 1) * tinv >> 20 : 0;
        w.rts = w.per_head * Hkv;
        w.ntiles = w.valid ? w.L / TR_TOK + (w.L % TR_TOK != 0) : 0;
        return w;
    }
    __device__ __forceinline__ long long start(const Seq &w, int j, int team) const {
        return (long long)j * (COST + w.ntiles);
    }
    __device__ __forceinline__ int row_tile_at(const Seq &w, long long u, int team) const {
        return min(w.rts / team - 1, (int)quick_div(u, COST + w.ntiles));
    }
    __device__ __forceinline__ bool in_teams(const Seq &w) const { return w.per_head % 2 == 0; }
    __device__ __forceinline__ int row_tiles(const Seq &w, int r) const { return w.ntiles; }
    __device__ __forceinline__ int first_tiles(const Seq &w, int r) const { return w.ntiles; }
    // kv head of a row tile, its first node (a tree is one row tile a head as a rule)
    __device__ __forceinline__ int head(const Seq &w, int r) const { return w.per_head == 1 ? r : r / w.per_head; }
    __device__ __forceinline__ int first_node(const Seq &w, int r) const {
        return w.per_head == 1 ? 0 : r % w.per_head * tile_toks;
    }
    __device__ __forceinline__ int cut_rows(const Seq &w, int r) const {
        return min(tile_toks, w.T - first_node(w, r)) * G;
    }
    __device__ __forceinline__ long long first_row(const Seq &w, int r) const {
        return (long long)(w.q0 + first_node(w, r)) * H + head(w, r) * G;
    }
    __device__ __forceinline__ bool seq_ok(int i) const { return query_start[i] <= query_start[i + 1]; }
    __device__ __forceinline__ bool ends_ok() const {
        return *query_start == 0 && query_start[num_seqs] == num_query_tokens;
    }
    // row m of a row tile, counted from the tile's first row in the output
    __device__ __forceinline__ long long row_at(int m) const {
        const int j = m * ginv >> 16;
        return (long long)j * H + (m - j * G);
    }
};

// Shared memory, tiles and threads of the kernel for a cache type and head_dim.
template <int KV, int D>
struct Tree {
    static constexpr bool F8 = KV == PA_KV_FP8_E4M3;
    static constexpr int MK = F8 ? PA_KV_F16 : KV;         // type of the MMAs' operands
    static constexpr int ROWS = F8 ? TR_HALF : TR_MAX_ROWS;
    static constexpr int BLOCK = TR_TOK * 128;             // 128 rows x 64 elements, 128-byte swizzle
    static constexpr int TILE = BLOCK * (D / 64);          // a key or value tile of 16-bit elements, a half's queries
    // Tiles on their way: of 16-bit caches key tiles in the first K_RING slots, value
    // tiles in the others; of FP8 caches staged codes likewise, and the converted tiles
    // in the order in which they are used.
    static constexpr int RING = F8 ? 3 : 10 / (D / 64), K_RING = (RING + 1) / 2;
    static constexpr int CODES = F8 ? TR_TOK * D : 0;      // a staged tile of codes
    static constexpr int STAGES = F8 ? 4 : 0, K_STAGES = 2;
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int OFF_STAGE = OFF_RING + RING * TILE;
    static constexpr int OFF_CTRL = OFF_STAGE + STAGES * CODES;
    static constexpr int CTRL = 3 * 1024;
    static constexpr int SMEM = OFF_CTRL + CTRL;
    static constexpr int THREADS = F8 ? 512 : 384;
    static constexpr int REGS_LAUNCH = F8 ? 128 : 168;     // per thread: 65536 / threads, rounded down to 8
    static constexpr int REGS_LOW = 104;                   // warps 0 - 3
    static constexpr int REGS_HIGH = F8 ? 152 : 200;       // the softmax warps
    static constexpr int REGS_CONV = 104;                  // the converting warps
    static constexpr int CONV_WARPS = 4;
    static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
    static_assert(128 * (REGS_LOW + 2 * REGS_HIGH + (F8 ? REGS_CONV : 0)) <= THREADS * REGS_LAUNCH,
                  "register split within the launch's pool");
};
constexpr int TR_TMEM = 512, TR_O = 256;   // S0, S1 at columns 0 and 128; O0, O1 at 256 and 384
constexpr int TR_MAX_RING = 10, TR_MAX_STAGES = 4;
constexpr int TR_MARKS = 16;               // pieces whose tiles can be on their way, and more
constexpr int TR_SEEN = PA_TREE_MAX_NODES / 32;
static_assert(2 * TR_SEEN == TR_MARKS, "set up by the same threads");

struct TrCtrl {
    uint64_t full[TR_MAX_RING], empty[TR_MAX_RING], stfull[TR_MAX_STAGES], stempty[TR_MAX_STAGES];
    uint64_t qfull[2], qempty[2];
    // by S buffer; one set for tiles whose columns both warpgroups share, one for
    // buffers of one warpgroup each
    uint64_t sfull[2][2], pfull[2][2], pvdone[2][2];
    uint64_t meet[2];       // of all softmax warps, at a piece's end and after it
    uint64_t done;
    uint32_t tmem;
    int abort;
    Plan plan;
    long long warp_sums[16];
    int bad[TR_MARKS];      // 1 + the number of a piece that met a block id out of range
    // Nodes whose values are not finite, as the softmax warps find them, by the
    // piece's parity (the next piece's set is emptied between the two meetings).
    uint32_t poison[2][TR_SEEN];
    float2 ml[2][TR_HALF];  // a row's maximum and sum as either warpgroup has them
};

// Where the softmax keeps four dims (32 k + 4 j ..) of a row, in float4: a store
// of a warp's 32 rows (rows 32 q .. of the row tile) is one run of 512 bytes.
template <int KV, int D>
__device__ __forceinline__ long long partial_at(int slot, int q, int k, int j, int lane) {
    return (((long long)slot * (Tree<KV, D>::ROWS / 32) + q) * (D / 32) + k) * 8 * 32 + j * 32 + lane;
}

// A piece of a row tile, in every role alike.
struct TrPiece {
    int g, node0, rows, n;   // kv head, first node, rows, KV tiles
    bool two;                // two halves
};
__device__ __forceinline__ TrPiece piece_of(const TreeArgs &a, const Walk<TreeArgs> &p) {
    TrPiece x;
    x.g = a.head(p.w, p.r);
    x.node0 = a.first_node(p.w, p.r);
    x.rows = a.cut_rows(p.w, p.r);
    x.n = p.t1 - p.t0;
    x.two = x.rows > TR_HALF;
    return x;
}
// A slot of a ring and the parity of its use.
struct TrSlot {
    int at;
    uint32_t parity;
};
__device__ __forceinline__ TrSlot slot_of(int first, int slots, int use) {
    return {first + use % slots, (uint32_t)(use / slots & 1)};
}
// Where the n-th key or value tile of a piece lies, `done` tiles after the CTA's
// first.  Converted tiles follow one another as K(0), then K(n + 1), V(n), the last V
// at the end.
template <int KV, int D>
__device__ __forceinline__ TrSlot k_slot(int done, int n) {
    using X = Tree<KV, D>;
    if (X::F8) return slot_of(0, X::RING, 2 * done + (n ? 2 * n - 1 : 0));
    return slot_of(0, X::K_RING, done + n);
}
template <int KV, int D>
__device__ __forceinline__ TrSlot v_slot(int done, int n, int all) {
    using X = Tree<KV, D>;
    if (X::F8) return slot_of(0, X::RING, 2 * done + (n + 1 < all ? 2 * n + 2 : 2 * all - 1));
    return slot_of(X::K_RING, X::RING - X::K_RING, done + n);
}

// A whole warp's bounded wait (for two barriers at once: a wait costs its latency
// even when it is over).
struct WarpWait {
    TrCtrl &c;
    long long limit;
    bool ok = true;
    __device__ __forceinline__ bool slow(uint64_t *bar, uint32_t parity) {
        volatile int *abort_flag = &c.abort;
        const bool got = ok && !*abort_flag && mbar_wait_bounded(smem_u32(bar), parity, limit);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) *abort_flag = 1;
        return ok;
    }
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity)) || slow(bar, parity);
    }
    __device__ __forceinline__ bool both(uint64_t *a, uint32_t pa, uint64_t *b, uint32_t pb) {
        const bool got_b = mbar_try_wait(smem_u32(b), pb), got_a = mbar_try_wait(smem_u32(a), pa);
        return __all_sync(0xffffffffu, got_a && got_b) || (slow(a, pa) && slow(b, pb));
    }
};

// One warp: the key tiles, or another one: the value tiles.  A lane finds a block's
// rows (its id is read a tile ahead of its use), and copies them as a box (two, of 64
// elements each).  (One warp for both worked 1830 clocks a tile over FP8 caches and
// bound the kernel, a single lane for each 1560.)
template <int KV, int D>
__device__ void tr_load(TrCtrl &c, const TreeArgs &a, Walk<TreeArgs> &p, uint32_t smem, const CUtensorMap *tm, bool values) {
    using X = Tree<KV, D>;
    constexpr int ROW = X::F8 ? D : 2 * D;        // bytes of a row
    constexpr int SLOTS = X::F8 ? X::STAGES : X::RING, KS = X::F8 ? X::K_STAGES : X::K_RING;
    constexpr int BYTES = X::F8 ? X::CODES : X::TILE;
    const int lane = threadIdx.x & 31;
    uint64_t *full = X::F8 ? c.stfull : c.full, *empty = X::F8 ? c.stempty : c.empty;
    const int first = values ? KS : 0, slots = values ? SLOTS - KS : KS;
    const uint32_t base = smem + (X::F8 ? X::OFF_STAGE : X::OFF_RING) + lane * a.bs * 128;
    const int boxes = TR_TOK / a.bs;
    const uint32_t num_blocks = (uint32_t)a.num_blocks;   // (rows of the caches are counted in 31 bits)
    const uint64_t once = policy_evict_first(), again = policy_evict_normal();
    WarpWait wait{c, a.wait_limit};
    int use = 0, at = 0;                          // tiles so far; the slot of the next (of this warp's)
    uint32_t parity = 1;
    while (wait.ok && p.next()) {
        const int g = a.head(p.w, p.r);
        const uint64_t policy = p.w.per_head > 1 ? again : once;
        const int32_t *table = a.block_tables + (long long)p.seq * a.mbps;
        const int blocks = (p.w.L - 1) / a.bs + 1;
        auto read = [&](int t) { return lane < boxes && t * boxes + lane < blocks ? table[t * boxes + lane] : 0; };
        int id = read(p.t0);
        for (int t = p.t0; t < p.t1; ++t) {
            const int some = min(boxes, blocks - t * boxes);   // the context ends in the last of them
            const bool out = (uint32_t)id >= num_blocks;
            // by the lane that arrives: its arrival publishes the mark to those that read it
            if (__any_sync(0xffffffffu, out) && lane == 0)
                *reinterpret_cast<volatile int *>(&c.bad[p.local % TR_MARKS]) = p.local + 1;
            const int row = ((out ? 0 : id) * a.Hkv + g) * a.bs;
            if (t + 1 < p.t1) id = read(t + 1);
            if (!wait(&empty[first + at], parity)) break;
            const uint32_t bar = smem_u32(&full[first + at]), dst = base + (first + at) * BYTES;
            if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(some * a.bs * ROW));
            __syncwarp();
            if (lane < some) {
                tma_load_2d(dst, tm, 0, row, bar, policy);
                if (!X::F8 && D == 128) tma_load_2d(dst + X::BLOCK, tm, 64, row, bar, policy);
            }
            ++use;
            if (++at == slots) at = 0, parity ^= 1;
        }
    }
    // the last copies into every slot have landed before the CTA leaves
    for (int s = 0; s < slots; ++s)
        if (use > s)
            mbar_wait_bounded(smem_u32(&full[first + (use - 1 - s) % slots]), (uint32_t)(((use - 1 - s) / slots) & 1),
                              WAIT_LIMIT);
}

// One warp: rows [from, to) of a half's queries, as the products read them, into the
// tile at dst (query row m0 of the row tile is the half's first); they are there on return.
template <int D>
__device__ __forceinline__ void load_queries(const TreeArgs &a, const uint16_t *first, int m0, int from, int to, uint32_t dst) {
    constexpr int CH = D / 8, BLOCK = TR_TOK * 128;   // 16-byte chunks of a row
    const int lane = threadIdx.x & 31, ch = lane % CH;
#pragma unroll 2
    for (int m = from + lane / CH; m < to; m += 32 / CH) {
        const uint16_t *src = first + a.row_at(m0 + m) * D + 8 * ch;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         dst + (ch / 8) * BLOCK + m * 128 + (((ch & 7) ^ (m & 7)) << 4)),
                     "l"(src)
                     : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    __syncwarp();
}

// One warp: the queries of all pieces but a CTA's first.  (That one's the softmax warps
// load, which have nothing else to do yet: a warp takes 60 clocks for 512 bytes, 256 rows
// 7700.)
template <int KV, int D>
__device__ void tr_query(uint8_t *smem, TrCtrl &c, const TreeArgs &a, Walk<TreeArgs> &p) {
    using X = Tree<KV, D>;
    const int lane = threadIdx.x & 31;
    WarpWait wait{c, a.wait_limit};
    uint32_t phase = 3;   // of the buffers' release (a bit each)
    int sel = 0;
    while (wait.ok && p.next()) {
        const TrPiece x = piece_of(a, p);
        const uint16_t *first = a.query + a.first_row(p.w, p.r) * D;
        for (int h = 0; wait.ok && h < (x.two ? 2 : 1); ++h) {
            const int b = x.two ? h : sel;
            phase ^= 1u << b;
            if (p.local == 0) continue;
            if (!wait(&c.qempty[b], phase >> b & 1u ^ 1u)) break;
            load_queries<D>(a, first, h * TR_HALF, 0, min(TR_HALF, x.rows - h * TR_HALF), smem_u32(smem) + b * X::TILE);
            if (lane == 0) mbar_arrive_many(smem_u32(&c.qfull[b]), TR_SOFTMAX_WARPS);
        }
        if (!x.two) sel ^= 1;
    }
}

// The converting warps (w of CONV_WARPS): staged codes to fp16 tiles of the same
// swizzled layout (every E4M3 value is an fp16 value).  A warp's eight lanes of a
// row store their 16-byte pieces so that all banks are covered: those of the
// second 64 dims their odd one first.
template <int KV, int D>
__device__ void tr_convert(uint8_t *smem, TrCtrl &c, const TreeArgs &a, Walk<TreeArgs> &p, int w) {
    using X = Tree<KV, D>;
    constexpr int N = X::CODES / 16 / (32 * X::CONV_WARPS);   // 16-byte chunks a thread
    const int lane = threadIdx.x & 31;
    WarpWait wait{c, a.wait_limit};
    int cnt = 0, kuse = 0, vuse = 0;
    while (wait.ok && p.next()) {
        for (int k = 0; wait.ok && k < 2 * (p.t1 - p.t0); ++k, ++cnt) {
            // in the order of their use: K(0), then K(n + 1), V(n), the last V
            const int s = cnt % X::RING, all = p.t1 - p.t0;
            const bool value = k > 0 && (k % 2 == 0 || k == 2 * all - 1);
            const TrSlot from_slot = value ? slot_of(X::K_STAGES, X::STAGES - X::K_STAGES, vuse++)
                                           : slot_of(0, X::K_STAGES, kuse++);
            const int st = from_slot.at;
            if (!wait(&c.stfull[st], from_slot.parity)) break;
            const uint8_t *from = smem + X::OFF_STAGE + st * X::CODES;
            uint4 v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = (w * N + i) * 32 + lane, m = at / 8, cc = at & 7;
                v[i] = *reinterpret_cast<const uint4 *>(from + m * 128 + ((cc ^ (m & 7)) << 4));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c.stempty[st]));
            if (!wait(&c.empty[s], (uint32_t)(((cnt / X::RING) & 1) ^ 1))) break;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = (w * N + i) * 32 + lane, m = at / 8, cc = at & 7;
                uint8_t *to = smem + X::OFF_RING + s * X::TILE + (cc >> 2) * X::BLOCK + m * 128;
                const uint4 lo = make_uint4(e4m3x2_lo_to_f16x2(v[i].x), e4m3x2_hi_to_f16x2(v[i].x),
                                            e4m3x2_lo_to_f16x2(v[i].y), e4m3x2_hi_to_f16x2(v[i].y));
                const uint4 hi = make_uint4(e4m3x2_lo_to_f16x2(v[i].z), e4m3x2_hi_to_f16x2(v[i].z),
                                            e4m3x2_lo_to_f16x2(v[i].w), e4m3x2_hi_to_f16x2(v[i].w));
                const int odd = cc >> 2, ch = (cc & 3) * 2;
                *reinterpret_cast<uint4 *>(to + (((ch + odd) ^ (m & 7)) << 4)) = odd ? hi : lo;
                *reinterpret_cast<uint4 *>(to + (((ch + 1 - odd) ^ (m & 7)) << 4)) = odd ? lo : hi;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c.full[s]));
        }
    }
}

// One lane: the MMAs.
template <int KV, int D>
__device__ void tr_mma(uint8_t *smem, TrCtrl &c, const TreeArgs &a, Walk<TreeArgs> &p, uint32_t tmem) {
    using X = Tree<KV, D>;
    const uint32_t base = smem_u32(smem);
    constexpr uint32_t ID_S = idesc_f16(TR_HALF, TR_TOK, X::MK == PA_KV_BF16, false);
    constexpr uint32_t ID_O = idesc_f16(TR_HALF, D, X::MK == PA_KV_BF16, true);
    const uint64_t dq0 = sw128_desc(base, 16, 1024);
    const uint64_t dk0 = sw128_desc(base + X::OFF_RING, 16, 1024);
    const uint64_t dv0 = sw128_desc(base + X::OFF_RING, X::BLOCK, 1024);
    volatile int *abort_flag = &c.abort;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(smem_u32(bar), parity)) return true;
        ok = ok && !*abort_flag && mbar_wait_bounded(smem_u32(bar), parity, a.wait_limit);
        if (!ok) *abort_flag = 1;
        return ok;
    };
    int done = 0, sel = 0;          // KV tiles before this piece; the next query buffer of one half
    uint32_t qphase = 0, phase = 0; // of the query barriers; of the P barriers: bits 0 and 1 of shared, 2 and 3 of own buffers
    auto q_wait = [&](int q) {
        const uint32_t now = qphase >> q & 1u;
        qphase ^= 1u << q;
        return wait(&c.qfull[q], now);
    };
    auto ring_wait = [&](const TrSlot &k) {
        const bool got = wait(&c.full[k.at], k.parity);
        tc_fence_after_sync();
        return got;
    };
    auto p_wait = [&](int own, int b) {
        const uint32_t now = phase >> (2 * own + b) & 1u;
        phase ^= 1u << (2 * own + b);
        const bool got = wait(&c.pfull[own][b], now);
        tc_fence_after_sync();
        return got;
    };
    auto release = [&](const TrSlot &k) { umma_commit(smem_u32(&c.empty[k.at])); };
    // S in buffer b = the queries of buffer q times the key tile at k
    auto issue_s = [&](int b, int q, const TrSlot &k) {
        const uint64_t dk = dk0 + (uint64_t)(k.at * (X::TILE >> 4)), dq = dq0 + (uint64_t)(q * (X::TILE >> 4));
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                umma_f16(tmem + b * TR_TOK, dq + h * (X::BLOCK >> 4) + 2 * j, dk + h * (X::BLOCK >> 4) + 2 * j, ID_S,
                         h > 0 || j > 0 ? 1u : 0u);
    };
    // O_h += the P in buffer h times the value tile at k (16 tokens: P columns 8 j .., V rows 16 j ..)
    auto issue_pv = [&](int h, const TrSlot &k, bool first) {
        const uint64_t dv = dv0 + (uint64_t)(k.at * (X::TILE >> 4));
#pragma unroll
        for (int j = 0; j < TR_TOK / 16; ++j)
            umma_f16_ts(tmem + TR_O + h * 128, tmem + h * TR_TOK + 8 * j, dv + (uint64_t)((j * 16 * 128) >> 4), ID_O,
                        !first || j > 0 ? 1u : 0u);
        umma_commit(smem_u32(&c.pvdone[1][h]));
    };
    while (ok && p.next()) {
        const TrPiece x = piece_of(a, p);
        const int N = x.n;
        if (!x.two) {   // S(n) in buffer n & 1, its columns 64 w .. the warpgroup w's, whose products go to O_w
            const TrSlot k0 = k_slot<KV, D>(done, 0);
            if (!q_wait(sel) || !ring_wait(k0)) break;
            issue_s(0, sel, k0);
            umma_commit(smem_u32(&c.sfull[0][0]));
            release(k0);
            if (N == 1) umma_commit(smem_u32(&c.qempty[sel]));
            for (int n = 0; n < N; ++n) {
                const int b = n & 1;
                const TrSlot v = v_slot<KV, D>(done, n, N);
                if (n + 1 < N) {   // buffer b ^ 1: its P has been taken by PV(n - 1)
                    const TrSlot k = k_slot<KV, D>(done, n + 1);
                    if (!ring_wait(k)) break;
                    issue_s(b ^ 1, sel, k);
                    umma_commit(smem_u32(&c.sfull[0][b ^ 1]));
                    release(k);
                    if (n + 2 == N) umma_commit(smem_u32(&c.qempty[sel]));
                }
                if (!p_wait(0, b) || !ring_wait(v)) break;
                const uint64_t dv = dv0 + (uint64_t)(v.at * (X::TILE >> 4));
#pragma unroll
                for (int j = 0; j < TR_TOK / 16; ++j)   // 16 tokens: P columns 64 w + 8 (j % 4) .., V rows 16 j ..
                    umma_f16_ts(tmem + TR_O + j / 4 * 128, tmem + b * TR_TOK + j / 4 * 64 + 8 * (j % 4),
                                dv + (uint64_t)((j * 16 * 128) >> 4), ID_O, n > 0 || j % 4 > 0 ? 1u : 0u);
                umma_commit(smem_u32(&c.pvdone[0][b]));
                release(v);
            }
            sel ^= 1;
        } else {        // half h in buffer h
            const TrSlot k0 = k_slot<KV, D>(done, 0);
            if (!q_wait(0) || !q_wait(1) || !ring_wait(k0)) break;
            for (int h = 0; h < 2; ++h) {
                issue_s(h, h, k0);
                umma_commit(smem_u32(&c.sfull[1][h]));
                if (N == 1) umma_commit(smem_u32(&c.qempty[h]));
            }
            release(k0);
            for (int n = 0; ok && n < N; ++n) {
                const bool more = n + 1 < N;
                const TrSlot v = v_slot<KV, D>(done, n, N), k = k_slot<KV, D>(done, n + 1);
                for (int h = 0; h < 2; ++h) {
                    if (!p_wait(1, h) || (h == 0 && !ring_wait(v))) break;
                    issue_pv(h, v, n == 0);
                    if (h == 1) release(v);
                    if (more) {
                        if (h == 0 && !ring_wait(k)) break;
                        issue_s(h, h, k);
                        umma_commit(smem_u32(&c.sfull[1][h]));
                        if (n + 2 == N) umma_commit(smem_u32(&c.qempty[h]));
                        if (h == 1) release(k);
                    }
                }
            }
        }
        done += N;
    }
    // every product issued has completed before tensor memory is freed
    umma_commit(smem_u32(&c.done));
    mbar_wait_bounded(smem_u32(&c.done), 0, WAIT_LIMIT);
}

// How the two softmax warpgroups share a piece: COLUMNS, each takes 64 columns of
// every tile (one half; S in turn in either buffer); HALVES, each takes its half's
// rows.
enum { COLUMNS, HALVES };

// A softmax warpgroup's state and its way through a piece's tiles, a row per thread.
template <int KV, int D>
struct TrRows {
    using X = Tree<KV, D>;
    static constexpr int MK = X::MK;
    TrCtrl &c;
    const TreeArgs &a;
    WarpWait wait;
    uint8_t *smem;
    uint32_t trow, ocol;
    int x, m, lane;
    uint32_t phase;        // of the S barriers: bits 0 and 1 of shared buffers, bit 2 of its own
    int done;              // KV tiles before this piece
    float mrun, l;
    bool lost;             // the chain of parents is broken

    template <int MODE>
    __device__ __forceinline__ void tiles(const Walk<TreeArgs> &p, const TrPiece &pc, bool mine, bool idle, int node,
                                          uint32_t *poison) {
        constexpr bool SHARED = MODE == COLUMNS;
        constexpr int COLS = SHARED ? TR_TOK / 2 : TR_TOK;
        const float sl2 = a.scale_log2;
        const int ctx = p.w.L - p.w.T;                 // positions before the tree
        const int32_t *parents = a.parents + p.w.q0;
        mrun = -INFINITY;
        l = 0.f;
        lost = false;
        for (int n = 0; n < pc.n; ++n) {
            const int b = SHARED ? n & 1 : x, bit = SHARED ? b : 2;
            const uint32_t now = phase >> bit & 1u;
            const uint32_t scol = (uint32_t)(b * TR_TOK + (SHARED ? x * COLS : 0));
            // S, and the products with this buffer's last P (done when S is; every phase
            // is seen, so that one waited for later is not taken for another)
            const bool there = n > (SHARED ? 1 : 0)
                                   ? wait.both(&c.sfull[!SHARED][b], now, &c.pvdone[!SHARED][b], now ^ 1u)
                                   : wait(&c.sfull[!SHARED][b], now);
            if (!there) return;
            tc_fence_after_sync();
            const int t0 = (p.t0 + n) * TR_TOK;
            const bool tail = ctx - t0 < TR_TOK;       // the tree's positions begin before the tile ends
            bool changed = false;
            if (tail && (x == 0 || SHARED)) {
                // Value rows that some row of the row tile does not see, where P is 0
                // and a product with an infinity or a NaN would not be: those behind the
                // context are zeroed, and so is what is not finite among the nodes' (the
                // rows that see it become NaN below).  Of two halves the first one's
                // warps do it for both: PV1(n) is issued after P0(n).
                const TrSlot at = v_slot<KV, D>(done, n, pc.n);
                if (!wait(&c.full[at.at], at.parity)) return;
                const int lo = max(0, ctx - t0), hi = p.w.L - t0, r0 = (SHARED ? x * COLS : 0) + m / 8;
#pragma unroll 1
                for (int h = 0; h < D / 64; ++h) {
                    uint4 *blk = reinterpret_cast<uint4 *>(smem + X::OFF_RING + at.at * X::TILE + h * X::BLOCK) +
                                 (SHARED ? x * COLS * 8 : 0);
                    // this thread's chunks m, m + 128, ..: row m / 8 + 16 i, from the first node's on
#pragma unroll 1
                    for (int i = max(0, (lo - r0 + 15) >> 4); i < COLS / 16; ++i) {
                        const int r = r0 + 16 * i;
                        uint4 &v = blk[m + TR_HALF * i];
                        if (r >= hi) {
                            v = make_uint4(0, 0, 0, 0);
                        } else if (not_finite<MK>(v)) {
                            v = make_uint4(finite_part<MK>(v.x), finite_part<MK>(v.y), finite_part<MK>(v.z),
                                           finite_part<MK>(v.w));
                            const int bad = t0 + r - ctx;
                            atomicOr(&poison[bad >> 5], 1u << (bad & 31));
                        }
                    }
                }
                changed = true;
            }
            if (!idle) {
                float s[COLS];
#pragma unroll
                for (int q = 0; q < COLS / 32; ++q) {
                    uint32_t r[32];
                    tmem_ld32(trow + scol + 32 * q, r);
#pragma unroll
                    for (int k = 0; k < 32; ++k) s[32 * q + k] = __uint_as_float(r[k]);
                }
                tmem_wait_ld();
                if (tail) {
                    // what the row sees of its columns, a bit each: the context, then its chain
                    const int c0 = t0 + (SHARED ? x * COLS : 0);
                    uint32_t see[COLS / 32];
#pragma unroll
                    for (int k = 0; k < COLS / 32; ++k) {
                        const int before = min(32, ctx - c0 - 32 * k);
                        see[k] = !mine || before <= 0 ? 0u : before == 32 ? ~0u : (1u << before) - 1u;
                    }
                    for (int j = mine ? node : -1; j >= 0;) {
                        const int at = ctx + j - c0;
#pragma unroll
                        for (int k = 0; k < COLS / 32; ++k)
                            if (at >> 5 == k) see[k] |= 1u << (at & 31);
                        const int up = parents[j];
                        lost = lost || up < -1 || up >= j;
                        j = lost ? -1 : up;
                    }
#pragma unroll
                    for (int k = 0; k < COLS; ++k) s[k] = see[k / 32] >> (k & 31) & 1u ? s[k] : -INFINITY;
                }
                float mp[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int k = 4; k + 8 <= COLS; k += 8)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mp[j] = max3(mp[j], s[k + 2 * j], s[k + 2 * j + 1]);
#pragma unroll
                for (int j = 0; j < 4; ++j) mp[j] = fmaxf(mp[j], s[COLS - 4 + j]);
                const float mx = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])) * sl2;
                // decided per row, done warp-wide (tensor-memory accesses are the
                // whole warp's); rows that do not grow scale by exactly 1
                const bool grow = mx > mrun + RESCALE_THRESHOLD;
                if (__any_sync(0xffffffffu, grow)) {
                    const float nm = grow ? mx : mrun;
                    const float alpha = grow ? fast_exp2(mrun - nm) : 1.f;
                    if (n > 0) {
                        // (a buffer of its own: the last products into O are complete, S(n) was issued after them)
                        if (SHARED && !wait(&c.pvdone[0][b ^ 1], (phase >> (b ^ 1) & 1u) ^ 1u)) return;
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
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
                const float mu = mrun == -INFINITY ? 0.f : mrun;   // a row that has seen nothing yet
                const uint64_t sl2x2 = pair_of(sl2, sl2), negm = pair_of(-mu, -mu);
                uint64_t lp[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) lp[j] = 0;
#pragma unroll
                for (int q = 0; q < COLS / 64; ++q) {
                    uint32_t r[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        float e0, e1;
                        pair_parts(pair_fma(pair_of(s[64 * q + 2 * k], s[64 * q + 2 * k + 1]), sl2x2, negm), e0, e1);
                        e0 = fast_exp2(e0);
                        e1 = fast_exp2(e1);
                        lp[k & 3] = pair_add(lp[k & 3], pair_of(e0, e1));
                        r[k] = pack_p<MK>(e0, e1);
                    }
                    tmem_st32(trow + scol + 32 * q, r);
                }
                float l0, l1;
                pair_parts(pair_add(pair_add(lp[0], lp[1]), pair_add(lp[2], lp[3])), l0, l1);
                l += l0 + l1;
                tmem_wait_st();
            }
            if (changed) fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();   // one arrival a warp: 32 atomics on one word hold up the shared-memory pipe
            if (lane == 0) mbar_arrive(smem_u32(&c.pfull[!SHARED][b]));
            phase ^= 1u << bit;
        }
        // the last products (and, of shared buffers, those before them)
        if (!SHARED) {
            wait(&c.pvdone[1][x], (phase >> 2 & 1u) ^ 1u);
        } else {
            const int b = (pc.n - 1) & 1;
            if (pc.n > 1) wait(&c.pvdone[0][b ^ 1], (phase >> (b ^ 1) & 1u) ^ 1u);
            wait(&c.pvdone[0][b], (phase >> b & 1u) ^ 1u);
        }
    }
};

// One warpgroup: the softmax and the output rows of half x, or of columns 64 x ..
template <int KV, int D>
__device__ void tr_softmax(uint8_t *smem, TrCtrl &c, const TreeArgs &a, Walk<TreeArgs> &p, uint32_t tmem, int x) {
    using X = Tree<KV, D>;
    constexpr int MK = X::MK;
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, m = quarter * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t ocol = (uint32_t)(TR_O + x * 128);
    TrRows<KV, D> rows{c, a, WarpWait{c, a.wait_limit}, smem, trow, ocol, x, m, lane, 0u, 0, 0.f, 0.f, false};
    WarpWait &wait = rows.wait;
    int met = 0;                    // pieces before this one
    auto meet = [&](int k) {        // all softmax warps
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.meet[k]));
        const bool got = wait(&c.meet[k], (uint32_t)(met & 1));
        tc_fence_after_sync();
        return got;
    };
    while (wait.ok && p.next()) {
        const TrPiece pc = piece_of(a, p);
        const int mm = pc.two ? x * TR_HALF + m : m;   // row of the row tile
        const bool mine = mm < pc.rows;
        const bool idle = !__any_sync(0xffffffffu, mine);
        if (p.local == 0) {   // its queries: a quarter of a half each, an eighth of one half
            const uint16_t *first = a.query + a.first_row(p.w, p.r) * D;
            const int some = pc.two ? 32 : 16, from = some * (pc.two ? quarter : 4 * x + quarter), b = pc.two ? x : 0;
            load_queries<D>(a, first, b * TR_HALF, from, min(from + some, pc.rows - b * TR_HALF), smem_u32(smem) + b * X::TILE);
            if (lane == 0) mbar_arrive_many(smem_u32(&c.qfull[b]), pc.two ? 2 : 1);
        }
        const int node = pc.node0 + (mm * a.ginv >> 16);
        const int32_t *parents = a.parents + p.w.q0;
        uint32_t *poison = c.poison[p.local & 1];
        if constexpr (!X::F8) {
            if (pc.two) rows.template tiles<HALVES>(p, pc, mine, idle, node, poison);
        }
        if (X::F8 || !pc.two) rows.template tiles<COLUMNS>(p, pc, mine, idle, node, poison);
        if (!wait.ok) break;
        rows.done += pc.n;
        float mrun = rows.mrun, l = rows.l;
        // ---- the piece's rows: finished, or a partial row
        if (rows.lost) l = __int_as_float(0x7fc00000);
        c.ml[x][m] = make_float2(mrun, l);
        if (!meet(0)) break;
        if (x == 0 && threadIdx.x % 128 < TR_SEEN) c.poison[(p.local & 1) ^ 1][threadIdx.x % 128] = 0;
        if (!idle) {
            const float2 other = c.ml[x ^ 1][m];
            const uint32_t any = lane < TR_SEEN ? *reinterpret_cast<volatile uint32_t *>(&poison[lane]) : 0u;
            bool nan = *reinterpret_cast<volatile int *>(&c.bad[p.local % TR_MARKS]) == p.local + 1;
            if (__any_sync(0xffffffffu, any != 0))
                for (int j = mine ? node : -1; j >= 0;) {
                    if (*reinterpret_cast<volatile uint32_t *>(&poison[j >> 5]) >> (j & 31) & 1u) nan = true;
                    const int up = parents[j];
                    j = up >= j ? -1 : up;   // (a broken chain has made its row NaN)
                }
            // one half: what both warpgroups saw joined, each of them makes half of the dims
            float wa = 1.f, wb = 0.f;
            if (!pc.two) {
                const float2 ma = x == 0 ? make_float2(mrun, l) : other, mb = x == 0 ? other : make_float2(mrun, l);
                mrun = fmaxf(ma.x, mb.x);
                const float mu = mrun == -INFINITY ? 0.f : mrun;
                wa = fast_exp2(ma.x - mu);
                wb = fast_exp2(mb.x - mu);
                l = ma.y * wa + mb.y * wb;
            }
            if (nan) l = __int_as_float(0x7fc00000);
            const bool whole = p.whole();
            if (!whole && mine && (pc.two || x == 0)) a.ml[(long long)p.slot() * X::ROWS + mm] = make_float2(mrun, l);
            const float out = whole ? a.v_scale / l : 1.f;
            wa *= out;
            wb *= out;
            uint16_t *orow = a.out + (a.first_row(p.w, p.r) + a.row_at(mm)) * D;
            const int q0 = pc.two ? 0 : x * (D / 64), q1 = pc.two ? D / 32 : q0 + D / 64;
#pragma unroll 1
            for (int q = q0; q < q1; ++q) {
                uint32_t o[32];
                tmem_ld32(trow + (pc.two ? ocol : (uint32_t)TR_O) + 32 * q, o);
                if (!pc.two) {
                    uint32_t o2[32];
                    tmem_ld32(trow + TR_O + 128 + 32 * q, o2);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        o[k] = __float_as_uint(fmaf(__uint_as_float(o2[k]), wb, __uint_as_float(o[k]) * wa));
                } else {
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * wa);
                }
                if (mine && whole) {
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = (uint32_t)out_bits<MK>(__uint_as_float(o[k + 2 * i])) |
                                   ((uint32_t)out_bits<MK>(__uint_as_float(o[k + 2 * i + 1])) << 16);
                        *reinterpret_cast<uint4 *>(orow + 32 * q + k) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else if (mine) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        *reinterpret_cast<uint4 *>(a.o + partial_at<KV, D>(p.slot(), mm / 32, q, k / 4, lane)) =
                            make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                }
                __syncwarp();   // the next load is the whole warp's
            }
        }
        if (!meet(1)) break;   // (both O's have been read, the marks and sums too)
        ++met;
    }
}

template <int KV, int D>
__global__ void __launch_bounds__(Tree<KV, D>::THREADS, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const TreeArgs a) {
    using X = Tree<KV, D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    TrCtrl &c = *reinterpret_cast<TrCtrl *>(smem + X::OFF_CTRL);
    static_assert(sizeof(TrCtrl) <= X::CTRL, "control block");
    const int warp = threadIdx.x >> 5;
    if ((smem_u32(smem) & 1023u) != 0) {   // tiles lie on 1024-byte boundaries (they do: nothing else is in shared memory)
        grid_wait();
        if (threadIdx.x == 0) a.status[blockIdx.x] = 1;
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < X::RING; ++s) {
            mbar_init(smem_u32(&c.full[s]), X::F8 ? X::CONV_WARPS : 1);
            mbar_init(smem_u32(&c.empty[s]), 1);
        }
        for (int s = 0; s < X::STAGES; ++s) {
            mbar_init(smem_u32(&c.stfull[s]), 1);
            mbar_init(smem_u32(&c.stempty[s]), X::CONV_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&c.qfull[b]), TR_SOFTMAX_WARPS);
            mbar_init(smem_u32(&c.qempty[b]), 1);
            for (int own = 0; own < 2; ++own) {
                mbar_init(smem_u32(&c.sfull[own][b]), 1);
                mbar_init(smem_u32(&c.pfull[own][b]), (own ? 1 : 2) * TR_HALF / 32);
                mbar_init(smem_u32(&c.pvdone[own][b]), 1);
            }
            mbar_init(smem_u32(&c.meet[b]), 2 * TR_HALF / 32);
        }
        mbar_init(smem_u32(&c.done), 1);
        c.abort = 0;
        fence_mbar_init();
        tma_prefetch_map(&tmk);
        tma_prefetch_map(&tmv);
    } else if (threadIdx.x >= 32 && threadIdx.x < 32 + TR_MARKS) {
        c.bad[threadIdx.x - 32] = 0;
        c.poison[(threadIdx.x - 32) / TR_SEEN][(threadIdx.x - 32) % TR_SEEN] = 0;
    }
    grid_wait();
    if (warp == 2) {   // (not before: an earlier kernel may still need its own)
        tmem_alloc(smem_u32(&c.tmem), TR_TMEM);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    make_plan(a, &c.plan, c.warp_sums);
    tc_fence_after_sync();
    const Plan plan = c.plan;
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&c.tmem);
    grid_release();   // the merge's CTAs may come as this kernel's leave (they wait for all of them)
    fill_idle_rows<D / 8>(a, plan, a.out, (long long)a.num_query_tokens * a.H,
                          X::MK == PA_KV_F16 ? 0x7e007e00u : 0x7fc07fc0u);
    if (plan.u0 < plan.u1) {   // the whole CTA has work, or none of it
        Walk<TreeArgs> p(a, plan);
        if (warp >= 4 && warp < 12) {
            regs_increase<X::REGS_HIGH>();
            tr_softmax<KV, D>(smem, c, a, p, tmem, (warp - 4) >> 2);
        } else if (warp >= 12) {
            if constexpr (X::F8) {
                regs_decrease<X::REGS_CONV>();
                tr_convert<KV, D>(smem, c, a, p, warp - 12);
            }
        } else {
            regs_decrease<X::REGS_LOW>();
            if (warp == 0 || warp == 3) {
                tr_load<KV, D>(c, a, p, smem_u32(smem), warp == 0 ? &tmk : &tmv, warp == 3);
            } else if (warp == 1) {
                tr_query<KV, D>(smem, c, a, p);
            } else if (warp == 2) {
                if (elect_one()) tr_mma<KV, D>(smem, c, a, p, tmem);
            }
            __syncwarp();
        }
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
    }
    if (warp == 2) tmem_dealloc(tmem, TR_TMEM);
    if (threadIdx.x == 0) a.status[blockIdx.x] = c.abort;
}

// Rows of the cut row tiles from their pieces' partial rows: blockIdx.x is the
// CTA whose range begins in the row tile; a warp takes 32 rows and eight of their
// dims, in the order in which the softmax left them.  When a CTA of the first
// kernel gave up, every row becomes NaN.
constexpr int TM_WARPS = 8;
static_assert(32 * TM_WARPS >= AXIS_MAX_CTAS, "a thread per CTA's status");

template <int KV, int D>
__global__ void __launch_bounds__(32 * TM_WARPS) tree_merge_kernel(const TreeArgs a, int ctas) {
    using X = Tree<KV, D>;
    constexpr int UNITS = D / 8;   // warps of 32 rows
    grid_release();
    grid_wait();
    const int cta = blockIdx.x, lane = threadIdx.x & 31;
    const int gave_up = threadIdx.x < ctas ? a.status[threadIdx.x] : 0;
    const Cut cut = a.cuts[cta];
    const int unit = blockIdx.y * TM_WARPS + (threadIdx.x >> 5), q = unit / UNITS;
    if (32 * (blockIdx.y * TM_WARPS / UNITS) >= cut.rows && (cta || blockIdx.y)) return;   // the whole block
    const bool failed = __syncthreads_or(gave_up);
    const uint32_t nan_pair = X::MK == PA_KV_F16 ? 0x7e007e00u : 0x7fc07fc0u;
    if (cta == 0 && blockIdx.y == 0) {
        if (threadIdx.x == 0) a.hdr->error = failed ? PA_ERR_TIMEOUT : PA_OK;
        if (failed) fill_rows(a.out, 0, (long long)a.num_query_tokens * a.H * (D / 8), nan_pair);
    }
    const int m = 32 * q + lane, k4 = unit % UNITS >> 2, j = 2 * (unit & 3);
    if (failed || m >= cut.rows || cut.pieces <= 1) return;
    float acc[8], l;
    join_pieces(
        cut.pieces, [&](int i) { return a.ml[(long long)piece_slot(cut, cta, i) * X::ROWS + m]; },
        [&](int i) { return a.o[partial_at<KV, D>(piece_slot(cut, cta, i), q, k4, j, lane)]; },
        [&](int i) { return a.o[partial_at<KV, D>(piece_slot(cut, cta, i), q, k4, j + 1, lane)]; }, acc, l);
    const float inv = a.v_scale / l;
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = (uint32_t)out_bits<X::MK>(acc[2 * i] * inv) | ((uint32_t)out_bits<X::MK>(acc[2 * i + 1] * inv) << 16);
    *reinterpret_cast<uint4 *>(a.out + (cut.row0 + a.row_at(m)) * D + 32 * k4 + 4 * j) = make_uint4(v[0], v[1], v[2], v[3]);
}

// ------------------------------------------------------------------ launch

struct TrLayout {
    size_t status, cuts, ml, o, total;
};

TrLayout tr_layout(int D) {
    TrLayout l;
    size_t at = 256;   // header
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at = (at + bytes + 255) / 256 * 256;
        return p;
    };
    l.status = take(sizeof(int) * AXIS_MAX_CTAS);
    l.cuts = take(sizeof(Cut) * AXIS_MAX_CTAS);
    l.ml = take(sizeof(float2) * 2 * AXIS_MAX_CTAS * TR_MAX_ROWS);
    l.o = take(sizeof(float) * 2 * AXIS_MAX_CTAS * TR_MAX_ROWS * (size_t)D);
    l.total = at;
    return l;
}

// A cache as [rows = num_blocks * Hkv * bs][D], boxes of 128 bytes by a block's rows.
bool block_map(CUtensorMap *map, const void *base, long long rows, int D, int bs, int kv) {
    auto enc = tma_encoder();
    if (!enc) return false;
    const bool fp8 = kv == PA_KV_FP8_E4M3;
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)D * (fp8 ? 1 : 2)};
    cuuint32_t box[2] = {fp8 ? 128u : 64u, (cuuint32_t)bs};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                        : kv == PA_KV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
               2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared-memory limits are set per device, on its first call; the kernel runs
// only if it was built with the registers that its split assumes (with another
// count the softmax warps' increase could wait forever).
template <int KV, int D>
int tr_setup() {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64 && done[dev]) return PA_OK;
    cudaFuncAttributes fa;
    if (cudaFuncSetAttribute(tree_kernel<KV, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tree<KV, D>::SMEM) !=
            cudaSuccess ||
        cudaFuncGetAttributes(&fa, tree_kernel<KV, D>) != cudaSuccess)
        return PA_ERR_CUDA;
    if (fa.numRegs != Tree<KV, D>::REGS_LAUNCH) return PA_ERR_UNSUPPORTED;
    if (dev < 64) done[dev] = true;
    return PA_OK;
}

template <int KV, int D>
int launch_tree(TreeArgs a, const void *k_cache, const void *v_cache, cudaStream_t st) {
    using X = Tree<KV, D>;
    if (const int e = tr_setup<KV, D>()) return e;
    const long long rows = a.num_blocks * a.Hkv * a.bs;
    CUtensorMap tmk, tmv;
    if (!block_map(&tmk, k_cache, rows, D, a.bs, KV) || !block_map(&tmv, v_cache, rows, D, a.bs, KV)) return PA_ERR_CUDA;
    a.tile_toks = X::ROWS / a.G;
    a.tinv = (1 << 20) / a.tile_toks + 1;
    const int ctas = std::min(num_sms(), AXIS_MAX_CTAS);
    if (const int e = launch_early(tree_kernel<KV, D>, dim3((unsigned)ctas), X::THREADS, X::SMEM, st, tmk, tmv, a))
        return e;
    const long long most = std::min<long long>(X::ROWS, (long long)a.num_query_tokens * a.G);
    const dim3 grid((unsigned)ctas, (unsigned)((most + 31) / 32 * (D / 8) / TM_WARPS));
    return launch_early(tree_merge_kernel<KV, D>, grid, 32 * TM_WARPS, 0, st, a, ctas);
}

// PA_DEBUG_VALIDATE: lengths, row offsets, block ids and parents.
int validate_tree(const TreeArgs &a, cudaStream_t st) try {
    if (const int e = validate_starts(a.query_start, a.num_seqs, a.num_query_tokens, true, st)) return e;
    const size_t n = (size_t)a.num_seqs;
    std::vector<int32_t> lens(n), qs(n + 1), parents((size_t)a.num_query_tokens);
    std::vector<int64_t> last(n);
    if (const int e = copy_to_host(lens.data(), a.context_lens, 4 * n, st)) return e;
    if (const int e = copy_to_host(qs.data(), a.query_start, 4 * (n + 1), st)) return e;
    if (const int e = copy_to_host(parents.data(), a.parents, 4 * parents.size(), st)) return e;
    for (size_t i = 0; i < n; ++i) {
        const int T = qs[i + 1] - qs[i];
        if (lens[i] < 0 || lens[i] > a.max_ctx || T > lens[i] || T > PA_TREE_MAX_NODES) return PA_ERR_INVALID_ARG;
        for (int j = 0; j < T; ++j)
            if (parents[(size_t)(qs[i] + j)] < -1 || parents[(size_t)(qs[i] + j)] >= j) return PA_ERR_INVALID_ARG;
        last[i] = lens[i];
    }
    return validate_tables(a.block_tables, last.data(), a.num_seqs, a.mbps, a.bs, a.num_blocks, st);
} catch (...) {   // no host memory for the check
    return PA_ERR_STATE;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_attention_tree_workspace_size(int num_seqs, int num_query_tokens, int num_heads, int num_kv_heads,
                                                   int head_dim, int max_context_len) {
    if (num_seqs < 0 || num_query_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        num_heads % num_kv_heads != 0 || head_dim <= 0 || max_context_len < 0)
        return 0;
    return tr_layout(head_dim).total;
}

extern "C" int pa_attention_tree(void *out, const void *query, const void *k_cache, const void *v_cache,
                                 const int32_t *block_tables, const int32_t *context_lens, const int32_t *query_start,
                                 const int32_t *parents, int num_seqs, int num_query_tokens, int num_heads,
                                 int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                                 int max_blocks_per_seq, int max_context_len, float scale, int kv_dtype, float k_scale,
                                 float v_scale, void *workspace, size_t workspace_bytes, void *stream) {
    if (num_seqs < 0 || num_query_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        num_heads % num_kv_heads != 0 || max_context_len < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
        !std::isfinite(scale) || !(scale > 0.f))
        return PA_ERR_INVALID_ARG;
    const int G = num_heads / num_kv_heads;
    const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
    if (!fp8 && kv_dtype != PA_KV_F16 && kv_dtype != PA_KV_BF16) return PA_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || (block_size != 8 && block_size != 16 && block_size != 32) || G > 16)
        return PA_ERR_UNSUPPORTED;
    if (fp8) {
        if (!std::isfinite(k_scale) || !(k_scale > 0.f) || !std::isfinite(v_scale) || !(v_scale > 0.f))
            return PA_ERR_INVALID_ARG;
        if (head_dim != 128) return PA_ERR_UNSUPPORTED;
    }
    if (num_query_tokens == 0) return PA_OK;
    if (num_seqs == 0) return PA_ERR_INVALID_ARG;
    if (!out || !query || !k_cache || !v_cache || !block_tables || !context_lens || !query_start || !parents)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache))
        return PA_ERR_INVALID_ARG;
    if ((long long)num_blocks * num_kv_heads * block_size >= (1LL << 31) ||
        (long long)num_query_tokens * num_heads >= (1LL << 31))
        return PA_ERR_UNSUPPORTED;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < pa_attention_tree_workspace_size(num_seqs, num_query_tokens, num_heads, num_kv_heads,
                                                           head_dim, max_context_len))
        return PA_ERR_WORKSPACE;
    TreeArgs a{};
    a.out = static_cast<uint16_t *>(out);
    a.query = static_cast<const uint16_t *>(query);
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.parents = parents;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const TrLayout lay = tr_layout(head_dim);
    a.hdr = reinterpret_cast<WsHeader *>(ws);
    a.status = reinterpret_cast<int *>(ws + lay.status);
    a.cuts = reinterpret_cast<Cut *>(ws + lay.cuts);
    a.ml = reinterpret_cast<float2 *>(ws + lay.ml);
    a.o = reinterpret_cast<float4 *>(ws + lay.o);
    a.num_seqs = num_seqs;
    a.num_query_tokens = num_query_tokens;
    a.H = num_heads;
    a.Hkv = num_kv_heads;
    a.G = G;
    a.ginv = 65536 / G + 1;
    a.wait_limit = pipeline_wait_limit();
    a.bs = block_size;
    a.mbps = max_blocks_per_seq;
    a.max_ctx = max_context_len;
    a.num_blocks = num_blocks;
    a.scale_log2 = scale * (fp8 ? k_scale : 1.f) * 1.4426950408889634f;
    a.v_scale = fp8 ? v_scale : 1.f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug_validate())
        if (const int e = validate_tree(a, st)) return e;
    if (fp8) return launch_tree<PA_KV_FP8_E4M3, 128>(a, k_cache, v_cache, st);
    if (kv_dtype == PA_KV_BF16)
        return head_dim == 128 ? launch_tree<PA_KV_BF16, 128>(a, k_cache, v_cache, st) : launch_tree<PA_KV_BF16, 64>(a, k_cache, v_cache, st);
    return head_dim == 128 ? launch_tree<PA_KV_F16, 128>(a, k_cache, v_cache, st) : launch_tree<PA_KV_F16, 64>(a, k_cache, v_cache, st);
}
