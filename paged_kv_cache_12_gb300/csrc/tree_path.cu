// Move of a verified path: K and V of the nodes that stand, from their positions
// in the tree to the ones that follow the context.
//
// The path rises (path[j] >= j, strictly), so row j's destination never lies
// behind the source of a later row: moved in order of j, every row is read before
// it is overwritten.  A thread moves the same 16 bytes of every row of one
// (layer, kv head, K or V) of a sequence, so that order is the thread's own and
// nothing has to be waited for.  One GB300: 64 sequences, up to eight rows of 128 bytes in
// each of 8 heads of 32 layers, 9.0 us (16.8 MB read and as much written, in pieces of
// 128 bytes); one layer of eight sequences 3.9 us, the launch.
//
// Sources: tokens are found through the block table ("PagedAttention de vLLM :
// comment la gestion de la VRAM soutient l'inference des grands modeles",
// deepsonar.com.cn, section 2.2); trees of drafted tokens are not on the pages.

#include <algorithm>
#include <climits>
#include <vector>

#include "common.cuh"

namespace pa {
namespace {

constexpr int MOVE_THREADS = 128;
constexpr int MOVE_BATCH = 4;   // rows on their way at once (64 x 8 rows of 32 layers: 9.0 us, with eight 9.6)

struct MoveArgs {
    uint8_t *k_cache, *v_cache;
    const int32_t *block_tables, *context_lens, *query_start, *path, *accepted;
    int num_seqs, max_depth, layers, hk, row_bytes, block_size, mbps;
    long long num_blocks;
};

// The slot of a sequence's position, or -1.
__device__ __forceinline__ long long slot_of(const MoveArgs &a, int seq, int pos) {
    const int b = pos / a.block_size;
    const long long blk = a.block_tables[(long long)seq * a.mbps + b];
    return blk < 0 || blk >= a.num_blocks ? -1 : blk * a.block_size + (pos - b * a.block_size);
}

// blockIdx.x = sequence; a thread per 16 bytes of (layer, K or V, kv head) over
// blockIdx.y.
__global__ void __launch_bounds__(MOVE_THREADS) move_path_kernel(const MoveArgs a) {
    __shared__ long long src[PA_TREE_MAX_NODES], dst[PA_TREE_MAX_NODES];
    const int seq = blockIdx.x;
    grid_release();
    grid_wait();
    const int32_t *path = a.path + (long long)seq * (a.max_depth + 1);
    const int first = threadIdx.x, here = first <= a.max_depth ? path[first] : 0;   // (read beside what it depends on)
    const int before = first > 0 && first <= a.max_depth ? path[first - 1] : -1;
    const int n = a.accepted[seq];
    const int q0 = a.query_start[seq], q1 = a.query_start[seq + 1], L = a.context_lens[seq];
    const int T = q0 >= 0 && q1 > q0 ? q1 - q0 : 0;   // (offsets of other signs may lie further apart than an int holds)
    bool ok = n >= 0 && n <= a.max_depth && T > 0 && T <= PA_TREE_MAX_NODES && n < T && T <= L &&
              L <= (long long)a.mbps * a.block_size;
    if (ok) {
        for (int j = first; j <= n; j += MOVE_THREADS) {
            const int p = j == first ? here : path[j];
            if (j == 0 ? p != 0 : p <= (j == first ? before : path[j - 1])) ok = false;
            if (p < 0 || p >= T) {
                ok = false;
                continue;
            }
            src[j] = slot_of(a, seq, L - T + p);
            dst[j] = slot_of(a, seq, L - T + j);
            if (src[j] < 0 || dst[j] < 0) ok = false;
        }
    }
    if (!__syncthreads_and(ok)) return;
    const int vecs = a.row_bytes / 16;
    const long long per_cache = (long long)a.layers * a.hk * vecs, head_rows = a.block_size;
    for (long long i = blockIdx.y * (long long)MOVE_THREADS + threadIdx.x; i < 2 * per_cache;
         i += (long long)gridDim.y * MOVE_THREADS) {
        const bool v = i >= per_cache;
        const long long k = v ? i - per_cache : i, lh = k / vecs;
        const int vec = (int)(k - lh * vecs);
        const long long layer = lh / a.hk;
        const int h = (int)(lh - layer * a.hk);
        uint4 *base = reinterpret_cast<uint4 *>(v ? a.v_cache : a.k_cache) +
                      layer * a.num_blocks * a.hk * head_rows * vecs + vec;
        auto at = [&](long long slot) {
            const long long blk = slot / a.block_size, off = slot - blk * a.block_size;
            return base + ((blk * a.hk + h) * head_rows + off) * vecs;
        };
        for (int j0 = 1; j0 <= n; j0 += MOVE_BATCH) {
            uint4 x[MOVE_BATCH];
#pragma unroll
            for (int u = 0; u < MOVE_BATCH; ++u)
                if (j0 + u <= n && src[j0 + u] != dst[j0 + u]) x[u] = *at(src[j0 + u]);
#pragma unroll
            for (int u = 0; u < MOVE_BATCH; ++u)
                if (j0 + u <= n && src[j0 + u] != dst[j0 + u]) *at(dst[j0 + u]) = x[u];
        }
    }
}

// PA_DEBUG_VALIDATE: what the kernel checks, as an error.
int validate_move(const MoveArgs &a, cudaStream_t st) try {
    if (const int e = validate_starts(a.query_start, a.num_seqs, INT_MAX, false, st)) return e;
    const size_t n = (size_t)a.num_seqs, w = (size_t)a.max_depth + 1;
    std::vector<int32_t> lens(n), qs(n + 1), acc(n), path(n * w);
    std::vector<int64_t> last(n);
    if (const int e = copy_to_host(lens.data(), a.context_lens, 4 * n, st)) return e;
    if (const int e = copy_to_host(qs.data(), a.query_start, 4 * (n + 1), st)) return e;
    if (const int e = copy_to_host(acc.data(), a.accepted, 4 * n, st)) return e;
    if (const int e = copy_to_host(path.data(), a.path, 4 * n * w, st)) return e;
    for (size_t i = 0; i < n; ++i) {
        const int T = qs[i + 1] - qs[i];
        if (T == 0 && acc[i] == -1) continue;
        if (acc[i] < 0 || acc[i] > a.max_depth || T > PA_TREE_MAX_NODES || acc[i] >= T || T > lens[i])
            return PA_ERR_INVALID_ARG;
        for (int j = 0; j <= acc[i]; ++j) {
            const int p = path[i * w + (size_t)j];
            if (p >= T || (j == 0 ? p != 0 : p <= path[i * w + (size_t)j - 1])) return PA_ERR_INVALID_ARG;
        }
        last[i] = lens[i];
    }
    return validate_tables(a.block_tables, last.data(), a.num_seqs, a.mbps, a.block_size, a.num_blocks, st);
} catch (...) {   // no host memory for the check
    return PA_ERR_STATE;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_kv_move_path(void *k_cache, void *v_cache, const int32_t *block_tables, const int32_t *context_lens,
                               const int32_t *query_start, const int32_t *path, const int32_t *accepted, int num_seqs,
                               int max_depth, int num_layers, int num_kv_heads, int head_dim, int block_size,
                               int64_t num_blocks, int max_blocks_per_seq, int kv_dtype, void *stream) {
    const bool fp8 = kv_dtype == PA_KV_FP8_E4M3;
    if (num_seqs < 0 || max_depth < 0 || num_layers <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || head_dim % (fp8 ? 16 : 8) != 0 || block_size <= 0 || num_blocks <= 0 ||
        max_blocks_per_seq <= 0 || (!fp8 && kv_dtype != PA_KV_F16 && kv_dtype != PA_KV_BF16))
        return PA_ERR_INVALID_ARG;
    // a path's entries and a row's bytes are counted in 32 bits
    if (max_depth > (1 << 30) || head_dim > (1 << 29)) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || max_depth == 0) return PA_OK;   // only node 0 can stand: it is in its place
    if (!k_cache || !v_cache || !block_tables || !context_lens || !query_start || !path || !accepted ||
        !aligned16(k_cache) || !aligned16(v_cache))
        return PA_ERR_INVALID_ARG;
    MoveArgs a{};
    a.k_cache = static_cast<uint8_t *>(k_cache);
    a.v_cache = static_cast<uint8_t *>(v_cache);
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.path = path;
    a.accepted = accepted;
    a.num_seqs = num_seqs;
    a.max_depth = max_depth;
    a.layers = num_layers;
    a.hk = num_kv_heads;
    a.row_bytes = head_dim * (fp8 ? 1 : 2);
    a.block_size = block_size;
    a.mbps = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (debug_validate())
        if (const int e = validate_move(a, st)) return e;
    const long long vecs = 2LL * num_layers * num_kv_heads * (a.row_bytes / 16);
    const unsigned gy = (unsigned)std::min<long long>((vecs + MOVE_THREADS - 1) / MOVE_THREADS, 65535);
    return launch_early(move_path_kernel, dim3((unsigned)num_seqs, gy), MOVE_THREADS, 0, st, a);
}
