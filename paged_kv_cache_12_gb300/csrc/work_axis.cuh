// Work shared out evenly over the CTAs of one launch, without a plan made on
// the host or in a launch of its own.
//
// The work of an attention call is a list of row tiles (some query rows of one
// sequence and the KV tiles that they see).  Laid end to end they make one axis
// of work units, a unit being a KV tile; each row tile has COST units more for
// its start and its end.  The axis is cut into equal ranges, one per CTA, and a
// CTA takes the pieces of row tiles inside its range.  A row tile that lies in
// one range is finished there; the pieces of a cut one leave partial rows (at
// most two pieces a CTA: one continued from the left, one to the right), which
// a second kernel merges.  Every CTA derives the cut by itself from the lengths,
// by one sum over the sequences.
//
// Where every sequence has an even number of row tiles over (nearly) the same KV
// tiles, the CTAs work in teams of two: a team takes a range of the axis of every
// second row tile, and its two CTAs a row tile each of the pairs in it, so that
// they read the same KV tiles at the same time (the second read comes from L2; one
// CTA after the other, both came from HBM).
//
// A problem P gives
//   P::COST                 units of a row tile besides its KV tiles
//   in_teams(w)             whether teams of two suit the sequence
//   P::Seq, seq_work(i)     what is needed of sequence i; Seq::rts row tiles
//   start(w, j, team)       first unit, within its sequence, of the j-th row tile
//                           of a team's axis (row tile j * team + member);
//                           start(w, w.rts / team, team) = the sequence's units
//   row_tiles(w, r)         KV tiles of row tile r
//   starts_ok()             whether the row offsets are in order (called by
//                           every thread of the block)
//   num_seqs, cuts          sequences; [AXIS_MAX_CTAS] what a cut row tile's merge
//                           needs, written by the CTA whose range begins in it
//   cut_rows(w, r)          rows of a row tile
//   first_row(w, r)         its first row in the output
//   first_tiles(w, r)       KV tiles that its first rows see (where the merge
//                           treats a row tile's rows alike: row_tiles)
#pragma once

#include <stdint.h>

namespace pa {
namespace {

constexpr int AXIS_MAX_CTAS = 160;   // CTAs of a launch: one per SM, at most this many

struct Plan {
    long long u0, u1, base;   // this CTA's range; first unit of sequence seq
    long long total;          // units of the axis (0 too if the row offsets are out of order)
    int seq;                  // the sequence in which the range begins
    int team;                 // CTAs of a team
    int ok;                   // the row offsets are in order
};

// A row tile whose first two pieces are the CTA's own and that of the CTA before
// it (a team before it), in cuts[CTA]: all that the merge needs of it.  rows = 0
// where there is none (the range begins with a row tile, or in one that an earlier
// range cuts as well).
struct Cut {
    long long row0;     // its first row in the output
    int rows;
    int pieces;         // its pieces, in consecutive teams from the one before on
    int pieces1;        // those that its first rows have tiles in (see first_tiles)
    int first, step;    // slots of their partial rows: first, then 2 CTA, 2 CTA + step, ..
    int pad;
};

// First unit of team k's range; `parts` = min(teams, total) teams have one, of at
// least a unit each.
__device__ __forceinline__ long long range_begin(long long total, int k, int parts) { return total * k / parts; }

// Whether the n + 1 device offsets are a non-decreasing cover of [0, end):
// every thread of the block calls it and gets the answer.
__device__ __forceinline__ bool offsets_ok(const int32_t *start, int n, int end) {
    bool ok = start[0] == 0 && start[n] == end;
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if (start[i] > start[i + 1]) ok = false;
    return __syncthreads_and(ok);
}

// The last of n sequences that starts at or before row `row`.
__device__ __forceinline__ int sequence_of(const int32_t *start, int n, int row) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= row) lo = mid; else hi = mid;
    }
    return lo;
}

// The last of a team's row tiles (numbered as the axis has them) that starts at
// or before unit u of the sequence.
template <class P>
__device__ __forceinline__ int row_tile_at(const P &a, const typename P::Seq &w, int team, long long u) {
    int r = 0, hi = w.rts / team;
    while (hi - r > 1) {
        const int mid = (r + hi) >> 1;
        if (a.start(w, mid, team) <= u) r = mid; else hi = mid;
    }
    return r;
}

// This block's plan (warp_sums: one number per warp, in shared memory).
template <class P>
__device__ __forceinline__ void make_plan(const P &a, Plan *plan, long long *warp_sums) {
    const bool ok = a.starts_ok();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int per = (a.num_seqs + blockDim.x - 1) / blockDim.x;
    const int i0 = min(a.num_seqs, (int)threadIdx.x * per), i1 = min(a.num_seqs, i0 + per);
    bool pairs = true;
    for (int i = i0; ok && i < i1; ++i) pairs = pairs && a.in_teams(a.seq_work(i));
    const int team = __syncthreads_and(pairs) ? 2 : 1;
    auto units = [&](int i) {
        const typename P::Seq w = a.seq_work(i);
        return a.start(w, w.rts / team, team);
    };
    long long mine = 0;
    for (int i = i0; ok && i < i1; ++i) mine += units(i);
    long long upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += x;
    }
    if (lane == 31) warp_sums[warp] = upto;
    __syncthreads();
    long long before = 0, total = 0;
    for (int j = 0; j < nwarps; ++j) {
        if (j < warp) before += warp_sums[j];
        total += warp_sums[j];
    }
    const long long begin = before + upto - mine, end = before + upto;
    const int parts = (int)min((long long)(gridDim.x / team), total), cta = blockIdx.x, k = cta / team;
    const long long u0 = k < parts ? range_begin(total, k, parts) : 0;
    const long long u1 = k < parts ? range_begin(total, k + 1, parts) : 0;
    if (threadIdx.x == 0) {
        plan->u0 = u0;
        plan->u1 = u1;
        plan->total = total;
        plan->team = team;
        plan->ok = ok;
        if (u0 >= u1) {
            a.cuts[cta].rows = 0;
            plan->seq = a.num_seqs;
        }
    }
    if (u0 < u1 && begin <= u0 && u0 < end) {   // one thread
        long long s = begin;
        int i = i0;
        for (;; ++i) {
            const long long n = units(i);
            if (u0 < s + n) break;
            s += n;
        }
        plan->seq = i;
        plan->base = s;
        // the row tile in which the range begins: cut here if a KV tile of it lies on either side
        const typename P::Seq w = a.seq_work(i);
        const int j = row_tile_at(a, w, team, u0 - s), r = j * team + cta % team;
        const long long at = s + a.start(w, j, team), first = at + P::COST;
        const int ntiles = a.row_tiles(w, r);
        Cut cut{};
        if (k > 0 && first < u0 && u0 < first + ntiles && range_begin(total, k - 1, parts) <= first) {
            auto pieces = [&](int tiles) {   // of the row tile's first `tiles` KV tiles
                int n = 1;
                while (range_begin(total, k - 1 + n, parts) < first + tiles) ++n;
                return n;
            };
            cut.row0 = a.first_row(w, r);
            cut.rows = a.cut_rows(w, r);
            cut.pieces = pieces(ntiles);
            cut.pieces1 = pieces(a.first_tiles(w, r));
            cut.first = 2 * (cta - team) + (at < range_begin(total, k - 1, parts) ? 0 : 1);
            cut.step = 2 * team;
        }
        a.cuts[cta] = cut;
    }
    __syncthreads();
}

// Walks the pieces of a CTA's range, in every role alike.
template <class P>
struct Walk {
    const P &a;
    long long u0, u1, base, s;   // the range; first unit of the sequence, and of row tile r
    int team, seq, j, r;         // row tile r is the j-th of the team's axis
    typename P::Seq w;
    int t0, t1, ntiles, local;   // the piece: KV tiles [t0, t1) of ntiles; its number in this CTA

    __device__ Walk(const P &args, const Plan &p) : a(args), u0(p.u0), u1(p.u1), base(p.base), team(p.team), seq(p.seq), j(0) {
        local = -1;
        if (u0 >= u1) return;
        w = a.seq_work(seq);
        j = row_tile_at(a, w, team, u0 - base) - 1;
    }
    // The next piece; false at the end of the range.
    __device__ bool next() {
        if (u0 >= u1) return false;
        for (;;) {
            ++j;
            while (j >= w.rts / team) {   // on to the next sequence
                base += a.start(w, w.rts / team, team);
                if (base >= u1 || ++seq >= a.num_seqs) return false;
                w = a.seq_work(seq);
                j = 0;
            }
            s = base + a.start(w, j, team);
            if (s >= u1) return false;
            r = j * team + (int)blockIdx.x % team;
            ntiles = a.row_tiles(w, r);
            t0 = (int)max(0LL, min((long long)ntiles, u0 - s - P::COST));
            t1 = (int)max(0LL, min((long long)ntiles, u1 - s - P::COST));
            if (t1 > t0) {
                ++local;
                return true;
            }
        }
    }
    __device__ bool whole() const { return t0 == 0 && t1 == ntiles; }
    // slot of this piece's partial rows: 0 if the row tile began before the range
    __device__ int slot() const { return 2 * (int)blockIdx.x + (s < u0 ? 0 : 1); }
};

// The slot of a cut row tile's i-th piece (it began before every later piece's range).
__device__ __forceinline__ int piece_slot(const Cut &cut, int cta, int i) {
    return i ? 2 * cta + (i - 1) * cut.step : cut.first;
}

// Whether a CTA of the first kernel gave up (called by the whole block).
__device__ __forceinline__ bool any_gave_up(const int *status, int ctas) {
    int failed = 0;
    for (int i = threadIdx.x; i < ctas; i += blockDim.x) failed |= status[i];
    return __syncthreads_or(failed);
}

// The block writes `bits` to 16-byte vectors [from, to) of out.
__device__ __forceinline__ void fill_rows(uint16_t *out, long long from, long long to, uint32_t bits) {
    uint4 *o = reinterpret_cast<uint4 *>(out);
    for (long long i = from + threadIdx.x; i < to; i += blockDim.x) o[i] = make_uint4(bits, bits, bits, bits);
}

// Rows that no KV tile makes: zeros for an empty context, NaN for an invalid
// sequence, and NaN for every row when the row offsets are out of order.  Each
// CTA takes every gridDim-th sequence.  VEC: 16-byte vectors of an output row.
template <int VEC, class P>
__device__ __forceinline__ void fill_idle_rows(const P &a, const Plan &plan, uint16_t *out, long long all_rows,
                                               uint32_t nan_pair) {
    if (!plan.ok) {
        const long long n = all_rows * VEC;
        fill_rows(out, range_begin(n, blockIdx.x, gridDim.x), range_begin(n, blockIdx.x + 1, gridDim.x), nan_pair);
        return;
    }
    for (int i = blockIdx.x; i < a.num_seqs; i += gridDim.x) {
        const typename P::Seq w = a.seq_work(i);
        if (w.rts == 0 && w.T > 0)
            fill_rows(out, (long long)w.q0 * a.H * VEC, ((long long)w.q0 + w.T) * a.H * VEC, w.valid ? 0u : nan_pair);
    }
}

}  // namespace
}  // namespace pa
