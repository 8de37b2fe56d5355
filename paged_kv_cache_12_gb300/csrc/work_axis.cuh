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
//   row_tile_at(w, u, team) the last of those that start at or before unit u
//   row_tiles(w, r)         KV tiles of row tile r
//   seq_ok(i), ends_ok()    whether sequence i's row offsets are in order, and
//                           all of them a cover of the rows
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
constexpr int AXIS_MIN_UNITS = 2;    // units of a range, at least (600 tokens, 16 heads, absorbed: 13.0 us with 1, 12.4
                                     // with 2, 14.1 with 3; expanded 24.3, 24.3 and 25.6)

struct Plan {
    long long u0, u1, base;   // this CTA's range; first unit of sequence seq
    long long total;          // units of the axis (0 too if the row offsets are out of order)
    int seq, j;               // the sequence in which the range begins, and its row tile (numbered as the axis has them)
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

// a / b for a, b >= 0: a 64-bit division takes several times a 32-bit one's time,
// and the plan is most of a short call's start.
__device__ __forceinline__ long long quick_div(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (uint32_t)a / (uint32_t)b : a / b;
}

// First unit of team k's range; `parts` teams have one, of AXIS_MIN_UNITS units each
// at least.
__device__ __forceinline__ long long range_begin(long long total, int k, int parts) { return quick_div(total * k, parts); }

// The first team whose range begins at unit u > 0 or later (`parts` if there is none).
__device__ __forceinline__ int team_from(long long total, long long u, int parts) {
    return (int)quick_div(u * parts + total - 1, total);
}

// This block's plan (warp_sums: one number per warp, in shared memory).
template <class P>
__device__ __forceinline__ void make_plan(const P &a, Plan *plan, long long *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int per = (a.num_seqs + blockDim.x - 1) / blockDim.x;
    const int i0 = min(a.num_seqs, (int)threadIdx.x * per), i1 = min(a.num_seqs, i0 + per);
    bool in_order = a.ends_ok(), pairs = true;
    long long one = 0, two = 0;   // units without teams and in teams
    for (int i = i0; i < i1; ++i) {
        const typename P::Seq w = a.seq_work(i);
        in_order = in_order && a.seq_ok(i);
        pairs = pairs && a.in_teams(w);
        one += a.start(w, w.rts, 1);
        if (pairs) two += a.start(w, w.rts / 2, 2);
    }
    const bool ok = __syncthreads_and(in_order);
    const int team = __syncthreads_and(pairs) ? 2 : 1;
    auto units = [&](int i) {
        const typename P::Seq w = a.seq_work(i);
        return a.start(w, w.rts / team, team);
    };
    const long long mine = !ok ? 0 : team == 2 ? two : one;
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
    const int cta = blockIdx.x, k = cta / team;
    const long long most = min(total, max(1LL, quick_div(total, AXIS_MIN_UNITS)));   // teams with work
    const int parts = (int)min((long long)(gridDim.x / team), most);
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
            plan->j = 0;
        }
    }
    if (u0 < u1 && begin <= u0 && u0 < end) {   // one thread
        long long s = begin;
        int i = i0;
        for (; i + 1 < i1; ++i) {
            const long long n = units(i);
            if (u0 < s + n) break;
            s += n;
        }
        plan->seq = i;
        plan->base = s;
        // the row tile in which the range begins: cut here if a KV tile of it lies on either side
        const typename P::Seq w = a.seq_work(i);
        const int j = a.row_tile_at(w, u0 - s, team), r = j * team + cta % team;
        plan->j = j;
        const long long at = s + a.start(w, j, team), first = at + P::COST;
        const int ntiles = a.row_tiles(w, r);
        Cut cut{};
        if (k > 0 && first < u0 && u0 < first + ntiles && range_begin(total, k - 1, parts) <= first) {
            // of the row tile's first `tiles` KV tiles: the teams from k - 1 on whose ranges begin before their end
            auto pieces = [&](int tiles) { return max(1, team_from(total, first + tiles, parts) - (k - 1)); };
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

    __device__ Walk(const P &args, const Plan &p) : a(args), u0(p.u0), u1(p.u1), base(p.base), team(p.team), seq(p.seq), j(p.j - 1) {
        local = -1;
        if (u0 < u1) w = a.seq_work(seq);
    }
    // The next piece; false at the end of the range.
    __device__ bool next() {
        if (u0 >= u1) return false;
        for (;;) {
            ++j;
            while (j >= w.rts >> (team - 1)) {   // on to the next sequence
                base += a.start(w, w.rts >> (team - 1), team);
                if (base >= u1 || ++seq >= a.num_seqs) return false;
                w = a.seq_work(seq);
                j = 0;
            }
            s = base + a.start(w, j, team);
            if (s >= u1) return false;
            r = j * team + ((int)blockIdx.x & (team - 1));
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

// Joins a cut row tile's pieces for one row and eight of its dims: piece i has the
// maximum (log2 units) and sum ml(i) and the unnormalised x(i), y(i).  Four pieces
// at a time, so that their loads are on their way together.
template <class ML, class X, class Y>
__device__ __forceinline__ void join_pieces(int pieces, ML ml, X x, Y y, float (&acc)[8], float &l) {
    constexpr int N = 4;
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    l = 0.f;
    for (int i0 = 0; i0 < pieces; i0 += N) {
        float2 s[N];
        float4 v[N], w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i0 + i < pieces) {
                s[i] = ml(i0 + i), v[i] = x(i0 + i), w[i] = y(i0 + i);
            } else {
                s[i] = make_float2(-INFINITY, 0.f), v[i] = w[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        float m = M;
#pragma unroll
        for (int i = 0; i < N; ++i) m = fmaxf(m, s[i].x);
        const float mu = m == -INFINITY ? 0.f : m;   // nothing seen yet
        const float old = fast_exp2(M - mu);
        l *= old;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] *= old;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float wt = fast_exp2(s[i].x - mu);
            const float o[8] = {v[i].x, v[i].y, v[i].z, v[i].w, w[i].x, w[i].y, w[i].z, w[i].w};
            l = fmaf(s[i].y, wt, l);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = fmaf(o[k], wt, acc[k]);
        }
        M = m;
    }
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
