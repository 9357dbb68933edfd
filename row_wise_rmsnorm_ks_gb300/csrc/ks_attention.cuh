// What the paged-attention kernels share: the call's shape, the division of its work over CTAs,
// which query row a tile's row is, and the join of split rows.
//
// Division of the work. The queries of one sequence and one key/value head (all heads of its
// group, token after token) are cut into row tiles of at most M rows, and the keys a row tile sees
// into units of TN keys. A row tile costs its units and a few more for its beginning and end
// (tile_cost). All cost of a call, in the order sequence, head, row tile, unit, is shared out evenly:
// CTA c of G takes [U c / G, U (c + 1) / G), G no more than U. A row tile whose units fall to several
// CTAs is split over its long axis; each of them leaves its running maximum, sum and unnormalised
// output in the workspace and a second kernel joins them in a fixed order, so results do not depend
// on timing. The lengths are read on the device: the launch depends on host-known
// sizes only, and a captured graph may be replayed with other lengths.
#pragma once

#include "ks_decode.cuh"

namespace ks {

struct AttnArgs {
    ks_attention_args_t a;
    int32_t group;       // query heads per key/value head
    int32_t tile_heads;  // heads of a group in a row tile
    int32_t head_splits; // row tiles a token's group is cut into (1 unless group > M)
    int32_t tile_tokens; // tokens in a row tile
    int32_t unit_shift;  // log2 of the keys per unit (TN)
    int32_t rows;        // rows of a tile (M)
    int32_t tile_cost;   // units that a row tile costs beside its own
    float scale_log2;    // scale * log2(e)
};

// What a CTA left in its second partial slot: the beginning of a row tile that later CTAs finish.
struct AttnJoin {
    int32_t pieces;      // 0: nothing to join
    int32_t seq, head, row_tile;
    int32_t q0, q_len;
    int32_t pad[2];
};

constexpr int kJoinThreads = 128;
constexpr int kMaxKeys = 0x7ffffc00;  // keys of a sequence: indices a few steps behind them still fit 31 bits
constexpr int kMaxTokens = 0x7ffffc00;  // the same for a row tile's rows behind the last token
constexpr int kMaxSeqs = 1 << 30;       // and for the last thread's share of the sequences

// A sequence's new tokens [q0, q0 + n) and key count, brought into range (and reported) where the
// given indices are not: nothing outside the tensors is ever addressed.
struct AttnSeq {
    int32_t q0, n, keys;
};

__device__ __forceinline__ AttnSeq attn_seq(const ks_attention_args_t &a, int b) {
    const int64_t tokens = a.tokens, room = min(a.table_pages * a.page_size, (int64_t)kMaxKeys);
    const int32_t q0 = a.q_starts[b], q1 = a.q_starts[b + 1], keys = a.kv_lens[b];
    AttnSeq s;
    s.q0 = (int32_t)min(max((int64_t)q0, (int64_t)0), tokens);
    const int32_t end = (int32_t)min(max((int64_t)q1, (int64_t)s.q0), tokens);
    s.n = end - s.q0;
    s.keys = (int32_t)min(max((int64_t)keys, (int64_t)0), room);
    if (s.q0 != q0 || end != q1 || s.keys != keys) atomicOr(&g_fault_flags, kFaultBadIndex);
    return s;
}

// a / b for a, b >= 0: by 32 bits where they fit (a fifth of the time of the 64-bit routine).
__device__ inline int64_t quotient(int64_t a, int64_t b) {
    if (((uint64_t)a | (uint64_t)b) >> 32 == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// sum over i in [0, n) of floor((a i + b) / 2^shift), for a n + b below 2^32: the whole multiples of the
// divisor in a and b sum in closed form; for what is left, the points under the line are counted along
// the other axis, which is the same sum with a and the divisor changed over.
__device__ inline int64_t floor_sum(uint32_t n, int shift, uint32_t a, uint32_t b) {
    uint32_t m = 1u << shift;
    int64_t total = (int64_t)(a >> shift) * ((int64_t)n * (n - 1) / 2) + (int64_t)(b >> shift) * n;
    a &= m - 1;
    b &= m - 1;
    uint32_t top = a * n + b;  // m times the line's height at n
    if (top < m) return total;
    n = top >> shift;
    b = top & (m - 1);
    while (true) {
        const uint32_t t = a;  // axes changed over
        a = m;
        m = t;
        const uint32_t qa = a / m, qb = b / m;
        total += (int64_t)qa * ((int64_t)n * (n - 1) / 2) + (int64_t)qb * n;
        a -= qa * m;
        b -= qb * m;
        top = a * n + b;
        if (top < m) return total;
        n = top / m;
        b = top - n * m;
    }
}

// Row tiles of a sequence for one head (head splits aside).
__device__ __forceinline__ int attn_row_tiles(const AttnArgs &s, const AttnSeq &q) {
    return q.n <= s.tile_tokens ? q.n > 0 : (q.n + s.tile_tokens - 1) / s.tile_tokens;
}

// Keys that the last token of row tile `rt` sees (the most any row of it sees), 0 if none.
__device__ __forceinline__ int attn_tile_keys(const AttnArgs &s, const AttnSeq &q, int rt) {
    if (!(s.a.flags & KS_ATTENTION_CAUSAL)) return q.keys;
    const int64_t last = min((int64_t)(rt + 1) * s.tile_tokens, (int64_t)q.n);
    return (int)max((int64_t)0, min((int64_t)q.keys, (int64_t)q.keys - q.n + last));
}

// Units of row tile `rt`: at least one, so that a tile that sees nothing still writes its zeros.
__device__ __forceinline__ int attn_tile_units(const AttnArgs &s, const AttnSeq &q, int rt) {
    return max(1, (int)(((uint32_t)attn_tile_keys(s, q, rt) + (1u << s.unit_shift) - 1) >> s.unit_shift));
}

// Cost of the row tiles [0, k) of one head, of `tiles` in all.
__device__ __forceinline__ int64_t attn_cost_before(const AttnArgs &s, const AttnSeq &q, int tiles, int k) {
    if (k <= 0) return 0;
    if (k == 1) return attn_tile_units(s, q, 0) + s.tile_cost;
    if (!(s.a.flags & KS_ATTENTION_CAUSAL)) return (int64_t)k * (attn_tile_units(s, q, 0) + s.tile_cost);
    int64_t total = (int64_t)k * s.tile_cost;
    if (k == tiles) {  // the last tile is cut off at the last token: by itself
        total += attn_tile_units(s, q, tiles - 1);
        --k;
    }
    // tile i < tiles - 1 sees past + (i + 1) tile_tokens keys; up to one unit of them counts as one
    const int past = q.keys - q.n, tt = s.tile_tokens, un = 1 << s.unit_shift;
    int one = 0;  // tiles i with past + (i + 1) tt <= un
    if (past < un) one = (int)min((uint32_t)k, ((uint32_t)un - (uint32_t)past) / (uint32_t)tt);
    if (one == k) return total + k;
    return total + one + floor_sum((uint32_t)(k - one), s.unit_shift, (uint32_t)tt,
                                   (uint32_t)(past + (one + 1) * (int64_t)tt + un - 1));
}

// A CTA's place in the call's units.
struct AttnCursor {
    int32_t seq, head, row_tile;  // head: key/value head * head_splits + split
    int32_t pos;                  // place in the row tile's cost: tile_cost, then its units
    int64_t left;                 // cost this CTA still has to do
    int64_t at;                   // place in the call's cost
    int64_t units;                // the call's cost
    int32_t ctas;                 // CTAs that have some
};

// The CTA's part of the row tile it is at: units [first, last) of `units`, none if first == last (its
// share ends in the tile's extra cost: the next CTA begins the tile).
struct AttnSpan {
    int32_t first, last, units, cost;
};

__device__ __forceinline__ AttnSpan attn_span(const AttnArgs &s, const AttnCursor &c, const AttnSeq &q) {
    AttnSpan p;
    p.units = attn_tile_units(s, q, c.row_tile);
    const int end = (int)min((int64_t)p.units + s.tile_cost, c.pos + c.left);
    p.first = max(0, c.pos - s.tile_cost);
    p.last = max(0, end - s.tile_cost);
    p.cost = end - c.pos;
    return p;
}

// The CTA that has place u of the cost U: the last c with U c / G < u + 1.
__device__ __forceinline__ int64_t attn_owner(const AttnCursor &c, int64_t u) {
    return quotient((u + 1) * c.ctas - 1, c.units);
}

// Finds the CTA's first unit: the sequences' units are summed by the block (a contiguous run of
// sequences per thread, a scan over the threads), the thread whose run holds the CTA's first unit
// names its sequence, and one warp searches that sequence's row tiles, 32 places at a time. All threads
// of the block call it; kThreads a multiple of 32, at most 1024. The result is in shared memory.
// It is one chain of latencies (2 to 3 us, most of it fetching code that no cache holds yet), which is
// why it divides by shifts where it can and computes nothing twice.
template <int kThreads>
__device__ inline const AttnCursor &attn_begin(const AttnArgs &s, int cta, int ctas) {
    constexpr int kWarps = kThreads / 32;
    __shared__ int64_t warp_units[kWarps];
    __shared__ int64_t found_before, found_per_head;
    __shared__ AttnCursor result;
    const int t = threadIdx.x, lane = t & 31, seqs = (int)s.a.seqs;
    const int per = seqs <= kThreads ? 1 : (seqs + kThreads - 1) / kThreads;
    const int64_t heads = (int64_t)s.a.kv_heads * s.head_splits;
    const int lo = min(seqs, t * per), hi = min(seqs, lo + per);
    int64_t mine = 0, per_head = 0;
    for (int b = lo; b < hi; ++b) {
        const AttnSeq q = attn_seq(s.a, b);
        const int tiles = attn_row_tiles(s, q);
        per_head = attn_cost_before(s, q, tiles, tiles);
        mine += heads * per_head;
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) warp_units[t / 32] = upto;
    __syncthreads();
    int64_t sums = lane < kWarps ? warp_units[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, sums, o);
        if (lane >= o) sums += v;
    }
    AttnCursor c = {};
    c.units = __shfl_sync(0xFFFFFFFFu, sums, kWarps - 1);
    const int64_t warps_before = __shfl_sync(0xFFFFFFFFu, sums, max(t / 32 - 1, 0));
    if (t >= 32) upto += warps_before;
    // with fewer units than CTAs, the first CTAs take one each: a row tile's pieces are then always
    // those of consecutive CTAs
    c.ctas = (int32_t)min((int64_t)ctas, c.units);
    if (cta >= c.ctas) {  // the whole block
        if (t == 0) result = c;
        __syncthreads();
        return result;
    }
    c.at = quotient(c.units * cta, c.ctas);
    c.left = quotient(c.units * (cta + 1), c.ctas) - c.at;
    int64_t before = upto - mine;
    if (before <= c.at && c.at < upto) {  // one thread, since some sequence has the unit
        c.seq = lo;
        for (int b = lo; per > 1; ++b) {
            const AttnSeq q = attn_seq(s.a, b);
            const int tiles = attn_row_tiles(s, q);
            per_head = attn_cost_before(s, q, tiles, tiles);
            c.seq = b;
            if (c.at < before + heads * per_head) break;
            before += heads * per_head;
        }
        result = c;
        found_before = before;
        found_per_head = per_head;
    }
    __syncthreads();
    if (t < 32) {
        const AttnSeq q = attn_seq(s.a, result.seq);
        const int tiles = attn_row_tiles(s, q);
        const int64_t begin = c.at - found_before;
        const int head = (int)quotient(begin, found_per_head);
        const int64_t u = begin - head * found_per_head;
        int low = 0, size = tiles;  // the wanted tile, the last that begins at or before u, is one of size from low on
        int64_t begins = 0;         // units before `low`
        while (size > 1) {
            const int step = (size + 31) >> 5;
            const int64_t mine_begins = lane * step < size ? attn_cost_before(s, q, tiles, low + lane * step) : u + 1;
            const int place = __popc(__ballot_sync(0xFFFFFFFFu, mine_begins <= u)) - 1;
            begins = __shfl_sync(0xFFFFFFFFu, mine_begins, place);
            low += place * step;
            size = min(step, size - place * step);
        }
        if (lane == 0) {
            result.head = head;
            result.row_tile = low;
            result.pos = (int32_t)(u - begins);
        }
    }
    __syncthreads();
    return result;
}

// Moves to the next row tile with units (called only while units are left).
__device__ __forceinline__ void attn_next(const AttnArgs &s, AttnCursor &c, AttnSeq &q) {
    c.pos = 0;
    if (++c.row_tile < attn_row_tiles(s, q)) return;
    c.row_tile = 0;
    if (++c.head < s.a.kv_heads * s.head_splits) return;
    c.head = 0;
    do {
        ++c.seq;
        if (c.seq >= s.a.seqs) return;  // not reached while units are left
        q = attn_seq(s.a, c.seq);
    } while (q.n == 0);
}

// Row r of a row tile: its token among all and its query head; false if the tile has no such row.
__device__ __forceinline__ bool attn_row(const AttnArgs &s, int q0, int n, int head, int row_tile,
                                         int r, int *token, int *q_head) {
    const int i = r / s.tile_heads, g = (head % s.head_splits) * s.tile_heads + r % s.tile_heads;
    const int in_seq = row_tile * s.tile_tokens + i;
    *token = q0 + in_seq;
    *q_head = (head / s.head_splits) * s.group + g;
    return i < s.tile_tokens && in_seq < n && g < s.group;
}

// Pieces of the row tile that the CTA begins: up to the CTA that has its last unit.
__device__ __forceinline__ int attn_pieces(const AttnArgs &s, const AttnCursor &c, const AttnSpan &p, int cta) {
    return (int)(attn_owner(c, c.at - c.pos + s.tile_cost + p.units - 1) - cta + 1);
}

// Workspace: per CTA two slots of rows * (dim + 2) floats (outputs, maxima, sums), then an AttnJoin per
// CTA. Outputs lie as the matrix instructions hand them out, so that a warp reads and writes 512 bytes
// in a row: by 16 rows and 8 columns, then four floats a lane, columns 2 (lane % 4) and the next of row
// lane / 4, then of row lane / 4 + 8.
__host__ __device__ inline int64_t attn_slot_floats(int64_t rows, int64_t dim) {
    return rows * (dim + 2);
}

__device__ __forceinline__ float *attn_slot(const AttnArgs &s, int64_t cta, int slot) {
    return (float *)s.a.workspace + (cta * 2 + slot) * attn_slot_floats(s.rows, s.a.head_dim);
}

__device__ __forceinline__ AttnJoin *attn_joins(const AttnArgs &s, int64_t ctas) {
    return (AttnJoin *)((float *)s.a.workspace + ctas * 2 * attn_slot_floats(s.rows, s.a.head_dim));
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / l, and 0 for a row that saw no key.
__device__ __forceinline__ float attn_inverse(float l) { return l == 0.0f ? 0.0f : __frcp_rn(l); }

// A maximum that can be subtracted: of a row that saw nothing yet, 0.
__device__ __forceinline__ float attn_base(float m) { return m == -INFINITY ? 0.0f : m; }

__device__ __forceinline__ float4 *attn_part(const AttnArgs &s, float *slot, int row_group, int col_group, int lane) {
    return reinterpret_cast<float4 *>(slot) + (row_group * ((int)s.a.head_dim / 8) + col_group) * 32 + lane;
}

// The tensor-core kernel (ks_attention_tc.cu): whether it takes a call's sizes, and its strides too,
// the rows and keys of its tiles, and its launch.
bool attn_tc_sizes(const ks_attention_args_t &a);
bool attn_tc_fits(const ks_attention_args_t &a);
int attn_tc_rows();
int attn_tc_unit();
int attn_tc_tile_cost();
cudaError_t attn_tc_launch(const AttnArgs &s, int ctas, cudaStream_t stream, bool pdl);

}  // namespace ks
