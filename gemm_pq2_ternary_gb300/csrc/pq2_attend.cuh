// What the attention kernels share: the list of work (sequences, tiles of query
// rows, heads, tiles of tokens), how it is dealt out, and how results are
// written and joined.
#pragma once

#include <climits>

#include "pq2_cache.cuh"
#include "pq2_elem.cuh"

namespace pq2 {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Rows of a warp that do not see the same values.  The values' reference is a power of two; scales
// over it are below 2.  With one that goes by all values a row's weights could sink below fp16's
// numbers next to values that other rows alone see.  So it goes by the row that sees the smallest
// ones, and a row that sees values larger by 2^kApart and more has its maximum raised by b, the
// difference of the two, which takes its weights down as much.  (Rows whose maximum is so large
// that this is not exact have no b.)
constexpr int kApart = 4;
constexpr float kHuge = 0x1p22f;

// b of a lane's rows, 8 bits each.
__device__ __forceinline__ int row_b(uint32_t bs, int r) { return bs >> (8 * r) & 255; }

// A scale's power of two, fp16's smallest number at least; and such powers' quotient, as an exponent.
__device__ __forceinline__ float scale_power(float x) {
    return __uint_as_float(__float_as_uint(fmaxf(x, 0x1p-24f)) & 0x7f800000u);
}
__device__ __forceinline__ int power_between(float lo, float hi) {
    return static_cast<int>(__float_as_uint(hi) >> 23) - static_cast<int>(__float_as_uint(lo) >> 23);
}

// 2^n for whole |n| < 127; 0 from -126 on.
__device__ __forceinline__ float power_of_two(float n) {
    return n > -126.0f ? __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(n)) << 23) : 0.0f;
}

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// What the rows that have seen something need of the reference: `lo` and `hi` for the smallest and largest
// of their values, `huge` for the largest of the rows without a b.
struct Apart {
    float lo = 0x1p30f, hi = 0.0f, huge = 0.0f;
    __device__ __forceinline__ void row(float max, float own, float empty) {
        if (max == empty) return;
        lo = fminf(lo, own);
        hi = fmaxf(hi, own);
        if (fabsf(max) >= kHuge) huge = fmaxf(huge, own);
    }
    __device__ __forceinline__ float reference(float ref) const {
        const float least = fmaxf(-warp_max(-lo), warp_max(huge)), most = warp_max(hi);
        return most == 0.0f ? ref : most < least * (1 << kApart) ? most : least;
    }
};

// A head whose tiles lie in more than one CTA: the CTA that has its first
// ones writes down which partial results belong together.
struct AttendJoin {
    int b, row_tile, head;
    int parts;       // 0: nothing to join
    int first_slot;  // the others are the first slots of the CTAs that follow
};

constexpr int kAttendCtas = 512;  // CTAs that a list is dealt out to, at most

// Partial results in the workspace.
struct AttendWork {
    float* o;          // [2 CTAs][rows][dim] outputs, not yet divided
    float2* ml;        // [2 CTAs][rows] maximum, sum of weights
    AttendJoin* join;  // [CTAs]
    int rows;          // of a partial result
    long long o_elems, ml_elems;  // for the bounds-checked build
};

// One tile of query rows of one sequence and key/value head.  Row i of the
// sequence's n G rows is query head i % G of token i / G.
struct AttendItem {
    int b, row_tile, head;
    int n;              // the sequence's tokens in this call; 0: no such item
    int row0, pos0;     // its first token's row and position
    int tile0, tile1;   // tiles of 16 tokens that the rows see something of
    int first_hi, last_lo;  // positions that all rows see all of: first_hi .. last_lo
};

// What of a sequence its items are made from.
struct AttendSequence {
    int n, row0, pos0;  // n == 0: nothing for this kernel
};

__device__ __forceinline__ AttendSequence attend_sequence(const pq2h::AttendParams& p, int b) {
    const int r0 = __ldcg(p.cache.row_start + b), r1 = __ldcg(p.cache.row_start + b + 1);
    const int len = __ldcg(p.cache.lens + b);
    const int most = p.cache.W * p.cache.T;
    const int n = r1 - r0;
    const bool bad = r0 < 0 || r1 < r0 || r1 > p.M || n > p.max_rows;
    if (bad || len < 0 || len > most) atomicOr(p.ctl.err, DEVERR_BAD_INDEX);
    if (bad || n == 0) return {0, 0, 0};
    const int rows = n * (p.q_heads / p.cache.heads);
    if (rows <= p.over || rows > p.upto) return {0, 0, 0};  // (another kernel's)
    return {n, r0, min(max(len, 0), most) - n};
}

template <int ROWS>
__device__ __forceinline__ AttendItem attend_item(const pq2h::AttendParams& p, const AttendSequence& q, int b, int row_tile,
                                                  int head) {
    AttendItem it = {b, row_tile, head, 0, 0, 0, 0, 0, 0, -1};
    const int G = p.q_heads / p.cache.heads;
    if (static_cast<long long>(row_tile) * ROWS >= static_cast<long long>(q.n) * G) return it;
    const int first = row_tile * ROWS / G, last = min(q.n - 1, (row_tile * ROWS + ROWS - 1) / G);
    it.n = q.n;
    it.row0 = q.row0;
    it.pos0 = q.pos0;
    const int lo = it.pos0 + first, hi = it.pos0 + last;
    if (hi >= 0) {
        it.tile1 = hi / kTileTokens + 1;
        if (p.window > 0 && lo - p.window + 1 > 0) it.tile0 = (lo - p.window + 1) / kTileTokens;
    }
    it.first_hi = p.window > 0 ? max(hi - p.window + 1, 0) : 0;
    it.last_lo = lo;
    return it;
}

template <int ROWS>
__device__ __forceinline__ AttendItem attend_item(const pq2h::AttendParams& p, int b, int row_tile, int head) {
    return attend_item<ROWS>(p, attend_sequence(p, b), b, row_tile, head);
}

// Units of an item: its tiles of `per` times 16 tokens, at least one (an item without
// any still has outputs to write), and before them `extra` for its rows.
__device__ __forceinline__ int attend_units(const AttendItem& it, int per, int extra) {
    if (it.n == 0) return 0;
    const int n = (it.tile1 + per - 1) / per - it.tile0 / per;
    return (it.tile1 > it.tile0 ? n : 1) + extra;
}

// A CTA's part of the list of units, and where a walk through it is.  The
// list's entries are the sequences' tiles of rows; an entry's heads follow one another.
struct AttendSpan {
    long long u0, u1, total;
    int ctas;
    int b, row_tile, tiles;  // an entry; its sequence's tiles of rows
    AttendSequence sequence;
    int units;               // the entry's, per head
    long long before;        // units before it
};

// A sequence's tiles of rows.
template <int ROWS>
__device__ __forceinline__ int attend_row_tiles(const pq2h::AttendParams& p, const AttendSequence& q) {
    return static_cast<int>((static_cast<long long>(q.n) * (p.q_heads / p.cache.heads) + ROWS - 1) / ROWS);
}

template <int ROWS>
__device__ __forceinline__ int attend_entry_units(const pq2h::AttendParams& p, const AttendSequence& q, int row_tile, int per,
                                                  int extra) {
    return attend_units(attend_item<ROWS>(p, q, 0, row_tile, 0), per, extra);
}

// That of a lane, for all.
__device__ __forceinline__ AttendSequence attend_sequence_of(const AttendSequence& q, int lane) {
    return {__shfl_sync(0xffffffffu, q.n, lane), __shfl_sync(0xffffffffu, q.row0, lane), __shfl_sync(0xffffffffu, q.pos0, lane)};
}

// The sum over a warp's lanes, and up to a lane.
__device__ __forceinline__ long long warp_scan(long long v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Units per head of a lane's sequence.  A few tiles of rows are its lane's
// work, more are all lanes'.
template <int ROWS>
__device__ __forceinline__ long long attend_sequence_units(const pq2h::AttendParams& p, const AttendSequence& q, int per,
                                                           int extra) {
    constexpr int kFew = 4;
    const int lane = threadIdx.x & 31, tiles = attend_row_tiles<ROWS>(p, q);
    long long units = 0;
#pragma unroll 1
    for (int r = 0; r < (tiles > kFew ? 0 : tiles); ++r) units += attend_entry_units<ROWS>(p, q, r, per, extra);
    __syncwarp();
#pragma unroll 1
    for (unsigned longer = __ballot_sync(0xffffffffu, tiles > kFew); longer; longer &= longer - 1) {
        const int from = __ffs(longer) - 1, n = __shfl_sync(0xffffffffu, tiles, from);
        const AttendSequence other = attend_sequence_of(q, from);
        long long sum = 0;
        for (int r = lane; r < n; r += 32) sum += attend_entry_units<ROWS>(p, other, r, per, extra);
        sum = __shfl_sync(0xffffffffu, warp_scan(sum), 31);
        if (lane == from) units = sum;
    }
    return units;
}

// The CTA's share of `total` units, at least `least` to a CTA (unless there are fewer).
__device__ __forceinline__ void attend_share(AttendSpan& s, long long total, int least) {
    s.total = total;
    s.ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), max(total / least, 1ll)));
    s.u0 = s.u1 = 0;
    s.b = 0, s.row_tile = 0, s.tiles = 0, s.units = 0, s.before = 0;
    s.sequence = {0, 0, 0};
    const int cta = blockIdx.x;
    if (cta >= s.ctas) return;
    s.u0 = cta * total / s.ctas;
    s.u1 = (cta + 1) * total / s.ctas;
}

// All threads of the CTA call it; the sequences are split over its warps.
template <int ROWS, int WARPS>
__device__ __forceinline__ void attend_span(const pq2h::AttendParams& p, int per, int extra, int least, AttendSpan& s) {
    __shared__ long long sums[WARPS];
    __shared__ long long found_before;
    __shared__ int found[4];  // b, row_tile, tiles, units
    __shared__ AttendSequence found_sequence;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, B = p.cache.B, H = p.cache.heads;
    const int share = (B + WARPS - 1) / WARPS;
    const int b0 = min(warp * share, B), b1 = min(b0 + share, B);
    long long mine = 0;
    const auto sequence_at = [&](int b) { return b < b1 ? attend_sequence(p, b) : AttendSequence{0, 0, 0}; };
    for (int b = b0; b < b1; b += 32)
        mine += __shfl_sync(0xffffffffu, warp_scan(attend_sequence_units<ROWS>(p, sequence_at(b + lane), per, extra)), 31);
    if (lane == 0) sums[warp] = mine * H;
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w == warp) before = total;
        total += sums[w];
    }
    attend_share(s, total, least);
    if (s.u0 >= s.u1) return;  // (all threads alike)
    if (before <= s.u0 && s.u0 < before + mine * H) {
        for (int b = b0; b < b1; b += 32) {
            const AttendSequence mine_q = sequence_at(b + lane);
            const long long c = attend_sequence_units<ROWS>(p, mine_q, per, extra), inc = warp_scan(c);
            const unsigned past = __ballot_sync(0xffffffffu, before + inc * H > s.u0);
            if (past) {
                // the sequence; then its tile of rows
                const int at = __ffs(past) - 1;
                before += __shfl_sync(0xffffffffu, inc - c, at) * H;
                const AttendSequence q = attend_sequence_of(mine_q, at);
                const int tiles = attend_row_tiles<ROWS>(p, q);
                for (int r = 0; r < tiles; r += 32) {
                    const int units = r + lane < tiles ? attend_entry_units<ROWS>(p, q, r + lane, per, extra) : 0;
                    const long long upto = warp_scan(units);
                    const unsigned here = __ballot_sync(0xffffffffu, before + upto * H > s.u0);
                    if (here) {
                        if (lane == __ffs(here) - 1) {
                            found[0] = b + at, found[1] = r + lane, found[2] = tiles, found[3] = units;
                            found_before = before + (upto - units) * H;
                            found_sequence = q;
                        }
                        break;
                    }
                    before += __shfl_sync(0xffffffffu, upto, 31) * H;
                }
                break;
            }
            before += __shfl_sync(0xffffffffu, inc, 31) * H;
        }
    }
    __syncthreads();
    s.b = found[0], s.row_tile = found[1], s.tiles = found[2], s.units = found[3];
    s.before = found_before;
    s.sequence = found_sequence;
}

// The piece of work that begins at unit u: `units` units of an item, in them
// `count` of its `of` tiles, from its tile `first` on; `end`: unit behind the item.
struct AttendStep {
    int b, row_tile, head, first, count, of, units;
    long long end;
};
// (by whole warps: sequences without work are passed over 32 at a time)
template <int ROWS>
__device__ __forceinline__ AttendStep attend_step(const pq2h::AttendParams& p, int per, int extra, AttendSpan& s,
                                                  long long u) {
    const int H = p.cache.heads, lane = threadIdx.x & 31;
    while (u >= s.before + static_cast<long long>(s.units) * H) {
        s.before += static_cast<long long>(s.units) * H;
        if (++s.row_tile >= s.tiles) {
            s.row_tile = 0;
            unsigned some = 0;
            int b = s.b + 1;
            for (; some == 0 && b < p.cache.B; b += 32) {
                const AttendSequence q = b + lane < p.cache.B ? attend_sequence(p, b + lane) : AttendSequence{0, 0, 0};
                const int tiles = attend_row_tiles<ROWS>(p, q);
                some = __ballot_sync(0xffffffffu, tiles > 0);
                if (some == 0) continue;
                s.b = b + __ffs(some) - 1;
                s.tiles = __shfl_sync(0xffffffffu, tiles, __ffs(some) - 1);
                s.sequence = attend_sequence_of(q, __ffs(some) - 1);
            }
            if (some == 0) {  // (only where the inputs have changed under way)
                s.units = INT_MAX;
                break;
            }
        }
        s.units = attend_entry_units<ROWS>(p, s.sequence, s.row_tile, per, extra);
    }
    const long long in = u - s.before;
    AttendStep st;
    st.b = s.b;
    st.row_tile = s.row_tile;
    st.head = static_cast<int>(in / s.units);
    const int at = static_cast<int>(in - static_cast<long long>(st.head) * s.units);
    st.units = static_cast<int>(min(static_cast<long long>(s.units - at), s.u1 - u));
    st.first = max(at - extra, 0);
    st.count = max(at + st.units - extra, 0) - st.first;
    st.of = s.units - extra;
    st.end = u - at + s.units;
    return st;
}

// The CTA that has unit u: the last with floor(cta total / ctas) <= u.
__device__ __forceinline__ int attend_cta_of(const AttendSpan& s, long long u) {
    return static_cast<int>(((u + 1) * s.ctas - 1) / s.total);
}

// N neighbouring outputs of one query row, from dim d on.
template <int N>
__device__ __forceinline__ void write_row(const pq2h::AttendParams& p, const AttendItem& it, int rows, int row, int d,
                                          float l, const float (&o)[N]) {
    const int G = p.q_heads / p.cache.heads;
    const int i = it.row_tile * rows + row, token = i / G;
    if (token >= it.n) return;
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const long long at = static_cast<long long>(it.row0 + token) * p.ld_out +
                         static_cast<long long>(it.head * G + i % G) * p.hs_out + d;
    if (!store_ok(p.ctl, at, N, p.out_elems)) return;
    const int type = p.bf16 ? PQ2_BF16 : PQ2_F16;
    uint32_t w[N / 2];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) w[k] = f32x2_to_elem16(o[2 * k] * inv, o[2 * k + 1] * inv, type);
    if constexpr (N == 2)
        *reinterpret_cast<uint32_t*>(p.out + at) = w[0];
    else if constexpr (N == 4)
        *reinterpret_cast<uint2*>(p.out + at) = make_uint2(w[0], w[1]);
    else
#pragma unroll
        for (int k = 0; k < N / 8; ++k)
            *reinterpret_cast<uint4*>(p.out + at + 8 * k) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
}

}  // namespace pq2
