// What the attention kernels share: the list of work (sequences, tiles of query
// rows, heads, tiles of tokens), how it is dealt out, and how results are
// written and joined.
#pragma once

#include "pq2_cache.cuh"
#include "pq2_elem.cuh"

namespace pq2 {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

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

template <int ROWS>
__device__ __forceinline__ AttendItem attend_item(const pq2h::AttendParams& p, int b, int row_tile, int head) {
    AttendItem it = {b, row_tile, head, 0, 0, 0, 0, 0, 0, -1};
    const int G = p.q_heads / p.cache.heads;
    const int r0 = __ldcg(p.cache.row_start + b), r1 = __ldcg(p.cache.row_start + b + 1);
    const int len = __ldcg(p.cache.lens + b);
    const int most = p.cache.W * p.cache.T;
    const int n = r1 - r0;
    if (r0 < 0 || r1 < r0 || r1 > p.M || n > p.max_rows || len < 0 || len > most) {
        atomicOr(p.ctl.err, DEVERR_BAD_INDEX);
        if (!(len < 0 || len > most)) return it;
        if (r0 < 0 || r1 < r0 || r1 > p.M || n > p.max_rows) return it;
    }
    if (static_cast<long long>(row_tile) * ROWS >= static_cast<long long>(n) * G) return it;
    if (n * G <= p.over || n * G > p.upto) return it;  // (another kernel's)
    const int first = row_tile * ROWS / G, last = min(n - 1, (row_tile * ROWS + ROWS - 1) / G);
    it.n = n;
    it.row0 = r0;
    it.pos0 = min(max(len, 0), most) - n;
    const int lo = it.pos0 + first, hi = it.pos0 + last;
    if (hi >= 0) {
        it.tile1 = hi / kTileTokens + 1;
        if (p.window > 0 && lo - p.window + 1 > 0) it.tile0 = (lo - p.window + 1) / kTileTokens;
    }
    it.first_hi = p.window > 0 ? max(hi - p.window + 1, 0) : 0;
    it.last_lo = lo;
    return it;
}

// Units of an item: its tiles of `per` times 16 tokens, at least one (an item without
// any still has outputs to write), and before them `extra` for its rows.
__device__ __forceinline__ int attend_units(const AttendItem& it, int per, int extra) {
    if (it.n == 0) return 0;
    const int n = (it.tile1 + per - 1) / per - it.tile0 / per;
    return (it.tile1 > it.tile0 ? n : 1) + extra;
}

// A CTA's part of the list of units, and where a walk through it is.  The
// list's entries are (sequence, tile of rows), `row_tiles` for every sequence (those
// that it does not have are empty); an entry's heads follow one another.
struct AttendSpan {
    long long u0, u1, total;
    int ctas;
    int entry, units;   // an entry, its units per head
    long long before;   // units before it
};

template <int ROWS>
__device__ __forceinline__ int attend_entry_units(const pq2h::AttendParams& p, long long entry, int row_tiles, int per,
                                                  int extra) {
    const int b = static_cast<int>(entry / row_tiles);
    return attend_units(attend_item<ROWS>(p, b, static_cast<int>(entry - static_cast<long long>(b) * row_tiles), 0), per,
                        extra);
}

// The CTA's share of `total` units, at least `least` to a CTA (unless there are fewer).
__device__ __forceinline__ void attend_share(AttendSpan& s, long long total, int least) {
    s.total = total;
    s.ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), max(total / least, 1ll)));
    s.u0 = s.u1 = 0;
    s.entry = 0, s.units = 0, s.before = 0;
    const int cta = blockIdx.x;
    if (cta >= s.ctas) return;
    s.u0 = cta * total / s.ctas;
    s.u1 = (cta + 1) * total / s.ctas;
}

// All threads of the CTA call it (every warp finds the same).
template <int ROWS>
__device__ __forceinline__ void attend_span(const pq2h::AttendParams& p, int per, int extra, int least, AttendSpan& s) {
    const int lane = threadIdx.x & 31, B = p.cache.B, H = p.cache.heads;
    long long total = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
        int c = 0;
        if (b0 + lane < B) c = attend_entry_units<ROWS>(p, b0 + lane, 1, per, extra);
        total += __reduce_add_sync(0xffffffffu, c);
    }
    attend_share(s, total * H, least);
    if (s.u0 >= s.u1) return;
    for (int b0 = 0; b0 < B; b0 += 32) {
        int c = 0;
        if (b0 + lane < B) c = attend_entry_units<ROWS>(p, b0 + lane, 1, per, extra);
        int inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        const unsigned past = __ballot_sync(0xffffffffu, s.before + static_cast<long long>(inc) * H > s.u0);
        if (past) {
            const int at = __ffs(past) - 1;
            s.entry = b0 + at;
            s.units = __shfl_sync(0xffffffffu, c, at);
            s.before += static_cast<long long>(__shfl_sync(0xffffffffu, inc - c, at)) * H;
            return;
        }
        s.before += static_cast<long long>(__shfl_sync(0xffffffffu, inc, 31)) * H;
    }
}

// The same with the work on many entries split over the CTA's warps.
template <int ROWS, int WARPS>
__device__ __forceinline__ void attend_span_block(const pq2h::AttendParams& p, int row_tiles, int per, int extra, int least,
                                                  AttendSpan& s) {
    __shared__ long long sums[WARPS];
    __shared__ long long found_before;
    __shared__ int found_entry, found_units;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, H = p.cache.heads;
    const long long entries = static_cast<long long>(p.cache.B) * row_tiles;
    const long long share = (entries + WARPS - 1) / WARPS;
    const long long e0 = min(warp * share, entries), e1 = min(e0 + share, entries);
    long long mine = 0;
    for (long long e = e0; e < e1; e += 32)
        mine += __reduce_add_sync(0xffffffffu, e + lane < e1 ? attend_entry_units<ROWS>(p, e + lane, row_tiles, per, extra) : 0);
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
        for (long long e = e0; e < e1; e += 32) {
            const int c = e + lane < e1 ? attend_entry_units<ROWS>(p, e + lane, row_tiles, per, extra) : 0;
            int inc = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += u;
            }
            const unsigned past = __ballot_sync(0xffffffffu, before + static_cast<long long>(inc) * H > s.u0);
            if (past) {
                if (lane == __ffs(past) - 1) {
                    found_entry = static_cast<int>(e + lane);
                    found_units = c;
                    found_before = before + static_cast<long long>(inc - c) * H;
                }
                break;
            }
            before += static_cast<long long>(__shfl_sync(0xffffffffu, inc, 31)) * H;
        }
    }
    __syncthreads();
    s.entry = found_entry;
    s.units = found_units;
    s.before = found_before;
}

// The piece of work that begins at unit u: `units` units of an item, in them
// `count` of its `of` tiles, from its tile `first` on; `end`: unit behind the item.
struct AttendStep {
    int b, row_tile, head, first, count, of, units;
    long long end;
};
template <int ROWS>
__device__ __forceinline__ AttendStep attend_step(const pq2h::AttendParams& p, int row_tiles, int per, int extra,
                                                  AttendSpan& s, long long u) {
    const int H = p.cache.heads;
    while (u >= s.before + static_cast<long long>(s.units) * H) {
        s.before += static_cast<long long>(s.units) * H;
        ++s.entry;
        s.units = attend_entry_units<ROWS>(p, s.entry, row_tiles, per, extra);
    }
    const long long in = u - s.before;
    AttendStep st;
    st.b = s.entry / row_tiles;
    st.row_tile = s.entry - st.b * row_tiles;
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
