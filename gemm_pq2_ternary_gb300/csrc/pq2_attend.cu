// Attention over a cache held in 4 bits, a few query rows for each key/value
// head (decode and a few drafts).
//
// With codes c, scales s and offsets z of the rows of keys and values,
//   q . k_j = s_j (q . c_j) + z_j sum(q),
//   sum_j w_j v_j = sum_j (w_j s_j) (c_j - 8) + sum_j w_j (z_j + 8 s_j),
// so the products run on the codes alone, and scales and offsets touch one number per key.
// The fp16 whose bits are a small whole number n is n 2^-24 exactly (a
// subnormal), so a key's code becomes an operand by one AND: w & 0x000f000f is the
// pair of codes 0 and 4 of a word, w & 0x00f000f0 codes 1 and 5 times 16 (the
// query / 16 for those), and the same of w >> 8 the other four: 5 instructions for 8
// operands.  Values' codes take a subtraction more: products of codes around 8
// would leave sums many times the result, and the tensor cores cut off sums' low bits (over
// 131071 tokens 7e-4 of the result was lost, with codes around 0 nothing).
//
// Bound by HBM: (D + 8) bytes a token and head, each read once.  Scores are computed as
// K q^T (m16n8k16: 16 keys by 8 query rows), outputs as V^T w^T (16 dims by 8
// rows), so that up to 8 rows (a group of query heads) share one pass over the codes.
// A warp takes tiles of 16 tokens straight from memory into registers,
// two tiles ahead, with a maximum, sums and outputs of its own.  Maxima are
// raised only when a score exceeds the present one by 2^kSlack (a vote, not a
// reduction per tile): weights stay below 4, and times the values' scales (over a
// power of two, raised likewise, below 2) times kWeight below 2^15, with 2^-26
// of the largest still at fp16's full precision.
//
// The tiles of all sequences and heads form one list, dealt out evenly to the CTAs.
// A CTA joins its warps' results in shared memory; a head whose tiles lie
// in several CTAs is joined by a second kernel, in the CTAs' order.
#include <algorithm>

#include "pq2_attend.cuh"

namespace pq2 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 8;            // query rows of a pass
constexpr int kFewRows = 32;        // rows of a sequence and head that this kernel takes, at most
constexpr int kExtra = 16;          // what an item takes besides its tiles, in tiles
constexpr float kEmpty = -1e30f;    // maximum of a row that has seen nothing
constexpr float kSlack = 2.0f;      // how far (as a power of two) a score may exceed the maximum
constexpr float kWeight = 4096.0f;  // weights enter the product times this

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Two codes (HIGH: the high halves of their bytes, times 16) less 8, as fp16:
// 1024 + c has c in its last bits.
template <int HIGH>
__device__ __forceinline__ uint32_t centred(uint32_t w) {
    const uint32_t v = HIGH ? (w & 0x00f000f0u) | 0x64006400u : (w & 0x000f000fu) | 0x64006400u;
    const uint32_t c = HIGH ? 0x64806480u : 0x64086408u;
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&d);
}

// One tile as a lane (g, t) = (lane / 4, lane % 4) holds it.  The token in
// place r of the products' 16 is key_of(r), so that each load of a warp covers whole lines: keys of
// places g and g + 8 (a quarter t of each row), values of places 2t, 2t + 1,
// 2t + 8, 2t + 9 (an eighth g of each).
__device__ __forceinline__ int key_of(int place) { return (place & 8) + ((place & 7) >> 1) + 4 * (place & 1); }

template <int D>
struct Tile {
    uint32_t k[2][D / 32];
    uint32_t v[4][D / 64];
    uint32_t kp[2], vp[2];  // (scale, offset) of places g and g + 8
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t* p) {
    if constexpr (N == 1) {
        w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else if constexpr (N == 2) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = u.x, w[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
    }
}

template <int D>
__device__ __forceinline__ void load_keys(Tile<D>& x, const uint8_t* tile, int g, int t) {
#pragma unroll
    for (int r = 0; r < 2; ++r) load_words(x.k[r], tile + (key_of(g) + 8 * r) * (D / 2) + t * (D / 8));
}
template <int D>
__device__ __forceinline__ void load_pairs(Tile<D>& x, const uint8_t* tile, int g) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        x.kp[r] = __ldg(reinterpret_cast<const uint32_t*>(tile + tile_pairs(D, 0)) + key_of(g) + 8 * r);
        x.vp[r] = __ldg(reinterpret_cast<const uint32_t*>(tile + tile_pairs(D, 1)) + key_of(g) + 8 * r);
    }
}
template <int D>
__device__ __forceinline__ void load_values(Tile<D>& x, const uint8_t* tile, int g, int t) {
#pragma unroll
    for (int r = 0; r < 4; ++r) load_words(x.v[r], tile + tile_codes(D, 1) + (t + 4 * r) * (D / 2) + g * (D / 16));
}

__device__ __forceinline__ float pair_scale(uint32_t p) { return __half2float(__ushort_as_half(p & 0xffffu)); }
__device__ __forceinline__ float pair_offset(uint32_t p) { return __half2float(__ushort_as_half(p >> 16)); }

// What a warp holds of 8 query rows.  Columns of the products are rows of
// queries: a lane has rows 2t and 2t + 1 of maxima, sums and outputs.
template <int D>
struct Rows {
    float fq[2], sq[2];     // factor of the products, sum of the row (both in powers of two: times log2 e)
    int first[2], last[2];  // positions that the row sees
    float m[2], l[2], z[2]; // maximum, sum of weights, sum of weights times offsets
    float ref;              // values' scales over this (a power of two) are below 2
    float o[D / 16][4];     // outputs: dims 2j and 2j + 1 (times 16) of the lane's eighth
};

template <int D>
__device__ __forceinline__ void clear(Rows<D>& r) {
#pragma unroll
    for (int c = 0; c < 2; ++c) r.m[c] = kEmpty, r.l[c] = 0.0f, r.z[c] = 0.0f;
    r.ref = 0x1p-24f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) r.o[j][i] = 0.0f;
}

// The query rows of item `it`: lane (g, t) loads quarter t of row g.  `q`: the
// lane's place for the products' operands (in shared memory: in registers they would be spilled).
template <int D>
__device__ __forceinline__ void load_rows(Rows<D>& r, uint4* q, const pq2h::AttendParams& p, const AttendItem& it, int g,
                                          int t) {
    const int G = p.q_heads / p.cache.heads;
    const int i = it.row_tile * kRows + g, token = i / G;
    const bool there = token < it.n;
    float v[D / 32][8];
    float top = 0.0f, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (there)
            u = __ldg(reinterpret_cast<const uint4*>(p.q + static_cast<long long>(it.row0 + token) * p.ld_q +
                                                     static_cast<long long>(it.head * G + i % G) * p.hs_q + t * (D / 4)) + w);
        const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (p.bf16) {
                v[w][2 * k] = __uint_as_float(a[k] << 16);
                v[w][2 * k + 1] = __uint_as_float(a[k] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a[k]));
                v[w][2 * k] = f.x;
                v[w][2 * k + 1] = f.y;
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[w][k])), sum += v[w][k];
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    // the row times a power of two, its largest value in [2^7, 2^8): an eighth
    // of the steps below fp16's smallest normal number is 2^-32 of it
    const int e = top > 0.0f ? 134 - static_cast<int>(__float_as_uint(fmaxf(top, 0x1p-100f)) >> 23) : 0;
    const float up = __uint_as_float(static_cast<uint32_t>(127 + min(e, 126)) << 23);
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[w][k] *= up;
        q[32 * w] = make_uint4(half2_bits(v[w][0], v[w][4]), half2_bits(v[w][1] * 0.0625f, v[w][5] * 0.0625f),
                               half2_bits(v[w][2], v[w][6]), half2_bits(v[w][3] * 0.0625f, v[w][7] * 0.0625f));
    }
    const float k = p.scale * 1.4426950408889634f;
    const float f = k * 0x1p24f / up, s = k * sum;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        // row 2t + c is held by lanes (2t + c, *)
        r.fq[c] = __shfl_sync(0xffffffffu, f, (2 * t + c) * 4);
        r.sq[c] = __shfl_sync(0xffffffffu, s, (2 * t + c) * 4);
        const int token_c = (it.row_tile * kRows + 2 * t + c) / G;
        r.last[c] = token_c < it.n ? it.pos0 + token_c : it.pos0 + it.n - 1;
        r.first[c] = p.window > 0 ? r.last[c] - p.window + 1 : 0;
    }
}

// Raises maxima and the values' reference where this tile needs it.
template <int D>
__device__ __forceinline__ void raise(Rows<D>& r, const float (&x)[2][2], const float (&s)[2]) {
    float alpha[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float top = fmaxf(x[0][c], x[1][c]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, r.m[c]);
        alpha[c] = ex2(r.m[c] - top);
        r.m[c] = top;
        r.l[c] *= alpha[c];
        r.z[c] *= alpha[c];
    }
    float ref = fmaxf(fmaxf(s[0], s[1]), r.ref);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
    ref = __uint_as_float(__float_as_uint(ref) & 0x7f800000u);
    const float down = r.ref / ref;
    r.ref = ref;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = alpha[i & 1] * down;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) r.o[j][i] *= a;
    }
}

// Tokens key0 .. key0 + 15 into the warp's rows; what of the tile has been used makes
// room for tile `next` (null: there is none).
template <int D>
__device__ __forceinline__ void take_tile(Rows<D>& r, const uint4* q, Tile<D>& x, int key0, bool inside,
                                          const uint8_t* next, int g, int t) {
    float a[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        const uint32_t k0 = x.k[0][w], k1 = x.k[1][w];
        const uint4 b = q[32 * w];
        mma16816(a[0], k0 & 0x000f000fu, k1 & 0x000f000fu, k0 & 0x00f000f0u, k1 & 0x00f000f0u, b.x, b.y);
        const uint32_t h0 = k0 >> 8, h1 = k1 >> 8;
        mma16816(a[1], h0 & 0x000f000fu, h1 & 0x000f000fu, h0 & 0x00f000f0u, h1 & 0x00f000f0u, b.z, b.w);
    }
    if (next) load_keys<D>(x, next, g, t);
    float y[2][2], s[2], z[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        s[i] = pair_scale(x.vp[i]);
        z[i] = pair_offset(x.vp[i]);
        const float ks = pair_scale(x.kp[i]), kz = pair_offset(x.kp[i]);
#pragma unroll
        for (int c = 0; c < 2; ++c)
            y[i][c] = fmaf(a[0][2 * i + c] + a[1][2 * i + c], ks * r.fq[c], kz * r.sq[c]);
    }
    if (next) load_pairs<D>(x, next, g);
    if (!inside) {
        // tokens that a row does not see; what lies behind a sequence's last
        // token may be anything, a NaN included
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int key = key0 + key_of(g) + 8 * i;
            bool seen = false;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const bool in = key >= r.first[c] && key <= r.last[c];
                if (!in) y[i][c] = __uint_as_float(0xff800000u);
                seen |= in;
            }
            if (!seen) s[i] = 0.0f, z[i] = 0.0f;
        }
    }
    const bool more = y[0][0] > r.m[0] + kSlack || y[1][0] > r.m[0] + kSlack || y[0][1] > r.m[1] + kSlack ||
                      y[1][1] > r.m[1] + kSlack || s[0] >= 2.0f * r.ref || s[1] >= 2.0f * r.ref;
    if (__any_sync(0xffffffffu, more)) raise<D>(r, y, s);
    const float f = kWeight / r.ref;
    uint32_t b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float w[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            w[c] = ex2(y[i][c] - r.m[c]);
            r.l[c] += w[c];
            r.z[c] = fmaf(w[c], fmaf(8.0f, s[i], z[i]), r.z[c]);
        }
        const float sf = s[i] * f;
        b[i] = transpose8x8(half2_bits(w[0] * sf, w[1] * sf));
    }
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __byte_perm(x.v[0][w], x.v[1][w], h ? 0x7632 : 0x5410);
            const uint32_t hi = __byte_perm(x.v[2][w], x.v[3][w], h ? 0x7632 : 0x5410);
            mma16816(r.o[w * 4 + 2 * h], centred<0>(lo), centred<1>(lo), centred<0>(hi), centred<1>(hi), b[0], b[1]);
            const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
            mma16816(r.o[w * 4 + 2 * h + 1], centred<0>(lo8), centred<1>(lo8), centred<0>(hi8), centred<1>(hi8), b[0],
                     b[1]);
        }
    }
    if (next) load_values<D>(x, next, g, t);
}

template <int D>
constexpr int so_row() {
    return D + 4;
}
// Floats before the warps' queries.
template <int D>
constexpr int q_at() {
    return kWarps * kRows * (so_row<D>() + 2);
}
template <int D>
constexpr size_t smem_bytes() {
    return static_cast<size_t>(q_at<D>()) * 4 + static_cast<size_t>(kWarps) * D * 16;
}

// The segment of item `it` in tiles [t0, t1): every warp its own tiles, then
// joined.  `whole`: all of the item (the outputs are final), else its partial
// result goes to `slot`.
template <int D>
__device__ __forceinline__ void segment(const pq2h::AttendParams& p, const AttendWork& wk, const AttendItem& it, int t0,
                                        int t1, bool whole, int slot, float* smem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    Rows<D> r;
    uint4* q = reinterpret_cast<uint4*>(smem + q_at<D>()) + warp * D + lane;
    load_rows<D>(r, q, p, it, g, t);
    clear<D>(r);
    const int per_page = p.cache.T / kTileTokens;
    const long long head_at = static_cast<long long>(it.head) * per_page * tile_bytes(D);
    const int mine = t1 - t0 > warp ? (t1 - t0 - warp + kWarps - 1) / kWarps : 0;
    // tiles that every row sees all of
    const int in0 = it.first_hi, in1 = it.last_lo;
    int page_lane = 0;
    const auto look_up = [&](int i) {  // pages of the warp's tiles i .. i + 31, one a lane
        const int tile = t0 + warp + kWarps * (i + lane);
        int page = -1;
        if (tile < t1) {
            page = __ldg(p.cache.pages + it.b * p.cache.ld_pages + tile / per_page);
            if (page < 0 || page >= p.cache.num_pages) {
                page = -1;
                atomicOr(p.ctl.err, DEVERR_BAD_INDEX);
            }
        }
        page_lane = page;
    };
    const auto place = [&](int i) -> const uint8_t* {  // tile i's bytes, null outside the pool
        const int page = __shfl_sync(0xffffffffu, page_lane, i & 31);
        if (page < 0) return nullptr;
        const int tile = t0 + warp + kWarps * i;
        return p.cache.pool + page * p.cache.page_stride + head_at +
               static_cast<long long>(tile % per_page) * tile_bytes(D);
    };
    Tile<D> x;
    const uint8_t* from = nullptr;
    if (mine > 0) {
        look_up(0);
        from = place(0);
    }
    if (from) {
        load_keys<D>(x, from, g, t);
        load_pairs<D>(x, from, g);
        load_values<D>(x, from, g, t);
    }
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
        const uint8_t* next = nullptr;
        if (i + 1 < mine) {
            if (((i + 1) & 31) == 0) look_up(i + 1);
            next = place(i + 1);
        }
        if (from) {
            const int key0 = (t0 + warp + kWarps * i) * kTileTokens;
            take_tile<D>(r, q, x, key0, key0 >= in0 && key0 + kTileTokens - 1 <= in1, next, g, t);
        } else if (next) {
            load_keys<D>(x, next, g, t);
            load_pairs<D>(x, next, g);
            load_values<D>(x, next, g, t);
        }
        from = next;
    }
    // the warps' results: [warp][row][D] with maxima and sums behind them
    float* so = smem;
    float* sm = smem + kWarps * kRows * so_row<D>();
    float* sl = sm + kWarps * kRows;
    __syncthreads();  // (the segment before may still be read)
    const float f = r.ref / kWeight;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            r.l[c] += __shfl_xor_sync(0xffffffffu, r.l[c], o);
            r.z[c] += __shfl_xor_sync(0xffffffffu, r.z[c], o);
        }
        const int row = warp * kRows + 2 * t + c;
        if (g == 0) sm[row] = r.m[c], sl[row] = r.l[c];
        float* to = so + row * so_row<D>() + g * (D / 8);
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
            *reinterpret_cast<float2*>(to + 2 * j) =
                make_float2(fmaf(r.o[j][c], f, r.z[c]), fmaf(r.o[j][2 + c], f * 0.0625f, r.z[c]));
    }
    __syncthreads();
    // warp w joins row w, a lane D / 32 dims of it
    const int row = warp;
    float m = kEmpty;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm[w * kRows + row]);
    float l = 0.0f, o[D / 32];
#pragma unroll
    for (int j = 0; j < D / 32; ++j) o[j] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float a = ex2(sm[w * kRows + row] - m);
        l = fmaf(a, sl[w * kRows + row], l);
        const float* from_w = so + (w * kRows + row) * so_row<D>() + lane * (D / 32);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) o[j] = fmaf(a, from_w[j], o[j]);
    }
    const int d = lane * (D / 32);
    if (whole) {
        write_row<D / 32>(p, it, kRows, row, d, l, o);
        return;
    }
    const long long at = (static_cast<long long>(slot) * kRows + row) * D + d;
    if (store_ok(p.ctl, at, D / 32, wk.o_elems)) {
#pragma unroll
        for (int j = 0; j < D / 32; j += 2) *reinterpret_cast<float2*>(wk.o + at + j) = make_float2(o[j], o[j + 1]);
    }
    if (lane == 0 && store_ok(p.ctl, slot * kRows + row, 1, wk.ml_elems)) wk.ml[slot * kRows + row] = make_float2(m, l);
}

// The list's tiles, dealt out.
template <int D>
__global__ void __launch_bounds__(kThreads, D == 256 ? 1 : 2)
    attend_kernel(const __grid_constant__ pq2h::AttendParams p, const __grid_constant__ AttendWork wk, int row_tiles) {
    extern __shared__ __align__(16) float smem[];
    pdl_wait();
    pdl_launch_dependents();
    // (the walk through the list is thread 0's: in registers of all threads it
    // would be in the way of the tiles')
    __shared__ AttendSpan walk;
    __shared__ AttendStep step;
    long long u, u1;
    {
        AttendSpan span;
        if (row_tiles == 1)
            attend_span<kRows>(p, 1, kExtra, 2 * kWarps, span);
        else
            attend_span_block<kRows, kWarps>(p, row_tiles, 1, kExtra, 2 * kWarps, span);
        if (threadIdx.x == 0) {
            walk = span;
            wk.join[blockIdx.x] = {0, 0, 0, 0, 0};
        }
        u = span.u0, u1 = span.u1;
    }
    for (int n = 0; u < u1; ++n) {
        __syncthreads();
        if (threadIdx.x == 0) step = attend_step<kRows>(p, row_tiles, 1, kExtra, walk, u);
        __syncthreads();
        const AttendStep s = step;
        u += s.units;
        if (s.count == 0) continue;
        const AttendItem it = attend_item<kRows>(p, s.b, s.row_tile, s.head);
        const int t0 = it.tile0 + s.first, slot = 2 * blockIdx.x + (n > 0);
        if (threadIdx.x == 0 && s.first == 0 && s.count < s.of)
            wk.join[blockIdx.x] = {s.b, s.row_tile, s.head,
                                   attend_cta_of(walk, s.end - 1) - static_cast<int>(blockIdx.x) + 1, slot};
        segment<D>(p, wk, it, t0, min(t0 + s.count, it.tile1), s.count == s.of, slot, smem);
    }
}

// CTA (c, row): row `row` of the item whose first part is CTA c's.  Each of
// the warps takes every kJoinWarps-th part, a lane D / 32 dims.
constexpr int kJoinWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
    attend_join_kernel(const __grid_constant__ pq2h::AttendParams p, const __grid_constant__ AttendWork wk) {
    __shared__ float so[kJoinWarps][D];
    __shared__ float sm[kJoinWarps], sl[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y;
    pdl_wait();
    pdl_launch_dependents();
    const AttendJoin j = wk.join[blockIdx.x];
    if (j.parts == 0) return;
    const auto slot_of = [&](int i) { return i == 0 ? j.first_slot : 2 * (static_cast<int>(blockIdx.x) + i); };
    float m = kEmpty, l = 0.0f, o[D / 32];
#pragma unroll
    for (int k = 0; k < D / 32; ++k) o[k] = 0.0f;
    for (int i = warp; i < j.parts; i += kJoinWarps) m = fmaxf(m, wk.ml[slot_of(i) * kRows + row].x);
    for (int i = warp; i < j.parts; i += kJoinWarps) {
        const long long at = static_cast<long long>(slot_of(i)) * kRows + row;
        const float2 ml = wk.ml[at];
        const float a = ex2(ml.x - m);
        l = fmaf(a, ml.y, l);
        const float2* f = reinterpret_cast<const float2*>(wk.o + at * D + lane * (D / 32));
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
            const float2 v = f[k];
            o[2 * k] = fmaf(a, v.x, o[2 * k]);
            o[2 * k + 1] = fmaf(a, v.y, o[2 * k + 1]);
        }
    }
#pragma unroll
    for (int k = 0; k < D / 32; ++k) so[warp][lane * (D / 32) + k] = o[k];
    if (lane == 0) sm[warp] = m, sl[warp] = l;
    __syncthreads();
    if (warp != 0) return;
    float top = kEmpty;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, sm[w]);
    l = 0.0f;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) o[k] = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        const float a = ex2(sm[w] - top);
        l = fmaf(a, sl[w], l);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) o[k] = fmaf(a, so[w][lane * (D / 32) + k], o[k]);
    }
    const AttendItem it = attend_item<kRows>(p, j.b, j.row_tile, j.head);
    write_row<D / 32>(p, it, kRows, row, lane * (D / 32), l, o);
}

}  // namespace
}  // namespace pq2

namespace pq2h {

namespace {

size_t pad(size_t b) { return (b + 255) & ~size_t(255); }

template <int D>
cudaError_t launch_few(const AttendParams& p, const pq2::AttendWork& wk, cudaStream_t st, const DeviceInfo& dev) {
    static SmemLimit lim;
    const size_t smem = pq2::smem_bytes<D>();
    cudaError_t e = raise_smem(lim, pq2::attend_kernel<D>, smem);
    if (e != cudaSuccess) return e;
    const int G = p.q_heads / p.cache.heads, row_tiles = (p.max_rows * G + pq2::kRows - 1) / pq2::kRows;
    const int64_t ctas = std::min<int64_t>(dev.num_sms * (D == 256 ? 1 : 2), pq2::kAttendCtas);
    e = launch(pq2::attend_kernel<D>, dim3(static_cast<unsigned>(ctas)), dim3(pq2::kThreads), smem, st, true, p, wk, row_tiles);
    if (e != cudaSuccess) return e;
    return launch(pq2::attend_join_kernel<D>, dim3(static_cast<unsigned>(ctas), pq2::kRows),
                  dim3(32 * pq2::kJoinWarps), 0, st, true, p, wk);
}

}  // namespace

size_t attend_workspace_bytes(int64_t M, int64_t q_heads, int64_t heads, int64_t dim) {
    const size_t rows = 2ull * pq2::kAttendCtas * pq2::kRows;
    const size_t few = pad(rows * dim * 4) + pad(rows * 8) + pad(pq2::kAttendCtas * sizeof(pq2::AttendJoin));
    return M * (q_heads / heads) > pq2::kFewRows ? std::max(few, attend_many_workspace_bytes(M, q_heads, heads, dim)) : few;
}

cudaError_t launch_attend(const AttendParams& p, void* workspace, cudaStream_t st, const DeviceInfo& dev) {
    const int64_t G = p.q_heads / p.cache.heads;
    if (p.max_rows * G > pq2::kFewRows) return launch_attend_many(p, workspace, st, dev);
    pq2::AttendWork wk = {};
    wk.rows = pq2::kRows;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    const size_t rows = 2ull * pq2::kAttendCtas * pq2::kRows;
    wk.o = reinterpret_cast<float*>(w);
    wk.o_elems = rows * p.dim;
    w += pad(rows * p.dim * 4);
    wk.ml = reinterpret_cast<float2*>(w);
    wk.ml_elems = rows;
    w += pad(rows * 8);
    wk.join = reinterpret_cast<pq2::AttendJoin*>(w);
    switch (p.dim) {
        case 64: return launch_few<64>(p, wk, st, dev);
        case 128: return launch_few<128>(p, wk, st, dev);
    }
    return launch_few<256>(p, wk, st, dev);
}

}  // namespace pq2h
