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
// Has to read (D + 8) bytes a token and head once.  Scores are computed as K q^T
// (m16n8k16: 16 keys by 8 query rows), outputs as V^T w^T (16 dims by 8 rows), so
// that up to 8 rows (a group of query heads), or 16 in two products, share one pass over
// the codes.  A warp takes tiles of 16 tokens from a ring of its own in shared memory, which
// bulk copies fill three tiles ahead, with a maximum, sums and outputs of its own.
// Maxima are raised only when a score exceeds the present one by 2^kSlack (a vote,
// not a reduction per tile): weights stay below 32, and times the values' scales (over
// a power of two, raised likewise, below 2) times kWeight below 2^15, with weights down to
// 2^-23 at fp16's full precision (where all rows see values of like size; pq2_attend.cuh).
//
// The tiles of all sequences and heads form one list, dealt out evenly to the CTAs;
// an item (a sequence's tile of rows and head) counts for kExtra tiles more.  A CTA joins its warps'
// results in shared memory; a head whose tiles lie in several CTAs is joined by a second
// kernel, in the CTAs' order.
//
// Bound by instructions and their latency: 497 warp instructions a tile of 16 tokens and head of
// 128 dims, 632 of 256, most of them on the integer pipe (operands from codes), issued at 52% and
// 45% of the rate.  On GB300: 131071 tokens, 24 heads of 256 on 4: 45 us, 3.1 TB/s (58 with
// loads into registers, 8 warps an SM and a join of one warp's loads at a time); 64 sequences of up
// to 8192, 48 heads of 128 on 8: 94 us, 3.0 TB/s (107 to 147 while the list counted tiles alone
// and registers were spilled); 75 tokens of 24 sequences of up to 5003, 40 heads of 128 on 8: 60 us
// (62 with 8 rows a pass).  Two groups of rows of 128 dims spill 284 bytes.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <type_traits>

#include "pq2_attend.cuh"

namespace pq2 {
namespace {

// A pass takes RG groups of 8 query rows: two of them share a tile's operands.
// Warps of a CTA and CTAs of an SM: as many as registers allow.
template <int D, int RG>
constexpr int kWarps = D == 256 && RG == 1 ? 12 : 8;
template <int D>
constexpr int kBlocks = D == 256 ? 1 : 2;
// Rows of a sequence and head that this kernel takes, at most; more go to
// pq2_attend_many.cu.  Both, in us (this one first).  24 sequences of 5003 tokens: heads of
// 128, 25 rows 120 and 166, 40 rows 161 and 164, 65 rows 246 and 166; of 256, 18 rows 111 and
// 106, 30 rows 111 and 108, 48 rows 151 and 109; of 64, 48 rows 112 and 125, 64 rows 141 and
// 130.  One sequence of 30000: heads of 128, 50 rows 62 and 65; of 256, 78 rows 70 and 90.
constexpr int few_rows(int64_t dim) { return dim == 256 ? 32 : 48; }
constexpr int kMostRows = 16;       // of a pass
// What an item takes besides its tiles, in tiles (64 sequences, 8 rows: 8 111 us, 16 107, 32 95,
// 64 96, 96 99; drafts, 25 rows: 16 69 us, 32 59, 48 57).
template <int RG>
constexpr int kExtra = RG == 1 ? 32 : 48;
constexpr float kEmpty = -FLT_MAX;  // maximum of a row that has seen nothing: below any score
constexpr float kSlack = 5.0f;      // how far (as a power of two) a score may exceed the maximum
constexpr float kWeight = 512.0f;  // weights enter the product times this

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

// One tile as a lane (g, t) = (lane / 4, lane % 4) takes it from shared memory: keys
// of places g and g + 8 of the products' 16 (a quarter t of each row), values of
// places 2t, 2t + 1, 2t + 8, 2t + 9 (an eighth g of each).  The token in a place:
// of two neighbouring places one is odd, of four values taken at once two are, so that
// with rows of 64 bytes keys meet every bank once and values twice.
__device__ __forceinline__ int key_of(int place) { return place ^ ((place >> 1) & 1); }

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t* p) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        w[0] = u.x, w[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 u = *(reinterpret_cast<const uint4*>(p) + i);
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
    }
}

__device__ __forceinline__ float pair_scale(uint32_t p) { return __half2float(__ushort_as_half(p & 0xffffu)); }
__device__ __forceinline__ float pair_offset(uint32_t p) { return __half2float(__ushort_as_half(p >> 16)); }

// What a warp holds of 8 query rows.  Columns of the products are rows of
// queries: a lane has rows 2t and 2t + 1 of maxima, sums and outputs.
template <int D, int RG>
struct Rows {
    static constexpr bool kShared = D == 256 || RG == 2;  // products' operands stay in shared memory
    uint4 q[kShared ? 1 : D / 32];
    float fq[RG][2], sq[RG][2];      // factor of the products, sum of the row (both in powers of two: times log2 e)
    int first[RG][2], last[RG][2];   // positions that the row sees
    float m[RG][2], l[RG][2], z[RG][2];  // maximum, sum of weights, sum of weights times offsets
    float ref;                       // values' scales over this (a power of two) are below 2
    float slack;                     // kSlack less the largest b (pq2_attend.cuh)
    uint32_t bs;
    float o[RG][D / 16][4];          // outputs: dims 2j and 2j + 1 (times 16) of the lane's eighth
    __device__ __forceinline__ uint4 query(const uint4* shared, int u, int w) const {
        if constexpr (kShared)
            return shared[32 * (u * (D / 32) + w)];
        else
            return q[w];
    }
};

template <int D, int RG>
__device__ __forceinline__ void clear(Rows<D, RG>& r) {
    r.ref = 0x1p-24f, r.slack = kSlack, r.bs = 0;
#pragma unroll
    for (int u = 0; u < RG; ++u) {
#pragma unroll
        for (int c = 0; c < 2; ++c) r.m[u][c] = kEmpty, r.l[u][c] = 0.0f, r.z[u][c] = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) r.o[u][j][i] = 0.0f;
    }
}

// The query rows of item `it`: lane (g, t) loads quarter t of row g.  `q`: the
// lane's place for those of 256 dims.
template <int D, int RG>
__device__ __forceinline__ void load_rows(Rows<D, RG>& r, uint4* q, const pq2h::AttendParams& p, const AttendItem& it, int u,
                                          int g, int t) {
    const int G = p.q_heads / p.cache.heads;
    const int i = it.row_tile * 8 * RG + 8 * u + g, token = i / G;
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
    // the row times a power of two, its largest value in [2^7, 2^8): half a step of a
    // sixteenth below fp16's smallest normal number is 2^-28 of it
    const int e = top > 0.0f ? 134 - static_cast<int>(__float_as_uint(fmaxf(top, 0x1p-100f)) >> 23) : 0;
    const float up = __uint_as_float(static_cast<uint32_t>(127 + min(e, 126)) << 23);
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[w][k] *= up;
        const uint4 b = make_uint4(half2_bits(v[w][0], v[w][4]), half2_bits(v[w][1] * 0.0625f, v[w][5] * 0.0625f),
                                   half2_bits(v[w][2], v[w][6]), half2_bits(v[w][3] * 0.0625f, v[w][7] * 0.0625f));
        if constexpr (!Rows<D, RG>::kShared)
            r.q[w] = b;
        else if (threadIdx.x < 32)  // (all warps have the same)
            q[32 * (u * (D / 32) + w)] = b;
    }
    const float k = p.scale * 1.4426950408889634f;
    const float f = k * 0x1p24f / up, s = k * sum;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        // row 2t + c is held by lanes (2t + c, *)
        r.fq[u][c] = __shfl_sync(0xffffffffu, f, (2 * t + c) * 4);
        r.sq[u][c] = __shfl_sync(0xffffffffu, s, (2 * t + c) * 4);
        const int token_c = (it.row_tile * 8 * RG + 8 * u + 2 * t + c) / G;
        r.last[u][c] = token_c < it.n ? it.pos0 + token_c : it.pos0 + it.n - 1;
        r.first[u][c] = p.window > 0 ? r.last[u][c] - p.window + 1 : 0;
    }
}

// 1 / x of a power of two.
__device__ __forceinline__ float inverse(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }

// Raises maxima and the values' reference where this tile (its keys from `key` on, and
// key + 8) needs it.  With `inside` all rows see all of it.
template <int D, int RG>
__device__ __forceinline__ void raise(Rows<D, RG>& r, const float (&x)[RG][2][2], const float (&s)[2], bool inside, int key) {
    float ref, top[RG][2];
#pragma unroll
    for (int u = 0; u < RG; ++u)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            top[u][c] = fmaxf(x[u][0][c], x[u][1][c]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top[u][c] = fmaxf(top[u][c], __shfl_xor_sync(0xffffffffu, top[u][c], o));
        }
    if (__all_sync(0xffffffffu, inside && r.bs == 0)) {  // all rows see the same
        ref = scale_power(fmaxf(warp_max(fmaxf(s[0], s[1])), r.ref));
#pragma unroll
        for (int u = 0; u < RG; ++u)
#pragma unroll
            for (int c = 0; c < 2; ++c) top[u][c] = fmaxf(top[u][c], r.m[u][c]);
    } else {
        Apart apart;
        float own[RG][2];  // the largest scale of the values that the row sees
#pragma unroll
        for (int u = 0; u < RG; ++u)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float most = 0.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (key + 8 * i >= r.first[u][c] && key + 8 * i <= r.last[u][c]) most = fmaxf(most, s[i]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                const float b = static_cast<float>(row_b(r.bs, 2 * u + c));
                const bool empty = r.m[u][c] == kEmpty;
                own[u][c] = fmaxf(scale_power(most), empty ? 0.0f : r.ref * power_of_two(b));
                top[u][c] = fmaxf(top[u][c], empty ? kEmpty : r.m[u][c] - b);
                apart.row(top[u][c], own[u][c], kEmpty);
            }
        ref = apart.reference(r.ref);
        r.bs = 0;
        float most = 0.0f;
#pragma unroll
        for (int u = 0; u < RG; ++u)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int b = top[u][c] == kEmpty ? 0 : max(power_between(ref, own[u][c]), 0);
                r.bs |= static_cast<uint32_t>(b) << (8 * (2 * u + c));
                top[u][c] += static_cast<float>(b);
                most = fmaxf(most, static_cast<float>(b));
            }
        r.slack = kSlack - warp_max(most);
    }
    const float down = r.ref * inverse(ref);
    r.ref = ref;
#pragma unroll
    for (int u = 0; u < RG; ++u) {
        float alpha[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            alpha[c] = r.m[u][c] == kEmpty ? 0.0f : ex2(r.m[u][c] - top[u][c]);
            r.m[u][c] = top[u][c];
            r.l[u][c] *= alpha[c];
            r.z[u][c] *= alpha[c];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = alpha[i & 1] * down;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) r.o[u][j][i] *= a;
        }
    }
}

// Tokens key0 .. key0 + 15, in shared memory, into the warp's rows.
template <int D, int RG>
__device__ __forceinline__ void take_tile(Rows<D, RG>& r, const uint4* q, const uint8_t* tile, int key0, bool inside, int g,
                                          int t) {
    uint32_t k[2][D / 32], kp[2], vp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int key = key_of(g) + 8 * i;
        load_words(k[i], tile + key * (D / 2) + t * (D / 8));
        kp[i] = reinterpret_cast<const uint32_t*>(tile + tile_pairs(D, 0))[key];
        vp[i] = reinterpret_cast<const uint32_t*>(tile + tile_pairs(D, 1))[key];
    }
    float a[RG][2][4];
#pragma unroll
    for (int u = 0; u < RG; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) a[u][i >> 2][i & 3] = 0.0f;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        const uint32_t k0 = k[0][w], k1 = k[1][w], h0 = k0 >> 8, h1 = k1 >> 8;
#pragma unroll
        for (int u = 0; u < RG; ++u) {
            const uint4 b = r.query(q, u, w);
            mma16816(a[u][0], k0 & 0x000f000fu, k1 & 0x000f000fu, k0 & 0x00f000f0u, k1 & 0x00f000f0u, b.x, b.y);
            mma16816(a[u][1], h0 & 0x000f000fu, h1 & 0x000f000fu, h0 & 0x00f000f0u, h1 & 0x00f000f0u, b.z, b.w);
        }
    }
    // (in flight meanwhile)
    uint32_t v[4][D / 64];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int key = key_of(2 * t + (i & 1) + 8 * (i >> 1));
        load_words(v[i], tile + tile_codes(D, 1) + key * (D / 2) + g * (D / 16));
    }
    float y[RG][2][2], s[2], z[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        s[i] = pair_scale(vp[i]);
        z[i] = pair_offset(vp[i]);
        const float ks = pair_scale(kp[i]), kz = pair_offset(kp[i]);
#pragma unroll
        for (int u = 0; u < RG; ++u)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                y[u][i][c] = fmaf(a[u][0][2 * i + c] + a[u][1][2 * i + c], ks * r.fq[u][c], kz * r.sq[u][c]);
    }
    if (!inside) {
        // tokens that a row does not see; what lies behind a sequence's last
        // token may be anything, a NaN included
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int key = key0 + key_of(g) + 8 * i;
            bool seen = false;
#pragma unroll
            for (int u = 0; u < RG; ++u)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const bool in = key >= r.first[u][c] && key <= r.last[u][c];
                    if (!in) y[u][i][c] = __uint_as_float(0xff800000u);
                    seen |= in;
                }
            if (!seen) s[i] = 0.0f, z[i] = 0.0f;
        }
    }
    bool more = s[0] >= 2.0f * r.ref || s[1] >= 2.0f * r.ref;
#pragma unroll
    for (int u = 0; u < RG; ++u)
#pragma unroll
        for (int c = 0; c < 2; ++c) more |= fmaxf(y[u][0][c], y[u][1][c]) > r.m[u][c] + r.slack;
    if (__any_sync(0xffffffffu, more)) raise<D, RG>(r, y, s, inside, key0 + key_of(g));
    const float f = kWeight * inverse(r.ref);
    uint32_t b[RG][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float sf = s[i] * f, zf = fmaf(8.0f, s[i], z[i]);
#pragma unroll
        for (int u = 0; u < RG; ++u) {
            float w[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                w[c] = ex2(y[u][i][c] - r.m[u][c]);
                r.l[u][c] += w[c];
                r.z[u][c] = fmaf(w[c], zf, r.z[u][c]);
            }
            b[u][i] = transpose8x8(half2_bits(w[0] * sf, w[1] * sf));
        }
    }
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __byte_perm(v[0][w], v[1][w], h ? 0x7632 : 0x5410);
            const uint32_t hi = __byte_perm(v[2][w], v[3][w], h ? 0x7632 : 0x5410);
            const uint32_t a0 = centred<0>(lo), a1 = centred<1>(lo), a2 = centred<0>(hi), a3 = centred<1>(hi);
#pragma unroll
            for (int u = 0; u < RG; ++u) mma16816(r.o[u][w * 4 + 2 * h], a0, a1, a2, a3, b[u][0], b[u][1]);
            const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
            const uint32_t c0 = centred<0>(lo8), c1 = centred<1>(lo8), c2 = centred<0>(hi8), c3 = centred<1>(hi8);
#pragma unroll
            for (int u = 0; u < RG; ++u) mma16816(r.o[u][w * 4 + 2 * h + 1], c0, c1, c2, c3, b[u][0], b[u][1]);
        }
    }
}

template <int D>
constexpr int so_row() {
    return D + 4;
}
// Shared memory: every warp's ring of tiles, in whose place the warps' results
// are joined, and the queries of 256 dims.
constexpr int kStages = 4;
template <int D>
constexpr size_t ring_bytes() {
    return static_cast<size_t>(kStages) * tile_bytes(D);
}
template <int D, int RG>
constexpr size_t q_at() {
    const size_t rings = kWarps<D, RG> * ring_bytes<D>();
    const size_t join = static_cast<size_t>(kWarps<D, RG>) * 8 * RG * (so_row<D>() + 2) * 4;
    return (rings > join ? rings : join) + 15 & ~size_t(15);
}
template <int D, int RG>
constexpr size_t smem_bytes() {
    return q_at<D, RG>() + (Rows<D, RG>::kShared ? RG * D * 16 : 0);
}

// A warp's tiles of a segment on their way through its ring: contiguous in memory, so
// that one lane's bulk copy brings one, three ahead of the one that is worked on.
// (Loads into registers, one tile ahead, left too few bytes on their way.)
struct Ring {
    uint8_t* at;
    uint64_t* bars;
    uint32_t count;  // tiles so far
    uint32_t bad;    // stages whose tile has no page
    bool stuck;      // a copy did not come: no further ones
};

// The segment of item `it` in tiles [t0, t1): every warp its own tiles, then
// joined.  `whole`: all of the item (the outputs are final), else its partial
// result goes to `slot`.
template <int D, int RG>
__device__ __forceinline__ void segment(const pq2h::AttendParams& p, const AttendWork& wk, const AttendItem& it, int t0,
                                        int t1, bool whole, int slot, uint8_t* shared, Ring& ring) {
    constexpr int kW = kWarps<D, RG>, kR = 8 * RG;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int per_page = p.cache.T / kTileTokens;
    const long long head_at = static_cast<long long>(it.head) * per_page * tile_bytes(D);
    const int mine = t1 - t0 > warp ? (t1 - t0 - warp + kW - 1) / kW : 0;
    // tiles that every row sees all of
    const int in0 = it.first_hi, in1 = it.last_lo;
    int page_lane = 0;
    const auto look_up = [&](int i) {  // pages of the warp's tiles i .. i + 31, one a lane
        const int tile = t0 + warp + kW * (i + lane);
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
    // tiles are asked for in order: the next one's place in its page
    const int step = kW % per_page;
    int in_page = (t0 + warp) % per_page;
    const auto fetch = [&](int i) {
        if ((i & 31) == 0) look_up(i);
        const int page = __shfl_sync(0xffffffffu, page_lane, i & 31), in = in_page;
        in_page += step;
        if (in_page >= per_page) in_page -= per_page;
        const uint32_t stage = (ring.count + i) % kStages;
        ring.bad = page < 0 ? ring.bad | (1u << stage) : ring.bad & ~(1u << stage);
        if (lane != 0 || static_cast<int>(ring.count + i) == p.ctl.debug_skip_stage) return;
        if (page < 0) {
            mbar_arrive(&ring.bars[stage]);
            return;
        }
        const uint8_t* from = p.cache.pool + page * p.cache.page_stride + head_at +
                              in * tile_bytes(D);
        mbar_arrive_expect_tx(&ring.bars[stage], tile_bytes(D));
        bulk_g2s(ring.at + stage * tile_bytes(D), from, tile_bytes(D), &ring.bars[stage]);
    };
    const auto wait = [&](uint32_t n) {
        unsigned long long since = 0;
        for (uint32_t i = 0; !__all_sync(0xffffffffu, mbar_try_wait(&ring.bars[n % kStages], (n / kStages) & 1)); ++i) {
            if (i % 64 != 63) continue;
            if (since == 0) since = globaltimer_ns();
            if (__any_sync(0xffffffffu, globaltimer_ns() - since > p.ctl.wait_limit_ns)) {
                if (lane == 0) atomicOr(p.ctl.err, DEVERR_TIMEOUT);
                return false;
            }
        }
        return true;
    };
    // the segment before's results, in the rings' place, have been read
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    if (!ring.stuck)
        for (int i = 0; i < min(kStages - 1, mine); ++i) fetch(i);
    Rows<D, RG> r;
    uint4* q = reinterpret_cast<uint4*>(shared + q_at<D, RG>()) + lane;
#pragma unroll
    for (int u = 0; u < RG; ++u) load_rows<D, RG>(r, q, p, it, u, g, t);
    clear<D, RG>(r);
    if constexpr (Rows<D, RG>::kShared) __syncthreads();
#pragma unroll 1
    for (int i = 0; i < mine && !ring.stuck; ++i) {
        if (i + kStages - 1 < mine) fetch(i + kStages - 1);
        const uint32_t n = ring.count + i, stage = n % kStages;
        if (!wait(n)) {
            // (not before the others are here, or have not come either)
            for (int k = 1; k < kStages && i + k < mine; ++k) wait(n + k);
            ring.stuck = true;
            break;
        }
        const int key0 = (t0 + warp + kW * i) * kTileTokens;
        if (!(ring.bad >> stage & 1))
            take_tile<D, RG>(r, q, ring.at + stage * tile_bytes(D), key0, key0 >= in0 && key0 + kTileTokens - 1 <= in1, g, t);
        __syncwarp();
    }
    ring.count += mine;
    float* smem = reinterpret_cast<float*>(shared);
    // the warps' results: [warp][row][D] with maxima and sums behind them
    float* so = smem;
    float* sm = smem + kW * kR * so_row<D>();
    float* sl = sm + kW * kR;
    __syncthreads();  // (other warps' tiles)
    const float f = r.ref / kWeight;
#pragma unroll
    for (int u = 0; u < RG; ++u)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float l = r.l[u][c], z = r.z[u][c];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l += __shfl_xor_sync(0xffffffffu, l, o);
                z += __shfl_xor_sync(0xffffffffu, z, o);
            }
            const int row = warp * kR + 8 * u + 2 * t + c;
            if (g == 0) sm[row] = r.m[u][c], sl[row] = l;
            float* to = so + row * so_row<D>() + g * (D / 8);
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                *reinterpret_cast<float2*>(to + 2 * j) =
                    make_float2(fmaf(r.o[u][j][c], f, z), fmaf(r.o[u][j][2 + c], f * 0.0625f, z));
        }
    __syncthreads();
    // warp w joins row w, a lane D / 32 dims of it
    for (int row = warp; row < kR; row += kW) {
    float m = kEmpty;
#pragma unroll
    for (int w = 0; w < kW; ++w) m = fmaxf(m, sm[w * kR + row]);
    float l = 0.0f, o[D / 32];
#pragma unroll
    for (int j = 0; j < D / 32; ++j) o[j] = 0.0f;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
        const float a = ex2(sm[w * kR + row] - m);
        l = fmaf(a, sl[w * kR + row], l);
        const float* from_w = so + (w * kR + row) * so_row<D>() + lane * (D / 32);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) o[j] = fmaf(a, from_w[j], o[j]);
    }
    const int d = lane * (D / 32);
    if (whole) {
        write_row<D / 32>(p, it, kR, row, d, l, o);
        continue;
    }
    const long long at = (static_cast<long long>(slot) * kR + row) * D + d;
    if (store_ok(p.ctl, at, D / 32, wk.o_elems)) {
#pragma unroll
        for (int j = 0; j < D / 32; j += 2) *reinterpret_cast<float2*>(wk.o + at + j) = make_float2(o[j], o[j + 1]);
    }
    if (lane == 0 && store_ok(p.ctl, slot * kR + row, 1, wk.ml_elems)) wk.ml[slot * kR + row] = make_float2(m, l);
    }
}

// The list's tiles, dealt out.
template <int D, int RG>
__global__ void __launch_bounds__(32 * kWarps<D, RG>, kBlocks<D>)
    attend_kernel(const __grid_constant__ pq2h::AttendParams p, const __grid_constant__ AttendWork wk) {
    constexpr int kR = 8 * RG;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint64_t bars[kWarps<D, RG>][kStages];
    pdl_wait();
    pdl_launch_dependents();
    // (the walk through the list is warp 0's: in registers of all threads it
    // would be in the way of the tiles')
    __shared__ AttendSpan walk;
    __shared__ AttendStep step;
    const int warp = threadIdx.x >> 5;
    Ring ring = {smem + warp * ring_bytes<D>(), bars[warp], 0, 0, false};
    if (threadIdx.x % 32 < kStages) mbar_init(&bars[warp][threadIdx.x % 32], 1);
    fence_mbar_init();
    __syncwarp();
    long long u, u1;
    {
        AttendSpan span;
        attend_span<kR, kWarps<D, RG>>(p, 1, kExtra<RG>, kWarps<D, RG>, span);
        if (threadIdx.x == 0) {
            walk = span;
            wk.join[blockIdx.x] = {0, 0, 0, 0, 0};
        }
        u = span.u0, u1 = span.u1;
    }
    for (int n = 0; u < u1; ++n) {
        __syncthreads();
        if (warp == 0) {
            AttendSpan span = walk;
            const AttendStep next = attend_step<kR>(p, 1, kExtra<RG>, span, u);
            __syncwarp();
            if (threadIdx.x == 0) step = next, walk = span;
        }
        __syncthreads();
        const AttendStep s = step;
        u += s.units;
        if (s.count == 0) continue;
        const AttendItem it = attend_item<kR>(p, s.b, s.row_tile, s.head);
        const int t0 = it.tile0 + s.first, slot = 2 * blockIdx.x + (n > 0);
        if (threadIdx.x == 0 && s.first == 0 && s.count < s.of)
            wk.join[blockIdx.x] = {s.b, s.row_tile, s.head,
                                   attend_cta_of(walk, s.end - 1) - static_cast<int>(blockIdx.x) + 1, slot};
        segment<D, RG>(p, wk, it, t0, min(t0 + s.count, it.tile1), s.count == s.of, slot, smem, ring);
    }
}

// CTA (c, row): row `row` of the item whose first part is CTA c's.  Every warp
// finds the weights of all parts, one a lane, and adds up every kJoinWarps-th part's
// outputs, a lane D / 32 dims.
constexpr int kJoinWarps = 8;

template <int D, int RG>
__global__ void __launch_bounds__(32 * kJoinWarps)
    attend_join_kernel(const __grid_constant__ pq2h::AttendParams p, const __grid_constant__ AttendWork wk) {
    constexpr int kN = D / 32, kR = 8 * RG;
    __shared__ float so[kJoinWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y;
    pdl_wait();
    pdl_launch_dependents();
    const AttendJoin j = wk.join[blockIdx.x];
    if (j.parts == 0) return;
    const auto place = [&](int i) {
        return static_cast<long long>(i == 0 ? j.first_slot : 2 * (static_cast<int>(blockIdx.x) + i)) * kR + row;
    };
    float m = kEmpty;
    for (int i = lane; i < j.parts; i += 32) m = fmaxf(m, wk.ml[place(i)].x);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    float l = 0.0f, o[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) o[k] = 0.0f;
    for (int i0 = 0; i0 < j.parts; i0 += 32) {
        float a = 0.0f;
        if (i0 + lane < j.parts) {
            const float2 ml = wk.ml[place(i0 + lane)];
            a = ex2(ml.x - m);
            l = fmaf(a, ml.y, l);
        }
#pragma unroll
        for (int k = 0; k < 32 / kJoinWarps; ++k) {
            const int i = warp + kJoinWarps * k;
            const float ai = __shfl_sync(0xffffffffu, a, i);
            if (i0 + i >= j.parts) continue;
            const float2* from = reinterpret_cast<const float2*>(wk.o + place(i0 + i) * D + lane * kN);
#pragma unroll
            for (int x = 0; x < kN / 2; ++x) {
                const float2 v = from[x];
                o[2 * x] = fmaf(ai, v.x, o[2 * x]);
                o[2 * x + 1] = fmaf(ai, v.y, o[2 * x + 1]);
            }
        }
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
#pragma unroll
    for (int k = 0; k < kN; ++k) so[warp][lane * kN + k] = o[k];
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
        for (int k = 0; k < kN; ++k) o[k] += so[w][lane * kN + k];
    const AttendItem it = attend_item<kR>(p, j.b, j.row_tile, j.head);
    write_row<D / 32>(p, it, kR, row, lane * (D / 32), l, o);
}

}  // namespace
}  // namespace pq2

namespace pq2h {

namespace {

size_t pad(size_t b) { return (b + 255) & ~size_t(255); }

template <int D, int RG>
cudaError_t launch_few(const AttendParams& p, const pq2::AttendWork& wk, cudaStream_t st, const DeviceInfo& dev) {
    static SmemLimit lim;
    const size_t smem = pq2::smem_bytes<D, RG>();
    cudaError_t e = raise_smem(lim, pq2::attend_kernel<D, RG>, smem);
    if (e != cudaSuccess) return e;
    const int64_t ctas = std::min<int64_t>(dev.num_sms * pq2::kBlocks<D>, pq2::kAttendCtas);
    e = launch(pq2::attend_kernel<D, RG>, dim3(static_cast<unsigned>(ctas)), dim3(32 * pq2::kWarps<D, RG>), smem, st, true, p, wk);
    if (e != cudaSuccess) return e;
    return launch(pq2::attend_join_kernel<D, RG>, dim3(static_cast<unsigned>(ctas), 8 * RG),
                  dim3(32 * pq2::kJoinWarps), 0, st, true, p, wk);
}

}  // namespace

size_t attend_workspace_bytes(int64_t M, int64_t q_heads, int64_t heads, int64_t dim) {
    const size_t rows = 2ull * pq2::kAttendCtas * pq2::kMostRows;
    const size_t few = pad(rows * dim * 4) + pad(rows * 8) + pad(pq2::kAttendCtas * sizeof(pq2::AttendJoin));
    return M * (q_heads / heads) > pq2::few_rows(dim) ? std::max(few, attend_many_workspace_bytes(M, q_heads, heads, dim)) : few;
}

cudaError_t launch_attend(const AttendParams& args, void* workspace, cudaStream_t st, const DeviceInfo& dev) {
    AttendParams p = args;
    const int64_t G = p.q_heads / p.cache.heads;
    p.over = -1, p.upto = INT_MAX;
    const bool many = p.max_rows * G > pq2::few_rows(p.dim);
    // one sequence has as many rows as the call; of several some may have few
    if (many && p.cache.B == 1) return launch_attend_many(p, workspace, st, dev);
    if (many) p.upto = pq2::few_rows(p.dim);
    pq2::AttendWork wk = {};
    wk.rows = pq2::kMostRows;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    const size_t rows = 2ull * pq2::kAttendCtas * pq2::kMostRows;
    wk.o = reinterpret_cast<float*>(w);
    wk.o_elems = rows * p.dim;
    w += pad(rows * p.dim * 4);
    wk.ml = reinterpret_cast<float2*>(w);
    wk.ml_elems = rows;
    w += pad(rows * 8);
    wk.join = reinterpret_cast<pq2::AttendJoin*>(w);
    const auto run = [&](auto rows) {
        constexpr int RG = decltype(rows)::value;
        switch (p.dim) {
            case 64: return launch_few<64, RG>(p, wk, st, dev);
            case 128: return launch_few<128, RG>(p, wk, st, dev);
        }
        return launch_few<256, RG>(p, wk, st, dev);
    };
    if (!many) return p.max_rows * G > 8 ? run(std::integral_constant<int, 2>()) : run(std::integral_constant<int, 1>());
    // Prompts and decoding sequences in one call: each to its kernel, one after the
    // other, in the same workspace.  2000 tokens behind 500, 40 heads of 128 on 8, with 256
    // sequences of one token behind 1000: 278 us, all by the other kernel 800; with 64 of 3 behind
    // 2000: 264 and 447; with 24 of 9 behind 3000: 309 and 320.  24 heads of 256 on 4 with
    // 256 of one: 279 and 380; with 24 of 5 behind 3000: 253 and 193 (the worst case of this rule).
    // 8 rows a pass: nothing bounds the rows of the short sequences, and most have one token.
    // With 16 the five took 325, 246, 275, 313 and 237 us.
    const cudaError_t e = run(std::integral_constant<int, 1>());
    if (e != cudaSuccess) return e;
    p.over = p.upto, p.upto = INT_MAX;
    return launch_attend_many(p, workspace, st, dev);
}

}  // namespace pq2h
