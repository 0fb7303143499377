// Low-rank adapters of many requests beside a shared projection:
//
//   v[m]  = A[id(m)] x[m]                       (rank values, fp32)
//   y'[m] = y[m] + scale[id(m)] * B[id(m)] v[m]
//
// A is [L][R][K], B [L][N][R], fp16 or bf16 like x; y is the projection's
// output.  Two kernels, "shrink" (x -> v) and "expand" (v -> y').
//
// Two forms:
//   few tokens (to 128 at most): every CTA finds its tile of at most 8 tokens of one
//     adapter itself, and expand adds up the K-split partials of shrink in a
//     fixed order.  Two launches.
//   more tokens: a plan kernel sorts the tokens by adapter into tiles of at
//     most 64 (stable counting sort in shared memory); shrink computes a tile
//     in a cluster of CTAs that split K and join their partials through
//     distributed shared memory; expand streams y and B through a ring in
//     shared memory against v's 16-bit terms.  Three launches.
// Results do not depend on which tokens share a tile: deterministic.
//
// The few-token form runs on the warp-level tensor instructions
// (mma.m16n8k16, fp32 accumulators) with the weights as the 16-row operand
// and the tokens as the 8 columns: a decode step has one or a few tokens per
// adapter, and 8 columns waste the least.  The sum index may be visited in
// any order, so a lane feeds the instructions from 16-byte loads of 8
// consecutive values (columns 8t .. 8t + 7 of a block of 32, t = lane % 4):
// the first instruction takes their first four, the second the others, the
// same for both operands.  Weights go from global memory straight to
// registers, with no shared-memory stage: each is used once per tile of
// tokens.  The planned form runs on tcgen05 with accumulators in tensor memory
// (shrink above 32 ranks; expand for fp32 y where two stages of its ring fit:
// up to rank 128, in tiles of 16 tokens any rank), else on the same
// instructions from shared memory.
//
// Precision.  v stays fp32 and would lose 13 bits (16 for bf16) as an operand
// of the expand product, so it enters as a sum of 16-bit terms: hi + lo for
// fp16 (22 bits below the largest |v| of the token; each token is scaled by a
// power of two, undone in fp32, so no term overflows), hi + mid + lo for
// bf16 (24 bits).  Tensor accumulation may round towards zero: chains are cut
// every 16 instructions and added up in fp32.
//
// Bounds: bytes.  Decode: A and B of the adapters in use; prompts: y in and
// out (8 N bytes per token against 2 K + 2 R (K + N) / tokens).  Measured: one
// token, rank 16, 5120 -> 17408: 4.6 us (the two launches); 48 tokens over 32
// adapters of rank 32, 6144 -> 5120: 11.4 us (1.7 TB/s); 4096 tokens, rank 64,
// 5120 -> 17408: 113.9 us (5.5 TB/s, 82% of the copy rate).
#include <algorithm>
#include <cstddef>
#include <type_traits>

#include <cuda_bf16.h>

#include "pq2_common.cuh"
#include "pq2_internal.h"
#include "pq2_step.cuh"

namespace pq2 {
namespace {

constexpr int kFewTokens = 128;
constexpr int kFewTile = 8;       // tokens per tile of the few-token form
constexpr int kTile = 64;        // tokens per tile of the planned form
constexpr int kSmallTile = 16;   // where adapters have few tokens each
constexpr int kShrinkWarps = 8;
constexpr int kExpandWarps = 4;   // 32 outputs each
constexpr int kExpandMaxWarps = 8;
constexpr int kMaxSplits = 64;
constexpr int kFlush = 8;        // k32 blocks (16 MMAs) per accumulator chain

// d += a . b (16 x 8 x 16), fp32 accumulators.
template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The two instructions of a block of 32: rows g and g + 8 from r0 and r1.
template <bool BF>
__device__ __forceinline__ void mma_block(float (&d)[4], const uint4& r0, const uint4& r1,
                                          const uint4& c) {
    mma16816<BF>(d, r0.x, r1.x, r0.y, r1.y, c.x, c.y);
    mma16816<BF>(d, r0.z, r1.z, r0.w, r1.w, c.z, c.w);
}

__device__ __forceinline__ uint4 zero4() { return make_uint4(0, 0, 0, 0); }

__device__ __forceinline__ uint4 load16(const uint16_t* p) {
    return *reinterpret_cast<const uint4*>(p);
}
// Past L1, for what a kernel reads before its dependency wait (or once).
__device__ __forceinline__ uint4 load16_cg(const uint16_t* p) {
    return __ldcg(reinterpret_cast<const uint4*>(p));
}

// Keeps the first n of 8 values (n <= 0: none): a row's padding may hold
// anything, NaN included.
__device__ __forceinline__ uint4 keep_first(uint4 v, int n) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (2 * i >= n) w[i] = 0;
        else if (2 * i + 1 >= n) w[i] &= 0xffffu;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ int rank_of(const pq2h::LoraParams& p, int l) {
    return p.ranks ? max(0, min(__ldcg(p.ranks + l), p.R)) : p.R;
}

// Adapter of token m: -1 if none.
__device__ __forceinline__ int adapter_of(const pq2h::LoraParams& p, int m, bool report) {
    const int id = __ldcg(p.ids + m);
    if (id >= p.L) {
        if (report) atomicOr(p.ctl.err, DEVERR_BAD_INDEX);
        return -1;
    }
    return id < 0 ? -1 : id;
}

// The few-token form's tiles: the tokens of an adapter in their order, cut by
// eights; a tile counts where its first token stands.  Every CTA works out its
// own tile (the ids are one load, the rest is a few hundred instructions)
// instead of waiting for another kernel to do it.  kNone: tokens without an
// adapter form tiles too (adapter -1).
struct alignas(16) FewTile {
    int ids[kFewTokens];    // read by fours: on its 16 bytes
    int tok[kFewTile];
    int adapter;
    int count;              // 0: there is no such tile
    int starts[kFewTokens / 32];
    int sel[2];
};
static_assert(offsetof(FewTile, ids) % 16 == 0, "int4 reads");
// All threads of the CTA (at least 128 of them where M > 32); the answer is
// in `f` after the last barrier.
template <bool kNone>
__device__ __forceinline__ void find_tile(const pq2h::LoraParams& p, int index, bool report,
                                          FewTile& f) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.M <= 32) {
        if (warp == 0) {
            const int id = lane < p.M ? adapter_of(p, lane, report) : -2;
            const unsigned same = __match_any_sync(0xffffffffu, id);
            const int rank = __popc(same & ((1u << lane) - 1u));
            const bool starts = (kNone ? id >= -1 : id >= 0) && rank % kFewTile == 0;
            unsigned lead = __ballot_sync(0xffffffffu, starts);
            for (int k = 0; k < index; ++k) lead &= lead - 1;
            const int src = lead ? __ffs(lead) - 1 : 0;
            const int sid = __shfl_sync(0xffffffffu, id, src), sr = __shfl_sync(0xffffffffu, rank, src);
            const bool member = lead && id == sid && rank / kFewTile == sr / kFewTile;
            const unsigned all = __ballot_sync(0xffffffffu, member);
            if (member) f.tok[rank % kFewTile] = lane;
            if (lane == 0) f.adapter = sid, f.count = __popc(all);
        }
        __syncthreads();
        return;
    }
    const int id = tid < p.M ? adapter_of(p, tid, report) : -2;
    if (tid < kFewTokens) f.ids[tid] = id;
    if (tid == 0) f.sel[0] = -3;
    __syncthreads();
    int rank = 0;
    if (tid < p.M) {
        const int4* v = reinterpret_cast<const int4*>(f.ids);
        for (int j = 0; j < tid / 4; ++j) {
            const int4 q = v[j];
            rank += (q.x == id) + (q.y == id) + (q.z == id) + (q.w == id);
        }
        for (int j = tid / 4 * 4; j < tid; ++j) rank += f.ids[j] == id;
    }
    const bool starts = tid < p.M && (kNone ? id >= -1 : id >= 0) && rank % kFewTile == 0;
    const unsigned lead = __ballot_sync(0xffffffffu, starts);
    if (lane == 0 && warp < kFewTokens / 32) f.starts[warp] = __popc(lead);
    __syncthreads();
    if (starts) {
        int at = __popc(lead & ((1u << lane) - 1u));
        for (int w = 0; w < warp; ++w) at += f.starts[w];
        if (at == index) f.sel[0] = id, f.sel[1] = rank / kFewTile;
    }
    __syncthreads();
    const bool member = tid < p.M && id == f.sel[0] && rank / kFewTile == f.sel[1];
    if (member) f.tok[rank % kFewTile] = tid;
    const int count = __syncthreads_count(member);
    if (tid == 0) f.adapter = f.sel[0], f.count = count;
    __syncthreads();
}
// Tiles there can be among M tokens of L adapters.
constexpr int64_t few_tiles(int64_t M, int64_t groups) {
    return groups + M / kFewTile < M ? groups + M / kFewTile : M;
}

// v's token as 16-bit terms.  fp16: the token is scaled by 2^-e first.
template <bool BF>
__device__ __forceinline__ void split_terms(float v, uint16_t (&t)[3]) {
    if constexpr (BF) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const __nv_bfloat16 h = __float2bfloat16_rn(v);
            t[i] = *reinterpret_cast<const uint16_t*>(&h);
            v -= __bfloat162float(h);
        }
    } else {
        const __half h = __float2half_rn(v);
        t[0] = __half_as_ushort(h);
        t[1] = __half_as_ushort(__float2half_rn(v - __half2float(h)));
        t[2] = 0;
    }
}
template <bool BF>
constexpr int terms() {
    return BF ? 3 : 2;
}

// 2^e with e the exponent of the token's largest |v| (kept in the range where
// 2^e and 2^-e are normal numbers); 1 for bf16, whose terms have fp32's range.
template <bool BF>
__device__ __forceinline__ float pow2_below(float top) {
    if constexpr (BF) return 1.0f;
    const int e = min(max(static_cast<int>((__float_as_uint(top) >> 23) & 0xff), 27), 227);
    return top > 0.0f ? __uint_as_float(static_cast<uint32_t>(e) << 23) : 1.0f;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// Rows of v's terms in shared memory: a block of 32 ranks is 16 words; an
// odd number of 16-word blocks per row keeps the 16-byte reads of two
// neighbouring tokens in different banks.
__host__ __device__ __forceinline__ int term_pitch(int blocks) { return (blocks | 1) * 32; }

// ----------------------------------------------------------------------------
// shrink
// ----------------------------------------------------------------------------

// Warps per rank tile of 16 within a CTA (the others split K).
__device__ __forceinline__ int k_warps(int rank_tiles) {
    return rank_tiles == 1 ? 8 : rank_tiles == 2 ? 4 : rank_tiles <= 4 ? 2 : 1;
}

// Few tokens: CTA (split, tile): the ranks of the tile's adapter times its
// tokens over one share of K, straight from global memory, eight blocks of 32
// columns in flight per warp.  part [splits][M][R].
template <bool BF>
__global__ void __launch_bounds__(kShrinkWarps * 32)
    lora_shrink_few(pq2h::LoraParams p, float* part, int k_split) {
    __shared__ float red[kShrinkWarps * 16 * kFewTile];
    __shared__ FewTile tile;
    pdl_wait();
    pdl_launch_dependents();
    find_tile<false>(p, blockIdx.y, blockIdx.x + blockIdx.y == 0, tile);
    const int count = tile.count, l = tile.adapter;
    if (count == 0) return;  // uniform over the CTA
    const int rank = rank_of(p, l);
    const int k0 = blockIdx.x * k_split, k1 = min(k0 + k_split, p.K);
    const long long out0 = static_cast<long long>(blockIdx.x) * p.M * p.R;
    const long long part_elems = static_cast<long long>(gridDim.x) * p.M * p.R;
    const auto put = [&](int j, int r, float v) {
        const long long o = out0 + static_cast<long long>(tile.tok[j]) * p.R + r;
        if (store_ok(p.ctl, o, 1, part_elems)) part[o] = v;
    };
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int rank_tiles = (rank + 15) / 16;
    const int kw = k_warps(rank_tiles);
    const int per_round = kShrinkWarps / kw;
    const int ks = warp % kw;
    const uint16_t* x = g < count ? p.x + static_cast<size_t>(tile.tok[g]) * p.ld_x : nullptr;
    // more than one round only with kw == 1, where `red` is not used
    for (int rt = warp / kw; rt < rank_tiles; rt += per_round) {
        const int ra = rt * 16 + g, rb = ra + 8;
        const uint16_t* a0 = p.A + (static_cast<size_t>(l) * p.R + ra) * p.K;
        const uint16_t* a1 = a0 + static_cast<size_t>(8) * p.K;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        constexpr int U = kFlush;  // blocks in flight, and in a chain
        for (int kb = k0 + ks * 32; kb < k1; kb += kw * 32 * U) {
            uint4 fa[U], fb[U], fx[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = kb + u * kw * 32 + 8 * t;
                fa[u] = k < k1 && ra < rank ? load16(a0 + k) : zero4();
                fb[u] = k < k1 && rb < rank ? load16(a1 + k) : zero4();
                fx[u] = k < k1 && x ? load16(x + k) : zero4();
            }
            // four accumulators: a dependent instruction waits some 150 cycles
            float acc[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][c] = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float(&lo)[4] = acc[u % 2 * 2];
                float(&hi)[4] = acc[u % 2 * 2 + 1];
                mma16816<BF>(lo, fa[u].x, fb[u].x, fa[u].y, fb[u].y, fx[u].x, fx[u].y);
                mma16816<BF>(hi, fa[u].z, fb[u].z, fa[u].w, fb[u].w, fx[u].z, fx[u].w);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[c] += (acc[0][c] + acc[1][c]) + (acc[2][c] + acc[3][c]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int r = (c >> 1) * 8 + g, j = 2 * t + (c & 1);
            if (kw > 1)
                red[(warp * 16 + r) * kFewTile + j] = sum[c];
            else if (j < count && rt * 16 + r < rank)
                put(j, rt * 16 + r, sum[c]);
        }
    }
    if (kw > 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < rank_tiles * 16 * count; i += kShrinkWarps * 32) {
            const int r = i % (rank_tiles * 16), j = i / (rank_tiles * 16);
            if (r >= rank) continue;
            const float* src = red + ((r / 16) * kw * 16 + r % 16) * kFewTile + j;
            float v = 0.0f;
            for (int w = 0; w < kw; ++w) v += src[w * 16 * kFewTile];
            put(j, r, v);
        }
    }
}

// ----------------------------------------------------------------------------
// expand
// ----------------------------------------------------------------------------

// Four consecutive values of y (n .. n + 3 of a row).
template <int YT>
__device__ __forceinline__ float4 y_load(const void* y, size_t i, int left, bool vec) {
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (YT == PQ2_F32) {
        const float* s = static_cast<const float*>(y) + i;
        if (vec && left >= 4) return __ldcg(reinterpret_cast<const float4*>(s));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < left) v[j] = __ldcg(s + j);
    } else {
        const uint16_t* s = static_cast<const uint16_t*>(y) + i;
        if (vec && left >= 4) {
            const uint2 u = __ldcg(reinterpret_cast<const uint2*>(s));
            return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                               __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < left) v[j] = __uint_as_float(static_cast<uint32_t>(__ldcg(s + j)) << 16);
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

template <int YT>
__device__ __forceinline__ void y_store(const pq2h::LoraParams& p, size_t i, int left, bool vec,
                                        const float4& v) {
    const long long elems = static_cast<long long>(p.M - 1) * p.ld_out + p.N;
    const float w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (YT == PQ2_F32) {
        float* d = static_cast<float*>(p.y_out) + i;
        if (vec && left >= 4) {
            if (store_ok(p.ctl, i, 4, elems)) *reinterpret_cast<float4*>(d) = v;
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < left && store_ok(p.ctl, i + j, 1, elems)) d[j] = w[j];
    } else {
        uint16_t* d = static_cast<uint16_t*>(p.y_out) + i;
        if (vec && left >= 4) {
            if (store_ok(p.ctl, i, 4, elems))
                *reinterpret_cast<uint2*>(d) = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < left && store_ok(p.ctl, i + j, 1, elems))
                d[j] = static_cast<uint16_t>(bf16x2(w[j], 0.0f) & 0xffffu);
    }
}

// The four rows of B of this lane (outputs n .. n + 3) in block `blk` of 32
// ranks: rows g and g + 8 of two instructions' operands.
struct BRows {
    uint4 r[4];
};
__device__ __forceinline__ BRows b_load(const pq2h::LoraParams& p, int l, int rank, int n, int blk) {
    BRows b;
    const int r0 = blk * 32 + 8 * (threadIdx.x & 3);
    const int left = rank - r0;
    const uint16_t* src = p.B + (static_cast<size_t>(l) * p.N + n) * p.R + r0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        b.r[i] = left > 0 && n + i < p.N ? load16_cg(src + static_cast<size_t>(i) * p.R) : zero4();
    }
    // only a rank that is no multiple of 8 leaves a piece half used (asking
    // about a value just loaded would wait for it)
    if (rank % 8 != 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) b.r[i] = keep_first(b.r[i], left);
    }
    return b;
}

// acc += B rows x v terms of one block of 32 ranks, for NT groups of 8
// tokens (those below `count`).  sv: terms of token 0, block 0.
template <bool BF, int NT>
__device__ __forceinline__ void expand_block(float (&acc)[2][NT][4], const BRows& b,
                                             const uint16_t* sv, int pitch, int term_size, int blk,
                                             int count) {
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        if (i * 8 >= count) break;
        const uint16_t* src = sv + (i * 8 + g) * pitch + blk * 32 + 8 * t;
#pragma unroll
        for (int q = 0; q < terms<BF>(); ++q) {
            const uint4 c = *reinterpret_cast<const uint4*>(src + q * term_size);
            mma_block<BF>(acc[0][i], b.r[0], b.r[1], c);
            mma_block<BF>(acc[1][i], b.r[2], b.r[3], c);
        }
    }
}

// y' = y + f acc for this lane's two tokens of each group of 8 (f: scale and
// the token's power of two).
template <int YT, int NT>
__device__ __forceinline__ void expand_store(const pq2h::LoraParams& p, const float (&acc)[2][NT][4],
                                             const float4 (&y)[NT][2], const int* tok,
                                             const float* f, int count, int n, bool vec) {
    const int t = threadIdx.x & 3;
    if (n >= p.N) return;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = i * 8 + 2 * t + h;
            if (j >= count) continue;
            const float s = f[j];
            float4 o = y[i][h];
            o.x = fmaf(s, acc[0][i][h], o.x);
            o.y = fmaf(s, acc[0][i][2 + h], o.y);
            o.z = fmaf(s, acc[1][i][h], o.z);
            o.w = fmaf(s, acc[1][i][2 + h], o.w);
            y_store<YT>(p, static_cast<size_t>(tok[j]) * p.ld_out + n, p.N - n, vec, o);
        }
}

template <int YT, int NT>
__device__ __forceinline__ void y_fetch(const pq2h::LoraParams& p, float4 (&y)[NT][2], const int* tok,
                                        int count, int n, bool vec) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = i * 8 + 2 * t + h;
            y[i][h] = j < count && n < p.N
                          ? y_load<YT>(p.y_in, static_cast<size_t>(tok[j]) * p.ld_in + n, p.N - n, vec)
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
}

// Rounds a CTA from which a round's lines are asked for as whole lines, before
// its loads take them in pieces of 64 bytes (us with and without: 64 tokens over
// 64 adapters of rank 64, 17408 outputs, 17 rounds, 50.0 and 52.2; 32 over 32 of
// rank 128 41.0 and 42.7; at 4 rounds, 48 tokens over 32 adapters of rank 32,
// 5120 outputs, 10.8 and 10.5).
constexpr int kAskRounds = 8;

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Few tokens: CTA (32 outputs a warp, tile).  The operands that do not come
// from shrink (B, y) are loaded before the dependency wait: shrink lets this
// kernel start only after its own wait, so everything before it is done.
// kOne: the adapters' rows of B are one block of 32 ranks, and the next
// round's operands are loaded during this one (64 requests with adapters of
// rank 16, 17408 outputs: 33 us against 44).  Else two blocks of this round
// are.
template <bool BF, int YT, bool kOne>
__global__ void __launch_bounds__(kExpandMaxWarps * 32)
    lora_expand_few(pq2h::LoraParams p, const float* part, int splits, int rounds, int vec) {
    extern __shared__ __align__(16) uint16_t sv[];
    __shared__ FewTile tile;
    __shared__ float f[kFewTile];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    find_tile<true>(p, blockIdx.y, false, tile);
    const int count = tile.count, l = tile.adapter;
    const int* tok = tile.tok;
    if (count == 0) {  // uniform over the CTA
        pdl_wait();
        return;
    }
    const int rank = l >= 0 ? rank_of(p, l) : 0;
    const int blocks = (rank + 31) / 32;
    // this warp's outputs: 32 a round, the rounds a CTA's width apart
    const int step = nwarps * 32;
    int n = blockIdx.x * rounds * step + warp * 32 + 4 * (lane >> 2);
    constexpr int kAhead = 2;  // blocks of B in registers
    BRows b[kAhead];
    float4 y[kOne ? 2 : 1][1][2];
    const auto load_b = [&](int slot, int blk, int at) {
        if (blk < blocks) b[slot] = b_load(p, l, rank, at, blk);
    };
    load_b(0, 0, n);
    if (!kOne) load_b(1, 1, n);
    y_fetch<YT, 1>(p, y[0], tok, count, n, vec != 0);
    // the lines of a round: B a row per lane, y a token per lane
    const auto ask = [&](int first) {   // the warp's first output there
        if (first + lane < p.N) {
            const uint8_t* rows = reinterpret_cast<const uint8_t*>(
                p.B + (static_cast<size_t>(max(l, 0)) * p.N + first + lane) * p.R);
            for (int c = 0; c < rank * 2; c += 128) prefetch_l2(rows + c);
        }
        if (lane < count && first < p.N)
            prefetch_l2(static_cast<const uint8_t*>(p.y_in) +
                        (static_cast<size_t>(tok[lane]) * p.ld_in + first) * (YT == PQ2_F32 ? 4 : 2));
    };
    const int first = n - 4 * (lane >> 2);
    const bool asks = rounds >= kAskRounds;
    const float scale = l >= 0 && p.scales ? __ldcg(p.scales + l) : 1.0f;

    pdl_wait();
    pdl_launch_dependents();
    // v: the K-split partials in order, a warp per token and 32 ranks; then the
    // token's 16-bit terms
    const int pitch = term_pitch((p.R + 31) / 32), term_size = kFewTile * pitch;
    float* sf = reinterpret_cast<float*>(sv + terms<BF>() * term_size);   // [token][blocks][32]
    for (int i = warp; i < count * blocks; i += nwarps) {
        const int j = i / blocks, r = i % blocks * 32 + lane;
        float v = 0.0f;
        if (r < rank) {
            const float* src = part + static_cast<size_t>(tok[j]) * p.R + r;
            const size_t step = static_cast<size_t>(p.M) * p.R;
            for (int s0 = 0; s0 < splits; s0 += 16) {
                float w[16];
#pragma unroll
                for (int s = 0; s < 16; ++s) w[s] = s0 + s < splits ? src[(s0 + s) * step] : 0.0f;
#pragma unroll
                for (int s = 0; s < 16; ++s) v += w[s];
            }
        }
        sf[i * 32 + lane] = v;
    }
    __syncthreads();
    for (int j = warp; j < count && blocks > 0; j += nwarps) {
        float top = 0.0f;
        for (int i = 0; i < blocks; ++i) top = fmaxf(top, fabsf(sf[(j * blocks + i) * 32 + lane]));
        const float up = pow2_below<BF>(warp_max(top)), down = 1.0f / up;
        for (int i = 0; i < blocks; ++i) {
            uint16_t w[3];
            split_terms<BF>(sf[(j * blocks + i) * 32 + lane] * down, w);
#pragma unroll
            for (int q = 0; q < terms<BF>(); ++q)
                sv[q * term_size + j * pitch + i * 32 + lane] = w[q];
        }
        if (lane == 0) f[j] = scale * up;
    }
    if (blocks == 0) {
        if (p.y_in == p.y_out && p.ld_in == p.ld_out) return;
        if (threadIdx.x < kFewTile) f[threadIdx.x] = 0.0f;
    }
    __syncthreads();
    // an accumulator for either half of a block: a dependent instruction waits
    // some 150 cycles
    float acc[2][1][4], half[2][4];
    const auto clear = [&] {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[h][0][c] = half[h][c] = 0.0f;
    };
    const auto product = [&](const BRows& rows, int blk) {
        const uint16_t* src = sv + (lane >> 2) * pitch + blk * 32 + 8 * (lane & 3);
        const uint4* r = rows.r;
#pragma unroll
        for (int q = 0; q < terms<BF>(); ++q) {
            const uint4 c = *reinterpret_cast<const uint4*>(src + q * term_size);
            mma16816<BF>(acc[0][0], r[0].x, r[1].x, r[0].y, r[1].y, c.x, c.y);
            mma16816<BF>(acc[1][0], r[2].x, r[3].x, r[2].y, r[3].y, c.x, c.y);
            mma16816<BF>(half[0], r[0].z, r[1].z, r[0].w, r[1].w, c.z, c.w);
            mma16816<BF>(half[1], r[2].z, r[3].z, r[2].w, r[3].w, c.z, c.w);
        }
    };
    const auto store = [&](const float4(&yv)[1][2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[h][0][c] += half[h][c];
        expand_store<YT, 1>(p, acc, yv, tok, f, count, n, vec != 0);
    };
    for (int round = 0; round < rounds; round += kOne ? 2 : 1) {
        // a warp past the end of the row loads and stores nothing
        if constexpr (kOne) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (round + s >= rounds) return;
                if (round + s + 1 < rounds) {
                    if (asks) ask(first + (round + s + 1) * step);
                    load_b(1 - s, 0, n + step);
                    y_fetch<YT, 1>(p, y[1 - s], tok, count, n + step, vec != 0);
                }
                clear();
                if (blocks > 0) product(b[s], 0);
                store(y[s]);
                n += step;
            }
        } else {
            if (round > 0) {
                if (asks) ask(first + round * step);
                load_b(0, 0, n);
                load_b(1, 1, n);
                y_fetch<YT, 1>(p, y[0], tok, count, n, vec != 0);
            }
            clear();
            for (int blk = 0; blk < blocks; blk += kAhead) {
                if (blk > 0) {
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) load_b(i, blk + i, n);
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    if (blk + i < blocks) product(b[i], blk + i);
            }
            store(y[0]);
            n += step;
        }
    }
}

// ----------------------------------------------------------------------------
// More tokens: plan, shrink, expand over tiles
// ----------------------------------------------------------------------------

struct Plan {
    int* perm;           // [M] tokens, sorted by adapter
    int4* tiles;         // adapter (-1: none), first position, tokens, rank
    int* num_tiles;      // [0] tiles, [1] those with an adapter
    int tile;            // tokens of a tile, at most: kTile or kSmallTile
    unsigned* taken;     // times that expand took items from the counter
    uint16_t* terms;     // [terms][M][rp], by position
    float* f;            // [M] scale and power of two, by position
    int max_tiles;
    int rp;              // R rounded up to 32
};

// One CTA: stable counting sort of the tokens by adapter (tokens without one
// last), cut into tiles of at most pl.tile.  Every warp counts and places a
// contiguous range of tokens in its own histogram, so the order is fixed.
// Bound by its chain of barriers and shared-memory trips: 3 us for 333 tokens,
// 6 for 4096.
// ranks_here: there is room for the bins' ranks too (else they are asked for
// again, a trip to L2 a bin).
__global__ void __launch_bounds__(1024) lora_plan_kernel(pq2h::LoraParams p, Plan pl, int warps,
                                                         int ranks_here) {
    // [warps][bins], then offsets [bins + 1], tiles [bins] and ranks [bins]
    extern __shared__ int hist[];
    __shared__ int ws[2][32];
    const int bins = p.L + 1;
    int* off = hist + warps * bins;
    int* tfirst = off + bins + 1;
    int* rank = tfirst + bins;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nthreads = blockDim.x;
    for (int i = threadIdx.x; i < warps * bins; i += nthreads) hist[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    const int per = ((p.M + warps - 1) / warps + 31) / 32 * 32;
    const int m0 = warp * per, m1 = min(m0 + per, p.M);
    int* mine = hist + warp * bins;
    // each thread's bins: their ranks are on the way meanwhile
    const int span = (bins + nthreads - 1) / nthreads;
    const int b0 = min(static_cast<int>(threadIdx.x) * span, bins), b1 = min(b0 + span, bins);
    const int first_rank = b0 < b1 && b0 < p.L ? rank_of(p, b0) : 0;
    // the tokens four at a time a lane, loaded together
    constexpr int kBatch = 4;
    int keys[kBatch];
    unsigned same[kBatch];   // lanes with the same key
    auto load_keys = [&](int base, bool report) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int m = base + i * 32 + lane;
            keys[i] = m < m1 ? adapter_of(p, m, report) : -2;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            keys[i] = keys[i] == -1 ? p.L : keys[i];
            same[i] = __match_any_sync(0xffffffffu, keys[i]);
        }
    };
    for (int base = m0; base < m1; base += 32 * kBatch) {
        load_keys(base, true);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (base + i * 32 >= m1) break;
            if (keys[i] >= 0 && __ffs(same[i]) - 1 == lane) mine[keys[i]] += __popc(same[i]);
            __syncwarp();
        }
    }
    __syncthreads();
    // a warp per bin: its counts by warp to offsets within the bin
    const int nwarps = nthreads >> 5;
    for (int b = warp; b < bins; b += nwarps) {
        const int c = lane < warps ? hist[lane * bins + b] : 0;
        int sum = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (lane < warps) hist[lane * bins + b] = sum - c;
        if (lane == 31) off[b] = sum;
    }
    __syncthreads();
    // a scan over the bins, each thread owning a contiguous span
    int n_tok = 0, n_tile = 0;
    for (int b = b0; b < b1; ++b) {
        if (ranks_here) rank[b] = b == b0 ? first_rank : b < p.L ? rank_of(p, b) : 0;
        n_tok += off[b];
        n_tile += (off[b] + pl.tile - 1) / pl.tile;
    }
    int s_tok = n_tok, s_tile = n_tile;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, s_tok, o), c = __shfl_up_sync(0xffffffffu, s_tile, o);
        if (lane >= o) s_tok += v, s_tile += c;
    }
    if (lane == 31) ws[0][warp] = s_tok, ws[1][warp] = s_tile;
    __syncthreads();
    int at_tok = s_tok - n_tok, at_tile = s_tile - n_tile;
    for (int w = 0; w < warp; ++w) at_tok += ws[0][w], at_tile += ws[1][w];
    for (int b = b0; b < b1; ++b) {
        const int total = off[b];
        off[b] = at_tok;
        tfirst[b] = at_tile;
        // tokens without an adapter come last: the tiles before theirs.  By this
        // bin's own thread; the last thread's count of all tiles needs no other's
        if (b == p.L) pl.num_tiles[1] = at_tile;
        at_tok += total;
        at_tile += (total + pl.tile - 1) / pl.tile;
    }
    if (threadIdx.x == nthreads - 1) {
        pl.num_tiles[0] = at_tile;
        *pl.taken = 0u;
        off[bins] = p.M;
    }
    __syncthreads();
    // tiles: a warp per bin again
    for (int b = warp; b < bins; b += nwarps) {
        const int first = off[b], total = off[b + 1] - first;
        if (total == 0) continue;
        const int r = ranks_here ? rank[b] : b < p.L ? rank_of(p, b) : 0;
        for (int k = lane * pl.tile; k < total; k += 32 * pl.tile)
            pl.tiles[tfirst[b] + k / pl.tile] =
                make_int4(b < p.L ? b : -1, first + k, min(pl.tile, total - k), r);
    }
    for (int base = m0; base < m1; base += 32 * kBatch) {
        if (per > 32 * kBatch) load_keys(base, false);   // else still there
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (base + i * 32 >= m1) break;
            const int key = keys[i], leader = __ffs(same[i]) - 1;
            int at = 0;
            if (key >= 0 && leader == lane) {
                at = mine[key];
                mine[key] = at + __popc(same[i]);
            }
            at = __shfl_sync(0xffffffffu, at, leader);
            if (key >= 0)
                pl.perm[off[key] + at + __popc(same[i] & ((1u << lane) - 1u))] = base + i * 32 + lane;
            __syncwarp();
        }
    }
}

// 16-byte asynchronous copy to shared memory; `bytes` 0 writes zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
// Asynchronous copy of 4 or 16 bytes to shared memory.
template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// One arrival on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every CTA's earlier stores to shared memory are visible to the cluster.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// First phase of the barrier apart: this CTA has started (and orders nothing).
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

constexpr int kTcNB = 128;          // rows of a product's first operand

// Matrix descriptor: K-major, 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(1) << 16;             // leading offset (unused here)
    d |= static_cast<uint64_t>(1024 >> 4) << 32;     // stride offset
    d |= static_cast<uint64_t>(1) << 46;             // descriptor version
    d |= static_cast<uint64_t>(2) << 61;             // 128-byte swizzle
    return d;
}

// D[128 x T] (+)= A[128 x 16] . B[T x 16]^T; both operands fp16, or both bf16.
template <bool BF, int T>
__device__ __forceinline__ void tc_mma(uint32_t d_tmem, uint64_t a, uint64_t b, bool add) {
    constexpr uint32_t idesc = (1u << 4) | ((BF ? 1u : 0u) << 7) | ((BF ? 1u : 0u) << 10) |
                               (static_cast<uint32_t>(T >> 3) << 17) |
                               (static_cast<uint32_t>(kTcNB >> 4) << 24);
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u));
}
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_ld(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_ld(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_ld(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

constexpr int kStageK = 64;         // columns of K per pipeline stage: rows of 128 bytes
constexpr int kFlushStages = kFlush * 32 / kStageK;
constexpr int kShrinkMaxStages = 8;
constexpr int kShrinkLoaders = 4;

// The loader warps' share (pt: thread of them): stages of 64 columns from k0 to
// k1.  Thread -> chunk `chunk` of rows row0 + 16 i, the first of them to dst0.
__device__ __forceinline__ void shrink_load(const pq2h::LoraParams& p, const Plan& pl,
                                            const CUtensorMap* map_a, uint8_t* smem, uint64_t* full,
                                            uint64_t* empty, int stages, int stage_bytes, int steps,
                                            int k0, int k1, int l, int rank, int first, int count,
                                            int pt, int chunk, int row0, uint32_t dst0,
                                            volatile int* abort_flag) {
    const int lane = pt & 31;
    // Rows past the rank or the tile hold anything: a row of A only reaches its
    // own rank's sums, a row of x its own token's, and those are not stored.
    // Columns past K enter every sum: zeros, in x here and in A past the map's
    // end (a share of K ends on a multiple of 64 otherwise).
    constexpr int kRows = kShrinkLoaders * 4;   // rows per round
    constexpr int kXRounds = kTile / kRows;
    const uint16_t* xs[kXRounds];
#pragma unroll
    for (int i = 0; i < kXRounds; ++i) {
        const int j = row0 + kRows * i;
        xs[i] = j < count ? p.x + static_cast<size_t>(pl.perm[first + j]) * p.ld_x + k0 + chunk * 8
                          : nullptr;
    }
    const int boxes = (rank + 15) / 16;
    int s = 0, issued = 0;
    uint32_t turn = 0;
    for (; issued < steps; ++issued) {
        if (turn > 0 && !mbar_ready_warp(&empty[s], (turn - 1) & 1, p.ctl, abort_flag)) break;
        if (issued != p.ctl.debug_skip_stage) {  // else withheld (timeout test)
            const uint32_t st = dst0 + s * stage_bytes;
            const int k = issued * kStageK;
            if (pt < 32) {
                if (lane == 0) mbar_arrive_expect_tx(&full[s], boxes * 16 * 128);
                __syncwarp();
                if (lane < boxes)
                    tma_load_2d(smem + s * stage_bytes + (kTile + lane * 16) * 128, map_a, k0 + k,
                                l * p.R + lane * 16, &full[s]);
            }
            if (k0 + k + kStageK <= k1) {
#pragma unroll
                for (int i = 0; i < kXRounds; ++i)
                    if (xs[i]) cp_async<16>(st + i * kRows * 128, xs[i] + k);
            } else {
                const bool in = k0 + k + chunk * 8 < k1;
#pragma unroll
                for (int i = 0; i < kXRounds; ++i)
                    if (xs[i]) cp_async16(st + i * kRows * 128, in ? xs[i] + k : p.x, in ? 16 : 0);
            }
            cp_async_arrive(&full[s]);
        }
        if (++s == stages) s = 0, ++turn;
    }
    // the last copies land before the CTA ends, whatever the others do
    for (int k = max(0, issued - stages); k < issued; ++k)
        if (k != p.ctl.debug_skip_stage)
            mbar_ready_warp(&full[k % stages], static_cast<uint32_t>(k / stages) & 1, p.ctl);
    cp_async_wait<0>();
}

// The cluster's partials of this CTA's tokens (in its inbox, [from CTA][token /
// splits][r16]) added up in order, scaled and split into 16-bit terms, a warp
// per token.
template <bool BF>
__device__ __forceinline__ void shrink_finish(const pq2h::LoraParams& p, const Plan& pl, const float* inbox,
                                              int part, int splits, int per_cta, int r16, int l,
                                              int rank, int first, int count, int warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float scale = p.scales ? p.scales[l] : 1.0f;
    const size_t term_size = static_cast<size_t>(p.M) * pl.rp;
    const int blocks = (rank + 31) / 32;
    for (int j = part + splits * warp; j < count; j += splits * warps) {
        float v[8], top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 32 + lane;
            v[i] = 0.0f;
            if (i >= blocks || r >= rank) continue;
            const float* src = inbox + (j / splits) * r16 + r;
            for (int s = 0; s < splits; ++s) v[i] += src[s * per_cta * r16];
            top = fmaxf(top, fabsf(v[i]));
        }
        const float up = pow2_below<BF>(warp_max(top)), down = 1.0f / up;
        if (lane == 0 && store_ok(p.ctl, first + j, 1, p.M)) pl.f[first + j] = scale * up;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= blocks) break;
            uint16_t w[3];
            split_terms<BF>(v[i] * down, w);
#pragma unroll
            for (int q = 0; q < terms<BF>(); ++q) {
                const size_t o = q * term_size + static_cast<size_t>(first + j) * pl.rp + i * 32 + lane;
                if (store_ok(p.ctl, o, 1, terms<BF>() * term_size)) pl.terms[o] = w[q];
            }
        }
    }
}

// Up to 32 ranks.  A cluster of CTAs computes one tile: v[64 tokens][R] over
// its share of K each, through a ring: A by TMA, 16 ranks x 64 columns a box, x
// by the loader warps' asynchronous copies (its rows are gathered; these copies
// reach some 17 bytes a cycle and SM, so A does not go the same way).  A row is
// 8 chunks of 16 bytes; in x's odd rows the halves are swapped, in A's rows the
// chunks are permuted by the 128-byte swizzle, and a lane takes the rank whose
// row puts the 8 lanes of a 16-byte read (two rows, four chunks) into different
// banks.  A consumer warp owns one rank tile of 16 and WN groups of 8 tokens,
// and waits for nothing but its stage.  Every CTA stores its partials of token j
// into the shared memory of CTA j % splits of the cluster, which adds them up,
// CTA by CTA in order, and writes the token's 16-bit terms: one cluster
// barrier, and nobody has to stay for the others.
// An accumulator set per half of a block of 32 columns (WN 1: and per block):
// a dependent mma.sync waits some 150 cycles, and a stage brings four in a row.
template <bool BF, int WN>
__global__ void __launch_bounds__((kShrinkWarps + kShrinkLoaders) * 32)
    lora_shrink_small(pq2h::LoraParams p, Plan pl, const __grid_constant__ CUtensorMap map_a,
                      int splits, int k_split, int stages) {
    constexpr int kSets = 4 / WN;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);   // swizzled rows
    __shared__ __align__(8) uint64_t full[kShrinkMaxStages], empty[kShrinkMaxStages];
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    pdl_wait();
    pdl_launch_dependents();
    const int index = blockIdx.x / splits;
    const int4 tile = pl.tiles[index];    // there for every index; a tile if below num_tiles
    const int l = tile.x, first = tile.y, count = tile.z, rank = tile.w;
    if (index >= *pl.num_tiles || rank == 0) return;   // the whole cluster
    // warps that have ranks and tokens
    constexpr int kTokenWarps = kTile / 8 / WN;
    const int busy = ((rank + 15) / 16) * ((count + 8 * WN - 1) / (8 * WN));
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], kShrinkLoaders * 32 + 1);
            mbar_init(&empty[s], busy);
        }
        abort_word = 0;
        fence_mbar_init();
    }
    if (splits > 1) cluster_arrive_relaxed();
    __syncthreads();
    const int part = splits > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int k0 = part * k_split, k1 = min(k0 + k_split, p.K);
    const int steps = (max(k1 - k0, 0) + kStageK - 1) / kStageK;
    const int r16 = (p.R + 15) / 16 * 16;   // rows of A per stage
    const int stage_bytes = (kTile + r16) * 128;
    const uint32_t base = smem_u32(smem);
    const int r0 = warp / kTokenWarps * 16, n0 = warp % kTokenWarps * WN;
    // the rank (of 8) that this lane's row of a fragment stands for: lanes g
    // and g + 1 of a read take rows 4 apart, whose chunks lie 4 apart
    const int gr = (g >> 1) | ((g & 1) << 2);
    const bool works = warp < kShrinkWarps && r0 < rank && n0 * 8 < count;
    float sum[WN][4];
#pragma unroll
    for (int i = 0; i < WN; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) sum[i][c] = 0.0f;

    if (warp >= kShrinkWarps) {
        const int pt = tid - kShrinkWarps * 32, chunk = pt & 7, row0 = pt >> 3;
        shrink_load(p, pl, &map_a, smem, full, empty, stages, stage_bytes, steps, k0, k1, l, rank, first,
                    count, pt, chunk, row0, base + row0 * 128 + ((chunk ^ ((row0 & 1) * 4)) * 16), abort_flag);
    } else if (works) {
        const uint32_t xat[2] = {static_cast<uint32_t>((t ^ ((g & 1) * 4)) * 16),
                                 static_cast<uint32_t>(((4 + t) ^ ((g & 1) * 4)) * 16)};
        const uint32_t aat[2] = {static_cast<uint32_t>((t ^ gr) * 16),
                                 static_cast<uint32_t>(((4 + t) ^ gr) * 16)};
        float acc[kSets][WN][4];
#pragma unroll
        for (int q = 0; q < kSets; ++q)
#pragma unroll
            for (int i = 0; i < WN; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[q][i][c] = 0.0f;
        int s = 0;
        uint32_t turn = 0;
        for (int step = 0; step < steps; ++step) {
            if (!mbar_ready_warp(&full[s], turn & 1, p.ctl, abort_flag)) {
                *abort_flag = 1;   // the host reads the error; v is not used
                break;
            }
            const uint32_t st = base + s * stage_bytes;
            const uint32_t x0 = st + (n0 * 8 + g) * 128, a0 = st + (kTile + r0 + gr) * 128;
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
                const uint4 a = lds_v4(a0 + aat[blk]), b = lds_v4(a0 + 8 * 128 + aat[blk]);
                uint4 c[WN];   // columns past the tile's last token hold anything and are not stored
#pragma unroll
                for (int i = 0; i < WN; ++i) c[i] = lds_v4(x0 + i * 8 * 128 + xat[blk]);
#pragma unroll
                for (int i = 0; i < WN; ++i)
                    mma16816<BF>(acc[(2 * blk) % kSets][i], a.x, b.x, a.y, b.y, c[i].x, c[i].y);
#pragma unroll
                for (int i = 0; i < WN; ++i)
                    mma16816<BF>(acc[(2 * blk + 1) % kSets][i], a.z, b.z, a.w, b.w, c[i].z, c[i].w);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (++s == stages) s = 0, ++turn;
            if ((step + 1) % kFlushStages == 0 || step + 1 == steps) {
#pragma unroll
                for (int q = 0; q < kSets; ++q)
#pragma unroll
                    for (int i = 0; i < WN; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            sum[i][c] += acc[q][i][c];
                            acc[q][i][c] = 0.0f;
                        }
            }
        }
    }
    // partials [from CTA][token / splits][r16], in the owner's shared memory
    float* inbox = reinterpret_cast<float*>(smem + stages * stage_bytes);
    const int per_cta = (kTile + splits - 1) / splits;
    __syncwarp();
    if (splits > 1) cluster_wait();   // all of the cluster have started
    if (works) {
        const uint32_t mine = smem_u32(inbox) + part * per_cta * r16 * 4;
#pragma unroll
        for (int i = 0; i < WN; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = (n0 + i) * 8 + 2 * t + h;
                if (j >= count) continue;
                uint32_t to = mine + (j / splits) * r16 * 4;
                if (splits > 1) to = map_to_rank(to, j % splits);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = r0 + c * 8 + gr;
                    if (r >= rank) continue;
                    if (splits > 1)
                        st_cluster_f32(to + r * 4, sum[i][c * 2 + h]);
                    else
                        sts_f32(to + r * 4, sum[i][c * 2 + h]);
                }
            }
    }
    __syncwarp();
    if (splits > 1)
        cluster_sync();
    else
        __syncthreads();
    shrink_finish<BF>(p, pl, inbox, part, splits, per_cta, r16, l, rank, first, count,
                      kShrinkWarps + kShrinkLoaders);
}

// More ranks, on the fifth-generation tensor cores: the same ring, x's rows too
// with the 128-byte swizzle, so that both lie as the product's operands.  One
// warp issues the products, A's ranks as the 128 rows of an accumulator (rows
// past the rank hold anything and reach only their own sums), the tokens as its
// 64 columns.  256 columns of K are summed in tensor memory and then added to
// the epilogue warps' registers in fp32, a lane per rank, while the next 256 go
// to the other accumulator.  With mma.sync a stage took 950 cycles (rank 64: 32
// instructions a scheduler), against 480 for its copies.  The longer way from
// the copies to the sums costs up to 2 us: 333 tokens of 17408 columns, rank
// 64, 26.5 us against 28.8 with mma.sync; 400 of rank 128 30.4 and 48.3; 4096
// of 5120 columns, rank 64, 113.9 and 115.6; but 1000 tokens of rank 32 27.3
// and 26.1, 4000 of rank 8 58.9 and 56.6.  MB: accumulators of 128 ranks.
template <int MB>
constexpr int shrink_threads() {
    return (8 * MB + kShrinkLoaders + 1) * 32;
}

template <bool BF, int MB>
__global__ void __launch_bounds__(shrink_threads<MB>(), MB == 1 ? 2 : 1)
    lora_shrink_tiles(pq2h::LoraParams p, Plan pl, const __grid_constant__ CUtensorMap map_a,
                      int splits, int k_split, int stages) {
    constexpr int kEpilogue = 8 * MB, kIssuer = kEpilogue + kShrinkLoaders;
    constexpr int kHalf = kTile / 2;             // tokens of an epilogue warp
    constexpr uint32_t kCols = 2 * MB * kTile;   // tensor memory
    extern __shared__ __align__(128) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);   // swizzled rows
    __shared__ __align__(8) uint64_t full[kShrinkMaxStages], empty[kShrinkMaxStages], dfull[2], dempty[2];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], kShrinkLoaders * 32 + 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dempty[i], kEpilogue);
        }
        abort_word = 0;
        fence_mbar_init();
    }
    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tmem_base)),
                     "r"(kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    const auto release = [&] {
        if (warp == kIssuer)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
    };
    pdl_wait();
    pdl_launch_dependents();
    const int index = blockIdx.x / splits;
    const int4 tile = pl.tiles[index];    // there for every index; a tile if below num_tiles
    const int l = tile.x, first = tile.y, count = tile.z;
    const int rank = tile.w;
    if (index >= *pl.num_tiles || rank == 0) {   // the whole cluster
        release();
        return;
    }
    if (splits > 1) cluster_arrive_relaxed();
    const int part = splits > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int k0 = part * k_split, k1 = min(k0 + k_split, p.K);
    const int steps = (max(k1 - k0, 0) + kStageK - 1) / kStageK;
    const int r16 = (p.R + 15) / 16 * 16;   // rows of A per stage
    const int stage_bytes = (kTile + r16) * 128;
    const uint32_t base = smem_u32(smem);
    // an epilogue warp's ranks and tokens
    const int r0 = (warp / 8 * 4 + warp % 4) * 32, j0 = warp / 4 % 2 * kHalf;
    const bool works = warp < kEpilogue && r0 < rank && j0 < count;
    float sum[kHalf];

    if (warp >= kEpilogue && warp < kIssuer) {
        const int pt = tid - kEpilogue * 32, chunk = pt & 7, row0 = pt >> 3;
        shrink_load(p, pl, &map_a, smem, full, empty, stages, stage_bytes, steps, k0, k1, l, rank, first,
                    count, pt, chunk, row0, base + row0 * 128 + ((chunk ^ (row0 & 7)) * 16), abort_flag);
    } else if (warp == kIssuer) {
        int s = 0, last_s = -1;
        uint32_t turn = 0, last_phase = 0;
        for (int step = 0; step < steps; ++step) {
            const int g = step / kFlushStages, d = g & 1;
            const bool opens = step % kFlushStages == 0;
            if (!mbar_ready_warp(&full[s], turn & 1, p.ctl, abort_flag) ||
                (opens && g >= 2 &&
                 !mbar_ready_warp(&dempty[d], static_cast<uint32_t>(g / 2 - 1) & 1, p.ctl, abort_flag))) {
                *abort_flag = 1;   // the host reads the error; v is not used
                break;
            }
            // x was written through the generic proxy
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_after();
            const uint32_t x0 = base + s * stage_bytes, a0 = x0 + kTile * 128;
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < kStageK / 16; ++i)
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        tc_mma<BF, kTile>(tmem + (d * MB + m) * kTile, sw128_desc(a0 + m * 128 * 128 + i * 32),
                                          sw128_desc(x0 + i * 32), !opens || i > 0);
                tc_commit(&empty[s]);
                if ((step + 1) % kFlushStages == 0 || step + 1 == steps) tc_commit(&dfull[d]);
            }
            __syncwarp();
            last_s = s;
            last_phase = turn & 1;
            if (++s == stages) s = 0, ++turn;
        }
        // no product may still be running when tensor memory is released
        if (last_s >= 0) mbar_ready_warp(&empty[last_s], last_phase, p.ctl);
    } else {
#pragma unroll
        for (int j = 0; j < kHalf; ++j) sum[j] = 0.0f;
        const uint32_t from = tmem + warp / 8 * kTile + j0 + (static_cast<uint32_t>(warp % 4 * 32) << 16);
        const int groups = (steps + kFlushStages - 1) / kFlushStages;
        for (int g = 0; g < groups; ++g) {
            const int d = g & 1;
            if (!mbar_ready_warp(&dfull[d], static_cast<uint32_t>(g / 2) & 1, p.ctl, abort_flag)) {
                *abort_flag = 1;
                break;
            }
            if (works) {
                tc_fence_after();
                const auto add = [&](auto at) {   // 16 tokens from there on
                    constexpr int A = decltype(at)::value;
                    float v[16];
                    tc_ld(from + d * MB * kTile + A, v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) sum[A + j] += v[j];
                };
                add(std::integral_constant<int, 0>{});
                if (count - j0 > 16) add(std::integral_constant<int, 16>{});
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&dempty[d]);
        }
    }
    // partials [from CTA][token / splits][r16], in the owner's shared memory
    float* inbox = reinterpret_cast<float*>(smem + stages * stage_bytes);
    const int per_cta = (kTile + splits - 1) / splits;
    __syncwarp();
    if (splits > 1) cluster_wait();   // all of the cluster have started
    if (works) {
        const int r = r0 + lane, shift = 31 - __clz(splits);
        const uint32_t mine = smem_u32(inbox) + (part * per_cta * r16 + r) * 4;
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
            const int j = j0 + i;
            if (j >= count || r >= rank) continue;
            const uint32_t to = mine + (j >> shift) * r16 * 4;
            if (splits > 1)
                st_cluster_f32(map_to_rank(to, j & (splits - 1)), sum[i]);
            else
                sts_f32(to, sum[i]);
        }
    }
    __syncwarp();
    tc_fence_before();
    if (splits > 1)
        cluster_sync();
    else
        __syncthreads();
    tc_fence_after();
    release();
    shrink_finish<BF>(p, pl, inbox, part, splits, per_cta, r16, l, rank, first, count,
                      shrink_threads<MB>() / 32);
}

// CTA (rounds x 128 outputs, tile): v's terms in shared memory, then per 32
// outputs and warp: y loads first, the product meanwhile, one store.
template <bool BF, int YT>
__global__ void __launch_bounds__(kExpandWarps * 32, 3)
    lora_expand_tiles(pq2h::LoraParams p, Plan pl, int rounds, int vec) {
    constexpr int NT = kTile / 8;
    extern __shared__ __align__(16) uint16_t sv[];
    __shared__ int tok[kTile];
    __shared__ float f[kTile];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the plan is complete before shrink lets this kernel start
    const bool here = static_cast<int>(blockIdx.y) < __ldcg(pl.num_tiles);
    const int4 tile = here ? __ldcg(pl.tiles + blockIdx.y) : make_int4(-1, 0, 0, 0);
    const int l = tile.x, first = tile.y, count = tile.z;
    const int rank = tile.w;
    const int blocks = (rank + 31) / 32;
    const bool in_place = p.y_in == p.y_out && p.ld_in == p.ld_out;
    if (!here || (rank == 0 && in_place)) {  // uniform over the CTA
        pdl_wait();
        return;
    }
    if (threadIdx.x < count) tok[threadIdx.x] = __ldcg(pl.perm + first + threadIdx.x);
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const int pitch = term_pitch(blocks), term_size = kTile * pitch;
    if (threadIdx.x < kTile)
        f[threadIdx.x] = rank > 0 && static_cast<int>(threadIdx.x) < count ? pl.f[first + threadIdx.x] : 0.0f;
    const int per_row = blocks * 4;  // 16-byte pieces
    for (int i = threadIdx.x; i < terms<BF>() * kTile * per_row; i += kExpandWarps * 32) {
        const int c = i % per_row, j = (i / per_row) % kTile, q = i / (per_row * kTile);
        *reinterpret_cast<uint4*>(sv + q * term_size + j * pitch + c * 8) =
            j < count ? load16(pl.terms + (static_cast<size_t>(q) * p.M + first + j) * pl.rp + c * 8)
                      : zero4();
    }
    __syncthreads();
    for (int round = 0; round < rounds; ++round) {
        const int n = (blockIdx.x * rounds + round) * (kExpandWarps * 32) + warp * 32 + 4 * (lane >> 2);
        float4 y[NT][2];
        y_fetch<YT, NT>(p, y, tok, count, n, vec != 0);
        float acc[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[h][i][c] = 0.0f;
        for (int blk = 0; blk < blocks; ++blk) {
            const BRows b = b_load(p, l, rank, n, blk);
            expand_block<BF, NT>(acc, b, sv, pitch, term_size, blk, count);
        }
        expand_store<YT, NT>(p, acc, y, tok, f, count, n, vec != 0);
    }
}

// The same over a ring in shared memory.  One CTA per SM takes a contiguous
// range of the items (tile, kNB outputs), so that v's terms rarely change;
// producer warps keep the next items' y and B on their way while groups of
// consumer warps take the items in turn.  y comes by asynchronous copies of
// kPiece bytes a thread (a warp per token row; bulk copies of 512-byte rows
// topped out at one per 46 ns and SM, half the rate needed), B by one bulk
// copy: kNB rows of B are contiguous.  A group has a warp per 32 outputs and
// goes over the tile's tokens by 32: eight accumulators a warp and three
// items at once, because a dependent mma.sync returns after some 150 cycles
// here (one item at a time took 3600 cycles for 64 tokens x 128 outputs of
// rank 64, against 2800 for its bytes).  Token rows of y are 16 bytes longer
// in shared memory, so that the 4 tokens of an access lie in different banks.
constexpr int kRingWarps = 12;      // consumers: 128 registers a thread
constexpr int kRingLoaders = 4;     // producer warps
constexpr int kRingMaxStages = 8;

// One item's product for a warp: 32 outputs x NI groups of 8 tokens.  bp: this
// lane's first row of B (shared-memory address, rows b_step apart), vp: its
// terms (groups i_step, terms q_step apart).  A column past the tile's last
// token holds anything and is not stored.
template <bool BF, int NI>
__device__ __forceinline__ void ring_product(float (&acc)[2][NI][4], uint32_t bp, uint32_t b_step,
                                             uint32_t vp, uint32_t i_step, uint32_t q_step,
                                             int blocks, int rank) {
    const int t = threadIdx.x & 3;
    for (int blk = 0; blk < blocks; ++blk, bp += 64, vp += 64) {
        uint4 b[4];
        if (blk * 32 + 32 <= rank) {
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = lds_v4(bp + i * b_step);
        } else {
            const int left = rank - blk * 32 - 8 * t;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[i] = left > 0 ? lds_v4(bp + i * b_step) : zero4();
            if (rank % 8 != 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = keep_first(b[i], left);
            }
        }
#pragma unroll
        for (int q = 0; q < terms<BF>(); ++q) {
            uint4 c[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) c[i] = lds_v4(vp + q * q_step + i * i_step);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                mma16816<BF>(acc[0][i], b[0].x, b[1].x, b[0].y, b[1].y, c[i].x, c[i].y);
                mma16816<BF>(acc[1][i], b[2].x, b[3].x, b[2].y, b[3].y, c[i].x, c[i].y);
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                mma16816<BF>(acc[0][i], b[0].z, b[1].z, b[0].w, b[1].w, c[i].z, c[i].w);
                mma16816<BF>(acc[1][i], b[2].z, b[3].z, b[2].w, b[3].w, c[i].z, c[i].w);
            }
        }
    }
}

// y' = y + f acc of NI groups of tokens, y from shared memory (sy: this lane's
// first), y' to global memory.  f, row: scale and start of y' of the lane's
// first token; n: its first output; left: tokens from the first group on.
template <int YT, int NI, int kYPitch, bool kWhole>
__device__ __forceinline__ void ring_store(const pq2h::LoraParams& p, const float (&acc)[2][NI][4],
                                           uint32_t sy, const float* f, const long long* row, int n,
                                           int left, bool vec) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!kWhole && i * 8 + 2 * t + h >= left) continue;
            const uint32_t a = sy + (i * 8 + h) * kYPitch;
            float4 o;
            if constexpr (YT == PQ2_F32) {
                const uint4 u = lds_v4(a);
                o = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                                __uint_as_float(u.w));
            } else {
                uint2 u;
                asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(u.x), "=r"(u.y) : "r"(a));
                o = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                                __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
            }
            const float s = f[i * 8 + h];
            o.x = fmaf(s, acc[0][i][h], o.x);
            o.y = fmaf(s, acc[0][i][2 + h], o.y);
            o.z = fmaf(s, acc[1][i][h], o.z);
            o.w = fmaf(s, acc[1][i][2 + h], o.w);
            y_store<YT>(p, row[i * 8 + h] + n, kWhole ? 4 : p.N - n, kWhole || vec, o);
        }
}

template <bool BF, int YT, int kNB, int kPiece>
__global__ void __launch_bounds__((kRingWarps + kRingLoaders) * 32, 1)
    lora_expand_ring(pq2h::LoraParams p, Plan pl, int groups, int stages, int stage_bytes,
                     int term_bytes) {
    constexpr int kUnit = YT == PQ2_F32 ? 4 : 2;
    constexpr int kYPitch = kNB * kUnit + 16;
    constexpr int kGroupWarps = kNB / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kRingMaxStages], empty[kRingMaxStages];
    __shared__ long long row[kTile];   // start of each token's y'
    __shared__ float f[kTile];
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    uint16_t* sv = reinterpret_cast<uint16_t*>(smem);
    uint8_t* ring = smem + term_bytes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], kRingLoaders * 32 + 1);
            mbar_init(&empty[s], kGroupWarps);
        }
        abort_word = 0;
        fence_mbar_init();
    }
    __syncthreads();
    const int nblocks = (p.N + kNB - 1) / kNB;
    const bool in_place = p.y_in == p.y_out && p.ld_in == p.ld_out;
    // the plan is complete before shrink lets this kernel start, as are y and
    // B; v's terms are not
    const long long total = static_cast<long long>(__ldcg(pl.num_tiles)) * nblocks;
    const long long it0 = total * blockIdx.x / gridDim.x, it1 = total * (blockIdx.x + 1) / gridDim.x;
    int index = static_cast<int>(it0 / nblocks), nb = static_cast<int>(it0 - static_cast<long long>(index) * nblocks);
    int left = static_cast<int>(it1 - it0);

    if (warp >= kRingWarps) {
        constexpr int kPieces = kNB * kUnit / kPiece;            // of a token row
        constexpr int kRows = kRingLoaders * 32 / kPieces;       // rows per round of the loaders
        static_assert(kRows >= 1, "a row is at most one round");
        const int pt = tid - kRingWarps * 32;
        const int row0 = pt / kPieces, piece = pt % kPieces;     // row0 is a warp's, or two
        const uint8_t* yb = static_cast<const uint8_t*>(p.y_in) + piece * kPiece;
        const long long ld = p.ld_in * kUnit;
        // each thread's rows by their addresses where they are few, else the
        // tile's tokens (lane, lane + 32) shared by shuffles
        constexpr int kRounds = kTile / kRows;
        constexpr bool kByAddress = kRounds <= 16;
        const uint8_t* rows[kByAddress ? kRounds : 1];
        int tk[2] = {0, 0};
        int cached = -1, l = -1, rank = 0, count = 0;
        int issued = 0, s = 0;
        uint32_t turn = 0;
        for (; left > 0; --left) {
            if (index != cached) {
                const int4 tile = __ldcg(pl.tiles + index);
                cached = index, l = tile.x, count = tile.z;
                rank = tile.w;
                if constexpr (kByAddress) {
#pragma unroll
                    for (int i = 0; i < kRounds; ++i) {
                        const int j = row0 + kRows * i;
                        rows[i] = j < count ? yb + __ldcg(pl.perm + tile.y + j) * ld : nullptr;
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (lane + 32 * h < count) tk[h] = __ldcg(pl.perm + tile.y + lane + 32 * h);
                }
            }
            const int n0 = nb * kNB, n = min(kNB, p.N - n0);
            if (++nb == nblocks) nb = 0, ++index;
            if (rank == 0 && in_place) continue;   // nothing to read or write
            if (turn > 0 && !mbar_ready_warp(&empty[s], (turn - 1) & 1, p.ctl, abort_flag)) break;
            if (issued != p.ctl.debug_skip_stage) {  // else withheld (timeout test)
                uint8_t* st = ring + static_cast<size_t>(s) * stage_bytes;
                if (pt == 0) {
                    const uint32_t brow = rank > 0 ? n * p.R * 2 : 0;
                    mbar_arrive_expect_tx(&full[s], brow);
                    if (rank > 0)
                        bulk_g2s(st + kTile * kYPitch,
                                 p.B + (static_cast<size_t>(l) * p.N + n0) * p.R, brow, &full[s]);
                }
                __syncwarp();
                const uint32_t dst = smem_u32(st) + row0 * kYPitch + piece * kPiece;
                if (kByAddress) {
                    if (piece * kPiece < n * kUnit) {
#pragma unroll
                        for (int i = 0; i < (kByAddress ? kRounds : 0); ++i)
                            if (rows[i])
                                cp_async<kPiece>(dst + i * kRows * kYPitch,
                                                 rows[i] + static_cast<size_t>(n0) * kUnit);
                    }
                } else {
                    const uint8_t* src = yb + static_cast<size_t>(n0) * kUnit;
                    const bool in = piece * kPiece < n * kUnit;
#pragma unroll 8
                    for (int i = 0; i * kRows < count; ++i) {
                        const int j = row0 + i * kRows;
                        const int lo = __shfl_sync(0xffffffffu, tk[0], j & 31);
                        const int hi = __shfl_sync(0xffffffffu, tk[1], j & 31);
                        if (in && j < count)
                            cp_async<kPiece>(dst + i * kRows * kYPitch, src + (j & 32 ? hi : lo) * ld);
                    }
                }
                cp_async_arrive(&full[s]);
            }
            ++issued;
            if (++s == stages) s = 0, ++turn;
        }
        // the last copies land before the CTA ends, whatever the consumers do
        for (int k = max(0, issued - stages); k < issued; ++k)
            if (k != p.ctl.debug_skip_stage)
                mbar_ready_warp(&full[k % stages], static_cast<uint32_t>(k / stages) & 1, p.ctl);
        cp_async_wait<0>();
        pdl_wait();
        return;
    }

    const int g = lane >> 2, t = lane & 3;
    const int group = warp / kGroupWarps;
    const int wn = (warp % kGroupWarps) * 32 + 4 * g;   // this lane's outputs within the item
    int cached = -1, rank = 0, count = 0, blocks = 0;
    const int pitch = term_pitch(pl.rp / 32), term_size = kTile * pitch;
    const uint32_t b_step = p.R * 2, i_step = 8 * pitch * 2, q_step = term_size * 2;
    const uint32_t ring_base = smem_u32(ring);
    const uint32_t b_off = kTile * kYPitch + (wn * p.R + 8 * t) * 2;
    const uint32_t y_off = 2 * t * kYPitch + wn * kUnit;
    const uint32_t v_base = smem_u32(sv + g * pitch + 8 * t);
    int s = 0, turn_of = 0;      // stage, and the group whose turn it is
    uint32_t turn = 0;
    bool ok = true;
    // the tile's record a tile ahead
    int4 next = __ldcg(pl.tiles + min(index, pl.max_tiles - 1));
    pdl_wait();
    pdl_launch_dependents();
    for (; left > 0; --left) {
        if (index != cached) {
            // every warp is done with the old tile; a failed wait reaches all
            if (named_bar_any(1, kRingWarps * 32, !ok)) return;
            const int4 tile = next;
            cached = index, count = tile.z;
            next = __ldcg(pl.tiles + min(index + 1, pl.max_tiles - 1));
            const int pieces = pl.rp / 8;   // of 16 bytes, at most 32
            float fv = 0.0f;
            int tv = 0;
            if (tid < count) {
                tv = __ldcg(pl.perm + tile.y + tid);
                fv = __ldcg(pl.f + tile.y + tid);
            }
            rank = tile.w;
            for (int i = warp; i < terms<BF>() * count && tile.x >= 0; i += kRingWarps) {
                const int q = i % terms<BF>(), j = i / terms<BF>();
                if (lane < pieces)
                    *reinterpret_cast<uint4*>(sv + q * term_size + j * pitch + lane * 8) =
                        load16_cg(pl.terms + (static_cast<size_t>(q) * p.M + tile.y + j) * pl.rp + lane * 8);
            }
            blocks = (rank + 31) / 32;
            if (tid < kTile) {
                row[tid] = tv * p.ld_out;
                f[tid] = rank > 0 ? fv : 0.0f;
            }
            named_bar_sync(2, kRingWarps * 32);
        }
        const int n = nb * kNB + wn;
        if (++nb == nblocks) nb = 0, ++index;
        if (rank == 0 && in_place) continue;
        const int stage = s;
        const uint32_t parity = turn & 1;
        const bool mine = turn_of == group;
        if (++s == stages) s = 0, ++turn;
        if (++turn_of == groups) turn_of = 0;
        if (!mine) continue;
        if (ok) ok = mbar_ready_warp(&full[stage], parity, p.ctl, abort_flag);
        if (!ok) {
            *abort_flag = 1;
            continue;   // to the next tile's barrier
        }
        const uint32_t st = ring_base + stage * stage_bytes;
        // tokens by 32, or by one group of 8
        auto part = [&](auto groups, int j) {
            constexpr int NI = decltype(groups)::value;
            float acc[2][NI][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[h][i][c] = 0.0f;
            ring_product<BF, NI>(acc, st + b_off, b_step, v_base + (j / 8) * i_step, i_step, q_step,
                                 blocks, rank);
            const uint32_t sy = st + y_off + j * kYPitch;
            const float* fj = f + j + 2 * t;
            const long long* rj = row + j + 2 * t;
            if (kPiece == 16 && count - j >= NI * 8 && n - wn + kNB <= p.N)
                ring_store<YT, NI, kYPitch, true>(p, acc, sy, fj, rj, n, count - j, true);
            else if (n < p.N)
                ring_store<YT, NI, kYPitch, false>(p, acc, sy, fj, rj, n, count - j, kPiece == 16);
        };
        for (int j = 0; j < count; j += 32) {
            if (count - j > 8)
                part(std::integral_constant<int, 4>{}, j);
            else
                part(std::integral_constant<int, 1>{}, j);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
    }
}

// ----------------------------------------------------------------------------
// expand on the 5th-generation tensor cores
// ----------------------------------------------------------------------------

// The ring's expand for fp32 y: the same items, with the product on tcgen05
// (kind::f16).  128 outputs are the rows of A (B's rows, K-major, 128-byte
// swizzle, by TMA), the tile's tokens the rows of B (v's terms, a pass of the
// product each), and the sum arrives in tensor memory, a column per token,
// several items in flight.  The epilogue's warps only add, store and hand
// back: 200 instructions a warp and item where the mma.sync form takes 800 and
// waits for its own results.  A lane is an output: y is read and written 128
// bytes a warp, one value a lane, so its rows need no alignment for that.
//
// A CTA takes a contiguous share of the items; where there are many, the
// shares stop at three quarters and the rest is taken from a counter, two
// items at a time (with shares alone the median CTA of 4096 tokens was done at
// 116 us and the last at 134: 130.4 us for the call against 117.1).  The items
// of one tile that a CTA takes in a row, eight at most, are a unit.  The
// scheduler warp fixes the units ahead and publishes them to the others; one
// warp loads a unit's terms while the unit before is under way (a tile change
// took 3 us otherwise); one looks at each item between its copies and its
// product: where the rank is no multiple of 16, it puts zeros over the ranks
// past it that the product would read (they may hold anything, and v's zero
// times a NaN is a NaN).
// Everyone who waits on a barrier sees each of its phases: a parity tells the
// phase meant only from the one before.
// Bound by HBM: 4096 tokens, rank 64, 17408 outputs 93 us alone, 5.8 TB/s.
constexpr int kTcEpilogue = 8;      // warps, two per quarter of the lanes
constexpr int kTcIssuer = 8, kTcProducer = 9, kTcFixer = 10, kTcTerms = 11, kTcScheduler = 12;
constexpr int kTcIssuer2 = 13;      // where there are two groups
constexpr int kTcLoaders = 4;       // the last, where y does not come by TMA
template <int T>
constexpr int tc_loader0() {
    return T == kTile ? kTcIssuer2 : kTcIssuer2 + 1;
}
template <bool kTma, int T>
constexpr int tc_threads() {
    return (tc_loader0<T>() + (kTma ? 0 : kTcLoaders)) * 32;
}
constexpr int kTcUnit = 8;          // items of a unit, at most
constexpr int kTcTail = 2;          // items taken at a time from the counter
constexpr int kTcShares = 16;       // items a CTA from which there is a counter
constexpr int kTcUnits = 2;         // units known at a time
constexpr int kTcMaxStages = 8;
constexpr int kTcABlock = kTcNB * 128;    // bytes of 64 ranks of an item's rows of B
// For tiles of at most T tokens:
template <int T>
struct Tc {
    // the epilogue's warps as groups that take the items in turn (an item of
    // few tokens is mostly waits); else they share each item's tokens
    static constexpr int kGroups = T == kTile ? 1 : 2;
    static constexpr int kItemWarps = kTcEpilogue / kGroups;
    static constexpr int kWarpTokens = T * 4 / kItemWarps;
    static constexpr int kDBufs = T == kTile ? 4 : 8;   // products in tensor memory
    static constexpr uint32_t kTmemCols = kDBufs * T;
    static constexpr int kVBlock = T * 128;             // bytes of 64 ranks of the terms
    static constexpr int kYBytes = T * kTcNB * 4;
};
constexpr int kTcMaxDBufs = 8;

// Tensor maps: y_in fp32 [M][N], box 128 x 1 (gathered by four rows); B 16-bit
// [L * N][R], box 64 x 128, 128-byte swizzle, zeros past R; v's terms 16-bit
// [terms * M][rp], box 64 x 64, the same.
struct TcMaps {
    CUtensorMap y, b, terms;
};

// Rows r0 .. r3 of columns x .. x + 127 (x a multiple of 4) to four rows of
// 512 bytes in shared memory; a row past the tensor's last gives zeros.
__device__ __forceinline__ void tma_gather4(void* dst, const void* map, int x, int r0, int r1, int r2,
                                            int r3, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3),
        "r"(smem_u32(bar))
        : "memory");
}

// kTma: y's rows start on 16-byte boundaries and come by TMA, four tokens an
// instruction; else value by value, by warps of their own.
struct TcUnit {
    int adapter, first, count, rank;   // count 0: no more units
    int nb0, nb1;
    int slot;
};
struct TcShared {
    uint64_t full[kTcMaxStages];    // an item's y and B are there
    uint64_t ready[kTcMaxStages];   // B as the product may read it
    uint64_t empty[kTcMaxStages];   // everyone is done with the stage
    uint64_t dfull[kTcMaxDBufs];     // an item's product is there
    uint64_t dempty[kTcMaxDBufs];     // read by the epilogue's warps
    uint64_t vfull[2];              // a unit's terms, rows and scales are there
    uint64_t vempty[2];             // everyone is done with them
    uint64_t ufull[kTcUnits];       // a unit is published
    uint64_t uempty[kTcUnits];      // everyone has taken it
    // read as 16-byte vectors
    alignas(16) int row[2][kTile];  // start of each token's y'
    alignas(16) float f[2][kTile];
    alignas(16) int token[kTcUnits][kTile];   // a unit's tokens (M past its count)
    TcUnit unit[kTcUnits];
    uint32_t tmem_base;
    int abort_word;
};

// Two stages of rank 128 and bf16 terms take 230400 bytes beside it, of 232448
// a CTA may have: a larger struct would send them to the other ring.
static_assert(sizeof(TcShared) <= 2048, "two stages fit up to rank 128");

// The k-th unit, for every warp but the scheduler's; false: no more, or a wait
// ran out.  A warp is done with its place (u.slot) when it calls release_unit.
__device__ __forceinline__ bool take_unit(TcShared& sh, int k, TcUnit& u, const DevCtl& ctl) {
    volatile int* abort_flag = &sh.abort_word;
    const int slot = k % kTcUnits;
    if (!mbar_ready_warp(&sh.ufull[slot], static_cast<uint32_t>(k / kTcUnits) & 1, ctl, abort_flag)) {
        *abort_flag = 1;
        return false;
    }
    u = sh.unit[slot];
    return u.count > 0;
}
__device__ __forceinline__ void release_unit(TcShared& sh, const TcUnit& u) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.uempty[u.slot]);
}

template <bool BF, bool kTma, int T>
__global__ void __launch_bounds__(tc_threads<kTma, T>(), 1)
    lora_expand_tc(pq2h::LoraParams p, Plan pl, const __grid_constant__ TcMaps maps, int stages,
                   int stage_bytes, int term_bytes) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ __align__(16) TcShared sh;
    volatile int* abort_flag = &sh.abort_word;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // terms of two units, then the stages; swizzled rows from 1024 on
    uint8_t* sv = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* ring = sv + 2 * term_bytes;
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&sh.full[s], kTma ? 1 : kTcLoaders * 32 + 1);
            mbar_init(&sh.ready[s], 1);
            mbar_init(&sh.empty[s], Tc<T>::kItemWarps + 1);
        }
        for (int i = 0; i < Tc<T>::kDBufs; ++i) {
            mbar_init(&sh.dfull[i], 1);
            mbar_init(&sh.dempty[i], Tc<T>::kItemWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.vfull[i], 2);
            mbar_init(&sh.vempty[i], kTcEpilogue);
        }
        for (int i = 0; i < kTcUnits; ++i) {
            mbar_init(&sh.ufull[i], 1);
            mbar_init(&sh.uempty[i], kTcEpilogue + 3 + Tc<T>::kGroups + (kTma ? 0 : kTcLoaders));
        }
        sh.abort_word = 0;
        fence_mbar_init();
    }
    if (warp == kTcIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sh.tmem_base)),
                     "r"(Tc<T>::kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    const int vblocks = (p.R + 63) / 64;
    TcUnit u;

    if (warp == kTcScheduler) {
        // ------------------------------ scheduler ------------------------------
        // the plan is complete before shrink lets this kernel start
        const bool in_place = p.y_in == p.y_out && p.ld_in == p.ld_out;
        const int nblocks = (p.N + kTcNB - 1) / kTcNB;
        const long long total = static_cast<long long>(__ldcg(pl.num_tiles + (in_place ? 1 : 0))) * nblocks;
        const long long grid = gridDim.x, shared = total >= kTcShares * grid ? total / 4 * 3 : total;
        long long pos = shared * blockIdx.x / grid, end = shared * (blockIdx.x + 1) / grid;
        for (int k = 0;;) {
            if (pos >= end && shared < total) {
                int got = 0;
                if (lane == 0) got = static_cast<int>(atomicAdd(pl.taken, 1u));
                pos = shared + static_cast<long long>(__shfl_sync(0xffffffffu, got, 0)) * kTcTail;
                end = min(pos + kTcTail, total);
            }
            const int slot = k % kTcUnits;
            TcUnit r = {-1, 0, 0, 0, 0, 0, slot};
            int tok[2] = {p.M, p.M};
            if (pos < end) {
                const int4 tile = __ldcg(pl.tiles + pos / nblocks);
                const int nb0 = static_cast<int>(pos % nblocks);
                const int n = static_cast<int>(min(static_cast<long long>(min(kTcUnit, nblocks - nb0)), end - pos));
                const int rank = tile.w;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (lane + 32 * h < tile.z) tok[h] = __ldcg(pl.perm + tile.y + lane + 32 * h);
                pos += n;
                if (rank == 0 && in_place) continue;
                r = {tile.x, tile.y, tile.z, rank, nb0, nb0 + n, slot};
            }
            if (k >= kTcUnits &&
                !mbar_ready_warp(&sh.uempty[slot], static_cast<uint32_t>(k / kTcUnits - 1) & 1, p.ctl,
                                 abort_flag)) {
                *abort_flag = 1;
                break;
            }
            sh.token[slot][lane] = tok[0];
            sh.token[slot][lane + 32] = tok[1];
            if (lane == 0) sh.unit[slot] = r;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.ufull[slot]);
            if (r.count == 0) break;
            ++k;
        }
        pdl_wait();
    } else if (warp == kTcProducer) {
        // ------------------------------ producer ------------------------------
        // y and B are older than the kernel before; v's terms are not
        int issued = 0, s = 0;
        uint32_t turn = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (!take_unit(sh, k, u, p.ctl)) break;
            const int used = (u.rank + 63) / 64, fours = (u.count + 3) / 4;
            const int4 tk = *reinterpret_cast<const int4*>(&sh.token[u.slot][(lane & 15) * 4]);
            release_unit(sh, u);
            for (int nb = u.nb0; nb < u.nb1; ++nb) {
                if (turn > 0 && !mbar_ready_warp(&sh.empty[s], (turn - 1) & 1, p.ctl, abort_flag)) {
                    ok = false;
                    break;
                }
                if (issued != p.ctl.debug_skip_stage) {  // else withheld (timeout test)
                    uint8_t* stage = ring + static_cast<size_t>(s) * stage_bytes;
                    if (lane == 0)
                        mbar_arrive_expect_tx(&sh.full[s],
                                              (kTma ? fours * 4 * kTcNB * 4 : 0) + used * kTcABlock);
                    __syncwarp();
                    if (lane < used)
                        tma_load_2d(stage + lane * kTcABlock, &maps.b, lane * 64,
                                    u.adapter * p.N + nb * kTcNB, &sh.full[s]);
                    if (kTma && lane < fours)
                        tma_gather4(stage + vblocks * kTcABlock + lane * 4 * kTcNB * 4, &maps.y, nb * kTcNB,
                                    tk.x, tk.y, tk.z, tk.w, &sh.full[s]);
                }
                ++issued;
                if (++s == stages) s = 0, ++turn;
            }
        }
        // the last copies land before the CTA ends, whatever the others do
        for (int k = max(0, issued - stages); k < issued; ++k)
            if (k != p.ctl.debug_skip_stage)
                mbar_ready_warp(&sh.full[k % stages], static_cast<uint32_t>(k / stages) & 1, p.ctl);
        pdl_wait();
    } else if (warp == kTcFixer) {
        // ------------------------------ fixer ------------------------------
        int s = 0;
        uint32_t turn = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (!take_unit(sh, k, u, p.ctl)) break;
            release_unit(sh, u);
            for (int nb = u.nb0; nb < u.nb1; ++nb) {
                ok = mbar_ready_warp(&sh.full[s], turn & 1, p.ctl, abort_flag);
                if (!ok) {
                    *abort_flag = 1;
                    break;
                }
                if (u.rank % 16 != 0) {
                    const uint32_t st = smem_u32(ring) + s * stage_bytes;
                    for (int r = lane; r < kTcNB; r += 32)
                        for (int c = u.rank / 8; c < (u.rank + 15) / 16 * 2; ++c) {
                            const uint32_t at = st + c / 8 * kTcABlock + r * 128 + (((c % 8) ^ (r & 7)) * 16);
                            const uint4 v = c * 8 < u.rank ? keep_first(lds_v4(at), u.rank - c * 8) : zero4();
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x),
                                         "r"(v.y), "r"(v.z), "r"(v.w)
                                         : "memory");
                        }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.ready[s]);
                    mbar_arrive(&sh.empty[s]);
                }
                if (++s == stages) s = 0, ++turn;
            }
        }
        pdl_wait();
    } else if (warp == kTcTerms) {
        // ------------------------------ terms ------------------------------
        pdl_wait();
        int k = 0;
        for (;; ++k) {
            if (!take_unit(sh, k, u, p.ctl)) break;
            const int b = k & 1;
            const int tok[2] = {sh.token[u.slot][lane], sh.token[u.slot][lane + 32]};
            release_unit(sh, u);
            if (k >= 2 && !mbar_ready_warp(&sh.vempty[b], static_cast<uint32_t>(k / 2 - 1) & 1, p.ctl, abort_flag)) {
                *abort_flag = 1;
                break;
            }
            const int used = (u.rank + 63) / 64, boxes = terms<BF>() * used;
            if (lane == 0) mbar_arrive_expect_tx(&sh.vfull[b], boxes * Tc<T>::kVBlock);
            __syncwarp();
            // rows past the tile's are its neighbours' and give columns that
            // are not stored
            if (lane < boxes) {
                const int q = lane / used, c = lane % used;
                tma_load_2d(sv + b * term_bytes + (q * vblocks + c) * Tc<T>::kVBlock, &maps.terms, c * 64,
                            q * p.M + u.first, &sh.vfull[b]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (lane + 32 * h < u.count) {
                    sh.row[b][lane + 32 * h] = static_cast<int>(tok[h] * p.ld_out);
                    sh.f[b][lane + 32 * h] = u.rank > 0 ? __ldcg(pl.f + u.first + lane + 32 * h) : 0.0f;
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.vfull[b]);
        }
        // the last copies land before the CTA ends, whatever the others do
        for (int i = max(0, k - 2); i < k; ++i)
            mbar_ready_warp(&sh.vfull[i & 1], static_cast<uint32_t>(i / 2) & 1, p.ctl);
    } else if (!kTma && warp >= tc_loader0<T>()) {
        // ------------------------------ loaders of y ------------------------------
        const int pt = tid - tc_loader0<T>() * 32;
        const uint8_t* yb = reinterpret_cast<const uint8_t*>(p.y_in) + pt * 4;
        const long long ld = p.ld_in * 4;
        int issued = 0, s = 0;
        uint32_t turn = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (!take_unit(sh, k, u, p.ctl)) break;
            const int tk[2] = {sh.token[u.slot][lane], sh.token[u.slot][lane + 32]};
            release_unit(sh, u);
            for (int nb = u.nb0; nb < u.nb1; ++nb) {
                const int n0 = nb * kTcNB, n = min(kTcNB, p.N - n0);
                if (turn > 0 && !mbar_ready_warp(&sh.empty[s], (turn - 1) & 1, p.ctl, abort_flag)) {
                    ok = false;
                    break;
                }
                if (issued != p.ctl.debug_skip_stage) {
                    const uint32_t ys = smem_u32(ring) + s * stage_bytes + vblocks * kTcABlock + pt * 4;
                    const uint8_t* src = yb + static_cast<size_t>(n0) * 4;
#pragma unroll 8
                    for (int j = 0; j < u.count; ++j) {
                        const int lo = __shfl_sync(0xffffffffu, tk[0], j & 31);
                        const int hi = __shfl_sync(0xffffffffu, tk[1], j & 31);
                        if (pt < n) cp_async<4>(ys + j * kTcNB * 4, src + (j & 32 ? hi : lo) * ld);
                    }
                    cp_async_arrive(&sh.full[s]);
                }
                ++issued;
                if (++s == stages) s = 0, ++turn;
            }
        }
        cp_async_wait<0>();
        pdl_wait();
    } else if (warp == kTcIssuer || (Tc<T>::kGroups > 1 && warp == kTcIssuer2)) {
        // ------------------------------ issuer ------------------------------
        // one for each group of the epilogue.  The warp stays together up to
        // the products themselves: under a branch of one lane their operands
        // took several hundred cycles an item to reach the uniform registers
        const int group = warp == kTcIssuer ? 0 : 1;
        int s = 0, d = 0, next = 0;
        uint32_t turn = 0, dturn = 0;
        int last_d = -1;              // of the last product issued, and its phase
        uint32_t last_phase = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (!take_unit(sh, k, u, p.ctl)) break;
            release_unit(sh, u);
            const int steps = (u.rank + 15) / 16;
            const uint32_t v0 = smem_u32(sv) + (k & 1) * term_bytes;
            ok = mbar_ready_warp(&sh.vfull[k & 1], static_cast<uint32_t>(k / 2) & 1, p.ctl, abort_flag);
            for (int nb = u.nb0; nb < u.nb1 && ok; ++nb) {
                if (next == group) {
                    ok = mbar_ready_warp(&sh.ready[s], turn & 1, p.ctl, abort_flag) &&
                         (dturn == 0 || mbar_ready_warp(&sh.dempty[d], (dturn - 1) & 1, p.ctl, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(ring) + s * stage_bytes;
                    if (elect_one()) {
#pragma unroll
                        for (int q = 0; q < terms<BF>(); ++q)
                            for (int i = 0; i < steps; ++i) {
                                const uint32_t off = (i & 3) * 32;
                                tc_mma<BF, T>(tmem + d * T, sw128_desc(a0 + (i >> 2) * kTcABlock + off),
                                              sw128_desc(v0 + (q * vblocks + (i >> 2)) * Tc<T>::kVBlock + off),
                                              q + i > 0);
                            }
                        tc_commit(&sh.dfull[d]);   // at once where the rank is 0
                    }
                    __syncwarp();
                    last_d = d;
                    last_phase = dturn & 1;
                }
                if (++next == Tc<T>::kGroups) next = 0;
                if (++d == Tc<T>::kDBufs) d = 0, ++dturn;
                if (++s == stages) s = 0, ++turn;
            }
        }
        if (!ok) *abort_flag = 1;
        // no product may still be running when tensor memory is released
        if (last_d >= 0) mbar_ready_warp(&sh.dfull[last_d], last_phase, p.ctl);
        pdl_wait();
    } else {
        // ------------------------------ epilogue ------------------------------
        const int quarter = warp & 3, part_of = warp >> 2;   // 32 outputs; a group or a part of the tokens
        const int group = Tc<T>::kGroups > 1 ? part_of : 0;
        const int j0 = Tc<T>::kGroups > 1 ? 0 : part_of * Tc<T>::kWarpTokens;
        int next = 0;    // the group whose item it is
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        float* yout = static_cast<float*>(p.y_out);
        const long long out_elems = static_cast<long long>(p.M - 1) * p.ld_out + p.N;
        int s = 0, d = 0;
        uint32_t turn = 0, dturn = 0;
        pdl_wait();
        pdl_launch_dependents();
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (!take_unit(sh, k, u, p.ctl)) break;
            release_unit(sh, u);
            const int vb = k & 1;
            ok = mbar_ready_warp(&sh.vfull[vb], static_cast<uint32_t>(k / 2) & 1, p.ctl, abort_flag);
            for (int nb = u.nb0; nb < u.nb1 && ok; ++nb) {
                const int n = nb * kTcNB + quarter * 32 + lane;
                const bool mine = next == group;
                if (++next == Tc<T>::kGroups) next = 0;
                if (mine) {
                    ok = mbar_ready_warp(&sh.full[s], turn & 1, p.ctl, abort_flag) &&
                         mbar_ready_warp(&sh.dfull[d], dturn & 1, p.ctl, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const float* sy = reinterpret_cast<const float*>(ring + static_cast<size_t>(s) * stage_bytes +
                                                                     vblocks * kTcABlock) +
                                      j0 * kTcNB + quarter * 32 + lane;
                    // the first 8 tokens of this half, or all of them
                    const auto part = [&](auto tokens) {
                        constexpr int W = decltype(tokens)::value;
                        float acc[W], y[W];
                        if (u.rank > 0) {
                            tc_ld(tmem + d * T + j0 + lane_off, acc);
                        } else {
#pragma unroll
                            for (int j = 0; j < W; ++j) acc[j] = 0.0f;
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.dempty[d]);
#pragma unroll
                        for (int j = 0; j < W; ++j) y[j] = sy[j * kTcNB];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.empty[s]);   // the stage is in registers
#pragma unroll
                        for (int j = 0; j < W; j += 4) {
                            const int4 rj = *reinterpret_cast<const int4*>(&sh.row[vb][j0 + j]);
                            const float4 fj = *reinterpret_cast<const float4*>(&sh.f[vb][j0 + j]);
                            const int o[4] = {rj.x + n, rj.y + n, rj.z + n, rj.w + n};
                            const float g[4] = {fj.x, fj.y, fj.z, fj.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (n < p.N && j0 + j + i < u.count && store_ok(p.ctl, o[i], 1, out_elems))
                                    yout[o[i]] = fmaf(g[i], acc[j + i], y[j + i]);
                        }
                    };
                    if (u.count - j0 > 8) {
                        part(std::integral_constant<int, Tc<T>::kWarpTokens>{});
                    } else if (u.count - j0 > 0) {
                        part(std::integral_constant<int, 8>{});
                    } else {
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&sh.dempty[d]);
                            mbar_arrive(&sh.empty[s]);
                        }
                    }
                    __syncwarp();
                }
                if (++d == Tc<T>::kDBufs) d = 0, ++dturn;
                if (++s == stages) s = 0, ++turn;
            }
            __syncwarp();
            if (!ok) *abort_flag = 1;
            else if (lane == 0) mbar_arrive(&sh.vempty[vb]);
        }
    }
    // every role is done with tensor memory
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kTcIssuer)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(Tc<T>::kTmemCols));
}

}  // namespace
}  // namespace pq2

namespace pq2h {

namespace {

using pq2::kFewTokens;
using pq2::kMaxSplits;
using pq2::kSmallTile;
using pq2::kTile;

// The GPU's SMs: the K splits are sized for it on the host, before a device
// is known (pq2_lora_workspace_bytes).
constexpr int64_t kSms = 152;

size_t pad(size_t b) { return (b + 255) & ~size_t(255); }

struct Layout {
    bool few;
    int splits, k_split, tile, max_tiles, rp;
    size_t part, terms, f, perm, tiles, num_tiles, bytes;
};

// The few-token form up to kFewTokens tokens; the planned one already above 64
// where tokens and their adapters' B are many, since its copies run further
// ahead and read B once for 16 tokens (17408 outputs, us few and planned: 128
// tokens over 64 adapters of rank 64 56.5 and 51.7, over 30 of rank 128 54.5 and
// 38.4; 66 over 64 of rank 128 71.3 and 64.9; but 80 over 64 of rank 64 47.3 and
// 53.0; 128 over 64 of rank 128 with 5120 outputs 50.2 and 59.9).
bool few_tokens(int64_t M, int64_t N, int64_t L, int64_t R) {
    return M <= 64 || (M <= kFewTokens && M * std::min(M, L) * N * R * 2 <= 15000000000);
}

Layout layout(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R) {
    Layout y = {};
    y.few = few_tokens(M, N, L, R);
    int64_t s;
    if (y.few) {
        // K splits: two CTAs per SM over the tiles that may appear, at
        // least 16 KB of A each
        const int64_t tiles = pq2::few_tiles(M, std::min(M, L));
        s = (2 * kSms + tiles - 1) / tiles;
        s = std::min(s, std::max<int64_t>(1, K * R * 2 / 16384));
        s = std::min<int64_t>(s, kMaxSplits);
    } else {
        // a cluster per tile: one and a half CTAs per SM over the tiles that
        // are likely, at least 256 columns each; more than 8 CTAs (the portable
        // cluster size) from 512 columns each
        // small tiles up to 32 tokens an adapter: expand's stages are smaller, so
        // there are more, and more items.  129 tokens over 64 adapters of rank 64,
        // 17408 outputs: 49.0 us against 60.7 with 64; 1000 over 64 of rank 16 38.9
        // and 44.1; 250 over 10 of rank 64 26.7 and 29.4; but 600 over 10 of rank
        // 32 30.9 and 23.7, 1000 over 30 of rank 24 84.6 and 42.0.  The rule goes by
        // the stack's adapters, which may be more than have tokens, and not by N or
        // the rank: a rank that is no multiple of 16, whose items all pass the
        // fixing warp, is better off with 64 well below 32 tokens an adapter
        y.tile = M <= 32 * L ? kSmallTile : kTile;
        const int64_t tiles = (M + y.tile - 1) / y.tile + std::min(L, M / 2);
        s = 1;
        while (s < 16 && s * tiles * 2 < 3 * kSms && K / (2 * s) >= (s < 8 ? 256 : 512)) s *= 2;
    }
    y.k_split = static_cast<int>(((K + s - 1) / s + 127) / 128 * 128);
    y.splits = y.few ? static_cast<int>((K + y.k_split - 1) / y.k_split) : static_cast<int>(s);
    y.rp = static_cast<int>((R + 31) / 32 * 32);
    size_t o = 0;
    if (y.few) {
        y.part = o;
        o += pad(static_cast<size_t>(y.splits) * M * R * 4);
    } else {
        y.max_tiles = static_cast<int>((M + y.tile - 1) / y.tile + std::min(L + 1, M));
        y.terms = o;
        o += pad(static_cast<size_t>(3) * M * y.rp * 2);
        y.f = o;
        o += pad(static_cast<size_t>(M) * 4);
        y.perm = o;
        o += pad(static_cast<size_t>(M) * 4);
        y.tiles = o;   // with room for as many as any M up to this one has
        o += pad(static_cast<size_t>((M + kSmallTile - 1) / kSmallTile + std::min(L + 1, M)) * 16);
        y.num_tiles = o;
        o += 256;
    }
    y.bytes = o;
    return y;
}

template <bool BF, int YT>
cudaError_t run_few(const LoraParams& p, const Layout& lay, uint8_t* ws, int vec, cudaStream_t st) {
    float* part = reinterpret_cast<float*>(ws + lay.part);
    const int64_t with = pq2::few_tiles(p.M, std::min(p.M, p.L));
    cudaError_t e = launch(pq2::lora_shrink_few<BF>, dim3(lay.splits, static_cast<unsigned>(with)),
                           dim3(pq2::kShrinkWarps * 32), 0, st, true, p, part, lay.k_split);
    if (e != cudaSuccess) return e;
    static SmemLimit lim[2];
    const int rb = (p.R + 31) / 32;
    auto kern = rb == 1 ? pq2::lora_expand_few<BF, YT, true> : pq2::lora_expand_few<BF, YT, false>;
    const size_t smem = static_cast<size_t>(pq2::terms<BF>()) * pq2::kFewTile * pq2::term_pitch(rb) * 2 +
                        static_cast<size_t>(pq2::kFewTile) * rb * 32 * 4;
    e = raise_smem(lim[rb == 1], kern, smem);
    if (e != cudaSuccess) return e;
    // 128 outputs a CTA while the GPU has SMs to spare; else 256, and as many
    // rounds of them as keep the CTAs to about one residency (two per SM): a
    // CTA's start (its tile, v) costs several trips to L2.  Rounded up, since
    // `all` is the most tiles that may appear (64 tokens over 64 adapters of rank
    // 64, 17408 outputs: 45.3 us, rounded down 50.0, with 2.5 per SM 58.6)
    const int64_t all = pq2::few_tiles(p.M, std::min(p.M, p.L + 1));
    const bool spare = (p.N + 127) / 128 * all <= 2 * kSms;
    const int cols = (spare ? pq2::kExpandWarps : pq2::kExpandMaxWarps) * 32;
    const int64_t blocks = (p.N + cols - 1) / cols;
    const int64_t per_tile = (2 * kSms + all - 1) / all;
    const int rounds = spare ? 1 : static_cast<int>((blocks + per_tile - 1) / per_tile);
    return launch(kern,
                  dim3(static_cast<unsigned>((blocks + rounds - 1) / rounds), static_cast<unsigned>(all)),
                  dim3(cols), smem, st, true, p, part, lay.splits, rounds, vec);
}

template <typename Kern>
cudaError_t ensure_wide_cluster(SmemLimit& done, Kern kern) {
    int dev = -1;
    const bool known = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kSmemLimitDevices;
    if (known && done.bytes[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && known) done.bytes[dev].store(1, std::memory_order_release);
    return e;
}

// MB 0: lora_shrink_small, over p.R / 16 rank tiles.
template <bool BF, int MB, int WN>
cudaError_t run_shrink(const LoraParams& p, const pq2::Plan& pl, const Layout& lay, cudaStream_t st,
                       const DeviceInfo& dev) {
    const auto kern = [] {
        if constexpr (MB == 0)
            return pq2::lora_shrink_small<BF, WN>;
        else
            return pq2::lora_shrink_tiles<BF, MB>;
    }();
    static SmemLimit lim;
    const int r16 = (p.R + 15) / 16 * 16, stage = (kTile + r16) * 128;
    const int inbox = lay.splits * ((kTile + lay.splits - 1) / lay.splits) * r16 * 4;
    // two CTAs per SM (1 KB each is the system's), above 128 ranks one
    const int room = (MB < 2 ? (dev.max_smem_optin + 1024) / 2 - 1024 : dev.max_smem_optin) - 2048;
    const int stages = std::min(pq2::kShrinkMaxStages, (room - inbox) / stage);
    // a product reads MB * 128 rows of A, whatever follows the last stage's
    const size_t smem = 1024 + std::max<size_t>(static_cast<size_t>(stages) * stage + inbox,
                                                static_cast<size_t>(stages - 1) * stage +
                                                    (kTile + MB * 128) * 128);
    CUtensorMap map_a;
    if (!encode_tmap_2d(&map_a, BF ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        p.A, p.K, static_cast<uint64_t>(p.L) * p.R, static_cast<uint64_t>(p.K) * 2,
                        pq2::kStageK, 16, true))
        return cudaErrorUnknown;
    cudaError_t e = raise_smem(lim, kern, smem);
    if (e != cudaSuccess) return e;
    if (lay.splits > 8) {
        // clusters past the portable size are asked for once per kernel
        static SmemLimit wide;
        e = ensure_wide_cluster(wide, kern);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(lay.splits * lay.max_tiles));
    cfg.blockDim = dim3(MB == 0 ? (pq2::kShrinkWarps + pq2::kShrinkLoaders) * 32 : pq2::shrink_threads<MB>());
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(lay.splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = lay.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p, pl, map_a, lay.splits, lay.k_split, stages);
}

// The ring's shared memory: v's terms, then as many stages as fit (0: fewer
// than two).
template <bool BF, int YT, int kNB>
int ring_stages(const LoraParams& p, const DeviceInfo& dev, int* stage_bytes, int* term_bytes) {
    constexpr int kUnit = YT == PQ2_F32 ? 4 : 2;
    *term_bytes = pq2::terms<BF>() * kTile * pq2::term_pitch((p.R + 31) / 32) * 2;
    *stage_bytes = kTile * (kNB * kUnit + 16) + kNB * p.R * 2;
    const int stages = (dev.max_smem_optin - 2048 - *term_bytes) / *stage_bytes;
    return stages < 2 ? 0 : std::min(stages, pq2::kRingMaxStages);
}

template <bool BF, int YT, int kNB, int kPiece>
cudaError_t run_ring(const LoraParams& p, const pq2::Plan& pl, int stages, int stage_bytes,
                     int term_bytes, cudaStream_t st, const DeviceInfo& dev) {
    auto kern = pq2::lora_expand_ring<BF, YT, kNB, kPiece>;
    // whole turns of the groups (see the kernel).  128 outputs: two stages a
    // group where they are few (4096 tokens of rank 64: two groups on four
    // stages 149 us, three on three 158); 64 outputs, for ranks above 64 or so:
    // as many groups as stages (rank 128: 167 us against 189 with two)
    const int groups = kNB == 128 ? std::min(3, stages / 2) : std::min(6, stages);
    stages -= stages % groups;
    static SmemLimit lim;
    const size_t smem = static_cast<size_t>(term_bytes) + static_cast<size_t>(stages) * stage_bytes;
    const cudaError_t e = raise_smem(lim, kern, smem);
    if (e != cudaSuccess) return e;
    return launch(kern, dim3(dev.num_sms), dim3((pq2::kRingWarps + pq2::kRingLoaders) * 32), smem, st,
                  true, p, pl, groups, stages, stage_bytes, term_bytes);
}

// 128 outputs an item where three stages fit beside v's terms (they take two
// thirds of the barriers and shuffles of 64), else 64.
template <bool BF, int YT, int kPiece>
cudaError_t run_ring(const LoraParams& p, const pq2::Plan& pl, cudaStream_t st, const DeviceInfo& dev) {
    int sb, tb;
    int stages = ring_stages<BF, YT, 128>(p, dev, &sb, &tb);
    if (stages >= 3) return run_ring<BF, YT, 128, kPiece>(p, pl, stages, sb, tb, st, dev);
    stages = ring_stages<BF, YT, 64>(p, dev, &sb, &tb);
    return run_ring<BF, YT, 64, kPiece>(p, pl, stages, sb, tb, st, dev);
}

// fp32 y on the tensor-memory form, where two stages fit and y's offsets and
// B's rows count in 31 bits (us with it, and on the ring of mma.sync: 4096
// tokens, rank 64, 17408 outputs 114.0 and 147.0; 1000 47.8 and 57.6; 4000 of
// rank 8, 5120 outputs 56.7 and 62.2; 300 of rank 128 22.6 and 23.5; 129 of rank
// 16, 5120 outputs 16.1 and 15.8).
template <bool BF, bool kTma, int T>
cudaError_t run_tc(const LoraParams& p, const pq2::Plan& pl, cudaStream_t st, const DeviceInfo& dev,
                   bool* taken) {
    const int vblocks = (p.R + 63) / 64;
    const int term_bytes = pq2::terms<BF>() * vblocks * pq2::Tc<T>::kVBlock;
    const int stage_bytes = vblocks * pq2::kTcABlock + pq2::Tc<T>::kYBytes;
    int stages =
        std::min(pq2::kTcMaxStages, (dev.max_smem_optin - static_cast<int>(sizeof(pq2::TcShared)) - 1024 -
                                     2 * term_bytes) / stage_bytes);
    stages -= stages % pq2::Tc<T>::kGroups;   // a stage is always the same group's
    *taken = stages >= 2 && (static_cast<int64_t>(p.M) - 1) * p.ld_out + p.N < (int64_t(1) << 31) &&
             static_cast<int64_t>(p.L) * p.N + pq2::kTcNB < (int64_t(1) << 31);
    if (!*taken) return cudaSuccess;
    pq2::TcMaps maps = {};
    if ((kTma && !encode_tmap_2d(&maps.y, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.y_in, p.N, p.M,
                                 static_cast<uint64_t>(p.ld_in) * 4, pq2::kTcNB, 1, false)) ||
        !encode_tmap_2d(&maps.b, BF ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        p.B, p.R, static_cast<uint64_t>(p.L) * p.N, static_cast<uint64_t>(p.R) * 2, 64,
                        pq2::kTcNB, true) ||
        !encode_tmap_2d(&maps.terms, BF ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        pl.terms, pl.rp, static_cast<uint64_t>(pq2::terms<BF>()) * p.M,
                        static_cast<uint64_t>(pl.rp) * 2, 64, T, true))
        return cudaErrorUnknown;
    auto kern = pq2::lora_expand_tc<BF, kTma, T>;
    static SmemLimit lim;
    const size_t smem = 1024 + 2 * static_cast<size_t>(term_bytes) + static_cast<size_t>(stages) * stage_bytes;
    const cudaError_t e = raise_smem(lim, kern, smem);
    if (e != cudaSuccess) return e;
    return launch(kern, dim3(dev.num_sms), dim3(pq2::tc_threads<kTma, T>()), smem, st, true, p, pl, maps, stages,
                  stage_bytes, term_bytes);
}

SmemLimit g_plan_smem;  // one for the kernel: run() has several instantiations

template <bool BF, int YT>
cudaError_t run(const LoraParams& p, const Layout& lay, uint8_t* ws, int vec, cudaStream_t st,
                const DeviceInfo& dev) {
    if (lay.few) return run_few<BF, YT>(p, lay, ws, vec, st);
    pq2::Plan pl = {};
    pl.terms = reinterpret_cast<uint16_t*>(ws + lay.terms);
    pl.f = reinterpret_cast<float*>(ws + lay.f);
    pl.perm = reinterpret_cast<int*>(ws + lay.perm);
    pl.tiles = reinterpret_cast<int4*>(ws + lay.tiles);
    pl.num_tiles = reinterpret_cast<int*>(ws + lay.num_tiles);
    pl.taken = reinterpret_cast<unsigned*>(ws + lay.num_tiles + 128);
    pl.max_tiles = lay.max_tiles;
    pl.tile = lay.tile;
    pl.rp = lay.rp;
    // as many warps as have tokens and fit their histograms in 200 KB; one
    // warp's and the ranks fit up to some 14500 adapters, without the ranks the
    // most there can be do
    const int bins = p.L + 1;
    int warps = 32;
    while (warps > 1 && (warps / 2 * 32 >= p.M || static_cast<size_t>(warps + 3) * bins * 4 > 200 * 1024))
        warps /= 2;
    const auto plan_bytes = [&](int arrays) { return (static_cast<size_t>(arrays) * bins + 1) * 4; };
    static_assert((3 * (PQ2_LORA_MAX_L + 1) + 1) * 4 <= 200 * 1024, "one warp's plan fits");
    const int ranks_here = plan_bytes(warps + 3) + 512 <= static_cast<size_t>(dev.max_smem_optin);
    const size_t plan_smem = plan_bytes(warps + 2 + ranks_here);
    cudaError_t e = raise_smem(g_plan_smem, pq2::lora_plan_kernel, plan_smem);
    if (e != cudaSuccess) return e;
    e = launch(pq2::lora_plan_kernel, dim3(1), dim3(warps * 32), plan_smem, st, true, p, pl, warps,
               ranks_here);
    if (e != cudaSuccess) return e;
    e = p.R <= 16    ? run_shrink<BF, 0, 1>(p, pl, lay, st, dev)
        : p.R <= 32  ? run_shrink<BF, 0, 2>(p, pl, lay, st, dev)
        : p.R <= 128 ? run_shrink<BF, 1, 0>(p, pl, lay, st, dev)
                     : run_shrink<BF, 2, 0>(p, pl, lay, st, dev);
    if (e != cudaSuccess) return e;
    // the ring, by 16-byte pieces of y where its rows allow, else (fp32) by
    // values; bf16 rows off their 16 bytes go by plain loads
    constexpr int kPer16 = YT == PQ2_F32 ? 4 : 8;
    const bool by16 = p.N % kPer16 == 0 && p.ld_in % kPer16 == 0 &&
                      reinterpret_cast<uintptr_t>(p.y_in) % 16 == 0;
    if constexpr (YT == PQ2_F32) {
        bool taken = false;
        if (lay.tile == kTile)
            e = by16 ? run_tc<BF, true, kTile>(p, pl, st, dev, &taken)
                     : run_tc<BF, false, kTile>(p, pl, st, dev, &taken);
        else
            e = by16 ? run_tc<BF, true, kSmallTile>(p, pl, st, dev, &taken)
                     : run_tc<BF, false, kSmallTile>(p, pl, st, dev, &taken);
        if (taken || e != cudaSuccess) return e;
    }
    if (by16 && p.ld_out % 4 == 0 && vec) return run_ring<BF, YT, 16>(p, pl, st, dev);
    if constexpr (YT == PQ2_F32) {
        return run_ring<BF, YT, 4>(p, pl, st, dev);
    } else {
        static SmemLimit lim;
        const size_t smem = static_cast<size_t>(pq2::terms<BF>()) * kTile *
                            pq2::term_pitch((p.R + 31) / 32) * 2;
        e = raise_smem(lim, pq2::lora_expand_tiles<BF, YT>, smem);
        if (e != cudaSuccess) return e;
        const int rounds = p.M <= 512 ? 1 : 4;
        const int cols = pq2::kExpandWarps * 32 * rounds;
        return launch(pq2::lora_expand_tiles<BF, YT>, dim3((p.N + cols - 1) / cols, lay.max_tiles),
                      dim3(pq2::kExpandWarps * 32), smem, st, true, p, pl, rounds, vec);
    }
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R) {
    // enough for any smaller M: few tokens may take more than many (their
    // partial sums over K are in memory)
    size_t most = layout(M, N, K, L, R).bytes;
    for (int64_t m = 1; m < std::min<int64_t>(M, kFewTokens + 1); ++m)
        most = std::max(most, layout(m, N, K, L, R).bytes);
    return most;
}

size_t lora_workspace_needed(const LoraParams& p) { return layout(p.M, p.N, p.K, p.L, p.R).bytes; }

cudaError_t launch_lora(const LoraParams& p, void* workspace, cudaStream_t st,
                        const DeviceInfo& dev) {
    const Layout lay = layout(p.M, p.N, p.K, p.L, p.R);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    // 4-wide accesses to y: every row starts on their boundary
    const size_t unit = p.y_type == PQ2_F32 ? 16 : 8;
    const bool vec = p.ld_in % 4 == 0 && p.ld_out % 4 == 0 &&
                     reinterpret_cast<uintptr_t>(p.y_in) % unit == 0 &&
                     reinterpret_cast<uintptr_t>(p.y_out) % unit == 0;
    if (p.bf16)
        return p.y_type == PQ2_F32 ? run<true, PQ2_F32>(p, lay, ws, vec, st, dev)
                                   : run<true, PQ2_BF16>(p, lay, ws, vec, st, dev);
    return p.y_type == PQ2_F32 ? run<false, PQ2_F32>(p, lay, ws, vec, st, dev)
                               : run<false, PQ2_BF16>(p, lay, ws, vec, st, dev);
}

}  // namespace pq2h
