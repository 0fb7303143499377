// Rotary positions, and new tokens into a cache held in 4 bits.
//
// Every pair (a, b) of a head's first `rot` values is turned by its token's
// angle: a' = a cos - b sin, b' = b cos + a sin, each operation one fp32
// rounding (so a plain restatement gets the same bits, and with them the same
// 4-bit codes).  Cosines and sines come from a table made once
// (rope_table_kernel, in 64 bits: at position 262144 a 32-bit angle would be off by
// up to 0.016): a row of it serves all heads of a token.
//
// Each value is read once and written once (2 or 4 bytes, or half a byte), with a few
// operations between.  head_kernel gives a warp a head's row of D values, D/32
// neighbours a lane, and two heads at once so that their loads are in flight together;
// in long calls it goes on to the token's other heads, so that place and angles
// are found once.  A pair's other half is loaded by both lanes that need it (the second
// time from L1).  A row's least and largest value, which its scale and offset come
// from, are one reduction over the warp each.  With inputs' type and pairing known when it
// is compiled it is held to 64 registers (80 with the cache), so that 32 (24) warps of an SM
// keep memory busy.  Neighbours fit (of 256 dims into the cache but for 12 bytes); halves of
// 256 dims spill 112 to 156 bytes (into the cache 24 to 132, of 128 dims 20).  4096 tokens of 28
// heads of 256 (fp32 in, bf16 out), floor 26.9 us: neighbours 30.6 us, halves 47.8; bf16
// in, floor 18.2: 29.3 and 43.3.  Parts whose half is no multiple of a lane's values, loaded
// one at a time: 52 and 75 us (fp32, 122 of 256).  Into the cache the issue of instructions
// is the limit: 3369 tokens of 64 heads of 128 in 49 us (floor 24; bf16 in 60), and read
// back in 10 (floor 3.2), where a lane's loads are small.
#include <algorithm>
#include <cmath>

#include "pq2_cache.cuh"
#include "pq2_elem.cuh"

namespace pq2 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlots = 2;  // heads of one token that a warp has in flight

// E neighbouring elements from element i on; VEC: on a boundary of their size.
template <int E, bool VEC>
__device__ __forceinline__ void load_elems(const void* base, int type, long long i, float (&v)[E]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < E; ++j)
            v[j] = type == PQ2_F32 ? static_cast<const float*>(base)[i + j]
                                   : elem_to_f32(static_cast<const uint16_t*>(base)[i + j], type);
    } else if (type == PQ2_F32) {
        const float* p = static_cast<const float*>(base) + i;
        if constexpr (E == 2) {
            const float2 f = *reinterpret_cast<const float2*>(p);
            v[0] = f.x, v[1] = f.y;
        } else {
#pragma unroll
            for (int k = 0; k < E / 4; ++k) {
                const float4 f = reinterpret_cast<const float4*>(p)[k];
                v[4 * k] = f.x, v[4 * k + 1] = f.y, v[4 * k + 2] = f.z, v[4 * k + 3] = f.w;
            }
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(base) + i;
        uint32_t w[E / 2];
        if constexpr (E == 2) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (E == 4) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            w[0] = u.x, w[1] = u.y;
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        }
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
            v[2 * k] = elem_to_f32(w[k] & 0xffffu, type);
            v[2 * k + 1] = elem_to_f32(w[k] >> 16, type);
        }
    }
}

template <int E, bool VEC>
__device__ __forceinline__ void store_elems(void* base, int type, long long i, const float (&v)[E]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < E; ++j) {
            if (type == PQ2_F32)
                static_cast<float*>(base)[i + j] = v[j];
            else
                static_cast<uint16_t*>(base)[i + j] = f32_to_elem16(v[j], type);
        }
    } else if (type == PQ2_F32) {
        float* p = static_cast<float*>(base) + i;
        if constexpr (E == 2) {
            *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
        } else {
#pragma unroll
            for (int k = 0; k < E / 4; ++k)
                reinterpret_cast<float4*>(p)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(base) + i;
        uint32_t w[E / 2];
#pragma unroll
        for (int k = 0; k < E / 2; ++k) w[k] = f32x2_to_elem16(v[2 * k], v[2 * k + 1], type);
        if constexpr (E == 2)
            *reinterpret_cast<uint32_t*>(p) = w[0];
        else if constexpr (E == 4)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

__device__ __forceinline__ float turned(float x, float other, float c, float s, bool second) {
    return second ? __fadd_rn(__fmul_rn(x, c), __fmul_rn(other, s))
                  : __fsub_rn(__fmul_rn(x, c), __fmul_rn(other, s));
}

__device__ __forceinline__ float warp_min(float v) {
    float r;
    asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// A row of 32 E values to E codes a lane (value j in bits 4j..) and the row's
// (scale, offset) as two fp16.
template <int E>
__device__ __forceinline__ uint32_t quantise_row(const float (&x)[E], uint32_t& pair) {
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int j = 1; j < E; ++j) lo = fminf(lo, x[j]), hi = fmaxf(hi, x[j]);
    lo = warp_min(lo);
    hi = warp_max(hi);
    const float range = __fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f);
    const __half s = __float2half_rn(fminf(range, 65504.0f));
    const __half z = __float2half_rn(fminf(fmaxf(lo, -65504.0f), 65504.0f));
    pair = __half_as_ushort(s) | (static_cast<uint32_t>(__half_as_ushort(z)) << 16);
    const float sf = __half2float(s), zf = __half2float(z);
    const float inv = sf > 0.0f ? __fdiv_rn(1.0f, sf) : 0.0f;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
        // clamped first, then rounded by adding 1.5 * 2^23 (half to even; the
        // integer is in the low bits): the same as rounded and clamped
        const float t = fminf(fmaxf(__fmul_rn(__fsub_rn(x[j], zf), inv), 0.0f), 15.0f);
        w |= (__float_as_uint(__fadd_rn(t, 12582912.0f)) & 15u) << (4 * j);
    }
    return w;
}

// Where a token stands in the cache; page < 0: nowhere, pos < 0: its position is out of range too.
struct Place {
    long long pos;
    long long page;
};

__device__ __forceinline__ Place place_of(const pq2h::CacheParams& c, int row, const DevCtl& ctl, bool& mine) {
    int end;
    const int seq = seq_of_row(c.row_start, c.B, row, end);
    mine = seq >= 0;
    Place at = {-1, -1};
    if (!mine) return at;
    at.pos = static_cast<long long>(__ldcg(c.lens + seq)) - end + row;
    bool bad = at.pos < 0 || at.pos >= static_cast<long long>(c.W) * c.T;
    if (bad) {
        at.pos = -1;
    } else {
        const int p = __ldcg(c.pages + seq * c.ld_pages + at.pos / c.T);
        bad = p < 0 || p >= c.num_pages;
        if (!bad) at.page = p;
    }
    if (bad && (threadIdx.x & 31) == 0) atomicOr(ctl.err, DEVERR_BAD_INDEX);
    return at;
}

// A warp takes a part of one token's heads (all of them in long calls), kSlots at a
// time.  Slots of a token: heads[0] of array 0, heads[1] of array 1 (both
// turned), heads[2] of array 2 (values as they are); where CACHE, arrays 1 and 2 go
// to the cache.
// MODE: kAny, or of values on boundaries of a lane's size kF32 (inputs are fp32) + kNear
// (neighbours make pairs): with both known a warp needs half of the registers.
constexpr int kAny = -1, kF32 = 1, kNear = 2;

template <int E, int MODE, bool CACHE>
__global__ void __launch_bounds__(kThreads, MODE == kAny ? 2 : CACHE ? 3 : 4) head_kernel(const __grid_constant__ pq2h::RopeParams p) {
    constexpr bool VEC = MODE != kAny;
    constexpr int D = 32 * E, kN = kSlots;
    const int x_type = VEC && (MODE & kF32) ? PQ2_F32 : p.x_type;
    if (VEC && !(MODE & kF32)) __builtin_assume(x_type != PQ2_F32);
    const int lane = threadIdx.x & 31;
    const int slots = p.heads[0] + p.heads[1] + p.heads[2];
    const int per_part = ((slots + kN - 1) / kN + p.parts - 1) / p.parts * kN;
    const long long total = p.M * p.parts;
    const int d = lane * E, half = p.rot >> 1;
    const bool near = VEC ? (MODE & kNear) != 0 : (p.flags & PQ2_ROPE_NEIGHBOURS) != 0;
    pdl_wait();
    pdl_launch_dependents();
    for (long long w = blockIdx.x * static_cast<long long>(kWarps) + (threadIdx.x >> 5); w < total;
         w += static_cast<long long>(gridDim.x) * kWarps) {
        const long long row = p.parts == 1 ? w : w / p.parts;
        const int first = static_cast<int>(w - row * p.parts) * per_part, end = min(first + per_part, slots);
        if (first >= end) continue;
        Place place = {0, 0};
        if constexpr (CACHE) {
            bool mine;
            place = place_of(p.cache, static_cast<int>(row), p.ctl, mine);
            if (!mine || place.pos < 0) continue;
        }
        float c[E], s[E];
#pragma unroll
        for (int j = 0; j < E; ++j) c[j] = 1.0f, s[j] = 0.0f;
        if (p.rot > 0) {
            const long long at = p.positions ? __ldcg(p.positions + row) : place.pos;
            if (at < 0 || at >= p.table_rows) {
                if (lane == 0) atomicOr(p.ctl.err, DEVERR_BAD_INDEX);
                continue;
            }
            const float* t = p.table + at * p.rot;
            if (VEC && d < p.rot) {
                if (near) {
                    float cs[E];
                    load_elems<E, true>(t, PQ2_F32, d, cs);
#pragma unroll
                    for (int j = 0; j < E; ++j) c[j] = cs[j & ~1], s[j] = cs[j | 1];
                } else {
                    float cs[E];
                    const int i0 = 2 * (d < half ? d : d - half);
                    load_elems<E, true>(t, PQ2_F32, i0, cs);
#pragma unroll
                    for (int j = 0; j < E / 2; ++j) c[j] = cs[2 * j], s[j] = cs[2 * j + 1];
                    load_elems<E, true>(t, PQ2_F32, i0 + E, cs);
#pragma unroll
                    for (int j = 0; j < E / 2; ++j) c[E / 2 + j] = cs[2 * j], s[E / 2 + j] = cs[2 * j + 1];
                }
            } else if (!VEC) {
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const int e = d + j;
                    if (e >= p.rot) continue;
                    const int i = near ? e >> 1 : e < half ? e : e - half;
                    c[j] = t[2 * i], s[j] = t[2 * i + 1];
                }
            }
            if (p.flags & PQ2_ROPE_INVERSE) {
#pragma unroll
                for (int j = 0; j < E; ++j) s[j] = -s[j];
            }
        }
        // (an array at a time: what depends on it alone is found once)
        int off = 0;
#pragma unroll 1
        for (int k = 0; k < 3; off += p.heads[k], ++k) {
            const int h1 = min(end - off, p.heads[k]);
            int h = max(first - off, 0);
            if (h >= h1) continue;
            const bool cached = CACHE && k > 0, turn = k < 2 && p.rot > 0;
            if (cached && place.page < 0) continue;
            const long long hs = p.hs[k];
            long long in = row * p.ld[k] + h * hs + d, out = 0, out_hs = 0;
            int pair_at = 0;
            if (cached) {
                const int T = p.cache.T, t = static_cast<int>(place.pos % T);
                out_hs = static_cast<long long>(T / kTileTokens) * tile_bytes(D);
                out = place.page * p.cache.page_stride + h * out_hs + t / kTileTokens * tile_bytes(D);
                pair_at = tile_pairs(D, k - 1) + (t % kTileTokens) * 4;
                out += tile_codes(D, k - 1) + (t % kTileTokens) * (D / 2) + lane * (E / 2);
                pair_at -= tile_codes(D, k - 1) + (t % kTileTokens) * (D / 2);
            } else {
                out_hs = p.hso[k];
                out = row * p.ldo[k] + h * out_hs + d;
            }
            const long long other = d < half ? half : -half;
#pragma unroll 1
            for (; h < h1; h += kN, in += kN * hs, out += kN * out_hs) {
                float x[kN][E], o[kN][E];
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    if (h + i >= h1) continue;
                    const long long at = in + i * hs;
                    load_elems<E, VEC>(p.x[k], x_type, at, x[i]);
                    if (!turn || near) continue;
                    if constexpr (VEC) {
                        // (rot / 2 is a multiple of E: a lane is on one side)
                        if (d < p.rot) load_elems<E, true>(p.x[k], x_type, at + other, o[i]);
                    } else {
#pragma unroll
                        for (int j = 0; j < E; ++j) {
                            const int e = d + j;
                            float one[1] = {0.0f};
                            if (e < p.rot) load_elems<1, false>(p.x[k], x_type, at + j + (e < half ? half : -half), one);
                            o[i][j] = one[0];
                        }
                    }
                }
                // in place: everything that the warp reads of these heads is read before it writes
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    if (h + i >= h1) continue;
                    if (turn) {
                        float y[E];
#pragma unroll
                        for (int j = 0; j < E; ++j) {
                            const int e = d + j;
                            y[j] = x[i][j];
                            if (e < p.rot)
                                y[j] = near ? turned(x[i][j], x[i][j ^ 1], c[j], s[j], e & 1)
                                            : turned(x[i][j], o[i][j], c[j], s[j], e >= half);
                        }
#pragma unroll
                        for (int j = 0; j < E; ++j) x[i][j] = y[j];
                    }
                    const long long at = out + i * out_hs;
                    if (!cached) {
                        if (store_ok(p.ctl, at, E, p.out_elems[k])) store_elems<E, VEC>(p.out[k], p.out_type, at, x[i]);
                        continue;
                    }
                    uint32_t pair;
                    const uint32_t codes = quantise_row<E>(x[i], pair);
                    if (store_ok(p.ctl, at, E / 2, p.cache.pool_bytes)) {
                        if constexpr (E == 8)
                            *reinterpret_cast<uint32_t*>(p.cache.pool + at) = codes;
                        else if constexpr (E == 4)
                            *reinterpret_cast<uint16_t*>(p.cache.pool + at) = static_cast<uint16_t>(codes);
                        else
                            p.cache.pool[at] = static_cast<uint8_t>(codes);
                    }
                    if (lane == 0 && store_ok(p.ctl, at + pair_at, 4, p.cache.pool_bytes))
                        *reinterpret_cast<uint32_t*>(p.cache.pool + at + pair_at) = pair;
                }
            }
        }
    }
}

// Heads of any size: a warp per head's row, a pair (or a value behind the
// turned part) a lane.
__global__ void __launch_bounds__(kThreads) any_head_kernel(const __grid_constant__ pq2h::RopeParams p) {
    const int lane = threadIdx.x & 31, half = p.rot >> 1;
    const int slots = p.heads[0] + p.heads[1];
    const long long total = p.M * slots;
    const bool near = p.flags & PQ2_ROPE_NEIGHBOURS;
    pdl_wait();
    pdl_launch_dependents();
    for (long long w = blockIdx.x * static_cast<long long>(kWarps) + (threadIdx.x >> 5); w < total;
         w += static_cast<long long>(gridDim.x) * kWarps) {
        const long long row = w / slots;
        int h = static_cast<int>(w - row * slots), k = 0;
        if (h >= p.heads[0]) h -= p.heads[0], k = 1;
        const float* t = nullptr;
        if (p.rot > 0) {
            const int at = __ldcg(p.positions + row);
            if (at < 0 || at >= p.table_rows) {
                if (lane == 0) atomicOr(p.ctl.err, DEVERR_BAD_INDEX);
                continue;
            }
            t = p.table + static_cast<long long>(at) * p.rot;
        }
        const long long in = row * p.ld[k] + h * p.hs[k], out = row * p.ldo[k] + h * p.hso[k];
        // a pair's (or a value's) two places are read and written by one lane
        for (int i = lane; i < half + p.dim - p.rot; i += 32) {
            float a[1], b[1];
            if (i >= half) {
                load_elems<1, false>(p.x[k], p.x_type, in + i + half, a);
                if (store_ok(p.ctl, out + i + half, 1, p.out_elems[k]))
                    store_elems<1, false>(p.out[k], p.out_type, out + i + half, a);
                continue;
            }
            const int i0 = near ? 2 * i : i, i1 = near ? 2 * i + 1 : i + half;
            load_elems<1, false>(p.x[k], p.x_type, in + i0, a);
            load_elems<1, false>(p.x[k], p.x_type, in + i1, b);
            const float c = t[2 * i], s = (p.flags & PQ2_ROPE_INVERSE) ? -t[2 * i + 1] : t[2 * i + 1];
            const float a2[1] = {turned(a[0], b[0], c, s, false)}, b2[1] = {turned(b[0], a[0], c, s, true)};
            if (store_ok(p.ctl, out + i0, 1, p.out_elems[k])) store_elems<1, false>(p.out[k], p.out_type, out + i0, a2);
            if (store_ok(p.ctl, out + i1, 1, p.out_elems[k])) store_elems<1, false>(p.out[k], p.out_type, out + i1, b2);
        }
    }
}

// The cache's values of a call's token rows: a warp takes a part of a token's
// rows of D values (all of them in long calls), kReads at a time.
constexpr int kReads = 4;

template <int E, bool VEC>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ pq2h::RopeParams p) {
    constexpr int D = 32 * E;
    const int lane = threadIdx.x & 31;
    const int slots = p.heads[0] + p.heads[1];
    const int per_part = ((slots + kReads - 1) / kReads + p.parts - 1) / p.parts * kReads;
    const long long total = p.M * p.parts;
    pdl_wait();
    pdl_launch_dependents();
    for (long long w = blockIdx.x * static_cast<long long>(kWarps) + (threadIdx.x >> 5); w < total;
         w += static_cast<long long>(gridDim.x) * kWarps) {
        const long long row = p.parts == 1 ? w : w / p.parts;
        const int first = static_cast<int>(w - row * p.parts) * per_part, end = min(first + per_part, slots);
        if (first >= end) continue;
        bool mine;
        const Place place = place_of(p.cache, static_cast<int>(row), p.ctl, mine);
        if (!mine || place.page < 0) continue;
        const int T = p.cache.T, t = static_cast<int>(place.pos % T);
        const long long head_bytes = static_cast<long long>(T / kTileTokens) * tile_bytes(D);
        const uint8_t* tile = p.cache.pool + place.page * p.cache.page_stride + t / kTileTokens * tile_bytes(D);
        int off = 0;
#pragma unroll 1
        for (int k = 0; k < 2; off += p.heads[k], ++k) {
            const int h1 = min(end - off, p.heads[k]), value = p.read_kind[k];
            const int code_at = tile_codes(D, value) + (t % kTileTokens) * (D / 2) + lane * (E / 2);
            const int pair_at = tile_pairs(D, value) + (t % kTileTokens) * 4;
#pragma unroll 1
            for (int h = max(first - off, 0); h < h1; h += kReads) {
                uint32_t codes[kReads], pair[kReads];
#pragma unroll
                for (int i = 0; i < kReads; ++i) {
                    if (h + i >= h1) continue;
                    const uint8_t* at = tile + (h + i) * head_bytes;
                    if constexpr (E == 8)
                        codes[i] = *reinterpret_cast<const uint32_t*>(at + code_at);
                    else if constexpr (E == 4)
                        codes[i] = *reinterpret_cast<const uint16_t*>(at + code_at);
                    else
                        codes[i] = at[code_at];
                    pair[i] = *reinterpret_cast<const uint32_t*>(at + pair_at);
                }
#pragma unroll
                for (int i = 0; i < kReads; ++i) {
                    if (h + i >= h1) continue;
                    const float s = elem_to_f32(pair[i] & 0xffffu, PQ2_F16), z = elem_to_f32(pair[i] >> 16, PQ2_F16);
                    float v[E];
#pragma unroll
                    for (int j = 0; j < E; ++j)  // (code * scale is exact: 4 + 11 bits)
                        v[j] = __fadd_rn(__fmul_rn(static_cast<float>((codes[i] >> (4 * j)) & 15u), s), z);
                    const long long out = row * p.ldo[k] + (h + i) * p.hso[k] + lane * E;
                    if (store_ok(p.ctl, out, E, p.out_elems[k])) store_elems<E, VEC>(p.out[k], p.out_type, out, v);
                }
            }
        }
    }
}

// One thread per (position, pair).
__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ pq2h::RopeTableParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int half = p.rot / 2;
    const long long total = p.count * half;
    for (long long n = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; n < total;
         n += static_cast<long long>(gridDim.x) * kThreads) {
        const long long pos = n / half;
        const int i = static_cast<int>(n - pos * half);
        double f = exp(-2.0 * i / p.rot * p.log_base);
        const double slow = f / p.factor;
        if (p.kind == PQ2_ROPE_LINEAR) {
            f = slow;
        } else if (p.kind == PQ2_ROPE_RAMP) {
            const double t = fmin(fmax((i - p.low) / (p.high - p.low), 0.0), 1.0);
            f = f + (slow - f) * t;
        } else if (p.kind == PQ2_ROPE_BANDS) {
            const double turns = p.old_len * f / 6.283185307179586476925;
            if (turns < p.low)
                f = slow;
            else if (turns <= p.high) {
                const double t = (turns - p.low) / (p.high - p.low);
                f = (1.0 - t) * slow + t * f;
            }
        }
        double sn, cs;
        sincos(static_cast<double>(p.first + pos) * f, &sn, &cs);
        if (store_ok(p.ctl, 2 * n, 2, 2 * total))
            reinterpret_cast<float2*>(p.table)[n] = make_float2(static_cast<float>(cs * p.magnitude),
                                                                static_cast<float>(sn * p.magnitude));
    }
}

}  // namespace
}  // namespace pq2

namespace pq2h {

namespace {

unsigned grid_for(long long warps) {
    // (longer ones are walked by the loop)
    return static_cast<unsigned>(std::min<long long>((warps + pq2::kWarps - 1) / pq2::kWarps, 1 << 24));
}

bool fits(const void* p, long long ld, long long hs, int unit_elems, int elem) {
    const int bytes = std::min(16, unit_elems * elem);
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * elem % bytes == 0 && hs * elem % bytes == 0;
}

int size_of(int type) { return type == PQ2_F32 ? 4 : 2; }

bool vector_path(const RopeParams& p, int E, bool cache) {
    const int per = (p.flags & PQ2_ROPE_NEIGHBOURS) ? p.rot : p.rot / 2;
    if (per % E != 0 || p.rot % 2 != 0) return false;
    for (int k = 0; k < 3; ++k) {
        if (p.heads[k] == 0) continue;
        if (!fits(p.x[k], p.ld[k], p.hs[k], E, size_of(p.x_type))) return false;
        if ((!cache || k == 0) && !fits(p.out[k], p.ldo[k], p.hso[k], E, size_of(p.out_type))) return false;
    }
    return true;
}

constexpr long long kEnoughWarps = 152 * 48;  // (four times as many: 88 us for 3369 tokens appended
                                               // and read back, when this took 75)

// Warps for each of M tokens: a token's place and angles are found once for all
// its heads where there are tokens enough to keep all SMs busy.
int parts_for(long long M, int slots, int at_once) {
    const long long most = std::max((slots + at_once - 1) / at_once, 1);
    return static_cast<int>(std::min(most, std::max(kEnoughWarps / std::max(M, 1ll), 1ll)));
}

template <int E, bool CACHE>
cudaError_t launch_heads(const RopeParams& args, cudaStream_t st) {
    RopeParams p = args;
    const int slots = p.heads[0] + p.heads[1] + p.heads[2];
    p.parts = parts_for(p.M, slots, pq2::kSlots);
    const unsigned grid = grid_for(p.M * p.parts);
    const auto go = [&](auto kernel) { return launch(kernel, dim3(grid), dim3(pq2::kThreads), 0, st, true, p); };
    if (!vector_path(p, E, CACHE)) return go(pq2::head_kernel<E, pq2::kAny, CACHE>);
    const bool f32 = p.x_type == PQ2_F32, near = p.flags & PQ2_ROPE_NEIGHBOURS;
    if (near) return f32 ? go(pq2::head_kernel<E, pq2::kF32 + pq2::kNear, CACHE>) : go(pq2::head_kernel<E, pq2::kNear, CACHE>);
    return f32 ? go(pq2::head_kernel<E, pq2::kF32, CACHE>) : go(pq2::head_kernel<E, 0, CACHE>);
}

template <int E>
cudaError_t launch_read(const RopeParams& args, cudaStream_t st) {
    RopeParams p = args;
    p.parts = parts_for(p.M, p.heads[0] + p.heads[1], pq2::kReads);
    const unsigned grid = grid_for(p.M * p.parts);
    bool vec = true;
    for (int k = 0; k < 2; ++k)
        if (p.heads[k]) vec = vec && fits(p.out[k], p.ldo[k], p.hso[k], E, size_of(p.out_type));
    if (vec) return launch(pq2::read_kernel<E, true>, dim3(grid), dim3(pq2::kThreads), 0, st, true, p);
    return launch(pq2::read_kernel<E, false>, dim3(grid), dim3(pq2::kThreads), 0, st, true, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t st) {
    switch (p.dim) {
        case 64: return launch_heads<2, false>(p, st);
        case 128: return launch_heads<4, false>(p, st);
        case 256: return launch_heads<8, false>(p, st);
    }
    return launch(pq2::any_head_kernel, dim3(grid_for(p.M * (p.heads[0] + p.heads[1]))),
                  dim3(pq2::kThreads), 0, st, true, p);
}

cudaError_t launch_cache_append(const RopeParams& p, cudaStream_t st) {
    switch (p.dim) {
        case 64: return launch_heads<2, true>(p, st);
        case 128: return launch_heads<4, true>(p, st);
    }
    return launch_heads<8, true>(p, st);
}

cudaError_t launch_cache_read(const RopeParams& p, cudaStream_t st) {
    switch (p.dim) {
        case 64: return launch_read<2>(p, st);
        case 128: return launch_read<4>(p, st);
    }
    return launch_read<8>(p, st);
}

cudaError_t launch_rope_table(const RopeTableParams& p, cudaStream_t st) {
    const long long total = p.count * (p.rot / 2);
    const unsigned grid = static_cast<unsigned>(
        std::min<long long>((total + pq2::kThreads - 1) / pq2::kThreads, 1 << 20));
    return launch(pq2::rope_table_kernel, dim3(grid), dim3(pq2::kThreads), 0, st, true, p);
}

}  // namespace pq2h
