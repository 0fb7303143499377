// Norms around a block of a serving step.  The pages time the projections;
// what stands between two of them is one pass over the residual stream:
//
//   before a block   x  = rms(r) * w
//   after a block    n  = rms(y) * w_post            (or y * w_post)
//                    r' = r + alpha * act(gate) * n
//                    x  = rms(r') * w_next           (the next block's input)
//   rms(v) = v / sqrt(mean(v^2) + eps)
//
// Every value is read and written once: a row stays in registers (or, for
// rows wider than that, in shared memory) from its loads to its stores, through both
// reductions.  All arithmetic is fp32; r' and x are rounded once each, and x
// comes from the unrounded r'.
//
// The kernel is bound by HBM bytes for many rows and by the latency of two
// reductions for few.  One CTA per row, as many CTAs as fit the GPU, each
// walking over rows with both weight vectors kept in registers (they would
// otherwise come through L2 again for every row).  Rows of at most 512
// values go one to a warp, without barriers.  Measured: one row of 5120 3.1 us
// (the launch, the reductions), 64 rows 4.0; 4096 rows of 5120 through the ring
// below 36.0 us, 5.8 TB/s, 87% of the copy rate.
#include <algorithm>

#include "pq2_common.cuh"
#include "pq2_elem.cuh"
#include "pq2_internal.h"
#include "pq2_step.cuh"

namespace pq2 {
namespace {

constexpr int kMaxWarps = 32;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Sum over the CTA, the same bits in every thread: warp sums, then every
// thread adds the warps' sums in order.  `slot` alternates between calls, so
// one barrier per sum is enough.
__device__ __forceinline__ float block_sum(float v, float (*slot)[kMaxWarps], int which) {
    v = warp_sum(v);
    const int warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    if (nwarps == 1) return v;
    if ((threadIdx.x & 31) == 0) slot[which][warp] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < nwarps; ++w) s += slot[which][w];
    return s;
}

__device__ __forceinline__ float act_of(float g, uint32_t flags) {
    if (flags & (PQ2_GATE_SIGMOID | PQ2_GATE_SILU)) {
        // the fast exponential and quotient: within 4 + 1.2 |g| ulp of the factor.
        // exp overflows to inf for a very negative g: the quotient is then 0
        const float s = __fdividef(1.0f, 1.0f + __expf(-g));
        return flags & PQ2_GATE_SILU ? g * s : s;
    }
    return g;
}

// The values of a row that a thread owns: vectors tid, tid + T, ... of V.
template <int V, int VPT, bool kAfter, bool kWarpRow>
__global__ void __launch_bounds__(512)
    norm_kernel(pq2h::NormParams p) {
    __shared__ float slot[2][kMaxWarps];
    const int T = kWarpRow ? 32 : static_cast<int>(blockDim.x);
    const int tid = kWarpRow ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
    const int rows_per_cta = kWarpRow ? static_cast<int>(blockDim.x >> 5) : 1;
    long long row = static_cast<long long>(blockIdx.x) * rows_per_cta +
                    (kWarpRow ? (threadIdx.x >> 5) : 0);
    const long long step = static_cast<long long>(gridDim.x) * rows_per_cta;
    const float inv_h = 1.0f / static_cast<float>(p.H);

    int idx[VPT];
    bool in[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        idx[i] = (tid + i * T) * V;
        in[i] = idx[i] < p.H;
    }
    if (!p.weights_static) pdl_wait();
    // the weights, once per CTA
    RawVec<V> wp[VPT], wn[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        wp[i] = wn[i] = raw_zero<V>();
        if (in[i] && kAfter && p.w_post) wp[i] = raw_load<V>(p.w_post, p.w_type, idx[i]);
        if (in[i] && p.w_next) wn[i] = raw_load<V>(p.w_next, p.w_type, idx[i]);
    }
    if (p.weights_static) pdl_wait();
    pdl_launch_dependents();

    for (; row < p.M; row += step) {
        RawVec<V> ry[VPT], rr[VPT], rg[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            ry[i] = rr[i] = rg[i] = raw_zero<V>();
            if (!in[i]) continue;
            if constexpr (kAfter) ry[i] = raw_load<V>(p.y, p.y_type, row * p.ld_y + idx[i]);
            rr[i] = raw_load<V>(p.r, p.r_type, row * p.ld_r + idx[i]);
            if (kAfter && p.gate) rg[i] = raw_load<V>(p.gate, p.gate_type, row * p.ld_gate + idx[i]);
        }
        float r[VPT][V];
        float ss = 0.0f;
        if constexpr (kAfter) {
            float y[VPT][V];
#pragma unroll
            for (int i = 0; i < VPT; ++i) raw_to_f32<V>(ry[i], p.y_type, y[i]);
            float scale = p.alpha;
            if (!(p.flags & PQ2_NORM_NO_POST)) {
                float s2 = 0.0f;
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) s2 = fmaf(y[i][j], y[i][j], s2);
                s2 = kWarpRow ? warp_sum(s2) : block_sum(s2, slot, 0);
                scale *= rsqrtf(s2 * inv_h + p.eps);
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float w[V], g[V];
                raw_to_f32<V>(wp[i], p.w_type, w);
                raw_to_f32<V>(rg[i], p.gate_type, g);
                raw_to_f32<V>(rr[i], p.r_type, r[i]);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float n = y[i][j] * scale;
                    if (p.w_post) n *= w[j] + p.w_offset;
                    if (p.gate) n *= act_of(g[j], p.flags);
                    r[i][j] += n;
                    ss = in[i] ? fmaf(r[i][j], r[i][j], ss) : ss;
                }
                const long long o = row * p.ld_ro + idx[i];
                if (in[i] && store_ok(p.ctl, o, V, p.ro_elems))
                    store_f32<V>(p.r_out, p.r_type, o, r[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                raw_to_f32<V>(rr[i], p.r_type, r[i]);
#pragma unroll
                for (int j = 0; j < V; ++j) ss = fmaf(r[i][j], r[i][j], ss);
            }
        }
        if (p.x) {
            ss = kWarpRow ? warp_sum(ss) : block_sum(ss, slot, 1);
            const float scale = rsqrtf(ss * inv_h + p.eps);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float w[V];
                raw_to_f32<V>(wn[i], p.w_type, w);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    r[i][j] *= scale;
                    if (p.w_next) r[i][j] *= w[j] + p.w_offset;
                }
                const long long o = row * p.ld_x + idx[i];
                if (in[i] && store_ok(p.ctl, o, V, p.x_elems))
                    store_f32<V>(p.x, p.x_type, o, r[i]);
            }
        }
        // slot 0 of the next row is written only after every thread has
        // passed this row's second barrier; without one (no x), and for a
        // norm before a block alone (slot 1 every time), wait here
        if (!kWarpRow && (!kAfter || !p.x || (p.flags & PQ2_NORM_NO_POST))) __syncthreads();
    }
}

// Rows of any width up to PQ2_NORM_MAX_H: the row (y, then r') waits in
// shared memory as fp32 between the passes.
template <bool kAfter>
__global__ void __launch_bounds__(1024) norm_wide_kernel(pq2h::NormParams p) {
    extern __shared__ float buf[];
    __shared__ float slot[2][kMaxWarps];
    const float inv_h = 1.0f / static_cast<float>(p.H);
    pdl_wait();
    pdl_launch_dependents();
    for (long long row = blockIdx.x; row < p.M; row += gridDim.x) {
        float scale = p.alpha;
        float ss = 0.0f;
        if constexpr (kAfter) {
            float s2 = 0.0f;
            for (int e = threadIdx.x; e < p.H; e += blockDim.x) {
                float v[1];
                raw_to_f32<1>(raw_load<1>(p.y, p.y_type, row * p.ld_y + e), p.y_type, v);
                buf[e] = v[0];  // read again by the same thread only
                s2 = fmaf(v[0], v[0], s2);
            }
            if (!(p.flags & PQ2_NORM_NO_POST)) {
                s2 = block_sum(s2, slot, 0);
                scale *= rsqrtf(s2 * inv_h + p.eps);
            }
        }
        for (int e = threadIdx.x; e < p.H; e += blockDim.x) {
            float r[1], w[1], g[1];
            raw_to_f32<1>(raw_load<1>(p.r, p.r_type, row * p.ld_r + e), p.r_type, r);
            if constexpr (kAfter) {
                float n = buf[e] * scale;
                if (p.w_post) {
                    raw_to_f32<1>(raw_load<1>(p.w_post, p.w_type, e), p.w_type, w);
                    n *= w[0] + p.w_offset;
                }
                if (p.gate) {
                    raw_to_f32<1>(raw_load<1>(p.gate, p.gate_type, row * p.ld_gate + e), p.gate_type,
                                  g);
                    n *= act_of(g[0], p.flags);
                }
                r[0] += n;
                const long long o = row * p.ld_ro + e;
                if (store_ok(p.ctl, o, 1, p.ro_elems)) store_f32<1>(p.r_out, p.r_type, o, r);
            }
            buf[e] = r[0];
            ss = fmaf(r[0], r[0], ss);
        }
        if (p.x) {
            ss = block_sum(ss, slot, 1);
            const float sx = rsqrtf(ss * inv_h + p.eps);
            for (int e = threadIdx.x; e < p.H; e += blockDim.x) {
                float v[1] = {buf[e] * sx}, w[1];
                if (p.w_next) {
                    raw_to_f32<1>(raw_load<1>(p.w_next, p.w_type, e), p.w_type, w);
                    v[0] *= w[0] + p.w_offset;
                }
                const long long o = row * p.ld_x + e;
                if (store_ok(p.ctl, o, 1, p.x_elems)) store_f32<1>(p.x, p.x_type, o, v);
            }
        }
        __syncthreads();  // the slots are free for the next row
    }
}

// Many rows: a bulk-copy ring.  One CTA per SM walks over rows; a producer
// warp keeps the next rows' y, r and gate on their way into shared memory
// (stages rows deep, whatever registers and barriers are doing), and groups of
// warps take the rows in turn, one row a group.  Both weight vectors (a gate
// that is one vector is folded into the first) wait in shared memory as fp32.
constexpr int kRingVpt = 4;            // vectors of 4 values per thread
constexpr int kRingMaxGroups = 12;     // named barriers 1 .. 12
constexpr int kRingMaxWarps = 23;      // consumer warps (and one producer): 80 registers
constexpr int kRingMaxStages = 16;

// This thread's values of a row in shared memory (vectors t, t + threads, ...
// of 4; zeros past H, which no thread has where kFull).  The type is asked once per row, not per vector.
template <int kType, bool kFull>
__device__ __forceinline__ void lds_values(const uint8_t* base, int t, int threads, int H,
                                           float (&v)[kRingVpt][4]) {
#pragma unroll
    for (int k = 0; k < kRingVpt; ++k) {
        const int e = (t + k * threads) * 4;
        if constexpr (kType == PQ2_F32) {
            const float4 f = kFull || e < H ? *reinterpret_cast<const float4*>(base + e * 4)
                                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            v[k][0] = f.x, v[k][1] = f.y, v[k][2] = f.z, v[k][3] = f.w;
        } else {
            const uint2 u = kFull || e < H ? *reinterpret_cast<const uint2*>(base + e * 2) : make_uint2(0, 0);
            const uint32_t w[2] = {u.x, u.y};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if constexpr (kType == PQ2_BF16) {
                    v[k][2 * j] = __uint_as_float(w[j] << 16);
                    v[k][2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                    v[k][2 * j] = f.x;
                    v[k][2 * j + 1] = f.y;
                }
            }
        }
    }
}
template <bool kFull>
__device__ __forceinline__ void lds_row(const uint8_t* base, int type, int t, int threads, int H,
                                        float (&v)[kRingVpt][4]) {
    if (type == PQ2_F32)
        lds_values<PQ2_F32, kFull>(base, t, threads, H, v);
    else if (type == PQ2_BF16)
        lds_values<PQ2_BF16, kFull>(base, t, threads, H, v);
    else
        lds_values<PQ2_F16, kFull>(base, t, threads, H, v);
}

template <int kType, bool kFull>
__device__ __forceinline__ void store_values(const DevCtl& ctl, void* out, long long o, long long n,
                                             int t, int threads, int H,
                                             const float (&v)[kRingVpt][4]) {
#pragma unroll
    for (int k = 0; k < kRingVpt; ++k) {
        const int e = (t + k * threads) * 4;
        if ((!kFull && e >= H) || !store_ok(ctl, o + e, 4, n)) continue;
        if constexpr (kType == PQ2_F32)
            *reinterpret_cast<float4*>(static_cast<float*>(out) + o + e) =
                make_float4(v[k][0], v[k][1], v[k][2], v[k][3]);
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + o + e) = make_uint2(
                f32x2_to_elem16(v[k][0], v[k][1], kType), f32x2_to_elem16(v[k][2], v[k][3], kType));
    }
}
template <bool kFull>
__device__ __forceinline__ void store_row(const DevCtl& ctl, void* out, int type, long long o,
                                          long long n, int t, int threads, int H,
                                          const float (&v)[kRingVpt][4]) {
    if (type == PQ2_F32)
        store_values<PQ2_F32, kFull>(ctl, out, o, n, t, threads, H, v);
    else if (type == PQ2_BF16)
        store_values<PQ2_BF16, kFull>(ctl, out, o, n, t, threads, H, v);
    else
        store_values<PQ2_F16, kFull>(ctl, out, o, n, t, threads, H, v);
}

// Four chains, so that no addition waits for the one before it.
__device__ __forceinline__ float sum_squares(const float (&v)[kRingVpt][4]) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kRingVpt; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = fmaf(v[k][j], v[k][j], s[j]);
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// Sum over a group of `threads` threads (named barrier `bar`); `bad` of any of
// them reaches all in `any`.
__device__ __forceinline__ float group_sum(float v, float* slot, int bar, int threads, bool bad,
                                           bool& any) {
    v = warp_sum(v);
    if (threads == 32) {
        any = bad;  // warp-uniform
        return v;
    }
    const int warp = (threadIdx.x % threads) >> 5, nwarps = threads >> 5, lane = threadIdx.x & 31;
    if (lane == 0) slot[warp] = v;
    any = named_bar_any(bar, threads, bad);
    // the warps' sums, added in the same order by every warp
    return warp_sum(lane < nwarps ? slot[lane] : 0.0f);
}

template <bool kAfter, bool kFull>
__global__ void __launch_bounds__((kRingMaxWarps + 1) * 32, 1)
    norm_ring_kernel(pq2h::NormParams p, int threads, int groups, int stages, int stage_bytes) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kRingMaxStages], empty[kRingMaxStages];
    __shared__ float slot[kRingMaxGroups][2][kRingMaxWarps];
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    uint8_t* ring = smem;
    float* w_post = reinterpret_cast<float*>(smem + static_cast<size_t>(stages) * stage_bytes);
    float* w_next = w_post + p.H;
    const int tid = threadIdx.x, lane = tid & 31;
    const int consumers = threads * groups;
    const bool producer = tid >= consumers;
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], threads / 32);
        }
        abort_word = 0;
        fence_mbar_init();
    }
    const int y_bytes = kAfter ? p.H * (p.y_type == PQ2_F32 ? 4 : 2) : 0;
    const int r_bytes = p.H * (p.r_type == PQ2_F32 ? 4 : 2);
    const bool gate_rows = kAfter && p.gate && p.ld_gate != 0;
    const bool gate_vec = kAfter && p.gate && p.ld_gate == 0;
    const int g_bytes = gate_rows ? p.H * (p.gate_type == PQ2_F32 ? 4 : 2) : 0;
    // rows of this CTA: blockIdx.x + i * gridDim.x, i < count
    const int count = static_cast<int>((p.M - blockIdx.x + gridDim.x - 1) / gridDim.x);
    __syncthreads();  // the barriers are there
    if (producer) {
        pdl_wait();
        pdl_launch_dependents();
        // lanes 0, 1, 2: the copies of y, r and the gate
        const int bytes = lane == 0 ? y_bytes : lane == 1 ? r_bytes : lane == 2 ? g_bytes : 0;
        const int at = lane == 0 ? 0 : lane == 1 ? y_bytes : y_bytes + r_bytes;
        const uint8_t* src = static_cast<const uint8_t*>(lane == 0 ? p.y : lane == 1 ? p.r : p.gate);
        const long long ld =
            lane == 0 ? p.ld_y * (y_bytes / p.H)
                      : lane == 1 ? p.ld_r * (r_bytes / p.H) : p.ld_gate * (g_bytes / p.H);
        src += blockIdx.x * ld;
        int i = 0, s = 0;
        uint32_t turn = 0;  // times the ring has gone round
        for (; i < count; ++i) {
            if (turn > 0 && !mbar_ready_warp(&empty[s], (turn - 1) & 1, p.ctl, abort_flag)) break;
            if (i != p.ctl.debug_skip_stage) {  // else withheld (timeout test)
                if (lane == 0) mbar_arrive_expect_tx(&full[s], y_bytes + r_bytes + g_bytes);
                __syncwarp();
                if (bytes > 0)
                    bulk_g2s(ring + static_cast<size_t>(s) * stage_bytes + at,
                             src + static_cast<long long>(i) * gridDim.x * ld, bytes, &full[s]);
            }
            if (++s == stages) s = 0, ++turn;
        }
        // the last copies land before the CTA ends, whatever the consumers do
        for (int k = max(0, i - stages); k < i; ++k)
            if (k != p.ctl.debug_skip_stage)
                mbar_ready_warp(&full[k % stages], static_cast<uint32_t>(k / stages) & 1, p.ctl);
        return;
    }
    if (!p.weights_static) pdl_wait();
    // eight weights a thread, every load before the first conversion: one
    // trip to L2 (value by value this took 9 us).  A gate vector is no weight:
    // the kernel before may be writing it, whatever the flag says
    for (int e = tid * 8; e < p.H; e += consumers * 8) {
        RawVec<8> rp = raw_zero<8>(), rg = rp, rn = rp;
        if (kAfter && p.w_post) rp = raw_load<8>(p.w_post, p.w_type, e);
        if (p.w_next) rn = raw_load<8>(p.w_next, p.w_type, e);
        if (gate_vec) {
            pdl_wait();   // at once where it has been waited for
            rg = raw_load<8>(p.gate, p.gate_type, e);
        }
        float v[8], g[8], n[8];
        raw_to_f32<8>(rp, p.w_type, v);
        raw_to_f32<8>(rg, p.gate_type, g);
        raw_to_f32<8>(rn, p.w_type, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = p.w_post ? v[j] + p.w_offset : 1.0f;
            if (gate_vec) v[j] *= act_of(g[j], p.flags);
            w_post[e + j] = v[j];
            w_next[e + j] = p.w_next ? n[j] + p.w_offset : 1.0f;
        }
    }
    if (p.weights_static) pdl_wait();
    pdl_launch_dependents();
    named_bar_sync(kRingMaxGroups + 1, consumers);  // the weights are there

    const int group = tid / threads, t = tid % threads;
    const int bar = 1 + group;
    const float inv_h = 1.0f / static_cast<float>(p.H);
    int s = group % stages;
    uint32_t turn = group / stages;
    for (int i = group; i < count; i += groups) {
        const long long row = blockIdx.x + static_cast<long long>(i) * gridDim.x;
        const bool ok = mbar_ready_warp(&full[s], turn & 1, p.ctl, abort_flag);
        if (!ok) *abort_flag = 1;
        const uint8_t* st = ring + static_cast<size_t>(s) * stage_bytes;
        float y[kRingVpt][4], r[kRingVpt][4];
        bool failed = false;
        float scale = p.alpha;
        if constexpr (kAfter) {
            lds_row<kFull>(st, p.y_type, t, threads, p.H, y);
            if (!(p.flags & PQ2_NORM_NO_POST)) {
                float s2 = sum_squares(y);
                s2 = group_sum(s2, slot[group][0], bar, threads, !ok, failed);
                scale *= rsqrtf(s2 * inv_h + p.eps);
            }
            if (gate_rows) {
                lds_row<kFull>(st + y_bytes + r_bytes, p.gate_type, t, threads, p.H, r);
                if (p.flags & (PQ2_GATE_SIGMOID | PQ2_GATE_SILU)) {
#pragma unroll
                    for (int k = 0; k < kRingVpt; ++k)
#pragma unroll
                        for (int j = 0; j < 4; ++j) r[k][j] = act_of(r[k][j], p.flags);
                }
#pragma unroll
                for (int k = 0; k < kRingVpt; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[k][j] *= r[k][j];
            }
        }
        lds_row<kFull>(st + y_bytes, p.r_type, t, threads, p.H, r);
        // every value of the stage is in registers: back to the producer
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&empty[s]);
        s += groups;
        while (s >= stages) s -= stages, ++turn;
        if (failed || (!ok && threads == 32)) return;  // uniform over the group
#pragma unroll
        for (int k = 0; k < kRingVpt; ++k) {
            if constexpr (kAfter) {
                const int e = (t + k * threads) * 4;
                const float4 w = kFull || e < p.H ? *reinterpret_cast<const float4*>(w_post + e)
                                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                r[k][0] = fmaf(y[k][0] * scale, w.x, r[k][0]);
                r[k][1] = fmaf(y[k][1] * scale, w.y, r[k][1]);
                r[k][2] = fmaf(y[k][2] * scale, w.z, r[k][2]);
                r[k][3] = fmaf(y[k][3] * scale, w.w, r[k][3]);
            }
        }
        if (kAfter && ok)
            store_row<kFull>(p.ctl, p.r_out, p.r_type, row * p.ld_ro, p.ro_elems, t, threads, p.H, r);
        if (p.x) {
            const float ss = group_sum(sum_squares(r), slot[group][1], bar, threads, !ok, failed);
            if (failed) return;
            const float sx = rsqrtf(ss * inv_h + p.eps);
#pragma unroll
            for (int k = 0; k < kRingVpt; ++k) {
                const int e = (t + k * threads) * 4;
                const float4 w = kFull || e < p.H ? *reinterpret_cast<const float4*>(w_next + e)
                                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                r[k][0] *= sx * w.x, r[k][1] *= sx * w.y, r[k][2] *= sx * w.z, r[k][3] *= sx * w.w;
            }
            store_row<kFull>(p.ctl, p.x, p.x_type, row * p.ld_x, p.x_elems, t, threads, p.H, r);
        }
        // slot 1 (or 0) may be written again only once all have read it:
        // the other sum's barrier separates two rows; with one sum a row,
        // or none, this one does (and agrees on a failed wait)
        if (threads > 32 && (!kAfter || !p.x || (p.flags & PQ2_NORM_NO_POST)) &&
            named_bar_any(bar, threads, !ok))
            return;
    }
}

}  // namespace
}  // namespace pq2

namespace pq2h {

namespace {

constexpr int kRingMaxH = 8192;
// The ring from four rows per SM on, wide rows from one: it keeps one row's
// loads in flight while another is summed, but starts later (both weight
// vectors into shared memory first).  bf16 r, fp16 y, us with and without it:
// 4096 rows of 5120 35.8 and 82.8, of 1024 10.7 and 13.2; 1000 of 2560 5.8 and
// 9.5; 200 of 5120 5.0 and 5.9; 608 of 1024 3.3 and 3.0; 320 of 2560 3.7 and
// 3.6; 128 of 5120 4.5 and 3.3.  Where the ring begins the two are within 0.3 us
// of each other (narrow rows are a little better off without it there).
constexpr int kRingMinRows = 4;
constexpr int64_t kRingMinValues = 900000;

bool takes_ring(int64_t M, int64_t H, int64_t sms) {
    return H > 512 && H <= kRingMaxH &&
           (M >= kRingMinRows * sms || (M >= sms && M * H >= kRingMinValues));
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// 16-byte vectors of 8 elements: every row starts on a 16-byte boundary
// (row strides are multiples of 8 elements where they are used).
bool rows_on16(const void* p, int64_t ld) { return !p || (on16(p) && ld % 8 == 0); }

template <int V, int VPT, bool kAfter, bool kWarpRow>
cudaError_t go(const NormParams& p, int threads, int rows_per_cta, int64_t ctas, cudaStream_t st) {
    const int64_t need = (p.M + rows_per_cta - 1) / rows_per_cta;
    return launch(pq2::norm_kernel<V, VPT, kAfter, kWarpRow>,
                  dim3(static_cast<unsigned>(std::min(need, ctas))), dim3(threads), 0, st, true, p);
}

template <bool kAfter>
cudaError_t route(const NormParams& p, cudaStream_t st, const DeviceInfo& dev) {
    const int H = static_cast<int>(p.H);
    const bool vec = H % 8 == 0 && rows_on16(p.y, p.ld_y) && rows_on16(p.r, p.ld_r) &&
                     rows_on16(p.r_out, p.ld_ro) && rows_on16(p.gate, p.ld_gate) &&
                     rows_on16(p.x, p.ld_x) && rows_on16(p.w_post, 0) && rows_on16(p.w_next, 0);
    const int64_t sms = dev.num_sms;
    if (vec && takes_ring(p.M, H, sms)) {
        // whole warps of 16 values a thread, as many groups as fit 23 warps
        const int threads = (H / 4 + pq2::kRingVpt * 32 - 1) / (pq2::kRingVpt * 32) * 32;
        int groups = std::min(pq2::kRingMaxGroups, pq2::kRingMaxWarps * 32 / threads);
        auto bytes = [&](int type) { return H * (type == PQ2_F32 ? 4 : 2); };
        const int stage = bytes(p.r_type) + (kAfter ? bytes(p.y_type) : 0) +
                          (kAfter && p.gate && p.ld_gate != 0 ? bytes(p.gate_type) : 0);
        const int room = dev.max_smem_optin - 4096 - 8 * H;
        int stages = std::min(pq2::kRingMaxStages, room / stage);
        if (stages >= 3) {
            // whole turns of the groups: a stage is always the same group's,
            // which sees each phase of its barrier (a parity says no more)
            groups = std::min(groups, stages);
            stages -= stages % groups;
            const bool full = H == threads * pq2::kRingVpt * 4;
            auto kern = full ? pq2::norm_ring_kernel<kAfter, true> : pq2::norm_ring_kernel<kAfter, false>;
            static SmemLimit lim[2];
            const size_t smem = static_cast<size_t>(stages) * stage + 8 * static_cast<size_t>(H);
            const cudaError_t e = raise_smem(lim[full], kern, smem);
            if (e != cudaSuccess) return e;
            return launch(kern, dim3(static_cast<unsigned>(sms)), dim3(threads * groups + 32), smem, st,
                          true, p, threads, groups, stages, stage);
        }
    }
    // a warp per row: 4096 rows of 512 5.9 us against 6.0 a CTA each, of 128 5.1
    // and 5.2, of 255 values one by one 6.7 and 6.7; 64 of 255 3.3 and 3.5
    if (vec && H <= 512) return go<8, 2, kAfter, true>(p, 256, 8, sms * 4, st);
    if (vec && H <= 8192) {
        // two vectors of 8 a thread: H may end half way through the last one's
        const int threads = ((H + 15) / 16 + 31) / 32 * 32;
        return go<8, 2, kAfter, false>(p, threads, 1, sms * std::max(1, 1280 / threads), st);
    }
    if (H <= 256) return go<1, 8, kAfter, true>(p, 256, 8, sms * 4, st);
    if (H <= 4096) {
        const int threads = ((H + 7) / 8 + 31) / 32 * 32;
        return go<1, 8, kAfter, false>(p, threads, 1, sms * std::max(1, 1280 / threads), st);
    }
    static SmemLimit lim;
    const size_t smem = static_cast<size_t>(H) * 4;
    cudaError_t e = raise_smem(lim, pq2::norm_wide_kernel<kAfter>, smem);
    if (e != cudaSuccess) return e;
    return launch(pq2::norm_wide_kernel<kAfter>,
                  dim3(static_cast<unsigned>(std::min<int64_t>(p.M, sms * 2))), dim3(1024), smem, st,
                  true, p);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t st, const DeviceInfo& dev) {
    return p.y ? route<true>(p, st, dev) : route<false>(p, st, dev);
}

}  // namespace pq2h
