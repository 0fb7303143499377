// Norms around a block of a serving step.  The pages time the projections;
// what stands between two of them is one pass over the residual stream:
//
//   before a block   x  = rms(r) * w
//   after a block    n  = rms(y) * w_post            (or n = y)
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
// values go one to a warp, without barriers.
#include <algorithm>

#include "pq2_common.cuh"
#include "pq2_elem.cuh"
#include "pq2_internal.h"

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

}  // namespace
}  // namespace pq2

namespace pq2h {

namespace {

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
    if (vec && H <= 512) return go<8, 2, kAfter, true>(p, 256, 8, sms * 4, st);
    if (vec && H <= 8192) {
        const int threads = (H / 16 + 31) / 32 * 32;
        return go<8, 2, kAfter, false>(p, threads, 1, sms * std::max(1, 1280 / threads), st);
    }
    if (H <= 256) return go<1, 8, kAfter, true>(p, 256, 8, sms * 4, st);
    if (H <= 4096) {
        const int threads = ((H + 7) / 8 + 31) / 32 * 32;
        return go<1, 8, kAfter, false>(p, threads, 1, sms * std::max(1, 1280 / threads), st);
    }
    static SmemLimit lim;
    const size_t smem = static_cast<size_t>(H) * 4;
    cudaError_t e = ensure_smem(lim, pq2::norm_wide_kernel<kAfter>, smem);
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
