// Verification of drafted tokens: the step after the lm_head when M = drafts
// + 1 token rows of a sequence went through the model at once.  For each
// sequence, with p_i = softmax(logits_i / T) and q_i the drafter's
// probabilities at position i:
//
//   draft d_i is taken while u_i q_i(d_i) < p_i(d_i);
//   the token after the taken ones is argmax_v w(v) / e(v), e(v) ~ Exp(1),
//   w = max(p_i - q_i, 0) at the first refused draft, w = p_n if none is.
//
// argmax_v w(v) / e(v) draws v with probability w(v) / sum w (the smallest of
// exponential variables e(v) / w(v)), so the drawn tokens follow the target's
// distribution, and no prefix sum over the vocabulary is needed.
// T = 0: drafts are taken while they are the argmax, and the argmax follows.
//
// Bound by HBM: one pass over all logits rows, and one over a single row of
// logits (mostly still in L2), q and e per sequence.  Two kernels:
//   verify_stats_kernel  splits every row into pieces of kPiece values; a
//       thread holds its values in registers, so maximum and sum of
//       exponentials take one read and no rescaling within a piece.
//   verify_pick_kernel   spans of each sequence's chosen row; every CTA joins
//       the pieces' statistics of the sequence's rows, finds the first refusal
//       (the same arithmetic in each CTA) and reduces its span to one 64-bit
//       key (score bits, then lowest index first).  atomicMax
//       joins the keys: the maximum does not depend on the order.  The last
//       CTA of a sequence writes the result.
// Measured: one sequence of 4 rows of 248320 6.9 us; 64 of them 76 us, 5.0
// TB/s of the bytes that the call cannot do without (the first kernel alone 5.6
// TB/s).
#include <algorithm>
#include <cfloat>
#include <climits>

#include "pq2_common.cuh"
#include "pq2_internal.h"
#include "pq2_step.cuh"

namespace pq2 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 2;                            // 16-byte vectors per thread and array at once
constexpr int kStatVecs = 8;                        // of stats (4: 5 us more for 256 rows)
constexpr int kPiece = kThreads * kStatVecs * 4;    // values of a row per CTA of stats
constexpr int kPickPiece = kThreads * kVecs * 4;    // and per round of a CTA of pick
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Values e .. e + 3 of a row of V values, with `fill` outside [0, V); `vec`:
// e is on a 16-byte boundary of the row's memory.
__device__ __forceinline__ float4 load4(const float* row, int e, int V, bool vec, float fill) {
    if (vec && e >= 0 && e + 3 < V) return *reinterpret_cast<const float4*>(row + e);
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (e + j >= 0 && e + j < V) ? row[e + j] : fill;
    return make_float4(v[0], v[1], v[2], v[3]);
}

// Number of values between the 16-byte boundary below `p` and `p`.
__device__ __forceinline__ int lead(const float* p) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(p) >> 2) & 3u);
}

// 1 / temperature in units of log2(e); 0 selects the greedy rule.  A
// temperature is never taken for greedy because it is large (infinite: every
// allowed value alike), and 0 times a tiny one's scale stays 0: the scale is
// kept between the smallest and the largest finite number.
__device__ __forceinline__ float scale_of(float temperature) {
    return temperature > 0.0f ? fminf(fmaxf(kLog2e / temperature, FLT_TRUE_MIN), FLT_MAX) : 0.0f;
}

// The later of two (maximum, lowest index) pairs.
__device__ __forceinline__ void best_of(float& m, int& at, float m2, int at2) {
    if (m2 > m || (m2 == m && at2 < at)) {
        m = m2;
        at = at2;
    }
}

// (maximum, sum of exponentials relative to it) of two pieces.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2, float c) {
    const float top = fmaxf(m, m2);
    if (top == neg_inf()) return;  // both empty: s = 0
    s = s * ex2((m - top) * c) + s2 * ex2((m2 - top) * c);
    m = top;
}

__global__ void __launch_bounds__(kThreads) verify_stats_kernel(pq2h::VerifyParams p) {
    __shared__ float sm[kWarps], ss[kWarps];
    __shared__ int si[kWarps];
    __shared__ float s_scale;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x / p.chunks;
    const int chunk = static_cast<int>(blockIdx.x - row * p.chunks);
    pdl_wait();
    pdl_launch_dependents();
    const float* l = p.logits + row * p.ld_logits;
    const int e0 = chunk * kPiece - lead(l);
    float v[kStatVecs][4];
#pragma unroll
    for (int i = 0; i < kStatVecs; ++i) {
        const float4 f = load4(l, e0 + (i * kThreads + tid) * 4, p.V, true, neg_inf());
        v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
    }
    if (blockIdx.x == 0) {
        for (long long b = tid; b < p.B; b += kThreads) {
            p.keys[2 * b] = p.keys[2 * b + 1] = 0ull;
            p.done[b] = 0u;
        }
    }
    // the temperature of the row's sequence, the one whose range is sound and
    // has the row (a broken range elsewhere says nothing about this row); loaded
    // with the ranges, not after them (one sequence: 6.9 us against 7.1)
    bool found = false;
    for (long long b = tid; b < p.B; b += kThreads) {
        const int r0 = p.row_start[b], r1 = p.row_start[b + 1];
        const float temperature = p.temperature[b];
        if (r0 >= 0 && r0 <= row && row < r1 && r1 <= p.rows) {
            s_scale = scale_of(temperature);
            found = true;
        }
    }
    const float c = __syncthreads_or(found) ? s_scale : 0.0f;

    float m = neg_inf();
    int at = INT_MAX;
#pragma unroll
    for (int i = 0; i < kStatVecs; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (v[i][j] > m) {
                m = v[i][j];
                at = e0 + (i * kThreads + tid) * 4 + j;
            }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        best_of(m, at, __shfl_xor_sync(0xffffffffu, m, off), __shfl_xor_sync(0xffffffffu, at, off));
    if (lane == 0) sm[warp] = m, si[warp] = at;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) best_of(m, at, sm[w], si[w]);
    float s = 0.0f;
    if (m > neg_inf()) {
#pragma unroll
        for (int i = 0; i < kStatVecs; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s += ex2((v[i][j] - m) * c);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) ss[warp] = s;
    __syncthreads();
    if (tid == 0) {
        s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += ss[w];
        if (store_ok(p.ctl, blockIdx.x, 1, p.rows * p.chunks)) {
            p.stats[blockIdx.x] = make_float2(m, s);
            p.best[blockIdx.x] = at;
        }
    }
}

// Score and index as one key: larger scores first, then lower indexes; 0 for
// a value that cannot be drawn.
__device__ __forceinline__ unsigned long long key_of(float score, int at) {
    return score > 0.0f ? (static_cast<unsigned long long>(__float_as_uint(score)) << 32) |
                              (0xffffffffu - static_cast<unsigned>(at))
                        : 0ull;
}

// What a warp needs to decide one row's draft; none of it comes from
// verify_stats_kernel.
struct RowTest {
    bool last;          // no draft to test: the sequence ends here
    int d;
    float l, q, u;      // its logit, the drafter's probability, the uniform
};
__device__ __forceinline__ RowTest row_test(const pq2h::VerifyParams& p, int row, int r1,
                                            bool greedy) {
    RowTest r = {true, 0, 0.0f, 1.0f, 0.0f};
    if (row >= r1) return r;
    r.d = __ldcg(p.drafts + row);
    r.last = row == r1 - 1 || r.d < 0 || r.d >= p.V;
    if (!r.last && !greedy) {
        r.l = __ldcg(p.logits + row * p.ld_logits + r.d);
        r.u = __ldcg(p.u + row);
        if (p.q) r.q = __ldcg(p.q + row * p.ld_q + r.d);
    }
    return r;
}

// CTA (span of pieces, sequence).  What does not come from
// verify_stats_kernel is read before the dependency wait: that kernel lets
// this one start only after its own wait, so everything before it is done.
__global__ void __launch_bounds__(kThreads) verify_pick_kernel(pq2h::VerifyParams p, int spans,
                                                               int pieces) {
    __shared__ int s_stop;
    __shared__ float s_max, s_inv;
    __shared__ int s_best, s_refused, s_draft;
    __shared__ unsigned long long sk[2][kWarps];
    __shared__ bool s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / spans, span = blockIdx.x - b * spans;
    if (tid == 0) s_stop = INT_MAX;
    const int r0 = __ldcg(p.row_start + b), r1 = __ldcg(p.row_start + b + 1);
    const float c = scale_of(__ldcg(p.temperature + b));
    const bool greedy = c == 0.0f;
    const bool bad = r0 < 0 || r1 < r0 || r1 > p.rows;
    if (bad || r0 == r1) {  // uniform over the CTA
        pdl_wait();
        if (tid == 0 && span == 0) {
            if (bad) atomicOr(p.ctl.err, DEVERR_BAD_INDEX);
            if (store_ok(p.ctl, b, 1, p.B)) p.accepted[b] = 0;
        }
        return;
    }
    RowTest test = row_test(p, r0 + warp, r1, greedy);
    const float* e = p.e + b * p.ld_e;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    // A warp per row, a round of kWarps rows at a time: join the row's pieces
    // and decide its draft.  The first row that stops ends the search.
    for (int base = r0; base < r1; base += kWarps) {
        const int row = base + warp;
        if (base > r0) test = row_test(p, row, r1, greedy);
        float m = neg_inf(), s = 0.0f;
        int at = INT_MAX;
        bool stops = false, refused = false;
        if (row < r1) {
            const long long o = static_cast<long long>(row) * p.chunks;
            for (int k = lane; k < p.chunks; k += 32) {
                const float2 f = p.stats[o + k];
                if (greedy) {
                    best_of(m, at, f.x, p.best[o + k]);
                } else {
                    join(m, s, f.x, f.y, c);
                }
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                const float m2 = __shfl_xor_sync(0xffffffffu, m, off);
                const float s2 = __shfl_xor_sync(0xffffffffu, s, off);
                const int at2 = __shfl_xor_sync(0xffffffffu, at, off);
                if (greedy)
                    best_of(m, at, m2, at2);
                else
                    join(m, s, m2, s2, c);
            }
            bool take = false;
            if (!test.last) {
                if (greedy)
                    take = test.d == at;
                else if (s > 0.0f)
                    take = test.u * test.q < ex2((test.l - m) * c) / s;
            }
            stops = !take;
            refused = stops && !test.last;
            if (stops && lane == 0) atomicMin(&s_stop, row);
        }
        __syncthreads();
        const int stop = s_stop;
        __syncthreads();  // read by all before the next round's atomicMin
        if (stop != INT_MAX) {
            if (row == stop && lane == 0) {
                s_max = m;
                s_inv = s > 0.0f ? 1.0f / s : 0.0f;
                s_best = at;
                s_refused = refused;
                s_draft = test.d;
            }
            break;
        }
    }
    __syncthreads();
    const int stop = s_stop;
    const bool refused = s_refused != 0;
    if (greedy) {
        if (span != 0) return;
    } else {
        const float m = s_max, inv = s_inv;
        const int d = s_draft;
        const float* l = p.logits + stop * p.ld_logits;
        const float* q = refused && p.q ? p.q + stop * p.ld_q : nullptr;
        const int off = lead(l);
        const bool ve = lead(e) == off, vq = q && lead(q) == off;
        unsigned long long k0 = 0, k1 = 0;
        // two pieces in turn: one is on its way while the other is reduced
        float4 lv[2][kVecs], ev[2][kVecs], qv[2][kVecs];
        const auto fetch = [&](int slot, int piece) {
            const int e0 = (span * pieces + piece) * kPickPiece - off;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int v0 = e0 + (i * kThreads + tid) * 4;
                lv[slot][i] = load4(l, v0, p.V, true, neg_inf());
                ev[slot][i] = load4(e, v0, p.V, ve, 1.0f);
                qv[slot][i] = q ? load4(q, v0, p.V, vq, 0.0f) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
        };
        const auto reduce = [&](int slot, int piece) {
            const int e0 = (span * pieces + piece) * kPickPiece - off;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int v0 = e0 + (i * kThreads + tid) * 4;
                const float4 lf = lv[slot][i], ef = ev[slot][i], qf = qv[slot][i];
                const float lj[4] = {lf.x, lf.y, lf.z, lf.w};
                const float ej[4] = {ef.x, ef.y, ef.z, ef.w};
                const float qj[4] = {qf.x, qf.y, qf.z, qf.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float pv = ex2((lj[j] - m) * c) * inv;
                    float w = pv;
                    if (refused) w = q ? pv - qj[j] : (v0 + j == d ? 0.0f : pv);
                    const unsigned long long a = key_of(__fdividef(w, ej[j]), v0 + j);
                    k0 = a > k0 ? a : k0;
                    if (refused) {
                        const unsigned long long t = key_of(__fdividef(pv, ej[j]), v0 + j);
                        k1 = t > k1 ? t : k1;
                    }
                }
            }
        };
        if (m > neg_inf()) {
            fetch(0, 0);
            for (int piece = 0; piece < pieces; piece += 2) {
                if (piece + 1 < pieces) fetch(1, piece + 1);
                reduce(0, piece);
                if (piece + 1 == pieces) break;
                if (piece + 2 < pieces) fetch(0, piece + 2);
                reduce(1, piece + 1);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long a = __shfl_xor_sync(0xffffffffu, k0, o);
            const unsigned long long t = __shfl_xor_sync(0xffffffffu, k1, o);
            k0 = a > k0 ? a : k0;
            k1 = t > k1 ? t : k1;
        }
        if (lane == 0) sk[0][warp] = k0, sk[1][warp] = k1;
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < kWarps; ++w) {
                k0 = sk[0][w] > k0 ? sk[0][w] : k0;
                k1 = sk[1][w] > k1 ? sk[1][w] : k1;
            }
            // k1 counts only where no span has a k0
            if (k0)
                atomicMax(&p.keys[2 * b], k0);
            else if (k1)
                atomicMax(&p.keys[2 * b + 1], k1);
            s_last = atom_add_acq_rel_gpu(&p.done[b], 1u) + 1u == static_cast<unsigned>(spans);
        }
        __syncthreads();
        if (!s_last) return;
    }
    // the sequence's result
    int token;
    if (greedy) {
        token = s_max > neg_inf() ? s_best : -1;
    } else {
        unsigned long long k = __ldcg(&p.keys[2 * b]);
        if (k == 0) k = __ldcg(&p.keys[2 * b + 1]);  // p <= q everywhere: from p itself
        token = k ? static_cast<int>(0xffffffffu - static_cast<unsigned>(k)) : -1;
    }
    if (tid == 0 && store_ok(p.ctl, b, 1, p.B)) p.accepted[b] = stop - r0;
    for (int row = r0 + tid; row < r1; row += kThreads) {
        const int t = row < stop ? p.drafts[row] : row == stop ? token : -1;
        if (store_ok(p.ctl, row, 1, p.rows)) p.tokens[row] = t;
    }
}

}  // namespace
}  // namespace pq2

namespace pq2h {

namespace {

constexpr int64_t kPickCtas = 456;

int verify_chunks(int64_t V) {
    // up to three values before the first 16-byte boundary of a row
    return static_cast<int>((V + 3 + pq2::kPiece - 1) / pq2::kPiece);
}

size_t pad(size_t b) { return (b + 255) & ~size_t(255); }

}  // namespace

size_t verify_workspace_bytes(int64_t B, int64_t rows, int64_t V) {
    const size_t pieces = static_cast<size_t>(rows) * verify_chunks(V);
    return pad(pieces * 8) + pad(pieces * 4) + pad(static_cast<size_t>(B) * 16) +
           pad(static_cast<size_t>(B) * 4);
}

cudaError_t launch_verify(VerifyParams p, void* workspace, cudaStream_t st) {
    p.chunks = verify_chunks(p.V);
    const size_t pieces = static_cast<size_t>(p.rows) * p.chunks;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    p.stats = reinterpret_cast<float2*>(w);
    w += pad(pieces * 8);
    p.best = reinterpret_cast<int32_t*>(w);
    w += pad(pieces * 4);
    p.keys = reinterpret_cast<unsigned long long*>(w);
    w += pad(static_cast<size_t>(p.B) * 16);
    p.done = reinterpret_cast<unsigned*>(w);
    // without rows every sequence is empty: nothing to prepare for pick, which
    // then starts after all before it (it reads ahead of its dependency wait
    // because the statistics kernel has waited by then)
    if (pieces > 0) {
        const cudaError_t e = launch(pq2::verify_stats_kernel, dim3(static_cast<unsigned>(pieces)),
                                     dim3(pq2::kThreads), 0, st, true, p);
        if (e != cudaSuccess) return e;
    }
    // a CTA's start (the row's statistics, the decision) costs several trips to
    // L2: one residency in all (three CTAs per SM), each over a span of pieces.
    // 64 sequences of 248320: 76.2 us, with a third more 87.3; 16 sequences of
    // 128000: 17.5 and 20.1
    const int all = static_cast<int>((p.V + 3 + pq2::kPickPiece - 1) / pq2::kPickPiece);
    const int64_t most = std::max<int64_t>(1, kPickCtas / p.B);
    const int rounds = static_cast<int>((all + most - 1) / most);
    const int spans = (all + rounds - 1) / rounds;
    return launch(pq2::verify_pick_kernel, dim3(static_cast<unsigned>(p.B * spans)),
                  dim3(pq2::kThreads), 0, st, pieces > 0, p, spans, rounds);
}

}  // namespace pq2h
