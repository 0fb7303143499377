// The pages of a cache between two steps: which page each slot keeps, shares,
// copies or gets (update), which pages move so that those in use come first
// (compact), and the copies themselves.
//
// Update and compact are whole-number work on small arrays in L2 (a step of 64
// slots over 3400 pages: 45 KB), so they are bound by latency: one cluster
// of kCtas CTAs per call, its phases separated by cluster barriers.  Free
// pages, wanted pages and moves are numbered by prefix sums over pages and
// slots, and counts are joined by integer atomics, so the result does not
// depend on the order of anything.
//
// Copies are bound by memory: a page (a pair's whole row of heads) is cut into
// pieces of kPiece bytes, and the pieces of all pairs are dealt out to CTAs.
#include <algorithm>
#include <climits>

#include "pq2_common.cuh"
#include "pq2_internal.h"
#include "pq2_step.cuh"

namespace pq2 {
namespace {

constexpr int kCtas = 8;
constexpr int kThreads = 1024;
constexpr int kAll = kCtas * kThreads;

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sum of v over the threads before this one in the CTA, and over all of them.
__device__ __forceinline__ int scan(int v, int& total) {
    __shared__ int sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();  // (sums may still be read from the scan before)
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    const int w = sums[lane];
    int winc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, winc, o);
        if (lane >= o) winc += u;
    }
    total = __shfl_sync(0xffffffffu, winc, 31);
    return inc - v + (warp ? __shfl_sync(0xffffffffu, winc, warp - 1) : 0);
}

// The CTA's part of n things, and this thread's part of that, as [lo, hi).
struct Part {
    int lo, hi;
};
__device__ __forceinline__ Part part_of(int n) {
    const int per = (n + kAll - 1) / kAll;
    const long long i = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) * per;
    return {static_cast<int>(min(i, static_cast<long long>(n))), static_cast<int>(min(i + per, static_cast<long long>(n)))};
}

// The sums of the CTAs before this one (each has put its own into
// sums[blockIdx.x] before a cluster barrier), and of all.
__device__ __forceinline__ int before(const int32_t* sums, int& total) {
    int b = 0;
    total = 0;
    int v[kCtas];
#pragma unroll
    for (int c = 0; c < kCtas; ++c) v[c] = __ldcg(sums + c);
#pragma unroll
    for (int c = 0; c < kCtas; ++c) {
        if (c < static_cast<int>(blockIdx.x)) b += v[c];
        total += v[c];
    }
    return b;
}

__device__ __forceinline__ int up(int n, int T) { return n / T + (n % T != 0); }

// A slot's token count, kept within [0, W T].
__device__ __forceinline__ int in_range(int n, int most, bool& bad) {
    bad |= n < 0 || n > most;
    return min(max(n, 0), most);
}

__device__ __forceinline__ int page_at(const pq2h::PagesParams& p, int b, int j) {
    const int page = __ldcg(p.pages + b * p.ld_pages + j);
    return page >= 0 && page < p.P ? page : -1;
}

// What slot b keeps.
struct Keeps {
    int source, full, want;
    bool part;
};
__device__ __forceinline__ Keeps keeps_of(const pq2h::PagesParams& p, int b, bool& bad) {
    const int most = p.W * p.T;
    Keeps k;
    k.source = __ldcg(p.source + b);
    if (k.source >= p.B) k.source = -1, bad = true;
    const int wanted = in_range(__ldcg(p.new_lens + b), most, bad);
    int kept = 0;
    if (k.source >= 0) {
        bool other = false;  // (that slot reports its own)
        kept = min(min(in_range(__ldcg(p.keep + b), most, bad), wanted),
                   in_range(__ldcg(p.lens + k.source), most, other));
    }
    k.full = kept / p.T;
    k.part = kept % p.T != 0;
    k.want = up(wanted, p.T);
    return k;
}

// w0: holders outside the table, w1: holders of the whole page in the new
// table, w2: the lowest slot that keeps a part of it, w3: the free pages in
// ascending order.  s0: pages a slot has before it wants more, s1: its first
// wanted page's number, s2: its partly kept page, as the one it stays with
// (>= 0), the one it copies (-2 - page) or none (-1).
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    pages_update_kernel(const __grid_constant__ pq2h::PagesParams p) {
    const int tid = blockIdx.x * kThreads + threadIdx.x, lane = threadIdx.x & 31;
    const int warp = tid >> 5, warps = kAll / 32;
    bool bad = false;
    pdl_wait();
    pdl_launch_dependents();
    for (int i = tid; i < p.P; i += kAll) {
        p.w0[i] = __ldcg(p.refs + i);
        p.w1[i] = 0;
        p.w2[i] = INT_MAX;
    }
    cluster_sync();
    // a warp per slot: the pages that it held, and those that it goes on with
    for (int b = warp; b < p.B; b += warps) {
        const int held = up(in_range(__ldcg(p.lens + b), p.W * p.T, bad), p.T);
        const Keeps k = keeps_of(p, b, bad);
        for (int j = lane; j < max(held, k.full + k.part); j += 32) {
            if (j < held) {
                const int page = page_at(p, b, j);
                bad |= page < 0;
                if (page >= 0) atomicSub(p.w0 + page, 1);
            }
            if (j < k.full + k.part) {
                const int page = page_at(p, k.source, j);
                if (j < k.full) {
                    if (page >= 0) atomicAdd(p.w1 + page, 1);
                    if (store_ok(p.ctl, b * p.ld_out + j, 1, (p.B - 1) * p.ld_out + p.W))
                        p.pages_out[b * p.ld_out + j] = page;
                } else if (page >= 0) {
                    atomicMin(p.w2 + page, b);
                }
            }
        }
    }
    cluster_sync();
    // number the slots' wanted pages and the free pages
    const Part slots = part_of(p.B), pages = part_of(p.P);
    int wants = 0, frees = 0;
    for (int b = slots.lo; b < slots.hi; ++b) {
        const Keeps k = keeps_of(p, b, bad);
        int state = -1;
        if (k.part) {
            const int page = page_at(p, k.source, k.full);
            if (page >= 0)
                state = __ldcg(p.w0 + page) <= 0 && __ldcg(p.w1 + page) == 0 && __ldcg(p.w2 + page) == b
                            ? page
                            : -2 - page;
        }
        const int have = k.full + (state >= 0);
        p.s0[b] = have;
        p.s2[b] = state;
        wants += k.want - have;
    }
    for (int i = pages.lo; i < pages.hi; ++i)
        frees += __ldcg(p.w0 + i) <= 0 && __ldcg(p.w1 + i) == 0 && __ldcg(p.w2 + i) == INT_MAX;
    int all_wants, all_frees;
    const int want0 = scan(wants, all_wants), free0 = scan(frees, all_frees);
    if (threadIdx.x == 0) {
        p.sums[blockIdx.x] = all_wants;
        p.sums[kCtas + blockIdx.x] = all_frees;
    }
    cluster_sync();
    int w = want0 + before(p.sums, all_wants), f = free0 + before(p.sums + kCtas, all_frees);
    for (int b = slots.lo; b < slots.hi; ++b) {
        const Keeps k = keeps_of(p, b, bad);
        p.s1[b] = w;
        w += k.want - p.s0[b];
    }
    for (int i = pages.lo; i < pages.hi; ++i) {
        const int outside = __ldcg(p.w0 + i), whole = __ldcg(p.w1 + i);
        if (outside <= 0 && whole == 0 && __ldcg(p.w2 + i) == INT_MAX) p.w3[f++] = i;
        if (store_ok(p.ctl, i, 1, p.P)) p.refs_out[i] = max(outside, 0) + whole;
    }
    if (tid == 0) {
        if (store_ok(p.ctl, 0, 2, 2)) {
            p.info[0] = max(all_frees - all_wants, 0);
            p.info[1] = max(all_wants - all_frees, 0);
        }
    }
    cluster_sync();
    // a warp per slot: the partly kept page, the wanted ones, and nothing behind
    for (int b = warp; b < p.B; b += warps) {
        bool again = false;
        const Keeps k = keeps_of(p, b, again);
        const int have = __ldcg(p.s0 + b), first = __ldcg(p.s1 + b), state = __ldcg(p.s2 + b);
        int copied = -1;
        for (int j = k.full + lane; j < p.W; j += 32) {
            int page = -1;
            if (j < have) {
                page = state;
            } else if (j < k.want) {
                const int n = first + j - have;
                if (n < all_frees) page = __ldcg(p.w3 + n);
                if (j == k.full && state <= -2) copied = page;
            }
            if (page >= 0 && store_ok(p.ctl, page, 1, p.P)) p.refs_out[page] = 1;  // its only holder
            if (store_ok(p.ctl, b * p.ld_out + j, 1, (p.B - 1) * p.ld_out + p.W)) p.pages_out[b * p.ld_out + j] = page;
        }
        if (lane == 0 && store_ok(p.ctl, 2 * b, 2, 2ll * p.B)) {
            // (copied: lane 0 has j == full)
            p.copies[2 * b] = copied >= 0 ? -2 - state : -1;
            p.copies[2 * b + 1] = copied;
        }
    }
    if (bad) atomicOr(p.ctl.err, DEVERR_BAD_INDEX);
}

// w0: where a page in use goes (itself, or its new place), w1: the free pages below n
// in order, w2: the pages in use from n on in order.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    pages_compact_kernel(const __grid_constant__ pq2h::PagesParams p) {
    const int tid = blockIdx.x * kThreads + threadIdx.x, lane = threadIdx.x & 31;
    const int warp = tid >> 5, warps = kAll / 32;
    bool bad = false;
    pdl_wait();
    pdl_launch_dependents();
    const Part pages = part_of(p.P);
    int used = 0;
    for (int i = pages.lo; i < pages.hi; ++i) used += __ldcg(p.refs + i) > 0;
    int total, below;
    const int used0 = scan(used, total);
    if (threadIdx.x == 0) p.sums[blockIdx.x] = total;
    cluster_sync();
    const int offset = before(p.sums, total);  // total: pages in use
    // those in use below `total`: the rest of them move
    int low = 0;
    for (int i = pages.lo; i < min(pages.hi, total); ++i) low += __ldcg(p.refs + i) > 0;
    scan(low, below);
    if (threadIdx.x == 0) p.sums[kCtas + blockIdx.x] = below;
    cluster_sync();
    before(p.sums + kCtas, below);
    const int moves = total - below;
    int u = used0 + offset;  // pages in use before i
    for (int i = pages.lo; i < pages.hi; ++i) {
        const bool in_use = __ldcg(p.refs + i) > 0;
        if (in_use && i >= total) p.w2[u - below] = i;
        if (!in_use && i < total) p.w1[i - u] = i;
        if (!in_use || i < total) p.w0[i] = in_use ? i : -1;
        u += in_use;
    }
    cluster_sync();
    for (int i = tid; i < p.P / 2; i += kAll) {
        int from = -1, to = -1;
        if (i < moves) {
            from = __ldcg(p.w2 + i);
            to = __ldcg(p.w1 + i);
            p.w0[from] = to;
            p.w3[i] = __ldcg(p.refs + from);
        }
        if (store_ok(p.ctl, 2ll * i, 2, 2ll * (p.P / 2))) {
            p.copies[2ll * i] = from;
            p.copies[2ll * i + 1] = to;
        }
    }
    if (tid == 0 && store_ok(p.ctl, 0, 2, 2)) {
        p.info[0] = total;
        p.info[1] = moves;
    }
    cluster_sync();  // (refs has been read: refs_out may be refs from here on)
    for (int i = tid; i < p.P; i += kAll) {
        // (a hole's count is its page's, below)
        const int r = i < total ? __ldcg(p.refs + i) : 0;
        if ((i >= total || r > 0) && store_ok(p.ctl, i, 1, p.P)) p.refs_out[i] = r;
    }
    for (int i = tid; i < moves; i += kAll) {
        const int to = __ldcg(p.w1 + i);
        if (store_ok(p.ctl, to, 1, p.P)) p.refs_out[to] = __ldcg(p.w3 + i);
    }
    for (int b = warp; b < p.B; b += warps) {
        const int held = up(in_range(__ldcg(p.lens + b), p.W * p.T, bad), p.T);
        for (int j = lane; j < p.W; j += 32) {
            int page = -1;
            if (j < held) {
                page = page_at(p, b, j);
                // (-1 for a page that nobody counts: it has no new place)
                if (page >= 0) page = __ldcg(p.w0 + page);
                bad |= page < 0;
            }
            if (store_ok(p.ctl, b * p.ld_out + j, 1, (p.B - 1) * p.ld_out + p.W)) p.pages_out[b * p.ld_out + j] = page;
        }
    }
    if (bad) atomicOr(p.ctl.err, DEVERR_BAD_INDEX);
}

constexpr int kPiece = 8192;       // bytes of a page that a CTA copies at once
constexpr int kCopyThreads = 256;  // two 16-byte loads a thread in flight

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ pq2h::PagesCopyParams p) {
    const long long pieces = (p.page_bytes + kPiece - 1) / kPiece;
    const long long total = p.n * pieces * p.layers;
    pdl_wait();
    pdl_launch_dependents();
    for (long long i = blockIdx.x; i < total; i += gridDim.x) {
        // neighbouring CTAs take neighbouring pairs: those that say nothing are spread
        const long long piece = i / p.n, n = i - piece * p.n;
        const int2 pair = __ldcg(reinterpret_cast<const int2*>(p.pairs) + n);
        if (pair.x < 0 || pair.y < 0) continue;
        if (pair.x >= p.P || pair.y >= p.P) {
            if (threadIdx.x == 0) atomicOr(p.ctl.err, DEVERR_BAD_INDEX);
            continue;
        }
        const long long layer = piece / pieces, at = (piece - layer * pieces) * kPiece;
        const uint8_t* from = p.pool + layer * p.layer_stride + pair.x * p.page_stride + at;
        uint8_t* to = p.pool + layer * p.layer_stride + pair.y * p.page_stride + at;
        const int bytes = static_cast<int>(min(p.page_bytes - at, static_cast<long long>(kPiece)));
        uint4 v[kPiece / 16 / kCopyThreads];
#pragma unroll
        for (int k = 0; k < kPiece / 16 / kCopyThreads; ++k) {
            const int o = (k * kCopyThreads + threadIdx.x) * 16;
            if (o < bytes) v[k] = *reinterpret_cast<const uint4*>(from + o);
        }
#pragma unroll
        for (int k = 0; k < kPiece / 16 / kCopyThreads; ++k) {
            const int o = (k * kCopyThreads + threadIdx.x) * 16;
            if (o < bytes && store_ok(p.ctl, at + o, 16, p.page_bytes)) *reinterpret_cast<uint4*>(to + o) = v[k];
        }
    }
}

}  // namespace
}  // namespace pq2

namespace pq2h {

namespace {
size_t pad(size_t b) { return (b + 255) & ~size_t(255); }

void lay_out(PagesParams& p, void* workspace) {
    uint8_t* w = static_cast<uint8_t*>(workspace);
    const auto take = [&](size_t n) {
        int32_t* at = reinterpret_cast<int32_t*>(w);
        w += pad(n * 4);
        return at;
    };
    p.w0 = take(p.P), p.w1 = take(p.P), p.w2 = take(p.P), p.w3 = take(p.P);
    p.s0 = take(p.B), p.s1 = take(p.B), p.s2 = take(p.B);
    p.sums = take(2 * pq2::kCtas);
}
}  // namespace

size_t pages_workspace_bytes(int64_t B, int64_t P) {
    return 4 * pad(static_cast<size_t>(P) * 4) + 3 * pad(static_cast<size_t>(B) * 4) + pad(2 * pq2::kCtas * 4);
}

cudaError_t launch_pages_update(PagesParams p, void* workspace, cudaStream_t st) {
    lay_out(p, workspace);
    return launch(pq2::pages_update_kernel, dim3(pq2::kCtas), dim3(pq2::kThreads), 0, st, true, p);
}

cudaError_t launch_pages_compact(PagesParams p, void* workspace, cudaStream_t st) {
    lay_out(p, workspace);
    return launch(pq2::pages_compact_kernel, dim3(pq2::kCtas), dim3(pq2::kThreads), 0, st, true, p);
}

cudaError_t launch_pages_copy(const PagesCopyParams& p, cudaStream_t st, const DeviceInfo& dev) {
    const long long pieces = (p.page_bytes + pq2::kPiece - 1) / pq2::kPiece;
    const long long total = p.n * pieces * p.layers;
    const long long most = static_cast<long long>(dev.num_sms) * 8;
    return launch(pq2::pages_copy_kernel, dim3(static_cast<unsigned>(std::min(total, most))),
                  dim3(pq2::kCopyThreads), 0, st, true, p);
}

}  // namespace pq2h
