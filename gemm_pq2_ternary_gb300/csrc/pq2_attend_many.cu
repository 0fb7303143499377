// Attention over a cache held in 4 bits, many query rows for each key/value
// head (prompts, chunks of them), on tcgen05 with accumulators in tensor memory.
//
// With c' = code - 8, z' = offset + 8 scale:
//   q . k_j = s_j (q . c_j + r_j sum(q)),  r_j = offset_j / s_j
//   sum_j w_j v_j = sum_j (w_j s_j) c'_j + sum_j w_j z'_j
// Both products run on codes (exact in fp16; keys' as subnormals c 2^-24, as in
// pq2_attend.cu), the first with one more step of 16 for r_j sum(q).  What is left for the
// softmax is one factor per key for the scores (s_j with the softmax scale), and
// two for the weights (s_j of values, z'_j): keys and values enter as exactly
// as the cache holds them, only the weights are rounded (to fp16, as in
// pq2_attend.cu, maxima raised and values' scales kept in range in the same way).
//
// A CTA works on 256 rows (128 of 256 dims), two accumulators of 128 rows that take
// turns: the tensor cores multiply for one while the other's weights are computed.
// Rows are (token, head of the group) pairs, so that a group shares the expanded keys.
// 20 warps:
//   0-7    softmax: scores from tensor memory as 16x256b fragments (a lane has
//          a quarter of the keys of four rows: with a row a lane, every factor would be
//          loaded by every lane, and shared memory cannot give that), weights back to it as
//          the second product's first operand; at the end the outputs
//   8-11   expand codes of keys (K-major: 64 dims of 128 keys to 16 KB), and
//   12-15  of values (MN-major, as they are: a row of dims per key); both are rows of
//          128 bytes with the 128-byte swizzle, in two buffers each
//   16     issues the products
//   17-19  look up pages and compute the keys' factors, a tile of 128 keys each in turn
// Work is dealt out in tiles of 128 keys as in pq2_attend.cu; a CTA that has
// only a part of an item's keys writes a partial result, and attend_many_join_kernel joins them.
//
// Bound by what happens between the products: with the issuing and expanding warps' waits
// out of the way a tile takes 5500 cycles of 2100 that its products need (256 dims;
// 128 dims 6500 of 2200), most of it the softmax of its 128 (256) rows in 8 warps, some
// 4000 cycles for 1400 instructions a warp.  What held it up before: local memory (arrays
// indexed at run time, too few registers for a role), operands' descriptors in
// registers that had to be moved to uniform ones (100 cycles a product), waits one
// by one, an address read from shared memory before every load of codes, and items that
// counted for their tiles alone.  On GB300: 4096 tokens behind 4096, 24 heads of 256 on 4:
// 717 us, 863 TFLOP/s, for the first calls after a pause, and 757 us, 817 TFLOP/s, in a row of a hundred
// (in a graph as from the host; the SM clock reads its maximum throughout, at 900 W); chunks of 1000,
// 948 and 895 tokens, the last of 6000, 948 and 1895, 40 heads of 128 on 8: 304 us (mma.sync, 8
// rows at a time: 4528 and 1250 us).  That rows do not share their values' reference
// (pq2_attend.cuh) costs 9 of the 304, none of the 717.
#include <algorithm>
#include <cfloat>

#include "pq2_attend.cuh"

namespace pq2 {
namespace {

constexpr int kThreads = 640;
constexpr int kKeys = 128;                // keys of a tile
constexpr int kPer = kKeys / kTileTokens;
constexpr int kChunk = 16384;             // bytes
constexpr int kSlots = 4;                 // tiles whose factors are held
constexpr int kExtra = 6;                 // what an item's queries and outputs take, in tiles (2: 390 us for
                                          // chunks behind 6000 tokens, 3: 333, 4: 324, 6: 316)
constexpr float kEmpty = -FLT_MAX;
// (Larger and smaller than pq2_attend.cu's 5 and 512: a raise touches all outputs in
// tensor memory.  A prompt took 862, 776 and 731 us with 2, 5 and 8, chunks 356, 315 and 296.)
constexpr float kSlack = 8.0f;
constexpr float kWeight = 64.0f;
constexpr int kExpandWarps = 8;
constexpr int kFactorWarps = 3;
constexpr int kIssuer = 16;
constexpr int kSkipValues = 1 << 16;  // (timeout tests) from here on it is a piece of values that is withheld
constexpr int kRegsSoftmax = 128, kRegsExpand = 72, kRegsOther = 80;
constexpr int kRegsNeeded = 256 * kRegsSoftmax + 256 * kRegsExpand + 128 * kRegsOther;
static_assert(kRegsNeeded <= kThreads * 96, "the launch's registers");

// Factors of a tile's keys.  Key 8 n + 2 t + i stands at t * kQuarter + 2 n + i: a lane
// (g, t) reads its quarter in 16-byte pieces, the four quarters from different banks.
constexpr int kQuarter = 36;
struct Slot {
    uint8_t aug[kKeys * 16];      // the first product's last step: 8 of its 16 columns (the others are zeros)
    float scale[4 * kQuarter];    // of the scores
    float value[4 * kQuarter];    // values' scales
    float offset[4 * kQuarter];   // values' z'
    long long base[kPer];         // byte offset in the pool of the tiles of 16 keys, -1: none
    float ref;                    // power of two with values' scales below twice it
    int last, two;                // 1: the tile is its segment's last, 2: and the CTA's; more than 128 rows
    int key0;                     // the tile's first key where some row does not see all of it, else -1
    // of the tile's segment: rows of its tile of rows, the item, where its
    // outputs go (a partial result's place, -1: they are final)
    int rows, row_tile, head, n, row0, pos0, part, pad;
};
static_assert(sizeof(Slot) % 16 == 0, "");

struct Bars {
    uint64_t full[2][2], empty[2][2];  // of keys and of values, by buffer
    uint64_t slot_full[kSlots], slot_empty[kSlots];
    uint64_t q_full;
    uint64_t s_full[2], p_full[2][2], pv_done[2];  // p_full: of each warpgroup
    uint64_t out_full[2];  // all products of an accumulator's segment
    int abort_word;
    uint32_t tmem;
    float back[256];  // inverses of the powers of two that the rows of queries are multiplied by
};

template <int D>
struct Cfg {
    static constexpr int kParts = D / 64;                 // chunks of a tile's keys, and of its values
    static constexpr int kTiles = D == 256 ? 1 : 2;       // accumulators of 128 rows
    static constexpr int kHalves = D == 256 ? 2 : 1;      // pieces of a tile that are expanded at a time
    static constexpr int kRows = 128 * kTiles;
    static constexpr int kPartKeys = kKeys / kParts;      // keys of a chunk of values
    static constexpr size_t kQ = static_cast<size_t>(kTiles) * kParts * kChunk;
    static constexpr int kPieceParts = kParts / kHalves;  // chunks of a piece
    static constexpr size_t kPieceBytes = static_cast<size_t>(kPieceParts) * kChunk;  // of expanded keys, or values
    static constexpr size_t kKeysAt = kQ;
    static constexpr size_t kValuesAt = kKeysAt + 2 * kPieceBytes;
    static constexpr size_t kAugAt = kValuesAt + 2 * kPieceBytes;
    static constexpr size_t kSlotAt = kAugAt + static_cast<size_t>(kTiles) * 2048;
    static constexpr size_t kZeroAt = kSlotAt + kSlots * sizeof(Slot);   // the last steps' other columns
    static constexpr size_t kBarAt = kZeroAt + 2048;
    static constexpr size_t kSmem = kBarAt + sizeof(Bars) + 1024;  // (the base is rounded up)
};
static_assert(Cfg<128>::kSmem <= 232448 && Cfg<256>::kSmem <= 232448, "shared memory of a CTA");

// ---------------------------------------------------------------------------
// tcgen05
// ---------------------------------------------------------------------------
// Descriptors of operands in shared memory.  Their upper words are constants: the distance of
// groups of 8 rows and the swizzle.  The lower ones are the address and a distance.
constexpr uint32_t desc_hi(uint32_t stride, uint32_t swizzle) { return (stride >> 4) | (1u << 14) | (swizzle << 29); }
// rows of 128 bytes, swizzled, groups of 8 of them 1024 bytes apart; K-major,
// or MN-major with blocks of 64 values `leading` bytes apart
constexpr uint32_t kRowsHi = desc_hi(1024, 2);
// rows of 16 bytes, not swizzled, and as many zeros `leading` bytes behind them
constexpr uint32_t kAugHi = desc_hi(128, 0);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t leading) { return (saddr >> 4) | ((leading >> 4) << 16); }
// What all lanes have alike, told to the compiler: the products' operands then stay in
// uniform registers (moved there one by one they took 100 cycles a product).
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// fp16 operands, fp32 accumulators, 128 rows by N; MN: the second operand is MN-major
template <int N, bool MN>
constexpr uint32_t kInstr = (1u << 4) | (MN ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);

template <int N, bool MN, uint32_t HI>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(HI), "r"(kInstr<N, MN>), "r"(add));
}
template <int N, bool MN, uint32_t HI>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(HI), "r"(kInstr<N, MN>), "r"(add));
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Operand lists of the loads and stores below.
#define PQ2_R8(x, i) x(i), x(i + 1), x(i + 2), x(i + 3), x(i + 4), x(i + 5), x(i + 6), x(i + 7)
#define PQ2_R16(x, i) PQ2_R8(x, i), PQ2_R8(x, i + 8)
// 16 rows by 32 columns; lane (g, t): v[4 n], v[4 n + 1] row g, columns
// 8 n + 2 t and the next, v[4 n + 2], v[4 n + 3] row g + 8.  Load and wait are one
// statement: a copy of a register between the two would copy what was in it before.
#define PQ2_OUT(i) "=f"(v[i])
__device__ __forceinline__ void tc_load(uint32_t addr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : PQ2_R16(PQ2_OUT, 0)
        : "r"(addr)
        : "memory");
}
#undef PQ2_OUT
// 32 columns of both groups of 16 rows of a warp.
#define PQ2_OUT0(i) "=f"(v0[i])
#define PQ2_OUT1(i) "=f"(v1[i])
__device__ __forceinline__ void tc_load2(uint32_t addr0, uint32_t addr1, float (&v0)[16], float (&v1)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : PQ2_R16(PQ2_OUT0, 0), PQ2_R16(PQ2_OUT1, 0)
        : "r"(addr0), "r"(addr1)
        : "memory");
}
#undef PQ2_OUT0
#undef PQ2_OUT1
#define PQ2_IN(i) "r"(__float_as_uint(v[i]))
__device__ __forceinline__ void tc_store(uint32_t addr, const float (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
                 PQ2_R16(PQ2_IN, 0)
                 : "memory");
}
#undef PQ2_IN
// 16 rows by 16 columns of two fp16; lane (g, t): w[2 n] row g, column 4 n + t, w[2 n + 1] row g + 8.
#define PQ2_IN(i) "r"(w[i])
__device__ __forceinline__ void tc_store_weights(uint32_t addr, const uint32_t (&w)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), PQ2_R8(PQ2_IN, 0)
                 : "memory");
}
#undef PQ2_IN
#define PQ2_OUT(i) "=r"(w[i])
__device__ __forceinline__ void tc_load_weights(uint32_t addr, uint32_t (&w)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : PQ2_R8(PQ2_OUT, 0)
        : "r"(addr)
        : "memory");
}
#undef PQ2_OUT

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---------------------------------------------------------------------------
// What every role knows
// ---------------------------------------------------------------------------
// r (of a key) and sum(q) are two fp16 each, hi + lo; three of their products are
// summed: hi hi + (hi kAugLo) (lo / kAugLo) + (lo kAugHi2) (hi / kAugHi2).  With those powers of
// two no factor falls so far below fp16's normal numbers that the scores notice.
constexpr float kAugLo = 0x1p-6f, kAugHi2 = 0x1p3f;
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// All waits are by whole warps, none of whose lanes goes apart from the others
// (a branch for one lane and the shuffle after it take some 300 cycles), and
// short in code.  The issuing warp, without which nothing goes on, also watches
// the time: it stops the others.
constexpr uint32_t kPolls = 1u << 26;  // of any other wait: far behind that
struct Ctl {
    const pq2h::AttendParams& p;
    Bars& bars;
    volatile int* stop;

    // false: give up
    __device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) const {
        for (uint32_t i = 0; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++i)
            if (__any_sync(0xffffffffu, *stop || i == kPolls)) return false;
        return true;
    }
    // every lane (that `need`s to) its own barrier
    __device__ __forceinline__ bool timed_wait(uint64_t* bar, uint32_t parity, bool need) const {
        unsigned long long t0 = 0;
        for (uint32_t i = 0; !__all_sync(0xffffffffu, !need || mbar_try_wait(bar, parity)); ++i) {
            if (i % 64 != 63) continue;
            if (t0 == 0) t0 = globaltimer_ns();
            if (__any_sync(0xffffffffu, *stop || globaltimer_ns() - t0 > p.ctl.wait_limit_ns)) {
                if ((threadIdx.x & 31) == 0) atomicOr(p.ctl.err, DEVERR_TIMEOUT);
                *stop = 1;
                return false;
            }
        }
        return true;
    }
};

// A segment: `units` units of one item, in them `count` tiles of keys, from tile `tile` on.
struct Segment {
    AttendItem it;
    int tile, count, units;
    bool whole, starts;   // all of the item's tiles; its first ones
    long long end;        // the item's last unit and one
};

template <int D>
__device__ __forceinline__ Segment segment_at(const pq2h::AttendParams& p, AttendSpan& span, long long u) {
    const AttendStep s = attend_step<Cfg<D>::kRows>(p, kPer, kExtra, span, u);
    Segment g;
    g.it = attend_item<Cfg<D>::kRows>(p, s.b, s.row_tile, s.head);
    g.units = s.units;
    g.tile = g.it.tile0 / kPer + s.first;
    g.count = s.count;
    g.whole = s.count == s.of;
    g.starts = s.first == 0;
    g.end = s.end;
    return g;
}

// ---------------------------------------------------------------------------
// Warps 17-19: pages and factors
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void factors(const Ctl& k, const AttendWork& wk, AttendSpan span, Slot* slots,
                                        uint32_t w) {
    const pq2h::AttendParams& p = k.p;
    const int G = p.q_heads / p.cache.heads;
    const int lane = threadIdx.x & 31;
    const int per_page = p.cache.T / kTileTokens;
    uint32_t n = 0, next = w;  // tiles so far; this warp's next
    const float to_score = p.scale * 1.4426950408889634f * 0x1p24f;
    for (long long u = span.u0; u < span.u1;) {
        const Segment g = segment_at<D>(p, span, u);
        const int part = 2 * blockIdx.x + (u == span.u0 ? 0 : 1);
        if (g.count > 0 && n == next && g.starts && !g.whole && lane == 0)
            wk.join[blockIdx.x] = {g.it.b, g.it.row_tile, g.it.head,
                                   attend_cta_of(span, g.end - 1) - static_cast<int>(blockIdx.x) + 1, part};
        u += g.units;
        // (an item has at least one tile behind its kExtra units)
        const int last = span.u1 - u > kExtra ? 1 : 2;
        // keys that some row sees (what is before a window may have lost its page)
        const int key_lo = g.it.tile0 * kTileTokens, key_hi = min(g.it.tile1 * kTileTokens, g.it.pos0 + g.it.n);
        const long long head_at = static_cast<long long>(g.it.head) * per_page * tile_bytes(D);
        for (int j = 0; j < g.count; ++j, ++n) {
            if (n != next) continue;
            next += kFactorWarps;
            Slot& slot = slots[n % kSlots];
            long long base[4];
            uint32_t kp[4], vp[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = (g.tile + j) * kKeys + lane + 32 * i;
                base[i] = -1;
                kp[i] = vp[i] = 0;
                if (key < key_lo || key >= key_hi) continue;
                const int page = __ldg(p.cache.pages + g.it.b * p.cache.ld_pages + key / p.cache.T);
                if (page < 0 || page >= p.cache.num_pages) {
                    atomicOr(p.ctl.err, DEVERR_BAD_INDEX);
                    continue;
                }
                const int in = key % p.cache.T;
                const long long tile = page * p.cache.page_stride + head_at +
                                       static_cast<long long>(in / kTileTokens) * tile_bytes(D);
                base[i] = tile;
                const uint8_t* at = p.cache.pool + tile + (in % kTileTokens) * 4;
                kp[i] = __ldg(reinterpret_cast<const uint32_t*>(at + tile_pairs(D, 0)));
                vp[i] = __ldg(reinterpret_cast<const uint32_t*>(at + tile_pairs(D, 1)));
            }
            float top = 0x1p-24f;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, __half2float(__ushort_as_half(vp[i] & 0xffffu)));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (n >= kSlots && !k.warp_wait(&k.bars.slot_empty[n % kSlots], (n / kSlots - 1) & 1)) return;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = lane + 32 * i;
                const int at = ((key & 7) >> 1) * kQuarter + 2 * (key >> 3) + (key & 1);
                float s = __half2float(__ushort_as_half(kp[i] & 0xffffu));
                const float z = __half2float(__ushort_as_half(kp[i] >> 16));
                // (2^-10 r has to stay below fp16's largest: a scale below 2^-25 of
                // the offset counts as that)
                s = fmaxf(s, fmaxf(fabsf(z) * 0x1p-25f, 0x1p-24f));
                const float r = 0x1p-10f * z / s;
                const __half hi = __float2half_rn(r);
                const float hf = __half2float(hi);
                *reinterpret_cast<uint4*>(slot.aug + key * 16) =
                    make_uint4(half2_bits(hf, hf * kAugLo), half2_bits((r - hf) * kAugHi2, 0.0f), 0u, 0u);
                const float vs = __half2float(__ushort_as_half(vp[i] & 0xffffu));
                slot.scale[at] = s * to_score;
                slot.value[at] = vs;
                slot.offset[at] = fmaf(8.0f, vs, __half2float(__ushort_as_half(vp[i] >> 16)));
                if (lane % kTileTokens == 0) slot.base[key / kTileTokens] = base[i];
            }
            if (lane == 0) {
                slot.ref = scale_power(top);
                slot.last = j == g.count - 1 ? last : 0;
                slot.rows = static_cast<int>(min(static_cast<long long>(g.it.n) * G -
                                                     static_cast<long long>(g.it.row_tile) * Cfg<D>::kRows,
                                                 static_cast<long long>(Cfg<D>::kRows)));
                slot.two = Cfg<D>::kTiles == 2 && slot.rows > 128;
                slot.row_tile = g.it.row_tile;
                slot.head = g.it.head;
                slot.n = g.it.n;
                slot.row0 = g.it.row0;
                slot.pos0 = g.it.pos0;
                slot.part = g.whole ? -1 : part;
                const int key0 = (g.tile + j) * kKeys;
                slot.key0 = key0 < g.it.first_hi || key0 + kKeys - 1 > g.it.last_lo ? key0 : -1;
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&k.bars.slot_full[n % kSlots]);
        }
    }
}

// ---------------------------------------------------------------------------
// Warps 8-15: codes to operands
// ---------------------------------------------------------------------------
// Two codes less 8 of four bytes (HIGH: the high halves, times 16).
template <int HIGH>
__device__ __forceinline__ uint32_t centred(uint32_t w) {
    const uint32_t v = HIGH ? (w & 0x00f000f0u) | 0x64006400u : (w & 0x000f000fu) | 0x64006400u;
    const uint32_t c = HIGH ? 0x64806480u : 0x64086408u;
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&d);
}

// Two codes as fp16 subnormals, code 2^-24 (HIGH: times 16).
template <int HIGH>
__device__ __forceinline__ uint32_t plain(uint32_t w) {
    return HIGH ? w & 0x00f000f0u : w & 0x000f000fu;
}

// Four warps expand keys and four values, in pieces: whole tiles, or (256 dims, where there is
// no room for two) halves: of keys 128 dims, of values 64 keys.  A lane takes 16
// bytes (32 codes) at a time and stores four pieces of 16; of the eight lanes of a
// load's or a store's phase two have the same row and four have neighbouring ones.  So
// loads take whole sectors of 32 bytes, and stores, swizzled, meet every bank once
// without a different order for each lane.  The next codes are asked for as soon as
// these are used.
template <int D, bool VALUES>
__device__ __forceinline__ void expand(const Ctl& k, const Slot* slots, uint8_t* smem, int warp) {
    using C = Cfg<D>;
    constexpr int kDims = VALUES ? D : D / C::kHalves;              // of a row of a piece
    constexpr int kRows = (VALUES ? kKeys / C::kHalves : kKeys) / 4;  // of a piece for the warp
    constexpr int kRowsAtOnce = 1024 / kDims, kLoads = kRows / kRowsAtOnce;
    const int lane = threadIdx.x & 31, phase = lane >> 3;
    const int j = (lane & 1) + 2 * (kDims == 256 ? phase : kDims == 128 ? phase & 1 : 0);
    const int in16 = ((lane >> 1) & 3) + 4 * (kDims == 256 ? 0 : kDims == 128 ? phase >> 1 : phase);
    const int row0 = kRows * warp + in16;
    const int skip = k.p.ctl.debug_skip_stage - (VALUES ? kSkipValues : 0);
    // where the lane's rows are in a piece (its 64 dims are block j / 2), and its
    // 16 bytes in a row: with 4 rows at a time every other row has the other half's
    // (a warp's rows are in one chunk of values: kPartKeys is a multiple of them)
    const uint32_t row_at =
        VALUES ? (row0 / C::kPartKeys) * kChunk + (j >> 1) * (C::kPartKeys * 128) + (row0 % C::kPartKeys) * 128
               : (j >> 1) * kChunk + row0 * 128;
    const uint32_t at = (((j & 1) * 4) ^ (row0 & 7)) << 4;
    // piece e: half e % kHalves of tile e / kHalves; the warp's rows lie in kGroups tiles
    // of 16 (what is behind the last token is read too: any codes will do)
    constexpr int kGroups = kRows / kTileTokens;
    const uint8_t* pool = k.p.cache.pool + (VALUES ? tile_codes(D, 1) : 0) + 16 * j + in16 * (D / 2);
    uint4 raw[kLoads];
    long long base[kGroups];
    bool ends = false;  // whether the piece is the CTA's last
    const auto places = [&](uint32_t e) {
        const uint32_t half = e % C::kHalves;
        const int group = kGroups * warp + (VALUES ? half * (4 * kGroups) : 0);
#pragma unroll
        for (int x = 0; x < kGroups; ++x) {
            base[x] = slots[e / C::kHalves % kSlots].base[group + x];
            if (!VALUES && C::kHalves == 2 && base[x] >= 0) base[x] += half * (kDims / 2);
        }
        ends = half == C::kHalves - 1 && slots[e / C::kHalves % kSlots].last == 2;
    };
    const auto load = [&](int i) {
        const long long from = base[kRowsAtOnce * i / kTileTokens];
        raw[i] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);  // codes 8
        if (from >= 0) raw[i] = __ldg(reinterpret_cast<const uint4*>(pool + from + kRowsAtOnce * i % kTileTokens * (D / 2)));
    };
    // once a piece's codes have been asked for
    const auto give_back = [&](uint32_t e) {
        if (e % C::kHalves != C::kHalves - 1) return;
        __syncwarp();
        if (lane == 0) mbar_arrive(&k.bars.slot_empty[e / C::kHalves % kSlots]);
    };
    if (!k.warp_wait(&k.bars.slot_full[0], 0)) return;
    places(0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load(i);
    give_back(0);
#pragma unroll 1
    for (uint32_t e = 0;; ++e) {
        const uint32_t buf = e & 1, next = (e + 1) / C::kHalves;  // (the next piece's tile)
        const bool more = !ends;
        // a lane looks whether the next tile's factors are there (they may have to wait for this
        // tile's products), the others wait for the buffer
        const bool early = more && __all_sync(0xffffffffu, mbar_test_wait(&k.bars.slot_full[next % kSlots], (next / kSlots) & 1));
        if (early) places(e + 1);
        if (e >= 2 && !k.warp_wait(&k.bars.empty[VALUES][buf], (e / 2 - 1) & 1)) return;
        uint8_t* to = smem + (VALUES ? C::kValuesAt : C::kKeysAt) + buf * C::kPieceBytes + row_at;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            uint8_t* row = to + kRowsAtOnce * i * 128;
            const uint32_t half = (kRowsAtOnce * i & 4) << 4;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t w8 = w[x] >> 8;
                *reinterpret_cast<uint4*>(row + (at ^ half ^ (x << 4))) =
                    VALUES ? make_uint4(centred<0>(w[x]), centred<1>(w[x]), centred<0>(w8), centred<1>(w8))
                           : make_uint4(plain<0>(w[x]), plain<1>(w[x]), plain<0>(w8), plain<1>(w8));
            }
            if (early) load(i);
        }
        fence_async();
        __syncwarp();
        if (lane == 0 && static_cast<int>(e) != skip) mbar_arrive(&k.bars.full[VALUES][buf]);
        if (!more) return;
        if (!early) {
            if (!k.warp_wait(&k.bars.slot_full[next % kSlots], (next / kSlots) & 1)) return;
            places(e + 1);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) load(i);
        }
        give_back(e + 1);
    }
}

// ---------------------------------------------------------------------------
// Warp 16: the products (one thread)
// ---------------------------------------------------------------------------
// A wait of a barrier that is ready takes some 300 cycles while the expanding warps keep
// shared memory busy, and the tensor cores run dry meanwhile: all that a step
// needs is waited for at once, a barrier a lane.
template <int D>
struct Issue {
    using C = Cfg<D>;
    const Ctl& k;
    const Slot* slots;
    uint32_t smem;
    uint32_t weights;  // parity of the weights' next phase, bit 2 * warpgroup + buffer

    // Waits for what is asked for: keys of tile m, values of tile n, weights of
    // the warpgroups in `from` in buffer buf, the queries of segment seg.
    __device__ __forceinline__ bool wait(bool keys, uint32_t m, bool values, uint32_t n, uint32_t from, uint32_t buf,
                                         bool queries, uint32_t seg) {
        const uint32_t lane = threadIdx.x & 31, i = lane & 1;
        const uint32_t e = (lane < 2 ? m : n) * C::kHalves + i;  // a piece of keys (lanes 0, 1) or values (2, 3)
        uint64_t* bar = &k.bars.full[lane >> 1 & 1][e & 1];
        uint32_t parity = e >> 1 & 1;
        bool need = lane < 2 ? keys && i < C::kHalves : lane < 4 && values && i < C::kHalves;
        if (lane == 4 || lane == 5) {
            bar = &k.bars.p_full[i][buf];
            parity = weights >> (2 * i + buf) & 1;
            need = from >> i & 1;
        }
        if (lane == 6) bar = &k.bars.q_full, parity = seg & 1, need = queries;
        weights ^= (from & 1) << buf | (from >> 1) << (2 + buf);
        if (!k.timed_wait(bar, parity, need)) return false;
        tc_after();
        return true;
    }
    // Scores of accumulator t with tile n's keys; `last`: the last use of these.
    __device__ __forceinline__ void keys(int t, uint32_t n, uint32_t buf, bool last) {
        const uint32_t zeros = smem + static_cast<uint32_t>(C::kZeroAt);
        const uint32_t aug_q = smem + static_cast<uint32_t>(C::kAugAt) + t * 2048;
        const uint32_t aug_k = smem + static_cast<uint32_t>(C::kSlotAt + (n % kSlots) * sizeof(Slot));
        // (halves: of every tile the first is in the first buffer)
        const uint32_t in = C::kHalves == 2 ? 0 : n & 1;
        const uint32_t d = uniform(256 + buf * 128);
        const uint32_t a = uniform(desc_lo(smem + t * C::kParts * kChunk, 16));
        const uint32_t b = uniform(desc_lo(smem + static_cast<uint32_t>(C::kKeysAt + in * C::kPieceBytes), 16));
        const uint32_t qa = uniform(desc_lo(aug_q, zeros - aug_q)), ka = uniform(desc_lo(aug_k, zeros - aug_k));
        if (elect_one()) {
#pragma unroll
            for (int i = 0; i < C::kParts; ++i) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    mma_ss<128, false, kRowsHi>(d, a + (i * kChunk / 16 + 2 * x), b + (i * kChunk / 16 + 2 * x),
                                                i > 0 || x > 0 ? 1u : 0u);
                if (C::kHalves == 2 && i == C::kPieceParts - 1 && last) tc_commit(&k.bars.empty[0][0]);
            }
            mma_ss<128, false, kAugHi>(d, qa, ka, 1);
            if (last) tc_commit(&k.bars.empty[0][C::kHalves == 2 ? 1 : in]);
            tc_commit(&k.bars.s_full[buf]);
        }
    }
    // Outputs of accumulator t with tile n's values and the weights in buffer buf.
    __device__ __forceinline__ void values(int t, uint32_t n, uint32_t buf, bool first, bool last, bool ends) {
        const uint32_t in = C::kHalves == 2 ? 0 : n & 1;
        const uint32_t d = uniform(t * D), a = uniform(256 + buf * 128), add = uniform(first ? 0u : 1u);
        const uint32_t b = uniform(desc_lo(smem + static_cast<uint32_t>(C::kValuesAt + in * C::kPieceBytes), C::kPartKeys * 128));
        if (elect_one()) {
#pragma unroll
            for (int i = 0; i < C::kParts; ++i) {
#pragma unroll
                for (int x = 0; x < C::kPartKeys / 16; ++x)
                    mma_ts<D, true, kRowsHi>(d, a + (i * C::kPartKeys + 16 * x) / 2, b + (i * kChunk / 16 + 128 * x),
                                             i > 0 || x > 0 ? 1u : add);
                if (C::kHalves == 2 && i == C::kPieceParts - 1 && last) tc_commit(&k.bars.empty[1][0]);
            }
            if (last) tc_commit(&k.bars.empty[1][C::kHalves == 2 ? 1 : in]);
            tc_commit(&k.bars.pv_done[t]);
            if (ends) tc_commit(&k.bars.out_full[t]);
        }
    }
    __device__ __forceinline__ void run() {
        uint32_t seg = 0, n = 0;
#pragma unroll 1
        for (int last = 0; last != 2; ++seg) {
            // a segment: from tile n to the one that says it is the last
            if (!k.timed_wait(&k.bars.slot_full[n % kSlots], (n / kSlots) & 1, true)) return;
            const int acc = C::kTiles == 2 && slots[n % kSlots].two ? 2 : 1;
            const bool alone = acc == 1;
            bool first = true;
            int next_last = 0;
            last = slots[n % kSlots].last;
            // one pass more than tiles: scores of tile m = n + 1 behind outputs of tile n
            // (before them with one accumulator, which has both buffers of scores)
            bool primed = false;
#pragma unroll 1
            for (;;) {
                const bool more = !primed || !last;
                const uint32_t m = primed ? n + 1 : n;
#pragma unroll 1
                for (int o = 0; o < 2 * acc; ++o) {
                    const int t = alone ? 0 : o >> 1;
                    const bool is_keys = alone ? o == 0 : o & 1;
                    const uint32_t buf = alone ? (is_keys ? m : n) & 1 : t;
                    // alone: a wait for each product (a warpgroup has written half of the
                    // weights); else one for both
                    const bool k_here = more && (alone ? is_keys : o == 0), v_here = primed && (alone ? !is_keys : o == 0);
                    const uint32_t from = !primed || is_keys ? 0 : alone ? 3 : 1u << t;
                    if (k_here || from != 0) {
                        if (!wait(k_here, m, v_here, n, from, buf, k_here && !primed, seg)) return;
                        // (the last tile's slot may be another's by the time of its values)
                        if (k_here && primed) next_last = slots[m % kSlots].last;
                    }
                    if (is_keys) {
                        if (more) keys(t, m, buf, t == acc - 1);
                    } else if (primed) {
                        values(t, n, buf, first, t == acc - 1, last);
                    }
                }
                if (primed) {
                    first = false;
                    ++n;
                    if (last) break;
                    last = next_last;
                }
                primed = true;
            }
        }
    }
};

// ---------------------------------------------------------------------------
// Warps 0-7
// ---------------------------------------------------------------------------
__device__ __forceinline__ float4 lds4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// What a softmax warp counts over all segments.
struct Counts {
    uint32_t n;          // tiles
    bool ends;           // the CTA's last is among them
    uint32_t phases;     // parities of the next phases: of products of keys by buffer (bits 0, 1),
                         // of the last of values by accumulator (2, 3), of segments (4, 5)
};

// A segment's rows and outputs, as in the slots of its tiles.
struct Rows {
    int rows, row_tile, head, n, row0, pos0, part;
};

// Where the 16-byte piece `col` of a row of queries is.
template <int D>
__device__ __forceinline__ uint32_t q_place(int row, int col) {
    return ((row >> 7) * Cfg<D>::kParts + (col >> 3)) * kChunk + (row & 127) * 128 + (((col & 7) ^ (row & 7)) << 4);
}
// First of the rows that a softmax warp loads the queries of.
template <int D>
__device__ __forceinline__ int own_row(int warp) {
    return D == 256 ? (warp & 3) * 32 + 16 * (warp >> 2) : 32 * warp;
}

// The tiles of a segment and its outputs, for a warp with NS groups of 16 rows.
// Two accumulators: a warpgroup each, a warp all 32 rows of its part of the
// lanes.  One: both warpgroups, a warp 16 of them.
template <int D, int NS>
__device__ __forceinline__ bool rows_of_segment(const Ctl& k, const AttendWork& wk, const Rows& s, uint8_t* smem,
                                                uint32_t tmem, Counts& count) {
    using C = Cfg<D>;
    constexpr int kR = 2 * NS;  // rows of a lane
    const pq2h::AttendParams& p = k.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3, wg = warp >> 2;
    const int tile = NS == 2 ? wg : 0;
    // first row of the warp's (of its accumulator), and its tensor memory lanes
    const int row0 = (warp & 3) * 32 + (NS == 2 ? 0 : 16 * wg);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(row0) << 16);
    const Slot* slots = reinterpret_cast<const Slot*>(smem + C::kSlotAt);
    const int G = p.q_heads / p.cache.heads;
    const bool there = tile * 128 + row0 < s.rows;  // the warp has rows
    const bool whole = s.part < 0;
    float m[kR], ref = 0x1p-24f, back[kR];
    float slack = kSlack;  // (less the largest b)
    uint32_t bs = 0;
    float l[kR], z[kR];
    int last[kR];
    const int back_to = p.window > 0 ? p.window - 1 : s.pos0 + s.n;  // positions that a row sees before its own
#pragma unroll
    for (int r = 0; r < kR; ++r) {
        m[r] = kEmpty;
        l[r] = z[r] = 0.0f;
        const int row = tile * 128 + row0 + (r >> 1) * 16 + (r & 1) * 8 + g;
        last[r] = s.pos0 + min((s.row_tile * C::kRows + row) / G, s.n - 1);
        back[r] = k.bars.back[row];
    }
    bool more_tiles = true;
#pragma unroll 1
    for (int j = 0; more_tiles; ++j, ++count.n) {
        const int buf = NS == 2 ? tile : count.n & 1;
        const Slot& slot = slots[count.n % kSlots];
        if (!k.warp_wait(&k.bars.slot_full[count.n % kSlots], (count.n / kSlots) & 1)) return false;
        if (!k.warp_wait(&k.bars.s_full[buf], (count.phases >> buf) & 1)) return false;
        count.phases ^= NS == 2 ? 3u : 1u << buf;
        tc_after();
        more_tiles = slot.last == 0;
        count.ends = slot.last == 2;
        if (there) {
            const int key0 = slot.key0;  // (-1: all rows see the whole tile)
            const uint32_t at_s = lanes + 256 + buf * 128;
            // 32 keys at a time, in a loop: with a tile's code unrolled, the roles'
            // instructions do not fit the instruction caches (64 at a time with one
            // group of rows: 750 us for a prompt, not 701)
            constexpr int kStep = 32, kGroups = kStep / 8;
#pragma unroll 1
            for (int q = 0; q < kKeys; q += kStep) {
                float x[NS][kStep / 2];
                if constexpr (NS == 2)
                    tc_load2(at_s + q, at_s + (16u << 16) + q, x[0], x[NS - 1]);
                else
                    tc_load(at_s + q, x[0]);
                const int at_f = t * kQuarter + q / 4;
                // (plain fp32 operations: pairs of them in one instruction cost more
                // in moves than they save)
#pragma unroll
                for (int c = 0; c < kGroups; c += 2) {
                    const float4 f4 = lds4(slot.scale + at_f + 2 * c);
                    const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                    for (int i = 0; i < NS; ++i)
#pragma unroll
                        for (int h = 0; h < 8; ++h) x[i][4 * c + h] *= f[2 * (h >> 2) + (h & 1)];
                }
                if (__builtin_expect(key0 >= 0, 0)) {
                    const int key1 = key0 + q + 2 * t;
#pragma unroll
                    for (int c = 0; c < kGroups; ++c)
#pragma unroll
                        for (int i = 0; i < NS; ++i)
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                const int key = key1 + 8 * c + (h & 1), r = 2 * i + (h >> 1);
                                if (key < last[r] - back_to || key > last[r]) x[i][4 * c + h] = __uint_as_float(0xff800000u);
                            }
                }
                float top[kR];
                bool more = slot.ref > ref;
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const float* v = x[r >> 1] + 2 * (r & 1);
                    top[r] = fmaxf(v[0], v[1]);
#pragma unroll
                    for (int c = 1; c < kGroups; ++c) top[r] = fmaxf(fmaxf(top[r], v[4 * c]), v[4 * c + 1]);
                    top[r] *= back[r];
                    more |= top[r] > m[r] + slack;
                }
                if (__builtin_expect(__any_sync(0xffffffffu, more), 0)) {
                    // raise the values' reference, and maxima where a row needs it, to whole
                    // numbers (what was rounded is scaled exactly; from 2^23 on every fp32 number is
                    // one, and the maximum is the score): sums and outputs are scaled down
                    // (a row's lanes are four neighbours)
                    float alpha[kR], to_ref = fmaxf(ref, slot.ref);
#pragma unroll
                    for (int r = 0; r < kR; ++r) {
                        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
                    }
                    if (__all_sync(0xffffffffu, key0 < 0 && bs == 0)) {  // all rows see the same
#pragma unroll
                        for (int r = 0; r < kR; ++r) {
                            const float to = top[r] > m[r] + kSlack ? ceilf(top[r]) : m[r];
                            alpha[r] = power_of_two(m[r] - to);
                            m[r] = to;
                        }
                    } else {
                        float own[kR];  // the largest scale of the values that the row sees
#pragma unroll
                        for (int r = 0; r < kR; ++r) own[r] = 0.0f;
#pragma unroll 1
                        for (int c = 0; c < kStep / 4; ++c) {
                            const int key = key0 + q + 2 * t + 8 * (c >> 1) + (c & 1);
                            const float v = slot.value[at_f + c];
#pragma unroll
                            for (int r = 0; r < kR; ++r)
                                if (key0 < 0 || (key >= last[r] - back_to && key <= last[r])) own[r] = fmaxf(own[r], v);
                        }
                        float max[kR];
                        Apart apart;
#pragma unroll
                        for (int r = 0; r < kR; ++r) {
                            own[r] = fmaxf(own[r], __shfl_xor_sync(0xffffffffu, own[r], 1));
                            own[r] = scale_power(fmaxf(own[r], __shfl_xor_sync(0xffffffffu, own[r], 2)));
                            const float b = static_cast<float>(row_b(bs, r));
                            max[r] = m[r] == kEmpty ? kEmpty : m[r] - b;
                            if (m[r] != kEmpty) own[r] = fmaxf(own[r], ref * power_of_two(b));
                            max[r] = top[r] > max[r] + kSlack ? ceilf(top[r]) : max[r];
                            apart.row(max[r], own[r], kEmpty);
                        }
                        to_ref = apart.reference(ref);
                        bs = 0;
                        float most = 0.0f;
#pragma unroll
                        for (int r = 0; r < kR; ++r) {
                            const int b = max[r] == kEmpty ? 0 : ::max(power_between(to_ref, own[r]), 0);
                            bs |= static_cast<uint32_t>(b) << (8 * r);
                            max[r] += static_cast<float>(b);
                            most = fmaxf(most, static_cast<float>(b));
                            alpha[r] = m[r] == kEmpty ? 0.0f : power_of_two(m[r] - max[r]);
                            m[r] = max[r];
                        }
                        slack = kSlack - warp_max(most);
                    }
                    const float down = ref / to_ref;
                    ref = to_ref;
#pragma unroll
                    for (int r = 0; r < kR; ++r) {
                        l[r] *= alpha[r];
                        z[r] *= alpha[r];
                        alpha[r] *= down;
                    }
                    // the tile's weights so far
                    tc_wait_st();
#pragma unroll 1
                    for (int before = 0; before < q; before += 32) {
#pragma unroll
                        for (int i = 0; i < NS; ++i) {
                            const uint32_t at = at_s + (static_cast<uint32_t>(16 * i) << 16) + before / 2;
                            uint32_t w[8];
                            tc_load_weights(at, w);
#pragma unroll
                            for (int y = 0; y < 8; ++y) {
                                const __half2 v2 = __hmul2(*reinterpret_cast<const __half2*>(&w[y]),
                                                           __float2half2_rn(alpha[2 * i + (y & 1)]));
                                w[y] = *reinterpret_cast<const uint32_t*>(&v2);
                            }
                            tc_store_weights(at, w);
                        }
                    }
                    if (j > 0) {
                        if (!k.warp_wait(&k.bars.pv_done[tile], ((count.phases >> (2 + tile)) & 1) ^ 1)) return false;
                        tc_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32)
#pragma unroll
                            for (int i = 0; i < NS; ++i) {
                                const uint32_t at = lanes + (static_cast<uint32_t>(16 * i) << 16) + tile * D + c;
                                float o[16];
                                tc_load(at, o);
#pragma unroll
                                for (int y = 0; y < 16; ++y) o[y] *= alpha[2 * i + ((y >> 1) & 1)];
                                tc_store(at, o);
                            }
                        tc_wait_st();
                    }
                }
                const float vf = kWeight / ref;
                uint32_t w[NS][kStep / 4];
#pragma unroll
                for (int c = 0; c < kGroups; c += 2) {
                    const float4 f4 = lds4(slot.value + at_f + 2 * c);
                    const float4 z4 = lds4(slot.offset + at_f + 2 * c);
                    const float f[4] = {f4.x * vf, f4.y * vf, f4.z * vf, f4.w * vf};
                    const float zs[4] = {z4.x, z4.y, z4.z, z4.w};
#pragma unroll
                    for (int i = 0; i < NS; ++i)
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const int at = 4 * c + 2 * h, r = 2 * i + (h & 1), key = 2 * (h >> 1);
                            const float w0 = ex2(fmaf(x[i][at], back[r], -m[r])), w1 = ex2(fmaf(x[i][at + 1], back[r], -m[r]));
                            l[r] += w0 + w1;
                            z[r] = fmaf(w1, zs[key + 1], fmaf(w0, zs[key], z[r]));
                            w[i][2 * c + h] = half2_bits(w0 * f[key], w1 * f[key + 1]);
                        }
                }
                // (over scores that have been read)
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    tc_store_weights(at_s + (static_cast<uint32_t>(16 * i) << 16) + q / 2, w[i]);
            }
            tc_wait_st();
        }
        count.phases ^= NS == 2 ? 12u : 4u;
        tc_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&k.bars.p_full[wg][buf]);
            mbar_arrive(&k.bars.slot_empty[count.n % kSlots]);
        }
    }
    // --- the outputs -----------------------------------------------------
    // (pv_done's last phase could be mistaken for the one but last: with one
    // accumulator either may be done)
    if (!k.warp_wait(&k.bars.out_full[tile], (count.phases >> (4 + tile)) & 1)) return false;
    count.phases ^= NS == 2 ? 48u : 16u;
    tc_after();
    if (!there) return true;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
            z[r] += __shfl_xor_sync(0xffffffffu, z[r], o);
        }
    }
    // a lane's columns 8 c + 2 t and the next are dims 8 c + t and 8 c + t + 4
    const float f = ref / kWeight * (t & 1 ? 0.0625f : 1.0f);
    // staged in the warp's rows of queries, which all products are done with
    const int stage0 = own_row<D>(warp);
    const int type = p.bf16 ? PQ2_BF16 : PQ2_F16;
    // output = a o + b; a row that has seen nothing gives zeros
    float a[kR], b[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
        l[r] = l[r] > 0.0f ? l[r] : 0.0f;
        const float inv = l[r] == 0.0f ? 0.0f : whole ? 1.0f / l[r] : 1.0f;
        a[r] = f * inv;
        b[r] = l[r] == 0.0f ? 0.0f : z[r] * inv;
        if (l[r] == 0.0f) a[r] = 0.0f;
    }
    // of neighbouring lanes the even one takes both dims 8 c + t, the odd one both 8 c + 4 + t
    const int dt = (t >> 1) * 2 + (t & 1) * 4;
    const long long part0 = (static_cast<long long>(s.part) * wk.rows + tile * 128 + row0 + g) * D + dt;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            float o[16];
            tc_load(lanes + (static_cast<uint32_t>(16 * i) << 16) + tile * D + c0, o);
#pragma unroll
            for (int y = 0; y < 16; y += 2) {
                const int h = (y >> 1) & 1, r = 2 * i + h, in = 16 * i + 8 * h + g;
                const float v0 = fmaf(o[y], a[r], b[r]), v1 = fmaf(o[y + 1], a[r], b[r]);
                const float other = __shfl_xor_sync(0xffffffffu, t & 1 ? v0 : v1, 1);
                o[y] = t & 1 ? other : v0;
                o[y + 1] = t & 1 ? v1 : other;
                if (whole)
                    *reinterpret_cast<uint32_t*>(smem + q_place<D>(stage0 + in, (c0 >> 3) + (y >> 2)) + dt * 2) =
                        f32x2_to_elem16(o[y], o[y + 1], type);
            }
            if (whole) continue;
#pragma unroll
            for (int y = 0; y < 16; y += 2) {
                const int in = 16 * i + 8 * ((y >> 1) & 1);
                const long long at = part0 + static_cast<long long>(in) * D + c0 + 8 * (y >> 2);
                if (tile * 128 + row0 + in + g < s.rows && store_ok(p.ctl, at, 2, wk.o_elems))
                    *reinterpret_cast<float2*>(wk.o + at) = make_float2(o[y], o[y + 1]);
            }
        }
    }
    if (!whole) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const int row = tile * 128 + row0 + (r >> 1) * 16 + (r & 1) * 8 + g;
            const long long at = static_cast<long long>(s.part) * wk.rows + row;
            if (t == 0 && row < s.rows && store_ok(p.ctl, at, 1, wk.ml_elems)) wk.ml[at] = make_float2(m[r], l[r]);
        }
        return true;
    }
    __syncwarp();
    constexpr int kPer16 = D / 8;
#pragma unroll 1
    for (int piece = lane; piece < 16 * NS * kPer16; piece += 32) {
        const int in = piece / kPer16, col = piece % kPer16, row = tile * 128 + row0 + in;
        if (row >= s.rows) continue;
        const int r = s.row_tile * C::kRows + row;
        const long long at = static_cast<long long>(s.row0 + r / G) * p.ld_out +
                             static_cast<long long>(s.head * G + r % G) * p.hs_out + col * 8;
        if (store_ok(p.ctl, at, 8, p.out_elems))
            *reinterpret_cast<uint4*>(p.out + at) = *reinterpret_cast<const uint4*>(smem + q_place<D>(stage0 + in, col));
    }
    __syncwarp();
    return true;
}

template <int D>
__device__ __forceinline__ void softmax(const Ctl& k, const AttendWork& wk, uint8_t* smem, uint32_t tmem) {
    using C = Cfg<D>;
    const pq2h::AttendParams& p = k.p;
    const int tid = threadIdx.x, lane = tid & 31;
    const int G = p.q_heads / p.cache.heads;
    const Slot* slots = reinterpret_cast<const Slot*>(smem + C::kSlotAt);
    uint32_t seg = 0;
    Counts count = {0, false, 0};
#pragma unroll 1
    for (; !count.ends; ++seg) {
        if (!k.warp_wait(&k.bars.slot_full[count.n % kSlots], (count.n / kSlots) & 1)) return;
        const Slot& its = slots[count.n % kSlots];
        const Rows s = {its.rows, its.row_tile, its.head, its.n, its.row0, its.pos0, its.part};
        const bool two = its.two;
        // --- the queries ---------------------------------------------------
        {
            // pieces of 8 values: as they are to their places, then the operands, every row
            // with a power of two of its own, so that it does not depend on the rows beside it
            // (one for all rows was no faster: a prompt 715 us, not 714).  (Kept in
            // registers between the two, their code would be 16 times as long, and code
            // that is run once a segment comes from L2.)
            constexpr int kPieces = C::kRows * (D / 8) / 256;  // a thread
            constexpr int kStride = 32 / (D / 8);              // rows between a thread's pieces
            constexpr int kBatch = 8;
            // A warp's rows are those that it stages its outputs in: it need not wait
            // for the others' outputs.
            const int col = lane % (D / 8), row0 = own_row<D>(tid >> 5) + lane / (D / 8);
            const auto place = [&](int i) -> uint4* {
                return reinterpret_cast<uint4*>(smem + q_place<D>(row0 + i * kStride, col));
            };
            const auto value = [&](uint32_t a, float& lo, float& hi) {
                if (p.bf16) {
                    lo = __uint_as_float(a << 16);
                    hi = __uint_as_float(a & 0xffff0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a));
                    lo = f.x;
                    hi = f.y;
                }
            };
            const auto values = [&](const uint4& q, float (&v)[8]) {
                value(q.x, v[0], v[1]), value(q.y, v[2], v[3]), value(q.z, v[4], v[5]), value(q.w, v[6], v[7]);
            };
            const int r0 = s.row_tile * C::kRows + row0;
            int token = r0 / G, head = r0 - token * G;
            const int tokens = kStride / G, heads = kStride - tokens * G;
            const uint16_t* from = p.q + static_cast<long long>(s.head * G) * p.hs_q + col * 8;
#pragma unroll 1
            for (int i0 = 0; i0 < kPieces; i0 += kBatch) {
                uint4 raw[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    raw[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (row0 + (i0 + i) * kStride < s.rows)
                        raw[i] = __ldg(reinterpret_cast<const uint4*>(from + static_cast<long long>(s.row0 + token) * p.ld_q +
                                                                      static_cast<long long>(head) * p.hs_q));
                    token += tokens, head += heads;
                    if (head >= G) head -= G, ++token;
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) *place(i0 + i) = raw[i];
            }
#pragma unroll 2
            for (int i = 0; i < kPieces; ++i) {
                const int row = row0 + i * kStride;
                float v[8], sum = 0.0f, top = 0.0f;
                values(*place(i), v);
#pragma unroll
                for (int x = 0; x < 8; ++x) top = fmaxf(top, fabsf(v[x]));
#pragma unroll
                for (int o = D / 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                // every row times a power of two of its own, its largest value in [2^14, 2^15): half
                // a step of a sixteenth below fp16's smallest normal number is 2^-35 of it
                const int e = top > 0.0f ? 141 - static_cast<int>(__float_as_uint(fmaxf(top, 0x1p-100f)) >> 23) : 0;
                const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                uint32_t h[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    // order of the expanded codes: 0 4 | 1 5 (over 16) | 2 6 | 3 7 (over 16)
                    const float f = x & 1 ? up * 0.0625f : up;
                    const __half2 b = __floats2half2_rn(v[x] * f, v[x + 4] * f);
                    h[x] = *reinterpret_cast<const uint32_t*>(&b);
                    const float2 c = __half22float2(b);
                    sum += (c.x + c.y) * (x & 1 ? 16.0f : 1.0f);
                }
                const int at = row >> 7, r = row & 127;
                *place(i) = make_uint4(h[0], h[1], h[2], h[3]);
#pragma unroll
                for (int o = D / 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (col == 0) {
                    k.bars.back[row] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                    sum *= 0x1p-14f;
                    const float hi = __half2float(__float2half_rn(sum));
                    *reinterpret_cast<uint4*>(smem + C::kAugAt + at * 2048 + r * 16) =
                        make_uint4(half2_bits(hi, (sum - hi) / kAugLo), half2_bits(hi / kAugHi2, 0.0f), 0u, 0u);
                }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&k.bars.q_full);
            // (a warp's rows of scores may be others' of queries)
            if (!k.warp_wait(&k.bars.q_full, seg & 1)) return;
        }
        // --- the tiles and the outputs ---------------------------------------
        if constexpr (C::kTiles == 2) {
            if (two) {
                if (!rows_of_segment<D, 2>(k, wk, s, smem, tmem, count)) return;
                continue;
            }
        }
        if (!rows_of_segment<D, 1>(k, wk, s, smem, tmem, count)) return;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attend_many_kernel(const __grid_constant__ pq2h::AttendParams p, const __grid_constant__ AttendWork wk) {
    using C = Cfg<D>;
    extern __shared__ uint8_t dynamic_smem[];
    const int tid = threadIdx.x, warp = tid >> 5;
    uint8_t* smem = dynamic_smem + ((1024u - (smem_u32(dynamic_smem) & 1023u)) & 1023u);
    Bars& bars = *reinterpret_cast<Bars*>(smem + C::kBarAt);
    Slot* slots = reinterpret_cast<Slot*>(smem + C::kSlotAt);
    pdl_wait();
    pdl_launch_dependents();
    AttendSpan span;
    // (at least one tile behind an item's kExtra units)
    attend_span<C::kRows, kThreads / 32>(p, kPer, kExtra, kExtra + 1, span);
    if (span.u0 >= span.u1) {  // (all threads alike)
        if (tid == 0) wk.join[blockIdx.x] = {0, 0, 0, 0, 0};
        return;
    }
    if (tid == 0) {
        wk.join[blockIdx.x] = {0, 0, 0, 0, 0};
        for (int i = 0; i < kSlots; ++i) mbar_init(&bars.slot_full[i], 1), mbar_init(&bars.slot_empty[i], 8 + kExpandWarps);
        mbar_init(&bars.q_full, 8);
        for (int i = 0; i < 2; ++i) {
            for (int b = 0; b < 2; ++b) mbar_init(&bars.full[i][b], kExpandWarps / 2), mbar_init(&bars.empty[i][b], 1);
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i][0], 4), mbar_init(&bars.p_full[i][1], 4);
            mbar_init(&bars.pv_done[i], 1);
            mbar_init(&bars.out_full[i], 1);
        }
        bars.abort_word = 0;
        fence_mbar_init();
    }
    if (tid < 128) reinterpret_cast<uint4*>(smem + C::kZeroAt)[tid] = make_uint4(0u, 0u, 0u, 0u);
    fence_async();
    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_before();
    __syncthreads();
    tc_after();
    constexpr uint32_t tmem = 0;  // all of it: from the first lane and column on
    const Ctl k = {p, bars, &bars.abort_word};
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        softmax<D>(k, wk, smem, tmem);
    } else if (warp < kIssuer) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsExpand));
        if (warp < 12)
            expand<D, false>(k, slots, smem, warp - 8);
        else
            expand<D, true>(k, slots, smem, warp - 12);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp > kIssuer)
            factors<D>(k, wk, span, slots, warp - kIssuer - 1);
        else
            Issue<D>{k, slots, smem_u32(smem), 0}.run();
        __syncwarp();
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == kIssuer)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

// CTA (c, r): rows 32 r .. of the item whose first part is CTA c's, a warp a row at a time.
template <int D>
__global__ void __launch_bounds__(256)
    attend_many_join_kernel(const __grid_constant__ pq2h::AttendParams p, const __grid_constant__ AttendWork wk) {
    constexpr int kN = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const AttendJoin j = wk.join[blockIdx.x];
    if (j.parts == 0) return;
    const AttendItem it = attend_item<Cfg<D>::kRows>(p, j.b, j.row_tile, j.head);
    const int G = p.q_heads / p.cache.heads;
    const int rows = min(static_cast<long long>(it.n) * G - static_cast<long long>(it.row_tile) * Cfg<D>::kRows,
                         static_cast<long long>(Cfg<D>::kRows));
    const auto slot_of = [&](int i) { return i == 0 ? j.first_slot : 2 * (static_cast<int>(blockIdx.x) + i); };
    for (int row = 32 * blockIdx.y + warp; row < min(rows, 32 * static_cast<int>(blockIdx.y) + 32); row += 8) {
        float m = kEmpty, l = 0.0f, o[kN];
#pragma unroll
        for (int x = 0; x < kN; ++x) o[x] = 0.0f;
        for (int i = 0; i < j.parts; ++i) m = fmaxf(m, wk.ml[static_cast<long long>(slot_of(i)) * wk.rows + row].x);
        for (int i = 0; i < j.parts; ++i) {
            const long long at = static_cast<long long>(slot_of(i)) * wk.rows + row;
            const float2 ml = wk.ml[at];
            const float a = ex2(ml.x - m);
            l = fmaf(a, ml.y, l);
            const float2* f = reinterpret_cast<const float2*>(wk.o + at * D + lane * kN);
#pragma unroll
            for (int x = 0; x < kN / 2; ++x) {
                const float2 v = f[x];
                o[2 * x] = fmaf(a, v.x, o[2 * x]);
                o[2 * x + 1] = fmaf(a, v.y, o[2 * x + 1]);
            }
        }
        write_row<kN>(p, it, Cfg<D>::kRows, row, lane * kN, l, o);
    }
}

size_t pad(size_t b) { return (b + 255) & ~size_t(255); }

// Rows of a partial result: all of a tile's, or as many as the call has.
int part_rows(int64_t M, int64_t G, int64_t dim) {
    const int64_t rows = dim == 256 ? 128 : 256;
    return static_cast<int>(std::min(rows, (M * G + 31) / 32 * 32));
}

constexpr int kMostCtas = 160;

template <int D>
cudaError_t launch_many(const pq2h::AttendParams& p, const AttendWork& wk, cudaStream_t st, const pq2h::DeviceInfo& dev) {
    static pq2h::SmemLimit lim;
    cudaError_t e = pq2h::raise_smem(lim, attend_many_kernel<D>, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    // the softmax warps' registers come from what the block is launched with:
    // with fewer they would wait for ever
    static const bool fits = [] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, attend_many_kernel<D>) == cudaSuccess && fa.numRegs * kThreads >= kRegsNeeded;
    }();
    if (!fits) return cudaErrorLaunchOutOfResources;
    const int ctas = std::min(dev.num_sms, kMostCtas);
    e = pq2h::launch(attend_many_kernel<D>, dim3(ctas), dim3(kThreads), Cfg<D>::kSmem, st, true, p, wk);
    if (e != cudaSuccess) return e;
    return pq2h::launch(attend_many_join_kernel<D>, dim3(ctas, (wk.rows + 31) / 32), dim3(256), 0, st, true, p, wk);
}

}  // namespace
}  // namespace pq2

namespace pq2h {

size_t attend_many_workspace_bytes(int64_t M, int64_t q_heads, int64_t heads, int64_t dim) {
    const size_t rows = 2ull * pq2::kMostCtas * pq2::part_rows(M, q_heads / heads, dim);
    return pq2::pad(rows * dim * 4) + pq2::pad(rows * 8) + pq2::pad(pq2::kMostCtas * sizeof(pq2::AttendJoin));
}

cudaError_t launch_attend_many(const AttendParams& p, void* workspace, cudaStream_t st, const DeviceInfo& dev) {
    pq2::AttendWork wk = {};
    uint8_t* w = static_cast<uint8_t*>(workspace);
    wk.rows = pq2::part_rows(p.M, p.q_heads / p.cache.heads, p.dim);
    const size_t rows = 2ull * pq2::kMostCtas * wk.rows;
    wk.o = reinterpret_cast<float*>(w);
    wk.o_elems = rows * p.dim;
    w += pq2::pad(rows * p.dim * 4);
    wk.ml = reinterpret_cast<float2*>(w);
    wk.ml_elems = rows;
    w += pq2::pad(rows * 8);
    wk.join = reinterpret_cast<pq2::AttendJoin*>(w);
    switch (p.dim) {
        case 64: return pq2::launch_many<64>(p, wk, st, dev);
        case 128: return pq2::launch_many<128>(p, wk, st, dev);
    }
    return pq2::launch_many<256>(p, wk, st, dev);
}

}  // namespace pq2h
