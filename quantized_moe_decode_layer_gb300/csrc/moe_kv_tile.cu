// Attention of many rows against one key/value head, on the 5th-generation tensor
// cores (tcgen05, accumulators in tensor memory): prompts with a sliding window
// and first positions, more than 16 rows of a cache's sequence, and a batch's rows against the prefix that they share.
//
// The rows that share a key/value head (query rows times heads per key/value
// head) are packed into tiles of 128, the positions that any of a CTA's rows
// sees into tiles of two halves of 64 slots: the first ones, then the window from where it begins (in a ring, the slots that it
// lies in; each slot's position follows from where the window starts).  Per tile of positions
//     S = Q K^T            128 x 128, fp32 in tensor memory
//     P = 2^(c (S - ref))  16 bits, in tensor memory over S;  l += row sums
//     O += P V             128 x D, fp32 in tensor memory
// with c = scale log2(e) and ref a running maximum that follows only when the true one is above it by
// more than 8 / c: the weights stay below 2^8, far from any type's end, and O is
// hardly ever rescaled.  A weight is rounded to 16 bits for its product, an error of half a step of the type, as the output's own
// rounding is; l has it as it was.  fp16 holds weights 2^kUp times as large, below 2^15: its steps end at 2^-24, so those below 2^-21
// of the reference are off by 2^-32 of it (kv_up in moe_kv.h).
//
// Two streams of steps alternate on the tensor core, so that it has one's
// products while the other's softmax runs: with D <= 128 two row tiles
// (tensor memory holds their S and two O), with D = 256 the even and the odd position
// tiles of one row tile (two S, one O); those hand the reference on from
// one to the other.  A CTA is persistent and goes through items (row tiles of a head) that warp 11 finds
// ahead of the others.  Warps 0-3 and 4-7 are the streams' softmax (thread = row),
// warp 8 loads K and V by TMA (boxes of 64 positions x 64 elements, 128-byte swizzle), one thread of
// warp 9 issues the products, warps 10 and 11 load q.  V is taken as it lies, [position][d] with d
// contiguous (an MN-major operand), P from tensor memory; outputs leave through a box in shared memory.
//
// Bound by the tensor core with D = 256 (a prompt of 16K, window 4096, 16/2/256: 0.57 to 0.61 ms, 1.6 PFLOP/s of the
// pairs that are seen, 85 % of the measured rate), by a stream's chain of S, softmax and P V with D = 128 (32/8/128:
// 0.66 ms), by the latency of the softmax warps, two a scheduler, with D = 64 (32/8/64: 0.50 ms).
//
// Every wait is bounded; one that runs out sets *err, the roles stop, the CTA waits
// (bounded) for its copies and products and frees its tensor memory.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include <algorithm>
#include <climits>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "moe_kv.h"
#include "moe_kv8.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;            // rows of a tile (MMA M)
constexpr int kKeys = 128;            // positions of a tile (MMA N of the scores)
constexpr int kHalf = kKeys / 2;      // they come in halves
constexpr int kBox = 128 * 128;       // 128 rows or positions of 64 elements
constexpr int kTThreads = 384;        // softmax: warps 0-3, 4-7; loads 8; products 9; q 10, 11
constexpr int kQThreads = 64;
constexpr int kErrTimeout = 4;
constexpr int kItems = 4, kItemBytes = 48;   // items known ahead

template <int D>
struct TLay {
    static constexpr bool kPair = D <= 128;                   // two row tiles a CTA
    // S in tensor memory: one for each stream, or three that all steps take in turn, so that a stream's next scores come
    // before its P has been read
    static constexpr bool kTurns = D == 64;
    static constexpr int NB = kTurns ? 3 : 2;
    static constexpr bool kAhead = !kPair || kTurns;          // the next tile's scores come before this one's values
    static constexpr int NQ = kPair ? 2 : 1;
    static constexpr int RT = NQ * kRows;
    static constexpr int kUnit = D == 64 ? kBox : 2 * kBox;   // 128 positions x min(D, 128)
    static constexpr int UPT = D == 256 ? 2 : 1;              // units of a tile of keys or values
    static constexpr int NU = D == 64 ? 8 : 4;                // (5 at 128, 256 measured no faster)
    static constexpr int q = 0;
    static constexpr int ring = NQ * (D / 64) * kBox;
    static constexpr int stage = ring + NU * kUnit;           // outputs on their way, a box a stream
    static constexpr int bars = stage + 2 * kBox;
    static constexpr int kBars = 2 * NU + 3 * NB + 2 + 8 + 4 + 2 * kItems;
    static constexpr int misc = bars + kBars * 8;             // tensor-memory address, abort flag
    static constexpr int refs = misc + 8;                     // [128] references, [2][128] sums (one row tile)
    static constexpr int items = (refs + 3 * 128 * 4 + 15) / 16 * 16;   // [kItems] items, read 16 bytes at a time
    static constexpr int total = items + kItems * kItemBytes;
    static_assert(bars % 1024 == 0 && misc % 8 == 0 && refs % 4 == 0 && items % 16 == 0 && kItemBytes % 16 == 0, "alignment");
};
static_assert(TLay<64>::total + 1024 <= kSmemMax && TLay<128>::total + 1024 <= kSmemMax && TLay<256>::total + 1024 <= kSmemMax,
              "shared memory");
// tensor memory: S at columns 0 and 128 (and 384), O from 256 on, P over S
constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t s_col(int b) { return b == 2 ? 384u : 128u * (uint32_t)b; }
// A weight's exponent is c s - c ref, one fused product and sum with the rounded product c ref, so a row's largest one is off by
// that rounding: up to half a spacing of c ref, 2^-14 at 2^10 and 64 at 2^30, which no 16-bit weight holds.  Rows whose c ref
// is beyond 2^10 take c (s - ref) instead, where the largest is exact.  (Found by the vote that a rising reference needs anyway: 8195
// rows, window 1024, 32/8/128: 125 -> 127 us, by a vote of its own 129.)
constexpr float kFar = 1024.f;
// registers a thread: launched with 168; the softmax warps take what the others leave
constexpr int kRegsSoft = 208, kRegsRest = 88;
static_assert(256 * kRegsSoft + 128 * kRegsRest <= kTThreads * 168, "registers");

struct Once {
    std::once_flag flag[64];
    int sms[64];
};

struct TileParams {
    CUtensorMap tk, tv, tq, to;
    KvCall c;
    int qmap, omap;   // q and outputs by TMA: 128 packed rows are a rectangle of theirs
    int ntile;     // row tiles (CTAs' worth) of a head
    int nsplit;
    int items;     // row tiles times parts times heads (times sequences)
    int full;      // items from there on are cut into two of one row tile
};

__device__ __forceinline__ uint32_t su32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ unsigned long long gtime()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ void bar_init(uint32_t b, unsigned n)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(b), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t b)
{
    asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(b) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t b, unsigned bytes)
{
    asm volatile("{ .reg .b64 st; mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1; }" ::"r"(b), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t b, unsigned parity)
{
    uint32_t done;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(done)
                 : "r"(b), "r"(parity)
                 : "memory");
    return done != 0;
}
// At a CTA's end: a phase that copies or products in flight complete.  A second at least, whatever the time limit of the
// waits: what is in flight lands in microseconds, and must not land after the CTA.
__device__ __forceinline__ void bar_drain(uint32_t b, unsigned parity, const KvCall &c)
{
    const unsigned long long t0 = gtime();
    while (!bar_test(b, parity) && (long long)(gtime() - t0) <= max(c.timeout_ns, 1000000000LL)) {}
}

// Bounded wait on an mbarrier phase; gives up when the CTA's abort flag is
// set, or sets it (and the error word) when the time runs out.
__device__ __forceinline__ bool bar_wait(uint32_t b, unsigned parity, volatile int *abort, const KvCall &c)
{
    if (bar_test(b, parity)) return true;
    const unsigned long long t0 = gtime();
#pragma unroll 1
    for (;;) {
        if (bar_test(b, parity)) return true;
        if (*abort) return false;
        if ((long long)(gtime() - t0) > c.timeout_ns) {
            *abort = 1;
            atomicOr(c.err, kErrTimeout);
            return false;
        }
    }
}

// Shared-memory descriptors (tcgen05, version 1), 128-byte swizzle: the low word has the address
// (in 16 bytes), the high word is the same for all.  K-major: rows of 64 elements, 8-row
// groups 1024 bytes apart; 16 elements on are 32 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); }
// MN-major: 64 elements of N in a row of 128 bytes, the next 64 a box further; rows are
// K, 8-row groups 1024 bytes apart; 16 of K on are 2048 bytes.
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | ((uint32_t)(kBox >> 4) << 16); }
// kind::f16, fp32 accumulator, M = 128; b_mn: B is MN-major.
template <bool F16>
__device__ __forceinline__ constexpr uint32_t idesc(int n, bool b_mn)
{
    return (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}
// One thread of the warp, the same each time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(r)::"memory");
    return r != 0;
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc)
{
    asm volatile("{ .reg .pred p; .reg .b64 x, y; setp.ne.b32 p, %4, 0; mov.b64 x, {%1, %5}; mov.b64 y, {%2, %5}; "
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p; }" ::"r"(d),
                 "r"(a), "r"(b), "r"(id), "r"(acc), "n"(kDescHi)
                 : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc)
{
    asm volatile("{ .reg .pred p; .reg .b64 y; setp.ne.b32 p, %4, 0; mov.b64 y, {%2, %5}; "
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p; }" ::"r"(d),
                 "r"(a), "r"(b), "r"(id), "r"(acc), "n"(kDescHi)
                 : "memory");
}
__device__ __forceinline__ void umma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define R4(a, i) "=r"(a[i]), "=r"(a[(i) + 1]), "=r"(a[(i) + 2]), "=r"(a[(i) + 3])
#define R16(a, i) R4(a, i), R4(a, (i) + 4), R4(a, (i) + 8), R4(a, (i) + 12)
#define I4(a, i) "r"(a[i]), "r"(a[(i) + 1]), "r"(a[(i) + 2]), "r"(a[(i) + 3])
#define I16(a, i) I4(a, i), I4(a, (i) + 4), I4(a, (i) + 8), I4(a, (i) + 12)
// 32 columns of the warp's lanes
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : R16(r, 0), R16(r, 16)
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::I16(r, 0),
                 I16(r, 16), "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15};" ::I16(r, 0),
                 "r"(at)
                 : "memory");
}

__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load5(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, int c4, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_store5(const CUtensorMap *map, uint32_t src, int c0, int c1, int c2, int c3, int c4)
{
    asm volatile("cp.async.bulk.tensor.5d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5, %6}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
                 : "memory");
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint64_t two(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split2(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Rows of sequence b that the call works on, and the first one's position.
__device__ __forceinline__ int rows_of(const KvCall &p, int b, int &p0, bool &bad)
{
    const int32_t last = p.T - p.M;
    return kv8_rows(p.pos ? p.pos + b : &last, p.counts ? p.counts + b : nullptr, 0, p.M, p.limit, p0, bad);
}

// The order in which tiles of keys and values are loaded: as the steps first use them.
// K0 V0 K1 V1 ..., or, ahead, K0 K1 V0 K2 V1 ...
template <bool AHEAD>
__device__ __forceinline__ int v_order(int t, int nt) { return !AHEAD ? 2 * t + 1 : t == nt - 1 ? 2 * nt - 1 : 2 * t + 2; }

// A CTA's worth of work: row tile(s) r0 .. of one head against nt tiles of positions: halves 2 i0 .. of the list that
// has nfront halves of a tile from slot 0 on and then those from slot `from` on.
// A window's halves begin at its first position, not at a multiple of their size: a window of 128 k positions and
// its rows' 64 or so take k + 1 tiles wherever they begin, and not k + 2 (8192 positions, 16/2/256, window 100:
// 58 -> 43 us, 600: 109 -> 90; 32/8/128, 1700: 195 -> 182).  The first tokens take a half and not a tile (32/8/128,
// window 1024 and 4 first tokens: 147 -> 133 us, window 100: 76 -> 61).
struct Item {
    int z, g, b, r0;
    int one;        // one row tile of a pair, by itself
    int p0, cnt;
    int from, nfront, i0, nt;
    int sl, off;    // slot of the first position in the window; that position less its slot
    __device__ __forceinline__ int first_key(int t, int half) const
    {
        const int j = 2 * (i0 + t) + half;
        return j < nfront ? kHalf * j : from + kHalf * (j - nfront);
    }
};
template <int RT, bool PREFIX>
__device__ __forceinline__ Item item_of(const TileParams &tp, int x)
{
    const KvCall &p = tp.c;
    Item it;
    const int seqs = PREFIX ? 1 : p.B;
    it.one = x >= tp.full;
    const int second = it.one ? x - tp.full & 1 : 0, rt = it.one ? kRows : RT;
    if (it.one) x = tp.full + (x - tp.full >> 1);
    it.z = x % tp.nsplit;
    x /= tp.nsplit;
    it.g = x % p.Hkv;
    x /= p.Hkv;
    it.b = x % seqs;
    const int tile = tp.ntile - 1 - x / seqs;   // later row tiles, which see more, first
    it.r0 = tile * RT + kRows * second;
    it.p0 = it.from = it.nfront = it.nt = it.sl = it.off = 0;
    it.cnt = p.M;
    if (PREFIX) {
        if (it.r0 < p.B * p.M * p.G) it.nt = (p.P + kKeys - 1) / kKeys;
    } else {
        bool bad;
        it.cnt = rows_of(p, it.b, it.p0, bad);
        if (bad) atomicOr(p.err, kKv8ErrRange);
        const int first = p.by_g(it.r0), last = min(p.by_g(it.r0 + rt - 1), it.cnt - 1);
        if (first < it.cnt) {
            // positions lo .. hi, slots sl .. T - 1 and (a ring that they wrap around in) on from S
            const int lo = max(0, it.p0 + first - p.W + 1), hi = it.p0 + last;
            it.sl = lo < p.T ? lo : p.S + (lo - p.S) % (p.T - p.S);
            it.off = lo - it.sl;
            const int end = it.sl + (hi - lo);
            const int low = max(min(p.S, lo), end >= p.T ? p.S + end - p.T + 1 : 0);   // slots from 0 on
            it.from = it.sl;
            it.nfront = (low + kHalf - 1) / kHalf;
            if (kHalf * it.nfront >= it.sl) it.from = it.nfront = 0;   // one row of them
            it.nt = (it.nfront + (min(end, p.T - 1) - it.from) / kHalf + 2) / 2;
        }
    }
    const int each = (it.nt + tp.nsplit - 1) / tp.nsplit;
    it.i0 = min(it.nt, it.z * each);
    it.nt = min(it.nt - it.i0, each);
    return it;
}

static_assert(sizeof(Item) <= kItemBytes + 4, "an item's words (the last bit of r0 is `one`)");

// The items of a CTA, in turn.
struct Items {
    uint8_t *ring;
    uint64_t *ready, *read;
    // The n-th, once it is there.  After the last of a role's threads has it: done(n).  Where the wait gave up it holds anything, and
    // done is not called any more: an item's place is not written again while some thread may still read it.
    __device__ __forceinline__ bool get(int n, Item &it, volatile int *abort, const KvCall &c) const
    {
        const int s = n % kItems;
        const bool ok = bar_wait(su32(&ready[s]), (unsigned)(n / kItems) & 1u, abort, c);
        const int4 *w = reinterpret_cast<const int4 *>(ring + s * kItemBytes);
        const int4 a = w[0], b = w[1], d = w[2];
        it.z = a.x, it.g = a.y, it.b = a.z, it.r0 = a.w & ~1, it.one = a.w & 1;
        it.p0 = b.x, it.cnt = b.y, it.off = b.z, it.from = b.w;
        it.nfront = d.x, it.i0 = d.y, it.nt = d.z, it.sl = d.w;
        return ok;
    }
    __device__ __forceinline__ void done(int n) const { bar_arrive(su32(&read[n % kItems])); }
    __device__ __forceinline__ void put(int n, const Item &it) const
    {
        int4 *w = reinterpret_cast<int4 *>(ring + n % kItems * kItemBytes);
        w[0] = make_int4(it.z, it.g, it.b, it.r0 | it.one);
        w[1] = make_int4(it.p0, it.cnt, it.off, it.from);
        w[2] = make_int4(it.nfront, it.i0, it.nt, it.sl);
        bar_arrive(su32(&ready[n % kItems]));
    }
};

// Four lanes with 64 bytes each (16 words): lane j gets the j-th 16 bytes of each of the four, so that a store
// of the warp has 64 bytes in a row instead of 16 (128 x 128 outputs: 3 us -> below 1).
__device__ __forceinline__ void quad_transpose(uint32_t (&v)[16], int lane)
{
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            if (a & d) continue;
            const bool up = lane & d;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t &lo = v[4 * a + j], &hi = v[4 * (a + d) + j];
                const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? lo : hi, d);
                if (up) lo = got;
                else hi = got;
            }
        }
}

template <bool F16, int D, bool PREFIX>
__global__ void __launch_bounds__(kTThreads, 1) kv_tile_kernel(const __grid_constant__ TileParams tp)
{
    using L = TLay<D>;
    constexpr bool PAIR = L::kPair, AHEAD = L::kAhead, TURNS = L::kTurns;
    constexpr int KS = kHalf, NB = L::NB;
    constexpr int NU = L::NU, UPT = L::UPT, RT = L::RT;
    constexpr float kUp = kv_up(F16), kDown = 1.f / (float)(1 << (int)kUp);
    const KvCall &p = tp.c;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // (warp: uniform, as the products' operands have to be)
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    // barriers: S is there, P is there, P V is done (one for each S: none gets two phases ahead of who waits); O has been
    // read (one for each stream)
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::bars), *empty = full + NU;
    uint64_t *s_full = empty + NU, *p_full = s_full + NB, *o_done = p_full + NB,
             *o_free = o_done + NB, *ref_rdy = o_free + 2, *q_full = ref_rdy + 8, *q_free = q_full + 1, *all_done = q_free + 1,
             *alone = all_done + 1, *i_ready = alone + 1, *i_read = i_ready + kItems;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::misc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *refs = reinterpret_cast<float *>(sm + L::refs), *sums = refs + 128;

    if (tid == 0) {
        for (int s = 0; s < NU; ++s) {
            bar_init(su32(&full[s]), 1);
            bar_init(su32(&empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(su32(&o_free[s]), PAIR ? 4 : 8);
        }
        for (int s = 0; s < NB; ++s) {
            bar_init(su32(&s_full[s]), 1);
            bar_init(su32(&p_full[s]), 4);
            bar_init(su32(&o_done[s]), 1);
        }
        for (int s = 0; s < 8; ++s) bar_init(su32(&ref_rdy[s]), 1);
        for (int s = 0; s < kItems; ++s) {
            bar_init(su32(&i_ready[s]), 1);
            bar_init(su32(&i_read[s]), 12);   // the softmax warps, loads, products, q
        }
        bar_init(su32(q_full), tp.qmap ? 1 : kQThreads);
        bar_init(su32(q_free), 1);
        bar_init(su32(all_done), 1);
        bar_init(su32(alone), 8);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)), "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (p.late) place_next();
    else after_previous();
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
    const long long rows = (long long)p.M * p.G * (PREFIX ? p.B : 1);   // of a head (and sequence)
    const bool parts = p.P > 0 || tp.nsplit > 1;
    const KvCall::Parts &to_parts = PREFIX ? p.prefix : p.own;
    // whether a pair's second row tile has rows that see anything
    auto two_tiles = [&](const Item &it) { return PAIR && !it.one && it.r0 + kRows < (PREFIX ? rows : (long long)it.cnt * p.G); };
    const Items items = {sm + L::items, i_ready, i_read};
    // items of the CTA: of every turn one, of odd turns from the other end, as they are sorted by what they see (prompts of 4096,
    // all seen, 32/8/128: 124 -> 104 us, of 8192 402 -> 366).  Not where some may have nothing to do: a CTA would get the
    // same few rows from both ends (5 of up to 3000: 119 -> 150).
    const int ctas = gridDim.x, turns = tp.items / ctas;
    const bool back = !p.counts;
    auto item_no = [&](int k) { return k * ctas + (back && k & 1 ? ctas - 1 - (int)blockIdx.x : (int)blockIdx.x); };
    const int mine = turns + (item_no(turns) < tp.items ? 1 : 0);

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
        if (warp == 8) {
            // ------------------------------------------------------------- loads
            if (lane == 0) {
                bool go = true;
                int slot = 0, turn = 0, n = 0;   // of the next unit; units issued
                for (int k = 0; k < mine && go; ++k) {
                    Item it;
                    go = items.get(k, it, abort_flag, p);
                    if (!go) break;
                    items.done(k);
                    auto load = [&](const CUtensorMap *map, int t) {
                        const int key0 = it.first_key(t, 0), key1 = it.first_key(t, 1);
                        for (int u = 0; u < UPT && go; ++u) {
                            if (turn > 0 && !bar_wait(su32(&empty[slot]), (unsigned)(turn - 1) & 1u, abort_flag, p)) {
                                go = false;
                                return;
                            }
                            const uint32_t dst = su32(sm + L::ring + slot * L::kUnit), fb = su32(&full[slot]);
                            bar_expect(fb, L::kUnit);
#pragma unroll
                            for (int h = 0; h < L::kUnit / kBox; ++h) {
                                tma_load4(dst + h * kBox, map, 128 * u + 64 * h, key0, it.g, PREFIX ? 0 : it.b, fb);
                                tma_load4(dst + h * kBox + kBox / 2, map, 128 * u + 64 * h, key1, it.g, PREFIX ? 0 : it.b, fb);
                            }
                            ++n;
                            if (++slot == NU) {
                                slot = 0;
                                ++turn;
                            }
                        }
                    };
                    if (AHEAD && it.nt > 0) load(&tp.tk, 0);
                    for (int t = 0; t < it.nt && go; ++t) {
                        const int kt = AHEAD ? t + 1 : t;
                        if (kt < it.nt) load(&tp.tk, kt);
                        if (go) load(&tp.tv, t);
                    }
                }
                // every copy issued has landed before the CTA ends
                for (int s = 0; s < NU && s < n; ++s) bar_drain(su32(&full[s]), (unsigned)((n - 1 - s) / NU) & 1u, p);
            }
        } else if (warp >= 10) {
            // ---------------------------------------------------- q, packed into rows
            // and, ahead of all others, which items there are: warp 11 writes two more than are worked on
            constexpr int CH = D / 8;
            const int t = tid - 320;
            int qn = 0;
            bool go = true;
            auto tell = [&](int k) {
                if (warp != 11 || lane != 0 || k >= mine) return;
                const Item it = item_of<RT, PREFIX>(tp, item_no(k));
                if (k >= kItems && !bar_wait(su32(&i_read[k % kItems]), (unsigned)(k / kItems - 1) & 1u, abort_flag, p)) return;
                items.put(k, it);
            };
            tell(0);
            tell(1);
            for (int k = 0; k < mine; ++k) {
                Item it;
                go = __all_sync(0xFFFFFFFFu, items.get(k, it, abort_flag, p));
                if (!go) break;
                if (lane == 0) items.done(k);
                // (warp 11 only where it loads, too: else q could be freed twice before it looks, and it would wait for a phase
                // that is gone)
                if (it.nt > 0 && qn > 0 && (warp == 10 || !tp.qmap)) go = bar_wait(su32(q_free), (unsigned)(qn - 1) & 1u, abort_flag, p);
                go = __all_sync(0xFFFFFFFFu, go);
                if (!go) break;
                if (it.nt == 0) {
                    tell(k + 2);
                    __syncwarp();
                    continue;
                }
                ++qn;
                if (tp.qmap) {
                    if (t == 0) {
                        const int nq = it.one ? 1 : L::NQ;
                        bar_expect(su32(q_full), nq * (D / 64) * kBox);
                        // packed rows r0 .. : the token of r0 (of all sequences' in turn, for a prefix)
                        const int m = p.by_g(it.r0);
#pragma unroll
                        for (int j = 0; j < L::NQ; ++j) {
                            if (j == nq) break;
#pragma unroll
                            for (int h = 0; h < D / 64; ++h)
                                tma_load5(su32(sm + L::q) + (j * (D / 64) + h) * kBox, &tp.tq, 64 * h, 0, it.g, m + j * (kRows / p.G),
                                          PREFIX ? 0 : it.b, su32(q_full));
                        }
                    }
                    tell(k + 2);    // (behind the loads, which others wait for)
                    __syncwarp();
                    continue;
                }
                // (rows of idle sequences and padding are read like the others; nothing of them is used)
                constexpr int STEP = kQThreads / CH;   // rows a pass
                const int rt = it.one ? kRows : RT;
                const int c = t % CH, rr0 = t / CH;
                int r = it.r0 + rr0, m = p.by_g(r), h = r - m * p.G, bb = it.b;
                if (PREFIX) {
                    bb = m / p.M;
                    m -= bb * p.M;
                }
                const uint16_t *src = p.q + (long long)bb * p.qb + (long long)m * p.qm + (long long)(it.g * p.G + h) * p.qh + 8 * c;
#pragma unroll 4
                for (int rr = rr0; rr < rt; rr += STEP) {
                    const bool ok = r < rows;   // rows that are not there are zeros
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                     su32(sm + L::q) + ((rr >> 7) * (D / 64) + (c >> 3)) * kBox + (rr & 127) * 128 + (((c & 7) ^ (rr & 7)) << 4)),
                                 "l"(ok ? src : p.q), "r"(ok ? 16 : 0)
                                 : "memory");
                    r += STEP;
                    h += STEP;
                    src += STEP * p.qh;
                    while (h >= p.G) {   // the next query row
                        h -= p.G;
                        src += p.qm - p.G * p.qh;
                        if (PREFIX && ++m == p.M) {
                            m = 0;
                            src += p.qb - p.M * p.qm;
                        }
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                bar_arrive(su32(q_full));
                tell(k + 2);
                __syncwarp();
            }
            // the last copies have landed before the CTA ends
            if (tp.qmap && t == 0 && qn > 0) bar_drain(su32(q_full), (unsigned)(qn - 1) & 1u, p);
        } else {
            // ---------------------------------------------------------- products
            // One thread, and as few instructions between the products as can be: they are issued in order,
            // and a step's 16 of 128 x 128 x 16 take the tensor core about 1000 cycles.
            if (elect_one()) {
                bool go = true;
                constexpr uint32_t id_s = idesc<F16>(kKeys, false), id_o = idesc<F16>(D < 128 ? D : 128, true);
                const uint32_t ring = su32(sm + L::ring), qd = desc_k(su32(sm + L::q));
                auto wait = [&](uint64_t *bar, int parity) { go = go && bar_wait(su32(bar), (unsigned)parity & 1u, abort_flag, p); };
                struct Place {   // of a unit in the ring, with its phase
                    int slot, phase;
                    __device__ __forceinline__ void move(int by)
                    {
                        slot += by;
                        if (slot >= NU) {
                            slot -= NU;
                            phase ^= 1;
                        }
                    }
                };
                Place base = {0, 0};
                int qn = 0, turns[2] = {0, 0};    // items, those of each stream
                int sb = 0, pb = 0, pphase = 0;   // taken in turn: S of the next scores; P of the next values, with its phase
                int phase0 = 0, phase1 = 0;       // else the phases of the streams' P
                for (int n = 0; n < mine && go; ++n) {
                    Item it;
                    go = items.get(n, it, abort_flag, p);
                    if (!go) break;
                    items.done(n);
                    const int nt = it.nt;
                    if (nt == 0) continue;
                    auto work = [&](auto duo_v) {
                        constexpr bool duo = decltype(duo_v)::value;   // a pair's second stream has something to do
                        constexpr bool both = !PAIR || duo;            // the streams take turns
                        const int n = duo ? 2 * nt : nt;               // steps
                        Place kp = base, vp = base;                    // of the next tile of keys, of values
                        vp.move(AHEAD && nt > 1 ? 2 * UPT : UPT);
                        auto scores = [&](int j, int xs) {
                            Place at = kp;
                            const int sn = TURNS ? sb : xs;
                            const uint32_t to = tmem + s_col(sn);
    #pragma unroll
                            for (int u = 0; u < UPT; ++u) {
                                if (!duo || xs == 0) wait(&full[at.slot], at.phase);
                                if (!go) return;
                                fence_after();
                                const uint32_t a0 = qd + (uint32_t)((((PAIR ? xs : 0) * (D / 64) + 2 * u) * kBox) >> 4);
                                const uint32_t b0 = desc_k(ring + at.slot * L::kUnit);
    #pragma unroll
                                for (int k = 0; k < (D < 128 ? D : 128) / 16; ++k) {
                                    const uint32_t off = (uint32_t)((k >> 2) * kBox + (k & 3) * 32) >> 4;
                                    umma_ss(to, a0 + off, b0 + off, id_s, (u | k) != 0 ? 1u : 0u);
                                }
                                if (!duo || xs == 1) umma_commit(su32(&empty[at.slot]));
                                at.move(1);
                            }
                            umma_commit(su32(&s_full[sn]));
                            if (j == n - 1) umma_commit(su32(q_free));
                            if (TURNS && ++sb == NB) sb = 0;
                            if (!duo || xs == 1) kp.move(AHEAD && (duo ? j < 2 : j < 1) ? UPT : 2 * UPT);
                        };
                        auto values = [&](int j, int xs) {
                            const int t = duo ? j >> 1 : j;
                            if (t == 0 && turns[xs] > 0) wait(&o_free[PAIR ? xs : 0], turns[xs] - 1);
                            if (!duo || xs == 0) {
                                Place at = vp;
    #pragma unroll
                                for (int u = 0; u < UPT; ++u) {
                                    wait(&full[at.slot], at.phase);
                                    at.move(1);
                                }
                            }
                            const int pn = TURNS ? pb : xs;
                            wait(&p_full[pn], TURNS ? pphase : xs ? phase1 : phase0);
                            if (!go) return;
                            fence_after();
                            Place at = vp;
                            const uint32_t from = tmem + s_col(pn);
    #pragma unroll
                            for (int u = 0; u < UPT; ++u) {
                                const uint32_t o = tmem + 256u + (PAIR ? (uint32_t)(D * xs) : 128u * u);
                                const uint32_t b0 = desc_mn(ring + at.slot * L::kUnit);
    #pragma unroll
                                for (int k = 0; k < kKeys / 16; ++k)
                                    umma_ts(o, from + 8u * k, b0 + 128u * k, id_o, (t | k) != 0 ? 1u : 0u);
                                if (!duo || xs == 1) umma_commit(su32(&empty[at.slot]));
                                at.move(1);
                            }
                            umma_commit(su32(&o_done[pn]));
                            if (!TURNS) {
                                if (xs) phase1 ^= 1;
                                else phase0 ^= 1;
                            } else if (++pb == NB) {
                                pb = 0;
                                pphase ^= 1;
                            }
                            if (!duo || xs == 1) vp.move(AHEAD && t + 2 >= nt ? UPT : 2 * UPT);
                        };
                        constexpr int second = both ? 1 : 0, ahead = TURNS || both ? NB : 1;   // (a stream alone with its S waits for its P)
                        auto step = [&](int j, int xs) {
                            values(j, xs);
                            if (go && j + ahead < n) scores(j + ahead, both && TURNS ? xs ^ 1 : xs);
                        };
                        wait(q_full, qn);
                        if (go) scores(0, 0);
                        if (go && ahead > 1 && n > 1) scores(1, second);
                        if (go && ahead > 2 && n > 2) scores(2, 0);
    #pragma unroll 1
                        for (int j = 0; j < n && go; j += 2) {
                            step(j, 0);
                            if (go && j + 1 < n) step(j + 1, second);
                        }
                        for (int j = 0; j < (2 * nt) % NU; ++j) base.move(UPT);
                        base.phase ^= (2 * nt / NU * UPT) & 1;
                        ++turns[0];
                        turns[1] += duo;
                        ++qn;
                    };
                    if (PAIR && two_tiles(it)) work(std::true_type());
                    else work(std::false_type());
                }
                // every product issued has finished before tensor memory is freed
                umma_commit(su32(all_done));
                bar_drain(su32(all_done), 0u, p);
            }
        }
        __syncwarp();
    } else {
        // --------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
        const int xs = warp >> 2, w = warp & 3, row = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
        const uint32_t oc = lanes + 256u + (PAIR ? (uint32_t)(D * xs) : 0u);
        const float c = p.c;
        const uint64_t c2 = two(c, c);
        int alones = 0;   // items of the first stream alone
        int done[2] = {0, 0}, all = 0, units = 0;   // steps of the streams and of both, units of the ring before this item
        bool go = true;
        auto wait = [&](uint64_t *bar, int parity) {
            go = __all_sync(0xFFFFFFFFu, go && bar_wait(su32(bar), (unsigned)parity & 1u, abort_flag, p));
        };
        // After a wait has given up a warp goes through the rest without work, as all warps of a stream still meet at each
        // item's barriers: whether they do must not depend on an item, which may be half written then.
#pragma unroll 1
        for (int n = 0; n < mine; ++n) {
            Item it;
            {
                const bool ok = items.get(n, it, abort_flag, p);
                go = __all_sync(0xFFFFFFFFu, go && ok);
                if (go && lane == 0) items.done(n);
            }
            const bool duo = two_tiles(it);
            const int nt = !go || (PAIR && xs == 1 && !duo) ? 0 : it.nt, nsteps = PAIR ? 2 * nt : nt, r = it.r0 + (PAIR ? 128 * xs : 0) + row;
            const size_t part0 = ((size_t)it.z * p.Hkv + it.g) * ((size_t)p.B * p.M * p.G) + (PREFIX ? 0 : (size_t)it.b * p.M * p.G);
            // The row is at position pos.  Slot s has position s (s < S), else s + off (s >= sl),
            // else s + off + R; it is seen if pos - W < position <= pos, or s < S.
            // Slots hole0 .. hole1 - 1 and from valid on may hold anything.  In a ring: all that none of the item's rows sees, as rows that
            // were appended and rejected lie behind the last position some way around.
            int pos = 0, valid = INT_MAX, hole0 = 0, hole1 = 0;
            const int R = p.ring ? p.T - p.S : kKvAll;
            // halves that all rows see all of: `inner` of the window's from inner0 on (others that are take the slower way)
            int inner0 = 0, inner = p.P / kHalf - 2 * it.i0;
            if (!PREFIX) {
                const int ra = it.r0 + (PAIR ? 128 * xs : 0);
                const int pos_lo = it.p0 + p.by_g(ra), pos_hi = it.p0 + p.by_g(ra + kRows - 1);
                pos = it.p0 + p.by_g(r);
                if (it.p0 + it.cnt <= p.T) valid = it.p0 + it.cnt;
                if (p.ring) {
                    const int last = min(p.by_g(it.r0 + (it.one ? kRows : RT) - 1), it.cnt - 1), end = it.p0 + last - it.off;
                    hole0 = max(min(p.S, it.sl + it.off), end >= p.T ? p.S + end - p.T + 1 : 0);
                    hole1 = it.sl;
                    valid = end < p.T - 1 ? end + 1 : INT_MAX;
                }
                int lo = pos_hi - it.off - p.W + 1;
                if (lo <= max(it.sl, p.S)) lo = it.sl;
                inner0 = it.nfront + (lo - it.from + kHalf - 1) / kHalf;
                inner = it.nfront + (min(p.T, pos_lo - it.off + 1) - it.from) / kHalf - inner0;
                inner0 -= 2 * it.i0;
            }
            inner = max(inner, 0);
            float l = 0.f, ref = -INFINITY;    // of the row, as the stream knows them
#pragma unroll 1
            for (int i = xs; i < nsteps && go; i += 2) {
                const int t = PAIR ? i >> 1 : i;
                const int turn = TURNS ? all + (duo ? i : t) : done[xs] + (i >> 1), sb = TURNS ? turn % NB : xs;   // the step's turn at its S
                const uint32_t sc = lanes + s_col(sb);
                wait(&s_full[sb], TURNS ? turn / NB : turn);
                if (!go) break;
                fence_after();
                auto all_seen = [&](int half) { return (unsigned)(2 * t + half - inner0) < (unsigned)inner; };
                auto any_left = [&](int key) { return valid < key + kHalf || max(key, hole0) < min(key + kHalf, hole1); };
                if (!PREFIX && !(all_seen(0) && all_seen(1)) && (any_left(it.first_key(t, 0)) || any_left(it.first_key(t, 1))) && (!PAIR || xs == 0)) {
                    // values that may be anything: zeros
                    const int n0 = units + UPT * v_order<AHEAD>(t, nt);
                    // Their place's phase before has to be over, or the wait below would take the one before that for it.  It is that of values
                    // whose product came before these scores, or of keys; with one row tile, of the values of the tile before, which nothing
                    // has waited for yet.  (The last tile's place had its own keys.)
                    if (!PAIR && t > 0 && t + 1 < nt) wait(&o_done[xs ^ 1], done[xs ^ 1] + ((i - 1) >> 1));
#pragma unroll 1
                    for (int u = n0; u < n0 + UPT; ++u) {
                        wait(&full[u % NU], u / NU);
                        if (!go) break;
                        uint8_t *unit = sm + L::ring + (u % NU) * L::kUnit;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int key = it.first_key(t, half);
                            for (int j = row; j < kHalf * 8; j += 128) {
                                const int slot = key + (j >> 3);
                                if (slot < valid && (slot < hole0 || slot >= hole1)) continue;
#pragma unroll
                                for (int h = 0; h < L::kUnit / kBox; ++h)
                                    *reinterpret_cast<uint4 *>(unit + h * kBox + half * (kBox / 2) + j * 16) = make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                    }
                    if (!go) break;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                uint32_t s0[KS], s1[KS];    // the positions' halves
                uint32_t pk[kKeys / 2];
                uint64_t add[2] = {0ull, 0ull};
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto load = [&](int half, uint32_t *s) {
#pragma unroll
                    for (int k = 0; k < KS / 32; ++k) tmem_ld32(sc + (uint32_t)(KS * half + 32 * k), s + 32 * k);
                };
                auto hide = [&](int half, uint32_t *s) {
                    if (all_seen(half)) return;
                    const int key = it.first_key(t, half);
                    auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
#pragma unroll
                    for (int k = 0; k < KS / 32; ++k) {
                        const int at = key + 32 * k;
                        uint32_t sees = below(p.P - at);
                        if (!PREFIX) {
                            const int a = pos - it.off + 1;      // past the last slot
                            sees = below(min(p.S, pos + 1) - at) | (below(min(a, p.T) - at) & ~below(max(a - p.W, max(it.sl, p.S)) - at));
                            if (p.ring) sees |= below(min(a - R, it.sl) - at) & ~below(max(a - R - p.W, p.S) - at);   // on the other side of sl
                        }
                        if (__all_sync(0xFFFFFFFFu, sees == ~0u)) continue;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(sees >> j & 1u)) s[32 * k + j] = 0xFF800000u;
                    }
                };
                auto largest = [&](const uint32_t *s) {
#pragma unroll
                    for (int k = 0; k < KS; k += 8)
#pragma unroll
                        for (int j = 0; j < 4; ++j) mx[j] = max3(mx[j], __uint_as_float(s[k + j]), __uint_as_float(s[k + 4 + j]));
                };
                auto weights = [&](int half, const uint32_t *s, uint64_t sub2) {
#pragma unroll
                    for (int j = 0; j < KS / 2; ++j) {
                        float e0, e1;
                        split2(fma2(two(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), c2, sub2), e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        add[j & 1] = add2(add[j & 1], two(e0, e1));
                        pk[KS / 2 * half + j] = pack2<F16>(e0, e1);
                    }
                };
                load(0, s0);
                tmem_wait_ld();
                load(1, s1);
                hide(0, s0);
                largest(s0);
                tmem_wait_ld();
                hide(1, s1);
                largest(s1);
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                float was = ref;
                if (!PAIR && i > 0) {   // the reference, from the stream that has the tile before
                    wait(&ref_rdy[4 * (xs ^ 1) + w], done[xs ^ 1] + ((i - 1) >> 1));
                    if (!go) break;
                    was = refs[row];
                }
                const bool raise = __fsub_rn(top, was) * c > 8.f;   // (a sum of was and the slack would round past top where scores are far apart)
                const float now = raise ? top : was;
                if (!PAIR) {
                    refs[row] = now;
                    __syncwarp();
                    if (lane == 0) bar_arrive(su32(&ref_rdy[4 * xs + w]));
                }
                if (now != ref) l *= ref == -INFINITY ? 0.f : ex2((ref - now) * c);
                ref = now;
                float sub = ref == -INFINITY ? 0.f : __fmaf_rn(-ref, c, kUp);
                const bool far = fabsf(sub) > kFar;
                if (__any_sync(0xFFFFFFFFu, raise || far)) {     // (hardly ever)
                    if (__any_sync(0xFFFFFFFFu, raise) && t > 0) {
                        // O, which has the tiles up to the one before, in the new reference's units
                        if (TURNS) {
                            const int before = turn - (duo ? 2 : 1);
                            wait(&o_done[before % NB], before / NB);
                        } else {
                            wait(&o_done[PAIR ? xs : xs ^ 1], PAIR ? turn - 1 : done[xs ^ 1] + ((i - 1) >> 1));
                        }
                        if (!go) break;
                        fence_after();
                        const float f = raise ? ex2((was - now) * c) : 1.f;
#pragma unroll 1
                        for (int k = 0; k < D; k += 32) {
                            uint32_t o[32];
                            tmem_ld32(oc + k, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st32(oc + k, o);
                        }
                    }
                    if (__any_sync(0xFFFFFFFFu, far)) {
                        const float shift = far ? -ref : 0.f;   // (0 changes nothing)
                        const uint64_t shift2 = two(shift, shift);
                        auto move = [&](uint32_t *s) {
#pragma unroll
                            for (int j = 0; j < KS; j += 2) {
                                float a, b;
                                split2(add2(two(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), shift2), a, b);
                                s[j] = __float_as_uint(a);
                                s[j + 1] = __float_as_uint(b);
                            }
                        };
                        move(s0);
                        move(s1);
                        if (far) sub = kUp;
                    }
                }
                weights(0, s0, two(sub, sub));
                // (one half's P on its way while the other's is computed: 16384 positions, all seen, 1157 -> 1132 us with 64
                // columns, 1547 -> 1528 with 128, 1294 -> 1312 with 256)
#pragma unroll
                for (int k = 0; k < 2; ++k) tmem_st16(sc + 16u * k, pk + 16 * k);
                weights(1, s1, two(sub, sub));
                float a0, a1;
                split2(add2(add[0], add[1]), a0, a1);
                l += a0 + a1;
#pragma unroll
                for (int k = 2; k < 4; ++k) tmem_st16(sc + 16u * k, pk + 16 * k);
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(su32(&p_full[sb]));
            }

            // -------------------------------------------------------------- outputs
            // thread = row; with one row tile a CTA the warp groups take half of the columns each
            constexpr int NC = PAIR ? D : 128;
            const int col0 = PAIR ? 0 : 128 * xs;
            if (!PAIR) {
                asm volatile("bar.sync 1, 256;" ::: "memory");    // the references are final
                const float end = refs[row];
                sums[128 * xs + row] = ref == -INFINITY ? l : l * ex2((ref - end) * c);   // (without a reference l is 0 or NaN)
                ref = end;
                asm volatile("bar.sync 1, 256;" ::: "memory");
                l = sums[row] + sums[128 + row];
                if (nt == 0) l = 0.f, ref = -INFINITY;
            }
            if (nt > 0) {
                if (TURNS) {
                    const int last = all + (duo ? 2 * nt - 2 + xs : nt - 1);
                    wait(&o_done[last % NB], last / NB);
                } else if (PAIR) {
                    wait(&o_done[xs], done[xs] + nt - 1);
                } else {
                    // the last step's, and the one's before (one of them is the other stream's, whose phases are not followed else)
                    if (nt > 1) wait(&o_done[nt & 1], done[nt & 1] + ((nt - 2) >> 1));
                    wait(&o_done[(nt - 1) & 1], done[(nt - 1) & 1] + ((nt - 1) >> 1));
                }
                if (go) fence_after();
            }
            // A second stream without work stays behind the first: its next wait is for the phase after this item's.
            if (TURNS && go && !duo && it.nt > 0) {
                __syncwarp();
                if (lane == 0) bar_arrive(su32(alone));
                wait(alone, alones++);
            }
            done[0] += PAIR ? nt : (nt + 1) / 2;
            done[1] += PAIR ? nt : nt / 2;
            all += duo ? 2 * it.nt : it.nt;
            units += 2 * it.nt * UPT;
            const bool live = PREFIX || p.by_g(r) < it.cnt;
            const float inv = live && nt > 0 && l != 0.f ? 1.f / l : 0.f;
            if (l != l && ref == -INFINITY) ref = 0.f;   // a row of NaN alone has no maximum, but is not empty
            const bool mine_too = go && !(PAIR && xs == 1 && it.one);   // (else another item's)
            if (!PREFIX && tp.omap) {
                // 64 columns at a time into the stream's box, and from there by TMA while the next item starts
                uint8_t *box = sm + L::stage + xs * kBox;
#pragma unroll 1
                for (int k = 0; k < NC / 64; ++k) {
                    if ((tid & 127) == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    asm volatile("bar.sync %0, 128;" ::"r"(2 + xs) : "memory");   // the box is free
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (!mine_too) break;
                        uint32_t o[32];
                        tmem_ld32(oc + col0 + 64 * k + 32 * half, o);   // (not used where there is nothing to see)
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t v[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                v[q] = live && nt > 0 ? pack2<F16>(__uint_as_float(o[8 * j + 2 * q]) * inv, __uint_as_float(o[8 * j + 2 * q + 1]) * inv) : 0u;
                            *reinterpret_cast<uint4 *>(box + row * 128 + (((4 * half + j) ^ (row & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    asm volatile("bar.sync %0, 128;" ::"r"(2 + xs) : "memory");   // and full
                    const int m = p.by_g(r);
                    if ((tid & 127) == 0 && mine_too && m < p.M) {
                        tma_store5(&tp.to, su32(box), col0 + 64 * k, 0, it.g, m, it.b);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                }
            } else if (mine_too) {
                // Four lanes exchange 64-byte pieces: lane 4 a + j then has piece j of rows 4 a .. 4 a + 3.
                if (parts && r < rows && col0 == 0) *reinterpret_cast<float2 *>(to_parts.ml + (part0 + r) * 2) = make_float2(ref * c, l * kDown);
                const int rq = r - (lane & 3);
                uint8_t *to[4];     // the four rows' places
                int m = p.by_g(rq), h = rq - m * p.G - 1;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (++h == p.G) {
                        h = 0;
                        ++m;
                    }
                    to[j] = parts ? reinterpret_cast<uint8_t *>(to_parts.o + (part0 + rq + j) * D + col0)
                                  : reinterpret_cast<uint8_t *>(static_cast<uint16_t *>(p.o) +
                                                                (((size_t)it.b * p.M + m) * p.Hq + it.g * p.G + h) * D + col0);
                    to[j] += 16 * (lane & 3);
                }
#pragma unroll 1
                for (int k = 0; k < NC / 32; ++k) {
                    uint32_t o[32];
                    if (nt > 0) {
                        tmem_ld32(oc + col0 + 32 * k, o);
                        tmem_wait_ld();
                    } else if (parts) {
                        break;      // an empty part
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (!parts && half) break;
                        uint32_t v[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (parts) v[j] = __float_as_uint(__uint_as_float(o[16 * half + j]) * kDown);
                            else v[j] = live && nt > 0 ? pack2<F16>(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv) : 0u;
                        }
                        quad_transpose(v, lane);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (rq + j < rows)
                                *reinterpret_cast<uint4 *>(to[j] + (parts ? 128 * k + 64 * half : 64 * k)) =
                                    make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    }
                }
            }
            if (nt > 0 && go) {
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(su32(&o_free[PAIR ? xs : 0]));
            }
        }
        if (!PREFIX && tp.omap && (tid & 127) == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    if (p.late) wait_for_previous();   // the end of this kernel means the end of the one before
    fence_before();
    __syncthreads();
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &qr) == cudaSuccess &&
            qr == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// The encoder needs a current context, which a thread without a CUDA call so far has none of.
bool bind_context()
{
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
}

// [sequence][head][position][d], strides in elements; a dimension of one entry may have any.  (A call's first map is one of these.)
bool map_of(CUtensorMap *map, const uint16_t *base, bool f16, int D, int T, int heads, int seqs, long long row, long long head,
            long long seq)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)T, (cuuint64_t)heads, (cuuint64_t)seqs};
    auto bytes = [&](long long s, int n) { return (cuuint64_t)(n > 1 ? s * 2 : D * 2); };
    const cuuint64_t strides[3] = {bytes(row, T), bytes(head, heads), bytes(seq, seqs)};
    const cuuint32_t box[4] = {64, (cuuint32_t)kHalf, 1, 1}, es[4] = {1, 1, 1, 1};
    auto done = [&] {
        return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(base), dims,
                   strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    return done() || (bind_context() && done());
}

// Packed rows as rectangles of a tensor: [sequence][token][key/value head][head of the group][d].  Needs a group
// that divides a row tile, and strides that are not 0 (an expanded q is left to plain loads).
bool packed_map(CUtensorMap *map, const KvCall &c, const void *base, long long tokens, int seqs, long long head, long long token,
                long long seq)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc || kRows % c.G != 0 || tokens > INT_MAX) return false;
    if ((c.Hq > 1 && head == 0) || (tokens > 1 && token == 0) || (seqs > 1 && seq == 0)) return false;
    const cuuint64_t dims[5] = {(cuuint64_t)c.D, (cuuint64_t)c.G, (cuuint64_t)c.Hkv, (cuuint64_t)tokens, (cuuint64_t)seqs};
    auto bytes = [&](long long s, long long n) { return (cuuint64_t)(n > 1 ? s * 2 : c.D * 2); };   // (one entry: any stride)
    const cuuint64_t strides[4] = {bytes(head, c.G), bytes(c.G * head, c.Hkv), bytes(token, tokens), bytes(seq, seqs)};
    const cuuint32_t box[5] = {64, (cuuint32_t)c.G, 1, (cuuint32_t)(kRows / c.G), 1}, es[5] = {1, 1, 1, 1, 1};
    return enc(map, c.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims,
               strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int row_tile(int D) { return D == 256 ? kRows : 2 * kRows; }

}  // namespace

long long kv_row_tiles(long long rows, int D) { return (rows + row_tile(D) - 1) / row_tile(D); }

// Parts that the positions of each row tile are cut into: as many as fill the SMs in as few
// turns as possible.  `ctas` row tiles of all heads, `tiles` tiles of positions each; an item costs about four
// tiles besides, one that leaves a part four more, and the merge that `rows` rows of all heads then need (0: they have it
// anyway) two and a third of one for each thousand rows.  (32/8/64: 512 rows at 512 positions are 28 us in two parts, 10 in one; 64 at
// 4096 are 15 in 16 parts, 34 in one.)  Where rows are few (a cache's attention: bound by HBM, loads run ahead into the next item) and more
// than the SMs, shorter items, none below four tiles, even out what the lengths, which the host does not know, differ by
// (256 of 100 to 2000 positions: 80 -> 56 us).
int kv_tile_most(long long ctas, bool ragged) { return (int)std::max<long long>(1, (ragged ? 4 : 3) * 152 / ctas); }
int kv_tile_splits(long long ctas, long long tiles, bool ragged, long long rows)
{
    const int most = kv_tile_most(ctas, ragged);
    if (ragged && ctas >= 152) return (int)std::max<long long>(1, std::min<long long>(most, tiles / 4));
    int best = 1;
    double cost = 1e30;
    for (int s = 1; s <= most && s <= tiles; ++s) {
        const bool cut = s > 1 && rows > 0;
        const double turns = (double)((ctas * s + 151) / 152), item = (double)((tiles + s - 1) / s) + (cut ? 8.0 : 4.0);
        const double c = turns * item + 0.05 * s + (cut ? 2.5 + rows / 3000.0 : 0.0);
        if (c < cost) {
            cost = c;
            best = s;
        }
    }
    return best;
}

int launch_kv_tiles(const KvCall &c, bool prefix, cudaStream_t stream)
{
    TileParams tp;
    memset(&tp, 0, sizeof tp);
    tp.c = c;
    bool ok;
    if (prefix)
        ok = map_of(&tp.tk, c.pk, c.f16, c.D, c.P, c.Hkv, 1, c.pkm, c.pkh, 0) &&
             map_of(&tp.tv, c.pv, c.f16, c.D, c.P, c.Hkv, 1, c.pvm, c.pvh, 0);
    else
        ok = map_of(&tp.tk, c.k, c.f16, c.D, c.T, c.Hkv, c.B, c.km, c.kh, c.kb) &&
             map_of(&tp.tv, c.v, c.f16, c.D, c.T, c.Hkv, c.B, c.vm, c.vh, c.vb);
    if (!ok) return MOE_ERR_UNSUPPORTED;
    if (!prefix) {
        tp.qmap = packed_map(&tp.tq, c, c.q, c.M, c.B, c.qh, c.qm, c.qb);
        const long long row = (long long)c.Hq * c.D;
        tp.omap = c.own.n == 1 && c.P == 0 && packed_map(&tp.to, c, c.o, c.M, c.B, c.D, row, row * c.M);
    } else if (c.B == 1 || c.M == 1 || c.qb == c.M * c.qm) {   // the batch's tokens have one stride
        tp.qmap = packed_map(&tp.tq, c, c.q, (long long)c.B * c.M, 1, c.qh, c.M == 1 ? c.qb : c.qm, 0);
    }
    const long long rows = (long long)c.M * c.G * (prefix ? c.B : 1);
    tp.nsplit = prefix ? c.prefix.n : c.own.n;
    const long long ntile = kv_row_tiles(rows, c.D), ctas = ntile * tp.nsplit * c.Hkv * (prefix ? 1 : c.B);
    if (rows > INT_MAX - 1024 || ctas > INT_MAX - 1024) return MOE_ERR_UNSUPPORTED;
    tp.ntile = (int)ntile;
    tp.items = (int)ctas;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
    auto go = [&](auto kernel, int smem, Once &once) {
        std::call_once(once.flag[dev], [&] {
            e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
            if (e == cudaSuccess) e = cudaDeviceGetAttribute(&once.sms[dev], cudaDevAttrMultiProcessorCount, dev);
        });
        if (e == cudaSuccess && once.sms[dev] < 1) e = cudaErrorInvalidDevice;
        // The last turn's pairs, where they leave half of the SMs without any, are cut: with 128 columns 2 x 2048 rows
        // behind 6001, window 2048: 129 -> 121 us, 3 x 1700: 82 -> 79.  (With 64 a stream alone is no faster: 97 -> 94, 61 -> 64.)
        const int left = e == cudaSuccess ? tp.items % once.sms[dev] : 0;
        tp.full = tp.items;
        if (c.D == 128 && rows > kRows && 2 * left <= once.sms[dev]) {
            tp.full -= left;
            tp.items += left;
        }
        if (e == cudaSuccess)
            e = launch_after(kernel, dim3((unsigned)std::min(tp.items, once.sms[dev])), kTThreads, smem, 0, stream, tp);
    };
#define KV_TILE(F, D, P)                                                 \
    do {                                                                 \
        static Once once;                                                \
        go(kv_tile_kernel<F, D, P>, TLay<D>::total + 1024, once);        \
    } while (0)
#define KV_TILE_P(F, D)                  \
    do {                                 \
        if (prefix) KV_TILE(F, D, true); \
        else KV_TILE(F, D, false);       \
    } while (0)
#define KV_TILE_D(F)                              \
    do {                                          \
        if (c.D == 256) KV_TILE_P(F, 256);        \
        else if (c.D == 128) KV_TILE_P(F, 128);   \
        else KV_TILE_P(F, 64);                    \
    } while (0)
    if (c.f16) KV_TILE_D(true);
    else KV_TILE_D(false);
#undef KV_TILE_D
#undef KV_TILE_P
#undef KV_TILE
    if (e != cudaSuccess) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
    note_launch();
    return MOE_OK;
}

}  // namespace moe
