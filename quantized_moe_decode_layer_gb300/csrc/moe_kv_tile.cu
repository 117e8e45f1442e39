// Attention of many rows against one key/value head, on the 5th-generation tensor
// cores (tcgen05, accumulators in tensor memory): prompts with a sliding window
// and first positions, and a batch's rows against the prefix that they share.
//
// The rows that share a key/value head (query rows times heads per key/value
// head) are packed into tiles of 128, the positions that any of a CTA's rows
// sees into tiles of 128 positions: the first ones, then the window.  Per tile
// of positions
//     S = Q K^T            128 x 128, fp32 in tensor memory
//     P = 2^(c S - ref)    16 bits, in tensor memory over S;  l += row sums
//     O += P V             128 x D, fp32 in tensor memory
// with ref a running maximum that follows only when the true one is above it by
// more than 8: the weights stay below 2^8, far from any type's end, and O is
// hardly ever rescaled.
//
// Two streams of steps alternate on the tensor core, so that it has one's
// products while the other's softmax runs: with D <= 128 two row tiles
// (tensor memory holds two S and two O), with D = 256 the even and the odd position
// tiles of one row tile (two S, one O); those hand the reference on from
// one to the other.  Warps 0-3 and 4-7 are the streams' softmax (thread = row),
// warp 8 loads by TMA (boxes of 128 positions x 64 elements, 128-byte swizzle),
// warp 9 issues the products.  V is taken as it lies, [position][d] with d
// contiguous (an MN-major operand), P from tensor memory.
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

#include "moe_kv.h"
#include "moe_kv8.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;            // rows of a tile (MMA M)
constexpr int kKeys = 128;            // positions of a tile (MMA N of the scores)
constexpr int kBox = 128 * 128;       // one TMA box: 128 positions of 64 elements
constexpr int kTThreads = 320;
constexpr int kErrTimeout = 4;

template <int D>
struct TLay {
    static constexpr bool kPair = D <= 128;                   // two row tiles a CTA
    static constexpr int NQ = kPair ? 2 : 1;
    static constexpr int RT = NQ * kRows;
    static constexpr int kUnit = D == 64 ? kBox : 2 * kBox;   // 128 positions x min(D, 128)
    static constexpr int UPT = D == 256 ? 2 : 1;              // units of a tile of keys or values
    static constexpr int NU = D == 64 ? 8 : 5;
    static constexpr int q = 0;
    static constexpr int ring = NQ * (D / 64) * kBox;
    static constexpr int bars = ring + NU * kUnit;
    static constexpr int kBars = 2 * NU + 2 + 2 + 2 + 8 + 1;
    static constexpr int misc = bars + kBars * 8;             // tensor-memory address, abort flag
    static constexpr int refs = misc + 8;                     // [128] references
    static constexpr int total = refs + 128 * 4;
};
static_assert(TLay<64>::total + 1024 <= kSmemMax && TLay<128>::total + 1024 <= kSmemMax && TLay<256>::total + 1024 <= kSmemMax,
              "shared memory");
// tensor memory: S of the streams at columns 0 and 128, O from 256 on
constexpr uint32_t kTmemCols = 512;

struct TileParams {
    CUtensorMap tk, tv;
    KvCall c;
    int ntile;     // row tiles (CTAs' worth) of a head
    int nsplit;
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
// Bounded wait on an mbarrier phase; gives up when the CTA's abort flag is
// set, or sets it (and the error word) when the time runs out.
__device__ __noinline__ bool bar_wait_slow(uint32_t b, unsigned parity, volatile int *abort, long long timeout_ns, int *err)
{
    const unsigned long long t0 = gtime();
#pragma unroll 1
    for (;;) {
        if (bar_test(b, parity)) return true;
        if (*abort) return false;
        if ((long long)(gtime() - t0) > timeout_ns) {
            *abort = 1;
            atomicOr(err, kErrTimeout);
            return false;
        }
    }
}
__device__ __forceinline__ bool bar_wait(uint32_t b, unsigned parity, volatile int *abort, const KvCall &c)
{
    return bar_test(b, parity) || bar_wait_slow(b, parity, abort, c.timeout_ns, c.err);
}

// Shared-memory descriptors (tcgen05, version 1), 128-byte swizzle.  K-major:
// rows of 64 elements, 8-row groups 1024 bytes apart; 16 elements on are 32 bytes.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// MN-major: 64 elements of N in a row of 128 bytes, the next 64 a box further; rows are
// K, 8-row groups 1024 bytes apart; 16 of K on are 2048 bytes.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(kBox >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
// kind::f16, fp32 accumulator, M = 128; b_mn: B is MN-major.
template <bool F16>
__device__ __forceinline__ constexpr uint32_t idesc(int n, bool b_mn)
{
    return (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc)
{
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc)
{
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
                 "r"(a), "l"(b), "r"(id), "r"(acc)
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

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
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

// The order in which a tile's keys (or values) are loaded: as the steps first use them.
template <bool PAIR>
__device__ __forceinline__ int k_order(int t) { return PAIR ? 2 * t : t == 0 ? 0 : 2 * t - 1; }
template <bool PAIR>
__device__ __forceinline__ int v_order(int t, int nt) { return PAIR ? 2 * t + 1 : t == nt - 1 ? 2 * nt - 1 : 2 * t + 2; }

template <bool F16, int D, bool PREFIX>
__global__ void __launch_bounds__(kTThreads, 1) kv_tile_kernel(const __grid_constant__ TileParams tp)
{
    using L = TLay<D>;
    constexpr bool PAIR = L::kPair;
    constexpr int NU = L::NU, UPT = L::UPT;
    const KvCall &p = tp.c;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::bars), *empty = full + NU;
    uint64_t *s_full = empty + NU, *p_full = s_full + 2, *o_done = p_full + 2, *ref_rdy = o_done + 2, *all_done = ref_rdy + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::misc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *refs = reinterpret_cast<float *>(sm + L::refs);

    // which rows and positions: later row tiles, which see more, first
    int x = blockIdx.x;
    const int tile = tp.ntile - 1 - x % tp.ntile;
    x /= tp.ntile;
    const int z = x % tp.nsplit;
    x /= tp.nsplit;
    const int g = x % p.Hkv, b = x / p.Hkv;
    const int r0 = tile * L::RT;
    after_previous();
    // tiles of positions i0 .. i0 + nt - 1 of the list: the first nsink, then from kt_lo on
    int p0 = 0, cnt = p.M, kt_lo = 0, nsink = 0, nt = 0, i0 = 0, nvalid = INT_MAX;
    if (PREFIX) {
        nt = (p.P + kKeys - 1) / kKeys;
    } else {
        bool bad;
        cnt = rows_of(p, b, p0, bad);
        if (bad && tile == 0 && g == 0 && z == 0 && tid == 0) atomicOr(p.err, kKv8ErrRange);
        const int first = r0 / p.G, last = min((r0 + L::RT - 1) / p.G, cnt - 1);
        nvalid = p0 + cnt;
        if (first < cnt) {
            kt_lo = max(0, p0 + first - p.W + 1) / kKeys;
            nsink = min((p.S + kKeys - 1) / kKeys, kt_lo);
            nt = nsink + (p0 + last) / kKeys - kt_lo + 1;
        }
    }
    {
        const int each = (nt + tp.nsplit - 1) / tp.nsplit;
        i0 = min(nt, z * each);
        nt = min(nt - i0, each);
    }
    auto first_key = [&](int t) { return kKeys * (i0 + t < nsink ? i0 + t : kt_lo + i0 + t - nsink); };
    const long long rows = PREFIX ? (long long)p.B * p.M * p.G : (long long)p.M * p.G;   // of a head (and sequence)
    const bool parts = PREFIX || tp.nsplit > 1;
    const size_t part0 = ((size_t)z * p.Hkv + g) * ((size_t)p.B * p.M * p.G) + (PREFIX ? 0 : (size_t)b * p.M * p.G);
    uint16_t *const out = static_cast<uint16_t *>(p.o);
    if (nt == 0) {
        // nothing to see: zeros, or an empty part
        for (int i = tid; i < L::RT; i += kTThreads)
            if (parts && r0 + i < rows) *reinterpret_cast<float2 *>(p.tile_ml + (part0 + r0 + i) * 2) = make_float2(-INFINITY, 0.f);
        if (!parts)
            for (int i = tid; i < L::RT * (D / 8); i += kTThreads) {
                const int r = r0 + i / (D / 8), c = i % (D / 8);
                if (r < rows) {
                    const int m = r / p.G, h = r - m * p.G;
                    *reinterpret_cast<uint4 *>(out + (((size_t)b * p.M + m) * p.Hq + g * p.G + h) * D + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
                }
            }
        return;
    }
    const int nsteps = PAIR ? 2 * nt : nt;

    if (tid == 0) {
        for (int s = 0; s < NU; ++s) {
            bar_init(su32(&full[s]), 1);
            bar_init(su32(&empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(su32(&s_full[s]), 1);
            bar_init(su32(&p_full[s]), 4);
            bar_init(su32(&o_done[s]), 1);
        }
        for (int s = 0; s < 8; ++s) bar_init(su32(&ref_rdy[s]), 1);
        bar_init(su32(all_done), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)), "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;

    float l = 0.f, ref = -INFINITY;    // of the thread's row, as its stream knows them
    if (warp == 8) {
        // ---------------------------------------------------------------- loads
        if (lane == 0) {
            bool go = true;
            int n = 0;   // units issued
            auto load = [&](const CUtensorMap *map, int t) {
                const int key = first_key(t);
                for (int u = 0; u < UPT && go; ++u) {
                    const int s = n % NU, turn = n / NU;
                    if (turn > 0 && !bar_wait(su32(&empty[s]), (unsigned)(turn - 1) & 1u, abort_flag, p)) {
                        go = false;
                        return;
                    }
                    const uint32_t dst = su32(sm + L::ring + s * L::kUnit), fb = su32(&full[s]);
                    bar_expect(fb, L::kUnit);
#pragma unroll
                    for (int h = 0; h < L::kUnit / kBox; ++h) tma_load4(dst + h * kBox, map, 128 * u + 64 * h, key, g, PREFIX ? 0 : b, fb);
                    ++n;
                }
            };
            if (PAIR) {
                for (int t = 0; t < nt && go; ++t) {
                    load(&tp.tk, t);
                    if (go) load(&tp.tv, t);
                }
            } else {
                load(&tp.tk, 0);
                if (go && nt > 1) load(&tp.tk, 1);
                for (int t = 0; t < nt && go; ++t) {
                    load(&tp.tv, t);
                    if (go && t + 2 < nt) load(&tp.tk, t + 2);
                }
            }
            // every copy issued has landed before the CTA ends
            const unsigned long long t0 = gtime();
            for (int s = 0; s < NU && s < n; ++s) {
                const unsigned last = (unsigned)((n - 1 - s) / NU) & 1u;
                while (!bar_test(su32(&full[s]), last) && (long long)(gtime() - t0) <= p.timeout_ns) {}
            }
        }
        __syncwarp();
    } else {
        // q, packed: rows that are not there are zeros
        if (warp != 9) {
            constexpr int CH = D / 8;
            for (int i = tid; i < L::RT * CH; i += 256) {
                const int rr = i / CH, c = i % CH, r = r0 + rr;
                bool ok = r < rows;
                int bb = b, m = r / p.G;
                const int h = r - m * p.G;
                if (PREFIX) {
                    bb = m / p.M;
                    m -= bb * p.M;
                    int q0;
                    bool bad;
                    ok = ok && m < rows_of(p, bb, q0, bad);
                } else {
                    ok = ok && m < cnt;
                }
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (ok) v = __ldg(reinterpret_cast<const uint4 *>(p.q + bb * p.qb + m * p.qm + (long long)(g * p.G + h) * p.qh) + c);
                *reinterpret_cast<uint4 *>(sm + L::q + ((rr >> 7) * (D / 64) + (c >> 3)) * kBox + (rr & 127) * 128 +
                                           (((c & 7) ^ (rr & 7)) << 4)) = v;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        asm volatile("bar.sync 1, 288;" ::: "memory");   // q is there: softmax warps and the products' warp

        if (warp == 9) {
            // ---------------------------------------------------------- products
            bool go = true;
            const uint32_t id_s = idesc<F16>(kKeys, false), id_o = idesc<F16>(D < 128 ? D : 128, true);
            auto wait = [&](uint64_t *bar, int parity) {
                go = __all_sync(0xFFFFFFFFu, go && bar_wait(su32(bar), (unsigned)parity & 1u, abort_flag, p));
                fence_after();
            };
            auto scores = [&](int i) {
                const int xs = i & 1, t = PAIR ? i >> 1 : i, n0 = UPT * k_order<PAIR>(t);
#pragma unroll
                for (int u = 0; u < UPT; ++u) {
                    const int s = (n0 + u) % NU;
                    if (go) wait(&full[s], (n0 + u) / NU);
                    if (!go) return;
                    if (lane == 0) {
                        const uint32_t a0 = su32(sm + L::q + ((PAIR ? xs : 0) * (D / 64) + 2 * u) * kBox);
                        const uint32_t b0 = su32(sm + L::ring + s * L::kUnit);
#pragma unroll
                        for (int k = 0; k < (D < 128 ? D : 128) / 16; ++k) {
                            const uint32_t off = (uint32_t)((k >> 2) * kBox + (k & 3) * 32);
                            umma_ss(tmem + 128u * xs, desc_k(a0 + off), desc_k(b0 + off), id_s, (u | k) != 0 ? 1u : 0u);
                        }
                        if (!PAIR || xs == 1) umma_commit(su32(&empty[s]));
                    }
                }
                if (lane == 0) umma_commit(su32(&s_full[xs]));
                __syncwarp();
            };
            auto values = [&](int i) {
                const int xs = i & 1, t = PAIR ? i >> 1 : i, n0 = UPT * v_order<PAIR>(t, nt);
                const int gone = nvalid - first_key(t);   // positions from here on hold anything
                if (go) wait(&p_full[xs], i >> 1);
#pragma unroll
                for (int u = 0; u < UPT; ++u) {
                    const int s = (n0 + u) % NU;
                    if (go) wait(&full[s], (n0 + u) / NU);
                    if (!go) return;
                    uint8_t *unit = sm + L::ring + s * L::kUnit;
                    if (!PREFIX && gone < kKeys && (!PAIR || xs == 0)) {
                        for (int j = lane; j < (kKeys - gone) * 8; j += 32)
#pragma unroll
                            for (int h = 0; h < L::kUnit / kBox; ++h)
                                *reinterpret_cast<uint4 *>(unit + h * kBox + gone * 128 + j * 16) = make_uint4(0u, 0u, 0u, 0u);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                    if (lane == 0) {
                        const uint32_t o = tmem + 256u + (PAIR ? (uint32_t)(D * xs) : 128u * u);
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k)
                            umma_ts(o, tmem + 128u * xs + 8u * k, desc_mn(su32(unit) + 2048u * k), id_o, (t | k) != 0 ? 1u : 0u);
                        if (!PAIR || xs == 1) umma_commit(su32(&empty[s]));
                    }
                }
                if (lane == 0) umma_commit(su32(&o_done[xs]));
                __syncwarp();
            };
            scores(0);
            if (nsteps > 1) scores(1);
#pragma unroll 1
            for (int i = 0; i < nsteps && go; ++i) {
                values(i);
                if (go && i + 2 < nsteps) scores(i + 2);
            }
            // every product issued has finished before O is read or tensor memory freed
            if (lane == 0) {
                umma_commit(su32(all_done));
                const unsigned long long t0 = gtime();
                while (!bar_test(su32(all_done), 0u) && (long long)(gtime() - t0) <= p.timeout_ns) {}
            }
            __syncwarp();
        } else {
            // ----------------------------------------------------------- softmax
            const int xs = warp >> 2, w = warp & 3, r = r0 + (PAIR ? 128 * xs : 0) + (tid & 127);
            const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16), sc = lanes + 128u * xs;
            const uint32_t oc = lanes + 256u + (PAIR ? (uint32_t)(D * xs) : 0u);
            // positions t the row sees: t <= high and (t > low or t < S)
            int high, low, all_high, all_low;   // of the row; that all the warp group's rows have at least (at most)
            if (PREFIX) {
                high = all_high = p.P - 1;
                low = all_low = -1;
            } else {
                const int ra = r0 + (PAIR ? 128 * xs : 0);
                high = p0 + r / p.G;
                low = high - p.W;
                all_high = p0 + ra / p.G;
                all_low = p0 + (ra + kRows - 1) / p.G - p.W;
            }
            const float c = p.c;
            bool ok = true;
#pragma unroll 1
            for (int i = xs; i < nsteps; i += 2) {
                const int t = PAIR ? i >> 1 : i, key = first_key(t);
                ok = bar_wait(su32(&s_full[xs]), (unsigned)(i >> 1) & 1u, abort_flag, p);
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
                fence_after();
                uint32_t s[kKeys];
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld32(sc + 32u * k, s + 32 * k);
                tmem_wait_ld();
                // a tile that some row does not see all of
                if (key + kKeys - 1 > all_high || (key <= all_low && key + kKeys > p.S)) {
                    const int a = high - key, lo = low - key, f = p.S - key;
#pragma unroll
                    for (int k = 0; k < kKeys; ++k)
                        if (!(k <= a && (k > lo || k < f))) s[k] = 0xFF800000u;
                }
                float mx[4] = {__uint_as_float(s[0]), __uint_as_float(s[1]), __uint_as_float(s[2]), __uint_as_float(s[3])};
#pragma unroll
                for (int k = 4; k < kKeys; k += 4)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mx[j] = fmaxf(mx[j], __uint_as_float(s[k + j]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                float was = ref;
                if (!PAIR && i > 0) {   // the reference, from the stream that has the tile before
                    ok = bar_wait(su32(&ref_rdy[4 * (xs ^ 1) + w]), (unsigned)((i - 1) >> 1) & 1u, abort_flag, p);
                    if (!__all_sync(0xFFFFFFFFu, ok)) break;
                    was = refs[tid & 127];
                }
                const bool raise = top > was + 8.f;
                const float now = raise ? top : was;
                if (!PAIR) {
                    refs[tid & 127] = now;
                    __syncwarp();
                    if (lane == 0) bar_arrive(su32(&ref_rdy[4 * xs + w]));
                }
                if (now != ref) l *= ref == -INFINITY ? 0.f : ex2(ref - now);
                ref = now;
                if (__any_sync(0xFFFFFFFFu, raise) && t > 0) {
                    // O, which has the tiles up to the one before, in the new reference's units
                    const int before = PAIR ? i - 2 : i - 1;
                    ok = bar_wait(su32(&o_done[PAIR ? xs : xs ^ 1]), (unsigned)(before >> 1) & 1u, abort_flag, p);
                    if (!__all_sync(0xFFFFFFFFu, ok)) break;
                    fence_after();
                    const float f = raise ? ex2(was - now) : 1.f;
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
                const float sub = ref == -INFINITY ? 0.f : ref;
                float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t pk[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float e0 = ex2(fmaf(__uint_as_float(s[32 * k + 2 * j]), c, -sub));
                        const float e1 = ex2(fmaf(__uint_as_float(s[32 * k + 2 * j + 1]), c, -sub));
                        add[(2 * j) & 3] += e0;
                        add[(2 * j + 1) & 3] += e1;
                        pk[j] = pack2<F16>(e0, e1);
                    }
                    tmem_st16(sc + 16u * k, pk);
                }
                l += (add[0] + add[1]) + (add[2] + add[3]);
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(su32(&p_full[xs]));
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    float *lsum = reinterpret_cast<float *>(sm + L::ring), *lref = lsum + 256;   // the ring is done with
    if (!PAIR) {
        if (warp < 8) {
            lsum[tid] = l;
            lref[tid] = ref;
        }
        __syncthreads();
    }
    if (warp < 8 && *abort_flag == 0) {
        // --------------------------------------------------------------- outputs
        // thread = row; with one row tile a CTA the warp groups take half of the columns each
        const int xs = warp >> 2, w = warp & 3, r = r0 + (PAIR ? 128 * xs : 0) + (tid & 127);
        constexpr int NC = PAIR ? D : 128;
        const int col0 = PAIR ? 0 : 128 * xs;
        const uint32_t oc = tmem + ((uint32_t)(32 * w) << 16) + 256u + (PAIR ? (uint32_t)(D * xs) : (uint32_t)col0);
        if (!PAIR) {
            ref = refs[tid & 127];
            l = 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float rk = lref[128 * k + (tid & 127)];
                if (rk != -INFINITY) l += lsum[128 * k + (tid & 127)] * ex2(rk - ref);
            }
        }
        const int m = r / p.G, h = r - m * p.G;   // windows only
        const float inv = parts ? 1.f : l != 0.f ? 1.f / l : 0.f;
        const bool live = PREFIX || m < cnt;
#pragma unroll 1
        for (int k = 0; k < NC; k += 32) {
            uint32_t o[32];
            tmem_ld32(oc + k, o);
            tmem_wait_ld();
            if (r >= rows) continue;
            if (parts) {
                float4 *to = reinterpret_cast<float4 *>(p.tile_o + (part0 + r) * D + col0 + k);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    to[j] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]), __uint_as_float(o[4 * j + 2]),
                                        __uint_as_float(o[4 * j + 3]));
            } else {
                uint4 *to = reinterpret_cast<uint4 *>(out + (((size_t)b * p.M + m) * p.Hq + g * p.G + h) * D + col0 + k);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        v[q] = live ? pack2<F16>(__uint_as_float(o[8 * j + 2 * q]) * inv, __uint_as_float(o[8 * j + 2 * q + 1]) * inv) : 0u;
                    to[j] = make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
        }
        if (parts && r < rows && col0 == 0) *reinterpret_cast<float2 *>(p.tile_ml + (part0 + r) * 2) = make_float2(ref, l);
        fence_before();
    }
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

// [sequence][head][position][d], strides in elements; a dimension of one entry may have any.
bool map_of(CUtensorMap *map, const uint16_t *base, bool f16, int D, int T, int heads, int seqs, long long row, long long head,
            long long seq)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)T, (cuuint64_t)heads, (cuuint64_t)seqs};
    auto bytes = [&](long long s, int n) { return (cuuint64_t)(n > 1 ? s * 2 : D * 2); };
    const cuuint64_t strides[3] = {bytes(row, T), bytes(head, heads), bytes(seq, seqs)};
    const cuuint32_t box[4] = {64, (cuuint32_t)kKeys, 1, 1}, es[4] = {1, 1, 1, 1};
    return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(base), dims,
               strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int row_tile(int D) { return D == 256 ? kRows : 2 * kRows; }

}  // namespace

long long kv_row_tiles(long long rows, int D) { return (rows + row_tile(D) - 1) / row_tile(D); }

// Parts that the positions of each row tile are cut into: as many as fill the SMs in as few
// turns as possible.  `ctas` row tiles of all heads, `tiles` tiles of positions each.
int kv_tile_most(long long ctas) { return (int)std::max<long long>(1, 3 * 152 / ctas); }
int kv_tile_splits(long long ctas, long long tiles)
{
    int best = 1;
    double cost = 1e30;
    for (int s = 1; s <= kv_tile_most(ctas) && s <= tiles; ++s) {
        const double turns = (double)((ctas * s + 151) / 152), c = turns * ((double)((tiles + s - 1) / s) + 4.0) + 0.05 * s;
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
    const long long rows = (long long)c.M * c.G * (prefix ? c.B : 1);
    tp.nsplit = c.nsplit;
    const long long ntile = kv_row_tiles(rows, c.D), ctas = ntile * c.nsplit * c.Hkv * (prefix ? 1 : c.B);
    if (rows > INT_MAX - 1024 || ctas > INT_MAX) return MOE_ERR_UNSUPPORTED;
    tp.ntile = (int)ntile;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
    auto go = [&](auto kernel, int smem, std::once_flag *once) {
        std::call_once(once[dev], [&] {
            e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        });
        if (e == cudaSuccess) e = launch_after(kernel, dim3((unsigned)ctas), kTThreads, smem, 0, stream, tp);
    };
#define KV_TILE(F, D, P)                                                 \
    do {                                                                 \
        static std::once_flag once[64];                                  \
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
