// Decode attention over the 8-bit key/value cache (moe_kv8.cuh), for a batch
// of sequences of unequal lengths that live on the device.
//
// Row m of sequence b (m < its rows) is at position pos[b] + m:
//     s_t = scale q . k_t,  t <= pos[b] + m;  p = softmax(s);  o = sum_t p_t v_t
// and, on request, what weight each position received from the rows and query
// heads that share its key/value head:
//     acc[t] = decay acc_in[t] (t < pos[b], 0 from there on) + sum p_t.
//
// Split: the positions are cut into chunks whose size is a rule of the cache
// alone (kv8_chunk), so a row's result depends neither on the other rows nor
// on the other sequences.  A chunk yields, per query column (row and head of
// a key/value head's group), a reference exponent near its maximum, the sum
// of exp(s - reference), and the unnormalised output with a unit of its own;
// the merge kernel joins a row's chunks in an order that is fixed as well.
// What only other rows see (later positions of the same call) adds exact zeros.
#include <algorithm>
#include <climits>
#include <mutex>

#include "moe_kv8.cuh"

namespace moe {
namespace {

// n / d for n < 2^31 by a product: m = 2^32 (2^s - d) / d + 1 rounded down, s = log2 d rounded up.
struct Div {
    unsigned d, m, s;
    __device__ __forceinline__ int by(int &n) const   // n becomes the remainder
    {
        const unsigned q = (__umulhi((unsigned)n, m) + (unsigned)n) >> s;
        n -= (int)(q * d);
        return (int)q;
    }
};
Div div_of(unsigned d)
{
    Div v = {d, 0u, 0u};
    while ((1ull << v.s) < d) ++v.s;
    v.m = (unsigned)((((1ull << v.s) - d) << 32) / d + 1);
    return v;
}

struct AttnP {
    const void *q;
    long long qb, qm, qh;           // strides in elements: sequence, row, head
    const uint8_t *k, *v;
    const float *ks, *vs;
    const int32_t *pos, *counts;
    float *part_o, *part_ml, *part_e;     // chunks' results: output, (reference, sum), log2 of the output's unit
    float *fin, *sc;                      // joined (reference, 1 / sum); scores [B][Hkv][T_cap][C] or NULL
    void *o;                        // [B][M][Hq][D]
    const float *acc_in;
    float *acc;
    float decay, scale_log2;        // scale * log2(e)
    int *err, *counter;                   // counter: items taken beyond the first of each CTA, or NULL (in turn)
    Div by_pass, by_head, by_group;       // column passes, key/value heads, G
    int B, Hq, Hkv, G, M, C, T_cap, chunk, nchunk, blk_log, nblk, f16, qvec, o_type, streams;
};

// ------------------------------------------------------------------ chunks
// Persistent CTAs of 4 warps, three on an SM, take (sequence, chunk,
// key/value head, column pass) items, in turn or, in long runs, from a counter
// (8 x 128K of 256: 162 us against 168).  Within a chunk a warp works alone on
// tiles of 16 R positions (R = 256 / D: 4 KB of keys and 4 KB of values), every
// fourth one, through a ring of two tiles of its own that cp.async fills
// ahead, across items.  At the end of a chunk the warps join their outputs
// through the ring slots that their last tiles left, while the other slots and
// the other CTAs keep the loads going.  (Warps with chunks of their own, 12 to
// an SM, wrote four times the results and took 183 us where this took 163.)
//
// Bound, at 8 columns: the read of the cache (8 x 128K of 256: 1.07 GB of
// capacity, 85% of the copy bandwidth over the whole call) and, for int8,
// issuing the 665 instructions that 8 KB of codes take; below some 100 MB the
// launches, the first loads and the last chunks (8 us) weigh as much.
//
// Per 16 positions and 8 query columns, on m16n8k16 fp16 MMAs:
//     S^T [16 positions x 8] = K Q^T,   O^T [D x 8] += V^T P^T.
// Codes are exact in fp16; queries are, after a power of two per row, but for
// elements below 2^-26 of the row's largest.  The
// contraction index may be any order of the dimensions as long as both
// operands share it, so a lane's 16 loaded bytes of a key row are its elements
// of four MMAs as they come.  Values need pairs of positions in one register:
// byte permutes of two rows' words.  P^T's transpose is movmatrix.  The
// weights go in as two fp16 halves (22 bits; below for what is smaller): an
// fp32 output means something.
//
// 12 warps on an SM leave 168 registers a thread: the output of 8 columns of
// 256 dimensions (64), or 16 of 128 or 64, the queries in registers where they
// take 16 or less and in shared memory otherwise.  (16 columns of 128 or 64, and the
// change of units, spill up to 122 bytes.)  16 columns of 256 run with
// two CTAs on an SM and 255 registers: expanding the codes is most of the
// work, and it is done once per column pass.  A column's arithmetic is the
// same either way, to the bit.  (16 warps with 128 registers and slots of half
// a tile took 178 us where this takes 163.)
constexpr int kWarps = 4, kThreads = 32 * kWarps, kStages = 2;
constexpr int kTileBytes = 4096;                       // keys (or values) of a warp's tile
constexpr int kStageBytes = 2 * kTileBytes + 64;       // and the steps of its up to 4 groups of 16 positions
// A column's softmax is taken against m, a whole number that follows its
// maximum when that has grown by more than 2^8 (with 8 columns every other tile
// has a new maximum), and its output is held in a unit of its own: weights
// go into the product as exp2(s - m) * step * 2^off, where step is the
// values' of the position, and off a whole number.  Changes of either are
// exact.  off leaves the largest such weight of a tile between 2^-7 and
// 2^15: it is chosen anew, for 2^8, when a tile's falls outside.  A
// weight's two halves reach down to 2^-24, so it is off by 2^-22 of itself or 2^-18
// of the largest weight * step of its tile (2^-14 where the tile's steps differ, by up
// to the factor of 16 that is not looked into), whatever the steps of other tiles.
// (One unit for all columns, of the largest step so far, lost what came after a
// block of values 2^24 times larger, however little weight that block had.)
// Following it costs nothing to speak of where a tile's largest weight is within
// a few octaves of the first one's; with scores of a standard deviation of 7 (nats) and
// 16 columns a tile, most tiles move some column: 4 rows at 128K of 2 heads of 256 take
// 87 us for 73.
constexpr float kSlack = 8.f, kTop = 0x1p15f, kLow = 0x1p-7f;
constexpr int kAim = 8, kOffMin = -126, kOffMax = 120;  // the latter: values below 2^-100 need no finer unit
constexpr int kOutTop = 90;                             // a finer unit takes no output beyond 2^91

// Column tiles of 8 that a warp holds.  (Four for 32 columns and more, of 64 or
// 128 dimensions with 255 registers, took 0.9 to 1.7 times as long.)
__host__ __device__ constexpr int kv8_nt(int C) { return C <= 8 ? 1 : 2; }
template <int D, int NT>
struct Lay {
    static constexpr bool wide = NT * D >= 256;                      // queries in shared memory
    static constexpr int ctas = NT * D > 256 ? 2 : 3, NC = 8 * NT;
    static constexpr int ring = 0, ml = kWarps * kStages * kStageBytes, off = ml + kWarps * NC * 8, slot = off + kWarps * NC * 4,
                         items = slot + kWarps * 4, q = items + 4 * 32, qf = q + NT * D * 16, first = qf + NC * 4;
    static constexpr int total(int B) { return first + (3 * B + 1) * 4; }   // first[B + 1], then position and rows of each sequence
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint64_t policy)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
__device__ __forceinline__ void cp16z(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4z(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2 of a positive number, rounded down; -127 of one below 2^-126.
__device__ __forceinline__ int log2_of(float v) { return (int)(__float_as_uint(v) >> 23) - 127; }

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first of a chain: nothing to add to.
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t movtrans(uint32_t a)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Two rows' words: fp16 pairs (row 0, row 1) of dimensions 0 .. 3.
template <int FMT>
__device__ __forceinline__ void cross(uint32_t r0, uint32_t r1, uint32_t (&d)[4])
{
    if (FMT == MOE_KV8_INT8) {
        pairs<FMT>(__byte_perm(r0, r1, 0x5410), d[0], d[1]);
        pairs<FMT>(__byte_perm(r0, r1, 0x7632), d[2], d[3]);
    } else {
        pairs<FMT>(__byte_perm(r0, r1, 0x5140), d[0], d[1]);
        pairs<FMT>(__byte_perm(r0, r1, 0x7362), d[2], d[3]);
    }
}

// One (sequence, chunk, head, column pass); b < 0: no more.
struct __align__(16) Item {
    int b, g, cp, k0, k1, p0, rows, nth;   // positions k0 .. k1 - 1, the nth chunk
};

__device__ __forceinline__ Item decode_item(const AttnP &p, const int *first, int item, int total)
{
    Item it;
    if (item >= total) {
        it.b = -1;
        it.g = it.cp = it.k0 = it.k1 = it.p0 = it.rows = it.nth = 0;
        return it;
    }
    it.cp = item;
    item = p.by_pass.by(it.cp);
    it.g = item;
    item = p.by_head.by(it.g);
    int lo = 0, hi = p.B;              // first[lo] <= item < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= item) lo = mid;
        else hi = mid;
    }
    it.b = lo;
    it.p0 = first[p.B + 1 + lo];
    it.rows = first[2 * p.B + 1 + lo];
    it.nth = item - first[lo];
    it.k0 = it.nth * p.chunk;
    it.k1 = min(it.k0 + p.chunk, it.p0 + it.rows);
    return it;
}

// An item's queries into shared memory, each warp 512 / D of its columns: as
// the B operands of the k-steps, [column tile][two k-steps][lane], in the order
// of pairs(); scaled by a power of two (exactly; the row's largest to 2^12 ..
// 2^13, so that only elements 2^26 times smaller lose bits).
template <int FMT, int D, int NT>
__device__ __forceinline__ void stage_q(const AttnP &p, const Item &it, uint4 *qs, float *qf)
{
    constexpr int kLanes = D / 16, kCols = 32 / kLanes;              // lanes (16 elements each) of a column, columns at once
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = lane % kLanes;
#pragma unroll
    for (int u = 0; u < (8 * NT / kCols + kWarps - 1) / kWarps; ++u) {
        const int col = (u * kWarps + warp) * kCols + lane / kLanes, c = it.cp * 8 * NT + col;
        if ((u * kWarps + warp) * kCols >= 8 * NT) break;
        int h = c;
        const int m = p.by_group.by(h);
        const bool in = c < p.C && m < it.rows;
        const uint16_t *src = static_cast<const uint16_t *>(p.q) + it.b * p.qb + m * p.qm + (it.g * p.G + h) * p.qh + 16 * e0;
        uint16_t raw[16];
        if (p.qvec) {
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4 *>(raw) = in ? __ldg(reinterpret_cast<const uint4 *>(src)) : zero;
            *reinterpret_cast<uint4 *>(raw + 8) = in ? __ldg(reinterpret_cast<const uint4 *>(src) + 1) : zero;
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) raw[j] = in ? __ldg(src + j) : (uint16_t)0;
        }
        float v[16], a = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            v[j] = p.f16 ? __half2float(__ushort_as_half(raw[j])) : __uint_as_float((uint32_t)raw[j] << 16);
            a = fmaxf(a, fabsf(v[j]));
        }
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
        const int e = (int)(__float_as_uint(a) >> 23) - 127;
        const bool odd = a == 0.f || e == 128;                       // zero or infinite: as it is
        const int up = odd ? 0 : max(-126, min(126, 12 - e));
        const float f = pow2f(up);
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int x = FMT == MOE_KV8_INT8 ? 4 * (j >> 1) + (j & 1) : 2 * j, y = FMT == MOE_KV8_INT8 ? x + 2 : x + 1;
            const __half2 t = __floats2half2_rn(v[x] * f, v[y] * f);
            w[j] = *reinterpret_cast<const uint32_t *>(&t);
        }
        // elements 64 i + 16 t ..: k-steps 4 i .. 4 i + 3 of lane (column, t)
        uint4 *dst = qs + ((col / 8 * (D / 16) + 4 * (e0 / 4)) / 2) * 32 + col % 8 * 4 + e0 % 4;
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[32] = make_uint4(w[4], w[5], w[6], w[7]);
        if (e0 == 0) qf[col] = __fmul_rn(p.scale_log2, pow2f(-up));
    }
}

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(kThreads, Lay<D, NT>::ctas) kv8_chunk_kernel(const AttnP p)
{
    using L = Lay<D, NT>;
    constexpr int R = 256 / D, TK = 16 * R, KS = D / 16, NC = 8 * NT;   // KS: k-steps of S, m-tiles of O
    extern __shared__ __align__(128) uint8_t sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
    int *first = reinterpret_cast<int *>(sm + L::first);
    Item *items = reinterpret_cast<Item *>(sm + L::items);          // the nth in slot n mod 4
    float2 *red_ml = reinterpret_cast<float2 *>(sm + L::ml);
    float *red_off = reinterpret_cast<float *>(sm + L::off);
    int *red_slot = reinterpret_cast<int *>(sm + L::slot);
    const int passes = (p.C + NC - 1) / NC;

    after_previous();
    int claim = 0;                     // thread 0: the item after next
    if (tid == 0) claim = gridDim.x + (p.counter ? atomicAdd(p.counter, 1) : (int)blockIdx.x);
    // chunks before each sequence's
    for (int b = tid; b < p.B; b += kThreads) {
        int p0;
        bool bad;
        const int rows = kv8_rows(p.pos, p.counts, b, p.M, p.T_cap, p0, bad);
        if (bad && blockIdx.x == 0) atomicOr(p.err, kKv8ErrRange);
        first[b + 1] = rows > 0 ? (p0 + rows + p.chunk - 1) / p.chunk : 0;
        first[p.B + 1 + b] = p0;
        first[2 * p.B + 1 + b] = rows;
    }
    __syncthreads();
    if (warp == 0) {
        int before = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            int v = b0 + lane < p.B ? first[b0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
                if (lane >= o) v += u;
            }
            if (b0 + lane < p.B) first[b0 + lane + 1] = before + v;
            before += __shfl_sync(0xFFFFFFFFu, v, 31);
        }
        if (lane == 0) first[0] = 0;
    }
    __syncthreads();
    const int total = first[p.B] * p.Hkv * passes;
    if ((int)blockIdx.x >= total) return;
    if (warp == 0) {
        const int second = __shfl_sync(0xFFFFFFFFu, claim, 0);
        if (lane < 2) items[lane] = decode_item(p, first, lane ? second : (int)blockIdx.x, total);
    }
    uint4 *const qs = reinterpret_cast<uint4 *>(sm + L::q);
    float *const qf = reinterpret_cast<float *>(sm + L::qf);
    __syncthreads();

    uint8_t *ring = sm + L::ring + warp * kStages * kStageBytes;
    const uint32_t ring_u = smem_u32(ring);

    // The load cursor runs up to two tiles ahead of the compute cursor, and
    // up to one item.  A lane's i-th 16 bytes of a tile are row lr + i 512 /
    // D, chunk lc; chunks are swapped within a row so that the reads below hit
    // every bank once.
    const int lr = lane / (D / 16), lc = lane % (D / 16);
    const uint32_t k_lane = lr * D + (D == 64 ? lc : lc ^ ((lr & 1) << 2)) * 16;
    constexpr int VX = D == 256 ? 4 : D == 128 ? 2 : 1;   // the values' swap depends on i mod VX
    uint32_t v_lane[VX];
#pragma unroll
    for (int i = 0; i < VX; ++i) v_lane[i] = lr * D + (lc ^ ((lr + i * (512 / D)) & (D == 64 ? 2 : 6))) * 16;
    // a cache that L2 cannot keep leaves it to the chunks' results
    uint64_t policy;
    if (p.streams) asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    else asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    int nth = 0, ld_nth = -1, ld_t = 0, ld_k1 = 0, ld_stage = 0, free_slots = kStages;
    const uint8_t *ld_k = nullptr, *ld_v = nullptr;
    const float *ld_s = nullptr;
    bool ld_more = true;
    auto fill = [&]() {
        while (free_slots > 0) {
            while (ld_t >= ld_k1) {
                if (ld_nth > nth || !ld_more) return;
                const Item x = items[++ld_nth & 3];
                ld_more = x.b >= 0;
                if (!ld_more) return;
                const size_t head = (size_t)x.b * p.Hkv + x.g;
                ld_t = x.k0 + warp * TK;
                ld_k1 = x.k1;
                ld_k = p.k + (head * p.T_cap + ld_t) * D + lane * 16;
                ld_v = p.v + (head * p.T_cap + ld_t) * D + lane * 16;
                ld_s = (lane & 1 ? p.vs : p.ks) + head * p.nblk;
            }
            const uint32_t dst = ring_u + ld_stage * kStageBytes;
            if (ld_t + TK <= ld_k1) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    cp16(dst + k_lane + i * 512, ld_k + i * 512, policy);
                    cp16(dst + kTileBytes + v_lane[i % VX] + i * 512, ld_v + i * 512, policy);
                }
            } else {
                // rows past the end are zeros, not what lies there
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool in = ld_t + lr + i * (512 / D) < ld_k1;
                    cp16z(dst + k_lane + i * 512, in ? ld_k + i * 512 : p.k, in);
                    cp16z(dst + kTileBytes + v_lane[i % VX] + i * 512, in ? ld_v + i * 512 : p.v, in);
                }
            }
            if (lane < 2 * R) {
                const int t = ld_t + 16 * (lane >> 1);
                const bool in = t < ld_k1;
                cp4z(dst + 2 * kTileBytes + lane * 4, in ? ld_s + (t >> p.blk_log) : ld_s, in);
            }
            cp_commit();
            ld_t += kWarps * TK;
            ld_k += kWarps * kTileBytes;
            ld_v += kWarps * kTileBytes;
            ld_stage ^= 1;
            --free_slots;
        }
    };
    static_assert(kStages == 2, "stages alternate");
    fill();
    stage_q<FMT, D, NT>(p, items[0], qs, qf);
    __syncthreads();

    // A lane's reads of a tile: chunk 4 i + t of key rows g and g + 8 (the
    // swap turns i even into i + 1 and back in odd rows), 16 (8) bytes of
    // value rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9.
    const int k_even = gq * D + tq * 16 + (D == 64 ? 0 : (gq & 1) * 64), k_odd = gq * D + tq * 16 - (D == 64 ? 0 : (gq & 1) * 64);
    const int v_at = 2 * tq * D + (D == 64 ? ((gq >> 1) ^ ((tq & 1) * 2)) * 16 + (gq & 1) * 8 : (gq ^ (2 * tq)) * 16);
    int stage = 0;
#pragma unroll 1
    for (;;) {
        const Item it = items[nth & 3];
        if (tid == 0) claim = p.counter ? gridDim.x + atomicAdd(p.counter, 1) : claim + gridDim.x;
        float f[NT][2], m[NT][2], l[NT][2], o[NT][KS][4];
        int off[NT][2];                // off in an exponent's place
        bool fresh = true;             // no tile yet: m = -inf, everything else 0
        uint32_t qr[L::wide ? 1 : NT][L::wide ? 1 : KS][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if constexpr (!L::wide) {
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    const uint4 x = qs[(n * KS + k) * 16 + lane];
                    qr[n][k][0] = x.x;
                    qr[n][k][1] = x.y;
                    qr[n][k + 1][0] = x.z;
                    qr[n][k + 1][1] = x.w;
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                f[n][c] = qf[8 * n + 2 * tq + c];
                m[n][c] = -INFINITY;
                l[n][c] = 0.f;
                off[n][c] = 0;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[n][k][c] = 0.f;
        }

#pragma unroll 1
        for (int t0 = it.k0 + warp * TK; t0 < it.k1; t0 += kWarps * TK) {
            if (free_slots == 0) cp_wait<1>();
            else cp_wait<0>();
            __syncwarp();
            const uint8_t *kt = ring + stage * kStageBytes;
            const float *steps = reinterpret_cast<const float *>(kt + 2 * kTileBytes);
            // ---- scores
            float s[R][NT][4];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                constexpr int kChains = D == 64 ? 1 : 2;           // of 4 to 8 MMAs that wait on one another
                float acc[NT][kChains][4];
                uint4 qw[NT];
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const uint8_t *src = kt + (i & 1 ? k_odd : k_even) + 16 * r * D + 64 * i;
                    const uint4 u = *reinterpret_cast<const uint4 *>(src);
                    const uint4 w = *reinterpret_cast<const uint4 *>(src + 8 * D);
                    const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (L::wide && !(j & 1)) {
#pragma unroll
                            for (int n = 0; n < NT; ++n) qw[n] = qs[(n * KS + 4 * i + j) * 16 + lane];
                        }
                        uint32_t a0, a1, a2, a3;
                        pairs<FMT>(uw[j], a0, a2);
                        pairs<FMT>(ww[j], a1, a3);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                        {
                            uint32_t b0, b1;
                            if constexpr (L::wide) {
                                b0 = j & 1 ? qw[n].z : qw[n].x;
                                b1 = j & 1 ? qw[n].w : qw[n].y;
                            } else {
                                b0 = qr[n][4 * i + j][0];
                                b1 = qr[n][4 * i + j][1];
                            }
                            if (4 * i + j < kChains) mma_first(acc[n][j % kChains], a0, a1, a2, a3, b0, b1);
                            else mma(acc[n][j % kChains], a0, a1, a2, a3, b0, b1);
                        }
                    }
                }
                const float ks = steps[2 * r];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        s[r][n][c] = __fmul_rn(kChains == 1 ? acc[n][0][c] : __fadd_rn(acc[n][0][c], acc[n][kChains - 1][c]),
                                               __fmul_rn(ks, f[n][c & 1]));
            }
            if (p.sc) {
                float *dst = p.sc + (((size_t)it.b * p.Hkv + it.g) * p.T_cap + t0 + gq) * p.C + it.cp * NC + 2 * tq;
                const int end = it.k1 - t0 - gq, cols = p.C - it.cp * NC - 2 * tq, step = 8 * p.C;
                const bool two = !(p.C & 1);                       // pairs are aligned, and whole
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int c = 0; c < 4; c += 2, dst += step)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (16 * r + 4 * c >= end || 8 * n >= cols) continue;
                            if (two) *reinterpret_cast<float2 *>(dst + 8 * n) = make_float2(s[r][n][c], s[r][n][c + 1]);
                            else {
                                dst[8 * n] = s[r][n][c];
                                if (8 * n + 1 < cols) dst[8 * n + 1] = s[r][n][c + 1];
                            }
                        }
            }
            // ---- positions that a row does not see (the call's own rows, and the end)
            if (t0 + TK > it.p0 + 1) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        int col = it.cp * NC + 8 * n + 2 * tq + c;
                        const int see = min(it.p0 + 1 + p.by_group.by(col), it.k1);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            if (t0 + 16 * r + gq >= see) s[r][n][c] = -INFINITY;
                            if (t0 + 16 * r + gq + 8 >= see) s[r][n][c + 2] = -INFINITY;
                        }
                    }
            }
            // ---- reference exponents and units
            float most = steps[1], least = steps[1];
#pragma unroll
            for (int r = 1; r < R; ++r) {
                most = fmaxf(most, steps[2 * r + 1]);
                least = fminf(least, steps[2 * r + 1]);
            }
            const bool near = R == 1 || most <= 16.f * least, whole = R == 1 || (near && t0 + TK <= it.p0 + 1);
            auto all = [](float v) {                               // over a column's lanes
                v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
                v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
                return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
            };
            // Where a column sees the whole tile and the steps are within a factor of
            // 16, its largest weight is taken to be that of its largest score and the largest step.
            float x[NT][2];                                        // the largest score
            bool move = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float a = fmaxf(s[0][n][c], s[0][n][c + 2]);
#pragma unroll
                    for (int r = 1; r < R; ++r) a = fmaxf(a, fmaxf(s[r][n][c], s[r][n][c + 2]));
                    x[n][c] = all(a);
                    // the difference: a sum would round past x where scores are 16 apart
                    const float d = __fsub_rn(x[n][c], m[n][c]), top = __fmul_rn(ex2(d), __fmul_rn(most, __int_as_float(off[n][c] + 0x3F800000)));
                    move |= d > kSlack || top >= kTop || top < kLow;
                }
            if (fresh && whole) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        m[n][c] = ceilf(x[n][c]);
                        const int e = log2_of(__fmul_rn(ex2(__fsub_rn(x[n][c], m[n][c])), most));
                        off[n][c] = max(kOffMin, min(kOffMax, kAim - e)) << 23;
                    }
                fresh = false;
            } else if (!whole || __any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    int by[2];                                     // the output's change, as a power of two
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        int want = off[n][c] >> 23;                // of the same unit under the new m
                        const bool first = m[n][c] == -INFINITY;   // nothing there: any unit
                        if (__fsub_rn(x[n][c], m[n][c]) > kSlack) {
                            const float mn = ceilf(x[n][c]);
                            const int up = (int)fminf(__fsub_rn(mn, m[n][c]), 1024.f);
                            l[n][c] = up > 126 ? 0.f : __fmul_rn(l[n][c], pow2f(-up));
                            want += up;
                            m[n][c] = mn;
                        }
                        // the largest exp2(s - m) * step (of up to 2^130: in units of 2^8), and
                        // the largest step that the column sees
                        float top = __fmul_rn(ex2(__fsub_rn(x[n][c], m[n][c])), most * 0x1p-8f), big = most;
                        if (R > 1 && !whole) {
                            int col = it.cp * NC + 8 * n + 2 * tq + c;
                            float a = 0.f, b = 0.f;
#pragma unroll
                            for (int r = 0; r < R; ++r) {
                                const float y = fmaxf(s[r][n][c], s[r][n][c + 2]);
                                a = fmaxf(a, __fmul_rn(ex2(__fsub_rn(y, m[n][c])), steps[2 * r + 1] * 0x1p-8f));
                                if (y > -INFINITY) b = fmaxf(b, steps[2 * r + 1]);
                            }
                            a = all(a);
                            b = all(b);
                            if (!near || t0 + TK > it.p0 + 1 + p.by_group.by(col)) {
                                top = a;
                                big = b;
                            }
                        }
                        // as above, so that a column does not depend on who else moves
                        const int e = log2_of(top) + 8;
                        int next = want;
                        if (e > -119) {                            // else a tile of no weight
                            if (e + want > 14 || e + want < -7) next = kAim - e;
                            next = min(next, 127 - log2_of(big));  // 2^off step is finite
                        }
                        next = max(kOffMin, min(kOffMax, next));
                        by[c] = first ? 0 : next - want;
                        off[n][c] = next << 23;
                    }
                    if (!__any_sync(0xFFFFFFFFu, (by[0] | by[1]) != 0)) continue;
                    if (__any_sync(0xFFFFFFFFu, max(by[0], by[1]) > 0)) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float a = 0.f;
#pragma unroll
                            for (int k = 0; k < KS; ++k) a = fmaxf(a, fmaxf(fabsf(o[n][k][c]), fabsf(o[n][k][c + 2])));
                            a = all(a);
                            if (by[c] > 0 && a > 0.f) {            // where there is nothing yet, any unit
                                const int cut = min(by[c], max(0, min(127, kOutTop - log2_of(a))));
                                off[n][c] -= (by[c] - cut) << 23;
                                by[c] = cut;
                            }
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float al = by[c] < -126 ? 0.f : pow2f(min(by[c], 127));
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            o[n][k][c] = __fmul_rn(o[n][k][c], al);
                            o[n][k][c + 2] = __fmul_rn(o[n][k][c + 2], al);
                        }
                    }
                }
                fresh = false;
            }
            // ---- weights, their sums, and the output
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int vstep = __float_as_int(steps[2 * r + 1]);
                uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    // step * 2^off by adding exponents; below 2^-126 and where it is too
                    // large (of positions that are not seen) zero
                    float unit[2], w[4];
#pragma unroll
                    for (int c = 0; c < 2; ++c) unit[c] = __int_as_float(__viaddmin_s32_relu(vstep, off[n][c], 0x7F000000));
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float base = m[n][c & 1] == -INFINITY ? 0.f : m[n][c & 1];
                        const float x = ex2(__fsub_rn(s[r][n][c], base));
                        l[n][c & 1] = __fadd_rn(l[n][c & 1], x);
                        w[c] = __fmul_rn(x, unit[c & 1]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const __half2 hi = __floats2half2_rn(w[2 * h], w[2 * h + 1]);
                        const float2 back = __half22float2(hi);
                        const __half2 lo = __floats2half2_rn(__fsub_rn(w[2 * h], back.x), __fsub_rn(w[2 * h + 1], back.y));
                        ph[n][h] = movtrans(*reinterpret_cast<const uint32_t *>(&hi));
                        pl[n][h] = movtrans(*reinterpret_cast<const uint32_t *>(&lo));
                    }
                }
                constexpr int VW = D >= 128 ? 4 : 2;             // words of a row per load
#pragma unroll
                for (int h = 0; h < (D + 127) / 128; ++h) {
                    uint32_t v[4][VW];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint8_t *src = kt + v_at + kTileBytes + (16 * r + (x & 1) + 8 * (x >> 1)) * D + 128 * h;
                        if (D >= 128) {
                            const uint4 u = *reinterpret_cast<const uint4 *>(src);
                            v[x][0] = u.x;
                            v[x][1] = u.y;
                            v[x][VW - 2] = u.z;
                            v[x][VW - 1] = u.w;
                        } else {
                            const uint2 u = *reinterpret_cast<const uint2 *>(src);
                            v[x][0] = u.x;
                            v[x][1] = u.y;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        uint32_t a[4], b[4];
                        cross<FMT>(v[0][w], v[1][w], a);
                        cross<FMT>(v[2][w], v[3][w], b);
                        const int k = (VW * h + w) * 2;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma(o[n][k], a[0], a[1], b[0], b[1], ph[n][0], ph[n][1]);
                            mma(o[n][k + 1], a[2], a[3], b[2], b[3], ph[n][0], ph[n][1]);
                            mma(o[n][k], a[0], a[1], b[0], b[1], pl[n][0], pl[n][1]);
                            mma(o[n][k + 1], a[2], a[3], b[2], b[3], pl[n][0], pl[n][1]);
                        }
                    }
                }
            }
            __syncwarp();                                          // the tile is read before its slot is filled again
            ++free_slots;
            stage ^= 1;
            if (t0 + kWarps * TK < it.k1) fill();                  // the last tile's slot serves the join first
        }

        // ---- the chunk's result from the warps' that had a tile
        const int having = min(kWarps, (it.k1 - it.k0 + TK - 1) / TK), cols = min(NC, p.C - it.cp * NC);
        const size_t slot = (((size_t)it.b * p.nchunk + it.nth) * p.Hkv + it.g) * passes + it.cp;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x = l[n][c];
                x = __fadd_rn(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                x = __fadd_rn(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                x = __fadd_rn(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                if (gq == 0) {
                    red_ml[warp * NC + 8 * n + 2 * tq + c] = make_float2(m[n][c], x);
                    red_off[warp * NC + 8 * n + 2 * tq + c] = (float)(off[n][c] >> 23);
                }
            }
        if (lane == 0) red_slot[warp] = stage ^ 1;
        constexpr int kAll = NT * KS, kRound = kAll < 16 ? kAll : 16;    // m-tiles, and of them a slot's worth
#pragma unroll
        for (int h = 0; h < kAll / kRound; ++h) {
            if (warp < having) {
                float4 *dst = reinterpret_cast<float4 *>(ring + (stage ^ 1) * kStageBytes) + lane;
#pragma unroll
                for (int x = 0; x < kRound; ++x) {
                    const float *v = o[(h * kRound + x) / KS][(h * kRound + x) % KS];
                    dst[x * 32] = make_float4(v[0], v[1], v[2], v[3]);
                }
            }
            __syncthreads();
            if (h == 0) {                                          // every warp is done with the item and its queries
                if (tid == 0) items[(nth + 2) & 3] = decode_item(p, first, claim, total);
                const Item x = items[(nth + 1) & 3];
                if (x.b >= 0) stage_q<FMT, D, NT>(p, x, qs, qf);
            }
            constexpr int kShare = kRound / kWarps;                // m-tiles a warp adds up, of one column tile
            const int x0 = h * kRound + warp * kShare, n = x0 / KS;
            float cf[kWarps][2], mx[2] = {-INFINITY, -INFINITY}, top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
            const float4 *src[kWarps];
#pragma unroll
            for (int v = 0; v < kWarps; ++v)
                if (v < having) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) mx[c] = fmaxf(mx[c], red_ml[v * NC + 8 * n + 2 * tq + c].x);
                }
            // in the coarsest unit of the warps'
#pragma unroll
            for (int v = 0; v < kWarps; ++v)
                if (v < having) {
                    src[v] = reinterpret_cast<const float4 *>(sm + L::ring + (v * kStages + red_slot[v]) * kStageBytes) +
                             (x0 - h * kRound) * 32 + lane;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float2 x = red_ml[v * NC + 8 * n + 2 * tq + c];
                        const float d = x.x == -INFINITY ? x.x : __fsub_rn(x.x, mx[c]);
                        sum[c] = __fmaf_rn(ex2(d), x.y, sum[c]);
                        cf[v][c] = __fsub_rn(d, red_off[v * NC + 8 * n + 2 * tq + c]);
                        top[c] = fmaxf(top[c], cf[v][c]);
                    }
                }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (top[c] == -INFINITY) top[c] = 0.f;             // no weight at all
#pragma unroll
                for (int v = 0; v < kWarps; ++v)
                    if (v < having) cf[v][c] = ex2(__fsub_rn(cf[v][c], top[c]));
            }
            if (8 * n + 2 * tq < cols) {
                if (x0 % KS == 0 && gq == 0) {
                    *reinterpret_cast<float4 *>(p.part_ml + (slot * NC + 8 * n + 2 * tq) * 2) = make_float4(mx[0], sum[0], mx[1], sum[1]);
                    *reinterpret_cast<float2 *>(p.part_e + slot * NC + 8 * n + 2 * tq) = make_float2(top[0], top[1]);
                }
                float4 *dst = reinterpret_cast<float4 *>(p.part_o) + (slot * kAll + x0) * 32 + lane;
#pragma unroll
                for (int x = 0; x < kShare; ++x) {
                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int v = 0; v < kWarps; ++v)
                        if (v < having) {
                            const float4 y = src[v][x * 32];
                            a.x = __fmaf_rn(cf[v][0], y.x, a.x);
                            a.y = __fmaf_rn(cf[v][1], y.y, a.y);
                            a.z = __fmaf_rn(cf[v][0], y.z, a.z);
                            a.w = __fmaf_rn(cf[v][1], y.w, a.w);
                        }
                    dst[x * 32] = a;
                }
            }
            __syncthreads();
        }
        if (items[++nth & 3].b < 0) break;
        fill();
    }
    cp_wait<0>();
}

// A mean of values of up to 2^128: bf16 and fp32 keep to finite numbers.
__device__ __forceinline__ void store_out(void *o, int type, size_t i, float v)
{
    if (type == MOE_BF16) static_cast<uint16_t *>(o)[i] = (uint16_t)bf16_pair(v, 0.f);
    else if (type == MOE_F16) static_cast<__half *>(o)[i] = __float2half_rn(v);
    else static_cast<float *>(o)[i] = fabsf(v) == INFINITY ? copysignf(__uint_as_float(0x7F7FFFFFu), v) : v;
}

// ------------------------------------------------------------------- merge
// Joins the chunks of a (sequence, head, column tile): a CTA per two m-tiles
// (4 dimensions for each group of 4 lanes) and share of the chunks, the shares
// of a cluster joined through its first CTA's shared memory.  Within a CTA
// 4 warps per m-tile take every 4th chunk, so the order of additions depends
// on the number of chunks and the cache's shape alone; chunks that a column does not see
// (another row's) add exact zeros.  Bound by latency: up to 304 CTAs load all
// their chunks at once, U in flight (one of 128K of 2 heads of 256: 32.9 us a
// call with U = 4, 31.8 with 8); more CTAs take little of the registers, so as to
// run beside the chunks that end last (32 of up to 16K of 8 heads of 128: 106 us
// with 4, 104 with 2).  U changes no addition's place.
constexpr int kMergeThreads = 256, kMergeShares = 8;

// A column pair's share: references, sums, log2 of the outputs' units, outputs.
struct Share {
    float m[2], l[2], e[2];
    float4 o;

    __device__ __forceinline__ float4 ml() const { return make_float4(m[0], l[0], m[1], l[1]); }
    __device__ __forceinline__ float2 unit() const { return make_float2(e[0], e[1]); }
    // += another; reference -inf: nothing.  Units keep what they hold: the
    // output is a sum of its terms in the coarser of two.
    __device__ __forceinline__ void join(const float4 &ml, const float2 &unit, const float4 &x)
    {
        const float bm[2] = {ml.x, ml.z}, bl[2] = {ml.y, ml.w}, be[2] = {unit.x, unit.y};
        float fa[2], fb[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float r = fmaxf(m[c], bm[c]), base = r == -INFINITY ? 0.f : r, da = m[c] - base, db = bm[c] - base;
            l[c] = l[c] * ex2(da) + ex2(db) * bl[c];
            m[c] = r;
            const float ea = da + e[c], eb = db + be[c], top = fmaxf(ea, eb);
            e[c] = top == -INFINITY ? 0.f : top;
            fa[c] = ex2(ea - e[c]);
            fb[c] = ex2(eb - e[c]);
        }
        o.x = o.x * fa[0] + fb[0] * x.x;
        o.y = o.y * fa[1] + fb[1] * x.y;
        o.z = o.z * fa[0] + fb[0] * x.z;
        o.w = o.w * fa[1] + fb[1] * x.w;
    }
};

template <int U>
__global__ void __launch_bounds__(kMergeThreads) kv8_merge_kernel(const AttnP p, int D, int shares)
{
    __shared__ float4 so[8][32], sml[8][32];
    __shared__ float2 se[8][32];
    __shared__ float4 co[kMergeShares][64], cml[kMergeShares][64];   // the shares' results, in the cluster's first CTA
    __shared__ float2 ce[kMergeShares][64];
    place_next();
    if (shares > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
    const int KS = D / 16, nt = kv8_nt(p.C), NC = 8 * nt, passes = (p.C + NC - 1) / NC;
    // blockIdx.x: share, then pair of m-tiles, then column tile
    const int share = blockIdx.x % shares, pair = blockIdx.x / shares % (KS / 2), ct = blockIdx.x / shares / (KS / 2);
    const int g = blockIdx.y, b = blockIdx.z, k = 2 * pair + (warp & 1);
    int p0;
    bool bad;
    const int rows = kv8_rows(p.pos, p.counts, b, p.M, p.T_cap, p0, bad);
    const int n = rows > 0 ? p0 + rows : 0, nch = (n + p.chunk - 1) / p.chunk;
    wait_for_previous();                                             // the chunks' results
    Share a = {{-INFINITY, -INFINITY}, {0.f, 0.f}, {0.f, 0.f}, make_float4(0.f, 0.f, 0.f, 0.f)};
    const bool on = 8 * ct + 2 * tq < p.C;
    const int stride = 4 * shares;
    auto slot = [&](int j) { return (((size_t)b * p.nchunk + j) * p.Hkv + g) * passes + ct / nt; };
    if (on) {
        for (int j = share * 4 + (warp >> 1); j < nch; j += U * stride) {
            float4 ml[U], x[U];
            float2 e[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int ju = j + u * stride;
                ml[u] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
                x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                e[u] = make_float2(0.f, 0.f);
                if (ju < nch) {
                    const size_t s = slot(ju);
                    ml[u] = __ldcg(reinterpret_cast<const float4 *>(p.part_ml + (s * NC + 8 * (ct % nt) + 2 * tq) * 2));
                    e[u] = __ldcg(reinterpret_cast<const float2 *>(p.part_e + s * NC + 8 * (ct % nt) + 2 * tq));
                    x[u] = __ldcg(reinterpret_cast<const float4 *>(p.part_o) + ((s * nt + ct % nt) * KS + k) * 32 + lane);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j + u * stride < nch) a.join(ml[u], e[u], x[u]);
        }
    }
    so[warp][lane] = a.o;
    sml[warp][lane] = a.ml();
    se[warp][lane] = a.unit();
    __syncthreads();
    if (warp < 2) {
#pragma unroll
        for (int w = 1; w < 4; ++w) a.join(sml[warp + 2 * w][lane], se[warp + 2 * w][lane], so[warp + 2 * w][lane]);
    }
    if (shares > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // the first CTA has started: its shared memory is there
        if (warp < 2) {
            // to the first CTA of the cluster
            uint32_t dst;
            const float4 ml = a.ml(), o = a.o;
            const float2 e = a.unit();
            asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(dst) : "r"(smem_u32(&co[share][warp * 32 + lane])));
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "f"(o.x), "f"(o.y), "f"(o.z), "f"(o.w) : "memory");
            asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(dst) : "r"(smem_u32(&cml[share][warp * 32 + lane])));
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "f"(ml.x), "f"(ml.y), "f"(ml.z), "f"(ml.w) : "memory");
            asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(dst) : "r"(smem_u32(&ce[share][warp * 32 + lane])));
            asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dst), "f"(e.x), "f"(e.y) : "memory");
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (share != 0) return;
        if (warp < 2)
            for (int s = 1; s < shares; ++s) a.join(cml[s][warp * 32 + lane], ce[s][warp * 32 + lane], co[s][warp * 32 + lane]);
    }
    if (warp >= 2) return;
    // dimensions of m-tile k: d (rows g) and d + 1 (rows g + 8)
    const int VW = D >= 128 ? 4 : 2, d = 4 * VW * (gq + 8 * (k / (2 * VW))) + 4 * (k / 2 % VW) + 2 * (k & 1);
    const float v[4] = {a.o.x, a.o.y, a.o.z, a.o.w};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int col = 8 * ct + 2 * tq + c;
        if (col >= p.C) continue;
        const int row = col / p.G, h = g * p.G + col % p.G;
        const size_t out = (((size_t)b * p.M + row) * p.Hq + h) * D + d;
        const bool seen = row < rows;
        const int e = (int)a.e[c];
        store_out(p.o, p.o_type, out, seen ? scalbnf(v[c] / a.l[c], e) : 0.f);
        store_out(p.o, p.o_type, out + 1, seen ? scalbnf(v[2 + c] / a.l[c], e) : 0.f);
        if (p.sc && k == 0 && gq == 0) {
            float *fin = p.fin + (((size_t)b * p.Hkv + g) * p.C + col) * 2;
            fin[0] = a.m[c];
            fin[1] = 1.f / a.l[c];
        }
    }
}

// Weight received by each position: the stored scores against the columns'
// joined references and sums, in column order.  Bound by reading the scores
// (from L2, mostly), four columns a load where a position's scores are aligned.
constexpr int kAccThreads = 256, kAccPer = 4, kAccSpan = kAccThreads * kAccPer;

__global__ void __launch_bounds__(kAccThreads) kv8_weights_kernel(const AttnP p)
{
    extern __shared__ float st[];   // [C][2]: reference, 1 / sum
    place_next();
    const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    int p0;
    bool bad;
    const int rows = kv8_rows(p.pos, p.counts, b, p.M, p.T_cap, p0, bad);
    const int n = rows > 0 ? p0 + rows : 0, t0 = blockIdx.x * kAccSpan + tid;
    if (t0 - tid >= n) {
        wait_for_previous();
        return;
    }
    const size_t head = (size_t)b * p.Hkv + g;
    // what does not come from the merge is loaded ahead of it
    float a[kAccPer];
#pragma unroll
    for (int i = 0; i < kAccPer; ++i) {
        const int t = t0 + i * kAccThreads;
        a[i] = t < min(p0, n) && p.acc_in ? p.decay * p.acc_in[head * p.T_cap + t] : 0.f;
    }
    wait_for_previous();
    for (int i = tid; i < 2 * p.C; i += kAccThreads) st[i] = __ldcg(p.fin + head * p.C * 2 + i);
    __syncthreads();
    const float *sc = p.sc + (head * p.T_cap + t0) * p.C;
    auto add = [&](int i, int c, int m, float s) {
        if (m < rows && t0 + i * kAccThreads <= p0 + m) a[i] = fmaf(exp2f(s - st[2 * c]), st[2 * c + 1], a[i]);
    };
    if (p.C % 4 == 0) {
#pragma unroll 2
        for (int c = 0; c < p.C; c += 4) {
            float4 v[kAccPer];
#pragma unroll
            for (int i = 0; i < kAccPer; ++i)
                v[i] = t0 + i * kAccThreads < n ? __ldcg(reinterpret_cast<const float4 *>(sc + (size_t)i * kAccThreads * p.C + c))
                                                : make_float4(0.f, 0.f, 0.f, 0.f);
            int m[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                int h = c + k;
                m[k] = p.by_group.by(h);
            }
#pragma unroll
            for (int i = 0; i < kAccPer; ++i) {
                add(i, c, m[0], v[i].x);
                add(i, c + 1, m[1], v[i].y);
                add(i, c + 2, m[2], v[i].z);
                add(i, c + 3, m[3], v[i].w);
            }
        }
    } else
        for (int c = 0; c < p.C; ++c) {
            int h = c;
            const int m = p.by_group.by(h);
#pragma unroll
            for (int i = 0; i < kAccPer; ++i)
                add(i, c, m, t0 + i * kAccThreads < n ? __ldcg(sc + (size_t)i * kAccThreads * p.C + c) : 0.f);
        }
#pragma unroll
    for (int i = 0; i < kAccPer; ++i)
        if (t0 + i * kAccThreads < n) p.acc[head * p.T_cap + t0 + i * kAccThreads] = a[i];
}

// Positions per chunk: r tiles a warp, from the cache's shape alone, so that a
// row's result does not depend on the call.  152 SMs take three CTAs each (two
// of two column tiles of 256), so chunks run in waves of 456.  A batch is taken
// as three quarters full with half a chunk more per head: the smallest r that
// runs in one wave, and at most 2048 positions, which leave uneven lengths
// something to share out.  One sequence is taken as full; a chunk's end costs
// about two tiles, and its last wave takes 7 (12) of a wave's 17 parts of time
// when it has at most one chunk (two) for an SM.
// (Microseconds a call among other kernels at r = 3, 4, 5, 6, 8, 10, 16: 8 x 8K of
// 2 heads of 256: 25, 19, 20, 21, 21, 22, 23, with four rows a sequence 55, 47, 46,
// 37, 43, 44, 37; 4 x 64K of 2 heads of 256: 57, 53, 53, 52, 46, 52, 42; 16 x 16K of
// 8 heads of 128, e4m3: 86, 81, 79, 79, 78, 78, 73; 8 x 24K of 8 heads of 64 with
// uneven lengths and weights: 47, 44, 42, 45, 41, 41, 50; one of 40K of 2
// heads of 256: 18, 19, 18, 19, 20, 19, 24, with four rows 38, 42, 33, 36, 40, 28, 37;
// one of 132K: 46, 43, 36, 39, 44, 33, 32; one of 32K of 8 heads of 128: 25, 26, 21,
// 22, 21, 22, 23.  The rule takes 6, 16, 16, 8, 10, 10 and 5 for these caches; its two tiles
// and its 7 and 12 of 17 are fitted to such figures and stand for nothing else.)  A cache that is
// mostly empty pays for it: at 2K positions one sequence of 2 heads of 256
// takes 17 us in a capacity of 132K and 8 in one of 2K.
int kv8_chunk(const moe_kv8 &c)
{
    const int round = kWarps * kTileBytes / c.head_dim;
    const long long heads = (long long)c.batch * c.kv_heads, slots = 456, quarters = c.head_dim == 256 ? 1216 : 1824;
    long long least = LLONG_MAX;                                     // in seventeenths of a tile
    int best = 1;
    for (const int r : {1, 2, 3, 4, 5, 6, 8, 10, 16}) {
        if (c.batch > 1) {
            if (r * round > 2048)
                break;
            best = r;
            if (heads * (3LL * c.T_cap / (r * round) + 2) <= quarters)
                break;
            continue;
        }
        const long long n = heads * ((c.T_cap + r * round - 1) / (r * round)), rest = n % slots;
        const long long cost = (n / slots * 17 + (rest == 0 ? 0 : rest <= 152 ? 7 : rest <= 304 ? 12 : 17)) * (r + 2);
        if (cost <= least) {
            least = cost;
            best = r;
        }
    }
    return best * round;
}

// Once per kernel and device.
struct Once {
    std::once_flag flag[64];
    int sms[64] = {};
};

struct Kv8Ws {
    size_t cnt, ml, e, o, fin, sc, total;
};
Kv8Ws kv8_ws(const moe_kv8 &c, int M, bool weights)
{
    const size_t slots = (size_t)c.batch * ((c.T_cap + kv8_chunk(c) - 1) / kv8_chunk(c)) * c.kv_heads;
    const int C = c.q_heads / c.kv_heads * M, NC = 8 * kv8_nt(C);
    const size_t cols = (size_t)(C + NC - 1) / NC * NC;
    Kv8Ws w;
    w.cnt = 0;
    w.ml = 256;
    w.e = align_up(w.ml + slots * cols * 2 * sizeof(float), 256);
    w.o = align_up(w.e + slots * cols * sizeof(float), 256);
    w.fin = align_up(w.o + slots * cols * c.head_dim * sizeof(float), 256);
    w.sc = align_up(w.fin + (size_t)c.batch * c.kv_heads * C * 2 * sizeof(float), 256);
    w.total = weights ? align_up(w.sc + (size_t)c.batch * c.kv_heads * c.T_cap * C * sizeof(float), 256) : w.sc;
    return w;
}

}  // namespace

size_t kv8_attn_workspace_bytes(const moe_kv8 &c, int M, bool weights) { return kv8_ws(c, M, weights).total; }

int launch_kv8_attn(const moe_kv8 &c, const moe_rows &q, int M, const int32_t *pos, const int32_t *counts, float scale,
                    void *o, int o_type, const float *acc_in, float *acc, float decay, void *ws, int *err,
                    cudaStream_t stream)
{
    AttnP p;
    const Kv8Ws w = kv8_ws(c, M, acc != nullptr);
    uint8_t *base = static_cast<uint8_t *>(ws);
    p.q = q.data_dev;
    p.qb = q.seq;
    p.qm = q.row;
    p.qh = q.head;
    p.k = static_cast<const uint8_t *>(c.k_dev);
    p.v = static_cast<const uint8_t *>(c.v_dev);
    p.ks = c.k_scale_dev;
    p.vs = c.v_scale_dev;
    p.pos = pos;
    p.counts = counts;
    p.part_ml = reinterpret_cast<float *>(base + w.ml);
    p.part_e = reinterpret_cast<float *>(base + w.e);
    p.part_o = reinterpret_cast<float *>(base + w.o);
    p.fin = reinterpret_cast<float *>(base + w.fin);
    p.sc = acc ? reinterpret_cast<float *>(base + w.sc) : nullptr;
    p.o = o;
    p.acc_in = acc_in;
    p.acc = acc;
    p.decay = decay;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.err = err;
    p.B = c.batch;
    p.Hq = c.q_heads;
    p.Hkv = c.kv_heads;
    p.G = c.q_heads / c.kv_heads;
    p.M = M;
    p.C = p.G * M;
    p.T_cap = c.T_cap;
    p.chunk = kv8_chunk(c);
    p.nchunk = (c.T_cap + p.chunk - 1) / p.chunk;
    p.blk_log = 0;
    while ((1 << p.blk_log) < c.block) ++p.blk_log;
    p.nblk = c.T_cap / c.block;
    p.by_head = div_of(p.Hkv);
    p.by_group = div_of(p.G);
    p.f16 = q.type == MOE_F16;
    p.o_type = o_type;
    p.streams = 2LL * c.batch * c.kv_heads * c.T_cap * c.head_dim > (96LL << 20);
    p.qvec = reinterpret_cast<uintptr_t>(q.data_dev) % 16 == 0 && q.seq % 8 == 0 && q.row % 8 == 0 && q.head % 8 == 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
    const int nt = kv8_nt(p.C);
    p.by_pass = div_of((p.C + 8 * nt - 1) / (8 * nt));
    const long long items = (long long)p.nchunk * p.B * p.Hkv * ((p.C + 8 * nt - 1) / (8 * nt));
    if (items > INT_MAX / 2) return MOE_ERR_UNSUPPORTED;
    auto go = [&](auto kernel, int smem, int ctas, Once &once) {
        std::call_once(once.flag[dev], [&] {
            e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         (int)cudaSharedmemCarveoutMaxShared);
            if (e == cudaSuccess) e = cudaDeviceGetAttribute(&once.sms[dev], cudaDevAttrMultiProcessorCount, dev);
        });
        if (e == cudaSuccess && once.sms[dev] < 1) e = cudaErrorInvalidDevice;
        if (e != cudaSuccess) return;
        const int grid = (int)std::min<long long>(items, (long long)once.sms[dev] * ctas);
        p.counter = nullptr;
        if (items >= 3LL * grid) {
            p.counter = reinterpret_cast<int *>(base + w.cnt);
            e = cudaMemsetAsync(p.counter, 0, sizeof(int), stream);
            if (e != cudaSuccess) return;
        }
        // One or two CTAs on every SM rather than more on some, which a call
        // right behind another otherwise gets (one of 40K of 2 heads of 256: 21.6 us
        // against 18.8 where it does not).
        if (grid <= 2 * once.sms[dev]) smem = std::max(smem, grid <= once.sms[dev] ? 116 << 10 : 78 << 10);
        e = launch_after(kernel, dim3(grid), kThreads, smem, 0, stream, p);
    };
#define KV8_GO(F, D, N)                                                                      \
    do {                                                                                     \
        static Once once;                                                                    \
        static_assert(Lay<D, N>::total(MOE_KV8_MAX_BATCH) <= kSmemMax, "shared memory");     \
        go(kv8_chunk_kernel<F, D, N>, Lay<D, N>::total(p.B), Lay<D, N>::ctas, once);         \
    } while (0)
#define KV8_GO_D(F, D)                \
    do {                              \
        if (nt == 1) KV8_GO(F, D, 1); \
        else KV8_GO(F, D, 2);         \
    } while (0)
#define KV8_GO_F(F)                                \
    do {                                           \
        if (c.head_dim == 256) KV8_GO_D(F, 256);   \
        else if (c.head_dim == 128) KV8_GO_D(F, 128); \
        else KV8_GO_D(F, 64);                      \
    } while (0)
    if (c.format == MOE_KV8_INT8) KV8_GO_F(MOE_KV8_INT8);
    else KV8_GO_F(MOE_KV8_E4M3);
#undef KV8_GO_F
#undef KV8_GO_D
#undef KV8_GO
    if (e != cudaSuccess) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
    note_launch();
    {
        int shares = 1;
        while (shares < kMergeShares && p.nchunk > 32 * shares) shares *= 2;
        const int each = (p.nchunk + 4 * shares - 1) / (4 * shares);             // chunks a warp
        const dim3 grid(shares * (c.head_dim / 32) * ((p.C + 7) / 8), p.Hkv, p.B);
        const bool few = (long long)grid.x * grid.y * grid.z <= 304;
        e = launch_after(few && each > 4 ? kv8_merge_kernel<8> : few && each > 2 ? kv8_merge_kernel<4> : kv8_merge_kernel<2>, grid,
                         kMergeThreads, 0, shares, stream, p, c.head_dim, shares);
        if (e != cudaSuccess) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
    }
    note_launch();
    if (acc) {
        e = launch_after(kv8_weights_kernel, dim3((c.T_cap + kAccSpan - 1) / kAccSpan, p.Hkv, p.B), kAccThreads,
                         p.C * 2 * (int)sizeof(float), 0, stream, p);
        if (e != cudaSuccess) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
        note_launch();
    }
    return MOE_OK;
}

}  // namespace moe
