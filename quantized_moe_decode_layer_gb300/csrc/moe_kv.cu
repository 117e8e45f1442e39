// 16-bit key/value cache of a batch of sequences: appending rows, and attention
// of at most 16 rows a key/value head (tokens, drafts, questions about one document)
// over it; and the merge of partial results, moe_kv_tile.cu's too.
//
// What it computes: query row at position p, head h, g = h / (Hq / Hkv):
//     s_t = scale q . k_t,  t <= p and (t > p - W or t < S)
//     o   = sum_t softmax(s)_t v_t
// and, behind a shared prefix, the prefix's positions in the same softmax.
//
// Split kernel.  A problem is the rows of one sequence that share a key/value
// head (M rows times Hq / Hkv heads) against the positions that any of them sees,
// counted through: the first S, then the window.  The prefix of a small batch is one more
// problem per head with the whole batch's rows: its keys are read once.  Every problem is
// cut into tiles of 64 positions, the tiles of all problems lie in one line, and each
// CTA takes an equal stretch of it: whatever the lengths are (they are read on the device),
// all CTAs move about the same number of bytes.  A stretch that holds a whole problem writes its
// outputs; a part of one leaves its unnormalised sum, maximum and sum of weights (the
// running maximum and sum of a softmax), which the merge kernel joins in
// order.  Slot (CTA + problem) is a part's own: along the line either grows.
//
// It is bound by HBM: keys and values come through cp.async as units of 64 positions into a ring
// that runs ahead across problems (96 to 200 KB an SM in flight); the products (m16n8k16, 16
// rows) take less than half a tile's time.  16 rows leave tcgen05's 128-row tiles seven
// eighths empty; more rows are taken there (32 rows here: twice its time).  48
// sequences of up to 4096 positions, 8 heads of 128: 115 us, 6.6 TB/s, 97 to 99 % of a copy's rate.
//
// Scores, maxima, sums and outputs are fp32; the weights are rounded to the
// cache's 16-bit type for the second product, an error of half a step, as the
// output's own rounding is (fp16's smallest weights: kv_up in moe_kv.h).
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include "moe_kv.h"
#include "moe_kv8.cuh"

namespace moe {
namespace {


struct Once {
    std::once_flag flag[64];
    int sms[64];
};

__device__ __forceinline__ uint32_t su32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Rows of sequence b that the call works on, and the first one's position.
__device__ __forceinline__ int rows_of(const KvCall &p, int b, int &p0, bool &bad)
{
    const int32_t last = p.T - p.M;
    return kv8_rows(p.pos ? p.pos + b : &last, p.counts ? p.counts + b : nullptr, 0, p.M, p.limit, p0, bad);
}

// Positions that any of a sequence's n rows from p0 on sees: 0 .. ns - 1, then lo .. p0 + n - 1.
__device__ __forceinline__ int visible(const KvCall &p, int p0, int n, int &lo, int &ns)
{
    lo = ns = 0;
    if (n == 0) return 0;
    lo = max(0, p0 - p.W + 1);
    ns = min(p.S, lo);
    return ns + p0 + n - lo;
}

// The line of tiles: the prefix's (all of head 0's, then head 1's ...), then for
// each sequence its heads'.  A sequence's problem has w more places ahead of its tiles, for what its start and end
// cost, so that a CTA of many short problems has fewer tiles (32 sequences of up to 2000, 32/8/128: 25 -> 22 us; 64 behind a
// prefix: 65 -> 59); none where a CTA has few tiles.
struct Line {
    int NP;             // problems of the prefix: its heads, or none
    int ptiles;         // tiles of one of them
    int w;
    int total, share;   // places; places a CTA
};
constexpr int kPlaces = 2;
__device__ __forceinline__ Line line_of(const KvCall &p, int seq_tiles, int ctas)
{
    Line l;
    l.NP = p.split_prefix ? p.Hkv : 0;
    l.ptiles = p.split_prefix ? (p.P + kKvTile - 1) / kKvTile : 0;
    l.w = l.NP * l.ptiles + seq_tiles * p.Hkv >= 4 * ctas ? kPlaces : 0;
    l.total = l.NP * l.ptiles + (seq_tiles + l.w * p.B) * p.Hkv;
    l.share = max(1, (l.total + ctas - 1) / ctas);
    return l;
}

// What the threads need to know of a problem while its tiles are computed.
struct Problem {
    int id;         // slot = CTA + id
    int n, ns, lo;  // positions seen; the first ns are 0 .. ns - 1, then from lo on
    int p0, cnt;    // first row's position, rows; the prefix: every row of the batch sees all of it
    int tiles;
    int whole;      // the CTA has all its tiles: outputs are written at once
    int b, g;       // sequence (-1: the prefix), head
};

// A CTA: four groups of 16 of a tile's positions, times WD parts of the output's columns (the warps of every
// column part take the scores of their positions themselves).  With 256 columns a warp's output takes 128
// registers, so two warps share it.
template <int D>
struct Lay {
    static constexpr int WD = D == 256 ? 2 : 1;
    static constexpr int WK = 4, KW = kKvTile / WK;        // position groups, positions of one
    static constexpr int kThreads = 32 * WK * WD;
    static constexpr int RB = kKvFewRows;
    static constexpr int kRow = D * 2;
    static constexpr int kUnit = kKvTile * kRow;           // keys or values of a tile
    static constexpr int kQ = RB * kRow;
    static constexpr int ctas = D == 256 ? 1 : D == 128 ? 2 : 3;
    // units in the ring, and problems whose q is there: the one whose keys are waited for, and those that the NU - 1
    // units ahead may have begun (q goes to registers with a problem's first keys)
    static constexpr int NU = D == 64 ? 8 : 6, NQ = NU / 2;
    static constexpr int q = NU * kUnit;
    static constexpr int probs = q + NQ * kQ;
    static constexpr int misc = probs + (NQ + 1) * (int)sizeof(Problem);   // maxima and sums of the position groups
    static constexpr int cum = misc + (2 * WK * RB + 8) * 4;               // tiles before a sequence; its first row's position; its rows
    static constexpr int total(int B) { return cum + (B + 1) * 4 + B * 5; }
    static_assert(q % 128 == 0 && probs % 4 == 0 && misc % 4 == 0 && cum % 4 == 0, "alignment");
};

// 16-byte chunk c of row r of a tile, swizzled so that eight rows' equal chunks lie in eight banks' groups.
template <int D>
__device__ __forceinline__ uint32_t at(int r, int c) { return (uint32_t)(r * (D * 2) + ((c ^ (r & 7)) << 4)); }

template <bool F16, int D>
__global__ void __launch_bounds__(Lay<D>::kThreads, Lay<D>::ctas) kv_split_kernel(const KvCall p)
{
    using L = Lay<D>;
    constexpr int RB = L::RB, WK = L::WK, WD = L::WD, KW = L::KW, NU = L::NU, kThreads = L::kThreads;
    constexpr int DW = D / WD;      // a warp's columns
    constexpr float kUp = kv_up(F16);
    extern __shared__ __align__(128) uint8_t sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Problem *probs = reinterpret_cast<Problem *>(sm + L::probs);
    float *gm = reinterpret_cast<float *>(sm + L::misc), *gl = gm + WK * RB;
    int *wsum = reinterpret_cast<int *>(gl + WK * RB);
    int *cum = reinterpret_cast<int *>(sm + L::cum), *first_pos = cum + p.B + 1;
    uint8_t *n_rows = reinterpret_cast<uint8_t *>(first_pos + p.B);
    if (p.late) place_next();
    else after_previous();

    // tiles of every sequence, summed up
    {
        const int per = (p.B + kThreads - 1) / kThreads, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
        int sum = 0;
        for (int b = b0; b < b1; ++b) {
            int p0, lo, ns;
            bool bad;
            const int n = rows_of(p, b, p0, bad);
            if (bad && blockIdx.x == 0) atomicOr(p.err, kKv8ErrRange);
            first_pos[b] = p0;
            n_rows[b] = (uint8_t)n;
            sum += (visible(p, p0, n, lo, ns) + kKvTile - 1) / kKvTile;
            cum[b + 1] = sum;
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int before = incl - sum;
        for (int w = 0; w < warp; ++w) before += wsum[w];
        for (int b = b0; b < b1; ++b) cum[b + 1] += before;
        if (tid == 0) cum[0] = 0;
        __syncthreads();
    }
    const Line ln = line_of(p, cum[p.B], gridDim.x);
    const int t0 = min(ln.total, (int)blockIdx.x * ln.share), t1 = min(ln.total, t0 + ln.share);
    // the problem and tile that t0 falls on, or the first behind it; tiles up to t1
    int id0 = -1, i0 = 0, ntiles = 0;
    {
        const int pt = ln.NP * ln.ptiles;
        int left = t1 - t0;
        if (t0 < pt && left > 0) {
            id0 = t0 / ln.ptiles;
            i0 = t0 - id0 * ln.ptiles;
            ntiles = min(left, pt - t0);
            left -= ntiles;
        }
        if (left > 0) {
            const int x = max(t0 - pt, 0);
            int lo = 0, hi = p.B - 1;   // the last b with the places before it <= x
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if ((cum[mid] + ln.w * mid) * p.Hkv <= x) lo = mid;
                else hi = mid - 1;
            }
            int each = cum[lo + 1] - cum[lo], y = x - (cum[lo] + ln.w * lo) * p.Hkv, j = y / (each + ln.w), at = y - j * (each + ln.w);
            while (left > 0) {
                const int take = min(left, each + ln.w - at), from = max(at - ln.w, 0), n = max(at + take - ln.w, 0) - from;
                if (n > 0 && id0 < 0) {
                    id0 = ln.NP + lo * p.Hkv + j;
                    i0 = from;
                }
                ntiles += n;
                left -= take;
                at = 0;
                if (++j == p.Hkv || each + ln.w == 0) {
                    j = 0;
                    if (++lo == p.B) break;
                    each = cum[lo + 1] - cum[lo];
                }
            }
        }
    }
    if (ntiles == 0) {
        if (p.late) wait_for_previous();
        return;
    }

    // ------------------------------------------------------------- loading
    // cursor of the loads: unit (keys, then values) of tile li of problem lp, NU - 1 units ahead
    Problem lp;
    int li, lcount = -1, lvalues = 0;   // lcount: problems opened by this CTA, less one
    const uint16_t *lk, *lv;
    long long lkm, lvm;
    int lbase;                          // slot of position lo

    auto open = [&](int id, int i) {
        lp.id = id;
        if (id < ln.NP) {
            lp.b = -1;
            lp.g = id;
            lp.n = p.P;
            lp.ns = lp.lo = 0;
            lp.p0 = INT_MAX;
            lp.cnt = p.M;
            lk = p.pk + lp.g * p.pkh;
            lv = p.pv + lp.g * p.pvh;
            lkm = p.pkm;
            lvm = p.pvm;
            lbase = 0;
        } else {
            const int x = id - ln.NP, b = x / p.Hkv;
            lp.b = b;
            lp.g = x - b * p.Hkv;
            lp.cnt = n_rows[b];
            lp.p0 = first_pos[b];
            lp.n = visible(p, lp.p0, lp.cnt, lp.lo, lp.ns);
            lk = p.k + b * p.kb + lp.g * p.kh;
            lv = p.v + b * p.vb + lp.g * p.vh;
            lkm = p.km;
            lvm = p.vm;
            lbase = lp.lo < p.T ? lp.lo : p.S + (lp.lo - p.S) % (p.T - p.S);
        }
        lp.tiles = (lp.n + kKvTile - 1) / kKvTile;
        li = i;
        lp.whole = i == 0 && lp.tiles <= ntiles;
        ++lcount;
        // its rows of q (those of idle sequences and padding are loaded like the others; nothing of them is used)
        constexpr int CH = D / 8;
        uint8_t *qs = sm + L::q + (lcount % L::NQ) * L::kQ;
        const int R = lp.b < 0 ? p.B * p.M * p.G : p.M * p.G;
        for (int x = tid; x < RB * CH; x += kThreads) {
            const int r = x / CH, c = x % CH;
            int m = p.by_g(r), b = lp.b;
            const int h = r - m * p.G;
            if (b < 0) {
                b = m / p.M;
                m -= b * p.M;
            }
            const bool ok = r < R;
            const uint16_t *src = ok ? p.q + b * p.qb + m * p.qm + (long long)(lp.g * p.G + h) * p.qh + 8 * c : p.q;
            cp16(su32(qs) + at<D>(r, c), src, ok);
        }
    };
    auto load = [&](int slot_of_ring) {
        constexpr int CH = D / 8, RPI = kThreads / CH;
        const uint32_t to = su32(sm + slot_of_ring * L::kUnit);
        const uint16_t *src = lvalues ? lv : lk;
        const long long step = lvalues ? lvm : lkm;
        static_assert(RPI % 8 == 0, "a thread's rows have one swizzle");
        const int c = tid % CH, r0 = tid / CH, v0 = li * kKvTile;
        const uint32_t dst = to + at<D>(r0, c);
        int first = lbase + v0 - lp.ns;     // slot of the tile's first position, where it is not among the first S
        if (lp.b >= 0 && first >= p.T) first -= p.T - p.S;
        if (v0 >= lp.ns && v0 + kKvTile <= lp.n && (lp.b < 0 || first + kKvTile <= p.T)) {   // 64 slots in a row
            const uint16_t *from = src + (first + r0) * step + 8 * c;
#pragma unroll
            for (int i = 0; i < kKvTile / RPI; ++i) {
                cp16(dst + (uint32_t)(i * RPI * L::kRow), from, true);
                from += RPI * step;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kKvTile / RPI; ++i) {
            const int v = v0 + r0 + i * RPI;
            int slot = v;
            if (v >= lp.ns) {
                slot = lbase + (v - lp.ns);
                if (lp.b >= 0 && slot >= p.T) slot -= p.T - p.S;
            }
            const bool ok = v < lp.n;   // behind the last: zeros
            if (!ok) slot = 0;
            cp16(dst + (uint32_t)(i * RPI * L::kRow), src + slot * step + 8 * c, ok);
        }
    };

    int left = ntiles;   // tiles whose values are not yet loaded
    open(id0, i0);
    if (tid == 0) probs[0] = lp;
    // the next unit of the line into the ring
    auto next = [&](int slot_of_ring) {
        if (left > 0) {
            if (li == lp.tiles) {
                int id = lp.id + 1;
                if (id >= ln.NP) {
                    int b = (id - ln.NP) / p.Hkv;
                    if (cum[b + 1] == cum[b]) {     // sequences without tiles (some with are behind)
                        do ++b;
                        while (cum[b + 1] == cum[b]);
                        id = ln.NP + b * p.Hkv;
                    }
                }
                open(id, 0);
                lp.whole = lp.tiles <= left;
                if (tid == 0) probs[lcount % (L::NQ + 1)] = lp;
            }
            load(slot_of_ring);
            lvalues ^= 1;
            if (lvalues == 0) {
                --left;
                ++li;
            }
        }
        cp_commit();
    };
#pragma unroll 1
    for (int u = 0; u < NU - 1; ++u) next(u);

    // ----------------------------------------------------------- computing
    const int wd = warp % WD, wk = warp / WD;
    const int rA = lane >> 2;                      // this thread's rows: rA, rA + 8
    const int key0 = wk * KW;
    uint32_t qf[D / 16][4];                        // the rows of q, as operands
    float acc[DW / 8][4];
    float mrun[2], lrun[2];
    int lowA = 0, highA = 0, lowB = 0, highB = 0;  // positions rows see: low < t <= high, or t < S
    Problem cp;
    int ci = -1, ccount = -1, slot = 0;

#pragma unroll 1
    for (int it = 0; it < ntiles; ++it) {
        cp_wait<NU - 2>();
        __syncthreads();
        next(slot == 0 ? NU - 1 : slot - 1);
        if (ci < 0 || ++ci == cp.tiles) {
            ++ccount;
            cp = probs[ccount % (L::NQ + 1)];
            ci = ci < 0 ? i0 : 0;   // (the CTA's first starts where the CTA does)
#pragma unroll
            for (int i = 0; i < DW / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
            mrun[0] = mrun[1] = -INFINITY;
            lrun[0] = lrun[1] = 0.f;
            auto limits = [&](int r, int &low, int &high) {
                const int m = p.by_g(r);
                high = cp.b < 0 ? INT_MAX : m < cp.cnt ? cp.p0 + m : -1;
                low = cp.b < 0 || m >= cp.cnt ? -1 : cp.p0 + m - p.W;
            };
            limits(rA, lowA, highA);
            limits(rA + 8, lowB, highB);
            const uint32_t qs = su32(sm + L::q + (ccount % L::NQ) * L::kQ);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) ldsm(qf[kk], qs + at<D>(lane & 15, 2 * kk + (lane >> 4)));
        }

        // scores
        float s[KW / 8][4];
        {
            const uint32_t ks = su32(sm + slot * L::kUnit);
#pragma unroll
            for (int j = 0; j < KW / 8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int j = 0; j < KW / 16; ++j) {
                    uint32_t b[4];
                    ldsm(b, ks + at<D>(key0 + 16 * j + (lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)));
                    mma<F16>(s[2 * j], qf[kk], b[0], b[1]);
                    mma<F16>(s[2 * j + 1], qf[kk], b[2], b[3]);
                }
        }
        if (++slot == NU) slot = 0;
        // in units of log2; positions that a row does not see
        const int v0 = ci * kKvTile + key0 + 2 * (lane & 3);
        const int first = ci * kKvTile, last = min(first + kKvTile, cp.n) - 1;
        const bool edge = first + kKvTile > cp.n ||
                          (cp.b >= 0 && cp.cnt > 1 && last >= cp.ns &&
                           (cp.lo + last - cp.ns > cp.p0 || cp.lo + max(first - cp.ns, 0) <= cp.p0 + cp.cnt - 1 - p.W));
#pragma unroll
        for (int j = 0; j < KW / 8; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[j][x] = __fmul_rn(s[j][x], p.c);
        if (edge) {
#pragma unroll
            for (int j = 0; j < KW / 8; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int v = v0 + 8 * j + (x & 1), t = v < cp.ns ? v : cp.lo + v - cp.ns;
                    const int low = x < 2 ? lowA : lowB, high = x < 2 ? highA : highB;
                    if (!(v < cp.n && t <= high && (t > low || t < p.S))) s[j][x] = -INFINITY;
                }
        }
        // running maximum and sum
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < KW / 8; ++j) {
            mx[0] = fmaxf(mx[0], fmaxf(s[j][0], s[j][1]));
            mx[1] = fmaxf(mx[1], fmaxf(s[j][2], s[j][3]));
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xFFFFFFFFu, mx[0], o));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xFFFFFFFFu, mx[1], o));
        }
        // The reference, kUp below a maximum, follows it only when that has grown by more
        // than 8 (a factor of 256, far from fp16's and fp32's ends): the
        // output is hardly ever rescaled.  (The difference: a sum would round past the maximum where scores are 16 apart.)
        const bool raise[2] = {__fsub_rn(mx[0], mrun[0]) > 8.f + kUp, __fsub_rn(mx[1], mrun[1]) > 8.f + kUp};
        if (__any_sync(0xFFFFFFFFu, raise[0] || raise[1])) {
            float al[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float mn = raise[x] ? __fsub_rn(mx[x], kUp) : mrun[x];
                al[x] = mrun[x] == mn ? 1.f : ex2(mrun[x] - mn);
                mrun[x] = mn;
                lrun[x] *= al[x];
            }
#pragma unroll
            for (int i = 0; i < DW / 8; ++i) {
                acc[i][0] *= al[0];
                acc[i][1] *= al[0];
                acc[i][2] *= al[1];
                acc[i][3] *= al[1];
            }
        }
        const float ref[2] = {mrun[0] == -INFINITY ? 0.f : mrun[0], mrun[1] == -INFINITY ? 0.f : mrun[1]};
        uint32_t w16[KW / 8][2];
#pragma unroll
        for (int j = 0; j < KW / 8; ++j) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s[j][x] = ex2(s[j][x] - ref[x >> 1]);
                lrun[x >> 1] += s[j][x];
            }
            w16[j][0] = pack2<F16>(s[j][0], s[j][1]);
            w16[j][1] = pack2<F16>(s[j][2], s[j][3]);
        }
        // weighted values
        cp_wait<NU - 2>();
        __syncthreads();
        next(slot == 0 ? NU - 1 : slot - 1);
        const uint32_t vs = su32(sm + slot * L::kUnit);
#pragma unroll
        for (int j = 0; j < KW / 16; ++j) {
            const uint32_t a[4] = {w16[2 * j][0], w16[2 * j][1], w16[2 * j + 1][0], w16[2 * j + 1][1]};
#pragma unroll
            for (int dd = 0; dd < DW / 16; ++dd) {
                uint32_t b[4];
                ldsm_t(b, vs + at<D>(key0 + 16 * j + (lane & 15), wd * (DW / 8) + 2 * dd + (lane >> 4)));
                mma<F16>(acc[2 * dd], a, b[0], b[1]);
                mma<F16>(acc[2 * dd + 1], a, b[2], b[3]);
            }
        }
        const int used = slot;
        if (++slot == NU) slot = 0;
        if (ci + 1 < cp.tiles && it + 1 < ntiles) continue;

        // ---------------------------------------- the problem's or CTA's end
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            lrun[0] += __shfl_xor_sync(0xFFFFFFFFu, lrun[0], o);
            lrun[1] += __shfl_xor_sync(0xFFFFFFFFu, lrun[1], o);
        }
        // a row of NaN alone has no maximum, but is not empty
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (lrun[x] != lrun[x] && mrun[x] == -INFINITY) mrun[x] = 0.f;
        const bool direct = cp.whole && p.P == 0;
        const int R = cp.b < 0 ? p.B * p.M * p.G : p.M * p.G;
        const size_t part = ((size_t)blockIdx.x + cp.id) * RB;
        // The position groups' outputs are joined in the unit that was just read (its next load comes after the
        // next barrier), eight rows at a time: every group's as they are, then their weighted sum.
        if ((lane & 3) == 0 && wd == 0) {
            gm[wk * RB + rA] = mrun[0];
            gm[wk * RB + rA + 8] = mrun[1];
            gl[wk * RB + rA] = lrun[0];
            gl[wk * RB + rA + 8] = lrun[1];
        }
        float *out = reinterpret_cast<float *>(sm + used * L::kUnit);   // [WK][8][D]
        static_assert(WK * 8 * D * 4 <= L::kUnit, "outputs in a unit");
        __syncthreads();                                                // the unit has been read by all
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (8 * half >= R) break;
            if (half) __syncthreads();
#pragma unroll
            for (int i = 0; i < DW / 8; ++i) {
                // columns in an order that spreads a warp's rows over the banks
                const int c = wd * DW + 8 * i + 2 * (lane & 3);
                *reinterpret_cast<float2 *>(out + (wk * 8 + rA) * D + (c ^ (8 * (rA & 3)))) = make_float2(acc[i][2 * half], acc[i][2 * half + 1]);
            }
            __syncthreads();
            constexpr int C4 = D / 4;
            for (int x = tid; x < 8 * C4; x += kThreads) {
                const int rr = x / C4, r = 8 * half + rr, c = 4 * (x % C4);
                if (r >= R) break;
                float m = gm[r], l = 0.f;
#pragma unroll
                for (int k = 1; k < WK; ++k) m = fmaxf(m, gm[k * RB + r]);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < WK; ++k) {
                    const float mk = gm[k * RB + r], w = mk == -INFINITY ? 0.f : ex2(mk - m);
                    const float4 u = *reinterpret_cast<const float4 *>(out + (k * 8 + rr) * D + (c ^ (8 * (rr & 3))));
                    l = fmaf(gl[k * RB + r], w, l);
                    v.x = fmaf(u.x, w, v.x);
                    v.y = fmaf(u.y, w, v.y);
                    v.z = fmaf(u.z, w, v.z);
                    v.w = fmaf(u.w, w, v.w);
                }
                if (direct) {
                    const int mm = p.by_g(r), h = r - mm * p.G;
                    const float f = l != 0.f ? 1.f / l : 0.f;
                    uint2 u = make_uint2(0u, 0u);
                    if (mm < cp.cnt) u = make_uint2(pack2<F16>(v.x * f, v.y * f), pack2<F16>(v.z * f, v.w * f));
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + (((size_t)cp.b * p.M + mm) * p.Hq + cp.g * p.G + h) * D + c) = u;
                } else {
                    *reinterpret_cast<float4 *>(p.part_o + (part + r) * D + c) = v;
                    if (c == 0) *reinterpret_cast<float2 *>(p.part_ml + (part + r) * 2) = make_float2(m, l);
                }
            }
        }
    }
    if (p.late) wait_for_previous();   // the end of this kernel means the end of the one before
}

// Joins a row's parts in order: o = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m)
// l_i with m the largest m_i.  One CTA per row and head; each warp takes every
// kMergeWarps-th part with a running maximum, its lanes the columns, and the warps' sums are joined.  Which parts there are
// follows from the lengths, which are there before the kernel in front has ended.  Rows without positions get zeros.
// ONE: a warp per row, its CTA's other warps have other heads of the same row: where there are many rows, most CTAs would
// wait for a place on an SM (512 prompt rows of 32 heads in two parts: 18 -> 10 us; 2048 rows behind a prefix: 9 -> 11).
constexpr int kMergeWarps = 4, kMergeMany = 4096;
template <int D, bool ONE>
__global__ void __launch_bounds__(32 * kMergeWarps) kv_merge_kernel(const KvCall p, int ctas)
{
    constexpr int VEC = D / 32, kThreads = 32 * kMergeWarps;
    __shared__ float red[kMergeWarps][D + 2];
    __shared__ int tsum[2][kMergeWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int STEP = ONE ? 1 : kMergeWarps;   // warps of a row
    const int x0 = ONE ? blockIdx.x * kMergeWarps + warp : blockIdx.x;
    const int hq = x0 % p.Hq, bm = x0 / p.Hq, m = bm % p.M, b = bm / p.M;
    const int g = hq / p.G, h = hq - g * p.G;
    uint16_t *o = static_cast<uint16_t *>(p.o) + ((size_t)bm * p.Hq + hq) * D;
    int p0, lo, ns;
    bool bad;
    const int cnt = rows_of(p, b, p0, bad);
    // parts of the own positions, then of the prefix's: of the tile kernel, or slots of the split kernel
    const int row = (b * p.M + m) * p.G + h;
    const size_t rows = (size_t)p.B * p.M * p.G;
    size_t first = 0, pfirst = 0;
    int n1 = p.own.n, n2 = p.prefix.n;
    if (p.split_own && m < cnt) {
        // tiles of all sequences, and of those before
        int all = 0, before = 0;
        for (int x = tid; x < p.B; x += kThreads) {
            int q0, xlo, xns;
            const int n = rows_of(p, x, q0, bad), t = (visible(p, q0, n, xlo, xns) + kKvTile - 1) / kKvTile;
            all += t;
            before += x < b ? t : 0;
        }
        all = __reduce_add_sync(0xFFFFFFFFu, all);
        before = __reduce_add_sync(0xFFFFFFFFu, before);
        if (lane == 0) {
            tsum[0][warp] = all;
            tsum[1][warp] = before;
        }
        __syncthreads();
        all = before = 0;
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
            all += tsum[0][w];
            before += tsum[1][w];
        }
        const Line ln = line_of(p, all, ctas);
        const int each = (visible(p, p0, cnt, lo, ns) + kKvTile - 1) / kKvTile, j = b * p.Hkv + g;
        const int T0 = ln.NP * ln.ptiles + (before + ln.w * b) * p.Hkv + g * (each + ln.w) + ln.w, c0 = T0 / ln.share;
        n1 = (T0 + each - 1) / ln.share - c0 + 1;
        first = ((size_t)c0 + ln.NP + j) * kKvFewRows + m * p.G + h;
        if (p.split_prefix) {
            const int q0 = g * ln.ptiles, a = q0 / ln.share;
            n2 = (q0 + ln.ptiles - 1) / ln.share - a + 1;
            pfirst = ((size_t)a + g) * kKvFewRows + row;
        }
    }
    wait_for_previous();
    if (m >= cnt) {
        for (int d = ONE ? lane : tid; d < D; d += 32 * STEP) o[d] = 0;
        return;
    }
    if (p.split_own && n1 == 1 && p.P == 0) return;   // written by the split kernel
    auto part = [&](int i, const float *&po) -> const float * {
        const bool own = i < n1;
        if (!own) i -= n1;
        if (own ? p.split_own : p.split_prefix) {
            const size_t x = (own ? first : pfirst) + (size_t)i * kKvFewRows;
            po = p.part_o + x * D;
            return p.part_ml + x * 2;
        }
        const KvCall::Parts &t = own ? p.own : p.prefix;
        const size_t x = ((size_t)i * p.Hkv + g) * rows + row;
        po = t.o + x * D;
        return t.ml + x * 2;
    };
    const int n = n1 + n2;
    float acc[VEC] = {}, l = 0.f, mx = -INFINITY;
    constexpr int AHEAD = 4;    // parts whose loads are in flight
    for (int i0 = ONE ? 0 : warp; i0 < n; i0 += AHEAD * STEP) {
        float2 ml[AHEAD], y[AHEAD][VEC / 2];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int i = i0 + k * STEP;
            ml[k] = make_float2(-INFINITY, 0.f);
            if (i < n) {
                const float *po, *at = part(i, po);
                ml[k] = __ldcg(reinterpret_cast<const float2 *>(at));
#pragma unroll
                for (int v = 0; v < VEC / 2; ++v) y[k][v] = __ldcg(reinterpret_cast<const float2 *>(po) + v * 32 + lane);
            }
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (ml[k].x == -INFINITY) continue;   // none, or empty: its output was not written
            const float top = fmaxf(mx, ml[k].x), f = mx == -INFINITY ? 0.f : ex2(mx - top), w = ex2(ml[k].x - top);
            mx = top;
            l = fmaf(l, f, ml[k].y * w);
#pragma unroll
            for (int v = 0; v < VEC / 2; ++v) {
                acc[2 * v] = fmaf(acc[2 * v], f, y[k][v].x * w);
                acc[2 * v + 1] = fmaf(acc[2 * v + 1], f, y[k][v].y * w);
            }
        }
    }
    if constexpr (ONE) {
        const float f = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int v = 0; v < VEC / 2; ++v)
            *reinterpret_cast<uint32_t *>(o + 64 * v + 2 * lane) =
                p.f16 ? pack2<true>(acc[2 * v] * f, acc[2 * v + 1] * f) : pack2<false>(acc[2 * v] * f, acc[2 * v + 1] * f);
    } else {
#pragma unroll
        for (int v = 0; v < VEC / 2; ++v) {
            red[warp][64 * v + 2 * lane] = acc[2 * v];
            red[warp][64 * v + 2 * lane + 1] = acc[2 * v + 1];
        }
        if (lane == 0) {
            red[warp][D] = l;
            red[warp][D + 1] = mx;
        }
        __syncthreads();
        float top = -INFINITY, w[kMergeWarps], ls = 0.f;
#pragma unroll
        for (int k = 0; k < kMergeWarps; ++k) top = fmaxf(top, red[k][D + 1]);
#pragma unroll
        for (int k = 0; k < kMergeWarps; ++k) {
            w[k] = red[k][D + 1] == -INFINITY ? 0.f : ex2(red[k][D + 1] - top);
            ls = fmaf(red[k][D], w[k], ls);
        }
        const float f = ls != 0.f ? 1.f / ls : 0.f;
        for (int d = 2 * tid; d < D; d += 2 * kThreads) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int k = 0; k < kMergeWarps; ++k) {
                x = fmaf(red[k][d], w[k], x);
                y = fmaf(red[k][d + 1], w[k], y);
            }
            *reinterpret_cast<uint32_t *>(o + d) = p.f16 ? pack2<true>(x * f, y * f) : pack2<false>(x * f, y * f);
        }
    }
}

// ------------------------------------------------------------------ append

// Rows of a call that stay: of each sequence the last T - S (T where it has no
// window), and those at the first S positions.  Thread: 8 elements of a row's head.
struct AppendCall {
    const void *k, *v;
    long long kb, km, kh, vb, vm, vh;
    uint16_t *to_k, *to_v;
    const int32_t *pos, *counts;
    int *err;
    int B, M, Hkv, D, T, S, limit, f16, type, vec;
    int nring, nfirst;   // candidates a sequence: in the ring, at the first positions
};

template <int TYPE>
__device__ __forceinline__ void get8(const void *base, long long at, bool vec, float (&x)[8])
{
    if (TYPE == MOE_F32) {
        const float *f = static_cast<const float *>(base) + at;
        if (vec) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(f)), b = __ldg(reinterpret_cast<const float4 *>(f) + 1);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __ldg(f + i);
        }
    } else {
        const uint16_t *h = static_cast<const uint16_t *>(base) + at;
        uint32_t w[4];
        if (vec) {
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(h));
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __ldg(h + 2 * i) | (uint32_t)__ldg(h + 2 * i + 1) << 16;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (TYPE == MOE_F16) {
                const float2 f = __half22float2(as_half2(w[i]));
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
}

template <int TYPE>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendCall p)
{
    after_previous();
    const int CH = p.D / 8, b = blockIdx.y;
    int p0;
    bool bad;
    const int n = kv8_rows(p.pos, p.counts, b, p.M, p.limit, p0, bad);
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, kKv8ErrRange);
    if (n == 0) return;
    const long long per = (long long)p.Hkv * CH, all = per * (p.nring + p.nfirst) * 2;
    for (long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x; x < all; x += (long long)gridDim.x * blockDim.x) {
        const int is_v = x >= all / 2;
        const long long y = is_v ? x - all / 2 : x;
        const int u = (int)(y / per), e = (int)(y - u * per), g = e / CH, c = e - g * CH;
        int t;
        if (u < p.nring) {
            t = p0 + n - 1 - u;
            if (t < p0 || t < p.S) continue;
        } else {
            t = p0 + (u - p.nring);
            if (t >= p0 + n || t >= p.S) continue;
        }
        const int slot = t < p.T ? t : p.S + (t - p.S) % (p.T - p.S);
        float f[8];
        if (is_v) get8<TYPE>(p.v, b * p.vb + (long long)(t - p0) * p.vm + g * p.vh + 8 * c, p.vec, f);
        else get8<TYPE>(p.k, b * p.kb + (long long)(t - p0) * p.km + g * p.kh + 8 * c, p.vec, f);
        uint4 w;
        if (p.f16) w = make_uint4(pack2<true>(f[0], f[1]), pack2<true>(f[2], f[3]), pack2<true>(f[4], f[5]), pack2<true>(f[6], f[7]));
        else w = make_uint4(pack2<false>(f[0], f[1]), pack2<false>(f[2], f[3]), pack2<false>(f[4], f[5]), pack2<false>(f[6], f[7]));
        *reinterpret_cast<uint4 *>((is_v ? p.to_v : p.to_k) + (((long long)b * p.Hkv + g) * p.T + slot) * p.D + 8 * c) = w;
    }
}

struct KvWs {
    size_t ml, o, own_ml, own_o, pre_ml, pre_o, total;
    long long own_ctas, pre_ctas;   // row tiles of the tile kernel (0: the split kernel's)
    int own_n, pre_most;            // parts of the own positions; of a prefix at most
};

// T, window, sinks: what a row tile sees at most sets the parts that it is cut into.
KvWs kv_ws(int B, int Hkv, int G, int D, long long M, int T, int W, int S, int P)
{
    KvWs w = {};
    const long long rows = M * G, prows = B * rows;
    const bool split_own = rows <= kKvFewRows, split_pre = P > 0 && prows <= kKvFewRows;
    const size_t slots = split_own ? (size_t)B * Hkv + (split_pre ? Hkv : 0) + kKvMaxCtas : 0;
    if (!split_own) {
        w.own_ctas = kv_row_tiles(rows, D) * Hkv * B;
        const long long seen = std::min<long long>((long long)W + S + 256 / G + 1, T);
        w.own_n = kv_tile_splits(w.own_ctas, (seen + 127) / 128, rows <= 128, P > 0 ? 0 : prows * Hkv);
    }
    if (P > 0 && !split_pre) {
        w.pre_ctas = kv_row_tiles(prows, D) * Hkv;
        w.pre_most = kv_tile_most(w.pre_ctas, false);
    }
    const size_t own = w.own_n > 1 || P > 0 ? (size_t)w.own_n * Hkv * prows : 0, pre = (size_t)w.pre_most * Hkv * prows;
    w.ml = 0;
    w.o = align_up(w.ml + slots * kKvFewRows * 8, 256);
    w.own_ml = align_up(w.o + slots * kKvFewRows * D * 4, 256);
    w.own_o = align_up(w.own_ml + own * 8, 256);
    w.pre_ml = align_up(w.own_o + own * D * 4, 256);
    w.pre_o = align_up(w.pre_ml + pre * 8, 256);
    w.total = align_up(w.pre_o + pre * D * 4, 256);
    return w;
}

}  // namespace

size_t kv_attn_workspace_bytes(int batch, int kv_heads, int group, int head_dim, long long M, int T, int window, int sinks, int P)
{
    return kv_ws(batch, kv_heads, group, head_dim, M, T, window ? window : kKvAll, sinks, P).total;
}

int launch_kv_append(const moe_kv &c, const moe_rows &k_new, const moe_rows &v_new, int M, const int32_t *pos,
                     const int32_t *counts, int *err, cudaStream_t stream)
{
    AppendCall p;
    memset(&p, 0, sizeof p);
    p.k = k_new.data_dev;
    p.kb = k_new.seq;
    p.km = k_new.row;
    p.kh = k_new.head;
    p.v = v_new.data_dev;
    p.vb = v_new.seq;
    p.vm = v_new.row;
    p.vh = v_new.head;
    p.to_k = static_cast<uint16_t *>(c.k_dev);
    p.to_v = static_cast<uint16_t *>(c.v_dev);
    p.pos = pos;
    p.counts = counts;
    p.err = err;
    p.B = c.batch;
    p.M = M;
    p.Hkv = c.kv_heads;
    p.D = c.head_dim;
    p.T = c.T_cap;
    p.S = c.window ? c.sinks : 0;
    p.limit = c.window ? kKvMaxPos : c.T_cap;
    p.f16 = c.type == MOE_F16;
    p.nring = std::min(M, c.T_cap - p.S);
    p.nfirst = std::min(M, p.S);
    const int unit = k_new.type == MOE_F32 ? 4 : 8;
    auto wide = [&](const moe_rows &r) {
        return reinterpret_cast<uintptr_t>(r.data_dev) % 16 == 0 && r.seq % unit == 0 && r.row % unit == 0 && r.head % unit == 0;
    };
    p.vec = wide(k_new) && wide(v_new);
    const long long all = 2LL * p.Hkv * (p.D / 8) * (p.nring + p.nfirst);
    const dim3 grid((unsigned)std::min<long long>((all + 255) / 256, std::max(1, 8192 / p.B)), p.B);
    auto *kernel = k_new.type == MOE_F32 ? kv_append_kernel<MOE_F32> : k_new.type == MOE_F16 ? kv_append_kernel<MOE_F16> : kv_append_kernel<MOE_BF16>;
    const cudaError_t e = launch_after(kernel, grid, 256, 0, 0, stream, p);
    if (e != cudaSuccess) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
    note_launch();
    return MOE_OK;
}

int launch_kv_attn(KvCall &p, void *ws, cudaStream_t stream)
{
    const KvWs w = kv_ws(p.B, p.Hkv, p.G, p.D, p.M, p.T, p.W, p.S, p.P);
    uint8_t *base = static_cast<uint8_t *>(ws);
    auto f = [&](size_t at) { return reinterpret_cast<float *>(base + at); };
    p.split_own = w.own_ctas == 0;
    p.split_prefix = p.P > 0 && w.pre_ctas == 0;
    p.late = 0;
    p.part_ml = f(w.ml);
    p.part_o = f(w.o);
    p.own = {0, f(w.own_o), f(w.own_ml)};
    p.prefix = {0, f(w.pre_o), f(w.pre_ml)};
    const long long merged = (long long)p.B * p.M * p.Hq;
    if (w.pre_ctas) {
        p.prefix.n = kv_tile_splits(w.pre_ctas, (p.P + 127) / 128, false, 0);
        const int rc = launch_kv_tiles(p, true, stream);
        if (rc) return rc;
        p.late = 1;   // the own positions' kernel runs beside
    }
    int grid = 1;
    if (w.own_ctas) {
        p.own.n = w.own_n;
        const int rc = launch_kv_tiles(p, false, stream);
        if (rc || (p.own.n == 1 && p.P == 0)) return rc;
    } else {
        // the line's length has to fit an int
        const long long seen = std::min<long long>((long long)p.W + p.S + p.M, p.T);
        const long long most = (seen / kKvTile + 2) * p.B * p.Hkv + (p.split_prefix ? ((long long)p.P / kKvTile + 1) * p.Hkv : 0);
        if (most > INT_MAX / 2) return MOE_ERR_UNSUPPORTED;
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess || dev < 0 || dev >= 64) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
        auto go = [&](auto kernel, int smem, int threads, int ctas, Once &once) {
            std::call_once(once.flag[dev], [&] {
                e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
                if (e == cudaSuccess)
                    e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                             (int)cudaSharedmemCarveoutMaxShared);
                if (e == cudaSuccess) e = cudaDeviceGetAttribute(&once.sms[dev], cudaDevAttrMultiProcessorCount, dev);
            });
            if (e == cudaSuccess && once.sms[dev] < 1) e = cudaErrorInvalidDevice;
            if (e != cudaSuccess) return;
            grid = (int)std::min<long long>(most, (long long)std::min(once.sms[dev], kMaxCtas) * ctas);
            e = launch_after(kernel, dim3(grid), threads, smem, 0, stream, p);
        };
#define KV_GO(F, D)                                                                         \
    do {                                                                                    \
        static Once once;                                                                   \
        static_assert(Lay<D>::total(MOE_KV_MAX_BATCH) <= kSmemMax, "shared memory");        \
        go(kv_split_kernel<F, D>, Lay<D>::total(p.B), Lay<D>::kThreads, Lay<D>::ctas, once); \
    } while (0)
#define KV_GO_F(F)                        \
    do {                                  \
        if (p.D == 256) KV_GO(F, 256);    \
        else if (p.D == 128) KV_GO(F, 128); \
        else KV_GO(F, 64);                \
    } while (0)
        if (p.f16) KV_GO_F(true);
        else KV_GO_F(false);
#undef KV_GO_F
#undef KV_GO
        if (e != cudaSuccess) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
        note_launch();
    }
    if (merged > INT_MAX) return MOE_ERR_UNSUPPORTED;
    const bool one = merged >= kMergeMany && p.Hq % kMergeWarps == 0;
    auto *merge = p.D == 256   ? (one ? kv_merge_kernel<256, true> : kv_merge_kernel<256, false>)
                  : p.D == 128 ? (one ? kv_merge_kernel<128, true> : kv_merge_kernel<128, false>)
                               : (one ? kv_merge_kernel<64, true> : kv_merge_kernel<64, false>);
    const cudaError_t e = launch_after(merge, dim3((unsigned)(one ? merged / kMergeWarps : merged)), 32 * kMergeWarps, 0, 0, stream, p, grid);
    if (e != cudaSuccess) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
    note_launch();
    return MOE_OK;
}

}  // namespace moe
