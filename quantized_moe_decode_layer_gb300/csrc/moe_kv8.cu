// The 8-bit key/value cache (moe_kv8.cuh): appending rows, reading values
// back, and eviction by accumulated attention weight.  The attention over it
// is moe_kv8_attn.cu.
#include <algorithm>
#include <mutex>

#include "moe_kv8.cuh"

namespace moe {
namespace {

// A block of positions of one head and tensor belongs to (block / 8) (D / 8)
// consecutive threads, 16 to 512 of them: a thread holds 8 consecutive values
// of 8 rows, so a block is read once, its maximum taken, and written from
// registers.  CTAs hold as many blocks as 256 threads do.
struct Place {
    int j, row, d, threads;        // block within the CTA's blocks, first of the thread's rows, dimension, threads per block
};
__device__ __forceinline__ Place place_of(int blk, int D)
{
    Place q;
    q.threads = (blk >> 3) * (D >> 3);
    const int r = threadIdx.x & (q.threads - 1);
    q.j = threadIdx.x / q.threads;
    q.row = r / (D >> 3);
    q.d = r % (D >> 3) * 8;
    return q;
}

// Maximum over a block's threads (a power of two); `red` holds a float per warp.
__device__ __forceinline__ float place_max(float v, const Place &q, float *red)
{
    for (int o = min(q.threads, 32) >> 1; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (q.threads <= 32) return v;
    const int warp = threadIdx.x >> 5, nw = q.threads >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    for (int w = 0; w < nw; ++w) v = fmaxf(v, red[(warp & ~(nw - 1)) + w]);
    return v;
}
int place_threads(int blk, int D) { return std::max(256, blk / 8 * (D / 8)); }
int place_blocks(int blk, int D) { return place_threads(blk, D) / (blk / 8 * (D / 8)); }

// ------------------------------------------------------------------ append
// The blocks that a sequence's new rows touch.  A block's step is the
// smallest that holds the new rows, and no smaller than that of its earlier
// rows, whose codes are rounded again when it grew.  Bound by the copy: two (four)
// bytes in and one out per value.
struct AppendParams {
    const void *src[2];            // new keys, values
    uint8_t *codes[2];
    float *scale[2];
    long long sb[2], sm[2], sh[2]; // strides of src in elements: sequence, row, head
    const int32_t *pos, *counts;
    int *err;
    int M, Hkv, D, T_cap, blk, nblk;
    int vec;                       // 16-byte loads of 8 (4) consecutive values
};

// 8 consecutive elements as they lie, and their values.
template <int TYPE>
struct Raw {
    uint32_t w[TYPE == MOE_F32 ? 8 : 4];

    __device__ __forceinline__ void load(const void *src, long long i, bool vec)
    {
        const uint8_t *p = static_cast<const uint8_t *>(src) + i * (TYPE == MOE_F32 ? 4 : 2);
        if (vec) {
#pragma unroll
            for (int j = 0; j < (TYPE == MOE_F32 ? 2 : 1); ++j)
                *reinterpret_cast<uint4 *>(w + 4 * j) = __ldg(reinterpret_cast<const uint4 *>(p) + j);
        } else if (TYPE == MOE_F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[TYPE == MOE_F32 ? j : 0] = __ldg(reinterpret_cast<const uint32_t *>(p) + j);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(p) + 2 * j) |
                       (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(p) + 2 * j + 1) << 16;
        }
    }
    // Largest of m and the magnitudes' bits, which order as the magnitudes do:
    // two 16-bit halves, or one word.
    __device__ __forceinline__ uint32_t amax(uint32_t m) const
    {
#pragma unroll
        for (int j = 0; j < (TYPE == MOE_F32 ? 8 : 4); ++j)
            m = TYPE == MOE_F32 ? max(m, w[j] & 0x7FFFFFFFu) : __vmaxu2(m, w[j] & 0x7FFF7FFFu);
        return m;
    }
    // Their value; infinite or NaN: not finite.
    static __device__ __forceinline__ float magnitude(uint32_t m)
    {
        if (TYPE == MOE_F32) return __uint_as_float(m);
        m = max(m & 0xFFFFu, m >> 16);
        return TYPE == MOE_BF16 ? __uint_as_float(m << 16) : __half2float(__ushort_as_half((uint16_t)m));
    }
    // CLEAN: with infinities as the type's largest value and NaN as zero.
    template <bool CLEAN>
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
        const float big = TYPE == MOE_BF16 ? __uint_as_float(0x7F7F0000u) : TYPE == MOE_F16 ? 65504.f : __uint_as_float(0x7F7FFFFFu);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (TYPE == MOE_F32) v[j] = __uint_as_float(w[TYPE == MOE_F32 ? j : 0]);
            else if (TYPE == MOE_BF16) v[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
            else v[j] = __half2float(__ushort_as_half((uint16_t)(w[j / 2] >> (16 * (j & 1)))));
            if (CLEAN && !(fabsf(v[j]) <= big)) v[j] = v[j] != v[j] ? 0.f : copysignf(big, v[j]);
        }
    }
};

template <int FMT, int TYPE, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? (TYPE == MOE_F32 ? 1 : 2) : TYPE == MOE_F32 ? 2 : 4) kv8_append_kernel(const AppendParams p)
{
    __shared__ float red[16];
    after_previous();
    const int b = blockIdx.z, g = blockIdx.y >> 1, which = blockIdx.y & 1;
    int p0;
    bool bad;
    const int n = kv8_rows(p.pos, p.counts, b, p.M, p.T_cap, p0, bad);
    if (bad && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(p.err, kKv8ErrRange);
    if (n <= 0) return;
    const Place q = place_of(p.blk, p.D);
    const int j = p0 / p.blk + blockIdx.x * (blockDim.x / q.threads) + q.j, t0 = j * p.blk;
    const int first = max(t0, p0), last = min(t0 + p.blk, p0 + n);   // new rows: positions first .. last - 1, none past the call's blocks
    const size_t head = (size_t)b * p.Hkv + g;
    const long long s0 = b * p.sb[which] + g * p.sh[which] + q.d, sm = p.sm[which];
    Raw<TYPE> raw[8];
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int t = t0 + q.row + i * (p.blk >> 3);
        if (t >= first && t < last) raw[i].load(p.src[which], s0 + (t - p0) * sm, p.vec);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int t = t0 + q.row + i * (p.blk >> 3);
        if (t >= first && t < last) most = raw[i].amax(most);
    }
    float amax = Raw<TYPE>::magnitude(most);
    const bool odd = !(amax <= __uint_as_float(0x7F7FFFFFu));        // an infinity or NaN among the thread's values
    if (odd) {
        atomicOr(p.err, kKv8ErrNonFinite);
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int t = t0 + q.row + i * (p.blk >> 3);
            if (t >= first && t < last) {
                float v[8];
                raw[i].template values<true>(v);
#pragma unroll
                for (int c = 0; c < 8; ++c) amax = fmaxf(amax, fabsf(v[c]));
            }
        }
    }
    const bool mixed = first > t0 && first < last;                   // earlier rows in the block
    float *scale = p.scale[which] + head * p.nblk + j;
    const float was = mixed ? *scale : 0.f;
    amax = place_max(amax, q, red);
    __syncthreads();                                                 // every thread has read the old step
    if (first >= last) return;
    int e = step_exp<FMT>(amax);
    uint8_t *codes = p.codes[which] + head * p.T_cap * p.D + q.d;
    if (mixed) {
        const int e_old = max((int)(__float_as_uint(was) >> 23) - 127, kKv8MinExp);
        if (e > e_old) {
            // 2^(e_old - e), zero where no code can survive (or the block had no step)
            const float down = was > 0.f && e - e_old <= 126 ? pow2f(e_old - e) : 0.f;
            for (int t = t0 + q.row; t < first; t += p.blk >> 3) {
                uint2 *w = reinterpret_cast<uint2 *>(codes + (size_t)t * p.D);
                *w = recode8<FMT>(*w, down);
            }
        }
        e = max(e, e_old);
    }
    if (q.row == 0 && q.d == 0) *scale = pow2f(e);
    const float inv = pow2f(-e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int t = t0 + q.row + i * (p.blk >> 3);
        if (t >= first && t < last) {
            float v[8];
            if (odd) raw[i].template values<true>(v);
            else raw[i].template values<false>(v);
            *reinterpret_cast<uint2 *>(codes + (size_t)t * p.D) =
                make_uint2(encode4<FMT>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                           encode4<FMT>(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
        }
    }
}

// -------------------------------------------------------------------- read
// bf16 values of positions start[b] .. start[b] + n - 1 (zero outside the
// cache or from lens[b] on): one thread per 8 values of keys and of values.
struct ReadParams {
    const uint8_t *codes[2];
    const float *scale[2];
    uint16_t *out[2];              // [B][n][Hkv][D]
    const int32_t *start, *lens;   // NULL: 0, T_cap
    int n, Hkv, D, T_cap, blk_log, nblk;
};

template <int FMT>
__global__ void __launch_bounds__(256) kv8_read_kernel(const ReadParams p)
{
    after_previous();
    const int lanes = p.D / 8, b = blockIdx.y;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;   // (row, head, 8 values)
    if (i >= (long long)p.n * p.Hkv * lanes) return;
    const int d = (int)(i % lanes) * 8, g = (int)(i / lanes % p.Hkv), r = (int)(i / lanes / p.Hkv);
    const long long t = (long long)(p.start ? p.start[b] : 0) + r;
    const int end = p.lens ? min(p.lens[b], p.T_cap) : p.T_cap;
    const size_t head = (size_t)b * p.Hkv + g;
    const bool in = t >= 0 && t < end;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        uint4 o = make_uint4(0u, 0u, 0u, 0u);
        if (in) {
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p.codes[which] + (head * p.T_cap + t) * p.D + d));
            const float s = __ldg(p.scale[which] + head * p.nblk + (t >> p.blk_log));
            float a[4], c[4];
            decode4<FMT>(w.x, a);
            decode4<FMT>(w.y, c);
            __nv_bfloat162 h[4] = {__floats2bfloat162_rn(a[0] * s, a[1] * s), __floats2bfloat162_rn(a[2] * s, a[3] * s),
                                   __floats2bfloat162_rn(c[0] * s, c[1] * s), __floats2bfloat162_rn(c[2] * s, c[3] * s)};
            // 2^128, which a code may stand for, is no bf16: the largest finite one
            // (8 heads of 16K rows of 256 33.9 us for 33.1; by the saturating conversion, or a
            // branch on the step, 37.7)
            const __nv_bfloat162 top = __halves2bfloat162(__ushort_as_bfloat16(0x7F7F), __ushort_as_bfloat16(0x7F7F));
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = __hmax2(__hmin2(h[k], top), __hneg2(top));
            o = *reinterpret_cast<uint4 *>(h);
        }
        *reinterpret_cast<uint4 *>(p.out[which] + ((size_t)b * p.n * p.Hkv * lanes + i) * 8) = o;
    }
}

// ------------------------------------------------------------------- evict
// Selection: a cluster of 1 to 8 CTAs per (sequence, head), a slice of the
// positions each.  Of n > budget positions the first `sinks` and last `recent`
// stay, and the rest are ranked by weight (larger first, then the lower
// position).  A radix select over 32-bit keys, 8 bits at a time, finds the
// weight of the last one that stays and how many of its equals do; then every
// warp counts what its part keeps, and writes it behind what the parts before
// it do.  Bound by latency: four passes over keys in shared memory (in L2 where
// a slice has more than 16K), a cluster barrier each, the slices' 256 counts
// added up through distributed shared memory (2048 counts, in three passes,
// took 25 us where these take fewer), and no more passes once all of a bin stays:
// distinct weights take three.  (8 heads of 32K: 13.4 us, 8 of 128K: 25; with
// the keys in registers and 32 copies of the counts 15.4 and 23.)  Weights share
// few exponents, so a CTA counts in 8 copies, a lane in its own.
constexpr int kSelThreads = 1024, kSelKeys = 16384, kSelBins = 256, kSelCopies = 8, kSelCtas = 8, kSelSlice = 4096;

struct EvictParams {
    const uint8_t *codes[2];
    const float *scale[2];
    const float *acc;
    const int32_t *lens;
    uint8_t *dcodes[2];
    float *dscale[2];
    float *dacc;                   // or NULL
    int32_t *idx, *lens_out;
    int *err;
    int Hkv, D, T_cap, blk, blk_log, nblk, dT_cap, dnblk, budget, sinks, recent;
};

// Larger weight, larger key; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float v)
{
    const uint32_t u = __float_as_uint(v + 0.f);
    if (v != v) return 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ void cluster_sync(int ctas)
{
    if (ctas == 1) __syncthreads();
    else asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Word of another CTA of the cluster at the place that p has in this one.
__device__ __forceinline__ int peer(const int *p, int rank)
{
    uint32_t a;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__global__ void __launch_bounds__(kSelThreads) kv8_select_kernel(const EvictParams p, int ctas)
{
    extern __shared__ __align__(16) uint32_t sel[];
    static_assert(__alignof__(sel) >= alignof(int4), "the counts are read four at a time");
    int *copies = reinterpret_cast<int *>(sel);                     // [bins][copies]
    float *weights = reinterpret_cast<float *>(sel + kSelBins * kSelCopies);   // [kSelKeys]: this slice's
    __shared__ int hist[2][kSelBins], wsum[32], weq[32], total[2], sh_digit, sh_need, sh_all;   // hist: the passes take turns
    after_previous();
    const int rank = blockIdx.x % ctas, g = blockIdx.x / ctas, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = p.lens[b];
    if (len > p.T_cap && blockIdx.x == 0 && tid == 0) atomicOr(p.err, kKv8ErrRange);
    const int n = max(0, min(len, p.T_cap)), kept = min(n, p.budget);
    const size_t head = (size_t)b * p.Hkv + g;
    const float *acc = p.acc + head * p.T_cap;
    int32_t *idx = p.idx + head * p.budget;
    float *dacc = p.dacc ? p.dacc + head * p.dT_cap : nullptr;
    if (blockIdx.x == 0 && tid == 0) p.lens_out[b] = kept;
    for (int i = kept + rank * kSelThreads + tid; i < p.budget; i += ctas * kSelThreads) idx[i] = -1;
    if (n <= p.budget) {
        for (int i = rank * kSelThreads + tid; i < n; i += ctas * kSelThreads) {
            idx[i] = i;
            if (dacc) dacc[i] = acc[i];
        }
        return;
    }
    const int lo = p.sinks, hi = n - p.recent;                      // candidates: positions lo .. hi - 1
    int need = p.budget - p.sinks - p.recent;                       // 0 <= need < hi - lo
    const bool any = need > 0;
    // this CTA's positions s0 .. s1 - 1, a warp's w0 .. w1 - 1
    const int slice = ((n + ctas - 1) / ctas + 31) & ~31, s0 = min(rank * slice, n), s1 = min(s0 + slice, n);
    const int part = ((slice + 31) / 32 + 31) & ~31, w0 = min(s0 + warp * part, s1), w1 = min(w0 + part, s1);
    const bool local = slice <= kSelKeys;
    if (local) {
#pragma unroll 4
        for (int t = s0 + tid; t < s1; t += kSelThreads) weights[t - s0] = acc[t];
    }
    auto weight = [&](int t) { return local ? weights[t - s0] : acc[t]; };
    auto key = [&](int t) { return weight_key(weight(t)); };
    uint32_t prefix = 0u, mask = 0u;
    const int c0 = max(lo, s0), c1 = min(hi, s1);
    bool open = any;                                                // the bin holds more than stay
    for (int pass = 0; pass < 4 && open; ++pass) {
        const int shift = 24 - 8 * pass;
        int *h = hist[pass & 1];
        for (int i = tid; i < kSelBins * kSelCopies; i += kSelThreads) copies[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int t = c0 + tid; t < c1; t += kSelThreads) {
            const uint32_t k = key(t);
            if ((k & mask) == prefix) atomicAdd(&copies[((k >> shift) & 255u) * kSelCopies + (lane & (kSelCopies - 1))], 1);
        }
        __syncthreads();
        const int bin = 255 - tid;                                  // from the largest down
        if (tid < kSelBins) {
            const int4 u = reinterpret_cast<const int4 *>(copies)[2 * bin], v = reinterpret_cast<const int4 *>(copies)[2 * bin + 1];
            h[bin] = u.x + u.y + u.z + u.w + v.x + v.y + v.z + v.w;
        }
        cluster_sync(ctas);
        // the bin in which the need-th largest lies
        int c = 0, before = 0;
        if (tid < kSelBins) {
            if (ctas == 1) c = h[bin];
            else {
                int v[kSelCtas];                                    // all on their way at once
#pragma unroll
                for (int r = 0; r < kSelCtas; ++r) v[r] = r < ctas ? peer(h + bin, r) : 0;
#pragma unroll
                for (int r = 0; r < kSelCtas; ++r) c += v[r];
            }
            before = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xFFFFFFFFu, before, o);
                if (lane >= o) before += u;
            }
            if (lane == 31) wsum[warp] = before;
        }
        __syncthreads();
        if (tid < kSelBins) {
            for (int w = 0; w < warp; ++w) before += wsum[w];
            before -= c;
            if (before < need && need <= before + c) {
                sh_digit = bin;
                sh_need = need - before;
                sh_all = need == before + c;
            }
        }
        __syncthreads();
        prefix |= (uint32_t)sh_digit << shift;
        mask |= 255u << shift;
        need = sh_need;
        open = !sh_all;
    }
    if (!any) __syncthreads();
    // kept: sinks, recent, keys above `prefix` in the digits seen, and the first `need` equal to it
    auto kind = [&](int t, bool &above, bool &equal) {
        above = equal = false;
        if (t >= w1) return;
        if (t < lo || t >= hi) above = true;
        else if (any) {
            const uint32_t k = key(t) & mask;
            above = k > prefix;
            equal = k == prefix;
        }
    };
    int na = 0, ne = 0;
#pragma unroll 4
    for (int t = w0 + lane; t - lane < w1; t += 32) {
        bool above, equal;
        kind(t, above, equal);
        na += __popc(__ballot_sync(0xFFFFFFFFu, above));
        ne += __popc(__ballot_sync(0xFFFFFFFFu, equal));
    }
    __syncthreads();                                                // wsum is read
    if (lane == 0) {
        wsum[warp] = na;
        weq[warp] = ne;
    }
    __syncthreads();
    if (warp == 0) {
        const int a = __reduce_add_sync(0xFFFFFFFFu, wsum[lane]), q = __reduce_add_sync(0xFFFFFFFFu, weq[lane]);
        if (lane == 0) {
            total[0] = a;
            total[1] = q;
        }
    }
    cluster_sync(ctas);
    int a0 = 0, e0 = 0;                                             // above and equal before this warp's part
    if (lane < rank) {
        a0 = peer(&total[0], lane);
        e0 = peer(&total[1], lane);
    }
    if (lane < warp) {
        a0 += wsum[lane];
        e0 += weq[lane];
    }
    a0 = __reduce_add_sync(0xFFFFFFFFu, a0);
    e0 = __reduce_add_sync(0xFFFFFFFFu, e0);
#pragma unroll 4
    for (int t = w0 + lane; t - lane < w1; t += 32) {
        bool above, equal;
        kind(t, above, equal);
        const unsigned below = (1u << lane) - 1u, be = __ballot_sync(0xFFFFFFFFu, equal), ba = __ballot_sync(0xFFFFFFFFu, above);
        const int le = e0 + __popc(be & below);
        if (above || (equal && le < need)) {
            const int i = a0 + __popc(ba & below) + min(le, need);
            idx[i] = t;
            if (dacc) dacc[i] = weight(t);
        }
        a0 += __popc(ba);
        e0 += __popc(be);
    }
    cluster_sync(ctas);                                             // nobody leaves while its words are read
}

// Moving: a destination block's step is the smallest that holds its values; a
// code whose own step was smaller is rounded to it, one whose step was larger
// is exact.  As many threads to a block as above, here with 16 codes of 4 rows
// each.  Bound by gathering rows of D bytes, hence four CTAs on an SM (three:
// 8 heads of 16K rows of 256 take 3 us longer), whose 64 registers a thread spill 16 bytes.
template <int FMT, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 2 : 4) kv8_move_kernel(const EvictParams p)
{
    __shared__ float red[16];
    const int g = blockIdx.y >> 1, which = blockIdx.y & 1, b = blockIdx.z;
    Place q = place_of(p.blk, p.D);
    const int r = threadIdx.x & (q.threads - 1), step = p.blk >> 2;
    q.row = r / (p.D >> 4);
    q.d = r % (p.D >> 4) * 16;
    place_next();
    wait_for_previous();
    const int kept = __ldcg(p.lens_out + b), j = blockIdx.x * (THREADS / q.threads) + q.j, i0 = j * p.blk;
    if ((int)(blockIdx.x * (THREADS / q.threads)) * p.blk >= kept) return;
    const size_t head = (size_t)b * p.Hkv + g;
    const uint8_t *src = p.codes[which] + head * p.T_cap * p.D + q.d;
    const float *scale = p.scale[which] + head * p.nblk;
    const int32_t *idx = p.idx + head * p.budget;
    uint4 w[4];
    float s[4], amax = 0.f;
    int t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = i0 + q.row + i * step;
        t[i] = at < kept ? __ldcg(idx + at) : -1;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        s[i] = 0.f;
        if (t[i] >= 0) {
            w[i] = __ldg(reinterpret_cast<const uint4 *>(src + (size_t)t[i] * p.D));
            s[i] = __ldg(scale + (t[i] >> p.blk_log));
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        amax = fmaxf(amax, fmaxf(amax8<FMT>(make_uint2(w[i].x, w[i].y)), amax8<FMT>(make_uint2(w[i].z, w[i].w))) * s[i]);
    amax = place_max(amax, q, red);
    if (i0 >= kept) return;
    const int e = step_exp<FMT>(amax);
    const float inv = pow2f(-e);
    if (r == 0) p.dscale[which][head * p.dnblk + j] = pow2f(e);
    uint8_t *dst = p.dcodes[which] + head * p.dT_cap * p.D + q.d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i0 + q.row + i * step >= kept) continue;
        // no more than 2^17, see recode4; a row of zeros may have any step
        const float ratio = fminf(s[i] * inv, 131072.f);
        if (ratio != 1.f)
            w[i] = make_uint4(recode4<FMT>(w[i].x, ratio), recode4<FMT>(w[i].y, ratio), recode4<FMT>(w[i].z, ratio),
                              recode4<FMT>(w[i].w, ratio));
        *reinterpret_cast<uint4 *>(dst + (size_t)(i0 + q.row + i * step) * p.D) = w[i];
    }
}

int ilog2(int v)
{
    int r = 0;
    while ((1 << r) < v) ++r;
    return r;
}

int launched(cudaError_t e)
{
    if (e != cudaSuccess) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
    note_launch();
    return MOE_OK;
}

}  // namespace

int launch_kv8_append(const moe_kv8 &c, const moe_rows &k_new, const moe_rows &v_new, int M, const int32_t *pos,
                      const int32_t *counts, int *err, cudaStream_t stream)
{
    AppendParams p;
    const int type = k_new.type, unit = type == MOE_F32 ? 4 : 8;
    p.vec = 1;
    for (int i = 0; i < 2; ++i) {
        const moe_rows &r = i ? v_new : k_new;
        p.src[i] = r.data_dev;
        p.sb[i] = r.seq;
        p.sm[i] = r.row;
        p.sh[i] = r.head;
        if (reinterpret_cast<uintptr_t>(r.data_dev) % 16 || r.seq % unit || r.row % unit || r.head % unit) p.vec = 0;
    }
    p.codes[0] = static_cast<uint8_t *>(c.k_dev);
    p.codes[1] = static_cast<uint8_t *>(c.v_dev);
    p.scale[0] = c.k_scale_dev;
    p.scale[1] = c.v_scale_dev;
    p.pos = pos;
    p.counts = counts;
    p.err = err;
    p.M = M;
    p.Hkv = c.kv_heads;
    p.D = c.head_dim;
    p.T_cap = c.T_cap;
    p.blk = c.block;
    p.nblk = c.T_cap / c.block;
    const int per = place_blocks(c.block, c.head_dim), threads = place_threads(c.block, c.head_dim);
    const dim3 grid((min((M - 1) / c.block + 2, p.nblk) + per - 1) / per, 2 * c.kv_heads, c.batch);
    cudaError_t e;
#define KV8_APPEND(F, T)                                                                    \
    do {                                                                                    \
        if (threads == 256) e = launch_after(kv8_append_kernel<F, T, 256>, grid, 256, 0, 0, stream, p); \
        else e = launch_after(kv8_append_kernel<F, T, 512>, grid, 512, 0, 0, stream, p);    \
    } while (0)
    if (c.format == MOE_KV8_INT8) {
        if (type == MOE_BF16) KV8_APPEND(MOE_KV8_INT8, MOE_BF16);
        else if (type == MOE_F16) KV8_APPEND(MOE_KV8_INT8, MOE_F16);
        else KV8_APPEND(MOE_KV8_INT8, MOE_F32);
    } else {
        if (type == MOE_BF16) KV8_APPEND(MOE_KV8_E4M3, MOE_BF16);
        else if (type == MOE_F16) KV8_APPEND(MOE_KV8_E4M3, MOE_F16);
        else KV8_APPEND(MOE_KV8_E4M3, MOE_F32);
    }
#undef KV8_APPEND
    return launched(e);
}

int launch_kv8_read(const moe_kv8 &c, const int32_t *start, int n, const int32_t *lens, uint16_t *k_out, uint16_t *v_out,
                    cudaStream_t stream)
{
    ReadParams p;
    p.codes[0] = static_cast<const uint8_t *>(c.k_dev);
    p.codes[1] = static_cast<const uint8_t *>(c.v_dev);
    p.scale[0] = c.k_scale_dev;
    p.scale[1] = c.v_scale_dev;
    p.out[0] = k_out;
    p.out[1] = v_out;
    p.start = start;
    p.lens = lens;
    p.n = n;
    p.Hkv = c.kv_heads;
    p.D = c.head_dim;
    p.T_cap = c.T_cap;
    p.blk_log = ilog2(c.block);
    p.nblk = c.T_cap / c.block;
    const long long items = (long long)n * c.kv_heads * (c.head_dim / 8);
    const dim3 grid((unsigned)((items + 255) / 256), c.batch);
    return launched(launch_after(c.format == MOE_KV8_INT8 ? kv8_read_kernel<MOE_KV8_INT8> : kv8_read_kernel<MOE_KV8_E4M3>, grid,
                                 256, 0, 0, stream, p));
}

int launch_kv8_evict(const moe_kv8 &c, const moe_kv8 &d, const int32_t *lens, const float *acc, int budget, int sinks,
                     int recent, float *dacc, int32_t *idx, int32_t *lens_out, int *err, cudaStream_t stream)
{
    EvictParams p;
    p.codes[0] = static_cast<const uint8_t *>(c.k_dev);
    p.codes[1] = static_cast<const uint8_t *>(c.v_dev);
    p.scale[0] = c.k_scale_dev;
    p.scale[1] = c.v_scale_dev;
    p.acc = acc;
    p.lens = lens;
    p.dcodes[0] = static_cast<uint8_t *>(d.k_dev);
    p.dcodes[1] = static_cast<uint8_t *>(d.v_dev);
    p.dscale[0] = d.k_scale_dev;
    p.dscale[1] = d.v_scale_dev;
    p.dacc = dacc;
    p.idx = idx;
    p.lens_out = lens_out;
    p.err = err;
    p.Hkv = c.kv_heads;
    p.D = c.head_dim;
    p.T_cap = c.T_cap;
    p.blk = c.block;
    p.blk_log = ilog2(c.block);
    p.nblk = c.T_cap / c.block;
    p.dT_cap = d.T_cap;
    p.dnblk = d.T_cap / d.block;
    p.budget = budget;
    p.sinks = sinks;
    p.recent = recent;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
    // CTAs per head: as many as slices of 4K positions of a full cache (8 heads of
    // 32K: 1, 2, 4, 8 CTAs take 33, 22, 16, 14 us; one of 2K in two slices 10 for 8)
    int ctas = 1;
    while (ctas < kSelCtas && c.T_cap > kSelSlice * ctas) ctas *= 2;
    const int smem = (kSelBins * kSelCopies + kSelKeys) * (int)sizeof(uint32_t);
    static std::once_flag once[64];
    std::call_once(once[dev], [&] {
        e = cudaFuncSetAttribute((const void *)kv8_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e == cudaSuccess)
        e = launch_after(kv8_select_kernel, dim3(ctas * c.kv_heads, c.batch), kSelThreads, smem, ctas, stream, p, ctas);
    if (const int rc = launched(e)) return rc;
    const int per = place_blocks(c.block, c.head_dim), threads = place_threads(c.block, c.head_dim);
    const dim3 grid(((budget + c.block - 1) / c.block + per - 1) / per, 2 * c.kv_heads, c.batch);
    const bool i8 = c.format == MOE_KV8_INT8;
    return launched(
        threads == 256
            ? launch_after(i8 ? kv8_move_kernel<MOE_KV8_INT8, 256> : kv8_move_kernel<MOE_KV8_E4M3, 256>, grid, 256, 0, 0, stream, p)
            : launch_after(i8 ? kv8_move_kernel<MOE_KV8_INT8, 512> : kv8_move_kernel<MOE_KV8_E4M3, 512>, grid, 512, 0, 0, stream, p));
}

}  // namespace moe
