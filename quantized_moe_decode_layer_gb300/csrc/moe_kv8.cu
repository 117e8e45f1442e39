// The 8-bit key/value cache (moe_kv8.cuh): appending rows, reading values
// back, and eviction by accumulated attention weight.  The attention over it
// is moe_kv8_attn.cu.
#include "moe_kv8.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------------ append
// One CTA per (block of positions that the rows can touch, head and tensor,
// sequence).  The block's step is the smallest that holds the new rows, and
// no smaller than that of its earlier rows, whose codes are rounded again
// when it grew.  A thread holds 8 consecutive values of a row.
constexpr int kAppThreads = 256;

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

template <int TYPE>
__device__ __forceinline__ void load8(const void *src, long long i, int vec, float (&v)[8])
{
    if (TYPE == MOE_F32) {
        const float *p = static_cast<const float *>(src) + i;
        if (vec) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __ldg(p + j);
        }
        return;
    }
    uint16_t h[8];
    const uint16_t *p = static_cast<const uint16_t *>(src) + i;
    if (vec) {
        *reinterpret_cast<uint4 *>(h) = __ldg(reinterpret_cast<const uint4 *>(p));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = __ldg(p + j);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = TYPE == MOE_BF16 ? __uint_as_float((uint32_t)h[j] << 16) : __half2float(__ushort_as_half(h[j]));
}

// Infinities become the type's largest value, NaN zero; says whether there was any.
template <int TYPE>
__device__ __forceinline__ bool make_finite(float (&v)[8])
{
    const float big = TYPE == MOE_BF16 ? __uint_as_float(0x7F7F0000u) : TYPE == MOE_F16 ? 65504.f : __uint_as_float(0x7F7FFFFFu);
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (!(fabsf(v[j]) <= big)) {
            odd = true;
            v[j] = v[j] != v[j] ? 0.f : copysignf(big, v[j]);
        }
    return odd;
}

template <int FMT, int TYPE>
__global__ void __launch_bounds__(kAppThreads) kv8_append_kernel(const AppendParams p)
{
    __shared__ float red[33];
    const int b = blockIdx.z, g = blockIdx.y >> 1, which = blockIdx.y & 1;
    int p0;
    bool bad;
    const int n = kv8_rows(p.pos, p.counts, b, p.M, p.T_cap, p0, bad);
    if (bad && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(p.err, kKv8ErrRange);
    if (n <= 0) return;
    const int j = p0 / p.blk + blockIdx.x, t0 = j * p.blk;
    if (t0 >= p0 + n) return;
    const int first = max(t0, p0), last = min(t0 + p.blk, p0 + n);   // new rows: positions first .. last - 1
    const int lanes = p.D / 8, r0 = threadIdx.x / lanes, d = threadIdx.x % lanes * 8, dr = kAppThreads / lanes;
    const long long s0 = b * p.sb[which] + g * p.sh[which] + d, sm = p.sm[which];
    float amax = 0.f;
    bool odd = false;
    for (int t = first + r0; t < last; t += dr) {
        float v[8];
        load8<TYPE>(p.src[which], s0 + (t - p0) * sm, p.vec, v);
        odd |= make_finite<TYPE>(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
    }
    if (odd) atomicOr(p.err, kKv8ErrNonFinite);
    amax = cta_max(amax, red);
    int e = step_exp<FMT>(amax);
    const size_t head = (size_t)b * p.Hkv + g;
    float *scale = p.scale[which] + head * p.nblk + j;
    uint8_t *codes = p.codes[which] + head * p.T_cap * p.D + d;
    if (first > t0) {
        const float was = *scale;
        const int e_old = max((int)(__float_as_uint(was) >> 23) - 127, kKv8MinExp);
        if (e > e_old) {
            // 2^(e_old - e), zero where no code can survive (or the block had no step)
            const float down = was > 0.f && e - e_old <= 126 ? pow2f(e_old - e) : 0.f;
            for (int t = t0 + r0; t < first; t += dr) {
                uint2 *w = reinterpret_cast<uint2 *>(codes + (size_t)t * p.D);
                *w = recode8<FMT>(*w, down);
            }
        }
        e = max(e, e_old);
    }
    __syncthreads();   // every thread has read the old step
    if (threadIdx.x == 0) *scale = pow2f(e);
    const float inv = pow2f(-e);
    for (int t = first + r0; t < last; t += dr) {
        float v[8];
        load8<TYPE>(p.src[which], s0 + (t - p0) * sm, p.vec, v);
        make_finite<TYPE>(v);
        *reinterpret_cast<uint2 *>(codes + (size_t)t * p.D) =
            make_uint2(encode4<FMT>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                       encode4<FMT>(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
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
            o = *reinterpret_cast<uint4 *>(h);
        }
        *reinterpret_cast<uint4 *>(p.out[which] + ((size_t)b * p.n * p.Hkv * lanes + i) * 8) = o;
    }
}

// ------------------------------------------------------------------- evict
// Selection: one CTA per (sequence, head).  Of n > budget positions the
// first `sinks` and last `recent` stay, and the rest are ranked by weight
// (larger first, then the lower position): a radix select over 32-bit keys
// finds the weight of the last one that stays and how many of its equals do,
// and a scan in position order writes the kept positions.
constexpr int kSelThreads = 1024;

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

__device__ __forceinline__ int cta_sum(int v, int *red)
{
    v = __reduce_add_sync(0xFFFFFFFFu, v);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) red[warp] = v;
    __syncthreads();
    int s = 0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += red[w];
    return s;
}

__global__ void __launch_bounds__(kSelThreads) kv8_select_kernel(const EvictParams p)
{
    __shared__ unsigned hist[256];
    __shared__ int red[32], sh_digit, sh_need;
    const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = p.lens[b];
    if (len > p.T_cap && g == 0 && tid == 0) atomicOr(p.err, kKv8ErrRange);
    const int n = max(0, min(len, p.T_cap)), kept = min(n, p.budget);
    const size_t head = (size_t)b * p.Hkv + g;
    const float *acc = p.acc + head * p.T_cap;
    int32_t *idx = p.idx + head * p.budget;
    if (g == 0 && tid == 0) p.lens_out[b] = kept;
    for (int i = kept + tid; i < p.budget; i += kSelThreads) idx[i] = -1;
    if (n <= p.budget) {
        for (int i = tid; i < n; i += kSelThreads) {
            idx[i] = i;
            if (p.dacc) p.dacc[head * p.dT_cap + i] = acc[i];
        }
        return;
    }
    const int lo = p.sinks, hi = n - p.recent;          // candidates: positions lo .. hi - 1
    int need = p.budget - p.sinks - p.recent;           // 0 <= need < hi - lo
    uint32_t prefix = 0u;
    for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0u;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
        for (int t = lo + tid; t < hi; t += kSelThreads) {
            const uint32_t k = weight_key(acc[t]);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {
            // digits from the largest down: the one in which the need-th largest lies
            int before = 0;
            for (int base = 248; base >= 0; base -= 8) {
                int c = 0;
                for (int i = 0; i < 8; ++i) c += (int)hist[base + i];
                if (before + c >= need) {
                    int dgt = base + 7;
                    while (before + (int)hist[dgt] < need) before += (int)hist[dgt--];
                    if (lane == 0) { sh_digit = dgt; sh_need = need - before; }
                    break;
                }
                before += c;
            }
        }
        __syncthreads();
        prefix |= (uint32_t)sh_digit << shift;
        need = sh_need;
        __syncthreads();
    }
    // kept: sinks, recent, keys above `prefix`, and the first `need` equal to it
    const bool any = p.budget > p.sinks + p.recent;
    int done = 0, equals = 0;
    for (int base = 0; base < n; base += kSelThreads) {
        const int t = base + tid;
        bool above = false, equal = false;
        if (t < n) {
            if (t < lo || t >= hi) above = true;
            else if (any) {
                const uint32_t k = weight_key(acc[t]);
                above = k > prefix;
                equal = k == prefix;
            }
        }
        const unsigned below = (1u << lane) - 1u;
        const unsigned be = __ballot_sync(0xFFFFFFFFu, equal);
        __syncthreads();
        if (lane == 0) red[warp] = __popc(be);
        __syncthreads();
        int before = equals, total = 0;
        for (int w = 0; w < 32; ++w) {
            before += w < warp ? red[w] : 0;
            total += red[w];
        }
        const bool keep = above || (equal && before + __popc(be & below) < need);
        equals += total;
        const unsigned bk = __ballot_sync(0xFFFFFFFFu, keep);
        __syncthreads();
        if (lane == 0) red[warp] = __popc(bk);
        __syncthreads();
        int at = done;
        total = 0;
        for (int w = 0; w < 32; ++w) {
            at += w < warp ? red[w] : 0;
            total += red[w];
        }
        if (keep) {
            const int i = at + __popc(bk & below);
            idx[i] = t;
            if (p.dacc) p.dacc[head * p.dT_cap + i] = acc[t];
        }
        done += total;
    }
}

// Moving: one CTA per (destination block, head and tensor, sequence).  The
// block's step is the smallest that holds its values; a code whose own step
// was smaller is rounded to it, one whose step was larger is exact.
constexpr int kMoveThreads = 256;

template <int FMT>
__global__ void __launch_bounds__(kMoveThreads) kv8_move_kernel(const EvictParams p)
{
    __shared__ float red[33];
    const int j = blockIdx.x, g = blockIdx.y >> 1, which = blockIdx.y & 1, b = blockIdx.z;
    const int kept = p.lens_out[b], i0 = j * p.blk, i1 = min(i0 + p.blk, kept);
    if (i0 >= kept) return;
    const size_t head = (size_t)b * p.Hkv + g;
    const int lanes = p.D / 8, r0 = threadIdx.x / lanes, d = threadIdx.x % lanes * 8, dr = kMoveThreads / lanes;
    const uint8_t *src = p.codes[which] + head * p.T_cap * p.D + d;
    const float *scale = p.scale[which] + head * p.nblk;
    const int32_t *idx = p.idx + head * p.budget;
    float amax = 0.f;
    for (int i = i0 + r0; i < i1; i += dr) {
        const int t = idx[i];
        amax = fmaxf(amax, amax8<FMT>(__ldg(reinterpret_cast<const uint2 *>(src + (size_t)t * p.D))) * scale[t >> p.blk_log]);
    }
    amax = cta_max(amax, red);
    const int e = step_exp<FMT>(amax);
    const float inv = pow2f(-e);
    if (threadIdx.x == 0) p.dscale[which][head * p.dnblk + j] = pow2f(e);
    uint8_t *dst = p.dcodes[which] + head * p.dT_cap * p.D + d;
    for (int i = i0 + r0; i < i1; i += dr) {
        const int t = idx[i];
        const float s = scale[t >> p.blk_log];
        // values, then units of the new step: the product of the two powers
        // could leave fp32's range, each factor alone cannot
        float a[4], c[4];
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(src + (size_t)t * p.D));
        decode4<FMT>(w.x, a);
        decode4<FMT>(w.y, c);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[k] = a[k] * s * inv;
            c[k] = c[k] * s * inv;
        }
        *reinterpret_cast<uint2 *>(dst + (size_t)i * p.D) =
            make_uint2(encode4<FMT>(a[0], a[1], a[2], a[3]), encode4<FMT>(c[0], c[1], c[2], c[3]));
    }
}

int ilog2(int v)
{
    int r = 0;
    while ((1 << r) < v) ++r;
    return r;
}

int launched()
{
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
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
    const dim3 grid(min((M - 1) / c.block + 2, p.nblk), 2 * c.kv_heads, c.batch);
    auto go = [&](auto kernel) { kernel<<<grid, kAppThreads, 0, stream>>>(p); };
    if (c.format == MOE_KV8_INT8) {
        if (type == MOE_BF16) go(kv8_append_kernel<MOE_KV8_INT8, MOE_BF16>);
        else if (type == MOE_F16) go(kv8_append_kernel<MOE_KV8_INT8, MOE_F16>);
        else go(kv8_append_kernel<MOE_KV8_INT8, MOE_F32>);
    } else {
        if (type == MOE_BF16) go(kv8_append_kernel<MOE_KV8_E4M3, MOE_BF16>);
        else if (type == MOE_F16) go(kv8_append_kernel<MOE_KV8_E4M3, MOE_F16>);
        else go(kv8_append_kernel<MOE_KV8_E4M3, MOE_F32>);
    }
    note_launch();
    return launched();
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
    if (c.format == MOE_KV8_INT8) kv8_read_kernel<MOE_KV8_INT8><<<grid, 256, 0, stream>>>(p);
    else kv8_read_kernel<MOE_KV8_E4M3><<<grid, 256, 0, stream>>>(p);
    note_launch();
    return launched();
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
    kv8_select_kernel<<<dim3(c.kv_heads, c.batch), kSelThreads, 0, stream>>>(p);
    note_launch();
    const dim3 grid((budget + c.block - 1) / c.block, 2 * c.kv_heads, c.batch);
    if (c.format == MOE_KV8_INT8) kv8_move_kernel<MOE_KV8_INT8><<<grid, kMoveThreads, 0, stream>>>(p);
    else kv8_move_kernel<MOE_KV8_E4M3><<<grid, kMoveThreads, 0, stream>>>(p);
    note_launch();
    return launched();
}

}  // namespace moe
