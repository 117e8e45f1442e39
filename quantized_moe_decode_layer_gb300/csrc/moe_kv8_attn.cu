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
// a key/value head's group), the maximum, the sum of exp(s - max) and the
// unnormalised output; the merge kernel joins a row's chunks in order.
#include "moe_kv8.cuh"

namespace moe {
namespace {

struct AttnP {
    const void *q;
    long long qb, qm, qh;           // strides in elements: sequence, row, head
    const uint8_t *k, *v;
    const float *ks, *vs;
    const int32_t *pos, *counts;
    float *part_o, *part_ml, *sc;   // sc: scores [B][Hkv][T_cap][C], or NULL
    void *o;                        // [B][M][Hq][D]
    const float *acc_in;
    float *acc;
    float decay, scale_log2;        // scale * log2(e)
    int *err;
    int B, Hq, Hkv, G, M, C, T_cap, chunk, nchunk, blk_log, nblk, f16, o_type;
};

constexpr int kPlainThreads = 128, kPlainCols = 8;

// The simplest form, in fp32: a CTA takes one chunk of one key/value head for
// up to 8 query columns; a thread scores one position at a time, then
// gathers one value dimension.
template <int FMT, int D>
__global__ void __launch_bounds__(kPlainThreads) kv8_attn_plain_kernel(const AttnP p)
{
    __shared__ float q[kPlainCols][D], sc[kPlainCols][kPlainThreads], red[33];
    const int chunk = blockIdx.x, g = blockIdx.y % p.Hkv, c0 = blockIdx.y / p.Hkv * kPlainCols, b = blockIdx.z, tid = threadIdx.x;
    int p0;
    bool bad;
    const int rows = kv8_rows(p.pos, p.counts, b, p.M, p.T_cap, p0, bad);
    if (bad && chunk == 0 && blockIdx.y == 0 && tid == 0) atomicOr(p.err, kKv8ErrRange);
    const int n = rows > 0 ? p0 + rows : 0, k0 = chunk * p.chunk, k1 = min(k0 + p.chunk, n), nc = min(kPlainCols, p.C - c0);
    if (k0 >= k1) return;
    for (int i = tid; i < nc * D; i += kPlainThreads) {
        const int c = c0 + i / D, m = c / p.G, h = g * p.G + c % p.G;
        const long long at = b * p.qb + m * p.qm + h * p.qh + i % D;
        q[i / D][i % D] = p.f16 ? __half2float(static_cast<const __half *>(p.q)[at])
                                : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.q)[at]);
    }
    const size_t head = (size_t)b * p.Hkv + g;
    const uint8_t *K = p.k + head * p.T_cap * D, *V = p.v + head * p.T_cap * D;
    const float *ks = p.ks + head * p.nblk, *vs = p.vs + head * p.nblk;
    float mx[kPlainCols], l[kPlainCols], o[kPlainCols][(D + kPlainThreads - 1) / kPlainThreads];
    for (int c = 0; c < kPlainCols; ++c) {
        mx[c] = -INFINITY;
        l[c] = 0.f;
        for (float &x : o[c]) x = 0.f;
    }
    for (int t0 = k0; t0 < k1; t0 += kPlainThreads) {
        const int t = t0 + tid;
        float s[kPlainCols];
        for (float &x : s) x = 0.f;
        __syncthreads();
        if (t < k1) {
            const float f = ks[t >> p.blk_log] * p.scale_log2;
            for (int d = 0; d < D; d += 4) {
                float x[4];
                decode4<FMT>(__ldg(reinterpret_cast<const uint32_t *>(K + (size_t)t * D + d)), x);
                for (int c = 0; c < kPlainCols; ++c)
                    if (c < nc)
                        for (int i = 0; i < 4; ++i) s[c] = fmaf(q[c][d + i], x[i], s[c]);
            }
            for (int c = 0; c < kPlainCols; ++c)
                if (c < nc) {
                    s[c] *= f;
                    if (p.sc) p.sc[(head * p.T_cap + t) * p.C + c0 + c] = s[c];
                }
        }
        for (int c = 0; c < nc; ++c) {
            const bool see = t < k1 && t <= p0 + (c0 + c) / p.G && (c0 + c) / p.G < rows;
            const float tm = cta_max(see ? s[c] : -INFINITY, red);
            const float nm = fmaxf(mx[c], tm), base = nm == -INFINITY ? 0.f : nm;
            const float w = see ? exp2f(s[c] - base) : 0.f, al = exp2f(mx[c] - base);
            sc[c][tid] = w;
            mx[c] = nm;
            l[c] *= al;
            for (float &x : o[c]) x *= al;
        }
        __syncthreads();
        for (int i = 0; i < min(kPlainThreads, k1 - t0); ++i) {
            const float f = vs[(t0 + i) >> p.blk_log];
            for (int c = 0; c < nc; ++c) l[c] += sc[c][i];
            for (int j = 0; j < (D + kPlainThreads - 1) / kPlainThreads; ++j) {
                const int d = tid + j * kPlainThreads;
                if (d < D) {
                    float x[4];
                    decode4<FMT>(V[(size_t)(t0 + i) * D + d], x);
                    for (int c = 0; c < nc; ++c) o[c][j] = fmaf(sc[c][i], x[0] * f, o[c][j]);
                }
            }
        }
    }
    const size_t slot = ((size_t)b * p.nchunk + chunk) * p.Hkv + g;
    for (int c = 0; c < nc; ++c) {
        if (tid == 0) {
            p.part_ml[(slot * p.C + c0 + c) * 2] = mx[c];
            p.part_ml[(slot * p.C + c0 + c) * 2 + 1] = l[c];
        }
        for (int j = 0; j < (D + kPlainThreads - 1) / kPlainThreads; ++j)
            if (tid + j * kPlainThreads < D) p.part_o[(slot * p.C + c0 + c) * D + tid + j * kPlainThreads] = o[c][j];
    }
}

__device__ __forceinline__ void store_out(void *o, int type, size_t i, float v)
{
    if (type == MOE_BF16) static_cast<__nv_bfloat16 *>(o)[i] = __float2bfloat16_rn(v);
    else if (type == MOE_F16) static_cast<__half *>(o)[i] = __float2half_rn(v);
    else static_cast<float *>(o)[i] = v;
}

// Joins a row's chunks in order: one CTA per (row and query head, sequence), a thread per value dimension.
__global__ void kv8_merge_kernel(const AttnP p)
{
    const int D = blockDim.x, m = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq, b = blockIdx.y, d = threadIdx.x;
    const int g = h / p.G, c = m * p.G + h % p.G;
    int p0;
    bool bad;
    const int rows = kv8_rows(p.pos, p.counts, b, p.M, p.T_cap, p0, bad);
    const int n = m < rows ? p0 + m + 1 : 0, nch = (n + p.chunk - 1) / p.chunk;
    const size_t out = ((size_t)(b * p.M + m) * p.Hq + h) * D + d;
    if (nch == 0) {
        store_out(p.o, p.o_type, out, 0.f);
        return;
    }
    const size_t slot0 = (size_t)b * p.nchunk * p.Hkv + g;
    float mx = -INFINITY;
    for (int j = 0; j < nch; ++j) {
        const float v = __ldg(p.part_ml + ((slot0 + (size_t)j * p.Hkv) * p.C + c) * 2);
        mx = v > mx || v != v ? v : mx;   // a NaN stays
    }
    float o = 0.f, l = 0.f;
    for (int j = 0; j < nch; ++j) {
        const size_t i = (slot0 + (size_t)j * p.Hkv) * p.C + c;
        const float w = exp2f(__ldg(p.part_ml + i * 2) - mx);
        l = fmaf(w, __ldg(p.part_ml + i * 2 + 1), l);
        o = fmaf(w, __ldg(p.part_o + i * D + d), o);
    }
    store_out(p.o, p.o_type, out, o / l);
}

// Weight received by each position: every CTA joins the columns' maxima and
// sums, then adds its positions' normalised weights in column order.
constexpr int kAccThreads = 256;

__global__ void __launch_bounds__(kAccThreads) kv8_weights_kernel(const AttnP p)
{
    extern __shared__ float st[];   // [C][2]: maximum, 1 / sum
    const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    int p0;
    bool bad;
    const int rows = kv8_rows(p.pos, p.counts, b, p.M, p.T_cap, p0, bad);
    const int n = rows > 0 ? p0 + rows : 0, t0 = blockIdx.x * kAccThreads;
    if (t0 >= n) return;
    const size_t slot0 = (size_t)b * p.nchunk * p.Hkv + g;
    for (int c = tid; c < p.C; c += kAccThreads) {
        const int m = c / p.G, nch = m < rows ? (p0 + m + p.chunk) / p.chunk : 0;
        float mx = -INFINITY, l = 0.f;
        for (int j = 0; j < nch; ++j) {
            const float v = __ldg(p.part_ml + ((slot0 + (size_t)j * p.Hkv) * p.C + c) * 2);
            mx = v > mx || v != v ? v : mx;
        }
        for (int j = 0; j < nch; ++j) {
            const size_t i = (slot0 + (size_t)j * p.Hkv) * p.C + c;
            l = fmaf(exp2f(__ldg(p.part_ml + i * 2) - mx), __ldg(p.part_ml + i * 2 + 1), l);
        }
        st[2 * c] = mx;
        st[2 * c + 1] = 1.f / l;
    }
    __syncthreads();
    const int t = t0 + tid;
    if (t >= n) return;
    const size_t head = (size_t)b * p.Hkv + g;
    float a = t < p0 && p.acc_in ? p.decay * p.acc_in[head * p.T_cap + t] : 0.f;
    for (int c = 0; c < p.C; ++c)
        if (c / p.G < rows && t <= p0 + c / p.G)
            a = fmaf(exp2f(__ldg(p.sc + (head * p.T_cap + t) * p.C + c) - st[2 * c]), st[2 * c + 1], a);
    p.acc[head * p.T_cap + t] = a;
}

// Positions per chunk.
int kv8_chunk(const moe_kv8 &c) { return c.T_cap <= 8192 ? 256 : 512; }

struct Kv8Ws {
    size_t ml, o, sc, total;
};
Kv8Ws kv8_ws(const moe_kv8 &c, int M, bool weights)
{
    const size_t slots = (size_t)c.batch * ((c.T_cap + kv8_chunk(c) - 1) / kv8_chunk(c)) * c.kv_heads;
    const size_t cols = (size_t)(c.q_heads / c.kv_heads) * M;
    Kv8Ws w;
    w.ml = 0;
    w.o = align_up(slots * cols * 2 * sizeof(float), 256);
    w.sc = align_up(w.o + slots * cols * c.head_dim * sizeof(float), 256);
    w.total = weights ? align_up(w.sc + (size_t)c.batch * c.kv_heads * c.T_cap * cols * sizeof(float), 256) : w.sc;
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
    p.part_o = reinterpret_cast<float *>(base + w.o);
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
    p.f16 = q.type == MOE_F16;
    p.o_type = o_type;
    const dim3 grid(p.nchunk, c.kv_heads * ((p.C + kPlainCols - 1) / kPlainCols), c.batch);
    auto go = [&](auto kernel) { kernel<<<grid, kPlainThreads, 0, stream>>>(p); };
    if (c.format == MOE_KV8_INT8) {
        if (c.head_dim == 64) go(kv8_attn_plain_kernel<MOE_KV8_INT8, 64>);
        else if (c.head_dim == 128) go(kv8_attn_plain_kernel<MOE_KV8_INT8, 128>);
        else go(kv8_attn_plain_kernel<MOE_KV8_INT8, 256>);
    } else {
        if (c.head_dim == 64) go(kv8_attn_plain_kernel<MOE_KV8_E4M3, 64>);
        else if (c.head_dim == 128) go(kv8_attn_plain_kernel<MOE_KV8_E4M3, 128>);
        else go(kv8_attn_plain_kernel<MOE_KV8_E4M3, 256>);
    }
    note_launch();
    kv8_merge_kernel<<<dim3(M * c.q_heads, c.batch), c.head_dim, 0, stream>>>(p);
    note_launch();
    if (acc) {
        kv8_weights_kernel<<<dim3((c.T_cap + kAccThreads - 1) / kAccThreads, c.kv_heads, c.batch), kAccThreads,
                             p.C * 2 * sizeof(float), stream>>>(p);
        note_launch();
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) { note_cuda_error((int)e); return MOE_ERR_CUDA; }
    return MOE_OK;
}

}  // namespace moe
