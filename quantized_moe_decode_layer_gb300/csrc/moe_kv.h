// Launches of the 16-bit key/value cache (moe_kv.cu, moe_kv_tile.cu) and the
// parameters that its kernels share.
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int kKvTile = 64;           // positions a tile of the split kernel
constexpr int kKvFewRows = 16;        // rows that it takes; more go through the tile kernel
constexpr int kKvMaxCtas = 4 * kMaxCtas;
constexpr int kKvMaxPos = 1 << 30;    // positions of a sequence whose cache is a ring
constexpr int kKvAll = 1 << 30;       // window of a sequence that sees everything

// Weights are held 2^kv_up times as large as the reference says.  fp16's smallest step is 2^-24: with 2^7, weights from 2^-21 of the
// reference on have all bits, and what smaller ones lose is at most 2^-32 of the reference for each (131071 of 2^-25 behind one of
// 1 were zeros, and are off by less than 1 %).  With the 2^8 that the maximum may be above it they stay below 2^15.  bf16 has fp32's exponents.
constexpr __host__ __device__ float kv_up(bool f16) { return f16 ? 7.f : 0.f; }

// Division of 0 <= x < 2^31 by a number of heads (at most 2^20), exactly: x m / 2^s.
struct Div {
    uint32_t m;
    int s;
    __host__ __device__ int operator()(int x) const { return (int)(((unsigned long long)(uint32_t)x * m) >> s); }
};
inline Div div_by(uint32_t d)
{
    int l = 0;
    while ((1ull << l) < d) ++l;
    return {(uint32_t)((1ull << (31 + l)) / d + 1), 31 + l};
}

// One attention call: q, k, v as they lie (strides in elements), the visible
// positions, and where partial results go.
struct KvCall {
    const uint16_t *q, *k, *v, *pk, *pv;
    long long qb, qm, qh;             // q: sequence, row, head
    long long kb, km, kh, vb, vm, vh; // keys, values: sequence, position (slot), head
    long long pkm, pkh, pvm, pvh;     // the prefix's: position, head
    const int32_t *pos, *counts;      // pos NULL: T - M
    int *err;
    void *o;                          // [B][M][Hq][D], q's type
    int B, M, Hq, Hkv, G, D;
    Div by_g;                         // G
    int T;                            // slots of a sequence
    int limit;                        // positions that a sequence may have
    int W, S;                         // window (kKvAll: none), first positions that stay visible
    int P;                            // prefix positions (0: none)
    int f16;
    float c;                          // scale * log2(e)
    int ring;                         // positions from T on lie in the slots from S on, again and again
    // split kernel: of the sequences' own positions, of the prefix's
    int split_own, split_prefix;
    int late;                         // the call's second kernel: beside the first, whose end it waits for at its own
    float *part_o, *part_ml;          // [slot][16][D], [slot][16][2]: unnormalised output; reference (log2), sum
    // tile kernel: parts of the own positions, of the prefix's
    struct Parts {
        int n;                        // 0: not taken; own positions, 1 without a prefix: outputs are written
        float *o, *ml;                // [part][Hkv][B M G][D], [...][2]
    } own, prefix;
    long long timeout_ns;
};

size_t kv_attn_workspace_bytes(int batch, int kv_heads, int group, int head_dim, long long M, int T, int window, int sinks, int P);
int launch_kv_append(const moe_kv &c, const moe_rows &k_new, const moe_rows &v_new, int M, const int32_t *pos,
                     const int32_t *counts, int *err, cudaStream_t stream);
// Attention over a cache, or of a prompt.  p: q, k, v, the prefix, lengths, shapes, scale and output; the rest is set there.
int launch_kv_attn(KvCall &p, void *ws, cudaStream_t stream);
// Tiles of 128 rows against the own positions, or the prefix.
int launch_kv_tiles(const KvCall &p, bool prefix, cudaStream_t stream);
long long kv_row_tiles(long long rows, int D);
// Parts of a row tile's positions: at most, and taken.  `ragged`: lengths that the host does not know, few rows.  `rows`: to
// be joined if there is more than one.
int kv_tile_most(long long ctas, bool ragged);
int kv_tile_splits(long long ctas, long long tiles, bool ragged, long long rows);

}  // namespace moe
