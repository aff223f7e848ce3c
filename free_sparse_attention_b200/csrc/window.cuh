// Window attention with sinks: arguments and the visibility rule shared by its kernels.
//
// Token positions fall into frames of `frame` tokens, f(x) = x / frame.  The query at
// position p sees key j iff
//   j < k_len,  f(j) <= f(p) + right,  and  f(j) >= f(p) - left  or  f(j) < sinks,
// i.e. the keys [0, s) and [lo, hi) with hi = min(k_len, (f(p) + right + 1) frame),
// lo = min(hi, max(0, (f(p) - left) frame)) and s = min(lo, sinks * frame).  All three grow
// with p, so the limits of a run of queries follow from its first and last one.
#pragma once

#include "common.cuh"
#include "early.cuh"

namespace scope {

struct WinLayout {
    long long b, h, n;   // strides in elements; channels are contiguous
};

// dK, dV: a block owns a tile of keys and walks the queries that see it.  Tiles of sinks, which
// every later query sees, and tiles under long windows are cut into shares of the walk, whose sums
// lie in `part` as fp32 (dK, then dV of each share, `rows` keys a tile) until window_kv_join.
// Items in order: sink tiles (tile, then unit, then share), then the others (unit, tile, share).
struct KeyShares {
    int units, tiles, sink;   // B * Hkv; key tiles; tiles of sinks among them
    int of_sink, of_other;    // shares (1: written to dK, dV directly)
    float *part;
    __host__ __device__ long long sink_items() const { return (long long)units * sink * of_sink; }
    __host__ __device__ long long items() const { return sink_items() + (long long)units * (tiles - sink) * of_other; }
    // shares that are joined, and their place in `part`: sink items first
    __host__ __device__ long long parts() const
    {
        return (of_sink > 1 ? sink_items() : 0) + (of_other > 1 ? items() - sink_items() : 0);
    }
    __host__ __device__ int shares(int tile) const { return tile < sink ? of_sink : of_other; }
    __host__ __device__ long long item(int tile, int unit) const   // of share 0
    {
        return tile < sink ? ((long long)tile * units + unit) * of_sink
                           : sink_items() + ((long long)unit * (tiles - sink) + tile - sink) * of_other;
    }
    __device__ __forceinline__ void at(int it, int &tile, int &unit, int &share) const   // items() < 2^31
    {
        const int sinks = units * sink * of_sink;
        const bool is_sink = it < sinks;
        const int of = is_sink ? of_sink : of_other, step = is_sink ? units : tiles - sink;
        it -= is_sink ? 0 : sinks;
        share = 0;
        if (of > 1) {
            share = it % of;
            it /= of;
        }
        const int hi = it / step, lo = it - hi * step;
        tile = is_sink ? hi : sink + lo;
        unit = is_sink ? lo : hi;
    }
    // place of an item's sums (dK; dV behind it) for tiles of `rows` keys and d channels
    __device__ float *sums(long long it, int rows, int d) const
    {
        return part + (it - (of_sink > 1 ? 0 : sink_items())) * 2 * rows * d;
    }
};

struct WinArgs {
    const void *Q, *K, *V, *G;   // G: gradient of O (backward)
    void *O;                     // forward output; backward: the forward's output (read)
    void *dQ, *dK, *dV;
    float *lse;                  // [B, H, Nq] natural log, or NULL (forward); read in backward
    float *delta, *nlse;         // [B, H, Nq] rowsum(G o O), negated in the bf16 form, and (bf16)
                                 // -lse log2 e (backward workspace)
    WinLayout lq, lk, lv, lo, lg, ldq, ldk, ldv;
    const int32_t *q_first;      // [B] or NULL: position of each entry's first query
    const int32_t *k_len;        // [B] or NULL: keys of each entry
    int first0;                  // position of the first query when q_first is NULL
    int B, H, Hkv, Nq, Nk, d, is_bf16;
    int frame, left, right, sinks;
    int pack;                    // query heads whose rows share a tile (few-row forms), or 1
    int splits;                  // key ranges of one row tile, joined afterwards (1: no join)
    float *part_o, *part_lse;    // [B*H*Nq, splits, d], [B*H*Nq, splits] (log2)
    KeyShares kv;                // how dK, dV cut the query rows of a key tile
    float scale, scale_log2;     // 1/sqrt(d), log2(e)/sqrt(d)
    int32_t *status, *counter;
    int num_sms;
    unsigned long long wait_ns;
};

constexpr int kWinUnbounded = 1 << 30;   // left / right of -1
constexpr int kFewCluster = 6;           // few rows, bf16: up to as many shares join as a cluster

struct WinRow {
    int s, lo, hi;
};

__device__ __forceinline__ int win_first(const WinArgs &a, int b)
{
    const int f = a.q_first ? a.q_first[b] : a.first0;
    return min(max(f, 0), 1 << 30);
}

__device__ __forceinline__ int win_klen(const WinArgs &a, int b)
{
    return a.k_len ? min(max(a.k_len[b], 0), a.Nk) : a.Nk;
}

// Limits of the query at position p.
__device__ __forceinline__ WinRow win_row(const WinArgs &a, int p, int k_len)
{
    const long long f = p / a.frame;
    const long long hi = min((long long)k_len, (f + a.right + 1) * a.frame);
    const long long lo = min(hi, max(0ll, (f - a.left) * a.frame));
    WinRow r;
    r.hi = (int)hi;
    r.lo = (int)lo;
    r.s = (int)min(lo, (long long)a.sinks * a.frame);
    return r;
}

// Key tiles (BN keys) that the queries between rows `a` (first) and `z` (last) see: the
// tiles [0, sink) and [begin, end), begin >= sink.
struct WinTiles {
    int sink, begin, end;
    __device__ __forceinline__ int count() const { return sink + end - begin; }
    __device__ __forceinline__ int at(int i) const { return i < sink ? i : begin + i - sink; }
};

template <int BN>
__device__ __forceinline__ WinTiles win_tiles(const WinRow &a, const WinRow &z)
{
    WinTiles t;
    t.sink = (min(a.s, z.hi) + BN - 1) / BN;
    t.end = a.lo < z.hi ? (z.hi + BN - 1) / BN : t.sink;
    t.begin = max(t.sink, a.lo / BN);
    t.end = max(t.end, t.begin);
    return t;
}

// Whether every query between rows a (first) and z (last) sees all of the keys [j0, j1).
__device__ __forceinline__ bool win_all(const WinRow &a, const WinRow &z, int j0, int j1)
{
    return j1 <= a.s || (j0 >= z.lo && j1 <= a.hi);
}

// Query rows [x, y) of a run of n queries from position `first` that may see one of the keys
// [j0, j1).
__device__ __forceinline__ int2 win_queries(const WinArgs &a, int first, int k_len, int n, int j0, int j1)
{
    if (j0 >= k_len) return make_int2(0, 0);
    const long long x = max(0ll, ((long long)(j0 / a.frame) - a.right) * a.frame - first);
    const long long y = ((long long)((j1 - 1) / a.frame) + a.left + 1) * a.frame - first;
    const bool sink = j0 < (long long)a.sinks * a.frame;
    const int lo = (int)min((long long)n, x);
    const int hi = sink ? n : (int)min((long long)n, max((long long)lo, y));
    return make_int2(lo, hi);
}

// Rows of one unit (b, group of `pack` query heads): row r is query i of head h.
__device__ __forceinline__ long long win_row_index(const WinArgs &a, int b, int h, int i)
{
    return ((long long)b * a.H + h) * a.Nq + i;
}

// Launchers (enqueue only).
cudaError_t window_tc_forward(const WinArgs &a, cudaStream_t s);    // bf16; clears the header itself
cudaError_t window_tc_backward(const WinArgs &a, cudaStream_t s);   // bf16; clears the header itself
cudaError_t window_few_forward(const WinArgs &a, cudaStream_t s);   // bf16, pack * Nq <= 16
cudaError_t window_simt_forward(const WinArgs &a, cudaStream_t s);    // fp32
cudaError_t window_simt_backward(const WinArgs &a, cudaStream_t s);   // fp32
cudaError_t window_join(const WinArgs &a, cudaStream_t s);
cudaError_t window_kv_join(const WinArgs &a, int tile, cudaStream_t s);   // tile: keys a tile

}  // namespace scope
