// Window attention with sinks on the CUDA cores: the fp32 form, forward and backward.
//
//   s_ij = q_i . k_j / sqrt d over the visible keys (window.cuh),  p = softmax(s),  O = p V
//   with D_i = dO_i . O_i:  dV_j = sum_i p_ij dO_i,  ds_ij = p_ij (dO_i . v_j - D_i) / sqrt d,
//   dQ_i = sum_j ds_ij k_j,  dK_j = sum_i ds_ij q_i.
//
// A block of 128 threads holds 32 rows against tiles of 64 columns; both sides lie row-major in
// shared memory with rows padded by 4 floats, so that the 16-byte reads of 16 neighbouring
// rows meet different banks.  A thread owns rows ty + 8 i and columns tx + 16 j of a score tile
// (4 x 4 scores from 8 16-byte reads per 4 channels, 64 FMAs in 32 packed instructions), and rows ty + 8 i and channels
// 4 tx + 64 j .. + 3 of an output.  Tiles arrive by cp.async as soon as their place is free (K and V
// of a tile in turn in one place), and three blocks (d 128) or four (d 64) share an SM, so that one computes while
// another waits (dK, dV copy Q twice a tile for the third: 389 us against 412 with two of twice the room).
// Scores, softmax statistics and all sums are fp32.  Bound by the FMA pipe (51 to 58 % busy over all
// SMs: 10 to 12 warps an SM do not hide the tile's barriers), the tiles' masked parts and the last blocks' end: the forward of 2 x 6
// heads x 1777 rows, d 64, window 300, takes 78 us; 8 heads x 1430 rows, d 128, frames of 143, two before
// and one after: forward 163 us and 9 to join, gradients 389 us, 4 for D and 7 to join.
#include "window.cuh"

namespace scope {

namespace {

// threads: 8 (ty) x 16 (tx); a warp holds 2 x 16, neighbouring lanes at the same column, so that a
// 16-byte read of 16 columns by 32 lanes is two wavefronts and one of 2 rows a single one
constexpr int kTh = 128;
constexpr int kBN = 64;      // columns of a score tile
constexpr int kBM = 32;      // rows of the ordinary form
constexpr int kLdP = kBN + 4;

__device__ __forceinline__ float4 load4(const float *p)
{
    return *reinterpret_cast<const float4 *>(p);
}

__device__ __forceinline__ void store4(float *p, float4 v)
{
    *reinterpret_cast<float4 *>(p) = v;
}

__device__ __forceinline__ void commit()
{
    asm volatile("cp.async.commit_group;\n" ::: "memory");
}

// Waits for all but the last N groups of copies, then for the block.
template <int N>
__device__ __forceinline__ void arrived()
{
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
    __syncthreads();
}

// Starts the copy of one tile's rows to shared memory (leading dimension D + 4), as one group;
// src(r) is row r's address or NULL for a row of zeros.  any: a valid address.
template <int D, int ROWS, typename Src>
__device__ __forceinline__ void load_tile(float *dst, const float *any, Src src)
{
    constexpr int C4 = D / 4;
#pragma unroll 4
    for (int e = threadIdx.x; e < ROWS * C4; e += kTh) {
        const int r = e / C4, c = (e % C4) * 4;
        const float *p = src(r);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(dst + r * (D + 4) + c)),
                     "l"(p ? p + c : any), "r"(p ? 16 : 0)
                     : "memory");
    }
    commit();
}

__device__ __forceinline__ void dot4(float &acc, float4 x, float4 y)
{
    acc = fmaf(x.x, y.x, acc);
    acc = fmaf(x.y, y.y, acc);
    acc = fmaf(x.z, y.z, acc);
    acc = fmaf(x.w, y.w, acc);
}

// Two products and sums in one instruction: the blocks are bound by instruction issue before the
// FMA pipe (96 % against 73 % of the busiest SM's cycles with scalar FMAs).
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t acc)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(acc));
    return d;
}

__device__ __forceinline__ uint64_t pair(float x, float y)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}

__device__ __forceinline__ float2 unpair(uint64_t v)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}

__device__ __forceinline__ ulonglong2 load22(const float *p)
{
    return *reinterpret_cast<const ulonglong2 *>(p);
}

// acc[i][j] = rows[ty + 8 i] . cols[tx + 16 j], j < NJ: even and odd channels summed apart.
template <int D, int MI, int NJ>
__device__ __forceinline__ void scores_of(float (&acc)[MI][4], const float *rows, const float *cols, int ty, int tx)
{
    uint64_t s[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[i][j] = 0ull;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        ulonglong2 x[MI], y[NJ];
#pragma unroll
        for (int i = 0; i < MI; ++i) x[i] = load22(rows + (ty + 8 * i) * (D + 4) + c);
#pragma unroll
        for (int j = 0; j < NJ; ++j) y[j] = load22(cols + (tx + 16 * j) * (D + 4) + c);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) s[i][j] = fma2(x[i].y, y[j].y, fma2(x[i].x, y[j].x, s[i][j]));
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = j < NJ ? unpair(s[i][j < NJ ? j : 0]) : make_float2(0.f, 0.f);
            acc[i][j] = f.x + f.y;
        }
}

// Groups of 16 columns of a tile that some row of the block meets: tiles at a window's edges and the
// last of the sinks are often partly empty, and half a tile or more that nobody sees is left out.
struct Groups {
    int lo, n;   // groups lo .. lo + n - 1: one, two or all four
};

__device__ __forceinline__ Groups groups(int lo, int end)
{
    return end - lo > 2 ? Groups{0, 4} : Groups{lo, end - lo};
}

// The groups of key tile j0 between rows ra (first) and rz (last).
__device__ __forceinline__ Groups key_groups(const WinRow &ra, const WinRow &rz, int j0)
{
    const int lo = j0 < ra.s ? 0 : max(0, ra.lo - j0) >> 4;
    const int end = max(min(ra.s - j0, kBN), ra.lo < j0 + kBN ? min(rz.hi - j0, kBN) : 0);
    return groups(min(lo, 3), max(min(lo, 3) + 1, (end + 15) >> 4));
}

// acc[i][j] = rows[ty + 8 i] . cols[16 (g.lo + j) + tx], j < g.n; zeros for the others.
template <int D, int MI>
__device__ __forceinline__ void scores(float (&acc)[MI][4], const float *rows, const float *cols, int ty, int tx, Groups g)
{
    cols += 16 * g.lo * (D + 4);
    if (g.n == 4)
        scores_of<D, MI, 4>(acc, rows, cols, ty, tx);
    else if (g.n == 2)
        scores_of<D, MI, 2>(acc, rows, cols, ty, tx);
    else
        scores_of<D, MI, 1>(acc, rows, cols, ty, tx);
}

// out[i][2 jj], [2 jj + 1] (channels 4 tx + 64 jj .. + 3 in pairs) += sum_k w[ty + 8 i][k] cols[k][...],
// k over the columns of the groups; w[.][k] starts at the first of them.
template <int D, int MI>
__device__ __forceinline__ void accumulate(uint64_t (&out)[MI][D / 32], const float *w, const float *cols, int ty, int tx, Groups g)
{
    cols += 16 * g.lo * (D + 4);
    const int n = 16 * g.n;
#pragma unroll 2
    for (int k = 0; k < n; k += 4) {
        float4 p[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) p[i] = load4(w + (ty + 8 * i) * kLdP + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            uint64_t pk[MI];
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const float v = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                pk[i] = pair(v, v);
            }
#pragma unroll
            for (int jj = 0; jj < D / 64; ++jj) {
                const ulonglong2 v = load22(cols + (k + kk) * (D + 4) + 4 * tx + 64 * jj);
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    out[i][2 * jj] = fma2(pk[i], v.x, out[i][2 * jj]);
                    out[i][2 * jj + 1] = fma2(pk[i], v.y, out[i][2 * jj + 1]);
                }
            }
        }
    }
}

// 4 channels 4 tx + 64 jj .. + 3 of one row, scaled.
__device__ __forceinline__ void store_scaled(float *p, const uint64_t *v, float scale)
{
    const float2 x = unpair(v[0]), y = unpair(v[1]);
    store4(p, make_float4(x.x * scale, x.y * scale, y.x * scale, y.y * scale));
}

// Forward: BM rows of one unit (b, group of a.pack query heads) against one share of the key
// tiles they see.  BM = 32, or 16 (two rows per thread) where a unit's rows fill no more.
template <int D, int BM>
__global__ void __launch_bounds__(kTh, D == 64 ? 4 : 3) window_fwd_kernel(WinArgs a)
{
    constexpr int MI = BM / 8;
    extern __shared__ __align__(16) float sm[];
    early_next();
    early_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;   // this path has no device conditions
    float *sq = sm, *sc = sq + BM * (D + 4), *sp = sc + kBN * (D + 4);   // sc: K, then V of a tile
    const int tx = (threadIdx.x >> 1) & 15, ty = (threadIdx.x & 1) + 2 * (threadIdx.x >> 5);
    const int rows = a.pack * a.Nq, tiles = (rows + BM - 1) / BM;
    // item = ((unit * tiles) + tile) * splits + split
    long long it = blockIdx.x;
    const int split = (int)(it % a.splits);
    it /= a.splits;
    const int tile = (int)(it % tiles), unit = (int)(it / tiles);
    const int groups = a.H / a.pack, b = unit / groups, h0 = (unit - b * groups) * a.pack;
    const int hk = h0 / (a.H / a.Hkv);
    const int r0 = tile * BM, r1 = min(rows, r0 + BM);
    const int first = win_first(a, b), kl = win_klen(a, b);
    // query range of the tile: rows r -> (head h0 + r / Nq, query r % Nq)
    const bool wraps = r0 / a.Nq != (r1 - 1) / a.Nq;
    const int ia = wraps ? 0 : r0 % a.Nq, iz = wraps ? a.Nq - 1 : (r1 - 1) % a.Nq;
    const WinRow ra = win_row(a, first + ia, kl), rz = win_row(a, first + iz, kl);
    const WinTiles wt = win_tiles<kBN>(ra, rz);
    const int nt = wt.count(), t0 = (int)((long long)nt * split / a.splits), t1 = (int)((long long)nt * (split + 1) / a.splits);
    const float *qb = static_cast<const float *>(a.Q) + b * a.lq.b;
    const float *kb = static_cast<const float *>(a.K) + b * a.lk.b + hk * a.lk.h;
    const float *vb = static_cast<const float *>(a.V) + b * a.lv.b + hk * a.lv.h;
    // a key tile of K or V; rows that no row of the tile sees are not read (they may hold anything)
    auto keys = [&](float *dst, const float *base, long long stride, int t) {
        if (t >= t1) return commit();
        const int j0 = wt.at(t) * kBN;
        load_tile<D, kBN>(dst, base, [&](int r) -> const float * {
            const int j = j0 + r;
            return j < ra.s || (j >= ra.lo && j < rz.hi) ? base + j * stride : nullptr;
        });
    };
    load_tile<D, BM>(sq, qb, [&](int r) -> const float * {
        const int rr = r0 + r;
        return rr < r1 ? qb + (h0 + rr / a.Nq) * a.lq.h + (rr % a.Nq) * a.lq.n : nullptr;
    });
    keys(sc, kb, a.lk.n, t0);
    WinRow lim[MI];
    float m[MI], l[MI];
    uint64_t o[MI][D / 32];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int rr = r0 + ty + 8 * i;
        lim[i] = rr < r1 ? win_row(a, first + rr % a.Nq, kl) : WinRow{0, 0, 0};
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) o[i][e] = 0ull;
    }
    for (int t = t0; t < t1; ++t) {
        const int j0 = wt.at(t) * kBN;
        arrived<0>();
        const Groups g = key_groups(ra, rz, j0);
        float s[MI][4];
        scores<D, MI>(s, sq, sc, ty, tx, g);
        __syncthreads();
        keys(sc, vb, a.lv.n, t);
        const bool all = win_all(ra, rz, j0, j0 + kBN);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            float mt = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = j0 + 16 * (g.lo + j) + tx;
                const bool vis = all || (j < g.n && (key < lim[i].s || (key >= lim[i].lo && key < lim[i].hi)));
                s[i][j] = vis ? s[i][j] * a.scale_log2 : -INFINITY;
                mt = fmaxf(mt, s[i][j]);
            }
#pragma unroll
            for (int x = 16; x > 1; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
            const float mn = fmaxf(m[i], mt), base = mn == -INFINITY ? 0.f : mn;
            const float corr = exp2f(m[i] - base);
            float ls = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = exp2f(s[i][j] - base);
                ls += s[i][j];
                sp[(ty + 8 * i) * kLdP + tx + 16 * j] = s[i][j];
            }
            l[i] = l[i] * corr + ls;   // of this thread's columns; joined at the end
            m[i] = mn;
            const uint64_t c2 = pair(corr, corr);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) o[i][e] = fma2(o[i][e], c2, 0ull);
        }
        arrived<0>();
        accumulate<D, MI>(o, sp, sc, ty, tx, g);
        __syncthreads();
        keys(sc, kb, a.lk.n, t + 1);
    }
    arrived<0>();
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int x = 16; x > 1; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
        const int rr = r0 + ty + 8 * i;
        if (rr >= r1) continue;
        const int h = h0 + rr / a.Nq, q = rr % a.Nq;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];   // no visible key: zeros; NaN stays NaN
        const float lse2 = l[i] == 0.f ? -INFINITY : m[i] + log2f(l[i]);
        const long long row = win_row_index(a, b, h, q);
        float *dst = a.splits > 1 ? a.part_o + (row * a.splits + split) * D
                                  : static_cast<float *>(a.O) + b * a.lo.b + h * a.lo.h + q * a.lo.n;
#pragma unroll
        for (int jj = 0; jj < D / 64; ++jj)
            store_scaled(dst + 4 * tx + 64 * jj, &o[i][2 * jj], inv);
        if (tx == 0) {
            if (a.splits > 1) a.part_lse[row * a.splits + split] = lse2;
            else if (a.lse) a.lse[row] = lse2 * 0.6931471805599453f;
        }
    }
}

// Joins the key shares of every row: O = sum_s 2^(L_s - L) O_s with L = log2 sum_s 2^L_s.
// One warp per row, shares in order (the result does not depend on the schedule).
template <typename T, int D>
__global__ void __launch_bounds__(128) window_join_kernel(WinArgs a)
{
    constexpr int PER = D / 32;
    early_next();
    early_wait();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (long long)a.B * a.H * a.Nq) return;
    const float *pl = a.part_lse + row * a.splits, *po = a.part_o + row * a.splits * D + lane * PER;
    float m = -INFINITY;
    for (int s = 0; s < a.splits; ++s) m = (pl[s] > m || pl[s] != pl[s]) ? pl[s] : m;   // keeps a NaN
    float sum = 0.f, o[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = 0.f;
    if (m != -INFINITY)
        for (int s = 0; s < a.splits; ++s) {
            const float w = exp2f(pl[s] - m);
            sum += w;
#pragma unroll
            for (int e = 0; e < PER; ++e) o[e] = fmaf(w, po[(long long)s * D + e], o[e]);
        }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int i = (int)(row % a.Nq), h = (int)(row / a.Nq % a.H), b = (int)(row / a.Nq / a.H);
    T *dst = static_cast<T *>(a.O) + b * a.lo.b + h * a.lo.h + i * a.lo.n + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        if constexpr (sizeof(T) == 2)
            dst[e] = __float2bfloat16(o[e] * inv);
        else
            dst[e] = o[e] * inv;
    }
    if (lane == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
}

// Joins the shares of the key tiles that were cut, in order: blockIdx.y is the tile, a thread 4
// channels of dK (blockIdx.z = 0) or dV of one key.
template <typename T, int D>
__global__ void __launch_bounds__(128) window_kv_join_kernel(WinArgs a, int rows)
{
    early_next();
    early_wait();
    const int tile = blockIdx.y + (a.kv.of_sink > 1 ? 0 : a.kv.sink), e = (int)threadIdx.x % (D / 4);
    const long long r = (long long)blockIdx.x * (128 / (D / 4)) + threadIdx.x / (D / 4);   // unit, key of the tile
    const int unit = (int)(r / rows), key = (int)(r % rows), j = tile * rows + key;
    if (unit >= a.kv.units || j >= a.Nk) return;
    const float *p = a.kv.sums(a.kv.item(tile, unit), rows, D) + (long long)blockIdx.z * rows * D + (long long)key * D + 4 * e;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = a.kv.shares(tile); s > 0; --s, p += 2ll * rows * D) {
        const float4 v = load4(p);
        x[0] += v.x;
        x[1] += v.y;
        x[2] += v.z;
        x[3] += v.w;
    }
    const WinLayout lay = blockIdx.z ? a.ldv : a.ldk;
    T *dst = static_cast<T *>(blockIdx.z ? a.dV : a.dK) + unit / a.Hkv * lay.b + unit % a.Hkv * lay.h + j * lay.n + 4 * e;
    if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
        *reinterpret_cast<uint2 *>(dst) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    } else {
        store4(dst, make_float4(x[0], x[1], x[2], x[3]));
    }
}

// D_i = dO_i . O_i, one warp per row.
template <int D>
__global__ void __launch_bounds__(kTh) window_delta_kernel(WinArgs a)
{
    early_next();
    early_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    const long long row = (long long)blockIdx.x * (kTh / 32) + (threadIdx.x >> 5);
    if (row >= (long long)a.B * a.H * a.Nq) return;
    const int i = (int)(row % a.Nq), h = (int)(row / a.Nq % a.H), b = (int)(row / a.Nq / a.H), c = 4 * (threadIdx.x & 31);
    float s = 0.f;
    if (c < D)
        dot4(s, load4(static_cast<const float *>(a.O) + b * a.lo.b + h * a.lo.h + i * a.lo.n + c),
             load4(static_cast<const float *>(a.G) + b * a.lg.b + h * a.lg.h + i * a.lg.n + c));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    if (c == 0) a.delta[row] = s;
}

// A row that sees one key: P = 1 whatever the score, so dS = 0, which dP - D only meets to rounding.
__device__ __forceinline__ bool alone(const WinRow &r)
{
    return r.s + r.hi - r.lo == 1;
}

// dQ: 32 query rows of one head against the key tiles they see.
template <int D>
__device__ __forceinline__ void dq_block(const WinArgs &a, float *sm, long long block)
{
    constexpr int MI = kBM / 8;
    float *sq = sm, *sg = sq + kBM * (D + 4), *sc = sg + kBM * (D + 4), *sp = sc + kBN * (D + 4);   // sc: V, then K of a tile
    const int tx = (threadIdx.x >> 1) & 15, ty = (threadIdx.x & 1) + 2 * (threadIdx.x >> 5);
    const int tiles = (a.Nq + kBM - 1) / kBM;
    const int tile = (int)(block % tiles), bh = (int)(block / tiles);
    const int b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hkv);
    const int r0 = tile * kBM, r1 = min(a.Nq, r0 + kBM);
    const int first = win_first(a, b), kl = win_klen(a, b);
    const WinRow ra = win_row(a, first + r0, kl), rz = win_row(a, first + r1 - 1, kl);
    const WinTiles wt = win_tiles<kBN>(ra, rz);
    const int nt = wt.count();
    const float *qb = static_cast<const float *>(a.Q) + b * a.lq.b + h * a.lq.h;
    const float *gb = static_cast<const float *>(a.G) + b * a.lg.b + h * a.lg.h;
    const float *kb = static_cast<const float *>(a.K) + b * a.lk.b + hk * a.lk.h;
    const float *vb = static_cast<const float *>(a.V) + b * a.lv.b + hk * a.lv.h;
    auto keys = [&](float *dst, const float *base, long long stride, int t) {
        if (t >= nt) return commit();
        const int j0 = wt.at(t) * kBN;
        load_tile<D, kBN>(dst, base, [&](int r) -> const float * {
            const int j = j0 + r;
            return j < ra.s || (j >= ra.lo && j < rz.hi) ? base + j * stride : nullptr;
        });
    };
    load_tile<D, kBM>(sq, qb, [&](int r) -> const float * { return r0 + r < r1 ? qb + (r0 + r) * a.lq.n : nullptr; });
    load_tile<D, kBM>(sg, gb, [&](int r) -> const float * { return r0 + r < r1 ? gb + (r0 + r) * a.lg.n : nullptr; });
    keys(sc, vb, a.lv.n, 0);
    arrived<1>();
    WinRow lim[MI];
    float lse[MI], dl[MI];
    uint64_t dq[MI][D / 32];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int q = r0 + ty + 8 * i;
        const bool in = q < r1;
        lim[i] = in ? win_row(a, first + q, kl) : WinRow{0, 0, 0};
        if (alone(lim[i])) lim[i] = WinRow{0, 0, 0};
        const long long row = win_row_index(a, b, h, in ? q : r0);
        lse[i] = in ? a.lse[row] * 1.4426950408889634f : -INFINITY;
        dl[i] = in ? a.delta[row] : 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) dq[i][e] = 0ull;
    }
    for (int t = 0; t < nt; ++t) {
        const int j0 = wt.at(t) * kBN;
        arrived<0>();
        const Groups g = key_groups(ra, rz, j0);
        float s[MI][4], dp[MI][4];
        scores<D, MI>(dp, sg, sc, ty, tx, g);
        __syncthreads();
        keys(sc, kb, a.lk.n, t);
        arrived<0>();
        scores<D, MI>(s, sq, sc, ty, tx, g);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = j0 + 16 * (g.lo + j) + tx;
                const bool vis = j < g.n && (key < lim[i].s || (key >= lim[i].lo && key < lim[i].hi));
                sp[(ty + 8 * i) * kLdP + tx + 16 * j] =
                    vis ? exp2f(fmaf(s[i][j], a.scale_log2, -lse[i])) * (dp[i][j] - dl[i]) : 0.f;
            }
        __syncwarp();   // a row of sp is written and read by one warp
        accumulate<D, MI>(dq, sp, sc, ty, tx, g);
        __syncthreads();
        keys(sc, vb, a.lv.n, t + 1);
    }
    arrived<0>();
    float *dst = static_cast<float *>(a.dQ) + b * a.ldq.b + h * a.ldq.h;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int q = r0 + ty + 8 * i;
        if (q >= r1) continue;
#pragma unroll
        for (int jj = 0; jj < D / 64; ++jj)
            store_scaled(dst + q * a.ldq.n + 4 * tx + 64 * jj, &dq[i][2 * jj], a.scale);
    }
}

// dK, dV: 32 keys of one key head against every query (of all its query heads, in order) that
// may see one of them.  Scores are taken transposed: rows are keys, columns are queries.
template <int D>
__device__ __forceinline__ void dkv_block(const WinArgs &a, float *sm, long long block)
{
    constexpr int MI = kBM / 8;
    float *sk = sm, *sv = sk + kBM * (D + 4), *sc = sv + kBM * (D + 4), *sp = sc + kBN * (D + 4);   // sc: Q, dO and Q of a tile
    const int tx = (threadIdx.x >> 1) & 15, ty = (threadIdx.x & 1) + 2 * (threadIdx.x >> 5);
    // sink blocks meet every later query: they come first in launch order
    int tile, bh, share;
    a.kv.at((int)block, tile, bh, share);
    const int shares = a.kv.shares(tile);
    const int b = bh / a.Hkv, hk = bh - b * a.Hkv, G = a.H / a.Hkv;
    const int j0 = tile * kBM, j1 = min(a.Nk, j0 + kBM);
    const int first = win_first(a, b), kl = win_klen(a, b);
    const int2 qr = win_queries(a, first, kl, a.Nq, j0, j1);
    const int per = (qr.y - qr.x + kBN - 1) / kBN, all = per * G;   // column tiles: per query head, in all
    const int t0 = (int)((long long)all * share / shares), nt = (int)((long long)all * (share + 1) / shares);
    const float *kb = static_cast<const float *>(a.K) + b * a.lk.b + hk * a.lk.h;
    const float *vb = static_cast<const float *>(a.V) + b * a.lv.b + hk * a.lv.h;
    auto queries = [&](float *dst, const void *tensor, const WinLayout &lay, int t) {
        if (t >= nt) return commit();
        const float *base = static_cast<const float *>(tensor) + b * lay.b + (hk * G + t / per) * lay.h;
        const int i0 = qr.x + t % per * kBN;
        load_tile<D, kBN>(dst, base, [&](int r) -> const float * { return i0 + r < qr.y ? base + (i0 + r) * lay.n : nullptr; });
    };
    load_tile<D, kBM>(sk, kb, [&](int r) -> const float * { return j0 + r < min(j1, kl) ? kb + (j0 + r) * a.lk.n : nullptr; });
    load_tile<D, kBM>(sv, vb, [&](int r) -> const float * { return j0 + r < min(j1, kl) ? vb + (j0 + r) * a.lv.n : nullptr; });
    queries(sc, a.Q, a.lq, t0);
    uint64_t dk[MI][D / 32], dv[MI][D / 32];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < D / 32; ++e) dk[i][e] = dv[i][e] = 0ull;
    for (int t = t0; t < nt; ++t) {
        const int h = hk * G + t / per, i0 = qr.x + t % per * kBN;
        float lse[4], dl[4];   // under way while the tile is
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int q = i0 + tx + 16 * j;
            const long long row = win_row_index(a, b, h, q < qr.y ? q : 0);
            lse[j] = a.lse[row];
            dl[j] = a.delta[row];
        }
        arrived<0>();   // Q
        float s[MI][4], dp[MI][4];
        const Groups g = groups(0, min(4, (qr.y - i0 + 15) >> 4));
        scores<D, MI>(s, sk, sc, ty, tx, g);
        __syncthreads();
        queries(sc, a.G, a.lg, t);
        uint32_t some = 0;   // bit 4 i + j: the score has a gradient
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int q = i0 + tx + 16 * j;
            const WinRow lim = q < qr.y ? win_row(a, first + q, kl) : WinRow{0, 0, 0};
            const float nlse = lse[j] * -1.4426950408889634f;
            const bool lone = alone(lim);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int key = j0 + ty + 8 * i;
                const bool vis = key < lim.s || (key >= lim.lo && key < lim.hi);
                s[i][j] = vis ? exp2f(fmaf(s[i][j], a.scale_log2, nlse)) : 0.f;
                some |= (uint32_t)(vis && !lone) << (4 * i + j);
                sp[(ty + 8 * i) * kLdP + tx + 16 * j] = s[i][j];
            }
        }
        arrived<0>();   // dO
        scores<D, MI>(dp, sv, sc, ty, tx, g);
        accumulate<D, MI>(dv, sp, sc, ty, tx, g);
        __syncthreads();
        queries(sc, a.Q, a.lq, t);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sp[(ty + 8 * i) * kLdP + tx + 16 * j] = (some >> (4 * i + j)) & 1u ? s[i][j] * (dp[i][j] - dl[j]) : 0.f;
        arrived<0>();   // Q again
        accumulate<D, MI>(dk, sp, sc, ty, tx, g);
        __syncthreads();
        queries(sc, a.Q, a.lq, t + 1);
    }
    arrived<0>();
    float *dkb = static_cast<float *>(a.dK) + b * a.ldk.b + hk * a.ldk.h, *dvb = static_cast<float *>(a.dV) + b * a.ldv.b + hk * a.ldv.h;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int j = j0 + ty + 8 * i;
        if (j >= j1) continue;
        if (shares > 1) {
            float *sum = a.kv.sums(block, kBM, D) + (ty + 8 * i) * D + 4 * tx;
#pragma unroll
            for (int jj = 0; jj < D / 64; ++jj) {
                store_scaled(sum + 64 * jj, &dk[i][2 * jj], a.scale);
                store_scaled(sum + kBM * D + 64 * jj, &dv[i][2 * jj], 1.f);
            }
            continue;
        }
#pragma unroll
        for (int jj = 0; jj < D / 64; ++jj) {
            const int c = 4 * tx + 64 * jj;
            store_scaled(dkb + j * a.ldk.n + c, &dk[i][2 * jj], a.scale);
            store_scaled(dvb + j * a.ldv.n + c, &dv[i][2 * jj], 1.f);
        }
    }
}

// Both gradients in one grid, so that the end of one kind's blocks is filled by the other's (8 heads
// x 1430, 360 blocks of each: as two grids the busiest SM had 1.48 and 1.33 times the mean's work).
template <int D>
__global__ void __launch_bounds__(kTh, D == 64 ? 4 : 3) window_bwd_kernel(WinArgs a)
{
    extern __shared__ __align__(16) float sm[];
    early_next();
    early_wait();
    // dQ's blocks first: those of dK, dV are cut finer (410 us against 458 the other way round, 8 heads x 1430, d 128)
    const long long q = (long long)a.B * a.H * ((a.Nq + kBM - 1) / kBM);
    if (blockIdx.x < q)
        dq_block<D>(a, sm, blockIdx.x);
    else
        dkv_block<D>(a, sm, blockIdx.x - q);
}

template <typename F>
cudaError_t launch(F *kernel, long long grid, int smem, const WinArgs &a, cudaStream_t s)
{
    if (grid < 1 || grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    return launch_early(kernel, dim3((unsigned)grid), kTh, smem, s, 1, a);
}

template <int D>
cudaError_t forward(const WinArgs &a, cudaStream_t s)
{
    // 16-row tiles when a unit's rows fill no more than one
    const long long rows = (long long)a.pack * a.Nq, units = (long long)a.B * (a.H / a.pack);
    if (rows <= 16)
        return launch(window_fwd_kernel<D, 16>, units * a.splits, (16 + kBN) * (D + 4) * 4 + 16 * kLdP * 4, a, s);
    return launch(window_fwd_kernel<D, kBM>, units * ((rows + kBM - 1) / kBM) * a.splits,
                  (kBM + kBN) * (D + 4) * 4 + kBM * kLdP * 4, a, s);
}

template <int D>
cudaError_t backward(const WinArgs &a, cudaStream_t s)
{
    const long long rows = (long long)a.B * a.H * a.Nq;
    cudaError_t e = launch(window_delta_kernel<D>, (rows + kTh / 32 - 1) / (kTh / 32), 0, a, s);
    if (e != cudaSuccess) return e;
    e = launch(window_bwd_kernel<D>, a.kv.items() + (long long)a.B * a.H * ((a.Nq + kBM - 1) / kBM),
               (2 * kBM + kBN) * (D + 4) * 4 + kBM * kLdP * 4, a, s);
    return e == cudaSuccess && a.kv.parts() > 0 ? window_kv_join(a, kBM, s) : e;
}

}  // namespace

cudaError_t window_simt_forward(const WinArgs &a, cudaStream_t s)
{
    return a.d == 64 ? forward<64>(a, s) : forward<128>(a, s);
}

cudaError_t window_simt_backward(const WinArgs &a, cudaStream_t s)
{
    return a.d == 64 ? backward<64>(a, s) : backward<128>(a, s);
}

cudaError_t window_kv_join(const WinArgs &a, int tile, cudaStream_t s)
{
    const int from = a.kv.of_sink > 1 ? 0 : a.kv.sink, to = a.kv.of_other > 1 ? a.kv.tiles : a.kv.sink;
    const int per = 128 / (a.d / 4);
    const dim3 grid((unsigned)(((long long)a.kv.units * tile + per - 1) / per), (unsigned)(to - from), 2);
    if (a.is_bf16)
        return a.d == 64 ? launch_early(window_kv_join_kernel<__nv_bfloat16, 64>, grid, 128, 0, s, 1, a, tile)
                         : launch_early(window_kv_join_kernel<__nv_bfloat16, 128>, grid, 128, 0, s, 1, a, tile);
    return a.d == 64 ? launch_early(window_kv_join_kernel<float, 64>, grid, 128, 0, s, 1, a, tile)
                     : launch_early(window_kv_join_kernel<float, 128>, grid, 128, 0, s, 1, a, tile);
}

cudaError_t window_join(const WinArgs &a, cudaStream_t s)
{
    const long long blocks = ((long long)a.B * a.H * a.Nq + 3) / 4;
    if (a.is_bf16)
        return a.d == 64 ? launch(window_join_kernel<__nv_bfloat16, 64>, blocks, 0, a, s)
                         : launch(window_join_kernel<__nv_bfloat16, 128>, blocks, 0, a, s);
    return a.d == 64 ? launch(window_join_kernel<float, 64>, blocks, 0, a, s)
                     : launch(window_join_kernel<float, 128>, blocks, 0, a, s);
}

}  // namespace scope
