// Window attention with sinks on the Blackwell tensor cores (tcgen05, sm_100a): the bf16
// gradients.
//
// With P = 2^(c Q K^T - lse), D_i = dO_i . O_i and dS = P o (dO V^T - D):
//   dQ = dS K / sqrt d,  dK = dS^T Q / sqrt d,  dV = P^T dO.
// Two kernels of one shape, so that every sum has one owner and a fixed order (no atomics, no
// fp32 gradient in memory; S and dO V^T are computed in both, 7 products instead of 5).  A CTA
// owns 128 rows and walks column tiles of 64:
//            rows R1, R2   columns C1, C2   S = R1 C1^T  dP = R2 C2^T   results
//   dQ       Q, dO         K, V             S            dP             dQ += dS C1
//   dK, dV   K, V          Q, dO            S^T          dP^T           dK += dS C1, dV += P C2
// Per CTA (persistent, one per SM): warps 0-3 / 4-7 turn S and dP of even / odd steps into P and
// dS (thread r owns row r = TMEM lane r); warp 8 loads rows and column tiles by TMA (and lse and D
// of the columns, for dK, dV) and hands out the items; warps 10 and 9 issue S and dP, warp 11 the
// products of P and dS, read as operands from TMEM.
// What bounds a step is the chain product -> commit -> wait -> arithmetic -> arrive -> product
// (about 3500 cycles when one buffer goes through all of it), so the chain is cut where TMEM has
// room: S and dP are released as soon as they are in registers, P and dS have columns of their
// own, and every operand has its own barrier (dV starts on P while dS is computed).  Only dK, dV
// at d = 128 has no such room (2 x 128 columns of results): there P and dS replace S and dP.
// P and dS are rounded to bf16 once, as operands; everything summed is fp32.
// Measured (B200): 48 heads x 17550, d 64, frames of 1350, one to either side and the first: dQ 2.10 ms =
// 766 TFLOP/s, dK dV 2.85 ms = 755; 3 x 16 heads of 4 key heads x 4001, d 128, window 1024: 184 and 222 us.
#include "window_tc.cuh"

#include <algorithm>

namespace scope {

namespace {

constexpr int kBM = 128, kBN = 64;
constexpr int kWarps = 12, kThreads = kWarps * 32;
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 216, kOtherRegs = 72;   // 65536 / 384, a multiple of 8
static_assert(2 * kSoftmaxRegs + kOtherRegs == 3 * kLaunchRegs, "register split");
constexpr int kMaxStages = 8, kMaxBuf = 3, kRing = 4;
constexpr uint32_t kTmemCols = 512;

struct __align__(8) Bars {
    uint64_t r_full, r_empty, land[2], out_full, out_free, sums_full, sums_free;
    uint64_t c_full[kMaxStages], c_empty[kMaxStages], ls_full[kMaxStages];
    uint64_t s_full[kMaxBuf], d_full[kMaxBuf], s_free[kMaxBuf], d_free[kMaxBuf];   // S and dP buffers
    uint64_t p_full[2], ds_full[2], pd_free[2], drain[3];                          // P and dS buffers
    uint64_t item_full[kRing], item_empty[kRing];
};

// TMEM columns: kBuf buffers of S (64) and dP (64); then, unless they share those, two buffers
// of P (dK, dV only) and dS (32 each); then the results (D each).
template <bool DKV, int D>
struct Cols {
    static constexpr bool kShared = DKV && D == 128;   // P and dS replace S and dP
    static constexpr int kBuf = !DKV && D == 64 ? 3 : 2;
    static constexpr int kPd = kBuf * 128;
    static constexpr int kPdBuf = kShared ? 0 : (DKV ? 64 : 32);
    static constexpr int kOut = kPd + 2 * kPdBuf;
    static_assert(kOut + (DKV ? 2 : 1) * D <= (int)kTmemCols, "TMEM columns");
    // column of the bf16 pairs of columns 16 kk .. 16 kk + 15 of P / dS of step g
    static constexpr __device__ __forceinline__ uint32_t p(uint32_t g, int kk)
    {
        return kShared ? (g % 2) * 128 + (kk >> 1) * 32 + (kk & 1) * 8 : kPd + (g & 1) * kPdBuf + kk * 8;
    }
    static constexpr __device__ __forceinline__ uint32_t ds(uint32_t g, int kk)
    {
        return kShared ? p(g, kk) + 64 : kPd + (g & 1) * kPdBuf + (DKV ? 32 : 0) + kk * 8;
    }
};

// One item: 128 rows of one head, and its column tiles in order.
template <bool DKV>
struct Item {
    int b, h, r0, nrows;   // h: query head (dQ) or key head (dK, dV)
    int first, kl;
    WinRow a, z;           // dQ: limits of the first and last row
    WinTiles wt;           // dQ: key tiles
    int n;                 // dQ: their number, walked twice if a row sees few keys (below)
    int c0, per, steps;    // dK, dV: first query tile and tiles per query head; steps of the share
    int from;              // dK, dV: the share's first step
    float *part;           // dK, dV: place of the share's sums, or NULL: dK, dV themselves
};

template <bool DKV, int D>
struct Smem {
    static constexpr int kStages = D == 128 ? (DKV ? 4 : 5) : 8;
    static constexpr int kRows = kBM * D * 2, kTile = kBN * D * 2;
    static constexpr int kR1 = 0, kR2 = kRows, kC = 2 * kRows;               // stage s: C1, C2
    static constexpr int kLs = kC + kStages * 2 * kTile;                     // stage s: lse [64], D [64]
    static constexpr int kSums = kLs;                                        // dQ: [2][128] row sums of dS
    static constexpr int kBars = kLs + (DKV ? kStages * 2 * kBN * 4 : 2 * kBM * 4);
    static constexpr int kMisc = kBars + (int)sizeof(Bars);
    static constexpr int kItems = kMisc + 64;                                // the ring's items
    static constexpr int kAlloc = kItems + kRing * (int)sizeof(Item<DKV>) + 1024;
    static_assert(kAlloc <= 232448, "shared memory budget");
    static_assert(kAlloc > 232448 / 2, "one CTA (and its 512 TMEM columns) per SM");
    static_assert(kStages <= kMaxStages, "ring depth");
};

// D_i = dO_i . O_i carries the rounding of O to bf16, a share 2^-9 |O| |dO| that matters where a row
// averages few values: at 4 visible keys it is as large as the rounding of dS, at 256 it is lost in
// it.  A tile with such rows is walked twice: the first walk gives sum_j dS_ij = (exact D_i) - D_i in
// fp32 (sum_j P_ij = 1), the second uses the corrected D_i, and so do dK and dV.  Those tiles are
// short by nature.
constexpr int kFewKeys = 256;

template <bool DKV, bool PLUS>
__device__ __forceinline__ Item<DKV> item_of(const WinArgs &a, int it)
{
    Item<DKV> x;
    const int n = DKV ? a.Nk : a.Nq, heads = DKV ? a.Hkv : a.H, tiles = (n + kBM - 1) / kBM;
    int bh, tile, share = 0;
    x.from = 0;
    x.part = nullptr;
    if (DKV) {
        // sink tiles meet every later query: those of all heads first; then head by head
        a.kv.at(it, tile, bh, share);
    } else {
        bh = it / tiles;
        tile = tiles - 1 - it % tiles;
    }
    x.b = bh / heads;
    x.h = bh % heads;
    x.r0 = tile * kBM;
    x.nrows = min(kBM, n - x.r0);
    x.first = win_first(a, x.b);
    x.kl = win_klen(a, x.b);
    if (DKV) {
        const int2 qr = win_queries(a, x.first, x.kl, a.Nq, x.r0, x.r0 + x.nrows);
        x.c0 = qr.x / kBN;
        x.per = qr.y > qr.x ? (qr.y + kBN - 1) / kBN - x.c0 : 0;
        const int all = x.per * (a.H / a.Hkv), shares = PLUS ? a.kv.shares(tile) : 1;
        x.steps = all;
        if (PLUS && shares > 1) {
            x.from = (int)((long long)all * share / shares);
            x.steps = (int)((long long)all * (share + 1) / shares) - x.from;
            x.part = a.kv.sums(it, kBM, a.d);
        }
    } else {
        x.a = win_row(a, x.first + x.r0, x.kl);
        x.z = win_row(a, x.first + x.r0 + x.nrows - 1, x.kl);
        x.wt = win_tiles<kBN>(x.a, x.z);
        x.n = x.wt.count();
        // the number of visible keys rises, stays and falls along the rows: least at an end
        const int least = min(x.a.s + x.a.hi - x.a.lo, x.z.s + x.z.hi - x.z.lo);
        x.steps = PLUS && least < kFewKeys ? 2 * x.n : x.n;
    }
    return x;
}

// Column tile t of an item: head and first column.
template <bool DKV>
__device__ __forceinline__ int2 column_of(const WinArgs &a, const Item<DKV> &x, int t)
{
    if (DKV) {
        t += x.from;   // 0 without shares
        return make_int2(x.h * (a.H / a.Hkv) + t / x.per, (x.c0 + t % x.per) * kBN);
    }
    return make_int2(x.h / (a.H / a.Hkv), x.wt.at(t < x.n ? t : t - x.n) * kBN);
}

// 32 values of this thread's row as bf16 pairs in 16 TMEM columns.
__device__ __forceinline__ void store_half(uint32_t taddr, const float *v)
{
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        __nv_bfloat162 h2 = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
        pk[e] = *reinterpret_cast<uint32_t *>(&h2);
    }
    tmem_st16(taddr, pk);
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const float *src, bool in)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}

// PLUS: some tile of the dQ pass may have rows that see few keys (the exact D costs every tile of
// the pass 5 to 8 %, for the code it brings into the step loop, so it is left out where no row can),
// or some tile of the dK, dV pass is cut into shares (2 to 3 %).
template <bool DKV, int D, bool PLUS>
__global__ void __launch_bounds__(kThreads, 1)
    window_bwd_tc_kernel(const __grid_constant__ CUtensorMap tmR1, const __grid_constant__ CUtensorMap tmR2,
                         const __grid_constant__ CUtensorMap tmC1, const __grid_constant__ CUtensorMap tmC2,
                         const __grid_constant__ WinArgs a, int n_items)
{
    using L = Smem<DKV, D>;
    using T = Cols<DKV, D>;
    constexpr bool FEW = PLUS && !DKV, CUT = PLUS && DKV;
    constexpr int NB = D / 64, NS = L::kStages, NBUF = T::kBuf;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars *bars = reinterpret_cast<Bars *>(sm + L::kBars);
    int *misc = reinterpret_cast<int *>(sm + L::kMisc);
    volatile int *abort_flag = misc;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + 1);
    volatile int *ring = misc + 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sbase = smem_u32(sm);
    const Waiter W{abort_flag, a.status, a.wait_ns};
    const uint32_t bar_base = sbase + L::kBars;
#define BAR(member) (bar_base + (uint32_t)offsetof(Bars, member))
    int32_t *counter = a.counter + (DKV ? 1 : 0);

    if (threadIdx.x == 0) {
        misc[0] = 0;
        bar_init(&bars->r_full, 1);
        bar_init(&bars->r_empty, 2);
        bar_init(&bars->land[0], 1);
        bar_init(&bars->land[1], 1);
        bar_init(&bars->out_full, 1);
        bar_init(&bars->out_free, 8);
        bar_init(&bars->sums_full, 8);
        bar_init(&bars->sums_free, 8);
        for (int s = 0; s < kMaxStages; ++s) {
            bar_init(&bars->c_full[s], 1);
            bar_init(&bars->c_empty[s], 1);
            bar_init(&bars->ls_full[s], 32);
        }
        for (int w = 0; w < kMaxBuf; ++w) {
            bar_init(&bars->s_full[w], 1);
            bar_init(&bars->d_full[w], 1);
            bar_init(&bars->s_free[w], T::kShared ? 1 : 4);   // the product's commit, or the 4 warps
            bar_init(&bars->d_free[w], T::kShared ? 1 : 4);
        }
        for (int w = 0; w < 2; ++w) {
            bar_init(&bars->p_full[w], 4);
            bar_init(&bars->ds_full[w], 4);
            bar_init(&bars->pd_free[w], 1);
        }
        for (int w = 0; w < 3; ++w) bar_init(&bars->drain[w], 1);
        for (int k = 0; k < kRing; ++k) {
            bar_init(&bars->item_full[k], 1);
            bar_init(&bars->item_empty[k], kWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 10) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t out1 = tmem + T::kOut, out2 = out1 + D;   // dQ or dK; dV
    // lane 0 of warp 8 is the item scheduler: it decodes an item ahead, for all
    Item<DKV> *const items_ring = reinterpret_cast<Item<DKV> *>(sm + L::kItems);
    auto fetch = [&](uint32_t k) -> bool {
        const int slot = k % kRing;
        if (!wait1(BAR(item_empty) + 8u * (slot), ((k / kRing) & 1) ^ 1, W)) return false;
        const int it = atomicAdd(counter, 1);
        if (it < n_items) items_ring[slot] = item_of<DKV, PLUS>(a, it);
        ring[slot] = it < n_items ? it : -1;
        bar_arrive(BAR(item_full) + 8u * (slot));
        return true;
    };
    auto next_item = [&](uint32_t k, Item<DKV> &x) -> int {
        const int slot = k % kRing;
        if (!waitw(BAR(item_full) + 8u * (slot), (k / kRing) & 1, W)) return -1;
        const int it = ring[slot];
        x = items_ring[slot];
        __syncwarp();
        if (lane == 0) bar_arrive(BAR(item_empty) + 8u * (slot));
        if (warp == 8 && it >= 0) {
            int ok = 1;
            if (lane == 0) ok = fetch(k + 1) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) return -1;
        }
        return it;
    };
    early_next();
    early_wait();
    if (warp == 8 && lane == 0) fetch(0);

    // Every role counts the CTA's steps in g: step g uses S / dP buffer g % NBUF, P / dS buffer
    // g % 2 and column stage g % NS; phase parities follow from the quotients.
    uint32_t g = 0;
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8) {
            // ------------------------------------------------------------------ loads
            uint32_t r_it = 0, land = 0;
            // dQ: a tile with key rows that no row of the item sees lands on a barrier of its own, and
            // those rows are zeroed (0 x NaN would reach dQ) once the next tile's copy is on its way
            constexpr uint32_t kNone = ~0u;
            uint32_t edge = kNone, edge_next = kNone;   // its step; that of a second one when waits gave up
            int edge_y = 0;                             // its first key
            auto finish_edge = [&](const Item<DKV> &x, int ok) -> int {
                if (edge == kNone || !ok) return ok;
                if (!waitw(BAR(land) + 8u * (land & 1), (land >> 1) & 1, W)) return 0;
                ++land;
                for (int e = lane; e < kBN * NB * 8; e += 32) {
                    const int r = e / (NB * 8), j = edge_y + r;
                    if (!(j < x.a.s || (j >= x.a.lo && j < x.z.hi)))
                        *reinterpret_cast<uint4 *>(sm + L::kC + edge % NS * 2 * L::kTile + (e / 8 % NB) * (kBN * 128) + r * 128 +
                                                   (e % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) bar_arrive(BAR(c_full) + 8u * (edge % NS));
                edge = kNone;
                return 1;
            };
            for (uint32_t item_k = 0; !warp_aborted(abort_flag); ++item_k) {
                Item<DKV> x;
                if (next_item(item_k, x) < 0) break;
                if (x.steps == 0) continue;
                int ok = 1;
                if (lane == 0) {
                    ok = wait1(BAR(r_empty), (r_it & 1) ^ 1, W);
                    if (ok) {
                        bar_expect_tx(BAR(r_full), 2 * L::kRows);
#pragma unroll
                        for (int k = 0; k < NB; ++k) {
                            tma_rows(sbase + L::kR1 + k * (kBM * 128), &tmR1, k * 64, x.r0, x.h, x.b, BAR(r_full));
                            tma_rows(sbase + L::kR2 + k * (kBM * 128), &tmR2, k * 64, x.r0, x.h, x.b, BAR(r_full));
                        }
                        ++r_it;
                    }
                }
                // lane 0: waits for the step's stage and starts its copies, which arrive on `bar`
                auto copy = [&](int2 col, uint32_t bar) -> int {
                    const int s = g % NS;
                    if (!wait1(BAR(c_empty) + 8u * (s), ((g / NS) & 1) ^ 1, W)) return 0;
                    bar_expect_tx(bar, 2 * L::kTile);
                    const uint32_t dst = sbase + L::kC + s * 2 * L::kTile;
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        tma_rows(dst + k * (kBN * 128), &tmC1, k * 64, col.y, col.x, x.b, bar);
                        tma_rows(dst + L::kTile + k * (kBN * 128), &tmC2, k * 64, col.y, col.x, x.b, bar);
                    }
                    return 1;
                };
                if constexpr (DKV) {
                    for (int t = 0; t < x.steps; ++t, ++g) {
                        const int s = g % NS;
                        const int2 col = column_of<DKV>(a, x, t);
                        if (lane == 0 && ok) ok = copy(col, BAR(c_full) + 8u * s);
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (!ok) break;
                        __syncwarp();
                        // -lse log2 e and -D of the columns beside the tile; the copies arrive on
                        // the barrier themselves
                        const uint32_t ls = sbase + L::kLs + s * (2 * kBN * 4) + lane * 4;
                        const long long row = win_row_index(a, x.b, col.x, col.y) + lane;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const bool in = col.y + lane + 32 * k < a.Nq;
                            cp_async4(ls + 128 * k, a.nlse + (in ? row + 32 * k : 0), in);
                            cp_async4(ls + kBN * 4 + 128 * k, a.delta + (in ? row + 32 * k : 0), in);
                        }
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(BAR(ls_full) + 8u * s) : "memory");
                    }
                } else {
                    for (int t = 0; t < x.steps && ok;) {
                        // lane 0 alone, up to an edge tile, or one tile while an edge tile lands
                        int whole = 1, y = 0;
                        if (lane == 0)
                            do {
                                const int2 col = column_of<DKV>(a, x, t);
                                y = col.y;
                                whole = y + kBN <= x.a.s || (y >= x.a.lo && y + kBN <= x.z.hi);
                                ok = copy(col, whole ? BAR(c_full) + 8u * (g % NS)
                                                     : BAR(land) + 8u * ((land + (edge != kNone ? 1 : 0)) & 1));
                                if (!ok) break;
                                ++g;
                                ++t;
                            } while (whole && edge == kNone && t < x.steps);
                        g = __shfl_sync(0xffffffffu, g, 0);
                        t = __shfl_sync(0xffffffffu, t, 0);
                        y = __shfl_sync(0xffffffffu, y, 0);
                        whole = __shfl_sync(0xffffffffu, whole, 0);
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (!ok) break;
                        ok = finish_edge(x, ok);
                        if (!whole) {
                            (ok ? edge : edge_next) = g - 1;
                            edge_y = y;
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if constexpr (!DKV) ok = finish_edge(x, ok);
                if (!ok) break;
            }
            asm volatile("cp.async.wait_all;\n" ::: "memory");
            if (lane == 0) {   // copies already issued land before the CTA exits
                for (uint32_t v = g > (uint32_t)NS ? g - NS : 0; v < g; ++v)
                    if (v != edge && v != edge_next) drain_wait(BAR(c_full) + 8u * (v % NS), (v / NS) & 1, W.limit_ns);
                for (uint32_t v = land; v < land + (edge != kNone) + (edge_next != kNone); ++v)
                    drain_wait(BAR(land) + 8u * (v & 1), (v >> 1) & 1, W.limit_ns);
                if (r_it > 0) drain_wait(BAR(r_full), (r_it - 1) & 1, W.limit_ns);
            }
            __syncwarp();
        } else if (lane == 0) {
            // ------------------------------------------------------------------ product issuers
            constexpr uint32_t idesc_s = f16_idesc(kBM, kBN, false), idesc_o = f16_idesc(kBM, D, true);
            // warp 9: dP, warp 10: S, warp 11: the products of P and dS.  A thread's commits and
            // waits leave the tensor pipe idle unless another thread's products are queued behind.
            const bool first_products = warp < 11, is_s = warp == 10;
            const uint64_t r_desc = sw128_desc(sbase + (is_s ? L::kR1 : L::kR2), 16, 1024);
            uint32_t items = 0;
            bool issued = false;
            for (uint32_t item_k = 0; !*abort_flag; ++item_k) {
                const int slot = item_k % kRing;
                if (!wait1(BAR(item_full) + 8u * (slot), (item_k / kRing) & 1, W)) break;
                const int it = ring[slot];
                const Item<DKV> x = items_ring[slot];
                bar_arrive(BAR(item_empty) + 8u * (slot));
                if (it < 0) break;
                const int steps = x.steps;
                if (steps == 0) continue;
                bool ok = true;
                issued = true;
                if (first_products) {
                    ok = wait1(BAR(r_full), items & 1, W);
                    for (int t = 0; t < steps && ok; ++t, ++g) {
                        const int s = g % NS, w = g % NBUF;
                        ok = wait1(BAR(c_full) + 8u * (s), (g / NS) & 1, W) &&
                             wait1(is_s ? BAR(s_free) + 8u * (w) : BAR(d_free) + 8u * (w), ((g / NBUF) & 1) ^ 1, W);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t c_desc = sw128_desc(sbase + L::kC + s * 2 * L::kTile + (is_s ? 0 : L::kTile), 16, 1024);
                        const uint32_t dst = tmem + 128 * w + (is_s ? 0 : 64);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t offa = (uint64_t)(((kk >> 2) * (kBM * 128) + (kk & 3) * 32) >> 4);
                            const uint64_t offb = (uint64_t)(((kk >> 2) * (kBN * 128) + (kk & 3) * 32) >> 4);
                            mma_bf16(dst, r_desc + offa, c_desc + offb, idesc_s, kk > 0);
                        }
                        mma_commit(is_s ? BAR(s_full) + 8u * (w) : BAR(d_full) + 8u * (w));
                        if (t == steps - 1) mma_commit(BAR(r_empty));
                    }
                } else {
                    for (int t = 0; t < steps && ok; ++t, ++g) {
                        const int s = g % NS, w = g & 1;
                        const uint32_t use = (g >> 1) & 1;
                        const uint32_t cb = sbase + L::kC + s * 2 * L::kTile;
                        ok = wait1(BAR(c_full) + 8u * (s), (g / NS) & 1, W);
                        if (ok && t == 0) ok = wait1(BAR(out_free), (items & 1) ^ 1, W);
                        if (!ok) break;
                        if constexpr (DKV) {
                            const uint64_t c2 = sw128_desc(cb + L::kTile, kBN * 128, 1024);
                            ok = wait1(BAR(p_full) + 8u * (w), use, W);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int kk = 0; kk < kBN / 16; ++kk)
                                mma_bf16_ts(out2, tmem + T::p(g, kk), c2 + (uint64_t)(kk * 2048 >> 4), idesc_o,
                                            (t > 0 || kk > 0) ? 1u : 0u);
                            if constexpr (T::kShared) mma_commit(BAR(s_free) + 8u * (w));
                        }
                        const uint64_t c1 = sw128_desc(cb, kBN * 128, 1024);
                        const bool fresh = t == 0 || (FEW && t == x.n);   // a walk's first step
                        ok = wait1(BAR(ds_full) + 8u * (w), use, W);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < kBN / 16; ++kk)
                            mma_bf16_ts(out1, tmem + T::ds(g, kk), c1 + (uint64_t)(kk * 2048 >> 4), idesc_o,
                                        (!fresh || kk > 0) ? 1u : 0u);
                        mma_commit(T::kShared ? BAR(d_free) + 8u * (w) : BAR(pd_free) + 8u * (w));
                        mma_commit(BAR(c_empty) + 8u * (s));
                        if (t == steps - 1) mma_commit(BAR(out_full));
                    }
                }
                if (!ok) break;
                ++items;
            }
            if (issued) {   // every product issued completes before TMEM is freed
                mma_commit(BAR(drain) + 8u * (warp - 9));
                drain_wait(BAR(drain) + 8u * (warp - 9), 0, W.limit_ns);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------------- P and dS, epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // the warpgroup's steps are those of its parity: two steps in work at a time
        const int odd = warp >> 2, row = threadIdx.x & (kBM - 1);
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        uint32_t items = 0;
        // the warpgroup's next step, with its buffers and their phases: S / dP buffer w, P / dS
        // buffer `odd`, column stage s
        uint32_t mine = odd, w = odd, s = odd, use = 0, pd_use = 0, s_use = 0, sums_use = 0;
        auto below = [&](int e) { return e <= 0 ? 0ull : (e >= 64 ? ~0ull : (1ull << e) - 1ull); };
        // the item, what this thread's row sees of it (columns [0, s) and [lo, hi) of dQ, [lo, hi) of
        // dK, dV) and its -lse log2 e and -D: taken while the last products of the item before it run
        Item<DKV> next;
        WinRow next_lim{0, 0, 0};
        float next_nlse = 0.f, next_ndelta = 0.f;
        uint32_t item_k = 0;
        auto take = [&]() -> int {
            const int it = next_item(item_k++, next);
            next_lim = WinRow{0, 0, 0};
            if (it < 0 || row >= next.nrows) return it;
            if constexpr (DKV) {
                const int2 qr = win_queries(a, next.first, next.kl, a.Nq, next.r0 + row, next.r0 + row + 1);
                next_lim.lo = qr.x;
                next_lim.hi = qr.y;
            } else {
                next_lim = win_row(a, next.first + next.r0 + row, next.kl);
                const long long ix = win_row_index(a, next.b, next.h, next.r0 + row);
                next_nlse = a.nlse[ix];
                next_ndelta = a.delta[ix];
            }
            return it;
        };
        int it = take();
        while (it >= 0 && !warp_aborted(abort_flag)) {
            const Item<DKV> x = next;
            const WinRow lim = next_lim;
            const float nlse = next_nlse;
            float ndelta = next_ndelta;
            const bool valid = row < x.nrows;
            const unsigned long long c2 = f2pack(a.scale_log2, a.scale_log2), nlse2 = f2pack(nlse, nlse);
            unsigned long long ndelta2 = f2pack(ndelta, ndelta), sum2 = 0ull;
            const bool twice = FEW && x.steps > x.n;
            bool ok = true, summing = twice;
            // the end of a first walk: the rows' sums over both warpgroups' steps correct D
            auto correct = [&]() {
                float *sums = reinterpret_cast<float *>(sm + L::kSums);
                const float2 part = f2unpack(sum2);
                ok &= waitw(BAR(sums_free), (sums_use & 1) ^ 1, W);
                sums[odd * kBM + row] = part.x + part.y;
                __syncwarp();
                warp_arrive(BAR(sums_full), lane);
                ok &= waitw(BAR(sums_full), sums_use & 1, W);
                ++sums_use;
                ndelta -= sums[row] + sums[kBM + row];
                __syncwarp();
                warp_arrive(BAR(sums_free), lane);
                ndelta2 = f2pack(ndelta, ndelta);
                if (odd == 0 && valid) a.delta[win_row_index(a, x.b, x.h, x.r0 + row)] = ndelta;
                summing = false;
            };
            // this warpgroup's steps: mine, mine + 2, ... below g + steps.  The column tile follows
            // without a division: position `at` of the query tiles of a head (dK, dV)
            int at = (int)(mine - g);
            if constexpr (DKV) {
                if (CUT && x.per > 0) at = (at + x.from) % x.per;
                while (at >= x.per && x.per > 0) at -= x.per;
            }
            for (uint32_t from = g, walks = FEW && x.steps > x.n ? 2 : 1; walks > 0 && ok; --walks) {
            for (; ok && mine - from < (uint32_t)(DKV ? x.steps : x.n); mine += 2) {
                const int j0 = (DKV ? (x.c0 + at) : x.wt.at((int)(mine - from))) * kBN;
                const uint32_t sb = tmem + lane_base + 128 * w;   // S; dP at + 64
                const bool whole =
                    __all_sync(0xffffffffu, j0 + kBN <= lim.s || (lim.lo <= j0 && j0 + kBN <= lim.hi));
                // a wait that gave up leaves the loop at the end of the step: what the step computes
                // from then on goes nowhere, and nothing else waits for long
                if constexpr (DKV) ok &= waitw(BAR(ls_full) + 8u * s, s_use, W);
                ok &= waitw(BAR(s_full) + 8u * w, use, W);
                tc_fence_after();
                float v[kBN];
                tmem_ld32(sb, v);
                tmem_ld32(sb + 32, v + 32);
                tmem_wait_ld(v);
                if constexpr (!T::kShared) {
                    tc_fence_before();
                    __syncwarp();
                    warp_arrive(BAR(s_free) + 8u * w, lane);
                }
                // P of the columns the row sees, 0 elsewhere
                const float *ls = reinterpret_cast<const float *>(sm + L::kLs) + s * 2 * kBN;
#pragma unroll
                for (int e = 0; e < kBN; e += 4) {
                    unsigned long long l0 = nlse2, l1 = nlse2;
                    if constexpr (DKV) {
                        const ulonglong2 l4 = *reinterpret_cast<const ulonglong2 *>(ls + e);
                        l0 = l4.x;
                        l1 = l4.y;
                    }
                    const float2 x0 = f2unpack(f2fma(f2pack(v[e], v[e + 1]), c2, l0));
                    const float2 x1 = f2unpack(f2fma(f2pack(v[e + 2], v[e + 3]), c2, l1));
                    v[e] = fast_exp2(x0.x);
                    v[e + 1] = fast_exp2(x0.y);
                    v[e + 2] = fast_exp2(x1.x);
                    v[e + 3] = fast_exp2(x1.y);
                }
                unsigned long long vis = ~0ull;
                if (__builtin_expect(!whole, 0)) {
                    vis = below(lim.s - j0) | (below(lim.hi - j0) & ~below(lim.lo - j0));
#pragma unroll
                    for (int e = 0; e < kBN; ++e) v[e] = (vis >> e) & 1ull ? v[e] : 0.f;
                }
                if constexpr (DKV) {
                    if constexpr (!T::kShared) {
                        ok &= waitw(BAR(pd_free) + 8u * odd, pd_use ^ 1, W);
                        tc_fence_after();
                    }
                    store_half(tmem + lane_base + T::p(odd, 0), v);
                    store_half(tmem + lane_base + T::p(odd, 2), v + 32);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    warp_arrive(BAR(p_full) + 8u * odd, lane);
                }
                ok &= waitw(BAR(d_full) + 8u * w, use, W);
                tc_fence_after();
                float dv[kBN];
                tmem_ld32(sb + 64, dv);
                tmem_ld32(sb + 96, dv + 32);
                tmem_wait_ld(dv);
                if constexpr (!T::kShared) {
                    tc_fence_before();
                    __syncwarp();
                    warp_arrive(BAR(d_free) + 8u * w, lane);
                }
#pragma unroll
                for (int e = 0; e < kBN; e += 4) {
                    unsigned long long d0 = ndelta2, d1 = ndelta2;
                    if constexpr (DKV) {
                        const ulonglong2 d4 = *reinterpret_cast<const ulonglong2 *>(ls + kBN + e);
                        d0 = d4.x;
                        d1 = d4.y;
                    }
                    const float2 x0 = f2unpack(f2mul(f2pack(v[e], v[e + 1]), f2add(f2pack(dv[e], dv[e + 1]), d0)));
                    const float2 x1 = f2unpack(f2mul(f2pack(v[e + 2], v[e + 3]), f2add(f2pack(dv[e + 2], dv[e + 3]), d1)));
                    v[e] = x0.x;
                    v[e + 1] = x0.y;
                    v[e + 2] = x1.x;
                    v[e + 3] = x1.y;
                }
                if (__builtin_expect(!whole, 0)) {   // 0 x what a hidden column holds
#pragma unroll
                    for (int e = 0; e < kBN; ++e) v[e] = (vis >> e) & 1ull ? v[e] : 0.f;
                }
                if constexpr (!DKV) {
                    if (FEW && __builtin_expect(summing, 0)) {
#pragma unroll
                        for (int e = 0; e < kBN; e += 2) sum2 = f2add(sum2, f2pack(v[e], v[e + 1]));
                    }
                    ok &= waitw(BAR(pd_free) + 8u * odd, pd_use ^ 1, W);
                    tc_fence_after();
                }
                store_half(tmem + lane_base + T::ds(odd, 0), v);
                store_half(tmem + lane_base + T::ds(odd, 2), v + 32);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                warp_arrive(BAR(ds_full) + 8u * odd, lane);
                // the next but one step's buffers and phases
                pd_use ^= 1;
                if (NBUF == 2) {
                    use ^= 1;
                } else {
                    w += 2;
                    if (w >= NBUF) {
                        w -= NBUF;
                        use ^= 1;
                    }
                }
                s += 2;
                if (s >= NS) {
                    s -= NS;
                    s_use ^= 1;
                }
                if constexpr (DKV) {
                    at += 2;
                    while (at >= x.per) at -= x.per;
                }
            }
            if constexpr (FEW) {
                if (summing && ok) correct();
                from += x.n;
            }
            }
            g += x.steps;
            if (!ok) break;
            it = take();
            // epilogue: dK by warpgroup 0 and dV by 1; of dQ, half the channels each
            if (x.steps > 0) {
                if (!waitw(BAR(out_full), items & 1, W)) break;
                ++items;
                tc_fence_after();
            }
            constexpr int CH = DKV ? D : D / 2;   // channels of one warpgroup
            const int ch0 = DKV ? 0 : odd * CH;
            const uint32_t src = (DKV && odd ? out2 : out1) + lane_base + ch0;
            const float scale = DKV && odd ? 1.f : a.scale;
            const WinLayout lay = DKV ? (odd ? a.ldv : a.ldk) : a.ldq;
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(DKV ? (odd ? a.dV : a.dK) : a.dQ) + x.b * lay.b + x.h * lay.h +
                                 (x.r0 + row) * lay.n + ch0;
#pragma unroll 1
            for (int h = 0; h < CH / 16; ++h) {
                float o[16];
                if (x.steps > 0) {
                    tmem_ld16(src + h * 16, o);
                    tmem_wait_ld(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = 0.f;
                }
                if (!valid) continue;
                if (CUT && x.part) {
                    float *sum = x.part + odd * (kBM * D) + row * D + h * 16;
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<float4 *>(sum + e) =
                            make_float4(o[e] * scale, o[e + 1] * scale, o[e + 2] * scale, o[e + 3] * scale);
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    uint32_t pk[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        __nv_bfloat162 hh = __floats2bfloat162_rn(o[e + 2 * k] * scale, o[e + 2 * k + 1] * scale);
                        pk[k] = *reinterpret_cast<uint32_t *>(&hh);
                    }
                    *reinterpret_cast<uint4 *>(dst + h * 16 + e) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
            }
            if (x.steps > 0) {
                tc_fence_before();
                __syncwarp();
                warp_arrive(BAR(out_free), lane);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 10)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// -D_i = -dO_i . O_i and -lse_i log2 e for the two passes, D / 8 threads per row; clears the status word and the item counters first
// (this launch precedes the two kernels above on the stream).
template <int D>
__global__ void __launch_bounds__(256) window_delta_kernel(WinArgs a)
{
    constexpr int TPR = D / 8;
    early_next();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *a.status = 0;
        a.counter[0] = a.counter[1] = 0;
    }
    const long long row = (long long)blockIdx.x * (256 / TPR) + threadIdx.x / TPR, rows = (long long)a.B * a.H * a.Nq;
    const int g = threadIdx.x % TPR;
    float s = 0.f;
    if (row < rows) {
        const int i = (int)(row % a.Nq), h = (int)(row / a.Nq % a.H), b = (int)(row / a.Nq / a.H);
        const uint4 o = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.O) + b * a.lo.b + h * a.lo.h +
                                                         i * a.lo.n + 8 * g);
        const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.G) + b * a.lg.b + h * a.lg.h +
                                                         i * a.lg.n + 8 * g);
        const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, gw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            s = fmaf(__uint_as_float(ow[k] << 16), __uint_as_float(gw[k] << 16), s);
            s = fmaf(__uint_as_float(ow[k] & 0xFFFF0000u), __uint_as_float(gw[k] & 0xFFFF0000u), s);
        }
    }
#pragma unroll
    for (int x = TPR / 2; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    if (g == 0 && row < rows) {
        a.delta[row] = -s;
        a.nlse[row] = a.lse[row] * -1.4426950408889634f;
    }
}

template <bool DKV, int D, bool PLUS>
cudaError_t launch_pass(const WinArgs &a, cudaStream_t s)
{
    CUtensorMap r1, r2, c1, c2;
    const int rows = DKV ? kBN : kBM, keys = DKV ? kBM : kBN;   // rows of a query and of a key tile
    CUtensorMap &q = DKV ? c1 : r1, &g = DKV ? c2 : r2, &k = DKV ? r1 : c1, &v = DKV ? r2 : c2;
    if (!rows_map(&q, a.Q, a.lq, a.B, a.H, a.Nq, D, rows) || !rows_map(&g, a.G, a.lg, a.B, a.H, a.Nq, D, rows) ||
        !rows_map(&k, a.K, a.lk, a.B, a.Hkv, a.Nk, D, keys) || !rows_map(&v, a.V, a.lv, a.B, a.Hkv, a.Nk, D, keys))
        return cudaErrorInvalidValue;
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, window_bwd_tc_kernel<DKV, D, PLUS>) != cudaSuccess || fa.numRegs != kLaunchRegs)
        return cudaErrorInvalidDeviceFunction;
    const long long items = DKV ? a.kv.items() : (long long)a.B * a.H * ((a.Nq + kBM - 1) / kBM);
    if (items > 0x7ffffff0ll) return cudaErrorInvalidConfiguration;
    const int smem = Smem<DKV, D>::kAlloc;
    cudaError_t e = cudaFuncSetAttribute(window_bwd_tc_kernel<DKV, D, PLUS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_early(window_bwd_tc_kernel<DKV, D, PLUS>, dim3((unsigned)(items < a.num_sms ? items : a.num_sms)), kThreads, smem,
                        s, 1, r1, r2, c1, c2, a, (int)items);
}

template <int D>
cudaError_t backward(const WinArgs &a, cudaStream_t s)
{
    const long long rows = (long long)a.B * a.H * a.Nq;
    const int per = 256 / (D / 8);
    // not early: its many small blocks would take the SMs' threads while the forward ends (608 us
    // against 598 for the whole step of 3 x 16/4 heads x 4001)
    window_delta_kernel<D><<<(unsigned)((rows + per - 1) / per), 256, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    // the first and the last query see the fewest keys
    bool few = a.q_first || a.k_len;
    for (const long long p : {(long long)a.first0, (long long)a.first0 + a.Nq - 1}) {
        const long long f = p / a.frame, hi = std::min((long long)a.Nk, (f + a.right + 1) * a.frame),
                        lo = std::min(hi, std::max(0ll, (f - a.left) * a.frame));
        few = few || hi - lo + std::min(lo, (long long)a.sinks * a.frame) < kFewKeys;
    }
    if (e == cudaSuccess) e = few ? launch_pass<false, D, true>(a, s) : launch_pass<false, D, false>(a, s);
    const bool cut = a.kv.parts() > 0;
    if (e == cudaSuccess) e = cut ? launch_pass<true, D, true>(a, s) : launch_pass<true, D, false>(a, s);
    if (e == cudaSuccess && cut) e = window_kv_join(a, kBM, s);
    return e;
}

#undef BAR

}  // namespace

cudaError_t window_tc_backward(const WinArgs &a, cudaStream_t s)
{
    return a.d == 64 ? backward<64>(a, s) : backward<128>(a, s);
}

}  // namespace scope
