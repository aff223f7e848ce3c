// Window attention with sinks on the Blackwell tensor cores (tcgen05, sm_100a), bf16 forward.
//
//   S = Q K^T over the key tiles that the rows see (window.cuh), P = 2^(c S - m), O = P V / l,
//   with the running row maximum m (in the exp2 domain) and row sum l in fp32.
//
// An item is 256 query rows of one head (two Q tiles of 128) against one share of the 64-key
// tiles that they see; tiles that only one Q tile sees cost the other nothing but a stage
// release.  Per CTA (persistent, one per SM, items handed out in order by a global counter):
//   warps 0-3 / 4-7  softmax + epilogue of Q tile 0 / 1 (thread r owns row r = TMEM lane r)
//   warp 8           TMA of Q and K, and the item scheduler
//   warp 9           TMA of V; zeroes the rows of edge tiles that no row of the item sees, so
//                    that what lies there (0 x NaN) cannot reach the product
//   warps 10 / 11    issue S = Q K^T of Q tile 0 / 1, warps 12 / 13 P V (one thread each: after a
//                    commit a thread's next wait takes some 400 cycles, in which the others'
//                    products keep the tensor pipe fed)
// TMEM: NSB buffers of S per Q tile (64 fp32 columns; P as bf16 pairs over the first 32 columns
// of its own buffer) and two O tiles.  S(n + NSB) follows P V(n), which frees its buffer.
// Only tiles that some row sees in part pay for the mask (one 64-bit word per row and tile).
// A step of 256 rows x 64 keys is bound by the chain S -> softmax -> P -> P V of either Q tile, about
// 2100 cycles at d 128 against 1024 of exponentials and 1280 of products.  Measured (B200): 40 heads x
// 32760, d 128, frames of 1560, two to either side and the first: 5.4 ms cold = 1080 TFLOP/s, 6.2 ms in a
// long run under the power limit; 48 heads x 17550, d 64: 1.78 ms.
#include "window_tc.cuh"

namespace scope {

namespace {

constexpr int kBM = 128;           // queries per Q tile (TMEM lanes)
constexpr int kBN = 64;            // keys per tile
constexpr int kThreads = 512;      // 16 warps, the last two idle (register splits are by warpgroup)
constexpr int kItemWarps = 14;     // warps that read the items
constexpr int kLaunchRegs = 128;   // 65536 / 512
constexpr int kSoftmaxRegs = 192;  // 2 warpgroups x 128 threads
constexpr int kOtherRegs = 64;     // 2 warpgroups
static_assert(2 * kSoftmaxRegs + 2 * kOtherRegs == 4 * kLaunchRegs, "register split");
constexpr int kMaxStages = 8, kMaxSB = 3, kRing = 4;
constexpr uint32_t kTmemCols = 512;

template <int D>
struct SBuf {
    static constexpr int n = D == 128 ? 2 : 3;   // 2 (n 64 + D) <= 512 columns
};

struct __align__(8) Bars {
    uint64_t q_full, q_empty, v_land;
    uint64_t k_full[kMaxStages], k_empty[kMaxStages];
    uint64_t v_full[kMaxStages], v_empty[kMaxStages];
    uint64_t s_full[2][kMaxSB], p_full[2][kMaxSB], o_done[2][kMaxSB];
    uint64_t o_free[2], drain[4];
    uint64_t item_full[kRing], item_empty[kRing];
};

// One item of the forward pass.
struct Item {
    int b, h, hk, r0, nrows, split, kl, first;
    WinRow a[2], z[2];   // limits of the first and last row of each Q tile (nrows > 128 q)
    WinTiles all, q[2];  // key tiles of the item and of each Q tile
    int t0, t1;          // the item's share of `all`
};

template <int D>
struct Smem {
    static constexpr int kStages = D == 128 ? 5 : 8;   // K and V rings
    static constexpr int kQTile = kBM * D * 2;
    static constexpr int kTile = kBN * D * 2;
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + 2 * kQTile;
    static constexpr int kV = kK + kStages * kTile;
    static constexpr int kBars = kV + kStages * kTile;
    static constexpr int kMisc = kBars + (int)sizeof(Bars);
    static constexpr int kItems = kMisc + 64;          // the ring's items
    static constexpr int kAlloc = kItems + kRing * (int)sizeof(Item) + 1024;
    static_assert(kAlloc <= 232448, "shared memory budget");
    static_assert(kAlloc > 232448 / 2, "one CTA (and its 512 TMEM columns) per SM");
};

// Whether the rows with key tiles w see key tile k.
__device__ __forceinline__ bool sees(const WinTiles &w, int k)
{
    return k < w.sink || (k >= w.begin && k < w.end);
}

template <typename T>
__device__ __forceinline__ T pick(bool second, const T (&v)[2])
{
    return second ? v[1] : v[0];   // by value: no indexed local memory
}

__device__ __forceinline__ Item item_of(const WinArgs &a, int it, int tiles)
{
    Item x;
    x.split = it % a.splits;
    it /= a.splits;
    const int bh = it / tiles;
    x.r0 = (tiles - 1 - (it - bh * tiles)) * (2 * kBM);   // late rows first: they see most under a causal bound
    x.b = bh / a.H;
    x.h = bh - x.b * a.H;
    x.hk = x.h / (a.H / a.Hkv);
    x.nrows = min(2 * kBM, a.Nq - x.r0);
    x.first = win_first(a, x.b) + x.r0;
    x.kl = win_klen(a, x.b);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int n = min(kBM, x.nrows - q * kBM);
        if (n > 0) {
            x.a[q] = win_row(a, x.first + q * kBM, x.kl);
            x.z[q] = win_row(a, x.first + q * kBM + n - 1, x.kl);
            x.q[q] = win_tiles<kBN>(x.a[q], x.z[q]);
        } else {
            x.a[q] = x.z[q] = WinRow{0, 0, 0};
            x.q[q] = WinTiles{0, 0, 0};
        }
    }
    x.all = win_tiles<kBN>(x.a[0], x.nrows > kBM ? x.z[1] : x.z[0]);
    const int n = x.all.count();
    x.t0 = (int)((long long)n * x.split / a.splits);
    x.t1 = (int)((long long)n * (x.split + 1) / a.splits);
    return x;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ WinArgs a, int n_items)
{
    using L = Smem<D>;
    constexpr int NB = D / 64, NSB = SBuf<D>::n, NS = L::kStages;
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
    const int tiles = (a.Nq + 2 * kBM - 1) / (2 * kBM);

    if (threadIdx.x == 0) {
        misc[0] = 0;
        bar_init(&bars->q_full, 1);
        bar_init(&bars->q_empty, 2);
        bar_init(&bars->v_land, 1);
        for (int s = 0; s < kMaxStages; ++s) {
            bar_init(&bars->k_full[s], 1);
            bar_init(&bars->v_full[s], 1);
            bar_init(&bars->k_empty[s], 2);
            bar_init(&bars->v_empty[s], 2);
        }
        for (int q = 0; q < 2; ++q) {
            for (int b = 0; b < kMaxSB; ++b) {
                bar_init(&bars->s_full[q][b], 1);
                bar_init(&bars->p_full[q][b], 4);
                bar_init(&bars->o_done[q][b], 1);
            }
            bar_init(&bars->o_free[q], 4);
        }
        for (int k = 0; k < 4; ++k) bar_init(&bars->drain[k], 1);
        for (int k = 0; k < kRing; ++k) {
            bar_init(&bars->item_full[k], 1);
            bar_init(&bars->item_empty[k], kItemWarps);
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
    // Scheduler: lane 0 of warp 8 takes item indices from the counter (or, where there are no more
    // items than CTAs, which then do without one, its CTA's) one item ahead and
    // publishes the items in a ring that every warp reads; -1 ends the work.
    Item *const items_ring = reinterpret_cast<Item *>(sm + L::kItems);
    auto fetch = [&](uint32_t k) -> bool {
        const int slot = k % kRing;
        if (!wait1(BAR(item_empty) + 8u * (slot), ((k / kRing) & 1) ^ 1, W)) return false;
        const int it = a.counter ? atomicAdd(a.counter, 1) : (k == 0 ? (int)blockIdx.x : n_items);
        if (it < n_items) items_ring[slot] = item_of(a, it, tiles);
        ring[slot] = it < n_items ? it : -1;
        bar_arrive(BAR(item_full) + 8u * (slot));
        return true;
    };
    auto next_item = [&](uint32_t k, Item &x) -> int {
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
    if (!a.counter && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    if (warp == 8 && lane == 0) fetch(0);

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8) {
            // -------------------------------------------------------------- Q and K loads
            uint32_t k_it = 0, q_it = 0;
            for (uint32_t item_k = 0; !warp_aborted(abort_flag); ++item_k) {
                Item x;
                if (next_item(item_k, x) < 0) break;
                if (x.t0 == x.t1) continue;
                int ok = 1;
                if (lane == 0) {
                    ok = wait1(BAR(q_empty), (q_it & 1) ^ 1, W);
                    if (ok) {
                        const int nq = x.nrows > kBM ? 2 : 1;
                        bar_expect_tx(BAR(q_full), nq * L::kQTile);
                        for (int q = 0; q < nq; ++q)
#pragma unroll
                            for (int b = 0; b < NB; ++b)
                                tma_rows(sbase + L::kQ + q * L::kQTile + b * (kBM * 128), &tmQ, b * 64, x.r0 + q * kBM, x.h,
                                         x.b, BAR(q_full));
                    }
                    for (int t = x.t0; t < x.t1 && ok; ++t) {
                        const int s = k_it % NS;
                        ok = wait1(BAR(k_empty) + 8u * (s), ((k_it / NS) & 1) ^ 1, W);
                        if (!ok) break;
                        bar_expect_tx(BAR(k_full) + 8u * (s), L::kTile);
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            tma_rows(sbase + L::kK + s * L::kTile + b * (kBN * 128), &tmK, b * 64, x.all.at(t) * kBN, x.hk, x.b,
                                     BAR(k_full) + 8u * (s));
                        ++k_it;
                    }
                    ++q_it;
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
            }
            if (lane == 0) {   // loads already issued land before the CTA exits
                for (uint32_t v = k_it > (uint32_t)NS ? k_it - NS : 0; v < k_it; ++v)
                    drain_wait(BAR(k_full) + 8u * (v % NS), (v / NS) & 1, W.limit_ns);
                if (q_it > 0) drain_wait(BAR(q_full), (q_it - 1) & 1, W.limit_ns);
            }
            __syncwarp();
        } else if (warp == 9) {
            // -------------------------------------------------------------- V loads
            uint32_t v_it = 0, land = 0;
            bool landing = false;   // an edge tile's copy was issued and not yet waited for
            for (uint32_t item_k = 0; !warp_aborted(abort_flag); ++item_k) {
                Item x;
                if (next_item(item_k, x) < 0) break;
                const WinRow za = x.a[0], zz = x.nrows > kBM ? x.z[1] : x.z[0];
                int ok = 1;
                for (int t = x.t0; t < x.t1 && ok; ++t) {
                    const int s = v_it % NS, j0 = x.all.at(t) * kBN;
                    const uint32_t dst = sbase + L::kV + s * L::kTile;
                    // every row of the tile seen by some row of the item: straight to the issuers
                    const bool whole = j0 + kBN <= za.s || (j0 >= za.lo && j0 + kBN <= zz.hi);
                    if (lane == 0) {
                        ok = wait1(BAR(v_empty) + 8u * (s), ((v_it / NS) & 1) ^ 1, W);
                        if (ok) {
                            const uint32_t bar = whole ? BAR(v_full) + 8u * (s) : BAR(v_land);
                            bar_expect_tx(bar, L::kTile);
#pragma unroll
                            for (int b = 0; b < NB; ++b)
                                tma_rows(dst + b * (kBN * 128), &tmV, b * 64, j0, x.hk, x.b, bar);
                            if (!whole) {
                                landing = true;
                                ok = wait1(BAR(v_land), land & 1, W);
                                landing = !ok;
                            }
                        }
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    __syncwarp();
                    if (!whole) {
                        ++land;
                        // a row is 128 bytes in each 64-channel box, whatever the swizzle does inside
                        for (int e = lane; e < kBN * NB * 8; e += 32) {
                            const int r = e / (NB * 8), j = j0 + r;
                            if (!(j < za.s || (j >= za.lo && j < zz.hi)))
                                *reinterpret_cast<uint4 *>(sm + L::kV + s * L::kTile + (e / 8 % NB) * (kBN * 128) + r * 128 +
                                                           (e % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) bar_arrive(BAR(v_full) + 8u * (s));
                    }
                    ++v_it;
                }
                if (!ok) break;
            }
            if (lane == 0)
                for (uint32_t v = v_it > (uint32_t)NS ? v_it - NS : 0; v < v_it; ++v)
                    drain_wait(BAR(v_full) + 8u * (v % NS), (v / NS) & 1, W.limit_ns);
            if (lane == 0 && landing) drain_wait(BAR(v_land), land & 1, W.limit_ns);
            __syncwarp();
        } else {
            // -------------------------------------------------------------- product issuers
            const int q = warp & 1;
            bool issued = false;
            if (lane == 0 && warp < 14) {
                constexpr uint32_t idesc_qk = f16_idesc(kBM, kBN, false), idesc_pv = f16_idesc(kBM, D, true);
                uint32_t it_s = 0, items = 0;   // stages and items (with products) so far
                uint32_t par = 0;               // bit b: parity of the next phase of buffer b that is waited for
                const uint32_t s_base = tmem + q * NSB * kBN, o_tm = tmem + 2 * NSB * kBN + q * D;
                const uint64_t qd = sw128_desc(sbase + L::kQ + q * L::kQTile, 16, 1024);
                for (uint32_t item_k = 0; !*abort_flag; ++item_k) {
                    const int slot = item_k % kRing;
                    if (!wait1(BAR(item_full) + 8u * (slot), (item_k / kRing) & 1, W)) break;
                    const int it = ring[slot];
                    const Item x = items_ring[slot];
                    bar_arrive(BAR(item_empty) + 8u * (slot));
                    if (it < 0) break;
                    if (x.t0 == x.t1) continue;
                    const WinTiles mine = pick(q == 1, x.q);
                    bool ok = true;
                    int n = 0;   // this Q tile's products in the item
                    issued = true;
                    if (warp < 12) {
                        // S(n) into buffer n % NSB, once P V has read what was there
                        ok = wait1(BAR(q_full), items & 1, W);
                        ++items;
                        for (int t = x.t0; t < x.t1 && ok; ++t, ++it_s) {
                            const int ks = it_s % NS;
                            ok = wait1(BAR(k_full) + 8u * ks, (it_s / NS) & 1, W);
                            if (ok && sees(mine, x.all.at(t))) {
                                const int buf = n % NSB;
                                ok = wait1(BAR(o_done) + 8u * (kMaxSB * q + buf), ((par >> buf) & 1u) ^ 1, W);
                                if (!ok) break;
                                par ^= 1u << buf;
                                tc_fence_after();
                                const uint64_t kd = sw128_desc(sbase + L::kK + ks * L::kTile, 16, 1024);
#pragma unroll
                                for (int kk = 0; kk < D / 16; ++kk) {
                                    const uint64_t offa = (uint64_t)(((kk >> 2) * (kBM * 128) + (kk & 3) * 32) >> 4);
                                    const uint64_t offb = (uint64_t)(((kk >> 2) * (kBN * 128) + (kk & 3) * 32) >> 4);
                                    mma_bf16(s_base + buf * kBN, qd + offa, kd + offb, idesc_qk, kk > 0);
                                }
                                mma_commit(BAR(s_full) + 8u * (kMaxSB * q + buf));
                                ++n;
                            }
                            if (!ok) break;
                            mma_commit(BAR(k_empty) + 8u * ks);
                            if (t == x.t1 - 1) mma_commit(BAR(q_empty));
                        }
                    } else {
                        // O += P(n) V
                        for (int t = x.t0; t < x.t1 && ok; ++t, ++it_s) {
                            const int vs = it_s % NS;
                            ok = wait1(BAR(v_full) + 8u * vs, (it_s / NS) & 1, W);
                            if (ok && sees(mine, x.all.at(t))) {
                                const int buf = n % NSB;
                                ok = wait1(BAR(p_full) + 8u * (kMaxSB * q + buf), (par >> buf) & 1u, W);
                                if (ok && n == 0) {
                                    ok = wait1(BAR(o_free) + 8u * q, (items & 1) ^ 1, W);
                                    ++items;
                                }
                                if (!ok) break;
                                par ^= 1u << buf;
                                tc_fence_after();
                                const uint64_t vd = sw128_desc(sbase + L::kV + vs * L::kTile, kBN * 128, 1024);
#pragma unroll
                                for (int kk = 0; kk < kBN / 16; ++kk)
                                    mma_bf16_ts(o_tm, s_base + buf * kBN + kk * 8, vd + (uint64_t)(kk * 2048 >> 4), idesc_pv,
                                                (n > 0 || kk > 0) ? 1u : 0u);
                                mma_commit(BAR(o_done) + 8u * (kMaxSB * q + buf));
                                ++n;
                            }
                            if (!ok) break;
                            mma_commit(BAR(v_empty) + 8u * vs);
                        }
                    }
                    if (!ok) break;
                }
                if (issued) {   // every product issued completes before TMEM is freed
                    mma_commit(BAR(drain) + 8u * (warp - 10));
                    drain_wait(BAR(drain) + 8u * (warp - 10), 0, W.limit_ns);
                }
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------------ softmax + epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int q = warp >> 2, row = threadIdx.x - q * kBM;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_col = q * NSB * kBN, o_col = 2 * NSB * kBN + q * D;
        uint32_t s_par = 0, o_par = 0;   // parities of the next s_full / of the o_done before the item
        const float c = a.scale_log2;
        auto pv_parity = [&](int j) -> uint32_t { return ((o_par >> (j % NSB)) + (uint32_t)(j / NSB)) & 1u; };
        // the item, and what this thread's row sees of it: taken while the last product of the item
        // before it runs
        const int r = q * kBM + row;
        Item next;
        WinRow next_lim;
        uint32_t item_k = 0;
        auto take = [&]() -> int {
            const int it = next_item(item_k++, next);
            if (it >= 0) next_lim = r < next.nrows ? win_row(a, next.first + r, next.kl) : WinRow{0, 0, 0};
            return it;
        };
        int it = take();
        while (it >= 0 && !warp_aborted(abort_flag)) {
            const Item x = next;
            const WinRow lim = next_lim;
            if (q * kBM >= x.nrows) {
                it = take();
                continue;
            }
            const bool valid = r < x.nrows;
            const WinTiles mine = pick(q == 1, x.q);
            const WinRow first_row = pick(q == 1, x.a), last_row = pick(q == 1, x.z);
            float m_run = -INFINITY, l = 0.f;
            int n = 0;
            bool ok = true;
            for (int t = x.t0; t < x.t1; ++t) {
                const int kt = x.all.at(t);
                if (!sees(mine, kt)) continue;
                const int b = n % NSB, j0 = kt * kBN;
                ok = waitw(BAR(s_full) + 8u * (kMaxSB * (q) + (b)), (s_par >> b) & 1u, W);
                if (!ok) break;
                s_par ^= 1u << b;
                tc_fence_after();
                const uint32_t sb_col = s_col + b * kBN;
                float s[kBN];
#pragma unroll
                for (int h = 0; h < kBN / 32; ++h) tmem_ld32(tmem + lane_base + sb_col + h * 32, s + h * 32);
                tmem_wait_ld(s);
                if (__builtin_expect(!win_all(first_row, last_row, j0, j0 + kBN), 0)) {
                    // bit j: whether the row sees key j0 + j
                    auto below = [&](int e) { return e <= 0 ? 0ull : (e >= 64 ? ~0ull : (1ull << e) - 1ull); };
                    const unsigned long long vis = below(lim.s - j0) | (below(lim.hi - j0) & ~below(lim.lo - j0));
                    const uint32_t v0 = (uint32_t)vis, v1 = (uint32_t)(vis >> 32);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (!((v0 >> j) & 1u)) s[j] = -INFINITY;
                        if (!((v1 >> j) & 1u)) s[32 + j] = -INFINITY;
                    }
                }
                float m8[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) m8[k] = s[k];
#pragma unroll
                for (int j = 8; j < kBN; j += 16)
#pragma unroll
                    for (int k = 0; k < 8; ++k) m8[k] = j + 8 < kBN ? fmax3(m8[k], s[j + k], s[j + 8 + k]) : fmaxf(m8[k], s[j + k]);
                const float mt = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])) * c;
                // the maximum that O and l are scaled by follows the row's only when it lags by
                // more than 8 (P <= 2^8, sums in fp32); -inf until the row has seen a key
                const bool need = mt > m_run + 8.f;
                if (__builtin_expect(n > 0 && __any_sync(0xffffffffu, need), 0)) {
                    ok = waitw(BAR(o_done) + 8u * (kMaxSB * (q) + ((n - 1) % NSB)), pv_parity(n - 1), W);
                    if (!ok) break;
                    tc_fence_after();
                    const float alpha = need ? fast_exp2(m_run - mt) : 1.f;
#pragma unroll 1
                    for (int h = 0; h < D / 32; ++h) {
                        float o[32];
                        tmem_ld32(tmem + lane_base + o_col + h * 32, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= alpha;
                        tmem_st32(tmem + lane_base + o_col + h * 32, o);
                    }
                    if (need) l *= alpha;
                }
                if (need) m_run = mt;
                const float m_use = m_run == -INFINITY ? 0.f : m_run;
                const unsigned long long c2 = f2pack(c, c), nm2 = f2pack(-m_use, -m_use);
                unsigned long long ls2[2] = {0ull, 0ull};
#pragma unroll
                for (int h = 0; h < kBN / 32; ++h) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 av = f2unpack(f2fma(f2pack(s[h * 32 + 2 * e], s[h * 32 + 2 * e + 1]), c2, nm2));
                        const float p0 = fast_exp2(av.x), p1 = fast_exp2(av.y);
                        ls2[e & 1] = f2add(ls2[e & 1], f2pack(p0, p1));
                        // P to bf16 for the product (half a step of 2^-7; l sums the fp32 values)
                        __nv_bfloat162 hh = __floats2bfloat162_rn(p0, p1);
                        pk[e] = *reinterpret_cast<uint32_t *>(&hh);
                    }
                    tmem_st16(tmem + lane_base + sb_col + h * 16, pk);
                }
                const float2 la = f2unpack(ls2[0]), lb = f2unpack(ls2[1]);
                l += (la.x + la.y) + (lb.x + lb.y);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                warp_arrive(BAR(p_full) + 8u * (kMaxSB * (q) + (b)), lane);
                ++n;
            }
            if (!ok) break;
            it = take();
            if (n > 0) {
                if (!waitw(BAR(o_done) + 8u * (kMaxSB * (q) + ((n - 1) % NSB)), pv_parity(n - 1), W)) break;
#pragma unroll
                for (int b = 0; b < NSB; ++b) o_par ^= (uint32_t)(((n + NSB - 1 - b) / NSB) & 1) << b;
                tc_fence_after();
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float lse2 = l == 0.f ? -INFINITY : m_run + log2f(l);
            const long long rix = win_row_index(a, x.b, x.h, x.r0 + (valid ? r : 0));
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.O) + x.b * a.lo.b + x.h * a.lo.h + (x.r0 + r) * a.lo.n;
            float *part = a.part_o + (rix * a.splits + x.split) * D;
#pragma unroll 1
            for (int h = 0; h < D / 32; ++h) {
                float o[32];
                if (n > 0) {
                    tmem_ld32(tmem + lane_base + o_col + h * 32, o);
                    tmem_wait_ld(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                if (!valid) continue;
                if (a.splits > 1) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4 *>(part + h * 32 + e) =
                            make_float4(o[e] * inv, o[e + 1] * inv, o[e + 2] * inv, o[e + 3] * inv);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t pk[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            __nv_bfloat162 hh = __floats2bfloat162_rn(o[e + 2 * k] * inv, o[e + 2 * k + 1] * inv);
                            pk[k] = *reinterpret_cast<uint32_t *>(&hh);
                        }
                        *reinterpret_cast<uint4 *>(dst + h * 32 + e) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                }
            }
            if (valid) {
                if (a.splits > 1) a.part_lse[rix * a.splits + x.split] = lse2;
                else if (a.lse) a.lse[rix] = lse2 * 0.6931471805599453f;
            }
            if (n > 0) {
                tc_fence_before();
                __syncwarp();
                warp_arrive(BAR(o_free) + 8u * (q), lane);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 10)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

template <int D>
cudaError_t launch_forward(WinArgs a, cudaStream_t s)
{
    CUtensorMap tq, tk, tv;
    if (!rows_map(&tq, a.Q, a.lq, a.B, a.H, a.Nq, D, kBM) || !rows_map(&tk, a.K, a.lk, a.B, a.Hkv, a.Nk, D, kBN) ||
        !rows_map(&tv, a.V, a.lv, a.B, a.Hkv, a.Nk, D, kBN))
        return cudaErrorInvalidValue;
    // the setmaxnreg split only adds up if the kernel was compiled to exactly kLaunchRegs
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, window_tc_kernel<D>) != cudaSuccess || fa.numRegs != kLaunchRegs)
        return cudaErrorInvalidDeviceFunction;
    const long long items = (long long)a.B * a.H * ((a.Nq + 2 * kBM - 1) / (2 * kBM)) * a.splits;
    if (items > 0x7ffffff0ll) return cudaErrorInvalidConfiguration;
    const int smem = Smem<D>::kAlloc;
    cudaError_t e = cudaFuncSetAttribute(window_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (items <= a.num_sms)
        a.counter = nullptr;   // nothing to clear first (some 2 us of a call)
    else if ((e = cudaMemsetAsync(a.status, 0, (char *)(a.counter + 1) - (char *)a.status, s)) != cudaSuccess)
        return e;
    return launch_early(window_tc_kernel<D>, dim3((unsigned)(items < a.num_sms ? items : a.num_sms)), kThreads, smem, s, 1, tq, tk,
                        tv, a, (int)items);
}

#undef BAR

}  // namespace

cudaError_t window_tc_forward(const WinArgs &a, cudaStream_t s)
{
    return a.d == 64 ? launch_forward<64>(a, s) : launch_forward<128>(a, s);
}

}  // namespace scope
