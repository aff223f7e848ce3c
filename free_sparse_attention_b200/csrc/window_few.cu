// Window attention for few query rows over a long cache (bf16): tiles of up to 16 rows, query heads
// of one key head together, so that a key and its value are read once for all of them.
//
// Bound by HBM: 4 d bytes per key and key head against 4 d flops per row.  A block of 4 warps
// owns one share of the unit's keys; each warp walks its own 16-key tiles through its own ring
// in shared memory (cp.async, no block barrier in the loop): S = Q K^T as mma m16n8k16 with the
// 16 rows as M, a running maximum and sum per row in fp32, O += P V.  With 16 rows the legacy
// matrix instructions take a fifth of the time the loads need; a tcgen05 tile would be 7/8 idle
// rows and pay the TMEM round trip.  Two blocks share an SM: 3 tiles of 8 KB per warp keep
// 128 KB of loads in flight there.  The warps join through shared memory, and the shares of a unit,
// up to 6, as one cluster through distributed shared memory, in order.
// Measured (B200): one row of 40 heads over 9360 visible keys of 32760, d 128: 35.7 us = 5.4 TB/s.
// Rows of a 16-key tile lie at 2 d bytes, 16-byte chunk c of row r at c ^ (r mod 8): the 8 rows
// of an ldmatrix meet different banks.
#include "window.cuh"

#include <cooperative_groups.h>

namespace scope {

namespace {

constexpr int kTileKeys = 16, kFewWarps = 4, kStages = 3;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool fill)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// c += a b, m16n8k16: rows lane / 4 and + 8, columns 2 (lane % 4) and + 1.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2(float x, float y)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float quad_max(float v)
{
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

__device__ __forceinline__ float quad_sum(float v)
{
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// CLUSTER: the shares of a unit are one thread-block cluster and join through distributed shared
// memory; otherwise window_join_kernel joins them.
template <int D, bool CLUSTER>
__global__ void __launch_bounds__(kFewWarps * 32, 2) window_few_kernel(WinArgs a)
{
    constexpr int CH = D / 8;                       // 16-byte chunks of a row
    constexpr int kTileBytes = kTileKeys * D * 2;   // K or V
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float sm_m[kFewWarps][16], sm_l[kFewWarps][16], sm_bm[16], sm_bl[16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tg = lane & 3, tr = lane >> 2;
    early_next();
    early_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;   // this path has no device conditions
    const int split = blockIdx.x % a.splits, unit = blockIdx.x / a.splits;
    const int groups = a.H / a.pack, b = unit / groups, h0 = (unit - b * groups) * a.pack, hk = h0 / (a.H / a.Hkv);
    const int rows = a.pack * a.Nq;
    const int first = win_first(a, b), kl = win_klen(a, b);
    const WinRow ra = win_row(a, first, kl), rz = win_row(a, first + a.Nq - 1, kl);
    const WinTiles wt = win_tiles<kTileKeys>(ra, rz);
    const int nt = wt.count(), t0 = (int)((long long)nt * split / a.splits), t1 = (int)((long long)nt * (split + 1) / a.splits);

    const __nv_bfloat16 *kb = static_cast<const __nv_bfloat16 *>(a.K) + b * a.lk.b + hk * a.lk.h;
    const __nv_bfloat16 *vb = static_cast<const __nv_bfloat16 *>(a.V) + b * a.lv.b + hk * a.lv.h;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (kStages * 2 * kTileBytes);
    // this lane's part of a tile: chunk `chunk` of rows lane_row, lane_row + step, ...
    constexpr int STEP = 32 / CH > 0 ? 32 / CH : 1;
    const int chunk = lane % CH, lane_row = lane / CH;
    const __nv_bfloat16 *kl0 = kb + lane_row * a.lk.n + 8 * chunk, *vl0 = vb + lane_row * a.lv.n + 8 * chunk;
    auto issue = [&](int t, int s) {   // tile t (of this warp) into stage s; rows nobody sees become zeros
        if (t < t1) {
            const int j0 = wt.at(t) * kTileKeys;
            const uint32_t dst = ring + s * (2 * kTileBytes);
            const __nv_bfloat16 *kp = kl0 + j0 * a.lk.n, *vp = vl0 + j0 * a.lv.n;
            const bool whole = j0 + kTileKeys <= ra.s || (j0 >= ra.lo && j0 + kTileKeys <= rz.hi);
#pragma unroll
            for (int i = 0; i < kTileKeys / STEP; ++i) {
                const int r = lane_row + i * STEP, j = j0 + r;
                const bool seen = whole || j < ra.s || (j >= ra.lo && j < rz.hi);
                const uint32_t off = r * (2 * D) + ((chunk ^ (r & 7)) << 4);
                cp_async16(dst + off, seen ? kp : kb, seen);
                cp_async16(dst + kTileBytes + off, seen ? vp : vb, seen);
                kp += STEP * a.lk.n;
                vp += STEP * a.lv.n;
            }
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue(t0 + warp + s * kFewWarps, s);

    // Q as A fragments: rows tr and tr + 8 (row r: head h0 + r / Nq, query r % Nq)
    uint32_t qf[D / 16][4];
    WinRow lim[2];
    const __nv_bfloat16 *qp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = tr + 8 * i;
        const bool in = r < rows;
        const int h = h0 + (in ? r / a.Nq : 0), q = in ? r % a.Nq : 0;
        qp[i] = in ? static_cast<const __nv_bfloat16 *>(a.Q) + b * a.lq.b + h * a.lq.h + q * a.lq.n : nullptr;
        lim[i] = in ? win_row(a, first + q, kl) : WinRow{0, 0, 0};
    }
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat16 *p = qp[e & 1];
            qf[kk][e] = p ? *reinterpret_cast<const uint32_t *>(p + kk * 16 + 2 * tg + (e >> 1) * 8) : 0u;
        }

    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < D / 8; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
    // this lane's row of the four 8 x 8 matrices of an ldmatrix, for K and (transposed) for V
    const int kr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
    const int vr = (lane & 7) + (((lane >> 3) & 1) << 3), vc = lane >> 4;
    int s = 0;
    for (int t = t0 + warp; t < t1; t += kFewWarps) {
        issue(t + (kStages - 1) * kFewWarps, s == 0 ? kStages - 1 : s - 1);
        asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        const uint32_t base = ring + s * (2 * kTileBytes);
        const int j0 = wt.at(t) * kTileKeys;
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t kf[4];
            ldmatrix4(kf, base + kr * (2 * D) + (((2 * kk + kc) ^ (kr & 7)) << 4));
            mma16816(sc[0], qf[kk], kf[0], kf[1]);
            mma16816(sc[1], qf[kk], kf[2], kf[3]);
        }
        const bool all = win_all(ra, rz, j0, j0 + kTileKeys);
        float p[2][4], corr[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // row tr + 8 i: values 2 i, 2 i + 1 of each 8-key half
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = j0 + (e >> 1) * 8 + 2 * tg + (e & 1);
                const bool vis = all || j < lim[i].s || (j >= lim[i].lo && j < lim[i].hi);
                v[e] = vis ? sc[e >> 1][2 * i + (e & 1)] * a.scale_log2 : -INFINITY;
            }
            const float mn = fmaxf(m[i], quad_max(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]))));
            const float use = mn == -INFINITY ? 0.f : mn;
            corr[i] = exp2f(m[i] - use);
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[i][e] = exp2f(v[e] - use);
                sum += p[i][e];
            }
            l[i] = l[i] * corr[i] + sum;
            m[i] = mn;
        }
        if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                o[c][0] *= corr[0];
                o[c][1] *= corr[0];
                o[c][2] *= corr[1];
                o[c][3] *= corr[1];
            }
        }
        // P (16 rows x 16 keys) as the A operand, rounded to bf16
        const uint32_t pf[4] = {pack2(p[0][0], p[0][1]), pack2(p[1][0], p[1][1]), pack2(p[0][2], p[0][3]),
                                pack2(p[1][2], p[1][3])};
#pragma unroll
        for (int c = 0; c < D / 8; c += 2) {
            uint32_t vf[4];
            ldmatrix4_trans(vf, base + kTileBytes + vr * (2 * D) + (((c + vc) ^ (vr & 7)) << 4));
            mma16816(o[c], pf, vf[0], vf[1]);
            mma16816(o[c + 1], pf, vf[2], vf[3]);
        }
        __syncwarp();   // every lane is done with the stage before it is filled again
        s = s + 1 == kStages ? 0 : s + 1;
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    __syncthreads();

    // join the warps: all scaled to the largest of their maxima (a NaN stays one)
    float *so = reinterpret_cast<float *>(smem);   // [warp][16][D]
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] = quad_sum(l[i]);
        if (tg == 0) {
            sm_m[warp][tr + 8 * i] = m[i];
            sm_l[warp][tr + 8 * i] = l[i];
        }
    }
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float2 *>(so + (warp * 16 + tr + 8 * i) * D + c * 8 + 2 * tg) =
                make_float2(o[c][2 * i], o[c][2 * i + 1]);
    __syncthreads();
    // 4 channels of row r: out (already divided by the row sum), lse2 by the thread of channel 0
    auto write = [&](int r, int c, const float (&x)[4], float lse2) {
        const int h = h0 + r / a.Nq, q = r % a.Nq;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.O) + b * a.lo.b + h * a.lo.h + q * a.lo.n + c;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
        if (c == 0 && a.lse) a.lse[win_row_index(a, b, h, q)] = lse2 * 0.6931471805599453f;
    };
    for (int e = threadIdx.x; e < rows * (D / 4); e += kFewWarps * 32) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) mm = fmaxf(mm, sm_m[w][r]);
        const float use = mm == -INFINITY ? 0.f : mm;
        float sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            const float f = exp2f(sm_m[w][r] - use);
            const float4 y = *reinterpret_cast<const float4 *>(so + (w * 16 + r) * D + c);
            sum = fmaf(f, sm_l[w][r], sum);
            x[0] = fmaf(f, y.x, x[0]);
            x[1] = fmaf(f, y.y, x[1]);
            x[2] = fmaf(f, y.z, x[2]);
            x[3] = fmaf(f, y.w, x[3]);
        }
        if (CLUSTER) {   // this share's row, for the cluster: the thread overwrites what it alone read
            *reinterpret_cast<float4 *>(so + r * D + c) = make_float4(x[0], x[1], x[2], x[3]);
            if (c == 0) {
                sm_bm[r] = mm;
                sm_bl[r] = sum;
            }
            continue;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const float lse2 = sum == 0.f ? -INFINITY : use + log2f(sum);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] *= inv;
        if (a.splits > 1) {
            const long long row = win_row_index(a, b, h0 + r / a.Nq, r % a.Nq);
            *reinterpret_cast<float4 *>(a.part_o + (row * a.splits + split) * D + c) = make_float4(x[0], x[1], x[2], x[3]);
            if (c == 0) a.part_lse[row * a.splits + split] = lse2;
        } else {
            write(r, c, x, lse2);
        }
    }
    if constexpr (CLUSTER) {
        // every block joins its part of the rows over all shares, in order
        const auto cluster = cooperative_groups::this_cluster();
        cluster.sync();
        for (int e = split * (kFewWarps * 32) + threadIdx.x; e < rows * (D / 4); e += a.splits * (kFewWarps * 32)) {
            const int r = e / (D / 4), c = (e % (D / 4)) * 4;
            float mm = -INFINITY;
            for (int k = 0; k < a.splits; ++k) mm = fmaxf(mm, cluster.map_shared_rank(sm_bm, k)[r]);
            const float use = mm == -INFINITY ? 0.f : mm;
            float sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
            for (int k = 0; k < a.splits; ++k) {
                const float f = exp2f(cluster.map_shared_rank(sm_bm, k)[r] - use);
                const float4 y = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(so, k) + r * D + c);
                sum = fmaf(f, cluster.map_shared_rank(sm_bl, k)[r], sum);
                x[0] = fmaf(f, y.x, x[0]);
                x[1] = fmaf(f, y.y, x[1]);
                x[2] = fmaf(f, y.z, x[2]);
                x[3] = fmaf(f, y.w, x[3]);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] *= inv;
            write(r, c, x, sum == 0.f ? -INFINITY : use + log2f(sum));
        }
        cluster.sync();   // no block leaves while another reads its memory
    }
}

template <int D, bool CLUSTER>
cudaError_t launch(const WinArgs &a, cudaStream_t s)
{
    const int smem = kFewWarps * kStages * 2 * kTileKeys * D * 2;
    static_assert(kFewWarps * 16 * D * 4 <= kFewWarps * kStages * 2 * kTileKeys * D * 2, "the join fits in the ring");
    const long long grid = (long long)a.B * (a.H / a.pack) * a.splits;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(window_few_kernel<D, CLUSTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_early(window_few_kernel<D, CLUSTER>, dim3((unsigned)grid), kFewWarps * 32, smem, s,
                        CLUSTER ? (unsigned)a.splits : 1u, a);
}

template <int D>
cudaError_t forward(const WinArgs &a, cudaStream_t s)
{
    // Up to 6 shares as a cluster (16 x 8 units of 2: 50 us against 53 with a second kernel; 40 units of
    // 6: 39.5 against 41.5); larger ones leave slots of a GPC empty (40 units of 7: 60 us against 42).
    if (a.splits > 1 && a.splits <= kFewCluster) return launch<D, true>(a, s);
    cudaError_t e = launch<D, false>(a, s);
    return e == cudaSuccess && a.splits > 1 ? window_join(a, s) : e;
}

}  // namespace

cudaError_t window_few_forward(const WinArgs &a, cudaStream_t s)
{
    return a.d == 64 ? forward<64>(a, s) : forward<128>(a, s);
}

}  // namespace scope
