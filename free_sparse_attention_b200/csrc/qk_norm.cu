// RMS norm of queries and keys per head, a weight per channel, and 3D RoPE, in one pass;
// and its gradients.
//
//   r = 1 / sqrt(mean_c x_c^2 + eps),  xh = x r,  u = w o xh,  y = R u,
// R turning the pairs (2i, 2i+1) of each axis range by phi = position * base^(-2i / d_axis).
// Backward, with g = R^T dy:  dw = sum over rows of g o xh,
//   dx = r (w o g - xh mean_c(w o g o xh)).
//
// HBM-bound: every element is read once and written once.  A block owns a run of consecutive
// tokens and walks the heads: a thread keeps 8 channels of one token, so cos and sin of its 4
// pairs are computed once and serve all its heads, with no table in memory (any position, any
// frame size).  The angle is taken in turns in binary64 and reduced there (position times a
// frequency that was rounded to binary64 once: the fraction is off by about 2^-52 of the turns),
// then cos and sin in fp32.  Statistics, products and the weight gradients are fp32; the result is rounded once.
// Measured (B200): 80 heads x 32760 tokens, d 128, bf16 207 us = 6.5 TB/s, the device's copy rate;
// backward of 96 heads x 17550, d 64: 111 to 122 us = 5.3 to 5.8 TB/s, bound by instruction issue
// (79 %) before the memory.
#include "qk_norm.cuh"
#include "early.cuh"

#include <algorithm>

namespace scope {

namespace {

constexpr int kThreads = 256;
template <typename T>
constexpr int kFwdBlocks = sizeof(T) == 2 ? 4 : 3;   // blocks per SM (registers)
template <typename T>
constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;       // forward: rows of a thread in flight while it works on as many
template <typename T>
constexpr int kBwdBlocks = sizeof(T) == 2 ? 4 : 2;
template <typename T>
constexpr int kBwdStages = sizeof(T) == 2 ? 6 : 3;   // backward: rows of the ring (see Feed)

__device__ __forceinline__ void get8(const __nv_bfloat16 *p, float (&x)[8])
{
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        x[2 * q] = __uint_as_float(w[q] << 16);
        x[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void get8(const float *p, float (&x)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&y)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * q], y[2 * q + 1]);
        w[q] = *reinterpret_cast<const uint32_t *>(&h);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

__device__ __forceinline__ void store8(float *p, const float (&y)[8])
{
    __stcs(reinterpret_cast<float4 *>(p), make_float4(y[0], y[1], y[2], y[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(y[4], y[5], y[6], y[7]));
}

// cos and sin of the 4 pairs of channel group g at token position pos.
__device__ __forceinline__ void pair_angles(const NormArgs &a, int g, int pos, float (&cs)[4], float (&sn)[4])
{
    const int plane = a.Hg * a.Wg, t = pos / plane, rem = pos - t * plane, h = rem / a.Wg, w = rem - h * a.Wg;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int c = 8 * g + 2 * q;
        const double p = c < a.dt ? t : (c < a.dt + a.dh ? h : w);
        double turns = p * a.freq[c / 2];
        turns -= rint(turns);
        sincospif((float)(2.0 * turns), &sn[q], &cs[q]);
    }
}

template <int TPR>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int x = TPR / 2; x; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
    return v;
}

// A block's place: token run, batch entry and a chunk of the heads of q (which = 0) or k (1).
struct Place {
    int b, tile, h0, h1;
};

__device__ __forceinline__ Place place_of(const NormArgs &a, int which, long long it)
{
    const int chunks = which ? a.chunks_k : a.chunks_q;
    Place p;
    p.h0 = (int)(it % chunks) * a.chunk;
    it /= chunks;
    p.tile = (int)(it % a.tiles);
    p.b = (int)(it / a.tiles);
    p.h1 = min(which ? a.Hkv : a.H, p.h0 + a.chunk);
    return p;
}

// Backward: the token runs times the heads of q (or k), head after head, are cut evenly over the
// blocks.  The place at position `pos` of a block's share, which ends at `end`: heads of one token
// run, no more than 32 of them.
__device__ __forceinline__ Place span_of(const NormArgs &a, int which, int pos, int end)
{
    const int heads = which ? a.Hkv : a.H, run = pos / heads;
    Place p;
    p.h0 = pos - run * heads;
    p.h1 = min(min(heads, p.h0 + 32), p.h0 + end - pos);
    p.b = run / a.tiles;
    p.tile = run - p.b * a.tiles;
    return p;
}

// The rows of a thread's places, in order, streamed through a ring of its own in shared memory
// (cp.async; no thread reads another's slots): STAGES - 1 rows of X (and G) are in flight
// whatever the registers hold, across the ends of places too.
template <typename T, int D, bool GRAD, int STAGES>
struct Feed {
    static constexpr int TPR = D / 8, ROWS = kThreads / TPR, BYTES = 8 * sizeof(T);   // of one thread's 8 channels
    static constexpr int kSmem = STAGES * (GRAD ? 2 : 1) * kThreads * BYTES;
    const NormArgs &a;
    const NormTensor &x;
    const int which, end;
    int pos;               // of the next row to load, its head, and the end of the place's heads
    int h, h1;
    const T *src, *grd;
    T *slots;              // slot s of X at s * kThreads * 8, of G behind the STAGES slots of X
    int fill;

    __device__ __forceinline__ Feed(const NormArgs &args, int w, int from, int to, void *smem)
        : a(args), x(w ? args.k : args.q), which(w), end(to), pos(from), h(0), h1(0),
          slots(static_cast<T *>(smem) + threadIdx.x * 8), fill(0)
    {
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) next();
    }

    __device__ __forceinline__ T *slot(int s, int tensor) const { return slots + (tensor * STAGES + s) * (kThreads * 8); }

    __device__ __forceinline__ void next()
    {
        if (pos < end) {
            if (h == h1) {
                const Place p = span_of(a, which, pos, end);
                const int n = min(p.tile * ROWS + (int)threadIdx.x / TPR, a.N - 1), c = 8 * (threadIdx.x % TPR);
                h = p.h0;
                h1 = p.h1;
                src = static_cast<const T *>(x.X) + p.b * x.lx.b + n * x.lx.n + h * x.lx.h + c;
                if (GRAD) grd = static_cast<const T *>(x.G) + p.b * x.lg.b + n * x.lg.n + h * x.lg.h + c;
            }
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i) {
                copy16(slot(fill, 0) + i * (16 / sizeof(T)), src + i * (16 / sizeof(T)));
                if (GRAD) copy16(slot(fill, 1) + i * (16 / sizeof(T)), grd + i * (16 / sizeof(T)));
            }
            ++pos;
            ++h;
            src += x.lx.h;
            if (GRAD) grd += x.lg.h;
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");   // one group per row, empty past the end
        fill = fill + 1 == STAGES ? 0 : fill + 1;
    }

    static __device__ __forceinline__ void copy16(T *dst, const T *from)
    {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(from)
                     : "memory");
    }
};


// 8 channels of a row as they lie in memory.
template <typename T>
struct Row8 {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    }
};


// Forward.  One place per block (the hardware's block scheduler balances them), rows in
// registers one batch ahead.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kFwdBlocks<T>) qk_norm_kernel(NormArgs a)
{
    constexpr int TPR = D / 8, M = kBatch<T>;
    early_next();
    early_wait();
    const int which = blockIdx.x >= a.blocks_q;
    const Place pl = place_of(a, which, which ? blockIdx.x - a.blocks_q : blockIdx.x);
    const int g = threadIdx.x % TPR, n = pl.tile * (kThreads / TPR) + threadIdx.x / TPR;
    const bool in = n < a.N;
    const int nn = in ? n : a.N - 1;   // idle threads repeat the last token and store nothing
    const NormTensor &x = which ? a.k : a.q;
    const T *src = static_cast<const T *>(x.X) + pl.b * x.lx.b + nn * x.lx.n + pl.h0 * x.lx.h + 8 * g;
    T *dst = static_cast<T *>(x.Y) + pl.b * x.ly.b + nn * x.ly.n + pl.h0 * x.ly.h + 8 * g;
    const int heads = pl.h1 - pl.h0;
    Row8<T> next[M];
#pragma unroll
    for (int j = 0; j < M; ++j)
        if (j < heads) next[j].load(src + j * x.lx.h);
    float w[8], cs[4], sn[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = x.w ? x.w[8 * g + e] : 1.f;
    pair_angles(a, g, norm_first(a, pl.b) + nn, cs, sn);
    for (int h = 0; h < heads; h += M) {
        Row8<T> now[M];
        src += M * x.lx.h;
#pragma unroll
        for (int j = 0; j < M; ++j) {
            now[j] = next[j];
            if (h + M + j < heads) next[j].load(src + j * x.lx.h);
        }
#pragma unroll
        for (int j = 0; j < M; ++j) {
            if (h + j >= heads) break;
            float v[8], y[8], s = 0.f;
            get8(reinterpret_cast<const T *>(now[j].v), v);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(v[e], v[e], s);
            const float r = __frsqrt_rn(group_sum<TPR>(s) * (1.f / D) + a.eps);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float u0 = v[2 * q] * r * w[2 * q], u1 = v[2 * q + 1] * r * w[2 * q + 1];
                y[2 * q] = fmaf(u0, cs[q], -u1 * sn[q]);
                y[2 * q + 1] = fmaf(u0, sn[q], u1 * cs[q]);
            }
            if (in) store8(dst, y);
            dst += x.ly.h;
        }
    }
}

// Backward.  A thread sums its weight gradients over its rows (one sum per place, added to the
// thread's total, so that no sum runs over more than 32 heads before it joins the next
// level), the block adds its token rows up in shared memory and writes one partial, and
// qk_norm_dw_kernel adds the partials in block order.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kBwdBlocks<T>) qk_norm_bwd_kernel(NormArgs a)
{
    constexpr int TPR = D / 8, ROWS = kThreads / TPR, STAGES = kBwdStages<T>;
    extern __shared__ __align__(16) unsigned char smem[];
    early_next();
    early_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    const int which = blockIdx.x >= a.blocks_q, first = which ? blockIdx.x - a.blocks_q : blockIdx.x,
              blocks = which ? gridDim.x - a.blocks_q : a.blocks_q;
    const long long rows = (long long)a.B * a.tiles * (which ? a.Hkv : a.H);
    const int from = (int)(rows * first / blocks), to = (int)(rows * (first + 1) / blocks);
    Feed<T, D, true, STAGES> feed(a, which, from, to, smem);
    const NormTensor &x = which ? a.k : a.q;
    const int g = threadIdx.x % TPR;
    float dw[8], w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        dw[e] = 0.f;
        w[e] = x.w ? x.w[8 * g + e] : 1.f;
    }
    int take = 0;
    for (int pos = from; pos < to;) {
        const Place pl = span_of(a, which, pos, to);
        pos += pl.h1 - pl.h0;
        const int n = pl.tile * ROWS + threadIdx.x / TPR;
        const bool in = n < a.N;
        T *dst = static_cast<T *>(x.Y) + pl.b * x.ly.b + n * x.ly.n + pl.h0 * x.ly.h + 8 * g;
        float cs[4], sn[4], sum[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = 0.f;
        pair_angles(a, g, norm_first(a, pl.b) + min(n, a.N - 1), cs, sn);
        for (int h = pl.h0; h < pl.h1; ++h) {
            feed.next();
            asm volatile("cp.async.wait_group %0;\n" ::"n"(STAGES - 1) : "memory");
            float v[8], gr[8], s = 0.f, t = 0.f;
            get8(feed.slot(take, 0), v);
            get8(feed.slot(take, 1), gr);
            take = take + 1 == STAGES ? 0 : take + 1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float d0 = gr[2 * q], d1 = gr[2 * q + 1];
                gr[2 * q] = fmaf(d0, cs[q], d1 * sn[q]);
                gr[2 * q + 1] = fmaf(d1, cs[q], -d0 * sn[q]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s = fmaf(v[e], v[e], s);
                t = fmaf(gr[e] * w[e], v[e], t);
            }
            const float r = __frsqrt_rn(group_sum<TPR>(s) * (1.f / D) + a.eps);
            const float c = group_sum<TPR>(t) * (1.f / D) * r * r;   // xh * mean(w g xh) = v * c
            float dx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dx[e] = r * fmaf(gr[e], w[e], -v[e] * c);
                sum[e] = fmaf(gr[e], v[e] * r, sum[e]);
            }
            if (in) store8(dst, dx);
            dst += x.ly.h;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] += in ? sum[e] : 0.f;
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);   // [ROWS][D]
    static_assert(ROWS * D * 4 <= Feed<T, D, true, STAGES>::kSmem, "the partials fit in the ring");
#pragma unroll
    for (int e = 0; e < 8; ++e) red[threadIdx.x / TPR * D + 8 * g + e] = dw[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < ROWS; ++k) s += red[k * D + threadIdx.x];
        a.partial[(long long)blockIdx.x * D + threadIdx.x] = s;
    }
}

// dw[c] = sum over the blocks of q (or k) of partial[block][c]: 32 channels per block, 32
// threads per channel each adding every 32nd partial, joined in a fixed order.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(NormArgs a, int blocks, int D)
{
    __shared__ float red[32][33];
    early_wait();
    const int which = blockIdx.x / (D / 32), c = (blockIdx.x % (D / 32)) * 32 + threadIdx.x % 32, k = threadIdx.x / 32;
    const int first = which ? a.blocks_q : 0, last = which ? blocks : a.blocks_q;
    float s = 0.f;
    for (int j = first + k; j < last; j += 32) s += a.partial[(long long)j * D + c];
    red[k][threadIdx.x % 32] = s;
    __syncthreads();
    s = red[threadIdx.x % 32][k];   // warp k: channel k of the 32
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    float *dw = which ? a.k.dw : a.q.dw;
    if (threadIdx.x % 32 == 0 && dw) dw[(blockIdx.x % (D / 32)) * 32 + k] = s;
}

// Heads per place, in equal chunks of q's heads: as many as leave 16 places per SM, but 4 to 20.
// Fewer than 4 and the evaluation of the angles outweighs the rows (2 heads: 16 us against 12 at
// 16 heads x 8194 tokens fp32); more than 20 gain nothing on it and leave a longer tail
// (40 heads: 212 us against 207 at 80 heads x 32760 tokens).
void plan(NormArgs &a, int num_sms)
{
    a.tiles = (a.N + kThreads / (a.d / 8) - 1) / (kThreads / (a.d / 8));
    const int heads = a.H + (a.k.X ? a.Hkv : 0);
    const long long runs = (long long)a.B * a.tiles, want = 16ll * num_sms;
    const int per = (int)std::min<long long>((want + runs - 1) / runs, heads);   // places wanted per token run
    const int chunk = std::min(std::max((heads + per - 1) / per, 4), 20), parts = (a.H + chunk - 1) / chunk;
    a.chunk = (a.H + parts - 1) / parts;
    a.chunks_q = parts;
    a.chunks_k = a.k.X ? (a.Hkv + a.chunk - 1) / a.chunk : 0;
}

template <typename T, int D>
cudaError_t forward(NormArgs a, int num_sms, cudaStream_t s)
{
    plan(a, num_sms);
    const long long runs = (long long)a.B * a.tiles, grid = runs * (a.chunks_q + a.chunks_k);
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    a.blocks_q = (int)(runs * a.chunks_q);
    return launch_early(qk_norm_kernel<T, D>, dim3((unsigned)grid), kThreads, 0, s, 1, a);
}

template <typename T, int D>
cudaError_t backward(NormArgs a, int num_sms, cudaStream_t s)
{
    const int per_sm = kBwdBlocks<T>, sms = std::min(num_sms, kNormMaxBlocks / per_sm);
    a.tiles = (a.N + kThreads / (D / 8) - 1) / (kThreads / (D / 8));
    // blocks in proportion to the rows of q and of k, at least one each, of 4 heads or more
    const long long rows = (long long)a.B * a.tiles * (a.H + (a.k.X ? a.Hkv : 0));
    const int grid = (int)std::max<long long>(a.k.X ? 2 : 1, std::min<long long>(rows / 4, (long long)sms * per_sm));
    a.blocks_q = grid;
    if (a.k.X) a.blocks_q = std::min(std::max(1, (int)((long long)grid * a.H / (a.H + a.Hkv))), grid - 1);
    const int smem = Feed<T, D, true, kBwdStages<T>>::kSmem;
    cudaError_t e = cudaFuncSetAttribute(qk_norm_bwd_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if ((e = launch_early(qk_norm_bwd_kernel<T, D>, dim3(grid), kThreads, smem, s, 1, a)) != cudaSuccess) return e;
    return launch_early(qk_norm_dw_kernel, dim3(2 * (D / 32)), 1024, 0, s, 1, a, grid, D);
}

}  // namespace

cudaError_t qk_norm_forward(const NormArgs &a, int num_sms, cudaStream_t s)
{
    if (a.is_bf16) return a.d == 64 ? forward<__nv_bfloat16, 64>(a, num_sms, s) : forward<__nv_bfloat16, 128>(a, num_sms, s);
    return a.d == 64 ? forward<float, 64>(a, num_sms, s) : forward<float, 128>(a, num_sms, s);
}

cudaError_t qk_norm_backward(const NormArgs &a, int num_sms, cudaStream_t s)
{
    if (a.is_bf16) return a.d == 64 ? backward<__nv_bfloat16, 64>(a, num_sms, s) : backward<__nv_bfloat16, 128>(a, num_sms, s);
    return a.d == 64 ? backward<float, 64>(a, num_sms, s) : backward<float, 128>(a, num_sms, s);
}

}  // namespace scope
