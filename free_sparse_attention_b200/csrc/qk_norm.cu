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
// binary64 frequency: the error of the fraction is below 2^-52 of the turns), then cos and sin
// in fp32.  Statistics, products and the weight gradients are fp32; the result is rounded once.
// HEADS rows per thread are in flight at a time.
#include "qk_norm.cuh"

namespace scope {

namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;   // rows of one thread in flight

// 8 channels of one row in fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8])
{
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        x[2 * q] = __uint_as_float(w[q] << 16);
        x[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void load8(const float *p, float (&x)[8])
{
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
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
    int b, tile, which, h0, h1;
};

__device__ __forceinline__ Place place_of(const NormArgs &a, long long it)
{
    Place p;
    const int c = (int)(it % (a.chunks_q + a.chunks_k));
    it /= a.chunks_q + a.chunks_k;
    p.tile = (int)(it % a.tiles);
    p.b = (int)(it / a.tiles);
    p.which = c >= a.chunks_q;
    const int k = p.which ? c - a.chunks_q : c;
    p.h0 = k * a.chunk;
    p.h1 = min(p.which ? a.Hkv : a.H, p.h0 + a.chunk);
    return p;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(NormArgs a)
{
    constexpr int TPR = D / 8;
    const Place pl = place_of(a, blockIdx.x);
    const int g = threadIdx.x % TPR, n = pl.tile * (kThreads / TPR) + threadIdx.x / TPR;
    const bool in = n < a.N;
    const int nn = in ? n : a.N - 1;   // idle threads repeat the last token and store nothing
    const NormTensor &x = pl.which ? a.k : a.q;
    const T *src = static_cast<const T *>(x.X) + pl.b * x.lx.b + nn * x.lx.n + 8 * g;
    T *dst = static_cast<T *>(x.Y) + pl.b * x.ly.b + nn * x.ly.n + 8 * g;
    float v[kHeads][8];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) load8(src + min(pl.h0 + j, pl.h1 - 1) * x.lx.h, v[j]);
    float w[8], cs[4], sn[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = x.w ? x.w[8 * g + e] : 1.f;
    pair_angles(a, g, norm_first(a, pl.b) + nn, cs, sn);
    for (int h = pl.h0; h < pl.h1; h += kHeads) {
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(v[j][e], v[j][e], s);
            const float r = __frsqrt_rn(group_sum<TPR>(s) * (1.f / D) + a.eps);
            float y[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float u0 = v[j][2 * q] * r * w[2 * q], u1 = v[j][2 * q + 1] * r * w[2 * q + 1];
                y[2 * q] = fmaf(u0, cs[q], -u1 * sn[q]);
                y[2 * q + 1] = fmaf(u0, sn[q], u1 * cs[q]);
            }
            if (in && h + j < pl.h1) store8(dst + (h + j) * x.ly.h, y);
        }
        if (h + kHeads < pl.h1)
#pragma unroll
            for (int j = 0; j < kHeads; ++j) load8(src + min(h + kHeads + j, pl.h1 - 1) * x.lx.h, v[j]);
    }
}

// Backward: a persistent grid; every thread sums its weight gradients over its rows (one sum
// per place, added to the thread's total, so that no sum runs over more than a chunk of heads
// before it joins the next level), the block adds its token rows up in shared memory and
// writes one partial per tensor, and qk_norm_dw_kernel adds the partials in block order.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) qk_norm_bwd_kernel(NormArgs a)
{
    constexpr int TPR = D / 8, ROWS = kThreads / TPR;
    __shared__ float red[ROWS][D];
    const int g = threadIdx.x % TPR;
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.status) *a.status = 0;
    const long long places = (long long)a.B * a.tiles * (a.chunks_q + a.chunks_k);
    float dw[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.f;
    for (long long it = blockIdx.x; it < places; it += gridDim.x) {
        const Place pl = place_of(a, it);
        const int n = pl.tile * ROWS + threadIdx.x / TPR;
        const bool in = n < a.N;
        const int nn = in ? n : a.N - 1;
        const NormTensor &x = pl.which ? a.k : a.q;
        const T *src = static_cast<const T *>(x.X) + pl.b * x.lx.b + nn * x.lx.n + 8 * g;
        const T *grd = static_cast<const T *>(x.G) + pl.b * x.lg.b + nn * x.lg.n + 8 * g;
        T *dst = static_cast<T *>(x.Y) + pl.b * x.ly.b + nn * x.ly.n + 8 * g;
        float w[8], cs[4], sn[4], sum[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[e] = x.w ? x.w[8 * g + e] : 1.f;
            sum[e] = 0.f;
        }
        pair_angles(a, g, norm_first(a, pl.b) + nn, cs, sn);
#pragma unroll 2
        for (int h = pl.h0; h < pl.h1; ++h) {
            float v[8], dy[8], gr[8];
            load8(src + h * x.lx.h, v);
            load8(grd + h * x.lg.h, dy);
            float s = 0.f, t = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                gr[2 * q] = fmaf(dy[2 * q], cs[q], dy[2 * q + 1] * sn[q]);
                gr[2 * q + 1] = fmaf(dy[2 * q + 1], cs[q], -dy[2 * q] * sn[q]);
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
            if (in) store8(dst + h * x.ly.h, dx);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float add = in ? sum[e] : 0.f;
            dw[0][e] += pl.which ? 0.f : add;
            dw[1][e] += pl.which ? add : 0.f;
        }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) red[threadIdx.x / TPR][8 * g + e] = dw[which][e];
        __syncthreads();
        if (threadIdx.x < D) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < ROWS; ++k) s += red[k][threadIdx.x];
            a.partial[((long long)which * gridDim.x + blockIdx.x) * D + threadIdx.x] = s;
        }
    }
}

// dw[c] = sum over blocks of partial[which][block][c]: 32 channels per block, 32 threads per
// channel each adding every 32nd partial, joined in a fixed order.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(NormArgs a, int blocks, int D)
{
    __shared__ float red[32][33];
    const int which = blockIdx.x / (D / 32), c = (blockIdx.x % (D / 32)) * 32 + threadIdx.x % 32, k = threadIdx.x / 32;
    const float *p = a.partial + (long long)which * blocks * D + c;
    float s = 0.f;
    for (int j = k; j < blocks; j += 32) s += p[(long long)j * D];
    red[k][threadIdx.x % 32] = s;
    __syncthreads();
    s = red[threadIdx.x % 32][k];   // warp k: channel k of the 32
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    float *dw = which ? a.k.dw : a.q.dw;
    if (threadIdx.x % 32 == 0 && dw) dw[(blockIdx.x % (D / 32)) * 32 + k] = s;
}

// Heads per place: all of them when the token runs alone fill the device several times over
// (one evaluation of the angles per token and tensor), fewer otherwise.
void plan(NormArgs &a, int num_sms)
{
    a.tiles = (a.N + kThreads / (a.d / 8) - 1) / (kThreads / (a.d / 8));
    const long long runs = (long long)a.B * a.tiles, want = 16ll * num_sms;
    const int heads = a.H > a.Hkv ? a.H : a.Hkv;
    long long per = (want + runs - 1) / runs;            // places wanted per token run
    long long chunk = (a.H + a.Hkv + per - 1) / per;
    chunk = (chunk + kHeads - 1) / kHeads * kHeads;
    a.chunk = (int)(chunk < heads ? chunk : heads);
    a.chunks_q = (a.H + a.chunk - 1) / a.chunk;
    a.chunks_k = a.k.X ? (a.Hkv + a.chunk - 1) / a.chunk : 0;
}

}  // namespace

cudaError_t qk_norm_forward(const NormArgs &a_in, int num_sms, cudaStream_t s)
{
    NormArgs a = a_in;
    plan(a, num_sms);
    const long long grid = (long long)a.B * a.tiles * (a.chunks_q + a.chunks_k);
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    if (a.is_bf16) {
        if (a.d == 64) qk_norm_kernel<__nv_bfloat16, 64><<<(unsigned)grid, kThreads, 0, s>>>(a);
        else qk_norm_kernel<__nv_bfloat16, 128><<<(unsigned)grid, kThreads, 0, s>>>(a);
    } else {
        if (a.d == 64) qk_norm_kernel<float, 64><<<(unsigned)grid, kThreads, 0, s>>>(a);
        else qk_norm_kernel<float, 128><<<(unsigned)grid, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t qk_norm_backward(const NormArgs &a_in, int num_sms, cudaStream_t s)
{
    NormArgs a = a_in;
    plan(a, num_sms);
    const long long places = (long long)a.B * a.tiles * (a.chunks_q + a.chunks_k);
    const int grid = (int)(places < kNormMaxBlocks ? places : kNormMaxBlocks);
    if (a.is_bf16) {
        if (a.d == 64) qk_norm_bwd_kernel<__nv_bfloat16, 64><<<grid, kThreads, 0, s>>>(a);
        else qk_norm_bwd_kernel<__nv_bfloat16, 128><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (a.d == 64) qk_norm_bwd_kernel<float, 64><<<grid, kThreads, 0, s>>>(a);
        else qk_norm_bwd_kernel<float, 128><<<grid, kThreads, 0, s>>>(a);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    qk_norm_dw_kernel<<<2 * (a.d / 32), 1024, 0, s>>>(a, grid, a.d);
    return cudaGetLastError();
}

}  // namespace scope
