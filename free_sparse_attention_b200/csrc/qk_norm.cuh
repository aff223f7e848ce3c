// Query/key norm with 3D RoPE: arguments shared by the kernels and the C ABI.
#pragma once

#include "window.cuh"

namespace scope {

struct NormTensor {
    const void *X, *G;   // input; gradient of the output (backward)
    void *Y;             // output; gradient of the input (backward)
    const float *w;      // [d] or NULL (ones)
    float *dw;           // [d] or NULL (backward)
    WinLayout lx, lg, ly;
};

struct NormArgs {
    NormTensor q, k;     // k.X NULL: queries only
    int B, H, Hkv, N, d, dt, dh, Hg, Wg, is_bf16;
    const int32_t *first;   // [B] or NULL: position of each entry's first token
    int first0;
    float eps;
    double freq[64];     // turns per position of channel pair i
    float *partial;      // [blocks, d] weight-gradient partials (backward)
    int32_t *status;     // cleared by the backward kernel
    int tiles, chunk, chunks_q, chunks_k, blocks_q;   // filled by the launchers
};

constexpr int kNormMaxBlocks = 148 * 4;   // most blocks of the backward pass (partials in the workspace)

__device__ __forceinline__ int norm_first(const NormArgs &a, int b)
{
    const int f = a.first ? a.first[b] : a.first0;
    return min(max(f, 0), 1 << 30);
}

cudaError_t qk_norm_forward(const NormArgs &a, int num_sms, cudaStream_t s);
cudaError_t qk_norm_backward(const NormArgs &a, int num_sms, cudaStream_t s);

}  // namespace scope
