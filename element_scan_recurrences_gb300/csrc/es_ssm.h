// es_ssm.h -- launches of the state-space layer's kernels: the short causal
// convolution (k_conv.cu), the selective scan (k_sscan.cu, k_sscan_bwd.cu) and
// the group norm with a gate (k_group_norm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "es.h"

namespace es {

constexpr int kMaxTaps = 8;
constexpr int kMaxStates = 64;
constexpr int kMaxNormDim = 8192;

// ---------------------------------------------------------------------------
// convolution

struct ConvLaunch {
    int bf16, w_bf16, taps, act;
    int run;                    // tokens a thread takes (the launch sets it)
    int64_t B, T, C;
    es_rows x, out;             // backward: out is grad_x
    const void *w, *bias;
    const int32_t* lengths;
    const void* init;
    void* fin;                  // backward: grad_initial_state
    // backward
    es_rows g;                  // grad_out
    const void* gfin;
    void *gw, *gb;
    float* partial;             // [blocks over batch and tokens][taps + 1][C]
    cudaStream_t stream;
};

// blocks over batch and tokens of a backward call (each keeps a row of `partial`)
int64_t conv_backward_rows(const ConvLaunch& L);
cudaError_t launch_conv(ConvLaunch L, int* kernels);
cudaError_t launch_conv_backward(ConvLaunch L, int* kernels);
cudaError_t launch_conv_step(const ConvLaunch& L);

// ---------------------------------------------------------------------------
// selective scan

// Tokens between two kept states, and of one tile of the kernels' loads.
constexpr int kScanChunk = 16;

struct ScanLaunch {
    int bf16, softplus;
    int64_t B, T, C;
    int N, G;
    int wide;                   // states in 16-byte pieces: N a multiple of 4, addresses of 16
    es_rows x, delta, gate, out;
    es_heads b, c;
    const float *a, *skip, *bias;
    const int32_t* lengths;
    const float* init;
    float* fin;
    float* kept;                // [B][chunks][C][N]: the state before each chunk (null: not kept)
    int64_t chunks;             // ceil(T / kScanChunk)
    // segments: `segs` of `seg_chunks` chunks; the state a segment makes of its own tokens and the sum of its steps
    int segs;
    int64_t seg_chunks;
    float *seg_state, *seg_sum; // [segs][B][C][N] ([0] counts from init), [segs][B][C]
    float* first;               // [B][C][N]: a copy of init that outlives it (null: init does)
    cudaStream_t stream;
};

struct ScanBackward {
    ScanLaunch f;               // out unused; kept set
    es_rows g, gx, gdelta, ggate;
    es_heads gb, gc;
    float *ga, *gskip, *gbias;
    const float* gfin;
    float* ginit;
    float *part_bc;             // [channel blocks][B][T][2][N]
    float *part_c;              // [segs * B][C][N + 2]: of a, skip, bias
};

// channels a CTA takes, forwards and backwards, and CTAs over the channels of a group
inline int scan_channels(int N) { return N <= 8 ? 64 : N <= 16 ? 32 : N <= 32 ? 16 : 8; }
inline int scan_bwd_channels(int N) { return 4 * scan_channels(N); }
inline int64_t scan_blocks(int64_t C, int G, int channels) { return (C / G + channels - 1) / channels; }
// `keep_only`: nothing but the kept states is computed
cudaError_t launch_scan(const ScanLaunch& L, bool keep_only, int* kernels);
// gradients that the segments' own tokens leave (seg_state, seg_sum, from the second segment on)
cudaError_t launch_scan_own_grads(const ScanBackward& L);
cudaError_t launch_scan_backward(const ScanBackward& L, int* kernels);
// gB and gC from the channel blocks' parts (without channels zeros); B, T > 0
cudaError_t launch_scan_sum_bc(const ScanBackward& L);
cudaError_t launch_scan_step(const ScanLaunch& L);

// ---------------------------------------------------------------------------
// group norm

struct NormLaunch {
    int bf16, w_bf16, center, first, act;
    int64_t B, T;
    int H, D;
    float eps;
    es_heads x, gate, out;      // backward: out is grad_x
    const void *w, *bias;
    // backward
    es_heads g, ggate;
    void *gw, *gb;
    float* partial;             // [norm_rows][2][H * D]
    cudaStream_t stream;
};

int64_t norm_backward_rows(const NormLaunch& L);
cudaError_t launch_norm(const NormLaunch& L, bool backward, int* kernels);

}  // namespace es
