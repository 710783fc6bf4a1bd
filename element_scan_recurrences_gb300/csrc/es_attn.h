// es_attn.h -- launch descriptions of linear attention and of the query/key
// norm with rotation, shared by the entry points (es_attn_api.cu) and the
// kernels (k_attn_*.cu, k_rotate.cu).  Not part of the ABI.
#pragma once

#include <cuda_bf16.h>

#include "es_internal.h"

namespace es {

// GB300's SMs.  Workspaces and grids are counted by this number and not by the
// device's, for a workspace may be asked for where there is no GPU.
constexpr int kSms = 152;

// [B, T, heads, dim] operand, innermost stride 1 (strides in elements); head h
// of the call reads operand head h / div.
struct AttnOperand {
    const void* p;
    int64_t sb, st, sh;
    int div;
};

// One run of the recurrence over the sequences of a call:
//
//     state[t] = e^{g[t]} state[t-1] + u y[t] z[t]^T,   out[t] = r x[t] state[t]
//
// or, reversed, from the last token to the first,
//
//     state[t] = e^{g[t+1]} state[t+1] + u y[t] z[t]^T, out[t] = r x[t] state[t]
//
// with a state of dx x dz values.  u and r are update_scale and read_scale, one
// of them the call's scale (out_scale, their product) and the other one: the
// states are then the ones that the call takes and gives, at any scale.
// The forward pass is one run (x, y, z) = (q, k, v); the gradients are three
// more over the same data:
//     grad_q  forward  (grad_out, v, k),  the state transposed
//     grad_v  reversed (k, q, grad_out)
//     grad_k  reversed (v, grad_out, q),  the state transposed
struct AttnRun {
    AttnOperand x, y, z;
    void* out;                   // [B, T, H, dz] by strides, bf16 or f32
    int64_t ob, ot, oh;
    int out_f32;                 // out is f32 whatever the operands' type
    const float* init;           // value (a, c) of the state of (b, h) at [(b*H + h)*dx*dz + a*sa + c*sc], or null (zero)
    float* fin;                  // state after the last trip, the same layout, or null
    int64_t sa, sc;
    float update_scale, read_scale, out_scale;
    int reverse;
    int state_result;            // the run's last state can be asked for (its results do not depend on whether it is)
    // For the decays' gradient: out[t] (unrounded) . w[t], per slice of dz
    // columns, [slices, B*H, T]; null: not wanted.
    AttnOperand w;
    float* dots;
    // The run's state at the end of every anchor block (kAttnAnchorTokens) and
    // of the row: a forward run's after the block, a reversed run's before it;
    // value (a, c) at anchors[((b*H + h)*n + m)*dx*dz + a*dz + c].
    float* anchors;
    int dx, dz;
};

struct AttnLaunch {
    AttnRun run[3];
    int runs;
    int bf16;
    int64_t B, T;
    int H;
    const float* g;              // log decays, strides in elements; null: none
    int64_t gb, gt, gh;
    const int* lengths;          // [B] or null
    int64_t n_anchors;           // per (b, h)
    // segments of tokens: each a CTA's, with a pass before for the states between them
    int64_t seg_chunks;          // chunks a segment
    int n_segs;
    float* seg_states;
    float* seg_decays;
    unsigned int* status;
    uint64_t wait_ns;
    int64_t drop_tile;
    cudaStream_t stream;
    EncodeTiledFn encode;
};

// chunk of tokens and slice of value columns of the direct kernel
constexpr int kAttnChunk = 32;
constexpr int kAttnSlice = 32;
constexpr int kAttnMaxDim = 256;

cudaError_t launch_attn_direct(const AttnLaunch& L, int* kernels);

// Tokens between the states the decays' gradient starts from: its sums of
// differences run within such a block (see k_attn_decay_grad).
constexpr int kAttnAnchorTokens = 256;

// the tensor-core kernel: chunk of tokens, and whether it can load an operand
constexpr int kAttnTcChunk = 64;
bool attn_tc_operand_ok(const AttnOperand& o, int heads, int d, int64_t T, int64_t B);
cudaError_t launch_attn_tc(const AttnLaunch& L, int* kernels, const char** err);

// The states between segments from each segment's own (launch_attn_join).
struct AttnJoin {
    int reverse[3], init[3];     // of each run: direction, and whether a first state came
    int64_t size, T, BH;
    int H, chunk, n_segs;
    int64_t seg_chunks;
    const int* lengths;
    float* states;               // [runs][BH][n_segs][size]
    const float* decays;         // [runs][BH][n_segs]
};
cudaError_t launch_attn_join(const AttnLaunch& L, int chunk);

// The decays' gradient from the two runs' dots and states: for each token t of
// anchor block m, sum over s >= t of the block of (dq[s] - dk[s]) + e[m], with
// e[m] = <state_q, state_k> at the block's end, corrected in proportion so that
// it meets e[m - 1] at the block's start.
struct AttnDecayGrad {
    const float* dots_q;         // [slices, B*H, T]
    const float* dots_k;
    const float* states_q;       // [B*H, n, size]
    const float* states_k;
    const float* initial;        // [B*H, size]: the first state and its gradient, or null
    const float* grad_initial;
    float* ends;                 // [B*H, n + 1]: e[-1], e[0], ..
    int slices;
    int64_t size;
    int64_t B, T;
    int H;
    const int* lengths;
    int64_t n;                   // anchor blocks per (b, h)
    float* grad;                 // [B, T, H], or null
    float* partial;              // per head: [H, B*n] block sums, then summed to `grad_h`
    float* grad_h;               // [H], or null
    cudaStream_t stream;
};
cudaError_t launch_attn_decay_grad(const AttnDecayGrad& G, int* kernels);

// grads of operand heads read by several heads: out[b,t,j,:] = sum of part[b,t,j*div+r,:] over r
struct AttnFold {
    const float* part;           // [B, T, H, d] dense
    void* out;
    int64_t ob, ot, oh;
    int bf16;
    int64_t B, T;
    int heads, div, d;
    cudaStream_t stream;
};
cudaError_t launch_attn_folds(const AttnFold* folds, int n);      // one launch for all

struct AttnStep {
    AttnOperand q, k, v;         // st unused
    void* out;                   // [B, H, dv] by strides
    int64_t ob, oh;
    int bf16;
    const float* g;
    int64_t gb, gh;
    const float* state;          // [B, H, dk, dv] dense
    float* state_out;
    float scale;
    int64_t B;
    int H, dk, dv;
    cudaStream_t stream;
};
cudaError_t launch_attn_step(const AttnStep& S);

// ---------------------------------------------------------------------------
// norm of queries and keys with the position rotation

struct RotateSide {
    const void* x;               // [B, T, heads, d]
    int64_t xb, xt, xh;
    const void* g;               // gradient of the output (backward)
    int64_t gb, gt, gh;
    void* out;                   // forward: the output; backward: the gradient of x
    int64_t ob, ot, oh;
    const void* w;               // [d] or null
    void* gw;                    // backward: gradient of w, or null
    int heads;
};

struct RotateLaunch {
    RotateSide side[2];          // queries, keys
    int bf16, w_bf16;
    int64_t B, T;
    int d, turned, neighbours;
    float eps;
    const float* cos;
    const float* sin;            // [rows, turned / 2]
    int64_t rows;
    const void* positions;       // [B, T] by strides, or null (0, 1, ...)
    int pos64;
    int64_t pb, pt;
    float* partial;              // backward: [blocks, d] partial sums of both weights' gradients
    int backward;
    cudaStream_t stream;
};
int rotate_blocks(const RotateLaunch& L, int side);
int64_t rotate_units(const RotateLaunch& L, int side);     // below 2^31 - 2^20: the kernel counts them in 32 bits
cudaError_t launch_rotate(const RotateLaunch& L, int* kernels);

}  // namespace es
