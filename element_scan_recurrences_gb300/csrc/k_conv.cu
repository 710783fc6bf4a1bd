// k_conv.cu -- the short causal convolution of every channel, its gradients, and
// its form for one token:
//
//     p[t] = bias + sum_j w[j] x[t - W + 1 + j],   out = p / (1 + e^-p)
//
// Bounded by HBM: 2 W + 4 operations against 4 bytes an element in bf16.  A thread
// takes 16 bytes of channels through a run of tokens with the last W - 1 inputs in
// registers, so each input is read once but for W - 1 tokens a run; a warp's
// accesses are whole 512-byte rows, and the unrolled loop keeps several in flight.
// The gradient is one pass over x and the gradient of out the same way: p is formed
// again, and the gradients of the last W tokens' p in registers give that of the
// input W - 1 tokens back.  The weights' sums over a run stay in registers and meet
// in a second launch, always in one order.
#include "es_attn.h"
#include "es_ssm.cuh"
#include "es_ssm.h"

namespace es {
namespace {

constexpr int kThreads = 128;
constexpr int kRun = 32;            // tokens a thread, forwards
constexpr int kRunBack = 64;        // and backwards: fewer partial sums of the weights

// The input at token t of a row (the carried one before the first, zeros without).
template <typename T, int V, int W>
__device__ __forceinline__ void input_at(const ConvLaunch& L, const T* x, int64_t b, int64_t c, int64_t t, float (&r)[V]) {
    if (t >= 0) load_pack<T, V>(x + t * L.x.stride_t, r);
    else if (L.init != nullptr && t >= 1 - W) load_pack<T, V>(static_cast<const T*>(L.init) + (b * (W - 1) + t + W - 1) * L.C + c, r);
    else zero(r);
}

template <typename T, int V, int W>
__device__ __forceinline__ void load_weights(const ConvLaunch& L, int64_t c, float (&w)[W][V], float (&bias)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][i] = weight_at(L.w, L.w_bf16, (c + i) * W + j);
        bias[i] = L.bias != nullptr ? weight_at(L.bias, L.w_bf16, c + i) : 0.0f;
    }
}

struct ConvPlace {
    int64_t b, c, begin;
};
// a thread's batch row, channels and first token; false past the last channel
template <int V, int RUN>
__device__ __forceinline__ bool conv_place(const ConvLaunch& L, ConvPlace* p) {
    const int64_t across = (L.C / V + kThreads - 1) / kThreads, runs = L.T == 0 ? 1 : (L.T + RUN - 1) / RUN;
    int64_t i = blockIdx.x;
    p->c = (i % across * kThreads + threadIdx.x) * V;
    i /= across;
    p->begin = i % runs * RUN;
    p->b = i / runs;
    return p->c < L.C;
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) k_conv(const __grid_constant__ ConvLaunch L) {
    ConvPlace p;
    if (!conv_place<V, kRun>(L, &p)) return;
    const int64_t len = live_tokens(L.lengths, p.b, L.T);
    const int64_t stop = p.begin + kRun < L.T ? p.begin + kRun : L.T, end = stop < len ? stop : len;
    const T* const x = static_cast<const T*>(L.x.data) + p.b * L.x.stride_b + p.c;
    T* const out = static_cast<T*>(L.out.data) + p.b * L.out.stride_b + p.c;
    float w[W][V], bias[V], row[W][V];
    if (p.begin < end || p.begin == 0) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) input_at<T, V, W>(L, x, p.b, p.c, p.begin - (W - 1) + j, row[j]);
    }
    if (p.begin == 0 && L.fin != nullptr) {
        // the carried inputs may lie where the last ones go: only this thread reads them, and has by now
        float last[W - 1][V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) input_at<T, V, W>(L, x, p.b, p.c, len - (W - 1) + j, last[j]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) store_pack<T, V>(static_cast<T*>(L.fin) + (p.b * (W - 1) + j) * L.C + p.c, last[j]);
    }
    load_weights<T, V, W>(L, p.c, w, bias);
#pragma unroll 4
    for (int64_t t = p.begin; t < end; ++t) {
        load_pack<T, V>(x + t * L.x.stride_t, row[W - 1]);
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float s = bias[i];
#pragma unroll
            for (int j = 0; j < W; ++j) s = fmaf(w[j][i], row[j][i], s);
            o[i] = L.act ? s * logistic(s) : s;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) row[j][i] = row[j + 1][i];
        }
        store_pack<T, V>(out + t * L.out.stride_t, o);
    }
    float none[V];
    zero(none);
    for (int64_t t = end > p.begin ? end : p.begin; t < stop; ++t) store_pack<T, V>(out + t * L.out.stride_t, none);
}

// Token u gives the gradient gp of its p, and with the W - 1 before it that of the
// input at token u - (W - 1); before the first token those are the carried inputs.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) k_conv_bwd(const __grid_constant__ ConvLaunch L) {
    ConvPlace p;
    if (!conv_place<V, kRunBack>(L, &p)) return;
    const int64_t len = live_tokens(L.lengths, p.b, L.T);
    const int64_t stop = p.begin + kRunBack < L.T ? p.begin + kRunBack : L.T;
    const T* const x = static_cast<const T*>(L.x.data) + p.b * L.x.stride_b + p.c;
    const T* const g = static_cast<const T*>(L.g.data) + p.b * L.g.stride_b + p.c;
    T* const out = static_cast<T*>(L.out.data) + p.b * L.out.stride_b + p.c;
    float w[W][V], bias[V], row[W][V], gp[W][V], gw[W][V], gb[V];
    load_weights<T, V, W>(L, p.c, w, bias);
    zero(gb);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        zero(gw[j]);
        zero(gp[j]);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        if (p.begin - (W - 1) + j < len) input_at<T, V, W>(L, x, p.b, p.c, p.begin - (W - 1) + j, row[j]);
        else zero(row[j]);
    }
#pragma unroll 2
    for (int64_t u = p.begin; u < stop + W - 1; ++u) {
        const bool live = u < len;
        float go[V];
        if (live) {
            load_pack<T, V>(x + u * L.x.stride_t, row[W - 1]);
            load_pack<T, V>(g + u * L.g.stride_t, go);
        } else {
            zero(row[W - 1]);
            zero(go);
        }
        const int64_t t = u - (W - 1), j = t - len + W - 1;      // the input, its place in the state after
        float gx[V];
        zero(gx);
        if (j >= 0 && j < W - 1 && L.gfin != nullptr && (t >= p.begin || p.begin == 0))
            load_pack<T, V>(static_cast<const T*>(L.gfin) + (p.b * (W - 1) + j) * L.C + p.c, gx);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float q = go[i];
            if (L.act) {
                float s = bias[i];
#pragma unroll
                for (int m = 0; m < W; ++m) s = fmaf(w[m][i], row[m][i], s);
                q *= silu_slope(s, logistic(s));
            }
            gp[W - 1][i] = q;
            if (u < stop) {
                gb[i] += q;
#pragma unroll
                for (int m = 0; m < W; ++m) gw[m][i] = fmaf(q, row[m][i], gw[m][i]);
            }
#pragma unroll
            for (int m = 0; m < W; ++m) gx[i] = fmaf(w[W - 1 - m][i], gp[m][i], gx[i]);
#pragma unroll
            for (int m = 0; m < W - 1; ++m) {
                gp[m][i] = gp[m + 1][i];
                row[m][i] = row[m + 1][i];
            }
        }
        if (t >= p.begin) store_pack<T, V>(out + t * L.out.stride_t, gx);
        else if (t < 0 && L.fin != nullptr) store_pack<T, V>(static_cast<T*>(L.fin) + (p.b * (W - 1) + u) * L.C + p.c, gx);
    }
    if (L.partial == nullptr) return;
    const int64_t runs = L.T == 0 ? 1 : (L.T + kRunBack - 1) / kRunBack;
    float* const q = L.partial + (p.b * runs + p.begin / kRunBack) * (W + 1) * L.C + p.c;
#pragma unroll
    for (int j = 0; j < W; ++j) store_pack<float, V>(q + j * L.C, gw[j]);
    store_pack<float, V>(q + W * L.C, gb);
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) k_conv_step(const __grid_constant__ ConvLaunch L) {
    const int64_t across = (L.C / V + kThreads - 1) / kThreads, b = blockIdx.x / across;
    const int64_t c = (blockIdx.x % across * kThreads + threadIdx.x) * V;
    if (c >= L.C) return;
    float w[W][V], bias[V], row[W][V], o[V];
    const T* const from = static_cast<const T*>(L.init) + b * (W - 1) * L.C + c;
    T* const to = static_cast<T*>(L.fin) + b * (W - 1) * L.C + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_pack<T, V>(from + j * L.C, row[j]);
    load_pack<T, V>(static_cast<const T*>(L.x.data) + b * L.x.stride_b + c, row[W - 1]);
    load_weights<T, V, W>(L, c, w, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float s = bias[i];
#pragma unroll
        for (int j = 0; j < W; ++j) s = fmaf(w[j][i], row[j][i], s);
        o[i] = L.act ? s * logistic(s) : s;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_pack<T, V>(to + j * L.C, row[j + 1]);
    store_pack<T, V>(static_cast<T*>(L.out.data) + b * L.out.stride_b + c, o);
}

enum Kind { kForward, kBackward, kStep };

template <typename T, int V, int W, Kind KIND>
cudaError_t go(const ConvLaunch& L) {
    const int64_t across = (L.C / V + kThreads - 1) / kThreads, run = KIND == kBackward ? kRunBack : kRun;
    const int64_t runs = KIND == kStep || L.T == 0 ? 1 : (L.T + run - 1) / run;
    const unsigned grid = static_cast<unsigned>(across * runs * L.B);
    if (KIND == kForward) k_conv<T, V, W><<<grid, kThreads, 0, L.stream>>>(L);
    else if (KIND == kBackward) k_conv_bwd<T, V, W><<<grid, kThreads, 0, L.stream>>>(L);
    else k_conv_step<T, V, W><<<grid, kThreads, 0, L.stream>>>(L);
    return cudaGetLastError();
}

template <typename T, int V, Kind KIND>
cudaError_t by_taps(const ConvLaunch& L) {
    switch (L.taps) {
        case 2: return go<T, V, 2, KIND>(L);
        case 3: return go<T, V, 3, KIND>(L);
        case 4: return go<T, V, 4, KIND>(L);
        case 5: return go<T, V, 5, KIND>(L);
        case 6: return go<T, V, 6, KIND>(L);
        case 7: return go<T, V, 7, KIND>(L);
        default: return go<T, V, 8, KIND>(L);
    }
}

// `unit`-byte accesses: addresses, strides and channels in them
bool in_units(const ConvLaunch& L, int unit) {
    const int64_t V = unit / (L.bf16 ? 2 : 4);
    if (L.C % V != 0) return false;
    for (const es_rows* r : {&L.x, &L.out, &L.g})
        if (r->data != nullptr && (reinterpret_cast<uintptr_t>(r->data) % unit != 0 || (L.B > 1 && r->stride_b % V != 0) ||
                                   (L.T > 1 && r->stride_t % V != 0)))
            return false;
    for (const void* s : {L.init, static_cast<const void*>(L.fin), L.gfin})
        if (reinterpret_cast<uintptr_t>(s) % unit != 0) return false;
    return true;
}

template <Kind KIND>
cudaError_t by_type(const ConvLaunch& L) {
    const bool vec = in_units(L, 16);
    if (L.bf16) return vec ? by_taps<__nv_bfloat16, 8, KIND>(L) : by_taps<__nv_bfloat16, 1, KIND>(L);
    return vec ? by_taps<float, 4, KIND>(L) : by_taps<float, 1, KIND>(L);
}

// a column of the partial sums: tap (or bias) j of channel c
struct PutConv {
    void *gw, *gb;
    int64_t C;
    int taps, bf16;
    __device__ __forceinline__ void operator()(int64_t i, float s) const {
        const int64_t j = i / C, c = i % C;
        if (j < taps) put_weight(gw, bf16, c * taps + j, s);
        else put_weight(gb, bf16, c, s);
    }
};

}  // namespace

int64_t conv_backward_rows(const ConvLaunch& L) { return L.B * (L.T == 0 ? 1 : (L.T + kRunBack - 1) / kRunBack); }

cudaError_t launch_conv(const ConvLaunch& L, int* kernels) {
    *kernels = 1;
    return by_type<kForward>(L);
}

cudaError_t launch_conv_backward(const ConvLaunch& L, int* kernels) {
    *kernels = 1;
    const cudaError_t e = by_type<kBackward>(L);
    if (e != cudaSuccess || L.partial == nullptr) return e;
    ++*kernels;
    return sum_rows(L.partial, conv_backward_rows(L), (L.taps + 1) * L.C, PutConv{L.gw, L.gb, L.C, L.taps, L.w_bf16}, L.stream);
}

cudaError_t launch_conv_step(const ConvLaunch& L) { return by_type<kStep>(L); }

}  // namespace es
