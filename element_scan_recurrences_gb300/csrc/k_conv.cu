// k_conv.cu -- the short causal convolution of every channel, its gradients, and
// its form for one token:
//
//     p[t] = bias + sum_j w[j] x[t - W + 1 + j],   out = p / (1 + e^-p)
//
// Bounded by HBM: 2 W + 4 operations against 4 bytes an element in bf16.  A thread
// takes 16 bytes of channels (8 backwards) through a run of tokens with the last
// W - 1 inputs in registers, so each input is read once but for W - 1 tokens a run;
// a warp's accesses are whole rows of 256 bytes or more.  Tokens come in blocks through
// places of the thread's own in shared memory (cp.async, no barrier), two blocks on
// their way: that many bytes in flight hide HBM's latency, where in registers there
// was room for one block (8 x 2048 x 4096 ragged prompts in bf16 54 us, now 40, 0.94
// of the measured copy rate with the call; the gradient of 4 x 2047 x 4096 77, now 54).  Products and sums are made two channels an
// instruction.  The gradient is one pass over x and the gradient of out the same
// way: p is formed again, and the gradients of the last W tokens' p in registers give
// that of the input W - 1 tokens back.  The weights' sums over a run stay in
// registers and meet in a second launch, always in one order.
#include "es_attn.h"
#include "es_ssm.cuh"
#include "es_ssm.h"

namespace es {
namespace {

constexpr int kThreads = 128;

template <int V>
constexpr int kPairs = (V + 1) / 2;
// tokens a block: at least 4, whole rounds of the W places that the last inputs go around
template <int W>
constexpr int kBlock = W >= 4 ? W : W == 3 ? 6 : 4;

// The input at token t of a row (the carried one before the first, zeros without).
template <typename T, int V, int W>
__device__ __forceinline__ void input_at(const ConvLaunch& L, const T* x, int64_t b, int64_t c, int64_t t, float2 (&r)[kPairs<V>]) {
    if (t >= 0) unpack<T, V>(load_raw<T, V>(x + t * L.x.stride_t), r);
    else if (L.init != nullptr && t >= 1 - W)
        unpack<T, V>(load_raw<T, V>(static_cast<const T*>(L.init) + (b * (W - 1) + t + W - 1) * L.C + c), r);
    else zero(r);
}

// The weights of V channels lie side by side.
template <typename W_, int V, int W>
__device__ __forceinline__ void weights_of(const W_* p, bool wide, float2 (&w)[W][kPairs<V>]) {
    constexpr int N = V * W, S = 16 / sizeof(W_);
    float f[N];
    if (N % S == 0 && wide) {
#pragma unroll
        for (int i = 0; i < N / S; ++i) {
            const Pack<W_, S> q = load_raw<W_, S>(p + i * S);
#pragma unroll
            for (int j = 0; j < S; ++j) f[i * S + j] = to_f32(q.v[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = to_f32(p[i]);
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int i = 0; i < kPairs<V>; ++i)
            w[j][i] = make_float2(f[2 * i * W + j], 2 * i + 1 < V ? f[(2 * i + 1 < V ? 2 * i + 1 : 0) * W + j] : 0.0f);
}
template <int V, int W>
__device__ __forceinline__ void load_weights(const ConvLaunch& L, int64_t c, float2 (&w)[W][kPairs<V>], float2 (&bias)[kPairs<V>]) {
    const bool wide = reinterpret_cast<uintptr_t>(L.w) % 16 == 0;
    if (L.w_bf16) weights_of<__nv_bfloat16, V, W>(static_cast<const __nv_bfloat16*>(L.w) + c * W, wide, w);
    else weights_of<float, V, W>(static_cast<const float*>(L.w) + c * W, wide, w);
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) {
        bias[i] = pair_of(0.f);
        if (L.bias != nullptr) {
            bias[i].x = weight_at(L.bias, L.w_bf16, c + 2 * i);
            if (2 * i + 1 < V) bias[i].y = weight_at(L.bias, L.w_bf16, c + 2 * i + 1);
        }
    }
}

// A thread's blocks of tokens on their way, kAheadBlocks of them
constexpr int kAheadBlocks = 2, kPlaces = kAheadBlocks + 1;

template <bool B>
struct Flag {
    static constexpr bool value = B;
};

struct ConvPlace {
    int64_t b, c, begin;
};
// a thread's batch row, channels and first token; false past the last channel
template <int V>
__device__ __forceinline__ bool conv_place(const ConvLaunch& L, ConvPlace* p) {
    const int64_t across = (L.C / V + kThreads - 1) / kThreads, runs = L.T == 0 ? 1 : (L.T + L.run - 1) / L.run;
    int64_t i = blockIdx.x;
    p->c = (i % across * kThreads + threadIdx.x) * V;
    i /= across;
    p->begin = i % runs * L.run;
    p->b = i / runs;
    return p->c < L.C;
}

// (The launch bounds hold the registers to what keeps 3 blocks of the common widths on
// an SM; 4 spill, 46 -> 52 us for 4 x 2047 x 4096.)
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads, V * W <= 32 ? 3 : 2) k_conv(const __grid_constant__ ConvLaunch L) {
    constexpr int P = kPairs<V>, BLK = kBlock<W>;
    ConvPlace p;
    if (!conv_place<V>(L, &p)) return;
    const int64_t len = live_tokens(L.lengths, p.b, L.T);
    const int64_t stop = p.begin + L.run < L.T ? p.begin + L.run : L.T, end = stop < len ? stop : len;
    const T* const x = static_cast<const T*>(L.x.data) + p.b * L.x.stride_b + p.c;
    T* const out = static_cast<T*>(L.out.data) + p.b * L.out.stride_b + p.c;
    float2 w[W][P], bias[P], row[W][P];              // token t's input at place (t - begin + W - 1) % W of `row`
    using Raw = Pack<T, V>;
    __shared__ Raw ring[kPlaces][BLK][kThreads];
    const int count = end > p.begin ? static_cast<int>(end - p.begin) : 0;
    const T* px = x + p.begin * L.x.stride_t;        // of the next block
    T* po = out + p.begin * L.out.stride_t;
    auto fetch = [&](int left, int place) {
#pragma unroll
        for (int k = 0; k < BLK; ++k)
            if (k < left) copy_async<sizeof(Raw)>(&ring[place][k][threadIdx.x], px + k * L.x.stride_t);
        copies_done();
        px += BLK * L.x.stride_t;
    };
#pragma unroll
    for (int i = 0; i < kAheadBlocks; ++i) fetch(count - i * BLK, i);
    int place = 0;
    if (p.begin < end || p.begin == 0) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) input_at<T, V, W>(L, x, p.b, p.c, p.begin - (W - 1) + j, row[j]);
    }
    if (p.begin == 0 && L.fin != nullptr) {
        // the carried inputs may lie where the last ones go: only this thread reads them, and has by now
        float2 last[W - 1][P];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) input_at<T, V, W>(L, x, p.b, p.c, len - (W - 1) + j, last[j]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            *reinterpret_cast<Pack<T, V>*>(static_cast<T*>(L.fin) + (p.b * (W - 1) + j) * L.C + p.c) = pack<T, V>(last[j]);
    }
    load_weights<V, W>(L, p.c, w, bias);
    // blocks whole and the last: without tests between their tokens they run into one another
    auto block = [&](int left, auto whole) {
        copies_wait<kAheadBlocks - 1>();
        // the place read a block ago takes the block that comes kAheadBlocks after this
        fetch(left - kAheadBlocks * BLK, place == 0 ? kAheadBlocks : place - 1);
        const auto& now = ring[place];
        if (++place == kPlaces) place = 0;
#pragma unroll
        for (int k = 0; k < BLK; ++k) {
            if (!decltype(whole)::value && k >= left) break;
            unpack<T, V>(now[k][threadIdx.x], row[(k + W - 1) % W]);
            float2 o[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                o[i] = bias[i];
#pragma unroll
                for (int j = 0; j < W; ++j) o[i] = pair_fma(w[j][i], row[(k + j) % W][i], o[i]);
            }
            if (L.act) {
#pragma unroll
                for (int i = 0; i < P; ++i) o[i] = pair_mul(o[i], pair_logistic<sizeof(T) == 4>(o[i]));
            }
            *reinterpret_cast<Pack<T, V>*>(po + k * L.out.stride_t) = pack<T, V>(o);
        }
        po += BLK * L.out.stride_t;
    };
    int left = count;
    for (; left >= BLK; left -= BLK) block(left, Flag<true>{});
    if (left > 0) block(left, Flag<false>{});
    float2 none[P];
    zero(none);
    for (int64_t t = end > p.begin ? end : p.begin; t < stop; ++t)
        *reinterpret_cast<Pack<T, V>*>(out + t * L.out.stride_t) = pack<T, V>(none);
}

// Token u gives the gradient gp of its p, and with the W - 1 before it that of the
// input at token u - (W - 1); before the first token those are the carried inputs.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads, V * W <= 16 ? 4 : 2) k_conv_bwd(const __grid_constant__ ConvLaunch L) {
    constexpr int P = kPairs<V>, BLK = kBlock<W>;
    ConvPlace p;
    if (!conv_place<V>(L, &p)) return;
    const int64_t len = live_tokens(L.lengths, p.b, L.T);
    const int64_t stop = p.begin + L.run < L.T ? p.begin + L.run : L.T;
    const T* const x = static_cast<const T*>(L.x.data) + p.b * L.x.stride_b + p.c;
    const T* const g = static_cast<const T*>(L.g.data) + p.b * L.g.stride_b + p.c;
    T* const out = static_cast<T*>(L.out.data) + p.b * L.out.stride_b + p.c;
    float2 w[W][P], bias[P], row[W][P], gp[W][P], gw[W][P], gb[P];      // `row` and `gp` go around as in k_conv
    using Raw = Pack<T, V>;
    __shared__ Raw ring[kPlaces][2][BLK][kThreads];
    // the tokens whose p this run needs: W - 1 past its own
    const int64_t until = stop + W - 1 < len ? stop + W - 1 : len;
    const T *px = x + p.begin * L.x.stride_t, *pg = g + p.begin * L.g.stride_t;      // of the next block
    auto fetch = [&](int left, int place) {
#pragma unroll
        for (int k = 0; k < BLK; ++k)
            if (k < left) {
                copy_async<sizeof(Raw)>(&ring[place][0][k][threadIdx.x], px + k * L.x.stride_t);
                copy_async<sizeof(Raw)>(&ring[place][1][k][threadIdx.x], pg + k * L.g.stride_t);
            }
        copies_done();
        px += BLK * L.x.stride_t;
        pg += BLK * L.g.stride_t;
    };
    // tokens from the run's first: those with p, with p of its own, all that the loop makes
    const int live = until > p.begin ? static_cast<int>(until - p.begin) : 0, own = static_cast<int>(stop - p.begin);
#pragma unroll
    for (int i = 0; i < kAheadBlocks; ++i) fetch(live - i * BLK, i);
    int place = 0;
    load_weights<V, W>(L, p.c, w, bias);
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
    // `inside`: every token of the block, and every input whose gradient it completes, is the
    // run's own and reads no state's gradient
    auto block = [&](int u0, auto inside) {
        constexpr bool kInside = decltype(inside)::value;
        copies_wait<kAheadBlocks - 1>();
        fetch(live - u0 - kAheadBlocks * BLK, place == 0 ? kAheadBlocks : place - 1);
        const auto& now = ring[place];
        if (++place == kPlaces) place = 0;
#pragma unroll
        for (int k = 0; k < BLK; ++k) {
            const int u = u0 + k;
            if (!kInside && u >= own + W - 1) break;
            auto& q = gp[(k + W - 1) % W];
            auto& in = row[(k + W - 1) % W];
            if (kInside || u < live) {
                unpack<T, V>(now[0][k][threadIdx.x], in);
                unpack<T, V>(now[1][k][threadIdx.x], q);
                if (L.act) {
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        float2 s = bias[i];
#pragma unroll
                        for (int m = 0; m < W; ++m) s = pair_fma(w[m][i], row[(k + m) % W][i], s);
                        const float2 l = pair_logistic<sizeof(T) == 4>(s);
                        // l + s l (1 - l)
                        q[i] = pair_mul(q[i], pair_fma(pair_mul(s, l), pair_fma(l, pair_of(-1.f), pair_of(1.f)), l));
                    }
                }
            } else {
                zero(in);
                zero(q);
            }
            if (kInside || u < own) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    gb[i] = pair_add(gb[i], q[i]);
#pragma unroll
                    for (int m = 0; m < W; ++m) gw[m][i] = pair_fma(q[i], row[(k + m) % W][i], gw[m][i]);
                }
            }
            float2 gx[P];
            zero(gx);
            const int64_t t = p.begin + u - (W - 1);
            if (!kInside) {
                const int64_t j = t - len + W - 1;       // the input's place in the state after
                if (j >= 0 && j < W - 1 && L.gfin != nullptr && (u >= W - 1 || p.begin == 0))
                    unpack<T, V>(load_raw<T, V>(static_cast<const T*>(L.gfin) + (p.b * (W - 1) + j) * L.C + p.c), gx);
            }
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int m = 0; m < W; ++m) gx[i] = pair_fma(w[W - 1 - m][i], gp[(k + m) % W][i], gx[i]);
            if (kInside || u >= W - 1) *reinterpret_cast<Pack<T, V>*>(out + t * L.out.stride_t) = pack<T, V>(gx);
            else if (t < 0 && L.fin != nullptr)
                *reinterpret_cast<Pack<T, V>*>(static_cast<T*>(L.fin) + (p.b * (W - 1) + u) * L.C + p.c) = pack<T, V>(gx);
        }
    };
    // inputs from len - (W - 1) on take the state's gradient
    const int whole = static_cast<int>(len - p.begin < own ? (len > p.begin ? len - p.begin : 0) : own);
    for (int u0 = 0; u0 < own + W - 1; u0 += BLK) {
        if (u0 >= W - 1 && u0 + BLK <= whole) block(u0, Flag<true>{});
        else block(u0, Flag<false>{});
    }
    if (L.partial == nullptr) return;
    const int64_t runs = L.T == 0 ? 1 : (L.T + L.run - 1) / L.run;
    float* const q = L.partial + (p.b * runs + p.begin / L.run) * (W + 1) * L.C + p.c;
#pragma unroll
    for (int j = 0; j < W; ++j) *reinterpret_cast<Pack<float, V>*>(q + j * L.C) = pack<float, V>(gw[j]);
    *reinterpret_cast<Pack<float, V>*>(q + W * L.C) = pack<float, V>(gb);
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) k_conv_step(const __grid_constant__ ConvLaunch L) {
    constexpr int P = kPairs<V>;
    const int64_t across = (L.C / V + kThreads - 1) / kThreads, b = blockIdx.x / across;
    const int64_t c = (blockIdx.x % across * kThreads + threadIdx.x) * V;
    if (c >= L.C) return;
    float2 w[W][P], bias[P], x[P], o[P];
    Pack<T, V> row[W];
    const T* const from = static_cast<const T*>(L.init) + b * (W - 1) * L.C + c;
    T* const to = static_cast<T*>(L.fin) + b * (W - 1) * L.C + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row[j] = load_raw<T, V>(from + j * L.C);
    row[W - 1] = load_raw<T, V>(static_cast<const T*>(L.x.data) + b * L.x.stride_b + c);
    load_weights<V, W>(L, c, w, bias);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) *reinterpret_cast<Pack<T, V>*>(to + j * L.C) = row[j + 1];
#pragma unroll
    for (int i = 0; i < P; ++i) o[i] = bias[i];
#pragma unroll
    for (int j = 0; j < W; ++j) {
        unpack<T, V>(row[j], x);
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = pair_fma(w[j][i], x[i], o[i]);
    }
    if (L.act) {
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = pair_mul(o[i], pair_logistic<sizeof(T) == 4>(o[i]));
    }
    *reinterpret_cast<Pack<T, V>*>(static_cast<T*>(L.out.data) + b * L.out.stride_b + c) = pack<T, V>(o);
}

enum Kind { kForward, kBackward, kStep };

template <typename T, int V, int W, Kind KIND>
cudaError_t go(const ConvLaunch& L) {
    const int64_t across = (L.C / V + kThreads - 1) / kThreads, runs = KIND == kStep || L.T == 0 ? 1 : (L.T + L.run - 1) / L.run;
    const unsigned grid = static_cast<unsigned>(across * runs * L.B);
    if constexpr (KIND == kForward) k_conv<T, V, W><<<grid, kThreads, 0, L.stream>>>(L);
    else if constexpr (KIND == kBackward) k_conv_bwd<T, V, W><<<grid, kThreads, 0, L.stream>>>(L);
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

// channels a thread
int width_of(const ConvLaunch& L, bool backward) {
    const int unit = backward ? 8 : 16;              // bytes
    return in_units(L, unit) ? unit / (L.bf16 ? 2 : 4) : 1;
}

template <Kind KIND>
cudaError_t by_type(const ConvLaunch& L) {
    const int V = width_of(L, KIND == kBackward);
    if (L.bf16) {
        if (V == 1) return by_taps<__nv_bfloat16, 1, KIND>(L);
        return by_taps<__nv_bfloat16, KIND == kBackward ? 4 : 8, KIND>(L);
    }
    return V == 1 ? by_taps<float, 1, KIND>(L) : by_taps<float, KIND == kBackward ? 2 : 4, KIND>(L);
}

// Tokens a run: long ones read fewer inputs twice and leave fewer partial sums,
// short ones fill the GPU (1024 threads an SM) when there are few rows and channels.
int run_of(const ConvLaunch& L, bool backward) {
    int run = backward ? 128 : 64;
    const int64_t across = L.C / width_of(L, backward);
    while (run > 8 && L.B * across * ((L.T + run - 1) / run) < static_cast<int64_t>(kSms) * 1024) run /= 2;
    return run;
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

int64_t conv_backward_rows(const ConvLaunch& L) {
    const int run = run_of(L, true);
    return L.B * (L.T == 0 ? 1 : (L.T + run - 1) / run);
}

cudaError_t launch_conv(ConvLaunch L, int* kernels) {
    *kernels = 1;
    L.run = run_of(L, false);
    return by_type<kForward>(L);
}

cudaError_t launch_conv_backward(ConvLaunch L, int* kernels) {
    *kernels = 1;
    L.run = run_of(L, true);
    const cudaError_t e = by_type<kBackward>(L);
    if (e != cudaSuccess || L.partial == nullptr) return e;
    ++*kernels;
    return sum_rows(L.partial, conv_backward_rows(L), (L.taps + 1) * L.C, PutConv{L.gw, L.gb, L.C, L.taps, L.w_bf16}, L.stream);
}

cudaError_t launch_conv_step(const ConvLaunch& L) { return by_type<kStep>(L); }

}  // namespace es
