// k_sscan.cu -- the selective scan over whole sequences and for one token:
//
//     h[n] = e^(d A[n]) h[n] + d x B[n],   y = sum_n C[n] h[n] + D x
//
// for every (batch row, channel), d = log(1 + e^(delta + bias)).
//
// Each token, channel and state costs one exponential (32 a clock an SM) and
// four products or sums (128 a clock), against 1/2 byte of traffic at 16 states
// in bf16: the exponentials bound it, not HBM.  So a thread owns one channel and
// up to 16 states in registers (more states: 2 or 4 lanes a channel): what is
// made once a token and channel (d, the gate) is made by one thread, the sum over
// states needs no exchange, and B and C are one broadcast read for the warp.
// Tokens come in tiles of kScanChunk through two stages of shared memory
// (cp.async; B and C widened to f32 on the way).
//
// A channel's tokens are a chain, so few channels leave the GPU idle: then the
// tokens are cut into segments, a first pass finds the state each segment makes
// of its own tokens, and the main pass enters each segment with
// h = e^(A sum d) h + own over the segments before it.
#include "es_attn.h"
#include "es_sscan.cuh"

namespace es {
namespace {

constexpr int kThreads = kScanThreads;
constexpr int K = kScanChunk;

enum Mode { kMain, kOwnState, kOwnGrad };

template <typename T, int LANES, int RN>
struct Tile {
    static constexpr int CB = kThreads / LANES;      // channels a CTA
    static constexpr int NP = LANES * RN;            // states, padded
    T x[K][CB], delta[K][CB], gate[K][CB];
    float b[K][NP], c[K][NP];
};

template <typename T, int LANES, int RN, bool VEC, Mode MODE>
__global__ void __launch_bounds__(kThreads) k_sscan(const __grid_constant__ ScanArgs A) {
    using Buf = Tile<T, LANES, RN>;
    constexpr int CB = Buf::CB, NP = Buf::NP, P = RN / 2;
    extern __shared__ __align__(128) unsigned char smem[];
    Buf* const buf = reinterpret_cast<Buf*>(smem);
    const ScanLaunch& L = A.L;
    Place p = place_of<CB>(A);
    if constexpr (MODE == kOwnGrad) p.seg += 1;      // the first segment's gradient enters none
    const int sub = threadIdx.x % LANES, ch = threadIdx.x / LANES, n0 = sub * RN;
    const int64_t c = p.first + ch;
    const bool mine = c < p.last, wide = L.wide;
    const int64_t len = live_tokens(L.lengths, p.b, L.T);
    const int64_t begin = p.seg * L.seg_chunks * K;
    const int64_t stop = begin + L.seg_chunks * K < L.T ? begin + L.seg_chunks * K : L.T;
    const int64_t end = stop < len ? stop : len;
    const int tiles = end > begin ? static_cast<int>((end - begin + K - 1) / K) : 0;

    float2 h[P], a2[P];
    float skip = 0.0f, bias = 0.0f, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) h[i] = a2[i] = make_float2(0.f, 0.f);
    const int64_t row = (p.b * L.C + c) * L.N;       // of a [B, C, N] tensor
    const int64_t seg_row = L.B * L.C * L.N;
    if (mine) {
        load_states<RN>(L.a + c * L.N, n0, L.N, wide, a2);
#pragma unroll
        for (int i = 0; i < P; ++i) a2[i] = pair_mul(a2[i], make_float2(kLog2e, kLog2e));
        if (L.skip != nullptr) skip = L.skip[c];
        if (L.bias != nullptr) bias = L.bias[c];
        if constexpr (MODE == kOwnGrad) {
            if (p.seg == L.segs - 1 && A.gfin != nullptr) load_states<RN>(A.gfin + row, n0, L.N, wide, h);
        } else if (p.seg == 0) {
            const float* from = MODE == kMain && L.first != nullptr ? L.first : L.init;
            if (from != nullptr) load_states<RN>(from + row, n0, L.N, wide, h);
            if (MODE == kOwnState && L.first != nullptr) store_states<RN>(L.first + row, n0, L.N, wide, h);
        } else if constexpr (MODE == kMain) {
            load_states<RN>(L.seg_state + row, n0, L.N, wide, h);
            for (int s = 1; s < p.seg; ++s) {
                const float d = L.seg_sum[(s * L.B + p.b) * L.C + c];
                float2 own[P];
                load_states<RN>(L.seg_state + s * seg_row + row, n0, L.N, wide, own);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float2 q = pair_mul(make_float2(d, d), a2[i]);
                    h[i] = pair_fma(make_float2(exp2_hw(q.x), exp2_hw(q.y)), h[i], own[i]);
                }
            }
        }
    }

    constexpr bool kReads = MODE != kOwnGrad;        // x and B; else the gradient, the gate and C
    const bool gated = L.gate.data != nullptr && MODE != kOwnState;
    Ahead<T, NP> ab, ac;
    // tile i of the pass: the i-th from the front, or from the back of the gradient's
    auto start = [&](int i) { return begin + static_cast<int64_t>(MODE == kOwnGrad ? tiles - 1 - i : i) * K; };
    auto count = [&](int64_t t0) { return static_cast<int>(end - t0 < K ? end - t0 : K); };
    auto fetch = [&](int i) {
        const int64_t t0 = start(i);
        const int live = count(t0);
        Buf& to = buf[i & 1];
        load_rows<T, VEC, CB>(to.x, kReads ? L.x : A.g, p, t0, live);
        load_rows<T, VEC, CB>(to.delta, L.delta, p, t0, live);
        if (gated && !A.keep_only) load_rows<T, VEC, CB>(to.gate, L.gate, p, t0, live);
        copies_done();
        if (kReads) ab.load(L.b, p.b, p.group, L.N, t0, live);
        if (MODE != kOwnState) ac.load(L.c, p.b, p.group, L.N, t0, live);
    };
    auto land = [&](int i) {
        if (kReads) ab.put(buf[i & 1].b);
        if (MODE != kOwnState) ac.put(buf[i & 1].c);
    };
    T* const out = static_cast<T*>(L.out.data) + p.b * L.out.stride_b + c;
    if (tiles > 0) {
        fetch(0);
        land(0);
    }
    for (int i = 0; i < tiles; ++i) {
        if (i + 1 < tiles) fetch(i + 1);
        else copies_done();
        copies_wait<1>();
        __syncthreads();
        const Buf& at = buf[i & 1];
        const int64_t t0 = start(i);
        const int live = count(t0);
        if (MODE == kMain && L.kept != nullptr && mine)
            store_states<RN>(L.kept + ((p.b * L.chunks + t0 / K) * L.C + c) * L.N, n0, L.N, wide, h);
#pragma unroll 2
        for (int k = 0; k < live; ++k) {
            const int tt = MODE == kOwnGrad ? live - 1 - k : k;
            const float xv = to_f32(at.x[tt][ch]);
            float d = to_f32(at.delta[tt][ch]) + bias;
            if (L.softplus) d = softplus(d);
            if constexpr (MODE != kMain) sum += d;
            const float2 dd = make_float2(d, d);
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            if constexpr (MODE == kOwnGrad) {
                float gy = xv;
                if (gated) {
                    const float z = to_f32(at.gate[tt][ch]);
                    gy *= z * logistic(z);
                }
                const float2 gg = make_float2(gy, gy);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 q = pair_mul(dd, a2[j]);
                    h[j] = pair_mul(make_float2(exp2_hw(q.x), exp2_hw(q.y)),
                                    pair_fma(gg, *reinterpret_cast<const float2*>(&at.c[tt][n0 + 2 * j]), h[j]));
                }
            } else {
                const float dx = d * xv;
                const float2 xx = make_float2(dx, dx);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 q = pair_mul(dd, a2[j]);
                    h[j] = pair_fma(make_float2(exp2_hw(q.x), exp2_hw(q.y)), h[j],
                                    pair_mul(xx, *reinterpret_cast<const float2*>(&at.b[tt][n0 + 2 * j])));
                    if (MODE == kMain)
                        acc[j & 1] = pair_fma(*reinterpret_cast<const float2*>(&at.c[tt][n0 + 2 * j]), h[j], acc[j & 1]);
                }
                if (MODE == kMain && !A.keep_only) {
                    const float2 both = pair_add(acc[0], acc[1]);
                    float y = both.x + both.y;
#pragma unroll
                    for (int m = 1; m < LANES; m *= 2) y += __shfl_xor_sync(0xffffffffu, y, m, LANES);
                    y = fmaf(skip, xv, y);
                    if (gated) {
                        const float z = to_f32(at.gate[tt][ch]);
                        y *= z * logistic(z);
                    }
                    if (sub == 0 && mine) out[(t0 + tt) * L.out.stride_t] = from_f32<T>(y);
                }
            }
        }
        __syncthreads();
        if (i + 1 < tiles) land(i + 1);
    }
    if (!mine) return;
    if constexpr (MODE == kMain) {
        if (!A.keep_only && sub == 0)
            for (int64_t t = end > begin ? end : begin; t < stop; ++t) out[t * L.out.stride_t] = from_f32<T>(0.0f);
        if (L.fin != nullptr && p.seg == L.segs - 1) store_states<RN>(L.fin + row, n0, L.N, wide, h);
    } else {
        store_states<RN>(L.seg_state + p.seg * seg_row + row, n0, L.N, wide, h);
        if (sub == 0) L.seg_sum[(p.seg * L.B + p.b) * L.C + c] = sum;
    }
}

template <typename T, int LANES, int RN, bool VEC, Mode MODE>
cudaError_t go(const ScanArgs& A, int64_t segs) {
    const int bytes = 2 * static_cast<int>(sizeof(Tile<T, LANES, RN>));
    auto* kernel = k_sscan<T, LANES, RN, VEC, MODE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(A.L.G * A.blocks * A.L.B * segs), kThreads, bytes, A.L.stream>>>(A);
    return cudaGetLastError();
}

template <typename T, bool VEC, Mode MODE>
cudaError_t by_states(const ScanArgs& A, int64_t segs) {
    if (A.L.N <= 8) return go<T, 1, 8, VEC, MODE>(A, segs);
    if (A.L.N <= 16) return go<T, 1, 16, VEC, MODE>(A, segs);
    if (A.L.N <= 32) return go<T, 2, 16, VEC, MODE>(A, segs);
    return go<T, 4, 16, VEC, MODE>(A, segs);
}

template <Mode MODE>
cudaError_t by_type(const ScanArgs& A, bool vec, int64_t segs) {
    if (A.L.bf16) return vec ? by_states<__nv_bfloat16, true, MODE>(A, segs) : by_states<__nv_bfloat16, false, MODE>(A, segs);
    return vec ? by_states<float, true, MODE>(A, segs) : by_states<float, false, MODE>(A, segs);
}

// ---------------------------------------------------------------------------
// one token: bound by the states' bytes (read and written once).  A lane holds
// VEC of a channel's states, `lanes` of them a channel, and takes ROWS batch rows
// with the channel's A in registers, their states' loads all in flight.
constexpr int ROWS = 4;

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) k_sscan_step(const __grid_constant__ ScanLaunch L, int lanes) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int sub = static_cast<int>(at % lanes), n0 = sub * VEC;
    const int64_t c = at / lanes;
    const bool mine = c < L.C && n0 < L.N;
    const int64_t cc = c < L.C ? c : L.C - 1, group = cc / (L.C / L.G);
    const int64_t b0 = static_cast<int64_t>(blockIdx.y) * ROWS;
    const int rows = static_cast<int>(L.B - b0 < ROWS ? L.B - b0 : ROWS);
    float a[VEC], h[ROWS][VEC], bv[ROWS][VEC], cv[ROWS][VEC], xv[ROWS], dv[ROWS], zv[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t b = b0 + (r < rows ? r : 0);
        const float* s = L.init + (b * L.C + cc) * L.N + n0;
        const T* pb = static_cast<const T*>(L.b.data) + b * L.b.stride_b + group * L.b.stride_h + n0;
        const T* pc = static_cast<const T*>(L.c.data) + b * L.c.stride_b + group * L.c.stride_h + n0;
        if constexpr (VEC == 4) {
            const float4 v = mine ? *reinterpret_cast<const float4*>(s) : make_float4(0.f, 0.f, 0.f, 0.f);
            h[r][0] = v.x, h[r][1] = v.y, h[r][2] = v.z, h[r][3] = v.w;
        } else {
            h[r][0] = mine ? *s : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            bv[r][j] = mine ? to_f32(pb[j]) : 0.0f;
            cv[r][j] = mine ? to_f32(pc[j]) : 0.0f;
        }
        xv[r] = to_f32((static_cast<const T*>(L.x.data) + b * L.x.stride_b)[cc]);
        dv[r] = to_f32((static_cast<const T*>(L.delta.data) + b * L.delta.stride_b)[cc]);
        zv[r] = L.gate.data != nullptr ? to_f32((static_cast<const T*>(L.gate.data) + b * L.gate.stride_b)[cc]) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) a[j] = mine ? L.a[cc * L.N + n0 + j] * kLog2e : 0.0f;
    const float skip = L.skip != nullptr ? L.skip[cc] : 0.0f, bias = L.bias != nullptr ? L.bias[cc] : 0.0f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (r >= rows) break;
        const int64_t b = b0 + r;
        float d = dv[r] + bias;
        if (L.softplus) d = softplus(d);
        const float dx = d * xv[r];
        float y = 0.0f;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            h[r][j] = fmaf(exp2_hw(d * a[j]), h[r][j], dx * bv[r][j]);
            y = fmaf(cv[r][j], h[r][j], y);
        }
        if (mine) {
            float* s = L.fin + (b * L.C + cc) * L.N + n0;
            if constexpr (VEC == 4) *reinterpret_cast<float4*>(s) = make_float4(h[r][0], h[r][1], h[r][2], h[r][3]);
            else *s = h[r][0];
        }
        for (int m = 1; m < lanes && m < 32; m *= 2) y += __shfl_xor_sync(0xffffffffu, y, m);
        if constexpr (VEC == 1) {
            // 64 states of one value a lane are two warps
            if (lanes > 32) {
                __shared__ float half[kThreads / 32];
                __syncthreads();
                if (threadIdx.x % 32 == 0) half[threadIdx.x / 32] = y;
                __syncthreads();
                y = half[threadIdx.x / 64 * 2] + half[threadIdx.x / 64 * 2 + 1];
            }
        }
        y = fmaf(skip, xv[r], y);
        if (L.gate.data != nullptr) y *= zv[r] * logistic(zv[r]);
        if (sub == 0 && c < L.C) (static_cast<T*>(L.out.data) + b * L.out.stride_b)[cc] = from_f32<T>(y);
    }
}

}  // namespace

cudaError_t launch_scan(const ScanLaunch& L, bool keep_only, int* kernels) {
    ScanArgs A = scan_args(L);
    A.keep_only = keep_only;
    const bool vec = scan_vectors(L, nullptr);
    cudaError_t e;
    *kernels = 0;
    if (L.segs > 1) {
        if ((e = by_type<kOwnState>(A, vec, L.segs - 1)) != cudaSuccess) return e;
        ++*kernels;
    }
    ++*kernels;
    return by_type<kMain>(A, vec, L.segs);
}

// the gradients that the segments' own tokens leave (seg_state, seg_sum; from the second segment on)
cudaError_t launch_scan_own_grads(const ScanBackward& S) {
    ScanArgs A = scan_args(S.f);
    A.g = S.g;
    A.gfin = S.gfin;
    return by_type<kOwnGrad>(A, scan_vectors(S.f, &S.g), S.f.segs - 1);
}

cudaError_t launch_scan_step(const ScanLaunch& L) {
    const bool vec = L.wide;
    int lanes = 1;
    while (lanes * (vec ? 4 : 1) < L.N) lanes *= 2;
    const dim3 grid(static_cast<unsigned>((L.C * lanes + kThreads - 1) / kThreads), static_cast<unsigned>((L.B + ROWS - 1) / ROWS));
    if (L.bf16) {
        if (vec) k_sscan_step<__nv_bfloat16, 4><<<grid, kThreads, 0, L.stream>>>(L, lanes);
        else k_sscan_step<__nv_bfloat16, 1><<<grid, kThreads, 0, L.stream>>>(L, lanes);
    } else {
        if (vec) k_sscan_step<float, 4><<<grid, kThreads, 0, L.stream>>>(L, lanes);
        else k_sscan_step<float, 1><<<grid, kThreads, 0, L.stream>>>(L, lanes);
    }
    return cudaGetLastError();
}

}  // namespace es
