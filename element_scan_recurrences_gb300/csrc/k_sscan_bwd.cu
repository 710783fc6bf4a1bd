// k_sscan_bwd.cu -- gradients of the selective scan.
//
// With gy the gradient of y = C.h + D x, and dh that of the state, tokens from the
// last to the first:
//
//     dh = dh + gy C,   gC += gy h,   gB += dh d x,   gx = gy D + d (dh.B)
//     u = dh a h' (h' the state before),  gA += u d,  gd = u.A + x (dh.B),   dh = a dh
//
// The states come from those kept every kScanChunk tokens (by the forward call, or
// found first): a chunk's states are formed again forwards, a h' of every token
// stays in shared memory, and the reverse pass forms the decays anew.  A token,
// channel and state costs 14 products and sums and two exponentials, and takes
// part in sums along both the states (y, dh.B, u.A) and the channels (gB, gC).  So
// a warp is 8 lanes of channels by 4 lanes of states, and a lane holds a tile of
// RC channels by RN states of one batch row: sums within the tile are products
// already made, and what is left crosses lanes in exchanges that halve the values
// each time.  gB and gC are summed over the CTA's channels here and over the CTAs
// by a second launch, always in one order.
#include "es_attn.h"
#include "es_sscan.cuh"

namespace es {
namespace {

constexpr int kThreads = kScanThreads, kWarps = kThreads / 32;
constexpr int K = kScanChunk;

struct BwdArgs {
    ScanArgs A;
    ScanBackward S;
};

template <typename T, int RN>
struct Shape {
    static constexpr int RC = RN <= 4 ? 4 : 16 / RN;     // channels a lane
    static constexpr int CW = 8 * RC, CB = kWarps * CW;  // channels a warp, a CTA
    static constexpr int NP = 4 * RN, P = RN / 2;
    static constexpr int Q = RC * RN / 4;                // float4 of a lane's tile
    struct Buf {
        T x[K][CB], delta[K][CB], gate[K][CB], g[K][CB];
        float b[K][NP], c[K][NP];
        float d[K][CB], dx[K][CB], gy[K][CB], y[K][CB];
        float part[K][kWarps][2 * NP];
        float4 stash[K][Q][kThreads];
    };
};

// v[r] summed over the 4 lanes of states; lane r of them (of RC) gets channel r's
template <int RC>
__device__ __forceinline__ float over_states(const float (&v)[RC], int lane) {
    if constexpr (RC == 4) {
        const bool hi = lane & 2, odd = lane & 1;
        const float k0 = (hi ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 2);
        const float k1 = (hi ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 2);
        return (odd ? k1 : k0) + __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 1);
    } else {
        float s;
        if constexpr (RC == 2) {
            const bool odd = lane & 1;
            s = (odd ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
        } else {
            s = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
        }
        return s + __shfl_xor_sync(0xffffffffu, s, 2);
    }
}

// w[0..N) summed over the lanes that differ in bits MASK, MASK / 2 .. 4 (those of
// channels): each lane is left with every 8th part of the sums (one at least) in
// w[0..), those from the returned index on
template <int N, int MASK, int M>
__device__ __forceinline__ int over_channels(float (&w)[M], int lane) {
    if constexpr (MASK < 4) {
        return 0;
    } else if constexpr (N == 1) {
        w[0] += __shfl_xor_sync(0xffffffffu, w[0], MASK);
        return over_channels<1, MASK / 2>(w, lane);
    } else {
        const bool hi = lane & MASK;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float keep = hi ? w[i + N / 2] : w[i], send = hi ? w[i] : w[i + N / 2];
            w[i] = keep + __shfl_xor_sync(0xffffffffu, send, MASK);
        }
        return (hi ? N / 2 : 0) + over_channels<N / 2, MASK / 2>(w, lane);
    }
}

template <typename T, int RN, bool VEC>
__global__ void __launch_bounds__(kThreads) k_sscan_bwd(const __grid_constant__ BwdArgs B) {
    using S = Shape<T, RN>;
    constexpr int RC = S::RC, CW = S::CW, CB = S::CB, NP = S::NP, P = S::P;
    extern __shared__ __align__(128) unsigned char smem[];
    auto& at = *reinterpret_cast<typename S::Buf*>(smem);
    const ScanLaunch& L = B.A.L;
    const Place p = place_of<CB>(B.A);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, quad = lane & 3, n0 = quad * RN;
    const int tile = warp * CW + (lane >> 2) * RC;          // the lane's channels, from p.first
    const int own = tile + (quad < RC ? quad : 0);          // the channel whose sums over states the lane gets
    const bool owner = quad < RC && p.first + own < p.last, wide = L.wide;
    const bool gated = L.gate.data != nullptr;
    const int64_t len = live_tokens(L.lengths, p.b, L.T);
    const int64_t begin = p.seg * L.seg_chunks * K;
    const int64_t stop = begin + L.seg_chunks * K < L.T ? begin + L.seg_chunks * K : L.T;
    const int64_t end = stop < len ? stop : len;
    const int tiles = end > begin ? static_cast<int>((end - begin + K - 1) / K) : 0;
    const int64_t seg_row = L.B * L.C * L.N;

    float2 a2[RC][P], dh[RC][P], ga[RC][P];
    float bias[RC];
#pragma unroll
    for (int r = 0; r < RC; ++r) {
        const int64_t c = p.first + tile + r, row = (p.b * L.C + c) * L.N;
#pragma unroll
        for (int i = 0; i < P; ++i) a2[r][i] = dh[r][i] = ga[r][i] = make_float2(0.f, 0.f);
        bias[r] = 0.0f;
        if (c < p.last) {
            load_states<RN>(L.a + c * L.N, n0, L.N, wide, a2[r]);
#pragma unroll
            for (int i = 0; i < P; ++i) a2[r][i] = pair_mul(a2[r][i], make_float2(kLog2e, kLog2e));
            if (p.seg == L.segs - 1) {
                if (B.S.gfin != nullptr) load_states<RN>(B.S.gfin + row, n0, L.N, wide, dh[r]);
            } else {
                load_states<RN>(L.seg_state + (L.segs - 1) * seg_row + row, n0, L.N, wide, dh[r]);
                for (int s = L.segs - 2; s > p.seg; --s) {
                    const float d = L.seg_sum[(s * L.B + p.b) * L.C + c];
                    float2 own_grad[P];
                    load_states<RN>(L.seg_state + s * seg_row + row, n0, L.N, wide, own_grad);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const float2 q = pair_mul(make_float2(d, d), a2[r][i]);
                        dh[r][i] = pair_fma(make_float2(exp2_hw(q.x), exp2_hw(q.y)), dh[r][i], own_grad[i]);
                    }
                }
            }
        }
    }
    const int64_t oc = p.first + own;
    const float skip = L.skip != nullptr && owner ? L.skip[oc] : 0.0f, own_bias = L.bias != nullptr && owner ? L.bias[oc] : 0.0f;
    float gskip = 0.0f, gbias = 0.0f;
    T* const gx = static_cast<T*>(B.S.gx.data) + p.b * B.S.gx.stride_b + oc;
    T* const gdelta = static_cast<T*>(B.S.gdelta.data) + p.b * B.S.gdelta.stride_b + oc;
    T* const ggate = gated ? static_cast<T*>(B.S.ggate.data) + p.b * B.S.ggate.stride_b + oc : nullptr;
    const int64_t across = L.G * B.A.blocks;
    float* const bc = B.S.part_bc + ((blockIdx.x % across) * L.B + p.b) * L.T * 2 * L.N;

    for (int i = tiles - 1; i >= 0; --i) {
        const int64_t t0 = begin + static_cast<int64_t>(i) * K;
        const int live = static_cast<int>(end - t0 < K ? end - t0 : K);
        load_rows<T, VEC, CB>(at.x, L.x, p, t0, live);
        load_rows<T, VEC, CB>(at.delta, L.delta, p, t0, live);
        load_rows<T, VEC, CB>(at.g, B.A.g, p, t0, live);
        if (gated) load_rows<T, VEC, CB>(at.gate, L.gate, p, t0, live);
        copies_done();
        {
            Ahead<T, NP> ab, ac;
            ab.load(L.b, p.b, p.group, L.N, t0, live);
            ac.load(L.c, p.b, p.group, L.N, t0, live);
            ab.put(at.b);
            ac.put(at.c);
        }
        float2 h[RC][P];
#pragma unroll
        for (int r = 0; r < RC; ++r) {
#pragma unroll
            for (int j = 0; j < P; ++j) h[r][j] = make_float2(0.f, 0.f);
            const int64_t c = p.first + tile + r;
            if (c < p.last) load_states<RN>(L.kept + ((p.b * L.chunks + t0 / K) * L.C + c) * L.N, n0, L.N, wide, h[r]);
        }
        copies_wait<0>();
        __syncthreads();
        // what the tile's lanes share: d, d x and gy of the warp's channels
        for (int k = lane; k < K * CW; k += 32) {
            const int tt = k / CW, ch = warp * CW + k % CW;
            const int64_t c = p.first + ch;
            float d = to_f32(at.delta[tt][ch]) + (L.bias != nullptr && c < p.last ? L.bias[c] : 0.0f);
            if (L.softplus) d = softplus(d);
            float gy = to_f32(at.g[tt][ch]);
            if (gated) {
                const float z = to_f32(at.gate[tt][ch]);
                gy *= z * logistic(z);
            }
            at.d[tt][ch] = d;
            at.dx[tt][ch] = d * to_f32(at.x[tt][ch]);
            at.gy[tt][ch] = gy;
        }
        __syncwarp();
        for (int tt = 0; tt < live; ++tt) {
            float y[RC];
#pragma unroll
            for (int r = 0; r < RC; ++r) {
                const float d = at.d[tt][tile + r], dx = at.dx[tt][tile + r];
                float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 q = pair_mul(make_float2(d, d), a2[r][j]);
                    const float2 ah = pair_mul(make_float2(exp2_hw(q.x), exp2_hw(q.y)), h[r][j]);
                    reinterpret_cast<float2*>(&at.stash[tt][(r * P + j) / 2][threadIdx.x])[(r * P + j) & 1] = ah;
                    h[r][j] = pair_fma(make_float2(dx, dx), *reinterpret_cast<const float2*>(&at.b[tt][n0 + 2 * j]), ah);
                    acc = pair_fma(*reinterpret_cast<const float2*>(&at.c[tt][n0 + 2 * j]), h[r][j], acc);
                }
                y[r] = acc.x + acc.y;
            }
            if (gated) {
                const float whole = over_states<RC>(y, lane);
                if (quad < RC) at.y[tt][own] = whole;
            }
        }
        for (int tt = live - 1; tt >= 0; --tt) {
            float w[2 * RN], s1[RC], s2[RC];
#pragma unroll
            for (int j = 0; j < 2 * RN; ++j) w[j] = 0.0f;
#pragma unroll
            for (int r = 0; r < RC; ++r) {
                const float d = at.d[tt][tile + r], dx = at.dx[tt][tile + r], gy = at.gy[tt][tile + r];
                float2 sb = make_float2(0.f, 0.f), sa = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 bb = *reinterpret_cast<const float2*>(&at.b[tt][n0 + 2 * j]);
                    const float2 cc = *reinterpret_cast<const float2*>(&at.c[tt][n0 + 2 * j]);
                    const float2 ah = reinterpret_cast<const float2*>(&at.stash[tt][(r * P + j) / 2][threadIdx.x])[(r * P + j) & 1];
                    const float2 q = pair_mul(make_float2(d, d), a2[r][j]);
                    const float2 a = make_float2(exp2_hw(q.x), exp2_hw(q.y));
                    const float2 now = pair_fma(make_float2(dx, dx), bb, ah);
                    float2 g = pair_fma(make_float2(gy, gy), cc, dh[r][j]);
                    const float2 pb = pair_fma(g, make_float2(dx, dx), make_float2(w[2 * j], w[2 * j + 1]));
                    const float2 pc = pair_fma(now, make_float2(gy, gy), make_float2(w[RN + 2 * j], w[RN + 2 * j + 1]));
                    w[2 * j] = pb.x, w[2 * j + 1] = pb.y, w[RN + 2 * j] = pc.x, w[RN + 2 * j + 1] = pc.y;
                    sb = pair_fma(g, bb, sb);
                    const float2 u = pair_mul(g, ah);
                    sa = pair_fma(u, a2[r][j], sa);
                    ga[r][j] = pair_fma(u, make_float2(d, d), ga[r][j]);
                    dh[r][j] = pair_mul(g, a);
                }
                s1[r] = sb.x + sb.y;
                s2[r] = sa.x + sa.y;
            }
            const float of_b = over_states<RC>(s1, lane), of_a = over_states<RC>(s2, lane);
            if (owner) {
                const float d = at.d[tt][own], x = to_f32(at.x[tt][own]), gy = at.gy[tt][own];
                float gd = fmaf(of_a, kLn2, of_b * x);
                if (L.softplus) gd *= logistic(to_f32(at.delta[tt][own]) + own_bias);
                gskip = fmaf(gy, x, gskip);
                gbias += gd;
                const int64_t t = t0 + tt;
                gx[t * B.S.gx.stride_t] = from_f32<T>(fmaf(of_b, d, gy * skip));
                gdelta[t * B.S.gdelta.stride_t] = from_f32<T>(gd);
                if (gated) {
                    const float z = to_f32(at.gate[tt][own]);
                    ggate[t * B.S.ggate.stride_t] =
                        from_f32<T>(to_f32(at.g[tt][own]) * fmaf(skip, x, at.y[tt][own]) * silu_slope(z, logistic(z)));
                }
            }
            const int first = over_channels<2 * RN, 16>(w, lane);
            constexpr int LEFT = 2 * RN >= 8 ? 2 * RN / 8 : 1;
#pragma unroll
            for (int j = 0; j < LEFT; ++j) {
                const int e = first + j;
                at.part[tt][warp][(e / RN) * NP + n0 + e % RN] = w[j];
            }
        }
        __syncthreads();
        for (int k = threadIdx.x; k < K * 2 * NP; k += kThreads) {
            const int tt = k / (2 * NP), e = k % (2 * NP), n = e % NP;
            if (tt < live && n < L.N) {
                float s = at.part[tt][0][e];
#pragma unroll
                for (int v = 1; v < kWarps; ++v) s += at.part[tt][v][e];
                bc[(t0 + tt) * 2 * L.N + (e / NP) * L.N + n] = s;
            }
        }
        __syncthreads();
    }
    // tokens past the row's length
    if (owner)
        for (int64_t t = end > begin ? end : begin; t < stop; ++t) {
            gx[t * B.S.gx.stride_t] = from_f32<T>(0.0f);
            gdelta[t * B.S.gdelta.stride_t] = from_f32<T>(0.0f);
            if (gated) ggate[t * B.S.ggate.stride_t] = from_f32<T>(0.0f);
        }
    const int64_t part_row = (static_cast<int64_t>(p.seg) * L.B + p.b) * L.C;
#pragma unroll
    for (int r = 0; r < RC; ++r) {
        const int64_t c = p.first + tile + r;
        if (c >= p.last) continue;
        if (p.seg == 0 && B.S.ginit != nullptr) store_states<RN>(B.S.ginit + (p.b * L.C + c) * L.N, n0, L.N, wide, dh[r]);
        store_states<RN>(B.S.part_c + (part_row + c) * (L.N + 2), n0, L.N, false, ga[r]);
    }
    if (owner) {
        float* const q = B.S.part_c + (part_row + oc) * (L.N + 2) + L.N;
        q[0] = gskip;
        q[1] = gbias;
    }
}

// gB and gC: the sums over the CTAs of a group, token by token
template <typename T>
__global__ void __launch_bounds__(256) k_sscan_sum_bc(const __grid_constant__ BwdArgs B) {
    const ScanLaunch& L = B.A.L;
    const int64_t tokens = L.B * L.T, per = 2 * L.N, all = tokens * L.G * per;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < all; i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t e = i % per, token = i / per % tokens, g = i / per / tokens, b = token / L.T, t = token % L.T;
        float s = 0.0f;
        if (t < live_tokens(L.lengths, b, L.T))
            for (int64_t k = 0; k < B.A.blocks; ++k) s += B.S.part_bc[((g * B.A.blocks + k) * tokens + token) * per + e];
        const es_heads& o = e < L.N ? B.S.gb : B.S.gc;
        static_cast<T*>(o.data)[b * o.stride_b + t * o.stride_t + g * o.stride_h + e % L.N] = from_f32<T>(s);
    }
}

// gA, gskip, gbias: the sums over batch rows and segments
__global__ void __launch_bounds__(256) k_sscan_sum_c(const __grid_constant__ BwdArgs B) {
    const ScanLaunch& L = B.A.L;
    const int64_t per = L.N + 2, all = L.C * per, rows = L.B * L.segs;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= all) return;
    const int64_t c = i / per, e = i % per;
    float* const to = e < L.N ? B.S.ga : e == L.N ? B.S.gskip : B.S.gbias;
    if (to == nullptr) return;
    float s = 0.0f;
    for (int64_t r = 0; r < rows; ++r) s += B.S.part_c[r * all + i];
    to[e < L.N ? c * L.N + e : c] = s;
}

template <typename T, int RN, bool VEC>
cudaError_t go(const BwdArgs& B) {
    const int bytes = static_cast<int>(sizeof(typename Shape<T, RN>::Buf));
    auto* kernel = k_sscan_bwd<T, RN, VEC>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const ScanLaunch& L = B.A.L;
    kernel<<<static_cast<unsigned>(L.G * B.A.blocks * L.B * L.segs), kThreads, bytes, L.stream>>>(B);
    return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t by_states(const BwdArgs& B) {
    const int N = B.A.L.N;
    if (N <= 8) return go<T, 2, VEC>(B);
    if (N <= 16) return go<T, 4, VEC>(B);
    if (N <= 32) return go<T, 8, VEC>(B);
    return go<T, 16, VEC>(B);
}

}  // namespace

cudaError_t launch_scan_backward(const ScanBackward& S, int* kernels) {
    BwdArgs B{scan_args(S.f), S};
    B.A.g = S.g;
    const ScanLaunch& L = S.f;
    const bool vec = scan_vectors(L, &S.g);
    cudaError_t e;
    *kernels = 0;
    if (L.segs > 1) {
        if ((e = launch_scan_own_grads(S)) != cudaSuccess) return e;
        ++*kernels;
    }
    if (L.bf16) e = vec ? by_states<__nv_bfloat16, true>(B) : by_states<__nv_bfloat16, false>(B);
    else e = vec ? by_states<float, true>(B) : by_states<float, false>(B);
    if (e != cudaSuccess) return e;
    ++*kernels;
    if (L.T > 0) {
        const int64_t all = L.B * L.T * L.G * 2 * L.N, most = static_cast<int64_t>(kSms) * 16;
        const int64_t want = (all + 255) / 256;
        const unsigned blocks = static_cast<unsigned>(want < most ? want : most);
        if (L.bf16) k_sscan_sum_bc<__nv_bfloat16><<<blocks, 256, 0, L.stream>>>(B);
        else k_sscan_sum_bc<float><<<blocks, 256, 0, L.stream>>>(B);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        ++*kernels;
    }
    k_sscan_sum_c<<<static_cast<unsigned>((L.C * (L.N + 2) + 255) / 256), 256, 0, L.stream>>>(B);
    ++*kernels;
    return cudaGetLastError();
}

}  // namespace es
