// k_group_norm.cu -- the norm of each group of a token's channels with its gate,
// and the gradients.
//
//     n = (u - mean) / sqrt(var + eps),  y = n w + b,  out = y s(gate)
//
// (u = x, or x s(gate) first; with or without the mean).  Bounded by HBM: x, gate
// and out once.  A team of 8 to 512 threads holds a group in registers as it was
// loaded, so the variance is the mean square distance from the mean and the
// gradient's sums see the same values; a team keeps one group of channels and
// walks over the tokens, with the weights and their gradients' sums in registers.
// Those meet in a second launch, always in one order.
#include "es_attn.h"
#include "es_ssm.cuh"
#include "es_ssm.h"

namespace es {
namespace {

template <int TEAM>
constexpr int kThreadsOf = TEAM <= 32 ? 256 : TEAM;

// N sums over the threads of a team
template <int TEAM, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*part)[N]) {
#pragma unroll
    for (int m = 1; m < (TEAM < 32 ? TEAM : 32); m *= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
    if constexpr (TEAM > 32) {
        constexpr int WARPS = TEAM / 32;
        __syncthreads();                 // the last sums have been read
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) part[threadIdx.x / 32][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = part[threadIdx.x % WARPS][i];
#pragma unroll
            for (int m = 1; m < WARPS; m *= 2) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
        }
    }
}

struct NormArgs {
    NormLaunch L;
    int heads, rows;        // heads and rows of a block at a time
};

template <typename T, int V, int NV, int TEAM, bool BWD>
__global__ void __launch_bounds__(kThreadsOf<TEAM>) k_group_norm(const __grid_constant__ NormArgs A) {
    constexpr int E = NV * V, TEAMS = kThreadsOf<TEAM> / TEAM;
    __shared__ float part1[32][1];
    __shared__ float part2[32][2];
    const NormLaunch& L = A.L;
    const int team = threadIdx.x / TEAM, lane = threadIdx.x % TEAM;
    const int hs = TEAMS == 1 ? 0 : team % A.heads, rs = TEAMS == 1 ? 0 : team / A.heads;
    const int64_t h = static_cast<int64_t>(blockIdx.y) * A.heads + hs;
    const bool team_in = rs < A.rows && h < L.H;
    const int64_t rows = L.B * L.T, step = static_cast<int64_t>(gridDim.x) * A.rows;
    const float inv = 1.0f / static_cast<float>(L.D);
    const bool gated = L.gate.data != nullptr;
    float w[E], bias[E], gw[BWD ? E : 1], gb[BWD ? E : 1];
    int col[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        col[k] = (k * TEAM + lane) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool in = team_in && col[k] < L.D;
            w[k * V + i] = in && L.w != nullptr ? weight_at(L.w, L.w_bf16, h * L.D + col[k] + i) : 1.0f;
            bias[k * V + i] = in && L.bias != nullptr ? weight_at(L.bias, L.w_bf16, h * L.D + col[k] + i) : 0.0f;
            if constexpr (BWD) gw[k * V + i] = gb[k * V + i] = 0.0f;
        }
    }
    // every team of a warp (of a block) makes every turn: the sums are taken together
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * A.rows; r0 < rows; r0 += step) {
        const int64_t r = r0 + rs;
        const bool in = team_in && r < rows;
        const int64_t b = in ? r / L.T : 0, t = in ? r % L.T : 0;
        auto place = [&](const es_heads& v) { return b * v.stride_b + t * v.stride_t + h * v.stride_h; };
        float x[E], z[E], g[BWD ? E : 1];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const bool here = in && col[k] < L.D;
            float v[V];
            zero(v);
            if (here) load_pack<T, V>(static_cast<const T*>(L.x.data) + place(L.x) + col[k], v);
#pragma unroll
            for (int i = 0; i < V; ++i) x[k * V + i] = v[i];
            zero(v);
            if (here && gated) load_pack<T, V>(static_cast<const T*>(L.gate.data) + place(L.gate) + col[k], v);
#pragma unroll
            for (int i = 0; i < V; ++i) z[k * V + i] = v[i];
            if constexpr (BWD) {
                zero(v);
                if (here) load_pack<T, V>(static_cast<const T*>(L.g.data) + place(L.g) + col[k], v);
#pragma unroll
                for (int i = 0; i < V; ++i) g[k * V + i] = v[i];
            }
        }
        float u[E];
#pragma unroll
        for (int e = 0; e < E; ++e) u[e] = gated && L.first ? x[e] * (z[e] * logistic(z[e])) : x[e];
        if (L.center) {
            float s[1] = {0.0f};
#pragma unroll
            for (int e = 0; e < E; ++e) s[0] += u[e];
            team_sum<TEAM>(s, part1);
            const float mean = s[0] * inv;
#pragma unroll
            for (int e = 0; e < E; ++e) u[e] = col[e / V] < L.D ? u[e] - mean : 0.0f;
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int e = 0; e < E; ++e) s[0] = fmaf(u[e], u[e], s[0]);
        team_sum<TEAM>(s, part1);
        const float size = rsqrtf(fmaf(s[0], inv, L.eps));
        if constexpr (!BWD) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = k * V + i;
                    o[i] = fmaf(u[e] * size, w[e], bias[e]);
                    if (gated && !L.first) o[i] *= z[e] * logistic(z[e]);
                    if (L.act) o[i] *= logistic(o[i]);
                }
                if (in && col[k] < L.D) store_pack<T, V>(static_cast<T*>(L.out.data) + place(L.out) + col[k], o);
            }
        } else {
            float two[2] = {0.0f, 0.0f};
            // from here on g is the gradient of n, u is n
#pragma unroll
            for (int e = 0; e < E; ++e) {
                u[e] *= size;
                const float y = fmaf(u[e], w[e], bias[e]);
                if (gated && !L.first) {
                    const float q = logistic(z[e]), of_gate = g[e] * y * silu_slope(z[e], q);
                    g[e] *= z[e] * q;
                    z[e] = of_gate;
                } else if (L.act) {
                    g[e] *= silu_slope(y, logistic(y));
                }
                gw[e] = fmaf(g[e], u[e], gw[e]);
                gb[e] += g[e];
                g[e] *= w[e];
                two[0] += g[e];
                two[1] = fmaf(g[e], u[e], two[1]);
            }
            team_sum<TEAM>(two, part2);
            const float of_mean = L.center ? two[0] * inv : 0.0f, of_size = two[1] * inv;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float gx[V], gz[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = k * V + i;
                    gx[i] = (g[e] - of_mean - u[e] * of_size) * size;
                    gz[i] = z[e];
                    if (gated && L.first) {
                        const float q = logistic(z[e]);
                        gz[i] = gx[i] * x[e] * silu_slope(z[e], q);
                        gx[i] *= z[e] * q;
                    }
                }
                if (in && col[k] < L.D) {
                    store_pack<T, V>(static_cast<T*>(L.out.data) + place(L.out) + col[k], gx);
                    if (gated) store_pack<T, V>(static_cast<T*>(L.ggate.data) + place(L.ggate) + col[k], gz);
                }
            }
        }
    }
    if constexpr (BWD) {
        if (L.partial == nullptr || !team_in) return;
        const int64_t all = static_cast<int64_t>(L.H) * L.D;
        float* const q = L.partial + (static_cast<int64_t>(blockIdx.x) * A.rows + rs) * 2 * all + h * L.D;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (col[e / V] < L.D) {
                q[col[e / V] + e % V] = gw[e];
                q[all + col[e / V] + e % V] = gb[e];
            }
    }
}

struct PutNorm {
    void *gw, *gb;
    int64_t all;
    int bf16;
    __device__ __forceinline__ void operator()(int64_t i, float s) const {
        if (i < all) put_weight(gw, bf16, i, s);
        else put_weight(gb, bf16, i - all, s);
    }
};

// 16-byte accesses: addresses, strides and widths in them
bool vectors(const NormLaunch& L) {
    const int V = L.bf16 ? 8 : 4;
    if (L.D % V != 0) return false;
    for (const es_heads* v : {&L.x, &L.gate, &L.out, &L.g, &L.ggate})
        if (v->data != nullptr && (reinterpret_cast<uintptr_t>(v->data) % 16 != 0 || (L.B > 1 && v->stride_b % V != 0) ||
                                   (L.T > 1 && v->stride_t % V != 0) || (L.H > 1 && v->stride_h % V != 0)))
            return false;
    return true;
}

// The team that a group of D values takes (V values a thread and access).
struct Team {
    int threads, accesses;
};
Team team_of(const NormLaunch& L, bool vec) {
    const int D = L.D;
    if (!vec) return D <= 128 ? Team{32, 4} : D <= 512 ? Team{32, 16} : D <= 2048 ? Team{128, 16} : Team{512, 16};
    if (L.bf16)
        return D <= 64 ? Team{8, 1} : D <= 128 ? Team{16, 1} : D <= 256 ? Team{32, 1} : D <= 512 ? Team{32, 2} : D <= 1024 ? Team{128, 1}
             : D <= 2048 ? Team{128, 2} : D <= 4096 ? Team{512, 1} : Team{512, 2};
    return D <= 32 ? Team{8, 1} : D <= 64 ? Team{16, 1} : D <= 128 ? Team{32, 1} : D <= 256 ? Team{32, 2} : D <= 512 ? Team{32, 4}
         : D <= 1024 ? Team{128, 2} : D <= 2048 ? Team{128, 4} : D <= 4096 ? Team{512, 2} : Team{512, 4};
}

// Blocks: as many as stay resident, so that each reads the weights once.
struct Grid {
    int heads, rows;
    unsigned x, y;
};
Grid grid_of(const NormLaunch& L, bool backward) {
    const int threads = team_of(L, vectors(L)).threads, teams = threads <= 32 ? 256 / threads : 1;
    Grid G;
    G.heads = L.H < teams ? L.H : teams;
    G.rows = teams / G.heads;
    G.y = static_cast<unsigned>((L.H + G.heads - 1) / G.heads);
    const int64_t want = (L.B * L.T + G.rows - 1) / G.rows;
    const int block = threads <= 32 ? 256 : threads;
    int64_t most = static_cast<int64_t>(kSms) * ((backward ? 768 : 1536) / block) / G.y;
    if (most < 1) most = 1;
    G.x = static_cast<unsigned>(want < most ? want : most);
    return G;
}

template <typename T, int V, int NV, int TEAM>
cudaError_t go(const NormLaunch& L, bool backward) {
    const Grid G = grid_of(L, backward);
    const NormArgs A{L, G.heads, G.rows};
    if (backward) k_group_norm<T, V, NV, TEAM, true><<<dim3(G.x, G.y), kThreadsOf<TEAM>, 0, L.stream>>>(A);
    else k_group_norm<T, V, NV, TEAM, false><<<dim3(G.x, G.y), kThreadsOf<TEAM>, 0, L.stream>>>(A);
    return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const NormLaunch& L, bool backward) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = vectors(L);
    const Team t = team_of(L, vec);
    if (!vec) {
        if (t.threads == 32) return t.accesses == 4 ? go<T, 1, 4, 32>(L, backward) : go<T, 1, 16, 32>(L, backward);
        return t.threads == 128 ? go<T, 1, 16, 128>(L, backward) : go<T, 1, 16, 512>(L, backward);
    }
    if (t.threads == 8) return go<T, V, 1, 8>(L, backward);
    if (t.threads == 16) return go<T, V, 1, 16>(L, backward);
    if constexpr (sizeof(T) == 2) {
        if (t.threads == 32) return t.accesses == 1 ? go<T, V, 1, 32>(L, backward) : go<T, V, 2, 32>(L, backward);
        if (t.threads == 128) return t.accesses == 1 ? go<T, V, 1, 128>(L, backward) : go<T, V, 2, 128>(L, backward);
        return t.accesses == 1 ? go<T, V, 1, 512>(L, backward) : go<T, V, 2, 512>(L, backward);
    } else {
        if (t.threads == 32)
            return t.accesses == 1 ? go<T, V, 1, 32>(L, backward) : t.accesses == 2 ? go<T, V, 2, 32>(L, backward) : go<T, V, 4, 32>(L, backward);
        if (t.threads == 128) return t.accesses == 2 ? go<T, V, 2, 128>(L, backward) : go<T, V, 4, 128>(L, backward);
        return t.accesses == 2 ? go<T, V, 2, 512>(L, backward) : go<T, V, 4, 512>(L, backward);
    }
}

}  // namespace

int64_t norm_backward_rows(const NormLaunch& L) {
    const Grid G = grid_of(L, true);
    return static_cast<int64_t>(G.x) * G.rows;
}

cudaError_t launch_norm(const NormLaunch& L, bool backward, int* kernels) {
    *kernels = 1;
    const cudaError_t e = L.bf16 ? pick<__nv_bfloat16>(L, backward) : pick<float>(L, backward);
    if (e != cudaSuccess || L.partial == nullptr) return e;
    ++*kernels;
    const int64_t all = static_cast<int64_t>(L.H) * L.D;
    return sum_rows(L.partial, norm_backward_rows(L), 2 * all, PutNorm{L.gw, L.gb, all, L.w_bf16}, L.stream);
}

}  // namespace es
