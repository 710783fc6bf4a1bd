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
// Threads an SM holds, which the registers are fitted to.
constexpr int kResident = 768, kResidentBack = 512;
// What hides HBM's latency is the bytes in flight: a thread's rows come through places
// of its own in shared memory (cp.async, no barrier), kAhead of them on their way.  In
// registers there was room for one: 16384 x 16 x 128 in bf16 51 us forwards, now 37
// (0.8 of the measured copy rate), and 87 backwards, now 63 (0.78).
template <int NV, int V>
constexpr int kAhead = V == 1 || NV >= 4 ? 1 : NV == 2 ? 2 : 4;

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

// where the gate goes
enum Gate { kAfter, kFirst, kNone };

template <typename T, int V, int NV, int TEAM, bool BWD, Gate GATE>
__global__ void __launch_bounds__(kThreadsOf<TEAM>, (BWD || NV * V == 16 ? 512 : kResident) / kThreadsOf<TEAM>)
    k_group_norm(const __grid_constant__ NormArgs A) {
    constexpr int E = NV * V, P = E / 2, TEAMS = kThreadsOf<TEAM> / TEAM;
    constexpr bool kWide = sizeof(T) == 4;
    using Raw = Pack<T, V>;
    __shared__ float part1[32][1];
    __shared__ float part2[32][2];
    const NormLaunch& L = A.L;
    const int team = threadIdx.x / TEAM, lane = threadIdx.x % TEAM;
    const int hs = TEAMS == 1 ? 0 : team % A.heads, rs = TEAMS == 1 ? 0 : team / A.heads;
    const int64_t h = static_cast<int64_t>(blockIdx.y) * A.heads + hs;
    const bool team_in = rs < A.rows && h < L.H;
    const int64_t rows = L.B * L.T, step = static_cast<int64_t>(gridDim.x) * A.rows;
    const float inv = 1.0f / static_cast<float>(L.D);
    constexpr bool gated = GATE != kNone;
    // values e and e + 1 of a thread, as pairs; those past the group's last are zeros, and so are their weights
    float2 w[P], bias[P], gw[BWD ? P : 1], gb[BWD ? P : 1];
    auto col = [&](int e) { return (e / V * TEAM + lane) * V + e % V; };
    const bool whole = L.D == TEAM * E;
    auto both = [&](int i, float2 v) {           // v where it is a value of the group
        if (whole) return v;
        return make_float2(col(2 * i) < L.D ? v.x : 0.0f, col(2 * i + 1) < L.D ? v.y : 0.0f);
    };
#pragma unroll
    for (int i = 0; i < P; ++i) {
        w[i] = bias[i] = pair_of(0.f);
        if (BWD) gw[BWD ? i : 0] = gb[BWD ? i : 0] = pair_of(0.f);
        if (team_in) {
            w[i] = both(i, pair_of(1.f));
            const int64_t at = h * L.D;
            const bool in0 = col(2 * i) < L.D, in1 = col(2 * i + 1) < L.D;
            if (L.w != nullptr) {
                if (in0) w[i].x = weight_at(L.w, L.w_bf16, at + col(2 * i));
                if (in1) w[i].y = weight_at(L.w, L.w_bf16, at + col(2 * i + 1));
            }
            if (L.bias != nullptr) {
                if (in0) bias[i].x = weight_at(L.bias, L.w_bf16, at + col(2 * i));
                if (in1) bias[i].y = weight_at(L.bias, L.w_bf16, at + col(2 * i + 1));
            }
        }
    }
    constexpr int AHEAD = kAhead<NV, V>, SLOTS = AHEAD + 1, KINDS = BWD ? 3 : 2;
    extern __shared__ __align__(16) unsigned char smem[];
    auto slot = [&](int64_t turn, int kind, int k) -> Raw& {
        return reinterpret_cast<Raw*>(smem)[((turn * KINDS + kind) * NV + k) * kThreadsOf<TEAM> + threadIdx.x];
    };
    // Rows come `step` apart: a tensor's place moves by as much from turn to turn, and by
    // the difference where the tokens of a batch row end.
    const int64_t step_b = step / L.T, step_t = step % L.T, first = static_cast<int64_t>(blockIdx.x) * A.rows + rs;
    auto place = [&](const es_heads& v) {
        return static_cast<const T*>(v.data) + first / L.T * v.stride_b + first % L.T * v.stride_t + h * v.stride_h + lane * V;
    };
    auto on = [&](const T*& p, const es_heads& v, bool wrapped) {
        p += step_b * v.stride_b + step_t * v.stride_t;
        if (wrapped) p += v.stride_b - L.T * v.stride_t;
    };
    const T *px = place(L.x), *pz = gated ? place(L.gate) : nullptr, *pg = BWD ? place(L.g) : nullptr;      // of the row after this
    const T *po = place(L.out), *pgz = BWD && gated ? place(L.ggate) : nullptr;                             // of this row
    const int64_t last = rows - 1;
    auto move = [&](Raw& to, const T* from) {
        if constexpr (V == 1) to = load_raw<T, V>(from);
        else copy16(&to, from, 16);
    };
    // the row at (px, pz, pg) into the places of a turn, and on to the next one
    int64_t t_next = first % L.T;                // the token of the row that px stands at
    auto fetch = [&](int64_t r, int turn) {
        if (team_in && r <= last) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (!whole && (k * TEAM + lane) * V >= L.D) continue;
                move(slot(turn, 0, k), px + k * TEAM * V);
                if (gated) move(slot(turn, 1, k), pz + k * TEAM * V);
                if (BWD) move(slot(turn, KINDS - 1, k), pg + k * TEAM * V);
            }
        }
        copies_done();
        t_next += step_t;
        const bool wrapped = t_next >= L.T;
        if (wrapped) t_next -= L.T;
        on(px, L.x, wrapped);
        if (gated) on(pz, L.gate, wrapped);
        if (BWD) on(pg, L.g, wrapped);
    };
    auto spread = [&](const Raw (&q)[NV], float2 (&r)[P]) {
#pragma unroll
        for (int i = 0; i < P; ++i) r[i] = make_float2(to_f32(q[2 * i / V].v[2 * i % V]), to_f32(q[(2 * i + 1) / V].v[(2 * i + 1) % V]));
    };
    auto put = [&](const T* p, const float2 (&q)[P]) {
        T* const o = const_cast<T*>(p);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (!whole && (k * TEAM + lane) * V >= L.D) continue;
            Raw raw;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = k * V + i;
                if (V == 1) raw.v[i] = from_f32<T>(e % 2 ? q[e / 2].y : q[e / 2].x);
                else if (i % 2 == 0) store_two(&raw.v[i], q[e / 2]);
            }
            *reinterpret_cast<Raw*>(o + k * TEAM * V) = raw;
        }
    };
    // places past the group's last value and of rows past the last hold zeros
    for (int i = 0; i < SLOTS * KINDS * NV; ++i) reinterpret_cast<Raw*>(smem)[i * kThreadsOf<TEAM> + threadIdx.x] = Raw{};
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(first + i * step, i);
    int turn = 0;
    int64_t t_out = first % L.T;
    // every team of a warp (of a block) makes every turn: the sums are taken together
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * A.rows; r0 < rows; r0 += step) {
        const bool in = team_in && r0 + rs <= last;
        copies_wait<AHEAD - 1>();
        // as loaded until they are needed, which takes half the registers in bf16
        Raw raw_x[NV], raw_z[NV], raw_g[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            raw_x[k] = slot(turn, 0, k);
            if (gated) raw_z[k] = slot(turn, 1, k);
            if (BWD) raw_g[k] = slot(turn, KINDS - 1, k);
        }
        // the place read a turn ago takes the row that comes kAhead after this
        fetch(r0 + rs + AHEAD * step, turn == 0 ? AHEAD : turn - 1);
        if (++turn == SLOTS) turn = 0;
        float2 u[P], of_z[P], slope[P];          // of_z: the gate's factor z s(z)
        auto gate = [&]() {
            spread(raw_z, of_z);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 s = pair_logistic<kWide>(of_z[i]);
                of_z[i] = pair_mul(of_z[i], s);
                if (BWD) slope[i] = pair_fma(of_z[i], pair_fma(s, pair_of(-1.f), pair_of(1.f)), s);      // s + z s (1 - s)
            }
        };
        spread(raw_x, u);
        if constexpr (GATE == kFirst) {
            gate();
#pragma unroll
            for (int i = 0; i < P; ++i) u[i] = pair_mul(u[i], of_z[i]);
        }
        if (L.center) {
            float2 t = pair_of(0.f);
#pragma unroll
            for (int i = 0; i < P; ++i) t = pair_add(t, u[i]);
            float s[1] = {t.x + t.y};
            team_sum<TEAM>(s, part1);
            const float mean = s[0] * inv;
#pragma unroll
            for (int i = 0; i < P; ++i) u[i] = both(i, pair_add(u[i], pair_of(-mean)));
        }
        float2 t = pair_of(0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) t = pair_fma(u[i], u[i], t);
        float s[1] = {t.x + t.y};
        team_sum<TEAM>(s, part1);
        // (0 for a team without a row: its places may hold nothing but zeros, whose reciprocal
        // deviation is infinite where eps is 0, and 0 times that would enter the weights' sums;
        // a team that has its block to itself has a row in every turn)
        const float2 size = pair_of(BWD && TEAMS > 1 && !in ? 0.0f : rsqrtf(fmaf(s[0], inv, L.eps)));
        if constexpr (GATE == kAfter) gate();
        if constexpr (!BWD) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                u[i] = pair_fma(pair_mul(u[i], size), w[i], bias[i]);
                if constexpr (GATE == kAfter) u[i] = pair_mul(u[i], of_z[i]);
                if (GATE == kNone && L.act) u[i] = pair_mul(u[i], pair_logistic<kWide>(u[i]));
            }
            if (in) put(po, u);
        } else {
            // g becomes the gradient of n, u is n, `slope` that of the gate
            float2 g[P];
            spread(raw_g, g);
            float2 t0 = pair_of(0.f), t1 = pair_of(0.f);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                u[i] = pair_mul(u[i], size);
                if (!in) g[i] = pair_of(0.f);
                const float2 y = pair_fma(u[i], w[i], bias[i]);
                if constexpr (GATE == kAfter) {
                    slope[i] = pair_mul(pair_mul(g[i], y), slope[i]);
                    g[i] = pair_mul(g[i], of_z[i]);
                } else if (GATE == kNone && L.act) {
                    const float2 q = pair_logistic<kWide>(y);
                    g[i] = pair_mul(g[i], pair_fma(pair_mul(y, q), pair_fma(q, pair_of(-1.f), pair_of(1.f)), q));
                }
                gw[i] = pair_fma(g[i], u[i], gw[i]);
                gb[i] = pair_add(gb[i], g[i]);
                g[i] = pair_mul(g[i], w[i]);
                t0 = pair_add(t0, g[i]);
                t1 = pair_fma(g[i], u[i], t1);
            }
            float two[2] = {t0.x + t0.y, t1.x + t1.y};
            team_sum<TEAM>(two, part2);
            float2 x[P];
            if constexpr (GATE == kFirst) spread(raw_x, x);
            const float2 of_mean = pair_of(L.center ? -two[0] * inv : 0.0f), of_size = pair_of(-two[1] * inv);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                g[i] = pair_mul(pair_fma(u[i], of_size, pair_add(g[i], of_mean)), size);
                if constexpr (GATE == kFirst) {
                    slope[i] = pair_mul(pair_mul(g[i], x[i]), slope[i]);
                    g[i] = pair_mul(g[i], of_z[i]);
                }
            }
            if (in) {
                put(po, g);
                if (gated) put(pgz, slope);
            }
        }
        t_out += step_t;
        const bool wrapped = t_out >= L.T;
        if (wrapped) t_out -= L.T;
        on(po, L.out, wrapped);
        if (BWD && gated) on(pgz, L.ggate, wrapped);
    }
    if constexpr (BWD) {
        if (L.partial == nullptr || !team_in) return;
        const int64_t all = static_cast<int64_t>(L.H) * L.D;
        float* const q = L.partial + (static_cast<int64_t>(blockIdx.x) * A.rows + rs) * 2 * all + h * L.D;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (col(e) < L.D) {
                q[col(e)] = e % 2 ? gw[e / 2].y : gw[e / 2].x;
                q[all + col(e)] = e % 2 ? gb[e / 2].y : gb[e / 2].x;
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

// The team that a group of D values takes: 8 values a thread, where 512 threads
// are enough for that (16 of them hold a backward call's registers to 128 only by
// spilling), 16 beyond; without 16-byte accesses whole warps.
struct Team {
    int threads, values;
};
Team team_of(const NormLaunch& L, bool vec) {
    if (L.D > 4096) return Team{512, 16};
    int n = vec ? 8 : 32;
    while (n * 8 < L.D) n *= vec ? 2 : 4;
    return Team{n, 8};
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
    int64_t most = static_cast<int64_t>(kSms) * ((backward ? kResidentBack : kResident) / block) / G.y;
    if (most < 1) most = 1;
    G.x = static_cast<unsigned>(want < most ? want : most);
    return G;
}

template <typename T, int V, int E, int TEAM>
cudaError_t go(const NormLaunch& L, bool backward) {
    const Grid G = grid_of(L, backward);
    const NormArgs A{L, G.heads, G.rows};
    const dim3 grid(G.x, G.y);
    const Gate gate = L.gate.data == nullptr ? kNone : L.first ? kFirst : kAfter;
    auto* kernel = backward ? (gate == kNone ? k_group_norm<T, V, E / V, TEAM, true, kNone> : gate == kFirst ? k_group_norm<T, V, E / V, TEAM, true, kFirst> : k_group_norm<T, V, E / V, TEAM, true, kAfter>)
                            : (gate == kNone ? k_group_norm<T, V, E / V, TEAM, false, kNone> : gate == kFirst ? k_group_norm<T, V, E / V, TEAM, false, kFirst> : k_group_norm<T, V, E / V, TEAM, false, kAfter>);
    const int bytes = (kAhead<E / V, V> + 1) * (backward ? 3 : 2) * E * static_cast<int>(sizeof(T)) * kThreadsOf<TEAM>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreadsOf<TEAM>, bytes, L.stream>>>(A);
    return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const NormLaunch& L, bool backward) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = vectors(L);
    const Team t = team_of(L, vec);
    if (t.values == 16) return vec ? go<T, V, 16, 512>(L, backward) : go<T, 1, 16, 512>(L, backward);
    if (!vec)
        return t.threads == 32 ? go<T, 1, 8, 32>(L, backward) : t.threads == 128 ? go<T, 1, 8, 128>(L, backward) : go<T, 1, 8, 512>(L, backward);
    switch (t.threads) {
        case 8: return go<T, V, 8, 8>(L, backward);
        case 16: return go<T, V, 8, 16>(L, backward);
        case 32: return go<T, V, 8, 32>(L, backward);
        case 64: return go<T, V, 8, 64>(L, backward);
        case 128: return go<T, V, 8, 128>(L, backward);
        case 256: return go<T, V, 8, 256>(L, backward);
        default: return go<T, V, 8, 512>(L, backward);
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
