// k_sscan.cu -- the selective scan over whole sequences and for one token:
//
//     h[n] = e^(d A[n]) h[n] + d x B[n],   y = sum_n C[n] h[n] + D x
//
// for every (batch row, channel), d = log(1 + e^(delta + bias)).
//
// Each token, channel and state costs one exponential (32 a clock an SM) and
// four products or sums (128 a clock), against 1/2 byte of traffic at 16 states
// in bf16: the exponentials bound it, not HBM.  What else could: shared memory
// gives a warp 128 bytes a clock whether its lanes read one address or many, so
// B and C cost 2 of 32 words a state if a lane has one channel.  So a lane holds 4
// states of each of 4 channels (as pairs of channels, two products an instruction)
// and 12 words serve 16 states; sums over states cross NL lanes in exchanges
// that halve the values.
//
// Tokens come in tiles of kScanChunk.  Half of a CTA's warps run the states through
// a tile, where the only chain from token to token is one product and sum; the
// other half at the same time make what the next tile's tokens and channels need once
// (d and d x), and the last tile's results, two channels an instruction: some 50 of
// the 131 instructions a token and channel, and half of the warps that hide each
// other's latencies (with every warp doing all three in turn 1.7 of them were there a
// scheduler, and it issued in 38 of 100 clocks).  One barrier a tile.  8 x 1024 x 4096
// channels x 16 states in bf16: 213 us (57 for the exponentials alone), 57 of 100
// clocks issue.  Eight tokens a block of the inner loop: with two it took 7 us more,
// four 12, sixteen 20.
//
// A channel's tokens are a chain, so few channels leave the GPU idle: then the
// tokens are cut into segments, a first pass finds the state each segment makes
// of its own tokens, and the main pass enters each segment with
// h = e^(A sum d) h + own over the segments before it.
#include "es_attn.h"
#include "es_sscan.cuh"

namespace es {
namespace {

constexpr int kThreads = 64, kHalf = 32;             // a CTA's threads, those of either kind
constexpr int K = kScanChunk;
constexpr int kStages = 4;                           // tiles arriving, made ready, run, finished

enum Mode { kMain, kOwnState, kOwnGrad };

template <typename T, int NL>
struct Tile {
    static constexpr int CB = kHalf / 32 * Lanes<NL>::CW, NP = Lanes<NL>::NP;
    struct Stage {
        T x[K][CB], delta[K][CB], gate[K][CB], b[K][NP], c[K][NP];
    };
    Stage stage[kStages];
    float d[2][K][CB], v[2][K][CB];                  // v: d x, or the gradient of y
    float y[2][K][CB];
};

// What both kinds of warps know.
struct Run {
    Place p;
    int64_t begin, stop, end;    // the segment's tokens, those that count
    int tiles;
    template <Mode MODE>
    __device__ __forceinline__ int64_t start(int i) const {      // tile i of the pass: from the back for the gradient's
        return begin + static_cast<int64_t>(MODE == kOwnGrad ? tiles - 1 - i : i) * K;
    }
    __device__ __forceinline__ int live(int64_t t0) const { return static_cast<int>(end - t0 < K ? end - t0 : K); }
};

// The warps that make steps and results.
template <typename T, int NL, Mode MODE>
__device__ __forceinline__ void help(const ScanArgs& A, const Run& R, Tile<T, NL>& buf) {
    constexpr int CB = Tile<T, NL>::CB, NP = Tile<T, NL>::NP, CW = Lanes<NL>::CW, PAIRS = Lanes<NL>::PAIRS, STEP = Lanes<NL>::STEP;
    constexpr bool kWide = sizeof(T) == 4, kReads = MODE != kOwnGrad;      // kReads: x and B; else the gradient, the gate and C
    const ScanLaunch& L = A.L;
    const Place& p = R.p;
    const int id = threadIdx.x % kHalf, lane = id % 32, warp = id / 32;
    const int two = warp * CW + lane % PAIRS * 2, at0 = lane / PAIRS;
    const int64_t c2 = p.first + two;
    const bool in0 = c2 < p.last, in1 = c2 + 1 < p.last;
    float2 skip = pair_of(0.f), bias = pair_of(0.f), sum = pair_of(0.f);
    if (L.skip != nullptr) skip = make_float2(in0 ? L.skip[c2] : 0.f, in1 ? L.skip[c2 + 1] : 0.f);
    if (L.bias != nullptr) bias = make_float2(in0 ? L.bias[c2] : 0.f, in1 ? L.bias[c2 + 1] : 0.f);
    const bool results = MODE == kMain && !A.keep_only, gated = L.gate.data != nullptr && (results || MODE == kOwnGrad);
    const int width = static_cast<int>(p.last - p.first);
    auto from = [&](const es_rows& r, int64_t t0) { return static_cast<const T*>(r.data) + p.b * r.stride_b + t0 * r.stride_t + p.first; };
    auto of_group = [&](const es_heads& r, int64_t t0) {
        return static_cast<const T*>(r.data) + p.b * r.stride_b + t0 * r.stride_t + p.group * r.stride_h;
    };
    auto fetch = [&](int i) {
        const int64_t t0 = R.start<MODE>(i);
        const int live = R.live(t0);
        auto& to = buf.stage[i % kStages];
        load_tile<T, CB, kHalf>(id, to.x, from(kReads ? L.x : A.g, t0), kReads ? L.x.stride_t : A.g.stride_t, width, live, A.vec);
        load_tile<T, CB, kHalf>(id, to.delta, from(L.delta, t0), L.delta.stride_t, width, live, A.vec);
        if (gated) load_tile<T, CB, kHalf>(id, to.gate, from(L.gate, t0), L.gate.stride_t, width, live, A.vec);
        if (kReads) load_tile<T, NP, kHalf>(id, to.b, of_group(L.b, t0), L.b.stride_t, L.N, live, A.vec_bc);
        if (MODE != kOwnState) load_tile<T, NP, kHalf>(id, to.c, of_group(L.c, t0), L.c.stride_t, L.N, live, A.vec_bc);
    };
    T* const out = static_cast<T*>(L.out.data) + p.b * L.out.stride_b + c2;
    if (R.tiles > 0) fetch(0);
    copies_wait<0>();
    __syncthreads();
    for (int i = 0; i < R.tiles + 2; ++i) {
        if (i + 1 < R.tiles) fetch(i + 1);
        if (i < R.tiles) {
            const auto& at = buf.stage[i % kStages];
            const int live = R.live(R.start<MODE>(i));
            float2 d[K / STEP], v[K / STEP];
#pragma unroll
            for (int k = 0; k < K / STEP; ++k) {
                d[k] = pair_add(load_two(&at.delta[at0 + k * STEP][two]), bias);
                v[k] = load_two(&at.x[at0 + k * STEP][two]);
            }
            if (L.softplus) {
#pragma unroll
                for (int k = 0; k < K / STEP; ++k) d[k] = pair_softplus(d[k]);
            }
            if constexpr (MODE == kOwnGrad) {
                if (gated) {
#pragma unroll
                    for (int k = 0; k < K / STEP; ++k) {
                        const float2 z = load_two(&at.gate[at0 + k * STEP][two]);
                        v[k] = pair_mul(v[k], pair_mul(z, pair_logistic<kWide>(z)));
                    }
                }
            }
            // tokens past the last take no step
#pragma unroll
            for (int k = 0; k < K / STEP; ++k) {
                const int tt = at0 + k * STEP;
                if (tt >= live) d[k] = v[k] = pair_of(0.f);
                if (MODE != kMain) sum = pair_add(sum, d[k]);
                store_two(&buf.d[i & 1][tt][two], d[k]);
                store_two(&buf.v[i & 1][tt][two], MODE == kOwnGrad ? v[k] : pair_mul(d[k], v[k]));
            }
        }
        if (results && i >= 2) {
            const auto& at = buf.stage[(i - 2) % kStages];
            const int64_t t0 = R.start<MODE>(i - 2);
            const int live = R.live(t0);
            float2 y[K / STEP];
#pragma unroll
            for (int k = 0; k < K / STEP; ++k) {
                const int tt = at0 + k * STEP;
                y[k] = pair_fma(skip, load_two(&at.x[tt][two]), load_two(&buf.y[i & 1][tt][two]));
            }
            if (gated) {
#pragma unroll
                for (int k = 0; k < K / STEP; ++k) {
                    const float2 z = load_two(&at.gate[at0 + k * STEP][two]);
                    y[k] = pair_mul(y[k], pair_mul(z, pair_logistic<kWide>(z)));
                }
            }
            T* o = out + (t0 + at0) * L.out.stride_t;
            if (A.pairs) {
#pragma unroll
                for (int k = 0; k < K / STEP; ++k) {
                    if (in0 && at0 + k * STEP < live) store_two(o, y[k]);
                    o += STEP * L.out.stride_t;
                }
            } else {
#pragma unroll
                for (int k = 0; k < K / STEP; ++k) {
                    if (in0 && at0 + k * STEP < live) o[0] = from_f32<T>(y[k].x);
                    if (in1 && at0 + k * STEP < live) o[1] = from_f32<T>(y[k].y);
                    o += STEP * L.out.stride_t;
                }
            }
        }
        copies_wait<0>();
        __syncthreads();
    }
    if (results && in0)
        for (int64_t t = (R.end > R.begin ? R.end : R.begin) + at0; t < R.stop; t += STEP) {
            out[t * L.out.stride_t] = from_f32<T>(0.0f);
            if (in1) out[t * L.out.stride_t + 1] = from_f32<T>(0.0f);
        }
    if constexpr (MODE != kMain) {
        // the steps' sums, of the lanes that took every STEP-th token
#pragma unroll
        for (int m = PAIRS; m < 32; m *= 2) {
            sum.x += __shfl_xor_sync(0xffffffffu, sum.x, m);
            sum.y += __shfl_xor_sync(0xffffffffu, sum.y, m);
        }
        float* const to = L.seg_sum + (p.seg * L.B + p.b) * L.C + c2;
        if (at0 == 0 && in0) to[0] = sum.x;
        if (at0 == 0 && in1) to[1] = sum.y;
    }
}

// The warps that run the states.
template <typename T, int NL, Mode MODE>
__device__ __forceinline__ void run(const ScanArgs& A, const Run& R, Tile<T, NL>& buf) {
    constexpr int CW = Lanes<NL>::CW;
    constexpr bool kReads = MODE != kOwnGrad;
    const ScanLaunch& L = A.L;
    const Place& p = R.p;
    const int lane = threadIdx.x % 32, warp = threadIdx.x % kHalf / 32, sub = lane % NL, n0 = 4 * sub;
    const int tile = warp * CW + lane / NL * 4;      // the lane's channels, from p.first
    const int64_t c = p.first + tile;
    const bool wide = L.wide;
    Block h, a2;
    const int64_t rows = L.C * L.N, seg_rows = L.B * rows;      // of a [C, N] table, of a segment's
    load_block(L.a, c, p.last, n0, L.N, wide, a2);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            a2[n][r] = pair_mul(a2[n][r], pair_of(kLog2e));
            h[n][r] = pair_of(0.f);
        }
    if constexpr (MODE == kOwnGrad) {
        if (p.seg == L.segs - 1 && A.gfin != nullptr) load_block(A.gfin + p.b * rows, c, p.last, n0, L.N, wide, h);
    } else if (p.seg == 0) {
        const float* from = MODE == kMain && L.first != nullptr ? L.first : L.init;
        if (from != nullptr) load_block(from + p.b * rows, c, p.last, n0, L.N, wide, h);
        if (MODE == kOwnState && L.first != nullptr) store_block(L.first + p.b * rows, L.N, c, p.last, n0, L.N, wide, h);
    } else if constexpr (MODE == kMain) {
        load_block(L.seg_state + p.b * rows, c, p.last, n0, L.N, wide, h);
        for (int s = 1; s < p.seg; ++s) enter_segment(L, p, s, c, n0, a2, h);
    }
    __syncthreads();
    for (int i = -1; i < R.tiles + 1; ++i) {
        if (i >= 0 && i < R.tiles) {
            const auto& at = buf.stage[i % kStages];
            const int64_t t0 = R.start<MODE>(i);
            const int live = R.live(t0);
            const float *const ds = &buf.d[i & 1][0][tile], *const vs = &buf.v[i & 1][0][tile];
            constexpr int CB = Tile<T, NL>::CB;
            if (MODE == kMain && L.kept != nullptr)
                store_block(L.kept + (p.b * L.chunks + t0 / K) * rows, L.N, c, p.last, n0, L.N, wide, h);
            // what makes up for the exponentials' mean error, by their size at the tile's first (last) token
            Block mend;
            {
                const float4 d = *reinterpret_cast<const float4*>(ds + (MODE == kOwnGrad ? live - 1 : 0) * CB);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    mend[n][0] = decay_mend(pair_mul(make_float2(d.x, d.y), a2[n][0]));
                    mend[n][1] = decay_mend(pair_mul(make_float2(d.z, d.w), a2[n][1]));
                }
            }
            // kBlock tokens at a time: their reads come before the writes of their sums
            constexpr int kBlock = 8;
#pragma unroll 1
            for (int k0 = 0; k0 < live; k0 += kBlock) {
                float2 y[kBlock];
#pragma unroll
                for (int k = 0; k < kBlock; ++k) {
                    const int tt = MODE == kOwnGrad ? (live - 1) / kBlock * kBlock - k0 + kBlock - 1 - k : k0 + k;
                    const float4 d4 = *reinterpret_cast<const float4*>(ds + tt * CB), v4 = *reinterpret_cast<const float4*>(vs + tt * CB);
                    const float2 d[2] = {make_float2(d4.x, d4.y), make_float2(d4.z, d4.w)};
                    const float2 v[2] = {make_float2(v4.x, v4.y), make_float2(v4.z, v4.w)};
                    float4 bv, cv;
                    if (kReads) bv = load_four(&at.b[tt][n0]);
                    if (MODE != kOwnState) cv = load_four(&at.c[tt][n0]);
                    float2 part[2] = {pair_of(0.f), pair_of(0.f)};
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float2 q = pair_fma(d[r], a2[n][r], mend[n][r]);
                            const float2 a = make_float2(exp2_hw(q.x), exp2_hw(q.y));
                            if constexpr (MODE == kOwnGrad) {
                                h[n][r] = pair_mul(a, pair_fma(v[r], pair_of(of_four(cv, n)), h[n][r]));
                            } else {
                                h[n][r] = pair_fma(a, h[n][r], pair_mul(v[r], pair_of(of_four(bv, n))));
                                if (MODE == kMain) {
                                    const float2 cn = pair_of(of_four(cv, n));
                                    part[r] = n == 0 ? pair_mul(cn, h[n][r]) : pair_fma(cn, h[n][r], part[r]);
                                }
                            }
                        }
                    if constexpr (MODE == kMain) y[k] = over_states<NL>(part, sub);
                }
                if constexpr (MODE == kMain) {
#pragma unroll
                    for (int k = 0; k < kBlock; ++k) put_sum<NL>(&buf.y[i & 1][k0 + k][tile], y[k], sub);
                }
            }
        }
        __syncthreads();
    }
    if constexpr (MODE == kMain) {
        if (L.fin != nullptr && p.seg == L.segs - 1) store_block(L.fin + p.b * rows, L.N, c, p.last, n0, L.N, wide, h);
    } else {
        store_block(L.seg_state + p.seg * seg_rows + p.b * rows, L.N, c, p.last, n0, L.N, wide, h);
    }
}

template <typename T, int NL, Mode MODE>
__global__ void __launch_bounds__(kThreads, 7) k_sscan(const __grid_constant__ ScanArgs A) {
    extern __shared__ __align__(128) unsigned char smem[];
    auto& buf = *reinterpret_cast<Tile<T, NL>*>(smem);
    const ScanLaunch& L = A.L;
    Run R;
    R.p = place_of<Tile<T, NL>::CB>(A);
    if constexpr (MODE == kOwnGrad) R.p.seg += 1;    // the first segment's gradient enters none
    const int64_t len = live_tokens(L.lengths, R.p.b, L.T);
    R.begin = R.p.seg * L.seg_chunks * K;
    R.stop = R.begin + L.seg_chunks * K < L.T ? R.begin + L.seg_chunks * K : L.T;
    R.end = R.stop < len ? R.stop : len;
    R.tiles = R.end > R.begin ? static_cast<int>((R.end - R.begin + K - 1) / K) : 0;
    // A warp's place on the SM fixes its scheduler: neighbouring CTAs give the two kinds
    // of warps the other way round, so that each scheduler has as much of both.
    __shared__ uint32_t slot;
    if (threadIdx.x == 0) asm volatile("mov.u32 %0, %%warpid;" : "=r"(slot));
    __syncthreads();
    if ((threadIdx.x < kHalf) == ((slot >> 2 & 1) == 0)) run<T, NL, MODE>(A, R, buf);
    else help<T, NL, MODE>(A, R, buf);
}

template <typename T, int NL, Mode MODE>
cudaError_t go(const ScanArgs& A, int64_t segs) {
    const int bytes = static_cast<int>(sizeof(Tile<T, NL>));
    auto* kernel = k_sscan<T, NL, MODE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(A.L.G * A.blocks * A.L.B * segs), kThreads, bytes, A.L.stream>>>(A);
    return cudaGetLastError();
}

template <typename T, Mode MODE>
cudaError_t by_states(const ScanArgs& A, int64_t segs) {
    if (A.L.N <= 8) return go<T, 2, MODE>(A, segs);
    if (A.L.N <= 16) return go<T, 4, MODE>(A, segs);
    if (A.L.N <= 32) return go<T, 8, MODE>(A, segs);
    return go<T, 16, MODE>(A, segs);
}

template <Mode MODE>
cudaError_t by_type(const ScanArgs& A, int64_t segs) {
    return A.L.bf16 ? by_states<__nv_bfloat16, MODE>(A, segs) : by_states<float, MODE>(A, segs);
}

// ---------------------------------------------------------------------------
// one token: bound by the states' bytes (read and written once).  A lane holds
// VEC of a channel's states, 2^log_lanes of them a channel, and takes ROWS batch rows
// with the channel's A in registers, their states' loads all in flight.  What a row
// and channel need once (the step, the gate, the result) is made by one of the
// channel's lanes: SHARE of them take the rows in turn.
// 256 x 4096 x 16 states: 4 rows and registers for 8 blocks an SM 32.6 us, with ordinary
// instead of streaming accesses 37, 8 rows 42 to 50; the exponents one by one instead of
// in pairs 33.4.  A state's sums are the prompt's, so a token costs it the same bits.
constexpr int kStepThreads = 128, ROWS = 4, kStepBlocks = 8;

template <typename T, int VEC, int SHARE>
__global__ void __launch_bounds__(kStepThreads, kStepBlocks) k_sscan_step(const __grid_constant__ ScanLaunch L, int log_lanes, int fours) {
    constexpr int OWN = ROWS / SHARE;                // rows whose once-a-row work a lane does: those with r % SHARE == sub % SHARE
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kStepThreads + threadIdx.x;
    const int sub = static_cast<int>(at) & ((1 << log_lanes) - 1), n0 = sub * VEC, turn = sub & (SHARE - 1);
    const int64_t c = at >> log_lanes;
    const bool mine = c < L.C && n0 < L.N;
    const int64_t cc = c < L.C ? c : L.C - 1;
    const int64_t group = L.G == 1 ? 0 : static_cast<uint32_t>(cc) / static_cast<uint32_t>(L.C / L.G);
    const int64_t b0 = static_cast<int64_t>(blockIdx.y) * ROWS;
    const int rows = static_cast<int>(L.B - b0 < ROWS ? L.B - b0 : ROWS);
    const int64_t pitch = L.C * L.N, offset = b0 * pitch + cc * L.N + n0;
    const float* const s = L.init + offset;
    const T* const pb = static_cast<const T*>(L.b.data) + b0 * L.b.stride_b + group * L.b.stride_h + n0;
    const T* const pc = static_cast<const T*>(L.c.data) + b0 * L.c.stride_b + group * L.c.stride_h + n0;
    float a[VEC], h[ROWS][VEC], bv[ROWS][VEC], cv[ROWS][VEC];
    float x[OWN], d[OWN], z[OWN], y[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const bool on = mine && r < rows;
        if constexpr (VEC == 4) {
            const float4 v = on ? __ldcs(reinterpret_cast<const float4*>(s + r * pitch)) : make_float4(0.f, 0.f, 0.f, 0.f);
            h[r][0] = v.x, h[r][1] = v.y, h[r][2] = v.z, h[r][3] = v.w;
        } else {
            h[r][0] = on ? s[r * pitch] : 0.0f;
        }
        if (VEC == 4 && fours) {
            Pack<T, VEC> qb{}, qc{};
            if (on) {
                qb = load_raw<T, VEC>(pb + r * L.b.stride_b);
                qc = load_raw<T, VEC>(pc + r * L.c.stride_b);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                bv[r][j] = to_f32(qb.v[j]);
                cv[r][j] = to_f32(qc.v[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                bv[r][j] = on ? to_f32(pb[r * L.b.stride_b + j]) : 0.0f;
                cv[r][j] = on ? to_f32(pc[r * L.c.stride_b + j]) : 0.0f;
            }
        }
    }
    const float skip = L.skip != nullptr ? L.skip[cc] : 0.0f, bias = L.bias != nullptr ? L.bias[cc] : 0.0f;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int r = i * SHARE + turn;
        const int64_t b = b0 + (r < rows ? r : 0);
        x[i] = to_f32((static_cast<const T*>(L.x.data) + b * L.x.stride_b)[cc]);
        d[i] = to_f32((static_cast<const T*>(L.delta.data) + b * L.delta.stride_b)[cc]) + bias;
        z[i] = L.gate.data != nullptr ? to_f32((static_cast<const T*>(L.gate.data) + b * L.gate.stride_b)[cc]) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) a[j] = 0.0f;
    if (mine) {
        const Pack<float, VEC> q = load_raw<float, VEC>(L.a + cc * L.N + n0);
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[j] = q.v[j] * kLog2e;
    }
    if (L.softplus) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) d[i] = softplus(d[i]);
    }
    float* const to = L.fin + offset;
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int from = (lane & ~(SHARE - 1)) + r % SHARE;
        const float dr = __shfl_sync(0xffffffffu, d[r / SHARE], from), dx = __shfl_sync(0xffffffffu, d[r / SHARE] * x[r / SHARE], from);
        y[r] = 0.0f;
        float q[VEC];
        if constexpr (VEC == 1) {
            q[0] = fmaf(dr, a[0], decay_mend(dr * a[0]));
        } else {
#pragma unroll
            for (int j = 0; j < VEC; j += 2) {
                const float2 d2 = pair_of(dr), a2 = make_float2(a[j], a[j + 1]);
                const float2 v = pair_fma(d2, a2, decay_mend(pair_mul(d2, a2)));
                q[j] = v.x, q[j + 1] = v.y;
            }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            h[r][j] = fmaf(exp2_hw(q[j]), h[r][j], dx * bv[r][j]);
            y[r] = fmaf(cv[r][j], h[r][j], y[r]);
        }
        if (mine && r < rows) {
            if constexpr (VEC == 4) __stcs(reinterpret_cast<float4*>(to + r * pitch), make_float4(h[r][0], h[r][1], h[r][2], h[r][3]));
            else to[r * pitch] = h[r][0];
        }
    }
    // the sums over a channel's lanes: first each lane gets its own rows' of SHARE lanes
    float own[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        float v[SHARE];
#pragma unroll
        for (int j = 0; j < SHARE; ++j) v[j] = y[i * SHARE + j];
#pragma unroll
        for (int n = SHARE / 2; n >= 1; n /= 2) {
            const bool hi = turn & n;
#pragma unroll
            for (int j = 0; j < n; ++j) {
                const float keep = hi ? v[j + n] : v[j], send = hi ? v[j] : v[j + n];
                v[j] = keep + __shfl_xor_sync(0xffffffffu, send, n);
            }
        }
        own[i] = v[0];
        for (int m = SHARE; m < 1 << log_lanes && m < 32; m *= 2) own[i] += __shfl_xor_sync(0xffffffffu, own[i], m);
    }
    if constexpr (VEC == 1 && SHARE == 4) {
        // 64 states of one value a lane are two warps
        if (log_lanes > 5) {
            __shared__ float half[kStepThreads / 32][SHARE];
            if (lane < SHARE) half[threadIdx.x / 32][lane] = own[0];
            __syncthreads();
            own[0] = half[threadIdx.x / 64 * 2][turn] + half[threadIdx.x / 64 * 2 + 1][turn];
        }
    }
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int r = i * SHARE + turn;
        float v = fmaf(skip, x[i], own[i]);
        if (L.gate.data != nullptr) v *= z[i] * logistic(z[i]);
        if (sub < SHARE && c < L.C && r < rows) (static_cast<T*>(L.out.data) + (b0 + r) * L.out.stride_b)[cc] = from_f32<T>(v);
    }
}

template <typename T, int VEC>
cudaError_t step(const ScanLaunch& L, int log_lanes, int fours) {
    const dim3 grid(static_cast<unsigned>(((L.C << log_lanes) + kStepThreads - 1) / kStepThreads), static_cast<unsigned>((L.B + ROWS - 1) / ROWS));
    auto* kernel = log_lanes == 0 ? k_sscan_step<T, VEC, 1> : log_lanes == 1 ? k_sscan_step<T, VEC, 2> : k_sscan_step<T, VEC, 4>;
    kernel<<<grid, kStepThreads, 0, L.stream>>>(L, log_lanes, fours);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan(const ScanLaunch& L, bool keep_only, int* kernels) {
    ScanArgs A = scan_args(L, scan_channels(L.N));
    A.keep_only = keep_only;
    A.vec = scan_vectors(L, nullptr);
    A.pairs = scan_pairs(L, L.out);
    cudaError_t e;
    *kernels = 0;
    if (L.segs > 1) {
        if ((e = by_type<kOwnState>(A, L.segs - 1)) != cudaSuccess) return e;
        ++*kernels;
    }
    ++*kernels;
    return by_type<kMain>(A, L.segs);
}

// the gradients that the segments' own tokens leave (seg_state, seg_sum; from the second segment on)
cudaError_t launch_scan_own_grads(const ScanBackward& S) {
    ScanArgs A = scan_args(S.f, scan_channels(S.f.N));
    A.g = S.g;
    A.gfin = S.gfin;
    A.vec = scan_vectors(S.f, &S.g);
    return by_type<kOwnGrad>(A, S.f.segs - 1);
}

cudaError_t launch_scan_step(const ScanLaunch& L) {
    const bool vec = L.wide;
    int log_lanes = 0;
    while ((vec ? 4 : 1) << log_lanes < L.N) ++log_lanes;
    // four neighbouring values of B and C in one access
    const int size = L.bf16 ? 2 : 4;
    int fours = vec;
    for (const es_heads* r : {&L.b, &L.c})
        if (reinterpret_cast<uintptr_t>(r->data) % (4 * size) != 0 || (L.B > 1 && r->stride_b % 4 != 0) || (L.G > 1 && r->stride_h % 4 != 0))
            fours = 0;
    if (L.bf16) return vec ? step<__nv_bfloat16, 4>(L, log_lanes, fours) : step<__nv_bfloat16, 1>(L, log_lanes, fours);
    return vec ? step<float, 4>(L, log_lanes, fours) : step<float, 1>(L, log_lanes, fours);
}

}  // namespace es
