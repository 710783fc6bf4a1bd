// k_sscan_bwd.cu -- gradients of the selective scan.
//
// With gy the gradient of y = C.h + D x, and dh that of the state, tokens from the
// last to the first:
//
//     dh = dh + gy C,   gC += gy h,   gB += dh d x,   gx = gy D + d (dh.B)
//     dh = a dh,   u = dh h' (h' the state before),   gA += u d,   gd = u.A + x (dh.B)
//
// The states come from those kept every kScanChunk tokens (by the forward call, or
// found first): a chunk's states are formed again forwards and stay in tensor
// memory, 16 words a thread and token, which no product uses here; the reverse pass
// forms the decays anew.  A token, channel and state costs 13 products and sums
// (128 a clock an SM) and two exponentials (32), and takes part in sums along both
// the states (y, dh.B, u.A) and the channels (gB, gC): the products bound it, then
// the instructions of the sums.  A lane holds 4 states of each of 4 channels: sums
// within the tile are products already made, sums over states cross NL lanes in
// exchanges, sums over the CTA's channels go through shared memory (each lane's 8
// values of a token, four instructions to write and read them where exchanges took
// 28), those over the CTAs of a group through a second launch, always in one order.
//
// 4 x 2048 x 4096 channels x 16 states in bf16: 762 us, 0.43 of the issue slots taken
// by 362 instructions a token and channel.  What keeps it there is 1.7 warps a
// scheduler: 255 registers a thread, and tensor memory for two CTAs (at up to 8 states
// shared memory for one: 149 KB, in f32 182).  Other warps for what is made once a token
// and channel, as the forward kernel has them, cost five barriers a chunk and took 1099 us.
#include "es_attn.h"
#include "es_sscan.cuh"
#include "es_tcgen05.cuh"

namespace es {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int K = kScanChunk;
constexpr int kGroup = 8;                            // tokens whose sums over channels are taken at once
constexpr int kPitch = kThreads + 4;                 // of a row of their terms: reads of neighbouring rows miss each other's banks
constexpr uint32_t kColumns = 16 * K;                // tensor memory: two CTAs an SM
constexpr int kLeastBytes = 77 * 1024;               // of shared memory, for the same reason

struct BwdArgs {
    ScanArgs A;
    ScanBackward S;
};

template <typename T, int NL>
struct BwdTile {
    static constexpr int CB = kWarps * Lanes<NL>::CW, NP = Lanes<NL>::NP;
    static constexpr int STAGES = sizeof(T) == 2 && NL >= 4 ? 2 : 1;      // two where two CTAs still fit an SM
    struct Stage {
        T x[K][CB], delta[K][CB], gate[K][CB], g[K][CB], b[K][NP], c[K][NP];
    };
    Stage stage[STAGES];
    float d[K][CB], dx[K][CB], gy[K][CB], of_b[K][CB], of_a[K][CB];       // dx: later y
    float4 terms[kGroup][2][kPitch];
    uint32_t tmem;
};

__device__ __forceinline__ void stash(uint32_t addr, const Block& h) {
    uint32_t r[16];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            r[4 * n + 2 * j] = __float_as_uint(h[n][j].x);
            r[4 * n + 2 * j + 1] = __float_as_uint(h[n][j].y);
        }
    tc::st(addr, r);
}
__device__ __forceinline__ float2 stashed(const uint32_t (&r)[16], int n, int j) {
    return make_float2(__uint_as_float(r[4 * n + 2 * j]), __uint_as_float(r[4 * n + 2 * j + 1]));
}

template <typename T, int NL>
__global__ void __launch_bounds__(kThreads, 2) k_sscan_bwd(const __grid_constant__ BwdArgs B) {
    using Buf = BwdTile<T, NL>;
    constexpr int CB = Buf::CB, NP = Buf::NP, CW = Lanes<NL>::CW, PAIRS = Lanes<NL>::PAIRS, STEP = Lanes<NL>::STEP;
    constexpr bool kWide = sizeof(T) == 4;
    extern __shared__ __align__(128) unsigned char smem[];
    Buf& buf = *reinterpret_cast<Buf*>(smem);
    const ScanLaunch& L = B.A.L;
    const Place p = place_of<CB>(B.A);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, sub = lane % NL, n0 = 4 * sub;
    const int tile = warp * CW + lane / NL * 4;      // the lane's channels, from p.first
    const int two = warp * CW + lane % PAIRS * 2, at0 = lane / PAIRS;      // what it does once a token and channel
    const int64_t c = p.first + tile, c2 = p.first + two;
    const bool wide = L.wide, gated = L.gate.data != nullptr;
    const int64_t len = live_tokens(L.lengths, p.b, L.T);
    const int64_t begin = p.seg * L.seg_chunks * K;
    const int64_t stop = begin + L.seg_chunks * K < L.T ? begin + L.seg_chunks * K : L.T;
    const int64_t end = stop < len ? stop : len;
    const int tiles = end > begin ? static_cast<int>((end - begin + K - 1) / K) : 0;
    const int64_t rows = L.C * L.N;                  // of a [C, N] table
    if (warp == 0) tc::alloc(&buf.tmem, kColumns);

    Block a2, dh, ga;
    float2 skip = pair_of(0.f), bias = pair_of(0.f), gskip = pair_of(0.f), gbias = pair_of(0.f);
    if (L.skip != nullptr) skip = make_float2(c2 < p.last ? L.skip[c2] : 0.f, c2 + 1 < p.last ? L.skip[c2 + 1] : 0.f);
    if (L.bias != nullptr) bias = make_float2(c2 < p.last ? L.bias[c2] : 0.f, c2 + 1 < p.last ? L.bias[c2 + 1] : 0.f);
    load_block(L.a, c, p.last, n0, L.N, wide, a2);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            a2[n][r] = pair_mul(a2[n][r], pair_of(kLog2e));
            dh[n][r] = ga[n][r] = pair_of(0.f);
        }
    if (p.seg == L.segs - 1) {
        if (B.S.gfin != nullptr) load_block(B.S.gfin + p.b * rows, c, p.last, n0, L.N, wide, dh);
    } else {
        load_block(L.seg_state + ((L.segs - 1) * L.B + p.b) * rows, c, p.last, n0, L.N, wide, dh);
        for (int s = L.segs - 2; s > p.seg; --s) enter_segment(L, p, s, c, n0, a2, dh);
    }

    const int width = static_cast<int>(p.last - p.first);
    auto start = [&](int i) { return begin + static_cast<int64_t>(i) * K; };
    auto count = [&](int64_t t0) { return static_cast<int>(end - t0 < K ? end - t0 : K); };
    auto from = [&](const es_rows& r, int64_t t0) { return static_cast<const T*>(r.data) + p.b * r.stride_b + t0 * r.stride_t + p.first; };
    auto of_group = [&](const es_heads& r, int64_t t0) {
        return static_cast<const T*>(r.data) + p.b * r.stride_b + t0 * r.stride_t + p.group * r.stride_h;
    };
    auto fetch = [&](int i) {
        const int64_t t0 = start(i);
        const int live = count(t0);
        auto& to = buf.stage[i % Buf::STAGES];
        load_tile<T, CB, kThreads>(threadIdx.x, to.x, from(L.x, t0), L.x.stride_t, width, live, B.A.vec);
        load_tile<T, CB, kThreads>(threadIdx.x, to.delta, from(L.delta, t0), L.delta.stride_t, width, live, B.A.vec);
        load_tile<T, CB, kThreads>(threadIdx.x, to.g, from(B.A.g, t0), B.A.g.stride_t, width, live, B.A.vec);
        if (gated) load_tile<T, CB, kThreads>(threadIdx.x, to.gate, from(L.gate, t0), L.gate.stride_t, width, live, B.A.vec);
        load_tile<T, NP, kThreads>(threadIdx.x, to.b, of_group(L.b, t0), L.b.stride_t, L.N, live, B.A.vec_bc);
        load_tile<T, NP, kThreads>(threadIdx.x, to.c, of_group(L.c, t0), L.c.stride_t, L.N, live, B.A.vec_bc);
    };
    T* const gx = static_cast<T*>(B.S.gx.data) + p.b * B.S.gx.stride_b + c2;
    T* const gdelta = static_cast<T*>(B.S.gdelta.data) + p.b * B.S.gdelta.stride_b + c2;
    T* const ggate = gated ? static_cast<T*>(B.S.ggate.data) + p.b * B.S.ggate.stride_b + c2 : nullptr;
    auto put = [&](T* o, float2 v) {
        if (B.A.pairs) {
            if (c2 < p.last) store_two(o, v);
        } else {
            if (c2 < p.last) o[0] = from_f32<T>(v.x);
            if (c2 + 1 < p.last) o[1] = from_f32<T>(v.y);
        }
    };
    const int64_t across = L.G * B.A.blocks;
    float* const bc = B.S.part_bc + ((blockIdx.x % across) * L.B + p.b) * L.T * 2 * L.N;

    if (tiles > 0) fetch(tiles - 1);
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = buf.tmem + (static_cast<uint32_t>(warp) << 21);      // the warp's 32 lanes

    for (int i = tiles - 1; i >= 0; --i) {
        const int64_t t0 = start(i);
        const int live = count(t0);
        Block h;
        load_block(L.kept + (p.b * L.chunks + t0 / K) * rows, c, p.last, n0, L.N, wide, h);
        copies_wait<0>();
        __syncthreads();
        // the other stage has been read by all: the next chunk's operands on their way
        if (Buf::STAGES == 2 && i > 0) fetch(i - 1);
        const auto& at = buf.stage[i % Buf::STAGES];
        // once a token and channel, some tokens at a time
        constexpr int SOME = K / STEP < 8 ? K / STEP : 8;
#pragma unroll 1
        for (int k0 = 0; k0 < K / STEP; k0 += SOME) {
            float2 d[SOME], gy[SOME];
            const int first = at0 + k0 * STEP;
#pragma unroll
            for (int k = 0; k < SOME; ++k) {
                d[k] = pair_add(load_two(&at.delta[first + k * STEP][two]), bias);
                gy[k] = load_two(&at.g[first + k * STEP][two]);
            }
            if (L.softplus) {
#pragma unroll
                for (int k = 0; k < SOME; ++k) d[k] = pair_softplus(d[k]);
            }
            if (gated) {
#pragma unroll
                for (int k = 0; k < SOME; ++k) {
                    const float2 z = load_two(&at.gate[first + k * STEP][two]);
                    gy[k] = pair_mul(gy[k], pair_mul(z, pair_logistic<kWide>(z)));
                }
            }
            // tokens past the last take no step
#pragma unroll
            for (int k = 0; k < SOME; ++k) {
                const int tt = first + k * STEP;
                if (tt >= live) d[k] = pair_of(0.f);
                store_two(&buf.d[tt][two], d[k]);
                store_two(&buf.dx[tt][two], pair_mul(d[k], load_two(&at.x[tt][two])));
                store_two(&buf.gy[tt][two], gy[k]);
            }
        }
        __syncwarp();
        Block mend;
        {
            const float4 d = *reinterpret_cast<const float4*>(&buf.d[0][tile]);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                mend[n][0] = decay_mend(pair_mul(make_float2(d.x, d.y), a2[n][0]));
                mend[n][1] = decay_mend(pair_mul(make_float2(d.z, d.w), a2[n][1]));
            }
        }
        // the states before each token; tokens past the last leave them as they are
#pragma unroll 4
        for (int tt = 0; tt < K; ++tt) {
            const float4 d4 = *reinterpret_cast<const float4*>(&buf.d[tt][tile]), v4 = *reinterpret_cast<const float4*>(&buf.dx[tt][tile]);
            const float2 d[2] = {make_float2(d4.x, d4.y), make_float2(d4.z, d4.w)};
            const float2 v[2] = {make_float2(v4.x, v4.y), make_float2(v4.z, v4.w)};
            const float4 bv = load_four(&at.b[tt][n0]);
            stash(tmem + 16 * tt, h);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 q = pair_fma(d[r], a2[n][r], mend[n][r]);
                    h[n][r] = pair_fma(make_float2(exp2_hw(q.x), exp2_hw(q.y)), h[n][r], pair_mul(v[r], pair_of(of_four(bv, n))));
                }
        }
        tc::wait_st();
        uint32_t one[16], other[16];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                one[4 * n + 2 * r] = __float_as_uint(h[n][r].x);
                one[4 * n + 2 * r + 1] = __float_as_uint(h[n][r].y);
            }
        tc::ld(tmem + 16 * (K - 1), other);
        // token tt: `now` holds the state after it, `before` (on its way) the one before
        auto step = [&](int tt, uint32_t(&now)[16], uint32_t(&before)[16], float4& tb, float4& tg, float2(&sums)[3]) {
            const float4 d4 = *reinterpret_cast<const float4*>(&buf.d[tt][tile]), v4 = *reinterpret_cast<const float4*>(&buf.dx[tt][tile]),
                         g4 = *reinterpret_cast<const float4*>(&buf.gy[tt][tile]);
            const float2 d[2] = {make_float2(d4.x, d4.y), make_float2(d4.z, d4.w)};
            const float2 v[2] = {make_float2(v4.x, v4.y), make_float2(v4.z, v4.w)};
            const float2 g[2] = {make_float2(g4.x, g4.y), make_float2(g4.z, g4.w)};
            const float4 bv = load_four(&at.b[tt][n0]), cv = load_four(&at.c[tt][n0]);
            float2 y[2], of_b[2], of_a[2];
            float wb[4], wc[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float2 bn = pair_of(of_four(bv, n)), cn = pair_of(of_four(cv, n));
                float2 sb, sc;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 s = stashed(now, n, r), grad = pair_fma(g[r], cn, dh[n][r]);
                    sc = r == 0 ? pair_mul(g[r], s) : pair_fma(g[r], s, sc);
                    sb = r == 0 ? pair_mul(grad, v[r]) : pair_fma(grad, v[r], sb);
                    y[r] = n == 0 ? pair_mul(cn, s) : pair_fma(cn, s, y[r]);
                    of_b[r] = n == 0 ? pair_mul(grad, bn) : pair_fma(grad, bn, of_b[r]);
                    const float2 q = pair_fma(d[r], a2[n][r], mend[n][r]);
                    dh[n][r] = pair_mul(grad, make_float2(exp2_hw(q.x), exp2_hw(q.y)));
                }
                wb[n] = sb.x + sb.y;
                wc[n] = sc.x + sc.y;
            }
            tb = make_float4(wb[0], wb[1], wb[2], wb[3]);
            tg = make_float4(wc[0], wc[1], wc[2], wc[3]);
            tc::wait_ld();
            tc::loaded(before);
            if (tt > 0) tc::ld(tmem + 16 * (tt - 1), now);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 u = pair_mul(dh[n][r], stashed(before, n, r));
                    of_a[r] = n == 0 ? pair_mul(u, a2[n][r]) : pair_fma(u, a2[n][r], of_a[r]);
                    ga[n][r] = pair_fma(u, d[r], ga[n][r]);
                }
            sums[0] = over_states<NL>(of_b, sub);
            sums[1] = over_states<NL>(of_a, sub);
            if (gated) sums[2] = over_states<NL>(y, sub);
        };
        // the tokens in groups whose sums over channels are taken at once, and in twos whose
        // reads come before the writes of their sums
#pragma unroll 1
        for (int k0 = K - kGroup; k0 >= 0; k0 -= kGroup) {
#pragma unroll 1
            for (int k = kGroup - 2; k >= 0; k -= 2) {
                float4 tb[2], tg[2];
                float2 sums[2][3];
                step(k0 + k + 1, one, other, tb[1], tg[1], sums[1]);
                step(k0 + k, other, one, tb[0], tg[0], sums[0]);
                __syncwarp();                        // every lane has read its d x of these tokens, where y goes
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int tt = k0 + k + m;
                    buf.terms[k + m][0][threadIdx.x] = tb[m];
                    buf.terms[k + m][1][threadIdx.x] = tg[m];
                    put_sum<NL>(&buf.of_b[tt][tile], sums[m][0], sub);
                    put_sum<NL>(&buf.of_a[tt][tile], sums[m][1], sub);
                    if (gated) put_sum<NL>(&buf.dx[tt][tile], sums[m][2], sub);
                }
            }
            __syncthreads();
            // gB and gC of these tokens: 16 rows (a token's two) of NL float4 each, the sum of 128 / NL terms
            constexpr int PARTS = 8 / NL > 0 ? 8 / NL : 1, TERMS = kThreads / NL / PARTS, EACH = kThreads / (NL * PARTS);
#pragma unroll
            for (int q = 0; q < 2 * kGroup; q += EACH) {
                const int r = q + threadIdx.x / (NL * PARTS), s = threadIdx.x % NL, part = threadIdx.x / NL % PARTS;
                const float4* const f = &buf.terms[r / 2][r % 2][s + NL * part];
                float4 v = f[0];
#pragma unroll 8
                for (int j = 1; j < TERMS; ++j) {
                    const float4 t = f[j * NL * PARTS];
                    v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
                }
#pragma unroll
                for (int m = NL; m < NL * PARTS; m *= 2) {
                    v.x += __shfl_xor_sync(0xffffffffu, v.x, m);
                    v.y += __shfl_xor_sync(0xffffffffu, v.y, m);
                    v.z += __shfl_xor_sync(0xffffffffu, v.z, m);
                    v.w += __shfl_xor_sync(0xffffffffu, v.w, m);
                }
                const int token = k0 + r / 2;
                if (part == 0 && token < live) {
                    float* const o = bc + ((t0 + token) * 2 + r % 2) * L.N + 4 * s;
                    if (L.N % 4 == 0) {
                        if (4 * s < L.N) *reinterpret_cast<float4*>(o) = v;
                    } else {
                        if (4 * s < L.N) o[0] = v.x;
                        if (4 * s + 1 < L.N) o[1] = v.y;
                        if (4 * s + 2 < L.N) o[2] = v.z;
                        if (4 * s + 3 < L.N) o[3] = v.w;
                    }
                }
            }
            __syncthreads();
        }
#pragma unroll 1
        for (int k0 = 0; k0 < K / STEP; k0 += SOME) {
            float2 gd[SOME], x[SOME], of_z[SOME];
            const int first = at0 + k0 * STEP;
#pragma unroll
            for (int k = 0; k < SOME; ++k) {
                const int t = first + k * STEP;
                x[k] = load_two(&at.x[t][two]);
                gd[k] = pair_fma(load_two(&buf.of_a[t][two]), pair_of(kLn2), pair_mul(load_two(&buf.of_b[t][two]), x[k]));
            }
            if (L.softplus) {
#pragma unroll
                for (int k = 0; k < SOME; ++k)
                    gd[k] = pair_mul(gd[k], pair_logistic<true>(pair_add(load_two(&at.delta[first + k * STEP][two]), bias)));
            }
            if (gated) {
#pragma unroll
                for (int k = 0; k < SOME; ++k) {
                    const int t = first + k * STEP;
                    const float2 z = load_two(&at.gate[t][two]), s = pair_logistic<kWide>(z);
                    const float2 slope = pair_fma(pair_mul(z, s), pair_fma(s, pair_of(-1.f), pair_of(1.f)), s);
                    of_z[k] = pair_mul(pair_mul(load_two(&at.g[t][two]), pair_fma(skip, x[k], load_two(&buf.dx[t][two]))), slope);
                }
            }
#pragma unroll
            for (int k = 0; k < SOME; ++k) {
                const int t = first + k * STEP;
                if (t >= live) break;
                const float2 gy = load_two(&buf.gy[t][two]);
                gskip = pair_fma(gy, x[k], gskip);
                gbias = pair_add(gbias, gd[k]);
                put(gx + (t0 + t) * B.S.gx.stride_t, pair_fma(load_two(&buf.of_b[t][two]), load_two(&buf.d[t][two]), pair_mul(gy, skip)));
                put(gdelta + (t0 + t) * B.S.gdelta.stride_t, gd[k]);
                if (gated) put(ggate + (t0 + t) * B.S.ggate.stride_t, of_z[k]);
            }
        }
        if (Buf::STAGES == 1) {
            __syncthreads();
            if (i > 0) fetch(i - 1);
        }
    }
    // tokens past the row's length
    if (c2 < p.last)
        for (int64_t t = (end > begin ? end : begin) + at0; t < stop; t += STEP) {
            put(gx + t * B.S.gx.stride_t, pair_of(0.f));
            put(gdelta + t * B.S.gdelta.stride_t, pair_of(0.f));
            if (gated) put(ggate + t * B.S.ggate.stride_t, pair_of(0.f));
        }
    if (p.seg == 0 && B.S.ginit != nullptr) store_block(B.S.ginit + p.b * rows, L.N, c, p.last, n0, L.N, wide, dh);
    float* const part = B.S.part_c + (static_cast<int64_t>(p.seg) * L.B + p.b) * L.C * (L.N + 2);
    store_block(part, L.N + 2, c, p.last, n0, L.N, false, ga);
    // the sums of the lanes that took every STEP-th token
#pragma unroll
    for (int m = PAIRS; m < 32; m *= 2) {
        gskip.x += __shfl_xor_sync(0xffffffffu, gskip.x, m);
        gskip.y += __shfl_xor_sync(0xffffffffu, gskip.y, m);
        gbias.x += __shfl_xor_sync(0xffffffffu, gbias.x, m);
        gbias.y += __shfl_xor_sync(0xffffffffu, gbias.y, m);
    }
    if (at0 == 0) {
        float* const q = part + c2 * (L.N + 2) + L.N;
        if (c2 < p.last) q[0] = gskip.x, q[1] = gbias.x;
        if (c2 + 1 < p.last) q[L.N + 2] = gskip.y, q[L.N + 3] = gbias.y;
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::dealloc(buf.tmem, kColumns);
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

template <typename T, int NL>
cudaError_t go(const BwdArgs& B) {
    const int size = static_cast<int>(sizeof(BwdTile<T, NL>)), bytes = size > kLeastBytes ? size : kLeastBytes;
    auto* kernel = k_sscan_bwd<T, NL>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const ScanLaunch& L = B.A.L;
    kernel<<<static_cast<unsigned>(L.G * B.A.blocks * L.B * L.segs), kThreads, bytes, L.stream>>>(B);
    return cudaGetLastError();
}

template <typename T>
cudaError_t by_states(const BwdArgs& B) {
    const int N = B.A.L.N;
    if (N <= 8) return go<T, 2>(B);
    if (N <= 16) return go<T, 4>(B);
    if (N <= 32) return go<T, 8>(B);
    return go<T, 16>(B);
}

}  // namespace

cudaError_t launch_scan_sum_bc(const ScanBackward& S) {
    const BwdArgs B{scan_args(S.f, scan_bwd_channels(S.f.N)), S};
    const ScanLaunch& L = S.f;
    const int64_t all = L.B * L.T * L.G * 2 * L.N, most = static_cast<int64_t>(kSms) * 16;
    const int64_t want = (all + 255) / 256;
    const unsigned blocks = static_cast<unsigned>(want < most ? want : most);
    if (L.bf16) k_sscan_sum_bc<__nv_bfloat16><<<blocks, 256, 0, L.stream>>>(B);
    else k_sscan_sum_bc<float><<<blocks, 256, 0, L.stream>>>(B);
    return cudaGetLastError();
}

cudaError_t launch_scan_backward(const ScanBackward& S, int* kernels) {
    BwdArgs B{scan_args(S.f, scan_bwd_channels(S.f.N)), S};
    B.A.g = S.g;
    const ScanLaunch& L = S.f;
    B.A.vec = scan_vectors(L, &S.g);
    B.A.pairs = scan_pairs(L, S.gx) && scan_pairs(L, S.gdelta) && (S.ggate.data == nullptr || scan_pairs(L, S.ggate));
    cudaError_t e;
    *kernels = 0;
    if (L.segs > 1) {
        if ((e = launch_scan_own_grads(S)) != cudaSuccess) return e;
        ++*kernels;
    }
    e = L.bf16 ? by_states<__nv_bfloat16>(B) : by_states<float>(B);
    if (e != cudaSuccess) return e;
    ++*kernels;
    if (L.T > 0) {
        if ((e = launch_scan_sum_bc(S)) != cudaSuccess) return e;
        ++*kernels;
    }
    k_sscan_sum_c<<<static_cast<unsigned>((L.C * (L.N + 2) + 255) / 256), 256, 0, L.stream>>>(B);
    ++*kernels;
    return cudaGetLastError();
}

}  // namespace es
