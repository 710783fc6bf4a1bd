// k_attn_direct.cu -- linear attention in chunks on the FMA units: any head
// widths up to 256, any strides and alignment, f32 or bf16 operands, every sum
// in f32.  Also the kernels that finish the gradients: the decays' gradient
// from the row products and the sum over heads that share an operand.
//
// One CTA runs one (batch row, head) and a slice of 32 value columns through
// the tokens, 32 at a time.  With G the inclusive sum of the chunk's log
// decays,
//
//     out_i  = sum_{j<=i} e^{G_i-G_j} (x_i.y_j) z_j + e^{G_i} x_i state
//     state' = e^{G_C} state + sum_j e^{G_C-G_j} y_j z_j^T
//
// (reversed: j >= i, e^{G_j-G_i}, and the two chunk coefficients swapped).  G
// is held as two floats, the second what the first lost: after a few strong
// decays it is in the thousands, while the weights that count are those between
// later tokens some hundredths apart (in one float, half of the tokens at -100:
// results off by 3e-5 instead of 1e-7).  A log decay below -104 makes e^g zero
// in f32: such a token starts a new group and contributes nothing to G, so a
// decay of -inf needs no other care.
#include "es_attn.h"
#include "es_device.cuh"
#include "es_pairs.cuh"
#include "es_segments.h"

namespace es {
namespace {

constexpr int C = kAttnChunk;
constexpr int ZS = kAttnSlice;
constexpr int kThreads = 128;
constexpr int kPLd = C + 4;          // rows of P: on 16 bytes
constexpr int kAnchorChunks = kAttnAnchorTokens / C;

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    return static_cast<float>(v);
}

// state = decay state + sum over the chunk's tokens of y u^T, a thread tiles of A rows by 4 columns
template <int A>
__device__ __forceinline__ void update(float* sS, const float* sY, const float* sU, int dxp, int ld, float decay, int tid) {
    for (int tile = tid; tile < (dxp / A) * (ZS / 4); tile += kThreads) {
        const int a = (tile / (ZS / 4)) * A, c = (tile % (ZS / 4)) * 4;
        float2 acc[A][2];
        const float2 d = make_float2(decay, decay);
#pragma unroll
        for (int r = 0; r < A; ++r) {
            const float4 v = *reinterpret_cast<const float4*>(sS + (a + r) * ZS + c);
            acc[r][0] = pair_mul(d, make_float2(v.x, v.y));
            acc[r][1] = pair_mul(d, make_float2(v.z, v.w));
        }
#pragma unroll 8
        for (int j = 0; j < C; ++j) {
            float ya[A];
            if constexpr (A == 4) {
                const float4 yv = *reinterpret_cast<const float4*>(sY + j * ld + a);
                ya[0] = yv.x;
                ya[1] = yv.y;
                ya[2] = yv.z;
                ya[3] = yv.w;
            } else {
                const float2 yv = *reinterpret_cast<const float2*>(sY + j * ld + a);
                ya[0] = yv.x;
                ya[1] = yv.y;
            }
            const float4 uv = *reinterpret_cast<const float4*>(sU + j * ZS + c);
#pragma unroll
            for (int r = 0; r < A; ++r) {
                acc[r][0] = pair_fma(make_float2(ya[r], ya[r]), make_float2(uv.x, uv.y), acc[r][0]);
                acc[r][1] = pair_fma(make_float2(ya[r], ya[r]), make_float2(uv.z, uv.w), acc[r][1]);
            }
        }
#pragma unroll
        for (int r = 0; r < A; ++r)
            *reinterpret_cast<float4*>(sS + (a + r) * ZS + c) = make_float4(acc[r][0].x, acc[r][0].y, acc[r][1].x, acc[r][1].y);
    }
}

struct DirectArgs {
    AttnRun run[3];
    int64_t T;
    int H;
    const float* g;
    int64_t gb, gt, gh;
    const int* lengths;
    int64_t n_anchors;
    int64_t BH;
    int n_segs;
    int64_t seg_chunks;
    float* seg_states;           // [runs][BH][n_segs][dx * dz]: the state entering each segment's successor
    float* seg_decays;           // [runs][BH][n_segs]
};

// Bounded on GB300 by the latency of shared-memory reads and by their number
// (in the main pass shared memory is 64 % busy and 47 % of issue slots are used),
// not by HBM: for one chunk and slice, dx = 128, 426 K FMAs (the 32 x 32 products
// of x and y are formed again in every slice).  So few threads with 4 rows of the
// products each: 256 threads with 2 rows read half as much again, and the training
// pass of 4 x 1000 x 16 heads of 128 took 1451 us instead of 1165 (2 x 501 x 8
// heads of 64: 122 instead of 103; a lone CTA an SM favours them, 4 x 300 x 12
// heads of 96 took 62 instead of 72).  It serves the calls the tensor-core
// kernel cannot take.
//
// The next chunk's operands are on their way in registers (XC columns of 8 rows a
// thread of x and of y) while this one's are worked on; widths above 128 would take
// too many (XC = 0) and wait for theirs.
//
// kStateOnly: a segment's own state, from zero, and its decay (slice 0); x is not read.
template <typename T, int XC, bool kStateOnly>
__global__ void __launch_bounds__(kThreads, XC == 2 ? 4 : XC == 4 ? 3 : 2) k_attn_direct(const __grid_constant__ DirectArgs A) {
    extern __shared__ __align__(16) float sm[];
    const AttnRun& R = A.run[blockIdx.z];
    const int slice = blockIdx.y;
    const int z0 = slice * ZS;
    if (z0 >= R.dz) return;
    const int64_t bh = blockIdx.x / A.n_segs;
    const int seg = static_cast<int>(blockIdx.x % A.n_segs);
    const int64_t b = bh / A.H;
    const int h = static_cast<int>(bh % A.H);
    const int tid = threadIdx.x;
    const int dx = R.dx, dxp = (dx + 3) & ~3, ld = dxp + 4;
    const int nz = min(ZS, R.dz - z0);

    float* sX = sm;                       // [C][ld]
    float* sY = sX + C * ld;              // [C][ld]
    float* sS = sY + C * ld;              // state slice [dxp][ZS]
    float* sZ = sS + dxp * ZS;            // [C][ZS]
    float* sU = sZ + C * ZS;              // z scaled by its chunk coefficient
    float* sP = sU + C * ZS;              // [C][kPLd]
    float* sG = sP + C * kPLd;            // G and what it lost, and per token: coefficient of the read, of the update
    float* sGl = sG + C;
    float* sRead = sGl + C;
    float* sUpd = sRead + C;
    int* sLo = reinterpret_cast<int*>(sUpd + C);    // first token of the group of token i
    float* sDecay = reinterpret_cast<float*>(sLo + C);

    int64_t len = A.T;
    if (A.lengths != nullptr) {
        const int64_t l = A.lengths[b];
        len = l < 0 ? 0 : l < A.T ? l : A.T;
    }
    const T* X = static_cast<const T*>(R.x.p) + b * R.x.sb + (h / R.x.div) * R.x.sh;
    const T* Y = static_cast<const T*>(R.y.p) + b * R.y.sb + (h / R.y.div) * R.y.sh;
    const T* Z = static_cast<const T*>(R.z.p) + b * R.z.sb + (h / R.z.div) * R.z.sh + z0;
    const T* Wd = R.dots != nullptr ? static_cast<const T*>(R.w.p) + b * R.w.sb + (h / R.w.div) * R.w.sh + z0 : nullptr;
    const float* G = A.g != nullptr ? A.g + b * A.gb + h * A.gh : nullptr;
    // the segment's chunks [c0, c1) of the row's `chunks`, and whether they begin or end the run
    const int chunks = static_cast<int>((len + C - 1) / C);
    const SegmentPart part = segment_part(seg, A.n_segs, static_cast<int>(A.seg_chunks), chunks, R.reverse != 0);
    const int64_t c0 = part.c0, c1 = part.c1, n_chunks = c1 > c0 ? c1 - c0 : 0;
    float* dots = R.dots != nullptr ? R.dots + (slice * A.BH + bh) * A.T : nullptr;
    const int64_t out_at = b * R.ob + static_cast<int64_t>(h) * R.oh + z0;
    const bool store_f32 = R.out_f32 != 0;

    // the first state
    const int64_t sbase = bh * R.dx * static_cast<int64_t>(R.dz);
    float* slots = A.n_segs > 1 ? A.seg_states + (blockIdx.z * A.BH + bh) * A.n_segs * R.dx * static_cast<int64_t>(R.dz) : nullptr;
    auto slot = [&](int s) { return slots + s * (R.dx * static_cast<int64_t>(R.dz)) + z0; };
    if constexpr (kStateOnly) {
        if (seg > part.last) return;
        if (part.ends) {
            // no successor: its place keeps the first state, which the last one may take the place of
            if (R.init != nullptr)
                for (int e = tid; e < dx * ZS; e += kThreads)
                    if (e % ZS < nz)
                        slot(seg)[(e / ZS) * static_cast<int64_t>(R.dz) + e % ZS] =
                            R.init[sbase + (e / ZS) * R.sa + (z0 + e % ZS) * R.sc];
            return;
        }
    }
    const float* from = nullptr;
    if (!kStateOnly && part.entry >= 0 && (!part.begins || R.init != nullptr)) from = slot(part.entry);
    for (int e = tid; e < dxp * ZS; e += kThreads) {
        const int a = e / ZS, c = e % ZS;
        float v = 0.0f;
        if (!kStateOnly && a < dx && c < nz) {
            if (from != nullptr) v = from[a * static_cast<int64_t>(R.dz) + c];
            else if (A.n_segs == 1 && R.init != nullptr) v = R.init[sbase + a * R.sa + (z0 + c) * R.sc];
        }
        sS[e] = v;
    }
    // the segment's rows past the length: zero
    if constexpr (!kStateOnly) {
        const int64_t lo = len > c0 * C ? len : c0 * C;
        const int64_t hi = seg == A.n_segs - 1 || (c0 + A.seg_chunks) * C > A.T ? A.T : (c0 + A.seg_chunks) * C;
        for (int64_t e = lo * nz + tid; e < hi * nz; e += kThreads) {
            const int64_t t = e / nz, at = out_at + t * R.ot + e % nz;
            if (store_f32) static_cast<float*>(R.out)[at] = 0.0f;
            else static_cast<T*>(R.out)[at] = static_cast<T>(0.0f);
        }
    }
    float all_decay = 1.0f;
    const int ty = tid / 16, tx = tid % 16;

    // Thread (t4, a) of 4 rows holds rows t4, t4 + 4, .. of columns a, a + 32, .. of x and y
    constexpr int PC = XC > 0 ? XC : 1, PR = C / 4;
    T px[PC][PR], py[PC][PR], pz[PR];
    float pg = 0.0f, cur_g = 0.0f;
    const int t4 = tid / 32, al = tid % 32;
    auto fetch = [&](int64_t k) {
        const int64_t t0 = (R.reverse ? c1 - 1 - k : c0 + k) * C;
#pragma unroll
        for (int r = 0; r < PR; ++r) {
            const int64_t t = t0 + t4 + 4 * r;
            const bool live = t < len;
            const T* xr = X + t * R.x.st;
            const T* yr = Y + t * R.y.st;
#pragma unroll
            for (int c = 0; c < PC; ++c) {
                const int a = al + 32 * c;
                if constexpr (!kStateOnly) px[c][r] = live && a < dx ? xr[a] : static_cast<T>(0.0f);
                py[c][r] = live && a < dx ? yr[a] : static_cast<T>(0.0f);
            }
            pz[r] = live && al < nz ? Z[t * R.z.st + al] : static_cast<T>(0.0f);
        }
        if (tid < 32) pg = G != nullptr && t0 + tid < len ? G[(t0 + tid) * A.gt] : 0.0f;
    };
    auto put = [&]() {
#pragma unroll
        for (int r = 0; r < PR; ++r) {
            const int t = t4 + 4 * r;
#pragma unroll
            for (int c = 0; c < PC; ++c) {
                const int a = al + 32 * c;
                if (a < dxp) {
                    if constexpr (!kStateOnly) sX[t * ld + a] = to_f32(px[c][r]);
                    sY[t * ld + a] = to_f32(py[c][r]);
                }
            }
            sZ[t * ZS + al] = to_f32(pz[r]);
        }
        cur_g = pg;
    };
    if constexpr (XC > 0) {
        if (n_chunks > 0) fetch(0);
    }

    for (int64_t k = 0; k < n_chunks; ++k) {
        const int64_t ci = R.reverse ? c1 - 1 - k : c0 + k;
        const int64_t t0 = ci * C;
        const int n = static_cast<int>(len - t0 < C ? len - t0 : C);
        __syncthreads();
        // for the decays' gradient: the state at the end of an anchor block
        const bool at_anchor = !kStateOnly && R.anchors != nullptr && ((ci + 1) % kAnchorChunks == 0 || ci == chunks - 1);
        auto keep = [&]() {
            float* an = R.anchors + (bh * A.n_anchors + ci / kAnchorChunks) * R.dx * static_cast<int64_t>(R.dz);
            for (int e = tid; e < dx * ZS; e += kThreads) {
                const int a = e / ZS, c = e % ZS;
                if (c < nz) an[static_cast<int64_t>(a) * R.dz + z0 + c] = sS[e];
            }
        };
        if (at_anchor && R.reverse) keep();
        if constexpr (XC > 0) {
            put();
            if (k + 1 < n_chunks) fetch(k + 1);
        } else {
            for (int e = tid; e < C * dxp; e += kThreads) {
                const int t = e / dxp, a = e % dxp;
                const bool in = t < n && a < dx;
                if constexpr (!kStateOnly) sX[t * ld + a] = in ? to_f32(X[(t0 + t) * R.x.st + a]) : 0.0f;
                sY[t * ld + a] = in ? to_f32(Y[(t0 + t) * R.y.st + a]) : 0.0f;
            }
            for (int e = tid; e < C * ZS; e += kThreads) {
                const int t = e / ZS, c = e % ZS;
                sZ[e] = (t < n && c < nz) ? to_f32(Z[(t0 + t) * R.z.st + c]) : 0.0f;
            }
        }
        if (tid < 32) {
            // one token a lane: G, the sum after it, and its group
            float g = cur_g;
            if constexpr (XC == 0) g = G != nullptr && tid < n ? G[(t0 + tid) * A.gt] : 0.0f;
            const bool cut = g < -104.0f;
            g = cut ? 0.0f : g;
            float pre = g, low = 0.0f, nxt = __shfl_down_sync(0xffffffffu, g, 1);
            float suf = tid == 31 ? 0.0f : nxt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float p = __shfl_up_sync(0xffffffffu, pre, o), pl = __shfl_up_sync(0xffffffffu, low, o);
                const float q = __shfl_down_sync(0xffffffffu, suf, o);
                if (tid >= o) {
                    float lost;
                    pre = two_sum(pre, p, lost);
                    low += pl + lost;
                }
                if (tid + o < 32) suf += q;
            }
            const unsigned cuts = __ballot_sync(0xffffffffu, cut);
            const unsigned upto = cuts & (0xffffffffu >> (31 - tid));
            const unsigned after = tid == 31 ? 0u : cuts >> (tid + 1);
            sG[tid] = pre;
            sGl[tid] = low;
            sLo[tid] = upto ? 31 - __clz(upto) : 0;
            const float er = upto ? 0.0f : expf(pre), eu = after ? 0.0f : expf(suf);
            sRead[tid] = (R.reverse ? eu : er) * R.read_scale;
            sUpd[tid] = (R.reverse ? er : eu) * R.update_scale;
            if (tid == 31) *sDecay = cuts ? 0.0f : expf(pre);
        }
        __syncthreads();
        // x_i . y_j with its decay: thread (ty, tx) rows ty + 8r, columns tx, tx + 16
        if constexpr (!kStateOnly) {
            float2 s[4][2];       // even and odd values apart
#pragma unroll
            for (int r = 0; r < 8; ++r) s[r / 2][r % 2] = make_float2(0.0f, 0.0f);
#pragma unroll 4
            for (int a = 0; a < dxp; a += 4) {
                float4 xv[4], yv[2];
#pragma unroll
                for (int r = 0; r < 4; ++r) xv[r] = *reinterpret_cast<const float4*>(sX + (ty + 8 * r) * ld + a);
#pragma unroll
                for (int c = 0; c < 2; ++c) yv[c] = *reinterpret_cast<const float4*>(sY + (tx + 16 * c) * ld + a);
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        s[r][c] = pair_fma(make_float2(xv[r].x, xv[r].y), make_float2(yv[c].x, yv[c].y), s[r][c]);
                        s[r][c] = pair_fma(make_float2(xv[r].z, xv[r].w), make_float2(yv[c].z, yv[c].w), s[r][c]);
                    }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int i = ty + 8 * r, j = tx + 16 * c;
                    const int late = R.reverse ? j : i, early = R.reverse ? i : j;
                    const bool in = early <= late && early >= sLo[late];
                    const float w = expf((sG[late] - sG[early]) + (sGl[late] - sGl[early])) * R.out_scale;
                    sP[i * kPLd + j] = in ? (s[r][c].x + s[r][c].y) * w : 0.0f;
                }
        }
        for (int e = tid; e < C * ZS; e += kThreads) sU[e] = sZ[e] * sUpd[e / ZS];
        __syncthreads();
        // out: thread (ty, tx) rows ty + 8r, columns 2tx, 2tx + 1; what the state gives first, then the chunk
        if constexpr (!kStateOnly) {
            float2 o[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = make_float2(0.0f, 0.0f);
            T wv[4][2];           // on their way meanwhile
            if (Wd != nullptr) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        wv[r][c] = ty + 8 * r < n && 2 * tx + c < nz ? Wd[(t0 + ty + 8 * r) * R.w.st + 2 * tx + c] : static_cast<T>(0.0f);
            }
            auto add = [&](const float* left, int stride, const float* right) {      // 4 terms
                float4 lv[4];
                float2 rv[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) lv[r] = *reinterpret_cast<const float4*>(left + (ty + 8 * r) * stride);
#pragma unroll
                for (int u = 0; u < 4; ++u) rv[u] = *reinterpret_cast<const float2*>(right + u * ZS + 2 * tx);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    o[r] = pair_fma(make_float2(lv[r].x, lv[r].x), rv[0], o[r]);
                    o[r] = pair_fma(make_float2(lv[r].y, lv[r].y), rv[1], o[r]);
                    o[r] = pair_fma(make_float2(lv[r].z, lv[r].z), rv[2], o[r]);
                    o[r] = pair_fma(make_float2(lv[r].w, lv[r].w), rv[3], o[r]);
                }
            };
#pragma unroll 4
            for (int a = 0; a < dxp; a += 4) add(sX + a, ld, sS + a * ZS);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float rd = sRead[ty + 8 * r];
                o[r] = pair_mul(o[r], make_float2(rd, rd));
            }
#pragma unroll 2
            for (int j = 0; j < C; j += 4) add(sP + j, kPLd, sZ + j * ZS);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = ty + 8 * r;
                float dot = 0.0f;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float v = c ? o[r].y : o[r].x;
                    const int zc = 2 * tx + c;
                    if (i < n && zc < nz) {
                        const int64_t at = out_at + (t0 + i) * R.ot + zc;
                        if (store_f32) static_cast<float*>(R.out)[at] = v;
                        else static_cast<T*>(R.out)[at] = static_cast<T>(v);
                        if (Wd != nullptr) dot += v * to_f32(wv[r][c]);
                    }
                }
                if (dots != nullptr) {
#pragma unroll
                    for (int s = 8; s; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
                    if (tx == 0 && i < n) dots[t0 + i] = dot;
                }
            }
        }
        __syncthreads();
        if constexpr (kStateOnly) all_decay *= *sDecay;
        // the state, in tiles of 4 key rows (2 where those would leave threads idle) by 4 columns
        if (dxp <= 32) update<2>(sS, sY, sU, dxp, ld, *sDecay, tid);
        else update<4>(sS, sY, sU, dxp, ld, *sDecay, tid);
        if (at_anchor && !R.reverse) {
            __syncthreads();
            keep();
        }
    }
    __syncthreads();
    if constexpr (kStateOnly) {
        for (int e = tid; e < dx * ZS; e += kThreads)
            if (e % ZS < nz) slot(seg)[(e / ZS) * static_cast<int64_t>(R.dz) + e % ZS] = sS[e];
        if (slice == 0 && tid == 0) A.seg_decays[(blockIdx.z * A.BH + bh) * A.n_segs + seg] = all_decay;
    } else if (R.fin != nullptr && part.ends) {
        for (int e = tid; e < dx * ZS; e += kThreads) {
            const int a = e / ZS, c = e % ZS;
            if (c < nz) R.fin[sbase + a * R.sa + (z0 + c) * R.sc] = sS[e];
        }
    }
}

// State entering each segment from the one before: in order along the run,
// what came in times segment s's decay, plus its own state.  The first state
// lies in the place of the run's last segment, which has no successor.
__global__ void __launch_bounds__(256) k_attn_join(const __grid_constant__ AttnJoin J) {
    const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (e >= J.size) return;
    const int64_t bh = blockIdx.z;
    int64_t len = J.T;
    if (J.lengths != nullptr) {
        const int64_t l = J.lengths[bh / J.H];
        len = l < 0 ? 0 : l < J.T ? l : J.T;
    }
    const int64_t chunks = (len + J.chunk - 1) / J.chunk;
    const int last_seg = chunks > 0 ? static_cast<int>((chunks - 1) / J.seg_chunks) : 0;
    const bool reverse = J.reverse[blockIdx.y];
    float* st = J.states + (blockIdx.y * J.BH + bh) * J.n_segs * J.size + e;
    const float* d = J.decays + (blockIdx.y * J.BH + bh) * J.n_segs;
    float v = J.init[blockIdx.y] ? st[(reverse ? 0 : last_seg) * J.size] : 0.0f;
#pragma unroll 4
    for (int s = 0; s < last_seg; ++s) {
        const int at = reverse ? last_seg - s : s;
        v = fmaf(d[at], v, st[at * J.size]);
        st[at * J.size] = v;
    }
}

// The decays' gradient meets, between the anchor blocks, the product of the
// state and its gradient.  One CTA a product: 8 bytes a value read once, all of
// this kernel's time.  Place 0 is the first state's (zero without one).
__global__ void __launch_bounds__(256) k_attn_state_products(const __grid_constant__ AttnDecayGrad G) {
    __shared__ float part[8];
    const int64_t bh = blockIdx.x / (G.n + 1), m = blockIdx.x % (G.n + 1) - 1;
    const int tid = threadIdx.x;
    int64_t len = G.T;
    if (G.lengths != nullptr) {
        const int64_t l = G.lengths[bh / G.H];
        len = l < 0 ? 0 : l < G.T ? l : G.T;
    }
    const float *a = nullptr, *c = nullptr;
    if (m >= 0) {
        if (m * kAttnAnchorTokens < len) {
            a = G.states_q + (bh * G.n + m) * G.size;
            c = G.states_k + (bh * G.n + m) * G.size;
        }
    } else if (G.initial != nullptr && G.grad_initial != nullptr) {
        a = G.initial + bh * G.size;
        c = G.grad_initial + bh * G.size;
    }
    float s = 0.0f;
    if (a != nullptr) {
        if (G.size % 4 == 0 && reinterpret_cast<uintptr_t>(a) % 16 == 0 && reinterpret_cast<uintptr_t>(c) % 16 == 0) {
            const float4* a4 = reinterpret_cast<const float4*>(a);
            const float4* c4 = reinterpret_cast<const float4*>(c);
#pragma unroll 8
            for (int64_t e = tid; e < G.size / 4; e += 256) {
                const float4 x = a4[e], y = c4[e];
                s += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
            }
        } else {
            for (int64_t e = tid; e < G.size; e += 256) s += a[e] * c[e];
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (tid % 32 == 0) part[tid / 32] = s;
    __syncthreads();
    if (tid == 0) {
        float all = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) all += part[w];
        G.ends[blockIdx.x] = all;
    }
}

// One CTA an anchor block: its tokens from its end, thread t the t-th from the
// end, summed by shuffles within a warp and across the warps through shared
// memory.  The sums are of differences whose terms cancel, so the terms'
// rounding drifts along the block; both of its ends are known, and what is
// missing at the start is spread over the block in proportion (a third of the
// drift's variance is left).
__global__ void __launch_bounds__(kAttnAnchorTokens) k_attn_decay_grad(const __grid_constant__ AttnDecayGrad G) {
    constexpr int kWarps = kAttnAnchorTokens / 32;
    __shared__ float part[kWarps], total[kWarps];
    const int64_t bh = blockIdx.x / G.n, m = blockIdx.x % G.n, BH = G.B * G.H, b = bh / G.H;
    const int h = static_cast<int>(bh % G.H);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    int64_t len = G.T;
    if (G.lengths != nullptr) {
        const int64_t l = G.lengths[b];
        len = l < 0 ? 0 : l < G.T ? l : G.T;
    }
    const int64_t lo = m * kAttnAnchorTokens, full = lo + kAttnAnchorTokens < G.T ? lo + kAttnAnchorTokens : G.T;
    const int64_t hi = full < len ? full : len;
    const int64_t t = hi - 1 - tid;
    const bool in = t >= lo;
    float v = 0.0f;
    if (in) {
        for (int s = 0; s < G.slices; ++s) v += G.dots_q[(s * BH + bh) * G.T + t];
        for (int s = 0; s < G.slices; ++s) v -= G.dots_k[(s * BH + bh) * G.T + t];
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float q = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += q;
    }
    if (lane == 31) total[warp] = v;
    __syncthreads();
    float whole = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) v += total[w];
        whole += total[w];
    }
    if (lo < hi) {
        const float end = G.ends[bh * (G.n + 1) + m + 1], start = G.ends[bh * (G.n + 1) + m];
        // the first block's start is known unless a first state's gradient is not asked for
        const bool known = m > 0 || G.initial == nullptr || G.grad_initial != nullptr;
        const float missing = known ? start - (end + whole) : 0.0f;
        v += end + missing * (static_cast<float>(tid + 1) / static_cast<float>(hi - lo));
    }
    if (in && G.grad != nullptr) G.grad[(b * G.T + t) * G.H + h] = v;
    if (G.grad != nullptr)
        for (int64_t p = (hi > lo ? hi : lo) + tid; p < full; p += kAttnAnchorTokens) G.grad[(b * G.T + p) * G.H + h] = 0.0f;
    if (G.partial != nullptr) {
        float sum = in ? v : 0.0f;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) part[warp] = sum;
        __syncthreads();
        if (tid == 0) {
            float all = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) all += part[w];
            G.partial[h * (G.B * G.n) + b * G.n + m] = all;
        }
    }
}

// [H, n] -> [H] in a fixed order (64-bit sums: a head's gradient adds every token of every row)
__global__ void __launch_bounds__(256) k_attn_sum_rows(const float* __restrict__ part, int64_t n, float* __restrict__ out) {
    __shared__ double s[8];
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 256) v += part[blockIdx.x * n + i];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
        for (int w = 0; w < 8; ++w) all += s[w];
        out[blockIdx.x] = static_cast<float>(all);
    }
}

// One thread four values (VEC) of an operand head: the f32 rows of the heads
// that read it, 16 bytes each, summed in order.  Bounded by their bytes.  grid y:
// which of the call's folds.
struct AttnFolds {
    AttnFold fold[3];
};
template <typename T, int VEC>
__global__ void __launch_bounds__(256) k_attn_fold(const __grid_constant__ AttnFolds A) {
    const AttnFold& F = A.fold[blockIdx.y];
    const uint32_t per = F.d / VEC, heads = F.heads;
    const int64_t n = F.B * F.T * heads * static_cast<int64_t>(per);
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < n; e += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = e / per, bt = row / heads, b = bt / F.T;
        const int c = static_cast<int>(e - row * per) * VEC, j = static_cast<int>(row - bt * heads);
        const float* p = F.part + row * F.div * F.d + c;
        float s[VEC];
#pragma unroll
        for (int u = 0; u < VEC; ++u) s[u] = 0.0f;
#pragma unroll 4
        for (int r = 0; r < F.div; ++r) {
            if constexpr (VEC == 4) {
                const float4 v = *reinterpret_cast<const float4*>(p + static_cast<int64_t>(r) * F.d);
                s[0] += v.x;
                s[1] += v.y;
                s[2] += v.z;
                s[3] += v.w;
            } else {
                s[0] += p[static_cast<int64_t>(r) * F.d];
            }
        }
        T* to = static_cast<T*>(F.out) + b * F.ob + (bt - b * F.T) * F.ot + j * F.oh + c;
#pragma unroll
        for (int u = 0; u < VEC; ++u) to[u] = static_cast<T>(s[u]);
    }
}

size_t direct_smem(int dx) {
    const size_t dxp = (dx + 3) & ~3;
    return sizeof(float) * (2 * C * (dxp + 4) + dxp * ZS + 2 * C * ZS + C * kPLd + 5 * C + 4);
}

}  // namespace

cudaError_t launch_attn_join(const AttnLaunch& L, int chunk) {
    AttnJoin J{};
    for (int r = 0; r < L.runs; ++r) {
        J.reverse[r] = L.run[r].reverse;
        J.init[r] = L.run[r].init != nullptr;
    }
    J.size = static_cast<int64_t>(L.run[0].dx) * L.run[0].dz;     // the same for every run of a call
    J.T = L.T;
    J.BH = L.B * L.H;
    J.H = L.H;
    J.chunk = chunk;
    J.n_segs = L.n_segs;
    J.seg_chunks = L.seg_chunks;
    J.lengths = L.lengths;
    J.states = L.seg_states;
    J.decays = L.seg_decays;
    k_attn_join<<<dim3(static_cast<unsigned>((J.size + 255) / 256), L.runs, static_cast<unsigned>(J.BH)), 256, 0, L.stream>>>(J);
    return cudaGetLastError();
}

template <typename T, int XC>
cudaError_t launch_direct(const DirectArgs& A, const AttnLaunch& L, dim3 grid, size_t smem) {
    cudaError_t e;
    if (A.n_segs > 1) {
        const auto state = k_attn_direct<T, XC, true>;
        if ((e = cudaFuncSetAttribute(state, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem))) != cudaSuccess) return e;
        state<<<grid, kThreads, smem, L.stream>>>(A);
        if ((e = cudaGetLastError()) != cudaSuccess || (e = launch_attn_join(L, C)) != cudaSuccess) return e;
    }
    const auto kernel = k_attn_direct<T, XC, false>;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem))) != cudaSuccess) return e;
    kernel<<<grid, kThreads, smem, L.stream>>>(A);
    return cudaGetLastError();
}

cudaError_t launch_attn_direct(const AttnLaunch& L, int* kernels) {
    DirectArgs A{};
    int dx = 0, dz = 0;
    for (int r = 0; r < L.runs; ++r) {
        A.run[r] = L.run[r];
        dx = L.run[r].dx > dx ? L.run[r].dx : dx;
        dz = L.run[r].dz > dz ? L.run[r].dz : dz;
    }
    A.T = L.T;
    A.H = L.H;
    A.g = L.g;
    A.gb = L.gb;
    A.gt = L.gt;
    A.gh = L.gh;
    A.lengths = L.lengths;
    A.n_anchors = L.n_anchors;
    A.BH = L.B * L.H;
    A.n_segs = L.n_segs;
    A.seg_chunks = L.seg_chunks;
    A.seg_states = L.seg_states;
    A.seg_decays = L.seg_decays;
    *kernels = L.n_segs > 1 ? 3 : 1;
    const size_t smem = direct_smem(dx);
    const dim3 grid(static_cast<unsigned>(A.BH * A.n_segs), (dz + ZS - 1) / ZS, L.runs);
    if (L.bf16)
        return dx <= 64    ? launch_direct<__nv_bfloat16, 2>(A, L, grid, smem)
               : dx <= 128 ? launch_direct<__nv_bfloat16, 4>(A, L, grid, smem)
                           : launch_direct<__nv_bfloat16, 0>(A, L, grid, smem);
    return dx <= 64    ? launch_direct<float, 2>(A, L, grid, smem)
           : dx <= 128 ? launch_direct<float, 4>(A, L, grid, smem)
                       : launch_direct<float, 0>(A, L, grid, smem);
}

cudaError_t launch_attn_decay_grad(const AttnDecayGrad& G, int* kernels) {
    *kernels = 2;
    k_attn_state_products<<<static_cast<unsigned>(G.B * G.H * (G.n + 1)), 256, 0, G.stream>>>(G);
    k_attn_decay_grad<<<static_cast<unsigned>(G.B * G.H * G.n), kAttnAnchorTokens, 0, G.stream>>>(G);
    if (G.grad_h != nullptr) {
        k_attn_sum_rows<<<G.H, 256, 0, G.stream>>>(G.partial, G.B * G.n, G.grad_h);
        ++*kernels;
    }
    return cudaGetLastError();
}

cudaError_t launch_attn_folds(const AttnFold* folds, int n) {
    AttnFolds A{};
    int64_t most = 0;
    bool vec = true;
    for (int i = 0; i < n; ++i) {
        A.fold[i] = folds[i];
        const int64_t values = folds[i].B * folds[i].T * folds[i].heads * static_cast<int64_t>(folds[i].d);
        most = values > most ? values : most;
        vec = vec && folds[i].d % 4 == 0 && reinterpret_cast<uintptr_t>(folds[i].part) % 16 == 0;
    }
    const int64_t blocks = (most / (vec ? 4 : 1) + 255) / 256;
    const dim3 grid(static_cast<unsigned>(blocks < kSms * 8 ? blocks : kSms * 8), n);
    const auto kernel = folds[0].bf16 ? (vec ? k_attn_fold<__nv_bfloat16, 4> : k_attn_fold<__nv_bfloat16, 1>)
                                      : (vec ? k_attn_fold<float, 4> : k_attn_fold<float, 1>);
    kernel<<<grid, 256, 0, folds[0].stream>>>(A);
    return cudaGetLastError();
}

}  // namespace es
