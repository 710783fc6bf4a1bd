// es_sscan.cuh -- what the selective scan's kernels share: a CTA's place, tiles of
// operands in shared memory.  A CTA takes scan_channels() (backwards
// scan_bwd_channels()) channels of one group, one batch row and one segment of its tokens.
#pragma once

#include "es_ssm.cuh"
#include "es_ssm.h"

namespace es {

// The hardware's 2^q is low in the mean, in parts of 2^24: for -1 < q < 0 by 0.09 where
// |q| < 2^-9, rising in a line to 0.42 at 2^-7 (0.11 at 0.0025, 0.21 at 0.0043, 0.33 at
// 0.006, 0.40 at 0.0076) and by 0.2 to 0.6 beyond (measured, 2^20 values in each
// twelfth of an octave; 0.5 to 0.7 at random about it).  Over the hundreds of tokens that
// a weak decay remembers the mean adds up where the rest does not (300 tokens of q =
// -0.0047: 4.3e-6 of a state), so it is put back with the exponent, in the sum that a
// product with it costs anyway: under 0.04 is left up to 2^-7, 0.25 up to 2^-6, and from
// 2^-9 on costs a state under 1.6e-6 (one value of 0.37 past 2^-8: 3.4e-6).  Over
// whole rows one q speaks for a tile of kScanChunk tokens (its first token's, or where a
// pass runs backwards its last's).
constexpr float kMendLow = 0.09f, kMendRise = 0.33f, kMendSlope = -62.0f / kMendRise, kMendFrom = -0.15f / kMendRise;
constexpr float kMendPart = 1.44269504f / 16777216.0f;           // of the exponent
__device__ __forceinline__ float mend_place(float q) { return __saturatef(fmaf(q, kMendSlope, kMendFrom)); }
__device__ __forceinline__ float decay_mend(float q) { return fmaf(mend_place(q), kMendRise * kMendPart, kMendLow * kMendPart); }
__device__ __forceinline__ float2 decay_mend(float2 q) {
    return pair_fma(make_float2(mend_place(q.x), mend_place(q.y)), pair_of(kMendRise * kMendPart), pair_of(kMendLow * kMendPart));
}

struct ScanArgs {
    ScanLaunch L;
    es_rows g;               // the gradient of out (backward)
    const float* gfin;
    int64_t per_group;       // channels of a group
    int64_t blocks;          // CTAs over a group's channels
    int keep_only;           // the kept states and no results
    int vec, vec_bc;         // loads in 16-byte pieces: of rows of channels, of B and C
    int pairs;               // stores of two values
};

// The part of a CTA's place that all kernels share.
struct Place {
    int64_t b, group, first, last;   // batch row, group, channels [first, last)
    int seg;
};
template <int CB>
__device__ __forceinline__ Place place_of(const ScanArgs& A) {
    const int64_t across = A.L.G * A.blocks;
    int64_t i = blockIdx.x;
    Place p;
    const int64_t cb = i % across;
    i /= across;
    p.b = i % A.L.B;
    p.seg = static_cast<int>(i / A.L.B);
    p.group = cb / A.blocks;
    p.first = p.group * A.per_group + (cb % A.blocks) * CB;
    const int64_t end = (p.group + 1) * A.per_group;
    p.last = p.first + CB < end ? p.first + CB : end;
    return p;
}

// `live` rows of up to W values, `stride` elements apart, into a tile of K rows;
// zeros elsewhere; thread `id` of THREADS.  `vec`: in 16-byte pieces, to be waited for.
template <typename T, int W, int THREADS>
__device__ __forceinline__ void load_tile(int id, T (*to)[W], const T* from, int64_t stride, int width, int live, bool vec) {
    if (vec) {
        constexpr int V = 16 / sizeof(T), ROW = W / V;
        const int v = id % ROW * V, left = width - v, bytes = (left < 0 ? 0 : left < V ? left : V) * static_cast<int>(sizeof(T));
        const T* f = from + (id / ROW) * stride + v;
#pragma unroll
        for (int i = 0; i < kScanChunk * ROW; i += THREADS) {
            const int tt = (i + id) / ROW;
            if (kScanChunk * ROW % THREADS == 0 || tt < kScanChunk) {
                const int n = tt < live ? bytes : 0;
                copy16(&to[tt][v], n > 0 ? f : from, n);
            }
            f += (THREADS / ROW) * stride;
        }
    } else {
        for (int i = id; i < kScanChunk * W; i += THREADS) {
            const int tt = i / W, v = i % W;
            to[tt][v] = tt < live && v < width ? from[tt * stride + v] : from_f32<T>(0.0f);
        }
    }
}

// How the lanes of a warp share its channels and their states: a lane holds 4
// states of each of 4 neighbouring channels, NL lanes (the low bits) the states of
// one channel.  Values of two neighbouring channels make a pair.
template <int NL>
struct Lanes {
    static constexpr int NP = 4 * NL;            // states, padded
    static constexpr int CW = 128 / NL;          // channels a warp
    static constexpr int PAIRS = CW / 2, STEP = 32 / PAIRS;      // what is done once a token and channel: a lane takes
                                                                 // two channels at every STEP-th token
};
using Block = float2[4][2];                      // [state][pair of channels]

// states n0.. of channels c.. (below `last`) of a [channels, N] table
__device__ __forceinline__ void load_block(const float* table, int64_t c, int64_t last, int n0, int N, bool wide, Block& h) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c + r < last) {
            const float* const q = table + (c + r) * N + n0;
            if (wide) {
                if (n0 < N) v = *reinterpret_cast<const float4*>(q);
            } else {
                v.x = n0 < N ? q[0] : 0.f;
                v.y = n0 + 1 < N ? q[1] : 0.f;
                v.z = n0 + 2 < N ? q[2] : 0.f;
                v.w = n0 + 3 < N ? q[3] : 0.f;
            }
        }
        (r & 1 ? h[0][r / 2].y : h[0][r / 2].x) = v.x;
        (r & 1 ? h[1][r / 2].y : h[1][r / 2].x) = v.y;
        (r & 1 ? h[2][r / 2].y : h[2][r / 2].x) = v.z;
        (r & 1 ? h[3][r / 2].y : h[3][r / 2].x) = v.w;
    }
}

__device__ __forceinline__ void store_block(float* table, int64_t pitch, int64_t c, int64_t last, int n0, int N, bool wide, const Block& h) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (c + r >= last) continue;
        float* const q = table + (c + r) * pitch + n0;
        const float4 v = r & 1 ? make_float4(h[0][r / 2].y, h[1][r / 2].y, h[2][r / 2].y, h[3][r / 2].y)
                               : make_float4(h[0][r / 2].x, h[1][r / 2].x, h[2][r / 2].x, h[3][r / 2].x);
        if (wide) {
            if (n0 < N) *reinterpret_cast<float4*>(q) = v;
        } else {
            if (n0 < N) q[0] = v.x;
            if (n0 + 1 < N) q[1] = v.y;
            if (n0 + 2 < N) q[2] = v.z;
            if (n0 + 3 < N) q[3] = v.w;
        }
    }
}

// the state (or its gradient) past segment s: what entered, through the segment's decays, and its own
__device__ __forceinline__ void enter_segment(const ScanLaunch& L, const Place& p, int s, int64_t c, int n0, const Block& a2, Block& h) {
    Block own;
    load_block(L.seg_state + (s * L.B + p.b) * L.C * L.N, c, p.last, n0, L.N, L.wide, own);
    const float* const sum = L.seg_sum + (s * L.B + p.b) * L.C + c;
    float2 d[2];
    d[0] = make_float2(c < p.last ? sum[0] : 0.f, c + 1 < p.last ? sum[1] : 0.f);
    d[1] = make_float2(c + 2 < p.last ? sum[2] : 0.f, c + 3 < p.last ? sum[3] : 0.f);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float2 q = pair_mul(d[r], a2[n][r]);
            h[n][r] = pair_fma(make_float2(exp2_hw(q.x), exp2_hw(q.y)), h[n][r], own[n][r]);
        }
}

// 4 neighbouring values of a row of B or C in shared memory
__device__ __forceinline__ float4 load_four(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load_four(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ float of_four(const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Sums of 4 channels' values over the NL lanes that share them: the exchanges halve
// the values each lane holds, then sum whole.  Each sum ends in a lane that has
// kept it: NL = 2 keeps two channels a lane, more lanes one (lanes 0..3 of them).
template <int NL>
__device__ __forceinline__ float2 over_states(const float2 (&v)[2], int sub) {
    const bool hi = sub & 1;
    const float2 keep = hi ? v[1] : v[0], send = hi ? v[0] : v[1];
    float2 s;
    s.x = keep.x + __shfl_xor_sync(0xffffffffu, send.x, 1);
    s.y = keep.y + __shfl_xor_sync(0xffffffffu, send.y, 1);
    if constexpr (NL >= 4) {
        const bool odd = sub & 2;
        s.x = (odd ? s.y : s.x) + __shfl_xor_sync(0xffffffffu, odd ? s.x : s.y, 2);
    }
    if constexpr (NL >= 8) s.x += __shfl_xor_sync(0xffffffffu, s.x, 4);
    if constexpr (NL >= 16) s.x += __shfl_xor_sync(0xffffffffu, s.x, 8);
    return s;
}
// ... and where they go, in a row of channels from the lane's first
template <int NL>
__device__ __forceinline__ void put_sum(float* row, float2 s, int sub) {
    if constexpr (NL == 2) *reinterpret_cast<float2*>(row + 2 * (sub & 1)) = s;
    else if (NL == 4 || sub < 4) row[2 * (sub & 1) + (sub >> 1 & 1)] = s.x;
}

// 16-byte pieces: of the rows of channels (addresses and strides in them, and no piece
// across two groups), of B and C
inline bool scan_vectors(const ScanLaunch& L, const es_rows* extra) {
    const int V = L.bf16 ? 8 : 4;
    const es_rows* rows[4] = {&L.x, &L.delta, &L.gate, extra};
    for (const es_rows* r : rows)
        if (r != nullptr && r->data != nullptr &&
            (reinterpret_cast<uintptr_t>(r->data) % 16 != 0 || (L.B > 1 && r->stride_b % V != 0) || (L.T > 1 && r->stride_t % V != 0)))
            return false;
    return L.G == 1 || (L.C / L.G) % V == 0;
}
inline bool scan_bc_vectors(const ScanLaunch& L) {
    const int V = L.bf16 ? 8 : 4;
    for (const es_heads* r : {&L.b, &L.c})
        if (reinterpret_cast<uintptr_t>(r->data) % 16 != 0 || (L.B > 1 && r->stride_b % V != 0) || (L.T > 1 && r->stride_t % V != 0) ||
            (L.G > 1 && r->stride_h % V != 0))
            return false;
    return true;
}

// accesses of two values: addresses, strides and a group's channels in pairs
inline bool scan_pairs(const ScanLaunch& L, const es_rows& r) {
    const int size = L.bf16 ? 2 : 4;
    return reinterpret_cast<uintptr_t>(r.data) % (2 * size) == 0 && (L.B == 1 || r.stride_b % 2 == 0) &&
           (L.T == 1 || r.stride_t % 2 == 0) && (L.C / L.G) % 2 == 0;
}

inline ScanArgs scan_args(const ScanLaunch& L, int channels) {
    ScanArgs A{};
    A.L = L;
    A.per_group = L.C / L.G;
    A.blocks = scan_blocks(L.C, L.G, channels);
    A.vec_bc = scan_bc_vectors(L);
    return A;
}

}  // namespace es
