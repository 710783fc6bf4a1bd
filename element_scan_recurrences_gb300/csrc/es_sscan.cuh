// es_sscan.cuh -- what the selective scan's kernels share: a CTA's place, tiles of
// operands in shared memory.  A CTA takes scan_block_channels() channels of one
// group, one batch row and one segment of its tokens.
#pragma once

#include "es_ssm.cuh"
#include "es_ssm.h"

namespace es {

constexpr int kScanThreads = 128;

struct ScanArgs {
    ScanLaunch L;
    es_rows g;               // the gradient of out (backward)
    const float* gfin;
    int64_t per_group;       // channels of a group
    int64_t blocks;          // CTAs over a group's channels
    int keep_only;
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

// `live` tokens from t0 of a [B, T, C] operand into a tile of CB channels
template <typename T, bool VEC, int CB>
__device__ __forceinline__ void load_rows(T (*to)[CB], const es_rows& r, const Place& p, int64_t t0, int live) {
    const T* from = static_cast<const T*>(r.data) + p.b * r.stride_b + t0 * r.stride_t + p.first;
    const int width = static_cast<int>(p.last - p.first);
    if constexpr (VEC) {
        constexpr int V = 16 / sizeof(T), ROW = CB / V > 0 ? CB / V : 1;
        for (int i = threadIdx.x; i < kScanChunk * ROW; i += kScanThreads) {
            const int tt = i / ROW, v = (i % ROW) * V;
            const int n = tt < live && v < width ? (width - v < V ? width - v : V) : 0;
            copy16(&to[tt][v], n > 0 ? from + tt * r.stride_t + v : from, n * static_cast<int>(sizeof(T)));
        }
    } else {
        for (int i = threadIdx.x; i < kScanChunk * CB; i += kScanThreads) {
            const int tt = i / CB, v = i % CB;
            to[tt][v] = tt < live && v < width ? from[tt * r.stride_t + v] : from_f32<T>(0.0f);
        }
    }
}

// B or C of a tile: read ahead into registers, widened into shared memory later
template <typename T, int NP>
struct Ahead {
    static constexpr int COUNT = kScanChunk * NP / kScanThreads;
    float v[COUNT];
    __device__ __forceinline__ void load(const es_heads& r, int64_t b, int64_t group, int N, int64_t t0, int live) {
        const T* from = static_cast<const T*>(r.data) + b * r.stride_b + group * r.stride_h;
#pragma unroll
        for (int j = 0; j < COUNT; ++j) {
            const int i = threadIdx.x + j * kScanThreads, tt = i / NP, n = i % NP;
            v[j] = tt < live && n < N ? to_f32(from[(t0 + tt) * r.stride_t + n]) : 0.0f;
        }
    }
    __device__ __forceinline__ void put(float (*to)[NP]) const {
#pragma unroll
        for (int j = 0; j < COUNT; ++j) {
            const int i = threadIdx.x + j * kScanThreads;
            to[i / NP][i % NP] = v[j];
        }
    }
};

// 16-byte pieces of every operand's rows: addresses and strides in them, and no piece across two groups
inline bool scan_vectors(const ScanLaunch& L, const es_rows* extra) {
    const int size = L.bf16 ? 2 : 4, V = 16 / size;
    const es_rows* rows[4] = {&L.x, &L.delta, &L.gate, extra};
    for (const es_rows* r : rows)
        if (r != nullptr && r->data != nullptr &&
            (reinterpret_cast<uintptr_t>(r->data) % 16 != 0 || (L.B > 1 && r->stride_b % V != 0) || (L.T > 1 && r->stride_t % V != 0)))
            return false;
    return L.G == 1 || (L.C / L.G) % V == 0;
}

inline ScanArgs scan_args(const ScanLaunch& L) {
    ScanArgs A{};
    A.L = L;
    A.per_group = L.C / L.G;
    A.blocks = scan_blocks(L.C, L.G, L.N);
    return A;
}

}  // namespace es
