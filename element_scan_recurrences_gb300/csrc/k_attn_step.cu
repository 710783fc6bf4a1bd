// k_attn_step.cu -- one token of linear attention:
//
//     state_out = e^g state + k v^T,   out = scale * q state_out
//
// for every (batch row, head), the state f32 [dk, dv].  Bounded by the states'
// bytes: each is read and written once, 8 dk dv bytes a head, and the token's
// own operands are under a hundredth of that.  A CTA takes a slice of the
// value columns of one head; each thread holds VEC neighbouring columns and
// every kRows-th row, its loads all issued before the first use; the products
// with q are summed over the rows in registers, then over the CTA through
// shared memory.
#include "es_attn.h"
#include "es_device.cuh"

namespace es {
namespace {

constexpr int kThreads = 128;

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    return static_cast<float>(v);
}

template <int VEC>
struct Pack {
    float v[VEC];
};

template <int VEC>
__device__ __forceinline__ Pack<VEC> load_pack(const float* p) {
    Pack<VEC> r;
    if constexpr (VEC == 4) {
        const float4 f = *reinterpret_cast<const float4*>(p);
        r.v[0] = f.x;
        r.v[1] = f.y;
        r.v[2] = f.z;
        r.v[3] = f.w;
    } else {
        r.v[0] = *p;
    }
    return r;
}

template <int VEC>
__device__ __forceinline__ void store_pack(float* p, const Pack<VEC>& r) {
    if constexpr (VEC == 4) *reinterpret_cast<float4*>(p) = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
    else *p = r.v[0];
}

// COLS threads across a row (COLS * VEC columns a CTA), kThreads / COLS rows a pass
template <typename T, int VEC, int COLS>
__global__ void __launch_bounds__(kThreads) k_attn_step(const __grid_constant__ AttnStep S) {
    constexpr int ROWS = kThreads / COLS;
    constexpr int U = 8;                       // rows in flight a thread
    __shared__ float sq[kAttnMaxDim], sk[kAttnMaxDim];
    __shared__ float part[ROWS][COLS * VEC + 1];
    const int64_t bh = blockIdx.x;
    const int64_t b = bh / S.H;
    const int h = static_cast<int>(bh % S.H);
    const int col = threadIdx.x % COLS, row = threadIdx.x / COLS;
    const int c0 = blockIdx.y * (COLS * VEC) + col * VEC;
    const bool live = c0 < S.dv;
    const float* st = S.state + bh * S.dk * static_cast<int64_t>(S.dv) + c0;
    float* so = S.state_out + bh * S.dk * static_cast<int64_t>(S.dv) + c0;
    const T* q = static_cast<const T*>(S.q.p) + b * S.q.sb + (h / S.q.div) * S.q.sh;
    const T* k = static_cast<const T*>(S.k.p) + b * S.k.sb + (h / S.k.div) * S.k.sh;
    const T* v = static_cast<const T*>(S.v.p) + b * S.v.sb + (h / S.v.div) * S.v.sh + c0;

    Pack<VEC> s[U];
    // the first rows' loads go out before anything waits
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int a = row + u * ROWS;
        if (live && a < S.dk) s[u] = load_pack<VEC>(st + static_cast<int64_t>(a) * S.dv);
    }
    const float g = S.g != nullptr ? S.g[b * S.gb + h * S.gh] : 0.0f;
    float vv[VEC], acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        vv[e] = live ? to_f32(v[e]) : 0.0f;
        acc[e] = 0.0f;
    }
    for (int a = threadIdx.x; a < S.dk; a += kThreads) {
        sq[a] = to_f32(q[a]);
        sk[a] = to_f32(k[a]);
    }
    const bool cut = g < -104.0f;              // e^g is zero in f32: whatever the state held is dropped
    const float decay = cut ? 0.0f : expf(g);
    __syncthreads();
    for (int a0 = row; a0 < S.dk; a0 += U * ROWS) {
        if (a0 != row) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int a = a0 + u * ROWS;
                if (live && a < S.dk) s[u] = load_pack<VEC>(st + static_cast<int64_t>(a) * S.dv);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int a = a0 + u * ROWS;
            if (live && a < S.dk) {
                const float ka = sk[a], qa = sq[a];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    s[u].v[e] = fmaf(ka, vv[e], cut ? 0.0f : decay * s[u].v[e]);
                    acc[e] = fmaf(qa, s[u].v[e], acc[e]);
                }
                store_pack<VEC>(so + static_cast<int64_t>(a) * S.dv, s[u]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) part[row][col * VEC + e] = acc[e];
    __syncthreads();
    const int c = blockIdx.y * (COLS * VEC) + threadIdx.x;
    if (threadIdx.x < COLS * VEC && c < S.dv) {
        float o = 0.0f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) o += part[r][threadIdx.x];
        static_cast<T*>(S.out)[b * S.ob + h * S.oh + c] = static_cast<T>(o * S.scale);
    }
}

template <typename T>
cudaError_t launch(const AttnStep& S) {
    const bool vec = S.dv % 4 == 0 && reinterpret_cast<uintptr_t>(S.state) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(S.state_out) % 16 == 0;
    const int64_t BH = S.B * S.H;
    if (vec)
        k_attn_step<T, 4, 8><<<dim3(static_cast<unsigned>(BH), (S.dv + 31) / 32), kThreads, 0, S.stream>>>(S);
    else
        k_attn_step<T, 1, 32><<<dim3(static_cast<unsigned>(BH), (S.dv + 31) / 32), kThreads, 0, S.stream>>>(S);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_step(const AttnStep& S) { return S.bf16 ? launch<__nv_bfloat16>(S) : launch<float>(S); }

}  // namespace es
