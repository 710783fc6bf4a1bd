// es_ssm.cuh -- device helpers of the state-space layer's kernels: element
// types, exponentials, the logistic function and log(1 + e^x), copies into
// shared memory.
#pragma once

#include <cuda_bf16.h>

#include "es_pairs.cuh"

namespace es {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLog2eLow = 1.92596299112661746887e-8f;      // log2(e) - kLog2e
constexpr float kLn2 = 0.69314718055994530942f;

// The hardware's 2^x (relative error below 2^-22; results under 2^-126 are 0).
__device__ __forceinline__ float exp2_hw(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_hw(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float2 pair_of(float v) { return make_float2(v, v); }

// e^-m (0 past 87).  EXACT, for m from -88.5 to 104: what m log2(e) loses in its
// rounding, |m| 2^-24 of the result, goes back in to first order; results rounded to
// bf16 go without.
template <bool EXACT>
__device__ __forceinline__ float2 pair_exp_minus(float2 m) {
    const float2 t = pair_mul(m, pair_of(-kLog2e));
    const float2 e = make_float2(exp2_hw(t.x), exp2_hw(t.y));
    if constexpr (!EXACT) return e;
    const float2 lost = pair_fma(m, pair_of(kLog2eLow), pair_fma(m, pair_of(kLog2e), t));
    return pair_fma(e, pair_mul(lost, pair_of(-kLn2)), e);
}

// 1 / (1 + e^-z), for any z: 0 below -88, where it would be subnormal, and 1 far above
// 0, so that z times it is 0 for the lowest finite values too.  The exponent's
// correction needs a finite power and product, hence EXACT's bounds (e^88.5 = 2.7e38,
// whose reciprocal the hardware flushes to 0).
template <bool EXACT>
__device__ __forceinline__ float2 pair_logistic(float2 z) {
    if constexpr (EXACT) z = make_float2(fminf(fmaxf(z.x, -88.5f), 104.0f), fminf(fmaxf(z.y, -88.5f), 104.0f));
    const float2 d = pair_add(pair_exp_minus<EXACT>(z), pair_of(1.0f));
    return make_float2(rcp_hw(d.x), rcp_hw(d.y));
}
__device__ __forceinline__ float logistic(float z) { return pair_logistic<true>(pair_of(z)).x; }

// max(v, 0), or NaN for a NaN
__device__ __forceinline__ float above_zero(float v) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
    return r;
}

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x| in [0, 1], 0 for x = -inf.
// log(1 + e) / e is a polynomial of degree 9, fitted for the least relative error on [0, 1]
// (5e-9; 1.3e-7 as evaluated in f32), so small results keep their bits.  A NaN stays one
// through the first term.
__device__ __forceinline__ float2 pair_softplus(float2 x) {
    const float2 e = pair_exp_minus<true>(make_float2(fminf(fabsf(x.x), 104.0f), fminf(fabsf(x.y), 104.0f)));
    float2 p = pair_fma(e, pair_of(-0.003244024235755205f), pair_of(0.019851457327604294f));
    p = pair_fma(p, e, pair_of(-0.056959524750709534f));
    p = pair_fma(p, e, pair_of(0.10603653639554977f));
    p = pair_fma(p, e, pair_of(-0.15305592119693756f));
    p = pair_fma(p, e, pair_of(0.1967593878507614f));
    p = pair_fma(p, e, pair_of(-0.24954134225845337f));
    p = pair_fma(p, e, pair_of(0.3332996368408203f));
    p = pair_fma(p, e, pair_of(-0.4999990165233612f));
    p = pair_fma(p, e, pair_of(1.0f));
    return pair_fma(p, e, make_float2(above_zero(x.x), above_zero(x.y)));
}
__device__ __forceinline__ float softplus(float x) { return pair_softplus(pair_of(x)).x; }

// two neighbouring values in shared memory
__device__ __forceinline__ float2 load_two(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 load_two(const __nv_bfloat16* p) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}
__device__ __forceinline__ void store_two(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
__device__ __forceinline__ void store_two(__nv_bfloat16* p, float2 v) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}

// V neighbouring values in one access
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

// as pairs (one half for V = 1), from what a load left in registers
template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V>& q, float2 (&r)[(V + 1) / 2]) {
    if constexpr (V == 1) {
        r[0] = make_float2(to_f32(q.v[0]), 0.0f);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) r[i] = make_float2(to_f32(q.v[2 * i]), to_f32(q.v[2 * i + 1]));
    }
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> pack(const float2 (&r)[(V + 1) / 2]) {
    Pack<T, V> q;
    if constexpr (V == 1) {
        q.v[0] = from_f32<T>(r[0].x);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) store_two(&q.v[2 * i], r[i]);
    }
    return q;
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_raw(const T* p) {
    return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <int P>
__device__ __forceinline__ void zero(float2 (&r)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) r[i] = make_float2(0.0f, 0.0f);
}

// a weight of either type
__device__ __forceinline__ float weight_at(const void* w, int bf16, int64_t i) {
    return bf16 ? to_f32(static_cast<const __nv_bfloat16*>(w)[i]) : static_cast<const float*>(w)[i];
}

// 16 bytes into shared memory; the bytes past `n` (0..16) are zeros and not read.
__device__ __forceinline__ void copy16(void* to, const void* from, int n) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(a), "l"(from), "r"(n) : "memory");
}
// BYTES (4, 8 or 16) into shared memory, to be waited for; fewer at once
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(a), "l"(from) : "memory");
    else if constexpr (BYTES >= 4) asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(a), "l"(from), "n"(BYTES) : "memory");
    else *static_cast<uint16_t*>(to) = *static_cast<const uint16_t*>(from);
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all groups but the LEFT last ones are there (0: every copy, in a group or not)
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    if constexpr (LEFT == 0) asm volatile("cp.async.wait_all;" ::: "memory");
    else asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// a row's tokens that count
__device__ __forceinline__ int64_t live_tokens(const int32_t* lengths, int64_t b, int64_t T) {
    if (lengths == nullptr) return T;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n < T ? n : T;
}

// Sums of the rows of a [rows][M] table, put(j, sum) for each column: a block takes
// 32 columns, its 8 warps every eighth row, always in one order.
constexpr int kSumLanes = 8;
template <typename Put>
__global__ void __launch_bounds__(32 * kSumLanes) k_sum_rows(const float* __restrict__ p, int64_t rows, int64_t M, const Put put) {
    __shared__ float part[kSumLanes][32];
    const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float s = 0.0f;
    if (j < M) {
        float t[4] = {0.f, 0.f, 0.f, 0.f};
        int64_t r = threadIdx.y;
        for (; r + 3 * kSumLanes < rows; r += 4 * kSumLanes)
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] += p[(r + i * kSumLanes) * M + j];
        for (; r < rows; r += kSumLanes) t[0] += p[r * M + j];
        s = (t[0] + t[1]) + (t[2] + t[3]);
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && j < M) {
#pragma unroll
        for (int i = 1; i < kSumLanes; ++i) s += part[i][threadIdx.x];
        put(j, s);
    }
}
template <typename Put>
cudaError_t sum_rows(const float* p, int64_t rows, int64_t M, const Put& put, cudaStream_t stream) {
    k_sum_rows<<<static_cast<unsigned>((M + 31) / 32), dim3(32, kSumLanes), 0, stream>>>(p, rows, M, put);
    return cudaGetLastError();
}

__device__ __forceinline__ void put_weight(void* w, int bf16, int64_t i, float v) {
    if (w == nullptr) return;
    if (bf16) static_cast<__nv_bfloat16*>(w)[i] = from_f32<__nv_bfloat16>(v);
    else static_cast<float*>(w)[i] = v;
}

}  // namespace es
