// k_rotate.cu -- the norm of queries and keys for each head, and the position
// rotation, in one pass over them, forward and backward.
//
//     u = x / sqrt(mean(x^2) + eps),  n = w u,  y = n with pairs of its first
//     `turned` values turned by the angles of the token's position
//
//     backward: z = y's gradient turned back,  dw = sum z u,
//               dx = (w z - u mean(w z u)) / sqrt(mean(x^2) + eps)
//
// Bounded by HBM: each value is read once and written once (backward: two
// read, one written).  A group of G lanes holds a head's row in registers,
// each lane two vectors of 16 bytes that turn into one another (halves) or
// within themselves (neighbours), so the rotation needs no exchange and the
// norm log2 G shuffles.  A warp takes one token and several of its heads, all
// of its loads issued before the first use, and reads the token's cosines and
// sines once for all of them.
#include "es_attn.h"
#include "es_device.cuh"
#include "es_pairs.cuh"

namespace es {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// CTAs an SM.  The forward's warps are many (6 CTAs, two rows a lane) and wait for
// their own loads; the backward's rows take twice the registers, so it has fewer
// warps (3 CTAs, two rows a lane) that fetch the next unit's rows before they work
// on this one's.  Measured, 16384 tokens x 40 heads of 128 bf16: forward 66 us (8
// CTAs 79, 5 CTAs 74, fetching ahead with 4 CTAs 69), backward 113 us (one row and
// 4 CTAs 125, without fetching ahead 165, 2 CTAs 148).
constexpr int resident(bool bwd) { return bwd ? 3 : 6; }

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    return static_cast<float>(v);
}

// VEC values of 16 bytes (or one value), as they lie in memory: rows wait for
// their turn in a quarter of the registers that f32 values would take
template <int VEC>
struct Raw {
    uint4 v;
};
template <>
struct Raw<1> {
    float v;
};

template <typename T, int VEC>
__device__ __forceinline__ void load_raw(const T* p, Raw<VEC>& r) {
    if constexpr (VEC == 1) r.v = to_f32(*p);
    else r.v = *reinterpret_cast<const uint4*>(p);
}

template <int VEC>
__device__ __forceinline__ void clear_raw(Raw<VEC>& r) {
    if constexpr (VEC == 1) r.v = 0.0f;
    else r.v = make_uint4(0, 0, 0, 0);
}

template <typename T, int VEC>
__device__ __forceinline__ void values_of(const Raw<VEC>& r, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] = r.v;
    } else if constexpr (sizeof(T) == 4) {
        f[0] = __uint_as_float(r.v.x);
        f[1] = __uint_as_float(r.v.y);
        f[2] = __uint_as_float(r.v.z);
        f[3] = __uint_as_float(r.v.w);
    } else {
        const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = __uint_as_float(w[e] << 16);
            f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[VEC]) {
    Raw<VEC> r;
    load_raw<T, VEC>(p, r);
    values_of<T, VEC>(r, f);
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        *p = static_cast<T>(f[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int VEC>
__device__ __forceinline__ void load_f32(const float* p, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] = *p;
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            const float4 r = *reinterpret_cast<const float4*>(p + e);
            f[e] = r.x;
            f[e + 1] = r.y;
            f[e + 2] = r.z;
            f[e + 3] = r.w;
        }
    }
}

template <int VEC>
__device__ __forceinline__ void load_weight(const void* w, int bf16, int at, float (&f)[VEC]) {
    if (w == nullptr) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = 1.0f;
    } else if (!bf16) {
        load_f32<VEC>(static_cast<const float*>(w) + at, f);
    } else if constexpr (VEC == 4) {
        const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + at);
        f[0] = __uint_as_float(r.x << 16);
        f[1] = __uint_as_float(r.x & 0xffff0000u);
        f[2] = __uint_as_float(r.y << 16);
        f[3] = __uint_as_float(r.y & 0xffff0000u);
    } else {
        load_vec<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(w) + at, f);
    }
}

struct RotateArgs {
    RotateLaunch L;
    int blocks0;                 // blocks of the queries' side (backward); the keys' follow
    uint32_t units[2];           // work units of each side
    uint32_t per[2];             // units a token
};

// Where item i of a row lies: two vectors at a and b (b < 0: none), turned if
// `pair` >= 0 by the angles from index `pair` on.
template <int VEC>
struct Item {
    int a, b, pair;
};

template <int VEC, bool NEIGH>
__device__ __forceinline__ Item<VEC> item_of(int i, int d, int turned) {
    Item<VEC> it;
    if constexpr (NEIGH) {
        it.a = VEC == 1 ? 2 * i : 2 * i * VEC;
        it.b = it.a + VEC;
        it.pair = it.a < turned ? it.a / 2 : -1;
    } else {
        const int half = turned / 2, nt = half / VEC;
        if (i < nt) {
            it.a = i * VEC;
            it.b = half + i * VEC;
            it.pair = i * VEC;
        } else {
            it.a = turned + 2 * (i - nt) * VEC;
            it.b = it.a + VEC;
            it.pair = -1;
        }
    }
    if (it.b >= d) it.b = -1;
    return it;
}

// The arithmetic on a lane's vectors, two values an instruction.
template <int VEC>
__device__ __forceinline__ float2 two(const float (&a)[VEC], int e) {
    return make_float2(a[e], a[e + 1]);
}

template <int VEC>
__device__ __forceinline__ void put(float (&a)[VEC], int e, float2 v) {
    a[e] = v.x;
    a[e + 1] = v.y;
}

// a *= w
template <int VEC>
__device__ __forceinline__ void times(float (&a)[VEC], const float (&w)[VEC]) {
    if constexpr (VEC == 1) {
        a[0] *= w[0];
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) put(a, e, pair_mul(two(a, e), two(w, e)));
    }
}

// a *= f
template <int VEC>
__device__ __forceinline__ void times(float (&a)[VEC], float f) {
    if constexpr (VEC == 1) {
        a[0] *= f;
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) put(a, e, pair_mul(two(a, e), make_float2(f, f)));
    }
}

// s += a b, the vector's even and odd values apart
template <int VEC>
__device__ __forceinline__ void add_dot(float2& s, const float (&a)[VEC], const float (&b)[VEC]) {
    if constexpr (VEC == 1) {
        s.x = fmaf(a[0], b[0], s.x);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) s = pair_fma(two(a, e), two(b, e), s);
    }
}

// d += a b value by value
template <int VEC>
__device__ __forceinline__ void add_product(float (&d)[VEC], const float (&a)[VEC], const float (&b)[VEC]) {
    if constexpr (VEC == 1) {
        d[0] = fmaf(a[0], b[0], d[0]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) put(d, e, pair_fma(two(a, e), two(b, e), two(d, e)));
    }
}

// a += b f
template <int VEC>
__device__ __forceinline__ void add_scaled(float (&a)[VEC], const float (&b)[VEC], float f) {
    if constexpr (VEC == 1) {
        a[0] = fmaf(b[0], f, a[0]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) put(a, e, pair_fma(two(b, e), make_float2(f, f), two(a, e)));
    }
}

// Turn (a, b) by the angles; the sines of the way back come negated.
template <int VEC, bool NEIGH>
__device__ __forceinline__ void turn(float (&a)[VEC], float (&b)[VEC], const float (&cs)[VEC], const float (&sn)[VEC]) {
    if constexpr (NEIGH && VEC > 1) {
        // cs, sn: the angles of a's pairs, then of b's
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            const float s0 = sn[e], s1 = sn[VEC / 2 + e];
            put(a, 2 * e, pair_fma(make_float2(a[2 * e + 1], a[2 * e]), make_float2(-s0, s0),
                                   pair_mul(two(a, 2 * e), make_float2(cs[e], cs[e]))));
            put(b, 2 * e, pair_fma(make_float2(b[2 * e + 1], b[2 * e]), make_float2(-s1, s1),
                                   pair_mul(two(b, 2 * e), make_float2(cs[VEC / 2 + e], cs[VEC / 2 + e]))));
        }
    } else if constexpr (VEC == 1) {
        const float a0 = a[0];
        a[0] = fmaf(-b[0], sn[0], a0 * cs[0]);
        b[0] = fmaf(a0, sn[0], b[0] * cs[0]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const float2 c = two(cs, e), s = two(sn, e), a0 = two(a, e), b0 = two(b, e);
            put(a, e, pair_fma(make_float2(-b0.x, -b0.y), s, pair_mul(a0, c)));
            put(b, e, pair_fma(a0, s, pair_mul(b0, c)));
        }
    }
}

// G lanes a row, ITEMS items a lane (more than one only without vectors), U
// rows a lane in flight.
template <typename T, int VEC, bool NEIGH, bool BWD, int G, int ITEMS, int U>
__global__ void __launch_bounds__(kThreads, resident(BWD)) k_rotate(const __grid_constant__ RotateArgs A) {
    constexpr int SLOTS = 32 / G;
    constexpr int HB = SLOTS * U;              // heads of a work unit
    const RotateLaunch& L = A.L;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int li = lane % G, slot = lane / G;
    const bool keys = static_cast<int>(blockIdx.x) >= A.blocks0;
    const RotateSide& S = L.side[keys ? 1 : 0];
    const uint32_t blk = keys ? blockIdx.x - A.blocks0 : blockIdx.x;
    const uint32_t nblk = keys ? gridDim.x - A.blocks0 : A.blocks0;
    const uint32_t units = A.units[keys ? 1 : 0], per = A.per[keys ? 1 : 0];
    const int d = L.d, half = L.turned / 2;
    const float inv_d = 1.0f / static_cast<float>(d);

    Item<VEC> it[ITEMS];
    bool on[ITEMS];
    float wa[ITEMS][VEC], wb[ITEMS][VEC];
    float dwa[ITEMS][VEC], dwb[ITEMS][VEC];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        it[i] = item_of<VEC, NEIGH>(li + i * G, d, L.turned);
        on[i] = it[i].a < d;
        if (!on[i]) it[i].a = 0, it[i].b = -1, it[i].pair = -1;
        load_weight<VEC>(S.w, L.w_bf16, it[i].a, wa[i]);
        load_weight<VEC>(S.w, L.w_bf16, it[i].b < 0 ? 0 : it[i].b, wb[i]);
        if constexpr (BWD) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) dwa[i][e] = dwb[i][e] = 0.0f;
        }
    }

    // a unit's rows as they lie in memory, and its position in the tables
    struct Unit {
        Raw<VEC> xa[U][ITEMS], xb[U][ITEMS], ga[BWD ? U : 1][ITEMS], gb[BWD ? U : 1][ITEMS];
        T* out;
        int64_t pos;
        int h0;
    };
    auto fetch = [&](uint32_t unit, Unit& f) {
        const uint32_t bt = unit / per;
        f.h0 = static_cast<int>(unit - bt * per) * HB + slot;
        const uint32_t b = bt / static_cast<uint32_t>(L.T), t = bt - b * static_cast<uint32_t>(L.T);
        // the token's position, clamped into the tables
        int64_t pos = t;
        if (L.positions != nullptr) {
            const int64_t at = b * L.pb + t * L.pt;
            pos = L.pos64 ? static_cast<const int64_t*>(L.positions)[at] : static_cast<const int32_t*>(L.positions)[at];
        }
        const T* x = static_cast<const T*>(S.x) + b * S.xb + t * S.xt;
        const T* gy = BWD ? static_cast<const T*>(S.g) + b * S.gb + t * S.gt : nullptr;
        f.out = static_cast<T*>(S.out) + b * S.ob + t * S.ot;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = f.h0 + u * SLOTS;
            const bool row = h < S.heads;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                clear_raw(f.xa[u][i]);
                clear_raw(f.xb[u][i]);
                if (row && on[i]) {
                    load_raw<T, VEC>(x + h * S.xh + it[i].a, f.xa[u][i]);
                    if (it[i].b >= 0) load_raw<T, VEC>(x + h * S.xh + it[i].b, f.xb[u][i]);
                }
                if constexpr (BWD) {
                    clear_raw(f.ga[u][i]);
                    clear_raw(f.gb[u][i]);
                    if (row && on[i]) {
                        load_raw<T, VEC>(gy + h * S.gh + it[i].a, f.ga[u][i]);
                        if (it[i].b >= 0) load_raw<T, VEC>(gy + h * S.gh + it[i].b, f.gb[u][i]);
                    }
                }
            }
        }
        f.pos = pos;
    };
    const uint32_t step = nblk * kWarps;
    uint32_t unit = blk * kWarps + warp;
    Unit now;
    if (BWD && unit < units) fetch(unit, now);
    for (; unit < units; unit += step) {
        Unit next;
        if constexpr (BWD) {
            if (units - unit > step) fetch(unit + step, next);
        } else {
            fetch(unit, now);
        }
        T* out = now.out;
        const int h0 = now.h0;
        const int64_t pos = now.pos < 0 ? 0 : now.pos < L.rows ? now.pos : L.rows - 1;
        float cs[ITEMS][VEC], sn[ITEMS][VEC];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (it[i].pair >= 0) {
                const float* c = L.cos + pos * half + it[i].pair;
                const float* s = L.sin + pos * half + it[i].pair;
                // neighbours in vectors: a's pairs and b's are VEC / 2 angles each, in a row (b's
                // may lie past the turned values: left as they are)
                if constexpr (NEIGH && VEC > 1) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const bool in = it[i].pair + e < half;
                        cs[i][e] = in ? c[e] : 1.0f;
                        sn[i][e] = in ? s[e] : 0.0f;
                    }
                } else {
                    load_f32<VEC>(c, cs[i]);
                    load_f32<VEC>(s, sn[i]);
                }
                if constexpr (BWD) times(sn[i], -1.0f);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * SLOTS;
            const bool row = h < S.heads;
            float va[ITEMS][VEC], vb[ITEMS][VEC];
            float2 sq2 = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                values_of<T, VEC>(now.xa[u][i], va[i]);
                values_of<T, VEC>(now.xb[u][i], vb[i]);
                add_dot(sq2, va[i], va[i]);
                add_dot(sq2, vb[i], vb[i]);
            }
            float sq = sq2.x + sq2.y;
#pragma unroll
            for (int o = G / 2; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
            const float r = row ? rsqrtf(sq * inv_d + L.eps) : 0.0f;
            if constexpr (!BWD) {
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) {
                    times(va[i], wa[i]);
                    times(vb[i], wb[i]);
                    if (it[i].pair >= 0) turn<VEC, NEIGH>(va[i], vb[i], cs[i], sn[i]);
                    times(va[i], r);
                    times(vb[i], r);
                    if (row && on[i]) {
                        store_vec<T, VEC>(out + h * S.oh + it[i].a, va[i]);
                        if (it[i].b >= 0) store_vec<T, VEC>(out + h * S.oh + it[i].b, vb[i]);
                    }
                }
            } else {
                float2 m2 = make_float2(0.0f, 0.0f);
                float za[ITEMS][VEC], zb[ITEMS][VEC];
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) {
                    values_of<T, VEC>(now.ga[u][i], za[i]);
                    values_of<T, VEC>(now.gb[u][i], zb[i]);
                    if (it[i].pair >= 0) turn<VEC, NEIGH>(za[i], zb[i], cs[i], sn[i]);
                    times(va[i], r);
                    times(vb[i], r);
                    add_product(dwa[i], za[i], va[i]);
                    add_product(dwb[i], zb[i], vb[i]);
                    times(za[i], wa[i]);
                    times(zb[i], wb[i]);
                    add_dot(m2, za[i], va[i]);
                    add_dot(m2, zb[i], vb[i]);
                }
                float m = m2.x + m2.y;
#pragma unroll
                for (int o = G / 2; o; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
                m *= -inv_d;
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) {
                    add_scaled(za[i], va[i], m);
                    add_scaled(zb[i], vb[i], m);
                    times(za[i], r);
                    times(zb[i], r);
                    if (row && on[i]) {
                        store_vec<T, VEC>(out + h * S.oh + it[i].a, za[i]);
                        if (it[i].b >= 0) store_vec<T, VEC>(out + h * S.oh + it[i].b, zb[i]);
                    }
                }
            }
        }
        if constexpr (BWD) now = next;
    }
    if constexpr (BWD) {
        if (S.gw == nullptr) return;           // the same for the whole block
        // the block's sum of each weight's gradient: over the warp's slots by
        // shuffles, then over the warps in order
        __shared__ float s[kWarps][kAttnMaxDim];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float p = dwa[i][e], q = dwb[i][e];
#pragma unroll
                for (int o = 16; o >= G; o >>= 1) {
                    p += __shfl_xor_sync(0xffffffffu, p, o);
                    q += __shfl_xor_sync(0xffffffffu, q, o);
                }
                if (slot == 0 && on[i]) {
                    s[warp][it[i].a + e] = p;
                    if (it[i].b >= 0) s[warp][it[i].b + e] = q;
                }
            }
        __syncthreads();
        for (int c = threadIdx.x; c < d; c += kThreads) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += s[w][c];
            L.partial[static_cast<int64_t>(blockIdx.x) * d + c] = v;
        }
    }
}

// Both weights' gradients from the blocks' sums, in a fixed order: a CTA a
// side and 8 columns, 128 threads a column, so that a column's 456 sums at most
// are four loads a thread.
constexpr int kSumParts = 128;
__global__ void __launch_bounds__(8 * kSumParts) k_rotate_sum(const __grid_constant__ RotateArgs A, int total) {
    const RotateLaunch& L = A.L;
    const int side = blockIdx.y;
    const RotateSide& S = L.side[side];
    if (S.gw == nullptr) return;
    const int lo = side ? A.blocks0 : 0, hi = side ? total : A.blocks0;
    const int col = threadIdx.x % 8, part = threadIdx.x / 8;
    const int c = blockIdx.x * 8 + col;
    __shared__ float s[kSumParts][9];
    float v = 0.0f;
    if (c < L.d)
#pragma unroll 4
        for (int k = lo + part; k < hi; k += kSumParts) v += L.partial[static_cast<int64_t>(k) * L.d + c];
    s[part][col] = v;
#pragma unroll
    for (int n = kSumParts / 2; n; n /= 2) {
        __syncthreads();
        if (part < n) s[part][col] += s[part + n][col];
    }
    if (part == 0 && c < L.d) {
        const float all = s[0][col];
        if (L.w_bf16) static_cast<__nv_bfloat16*>(S.gw)[c] = __float2bfloat16_rn(all);
        else static_cast<float*>(S.gw)[c] = all;
    }
}

// Vectors of 16 bytes serve rows whose halves, strides and addresses keep to
// them; anything else goes value by value.
bool vectors(const RotateLaunch& L) {
    const int vec = L.bf16 ? 8 : 4;
    const int64_t size = L.bf16 ? 2 : 4;
    if (L.d % vec != 0) return false;
    if (L.neighbours ? L.turned % vec != 0 : (L.turned / 2) % vec != 0) return false;
    auto fits = [&](const void* p, int64_t b, int64_t t, int64_t h) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && b * size % 16 == 0 && t * size % 16 == 0 && h * size % 16 == 0;
    };
    for (const RotateSide& S : L.side) {
        if (S.heads == 0) continue;
        if (reinterpret_cast<uintptr_t>(S.w) % 16 != 0) return false;
        if (!fits(S.x, S.xb, S.xt, S.xh) || !fits(S.out, S.ob, S.ot, S.oh)) return false;
        if (L.backward && !fits(S.g, S.gb, S.gt, S.gh)) return false;
    }
    return reinterpret_cast<uintptr_t>(L.cos) % 16 == 0 && reinterpret_cast<uintptr_t>(L.sin) % 16 == 0;
}

// lanes of a row's group: one item a lane with vectors, 32 without
int lanes(const RotateLaunch& L, bool vec) {
    if (!vec) return 32;
    const int n = (L.d / (L.bf16 ? 8 : 4) + 1) / 2;
    int g = 1;
    while (g < n) g *= 2;
    return g;
}

// Blocks of each side: as many as stay resident between them, shared out by
// heads, so that the weights are read once a thread and the backward's sums
// over blocks stay short.
struct Grid {
    int blocks[2];
    int64_t units[2];
    int per[2];
};

constexpr int unroll_of(bool vec) { return vec ? 2 : 1; }

Grid grid_of(const RotateLaunch& L) {
    Grid g{};
    const bool vec = vectors(L);
    const int hb = 32 / lanes(L, vec) * unroll_of(vec);
    int64_t heads = L.side[0].heads + L.side[1].heads;
    for (int s = 0; s < 2; ++s) {
        g.per[s] = (L.side[s].heads + hb - 1) / hb;
        g.units[s] = L.B * L.T * g.per[s];
        int64_t n = (g.units[s] + kWarps - 1) / kWarps;
        int64_t most = static_cast<int64_t>(kSms) * resident(L.backward) * L.side[s].heads / (heads > 0 ? heads : 1);
        if (most < 1) most = 1;
        n = n < most ? n : most;
        g.blocks[s] = static_cast<int>(n);
    }
    return g;
}

template <typename T, int VEC, bool NEIGH, bool BWD, int G, int ITEMS, int U>
cudaError_t go(const RotateArgs& A, int total) {
    k_rotate<T, VEC, NEIGH, BWD, G, ITEMS, U><<<total, kThreads, 0, A.L.stream>>>(A);
    return cudaGetLastError();
}

template <typename T, bool NEIGH, bool BWD>
cudaError_t pick(const RotateArgs& A, int total, bool vec, int g) {
    constexpr int VEC = sizeof(T) == 2 ? 8 : 4;
    constexpr int U = unroll_of(true);
    if (!vec) return go<T, 1, NEIGH, BWD, 32, 4, 1>(A, total);
    switch (g) {
        case 1: return go<T, VEC, NEIGH, BWD, 1, 1, U>(A, total);
        case 2: return go<T, VEC, NEIGH, BWD, 2, 1, U>(A, total);
        case 4: return go<T, VEC, NEIGH, BWD, 4, 1, U>(A, total);
        case 8: return go<T, VEC, NEIGH, BWD, 8, 1, U>(A, total);
        case 16: return go<T, VEC, NEIGH, BWD, 16, 1, U>(A, total);
        default: return go<T, VEC, NEIGH, BWD, 32, 1, U>(A, total);
    }
}

}  // namespace

int rotate_blocks(const RotateLaunch& L, int side) { return grid_of(L).blocks[side]; }

int64_t rotate_units(const RotateLaunch& L, int side) { return grid_of(L).units[side]; }

cudaError_t launch_rotate(const RotateLaunch& L, int* kernels) {
    const Grid g = grid_of(L);
    RotateArgs A{};
    A.L = L;
    A.blocks0 = g.blocks[0];
    for (int s = 0; s < 2; ++s) {
        A.units[s] = static_cast<uint32_t>(g.units[s]);
        A.per[s] = static_cast<uint32_t>(g.per[s]);
    }
    const int total = g.blocks[0] + g.blocks[1];
    const bool vec = vectors(L);
    const int lg = lanes(L, vec);
    *kernels = 1;
    cudaError_t e;
    if (L.bf16) {
        if (L.backward) e = L.neighbours ? pick<__nv_bfloat16, true, true>(A, total, vec, lg) : pick<__nv_bfloat16, false, true>(A, total, vec, lg);
        else e = L.neighbours ? pick<__nv_bfloat16, true, false>(A, total, vec, lg) : pick<__nv_bfloat16, false, false>(A, total, vec, lg);
    } else {
        if (L.backward) e = L.neighbours ? pick<float, true, true>(A, total, vec, lg) : pick<float, false, true>(A, total, vec, lg);
        else e = L.neighbours ? pick<float, true, false>(A, total, vec, lg) : pick<float, false, false>(A, total, vec, lg);
    }
    if (e != cudaSuccess) return e;
    if (L.backward && (L.side[0].gw != nullptr || L.side[1].gw != nullptr)) {
        k_rotate_sum<<<dim3((L.d + 7) / 8, 2), 8 * kSumParts, 0, L.stream>>>(A, total);
        ++*kernels;
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace es
