// es_tcgen05.cuh -- inline-PTX wrappers of the 5th-generation tensor core for
// sm_103a: tensor memory, its loads and stores, matrix products issued by one
// thread, their completion on mbarriers, and the descriptors they take.
#pragma once

#include <cuda_bf16.h>

#include "es_pairs.cuh"
#include "es_ptx.cuh"

namespace es {
namespace tc {

// ---------------------------------------------------------------------------
// tensor memory (128 lanes x 512 columns of 32 bits an SM)

// One warp allocates `cols` columns (a power of two, 32..512); the address is written to shared memory.
__device__ __forceinline__ void alloc(uint32_t* slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void dealloc(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// keeps the uses of loaded values behind the wait before it
template <int N>
__device__ __forceinline__ void loaded(uint32_t (&r)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) asm volatile("" : "+r"(r[e]));
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// N columns of the warp's 32 lanes: lane l of the warp holds its lane's N values
__device__ __forceinline__ void ld(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
}

__device__ __forceinline__ void st(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
                 ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ld(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
                 "%12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
}

__device__ __forceinline__ void st(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
                 "%11, %12, %13, %14, %15};"
                 ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void st(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
                 "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
                 "%29, %30, %31};"
                 ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
                 "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
                 "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
                 : "memory");
}

// Fragments: of 16 lanes (the address names the first), thread t holds lanes
// t / 4 and t / 4 + 8.  ld_pairs: per 8 columns two neighbouring values of each,
// columns 2 (t % 4) and the next; st_words: per 4 columns one of each, column t % 4.
__device__ __forceinline__ void ld_pairs(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void st_words(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
                 : "memory");
}

// Four 8 x 8 blocks of 16-bit values in shared memory, transposed: lane l names
// row l % 8 of block l / 8; thread t holds column t / 4 of rows 2 (t % 4) and the next.
__device__ __forceinline__ void ld_blocks(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void st_blocks(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%4], {%0, %1, %2, %3};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(addr)
                 : "memory");
}

// ---------------------------------------------------------------------------
// products

// Shared-memory operand descriptors, 128-byte swizzle: rows of 64 16-bit values
// in groups of 8 (1024 bytes, `sbo`).  K innermost: sbo is the step between
// groups of 8 rows, `lbo` unused.  Rows innermost (a transposed operand): sbo is
// the step between groups of 8 along K, lbo between panels of 64 rows.

// Instruction descriptor of bf16 operands with f32 sums, M = 128.
__host__ __device__ constexpr uint32_t instr_bf16(uint32_t n, bool a_rows_inner, bool b_rows_inner) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(a_rows_inner) << 15) |
           (static_cast<uint32_t>(b_rows_inner) << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// The products and commits below are run by the whole warp and done by one
// thread of it (`lead`): without a branch around them their operands stay in
// uniform registers, which they are read from; inside one, each operand is
// moved there first, and issuing takes longer than the product.

// one thread of the (whole) warp
__device__ __forceinline__ uint32_t elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

// Shared-memory descriptors differ in their low words only, which the callers
// count up; the high word holds `sbo` and the kind.
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) {
    return ((addr >> 4) & 0x3fffu) | (((lbo >> 4) & 0x3fffu) << 16);
}
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);     // sbo 1024, 128-byte swizzle

// d = a b (first) or d += a b, 16 along K; both operands in shared memory
template <bool kFirst = false>
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t instr) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(instr), "n"(kFirst ? 0 : 1), "r"(lead), "r"(kDescHigh)
        : "memory");
}

// the same with a in tensor memory (a row a lane, two bf16 a column)
template <bool kFirst = false>
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t instr) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(instr), "n"(kFirst ? 0 : 1), "r"(lead), "r"(kDescHigh)
        : "memory");
}

// arrive on `bar` once every product issued by that thread so far is done
__device__ __forceinline__ void commit(uint32_t lead, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(lead)
        : "memory");
}

// ---------------------------------------------------------------------------
// bf16 terms of f32 values

// two values rounded to bf16, the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float low_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// v less its own rounding `hi` to bf16, exact
__device__ __forceinline__ float2 rest_of(float2 v, uint32_t hi) {
    return pair_fma(make_float2(low_bf16(hi), high_bf16(hi)), make_float2(-1.0f, -1.0f), v);
}

// The next bf16 term of a pair of values, which keeps what is left of them.
// Rounded to nearest (2^-8 of the value is left at most) or cut off (2^-7): the
// conversion runs at a quarter of the rate of the byte permute that cuts.
template <bool kCut>
__device__ __forceinline__ uint32_t take_term(float2& v) {
    uint32_t t;
    if constexpr (kCut) {
        asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(t) : "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)));
        v = pair_fma(make_float2(high_bf16(__float_as_uint(v.x)), high_bf16(__float_as_uint(v.y))), make_float2(-1.0f, -1.0f), v);
    } else {
        t = pack_bf16(v.x, v.y);
        v = rest_of(v, t);
    }
    return t;
}

// the first two bf16 terms of a pair of values: 2^-17 of them is left at most, cut off 2^-16
template <bool kCut>
__device__ __forceinline__ void split2(float2 v, uint32_t& hi, uint32_t& lo) {
    hi = take_term<kCut>(v);
    lo = pack_bf16(v.x, v.y);
}

__device__ __forceinline__ float exp2_approx(float v) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

}  // namespace tc
}  // namespace es
