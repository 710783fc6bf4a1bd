// k_attn_tc.cu -- linear attention in chunks of 64 tokens on the tensor cores.
//
// One CTA takes one (batch row, head), or a segment of its tokens, through the
// chunks in order; its 32 warps are a pipeline of roles linked by mbarriers:
//
//     warp 2       TMA loads of the operands' tiles (X, Y, Z, and W for the
//                  decays' gradient), 128-byte swizzled panels of 64 values
//     warp 7       the chunk's decays (G, the coefficients of read and update);
//                  hands a loaded stage on, after clearing the rows of Y and Z
//                  past the length in a row's last, ragged chunk
//     warps 3, 6   issue the products (tcgen05.mma, one thread each): the
//                  scores' and the state's
//     warps 0,1,4,5  scores -> P: mask and decay, split into bf16 terms, to
//                  shared memory
//     warps 8-15   Z scaled by its update coefficients and transposed into
//                  tensor memory, two or three bf16 terms
//     warps 16-23  the state: f32 in tensor memory, decayed once a chunk, and
//                  its two bf16 terms for the read
//     warps 24-31  the outputs: read, joined, rounded once, stored
//
// The state lies transposed, a value column a lane and a key column a column,
// so that everything made from it or for it is the A operand, read from tensor
// memory, and X, Y and Z are used where TMA put them:
//
//     S[i, j]    = X Y^T              both K innermost; 128 rows asked of which
//                                     the chunk's 64 are used
//     H^T[c, a] += Z'^T Y             A = the scaled Z (tensor memory), B = Y
//                                     rows innermost
//     O2^T[c, i] = H^T X^T            A = the state's terms, B = X
//     O1^T[c, i] = Z^T P^T            A = Z rows innermost, B = P
//     out_i      = scale O1_i + read_i O2_i      (the scale of O2 in read)
//
// Precision: bf16 operands go in as they are.  Every f32 factor is split into
// bf16 terms that are multiplied in turn and summed in f32: P and the state as
// read in two (2^-16 of each factor, below the result's own rounding; 2^-17
// with the decays' gradient, which takes differences of these results that one
// term would spoil), Z' in three where the state is an f32 result (all of its
// 24 bits), else in two.
//
// Every wait is bounded: a role that gives up sets the status word and the
// abort flag, all roles leave their loops, copies and products in flight are
// waited for (bounded too), and tensor memory is freed.
#include "es_attn.h"
#include "es_device.cuh"
#include "es_segments.h"
#include "es_tcgen05.cuh"

namespace es {
namespace {

constexpr int C = kAttnTcChunk;               // 64 tokens
constexpr int kThreads = 1024;
constexpr int kAnchorChunks = kAttnAnchorTokens / C;
constexpr int kMaxStages = 4;
constexpr uint32_t kPanel = C * 128;          // bytes of a panel: 64 rows of 64 bf16
constexpr uint32_t kTmemCols = 512;

struct alignas(16) Coef {
    float g2[C];                              // inclusive sums of the log decays, base 2
    float low[C];                             // what they lost to rounding
    float read[C], upd[C];
    int bound[C];                             // forward: the first token row i sees; reversed: the last
    float decay;
    int wide;                                 // the sums are so large that what they lost counts
    float pad[2];
};

// Half of an ulp of a sum below 32 is 2^-20, and a weight is off by a few of them: less
// than the 2^-16 to which P is kept.  Above (half of the tokens at -100: 2^-12) the
// weights take the sums' second floats too.  With the decays' gradient only there
// (8 x 4096 x 16 x 128 both ways 762 us, for every chunk 769); without it for every
// chunk, which is the faster way round by the code it leaves (65536 tokens x 16 heads of
// 128 384 us, 391 with a branch).
constexpr float kWideSum = 32.0f;

struct TcRun {
    CUtensorMap x, y, z, w;
    void* out;
    int64_t ob, ot, oh;
    const float* init;
    float* fin;
    int64_t sa, sc;
    float update_scale, read_scale, out_scale;
    float* dots;
    float* anchors;
    int xdiv, ydiv, zdiv, wdiv;
    int xb, yb, zb, wb;                       // 1; 0: one batch row for all
    int dx, dz;                               // real widths
    int reverse, out_f32;
    int terms;                                // bf16 terms of the scaled Z: 3 where the state can be a result, else 2
    int wide;                                 // the result's addresses and strides keep to 16 bytes
};

struct TcArgs {
    TcRun run[3];
    int64_t T, BH;
    int H;
    int n_segs, seg_chunks;
    const float* g;
    int64_t gb, gt, gh;
    const int* lengths;
    int64_t n_anchors;
    float* seg_states;                        // [runs][BH][n_segs][dx * dz] states entering each segment's successor
    float* seg_decays;                        // [runs][BH][n_segs]
    int64_t seg_stride;                       // floats of one run's seg_states
    unsigned int* status;
    uint64_t wait_ns;
    int64_t drop_tile;
    int stages;
    uint32_t stage_bytes;
};

struct Shared {
    uint64_t full[kMaxStages], ready[kMaxStages], empty[kMaxStages];
    uint64_t s_done, p_ready, zh_ready[2], kv_done, state_done, o_done, o_read, drained[2];
    uint32_t tmem;
    int abort_flag;
    Coef coef[kMaxStages];
};

// A bounded wait that lets the hardware hold the thread, up to 20 us a try: a
// try without that hint comes back after some tens of cycles.  The clock and
// the abort flag are looked at after every 64 tries; what runs in between is
// kept short, for the roles' loops together have to stay in the instruction
// caches.
__device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag) {
    const uint32_t at = smem_u32(bar);
    uint64_t t0 = 0;
#pragma unroll 1
    while (true) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .u32 n;\n\tmov.u32 n, 64;\n"
            "TRY:\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "@p bra DONE;\n\t"
            "sub.u32 n, n, 1;\n\t"
            "setp.ne.u32 p, n, 0;\n\t"
            "@p bra TRY;\n\t"
            "setp.ne.u32 p, n, 0;\n"
            "DONE:\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(at), "r"(parity), "r"(20000u)
            : "memory");
        if (done) return true;
        if (abort_flag != nullptr && *abort_flag) return false;
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > limit_ns) return false;
    }
}

// A place in a ring of stages and the parity of its current round.
struct Ring {
    int s = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int n) {
        if (++s == n) {
            s = 0;
            parity ^= 1;
        }
    }
};

// one thread's wait
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag) {
    return mbar_try_wait(bar, parity) || wait_more(bar, parity, limit_ns, abort_flag);
}

// The whole warp's wait when its first try found the barrier not yet due.
__device__ __noinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag,
                                       unsigned int* status) {
    const bool ok = wait_more(bar, parity, limit_ns, abort_flag);
    if (__all_sync(0xffffffffu, ok)) return true;
    if (!ok && !*abort_flag) report_timeout(status, abort_flag);
    return false;
}

struct Wait {
    uint64_t ns;
    volatile int* flag;
    unsigned int* status;
    // the whole warp waits; false: leave the loop
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1))) return true;
        return wait_warp(bar, parity & 1, ns, flag, status);
    }
};

__device__ __forceinline__ void arrive_warp(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// Columns [lo, hi) of the warp's lanes of the state to `to` (one value column;
// null: none) and on every `stride` floats.
__device__ __noinline__ void state_out(uint32_t state, int lo, int hi, float* to, int64_t stride) {
#pragma unroll 1
    for (int a0 = lo; a0 < hi; a0 += 8) {
        uint32_t r[8];
        tc::ld(state + a0, r);
        tc::wait_ld();
        tc::loaded(r);
        if (to != nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) to[(a0 + e) * stride] = __uint_as_float(r[e]);
        }
    }
}

// kStateOnly: a segment's own state and decay, from zero: only Y and Z are read.
// It goes through the segment backwards, with the decays from each chunk to the
// segment's end in Z's coefficients, so the state is a plain sum and no role has
// to look at it on the way (65536 tokens x 16 heads of 128: 153 -> 113 us).
template <bool kStateOnly, bool kDots>
__global__ void __launch_bounds__(kThreads, 1) k_attn_tc(const __grid_constant__ TcArgs A) {
    extern __shared__ __align__(1024) unsigned char raw[];
    __shared__ Shared sh;
    unsigned char* tiles = raw + smem_align_pad(raw);
    const TcRun& R = A.run[blockIdx.y];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t bh = blockIdx.x / A.n_segs;
    const int seg = static_cast<int>(blockIdx.x % A.n_segs);
    const int b = static_cast<int>(bh / A.H), h = static_cast<int>(bh % A.H);
    int64_t len = A.T;
    if (A.lengths != nullptr) {
        const int64_t l = A.lengths[b];
        len = l < 0 ? 0 : l < A.T ? l : A.T;
    }
    // the segment's chunks [c0, c1) and whether they begin or end the run
    const int chunks = static_cast<int>((len + C - 1) / C);
    const SegmentPart part = segment_part(seg, A.n_segs, A.seg_chunks, chunks, R.reverse != 0);
    const int c0 = part.c0, c1 = part.c1, n = max(0, c1 - c0);
    if constexpr (kStateOnly) {
        if (seg > part.last) return;
        if (part.ends) {
            // No successor: its place keeps the initial state, which the main pass may find overwritten
            // (the last state may take its place) before its first segment reads it.
            if (R.init != nullptr) {
                const int64_t size = static_cast<int64_t>(R.dx) * R.dz;
                float* to = A.seg_states + blockIdx.y * A.seg_stride + (bh * A.n_segs + seg) * size;
                for (int64_t e = threadIdx.x; e < size; e += kThreads)
                    to[e] = R.init[bh * size + e / R.dz * R.sa + e % R.dz * R.sc];
            }
            return;
        }
    }
    const int dxp = (R.dx + 63) & ~63, dzp = (R.dz + 63) & ~63;
    const int px = dxp / 64, pz = dzp / 64;
    const bool dots = kDots && R.dots != nullptr;
    // (the decays' gradient takes differences of the results: its terms are rounded to nearest)
    constexpr bool kCut = !kDots;

    // a stage: X, Y, Z, and W's place, which is then the output tile's
    const uint32_t off_y = kStateOnly ? 0 : px * kPanel, off_z = off_y + px * kPanel, off_w = off_z + pz * kPanel;
    unsigned char* p_hi = tiles + A.stages * A.stage_bytes;
    unsigned char* p_lo = p_hi + kPanel;

    if (warp == 2) tc::alloc(&sh.tmem, kTmemCols);
    if (threadIdx.x == 0) {
        for (int s = 0; s < A.stages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.ready[s], 1);
            mbar_init(&sh.empty[s], 1 + 8 + (kStateOnly ? 0 : 8 + 1 + 4 + 8));   // products, Z; state, products, P, outputs
        }
        mbar_init(&sh.s_done, 1);
        mbar_init(&sh.p_ready, 4);
        mbar_init(&sh.zh_ready[0], kStateOnly ? 8 : 8 + 8);
        mbar_init(&sh.zh_ready[1], 8);
        mbar_init(&sh.kv_done, 1);
        mbar_init(&sh.state_done, 1);
        mbar_init(&sh.o_done, 2);                                    // O1, O2
        mbar_init(&sh.o_read, 8);
        mbar_init(&sh.drained[0], 1);
        mbar_init(&sh.drained[1], 1);
        sh.abort_flag = 0;
        mbar_fence_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    // all of the SM's tensor memory is this CTA's, so its address is 0
    constexpr uint32_t tmem = 0;
    const uint32_t t_h = tmem, t_hb = t_h + dxp, t_zt = t_hb + dxp, t_s = t_zt + C, t_o1 = t_s + C, t_o2 = t_o1 + C;
    const Wait wait{A.wait_ns, &sh.abort_flag, A.status};
    // Z's terms, the barrier that says they are there and the one of the state's products: a segment's own state has room
    // for two chunks' terms (in the place of the state's), which take turns.  So do their barriers: a warp may be one chunk
    // ahead of another (those past the value columns have nothing to do), and its arrival must not count for the other's.
    auto zt_of = [&](int k) { return kStateOnly ? t_hb + (k & 1) * C : t_zt; };
    auto zh_of = [&](int k) { return &sh.zh_ready[kStateOnly ? k & 1 : 0]; };
    auto kv_of = [&](int k) { return kStateOnly && (k & 1) ? &sh.s_done : &sh.kv_done; };
    auto chunk_of = [&](int k) { return (R.reverse != 0) != kStateOnly ? c1 - 1 - k : c0 + k; };

    if (warp == 2) {
        // ---- loads
        if (lane == 0) {
            if constexpr (!kStateOnly) tma_prefetch_desc(&R.x);
            tma_prefetch_desc(&R.y);
            tma_prefetch_desc(&R.z);
            const uint64_t pol = l2_policy_stream();
            const int hx = h / R.xdiv, hy = h / R.ydiv, hz = h / R.zdiv, hw = h / R.wdiv;
            const int bx = b * R.xb, by = b * R.yb, bz = b * R.zb, bw = b * R.wb;
            const uint32_t bytes = ((kStateOnly ? px : 2 * px) + (dots ? 2 * pz : pz)) * kPanel;
            int issued = 0;
            Ring ring;
#pragma unroll 1
            for (int k = 0; k < n; ++k, ring.next(A.stages)) {
                uint64_t* full = &sh.full[ring.s];
                if (k >= A.stages && !wait_bounded(&sh.empty[ring.s], ring.parity ^ 1, A.wait_ns, &sh.abort_flag)) {
                    report_timeout(A.status, &sh.abort_flag);
                    break;
                }
                issued = k + 1;
                if (k == A.drop_tile) continue;      // testing hook: this tile never arrives
                unsigned char* st = tiles + ring.s * A.stage_bytes;
                const int t0 = chunk_of(k) * C;
                mbar_arrive_expect_tx(full, bytes);
#pragma unroll 1
                for (int p = 0; p < px; ++p) {
                    if constexpr (!kStateOnly) tma_load_4d(st + p * kPanel, &R.x, p * 64, hx, t0, bx, full, pol);
                    tma_load_4d(st + off_y + p * kPanel, &R.y, p * 64, hy, t0, by, full, pol);
                }
#pragma unroll 1
                for (int p = 0; p < pz; ++p) {
                    tma_load_4d(st + off_z + p * kPanel, &R.z, p * 64, hz, t0, bz, full, pol);
                    if (dots) tma_load_4d(st + off_w + p * kPanel, &R.w, p * 64, hw, t0, bw, full, pol);
                }
            }
#pragma unroll 1
            for (int k = max(0, issued - A.stages); k < issued; ++k) {
                if (k == A.drop_tile) continue;
                if (!wait_bounded(&sh.full[k % A.stages], (k / A.stages) & 1, A.wait_ns, nullptr))
                    atomicOr(A.status, ES_DEVICE_TIMEOUT);
            }
        }
        __syncwarp();
    } else if (warp == 7) {
        // ---- the chunks' decays, tokens 2 lane and 2 lane + 1; then the stage is handed on
        const float* G = A.g != nullptr ? A.g + b * A.gb + h * A.gh : nullptr;
        auto load = [&](int k) {
            float2 g = make_float2(0.0f, 0.0f);
            if (G == nullptr || k >= n) return g;
            const int64_t t = static_cast<int64_t>(chunk_of(k)) * C + 2 * lane;
            if (t < len) g.x = __ldg(G + t * A.gt);
            if (t + 1 < len) g.y = __ldg(G + (t + 1) * A.gt);
            return g;
        };
        float2 g = load(0);
        float all = 1.0f;
        Ring ring;
#pragma unroll 1
        for (int k = 0; k < n; ++k, ring.next(A.stages)) {
            const float2 next = load(k + 1);
            const bool cut0 = g.x < -104.0f, cut1 = g.y < -104.0f;
            const float v0 = cut0 ? 0.0f : g.x * 1.4426950408889634f, v1 = cut1 ? 0.0f : g.y * 1.4426950408889634f;
            // inclusive sums of the pairs before (and what they lose), exclusive sums of the pairs after
            float lost;
            float pre = two_sum(v0, v1, lost), low = lost, suf = pre;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float p = __shfl_up_sync(0xffffffffu, pre, o), pl = __shfl_up_sync(0xffffffffu, low, o);
                const float q = __shfl_down_sync(0xffffffffu, suf, o);
                if (lane >= o) {
                    if constexpr (kStateOnly) {
                        pre += p;
                    } else {
                        pre = two_sum(pre, p, lost);
                        low += pl + lost;
                    }
                }
                if (lane + o < 32) suf += q;
            }
            const float whole = __shfl_sync(0xffffffffu, pre, 31);
            float before = __shfl_up_sync(0xffffffffu, pre, 1), after = __shfl_down_sync(0xffffffffu, suf, 1);
            float before_low = __shfl_up_sync(0xffffffffu, low, 1);
            if (lane == 0) before = before_low = 0.0f;
            if (lane == 31) after = 0.0f;
            const float2 g2 = make_float2(two_sum(before, v0, lost), pre);
            const float2 g2_low = make_float2(before_low + lost, low);
            float2 from_start = make_float2(tc::exp2_approx(g2.x), tc::exp2_approx(g2.y));
            float2 to_end = make_float2(tc::exp2_approx(after + v1), tc::exp2_approx(after));
            float decay = tc::exp2_approx(whole);
            int2 bound = R.reverse ? make_int2(63, 63) : make_int2(0, 0);
            if (__any_sync(0xffffffffu, cut0 || cut1)) {
                // some token starts afresh: coefficients that reach across it are zero, and rows end there
                const unsigned m0 = __ballot_sync(0xffffffffu, cut0), m1 = __ballot_sync(0xffffffffu, cut1);
                const unsigned upto = 0xffffffffu >> (31 - lane), below = upto >> 1, above = ~upto;
                // the last cut at or before each token, the first one after it
                auto last = [](unsigned even, unsigned odd) {
                    return max(even ? 2 * (31 - __clz(even)) : -1, odd ? 2 * (31 - __clz(odd)) + 1 : -1);
                };
                auto first = [](unsigned even, unsigned odd) {
                    return min(even ? 2 * (__ffs(even) - 1) : 64, odd ? 2 * (__ffs(odd) - 1) + 1 : 64);
                };
                const int l0 = last(m0 & upto, m1 & below), l1 = last(m0 & upto, m1 & upto);
                const int f0 = first(m0 & above, m1 & ~below), f1 = first(m0 & above, m1 & above);
                if (l0 >= 0) from_start.x = 0.0f;
                if (l1 >= 0) from_start.y = 0.0f;
                if (f0 < 64) to_end.x = 0.0f;
                if (f1 < 64) to_end.y = 0.0f;
                bound = R.reverse ? make_int2(f0 - 1, f1 - 1) : make_int2(max(l0, 0), max(l1, 0));
                decay = 0.0f;
            }
            if constexpr (kStateOnly) {
                // on to the segment's end
                from_start.x *= all;
                from_start.y *= all;
                to_end.x *= all;
                to_end.y *= all;
            }
            all *= decay;
            if (k >= A.stages && !wait(&sh.empty[ring.s], ring.parity ^ 1)) break;
            Coef& c = sh.coef[ring.s];
            if constexpr (!kStateOnly) {
                *reinterpret_cast<float2*>(&c.g2[2 * lane]) = g2;
                *reinterpret_cast<float2*>(&c.low[2 * lane]) = g2_low;
            }
            const float2 read = R.reverse ? to_end : from_start, upd = R.reverse ? from_start : to_end;
            *reinterpret_cast<float2*>(&c.read[2 * lane]) = pair_mul(read, make_float2(R.read_scale, R.read_scale));
            *reinterpret_cast<float2*>(&c.upd[2 * lane]) = pair_mul(upd, make_float2(R.update_scale, R.update_scale));
            *reinterpret_cast<int2*>(&c.bound[2 * lane]) = bound;
            if (lane == 0) {
                c.decay = decay;
                c.wide = !(fabsf(whole) < kWideSum);
            }
            if (!wait(&sh.full[ring.s], ring.parity)) break;
            const int left = static_cast<int>(min(static_cast<int64_t>(C), len - static_cast<int64_t>(chunk_of(k)) * C));
            if (left < C) {
                // rows past the length may hold anything (a NaN times a zero of P is a NaN): cleared
                unsigned char* st = tiles + ring.s * A.stage_bytes;
                const int rows = C - left;
#pragma unroll 1
                for (int p = 0; p < px + pz; ++p) {
                    uint4* panel = reinterpret_cast<uint4*>(st + off_y + p * kPanel + left * 128);
#pragma unroll 1
                    for (int e = lane; e < rows * 8; e += 32) panel[e] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            arrive_warp(&sh.ready[ring.s], lane);
            g = next;
        }
        if constexpr (kStateOnly) {
            if (lane == 0) A.seg_decays[(blockIdx.y * A.BH + bh) * A.n_segs + seg] = all;
        }
    } else if (warp == 3 || warp == 6) {
        // ---- products: warp 6 those of the state, warp 3 those of the scores, so that neither waits for the other's turn
        const uint32_t i_64 = tc::instr_bf16(C, false, false), i_o1 = tc::instr_bf16(C, true, false);
        const uint32_t i_kv = tc::instr_bf16(static_cast<uint32_t>(dxp), false, true);
        const uint32_t i_kv3 = tc::instr_bf16(static_cast<uint32_t>(dxp), true, true);
        const uint32_t base = smem_u32(tiles);
        const uint32_t lead = tc::elect();
        constexpr uint32_t kPanelStep = kPanel >> 4, kRows16 = 2048 >> 4;      // in descriptors' units
        Ring ring;
        if (warp == 6) {
#pragma unroll 1
            for (int k = 0; k < n; ++k, ring.next(A.stages)) {
                const uint32_t sx = base + ring.s * A.stage_bytes;
                if (!wait(&sh.ready[ring.s], ring.parity)) break;
                if (!wait(zh_of(k), kStateOnly ? k / 2 : k)) break;
                const uint32_t y = tc::desc_low(sx + off_y, kPanel);
                if constexpr (!kStateOnly) {
                    // O2's region: the last chunk's has to be read
                    if (k > 0 && !wait(&sh.o_read, k - 1)) break;
                    tc::fence_after();
                    const uint32_t x = tc::desc_low(sx, 16);
                    tc::mma_ts<true>(lead, t_o2, t_hb, x, i_64);
#pragma unroll
                    for (int q = 1; q < 4; ++q) tc::mma_ts(lead, t_o2, t_hb + 8 * q, x + 2 * q, i_64);
#pragma unroll 1
                    for (int p = 1; p < 2 * px; ++p) {
                        const uint32_t xp = x + (p < px ? p : p - px) * kPanelStep;
#pragma unroll
                        for (int q = 0; q < 4; ++q) tc::mma_ts(lead, t_o2, t_hb + 32 * p + 8 * q, xp + 2 * q, i_64);
                    }
                } else {
                    tc::fence_after();
                }
                const uint32_t zt = zt_of(k);
                if (kStateOnly && k == 0) tc::mma_ts<true>(lead, t_h, zt, y, i_kv);
                else tc::mma_ts(lead, t_h, zt, y, i_kv);
#pragma unroll
                for (int q = 1; q < 2 * C / 16; ++q) tc::mma_ts(lead, t_h, zt + q * 8, y + q % (C / 16) * kRows16, i_kv);
                if (R.terms == 3) {
                    const uint32_t w = tc::desc_low(sx + off_w, kPanel);
#pragma unroll
                    for (int q = 0; q < C / 16; ++q) tc::mma_ss(lead, t_h, w + q * kRows16, y + q * kRows16, i_kv3);
                }
                tc::commit(lead, kv_of(k));
                if constexpr (kStateOnly) {
                    if (k == n - 1) tc::commit(lead, &sh.state_done);
                } else {
                    tc::commit(lead, &sh.o_done);
                }
                tc::commit(lead, &sh.empty[ring.s]);
            }
        } else if constexpr (!kStateOnly) {
            const uint32_t phi = tc::desc_low(smem_u32(p_hi), 16);
            int last = 0;
#pragma unroll 1
            for (int k = 0; k <= n; ++k) {
                if (k > 0) {
                    // O1 of the last chunk
                    if (!wait(&sh.p_ready, k - 1)) break;
                    if (k > 1 && !wait(&sh.o_read, k - 2)) break;
                    tc::fence_after();
                    const uint32_t z = tc::desc_low(base + last * A.stage_bytes + off_z, kPanel);
                    tc::mma_ss<true>(lead, t_o1, z, phi, i_o1);
#pragma unroll
                    for (int q = 1; q < C / 16; ++q) tc::mma_ss(lead, t_o1, z + q * kRows16, phi + 2 * q, i_o1);
#pragma unroll
                    for (int q = 0; q < C / 16; ++q) tc::mma_ss(lead, t_o1, z + q * kRows16, phi + kPanelStep + 2 * q, i_o1);
                    tc::commit(lead, &sh.o_done);
                    tc::commit(lead, &sh.empty[last]);
                }
                if (k < n) {
                    // this chunk's scores; their commit stands for O1 too, so P's place is free by then
                    if (!wait(&sh.ready[ring.s], ring.parity)) break;
                    tc::fence_after();
                    const uint32_t sx = base + ring.s * A.stage_bytes;
                    const uint32_t x = tc::desc_low(sx, 16), y = tc::desc_low(sx + off_y, 16);
                    tc::mma_ss<true>(lead, t_s, x, y, i_64);
#pragma unroll
                    for (int q = 1; q < 4; ++q) tc::mma_ss(lead, t_s, x + 2 * q, y + 2 * q, i_64);
                    if (px == 2)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tc::mma_ss(lead, t_s, x + kPanelStep + 2 * q, y + kPanelStep + 2 * q, i_64);
                    tc::commit(lead, &sh.s_done);
                }
                last = ring.s;
                ring.next(A.stages);
            }
        }
        // nothing of this CTA's may still run when its tensor memory goes
        uint64_t* drained = &sh.drained[warp == 6];
        tc::commit(lead, drained);
        if (!__all_sync(0xffffffffu, wait_bounded(drained, 0, A.wait_ns, nullptr)) && lane == 0)
            atomicOr(A.status, ES_DEVICE_TIMEOUT);
    } else if (warp < 8) {
        // ---- P: row i, 32 columns
        if constexpr (!kStateOnly) {
            const int i = lane + 32 * (warp & 1), half = warp >> 2;
            const uint32_t from = t_s + (static_cast<uint32_t>(32 * (warp & 1)) << 16) + 32 * half;
            // rows of one half never see the columns of the other: forward rows 0-31 the late columns
            const float sign = R.reverse ? -1.0f : 1.0f;
            const bool none = R.reverse ? (warp & 1) > half : (warp & 1) < half;
            Ring ring;
#pragma unroll 1
            for (int k = 0; k < n; ++k, ring.next(A.stages)) {
                // the stage's coefficients, then the scores
                if (!wait(&sh.ready[ring.s], ring.parity) || !wait(&sh.s_done, k)) break;
                const Coef& c = sh.coef[ring.s];
                const uint32_t swz = i & 7;
                if (none) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t at = i * 128 + (((4 * half + q) ^ swz) << 4);
                        *reinterpret_cast<uint4*>(p_hi + at) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4*>(p_lo + at) = make_uint4(0, 0, 0, 0);
                    }
                } else {
                    tc::fence_after();
                    const float gs = sign * c.g2[i], gs_low = sign * c.low[i];
                    const int bound = c.bound[i], wide = c.wide;
                    // the half's columns that row i sees, as bits
                    const int first = max(0, (R.reverse ? i : bound) - 32 * half), last = min(31, (R.reverse ? bound : i) - 32 * half);
                    const uint32_t seen = first <= last ? (0xffffffffu >> (31 - (last - first))) << first : 0u;
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t r[8], hi[4], lo[4];
                        tc::ld(from + 8 * q, r);
                        const uint32_t mask = seen >> (8 * q);
                        const int j0 = 32 * half + 8 * q;
                        float2 d[4];
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float4 gj = *reinterpret_cast<const float4*>(&c.g2[j0 + 2 * e]);
                            float2 x = pair_fma(make_float2(gj.x, gj.y), make_float2(-sign, -sign), make_float2(gs, gs));
                            float2 y = pair_fma(make_float2(gj.z, gj.w), make_float2(-sign, -sign), make_float2(gs, gs));
                            if (!kDots || wide) {
                                const float4 lj = *reinterpret_cast<const float4*>(&c.low[j0 + 2 * e]);
                                x = pair_add(x, pair_fma(make_float2(lj.x, lj.y), make_float2(-sign, -sign), make_float2(gs_low, gs_low)));
                                y = pair_add(y, pair_fma(make_float2(lj.z, lj.w), make_float2(-sign, -sign), make_float2(gs_low, gs_low)));
                            }
                            d[e] = make_float2(tc::exp2_approx(x.x), tc::exp2_approx(x.y));
                            d[e + 1] = make_float2(tc::exp2_approx(y.x), tc::exp2_approx(y.y));
                        }
                        tc::wait_ld();
                        tc::loaded(r);
                        float2 v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = pair_mul(make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), d[e]);
                        if (!__all_sync(0xffffffffu, (mask & 0xffu) == 0xffu)) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (!(mask & (1u << (2 * e)))) v[e].x = 0.0f;
                                if (!(mask & (2u << (2 * e)))) v[e].y = 0.0f;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) tc::split2<kCut>(v[e], hi[e], lo[e]);
                        const uint32_t at = i * 128 + (((4 * half + q) ^ swz) << 4);
                        *reinterpret_cast<uint4*>(p_hi + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(p_lo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                fence_proxy_async_smem();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.p_ready);
                    mbar_arrive(&sh.empty[ring.s]);
                }
            }
        }
    } else if (warp < 16) {
        // ---- Z scaled and transposed: 32 value columns (lanes) and 32 of the tokens (pairs along the columns)
        const int slice = warp & 3, side = (warp - 8) / 4;
        const uint32_t to = 16 * side + (static_cast<uint32_t>(slice * 32) << 16);
        const bool on = slice * 32 < R.dz;
        // lane l names row l % 8 of block l / 8: two blocks of columns, two of tokens
        const uint32_t row = 32 * side + 8 * (lane / 16) + lane % 8, piece = 4 * (slice & 1) + (lane / 8) % 2;
        const uint32_t at0 = smem_u32(tiles) + off_z + (slice / 2) * kPanel + row * 128 + ((piece ^ (row & 7)) << 4);
        Ring ring;
#pragma unroll 1
        for (int k = 0; k < n; ++k, ring.next(A.stages)) {
            if (!wait(&sh.ready[ring.s], ring.parity)) break;
            if (kStateOnly ? k > 1 && !wait(kv_of(k), k / 2 - 1) : k > 0 && !wait(&sh.kv_done, k - 1)) break;
            tc::fence_after();
            if (on) {
                const float* upd = sh.coef[ring.s].upd + 32 * side + 2 * (lane % 4);
                const uint32_t at = at0 + ring.s * A.stage_bytes;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint32_t z[2][4], t[8];
                    float2 v[8];
                    // pieces 2 half and 2 half + 1 (the swizzle only flips that bit of the address)
                    tc::ld_blocks(at ^ (half << 5), z[0]);
                    tc::ld_blocks((at ^ (half << 5)) + 16 * 128, z[1]);
                    const uint32_t lanes = zt_of(k) + to + (static_cast<uint32_t>(16 * half) << 16);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 w = *reinterpret_cast<const float2*>(upd + 8 * (e / 2));
                        const uint32_t u = z[e / 4][e % 4];
                        v[e] = pair_mul(make_float2(tc::low_bf16(u), tc::high_bf16(u)), w);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) t[e] = tc::take_term<kCut>(v[e]);
                    tc::st_words(lanes, t);
                    if (R.terms == 3) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) t[e] = tc::take_term<kCut>(v[e]);
                        tc::st_words(lanes + 32, t);
                        // the third goes back as it came, to W's place, which this run leaves to the results
#pragma unroll
                        for (int e = 0; e < 8; ++e) z[e / 4][e % 4] = tc::pack_bf16(v[e].x, v[e].y);
                        tc::st_blocks((at ^ (half << 5)) + off_w - off_z, z[0]);
                        tc::st_blocks((at ^ (half << 5)) + off_w - off_z + 16 * 128, z[1]);
                        fence_proxy_async_smem();
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) t[e] = tc::pack_bf16(v[e].x, v[e].y);
                        tc::st_words(lanes + 32, t);
                    }
                }
                tc::wait_st();
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(zh_of(k));
                mbar_arrive(&sh.empty[ring.s]);
            }
        }
    } else if (warp < 24) {
        // ---- the state: lane = value column c, half of the key columns along
        const int slice = warp & 3, side = (warp - 16) / 4, a_lo = side * (dxp / 2), a_hi = a_lo + dxp / 2;
        const int c = slice * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(slice * 32) << 16;
        const bool on = slice * 32 < R.dz, real = c < R.dz;
        const int64_t size = static_cast<int64_t>(R.dx) * R.dz;
        // where the run's first state comes from
        const float* from = nullptr;
        int64_t fa = 0;
        if (real && !kStateOnly) {
            if (A.n_segs == 1) {
                if (R.init != nullptr) from = R.init + bh * size + c * R.sc;
                fa = R.sa;
            } else if (part.entry >= 0 && (!part.begins || R.init != nullptr)) {
                from = A.seg_states + blockIdx.y * A.seg_stride + (bh * A.n_segs + part.entry) * size + c;
                fa = R.dz;
            }
        }
        // the chunk's state leaves for its anchor block
        auto keep = [&](int at) {
            if ((at + 1) % kAnchorChunks == 0 || at == chunks - 1)
                state_out(t_h + lanes, a_lo, min(a_hi, R.dx), real ? R.anchors + (bh * A.n_anchors + at / kAnchorChunks) * size + c : nullptr,
                          R.dz);
        };
        if (on && !kStateOnly) {
            // 32 loads in flight: a short sequence is mostly this and the way in and out
#pragma unroll 1
            for (int a0 = a_lo; a0 < a_hi; a0 += 32) {
                uint32_t r[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = 0u;
                if (from != nullptr) {
                    const float* p = from + a0 * fa;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (a0 + e < R.dx) r[e] = __float_as_uint(p[e * fa]);
                }
                tc::st(t_h + lanes + a0, r);
            }
            tc::wait_st();
        }
        const bool anchored = !kStateOnly && R.anchors != nullptr && on;
        Ring ring;
        int k = 0;
#pragma unroll 1
        for (; k < n && !kStateOnly; ++k, ring.next(A.stages)) {
            if (!wait(&sh.ready[ring.s], ring.parity)) break;
            const float decay = sh.coef[ring.s].decay;
            if (k > 0 && !wait(&sh.kv_done, k - 1)) break;
            tc::fence_after();
            if (anchored && (R.reverse || k > 0)) keep(chunk_of(R.reverse ? k : k - 1));
            if (on) {
#pragma unroll 1
                for (int a0 = a_lo; a0 < a_hi; a0 += 16) {
                    uint32_t r[16], t[8], u[8];
                    tc::ld(t_h + lanes + a0, r);
                    tc::wait_ld();
                    tc::loaded(r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 v = make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
                        tc::split2<kCut>(v, t[e], u[e]);
                        const float2 d = pair_mul(v, make_float2(decay, decay));
                        r[2 * e] = __float_as_uint(d.x);
                        r[2 * e + 1] = __float_as_uint(d.y);
                    }
                    tc::st(t_hb + lanes + a0 / 2, t);
                    tc::st(t_hb + lanes + dxp / 2 + a0 / 2, u);
                    tc::st(t_h + lanes + a0, r);
                }
            }
            tc::wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(zh_of(k));
                mbar_arrive(&sh.empty[ring.s]);
            }
        }
        // the last state
        bool ok;
        if constexpr (kStateOnly) ok = wait(&sh.state_done, 0);
        else ok = k == n && (n == 0 || wait(&sh.kv_done, n - 1));
        if (ok) {
            tc::fence_after();
            if (anchored && !R.reverse && n > 0) keep(chunk_of(n - 1));
            if (on && kStateOnly)
                state_out(t_h + lanes, a_lo, min(a_hi, R.dx),
                          real ? A.seg_states + blockIdx.y * A.seg_stride + (bh * A.n_segs + seg) * size + c : nullptr, R.dz);
            else if (on && part.ends && R.fin != nullptr)
                state_out(t_h + lanes, a_lo, min(a_hi, R.dx), real ? R.fin + bh * size + c * R.sc : nullptr, R.sa);
        }
    } else {
        // ---- outputs: lane = value column c, tokens along the columns
        if constexpr (!kStateOnly) {
            const int slice = warp & 3, side = (warp - 24) / 4;       // 32 value columns, 32 of the tokens
            const int c = slice * 32 + lane;
            const uint32_t lanes = static_cast<uint32_t>(slice * 32) << 16;
            const bool on = slice * 32 < R.dz, real = c < R.dz;
            float* of = static_cast<float*>(R.out) + b * R.ob + static_cast<int64_t>(h) * R.oh;
            unsigned short* o16 = static_cast<unsigned short*>(R.out) + b * R.ob + static_cast<int64_t>(h) * R.oh;
            const bool wide = !R.out_f32 && R.wide;
            // the warp's part of the tile: lane l names row l % 8 of block l / 8 (blocks of 8 columns)
            const uint32_t row0 = 32 * side + lane % 8, w0 = off_w + (slice / 2) * kPanel;
            const uint32_t at0 = w0 + row0 * 128 + ((((4 * (slice & 1)) + lane / 8) ^ (row0 & 7)) << 4);
            const float2 scale = make_float2(R.out_scale, R.out_scale);
            Ring ring;
#pragma unroll 1
            for (int k = 0; k < n; ++k, ring.next(A.stages)) {
                // the stage's coefficients (and W), then the products
                if (!wait(&sh.ready[ring.s], ring.parity) || !wait(&sh.o_done, k)) break;
                tc::fence_after();
                const int64_t t0 = static_cast<int64_t>(chunk_of(k)) * C;
                const int left = static_cast<int>(min(static_cast<int64_t>(C), len - t0));
                const float* rd = sh.coef[ring.s].read + 32 * side + 2 * (lane % 4);
                unsigned char* st = tiles + ring.s * A.stage_bytes;
                if (on) {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        // 8 tokens: columns t / 4 of four blocks, two tokens
                        uint32_t o1[2][4], o2[2][4];
                        const uint32_t col = lanes + 32 * side + 8 * q;
                        tc::ld_pairs(t_o1 + col, o1[0]);
                        tc::ld_pairs(t_o1 + col + (16u << 16), o1[1]);
                        tc::ld_pairs(t_o2 + col, o2[0]);
                        tc::ld_pairs(t_o2 + col + (16u << 16), o2[1]);
                        const float2 r = *reinterpret_cast<const float2*>(rd + 8 * q);
                        tc::wait_ld();
                        tc::loaded(o1[0]);
                        tc::loaded(o1[1]);
                        tc::loaded(o2[0]);
                        tc::loaded(o2[1]);
                        if (q == 3) {
                            // the products of the next chunk may overwrite what was read
                            tc::fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sh.o_read);
                        }
                        float2 v[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const uint32_t* x1 = &o1[m / 2][2 * (m & 1)];
                            const uint32_t* x2 = &o2[m / 2][2 * (m & 1)];
                            v[m] = pair_fma(make_float2(__uint_as_float(x2[0]), __uint_as_float(x2[1])), r,
                                            pair_mul(make_float2(__uint_as_float(x1[0]), __uint_as_float(x1[1])), scale));
                        }
                        const uint32_t at = smem_u32(st) + at0 + 8 * q * 128;
                        const int row = 32 * side + 8 * q + 2 * (lane % 4);
                        if (kDots && dots) {
                            // out . w over the warp's columns (padded columns hold zeros)
                            uint32_t w[4];
                            tc::ld_blocks(at, w);
                            float2 d = make_float2(0.0f, 0.0f);
#pragma unroll
                            for (int m = 0; m < 4; ++m) d = pair_fma(v[m], make_float2(tc::low_bf16(w[m]), tc::high_bf16(w[m])), d);
                            // over the lanes of a token pair: half of them take the second token
                            const bool second = lane & 16;
                            float sum = second ? d.y : d.x;
                            sum += __shfl_xor_sync(0xffffffffu, second ? d.x : d.y, 16);
                            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                            const int mine = row + (second ? 1 : 0);
                            if ((lane & 12) == 0 && mine < left) R.dots[(slice * A.BH + bh) * A.T + t0 + mine] = sum;
                            __syncwarp();      // W's rows are read before the results take their place
                        }
                        if (!R.out_f32) {
                            uint32_t p[4];
#pragma unroll
                            for (int m = 0; m < 4; ++m) p[m] = tc::pack_bf16(v[m].x, v[m].y);
                            tc::st_blocks(at, p);
                        } else {
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const int cc = 32 * slice + 8 * m + lane / 4;
                                if (cc < R.dz && row < left) of[(t0 + row) * R.ot + cc] = v[m].x;
                                if (cc < R.dz && row + 1 < left) of[(t0 + row + 1) * R.ot + cc] = v[m].y;
                            }
                        }
                    }
                } else if (lane == 0) {
                    mbar_arrive(&sh.o_read);
                }
                // the next load of this place comes through the async proxy
                fence_proxy_async_smem();
                __syncwarp();
                if (on && !R.out_f32) {
                    // the warp's rows out, 64 bytes each, 16 a thread where the result's addresses allow it
                    const int piece = 4 * (slice & 1) + lane % 4, cc = 32 * slice + 8 * (lane % 4);
#pragma unroll 1
                    for (int row = 32 * side + lane / 4; row < min(left, 32 * side + 32); row += 8) {
                        const uint4 u = *reinterpret_cast<const uint4*>(st + w0 + row * 128 + ((piece ^ (row & 7)) << 4));
                        unsigned short* to = o16 + (t0 + row) * R.ot + cc;
                        if (wide) {
                            if (cc < R.dz) *reinterpret_cast<uint4*>(to) = u;
                        } else {
                            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (cc + e < R.dz) to[e] = static_cast<unsigned short>(e % 2 ? x[e / 2] >> 16 : x[e / 2]);
                        }
                    }
                }
                arrive_warp(&sh.empty[ring.s], lane);
            }
            // this segment's rows past the length are zero
            const int64_t lo = max(len, static_cast<int64_t>(c0) * C);
            const int64_t hi = seg == A.n_segs - 1 ? A.T : min(A.T, static_cast<int64_t>(c0 + A.seg_chunks) * C);
            if (wide) {
                const int cc = 32 * slice + 8 * (lane % 4);
                if (cc < R.dz)
#pragma unroll 4
                    for (int64_t t = lo + 8 * side + lane / 4; t < hi; t += 16)
                        *reinterpret_cast<uint4*>(o16 + t * R.ot + cc) = make_uint4(0, 0, 0, 0);
            } else if (real) {
#pragma unroll 1
                for (int64_t t = lo + side; t < hi; t += 2) {
                    if (R.out_f32) of[t * R.ot + c] = 0.0f;
                    else o16[t * R.ot + c] = 0;
                }
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 2) {
        tc::fence_after();
        tc::dealloc(sh.tmem, kTmemCols);
    }
}

bool encode(EncodeTiledFn fn, CUtensorMap* m, const AttnOperand& o, int heads, int d, int64_t T, int64_t B) {
    // a broadcast axis (stride 0) has an extent of one; extents of one take a stride that keeps the map valid
    if (o.sb == 0) B = 1;
    if (o.sh == 0) heads = 1;
    const int64_t row = (static_cast<int64_t>(d) * 2 + 15) & ~int64_t(15);
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(T),
                                static_cast<cuuint64_t>(B)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(heads > 1 ? o.sh * 2 : row), static_cast<cuuint64_t>(T > 1 ? o.st * 2 : row),
                                   static_cast<cuuint64_t>(B > 1 ? o.sb * 2 : row)};
    const cuuint32_t box[4] = {64, 1, C, 1}, one[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(o.p), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool attn_tc_operand_ok(const AttnOperand& o, int heads, int d, int64_t T, int64_t B) {
    if (d > 128 || d % 8 != 0) return false;
    if (reinterpret_cast<uintptr_t>(o.p) % 16 != 0) return false;
    auto fits = [](int64_t n, int64_t s) { return n <= 1 || (s % 8 == 0 && s < (int64_t(1) << 38)); };
    return fits(heads, o.sh) && fits(T, o.st) && fits(B, o.sb) && (T <= 1 || o.st > 0);
}

cudaError_t launch_attn_tc(const AttnLaunch& L, int* kernels, const char** err) {
    TcArgs A{};
    uint32_t stage = 0;
    bool any_dots = false;
    for (int r = 0; r < L.runs; ++r) {
        const AttnRun& f = L.run[r];
        TcRun& t = A.run[r];
        const bool maps = encode(L.encode, &t.x, f.x, L.H / f.x.div, f.dx, L.T, L.B) &&
                          encode(L.encode, &t.y, f.y, L.H / f.y.div, f.dx, L.T, L.B) &&
                          encode(L.encode, &t.z, f.z, L.H / f.z.div, f.dz, L.T, L.B) &&
                          (f.dots == nullptr || encode(L.encode, &t.w, f.w, L.H / f.w.div, f.dz, L.T, L.B));
        if (!maps) {
            *err = "cuTensorMapEncodeTiled failed";
            return cudaErrorInvalidValue;
        }
        t.out = f.out;
        t.ob = f.ob;
        t.ot = f.ot;
        t.oh = f.oh;
        t.init = f.init;
        t.fin = f.fin;
        t.sa = f.sa;
        t.sc = f.sc;
        t.update_scale = f.update_scale;
        t.read_scale = f.read_scale;
        t.out_scale = f.out_scale;
        t.dots = f.dots;
        any_dots = any_dots || f.dots != nullptr;
        t.anchors = f.anchors;
        t.xdiv = f.x.sh > 0 ? f.x.div : L.H;
        t.xb = f.x.sb > 0;
        t.ydiv = f.y.sh > 0 ? f.y.div : L.H;
        t.yb = f.y.sb > 0;
        t.zdiv = f.z.sh > 0 ? f.z.div : L.H;
        t.zb = f.z.sb > 0;
        t.wdiv = f.w.sh > 0 ? f.w.div : L.H;
        t.wb = f.w.sb > 0;
        t.dx = f.dx;
        t.dz = f.dz;
        t.reverse = f.reverse;
        t.out_f32 = f.out_f32;
        t.terms = f.state_result ? 3 : 2;
        t.wide = reinterpret_cast<uintptr_t>(f.out) % 16 == 0 && f.ob % 8 == 0 && f.ot % 8 == 0 && f.oh % 8 == 0;
        const uint32_t px = (f.dx + 63) / 64, pz = (f.dz + 63) / 64;
        const uint32_t bytes = (2 * px + 2 * pz) * kPanel;
        stage = bytes > stage ? bytes : stage;
        const int64_t size = static_cast<int64_t>(f.dx) * f.dz;
        A.seg_stride = L.B * L.H * L.n_segs * size;
    }
    A.T = L.T;
    A.BH = L.B * L.H;
    A.H = L.H;
    A.n_segs = L.n_segs;
    A.seg_chunks = static_cast<int>(L.seg_chunks);
    A.g = L.g;
    A.gb = L.gb;
    A.gt = L.gt;
    A.gh = L.gh;
    A.lengths = L.lengths;
    A.n_anchors = L.n_anchors;
    A.seg_states = L.seg_states;
    A.seg_decays = L.seg_decays;
    A.status = L.status;
    A.wait_ns = L.wait_ns;
    A.drop_tile = L.drop_tile;
    A.stage_bytes = stage;
    // tiles, P's two terms, alignment; the rest of the 227 KB is the static struct
    const uint32_t room = 227 * 1024 - static_cast<uint32_t>(sizeof(Shared)) - 1024 - 1024;
    const uint32_t fit = (room - 2 * kPanel) / stage;
    A.stages = static_cast<int>(fit < kMaxStages ? fit : kMaxStages);
    const size_t smem = A.stages * stage + 2 * kPanel + 1024;
    *kernels = 0;
    cudaError_t e;
    const unsigned blocks = static_cast<unsigned>(A.BH * A.n_segs);
    auto launch = [&](void (*kernel)(TcArgs)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        kernel<<<dim3(blocks, L.runs), kThreads, smem, L.stream>>>(A);
        return cudaGetLastError();
    };
    if (A.n_segs > 1) {
        if ((e = launch(k_attn_tc<true, false>)) != cudaSuccess) return e;
        if ((e = launch_attn_join(L, C)) != cudaSuccess) return e;
        *kernels += 2;
    }
    if ((e = launch(any_dots ? k_attn_tc<false, true> : k_attn_tc<false, false>)) != cudaSuccess) return e;
    ++*kernels;
    return cudaGetLastError();
}

}  // namespace es
