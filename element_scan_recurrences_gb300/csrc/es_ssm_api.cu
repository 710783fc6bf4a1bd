// es_ssm_api.cu -- entry points of the state-space layer's operators (es.h): the
// short causal convolution, the selective scan and the group norm with a gate.
// Validation, workspaces, segments and launches.
#include <cmath>

#include "es.h"
#include "es_attn.h"
#include "es_internal.h"
#include "es_ssm.h"
#include "es_views.h"

namespace es {
namespace {

bool known(int64_t dtype) { return dtype == ES_F32 || dtype == ES_BF16; }
int64_t size_of(int64_t dtype) { return dtype == ES_BF16 ? 2 : 4; }

// The spans a call reads and writes.
struct Spans {
    Span in[16], out[12];
    int n_in = 0, n_out = 0;
};

es_status add_rows(const char* fn, const char* name, const es_rows& r, int64_t B, int64_t T, int64_t C, int64_t size, bool output, Spans* S) {
    const es_heads v{r.data, r.stride_b, r.stride_t, 0, 1};
    return check_view(fn, name, v, B, T, C, size, output, output ? &S->out[S->n_out++] : &S->in[S->n_in++]);
}

es_status add_heads(const char* fn, const char* name, const es_heads& v, int64_t heads, int64_t B, int64_t T, int64_t dim, int64_t size,
                    bool output, Spans* S) {
    if (v.heads != heads)
        return api_fail(ES_E_DIM_001, "E-DIM-001 %s: `%s` has %lld heads, not %lld", fn, name, static_cast<long long>(v.heads),
                        static_cast<long long>(heads));
    return check_view(fn, name, v, B, T, dim, size, output, output ? &S->out[S->n_out++] : &S->in[S->n_in++]);
}

es_status add_dense(const char* fn, const char* name, const void* p, int64_t elements, int64_t size, bool output, Spans* S) {
    if (reinterpret_cast<uintptr_t>(p) % size != 0) return api_fail(ES_E_ARG, "%s: `%s` is not aligned to its elements", fn, name);
    (output ? S->out[S->n_out++] : S->in[S->n_in++]) = Span{name, p, p == nullptr ? 0 : elements * size};
    return ES_OK;
}

// a state to read and, for `to` at the same address, to write in its place
es_status add_states(const char* fn, const void* from, const void* to, int64_t elements, int64_t size, Spans* S) {
    es_status st = add_dense(fn, "initial_state", from, elements, size, false, S);
    if (st != ES_OK) return st;
    if (from == to) S->in[S->n_in - 1].bytes = 0;
    return add_dense(fn, "final_state", to, elements, size, true, S);
}

es_status no_overlap(const char* fn, const Spans& S, const void* ws, size_t bytes) {
    return check_outputs(fn, S.in, S.n_in, S.out, S.n_out, ws, bytes);
}

// [B, T, C] within the index arithmetic: blocks and rows below 2^31, elements below 2^56
es_status check_sizes(const char* fn, int64_t B, int64_t T, int64_t C) {
    if (B < 0 || T < 0 || C < 0) return api_fail(ES_E_DIM_001, "E-DIM-001 %s: a negative dimension", fn);
    int64_t x;
    if (T >= (int64_t(1) << 31) || C >= (int64_t(1) << 31) || __builtin_mul_overflow(B, T > 0 ? T : 1, &x) ||
        __builtin_mul_overflow(x, C > 0 ? C : 1, &x) || x >= (int64_t(1) << 48))
        return api_fail(ES_E_UNSUPPORTED, "%s: too many elements", fn);
    return ES_OK;
}

constexpr int64_t kMostBlocks = 0x7fffffff;

// ---------------------------------------------------------------------------
// convolution

struct ConvPlan {
    ConvLaunch L;
    bool empty;
    size_t bytes;
};

es_status plan_conv(const char* fn, const es_causal_conv_args* a, const es_causal_conv_grads* g, bool step, ConvPlan* P) {
    if (a == nullptr) return api_fail(ES_E_ARG, "%s: null arguments", fn);
    if (!known(a->dtype) || !known(a->weight_dtype))
        return api_fail(ES_E_DIM_002, "E-DIM-002 %s: dtypes %lld (weights %lld): f32 or bf16 are taken", fn,
                        static_cast<long long>(a->dtype), static_cast<long long>(a->weight_dtype));
    const int64_t B = a->batch, T = a->length, C = a->channels, W = a->taps;
    es_status st;
    if ((st = check_sizes(fn, B, T, C)) != ES_OK) return st;
    if (W < 2 || W > kMaxTaps)
        return api_fail(ES_E_UNSUPPORTED, "%s: %lld taps; 2..%d are supported", fn, static_cast<long long>(W), kMaxTaps);
    if (step && T != 1) return api_fail(ES_E_DIM_001, "E-DIM-001 %s: a step is one token, not %lld", fn, static_cast<long long>(T));
    if (step && a->lengths != nullptr) return api_fail(ES_E_ARG, "%s: a step takes no lengths", fn);
    const int64_t size = size_of(a->dtype), wsize = size_of(a->weight_dtype), n_state = B * (W - 1) * C;
    Spans S;
    if ((st = add_rows(fn, "x", a->x, B, T, C, size, false, &S)) != ES_OK) return st;
    if (C > 0 && a->weight == nullptr) return api_fail(ES_E_ARG, "%s: `weight` is a null pointer", fn);
    if ((st = add_dense(fn, "weight", a->weight, C * W, wsize, false, &S)) != ES_OK) return st;
    if ((st = add_dense(fn, "bias", a->bias, C, wsize, false, &S)) != ES_OK) return st;
    if ((st = add_dense(fn, "lengths", a->lengths, B, 4, false, &S)) != ES_OK) return st;
    *P = ConvPlan{};
    ConvLaunch& L = P->L;
    L.bf16 = a->dtype == ES_BF16;
    L.w_bf16 = a->weight_dtype == ES_BF16;
    L.taps = static_cast<int>(W);
    L.act = a->activation != 0;
    L.B = B;
    L.T = T;
    L.C = C;
    L.x = a->x;
    L.w = a->weight;
    L.bias = a->bias;
    L.lengths = a->lengths;
    L.init = a->initial_state;
    if (g == nullptr) {
        if (step && n_state > 0 && (a->initial_state == nullptr || a->final_state == nullptr))
            return api_fail(ES_E_ARG, "%s: a step needs the state and a place for the new one", fn);
        if ((st = add_rows(fn, "out", a->out, B, T, C, size, true, &S)) != ES_OK) return st;
        if ((st = add_states(fn, a->initial_state, a->final_state, n_state, size, &S)) != ES_OK) return st;
        L.out = a->out;
        L.fin = a->final_state;
    } else {
        if ((st = add_dense(fn, "initial_state", a->initial_state, n_state, size, false, &S)) != ES_OK) return st;
        if ((st = add_rows(fn, "grad_out", g->grad_out, B, T, C, size, false, &S)) != ES_OK) return st;
        if ((st = add_dense(fn, "grad_final_state", g->grad_final_state, n_state, size, false, &S)) != ES_OK) return st;
        if ((st = add_rows(fn, "grad_x", g->grad_x, B, T, C, size, true, &S)) != ES_OK) return st;
        if ((st = add_dense(fn, "grad_weight", g->grad_weight, C * W, wsize, true, &S)) != ES_OK) return st;
        if ((st = add_dense(fn, "grad_bias", g->grad_bias, C, wsize, true, &S)) != ES_OK) return st;
        if (g->grad_bias != nullptr && a->bias == nullptr) return api_fail(ES_E_ARG, "%s: a gradient of `bias`, which is null", fn);
        if ((st = add_dense(fn, "grad_initial_state", g->grad_initial_state, n_state, size, true, &S)) != ES_OK) return st;
        L.g = g->grad_out;
        L.out = g->grad_x;
        L.gfin = g->grad_final_state;
        L.fin = g->grad_initial_state;
        L.gw = g->grad_weight;
        L.gb = g->grad_bias;
        if (C > 0 && B > 0 && (L.gw != nullptr || L.gb != nullptr))
            P->bytes = static_cast<size_t>(conv_backward_rows(L)) * (W + 1) * C * 4;
    }
    P->empty = B == 0 || C == 0;
    const int64_t blocks = B * (T / 8 + 1) * (C / 128 + 1);
    if (blocks > kMostBlocks) return api_fail(ES_E_UNSUPPORTED, "%s: too many elements", fn);
    return no_overlap(fn, S, a->workspace, P->bytes);
}

// ---------------------------------------------------------------------------
// selective scan

struct ScanPlan {
    ScanBackward S;
    bool empty, find;            // find: a backward call without checkpoints
    size_t kept, seg_state, seg_sum, part_bc, part_c, bytes, kept_bytes;
    size_t first;                // offset of the copy of init, plus one (0: none)
    int fwd_segs;                // of the pass that finds the kept states
    int64_t fwd_seg_chunks;
};

// Segments a row's tokens are cut into.  A CTA takes a row's block of channels from
// token to token, and a chunk takes it the longer the more CTAs share its SM: 1 + 0.37
// us for each of them (7 at most; measured 2.0 us at 3.4, 3.5 at 6.7).  Segments make
// more CTAs of fewer chunks, for a pass over all but one of them that finds their own
// states at 0.6 of that, a launch, and at the start of each a read of those before it.
// More CTAs than the GPU holds even out what its SMs get: 65536 tokens x 2048 channels
// 1397 us in 16 segments, 1347 in 19, 1301 in 32, 1331 in 64.  Backwards (2 CTAs an SM
// at most, of 4 times the channels) a chunk takes 9.4 us alone, 13 by two, and a
// second wave would run alone.  4 x 2048 x 4096 whole and in two segments: forwards 249
// us, 290; backwards 1200, 874 (chosen: one, two).
//
// The paces and the CTAs an SM holds were measured in bf16 at 16 states.  By their tiles
// others hold fewer: forwards 4 at up to 8 states (f32 2, and 5 or 6 above), backwards
// one at up to 8 states.  They go by the same rule; compared were 4 x 1024 x 2048 channels
// whole, in two segments and as chosen, forwards and backwards: 8 states 131, 105, 78 us
// and 717, 421, 242 (f32 136, 107, 112 and 726, 435, 266), 16 states 103, 101, 102 and 594,
// 352, 250 (f32 126, 114, 113 and 593, 357, 258), 32 states 132, 140, 132 and 574, 425, 425,
// 64 states 181, 241, 181 and 758, 823, 758.
struct Pace {
    int resident, waves;
    double alone, more;          // us a chunk of one CTA an SM, what each further one adds
};
constexpr Pace kForwards{7, 4, 1.37, 0.37}, kBackwards{2, 1, 9.4, 3.7};

double chunk_us(const Pace& p, int64_t ctas) {
    const double each = static_cast<double>(ctas) / kSms;
    // (the last wave ends raggedly: a twentieth of one)
    if (each > p.resident) return (each / p.resident + 0.05) * (p.alone + (p.resident - 1) * p.more);
    return p.alone + (std::ceil(each) > 1.0 ? std::ceil(each) - 1.0 : 0.0) * p.more;
}

// `ctas` of the main pass, `first` of the pass before it, a segment
int scan_segments(const Pace& p, int64_t ctas, int64_t first, int64_t chunks, int64_t* seg_chunks) {
    *seg_chunks = chunks > 0 ? chunks : 1;
    const int64_t most = static_cast<int64_t>(kSms) * p.resident * p.waves / (ctas > 0 ? ctas : 1);
    double best = static_cast<double>(chunks) * chunk_us(p, ctas);
    int segs = 1;
    // (some forty numbers of segments, a hundred for a CTA or two: a plan is made at every call)
    for (int64_t s = 2; s <= most && s <= chunks; s += s < 16 ? 1 : s / 16) {
        const int64_t each = (chunks + s - 1) / s, n = (chunks + each - 1) / each;
        const double us = static_cast<double>(each) * (chunk_us(p, ctas * n) + 0.6 * chunk_us(kForwards, first * (n - 1))) + 5.0 + 0.6 * n;
        if (us < best) {
            best = us;
            segs = static_cast<int>(n);
            *seg_chunks = each;
        }
    }
    return segs;
}

es_status plan_scan(const char* fn, const es_selective_scan_args* a, const es_selective_scan_grads* g, bool step, ScanPlan* P) {
    if (a == nullptr) return api_fail(ES_E_ARG, "%s: null arguments", fn);
    if (!known(a->dtype))
        return api_fail(ES_E_DIM_002, "E-DIM-002 %s: dtype %lld is neither f32 nor bf16", fn, static_cast<long long>(a->dtype));
    const int64_t B = a->batch, T = a->length, C = a->channels, N = a->states, G = a->groups;
    es_status st;
    if ((st = check_sizes(fn, B, T, C)) != ES_OK) return st;
    if (N < 1 || N > kMaxStates)
        return api_fail(ES_E_UNSUPPORTED, "%s: %lld states a channel; 1..%d are supported", fn, static_cast<long long>(N), kMaxStates);
    if (G < 1 || C % G != 0)
        return api_fail(ES_E_DIM_001, "E-DIM-001 %s: %lld groups do not divide the %lld channels", fn, static_cast<long long>(G),
                        static_cast<long long>(C));
    // (channels bound the groups, but for none)
    if (C == 0 && (st = check_sizes(fn, B, T, G)) != ES_OK) return st;
    if (step && T != 1) return api_fail(ES_E_DIM_001, "E-DIM-001 %s: a step is one token, not %lld", fn, static_cast<long long>(T));
    if (step && (a->lengths != nullptr || a->checkpoints != nullptr))
        return api_fail(ES_E_ARG, "%s: a step takes no lengths and leaves no checkpoints", fn);
    const bool backward = g != nullptr, gated = a->gate.data != nullptr;
    const int64_t size = size_of(a->dtype), n_state = B * C * N;
    Spans S;
    if ((st = add_rows(fn, "x", a->x, B, T, C, size, false, &S)) != ES_OK) return st;
    if ((st = add_rows(fn, "delta", a->delta, B, T, C, size, false, &S)) != ES_OK) return st;
    if (gated && (st = add_rows(fn, "gate", a->gate, B, T, C, size, false, &S)) != ES_OK) return st;
    if ((st = add_heads(fn, "b", a->b, G, B, C > 0 ? T : 0, N, size, false, &S)) != ES_OK) return st;
    if ((st = add_heads(fn, "c", a->c, G, B, C > 0 ? T : 0, N, size, false, &S)) != ES_OK) return st;
    if (C > 0 && a->a == nullptr) return api_fail(ES_E_ARG, "%s: `a` is a null pointer", fn);
    if ((st = add_dense(fn, "a", a->a, C * N, 4, false, &S)) != ES_OK) return st;
    if ((st = add_dense(fn, "skip", a->skip, C, 4, false, &S)) != ES_OK) return st;
    if ((st = add_dense(fn, "delta_bias", a->delta_bias, C, 4, false, &S)) != ES_OK) return st;
    if ((st = add_dense(fn, "lengths", a->lengths, B, 4, false, &S)) != ES_OK) return st;

    *P = ScanPlan{};
    ScanLaunch& L = P->S.f;
    L.bf16 = a->dtype == ES_BF16;
    L.softplus = a->softplus != 0;
    L.B = B;
    L.T = T;
    L.C = C;
    L.N = static_cast<int>(N);
    L.G = static_cast<int>(G);
    L.x = a->x;
    L.delta = a->delta;
    L.gate = a->gate;
    L.b = a->b;
    L.c = a->c;
    L.a = a->a;
    L.skip = a->skip;
    L.bias = a->delta_bias;
    L.lengths = a->lengths;
    L.init = a->initial_state;
    L.chunks = (T + kScanChunk - 1) / kScanChunk;
    P->empty = B == 0 || C == 0;
    P->kept_bytes = static_cast<size_t>(L.chunks) * n_state * 4;
    auto wide = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    L.wide = N % 4 == 0 && wide(a->a) && wide(a->initial_state) && wide(a->final_state);
    if (!backward) {
        if (step && n_state > 0 && (a->initial_state == nullptr || a->final_state == nullptr))
            return api_fail(ES_E_ARG, "%s: a step needs the state and a place for the new one", fn);
        if ((st = add_rows(fn, "out", a->out, B, T, C, size, true, &S)) != ES_OK) return st;
        if ((st = add_states(fn, a->initial_state, a->final_state, n_state, 4, &S)) != ES_OK) return st;
        L.out = a->out;
        L.fin = a->final_state;
    } else {
        if ((st = add_dense(fn, "initial_state", a->initial_state, n_state, 4, false, &S)) != ES_OK) return st;
        if (gated != (g->grad_gate.data != nullptr))
            return api_fail(ES_E_ARG, "%s: `grad_gate` goes with `gate`", fn);
        if (g->grad_skip != nullptr && a->skip == nullptr) return api_fail(ES_E_ARG, "%s: a gradient of `skip`, which is null", fn);
        if (g->grad_delta_bias != nullptr && a->delta_bias == nullptr)
            return api_fail(ES_E_ARG, "%s: a gradient of `delta_bias`, which is null", fn);
        if ((st = add_rows(fn, "grad_out", g->grad_out, B, T, C, size, false, &S)) != ES_OK) return st;
        if ((st = add_dense(fn, "grad_final_state", g->grad_final_state, n_state, 4, false, &S)) != ES_OK) return st;
        if ((st = add_rows(fn, "grad_x", g->grad_x, B, T, C, size, true, &S)) != ES_OK) return st;
        if ((st = add_rows(fn, "grad_delta", g->grad_delta, B, T, C, size, true, &S)) != ES_OK) return st;
        if (gated && (st = add_rows(fn, "grad_gate", g->grad_gate, B, T, C, size, true, &S)) != ES_OK) return st;
        if ((st = add_heads(fn, "grad_b", g->grad_b, G, B, T, N, size, true, &S)) != ES_OK) return st;
        if ((st = add_heads(fn, "grad_c", g->grad_c, G, B, T, N, size, true, &S)) != ES_OK) return st;
        if ((st = add_dense(fn, "grad_a", g->grad_a, C * N, 4, true, &S)) != ES_OK) return st;
        if ((st = add_dense(fn, "grad_skip", g->grad_skip, C, 4, true, &S)) != ES_OK) return st;
        if ((st = add_dense(fn, "grad_delta_bias", g->grad_delta_bias, C, 4, true, &S)) != ES_OK) return st;
        if ((st = add_dense(fn, "grad_initial_state", g->grad_initial_state, n_state, 4, true, &S)) != ES_OK) return st;
        ScanBackward& Q = P->S;
        Q.g = g->grad_out;
        Q.gx = g->grad_x;
        Q.gdelta = g->grad_delta;
        Q.ggate = g->grad_gate;
        Q.gb = g->grad_b;
        Q.gc = g->grad_c;
        Q.ga = g->grad_a;
        Q.gskip = g->grad_skip;
        Q.gbias = g->grad_delta_bias;
        Q.gfin = g->grad_final_state;
        Q.ginit = g->grad_initial_state;
        L.wide = N % 4 == 0 && wide(a->a) && wide(a->initial_state) && wide(Q.gfin) && wide(Q.ginit);
    }
    if (a->checkpoints != nullptr) {
        if (a->checkpoints_bytes < 0 || static_cast<size_t>(a->checkpoints_bytes) < P->kept_bytes)
            return api_fail(ES_E_ARG, "%s: checkpoints of %lld bytes; %zu are needed", fn, static_cast<long long>(a->checkpoints_bytes),
                            P->kept_bytes);
        if (!wide(a->checkpoints)) return api_fail(ES_E_ARG, "%s: the checkpoints are not 16-byte aligned", fn);
        if ((st = add_dense(fn, "checkpoints", a->checkpoints, static_cast<int64_t>(P->kept_bytes / 4), 4, !backward, &S)) != ES_OK) return st;
        L.kept = static_cast<float*>(a->checkpoints);
    }
    L.segs = 1;
    L.seg_chunks = L.chunks > 0 ? L.chunks : 1;
    P->fwd_segs = 1;
    P->fwd_seg_chunks = L.seg_chunks;
    if (!P->empty) {
        const int g = static_cast<int>(G), n = static_cast<int>(N);
        const int64_t ctas = G * scan_blocks(C, g, scan_channels(n)) * B, back = G * scan_blocks(C, g, scan_bwd_channels(n)) * B;
        size_t at = 0;
        if (!step) P->fwd_segs = scan_segments(kForwards, ctas, ctas, L.chunks, &P->fwd_seg_chunks);
        if (!backward) {
            L.segs = P->fwd_segs;
            L.seg_chunks = P->fwd_seg_chunks;
        } else {
            L.segs = scan_segments(kBackwards, back, ctas, L.chunks, &L.seg_chunks);
            P->find = L.kept == nullptr && L.chunks > 0;
        }
        int64_t segs = L.segs;
        if (P->find && P->fwd_segs > segs) segs = P->fwd_segs;
        if (ctas > kMostBlocks / segs || (step && B > 4 * 65535))
            return api_fail(ES_E_UNSUPPORTED, "%s: too many rows and channels", fn);
        if (segs > 1) {
            P->seg_state = take(&at, 4 * segs * n_state);
            P->seg_sum = take(&at, 4 * segs * B * C);
            if (!backward && a->final_state != nullptr && a->final_state == a->initial_state) P->first = take(&at, 4 * n_state) + 1;
        }
        if (backward) {
            if (P->find) P->kept = take(&at, static_cast<int64_t>(P->kept_bytes));
            P->part_bc = take(&at, 4 * back * T * 2 * N);
            P->part_c = take(&at, 4 * segs * B * C * (N + 2));
        }
        P->bytes = at;
    }
    return no_overlap(fn, S, a->workspace, P->bytes);
}

// ---------------------------------------------------------------------------
// group norm

struct NormPlan {
    NormLaunch L;
    bool empty;
    size_t bytes;
};

es_status plan_norm(const char* fn, const es_group_norm_args* a, const es_group_norm_grads* g, NormPlan* P) {
    if (a == nullptr) return api_fail(ES_E_ARG, "%s: null arguments", fn);
    if (!known(a->dtype) || !known(a->weight_dtype))
        return api_fail(ES_E_DIM_002, "E-DIM-002 %s: dtypes %lld (weights %lld): f32 or bf16 are taken", fn,
                        static_cast<long long>(a->dtype), static_cast<long long>(a->weight_dtype));
    const int64_t B = a->batch, T = a->length, H = a->x.heads, D = a->dim;
    es_status st;
    if (H < 0) return api_fail(ES_E_DIM_001, "E-DIM-001 %s: a negative dimension", fn);
    if (D < 1 || D > kMaxNormDim)
        return api_fail(ES_E_UNSUPPORTED, "%s: groups of %lld values; 1..%d are supported", fn, static_cast<long long>(D), kMaxNormDim);
    if (H > 65535) return api_fail(ES_E_UNSUPPORTED, "%s: %lld groups a token; 65535 are supported", fn, static_cast<long long>(H));
    if ((st = check_sizes(fn, B, T, H * D)) != ES_OK) return st;
    if (!(a->eps >= 0) || !std::isfinite(a->eps)) return api_fail(ES_E_ARG, "%s: eps %g", fn, a->eps);
    const bool backward = g != nullptr, gated = a->gate.data != nullptr;
    if (gated && a->activation) return api_fail(ES_E_ARG, "%s: an activation goes without a gate only", fn);
    if (!gated && a->gate_first) return api_fail(ES_E_ARG, "%s: gate_first without a gate", fn);
    const int64_t size = size_of(a->dtype), wsize = size_of(a->weight_dtype);
    Spans S;
    if ((st = add_heads(fn, "x", a->x, H, B, T, D, size, false, &S)) != ES_OK) return st;
    if (gated && (st = add_heads(fn, "gate", a->gate, H, B, T, D, size, false, &S)) != ES_OK) return st;
    if ((st = add_dense(fn, "weight", a->weight, H * D, wsize, false, &S)) != ES_OK) return st;
    if ((st = add_dense(fn, "bias", a->bias, H * D, wsize, false, &S)) != ES_OK) return st;
    *P = NormPlan{};
    NormLaunch& L = P->L;
    L.bf16 = a->dtype == ES_BF16;
    L.w_bf16 = a->weight_dtype == ES_BF16;
    L.center = a->center != 0;
    L.first = a->gate_first != 0;
    L.act = a->activation != 0;
    L.B = B;
    L.T = T;
    L.H = static_cast<int>(H);
    L.D = static_cast<int>(D);
    L.eps = static_cast<float>(a->eps);
    L.x = a->x;
    L.gate = a->gate;
    L.w = a->weight;
    L.bias = a->bias;
    P->empty = B * T == 0 || H == 0;
    if (!backward) {
        if ((st = add_heads(fn, "out", a->out, H, B, T, D, size, true, &S)) != ES_OK) return st;
        L.out = a->out;
    } else {
        if (gated != (g->grad_gate.data != nullptr)) return api_fail(ES_E_ARG, "%s: `grad_gate` goes with `gate`", fn);
        if ((g->grad_weight != nullptr && a->weight == nullptr) || (g->grad_bias != nullptr && a->bias == nullptr))
            return api_fail(ES_E_ARG, "%s: a gradient of a weight that is null", fn);
        if ((st = add_heads(fn, "grad_out", g->grad_out, H, B, T, D, size, false, &S)) != ES_OK) return st;
        if ((st = add_heads(fn, "grad_x", g->grad_x, H, B, T, D, size, true, &S)) != ES_OK) return st;
        if (gated && (st = add_heads(fn, "grad_gate", g->grad_gate, H, B, T, D, size, true, &S)) != ES_OK) return st;
        if ((st = add_dense(fn, "grad_weight", g->grad_weight, H * D, wsize, true, &S)) != ES_OK) return st;
        if ((st = add_dense(fn, "grad_bias", g->grad_bias, H * D, wsize, true, &S)) != ES_OK) return st;
        L.g = g->grad_out;
        L.out = g->grad_x;
        L.ggate = g->grad_gate;
        L.gw = g->grad_weight;
        L.gb = g->grad_bias;
        if (!P->empty && (L.gw != nullptr || L.gb != nullptr)) P->bytes = static_cast<size_t>(norm_backward_rows(L)) * 2 * H * D * 4;
    }
    return no_overlap(fn, S, a->workspace, P->bytes);
}

es_status run_norm(const char* fn, const es_group_norm_args* a, const es_group_norm_grads* g, es_stream_t stream) {
    NormPlan P;
    es_status st = plan_norm(fn, a, g, &P);
    if (st != ES_OK) return st;
    NormLaunch& L = P.L;
    L.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (P.empty) {       // no rows: the weights' gradients are sums of nothing
        for (void* w : {L.gw, L.gb})
            if (w != nullptr && L.H > 0 && (e = cudaMemsetAsync(w, 0, static_cast<size_t>(L.H) * L.D * (L.w_bf16 ? 2 : 4), L.stream)) != cudaSuccess)
                return cuda_fail(fn, e);
        return ES_OK;
    }
    if ((st = check_workspace(fn, a->workspace, a->workspace_bytes, P.bytes)) != ES_OK) return st;
    L.partial = P.bytes > 0 ? static_cast<float*>(a->workspace) : nullptr;
    int n = 0;
    if ((e = launch_norm(L, g != nullptr, &n)) != cudaSuccess) return cuda_fail(fn, e);
    count_launch(n);
    return ES_OK;
}

float* at(void* workspace, size_t offset) { return reinterpret_cast<float*>(static_cast<char*>(workspace) + offset); }

}  // namespace
}  // namespace es

extern "C" {

es_status es_causal_conv(const es_causal_conv_args* args, es_stream_t stream) {
    const char* fn = "es_causal_conv";
    es::ConvPlan P;
    const es_status st = es::plan_conv(fn, args, nullptr, false, &P);
    if (st != ES_OK || P.empty) return st;
    if (P.L.T == 0 && P.L.fin == nullptr) return ES_OK;
    P.L.stream = reinterpret_cast<cudaStream_t>(stream);
    int n = 0;
    const cudaError_t e = es::launch_conv(P.L, &n);
    if (e != cudaSuccess) return es::cuda_fail(fn, e);
    es::count_launch(n);
    return ES_OK;
}

es_status es_causal_conv_backward(const es_causal_conv_args* args, const es_causal_conv_grads* grads, es_stream_t stream) {
    const char* fn = "es_causal_conv_backward";
    if (grads == nullptr) return es::api_fail(ES_E_ARG, "%s: null gradients", fn);
    es::ConvPlan P;
    es_status st = es::plan_conv(fn, args, grads, false, &P);
    if (st != ES_OK) return st;
    es::ConvLaunch& L = P.L;
    L.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (P.empty) {       // no rows: the weights' gradients are sums of nothing
        const size_t size = L.w_bf16 ? 2 : 4;
        if (L.C > 0 && ((L.gw != nullptr && (e = cudaMemsetAsync(L.gw, 0, L.C * L.taps * size, L.stream)) != cudaSuccess) ||
                        (L.gb != nullptr && (e = cudaMemsetAsync(L.gb, 0, L.C * size, L.stream)) != cudaSuccess)))
            return es::cuda_fail(fn, e);
        return ES_OK;
    }
    if ((st = es::check_workspace(fn, args->workspace, args->workspace_bytes, P.bytes)) != ES_OK) return st;
    L.partial = P.bytes > 0 ? static_cast<float*>(args->workspace) : nullptr;
    int n = 0;
    if ((e = es::launch_conv_backward(L, &n)) != cudaSuccess) return es::cuda_fail(fn, e);
    es::count_launch(n);
    return ES_OK;
}

es_status es_causal_conv_workspace(const es_causal_conv_args* args, const es_causal_conv_grads* grads, size_t* bytes) {
    if (bytes == nullptr) return es::api_fail(ES_E_ARG, "es_causal_conv_workspace: null result");
    es::ConvPlan P;
    const es_status st = es::plan_conv("es_causal_conv_workspace", args, grads, false, &P);
    if (st == ES_OK) *bytes = P.bytes;
    return st;
}

es_status es_plan_causal_conv(const es_causal_conv_args* args, const es_causal_conv_grads* grads, es_plan_info* info) {
    es::ConvPlan P;
    const es_status st = es::plan_conv("es_plan_causal_conv", args, grads, false, &P);
    if (st == ES_OK)
        es::fill_info(info, P.L.B, P.L.T, P.L.C, P.L.taps, P.L.B * P.L.T * P.L.C, P.empty ? ES_PATH_EMPTY : ES_PATH_GENERIC);
    return st;
}

es_status es_causal_conv_step(const es_causal_conv_args* args, es_stream_t stream) {
    const char* fn = "es_causal_conv_step";
    es::ConvPlan P;
    const es_status st = es::plan_conv(fn, args, nullptr, true, &P);
    if (st != ES_OK || P.empty) return st;
    P.L.stream = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = es::launch_conv_step(P.L);
    if (e != cudaSuccess) return es::cuda_fail(fn, e);
    es::count_launch();
    return ES_OK;
}

es_status es_selective_scan(const es_selective_scan_args* args, es_stream_t stream) {
    const char* fn = "es_selective_scan";
    es::ScanPlan P;
    es_status st = es::plan_scan(fn, args, nullptr, false, &P);
    if (st != ES_OK || P.empty) return st;
    if ((st = es::check_workspace(fn, args->workspace, args->workspace_bytes, P.bytes)) != ES_OK) return st;
    es::ScanLaunch& L = P.S.f;
    L.stream = reinterpret_cast<cudaStream_t>(stream);
    if (L.segs > 1) {
        L.seg_state = es::at(args->workspace, P.seg_state);
        L.seg_sum = es::at(args->workspace, P.seg_sum);
        if (P.first > 0) L.first = es::at(args->workspace, P.first - 1);
    }
    int n = 0;
    const cudaError_t e = es::launch_scan(L, false, &n);
    if (e != cudaSuccess) return es::cuda_fail(fn, e);
    es::count_launch(n);
    return ES_OK;
}

es_status es_selective_scan_backward(const es_selective_scan_args* args, const es_selective_scan_grads* grads, es_stream_t stream) {
    const char* fn = "es_selective_scan_backward";
    if (grads == nullptr) return es::api_fail(ES_E_ARG, "%s: null gradients", fn);
    es::ScanPlan P;
    es_status st = es::plan_scan(fn, args, grads, false, &P);
    if (st != ES_OK) return st;
    es::ScanBackward& S = P.S;
    es::ScanLaunch& L = S.f;
    L.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (P.empty) {       // no rows: the weights' gradients are sums of nothing
        if (L.C > 0 && ((S.ga != nullptr && (e = cudaMemsetAsync(S.ga, 0, L.C * L.N * 4, L.stream)) != cudaSuccess) ||
                        (S.gskip != nullptr && (e = cudaMemsetAsync(S.gskip, 0, L.C * 4, L.stream)) != cudaSuccess) ||
                        (S.gbias != nullptr && (e = cudaMemsetAsync(S.gbias, 0, L.C * 4, L.stream)) != cudaSuccess)))
            return es::cuda_fail(fn, e);
        // no channels: those of b and c too
        if (L.C == 0 && L.B > 0 && L.T > 0) {
            if ((e = es::launch_scan_sum_bc(S)) != cudaSuccess) return es::cuda_fail(fn, e);
            es::count_launch();
        }
        return ES_OK;
    }
    if ((st = es::check_workspace(fn, args->workspace, args->workspace_bytes, P.bytes)) != ES_OK) return st;
    void* const ws = args->workspace;
    L.seg_state = es::at(ws, P.seg_state);
    L.seg_sum = es::at(ws, P.seg_sum);
    S.part_bc = es::at(ws, P.part_bc);
    S.part_c = es::at(ws, P.part_c);
    int n = 0;
    if (P.find) {
        L.kept = es::at(ws, P.kept);
        es::ScanLaunch F = L;
        F.segs = P.fwd_segs;
        F.seg_chunks = P.fwd_seg_chunks;
        if ((e = es::launch_scan(F, true, &n)) != cudaSuccess) return es::cuda_fail(fn, e);
        es::count_launch(n);
    }
    if ((e = es::launch_scan_backward(S, &n)) != cudaSuccess) return es::cuda_fail(fn, e);
    es::count_launch(n);
    return ES_OK;
}

es_status es_selective_scan_workspace(const es_selective_scan_args* args, const es_selective_scan_grads* grads, size_t* bytes) {
    if (bytes == nullptr) return es::api_fail(ES_E_ARG, "es_selective_scan_workspace: null result");
    es::ScanPlan P;
    const es_status st = es::plan_scan("es_selective_scan_workspace", args, grads, false, &P);
    if (st == ES_OK) *bytes = P.bytes;
    return st;
}

es_status es_selective_scan_checkpoints(const es_selective_scan_args* args, size_t* bytes) {
    const char* fn = "es_selective_scan_checkpoints";
    if (bytes == nullptr) return es::api_fail(ES_E_ARG, "%s: null result", fn);
    if (args == nullptr) return es::api_fail(ES_E_ARG, "%s: null arguments", fn);
    es_selective_scan_args a = *args;
    a.checkpoints = nullptr;
    es::ScanPlan P;
    const es_status st = es::plan_scan(fn, &a, nullptr, false, &P);
    if (st == ES_OK) *bytes = P.kept_bytes;
    return st;
}

es_status es_plan_selective_scan(const es_selective_scan_args* args, const es_selective_scan_grads* grads, es_plan_info* info) {
    es::ScanPlan P;
    const es_status st = es::plan_scan("es_plan_selective_scan", args, grads, false, &P);
    if (st == ES_OK) {
        const es::ScanLaunch& L = P.S.f;
        es::fill_info(info, L.B, L.T, L.C, L.N, L.B * L.T * L.C, P.empty ? ES_PATH_EMPTY : ES_PATH_GENERIC);
    }
    return st;
}

es_status es_selective_scan_step(const es_selective_scan_args* args, es_stream_t stream) {
    const char* fn = "es_selective_scan_step";
    es::ScanPlan P;
    const es_status st = es::plan_scan(fn, args, nullptr, true, &P);
    if (st != ES_OK || P.empty) return st;
    P.S.f.stream = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = es::launch_scan_step(P.S.f);
    if (e != cudaSuccess) return es::cuda_fail(fn, e);
    es::count_launch();
    return ES_OK;
}

es_status es_group_norm(const es_group_norm_args* args, es_stream_t stream) { return es::run_norm("es_group_norm", args, nullptr, stream); }

es_status es_group_norm_backward(const es_group_norm_args* args, const es_group_norm_grads* grads, es_stream_t stream) {
    if (grads == nullptr) return es::api_fail(ES_E_ARG, "es_group_norm_backward: null gradients");
    return es::run_norm("es_group_norm_backward", args, grads, stream);
}

es_status es_group_norm_workspace(const es_group_norm_args* args, const es_group_norm_grads* grads, size_t* bytes) {
    if (bytes == nullptr) return es::api_fail(ES_E_ARG, "es_group_norm_workspace: null result");
    es::NormPlan P;
    const es_status st = es::plan_norm("es_group_norm_workspace", args, grads, &P);
    if (st == ES_OK) *bytes = P.bytes;
    return st;
}

es_status es_plan_group_norm(const es_group_norm_args* args, const es_group_norm_grads* grads, es_plan_info* info) {
    es::NormPlan P;
    const es_status st = es::plan_norm("es_plan_group_norm", args, grads, &P);
    if (st == ES_OK)
        es::fill_info(info, P.L.B, P.L.T, P.L.H, P.L.D, P.L.B * P.L.T * P.L.H * P.L.D, P.empty ? ES_PATH_EMPTY : ES_PATH_GENERIC);
    return st;
}

}  // extern "C"
