// es_attn_api.cu -- entry points of linear attention and of the query/key norm
// with rotation (es.h): validation, the runs a call consists of, workspaces,
// kernel choice and launch.
#include <cmath>

#include "es.h"
#include "es_attn.h"
#include "es_internal.h"
#include "es_views.h"

namespace es {
namespace {

AttnOperand operand(const es_heads& v, int64_t H) {
    return AttnOperand{v.data, v.stride_b, v.stride_t, v.stride_h, v.heads > 0 ? static_cast<int>(H / v.heads) : 1};
}

struct AttnPlan {
    AttnLaunch L;
    int path;
    bool empty;
    // backward: byte offsets into the workspace
    size_t seg_states, seg_decays, dots_q, dots_k, states_q, states_k, ends, partial, fold_q, fold_k, fold_v, bytes;
    int slices_k;                // slices of the runs that give the dots (key-wide outputs)
};

// Segments a sequence is cut into.  One CTA runs one (batch row, head, run, and on
// the direct path slice); with fewer of them than the GPU has places, the chunks
// are shared out among more CTAs, which costs a pass for the states between
// segments and two launches.  In hundredths of a main pass's chunk: on the tensor
// cores (one CTA an SM) 42 a chunk (113 of 268 us for 65536 tokens x 16 heads of
// 128) and 500 for the launches; on the direct path (four CTAs an SM at widths to
// 64, three to 128, two above; chunks of 32 tokens, 5 to 7 us each) 65 and 600.
// f32, whole against in segments: 4000 tokens x 4 heads of 128 851 and 107 us,
// 256 tokens x 4 heads of 64 48 and 24, 8 x 200 x 8 heads of 64 44 and 46,
// 8 x 1000 x 16 heads of 64 221 and 227.  With two CTAs an SM at all widths
// 4 x 1000 x 16 heads of 64 took 146 us instead of 120.
int segments(bool tensor, int64_t width, int64_t ctas, int64_t chunks, int64_t* seg_chunks) {
    const int64_t most = kSms * (tensor ? 1 : width <= 64 ? 4 : width <= 128 ? 3 : 2) / ctas;
    if (most < 2) return 1;
    const int64_t each = (chunks + most - 1) / most;
    if ((tensor ? 142 : 165) * each + (tensor ? 500 : 600) >= 100 * chunks) return 1;
    *seg_chunks = each;
    return static_cast<int>((chunks + each - 1) / each);
}

es_status plan_attn(const char* fn, const es_linear_attention_args* a, const es_linear_attention_grads* g, bool step,
                    AttnPlan* P) {
    if (a == nullptr) return api_fail(ES_E_ARG, "%s: null arguments", fn);
    if (a->dtype != ES_F32 && a->dtype != ES_BF16)
        return api_fail(ES_E_DIM_002, "E-DIM-002 %s: dtype %lld is neither f32 nor bf16", fn, static_cast<long long>(a->dtype));
    const int64_t B = a->batch, T = a->length, H = a->heads, dk = a->key_dim, dv = a->value_dim;
    if (B < 0 || T < 0 || H < 0) return api_fail(ES_E_DIM_001, "E-DIM-001 %s: a negative dimension", fn);
    if (dk < 1 || dk > kAttnMaxDim || dv < 1 || dv > kAttnMaxDim)
        return api_fail(ES_E_UNSUPPORTED, "%s: head widths %lld and %lld; 1..%d are supported", fn, static_cast<long long>(dk),
                        static_cast<long long>(dv), kAttnMaxDim);
    if (step && T != 1) return api_fail(ES_E_DIM_001, "E-DIM-001 %s: a step is one token, not %lld", fn, static_cast<long long>(T));
    if (step && a->lengths != nullptr) return api_fail(ES_E_ARG, "%s: a step takes no lengths", fn);
    const es_heads* ops[3] = {&a->q, &a->k, &a->v};
    const char* names[3] = {"q", "k", "v"};
    for (int i = 0; i < 3; ++i)
        if (H > 0 && (ops[i]->heads < 1 || H % ops[i]->heads != 0))
            return api_fail(ES_E_DIM_001, "E-DIM-001 %s: %lld heads of `%s` do not divide the %lld heads", fn,
                            static_cast<long long>(ops[i]->heads), names[i], static_cast<long long>(H));
    int64_t bh, x;
    if (__builtin_mul_overflow(B, H, &bh) || bh > 0x7fffffff)
        return api_fail(ES_E_UNSUPPORTED, "%s: %lld rows of %lld heads are too many", fn, static_cast<long long>(B),
                        static_cast<long long>(H));
    if (T >= (int64_t(1) << 31) || __builtin_mul_overflow(bh, T, &x) || __builtin_mul_overflow(x, int64_t(kAttnMaxDim) * 8, &x))
        return api_fail(ES_E_UNSUPPORTED, "%s: too many tokens", fn);
    if (!std::isfinite(a->scale) || static_cast<float>(a->scale) == 0.0f || !std::isfinite(static_cast<float>(a->scale)))
        return api_fail(ES_E_ARG, "%s: scale %g; it must be finite and not zero", fn, a->scale);
    const int64_t size = a->dtype == ES_BF16 ? 2 : 4;
    Span in[12], out[8];
    int n_in = 0, n_out = 0;
    es_status st;
    const int64_t dims[3] = {dk, dk, dv};
    for (int i = 0; i < 3; ++i)
        if ((st = check_view(fn, names[i], *ops[i], B, T, dims[i], size, false, &in[n_in++])) != ES_OK) return st;
    const int64_t n_state = bh * dk * dv;
    const bool backward = g != nullptr;
    Span init, fin;
    if ((st = check_dense(fn, "initial_state", a->initial_state, n_state, &init)) != ES_OK) return st;
    if ((st = check_dense(fn, "final_state", a->final_state, n_state, &fin)) != ES_OK) return st;
    in[n_in++] = init;
    if (a->log_decay != nullptr) {
        if (a->decay_b < 0 || a->decay_t < 0 || a->decay_h < 0)
            return api_fail(ES_E_ARG, "%s: `log_decay` has a negative stride", fn);
        const es_heads v{const_cast<float*>(a->log_decay), a->decay_per_head ? 0 : a->decay_b,
                         a->decay_per_head || step ? 0 : a->decay_t, a->decay_h, H};
        if ((st = check_view(fn, "log_decay", v, B, T, 1, 4, false, &in[n_in++])) != ES_OK) return st;
    }
    if ((st = check_dense(fn, "lengths", a->lengths, B, &in[n_in])) != ES_OK) return st;
    ++n_in;
    if (!backward) {
        if (a->out.heads != H)
            return api_fail(ES_E_DIM_001, "E-DIM-001 %s: `out` has %lld heads, not %lld", fn,
                            static_cast<long long>(a->out.heads), static_cast<long long>(H));
        if ((st = check_view(fn, "out", a->out, B, T, dv, size, true, &out[n_out++])) != ES_OK) return st;
        if (step && n_state > 0 && (a->initial_state == nullptr || a->final_state == nullptr))
            return api_fail(ES_E_ARG, "%s: a step needs the state and a place for the new one", fn);
        // the last state may take the first one's place
        out[n_out++] = fin;
        if (a->final_state == a->initial_state) in[3].bytes = 0;
    } else {
        const es_heads* gs[4] = {&g->grad_out, &g->grad_q, &g->grad_k, &g->grad_v};
        const char* gn[4] = {"grad_out", "grad_q", "grad_k", "grad_v"};
        const int64_t want[4] = {H, a->q.heads, a->k.heads, a->v.heads}, gd[4] = {dv, dk, dk, dv};
        for (int i = 0; i < 4; ++i) {
            if (gs[i]->heads != want[i])
                return api_fail(ES_E_DIM_001, "E-DIM-001 %s: `%s` has %lld heads, not %lld", fn, gn[i],
                                static_cast<long long>(gs[i]->heads), static_cast<long long>(want[i]));
            if ((st = check_view(fn, gn[i], *gs[i], B, T, gd[i], size, i > 0, i > 0 ? &out[n_out] : &in[n_in])) != ES_OK) return st;
            ++(i > 0 ? n_out : n_in);
        }
        if ((st = check_dense(fn, "grad_final_state", g->grad_final_state, n_state, &in[n_in])) != ES_OK) return st;
        ++n_in;
        if ((st = check_dense(fn, "grad_initial_state", g->grad_initial_state, n_state, &out[n_out])) != ES_OK) return st;
        ++n_out;
        if (g->grad_log_decay != nullptr && a->log_decay == nullptr)
            return api_fail(ES_E_ARG, "%s: a gradient of `log_decay`, which is null", fn);
        if ((st = check_dense(fn, "grad_log_decay", g->grad_log_decay, a->decay_per_head ? H : bh * T, &out[n_out])) != ES_OK) return st;
        ++n_out;
    }
    if ((st = check_outputs(fn, in, n_in, out, n_out)) != ES_OK) return st;

    *P = AttnPlan{};
    P->empty = bh == 0;
    AttnLaunch& L = P->L;
    L.bf16 = a->dtype == ES_BF16;
    L.B = B;
    L.T = T;
    L.H = static_cast<int>(H);
    L.g = a->log_decay;
    L.gb = a->decay_per_head ? 0 : a->decay_b;
    L.gt = a->decay_per_head || step ? 0 : a->decay_t;
    L.gh = a->decay_h;
    L.lengths = a->lengths;
    if (P->empty) {
        P->path = ES_PATH_EMPTY;
        return ES_OK;
    }
    const float scale = static_cast<float>(a->scale);
    AttnRun& f = L.run[0];
    if (!backward) {
        L.runs = 1;
        f.x = operand(a->q, H);
        f.y = operand(a->k, H);
        f.z = operand(a->v, H);
        f.out = a->out.data;
        f.ob = a->out.stride_b;
        f.ot = a->out.stride_t;
        f.oh = a->out.stride_h;
        f.init = a->initial_state;
        f.fin = a->final_state;
        f.sa = dv;
        f.sc = 1;
        f.update_scale = 1.0f;
        f.read_scale = f.out_scale = scale;
        f.state_result = 1;
        f.dx = static_cast<int>(dk);
        f.dz = static_cast<int>(dv);
    } else {
        L.runs = 3;
        AttnRun &rq = L.run[0], &rv = L.run[1], &rk = L.run[2];
        const AttnOperand q = operand(a->q, H), k = operand(a->k, H), v = operand(a->v, H), go = operand(g->grad_out, H);
        auto fill = [&](AttnRun& r, const AttnOperand& x, const AttnOperand& y, const AttnOperand& z, const es_heads& o, int64_t dx,
                        int64_t dz, bool turned) {
            r.x = x;
            r.y = y;
            r.z = z;
            r.out = o.data;
            r.ob = o.stride_b;
            r.ot = o.stride_t;
            r.oh = o.stride_h;
            r.sa = turned ? 1 : dv;
            r.sc = turned ? dv : 1;
            r.update_scale = 1.0f;
            r.read_scale = r.out_scale = scale;
            r.dx = static_cast<int>(dx);
            r.dz = static_cast<int>(dz);
        };
        fill(rq, go, v, k, g->grad_q, dv, dk, true);
        rq.init = a->initial_state;
        fill(rv, k, q, go, g->grad_v, dk, dv, false);
        fill(rk, v, go, q, g->grad_k, dv, dk, true);
        rv.reverse = rk.reverse = 1;
        rv.init = rk.init = g->grad_final_state;
        // the states of these are the gradients of the states
        rv.update_scale = rk.update_scale = scale;
        rv.read_scale = rk.read_scale = 1.0f;
        rv.fin = g->grad_initial_state;
        rv.state_result = 1;
    }
    // the path: every run's operands have to suit the tensor-core kernel's loads
    bool tensor = L.bf16 && T > 0 && !step;
    for (int r = 0; r < L.runs && tensor; ++r) {
        const AttnRun& u = L.run[r];
        tensor = attn_tc_operand_ok(u.x, L.H / u.x.div, u.dx, T, B) && attn_tc_operand_ok(u.y, L.H / u.y.div, u.dx, T, B) &&
                 attn_tc_operand_ok(u.z, L.H / u.z.div, u.dz, T, B);
    }
    const int forced = api_path_override();
    if (forced != ES_PATH_AUTO && forced != ES_PATH_GENERIC && !(forced == ES_PATH_TENSOR && tensor))
        return api_fail(ES_E_UNSUPPORTED, "%s: the forced kernel path %d cannot serve this call", fn, forced);
    P->path = tensor && forced != ES_PATH_GENERIC ? ES_PATH_TENSOR : ES_PATH_GENERIC;

    // workspace
    const int64_t chunk = P->path == ES_PATH_TENSOR ? kAttnTcChunk : kAttnChunk;
    L.n_anchors = (T + kAttnAnchorTokens - 1) / kAttnAnchorTokens;
    L.n_segs = 1;
    const int64_t chunks = (T + chunk - 1) / chunk;
    L.seg_chunks = chunks > 0 ? chunks : 1;
    const int64_t slices = ((dk > dv ? dk : dv) + kAttnSlice - 1) / kAttnSlice;
    if (chunks > 1 && !step)
        L.n_segs = segments(P->path == ES_PATH_TENSOR, dk > dv ? dk : dv, bh * L.runs * (P->path == ES_PATH_TENSOR ? 1 : slices),
                            chunks, &L.seg_chunks);
    P->slices_k = static_cast<int>((dk + kAttnSlice - 1) / kAttnSlice);
    size_t at = 0;
    if (L.n_segs > 1) {
        P->seg_states = take(&at, 4 * L.runs * bh * L.n_segs * dk * dv);
        P->seg_decays = take(&at, 4 * L.runs * bh * L.n_segs);
    }
    if (backward && T > 0) {
        if (g->grad_log_decay != nullptr) {
            P->dots_q = take(&at, 4 * P->slices_k * bh * T);
            P->dots_k = take(&at, 4 * P->slices_k * bh * T);
            P->states_q = take(&at, 4 * bh * L.n_anchors * dk * dv);
            P->states_k = take(&at, 4 * bh * L.n_anchors * dk * dv);
            P->ends = take(&at, 4 * bh * (L.n_anchors + 1));
            P->partial = take(&at, 4 * bh * L.n_anchors);
        }
        if (a->q.heads < H) P->fold_q = take(&at, 4 * bh * T * dk);
        if (a->k.heads < H) P->fold_k = take(&at, 4 * bh * T * dk);
        if (a->v.heads < H) P->fold_v = take(&at, 4 * bh * T * dv);
    }
    P->bytes = at;
    return check_outputs(fn, in, n_in, out, n_out, a->workspace, at);
}

es_status device_of(AttnLaunch* L, es_stream_t stream) {
    int dev = 0;
    DeviceState* ds = nullptr;
    es_status st = api_device(&dev, &ds);
    if (st != ES_OK) return st;
    L->status = ds->status;
    L->wait_ns = api_wait_ns();
    L->drop_tile = api_drop_tile();
    L->stream = reinterpret_cast<cudaStream_t>(stream);
    return ES_OK;
}

// one launch of P's path over `runs` of L
es_status launch_runs(const char* fn, const AttnPlan& P, AttnLaunch L, void* workspace) {
    cudaError_t e;
    int n = 0;
    if (L.n_segs > 1) {
        L.seg_states = reinterpret_cast<float*>(static_cast<char*>(workspace) + P.seg_states);
        L.seg_decays = reinterpret_cast<float*>(static_cast<char*>(workspace) + P.seg_decays);
    }
    if (P.path == ES_PATH_TENSOR) {
        es_status st = api_encoder(&L.encode);
        if (st != ES_OK) return st;
        const char* msg = nullptr;
        e = launch_attn_tc(L, &n, &msg);
        if (msg != nullptr) return api_fail(ES_E_CUDA, "%s: %s", fn, msg);
    } else {
        e = launch_attn_direct(L, &n);
    }
    if (e != cudaSuccess) return cuda_fail(fn, e);
    count_launch(n);
    return ES_OK;
}

es_status run_backward(const char* fn, const es_linear_attention_args* a, const es_linear_attention_grads* g, AttnPlan& P) {
    AttnLaunch& L = P.L;
    char* ws = static_cast<char*>(a->workspace);
    const int64_t H = a->heads;
    const int dk = static_cast<int>(a->key_dim), dv = static_cast<int>(a->value_dim);
    cudaError_t e;
    AttnRun &rq = L.run[0], &rv = L.run[1], &rk = L.run[2];
    const bool decay = g->grad_log_decay != nullptr && L.T > 0;
    if (decay) {
        rq.w = operand(a->q, H);
        rq.dots = reinterpret_cast<float*>(ws + P.dots_q);
        rq.anchors = reinterpret_cast<float*>(ws + P.states_q);
        rk.w = operand(a->k, H);
        rk.dots = reinterpret_cast<float*>(ws + P.dots_k);
        rk.anchors = reinterpret_cast<float*>(ws + P.states_k);
    }
    AttnFold fold[3];
    int folds = 0;
    auto shared = [&](AttnRun& r, const es_heads& o, size_t at, int d) {
        if (o.heads == H || L.T == 0) return;
        AttnFold& F = fold[folds++];
        F = AttnFold{reinterpret_cast<const float*>(ws + at), r.out, r.ob, r.ot, r.oh, L.bf16, L.B, L.T,
                     static_cast<int>(o.heads), static_cast<int>(H / o.heads), d, L.stream};
        r.out = ws + at;
        r.out_f32 = 1;
        r.oh = d;
        r.ot = H * d;
        r.ob = L.T * H * d;
    };
    shared(rq, g->grad_q, P.fold_q, dk);
    shared(rv, g->grad_v, P.fold_v, dv);
    shared(rk, g->grad_k, P.fold_k, dk);
    const es_status st = launch_runs(fn, P, L, a->workspace);
    if (st != ES_OK) return st;
    if (decay) {
        AttnDecayGrad D{};
        D.dots_q = rq.dots;
        D.dots_k = rk.dots;
        D.states_q = rq.anchors;
        D.states_k = rk.anchors;
        D.initial = a->initial_state;
        D.grad_initial = g->grad_initial_state;
        D.ends = reinterpret_cast<float*>(ws + P.ends);
        D.slices = P.slices_k;
        D.size = static_cast<int64_t>(dk) * dv;
        D.B = L.B;
        D.T = L.T;
        D.H = L.H;
        D.lengths = L.lengths;
        D.n = L.n_anchors;
        D.stream = L.stream;
        if (a->decay_per_head) {
            D.partial = reinterpret_cast<float*>(ws + P.partial);
            D.grad_h = g->grad_log_decay;
        } else {
            D.grad = g->grad_log_decay;
        }
        int n = 0;
        if ((e = launch_attn_decay_grad(D, &n)) != cudaSuccess) return cuda_fail(fn, e);
        count_launch(n);
    } else if (g->grad_log_decay != nullptr && a->decay_per_head) {
        // no tokens: a sum of nothing
        if ((e = cudaMemsetAsync(g->grad_log_decay, 0, H * 4, L.stream)) != cudaSuccess) return cuda_fail(fn, e);
    }
    if (folds > 0) {
        if ((e = launch_attn_folds(fold, folds)) != cudaSuccess) return cuda_fail(fn, e);
        count_launch();
    }
    return ES_OK;
}

// ---------------------------------------------------------------------------
// norm and rotation

struct RotatePlan {
    RotateLaunch L;
    bool empty;
    size_t bytes;
};

es_status plan_rotate(const char* fn, const es_qk_norm_rotate_args* a, const es_qk_norm_rotate_grads* g, RotatePlan* P) {
    if (a == nullptr) return api_fail(ES_E_ARG, "%s: null arguments", fn);
    if ((a->dtype != ES_F32 && a->dtype != ES_BF16) || (a->weight_dtype != ES_F32 && a->weight_dtype != ES_BF16))
        return api_fail(ES_E_DIM_002, "E-DIM-002 %s: dtypes %lld (weights %lld): f32 or bf16 are taken", fn,
                        static_cast<long long>(a->dtype), static_cast<long long>(a->weight_dtype));
    const int64_t B = a->batch, T = a->length, d = a->dim;
    if (B < 0 || T < 0 || a->q.heads < 0 || a->k.heads < 0) return api_fail(ES_E_DIM_001, "E-DIM-001 %s: a negative dimension", fn);
    if (d < 1 || d > kAttnMaxDim)
        return api_fail(ES_E_UNSUPPORTED, "%s: heads of %lld values; 1..%d are supported", fn, static_cast<long long>(d), kAttnMaxDim);
    if (a->turned < 0 || a->turned > d || a->turned % 2 != 0)
        return api_fail(ES_E_DIM_001, "E-DIM-001 %s: %lld of %lld values to turn: an even number of them is wanted", fn,
                        static_cast<long long>(a->turned), static_cast<long long>(d));
    if (!(a->eps >= 0) || !std::isfinite(a->eps)) return api_fail(ES_E_ARG, "%s: eps %g", fn, a->eps);
    if (a->q.heads > (1 << 20) || a->k.heads > (1 << 20)) return api_fail(ES_E_UNSUPPORTED, "%s: too many heads", fn);
    int64_t rows, x;
    if (__builtin_mul_overflow(B, T, &rows) || __builtin_mul_overflow(rows, int64_t(1) << 30, &x))
        return api_fail(ES_E_UNSUPPORTED, "%s: too many tokens", fn);
    const int64_t size = a->dtype == ES_BF16 ? 2 : 4, wsize = a->weight_dtype == ES_BF16 ? 2 : 4;
    const bool backward = g != nullptr;
    Span in[18], out[4];
    int n_in = 0, n_out = 0;
    es_status st;
    const es_heads* xs[2] = {&a->q, &a->k};
    const es_heads* os[2] = {&a->q_out, &a->k_out};
    const es_heads* gs[2] = {backward ? &g->grad_q_out : nullptr, backward ? &g->grad_k_out : nullptr};
    const void* ws[2] = {a->q_weight, a->k_weight};
    void* gw[2] = {backward ? g->grad_q_weight : nullptr, backward ? g->grad_k_weight : nullptr};
    const char* xn[2] = {"q", "k"};
    const char* on[2] = {backward ? "grad_q" : "q_out", backward ? "grad_k" : "k_out"};
    const char* gn[2] = {"grad_q_out", "grad_k_out"};
    const char* wn[2] = {"q_weight", "k_weight"};
    const char* gwn[2] = {"grad_q_weight", "grad_k_weight"};
    Span xsp[2], osp[2], gsp[2];
    for (int i = 0; i < 2; ++i) {
        if ((st = check_view(fn, xn[i], *xs[i], B, T, d, size, false, &xsp[i])) != ES_OK) return st;
        if (os[i]->heads != xs[i]->heads || (backward && gs[i]->heads != xs[i]->heads))
            return api_fail(ES_E_DIM_001, "E-DIM-001 %s: `%s` has %lld heads; its result or gradient another number", fn, xn[i],
                            static_cast<long long>(xs[i]->heads));
        if ((st = check_view(fn, on[i], *os[i], B, T, d, size, true, &osp[i])) != ES_OK) return st;
        if (backward && (st = check_view(fn, gn[i], *gs[i], B, T, d, size, false, &gsp[i])) != ES_OK) return st;
        if (reinterpret_cast<uintptr_t>(ws[i]) % wsize != 0 || reinterpret_cast<uintptr_t>(gw[i]) % wsize != 0)
            return api_fail(ES_E_ARG, "%s: `%s` or its gradient is not aligned to its elements", fn, wn[i]);
        in[n_in++] = Span{wn[i], ws[i], ws[i] == nullptr ? 0 : d * wsize};
        if (gw[i] != nullptr) out[n_out++] = Span{gwn[i], gw[i], d * wsize};
    }
    const int64_t half = a->turned / 2;
    if (half > 0 && rows > 0) {
        if (a->table_rows < 1) return api_fail(ES_E_DIM_001, "E-DIM-001 %s: tables without rows", fn);
        if (__builtin_mul_overflow(a->table_rows, half * 4, &x)) return api_fail(ES_E_UNSUPPORTED, "%s: tables too large", fn);
        if (a->cos == nullptr || a->sin == nullptr) return api_fail(ES_E_ARG, "%s: null `cos` or `sin`", fn);
        if ((st = check_dense(fn, "cos", a->cos, a->table_rows * half, &in[n_in])) != ES_OK) return st;
        ++n_in;
        if ((st = check_dense(fn, "sin", a->sin, a->table_rows * half, &in[n_in])) != ES_OK) return st;
        ++n_in;
    }
    if (a->positions != nullptr && rows > 0) {
        const int64_t ps = a->positions_64 ? 8 : 4;
        const es_heads v{const_cast<void*>(a->positions), a->position_b, a->position_t, 0, 1};
        if ((st = check_view(fn, "positions", v, B, T, 1, ps, false, &in[n_in])) != ES_OK) return st;
        ++n_in;
    }
    if ((st = check_outputs(fn, in, n_in, out, n_out)) != ES_OK) return st;
    // each side's result may take its own input's (its gradient's) place, or lie beside the others in one tensor
    auto same = [](const es_heads& p, const es_heads& q) {
        return p.data == q.data && p.stride_b == q.stride_b && p.stride_t == q.stride_t && p.stride_h == q.stride_h;
    };
    for (int i = 0; i < 2; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlap(osp[i], in[j])) return api_fail(ES_E_ARG, "%s: `%s` overlaps `%s`", fn, on[i], in[j].name);
        for (int j = 0; j < n_out; ++j)
            if (overlap(osp[i], out[j])) return api_fail(ES_E_ARG, "%s: `%s` overlaps `%s`", fn, on[i], out[j].name);
        for (int j = 0; j < 2; ++j) {
            if (overlap(osp[i], xsp[j]) && !(i == j && same(*os[i], *xs[j])) && !side_by_side(*os[i], *xs[j], d, d, size, B, T))
                return api_fail(ES_E_ARG, "%s: `%s` overlaps `%s`", fn, on[i], xn[j]);
            if (backward && overlap(osp[i], gsp[j]) && !(i == j && same(*os[i], *gs[j])) &&
                !side_by_side(*os[i], *gs[j], d, d, size, B, T))
                return api_fail(ES_E_ARG, "%s: `%s` overlaps `%s`", fn, on[i], gn[j]);
            for (int o = 0; o < n_out; ++o)
                if (overlap(out[o], xsp[j]) || (backward && overlap(out[o], gsp[j])))
                    return api_fail(ES_E_ARG, "%s: `%s` overlaps an input", fn, out[o].name);
        }
    }
    if (overlap(osp[0], osp[1]) && !side_by_side(*os[0], *os[1], d, d, size, B, T))
        return api_fail(ES_E_ARG, "%s: `%s` overlaps `%s`", fn, on[0], on[1]);

    *P = RotatePlan{};
    RotateLaunch& L = P->L;
    for (int i = 0; i < 2; ++i) {
        RotateSide& S = L.side[i];
        S.x = xs[i]->data;
        S.xb = xs[i]->stride_b;
        S.xt = xs[i]->stride_t;
        S.xh = xs[i]->stride_h;
        S.out = os[i]->data;
        S.ob = os[i]->stride_b;
        S.ot = os[i]->stride_t;
        S.oh = os[i]->stride_h;
        if (backward) {
            S.g = gs[i]->data;
            S.gb = gs[i]->stride_b;
            S.gt = gs[i]->stride_t;
            S.gh = gs[i]->stride_h;
        }
        S.w = ws[i];
        S.gw = gw[i];
        S.heads = static_cast<int>(xs[i]->heads);
    }
    L.bf16 = a->dtype == ES_BF16;
    L.w_bf16 = a->weight_dtype == ES_BF16;
    L.B = B;
    L.T = T;
    L.d = static_cast<int>(d);
    L.turned = static_cast<int>(a->turned);
    L.neighbours = a->neighbours ? 1 : 0;
    L.eps = static_cast<float>(a->eps);
    L.cos = a->cos;
    L.sin = a->sin;
    L.rows = half > 0 ? a->table_rows : 1;
    L.positions = a->positions;
    L.pos64 = a->positions_64 ? 1 : 0;
    L.pb = a->position_b;
    L.pt = a->position_t;
    L.backward = backward ? 1 : 0;
    P->empty = rows == 0 || a->q.heads + a->k.heads == 0;
    if (rows >= 0x7ff00000 || rotate_units(L, 0) >= 0x7ff00000 || rotate_units(L, 1) >= 0x7ff00000)
        return api_fail(ES_E_UNSUPPORTED, "%s: %lld tokens are too many", fn, static_cast<long long>(rows));
    if (!P->empty && (gw[0] != nullptr || gw[1] != nullptr))
        P->bytes = static_cast<size_t>(rotate_blocks(L, 0) + rotate_blocks(L, 1)) * d * 4;
    for (int i = 0; i < 2; ++i) {
        in[n_in++] = xsp[i];
        in[n_in++] = osp[i];
        if (backward) in[n_in++] = gsp[i];
    }
    return check_outputs(fn, in, n_in, out, n_out, a->workspace, P->bytes);
}

es_status run_rotate(const char* fn, const es_qk_norm_rotate_args* a, const es_qk_norm_rotate_grads* g, es_stream_t stream) {
    RotatePlan P;
    es_status st = plan_rotate(fn, a, g, &P);
    if (st != ES_OK) return st;
    RotateLaunch& L = P.L;
    L.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (P.empty) {
        for (int i = 0; i < 2; ++i)       // no rows: the weights' gradients are sums of nothing
            if (L.side[i].gw != nullptr &&
                (e = cudaMemsetAsync(L.side[i].gw, 0, L.d * (L.w_bf16 ? 2 : 4), L.stream)) != cudaSuccess)
                return cuda_fail(fn, e);
        return ES_OK;
    }
    if ((st = check_workspace(fn, a->workspace, a->workspace_bytes, P.bytes)) != ES_OK) return st;
    L.partial = static_cast<float*>(a->workspace);
    int n = 0;
    if ((e = launch_rotate(L, &n)) != cudaSuccess) return cuda_fail(fn, e);
    count_launch(n);
    return ES_OK;
}

}  // namespace
}  // namespace es

extern "C" {

es_status es_linear_attention(const es_linear_attention_args* args, es_stream_t stream) {
    const char* fn = "es_linear_attention";
    es::AttnPlan P;
    es_status st = es::plan_attn(fn, args, nullptr, false, &P);
    if (st != ES_OK || P.empty) return st;
    if ((st = es::check_workspace(fn, args->workspace, args->workspace_bytes, P.bytes)) != ES_OK) return st;
    if ((st = es::device_of(&P.L, stream)) != ES_OK) return st;
    return es::launch_runs(fn, P, P.L, args->workspace);
}

es_status es_linear_attention_backward(const es_linear_attention_args* args, const es_linear_attention_grads* grads,
                                       es_stream_t stream) {
    const char* fn = "es_linear_attention_backward";
    if (grads == nullptr) return es::api_fail(ES_E_ARG, "%s: null gradients", fn);
    es::AttnPlan P;
    es_status st = es::plan_attn(fn, args, grads, false, &P);
    if (st != ES_OK) return st;
    if (P.empty) {
        if (grads->grad_log_decay != nullptr && args->decay_per_head && args->heads > 0) {
            const cudaError_t e = cudaMemsetAsync(grads->grad_log_decay, 0, args->heads * 4, reinterpret_cast<cudaStream_t>(stream));
            if (e != cudaSuccess) return es::cuda_fail(fn, e);
        }
        return ES_OK;
    }
    if ((st = es::check_workspace(fn, args->workspace, args->workspace_bytes, P.bytes)) != ES_OK) return st;
    if ((st = es::device_of(&P.L, stream)) != ES_OK) return st;
    return es::run_backward(fn, args, grads, P);
}

es_status es_linear_attention_workspace(const es_linear_attention_args* args, const es_linear_attention_grads* grads,
                                        size_t* bytes) {
    if (bytes == nullptr) return es::api_fail(ES_E_ARG, "es_linear_attention_workspace: null result");
    es::AttnPlan P;
    const es_status st = es::plan_attn("es_linear_attention_workspace", args, grads, false, &P);
    if (st == ES_OK) *bytes = P.bytes;
    return st;
}

es_status es_plan_linear_attention(const es_linear_attention_args* args, const es_linear_attention_grads* grads,
                                   es_plan_info* info) {
    es::AttnPlan P;
    const es_status st = es::plan_attn("es_plan_linear_attention", args, grads, false, &P);
    if (st == ES_OK)
        es::fill_info(info, args->batch, args->length, args->heads, args->key_dim * args->value_dim,
                      args->batch * args->length * args->heads * args->value_dim, P.path);
    return st;
}

es_status es_linear_attention_step(const es_linear_attention_args* args, es_stream_t stream) {
    const char* fn = "es_linear_attention_step";
    es::AttnPlan P;
    es_status st = es::plan_attn(fn, args, nullptr, true, &P);
    if (st != ES_OK || P.empty) return st;
    const es::AttnLaunch& L = P.L;
    const es::AttnRun& r = L.run[0];
    es::AttnStep S{};
    S.q = r.x;
    S.k = r.y;
    S.v = r.z;
    S.out = r.out;
    S.ob = r.ob;
    S.oh = r.oh;
    S.bf16 = L.bf16;
    S.g = L.g;
    S.gb = L.gb;
    S.gh = L.gh;
    S.state = r.init;
    S.state_out = r.fin;
    S.scale = r.out_scale;
    S.B = L.B;
    S.H = L.H;
    S.dk = r.dx;
    S.dv = r.dz;
    S.stream = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = es::launch_attn_step(S);
    if (e != cudaSuccess) return es::cuda_fail(fn, e);
    es::count_launch();
    return ES_OK;
}

es_status es_qk_norm_rotate(const es_qk_norm_rotate_args* args, es_stream_t stream) {
    return es::run_rotate("es_qk_norm_rotate", args, nullptr, stream);
}

es_status es_qk_norm_rotate_backward(const es_qk_norm_rotate_args* args, const es_qk_norm_rotate_grads* grads,
                                     es_stream_t stream) {
    if (grads == nullptr) return es::api_fail(ES_E_ARG, "es_qk_norm_rotate_backward: null gradients");
    return es::run_rotate("es_qk_norm_rotate_backward", args, grads, stream);
}

es_status es_qk_norm_rotate_workspace(const es_qk_norm_rotate_args* args, const es_qk_norm_rotate_grads* grads,
                                      size_t* bytes) {
    if (bytes == nullptr) return es::api_fail(ES_E_ARG, "es_qk_norm_rotate_workspace: null result");
    es::RotatePlan P;
    const es_status st = es::plan_rotate("es_qk_norm_rotate_workspace", args, grads, &P);
    if (st == ES_OK) *bytes = P.bytes;
    return st;
}

es_status es_plan_qk_norm_rotate(const es_qk_norm_rotate_args* args, const es_qk_norm_rotate_grads* grads,
                                 es_plan_info* info) {
    es::RotatePlan P;
    const es_status st = es::plan_rotate("es_plan_qk_norm_rotate", args, grads, &P);
    if (st == ES_OK)
        es::fill_info(info, args->batch, args->length, args->q.heads + args->k.heads, args->dim,
                      args->batch * args->length * (args->q.heads + args->k.heads) * args->dim,
                      P.empty ? ES_PATH_EMPTY : ES_PATH_GENERIC);
    return st;
}

}  // extern "C"
