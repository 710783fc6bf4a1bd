// es_views.h -- checks that the entry points of the sequence-layer operators
// share: views' spans and alignment, overlaps, workspaces.  Host code.
#pragma once

#include <cstdint>
#include <cstring>

#include "es.h"
#include "es_internal.h"

namespace es {

// Bytes a view [B, T, heads, dim] spans, or -1 on overflow.
inline int64_t span_bytes(const es_heads& v, int64_t B, int64_t T, int64_t dim, int64_t size) {
    if (B == 0 || T == 0 || v.heads == 0 || dim == 0) return 0;
    const int64_t n[3] = {B - 1, T - 1, v.heads - 1}, s[3] = {v.stride_b, v.stride_t, v.stride_h};
    int64_t last = dim - 1;
    for (int i = 0; i < 3; ++i) {
        int64_t x;
        if (__builtin_mul_overflow(n[i], s[i], &x) || __builtin_add_overflow(last, x, &last)) return -1;
    }
    int64_t bytes;
    if (__builtin_add_overflow(last, int64_t(1), &last) || __builtin_mul_overflow(last, size, &bytes)) return -1;
    return bytes > (int64_t(1) << 60) ? -1 : bytes;
}

struct Span {
    const char* name;
    const void* p;
    int64_t bytes;
};

inline bool overlap(const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.bytes > 0 && b.bytes > 0 && x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

// Two views with the same batch and token strides whose tokens' rows lie side
// by side (as the parts of one fused projection do) share no element.  The
// stride of an axis with one entry means nothing; of two axes, one has to hold
// the other's entries whole, in either order.
inline bool side_by_side(const es_heads& a, const es_heads& b, int64_t da, int64_t db, int64_t size, int64_t B, int64_t T) {
    int64_t period = INT64_MAX;           // elements from one token's row to the next
    if (T > 1) {
        if (a.stride_t != b.stride_t) return false;
        period = a.stride_t;
    }
    if (B > 1) {
        if (a.stride_b != b.stride_b) return false;
        if (T > 1 && (a.stride_b >= a.stride_t ? a.stride_b < a.stride_t * T : a.stride_t < a.stride_b * B)) return false;
        period = a.stride_b < period ? a.stride_b : period;
    }
    const int64_t wa = (a.heads - 1) * a.stride_h + da, wb = (b.heads - 1) * b.stride_h + db;
    int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.data) - reinterpret_cast<uintptr_t>(b.data));
    if (d % size != 0) return false;
    d /= size;
    if (d >= 0) return d >= wb && d <= period - wa;
    return -d >= wa && -d <= period - wb;
}

inline es_status check_view(const char* fn, const char* name, const es_heads& v, int64_t B, int64_t T, int64_t dim, int64_t size,
                     bool output, Span* s) {
    if (v.stride_b < 0 || v.stride_t < 0 || v.stride_h < 0)
        return api_fail(ES_E_ARG, "%s: `%s` has a negative stride", fn, name);
    const int64_t bytes = span_bytes(v, B, T, dim, size);
    if (bytes < 0) return api_fail(ES_E_UNSUPPORTED, "%s: `%s` spans too many elements", fn, name);
    *s = Span{name, v.data, bytes};
    if (bytes == 0) return ES_OK;
    if (v.data == nullptr) return api_fail(ES_E_ARG, "%s: `%s` is a null pointer", fn, name);
    if (reinterpret_cast<uintptr_t>(v.data) % size != 0)
        return api_fail(ES_E_ARG, "%s: `%s` is not aligned to its elements", fn, name);
    if (output && ((B > 1 && v.stride_b == 0) || (T > 1 && v.stride_t == 0) || (v.heads > 1 && v.stride_h < dim)))
        return api_fail(ES_E_ARG, "%s: `%s` is an output whose elements share addresses", fn, name);
    return ES_OK;
}

inline es_status check_dense(const char* fn, const char* name, const void* p, int64_t elements, Span* s) {
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return api_fail(ES_E_ARG, "%s: `%s` is not 4-byte aligned", fn, name);
    *s = Span{name, p, p == nullptr ? 0 : elements * 4};
    return ES_OK;
}

// No output may touch another span, nor the workspace any of them.
inline es_status check_outputs(const char* fn, const Span* in, int n_in, const Span* out, int n_out, const void* ws = nullptr,
                        size_t ws_bytes = 0) {
    if (ws != nullptr && ws_bytes > 0) {
        const Span w{"workspace", ws, static_cast<int64_t>(ws_bytes)};
        for (int i = 0; i < n_in; ++i)
            if (overlap(w, in[i])) return api_fail(ES_E_ARG, "%s: the workspace overlaps `%s`", fn, in[i].name);
        for (int i = 0; i < n_out; ++i)
            if (overlap(w, out[i])) return api_fail(ES_E_ARG, "%s: the workspace overlaps `%s`", fn, out[i].name);
    }
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlap(out[i], in[j])) return api_fail(ES_E_ARG, "%s: `%s` overlaps `%s`", fn, out[i].name, in[j].name);
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return api_fail(ES_E_ARG, "%s: `%s` overlaps `%s`", fn, out[i].name, out[j].name);
    }
    return ES_OK;
}

// the next `bytes` of a workspace, from a 256-byte boundary
inline size_t take(size_t* at, int64_t bytes) {
    const size_t here = *at;
    *at += (static_cast<size_t>(bytes) + 255) & ~size_t(255);
    return here;
}

inline es_status check_workspace(const char* fn, void* ws, int64_t bytes, size_t need) {
    if (need == 0) return ES_OK;
    if (ws == nullptr || bytes < 0 || static_cast<size_t>(bytes) < need)
        return api_fail(ES_E_ARG, "%s: a workspace of %lld bytes; %zu are needed", fn,
                        static_cast<long long>(ws == nullptr ? 0 : bytes), need);
    if (reinterpret_cast<uintptr_t>(ws) % 16 != 0) return api_fail(ES_E_ARG, "%s: the workspace is not 16-byte aligned", fn);
    return ES_OK;
}

inline es_status cuda_fail(const char* fn, cudaError_t e) { return api_fail(ES_E_CUDA, "%s: %s", fn, cudaGetErrorString(e)); }

inline void fill_info(es_plan_info* info, int64_t O, int64_t T, int64_t J, int64_t W, int64_t elements, int path) {
    if (info == nullptr) return;
    std::memset(info, 0, sizeof(*info));
    info->O = O;
    info->T = T;
    info->J = J;
    info->W = W;
    info->elements = elements;
    info->path = path;
}

}  // namespace es
