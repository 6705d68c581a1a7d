// abi_cache.cu -- the extern "C" entry points of the target pass's cache and
// attention: host-side argument checks, then the launchers.
#include <algorithm>
#include <cmath>

#include "abi_util.cuh"
#include "cache.cuh"

using namespace dspark;

namespace {

dspark_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA; }

bool table_ok(int B, int P, int max_pages, int n_pages) {
    return B >= 1 && B <= 4096 && page_ok(P) && max_pages >= 1 && n_pages >= 1 &&
           (long long)n_pages * P <= 0x7fffffffLL && (long long)max_pages * P <= (1LL << 30);
}
bool heads_ok(int Hq, int Hkv) { return Hkv >= 1 && Hq >= Hkv && Hq <= 1024 && Hq % Hkv == 0; }
// 6 g, 512 * 6 g and their reciprocals stay normal fp32 numbers.
bool gain_ok(float g) { return g >= 0x1p-64f && g <= 0x1p64f; }
// Rows are read in 16-byte pieces: base and token stride on 16-byte boundaries,
// the stride at least the token's heads.
bool rows_ok(const void *p, long long stride, int heads, int D, int dtype) {
    const int per = dtype == DSPARK_BF16 ? 8 : 4;
    return aligned16(p) && stride >= (long long)heads * D && stride % per == 0;
}

// `T` tokens of `heads` heads, `stride` elements apart: the bytes they span.
struct Span {
    uintptr_t lo, hi;
    bool dense;   // nothing between the tokens
};
Span span_of(const void *p, int T, long long stride, int heads, int D, int dtype) {
    const long long e = dtype == DSPARK_BF16 ? 2 : 4, row = (long long)heads * D;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + (uintptr_t)(((T - 1) * stride + row) * e), T == 1 || stride == row};
}
bool disjoint(const Span &a, const Span &b) { return a.hi <= b.lo || b.hi <= a.lo; }
// An output over an input: the same dense rows (a thread reads its own rows
// before it writes them), or apart.
bool in_place_or_apart(const Span &out, const Span &in) { return disjoint(out, in) || (in.dense && out.lo == in.lo); }

dspark_status plan(const PlanArgs &a, size_t ws_bytes, void *stream) {
    if (!table_ok(a.B, a.P, a.max_pages, a.n_pages) || a.G < 0 || a.G > (1 << 20) || a.T < 0 || a.T > (1 << 24))
        return DSPARK_ERR_INVALID_ARG;
    if (!a.ctx || !a.ell || !a.table || !a.held || !a.free_list || !a.free_count || !a.q_start || !a.kv_len ||
        (a.T > 0 && (!a.slot || !a.pos)))
        return DSPARK_ERR_INVALID_ARG;
    if (dspark_status s = check_ws(a.hdr, ws_bytes, sizeof(WsHeader))) return s;
    return cuda_status(launch_cache_plan(a, static_cast<cudaStream_t>(stream)));
}

dspark_status commit(const CommitArgs &a, size_t ws_bytes, void *stream) {
    if (!table_ok(a.B, a.P, a.max_pages, a.n_pages) || a.G < 0 || a.G > (1 << 20)) return DSPARK_ERR_INVALID_ARG;
    if (!a.ctx || !a.q_start || !a.nout || !a.table || !a.held || !a.free_list || !a.free_count || !a.ctx_out)
        return DSPARK_ERR_INVALID_ARG;
    if (dspark_status s = check_ws(a.hdr, ws_bytes, sizeof(WsHeader))) return s;
    return cuda_status(launch_cache_commit(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t dspark_cache_record_bytes(int P, int D) {
    return page_ok(P) && cache_dim_ok(D) ? (size_t)record_bytes(P, D) : 0;
}

dspark_status dspark_cache_plan(const int32_t *ctx, const int32_t *ell, int B, int G, int P, int max_pages,
                                int n_pages, int32_t *table, int32_t *held, const int32_t *free_list,
                                int32_t *free_count, void *ws, size_t ws_bytes, int32_t *q_start_out,
                                int32_t *kv_len_out, int32_t *slot_out, int32_t *pos_out, void *stream) {
    if (dspark_status s = injected("dspark_cache_plan")) return s;
    const long long T = (long long)B * (G + 1LL);
    if (T < 0 || T > (1 << 24)) return DSPARK_ERR_INVALID_ARG;
    return plan({ctx, ell, B, G, P, max_pages, n_pages, table, held, free_list, free_count,
                 static_cast<WsHeader *>(ws), q_start_out, kv_len_out, slot_out, pos_out, (int)T, nullptr},
                ws_bytes, stream);
}

dspark_status dspark_cache_plan_rows(const int32_t *ctx, const int32_t *ell, int B, int G, int P, int max_pages,
                                     int n_pages, int32_t *table, int32_t *held, const int32_t *free_list,
                                     int32_t *free_count, int T, void *ws, size_t ws_bytes, int32_t *ell_out,
                                     int32_t *q_start_out, int32_t *kv_len_out, int32_t *slot_out, int32_t *pos_out,
                                     void *stream) {
    if (dspark_status s = injected("dspark_cache_plan_rows")) return s;
    return plan({ctx, ell, B, G, P, max_pages, n_pages, table, held, free_list, free_count,
                 static_cast<WsHeader *>(ws), q_start_out, kv_len_out, slot_out, pos_out, T, ell_out},
                ws_bytes, stream);
}

dspark_status dspark_cache_commit(const int32_t *ctx, const int32_t *q_start, const int32_t *nout,
                                  const int32_t *done, int B, int P, int max_pages, int n_pages, int32_t *table,
                                  int32_t *held, int32_t *free_list, int32_t *free_count, void *ws, size_t ws_bytes,
                                  int32_t *ctx_out, void *stream) {
    if (dspark_status s = injected("dspark_cache_commit")) return s;
    return commit({ctx, q_start, nout, done, B, P, max_pages, n_pages, table, held, free_list, free_count,
                   static_cast<WsHeader *>(ws), ctx_out, nullptr, nullptr, nullptr, 0},
                  ws_bytes, stream);
}

dspark_status dspark_cache_commit_round(const int32_t *ctx, const int32_t *q_start, int32_t *nout, int32_t *acc,
                                        int32_t *tokens, const int32_t *done, int B, int G, int P, int max_pages,
                                        int n_pages, int32_t *table, int32_t *held, int32_t *free_list,
                                        int32_t *free_count, void *ws, size_t ws_bytes, int32_t *ctx_out,
                                        void *stream) {
    if (dspark_status s = injected("dspark_cache_commit_round")) return s;
    return commit({ctx, q_start, nout, done, B, P, max_pages, n_pages, table, held, free_list, free_count,
                   static_cast<WsHeader *>(ws), ctx_out, nout, acc, tokens, G},
                  ws_bytes, stream);
}

dspark_status dspark_qk_norm_rope(const void *q, long long q_stride, const void *k, long long k_stride,
                                  const void *v, long long v_stride, const void *wq, const void *wk, float eps,
                                  const int32_t *pos, const float *inv_freq, int rot, int interleaved,
                                  const int32_t *n_rows, int T, int Hq, int Hkv, int D, int dtype, void *q_out,
                                  void *k_out, void *cache, const int32_t *slot, int P, int n_pages, float k_scale,
                                  float v_scale, void *ws, size_t ws_bytes, void *stream) {
    if (dspark_status s = injected("dspark_qk_norm_rope")) return s;
    if (!dtype_ok(dtype)) return DSPARK_ERR_UNSUPPORTED_DTYPE;
    if (T < 0 || T > (1 << 24) || !heads_ok(Hq, Hkv) || !cache_dim_ok(D) || rot < 0 || rot > D || rot % 32 != 0 ||
        !(eps >= 0.f))
        return DSPARK_ERR_INVALID_ARG;
    // An empty array may have no address.
    if (T > 0 && (!q || !k || !q_out || (!k_out && !cache) || (rot > 0 && (!pos || !inv_freq))))
        return DSPARK_ERR_INVALID_ARG;
    if (!rows_ok(q, q_stride, Hq, D, dtype) || !rows_ok(k, k_stride, Hkv, D, dtype) || !aligned16(q_out) ||
        !aligned16(k_out) || !aligned16(wq) || !aligned16(wk))
        return DSPARK_ERR_INVALID_ARG;
    if (cache != nullptr) {
        if ((T > 0 && (!v || !slot)) || !page_ok(P) || n_pages < 1 || (long long)n_pages * P > 0x7fffffffLL || !gain_ok(k_scale) ||
            !gain_ok(v_scale) || !aligned16(cache) || !rows_ok(v, v_stride, Hkv, D, dtype))
            return DSPARK_ERR_INVALID_ARG;
    }
    if (dspark_status s = check_ws(ws, ws_bytes, sizeof(WsHeader))) return s;
    if (T == 0) return DSPARK_OK;
    const Span sq = span_of(q, T, q_stride, Hq, D, dtype), sk = span_of(k, T, k_stride, Hkv, D, dtype);
    const Span oq = span_of(q_out, T, (long long)Hq * D, Hq, D, dtype);
    if (!in_place_or_apart(oq, sq) || !disjoint(oq, sk)) return DSPARK_ERR_INVALID_ARG;
    if (k_out) {
        const Span ok = span_of(k_out, T, (long long)Hkv * D, Hkv, D, dtype);
        if (!in_place_or_apart(ok, sk) || !disjoint(ok, sq) || !disjoint(ok, oq)) return DSPARK_ERR_INVALID_ARG;
        if (cache && !disjoint(ok, span_of(v, T, v_stride, Hkv, D, dtype))) return DSPARK_ERR_INVALID_ARG;
    }
    if (cache && !disjoint(oq, span_of(v, T, v_stride, Hkv, D, dtype))) return DSPARK_ERR_INVALID_ARG;
    NormArgs a{q, k, v, q_stride, k_stride, v_stride, wq, wk, eps, pos, inv_freq, rot, interleaved ? 1 : 0, n_rows,
               T, Hq, Hkv, D, dtype, q_out, k_out, static_cast<uint8_t *>(cache), slot, P, n_pages, k_scale, v_scale,
               static_cast<WsHeader *>(ws)};
    return cuda_status(launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

dspark_status dspark_cache_read(const void *cache, const int32_t *slot, int T, int Hkv, int D, int P, int n_pages,
                                float k_scale, float v_scale, int dtype, void *k_out, void *v_out, void *ws,
                                size_t ws_bytes, void *stream) {
    if (dspark_status s = injected("dspark_cache_read")) return s;
    if (!dtype_ok(dtype)) return DSPARK_ERR_UNSUPPORTED_DTYPE;
    if (T < 0 || T > (1 << 24) || !heads_ok(Hkv, Hkv) || !cache_dim_ok(D) || !page_ok(P) || n_pages < 1 ||
        (long long)n_pages * P > 0x7fffffffLL || !gain_ok(k_scale) || !gain_ok(v_scale))
        return DSPARK_ERR_INVALID_ARG;
    if (!cache || (T > 0 && (!slot || !k_out || !v_out)) || !aligned16(cache) || !aligned16(k_out) || !aligned16(v_out))
        return DSPARK_ERR_INVALID_ARG;
    if (dspark_status s = check_ws(ws, ws_bytes, sizeof(WsHeader))) return s;
    if (T == 0) return DSPARK_OK;
    ReadArgs a{static_cast<const uint8_t *>(cache), slot, T, Hkv, D, P, n_pages, dtype, k_scale, v_scale, k_out,
               v_out, static_cast<WsHeader *>(ws)};
    return cuda_status(launch_cache_read(a, static_cast<cudaStream_t>(stream)));
}

size_t dspark_cache_attention_workspace_size(int B, int Hq, int Hkv, int D) {
    if (B < 1 || B > 4096 || !heads_ok(Hq, Hkv) || !cache_dim_ok(D)) return 0;
    return attention_ws_bytes(D);
}

dspark_status dspark_cache_attention(const void *q, long long q_stride, const void *cache, const int32_t *table,
                                     const int32_t *q_start, const int32_t *kv_len, int B, int T, int Hq, int Hkv,
                                     int D, int P, int max_pages, int n_pages, float scale, float k_scale,
                                     float v_scale, int window, int dtype, void *ws, size_t ws_bytes, void *out,
                                     void *stream) {
    if (dspark_status s = injected("dspark_cache_attention")) return s;
    if (dtype != DSPARK_BF16) return DSPARK_ERR_UNSUPPORTED_DTYPE;
    if (!table_ok(B, P, max_pages, n_pages) || T < 0 || T > (1 << 24) || !heads_ok(Hq, Hkv) || !cache_dim_ok(D) ||
        window < 0 || !gain_ok(k_scale) || !gain_ok(v_scale) || !std::isfinite(scale * k_scale * kLog2e) ||
        (long long)T * Hq > 0x7fffffffLL)
        return DSPARK_ERR_INVALID_ARG;
    if ((T > 0 && (!q || !out)) || !cache || !table || !q_start || !kv_len || !rows_ok(q, q_stride, Hq, D, dtype) ||
        !aligned16(cache) || !attention_work_fits(B, T, Hkv, Hq / Hkv, P, max_pages))
        return DSPARK_ERR_INVALID_ARG;
    if (dspark_status s = check_ws(ws, ws_bytes, attention_ws_bytes(D))) return s;
    if (T == 0) return DSPARK_OK;
    // Parts of an item read its queries while another part's results are out.
    const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
    const uintptr_t q1 = q0 + ((size_t)(T - 1) * (size_t)q_stride + (size_t)Hq * D) * 2, o1 = o0 + (size_t)T * Hq * D * 2;
    if (q0 < o1 && o0 < q1) return DSPARK_ERR_INVALID_ARG;
    AttnArgs a{};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_stride = q_stride;
    a.cache = static_cast<const uint8_t *>(cache);
    a.table = table;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.B = B;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.group = Hq / Hkv;
    a.D = D;
    a.P = P;
    a.max_pages = max_pages;
    a.n_pages = n_pages;
    a.window = std::min(window, max_pages * P);   // no table holds more; positions less a window stay in 32 bits
    a.qk_mul = scale * k_scale * kLog2e;
    a.v_mul = v_scale;
    a.out = static_cast<__nv_bfloat16 *>(out);
    return cuda_status(launch_cache_attention(a, ws, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
