"""ctypes binding of libdspark (the C ABI declared in include/dspark.h).

Argument marshalling only: torch tensors supply device pointers and sizes,
torch streams supply the cudaStream_t.  Every step of the round runs in the
library's CUDA kernels; there is no fallback.  Importing this module on a
machine without the built library, or calling it without a CUDA device,
raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdspark.so")

DSPARK_F32 = 0
DSPARK_BF16 = 1
SCHED_ALL = 0
SCHED_GREEDY_EARLY_STOP = 1
SCHED_GLOBAL_ARGMAX = 2
SCHED_THRESHOLD = 3
SCHED_TOPK = 4

STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED_DTYPE", 3: "WORKSPACE", 4: "CUDA", 5: "TIMEOUT"}
DEV_TOKEN_RANGE, DEV_ELL_RANGE, DEV_BAD_TEMP, DEV_TIMEOUT, DEV_BAD_VALUE = 0x1, 0x2, 0x4, 0x8, 0x10
DEV_CACHE_FULL, DEV_PAGE_RANGE, DEV_LENGTH_RANGE = 0x20, 0x40, 0x80

EXPORTS = ("dspark_version", "dspark_draft_workspace_size", "dspark_draft_markov", "dspark_confidence",
           "dspark_schedule_workspace_size", "dspark_schedule", "dspark_verify_workspace_size",
           "dspark_verify", "dspark_get_device_status", "dspark_clear_device_status",
           "dspark_draft_noalloc_max_scratch", "dspark_draft_markov_noalloc", "dspark_schedule_threshold",
           "dspark_sts_workspace_size", "dspark_sts_fit", "dspark_survival_auc", "dspark_schedule_topk",
           "dspark_draft_noalloc_device_status", "dspark_draft_rnn", "dspark_verify_rnn", "dspark_get_near_ties",
           "dspark_exp2_fma", "dspark_gather_admitted_targets", "dspark_cache_record_bytes", "dspark_cache_plan",
           "dspark_cache_commit", "dspark_qk_norm_rope", "dspark_cache_read",
           "dspark_cache_attention_workspace_size", "dspark_cache_attention", "dspark_cache_plan_rows",
           "dspark_cache_commit_round")


class DsparkError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} returned {status} ({STATUS.get(status, '?')})")
        self.status = status


_lib = None
_vp, _i, _f, _sz, _d = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_double
_ll = ctypes.c_longlong


def load() -> ctypes.CDLL:
    """Load libdspark.so from the package directory (build it first with
    ``python -m speculative_decoding_draft_rank_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libdspark.so is not built ({LIB_PATH}); run the package build step")
    lib = ctypes.CDLL(LIB_PATH)
    lib.dspark_version.restype = ctypes.c_char_p
    lib.dspark_draft_workspace_size.restype = _sz
    lib.dspark_draft_workspace_size.argtypes = [_i] * 5
    lib.dspark_draft_markov.restype = _i
    lib.dspark_draft_markov.argtypes = [_vp] * 6 + [_i] * 5 + [_vp, _sz] + [_vp] * 5
    lib.dspark_confidence.restype = _i
    lib.dspark_confidence.argtypes = [_vp, _vp, _f, _vp, _i, _i, _i, _i, _vp, _vp, _vp]
    lib.dspark_schedule_workspace_size.restype = _sz
    lib.dspark_schedule_workspace_size.argtypes = [_i, _i]
    lib.dspark_schedule.restype = _i
    lib.dspark_schedule.argtypes = [_vp, _i, _i, _vp, _vp, _i, _i, _i, _vp, _sz, _vp, _vp, _vp, _vp, _vp]
    lib.dspark_schedule_threshold.restype = _i
    lib.dspark_schedule_threshold.argtypes = [_vp, _i, _i, _f, _i, _vp, _sz, _vp, _vp, _vp, _vp]
    lib.dspark_verify_workspace_size.restype = _sz
    lib.dspark_verify_workspace_size.argtypes = [_i] * 5
    lib.dspark_verify.restype = _i
    lib.dspark_verify.argtypes = [_vp] * 13 + [_i] * 5 + [_vp, _sz] + [_vp] * 5
    lib.dspark_get_device_status.restype = _i
    lib.dspark_get_device_status.argtypes = [_vp, _vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.dspark_exp2_fma.restype = _i
    lib.dspark_exp2_fma.argtypes = [_vp, _vp, _i, _vp]
    lib.dspark_get_near_ties.restype = _i
    lib.dspark_get_near_ties.argtypes = [_vp, _vp, ctypes.POINTER(ctypes.c_uint32), ctypes.POINTER(ctypes.c_uint32)]
    lib.dspark_clear_device_status.restype = _i
    lib.dspark_clear_device_status.argtypes = [_vp, _vp]
    lib.dspark_draft_noalloc_max_scratch.restype = _sz
    lib.dspark_draft_noalloc_max_scratch.argtypes = []
    lib.dspark_draft_markov_noalloc.restype = _i
    lib.dspark_draft_markov_noalloc.argtypes = [_vp] * 6 + [_i] * 5 + [_vp] * 5
    lib.dspark_draft_rnn.restype = _i
    lib.dspark_draft_rnn.argtypes = [_vp] * 7 + [_i] * 5 + [_vp, _sz] + [_vp] * 6
    lib.dspark_verify_rnn.restype = _i
    lib.dspark_verify_rnn.argtypes = [_vp] * 12 + [_i] * 5 + [_vp, _sz] + [_vp] * 5
    lib.dspark_draft_noalloc_device_status.restype = _i
    lib.dspark_draft_noalloc_device_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.dspark_schedule_topk.restype = _i
    lib.dspark_schedule_topk.argtypes = [_vp, _i, _i, _vp, _i, _vp, _sz, _vp, _vp, _vp, _vp]
    lib.dspark_sts_workspace_size.restype = _sz
    lib.dspark_sts_workspace_size.argtypes = [_i] * 4
    lib.dspark_sts_fit.restype = _i
    lib.dspark_sts_fit.argtypes = [_vp] * 3 + [_i] * 4 + [_vp, _sz] + [_vp] * 6
    lib.dspark_survival_auc.restype = _i
    lib.dspark_survival_auc.argtypes = [_vp, _vp, _i, _i, _vp, _vp, _vp]
    lib.dspark_gather_admitted_targets.restype = _i
    lib.dspark_gather_admitted_targets.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _vp]
    lib.dspark_cache_record_bytes.restype = _sz
    lib.dspark_cache_record_bytes.argtypes = [_i] * 2
    lib.dspark_cache_plan.restype = _i
    lib.dspark_cache_plan.argtypes = [_vp] * 2 + [_i] * 5 + [_vp] * 5 + [_sz] + [_vp] * 5
    lib.dspark_cache_commit.restype = _i
    lib.dspark_cache_commit.argtypes = [_vp] * 4 + [_i] * 4 + [_vp] * 5 + [_sz] + [_vp] * 2
    lib.dspark_cache_plan_rows.restype = _i
    lib.dspark_cache_plan_rows.argtypes = [_vp] * 2 + [_i] * 5 + [_vp] * 4 + [_i, _vp, _sz] + [_vp] * 6
    lib.dspark_cache_commit_round.restype = _i
    lib.dspark_cache_commit_round.argtypes = [_vp] * 6 + [_i] * 5 + [_vp] * 5 + [_sz] + [_vp] * 2
    lib.dspark_qk_norm_rope.restype = _i
    lib.dspark_qk_norm_rope.argtypes = ([_vp, _ll] * 3 + [_vp] * 2 + [_f] + [_vp] * 2 + [_i] * 2 + [_vp] + [_i] * 5 +
                                        [_vp] * 4 + [_i] * 2 + [_f] * 2 + [_vp, _sz, _vp])
    lib.dspark_cache_read.restype = _i
    lib.dspark_cache_read.argtypes = [_vp] * 2 + [_i] * 5 + [_f] * 2 + [_i] + [_vp] * 3 + [_sz, _vp]
    lib.dspark_cache_attention_workspace_size.restype = _sz
    lib.dspark_cache_attention_workspace_size.argtypes = [_i] * 4
    lib.dspark_cache_attention.restype = _i
    lib.dspark_cache_attention.argtypes = ([_vp, _ll] + [_vp] * 4 + [_i] * 8 + [_f] * 3 + [_i] * 2 +
                                           [_vp, _sz] + [_vp] * 2)
    _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libdspark takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libdspark takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype(t):
    if t.dtype == torch.bfloat16:
        return DSPARK_BF16
    if t.dtype == torch.float32:
        return DSPARK_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


def _call(fn, *args):
    st = getattr(load(), fn)(*args)
    if st != 0:
        raise DsparkError(fn, st)


def version() -> str:
    return load().dspark_version().decode()


def dspark_draft_workspace_size(B, G, V, r, dtype) -> int:
    return int(load().dspark_draft_workspace_size(B, G, V, r, dtype))


def dspark_schedule_workspace_size(B, G) -> int:
    return int(load().dspark_schedule_workspace_size(B, G))


def dspark_verify_workspace_size(B, G, V, r, dtype) -> int:
    return int(load().dspark_verify_workspace_size(B, G, V, r, dtype))


def dspark_draft_markov(L, U, Wt, x0, temp, u_draft, ws, x_out, pd_x_out, rowmax_out, rowsum_out,
                        stream=None):
    B, G, V = L.shape
    r = U.shape[1]
    _call("dspark_draft_markov", _ptr(L), _ptr(U), _ptr(Wt), _ptr(x0), _ptr(temp), _ptr(u_draft), B, G, V,
          r, _dtype(L), _ptr(ws), ws.numel() * ws.element_size(), _ptr(x_out), _ptr(pd_x_out),
          _ptr(rowmax_out), _ptr(rowsum_out), _stream(stream))


def dspark_draft_rnn(L, U, Arec, Wt, x0, temp, u_draft, ws, x_out, pd_x_out, rowmax_out, rowsum_out, H_out,
                     stream=None):
    """Drafting with the RNN head: Arec [r, r] bf16 recurrent matrix; H_out
    [B, G, r] fp32 receives the state that biased every position."""
    B, G, V = L.shape
    r = U.shape[1]
    _call("dspark_draft_rnn", _ptr(L), _ptr(U), _ptr(Arec), _ptr(Wt), _ptr(x0), _ptr(temp), _ptr(u_draft), B, G,
          V, r, _dtype(L), _ptr(ws), ws.numel() * ws.element_size(), _ptr(x_out), _ptr(pd_x_out), _ptr(rowmax_out),
          _ptr(rowsum_out), _ptr(H_out), _stream(stream))


def dspark_verify_rnn(Tlog, L, H, Wt, x, pd_x, rowmax, rowsum, temp, u_accept, u_final, ell, ws, acc_out,
                      tokens_out, nout_out, pt_x_out=None, stream=None):
    """Verification of RNN-head drafts (the states H from dspark_draft_rnn)."""
    B, G1, V = Tlog.shape
    r = H.shape[2]
    _call("dspark_verify_rnn", _ptr(Tlog), _ptr(L), _ptr(H), _ptr(Wt), _ptr(x), _ptr(pd_x), _ptr(rowmax),
          _ptr(rowsum), _ptr(temp), _ptr(u_accept), _ptr(u_final), _ptr(ell), B, G1 - 1, V, r, _dtype(Tlog),
          _ptr(ws), ws.numel() * ws.element_size(), _ptr(acc_out), _ptr(tokens_out), _ptr(nout_out),
          _ptr(pt_x_out), _stream(stream))


def dspark_draft_noalloc_max_scratch() -> int:
    return int(load().dspark_draft_noalloc_max_scratch())


def dspark_draft_markov_noalloc(L, U, Wt, x0, temp, u_draft, x_out, pd_x_out, rowmax_out, rowsum_out,
                                stream=None):
    """Drafting with the library's own fixed scratch instead of a workspace."""
    B, G, V = L.shape
    r = U.shape[1]
    _call("dspark_draft_markov_noalloc", _ptr(L), _ptr(U), _ptr(Wt), _ptr(x0), _ptr(temp), _ptr(u_draft), B,
          G, V, r, _dtype(L), _ptr(x_out), _ptr(pd_x_out), _ptr(rowmax_out), _ptr(rowsum_out), _stream(stream))


def dspark_draft_noalloc_device_status(stream=None) -> int:
    """Status word of the last allocation-free drafting call on `stream`
    (synchronises the stream)."""
    out = ctypes.c_uint32(0)
    _call("dspark_draft_noalloc_device_status", _stream(stream), ctypes.byref(out))
    return int(out.value)


def dspark_confidence(h, w, bias, tau, c_out, S_out, stream=None):
    B, G, d = h.shape
    _call("dspark_confidence", _ptr(h), _ptr(w), ctypes.c_float(bias), _ptr(tau), B, G, d, _dtype(h),
          _ptr(c_out), _ptr(S_out), _stream(stream))


def dspark_schedule(S, knots_n, knots_t, budget, mode, ws, ell_out, n_adm_out, theta_out, order_out=None,
                    stream=None):
    B, G = S.shape
    _call("dspark_schedule", _ptr(S), B, G, _ptr(knots_n), _ptr(knots_t), knots_n.numel(), int(budget),
          int(mode), _ptr(ws), ws.numel() * ws.element_size(), _ptr(ell_out), _ptr(n_adm_out),
          _ptr(theta_out), _ptr(order_out), _stream(stream))


def dspark_schedule_threshold(S, threshold, budget, ws, ell_out, n_adm_out, order_out=None, stream=None):
    """Static-threshold pruning: the sorted candidates with S >= threshold."""
    B, G = S.shape
    _call("dspark_schedule_threshold", _ptr(S), B, G, ctypes.c_float(threshold), int(budget), _ptr(ws),
          ws.numel() * ws.element_size(), _ptr(ell_out), _ptr(n_adm_out), _ptr(order_out), _stream(stream))


def dspark_schedule_topk(S, capacity, budget, ws, ell_out, n_adm_out, order_out=None, stream=None):
    """Dynamic top-K: the first *capacity (a device int32) candidates of the
    stable order by S."""
    B, G = S.shape
    _call("dspark_schedule_topk", _ptr(S), B, G, _ptr(capacity), int(budget), _ptr(ws),
          ws.numel() * ws.element_size(), _ptr(ell_out), _ptr(n_adm_out), _ptr(order_out), _stream(stream))


def dspark_verify(Tlog, L, U, Wt, x0, x, pd_x, rowmax, rowsum, temp, u_accept, u_final, ell, ws, acc_out,
                  tokens_out, nout_out, pt_x_out=None, stream=None):
    B, G1, V = Tlog.shape
    r = U.shape[1]
    _call("dspark_verify", _ptr(Tlog), _ptr(L), _ptr(U), _ptr(Wt), _ptr(x0), _ptr(x), _ptr(pd_x),
          _ptr(rowmax), _ptr(rowsum), _ptr(temp), _ptr(u_accept), _ptr(u_final), _ptr(ell), B, G1 - 1, V, r,
          _dtype(Tlog), _ptr(ws), ws.numel() * ws.element_size(), _ptr(acc_out), _ptr(tokens_out),
          _ptr(nout_out), _ptr(pt_x_out), _stream(stream))


def dspark_sts_workspace_size(N, G, K, n_bins) -> int:
    return int(load().dspark_sts_workspace_size(N, G, K, n_bins))


def dspark_sts_fit(z, acc, tau_grid, n_bins, ws, tau_out, ece_raw_out=None, ece_fit_out=None, ece_all_out=None,
                   S_out=None, stream=None):
    """Sequential temperature scaling: z [N, G] f32 logits, acc [N] int32,
    tau_grid [K] f32 candidates -> tau_out [G] f32 (and the optional ECEs,
    fp64, and fitted survivals S_out [N, G] f32)."""
    N, G = z.shape
    K = tau_grid.shape[0]
    _call("dspark_sts_fit", _ptr(z), _ptr(acc), _ptr(tau_grid), N, G, K, int(n_bins), _ptr(ws),
          ws.numel() * ws.element_size(), _ptr(tau_out), _ptr(ece_raw_out), _ptr(ece_fit_out), _ptr(ece_all_out),
          _ptr(S_out), _stream(stream))


def dspark_survival_auc(S, acc, twice_out, pairs_out, stream=None):
    """ROC-AUC pair counts per position: twice_out, pairs_out [G] int64
    tensors (uint64 bit patterns); AUC = twice / (2 * pairs)."""
    N, G = S.shape
    _call("dspark_survival_auc", _ptr(S), _ptr(acc), N, G, _ptr(twice_out), _ptr(pairs_out), _stream(stream))


def dspark_get_device_status(ws, stream=None) -> int:
    out = ctypes.c_uint32(0)
    _call("dspark_get_device_status", _ptr(ws), _stream(stream), ctypes.byref(out))
    return int(out.value)


def dspark_get_near_ties(ws, stream=None):
    """(drafting, verification) near-tie counts of a workspace since its last
    clear (synchronises the stream)."""
    d, v = ctypes.c_uint32(0), ctypes.c_uint32(0)
    _call("dspark_get_near_ties", _ptr(ws), _stream(stream), ctypes.byref(d), ctypes.byref(v))
    return int(d.value), int(v.value)


def dspark_gather_admitted_targets(Tlog_host, Tlog_dev, ell, stream=None):
    """Enqueue one kernel that copies rows 0..ell[b] of every request of the
    pinned host target logits [B, G+1, V] into the device buffer of the same
    layout; ell: the device int32 [B] of admitted lengths."""
    if Tlog_host.is_cuda or not Tlog_host.is_pinned() or not Tlog_host.is_contiguous():
        raise ValueError("Tlog_host must be a contiguous pinned host tensor")
    if Tlog_host.shape != Tlog_dev.shape or Tlog_host.dtype != Tlog_dev.dtype or ell.dtype != torch.int32:
        raise ValueError("Tlog_host and Tlog_dev differ in shape or dtype, or ell is not int32")
    B, G1, V = Tlog_dev.shape
    _call("dspark_gather_admitted_targets", ctypes.c_void_p(Tlog_host.data_ptr()), _ptr(Tlog_dev), _ptr(ell), B,
          G1 - 1, V, _dtype(Tlog_dev), _stream(stream))


# The calls of the target pass run once per layer and round, so their
# marshalling is kept short: plain integers for pointers, the raw stream, and
# one device comparison per tensor.
def _device_of(t):
    d = t.get_device()
    if d < 0:
        raise ValueError("libdspark takes device tensors")
    return d


def _dense(t, dev):
    """Pointer of a contiguous tensor on device `dev` (None passes)."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"libdspark takes tensors of one device: {t.device} and cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError("libdspark takes contiguous tensors")
    return t.data_ptr()


def _ints(t, dev, n, what):
    """Pointer of an int32 tensor of at least n elements."""
    if t.dtype is not torch.int32 or t.numel() < n:
        raise ValueError(f"{what}: an int32 tensor of at least {n} elements, got {t.dtype} of {t.numel()}")
    return _dense(t, dev)


def _rows(t, dev, what):
    """(pointer, token stride) of a [T, H, D] device tensor whose heads are dense; the tokens may lie apart (a
    slice of a fused projection)."""
    if t.get_device() != dev:
        raise ValueError(f"libdspark takes tensors of one device: {t.device} and cuda:{dev}")
    T, H, D = t.shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or (H > 1 and s1 != D):
        raise ValueError(f"{what}: the heads of a token must be dense")
    return t.data_ptr(), (s0 if T > 1 else H * D)   # of a single token the stride says nothing


def _launch(fn, dev, stream, *args):
    """Call `fn` with the stream appended, on device `dev` (which need not be the current one)."""
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    f = getattr(_lib or load(), fn)
    if dev == torch._C._cuda_getDevice():
        st = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = f(*args, raw)
    if st != 0:
        raise DsparkError(fn, st)


def _cache_dims(cache, page, D):
    """(n_pages, Hkv) of a cache tensor [n_pages, Hkv, record bytes]."""
    shape = cache.shape
    need = dspark_cache_record_bytes(page, D)
    if cache.dtype is not torch.uint8 or len(shape) != 3 or need == 0 or shape[2] != need:
        raise ValueError(f"cache: uint8 [n_pages, Hkv, {need}] for pages of {page} tokens and heads of {D}, got "
                         f"{cache.dtype} {tuple(shape)}")
    return shape[0], shape[1]


def dspark_cache_record_bytes(page, D) -> int:
    """Bytes of one (page, head) record of the 4-bit cache; 0 for an unsupported page size or head dim."""
    return (_lib or load()).dspark_cache_record_bytes(page, D)


def dspark_cache_plan(ctx, ell, G, table, held, free_list, free_count, page, ws, q_start_out, kv_len_out, slot_out,
                      pos_out, stream=None):
    """Rows, slots, positions and pages of a round from the cached lengths
    ctx [B] and admitted lengths ell [B]; table [B, max_pages], held [B] and
    free_count [1] are updated, free_list [n_pages] is read.  slot_out and
    pos_out hold B * (G + 1) entries, -1 behind the last row."""
    dev = _device_of(table)
    B, max_pages = table.shape
    T = B * (G + 1)
    _launch("dspark_cache_plan", dev, stream, _ints(ctx, dev, B, "ctx"), _ints(ell, dev, B, "ell"), B, int(G),
            int(page), max_pages, free_list.numel(), _ints(table, dev, 1, "table"), _ints(held, dev, B, "held"),
            _ints(free_list, dev, 1, "free_list"), _ints(free_count, dev, 1, "free_count"), _dense(ws, dev),
            ws.nbytes, _ints(q_start_out, dev, B + 1, "q_start_out"), _ints(kv_len_out, dev, B, "kv_len_out"),
            _ints(slot_out, dev, T, "slot_out"), _ints(pos_out, dev, T, "pos_out"))


def dspark_cache_plan_rows(ctx, ell, G, table, held, free_list, free_count, page, ws, q_start_out, kv_len_out, slot_out,
                           pos_out, ell_out=None, stream=None):
    """dspark_cache_plan for arrays slot_out and pos_out of any number of rows;
    ell_out [B] (may be ell) gets the admitted lengths that the plan covers."""
    dev = _device_of(table)
    B, max_pages = table.shape
    T = slot_out.numel()
    _launch("dspark_cache_plan_rows", dev, stream, _ints(ctx, dev, B, "ctx"), _ints(ell, dev, B, "ell"), B, int(G),
            int(page), max_pages, free_list.numel(), _ints(table, dev, 1, "table"), _ints(held, dev, B, "held"),
            _ints(free_list, dev, 1, "free_list"), _ints(free_count, dev, 1, "free_count"), T, _dense(ws, dev),
            ws.nbytes, None if ell_out is None else _ints(ell_out, dev, B, "ell_out"),
            _ints(q_start_out, dev, B + 1, "q_start_out"), _ints(kv_len_out, dev, B, "kv_len_out"),
            _ints(slot_out, dev, T, "slot_out"), _ints(pos_out, dev, T, "pos_out"))


def dspark_cache_commit(ctx, q_start, nout, done, table, held, free_list, free_count, page, ws, ctx_out,
                        stream=None):
    """After verification: ctx_out = ctx + nout (-1 where done [B], or None,
    is set), and the pages behind those tokens go back on the free list.
    ctx_out may be ctx."""
    dev = _device_of(table)
    B, max_pages = table.shape
    _launch("dspark_cache_commit", dev, stream, _ints(ctx, dev, B, "ctx"), _ints(q_start, dev, B + 1, "q_start"),
            _ints(nout, dev, B, "nout"), None if done is None else _ints(done, dev, B, "done"), B, int(page),
            max_pages, free_list.numel(), _ints(table, dev, 1, "table"), _ints(held, dev, B, "held"),
            _ints(free_list, dev, 1, "free_list"), _ints(free_count, dev, 1, "free_count"), _dense(ws, dev),
            ws.nbytes, _ints(ctx_out, dev, B, "ctx_out"))


def dspark_cache_commit_round(ctx, q_start, nout, acc, tokens, done, table, held, free_list, free_count, page, ws,
                              ctx_out, stream=None):
    """dspark_cache_commit after a round's verification: requests without
    planned rows emit nothing (nout and acc [B] become 0, tokens [B, G+1] -1,
    in place; acc and tokens may be None)."""
    dev = _device_of(table)
    B, max_pages = table.shape
    G = 0 if tokens is None else tokens.shape[1] - 1
    _launch("dspark_cache_commit_round", dev, stream, _ints(ctx, dev, B, "ctx"), _ints(q_start, dev, B + 1, "q_start"),
            _ints(nout, dev, B, "nout"), None if acc is None else _ints(acc, dev, B, "acc"),
            None if tokens is None else _ints(tokens, dev, B * (G + 1), "tokens"),
            None if done is None else _ints(done, dev, B, "done"), B, G, int(page), max_pages, free_list.numel(),
            _ints(table, dev, 1, "table"), _ints(held, dev, B, "held"), _ints(free_list, dev, 1, "free_list"),
            _ints(free_count, dev, 1, "free_count"), _dense(ws, dev), ws.nbytes, _ints(ctx_out, dev, B, "ctx_out"))


def dspark_qk_norm_rope(q, k, wq, wk, eps, pos, inv_freq, interleaved, n_rows, q_out, k_out, ws, v=None, cache=None,
                        slot=None, page=64, k_scale=1.0, v_scale=1.0, stream=None):
    """Head norms, rotation and (with cache, v and slot) the write of keys and
    values into the 4-bit cache.  q [T, Hq, D], k and v [T, Hkv, D] may be
    slices of one projection; inv_freq [rot/2] f32 (None: no rotation); wq, wk
    [D] or None (no norm); n_rows: device int32 tensor or None."""
    dev = _device_of(q)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    dt = q.dtype
    if k.shape != (T, Hkv, D) or q_out.shape != q.shape or (k_out is not None and k_out.shape != k.shape):
        raise ValueError("q, k, q_out and k_out differ in tokens, heads or dims")
    for t in (k, v, wq, wk, q_out, k_out):
        if t is not None and t.dtype is not dt:
            raise ValueError(f"one dtype for q, k, v, the weights and the outputs: {t.dtype} and {dt}")
    if (wq is not None and wq.numel() != D) or (wk is not None and wk.numel() != D):
        raise ValueError(f"norm weights have {D} elements")
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    if rot and inv_freq.dtype is not torch.float32:
        raise ValueError("inv_freq is float32")
    n_pages, cp, sp, vp, vs = 0, None, None, None, 0
    if cache is not None:
        n_pages, heads = _cache_dims(cache, page, D)
        if v is None or slot is None or v.shape != k.shape or heads != Hkv:
            raise ValueError("a cache write needs v like k, slot, and a cache of k's heads")
        cp, sp = _dense(cache, dev), _ints(slot, dev, T, "slot")
        vp, vs = _rows(v, dev, "v")
    qp, qs = _rows(q, dev, "q")
    kp, ks = _rows(k, dev, "k")
    _launch("dspark_qk_norm_rope", dev, stream, qp, qs, kp, ks, vp, vs, _dense(wq, dev), _dense(wk, dev), float(eps),
            _ints(pos, dev, T, "pos") if rot else None, _dense(inv_freq, dev) if rot else None, rot,
            1 if interleaved else 0, None if n_rows is None else _ints(n_rows, dev, 1, "n_rows"), T, Hq, Hkv, D,
            _dtype(q), _dense(q_out, dev), _dense(k_out, dev), cp, sp, int(page), n_pages, float(k_scale),
            float(v_scale), _dense(ws, dev), ws.nbytes)


def dspark_cache_read(cache, slot, page, k_out, v_out, ws, k_scale=1.0, v_scale=1.0, stream=None):
    """Keys and values of the cached tokens slot [T] -> k_out, v_out
    [T, Hkv, D]; rows with a negative slot are left alone."""
    dev = _device_of(cache)
    T, Hkv, D = k_out.shape
    n_pages, heads = _cache_dims(cache, page, D)
    if v_out.shape != k_out.shape or v_out.dtype is not k_out.dtype or heads != Hkv:
        raise ValueError("k_out, v_out and the cache differ in heads, dims or dtype")
    _launch("dspark_cache_read", dev, stream, _dense(cache, dev), _ints(slot, dev, T, "slot"), T, Hkv, D, int(page),
            n_pages, float(k_scale), float(v_scale), _dtype(k_out), _dense(k_out, dev), _dense(v_out, dev),
            _dense(ws, dev), ws.nbytes)


def dspark_cache_attention_workspace_size(B, Hq, Hkv, D) -> int:
    return int(load().dspark_cache_attention_workspace_size(B, Hq, Hkv, D))


def dspark_cache_attention(q, cache, table, q_start, kv_len, page, scale, window, ws, out, k_scale=1.0, v_scale=1.0,
                           stream=None):
    """Attention of the round's rows q [T, Hq, D] (bf16) over the 4-bit cache:
    causal inside each request's block, the last `window` keys only when
    window > 0; table, q_start and kv_len as dspark_cache_plan leaves them."""
    dev = _device_of(q)
    T, Hq, D = q.shape
    B, max_pages = table.shape
    n_pages, Hkv = _cache_dims(cache, page, D)
    if out.shape != q.shape or out.dtype is not q.dtype:
        raise ValueError("q and out differ in shape or dtype")
    qp, qs = _rows(q, dev, "q")
    _launch("dspark_cache_attention", dev, stream, qp, qs, _dense(cache, dev), _ints(table, dev, 1, "table"),
            _ints(q_start, dev, B + 1, "q_start"), _ints(kv_len, dev, B, "kv_len"), B, T, Hq, Hkv, D, int(page),
            max_pages, n_pages, float(scale), float(k_scale), float(v_scale), int(window), _dtype(q),
            _dense(ws, dev), ws.nbytes, _dense(out, dev))


def dspark_exp2_fma(x, y, stream=None):
    """y = 2^x (float32 device tensors of equal size) by the library's FMA-pipe polynomial."""
    _call("dspark_exp2_fma", _ptr(x), _ptr(y), int(x.numel()), _stream(stream))


def dspark_clear_device_status(ws, stream=None):
    _call("dspark_clear_device_status", _ptr(ws), _stream(stream))
