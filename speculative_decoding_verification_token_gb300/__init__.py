"""GB300 speculative-decoding verification: Python binding of ``libspecverify.so``.

The functions below carry the names of the C entry points declared in ``include/specverify.h`` and
do argument marshalling only: every step runs in the library's CUDA kernels.  Tensors must live on
the current CUDA device; outputs that are not supplied are allocated with torch, for the stream that
the call runs on.  The library is loaded on first use and its absence raises -- there is no other
implementation to fall back to.
"""
from __future__ import annotations

import ctypes as C
import functools
import importlib
import importlib.machinery
import os
import re
import threading
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")
FASTCALL_PATH = os.path.join(_HERE, "_fastcall" + importlib.machinery.EXTENSION_SUFFIXES[0])
HEADER = os.path.join(os.path.dirname(_HERE), "include", "specverify.h")

SV_OK, SV_ERR_INVALID, SV_ERR_UNSUPPORTED, SV_ERR_CUDA, SV_ERR_BAD_INPUT, SV_ERR_TIMEOUT = range(6)
SV_F32, SV_BF16 = 0, 1
SV_HISTORY_OUTPUT, SV_HISTORY_PROMPT = 0, 1
SV_FP4_E8M0_32, SV_FP4_E4M3_16 = 0, 1
SV_MAX_DRAFT_LEN = 64
SV_NOALLOC_SCRATCH_BYTES = 8 << 20  # scratch array of spec_verify_token_noalloc

_lock = threading.Lock()
_lib = None
_fast = None  # the _fastcall module, once the library is loaded


class SpecVerifyError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {status_string(code)}")


def declared_functions():
    """Names of the functions declared in include/specverify.h."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*"
                                 r"([a-z_][a-z0-9_]*)\s*\(", text, flags=re.M)))


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is not None:  # set once, complete
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = C.CDLL(LIB_PATH)
        P, i32, i64, u64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_uint64, C.c_size_t
        st = C.c_int
        verify_args = [P, P, st, i64, i64, P, P, P, i32, P, i32, u64, P, P, P, i64, P]
        sigs = {
            "sv_status_string": (C.c_char_p, [st]),
            "sv_version": (C.c_char_p, []),
            "sv_profile_enable": (st, [C.c_int]),
            "sv_selftest_wait": (st, [i32, i32, P, P]),
            "sv_profile_read": (st, [P]),
            "spec_verify_workspace_bytes": (sz, [i32, i32, i64, st]),
            "spec_verify_token": (st, verify_args + [P, P, P, sz, P]),
            "spec_verify_block": (st, verify_args + [P, P, P, P, sz, P]),
            "spec_verify_token_noalloc": (st, verify_args + [P, P, P]),
            "spec_sample_draft": (st, [P, st, i64, i64, P, P, i32, i32, u64, P, P, P, P, sz, P]),
            "dspark_markov_workspace_bytes": (sz, [i32, i32, i64, i32]),
            "dspark_markov_draft": (st, [P, i64, P, P, i64, P, P, P, i32, i32, i64, i32, u64, P,
                                         P, P, i64, P, P, P, P, sz, P]),
            "dspark_schedule_workspace_bytes": (sz, [i32, i32]),
            "dspark_schedule": (st, [P, P, i32, i32, P, i32, P, P, P, P, P, P, sz, P]),
            "spec_verify_shard_stats": (st, [P, P, st, i64, i64, i64, i64, P, P, P, i32, P, i32,
                                             P, P, P, P, sz, P]),
            "spec_verify_shard_merge": (st, [P, P, i32, i64, P, P, P]),
            "spec_verify_shard_race": (st, [P, P, st, i64, i64, i64, i64, P, P, P, i32, P, i32,
                                            u64, P, P, P, P, P, P, P, P, sz, P]),
            "spec_verify_shard_finish": (st, [P, i32, i32, P, P, P, P, i64, P, P, P]),
            "spec_verify_lmhead_workspace_bytes": (sz, [i32, i32, i64, i64]),
            "spec_verify_lmhead": (st, [P, P, i64, P, i64, i64, i64, P, P, P, i32, P, i32, u64,
                                        P, P, P, i64, P, P, P, P, P, sz, P]),
            "spec_history_append": (st, [P, i64, P, i32, P, i32, i32, i32, i64, i32, P, i64, P, P,
                                         i64, P, P]),
            "spec_process_logits": (st, [P, i64, P, i64, st, i64, P, P, P, i32, i32, i32, P, i32,
                                         P, i32, P, i64, P, P, i64, P, P, P, P, P, P, i64, P, i64,
                                         i32, P, P, P]),
            "spec_fp4_row_bytes": (i64, [i64]),
            "spec_fp4_scale_bytes": (sz, [i64, i64, i32]),
            "spec_quantize_fp4": (st, [P, st, i64, i64, i64, i32, P, P, P, P, i64, P, P]),
            "spec_project_fp4": (st, [P, P, P, i64, P, P, P, i64, i64, i32, P, st, i64, P, P]),
            "dspark_schedule_rule": (st, [P, P, i32, i32, P, i32, i32, P, P, P, P, P, P, sz, P]),
            "dspark_schedule_async": (st, [P, i32, i64, P, P, i32, i32, P, i32, i32, P, P, P, P, P,
                                           P, sz, P]),
            "dspark_acceptance_update": (st, [P, P, i32, i32, C.c_double, C.c_double, C.c_double,
                                              P, P, P, P, P, P]),
            "dspark_sts_fit": (st, [P, P, P, i32, i32, i32, C.c_double, C.c_double, i32, P, P, P,
                                    P, P, P, P]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _bind_fastcall(L)
        _lib = L
        return L


def _bind_fastcall(L):
    """Gives the marshalling module the entry points' addresses.  Where it is missing, or does not
    load, the library is called through ctypes alone."""
    global _fast
    if not os.path.exists(FASTCALL_PATH):
        return
    try:
        module = importlib.import_module("._fastcall", __name__)
    except ImportError as e:
        warnings.warn(f"_fastcall is not used, it does not load ({e}): build again", RuntimeWarning)
        return
    module.bind(*(C.cast(getattr(L, name), C.c_void_p).value for name in (
        "spec_history_append", "spec_process_logits", "spec_quantize_fp4", "spec_project_fp4")))
    _fast = module


def status_string(code):
    return lib().sv_status_string(int(code)).decode()


def version():
    return lib().sv_version().decode()


def sv_selftest_wait(which, limit_us, status, stream=None):
    """Make one of the kernels' bounded waits run out (see include/specverify.h)."""
    _check(lib().sv_selftest_wait(int(which), int(limit_us), _ptr(status), _stream(stream)),
           "sv_selftest_wait")


def sv_profile_enable(enable=True):
    _check(lib().sv_profile_enable(int(enable)), "sv_profile_enable")


def sv_profile_read():
    """Durations (ms) of the last profiled verify call: [streaming, decisions, race]."""
    out = (C.c_float * 3)()
    _check(lib().sv_profile_read(out), "sv_profile_read")
    return [float(x) for x in out]


def _check(code, where):
    if code != SV_OK:
        raise SpecVerifyError(code, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    # torch.cuda.current_stream().cuda_stream without the stream object (3 us of a short call)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _torch_stream(stream):
    """The torch stream of any object with a cuda_stream."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(stream.cuda_stream)


def _on_its_stream(call):
    """A call with a parameter `stream` whose own tensors -- outputs, status, workspace -- belong
    to the stream it runs on: their memory is not in use by work that the stream has still to wait
    for, and their fills are in order with the kernels.  Results are kept for the current stream
    too, for a caller who goes on with them there."""
    at = call.__code__.co_varnames.index("stream")

    @functools.wraps(call)
    def run(*args, stream=None, **kw):
        if len(args) > at:
            args, stream = args[:at] + (None,) + args[at + 1:], args[at]
        if stream is None:
            return call(*args, **kw)
        here = torch.cuda.current_stream()
        with torch.cuda.stream(_torch_stream(stream)):
            out = call(*args, **kw)
        results = out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,)
        for t in results:
            if t is not None and t.is_cuda:  # not an output of the caller's in pinned host memory
                t.record_stream(here)
        return out

    return run


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float32:
        return SV_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _dev(t, dtype=None, rows=False, strided=False):
    """Checks a device tensor; `rows` allows a row-strided 2-D view (logits with ld > V) and
    `strided` leaves the layout to the caller's own checks."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the library must be on a CUDA device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"expected {dtype}, got {t.dtype}")
    if rows:
        if t.dim() != 2 or t.stride(1) != 1:
            raise ValueError("logits must be a 2-D tensor with unit column stride")
    elif not strided and not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t


_ws_cache = {}


def workspace(nbytes, device=None):
    """A cached device buffer of at least `nbytes` bytes (256-byte aligned, from torch), one for each
    host thread and stream: calls on two streams must not share their scratch.  A larger request
    replaces it, so a captured graph that outlives that wants a workspace of its own."""
    device = torch.device(device or torch.cuda.current_device())
    index = torch.cuda.current_device() if device.index is None else device.index
    key = (index, threading.get_ident(), torch._C._cuda_getCurrentRawStream(index))
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


# ---- verification ----------------------------------------------------------------------------

def spec_verify_workspace_bytes(B, max_draft_len, V, dtype_code):
    return int(lib().spec_verify_workspace_bytes(B, max_draft_len, V, dtype_code))


def _verify(block, target, draft, target_row0, draft_row0, draft_len, max_draft_len,
            draft_tokens, seed, request_ids, out_ld, want_rows, status, ws, stream):
    _dev(target, rows=True), _dev(draft, rows=True)
    _dev(target_row0, torch.int64), _dev(draft_row0, torch.int64)
    _dev(draft_len, torch.int32), _dev(draft_tokens, torch.int32)
    _dev(request_ids)
    dt = _dtype_code(target)
    if draft.dtype != target.dtype:
        raise TypeError("target and draft logits must have the same dtype")
    V = target.shape[-1]
    ld = target.stride(0)
    if draft.stride(0) != ld:
        raise ValueError("target and draft rows must have the same stride")
    B = draft_len.numel()
    out_ld = out_ld or max_draft_len + 1
    dev = target.device
    accepted = torch.empty(B, dtype=torch.int32, device=dev)
    out_tokens = torch.empty((B, out_ld), dtype=torch.int32, device=dev)
    correction = torch.empty(B, dtype=torch.int32, device=dev)
    n_draft_rows = draft_tokens.numel()
    rows_a = torch.empty(n_draft_rows, dtype=torch.float32, device=dev) if want_rows else None
    rows_h = (torch.empty(n_draft_rows, dtype=torch.float32, device=dev)
              if (want_rows and block) else None)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    need = spec_verify_workspace_bytes(B, max_draft_len, V, dt)
    if ws is None:
        ws = workspace(need, dev)
    args = [_ptr(target), _ptr(draft), dt, V, ld, _ptr(target_row0), _ptr(draft_row0),
            _ptr(draft_len), int(max_draft_len), _ptr(draft_tokens), B, int(seed),
            _ptr(request_ids), _ptr(accepted), _ptr(out_tokens), out_ld, _ptr(correction)]
    if block:
        code = lib().spec_verify_block(*args, _ptr(rows_a), _ptr(rows_h), _ptr(status),
                                       _ptr(ws), ws.numel(), _stream(stream))
    else:
        code = lib().spec_verify_token(*args, _ptr(rows_a), _ptr(status), _ptr(ws), ws.numel(),
                                       _stream(stream))
    _check(code, "spec_verify_block" if block else "spec_verify_token")
    out = {"accepted_len": accepted, "out_tokens": out_tokens, "correction": correction,
           "status": status}
    if block:
        out["running_ratio"] = rows_a
        out["h"] = rows_h
    else:
        out["accept_ratio"] = rows_a
    return out


@_on_its_stream
def spec_verify_token(target, draft, target_row0, draft_row0, draft_len, max_draft_len,
                      draft_tokens, seed, request_ids=None, out_ld=None, want_ratio=True,
                      status=None, workspace=None, stream=None):
    """Token-level verification (see include/specverify.h).  Returns a dict of device tensors."""
    return _verify(False, target, draft, target_row0, draft_row0, draft_len, max_draft_len,
                   draft_tokens, seed, request_ids, out_ld, want_ratio, status, workspace, stream)


@_on_its_stream
def spec_verify_block(target, draft, target_row0, draft_row0, draft_len, max_draft_len,
                      draft_tokens, seed, request_ids=None, out_ld=None, want_rows=True,
                      status=None, workspace=None, stream=None):
    """Block verification (see include/specverify.h).  Returns a dict of device tensors."""
    return _verify(True, target, draft, target_row0, draft_row0, draft_len, max_draft_len,
                   draft_tokens, seed, request_ids, out_ld, want_rows, status, workspace, stream)


def spec_verify_lmhead_workspace_bytes(B, max_draft_len, V, H):
    return int(lib().spec_verify_lmhead_workspace_bytes(B, max_draft_len, V, H))


@_on_its_stream
def spec_verify_lmhead(target_hidden, draft_hidden, W, target_row0, draft_row0, draft_len,
                       max_draft_len, draft_tokens, seed, request_ids=None, out_ld=None,
                       want_ratio=True, status=None, workspace=None, stream=None):
    """Token-level verification from hidden states: logits = hidden rows x W^T (bf16 operands,
    W [V, H]), decided and sampled as spec_verify_token does (see include/specverify.h).
    Returns a dict of device tensors."""
    _dev(target_hidden, torch.bfloat16, rows=True), _dev(draft_hidden, torch.bfloat16, rows=True)
    _dev(W, torch.bfloat16, rows=True)
    _dev(target_row0, torch.int64), _dev(draft_row0, torch.int64)
    _dev(draft_len, torch.int32), _dev(draft_tokens, torch.int32)
    _dev(request_ids)
    H = target_hidden.shape[-1]
    if draft_hidden.shape[-1] != H or W.shape[-1] != H:
        raise ValueError("hidden rows and W must have the same width H")
    ldh = target_hidden.stride(0)
    if draft_hidden.stride(0) != ldh:
        raise ValueError("target and draft hidden rows must have the same stride")
    V = W.shape[0]
    B = draft_len.numel()
    out_ld = out_ld or max_draft_len + 1
    dev = target_hidden.device
    accepted = torch.empty(B, dtype=torch.int32, device=dev)
    out_tokens = torch.empty((B, out_ld), dtype=torch.int32, device=dev)
    correction = torch.empty(B, dtype=torch.int32, device=dev)
    ratio = (torch.empty(draft_tokens.numel(), dtype=torch.float32, device=dev)
             if want_ratio else None)
    recomputed = torch.zeros(1, dtype=torch.int32, device=dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    need = spec_verify_lmhead_workspace_bytes(B, max_draft_len, V, H)
    ws = workspace if workspace is not None else globals()["workspace"](need, dev)
    code = lib().spec_verify_lmhead(_ptr(target_hidden), _ptr(draft_hidden), ldh, _ptr(W),
                                    W.stride(0), H, V, _ptr(target_row0), _ptr(draft_row0),
                                    _ptr(draft_len), int(max_draft_len), _ptr(draft_tokens), B,
                                    int(seed), _ptr(request_ids), _ptr(accepted),
                                    _ptr(out_tokens), out_ld, _ptr(correction), _ptr(ratio),
                                    _ptr(recomputed), _ptr(status), _ptr(ws), ws.numel(),
                                    _stream(stream))
    _check(code, "spec_verify_lmhead")
    return {"accepted_len": accepted, "out_tokens": out_tokens, "correction": correction,
            "accept_ratio": ratio, "recomputed": recomputed, "status": status}


@_on_its_stream
def spec_sample_draft(draft, draft_row0, draft_len, max_draft_len, seed, request_ids=None,
                      draft_tokens=None, status=None, workspace=None, stream=None):
    """Sample draft tokens from q for every drafted row; returns the token tensor (by draft row)."""
    _dev(draft, rows=True), _dev(draft_row0, torch.int64), _dev(draft_len, torch.int32)
    dt = _dtype_code(draft)
    V = draft.shape[-1]
    ld = draft.stride(0)
    B = draft_len.numel()
    dev = draft.device
    if draft_tokens is None:
        draft_tokens = torch.full((draft.shape[0],), -1, dtype=torch.int32, device=dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    need = spec_verify_workspace_bytes(B, max_draft_len, V, dt)
    ws = workspace if workspace is not None else globals()["workspace"](need, dev)
    code = lib().spec_sample_draft(_ptr(draft), dt, V, ld, _ptr(draft_row0), _ptr(draft_len),
                                   int(max_draft_len), B, int(seed), _ptr(request_ids),
                                   _ptr(draft_tokens), _ptr(status), _ptr(ws), ws.numel(),
                                   _stream(stream))
    _check(code, "spec_sample_draft")
    return draft_tokens


# ---- vocabulary-sharded verification ------------------------------------------------------------

@_on_its_stream
def spec_verify_shard_stats(target, draft, v_off, V_total, target_row0, draft_row0, draft_len,
                            max_draft_len, draft_tokens, status=None, workspace=None, stream=None):
    """This shard's statistics of every drafted row pair and the drafted tokens' logits (-inf
    where the shard does not hold the token).  Returns (stats fp32 [B * gmax, 4], tok fp32
    [B * gmax, 2])."""
    _dev(target, rows=True), _dev(draft, rows=True)
    _dev(target_row0, torch.int64), _dev(draft_row0, torch.int64)
    _dev(draft_len, torch.int32), _dev(draft_tokens, torch.int32)
    dt = _dtype_code(target)
    Vs, ld = target.shape[-1], target.stride(0)
    B = draft_len.numel()
    dev = target.device
    units = max(1, B * max_draft_len)
    stats = torch.empty((units, 4), dtype=torch.float32, device=dev)
    tok = torch.empty((units, 2), dtype=torch.float32, device=dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    need = spec_verify_workspace_bytes(B, max_draft_len, Vs, dt)
    ws = workspace if workspace is not None else globals()["workspace"](need, dev)
    code = lib().spec_verify_shard_stats(_ptr(target), _ptr(draft), dt, Vs, ld, int(v_off),
                                         int(V_total), _ptr(target_row0), _ptr(draft_row0),
                                         _ptr(draft_len), int(max_draft_len), _ptr(draft_tokens),
                                         B, _ptr(stats), _ptr(tok), _ptr(status), _ptr(ws),
                                         ws.numel(), _stream(stream))
    _check(code, "spec_verify_shard_stats")
    return stats, tok


@_on_its_stream
def spec_verify_shard_merge(stats_all, tok_all, stream=None):
    """Statistics of every shard ([n, rows, 4]) merged in shard order; drafted-token logits
    ([n, rows, 2]) from the shard that holds each token."""
    _dev(stats_all, torch.float32), _dev(tok_all, torch.float32)
    n, rows = stats_all.shape[0], stats_all.shape[1]
    stats = torch.empty((rows, 4), dtype=torch.float32, device=stats_all.device)
    tok = torch.empty((rows, 2), dtype=torch.float32, device=stats_all.device)
    code = lib().spec_verify_shard_merge(_ptr(stats_all.contiguous()), _ptr(tok_all.contiguous()),
                                         n, rows, _ptr(stats), _ptr(tok), _stream(stream))
    _check(code, "spec_verify_shard_merge")
    return stats, tok


@_on_its_stream
def spec_verify_shard_race(target, draft, v_off, V_total, target_row0, draft_row0, draft_len,
                           max_draft_len, draft_tokens, seed, stats, tok, request_ids=None,
                           want_ratio=True, status=None, workspace=None, stream=None):
    """Every request decided from the merged statistics, then this shard's race.  Returns
    {"accepted_len", "winners" (int64 [B, 2], unsigned bit patterns), "accept_ratio", "status"}."""
    _dev(target, rows=True), _dev(draft, rows=True), _dev(request_ids)
    dt = _dtype_code(target)
    Vs, ld = target.shape[-1], target.stride(0)
    B = draft_len.numel()
    dev = target.device
    acc = torch.empty(B, dtype=torch.int32, device=dev)
    winners = torch.empty((B, 2), dtype=torch.int64, device=dev)
    ratio = (torch.empty(draft_tokens.numel(), dtype=torch.float32, device=dev)
             if want_ratio else None)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    need = spec_verify_workspace_bytes(B, max_draft_len, Vs, dt)
    ws = workspace if workspace is not None else globals()["workspace"](need, dev)
    code = lib().spec_verify_shard_race(_ptr(target), _ptr(draft), dt, Vs, ld, int(v_off),
                                        int(V_total), _ptr(target_row0), _ptr(draft_row0),
                                        _ptr(draft_len), int(max_draft_len), _ptr(draft_tokens),
                                        B, int(seed), _ptr(request_ids), _ptr(stats), _ptr(tok),
                                        _ptr(acc), _ptr(ratio), _ptr(winners), _ptr(status),
                                        _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "spec_verify_shard_race")
    return {"accepted_len": acc, "winners": winners, "accept_ratio": ratio, "status": status}


@_on_its_stream
def spec_verify_shard_finish(winners_all, accepted_len, draft_row0, draft_tokens, out_ld,
                             status=None, stream=None):
    """The largest winner over the shards ([n, B, 2]) and the request outputs."""
    _dev(winners_all, torch.int64), _dev(accepted_len, torch.int32)
    n, B = winners_all.shape[0], winners_all.shape[1]
    dev = winners_all.device
    out = torch.empty((B, out_ld), dtype=torch.int32, device=dev)
    corr = torch.empty(B, dtype=torch.int32, device=dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    code = lib().spec_verify_shard_finish(_ptr(winners_all.contiguous()), n, B,
                                          _ptr(accepted_len), _ptr(draft_row0),
                                          _ptr(draft_tokens), _ptr(out), int(out_ld),
                                          _ptr(corr), _ptr(status), _stream(stream))
    _check(code, "spec_verify_shard_finish")
    return {"out_tokens": out, "correction": corr, "accepted_len": accepted_len,
            "status": status}


def all_gather_stacked(t, group=None):
    """The tensor t of every rank of `group`, stacked in rank order (the shard order)."""
    import torch.distributed as dist
    parts = [torch.empty_like(t) for _ in range(dist.get_world_size(group))]
    dist.all_gather(parts, t.contiguous(), group=group)
    return torch.stack(parts)


def spec_verify_token_sharded(target, draft, v_off, V_total, target_row0, draft_row0, draft_len,
                              max_draft_len, draft_tokens, seed, request_ids=None, out_ld=None,
                              gather=all_gather_stacked, steps=None):
    """Token-level verification of this rank's vocabulary shard (columns v_off .. v_off + Vs of
    every row), rank r holding shard r: the four library calls with the two exchanges between
    them, `gather(t)` stacking every rank's t in rank order (all_gather over the default process
    group by default).  `steps` replaces the four calls (a dict with keys stats, merge, race,
    finish taking the same arguments) -- the exchanges stay the same."""
    st = steps or {"stats": spec_verify_shard_stats, "merge": spec_verify_shard_merge,
                   "race": spec_verify_shard_race, "finish": spec_verify_shard_finish}
    stats, tok = st["stats"](target, draft, v_off, V_total, target_row0, draft_row0, draft_len,
                             max_draft_len, draft_tokens)
    stats, tok = st["merge"](gather(stats), gather(tok))
    race = st["race"](target, draft, v_off, V_total, target_row0, draft_row0, draft_len,
                      max_draft_len, draft_tokens, seed, stats, tok, request_ids=request_ids)
    out = st["finish"](gather(race["winners"]), race["accepted_len"], draft_row0, draft_tokens,
                       out_ld or max_draft_len + 1)
    out["accept_ratio"] = race.get("accept_ratio")
    return out


# ---- logits before verification ----------------------------------------------------------------
# These calls are short, so that checking their arguments counts: _fastcall does it in C++ and makes
# the call, and declines (-1) all that is not plain -- the checks below then find out what it is.

def _load_fast():
    lib()
    return _fast


def _refuse(t, name, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)} with strides {t.stride()}")


def _device_of(t, name):
    """Index of the device a call works on: the tensor's, which must be the current one."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or (
            t.get_device() != torch._C._cuda_getDevice()):
        _refuse(t, name, None, "")
    return t.get_device()


def _vec(t, name, dtype, n, dev):
    """Pointer of a contiguous tensor [n] on device `dev` (n None: any length); None stays None."""
    if t is None:
        return None
    try:
        if (t.get_device() == dev and t.dtype == dtype and t.is_contiguous()
                and (n is None or t.shape == (n,))):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, "contiguous" if n is None else f"contiguous [{n}]")


def _mat(t, name, dtype, dev, rows=None, cols=1):
    """(pointer, row stride) of a 2-D tensor with unit column stride on device `dev`, of at least
    `cols` columns and exactly `rows` rows if given.  A single row's stride says nothing: the next
    multiple of 8 will do."""
    try:
        n, m = t.shape
        ld, step = t.stride()
        if (t.get_device() == dev and t.dtype == dtype and (step == 1 or m <= 1) and m >= cols
                and (rows is None or n == rows)):
            return t.data_ptr(), ld if n > 1 else (max(ld, m) + 7) // 8 * 8
    except (AttributeError, ValueError):
        pass
    _refuse(t, name, dtype, f"[{rows or 'rows'}, {cols} or more] with unit column stride")


def _empty(shape, dtype, dev, stream):
    """A tensor of the call's own, not filled, on device `dev`.  Given `stream`, it is that stream's:
    its memory is not in use by work that the stream has still to wait for, and is not given away
    before the call has written it.  It outlives the current stream's work too, for a caller who
    goes on with it there."""
    device = torch.device("cuda", dev)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream()
    with torch.cuda.stream(_torch_stream(stream)):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(here)
    return t


def _status_ptr(status, dev, stream):
    """The status word of a call that returns it, and its pointer; every call resets it."""
    if status is None:
        status = _empty(1, torch.int32, dev, stream)
    return status, _vec(status, "status", torch.int32, None, dev)


def _history(counts, prompt_bits, output_bits, dev):
    """Checks the history tensors; returns (counts, prompt bits, output bits, slots, strides, V)."""
    i32 = torch.int32
    c, ldc = _mat(counts, "counts", i32, dev)
    n_slots, V = counts.shape
    words = (V + 31) // 32
    pb, ldb = _mat(prompt_bits, "prompt_bits", i32, dev, n_slots, words)
    ob, ldo = _mat(output_bits, "output_bits", i32, dev, n_slots, words)
    if ldo != ldb and n_slots > 1:
        raise ValueError("prompt_bits and output_bits must have the same stride")
    return c, pb, ob, n_slots, ldc, ldb, V


def spec_history_append(tokens, counts, prompt_bits, output_bits, slots=None, lens=None,
                        prompt=False, reset=False, status=None, stream=None):
    """Adds tokens int32 [B, n] (negative: padding; only the first lens[r] columns if given) to
    the history of slots int32 [B] (default: row r in slot r), in place: counts int32 [S, V] and
    the bit rows int32 [S, ceil(V / 32)] (see include/specverify.h).  `prompt` marks them as prompt
    tokens instead of counting them; `reset` clears the listed slots first.  Returns the status."""
    if status is not None and (_fast or _load_fast()):
        code = _fast.history_append(tokens, counts, prompt_bits, output_bits, slots, lens, prompt,
                                    reset, status, stream)
        if code == 0:
            return status
        if code > 0:
            raise SpecVerifyError(code, "spec_history_append")
    dev = _device_of(tokens, "tokens")
    tk, ldt = _mat(tokens, "tokens", torch.int32, dev, cols=0)
    c, pb, ob, n_slots, ldc, ldb, V = _history(counts, prompt_bits, output_bits, dev)
    B, n = tokens.shape
    if slots is None and B > n_slots:
        raise ValueError("more rows than slots")
    status, st = _status_ptr(status, dev, stream)
    code = lib().spec_history_append(
        tk, ldt, _vec(lens, "lens", torch.int32, B, dev), n,
        _vec(slots, "slots", torch.int32, B, dev), B, int(prompt), int(reset), V, n_slots, c, ldc,
        pb, ob, ldb, st, _stream(stream))
    _check(code, "spec_history_append")
    return status


def spec_process_logits(logits, row0, draft_row0, draft_len, max_draft_len, draft_tokens,
                        first_row=0, bonus_row=True, slots=None, counts=None, prompt_bits=None,
                        output_bits=None, repetition=None, presence=None, frequency=None,
                        bias_start=None, bias_tokens=None, bias_values=None, mask=None,
                        mask_row=None, out=None, status=None, stream=None):
    """Repetition / presence / frequency penalties (fp32 [B]), logit biases (bias_start int32
    [B + 1] into ascending bias_tokens int32 and bias_values fp32) and grammar masks (mask int32
    [n, ceil(V / 32)] bit rows, mask_row int32 per logit row, -1: none) on the rows of a round
    (see include/specverify.h).  Works in place unless `out` is another tensor of the same shape
    and dtype.  Returns out.  Data errors go to `status`; without one they go unreported."""
    if out is None:
        out = logits
    if _fast or _load_fast():
        code = _fast.process_logits(
            logits, row0, draft_row0, draft_len, max_draft_len, draft_tokens, first_row, bonus_row,
            slots, counts, prompt_bits, output_bits, repetition, presence, frequency, bias_start,
            bias_tokens, bias_values, mask, mask_row, out, status, stream)
        if code == 0:
            return out
        if code > 0:
            raise SpecVerifyError(code, "spec_process_logits")
    dev = _device_of(logits, "logits")
    dt = _dtype_code(logits)
    lg, ld = _mat(logits, "logits", logits.dtype, dev)
    rows, V = logits.shape
    B = draft_len.numel()
    ot, ldo = _mat(out, "out", logits.dtype, dev, rows, V)
    if out.shape[1] != V:
        raise ValueError("out must have the shape of the logits")
    f32, i32, i64 = torch.float32, torch.int32, torch.int64
    rep = _vec(repetition, "repetition", f32, B, dev)
    pres = _vec(presence, "presence", f32, B, dev)
    freq = _vec(frequency, "frequency", f32, B, dev)
    c = pb = ob = sl = None
    n_slots = ldc = ldb = 0
    if rep is not None or pres is not None or freq is not None:
        if counts is None or prompt_bits is None or output_bits is None:
            raise ValueError("penalties need counts, prompt_bits and output_bits")
        c, pb, ob, n_slots, ldc, ldb, hv = _history(counts, prompt_bits, output_bits, dev)
        if hv != V:
            raise ValueError("the history's vocabulary differs from the logits'")
        sl = _vec(slots, "slots", i32, B, dev)
        if slots is None and B > n_slots:
            raise ValueError("more requests than slots")
    bs = _vec(bias_start, "bias_start", i32, B + 1, dev)
    bt = bv = None
    n_bias = 0
    if bs is not None:
        bt = _vec(bias_tokens, "bias_tokens", i32, None, dev)
        if bt is None or bias_values is None:
            raise ValueError("bias_start needs bias_tokens and bias_values")
        n_bias = bias_tokens.numel()
        bv = _vec(bias_values, "bias_values", f32, n_bias, dev)
    mr = _vec(mask_row, "mask_row", i32, rows, dev)
    mk = None
    n_mask = ldm = 0
    if mr is not None:
        mk, ldm = _mat(mask, "mask", i32, dev, None, (V + 31) // 32)
        n_mask = mask.shape[0]
    st = _vec(status, "status", torch.int32, None, dev)
    code = lib().spec_process_logits(
        lg, ld, ot, ldo, dt, V, _vec(row0, "row0", i64, B, dev),
        _vec(draft_row0, "draft_row0", i64, B, dev), _vec(draft_len, "draft_len", i32, B, dev),
        int(max_draft_len), int(first_row), int(bonus_row),
        _vec(draft_tokens, "draft_tokens", i32, None, dev), B, sl, n_slots, c, ldc, pb, ob, ldb,
        rep, pres, freq, bs, bt, bv, n_bias, mk, ldm, n_mask, mr, st, _stream(stream))
    _check(code, "spec_process_logits")
    return out


# ---- the output projection in 4 bits -------------------------------------------------------------

_FP4_BLOCK = {SV_FP4_E8M0_32: 32, SV_FP4_E4M3_16: 16}


def spec_fp4_row_bytes(H):
    return int(lib().spec_fp4_row_bytes(H))


def spec_fp4_scale_bytes(rows, H, fmt):
    return int(lib().spec_fp4_scale_bytes(rows, H, fmt))


def _fp4_sizes(rows, H, fmt):
    """(packed bytes of a row, bytes of all scales): 128-row tiles, 256-element spans."""
    return (H + 31) // 32 * 16, (rows + 127) // 128 * ((H + 255) // 256) * (32768 // _FP4_BLOCK[fmt])


def spec_quantize_fp4(x, fmt, packed=None, scales=None, row_scales=None, values=None, status=None,
                      stream=None):
    """Rows x [rows, H] (bf16 or fp32, any row stride) to blocks of 4-bit values in format `fmt`
    (see include/specverify.h).  Returns {"packed", "scales", "row_scales", "rows", "H", "format",
    "status"}, which spec_project_fp4 takes as an operand; `values`, a bf16 [rows, H] tensor, is
    filled with the numbers the codes stand for."""
    if status is not None and packed is not None and scales is not None and (_fast or _load_fast()):
        code = _fast.quantize_fp4(x, fmt, packed, scales, row_scales, values, status, stream)
        if code == 0:
            rows, H = x.shape
            return {"packed": packed, "scales": scales,
                    "row_scales": row_scales if fmt == SV_FP4_E4M3_16 else None, "rows": rows,
                    "H": H, "format": fmt, "status": status}
        if code > 0:
            raise SpecVerifyError(code, "spec_quantize_fp4")
    dev = _device_of(x, "x")
    dt = _dtype_code(x)
    xp, ldx = _mat(x, "x", x.dtype, dev)
    rows, H = x.shape
    if fmt not in _FP4_BLOCK:
        raise ValueError("fmt must be SV_FP4_E8M0_32 or SV_FP4_E4M3_16")
    rb, nbytes = _fp4_sizes(rows, H, fmt)
    if packed is None:
        packed = _empty((rows, rb), torch.uint8, dev, stream)
    elif packed.shape != (rows, rb):
        raise ValueError(f"packed must be [{rows}, {rb}]")
    if scales is None:
        scales = _empty(nbytes, torch.uint8, dev, stream)
    elif scales.numel() != nbytes:
        raise ValueError(f"scales must hold {nbytes} bytes")
    rs = None
    if fmt == SV_FP4_E4M3_16:
        if row_scales is None:
            row_scales = _empty(rows, torch.float32, dev, stream)
        rs = _vec(row_scales, "row_scales", torch.float32, rows, dev)
    else:
        row_scales = None
    vp, ldv = None, 0
    if values is not None:
        vp, ldv = _mat(values, "values", torch.bfloat16, dev, rows, H)
        if values.shape[1] != H:
            raise ValueError("values must have the shape of x")
    status, st = _status_ptr(status, dev, stream)
    u8 = torch.uint8
    code = lib().spec_quantize_fp4(xp, dt, rows, H, ldx, fmt,
                                   _vec(packed, "packed", u8, None, dev),
                                   _vec(scales, "scales", u8, None, dev), rs, vp, ldv, st,
                                   _stream(stream))
    _check(code, "spec_quantize_fp4")
    return {"packed": packed, "scales": scales, "row_scales": row_scales, "rows": rows, "H": H,
            "format": fmt, "status": status}


def _fp4_operand(t, name, dev):
    """(packed, scales, row scales, rows, H, format) of an operand, checked."""
    rows, H, fmt = t["rows"], t["H"], t["format"]
    if fmt not in _FP4_BLOCK:
        raise ValueError(f"{name}: unknown format {fmt}")
    rb, nbytes = _fp4_sizes(rows, H, fmt)
    packed, scales = t["packed"], t["scales"]
    if packed.shape != (rows, rb) or scales.numel() != nbytes:
        raise ValueError(f"{name}: packed and scales do not fit [{rows}, {H}]")
    rs = None
    if fmt == SV_FP4_E4M3_16:
        rs = _vec(t["row_scales"], name + " row_scales", torch.float32, rows, dev)
    return (_vec(packed, name + " packed", torch.uint8, None, dev),
            _vec(scales, name + " scales", torch.uint8, None, dev), rs, rows, H, fmt)


def spec_project_fp4(x, w, out=None, dtype=torch.bfloat16, status=None, stream=None):
    """Logits [M, V] = x w^T of two operands quantised by spec_quantize_fp4: hidden rows x [M, H]
    and the output projection w [V, H] (see include/specverify.h).  `out` (bf16 or fp32, rows
    16-byte aligned) is allocated in `dtype` if not given.  Returns it.  A wait that ran out is
    written to `status`; without one it goes unreported."""
    if out is not None and (_fast or _load_fast()) and (
            x["H"] == w["H"] and x["format"] == w["format"]):
        code = _fast.project_fp4(x["packed"], x["scales"], x["row_scales"], x["rows"], w["packed"],
                                 w["scales"], w["row_scales"], w["rows"], x["H"], x["format"], out,
                                 status, stream)
        if code == 0:
            return out
        if code > 0:
            raise SpecVerifyError(code, "spec_project_fp4")
    dev = _device_of(x["packed"], "x packed")
    xp, xs, xr, M, H, fmt = _fp4_operand(x, "x", dev)
    wp, ws, wr, V, Hw, fw = _fp4_operand(w, "w", dev)
    if Hw != H or fw != fmt:
        raise ValueError("x and w must have the same width and format")
    if out is None:
        ld = (V + 7) // 8 * 8  # rows start on 16-byte boundaries
        out = _empty((M, ld), dtype, dev, stream)[:, :V]
    dt = _dtype_code(out)
    op, ld = _mat(out, "out", out.dtype, dev, M, V)
    if out.shape[1] != V:
        raise ValueError(f"out must be [{M}, {V}]")
    st = _vec(status, "status", torch.int32, None, dev)
    code = lib().spec_project_fp4(xp, xs, xr, M, wp, ws, wr, V, H, fmt, op, dt, ld, st,
                                  _stream(stream))
    _check(code, "spec_project_fp4")
    return out


# ---- DSpark draft side ------------------------------------------------------------------------

def dspark_markov_workspace_bytes(B, K, V, R):
    return int(lib().dspark_markov_workspace_bytes(B, K, V, R))


@_on_its_stream
def dspark_markov_draft(backbone, U, Wt, anchor, conf_scores, sts_T, seed, request_ids=None,
                        want_logits=True, want_stats=True, status=None, workspace=None,
                        stream=None):
    """Markov-head drafting.  backbone bf16 [B, K, V] (rows may be padded: stride(1) = ldb,
    stride(0) = K * ldb); U bf16 [V, R]; Wt bf16 [V, R] (W stored transposed, rows may be padded);
    anchor int32 [B]; conf_scores fp32 [B, K] and sts_T fp32 [K], or both None (no confidence)."""
    _dev(backbone, torch.bfloat16, strided=True), _dev(U, torch.bfloat16)
    _dev(Wt, torch.bfloat16, strided=True), _dev(anchor, torch.int32)
    if conf_scores is not None:
        _dev(conf_scores, torch.float32), _dev(sts_T, torch.float32)
    B, K, V = backbone.shape
    R = U.shape[1]
    ldb = backbone.stride(1)
    if backbone.stride(2) != 1 or backbone.stride(0) != K * ldb:
        raise ValueError("backbone must be [B, K, V] with unit column stride and rows ldb apart")
    if U.stride(1) != 1 or U.stride(0) != R or Wt.stride(1) != 1 or Wt.shape[0] != V:
        raise ValueError("U must be a contiguous [V, R] tensor and Wt a [V, R] row-major tensor")
    dev = backbone.device
    tokens = torch.empty((B, K), dtype=torch.int32, device=dev)
    ldz = (V + 7) // 8 * 8  # rows of z start on 16-byte boundaries
    z = (torch.empty((B, K, ldz), dtype=torch.bfloat16, device=dev)[:, :, :V] if want_logits
         else None)
    stats = torch.empty((B, K, 2), dtype=torch.float32, device=dev) if want_stats else None
    conf = torch.empty((B, K), dtype=torch.float32, device=dev) if conf_scores is not None else None
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    need = dspark_markov_workspace_bytes(B, K, V, R)
    ws = workspace if workspace is not None else globals()["workspace"](need, dev)
    code = lib().dspark_markov_draft(_ptr(backbone), ldb, _ptr(U), _ptr(Wt), Wt.stride(0),
                                     _ptr(anchor), _ptr(conf_scores), _ptr(sts_T), B, K, V, R,
                                     int(seed), _ptr(request_ids), _ptr(tokens), _ptr(z),
                                     ldz, _ptr(stats), _ptr(conf), _ptr(status), _ptr(ws),
                                     ws.numel(), _stream(stream))
    _check(code, "dspark_markov_draft")
    return {"draft_tokens": tokens, "draft_logits": z, "row_stats": stats, "conf": conf,
            "status": status}


def dspark_schedule_workspace_bytes(N, K):
    return int(lib().dspark_schedule_workspace_bytes(N, K))


SV_STOP_FIRST_DROP = 0
SV_STOP_ARGMAX = 1
SV_STOP_FIXED_DEPTH = 2


@_on_its_stream
def dspark_schedule(cond_accept, max_len, sps, B_max, want_survival=True, status=None,
                    workspace=None, stream=None, rule=SV_STOP_FIRST_DROP):
    """Hardware-aware prefix scheduler.  cond_accept fp32 [N, K]; sps fp64 [B_max + 1]; rule:
    SV_STOP_FIRST_DROP (early stop), SV_STOP_ARGMAX (best budget over all) or
    SV_STOP_FIXED_DEPTH (one depth for every request)."""
    _dev(cond_accept, torch.float32), _dev(max_len, torch.int32), _dev(sps, torch.float64)
    N, K = cond_accept.shape
    dev = cond_accept.device
    sel = torch.empty(N, dtype=torch.int32, device=dev)
    surv = torch.empty((N, K), dtype=torch.float32, device=dev) if want_survival else None
    total = torch.empty(1, dtype=torch.int32, device=dev)
    obj = torch.empty(1, dtype=torch.float64, device=dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    need = dspark_schedule_workspace_bytes(N, K)
    ws = workspace if workspace is not None else globals()["workspace"](need, dev)
    code = lib().dspark_schedule_rule(_ptr(cond_accept), _ptr(max_len), N, K, _ptr(sps),
                                      int(B_max), int(rule), _ptr(sel), _ptr(surv), _ptr(total),
                                      _ptr(obj), _ptr(status), _ptr(ws), ws.numel(),
                                      _stream(stream))
    _check(code, "dspark_schedule_rule")
    return {"sel_len": sel, "survival": surv, "total_rows": total, "objective": obj,
            "status": status}


@_on_its_stream
def dspark_schedule_async(conf_ring, round_, cond_prior, max_len, sps, B_max, rule=SV_STOP_FIRST_DROP,
                          want_survival=True, status=None, workspace=None, stream=None):
    """Round `round_` scheduled with the confidences of round `round_` - 2: conf_ring fp32
    [depth >= 3, N, K] (round t's confidence head writes slot t % depth), cond_prior fp32 [N, K] for
    the first two rounds; otherwise as dspark_schedule."""
    _dev(conf_ring, torch.float32), _dev(cond_prior, torch.float32)
    _dev(max_len, torch.int32), _dev(sps, torch.float64)
    depth, N, K = conf_ring.shape
    if tuple(cond_prior.shape) != (N, K):
        raise ValueError("cond_prior must be [N, K] like one ring slot")
    dev = conf_ring.device
    sel = torch.empty(N, dtype=torch.int32, device=dev)
    surv = torch.empty((N, K), dtype=torch.float32, device=dev) if want_survival else None
    total = torch.empty(1, dtype=torch.int32, device=dev)
    obj = torch.empty(1, dtype=torch.float64, device=dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    need = dspark_schedule_workspace_bytes(N, K)
    ws = workspace if workspace is not None else globals()["workspace"](need, dev)
    code = lib().dspark_schedule_async(_ptr(conf_ring), int(depth), int(round_), _ptr(cond_prior),
                                       _ptr(max_len), N, K, _ptr(sps), int(B_max), int(rule),
                                       _ptr(sel), _ptr(surv), _ptr(total), _ptr(obj),
                                       _ptr(status), _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "dspark_schedule_async")
    return {"sel_len": sel, "survival": surv, "total_rows": total, "objective": obj,
            "status": status}


@_on_its_stream
def dspark_acceptance_update(sel_len, accepted_len, trials, accepts, decay=1.0, prior_a=1.0,
                             prior_b=1.0, alpha=None, cond_accept_out=None, status=None,
                             stream=None):
    """One verified round into the per-position acceptance counts (fp64 [K] device tensors,
    updated in place).  Returns {"alpha": fp32 [K], "cond_accept": fp32 [N, K] or None,
    "status"}."""
    _dev(sel_len, torch.int32), _dev(accepted_len, torch.int32)
    _dev(trials, torch.float64), _dev(accepts, torch.float64)
    N = sel_len.numel()
    K = trials.numel()
    if accepts.numel() != K or accepted_len.numel() != N:
        raise ValueError("inconsistent sizes")
    dev = trials.device
    if alpha is None:
        alpha = torch.empty(K, dtype=torch.float32, device=dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    code = lib().dspark_acceptance_update(_ptr(sel_len), _ptr(accepted_len), N, K, float(decay),
                                          float(prior_a), float(prior_b), _ptr(trials),
                                          _ptr(accepts), _ptr(alpha), _ptr(cond_accept_out),
                                          _ptr(status), _stream(stream))
    _check(code, "dspark_acceptance_update")
    return {"alpha": alpha, "cond_accept": cond_accept_out, "status": status}


@_on_its_stream
def dspark_sts_fit(scores, sel_len, accepted_len, iters=30, beta_min=1.0 / 16, beta_max=16.0,
                   nbins=15, status=None, stream=None):
    """Per-position temperatures of the confidence head fitted to verified outcomes (scores fp32
    [N, K], sel_len / accepted_len int32 [N], all on the device).  Returns device tensors T [K],
    nll, ece_raw, ece_fit (fp64 [K]), count (int32 [K]) and status."""
    _dev(scores, torch.float32), _dev(sel_len, torch.int32), _dev(accepted_len, torch.int32)
    N, K = scores.shape
    dev = scores.device
    out = {"T": torch.empty(K, dtype=torch.float32, device=dev),
           "nll": torch.empty(K, dtype=torch.float64, device=dev),
           "ece_raw": torch.empty(K, dtype=torch.float64, device=dev),
           "ece_fit": torch.empty(K, dtype=torch.float64, device=dev),
           "count": torch.empty(K, dtype=torch.int32, device=dev),
           "status": status if status is not None else torch.zeros(1, dtype=torch.int32,
                                                                   device=dev)}
    code = lib().dspark_sts_fit(_ptr(scores), _ptr(sel_len), _ptr(accepted_len), N, K,
                                int(iters), float(beta_min), float(beta_max), int(nbins),
                                _ptr(out["T"]), _ptr(out["nll"]), _ptr(out["ece_raw"]),
                                _ptr(out["ece_fit"]), _ptr(out["count"]), _ptr(out["status"]),
                                _stream(stream))
    _check(code, "dspark_sts_fit")
    return out
