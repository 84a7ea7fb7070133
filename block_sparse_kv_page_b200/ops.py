"""Python binding of libsparse_attn.so: the C-ABI calls under the same names,
taking torch tensors (device memory) and the current torch stream.

Argument marshalling only: every step of the path runs in the CUDA kernels
behind the C ABI.  Errors from the library raise SparseAttnError.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _abi
from ._abi import (SA_BUDGET_RATIO, SA_BUDGET_TOKENS, SA_BUDGET_TOPK, SA_SCORE_CENTROID,
                   SA_SCORE_ENVELOPE, sa_budget, sa_kv_desc, sa_paged_desc)

lib = _abi.load()

RULES = {"envelope": SA_SCORE_ENVELOPE, "centroid": SA_SCORE_CENTROID}


class SparseAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        msg = lib.sparse_attn_status_string(int(status)).decode()
        super().__init__(f"{where}: status {status} ({msg})")


def _check(st: int, where: str) -> None:
    if st != 0:
        raise SparseAttnError(st, where)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _rule(rule) -> int:
    return RULES[rule] if isinstance(rule, str) else int(rule)


class KvCache:
    """A cache view: K, V bf16 [B, Hkv, cap, 128] plus sequence lengths and,
    for variable chunks, the CSR chunk table.  Holds references to the
    tensors so the pointers in `desc` stay valid."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, seq_len: torch.Tensor, *,
                 page_size: int, max_pages: int, chunk_off: torch.Tensor | None = None,
                 n_chunks: torch.Tensor | None = None):
        for name, t in (("k", k), ("v", v)):
            if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous bf16 [B, Hkv, cap, D] tensor")
        if seq_len.dtype != torch.int32:
            raise ValueError("seq_len must be int32")
        if chunk_off is not None and (chunk_off.dtype != torch.int32 or not chunk_off.is_contiguous()):
            raise ValueError("chunk_off must be contiguous int32 [B, max_pages + 1]")
        self.k, self.v, self.seq_len = k, v, seq_len
        self.chunk_off, self.n_chunks = chunk_off, n_chunks
        B, Hkv, cap, D = k.shape
        self.page_size, self.max_pages = int(page_size), int(max_pages)
        self.desc = sa_kv_desc(B, Hkv, D, int(page_size), cap, k.data_ptr(), v.data_ptr(),
                               seq_len.data_ptr(), _ptr(chunk_off), _ptr(n_chunks), int(max_pages))

    @property
    def batch(self) -> int:
        return self.desc.batch

    @property
    def n_kv_heads(self) -> int:
        return self.desc.n_kv_heads

    def meta_buffer(self) -> torch.Tensor:
        return torch.empty((self.batch, self.n_kv_heads, self.max_pages, 512),
                           dtype=torch.uint8, device=self.k.device)


def budget_topk(k: int) -> sa_budget:
    return sa_budget(SA_BUDGET_TOPK, int(k), 0.0, 0, 0, 0, 0)


def budget_ratio(ratio: float, *, topk_val: int = 1, bos: int = 0, eos: int = 1) -> sa_budget:
    return sa_budget(SA_BUDGET_RATIO, 0, float(ratio), int(topk_val), int(bos), int(eos), 0)


def budget_tokens(n: int) -> sa_budget:
    return sa_budget(SA_BUDGET_TOKENS, 0, 0.0, 0, 0, 0, int(n))


def sparse_attn_workspace_size(kv: KvCache, n_q_heads: int, n_q_rows: int, max_sel: int) -> int:
    return int(lib.sparse_attn_workspace_size(C.byref(kv.desc), n_q_heads, n_q_rows, max_sel))


def _ws_call(ws: torch.Tensor, stream, fn, where: str, *args) -> None:
    """A call on a workspace alone, with its device current: on the given
    stream or that device's current one."""
    index = ws.get_device()
    if index < 0 or index == torch._C._cuda_getDevice():
        _check(fn(ws.data_ptr(), *args, _stream(stream)), where)
    else:
        with torch.cuda.device(index):
            _check(fn(ws.data_ptr(), *args, _stream(stream)), where)


def sparse_attn_workspace_init(ws: torch.Tensor, stream=None) -> None:
    _ws_call(ws, stream, lib.sparse_attn_workspace_init, "sparse_attn_workspace_init",
             ws.numel() * ws.element_size())


def make_workspace(kv: KvCache, n_q_heads: int, n_q_rows: int, max_sel: int, stream=None) -> torch.Tensor:
    n = sparse_attn_workspace_size(kv, n_q_heads, n_q_rows, max_sel)
    if n == 0:
        raise SparseAttnError(_abi.SA_ERR_INVALID, "sparse_attn_workspace_size")
    ws = torch.empty(n, dtype=torch.uint8, device=kv.k.device)
    sparse_attn_workspace_init(ws, stream)
    return ws


def sparse_attn_workspace_size_per_head(kv: KvCache, n_q_heads: int, max_sel: int) -> int:
    return int(lib.sparse_attn_workspace_size_per_head(C.byref(kv.desc), int(n_q_heads), int(max_sel)))


def make_workspace_per_head(kv: KvCache, n_q_heads: int, max_sel: int, stream=None) -> torch.Tensor:
    """Workspace for sparse_attn_select_per_head / sparse_attn_decode_per_head /
    sparse_attn_decode_step_per_head."""
    n = sparse_attn_workspace_size_per_head(kv, n_q_heads, max_sel)
    if n == 0:
        raise SparseAttnError(_abi.SA_ERR_INVALID, "sparse_attn_workspace_size_per_head")
    ws = torch.empty(n, dtype=torch.uint8, device=kv.k.device)
    sparse_attn_workspace_init(ws, stream)
    return ws


def sparse_attn_build_meta(kv: KvCache, rule, first_token: int, meta: torch.Tensor, stream=None) -> None:
    _check(lib.sparse_attn_build_meta(C.byref(kv.desc), _rule(rule), int(first_token),
                                      meta.data_ptr(), _stream(stream)), "sparse_attn_build_meta")


def sparse_attn_select(kv: KvCache, meta: torch.Tensor, rule, q: torch.Tensor, budget: sa_budget,
                       max_sel: int, sel_idx: torch.Tensor, sel_count: torch.Tensor,
                       scores_out: torch.Tensor | None, ws: torch.Tensor, stream=None) -> None:
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [B, Hq, 128]")
    _check(lib.sparse_attn_select(C.byref(kv.desc), meta.data_ptr(), _rule(rule), q.data_ptr(),
                                  q.shape[-2], C.byref(budget), int(max_sel), sel_idx.data_ptr(),
                                  sel_count.data_ptr(), _ptr(scores_out), ws.data_ptr(),
                                  ws.numel() * ws.element_size(), _stream(stream)),
           "sparse_attn_select")


def sparse_attn_select_per_head(kv: KvCache, meta: torch.Tensor, rule, q: torch.Tensor, budget: sa_budget,
                                max_sel: int, sel_idx: torch.Tensor, sel_count: torch.Tensor,
                                scores_out: torch.Tensor | None, ws: torch.Tensor, stream=None) -> None:
    """One page set per query head: sel_idx [B, Hq, max_sel], sel_count [B, Hq]."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [B, Hq, 128]")
    _check(lib.sparse_attn_select_per_head(C.byref(kv.desc), meta.data_ptr(), _rule(rule), q.data_ptr(),
                                           q.shape[-2], C.byref(budget), int(max_sel), sel_idx.data_ptr(),
                                           sel_count.data_ptr(), _ptr(scores_out), ws.data_ptr(),
                                           ws.numel() * ws.element_size(), _stream(stream)),
           "sparse_attn_select_per_head")


def sparse_attn_decode_per_head(kv: KvCache, q: torch.Tensor, scale: float, idx: torch.Tensor,
                                count: torch.Tensor, max_sel: int, out: torch.Tensor,
                                lse: torch.Tensor | None, ws: torch.Tensor, stream=None) -> None:
    """Decode where query head h attends its own page list idx[b, h]."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [B, Hq, 128]")
    if out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("out must be contiguous fp32")
    _check(lib.sparse_attn_decode_per_head(C.byref(kv.desc), q.data_ptr(), q.shape[-2], float(scale),
                                           idx.data_ptr(), count.data_ptr(), int(max_sel), out.data_ptr(),
                                           _ptr(lse), ws.data_ptr(), ws.numel() * ws.element_size(),
                                           _stream(stream)),
           "sparse_attn_decode_per_head")


def sparse_attn_decode(kv: KvCache, q: torch.Tensor, n_q_rows: int, q_pos0: int, tile_rows: int,
                       scale: float, idx: torch.Tensor, count: torch.Tensor, max_sel: int,
                       out: torch.Tensor, lse: torch.Tensor | None, ws: torch.Tensor,
                       stream=None) -> None:
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16")
    if out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("out must be contiguous fp32")
    _check(lib.sparse_attn_decode(C.byref(kv.desc), q.data_ptr(), q.shape[-2], int(n_q_rows),
                                  int(q_pos0), int(tile_rows), float(scale), idx.data_ptr(),
                                  count.data_ptr(), int(max_sel), out.data_ptr(), _ptr(lse),
                                  ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)),
           "sparse_attn_decode")


def sparse_attn_decode_step(kv: KvCache, meta: torch.Tensor, rule, q: torch.Tensor, budget: sa_budget,
                            max_sel: int, scale: float, sel_idx: torch.Tensor, sel_count: torch.Tensor,
                            out: torch.Tensor, lse: torch.Tensor | None, ws: torch.Tensor,
                            stream=None) -> None:
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [B, Hq, 128]")
    if out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("out must be contiguous fp32")
    _check(lib.sparse_attn_decode_step(C.byref(kv.desc), meta.data_ptr(), _rule(rule), q.data_ptr(),
                                       q.shape[-2], C.byref(budget), int(max_sel), float(scale),
                                       sel_idx.data_ptr(), sel_count.data_ptr(), out.data_ptr(),
                                       _ptr(lse), ws.data_ptr(), ws.numel() * ws.element_size(),
                                       _stream(stream)),
           "sparse_attn_decode_step")


def sparse_attn_decode_step_wait_test(kv: KvCache, meta: torch.Tensor, rule, q: torch.Tensor,
                                      budget: sa_budget, max_sel: int, scale: float, sel_idx: torch.Tensor,
                                      sel_count: torch.Tensor, out: torch.Tensor, lse: torch.Tensor | None,
                                      held_unit: int, flag_spin_limit: int, ws: torch.Tensor,
                                      stream=None) -> None:
    """The decode step with unit `held_unit`'s selection never published, so
    that its decode items run their bounded wait out (SA_ERR_TIMEOUT in the
    workspace status word).  A test of the error path; outputs unspecified."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [B, Hq, 128]")
    if out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("out must be contiguous fp32")
    _check(lib.sparse_attn_decode_step_wait_test(C.byref(kv.desc), meta.data_ptr(), _rule(rule), q.data_ptr(),
                                                 q.shape[-2], C.byref(budget), int(max_sel), float(scale),
                                                 sel_idx.data_ptr(), sel_count.data_ptr(), out.data_ptr(),
                                                 _ptr(lse), int(held_unit), int(flag_spin_limit),
                                                 ws.data_ptr(), ws.numel() * ws.element_size(),
                                                 _stream(stream)),
           "sparse_attn_decode_step_wait_test")


def sparse_attn_decode_step_per_head(kv: KvCache, meta: torch.Tensor, rule, q: torch.Tensor,
                                     budget: sa_budget, max_sel: int, scale: float, sel_idx: torch.Tensor,
                                     sel_count: torch.Tensor, out: torch.Tensor, lse: torch.Tensor | None,
                                     ws: torch.Tensor, stream=None) -> None:
    """The decode step with one page set per query head: sel_idx [B, Hq, max_sel],
    sel_count [B, Hq]; ws from make_workspace_per_head."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [B, Hq, 128]")
    if out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("out must be contiguous fp32")
    _check(lib.sparse_attn_decode_step_per_head(C.byref(kv.desc), meta.data_ptr(), _rule(rule), q.data_ptr(),
                                                q.shape[-2], C.byref(budget), int(max_sel), float(scale),
                                                sel_idx.data_ptr(), sel_count.data_ptr(), out.data_ptr(),
                                                _ptr(lse), ws.data_ptr(), ws.numel() * ws.element_size(),
                                                _stream(stream)),
           "sparse_attn_decode_step_per_head")


def sparse_attn_decode_step_append(kv: KvCache, meta: torch.Tensor, rule, q: torch.Tensor,
                                   k_new: torch.Tensor, v_new: torch.Tensor, budget: sa_budget,
                                   max_sel: int, scale: float, sel_idx: torch.Tensor,
                                   sel_count: torch.Tensor, out: torch.Tensor, lse: torch.Tensor | None,
                                   ws: torch.Tensor, stream=None) -> None:
    """The decode step with the newest token's key and value (bf16 [B, Hkv, 128])
    stored into the cache at row seq_len - 1 inside the same launch.  out is
    fp32 or bf16 [B, Hq, 128] (bf16: the fp32 result rounded to nearest even)."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [B, Hq, 128]")
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or tuple(t.shape) != (kv.batch, kv.k.shape[1], 128):
            raise ValueError(f"{name} must be contiguous bf16 [B, Hkv, 128]")
    if out.dtype not in (torch.float32, torch.bfloat16) or not out.is_contiguous():
        raise ValueError("out must be contiguous fp32 or bf16")
    out_dtype = _abi.SA_OUT_BF16 if out.dtype == torch.bfloat16 else _abi.SA_OUT_F32
    _check(lib.sparse_attn_decode_step_append(C.byref(kv.desc), meta.data_ptr(), _rule(rule), q.data_ptr(),
                                              q.shape[-2], k_new.data_ptr(), v_new.data_ptr(),
                                              C.byref(budget), int(max_sel), float(scale),
                                              sel_idx.data_ptr(), sel_count.data_ptr(), out.data_ptr(),
                                              out_dtype, _ptr(lse), ws.data_ptr(),
                                              ws.numel() * ws.element_size(), _stream(stream)),
           "sparse_attn_decode_step_append")


def sparse_attn_decode_static(kv: KvCache, q: torch.Tensor, n_q_rows: int, q_pos0: int,
                              tile_rows: int, scale: float, idx: torch.Tensor, count: torch.Tensor,
                              max_sel: int, out: torch.Tensor, lse: torch.Tensor | None,
                              device_status: torch.Tensor | None = None, stream=None) -> None:
    """sparse_attn_decode without a workspace, for callers that cannot
    allocate device memory where they run it: the scratch is an 8 MiB array
    inside the library, shared by every call, so calls must not overlap on
    the GPU.  One-row decode only (tile_rows == 1).  device_status: optional
    zeroed int32 device tensor that receives the first device-side error
    code; without it, device-side errors of the call are not reported."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16")
    if out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("out must be contiguous fp32")
    _check(lib.sparse_attn_decode_static(C.byref(kv.desc), q.data_ptr(), q.shape[-2], int(n_q_rows),
                                         int(q_pos0), int(tile_rows), float(scale), idx.data_ptr(),
                                         count.data_ptr(), int(max_sel), out.data_ptr(), _ptr(lse),
                                         _ptr(device_status), _stream(stream)),
           "sparse_attn_decode_static")


def sparse_attn_route_decode(kv: KvCache, meta: torch.Tensor, rule, q: torch.Tensor, k: int, rho: int,
                             quantile: float, tau: torch.Tensor | None, kv_idx: torch.Tensor,
                             kv_count: torch.Tensor, sigma: torch.Tensor, sigma_bar: torch.Tensor,
                             triggered: torch.Tensor, tau_out: torch.Tensor | None, ws: torch.Tensor,
                             stream=None) -> None:
    """The router with one-row tiles: every sequence's decode query is a tile.
    kv_idx [B, Hkv, rho*k] rank-ordered, -1 padded; kv_count [B, Hkv];
    sigma [B, Hkv]; sigma_bar [B]; triggered [B] uint8."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [B, Hq, 128]")
    _check(lib.sparse_attn_route_decode(C.byref(kv.desc), meta.data_ptr(), _rule(rule), q.data_ptr(),
                                        q.shape[-2], int(k), int(rho), float(quantile), _ptr(tau),
                                        kv_idx.data_ptr(), kv_count.data_ptr(), sigma.data_ptr(),
                                        sigma_bar.data_ptr(), triggered.data_ptr(), _ptr(tau_out),
                                        ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)),
           "sparse_attn_route_decode")


def sparse_attn_route_decode_step(kv: KvCache, meta: torch.Tensor, rule, q: torch.Tensor, k: int, rho: int,
                                  quantile: float, tau: torch.Tensor | None, scale: float, kv_idx: torch.Tensor,
                                  kv_count: torch.Tensor, sigma: torch.Tensor, sigma_bar: torch.Tensor,
                                  triggered: torch.Tensor, tau_out: torch.Tensor | None, out: torch.Tensor,
                                  lse: torch.Tensor | None, ws: torch.Tensor, stream=None) -> None:
    """The router on the decode batch and the decode over its lists in one
    launch (newest-page metadata refresh included): the outputs of
    sparse_attn_route_decode plus out [B, Hq, 128] fp32 and lse [B, Hq]."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [B, Hq, 128]")
    if out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("out must be contiguous fp32")
    _check(lib.sparse_attn_route_decode_step(C.byref(kv.desc), meta.data_ptr(), _rule(rule), q.data_ptr(),
                                             q.shape[-2], int(k), int(rho), float(quantile), _ptr(tau),
                                             float(scale), kv_idx.data_ptr(), kv_count.data_ptr(),
                                             sigma.data_ptr(), sigma_bar.data_ptr(), triggered.data_ptr(),
                                             _ptr(tau_out), out.data_ptr(), _ptr(lse), ws.data_ptr(),
                                             ws.numel() * ws.element_size(), _stream(stream)),
           "sparse_attn_route_decode_step")


def sparse_attn_route(kv: KvCache, meta: torch.Tensor, rule, q: torch.Tensor, n_q_rows: int,
                      q_pos0: int, tile_rows: int, k: int, rho: int, quantile: float,
                      tau: torch.Tensor | None, kv_idx: torch.Tensor, kv_count: torch.Tensor,
                      sigma: torch.Tensor, sigma_bar: torch.Tensor, triggered: torch.Tensor,
                      tau_out: torch.Tensor | None, ws: torch.Tensor, stream=None) -> None:
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [rows, Hq, 128]")
    _check(lib.sparse_attn_route(C.byref(kv.desc), meta.data_ptr(), _rule(rule), q.data_ptr(),
                                 q.shape[-2], int(n_q_rows), int(q_pos0), int(tile_rows), int(k),
                                 int(rho), float(quantile), _ptr(tau), kv_idx.data_ptr(),
                                 kv_count.data_ptr(), sigma.data_ptr(), sigma_bar.data_ptr(),
                                 triggered.data_ptr(), _ptr(tau_out), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), _stream(stream)),
           "sparse_attn_route")


def sparse_attn_get_device_status(ws: torch.Tensor, stream=None) -> int:
    out = C.c_int(0)
    _ws_call(ws, stream, lib.sparse_attn_get_device_status, "sparse_attn_get_device_status", C.byref(out))
    return int(out.value)


def sparse_attn_status_string(code: int) -> str:
    return lib.sparse_attn_status_string(int(code)).decode()


class PagedCache:
    """A cache held in pages: k, v [n_pages, Hkv, page_size, 128], bf16 or
    float8_e4m3fn, of the same strides (the last one 1), so token-major pages
    ([n_pages, page_size, Hkv, 128].transpose(1, 2)) fit; page_table int32
    [B, max_pages]; seq_len int32 [B], the tokens of each sequence with the
    new ones of a call.  float8_e4m3fn: k_scale, v_scale uint8 [n_pages, Hkv,
    page_size], a value being code * 2^(scale - 127).  Holds references to the
    tensors so the pointers in `desc` stay valid."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, seq_len: torch.Tensor, *,
                 k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be [n_pages, Hkv, page_size, D] tensors of one shape and type")
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError("k and v must be bf16 or float8_e4m3fn")
        n_pages, Hkv, page_size, D = k.shape
        if 0 in k.shape:
            raise ValueError("k and v must not be empty")

        def strides(t):  # the stride of an axis of one element says nothing: take one that fits
            s = list(t.stride())
            if D > 1 and s[3] != 1:
                raise ValueError("k and v must have contiguous rows (last stride 1)")
            if page_size == 1:
                s[2] = D
            if Hkv == 1:
                s[1] = page_size * s[2]
            if n_pages == 1:
                s[0] = max(Hkv * s[1], page_size * s[2])
            return s[:3]
        page_stride, head_stride, token_stride = strides(k)
        if strides(v) != strides(k):
            raise ValueError("k and v must have the same strides")
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_contiguous():
            raise ValueError("page_table must be contiguous int32 [B, max_pages]")
        B, max_pages = page_table.shape
        if seq_len.dtype != torch.int32 or tuple(seq_len.shape) != (B,) or not seq_len.is_contiguous():
            raise ValueError("seq_len must be contiguous int32 [B]")
        e4m3 = k.dtype == torch.float8_e4m3fn
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if e4m3 != (t is not None):
                raise ValueError(f"{name} is needed with a float8_e4m3fn cache, and only with it")
            if e4m3 and (t.dtype != torch.uint8 or tuple(t.shape) != (n_pages, Hkv, page_size)
                         or not t.is_contiguous()):
                raise ValueError(f"{name} must be contiguous uint8 [n_pages, Hkv, page_size]")
        self.device, self.index = k.device, k.get_device()
        for t in (v, page_table, seq_len, k_scale, v_scale):
            if t is not None and t.device != self.device:
                raise ValueError("the tensors of a cache must be on one device")
        self.k, self.v, self.page_table, self.seq_len = k, v, page_table, seq_len
        self.k_scale, self.v_scale = k_scale, v_scale
        self.n_kv_heads, self.page_size, self.batch = Hkv, page_size, B
        self.desc = sa_paged_desc(B, Hkv, D, page_size, n_pages, _abi.SA_KV_E4M3 if e4m3 else _abi.SA_KV_BF16,
                                  max_pages, k.data_ptr(), v.data_ptr(), page_stride, head_stride, token_stride,
                                  _ptr(k_scale), _ptr(v_scale), page_table.data_ptr(), seq_len.data_ptr())
        self.ref = C.byref(self.desc)


def _on(kv: PagedCache, stream, *tensors) -> int:
    """The stream of a call on the cache's device: the given one, or that
    device's current one.  All tensors of a call are on that device, which is
    a GPU (a cache in host memory can be described and sized only)."""
    index = kv.index
    if index < 0:
        raise ValueError("the tensors of a call must be on a CUDA device")
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError("the tensors of a call must be on the cache's device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return _stream(stream)


def _paged_call(kv: PagedCache, fn, where: str, *args) -> None:
    """Run a call with the cache's device current."""
    if kv.index == torch._C._cuda_getDevice():
        st = fn(*args)
    else:
        with torch.cuda.device(kv.index):
            st = fn(*args)
    if st != 0:
        raise SparseAttnError(st, where)


def _rows(t: torch.Tensor, name: str, heads: int | None = None) -> int:
    """The row stride (elements) of a packed bf16 [rows, heads, 128] array
    whose heads lie one after another, so parts of a projection's rows fit."""
    shape = t.shape
    if t.dtype is not torch.bfloat16 or len(shape) != 3 or shape[2] != 128 or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be a bf16 [rows, heads, 128] tensor of the call's heads")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != 128 and shape[1] > 1):
        raise ValueError(f"{name} must have its heads one after another in a row")
    return s0 if shape[0] > 1 else shape[1] * 128


def _row_off(row_off: torch.Tensor, kv: PagedCache) -> None:
    if row_off.dtype is not torch.int32 or row_off.shape != (kv.batch + 1,) or not row_off.is_contiguous():
        raise ValueError("row_off must be contiguous int32 [B + 1]")


def _int32(x) -> int:
    x = int(x)
    if not -(1 << 31) <= x < 1 << 31:  # (ctypes keeps the low bits of others)
        raise ValueError("first_token, window and sinks must fit 32 bits")
    return x


def _ws(ws: torch.Tensor | None) -> tuple[int | None, int]:
    return (None, 0) if ws is None else (ws.data_ptr(), ws.nbytes)


def sparse_attn_paged_workspace_size(kv: PagedCache, n_q_heads: int) -> int:
    """Bytes for the cache's device (they go by its number of SMs)."""
    if kv.index < 0 or kv.index == torch._C._cuda_getDevice():
        return int(lib.sparse_attn_paged_workspace_size(kv.ref, int(n_q_heads)))
    with torch.cuda.device(kv.index):
        return int(lib.sparse_attn_paged_workspace_size(kv.ref, int(n_q_heads)))


def make_paged_workspace(kv: PagedCache, n_q_heads: int, stream=None) -> torch.Tensor:
    """Workspace of the paged-cache calls; calls that may overlap on the GPU
    (other streams, other captured graphs) need one each."""
    n = sparse_attn_paged_workspace_size(kv, n_q_heads)
    if n == 0:
        raise SparseAttnError(_abi.SA_ERR_INVALID, "sparse_attn_paged_workspace_size")
    s = _on(kv, stream)
    ws = torch.empty(n, dtype=torch.uint8, device=kv.device)
    _paged_call(kv, lib.sparse_attn_workspace_init, "sparse_attn_workspace_init", ws.data_ptr(), n, s)
    return ws


def sparse_attn_cache_write(kv: PagedCache, k_new: torch.Tensor, v_new: torch.Tensor, row_off: torch.Tensor,
                            ws: torch.Tensor | None = None, stream=None) -> None:
    """Store the new rows (bf16 [rows, Hkv, 128], rows row_off[b] ..
    row_off[b + 1] - 1 being the last tokens of sequence b) in the cache,
    quantised if it holds e4m3.  ws: takes the status word; may be None."""
    Hkv = kv.n_kv_heads
    stride = _rows(k_new, "k_new", Hkv)
    rows = k_new.shape[0]
    if v_new.shape[0] != rows or _rows(v_new, "v_new", Hkv) != stride:
        raise ValueError("k_new and v_new must have the same rows and strides")
    _row_off(row_off, kv)
    s = _on(kv, stream, k_new, v_new, row_off, ws)
    if rows == 0:
        return
    _paged_call(kv, lib.sparse_attn_cache_write, "sparse_attn_cache_write", kv.ref, k_new.data_ptr(),
                v_new.data_ptr(), stride, row_off.data_ptr(), rows, *_ws(ws), s)


def sparse_attn_cache_read(kv: PagedCache, first_token: int, k_out: torch.Tensor, v_out: torch.Tensor,
                           ws: torch.Tensor | None = None, stream=None) -> None:
    """Read tokens back into a contiguous bf16 cache [B, Hkv, cap, 128] (the k
    and v of a KvCache): tokens first_token .. seq_len - 1 of every sequence,
    or its last -first_token ones.  Other rows are left as they are."""
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous() or t.shape != k_out.shape \
                or t.shape[0] != kv.batch or t.shape[1] != kv.n_kv_heads or t.shape[3] != 128:
            raise ValueError(f"{name} must be a contiguous bf16 [B, Hkv, cap, 128] tensor")
    first_token = _int32(first_token)
    s = _on(kv, stream, k_out, v_out, ws)
    _paged_call(kv, lib.sparse_attn_cache_read, "sparse_attn_cache_read", kv.ref, first_token,
                k_out.data_ptr(), v_out.data_ptr(), k_out.shape[2], *_ws(ws), s)


def _attn_out(rows: int, heads: int, out: torch.Tensor, lse: torch.Tensor | None) -> int:
    dtype = out.dtype
    if out.shape != (rows, heads, 128) or not out.is_contiguous() or dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out must be contiguous fp32 or bf16 [rows, Hq, 128]")
    if lse is not None and (lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.shape != (rows, heads)):
        raise ValueError("lse must be contiguous fp32 [rows, Hq]")
    return _abi.SA_OUT_BF16 if dtype is torch.bfloat16 else _abi.SA_OUT_F32


def sparse_attn_chunk(kv: PagedCache, q: torch.Tensor, row_off: torch.Tensor, scale: float, window: int, sinks: int,
                      out: torch.Tensor, lse: torch.Tensor | None, ws: torch.Tensor, stream=None) -> None:
    """Causal attention of the new rows q (bf16 [rows, Hq, 128]; rows
    row_off[b] .. row_off[b + 1] - 1 are the last tokens of sequence b, whose
    keys and values the cache already holds) over the cache.  window > 0: a row
    sees its last `window` tokens, itself included, and the first `sinks`."""
    stride = _rows(q, "q")
    rows, heads, _ = q.shape
    out_dtype = _attn_out(rows, heads, out, lse)
    _row_off(row_off, kv)
    window, sinks = _int32(window), _int32(sinks)
    s = _on(kv, stream, q, row_off, out, lse, ws)
    if rows == 0:
        return
    _paged_call(kv, lib.sparse_attn_chunk, "sparse_attn_chunk", kv.ref, q.data_ptr(), stride, heads,
                row_off.data_ptr(), rows, window, sinks, float(scale), out.data_ptr(), out_dtype,
                _ptr(lse), *_ws(ws), s)


def sparse_attn_paged_decode(kv: PagedCache, q: torch.Tensor, scale: float, window: int, sinks: int,
                             out: torch.Tensor, lse: torch.Tensor | None, ws: torch.Tensor, stream=None) -> None:
    """One row per sequence: q bf16 [B, Hq, 128], row b the newest token of
    sequence b; otherwise as sparse_attn_chunk."""
    stride = _rows(q, "q")
    rows, heads, _ = q.shape
    if rows != kv.batch:
        raise ValueError("q must have one row per sequence")
    out_dtype = _attn_out(rows, heads, out, lse)
    window, sinks = _int32(window), _int32(sinks)
    s = _on(kv, stream, q, out, lse, ws)
    _paged_call(kv, lib.sparse_attn_paged_decode, "sparse_attn_paged_decode", kv.ref, q.data_ptr(), stride,
                heads, window, sinks, float(scale), out.data_ptr(), out_dtype, _ptr(lse), *_ws(ws), s)
