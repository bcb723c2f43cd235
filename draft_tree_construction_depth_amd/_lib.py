"""ctypes binding of libddtree.so (C ABI in include/ddtree.h).

Argument marshalling only: every function below passes torch tensors' device
pointers and the current HIP stream to the function of the same name in the
library; all computation happens in the library's HIP kernels. There is no
fallback: if the library is missing, loading it raises.
"""

from __future__ import annotations

import ctypes as C
import functools
import os
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libddtree.so")

DDT_OK, DDT_EINVAL, DDT_ENOTSUP, DDT_EWORKSPACE, DDT_EHIP = 0, -1, -2, -3, -4
DDT_BF16, DDT_F32, DDT_F16 = 0, 1, 2

_lib = None


class DDTreeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


def lib() -> C.CDLL:
    """Load libddtree.so from the package directory (raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"HIP library not built: {LIB_PATH} is missing; run __graft_entry__.build()")
        L = C.CDLL(LIB_PATH)
        p, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
        L.ddt_abi_version.restype = C.c_int
        L.ddt_status_string.restype = C.c_char_p
        L.ddt_status_string.argtypes = [C.c_int]
        L.ddtree_build_workspace_size.restype = sz
        L.ddtree_build_workspace_size.argtypes = [i64, i32, i64, i32, C.c_int]
        L.ddtree_row_topk_workspace_size.restype = sz
        L.ddtree_row_topk_workspace_size.argtypes = [i64, i64, i32, C.c_int]
        L.ddtree_build.restype = C.c_int
        L.ddtree_build.argtypes = [p, C.c_int, i64, i32, i64, i32, p, p, p, p, p, p, p, sz, p]
        L.ddtree_build_noalloc.restype = C.c_int
        L.ddtree_build_noalloc.argtypes = [p, C.c_int, i64, i32, i64, i32, p, p, p, p, p, p, p]
        L.ddtree_select.restype = C.c_int
        L.ddtree_select.argtypes = [p, p, p, i64, i32, i32, i32, p, p, p, p, p, p, p]
        L.ddtree_mask.restype = C.c_int
        L.ddtree_mask.argtypes = [p, p, i64, i32, p, p]
        L.ddtree_accept.restype = C.c_int
        L.ddtree_accept.argtypes = [p, p, p, p, i64, i32, i32, p, p, p, p]
        L.ddtree_compact_kv.restype = C.c_int
        L.ddtree_compact_kv.argtypes = [p, p, i64, i64, i32, i64, i32, p, p, p, i32, p, p]
        L.ddtree_read_probe.restype = C.c_int
        L.ddtree_read_probe.argtypes = [p, i64, i64, p, p]
        L.ddtree_ts_load_probe.restype = C.c_int
        L.ddtree_ts_load_probe.argtypes = [p, p, p, i64, i32, i32, p, p]
        L.ddtree_row_topk.restype = C.c_int
        L.ddtree_row_topk.argtypes = [p, C.c_int, i64, i64, i32, p, p, p, p, sz, p]
        L.treespark_workspace_size.restype = sz
        L.treespark_workspace_size.argtypes = [i64, i32, i64, i32, i32, i32, i32]
        L.treespark_expand.restype = C.c_int
        L.treespark_expand.argtypes = [p, p, p, p, i64, i32, i64, i32, i32, i32, i32, p, p, p, p,
                                       p, p, sz, p]
        L.sparkling_build_workspace_size.restype = sz
        L.sparkling_build_workspace_size.argtypes = [i64, i32, i64, i32, i32, i32, C.c_int]
        L.sparkling_build.restype = C.c_int
        L.sparkling_build.argtypes = [p, C.c_int, p, p, i64, i32, i64, i32, i32, i32, p, p, p, p,
                                      p, p, p, sz, p]
        L.dspark_budget.restype = C.c_int
        L.dspark_budget.argtypes = [p, i64, i32, p, i32, p, p, p, p, p, p]
        L.sparkling_beam.restype = C.c_int
        L.sparkling_beam.argtypes = [p, C.c_int, p, p, i64, i32, i64, i32, i32, p, i32, p, p, p,
                                     p, p, p, p, sz, p]
        L.ddtree_append_kv.restype = C.c_int
        L.ddtree_append_kv.argtypes = [p, p, p, C.c_int, i64, i32, i32, i32, i32, i64, i64, i64, p,
                                       i64, i32, i32, p, p, p, p, i64, i64, i32, p, p, p, p]
        L.ddtree_attention_workspace_size.restype = sz
        L.ddtree_attention_workspace_size.argtypes = [i64, i32, i32, i32, i32, i64, i32]
        L.ddtree_attention.restype = C.c_int
        L.ddtree_attention.argtypes = [p, C.c_int, i64, i32, i32, i32, i32, p, p, p, i64, i64, i32,
                                       p, p, p, C.c_float, p, p, p, sz, p]
        L.ddtree_compact_kv_paged.restype = C.c_int
        L.ddtree_compact_kv_paged.argtypes = [p, p, i64, i64, i32, i32, i32, p, i64, i64, p, p, p,
                                              i32, p, p]
        L.ddtree_accept_sampled_workspace_size.restype = sz
        L.ddtree_accept_sampled_workspace_size.argtypes = [i64, i32, i32, i64, C.c_int]
        L.ddtree_accept_sampled.restype = C.c_int
        L.ddtree_accept_sampled.argtypes = [p, p, p, p, C.c_int, p, p, i64, i32, i32, i64, p, p, p,
                                            p, p, sz, p]
        L.dspark_accept_sampled_workspace_size.restype = sz
        L.dspark_accept_sampled_workspace_size.argtypes = [i64, i32, i64, C.c_int]
        L.dspark_accept_sampled.restype = C.c_int
        L.dspark_accept_sampled.argtypes = [p, p, p, p, C.c_int, p, p, i64, i32, i64, p, p, p, p,
                                            sz, p]
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().ddt_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _arg(t, name, dtypes, shape=None):
    """Check that a tensor argument is a contiguous device tensor of the
    expected dtype (and shape); the library reads raw row-major memory."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


_I32 = (torch.int32,)
_LOGITS = (torch.bfloat16, torch.float32)


def _stream(device):
    return C.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DDT_BF16
    if t.dtype == torch.float32:
        return DDT_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _check(fn, rc):
    if rc != DDT_OK:
        raise DDTreeError(fn, rc)


class _Workspaces(threading.local):
    """The calling thread's own workspaces. A call into the library releases the interpreter
    lock and enqueues several launches, so two threads' launches on one stream (the default one
    is every thread's) may lie between one another's: they must not share a workspace. A
    thread's buffers go with it; the allocator keeps their next use behind the stream's work."""

    def __init__(self):
        self.held: dict = {}

    def get(self, key):
        return self.held.get(key)

    def __setitem__(self, key, ws):
        self.held[key] = ws

    def __iter__(self):
        return iter(self.held)


_workspaces = _Workspaces()


def workspace(kind: str, size: int, device, key) -> torch.Tensor:
    """Scratch buffer cached per thread and (kind, device, stream, shape key).

    The library ignores a workspace's contents on entry, so one buffer per
    shape is reused across calls; calls on different streams may overlap and
    those of different threads interleave, and so get buffers of their own.
    """
    k = (kind, str(device), torch.cuda.current_stream(device).cuda_stream, key)
    ws = _workspaces.get(k)
    if ws is None or ws.numel() < size:
        ws = torch.empty(max(size, 1), dtype=torch.uint8, device=device)
        _workspaces[k] = ws
    return ws


def ddtree_build(logits: torch.Tensor, B: int, *, with_mask: bool = True, out: dict | None = None,
                 ws: torch.Tensor | None = None) -> dict:
    """Stages 1-2 (+3): logits [batch, L, V] (bf16/f32, cuda) -> tree tensors."""
    _arg(logits, "logits", _LOGITS)
    if logits.dim() != 3:
        raise ValueError("logits must be [batch, L, V]")
    batch, L, V = logits.shape
    dev = logits.device
    dt = _dtype_code(logits)
    if out is None:
        out = _tree_out(batch, B, dev, with_mask)
    size = lib().ddtree_build_workspace_size(batch, L, V, B, dt)
    if ws is None:
        ws = workspace("build", size, dev, (batch, L, V, B, dt))
    rc = lib().ddtree_build(_ptr(logits), dt, batch, L, V, B, _ptr(out["tree_tokens"]),
                            _ptr(out["parents"]), _ptr(out["logq"]), _ptr(out.get("depths")),
                            _ptr(out["num_nodes"]), _ptr(out.get("mask")), _ptr(ws),
                            ws.numel(), _stream(dev))
    _check("ddtree_build", rc)
    return out


def ddtree_build_noalloc(logits: torch.Tensor, B: int, *, with_mask: bool = True,
                         out: dict | None = None) -> dict:
    """ddtree_build on the library's static scratch (no workspace; the call
    allocates nothing on the device when out is given)."""
    _arg(logits, "logits", _LOGITS)
    if logits.dim() != 3:
        raise ValueError("logits must be [batch, L, V]")
    batch, L, V = logits.shape
    dev = logits.device
    dt = _dtype_code(logits)
    if out is None:
        out = _tree_out(batch, B, dev, with_mask)
    rc = lib().ddtree_build_noalloc(_ptr(logits), dt, batch, L, V, B, _ptr(out["tree_tokens"]),
                                    _ptr(out["parents"]), _ptr(out["logq"]),
                                    _ptr(out.get("depths")), _ptr(out["num_nodes"]),
                                    _ptr(out.get("mask")), _stream(dev))
    _check("ddtree_build_noalloc", rc)
    return out


def _tree_out(batch, B, dev, with_mask):
    out = dict(
        tree_tokens=torch.empty((batch, B), dtype=torch.int32, device=dev),
        parents=torch.empty((batch, B), dtype=torch.int32, device=dev),
        logq=torch.empty((batch, B), dtype=torch.float32, device=dev),
        depths=torch.empty((batch, B), dtype=torch.int32, device=dev),
        num_nodes=torch.empty((batch,), dtype=torch.int32, device=dev),
    )
    if with_mask:
        out["mask"] = torch.empty((batch, B + 1, (B + 1 + 63) // 64), dtype=torch.int64, device=dev)
    return out


def ddtree_select(vals: torch.Tensor, ids: torch.Tensor, lse: torch.Tensor, B: int, *,
                  with_mask: bool = True, out: dict | None = None) -> dict:
    """Stage 2 (+3) from tables vals/ids [batch, L, K] and lse [batch, L]."""
    _arg(vals, "vals", (torch.float32,))
    batch, L, K = vals.shape
    _arg(ids, "ids", _I32, (batch, L, K))
    _arg(lse, "lse", (torch.float64,), (batch, L))
    if out is None:
        out = _tree_out(batch, B, vals.device, with_mask)
    rc = lib().ddtree_select(_ptr(vals), _ptr(ids), _ptr(lse), batch, L, K, B,
                             _ptr(out["tree_tokens"]), _ptr(out["parents"]), _ptr(out["logq"]),
                             _ptr(out.get("depths")), _ptr(out["num_nodes"]), _ptr(out.get("mask")),
                             _stream(vals.device))
    _check("ddtree_select", rc)
    return out


def ddtree_mask(parents: torch.Tensor, num_nodes: torch.Tensor, B: int,
                mask: torch.Tensor | None = None) -> torch.Tensor:
    _arg(num_nodes, "num_nodes", _I32)
    batch = num_nodes.shape[0]
    _arg(parents, "parents", _I32, (batch, B))
    W = (B + 1 + 63) // 64
    if mask is None:
        mask = torch.empty((batch, B + 1, W), dtype=torch.int64, device=parents.device)
    rc = lib().ddtree_mask(_ptr(parents), _ptr(num_nodes), batch, B, _ptr(mask),
                           _stream(parents.device))
    _check("ddtree_mask", rc)
    return mask


def ddtree_accept(tree_tokens: torch.Tensor, parents: torch.Tensor, num_nodes: torch.Tensor,
                  target_tokens: torch.Tensor, L: int, out: dict | None = None) -> dict:
    _arg(tree_tokens, "tree_tokens", _I32)
    batch, B = tree_tokens.shape
    _arg(parents, "parents", _I32, (batch, B))
    _arg(num_nodes, "num_nodes", _I32, (batch,))
    _arg(target_tokens, "target_tokens", _I32, (batch, B + 1))
    dev = tree_tokens.device
    if out is None:
        out = dict(accepted_nodes=torch.empty((batch, L), dtype=torch.int32, device=dev),
                   accept_len=torch.empty((batch,), dtype=torch.int32, device=dev),
                   next_token=torch.empty((batch,), dtype=torch.int32, device=dev))
    rc = lib().ddtree_accept(_ptr(tree_tokens), _ptr(parents), _ptr(num_nodes),
                             _ptr(target_tokens), batch, B, L, _ptr(out["accepted_nodes"]),
                             _ptr(out["accept_len"]), _ptr(out["next_token"]), _stream(dev))
    _check("ddtree_accept", rc)
    return out


def ddtree_compact_kv(k_cache: torch.Tensor, v_cache: torch.Tensor, past_len: torch.Tensor,
                      accepted_nodes: torch.Tensor, accept_len: torch.Tensor,
                      new_len: torch.Tensor | None = None) -> torch.Tensor:
    """In place: caches [layers, batch, heads, cap, head_dim] keep the accepted path's
    rows (slots past_len+1 .. past_len+accept_len); returns new_len [batch]."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 5:
        raise ValueError("k_cache must be a 5-d tensor [layers, batch, heads, cap, head_dim]")
    _arg(k_cache, "k_cache", (k_cache.dtype,))
    _arg(v_cache, "v_cache", (k_cache.dtype,), tuple(k_cache.shape))
    layers, batch, heads, cap, dh = k_cache.shape
    _arg(past_len, "past_len", _I32, (batch,))
    _arg(accepted_nodes, "accepted_nodes", _I32)
    L = accepted_nodes.shape[-1]
    _arg(accepted_nodes, "accepted_nodes", _I32, (batch, L))
    _arg(accept_len, "accept_len", _I32, (batch,))
    dev = k_cache.device
    if new_len is None:
        new_len = torch.empty((batch,), dtype=torch.int32, device=dev)
    rc = lib().ddtree_compact_kv(_ptr(k_cache), _ptr(v_cache), layers, batch, heads, cap,
                                 dh * k_cache.element_size(), _ptr(past_len),
                                 _ptr(accepted_nodes), _ptr(accept_len), L, _ptr(new_len),
                                 _stream(dev))
    _check("ddtree_compact_kv", rc)
    return new_len


def ddtree_row_topk(logits: torch.Tensor, K: int, *, out: dict | None = None,
                    ws: torch.Tensor | None = None) -> dict:
    """Stage 1 alone: logits [..., V] -> ids/vals [rows, K], lse [rows] (float64)."""
    _arg(logits, "logits", _LOGITS)
    V = logits.shape[-1]
    rows = logits.numel() // V
    dev = logits.device
    dt = _dtype_code(logits)
    if out is None:
        out = dict(ids=torch.empty((rows, K), dtype=torch.int32, device=dev),
                   vals=torch.empty((rows, K), dtype=torch.float32, device=dev),
                   lse=torch.empty((rows,), dtype=torch.float64, device=dev))
    size = lib().ddtree_row_topk_workspace_size(rows, V, K, dt)
    if ws is None:
        ws = workspace("row_topk", size, dev, (rows, V, K, dt))
    rc = lib().ddtree_row_topk(_ptr(logits), dt, rows, V, K, _ptr(out["ids"]), _ptr(out["vals"]),
                               _ptr(out["lse"]), _ptr(ws), ws.numel(), _stream(dev))
    _check("ddtree_row_topk", rc)
    return out


_BF16 = (torch.bfloat16,)


def ddtree_read_probe(src: torch.Tensor, rows: int, row_bytes: int,
                      sink: torch.Tensor | None = None) -> torch.Tensor:
    """Measurement probe: stream rows x row_bytes bytes of src (stage 1's
    launch geometry, no compute); returns the XOR sink [rows, 4] (uint32 as int32)."""
    if not isinstance(src, torch.Tensor) or not src.is_cuda or not src.is_contiguous():
        raise ValueError("src must be a contiguous device tensor")
    if rows * row_bytes > src.numel() * src.element_size():
        raise ValueError("rows x row_bytes exceeds src")
    if sink is None:
        sink = torch.empty((rows, 4), dtype=torch.int32, device=src.device)
    _check("ddtree_read_probe", lib().ddtree_read_probe(_ptr(src), rows, row_bytes, _ptr(sink),
                                                        _stream(src.device)))
    return sink


def ddtree_ts_load_probe(W: torch.Tensor, E: torch.Tensor, ptok: torch.Tensor, variant: int,
                         sink: torch.Tensor | None = None) -> torch.Tensor:
    """Measurement probe: one TreeSpark head evaluation's loads (W [V, H] and
    the 128 parents' rows ptok of E [V, H], bf16) with nothing computed;
    variant 0-4 as in the header. Returns the sink [256] (int32)."""
    _arg(W, "W", _BF16)
    V, H = W.shape
    _arg(E, "E", _BF16, (V, H))
    _arg(ptok, "ptok", _I32, (128,))
    if sink is None:
        sink = torch.empty(256, dtype=torch.int32, device=W.device)
    _check("ddtree_ts_load_probe", lib().ddtree_ts_load_probe(_ptr(W), _ptr(E), _ptr(ptok), V, H,
                                                              variant, _ptr(sink),
                                                              _stream(W.device)))
    return sink


def treespark_expand(backbone: torch.Tensor, W: torch.Tensor, E: torch.Tensor,
                     anchor: torch.Tensor, *, k: int = 4, F: int = 4, N: int = 32,
                     out: dict | None = None, ws: torch.Tensor | None = None) -> dict:
    """TreeSpark expansion: backbone [batch, D, V], W / E [V, H] (bf16), anchor [batch]."""
    _arg(backbone, "backbone", _BF16)
    batch, D, V = backbone.shape
    _arg(W, "W", _BF16)
    Vw, H = W.shape
    if Vw != V:
        raise ValueError(f"W must have {V} rows, got {Vw}")
    _arg(E, "E", _BF16, (V, H))
    _arg(anchor, "anchor", _I32, (batch,))
    dev = backbone.device
    if out is None:
        out = dict(tree_tokens=torch.empty((batch, N), dtype=torch.int32, device=dev),
                   parents=torch.empty((batch, N), dtype=torch.int32, device=dev),
                   logq=torch.empty((batch, N), dtype=torch.float32, device=dev),
                   depths=torch.empty((batch, N), dtype=torch.int32, device=dev),
                   num_nodes=torch.empty((batch,), dtype=torch.int32, device=dev))
    size = lib().treespark_workspace_size(batch, D, V, H, k, F, N)
    if ws is None:
        ws = workspace("treespark", size, dev, (batch, D, V, H, k, F, N))
    rc = lib().treespark_expand(_ptr(backbone), _ptr(W), _ptr(E), _ptr(anchor), batch, D, V, H, k,
                                F, N, _ptr(out["tree_tokens"]), _ptr(out["parents"]),
                                _ptr(out["logq"]), _ptr(out.get("depths")),
                                _ptr(out["num_nodes"]), _ptr(ws), ws.numel(), _stream(dev))
    _check("treespark_expand", rc)
    return out


def sparkling_build(logits: torch.Tensor, W1: torch.Tensor, W2t: torch.Tensor, B: int, *,
                    C: int = 128, with_mask: bool = True, out: dict | None = None,
                    ws: torch.Tensor | None = None) -> dict:
    """SparklingTree: logits [batch, L, V] (bf16/f32), Markov head W1 / W2t [V, R] (bf16)
    -> tree tensors (as ddtree_build)."""
    _arg(logits, "logits", _LOGITS)
    if logits.dim() != 3:
        raise ValueError("logits must be [batch, L, V]")
    batch, L, V = logits.shape
    _arg(W1, "W1", _BF16)
    if W1.dim() != 2 or W1.shape[0] != V:
        raise ValueError(f"W1 must be [{V}, R]")
    R = W1.shape[1]
    _arg(W2t, "W2t", _BF16, (V, R))
    dev = logits.device
    dt = _dtype_code(logits)
    if out is None:
        out = _tree_out(batch, B, dev, with_mask)
    size = lib().sparkling_build_workspace_size(batch, L, V, C, R, B, dt)
    if ws is None:
        ws = workspace("sparkling", size, dev, (batch, L, V, C, R, B, dt))
    rc = lib().sparkling_build(_ptr(logits), dt, _ptr(W1), _ptr(W2t), batch, L, V, C, R, B,
                               _ptr(out["tree_tokens"]), _ptr(out["parents"]), _ptr(out["logq"]),
                               _ptr(out.get("depths")), _ptr(out["num_nodes"]),
                               _ptr(out.get("mask")), _ptr(ws), ws.numel(), _stream(dev))
    _check("sparkling_build", rc)
    return out


def dspark_budget(conf: torch.Tensor, cost_ms: torch.Tensor, *, out: dict | None = None) -> dict:
    """DSpark budget: conf [batch, P] float32, cost_ms [n_cost] float32 (cuda) ->
    keep [batch], n_keep [1], survival [batch, P], expected_tokens [1], objective [1]."""
    _arg(conf, "conf", (torch.float32,))
    if conf.dim() != 2:
        raise ValueError("conf must be [batch, P]")
    _arg(cost_ms, "cost_ms", (torch.float32,))
    if cost_ms.dim() != 1:
        raise ValueError("cost_ms must be 1-D")
    batch, P = conf.shape
    dev = conf.device
    if out is None:
        out = dict(keep=torch.empty((batch,), dtype=torch.int32, device=dev),
                   n_keep=torch.empty((1,), dtype=torch.int32, device=dev),
                   survival=torch.empty((batch, P), dtype=torch.float64, device=dev),
                   expected_tokens=torch.empty((1,), dtype=torch.float64, device=dev),
                   objective=torch.empty((1,), dtype=torch.float64, device=dev))
    rc = lib().dspark_budget(_ptr(conf), batch, P, _ptr(cost_ms), cost_ms.numel(),
                             _ptr(out["keep"]), _ptr(out.get("survival")), _ptr(out["n_keep"]),
                             _ptr(out.get("expected_tokens")), _ptr(out.get("objective")),
                             _stream(dev))
    _check("dspark_budget", rc)
    return out


def sparkling_beam(logits: torch.Tensor, W1: torch.Tensor, W2t: torch.Tensor, widths=None, *,
                   B: int | None = None, C: int = 128, with_mask: bool = True,
                   out: dict | None = None, ws: torch.Tensor | None = None) -> dict:
    """Beam tree on SparklingTree's rows: per-depth widths, or (widths None) the
    budget B spread evenly by the library."""
    _arg(logits, "logits", _LOGITS)
    if logits.dim() != 3:
        raise ValueError("logits must be [batch, L, V]")
    batch, L, V = logits.shape
    _arg(W1, "W1", _BF16)
    if W1.dim() != 2 or W1.shape[0] != V:
        raise ValueError(f"W1 must be [{V}, R]")
    R = W1.shape[1]
    _arg(W2t, "W2t", _BF16, (V, R))
    import ctypes  # (the argument C shadows the module alias)
    if widths is None:
        if B is None:
            raise ValueError("give widths or a budget B")
        Bt, wa = int(B), None
    else:
        widths = [int(w) for w in widths]
        if len(widths) != L:
            raise ValueError(f"widths must have {L} entries")
        Bt = sum(widths)
        wa = ctypes.cast((ctypes.c_int32 * L)(*widths), ctypes.c_void_p)
    dev = logits.device
    dt = _dtype_code(logits)
    if out is None:
        out = _tree_out(batch, max(Bt, 1), dev, with_mask)
    size = lib().sparkling_build_workspace_size(batch, L, V, C, R, max(Bt, 1), dt)
    if ws is None:
        ws = workspace("sparkling", size, dev, (batch, L, V, C, R, max(Bt, 1), dt))
    rc = lib().sparkling_beam(_ptr(logits), dt, _ptr(W1), _ptr(W2t), batch, L, V, C, R, wa,
                              0 if widths is not None else Bt,
                              _ptr(out["tree_tokens"]), _ptr(out["parents"]), _ptr(out["logq"]),
                              _ptr(out.get("depths")), _ptr(out["num_nodes"]),
                              _ptr(out.get("mask")), _ptr(ws), ws.numel(), _stream(dev))
    _check("sparkling_beam", rc)
    return out


# ---- the verification pass --------------------------------------------------
# Calls of a few microseconds on the device: the checks below are one test per
# tensor when it is right, and say what is wrong only when it is not.
_HALF = (torch.bfloat16, torch.float16)
_F32 = (torch.float32,)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _half_code(dtype) -> int:
    return DDT_BF16 if dtype == torch.bfloat16 else DDT_F16


def _dev_arg(t, name, dtype, shape, dev):
    """Device pointer of a contiguous tensor of this dtype and shape on device number dev."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype == dtype and \
            t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _arg(t, name, (dtype,), shape)
    raise ValueError(f"{name} must be on device {dev}, got {t.device}")


def _maybe_arg(t, name, dtype, shape, dev):
    return None if t is None else _dev_arg(t, name, dtype, shape, dev)


def _ws_arg(kind, size, ws, dev):
    """Pointer and size of the workspace of one call: the caller's, or this
    thread's own for the stream and kind (grown as needed), or, under graph
    capture, one of the graph's, so that no two graphs and no eager call share
    it. The second return value keeps it alive until the call is enqueued."""
    if ws is not None:
        if not isinstance(ws, torch.Tensor) or not ws.is_cuda or not ws.is_contiguous():
            raise ValueError("ws must be a contiguous device tensor")
        if ws.get_device() != dev:
            raise ValueError(f"ws must be on device {dev}, got {ws.device}")
        return ws.data_ptr(), ws, ws.numel() * ws.element_size()
    if torch.cuda.is_current_stream_capturing():
        ws = torch.empty(max(size, 1), dtype=torch.uint8, device=dev)
    else:
        key = (kind, dev, _raw_stream(dev))
        ws = _workspaces.get(key)
        if ws is None or ws.numel() < size:
            ws = torch.empty(max(size, 1), dtype=torch.uint8, device=dev)
            _workspaces[key] = ws
    return ws.data_ptr(), ws, ws.numel()


def _call(name, dev, args, kind=None, size=0, ws=None):
    """Calls the library with args, the workspace of `kind` if there is one and device dev's
    current stream, dev being the current device meanwhile; raises on an error status."""
    if torch.cuda.current_device() != dev:  # launches go to the current device
        with torch.cuda.device(dev):
            return _call(name, dev, args, kind, size, ws)
    fn = getattr(lib(), name)
    if kind is None:
        rc = fn(*args, _raw_stream(dev))
    else:
        wp, ws, size = _ws_arg(kind, size, ws, dev)
        rc = fn(*args, wp, size, _raw_stream(dev))
    if rc:
        _check(name, rc)


def _block_rows(t, name, dtype, batch, T, dh, dev):
    """Check [batch, T, heads, head_dim] rows at one distance; (pointer, heads, that distance)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on device {dev} like the caches, got {t.device}")
    shape = t.shape
    if len(shape) != 4 or shape[0] != batch or shape[1] != T or shape[3] != dh:
        raise ValueError(f"{name} must have shape ({batch}, {T}, heads, {dh}), got {tuple(shape)}")
    heads = shape[2]
    s0, s1, s2, s3 = t.stride()
    step = s1 if T > 1 else (s0 if batch > 1 else heads * dh)
    if (s3 != 1 and dh > 1) or (heads > 1 and s2 != dh) or (batch > 1 and s0 != T * step):
        raise ValueError(f"{name} must hold its heads side by side and its rows at one distance")
    return t.data_ptr(), heads, step


def _paged_cache(k_cache, v_cache, page_table, batch, dims):
    """Check a cache [(layers,) pages, kv_heads, page_size, head_dim] and its page
    table [batch, width]; (pointers, shape, width, device number)."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != dims:
        raise ValueError(f"k_cache must be a {dims}-d tensor "
                         f"[{'layers, ' if dims == 5 else ''}pages, kv_heads, page_size, head_dim]")
    shape, dev, dtype = k_cache.shape, k_cache.get_device(), k_cache.dtype
    if dev < 0:
        raise ValueError("k_cache must be a device tensor")
    k = _dev_arg(k_cache, "k_cache", dtype, shape, dev)
    v = _dev_arg(v_cache, "v_cache", dtype, shape, dev)
    if page_table is None:
        if shape[-4] != batch:
            raise ValueError(f"without a page table the cache must hold one page per request "
                             f"({batch}), got {shape[-4]}")
        return k, v, None, shape, 1, dev
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2 or \
            page_table.shape[0] != batch:
        raise ValueError(f"page_table must be a tensor of shape ({batch}, width)")
    table = page_table.shape
    return (k, v, _dev_arg(page_table, "page_table", torch.int32, table, dev), shape, table[1],
            dev)


def ddtree_append_kv(q, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, past_len: torch.Tensor, *,
                     rope: torch.Tensor | None = None, interleaved: bool = False,
                     page_table: torch.Tensor | None = None, depths: torch.Tensor | None = None,
                     num_nodes: torch.Tensor | None = None, q_out: torch.Tensor | None = None):
    """Verified block into one layer's cache: q [batch, T, q_heads, dh] (or None), k / v
    [batch, T, kv_heads, dh] (bf16/f16; slices of a fused projection are read in place), caches
    [pages, kv_heads, page_size, dh], rope [positions, rope_dim] float32 (cosines, then sines),
    depths [batch, T-1]; writes the caches and returns the rotated queries q_out (None for q None).
    Without q_out a new one is made and cleared first, a launch of its own."""
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be [batch, T, kv_heads, head_dim]")
    dt = k.dtype
    if dt not in _HALF:
        raise TypeError(f"k must have dtype {' or '.join(map(str, _HALF))}, got {dt}")
    batch, T, _, dh = k.shape
    kc, vc, table, shape, width, dev = _paged_cache(k_cache, v_cache, page_table, batch, 4)
    if k_cache.dtype != dt:
        raise TypeError(f"k_cache must have dtype {dt}, got {k_cache.dtype}")
    kp, kv_heads, ks = _block_rows(k, "k", dt, batch, T, dh, dev)
    vp, hv, vs = _block_rows(v, "v", dt, batch, T, dh, dev)
    pages, hc, page_size, dc = shape
    if hv != kv_heads or hc != kv_heads or dc != dh:
        raise ValueError("k, v and the caches must have the same heads and head_dim")
    qp, q_heads, qs, qo = None, 0, 0, None
    if q is None:
        q_out = None
    else:
        qp, q_heads, qs = _block_rows(q, "q", dt, batch, T, dh, dev)
        if q_out is None:
            q_out = torch.zeros((batch, T, q_heads, dh), dtype=dt, device=dev)
        qo = _dev_arg(q_out, "q_out", dt, (batch, T, q_heads, dh), dev)
    rp, rope_len, rot = None, 0, 0
    if rope is not None:
        if not isinstance(rope, torch.Tensor) or rope.dim() != 2:
            raise ValueError("rope must be [positions, rope_dim]")
        rope_len, rot = rope.shape
        rp = _dev_arg(rope, "rope", torch.float32, (rope_len, rot), dev)
    args = (qp, kp, vp, _half_code(dt), batch, T, q_heads, kv_heads, dh, qs, ks, vs, rp, rope_len,
            rot, 1 if interleaved else 0, _dev_arg(past_len, "past_len", torch.int32, (batch,), dev),
            _maybe_arg(depths, "depths", torch.int32, (batch, T - 1), dev),
            _maybe_arg(num_nodes, "num_nodes", torch.int32, (batch,), dev), table, width, pages,
            page_size, kc, vc, qo)
    _call("ddtree_append_kv", dev, args)
    return q_out


@functools.lru_cache(maxsize=1024)
def _attention_ws(*sizes) -> int:
    return lib().ddtree_attention_workspace_size(*sizes)


def ddtree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     past_len: torch.Tensor, *, page_table: torch.Tensor | None = None,
                     num_nodes: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                     scale: float | None = None, with_lse: bool = False, out: dict | None = None,
                     ws: torch.Tensor | None = None) -> dict:
    """Verified block's attention: q [batch, T, q_heads, dh] (bf16/f16) over one layer's caches
    [pages, kv_heads, page_size, dh] under the ancestor mask [batch, T, ceil(T/64)] (int64, as
    ddtree_mask's; None: a chain); scale defaults to dh ** -0.5. Returns out (and lse)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be [batch, T, q_heads, head_dim]")
    dt = q.dtype
    if dt not in _HALF:
        raise TypeError(f"q must have dtype {' or '.join(map(str, _HALF))}, got {dt}")
    batch, T, q_heads, dh = q.shape
    kc, vc, table, shape, width, dev = _paged_cache(k_cache, v_cache, page_table, batch, 4)
    qp = _dev_arg(q, "q", dt, q.shape, dev)
    if k_cache.dtype != dt:
        raise TypeError(f"k_cache must have dtype {dt}, got {k_cache.dtype}")
    pages, kv_heads, page_size, dc = shape
    if dc != dh:
        raise ValueError(f"the caches must have head_dim {dh}, got {dc}")
    if out is None:
        out = {"out": torch.empty_like(q)}
        if with_lse:
            out["lse"] = torch.empty((batch, T, q_heads), dtype=torch.float32, device=dev)
    args = (qp, _half_code(dt), batch, T, q_heads, kv_heads, dh, kc, vc, table, width, pages,
            page_size, _dev_arg(past_len, "past_len", torch.int32, (batch,), dev),
            _maybe_arg(num_nodes, "num_nodes", torch.int32, (batch,), dev),
            _maybe_arg(mask, "mask", torch.int64, (batch, T, (T + 63) // 64), dev),
            dh ** -0.5 if scale is None else float(scale),
            _dev_arg(out["out"], "out", dt, q.shape, dev),
            _maybe_arg(out.get("lse"), "lse", torch.float32, (batch, T, q_heads), dev))
    size = _attention_ws(batch, T, q_heads, kv_heads, dh, width, page_size)
    _call("ddtree_attention", dev, args, "attention", size, ws)
    return out


def ddtree_compact_kv_paged(k_cache: torch.Tensor, v_cache: torch.Tensor,
                            page_table: torch.Tensor, past_len: torch.Tensor,
                            accepted_nodes: torch.Tensor, accept_len: torch.Tensor,
                            new_len: torch.Tensor | None = None) -> torch.Tensor:
    """In place: paged caches [layers, pages, heads, page_size, head_dim] keep the accepted
    path's rows (page_table [batch, width]); returns new_len [batch]."""
    if not isinstance(past_len, torch.Tensor) or past_len.dim() != 1:
        raise ValueError("past_len must be [batch]")
    batch = past_len.shape[0]
    if page_table is None:
        raise ValueError("page_table is required; ddtree_compact_kv takes contiguous caches")
    kc, vc, table, shape, width, dev = _paged_cache(k_cache, v_cache, page_table, batch, 5)
    layers, pages, heads, page_size, dh = shape
    if not isinstance(accepted_nodes, torch.Tensor) or accepted_nodes.dim() != 2:
        raise ValueError("accepted_nodes must be [batch, L]")
    L = accepted_nodes.shape[1]
    if new_len is None:
        new_len = torch.empty((batch,), dtype=torch.int32, device=dev)
    args = (_dev_arg(past_len, "past_len", torch.int32, (batch,), dev),
            _dev_arg(accepted_nodes, "accepted_nodes", torch.int32, (batch, L), dev),
            _dev_arg(accept_len, "accept_len", torch.int32, (batch,), dev), L,
            _dev_arg(new_len, "new_len", torch.int32, (batch,), dev))
    _call("ddtree_compact_kv_paged", dev, (kc, vc, layers, pages, heads, page_size,
                                           dh * k_cache.element_size(), table, width, batch,
                                           *args))
    return new_len


@functools.lru_cache(maxsize=1024)
def _accept_ws(*sizes) -> int:
    return lib().ddtree_accept_sampled_workspace_size(*sizes)


@functools.lru_cache(maxsize=1024)
def _chain_ws(*sizes) -> int:
    return lib().dspark_accept_sampled_workspace_size(*sizes)


def _rows_arg(t, name, batch):
    """A [batch, n] tensor argument's n."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or (batch is not None and t.shape[0] != batch):
        raise ValueError(f"{name} must be [{'batch' if batch is None else batch}, n]")
    return t.shape[1]


def ddtree_accept_sampled(tree_tokens: torch.Tensor, parents: torch.Tensor,
                          num_nodes: torch.Tensor | None, target_logits: torch.Tensor,
                          temperature: torch.Tensor | None, u: torch.Tensor, *,
                          out: dict | None = None, ws: torch.Tensor | None = None) -> dict:
    """Tree acceptance at a temperature: target_logits [batch, B+1, V] (bf16/f32), temperature
    [batch] (None: 1; 0: greedy), u [batch, L+1] uniforms -> accepted_nodes [batch, L],
    accept_len, next_token, logp [batch, L+1]."""
    _arg(target_logits, "target_logits", _LOGITS)
    B = _rows_arg(tree_tokens, "tree_tokens", None)
    batch, V, dev = tree_tokens.shape[0], target_logits.shape[-1], target_logits.get_device()
    L = _rows_arg(u, "u", batch) - 1
    dt = DDT_BF16 if target_logits.dtype == torch.bfloat16 else DDT_F32
    if out is None:
        i32 = torch.empty((max(L, 0) + 2, batch), dtype=torch.int32, device=dev)
        out = dict(accepted_nodes=i32[2:].view(batch, max(L, 0)), accept_len=i32[0],
                   next_token=i32[1],
                   logp=torch.empty((batch, L + 1), dtype=torch.float32, device=dev))
    args = (_dev_arg(tree_tokens, "tree_tokens", torch.int32, (batch, B), dev),
            _dev_arg(parents, "parents", torch.int32, (batch, B), dev),
            _maybe_arg(num_nodes, "num_nodes", torch.int32, (batch,), dev),
            _dev_arg(target_logits, "target_logits", target_logits.dtype, (batch, B + 1, V), dev),
            dt, _maybe_arg(temperature, "temperature", torch.float32, (batch,), dev),
            _dev_arg(u, "u", torch.float32, (batch, L + 1), dev), batch, B, L, V,
            _dev_arg(out["accepted_nodes"], "accepted_nodes", torch.int32, (batch, L), dev),
            _dev_arg(out["accept_len"], "accept_len", torch.int32, (batch,), dev),
            _dev_arg(out["next_token"], "next_token", torch.int32, (batch,), dev),
            _maybe_arg(out.get("logp"), "logp", torch.float32, (batch, L + 1), dev))
    _call("ddtree_accept_sampled", dev, args, "accept_sampled", _accept_ws(batch, B, L, V, dt), ws)
    return out


def dspark_accept_sampled(tokens: torch.Tensor, target_logits: torch.Tensor,
                          draft_logits: torch.Tensor, temperature: torch.Tensor | None,
                          u: torch.Tensor, *, keep: torch.Tensor | None = None,
                          out: dict | None = None, ws: torch.Tensor | None = None) -> dict:
    """Verification of a sampled chain: tokens [batch, P], target_logits [batch, P+1, V],
    draft_logits [batch, P, V] (bf16/f32), temperature [batch] (None: 1; 0: greedy), u
    [batch, P+1] uniforms, keep [batch] -> accept_len, next_token, logp [batch, P+1]."""
    _arg(target_logits, "target_logits", _LOGITS)
    P = _rows_arg(tokens, "tokens", None)
    batch, V, dev = tokens.shape[0], target_logits.shape[-1], target_logits.get_device()
    dt = DDT_BF16 if target_logits.dtype == torch.bfloat16 else DDT_F32
    if out is None:
        i32 = torch.empty((2, batch), dtype=torch.int32, device=dev)
        out = dict(accept_len=i32[0], next_token=i32[1],
                   logp=torch.empty((batch, P + 1), dtype=torch.float32, device=dev))
    args = (_dev_arg(tokens, "tokens", torch.int32, (batch, P), dev),
            _maybe_arg(keep, "keep", torch.int32, (batch,), dev),
            _dev_arg(target_logits, "target_logits", target_logits.dtype, (batch, P + 1, V), dev),
            _dev_arg(draft_logits, "draft_logits", target_logits.dtype, (batch, P, V), dev), dt,
            _maybe_arg(temperature, "temperature", torch.float32, (batch,), dev),
            _dev_arg(u, "u", torch.float32, (batch, P + 1), dev), batch, P, V,
            _dev_arg(out["accept_len"], "accept_len", torch.int32, (batch,), dev),
            _dev_arg(out["next_token"], "next_token", torch.int32, (batch,), dev),
            _maybe_arg(out.get("logp"), "logp", torch.float32, (batch, P + 1), dev))
    _call("dspark_accept_sampled", dev, args, "chain_accept_sampled", _chain_ws(batch, P, V, dt),
          ws)
    return out
