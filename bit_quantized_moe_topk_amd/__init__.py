"""Routed MoE FFN over 2/3-bit block-quantized experts on one MI355X (gfx950).

Thin ctypes binding over ``libmoe.so`` (the C ABI in ``include/moe.h``). Every
step of the layer runs in the library's HIP kernels; this module only checks
tensor placement, allocates outputs and workspace with PyTorch and passes raw
device pointers plus the current HIP stream. There is no CPU fallback: without
the built library every call raises.

Calls, in the order a layer uses them:
    idx, gates = route_topk(logits, k)
    grp        = group(idx, E, has_shared)                  # optional
    ex         = Experts(qtype, E, has_shared, H, I, codes, hi, dm)
    y          = ffn_q(x, ex, idx, gates, grouping=grp, mode="fast" | "check")

Experts in microscaled 4-bit blocks, and a router in training:
    w  = mx4_quantize(weights)                              # [E (+ 1), N, K] -> Mx4
    y  = mx4_experts_matmul(x, w, grp, tokens=T)            # [A, N], in the groups' order
    dx = mx4_experts_matmul_backward(dy, w, grp, tokens=T)
    bl = balance_loss(logits, idx);  dlogits = balance_loss_backward(logits, bl, d_losses)
The *_backward calls are explicit: no call here records a graph for autograd.
"""
from __future__ import annotations

import ctypes as C
import functools
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP = 0, -1, -2, -3, -4
F32, BF16, MX4 = 0, 1, 4
Q2, Q3 = 2, 3
FAST, CHECK_F32 = 0, 2
MAX_E = 2048

_lib = None


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status} ({status_string(status)})")
        self.status = status


def lib() -> C.CDLL:
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m bit_quantized_moe_topk_amd.build`")
        L = C.CDLL(LIB_PATH)
        P, i32, sz = C.c_void_p, C.c_int32, C.c_size_t
        L.moe_status_string.argtypes = [i32]
        L.moe_status_string.restype = C.c_char_p
        L.moe_router_logits.argtypes = [P, i32, i32, i32, P, P, i32, P, P]
        L.moe_router_logits.restype = C.c_int
        L.moe_route_topk.argtypes = [P, i32, i32, i32, P, P, P]
        L.moe_route_topk.restype = C.c_int
        L.moe_group_workspace_size.argtypes = [i32, i32, i32]
        L.moe_group_workspace_size.restype = sz
        L.moe_group.argtypes = [P, i32, i32, i32, i32, P, P, P, P, P, sz, P]
        L.moe_group.restype = C.c_int
        L.moe_route_group.argtypes = [P, i32, i32, i32, i32, P, P, P, P, P, P, P, sz, P]
        L.moe_route_group.restype = C.c_int
        L.moe_experts_create.argtypes = [C.POINTER(P), i32, i32, i32, i32, i32, P, P, P]
        L.moe_experts_create.restype = C.c_int
        L.moe_experts_destroy.argtypes = [P]
        L.moe_experts_destroy.restype = C.c_int
        L.moe_experts_tiled_size.argtypes = [P]
        L.moe_experts_tiled_size.restype = sz
        L.moe_experts_attach_tiled.argtypes = [P, P, sz, P]
        L.moe_experts_attach_tiled.restype = C.c_int
        L.moe_ffn_q_workspace_size.argtypes = [P, i32, i32, i32]
        L.moe_ffn_q_workspace_size.restype = sz
        L.moe_ffn_q.argtypes = [P, i32, i32, P, P, P, i32, P, P, P, P, P, i32, P, sz, P]
        L.moe_ffn_q.restype = C.c_int
        L.moe_layer_workspace_size.argtypes = [P, i32, i32, i32]
        L.moe_layer_workspace_size.restype = sz
        L.moe_layer.argtypes = [P, P, i32, i32, P, i32, P, P, P, i32, P, sz, P]
        L.moe_layer.restype = C.c_int
        L.moe_layer_static.argtypes = [P, P, i32, i32, P, i32, P, P, P, i32, P]
        L.moe_layer_static.restype = C.c_int
        L.moe_router_topk.argtypes = [P, i32, i32, i32, P, P, i32, i32, P, P, P, P]
        L.moe_router_topk.restype = C.c_int
        L.moe_expert_gateup_fp8_workspace_size.argtypes = [P, i32]
        L.moe_expert_gateup_fp8_workspace_size.restype = sz
        L.moe_expert_gateup_fp8.argtypes = [P, i32, P, i32, P, P, sz, P]
        L.moe_expert_gateup_fp8.restype = C.c_int
        L.moe_layer_hidden_workspace_size.argtypes = [P, i32, i32, i32]
        L.moe_layer_hidden_workspace_size.restype = sz
        L.moe_layer_hidden.argtypes = [P, i32, i32, P, P, P, i32, P, P, P, P, i32, P, sz, P]
        L.moe_layer_hidden.restype = C.c_int
        i64, u = C.c_int64, P
        sigs = {
            "moe_mx4_quantize": [P, i32, i64, i32, i32, u, u, P],
            "moe_mx4_dequantize": [u, u, i32, i32, i32, P, P],
            "moe_mx4_matmul": [P, u, i32, i64, i32, u, u, i32, i32, P, i32, P],
            "moe_mx4_matmul_backward": [P, i32, i64, i32, u, u, i32, i32, P, i32, P],
            "moe_mx4_experts_matmul": [P, u, i32, i64, i32, i32, i32, i32, i32, P, P, u, u, i32, i32, P,
                                       i32, P, sz, P],
            "moe_mx4_experts_matmul_backward": [P, i32, i64, i32, i32, i32, i32, i32, P, P, u, u, i32,
                                                i32, P, i32, P, sz, P],
            "moe_balance_loss": [P, i32, i64, i32, i32, i32, P, P, P, P, P, P, sz, P],
            "moe_balance_loss_backward": [P, i32, i64, i32, i32, i32, P, P, P, P, P, P],
        }
        for name, args in sigs.items():
            getattr(L, name).argtypes = args
            getattr(L, name).restype = C.c_int
        L.moe_mx4_experts_matmul_workspace_size.argtypes = [i32] * 3
        L.moe_mx4_experts_matmul_workspace_size.restype = sz
        L.moe_mx4_experts_matmul_backward_workspace_size.argtypes = [i32] * 5
        L.moe_mx4_experts_matmul_backward_workspace_size.restype = sz
        L.moe_balance_loss_workspace_size.argtypes = [i32] * 3
        L.moe_balance_loss_workspace_size.restype = sz
        L.moe_profile_begin.argtypes = [i32]
        L.moe_profile_begin.restype = C.c_int
        L.moe_profile_end.argtypes = []
        L.moe_profile_end.restype = C.c_int
        L.moe_profile_count.argtypes = []
        L.moe_profile_count.restype = i32
        L.moe_profile_get.argtypes = [i32, C.POINTER(C.c_char_p), C.POINTER(i32),
                                      C.POINTER(C.c_double)]
        L.moe_profile_get.restype = C.c_int
        _lib = L
    return _lib


def profile_begin(max_launches: int = 65536) -> None:
    """Record HIP events around every library launch from now on."""
    _check("moe_profile_begin", lib().moe_profile_begin(max_launches))


def profile_end() -> dict:
    """Stop recording; return {kernel name: (launches, total ms)}."""
    L = lib()
    _check("moe_profile_end", L.moe_profile_end())
    out = {}
    for i in range(L.moe_profile_count()):
        name, n, ms = C.c_char_p(), C.c_int32(), C.c_double()
        _check("moe_profile_get", L.moe_profile_get(i, C.byref(name), C.byref(n), C.byref(ms)))
        out[name.value.decode()] = (n.value, ms.value)
    return out


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != OK:
        raise MoeError(fn, status)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream():
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need_cuda(name: str, t: torch.Tensor, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def router_logits(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None):
    """Router scores x . w[e] (+ bias[e]): float32 [T, E]. x: f32 or bf16 [T, H];
    w: bf16 [E, H] (or its uint16/int16 bit patterns); bias: f32 [E] or None."""
    _need_cuda("x", x, (torch.float32, torch.bfloat16))
    if w.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or not w.is_cuda or not w.is_contiguous():
        raise ValueError("w must be a contiguous CUDA bf16 (or 16-bit pattern) tensor [E, H]")
    if bias is not None:
        _need_cuda("bias", bias, torch.float32)
    T, H = x.shape
    E = w.shape[0]
    if w.shape[1] != H or (bias is not None and bias.numel() != E):
        raise ValueError("shape mismatch between x, w and bias")
    logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    xdt = F32 if x.dtype == torch.float32 else BF16
    _check("moe_router_logits", lib().moe_router_logits(_ptr(x), xdt, T, H, _ptr(w),
                                                        _ptr(bias) if bias is not None else None,
                                                        E, _ptr(logits), _stream()))
    return logits


def router_topk(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None, k: int):
    """moe_router_topk: router product and top-k in one launch (bf16 x [T, H],
    w bf16 [E, H]): returns (idx int32 [T, k], gates f32 [T, k], logits f32 [T, E])."""
    _need_cuda("x", x, torch.bfloat16)
    if w.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or not w.is_cuda or not w.is_contiguous():
        raise ValueError("w must be a contiguous CUDA bf16 (or 16-bit pattern) tensor [E, H]")
    if bias is not None:
        _need_cuda("bias", bias, torch.float32)
    T, H = x.shape
    E = w.shape[0]
    if w.shape[1] != H or (bias is not None and bias.numel() != E):
        raise ValueError("shape mismatch between x, w and bias")
    idx = torch.empty((T, k), dtype=torch.int32, device=x.device)
    gates = torch.empty((T, k), dtype=torch.float32, device=x.device)
    logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    _check("moe_router_topk", lib().moe_router_topk(_ptr(x), BF16, T, H, _ptr(w),
                                                    _ptr(bias) if bias is not None else None, E, k,
                                                    _ptr(idx), _ptr(gates), _ptr(logits), _stream()))
    return idx, gates, logits


def route_topk(logits: torch.Tensor, k: int):
    """Top-k experts per token and their softmax gates: (idx int32 [T,k], gates f32 [T,k])."""
    _need_cuda("logits", logits, torch.float32)
    T, E = logits.shape
    idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    gates = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check("moe_route_topk", lib().moe_route_topk(_ptr(logits), T, E, k, _ptr(idx), _ptr(gates),
                                                  _stream()))
    return idx, gates


@dataclass
class Grouping:
    counts: torch.Tensor   # int32 [E+1]
    offsets: torch.Tensor  # int32 [E+2]
    perm: torch.Tensor     # int32 [A]
    slot_of: torch.Tensor  # int32 [A]
    has_shared: bool | None = None  # set by group() and route_group()


def group(idx: torch.Tensor, E: int, has_shared: bool) -> Grouping:
    """Stable grouping of the assignments of ``idx`` by expert."""
    _need_cuda("idx", idx, torch.int32)
    T, k = idx.shape
    dev = idx.device
    A = T * (k + int(bool(has_shared)))
    g = Grouping(torch.empty(E + 1, dtype=torch.int32, device=dev),
                 torch.empty(E + 2, dtype=torch.int32, device=dev),
                 torch.empty(max(A, 1), dtype=torch.int32, device=dev),
                 torch.empty(max(A, 1), dtype=torch.int32, device=dev))
    nbytes = lib().moe_group_workspace_size(T, k, E)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _check("moe_group", lib().moe_group(_ptr(idx), T, k, E, int(bool(has_shared)), _ptr(g.counts),
                                        _ptr(g.offsets), _ptr(g.perm), _ptr(g.slot_of), _ptr(ws),
                                        nbytes, _stream()))
    g.perm = g.perm[:A]
    g.slot_of = g.slot_of[:A]
    g.has_shared = bool(has_shared)
    return g


def route_group(logits: torch.Tensor, k: int, has_shared: bool):
    """Top-k routing and the grouping in one call: (idx, gates, Grouping)."""
    _need_cuda("logits", logits, torch.float32)
    T, E = logits.shape
    dev = logits.device
    A = T * (k + int(bool(has_shared)))
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    gates = torch.empty((T, k), dtype=torch.float32, device=dev)
    g = Grouping(torch.empty(E + 1, dtype=torch.int32, device=dev),
                 torch.empty(E + 2, dtype=torch.int32, device=dev),
                 torch.empty(max(A, 1), dtype=torch.int32, device=dev),
                 torch.empty(max(A, 1), dtype=torch.int32, device=dev))
    nbytes = lib().moe_group_workspace_size(T, k, E)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _check("moe_route_group", lib().moe_route_group(
        _ptr(logits), T, E, k, int(bool(has_shared)), _ptr(idx), _ptr(gates), _ptr(g.counts),
        _ptr(g.offsets), _ptr(g.perm), _ptr(g.slot_of), _ptr(ws), nbytes, _stream()))
    g.perm = g.perm[:A]
    g.slot_of = g.slot_of[:A]
    g.has_shared = bool(has_shared)
    return idx, gates, g


class Experts:
    """One layer's packed experts (device planes in the canonical layout)."""

    def __init__(self, qtype: int, E: int, has_shared: bool, H: int, I: int,
                 codes: torch.Tensor, hi: torch.Tensor | None, dm: torch.Tensor):
        _need_cuda("codes", codes, torch.uint8)
        _need_cuda("dm", dm, (torch.uint16, torch.int16))
        if hi is not None:
            _need_cuda("hi", hi, torch.uint8)
        E_tot = E + int(bool(has_shared))
        nb = 3 * H * I // 32
        if codes.numel() != E_tot * nb * 8 or dm.numel() != E_tot * nb * 2:
            raise ValueError("plane sizes do not match the shape")
        if qtype == Q3 and (hi is None or hi.numel() != E_tot * nb * 4):
            raise ValueError("Q3 needs a high-bit plane of E_tot * NB * 4 bytes")
        self.qtype, self.E, self.has_shared, self.H, self.I = qtype, E, bool(has_shared), H, I
        self._planes = (codes, hi, dm)  # keep alive for the handle's lifetime
        h = C.c_void_p()
        _check("moe_experts_create",
               lib().moe_experts_create(C.byref(h), qtype, E, int(bool(has_shared)), H, I,
                                        _ptr(codes), _ptr(hi), _ptr(dm)))
        self._h = h

    @property
    def handle(self) -> C.c_void_p:
        return self._h

    def attach_tiled(self) -> None:
        """Build the tiled weight copy that the prefill matrix-core tiles read
        (a device buffer as large as the planes, kept by this object)."""
        import torch
        nbytes = int(lib().moe_experts_tiled_size(self._h))
        buf = torch.empty(nbytes, dtype=torch.uint8, device=self._planes[0].device)
        stream = C.c_void_p(torch.cuda.current_stream().cuda_stream)
        _check("moe_experts_attach_tiled",
               lib().moe_experts_attach_tiled(self._h, _ptr(buf), nbytes, stream))
        self._tiled = buf

    def detach_tiled(self) -> None:
        _check("moe_experts_attach_tiled", lib().moe_experts_attach_tiled(self._h, None, 0, None))
        self._tiled = None

    def workspace_size(self, T: int, k: int, mode: int = FAST) -> int:
        return int(lib().moe_ffn_q_workspace_size(self._h, T, k, mode))

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().moe_experts_destroy(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_MODES = {"fast": FAST, "check": CHECK_F32, FAST: FAST, CHECK_F32: CHECK_F32}


def ffn_q(x: torch.Tensor, ex: Experts, idx: torch.Tensor, gates: torch.Tensor,
          grouping: Grouping | None = None, mode="fast", workspace: torch.Tensor | None = None,
          out: torch.Tensor | None = None) -> torch.Tensor:
    """Expert FFN + gate-weighted combine for every token of ``x``.

    ``x``: [T, H] float32 or bfloat16. Returns ``y`` [T, H] with x's dtype in
    fast mode, float32 in check mode.
    """
    mode = _MODES[mode]
    _need_cuda("x", x, (torch.float32, torch.bfloat16))
    _need_cuda("idx", idx, torch.int32)
    _need_cuda("gates", gates, torch.float32)
    T, H = x.shape
    k = idx.shape[1]
    if H != ex.H or idx.shape[0] != T or tuple(gates.shape) != (T, k):
        raise ValueError("shape mismatch between x, idx, gates and the experts")
    xdt = F32 if x.dtype == torch.float32 else BF16
    ydtype = torch.float32 if mode == CHECK_F32 else x.dtype
    y = out if out is not None else torch.empty((T, H), dtype=ydtype, device=x.device)
    _need_cuda("out", y, ydtype)
    nbytes = ex.workspace_size(T, k, mode)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
    g = grouping
    _check("moe_ffn_q", lib().moe_ffn_q(
        _ptr(x), xdt, T, ex.handle, _ptr(idx), _ptr(gates), k,
        _ptr(g.counts) if g else None, _ptr(g.offsets) if g else None,
        _ptr(g.perm) if g else None, _ptr(g.slot_of) if g else None,
        _ptr(y), mode, _ptr(workspace), workspace.numel(), _stream()))
    return y


def layer(logits: torch.Tensor, x: torch.Tensor, ex: "Experts", k: int, mode="fast",
          workspace: torch.Tensor | None = None, out=None):
    """The whole layer (route, group, expert FFN, combine): returns (idx, gates, y).

    A caller-provided `workspace` (uint8, at least moe_layer_workspace_size
    bytes) must start zero-filled; the calls keep the counters in its first
    8192 bytes consistent from call to call. `out` = (idx, gates, y) writes
    into existing tensors (as a captured graph needs)."""
    mode = _MODES[mode]
    _need_cuda("logits", logits, torch.float32)
    _need_cuda("x", x, (torch.float32, torch.bfloat16))
    T, H = x.shape
    if H != ex.H or logits.shape[0] != T:
        raise ValueError("shape mismatch between logits, x and the experts")
    dev = x.device
    ydtype = torch.float32 if mode == CHECK_F32 else x.dtype
    if out is None:
        idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        gates = torch.empty((T, k), dtype=torch.float32, device=dev)
        y = torch.empty((T, H), dtype=ydtype, device=dev)
    else:
        idx, gates, y = out
        _need_cuda("idx", idx, torch.int32)
        _need_cuda("gates", gates, torch.float32)
        _need_cuda("y", y, ydtype)
        if tuple(idx.shape) != (T, k) or tuple(gates.shape) != (T, k) or tuple(y.shape) != (T, H):
            raise ValueError("out tensors do not match (T, k) and (T, H)")
    nbytes = int(lib().moe_layer_workspace_size(ex.handle, T, k, mode))
    if workspace is None:  # zero-filled: its head holds the decode window's counters
        workspace = torch.zeros(max(nbytes, 1), dtype=torch.uint8, device=dev)
    xdt = F32 if x.dtype == torch.float32 else BF16
    _check("moe_layer", lib().moe_layer(_ptr(logits), _ptr(x), xdt, T, ex.handle, k, _ptr(idx),
                                        _ptr(gates), _ptr(y), mode, _ptr(workspace),
                                        workspace.numel(), _stream()))
    return idx, gates, y


def layer_hidden(x: torch.Tensor, w_router: torch.Tensor, bias: torch.Tensor | None, ex: "Experts",
                 k: int, mode="fast", workspace: torch.Tensor | None = None, out=None,
                 logits: torch.Tensor | None = None):
    """moe_layer_hidden: the router product, then the whole layer, from the
    hidden states x [T, H]: returns (idx, gates, y, logits). w_router: bf16 [E, H]
    (or its 16-bit patterns); bias: f32 [E] or None. `logits` (f32 [T, E]) receives
    the router scores; when None, a new tensor does. `workspace` and `out` as
    for layer()."""
    mode = _MODES[mode]
    _need_cuda("x", x, (torch.float32, torch.bfloat16))
    if (w_router.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or not w_router.is_cuda
            or not w_router.is_contiguous()):
        raise ValueError("w_router must be a contiguous CUDA bf16 (or 16-bit pattern) tensor [E, H]")
    if bias is not None:
        _need_cuda("bias", bias, torch.float32)
    T, H = x.shape
    if H != ex.H or tuple(w_router.shape) != (ex.E, H) or (bias is not None and bias.numel() != ex.E):
        raise ValueError("shape mismatch between x, w_router, bias and the experts")
    dev = x.device
    ydtype = torch.float32 if mode == CHECK_F32 else x.dtype
    if out is None:
        idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        gates = torch.empty((T, k), dtype=torch.float32, device=dev)
        y = torch.empty((T, H), dtype=ydtype, device=dev)
    else:
        idx, gates, y = out
        _need_cuda("idx", idx, torch.int32)
        _need_cuda("gates", gates, torch.float32)
        _need_cuda("y", y, ydtype)
    if logits is None:
        logits = torch.empty((T, ex.E), dtype=torch.float32, device=dev)
    _need_cuda("logits", logits, torch.float32)
    nbytes = int(lib().moe_layer_hidden_workspace_size(ex.handle, T, k, mode))
    if workspace is None:  # zero-filled: its head holds the decode window's counters
        workspace = torch.zeros(max(nbytes, 1), dtype=torch.uint8, device=dev)
    xdt = F32 if x.dtype == torch.float32 else BF16
    _check("moe_layer_hidden", lib().moe_layer_hidden(
        _ptr(x), xdt, T, _ptr(w_router), _ptr(bias) if bias is not None else None, ex.handle, k,
        _ptr(idx), _ptr(gates), _ptr(y), _ptr(logits), mode, _ptr(workspace), workspace.numel(),
        _stream()))
    return idx, gates, y, logits


def expert_gateup_fp8(x: torch.Tensor, ex: "Experts", expert: int,
                      workspace: torch.Tensor | None = None) -> torch.Tensor:
    """moe_expert_gateup_fp8: h = silu(g) * u of one expert for every row of
    x (bf16 [T, H]) on the FP8 matrix cores (a measured variant): f32 [T, I]."""
    _need_cuda("x", x, torch.bfloat16)
    T, H = x.shape
    if H != ex.H:
        raise ValueError("x does not match the experts' H")
    h = torch.empty((T, ex.I), dtype=torch.float32, device=x.device)
    n = int(lib().moe_expert_gateup_fp8_workspace_size(ex.handle, T))
    if workspace is None:
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=x.device)
    _check("moe_expert_gateup_fp8", lib().moe_expert_gateup_fp8(
        _ptr(x), T, ex.handle, expert, _ptr(h), _ptr(workspace), workspace.numel(), _stream()))
    return h


def layer_static(logits: torch.Tensor, x: torch.Tensor, ex: "Experts", k: int, mode="fast"):
    """moe_layer_static: the whole layer on the library's own per-GPU scratch
    (no workspace argument, nothing allocated by the library): (idx, gates, y)."""
    mode = _MODES[mode]
    _need_cuda("logits", logits, torch.float32)
    _need_cuda("x", x, (torch.float32, torch.bfloat16))
    T, H = x.shape
    if H != ex.H or logits.shape[0] != T:
        raise ValueError("shape mismatch between logits, x and the experts")
    dev = x.device
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    gates = torch.empty((T, k), dtype=torch.float32, device=dev)
    y = torch.empty((T, H), dtype=torch.float32 if mode == CHECK_F32 else x.dtype, device=dev)
    xdt = F32 if x.dtype == torch.float32 else BF16
    _check("moe_layer_static", lib().moe_layer_static(_ptr(logits), _ptr(x), xdt, T, ex.handle, k,
                                                      _ptr(idx), _ptr(gates), _ptr(y), mode,
                                                      _stream()))
    return idx, gates, y


# ---- microscaled 4-bit operands ---------------------------------------------------

_FLOATS = {torch.float32: F32, torch.bfloat16: BF16}
_MOST = 2 ** 31 - 1  # sizes that the library's calls can be told


# The handle of a device's current stream (the first form builds no Stream object: small products
# take a few microseconds in all).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(name: str, dev: torch.device, *args) -> None:
    """Runs a library call on the current stream of the tensors' device."""
    fn = getattr(_lib or lib(), name)
    i = dev.index
    if i == torch.cuda.current_device():
        st = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(i))
    if st != OK:
        raise MoeError(name, st)


def _rows(name: str, t: torch.Tensor, n: int | None = None):
    """Checks rows of float values ([R, n], values adjacent): (type code, elements from row to row, R)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    code = _FLOATS.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {t.dtype}, expected float32 or bfloat16")
    shape = t.shape
    if len(shape) != 2 or (n is not None and shape[1] != n):
        raise ValueError(f"{name} must be [rows, {'n' if n is None else n}]: got {tuple(shape)}")
    R, m = shape
    if R > _MOST or m > _MOST:
        raise ValueError(f"{name} is too large: {tuple(shape)}")
    ld, inner = t.stride()
    if R <= 1:
        ld = m
    if ld < m or (inner != 1 and m > 1):
        raise ValueError(f"{name} must have adjacent values in each row, and rows that do not overlap")
    return code, ld, R


def _int32(name: str, t: torch.Tensor, dev: torch.device, n: int = 0):
    if t.dtype is not torch.int32 or t.device != dev or not t.is_contiguous() or t.numel() < n:
        _need_cuda(name, t, torch.int32)
        raise ValueError(f"{name} must be on {dev}" + (f" and hold {n} values" if n else ""))


def _result(out, shape, dtype, dev: torch.device) -> torch.Tensor:
    if dtype not in _FLOATS:
        raise TypeError(f"results are float32 or bfloat16, not {dtype}")
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _need_cuda("out", out, dtype)
    if tuple(out.shape) != tuple(shape) or out.device != dev:
        raise ValueError(f"out must be {tuple(shape)} on {dev}")
    return out


class Mx4:
    """Rows of K values in microscaled 4-bit blocks: codes uint8 [..., 16 B], scales uint8 [..., B],
    B = ceil(K / 32) blocks a row (the layout is in include/moe.h). [N, K] is a matrix or N rows of
    activations, [E, N, K] one matrix for each expert."""

    __slots__ = ("codes", "scales", "K")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, K: int):
        _need_cuda("codes", codes, torch.uint8)
        _need_cuda("scales", scales, torch.uint8)
        c, s = codes.shape, scales.shape
        if K < 1 or len(c) < 2 or s[-1] != (K + 31) // 32 or c[-1] != 16 * s[-1] or c[:-1] != s[:-1]:
            raise ValueError(f"codes {tuple(c)} and scales {tuple(s)} do not hold rows of {K}")
        if codes.device != scales.device:
            raise ValueError("codes and scales must be on one device")
        if K > _MOST or s[:-1].numel() > _MOST:
            raise ValueError(f"too many rows or values: {tuple(s[:-1])} rows of {K}")
        self.codes, self.scales, self.K = codes, scales, K

    @classmethod
    def _new(cls, shape, K: int, dev: torch.device) -> "Mx4":
        """Room for rows [*shape, K]."""
        self, B = object.__new__(cls), (K + 31) // 32
        self.codes = torch.empty((*shape, 16 * B), dtype=torch.uint8, device=dev)
        self.scales = torch.empty((*shape, B), dtype=torch.uint8, device=dev)
        self.K = K
        return self

    @property
    def shape(self) -> tuple:
        return (*self.codes.shape[:-1], self.K)

    @property
    def device(self) -> torch.device:
        return self.codes.device


def mx4_quantize(x: torch.Tensor, out: Mx4 | None = None) -> Mx4:
    """Rows x ([..., K], float32 or bfloat16) as microscaled 4-bit blocks (moe_mx4_quantize). More than
    two dimensions must be contiguous; of two, rows may lie further apart."""
    if isinstance(x, torch.Tensor) and x.dim() > 2 and not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if not isinstance(x, torch.Tensor) or x.dim() < 2 or x.shape[-1] < 1:
        raise ValueError("x must be a tensor [..., K] of two dimensions or more")
    K = x.shape[-1]
    flat = x if x.dim() == 2 else x.reshape(-1, K)
    code, ld, rows = _rows("x", flat)
    if out is None:
        out = Mx4._new(x.shape[:-1], K, x.device)
    elif out.shape != tuple(x.shape) or out.device != x.device:
        raise ValueError(f"out must be an Mx4 of {tuple(x.shape)} on {x.device}")
    _call("moe_mx4_quantize", x.device, flat.data_ptr(), code, ld, rows, K, out.codes.data_ptr(),
          out.scales.data_ptr())
    return out


def mx4_dequantize(q: Mx4, dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of q, [..., K], in float32 or bfloat16 (exact in both)."""
    y = _result(out, q.shape, dtype, q.device)
    _call("moe_mx4_dequantize", q.device, q.codes.data_ptr(), q.scales.data_ptr(), q.codes.shape[:-1].numel(), q.K,
          _FLOATS[dtype], y.data_ptr())
    return y


def _product_rows(x, K: int):
    """A product's rows: (data, scales, type code, row distance, rows, device, result type)."""
    if isinstance(x, Mx4):
        if x.codes.dim() != 2 or x.K != K:
            raise ValueError(f"x must be rows of {K} values: got {x.shape}")
        return x.codes.data_ptr(), x.scales.data_ptr(), MX4, 0, x.codes.shape[0], x.device, torch.bfloat16
    code, ld, R = _rows("x", x, K)
    return x.data_ptr(), None, code, ld, R, x.device, x.dtype


def _matrix(w: Mx4, dims: int) -> int:
    shape = w.codes.shape if isinstance(w, Mx4) else ()
    if len(shape) != dims or shape[-2] < 1:
        raise ValueError(f"w must be an Mx4 of {dims} dimensions, with a row at least")
    return shape[-2]


def _same(name: str, w: Mx4, dev: torch.device):
    if w.codes.device != dev:
        raise ValueError(f"{name} must be on {dev}")


def mx4_matmul(x, w: Mx4, dtype: torch.dtype | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """x W^T: [T, N] for rows x ([T, K]: float32, bfloat16, or an Mx4) and a matrix w ([N, K])
    (moe_mx4_matmul). The result has x's type (an Mx4: bfloat16) unless `dtype` says otherwise."""
    N = _matrix(w, 2)
    p, s, code, ld, T, dev, own = _product_rows(x, w.K)
    _same("w", w, dev)
    y = _result(out, (T, N), dtype or own, dev)
    _call("moe_mx4_matmul", dev, p, s, code, ld, T, w.codes.data_ptr(), w.scales.data_ptr(), N, w.K, y.data_ptr(),
          _FLOATS[y.dtype])
    return y


def mx4_matmul_backward(dy: torch.Tensor, w: Mx4, dtype: torch.dtype | None = None,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of mx4_matmul for its rows: dy W, [T, K], for dy [T, N] (float32 or bfloat16; the
    result has its type unless `dtype` says otherwise). w is not trained."""
    N = _matrix(w, 2)
    code, ld, T = _rows("dy", dy, N)
    _same("w", w, dy.device)
    dx = _result(out, (T, w.K), dtype or dy.dtype, dy.device)
    _call("moe_mx4_matmul_backward", dy.device, dy.data_ptr(), code, ld, T, w.codes.data_ptr(),
          w.scales.data_ptr(), N, w.K, dx.data_ptr(), _FLOATS[dx.dtype])
    return dx


def _groups(grouping: Grouping, w: Mx4, tokens: int | None, dev: torch.device):
    """(T, k, E, has_shared, A) of a grouping and the experts it is for. Without `tokens` every row of the
    groups counts as a token of its own."""
    E, A, n = grouping.counts.numel() - 1, grouping.perm.numel(), w.codes.shape[0]
    if n not in (E, E + 1) or E < 1 or (grouping.has_shared is not None and grouping.has_shared != (n == E + 1)):
        raise ValueError(f"w holds {n} experts, the grouping is for {E}"
                         + (" and a shared one" if grouping.has_shared else ""))
    _int32("grouping.offsets", grouping.offsets, dev, n + 1)
    shared = n - E
    if tokens is None:
        # one assignment a row; the shared expert's group is one of the groups
        return A, 1, n, 0, A
    if tokens < 0 or (A % tokens if tokens else A) or (tokens and A // tokens - shared < 1):
        raise ValueError(f"the grouping's {A} rows do not belong to {tokens} tokens")
    return tokens, max(1, A // tokens - shared if tokens else 1), E, shared, A


@functools.lru_cache(maxsize=256)
def _bytes(name: str, *sizes: int) -> int:
    """A *_workspace_size call's answer, which depends on the sizes alone."""
    return getattr(lib(), name)(*sizes)


def _workspace(given: torch.Tensor | None, n: int, dev: torch.device):
    """(pointer, bytes, tensor) of the caller's workspace, or of a new one of n bytes."""
    if given is None:
        if not n:
            return None, 0, None
        given = torch.empty(n, dtype=torch.uint8, device=dev)
    else:
        _need_cuda("workspace", given, torch.uint8)
        if given.device != dev:
            raise ValueError(f"workspace must be on {dev}")
    return given.data_ptr(), given.numel(), given


def mx4_experts_matmul(x, w: Mx4, grouping: Grouping, tokens: int | None = None, dtype: torch.dtype | None = None,
                       out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Rows grouped by expert, each times its expert's matrix (moe_mx4_experts_matmul): [A, N] in the
    groups' order. w: [E, N, K], or [E + 1, N, K] with the shared expert last. x ([.., K]: float32,
    bfloat16, or an Mx4) holds the A rows in the groups' order, or, where `tokens` gives their number,
    one row a token. Rows of `out` that are in no group are left as they were."""
    N = _matrix(w, 3)
    p, s, code, ld, R, dev, own = _product_rows(x, w.K)
    _same("w", w, dev)
    T, k, E, shared, A = _groups(grouping, w, tokens, dev)
    if R != T:
        raise ValueError(f"x has {R} rows, expected {T}")
    gather = tokens is not None
    if gather:
        _int32("grouping.perm", grouping.perm, dev, A)
    y = _result(out, (A, N), dtype or own, dev)
    wp, wn, keep = _workspace(workspace, _bytes("moe_mx4_experts_matmul_workspace_size", T, k, shared), dev)
    _call("moe_mx4_experts_matmul", dev, p, s, code, ld, T, k, E, shared, int(gather), grouping.offsets.data_ptr(),
          grouping.perm.data_ptr() if gather else None, w.codes.data_ptr(), w.scales.data_ptr(), N, w.K, y.data_ptr(),
          _FLOATS[y.dtype], wp, wn)
    return y


def mx4_experts_matmul_backward(dy: torch.Tensor, w: Mx4, grouping: Grouping, tokens: int | None = None,
                                dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of mx4_experts_matmul for x: dy [A, N] in the groups' order -> [A, K], or, where
    `tokens` gives their number, [tokens, K], the sum over each token's assignments. w is not trained."""
    N = _matrix(w, 3)
    code, ld, R = _rows("dy", dy, N)
    dev = dy.device
    _same("w", w, dev)
    T, k, E, shared, A = _groups(grouping, w, tokens, dev)
    if R != A:
        raise ValueError(f"dy has {R} rows, expected {A}")
    gather = tokens is not None
    if gather:
        _int32("grouping.slot_of", grouping.slot_of, dev, A)
    dx = _result(out, (T, w.K), dtype or dy.dtype, dev)
    wp, wn, keep = _workspace(
        workspace, _bytes("moe_mx4_experts_matmul_backward_workspace_size", T, k, shared, w.K, int(gather)), dev)
    _call("moe_mx4_experts_matmul_backward", dev, dy.data_ptr(), code, ld, T, k, E, shared, int(gather),
          grouping.offsets.data_ptr(), grouping.slot_of.data_ptr() if gather else None, w.codes.data_ptr(),
          w.scales.data_ptr(), N, w.K, dx.data_ptr(), _FLOATS[dx.dtype], wp, wn)
    return dx


# ---- balance loss ---------------------------------------------------------------------


@dataclass
class BalanceLoss:
    losses: torch.Tensor  # float32 [2]: balance loss, z loss
    counts: torch.Tensor  # int32 [E]: assignments of the kept tokens to each expert
    kept: torch.Tensor    # int32 [1]: how many tokens the mask keeps
    k: int                # experts per token


def _token_mask(mask: torch.Tensor | None, T: int, dev: torch.device):
    if mask is None:
        return None
    _need_cuda("token_mask", mask, (torch.bool, torch.uint8))
    if mask.numel() != T or mask.device != dev:
        raise ValueError(f"token_mask must hold {T} values on {dev}")
    return mask.data_ptr()


def balance_loss(logits: torch.Tensor, idx: torch.Tensor, token_mask: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, out: BalanceLoss | None = None) -> BalanceLoss:
    """Per-expert counts, balance loss and z loss of a routed batch (moe_balance_loss): logits [T, E]
    (float32 or bfloat16), idx int32 [T, k] as route_topk gives it, token_mask bool [T] (False: a token
    that does not count, as padding)."""
    code, ld, T = _rows("logits", logits)
    E = logits.shape[1]
    dev = logits.device
    _int32("idx", idx, dev)
    if idx.dim() != 2 or idx.shape[0] != T:
        raise ValueError(f"idx must be [{T}, k]: got {tuple(idx.shape)}")
    k = idx.shape[1]
    keep = _token_mask(token_mask, T, dev)
    need = _bytes("moe_balance_loss_workspace_size", T, k, E)
    inside = None
    if out is None:  # parts of one tensor, a small workspace (16-byte aligned, as the tensor is) among them
        n = (need + 15) // 16 * 4 if workspace is None and need <= 1 << 16 else 0
        room = torch.empty(n + E + 3, dtype=torch.int32, device=dev)
        scratch, losses, kept, counts = room.split_with_sizes((n, 2, 1, E))
        out = BalanceLoss(losses.view(torch.float32), counts, kept, k)
        if n:
            inside = (room.data_ptr(), 4 * n, room)
    else:
        _need_cuda("out.losses", out.losses, torch.float32)
        _int32("out.counts", out.counts, dev)
        _int32("out.kept", out.kept, dev)
        if out.losses.numel() != 2 or out.counts.numel() != E or out.kept.numel() != 1 or out.losses.device != dev:
            raise ValueError("out does not match the logits")
        out.k = k
    wp, wn, keep_ws = inside or _workspace(workspace, need, dev)
    _call("moe_balance_loss", dev, logits.data_ptr(), code, ld, T, E, k, idx.data_ptr(), keep, out.losses.data_ptr(),
          out.counts.data_ptr(), out.kept.data_ptr(), wp, wn)
    return out


def balance_loss_backward(logits: torch.Tensor, loss: BalanceLoss, d_losses: torch.Tensor,
                          token_mask: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of balance_loss for the logits, [T, E] in their type, from the gradients d_losses
    (float32 [2], on the device) of its two losses; `loss` and `token_mask` as the forward call had them."""
    code, ld, T = _rows("logits", logits)
    E = logits.shape[1]
    dev = logits.device
    _need_cuda("d_losses", d_losses, torch.float32)
    if d_losses.numel() != 2 or d_losses.device != dev:
        raise ValueError(f"d_losses must hold 2 values on {dev}")
    _int32("loss.counts", loss.counts, dev)
    _int32("loss.kept", loss.kept, dev, 1)
    if loss.counts.numel() != E:
        raise ValueError(f"loss is for {loss.counts.numel()} experts, the logits for {E}")
    keep = _token_mask(token_mask, T, dev)
    d = _result(out, (T, E), logits.dtype, dev)
    _call("moe_balance_loss_backward", dev, logits.data_ptr(), code, ld, T, E, loss.k, keep, loss.counts.data_ptr(),
          loss.kept.data_ptr(), d_losses.data_ptr(), d.data_ptr())
    return d


__all__ = ["layer", "layer_static", "profile_begin", "profile_end", "router_logits", "route_topk", "route_group", "group", "Grouping", "Experts", "ffn_q", "lib", "status_string",
           "MoeError", "Q2", "Q3", "F32", "BF16", "FAST", "CHECK_F32", "MAX_E", "LIB_PATH",
           "MX4", "Mx4", "mx4_quantize", "mx4_dequantize", "mx4_matmul", "mx4_matmul_backward",
           "mx4_experts_matmul", "mx4_experts_matmul_backward", "BalanceLoss", "balance_loss",
           "balance_loss_backward"]
