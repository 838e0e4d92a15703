"""Python binding of libmate: argument marshalling only.

Every step of the MATE block runs in the CUDA library (include/mate.h); PyTorch provides device memory
and the current stream.  There is no Python or CPU implementation behind these calls: if libmate.so is
missing, the first call raises ImportError.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import functools
from typing import Dict, Optional

import torch

from . import _lib

__all__ = ["MateBlock", "DitBlock", "dit_weights_to_device", "rms_permute", "rms_unpermute", "review_pool", "ssd_scan_bidir", "ssd_scan_bidir_pd",
           "ssd_scan_bidir_noalloc", "ssd_scan_bidir_backward", "tesa_forward", "tesa_backward", "project_bf16", "device_status",
           "torch_dtype", "weights_to_device", "scan_locality", "KernelTrace",
           "QkConfig", "rope_table", "qk_norm_rope", "qk_norm_rope_backward", "GatedScanConfig", "gated_scan",
           "gated_scan_states", "gated_scan_backward", "quantize_rows", "project_int8"]


def torch_dtype(cfg) -> torch.dtype:
    return torch.bfloat16 if cfg.dtype == "bf16" else torch.float32


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _s(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, dtype: torch.dtype, numel: int, name: str):
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous() or t.numel() != numel:
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor with {numel} elements, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


def weights_to_device(w: Dict, cfg, device="cuda") -> Dict[str, torch.Tensor]:
    """Host weight arrays (numpy / tensors) -> device tensors in the library's dtypes."""
    dt = torch_dtype(cfg)
    out = {}
    for k in ("W_in", "W_out", "W_qkv", "W_o", "W_z"):
        if k in w:   # W_z: the optional gate projection of the full Mamba2 block
            out[k] = torch.as_tensor(w[k]).to(device=device, dtype=dt).contiguous()
    for k in ("dt_bias", "A_log", "D", "dt_bias_b", "A_log_b", "D_b", "conv_w", "conv_b", "norm_w"):
        if k in w:   # optional: the backward-scan parameters, the convolution and the norm weight
            out[k] = torch.as_tensor(w[k]).to(device=device, dtype=torch.float32).contiguous()
    return out


class MateBlock:
    """One MATE block (MA + TE branches) with its weights resident on the GPU and a reusable workspace.
    Weights W_z, conv_w, conv_b and norm_w, given together, make the MA branch's core a full Mamba2 block
    (causal convolution + SiLU on x | B | C, SiLU(z) gate, gated RMSNorm).  The projection matrices are
    packed once here (mate_pack_weights); pack=False makes every forward pack them again instead."""

    def __init__(self, cfg, weights: Dict[str, torch.Tensor], device="cuda", pack: bool = True,
                 workspace: bool = True):
        lib = _lib.load()
        self.cfg = cfg
        ext = [k for k in ("W_z", "conv_w", "conv_b", "norm_w") if k in weights]
        if ext and len(ext) != 4:
            raise ValueError(f"Mamba2 extras: give W_z, conv_w, conv_b and norm_w together, got {ext}")
        self.extras = bool(ext)
        self.ccfg = _lib.make_config(cfg, self.extras)
        _lib.check(lib.mate_check_config(ctypes.byref(self.ccfg)), "mate_check_config")
        self.device = torch.device(device)
        self.dtype = torch_dtype(cfg)
        self.w = weights
        n_in = cfg.nh * cfg.P + 2 * cfg.N + cfg.nh
        _need(weights["W_in"], self.dtype, n_in * cfg.d, "W_in")
        _need(weights["W_out"], self.dtype, cfg.d * cfg.nh * cfg.P, "W_out")
        _need(weights["W_qkv"], self.dtype, 3 * cfg.th * cfg.tp * cfg.d, "W_qkv")
        _need(weights["W_o"], self.dtype, cfg.d * cfg.th * cfg.tp, "W_o")
        for k in ("dt_bias", "A_log", "D"):
            _need(weights[k], torch.float32, cfg.nh, k)
        bwd = [k for k in ("dt_bias_b", "A_log_b", "D_b") if k in weights]
        if bwd and len(bwd) != 3:
            raise ValueError(f"backward-scan parameters: give dt_bias_b, A_log_b and D_b together, got {bwd}")
        for k in bwd:
            _need(weights[k], torch.float32, cfg.nh, k)
        if self.extras:
            nP, Cx = cfg.nh * cfg.P, cfg.nh * cfg.P + 2 * cfg.N
            _need(weights["W_z"], self.dtype, nP * cfg.d, "W_z")
            _need(weights["conv_w"], torch.float32, Cx * 4, "conv_w")
            _need(weights["conv_b"], torch.float32, Cx, "conv_b")
            _need(weights["norm_w"], torch.float32, nP, "norm_w")
        self.cw = _lib.CWeights(*(weights[k].data_ptr() if k in weights else None for k in
                                  ("W_in", "dt_bias", "A_log", "D", "W_out", "W_qkv", "W_o", "dt_bias_b", "A_log_b",
                                   "D_b", "W_z", "conv_w", "conv_b", "norm_w")))
        self.packed = None
        if pack:
            nb = lib.mate_packed_weights_bytes(ctypes.byref(self.ccfg))
            self.packed = torch.empty(nb, dtype=torch.uint8, device=self.device)
            _lib.check(lib.mate_pack_weights(ctypes.byref(self.cw), ctypes.byref(self.ccfg), _p(self.packed), nb,
                                             _s(None)), "mate_pack_weights")
            self.cw.packed = self.packed.data_ptr()
        self.ws_bytes = lib.mate_workspace_bytes(ctypes.byref(self.ccfg))
        self.ws = torch.empty(self.ws_bytes if workspace else 0, dtype=torch.uint8, device=self.device)
        self.ws_host = None
        self.numel = cfg.B * cfg.T * cfg.H * cfg.W * cfg.d

    def forward(self, X: torch.Tensor, layer_idx: int, out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Out = MA(X) + TE(X) for X [B, T, H, W, d] on the GPU (stream-ordered, no synchronisation)."""
        _need(X, self.dtype, self.numel, "X")
        if out is None:
            out = torch.empty_like(X)
        _need(out, self.dtype, self.numel, "out")
        st = _lib.load().mate_forward(_p(X), ctypes.byref(self.cw), int(layer_idx), _p(out), ctypes.byref(self.ccfg),
                                      _p(self.ws), self.ws_bytes, _s(stream))
        _lib.check(st, "mate_forward")
        return out

    def forward_host(self, X_host: torch.Tensor, layer_idx: int, out_host: torch.Tensor,
                     stream: Optional[torch.cuda.Stream] = None, pipelined: bool = False) -> torch.Tensor:
        """mate_forward_host: host (page-locked) input and output, copies inside the call.  pipelined: the copies
        overlap the neighbouring calls' work (mate_forward_host_pipelined); out_host is then complete once the
        stream reaches the end of the next pipelined call or of flush_host()."""
        lib = _lib.load()
        if self.ws_host is None:
            nb = lib.mate_forward_host_workspace_bytes(ctypes.byref(self.ccfg))
            self.ws_host = torch.empty(nb, dtype=torch.uint8, device=self.device)
        for t, nm in ((X_host, "X_host"), (out_host, "out_host")):
            if t.is_cuda or t.dtype != self.dtype or t.numel() != self.numel or not t.is_contiguous():
                raise ValueError(f"{nm}: expected a contiguous host {self.dtype} tensor with {self.numel} elements")
        fn = lib.mate_forward_host_pipelined if pipelined else lib.mate_forward_host
        st = fn(_p(X_host), ctypes.byref(self.cw), int(layer_idx), _p(out_host), ctypes.byref(self.ccfg),
                _p(self.ws_host), self.ws_host.numel(), _s(stream))
        _lib.check(st, "mate_forward_host_pipelined" if pipelined else "mate_forward_host")
        return out_host

    @staticmethod
    def flush_host(stream: Optional[torch.cuda.Stream] = None):
        """mate_forward_host_flush: the stream waits for every pipelined call's output copy."""
        _lib.check(_lib.load().mate_forward_host_flush(_s(stream)), "mate_forward_host_flush")

    @staticmethod
    def last_launch_count() -> int:
        return _lib.load().mate_last_launch_count()


def dit_weights_to_device(w: Dict, cfg, device="cuda") -> Dict[str, torch.Tensor]:
    """Host DiT-block weights (W_ada [6d, dc], W1 [4d, d], W2 [d, 4d], b_ada, b1, b2) -> device tensors in the
    library's dtypes (matrices in the block's dtype, biases fp32)."""
    dt = torch_dtype(cfg)
    out = {k: torch.as_tensor(w[k]).to(device=device, dtype=dt).contiguous() for k in ("W_ada", "W1", "W2")}
    out.update({k: torch.as_tensor(w[k]).to(device=device, dtype=torch.float32).contiguous()
                for k in ("b_ada", "b1", "b2")})
    return out


class DitBlock:
    """A DiT block with the MATE block as its token mixer (mate_dit_block_forward): adaLN-Zero modulation
    from a per-sample conditioning vector c [B, dc], the mixer behind a gated residual, and a gated GELU MLP
    of width 4 d."""

    def __init__(self, cfg, mate_weights: Dict[str, torch.Tensor], dit_weights: Dict[str, torch.Tensor], dc: int,
                 device="cuda"):
        lib = _lib.load()
        self.cfg, self.dc = cfg, int(dc)
        self.mix = MateBlock(cfg, mate_weights, device, workspace=False)
        d = cfg.d
        dt = torch_dtype(cfg)
        _need(dit_weights["W_ada"], dt, 6 * d * self.dc, "W_ada")
        _need(dit_weights["W1"], dt, 4 * d * d, "W1")
        _need(dit_weights["W2"], dt, 4 * d * d, "W2")
        _need(dit_weights["b_ada"], torch.float32, 6 * d, "b_ada")
        _need(dit_weights["b1"], torch.float32, 4 * d, "b1")
        _need(dit_weights["b2"], torch.float32, d, "b2")
        self.w = dit_weights
        self.cw = _lib.CDitWeights(*(dit_weights[k].data_ptr() for k in ("W_ada", "b_ada", "W1", "b1", "W2", "b2")))
        self.ws_bytes = lib.mate_dit_workspace_bytes(ctypes.byref(self.mix.ccfg))
        if self.ws_bytes == 0:
            raise ValueError("mate_dit_workspace_bytes: configuration not supported by the DiT block")
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)

    def forward(self, X: torch.Tensor, c: torch.Tensor, layer_idx: int, out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        _need(X, self.mix.dtype, self.mix.numel, "X")
        _need(c, torch.float32, self.cfg.B * self.dc, "c")
        if out is None:
            out = torch.empty_like(X)
        _need(out, self.mix.dtype, self.mix.numel, "out")
        st = _lib.load().mate_dit_block_forward(_p(X), _p(c), self.dc, ctypes.byref(self.cw),
                                                ctypes.byref(self.mix.cw), int(layer_idx), _p(out),
                                                ctypes.byref(self.mix.ccfg), _p(self.ws), self.ws_bytes, _s(stream))
        _lib.check(st, "mate_dit_block_forward")
        return out


def _cfg(cfg):
    c = _lib.make_config(cfg)
    return c


def rms_permute(X: torch.Tensor, order: int, cfg, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    n = cfg.T * cfg.H * cfg.W
    if out is None:
        out = torch.empty((cfg.B, n, cfg.d), dtype=X.dtype, device=X.device)
    c = _cfg(cfg)
    _lib.check(_lib.load().rms_permute(_p(X), _p(out), int(order), ctypes.byref(c), _s(stream)), "rms_permute")
    return out


def rms_unpermute(Xp: torch.Tensor, order: int, cfg, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty((cfg.B, cfg.T, cfg.H, cfg.W, cfg.d), dtype=Xp.dtype, device=Xp.device)
    c = _cfg(cfg)
    _lib.check(_lib.load().rms_unpermute(_p(Xp), _p(out), int(order), ctypes.byref(c), _s(stream)), "rms_unpermute")
    return out


def review_pool(X: torch.Tensor, order: int, cfg, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty((cfg.B, cfg.R, cfg.d), dtype=X.dtype, device=X.device)
    c = _cfg(cfg)
    _lib.check(_lib.load().review_pool(_p(X), _p(out), int(order), ctypes.byref(c), _s(stream)), "review_pool")
    return out


def ssd_scan_bidir(x, Bm, Cm, dt, dt_bias, A_log, D, prefix_len: int, cfg, out=None, ws=None, stream=None):
    """Bidirectional selective scan over [prefix; video] rows: x [B, L, nh*P], Bm/Cm [B, L, N], dt [B, L, nh]
    (fp32, before softplus).  Returns y [B, T*H*W, nh*P] for the video rows."""
    lib = _lib.load()
    c = _cfg(cfg)
    n = cfg.T * cfg.H * cfg.W
    if out is None:
        out = torch.empty((cfg.B, n, cfg.nh * cfg.P), dtype=x.dtype, device=x.device)
    nb = lib.mate_ssd_workspace_bytes(ctypes.byref(c), int(prefix_len))
    if ws is None or ws.numel() < nb:
        ws = torch.empty(nb, dtype=torch.uint8, device=x.device)
    st = lib.ssd_scan_bidir(_p(x), _p(Bm), _p(Cm), _p(dt), _p(dt_bias), _p(A_log), _p(D), int(prefix_len), _p(out),
                            ctypes.byref(c), _p(ws), ws.numel(), _s(stream))
    _lib.check(st, "ssd_scan_bidir")
    return out


def ssd_scan_bidir_pd(x, Bm, Cm, dt, dt_bias, A_log, D, dt_bias_b, A_log_b, D_b, prefix_len: int, cfg, out=None,
                      ws=None, stream=None):
    """ssd_scan_bidir with the backward scan's own step-size bias, A_log and D ([nh] fp32 each)."""
    lib = _lib.load()
    c = _cfg(cfg)
    n = cfg.T * cfg.H * cfg.W
    if out is None:
        out = torch.empty((cfg.B, n, cfg.nh * cfg.P), dtype=x.dtype, device=x.device)
    nb = lib.mate_ssd_pd_workspace_bytes(ctypes.byref(c), int(prefix_len))
    if ws is None or ws.numel() < nb:
        ws = torch.empty(nb, dtype=torch.uint8, device=x.device)
    st = lib.ssd_scan_bidir_pd(_p(x), _p(Bm), _p(Cm), _p(dt), _p(dt_bias), _p(A_log), _p(D), _p(dt_bias_b),
                               _p(A_log_b), _p(D_b), int(prefix_len), _p(out), ctypes.byref(c), _p(ws), ws.numel(),
                               _s(stream))
    _lib.check(st, "ssd_scan_bidir_pd")
    return out


def ssd_scan_bidir_backward(x, Bm, Cm, dt, dt_bias, A_log, D, dy, prefix_len: int, cfg, ws=None, stream=None):
    """Gradients of ssd_scan_bidir (fp32 blocks) given the video rows' output gradient dy [B, T*H*W, nh*P]:
    a dict with dx, dB, dC (layouts of x, Bm, Cm), ddt (layout of dt) and ddt_bias, dA_log, dD [nh]."""
    lib = _lib.load()
    c = _cfg(cfg)
    L = cfg.n + int(prefix_len)
    for t, nm, numel in ((x, "x", cfg.B * L * cfg.nh * cfg.P), (Bm, "Bm", cfg.B * L * cfg.N),
                         (Cm, "Cm", cfg.B * L * cfg.N), (dt, "dt", cfg.B * L * cfg.nh),
                         (dy, "dy", cfg.B * cfg.n * cfg.nh * cfg.P), (dt_bias, "dt_bias", cfg.nh),
                         (A_log, "A_log", cfg.nh), (D, "D", cfg.nh)):
        _need(t, torch.float32, numel, nm)
    f32 = dict(dtype=torch.float32, device=x.device)
    g = dict(dx=torch.empty_like(x), dB=torch.empty_like(Bm), dC=torch.empty_like(Cm), ddt=torch.empty_like(dt),
             ddt_bias=torch.empty(cfg.nh, **f32), dA_log=torch.empty(cfg.nh, **f32), dD=torch.empty(cfg.nh, **f32))
    nb = lib.mate_ssd_backward_workspace_bytes(ctypes.byref(c), int(prefix_len))
    if ws is None or ws.numel() < nb:
        ws = torch.empty(nb, dtype=torch.uint8, device=x.device)
    st = lib.ssd_scan_bidir_backward(_p(x), _p(Bm), _p(Cm), _p(dt), _p(dt_bias), _p(A_log), _p(D), int(prefix_len),
                                     _p(dy), _p(g["dx"]), _p(g["dB"]), _p(g["dC"]), _p(g["ddt"]), _p(g["ddt_bias"]),
                                     _p(g["dA_log"]), _p(g["dD"]), ctypes.byref(c), _p(ws), ws.numel(), _s(stream))
    _lib.check(st, "ssd_scan_bidir_backward")
    return g


def ssd_scan_bidir_noalloc(x, Bm, Cm, dt, dt_bias, A_log, D, prefix_len: int, cfg, out, stream=None):
    """ssd_scan_bidir on the library's fixed device scratch, for callers that may not allocate device memory.
    Nothing is allocated here either: the caller passes the output `out` [B, T*H*W, nh*P]."""
    c = _cfg(cfg)
    st = _lib.load().ssd_scan_bidir_noalloc(_p(x), _p(Bm), _p(Cm), _p(dt), _p(dt_bias), _p(A_log), _p(D),
                                            int(prefix_len), _p(out), ctypes.byref(c), _s(stream))
    _lib.check(st, "ssd_scan_bidir_noalloc")
    return out


def tesa_forward(qkv: torch.Tensor, shifted: bool, cfg, out: Optional[torch.Tensor] = None, stream=None):
    if out is None:
        out = torch.empty((cfg.B, cfg.T, cfg.H, cfg.W, cfg.th * cfg.tp), dtype=qkv.dtype, device=qkv.device)
    c = _cfg(cfg)
    _lib.check(_lib.load().tesa_forward(_p(qkv), _p(out), int(bool(shifted)), ctypes.byref(c), _s(stream)),
               "tesa_forward")
    return out


def tesa_backward(qkv: torch.Tensor, O: torch.Tensor, dO: torch.Tensor, shifted: bool, cfg, out=None, ws=None,
                  stream=None) -> torch.Tensor:
    """Gradient of tesa_forward with respect to qkv [B, T, H, W, 3 th tp], given its output O and the output
    gradient dO [B, T, H, W, th tp] (bf16 blocks)."""
    lib = _lib.load()
    c = _cfg(cfg)
    a = cfg.th * cfg.tp
    n = cfg.B * cfg.T * cfg.H * cfg.W
    _need(qkv, torch.bfloat16, n * 3 * a, "qkv")
    _need(O, torch.bfloat16, n * a, "O")
    _need(dO, torch.bfloat16, n * a, "dO")
    if out is None:
        out = torch.empty_like(qkv)
    nb = lib.mate_tesa_backward_workspace_bytes(ctypes.byref(c))
    if ws is None or ws.numel() < nb:
        ws = torch.empty(nb, dtype=torch.uint8, device=qkv.device)
    _lib.check(lib.tesa_backward(_p(qkv), _p(O), _p(dO), _p(out), int(bool(shifted)), ctypes.byref(c), _p(ws),
                                 ws.numel(), _s(stream)), "tesa_backward")
    return out


def project_bf16(A: torch.Tensor, Wt: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None):
    """C = A W^T on tensor cores: A [M, K] bf16, Wt [N, K] bf16 -> C [M, N] bf16."""
    M, K = A.shape
    N = Wt.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    st = _lib.load().mate_project_bf16(_p(A), A.stride(0), M, K, _p(Wt), Wt.stride(0), N, _p(out), out.stride(0),
                                       _s(stream))
    _lib.check(st, "mate_project_bf16")
    return out


# ------------------------------------------------------------------------------ operators beside the block
# They take strided rows, tensors on any CUDA device (which need not be the current one) and an optional stream
# of that device; what they allocate belongs to the stream they run on.  Devices go by their index here, and streams
# by their raw handle: a call of few rows takes about as long on the host as on the GPU.
_HERE = contextlib.nullcontext()


def _on(index: int, stream: Optional[torch.cuda.Stream]):
    """Context in which device `index` and `stream` are current (nothing to do where they already are)."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"stream on {stream.device}, tensors on cuda:{index}")
        return torch.cuda.stream(stream)
    return _HERE if index == torch.cuda.current_device() else torch.cuda.device(index)


def _raw_stream(index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(index)


def _device_index(device) -> int:
    """Index of a CUDA device given as a name, an index or a torch.device."""
    d = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
    if d.type != "cuda":
        raise ValueError(f"device {d}: a CUDA device is needed")
    return torch.cuda.current_device() if d.index is None else d.index


def _rows(t: torch.Tensor, dtype: torch.dtype, rows: int, cols: int, index: int, name: str) -> int:
    """Row stride in elements of a tensor that holds `rows` evenly strided rows of `cols` elements (of one row: any
    stride that the library takes) on device `index`."""
    ok = t.dtype is dtype and t.get_device() == index and index >= 0 and t.numel() == rows * cols and \
        t.dim() >= 1 and t.shape[-1] == cols
    ld = cols if rows != 1 else (cols + 15) // 16 * 16
    if ok and t.is_contiguous():
        return ld
    ok = ok and (t.stride(-1) == 1 or cols == 1)
    if ok:
        step = None
        for size, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
            if size == 1:
                continue
            if step is None:
                ld = step = st
            ok = ok and st == step
            step *= size
    if not ok:
        raise ValueError(f"{name}: expected {rows} evenly strided rows of {cols} {dtype} elements on "
                         f"{'a CUDA device' if index < 0 else f'cuda:{index}'}, got {t.dtype} {tuple(t.shape)} with "
                         f"strides {t.stride()} on {t.device}")
    return ld


def _flat(t: Optional[torch.Tensor], dtype: torch.dtype, numel: int, index: int, name: str) -> Optional[int]:
    """Address of an optional contiguous tensor on device `index`."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != index or t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor with {numel} elements on cuda:{index}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _check(status: int, where: str, **tensors: Optional[torch.Tensor]) -> None:
    """check, naming the tensors whose start or rows the library may have refused."""
    if status == _lib.MATE_ERR_ARG:
        for name, t in tensors.items():
            step = t.stride(-2) * t.element_size() if t is not None and t.dim() > 1 else 0
            if t is not None and (t.data_ptr() % 16 or step % 16):
                where += f", {name}: starts {t.data_ptr() % 16} bytes behind a multiple of 16, rows {step} bytes apart"
    _lib.check(status, where)


def _workspace(ws: Optional[torch.Tensor], nbytes: int, like: torch.Tensor) -> Optional[torch.Tensor]:
    """The caller's workspace (uint8, checked), else a new one of the current stream; None where none is needed."""
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device) if nbytes else None
    if ws.dtype is not torch.uint8 or not ws.is_contiguous() or ws.device != like.device or ws.numel() < nbytes:
        raise ValueError(f"ws: expected at least {nbytes} contiguous uint8 elements on {like.device}, got {ws.dtype} "
                         f"{tuple(ws.shape)} on {ws.device}")
    return ws


def _int(value, name: str, bits: int = 32) -> int:
    """The value as an integer of the C interface (one that does not fit is refused, not cut)."""
    v = int(value)
    if not -(1 << bits - 1) <= v < (1 << bits - 1):
        raise ValueError(f"{name} = {v} does not fit a {bits}-bit int")
    return v


def _ints(obj, names):
    return [_int(getattr(obj, k), k) for k in names]


def _keep(obj, **values):
    """Derived values of a frozen configuration."""
    for k, v in values.items():
        object.__setattr__(obj, k, v)


class _Config:
    """Copies and pickles go by the fields: the C structure and the pointer to it are made anew."""

    def __reduce__(self):
        return type(self), tuple(getattr(self, f.name) for f in dataclasses.fields(self))


@dataclasses.dataclass(frozen=True)
class QkConfig(_Config):
    """Shape of qk_norm_rope's rows: B samples of T x H x W tokens, hq query, hk key and hv value heads of tp channels
    (tesa_forward's rows: all three th); rt / rh / rw of a head's first channels turn with the token's t / h / w
    position, in pairs of "adjacent" channels or of the "halves" of each axis' channels."""

    B: int
    T: int
    H: int
    W: int
    hq: int
    hk: int
    hv: int
    tp: int
    rt: int = 0
    rh: int = 0
    rw: int = 0
    pairing: str = "adjacent"
    eps: float = 1e-6
    dtype: str = "bf16"

    def __post_init__(self):
        if self.pairing not in ("adjacent", "halves") or self.dtype not in ("bf16", "f32"):
            raise ValueError(f"pairing {self.pairing!r} (adjacent, halves), dtype {self.dtype!r} (bf16, f32)")
        c = _lib.CQkConfig(*_ints(self, ("B", "T", "H", "W", "hq", "hk", "hv", "tp", "rt", "rh", "rw")),
                           int(self.pairing == "halves"), self.eps,
                           _lib.MATE_BF16 if self.dtype == "bf16" else _lib.MATE_F32)
        _keep(self, ccfg=c, ref=ctypes.byref(c), tdtype=torch_dtype(self), rows=self.B * self.T * self.H * self.W,
              width=(self.hq + self.hk + self.hv) * self.tp)

    @functools.cached_property
    def backward_workspace_bytes(self) -> int:
        return _lib.load().mate_qk_norm_rope_backward_workspace_bytes(self.ref)


def rope_table(count: int, dims: int, start: int = 0, theta: float = 10000.0, device="cuda",
               stream=None) -> torch.Tensor:
    """[count, dims / 2, 2] fp32: (cos, sin) of (start + p) theta^(-2 i / dims), the angle in 64 bits (made once)."""
    count, dims, start = _int(count, "count"), _int(dims, "dims"), _int(start, "start", 64)
    index = _device_index(device)
    with _on(index, stream):
        tab = torch.empty((max(count, 0), max(dims, 0) // 2, 2), dtype=torch.float32, device=f"cuda:{index}")
        st = 0 if dims == 0 else _lib.load().mate_rope_table(tab.data_ptr(), start, count, dims, float(theta),
                                                             _raw_stream(index))
    _lib.check(st, "mate_rope_table")
    return tab


def _qk_tables(tables, cfg: QkConfig, index: int):
    if len(tables) != 3:
        raise ValueError(f"tables: expected the t, h and w tables, got {len(tables)}")
    t, h, w = tables
    return (_flat(t, torch.float32, cfg.T * cfg.rt, index, "t table") if cfg.rt else None,
            _flat(h, torch.float32, cfg.H * cfg.rh, index, "h table") if cfg.rh else None,
            _flat(w, torch.float32, cfg.W * cfg.rw, index, "w table") if cfg.rw else None)


def qk_norm_rope(qkv: torch.Tensor, wq: Optional[torch.Tensor], wk: Optional[torch.Tensor], tables, cfg: QkConfig,
                 out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """RMS norm of every query and key head (weights wq, wk [tp] fp32 or None) and rotation by the token's position,
    on packed q | k | v rows; value columns pass.  tables: the (t, h, w) tables of rope_table (None for an axis with no
    channels).  out=qkv works in place."""
    dt, index = cfg.tdtype, qkv.get_device()
    ldi = _rows(qkv, dt, cfg.rows, cfg.width, index, "qkv")
    tabs = _qk_tables(tables, cfg, index)
    with _on(index, stream):
        if out is None:
            out, ldo = torch.empty_like(qkv, memory_format=torch.contiguous_format), cfg.width
        else:
            ldo = _rows(out, dt, cfg.rows, cfg.width, index, "out") if out is not qkv else ldi
        st = _lib.load().mate_qk_norm_rope(
            qkv.data_ptr(), ldi, _flat(wq, torch.float32, cfg.tp, index, "wq"),
            _flat(wk, torch.float32, cfg.tp, index, "wk"), *tabs, out.data_ptr(), ldo, cfg.ref, _raw_stream(index))
    if st:
        _check(st, "mate_qk_norm_rope", qkv=qkv, wq=wq, wk=wk, out=out)
    return out


def qk_norm_rope_backward(qkv: torch.Tensor, wq: Optional[torch.Tensor], wk: Optional[torch.Tensor], tables,
                          dout: torch.Tensor, cfg: QkConfig, dqkv: Optional[torch.Tensor] = None, ws=None,
                          stream=None) -> Dict[str, torch.Tensor]:
    """Gradients of qk_norm_rope from its input and the output gradient: dqkv (may be dout or qkv itself), dwq and dwk
    [tp] fp32 (summed over rows and heads in a fixed order)."""
    dt, index = cfg.tdtype, qkv.get_device()
    ldi = _rows(qkv, dt, cfg.rows, cfg.width, index, "qkv")
    ldg = _rows(dout, dt, cfg.rows, cfg.width, index, "dout")
    tabs = _qk_tables(tables, cfg, index)
    with _on(index, stream):
        if dqkv is None:
            dqkv = torch.empty_like(qkv, memory_format=torch.contiguous_format)
        ldd = _rows(dqkv, dt, cfg.rows, cfg.width, index, "dqkv")
        dwq = torch.empty(cfg.tp, dtype=torch.float32, device=qkv.device)
        dwk = torch.empty(cfg.tp, dtype=torch.float32, device=qkv.device)
        ws = _workspace(ws, cfg.backward_workspace_bytes, qkv)
        if ws is None:
            raise ValueError(f"qk_norm_rope_backward: {cfg} is not supported")
        st = _lib.load().mate_qk_norm_rope_backward(
            qkv.data_ptr(), ldi, _flat(wq, torch.float32, cfg.tp, index, "wq"),
            _flat(wk, torch.float32, cfg.tp, index, "wk"), *tabs, dout.data_ptr(), ldg, dqkv.data_ptr(), ldd,
            dwq.data_ptr(), dwk.data_ptr(), cfg.ref, ws.data_ptr(), ws.numel(), _raw_stream(index))
    if st:
        _check(st, "mate_qk_norm_rope_backward", qkv=qkv, wq=wq, wk=wk, dout=dout, dqkv=dqkv)
    return dict(dqkv=dqkv, dwq=dwq, dwk=dwk)


@dataclasses.dataclass(frozen=True)
class GatedScanConfig(_Config):
    """Shape of gated_scan: B samples of T x H x W tokens with D channels, walked along scan order `order` (as
    rms_permute), from its last position back if `reverse`."""

    B: int
    T: int
    H: int
    W: int
    D: int
    order: int = 0
    reverse: bool = False
    dtype: str = "bf16"

    def __post_init__(self):
        if self.dtype not in ("bf16", "f32"):
            raise ValueError(f"dtype {self.dtype!r} (bf16, f32)")
        c = _lib.CGatedScanConfig(*_ints(self, ("B", "T", "H", "W", "D", "order")), int(bool(self.reverse)),
                                  _lib.MATE_BF16 if self.dtype == "bf16" else _lib.MATE_F32)
        _keep(self, ccfg=c, ref=ctypes.byref(c), tdtype=torch_dtype(self), rows=self.B * self.T * self.H * self.W)

    @functools.cached_property
    def workspace_bytes(self) -> int:
        return _lib.load().mate_gated_scan_workspace_bytes(self.ref)

    @functools.cached_property
    def backward_workspace_bytes(self) -> int:
        return _lib.load().mate_gated_scan_backward_workspace_bytes(self.ref)

    @functools.cached_property
    def states_numel(self) -> int:
        return _lib.load().mate_gated_scan_states_bytes(self.ref) // 4


def gated_scan_states(cfg: GatedScanConfig, device="cuda", stream=None) -> torch.Tensor:
    """Buffer (fp32) for the states that gated_scan leaves for gated_scan_backward."""
    index = _device_index(device)
    if cfg.states_numel == 0:
        raise ValueError(f"gated_scan_states: {cfg} is not supported")
    with _on(index, stream):
        return torch.empty(cfg.states_numel, dtype=torch.float32, device=f"cuda:{index}")


def gated_scan(x: torch.Tensor, g: torch.Tensor, cfg: GatedScanConfig, bias: Optional[torch.Tensor] = None,
               h0: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
               h_last: Optional[torch.Tensor] = None, states: Optional[torch.Tensor] = None, ws=None, stream=None):
    """h_t = a_t h_{t-1} + (1 - a_t) x_t with a = sigmoid(g + bias), along the grid's scan order: (y, h_last).
    x, g: rows of D channels in grid order (strided rows allowed); bias [D], h0 and h_last [B, D] fp32.
    states (gated_scan_states): filled for gated_scan_backward."""
    dt, f32, index, rows, D = cfg.tdtype, torch.float32, x.get_device(), cfg.rows, cfg.D
    ldx = _rows(x, dt, rows, D, index, "x")
    ldg = _rows(g, dt, rows, D, index, "g")
    with _on(index, stream):
        if y is None:
            y, ldy = torch.empty_like(x, memory_format=torch.contiguous_format), D
        else:
            ldy = _rows(y, dt, rows, D, index, "y")
        if h_last is None:
            h_last = torch.empty((cfg.B, D), dtype=f32, device=x.device)
        ws = _workspace(ws, cfg.workspace_bytes, x)
        st = _lib.load().mate_gated_scan(
            x.data_ptr(), ldx, g.data_ptr(), ldg, _flat(bias, f32, D, index, "bias"),
            _flat(h0, f32, cfg.B * D, index, "h0"), y.data_ptr(), ldy, _flat(h_last, f32, cfg.B * D, index, "h_last"),
            None if states is None else _flat(states, f32, cfg.states_numel, index, "states"), cfg.ref,
            None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), _raw_stream(index))
    if st:
        _check(st, "mate_gated_scan", x=x, g=g, bias=bias, h0=h0, y=y, h_last=h_last, states=states)
    return y, h_last


def gated_scan_backward(x: torch.Tensor, g: torch.Tensor, states: torch.Tensor, dy: torch.Tensor, cfg: GatedScanConfig,
                        bias: Optional[torch.Tensor] = None, dh_last: Optional[torch.Tensor] = None,
                        dx: Optional[torch.Tensor] = None, dg: Optional[torch.Tensor] = None, ws=None,
                        stream=None) -> Dict[str, torch.Tensor]:
    """Gradients of gated_scan from its inputs, the states it left and the gradients dy of y and dh_last of h_last
    (None: zero): dx, dg, dh0 [B, D] and, with a bias, dbias [D]."""
    dt, f32, index, rows, D = cfg.tdtype, torch.float32, x.get_device(), cfg.rows, cfg.D
    ldx = _rows(x, dt, rows, D, index, "x")
    ldg = _rows(g, dt, rows, D, index, "g")
    lddy = _rows(dy, dt, rows, D, index, "dy")
    with _on(index, stream):
        if dx is None:
            dx = torch.empty_like(x, memory_format=torch.contiguous_format)
        if dg is None:
            dg = torch.empty_like(g, memory_format=torch.contiguous_format)
        grads = dict(dx=dx, dg=dg, dh0=torch.empty((cfg.B, D), dtype=f32, device=x.device))
        dbias = None
        if bias is not None:
            dbias = grads["dbias"] = torch.empty(D, dtype=f32, device=x.device)
        ws = _workspace(ws, cfg.backward_workspace_bytes, x)
        if ws is None:
            raise ValueError(f"gated_scan_backward: {cfg} is not supported")
        st = _lib.load().mate_gated_scan_backward(
            x.data_ptr(), ldx, g.data_ptr(), ldg, _flat(bias, f32, D, index, "bias"),
            _flat(states, f32, cfg.states_numel, index, "states"), dy.data_ptr(), lddy,
            _flat(dh_last, f32, cfg.B * D, index, "dh_last"), dx.data_ptr(), _rows(dx, dt, rows, D, index, "dx"),
            dg.data_ptr(), _rows(dg, dt, rows, D, index, "dg"), None if dbias is None else dbias.data_ptr(),
            grads["dh0"].data_ptr(), cfg.ref, ws.data_ptr(), ws.numel(), _raw_stream(index))
    if st:
        _check(st, "mate_gated_scan_backward", x=x, g=g, states=states, dy=dy, bias=bias, dh_last=dh_last, dx=dx, dg=dg)
    return grads


def _mate_dtype(dtype: torch.dtype, name: str) -> int:
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{name}: expected torch.bfloat16 or torch.float32, got {dtype}")
    return _lib.MATE_BF16 if dtype == torch.bfloat16 else _lib.MATE_F32


def quantize_rows(x: torch.Tensor, q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None, stream=None):
    """x [M, K] bf16 or fp32 (strided rows allowed) -> (q [M, K] int8, scale [M] fp32): scale = max|x| / 127 of the row,
    q = x / scale to the nearest integer, ties to even.  A new q has its rows padded to a multiple of 16 bytes."""
    if x.dim() != 2:
        raise ValueError(f"x: expected [M, K], got {tuple(x.shape)}")
    (M, K), index, code = x.shape, x.get_device(), _mate_dtype(x.dtype, "x")
    _int(K, "K")
    ldx = _rows(x, x.dtype, M, K, index, "x")
    with _on(index, stream):
        if q is None:
            ldq = (K + 15) // 16 * 16
            q = torch.empty((M, ldq), dtype=torch.int8, device=x.device)
            q = q if ldq == K else q[:, :K]
        else:
            ldq = _rows(q, torch.int8, M, K, index, "q")
        if scale is None:
            scale = torch.empty(M, dtype=torch.float32, device=x.device)
        st = _lib.load().mate_quantize_rows(x.data_ptr(), ldx, M, K, code, q.data_ptr(), ldq,
                                            _flat(scale, torch.float32, M, index, "scale"), _raw_stream(index)) if M else 0
    if st:
        _check(st, "mate_quantize_rows", x=x, q=q, scale=scale)
    return q, scale


def project_int8(A: torch.Tensor, a_scale: torch.Tensor, Wt: torch.Tensor, w_scale: torch.Tensor,
                 bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """C = (A W^T) a_scale[row] w_scale[column] + bias on tensor cores: A [M, K] and Wt [N, K] int8 (rows on 16 bytes),
    a_scale [M], w_scale [N], bias [N] fp32 -> C [M, N] bf16 or fp32.  The integer sums are exact."""
    if A.dim() != 2 or Wt.dim() != 2:
        raise ValueError(f"A and Wt: expected [M, K] and [N, K], got {tuple(A.shape)} and {tuple(Wt.shape)}")
    (M, K), N, index, f32 = A.shape, Wt.shape[0], A.get_device(), torch.float32
    _int(K, "K")
    _int(N, "N")
    lda = _rows(A, torch.int8, M, K, index, "A")
    ldw = _rows(Wt, torch.int8, N, K, index, "Wt")
    with _on(index, stream):
        if out is None:
            code, out, ldc = _mate_dtype(out_dtype, "out_dtype"), torch.empty((M, N), dtype=out_dtype, device=A.device), N
        else:
            code, ldc = _mate_dtype(out.dtype, "out"), _rows(out, out.dtype, M, N, index, "out")
        st = _lib.load().mate_project_int8(
            A.data_ptr(), lda, _flat(a_scale, f32, M, index, "a_scale"), M, K, Wt.data_ptr(), ldw,
            _flat(w_scale, f32, N, index, "w_scale"), N, _flat(bias, f32, N, index, "bias"), out.data_ptr(), ldc, code,
            _raw_stream(index)) if M else 0
    if st:
        _check(st, "mate_project_int8", A=A, a_scale=a_scale, Wt=Wt, w_scale=w_scale, bias=bias, out=out)
    return out


def device_status(stream=None) -> int:
    """Synchronise and read/clear the device status word (1 = a bounded wait ran out)."""
    flags = ctypes.c_uint(0)
    _lib.load().mate_device_status(_s(stream), ctypes.byref(flags))
    return int(flags.value)


class KernelTrace:
    """Per-launch device times of this library's kernels between start() and stop() (CUDA events around
    each launch, recorded by the library).  read() -> list of (kernel name, ms) in launch order."""

    def __init__(self, capacity: int):
        self.capacity = int(capacity)

    def start(self):
        _lib.check(_lib.load().mate_trace_start(self.capacity), "mate_trace_start")
        return self

    def stop(self):
        _lib.check(_lib.load().mate_trace_stop(), "mate_trace_stop")

    def read(self):
        lib = _lib.load()
        recs = (_lib.CTraceRecord * max(self.capacity, 1))()
        n = lib.mate_trace_read(recs, self.capacity)
        if n < 0:
            raise _lib.MateError(_lib.MATE_ERR_CUDA, "mate_trace_read")
        return [(lib.mate_kernel_name(recs[r].kernel).decode(), float(recs[r].ms)) for r in range(n)]


LOCALITY_MAPS = ("rms_order0", "rms_order1", "rms_order2", "rms_order3", "zigzag", "hilbert", "rms_rotation")


def scan_locality(T: int, H: int, W: int, kind: int, stream=None):
    """(sum of sequence distances, number of grid-adjacent pairs, largest distance) of index map `kind`
    over a T x H x W grid, computed on the GPU (see mate_scan_locality)."""
    out = torch.zeros(3, dtype=torch.int64, device="cuda")
    _lib.check(_lib.load().mate_scan_locality(int(T), int(H), int(W), int(kind), _p(out), _s(stream)),
               "mate_scan_locality")
    s, n, m = (int(v) for v in out.cpu().tolist())
    return s, n, m
