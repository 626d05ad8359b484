"""Python binding of ``libmoe.so`` — a DeepSeek-V4-Flash MoE layer for MI355X.

Argument marshalling only: every step of the layer runs in the HIP kernels of
``csrc/`` behind the C ABI of ``include/moe.h``. PyTorch provides device
memory and the current stream. There is no CPU fallback: if the library is
not built, or a call fails, an exception is raised.

Entry points (same names as the C ABI): ``route``, ``hash_route``,
``permute``, ``expert_ffn``, ``forward``; plus ``workspace_size``,
``Workspace`` and ``DeviceLayer`` (device copies of one layer's parameters).
Around the layer: ``quantize_mxfp4`` / ``dequantize_mxfp4`` (its weight
format), ``linear_mxfp4`` / ``linear_mxfp4_dx`` (plain products with MXFP4
weights) and ``gated_ffn`` / ``gated_ffn_backward`` (the expert's block with
bf16 weights, and its gradients).
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_EWORKSPACE, MOE_EHIP = 0, -1, -2, -3, -4
KERNELS = {"router": 1, "permute": 2, "routed_w13": 3, "routed_w2": 4, "shared_w13": 5, "shared_w2": 6,
           "combine": 7}


class MoEError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


class MoeLayerWeights(ctypes.Structure):
    """Mirror of ``moe_layer_weights`` (device pointers of one layer)."""
    _fields_ = [("gate_w", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("logit_offset", ctypes.c_void_p),
                ("tid2eid", ctypes.c_void_p), ("V", ctypes.c_int32), ("w13_codes", ctypes.c_void_p),
                ("w13_scales", ctypes.c_void_p), ("w2_codes", ctypes.c_void_p), ("w2_scales", ctypes.c_void_p),
                ("sh_w13", ctypes.c_void_p), ("sh_w13_scale", ctypes.c_void_p), ("sh_w2", ctypes.c_void_p),
                ("sh_w2_scale", ctypes.c_void_p)]


class MoeConfig(ctypes.Structure):
    """Mirror of ``moe_config`` (names of the checkpoint's config.json)."""
    _fields_ = [("hidden_size", ctypes.c_int32), ("n_routed_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("moe_intermediate", ctypes.c_int32),
                ("routed_scaling_factor", ctypes.c_float), ("swiglu_limit", ctypes.c_float),
                ("norm_topk_prob", ctypes.c_int32)]


def config(hidden_size=4096, n_routed_experts=256, top_k=6, moe_intermediate=2048,
           routed_scaling_factor=1.5, swiglu_limit=10.0, norm_topk_prob=1) -> MoeConfig:
    return MoeConfig(hidden_size, n_routed_experts, top_k, moe_intermediate, routed_scaling_factor,
                     swiglu_limit, norm_topk_prob)


def config_of(wl) -> MoeConfig:
    """Config of a workload description with fields H, E, k, I (e.g. ``synth.Workload``)."""
    return config(wl.H, wl.E, wl.k, wl.I, wl.routed_scaling_factor, wl.swiglu_limit)


_lib = None
_VP, _I32, _I64, _SZ, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_CFGP = ctypes.POINTER(MoeConfig)

_SIGNATURES = {
    "moe_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "moe_version": ([], ctypes.c_char_p),
    "moe_workspace_size": ([_CFGP, _I32], _SZ),
    "moe_workspace_init": ([_VP, _SZ, _VP], ctypes.c_int),
    "moe_route": ([_CFGP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_hash_route": ([_CFGP, _I32, _VP, _VP, _VP, _I32, _VP, _VP, _VP, _VP], ctypes.c_int),
    "moe_permute": ([_CFGP, _I32, _VP, _VP, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_expert_ffn": ([_CFGP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
                       ctypes.c_int),
    "moe_set_kernel_events": ([_I32, _VP, _VP], ctypes.c_int),
    "moe_device_flags": ([ctypes.POINTER(ctypes.c_uint32), _I32, _VP], ctypes.c_int),
    "moe_read_probe": ([_VP, _SZ, _I32, _VP, _VP], ctypes.c_int),
    "moe_set_option": ([_I32, _I32], ctypes.c_int),
    "moe_get_option": ([_I32], ctypes.c_int),
    "moe_forward_schedule": ([_CFGP, _I32, _I32], ctypes.c_int),
    "moe_noalloc_max_bytes": ([], _SZ),
    "moe_linear_workspace_size": ([_I32, _I32, _I32, _I32], _SZ),
    "moe_linear_w8a16": ([_I32, _I32, _I32, _I32, _VP, _VP, _VP, _VP, _I32, _VP, _SZ, _VP], ctypes.c_int),
    "moe_mxfp4_quantize": ([_I64, _I32, _I32, _VP, _I64, _VP, _VP, _VP], ctypes.c_int),
    "moe_mxfp4_dequantize": ([_I64, _I32, _VP, _VP, _I32, _VP, _VP], ctypes.c_int),
    "moe_linear_mxfp4_workspace_size": ([_I32, _I32, _I32, _I32], _SZ),
    "moe_linear_mxfp4": ([_I32, _I32, _I32, _VP, _VP, _VP, _I32, _VP, _I32, _VP, _SZ, _VP], ctypes.c_int),
    "moe_linear_mxfp4_dx_workspace_size": ([_I32, _I32, _I32], _SZ),
    "moe_linear_mxfp4_dx": ([_I32, _I32, _I32, _VP, _VP, _VP, _VP, _I32, _VP, _SZ, _VP], ctypes.c_int),
    "moe_gated_ffn_workspace_size": ([_I32, _I32, _I32], _SZ),
    "moe_gated_ffn": ([_I32, _I32, _I32, _F32, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP, _SZ, _VP], ctypes.c_int),
    "moe_gated_ffn_backward_workspace_size": ([_I32, _I32, _I32], _SZ),
    "moe_gated_ffn_backward": ([_I32, _I32, _I32, _F32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP, _SZ,
                                _VP], ctypes.c_int),
    "moe_forward_stack": ([_CFGP, _I32, _VP, _I32, _VP, _VP, _VP, _VP, _I32, _VP, _SZ, _VP], ctypes.c_int),
    "moe_forward_noalloc": ([_CFGP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP,
                             _VP, _VP, _VP, _I32, _VP, _VP, _VP], ctypes.c_int),
    "moe_forward": ([_CFGP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP,
                     _VP, _VP, _VP, _I32, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_forward_w2q3": ([_CFGP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                          _VP, _VP, _VP, _I32, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
}


def lib():
    """The loaded ``libmoe.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with mxfp4_moe_expert_amd/build.py "
                               "(or __graft_entry__.build()); there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def version() -> str:
    return lib().moe_version().decode()


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoEError(status, what)


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, dtype, shape, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: torch.Tensor expected")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a device (cuda/hip) tensor")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


def set_kernel_events(kernel: str | None, start_event=None, stop_event=None):
    """Bracket every launch of ``kernel`` (a KERNELS name) with the given
    hipEvent_t handles (ints or c_void_p); None stops. Measurement only."""
    kid = 0 if kernel is None else KERNELS[kernel]
    _check(lib().moe_set_kernel_events(kid, start_event, stop_event), "moe_set_kernel_events")


OPTIONS = {"prefill_block_scaled": 1}


def set_option(name: str, value: int):
    """Set a process-wide option (``OPTIONS``); returns the previous value."""
    prev = lib().moe_get_option(OPTIONS[name])
    _check(lib().moe_set_option(OPTIONS[name], int(value)), "moe_set_option")
    return prev


FLAGS = {"token_id": 1, "table_entry": 2, "expert_id": 4, "wait_expired": 8, "permutation": 16}


def read_probe(buf, blocks: int, sink, device=None) -> None:
    """Queues the library's streaming-read kernel over all of ``buf`` (a
    contiguous device tensor, 16-byte multiple) with ``blocks`` blocks on the
    current stream; ``sink`` is an int32/uint32 device tensor of at least
    ``blocks`` words (a measurement aid: time it to get the read rate)."""
    if not (buf.is_cuda and sink.is_cuda and buf.is_contiguous()):
        raise ValueError("read_probe: contiguous device tensors expected")
    if sink.numel() * sink.element_size() < 4 * blocks:
        raise ValueError("read_probe: sink smaller than one word per block")
    _check(lib().moe_read_probe(buf.data_ptr(), buf.numel() * buf.element_size(), int(blocks), sink.data_ptr(),
                                _stream(device)), "moe_read_probe")


def device_flags(clear: bool = False, device=None) -> set:
    """Names of the device error flags (``FLAGS``) set on the current device
    by work queued so far on the current stream; waits for that stream.
    ``clear`` resets them afterwards."""
    v = ctypes.c_uint32(0)
    _check(lib().moe_device_flags(ctypes.byref(v), 1 if clear else 0, _stream(device)), "moe_device_flags")
    return {name for name, bit in FLAGS.items() if v.value & bit}


SCHEDULES = {1: "single", 2: "tiny", 3: "decode", 4: "large"}


def forward_schedule(cfg: MoeConfig, T: int, hash_layer: bool = False) -> str:
    """Which launch sequence ``forward`` takes for T tokens on the current
    device: "single" (the whole layer in one launch), "tiny", "decode" or
    "large"."""
    rc = lib().moe_forward_schedule(ctypes.byref(cfg), T, 1 if hash_layer else 0)
    if rc < 0:
        raise MoEError(rc, "moe_forward_schedule")
    return SCHEDULES[rc]


def workspace_size(cfg: MoeConfig, T: int) -> int:
    n = lib().moe_workspace_size(ctypes.byref(cfg), T)
    if n == 0:
        raise MoEError(MOE_EUNSUPPORTED, "moe_workspace_size")
    return n


class Workspace:
    """Zero-initialised device scratch, grown on demand (one per device/stream user)."""

    def __init__(self, device=None):
        self.device = torch.device(device or "cuda")
        self.buf = None

    def get(self, cfg: MoeConfig, T: int) -> torch.Tensor:
        need = workspace_size(cfg, T)
        if self.buf is None or self.buf.numel() < need:
            self.buf = torch.zeros(need, dtype=torch.uint8, device=self.device)
            if self.buf.data_ptr() % 256:
                raise RuntimeError("workspace allocation is not 256-byte aligned")
        return self.buf


_default_ws: dict = {}


def _ws(cfg, T, device, ws):
    if ws is None:
        key = torch.device(device).index or 0
        ws = _default_ws.setdefault(key, Workspace(device))
    buf = ws.get(cfg, T)
    return buf, buf.numel()


# ------------------------------------------------------------------ device layer

@dataclass
class DeviceLayer:
    """Device tensors of one layer (layouts as in include/moe.h)."""
    gate_w: torch.Tensor
    bias: torch.Tensor
    logit_offset: torch.Tensor | None
    w13_codes: torch.Tensor
    w13_scales: torch.Tensor
    w2_codes: torch.Tensor
    w2_scales: torch.Tensor
    sh_w13: torch.Tensor
    sh_w13_scale: torch.Tensor
    sh_w2: torch.Tensor
    sh_w2_scale: torch.Tensor
    tid2eid: torch.Tensor | None = None

    @staticmethod
    def from_host(layer, device="cuda") -> "DeviceLayer":
        """Copy a host layer (numpy arrays with the same field names) to the device."""
        def d(a):
            return None if a is None else torch.from_numpy(a).to(device)
        return DeviceLayer(d(layer.gate_w), d(layer.bias), d(layer.logit_offset), d(layer.w13_codes),
                           d(layer.w13_scales), d(layer.w2_codes), d(layer.w2_scales), d(layer.sh_w13),
                           d(layer.sh_w13_scale), d(layer.sh_w2), d(layer.sh_w2_scale), d(layer.tid2eid))


def bf16_from_numpy(a, device="cuda") -> torch.Tensor:
    """uint16 bf16 bit patterns (numpy) -> a torch.bfloat16 device tensor."""
    import numpy as np

    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(device).view(torch.bfloat16)


# ------------------------------------------------------------------ entry points

def route(cfg: MoeConfig, x, gate_w, bias, logit_offset=None, ws=None, out=None):
    """Learned router -> (topk_ids int32 [T,k], topk_w fp32 [T,k])."""
    T, H, E, k = x.shape[0], cfg.hidden_size, cfg.n_routed_experts, cfg.top_k
    _need(x, _BF16, (T, H), "x")
    _need(gate_w, torch.float32, (E, H), "gate_w")
    _need(bias, torch.float32, (E,), "bias")
    if logit_offset is not None:
        _need(logit_offset, torch.float32, (E,), "logit_offset")
    ids, w = out if out is not None else (torch.empty(T, k, dtype=torch.int32, device=x.device),
                                          torch.empty(T, k, dtype=torch.float32, device=x.device))
    buf, nb = _ws(cfg, T, x.device, ws)
    _check(lib().moe_route(ctypes.byref(cfg), T, _ptr(x), _ptr(gate_w), _ptr(bias), _ptr(logit_offset),
                           _ptr(ids), _ptr(w), _ptr(buf), nb, _stream(x.device)), "moe_route")
    return ids, w


def hash_route(cfg: MoeConfig, x, token_ids, tid2eid, gate_w, out=None):
    """Hash-layer router -> (topk_ids, topk_w)."""
    T, H, E, k = x.shape[0], cfg.hidden_size, cfg.n_routed_experts, cfg.top_k
    _need(x, _BF16, (T, H), "x")
    _need(token_ids, torch.int32, (T,), "token_ids")
    _need(tid2eid, torch.int32, None, "tid2eid")
    if tid2eid.dim() != 2 or tid2eid.shape[1] != k:
        raise ValueError("tid2eid: shape [V, top_k] expected")
    _need(gate_w, torch.float32, (E, H), "gate_w")
    ids, w = out if out is not None else (torch.empty(T, k, dtype=torch.int32, device=x.device),
                                          torch.empty(T, k, dtype=torch.float32, device=x.device))
    _check(lib().moe_hash_route(ctypes.byref(cfg), T, _ptr(x), _ptr(token_ids), _ptr(tid2eid),
                                tid2eid.shape[0], _ptr(gate_w), _ptr(ids), _ptr(w), _stream(x.device)),
           "moe_hash_route")
    return ids, w


def permute(cfg: MoeConfig, topk_ids, ws=None):
    """Stable sort of slots by expert -> (expert_offsets [E+1], sorted_slots [T*k], slot_pos [T*k])."""
    T, k, E = topk_ids.shape[0], cfg.top_k, cfg.n_routed_experts
    _need(topk_ids, torch.int32, (T, k), "topk_ids")
    dev = topk_ids.device
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    sorted_slots = torch.empty(T * k, dtype=torch.int32, device=dev)
    slot_pos = torch.empty(T * k, dtype=torch.int32, device=dev)
    buf, nb = _ws(cfg, T, dev, ws)
    _check(lib().moe_permute(ctypes.byref(cfg), T, _ptr(topk_ids), _ptr(offsets), _ptr(sorted_slots),
                             _ptr(slot_pos), _ptr(buf), nb, _stream(dev)), "moe_permute")
    return offsets, sorted_slots, slot_pos


def expert_ffn(cfg: MoeConfig, x, expert_offsets, sorted_slots, topk_w, w13_codes, w13_scales, w2_codes,
               w2_scales, ws=None):
    """Routed experts only -> routed_out fp32 [T, H]."""
    T, H, E, k, I = x.shape[0], cfg.hidden_size, cfg.n_routed_experts, cfg.top_k, cfg.moe_intermediate
    _need(x, _BF16, (T, H), "x")
    _need(expert_offsets, torch.int32, (E + 1,), "expert_offsets")
    _need(sorted_slots, torch.int32, (T * k,), "sorted_slots")
    _need(topk_w, torch.float32, (T, k), "topk_w")
    _need(w13_codes, torch.uint8, (E, 2 * I, H // 2), "w13_codes")
    _need(w13_scales, torch.uint8, (E, 2 * I, H // 32), "w13_scales")
    _need(w2_codes, torch.uint8, (E, H, I // 2), "w2_codes")
    _need(w2_scales, torch.uint8, (E, H, I // 32), "w2_scales")
    out = torch.empty(T, H, dtype=torch.float32, device=x.device)
    buf, nb = _ws(cfg, T, x.device, ws)
    _check(lib().moe_expert_ffn(ctypes.byref(cfg), T, _ptr(x), _ptr(expert_offsets), _ptr(sorted_slots),
                                _ptr(topk_w), _ptr(w13_codes), _ptr(w13_scales), _ptr(w2_codes),
                                _ptr(w2_scales), _ptr(out), _ptr(buf), nb, _stream(x.device)),
           "moe_expert_ffn")
    return out


def forward(cfg: MoeConfig, x, layer: DeviceLayer, token_ids=None, out_fp32=False, return_routing=False,
            ws=None, out=None, routing_out=None):
    """The whole layer -> out [T, H] (bf16, or fp32 if out_fp32) [, (topk_ids, topk_w)]."""
    T, H, E, k, I = x.shape[0], cfg.hidden_size, cfg.n_routed_experts, cfg.top_k, cfg.moe_intermediate
    dev = x.device
    _need(x, _BF16, (T, H), "x")
    _need(layer.gate_w, torch.float32, (E, H), "gate_w")
    _need(layer.w13_codes, torch.uint8, (E, 2 * I, H // 2), "w13_codes")
    _need(layer.w13_scales, torch.uint8, (E, 2 * I, H // 32), "w13_scales")
    _need(layer.w2_codes, torch.uint8, (E, H, I // 2), "w2_codes")
    _need(layer.w2_scales, torch.uint8, (E, H, I // 32), "w2_scales")
    _need(layer.sh_w13, torch.int8, (2 * I, H), "sh_w13")
    _need(layer.sh_w13_scale, torch.float32, (2 * I,), "sh_w13_scale")
    _need(layer.sh_w2, torch.int8, (H, I), "sh_w2")
    _need(layer.sh_w2_scale, torch.float32, (H,), "sh_w2_scale")
    V = 0
    if token_ids is not None:
        _need(token_ids, torch.int32, (T,), "token_ids")
        if layer.tid2eid is None:
            raise ValueError("hash layer needs layer.tid2eid")
        _need(layer.tid2eid, torch.int32, None, "tid2eid")
        V = layer.tid2eid.shape[0]
    else:
        _need(layer.bias, torch.float32, (E,), "bias")
    if out is None:
        out = torch.empty(T, H, dtype=torch.float32 if out_fp32 else torch.bfloat16, device=dev)
    ids = w = None
    if return_routing:
        ids, w = routing_out if routing_out is not None else (
            torch.empty(T, k, dtype=torch.int32, device=dev), torch.empty(T, k, dtype=torch.float32, device=dev))
    buf, nb = _ws(cfg, T, dev, ws)
    _check(lib().moe_forward(
        ctypes.byref(cfg), T, _ptr(x), _ptr(layer.gate_w), _ptr(layer.bias), _ptr(layer.logit_offset),
        _ptr(token_ids), _ptr(layer.tid2eid if token_ids is not None else None), V, _ptr(layer.w13_codes),
        _ptr(layer.w13_scales), _ptr(layer.w2_codes), _ptr(layer.w2_scales), _ptr(layer.sh_w13),
        _ptr(layer.sh_w13_scale), _ptr(layer.sh_w2), _ptr(layer.sh_w2_scale), _ptr(out), int(out_fp32),
        _ptr(ids), _ptr(w), _ptr(buf), nb, _stream(dev)), "moe_forward")
    if return_routing:
        return out, (ids, w)
    return out


def forward_w2q3(cfg: MoeConfig, x, layer: DeviceLayer, w2_codes, w2_scales, w2_levels=None, token_ids=None,
                 out_fp32=False, return_routing=False, ws=None, out=None):
    """``forward`` with the routed experts' w2 in 3-bit blocks (moe_forward_w2q3):
    w2_codes uint8 [E, H, I/32*12], w2_scales int16/uint16 [E, H, I/32]
    (binary16 bits), w2_levels fp32 [E, 8] or None (the uniform code book).
    ``layer``'s own w2 tensors are not used."""
    T, H, E, k, I = x.shape[0], cfg.hidden_size, cfg.n_routed_experts, cfg.top_k, cfg.moe_intermediate
    dev = x.device
    _need(x, _BF16, (T, H), "x")
    _need(layer.gate_w, torch.float32, (E, H), "gate_w")
    _need(layer.w13_codes, torch.uint8, (E, 2 * I, H // 2), "w13_codes")
    _need(layer.w13_scales, torch.uint8, (E, 2 * I, H // 32), "w13_scales")
    _need(w2_codes, torch.uint8, (E, H, I // 32 * 12), "w2_codes")
    _need(w2_scales, (torch.int16, torch.uint16), (E, H, I // 32), "w2_scales")
    if w2_levels is not None:
        _need(w2_levels, torch.float32, (E, 8), "w2_levels")
    _need(layer.sh_w13, torch.int8, (2 * I, H), "sh_w13")
    _need(layer.sh_w2, torch.int8, (H, I), "sh_w2")
    V = 0
    if token_ids is not None:
        _need(token_ids, torch.int32, (T,), "token_ids")
        if layer.tid2eid is None:
            raise ValueError("hash layer needs layer.tid2eid")
        V = layer.tid2eid.shape[0]
    else:
        _need(layer.bias, torch.float32, (E,), "bias")
    if out is None:
        out = torch.empty(T, H, dtype=torch.float32 if out_fp32 else torch.bfloat16, device=dev)
    ids = w = None
    if return_routing:
        ids = torch.empty(T, k, dtype=torch.int32, device=dev)
        w = torch.empty(T, k, dtype=torch.float32, device=dev)
    buf, nb = _ws(cfg, T, dev, ws)
    _check(lib().moe_forward_w2q3(
        ctypes.byref(cfg), T, _ptr(x), _ptr(layer.gate_w), _ptr(layer.bias), _ptr(layer.logit_offset),
        _ptr(token_ids), _ptr(layer.tid2eid if token_ids is not None else None), V, _ptr(layer.w13_codes),
        _ptr(layer.w13_scales), _ptr(w2_codes), _ptr(w2_scales), _ptr(w2_levels), _ptr(layer.sh_w13),
        _ptr(layer.sh_w13_scale), _ptr(layer.sh_w2), _ptr(layer.sh_w2_scale), _ptr(out), int(out_fp32),
        _ptr(ids), _ptr(w), _ptr(buf), nb, _stream(dev)), "moe_forward_w2q3")
    if return_routing:
        return out, (ids, w)
    return out


def forward_noalloc(cfg: MoeConfig, x, layer: DeviceLayer, token_ids=None, out_fp32=False, out=None,
                    routing_out=None):
    """``forward`` through moe_forward_noalloc (no workspace: the library's
    fixed per-GPU scratch). ``out`` and ``routing_out`` may be preallocated
    so that the call itself allocates nothing."""
    T, H, E, k, I = x.shape[0], cfg.hidden_size, cfg.n_routed_experts, cfg.top_k, cfg.moe_intermediate
    dev = x.device
    _need(x, _BF16, (T, H), "x")
    _need(layer.w13_codes, torch.uint8, (E, 2 * I, H // 2), "w13_codes")
    _need(layer.w2_codes, torch.uint8, (E, H, I // 2), "w2_codes")
    _need(layer.sh_w13, torch.int8, (2 * I, H), "sh_w13")
    _need(layer.sh_w2, torch.int8, (H, I), "sh_w2")
    V = 0
    if token_ids is not None:
        _need(token_ids, torch.int32, (T,), "token_ids")
        V = layer.tid2eid.shape[0]
    if out is None:
        out = torch.empty(T, H, dtype=torch.float32 if out_fp32 else torch.bfloat16, device=dev)
    ids, w = routing_out if routing_out is not None else (None, None)
    _check(lib().moe_forward_noalloc(
        ctypes.byref(cfg), T, _ptr(x), _ptr(layer.gate_w), _ptr(layer.bias), _ptr(layer.logit_offset),
        _ptr(token_ids), _ptr(layer.tid2eid if token_ids is not None else None), V, _ptr(layer.w13_codes),
        _ptr(layer.w13_scales), _ptr(layer.w2_codes), _ptr(layer.w2_scales), _ptr(layer.sh_w13),
        _ptr(layer.sh_w13_scale), _ptr(layer.sh_w2), _ptr(layer.sh_w2_scale), _ptr(out), int(out_fp32),
        _ptr(ids), _ptr(w), _stream(dev)), "moe_forward_noalloc")
    return out


def layer_weights(layer: DeviceLayer) -> MoeLayerWeights:
    """The ``moe_layer_weights`` of a device layer (hash layer if it has a tid2eid table)."""
    def p(t):
        return None if t is None else t.data_ptr()
    V = 0 if layer.tid2eid is None else layer.tid2eid.shape[0]
    return MoeLayerWeights(p(layer.gate_w), p(layer.bias), p(layer.logit_offset), p(layer.tid2eid), V,
                           p(layer.w13_codes), p(layer.w13_scales), p(layer.w2_codes), p(layer.w2_scales),
                           p(layer.sh_w13), p(layer.sh_w13_scale), p(layer.sh_w2), p(layer.sh_w2_scale))


def forward_stack(cfg: MoeConfig, x, layers, token_ids=None, out_fp32=False, ws=None, act=None, out=None,
                  weights=None):
    """MoE layers back to back (moe_forward_stack): layer l + 1 reads layer l's
    bf16 output. ``layers``: DeviceLayers (hash layers carry tid2eid);
    ``weights``: their prebuilt ctypes array (optional, for repeated calls)."""
    T, H = x.shape[0], cfg.hidden_size
    dev = x.device
    _need(x, _BF16, (T, H), "x")
    n = len(layers)
    if weights is None:
        weights = (MoeLayerWeights * n)(*[layer_weights(L) for L in layers])
    if token_ids is not None:
        _need(token_ids, torch.int32, (T,), "token_ids")
    if act is None:
        act = torch.empty(2, T, H, dtype=torch.bfloat16, device=dev)
    if out is None:
        out = torch.empty(T, H, dtype=torch.float32 if out_fp32 else torch.bfloat16, device=dev)
    buf, nb = _ws(cfg, T, dev, ws)
    _check(lib().moe_forward_stack(ctypes.byref(cfg), n, weights, T, _ptr(x), _ptr(token_ids), _ptr(act),
                                   _ptr(out), int(out_fp32), _ptr(buf), nb, _stream(dev)), "moe_forward_stack")
    return out


_linear_ws: dict = {}


def linear_w8a16(x, q, scale, groups=1, out_fp32=False, out=None, ws=None):
    """int8 per-channel linear (moe_linear_w8a16): x [T][groups*K] bf16, q
    [groups*N][K] int8, scale [groups*N] f32 -> [T][groups*N] (bf16 or f32)."""
    T = x.shape[0]
    dev = x.device
    _need(x, _BF16, None, "x")
    _need(q, torch.int8, None, "q")
    _need(scale, torch.float32, None, "scale")
    if x.dim() != 2 or q.dim() != 2 or x.shape[1] % groups or q.shape[0] % groups:
        raise ValueError("x [T][groups*K], q [groups*N][K] expected")
    K, N = x.shape[1] // groups, q.shape[0] // groups
    if q.shape[1] != K or scale.shape != (groups * N,):
        raise ValueError("shapes of q / scale do not match x")
    need = lib().moe_linear_workspace_size(T, K, N, groups)
    if need == 0:
        raise MoEError(MOE_EUNSUPPORTED, "moe_linear_workspace_size")
    if ws is None:
        key = torch.device(dev).index or 0
        ws = _linear_ws.get(key)
        if ws is None or ws.numel() < need:
            ws = torch.zeros(max(need, 1 << 20), dtype=torch.uint8, device=dev)
            _linear_ws[key] = ws
    if out is None:
        out = torch.empty(T, groups * N, dtype=torch.float32 if out_fp32 else torch.bfloat16, device=dev)
    _check(lib().moe_linear_w8a16(T, K, N, groups, _ptr(x), _ptr(q), _ptr(scale), _ptr(out), int(out_fp32),
                                  _ptr(ws), ws.numel(), _stream(dev)), "moe_linear_w8a16")
    return out


# ------------------------------------------------------------------ MXFP4 tensors and products, the gated block
#
# These calls take their scratch from torch's allocator per call (or from
# ``ws``, a uint8 tensor of at least the size the C ABI names), so calls on
# different streams and captured graphs never share one by accident. They run
# on the device of their tensors, whatever the current device is. They are no
# autograd operations: outputs have no history, whatever their inputs require.
# Outputs and workspaces must not overlap each other or an input.

# Small calls last a few microseconds, so the argument checks here are the
# short forms; a check that fails is repeated by ``_need``, which words it.

_DTYPES = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}
_ACTS = {"bf16": 0, "mxfp4": 1}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _arg(t, dtype, shape, index, name):
    """t's pointer, t being a contiguous ``dtype`` tensor of ``shape`` on device ``index``."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        return t.data_ptr()
    _need(t, dtype, shape, name)
    raise ValueError(f"{name}: on {t.device}, expected cuda:{index}")


def _scale_bytes(t, shape, index):
    """Pointer of an MXFP4 tensor's scales, and the tensor it belongs to (to be kept until the call is queued). Cut out
    of a stacked tensor they start at any byte, N K / 32 being any number: the call then reads an aligned copy."""
    if (isinstance(t, torch.Tensor) and t.dtype is torch.uint8 and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        p = t.data_ptr()
        if p & 15:
            t = t.clone()
            p = t.data_ptr()
        return p, t
    return _arg(t, torch.uint8, shape, index, "scales"), t


def _matrix(t, dtype, name):
    """Rows, columns and device index of a 2-D tensor whose own checks follow."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not dtype:
        _need(t, dtype, None, name)
    if t.dim() != 2:
        raise ValueError(f"{name}: two dimensions expected")
    return t.shape[0], t.shape[1], t.get_device()


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(index, name, *args):
    """Calls a library function with device ``index`` current, its current stream appended."""
    fn = getattr(_lib or lib(), name)
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != MOE_OK:
        raise MoEError(status, _misaligned(name, args) if status == MOE_EINVAL else name)


# The pointer arguments of the calls, in order.
_POINTERS = {
    "moe_mxfp4_quantize": ("x", "codes", "scales"),
    "moe_mxfp4_dequantize": ("codes", "scales", "out"),
    "moe_linear_mxfp4": ("x", "codes", "scales", "out", "ws"),
    "moe_linear_mxfp4_dx": ("dy", "codes", "scales", "out", "ws"),
    "moe_gated_ffn": ("x", "w13", "w2", "saved[0]", "saved[1]", "out", "ws"),
    "moe_gated_ffn_backward": ("dy", "x", "w13", "w2", "saved[0]", "saved[1]", "dx", "dw13", "dw2", "ws"),
}


def _misaligned(name, args):
    """What a refused call is about: its first tensor off its border (16 bytes, workspaces 256), else the call."""
    pointers = [a for a, t in zip(args, _SIGNATURES[name][0]) if t is _VP]
    for what, p in zip(_POINTERS[name], pointers):
        border = 256 if what == "ws" else 16
        if p and p % border:
            return f"{name}, {what}: not {border}-byte aligned"
    return name


def _scratch(need, like, ws, what):
    """Pointer and size of the workspace, and its tensor (to be kept until the call is queued)."""
    if need == 0:
        raise MoEError(MOE_EUNSUPPORTED, what)
    if ws is None:
        ws = like.new_empty((need,), dtype=torch.uint8)
        return ws.data_ptr(), need, ws
    return _arg(ws, torch.uint8, ws.shape, like.get_device(), "ws"), ws.numel(), ws


def _result(out, shape, dtype, like, name="out"):
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    _arg(out, dtype, shape, like.get_device(), name)
    return out


def quantize_mxfp4(x, out=None):
    """x [..., K] (bf16, fp32 or fp16; K a multiple of 32) -> (codes uint8
    [..., K/2], scales uint8 [..., K/32]), the layer's MXFP4 layout
    (moe_mxfp4_quantize). x is contiguous, or 2-D with unit column stride and
    16-byte aligned rows."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x: torch.Tensor expected")
    if not x.is_cuda:
        raise ValueError("x: must be a device (cuda/hip) tensor")
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        raise TypeError(f"x: dtype {x.dtype}, expected bfloat16, float32 or float16")
    shape = x.shape
    K = shape[-1] if len(shape) else 0
    if K == 0 or K % 32:
        raise ValueError("x: last dimension must be a positive multiple of 32")
    ldx = K
    if not x.is_contiguous():
        if x.dim() != 2 or x.stride(1) != 1 or x.stride(0) < K:
            raise ValueError("x: contiguous, or 2-D with unit column stride, expected")
        ldx = x.stride(0)
    lead = tuple(shape[:-1])
    c, s = out if out is not None else (None, None)
    codes = _result(c, lead + (K // 2,), torch.uint8, x, "codes")
    scales = _result(s, lead + (K // 32,), torch.uint8, x, "scales")
    _call(x.get_device(), "moe_mxfp4_quantize", x.numel() // K, K, dt, x.data_ptr(), ldx, codes.data_ptr(),
          scales.data_ptr())
    return codes, scales


def dequantize_mxfp4(codes, scales, dtype=torch.bfloat16, out=None):
    """(codes [..., K/2], scales [..., K/32]) -> [..., K] in bf16 or fp32, exact (moe_mxfp4_dequantize). The scales
    may start at any byte, as those of one matrix of a stack do (here and in the products)."""
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError(f"dtype {dtype}, expected bfloat16 or float32")
    if not isinstance(codes, torch.Tensor) or not codes.is_cuda:
        _need(codes, torch.uint8, None, "codes")
    shape, index = codes.shape, codes.get_device()
    K = shape[-1] * 2 if len(shape) else 0
    if K == 0 or K % 32:
        raise ValueError("codes: last dimension must be a positive multiple of 16")
    lead = tuple(shape[:-1])
    pc = _arg(codes, torch.uint8, shape, index, "codes")
    ps, scales = _scale_bytes(scales, lead + (K // 32,), index)
    out = _result(out, lead + (K,), dtype, codes)
    _call(index, "moe_mxfp4_dequantize", codes.numel() * 2 // K, K, pc, ps, _DTYPES[dtype], out.data_ptr())
    return out


def _mxfp4_weight(codes, scales, index):
    """N, K and the pointers of an MXFP4 matrix [N][K] on device ``index``, and its scales' tensor (to be kept)."""
    if (isinstance(codes, torch.Tensor) and codes.dtype is torch.uint8 and codes.dim() == 2
            and codes.get_device() == index and codes.is_contiguous()):
        N, half = codes.shape
        if half and half % 16 == 0:
            ps, scales = _scale_bytes(scales, (N, half // 16), index)
            return N, half * 2, codes.data_ptr(), ps, scales
    _matrix(codes, torch.uint8, "codes")
    _arg(codes, torch.uint8, codes.shape, index, "codes")
    raise ValueError("codes: shape [N, K/2] with K a positive multiple of 32 expected")


def linear_mxfp4(x, codes, scales, act="bf16", out_fp32=False, out=None, ws=None):
    """y = x W^T (moe_linear_mxfp4): x [T][K] bf16, W [N][K] as codes
    [N][K/2] and scales [N][K/32] -> [T][N] (bf16 or fp32). act: "bf16", or
    "mxfp4" to round x to MXFP4 first. Autograd does not see it: its input
    gradient is ``linear_mxfp4_dx``."""
    mode = _ACTS.get(act)
    if mode is None:
        raise ValueError(f"act {act!r}, expected one of {sorted(_ACTS)}")
    T, cols, index = _matrix(x, torch.bfloat16, "x")
    N, K, pc, ps, scales = _mxfp4_weight(codes, scales, index)
    if cols != K or not x.is_contiguous():
        _need(x, torch.bfloat16, (T, K), "x")
    if out is None:
        out = x.new_empty((T, N), dtype=torch.float32) if out_fp32 else x.new_empty((T, N))
    else:
        _arg(out, torch.float32 if out_fp32 else torch.bfloat16, (T, N), index, "out")
    pw, nw = None, 0
    if T > 1 or ws is not None:  # one row is always streamed, without a workspace
        need = lib().moe_linear_mxfp4_workspace_size(T, K, N, mode)
        if need != 256 or ws is not None:
            pw, nw, ws = _scratch(need, x, ws, "moe_linear_mxfp4")
    _call(index, "moe_linear_mxfp4", T, K, N, x.data_ptr(), pc, ps, mode, out.data_ptr(), 1 if out_fp32 else 0, pw, nw)
    return out


def linear_mxfp4_dx(dy, codes, scales, out_fp32=False, out=None, ws=None):
    """dx = dy W, the input gradient of ``linear_mxfp4`` through frozen
    weights (moe_linear_mxfp4_dx): dy [T][N] bf16 -> [T][K] (bf16 or fp32)."""
    T, _, index = _matrix(dy, torch.bfloat16, "dy")
    N, K, pc, ps, scales = _mxfp4_weight(codes, scales, index)
    py = _arg(dy, torch.bfloat16, (T, N), index, "dy")
    out = _result(out, (T, K), torch.float32 if out_fp32 else torch.bfloat16, dy)
    pw, nw, ws = _scratch(lib().moe_linear_mxfp4_dx_workspace_size(T, K, N), dy, ws, "moe_linear_mxfp4_dx")
    _call(index, "moe_linear_mxfp4_dx", T, K, N, py, pc, ps, out.data_ptr(), 1 if out_fp32 else 0, pw, nw)
    return out


def _ffn_args(x, w13, w2):
    """T, H, I, the device index and the pointers of the block's inputs."""
    T, H, index = _matrix(x, torch.bfloat16, "x")
    h2, I, _ = _matrix(w2, torch.bfloat16, "w2")
    if h2 != H:
        raise ValueError(f"w2: shape {tuple(w2.shape)}, expected ({H}, I)")
    return (T, H, I, index, _arg(x, torch.bfloat16, (T, H), index, "x"),
            _arg(w13, torch.bfloat16, (2 * I, H), index, "w13"), _arg(w2, torch.bfloat16, (H, I), index, "w2"))


def gated_ffn(x, w13, w2, limit=10.0, save=False, out_fp32=False, out=None, ws=None):
    """The expert's block with bf16 weights (moe_gated_ffn): x [T][H], w13
    [2I][H] (gate rows, then up rows), w2 [H][I] -> y [T][H] (bf16 or fp32).
    save=True returns (y, saved), ``saved`` being what ``gated_ffn_backward``
    takes: (g and u [T][2I] fp32, h [T][I] bf16). Autograd does not see it: the
    gradients are ``gated_ffn_backward``'s."""
    T, H, I, index, px, p13, p2 = _ffn_args(x, w13, w2)
    out = _result(out, (T, H), torch.float32 if out_fp32 else torch.bfloat16, x)
    saved = (x.new_empty((T, 2 * I), dtype=torch.float32), x.new_empty((T, I))) if save else None
    pg, ph = (saved[0].data_ptr(), saved[1].data_ptr()) if save else (None, None)
    pw, nw, ws = _scratch(lib().moe_gated_ffn_workspace_size(T, H, I), x, ws, "moe_gated_ffn")
    _call(index, "moe_gated_ffn", T, H, I, limit, px, p13, p2, pg, ph, out.data_ptr(), 1 if out_fp32 else 0, pw, nw)
    return (out, saved) if save else out


def gated_ffn_backward(dy, x, w13, w2, saved, limit=10.0, need=(True, True, True), dw_fp32=False, ws=None):
    """Gradients of ``gated_ffn`` (moe_gated_ffn_backward) for dy [T][H] bf16:
    (dx [T][H] bf16, dw13 [2I][H], dw2 [H][I]; the weights' in bf16, or fp32
    if dw_fp32). ``saved`` and ``limit``: the forward call's. ``need``: which
    of the three to compute (None in the others' places)."""
    T, H, I, index, px, p13, p2 = _ffn_args(x, w13, w2)
    pd = _arg(dy, torch.bfloat16, (T, H), index, "dy")
    pg = _arg(saved[0], torch.float32, (T, 2 * I), index, "saved[0]")
    ph = _arg(saved[1], torch.bfloat16, (T, I), index, "saved[1]")
    wt = torch.float32 if dw_fp32 else torch.bfloat16
    dx = x.new_empty((T, H)) if need[0] else None
    dw13 = x.new_empty((2 * I, H), dtype=wt) if need[1] else None
    dw2 = x.new_empty((H, I), dtype=wt) if need[2] else None
    pw, nw, ws = _scratch(lib().moe_gated_ffn_backward_workspace_size(T, H, I), x, ws, "moe_gated_ffn_backward")
    _call(index, "moe_gated_ffn_backward", T, H, I, limit, pd, px, p13, p2, pg, ph,
          None if dx is None else dx.data_ptr(), None if dw13 is None else dw13.data_ptr(),
          None if dw2 is None else dw2.data_ptr(), 1 if dw_fp32 else 0, pw, nw)
    return dx, dw13, dw2
