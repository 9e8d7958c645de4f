"""ctypes binding over libmol.so (include/mol.h), with the same entry point names.

Argument marshalling only: tensors become device pointers, torch's current stream becomes
the hipStream_t, missing outputs are allocated with torch. Every step of the path runs in
the HIP kernels of libmol; there is no fallback of any kind - if the library is missing or
a call fails, this raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOL_LIBRARY names another build of the same library (the host-sanitizer build of the CPU
# tests); by default, the one built in-tree
LIB_PATH = os.environ.get("MOL_LIBRARY") or os.path.join(_PKG, "libmol.so")

MOL_OK, MOL_E_ARG, MOL_E_LIMIT, MOL_E_DTYPE, MOL_E_ALIGN, MOL_E_WORKSPACE, MOL_E_HIP = range(7)
MOL_F32, MOL_BF16 = 0, 1
MOL_MAX_BUCKETS = 8192
MOL_SCORE_SOFTMAX, MOL_SCORE_SIGMOID = 0, 1
MOL_MAX_ROUTER_TOPK = 64
MOL_ACT_NONE, MOL_ACT_SILU_MUL = 0, 1

# every symbol include/mol.h declares, with (restype, argtypes)
_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_F32 = ctypes.c_float
SIGNATURES = {
    "mol_status_string": (ctypes.c_char_p, [_I32]),
    "mol_abi_version": (_I32, []),
    "mol_virtual_topk": (_I32, [_P, _P, _I32, _I32, _I32, _I32, _P, _P]),
    "mol_align_max_blocks": (_I64, [_I64, _I32, _I32]),
    "mol_align_workspace_bytes": (_I64, [_I64, _I32, _I32]),
    "mol_plan_bytes": (_I64, [_I64, _I32, _I32]),
    "mol_align_block_size": (_I32, [_P, _P, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _SZ,
                                    _P, _SZ, _P]),
    "mol_lora_shrink": (_I32, [_I32, _P, _I64, _I32, _P, _I32, _I32, _I32, _P, _I32, _P, _P,
                               _P, _I32, _I32, _I32, _P, _P]),
    "mol_lora_expand": (_I32, [_I32, _P, _I32, _I32, _P, _I32, _P, _P, _I32, _P, _P, _P, _P,
                               _I32, _I32, _I32, _P, _I64, _P]),
    "mol_delta_workspace_bytes": (_I64, [_I32, _I32, _I32, _I32]),
    "mol_lora_delta": (_I32, [_I32, _P, _I64, _I32, _P, _I32, _I32, _I32, _P, _I32, _P, _P,
                              _I32, _P, _P, _P, _P, _I32, _I32, _I32, _P, _I64, _P, _SZ, _P]),
    "mol_lora_delta_noalloc": (_I32, [_I32, _P, _I64, _I32, _P, _I32, _I32, _I32, _P, _I32, _P,
                                      _P, _I32, _P, _P, _P, _P, _I32, _I32, _I32, _P, _I64,
                                      _P]),
    "mol_moe_gemm": (_I32, [_I32, _P, _I64, _I32, _P, _I32, _I32, _I32, _P, _P, _P, _I32, _I32,
                            _P, _I64, _P, _I32, _I32, _P, _P, _P, _P, _I32, _I32, _P]),
    "mol_moe_combine": (_I32, [_I32, _P, _I64, _P, _P, _I32, _I32, _I32, _I32, _P, _I64, _P]),
    "mol_lora_expand_combine": (_I32, [_I32, _P, _I32, _P, _I32, _P, _P, _P, _P, _P, _I32,
                                       _I32, _I32, _I32, _P, _I64, _P, _I64, _P]),
    "mol_router_topk": (_I32, [_I32, _P, _I64, _I32, _I32, _I32, _I32, _I32, _F32, _I32, _I32,
                               _P, _P, _P]),
    "mol_moe_gemm_q4": (_I32, [_I32, _P, _I64, _I32, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _P,
                               _P, _I32, _I32, _P, _I64, _P]),
    "mol_router_balance_workspace_bytes": (_I64, [_I32, _I32]),
    "mol_router_balance": (_I32, [_I32, _P, _I64, _P, _P, _I32, _I32, _I32, _I32, _F32, _P, _P, _P,
                                  _P, _SZ, _P]),
    "mol_router_balance_grad": (_I32, [_I32, _P, _I64, _P, _P, _P, _I32, _I32, _I32, _I32, _F32,
                                       _P, _I64, _P]),
    "mol_mx4_quantize": (_I32, [_I32, _I32, _P, _I64, _I64, _I32, _P, _P, _P]),
    "mol_mx4_dequantize": (_I32, [_I32, _P, _P, _I64, _I32, _P, _I64, _P]),
    "mol_moe_gemm_mx4": (_I32, [_I32, _P, _I64, _P, _I32, _P, _P, _I32, _I32, _I32, _P, _P, _P,
                                _I32, _I32, _P, _I64, _P]),
    "mol_moe_layer_workspace_bytes": (_I64, [_I32, _I32, _I32, _I32, _I32, _I32]),
    "mol_moe_layer": (_I32, [_P, _P, _P, _I64, _P, _P, _P, _I32, _I32, _P, _I64, _P, _SZ, _P]),
}


class MolError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmol.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m virtual_expert_routed_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().mol_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != MOL_OK:
        raise MolError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t=None):
    dev = t.device if t is not None and t.is_cuda else None
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOL_F32
    if t.dtype == torch.bfloat16:
        return MOL_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _need(t: torch.Tensor, name: str, dtype=None, contiguous=True):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ------------------------------------------------------------------------------- sizing


def mol_align_max_blocks(numel: int, num_virtual: int, block_m: int) -> int:
    v = lib().mol_align_max_blocks(numel, num_virtual, block_m)
    if v < 0:
        raise MolError("mol_align_max_blocks", -v)
    return int(v)


def mol_align_workspace_bytes(numel: int, num_virtual: int, block_m: int) -> int:
    v = lib().mol_align_workspace_bytes(numel, num_virtual, block_m)
    if v < 0:
        raise MolError("mol_align_workspace_bytes", -v)
    return int(v)


def mol_plan_bytes(numel: int, num_virtual: int, block_m: int) -> int:
    v = lib().mol_plan_bytes(numel, num_virtual, block_m)
    if v < 0:
        raise MolError("mol_plan_bytes", -v)
    return int(v)


def new_plan(numel: int, num_virtual: int, block_m: int, device):
    """A buffer for the align's work plan (int32; written by mol_align_block_size)."""
    n = mol_plan_bytes(numel, num_virtual, block_m)
    return torch.empty(max(64, n // 4), dtype=torch.int32, device=device)


def mol_delta_workspace_bytes(numel: int, R: int, num_virtual: int, block_m: int) -> int:
    v = lib().mol_delta_workspace_bytes(numel, R, num_virtual, block_m)
    if v < 0:
        raise MolError("mol_delta_workspace_bytes", -v)
    return int(v)


# -------------------------------------------------------------------------- entry points


def mol_virtual_topk(topk_ids, lora_ids, num_experts: int, num_slots: int, out=None):
    _need(topk_ids, "topk_ids", torch.int32)
    _need(lora_ids, "lora_ids", torch.int32)
    M, k = topk_ids.shape
    if out is None:
        out = torch.empty_like(topk_ids)
    _need(out, "out", torch.int32)
    _check("mol_virtual_topk", lib().mol_virtual_topk(
        _ptr(topk_ids), _ptr(lora_ids), M, k, num_experts, num_slots, _ptr(out),
        _stream(topk_ids)))
    return out


def mol_align_block_size(ids, lora_ids, num_experts: int, num_slots: int, block_m: int,
                         sorted_ids=None, expert_ids=None, num_post_padded=None,
                         workspace=None, plan=None):
    """Returns (sorted_ids, expert_ids, num_post_padded) sized by mol_align_max_blocks. With
    plan (an int32 tensor of mol_plan_bytes), the work plan is written there as well."""
    _need(ids, "ids", torch.int32)
    if lora_ids is not None:
        _need(lora_ids, "lora_ids", torch.int32)
    M, k = ids.shape
    V = num_experts * num_slots
    mb = mol_align_max_blocks(M * k, V, block_m)
    dev = ids.device
    if sorted_ids is None:
        sorted_ids = torch.empty(max(1, mb * block_m), dtype=torch.int32, device=dev)
    if expert_ids is None:
        expert_ids = torch.empty(max(1, mb), dtype=torch.int32, device=dev)
    if num_post_padded is None:
        num_post_padded = torch.empty(1, dtype=torch.int32, device=dev)
    wsb = mol_align_workspace_bytes(M * k, V, block_m)
    if wsb and workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    if plan is not None:
        _need(plan, "plan", torch.int32)
    _check("mol_align_block_size", lib().mol_align_block_size(
        _ptr(ids), _ptr(lora_ids), M, k, num_experts, num_slots, block_m, _ptr(sorted_ids),
        _ptr(expert_ids), _ptr(num_post_padded), _ptr(plan),
        plan.numel() * 4 if plan is not None else 0, _ptr(workspace) if wsb else None,
        workspace.numel() if (wsb and workspace is not None) else 0, _stream(ids)))
    return sorted_ids, expert_ids, num_post_padded


def _ranks(slot_ranks):
    if slot_ranks is not None:
        _need(slot_ranks, "slot_ranks", torch.int32)
    return _ptr(slot_ranks)


def mol_lora_shrink(xin, row_div: int, A, sorted_ids, expert_ids, num_post_padded,
                    numel: int, num_virtual: int, block_m: int, s=None, slices: int = 1,
                    slot_ranks=None, num_experts: int = None):
    _need(xin, "xin", contiguous=False)
    _need(A, "A")
    if xin.stride(1) != 1:
        raise ValueError("xin rows must be contiguous")
    V, R, K = A.shape
    if s is None:
        s = torch.empty((max(1, numel), R), dtype=torch.float32, device=A.device)
    _need(s, "s", torch.float32)
    E = num_virtual if num_experts is None else num_experts
    _check("mol_lora_shrink", lib().mol_lora_shrink(
        _dtype_code(A), _ptr(xin), xin.stride(0), row_div, _ptr(A), R, K, slices,
        _ranks(slot_ranks), E, _ptr(sorted_ids), _ptr(expert_ids), _ptr(num_post_padded),
        numel, num_virtual, block_m, _ptr(s), _stream(A)))
    return s


def mol_lora_expand(s, slices: int, B, slot_scale, num_experts: int, sorted_ids, expert_ids,
                    num_post_padded, numel: int, num_virtual: int, block_m: int, out,
                    slot_ranks=None, plan=None):
    _need(B, "B")
    _need(s, "s", torch.float32)
    _need(slot_scale, "slot_scale", torch.float32)
    _need(out, "out", B.dtype, contiguous=False)
    if out.stride(1) != 1:
        raise ValueError("out rows must be contiguous")
    V, N, r = B.shape
    _check("mol_lora_expand", lib().mol_lora_expand(
        _dtype_code(B), _ptr(s), s.shape[1], slices, _ptr(B), N, _ptr(slot_scale),
        _ranks(slot_ranks), num_experts, _ptr(sorted_ids), _ptr(expert_ids),
        _ptr(num_post_padded), _ptr(plan), numel, num_virtual, block_m, _ptr(out),
        out.stride(0), _stream(B)))
    return out


def new_delta_workspace(numel: int, R: int, num_virtual: int, block_m: int, device):
    """A workspace for mol_lora_delta (its contents need no initialisation)."""
    n = mol_delta_workspace_bytes(numel, R, num_virtual, block_m)
    return torch.empty(max(256, n), dtype=torch.uint8, device=device)


def mol_lora_delta(xin, row_div: int, A, slices: int, B, slot_scale, num_experts: int,
                   sorted_ids, expert_ids, num_post_padded, numel: int, num_virtual: int,
                   block_m: int, out, workspace, slot_ranks=None, plan=None):
    _need(xin, "xin", contiguous=False)
    _need(A, "A")
    _need(B, "B")
    _need(slot_scale, "slot_scale", torch.float32)
    _need(out, "out", B.dtype, contiguous=False)
    _need(workspace, "workspace", torch.uint8)
    if xin.stride(1) != 1 or out.stride(1) != 1:
        raise ValueError("xin and out rows must be contiguous")
    V, R, K = A.shape
    _, N, r = B.shape
    _check("mol_lora_delta", lib().mol_lora_delta(
        _dtype_code(A), _ptr(xin), xin.stride(0), row_div, _ptr(A), R, K, slices, _ptr(B), N,
        _ptr(slot_scale), _ranks(slot_ranks), num_experts, _ptr(sorted_ids), _ptr(expert_ids),
        _ptr(num_post_padded), _ptr(plan), numel, num_virtual, block_m, _ptr(out), out.stride(0),
        _ptr(workspace), workspace.numel(), _stream(A)))
    return out


def mol_lora_delta_noalloc(xin, row_div: int, A, slices: int, B, slot_scale, num_experts: int,
                           sorted_ids, expert_ids, num_post_padded, numel: int,
                           num_virtual: int, block_m: int, out, slot_ranks=None, plan=None):
    """mol_lora_delta with s in the library's own per-GPU scratch: no workspace argument and
    nothing allocated (numel * R <= MOL_DELTA_SCRATCH_FLOATS; calls that overlap on one
    GPU race)."""
    _need(xin, "xin", contiguous=False)
    _need(A, "A")
    _need(B, "B")
    _need(slot_scale, "slot_scale", torch.float32)
    _need(out, "out", B.dtype, contiguous=False)
    if xin.stride(1) != 1 or out.stride(1) != 1:
        raise ValueError("xin and out rows must be contiguous")
    V, R, K = A.shape
    _, N, r = B.shape
    _check("mol_lora_delta_noalloc", lib().mol_lora_delta_noalloc(
        _dtype_code(A), _ptr(xin), xin.stride(0), row_div, _ptr(A), R, K, slices, _ptr(B), N,
        _ptr(slot_scale), _ranks(slot_ranks), num_experts, _ptr(sorted_ids), _ptr(expert_ids),
        _ptr(num_post_padded), _ptr(plan), numel, num_virtual, block_m, _ptr(out), out.stride(0),
        _stream(A)))
    return out


MOL_DELTA_SCRATCH_FLOATS = 4 * 1024 * 1024


def mol_moe_combine(rows, topk_ids, topk_weights, num_experts: int, y=None):
    """y [M, N] = per token the router-weighted sum of its pair rows [M*topk, N]."""
    _need(rows, "rows", contiguous=False)
    _need(topk_ids, "topk_ids", torch.int32)
    _need(topk_weights, "topk_weights", torch.float32)
    if rows.stride(1) != 1:
        raise ValueError("rows must have contiguous rows")
    M, k = topk_ids.shape
    N = rows.shape[1]
    if y is None:
        y = torch.empty((M, N), dtype=rows.dtype, device=rows.device)
    _need(y, "y", rows.dtype, contiguous=False)
    _check("mol_moe_combine", lib().mol_moe_combine(
        _dtype_code(rows), _ptr(rows), rows.stride(0), _ptr(topk_ids), _ptr(topk_weights), M,
        k, num_experts, N, _ptr(y), y.stride(0), _stream(rows)))
    return y


def mol_lora_expand_combine(s, B, slot_scale, topk_ids, lora_ids, topk_weights,
                            num_experts: int, num_slots: int, base, y=None, slot_ranks=None):
    """The down stage's expand fused with the combine: y [M, N] from s [M*topk, R], B
    [E*S, N, R] and the pairs' base rows [M*topk, N]; the rows are not written."""
    _need(B, "B")
    _need(s, "s", torch.float32)
    _need(slot_scale, "slot_scale", torch.float32)
    _need(topk_ids, "topk_ids", torch.int32)
    _need(lora_ids, "lora_ids", torch.int32)
    _need(topk_weights, "topk_weights", torch.float32)
    _need(base, "base", B.dtype, contiguous=False)
    if base.stride(1) != 1:
        raise ValueError("base must have contiguous rows")
    V, N, R = B.shape
    M, k = topk_ids.shape
    if y is None:
        y = torch.empty((M, N), dtype=B.dtype, device=B.device)
    _need(y, "y", B.dtype, contiguous=False)
    _check("mol_lora_expand_combine", lib().mol_lora_expand_combine(
        _dtype_code(B), _ptr(s), R, _ptr(B), N, _ptr(slot_scale), _ranks(slot_ranks),
        _ptr(topk_ids), _ptr(lora_ids), _ptr(topk_weights), M, k, num_experts, num_slots,
        _ptr(base), base.stride(0), _ptr(y), y.stride(0), _stream(B)))
    return y


def mol_moe_gemm(xin, row_div: int, W, sorted_ids, expert_ids, num_post_padded, numel: int,
                 block_m: int, out, s=None, slices: int = 1, B=None, slot_scale=None,
                 lora_ids=None, topk: int = 1, num_slots: int = 1, slot_ranks=None):
    """The base grouped GEMM of a stage into out [numel, N] (routing by base expert); with
    s and B the LoRA delta is added before the one rounding."""
    _need(xin, "xin", contiguous=False)
    _need(W, "W")
    _need(out, "out", W.dtype, contiguous=False)
    if xin.stride(1) != 1 or out.stride(1) != 1:
        raise ValueError("xin and out rows must be contiguous")
    E, N, K = W.shape
    R = 0
    if s is not None:
        _need(s, "s", torch.float32)
        _need(B, "B", W.dtype)
        _need(slot_scale, "slot_scale", torch.float32)
        _need(lora_ids, "lora_ids", torch.int32)
        R = s.shape[1]
    _check("mol_moe_gemm", lib().mol_moe_gemm(
        _dtype_code(W), _ptr(xin), xin.stride(0), row_div, _ptr(W), K, N, E, _ptr(sorted_ids),
        _ptr(expert_ids), _ptr(num_post_padded), numel, block_m, _ptr(out), out.stride(0),
        _ptr(s), R, slices, _ptr(B), _ptr(slot_scale), _ranks(slot_ranks), _ptr(lora_ids), topk,
        num_slots, _stream(W)))
    return out


def _on(dev, name: str, t: torch.Tensor, dtype, shape):
    """t is on dev, contiguous, of this dtype and shape."""
    if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    _need(t, name, dtype)
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _fit(fn: str, *values) -> None:
    """Whole numbers that an int32 argument holds (ctypes would wrap others)."""
    if max(values) > 0x7fffffff or min(values) < -0x80000000:
        raise ValueError(f"{fn}: {max(values, key=abs)} does not fit 32 bits")


_fns = {}  # entry points by name
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda i: torch.cuda.current_stream(i).cuda_stream)


_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(dev, fn: str, *args) -> None:
    """The entry point on dev's current stream, with dev current for the launch."""
    if dev.type != "cuda":
        raise ValueError(f"{fn} needs device tensors, got {dev}")
    f = _fns.get(fn)
    if f is None:
        f = _fns[fn] = getattr(lib(), fn)
    index = dev.index
    if index == _device():
        status = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = f(*args, _raw_stream(index))
    if status != MOL_OK:
        raise MolError(fn, status)


def mol_router_topk(logits, topk: int, scoring: int = MOL_SCORE_SOFTMAX,
                    renormalize: bool = True, scale: float = 1.0, first_expert: int = 0,
                    num_local: int = None, topk_ids=None, topk_weights=None):
    """The top-k experts of each token from router logits [M, E] (rows may be strided):
    (topk_ids int32 [M, topk], topk_weights float32 [M, topk])."""
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be 2-d with contiguous rows")
    M, E = logits.shape
    if num_local is None:
        num_local = E
    _fit("mol_router_topk", M, E, topk, scoring, first_expert, num_local)
    dev = logits.device
    if topk_ids is None:
        topk_ids = torch.empty((M, topk), dtype=torch.int32, device=dev)
    else:
        _on(dev, "topk_ids", topk_ids, torch.int32, (M, topk))
    if topk_weights is None:
        topk_weights = torch.empty((M, topk), dtype=torch.float32, device=dev)
    else:
        _on(dev, "topk_weights", topk_weights, torch.float32, (M, topk))
    _call(dev, "mol_router_topk", _dtype_code(logits), logits.data_ptr(),
          logits.stride(0) if M > 1 else max(logits.stride(0), E), M, E, topk, scoring,
          1 if renormalize else 0, scale, first_expert, num_local,
          topk_ids.data_ptr(), topk_weights.data_ptr())
    return topk_ids, topk_weights


def _rows(t: torch.Tensor, name: str, dev, dtype, shape) -> int:
    """t is on dev, 2-d with contiguous rows, of this dtype and shape; its row stride."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev:
        if t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")
        _need(t, name, dtype, contiguous=False)
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return ld if shape[0] > 1 else max(ld, shape[1])


def _q4(W, scales, zeros, name: str, dev):
    """(N, K, group) of packed 4-bit weights [E, N, K/2] with scales (and zeros) [E, N, K/G]."""
    if W.dim() != 3 or scales.dim() != 3 or scales.shape[2] < 1:
        raise ValueError(f"{name} must be [E, N, K/2] with scales [E, N, K/group]")
    E, N, half = W.shape
    _fit(name, E, N, 2 * half)
    _on(dev, name, W, torch.uint8, (E, N, half))
    _on(dev, name + " scales", scales, scales.dtype, (E, N, scales.shape[2]))
    if zeros is not None:
        _on(dev, name + " zeros", zeros, torch.uint8, scales.shape)
    if 2 * half % scales.shape[2]:
        raise ValueError(f"{name}: {2 * half} columns are not whole groups of {scales.shape[2]}")
    return N, 2 * half, 2 * half // scales.shape[2]


def _routing(dev, E: int, numel: int, block_m: int, sorted_ids, expert_ids, num_post_padded):
    """The aligned blocks of a batch are on dev, and as long as any routing of numel pairs can be."""
    # the routing's bound on blocks, as mol_align_max_blocks has it (which the call checks again)
    blocks = -(-(numel + min(numel, E + 1) * (block_m - 1)) // block_m) if block_m > 0 else 0
    for t, name, least in ((sorted_ids, "sorted_ids", blocks * block_m),
                           (expert_ids, "expert_ids", blocks),
                           (num_post_padded, "num_post_padded", 1)):
        if t.dtype is not torch.int32 or t.device != dev or not t.is_contiguous():
            _on(dev, name, t, torch.int32, t.shape)
        if t.numel() < least:
            raise ValueError(f"{name} has {t.numel()} entries, fewer than the routing's {least}")


def mol_moe_gemm_q4(xin, row_div: int, W, scales, sorted_ids, expert_ids, num_post_padded,
                    numel: int, block_m: int, out, zeros=None):
    """The base grouped GEMM of a stage into out [numel, N] over 4-bit weights W uint8
    [E, N, K/2] with scales [E, N, K/group] (routing by base expert)."""
    _fit("mol_moe_gemm_q4", row_div, numel, block_m)
    dev = W.device
    N, K, group = _q4(W, scales, zeros, "W", dev)
    E = W.shape[0]
    dtype = scales.dtype
    ld_x = _rows(xin, "xin", dev, dtype, (xin.shape[0], K))
    if row_div < 1:
        raise ValueError(f"row_div must be at least 1, got {row_div}")
    if xin.shape[0] * row_div < numel:
        raise ValueError(f"xin has {xin.shape[0]} rows: {numel} pairs need "
                         f"{-(-numel // row_div)}")
    ld_out = _rows(out, "out", dev, dtype, (numel, N))
    _routing(dev, E, numel, block_m, sorted_ids, expert_ids, num_post_padded)
    _call(dev, "mol_moe_gemm_q4", _dtype_code(scales), xin.data_ptr(), ld_x, row_div,
          W.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(), group, K,
          N, E, sorted_ids.data_ptr(), expert_ids.data_ptr(), num_post_padded.data_ptr(), numel,
          block_m, out.data_ptr(), ld_out)
    return out


def mol_router_balance_workspace_bytes(M: int, num_experts: int) -> int:
    _fit("mol_router_balance_workspace_bytes", M, num_experts)
    v = lib().mol_router_balance_workspace_bytes(M, num_experts)
    if v < 0:
        raise MolError("mol_router_balance_workspace_bytes", -v)
    return int(v)


def new_router_balance_workspace(M: int, num_experts: int, device):
    """A workspace for mol_router_balance at up to M tokens (its contents need no initialisation)."""
    n = mol_router_balance_workspace_bytes(M, num_experts)
    return torch.empty(max(256, n), dtype=torch.uint8, device=device)


def _logits(fn: str, logits, topk: int, scoring: int, token_mask):
    """(M, E, row stride, mask pointer) of a batch's logits."""
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be 2-d with contiguous rows")
    M, E = logits.shape
    _fit(fn, M, E, topk, scoring)
    if token_mask is not None:
        if token_mask.dtype is not torch.bool and token_mask.dtype is not torch.uint8:
            raise TypeError(f"token_mask must be bool or uint8, got {token_mask.dtype}")
        _on(logits.device, "token_mask", token_mask, token_mask.dtype, (M,))
        token_mask = token_mask.data_ptr()
    return M, E, logits.stride(0) if M > 1 else max(logits.stride(0), E), token_mask


def mol_router_balance(logits, topk_ids, scoring: int = MOL_SCORE_SOFTMAX, alpha: float = 1.0,
                       token_mask=None, counts=None, prob_sums=None, loss=None, workspace=None):
    """The balance loss of a routed batch from its logits [M, E] (rows may be strided) and the ids
    [M, topk] chosen over all experts: (loss float32 [1], counts int32 [E + 1] with the number of tokens
    last, prob_sums float32 [E]). token_mask bool or uint8 [M]: 0 for tokens that do not count."""
    dev = logits.device
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids must be 2-d")
    topk = topk_ids.shape[1]
    M, E, ld, mask = _logits("mol_router_balance", logits, topk, scoring, token_mask)
    _on(dev, "topk_ids", topk_ids, torch.int32, (M, topk))
    if counts is None:
        counts = torch.empty(E + 1, dtype=torch.int32, device=dev)
    else:
        _on(dev, "counts", counts, torch.int32, (E + 1,))
    if prob_sums is None:
        prob_sums = torch.empty(E, dtype=torch.float32, device=dev)
    else:
        _on(dev, "prob_sums", prob_sums, torch.float32, (E,))
    if loss is None:
        loss = torch.empty(1, dtype=torch.float32, device=dev)
    else:
        _on(dev, "loss", loss, torch.float32, (1,))
    if workspace is None:
        workspace = new_router_balance_workspace(M, E, dev)
    _on(dev, "workspace", workspace, torch.uint8, workspace.shape)
    _call(dev, "mol_router_balance", _dtype_code(logits), logits.data_ptr(), ld, topk_ids.data_ptr(),
          mask, M, E, topk, scoring, alpha, counts.data_ptr(), prob_sums.data_ptr(), loss.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return loss, counts, prob_sums


def mol_router_balance_grad(logits, counts, topk: int, scoring: int = MOL_SCORE_SOFTMAX,
                            alpha: float = 1.0, token_mask=None, grad_loss=None, out=None):
    """The gradient of mol_router_balance's loss in the logits [M, E] (dtype of logits), from its counts (or
    their sums over ranks); grad_loss float32 [1], the gradient that arrives at the loss (None: 1)."""
    dev = logits.device
    M, E, ld, mask = _logits("mol_router_balance_grad", logits, topk, scoring, token_mask)
    _on(dev, "counts", counts, torch.int32, (E + 1,))
    if grad_loss is not None:
        _on(dev, "grad_loss", grad_loss, torch.float32, (1,))
    if out is None:
        out = torch.empty((M, E), dtype=logits.dtype, device=dev)
    ld_out = _rows(out, "out", dev, logits.dtype, (M, E))
    _call(dev, "mol_router_balance_grad", _dtype_code(logits), logits.data_ptr(), ld, mask,
          counts.data_ptr(), None if grad_loss is None else grad_loss.data_ptr(), M, E, topk, scoring,
          alpha, out.data_ptr(), ld_out)
    return out


def _as_rows(t: torch.Tensor, name: str):
    """(rows, width, row stride) of a tensor of one row dimension or more, the last dimension contiguous."""
    if t.dim() == 2:
        (rows, width), (ld, step) = t.shape, t.stride()
        if step != 1 and width > 1:
            raise ValueError(f"{name} must have contiguous rows")
        return rows, width, ld if rows > 1 else max(ld, width)
    if t.dim() < 2:
        raise ValueError(f"{name} must have rows: at least 2 dimensions")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, or 2-d with contiguous rows")
    width = t.shape[-1]
    return t.numel() // width if width else 0, width, width


def mol_mx4_quantize(x, activation: int = MOL_ACT_NONE, q=None, scales=None):
    """Rows [..., K] of bf16 or fp32 (strided rows if 2-d) as MX4: (q uint8 [..., K/2], scales uint8
    [..., K/32]). MOL_ACT_SILU_MUL: rows [..., 2 K], gate columns first, as SiLU(gate) * up."""
    rows, width, ld = _as_rows(x, "x")
    if activation == MOL_ACT_NONE:
        K = width
    elif activation == MOL_ACT_SILU_MUL:
        K = width // 2
    else:
        raise ValueError(f"unknown activation {activation}")
    if K < 1 or K % 32 or (K != width and width % 2):
        raise ValueError(f"rows of {width} are not whole blocks of 32 values")
    if K > 0x7fffffff:
        raise ValueError(f"mol_mx4_quantize: {K} does not fit 32 bits")
    dev = x.device
    lead = (rows,) if x.dim() == 2 else x.shape[:-1]
    codes_shape, scales_shape = (*lead, K // 2), (*lead, K // 32)
    if q is None:
        q = torch.empty(codes_shape, dtype=torch.uint8, device=dev)
    else:
        _on(dev, "q", q, torch.uint8, codes_shape)
    if scales is None:
        scales = torch.empty(scales_shape, dtype=torch.uint8, device=dev)
    else:
        _on(dev, "scales", scales, torch.uint8, scales_shape)
    _call(dev, "mol_mx4_quantize", _dtype_code(x), activation, x.data_ptr(), ld, rows, K, q.data_ptr(),
          scales.data_ptr())
    return q, scales


def mol_mx4_dequantize(q, scales, dtype=torch.bfloat16, out=None):
    """The values [..., K] of MX4 codes q uint8 [..., K/2] and scales uint8 [..., K/32], in dtype (that of
    out, whose rows may be strided if 2-d)."""
    dev, shape = q.device, q.shape
    if len(shape) < 2:
        raise ValueError("q must have rows: at least 2 dimensions")
    lead, K = shape[:-1], 2 * shape[-1]
    if K < 1 or K % 32:
        raise ValueError(f"rows of {K} are not whole blocks of 32 values")
    if K > 0x7fffffff:
        raise ValueError(f"mol_mx4_dequantize: {K} does not fit 32 bits")
    _on(dev, "q", q, torch.uint8, shape)
    _on(dev, "scales", scales, torch.uint8, (*lead, K // 32))
    if out is None:
        out = torch.empty((*lead, K), dtype=dtype, device=dev)
    elif out.shape != (*lead, K) or out.device != dev:
        raise ValueError(f"out must be {(*lead, K)} on {dev}, got {tuple(out.shape)} on {out.device}")
    rows, _, ld = _as_rows(out, "out")
    _call(dev, "mol_mx4_dequantize", _dtype_code(out), q.data_ptr(), scales.data_ptr(), rows, K,
          out.data_ptr(), ld)
    return out


def mol_moe_gemm_mx4(xin, row_div: int, W, scales, sorted_ids, expert_ids, num_post_padded,
                     numel: int, block_m: int, out, x_scales=None):
    """The base grouped GEMM of a stage into out [numel, N] (bf16 or fp32) over MX4 weights W uint8
    [E, N, K/2] with scales uint8 [E, N, K/32] (routing by base expert). xin: rows [., K] in the dtype of
    out, or with x_scales uint8 [., K/32] rows of MX4 codes uint8 [., K/2]."""
    _fit("mol_moe_gemm_mx4", row_div, numel, block_m)
    dev = W.device
    if W.dim() != 3:
        raise ValueError("W must be [E, N, K/2]")
    E, N, half = W.shape
    K = 2 * half
    _fit("mol_moe_gemm_mx4", E, N, K)
    if K < 1 or K % 32:
        raise ValueError(f"W: rows of {K} are not whole blocks of 32 values")
    _on(dev, "W", W, torch.uint8, (E, N, half))
    _on(dev, "scales", scales, torch.uint8, (E, N, K // 32))
    if xin.dim() != 2:
        raise ValueError("xin must be 2-d")
    rows, dtype = xin.shape[0], out.dtype
    if x_scales is None:
        ld_x = _rows(xin, "xin", dev, dtype, (rows, K))
    else:
        ld_x = 2 * _rows(xin, "xin", dev, torch.uint8, (rows, half))
        ld_s = _rows(x_scales, "x_scales", dev, torch.uint8, (rows, K // 32))
        if rows > 1 and ld_s * 32 != ld_x:
            raise ValueError(f"rows of xin are {ld_x} values apart, rows of x_scales {ld_s * 32}")
        if rows == 1:
            ld_x = K
    if row_div < 1:
        raise ValueError(f"row_div must be at least 1, got {row_div}")
    if rows * row_div < numel:
        raise ValueError(f"xin has {rows} rows: {numel} pairs need {-(-numel // row_div)}")
    ld_out = _rows(out, "out", dev, dtype, (numel, N))
    _routing(dev, E, numel, block_m, sorted_ids, expert_ids, num_post_padded)
    _call(dev, "mol_moe_gemm_mx4", _dtype_code(out), xin.data_ptr(), ld_x,
          None if x_scales is None else x_scales.data_ptr(), row_div, W.data_ptr(), scales.data_ptr(),
          K, N, E, sorted_ids.data_ptr(), expert_ids.data_ptr(), num_post_padded.data_ptr(), numel,
          block_m, out.data_ptr(), ld_out)
    return out


class _MoeWeightsC(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("dtype", "group", "num_experts", "hidden", "inter",
                                     "reserved")] +
                [(n, _P) for n in ("gate_up", "down", "gate_up_scales", "down_scales",
                                   "gate_up_zeros", "down_zeros")])


class _MoeAdaptersC(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("num_slots", "rank")] +
                [(n, _P) for n in ("gate_up_A", "gate_up_B", "down_A", "down_B", "slot_scale",
                                   "slot_ranks")])


class MoeWeights:
    """The base weights of a layer as mol_moe_layer takes them, described once: gate_up [E,
    2*inter, hidden] and down [E, hidden, inter] (bf16 or fp32), or packed 4-bit (uint8, last
    dimension halved) with scales and, optionally, zeros. Keeps the tensors alive."""

    def __init__(self, gate_up, down, gate_up_scales=None, down_scales=None,
                 gate_up_zeros=None, down_zeros=None):
        dev = gate_up.device
        q4 = gate_up_scales is not None or down_scales is not None
        if gate_up.dim() != 3 or down.dim() != 3:
            raise ValueError("gate_up and down must be 3-d")
        E, N1, _ = gate_up.shape
        if q4:
            if gate_up_scales is None or down_scales is None:
                raise ValueError("4-bit weights need both scales")
            N1, H, group = _q4(gate_up, gate_up_scales, gate_up_zeros, "gate_up", dev)
            N2, inter, g2 = _q4(down, down_scales, down_zeros, "down", dev)
            if g2 != group or down_scales.dtype != gate_up_scales.dtype:
                raise ValueError("gate_up and down must have one group size and scale dtype")
            self.dtype = gate_up_scales.dtype
        else:
            if gate_up_zeros is not None or down_zeros is not None:
                raise ValueError("zeros without scales")
            H, group = gate_up.shape[2], 0
            N2, inter = down.shape[1], down.shape[2]
            self.dtype = gate_up.dtype
            _on(dev, "gate_up", gate_up, self.dtype, (E, N1, H))
            _on(dev, "down", down, self.dtype, (E, N2, inter))
        if N1 != 2 * inter or N2 != H or down.shape[0] != E:
            raise ValueError(f"gate_up {tuple(gate_up.shape)} and down {tuple(down.shape)} are "
                             "not one layer's")
        self.device, self.num_experts, self.hidden, self.inter = dev, E, H, inter
        self.tensors = (gate_up, down, gate_up_scales, down_scales, gate_up_zeros, down_zeros)
        self.c = _MoeWeightsC(_dtype_code(gate_up_scales if q4 else gate_up), group, E, H, inter,
                              0, *(None if t is None else t.data_ptr() for t in self.tensors))


class MoeAdapters:
    """The adapters of a layer as mol_moe_layer takes them: gate_up_A [E*S, 2r, hidden],
    gate_up_B [E*S, 2*inter, r], down_A [E*S, r, inter], down_B [E*S, hidden, r], slot_scale
    [S], slot_ranks [S] or None. Keeps the tensors alive."""

    def __init__(self, gate_up_A, gate_up_B, down_A, down_B, slot_scale, slot_ranks=None):
        dev, dt = gate_up_A.device, gate_up_A.dtype
        _dtype_code(gate_up_A)
        S = slot_scale.shape[0]
        V, r2, H = gate_up_A.shape
        r, inter = r2 // 2, down_A.shape[2]
        if S < 1 or V % S:
            raise ValueError(f"{V} virtual experts are not a multiple of {S} slots")
        for t, name, shape in ((gate_up_A, "gate_up_A", (V, 2 * r, H)),
                               (gate_up_B, "gate_up_B", (V, 2 * inter, r)),
                               (down_A, "down_A", (V, r, inter)), (down_B, "down_B", (V, H, r))):
            _on(dev, name, t, dt, shape)
        _on(dev, "slot_scale", slot_scale, torch.float32, (S,))
        if slot_ranks is not None:
            _on(dev, "slot_ranks", slot_ranks, torch.int32, (S,))
        self.device, self.dtype, self.num_slots, self.rank = dev, dt, S, r
        self.num_virtual, self.hidden, self.inter = V, H, inter
        self.tensors = (gate_up_A, gate_up_B, down_A, down_B, slot_scale, slot_ranks)
        self.c = _MoeAdaptersC(S, r, *(None if t is None else t.data_ptr()
                                       for t in self.tensors))


def mol_moe_layer_workspace_bytes(w: MoeWeights, M: int, topk: int, adapters=None) -> int:
    _fit("mol_moe_layer_workspace_bytes", M, topk)
    v = lib().mol_moe_layer_workspace_bytes(w.c.dtype, M, topk, w.hidden, w.inter,
                                            0 if adapters is None else adapters.rank)
    if v < 0:
        raise MolError("mol_moe_layer_workspace_bytes", -v)
    return int(v)


def new_moe_layer_workspace(w: MoeWeights, M: int, topk: int, adapters=None):
    """A workspace for mol_moe_layer at up to M tokens (its contents need no initialisation)."""
    n = mol_moe_layer_workspace_bytes(w, M, topk, adapters)
    return torch.empty(max(256, n), dtype=torch.uint8, device=w.device)


def mol_moe_layer(w: MoeWeights, x, topk_ids, topk_weights, adapters=None, lora_ids=None,
                  y=None, workspace=None):
    """A whole layer for a few tokens: y [M, hidden] from x [M, hidden] and its routing."""
    dev = w.device
    M, topk = topk_ids.shape
    _fit("mol_moe_layer", M, topk)
    ld_x = _rows(x, "x", dev, w.dtype, (M, w.hidden))
    _on(dev, "topk_ids", topk_ids, torch.int32, (M, topk))
    _on(dev, "topk_weights", topk_weights, torch.float32, (M, topk))
    if adapters is not None:
        if (adapters.dtype != w.dtype or adapters.device != dev or adapters.hidden != w.hidden or
                adapters.inter != w.inter or
                adapters.num_virtual != w.num_experts * adapters.num_slots):
            raise ValueError("the adapters are not for these weights")
        if lora_ids is None:
            raise ValueError("adapters need lora_ids")
        _on(dev, "lora_ids", lora_ids, torch.int32, (M,))
    elif lora_ids is not None:
        raise ValueError("lora_ids without adapters")
    if y is None:
        y = torch.empty((M, w.hidden), dtype=w.dtype, device=dev)
    ld_y = _rows(y, "y", dev, w.dtype, (M, w.hidden))
    if workspace is None:
        workspace = new_moe_layer_workspace(w, M, topk, adapters)
    _on(dev, "workspace", workspace, torch.uint8, workspace.shape)
    _call(dev, "mol_moe_layer", ctypes.addressof(w.c),
          None if adapters is None else ctypes.addressof(adapters.c), x.data_ptr(), ld_x,
          topk_ids.data_ptr(), topk_weights.data_ptr(),
          None if lora_ids is None else lora_ids.data_ptr(), M, topk, y.data_ptr(), ld_y,
          workspace.data_ptr(), workspace.numel())
    return y
