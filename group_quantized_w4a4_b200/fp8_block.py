"""Block-scaled FP8, expert and block-norm entry points of the C ABI (include/apex_w4a4.h).

As in the package itself, every ``apex_*`` function has the name and arguments of the C entry
point with torch CUDA tensors for device pointers, and the functions without the prefix
allocate their outputs and workspaces (from torch's caching allocator, on the call's stream).
Tensors are contiguous and on one device, which the call makes current while it launches;
``stream`` defaults to that device's current stream.
"""
from __future__ import annotations

import ctypes

import torch

APEX_DTYPE_F16 = 0
APEX_DTYPE_BF16 = 1
APEX_DTYPE_F32 = 2
APEX_SCORE_SOFTMAX = 0
APEX_SCORE_SIGMOID = 1
APEX_GROUP_MAX = 0x100
APEX_MAX_EXPERTS = 512
APEX_MAX_TOP_K = 32

ENTRY_POINTS = [
    "apex_quantize_act_fp8_block", "apex_pack_weights_fp8_block", "apex_gemm_fp8_block",
    "apex_linear_fp8_block", "apex_linear_fp8_block_workspace_size", "apex_route_experts",
    "apex_plan_experts", "apex_route_plan_experts", "apex_moe_mlp_fp8_block", "apex_moe_mlp_fp8_block_workspace_size",
    "apex_block_norm",
]
CONVENIENCES = [
    "quantize_act_fp8_block", "pack_weights_fp8_block", "gemm_fp8_block", "linear_fp8_block",
    "route_experts", "plan_experts", "moe_mlp_fp8_block", "block_norm",
]
__all__ = ENTRY_POINTS + CONVENIENCES

_DTYPES = {torch.float16: APEX_DTYPE_F16, torch.bfloat16: APEX_DTYPE_BF16,
           torch.float32: APEX_DTYPE_F32}
_GROUP_SCORES = {"top2": 0, "max": APEX_GROUP_MAX}
_SCORES = {"softmax": APEX_SCORE_SOFTMAX, "sigmoid": APEX_SCORE_SIGMOID}


def _lib():
    from . import load_library
    return load_library()


def _check_stream(stream, tensor):
    """A stream of another device would leave the call on that device's own current stream, which
    the caller's waits do not order."""
    if tensor is not None and stream.device_index != tensor.get_device():
        raise ValueError("expected a stream of the tensors' device")


def _call(name, tensors, args, stream):
    """Launch entry point `name`: `tensors` are the tensor arguments (None where absent), all on
    one device; `args(p)` lists the C arguments but the stream, p the device pointers."""
    from . import ApexError
    device = None
    pointers = []
    for t in tensors:
        if t is None:
            pointers.append(None)
            continue
        if not t.is_cuda:
            raise ValueError("expected a CUDA tensor (device memory)")
        if not t.is_contiguous():
            raise ValueError("expected a contiguous tensor")
        index = t.get_device()
        if device is None:
            device = index
        elif device != index:
            raise ValueError("expected tensors on one device")
        pointers.append(t.data_ptr())
    fn = getattr(_lib(), name)
    if stream is not None and stream.device_index != device:
        raise ValueError("expected a stream of the tensors' device")
    if device == torch.cuda.current_device():
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream
        code = fn(*args(pointers), s)
    else:
        with torch.cuda.device(device):
            s = torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream
            code = fn(*args(pointers), s)
    if code != 0:
        raise ApexError(code, name)


def _dtype(t):
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise ValueError(f"expected fp16, bf16 or fp32, got {t.dtype}") from None


# ------------------------------------------------------------------ the torch binding

_native = None
# the entry points that the binding calls, in the order of its table
_BOUND = ["apex_quantize_act_fp8_block", "apex_gemm_fp8_block", "apex_linear_fp8_block",
          "apex_linear_fp8_block_workspace_size", "apex_route_experts", "apex_plan_experts",
          "apex_route_plan_experts", "apex_moe_mlp_fp8_block",
          "apex_moe_mlp_fp8_block_workspace_size", "apex_block_norm"]


def _load():
    """The compiled binding (csrc/torch_binding.cpp), built first if it is missing or stale."""
    global _native
    if _native is None:
        import importlib.machinery
        import importlib.util

        from . import ApexError, build
        lib = _lib()
        path = build.build_torch()
        loader = importlib.machinery.ExtensionFileLoader("apex_torch", path)
        spec = importlib.util.spec_from_loader("apex_torch", loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        module.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _BOUND),
                    ApexError)
        _native = module
    return _native


def _run(name, stream, *args):
    """Call `name` of the binding, on `stream` when one is given (its outputs and workspaces then
    belong to that stream too)."""
    fn = getattr(_native or _load(), name)
    if stream is None:
        return fn(*args)
    _check_stream(stream, next((a for a in args if isinstance(a, torch.Tensor)), None))
    with torch.cuda.stream(stream):
        return fn(*args)


# ------------------------------------------------------------------ the C entry points

def apex_quantize_act_fp8_block(x, M, K, codes, scales_f32, stream=None):
    _call("apex_quantize_act_fp8_block", (x, codes, scales_f32),
          lambda p: (p[0], _dtype(x), M, K, p[1], p[2]), stream)


def apex_pack_weights_fp8_block(w, E, N, K, codes, scales_f32, stream=None):
    _call("apex_pack_weights_fp8_block", (w, codes, scales_f32),
          lambda p: (p[0], _dtype(w), E, N, K, p[1], p[2]), stream)


def apex_gemm_fp8_block(M, N, K, a_codes, a_scales, w_codes, w_scales, y, stream=None):
    _call("apex_gemm_fp8_block", (a_codes, a_scales, w_codes, w_scales, y),
          lambda p: (M, N, K, p[0], p[1], p[2], p[3], _dtype(y), p[4]), stream)


def apex_linear_fp8_block_workspace_size(M, N, K) -> int:
    return int(_lib().apex_linear_fp8_block_workspace_size(M, N, K))


def apex_linear_fp8_block(M, N, K, x, w_codes, w_scales, y, workspace, workspace_bytes=None,
                          stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _call("apex_linear_fp8_block", (x, w_codes, w_scales, y, workspace),
          lambda p: (M, N, K, p[0], _dtype(x), p[1], p[2], p[3], p[4], workspace_bytes), stream)


def apex_route_experts(logits, T, E, k, score, bias_f32, groups, topk_groups, renormalize, scale,
                       mask_u8, weights_f32, ids_i32, stream=None):
    _call("apex_route_experts", (logits, bias_f32, mask_u8, weights_f32, ids_i32),
          lambda p: (p[0], _dtype(logits), T, E, k, score, p[1], groups, topk_groups,
                     1 if renormalize else 0, scale, p[2], p[3], p[4]), stream)


def apex_route_plan_experts(logits, T, E, k, score, bias_f32, groups, topk_groups, renormalize,
                            scale, mask_u8, weights_f32, ids_i32, offsets_i32, order_i32,
                            stream=None):
    _call("apex_route_plan_experts",
          (logits, bias_f32, mask_u8, weights_f32, ids_i32, offsets_i32, order_i32),
          lambda p: (p[0], _dtype(logits), T, E, k, score, p[1], groups, topk_groups,
                     1 if renormalize else 0, scale, *p[2:]), stream)


def apex_plan_experts(ids_i32, T, k, E, offsets_i32, order_i32, stream=None):
    _call("apex_plan_experts", (ids_i32, offsets_i32, order_i32),
          lambda p: (p[0], T, k, E, p[1], p[2]), stream)


def apex_moe_mlp_fp8_block_workspace_size(T, E, k, H, I) -> int:
    return int(_lib().apex_moe_mlp_fp8_block_workspace_size(T, E, k, H, I))


def apex_moe_mlp_fp8_block(T, E, k, H, I, x, weights_f32, ids_i32, offsets_i32, order_i32,
                           w13_codes, w13_scales, w2_codes, w2_scales, y, workspace,
                           workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _call("apex_moe_mlp_fp8_block",
          (x, weights_f32, ids_i32, offsets_i32, order_i32, w13_codes, w13_scales, w2_codes,
           w2_scales, y, workspace),
          lambda p: (T, E, k, H, I, p[0], _dtype(x), *p[1:], workspace_bytes), stream)


def apex_block_norm(x, T, H, residual, post_weight, gate, gate_rows, alpha, pre_weight, eps,
                    weight_offset, h, y, y_codes, y_scales_f32, stream=None):
    _call("apex_block_norm",
          (x, residual, post_weight, gate, pre_weight, h, y, y_codes, y_scales_f32),
          lambda p: (p[0], _dtype(x), T, H, p[1], p[2], p[3], gate_rows, alpha, p[4], eps,
                     weight_offset, p[5], p[6], p[7], p[8]), stream)


# ------------------------------------------------------------------ tensor conveniences

def quantize_act_fp8_block(x, stream=None):
    """fp16 / bf16 [M, K] -> (E4M3 codes uint8 [M, K], scales fp32 [M, ceil(K/128)])."""
    return _run("quantize_act", stream, x)


def pack_weights_fp8_block(w, stream=None):
    """fp16 / bf16 / fp32 [..., N, K] -> (E4M3 codes uint8 of w's shape, scales fp32
    [..., ceil(N/128), ceil(K/128)])."""
    N, K = w.shape[-2:]
    if stream is not None:
        _check_stream(stream, w)
    with torch.cuda.stream(stream):   # None: the current one
        codes = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
        scales = torch.empty((*w.shape[:-2], -(-N // 128), -(-K // 128)), dtype=torch.float32,
                             device=w.device)
        if w.numel():
            apex_pack_weights_fp8_block(w, w.numel() // (N * K), N, K, codes, scales)
    return codes, scales


def gemm_fp8_block(a_codes, a_scales, w_codes, w_scales, dtype=None, out=None, stream=None):
    """Y = block-scaled FP8 GEMM of quantized operands -> [M, N] of `dtype` (fp16 or bf16; None:
    out's, or bf16)."""
    if dtype is None:
        dtype = torch.bfloat16 if out is None else out.dtype
    elif out is not None and dtype != out.dtype:
        raise ValueError(f"dtype: out is {out.dtype}, not {dtype}")
    if dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"dtype: expected fp16 or bf16, got {dtype}")
    return _run("gemm", stream, a_codes, a_scales, w_codes, w_scales, dtype == torch.bfloat16,
                out)


def linear_fp8_block(x, w_codes, w_scales, out=None, stream=None):
    """y = x . W^T for x fp16 / bf16 [M, K], W from pack_weights_fp8_block -> [M, N] like x."""
    return _run("linear", stream, x, w_codes, w_scales, out)


def route_experts(logits, k, bias=None, score="softmax", groups=1, topk_groups=1,
                  renormalize=True, scale=1.0, mask=None, plan=False, stream=None,
                  group_score="top2"):
    """logits [T, E] -> (weights fp32 [T, k], ids int32 [T, k]); with plan also (offsets, order)
    of plan_experts.  bias fp32 [E]; mask bool [T] (False: the token takes no part).  group_score:
    a group is worth the sum of its two largest values ("top2") or its largest ("max")."""
    if score not in _SCORES:
        raise ValueError(f"score: expected one of {sorted(_SCORES)}, got {score!r}")
    if group_score not in _GROUP_SCORES:
        raise ValueError(f"group_score: expected one of {sorted(_GROUP_SCORES)}, got {group_score!r}")
    return _run("route", stream, logits, k, bias, _SCORES[score] | _GROUP_SCORES[group_score],
                groups, topk_groups, renormalize, scale, mask, plan)


def plan_experts(ids, experts, stream=None):
    """ids int32 [T, k] -> (offsets int32 [experts + 1], order int32 [T * k])."""
    return _run("plan", stream, ids, experts)


def moe_mlp_fp8_block(x, weights, ids, offsets, order, w13_codes, w13_scales, w2_codes,
                      w2_scales, out=None, stream=None):
    """The experts' gated MLP of x fp16 / bf16 [T, H] -> [T, H] like x.  weights, ids, offsets,
    order from route_experts(..., plan=True); w13 [E, 2, I, H] (gate, up) and w2 [E, H, I] from
    pack_weights_fp8_block."""
    return _run("moe", stream, x, weights, ids, offsets, order, w13_codes, w13_scales, w2_codes,
                w2_scales, out)


_NORM_OUT = {"codes": (False, True), "values": (True, False), "both": (True, True),
             "residual": (False, False)}


def block_norm(x, pre_weight=None, residual=None, post_weight=None, gate=None, alpha=1.0,
               eps=1e-6, weight_offset=0.0, out="codes", stream=None):
    """x [T, H] -> (h, y, codes, scales): the norm behind a block, gate, scaled residual and the
    norm before the next one.  out: "codes" (y None), "values" (codes and scales None), "both", or
    "residual" (h alone, without the second norm).  gate [rows, H], rows dividing T."""
    if out not in _NORM_OUT:
        raise ValueError(f"out: expected one of {sorted(_NORM_OUT)}, got {out!r}")
    if out != "residual" and pre_weight is None:
        raise ValueError(f"out={out!r} needs pre_weight")
    return _run("norm", stream, x, pre_weight, residual, post_weight, gate, alpha, eps,
                weight_offset, *_NORM_OUT[out])
