"""Python binding of libmoe.so: the MI355X MoE layer forward (C ABI in include/moe.h).

Argument marshalling only: every step runs in the library's HIP kernels.
Tensors are torch tensors on the GPU (PyTorch supplies device memory and the
stream); bf16 tensors may be torch.bfloat16 or 16-bit integer views of the
bit patterns. Every call checks the returned status and raises MoeError.
There is no fallback: without the compiled library every call fails.
"""
import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "moe.h")

STATUS = {0: "MOE_SUCCESS", 1: "MOE_ERROR_INVALID_VALUE", 2: "MOE_ERROR_UNSUPPORTED",
          3: "MOE_ERROR_WORKSPACE", 4: "MOE_ERROR_LAUNCH"}


class MoeError(RuntimeError):
    def __init__(self, fn, status, detail=""):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}{detail}")
        self.status = status


_lib = None
_I32 = ctypes.c_int32
_VP = ctypes.c_void_p
_SZ = ctypes.c_size_t

_SIGS = {
    "moe_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "moe_last_launch_error": ([], ctypes.c_char_p),
    "moe_partition": ([_I32, _I32, _I32, ctypes.POINTER(_I32), ctypes.POINTER(_I32)], ctypes.c_int),
    "moe_workspace_size": ([_I32] * 6 + [ctypes.POINTER(_SZ)], ctypes.c_int),
    "moe_router_logits": ([_VP, _VP, _VP, _I32, _I32, _I32, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_route": ([_VP, _I32, _I32, _I32, _VP, _VP, _VP], ctypes.c_int),
    "moe_permute": ([_VP, _I32, _I32, _I32, _I32, _I32, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
                    ctypes.c_int),
    "moe_route_permute": ([_VP, _I32, _I32, _I32, _I32, _I32] + [_VP] * 7 + [_SZ, _VP],
                          ctypes.c_int),
    "moe_route_permute_variant": ([_VP, _I32, _I32, _I32, _I32, _I32] + [_VP] * 7 +
                                  [_SZ, _I32, _VP], ctypes.c_int),
    "moe_routing_plan": ([_I32, _I32, _I32, _I32, ctypes.POINTER(_I32)], ctypes.c_int),
    "moe_grouped_ffn": ([_VP, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _VP, _VP, _VP, _VP, _SZ,
                         _VP], ctypes.c_int),
    "moe_grouped_ffn_fp8": ([_VP, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _VP, _VP, _VP, _VP, _VP,
                             _VP, _SZ, _VP], ctypes.c_int),
    "moe_combine": ([_VP, _VP, _VP, _I32, _I32, _I32, _VP, _VP], ctypes.c_int),
    "moe_forward": ([_VP, _VP, _VP, _VP, _VP] + [_I32] * 7 + [_VP, _VP, _VP, _VP, _VP, _SZ, _VP],
                    ctypes.c_int),
    "moe_forward_fp8": ([_VP] * 7 + [_I32] * 7 + [_VP, _VP, _VP, _VP, _VP, _SZ, _VP],
                        ctypes.c_int),
    "moe_grouped_matmul": ([_VP, _VP, _VP] + [_I32] * 6 + [_VP, _VP, _I32, _VP], ctypes.c_int),
    "moe_grouped_matmul_dx": ([_VP, _VP] + [_I32] * 4 + [_VP, _VP, _I32, _VP], ctypes.c_int),
    "moe_grouped_matmul_dw": ([_VP] * 4 + [_I32] * 6 + [_VP, _I32, _VP], ctypes.c_int),
    "moe_rms_norm": ([_VP, _VP, _VP, ctypes.c_float, _I32, _I32] + [_VP] * 5, ctypes.c_int),
    "moe_rms_norm_backward_workspace_size": ([_I32, _I32, ctypes.POINTER(_SZ)], ctypes.c_int),
    "moe_rms_norm_backward": ([_VP, _VP, _VP, ctypes.c_float, _I32, _I32] + [_VP] * 4 +
                              [_SZ, _VP], ctypes.c_int),
    "moe_quantize_mx": ([_VP, _I32, _I32, _I32, _I32, _VP, _VP, _VP], ctypes.c_int),
    "moe_swiglu_quantize_mx": ([_VP, _I32, _I32, _I32, _VP, _I32, _VP, _VP, _VP], ctypes.c_int),
    "moe_dequantize_mx": ([_VP, _VP, _I32, _I32, _I32, _VP, _I32, _VP], ctypes.c_int),
    "moe_grouped_matmul_mx": ([_VP, _VP, _I32, _VP, _VP] + [_I32] * 6 +
                              [_VP, _VP, _VP, _I32, _VP], ctypes.c_int),
    "moe_forward_no_alloc": ([_VP, _VP, _VP, _VP, _VP] + [_I32] * 7 + [_VP, _VP, _VP, _VP, _VP],
                             ctypes.c_int),
}

NO_ALLOC_SCRATCH_BYTES = 128 << 20


def lib():
    """Load libmoe.so (built in place by routing_grouped_expert_amd.build).

    torch is imported first: it carries its own HIP runtime under the same
    soname as the system one that libmoe.so names, and whichever is loaded
    first serves the whole process. Loading the library first would hand
    torch a runtime it was not built against (it then finds no GPU)."""
    global _lib
    if _lib is None:
        import torch  # noqa: F401  (see above)
        if not os.path.exists(LIB_PATH):
            from . import build
            build.build()
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _check(fn, st):
    if st != 0:
        detail = ""
        if st == 4:
            detail = f" ({lib().moe_last_launch_error().decode()})"
        raise MoeError(fn, st, detail)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, shape, esize, optional=False):
    """Raise ValueError unless t is a contiguous GPU tensor of `shape` whose
    elements are `esize` bytes (None allowed when optional). Checked before
    every call, so a host tensor, a strided view or a wrong shape never
    reaches a kernel."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.element_size() != esize:
        raise ValueError(f"{name} must have {esize}-byte elements, not {t.element_size()}")
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _need_ws(ws):
    if ws is None:
        return 0
    if not getattr(ws, "is_cuda", False) or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous GPU tensor")
    return ws.numel() * ws.element_size()


def _dims(t, name, nd):
    if t is None or t.dim() != nd:
        raise ValueError(f"{name} must be a {nd}-d tensor")
    return tuple(t.shape)


def _stream(stream):
    if stream is None:
        torch = _torch()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:  # the handle alone: a Stream object costs a few us a call
            return raw(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def partition(num_experts, num_shares, share):
    """(first_expert, num_local) of a contiguous ceil/floor expert share."""
    f, c = _I32(), _I32()
    _check("moe_partition", lib().moe_partition(num_experts, num_shares, share, ctypes.byref(f),
                                                ctypes.byref(c)))
    return f.value, c.value


def workspace_size(T, H, I, E, k, num_local):
    n = _SZ()
    _check("moe_workspace_size", lib().moe_workspace_size(T, H, I, E, k, num_local,
                                                          ctypes.byref(n)))
    return n.value


def router_logits(x, w_gate, bias, logits, ws, stream=None):
    T, H = _dims(x, "x", 2)
    E = _dims(w_gate, "w_gate", 2)[0]
    _need(x, "x", (T, H), 2)
    _need(w_gate, "w_gate", (E, H), 4)
    _need(bias, "bias", (E,), 4, optional=True)
    _need(logits, "logits", (T, E), 4)
    nws = _need_ws(ws)
    _check("moe_router_logits", lib().moe_router_logits(
        _ptr(x), _ptr(w_gate), _ptr(bias), T, H, E, _ptr(logits), _ptr(ws), nws,
        _stream(stream)))


def route(logits, k, topk_ids, topk_weights, stream=None):
    T, E = _dims(logits, "logits", 2)
    _need(logits, "logits", (T, E), 4)
    _need(topk_ids, "topk_ids", (T, k), 4)
    _need(topk_weights, "topk_weights", (T, k), 4)
    _check("moe_route", lib().moe_route(_ptr(logits), T, E, k, _ptr(topk_ids),
                                        _ptr(topk_weights), _stream(stream)))


def permute(topk_ids, num_experts, first_expert, num_local, expert_counts, expert_offsets,
            permuted_rows, expanded_to_permuted, ws, stream=None):
    T, k = _dims(topk_ids, "topk_ids", 2)
    _need(topk_ids, "topk_ids", (T, k), 4)
    _need(expert_counts, "expert_counts", (num_experts,), 4)
    _need(expert_offsets, "expert_offsets", (num_local + 1,), 4)
    _need(permuted_rows, "permuted_rows", (T * k,), 4)
    _need(expanded_to_permuted, "expanded_to_permuted", (T * k,), 4)
    nws = _need_ws(ws)
    _check("moe_permute", lib().moe_permute(
        _ptr(topk_ids), T, k, num_experts, first_expert, num_local, _ptr(expert_counts),
        _ptr(expert_offsets), _ptr(permuted_rows), _ptr(expanded_to_permuted), _ptr(ws), nws,
        _stream(stream)))


ROUTING_VARIANTS = {"auto": 0, "one_block": 1, "two_kernels": 2, "tiled": 3}


def routing_plan(T, E, k, num_local):
    """Name of the routing variant moe_route_permute runs for these sizes."""
    v = _I32()
    _check("moe_routing_plan", lib().moe_routing_plan(T, E, k, num_local, ctypes.byref(v)))
    return {c: n for n, c in ROUTING_VARIANTS.items()}[v.value]


def route_permute(logits, k, first_expert, num_local, topk_ids, topk_weights, expert_counts,
                  expert_offsets, permuted_rows, expanded_to_permuted, ws, stream=None,
                  variant="auto"):
    """moe_route_permute: routing then the permutation, in one call (variant:
    a key of ROUTING_VARIANTS; "auto" is the plan)."""
    T, E = _dims(logits, "logits", 2)
    _need(logits, "logits", (T, E), 4)
    _need(topk_ids, "topk_ids", (T, k), 4)
    _need(topk_weights, "topk_weights", (T, k), 4)
    _need(expert_counts, "expert_counts", (E,), 4)
    _need(expert_offsets, "expert_offsets", (num_local + 1,), 4)
    _need(permuted_rows, "permuted_rows", (T * k,), 4)
    _need(expanded_to_permuted, "expanded_to_permuted", (T * k,), 4)
    nws = _need_ws(ws)
    if variant == "auto":
        _check("moe_route_permute", lib().moe_route_permute(
            _ptr(logits), T, E, k, first_expert, num_local, _ptr(topk_ids), _ptr(topk_weights),
            _ptr(expert_counts), _ptr(expert_offsets), _ptr(permuted_rows),
            _ptr(expanded_to_permuted), _ptr(ws), nws, _stream(stream)))
        return
    _check("moe_route_permute_variant", lib().moe_route_permute_variant(
        _ptr(logits), T, E, k, first_expert, num_local, _ptr(topk_ids), _ptr(topk_weights),
        _ptr(expert_counts), _ptr(expert_offsets), _ptr(permuted_rows),
        _ptr(expanded_to_permuted), _ptr(ws), nws, ROUTING_VARIANTS[variant], _stream(stream)))


def _ffn_common(x, permuted_rows, expert_offsets, k, w2, expert_out):
    T, H = _dims(x, "x", 2)
    L = _dims(expert_offsets, "expert_offsets", 1)[0] - 1
    I = _dims(w2, "w2", 3)[2]
    _need(x, "x", (T, H), 2)
    _need(permuted_rows, "permuted_rows", (T * k,), 4)
    _need(expert_offsets, "expert_offsets", (L + 1,), 4)
    _need(expert_out, "expert_out", (T * k, H), 4)
    return T, H, L, I


def grouped_ffn(x, permuted_rows, expert_offsets, k, w1, w2, expert_out, ws, stream=None):
    T, H, L, I = _ffn_common(x, permuted_rows, expert_offsets, k, w2, expert_out)
    _need(w1, "w1", (L, 2 * I, H), 2)
    _need(w2, "w2", (L, H, I), 2)
    nws = _need_ws(ws)
    _check("moe_grouped_ffn", lib().moe_grouped_ffn(
        _ptr(x), _ptr(permuted_rows), _ptr(expert_offsets), L, T, k, H, I, _ptr(w1), _ptr(w2),
        _ptr(expert_out), _ptr(ws), nws, _stream(stream)))


def grouped_ffn_fp8(x, permuted_rows, expert_offsets, k, w1q, w1s, w2q, w2s, expert_out, ws,
                    stream=None):
    """moe_grouped_ffn_fp8: w1q [L, 2I, H] and w2q [L, H, I] uint8 E4M3 codes,
    w1s [L, 2I] and w2s [L, H] fp32 row scales."""
    T, H, L, I = _ffn_common(x, permuted_rows, expert_offsets, k, w2q, expert_out)
    _need(w1q, "w1q", (L, 2 * I, H), 1)
    _need(w1s, "w1s", (L, 2 * I), 4)
    _need(w2q, "w2q", (L, H, I), 1)
    _need(w2s, "w2s", (L, H), 4)
    nws = _need_ws(ws)
    _check("moe_grouped_ffn_fp8", lib().moe_grouped_ffn_fp8(
        _ptr(x), _ptr(permuted_rows), _ptr(expert_offsets), L, T, k, H, I, _ptr(w1q), _ptr(w1s),
        _ptr(w2q), _ptr(w2s), _ptr(expert_out), _ptr(ws), nws, _stream(stream)))


def combine(expert_out, expanded_to_permuted, topk_weights, y, stream=None):
    T, k = _dims(topk_weights, "topk_weights", 2)
    H = _dims(y, "y", 2)[1]
    _need(topk_weights, "topk_weights", (T, k), 4)
    _need(y, "y", (T, H), 2)
    _need(expert_out, "expert_out", (T * k, H), 4)
    _need(expanded_to_permuted, "expanded_to_permuted", (T * k,), 4)
    _check("moe_combine", lib().moe_combine(_ptr(expert_out), _ptr(expanded_to_permuted),
                                            _ptr(topk_weights), T, k, H, _ptr(y),
                                            _stream(stream)))


def _forward_common(x, w_gate, router_bias, k, y, logits_out, topk_ids_out, topk_weights_out):
    T, H = _dims(x, "x", 2)
    E = _dims(w_gate, "w_gate", 2)[0]
    _need(x, "x", (T, H), 2)
    _need(w_gate, "w_gate", (E, H), 4)
    _need(router_bias, "router_bias", (E,), 4, optional=True)
    _need(y, "y", (T, H), 2)
    _need(logits_out, "logits_out", (T, E), 4, optional=True)
    _need(topk_ids_out, "topk_ids_out", (T, k), 4, optional=True)
    _need(topk_weights_out, "topk_weights_out", (T, k), 4, optional=True)
    return T, H, E


def forward(x, w_gate, router_bias, w1, w2, k, first_expert, num_local, y, ws, logits_out=None,
            topk_ids_out=None, topk_weights_out=None, stream=None):
    T, H, E = _forward_common(x, w_gate, router_bias, k, y, logits_out, topk_ids_out,
                              topk_weights_out)
    I = _dims(w2, "w2", 3)[2]
    _need(w1, "w1", (num_local, 2 * I, H), 2)
    _need(w2, "w2", (num_local, H, I), 2)
    nws = _need_ws(ws)
    _check("moe_forward", lib().moe_forward(
        _ptr(x), _ptr(w_gate), _ptr(router_bias), _ptr(w1), _ptr(w2), T, H, I, E, k,
        first_expert, num_local, _ptr(y), _ptr(logits_out), _ptr(topk_ids_out),
        _ptr(topk_weights_out), _ptr(ws), nws, _stream(stream)))


def forward_fp8(x, w_gate, router_bias, w1q, w1s, w2q, w2s, k, first_expert, num_local, y, ws,
                logits_out=None, topk_ids_out=None, topk_weights_out=None, stream=None):
    """moe_forward_fp8: the layer with FP8 expert weights (codes and row scales
    as for grouped_ffn_fp8)."""
    T, H, E = _forward_common(x, w_gate, router_bias, k, y, logits_out, topk_ids_out,
                              topk_weights_out)
    I = _dims(w2q, "w2q", 3)[2]
    _need(w1q, "w1q", (num_local, 2 * I, H), 1)
    _need(w1s, "w1s", (num_local, 2 * I), 4)
    _need(w2q, "w2q", (num_local, H, I), 1)
    _need(w2s, "w2s", (num_local, H), 4)
    nws = _need_ws(ws)
    _check("moe_forward_fp8", lib().moe_forward_fp8(
        _ptr(x), _ptr(w_gate), _ptr(router_bias), _ptr(w1q), _ptr(w1s), _ptr(w2q), _ptr(w2s), T,
        H, I, E, k, first_expert, num_local, _ptr(y), _ptr(logits_out), _ptr(topk_ids_out),
        _ptr(topk_weights_out), _ptr(ws), nws, _stream(stream)))


def forward_no_alloc(x, w_gate, router_bias, w1, w2, k, first_expert, num_local, y,
                     logits_out=None, topk_ids_out=None, topk_weights_out=None, stream=None):
    """moe_forward_no_alloc: the layer on the library's own device scratch
    (no workspace argument; sizes whose workspace exceeds
    NO_ALLOC_SCRATCH_BYTES are rejected)."""
    T, H, E = _forward_common(x, w_gate, router_bias, k, y, logits_out, topk_ids_out,
                              topk_weights_out)
    I = _dims(w2, "w2", 3)[2]
    _need(w1, "w1", (num_local, 2 * I, H), 2)
    _need(w2, "w2", (num_local, H, I), 2)
    _check("moe_forward_no_alloc", lib().moe_forward_no_alloc(
        _ptr(x), _ptr(w_gate), _ptr(router_bias), _ptr(w1), _ptr(w2), T, H, I, E, k,
        first_expert, num_local, _ptr(y), _ptr(logits_out), _ptr(topk_ids_out),
        _ptr(topk_weights_out), _stream(stream)))


def _out_fp32(t, name):
    """0 / 1 for a bf16 (2-byte) or fp32 (4-byte) tensor."""
    if t is None or t.element_size() not in (2, 4):
        raise ValueError(f"{name} must be bf16 or fp32")
    return t.element_size() == 4


def _here(*tensors, whole=(), ws=None):
    """Raise ValueError unless the tensors are on the current device, the one
    the call launches on, and hold none of the types that have the size of an
    operand's without being it: `tensors` are values and codes (16- and 8-bit
    integers are taken as the bits they are; 4 bytes are fp32), `whole` offsets
    and selections (int32), ws a workspace of any type."""
    torch = _torch()
    d = torch.cuda.current_device()
    others = _other_types or _set_other_types(torch)
    for t in tensors + whole + (ws,):
        if t is not None and t.get_device() != d:
            raise ValueError(f"a tensor is on device {t.get_device()}, the current one is {d}")
    for t in tensors:
        if t is not None and t.dtype in others:
            raise ValueError(f"{t.dtype} is no type of an operand here")
    for t in whole:
        if t is not None and t.dtype is not torch.int32:
            raise ValueError(f"{t.dtype} is no type of offsets or selections, they are int32")


_other_types = None


def _set_other_types(torch):
    global _other_types
    names = ("float16", "float8_e4m3fnuz", "float8_e5m2", "float8_e5m2fnuz", "bool", "int32",
             "uint32", "complex32")
    _other_types = frozenset(getattr(torch, n) for n in names if hasattr(torch, n))
    return _other_types


def _grouped_rows(x, expert_offsets, permuted_rows, k, N):
    T, K = _dims(x, "x", 2)
    L = _dims(expert_offsets, "expert_offsets", 1)[0] - 1
    _need(expert_offsets, "expert_offsets", (L + 1,), 4)
    if permuted_rows is not None:
        _need(permuted_rows, "permuted_rows", (N,), 4)
    elif T != N or k != 1:
        raise ValueError(f"without permuted_rows x has one row for each of the {N} rows, and k is 1")
    return T, K, L


def grouped_matmul(x, expert_offsets, w, y, permuted_rows=None, k=1, stream=None):
    """moe_grouped_matmul: y[n] = w[i] . x[permuted_rows[n] // k] for the rows n
    of each local expert i. x [T, K] bf16, w [L, M, K] bf16, y [N, M] bf16 or
    fp32; without permuted_rows row n is x[n]."""
    N, M = _dims(y, "y", 2)
    T, K, L = _grouped_rows(x, expert_offsets, permuted_rows, k, N)
    _need(x, "x", (T, K), 2)
    _need(w, "w", (L, M, K), 2)
    f32 = _out_fp32(y, "y")
    _need(y, "y", (N, M), 4 if f32 else 2)
    _here(x, w, y, whole=(expert_offsets, permuted_rows))
    _check("moe_grouped_matmul", lib().moe_grouped_matmul(
        _ptr(x), _ptr(permuted_rows), _ptr(expert_offsets), L, T, k, N, K, M, _ptr(w), _ptr(y),
        f32, _stream(stream)))


def grouped_matmul_dx(dy, expert_offsets, w, dx, stream=None):
    """moe_grouped_matmul_dx: dx[n] = w[i]^T . dy[n]. dy [N, M] bf16, w
    [L, M, K] bf16, dx [N, K] bf16 or fp32, all in the experts' row order."""
    N, K = _dims(dx, "dx", 2)
    _, M, L = _grouped_rows(dy, expert_offsets, None, 1, N)
    _need(dy, "dy", (N, M), 2)
    _need(w, "w", (L, M, K), 2)
    f32 = _out_fp32(dx, "dx")
    _need(dx, "dx", (N, K), 4 if f32 else 2)
    _here(dy, w, dx, whole=(expert_offsets,))
    _check("moe_grouped_matmul_dx", lib().moe_grouped_matmul_dx(
        _ptr(dy), _ptr(expert_offsets), L, N, K, M, _ptr(w), _ptr(dx), f32, _stream(stream)))


def grouped_matmul_dw(dy, x, expert_offsets, dw, permuted_rows=None, k=1, stream=None):
    """moe_grouped_matmul_dw: dw[i] = sum over expert i's rows of
    dy[n] x[permuted_rows[n] // k]^T. dy [N, M] bf16, x [T, K] bf16, dw
    [L, M, K] bf16 or fp32."""
    N, M = _dims(dy, "dy", 2)
    T, K, L = _grouped_rows(x, expert_offsets, permuted_rows, k, N)
    _need(dy, "dy", (N, M), 2)
    _need(x, "x", (T, K), 2)
    f32 = _out_fp32(dw, "dw")
    _need(dw, "dw", (L, M, K), 4 if f32 else 2)
    _here(dy, x, dw, whole=(expert_offsets, permuted_rows))
    _check("moe_grouped_matmul_dw", lib().moe_grouped_matmul_dw(
        _ptr(dy), _ptr(x), _ptr(permuted_rows), _ptr(expert_offsets), L, T, k, N, K, M, _ptr(dw),
        f32, _stream(stream)))


def rms_norm(x, weight, eps, y=None, yq=None, ys=None, residual=None, residual_out=None,
             stream=None):
    """moe_rms_norm: h = x + residual (bf16, to residual_out), then
    h / sqrt(mean(h^2) + eps) * weight in bf16 (y) and / or MXFP8 (codes yq
    [T, H], scales ys [T, H // 32])."""
    T, H = _dims(x, "x", 2)
    _need(x, "x", (T, H), 2)
    _need(weight, "weight", (H,), 4)
    _need(residual, "residual", (T, H), 2, optional=True)
    _need(residual_out, "residual_out", (T, H), 2, optional=True)
    _need(y, "y", (T, H), 2, optional=True)
    _need(yq, "yq", (T, H), 1, optional=True)
    _need(ys, "ys", (T, H // 32), 1, optional=True)
    _here(x, weight, y, yq, ys, residual, residual_out)
    _check("moe_rms_norm", lib().moe_rms_norm(
        _ptr(x), _ptr(residual), _ptr(weight), eps, T, H, _ptr(residual_out), _ptr(y), _ptr(yq),
        _ptr(ys), _stream(stream)))


def rms_norm_backward_workspace_size(T, H):
    n = _SZ()
    _check("moe_rms_norm_backward_workspace_size",
           lib().moe_rms_norm_backward_workspace_size(T, H, ctypes.byref(n)))
    return n.value


def rms_norm_backward(dy, h, weight, eps, dx, dweight, ws, dresidual=None, stream=None):
    """moe_rms_norm_backward: dx (of x and of residual alike) and dweight from
    dy, the gradient of rms_norm's y, and h, its residual_out; dresidual is the
    gradient arriving at residual_out."""
    T, H = _dims(h, "h", 2)
    _need(dy, "dy", (T, H), 2)
    _need(h, "h", (T, H), 2)
    _need(weight, "weight", (H,), 4)
    _need(dx, "dx", (T, H), 2)
    _need(dweight, "dweight", (H,), 4)
    _need(dresidual, "dresidual", (T, H), 2, optional=True)
    nws = _need_ws(ws)
    _here(dy, h, weight, dx, dweight, dresidual, ws=ws)
    _check("moe_rms_norm_backward", lib().moe_rms_norm_backward(
        _ptr(dy), _ptr(h), _ptr(weight), eps, T, H, _ptr(dresidual), _ptr(dx), _ptr(dweight),
        _ptr(ws), nws, _stream(stream)))


def _mx_bits(codes, name, rows, width):
    """8 or 4: which microscaled format a code array of `width` values a row holds."""
    got = _dims(codes, name, 2)[1]
    bits = 4 if 2 * got == width else 8
    _need(codes, name, (rows, width * bits // 8), 1)
    return bits


def quantize_mx(x, codes, scales, stream=None):
    """moe_quantize_mx: x [R, K] bf16 or fp32 to MXFP8 (codes [R, K]) or MXFP4
    (codes [R, K // 2]) with scales [R, K // 32]."""
    R, K = _dims(x, "x", 2)
    f32 = _out_fp32(x, "x")
    _need(x, "x", (R, K), 4 if f32 else 2)
    bits = _mx_bits(codes, "codes", R, K)
    _need(scales, "scales", (R, K // 32), 1)
    _here(x, codes, scales)
    _check("moe_quantize_mx", lib().moe_quantize_mx(_ptr(x), f32, R, K, bits, _ptr(codes),
                                                    _ptr(scales), _stream(stream)))


def swiglu_quantize_mx(gu, codes, scales, rows=None, stream=None):
    """moe_swiglu_quantize_mx: silu(gu[:, :I]) * gu[:, I:] to MXFP8 or MXFP4;
    rows: a one-element int32 tensor with the number of rows to take (for
    instance expert_offsets[-1:]), all of them without it."""
    N, I2 = _dims(gu, "gu", 2)
    if I2 % 2:
        raise ValueError("gu holds gate and up columns: an even number")
    f32 = _out_fp32(gu, "gu")
    _need(gu, "gu", (N, I2), 4 if f32 else 2)
    bits = _mx_bits(codes, "codes", N, I2 // 2)
    _need(scales, "scales", (N, I2 // 64), 1)
    _need(rows, "rows", (1,), 4, optional=True)
    _here(gu, codes, scales, whole=(rows,))
    _check("moe_swiglu_quantize_mx", lib().moe_swiglu_quantize_mx(
        _ptr(gu), f32, N, I2 // 2, _ptr(rows), bits, _ptr(codes), _ptr(scales), _stream(stream)))


def dequantize_mx(codes, scales, out, stream=None):
    """moe_dequantize_mx: the values codes and scales stand for, to out [R, K]
    bf16 or fp32."""
    R, K = _dims(out, "out", 2)
    f32 = _out_fp32(out, "out")
    _need(out, "out", (R, K), 4 if f32 else 2)
    bits = _mx_bits(codes, "codes", R, K)
    _need(scales, "scales", (R, K // 32), 1)
    _here(codes, scales, out)
    _check("moe_dequantize_mx", lib().moe_dequantize_mx(_ptr(codes), _ptr(scales), R, K, bits,
                                                        _ptr(out), f32, _stream(stream)))


def grouped_matmul_mx(xq, xs, expert_offsets, wq, ws, y, permuted_rows=None, k=1, stream=None):
    """moe_grouped_matmul_mx: grouped_matmul of MXFP8 rows (xq [T, K]) or MXFP4
    rows (xq [T, K // 2]), scales xs [T, K // 32], with MXFP4 weights (wq
    [L, M, K // 2], ws [L, M, K // 32]); y [N, M] bf16 or fp32. Exact products,
    fp32 sums, for which MXFP8 rows are multiplied in two parts."""
    N, M = _dims(y, "y", 2)
    T, _, L = _grouped_rows(xq, expert_offsets, permuted_rows, k, N)
    K = 2 * _dims(wq, "wq", 3)[2]
    bits = _mx_bits(xq, "xq", T, K)
    _need(xs, "xs", (T, K // 32), 1)
    _need(wq, "wq", (L, M, K // 2), 1)
    _need(ws, "ws", (L, M, K // 32), 1)
    f32 = _out_fp32(y, "y")
    _need(y, "y", (N, M), 4 if f32 else 2)
    _here(xq, xs, wq, ws, y, whole=(expert_offsets, permuted_rows))
    _check("moe_grouped_matmul_mx", lib().moe_grouped_matmul_mx(
        _ptr(xq), _ptr(xs), bits, _ptr(permuted_rows), _ptr(expert_offsets), L, T, k, N, K, M,
        _ptr(wq), _ptr(ws), _ptr(y), f32, _stream(stream)))


def alloc_workspace(T, H, I, E, k, num_local, device="cuda"):
    """A uint8 torch tensor of moe_workspace_size bytes (torch allocations are
    256-byte aligned)."""
    import torch
    n = workspace_size(T, H, I, E, k, num_local)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)
