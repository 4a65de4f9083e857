"""Python binding of libbsf8, the block-scaled FP8 linear projection for MI355X.

Argument marshalling only: every step of the projection runs in the HIP
library (``libbsf8.so``, built by ``python -m block_scaled_fp8_linear_amd.build``).
PyTorch supplies device memory and the current stream.  There is no CPU path:
if the library is missing, importing works but every call raises.

Entry points mirror ``include/bsf8.h``:

* ``validate(...)``                     header-only geometry check, returns a status name
* ``BlockFP8Weight(members, ...)``      handle over borrowed device tensors
* ``quant_act(x)``                      per-token 1x128 E4M3 quantization -> (xq, xs)
* ``quant_norm(x, weight, ...)``        residual add, norms and gate between two blocks -> codes, scales, stream
* ``expert_plan(ids, n_experts)``       router choices -> row ranges of the experts, gather rows, slots
* ``linear_w8a16(w, x)``                F32-activation arm
* ``linear_w8a8_epilogue(w, xq, xs, ...)``  linear_w8a8 with bias, activation and residual in the same call
* ``ExpertsFP8Weight(members)``, ``linear_w8a8_experts(w, xq, xs, offsets, rows)``  products grouped by expert
* ``linear_w8a8(w, xq, xs)``            FP8 x FP8 arm with F32 epilogue
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, List, Optional, Sequence, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
# BSF8_LIBRARY may name another build of the same library (the host-sanitized
# build the CPU tests run under); by default the in-tree libbsf8.so is loaded.
LIB_PATH = os.environ.get("BSF8_LIBRARY") or os.path.join(_HERE, "libbsf8.so")

DT_INVALID, DT_F8_E4M3, DT_F8_E5M2, DT_BF16, DT_F16, DT_F32, DT_U8, DT_OTHER = range(8)
ARM_W8A16, ARM_W8A8, ARM_DENSE, ARM_W8A8_DYNAMIC, ARM_W8A8_EPILOGUE = 0, 1, 2, 3, 4
DTYPE_NAMES = {"F8_E4M3": DT_F8_E4M3, "F8_E5M2": DT_F8_E5M2, "BF16": DT_BF16, "F16": DT_F16,
               "F32": DT_F32, "U8": DT_U8}
MAX_MEMBERS = 8
BLOCK = 128


class BSF8Error(RuntimeError):
    def __init__(self, status: int, name: str, detail: str):
        super().__init__(f"{name}: {detail}")
        self.status, self.name, self.detail = status, name, detail


class TensorDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("rank", ctypes.c_int32), ("shape", ctypes.c_int64 * 4),
                ("data", ctypes.c_void_p)]


class MemberDesc(ctypes.Structure):
    _fields_ = [("weight", TensorDesc), ("scale_inv", ctypes.POINTER(TensorDesc)),
                ("scale", ctypes.POINTER(TensorDesc))]


class Decl(ctypes.Structure):
    _fields_ = [("quant_method_fp8", ctypes.c_int32), ("block_n", ctypes.c_int32), ("block_k", ctypes.c_int32)]


_i32, _i64, _f64, _ptr = ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_void_p


class NormArgs(ctypes.Structure):
    """bsf8_norm_args."""
    _fields_ = [("M", _i64), ("K", _i64), ("kind", _i32), ("eps", _f64), ("residual_scale", _f64), ("x", _ptr),
                ("x_dtype", _i32), ("ldx", _i64), ("x_rows", _i64), ("slots", _ptr), ("probs", _ptr), ("top", _i32),
                ("post_weight", _ptr), ("post_bias", _ptr), ("post_dtype", _i32), ("gate", _ptr),
                ("gate_dtype", _i32), ("ldg", _i64), ("residual", _ptr), ("ldr", _i64), ("h", _ptr), ("ldh", _i64),
                ("h_dtype", _i32), ("weight", _ptr), ("bias", _ptr), ("weight_dtype", _i32), ("n", _ptr),
                ("n_dtype", _i32), ("ldn", _i64), ("xq", _ptr), ("ldq", _i64), ("xs", _ptr), ("xs_sm", _i64),
                ("xs_sk", _i64)]


class Epilogue(ctypes.Structure):
    """bsf8_epilogue."""
    _fields_ = [("bias", _ptr), ("bias_dtype", _i32), ("activation", _i32), ("residual", _ptr),
                ("residual_dtype", _i32), ("ldr", _i64), ("residual_scale", ctypes.c_float)]


class Unit(ctypes.Structure):
    _fields_ = [("prefix", ctypes.c_char * 256), ("prefix_truncated", ctypes.c_int32), ("status", ctypes.c_int32),
                ("weight", TensorDesc), ("scale_inv", TensorDesc), ("scale", TensorDesc),
                ("has_scale_inv", ctypes.c_int32), ("has_scale", ctypes.c_int32),
                ("weight_offset", ctypes.c_int64), ("scale_offset", ctypes.c_int64)]


_lib = None

# (name, restype, argtypes) of every entry point the header declares.
EXPORTS = [
    ("bsf8_abi_version", ctypes.c_int32, []),
    ("bsf8_status_name", ctypes.c_char_p, [ctypes.c_int]),
    ("bsf8_last_error", ctypes.c_char_p, []),
    ("bsf8_validate", ctypes.c_int, [ctypes.POINTER(Decl), ctypes.POINTER(MemberDesc), ctypes.c_int32]),
    ("bsf8_weight_create", ctypes.c_int, [ctypes.POINTER(Decl), ctypes.POINTER(MemberDesc), ctypes.c_int32,
                                          ctypes.POINTER(ctypes.c_void_p)]),
    ("bsf8_weight_destroy", None, [ctypes.c_void_p]),
    ("bsf8_weight_geometry", ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int64),
                                            ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int32)]),
    ("bsf8_weight_scale_row", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(ctypes.c_int32),
                                             ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64)]),
    ("bsf8_quant_act", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                      ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]),
    ("bsf8_workspace_size", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                           ctypes.POINTER(ctypes.c_size_t)]),
    ("bsf8_linear_w8a16", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                         ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                         ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    ("bsf8_linear_w8a8", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.c_void_p]),
    ("bsf8_linear_w8a8_dynamic", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                                ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                                ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    ("bsf8_linear_w8a8_noalloc", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                                ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                                ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p]),
    ("bsf8_describe", ctypes.c_char_p, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64]),
    ("bsf8_read_stream", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    ("bsf8_parse_quant_config", ctypes.c_int, [ctypes.c_char_p, ctypes.POINTER(Decl)]),
    ("bsf8_inspect_safetensors", ctypes.c_int, [ctypes.c_char_p, ctypes.POINTER(Decl), ctypes.POINTER(Unit),
                                                ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)]),
    ("bsf8_quant_glu", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                      ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]),
    ("bsf8_glu_act", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                    ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
    ("bsf8_linear_w8a8_epilogue", ctypes.c_int, [_ptr, _ptr, _i64, _ptr, _i64, _i64, _i64, ctypes.POINTER(Epilogue),
                                                 _ptr, _i32, _i64, _ptr, ctypes.c_size_t, _ptr]),
    ("bsf8_experts_create", ctypes.c_int, [ctypes.POINTER(Decl), ctypes.POINTER(MemberDesc), _i32,
                                           ctypes.POINTER(_ptr)]),
    ("bsf8_experts_destroy", None, [_ptr]),
    ("bsf8_experts_geometry", ctypes.c_int, [_ptr, ctypes.POINTER(_i64), ctypes.POINTER(_i64), ctypes.POINTER(_i64)]),
    ("bsf8_linear_w8a8_experts", ctypes.c_int, [_ptr, _ptr, _i64, _ptr, _i64, _i64, _i64, _ptr, _ptr, _i64, _ptr,
                                                _i32, _i64, _ptr]),
    ("bsf8_experts_describe", ctypes.c_char_p, [_ptr, _i64]),
    ("bsf8_quant_norm", ctypes.c_int, [ctypes.POINTER(NormArgs), ctypes.c_void_p]),
    ("bsf8_expert_plan", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p]),
    ("bsf8_upcast", ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p]),
    ("bsf8_dense_workspace_size", ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                 ctypes.POINTER(ctypes.c_size_t)]),
    ("bsf8_linear_dense", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                         ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32,
                                         ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
]


def lib() -> ctypes.CDLL:
    """Load libbsf8.so once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run `python -m block_scaled_fp8_linear_amd.build` "
                              "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        for name, res, args in EXPORTS:
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def status_name(st: int) -> str:
    return lib().bsf8_status_name(st).decode()


def _check(st: int, what: str):
    if st != 0:
        raise BSF8Error(st, status_name(st), f"{what}: {lib().bsf8_last_error().decode()}")


def _tdesc(dtype, shape, addr) -> TensorDesc:
    d = TensorDesc()
    d.dtype = DTYPE_NAMES[dtype] if isinstance(dtype, str) else int(dtype)
    d.rank = len(shape)
    for i, s in enumerate(shape):
        d.shape[i] = int(s)
    d.data = int(addr) if addr else None
    return d


def _members_array(members: Sequence[dict]):
    """members: dicts with 'weight' (dtype, shape, addr) and optional 'scale_inv' / 'scale'."""
    keep = []
    arr = (MemberDesc * max(1, len(members)))()
    for i, m in enumerate(members):
        w = m["weight"]
        arr[i].weight = _tdesc(w["dtype"], w["shape"], w.get("addr"))
        for leaf in ("scale_inv", "scale"):
            s = m.get(leaf)
            if s is not None:
                d = _tdesc(s["dtype"], s["shape"], s.get("addr"))
                keep.append(d)
                setattr(arr[i], leaf, ctypes.pointer(d))
    return arr, keep


def _decl(quant_method: str = "fp8", block=(BLOCK, BLOCK)) -> Decl:
    d = Decl()
    d.quant_method_fp8 = 1 if quant_method == "fp8" else 0
    d.block_n, d.block_k = int(block[0]), int(block[1])
    return d


def validate(quant_method: str, block, members: Sequence[dict]) -> str:
    """Header-only validation (no device access); returns the status name."""
    decl = _decl(quant_method, block)
    arr, _keep = _members_array(members)
    return status_name(lib().bsf8_validate(ctypes.byref(decl), arr, len(members)))


# ------------------------------------------------------- checkpoint headers

_DT_NAME = {v: k for k, v in DTYPE_NAMES.items()}


def parse_quant_config(json_text: str) -> Tuple[str, Tuple[int, int]]:
    """(quant_method as 'fp8' or 'other', weight_block_size) from a config's JSON text;
    the block is (0, 0) when no weight_block_size is declared (per-tensor reading)."""
    d = Decl()
    _check(lib().bsf8_parse_quant_config(json_text.encode(), ctypes.byref(d)), "parse_quant_config")
    return ("fp8" if d.quant_method_fp8 else "other"), (d.block_n, d.block_k)


def _desc_dict(t: TensorDesc) -> dict:
    return dict(dtype=_DT_NAME.get(t.dtype, "OTHER"), shape=tuple(t.shape[i] for i in range(t.rank)))


def inspect_safetensors(path: str, quant_method: str = "fp8", block=(BLOCK, BLOCK)):
    """Header-only inspection of one safetensors file (no tensor byte is read).

    Returns (status name of the whole file, list of units); each unit is a dict
    with prefix, weight / scale_inv / scale descriptors, data offsets and its
    own status name."""
    L = lib()
    decl = _decl(quant_method, block)
    n = ctypes.c_int32()
    st = L.bsf8_inspect_safetensors(path.encode(), ctypes.byref(decl), None, 0, ctypes.byref(n))
    if status_name(st) == "INVALID_ARG":
        _check(st, "inspect_safetensors")
    units = (Unit * max(1, n.value))()
    st = L.bsf8_inspect_safetensors(path.encode(), ctypes.byref(decl), units, n.value, ctypes.byref(n))
    out = []
    for u in units[:n.value]:
        out.append(dict(prefix=u.prefix.decode(), status=status_name(u.status), weight=_desc_dict(u.weight),
                        scale_inv=_desc_dict(u.scale_inv) if u.has_scale_inv else None,
                        scale=_desc_dict(u.scale) if u.has_scale else None,
                        weight_offset=u.weight_offset, scale_offset=u.scale_offset))
    return status_name(st), out


# ------------------------------------------------------------------ torch glue

_T = None


def _torch():
    global _T
    if _T is None:
        import torch
        _T = torch
    return _T


_DT_OF: Dict[object, int] = {}


def _dt_of(t) -> int:
    if not _DT_OF:
        torch = _torch()
        _DT_OF.update({torch.float32: DT_F32, torch.bfloat16: DT_BF16, torch.float16: DT_F16, torch.uint8: DT_U8,
                       torch.float8_e4m3fn: DT_F8_E4M3, torch.float8_e5m2: DT_F8_E5M2})
    return _DT_OF.get(t.dtype, DT_OTHER)


def _on_device(device, **tensors):
    """Refuse, before any library call, a tensor that is not a GPU tensor on ``device``.

    The library takes raw device addresses: a host tensor's address would reach
    a kernel as if it were device memory, so every tensor argument is checked
    here (None entries are skipped)."""
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor (got one on {t.device})")
        if device is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _codes_dtype_ok(t) -> bool:
    torch = _torch()
    return t.dtype in (torch.uint8, torch.float8_e4m3fn)


def _stream_ptr(device) -> int:
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # no Stream object: 0.1 us in place of 2
    if raw is not None and device.index is not None:
        return raw(device.index)
    return torch.cuda.current_stream(device).cuda_stream


class BlockFP8Weight:
    """Immutable handle over a (possibly grouped) block-FP8 weight on the GPU.

    ``members``: list of (weight, scale_inv) device tensors; weight is uint8 or
    float8_e4m3fn [N_i, K] (contiguous), scale_inv is bfloat16 or float32
    [ceil(N_i/128), ceil(K/128)] (contiguous).  With ``block=(0, 0)`` the
    weight is per-tensor scaled instead: each member's scale is its single
    ``weight_scale`` value (a 0-d or one-element tensor), read as one block that
    covers the whole member.  The tensors are borrowed: this object keeps
    references so they stay alive, and never modifies them.
    """

    def __init__(self, members: Sequence[Tuple[object, object]], quant_method: str = "fp8", block=(BLOCK, BLOCK)):
        L = lib()
        descs = []
        self._tensors = []
        leaf = "scale" if tuple(int(b) for b in block) == (0, 0) else "scale_inv"
        self.per_tensor = leaf == "scale"
        if len(members) == 0:
            raise ValueError("a weight needs at least one member")
        dev0 = members[0][0].device
        for i, (w, s) in enumerate(members):
            _on_device(dev0 if dev0.type == "cuda" else None, **{f"member {i} weight": w, f"member {i} scale": s})
            if not (w.is_contiguous() and s.is_contiguous()):
                raise ValueError("weights and scale grids must be contiguous")
            wdt = DT_F8_E4M3 if _dt_of(w) in (DT_U8, DT_F8_E4M3) else _dt_of(w)
            descs.append({"weight": dict(dtype=wdt, shape=tuple(w.shape), addr=w.data_ptr()),
                          leaf: dict(dtype=_dt_of(s), shape=tuple(s.shape), addr=s.data_ptr())})
            self._tensors += [w, s]
        decl = _decl(quant_method, block)
        arr, keep = _members_array(descs)
        h = ctypes.c_void_p()
        _check(L.bsf8_weight_create(ctypes.byref(decl), arr, len(descs), ctypes.byref(h)), "weight_create")
        self._h = h
        self.device = members[0][0].device
        n, k, nm = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32()
        _check(L.bsf8_weight_geometry(h, ctypes.byref(n), ctypes.byref(k), ctypes.byref(nm)), "geometry")
        self.n_total, self.K, self.n_members = n.value, k.value, nm.value
        self._ws: Dict[tuple, object] = {}

    @property
    def handle(self):
        return self._h

    @property
    def members(self):
        """The borrowed (weight, scale_inv) device tensors, in member order."""
        return [(self._tensors[i], self._tensors[i + 1]) for i in range(0, len(self._tensors), 2)]

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.bsf8_weight_destroy(h)
            self._h = None

    def describe(self, arm: int, M: int) -> str:
        return lib().bsf8_describe(self._h, arm, M).decode()

    def scale_row(self, n: int) -> Tuple[int, int, int]:
        mi, lr, sr = ctypes.c_int32(), ctypes.c_int64(), ctypes.c_int64()
        _check(lib().bsf8_weight_scale_row(self._h, n, ctypes.byref(mi), ctypes.byref(lr), ctypes.byref(sr)),
               "scale_row")
        return mi.value, lr.value, sr.value

    def workspace_size(self, arm: int, M: int) -> int:
        """Workspace bytes of a call of M tokens on this weight's device (they go by its compute units)."""
        b = ctypes.c_size_t()
        idx = self.device.index
        if idx is None or _current()[0]() == idx:
            st = lib().bsf8_workspace_size(self._h, arm, M, ctypes.byref(b))
        else:
            with _torch().cuda.device(idx):
                st = lib().bsf8_workspace_size(self._h, arm, M, ctypes.byref(b))
        _check(st, "workspace_size")
        return b.value

    def workspace(self, arm: int, M: int):
        """A zero-filled device workspace, cached per stream and grown on demand."""
        torch = _torch()
        need = self.workspace_size(arm, M)
        if need == 0:
            return None, 0
        key = _stream_ptr(self.device)
        ws = self._ws.get(key)
        if ws is None or ws.numel() < need:
            ws = torch.zeros(need, dtype=torch.uint8, device=self.device)
            self._ws[key] = ws
        return ws, ws.numel()


def _out(out, M, N, dtype, device):
    torch = _torch()
    if out is None:
        return torch.empty((M, N), dtype=dtype, device=device)
    if out.dtype != dtype or out.dim() != 2 or out.shape[0] != M or out.shape[1] < N or out.stride(1) != 1:
        raise ValueError("out must be [M, >=N] with unit column stride and the requested dtype")
    return out


def scales_kmajor(M: int, Kb: int, device):
    """An uninitialised [M, Kb] float32 scale tensor in the K-major layout (token index
    contiguous: strides (1, M)), the layout the W8A8 product reads fastest."""
    torch = _torch()
    return torch.empty((Kb, M), dtype=torch.float32, device=device).t()


def quant_act(x, xq=None, xs=None):
    """Per-token 1x128 E4M3 quantization of x [M,K] (float32 or bfloat16) -> (xq uint8 [M,K], xs f32 [M,Kb]).
    xs may be any [M, Kb] float32 view in the token-major or the K-major layout; by default
    it is a new K-major one."""
    torch = _torch()
    _on_device(None, x=x)
    _on_device(x.device, xq=xq, xs=xs)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    Kb = -(-K // BLOCK)
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if xs is None:
        xs = scales_kmajor(M, Kb, x.device)
    if tuple(xq.shape) != (M, K) or tuple(xs.shape) != (M, Kb) or xs.dtype != torch.float32:
        raise ValueError(f"xq must be [M, K] = [{M}, {K}] and xs float32 [M, Kb] = [{M}, {Kb}]")
    if not _codes_dtype_ok(xq) or xq.stride(1) != 1:
        raise ValueError("xq must be uint8 or float8_e4m3fn with unit column stride")
    _check(lib().bsf8_quant_act(x.data_ptr(), _dt_of(x), M, K, x.stride(0), xq.data_ptr(), xq.stride(0),
                                xs.data_ptr(), xs.stride(0), xs.stride(1), _stream_ptr(x.device)), "quant_act")
    return xq, xs


def quant_glu(y, xq=None, xs=None):
    """Gate/up output y [M, 2F] (gate then up; float32 or bfloat16) -> the down projection's
    quantized input for silu(gate) * up: (xq uint8 [M, F], xs f32 [M, ceil(F/128)]; xs as for quant_act)."""
    torch = _torch()
    _on_device(None, y=y)
    _on_device(y.device, xq=xq, xs=xs)
    if y.dim() != 2 or y.stride(1) != 1 or y.shape[1] % 2:
        raise ValueError("y must be 2-D with an even number of columns and unit column stride")
    M, F = y.shape[0], y.shape[1] // 2
    Fb = -(-F // BLOCK)
    if xq is None:
        xq = torch.empty((M, F), dtype=torch.uint8, device=y.device)
    if xs is None:
        xs = scales_kmajor(M, Fb, y.device)
    if tuple(xq.shape) != (M, F) or tuple(xs.shape) != (M, Fb) or xs.dtype != torch.float32:
        raise ValueError(f"xq must be [M, F] = [{M}, {F}] and xs float32 [M, Fb] = [{M}, {Fb}]")
    if not _codes_dtype_ok(xq) or xq.stride(1) != 1:
        raise ValueError("xq must be uint8 or float8_e4m3fn with unit column stride")
    _check(lib().bsf8_quant_glu(y.data_ptr(), _dt_of(y), M, F, y.stride(0), xq.data_ptr(), xq.stride(0),
                                xs.data_ptr(), xs.stride(0), xs.stride(1), _stream_ptr(y.device)), "quant_glu")
    return xq, xs


def glu_act(y, out=None):
    """Gate/up output y [M, 2F] (gate then up; float32 or bfloat16) -> h = silu(gate) * up as float32 [M, F],
    the same values quant_glu quantizes."""
    torch = _torch()
    _on_device(None, y=y)
    _on_device(y.device, out=out)
    if y.dim() != 2 or y.stride(1) != 1 or y.shape[1] % 2:
        raise ValueError("y must be 2-D with an even number of columns and unit column stride")
    M, F = y.shape[0], y.shape[1] // 2
    if out is None:
        out = torch.empty((M, F), dtype=torch.float32, device=y.device)
    if out.dtype != torch.float32 or out.dim() != 2 or tuple(out.shape) != (M, F) or out.stride(1) != 1:
        raise ValueError(f"out must be float32 [M, F] = [{M}, {F}] with unit column stride")
    _check(lib().bsf8_glu_act(y.data_ptr(), _dt_of(y), M, F, y.stride(0), out.data_ptr(), out.stride(0),
                              _stream_ptr(y.device)), "glu_act")
    return out


# The calls below take few microseconds on the GPU, so their checks are made of
# few Python operations: device numbers instead of device objects, one stride
# tuple per tensor, no checks of what is allocated here.

def _same_device(idx, **tensors):
    """_on_device against the device number ``idx``, in one comparison per tensor where all is well."""
    for t in tensors.values():
        if t is not None and t.get_device() != idx:
            _on_device(_torch().device("cuda", idx), **tensors)


def _gpu_index(name, t) -> int:
    idx = t.get_device() if t.is_cuda else -1
    if idx < 0:
        _on_device(None, **{name: t})
    return idx


_CURRENT = None


def _current():
    """(current device number, raw stream of a device number): torch's own entry points without the objects around
    them where this torch has them (0.2 us in place of 0.7)."""
    global _CURRENT
    if _CURRENT is None:
        torch = _torch()
        _CURRENT = (getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device,
                    getattr(torch._C, "_cuda_getCurrentRawStream", None) or
                    (lambda idx: torch.cuda.current_stream(idx).cuda_stream))
    return _CURRENT


def _launch(what, idx, fn, *args):
    """fn(*args, stream) on device ``idx``, which is made the current one for the call where it is another."""
    device, stream = _current()
    if device() == idx:
        st = fn(*args, stream(idx))
    else:
        with _torch().cuda.device(idx):
            st = fn(*args, stream(idx))
    if st != 0:
        _check(st, what)


def _new_like(t, shape, dtype):
    """A new contiguous tensor on ``t``'s device, by the shorter call where ``t`` has its shape and type."""
    torch = _torch()
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty(shape, dtype=dtype, device=t.device)


def _pitch(name, t, M, K, dtypes) -> int:
    """Row pitch of ``t``, which must be [M, K] of one of ``dtypes`` with unit column stride and rows that do not
    overlap."""
    if t.shape == (M, K) and t.dtype in dtypes:
        s0, s1 = t.stride()
        if (s1 == 1 or K <= 1) and (s0 >= K or M <= 1):
            return s0 if s0 > K else K
    raise ValueError(f"{name} must be [{M}, {K}] with unit column stride, of one of {dtypes}")


def _vector(name, t, n, dtypes) -> int:
    if t.shape != (n,) or t.dtype not in dtypes or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{n}] tensor of one of {dtypes}")
    return t.data_ptr()


NORM_KINDS = {"rms": 0, "layer": 1}


def quant_norm(x, weight, *, bias=None, kind="rms", eps=1e-6, residual=None, residual_scale=1.0, gate=None,
               post_weight=None, post_bias=None, slots=None, probs=None, quantize=True, xq=None, xs=None, h=None,
               out_dtype=None, out=None):
    """The step between two blocks of a residual stream, in one pass:

        o = x, or sum_j probs[:, j] x[slots[:, j]]         h = residual_scale * residual + gate * post_norm(o)
        n = norm(h) * weight + bias                        (xq, xs) = quant_act(n)

    x: the block's output [M, K] (float32 or bfloat16), or with ``slots`` (int32 [M, top]) and ``probs``
    (float32 [M, top]) the rows of an expert product.  ``kind``: "rms" or "layer", of both norms; the one after
    the block runs when ``post_weight`` is given.  ``gate``: [K] or [M, K].  ``residual`` and ``h`` have one type
    (x's when there is no residual); ``h`` may be ``residual`` itself.  Returns (xq, xs, h, n): codes and scales
    as quant_act gives them (None with ``quantize=False``), the stream h (None when there is neither ``residual``
    nor ``h``), and n when ``out`` or ``out_dtype`` asks for it, else None."""
    torch = _torch()
    f32, bf16 = torch.float32, torch.bfloat16
    real = (f32, bf16)
    idx = _gpu_index("x", x)
    _same_device(idx, weight=weight, bias=bias, residual=residual, gate=gate, post_weight=post_weight,
                 post_bias=post_bias, slots=slots, probs=probs, xq=xq, xs=xs, h=h, out=out)
    if kind not in NORM_KINDS:
        raise ValueError(f"kind must be one of {sorted(NORM_KINDS)}")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    rows, K = x.shape
    a = NormArgs(rows, K, NORM_KINDS[kind], eps, residual_scale, x.data_ptr(), DT_BF16 if x.dtype is bf16 else DT_F32,
                 _pitch("x", x, rows, K, real), rows)
    M = rows
    if slots is not None or probs is not None:
        if slots is None or probs is None:
            raise ValueError("slots and probs: both or neither")
        if slots.dim() != 2 or slots.dtype != torch.int32 or not slots.is_contiguous() or probs.shape != slots.shape \
                or probs.dtype != f32 or not probs.is_contiguous():
            raise ValueError("slots must be int32 and probs float32, both contiguous [M, top]")
        M, top = slots.shape
        if top < 1:
            raise ValueError("slots and probs need at least one column")
        a.M, a.slots, a.probs, a.top = M, slots.data_ptr(), probs.data_ptr(), top
    a.weight, a.weight_dtype = _vector("weight", weight, K, real), _dt_of(weight)
    if bias is not None:
        a.bias = _vector("bias", bias, K, (weight.dtype,))
    if post_weight is not None:
        a.post_weight, a.post_dtype = _vector("post_weight", post_weight, K, real), _dt_of(post_weight)
    if post_bias is not None:
        if post_weight is None:
            raise ValueError("post_bias without post_weight")
        a.post_bias = _vector("post_bias", post_bias, K, (post_weight.dtype,))
    if gate is not None:
        if gate.dim() == 1:
            a.gate = _vector("gate", gate, K, real)
        else:
            a.gate, a.ldg = gate.data_ptr(), _pitch("gate", gate, M, K, real)
        a.gate_dtype = _dt_of(gate)
    stream_dtype = x.dtype
    if residual is not None:
        stream_dtype = residual.dtype
        a.residual, a.ldr = residual.data_ptr(), _pitch("residual", residual, M, K, real)
        if h is None:
            h = _new_like(residual, (M, K), stream_dtype)
            a.h, a.ldh = h.data_ptr(), K
        else:
            a.h, a.ldh = h.data_ptr(), _pitch("h", h, M, K, (stream_dtype,))
    elif h is not None:
        stream_dtype = h.dtype
        a.h, a.ldh = h.data_ptr(), _pitch("h", h, M, K, real)
    a.h_dtype = DT_BF16 if stream_dtype is bf16 else DT_F32
    if out is not None:
        a.n, a.ldn = out.data_ptr(), _pitch("out", out, M, K, real if out_dtype is None else (out_dtype,))
        a.n_dtype = _dt_of(out)
    elif out_dtype is not None:
        if out_dtype not in real:
            raise ValueError("out_dtype must be float32 or bfloat16")
        out = torch.empty((M, K), dtype=out_dtype, device=x.device)
        a.n, a.n_dtype, a.ldn = out.data_ptr(), _dt_of(out), K
    if quantize:
        Kb = -(-K // BLOCK)
        if xq is None:
            xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
            a.xq, a.ldq = xq.data_ptr(), K
        else:
            a.xq, a.ldq = xq.data_ptr(), _pitch("xq", xq, M, K, (torch.uint8, torch.float8_e4m3fn))
        if xs is None:
            xs = torch.empty_strided((M, Kb), (1, M), dtype=f32, device=x.device)
            a.xs, a.xs_sm, a.xs_sk = xs.data_ptr(), 1, M
        else:
            if xs.shape != (M, Kb) or xs.dtype != f32:
                raise ValueError(f"xs must be float32 [M, Kb] = [{M}, {Kb}]")
            a.xs, (a.xs_sm, a.xs_sk) = xs.data_ptr(), xs.stride()
    elif out is None or xq is not None or xs is not None:
        raise ValueError("without quantize, out or out_dtype is needed and xq and xs are not written")
    _launch("quant_norm", idx, lib().bsf8_quant_norm, ctypes.byref(a))
    return xq, xs, h, out


def expert_plan(ids, n_experts: int, offsets=None, rows=None, slots=None):
    """The router's choices ids [M, top] (int32 or int64, contiguous) -> (offsets int32 [n_experts + 1],
    rows int32 [M * top], slots int32 [M, top]): expert e has rows offsets[e] .. offsets[e+1] - 1, row r is token
    rows[r], choice (m, j) is row slots[m, j].  A number outside [0, n_experts) has no row and slot -1; entries of
    rows from offsets[n_experts] on keep what they hold."""
    torch = _torch()
    idx = _gpu_index("ids", ids)
    _same_device(idx, offsets=offsets, rows=rows, slots=slots)
    i32 = torch.int32
    if ids.dim() != 2 or ids.dtype not in (i32, torch.int64) or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 or int64 [M, top] tensor")
    M, top = ids.shape
    if n_experts < 1:
        raise ValueError("n_experts must be positive")
    for name, t, shape in (("offsets", offsets, (n_experts + 1,)), ("rows", rows, (M * top,)),
                           ("slots", slots, (M, top))):
        if t is not None and (t.shape != shape or t.dtype != i32 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor")
    if offsets is None:
        offsets = torch.empty(n_experts + 1, dtype=i32, device=ids.device)
    if rows is None:
        rows = torch.empty(M * top, dtype=i32, device=ids.device)
    if slots is None:
        slots = _new_like(ids, (M, top), i32)
    _launch("expert_plan", idx, lib().bsf8_expert_plan, ids.data_ptr(), ids.element_size(), M, top, n_experts,
            offsets.data_ptr(), rows.data_ptr(), slots.data_ptr())
    return offsets, rows, slots


def linear_w8a16(w: BlockFP8Weight, x, out_dtype=None, out=None, workspace=None):
    """F32-activation arm: y [M, N] = x . dequant(W)^T (float32 output unless out_dtype says bfloat16)."""
    torch = _torch()
    out_dtype = out_dtype or torch.float32
    _on_device(w.device, x=x, out=out, workspace=workspace[0] if workspace is not None else None)
    if x.dim() != 2 or x.stride(1) != 1 or x.shape[1] != w.K:
        raise ValueError("x must be [M, K] with unit column stride")
    M = x.shape[0]
    y = _out(out, M, w.n_total, out_dtype, x.device)
    ws, wsb = workspace if workspace is not None else w.workspace(ARM_W8A16, M)
    _check(lib().bsf8_linear_w8a16(w.handle, x.data_ptr(), _dt_of(x), M, x.stride(0), y.data_ptr(), _dt_of(y),
                                   y.stride(0), ws.data_ptr() if ws is not None else None, wsb,
                                   _stream_ptr(x.device)), "linear_w8a16")
    return y


def linear_w8a8(w: BlockFP8Weight, xq, xs, out_dtype=None, out=None, workspace=None):
    """FP8 x FP8 arm with F32 epilogue: y [M, N] (bfloat16 output unless out_dtype says float32)."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    _on_device(w.device, xq=xq, xs=xs, out=out, workspace=workspace[0] if workspace is not None else None)
    Kb = -(-w.K // BLOCK)
    if (xq.dim() != 2 or xq.shape[1] != w.K or xq.stride(1) != 1 or tuple(xs.shape) != (xq.shape[0], Kb)
            or xs.dtype != torch.float32):
        raise ValueError("xq must be [M, K] with unit column stride and xs float32 [M, ceil(K/128)]")
    if not _codes_dtype_ok(xq):
        raise ValueError("xq must be uint8 or float8_e4m3fn (the quantizer's E4M3 bytes)")
    M = xq.shape[0]
    y = _out(out, M, w.n_total, out_dtype, xq.device)
    ws, wsb = workspace if workspace is not None else w.workspace(ARM_W8A8, M)
    _check(lib().bsf8_linear_w8a8(w.handle, xq.data_ptr(), xq.stride(0), xs.data_ptr(), xs.stride(0), xs.stride(1), M,
                                  y.data_ptr(), _dt_of(y), y.stride(0),
                                  ws.data_ptr() if ws is not None else None, wsb, _stream_ptr(xq.device)),
           "linear_w8a8")
    return y


ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def _quantized(xq, xs, K):
    """(tokens, code pitch, scale strides) of a quantizer's output for K channels."""
    torch = _torch()
    if xq.dim() != 2:
        raise ValueError("xq must be 2-D")
    M = xq.shape[0]
    ldq = _pitch("xq", xq, M, K, (torch.uint8, torch.float8_e4m3fn))
    if xs.shape != (M, -(-K // BLOCK)) or xs.dtype != torch.float32:
        raise ValueError("xs must be float32 [M, ceil(K/128)]")
    sm, sk = xs.stride()
    return M, ldq, sm, sk


def _output(out, M, N, dtype, device):
    """(out, pitch): ``out`` checked, or a new [M, N] of ``dtype``."""
    if out is None:
        return _torch().empty((M, N), dtype=dtype, device=device), N
    out = _out(out, M, N, dtype, device)
    if M > 1 and out.stride(0) < N:
        raise ValueError("out's rows must not overlap")
    return out, max(out.stride(0), N)


def linear_w8a8_epilogue(w: BlockFP8Weight, xq, xs, *, bias=None, activation=None, residual=None, residual_scale=1.0,
                         out_dtype=None, out=None, workspace=None):
    """linear_w8a8 and what follows it in one call: y = activation(x . W^T + bias) + residual_scale * residual.

    bias: [N]; residual: [M, N], which may be ``out`` itself (float32 or bfloat16 both); activation: None, "relu",
    "silu", "gelu" or "gelu_tanh".  y is bfloat16 unless out_dtype says float32.  workspace: (tensor, bytes) as
    workspace_size(ARM_W8A8_EPILOGUE, M) says; without it a call that needs one takes its own from the allocator, so
    that graphs captured on one stream may be replayed at the same time."""
    torch = _torch()
    real = (torch.float32, torch.bfloat16)
    out_dtype = out_dtype or torch.bfloat16
    idx = w.device.index
    _same_device(idx, xq=xq, xs=xs, bias=bias, residual=residual, out=out,
                 workspace=workspace[0] if workspace is not None else None)
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}")
    M, ldq, sm, sk = _quantized(xq, xs, w.K)
    N = w.n_total
    e = Epilogue()
    e.activation = ACTIVATIONS[activation]
    if bias is not None:
        e.bias, e.bias_dtype = _vector("bias", bias, N, real), _dt_of(bias)
    if residual is not None:
        e.residual, e.ldr = residual.data_ptr(), _pitch("residual", residual, M, N, real)
        e.residual_dtype, e.residual_scale = _dt_of(residual), residual_scale
    y, ldy = _output(out, M, N, out_dtype, w.device)
    if workspace is not None:
        ws, wsb = workspace
        if wsb > (ws.numel() * ws.element_size() if ws is not None and ws.is_contiguous() else 0):
            raise ValueError(f"the workspace must be a contiguous tensor of at least the {wsb} bytes given")
    else:
        wsb = w.workspace_size(ARM_W8A8_EPILOGUE, M)
        ws = torch.empty(wsb, dtype=torch.uint8, device=w.device) if wsb else None
    _launch("linear_w8a8_epilogue", idx, lib().bsf8_linear_w8a8_epilogue, w.handle, xq.data_ptr(), ldq, xs.data_ptr(),
            sm, sk, M, ctypes.byref(e), y.data_ptr(), _dt_of(y), ldy, ws.data_ptr() if ws is not None else None, wsb)
    return y


class ExpertsFP8Weight:
    """Immutable handle over the block-FP8 weights of E experts on the GPU.

    ``members``: list of (weight, scale_inv) device tensors; weight is uint8 or float8_e4m3fn [E, N_i, K], scale_inv
    bfloat16 or float32 [E, ceil(N_i/128), ceil(K/128)], both contiguous.  A gated layer has two members, gate and
    up (or one that holds both, where their rows are a multiple of 128).  The tensors are borrowed, as
    BlockFP8Weight's are."""

    def __init__(self, members: Sequence[Tuple[object, object]], quant_method: str = "fp8", block=(BLOCK, BLOCK)):
        L = lib()
        if len(members) == 0:
            raise ValueError("a weight needs at least one member")
        descs, self._tensors = [], []
        dev0 = members[0][0].device
        for i, (w, s) in enumerate(members):
            _on_device(dev0 if dev0.type == "cuda" else None, **{f"member {i} weight": w, f"member {i} scale": s})
            if not (w.is_contiguous() and s.is_contiguous()):
                raise ValueError("weights and scale grids must be contiguous")
            if w.dim() > 4 or s.dim() > 4:
                raise ValueError("weights and scale grids must be 3-D")
            wdt = DT_F8_E4M3 if _dt_of(w) in (DT_U8, DT_F8_E4M3) else _dt_of(w)
            descs.append({"weight": dict(dtype=wdt, shape=tuple(w.shape), addr=w.data_ptr()),
                          "scale_inv": dict(dtype=_dt_of(s), shape=tuple(s.shape), addr=s.data_ptr())})
            self._tensors += [w, s]
        decl = _decl(quant_method, block)
        arr, _keep = _members_array(descs)
        h = ctypes.c_void_p()
        _check(L.bsf8_experts_create(ctypes.byref(decl), arr, len(descs), ctypes.byref(h)), "experts_create")
        self._h = h
        self.device = dev0
        e, n, k = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(L.bsf8_experts_geometry(h, ctypes.byref(e), ctypes.byref(n), ctypes.byref(k)), "experts_geometry")
        self.n_experts, self.n_total, self.K = e.value, n.value, k.value

    @property
    def handle(self):
        return self._h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.bsf8_experts_destroy(h)
            self._h = None

    def describe(self, R: int) -> str:
        return lib().bsf8_experts_describe(self._h, R).decode()


def linear_w8a8_experts(w: ExpertsFP8Weight, xq, xs, offsets, rows=None, out_dtype=None, out=None):
    """The experts' products of ragged row runs: y[r] = x[rows[r]] . W_e^T for r in [offsets[e], offsets[e+1]).

    xq, xs: M tokens as the quantizers give them; offsets: int32 [E + 1] and rows: int32 [R], on the GPU, as
    expert_plan gives them (without ``rows``, row r is token r and R = M).  y [R, N] is bfloat16 unless out_dtype
    says float32; rows outside every run keep what ``out`` holds, and a row whose token is outside [0, M) is zero.
    The runs are read on the GPU: nothing here waits for them, and a captured call follows their new values."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    idx = w.device.index
    _same_device(idx, xq=xq, xs=xs, offsets=offsets, rows=rows, out=out)
    M, ldq, sm, sk = _quantized(xq, xs, w.K)
    i32 = (torch.int32,)
    off = _vector("offsets", offsets, w.n_experts + 1, i32)
    R, at = M, None
    if rows is not None:
        R = rows.numel()
        at = _vector("rows", rows, R, i32)
    y, ldy = _output(out, R, w.n_total, out_dtype, w.device)
    _launch("linear_w8a8_experts", idx, lib().bsf8_linear_w8a8_experts, w.handle, xq.data_ptr(), ldq, xs.data_ptr(),
            sm, sk, M, off, at, R, y.data_ptr(), _dt_of(y), ldy)
    return y


def linear_w8a8_dynamic(w: BlockFP8Weight, x, out_dtype=None, out=None, workspace=None):
    """W8A8 arm on unquantized activations: x (float32 or bfloat16 [M, K]) is quantized per
    token in 1x128 groups as quant_act does and multiplied as linear_w8a8 does, bit for bit,
    in one call (bfloat16 output unless out_dtype says float32).  One aligned token is
    quantized inside the weight-streaming kernels; more go through the workspace."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    _on_device(w.device, x=x, out=out, workspace=workspace[0] if workspace is not None else None)
    if x.dim() != 2 or x.stride(1) != 1 or x.shape[1] != w.K:
        raise ValueError("x must be [M, K] with unit column stride")
    M = x.shape[0]
    y = _out(out, M, w.n_total, out_dtype, x.device)
    ws, wsb = workspace if workspace is not None else w.workspace(ARM_W8A8_DYNAMIC, M)
    _check(lib().bsf8_linear_w8a8_dynamic(w.handle, x.data_ptr(), _dt_of(x), M, x.stride(0), y.data_ptr(),
                                          _dt_of(y), y.stride(0), ws.data_ptr() if ws is not None else None, wsb,
                                          _stream_ptr(x.device)), "linear_w8a8_dynamic")
    return y


NOALLOC_SCRATCH_BYTES = 64 << 20   # BSF8_NOALLOC_SCRATCH_BYTES in include/bsf8.h


def linear_w8a8_noalloc(w: BlockFP8Weight, xq, xs, out):
    """linear_w8a8 for callers that cannot allocate: ``out`` (bfloat16 or float32 [M, >=N])
    must be given, and split-K partials go to the library's fixed per-device scratch
    instead of a workspace.  Calls that overlap in time on one device race."""
    torch = _torch()
    if out is None:
        raise ValueError("out must be given: the no-allocation call allocates nothing")
    _on_device(w.device, xq=xq, xs=xs, out=out)
    Kb = -(-w.K // BLOCK)
    if (xq.dim() != 2 or xq.shape[1] != w.K or xq.stride(1) != 1 or tuple(xs.shape) != (xq.shape[0], Kb)
            or xs.dtype != torch.float32):
        raise ValueError("xq must be [M, K] with unit column stride and xs float32 [M, ceil(K/128)]")
    if not _codes_dtype_ok(xq):
        raise ValueError("xq must be uint8 or float8_e4m3fn (the quantizer's E4M3 bytes)")
    M = xq.shape[0]
    y = _out(out, M, w.n_total, out.dtype, xq.device)
    _check(lib().bsf8_linear_w8a8_noalloc(w.handle, xq.data_ptr(), xq.stride(0), xs.data_ptr(), xs.stride(0),
                                          xs.stride(1), M, y.data_ptr(), _dt_of(y), y.stride(0),
                                          _stream_ptr(xq.device)), "linear_w8a8_noalloc")
    return y


def upcast(w: BlockFP8Weight, out_dtype=None, out=None):
    """Dense copy [N, K] of the weight (bfloat16 unless out_dtype says float32): the resident=False load step."""
    torch = _torch()
    out_dtype = out_dtype or torch.bfloat16
    _on_device(w.device, out=out)
    if out is None:
        out = torch.empty((w.n_total, w.K), dtype=out_dtype, device=w.device)
    if out.dtype != out_dtype or out.dim() != 2 or out.shape[0] != w.n_total or out.shape[1] < w.K \
            or out.stride(1) != 1:
        raise ValueError("out must be [N, >=K] with unit column stride and the requested dtype")
    _check(lib().bsf8_upcast(w.handle, out.data_ptr(), _dt_of(out), out.stride(0), _stream_ptr(out.device)), "upcast")
    return out


def dense_workspace_size(N: int, K: int, M: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().bsf8_dense_workspace_size(N, K, M, ctypes.byref(b)), "dense_workspace_size")
    return b.value


def linear_dense(wd, x, out_dtype=None, out=None, workspace=None):
    """Dense arm: y [M, N] = x . wd^T for bfloat16 wd [N, K] (contiguous) and bfloat16 x [M, K]
    (float32 output unless out_dtype says bfloat16).  ``workspace``: a uint8 device tensor of at
    least dense_workspace_size bytes, allocated here when omitted."""
    torch = _torch()
    out_dtype = out_dtype or torch.float32
    _on_device(None, wd=wd)
    _on_device(wd.device, x=x, out=out, workspace=workspace)
    if wd.dim() != 2 or not wd.is_contiguous() or wd.dtype != torch.bfloat16:
        raise ValueError("wd must be a contiguous bfloat16 [N, K] tensor")
    N, K = wd.shape
    if x.dim() != 2 or x.stride(1) != 1 or x.shape[1] != K or x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16 [M, K] with unit column stride")
    M = x.shape[0]
    y = _out(out, M, N, out_dtype, x.device)
    need = dense_workspace_size(N, K, M)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _check(lib().bsf8_linear_dense(wd.data_ptr(), N, K, x.data_ptr(), M, x.stride(0), y.data_ptr(), _dt_of(y),
                                   y.stride(0), workspace.data_ptr() if workspace is not None else None,
                                   workspace.numel() if workspace is not None else 0, _stream_ptr(x.device)),
           "linear_dense")
    return y


__all__ = ["BSF8Error", "BlockFP8Weight", "validate", "quant_act", "quant_glu", "glu_act", "quant_norm", "expert_plan", "linear_w8a16", "linear_w8a8",
           "linear_w8a8_dynamic", "linear_w8a8_noalloc", "linear_w8a8_epilogue", "linear_w8a8_experts",
           "ExpertsFP8Weight", "ARM_W8A8_EPILOGUE", "NOALLOC_SCRATCH_BYTES", "upcast",
           "linear_dense", "dense_workspace_size", "lib", "status_name", "ARM_W8A16", "ARM_W8A8", "ARM_DENSE",
           "ARM_W8A8_DYNAMIC",
           "EXPORTS", "LIB_PATH", "MAX_MEMBERS", "scales_kmajor"]


READ_STREAM_SINK_WORDS = 2048  # BSF8_READ_STREAM_SINK_WORDS in include/bsf8.h


def read_stream(buf, sink):
    """Measurement aid: a plain read of ``buf``'s bytes on the current stream.

    ``sink``: int32 device tensor of at least READ_STREAM_SINK_WORDS words; the
    launch overwrites its leading words with per-block XORs of what it read."""
    _on_device(None, buf=buf)
    _on_device(buf.device, sink=sink)
    if sink.numel() * sink.element_size() < 4 * READ_STREAM_SINK_WORDS:
        raise ValueError(f"read_stream sink needs {READ_STREAM_SINK_WORDS} 4-byte words")
    _check(lib().bsf8_read_stream(buf.data_ptr(), buf.numel() * buf.element_size(), sink.data_ptr(),
                                  _stream_ptr(buf.device)), "read_stream")
