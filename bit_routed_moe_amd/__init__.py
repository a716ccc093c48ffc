"""ds4moe: one routed-MoE layer over low-bit experts on an AMD Instinct MI355X.

A thin ctypes binding over ``libds4moe.so`` (built from ``csrc/`` by
``bit_routed_moe_amd.build``).  Every function takes caller-allocated torch
tensors, passes their device pointers and the current HIP stream to the C ABI
of the same name (see ``include/ds4moe.h``), and raises ``Ds4MoeError`` on a
non-OK status.  Nothing here computes: every step runs in the HIP kernels.
There is no CPU fallback; importing the package fails if the library has not
been built.
"""
import ctypes
import os

__all__ = [
    "Config", "Weights", "Ds4MoeError", "WFMT", "DTYPE", "ALGO", "LIB_PATH", "lib",
    "make_config", "make_weights", "router_logits", "route", "permute", "expert_ffn", "combine", "forward",
    "forward_noalloc", "forward_noalloc_max_bytes",
    "workspace_bytes", "workspace_region", "WS_REGION", "dequantize", "quantize_mxfp8", "status_string", "version",
    "EXPORTS", "STAGE", "set_stage_events",
    "ACT", "Matmul", "make_matmul", "matmul_workspace_bytes", "linear", "linear_backward", "grouped_matmul",
    "grouped_matmul_backward", "sample", "sample_workspace_bytes",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libds4moe.so")

WFMT = {"q2k": 1, "mxfp4": 2, "bf16": 3, "q4k": 4}
DTYPE = {"f32": 0, "bf16": 1, "fp8": 2}
ALGO = {"auto": 0, "gemv": 1, "grouped": 2}
ACT = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "swiglu": 5}

# Every entry point declared in include/ds4moe.h.
EXPORTS = (
    "ds4moe_router_logits", "ds4moe_route", "ds4moe_permute", "ds4moe_expert_ffn", "ds4moe_combine", "ds4moe_forward",
    "ds4moe_workspace_bytes", "ds4moe_dequantize", "ds4moe_status_string", "ds4moe_last_error",
    "ds4moe_version", "ds4moe_set_stage_events", "ds4moe_forward_path", "ds4moe_quantize_mxfp8",
    "ds4moe_workspace_region", "ds4moe_forward_noalloc", "ds4moe_forward_noalloc_max_bytes",
    "ds4moe_linear", "ds4moe_linear_backward", "ds4moe_grouped_matmul", "ds4moe_grouped_matmul_backward",
    "ds4moe_matmul_workspace_bytes", "ds4moe_sample", "ds4moe_sample_workspace_bytes",
)

WS_REGION = {"topk_idx": 0, "topk_w": 1, "offsets": 2, "sorted_pair": 3, "pair_pos": 4, "active": 5,
             "expert_out": 6, "shared_out": 7}

STAGE = {"route": 0, "permute": 1, "ffn_up": 2, "ffn_down": 3, "combine": 4, "router_proj": 5}


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "hidden", "ffn", "n_experts", "top_k", "shared_ffn", "wfmt", "act_dtype", "mma_dtype", "algo")]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "gate", "up", "down", "gate_scales", "up_scales", "down_scales", "sh_gate", "sh_up", "sh_down")]


class Matmul(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("in_dim", "out_dim", "groups", "dtype", "act", "grad_dtype")] +
                [(n, ctypes.c_int64) for n in ("ldx", "ldw", "ldy", "ldz")])


class Ds4MoeError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"ds4moe status {status}: {message}")
        self.status = status


def _load():
    # torch's HIP runtime must be the process's runtime before the library is
    # mapped: the library's libamdhip64.so.7 dependency then resolves to
    # torch's copy, and torch's pointers and streams are valid in its launches.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m bit_routed_moe_amd.build` "
                          "(hipcc, gfx950); there is no fallback")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    cfgp, wp = ctypes.POINTER(Config), ctypes.POINTER(Weights)
    mmp = ctypes.POINTER(Matmul)
    sigs = {
        "ds4moe_router_logits": (i32, [cfgp, i32, vp, vp, vp, vp]),
        "ds4moe_route": (i32, [cfgp, i32, vp, vp, vp, vp]),
        "ds4moe_permute": (i32, [cfgp, i32, vp, vp, vp, vp, vp, vp]),
        "ds4moe_expert_ffn": (i32, [cfgp, wp, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "ds4moe_combine": (i32, [cfgp, i32, vp, vp, vp, vp, vp, vp]),
        "ds4moe_forward": (i32, [cfgp, wp, i32, vp, vp, vp, vp, sz, vp]),
        "ds4moe_workspace_bytes": (sz, [cfgp, i32]),
        "ds4moe_dequantize": (i32, [i32, vp, vp, i64, vp, vp, vp]),
        "ds4moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "ds4moe_last_error": (ctypes.c_char_p, []),
        "ds4moe_version": (ctypes.c_char_p, []),
        "ds4moe_set_stage_events": (i32, [ctypes.c_int, vp, vp]),
        "ds4moe_forward_path": (i32, [cfgp, i32]),
        "ds4moe_quantize_mxfp8": (i32, [vp, i64, vp, vp, vp]),
        "ds4moe_workspace_region": (i32, [cfgp, i32, i32, ctypes.POINTER(sz), ctypes.POINTER(sz)]),
        "ds4moe_forward_noalloc": (i32, [cfgp, wp, i32, vp, vp, vp, vp]),
        "ds4moe_forward_noalloc_max_bytes": (sz, []),
        "ds4moe_linear": (i32, [mmp, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "ds4moe_linear_backward": (i32, [mmp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "ds4moe_grouped_matmul": (i32, [mmp, i32, vp, i32, vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]),
        "ds4moe_grouped_matmul_backward": (i32, [mmp, i32, vp, i32, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp]),
        "ds4moe_matmul_workspace_bytes": (sz, [mmp, i32, i32]),
        "ds4moe_sample": (i32, [i32, i32, vp, i64, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "ds4moe_sample_workspace_bytes": (sz, [i32, i32]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


lib = _load()


def status_string(st: int) -> str:
    return lib.ds4moe_status_string(st).decode()


def version() -> str:
    return lib.ds4moe_version().decode()


def _check(st: int):
    if st != 0:
        raise Ds4MoeError(st, f"{status_string(st)}: {lib.ds4moe_last_error().decode()}")


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _s(stream, dev=None):
    """Handle of a stream; None: the current one (of device `dev`, where its index is at hand)."""
    if stream is not None:
        return ctypes.c_void_p(stream if isinstance(stream, int) else stream.cuda_stream)
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def make_config(hidden, ffn, n_experts, top_k, shared_ffn=0, wfmt="q2k", act="bf16", mma="bf16",
                algo="auto") -> Config:
    return Config(hidden, ffn, n_experts, top_k, shared_ffn, WFMT[wfmt], DTYPE[act], DTYPE[mma], ALGO[algo])


def make_weights(gate, up, down, gate_scales=None, up_scales=None, down_scales=None,
                 sh_gate=None, sh_up=None, sh_down=None) -> Weights:
    """Device tensors -> the pointer struct.  The caller keeps the tensors alive."""
    ptr = lambda t: None if t is None else t.data_ptr()
    return Weights(ptr(gate), ptr(up), ptr(down), ptr(gate_scales), ptr(up_scales), ptr(down_scales),
                   ptr(sh_gate), ptr(sh_up), ptr(sh_down))


def workspace_bytes(cfg: Config, T_max: int) -> int:
    return int(lib.ds4moe_workspace_bytes(ctypes.byref(cfg), T_max))


def workspace_region(cfg: Config, T: int, region) -> tuple:
    """(byte offset, byte count) of a stage result inside forward's workspace
    ("topk_idx", "topk_w", "offsets", "sorted_pair", "pair_pos", "active",
    "expert_out", "shared_out")."""
    off, n = ctypes.c_size_t(0), ctypes.c_size_t(0)
    r = WS_REGION[region] if isinstance(region, str) else region
    _check(lib.ds4moe_workspace_region(ctypes.byref(cfg), T, r, ctypes.byref(off), ctypes.byref(n)))
    return int(off.value), int(n.value)


def router_logits(cfg, T, x, router_w, logits, stream=None):
    _check(lib.ds4moe_router_logits(ctypes.byref(cfg), T, _p(x), _p(router_w), _p(logits), _s(stream)))


def route(cfg, T, logits, topk_idx, topk_w, stream=None):
    _check(lib.ds4moe_route(ctypes.byref(cfg), T, _p(logits), _p(topk_idx), _p(topk_w), _s(stream)))


def permute(cfg, T, topk_idx, expert_offsets, sorted_pair, pair_pos, active, stream=None):
    _check(lib.ds4moe_permute(ctypes.byref(cfg), T, _p(topk_idx), _p(expert_offsets), _p(sorted_pair),
                              _p(pair_pos), _p(active), _s(stream)))


def expert_ffn(cfg, weights, T, x, expert_offsets, sorted_pair, active, expert_out, shared_out,
               workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.ds4moe_expert_ffn(ctypes.byref(cfg), ctypes.byref(weights), T, _p(x), _p(expert_offsets),
                                 _p(sorted_pair), _p(active), _p(expert_out), _p(shared_out),
                                 _p(workspace), nbytes, _s(stream)))


def combine(cfg, T, expert_out, pair_pos, topk_w, shared_out, y, stream=None):
    _check(lib.ds4moe_combine(ctypes.byref(cfg), T, _p(expert_out), _p(pair_pos), _p(topk_w),
                              _p(shared_out), _p(y), _s(stream)))


def forward(cfg, weights, T, x, logits, y, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.ds4moe_forward(ctypes.byref(cfg), ctypes.byref(weights), T, _p(x), _p(logits), _p(y),
                              _p(workspace), nbytes, _s(stream)))


def forward_noalloc(cfg, weights, T, x, logits, y, stream=None):
    """ds4moe_forward with its workspace in the library's fixed per-device
    array (no device allocation; overlapping calls on one device race)."""
    _check(lib.ds4moe_forward_noalloc(ctypes.byref(cfg), ctypes.byref(weights), T, _p(x), _p(logits), _p(y),
                                      _s(stream)))


def forward_noalloc_max_bytes() -> int:
    return int(lib.ds4moe_forward_noalloc_max_bytes())


def forward_path(cfg, T):
    """1: batch 1 in two launches; else route/permute/FFN/combine launches
    with the expert FFNs on the GEMV kernels (0) or the grouped GEMM (2)."""
    st = lib.ds4moe_forward_path(ctypes.byref(cfg), T)
    if st < 0:
        _check(st)
    return st


def dequantize(wfmt, data, scales, n, out_f32=None, out_bf16=None, stream=None):
    _check(lib.ds4moe_dequantize(WFMT[wfmt] if isinstance(wfmt, str) else wfmt, _p(data), _p(scales), n,
                                 _p(out_f32), _p(out_bf16), _s(stream)))


def quantize_mxfp8(x, n, codes, scales, stream=None):
    """MXFP8-E4M3 codes [n] and E8M0 scales [n/32] of n bf16 values."""
    _check(lib.ds4moe_quantize_mxfp8(_p(x), n, _p(codes), _p(scales), _s(stream)))


def set_stage_events(stage, start=None, stop=None):
    """Record torch.cuda.Event pair (created with enable_timing=True and
    already recorded once, so that it has a HIP event handle) around every
    launch of `stage` ("route", "permute", "ffn_up", "ffn_down", "combine")
    on this thread; "router_proj" times ds4moe_router_logits; no events clears."""
    h = lambda e: None if e is None else ctypes.c_void_p(e.cuda_event)
    _check(lib.ds4moe_set_stage_events(STAGE[stage] if isinstance(stage, str) else stage, h(start), h(stop)))


# ---- products at original precision -------------------------------------------

def make_matmul(in_dim, out_dim, groups=1, dtype="bf16", act="none", grad=None, ldx=0, ldw=0, ldy=0,
                ldz=0) -> Matmul:
    """Descriptor of a dense or grouped product: weights [groups][out_dim][in_dim],
    `act` a key of ACT, `grad` the type of dw and dbias (default: dtype), row
    strides in elements (0: no gaps)."""
    return Matmul(in_dim, out_dim, groups, DTYPE[dtype], ACT[act], DTYPE[grad or dtype], ldx, ldw, ldy, ldz)


def matmul_workspace_bytes(m: Matmul, rows: int, backward: bool = False) -> int:
    return int(lib.ds4moe_matmul_workspace_bytes(ctypes.byref(m), rows, int(backward)))


def _here():
    """Index of the current HIP device, None without one."""
    import torch
    cuda = torch.cuda
    return cuda.current_device() if cuda.is_initialized() or cuda.is_available() else None


def _vector(name, t, dtype, n, dev):
    """Device pointer of at least `n` contiguous elements of `dtype` on device
    `dev` (None: NULL)."""
    if t is None:
        return None
    if t.dtype != dtype and dtype is not None:   # (None: the library refuses the descriptor)
        raise Ds4MoeError(-1, f"{name} is {t.dtype}, not {dtype}")
    if t.numel() < n or not t.is_contiguous():
        raise Ds4MoeError(-2, f"{name} of shape {tuple(t.shape)}, strides {t.stride()}: not {n} contiguous elements")
    if t.get_device() != dev:
        raise Ds4MoeError(-1, f"{name} on {t.device}, not on the current HIP device {dev}")
    return t.data_ptr()


def _workspace(t, dev):
    """Device pointer and bytes of a workspace of any type (None: NULL, 0)."""
    if t is None:
        return None, 0
    if not t.is_contiguous():
        raise Ds4MoeError(-2, f"workspace of shape {tuple(t.shape)}, strides {t.stride()} is not contiguous")
    if t.get_device() != dev:
        raise Ds4MoeError(-1, f"workspace on {t.device}, not on the current HIP device {dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def _rows_apart(shape, strides, rows, cols, ld):
    """Whether a tensor's first `rows` rows, counted over all its dimensions but
    the last, are `cols` or more elements that start `ld` apart."""
    if not shape or 0 in shape or (cols > 1 and strides[-1] != 1):
        return False
    if len(shape) == 1:                      # memory without rows
        return shape[0] >= (rows - 1) * ld + cols and (strides[0] == 1 or shape[0] == 1)
    n, i = 1, len(shape) - 2
    while i >= 0 and n < rows:
        if shape[i] != 1 and strides[i] != n * ld:
            return False
        n *= shape[i]
        i -= 1
    return shape[-1] >= cols and n >= rows


def _matrix(name, t, dtype, rows, cols, ld, dev):
    """Device pointer of `rows` rows of `cols` elements of `dtype`, `ld` apart
    (0: without gaps), on device `dev` (None: NULL).  A tensor may have more
    rows and columns than that."""
    if t is None:
        return None
    if t.dtype != dtype and dtype is not None:   # (None: the library refuses the descriptor)
        raise Ds4MoeError(-1, f"{name} is {t.dtype}, not {dtype}")
    ld = ld or cols
    shape, strides = t.shape, t.stride()
    # (two dimensions, the ordinary case, first: this is host time of every call)
    if not ((len(shape) == 2 and strides[0] == ld and strides[1] == 1 and shape[0] >= rows and shape[1] >= cols)
            or _rows_apart(shape, strides, rows, cols, ld)):
        raise Ds4MoeError(-2, f"{name} of shape {tuple(shape)}, strides {strides}: not {rows} rows of {cols} "
                              f"elements, {ld} apart")
    if t.get_device() != dev:
        raise Ds4MoeError(-1, f"{name} on {t.device}, not on the current HIP device {dev}")
    return t.data_ptr()


def _mm_plan(m):
    """A descriptor's types (of its tensors, of their gradients, int32), rows of
    w, columns of y, and the current device."""
    import torch
    types = (torch.float32, torch.bfloat16)
    dt, gd, n = m.dtype, m.grad_dtype, m.out_dim
    return (types[dt] if 0 <= dt <= 1 else None, types[gd] if 0 <= gd <= 1 else None, torch.int32, m.groups * n,
            n // 2 if m.act == ACT["swiglu"] else n, _here())


def _x_rows(x, rows):
    """Rows of x that a grouped call does not state."""
    if x is None:
        return rows
    return x.shape[0] if x.dim() < 2 or x.shape[-1] == 0 else x.numel() // x.shape[-1]


def linear(m, rows, x, w, y, bias=None, residual=None, z=None, workspace=None, stream=None):
    """y = act(x W^T + bias) + residual; z (optional) receives the pre-activations.
    Tensors whose type, size or row stride is not the descriptor's are refused
    (a tensor may have more rows and columns); w [.., out_dim, in_dim] and bias
    are counted over all their leading dimensions."""
    dt, _, _, wrows, oc, dev = _mm_plan(m)
    k, n, ldy = m.in_dim, m.out_dim, m.ldy
    ws, nws = _workspace(workspace, dev)
    _check(lib.ds4moe_linear(
        ctypes.byref(m), rows, _matrix("x", x, dt, rows, k, m.ldx, dev), _matrix("w", w, dt, wrows, k, m.ldw, dev),
        _vector("bias", bias, dt, wrows, dev), _matrix("residual", residual, dt, rows, oc, ldy, dev),
        _matrix("y", y, dt, rows, oc, ldy, dev), _matrix("z", z, dt, rows, n, m.ldz, dev), ws, nws, _s(stream, dev)))


def linear_backward(m, rows, x, w, dy, z=None, dx=None, dw=None, dbias=None, workspace=None, stream=None):
    """Gradients of linear: each of dx, dw, dbias that is given."""
    dt, gd, _, wrows, oc, dev = _mm_plan(m)
    k, n, ldx, ldw = m.in_dim, m.out_dim, m.ldx, m.ldw
    # (what the call does not read may be anything)
    x, w, z = None if dw is None else x, None if dx is None else w, z if m.act else None
    ws, nws = _workspace(workspace, dev)
    _check(lib.ds4moe_linear_backward(
        ctypes.byref(m), rows, _matrix("x", x, dt, rows, k, ldx, dev), _matrix("w", w, dt, wrows, k, ldw, dev),
        _matrix("z", z, dt, rows, n, m.ldz, dev), _matrix("dy", dy, dt, rows, oc, m.ldy, dev),
        _matrix("dx", dx, dt, rows, k, ldx, dev), _matrix("dw", dw, gd, wrows, k, ldw, dev),
        _vector("dbias", dbias, gd, wrows, dev), ws, nws, _s(stream, dev)))


def grouped_matmul(m, rows, x, w, expert_offsets, y, sorted_pair=None, top_k=1, x_rows=None, bias=None, z=None,
                   workspace=None, stream=None):
    """Products of expert-sorted rows with their experts' weights, from
    permute's expert_offsets (and sorted_pair, when rows are read from the
    tokens' x), both int32.  x_rows: x's rows (default: all that it has)."""
    dt, _, i32, wrows, oc, dev = _mm_plan(m)
    k, xr = m.in_dim, _x_rows(x, rows) if x_rows is None else x_rows
    ws, nws = _workspace(workspace, dev)
    _check(lib.ds4moe_grouped_matmul(
        ctypes.byref(m), rows, _matrix("x", x, dt, xr, k, m.ldx, dev), xr,
        _matrix("w", w, dt, wrows, k, m.ldw, dev), _vector("bias", bias, dt, wrows, dev),
        _vector("expert_offsets", expert_offsets, i32, m.groups + 1, dev),
        _vector("sorted_pair", sorted_pair, i32, rows, dev), top_k, _matrix("y", y, dt, rows, oc, m.ldy, dev),
        _matrix("z", z, dt, rows, m.out_dim, m.ldz, dev), ws, nws, _s(stream, dev)))


def grouped_matmul_backward(m, rows, x, w, expert_offsets, dy, z=None, sorted_pair=None, top_k=1, x_rows=None,
                            dx=None, dw=None, dbias=None, workspace=None, stream=None):
    """Gradients of grouped_matmul: each of dx (a row per sorted row), dw,
    dbias that is given.  x is read for dw only, but its row count is always
    part of the call (x_rows, if x is None)."""
    dt, gd, i32, wrows, oc, dev = _mm_plan(m)
    k, ldx, ldw, xr = m.in_dim, m.ldx, m.ldw, _x_rows(x, rows) if x_rows is None else x_rows
    x, w, z = None if dw is None else x, None if dx is None else w, z if m.act else None
    ws, nws = _workspace(workspace, dev)
    _check(lib.ds4moe_grouped_matmul_backward(
        ctypes.byref(m), rows, _matrix("x", x, dt, xr, k, ldx, dev), xr, _matrix("w", w, dt, wrows, k, ldw, dev),
        _matrix("z", z, dt, rows, m.out_dim, m.ldz, dev), _matrix("dy", dy, dt, rows, oc, m.ldy, dev),
        _vector("expert_offsets", expert_offsets, i32, m.groups + 1, dev),
        _vector("sorted_pair", sorted_pair, i32, rows, dev), top_k, _matrix("dx", dx, dt, rows, k, ldx, dev),
        _matrix("dw", dw, gd, wrows, k, ldw, dev), _vector("dbias", dbias, gd, wrows, dev), ws, nws, _s(stream, dev)))


# ---- token sampling ------------------------------------------------------------

def sample_workspace_bytes(B: int, V: int) -> int:
    return int(lib.ds4moe_sample_workspace_bytes(B, V))


def sample(B, V, logits, u, token, temperature=None, top_k=None, top_p=None, min_p=None, prob=None, workspace=None,
           stream=None):
    """token[B] (and prob[B]) sampled from logits [B][V] (fp32 or bf16; rows may
    be logits.stride(0) apart) with the random numbers u[B]; the filters' values
    are per row, None switches one off.  top_k and token are int32, the other
    vectors fp32, all contiguous; anything else, or fewer rows or tokens than B
    and V, is refused."""
    import torch
    f32, i32, dev = torch.float32, torch.int32, _here()
    if logits.dtype not in (f32, torch.bfloat16) or logits.stride(-1) != 1:
        raise Ds4MoeError(-1, f"logits {logits.dtype} with strides {logits.stride()}")
    dtype, ld = 0 if logits.dtype == f32 else 1, V
    if logits.size(-1) < V or logits.size(0) < (B if logits.dim() > 1 else B * V):
        raise Ds4MoeError(-2, f"logits of shape {tuple(logits.shape)} for {B} rows of {V}")
    if B > 1:
        ld = logits.stride(0)
    if logits.get_device() != dev:
        raise Ds4MoeError(-1, f"logits on {logits.device}, not on the current HIP device {dev}")
    ws, nws = _workspace(workspace, dev)
    _check(lib.ds4moe_sample(
        B, V, logits.data_ptr(), ld, dtype, _vector("temperature", temperature, f32, B, dev),
        _vector("top_k", top_k, i32, B, dev), _vector("top_p", top_p, f32, B, dev),
        _vector("min_p", min_p, f32, B, dev), _vector("u", u, f32, B, dev), _vector("token", token, i32, B, dev),
        _vector("prob", prob, f32, B, dev), ws, nws, _s(stream, dev)))
