"""ctypes binding of libecho.so (include/echo.h), with the same call names.

Argument marshalling only: tensors become device pointers, torch streams become
cudaStream_t handles, status codes become exceptions.  Every step of the
all-reduce runs in the library's CUDA kernels; there is no fallback.  Importing
this module raises if the library has not been built
(``python -m bit_error_compensated_gb300.build``).
"""
from __future__ import annotations

import ctypes
import struct
from pathlib import Path

_LIB_PATH = Path(__file__).resolve().parent / "lib" / "libecho.so"
if not _LIB_PATH.exists():
    raise ImportError(f"{_LIB_PATH} is missing: build it with "
                      "`python -m bit_error_compensated_gb300.build` (needs nvcc)")
_lib = ctypes.CDLL(str(_LIB_PATH))

ECHO_OK = 0
ECHO_ERR_ARG = 1
ECHO_ERR_SHAPE = 2
ECHO_ERR_UNSUPPORTED = 3
ECHO_ERR_ALIGN = 4
ECHO_ERR_CUDA = 5
ECHO_ERR_OVERFLOW = 6
ECHO_ERR_TIMEOUT = 7
ECHO_ERR_TOO_LARGE = 8
ECHO_NOALLOC_SCRATCH_BYTES = 32 << 20
ECHO_MAX_RANKS = 16
ECHO_QUANT_ZERO_AWARE = 0
ECHO_QUANT_NAIVE_ZERO_POINT = 1
ECHO_QUANT_SYMMETRIC = 2
ECHO_TILE_OFF = 0
ECHO_TILE_AUTO = 1
ECHO_TILE_RANK_LOOP = 2
ECHO_TILE_RANK_PARALLEL = 3
ECHO_STATE_F32 = 0
ECHO_STATE_BF16 = 1
ECHO_STATE_F16 = 2
COMP_DEFAULT = ctypes.c_void_p(-1 & (2 ** 64 - 1))   # ECHO_COMP_DEFAULT
ECHO_F32 = 0
ECHO_BF16 = 1
ECHO_F16 = 2
ECHO_NORM_RMS = 0
ECHO_NORM_LAYER = 1
ECHO_NORM_MAX_WIDTH = 16384
ECHO_MATMUL_MAX_ROWS = 1048576
ECHO_MATMUL_MAX_DEPTH = 131071

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t


# The C structures of the block operators: nothing but 64-bit integers and
# pointers, packed into bytes (cheaper than a ctypes.Structure per call).
_NORM_PARAMS = struct.Struct("4q")        # echo_norm_params: w_post, b_post, w_pre, b_pre
_NORM_IO = struct.Struct("16q")           # echo_norm_io
_NORM_GRAD_IO = struct.Struct("18q")      # echo_norm_grad_io
_MATRIX = struct.Struct("3q")             # echo_matrix: data, ld, rank_stride
_FEW_TOKENS = 32                          # up to here no product needs a workspace

_SIGS = {
    "echo_plan": (_i32, [_i32, _i64, _i32, _i32, ctypes.POINTER(_vp)]),
    "echo_allreduce": (_i32, [_vp, ctypes.POINTER(_vp), ctypes.POINTER(_vp), _vp, _vp]),
    "echo_reset_comp": (_i32, [_vp]),
    "echo_reset_comp_async": (_i32, [_vp, _vp, _vp]),
    "echo_comp_bytes": (_sz, [_vp]),
    "echo_wire_bytes": (_sz, [_vp]),
    "echo_wire_layout": (_i32, [_vp, ctypes.POINTER(_i64)]),
    "echo_get_status": (_i32, [_vp, _vp, ctypes.POINTER(_i32)]),
    "echo_debug_wire": (_i32, [_vp, _vp, _sz, _vp]),
    "echo_set_fused": (_i32, [_vp, _i32]),
    "echo_set_timing": (_i32, [_vp, ctypes.POINTER(_vp), _i32]),
    "echo_set_quantizer": (_i32, [_vp, _i32]),
    "echo_set_state": (_i32, [_vp, _i32, ctypes.c_float]),
    "echo_set_persistent": (_i32, [_vp, _i32]),
    "echo_set_tile_fused": (_i32, [_vp, _i32]),
    "echo_debug_hold_push": (_i32, [_vp, _i64]),
    "echo_debug_set_grid": (_i32, [_vp, _i32]),
    "echo_debug_check_guards": (_i32, [_vp, ctypes.POINTER(_i32)]),
    "echo_allreduce_noalloc": (_i32, [_i32, _i64, _i32, ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                      _vp, _vp]),
    "echo_plan_destroy": (None, [_vp]),
    "echo_norm_plan": (_i32, [_i64, _i32, _i32, _i32, _i32, ctypes.c_float, ctypes.c_float,
                              ctypes.POINTER(_vp)]),
    "echo_norm_plan_destroy": (None, [_vp]),
    "echo_norm": (_i32, [_vp, _vp, _vp, _vp]),
    "echo_norm_backward": (_i32, [_vp, _vp, _vp, _vp, _vp]),
    "echo_quantize_tokens": (_i32, [_i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp]),
    "echo_matmul_int8": (_i32, [_i64, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _i32, _vp,
                                _vp, _sz, _vp]),
    "echo_matmul_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _vp, _vp]),
    "echo_matmul_status": (_i32, [_vp, ctypes.POINTER(_i32)]),
    "echo_debug_hold_product": (_i32, [_i32]),
    "echo_linear_int8": (_i32, [_i64, _i64, _i64, _i64, _i32, _vp, _vp, _vp, _i64, _vp, _vp, _vp,
                                _vp, _sz, _vp]),
    "echo_strerror": (ctypes.c_char_p, [_i32]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)


class EchoError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {_lib.echo_strerror(status).decode()} (status {status})")


def _check(status: int, call: str):
    if status != ECHO_OK:
        raise EchoError(status, call)


def _ptr(x) -> int | None:
    """A device pointer from a tensor, an int address, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if isinstance(x, ctypes.c_void_p):
        return x.value
    return x.data_ptr()


def _tensor_ptrs(*args) -> list:
    """_ptr over (buffer, name, dtypes, min_numel) tuples, with the checks a
    torch tensor allows: the dtype, contiguous, large enough -- for every
    buffer first -- then on a CUDA device.  Raw addresses pass unchecked."""
    import torch
    tensors = [a for a in args if isinstance(a[0], torch.Tensor)]
    for t, what, dtypes, min_numel in tensors:
        if t.dtype not in dtypes:
            raise ValueError(f"{what}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
        if not t.is_contiguous():
            raise ValueError(f"{what}: tensor must be contiguous")
        if t.numel() < min_numel:
            raise ValueError(f"{what}: {t.numel()} elements, at least {min_numel} needed")
    for t, what, _, _ in tensors:
        if not t.is_cuda:
            raise ValueError(f"{what}: tensor must be on a CUDA device")
    return [_ptr(a[0]) for a in args]


def _buffers(P: int, n: int, ins, outs, comp_state, state_fmt: int):
    """Checked pointers of one call's P inputs, P outputs and state."""
    if len(ins) != P or len(outs) != P:
        raise ValueError(f"expected {P} input and {P} output buffers")
    bf = _bf16()
    args = ([(t, f"in[{p}]", bf, n) for p, t in enumerate(ins)]
            + [(t, f"out[{p}]", bf, n) for p, t in enumerate(outs)]
            + [(None if comp_state is COMP_DEFAULT else comp_state, "comp_state",
                _state_dtypes(state_fmt), P * n)])
    ptrs = _tensor_ptrs(*args)
    comp = COMP_DEFAULT if comp_state is COMP_DEFAULT else ptrs[2 * P]
    return (_vp * P)(*ptrs[:P]), (_vp * P)(*ptrs[P:2 * P]), comp


def _bf16():
    import torch
    return (torch.bfloat16,)


def _state_dtypes(fmt: int):
    import torch
    return ((torch.float32,), (torch.bfloat16,), (torch.float16,))[fmt]


def _stream(stream, device=None) -> int | None:
    """The raw stream; of the current device (its number, where the caller has it) if None."""
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:                       # without making a Stream object: 0.1 us, not 3
            return raw(torch.cuda.current_device() if device is None else device)
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Plan:
    """Owning handle of an echo_plan_t; frees the plan when collected."""

    def __init__(self, handle: int, P: int, n: int, g: int, bits: int):
        self.handle = handle
        self.P, self.n, self.g, self.bits = P, n, g, bits
        self.state_fmt = ECHO_STATE_F32          # kept in step with echo_set_state

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            _lib.echo_plan_destroy(h)

    @property
    def _as_parameter_(self):
        return ctypes.c_void_p(self.handle)


def echo_plan(P: int, n: int, g: int = 128, bits: int = 4) -> Plan:
    h = _vp()
    _check(_lib.echo_plan(P, n, g, bits, ctypes.byref(h)), "echo_plan")
    return Plan(h.value, P, n, g, bits)


def echo_allreduce(plan: Plan, ins, outs, comp_state=None, stream=None) -> None:
    """ins/outs: sequences of P device tensors (or int addresses); comp_state:
    None (uncompensated), COMP_DEFAULT (the plan's own state) or a device
    buffer of echo_comp_bytes(plan) bytes."""
    arr_in, arr_out, comp = _buffers(plan.P, plan.n, ins, outs, comp_state, plan.state_fmt)
    _check(_lib.echo_allreduce(plan, arr_in, arr_out, comp, _stream(stream)), "echo_allreduce")


class PreparedCall:
    """echo_allreduce with its buffers checked and marshalled once, for a loop
    that repeats one call on the same buffers (an all-reduce site of a model,
    a benchmark): calling it issues only the C call, without re-checking the
    2P + 1 buffers (about 1 us a buffer in Python), which is what dominates the
    cost of a call on a small message.  It keeps references to the buffers so
    that they stay allocated; their addresses are taken once, so a buffer must
    not be resized or re-pointed while the prepared call is in use.  Calling it
    after the plan's state format changed, or after the plan was destroyed,
    raises ValueError."""

    __slots__ = ("plan", "_keep", "_fmt", "_args")

    def __init__(self, plan: Plan, ins, outs, comp_state=None):
        arr_in, arr_out, comp = _buffers(plan.P, plan.n, ins, outs, comp_state, plan.state_fmt)
        self.plan = plan
        self._keep = (tuple(ins), tuple(outs), comp_state)
        self._fmt = plan.state_fmt
        self._args = (_vp(plan.handle), arr_in, arr_out, comp)

    def __call__(self, stream=None) -> None:
        if self.plan.handle is None or self.plan.handle != self._args[0].value:
            raise ValueError("prepared call: its plan was destroyed")
        if self.plan.state_fmt != self._fmt:
            raise ValueError("prepared call: the plan's state format changed; prepare it again")
        _check(_lib.echo_allreduce(*self._args, _stream(stream)), "echo_allreduce")


def prepare_allreduce(plan: Plan, ins, outs, comp_state=None) -> PreparedCall:
    """A PreparedCall of echo_allreduce(plan, ins, outs, comp_state)."""
    return PreparedCall(plan, ins, outs, comp_state)


def echo_reset_comp(plan: Plan) -> None:
    _check(_lib.echo_reset_comp(plan), "echo_reset_comp")


def echo_reset_comp_async(plan: Plan, comp_state=COMP_DEFAULT, stream=None) -> None:
    comp = COMP_DEFAULT if comp_state is COMP_DEFAULT else _tensor_ptrs(
        (comp_state, "comp_state", _state_dtypes(plan.state_fmt), plan.P * plan.n))[0]
    _check(_lib.echo_reset_comp_async(plan, comp, _stream(stream)), "echo_reset_comp_async")


def echo_comp_bytes(plan: Plan) -> int:
    return int(_lib.echo_comp_bytes(plan))


def echo_wire_bytes(plan: Plan) -> int:
    return int(_lib.echo_wire_bytes(plan))


def echo_wire_layout(plan: Plan) -> dict:
    d = (_i64 * 8)()
    _check(_lib.echo_wire_layout(plan, d), "echo_wire_layout")
    keys = ("codes1", "meta1", "codes2", "meta2", "Gs", "Gs_pad", "code_bytes", "total")
    return dict(zip(keys, [int(v) for v in d]))


def echo_get_status(plan: Plan, stream=None) -> int:
    st = _i32(0)
    _check(_lib.echo_get_status(plan, _stream(stream), ctypes.byref(st)), "echo_get_status")
    return st.value


def echo_debug_wire(plan: Plan, stream=None) -> bytes:
    nbytes = echo_wire_bytes(plan)
    buf = (ctypes.c_uint8 * max(nbytes, 1))()
    _check(_lib.echo_debug_wire(plan, buf, nbytes, _stream(stream)), "echo_debug_wire")
    return bytes(buf)[:nbytes]


def echo_set_fused(plan: Plan, fused: bool) -> None:
    _check(_lib.echo_set_fused(plan, 1 if fused else 0), "echo_set_fused")


def echo_set_quantizer(plan: Plan, mode: int) -> None:
    _check(_lib.echo_set_quantizer(plan, mode), "echo_set_quantizer")


def echo_set_state(plan: Plan, fmt: int = ECHO_STATE_F32, decay: float = 1.0) -> None:
    _check(_lib.echo_set_state(plan, fmt, decay), "echo_set_state")
    plan.state_fmt = fmt


def echo_set_tile_fused(plan: Plan, on: int) -> None:
    """on: ECHO_TILE_OFF/AUTO/RANK_LOOP/RANK_PARALLEL; False and True mean OFF and AUTO."""
    _check(_lib.echo_set_tile_fused(plan, int(on)), "echo_set_tile_fused")


def echo_set_persistent(plan: Plan, on: bool) -> None:
    _check(_lib.echo_set_persistent(plan, 1 if on else 0), "echo_set_persistent")


def echo_debug_hold_push(plan: Plan, item: int) -> None:
    _check(_lib.echo_debug_hold_push(plan, item), "echo_debug_hold_push")


def echo_debug_set_grid(plan: Plan, blocks: int) -> None:
    _check(_lib.echo_debug_set_grid(plan, blocks), "echo_debug_set_grid")


def echo_debug_check_guards(plan: Plan) -> bool:
    intact = ctypes.c_int(0)
    _check(_lib.echo_debug_check_guards(plan, ctypes.byref(intact)), "echo_debug_check_guards")
    return bool(intact.value)


def echo_set_timing(plan: Plan, events) -> None:
    """events: four torch.cuda.Event (enable_timing=True), or None to disable."""
    if not events:
        _check(_lib.echo_set_timing(plan, None, 0), "echo_set_timing")
        return
    arr = (_vp * 4)(*[ev.cuda_event for ev in events])
    _check(_lib.echo_set_timing(plan, arr, 4), "echo_set_timing")


def echo_allreduce_noalloc(P: int, n: int, bits: int, ins, outs, comp_state=None,
                           stream=None) -> None:
    """The no-allocation call (see include/echo.h): no plan, receive slots in
    the library's fixed device array; comp_state is None or a caller buffer."""
    arr_in, arr_out, comp = _buffers(P, n, ins, outs, comp_state, ECHO_STATE_F32)
    _check(_lib.echo_allreduce_noalloc(P, n, bits, arr_in, arr_out, comp,
                                       _stream(stream)), "echo_allreduce_noalloc")


def echo_plan_destroy(plan: Plan) -> None:
    h, plan.handle = plan.handle, None
    if h:
        _lib.echo_plan_destroy(h)


# ---------------------------------------------------------------------------
# The operators on either side of the all-reduce.  Their arguments are tensors
# (strides and sizes are read from them); outputs are the caller's buffers.
# A decode loop makes these calls once a token and layer, so the checks are one
# cheap test of each tensor (_fits); only a tensor that fails it goes through
# _refuse, which says what is wrong.

_CODES = {}                                   # torch.dtype -> ECHO_*, filled by the first call


def _dtype_code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        import torch
        _CODES.update({torch.float32: ECHO_F32, torch.bfloat16: ECHO_BF16, torch.float16: ECHO_F16})
        code = _CODES.get(dtype)
    if code is None:
        raise ValueError(f"dtype {dtype}, expected float32, bfloat16 or float16")
    return code


def _fits(t, dtype, shape, device) -> bool:
    """Of this dtype, shape and device, the elements of a row contiguous."""
    return (t.dtype is dtype and t.shape == shape and t.get_device() == device
            and (t.stride()[-1] == 1 or shape[-1] <= 1))


def _refuse(t, what: str, dtype, shape, device) -> None:
    if t.dtype != dtype:
        raise ValueError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what}: elements of a row must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{what}: tensor must be on a CUDA device")
    raise ValueError(f"{what}: tensor on cuda:{t.get_device()}, but the call runs on cuda:{device}")


def _expect(t, what: str, dtype, shape, device) -> None:
    if not _fits(t, dtype, shape, device):
        _refuse(t, what, dtype, shape, device)


def _expect_contiguous(t, what: str, dtype, shape, device) -> None:
    if not _fits(t, dtype, shape, device):
        _refuse(t, what, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")


def _call_device(t, plan=None) -> int:
    """The device that a call runs on: the current one, and the plan's."""
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    import torch
    device = torch.cuda.current_device()
    if plan is not None and plan.device != device:
        raise ValueError(f"the plan belongs to cuda:{plan.device}, but the current device is cuda:{device}")
    return device


class NormPlan:
    """Owning handle of an echo_norm_plan_t; frees the plan when collected."""

    def __init__(self, handle, width, dtype, param_dtype, kind, post, device):
        self.handle = handle
        self.width, self.dtype, self.param_dtype = width, dtype, param_dtype
        self.kind, self.post, self.device = kind, post, device

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            _lib.echo_norm_plan_destroy(h)


def echo_norm_plan(width: int, dtype, param_dtype=None, kind: int = ECHO_NORM_RMS, post: bool = True,
                   eps: float = 1e-6, scale: float = 1.0) -> NormPlan:
    """A residual join (include/echo.h): rows of `width` elements of `dtype`,
    parameters and gate of `param_dtype` (dtype if None, or torch.float32)."""
    import torch
    param_dtype = dtype if param_dtype is None else param_dtype
    h = _vp()
    _check(_lib.echo_norm_plan(width, _dtype_code(dtype), _dtype_code(param_dtype), kind, int(post),
                               eps, scale, ctypes.byref(h)), "echo_norm_plan")
    return NormPlan(h.value, width, dtype, param_dtype, kind, bool(post), torch.cuda.current_device())


def echo_norm_plan_destroy(plan: NormPlan) -> None:
    h, plan.handle = plan.handle, None
    if h:
        _lib.echo_norm_plan_destroy(h)


class NormParams:
    """The weights and biases of a plan's norms (or their gradients), checked
    once: contiguous tensors of `width` elements of the plan's param_dtype, or
    None.  Keeps the tensors.  A call reads their addresses again (0.1 us each),
    and where one has changed (a module was moved, .data assigned) checks the
    tensors anew: it reads what they hold now, or raises ValueError."""

    __slots__ = ("_all", "_there", "_at", "_plan", "_packed")

    def __init__(self, plan: NormPlan, w_post=None, b_post=None, w_pre=None, b_pre=None):
        self._all = (w_post, b_post, w_pre, b_pre)
        self._there = tuple(t for t in self._all if t is not None)
        self._plan = plan
        self._check()

    def _check(self) -> None:
        plan = self._plan
        self._at = None                           # a call after a refusal checks again
        for t, what in zip(self._all, ("w_post", "b_post", "w_pre", "b_pre")):
            if t is not None:
                _expect_contiguous(t, what, plan.param_dtype, (plan.width,), plan.device)
                if t.data_ptr() == 0:
                    raise ValueError(f"{what}: the tensor's storage was freed")
        self._packed = _NORM_PARAMS.pack(*[0 if t is None else t.data_ptr() for t in self._all])
        self._at = [t.data_ptr() for t in self._there]


def _packed_params(plan: NormPlan, params):
    if params is None:
        return None
    if params._plan is not plan:
        raise ValueError("these parameters were checked for another plan")
    if [t.data_ptr() for t in params._there] != params._at:
        params._check()
    return params._packed


def _norm_rows(plan: NormPlan, x) -> int:
    if plan.handle is None:
        raise ValueError("the plan was destroyed")
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected (rows, {plan.width})")
    return x.shape[0]


def _norm_gate(plan: NormPlan, gate, dgate, rows: int) -> tuple:
    """(address, rows, columns) of a gate of [rows or fewer][width or 1]."""
    if gate is None:
        if dgate is not None:
            raise ValueError("dgate without gate")
        return 0, 0, 0
    shape = tuple(gate.shape)
    if len(shape) != 2 or shape[1] not in (plan.width, 1) or shape[0] < 1 or rows % shape[0]:
        raise ValueError(f"gate: shape {shape}, expected (rows of which {rows} is a multiple, "
                         f"{plan.width} or 1)")
    _expect_contiguous(gate, "gate", plan.param_dtype, shape, plan.device)
    if dgate is not None:
        _expect_contiguous(dgate, "dgate", plan.param_dtype, shape, plan.device)
    return gate.data_ptr(), shape[0], shape[1]


def echo_norm(plan: NormPlan, params: NormParams | None, x, y=None, r=None, h=None, gate=None,
              codes=None, scales=None, stats=None, stream=None) -> None:
    """x, y, r, h: [rows][width] tensors of the plan's dtype, any row distance
    (y, r, h may be None); gate: [gate rows][width or 1]; codes int8
    [rows][width] with scales fp32 [rows]; stats fp32 [rows][4]."""
    rows = _norm_rows(plan, x)
    shape, dtype, device = (rows, plan.width), plan.dtype, plan.device
    _expect(x, "x", dtype, shape, device)
    _call_device(x, plan)
    at_y = at_r = at_h = at_codes = at_scales = at_stats = ld_y = ld_r = ld_h = ld_codes = 0
    if y is not None:
        _expect(y, "y", dtype, shape, device)
        at_y, ld_y = y.data_ptr(), y.stride()[0]
    if r is not None:
        _expect(r, "r", dtype, shape, device)
        at_r, ld_r = r.data_ptr(), r.stride()[0]
    if h is not None:
        _expect(h, "h", dtype, shape, device)
        at_h, ld_h = h.data_ptr(), h.stride()[0]
    if (codes is None) != (scales is None):
        raise ValueError("codes and scales belong together")
    if codes is not None:
        import torch
        _expect(codes, "codes", torch.int8, shape, device)
        _expect_contiguous(scales, "scales", torch.float32, (rows,), device)
        at_codes, ld_codes, at_scales = codes.data_ptr(), codes.stride()[0], scales.data_ptr()
    if stats is not None:
        import torch
        _expect_contiguous(stats, "stats", torch.float32, (rows, 4), device)
        at_stats = stats.data_ptr()
    at_gate, gate_rows, gate_cols = _norm_gate(plan, gate, None, rows)
    io = _NORM_IO.pack(rows, x.data_ptr(), x.stride()[0], at_y, ld_y, at_gate, gate_rows, gate_cols,
                       at_r, ld_r, at_h, ld_h, at_codes, ld_codes, at_scales, at_stats)
    status = _lib.echo_norm(plan.handle, _packed_params(plan, params), io, _stream(stream, device))
    if status:
        raise EchoError(status, "echo_norm")


def echo_norm_backward(plan: NormPlan, params: NormParams | None, x, y, stats, dr, dh, dx=None,
                       dy=None, grads: NormParams | None = None, gate=None, dgate=None,
                       stream=None) -> None:
    """x, y, gate, stats as in the forward call; dr, dh: gradients of r and h
    (either may be None); dx, dy, dgate and grads (a NormParams of the plan
    holding the tensors to write) receive the gradients."""
    import torch
    rows = _norm_rows(plan, x)
    shape, device = (rows, plan.width), plan.device
    at = []
    for t, what in ((x, "x"), (y, "y"), (dr, "dr"), (dh, "dh"), (dx, "dx"), (dy, "dy")):
        if t is None:
            at += (0, 0)
        else:
            _expect(t, what, plan.dtype, shape, device)
            at += (t.data_ptr(), t.stride()[0])
    _call_device(x, plan)
    if stats is not None:
        _expect_contiguous(stats, "stats", torch.float32, (rows, 4), device)
    gate_args = _norm_gate(plan, gate, dgate, rows)
    io = _NORM_GRAD_IO.pack(rows, *at[:4], *gate_args, 0 if stats is None else stats.data_ptr(), *at[4:],
                            0 if dgate is None else dgate.data_ptr())
    status = _lib.echo_norm_backward(plan.handle, _packed_params(plan, params), io,
                                     _packed_params(plan, grads), _stream(stream, device))
    if status:
        raise EchoError(status, "echo_norm_backward")


def _matrix(t) -> bytes:
    """A [ranks][rows][cols] tensor, or a [rows][cols] one that all ranks share."""
    stride = t.stride()
    if len(stride) == 2:
        return _MATRIX.pack(t.data_ptr(), stride[0], 0)
    return _MATRIX.pack(t.data_ptr(), stride[1], stride[0] if t.shape[0] > 1 else 0)


def _expect_matrix(t, what: str, dtype, shape, device) -> bytes:
    """_expect and _matrix of a two- or three-dimensional shape in one."""
    stride = t.stride()
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == device
            and (stride[-1] == 1 or shape[-1] <= 1)):
        _refuse(t, what, dtype, shape, device)
    if len(stride) == 2:
        return _MATRIX.pack(t.data_ptr(), stride[0], 0)
    return _MATRIX.pack(t.data_ptr(), stride[1], stride[0] if shape[0] > 1 else 0)


def _batch(t, what: str) -> tuple:
    """(ranks, rows, columns) of a two- or three-dimensional tensor."""
    shape = t.shape
    if len(shape) == 2:
        return 1, shape[0], shape[1]
    if len(shape) == 3:
        return shape
    raise ValueError(f"{what}: shape {tuple(shape)}, expected two or three dimensions")


def _check_product(tokens_of, what: str, dtype, scales, w, w_scales, out, device: int) -> tuple:
    """(ranks, tokens, channels, depth, and the matrices of the tokens' tensor,
    w and out) of a product whose tensors fit: out [ranks][tokens][channels] or
    without ranks, the tokens' tensor and scales, w and w_scales each with the
    ranks' dimension or without it."""
    import torch
    ranks, tokens, channels = _batch(out, "out")
    depth = w.shape[-1]
    own = len(tokens_of.shape) == 3
    a = _expect_matrix(tokens_of, what, dtype, (ranks, tokens, depth) if own else (tokens, depth), device)
    _expect_contiguous(scales, "scales", torch.float32, (ranks, tokens) if own else (tokens,), device)
    wm = _expect_matrix(w, "w", torch.int8,
                        (ranks, channels, depth) if len(w.shape) == 3 else (channels, depth), device)
    _expect(w_scales, "w_scales", torch.float32,
            (ranks, channels) if len(w_scales.shape) == 2 else (channels,), device)
    return ranks, tokens, channels, depth, a, wm, _expect_matrix(out, "out", out.dtype, out.shape, device)


def _workspace(nbytes: int, device, stream) -> tuple:
    """(tensor or None, address) of a product's workspace, from torch's
    allocator: ordered by the stream that the call runs on."""
    if nbytes == 0:
        return None, None
    import torch
    buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if stream is not None:
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        if stream != torch.cuda.current_stream():
            stream.wait_stream(torch.cuda.current_stream())   # the memory's last use lies on this one
            buf.record_stream(stream)
    return buf, buf.data_ptr()


def echo_matmul_workspace_bytes(ranks: int, tokens: int, channels: int, depth: int, codes, w) -> int:
    """codes, w: the tensors of the call."""
    return int(_lib.echo_matmul_workspace_bytes(ranks, tokens, channels, depth, _matrix(codes), _matrix(w)))


def echo_quantize_tokens(x, codes, scales, stream=None) -> None:
    """x [ranks][tokens][depth] (or [tokens][depth]) to int8 codes of the same
    shape and one fp32 scale a token, [ranks][tokens] contiguous."""
    import torch
    ranks, tokens, depth = _batch(x, "x")
    dtype, shape = _dtype_code(x.dtype), x.shape
    device = _call_device(x)
    _expect(x, "x", x.dtype, shape, device)
    _expect(codes, "codes", torch.int8, shape, device)
    _expect_contiguous(scales, "scales", torch.float32, shape[:-1], device)
    status = _lib.echo_quantize_tokens(ranks, tokens, depth, dtype, _matrix(x), _matrix(codes),
                                       scales.data_ptr(), _stream(stream, device))
    if status:
        raise EchoError(status, "echo_quantize_tokens")


def echo_matmul_int8(codes, scales, w, w_scales, out, stream=None) -> None:
    """out[p][t][c] = sum_k codes[p][t][k] w[p][c][k] * scales[p][t] * w_scales[p][c].
    out: [ranks][tokens][channels], or without ranks; codes with scales, w and
    w_scales: with the ranks' dimension, or without it where all ranks share
    them (codes and scales both)."""
    import torch
    device = _call_device(out)
    ranks, tokens, channels, depth, a, wm, om = _check_product(codes, "codes", torch.int8, scales, w, w_scales,
                                                               out, device)
    keep, at, nbytes = None, None, 0
    if tokens > _FEW_TOKENS:
        nbytes = _lib.echo_matmul_workspace_bytes(ranks, tokens, channels, depth, a, wm)
        keep, at = _workspace(nbytes, out.device, stream)
    status = _lib.echo_matmul_int8(ranks, tokens, channels, depth, a, scales.data_ptr(),
                                   tokens if len(codes.shape) == 3 else 0, wm, w_scales.data_ptr(),
                                   w_scales.stride()[0] if len(w_scales.shape) == 2 else 0,
                                   _dtype_code(out.dtype), om, at, nbytes, _stream(stream, device))
    if status:
        raise EchoError(status, "echo_matmul_int8")


def echo_matmul_status(stream=None) -> int:
    st = _i32(0)
    _check(_lib.echo_matmul_status(_stream(stream), ctypes.byref(st)), "echo_matmul_status")
    return st.value


def echo_debug_hold_product(on: bool) -> None:
    _check(_lib.echo_debug_hold_product(1 if on else 0), "echo_debug_hold_product")


def echo_linear_int8(x, w, w_scales, out, codes, scales, stream=None) -> None:
    """echo_quantize_tokens(x, codes, scales), then echo_matmul_int8 of them:
    x [ranks][tokens][depth] (or without ranks) and out of one dtype; codes
    and scales are the caller's buffers for the quantized tokens."""
    import torch
    device = _call_device(out)
    ranks, tokens, channels, depth, a, wm, om = _check_product(codes, "codes", torch.int8, scales, w, w_scales,
                                                               out, device)
    if len(x.shape) != len(out.shape):
        raise ValueError(f"x: shape {tuple(x.shape)}, expected the {len(out.shape)} dimensions of out")
    xm = _expect_matrix(x, "x", out.dtype, codes.shape, device)
    keep, at, nbytes = None, None, 0
    if tokens > _FEW_TOKENS:
        nbytes = _lib.echo_matmul_workspace_bytes(ranks, tokens, channels, depth, a, wm)
        keep, at = _workspace(nbytes, out.device, stream)
    status = _lib.echo_linear_int8(ranks, tokens, channels, depth, _dtype_code(x.dtype), xm, wm,
                                   w_scales.data_ptr(),
                                   w_scales.stride()[0] if len(w_scales.shape) == 2 else 0,
                                   a, scales.data_ptr(), om, at, nbytes, _stream(stream, device))
    if status:
        raise EchoError(status, "echo_linear_int8")


def echo_strerror(status: int) -> str:
    return _lib.echo_strerror(status).decode()


def library_path() -> str:
    return str(_LIB_PATH)
