"""Host side of the block operators without a GPU: the C calls' argument checks
(reported before any CUDA call), the packed structures against include/echo.h,
and the binding's refusal of tensors that are not on a GPU."""
import ctypes
import re
from pathlib import Path

import pytest
import torch

ROOT = Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def lib():
    from bit_error_compensated_gb300.build import build_library
    return ctypes.CDLL(str(build_library()))


def test_packed_structures_follow_the_header():
    """Every field of the header's structures is 8 bytes, in the order and
    number that the binding packs."""
    from bit_error_compensated_gb300 import echo
    text = re.sub(r"/\*.*?\*/", "", (ROOT / "include" / "echo.h").read_text(), flags=re.S)
    for name, packed, fields in (
            ("echo_norm_params", echo._NORM_PARAMS, ["w_post", "b_post", "w_pre", "b_pre"]),
            ("echo_norm_io", echo._NORM_IO,
             ["rows", "x", "ld_x", "y", "ld_y", "gate", "gate_rows", "gate_cols", "r", "ld_r", "h", "ld_h",
              "codes", "ld_codes", "scales", "stats"]),
            ("echo_norm_grad_io", echo._NORM_GRAD_IO,
             ["rows", "x", "ld_x", "y", "ld_y", "gate", "gate_rows", "gate_cols", "stats", "dr", "ld_dr", "dh",
              "ld_dh", "dx", "ld_dx", "dy", "ld_dy", "dgate"]),
            ("echo_matrix", echo._MATRIX, ["data", "ld", "rank_stride"])):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)
        declared = []
        for line in body.split(";"):
            line = line.strip()
            if not line:
                continue
            assert line.startswith("int64_t ") or "*" in line, line          # 8 bytes each
            declared += [re.search(r"(\w+)\s*$", part).group(1) for part in line.split(",")]
        assert declared == fields
        assert packed.size == 8 * len(fields)


def test_constants_match_the_header():
    from bit_error_compensated_gb300 import echo
    text = (ROOT / "include" / "echo.h").read_text()
    for name in ("ECHO_F32", "ECHO_BF16", "ECHO_F16", "ECHO_NORM_RMS", "ECHO_NORM_LAYER", "ECHO_NORM_MAX_WIDTH",
                 "ECHO_MATMUL_MAX_ROWS", "ECHO_MATMUL_MAX_DEPTH"):
        m = re.search(rf"#define {name}\s+(\d+)", text)
        assert m and int(m.group(1)) == getattr(echo, name), name


def test_norm_arguments_are_checked_before_any_cuda_call(lib):
    from bit_error_compensated_gb300 import echo
    h = ctypes.c_void_p(1)
    plan = lib.echo_norm_plan
    plan.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float,
                     ctypes.c_float, ctypes.POINTER(ctypes.c_void_p)]

    def status(width=64, dtype=1, param=1, kind=0, post=1, eps=1e-6, scale=1.0, out=ctypes.byref(h)):
        return plan(width, dtype, param, kind, post, eps, scale, out)

    assert status(out=None) == echo.ECHO_ERR_ARG
    assert status(kind=2) == status(post=2) == echo.ECHO_ERR_ARG
    assert status(eps=-1.0) == status(eps=float("nan")) == status(scale=float("inf")) == echo.ECHO_ERR_ARG
    assert status(dtype=3) == status(param=2) == status(width=16385) == echo.ECHO_ERR_UNSUPPORTED
    assert status(dtype=0, param=1) == echo.ECHO_ERR_UNSUPPORTED
    assert status(width=0) == status(width=-4) == echo.ECHO_ERR_SHAPE
    assert h.value is None
    assert lib.echo_norm(None, None, None, None) == echo.ECHO_ERR_ARG
    assert lib.echo_norm_backward(None, None, None, None, None) == echo.ECHO_ERR_ARG
    lib.echo_norm_plan_destroy(None)


def test_product_arguments_are_checked_before_any_cuda_call(lib):
    from bit_error_compensated_gb300 import echo
    base = 1 << 20
    matrix = lambda at, ld, stride=0: echo._MATRIX.pack(at, ld, stride)          # noqa: E731

    def status(ranks=1, tokens=4, channels=8, depth=16, a=matrix(base, 16), sa=base * 2, w=matrix(base * 3, 16),
               sw=base * 4, dtype=1, out=matrix(base * 5, 8), workspace=None, nbytes=0):
        return echo._lib.echo_matmul_int8(ranks, tokens, channels, depth, a, sa, 0, w, sw, 0, dtype, out,
                                          workspace, nbytes, None)

    assert status(ranks=0) == status(ranks=17) == echo.ECHO_ERR_ARG
    assert status(tokens=-1) == status(depth=-1) == echo.ECHO_ERR_SHAPE
    assert status(depth=131072) == status(tokens=2 ** 20 + 1) == status(dtype=5) == echo.ECHO_ERR_UNSUPPORTED
    assert status(a=None) == status(sa=None) == status(out=matrix(0, 8)) == echo.ECHO_ERR_ARG
    assert status(a=matrix(base, 15)) == status(w=matrix(base * 3, 1)) == echo.ECHO_ERR_SHAPE
    assert status(out=matrix(base * 5 + 1, 8)) == status(sw=base * 4 + 2) == echo.ECHO_ERR_ALIGN
    assert status(out=matrix(base + 16, 8)) == echo.ECHO_ERR_ARG                 # over the codes
    assert status(ranks=2, out=matrix(base * 5, 8, 16)) == echo.ECHO_ERR_ARG     # ranks' results overlap
    assert status(tokens=33, a=matrix(base, 16)) == echo.ECHO_ERR_TOO_LARGE      # no workspace
    assert status(tokens=33, workspace=base * 9, nbytes=100) == echo.ECHO_ERR_TOO_LARGE
    assert status(tokens=33, workspace=base * 9 + 8, nbytes=1 << 20) == echo.ECHO_ERR_ALIGN
    assert echo._lib.echo_matmul_status(None, None) == echo.ECHO_ERR_ARG
    assert echo._lib.echo_debug_hold_product(2) == echo.ECHO_ERR_ARG


def test_workspace_bytes():
    """Two bytes a code of the tokens, rounded up to 128 x 128, ranks that share
    them once; a byte a code of channels whose rows are not aligned."""
    from bit_error_compensated_gb300 import echo
    z = lambda *s: torch.zeros(s, dtype=torch.int8)                              # noqa: E731
    need = echo.echo_matmul_workspace_bytes
    a, w = z(200, 144), z(64, 144)
    assert need(1, 200, 64, 144, a, w) == 2 * 256 * 256
    assert need(1, 32, 64, 144, z(32, 144), w) == 0 == need(1, 200, 64, 0, z(200, 0), z(64, 0))
    assert need(3, 200, 64, 144, a, w) == 2 * 256 * 256
    assert need(3, 200, 64, 144, z(3, 200, 144), w) == 3 * 2 * 256 * 256
    odd = z(64, 145)[:, :144]
    assert need(1, 200, 64, 144, a, odd) == 2 * 256 * 256 + 64 * 144
    assert need(2, 200, 64, 131, z(200, 131), z(2, 64, 131)) == 2 * 256 * 256 + 2 * 64 * 144


def test_tensors_have_to_be_on_the_gpu():
    from bit_error_compensated_gb300 import echo
    x = torch.zeros(4, 16)
    codes, scales, out = torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4), torch.zeros(4, 8)
    w, ws = torch.zeros(8, 16, dtype=torch.int8), torch.zeros(8)
    for call in (lambda: echo.echo_quantize_tokens(x, codes, scales),
                 lambda: echo.echo_matmul_int8(codes, scales, w, ws, out),
                 lambda: echo.echo_linear_int8(x, w, ws, out, codes, scales)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    plan = echo.NormPlan(0, 16, torch.float32, torch.float32, 0, True, 0)      # stands in for a plan
    with pytest.raises(ValueError, match="CUDA device"):
        echo.echo_norm(plan, None, x, x.clone(), x.clone())
    with pytest.raises(ValueError, match="CUDA device"):
        echo.NormParams(plan, w_pre=torch.zeros(16))
    with pytest.raises(ValueError, match="shape"):
        echo.NormParams(plan, w_pre=torch.zeros(15))
    with pytest.raises(ValueError, match="dtype"):
        echo.NormParams(plan, w_pre=torch.zeros(16, dtype=torch.float16))
    echo.echo_norm_plan_destroy(plan)
    with pytest.raises(ValueError, match="destroyed"):
        echo.echo_norm(plan, None, x)
    with pytest.raises(ValueError, match="dimensions"):
        echo.echo_quantize_tokens(torch.zeros(4), codes, scales)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        echo.echo_quantize_tokens(x.double(), codes, scales)


def test_parameters_that_move_are_read_where_they_are():
    """A tensor whose memory is another one since it was checked (module.to, an
    assignment to .data) is checked and packed anew by the next call; one that
    no longer fits, or whose memory is gone, is refused.  (The device number -1
    stands for the CPU.)"""
    from bit_error_compensated_gb300 import echo
    plan = echo.NormPlan(0, 16, torch.float32, torch.float32, 0, True, -1)
    w, b = torch.zeros(16), torch.ones(16)
    params = echo.NormParams(plan, w_pre=w, w_post=b)
    packed = lambda: echo._NORM_PARAMS.unpack(echo._packed_params(plan, params))          # noqa: E731
    assert packed() == (b.data_ptr(), 0, w.data_ptr(), 0)
    was, w.data = w.detach(), torch.ones(16)
    assert w.data_ptr() != was.data_ptr()
    assert packed() == (b.data_ptr(), 0, w.data_ptr(), 0)
    for bad, word in ((torch.ones(16, dtype=torch.float16), "dtype"), (torch.ones(15), "shape"),
                      (torch.ones(32)[::2], "contiguous")):
        good, w.data = w.detach(), bad
        for _ in range(2):
            with pytest.raises(ValueError, match="w_pre: .*" + word):
                packed()
        w.data = good
        assert packed() == (b.data_ptr(), 0, w.data_ptr(), 0)
    w.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="w_pre: .*freed"):
        packed()


def test_texts_of_errors_name_the_operators():
    """The text of a status says what it means for a norm and a product too."""
    from bit_error_compensated_gb300 import echo
    for status, words in ((echo.ECHO_ERR_SHAPE, ("multiple of P*g", "rows", "gate")),
                          (echo.ECHO_ERR_UNSUPPORTED, ("bits", "width", "product", "types")),
                          (echo.ECHO_ERR_ALIGN, ("aligned", "stats", "workspace")),
                          (echo.ECHO_ERR_TOO_LARGE, ("no-allocation", "workspace"))):
        text = echo.echo_strerror(status)
        assert all(w in text for w in words), text
