"""Rules that the block operators' kernels keep and whose breach no run shows:
a wrong order that only a slow or preempted block would meet, or an access that
is wrong by the programming model and right by luck.  Read from the sources."""
import re
from pathlib import Path

CSRC = Path(__file__).resolve().parents[1] / "bit_error_compensated_gb300" / "csrc"


def source(name):
    """The file without its comments."""
    text = (CSRC / name).read_text()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def body_after(text, opening):
    """The braces' contents that follow the first match of `opening`."""
    start = re.search(opening, text)
    assert start, opening
    at = text.index("{", start.start())
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i]
    raise AssertionError("unbalanced braces")


def test_a_block_that_gave_up_stays_so():
    """The flag of a block whose wait gave up is cleared only where the block
    begins: a warp that cleared it later would hide it from the others, and one
    that set it again would end the waits of those that clean up."""
    kernel = body_after(source("int8_pair.cu"), r"product_pair_kernel\(")
    writes = re.findall(r"\bgive_up\s*=[^=]\s*[^;]*;", kernel)
    assert writes == ["give_up = 0;"]
    assert kernel.index("give_up = 0;") < kernel.index("mbar_init(")


def test_issuing_warps_wait_for_what_they_issued():
    """Each of the three issuing warps ends with bounded waits that look at no
    flag, and makes them however its loop ended: another warp may give up after
    this one has issued its last."""
    kernel = body_after(source("int8_pair.cu"), r"product_pair_kernel\(")
    issuing = body_after(kernel, r"if \(warp >= kIssuer\)")
    drains = {"last": r"if \(one\)\s*", "landed": r"for \([^)]*kStages && issued > 0[^)]*\)\s*",
              "codes_full": r"for \([^)]*kGroups && g > 0[^)]*\)\s*"}
    for barrier, opening in drains.items():
        waits = [b for b in re.findall(opening + r"\{([^{}]*)\}", issuing) if "mbar_wait_bounded(" + barrier in b]
        assert len(waits) == 1, barrier
        assert "give_up" not in waits[0] and "wait_on" not in waits[0]
    assert "!ok &&" not in issuing


def test_warps_are_together_at_aligned_instructions():
    """A cluster's barrier, a load from tensor memory and a warp's matrix
    instruction ask that all lanes of a warp execute them together, and all
    three stand behind branches that part them.  So the barrier exists once,
    behind a __syncwarp, the load's function begins with one, and one stands
    between the loads of codes and the products of them."""
    files = ["ops_common.h", "norm_common.h", "norm_fwd.cu", "norm_bwd.cu", "int8_common.h", "int8_load.h",
             "int8_few.cu", "int8_quantize.cu", "int8_pair.cu"]
    assert sum(source(f).count("barrier.cluster.arrive") for f in files) == 1
    for name, opening, instruction in (("ops_common.h", r"void cluster_barrier\(\)", "barrier.cluster.arrive"),
                                       ("int8_pair.cu", r"void tmem_load16\(", "tcgen05.ld")):
        body = body_after(source(name), opening)
        assert 0 <= body.find("__syncwarp();") < body.index(instruction)
    assert source("int8_pair.cu").count("tcgen05.ld") == 1
    few = body_after(source("int8_few.cu"), r"product_few_kernel\(")
    loads, sync, products = (few.rindex("load(tokens"), few.rindex("__syncwarp();"), few.index("mma(sum"))
    assert loads < sync < products


def test_no_read_only_loads_of_what_the_kernel_before_writes():
    """Blocks of these kernels are in place while the kernel before still runs
    (programmatic launches), so its results are not read-only data for them:
    no __ldg, no ld.global.nc.  Loads that the compiler may move (not volatile)
    start from pointers that were pinned behind the wait; the channels' codes,
    which the kernel before does not write, may be read ahead of it."""
    for path in sorted(CSRC.glob("int8_*")) + sorted(CSRC.glob("norm_*")) + [CSRC / "ops_common.h"]:
        text = source(path.name)
        assert "__ldg" not in text and "global.nc" not in text, path.name
        for kernel in re.finditer(r"__global__", text):
            body = body_after(text[kernel.start():], r"__global__")
            assert "pdl_wait();" in body, path.name
    for name, pointers in (("norm_bwd.cu", ["stats"]), ("int8_few.cu", ["w[i]", "a[i]"])):
        text = source(name)
        for p in pointers:
            assert text.index("pdl_wait();") < text.index(p + " = pinned("), p
    early = body_after(source("int8_few.cu"), r"product_few_kernel\(")
    assert re.findall(r"\bload\([^)]*\);", early[:early.index("pdl_wait();")]) == ["load(codes, w, warp);"]
    assert source("int8_quantize.cu").count("load_codes<") == source("int8_quantize.cu").count(">(pinned(") == 2


def test_a_report_that_was_not_read_is_not_cleared():
    """A product on another stream may set its word between this call's read
    and its clearing: only words that were read as set are cleared."""
    body = body_after(source("int8_api.cu"), r"int echo_matmul_status\(")
    read = body.index("cudaStreamSynchronize")
    for i, t in enumerate(("float", "__nv_bfloat16", "__half")):
        clear = re.search(rf"if \(word\[{i}\]\) ECHO_OPS_CUDA\(clear_gave_up<{t}>\(s\)\);", body)
        assert clear and clear.start() > read
    assert body.count("clear_gave_up") == 3 and "cudaMemsetAsync" not in body
    assert "cudaMemsetAsync" not in body_after(source("int8_pair.cu"), r"read_gave_up<")
