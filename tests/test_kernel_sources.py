"""Rules of the kernels' sources that no run can show to be broken: what they order holds on the GPU either way, until a
compiler or a chip makes use of its freedom (no GPU needed)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_mixture_experts_rms_b200", "csrc")


def source(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(src, start):
    """The brace block that begins after `start`."""
    i = src.index("{", src.index(start))
    depth = 0
    for j in range(i, len(src)):
        depth += {"{": 1, "}": -1}.get(src[j], 0)
        if depth == 0:
            return src[i:j]
    raise AssertionError(start)


def test_sums_read_before_the_kernels_own_wait_come_from_l2():
    """linear_dbias_kernel<true> reads the column sums before its griddepcontrol.wait: only by loads that pass L1."""
    kernel = body(source("linear.cu"), "linear_dbias_kernel(")
    assert "if (AFTER) griddep_wait()" in kernel and kernel.index("part") < kernel.rindex("griddep_wait")
    assert re.findall(r"\bpart\b", kernel) and re.findall(r"\bpart\b", kernel) == re.findall(r"(?<=__ldcg\()part\b", kernel)


def test_a_wait_made_by_one_lane_is_shared_with_a_barrier():
    """A shuffle orders no memory: a wait's result reaches the other lanes through warp_take, whose barrier does."""
    assert "__syncwarp()" in body(source("ptx.cuh"), "bool warp_take(")
    files = [f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))]
    assert len(files) > 10
    for f in files:
        src = source(f).replace(body(source(f), "bool warp_take("), "") if f == "ptx.cuh" else source(f)
        assert not re.search(r"__shfl_sync\(\w+,\s*(got|ok)\b", src), f
    for f in ("few.cu", "linear_pair.cu"):
        assert source(f).count("warp_take(") == 2, f


def test_dependent_launches_read_without_the_read_only_path():
    """The linear kernels and the combine start while the kernel before may still be writing dy, z, the bias or y: no
    `ld.global.nc` (__ldg), which is for memory that nobody writes while the kernel runs."""
    for f in ("linear.cu", "linear.cuh", "linear_split.cu", "linear_pair.cu", "combine.cu"):
        src = source(f)
        assert "__ldg(" not in src and "global.nc" not in src and "__restrict__" not in src, f


def test_a_device_with_too_few_sms_is_told_so():
    """The few-token kernel needs an SM a token.  No GPU here has fewer than 64, so the check is read: it gives the
    documented status, before the launch."""
    call = body(source("api_few.cu"), "moe_status_t moe_layer_fwd_few(")
    check = call.index("if (sms < c.T) return MOE_ERR_UNSUPPORTED;")
    assert call.index("device_ready(&sms)) != MOE_OK) return st;\n  const moe_config_t& c") < check < call.index("launch_few(")
    with open(os.path.join(ROOT, "include", "moe.h")) as f:
        assert "with fewer than T SMs" in f.read()
