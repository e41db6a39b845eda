"""Device code of the products of quantized rows: what the compiler does not check for MFMAs and
conversions written as assembly, checked on the assembly of every instance of the four-wave tiles."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tensor_sharded_linear_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not installed")


@pytest.fixture(scope="module")
def bodies(tmp_path_factory):
    """{kernel: instructions} of gemm_fp8_tiled.hip."""
    from tensor_sharded_linear_amd.build import FLAGS
    flags = [f for f in FLAGS if f not in ("-shared", "-fPIC")]
    out = tmp_path_factory.mktemp("asm") / "gemm_fp8_tiled.s"
    res = subprocess.run([HIPCC, *flags, "--cuda-device-only", "-S", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                          os.path.join(CSRC, "gemm_fp8_tiled.hip"), "-o", str(out)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    text = out.read_text()
    found = {}
    for m in re.finditer(r"^(\S*gemm_fp8_nt_kernel\S*):", text, re.M):
        body = text[m.end():text.index("s_endpgm", m.end())].splitlines()
        found[m.group(1)] = [ln.strip() for ln in body if re.match(r"\s+[a-z]", ln) and not ln.strip().startswith(".")]
    return found


def registers(operand, kind):
    """The numbers of the registers of a kind ('v' or 'a') that an operand names."""
    m = re.fullmatch(kind + r"\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.fullmatch(kind + r"(\d+)", operand)
    return {int(m.group(1))} if m else set()


def operands(line):
    return [o.strip() for o in line.split(None, 1)[1].split(" op_sel")[0].split(",")] if " " in line else []


def test_every_instance_is_there(bodies):
    """8-bit: 4 shapes for each of the plain epilogues and 3 for SwiGLU; exact: 3 and 2; with bias or not."""
    assert len(bodies) == 2 * (4 + 4 + 3) + 2 * (3 + 3 + 2), sorted(bodies)


def test_no_accumulator_is_moved_among_the_mfmas(bodies):
    """Between the first MFMA and the wait after the last, no other instruction touches an accumulator."""
    for name, body in bodies.items():
        mfma = [i for i, ln in enumerate(body) if ln.startswith("v_mfma")]
        acc = set().union(*(registers(operands(body[i])[0], "a") for i in mfma))
        end = next(i for i, ln in enumerate(body) if ln.startswith("s_nop 7") and i > mfma[-1])
        for ln in body[mfma[0]:end]:
            if not ln.startswith("v_mfma"):
                used = set().union(*(registers(o, "a") for o in operands(ln))) if " " in ln else set()
                assert not used & acc, (name, ln)


def test_no_mfma_reads_what_the_two_instructions_before_it_wrote(bodies):
    """An MFMA needs two wait states after a VALU instruction that writes one of its operands."""
    for name, body in bodies.items():
        for i, ln in enumerate(body):
            if not ln.startswith("v_mfma"):
                continue
            reads = set().union(*(registers(o, "v") for o in operands(ln)[1:]))
            for prev in body[max(0, i - 2):i]:
                if prev.startswith("v_") and not prev.startswith("v_mfma"):
                    assert not registers(operands(prev)[0], "v") & reads, (name, prev, ln)
