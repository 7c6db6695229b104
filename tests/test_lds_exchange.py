"""How the 4-bit product's waves hand scales and rows' values to one another through LDS, read from the compiler's intermediate
form before optimisation: written in one width and read in another, the bytes go through types that may alias, and a fence of the
wave stands on either side of the writing, so that no optimisation may move a read above the write it depends on."""
import os
import re
import subprocess

import pytest

from moe_expert_layer_amd import build


@pytest.fixture(scope="module")
def functions(tmp_path_factory):
    """name -> lines, and the name of the type that a tbaa tag stands for"""
    out = tmp_path_factory.mktemp("ir") / "w4.ll"
    cmd = [build.hipcc(), *build.HIP_FLAGS, "-I", build.INCLUDE, "-I", build.CSRC, "-S", "-emit-llvm", "--offload-device-only",
           "-Xclang", "-disable-llvm-passes", os.path.join(build.CSRC, "w4_gemm.hip"), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    text = out.read_text()
    meta = dict(re.findall(r"^!(\d+) = (.*)$", text, re.M))

    def accessed(tag):
        node = meta[re.match(r"!\{!\d+, !(\d+)", meta[tag]).group(1)]
        return re.match(r'!\{!"([^"]*)"', node).group(1)

    fns = {m.group(1): m.group(0).split("\n") for m in re.finditer(r"^define [^\n]*@(\S+?)\(.*?^\}", text, re.M | re.S)}
    return fns, accessed


def accesses(lines, kind):
    """(line, tbaa tag) of the loads or stores that do not go to the function's own variables"""
    local = set()
    for l in lines:
        m = re.match(r"\s*(%\S+) = (?:alloca|addrspacecast ptr addrspace\(5\))", l)
        if m:
            local.add(m.group(1))
        m = re.match(r"\s*store .*, ptr (%\S+?),", l) if kind == "store" else re.match(r"\s*%\S+ = load [^,]*, ptr (%\S+?),", l)
        if m and m.group(1) not in local:
            yield l, re.search(r"!tbaa !(\d+)", l)


@pytest.mark.parametrize("pattern,kind", [(r"Items.*load_lds", "load"), (r"ScaleLds.*3putE", "store"), (r"ScaleLds.*4copyE", "store")])
def test_bytes_in_lds_go_through_types_that_may_alias(functions, pattern, kind):
    fns, accessed = functions
    seen = 0
    for name, lines in fns.items():
        if re.search(pattern, name):
            for line, tag in accesses(lines, kind):
                seen += 1
                assert tag is None or accessed(tag.group(1)) == "omnipotent char", (name, line)
    assert seen


def calls(lines, what):
    return [i for i, l in enumerate(lines) if " call " in l and what in l]


@pytest.mark.parametrize("pattern,written", [(r"ScaleLds.*3putE", "store i32"), (r"ScaleLds.*4copyE", "store i"),
                                             (r"few_rows.*ENKUl.*RZ?N.*Block.*", "turn")])
def test_a_fence_on_either_side_of_the_writing(functions, pattern, written):
    fns, _ = functions
    seen = 0
    for name, lines in fns.items():
        if not re.search(pattern, name):
            continue
        if written == "turn":
            at = calls(lines, "turnI")
        else:
            at = [lines.index(l) for l, _ in accesses(lines, "store") if written in l]
        if not at:
            continue
        seen += 1
        fences = calls(lines, "wave_fence")
        assert fences and fences[0] < min(at) and fences[-1] > max(at), name
    assert seen
    fence = [l for n, l in fns.items() if "wave_fence" in n]
    assert len(fence) == 1
    body = "\n".join(fence[0])
    assert re.search(r'fence syncscope\("wavefront"\) release.*wave\.barrier.*fence syncscope\("wavefront"\) acquire', body, re.S)
