"""Launches that may start beside their predecessor, read in the source: which kernels wait, and where."""
import os
import re

from sp_partitioned_transformer_gb300 import build


def _code(name):
    with open(os.path.join(build.CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//.*|/\*(?s:.*?)\*/", "", f.read())


def _bodies(code):
    """name -> body of every kernel."""
    found, code = {}, re.sub(r"__launch_bounds__\([^()]*\)", "", code)
    for m in re.finditer(r"__global__\s+void\s+(\w+)\s*\([^;{]*\)\s*\{", code):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(code[i], 0)
            i += 1
        found[m.group(1)] = code[m.end() : i]
    return found


def test_products_of_a_block_without_a_checkpoint_have_none_of_its_code():
    """They neither start early nor run dry, and nothing of either is asked for at run time."""
    code = _code("gemm_tc.cu")
    assert not re.search(r"\bp\.held\b", code)
    early = code.index("cudaLaunchAttributeProgrammaticStreamSerialization")
    assert code[:early].rstrip().endswith("{\n    attr[cfg.numAttrs].id =") and "if (HELD) {" in code[early - 60 : early]
    for name in ("gemm_kernel", "gemm_pair_kernel"):
        body = _bodies(code)[name]
        assert body.count("pdl_enter();") == body.count("if constexpr (HELD) pdl_enter();") + body.count("if (dry) pdl_enter();")
        assert "const bool dry = HELD && it < 0;" in body
