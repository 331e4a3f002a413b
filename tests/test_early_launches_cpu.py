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


def _starts(body):
    """A body's first statement behind its declarations of constants and shared memory."""
    return re.match(r"\s*(?:(?:using|constexpr|extern|__shared__)\b[^;]*;\s*)*([^;]*;)", body).group(1)


def test_kernels_of_the_layer_wait_before_anything_else():
    """act_kernel, launched as any other kernel, is the one that does not."""
    for name in ("checkpoint.cu", "norm_residual.cu"):
        code = _code(name)
        bodies = _bodies(code)
        assert len(bodies) == code.count("__global__")
        without = [k for k, b in bodies.items() if _starts(b) != "pdl_enter();"]
        assert without == (["act_kernel"] if name == "checkpoint.cu" else []), without
        assert set(re.findall(r"(\w+)<<<|::(\w+)<<<", code)) <= {("act_kernel", ""), ("", "act_kernel")}


def test_products_of_a_block_with_a_checkpoint_wait_in_all_three_roles():
    """The producer before its first load, the issuer before its first wait, the epilogue's warps behind their dry pass,
    which is their first, loads nothing and stores nothing."""
    bodies = _bodies(_code("gemm_tc.cu"))
    for name in ("gemm_kernel", "gemm_pair_kernel"):
        body = bodies[name]
        roles = re.split(r"(?:\}\s*else\s+)?if \(warp (?:==|>=) (\d)\) \{", body[body.index("const int num_tiles") :])
        producer, issuer, epilogue = (roles[roles.index(w) + 1] for w in "014")
        for part, first in ((producer, "tma_load"), (issuer, "mbar_wait_bounded")):
            assert part.count("pdl_enter();") == 1 and part.index("if constexpr (HELD) pdl_enter();") < part.index(first), name
            assert part.index("pdl_enter();") < part.index("for (int t = ")
        assert re.search(r"int it = HELD \? -1 : 0;\s*for \(int t = HELD \? \w+ - \w+ : \w+;", epilogue)
        assert "(dry ? no_row(p) :" in epilogue and epilogue.count("pdl_enter();") == 1
        assert epilogue.index("run_epilogue<") < epilogue.index("if (dry) pdl_enter();")
        assert "return" not in epilogue[: epilogue.index("run_epilogue<")]
    assert re.search(r"no_row\(const Params& p\) \{ return \(static_cast<int64_t>\(p\.M\) \+ 31\) / 32 \* 32; \}", _code("gemm_tc.cu"))
