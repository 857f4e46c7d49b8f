"""Rules of the kernels that no run shows, checked in their source (no GPU)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "pretraining_optimizer_b200", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _body(source, at):
    """The text of the braces that open first behind `at`."""
    begin = source.index("{", source.index(at))
    depth = 0
    for i in range(begin, len(source)):
        depth += {"{": 1, "}": -1}.get(source[i], 0)
        if depth == 0:
            return source[begin:i + 1]
    raise AssertionError(at)


def test_pair_kernels_commit_for_the_pair_only():
    """All tcgen05 instructions of a kernel name the same cta_group: a commit for one CTA does not have to track
    the pair's MMAs, which must be done before their TMEM is freed."""
    body = _body(_source("muonh_ns_gemm.cu"), " ns_gemm_pair_kernel(const")
    assert "umma_commit_pair(drain)" in body
    assert not re.search(r"\b(umma_commit|umma_f16|tmem_alloc|tmem_dealloc)\(", body)
    body = _body(_source("muonh_block_gemm.cu"), " block_matmul_kernel(const")
    assert "commit(drain)" in body
    # the one-CTA forms stand only where PAIR is false
    for form in ("umma_commit(", "umma_mxf8(", "copy_scales(", "tmem_alloc(", "tmem_dealloc("):
        for m in re.finditer(r"\b" + re.escape(form), body):
            assert re.search(r"else\s*$", body[:m.start()]), (form, body[m.start() - 80:m.start() + 40])


def test_both_ctas_of_a_pair_wait_for_the_last_commit():
    """It arrives in both, and neither may leave before it has."""
    for name, kernel in (("muonh_ns_gemm.cu", " ns_gemm_pair_kernel(const"), ("muonh_block_gemm.cu", " block_matmul_kernel(const")):
        body = _body(_source(name), kernel)
        wait = body.index("mbar_try_wait(drain")
        # the wait's braces hold no condition on the rank: walk outwards from it
        depth, opened = 0, []
        for i in range(wait, -1, -1):
            if body[i] == "}":
                depth += 1
            elif body[i] == "{":
                if depth == 0:
                    opened.append(body[max(0, i - 80):i].split(";")[-1].split("}")[-1])
                else:
                    depth -= 1
        assert not any("rank" in o for o in opened), (name, opened)
