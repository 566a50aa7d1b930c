"""Properties of the kernels' sources that no run on one GPU shows."""
import glob
import os
import re

import matrix_orthogonalizing_optimizer_shape_gb300 as d3

CSRC = os.path.join(os.path.dirname(d3.__file__), "csrc")


def sources():
    files = [f for pat in ("*.cu", "*.cuh", "*.h") for f in sorted(glob.glob(os.path.join(CSRC, pat)))]
    assert files
    return {os.path.basename(f): open(f).read() for f in files}


def test_only_commits_reach_several_ctas():
    """The library is loaded by one process a GPU: each CTA loads its own operands,
    and only the tensor cores' commits signal several CTAs of a cluster."""
    commits = 0
    for name, text in sources().items():
        for stmt in re.findall(r"\basm\b[^;]*?\(.*?\)\s*;", text, flags=re.S):
            if "multicast" in stmt:
                assert "tcgen05.commit" in stmt, f"{name}: {stmt[:200]}"
                commits += 1
    assert commits > 0


def test_cached_values_are_atomic():
    """Host threads may make their first calls together: what a function keeps in a
    static is an atomic, a once_flag, constant, or written under one of them."""
    guarded = re.compile(r"std::(atomic|once_flag|mutex)|const(expr)? |\bPFN_|\(")
    for name, text in sources().items():
        for m in re.finditer(r"^ +static (?!_)[^;{]*", text, flags=re.M):
            decl = m.group(0)
            locked = "std::mutex" in text[max(0, m.start() - 200):m.start()]  # declared right after its lock
            assert locked or guarded.search(decl), f"{name}: {decl.strip()}"


def test_every_wrapper_is_used():
    """tc_ops.cuh holds the instructions that the kernels issue, and no others."""
    texts = sources()
    names = re.findall(r"__forceinline__ \w+ (\w+)\(|constexpr \w+ (\w+)\(", texts["tc_ops.cuh"])
    assert len(names) > 20
    users = [texts["tc_ops.cuh"]] + [t for n, t in texts.items() if '"tc_ops.cuh"' in t]
    for name in (a or b for a, b in names):
        uses = sum(len(re.findall(rf"\b{name}\b", t)) for t in users)
        assert uses > 1, f"{name} is not used"
