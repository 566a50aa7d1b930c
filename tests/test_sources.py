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


def test_flags_of_waits_that_ran_out_are_read_between_barriers():
    """A thread that leaves a loop of block barriers alone hangs its block: the recurrence's
    flags are read where a barrier stands between every write and every read.  `late` is
    written by the kernels before a step (the call of enter) and read behind enter's first
    barrier; `stop` is written between enter's barriers and read behind the second."""
    text = re.sub(r"//[^\n]*", "", sources()["recurrence.cu"])
    start = text.index("enter(Shared<VEC>& sh")
    end = text.index("\n}\n", start)
    enter, others = text[start:end], text[:start] + text[end:]
    assert not re.search(r"sh\.(late|stop)\b(?! = )", others)  # written, never read
    assert not re.search(r"sh\.stop = 1", others) and len(re.findall(r"sh\.late = 1", others)) == 2
    before, between, behind = enter.split("__syncthreads();")
    assert not re.search(r"sh\.(late|stop)\b", before)
    assert re.findall(r"sh\.(?:late|stop)\b(?: = 1)?", between) == ["sh.late", "sh.stop = 1"]
    assert re.findall(r"sh\.(?:late|stop)\b(?: = 1)?", behind) == ["sh.stop"]
    for call in re.finditer(r"= enter<VEC>\(", others):  # each step's writes of `late` stand before its call
        assert "sh.late = 1" in others[others.rindex("in_flight.wait(step,", 0, call.start()):call.start()]


def test_large_clusters_are_asked_for():
    """A kernel that may run in clusters past the 8 blocks that every device holds asks
    whether this one (or the part of it that the process has) holds them."""
    found = 0
    for name, text in sources().items():
        for m in re.finditer(r"cudaFuncAttributeNonPortableClusterSizeAllowed", text):
            found += 1
            assert "cudaOccupancyMaxActiveClusters" in text[m.start():m.start() + 600], name
    assert found == 2
