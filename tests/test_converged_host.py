"""Warp-wide instructions stand behind a point where the warp is together.

TMEM loads and stores, the transposing shared-memory loads and cluster barriers
have .aligned forms: every lane of the warp has to execute the same one, or the
GPU may fault or hang.  After code that only some lanes run, nothing but a
warp-wide synchronisation says that the lanes are together again.  That cannot
be shown by running it, so the sources are read: between the last statement
that lanes may part on and such an instruction there has to be a meeting point,
also on the way from the end of a loop's body back to its start."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_mixer_gb300", "csrc")

ALIGNED = re.compile(r"\b(tmem_ld\w+|tmem_st\w+|ldsm4t|cluster_sync)\s*\(|bar\.sync")
MEET = re.compile(r"__syncwarp\(|__syncthreads\(|__all_sync\(|\bwarp_wait2?\(|\bcluster_sync\(")
CONDITIONAL = re.compile(r"\bif \(.*\) (ok =|cluster_sync)")
# What may part the lanes: tests of a lane's own values, and helpers that hold such tests.
PART = re.compile(r"\bif \([^;]*\b(lane|tid|t == 0|c\.y|inside|in_bounds|j >= len|row >= g\.M|rows)\b|"
                  r"\b(load_residual|prefetch_residual|store_run|load_rows|finish<\w+>|warp_arrive)\(")


def code(path):
    """The file's lines without comments."""
    with open(path) as f:
        return [line.split("//", 1)[0].rstrip() for line in f]


def blocks(lines):
    """For each line the innermost enclosing (first, last) lines of a braced block, and every block's parent."""
    stack, inner, span, parent = [], [], {}, {}
    for i, line in enumerate(lines):
        closed = len(line) - len(line.lstrip("} \t"))
        for ch in line[:closed].count("}") * "}":
            span[stack.pop()] = i
        inner.append(stack[-1] if stack else None)
        for ch in line[closed:]:
            if ch == "{":
                parent[i] = stack[-1] if stack else None
                stack.append(i)
            elif ch == "}":
                top = stack.pop()
                span[top] = i
    return inner, span, parent


def unsafe(lines):
    inner, span, parent = blocks(lines)
    bad = []

    def around(block):
        while block is not None:
            yield block
            block = parent[block]

    def parted(i, first):
        """Scanning back from line i to `first`: True if lanes parted last, False if they met last, None if neither.
        Meeting points that are passed on a condition do not count."""
        for n in range(i - 1, first, -1):
            if MEET.search(lines[n]) and not CONDITIONAL.search(lines[n]) and inner[n] in (first, *around(first)):
                return False
            if PART.search(lines[n]):
                return True
        return None

    for i, line in enumerate(lines):
        if not ALIGNED.search(line) or "__forceinline__" in line or "asm" in lines[i - 1]:
            continue
        at, block = i, inner[i]
        while block is not None and parent[block] is not None:
            p = parted(at, block)
            if p is None and re.search(r"\b(for|while) \(", lines[block]):
                p = parted(span[block], at)  # round the loop
            if p is not None:
                if p:
                    bad.append((i + 1, line.strip()))
                break
            at, block = block, parent[block]
    return bad


@pytest.mark.parametrize("name", ["linear_ex.cu", "linattn_chunked.cu", "gemm.cu"])
def test_aligned_instructions_follow_a_meeting_point(name):
    assert unsafe(code(os.path.join(CSRC, name))) == []


def test_the_reading_itself():
    good = ["namespace a {", "void k() {", "  for (int i = 0; i < n; ++i) {", "    __syncwarp();", "    tmem_ld32(t, v);",
            "    if (lane < rows) {", "      store();", "    }", "  }", "}", "}"]
    assert unsafe(good) == []
    assert [n for n, _ in unsafe([x for x in good if "__syncwarp" not in x])] == [4]
    assert [n for n, _ in unsafe([x.replace("__syncwarp();", "if (n) ok = warp_wait(b);") for x in good])] == [5]
    assert unsafe(["namespace a {", "void k() {", "  if (lane == 0) arrive();", "  cluster_sync();", "}", "}"]) == [(4, "cluster_sync();")]
