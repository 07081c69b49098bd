"""The order in which the parts of a cut pair of query tiles reach the CTA that joins them (fa_chunk.cu), from the
kernel's source and the rules of the PTX memory model (no GPU).

Two CTAs leave a part each; the one that counts last reads both.  From the source come, in their order, the
synchronising steps of a softmax warp between its last store of a part and its first load of the join.  Each thread
runs them (those of warp 0 or of lane 0 only there), and every synchronisation is an edge between threads:
  __syncwarp                        all lanes of a warp, both ways;
  mbar_arrive -> wait on it         release to acquire, within the CTA;
  atomicAdd of a CTA -> the later   only as fence; atomic -> atomic; fence, the fences in the program order of the
  atomicAdd of another              threads that do the atomics: a relaxed atomic alone orders nothing.
A store is visible to a load iff a path of program order and edges leads from one to the other."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WARPS, LANES = 3, 2  # as many as tell the cases apart: warp 0 and others, lane 0 and others

STEPS = [("fence", r"__threadfence\(\);"), ("syncwarp", r"__syncwarp\(\);"),
         ("arrive part", r"if \(lane == 0\) mbar_arrive\(&bar_part\);"), ("wait part", r"wait_warp\(&bar_part,"),
         ("atomic", r"atomicAdd\(&p\.counters"), ("arrive ticket", r"mbar_arrive\(&bar_ticket\);"),
         ("wait ticket", r"wait_warp\(&bar_ticket,"), ("load", r"join_parts<"),
         ("warp 0 {", r"if \(warp == 0\) \{"), ("lane 0 {", r"if \(lane == 0\) \{"), ("}", r"\n *\}")]


def steps_of_source():
    src = open(os.path.join(ROOT, "tiled_attention_08_gb300", "csrc", "fa_chunk.cu")).read()
    begin = src.index("const int n_parts = unit_cta(")
    text = re.sub(r"//[^\n]*", "", src[begin:src.index("join_parts<D, BF16>(p, sg.b", begin) + 20])
    found = sorted((m.start(), name) for name, pat in STEPS for m in re.finditer(pat, text))
    return [name for _, name in found]


def thread_program(steps, warp, lane):
    """(step, index) of those that this thread executes."""
    out, scope = [], []
    for i, s in enumerate(steps):
        if s.endswith("{"):
            scope.append(s)
        elif s == "}":
            if scope:
                scope.pop()
        elif not (("warp 0 {" in scope and warp != 0) or ("lane 0 {" in scope and lane != 0)):
            if not (s == "arrive part" and lane != 0):
                out.append((s, i))
    return out


def visible(steps):
    """Whether every thread of CTA 1 (the last to count) sees the parts of every thread of CTA 0."""
    nodes, edges = {}, {}

    def edge(a, b):
        edges.setdefault(a, set()).add(b)

    threads = [(c, w, l) for c in (0, 1) for w in range(WARPS) for l in range(LANES)]
    for t in threads:
        prog = [("store", -1)] + thread_program(steps, t[1], t[2])
        nodes[t] = prog
        for a, b in zip(prog, prog[1:]):
            edge((t, a), (t, b))
    for t in threads:
        for u in threads:
            for a in nodes[t]:
                for b in nodes[u]:
                    same_warp, same_cta = t[:2] == u[:2], t[0] == u[0]
                    if a == b and a[0] == "syncwarp" and same_warp:
                        # (what is in front of it there is in front of what is behind it here)
                        k, n = nodes[t].index(a), nodes[u].index(b)
                        if k > 0 and n + 1 < len(nodes[u]):
                            edge((t, nodes[t][k - 1]), (u, nodes[u][n + 1]))
                    if same_cta and (a[0], b[0]) in (("arrive part", "wait part"), ("arrive ticket", "wait ticket")):
                        edge((t, a), (u, b))
    for t in threads:
        for u in threads:
            at, au = ([x for x in nodes[y] if x[0] == "atomic"] for y in (t, u))
            if t[0] == 0 and u[0] == 1 and at and au:
                release = [x for x in nodes[t] if x[0] == "fence" and x[1] < at[0][1]]
                acquire = [x for x in nodes[u] if x[0] == "fence" and x[1] > au[0][1]]
                if release and acquire:
                    edge((t, release[-1]), (u, acquire[0]))
    for t in threads:
        if t[0] != 0:
            continue
        seen, todo = set(), [(t, ("store", -1))]
        while todo:
            for x in edges.get(todo.pop(), ()):
                if x not in seen:
                    seen.add(x)
                    todo.append(x)
        for u in threads:
            load = [x for x in nodes[u] if x[0] == "load"]
            if u[0] == 1 and not (load and (u, load[0]) in seen):
                return False
    return True


def test_the_source_is_read_whole():
    steps = steps_of_source()
    for s in ("arrive part", "wait part", "atomic", "arrive ticket", "wait ticket", "load"):
        assert steps.count(s) == 1, (s, steps)
    assert steps[-1] == "load"


def test_parts_are_visible_to_the_cta_that_joins_them():
    assert visible(steps_of_source()), steps_of_source()


RIGHT = ["syncwarp", "arrive part", "warp 0 {", "wait part", "lane 0 {", "fence", "atomic", "fence", "arrive ticket", "}",
         "syncwarp", "}", "wait ticket", "load"]


def without(i):
    return RIGHT[:i] + RIGHT[i + 1:]


def test_the_rules_tell_right_from_wrong():
    assert visible(RIGHT)
    # Fences in the threads that store and load, not in those that count.
    assert not visible(["fence", *without(5)])
    assert not visible([*without(7)[:-1], "fence", "load"])


@pytest.mark.parametrize("gone", [0, 1, 3, 5, 7, 8, 12])
def test_every_step_is_needed(gone):
    assert not visible(without(gone)), RIGHT[gone]
