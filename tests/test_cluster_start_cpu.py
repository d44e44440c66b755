"""Stores into another CTA's shared memory need a cluster barrier before them:
only behind one is it known that the other CTA has begun.  Read from the
sources, for such a store that comes too early need not show in any result."""
import os
import re

import pytest

from hybrid_linear_attention_gdn_gb300 import _build

REMOTE = re.compile(r"\bmap_shared_rank\b|\bmapa\b|shared::cluster\.(?:u32|u64|b32|b64|f32)")
BARRIER = re.compile(r"\bcluster\.sync\(\)|\bcluster_wait_acquire\(\)|\bcluster_sync\(\)")


def kernels(text):
    """(name, body without comments) of every __global__ function."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\((?:[^()]|\([^()]*\))*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[m.end():i - 1]


def unconditional(body):
    """The statements of a body that are in no block, branch or loop."""
    out, depth = [], 0
    for c in body:
        depth -= c == "}"
        out.append(c if depth == 0 and c not in "{}" else ";" if c == "}" and depth == 0 else "")
        depth += c == "{"
    return [s for s in "".join(out).split(";") if not re.match(r"\s*(if|for|while|else)\b", s)]


def unordered(text):
    """Kernels that reach into another CTA's shared memory before an
    unconditional barrier of the cluster."""
    bad = []
    for name, body in kernels(text):
        m = REMOTE.search(body)
        if m and not any(BARRIER.search(s) for s in unconditional(body[:m.start()])):
            bad.append(name)
    return bad


def sources():
    return sorted(s for s in os.listdir(_build.CSRC) if s.endswith((".cu", ".cuh")))


@pytest.mark.parametrize("name", sources())
def test_peers_have_begun(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        assert unordered(f.read()) == []


def test_the_reader_itself():
    head = "template <bool R>\n__global__ void __launch_bounds__(64) k(const A a) {\n  int v = 0;\n"
    store = "  *cluster.map_shared_rank(&c[0], 1) = v;\n}\n"
    assert unordered(head + store) == ["k"]
    assert unordered(head + "  if (R) {\n    cluster.sync();\n  }\n" + store) == ["k"]
    assert unordered(head + "  if (R) cluster.sync();\n" + store) == ["k"]
    assert unordered(head + "  // cluster.sync();\n" + store) == ["k"]
    assert unordered(head + "  if (R) {\n    v = 1;\n  }\n  cluster.sync();\n" + store) == []
