"""Orderings between blocks and kernels that no output can be made to depend on:
what the sources of the training-step operators have to say about them."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "ring_allreduce_compressed_gb300", "csrc")


def source(name):
    """The file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def body(text, name):
    """The braces of the function `name` and what is between them."""
    start = text.index("{", re.search(rf"\b{name}\(", text).end())
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError(f"{name}: no end")


def test_blocks_of_a_cluster_have_started_before_their_memory_is_written():
    sort = body(source("token_sort.cuh"), "cluster_sort_kernel")
    remote = sort.index("st.shared::cluster")
    waits = [sort.find(w) for w in ("cluster_wait()", "cluster_sync()")]
    assert any(0 <= w < remote for w in waits)
    # a wait of its own needs an arrival of its own, by every thread, before it
    if 0 <= waits[0] < remote:
        arrives = sort.index("cluster_started()")
        assert arrives < waits[0]
        assert sort[:arrives].count("{") == 1 and "return" not in sort[:waits[0]]
