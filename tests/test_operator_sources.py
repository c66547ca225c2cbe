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


def kernels(text):
    """(name, definition) of every kernel."""
    for part in re.split(r"\b__global__\b", text)[1:]:
        name = re.search(r"(\w+)\(\s*(?:const )?[\w<>]+ ?[*\w]", re.sub(
            r"__launch_bounds__\((?:[^()]|\([^()]*\))*\)", "", part)).group(1)
        yield name, part[:part.index("{")] + body(part, name)


def test_kernels_that_begin_early_do_not_read_through_the_read_only_path():
    """That path is for memory that nobody writes while the kernel lives; a
    chained kernel lives before the one ahead of it has done its writes."""
    found = set()
    for name in ("embedding.cu", "grad_norm.cu", "layer_norm.cu", "token_sort.cuh"):
        for kernel, text in kernels(source(name)):
            if "dependents_wait" in text or "dependents_launch" in text:
                found.add(kernel)
                assert "__restrict__" not in text and "__ldg" not in text, kernel
    assert {"lookup_kernel", "sum_kernel", "scale_kernel", "norm_grad_kernel",
            "cluster_sort_kernel"} <= found


def test_what_scaling_reads_before_its_wait_comes_from_l2():
    text = source("grad_norm.cu")
    assert re.search(r"scale_any<kThreads, true>\(.*?, factor\)", body(text, "scale_kernel"))
    tile = body(text, "scale_tile")
    before = tile[:tile.index("factor()")]
    # a tile's reads that stand before the factor is asked for
    loads = re.findall(r"[^;{}]*\bload_pack\w*<[^;]*;", before)
    assert loads and all("EARLY ? load_pack_l2" in x for x in loads)
    assert "__ldcg" in body(source("op_common.cuh"), "load_pack_l2")
