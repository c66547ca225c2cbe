"""Orderings and limits that no output shows: what the sources of the operators with
activations in 8 bits have to say about them."""
from test_operator_sources import body, kernels, source

FILES = ("layer_norm_saved.cu", "gated_ff.cu", "gated_rows.cu", "gated_gemm.cu", "row_group.cuh")


def test_kernels_that_begin_early_do_not_read_through_the_read_only_path():
    found = set()
    for name in FILES:
        for kernel, text in kernels(source(name)):
            if "dependents_wait" in text or "dependents_launch" in text:
                found.add(kernel)
                assert "__restrict__" not in text and "__ldg" not in text, kernel
                # and wait before they let the next one in
                assert text.index("dependents_wait") < text.index("dependents_launch"), kernel
    assert {"save_kernel", "restore_kernel", "saved_grad_kernel", "act_grad_kernel",
            "operand_kernel", "rows_kernel", "codes_kernel", "finish_kernel",
            "join_kernel"} <= found
    for name in ("saved.cuh", "ragged.cuh"):
        assert "__ldg" not in source(name) and "__restrict__" not in source(name)


def test_the_large_kernel_waits_for_nothing_but_its_own_block():
    text = source("gated_gemm.cu")
    for word in ("mbarrier", "cluster", "tcgen05", "while (", "for (;;", "volatile unsigned",
                 "cooperative"):
        assert word not in text, word
    # begun when what is ahead of it has ended, and keeps what is behind it back
    kernel = body(text, "gemm_kernel")
    assert "dependents_" not in kernel and "fn<<<" in text
    # what is outside of an operand is not read
    copy = body(text, "copy16")
    assert "row < x.rows" in copy and "x.cols - col" in copy
