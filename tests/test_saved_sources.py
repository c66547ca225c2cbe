"""Orderings and limits that no output shows: what the sources of the operators with
activations in 8 bits have to say about them."""
import re

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
            "operand_kernel", "rows_kernel", "codes_kernel", "gemm_kernel", "finish_kernel",
            "join_kernel"} <= found
    for name in ("saved.cuh", "ragged.cuh", "tc.cuh"):
        assert "__ldg" not in source(name) and "__restrict__" not in source(name)


def test_waits_of_the_large_kernel_have_a_limit():
    text = source("gated_gemm.cu")
    # every wait on a barrier in memory is the one with the limit
    assert "try_wait" not in text and text.count("wait_limited(") >= 5
    wait = body(source("tc.cuh"), "wait_limited")
    assert "kWaitLimitNs" in wait and "*stop" in wait
    # and the loops that wait go on only while it says so
    kernel = body(text, "gemm_kernel")
    for loop in re.findall(r"for \(int t = pair;([^;]*);", kernel):
        assert "ok &&" in loop


def test_a_kernel_that_gave_up_is_reported_by_the_next_call():
    text = source("gated_ff.cu")
    status = body(text, "stalled_status")
    assert "RRA_ERR_TIMEOUT" in status
    for call in ("ff", "ff_grad"):
        assert "stalled_status()" in body(text, rf"rra_status {call}")
