"""Order of a gradient's overlapping launches, read from the sources (no GPU
needed; a missing wait may go unnoticed for as long as it likes on one).

A launch may start before the one ahead of it has ended, and only its own
griddepcontrol.wait makes writes of the launch directly ahead visible.  So a
kernel that reads what another launch of the call wrote waits before its first
read, a kernel that does not wait first reads the call's inputs alone, and the
last block of every early launch waits before it ends."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "exact_second_order_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernel(name, function):
    text = source(name)
    start = re.search(r"\b" + function + r"\s*\([^;{]*\)\s*\{", text)
    return text[start.end():text.index("\n}\n", start.end())]


@pytest.mark.parametrize("name,function", [("tc_attn_dkv.cu", "tc_dkv_kernel"),
                                           ("attn_simt.cu", "attn_dkv_kernel")])
def test_row_state_is_waited_for_before_it_is_read(name, function):
    body = kernel(name, function)
    reads = [m.start() for m in re.finditer(r"__ldcg\(|bulk_load\(", body)]
    assert reads and 0 <= body.find("wait_ahead();") < min(reads)


@pytest.mark.parametrize("name,function", [("tc_attn_dq.cu", "tc_dq_kernel"),
                                           ("attn_simt.cu", "attn_dq_kernel")])
def test_a_launch_that_does_not_wait_first_reads_inputs_alone(name, function):
    body = kernel(name, function)
    assert "workspace" not in body and "grad_rows" not in body
    last = body.rstrip()
    assert last.endswith("wait_ahead();") and body.count("wait_ahead") == 1


@pytest.mark.parametrize("name,function,read", [("attn_rows.cu", "join_kernel", r"p\.ml\["),
                                                ("qk_norm.cu", "norm_dw_kernel", r"part\[")])
def test_joins_wait_first(name, function, read):
    body = kernel(name, function)
    assert 0 <= body.find("wait_ahead();") < re.search(read, body).start()


def test_dkv_is_launched_between_the_row_state_and_dq():
    api, simt = source("flashbob_api.cu"), source("attn_simt.cu")
    assert api.index("attn_grad_rows(a)") < api.index("tc_attn_dkv(a)") < api.index("tc_attn_dq(a)")
    assert simt.index("launch(attn_dkv_kernel") < simt.index("launch(attn_dq_kernel")
