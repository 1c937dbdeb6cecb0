"""Orders inside kernels that no run can be relied on to show, checked on the text."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_fp4_csa2_gb300", "csrc")


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_row_scales_after_the_block_before():
    """The sparse readout's workers write a block's scales only behind the wait for the
    products of the block before: until then slower warps read that block's."""
    body = text("attention.cu")
    loop = body[body.index("for (; cur_item < items; ++g)"):]
    loop = loop[:loop.index("mbar_arrive(&S.cols_full[p])")]
    assert loop.count("put_row_info") == 1
    assert loop.index("&S.cols_free[p]") < loop.index("put_row_info")
