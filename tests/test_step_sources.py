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


def bodies(source):
    """Name -> body of the device functions of a file (closing brace in the first column)."""
    return {m[1]: m[2] for m in re.finditer(r"__device__[^;{]*?(\w+)\([^{;]*\) \{\n(.*?)\n\}\n", source, re.S)}


def test_every_issuer_of_products_waits_for_its_own():
    """A commit tells of the products of the thread that makes it: each role that issues
    some ends with one of its own, which the teardown follows."""
    for name in ("window_attn.cu", "gather_attn.cu"):
        found = []
        for fn, body in bodies(text(name)).items():
            if "mma_f16" not in body:
                continue
            last = body.rindex("mma_")
            after = re.findall(r"drain\(&S\.done\[(\d)\]\)", body[last:])
            assert len(after) == 1, f"{name}: {fn} ends without a wait for its products"
            found += after
        assert sorted(found) == ["0", "1"], name
        drain = bodies(text(name))["drain"]
        assert drain.index("mma_commit(done)") < drain.index("mbar_wait(done, 0)")
