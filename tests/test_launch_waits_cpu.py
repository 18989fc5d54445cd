"""Every kernel that may be launched before the one in front of it is done waits for it before it looks at global memory, read from the
sources: what a load before the wait brings is not defined, and mostly right."""
import re

import pytest

from tests.test_gave_up_waits_cpu import block, source

FILES = ["zdmmv_attn.cuh", "zdmmv_attn_prompt.cuh", "zdmmv_attn_weights.cu", "zdmmv_kv.cu", "zdmmv_kv_keep.cu", "zdmmv_norm.cu"]


@pytest.mark.parametrize("name", FILES)
def test_the_wait_comes_first(name):
    text = source(name)
    kernels = [m.start() for m in re.finditer(r"__global__ void ", text)]
    assert kernels
    for at in kernels:
        head = text[at:text.index("{", at)]
        body = block(text, at)
        assert body.count("block_op_wait();") == 1, head
        before = body[:body.index("block_op_wait();")]
        # no pointer of the arguments is followed, and nothing is called that follows one
        assert not re.search(r"\b[aw]\.[\w.]+\s*\[|[=(,;{!&|+-]\s*\*\s*[aw]\.|attn_range|__ldg|ldg_|load_|cp_async|bulk_copy|\breturn;", before), head
        # and it is one of the kernel's own statements
        assert before.count("{") - before.count("}") == 1, head
