"""What the attention half's kernels do after a wait that gave up, read from their sources: such a wait cannot be brought about
without breaking a kernel."""
import os
import re

from gguf_block_quant_gb300 import _build


def source(name):
    text = open(os.path.join(_build.CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def block(text, at):
    """The braces' contents that begin at or after `at`."""
    i = text.index("{", at)
    depth, j = 0, i
    while True:
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        j += 1
        if depth == 0:
            return text[i:j]


def waits_that_report(text):
    return [block(text, m.start()) for m in re.finditer(r"if \([^{;]*mbar_wait\([^{;]*\)(?= (?:\{|atomicOr))", text)]


def test_the_prompt_kernel_poisons_its_result():
    """attn_store stores NaN where sh_bad is set: every wait that reports a fault sets it."""
    text = source("zdmmv_attn_prompt.cuh")
    reports = text.count("atomicOr(a.fault")
    assert reports >= 2
    assert sum("atomicOr(a.fault" in b and "sh_bad = 1" in b for b in waits_that_report(text)) == reports
