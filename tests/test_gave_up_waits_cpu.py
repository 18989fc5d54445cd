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
    """attn_store stores NaN where sh_bad is set: every wait that reports a fault marks its thread, and all three kinds of warps
    set sh_bad for a marked thread before the barrier in front of attn_store."""
    text = source("zdmmv_attn_prompt.cuh")
    reports = text.count("atomicOr(a.fault")
    assert reports >= 2
    assert sum("atomicOr(a.fault" in b and "dead = true" in b for b in waits_that_report(text)) == reports
    kernel = block(text, text.index("attn_prompt_kernel(AttnArgs a)"))
    roles = kernel.split("asm volatile(\"setmaxnreg.")[1:4]
    assert [r.count("if (dead) sh_bad = 1;") for r in roles] == [1, 1, 1]
    for r in roles:
        assert "wait(" not in r[r.index("if (dead) sh_bad = 1;"):].replace("tm_", "")


def test_the_append_rings_last_waits():
    """After a wait that gave up a warp of the prompts' kernel waits once for each copy that it still has in flight, on the slot
    and the parity that the copy completes, and for nothing else."""
    text = source("zdmmv_kv.cu")
    text = block(text, text.index("kv_append_stream_kernel(AppendArgs a, int n_jobs)"))
    slots = int(re.search(r"kStreamSlots = (\d+)", source("zdmmv_kv.cu")).group(1))
    waits = re.findall(r"[^\n]*mbar_wait\([^\n]*", text)
    assert len(waits) == 2 and "break;" in waits_that_report(text)[0]     # none in the loop once one gave up
    m = re.search(r"for \(int k = (.+?); k < (.+?); \+\+k\) \(void\)mbar_wait\(&full\[(.+?)\], (.+?)\);", text)
    lo, hi, slot, parity = (compile(x.replace("/", "//"), "zdmmv_kv.cu", "eval") for x in m.groups())
    for first, last in ((0, 1), (0, 9), (4, 6), (5, 20), (100, 103)):
        for lost in range(first, last):
            names = {"first": first, "last": last, "lost": lost, "kStreamSlots": slots, "min": min}
            got = [(eval(slot, {**names, "k": k}), eval(parity, {**names, "k": k})) for k in range(eval(lo, names), eval(hi, names))]
            # the ring as the loop runs it: job j in slot s, whose barrier's phase flips with every round
            issued, s, phase = list(range(first, min(first + slots, last))), 0, 0
            at = {}
            for job in range(first, last):
                at[job] = (s, phase)
                if job < lost and job + slots < last:
                    issued.append(job + slots)
                s += 1
                if s == slots:
                    s, phase = 0, phase ^ 1
            assert got == [at[j] for j in issued if j >= lost]
