"""The build says so when a kernel that shares its registers out was compiled with another number of them."""
import re

import pytest

from gguf_block_quant_gb300 import _build

LOG = """ptxas info    : Compiling entry function '_ZN5zdmmv18attn_prompt_kernelILi4EEEvNS_8AttnArgsE' for 'sm_103a'
ptxas info    : Function properties for _ZN5zdmmv18attn_prompt_kernelILi4EEEvNS_8AttnArgsE
    56 bytes stack frame, 72 bytes spill stores, 84 bytes spill loads
ptxas info    : Used {} registers, used 3 barriers, 56 bytes cumulative stack size, 3968 bytes smem
ptxas info    : Compiling entry function '_ZN5zdmmv5otherEv' for 'sm_103a'
ptxas info    : Used 32 registers
"""


@pytest.mark.parametrize("n", [80, 96])
def test_registers_are_read_from_the_compilers_report(n):
    assert _build.registers_of(LOG.format(n), "attn_prompt_kernel") == [n]
    assert _build.registers_of(LOG.format(n), "other") == [32]


def test_a_build_with_other_registers_fails(monkeypatch, tmp_path):
    class Done:
        returncode, stdout, stderr = 0, "", LOG.format(88)
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(_build.subprocess, "run", lambda *a, **k: Done)
    with pytest.raises(RuntimeError, match="attn_prompt_kernel: .88. registers"):
        _build.build()


def test_the_numbers_are_the_sources():
    import os
    text = open(os.path.join(_build.CSRC, "zdmmv_attn_prompt.cuh")).read()
    assert int(re.search(r"kRegsLaunch = (\d+)", text).group(1)) == _build.REGISTERS["zdmmv_attn_prompt.cu"][1]
