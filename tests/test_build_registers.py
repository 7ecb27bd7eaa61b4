"""Kernels that split registers between their warps: the build refuses any other number a thread than the split counts
on, of any of a kernel's forms."""
import os
import re

import pytest

from audio_video_flow_gb300 import _build

SOURCE = os.path.join(_build.CSRC, "k_attention_window.cu")


def log(*registers, kernel="attention_window_kernel"):
    return "".join(f"ptxas info    : Compiling entry function '_ZN2h323{kernel}ILi{i}EEEv14CUtensorMap_stS1_' for 'sm_103a'\n"
                   f"ptxas info    : Function properties for _ZN2h323{kernel}ILi{i}EEEv14CUtensorMap_stS1_\n"
                   f"    8 bytes stack frame, 4 bytes spill stores, 16 bytes spill loads\n"
                   f"ptxas info    : Used {n} registers, used 2 barriers, 8 bytes cumulative stack size\n"
                   for i, n in enumerate(registers))


def test_the_count_is_the_split_s():
    text = open(SOURCE).read()
    assert int(re.search(r"AW_REGS = (\d+)", text).group(1)) == _build.REGISTERS["attention_window_kernel"]
    _build.check_registers(SOURCE, log(168, 168, 168))


@pytest.mark.parametrize("text", [log(160, 168, 168), log(168, 168, 170), log(), log(168, kernel="another_kernel")])
def test_another_count_is_refused(text):
    with pytest.raises(RuntimeError, match="attention_window_kernel"):
        _build.check_registers(SOURCE, text)


def test_every_kernel_that_splits_registers_is_checked():
    for name in os.listdir(_build.CSRC):
        text = open(os.path.join(_build.CSRC, name)).read()
        if "setmaxnreg" in text:
            assert any(f" {k}(" in text.replace("\n", " ") for k in _build.REGISTERS), name
    for name in ("k_cache.cu", "k_norm.cu"):
        _build.check_registers(os.path.join(_build.CSRC, name), "")


def test_the_library_here_passes():
    _build.build()
    path = os.path.join(_build.BUILD, "k_attention_window.cu.log")
    _build.check_registers(SOURCE, open(path).read())
