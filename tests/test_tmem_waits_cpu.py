"""Loads from tensor memory that are in flight together: the one wait for them ties the registers of all, not only of
the first, so that the compiler can move no use of one above it."""
import os
import re

from audio_video_flow_gb300 import _build


def test_a_wait_ties_every_load_before_it():
    for name in sorted(os.listdir(_build.CSRC)):
        text = open(os.path.join(_build.CSRC, name)).read()
        if name != "h3_device.cuh":                        # (where the wait for several is made of that for one)
            assert not re.findall(r"tmem_ld_wait\(\w+\[0\]\)", text), name
        for loop in re.finditer(r"for \(int (\w+) = 0;[^\n]*\n?\s*tmem_ld32\([^;]*, (\w+)\[\1\]\);\n([^\n]*)", text):
            array, rest = loop.group(2), text[loop.end(2):loop.end(2) + 400]
            each = re.search(r"uint32_t\(&(\w+)\)\[32\] = %s\[\w+\];\s*tmem_ld_wait\(\1\);" % array, rest)
            assert each or re.search(r"tmem_ld_wait\(%s\);" % array, rest), (name, loop.group(0))
