"""Scratch and waves of the paged-cache kernels, read from the compiler (no GPU needed).

A token loop that spills runs at half its rate and still passes every numerics test, so no kernel
of the cache may use scratch, and the attention kernels must leave room for the waves that their
launch bounds and the plan of the call count on: two per SIMD, or one where the head is too wide.
Template arguments are read from the mangled names in order: kv_attention_kernel <IO, FP8, D, row
blocks, workgroups per CU>, kv_attention_wide_kernel <IO, FP8, D, row blocks, row groups>.
"""
import os
import re
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from hybrid_decode_replay_amd import build as hb
from test_kernel_budget_cpu import _remarks

UNITS = [u for u in hb.SOURCES if u.startswith("kv_")]


def _kernels(text):
    """(mangled name, scratch bytes per lane, waves per SIMD) of every kernel in the remarks."""
    name = scratch = None
    for line in text.splitlines():
        if m := re.search(r"Function Name: (\S+)", line):
            name = m.group(1)
        elif m := re.search(r"ScratchSize \[bytes/lane\]: (\d+)", line):
            scratch = int(m.group(1))
        elif m := re.search(r"Occupancy \[waves/SIMD\]: (\d+)", line):
            yield name, scratch, int(m.group(1))


@pytest.mark.skipif(not (os.path.exists(hb.HIPCC) or shutil.which(hb.HIPCC)), reason="hipcc not available")
def test_cache_kernels_use_no_scratch_and_leave_room_for_their_waves(tmp_path):
    with ThreadPoolExecutor(max_workers=len(UNITS)) as ex:
        found = [k for t in ex.map(lambda u: _remarks(u, str(tmp_path)), UNITS) for k in _kernels(t)]
    assert sum("kv_attention" in n for n, _, _ in found) == 4 * (3 * 2 + 2 + 2 + 1)     # types x (direct + wide by width)
    bad = []
    for name, scratch, waves in found:
        need = 1
        if "kv_attention" in name:
            last = int(re.findall(r"L[ib](\d+)E", name)[-1])
            need = 2 if "wide" in name else last
        if scratch > 0 or waves < need:
            bad.append(f"{name}: {scratch} B/lane scratch, {waves} waves/SIMD (needs {need})")
    assert not bad, "\n".join(bad)
