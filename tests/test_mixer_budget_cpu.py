"""Scratch and waves of the norm, E4M3 projection and prompt kernels, read from the compiler (no GPU needed).

Kernels that spill pass every numerics test at half their rate: none may use scratch, and each must leave room for the
waves that its launch bounds count on.  Template arguments are read from the mangled names in order: linear_tile_kernel
<..., waves a SIMD>, gdn_chunk_kernel, gdn_state_kernel and gdn_short_kernel <d_k, ...>.
"""
import os
import re
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from hybrid_decode_replay_amd import build as hb
from test_kernel_budget_cpu import _remarks
from test_kv_budget_cpu import _kernels

UNITS = ["norm.hip", "linear_fp8.hip", "gdn_prefill.hip", "gdn_chunks.hip", "gdn_short.hip"]


def waves_needed(name):
    args = [int(x) for x in re.findall(r"L[ib](\d+)E", name)]
    if "linear_tile" in name:
        return args[-1]
    if "gdn_tokens" in name or "norm" in name:
        return 1
    return 1 if args[0] == 256 else 3 if "gdn_chunk" in name else 2


@pytest.mark.skipif(not (os.path.exists(hb.HIPCC) or shutil.which(hb.HIPCC)), reason="hipcc not available")
def test_mixer_kernels_use_no_scratch_and_leave_room_for_their_waves(tmp_path):
    assert set(UNITS) <= set(hb.SOURCES)
    with ThreadPoolExecutor(max_workers=len(UNITS)) as ex:
        found = [k for t in ex.map(lambda u: _remarks(u, str(tmp_path)), UNITS) for k in _kernels(t)]
    for part in ("norm_kernel", "linear_tile_kernel", "gdn_tokens_kernel", "gdn_chunk_kernel", "gdn_state_kernel", "gdn_short_kernel"):
        assert any(part in n for n, _, _ in found)
    bad = [f"{n}: {scratch} B/lane scratch, {waves} waves/SIMD (needs {waves_needed(n)})" for n, scratch, waves in found
           if scratch > 0 or waves < waves_needed(n)]
    assert not bad, "\n".join(bad)


@pytest.mark.skipif(not (os.path.exists(hb.HIPCC) or shutil.which(hb.HIPCC)), reason="hipcc not available")
def test_four_workgroups_of_the_chunk_kernel_fit_a_cu(tmp_path):
    """Below d_k 256 its launch bounds, and the time of its launch, count on four waves a SIMD; three would pass the test above."""
    found = {n: waves for n, _, waves in _kernels(_remarks("gdn_chunks.hip", str(tmp_path))) if "gdn_chunk_kernel" in n}
    assert len(found) == 3
    assert all(waves >= 4 for n, waves in found.items() if "Li256E" not in n), found
