"""The largest sizes of the paged cache's calls, as far as the host refuses them (no GPU needed)."""
import ctypes

import pytest

from test_kv_abi_cpu import LIB, append, layer, pytestmark, rb, refused  # noqa: F401


@pytest.mark.parametrize("rows", [(1 << 25) - 1, 1 << 25, (1 << 31) - 1])
def test_rows_that_a_launch_cannot_hold(rows):
    """Two rows a workgroup of 256 lanes: a launch of 2^32 lanes is no launch."""
    b = rb()
    refused(b.lib().replay_kv_append(ctypes.byref(layer()), append(rows=rows), None), b.ERR_SHAPE)


# ---- how an attention call is cut (the library's own rule, called on the host) ----------------------
class Plan(ctypes.Structure):
    _fields_ = [("RB", ctypes.c_int), ("RW", ctypes.c_int), ("wide", ctypes.c_bool), ("rpc", ctypes.c_int),
                ("nchunk", ctypes.c_int), ("nwg", ctypes.c_int)]


def whole(D, fp8, rows, tokens, ranges):
    L = ctypes.CDLL(LIB)
    plan, rule = L._ZN2rs17kv_attention_planEibi, L._ZN2rs18kv_attention_wholeERKNS_6KvPlanEibxx
    plan.restype, plan.argtypes = Plan, [ctypes.c_int, ctypes.c_bool, ctypes.c_int]
    rule.restype = ctypes.c_bool
    rule.argtypes = [ctypes.POINTER(Plan), ctypes.c_int, ctypes.c_bool, ctypes.c_longlong, ctypes.c_longlong]
    p = plan(D, fp8, rows)
    return rule(ctypes.byref(p), D, fp8, tokens, ranges)


KINDS = [(D, fp8, rows) for D in (64, 128, 256) for fp8 in (False, True) for rows in (1, 4, 32, 64, 128)]


@pytest.mark.parametrize("D,fp8,rows", KINDS)
def test_the_cut_has_no_steps_at_certain_sizes(D, fp8, rows):
    """Shorter ranges than ones that are taken whole are so too, and where every workgroup has one it does not
    matter how many more there are."""
    sizes = list(range(32, 12000, 32))        # (35.5 us of 128 bytes a token are 11094 tokens)
    for ranges in (1, 7, 8, 192, 512, 2040, 2048, 2049, 30000):
        took = [whole(D, fp8, rows, n, ranges) for n in sizes]
        assert took == sorted(took, reverse=True)
        assert took[0] and not took[-1]
    for n in sizes:
        assert len({whole(D, fp8, rows, n, r) for r in (512, 1000, 2047, 2048, 4000)}) == 1


@pytest.mark.parametrize("D,fp8,rows", KINDS)
def test_few_ranges_are_split_by_their_bytes(D, fp8, rows):
    """Below some 7 us of one workgroup's work the join costs more than it saves, past some 12 it does not:
    40 GB/s, or 0.16 ns a channel and token through LDS."""
    us = lambda n: n * (0.16e-3 * D if rows > 32 else 2 * D * (1 if fp8 else 2) / 40e3)  # noqa: E731
    for ranges in (1, 8):
        for n in range(32, 3000, 32):
            if us(n) < 7:
                assert whole(D, fp8, rows, n, ranges)
            if us(n) > 12 + us(128):
                assert not whole(D, fp8, rows, n, ranges)


def test_tables_as_wide_as_a_context_say_nothing():
    for D, fp8, rows in KINDS:
        for ranges in (1, 512, 4096):
            assert not whole(D, fp8, rows, 32768, ranges)
