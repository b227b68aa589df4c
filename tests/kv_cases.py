"""Inputs and error bounds shared by the paged key/value cache tests."""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}      # half a step, relative
SUBNORMAL = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def rng(*seed):
    return np.random.default_rng(list(seed))


def f64(t):
    """A tensor's values in fp64 numpy (E4M3 decoded)."""
    return t.detach().float().cpu().numpy().astype(np.float64)


def normal(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(shape, generator=g)).to(dtype)


def paged(lens, page, npages, max_pages, seed):
    """A table of distinct pages in a seeded order, -1 behind each sequence's last."""
    r = rng(seed, 77)
    order = r.permutation(npages)
    table = np.full((len(lens), max_pages), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        k = -(-int(n) // page)
        assert at + k <= npages and k <= max_pages
        table[b, :k] = order[at:at + k]
        at += k
    return table


def attention_bounds(o, lse, top, a, D, longest, io):
    """Largest differences an output may have, element by element.

    Scores: D products summed in fp32, (D + 2) 2^-24 of scale sum |q k|; scale, log2(e) and the
    reference's rounding add at most 4 more.  exp2 is good to 2^-22.  Together a weight is off by
    eps relative.  Weights are carried as two io terms: what is left over is (half step)^2.  A
    lane's sums take longest / 16 + 64 additions of 2^-24.  Numerator and denominator both: twice.
    Then one rounding to the io type."""
    eps = (D + 6) * 2.0 ** -24 * top + 2.0 ** -22
    sums = (longest / 16 + 64) * 2.0 ** -24
    rel = 2 * (eps + sums) + HALF[io] ** 2
    bound_o = rel[..., None] * a
    bound_o = bound_o + HALF[io] * (np.abs(o) + bound_o) + SUBNORMAL[io]
    bound_lse = eps + sums + 2.0 ** -22 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))
    return bound_o, bound_lse


def check_attention(o, lse, ref, D, longest, io):
    ro, rl, top, a = ref
    bo, bl = attention_bounds(ro, rl, top, a, D, longest, io)
    got = f64(o)
    assert np.isfinite(got).all()
    worst = float((np.abs(got - ro) / bo).max())
    assert worst <= 1.0, f"output error {worst:.3f} of its bound"
    if lse is not None:
        gl = f64(lse)
        fin = np.isfinite(rl)
        assert (np.isneginf(gl) == ~fin).all()
        if fin.any():
            w = float((np.abs(gl[fin] - rl[fin]) / bl[fin]).max())
            assert w <= 1.0, f"lse error {w:.3f} of its bound"
    return worst
