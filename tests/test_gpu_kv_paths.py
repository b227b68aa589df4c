"""Paged decode attention over tables too wide to say how long the sequences are: few ranges and many
that are split, and ranges of like lengths that the kernel takes whole, for the kernels of few rows and
of many."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cases import rng  # noqa: E402
from test_gpu_kv_attention import BF, F16, problem  # noqa: E402
from test_gpu_kv_attention_split import verify  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


# rows of a head: one block of 16, two, two and four row groups
ROWS = [(2, 1), (8, 3), (12, 4), (12, 9)]
WIDE = 16 * 1024                               # tokens of a table (165 us of a workgroup at the least)


@pytest.mark.parametrize("io,fp8,D", [(BF, False, 64), (BF, True, 128), (F16, False, 256)])
@pytest.mark.parametrize("group,T", ROWS)
def test_few_ranges(group, T, io, fp8, D):
    verify(problem([701, 0, 40, 1300], 2 * group, 2, D, 64, T, io, fp8, D + T, max_pages=WIDE // 64))


@pytest.mark.parametrize("io,fp8,D", [(BF, False, 64), (BF, True, 64), (F16, False, 128)])
@pytest.mark.parametrize("group,T", ROWS)
def test_more_ranges_than_workgroups_on_the_line(group, T, io, fp8, D):
    """One sequence much longer than an even share."""
    r = rng(group, T, D)
    lens = [int(n) for n in r.integers(0, 40, 600)]
    lens[100] = 2600
    verify(problem(lens, group, 1, D, 16, T, io, fp8, 90 + T, max_pages=WIDE // 16))


@pytest.mark.parametrize("io,fp8,D", [(BF, False, 64), (BF, True, 64), (BF, True, 128), (F16, True, 256)])
@pytest.mark.parametrize("group,T", ROWS)
def test_like_lengths_by_length(group, T, io, fp8, D):
    """None longer than an even share (two tiles of 128 tokens, at least 1040 for 512 workgroups): whole,
    the longest first."""
    r = rng(group, T, D, 1)
    lens = [int(n) for n in r.integers(1, 200, 520)]
    verify(problem(lens, 2 * group, 2, D, 16, T, io, fp8, 91 + T, max_pages=WIDE // 16))
