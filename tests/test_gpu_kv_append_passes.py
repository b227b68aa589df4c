"""Cache appends whose rows have more items than a workgroup's one pass (512 pairs of 16-byte chunks for one
row, 768 for two), and the two-row kernel in every type and style."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_kv_append import BF, F16, call, setup, verify  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


KINDS = [(BF, False), (F16, False), (BF, True), (F16, True)]
# 640 items a row (a second pass of one row and of two); 1280 (a third); 352 (the second of the items in flight)
HEADS = [(64, 8, 128, 96), (64, 8, 256, 256), (66, 11, 64, 32)]


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("io,fp8", KINDS)
@pytest.mark.parametrize("Hq,Hkv,D,rot", HEADS)
def test_one_row_a_workgroup(Hq, Hkv, D, rot, io, fp8, style):
    p = setup(9, Hq, Hkv, D, 16, io, fp8, rot, style, 2, D + Hq)
    verify(p, *call(p))


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("io,fp8", KINDS)
@pytest.mark.parametrize("N,Hq,Hkv,D,rot", [(1027, 20, 10, 128, 64), (1026, 10, 2, 256, 64), (1029, 7, 7, 64, 0)])
def test_two_rows_a_workgroup(N, Hq, Hkv, D, rot, io, fp8, style):
    """640 items of two rows, 448 and 168; the last workgroup has one row or two."""
    p = setup(N, Hq, Hkv, D, 32, io, fp8, rot, style, 1, N, idle=0.25)
    verify(p, *call(p))


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("io,fp8", [(BF, False), (F16, True)])
def test_two_rows_in_two_passes(io, fp8, style):
    p = setup(1025, 64, 8, 128, 64, io, fp8, 32, style, 3, 5, idle=0.25)
    verify(p, *call(p))


def test_two_rows_without_queries():
    p = setup(1030, 64, 64, 128, 16, BF, False, 128, 0, 1, 6)
    p["axis"].zero_()
    _, K, V = call(p, with_q=False, axis=None)
    verify(p, None, K, V, axis=False)
