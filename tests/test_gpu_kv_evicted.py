"""Tables whose pages before a sliding window are gone: nobody sees them, so nothing changes and no
error is reported."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_kv_attention import BF, call, problem  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


@pytest.mark.parametrize("max_pages", [30, 300])
@pytest.mark.parametrize("group,T,D", [(4, 1, 64), (8, 3, 128), (16, 4, 64), (16, 4, 256)])
@pytest.mark.parametrize("gone", [None, -1, 10 ** 6])
def test_pages_before_the_window(gone, group, T, D, max_pages):
    lens, window, page = [100, 130, 33, 400], 50, 16
    p = problem(lens, group, 1, D, page, T, BF, False, 70 + D, max_pages=max_pages)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, wl = call(p, 0.1, window, err=err)
    assert int(err) == 0
    first = [max(0, n - T - window + 1) for n in lens]      # what the first draft sees first
    assert any(f % 32 >= 16 for f in first)                 # (a page that ends inside a block of 32)
    if gone is None:                                        # the first visible page itself
        p["table"][0, first[0] // page] = -1
        call(p, 0.1, window, err=err)
        assert int(err) == 4
        return
    for b, f in enumerate(first):
        p["table"][b, :f // page] = gone
    got, gl = call(p, 0.1, window, err=err)
    assert int(err) == 0
    assert torch.equal(got, want) and torch.equal(gl, wl)
