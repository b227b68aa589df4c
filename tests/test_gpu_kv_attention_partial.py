"""Values that are no number and that only some drafts see, at either end of what the drafts see of a long
sequence: they stay with those drafts and that channel.  All widths, one and two row blocks, more rows, E4M3."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_kv_attention import BF, F16, call, problem  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


@pytest.mark.parametrize("max_pages", [40, 1100])
@pytest.mark.parametrize("io,fp8", [(BF, False), (F16, False), (BF, True)])
@pytest.mark.parametrize("group,T,D", [(4, 4, 64), (4, 4, 128), (4, 4, 256), (8, 3, 128), (8, 3, 256), (12, 4, 64), (16, 4, 128),
                                       (16, 6, 256)])
def test_both_ends(group, T, D, io, fp8, max_pages):
    n = 600
    p = problem([n, 33], group, 1, D, 16, T, io, fp8, 21 + D, max_pages=max_pages)
    keep = [c for c in range(D) if c != 5]
    for window in (0, 400):
        want, wl = call(p, 0.1, window)
        first = n - T - window + 1                          # what the first draft alone sees of the window
        for j in [n - 1, n - 2] + ([first, first + 1] if window else []):
            V = p["V"].clone()
            raw = V.view(torch.uint8) if fp8 else V
            raw[p["table"][0, j // 16], :, j % 16, 5] = 0x7f if fp8 else float("nan")
            got, gl = call(dict(p, V=V), 0.1, window)
            sees = [n - T + t >= j and (not window or n - T + t - window < j) for t in range(T)]
            assert any(sees) and not all(sees)
            for t in range(T):
                assert torch.isnan(got[t, 0, :, 5]).all() == sees[t]
                assert torch.equal(got[t, 0][:, keep], want[t, 0][:, keep])
                if not sees[t]:
                    assert torch.equal(got[t, 0], want[t, 0])
            assert torch.equal(got[:, 1], want[:, 1]) and torch.equal(gl, wl)


@pytest.mark.parametrize("max_pages", [40, 1100])
@pytest.mark.parametrize("group,T,D", [(4, 1, 64), (8, 3, 128), (16, 4, 128), (16, 6, 256)])
def test_an_infinite_value_that_all_see(group, T, D, max_pages):
    """It leaves no number in its channel and changes no other."""
    p = problem([300, 33], group, 1, D, 16, T, BF, False, 23, max_pages=max_pages)
    want, wl = call(p, 0.1)
    V = p["V"].clone()
    V[p["table"][0, 6], :, 4, 5] = float("inf")             # position 100
    got, gl = call(dict(p, V=V), 0.1)
    keep = [c for c in range(D) if c != 5]
    assert not torch.isfinite(got[:, 0, :, 5]).any()
    assert torch.equal(got[:, 0][:, :, keep], want[:, 0][:, :, keep]) and torch.equal(got[:, 1], want[:, 1])
    assert torch.equal(gl, wl)
