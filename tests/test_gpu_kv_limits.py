"""The largest sizes of the paged cache's calls."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def test_a_count_and_rows_of_31_bits():
    """As many rows as the call can name (26 GB of slots and positions) and a count to fill them, which
    no table holds: every row is marked, nothing is taken.  The row index has to pass 2^31 to end."""
    from hybrid_decode_replay_amd import binding as rb
    rows = 2 ** 31 - 1
    pages = rb.KVPages(rb.kv_config(2, 8, 16, 8))
    slots = torch.zeros(rows, dtype=torch.int64, device="cuda")
    pos = torch.zeros(rows, dtype=torch.int32, device="cuda")
    counts = torch.tensor([3, rows], dtype=torch.int32, device="cuda")
    _, _, starts = pages.reserve(counts=counts, slots=slots, pos=pos)
    assert starts.tolist() == [0, 3, 2 ** 31 - 1] and pages.end.tolist() == [3, 0] and int(pages.err) == 2
    assert slots[:3].tolist() == [0, 1, 2] and pos[:3].tolist() == [0, 1, 2]
    for x in (slots, pos):
        assert int(x[3:].min()) == -1 and int(x[3:].max()) == -1
