"""README's example of a decode step over the paged cache, run as it stands there."""
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def example():
    path = os.path.join(ROOT, "README.md")
    if not os.path.exists(path):
        pytest.skip("a copy without its README")
    with open(path) as f:
        blocks = f.read().split("```")[1::2]
    found = [b for b in blocks if "rb.KVPages" in b]
    assert len(found) == 1
    return found[0]


@pytest.mark.parametrize("ntok", [1, 3])
def test_the_paged_step(ntok):
    from hybrid_decode_replay_amd import binding as rb
    batch, Hq, Hkv, D = 3, 4, 2, 64
    g = torch.Generator().manual_seed(ntok)
    rows = lambda heads: torch.randn((ntok * batch, heads * D), generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    words = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    mask = torch.tensor([1, 0, 1], dtype=torch.uint8, device="cuda")
    v = rows(Hkv)
    names = dict(rb=rb, torch=torch, batch=batch, npages=8, page_size=16, max_pages=4, Hq=Hq, Hkv=Hkv, D=D, ntok=ntok,
                 mask=mask, q=rows(Hq), k=rows(Hkv), v=v, freq=torch.rand(D // 2, generator=g).cuda(),
                 accepted=words(ntok, 0, 1), departed=torch.tensor([1, 0, 0], dtype=torch.uint8, device="cuda"))
    exec(example(), names)
    torch.cuda.synchronize()
    pages, o = names["pages"], names["o"]
    assert int(pages.err) == 0
    assert pages.len.tolist() == [0, 0, 1] and int(pages.nfree) == 7
    # the first new token sees itself alone: its output is its value
    first = v.view(ntok, batch, Hkv, D)[0].repeat_interleave(Hq // Hkv, 1)
    assert torch.equal(o[0, 0], first[0]) and torch.equal(o[0, 2], first[2]) and (o[:, 1] == 0).all()
