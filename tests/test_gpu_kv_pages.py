"""The page pool on the GPU against a sequential program: tables, slots, positions, free pages
and error bits are equal to the last number."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cases import rng  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def cuda(x, dtype):
    return torch.from_numpy(np.asarray(x, dtype=dtype)).cuda()


def pair(B, npages, page, mp):
    from hybrid_decode_replay_amd import binding as rb
    from oracle.kv_oracle import Pool
    return rb.KVPages(rb.kv_config(B, npages, page, mp)), Pool(B, npages, page, mp)


def same(pages, pool):
    nfree = int(pages.nfree)
    assert nfree == len(pool.free)
    assert pages.free[:nfree].tolist() == pool.free
    assert pages.len.tolist() == pool.len and pages.end.tolist() == pool.end
    assert pages.held.tolist() == [len(r) for r in pool.rows]
    assert (pages.table.cpu().numpy() == pool.table()).all()
    assert int(pages.err) == pool.err


@pytest.mark.parametrize("B,npages,page,mp,ntok", [(1, 1, 16, 1, 1), (1, 40, 16, 40, 16), (8, 60, 16, 9, 1),
                                                   (65, 300, 32, 6, 4), (300, 900, 64, 4, 7), (1500, 1200, 16, 3, 5),
                                                   (4096, 5000, 256, 2, 16)])
def test_steps(B, npages, page, mp, ntok):
    """Steps with idle sequences, partly accepted drafts, departures, until pages run out."""
    pages, pool = pair(B, npages, page, mp)
    same(pages, pool)
    r = rng(B, page, ntok)
    for step in range(9):
        active = (r.random(B) < 0.8).astype(np.uint8) if step % 3 else None
        slots, pos = pages.reserve(ntok, active=None if active is None else cuda(active, np.uint8))
        s, p, _ = pool.reserve([ntok] * B, active, "step")
        assert (slots.cpu().numpy() == s).all() and (pos.cpu().numpy() == p).all()
        same(pages, pool)
        if step % 2:
            acc = r.integers(-1, ntok + 2, B)
            pages.commit(cuda(acc, np.int32))
            pool.commit(acc)
        else:
            pages.commit()
            pool.commit()
        same(pages, pool)
        if step in (4, 6):
            mask = (r.random(B) < 0.4).astype(np.uint8)
            pages.release(cuda(mask, np.uint8))
            pool.release(mask)
            same(pages, pool)


@pytest.mark.parametrize("B,npages,page,mp,most,rows", [(1, 30, 16, 30, 400, 500), (5, 60, 16, 20, 300, 700),
                                                        (7, 5, 16, 20, 60, 400), (40, 400, 64, 12, 700, 9000),
                                                        (33, 300, 32, 8, 300, 900), (1100, 3000, 16, 4, 60, 40000)])
def test_arrivals(B, npages, page, mp, most, rows):
    """Ragged prompts in packed rows: empty ones, ones too long, rows and pages that run out; the rows
    behind the last sequence hold -1; a release undoes the reserve."""
    pages, pool = pair(B, npages, page, mp)
    r = rng(B, most)
    for turn in range(4):
        counts = r.integers(0, most + 1, B)
        counts[r.random(B) < 0.2] = 0
        if turn == 2:
            counts[B // 2] = -3
        active = (r.random(B) < 0.7).astype(np.uint8) if turn else None
        slots, pos, starts = pages.reserve(counts=cuda(counts, np.int32), rows=rows,
                                           active=None if active is None else cuda(active, np.uint8))
        s, p, st = pool.reserve(counts, active, "packed", rows)
        assert starts.tolist() == st
        assert (slots.cpu().numpy() == s).all() and (pos.cpu().numpy() == p).all()
        same(pages, pool)
        if turn == 1:
            pages.release()
            pool.release()
        else:
            pages.commit()
            pool.commit()
        same(pages, pool)


def test_release_is_the_reserves_inverse():
    pages, _ = pair(6, 64, 16, 20)
    pages.reserve(counts=cuda([5, 0, 40, 3, 100, 17], np.int32), rows=200)
    pages.commit()
    pages.release(cuda([0, 0, 1, 0, 1, 0], np.uint8))
    before = pages.mem.clone()
    args = dict(counts=cuda([9, 9, 200, 9, 33, 9], np.int32), active=cuda([0, 0, 1, 0, 1, 0], np.uint8), rows=300)
    first = pages.reserve(**args)
    pages.release(cuda([0, 0, 1, 0, 1, 0], np.uint8))
    n = int(pages.nfree)
    assert int(before[0]) == n
    again = pages.reserve(**args)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_sums_past_31_bits():
    """Counts whose sum passes 2^31: starts stay at 2^31 - 1, nobody behind is served."""
    pages, _ = pair(4, 8, 16, 8)
    slots, pos, starts = pages.reserve(counts=cuda([20, 2 ** 31 - 1, 2 ** 31 - 1, 5], np.int32), rows=64)
    assert starts.tolist() == [0, 20, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]
    assert pages.end.tolist() == [20, 0, 0, 0] and int(pages.err) == 2
    assert pos.tolist() == list(range(20)) + [-1] * 44
    assert (slots[20:] == -1).all()


def test_rows_behind_the_step():
    pages, _ = pair(3, 8, 16, 2)
    slots, pos = pages.reserve(2, rows=11)
    assert (slots[6:] == -1).all() and (pos[6:] == -1).all() and (pos[:6] == cuda([0, 0, 0, 1, 1, 1], np.int32)).all()
