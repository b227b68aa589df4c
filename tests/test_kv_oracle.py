"""The paged cache's references pinned by hand-made cases, by torch's own conversions and by the
reference's invariants."""
import numpy as np
import pytest

from oracle import kv_oracle as ko


def test_pool_by_hand():
    p = ko.Pool(2, 4, 16, 3)
    s, pos, st = p.reserve([17, 3], None, "packed", 24)
    assert st == [0, 17, 20]
    assert s.tolist() == list(range(16)) + [16] + [32, 33, 34] + [-1] * 4
    assert pos.tolist() == list(range(17)) + [0, 1, 2] + [-1] * 4
    p.commit()
    assert p.len == [17, 3] and p.free == [3]
    s, pos, _ = p.reserve([14, 14], None, "step")                # 31 tokens in two pages, 17 in one more
    assert p.free == [] and p.end == [31, 17] and p.err == 0
    assert pos.tolist() == [x for i in range(14) for x in (17 + i, 3 + i)]
    assert s[-2:].tolist() == [16 + 30 - 16, 3 * 16]
    p.commit([1, 99])
    assert p.len == [18, 17] and p.err == ko.CLAMPED


def test_pool_inverse_and_order():
    p = ko.Pool(3, 9, 16, 4)
    p.reserve([40, 1, 30], None, "packed", 100)
    table, free = p.table().copy(), list(p.free)
    p.release()
    p.reserve([40, 1, 30], None, "packed", 100)
    assert (p.table() == table).all() and p.free == free


def test_pool_runs_out_in_order():
    p = ko.Pool(4, 3, 16, 4)
    p.reserve([16, 40, 1, 0], None, "packed", 100)               # 1 + 3 + 1 + 0 pages of 3
    assert p.end == [16, 0, 0, 0] and p.err == ko.NO_PAGES and len(p.free) == 2
    p.commit([-1, 0, 0, 0])
    assert p.err == ko.NO_PAGES | ko.CLAMPED and p.len == [0] * 4


def test_rotation_by_hand():
    x = np.zeros((1, 1, 4))
    x[0, 0] = [1, 2, 3, 4]
    quarter = np.pi / 2
    assert np.allclose(ko.rotate(x, [[1]], [quarter, 0.0], None, 4, False)[0, 0], [-3, 2, 1, 4])
    assert np.allclose(ko.rotate(x, [[1]], [quarter, 0.0], None, 4, True)[0, 0], [-2, 1, 3, 4])
    assert np.allclose(ko.rotate(x, [[0], [2]], [quarter, quarter], [0, 1], 4, True)[0, 0], [1, 2, -3, -4])
    assert np.allclose(ko.rotate(x, [[1]], [quarter, quarter], [0, 1], 4, True)[0, 0], [-2, 1, 3, 4])


def test_e4m3_against_torch():
    torch = pytest.importorskip("torch")
    r = np.random.default_rng(0)
    x = (r.normal(size=20000) * np.exp(r.uniform(-12, 5, 20000))).astype(np.float32)
    x = np.concatenate([x, ko.e4m3_values(), (ko.e4m3_values()[1:] + ko.e4m3_values()[:-1]) / 2]).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (ko.to_e4m3(x) == want).all()


def test_attention_by_hand():
    K = np.zeros((2, 1, 16, 2))
    V = np.zeros((2, 1, 16, 2))
    K[1, 0, 0], V[1, 0, 0] = [1, 0], [10, 0]
    K[1, 0, 1], V[1, 0, 1] = [0, 1], [0, 10]
    q = np.array([[[[np.log(3.0), 0.0]]], [[[0.0, 0.0]]]])
    table = np.array([[1, -1]], np.int32)
    o, lse, _, _ = ko.attention(q, K, V, table, [2], 1.0)
    assert np.allclose(o[0, 0, 0], [10, 0]) and np.allclose(lse[0, 0, 0], np.log(3))     # sees token 0 alone
    assert np.allclose(o[1, 0, 0], [5, 5]) and np.allclose(lse[1, 0, 0], np.log(2))
    o, lse, _, _ = ko.attention(q, K, V, table, [2], 1.0, window=1)
    assert np.allclose(o[1, 0, 0], [0, 10])
    o, lse, _, _ = ko.attention(q, K, V, table, [1], 1.0)
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all() and np.allclose(o[1, 0, 0], [10, 0])
    o, lse, _, _ = ko.attention(q, K, V, np.array([[-1, 7]], np.int32), [20], 1.0)
    assert (o == 0).all() and np.isneginf(lse).all()
