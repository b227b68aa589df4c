"""Paged decode attention where ranges may be long, so that their tokens are split over workgroups
and joined: tables that hold more than 2560 tokens a sequence.  All widths, types and row counts,
with empty, short and long sequences, windows, masks and bad pages."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cases import check_attention, rng  # noqa: E402
from test_gpu_kv_attention import BF, F16, call, problem, reference  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def verify(p, scale=None, window=0, **kw):
    """Lanes of the many-row kernel sum a quarter of the tokens, four times the others' share."""
    D = p["layer"].head_dim
    scale = D ** -0.5 if scale is None else scale
    o, lse = call(p, scale, window, **kw)
    rows = p["T"] * p["layer"].nheads // p["layer"].nkv
    w = check_attention(o, lse, reference(p, scale, window), D, int(p["end"].max()) * (4 if rows > 32 else 1), p["io"])
    print(f"error {w:.3f} of the bound", flush=True)


# rows of a head: one, a product's 16, two products, a row past them, two and four row groups, two chunks
ROWS = [(1, 1), (16, 1), (32, 1), (11, 3), (16, 4), (13, 5), (16, 8), (27, 5)]
MIXED = [300, 0, 1, 129, 2049, 64]


@pytest.mark.parametrize("io,fp8", [(BF, False), (F16, False), (BF, True), (F16, True)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group,T", ROWS)
def test_rows_widths_and_types(group, T, D, io, fp8):
    verify(problem(MIXED, 2 * group, 2, D, 32, T, io, fp8, 7 * group + T + D, max_pages=90))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group,T", [(4, 1), (4, 6), (8, 6), (8, 16)])
@pytest.mark.parametrize("window", [1, 40, 1500, 2600])
def test_windows(window, group, T, D):
    """2600 positions are too many for a workgroup each, fewer are not."""
    verify(problem([2900, 5, 700], group, 1, D, 64, T, BF, False, window + T, max_pages=50), window=window)


@pytest.mark.parametrize("group,T,D", [(4, 1, 128), (8, 16, 128), (8, 5, 64), (16, 8, 256)])
def test_one_long_sequence(group, T, D):
    verify(problem([9011], group, 1, D, 16, T, BF, False, D + T))


@pytest.mark.parametrize("group,T", [(2, 1), (12, 4), (12, 12)])
def test_more_ranges_than_workgroups(group, T):
    r = rng(group, T)
    lens = [int(n) for n in r.integers(0, 70, 600)]
    lens[100] = 2600
    verify(problem(lens, 2 * group, 2, 64, 16, T, BF, False, 90 + T, max_pages=170))


def test_many_ranges_of_middling_length():
    """At least 2048 ranges of up to 2560 tokens: a workgroup each."""
    r = rng(4)
    lens = [int(n) for n in r.integers(0, 40, 1030)]
    lens[7], lens[1029] = 2560, 2100
    verify(problem(lens, 4, 2, 64, 16, 1, BF, False, 91, max_pages=160))


@pytest.mark.parametrize("max_pages", [20, 200])
@pytest.mark.parametrize("group,T,D", [(3, 2, 64), (8, 2, 256), (8, 5, 128), (8, 5, 256), (16, 8, 64)])
@pytest.mark.parametrize("fp8", [False, True])
def test_what_lies_in_masked_places(fp8, group, T, D, max_pages):
    """NaN behind the end, in unused pages and outside the window changes nothing."""
    p = problem([37, 0, 290, 4], group, 1, D, 16, T, BF, fp8, 12 + D, max_pages=max_pages)
    for window in (0, 24):
        want, wl = call(p, 0.09, window)
        raws = []
        for x in (p["K"].clone(), p["V"].clone()):
            seen = torch.zeros(x.shape[0], 16, dtype=torch.bool)
            for b, n in enumerate(p["end"].tolist()):
                for j in range(max(0, n - T - window + 1) if window else 0, n):
                    seen[p["table"][b, j // 16], j % 16] = True
            raw = x.view(torch.uint8) if fp8 else x
            raw.permute(0, 2, 1, 3)[~seen] = 0x7f if fp8 else float("nan")
            raws.append(x)
        got, gl = call(dict(p, K=raws[0], V=raws[1]), 0.09, window)
        assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("max_pages", [20, 200])
@pytest.mark.parametrize("group,T,D", [(4, 3, 64), (16, 3, 128), (16, 3, 256), (16, 8, 128)])
def test_a_drafts_nan_stays_with_those_who_see_it(group, T, D, max_pages):
    p = problem([70, 33], group, 1, D, 16, T, BF, False, 21, max_pages=max_pages)
    want, _ = call(p, 0.125)
    for back in (1, 2):                                     # the last draft's value, the one's before it
        V = p["V"].clone()
        j = 70 - back
        V[p["table"][0, j // 16], :, j % 16, 5] = float("nan")
        got, _ = call(dict(p, V=V), 0.125)
        assert torch.equal(got[:T - back], want[:T - back]) and torch.equal(got[:, 1], want[:, 1])
        assert torch.isnan(got[T - back:, 0, :, 5]).all()
        keep = [c for c in range(D) if c != 5]
        assert torch.equal(got[:, 0][:, :, keep], want[:, 0][:, :, keep])


@pytest.mark.parametrize("max_pages", [32, 300])
@pytest.mark.parametrize("group,T", [(2, 2), (16, 4), (16, 10)])
def test_bad_pages_and_ends(group, T, max_pages):
    """Pages outside the cache are masked, an end past the table is its end, a negative one empty."""
    p = problem([100, 64, 47, 30, 20], 2 * group, 2, 64, 16, T, BF, False, 44, max_pages=max_pages)
    p["table"][0, 2] = -1
    p["table"][1, :] = 10 ** 6
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = call(p, 0.125, err=err)
    check_attention(o, lse, reference(p, 0.125), 64, 128, BF)
    assert int(err) == 4 and (o[:, 1] == 0).all() and torch.isneginf(lse[:, 1]).all()
    q = problem([100, 64, 47, 30, 20], 2 * group, 2, 64, 16, T, BF, False, 44, max_pages=max_pages)
    err.zero_()
    want, _ = call(q, 0.125, err=err)
    assert int(err) == 0
    for bad in (-1, -2 ** 31):
        q["end"][3] = bad
        err.zero_()
        o, lse = call(q, 0.125, err=err)
        assert int(err) == 4 and (o[:, 3] == 0).all() and torch.isneginf(lse[:, 3]).all()
        assert torch.equal(o[:, :3], want[:, :3]) and torch.equal(o[:, 4], want[:, 4])
    # ... also the largest; a sequence that is idle reports nothing
    q["end"][3] = 2 ** 31 - 1
    err.zero_()
    active = torch.tensor([1, 1, 1, 0, 1], dtype=torch.uint8, device="cuda")
    o, lse = call(q, 0.125, err=err, active=active, o=torch.full_like(want, 3.0))
    assert int(err) == 0 and (o[:, 3] == 3.0).all() and (lse[:, 3] == 7.0).all() and torch.equal(o[:, :3], want[:, :3])


@pytest.mark.parametrize("max_pages", [40, 300])
@pytest.mark.parametrize("group,T", [(4, 1), (16, 4), (16, 10)])
def test_idle_sequences_keep_their_outputs(group, T, max_pages):
    p = problem([60, 0, 300, 8, 600], group, 1, 128, 16, T, BF, False, 50, max_pages=max_pages)
    want, wl = call(p, 0.09)
    for mask in ([1, 0, 0, 1, 1], [0, 1, 1, 0, 0], [0, 0, 0, 0, 0]):
        mark = torch.full_like(want, 3.0)
        got, gl = call(p, 0.09, active=torch.tensor(mask, dtype=torch.uint8, device="cuda"), o=mark)
        for b, on in enumerate(mask):
            if on:                                          # (the cut of the work moves with the mask: not bit for bit)
                assert torch.allclose(got[:, b].float(), want[:, b].float(), rtol=2.0 ** -6, atol=2.0 ** -6)
                assert torch.equal(torch.isneginf(gl[:, b]), torch.isneginf(wl[:, b]))
            else:
                assert (got[:, b] == 3.0).all() and (gl[:, b] == 7.0).all()


@pytest.mark.parametrize("max_pages", [40, 300])
@pytest.mark.parametrize("group,T", [(4, 1), (16, 4)])
def test_a_scale_of_zero_is_the_mean(group, T, max_pages):
    p = problem([60, 0, 300, 2], group, 1, 128, 16, T, BF, False, 51, max_pages=max_pages)
    o, lse = call(p, 0.0)
    check_attention(o, lse, reference(p, 0.0), 128, 4 * 300, BF)


@pytest.mark.parametrize("group,T", [(4, 1), (16, 4)])
def test_the_same_page_in_two_tables(group, T):
    """Shared prefixes: two sequences that read the same pages, and one that reads a page twice."""
    p = problem([640, 700, 64], group, 1, 64, 64, T, BF, False, 52, max_pages=60)
    p["table"][1, :9] = p["table"][0, :9]
    p["table"][0, 5] = p["table"][0, 4]
    verify(p)


def test_joined_results_repeat_on_a_graph():
    """A captured call gives the eager result again and again, lengths and tables read anew each time."""
    from hybrid_decode_replay_amd import binding as rb
    p = problem([9000, 50, 1700], 16, 2, 128, 64, 2, BF, False, 53, max_pages=160)
    c = lambda n: p[n].cuda()  # noqa: E731
    q, K, V, table, end = c("q"), c("K"), c("V"), c("table"), c("end")
    ws = torch.zeros(rb.kv_attention_workspace(p["layer"], 3, ntok=2), dtype=torch.uint8, device="cuda")
    o = torch.zeros((2, 3, 16, 128), dtype=BF, device="cuda")
    run = lambda: rb.kv_attention(p["layer"], q, K, V, table, end, ntok=2, ws=ws, o=o)  # noqa: E731
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        run()
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for lens in ([9000, 50, 1700], [3, 4000, 0], [0, 0, 0], [9000, 50, 1700]):
        lens = [min(n, m) for n, m in zip(lens, [9000, 50, 1700])]
        end.copy_(torch.tensor(lens, dtype=torch.int32))
        run()
        want = o.clone()
        o.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)


@pytest.mark.parametrize("group,T,D", [(2, 1, 64), (13, 5, 64), (13, 5, 256)])
def test_the_largest_batch(group, T, D):
    """4096 sequences: every seventh holds something; and once with all but one idle."""
    lens = [(b * 5) % 33 if b % 7 == 0 else 0 for b in range(4096)]
    p = problem(lens, group, 1, D, 16, T, BF, False, 95, max_pages=161)
    verify(p)
    want, wl = call(p, D ** -0.5)
    active = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    active[2800] = 1
    got, gl = call(p, D ** -0.5, active=active, o=torch.full_like(want, 3.0))
    assert torch.equal(got[:, 2800], want[:, 2800]) and torch.equal(gl[:, 2800], wl[:, 2800])
    assert (got[:, :2800] == 3.0).all() and (got[:, 2801:] == 3.0).all()


@pytest.mark.parametrize("max_pages", [20, 200])
@pytest.mark.parametrize("group,T", [(4, 1), (16, 4)])
def test_infinite_scores(group, T, max_pages):
    """A key whose score is -inf weighs nothing, also where whole blocks of them come first; one of
    +inf leaves no number, in the rows that see it."""
    p = problem([300, 40], group, 1, 128, 16, T, BF, False, 61, max_pages=max_pages)
    p["q"].view(-1, 128)[:, 9] = -1.0
    rows = p["table"][0, :19].long()
    gone = list(range(0, 200)) + [250]
    K = p["K"].clone()
    for j in gone:
        K[rows[j // 16], 0, j % 16, 9] = float("inf")
    got, lse = call(dict(p, K=K), 0.09)
    # the same positions with keys that weigh 2^-200 or less: 0.09 * 3e4 is 2700 below the others
    far = p["K"].clone()
    for j in gone:
        far[rows[j // 16], 0, j % 16, 9] = 3e4
    ro, rl, top, a = reference(dict(p, K=far), 0.09)
    clean = reference(p, 0.09)
    check_attention(got, lse, (ro, rl, clean[2], a), 128, 4 * 300, BF)
    K = p["K"].clone()
    K[rows[298 // 16], 0, 298 % 16, 9] = float("-inf")
    got, _ = call(dict(p, K=K), 0.09)
    want, _ = call(p, 0.09)
    first = max(0, T - 2)                                   # position 298 is seen by the last two drafts
    assert torch.isnan(got[first:, 0]).all() and torch.equal(got[:, 1], want[:, 1])
    assert torch.equal(got[:first, 0], want[:first, 0])


@pytest.mark.parametrize("max_pages", [160, 200])
@pytest.mark.parametrize("B,Hkv,group,T,D", [(700, 3, 2, 1, 64), (250, 9, 2, 2, 64), (1024, 2, 12, 4, 64), (70, 8, 3, 1, 256)])
def test_the_longest_first(B, Hkv, group, T, D, max_pages):
    """More ranges than workgroups, none longer than an even share: a workgroup each, by length."""
    r = rng(B, D)
    lens = [int(n) for n in r.integers(0, 300 if B < 1000 else 100, B)]
    lens[-1], lens[0] = 0, 3
    p = problem(lens, Hkv * group, Hkv, D, 16, T, BF, False, 97, max_pages=max_pages)
    verify(p)
    want, wl = call(p, D ** -0.5)
    on = r.integers(0, 5, B) > 0
    active = torch.from_numpy(on.astype(np.uint8)).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, gl = call(p, D ** -0.5, active=active, o=torch.full_like(want, 3.0), err=err)
    on = torch.from_numpy(on).cuda()
    assert torch.equal(got[:, on], want[:, on]) and torch.equal(gl[:, on], wl[:, on]) and int(err) == 0
    assert (got[:, ~on] == 3.0).all() and (gl[:, ~on] == 7.0).all()
    p["end"][B // 2] = 2 ** 31 - 1
    p["end"][B // 3] = -5
    call(p, D ** -0.5, err=err)
    assert int(err) == 4


def test_even_and_uneven_lengths_on_one_graph():
    """The cut follows the lengths that a replay finds: even ones, one long one, none."""
    from hybrid_decode_replay_amd import binding as rb
    full = [60] * 299 + [2900]
    p = problem(full, 4, 2, 64, 16, 1, BF, False, 54, max_pages=190)
    c = lambda n: p[n].cuda()  # noqa: E731
    q, K, V, table, end = c("q"), c("K"), c("V"), c("table"), c("end")
    ws = torch.zeros(rb.kv_attention_workspace(p["layer"], 300), dtype=torch.uint8, device="cuda")
    o = torch.zeros((1, 300, 4, 64), dtype=BF, device="cuda")
    run = lambda: rb.kv_attention(p["layer"], q, K, V, table, end, ws=ws, o=o)  # noqa: E731
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        run()
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for last in (2900, 60, 0, 2900, 61):
        end.copy_(torch.tensor([60] * 299 + [last], dtype=torch.int32))
        o.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        p["end"] = end.cpu()
        ref = reference(p, 64 ** -0.5)
        check_attention(o, None, ref, 64, 2900, BF)


def test_windows_past_every_position_are_none():
    import sys

    from hybrid_decode_replay_amd import binding as rb
    p = problem([300, 41], 4, 2, 64, 16, 2, BF, False, 98)
    want, wl = call(p, 0.125)
    for window in (20 * 16, 2 ** 31 - 1, 2 ** 32 + 5, sys.maxsize):
        got, gl = call(p, 0.125, window)
        assert torch.equal(got, want) and torch.equal(gl, wl)
    for window in (-1, -2 ** 32 + 5):
        with pytest.raises(rb.ReplayError) as e:
            call(p, 0.125, window)
        assert e.value.status == rb.ERR_ARG
