"""Paged decode attention against fp64, every element within a derived bound (tests/kv_cases.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cases import check_attention, f64, normal, paged, rng  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


BF, F16 = torch.bfloat16, torch.float16


def problem(lens, Hq, Hkv, D, page, T, io, fp8, seed, spare=3, std=1.0, max_pages=None):
    """Queries, pages with stale values everywhere, a table with a seeded order of pages."""
    from hybrid_decode_replay_amd import binding as rb
    need = sum(-(-n // page) for n in lens)
    npages = need + spare
    mp = max_pages or max(1, max(-(-n // page) for n in lens))
    table = paged(lens, page, npages, mp, seed)
    layer = rb.kv_layer(Hq, Hkv, D, npages, page, io_dtype=rb.BF16 if io == BF else rb.F16,
                        cache_dtype=rb.FP8_E4M3 if fp8 else None)
    shape = (npages, Hkv, page, D)
    kind = torch.float8_e4m3fn if fp8 else io
    K, V = normal(shape, torch.float32, seed + 1, 30.0 if fp8 else std), normal(shape, torch.float32, seed + 2, 30.0 if fp8 else 1.0)
    ks = vs = None
    if fp8:
        ks = torch.from_numpy(rng(seed, 5).uniform(0.02, 0.05, Hkv).astype(np.float32))
        vs = torch.from_numpy(rng(seed, 6).uniform(0.02, 0.05, Hkv).astype(np.float32))
    return dict(layer=layer, q=normal((T * len(lens), Hq * D), io, seed + 3, std), K=K.to(kind), V=V.to(kind),
                table=torch.from_numpy(table), end=torch.tensor(lens, dtype=torch.int32), ks=ks, vs=vs, T=T, io=io)


def reference(p, scale, window=0):
    from oracle import kv_oracle as ko
    B, Hq, D = len(p["end"]), p["layer"].nheads, p["layer"].head_dim
    K, V = f64(p["K"]), f64(p["V"])
    if p["ks"] is not None:
        K, V = K * f64(p["ks"])[None, :, None, None], V * f64(p["vs"])[None, :, None, None]
    return ko.attention(f64(p["q"]).reshape(p["T"], B, Hq, D), K, V, p["table"].numpy(), p["end"].numpy(), scale, window)


def call(p, scale, window=0, **kw):
    from hybrid_decode_replay_amd import binding as rb
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    B = len(p["end"])
    lse = torch.full((p["T"], B, p["layer"].nheads), 7.0, device="cuda")
    o = rb.kv_attention(p["layer"], c(p["q"]), c(p["K"]), c(p["V"]), c(p["table"]), c(p["end"]), ntok=p["T"], scale=scale,
                        window=window, k_scale=c(p["ks"]), v_scale=c(p["vs"]), lse=lse, **kw)
    torch.cuda.synchronize()
    return o, lse


def verify(p, scale=None, window=0):
    D = p["layer"].head_dim
    scale = D ** -0.5 if scale is None else scale
    o, lse = call(p, scale, window)
    w = check_attention(o, lse, reference(p, scale, window), D, int(p["end"].max()), p["io"])
    print(f"error {w:.3f} of the bound", flush=True)


@pytest.mark.parametrize("io,fp8", [(BF, False), (F16, False), (BF, True), (F16, True)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_types_and_widths(D, io, fp8):
    verify(problem([1, 15, 16, 17, 130, 333], 8, 2, D, 16, 1, io, fp8, 10 + D))


@pytest.mark.parametrize("lens", [[1], [0], [31], [32], [33], [127], [128], [129], [0, 1, 0, 2], [1000], [3, 700, 64]])
def test_lengths(lens):
    verify(problem(lens, 4, 1, 128, 32, 1, BF, False, 31 + sum(lens)))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (6, 2), (10, 2), (16, 1), (17, 1), (40, 2), (64, 1)])
def test_head_layouts(Hq, Hkv):
    verify(problem([200, 47], Hq, Hkv, 64, 16, 1, BF, False, Hq * 7 + Hkv))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(page):
    verify(problem([300, 513, 16], 8, 4, 128, page, 2, BF, False, page))


@pytest.mark.parametrize("T", [2, 3, 4, 7, 16])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (8, 1, 128), (16, 2, 256)])
def test_drafts(T, Hq, Hkv, D):
    """Also sequences shorter than the drafts: their first rows see nothing."""
    verify(problem([5, 40, 129, 257, 1, 0], Hq, Hkv, D, 16, T, BF, False, T * D))


@pytest.mark.parametrize("T", [16])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows(T, fp8, D):
    """More rows than one workgroup holds: 16 drafts of 10 queries."""
    verify(problem([161, 90], 10, 1, D, 32, T, F16, fp8, D + T))


@pytest.mark.parametrize("window", [1, 2, 16, 31, 100, 129, 5000])
@pytest.mark.parametrize("T", [1, 5])
def test_windows(window, T):
    verify(problem([300, 90, 33, 4], 8, 2, 64, 16, T, F16, False, window + T), window=window)


@pytest.mark.parametrize("io,fp8,D", [(BF, False, 128), (BF, True, 128), (F16, False, 64), (BF, False, 256)])
def test_split_and_joined(io, fp8, D):
    """One long sequence among short ones: its range is cut over many workgroups."""
    verify(problem([9001, 3, 0, 700], 4, 2, D, 64, 1, io, fp8, D + 99))


def test_large_scores_and_scale():
    """Scores of some hundreds: one weight dominates, references move."""
    verify(problem([513, 80], 8, 2, 128, 16, 2, BF, False, 5, std=4.0), scale=0.4)
    verify(problem([513, 80], 8, 2, 128, 16, 2, F16, False, 6, std=2.0), scale=-0.3)


def test_rising_scores():
    """Keys that grow with the position move the reference in every block."""
    p = problem([600], 4, 1, 128, 16, 1, BF, False, 8)
    at = p["table"][0].long()
    ramp = torch.linspace(0, 3, at.numel() * 16).view(-1, 1, 16, 1)
    K = p["K"].clone()
    K[at] = (p["q"].float().mean(0).view(4, 128)[0].view(1, 1, 1, 128) * ramp).to(BF)
    p["K"] = K
    verify(p)


def test_what_lies_in_masked_places():
    """NaN and infinities behind the end, in unused pages and outside the window change nothing."""
    p = problem([37, 161, 5], 8, 2, 128, 16, 3, BF, False, 12, spare=4)
    for window in (0, 24):
        want, wl = call(p, 0.09, window)
        K, V = p["K"].clone(), p["V"].clone()
        seen = torch.zeros(K.shape[0], 16, dtype=torch.bool)
        for b, n in enumerate(p["end"].tolist()):
            for j in range(max(0, n - 3 - window + 1) if window else 0, n):
                seen[p["table"][b, j // 16], j % 16] = True
        for x, bad in ((K, float("nan")), (V, float("inf"))):
            x.permute(0, 2, 1, 3)[~seen] = bad
        got, gl = call(dict(p, K=K, V=V), 0.09, window)
        assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_drafts_nan_stays_with_those_who_see_it(fp8):
    """The last draft's value is NaN (or its key): the drafts before it do not see it."""
    p = problem([70, 33], 4, 2, 64, 16, 3, F16, fp8, 21)
    want, _ = call(p, 0.125)
    for name in ("V", "K"):
        x = p[name].clone()
        b, n = 0, 70
        raw = x.view(torch.uint8) if fp8 else x
        raw[p["table"][b, (n - 1) // 16], :, (n - 1) % 16, 3] = 0x7f if fp8 else float("nan")
        got, _ = call(dict(p, **{name: x}), 0.125)
        assert torch.equal(got[:2], want[:2]) and torch.equal(got[2, 1], want[2, 1])
        assert torch.isnan(got[2, 0, :, 3]).all()
    x = p["V"].clone()
    raw = x.view(torch.uint8) if fp8 else x
    raw[p["table"][0, 68 // 16], :, 68 % 16, 5] = 0x7f if fp8 else float("nan")
    got, _ = call(dict(p, V=x), 0.125)
    assert torch.equal(got[0], want[0]) and torch.isnan(got[1:, 0, :, 5]).all()
    # the window's side: the first draft still sees it, the others do not
    want, _ = call(p, 0.125, 20)
    x = p["V"].clone()
    raw = x.view(torch.uint8) if fp8 else x
    j = 70 - 3 - 20 + 1
    raw[p["table"][0, j // 16], :, j % 16, 5] = 0x7f if fp8 else float("nan")
    got, _ = call(dict(p, V=x), 0.125, 20)
    assert torch.equal(got[1:], want[1:]) and torch.isnan(got[0, 0, :, 5]).all()


def test_infinite_and_nan_queries_stay_in_their_rows():
    p = problem([90, 50], 4, 2, 128, 16, 1, BF, False, 33)
    want, _ = call(p, 0.09)
    q = p["q"].clone()
    q[0, 128 * 1 + 7] = float("nan")
    got, _ = call(dict(p, q=q), 0.09)
    assert torch.isnan(got[0, 0, 1]).all()
    keep = torch.ones(2, 4, dtype=torch.bool)
    keep[0, 1] = False
    assert torch.equal(got[0][keep.cuda()], want[0][keep.cuda()])


def test_pages_outside_the_cache_are_masked():
    """Table entries of -1 or past the cache, and an end past the table: masked, with an error bit."""
    p = problem([100, 64, 47], 4, 2, 64, 16, 2, BF, False, 44, max_pages=8)
    p["table"][0, 2] = -1
    p["table"][1, :] = 10 ** 6
    p["end"][2] = 500                                       # pages 3.. of its row are -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = call(p, 0.125, err=err)
    check_attention(o, lse, reference(p, 0.125), 64, 128, BF)
    assert int(err) == 4
    assert (o[:, 1] == 0).all() and torch.isneginf(lse[:, 1]).all()


def test_idle_sequences_keep_their_outputs():
    p = problem([60, 0, 300, 8], 4, 2, 128, 16, 2, BF, False, 50)
    want, wl = call(p, 0.09)
    mark = torch.full_like(want, 3.0)
    active = torch.tensor([1, 0, 0, 1], dtype=torch.uint8, device="cuda")
    got, gl = call(p, 0.09, active=active, o=mark)
    for b in range(4):
        if active[b]:
            assert torch.equal(got[:, b], want[:, b]) and torch.equal(gl[:, b], wl[:, b])
        else:
            assert (got[:, b] == 3.0).all() and (gl[:, b] == 7.0).all()


def test_strided_queries_and_own_workspace():
    from hybrid_decode_replay_amd import binding as rb
    p = problem([60, 33], 8, 2, 64, 16, 1, BF, False, 60)
    want, _ = call(p, 0.125)
    wide = torch.zeros(2, 8 * 64 + 2 * 2 * 64, dtype=BF)
    wide[:, :8 * 64] = p["q"]
    ws = torch.full((rb.kv_attention_workspace(p["layer"], 2),), 255, dtype=torch.uint8, device="cuda")
    c = lambda t: t.cuda()  # noqa: E731
    got = rb.kv_attention(p["layer"], c(wide)[:, :8 * 64], c(p["K"]), c(p["V"]), c(p["table"]), c(p["end"]), scale=0.125,
                          ws=ws)
    assert torch.equal(got, want)


def test_many_sequences():
    r = rng(3)
    lens = [int(n) for n in r.integers(0, 90, 700)]
    verify(problem(lens, 2, 1, 64, 16, 1, BF, False, 70))


def test_results_repeat():
    p = problem([3000, 17, 900], 8, 2, 128, 16, 4, BF, False, 80)
    a, la = call(p, 0.09)
    for _ in range(3):
        b, lb = call(p, 0.09)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 values: pages at its far end."""
    from hybrid_decode_replay_amd import binding as rb
    Hkv, D, page = 8, 128, 256
    npages = (1 << 32) // (Hkv * D * page) + 9
    layer = rb.kv_layer(8, Hkv, D, npages, page)
    K = torch.empty((npages, Hkv, page, D), dtype=BF, device="cuda")
    V = torch.empty_like(K)
    g = torch.Generator(device="cuda").manual_seed(5)
    for x in (K, V):
        x[-2:] = torch.randn(x[-2:].shape, generator=g, device="cuda").to(BF)
    q = normal((1, 8 * D), BF, 4).cuda()
    table = torch.tensor([[npages - 1, npages - 2]], dtype=torch.int32, device="cuda")
    end = torch.tensor([300], dtype=torch.int32, device="cuda")
    far = rb.kv_attention(layer, q, K, V, table, end)
    small = rb.kv_layer(8, Hkv, D, 2, page)
    near = rb.kv_attention(small, q, K[-2:].flip(0).contiguous(), V[-2:].flip(0).contiguous(),
                           torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), end)
    assert torch.equal(far, near) and torch.isfinite(far).all()
