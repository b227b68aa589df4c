"""replay_gdn_prefill against the recurrence in 64 bits: lengths, head layouts, states, strides, gates at their limits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mixer_cases import HALF, TINY, gdn_inputs, gdn_plain, gen, normal  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def rb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from hybrid_decode_replay_amd import binding
    return binding


def starts_of(lens, first=0):
    return torch.tensor([first] + [first + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)


def check(o, S, q, k, v, a, b, starts, G, scale, S0, which=None):
    starts = starts.tolist()
    H = a.shape[1]
    for i, (lo, hi) in enumerate(zip(starts, starts[1:])):
        if which is not None and i not in which:
            continue
        wo, wS, bo, bS = gdn_plain(q[lo:hi], k[lo:hi], v[lo:hi], a[lo:hi], b[lo:hi], G, scale, None if S0 is None else S0[i])
        off = (S[i].cpu().double() - wS).norm(dim=-1)
        bound = bS + 2.0 ** -24 * wS.norm(dim=-1) + 2.0 ** -140
        assert (off <= bound).all(), (i, hi - lo, float((off / bound).max()))
        if hi > lo:
            got = o[lo:hi].cpu().double().view(hi - lo, H, -1)
            bound = bo + HALF[o.dtype] * (wo.abs() + bo) + TINY[o.dtype]
            assert ((got - wo).abs() <= bound).all(), (i, hi - lo, float(((got - wo).abs() / bound).max()))


def run(rb, lens, H, G, DK, DV, dtype, seed=0, state=True, scale=None, **kw):
    rows = sum(lens)
    scale = DK ** -0.5 if scale is None else scale
    q, k, v, a, b = gdn_inputs(seed, rows, H, G, DK, DV, dtype, **kw)
    starts = starts_of(lens)
    S0 = normal(gen(seed, 5), len(lens), H, DV, DK, std=0.3) if state else None
    o, S = rb.gdn_prefill(q.cuda(), k.cuda(), v.cuda(), a.cuda(), b.cuda(), starts.cuda(), ngroups=G, scale=scale,
                          state=None if S0 is None else S0.cuda())
    check(o, S, q, k, v, a, b, starts, G, scale, S0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("DK", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("DV", [16, 48, 128, 256])
def test_dimensions(rb, DK, DV, dtype):
    run(rb, [1, 70, 0, 17], 2, 1, DK, DV, dtype, seed=DK + DV)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,G", [(1, 1), (3, 3), (4, 2), (6, 1), (5, 5)])
def test_heads(rb, H, G, dtype):
    run(rb, [33, 66], H, G, 64, 64, dtype, seed=H * 10 + G, state=H % 2 == 0)


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 193, 256])
@pytest.mark.parametrize("state", [False, True])
def test_lengths(rb, n, state):
    run(rb, [n], 2, 2, 128, 128, BF, seed=n, state=state)


@pytest.mark.parametrize("lens", [[5, 0, 0, 130, 1, 64, 63], [0, 0, 3], [200, 0], [1] * 20, [64, 128, 192]])
def test_ragged(rb, lens):
    run(rb, lens, 2, 1, 128, 64, BF, seed=len(lens))


@pytest.mark.parametrize("lens", [[40, 3, 0, 1, 2, 5, 0, 33], [1, 90, 0, 0, 2, 2], [33] + [0] * 9, [20, 11, 0, 2]])
def test_one_long_among_few(rb, lens):
    run(rb, lens, 3, 3, 128, 48, BF, seed=sum(lens))


@pytest.mark.parametrize("B,H,DK,DV", [(40, 2, 64, 48), (40, 32, 64, 48), (64, 16, 64, 64), (70, 16, 64, 16), (131, 16, 64, 16),
                                       (33, 32, 128, 48), (33, 32, 256, 16)])
def test_long_among_short(rb, B, H, DK, DV):
    """Lengths of 0 to 130 whose mean is below 64, also of more sequences and heads than start at a time."""
    g = gen(B)
    lens = [(0, 1, 7, 31, 32, 33, 34, 50, 64, 65, 100, 130)[int(i)] for i in torch.randint(0, 12, (B,), generator=g)]
    assert sum(lens) < 64 * B
    run(rb, lens, H, 1, DK, DV, BF, seed=B)


def test_a_long_prompt(rb):
    run(rb, [1500], 1, 1, 128, 128, BF, seed=4)


@pytest.mark.parametrize("DK", [64, 128])
def test_gates_at_their_limits(rb, DK):
    """alpha 0 forgets all, alpha 1 nothing; beta 0 writes nothing, beta 1 replaces; keys that are all alike."""
    for alpha, beta, common in [(1.0, 1.0, 0.5), (1.0, 0.5, 50.0), (1.0, 1.0, 50.0), (0.0, 0.7, 0.5), (0.5, 0.0, 0.5),
                                (1e-30, 0.9, 0.5), (0.999, 0.3, 5.0)]:
        run(rb, [150, 40], 2, 2, DK, 64, BF, seed=7, alpha=alpha, beta=beta, common=common)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_forgetting_in_the_middle(rb, dtype):
    """Zeros among the alphas: what lies before leaves nothing behind."""
    H, DK, DV, n = 2, 128, 64, 200
    q, k, v, a, b = gdn_inputs(11, n, H, H, DK, DV, dtype)
    a[[0, 5, 63, 64, 100, 130]] = 0
    a[70:90] = 1e-20
    starts, S0 = starts_of([n]), normal(gen(1), 1, H, DV, DK)
    o, S = rb.gdn_prefill(q.cuda(), k.cuda(), v.cuda(), a.cuda(), b.cuda(), starts.cuda(), state=S0.cuda())
    check(o, S, q, k, v, a, b, starts, H, 1.0, S0)
    o2, S2 = rb.gdn_prefill(*(t[100:].contiguous().cuda() for t in (q, k, v, a, b)), starts_of([n - 100]).cuda())
    check(o2, S2, q[100:], k[100:], v[100:], a[100:], b[100:], starts_of([n - 100]), H, 1.0, None)


def test_rows_of_a_fused_projection(rb):
    """q, k and v as slices of one tensor's rows."""
    H, G, DK, DV, lens = 4, 2, 64, 128, [70, 9]
    rows = sum(lens)
    q, k, v, a, b = gdn_inputs(2, rows, H, G, DK, DV, BF)
    fused = torch.cat([q, torch.full((rows, 8), 9.0, dtype=BF), k, v], 1).cuda()
    wq = G * DK
    o, S = rb.gdn_prefill(fused[:, :wq], fused[:, wq + 8:2 * wq + 8], fused[:, 2 * wq + 8:], a.cuda(), b.cuda(),
                          starts_of(lens).cuda(), ngroups=G, scale=0.3)
    check(o, S, q, k, v, a, b, starts_of(lens), G, 0.3, None)


@pytest.mark.parametrize("dtype,DK", [(BF, 128), (BF, 32), (F32, 64)])
def test_rows_of_no_sequence(rb, dtype, DK):
    """A padded batch: rows before the first sequence and behind the last are not read (NaN there) and not written."""
    H, DV, lens = 2, 64, [40, 0, 81]
    n, pad = sum(lens), 29
    q, k, v, a, b = gdn_inputs(3, n, H, H, DK, DV, dtype)
    grown = [torch.cat([torch.full((pad, t.shape[1]), float("nan"), dtype=t.dtype), t,
                        torch.full((pad, t.shape[1]), float("nan"), dtype=t.dtype)]).cuda() for t in (q, k, v, a, b)]
    o = torch.full((n + 2 * pad, H * DV), 5.0, dtype=dtype, device="cuda")
    _, S = rb.gdn_prefill(*grown, starts_of(lens, pad).cuda(), o=o)
    assert (o[:pad] == 5).all() and (o[n + pad:] == 5).all()
    check(o[pad:n + pad], S, q, k, v, a, b, starts_of(lens), H, 1.0, None)


@pytest.mark.parametrize("B,H", [(1, 2), (2, 2), (70, 2), (1, 1024), (70, 16)])
@pytest.mark.parametrize("n", [1, 20, 32, 33, 40])
def test_few_of_the_rows(rb, n, B, H):
    """One sequence of n tokens in the middle of many more rows, alone or beside empty ones."""
    DK, DV, rows = 64, 32, 60 * B
    q, k, v, a, b = gdn_inputs(13, rows, H, H, DK, DV, BF)
    starts = torch.full((B + 1,), 20 + n, dtype=torch.int32)
    starts[:B // 2 + 1] = 20
    S0 = normal(gen(4), B, H, DV, DK)
    state = S0.cuda()
    o, S = rb.gdn_prefill(*(t.cuda() for t in (q, k, v, a, b)), starts.cuda(), state=state, state_out=state)
    check(o, S, q, k, v, a, b, starts, H, 1.0, S0)
    assert (o[:20] == 0).all() and (o[20 + n:] == 0).all()


@pytest.mark.parametrize("DK", [32, 128])
def test_starts_that_lie(rb, DK):
    """Entries outside the rows are taken into them; a sequence that ends before it starts has no rows."""
    H, DV, n = 2, 32, 100
    q, k, v, a, b = gdn_inputs(5, n, H, H, DK, DV, BF)
    S0 = normal(gen(2), 2, H, DV, DK)
    for starts, seen in (([-7, 60, 40], [0, 60, 60]), ([1 << 30, 50, (1 << 31) - 1], [50, 50, 100]), ([-(1 << 31), -5, 200], [0, 0, 100])):
        o, S = rb.gdn_prefill(*(t.cuda() for t in (q, k, v, a, b)), torch.tensor(starts, dtype=torch.int32).cuda(),
                              state=S0.cuda())
        check(o, S, q, k, v, a, b, torch.tensor(seen), H, 1.0, S0)
        rest = torch.ones(n, dtype=torch.bool)
        rest[seen[0]:seen[2]] = False
        assert (o[rest.cuda()] == 0).all()


@pytest.mark.parametrize("dtype,DK", [(BF, 128), (F32, 128), (BF, 64)])
def test_in_pieces_and_in_place(rb, dtype, DK):
    """A prompt in three calls, the state updated in place, is the prompt."""
    H, DV, n = 2, 128, 210
    q, k, v, a, b = gdn_inputs(6, n, H, H, DK, DV, dtype)
    state = torch.zeros((1, H, DV, DK), device="cuda")
    outs = []
    for lo, hi in ((0, 77), (77, 78), (78, n)):
        o, S = rb.gdn_prefill(*(t[lo:hi].cuda() for t in (q, k, v, a, b)), starts_of([hi - lo]).cuda(), state=state, state_out=state)
        assert S is state
        outs.append(o)
    check(torch.cat(outs), state, q, k, v, a, b, starts_of([n]), H, 1.0, None)


def test_no_rows_at_all(rb):
    S0 = normal(gen(4), 2, 3, 32, 64)
    z = lambda w, t=BF: torch.empty((0, w), dtype=t, device="cuda")  # noqa: E731
    o, S = rb.gdn_prefill(z(192), z(192), z(96), z(3, F32), z(3, F32), torch.zeros(3, dtype=torch.int32, device="cuda"), state=S0.cuda())
    assert o.shape == (0, 96) and torch.equal(S.cpu(), S0)
    _, S = rb.gdn_prefill(z(192), z(192), z(96), z(3, F32), z(3, F32), torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert (S == 0).all()


@pytest.mark.parametrize("dtype,DK", [(BF, 128), (F32, 32)])
def test_a_graph_and_another_stream(rb, dtype, DK):
    """Captured once; lengths, inputs and states of later replays differ."""
    H, DV, n = 2, 64, 150
    args = [t.cuda() for t in gdn_inputs(8, n, H, H, DK, DV, dtype)]
    starts, S0 = starts_of([100, 50]).cuda(), torch.zeros((2, H, DV, DK), device="cuda")
    o, S = torch.zeros((n, H * DV), dtype=dtype, device="cuda"), torch.zeros_like(S0)
    ws = torch.empty(max(1, rb.gdn_prefill_workspace(*args, starts)), dtype=torch.uint8, device="cuda")
    call = lambda o, S, ws=None: rb.gdn_prefill(*args, starts, state=S0, o=o, state_out=S, ws=ws)  # noqa: E731
    want, wS = (t.clone() for t in call(o, S))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o.zero_()
        call(o, S, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want) and torch.equal(S, wS)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(o, S, ws)
    for i, lens in enumerate(([150, 0], [1, 149], [64, 86])):
        for t, new in zip(args, gdn_inputs(20 + i, n, H, H, DK, DV, dtype)):
            t.copy_(new)
        starts.copy_(starts_of(lens))
        S0.copy_(normal(gen(i), 2, H, DV, DK))
        graph.replay()
        eo, eS = call(torch.zeros_like(o), torch.zeros_like(S))
        assert torch.equal(o, eo) and torch.equal(S, eS)


@pytest.mark.parametrize("DK,DV,n", [(64, 48, 100), (128, 64, 70), (128, 128, 130), (256, 32, 90), (128, 96, 30), (32, 32, 40)])
@pytest.mark.parametrize("what", ["q", "k", "v", "alpha", "beta", "state"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_a_token_must_not_see(rb, DK, DV, n, what, value):
    """An infinity or NaN at a token (or in a row of the state) reaches that token's outputs and what follows them in its head,
    and nothing before it, beside it or in the other sequence of the call."""
    H, j, in_place = 2, n * 2 // 3, what != "state"
    q, k, v, a, b = gdn_inputs(21, 2 * n, H, H, DK, DV, BF)
    S0 = normal(gen(8), 2, H, DV, DK, std=0.3)
    broken = [t.clone() for t in (q, k, v, a, b, S0)]
    at = {"q": (0, j, DK + 5), "k": (1, j, DK + 5), "v": (2, j, DV + 5), "alpha": (3, j, 1), "beta": (4, j, 1)}
    if what == "state":
        broken[5][0, 1, 5, 3] = value
    else:
        i, row, col = at[what]
        broken[i][row, col] = value
    args, state = [t.cuda() for t in broken[:5]], broken[5].cuda()
    starts = starts_of([n, n])
    o, S = rb.gdn_prefill(*args, starts.cuda(), state=state, state_out=state if in_place else None)
    check(o, S, q, k, v, a, b, starts, H, 1.0, S0, which=[1])
    o = o.cpu().double().view(2 * n, H, DV)
    for h in range(H):
        take = [t[:n].view(n, H, -1)[:, h] for t in (q, k, v)] + [t[:n, h:h + 1] for t in (a, b)]
        wo, wS, bo, bS = gdn_plain(*take, 1, 1.0, S0[0, h:h + 1])
        good = (o[:n, h] - wo[:, 0]).abs() <= bo[:, 0] + HALF[BF] * (wo[:, 0].abs() + bo[:, 0])
        fine = (S[0, h].cpu().double() - wS[0]).norm(dim=-1) <= bS[0] + 2.0 ** -24 * wS[0].norm(dim=-1)
        if h == 0:
            assert good.all() and fine.all()
            continue
        if what in ("v", "state"):                       # one column of the head
            rest = torch.ones(DV, dtype=torch.bool)
            rest[5] = False
            assert good[:, rest].all() and fine[rest].all()
            since = 0 if what == "state" else j
            assert good[:since, 5].all() and not o[since:n, 1, 5].isfinite().any() and not S[0, 1, 5].isfinite().all()
        elif what == "q":
            rest = torch.arange(n) != j
            assert good[rest].all() and fine.all() and not o[j, 1].isfinite().any()
        else:
            assert good[:j].all() and not o[j:n, 1].isfinite().any() and not S[0, 1].isfinite().all(-1).any()


@pytest.mark.parametrize("DK", [64, 128, 256])
@pytest.mark.parametrize("lens,H,DV", [([20], 2, 32), ([32], 1, 96), ([70], 2, 32), ([100, 30], 2, 48), ([66] * 4 + [0], 32, 80),
                                       ([40] + [9] * 39, 32, 48)])
def test_scores_that_overflow(rb, DK, lens, H, DV):
    """q and k whose products pass the fp32 range, over updates so small that every output and state is an ordinary number:
    short sequences alone, chunks with one and two strips a workgroup, long sequences among short ones."""
    rows = sum(lens)
    q, k, v, a, b = gdn_inputs(17, rows, H, 1, DK, DV, BF)
    q, k = (q.float() * 2.0 ** 100).to(BF), (k.float() * 2.0 ** 32).to(BF)
    v, b = (v.float() * 2.0 ** -34).to(BF), b * 2.0 ** -64
    starts = starts_of(lens)
    o, S = rb.gdn_prefill(*(t.cuda() for t in (q, k, v, a, b)), starts.cuda(), ngroups=1)
    assert o.isfinite().all() and S.isfinite().all()
    check(o, S, q, k, v, a, b, starts, 1, 1.0, None)


@pytest.mark.parametrize("DK,DV", [(64, 48), (128, 64), (256, 32)])
@pytest.mark.parametrize("n,at", [(4, (0, 1, 2, 3)), (20, (3, 9, 15, 19)), (32, (0, 1, 30, 31)), (40, (2, 5, 37, 39)),
                                  (64, (0, 31, 32, 63)), (150, (1, 60, 64, 149))])
def test_strong_decays_keep_their_bits(rb, n, at, DK, DV):
    """Four tokens that leave some 2^-25 of the state each, the others all, and nothing written: the state is its start times
    the alphas.  In chunks the product comes from logarithms.  A token's is off by at most 2^-24 (an fp32 logarithm below 1/2,
    two steps; the exponent is exact, and that of 1 is 0), which is ln 2 2^-24 of the product; each chunk adds the rounding of
    the power's part (ln 2 2^-25), the power (one step, 2^-23) and the state's product (2^-24)."""
    H = 8
    q, k, v, a, b = gdn_inputs(n, n, H, H, DK, DV, BF, alpha=1.0, beta=0.0)
    a[list(at)] = torch.exp2(-20 - 10 * torch.rand((4, H), generator=gen(n, 3)))
    S0 = normal(gen(n, 4), 1, H, DV, DK)
    o, S = rb.gdn_prefill(*(t.cuda() for t in (q, k, v, a, b)), starts_of([n]).cuda(), state=S0.cuda())
    want = S0.double() * a.double().prod(0)[:, None, None]
    bound = (4 * 0.694 + (n + 63) // 64 * (0.347 + 2 + 1)) * 2.0 ** -24
    off = (S.cpu().double() - want).abs() / want.abs()
    assert (off <= bound).all(), float(off.max()) / bound


WAYS = [([30], 2, 48), ([32], 1, 16), ([64], 2, 48), ([150, 7], 2, 64), ([33], 1, 16), ([70, 0, 65, 100, 64], 32, 80),
        ([40] + [9] * 39, 32, 48)]


def whole_numbers(lens, H, DK, DV, size, seed):
    """Keys and queries of one channel each (half the queries are their token's key), whole numbers up to `size` in v and
    some 2^23 in the states: all that is formed of them is a whole number of at most 24 bits."""
    rows, g = sum(lens), gen(seed, DK, DV, H)
    hot = lambda i: torch.zeros((rows, H, DK)).scatter_(2, i[..., None], 1.0).flatten(1).to(BF)  # noqa: E731
    ki = torch.randint(0, DK, (rows, H), generator=g)
    qi = torch.where(torch.rand((rows, H), generator=g) < 0.5, ki, torch.randint(0, DK, (rows, H), generator=g))
    v = torch.randint(-size, size + 1, (rows, H * DV), generator=g).to(BF)
    S0 = torch.randint(-2 ** 23 + 1024, 2 ** 23 - 1024, (len(lens), H, DV, DK), generator=g).float()
    return hot(qi), hot(ki), v, S0


def check_exact(rb, lens, H, q, k, v, a, b, scale, S0):
    starts = starts_of(lens)
    o, S = rb.gdn_prefill(*(t.cuda() for t in (q, k, v, a, b)), starts.cuda(), scale=scale, state=S0.cuda())
    o, S = o.cpu(), S.cpu()
    for i, (lo, hi) in enumerate(zip(starts.tolist(), starts.tolist()[1:])):
        T = S0[i].double().clone()
        for t in range(lo, hi):
            kt, qt, vt = (x[t].double().view(H, -1) for x in (k, q, v))
            T = T * a[t, :, None, None].double()
            u = b[t, :, None].double() * (vt - (T @ kt[..., None])[..., 0])
            T = T + u[..., None] * kt[:, None]
            want = (scale * (T @ qt[..., None])[..., 0]).float()
            assert torch.equal(o[t].view(H, -1), want.to(BF)), (i, t - lo)
        assert torch.equal(S[i].double(), T), i


@pytest.mark.parametrize("DK", [64, 128, 256])
@pytest.mark.parametrize("lens,H,DV", WAYS)
def test_whole_numbers(rb, DK, lens, H, DV):
    """Small values take the place of 24-bit ones: every step is exact in fp32, so states and outputs are, in chunks too.
    (Of S and U in 16 bits, an output that is v - (24 bits) + (24 bits) would be off by up to 2^7.)"""
    q, k, v, S0 = whole_numbers(lens, H, DK, DV, 255, 1)
    a = torch.ones((sum(lens), H))
    check_exact(rb, lens, H, q, k, v, a, torch.ones_like(a), 1.0, S0)


@pytest.mark.parametrize("DK", [64, 128, 256])
@pytest.mark.parametrize("lens,H,DV", WAYS)
def test_factors_of_many_bits(rb, DK, lens, H, DV):
    """beta, then scale, of 1 + 2^-9 + 2^-20 (three terms of eight bits) on numbers of three bits: the triangle's inverse and
    the masked scores hold 24 bits."""
    rows, g = sum(lens), gen(5, DK)
    order = torch.stack([torch.randperm(64, generator=g) for _ in range(H)], 1)         # no key twice in a chunk
    since = torch.cat([torch.arange(n) % 64 for n in lens])
    hot = torch.zeros((rows, H, DK)).scatter_(2, order[since][..., None], 1.0).flatten(1).to(BF)
    S0 = torch.randint(0, 4, (len(lens), H, DV, DK), generator=g).float()
    v = torch.randint(0, 4, (rows, H * DV), generator=g).to(BF)
    a, c = torch.ones((rows, H)), 1 + 2.0 ** -9 + 2.0 ** -20
    if max(lens) <= 64:
        check_exact(rb, lens, H, hot, hot, v, a, c * a, 1.0, S0)
    # (what replaces 5 2^10 is 0: scale s - scale s, each of 24 bits)
    check_exact(rb, lens, H, hot, hot, torch.zeros_like(v), a, a, c, 5 * 2.0 ** 10 * S0.clamp(max=1))


def way(rb, lens, H, DK, DV):
    """Which launches a call takes: "short", "chunks" or "mixed", and whether a workgroup of the chunks has two strips.  From
    the workspace, which counts the sequences that the chunks take at most (where that is all of them in either case: a mean of
    33 tokens and more: by the host's rule, a mean below 64 of 1024 sequence-heads and more)."""
    def units(rows, nseq):
        z = lambda w, t=BF: torch.empty((rows, w), dtype=t, device="cuda")  # noqa: E731
        return rb.gdn_prefill_workspace(z(H * DK), z(H * DK), z(H * DV), z(H, F32), z(H, F32),
                                        torch.empty(nseq + 1, dtype=torch.int32, device="cuda"))
    rows, nseq = sum(lens), len(lens)
    need = units(rows, nseq)
    if need == 0:
        return "short", False
    most = need * 2 // units(64, 1) - rows // 64
    few = min(nseq, rows // 33)
    assert most in (few, nseq)
    mixed = most < nseq if few < nseq else rows < 64 * nseq and nseq * H >= 1024
    return "mixed" if mixed else "chunks", DK < 256 and most * H * (DV // 16) > 512


@pytest.mark.parametrize("lens,H,G,DV", [([70, 0, 130, 64, 90], 32, 16, 64), ([100, 65, 33, 0, 200], 36, 9, 48),
                                         ([40, 90, 0, 64, 129, 100, 63], 15, 5, 80), ([30] * 30 + [0, 100, 33, 65, 1, 32] * 6, 2, 1, 64)])
@pytest.mark.parametrize("DK", [64, 128])
def test_two_strips_a_workgroup(rb, DK, lens, H, G, DV):
    """Batches of ordinary prompts: two strips a workgroup (the last one's alone where they are odd), the longest first up to
    64 sequences, heads spread over the chip or not."""
    assert way(rb, lens, H, DK, DV) == ("chunks", True)
    run(rb, lens, H, G, DK, DV, BF, seed=len(lens))


BAD = [([15, 15], 2, 96, "short", False), ([32], 2, 48, "short", False), ([9, 1, 20], 2, 256, "short", False),
       ([70, 0, 80, 66], 4, 48, "chunks", False), ([70, 0, 130, 64, 90], 44, 48, "chunks", True),
       ([9] * 38 + [40, 100], 32, 48, "mixed", True)]


@pytest.mark.parametrize("lens,H,DV,by,two", BAD)
@pytest.mark.parametrize("DK", [64, 128, 256])
@pytest.mark.parametrize("what", ["q", "k", "v", "alpha", "state"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_values_in_every_way(rb, DK, lens, H, DV, by, two, what, value):
    """An infinity or NaN in one head of the longest sequence (and of the shortest with rows, in a mixed call), states in place:
    what follows it in its head, and nothing else."""
    assert way(rb, lens, H, DK, DV) == (by, two and DK < 256)
    rows, starts = sum(lens), starts_of(lens)
    q, k, v, a, b = gdn_inputs(31, rows, H, H, DK, DV, BF)
    S0 = normal(gen(9), len(lens), H, DV, DK, std=0.3)
    hit = {lens.index(max(lens))} | ({0} if by == "mixed" else set())
    h, ch = H - 1, DV - 11                     # (the last strip)
    args, state = [t.clone() for t in (q, k, v, a, b)], S0.clone()
    for i in hit:
        j = int(starts[i]) + lens[i] * 2 // 3
        if what == "state":
            state[i, h, ch, 3] = value
        else:
            args["q k v alpha".split().index(what)][j, {"q": h * DK + 5, "k": h * DK + 5, "v": h * DV + ch, "alpha": h}[what]] = value
    state = state.cuda()
    o, S = rb.gdn_prefill(*(t.cuda() for t in args), starts.cuda(), state=state, state_out=state)
    near = {i for x in hit for i in (x - 1, x + 1) if 0 <= i < len(lens)} - hit
    check(o, S, q, k, v, a, b, starts, H, 1.0, S0, which=near | ({len(lens) - 1} - hit))
    for i in hit:
        lo, n = int(starts[i]), lens[i]
        at = slice(lo, lo + n)
        for one in (0, h - 1, h):
            take = [t[at].view(n, H, -1)[:, one] for t in (q, k, v)] + [t[at, one:one + 1] for t in (a, b)]
            wo, wS, bo, bS = gdn_plain(*take, 1, 1.0, S0[i, one:one + 1])
            got = o[at].cpu().double().view(n, H, DV)[:, one]
            good = (got - wo[:, 0]).abs() <= bo[:, 0] + HALF[BF] * (wo[:, 0].abs() + bo[:, 0])
            fine = (S[i, one].cpu().double() - wS[0]).norm(dim=-1) <= bS[0] + 2.0 ** -24 * wS[0].norm(dim=-1)
            since = 0 if what == "state" else n * 2 // 3
            if one != h:
                assert good.all() and fine.all(), (i, one)
            elif what in ("v", "state"):
                rest = torch.arange(DV) != ch
                assert good[:, rest].all() and fine[rest].all() and good[:since].all(), i
                assert not got[since:, ch].isfinite().any() and not S[i, h, ch].isfinite().all()
            elif what == "q":
                rest = torch.arange(n) != since
                assert good[rest].all() and fine.all() and not got[since].isfinite().any(), i
            else:
                assert good[:since].all() and not got[since:].isfinite().any() and not S[i, h].isfinite().all(-1).any(), i


def test_workgroups_go_on_after_a_bad_value(rb):
    """More heads of long sequences than start at a time: a workgroup that has gone over its first head once more takes its
    next one as if nothing had been."""
    H, DK, DV, lens = 64, 64, 80, [40] * 14 + [3] * 10
    assert way(rb, lens, H, DK, DV) == ("mixed", True)
    q, k, v, a, b = gdn_inputs(37, sum(lens), H, 1, DK, DV, BF)
    starts, bad = starts_of(lens), v.clone()
    bad[[25, 65, 110], ::16] = float("nan")
    o, S = rb.gdn_prefill(*(t.cuda() for t in (q, k, bad, a, b)), starts.cuda(), ngroups=1)
    check(o, S, q, k, v, a, b, starts, 1, 1.0, None, which=[3, 9, 10, 11, 12, 13, 14, 23])
    hit = torch.arange(H * DV) % 16 == 0
    assert not o[25:40].cpu()[:, hit].isfinite().any() and o[:25].isfinite().all() and o[:120].cpu()[:, ~hit].isfinite().all()
