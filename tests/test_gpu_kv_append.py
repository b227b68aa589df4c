"""Rows into the paged cache: rotation against fp64 within derived bounds, copies to the bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cases import HALF, SUBNORMAL, f64, normal, rng  # noqa: E402

BF, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def setup(N, Hq, Hkv, D, page, io, fp8, rot, style, axes, seed, far=5000, idle=0.2):
    from hybrid_decode_replay_amd import binding as rb
    npages = -(-N // page) + 2
    layer = rb.kv_layer(Hq, Hkv, D, npages, page, io_dtype=rb.BF16 if io == BF else rb.F16,
                        cache_dtype=rb.FP8_E4M3 if fp8 else None, rot_dim=rot, rot_style=style)
    r = rng(seed, N)
    slots = r.permutation(npages * page)[:N].astype(np.int64)
    slots[r.random(N) < idle] = -1
    ks = vs = None
    if fp8:
        ks, vs = (torch.from_numpy(r.uniform(0.01, 0.05, Hkv).astype(np.float32)) for _ in range(2))
    return dict(layer=layer, x=normal((N, (Hq + 2 * Hkv) * D), io, seed), slots=torch.from_numpy(slots),
                pos=torch.from_numpy(r.integers(0, far, (axes, N)).astype(np.int32)), axes=axes, io=io, ks=ks, vs=vs,
                axis=torch.from_numpy(r.integers(0, axes, rot // 2).astype(np.uint8)),
                freq=torch.from_numpy((1e5 ** -r.random(rot // 2)).astype(np.float32)))


def call(p, with_q=True, **kw):
    from hybrid_decode_replay_amd import binding as rb
    l, c = p["layer"], (lambda t: None if t is None else t.cuda())
    K, V = rb.kv_cache(l)
    for t in (K, V):
        t.view(torch.uint8).fill_(0x55)
    x = c(p["x"])
    nq, nk = l.nheads * l.head_dim, l.nkv * l.head_dim
    q_out = torch.full((x.shape[0], nq), 9.0, dtype=p["io"], device="cuda") if with_q else None
    rb.kv_append(l, K, V, x[:, nq:nq + nk], x[:, nq + nk:], c(p["slots"]), q=x[:, :nq] if with_q else None, q_out=q_out,
                 **{**dict(pos=c(p["pos"]), freq=c(p["freq"]), axis=c(p["axis"]), k_scale=c(p["ks"]), v_scale=c(p["vs"])),
                    **kw})
    torch.cuda.synchronize()
    return q_out, K, V


def verify(p, q_out, K, V, axis=True):
    from oracle import kv_oracle as ko
    l, io = p["layer"], p["io"]
    Hq, Hkv, D, page, rot = l.nheads, l.nkv, l.head_dim, l.page_size, l.rot_dim
    N = p["x"].shape[0]
    x = f64(p["x"]).reshape(N, -1, D)
    turn = lambda h: ko.rotate(h, p["pos"].numpy(), p["freq"].numpy(),  # noqa: E731
                               p["axis"].numpy() if axis else None, rot, l.rot_style == 1)
    # what a pair's two values can lose: cos and sin are good to 3 2^-23, two products and their sum
    # are rounded to 2^-24 each
    size = np.abs(x).copy()
    i, j = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if l.rot_style == 1 else (np.arange(rot // 2), np.arange(rot // 2, rot))
    size[:, :, i] = size[:, :, j] = np.abs(x[:, :, i]) + np.abs(x[:, :, j])
    lost = 6 * 2.0 ** -23 * size
    lost[:, :, rot:] = 0
    live = (p["slots"] >= 0).numpy()
    if q_out is not None:
        ref = turn(x[:, :Hq])
        err = np.abs(f64(q_out).reshape(N, Hq, D) - ref)
        bound = HALF[io] * (np.abs(ref) + lost[:, :Hq]) + lost[:, :Hq] + SUBNORMAL[io]
        assert (err <= bound)[live].all()
        assert (f64(q_out)[~live] == 9.0).all()
    at = p["slots"].numpy()[live]
    for name, cache, heads, scale, slack in (("K", K, turn(x[:, Hq:Hq + Hkv]), p["ks"], lost[:, Hq:Hq + Hkv]),
                                             ("V", V, x[:, Hq + Hkv:], p["vs"], 0 * lost[:, :Hkv])):
        raw = cache.view(torch.uint8).cpu().numpy().reshape(l.npages, Hkv, page, -1).transpose(0, 2, 1, 3)
        raw = raw.reshape(l.npages * page, Hkv, -1)
        untouched = np.ones(l.npages * page, bool)
        untouched[at] = False
        assert (raw[untouched] == 0x55).all()
        got = f64(cache).transpose(0, 2, 1, 3).reshape(l.npages * page, Hkv, D)[at]
        ref, slack = heads[live], np.broadcast_to(slack[live], heads[live].shape)
        if scale is None:
            bound = HALF[io] * (np.abs(ref) + slack) + slack + SUBNORMAL[io]
            assert (np.abs(got - ref) <= (bound if name == "K" and rot else 0)).all()
        else:
            s = f64(scale)[:, None]
            ref, slack = ref / s, slack / s + 2.0 ** -24 * np.abs(ref / s)
            if name == "V" or rot == 0:      # codes of the fp32 quotient, exactly
                quotient = heads[live].astype(np.float32) / scale.numpy()[:, None]
                assert (raw[at] == ko.to_e4m3(quotient.astype(np.float64))).all()
            else:
                lim = np.clip(ref, -448, 448)
                assert (np.abs(got - lim) <= 2.0 ** -4 * (np.abs(lim) + slack) + slack + 2.0 ** -10).all()


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("io,fp8", [(BF, False), (F16, False), (BF, True), (F16, True)])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 64), (256, 256), (128, 0)])
def test_types_widths_styles(D, rot, io, fp8, style):
    p = setup(37, 6, 2, D, 16, io, fp8, rot, style, 1, D + rot)
    verify(p, *call(p))


@pytest.mark.parametrize("axes", [1, 2, 3, 8])
@pytest.mark.parametrize("style", [0, 1])
def test_axes(axes, style):
    p = setup(50, 4, 1, 128, 32, F16, False, 96, style, axes, axes)
    verify(p, *call(p))
    p["axis"][::3] = 200                                        # no such axis: those pairs do not turn
    verify(p, *call(p))


@pytest.mark.parametrize("N", [1, 2, 255, 1024, 1025, 1027, 2310])
def test_row_counts(N):
    p = setup(N, 2, 1, 64, 64, BF, False, 64, 0, 2, N)
    verify(p, *call(p))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 7), (10, 2), (64, 1)])
def test_head_layouts(Hq, Hkv):
    p = setup(20, Hq, Hkv, 64, 256, BF, False, 32, 0, 1, Hq)
    verify(p, *call(p))


def test_far_positions():
    """A million positions: the angle is formed in 64 bits."""
    p = setup(64, 4, 2, 128, 16, F16, False, 128, 0, 1, 3, far=10 ** 6)
    p["pos"][0, :4] = torch.tensor([10 ** 6, 999983, 0, -777777], dtype=torch.int32)
    p["freq"][:3] = 1.0
    verify(p, *call(p))


def test_without_queries_and_without_axis_table():
    p = setup(33, 4, 2, 64, 16, BF, False, 64, 0, 1, 9)
    p["axis"].zero_()
    _, K, V = call(p, with_q=False, axis=None)
    verify(p, None, K, V, axis=False)
    verify(p, *call(p, axis=None, pos=p["pos"][0].cuda()), axis=False)


def test_slots_outside_the_cache_are_skipped():
    p = setup(10, 2, 1, 64, 16, BF, False, 0, 0, 1, 4, idle=0.0)
    p["slots"][3] = p["layer"].npages * 16
    p["slots"][7] = 1 << 40
    p["slots"][8] = -(1 << 40)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(p, err=err)
    assert int(err) == 4
    p["slots"][[3, 7]] = -1
    verify(p, *out)
    err.zero_()
    call(p, err=err)
    assert int(err) == 0


def test_no_rows():
    p = setup(0, 2, 1, 64, 16, BF, False, 64, 0, 1, 4)
    q_out, K, V = call(p)
    assert q_out.shape == (0, 128) and (K.view(torch.uint8) == 0x55).all()


def test_special_values():
    """Infinities, NaN, signed zeros and E4M3's border values arrive as they should."""
    from oracle import kv_oracle as ko
    vals = [float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 448.0, 464.0, 480.0, -1e4, 2.0 ** -9, 2.0 ** -10,
            3 * 2.0 ** -10, 2.0 ** -24, 17.0, 19.0, 1.0]
    for io in (BF, F16):
        p = setup(4, 1, 1, 64, 16, io, True, 0, 0, 1, 5, idle=0.0)
        p["x"][:, 64:] = torch.tensor(vals * 8, dtype=io)
        p["ks"][:], p["vs"][:] = 1.0, 2.0
        _, K, V = call(p)
        for cache, s, part in ((K, 1.0, slice(64, 128)), (V, 2.0, slice(128, 192))):
            raw = cache.view(torch.uint8).cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, 64)[p["slots"].numpy()]
            assert (raw == ko.to_e4m3(f64(p["x"][:, part]) / s)).all()
        p = setup(4, 1, 1, 64, 16, io, False, 0, 0, 1, 5, idle=0.0)
        p["x"][:] = torch.tensor(vals * 12, dtype=io)
        q_out, K, V = call(p)
        assert torch.equal(q_out.cpu().view(torch.int16)[0], p["x"].view(torch.int16)[0, :64])
