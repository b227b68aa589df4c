"""README's example of prompts through a Gated DeltaNet layer, run as it stands there."""
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mixer_cases import E4M3, gen, normal  # noqa: E402

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
    found = [b for b in blocks if "rb.gdn_prefill" in b]
    assert len(found) == 1
    return found[0]


def test_prompts_arrive():
    from hybrid_decode_replay_amd import binding as rb
    E, H, G, Dk, Dv, rows = 256, 4, 2, 64, 128, 90
    g = gen(3)
    ones = lambda n: torch.ones(n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    codes = lambda n, k: normal(g, n, k, std=50).to(E4M3).cuda()  # noqa: E731
    scales = lambda n, k: torch.full((-(-n // 128), k // 128), 1e-3, device="cuda")  # noqa: E731
    wide = 2 * G * Dk + H * Dv
    st = rb.ReplayState(rb.make_config(rb.GDN, 5, H, G, Dv, Dk, 4, rb.BF16, scale=Dk ** -0.5), device="cuda")
    st.load_checkpoint(torch.zeros((5, H, Dv, Dk), device="cuda"))
    x, stream = (normal(g, rows, E, dtype=torch.bfloat16).cuda() for _ in range(2))
    names = dict(rb=rb, torch=torch, H=H, G=G, Dk=Dk, x=x, stream=stream, w_norm=ones(E), w_head=ones(Dv),
                 unit=ones(Dk) * Dk ** -0.5, w_in=codes(wide, E), w_in_scale=scales(wide, E), w_out=codes(E, H * Dv),
                 w_out_scale=scales(E, H * Dv), alpha=torch.rand((rows, H), generator=g).cuda(),
                 beta=torch.rand((rows, H), generator=g).cuda(), state=st, slots=[3, 1],
                 starts=torch.tensor([0, 20, 90], dtype=torch.int32, device="cuda"))
    exec(example(), names)
    torch.cuda.synchronize()
    ck, S = st.read_checkpoint(), names["S"]
    assert torch.equal(ck[3], S[0]) and torch.equal(ck[1], S[1]) and (ck[[0, 2, 4]] == 0).all()
    assert S.abs().amax() > 0 and names["out"].shape == (rows, E) and names["out"].isfinite().all()
    # a first token sees an empty state: o = scale beta (q.k) v
    q, k = (names[n].float().view(rows, G, Dk).repeat_interleave(H // G, 1)[[0, 20]] for n in "qk")
    v = names["v"].float().view(rows, H, Dv)[[0, 20]]
    want = Dk ** -0.5 * names["beta"][[0, 20]][..., None] * (q * k).sum(-1, keepdim=True) * v
    o = names["o"].float().view(rows, H, Dv)[[0, 20]]
    # a rounding to bf16, and terms of 16 bits of |q| |k| |v| before it
    assert ((o - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -14 * v.abs()).all()


@pytest.mark.parametrize("Dk", [64, 128])
def test_heads_of_small_projections_have_length_one(Dk):
    """q and k of projections of some 2e-3: x / sqrt(x.x + 1e-6).  In lengths: eps 1e-6 / x.x / 2; a rounding of each value to
    bf16 and one of Dk ** -0.5 (which is exact for Dk 64), 2^-8 each; an fp32 norm."""
    from hybrid_decode_replay_amd import binding as rb
    E, H, G, Dv, rows = 256, 2, 2, 128, 40
    g = gen(4)
    ones = lambda n: torch.ones(n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    codes = lambda n, k: normal(g, n, k, std=50).to(E4M3).cuda()  # noqa: E731
    scales = lambda n, k, s: torch.full((-(-n // 128), k // 128), s, device="cuda")  # noqa: E731
    wide = 2 * G * Dk + H * Dv
    st = rb.ReplayState(rb.make_config(rb.GDN, 1, H, G, Dv, Dk, 4, rb.BF16, scale=Dk ** -0.5), device="cuda")
    x, stream = (normal(g, rows, E, dtype=torch.bfloat16).cuda() for _ in range(2))
    names = dict(rb=rb, torch=torch, H=H, G=G, Dk=Dk, x=x, stream=stream, w_norm=ones(E), w_head=ones(Dv),
                 unit=ones(Dk) * Dk ** -0.5, w_in=codes(wide, E), w_in_scale=scales(wide, E, 2.5e-6), w_out=codes(E, H * Dv),
                 w_out_scale=scales(E, H * Dv, 1e-3), alpha=torch.rand((rows, H), generator=g).cuda(),
                 beta=torch.rand((rows, H), generator=g).cuda(), state=st, slots=[0],
                 starts=torch.tensor([0, rows], dtype=torch.int32, device="cuda"))
    exec(example(), names)
    p = names["p"][:, :2 * G * Dk].double().view(rows, 2 * G, Dk)
    sq = p.square().sum(-1)
    assert 1e-4 < sq.min() and sq.max() < 1e-2
    got = torch.cat([names["q"], names["k"]], 1).double().view(rows, 2 * G, Dk).norm(dim=-1)
    want = (sq / (sq + 1e-6)).sqrt()
    assert ((got - want).abs() <= 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -16).all()
    assert ((got - 1).abs() <= 1e-6 / sq / 2 + 2.0 ** -7 + 2.0 ** -16).all()
