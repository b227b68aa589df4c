"""replay_norm against its definition in 64 bits: types, widths, heads, strides, residuals, extreme values."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from mixer_cases import E4M3, HALF, TINY, U, e4m3_half_step, e4m3_values, gen, group_plain, norm_eps, norm_plain, normal  # noqa: E402


@pytest.fixture(scope="module")
def rb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from hybrid_decode_replay_amd import binding
    return binding


def check(y, scale, total, x, w, heads, eps, res):
    """y (fp8: with its scales) and the sum against fp64."""
    s, want = norm_plain(x, w, heads, eps, res)
    n = want.shape[-1]
    rel = norm_eps(n)
    if total is not None:
        bound = (HALF[x.dtype] + 2 * U) * s.abs() + TINY[x.dtype]
        assert ((total.cpu().double().view_as(s) - s).abs() <= bound).all()
    if scale is None:
        got, want = y.cpu().double(), want.flatten(1)
        bound = (rel + HALF[x.dtype] * (1 + rel)) * want.abs() + TINY[x.dtype]
        assert ((got - want).abs() <= bound).all()
        return
    ws, wq = group_plain(want, n)
    assert ((scale.cpu().double() - ws).abs() <= (rel + 2 * U) * ws + 2.0 ** -149).all()
    got = e4m3_values(y).view_as(wq)
    bound = e4m3_half_step(wq) + 2 * (rel + 4 * U) * wq.abs()
    bad = (got - wq).abs() > bound
    assert not bad.any(), (got[bad][:4], wq[bad][:4])


SIZES = [(1, 1, 128), (3, 1, 256), (5, 1, 384), (2, 1, 512), (7, 1, 640), (257, 1, 1024), (3, 1, 1152), (33, 1, 2048),
         (2, 1, 2176), (65, 1, 4096), (3, 1, 5120), (5, 1, 8192), (1, 1, 8320), (2, 1, 16384), (19, 7, 128), (11, 3, 256),
         (3, 5, 640)]


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out", ["same", "fp8"])
@pytest.mark.parametrize("rows,heads,n", SIZES)
def test_sizes(rb, rows, heads, n, out, io):
    g = gen(rows, heads, n)
    x = normal(g, rows, heads * n, std=3, dtype=io)
    res = normal(g, rows, heads * n, dtype=io) if rows % 2 else None
    w = normal(g, n, dtype=io) if n != 256 else None
    total = torch.empty_like(x, device="cuda") if res is not None else None
    y, scale = rb.norm(x.cuda(), None if w is None else w.cuda(), heads=heads, eps=1e-5,
                       res=None if res is None else res.cuda(), res_out=total, out_dtype=E4M3 if out == "fp8" else None)
    check(y, scale, total, x, w, heads, 1e-5, res)


@pytest.mark.parametrize("n", [8, 16, 24, 72, 120, 136, 248, 504, 1016, 2040, 4104, 16376])
@pytest.mark.parametrize("heads", [1, 3])
def test_odd_widths(rb, n, heads):
    g = gen(n, heads)
    x = normal(g, 5, heads * n, dtype=torch.bfloat16)
    w = normal(g, n, dtype=torch.bfloat16)
    y, scale = rb.norm(x.cuda(), w.cuda(), heads=heads)
    assert scale is None
    check(y, None, None, x, w, heads, 1e-6, None)


@pytest.mark.parametrize("heads,n", [(4, 128), (1, 1024), (2, 64)])
def test_rows_of_a_wider_tensor(rb, heads, n):
    """x and res as slices of fused rows; nothing beside the outputs is written."""
    g = gen(heads, n, 5)
    wide = normal(g, 9, heads * n + 88, dtype=torch.bfloat16).cuda()
    other = normal(g, 9, 2 * heads * n, dtype=torch.bfloat16).cuda()
    x, res = wide[:, 40:40 + heads * n], other[:, heads * n:]
    keep_x, keep_r = wide.clone(), other.clone()
    guard = torch.full((11, heads * n), 7.0, dtype=torch.bfloat16, device="cuda")
    total = torch.empty((9, heads * n), dtype=torch.bfloat16, device="cuda")
    rb.norm(x, heads=heads, res=res, res_out=total, y=guard[1:10])
    check(guard[1:10], None, total, x.cpu(), None, heads, 1e-6, res.cpu())
    assert (guard[0] == 7).all() and (guard[10] == 7).all()
    assert torch.equal(wide, keep_x) and torch.equal(other, keep_r)


def test_the_sum_in_place(rb):
    """res_out may be res: the residual stream of a model, layer after layer."""
    g = gen(3)
    x, res = normal(g, 300, 4096, dtype=torch.bfloat16), normal(g, 300, 4096, dtype=torch.bfloat16)
    stream = res.cuda()
    y, scale = rb.norm(x.cuda(), res=stream, res_out=stream, out_dtype=E4M3)
    check(y, scale, stream, x, None, 1, 1e-6, res)


def test_zero_and_tiny_rows(rb):
    """A row of zeros has codes 0 and the least scale; groups whose values are below it stay finite."""
    x = torch.zeros((3, 256), dtype=torch.bfloat16)
    x[1] = 2.0 ** -120
    x[2, :128] = 1
    y, scale = rb.norm(x.cuda(), out_dtype=E4M3)
    assert (e4m3_values(y)[0] == 0).all() and (scale[0] == 2.0 ** -126).all()
    assert (e4m3_values(y)[2, 128:] == 0).all() and float(scale[2, 1]) == 2.0 ** -126
    check(y, scale, None, x, None, 1, 1e-6, None)
    y, _ = rb.norm(x.cuda())
    assert (y[0] == 0).all()


def test_what_is_no_number(rb):
    """A NaN or an infinity stays in its row; a NaN code leaves its group's scale to the others; an overflowing y saturates."""
    g = gen(8)
    x = normal(g, 6, 512, dtype=torch.bfloat16)
    clean = x.clone()
    x[1, 5] = float("nan")
    x[3, 300] = float("inf")
    y, scale = rb.norm(x.cuda(), out_dtype=E4M3)
    v = e4m3_values(y)
    assert v[1].isnan().all() and (y[1].view(torch.uint8) == 0x7f).all() and (scale[1] == 2.0 ** -126).all()
    assert v[3, 300].isnan() and (v[3].nan_to_num() == 0).all()
    rows = [0, 2, 4, 5]
    check(y[rows], scale[rows], None, clean[rows], None, 1, 1e-6, None)
    # one channel whose weight is no number
    w = torch.ones(512, dtype=torch.bfloat16)
    w[130] = float("nan")
    y, scale = rb.norm(clean.cuda(), w.cuda(), out_dtype=E4M3)
    v = e4m3_values(y)
    assert v[:, 130].isnan().all() and int(v.isnan().sum()) == 6
    w[130] = 0
    check(torch.where(v.isnan(), 0.0, v).to(E4M3), scale, None, clean, w, 1, 1e-6, None)
    # an infinite y: the largest fp32 number in its group's scale, the code of 448
    w[130] = float("inf")
    y, scale = rb.norm(clean.abs().cuda(), w.cuda(), out_dtype=E4M3)
    assert (e4m3_values(y)[:, 130] == 448).all() and scale.isfinite().all()


def test_sixteen_bit_outputs_keep_infinities(rb):
    x = torch.ones((1, 128), dtype=torch.float16)
    w = torch.ones(128, dtype=torch.float16)
    w[3], w[4] = float("inf"), float("nan")
    y, _ = rb.norm(x.cuda(), w.cuda())
    assert y[0, 3] == float("inf") and y[0, 4].isnan() and y[0, 5] == 1


def test_no_rows(rb):
    y, scale = rb.norm(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), out_dtype=E4M3)
    assert y.shape == (0, 256) and scale.shape == (0, 2)


@pytest.mark.parametrize("rows,heads,n", [(70001, 1, 128), (1 << 14, 40, 64)])
def test_many_runs(rb, rows, heads, n):
    """Every run against torch on the device, in 64 bits."""
    x = torch.randn((rows, heads * n), device="cuda", dtype=torch.bfloat16)
    y, _ = rb.norm(x, heads=heads, eps=0.0)
    s = x.double().unflatten(1, (heads, n))
    want = (s / s.square().mean(-1, keepdim=True).sqrt()).flatten(1)
    bound = (norm_eps(n) + HALF[x.dtype] * (1 + norm_eps(n))) * want.abs() + TINY[x.dtype]
    assert ((y.double() - want).abs() <= bound).all()


def test_another_stream_and_a_graph(rb):
    g = gen(21)
    x = normal(g, 64, 2048, dtype=torch.bfloat16).cuda()
    w = normal(g, 2048, dtype=torch.bfloat16).cuda()
    want, ws = rb.norm(x, w, out_dtype=E4M3)
    y, scale = torch.zeros_like(want.view(torch.uint8)).view(E4M3), torch.zeros_like(ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rb.norm(x, w, y=y, y_scale=scale)
    side.synchronize()
    assert torch.equal(y.view(torch.uint8), want.view(torch.uint8)) and torch.equal(scale, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rb.norm(x, w, y=y, y_scale=scale)
    for i in range(3):
        x.copy_(normal(gen(30 + i), 64, 2048, dtype=torch.bfloat16))
        graph.replay()
        want, ws = rb.norm(x, w, out_dtype=E4M3)
        assert torch.equal(y.view(torch.uint8), want.view(torch.uint8)) and torch.equal(scale, ws)


@pytest.mark.parametrize("n,heads,out", [(72, 3, None)] + [(n, h, out) for n, h in (
    (128, 5), (256, 3), (512, 1), (1024, 1), (2048, 1), (4096, 1), (8192, 1), (16384, 1)) for out in (None, E4M3)])
def test_squares_out_of_range(rb, n, heads, out):
    """Runs of 2^-126 to 2^126 beside ordinary ones, eps 0: their squares are out of the range of fp32."""
    g = gen(n, heads, 6)
    powers = [0, -126, -90, -75, -64, -55, -50, -45, 0, 55, 60, 64, 100, 124, 0]
    x = normal(g, len(powers), heads * n)
    x = (x * torch.exp2(torch.tensor(powers, dtype=torch.float32))[:, None]).to(torch.bfloat16)
    if heads > 1:                                     # (heads of a row differ too)
        x[:, n:2 * n] = normal(g, len(powers), n).to(torch.bfloat16)
    w = normal(g, n, dtype=torch.bfloat16)
    y, scale = rb.norm(x.cuda(), w.cuda(), heads=heads, eps=0.0, out_dtype=out)
    check(y, scale, None, x, w, heads, 0.0, None)
    res = x.flip(0).contiguous()
    total = torch.empty_like(x, device="cuda")
    y, scale = rb.norm(x.cuda(), w.cuda(), heads=heads, eps=1e-30, res=res.cuda(), res_out=total, out_dtype=out)
    check(y, scale, total, x, w, heads, 1e-30, res)
