"""A step in which reserve refuses a sequence: the mask of the served keeps it out of the attention and
of the replayed state's step, eagerly and in a captured step."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cases import normal  # noqa: E402
from test_gpu_kv_flow import Model, cuda  # noqa: E402

import numpy as np  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def test_the_served_mask():
    """Idle sequences, ones without new tokens, ones refused for want of pages or of table."""
    from hybrid_decode_replay_amd import binding as rb
    pages = rb.KVPages(rb.kv_config(5, 4, 16, 2))
    assert pages.served().tolist() == [0] * 5
    pages.reserve(counts=cuda([16, 0, 33, 10, 40], np.int32), rows=200)
    assert pages.served().tolist() == [1, 0, 0, 1, 0] and int(pages.err) == 2
    pages.commit()
    assert pages.served().tolist() == [0] * 5
    pages.reserve(2, active=cuda([1, 1, 1, 1, 0], np.uint8))
    assert pages.served().tolist() == [1, 1, 0, 1, 0] and int(pages.err) == 3
    assert pages.served().dtype == torch.uint8


def step(m, x, q_out, o, mask=None):
    """One token of every sequence (of mask) through layer 0; returns the mask of the served."""
    slots, pos = m.pages.reserve(1, active=mask)
    served = m.pages.served()
    K, V = m.cache[0]
    nq, nk = m.Hq * m.D, m.Hkv * m.D
    m.rb.kv_append(m.layer, K, V, x[:, nq:nq + nk], x[:, nq + nk:], slots, q=x[:, :nq], q_out=q_out, pos=pos, freq=m.freq,
                   err=m.pages.err)
    m.attend(0, q_out, 1, served, o=o)
    m.pages.commit()
    return served


@pytest.mark.parametrize("captured", [False, True])
def test_refused_sequences_keep_their_outputs(captured):
    """Five pages are held by sequences of 31, 32 and 16 tokens: the next token of the first has room, the
    others' have not; then nobody's has; then the second leaves and two pages are free.  What is served is
    what a pool with room gives for the same mask."""
    B = 3
    m, roomy = Model(B, 5, 16, 8), Model(B, 30, 16, 8)
    width = (m.Hq + 2 * m.Hkv) * m.D
    x = normal((79, width), torch.bfloat16, 8).cuda()
    for model in (m, roomy):
        slots, pos, _ = model.pages.reserve(counts=cuda([31, 32, 16], np.int32), rows=79)
        model.append(0, x, slots, pos)
        model.pages.commit()
    assert int(m.pages.nfree) == 0 and int(m.pages.err) == 0
    x = torch.zeros((B, width), dtype=torch.bfloat16, device="cuda")
    q_out, o = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((B, m.Hq * m.D), (1, B, m.Hq, m.D)))
    served = torch.zeros(B, dtype=torch.uint8, device="cuda")
    run = lambda: served.copy_(step(m, x, q_out, o))  # noqa: E731
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):                           # warm up on a pool of its own
            step(Model(B, 5, 16, 8), x, q_out.clone(), o.clone())
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        run = graph.replay
    for i, (mask, lens) in enumerate([([1, 0, 0], [32, 32, 16]), ([0, 0, 0], [32, 32, 16]), ([1, 1, 0], [33, 1, 16])]):
        if i == 2:
            for model in (m, roomy):
                model.pages.release(cuda([0, 1, 0], np.uint8))
        x.copy_(normal(tuple(x.shape), torch.bfloat16, 20 + i).cuda())
        q_out.fill_(5.0)
        o.fill_(3.0)
        run()
        torch.cuda.synchronize()
        want, wq = torch.full_like(o, 3.0), torch.full_like(q_out, 5.0)
        step(roomy, x, wq, want, cuda(mask, np.uint8))
        assert served.tolist() == mask and m.pages.len.tolist() == lens and int(m.pages.err) == 1
        assert torch.equal(o, want) and torch.equal(q_out, wq)
        for b in range(B):
            assert (o[:, b] == 3.0).all() == (not mask[b]) and (q_out[b] == 5.0).all() == (not mask[b])


def test_a_replayed_state_takes_the_same_mask():
    """The state of a refused sequence does not move when its step is given the served mask."""
    from hybrid_decode_replay_amd import binding as rb, synth
    B = 3
    pages = rb.KVPages(rb.kv_config(B, 2, 16, 4))
    ssm = rb.ReplayState(rb.make_config(rb.GDN, B, 2, 1, 16, 32, 8, rb.BF16))
    ssm.load_checkpoint(torch.zeros(ssm.ckpt_shape, device="cuda"))
    tok = {n: (torch.from_numpy(v).cuda() if n in ("alpha", "beta") else torch.from_numpy(v).cuda().to(torch.bfloat16))
           for n, v in synth.gdn_tokens(5, 1, B, 2, 1, 16, 32).items()}
    pages.reserve(1)
    ssm.decode(tok, active=pages.served())
    pages.commit()
    assert pages.len.tolist() == [1, 1, 0] and int(pages.err) == 1
    assert ssm.read_book()[0].tolist() == [1, 1, 0]
