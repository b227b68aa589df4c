"""The paged cache's operators together, as a serving loop uses them: beside replayed SSM states
with the same slots, drafts and commits, captured into a graph, on other streams."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cases import check_attention, f64, normal, rng  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def cuda(x, dtype):
    return torch.from_numpy(np.asarray(x, dtype=dtype)).cuda()


class Model:
    """Two attention layers over one pool; keeps every sequence's keys and values on the host."""

    def __init__(self, B, npages, page, mp, Hq=4, Hkv=2, D=64, rot=32):
        from hybrid_decode_replay_amd import binding as rb
        self.rb, self.B, self.Hq, self.Hkv, self.D = rb, B, Hq, Hkv, D
        self.pages = rb.KVPages(rb.kv_config(B, npages, page, mp))
        self.layer = rb.kv_layer(Hq, Hkv, D, npages, page, rot_dim=rot)
        self.cache = [rb.kv_cache(self.layer) for _ in range(2)]
        self.freq = cuda(1e4 ** (-np.arange(rot // 2) / (rot // 2)), np.float32)
        self.hist = [[[] for _ in range(B)] for _ in range(2)]

    def append(self, l, x, slots, pos):
        nq, nk = self.Hq * self.D, self.Hkv * self.D
        K, V = self.cache[l]
        return self.rb.kv_append(self.layer, K, V, x[:, nq:nq + nk], x[:, nq + nk:], slots, q=x[:, :nq], pos=pos,
                                 freq=self.freq, err=self.pages.err)

    def attend(self, l, q, T, active=None, o=None, lse=None):
        K, V = self.cache[l]
        return self.rb.kv_attention(self.layer, q, K, V, self.pages.table, self.pages.end, ntok=T, active=active, o=o,
                                    lse=lse, err=self.pages.err)

    def cached(self, l, x, slots, pos):
        """The keys and values of host rows as layer l's cache holds them, checked against the rotation
        (bounds as in test_gpu_kv_append.py); rows without a slot give zeros."""
        from oracle import kv_oracle as ko
        at = slots.cpu().numpy()
        live = at >= 0
        K, V = (f64(c).transpose(0, 2, 1, 3).reshape(-1, self.Hkv, self.D)[np.maximum(at, 0)] for c in self.cache[l])
        h = f64(x).reshape(len(at), -1, self.D)[:, self.Hq:]
        k = ko.rotate(h[:, :self.Hkv], [np.maximum(pos.cpu().numpy(), 0)], self.freq.cpu().numpy(), None,
                      self.layer.rot_dim, False)
        slack = 6 * 2.0 ** -23 * 2 * np.abs(h).max()
        assert (np.abs(K - k) <= 2.0 ** -8 * (np.abs(k) + slack) + slack)[live].all()
        assert (V == h[:, self.Hkv:])[live].all()
        return np.where(live[:, None, None], K, 0), np.where(live[:, None, None], V, 0)


def test_serving_loop_beside_a_replayed_state():
    """Arrivals, decode steps, draft rounds with partial acceptance and departures, with one mask and one
    acceptance for the replayed state and the pool: every attention output is that of the sequence's
    own history."""
    from hybrid_decode_replay_amd import binding as rb, synth
    from oracle import kv_oracle as ko
    B, page, mp, T = 5, 16, 12, 3
    m = Model(B, 40, page, mp)
    cfg = rb.make_config(rb.GDN, B, 2, 1, 16, 32, 8, rb.BF16)
    ssm = rb.ReplayState(cfg)
    ssm.load_checkpoint(torch.zeros(ssm.ckpt_shape, device="cuda"))
    r = rng(11)
    live = np.zeros(B, bool)

    def ssm_tokens(k, seed):
        t = synth.gdn_tokens(seed, k, B, 2, 1, 16, 32)
        return {n: (torch.from_numpy(v).cuda() if n in ("alpha", "beta") else torch.from_numpy(v).cuda().to(torch.bfloat16))
                for n, v in t.items()}

    def outputs(x, pos_of, T_, active, l):
        """Compares layer l's outputs of the step's rows with the histories."""
        slots, pos = pos_of
        q = m.append(l, x, slots, pos)
        lse = torch.zeros((T_, B, m.Hq), device="cuda")
        o = m.attend(l, q, T_, cuda(active, np.uint8), lse=lse)
        torch.cuda.synchronize()
        hk, hv = m.cached(l, x, slots, pos)
        got_q = f64(q).reshape(T_, B, m.Hq, m.D)
        for b in range(B):
            if not active[b]:
                assert (o[:, b] == 0).all() and (lse[:, b] == 0).all()
                continue
            keys = [k for k, _ in m.hist[l][b]] + [hk[t * B + b] for t in range(T_)]
            vals = [v for _, v in m.hist[l][b]] + [hv[t * B + b] for t in range(T_)]
            K, V = (np.stack(a)[None].transpose(0, 2, 1, 3) for a in (keys, vals))       # one page of all tokens
            ref = ko.attention(got_q[:, b:b + 1], K, V, np.zeros((1, 1), np.int32), [len(keys)], m.D ** -0.5)
            check_attention(o[:, b:b + 1], lse[:, b:b + 1], ref, m.D, len(keys), torch.bfloat16)
        return hk, hv

    for step in range(14):
        if step in (0, 4, 9):                       # arrivals
            new = ~live & (r.random(B) < (1.0 if step == 0 else 0.9))
            if step == 9:
                gone = live & (r.random(B) < 0.5)
                m.pages.release(cuda(gone, np.uint8))
                for b in np.flatnonzero(gone):
                    m.hist[0][b], m.hist[1][b] = [], []
                live &= ~gone
                new = ~live
            if step == 0:
                new[3] = False
            counts = np.where(new, r.integers(1, 40, B), 0)
            idx = np.flatnonzero(new)
            if len(idx):
                ssm.load_slots(idx.tolist(), torch.zeros((len(idx), 2, 16, 32), device="cuda"))
            rows = int(counts.sum()) + 3
            slots, pos, starts = m.pages.reserve(counts=cuda(counts, np.int32), active=cuda(new, np.uint8), rows=rows)
            for l in range(2):
                x = normal((rows, (m.Hq + 2 * m.Hkv) * m.D), torch.bfloat16, 1000 * step + l).cuda()
                m.append(l, x, slots, pos)
                hk, hv = m.cached(l, x, slots, pos)
                st = starts.tolist()
                for b in idx:
                    m.hist[l][b] = [(hk[i], hv[i]) for i in range(st[b], st[b] + counts[b])]
            m.pages.commit()
            live |= new
            assert m.pages.len.tolist() == [len(h) for h in m.hist[0]]
        active = live & (r.random(B) < 0.85)
        if not active.any():
            continue
        drafts = step % 2 == 1
        k = T if drafts else 1
        mask = cuda(active, np.uint8)
        pos_of = m.pages.reserve(k, active=mask)
        if drafts:
            ssm.spec_append(k, ssm_tokens(k, step), active=mask)
        else:
            ssm.decode(ssm_tokens(1, step), active=mask)
        new = [outputs(normal((k * B, (m.Hq + 2 * m.Hkv) * m.D), torch.bfloat16, 77 * step + l).cuda(), pos_of, k, active, l)
               for l in range(2)]
        acc = np.where(active, r.integers(0, k + 1, B) if drafts else 1, 0)
        accepted = cuda(acc, np.int32)
        if drafts:
            ssm.commit(accepted)
        m.pages.commit(accepted)
        for l in range(2):
            hk, hv = new[l]
            for b in range(B):
                m.hist[l][b] += [(hk[t * B + b], hv[t * B + b]) for t in range(acc[b])]
        assert m.pages.len.tolist() == [len(h) for h in m.hist[0]]
        assert int(m.pages.err) == 0
    held = [-(-n // page) for n in m.pages.len.tolist()]
    assert all(h >= n for h, n in zip(m.pages.held.tolist(), held))
    assert int(m.pages.nfree) == 40 - sum(m.pages.held.tolist())


def test_captured_decode_step_crosses_pages():
    """One graph of reserve, append, attention and commit, replayed over 40 tokens with eager work and
    synchronizations between, equals the same steps run eagerly."""
    B, T = 3, 2
    one, two = Model(B, 30, 16, 8), Model(B, 30, 16, 8)
    x = torch.zeros((T * B, (one.Hq + 2 * one.Hkv) * one.D), dtype=torch.bfloat16, device="cuda")
    accepted = torch.zeros(B, dtype=torch.int32, device="cuda")
    o = torch.zeros((2, T, B, one.Hq, one.D), dtype=torch.bfloat16, device="cuda")

    def step(m, out):
        slots, pos = m.pages.reserve(T)
        for l in range(2):
            m.attend(l, m.append(l, x, slots, pos), T, o=out[l])
        m.pages.commit(accepted)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                                # warm up on a pool of its own
        step(Model(B, 30, 16, 8), o.clone())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(one, o)
    r = rng(4)
    for i in range(20):
        x.copy_(normal(tuple(x.shape), torch.bfloat16, 300 + i).cuda())
        accepted.copy_(cuda(r.integers(0, T + 1, B), np.int32))
        graph.replay()
        if i % 3 == 0:
            torch.cuda.synchronize()
        want = torch.zeros_like(o)
        step(two, want)
        assert torch.equal(o, want)
        assert torch.equal(one.pages.mem[64:], two.pages.mem[64:])
    assert max(one.pages.len.tolist()) > 16


def test_two_calls_at_once_on_two_streams():
    m = Model(4, 100, 16, 20)
    counts = cuda([200, 31, 300, 5], np.int32)
    slots, pos, _ = m.pages.reserve(counts=counts, rows=536)
    x = normal((536, (m.Hq + 2 * m.Hkv) * m.D), torch.bfloat16, 9).cuda()
    for l in range(2):
        m.append(l, x if l else -x, slots, pos)
    q = [normal((4, m.Hq * m.D), torch.bfloat16, 20 + l).cuda() for l in range(2)]
    want = [m.attend(l, q[l], 1) for l in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [torch.zeros_like(w) for w in want]
        torch.cuda.synchronize()
        for l in range(2):
            with torch.cuda.stream(streams[l]):
                m.attend(l, q[l], 1, o=got[l])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_paged_equals_the_dense_stand_in():
    """The same keys and values in a dense cache: the stand-in attention and the paged one agree to
    their roundings (half a bf16 step each, and the stand-in's fp32 sums)."""
    from hybrid_decode_replay_amd import binding as rb
    B, Hq, Hkv, D, L, page = 3, 8, 2, 128, 300, 32
    layer = rb.kv_layer(Hq, Hkv, D, 32, page)
    K, V = rb.kv_cache(layer)
    Kd, Vd = (normal((B, Hkv, L, D), torch.bfloat16, s).cuda() for s in (1, 2))
    q = normal((B, Hq * D), torch.bfloat16, 3).cuda()
    pages = rb.KVPages(rb.kv_config(B, 32, page, 10))
    slots, pos, _ = pages.reserve(counts=cuda([L] * B, np.int32), rows=B * L)
    flat = lambda t: t.transpose(1, 2).reshape(B * L, Hkv * D)  # noqa: E731
    rb.kv_append(layer, K, V, flat(Kd), flat(Vd), slots)
    a = rb.kv_attention(layer, q, K, V, pages.table, pages.end)[0]
    b = rb.standin_attention(q, Kd, Vd, D ** -0.5)
    mean = f64(Vd).__abs__().max()
    assert np.abs(f64(a) - f64(b)).max() <= 2 * 2.0 ** -8 * np.abs(f64(b)).max() + 2.0 ** -14 * mean


def test_binding_checks():
    from hybrid_decode_replay_amd import binding as rb
    m = Model(2, 8, 16, 4)
    K, V = m.cache[0]
    q = torch.zeros((2, m.Hq * m.D), dtype=torch.bfloat16, device="cuda")
    ok = dict(table=m.pages.table, end=m.pages.end)
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=torch.zeros((m.Hq * m.D, 2), dtype=torch.bfloat16, device="cuda").t()),
                dict(K=K[:, :1]), dict(K=K.transpose(2, 3)), dict(V=V.float()), dict(table=m.pages.table.long()),
                dict(table=m.pages.table[:1]), dict(table=m.pages.table.t()), dict(end=m.pages.end.long()),
                dict(end=m.pages.end.cpu()), dict(q=q.cpu()), dict(active=torch.ones(3, dtype=torch.uint8, device="cuda")),
                dict(active=torch.ones(2, dtype=torch.bool, device="cuda")), dict(lse=torch.zeros(2, 4, device="cuda")),
                dict(o=torch.zeros(2, 4, 64, device="cuda", dtype=torch.bfloat16)),
                dict(ws=torch.zeros(8, dtype=torch.float32, device="cuda"))):
        a = {**dict(q=q, K=K, V=V), **ok, **bad}
        with pytest.raises(ValueError):
            rb.kv_attention(m.layer, a.pop("q"), a.pop("K"), a.pop("V"), a.pop("table"), a.pop("end"), **a)
    with pytest.raises(rb.ReplayError) as e:
        rb.kv_attention(m.layer, q, K, V, m.pages.table, m.pages.end, ws=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == rb.ERR_ALIGN
    k = torch.zeros((3, m.Hkv * m.D), dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (dict(v=k[:2]), dict(slots=slots.int()), dict(slots=slots[:2]), dict(pos=None), dict(freq=None),
                dict(pos=pos.long()), dict(freq=m.freq[:3]), dict(q_out=k), dict(k=k.half()), dict(axis=slots)):
        a = {**dict(k=k, v=k, slots=slots, pos=pos, freq=m.freq), **bad}
        with pytest.raises(ValueError):
            rb.kv_append(m.layer, K, V, a.pop("k"), a.pop("v"), a.pop("slots"), **a)
    with pytest.raises(ValueError):
        m.pages.reserve(counts=m.pages.len.clone())
    with pytest.raises(ValueError):
        m.pages.commit(torch.zeros(3, dtype=torch.int32, device="cuda"))
