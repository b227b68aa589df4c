"""The paged key/value cache of a hybrid model's attention layers, as operators to time and to compare: page tables
and slot maps built on the GPU, the append of rotated keys and values, decode attention over the pages.

Three kinds of case (`op`):

  tables     the page pool: a step's new tokens get pages and slots, a round of drafts is rolled back, requests
             leave and others arrive.  All state is one int32 region: word 0 the number of free pages, word 1 the
             error bits, from word 64 on len, end, held [B] each and 4 B words of scratch (each B rounded up to 64),
             then the table [B][max_pages] and the stack of free pages [npages].
  append     rows of a fused q/k/v projection: q and k rotated by their positions (one axis or several), q written
             out, k and v written to the pages their slots name.
  attention  the queries of one step (one token a sequence, or a few drafts) over the cached keys and values.

Where `own` is false every operator is computed in elementary torch operations, in 32 bits (angles in 64).
"""
import math

import numpy as np
import torch

own = False

_TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.float8_e4m3fn}


# ---- cases -----------------------------------------------------------------------------------------------------
def listed():
    return [
        # a small server's decode step: eight sequences, one token each
        _tables("tables step b8", batch=8, ntok=1, lo=100, hi=2001, page=16, active=1.0, arrive=False),
        # a speculative round of a full batch, a quarter of its slots idle, all drafts rejected
        _tables("tables drafts b512", batch=512, ntok=4, lo=33, hi=8190, page=64, active=0.75, arrive=False),
        # half of a batch leaves and prompts of up to 8000 tokens take the slots
        _tables("tables arrivals b256", batch=256, ntok=0, lo=61, hi=8011, page=16, active=0.5, arrive=True),
        # one sequence's next token
        _append("append one row", rows=1, hq=32, hkv=8, dim=128, rot=128, axes=1, adjacent=False, page=16, idle=0.0,
                io="bf16", cache="bf16"),
        # the drafts of 256 sequences, a part of each head rotated, a cache in 8 bits
        _append("append drafts fp8", rows=1024, hq=16, hkv=2, dim=256, rot=64, axes=1, adjacent=False, page=64,
                idle=0.25, io="bf16", cache="fp8"),
        # prompts with images: three axes, neighbouring pairs
        _append("append prompts 3 axes", rows=16387, hq=32, hkv=8, dim=128, rot=128, axes=3, adjacent=True, page=16,
                idle=0.02, io="f16", cache="f16"),
        # the smallest call: one sequence, a short chat
        _attention("attention b1 short", batch=1, lo=701, hi=701, ntok=1, hq=32, hkv=8, dim=128, page=16, window=0,
                   io="bf16", cache="bf16"),
        # ordinary serving: ragged chats
        _attention("attention b64 ragged", batch=64, lo=1023, hi=4097, ntok=1, hq=32, hkv=8, dim=128, page=16,
                   window=0, io="bf16", cache="bf16"),
        # the full batch with a cache in 8 bits
        _attention("attention b256 fp8", batch=256, lo=200, hi=2001, ntok=1, hq=32, hkv=8, dim=128, page=16, window=0,
                   io="bf16", cache="fp8"),
        # one sequence with a long document: the length has to be split
        _attention("attention b1 long", batch=1, lo=131063, hi=131063, ntok=1, hq=32, hkv=8, dim=128, page=64,
                   window=0, io="bf16", cache="bf16"),
        # drafts in a sliding window
        _attention("attention drafts window", batch=48, lo=701, hi=9001, ntok=4, hq=32, hkv=4, dim=64, page=32,
                   window=1024, io="f16", cache="f16"),
        # drafts over long contexts, wide heads shared by eight queries
        _attention("attention drafts long", batch=32, lo=8191, hi=32768, ntok=8, hq=16, hkv=2, dim=256, page=64,
                   window=0, io="bf16", cache="bf16"),
    ]


def _tables(name, **c):
    return {"name": name, "op": "tables", **c}


def _append(name, **c):
    return {"name": name, "op": "append", **c}


def _attention(name, **c):
    return {"name": name, "op": "attention", **c}


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["tables", "append", "append", "attention", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128, 256])
    io = rng.choice(["bf16", "bf16", "f16"])
    cache = rng.choice([io, io, "fp8"])
    hkv = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 4, 5, 8, 16])
    dim = rng.choice([64, 128, 128, 256])
    if kind == "tables":
        batch = _spread(rng, 1, 512)
        arrive = rng.random() < 0.4
        hi = _spread(rng, 20, min(8011, 500000 // batch))
        return {"op": "tables", "batch": batch, "ntok": 0 if arrive else rng.randint(1, 16),
                "lo": max(1, int(hi * rng.random())), "hi": hi, "page": page, "active": rng.choice([1.0, 0.75, 0.5]),
                "arrive": arrive}
    if kind == "append":
        most = min(16387, int(3.5e8 / (dim * (4 * group * hkv + 8 * hkv))))     # the bytes of the largest listed case
        return {"op": "append", "rows": _spread(rng, 1, most), "hq": group * hkv, "hkv": hkv, "dim": dim,
                "rot": rng.choice([0, dim, dim // 2, dim // 4]), "axes": rng.choice([1, 1, 2, 3, 4]),
                "adjacent": rng.random() < 0.5, "page": page, "idle": rng.choice([0.0, 0.0, 0.25]), "io": io,
                "cache": cache}
    ntok = rng.choice([1, 1, 1, 2, 3, 4, 7, 8, 16])
    window = rng.choice([0, 0, 0, _spread(rng, 8, 4099)])
    batch = _spread(rng, 1, 256)
    # no dearer than the largest listed case: its bytes of keys and values, and its products
    tokens = min(1.2e9 / (4 * hkv * dim), 1e10 / (ntok * hkv * group * dim / 2))
    hi = _spread(rng, 1, max(16, int(min(131063, tokens / batch))))
    return {"op": "attention", "batch": batch, "lo": max(1, int(hi * rng.choice([1.0, 0.5, 0.1]))), "hi": hi,
            "ntok": ntok, "hq": group * hkv, "hkv": hkv, "dim": dim, "page": page, "window": window, "io": io,
            "cache": cache}


def _ramp(lo, hi, n):
    """n whole numbers from lo to hi."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _shuffled(values, rng):
    values = np.asarray(values, dtype=np.int64)
    return values[rng.permutation(len(values))]


def _pages(tokens, page):
    return -(-tokens // page)


# ---- inputs ----------------------------------------------------------------------------------------------------
def prepare(case, seed):
    op = case["op"]
    return {"tables": _prepare_tables, "append": _prepare_append, "attention": _prepare_attention}[op](case, seed)


def _sizes(c):
    """(active sequences, counts of arriving tokens, max_pages, npages, rows) of a tables case."""
    B, page = c["batch"], c["page"]
    nact = max(1, int(B * c["active"]))
    counts = _ramp(c["lo"], c["hi"], nact)
    mp = _pages(c["hi"] + 16, page) + 1
    npages = sum(_pages(n, page) for n in _ramp(c["lo"], c["hi"], B)) + sum(_pages(n, page) for n in counts) + 2 * B + 3
    rows = sum(counts) + 77 if c["arrive"] else c["ntok"] * B
    return nact, counts, mp, npages, rows


def _views(batch, max_pages, npages, mem):
    """The parts of the pool's region."""
    bp = -(-batch // 64) * 64
    t = 64 + 7 * bp
    return {"nfree": mem[0:1], "err": mem[1:2], "len": mem[64:64 + batch], "end": mem[64 + bp:64 + bp + batch],
            "held": mem[64 + 2 * bp:64 + 2 * bp + batch],
            "table": mem[t:t + batch * max_pages].reshape(batch, max_pages),
            "free": mem[t + batch * max_pages:t + batch * max_pages + npages]}


def _prepare_tables(c, seed):
    rng = np.random.default_rng([seed, 1])
    B, page = c["batch"], c["page"]
    nact, counts, mp, npages, rows = _sizes(c)
    mem = np.zeros(64 + 7 * (-(-B // 64) * 64) + B * mp + npages, dtype=np.int32)
    v = _views(B, mp, npages, mem)
    lens = _shuffled(_ramp(c["lo"], c["hi"], B), rng)
    pool = rng.permutation(npages).astype(np.int32)
    held = _pages(lens, page)
    at = int(held.sum())
    v["table"][:] = -1
    v["table"][np.arange(mp)[None] < held[:, None]] = pool[:at]
    v["held"][:] = held
    v["len"][:] = lens
    v["end"][:] = lens
    v["nfree"][0] = npages - at
    v["free"][:npages - at] = pool[at:]
    active = np.zeros(B, dtype=np.uint8)
    active[rng.permutation(B)[:nact]] = 1
    new = np.zeros(B, dtype=np.int32)
    new[active != 0] = _shuffled(counts, rng)
    cuda = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return {"case": c, "mem": cuda(mem), "active": cuda(active), "counts": cuda(new), "max_pages": mp, "npages": npages,
            "rows": rows, "rejected": torch.zeros(B, dtype=torch.int32, device="cuda"),
            "slots": torch.zeros(rows, dtype=torch.int64, device="cuda"),
            "pos": torch.zeros(rows, dtype=torch.int32, device="cuda"),
            "starts": torch.zeros(B + 1, dtype=torch.int32, device="cuda")}


def _scales(case, n, gen):
    if case["cache"] != "fp8":
        return None
    return torch.rand(n, generator=gen, device="cuda") * 0.02 + 0.02


def _prepare_append(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7 + 3)
    rng = np.random.default_rng([seed, 2])
    N, Hq, Hkv, D, page, rot = c["rows"], c["hq"], c["hkv"], c["dim"], c["page"], c["rot"]
    io = _TORCH[c["io"]]
    npages = _pages(N, page) + 3
    # the projection's rows: a head's channels differ in size, as trained ones do
    width = (Hq + 2 * Hkv) * D
    qkv = torch.randn((N, width), generator=gen, device="cuda")
    qkv *= 0.5 + torch.rand(width, generator=gen, device="cuda")
    cache = torch.zeros((2, npages, Hkv, page, D), device="cuda", dtype=_TORCH[c["cache"]])
    # pages in any order, tokens in order within them; some rows belong to idle slots
    order = torch.from_numpy(rng.permutation(npages)).cuda()
    t = torch.arange(N, device="cuda")
    slots = order[t // page] * page + t % page
    idle = rng.permutation(N)[:int(N * c["idle"])]
    slots[torch.from_numpy(idle).cuda()] = -1
    far = [131071, 8191, 97, 61]
    pos = torch.from_numpy(np.stack([rng.integers(0, far[a], N) for a in range(c["axes"])]).astype(np.int32)).cuda()
    # sections of the rotated pairs belong to the axes in turn
    axis = torch.from_numpy((np.arange(rot // 2) * c["axes"] // max(1, rot // 2)).astype(np.uint8)).cuda()
    freq = torch.from_numpy((1e6 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)).cuda()
    return {"case": c, "qkv": qkv.to(io), "K": cache[0], "V": cache[1], "slots": slots, "pos": pos, "axis": axis,
            "freq": freq, "npages": npages, "q_out": torch.zeros((N, Hq * D), dtype=io, device="cuda"),
            "k_scale": _scales(c, Hkv, gen), "v_scale": _scales(c, Hkv, gen)}


def _prepare_attention(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 11 + 5)
    rng = np.random.default_rng([seed, 3])
    B, Hq, Hkv, D, page, T = c["batch"], c["hq"], c["hkv"], c["dim"], c["page"], c["ntok"]
    io, kind = _TORCH[c["io"]], _TORCH[c["cache"]]
    lens = _shuffled(_ramp(c["lo"], c["hi"], B), rng)
    mp = _pages(c["hi"], page)
    held = _pages(lens, page)
    npages = int(held.sum()) + 5
    pool = rng.permutation(npages)
    table = np.full((B, mp), -1, dtype=np.int32)
    table[np.arange(mp)[None] < held[:, None]] = pool[:held.sum()]

    def pages():
        x = torch.randn((npages, Hkv, page, D), generator=gen, device="cuda", dtype=io)
        return (x * 35).to(kind) if c["cache"] == "fp8" else x

    q = torch.randn((T * B, Hq * D), generator=gen, device="cuda", dtype=io) * 1.5
    return {"case": c, "q": q, "K": pages(), "V": pages(), "table": torch.from_numpy(table).cuda(),
            "end": torch.from_numpy(lens.astype(np.int32)).cuda(), "npages": npages, "scale": D ** -0.5,
            "o": torch.zeros((T, B, Hq, D), dtype=io, device="cuda"),
            "lse": torch.zeros((T, B, Hq), dtype=torch.float32, device="cuda"),
            "k_scale": _scales(c, Hkv, gen), "v_scale": _scales(c, Hkv, gen)}


# ---- one pass --------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"tables": _own_tables, "append": _own_append, "attention": _own_attention}[op](state)
    return {"tables": _plain_tables, "append": _plain_append, "attention": _plain_attention}[op](state)


def _binding():
    from hybrid_decode_replay_amd import binding
    return binding


def _own_tables(s):
    rb, c = _binding(), s["case"]
    pages = rb.KVPages(rb.kv_config(c["batch"], s["npages"], c["page"], s["max_pages"]), mem=s["mem"])
    if c["arrive"]:
        pages.release(s["active"])
        pages.reserve(counts=s["counts"], active=s["active"], slots=s["slots"], pos=s["pos"], starts=s["starts"])
    else:
        pages.reserve(c["ntok"], active=s["active"], slots=s["slots"], pos=s["pos"])
        pages.commit(s["rejected"])
    return _tables_out(s)


def _tables_out(s):
    c = s["case"]
    v = _views(c["batch"], s["max_pages"], s["npages"], s["mem"])
    return {**v, "slots": s["slots"], "pos": s["pos"], "starts": s["starts"]}


def _own_append(s):
    rb, c = _binding(), s["case"]
    layer = _layer(rb, s, rot_dim=c["rot"], rot_style=rb.ROT_ADJACENT if c["adjacent"] else rb.ROT_HALVES)
    nq, nk = c["hq"] * c["dim"], c["hkv"] * c["dim"]
    x = s["qkv"]
    rb.kv_append(layer, s["K"], s["V"], x[:, nq:nq + nk], x[:, nq + nk:], s["slots"], q=x[:, :nq], q_out=s["q_out"],
                 pos=s["pos"], freq=s["freq"], axis=s["axis"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"q": s["q_out"], "K": s["K"], "V": s["V"]}


def _layer(rb, s, **kw):
    c = s["case"]
    kinds = {"bf16": rb.BF16, "f16": rb.F16, "fp8": rb.FP8_E4M3}
    return rb.kv_layer(c["hq"], c["hkv"], c["dim"], s["npages"], c["page"], io_dtype=kinds[c["io"]],
                       cache_dtype=kinds[c["cache"]], **kw)


def _own_attention(s):
    rb, c = _binding(), s["case"]
    rb.kv_attention(_layer(rb, s), s["q"], s["K"], s["V"], s["table"], s["end"], ntok=c["ntok"], scale=s["scale"],
                    window=c["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], o=s["o"], lse=s["lse"])
    return {"o": s["o"], "lse": s["lse"]}


# ---- plain forms -----------------------------------------------------------------------------------------------
def _plain_tables(s):
    c = s["case"]
    v = _views(c["batch"], s["max_pages"], s["npages"], s["mem"])
    if c["arrive"]:
        _plain_release(v, s["active"])
        _plain_reserve(c, v, s["counts"].long() * (s["active"] != 0), s, True)
    else:
        _plain_reserve(c, v, c["ntok"] * (s["active"] != 0).long(), s, False)
        v["len"] += torch.minimum(s["rejected"].clamp(min=0), v["end"] - v["len"])
        v["end"].copy_(v["len"])
    return _tables_out(s)


def _plain_release(v, mask):
    """The marked sequences' pages go back on the stack, the last one first."""
    held = torch.where(mask != 0, v["held"], 0).long()
    total = held.sum()
    first = torch.cumsum(held, 0) - held
    i = torch.arange(v["table"].shape[1], device=held.device)
    taken = i[None] < held[:, None]
    at = (v["nfree"].long() + total - 1 - first[:, None] - i[None])[taken]
    v["free"][at] = v["table"][taken]
    v["table"][taken] = -1
    v["nfree"] += total.int()
    kept = (mask == 0).int()
    v["held"] *= kept
    v["len"] *= kept
    v["end"] *= kept


def _plain_reserve(c, v, new, s, packed):
    page, (B, mp) = c["page"], v["table"].shape
    dev = new.device
    lens, held = v["len"].long(), v["held"].long()
    start = torch.cumsum(new, 0) - new
    rows = s["rows"]
    fits = lens + new <= mp * page
    if packed:
        fits &= start + new <= rows
    need = torch.clamp((lens + new + page - 1) // page - held, min=0) * fits
    upto = torch.cumsum(need, 0)
    given = fits & ((need == 0) | (upto <= v["nfree"].long()))
    got = need * given
    i = torch.arange(mp, device=dev)
    fresh = (i[None] >= held[:, None]) & (i[None] < (held + got)[:, None])
    k = (upto - need)[:, None] + i[None] - held[:, None]
    v["table"][fresh] = v["free"][(v["nfree"].long() - 1 - k)[fresh]]
    v["nfree"] -= (upto * (got > 0)).max().int()
    v["held"] += got.int()
    v["end"].copy_(lens + new * given)
    r = torch.arange(rows, device=dev)
    if packed:
        total = new.sum()
        b = (torch.searchsorted(start + new, r, right=True)).clamp(max=B - 1)
        t = r - start[b]
        live = (r < total) & given[b]
        s["starts"][:B] = start
        s["starts"][B] = total
    else:
        b, t = r % B, r // B
        live = (t < new[b]) & given[b]
    p = lens[b] + t
    at = v["table"][b, (p // page).clamp(max=mp - 1)].long() * page + p % page
    s["slots"].copy_(torch.where(live, at, -1))
    s["pos"].copy_(torch.where(live, p, -1))


def _rotated(x, cos, sin, rot, adjacent):
    """x [N][H][D] in 32 bits, its first `rot` channels turned pair by pair; cos and sin [N][1][rot / 2]."""
    if rot == 0:
        return x
    if adjacent:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_append(s):
    c = s["case"]
    N, Hq, Hkv, D, rot, io = c["rows"], c["hq"], c["hkv"], c["dim"], c["rot"], _TORCH[c["io"]]
    x = s["qkv"].float().view(N, Hq + 2 * Hkv, D)
    angle = s["pos"].double()[s["axis"].long()].T * s["freq"].double()          # [N][rot / 2]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    live = s["slots"] >= 0
    q = _rotated(x[:, :Hq], cos, sin, rot, c["adjacent"]).reshape(N, Hq * D)
    s["q_out"].copy_(torch.where(live[:, None], q.to(io), s["q_out"]))
    k = _rotated(x[:, Hq:Hq + Hkv], cos, sin, rot, c["adjacent"])
    slot = s["slots"][live]
    _stored(s["K"], k[live], slot, s["k_scale"])
    _stored(s["V"], x[:, Hq + Hkv:][live], slot, s["v_scale"])
    return {"q": s["q_out"], "K": s["K"], "V": s["V"]}


def _stored(cache, rows, slot, scale):
    page = cache.shape[2]
    if scale is not None:
        rows = (rows / scale[:, None]).clamp(-448, 448).to(cache.dtype).view(torch.uint8)
        cache = cache.view(torch.uint8)
    cache[slot // page, :, slot % page] = rows.to(cache.dtype)


def _gathered(cache, table, scale):
    """[B][Hkv][max_pages * page][D] in 32 bits."""
    at = table.long().clamp(min=0)
    x = cache.view(torch.uint8)[at].view(cache.dtype) if scale is not None else cache[at]
    x = x.float().transpose(1, 2)
    if scale is not None:
        x = x * scale[None, :, None, None, None]
    return x.flatten(2, 3)


def _plain_attention(s):
    c = s["case"]
    B, Hq, Hkv, D, T, window = c["batch"], c["hq"], c["hkv"], c["dim"], c["ntok"], c["window"]
    k = _gathered(s["K"], s["table"], s["k_scale"])
    q = s["q"].float().view(T, B, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3, 4).reshape(B, Hkv, -1, D)
    score = (q @ k.transpose(-1, -2)).view(B, Hkv, T, Hq // Hkv, -1) * s["scale"]
    j = torch.arange(k.shape[2], device=k.device)
    p = s["end"][:, None].long() - T + torch.arange(T, device=k.device)         # [B][T]
    seen = j <= p[..., None]
    if window:
        seen &= j > p[..., None] - window
    score = torch.where(seen[:, None, :, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    del k, score
    v = _gathered(s["V"], s["table"], s["v_scale"])
    v = torch.where((j < s["end"][:, None])[:, None, :, None], v, 0.0)
    o = (e.flatten(2, 3) @ v).view(B, Hkv, T, Hq // Hkv, D)
    o = torch.where(total > 0, o / total, 0.0)
    s["o"].copy_(o.permute(2, 0, 1, 3, 4).reshape(T, B, Hq, D))
    s["lse"].copy_((top + total.log()).squeeze(-1).permute(2, 0, 1, 3).reshape(T, B, Hq))
    return {"o": s["o"], "lse": s["lse"]}


# ---- what a pass cannot do without -----------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "tables":
        nact, counts, mp, npages, rows = _sizes(c)
        if c["arrive"]:
            moved = 2 * sum(_pages(n, c["page"]) for n in counts)
            return {"bytes": 8 * moved + 12 * rows + 28 * c["batch"], "flops": rows}
        return {"bytes": 12 * rows + 33 * c["batch"], "flops": rows}
    size = {"bf16": 2, "f16": 2, "fp8": 1}
    if c["op"] == "append":
        live = c["rows"] - int(c["rows"] * c["idle"])
        per = c["dim"] * (2 * c["hq"] * size[c["io"]] + 2 * c["hkv"] * (size[c["io"]] + size[c["cache"]]))
        return {"bytes": live * (per + 8 + 4 * c["axes"]), "flops": 3 * live * (c["hq"] + c["hkv"]) * c["rot"]}
    T, window = c["ntok"], c["window"]
    lens = _ramp(c["lo"], c["hi"], c["batch"])
    tokens = sum(min(n, window + T - 1) if window else n for n in lens)
    pairs = sum(min(max(0, n - T + t + 1), window or n) for n in lens for t in range(T))
    rows = T * c["batch"] * c["hq"]
    return {"bytes": 2 * tokens * c["hkv"] * c["dim"] * size[c["cache"]] + rows * (2 * c["dim"] * size[c["io"]] + 4)
            + 4 * sum(_pages(n, c["page"]) for n in lens), "flops": 4 * pairs * c["hq"] * c["dim"]}


# ---- in 64 bits ------------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "tables":
        return None
    c, s = case, prepare(case, seed)
    if c["op"] == "append":
        return _exact_append(c, s)
    # attention sequence by sequence and token by token, over its visible positions alone
    B, Hq, Hkv, D, T, page = c["batch"], c["hq"], c["hkv"], c["dim"], c["ntok"], c["page"]
    o = torch.zeros((T, B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    q = s["q"].double().reshape(T, B, Hkv, Hq // Hkv, D)
    for b, n in enumerate(s["end"].tolist()):
        first = max(0, n - T + 1 - c["window"]) // page if c["window"] else 0
        at = s["table"][b, first:_pages(n, page)].long()
        k, v = _exact_tokens(s["K"], at, s["k_scale"]), _exact_tokens(s["V"], at, s["v_scale"])
        for t in range(T):
            last = n - T + t + 1 - first * page
            begin = max(0, last - c["window"]) if c["window"] else 0
            if last > begin:
                w = torch.matmul(k[:, begin:last], q[t, b].transpose(1, 2).contiguous()) * s["scale"]
                norm = torch.logsumexp(w, 1)                                    # [Hkv][Hq / Hkv]
                lse[t, b] = norm.flatten()
                w = torch.exp(w - norm[:, None]).transpose(1, 2).contiguous()
                o[t, b] = torch.matmul(w, v[:, begin:last]).reshape(Hq, D)
    return {"o": o, "lse": lse}


def _exact_tokens(cache, at, scale):
    """The tokens of pages `at` in order: [Hkv][tokens][D] in 64 bits."""
    x = cache[at] if scale is None else cache.view(torch.uint8)[at].view(cache.dtype)
    x = x.transpose(0, 1).flatten(1, 2).double()
    return x if scale is None else x * scale.double()[:, None, None]


def _exact_append(c, s):
    """Rotation as a product with e^(i angle)."""
    N, Hq, Hkv, D, page, rot = c["rows"], c["hq"], c["hkv"], c["dim"], c["page"], c["rot"]
    x = s["qkv"].double().reshape(N, -1, D)
    heads = x[:, :Hq + Hkv].clone()
    if rot:
        steps = torch.stack([s["pos"][int(a)].double() for a in s["axis"].tolist()], 1) * s["freq"].double()
        i = torch.arange(rot // 2, device="cuda")
        re, im = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + rot // 2)
        z = torch.complex(heads[..., re], heads[..., im]) * torch.complex(steps.cos(), steps.sin())[:, None]
        heads[..., re], heads[..., im] = z.real, z.imag
    slots = s["slots"]
    rows = torch.nonzero(slots >= 0).flatten()
    q = torch.zeros((N, Hq * D), dtype=torch.float64, device="cuda")
    q[rows] = heads[rows, :Hq].reshape(len(rows), -1)

    def cached(values, scale):
        out = torch.zeros((s["npages"] * page, Hkv, D), dtype=torch.float64, device="cuda")
        out[slots[rows]] = values[rows] / (1.0 if scale is None else scale.double()[:, None])
        return out.view(s["npages"], page, Hkv, D).transpose(1, 2).contiguous()

    return {"q": q, "K": cached(heads[:, Hq:], s["k_scale"]), "V": cached(x[:, Hq + Hkv:], s["v_scale"])}
