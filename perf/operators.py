"""The operators of the 8-bit prefix cache, and the calls on which their time is measured.

A prefix cache may be held in 8 bits: keys and values as e4m3 codes, with one
fp32 scale for each page (16 tokens) of each KV head, for K and for V.  A
cached value stands for ``code * scale``.  The operators are

* ``write``   quantise a whole prefix into such a cache, with the page min/max
              records of the keys that the cache now holds;
* ``append``  commit a finished block to it (the touched pages re-encoded);
* ``read``    read it back;
* ``dense``   attention of a block's queries over the whole cached prefix and
              the block itself (``B = 1``: one decoded token);
* ``step``    one LoSA denoising step over it.

``run`` computes one pass of an operator: in elementary torch operations where
``own`` is false, by the framework's calls where it is true.

The page scale is the smallest power of two, at least 2^-100, with which the
page's largest magnitude is at most 448, e4m3's largest number (1 for a page
of zeros); codes are rounded to nearest even.
"""
import math

import torch

own = False

D = 128       # head dimension
PS = 16       # tokens per page
E4M3_MAX = 448.0
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(op, S, Hkv, G, L, B, dtype="bf16", cap=0, ragged=False, A=0, budget=0, name=None):
    c = dict(op=op, S=S, Hkv=Hkv, G=G, L=L, B=B, dtype=dtype, cap=cap or L, ragged=ragged, A=A,
             budget=budget)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a 16K prompt of one GQA layer (8 KV heads) is quantised after its prefill
        _case("write", 1, 8, 4, 16384, 16, name="write_16k"),
        # three prompts of different, odd lengths, in fp32, with room to grow
        _case("write", 3, 2, 4, 2005, 16, "f32", cap=2080, ragged=True, name="write_f32_ragged"),
        # a block of 16 is committed to a 64K prefix, as after each block of a generation
        _case("append", 1, 8, 4, 65003, 16, cap=65536, name="append_64k"),
        # eight sequences of a batch commit blocks of 32 at their own odd lengths
        _case("append", 8, 8, 4, 1999, 32, cap=2048, ragged=True, name="append_batch8"),
        # the whole 64K prefix is read back (to move it, or for a path without 8-bit support)
        _case("read", 1, 8, 4, 65536, 16, name="read_64k"),
        # a short ragged fp32 batch is read back
        _case("read", 4, 2, 4, 1003, 16, "f32", cap=1024, ragged=True, name="read_f32_ragged"),
        # the first denoising step of a block of 16 over 64K of context
        _case("dense", 1, 8, 4, 65536, 16, name="dense_64k"),
        # one token decoded for each of eight sequences of up to 32K tokens
        _case("dense", 8, 8, 4, 32768, 1, ragged=True, name="dense_decode_batch8"),
        # a single fp32 head over a short prefix: where latency counts
        _case("dense", 1, 1, 1, 2048, 16, "f32", name="dense_f32_tiny"),
        # eight 32K sequences with blocks of 32: 128 query rows for each KV head
        _case("dense", 8, 8, 4, 32768, 32, name="dense_batch8"),
        # a denoising step of a block of 16 over 64K, 8 pages for each active query
        _case("step", 1, 8, 4, 65536, 16, A=4, budget=128, name="step_64k"),
        # a step of four sequences of different lengths up to 16K, 16 pages each
        _case("step", 4, 8, 4, 16333, 16, cap=16400, ragged=True, A=4, budget=256,
              name="step_batch4_ragged"),
    ]


def draw(rng):
    op = rng.choice(("write", "append", "read", "dense", "dense", "step"))
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    Hkv = rng.choice((1, 2, 4, 8))
    G = rng.choice((1, 2, 4, 8))
    # (an fp32 step keeps twice the bytes of a bf16 one on chip, and takes half its rows)
    rows = 128 if op != "step" else 32 if dtype == "f32" else 64
    B = rng.choice([b for b in (1, 2, 5, 8, 16, 31, 32) if G * b <= rows])
    S = rng.randint(1, 8)
    # the bytes of all sequences and heads together stay below the largest listed case's
    top = min(65536, (1 << (18 if dtype == "f32" else 19 if op in ("write", "read") else 20)) // (S * Hkv))
    L = int(round(math.exp(rng.uniform(0.0, math.log(top)))))
    A = budget = 0
    if op == "step":
        A = rng.randint(1, min(B, 8))
        budget = PS * rng.choice((1, 4, 8, 16, 32))
    cap = L + rng.choice((0, 0, 5, 32, 100)) + (B if op == "append" else 0)
    return _case(op, S, Hkv, G, L, B, dtype, cap, rng.random() < 0.5, A, budget)


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    SG, d = c["S"] * c["Hkv"], D
    rows = SG * c["G"] * c["B"]
    tokens = c["Hkv"] * _mean_tokens(c)                     # over all sequences and KV heads
    pages = tokens / PS
    rec = pages * (2 * d * e + 8)                           # page records and their norms
    q8 = 2 * tokens * d + 2 * pages * 4                     # the 8-bit K and V and their scales
    blk = 2 * SG * c["B"] * d * e
    state = rows * (d + 1) * 4                              # one fp32 [rows][d] and [rows]
    if c["op"] == "write":
        return {"bytes": 2 * tokens * d * e + q8 + rec, "flops": 6 * 2 * tokens * d}
    if c["op"] == "append":
        t = SG * c["B"]                                     # the new tokens, and half a page of old
        new = 2 * (t + SG * PS / 2) * d
        return {"bytes": blk + new + 2 * SG * PS / 2 * d + (t / PS + SG) * (8 + 2 * d * e),
                "flops": 6 * new}
    if c["op"] == "read":
        return {"bytes": q8 + 2 * tokens * d * e, "flops": 2 * tokens * d}
    if c["op"] == "dense":
        keys = tokens * c["G"] * c["B"] + rows * c["B"]     # (row, key) pairs
        return {"bytes": q8 + rows * d * e + blk + 2 * state, "flops": 4 * keys * d}
    k = min(c["budget"] // PS, -(-c["L"] // PS))
    act = SG * c["G"] * c["A"]
    sel = min(act * k, pages) * PS                          # tokens of the selected pages
    pairs = act * pages * 4 * d + (act * k * PS + rows * c["B"]) * 4 * d
    return {"bytes": rec + 2 * sel * d + 2 * rows * d * e + blk + 2 * state + act * (d + 1) * 4,
            "flops": pairs}


def _mean_tokens(c):
    """Tokens of all sequences: a ragged batch's other lengths are uniform in [1, L]."""
    return c["L"] + (c["S"] - 1) * ((c["L"] + 1) / 2 if c["ragged"] else c["L"])


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _pages(n):
    return -(-n // PS)


def prepare(case, seed):
    """What a program holds before the call: the cache (or the prefix to write
    into it), queries, block and outputs, and the workspace.  Keys and values
    are N(0, 1), some keys lean on a direction that the queries share, and a few
    channels of K are larger than the rest, as they are in trained models."""
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    S, Hkv, G, L, B, cap = (c[x] for x in ("S", "Hkv", "G", "L", "B", "cap"))
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    Hq = Hkv * G

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    st = {"case": c, "scale": 1.0 / math.sqrt(D)}
    st["lens"] = None
    if c["ragged"]:
        lens = torch.randint(1, L + 1, (S,), generator=gen, device=dev, dtype=torch.int32)
        lens[torch.randint(0, S, (1,), generator=gen, device=dev)] = L
        st["lens"] = lens
    chan = torch.ones(D, device=dev)
    chan[torch.randperm(D, generator=gen, device=dev)[:4]] = 2.0
    u = randn(Hkv, D)
    u = u / u.norm(dim=-1, keepdim=True)
    Pc = _pages(cap)
    K = torch.zeros(S, Hkv, cap, D, device=dev, dtype=dt)
    V = torch.zeros(S, Hkv, cap, D, device=dev, dtype=dt)
    hot = min(64, L)
    for s in range(S):
        k = randn(Hkv, L, D) * chan
        pos = torch.randint(0, L, (Hkv, hot), generator=gen, device=dev)
        k.scatter_add_(1, pos[..., None].expand(-1, -1, D), (4.0 * u)[:, None].expand(-1, hot, -1))
        K[s, :, :L] = k.to(dt)
        V[s, :, :L] = randn(Hkv, L, D).to(dt)
    if c["op"] == "write":
        st.update(k=K, v=V, k8=torch.zeros(S, Hkv, cap, D, device=dev, dtype=F8),
                  v8=torch.zeros(S, Hkv, cap, D, device=dev, dtype=F8),
                  ks=torch.ones(S, Hkv, Pc, device=dev), vs=torch.ones(S, Hkv, Pc, device=dev),
                  meta=torch.zeros(_meta_bytes(c), device=dev, dtype=torch.uint8))
    else:
        ok = _valid(c, st["lens"], dev)
        st["k8"], st["ks"] = _encode(K, ok)
        st["v8"], st["vs"] = _encode(V, ok)
        if c["op"] in ("append", "step"):
            st["meta"] = torch.zeros(_meta_bytes(c), device=dev, dtype=torch.uint8)
            _write_records(c, _decode(st["k8"], st["ks"]), ok, st["meta"])
        if c["op"] == "read":
            st["k"], st["v"] = torch.zeros_like(K), torch.zeros_like(V)
    del K, V
    if c["op"] in ("append", "dense", "step"):
        st["kb"] = (randn(S, Hkv, B, D) * chan).to(dt)
        st["vb"] = randn(S, Hkv, B, D).to(dt)
    if c["op"] in ("dense", "step"):
        q = randn(S, Hq, B, D) + 0.5 * u.repeat_interleave(G, 0)[None, :, None]
        st.update(q=q.to(dt), o_p=torch.zeros(S, Hq, B, D, device=dev),
                  l_p=torch.zeros(S, Hq, B, device=dev), out=torch.zeros(S, Hq, B, D, device=dev),
                  lse=torch.zeros(S, Hq, B, device=dev))
    if c["op"] == "step":
        # the next step's queries: A tokens of each head move a lot, the others a little
        act = torch.argsort(torch.rand(S, Hq, B, generator=gen, device=dev), -1) < c["A"]
        st["q_prev"] = st["q"]
        st["q"] = (q + torch.where(act, 1.0, 0.01)[..., None] * randn(S, Hq, B, D)).to(dt)
        # the state that the block's first step left (any finite one is a valid input)
        st["o_p"] = 0.1 * randn(S, Hq, B, D)
        st["l_p"] = math.log(L) + 0.5 * randn(S, Hq, B).abs()
        k = min(c["budget"] // PS, _pages(L))
        st["act"] = torch.zeros(S, Hq, c["A"], device=dev, dtype=torch.int32)
        st["pages"] = torch.zeros(S, Hq, c["A"], k, device=dev, dtype=torch.int32)
        st["union"] = torch.zeros(S, Hkv, device=dev, dtype=torch.int32)
    if own:  # the handle and the workspace that a program makes once
        from sparse_long_context_mse_b200 import api
        st["shape"] = api.make_shape(S, Hq, Hkv, D, L, PS, B, c["A"], c["budget"], c["dtype"],
                                     prefix_capacity=cap, prefix_lens=st["lens"])
        if c["op"] == "dense":
            st["ws"] = api.alloc_workspace(st["shape"], api.LOSA_WS_DENSE_QUANT, dev)
        elif c["op"] == "step":
            st["ws"] = api.alloc_workspace(st["shape"], api.LOSA_WS_STEP, dev)
    return st


def _valid(c, lens, dev):
    """[S, 1, cap]: the tokens that a sequence has."""
    pos = torch.arange(c["cap"], device=dev)
    n = lens.long() if lens is not None else torch.full((c["S"],), c["L"], device=dev)
    return (pos < n[:, None])[:, None]


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _page_scale(amax):
    """The smallest power of two >= 2^-100 with amax <= 448 * it; 1 for a zero page."""
    m, e = torch.frexp(amax / E4M3_MAX)                      # amax / 448 = m 2^e, m in [1/2, 1)
    e = torch.where(m == 0.5, e - 1, e).clamp(-100, 119)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))


def _paged(x, fill=0):
    """[..., n, D] -> [..., pages, PS, D], the last page filled up."""
    n = x.shape[-2]
    x = torch.nn.functional.pad(x, (0, 0, 0, _pages(n) * PS - n), value=fill)
    return x.unflatten(-2, (-1, PS))


def _encode(x, ok):
    """(codes, scales) of x [S, H, n, D]; tokens that are not `ok` become code 0."""
    n = x.shape[-2]
    xp = _paged(torch.where(ok[..., None], x.float(), 0.0))
    s = _page_scale(xp.abs().amax((-1, -2)))
    return (xp / s[..., None, None]).to(F8).flatten(-3, -2)[..., :n, :].contiguous(), s


def _decode(x8, s):
    n = x8.shape[-2]
    return x8.float() * s.repeat_interleave(PS, -1)[..., :n, None]


def _meta_bytes(c):
    e = 4 if c["dtype"] == "f32" else 2
    Pc = _pages(c["cap"])
    return c["S"] * c["Hkv"] * (Pc * 2 * D * e + _pages8(Pc) * 8)


def _pages8(Pc):
    return -(-Pc // 8) * 8


def _meta_parts(c, meta):
    """The records [S, Hkv, Pc, 2 D] (16-byte chunks in stored order) and the norm
    pairs [S, Hkv, Pn, 2] of a metadata buffer, as views."""
    e, dt = (4, torch.float32) if c["dtype"] == "f32" else (2, torch.bfloat16)
    Pc = _pages(c["cap"])
    nr = c["S"] * c["Hkv"] * Pc * 2 * D * e
    return (meta[:nr].view(dt).view(c["S"], c["Hkv"], Pc, 2 * D),
            meta[nr:].view(torch.float32).view(c["S"], c["Hkv"], _pages8(Pc), 2))


def _swizzled(c, x, first=0):
    """Chunks of 16 bytes of a record [..., P, 2 D] in the order they are stored in:
    chunk j of page p stands at place j ^ (p & 7).  The order is its own inverse."""
    per = 4 if c["dtype"] == "f32" else 8                    # elements of a chunk
    n = 2 * D // per
    p = torch.arange(first, first + x.shape[-2], device=x.device)
    at = torch.arange(n, device=x.device)[None] ^ (p[:, None] & 7)
    x = x.unflatten(-1, (n, per))
    return x.gather(-2, at[..., None].expand(x.shape)).flatten(-2)


def _minmax(k, ok):
    """Per page and channel the least and the greatest key of its `ok` tokens."""
    okp = _paged(ok[..., None].expand(*ok.shape, 1))
    kp = _paged(k)
    return (torch.where(okp, kp, math.inf).amin(-2), torch.where(okp, kp, -math.inf).amax(-2),
            okp.any(-2))


def _write_records(c, k, ok, meta):
    lo, hi, has = _minmax(k, ok)
    rec, nrm = _meta_parts(c, meta)
    rec.copy_(torch.where(has, _swizzled(c, torch.cat((lo, hi), -1).to(rec.dtype)), rec))
    # the norms are upper bounds: the exact one, rounded up
    n = torch.stack((lo.double().norm(dim=-1), hi.double().norm(dim=-1)), -1)
    n = torch.where(has, n, 0.0)
    up = n.float()
    up = torch.where(up.double() < n, torch.nextafter(up, torch.full_like(up, math.inf)), up)
    nrm[:, :, :up.shape[2]] = torch.where(has, up, nrm[:, :, :up.shape[2]])


def _plain_write(st):
    c = st["case"]
    ok = _valid(c, st["lens"], st["k"].device)
    for x, x8, s in ((st["k"], st["k8"], st["ks"]), (st["v"], st["v8"], st["vs"])):
        codes, scale = _encode(x, ok)
        x8.copy_(codes)
        s.copy_(scale)
    _write_records(c, _decode(st["k8"], st["ks"]), ok, st["meta"])


def _plain_append(st):
    c, dev = st["case"], st["kb"].device
    S, Hkv, B, cap = c["S"], c["Hkv"], c["B"], c["cap"]
    n = st["lens"].long() if st["lens"] is not None else torch.full((S,), c["L"], device=dev)
    # the pages that positions n .. n + B - 1 touch, as [S, pages]; one past the cache's end
    # stands for a page that this sequence does not touch
    p = n[:, None] // PS + torch.arange(_pages(B - 1) + 1, device=dev)
    mine = p <= (n[:, None] + B - 1) // PS
    pos = (p[..., None] * PS + torch.arange(PS, device=dev)).flatten(1)           # [S, tokens]
    ok = (pos < n[:, None] + B)[:, None]
    old = pos < n[:, None]
    at = pos.clamp(max=cap - 1)[:, None, :, None].expand(S, Hkv, -1, D)
    fr = (pos - n[:, None]).clamp(0, B - 1)[:, None, :, None].expand(S, Hkv, -1, D)
    sat = p.clamp(max=_pages(cap) - 1)[:, None].expand(S, Hkv, -1)
    w = (ok[:, 0] & mine.repeat_interleave(PS, 1)).nonzero(as_tuple=True)
    wp = mine.nonzero(as_tuple=True)
    for blk, x8, s in ((st["kb"], st["k8"], st["ks"]), (st["vb"], st["v8"], st["vs"])):
        bytes8 = x8.view(torch.uint8)
        was = bytes8.gather(2, at).view(F8).float() * s.gather(2, sat).repeat_interleave(PS, -1)[..., None]
        x = torch.where(old[:, None, :, None], was, blk.float().gather(2, fr))
        codes, scale = _encode(x, ok)
        bytes8[w[0], :, pos[w]] = codes.view(torch.uint8)[w[0], :, w[1]]
        s[wp[0], :, p[wp]] = scale[wp[0], :, wp[1]]
        if blk is st["kb"]:
            lo, hi, _ = _minmax(_decode(codes, scale), ok)
    rec, nrm = _meta_parts(c, st["meta"])
    r = torch.cat((lo, hi), -1).to(rec.dtype)[wp[0], :, wp[1]]                     # [touched, Hkv, 2 D]
    per = 4 if c["dtype"] == "f32" else 8
    chunks = 2 * D // per
    place = torch.arange(chunks, device=dev)[None] ^ (p[wp][:, None] & 7)
    r = r.unflatten(-1, (chunks, per))
    rec[wp[0], :, p[wp]] = r.gather(2, place[:, None, :, None].expand(r.shape)).flatten(-2)
    nn = torch.stack((lo.double().norm(dim=-1), hi.double().norm(dim=-1)), -1)[wp[0], :, wp[1]]
    nrm[wp[0], :, p[wp]] = nn.float()


def _plain_read(st):
    ok = _valid(st["case"], st["lens"], st["k"].device)[..., None]
    for x, x8, s in ((st["k"], st["k8"], st["ks"]), (st["v"], st["v8"], st["vs"])):
        x.copy_(torch.where(ok, _decode(x8, s).to(x.dtype), x))


def _attend(s, v):
    """Softmax of the scores s [..., n] over the values v [..., n, D]: output and
    log-normaliser."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / l, (m + torch.log(l)).squeeze(-1)


def _merge(o1, l1, o2, l2):
    m = torch.maximum(l1, l2)
    a, b = torch.exp(l1 - m), torch.exp(l2 - m)
    return (a[..., None] * o1 + b[..., None] * o2) / (a + b)[..., None], m + torch.log(a + b)


def _grouped(x, Hkv):
    """[S, Hq, ...] -> [S, Hkv, G, ...]"""
    return x.unflatten(1, (Hkv, -1))


def _suffix(st, q):
    c = st["case"]
    qg = _grouped(q, c["Hkv"]).flatten(2, 3)                                       # [S, Hkv, G B, D]
    o, l = _attend(torch.matmul(qg, st["kb"].float().transpose(-1, -2)) * st["scale"], st["vb"].float())
    return o.view(q.shape), l.view(q.shape[:-1])


def _plain_dense(st):
    c = st["case"]
    q = st["q"].float()
    ok = _valid(c, st["lens"], q.device)[:, :, None]
    qg = _grouped(q, c["Hkv"]).flatten(2, 3)
    # zeros past a sequence's end, so that 0 times whatever stands there is 0
    k = torch.where(ok.transpose(-1, -2), _decode(st["k8"], st["ks"]), 0.0)
    v = torch.where(ok.transpose(-1, -2), _decode(st["v8"], st["vs"]), 0.0)
    s = torch.matmul(qg, k.transpose(-1, -2)) * st["scale"]
    del k
    o, l = _attend(torch.where(ok, s, -math.inf), v)
    o, l = o.view(q.shape), l.view(q.shape[:-1])
    out, lse = _merge(o, l, *_suffix(st, q))
    for to, x in (("o_p", o), ("l_p", l), ("out", out), ("lse", lse)):
        st[to].copy_(x)


def _top(key, n):
    """The n largest, ties to the lower index, in ascending index order."""
    return torch.sort(key + 0.0, dim=-1, descending=True, stable=True).indices[..., :n].sort(-1).values


def _plain_step(st):
    c = st["case"]
    S, Hkv, G, L, B, A = (c[x] for x in ("S", "Hkv", "G", "L", "B", "A"))
    dev, P = st["q"].device, _pages(L)
    k = min(c["budget"] // PS, P)
    q = st["q"].float()
    mse = (q - st["q_prev"].float()).double().square().mean(-1)
    act = _top(mse, A)                                                             # [S, Hq, A]
    rows = act[..., None].expand(*act.shape, D)
    qa = _grouped(q.gather(2, rows), Hkv).flatten(2, 3)                            # [S, Hkv, G A, D]
    rec, _ = _meta_parts(c, st["meta"])
    rec = _swizzled(c, rec[:, :, :P]).float()
    lo, hi = rec[..., :D].transpose(-1, -2), rec[..., D:].transpose(-1, -2)        # [S, Hkv, D, P]
    # the bound that ranks the pages is defined in fp32, its channels added in order: pages
    # whose exact bounds nearly tie are ranked by that sum
    U = torch.zeros(S, Hkv, G * A, P, device=dev)
    for i in range(D):
        x = qa[..., i, None]
        U = U + torch.maximum(x * hi[:, :, None, i], x * lo[:, :, None, i])
    n = st["lens"].long() if st["lens"] is not None else torch.full((S,), L, device=dev)
    np_ = -(-n // PS)
    has = (torch.arange(P, device=dev) < np_[:, None])[:, None, None]
    pages = _top(torch.where(has, U, -math.inf), k)                                # [S, Hkv, G A, k]
    real = pages < np_[:, None, None, None]
    tok = (pages[..., None] * PS + torch.arange(PS, device=dev)).flatten(-2)       # [S, Hkv, G A, k PS]
    seen = tok < n[:, None, None, None]
    flat = tok.clamp(max=c["cap"] - 1).flatten(2)

    def gather(x8, s):
        b = x8.view(torch.uint8).gather(2, flat[..., None].expand(-1, -1, -1, D)).view(F8).float()
        b = b * s.gather(2, flat // PS)[..., None]
        return torch.where(seen.flatten(2)[..., None], b, 0.0).unflatten(2, (G * A, -1))

    s = torch.matmul(gather(st["k8"], st["ks"]), qa[..., None]).squeeze(-1) * st["scale"]
    o, l = _attend(torch.where(seen, s, -math.inf)[..., None, :], gather(st["v8"], st["vs"]))
    st["o_p"].scatter_(2, rows, o.reshape(S, Hkv * G, A, D))
    st["l_p"].scatter_(2, act, l.reshape(S, Hkv * G, A))
    out, lse = _merge(st["o_p"], st["l_p"], *_suffix(st, q))
    hit = torch.zeros(S, Hkv, P + 1, device=dev, dtype=torch.int32)
    hit.scatter_(2, torch.where(real, pages, P).flatten(2), 1)
    st["out"].copy_(out)
    st["lse"].copy_(lse)
    st["act"].copy_(act)
    st["pages"].copy_(torch.where(real, pages, -1).reshape(st["pages"].shape))
    st["union"].copy_(hit[..., :P].sum(-1))


_PLAIN = {"write": _plain_write, "append": _plain_append, "read": _plain_read,
          "dense": _plain_dense, "step": _plain_step}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own(st):
    from sparse_long_context_mse_b200 import api
    op, sh = st["case"]["op"], st["shape"]
    if op == "write":
        api.quantize_prefix(sh, st["k"], st["v"], st["k8"], st["v8"], st["ks"], st["vs"], st["meta"])
    elif op == "append":
        api.append_block_quant(sh, st["kb"], st["vb"], st["k8"], st["v8"], st["ks"], st["vs"],
                               st["meta"])
    elif op == "read":
        api.dequantize_prefix(sh, st["k8"], st["v8"], st["ks"], st["vs"], st["k"], st["v"])
    elif op == "dense":
        api.dense_prefix_quant(sh, st["q"], st["k8"], st["v8"], st["ks"], st["vs"], st["kb"],
                               st["vb"], st["o_p"], st["l_p"], st["out"], st["lse"], st["ws"])
    else:
        api.step_quant(sh, st["q"], st["q_prev"], st["k8"], st["v8"], st["ks"], st["vs"],
                       st["meta"], st["kb"], st["vb"], st["o_p"], st["l_p"], st["out"], st["lse"],
                       st["ws"], st["act"], st["pages"], st["union"])


_OUTPUTS = {"write": ("k8", "ks", "v8", "vs"), "append": ("k8", "ks", "v8", "vs"),
            "read": ("k", "v"), "dense": ("o_p", "l_p", "out", "lse"),
            "step": ("o_p", "l_p", "out", "lse", "act", "pages", "union")}


def run(state):
    if own:
        _own(state)
    else:
        _PLAIN[state["case"]["op"]](state)
    got = {n: state[n] for n in _OUTPUTS[state["case"]["op"]]}
    if state["case"]["op"] in ("write", "append"):
        got["records"], got["norms"] = _meta_parts(state["case"], state["meta"])
    return got


# ---------------------------------------------------------------------------
# 64 bits, from the definition
# ---------------------------------------------------------------------------
def _exact_codes(x):
    """(values in units of the scale, scale) of one page x [n, D] in 64 bits: e4m3
    has steps of 2^(e - 3) in [2^e, 2^(e + 1)), and of 2^-9 below 2^-6."""
    amax = float(x.abs().max()) if x.numel() else 0.0
    e = -100
    while amax > E4M3_MAX * 2.0 ** e:
        e += 1
    scale = 2.0 ** e if amax > 0 else 1.0
    y = x / scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, scale


def _exact_encode_all(x, lens):
    """The same for every page of x [S, H, cap, D], pages at once."""
    S, H, cap, _ = x.shape
    ok = torch.arange(cap, device=x.device)[None, None, :, None] < lens.view(S, 1, 1, 1)
    x = torch.nn.functional.pad(x.double() * ok, (0, 0, 0, _pages(cap) * PS - cap))
    x = x.view(S, H, -1, PS, D)
    amax = x.abs().flatten(-2).max(-1).values
    scale = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(-100, 119))
    # (a logarithm that was rounded across a whole number)
    scale = torch.where((scale > 2.0 ** -100) & (amax <= E4M3_MAX / 2 * scale), scale / 2, scale)
    scale = torch.where(amax > E4M3_MAX * scale, 2 * scale, scale)
    scale = torch.where(amax > 0, scale, torch.ones_like(scale))
    y = x / scale[..., None, None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).view(S, H, -1, D)[:, :, :cap], scale


def _exact_rec(c, meta, x, lens, first_page=None):
    """Records and norms of the cached keys x [S, H, cap, D] in 64 bits, laid out as
    stored; pages that a sequence does not have keep what `meta` holds."""
    rec, nrm = (t.double() for t in _meta_parts(c, meta))
    S, H, cap, _ = x.shape
    per = 4 if c["dtype"] == "f32" else 8
    x = torch.nn.functional.pad(x, (0, 0, 0, _pages(cap) * PS - cap)).view(S, H, -1, PS, D)
    j = torch.arange(2 * D, device=x.device)
    for s in range(S):
        n = int(lens[s])
        for p0 in range(0 if first_page is None else first_page[s], _pages(n), 512):
            p1 = min(_pages(n), p0 + 512)
            page = torch.arange(p0, p1, device=x.device)
            tok = page[:, None] * PS + torch.arange(PS, device=x.device)
            out = (tok >= n)[None, :, :, None]
            lo = x[s, :, p0:p1].masked_fill(out, math.inf).min(2).values
            hi = x[s, :, p0:p1].masked_fill(out, -math.inf).max(2).values
            both = torch.cat((lo, hi), -1)
            src = ((j[None] // per) ^ (page[:, None] & 7)) * per + j[None] % per
            rec[s, :, p0:p1] = both.gather(-1, src.expand(H, -1, -1))
            nrm[s, :, p0:p1, 0] = lo.square().sum(-1).sqrt()
            nrm[s, :, p0:p1, 1] = hi.square().sum(-1).sqrt()
    return rec, nrm


def _exact_bounds(q, lo, hi):
    """The pages' bounds for one query row q [D]: fp32 by definition, each product and
    each partial sum rounded once (64-bit sums of 32-bit numbers, rounded)."""
    a = (q * hi).float().double()                                                  # [P, D]
    b = (q * lo).float().double()
    t = torch.where(a > b, a, b)
    acc = torch.zeros(t.shape[0], device=q.device, dtype=torch.float64)
    for i in range(D):
        acc = (acc + t[:, i]).float().double()
    return acc


def exact(case, seed):
    c, st = case, prepare(case, seed)
    S, Hkv, G, B, cap = (c[x] for x in ("S", "Hkv", "G", "B", "cap"))
    first = st.get("k8")
    dev = first.device
    lens = st["lens"].long() if st["lens"] is not None else torch.full((S,), c["L"], device=dev)
    up = None
    if "ks" in st:
        up = lambda s: torch.repeat_interleave(s.double(), PS, 2)[:, :, :cap, None]  # noqa: E731
    if c["op"] == "write":
        (k8, ks), (v8, vs) = (_exact_encode_all(st[n], lens) for n in ("k", "v"))
        rec, nrm = _exact_rec(c, st["meta"], k8 * up(ks), lens)
        return {"k8": k8, "ks": ks, "v8": v8, "vs": vs, "records": rec, "norms": nrm}
    if c["op"] == "append":
        got = {}
        for n8, ns, nb in (("k8", "ks", "kb"), ("v8", "vs", "vb")):
            x, sc = st[n8].double(), st[ns].double()
            for s in range(S):
                n = int(lens[s])
                p0 = n // PS
                for h in range(Hkv):
                    old = x[s, h, p0 * PS:n] * sc[s, h, p0] if n % PS else x[s, h, n:n]
                    new = torch.cat((old, st[nb][s, h].double()))
                    for i in range(0, len(new), PS):
                        y, e = _exact_codes(new[i:i + PS])
                        x[s, h, p0 * PS + i:p0 * PS + i + len(y)] = y
                        sc[s, h, p0 + i // PS] = e
            got[n8], got[ns] = x, sc
        got["records"], got["norms"] = _exact_rec(c, st["meta"], got["k8"] * up(got["ks"]), lens + B,
                                                  [int(n) // PS for n in lens])
        return got
    if c["op"] == "read":
        ok = torch.arange(cap, device=dev)[None, None, :, None] < lens.view(S, 1, 1, 1)
        return {n: st[n + "8"].double() * up(st[n + "s"]) * ok for n in ("k", "v")}
    if c["op"] == "dense":
        got = {n: torch.empty(st[n].shape, device=dev, dtype=torch.float64) for n in ("o_p", "l_p", "out", "lse")}
        for s in range(S):
            n = int(lens[s])
            for g in range(Hkv):
                scale = lambda x: torch.repeat_interleave(x[s, g].double(), PS)[:n, None]  # noqa: E731
                K = torch.cat((st["k8"][s, g, :n].double() * scale(st["ks"]), st["kb"][s, g].double()))
                V = torch.cat((st["v8"][s, g, :n].double() * scale(st["vs"]), st["vb"][s, g].double()))
                h = slice(g * G, (g + 1) * G)
                w = torch.einsum("hbd,nd->hbn", st["q"][s, h].double(), K) * st["scale"]
                got["l_p"][s, h] = torch.logsumexp(w[..., :n], -1)
                got["lse"][s, h] = torch.logsumexp(w, -1)
                got["o_p"][s, h] = torch.softmax(w[..., :n], -1) @ V[:n]
                got["out"][s, h] = torch.softmax(w, -1) @ V
        return got
    # step: row by row
    got = {n: st[n].double() for n in ("o_p", "l_p")}
    got.update({n: torch.empty(st[n].shape, device=dev, dtype=torch.float64) for n in ("out", "lse")})
    got.update(act=None, pages=None, union=None)
    if S * Hkv * G * c["A"] > 1024:
        return None
    rec = _meta_parts(c, st["meta"])[0]
    per = 4 if c["dtype"] == "f32" else 8
    j = torch.arange(2 * D, device=dev)
    diff = (st["q"].double() - st["q_prev"].double()).square().sum(-1)
    for s in range(S):
        n = int(lens[s])
        P = _pages(n)
        page = torch.arange(P, device=dev)
        src = ((j[None] // per) ^ (page[:, None] & 7)) * per + j[None] % per
        for g in range(Hkv):
            r = rec[s, g, :P].double().gather(-1, src)
            Kb, Vb = st["kb"][s, g].double(), st["vb"][s, g].double()
            for h in range(g * G, (g + 1) * G):
                for t in torch.topk(diff[s, h], c["A"]).indices.tolist():
                    q = st["q"][s, h, t].double()
                    U = _exact_bounds(q, r[:, :D], r[:, D:])
                    k = min(c["budget"] // PS, P)
                    sel = torch.sort(U, descending=True, stable=True).indices[:k]
                    tok = (sel[:, None] * PS + torch.arange(PS, device=dev)).flatten()
                    tok = tok[tok < n]
                    K = st["k8"][s, g].view(torch.uint8)[tok].view(F8).double() * st["ks"][s, g, tok // PS, None].double()
                    V = st["v8"][s, g].view(torch.uint8)[tok].view(F8).double() * st["vs"][s, g, tok // PS, None].double()
                    w = (K @ q) * st["scale"]
                    got["o_p"][s, h, t] = torch.softmax(w, 0) @ V
                    got["l_p"][s, h, t] = torch.logsumexp(w, 0)
                # every row of the head: its prefix state and the block's keys
                w = (st["q"][s, h].double() @ Kb.T) * st["scale"]                  # [B, B]
                lse = torch.logsumexp(torch.cat((got["l_p"][s, h, :, None], w), -1), -1)
                got["out"][s, h] = (torch.exp(got["l_p"][s, h] - lse)[:, None] * got["o_p"][s, h]
                                    + torch.exp(w - lse[:, None]) @ Vb)
                got["lse"][s, h] = lse
    return got
