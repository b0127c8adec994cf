"""Attention over the 8-bit prefix cache: the dense pass against its 64-bit
formula, the step against the step over the read-back prefix (the same selections
and weights), 64 bits and the oracle, and a whole block's life -- write, dense pass,
steps, append, next block."""
import threading

import numpy as np
import pytest
import torch

import oracle
from losa_testutil import (DEV, TOL, gpu_dense, gpu_meta, gpu_step, maxabs,
                           oshape, random_case, scale_of, unswizzle_page_meta)
from quant_testutil import (F8, alloc_state, check_dense, dense_reference, f64, gpu_dense_quant,
                            random_prefix, read_back)
from sparse_long_context_mse_b200 import api

pytestmark = pytest.mark.gpu


def inputs(dtype, lens, Hkv, G, B, cap=0, seed=0, amp=1.0, A=0, budget=0, flags=0):
    """A shape, its quantised prefix (NaN past every sequence's length), its metadata,
    queries and block."""
    gen = torch.Generator().manual_seed(seed)
    t = torch.tensor(lens, dtype=torch.int32, device=DEV) if len(set(lens)) > 1 else None
    S, Hq = len(lens), Hkv * G
    sh = api.make_shape(S, Hq, Hkv, 128, max(lens), 16, B, A, budget, dtype, scale=scale_of(128),
                        prefix_capacity=cap, prefix_lens=t, flags=flags)
    K, V = random_prefix(sh, gen, DEV, amp=amp)
    cache = api.alloc_quant_prefix(sh, DEV)
    for x in cache[:2]:
        x.view(torch.uint8).fill_(0x7F)  # NaN
    for x in cache[2:]:
        x.fill_(float("nan"))
    meta = api.alloc_page_meta(sh, DEV)
    meta.fill_(0x5A)
    api.quantize_prefix(sh, K, V, *cache, meta)
    dt = sh.torch_dtype
    r = lambda *shape: torch.randn(*shape, generator=gen)
    q = [r(S, Hq, B, 128)]
    drift = torch.full((S, Hq, B, 1), 0.01)
    for s in range(S):
        for h in range(Hq):
            drift[s, h, torch.randperm(B, generator=gen)[:A]] = 1.0
    q.append(q[0] + drift * r(S, Hq, B, 128))
    q = [x.to(dt).to(DEV) for x in q]
    kb, vb = (r(S, Hkv, B, 128).to(dt).to(DEV) for _ in range(2))
    return sh, cache, meta, q, kb, vb


def dense_case(sh, cache, q, kb, vb, what=""):
    ws = api.alloc_workspace(sh, api.LOSA_WS_DENSE_QUANT, DEV)
    got = gpu_dense_quant(sh, q, cache, kb, vb, ws)
    assert api.read_device_status(ws) == api.LOSA_OK, what
    ref, bounds = dense_reference(sh, q, *cache, kb, vb)
    check_dense(got, ref, bounds, what)
    return got, ref, bounds


# rows of a KV head from 1 to 128, lengths from one token to many tiles, pages and tiles
# that end inside, ragged batches
DENSE = [("bf16", [1], 1, 1, 1), ("bf16", [16], 1, 1, 16), ("bf16", [127], 2, 4, 16),
         ("bf16", [128], 2, 4, 16), ("bf16", [129], 2, 4, 16), ("bf16", [2000], 2, 4, 1),
         ("bf16", [2000], 1, 8, 16), ("bf16", [2047], 1, 4, 32), ("bf16", [5000], 2, 1, 5),
         ("bf16", [5000], 1, 2, 31), ("bf16", [333], 8, 8, 2), ("f32", [1], 1, 1, 16),
         ("f32", [2048], 1, 1, 16), ("f32", [777], 2, 8, 16), ("f32", [1500], 2, 4, 1),
         ("bf16", [1000, 37, 1, 513], 2, 4, 16), ("f32", [1000, 37, 1, 513], 2, 4, 8),
         ("bf16", [3000, 1, 2, 2999, 129, 17, 128], 4, 8, 1), ("bf16", [4096], 8, 4, 32),
         ("bf16", [700, 41], 3, 5, 7)]


@pytest.mark.parametrize("dtype,lens,Hkv,G,B", DENSE)
def test_dense(dtype, lens, Hkv, G, B):
    sh, cache, _, q, kb, vb = inputs(dtype, lens, Hkv, G, B, cap=max(lens) + 5, seed=sum(lens) + B)
    dense_case(sh, cache, q[0], kb, vb)


@pytest.mark.parametrize("dtype,G,B", [("bf16", 4, 16), ("bf16", 4, 1), ("bf16", 8, 16), ("f32", 4, 16)])
def test_dense_long(dtype, G, B):
    """Many tiles for each CTA, and CTAs that cross from one KV head into the next."""
    sh, cache, _, q, kb, vb = inputs(dtype, [20000, 9001, 16384], 8, G, B, cap=20011, seed=21)
    dense_case(sh, cache, q[0], kb, vb)


@pytest.mark.parametrize("S,Hkv,G,B", [(70, 1, 4, 4), (33, 3, 2, 1), (150, 2, 1, 1)])
def test_dense_many_sequences(S, Hkv, G, B):
    """More sequences than a warp has lanes, and more KV heads than CTAs: the CTAs' places
    among the tiles come from sums over all lengths."""
    g = torch.Generator().manual_seed(S)
    lens = torch.randint(1, 700, (S,), generator=g).tolist()
    lens[S // 2] = 1500
    sh, cache, _, q, kb, vb = inputs("bf16", lens, Hkv, G, B, cap=1511, seed=S)
    dense_case(sh, cache, q[0], kb, vb)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dense_rows_of_different_sizes(dtype):
    """Query rows and parts of rows of very different sizes, in one head."""
    sh, cache, _, q, kb, vb = inputs(dtype, [900], 2, 4, 16, seed=32)
    g = torch.Generator().manual_seed(33)
    size = torch.exp2(torch.randint(-24, 3, (1, 8, 16, 1), generator=g).float())
    dense_case(sh, cache, (q[0].cpu().float() * size).to(sh.torch_dtype).to(DEV), kb, vb)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dense_growing_scores(dtype):
    """Scores that rise along the prefix, so that the running maximum moves many times,
    and large ones, whose softmax is one key."""
    sh, cache, _, q, kb, vb = inputs(dtype, [3001], 2, 4, 16, seed=31)
    k = torch.randn(1, 2, 3001, 128, generator=torch.Generator().manual_seed(1))
    k *= torch.linspace(0.1, 6.0, 3001)[None, None, :, None]
    v = torch.randn(1, 2, 3001, 128, generator=torch.Generator().manual_seed(2))
    api.quantize_prefix(sh, k.to(sh.torch_dtype).to(DEV), v.to(sh.torch_dtype).to(DEV), *cache)
    dense_case(sh, cache, q[0], kb, vb)
    big = torch.zeros(1, 2, 3001, 128)
    big[:, :, 2000] = 40.0
    api.quantize_prefix(sh, (k + big).to(sh.torch_dtype).to(DEV), v.to(sh.torch_dtype).to(DEV), *cache)
    dense_case(sh, cache, q[0], kb, vb)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dense_other_scales(dtype):
    """Scales that are no powers of two, of very different sizes from page to page, a
    negative K scale, V scales of zero, and values whose weight is elsewhere."""
    sh, cache, _, q, kb, vb = inputs(dtype, [1200, 455], 2, 4, 8, seed=41)
    g = torch.Generator().manual_seed(7)
    P = sh.capacity_pages
    cache[2].copy_((torch.randn(2, 2, P, generator=g) * 0.02).to(DEV))
    vs = torch.exp2(torch.randint(-30, 4, (2, 2, P), generator=g).float()) * 1.3
    vs[:, :, 3::5] = 0.0
    cache[3].copy_(vs.to(DEV))
    got, ref, bounds = dense_case(sh, cache, q[0], kb, vb)
    # where almost all the weight is on one page with small values, the output keeps
    # its relative accuracy: the bounds scale with that page's values
    cache[2].fill_(0.0)
    cache[2][:, :, 5] = 100.0
    cache[3].fill_(2.0 ** -8)
    cache[3][:, :, 5] = 2.0 ** -40
    qq = torch.ones_like(q[0])
    c5 = torch.zeros(2, 2, 16, 128, device=DEV)
    c5[:, :, 0] = 1.0
    cache[0].view(torch.uint8)[:, :, 80:96] = c5.to(F8).view(torch.uint8)
    got = gpu_dense_quant(sh, qq, cache, kb, vb)
    ref, _ = dense_reference(sh, qq, *cache, kb, vb)
    a, b = got["o_p"].cpu().double(), ref["o_p"]
    assert b.abs().max() < 1e-9 and (a - b).abs().max() <= 2.0 ** -14 * b.abs().max()


@pytest.mark.parametrize("dtype,lens,Hkv,G,B,outlier", [
    ("bf16", [3], 2, 1, 1, 1), ("bf16", [95, 60], 2, 8, 2, 1), ("bf16", [5000], 2, 4, 16, 1),
    ("f32", [700], 2, 4, 8, 1), ("bf16", [400], 2, 4, 16, 60), ("f32", [400], 2, 4, 4, 60)])
def test_dense_error_against_64_bits(dtype, lens, Hkv, G, B, outlier):
    """Relative to the results' norm.  Scores of N(0, 1) queries and keys are below 2^3 in
    base 2, those of rows with one channel 60 times larger below 2^7; the tensor core rounds
    them (16 accumulations of at most 2^-24 of that: 2^-17 and 2^-13 in the worst case), and
    the split of a row leaves 2^-21 of its maximum in a few channels, the less.  Independent
    roundings add as squares: an eighth of the worst case, 2^-20 and 2^-16."""
    sh, cache, _, q, kb, vb = inputs(dtype, lens, Hkv, G, B, seed=sum(lens))
    q[0][..., 5] *= outlier
    got, ref, _ = dense_case(sh, cache, q[0], kb, vb)
    for key in ("o_p", "out"):
        err = ((got[key].cpu().double() - ref[key]).norm() / ref[key].norm()).item()
        assert err <= (2.0 ** -20 if outlier == 1 else 2.0 ** -16), (key, err)


def test_dense_zero_and_tiny_queries():
    sh, cache, _, q, kb, vb = inputs("bf16", [500], 2, 4, 16, seed=51)
    q0 = q[0].clone()
    q0[:, :, 0] = 0.0
    q0[:, :, 1] *= 1e-30
    q0[:, :, 2, :64] *= 2.0 ** -12
    q0[:, :, 3, 5] = 1000.0
    dense_case(sh, cache, q0, kb, vb)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dense_huge_scores(dtype):
    """Scores so large that a unit is lost in their rounding: the softmax is one key, its
    value the output, and the log-normaliser its score (to 2^-20 of it: a product of
    exact numbers and three roundings)."""
    sh, cache, _, q, kb, vb = inputs(dtype, [700], 2, 2, 8, seed=52)
    k = torch.zeros(1, 2, 700, 128)
    k[:, :, 333] = 2.0 ** 24
    k[:, :, 500] = 2.0 ** 10
    v = torch.randn(1, 2, 700, 128, generator=torch.Generator().manual_seed(3))
    api.quantize_prefix(sh, k.to(sh.torch_dtype).to(DEV), v.to(sh.torch_dtype).to(DEV), *cache)
    qq = torch.full_like(q[0], 8.0)
    got = gpu_dense_quant(sh, qq, cache, kb, vb)
    ref, _ = dense_reference(sh, qq, *cache, kb, vb)
    want = read_back(cache[1], cache[3])[0, :, 333]
    for key in ("o_p", "out"):
        g = got[key].double().reshape(2, 16, 128)
        assert (g - want[:, None]).abs().max().item() <= 2.0 ** -20 * 8
    for key in ("l_p", "lse"):
        assert ((got[key].cpu().double() - ref[key]) / ref[key]).abs().max().item() <= 2.0 ** -20
    # and so small that all keys weigh the same
    got = gpu_dense_quant(sh, qq * 2.0 ** -60, cache, kb, vb)
    ref, _ = dense_reference(sh, qq * 2.0 ** -60, *cache, kb, vb)
    assert (got["o_p"].cpu().double() - ref["o_p"]).abs().max().item() <= 2.0 ** -18 * 5


def test_dense_matches_the_pass_over_the_read_back_prefix():
    sh, cache, _, q, kb, vb = inputs("bf16", [4000], 2, 4, 16, seed=61)
    got = gpu_dense_quant(sh, q[0], cache, kb, vb)
    K, V = (torch.zeros(1, 2, 4000, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    api.dequantize_prefix(sh, *cache, K, V)
    ref = gpu_dense(sh, q[0], K, V, kb, vb)
    for key in ("o_p", "l_p", "out", "lse"):
        assert maxabs(got[key].cpu().numpy(), ref[key].cpu().numpy()) <= TOL, key


def test_dense_bad_lengths_are_reported():
    """Lengths outside [1, L] are clamped and reported, as in losa_dense_prefix."""
    sh, cache, _, q, kb, vb = inputs("bf16", [300, 200], 2, 4, 16, seed=71)
    for t in cache[:2]:
        t.view(torch.uint8).fill_(0x38)
    for t in cache[2:]:
        t.fill_(1.0)
    ws = api.alloc_workspace(sh, api.LOSA_WS_DENSE_QUANT, DEV)
    sh._prefix_lens.copy_(torch.tensor([301, 0]))
    got = gpu_dense_quant(sh, q[0], cache, kb, vb, ws)
    assert api.read_device_status(ws) == api.LOSA_ERR_DEVICE_BOUNDS
    sh._prefix_lens.copy_(torch.tensor([300, 1]))
    ref, bounds = dense_reference(sh, q[0], *cache, kb, vb)
    check_dense(got, ref, bounds)
    gpu_dense_quant(sh, q[0], cache, kb, vb, ws)
    assert api.read_device_status(ws) == api.LOSA_OK


def test_dense_same_bits_again_and_with_a_used_workspace():
    sh, cache, _, q, kb, vb = inputs("bf16", [5000, 801], 4, 4, 16, seed=81)
    ws = api.alloc_workspace(sh, api.LOSA_WS_DENSE_QUANT, DEV)
    a = gpu_dense_quant(sh, q[0], cache, kb, vb, ws)
    ws[256:].fill_(0xFF)
    b = gpu_dense_quant(sh, q[0], cache, kb, vb, ws)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_dense_captured_two_streams_and_replay():
    """Two calls at once on two streams with their own workspaces, and a captured call
    replayed on other inputs and lengths."""
    cases = [inputs("bf16", [3000, 1700], 4, 4, 16, seed=91), inputs("bf16", [2500, 60], 2, 8, 1, seed=92)]
    st = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for (sh, cache, _, q, kb, vb), s in zip(cases, st):
        with torch.cuda.stream(s):
            ws = api.alloc_workspace(sh, api.LOSA_WS_DENSE_QUANT, DEV)
            got.append(gpu_dense_quant(sh, q[0], cache, kb, vb, ws))
    torch.cuda.synchronize()
    for (sh, cache, _, q, kb, vb), r in zip(cases, got):
        check_dense(r, *dense_reference(sh, q[0], *cache, kb, vb))
    sh, cache, _, q, kb, vb = cases[0]
    ws = api.alloc_workspace(sh, api.LOSA_WS_DENSE_QUANT, DEV)
    out = alloc_state(sh, torch.device(DEV))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.dense_prefix_quant(sh, q[0], *cache, kb, vb, out["o_p"], out["l_p"], out["out"], out["lse"], ws)
    q[0].copy_(q[1])
    sh._prefix_lens.copy_(torch.tensor([777, 1700]))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    check_dense(out, *dense_reference(sh, q[0], *cache, kb, vb))


@pytest.mark.parametrize("B", [1, 16])
def test_dense_calls_queued_behind_the_kernels_that_write_their_inputs(B):
    """Every call's queries, block and cache are written on the stream just before it, and
    its results and workspace are used again just after it, with no wait between."""
    cases = [inputs("bf16", [2500, 900], 2, 4, B, cap=2600, seed=97 + i) for i in range(6)]
    sh = cases[0][0]
    for other in cases[1:]:
        sh_i = other[0]
        assert [int(x) for x in sh_i._prefix_lens] == [int(x) for x in sh._prefix_lens]
    cache = api.alloc_quant_prefix(sh, DEV)
    q, kb, vb = (torch.empty_like(x) for x in (cases[0][3][0], *cases[0][4:]))
    ws = api.alloc_workspace(sh, api.LOSA_WS_DENSE_QUANT, DEV)
    out = alloc_state(sh, torch.device(DEV))
    got = []
    torch.cuda.synchronize()
    for _, c, _, qs, k, v in cases:
        for dst, src in zip((*cache, q, kb, vb), (*c, qs[0], k, v)):
            dst.copy_(src)
        for _ in range(2):  # (the second one's inputs are the first one's)
            api.dense_prefix_quant(sh, q, *cache, kb, vb, out["o_p"], out["l_p"], out["out"], out["lse"], ws)
        got.append({n: x.clone() for n, x in out.items()})
    for r, (_, c, _, qs, k, v) in zip(got, cases):
        check_dense(r, *dense_reference(sh, qs[0], *c, k, v))


def test_dense_from_two_threads():
    """Python threads, each with its own stream, tensors and workspace."""
    cases = [inputs("bf16", [1500, 60], 2, 4, 16, seed=111), inputs("bf16", [900], 2, 8, 1, seed=112)]
    got = [[], []]
    torch.cuda.synchronize()

    def work(i):
        sh, cache, _, q, kb, vb = cases[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            ws = api.alloc_workspace(sh, api.LOSA_WS_DENSE_QUANT, DEV)
            for _ in range(50):
                got[i].append(gpu_dense_quant(sh, q[0], cache, kb, vb, ws))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i, (sh, cache, _, q, kb, vb) in enumerate(cases):
        assert len(got[i]) == 50
        check_dense(got[i][0], *dense_reference(sh, q[0], *cache, kb, vb))
        assert all(torch.equal(r[k], got[i][0][k]) for r in got[i] for k in r)


def test_a_tensor_without_sizes_raises():
    sh, cache, _, q, kb, vb = inputs("bf16", [40], 2, 2, 4, seed=3)
    K, V = (torch.zeros(1, 2, 40, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    nested = torch.nested.nested_tensor([K[0], K[0]])
    with pytest.raises((RuntimeError, ValueError)):
        api.dequantize_prefix(sh, *cache, nested, V)


# ---------------------------------------------------------------------------
# the step
# ---------------------------------------------------------------------------
def gpu_step_quant(sh, qc, qp, cache, meta, kb, vb, o_p, l_p, q_ref=None, ws=None):
    rows = (sh.num_seqs, sh.n_q_heads, sh.block_size)
    A, k = sh.n_active, sh.pages_per_row
    r = {"out": torch.empty(*rows, 128, device=DEV), "lse": torch.empty(*rows, device=DEV),
         "o_p": o_p, "l_p": l_p,
         "active_idx": torch.full((*rows[:2], A), -7, dtype=torch.int32, device=DEV),
         "page_idx": torch.full((*rows[:2], A, k), -7, dtype=torch.int32, device=DEV),
         "union_count": torch.full((sh.num_seqs, sh.n_kv_heads), -7, dtype=torch.int32, device=DEV),
         "ws": api.alloc_workspace(sh, api.LOSA_WS_STEP, DEV) if ws is None else ws}
    tail = (*cache, meta, kb, vb, o_p, l_p, r["out"], r["lse"], r["ws"], r["active_idx"],
            r["page_idx"], r["union_count"])
    if q_ref is None:
        api.step_quant(sh, qc, qp, *tail)
    else:
        api.step_ref_quant(sh, qc, q_ref, *tail)
    return r


def state_of(sh, seed):
    g = torch.Generator().manual_seed(seed)
    rows = (sh.num_seqs, sh.n_q_heads, sh.block_size)
    return torch.randn(*rows, 128, generator=g).to(DEV), (3 + torch.rand(*rows, generator=g)).to(DEV)


KEYS = ("out", "lse", "o_p", "l_p", "active_idx", "page_idx", "union_count")
UNION = api.LOSA_STEP_ATTEND_UNION
STEP = [("bf16", [1000], 2, 4, 16, 4, 64, 0), ("f32", [1000], 2, 4, 8, 2, 64, 0),
        ("bf16", [1000], 2, 4, 16, 4, 64, UNION), ("f32", [333], 1, 2, 16, 4, 48, UNION),
        ("bf16", [1], 1, 1, 1, 1, 16, 0), ("bf16", [17], 2, 2, 5, 5, 512, 0),
        ("bf16", [700], 2, 4, 16, 16, 700 * 2, 0), ("bf16", [2000], 4, 2, 16, 0, 0, 0),
        ("bf16", [1000, 37, 1, 513], 2, 4, 16, 4, 64, 0), ("f32", [1000, 37, 1, 513], 2, 4, 4, 2, 64, 0),
        ("bf16", [1000, 37, 1, 513], 2, 4, 16, 4, 64, UNION), ("bf16", [9001], 8, 4, 16, 4, 256, 0),
        ("bf16", [3000], 1, 8, 8, 8, 512, 0), ("bf16", [4000, 4000], 2, 4, 32, 8, 256, 0)]


@pytest.mark.parametrize("dtype,lens,Hkv,G,B,A,budget,flags", STEP)
def test_step_equals_the_step_over_the_read_back_prefix(dtype, lens, Hkv, G, B, A, budget, flags):
    """With the scales that the library writes (powers of two) every score and weight of
    the two calls has the same bits: so have the selections and the log-normalisers, and in
    fp32 all results.  In bf16 the step over elements rounds a weight to two bf16 parts
    (within 2^-18), the 8-bit one to three, and they add up to 46 pages' products in 2 and 3
    accumulations of at most 2^-23 each: 2 * 2^-18 + 46 * 5 * 2^-23 < 2^-14 of max|v|."""
    sh, cache, meta, q, kb, vb = inputs(dtype, lens, Hkv, G, B, max(lens) + 5, sum(lens) + A,
                                        A=A, budget=budget, flags=flags)
    K, V = (torch.full((len(lens), Hkv, sh.capacity, 128), float("nan"), dtype=sh.torch_dtype,
                       device=DEV) for _ in range(2))
    api.dequantize_prefix(sh, *cache, K, V)
    o, l = state_of(sh, 3)
    a = gpu_step_quant(sh, q[1], q[0], cache, meta, kb, vb, o.clone(), l.clone())
    b = gpu_step(sh, q[1], q[0], K, V, meta, kb, vb, o.clone(), l.clone())
    assert api.read_device_status(a["ws"]) == api.LOSA_OK
    vmax = max(torch.nan_to_num(V).abs().max().item(), vb.abs().max().item(), o.abs().max().item())

    def check(a, b):
        for key in KEYS:
            if dtype == "bf16" and key in ("o_p", "out"):
                assert (a[key] - b[key]).abs().max().item() <= 2.0 ** -14 * vmax, key
            else:
                assert torch.equal(a[key], b[key]), key
    check(a, b)
    assert torch.isfinite(a["out"]).all()
    if A:  # the drift-safe form, its reference rewritten the same way
        ra, rb = q[0].clone(), q[0].clone()
        a = gpu_step_quant(sh, q[1], None, cache, meta, kb, vb, o.clone(), l.clone(), q_ref=ra)
        b = gpu_step(sh, q[1], None, K, V, meta, kb, vb, o.clone(), l.clone(), q_ref=rb)
        check(a, b)
        assert torch.equal(ra, rb) and not torch.equal(ra, q[0])


@pytest.mark.parametrize("dtype,lens,Hkv,G,B,A,budget,flags", [
    ("bf16", [3000, 2999, 1, 1700], 8, 4, 16, 4, 256, 0), ("bf16", [2500] * 8, 8, 4, 32, 8, 256, 0),
    ("f32", [1500] * 6, 4, 2, 8, 3, 64, 0), ("bf16", [900] * 5, 8, 8, 16, 8, 64, UNION),
    ("bf16", [40] * 20, 2, 1, 1, 1, 16, 0)])
def test_step_with_more_groups_than_run_at_once(dtype, lens, Hkv, G, B, A, budget, flags):
    """More (sequence, KV head) groups than clusters of 8 fit the GPU: the 8-bit step takes
    smaller clusters, so sums run in another order than in the step over the read-back
    prefix.  Selections are the same; each of the two carries weights within 2^-16 of the
    exact ones (two bf16 parts) and fp32 sums, so they differ by at most 2 * 2^-15 max|v|,
    and the log-normalisers by 2^-15."""
    sh, cache, meta, q, kb, vb = inputs(dtype, lens, Hkv, G, B, max(lens) + 3, sum(lens) + A, A=A,
                                        budget=budget, flags=flags)
    K, V = (torch.full((len(lens), Hkv, sh.capacity, 128), float("nan"), dtype=sh.torch_dtype,
                       device=DEV) for _ in range(2))
    api.dequantize_prefix(sh, *cache, K, V)
    o, l = state_of(sh, 3)
    a = gpu_step_quant(sh, q[1], q[0], cache, meta, kb, vb, o.clone(), l.clone())
    b = gpu_step(sh, q[1], q[0], K, V, meta, kb, vb, o.clone(), l.clone())
    assert api.read_device_status(a["ws"]) == api.LOSA_OK
    for key in ("active_idx", "page_idx", "union_count"):
        assert torch.equal(a[key], b[key]), key
    vmax = max(torch.nan_to_num(V).abs().max().item(), vb.abs().max().item(), o.abs().max().item())
    for key in ("o_p", "out", "l_p", "lse"):
        tol = 2.0 ** -14 * vmax if key in ("o_p", "out") else 2.0 ** -15
        assert (a[key] - b[key]).abs().max().item() <= tol, key
    again = gpu_step_quant(sh, q[1], q[0], cache, meta, kb, vb, o.clone(), l.clone())
    assert all(torch.equal(a[key], again[key]) for key in KEYS)


@pytest.mark.parametrize("dtype,lens,Hkv,G,B,A,budget", [
    ("bf16", [1], 2, 2, 1, 1, 16), ("bf16", [4], 2, 1, 1, 1, 16), ("bf16", [40], 1, 2, 5, 2, 512),
    ("bf16", [700], 2, 4, 16, 4, 128), ("f32", [300], 2, 2, 8, 3, 64)])
def test_step_error_against_64_bits(dtype, lens, Hkv, G, B, A, budget):
    """Relative to the results' norm: the weights keep 24 bits (three bf16 parts), the
    exponential is within 2^-22, the scores' roundings (at most 128 terms summed in 8
    accumulations, 2^-24 each of a score whose terms' sum is small at this scale) within
    2^-21, and a page's three products are added in as many accumulations of at most 2^-23 of
    the sum, over at most 4 pages of a warp: in all below 2^-19.  Independent roundings add as
    squares; half of that is allowed: 2^-20."""
    sh, cache, meta, q, kb, vb = inputs(dtype, lens, Hkv, G, B, seed=55, A=A, budget=budget)
    o, l = state_of(sh, 4)
    a = gpu_step_quant(sh, q[1], q[0], cache, meta, kb, vb, o.clone(), l.clone())
    K, V = read_back(cache[0], cache[2]), read_back(cache[1], cache[3])
    scale = sh.scale if sh.scale > 0 else 128 ** -0.5
    want = {"o_p": o.double(), "l_p": l.double()}
    want["out"], want["lse"] = torch.empty_like(want["o_p"]), torch.empty_like(want["l_p"])
    dbl = lambda x: x.double().to(DEV)
    for h in range(sh.n_q_heads):
        g = h // G
        for i, t in enumerate(a["active_idx"][0, h].tolist()):
            toks = torch.tensor([p * 16 + j for p in a["page_idx"][0, h, i].tolist() if p >= 0
                                 for j in range(16) if p * 16 + j < lens[0]], device=DEV)
            w = (K[0, g, toks] @ dbl(q[1][0, h, t])) * scale
            want["o_p"][0, h, t] = torch.softmax(w, 0) @ V[0, g, toks]
            want["l_p"][0, h, t] = torch.logsumexp(w, 0)
        w = dbl(q[1][0, h]) @ dbl(kb[0, g]).T * scale
        o_s, l_s = torch.softmax(w, -1) @ dbl(vb[0, g]), torch.logsumexp(w, -1)
        L = torch.logaddexp(want["l_p"][0, h], l_s)
        want["lse"][0, h] = L
        want["out"][0, h] = (torch.exp(want["l_p"][0, h] - L)[:, None] * want["o_p"][0, h]
                             + torch.exp(l_s - L)[:, None] * o_s)
    for key, ref in want.items():
        err = ((a[key].double() - ref).norm() / ref.norm()).item()
        assert err <= 2.0 ** -20, (key, err)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_other_scales(dtype):
    """Scales that are no powers of two, against the oracle on the read-back prefix (its
    metadata built from what the cache holds, rounded to the element type)."""
    sh, cache, _, q, kb, vb = inputs(dtype, [700], 2, 4, 8, seed=5, A=3, budget=64)
    g = torch.Generator().manual_seed(9)
    for t, lo in ((cache[2], 0.005), (cache[3], 0.002)):
        t.copy_((lo * (1 + torch.rand(t.shape, generator=g))).to(DEV))
    K, V = (torch.zeros(1, 2, 700, 128, dtype=sh.torch_dtype, device=DEV) for _ in range(2))
    api.dequantize_prefix(sh, *cache, K, V)
    meta = gpu_meta(sh, K)
    o, l = state_of(sh, 4)
    a = gpu_step_quant(sh, q[1], q[0], cache, meta, kb, vb, o.clone(), l.clone())
    kmin, kmax = (x.float().numpy() for x in unswizzle_page_meta(sh, meta))
    Kx, Vx = (read_back(cache[i], cache[2 + i]).float().cpu().numpy() for i in (0, 1))
    r = oracle.step(oshape(sh), q[1], q[0], Kx, Vx, kmin, kmax, kb, vb, o, l)
    for key in ("active_idx", "page_idx", "union_count"):
        assert np.array_equal(a[key].cpu().numpy(), r[key]), key
    for key in ("o_p", "l_p", "out", "lse"):
        assert maxabs(a[key].cpu().numpy(), r[key]) <= 2e-4, key  # (fp32 sums; see dense_bounds)


def test_step_captured_and_replayed():
    sh, cache, meta, q, kb, vb = inputs("bf16", [2000, 77], 2, 4, 16, 2010, 6, A=4, budget=128)
    o, l = state_of(sh, 8)
    want = gpu_step_quant(sh, q[1], q[0], cache, meta, kb, vb, o.clone(), l.clone())
    o2, l2 = o.clone(), l.clone()
    ws = api.alloc_workspace(sh, api.LOSA_WS_STEP, DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gpu_step_quant(sh, q[1], q[0], cache, meta, kb, vb, o2, l2, ws=ws)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for key in KEYS:
        assert torch.equal(got[key], want[key]), key


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,ragged", [("bf16", False), ("bf16", True), ("f32", False)])
def test_two_blocks_of_a_generation(dtype, ragged):
    """Write the prefix, then twice: the dense pass, three steps, the block appended.
    Every call is checked against the oracle on the read-back prefix of that time."""
    S, Hq, Hkv, B, A, budget = (2, 8, 2, 16, 4, 64)
    lens = [1000, 430] if ragged else [1000, 1000]
    c = random_case(S, Hq, Hkv, 1000, B, A, budget, dtype, seed=13)
    t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    sh = api.make_shape(S, Hq, Hkv, 128, 1000, 16, B, A, budget, dtype, scale=c.sh.scale,
                        prefix_capacity=1040, prefix_lens=t if ragged else None)
    K = torch.full((S, Hkv, 1040, 128), float("nan"), dtype=c.K.dtype, device=DEV)
    V = K.clone()
    K[:, :, :1000], V[:, :, :1000] = c.K, c.V
    cache = api.alloc_quant_prefix(sh, DEV)
    meta = api.alloc_page_meta(sh, DEV)
    api.quantize_prefix(sh, K, V, *cache, meta)
    ws_d = api.alloc_workspace(sh, api.LOSA_WS_DENSE_QUANT, DEV)
    ws_s = api.alloc_workspace(sh, api.LOSA_WS_STEP, DEV)
    g = torch.Generator().manual_seed(14)
    rnd = lambda *s: torch.randn(*s, generator=g).to(c.K.dtype).to(DEV)
    for block in range(2):
        if api.workspace_size(sh, api.LOSA_WS_DENSE_QUANT) > ws_d.numel():
            ws_d = api.alloc_workspace(sh, api.LOSA_WS_DENSE_QUANT, DEV)
        q = [rnd(S, Hq, B, 128)]
        kb, vb = rnd(S, Hkv, B, 128), rnd(S, Hkv, B, 128)
        st = gpu_dense_quant(sh, q[0], cache, kb, vb, ws_d)
        check_dense(st, *dense_reference(sh, q[0], *cache, kb, vb), f"block {block}")
        Kr, Vr = torch.zeros_like(K), torch.zeros_like(V)
        api.dequantize_prefix(sh, *cache, Kr, Vr)
        ref = {k: st[k].cpu().numpy() for k in ("o_p", "l_p")}
        for step in range(3):
            q.append((q[-1].float() + 0.3 * torch.randn(q[0].shape, generator=g).to(DEV)).to(c.K.dtype))
            kb, vb = rnd(S, Hkv, B, 128), rnd(S, Hkv, B, 128)
            r = gpu_step_quant(sh, q[-1], q[-2], cache, meta, kb, vb, st["o_p"], st["l_p"], ws=ws_s)
            osh = oracle.shape(S, Hq, Hkv, 128, sh.prefix_len, 16, B, A, budget, sh.scale)
            ref = oracle.step_varlen(osh, t.cpu().tolist() if ragged else [sh.prefix_len] * S, q[-1],
                                     q[-2], Kr, Vr, kb, vb, ref["o_p"], ref["l_p"])
            for key in ("active_idx", "page_idx", "union_count"):
                assert np.array_equal(r[key].cpu().numpy(), ref[key]), (block, step, key)
            for key in ("o_p", "l_p", "out", "lse"):
                assert maxabs(r[key].cpu().numpy(), ref[key]) <= 2e-4, (block, step, key)
        api.append_block_quant(sh, kb, vb, *cache, meta)
        sh.prefix_len += B
        t += B
    assert api.read_device_status(ws_d) == api.read_device_status(ws_s) == api.LOSA_OK
    assert np.isfinite(f64(cache[0][:, :, :400])).all()


def test_a_block_in_one_graph():
    """Copies from host memory, the write on a side stream, the dense pass, two steps and the
    append captured together and replayed on other inputs: the results of eager calls."""
    S, Hkv, G, B, L = 2, 2, 4, 16, 900
    sh = api.make_shape(S, Hkv * G, Hkv, 128, L, 16, B, 4, 64, "bf16", prefix_capacity=L + 40)
    g = torch.Generator().manual_seed(77)
    rnd = lambda *shape: torch.randn(*shape, generator=g).to(torch.bfloat16)
    sets = [[rnd(S, Hkv, L + 40, 128), rnd(S, Hkv, L + 40, 128), rnd(3, S, Hkv * G, B, 128),
             rnd(S, Hkv, B, 128), rnd(S, Hkv, B, 128)] for _ in range(2)]
    ws_d = api.alloc_workspace(sh, api.LOSA_WS_DENSE_QUANT, DEV)
    ws_s = api.alloc_workspace(sh, api.LOSA_WS_STEP, DEV)

    def buffers():
        return ([torch.empty_like(x, device=DEV) for x in sets[0]], api.alloc_quant_prefix(sh, DEV),
                api.alloc_page_meta(sh, DEV).zero_(), alloc_state(sh, torch.device(DEV), 0.0))

    def block(host, buf, side):
        (K, V, q, kb, vb), cache, meta, st = buf
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for dst, src in zip((K, V), host):
                dst.copy_(src, non_blocking=True)
            api.quantize_prefix(sh, K, V, *cache, meta)
        for dst, src in zip((q, kb, vb), host[2:]):
            dst.copy_(src, non_blocking=True)
        main.wait_stream(side)
        tail = (st["o_p"], st["l_p"], st["out"], st["lse"])
        api.dense_prefix_quant(sh, q[0], *cache, kb, vb, *tail, ws_d)
        for i in (1, 2):
            api.step_quant(sh, q[i], q[i - 1], *cache, meta, kb, vb, *tail, ws_s)
        api.append_block_quant(sh, kb, vb, *cache, meta)
        return [st[k] for k in ("o_p", "l_p", "out", "lse")] + [x.view(torch.uint8) for x in cache] + [meta]

    host = [x.clone().pin_memory() for x in sets[0]]
    buf, side = buffers(), torch.cuda.Stream()
    with torch.cuda.stream(torch.cuda.Stream()):
        block(host, buffers(), side)  # (warm-up)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(host, buf, side)
    for data in sets:
        for dst, src in zip(host, data):
            dst.copy_(src)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        want = block([x.pin_memory() for x in data], buffers(), torch.cuda.Stream())
        torch.cuda.synchronize()
        assert torch.isfinite(want[2]).all()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), i
    assert api.read_device_status(ws_d) == api.read_device_status(ws_s) == api.LOSA_OK
