"""The dense pass over the 8-bit prefix where the pages' V scales and the keys' weights are of
very different sizes: what holds the weight need not be what the output is made of.

Errors are relative to the results' norm, so that small values count as much as large ones."""
import math

import pytest
import torch

from losa_testutil import DEV
from quant_testutil import dense_reference, gpu_dense_quant
from sparse_long_context_mse_b200 import api
from test_gpu_quant_attention import gpu_step_quant, inputs, state_of

pytestmark = pytest.mark.gpu

PS = 16


def run(sh, cache, q, kb, vb):
    ws = api.alloc_workspace(sh, api.LOSA_WS_DENSE_QUANT, DEV)
    got = gpu_dense_quant(sh, q, cache, kb, vb, ws)
    assert api.read_device_status(ws) == api.LOSA_OK
    return got, dense_reference(sh, q, *cache, kb, vb)[0]


def errors(got, ref):
    """(worst relative error of o_p and out by norm, worst error of the log-normalisers)."""
    rel = [((got[k].cpu().double() - ref[k]).norm() / ref[k].norm()).item() for k in ("o_p", "out")]
    return max(rel), max((got[k].cpu().double() - ref[k]).abs().max().item() for k in ("l_p", "lse"))


# one row to 128, few tiles and many for each CTA, ragged, both types
SHAPES = [("bf16", [700], 2, 4, 16), ("bf16", [20000], 8, 4, 1), ("bf16", [9000, 501], 2, 4, 32),
          ("bf16", [1000], 1, 8, 4), ("f32", [3000], 2, 4, 4), ("f32", [700, 90], 1, 8, 16)]


@pytest.mark.parametrize("amp", [1e-2, 1e-4, 1e-9, 1e-20])
@pytest.mark.parametrize("dtype,lens,Hkv,G,B", SHAPES)
def test_small_values_beside_pages_of_zeros(dtype, lens, Hkv, G, B, amp):
    """A page of zeros has scale 1, whatever its neighbours have, and a share of the weight.
    The pass's roundings are relative to each key's own weight, so the bound is that of values
    of one size (test_dense_error_against_64_bits): 2^-20 of the norm."""
    sh, cache, _, q, kb, vb = inputs(dtype, lens, Hkv, G, B, seed=sum(lens) + 7)
    g = torch.Generator().manual_seed(5)
    K, V = (torch.randn(len(lens), Hkv, sh.capacity, 128, generator=g) for _ in range(2))
    V *= amp
    for p in range(3, sh.capacity_pages, 7):
        V[:, :, p * PS:(p + 1) * PS] = 0.0
    api.quantize_prefix(sh, K.to(sh.torch_dtype).to(DEV), V.to(sh.torch_dtype).to(DEV), *cache)
    assert (cache[3][:, :, 3] == 1.0).all()
    got, ref = run(sh, cache, q[0], kb, (vb.float() * amp).to(sh.torch_dtype))
    o, l = errors(got, ref)
    assert o <= 2.0 ** -20, o
    assert l <= 2.0 ** -19, l  # (a weight's relative error, and 2^-23 of its size, at most 10)


@pytest.mark.parametrize("binades", [12, 30, 60])
@pytest.mark.parametrize("dtype,lens,Hkv,G,B", SHAPES)
def test_zero_values_hold_the_weight(dtype, lens, Hkv, G, B, binades):
    """One token in 64 has a V of zeros and a score `binades` powers of two above the others:
    the output is the others' part.  Their scores have no large term, so among themselves they
    keep 2^-20; the normaliser is the heavy tokens' and carries their scores' error: t = 0.7 *
    binades + 3 (natural-log units), summed in 8 accumulations of at most 2^-24 t (16 in fp32,
    whose parts end in two accumulators) and rounded by half of 2^-23 t four times."""
    sh, cache, _, q, kb, vb = inputs(dtype, lens, Hkv, G, B, seed=sum(lens) + 11)
    g = torch.Generator().manual_seed(6)
    K, V = (torch.randn(len(lens), Hkv, sh.capacity, 128, generator=g) for _ in range(2))
    K[..., 0] = 0.0
    heavy = torch.arange(5, sh.capacity, 64)
    K[:, :, heavy, 0] = binades * math.log(2) / (8 * 128 ** -0.5)
    V[:, :, heavy] = 0.0
    api.quantize_prefix(sh, K.to(sh.torch_dtype).to(DEV), V.to(sh.torch_dtype).to(DEV), *cache)
    q[0][..., 0] = 8.0
    # (the block's tokens score like the light ones; its values are far smaller than the output)
    kb[..., 0] = 0.0
    got, ref = run(sh, cache, q[0], kb, torch.zeros_like(vb))
    o, l = errors(got, ref)
    t = 0.7 * binades + 3
    tol = 2.0 ** -20 + t * (16 + 4) * 2.0 ** -24
    assert ref["o_p"].norm() > 0 and o <= tol, (o, tol)
    assert l <= tol + 2.0 ** -22 * ref["lse"].abs().max().item(), l


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales_and_scores_against_each_other(dtype):
    """Pages of values 2^20 and of values 2^-20 whose scores make up for it, and the same with
    2^40 more between the two: the larger values' part is what the output is made of, or the
    smaller values' is."""
    sh, cache, _, q, kb, vb = inputs(dtype, [5000], 2, 4, 8, seed=71)
    for up, down in ((40, 0), (80, 0), (0, 0)):  # score of the small values' pages, binades
        g = torch.Generator().manual_seed(8)
        K, V = (torch.randn(1, 2, sh.capacity, 128, generator=g) for _ in range(2))
        K[..., 0] = 0.0
        for p in range(sh.capacity_pages):
            t = slice(p * PS, (p + 1) * PS)
            V[:, :, t] *= 2.0 ** (20 if p % 5 else -20)
            K[:, :, t, 0] = (down if p % 5 else up) * math.log(2) / (8 * 128 ** -0.5)
        api.quantize_prefix(sh, K.to(sh.torch_dtype).to(DEV), V.to(sh.torch_dtype).to(DEV), *cache)
        q[0][..., 0] = 8.0
        got, ref = run(sh, cache, q[0], kb, torch.zeros_like(vb))
        t = 0.7 * up + 3  # (as above)
        assert errors(got, ref)[0] <= 2.0 ** -20 + t * 20 * 2.0 ** -24


@pytest.mark.parametrize("dtype,n,Hkv,G,B", [("bf16", 140000, 1, 1, 1), ("f32", 131072, 1, 1, 1),
                                             ("bf16", 20000, 148, 1, 16)])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -120, 2.0 ** -100, 2.0 ** 119])
def test_the_smallest_and_largest_v_scales(dtype, n, Hkv, G, B, scale):
    """All V scales of a head the same, many keys of one score: the normaliser is their number
    and the output their mean, at any scale.  148 heads: one CTA has all keys of a head."""
    sh, cache, _, q, kb, vb = inputs(dtype, [64], Hkv, G, B, seed=3)
    sh = api.make_shape(1, Hkv * G, Hkv, 128, n, 16, B, 0, 0, dtype, scale=128 ** -0.5)
    cache = api.alloc_quant_prefix(sh, DEV)
    cache[1].view(torch.uint8).fill_(0x7E)  # 448
    cache[2].zero_()
    cache[3].fill_(scale)
    got = gpu_dense_quant(sh, torch.zeros_like(q[0]), cache, kb, torch.zeros_like(vb))
    # equal weights: sums of equal numbers, rounded a few times in fp32 (and truncated 24 times
    # a tile): 2^-18 in all
    assert (got["l_p"].double() - math.log(n)).abs().max().item() <= 2.0 ** -20 * math.log(n)
    assert (got["lse"].double() - math.log(n + B)).abs().max().item() <= 2.0 ** -20 * math.log(n)
    o = got["o_p"].double()
    assert torch.isfinite(got["out"]).all()
    if scale == 0.0:
        assert (o == 0).all()
    else:
        assert (o / (448 * scale) - 1).abs().max().item() <= 2.0 ** -18


@pytest.mark.parametrize("per_tile", [6, -6])
@pytest.mark.parametrize("dtype,B", [("bf16", 16), ("bf16", 1), ("f32", 4)])
def test_values_that_grow_or_shrink_along_the_prefix(dtype, B, per_tile):
    """Values 2^6 larger (smaller) from one 128 keys to the next, over 2^66 in all, with scores
    that make up for it and with flat ones: six tiles for each CTA."""
    sh, cache, _, q, kb, vb = inputs(dtype, [1500], 74, 1, B, seed=81)
    for flat in (False, True):
        g = torch.Generator().manual_seed(9)
        K, V = (torch.randn(1, 74, 1500, 128, generator=g) for _ in range(2))
        step = per_tile * (torch.arange(1500) // 128 - 5.5)
        V *= torch.exp2(step)[:, None]
        K[..., 0] = 0.0 if flat else -step * math.log(2) / (8 * 128 ** -0.5)
        api.quantize_prefix(sh, K.to(sh.torch_dtype).to(DEV), V.to(sh.torch_dtype).to(DEV), *cache)
        q[0][..., 0] = 8.0
        got, ref = run(sh, cache, q[0], kb, torch.zeros_like(vb))
        t = 3 if flat else 0.7 * 33 + 3  # (as above)
        assert errors(got, ref)[0] <= 2.0 ** -20 + t * 20 * 2.0 ** -24


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -100, 2.0 ** -60, 2.0 ** 100])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_v_scales(dtype, scale):
    """The step takes the V scales as they are: every token active on all pages is the dense
    pass, within 2^-20 of the results' norm (test_step_error_against_64_bits)."""
    sh, cache, meta, q, kb, vb = inputs(dtype, [60], 2, 4, 8, seed=85, A=8, budget=64)
    cache[3].fill_(scale)
    o, l = state_of(sh, 4)
    r = gpu_step_quant(sh, q[1], q[0], cache, meta, kb, vb, o, l)
    assert api.read_device_status(r["ws"]) == api.LOSA_OK
    ref = dense_reference(sh, q[1], *cache, kb, vb)[0]
    got = r["o_p"].cpu().double()
    if scale == 0.0:
        assert (got == 0).all()
    else:
        assert ((got - ref["o_p"]).norm() / ref["o_p"].norm()).item() <= 2.0 ** -20
    assert (r["l_p"].cpu().double() - ref["l_p"]).abs().max().item() <= 2.0 ** -19


@pytest.mark.parametrize("dtype,lens,Hkv,G,B", [("bf16", [700], 2, 4, 8), ("f32", [300, 90], 1, 8, 4)])
def test_the_smallest_weights(dtype, lens, Hkv, G, B):
    """Tokens of zeros hold all but 2^-116 of the weight: the other keys' weights, down to fp32's
    smallest normal number, keep their bits.  Rows are compared by direction (the factor that
    a row has in common is the heavy tokens' score, summed to within 2^-13).  An exponent of
    64 to 128 is rounded by at most half of 2^-17, which is ln 2 * 2^-18 of the weight; the
    rest is 2^-20 (test_dense_error_against_64_bits)."""
    sh, cache, _, q, kb, vb = inputs(dtype, lens, Hkv, G, B, seed=sum(lens) + 13)
    g = torch.Generator().manual_seed(6)
    K, V = (torch.randn(len(lens), Hkv, sh.capacity, 128, generator=g) for _ in range(2))
    K *= 0.5  # (scores within 2^+-5 of 2^-116)
    K[..., 0] = 0.0
    heavy = torch.arange(5, sh.capacity, 64)
    K[:, :, heavy, 0] = 116 * math.log(2) / (8 * 128 ** -0.5)
    V[:, :, heavy] = 0.0
    api.quantize_prefix(sh, K.to(sh.torch_dtype).to(DEV), V.to(sh.torch_dtype).to(DEV), *cache)
    q[0][..., 0] = 8.0
    got, ref = run(sh, cache, q[0], kb, torch.zeros_like(vb))
    a, b = got["o_p"].cpu().double(), ref["o_p"]
    assert (b.norm(dim=-1) > 0).all()
    a, b = a / a.norm(dim=-1, keepdim=True), b / b.norm(dim=-1, keepdim=True)
    assert (a - b).norm(dim=-1).max().item() <= math.log(2) * 2.0 ** -18 + 2.0 ** -20
