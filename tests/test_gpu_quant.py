"""Writing, growing and reading the 8-bit prefix cache: codes, scales and
records bit for bit what the definition gives, and nothing else written."""
import copy

import numpy as np
import pytest
import torch

from losa_testutil import DEV, page_norms, unswizzle_page_meta
from quant_testutil import F8, PS, encode, f64, lens_of, random_prefix, same
from sparse_long_context_mse_b200 import api

pytestmark = pytest.mark.gpu

FILL = 0x5A      # what an unwritten byte holds
SFILL = 12345.0  # what an unwritten scale holds


def make(dtype, lens, Hkv, cap=0, B=16):
    ragged = len(set(lens)) > 1
    t = torch.tensor(lens, dtype=torch.int32, device=DEV) if ragged else None
    return api.make_shape(len(lens), 2 * Hkv, Hkv, 128, max(lens), 16, B, 0, 0, dtype,
                          prefix_capacity=cap, prefix_lens=t)


def empty_cache(sh):
    k8, v8, ks, vs = api.alloc_quant_prefix(sh, DEV)
    for t in (k8, v8):
        t.view(torch.uint8).fill_(FILL)
    ks.fill_(SFILL)
    vs.fill_(SFILL)
    meta = api.alloc_page_meta(sh, DEV)
    meta.fill_(FILL)
    return (k8, v8, ks, vs), meta


def check_cache(sh, cache, K, V, what=""):
    """Every sequence's codes and scales against the definition; the rest untouched."""
    for x8, sc, X in ((cache[0], cache[2], K), (cache[1], cache[3], V)):
        val, raw, scale = f64(x8), x8.view(torch.uint8).cpu().numpy(), sc.cpu().numpy()
        for s, n in enumerate(lens_of(sh)):
            P = -(-n // PS)
            for g in range(sh.n_kv_heads):
                want, ws = encode(X[s][g][:n])
                assert np.array_equal(scale[s, g, :P], ws), (what, s, g)
                assert same(val[s, g, :n], want), (what, s, g)
            assert (raw[s, :, n:] == FILL).all() and (scale[s, :, P:] == SFILL).all(), (what, s)


def check_records(sh, meta, cache):
    """The records are what the metadata build gives for the read-back prefix, and the
    norms bound the records' from above; records past a sequence's pages untouched."""
    K = torch.full((sh.num_seqs, sh.n_kv_heads, sh.capacity, 128), float("nan"),
                   dtype=sh.torch_dtype, device=DEV)
    V = K.clone()
    api.dequantize_prefix(sh, *cache, K, V)
    ref = api.alloc_page_meta(sh, DEV)
    ref.fill_(FILL)
    api.build_page_meta(sh, K, ref)
    nrec = sh.num_seqs * sh.n_kv_heads * sh.capacity_pages * 256 * K.element_size()
    a, b = meta[:nrec].view(sh.torch_dtype).float(), ref[:nrec].view(sh.torch_dtype).float()
    assert torch.equal(a, b)  # (as numbers: a zero's sign is free)
    na, nb = page_norms(sh, meta).astype(np.float64), page_norms(sh, ref).astype(np.float64)
    lo, hi = (x.double().numpy() for x in unswizzle_page_meta(sh, meta))
    for s, n in enumerate(lens_of(sh)):
        P = -(-n // PS)
        for j, m in enumerate((lo, hi)):
            exact = np.sqrt((m[s, :, :P] ** 2).sum(-1))
            assert (na[s, :, :P, j] >= exact).all()
            assert (na[s, :, :P, j] <= exact * (1 + 2.0 ** -15) + 1e-30).all()
        assert np.array_equal(na[s, :, P:].view(np.uint64), nb[s, :, P:].view(np.uint64))


SHAPES = [  # dtype, lengths, KV heads, capacity
    ("bf16", [1], 1, 0), ("bf16", [16], 2, 0), ("bf16", [333], 2, 340), ("f32", [37, 1, 513], 2, 530),
    ("bf16", [1000, 37, 1, 513], 2, 1003), ("f32", [129], 1, 129), ("bf16", [4097, 2050], 8, 4100)]


@pytest.mark.parametrize("dtype,lens,Hkv,cap", SHAPES)
def test_write_and_read(dtype, lens, Hkv, cap):
    sh = make(dtype, lens, Hkv, cap)
    K, V = random_prefix(sh, torch.Generator().manual_seed(len(lens) + lens[0]), DEV)
    cache, meta = empty_cache(sh)
    api.quantize_prefix(sh, K, V, *cache, meta)
    check_cache(sh, cache, f64(K), f64(V))
    check_records(sh, meta, cache)
    # reading back is exact, and writes nothing past a sequence's length
    k, v = torch.full_like(K, 7.0), torch.full_like(V, 7.0)
    api.dequantize_prefix(sh, *cache, k, v)
    for x, x8, sc in ((k, cache[0], cache[2]), (v, cache[1], cache[3])):
        x, val, scale = f64(x), f64(x8), f64(sc)
        for s, n in enumerate(lens):
            want = val[s, :, :n] * np.repeat(scale[s], PS, axis=-1)[:, :n, None]
            assert np.array_equal(x[s, :, :n], want) and (x[s, :, n:] == 7.0).all()
    # without metadata the codes are the same
    again, _ = empty_cache(sh)
    api.quantize_prefix(sh, K, V, *again)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cache, again))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_special_values(dtype):
    sh = make(dtype, [16 * 12], 1)
    K = torch.zeros(1, 1, 192, 128)
    p = lambda i: K[0, 0, 16 * i:16 * i + 16]
    p(1)[3, 5] = 448.0                       # exactly e4m3's largest number: scale 1
    p(1)[4, 6] = -2.0 ** -9                  # its smallest subnormal
    p(1)[4, 7] = 2.0 ** -10                  # half of it: ties to zero
    p(1)[5, 7] = 3 * 2.0 ** -10              # ties to 2 * 2^-9
    p(2)[0, 0] = 450.0                       # just above: scale 2
    p(3)[:] = 2.0 ** -120                    # below the smallest scale's range
    p(4)[0] = 3e38                           # near the largest number
    p(5)[0, 0] = float("inf")
    p(5)[1, 0] = float("-inf")
    p(5)[2, 0] = 1.0
    p(6)[0, 0] = float("nan")
    p(6)[1] = 2.0
    p(7)[:] = -0.0
    p(8)[:] = torch.linspace(-1, 1, 16 * 128).view(16, 128)
    p(9)[:] = 1e-30
    p(10)[:, 64:] = 5.0
    p(11)[15, 127] = 2.0 ** -100
    K = K.to(sh.torch_dtype).to(DEV)
    cache, _ = empty_cache(sh)
    api.quantize_prefix(sh, K, K, *cache)
    check_cache(sh, cache, f64(K), f64(K))
    back = [torch.empty_like(K) for _ in range(2)]
    api.dequantize_prefix(sh, *cache, *back)
    assert torch.isnan(back[0][0, 0, 96, 0]) and torch.equal(back[0].isnan(), back[1].isnan())
    assert torch.isfinite(back[0][0, 0, :96]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_read_with_other_scales(dtype):
    """A cache of another program: every code, scales that are no powers of two."""
    sh = make(dtype, [70], 2, 80)
    g = torch.Generator().manual_seed(4)
    codes = torch.randint(0, 256, (2, 1, 2, 80, 128), generator=g, dtype=torch.uint8).to(DEV)
    sc = (torch.randn(2, 1, 2, 5, generator=g) * 3).to(DEV)
    k, v = (torch.full((1, 2, 80, 128), 7.0, dtype=sh.torch_dtype, device=DEV) for _ in range(2))
    api.dequantize_prefix(sh, codes[0].view(F8), codes[1].view(F8), sc[0], sc[1], k, v)
    for x, c, s in ((k, codes[0], sc[0]), (v, codes[1], sc[1])):
        want = f64(c.view(F8)) * np.repeat(f64(s), PS, axis=-1)[..., None]
        want = torch.tensor(want).float().to(sh.torch_dtype)  # (products of a 4- and a 24-bit number)
        assert torch.equal(torch.nan_to_num(x[:, :, :70].cpu()), torch.nan_to_num(want[:, :, :70]))
        assert torch.equal(x[:, :, :70].isnan().cpu(), want[:, :, :70].isnan())
        assert (x[:, :, 70:] == 7.0).all()


def run_appends(sh, B, n_appends, seed, amps, with_meta=True):
    gen = torch.Generator().manual_seed(seed)
    S, Hkv = sh.num_seqs, sh.n_kv_heads
    K, V = random_prefix(sh, gen, DEV)
    cache, meta = empty_cache(sh)
    api.quantize_prefix(sh, K, V, *cache, meta)
    m = meta if with_meta else None
    lens = sh._prefix_lens
    for i in range(n_appends):
        n = lens_of(sh)
        val = [f64(cache[j]) for j in (0, 1)]
        scl = [f64(cache[j]) for j in (2, 3)]
        raw = [cache[j].view(torch.uint8).cpu().numpy().copy() for j in (0, 1)]
        blk = [(amps[i] * torch.randn(S, Hkv, B, 128, generator=gen)).to(sh.torch_dtype).to(DEV)
               for _ in range(2)]
        api.append_block_quant(sh, *blk, *cache, m)
        if lens is not None:
            lens += B
        sh.prefix_len += B
        for j in (0, 1):
            got, sc = f64(cache[j]), f64(cache[2 + j])
            now = cache[j].view(torch.uint8).cpu().numpy()
            new = f64(blk[j])
            for s in range(S):
                p0, p1 = n[s] // PS, -(-(n[s] + B) // PS)
                for g in range(Hkv):
                    old = val[j][s, g, p0 * PS:n[s]] * scl[j][s, g, p0]
                    want, ws = encode(np.concatenate((old, new[s, g])))
                    assert same(got[s, g, p0 * PS:n[s] + B], want), (i, j, s, g)
                    assert np.array_equal(sc[s, g, p0:p1], ws), (i, j, s, g)
                # everything outside the touched pages is as it was
                assert np.array_equal(now[s, :, :p0 * PS], raw[j][s, :, :p0 * PS])
                assert np.array_equal(now[s, :, n[s] + B:], raw[j][s, :, n[s] + B:])
                assert np.array_equal(sc[s, :, :p0], scl[j][s, :, :p0])
                assert np.array_equal(sc[s, :, p1:], scl[j][s, :, p1:])
        if with_meta:
            check_records(sh, meta, cache)
        elif i == 0:
            assert (meta.cpu() == meta.cpu()).all()
    return cache


@pytest.mark.parametrize("dtype,lens,B", [
    ("bf16", [1000], 16), ("f32", [992], 16), ("bf16", [8], 1), ("bf16", [15], 2), ("f32", [1], 31),
    ("bf16", [1000, 37, 1, 513], 32), ("f32", [16, 33], 5)])
def test_append(dtype, lens, B):
    cap = max(lens) + 4 * B + 5
    # larger and smaller blocks than the prefix: the shared page's scale grows or not
    run_appends(make(dtype, lens, 2, cap, B), B, 4, 9 + B, (1.0, 100.0, 0.01, 1.0))


def test_append_without_metadata():
    run_appends(make("bf16", [100], 2, 140, 16), 16, 2, 3, (1.0, 1.0), with_meta=False)


def test_older_tokens_keep_their_values():
    """A block that does not raise the page's scale leaves the older tokens' values."""
    sh = make("bf16", [100], 2, 160)
    K, V = random_prefix(sh, torch.Generator().manual_seed(5), DEV)
    cache, _ = empty_cache(sh)
    api.quantize_prefix(sh, K, V, *cache)
    a = [torch.zeros_like(K) for _ in range(2)]
    api.dequantize_prefix(sh, *cache, *a)
    blk = torch.full((1, 2, 16, 128), 0.25, dtype=torch.bfloat16, device=DEV)
    api.append_block_quant(sh, blk, blk, *cache)
    sh.prefix_len += 16
    b = [torch.zeros_like(K) for _ in range(2)]
    api.dequantize_prefix(sh, *cache, *b)
    for x, y in zip(a, b):
        assert torch.equal(x[:, :, :100], y[:, :, :100])
        assert (y[:, :, 100:116] == 0.25).all() and (y[:, :, 116:] == 0).all()


def test_append_out_of_range_lengths_stay_inside():
    """Lengths outside [1, L] are clamped into it, as in losa_append_block."""
    sh = make("bf16", [100, 50], 1, 120)
    cache, meta = empty_cache(sh)
    K, V = random_prefix(sh, torch.Generator().manual_seed(6), DEV)
    api.quantize_prefix(sh, K, V, *cache, meta)
    sh._prefix_lens.copy_(torch.tensor([10 ** 6, -5]))
    blk = torch.ones(2, 1, 16, 128, dtype=torch.bfloat16, device=DEV)
    before = cache[0].view(torch.uint8).clone()
    api.append_block_quant(sh, blk, blk, *cache, meta)
    torch.cuda.synchronize()
    now = f64(cache[0]) * np.repeat(f64(cache[2]), PS, -1)[:, :, :120, None]
    assert (now[0, :, 100:116] == 1.0).all() and (now[1, :, 1:17] == 1.0).all()
    assert torch.equal(cache[0].view(torch.uint8)[0, :, 116:], before[0, :, 116:])
    assert torch.equal(cache[0].view(torch.uint8)[1, :, 32:], before[1, :, 32:])


def test_captured_and_on_another_stream():
    """Write, append and read on a stream of their own and inside a captured graph that
    is replayed on new contents."""
    sh = make("bf16", [100, 61], 2, 130)
    gen = torch.Generator().manual_seed(8)
    K, V = random_prefix(sh, gen, DEV)
    cache, meta = empty_cache(sh)
    back = [torch.full_like(K, 7.0) for _ in range(2)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        api.quantize_prefix(sh, K, V, *cache, meta, stream=st)
        api.dequantize_prefix(sh, *cache, *back, stream=st)
        with torch.cuda.graph(graph, stream=st):
            api.quantize_prefix(sh, K, V, *cache, meta)
            api.dequantize_prefix(sh, *cache, *back)
    torch.cuda.synchronize()
    K2, V2 = random_prefix(sh, gen, DEV, amp=30.0)
    K.copy_(K2)
    V.copy_(V2)
    sh._prefix_lens.copy_(torch.tensor([100, 33]))  # read when the graph runs
    (c2, m2) = empty_cache(sh)
    for t, u in zip((*cache, meta), (*c2, m2)):
        t.view(torch.uint8).copy_(u.view(torch.uint8))
    graph.replay()
    torch.cuda.synchronize()
    check_cache(sh, cache, f64(K), f64(V))
    check_records(sh, meta, cache)


def test_append_refuses_a_full_cache():
    sh = make("bf16", [100], 1, 115)
    cache, meta = empty_cache(sh)
    blk = torch.zeros(1, 1, 16, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(api.LosaError):
        api.append_block_quant(sh, blk, blk, *cache, meta)
    sh2 = copy.copy(sh)
    sh2.block_size = 15
    api.append_block_quant(sh2, blk[:, :, :15].contiguous(), blk[:, :, :15].contiguous(), *cache, meta)
    torch.cuda.synchronize()
