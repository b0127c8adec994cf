"""Forms of the 8-bit calls that their documentation allows: without metadata and other
optional results, scales that are a slice of a larger array, explicit streams, two steps at
once, and the drift-safe step with small clusters and in a replayed graph."""
import pytest
import torch

from losa_testutil import DEV, gpu_step
from quant_testutil import alloc_state, check_dense, dense_reference, gpu_dense_quant
from sparse_long_context_mse_b200 import api
from test_gpu_quant_attention import KEYS, UNION, gpu_step_quant, inputs, state_of

pytestmark = pytest.mark.gpu


def bytes_of(t):
    return t.reshape(-1).view(torch.uint8)


@pytest.mark.parametrize("dtype,lens,B", [("bf16", [100], 16), ("f32", [77, 20, 1], 5)])
def test_write_and_append_without_metadata(dtype, lens, B):
    """The same codes and scales as with it, and the records stay as they were."""
    sh, _, _, _, kb, vb = inputs(dtype, lens, 2, 2, B, cap=max(lens) + B + 3, seed=5)
    g = torch.Generator().manual_seed(6)
    K, V = (torch.randn(len(lens), 2, sh.capacity, 128, generator=g).to(sh.torch_dtype).to(DEV)
            for _ in range(2))
    caches = [api.alloc_quant_prefix(sh, DEV) for _ in range(2)]
    metas = [api.alloc_page_meta(sh, DEV).fill_(0x5A) for _ in range(2)]
    for cache, meta in zip(caches, (metas[0], None)):
        api.quantize_prefix(sh, K, V, *cache, meta)
    assert (metas[1] == 0x5A).all() and not (metas[0] == 0x5A).all()
    metas[1].copy_(metas[0])
    for cache, meta in zip(caches, (metas[0], None)):
        api.append_block_quant(sh, kb, vb, *cache, meta)
    for a, b in zip(*caches):
        assert torch.equal(bytes_of(a), bytes_of(b))
    before = api.alloc_page_meta(sh, DEV).fill_(0x5A)
    api.quantize_prefix(sh, K, V, *api.alloc_quant_prefix(sh, DEV), before)
    assert torch.equal(metas[1], before) and not torch.equal(metas[0], before)


def test_scales_of_a_slice_of_a_larger_array():
    """Scale arrays at an odd multiple of four bytes: every call gives the same bits."""
    sh, cache, meta, q, kb, vb = inputs("bf16", [500, 333], 3, 2, 8, cap=516, seed=7, A=3, budget=64)
    n = cache[2].numel()
    big = torch.full((4 * n + 9,), float("nan"), device=DEV)
    odd = [big[1:1 + n].view(cache[2].shape), big[2 * n + 3:3 * n + 3].view(cache[2].shape)]
    assert all(t.data_ptr() % 16 for t in odd)
    other = [cache[0].clone(), cache[1].clone(), *odd]
    for a, b in zip(odd, cache[2:]):
        a.copy_(b)
    o, l = state_of(sh, 1)
    got = []
    for c in (cache, other):
        K, V = (torch.zeros(2, 3, sh.capacity, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        m = meta.clone()
        d = gpu_dense_quant(sh, q[0], c, kb, vb)
        s = gpu_step_quant(sh, q[1], q[0], c, m, kb, vb, o.clone(), l.clone())
        api.append_block_quant(sh, kb, vb, *c, m)
        api.dequantize_prefix(sh, *c, K, V)
        got.append([*d.values(), *(s[k] for k in KEYS), m, K, V, *c[:2], *(x.clone() for x in c[2:])])
    for a, b in zip(*got):
        assert torch.equal(bytes_of(a), bytes_of(b))
    # nothing beside the slices was written
    rest = torch.ones_like(big, dtype=torch.bool)
    rest[1:1 + n] = rest[2 * n + 3:3 * n + 3] = False
    assert torch.isnan(big[rest]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_optional_results_and_on_a_given_stream(dtype):
    sh, cache, meta, q, kb, vb = inputs(dtype, [700, 41], 2, 4, 8, seed=9, A=2, budget=64)
    o, l = state_of(sh, 2)
    want = gpu_step_quant(sh, q[1], q[0], cache, meta, kb, vb, o.clone(), l.clone())
    dense = gpu_dense_quant(sh, q[0], cache, kb, vb)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    ws_d = api.alloc_workspace(sh, api.LOSA_WS_DENSE_QUANT, DEV)
    ws_s = api.alloc_workspace(sh, api.LOSA_WS_STEP, DEV)
    out = alloc_state(sh, torch.device(DEV))
    o2, l2, out2 = o.clone(), l.clone(), torch.empty_like(want["out"])
    torch.cuda.synchronize()
    api.dense_prefix_quant(sh, q[0], *cache, kb, vb, out["o_p"], out["l_p"], out["out"], None, ws_d,
                           stream=st)
    api.step_quant(sh, q[1], q[0], *cache, meta, kb, vb, o2, l2, out2, None, ws_s, stream=st)
    st.synchronize()
    for k in ("o_p", "l_p", "out"):
        assert torch.equal(out[k], dense[k]), k
    for a, k in ((o2, "o_p"), (l2, "l_p"), (out2, "out")):
        assert torch.equal(a, want[k]), k


def test_two_steps_at_once():
    """Two streams, each with its own state and workspace."""
    cases = [inputs("bf16", [3000, 100], 4, 4, 16, seed=11, A=4, budget=128),
             inputs("f32", [2000], 2, 2, 8, seed=12, A=2, budget=64)]
    want, got = [], []
    for sh, cache, meta, q, kb, vb in cases:
        want.append(gpu_step_quant(sh, q[1], q[0], cache, meta, kb, vb, *state_of(sh, 3)))
    states = [state_of(c[0], 3) for c in cases]
    ws = [api.alloc_workspace(c[0], api.LOSA_WS_STEP, DEV) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for (sh, cache, meta, q, kb, vb), s, st, w in zip(cases, states, streams, ws):
        with torch.cuda.stream(st):
            got.append(gpu_step_quant(sh, q[1], q[0], cache, meta, kb, vb, *s, ws=w))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(a[k], b[k]) for k in KEYS)


@pytest.mark.parametrize("dtype,lens,Hkv,G,B,A,budget,flags", [
    ("bf16", [3000, 2999, 1, 1700], 8, 4, 16, 4, 256, 0), ("bf16", [2500] * 8, 8, 4, 32, 8, 256, 0),
    ("f32", [1500] * 6, 4, 2, 8, 3, 64, 0), ("bf16", [900] * 5, 8, 8, 16, 8, 64, UNION)])
def test_drift_safe_step_with_more_groups_than_run_at_once(dtype, lens, Hkv, G, B, A, budget, flags):
    """The drift-safe step in clusters smaller than 8, against the one over the read-back
    prefix: the same selections and the same rewritten reference queries, results within the
    bounds of test_step_with_more_groups_than_run_at_once; twice, so that the second call
    scores against references that the first one wrote."""
    sh, cache, meta, q, kb, vb = inputs(dtype, lens, Hkv, G, B, max(lens) + 3, sum(lens) + A, A=A,
                                        budget=budget, flags=flags)
    K, V = (torch.full((len(lens), Hkv, sh.capacity, 128), float("nan"), dtype=sh.torch_dtype,
                       device=DEV) for _ in range(2))
    api.dequantize_prefix(sh, *cache, K, V)
    o, l = state_of(sh, 3)
    refs = [q[0].clone(), q[0].clone()]
    vmax = max(torch.nan_to_num(V).abs().max().item(), vb.abs().max().item(), o.abs().max().item())
    for qc in (q[1], (q[1].float() + 0.05 * q[0].float()).to(sh.torch_dtype)):
        a = gpu_step_quant(sh, qc, None, cache, meta, kb, vb, o.clone(), l.clone(), q_ref=refs[0])
        b = gpu_step(sh, qc, None, K, V, meta, kb, vb, o.clone(), l.clone(), q_ref=refs[1])
        assert api.read_device_status(a["ws"]) == api.LOSA_OK
        for key in ("active_idx", "page_idx", "union_count"):
            assert torch.equal(a[key], b[key]), key
        for key in ("o_p", "out", "l_p", "lse"):
            tol = 2.0 ** -14 * vmax if key in ("o_p", "out") else 2.0 ** -15
            assert (a[key] - b[key]).abs().max().item() <= tol, key
        assert torch.equal(refs[0], refs[1])
        # exactly the active rows' references are this call's queries
        act = torch.zeros(q[0].shape[:3], dtype=torch.bool, device=DEV)
        act.scatter_(2, a["active_idx"].long(), True)
        assert torch.equal(refs[0][act], qc[act])
    assert not torch.equal(refs[0], q[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_drift_safe_step_captured_and_replayed(dtype):
    """Each replay scores against the references that the one before wrote: as many eager
    calls give the same bits."""
    sh, cache, meta, q, kb, vb = inputs(dtype, [2000, 77], 2, 4, 16, 2010, 6, A=4, budget=128)
    o, l = state_of(sh, 8)
    qc = [q[1], (q[1].float() * 1.1).to(sh.torch_dtype), q[0]]
    ws = api.alloc_workspace(sh, api.LOSA_WS_STEP, DEV)
    cur, ref, o2, l2 = q[1].clone(), q[0].clone(), o.clone(), l.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gpu_step_quant(sh, cur, None, cache, meta, kb, vb, o2, l2, q_ref=ref, ws=ws)
    eager_ref, o1, l1 = q[0].clone(), o.clone(), l.clone()
    for x in qc:
        want = gpu_step_quant(sh, x, None, cache, meta, kb, vb, o1, l1, q_ref=eager_ref)
        cur.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ref, eager_ref)
        for key in KEYS:
            assert torch.equal(got[key], want[key]), key
    assert api.read_device_status(ws) == api.LOSA_OK


def test_dense_of_one_head_among_many_rows():
    """127 and 128 query rows of a KV head: the second CTA of a range has a row less, or all."""
    for G, B in ((127, 1), (128, 1), (4, 32), (65, 1)):
        sh, cache, _, q, kb, vb = inputs("bf16", [700], 1, G, B, seed=G)
        got = gpu_dense_quant(sh, q[0], cache, kb, vb)
        check_dense(got, *dense_reference(sh, q[0], *cache, kb, vb), f"{G} {B}")


@pytest.mark.parametrize("dtype,L,Hkv", [("bf16", 131072, 8), ("bf16", 131069, 4), ("f32", 65530, 4)])
def test_long_prefix(dtype, L, Hkv):
    """The longest prefix that the framework's own workloads have: the step against the one
    over the read-back prefix (bounds as in test_step_equals_the_step_over_the_read_back_prefix),
    the dense pass against 64 bits, and a block appended behind it."""
    B = 16
    sh, cache, meta, q, kb, vb = inputs(dtype, [L], Hkv, 4, B, L + 20, 17, A=4, budget=128)
    got = gpu_dense_quant(sh, q[0], cache, kb, vb)
    check_dense(got, *dense_reference(sh, q[0], *cache, kb, vb))
    K, V = (torch.zeros(1, Hkv, sh.capacity, 128, dtype=sh.torch_dtype, device=DEV) for _ in range(2))
    for _ in range(2):
        api.dequantize_prefix(sh, *cache, K, V)
        o, l = state_of(sh, 3)
        a = gpu_step_quant(sh, q[1], q[0], cache, meta, kb, vb, o.clone(), l.clone())
        b = gpu_step(sh, q[1], q[0], K, V, meta, kb, vb, o.clone(), l.clone())
        assert api.read_device_status(a["ws"]) == api.LOSA_OK
        for key in KEYS:
            if dtype == "bf16" and key in ("o_p", "out"):
                vmax = max(V.abs().max().item(), vb.abs().max().item(), o.abs().max().item())
                assert (a[key] - b[key]).abs().max().item() <= 2.0 ** -14 * vmax, key
            else:
                assert torch.equal(a[key], b[key]), key
        if sh.prefix_len == L:
            api.append_block_quant(sh, kb, vb, *cache, meta)
            sh.prefix_len += B
