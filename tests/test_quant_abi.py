"""The 8-bit prefix cache's calls without a GPU: sizes, argument validation
before any launch, the binding's checks, and the tests' own model of the format."""
import ctypes

import numpy as np
import pytest
import torch

from quant_testutil import VALUES, encode, encode_value, page_scale
from sparse_long_context_mse_b200 import api, build

INV, UNS = api.LOSA_ERR_INVALID_ARG, api.LOSA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


@pytest.fixture
def no_device():
    """Tests that pass fake addresses: a call that wrongly passed validation would
    launch on them, so they run only without a GPU."""
    if torch.cuda.is_available():
        pytest.skip("fake device addresses: CPU-only validation test")


def S(**kw):
    base = dict(num_seqs=1, n_q_heads=32, n_kv_heads=8, head_dim=128, prefix_len=65536,
                page_size=16, block_size=16, n_active=4, token_budget=128, dtype="bf16")
    base.update(kw)
    return api.make_shape(**base)


FAR = [(i + 1) << 36 for i in range(20)]  # no two buffers of a call overlap


def P(ptrs):
    return [ctypes.c_void_p(p) if p is not None else None for p in ptrs]


def test_workspace_size(L):
    for kw in (dict(), dict(dtype="f32"), dict(block_size=1, n_active=0, token_budget=0),
               dict(num_seqs=8, prefix_len=32768, block_size=32, n_active=8, token_budget=256),
               dict(prefix_len=1, n_active=0, token_budget=0)):
        n = api.workspace_size(S(**kw), api.LOSA_WS_DENSE_QUANT)
        assert n > 0 and n % 256 == 0
    assert api.workspace_size(S(prefix_len=0), api.LOSA_WS_DENSE_QUANT) == 0
    assert api.workspace_size(S(block_size=64, n_active=4), api.LOSA_WS_DENSE_QUANT) == 0


# (call, pointers, indices of the optional ones, (written, other) pairs)
def calls(L):
    return {
        # 0 k_prefix 1 v_prefix 2 k8 3 v8 4 k_scale 5 v_scale 6 page_meta
        "write": (L.losa_quantize_prefix, 7, (6,),
                  ((2, 0), (2, 1), (3, 0), (3, 2), (4, 1), (5, 3), (5, 4), (6, 0), (6, 2), (6, 5))),
        # 0 k_blk 1 v_blk 2 k8 3 v8 4 k_scale 5 v_scale 6 page_meta
        "append": (L.losa_append_block_quant, 7, (6,),
                   ((2, 0), (3, 1), (3, 2), (4, 0), (5, 2), (6, 3), (6, 4), (6, 1))),
        # 0 k8 1 v8 2 k_scale 3 v_scale 4 k_prefix 5 v_prefix
        "read": (L.losa_dequantize_prefix, 6, (), ((4, 0), (4, 1), (5, 2), (5, 3), (5, 4))),
        # 0 q 1 k8 2 v8 3 k_scale 4 v_scale 5 k_blk 6 v_blk 7 o_p 8 l_p 9 out 10 lse 11 workspace
        "dense": (L.losa_dense_prefix_quant, 12, (10,),
                  ((7, 0), (7, 1), (8, 2), (8, 3), (9, 4), (9, 5), (10, 6), (9, 7), (11, 1), (11, 9))),
        # 0 q_cur 1 q_prev 2 k8 3 v8 4 k_scale 5 v_scale 6 page_meta 7 k_blk 8 v_blk 9 o_p 10 l_p
        # 11 out 12 lse 13 active 14 pages 15 union 16 workspace
        "step": (L.losa_step_quant, 17, (12, 13, 14, 15),
                 ((9, 0), (9, 2), (10, 3), (11, 4), (11, 5), (12, 6), (13, 7), (14, 8), (15, 9),
                  (16, 4), (16, 11))),
        "step_ref": (L.losa_step_ref_quant, 17, (12, 13, 14, 15),
                     ((1, 0), (1, 2), (1, 4), (9, 1), (11, 5), (16, 1))),
    }


def invoke(L, name, sh, ptrs, ws_bytes=None):
    fn, n, _, _ = calls(L)[name]
    args = P(ptrs[:n])
    if name in ("dense", "step", "step_ref"):
        which = api.LOSA_WS_DENSE_QUANT if name == "dense" else api.LOSA_WS_STEP
        args.append(api.workspace_size(sh, which) if ws_bytes is None else ws_bytes)
    return fn(ctypes.byref(sh) if sh is not None else None, *args, None)


SCALES = {"write": (4, 5), "append": (4, 5), "read": (2, 3), "dense": (3, 4), "step": (4, 5),
          "step_ref": (4, 5)}
NAMES = ("write", "append", "read", "dense", "step", "step_ref")


@pytest.mark.parametrize("name", NAMES)
def test_pointer_validation(L, name, no_device):
    sh = S(prefix_capacity=65536 + 64)
    _, n, optional, _ = calls(L)[name]
    for i in range(n):
        p = list(FAR)
        # misaligned (16 bytes; a scale 4, the workspace 256)
        p[i] = FAR[i] + (2 if i in SCALES[name] else 8)
        assert invoke(L, name, sh, p) == INV, i
        if i not in optional:
            p[i] = None
            assert invoke(L, name, sh, p) == INV, i
    assert invoke(L, name, None, FAR, 1 << 40) == INV
    if name in ("dense", "step", "step_ref"):
        which = api.LOSA_WS_DENSE_QUANT if name == "dense" else api.LOSA_WS_STEP
        assert invoke(L, name, sh, FAR, api.workspace_size(sh, which) - 1) == INV
        p = list(FAR)
        p[n - 1] = FAR[n - 1] + 128
        assert invoke(L, name, sh, p) == INV


@pytest.mark.parametrize("name", NAMES)
def test_written_aliases_are_refused(L, name, no_device):
    sh = S(prefix_capacity=65536 + 64)
    for w, o in calls(L)[name][3]:
        p = list(FAR)
        p[w] = FAR[o] + (0 if name == "step_ref" and w == 1 else 256)
        assert invoke(L, name, sh, p) == INV, (w, o)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("kw,code", [
    (dict(n_q_heads=30), INV), (dict(prefix_len=0), INV), (dict(scale=-1.0), INV),
    (dict(prefix_capacity=65535), INV), (dict(flags=2), INV), (dict(num_seqs=0), INV),
    (dict(head_dim=64), UNS), (dict(page_size=32), UNS), (dict(block_size=64), UNS),
    (dict(n_q_heads=64, n_kv_heads=2, block_size=8), UNS)])
def test_shape_validation(L, name, kw, code, no_device):
    assert invoke(L, name, S(**kw), FAR, 1 << 40) == code


def test_append_needs_room(L, no_device):
    for cap in (0, 65536 + 15):
        assert invoke(L, "append", S(prefix_capacity=cap), FAR) == INV


def test_too_many_groups(L, no_device):
    sh = S(num_seqs=65536, n_q_heads=1, n_kv_heads=1, prefix_len=16, prefix_capacity=64,
           n_active=0, token_budget=0)
    for name in NAMES:
        assert invoke(L, name, sh, [(i + 1) << 42 for i in range(20)]) == UNS, name


def test_binding_refuses_host_tensors_and_wrong_types(L, monkeypatch):
    sh = S(prefix_len=32)
    k = torch.zeros(1, 8, 32, 128, dtype=torch.bfloat16)
    c8 = torch.zeros(1, 8, 32, 128, dtype=torch.float8_e4m3fn)
    sc = torch.ones(1, 8, 2)
    for bad in ((k, k, c8, c8, sc, sc), (k, k, c8, c8, sc, sc, torch.zeros(3, dtype=torch.uint8))):
        with pytest.raises(ValueError):  # host tensors
            api.quantize_prefix(sh, *bad)
    with pytest.raises(TypeError):
        api.quantize_prefix(sh, [0.0], k, c8, c8, sc, sc)
    monkeypatch.setattr(api, "_device_of", lambda t: t.device)
    with pytest.raises(TypeError):  # only the metadata may be left out
        api.quantize_prefix(sh, k, k, c8, None, sc, sc)


@pytest.mark.parametrize("kind,good,bad", [
    ("8", torch.zeros(1, 8, 32, 128, dtype=torch.float8_e4m3fn),
     [torch.zeros(1, 8, 32, 128, dtype=torch.uint8), torch.zeros(1, 8, 31, 128, dtype=torch.float8_e4m3fn),
      torch.zeros(1, 8, 32, 256, dtype=torch.float8_e4m3fn)[..., ::2]]),
    ("s", torch.ones(1, 8, 2), [torch.ones(1, 8, 3), torch.ones(1, 8, 2).double(), torch.ones(8, 2)]),
    ("b", torch.zeros(1, 8, 16, 128, dtype=torch.bfloat16),
     [torch.zeros(1, 8, 16, 128), torch.zeros(1, 8, 16, 256, dtype=torch.bfloat16)[..., ::2]]),
    ("m", None, [torch.zeros(5, dtype=torch.uint8)])])
def test_binding_says_which_tensor_is_wrong(L, monkeypatch, kind, good, bad):
    """The message names the tensor (host tensors stand in: only the device check is
    taken out)."""
    monkeypatch.setattr(api, "_device_of", lambda t: t.device)
    sh = S(prefix_len=32)
    first = torch.zeros(1, 32, 16, 128, dtype=torch.bfloat16)
    for t in bad:
        with pytest.raises(ValueError, match="the_one"):
            api._refuse(sh, "Q" + kind, ("q", "the_one"), (first, t))
    with pytest.raises(ValueError, match="not what its shape says"):  # nothing to name
        api._refuse(sh, "Q" + kind, ("q", "the_one"), (first, good))


def test_missing_native_checks_fail_loudly(L, monkeypatch, tmp_path):
    monkeypatch.setattr(api, "_binding", None)
    monkeypatch.setattr(api, "_PKG", str(tmp_path))
    with pytest.raises(RuntimeError, match="missing"):
        api._native()


def test_kinds_match_the_entry_points(L):
    """One kind and one name per pointer argument of each entry point."""
    for fn, kinds, names in (
            (L.losa_quantize_prefix, "KK88ssm", 7), (L.losa_append_block_quant, "bb88ssm", 7),
            (L.losa_dequantize_prefix, "88ssKK", 6),
            (L.losa_dense_prefix_quant, "Q88ssbbOLOlW", len(api._DENSE_NAMES)),
            (L.losa_step_quant, "QQ88ssMbbOLOlapuW", len(api._STEP_NAMES))):
        ws = "W" in kinds
        assert len(kinds) == names == len(fn.argtypes) - 2 - ws
        for k in kinds:
            api._expected(S(), k)


# ---- the model the GPU tests compare with ---------------------------------
def test_encode_value_is_the_nearest_code():
    v = np.unique(VALUES[~np.isnan(VALUES)])
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-460, 460, 2000), rng.normal(0, 0.01, 2000), v,
                        (v[1:] + v[:-1]) / 2])
    y = encode_value(x)
    assert np.isin(y, v).all()
    best = np.abs(x[:, None] - v[None]).min(1)
    assert np.array_equal(np.abs(x - y), best)
    # ties go to the even code, and torch's conversion agrees
    t = torch.tensor(x[np.abs(x) < 448], dtype=torch.float32)
    assert np.array_equal(encode_value(t.numpy()), t.to(torch.float8_e4m3fn).float().numpy())


def test_page_scale():
    for amax, want in ((448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (0.0, 1.0),
                       (3.5, 2.0 ** -7), (1e-38, 2.0 ** -100), (448 * 2.0 ** 119, 2.0 ** 119),
                       (3.3e38, 2.0 ** 119), (np.inf, 2.0 ** 119)):
        assert page_scale(np.array([amax, -amax / 3])) == want, amax
    vals, sc = encode(np.full((17, 128), 3.0))
    assert sc.shape == (2,) and np.array_equal(vals * np.repeat(sc, 16)[:17, None], np.full((17, 128), 3.0))
