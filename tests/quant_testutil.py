"""The 8-bit prefix cache in 64 bits, from its definition: what the GPU tests
compare the library's calls with.

A page (16 tokens) of K or V of one KV head is stored as e4m3 codes and a
scale: the smallest power of two >= 2^-100 with amax <= 448 * scale (1 for a
page of zeros), codes rounded to nearest, ties to even, saturating."""
from __future__ import annotations

import math

import numpy as np
import torch

from sparse_long_context_mse_b200 import api

PS, D = 16, 128
F8 = torch.float8_e4m3fn


def e4m3_values() -> np.ndarray:
    """The 256 codes' values (NaN for 0x7f and 0xff), from the format: 1 sign, 4
    exponent (bias 7) and 3 mantissa bits."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = math.nan if (c & 127) == 127 else x
    v[128:] = -v[128:]
    return v


VALUES = e4m3_values()


def encode_value(x: np.ndarray) -> np.ndarray:
    """The e4m3 numbers nearest to x (ties to the even code), as float64."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -60))), -6)
    e = np.where(2.0 ** (e + 1) <= a, e + 1, np.where(2.0 ** e > a, e - 1, e))
    step = 2.0 ** (np.maximum(e, -6) - 3)
    y = np.minimum(np.rint(a / step) * step, 448.0)  # (np.rint: ties to even)
    return np.where(np.isnan(x), np.nan, np.copysign(y, x))


def page_scale(page: np.ndarray) -> float:
    a = np.abs(np.asarray(page, np.float64))
    a = a[~np.isnan(a)]
    amax = float(a.max()) if a.size else 0.0
    if amax == 0.0:
        return 1.0
    e = -100
    while e < 119 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def encode(x: np.ndarray):
    """(values of the codes [n][D], scales [pages]) of the n >= 1 tokens of one KV head."""
    x = np.asarray(x, np.float64)
    out, sc = np.empty_like(x), []
    with np.errstate(over="ignore", invalid="ignore"):
        for j in range(0, len(x), PS):
            s = page_scale(x[j:j + PS])
            out[j:j + PS] = encode_value(x[j:j + PS] / s)
            sc.append(s)
    return out, np.array(sc)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy().astype(np.float64)


def same(a, b) -> bool:
    """Equal as numbers, NaN equal to NaN."""
    return np.array_equal(np.asarray(a), np.asarray(b), equal_nan=True)


def lens_of(sh) -> list:
    t = getattr(sh, "_prefix_lens", None)
    return [sh.prefix_len] * sh.num_seqs if t is None else [int(v) for v in t.cpu()]


def read_back(k8: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    """code * scale of every token, in float64, on the tensors' device."""
    n = k8.shape[2]
    return k8.float().double() * scale.double().repeat_interleave(PS, 2)[:, :, :n, None]


def random_prefix(sh, gen, device, tail=float("nan"), amp=1.0):
    """K and V of the shape's capacity, N(0, amp^2) up to each sequence's length and
    `tail` past it."""
    kv = (sh.num_seqs, sh.n_kv_heads, sh.capacity, D)
    out = []
    for _ in range(2):
        x = amp * torch.randn(kv, generator=gen)
        for s, n in enumerate(lens_of(sh)):
            x[s, :, n:] = tail
        out.append(x.to(sh.torch_dtype).to(device))
    return out


def attention(q, k, v, scale):
    """Softmax attention in float64: q [.., r, D], k and v [.., n, D] -> (o, lse, T), T the
    largest sum of |terms| of a score (natural-log units)."""
    w = torch.matmul(q, k.transpose(-1, -2)) * scale
    t = torch.matmul(q.abs(), k.abs().transpose(-1, -2)).max().item() * scale if k.shape[-2] else 0.0
    return torch.matmul(torch.softmax(w, -1), v), torch.logsumexp(w, -1), t


def dense_reference(sh, q, k8, v8, ks, vs, kb, vb):
    """losa_dense_prefix_quant's results in float64, and the error bounds of its fp32
    arithmetic: see `dense_bounds`."""
    S, Hq, Hkv, B = sh.num_seqs, sh.n_q_heads, sh.n_kv_heads, sh.block_size
    G = Hq // Hkv
    scale = sh.scale if sh.scale > 0 else 1 / math.sqrt(D)
    K, V = read_back(k8, ks), read_back(v8, vs)
    got = {"o_p": torch.empty(S, Hq, B, D, dtype=torch.float64), "l_p": torch.empty(S, Hq, B, dtype=torch.float64)}
    got["out"], got["lse"] = torch.empty_like(got["o_p"]), torch.empty_like(got["l_p"])
    tmax, small, vmax = 0.0, 0.0, 0.0
    for s, n in enumerate(lens_of(sh)):
        for g in range(Hkv):
            h = slice(g * G, (g + 1) * G)
            qq = q[s, h].double().reshape(G * B, D)
            kk, vv = K[s, g, :n], V[s, g, :n]
            o, l, t = attention(qq, kk, vv, scale)
            ka = torch.cat((kk, kb[s, g].double()))
            va = torch.cat((vv, vb[s, g].double()))
            oa, la, ta = attention(qq, ka, va, scale)
            got["o_p"][s, h], got["l_p"][s, h] = o.reshape(G, B, D).cpu(), l.reshape(G, B).cpu()
            got["out"][s, h], got["lse"][s, h] = oa.reshape(G, B, D).cpu(), la.reshape(G, B).cpu()
            tmax = max(tmax, t, ta)
            small = max(small, qq.abs().max().item() * ka.abs().sum(-1).max().item() * scale)
            vmax = max(vmax, va.abs().max().item())
    return got, dense_bounds(tmax, small, vmax, got["lse"].abs().max().item())


def dense_bounds(T, small, vmax, lse):
    """Error bounds of the dense pass.  T: the largest sum of |terms| of a score; small:
    the largest (row maximum of |q|) * (sum of |k|), both in natural-log units.

    * A query row is split into 8-bit parts: bf16 rows into two, exact but for elements near
      the bottom of the row's range, where the error is at most 2^-21 of the row's maximum
      (2^-29 with the six parts of an fp32 row): 2^-21 small.
    * The score is summed in fp32 by the tensor core, at most 16 accumulations of
      2^-24 T (or one rounding per channel on CUDA cores: 128 of 2^-24 T): 2^-17 T.
    * Scaling the score and the exponential add 2^-20 in all.
    The sum d of these is the relative error of a weight.  Output: both the weighted sum
    and the normaliser carry d, and the weights' rounding (2^-21), the truncating
    accumulations of a tile (16 of 2^-24), the sums over tiles and the merges add 2^-16 of
    max|v|.  Log-normaliser: d, and 2^-22 of its own size."""
    d = 2.0 ** -21 * small + 2.0 ** -17 * T + 2.0 ** -20
    return {"o": (2 * d + 2.0 ** -16) * vmax, "l": d + 2.0 ** -20 + 2.0 ** -22 * lse}


def alloc_state(sh, device, fill=float("nan")):
    rows = (sh.num_seqs, sh.n_q_heads, sh.block_size)
    mk = lambda *t: torch.full((*rows, *t), fill, device=device)
    return {"o_p": mk(D), "l_p": mk(), "out": mk(D), "lse": mk()}


def gpu_dense_quant(sh, q, cache, kb, vb, ws=None, stream=None):
    st = alloc_state(sh, q.device)
    if ws is None:
        ws = api.alloc_workspace(sh, api.LOSA_WS_DENSE_QUANT, q.device)
    api.dense_prefix_quant(sh, q, *cache, kb, vb, st["o_p"], st["l_p"], st["out"], st["lse"], ws,
                           stream=stream)
    return st


def check_dense(got, ref, bounds, what=""):
    for key in ("o_p", "out", "l_p", "lse"):
        g = got[key].cpu().double()
        assert torch.isfinite(g).all(), (what, key)
        err = (g - ref[key]).abs().max().item()
        tol = bounds["o" if key in ("o_p", "out") else "l"]
        assert err <= tol, f"{what} {key}: max-abs error {err:.3g} > {tol:.3g}"
