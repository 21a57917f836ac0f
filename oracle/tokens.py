"""Single tokens and the 4-bit cache: norm of the query and key heads with rotary positions, the paged
4-bit key / value cache and attention over it, and the layer for a few rows with 16-bit activations.

TEST INFRASTRUCTURE ONLY (see the package docstring).  The pages fix none of these operators; each is
defined by the formulas here, in float64 but for the roundings that belong to the definition:

  qk     z = x·γ / sqrt(mean x² + eps) per head, then the turn of oracle/attention.py's rope
  cache  pages of 64 tokens; per token, head and 32 channels an MXFP4 block (oracle/mx.py) with the
         exponent within [-110, 85] (-110 for zeros); a block with an infinity or NaN: scale byte 255,
         codes 0
  attn   oracle/attention.py's attention over those values
  gemv   x̂ = bf16(fl32(x·fl32(1/λ))); Σ x̂·w + (x̂·downᵀ)·upᵀ with w the dequantised weight
"""
import numpy as np

from .formats import (bf16_bits_to_f32, bf16_round_f32, e2m1_decode, e4m3_decode, pack_nibbles,
                      unpack_nibbles)
from . import attention as OA, mx

F32 = np.float32
PAGE = OA.PAGE
E_MIN, E_MAX = -110, 85
NAN_SCALE = 255


def qk_norm_rope(x, q_heads, gamma_q_bits, gamma_k_bits, eps, pos, freq, axis_dims, interleaved):
    """x float [M, heads, dim]: (float64 values before the output rounding, the normed heads z)."""
    z = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        z = z * (1.0 / np.sqrt(np.mean(z * z, axis=2, keepdims=True) + np.float64(F32(eps))))
        for part, g in ((z[:, :q_heads], gamma_q_bits), (z[:, q_heads:], gamma_k_bits)):
            if g is not None:
                part *= bf16_bits_to_f32(g).astype(np.float64)
        return OA.rope(z, pos, freq, axis_dims, interleaved, False), z


# ------------------------------------------------------------------------------------------
# the cache
# ------------------------------------------------------------------------------------------

def k_place(t, d, dim):
    return ((t // 32 * (dim // 64) + d // 64) * 64 + d // 32 % 2 * 32 + t % 32) * 16 + d % 32 // 2


def k_scale_place(t, d, dim):
    return (d // 32 % 2 * 32 + t % 32) * (dim // 32) + t // 32 * (dim // 64) + d // 64


def v_place(t, d, dim):
    return ((d // 64 * 2 + t // 32) * 64 + t // 4 % 2 * 32 + d // 2 % 32) * 16 + t // 16 % 2 * 8 \
        + t // 8 % 2 * 4 + t % 4


def v_scale_place(t, d, dim):
    return (d // 32 * 2 + t // 4 % 2) * 32 + t // 16 * 8 + t // 8 % 2 * 4 + t % 4


def _places(dim, is_v):
    """Code bytes [64, dim / 2] and scale bytes [64, dim / 32] of a page's tokens."""
    t = np.arange(PAGE)[:, None]
    code, scale = (v_place, v_scale_place) if is_v else (k_place, k_scale_place)
    return code(t, np.arange(0, dim, 2)[None], dim), scale(t, np.arange(0, dim, 32)[None], dim)


def quantise(x):
    """Tokens x float32 [..., dim]: (codes packed [..., dim / 2], scale bytes [..., dim / 32])."""
    x = np.asarray(x, F32)
    lead, dim = x.shape[:-1], x.shape[-1]
    blk = x.reshape(*lead, dim // 32, 32)
    bad = ~np.isfinite(blk).all(axis=-1)
    blk = np.where(bad[..., None], F32(0), blk)
    a = np.abs(blk).max(axis=-1, initial=0)
    e = np.clip(np.where(a == 0, E_MIN, mx.mx_exponent(a, "e2m1")), E_MIN, E_MAX)
    with np.errstate(over="ignore"):
        codes = mx.mx_element_codes(blk, np.broadcast_to(e[..., None], blk.shape), "e2m1")
    return (pack_nibbles(codes.reshape(-1, dim)).reshape(*lead, dim // 2),
            np.where(bad, NAN_SCALE, e + 127).astype(np.uint8))


def dequantise(codes, scales):
    """float64 values [..., dim] of packed codes [..., dim / 2]."""
    v = e2m1_decode(unpack_nibbles(codes.reshape(-1, codes.shape[-1])))
    v = v.reshape(*scales.shape, 32) * np.ldexp(1.0, scales.astype(np.int64) - 127)[..., None]
    return np.where((scales == NAN_SCALE)[..., None], np.nan, v).reshape(*scales.shape[:-1], 2 * codes.shape[-1])


def new_cache(n_pages, heads, dim, fill=0):
    """kc, vc [pages, heads, 32·dim], ks, vs [pages, heads, 2·dim], every byte `fill`."""
    z = lambda n: np.full((n_pages, heads, n), fill, np.uint8)  # noqa: E731
    return dict(kc=z(32 * dim), vc=z(32 * dim), ks=z(2 * dim), vs=z(2 * dim), dim=dim)


def kv_write(cache, K_bits, V_bits, table, cu, start):
    """Appends in place; pages outside the table or the cache are skipped."""
    dim, (n_pages, heads) = cache["dim"], cache["ks"].shape[:2]
    for is_v, bits, codes, scales in ((0, K_bits, cache["kc"], cache["ks"]),
                                      (1, V_bits, cache["vc"], cache["vs"])):
        c, s = quantise(bf16_bits_to_f32(bits).reshape(-1, heads, dim))
        at_c, at_s = _places(dim, is_v)
        for b in range(len(cu) - 1):
            for i in range(cu[b + 1] - cu[b]):
                p, t = divmod(int(start[b]) + i, PAGE)
                if p >= table.shape[1] or not 0 <= table[b, p] < n_pages:
                    continue
                codes[table[b, p], :, at_c[t]] = c[cu[b] + i].T
                scales[table[b, p], :, at_s[t]] = s[cu[b] + i].T


def kv_values(cache, table_row, n, head, is_v):
    """float64 values [n, dim] of a sequence's first n tokens, and which exist (a valid page)."""
    dim, n_pages = cache["dim"], cache["ks"].shape[0]
    codes, scales = (cache["vc"], cache["vs"]) if is_v else (cache["kc"], cache["ks"])
    at_c, at_s = _places(dim, is_v)
    out, ok = np.zeros((n, dim)), np.zeros(n, bool)
    for p in range((n + PAGE - 1) // PAGE):
        if p >= len(table_row) or not 0 <= table_row[p] < n_pages:
            continue
        m = min(PAGE, n - PAGE * p)
        page = table_row[p], head
        out[PAGE * p:PAGE * p + m] = dequantise(codes[page][at_c[:m]], scales[page][at_s[:m]])
        ok[PAGE * p:PAGE * p + m] = True
    return out, ok


def attention(Q, cache, table, cu, kv_len, scale, causal):
    return OA.attention(Q, cache, table, cu, kv_len, scale, causal, values=kv_values)


# ------------------------------------------------------------------------------------------
# the layer for a few rows
# ------------------------------------------------------------------------------------------

def weight_values(codes, scales, g, fmt):
    """float64 [N, K] of a prepared weight (oracle/layer.py's fields)."""
    nib = unpack_nibbles(codes)
    if fmt == "int4":
        v, s, n = np.where(nib > 7, nib.astype(np.int64) - 16, nib).astype(np.float64), scales.astype(np.float64), 64
    elif fmt == "nvfp4":
        v, s, n = e2m1_decode(nib), e4m3_decode(scales).astype(np.float64) * np.float64(g), 16
    else:
        v, s, n = e2m1_decode(nib), np.ldexp(1.0, scales.astype(np.int64) - 127), 32
    return (v.reshape(len(v), -1, n) * s[..., None]).reshape(v.shape)


def gemv(X_bits, lam, down_bits, up_bits, w):
    """(float64 Y, A: the sum of the magnitudes of the products that make it up)."""
    x = bf16_bits_to_f32(X_bits)
    if lam is not None:
        x = bf16_round_f32(x * (F32(1) / lam.astype(F32)))
    x = x.astype(np.float64)
    y, a = x @ w.T, np.abs(x) @ np.abs(w).T
    if down_bits is not None:
        d, u = (bf16_bits_to_f32(v).astype(np.float64) for v in (down_bits, up_bits))
        y = y + (x @ d.T) @ u.T
        a = a + (np.abs(x) @ np.abs(d).T) @ np.abs(u).T
    return y, a
