"""The attention half of the block around the projections: RMS norm with 8-bit output, rotary
positions with several axes, the paged 8-bit key / value cache, and attention over it.

TEST INFRASTRUCTURE ONLY (see the package docstring).  The pages fix none of these operators; each
is defined by the formulas here:

  norm   h = bf16(fp32(x + res)); inv = fp32(1 / sqrt(mean h² + eps)), mean in float64;
         x̂ = ((h·inv)·γ)·fp32(1/λ), each product rounded to float32; MXFP8 of x̂ (oracle/mx.py)
  rope   pair (u, v) of axis a turns by pos[m, a]·freq[i], all in float64
  cache  pages of 64 tokens; per page and head (K and V apart) value = code·2^(byte - 127), the
         exponent the smallest e with max|x| <= 448·2^e in [-110, 119] (-110 for an all-zero
         page); on a page with earlier tokens not below the stored one, the earlier codes rounded
         again where it grows; infinities and NaN have no part in it and become code 0xFF
  attn   softmax over the visible tokens in float64; a row that sees none: 0, lse -inf
"""
import numpy as np

from .formats import bf16_bits_to_f32, bf16_rne, bf16_round_f32, e4m3_decode, e4m3_encode_signed
from . import mx

F32 = np.float32
PAGE = 64
E_MIN, E_MAX = -110, 119


def rmsnorm_quant(X_bits, res_bits, gamma_bits, eps, lam, down_bits):
    """dict(H bits, xhat float32, codes, scales, D float64 or None)."""
    x = bf16_bits_to_f32(X_bits)
    H = X_bits if res_bits is None else bf16_rne(x + bf16_bits_to_f32(res_bits))
    h = bf16_bits_to_f32(H)
    mean = np.sum(h.astype(np.float64) ** 2, axis=1) / h.shape[1]
    inv = (1.0 / np.sqrt(mean + np.float64(F32(eps)))).astype(F32)
    y = h * inv[:, None]
    if gamma_bits is not None:
        y = y * bf16_bits_to_f32(gamma_bits)
    if lam is not None:
        y = y * (F32(1) / lam.astype(F32))
    assert y.dtype == F32
    codes, scales = mx.mx_quantize(y, "e4m3")
    D = None
    if down_bits is not None:
        D = bf16_round_f32(y).astype(np.float64) @ bf16_bits_to_f32(down_bits).astype(np.float64).T
    return dict(H=H, xhat=y, codes=codes, scales=scales, D=D)


def rope(x, pos, freq, axis_dims, interleaved, inverse):
    """x float [M, heads, dim]; float64 values before the output rounding."""
    y = np.asarray(x, np.float64).copy()
    n = sum(axis_dims) // 2
    axis = np.repeat(np.arange(len(axis_dims)), [d // 2 for d in axis_dims])
    ang = pos.astype(np.float64)[:, axis] * freq * (-1.0 if inverse else 1.0)
    c, s = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    u, v = y[:, :, a].copy(), y[:, :, b].copy()
    y[:, :, a] = u * c - v * s
    y[:, :, b] = u * s + v * c
    return y


def k_offset(t, d, dim):
    return ((((t // 32) * (dim // 64) + d // 64) * 2 + d // 16 % 2) * 64 + d // 32 % 2 * 32
            + t % 32) * 16 + d % 16


def v_offset(t, d, dim):
    return (((d // 32) * 2 + t // 32) * 64 + t // 4 % 2 * 32 + d % 32) * 16 + t // 16 % 2 * 8 \
        + t // 8 % 2 * 4 + t % 4


def _place(dim, is_v):
    t, d = np.meshgrid(np.arange(PAGE), np.arange(dim), indexing="ij")
    return (v_offset if is_v else k_offset)(t, d, dim)


def page_exponent(a):
    """Smallest e with a <= 448·2^e, clamped."""
    if a == 0:
        return E_MIN
    e = E_MIN
    while e < E_MAX and float(a) > 448.0 * 2.0 ** e:
        e += 1
    return e


def _encode(x):
    """E4M3 codes, 0xFF for NaN."""
    c = e4m3_encode_signed(np.where(np.isnan(x), 0, x).astype(F32))
    return np.where(np.isnan(x), np.uint8(0xFF), c)


def _decode(codes):
    nan = (codes & 0x7F) == 0x7F
    return np.where(nan, np.nan, e4m3_decode(np.where(nan, np.uint8(0), codes)))


def new_cache(n_pages, heads, dim, fill=0):
    """kc, vc [pages, heads, 64·dim], ks, vs [pages, heads], every byte `fill`."""
    return dict(kc=np.full((n_pages, heads, PAGE * dim), fill, np.uint8),
                vc=np.full((n_pages, heads, PAGE * dim), fill, np.uint8),
                ks=np.full((n_pages, heads), fill, np.uint8),
                vs=np.full((n_pages, heads), fill, np.uint8), dim=dim)


def kv_write(cache, K_bits, V_bits, table, cu, start):
    """Appends in place; pages outside the table or the cache are skipped.  Infinities and NaN have
    no part in the scale and become the code 0xFF."""
    dim, (n_pages, heads) = cache["dim"], cache["ks"].shape
    for is_v, bits, codes, scales in ((0, K_bits, cache["kc"], cache["ks"]),
                                      (1, V_bits, cache["vc"], cache["vs"])):
        x = bf16_bits_to_f32(bits).reshape(-1, heads, dim)
        x = np.where(np.isfinite(x), x, F32(np.nan))
        place = _place(dim, is_v)
        for b in range(len(cu) - 1):
            n, s = cu[b + 1] - cu[b], start[b]
            for p in range(s // PAGE, (s + n + PAGE - 1) // PAGE if n else s // PAGE):
                if p >= table.shape[1] or not 0 <= table[b, p] < n_pages:
                    continue
                page = table[b, p]
                lo, hi = max(0, s - PAGE * p), min(PAGE, s + n - PAGE * p)
                rows = x[cu[b] + PAGE * p + lo - s:cu[b] + PAGE * p + hi - s]
                for h in range(heads):
                    e = page_exponent(np.nan_to_num(np.abs(rows[:, h]), nan=0.0).max())
                    if lo > 0:
                        e0 = int(np.clip(int(scales[page, h]) - 127, E_MIN, E_MAX))
                        e = max(e, e0)
                        if e > e0:
                            at = place[:lo]
                            old = _decode(codes[page, h, at]) * 2.0 ** (e0 - e)
                            codes[page, h, at] = _encode(old)
                    scaled = (rows[:, h].astype(np.float64) * 2.0 ** -e).astype(F32)
                    codes[page, h, place[lo:hi]] = _encode(scaled)
                    scales[page, h] = e + 127


def kv_values(cache, table_row, n, head, is_v):
    """float64 values [n, dim] of a sequence's first n tokens, and which exist (a valid page)."""
    dim, n_pages = cache["dim"], cache["ks"].shape[0]
    codes, scales = (cache["vc"], cache["vs"]) if is_v else (cache["kc"], cache["ks"])
    place = _place(dim, is_v)
    out, ok = np.zeros((n, dim)), np.zeros(n, bool)
    for p in range((n + PAGE - 1) // PAGE):
        if p >= len(table_row) or not 0 <= table_row[p] < n_pages:
            continue
        m = min(PAGE, n - PAGE * p)
        v = _decode(codes[table_row[p], head, place[:m]])
        out[PAGE * p:PAGE * p + m] = v * 2.0 ** (int(scales[table_row[p], head]) - 127)
        ok[PAGE * p:PAGE * p + m] = True
    return out, ok


def attention(Q, cache, table, cu, kv_len, scale, causal, values=kv_values):
    """Q float [rows, q_heads, dim]: dict(O, lse float64, absO = Σ p|v|, absz = scale·max_t
    Σ_d |q_d k_td| of every row, the magnitudes that rounding errors are relative to).  What a row
    does not see has no part in it, NaN included; a query with an infinity or NaN is NaN.  values:
    what reads the cache."""
    rows, Hq, dim = Q.shape
    H = cache["ks"].shape[1]
    G = Hq // H
    O, absO = np.zeros((rows, Hq, dim)), np.zeros((rows, Hq, dim))
    lse, absz = np.full((rows, Hq), -np.inf), np.zeros((rows, Hq))
    for b in range(len(cu) - 1):
        n, kv = cu[b + 1] - cu[b], min(int(kv_len[b]), PAGE * table.shape[1])
        if n <= 0 or kv <= 0:
            continue
        see = np.arange(kv)[None, :] < ((kv - n + np.arange(n) + 1)[:, None] if causal else kv)
        for h in range(H):
            k, ok = values(cache, table[b], kv, h, 0)
            v, _ = values(cache, table[b], kv, h, 1)
            vis = see & ok[None, :]
            for g in range(G):
                j = h * G + g
                q = Q[cu[b]:cu[b + 1], j].astype(np.float64)
                q = np.where(np.isfinite(q).all(axis=1, keepdims=True), q, np.nan)
                z = np.where(vis, scale * (q @ k.T), -np.inf)
                m = z.max(axis=1, keepdims=True)
                m = np.where(np.isneginf(m), 0.0, m)
                p = np.exp(z - m)
                l = p.sum(axis=1, keepdims=True)
                some = l[:, 0] != 0
                p = p / np.where(l != 0, l, 1.0)
                seen_nan = np.where(vis.astype(np.float64) @ np.isnan(v) > 0, np.nan, 0.0)
                v0 = np.nan_to_num(v, nan=0.0)
                O[cu[b]:cu[b + 1], j] = p @ v0 + seen_nan
                absO[cu[b]:cu[b + 1], j] = p @ np.abs(v0)
                absz[cu[b]:cu[b + 1], j] = scale * np.nan_to_num(
                    np.abs(q) @ np.nan_to_num(np.abs(k)).T).max(axis=1)
                with np.errstate(divide="ignore"):
                    lse[cu[b]:cu[b + 1], j] = np.where(some, m[:, 0] + np.log(l[:, 0]), -np.inf)
    return dict(O=O, lse=lse, absO=absO, absz=absz)
