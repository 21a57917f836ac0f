"""Allocating helpers over the C ABI for the W4A4 layer (torch provides memory and streams).

Every numeric step runs in libsvdq.so; these functions only allocate outputs and call the
entry points in order: calibration -> weight preparation -> activation quantisation with the
low-rank down-projection -> W4A4 GEMM.
"""
from dataclasses import dataclass

from . import _lib
from ._lib import NVFP4, INT4_G64, MXFP4, MXFP8  # noqa: F401


def _torch():
    import torch
    return torch


@dataclass
class PreparedWeight:
    fmt: int
    N: int
    K: int
    r: int
    codes: object        # uint8 [N, K/2] (MXFP8: [N, K])
    scales: object       # uint8 [N, K/16] (E4M3), float16 [N, K/64] or uint8 [N, K/32] (E8M0)
    g: object            # float32 [1] (NVFP4) or None
    lora_up: object      # bf16 [N, r] or None


def _alloc_codes_scales(fmt, rows, K, dev):
    """Code and scale tensors of one format; the NVFP4 tensor scale (else None)."""
    torch = _torch()
    codes = torch.empty(rows, K if fmt == MXFP8 else K // 2, dtype=torch.uint8, device=dev)
    g = None
    if fmt == NVFP4:
        scales = torch.empty(rows, K // 16, dtype=torch.uint8, device=dev)
        g = torch.empty(1, dtype=torch.float32, device=dev)
    elif fmt == INT4_G64:
        scales = torch.empty(rows, K // 64, dtype=torch.float16, device=dev)
    else:
        scales = torch.empty(rows, K // 32, dtype=torch.uint8, device=dev)
    return codes, scales, g


def calibrate(X, seg, W=None, mask=7, alpha=0.5, state=None):
    """λ calibration on X [M, K]; pass the previous result as `state` to accumulate batches."""
    torch = _torch()
    K = X.shape[1]
    dev = X.device
    if state is None:
        state = dict(ax=torch.empty(3, K, device=dev), aw=torch.empty(K, device=dev),
                     **{"lambda": torch.empty(K, device=dev)},
                     act_amax=torch.empty(1, device=dev))
        acc = 0
    else:
        acc = 1
    _lib.svdq_calibrate_lambda(X, seg, W, mask, alpha, acc, state["ax"], state["aw"],
                               state["lambda"], state["act_amax"])
    return state


def bits_lost(ax, lam=None, block=16):
    """Bits-lost proxy per modality (float64 [3]) of the smoothing λ for per-modality channel
    maxima ax [3, K] (the `ax` of a calibration state); block = the quantiser's group size."""
    torch = _torch()
    out = torch.empty(3, dtype=torch.float64, device=ax.device)
    _lib.svdq_bits_lost(ax, lam, block, out)
    return out


def lowrank_factors(W, lam, omega, r, power_iters=2):
    """Randomized rank-r factors of diag(λ)·Wᵀ on the GPU: (lora_down [r, K], lora_up [N, r],
    sigma [r]).  omega [N, ell] fp32 is the caller's random matrix (ell >= r)."""
    torch = _torch()
    N, K = W.shape
    ell = omega.shape[1]
    dev = W.device
    down = torch.empty(r, K, dtype=torch.bfloat16, device=dev)
    up = torch.empty(N, r, dtype=torch.bfloat16, device=dev)
    sigma = torch.empty(r, dtype=torch.float32, device=dev)
    nbytes = _lib.svdq_lowrank_workspace_bytes(N, K, ell)
    if nbytes < 0:
        raise ValueError(f"unsupported sketch width {ell}")
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=dev)
    off = (-ws.data_ptr()) % 256
    _lib.svdq_lowrank_factors(W, lam, omega, r, power_iters, down, up, sigma,
                              ws[off:off + nbytes])
    return down, up, sigma


# The 39 migration strengths α = i/40 of the λ grid (λ_k = a_k^α / w_k^(1−α)).
ALPHA_GRID = tuple(i / 40.0 for i in range(1, 40))


def lambda_search(X, W, state, alphas, rows, fmt=NVFP4, omega=None, r=32, power_iters=2,
                  mask=7, refit_iters=0, per_iterate=False):
    """λ grid search on the GPU: for each α the layer's output error on the sampled rows
    (device int32 indices into X), the smallest over refit_iters refits of the low-rank branch.
    Returns dict(scores fp64 [n_alpha], lam (the winner's λ), index, and when r > 0 the
    winner's best factors lora_down [r, K] / lora_up [N, r]; with per_iterate the score of
    every iterate, fp64 [n_alpha, refit_iters + 1])."""
    torch = _torch()
    N, K = W.shape
    dev = X.device
    ell = omega.shape[1] if omega is not None else 0
    n = len(alphas)
    out = dict(scores=torch.empty(n, dtype=torch.float64, device=dev),
               lam=torch.empty(K, dtype=torch.float32, device=dev),
               index=torch.empty(1, dtype=torch.int32, device=dev))
    if per_iterate:
        out["iter_scores"] = torch.empty(n, refit_iters + 1, dtype=torch.float64, device=dev)
    if r > 0:
        out["lora_down"] = torch.empty(r, K, dtype=torch.bfloat16, device=dev)
        out["lora_up"] = torch.empty(N, r, dtype=torch.bfloat16, device=dev)
    nbytes = _lib.svdq_lambda_search_workspace_bytes(fmt, N, K, ell, r, rows.numel(), n,
                                                     refit_iters)
    if nbytes < 0:
        raise ValueError("unsupported search shape")
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=dev)
    off = (-ws.data_ptr()) % 256
    _lib.svdq_lambda_search(X, W, state["ax"], state["aw"], mask, alphas, fmt, omega, r,
                            power_iters, refit_iters, rows, out["scores"], out.get("iter_scores"),
                            out["lam"], out["index"], out.get("lora_down"), out.get("lora_up"),
                            ws[off:off + nbytes])
    return out


def prepare_weight(W, lam, lora_down, lora_up, fmt=NVFP4, workspace=None):
    """Quantised residual of diag(λ)·W − L1·L2 (W [N, K] bf16).  With `workspace` (uint8, at
    least quantize_weight_workspace_bytes, 256-byte aligned) the NVFP4 residual is formed once."""
    torch = _torch()
    N, K = W.shape
    r = 0 if lora_down is None else lora_down.shape[0]
    codes, scales, g = _alloc_codes_scales(fmt, N, K, W.device)
    if workspace is None:
        _lib.svdq_quantize_weight(fmt, W, lam, lora_down, lora_up, r, codes, scales, g)
    else:
        _lib.svdq_quantize_weight_ws(fmt, W, lam, lora_down, lora_up, r, codes, scales, g,
                                     workspace)
    return PreparedWeight(fmt, N, K, r, codes, scales, g, lora_up)


def quantize_weight_workspace(N, K, fmt=NVFP4, device="cuda"):
    """A 256-byte aligned workspace for prepare_weight(..., workspace=...)."""
    torch = _torch()
    nb = _lib.svdq_quantize_weight_workspace_bytes(fmt, N, K)
    buf = torch.empty(nb + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + nb]


def gptq_hessian(X, lam, H=None):
    """H [K, K] fp64 (+)= X̂ᵀX̂ of the calibration rows X; pass H back to accumulate batches."""
    torch = _torch()
    K = X.shape[1]
    if H is None:
        H = torch.empty(K, K, dtype=torch.float64, device=X.device)
        _lib.svdq_gptq_hessian(X, lam, H, accumulate=False)
    else:
        _lib.svdq_gptq_hessian(X, lam, H, accumulate=True)
    return H


def prepare_weight_gptq(W, lam, lora_down, lora_up, H, fmt=NVFP4):
    """prepare_weight with the residual GPTQ-rounded under the Hessian H."""
    torch = _torch()
    N, K = W.shape
    r = 0 if lora_down is None else lora_down.shape[0]
    codes, scales, g = _alloc_codes_scales(fmt, N, K, W.device)
    nbytes = _lib.svdq_gptq_workspace_bytes(N, K)
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=W.device)
    off = (-ws.data_ptr()) % 256
    _lib.svdq_gptq_quantize_weight(fmt, W, lam, lora_down, lora_up, r, H, codes, scales, g,
                                   ws[off:off + nbytes])
    return PreparedWeight(fmt, N, K, r, codes, scales, g, lora_up)


def quantize_activation(X, lam, act_amax, lora_down, fmt=NVFP4, sat_count=None):
    """(codes, scales, g_a, D) of X [M, K]."""
    torch = _torch()
    M, K = X.shape
    r = 0 if lora_down is None else lora_down.shape[0]
    dev = X.device
    codes, scales, g = _alloc_codes_scales(fmt, M, K, dev)
    D = torch.empty(M, r, dtype=torch.float32, device=dev) if r else None
    _lib.svdq_quant_act_lowrank_down(fmt, X, lam, act_amax, lora_down, r, codes, scales, g, D,
                                     sat_count)
    return codes, scales, g, D


def cube_geometry(T, H, W, ct, ch, cw, n_text, n_audio, cube1d, device="cuda"):
    """DeltaQuant geometry on the host, uploaded: dict(row_to_cube, cube_ptr, cube_rows,
    group_ptr (device int32), n_cubes, host (the numpy arrays))."""
    import numpy as np
    torch = _torch()
    r2c, ptr, rows = _lib.svdq_cube_geometry(T, H, W, ct, ch, cw, n_text, n_audio, cube1d)
    gp = _lib.svdq_cube_groups(ptr)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
    return dict(row_to_cube=up(r2c), cube_ptr=up(ptr), cube_rows=up(rows), group_ptr=up(gp),
                n_cubes=len(ptr) - 1, host=dict(row_to_cube=r2c, cube_ptr=ptr, cube_rows=rows,
                                                group_ptr=gp))


def delta_quantize_activation(X, lam, act_amax, geo, lora_down, out=None, sat_count=None):
    """DeltaQuant activations of X [M, K] for the cube geometry `geo` (cube_geometry, or a dict
    with device cube_ptr / cube_rows / group_ptr and n_cubes): dict with core codes cc
    [n_cubes, K], core scales cs [n_cubes], delta codes dc [M, K/2] and scales dsc [M, K/16],
    g_delta gd [1], D [M, r] (fp32) and the fp32 core workspace ws.  Pass `out` to reuse its
    tensors."""
    torch = _torch()
    M, K = X.shape
    r = 0 if lora_down is None else lora_down.shape[0]
    dev = X.device
    u8 = torch.uint8
    nc = geo["n_cubes"]
    if out is None:
        nbytes = _lib.svdq_delta_workspace_bytes(nc, K)
        ws = torch.empty(nbytes + 256, dtype=u8, device=dev)
        off = (-ws.data_ptr()) % 256
        out = dict(cc=torch.empty(nc, K, dtype=u8, device=dev),
                   cs=torch.empty(nc, device=dev),
                   dc=torch.empty(M, K // 2, dtype=u8, device=dev),
                   dsc=torch.empty(M, K // 16, dtype=u8, device=dev),
                   gd=torch.empty(1, device=dev),
                   D=torch.empty(M, r, device=dev) if r else None,
                   ws=ws[off:off + nbytes])
    _lib.svdq_delta_quant_act(X, lam, act_amax, geo["cube_ptr"], geo["cube_rows"], nc,
                              geo["group_ptr"], lora_down, r, out["cc"], out["cs"], out["dc"],
                              out["dsc"], out["gd"], out.get("D"), sat_count, out["ws"])
    return out


def gemm(codes, scales, g_a, D, pw, M, out=None, core_out=None, row_to_cube=None):
    torch = _torch()
    Y = out if out is not None else torch.empty(M, pw.N, dtype=torch.bfloat16, device=codes.device)
    _lib.svdq_w4a4_gemm(pw.fmt, M, pw.N, pw.K, codes, scales, g_a, pw.codes, pw.scales, pw.g, D,
                        pw.lora_up, pw.r, Y, core_out, row_to_cube)
    return Y


def forward(X, pw, act_amax, lam, lora_down, out=None):
    """Y = X̂·L1·L2 + Q(X̂)·Q(R) for X [..., K]; leading dimensions are flattened exactly once."""
    lead = X.shape[:-1]
    X2 = X.reshape(-1, X.shape[-1])
    codes, scales, g, D = quantize_activation(X2, lam, act_amax, lora_down, pw.fmt)
    Y = gemm(codes, scales, g, D, pw, X2.shape[0], out=out)
    return Y.reshape(*lead, pw.N)


def _bytes(n, device):
    """A 256-byte aligned workspace of n bytes."""
    buf = _torch().empty(n + 256, dtype=_torch().uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + n]


def gemv_workspace(rows, pw, device="cuda"):
    """A workspace for gemv() of so many rows."""
    nb = _lib.svdq_w4a16_gemv_workspace_bytes(rows, pw.N, pw.K, pw.r)
    if nb < 0:
        raise ValueError(f"unsupported: {rows} rows (at most 64), N={pw.N}, K={pw.K}, rank {pw.r}")
    return _bytes(nb, device)


def gemv(X, pw, lam, lora_down, out=None, workspace=None):
    """forward() of at most 64 rows without activation quantisation: Y = X̂·L1·L2 + X̂·Q(R) with the
    16-bit X̂ = bf16(X / λ) for X [..., K] bf16 and a 4-bit weight pw (NVFP4, INT4_G64, MXFP4); out: bf16
    [rows, N].  For single tokens and small batches, where the weight's bytes are the work."""
    torch = _torch()
    lead = X.shape[:-1]
    X2 = X if X.dim() == 2 else X.reshape(-1, X.shape[-1])
    M = X2.shape[0]
    Y = out if out is not None else torch.empty(M, pw.N, dtype=torch.bfloat16, device=X.device)
    if workspace is None and M:
        workspace = gemv_workspace(M, pw, X.device)
    _lib.svdq_w4a16_gemv(pw.fmt, X2, lam, lora_down, pw.r, pw.codes, pw.scales, pw.g, pw.lora_up, pw.N,
                         Y, workspace)
    return Y if len(lead) == 1 else Y.reshape(*lead, pw.N)


# ------------------------------------------------------------------------------------------
# the attention half of the block
# ------------------------------------------------------------------------------------------

KV_PAGE = 64   # tokens of a cache page


def norm_quantize_activation(X, gamma, lam, lora_down, eps=1e-6, residual=None, out_residual=None):
    """MXFP8 activations (codes, scales, D, H) of the RMS norm of X + residual, [M, K] bf16:
    what gemm() of an MXFP8 weight takes, and the new residual stream H (X itself without a
    residual).  out_residual: where H goes (X or residual: in place)."""
    torch = _torch()
    M, K = X.shape
    r = 0 if lora_down is None else lora_down.shape[0]
    dev = X.device
    codes = torch.empty(M, K, dtype=torch.uint8, device=dev)
    scales = torch.empty(M, K // 32, dtype=torch.uint8, device=dev)
    D = torch.empty(M, r, dtype=torch.float32, device=dev) if r else None
    H = X
    if residual is not None:
        H = out_residual if out_residual is not None else torch.empty(M, K, dtype=X.dtype,
                                                                      device=dev)
    _lib.svdq_rmsnorm_quant_act(X, residual, H if residual is not None else None, gamma, eps, lam,
                                lora_down, r, codes, scales, D)
    return codes, scales, D, H


def rope_frequencies(axis_dims, theta=10000.0, device="cuda"):
    """Frequencies of rope(): device float64 [sum(axis_dims) / 2]."""
    torch = _torch()
    return torch.from_numpy(_lib.svdq_rope_frequencies(axis_dims, theta)).to(device)


def rope(X, pos, freq, axis_dims, dim, interleaved=True, inverse=False, out=None):
    """Rotary positions of the heads of X [M, heads·dim] bf16; pos int32 [M, axes] (time, height,
    width of every row), freq from rope_frequencies.  out=X turns in place."""
    torch = _torch()
    Y = out if out is not None else torch.empty(X.shape, dtype=X.dtype, device=X.device)
    _lib.svdq_rope_axes(X, X.shape[1] // dim, dim, pos, freq, axis_dims, interleaved, inverse, Y)
    return Y


def qk_norm_rope(X, pos, freq, axis_dims, dim, q_heads, gamma_q, gamma_k, eps=1e-6, interleaved=True,
                 out=None):
    """RMS norm of every head of X [M, heads·dim] bf16 with the rotary positions in the same pass: the
    first q_heads heads with gamma_q, the others (keys) with gamma_k (bf16 [dim]; None: 1).  pos, freq
    and axis_dims as rope() takes them.  out=X works in place."""
    # (empty_like: 0.7 us instead of 2 for the same by shape, type and device, of a call of 10)
    Y = out if out is not None else _torch().empty_like(X)
    _lib.svdq_qk_norm_rope(X, q_heads, X.shape[1] // dim - q_heads, dim, gamma_q, gamma_k, eps, pos,
                           freq, axis_dims, interleaved, Y)
    return Y


@dataclass
class KVCache:
    k_codes: object      # uint8 [pages, heads, 64·dim], operand order (include/svdq.h); 4 bits: 32·dim
    v_codes: object
    k_scales: object     # uint8 [pages, heads]: the page's exponent + 127; 4 bits: [pages, heads, 2·dim]
    v_scales: object
    dim: int
    bits: int = 8        # 8: E4M3 codes, a scale per page and head; 4: MXFP4, one per token and 32 channels


def _by_bits(bits, eight, four):
    if bits not in (4, 8):
        raise ValueError(f"a cache of {bits} bits: must be 4 or 8")
    return eight if bits == 8 else four


def kv_cache(n_pages, heads, dim, device="cuda", bits=8):
    """An empty paged cache of n_pages pages of 64 tokens, of 8 or 4 bits."""
    torch = _torch()
    if bits not in (4, 8):
        raise ValueError(f"a cache of {bits} bits: must be 4 or 8")
    codes = [torch.zeros(n_pages, heads, KV_PAGE * dim * bits // 8, dtype=torch.uint8, device=device)
             for _ in range(2)]
    shape = (n_pages, heads) if bits == 8 else (n_pages, heads, 2 * dim)
    scales = [torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2)]
    return KVCache(codes[0], codes[1], scales[0], scales[1], dim, bits)


def kv_write(cache, K, V, block_table, cu_rows, start, max_rows):
    """Append the packed rows K, V [rows, heads·dim] bf16: sequence b's rows cu_rows[b] ..
    cu_rows[b + 1] become its tokens start[b] onward, quantised with one scale a page and head (8
    bits) or a token and 32 channels (4 bits)."""
    _by_bits(cache.bits, _lib.svdq_kv_write, _lib.svdq_kv4_write)(
        K, V, cache.dim, cu_rows, start, max_rows, block_table, cache.k_codes, cache.v_codes,
        cache.k_scales, cache.v_scales)


def kv_read(cache, block_table, cu_rows, start, rows, max_rows, out=None):
    """(K, V) [rows, heads·dim] bf16 of tokens start[b] onward of each sequence."""
    torch = _torch()
    if out is None:
        K = torch.empty(rows, cache.k_codes.shape[1] * cache.dim, dtype=torch.bfloat16,
                        device=cache.k_codes.device)
        out = [K, torch.empty_like(K)]
    _by_bits(cache.bits, _lib.svdq_kv_read, _lib.svdq_kv4_read)(
        out[0], out[1], cache.dim, cu_rows, start, max_rows, block_table, cache.k_codes, cache.v_codes,
        cache.k_scales, cache.v_scales)
    return out[0], out[1]


def attention_workspace(rows, q_heads, kv_heads, dim, B, max_rows, max_kv, device="cuda", bits=8):
    """A workspace for attention() of these sizes over a cache of `bits` bits (None when none is
    needed)."""
    nb = _by_bits(bits, _lib.svdq_attn_kv8_workspace_bytes, _lib.svdq_attn_kv4_workspace_bytes)(
        rows, q_heads, kv_heads, dim, B, max_rows, max_kv)
    if nb < 0:
        raise ValueError("unsupported attention shape")
    return _bytes(nb, device) if nb else None


def attention(Q, cache, block_table, cu_rows, kv_len, max_rows, max_kv, scale=None, causal=False,
              out=None, workspace=None, return_lse=False):
    """softmax(scale·Q·Kᵀ)·V of Q [rows, q_heads·dim] bf16 over the cached tokens [0, kv_len[b]) of
    each sequence (causal: row i of n sees kv_len − n + i + 1 of them); scale defaults to
    dim^−1/2.  Returns O, or (O, lse) with lse fp32 [rows, q_heads]."""
    torch = _torch()
    dim, heads = cache.dim, cache.k_codes.shape[1]
    rows, q_heads = Q.shape[0], Q.shape[1] // dim
    O = out if out is not None else torch.empty(rows, q_heads * dim, dtype=torch.bfloat16,
                                                device=Q.device)
    lse = torch.empty(rows, q_heads, dtype=torch.float32, device=Q.device) if return_lse else None
    if workspace is None:
        workspace = attention_workspace(rows, q_heads, heads, dim, block_table.shape[0], max_rows,
                                        max_kv, Q.device, cache.bits)
    _by_bits(cache.bits, _lib.svdq_attn_kv8, _lib.svdq_attn_kv4)(
        Q, dim, cu_rows, kv_len, max_rows, max_kv, block_table, cache.k_codes, cache.v_codes,
        cache.k_scales, cache.v_scales, dim ** -0.5 if scale is None else scale, causal, O, lse,
        workspace)
    return (O, lse) if return_lse else O
