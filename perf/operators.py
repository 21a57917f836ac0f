"""The attention half of a packed [text | video | audio] transformer block around the quantised
projections: cases, inputs, plain forms and 64-bit values of

  norm   residual addition, root-mean-square norm, smoothing, MXFP8 codes and the low-rank
         down-projection, as the projection that follows reads them;
  rope   rotary positions over (time, height, width) of all query and key heads of a packed row;
  cache  tokens appended to a paged 8-bit key / value cache and the touched pages read back;
  attn   softmax attention of ragged query rows over that cache.

With `own` false the plain torch form runs, with `own` true the calls a user makes of
w4a4_quantized_dit_amd.layer.  Both read the same buffers, the cache's page layout included:
64 tokens a page; per page and head `kc` holds the codes of K in order
(token/32, d/32, (d/16)%2 ...) and `vc` those of V with the token order of a matrix operand; the
two index maps below (k_place, v_place) state them.
"""
import functools
import math

import torch

own = False

PAGE = 64
E_MIN, E_MAX = -110, 119          # exponents of a page's power-of-two scale


# ------------------------------------------------------------------------------------------
# cases (5120 = 40 heads of 128; 31 x 24 x 42 is the grid of the DeltaQuant workload)
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # one row through the norm: a single conditioning token, where latency counts
        dict(name="norm-row", op="norm", M=1, K=5120, r=0, residual=True, smooth=True, pad=0),
        # an attention projection's rows without the low-rank branch
        dict(name="norm-proj", op="norm", M=16384, K=5120, r=0, residual=True, smooth=True, pad=0),
        # the packed 31 x 24 x 42 grid with the rank-128 branch, rows strided
        dict(name="norm-grid-r128", op="norm", M=31688, K=5120, r=128, residual=True, smooth=True,
             pad=256),
        # query and key heads of a few rows of a packed q|k|v buffer
        dict(name="rope-few", op="rope", M=33, heads=48, tail=8, D=128, axes="44,42,42",
             interleaved=True, inverse=False, far=False),
        # query and key heads of the whole grid
        dict(name="rope-grid", op="rope", M=31688, heads=80, tail=40, D=128, axes="44,42,42",
             interleaved=True, inverse=False, far=True),
        # one token for each of 32 streams: appended in the middle of a page
        dict(name="cache-token", op="cache", B=32, new=1, prior=777, H=8, D=128, ragged=False),
        # one frame (24 x 42 tokens) of two streams behind a ragged history
        dict(name="cache-frame", op="cache", B=2, new=1008, prior=5041, H=40, D=128, ragged=True),
        # a whole clip at once
        dict(name="cache-clip", op="cache", B=1, new=16384, prior=0, H=40, D=128, ragged=False),
        # single tokens of 32 ragged streams over shared heads
        dict(name="attn-token", op="attn", B=32, q=1, kv=8191, Hq=40, Hkv=8, D=128, causal=True,
             ragged=True),
        # a causal prompt of two ragged streams, narrow heads
        dict(name="attn-causal", op="attn", B=2, q=4001, kv=4001, Hq=32, Hkv=8, D=64, causal=True,
             ragged=True),
        # one frame against the cached grid
        dict(name="attn-frame", op="attn", B=1, q=1008, kv=31688, Hq=40, Hkv=40, D=128,
             causal=False, ragged=False),
        # a clip against itself
        dict(name="attn-clip", op="attn", B=1, q=16384, kv=16384, Hq=40, Hkv=40, D=128,
             causal=False, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rope", "cache", "attn"])
    if op == "norm":
        r = rng.choice([0, 8, 32, 64, 128])
        return dict(op=op, M=_log(rng, 1, 24000), K=256 * rng.randint(1, 28), r=r,
                    residual=rng.random() < 0.7, smooth=rng.random() < 0.7,
                    pad=rng.choice([0, 8, 256]))
    if op == "rope":
        D, axes = rng.choice([(128, "44,42,42"), (128, "16,56,56"), (64, "16,24,24"),
                              (128, "32,32"), (64, "64"), (256, "64,96,96")])
        return dict(op=op, M=_log(rng, 1, 12000), heads=rng.randint(1, 96),
                    tail=rng.randint(0, 40), D=D, axes=axes, interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.3, far=rng.random() < 0.3)
    B = _log(rng, 1, 32)
    D = rng.choice([64, 128])
    if op == "cache":
        new = _log(rng, 1, max(1, 12000 // B))
        return dict(op=op, B=B, new=new, prior=rng.choice([0, rng.randint(1, 4000)]),
                    H=rng.choice([1, 5, 8, 24, 40]), D=D, ragged=rng.random() < 0.6)
    Hkv = rng.choice([1, 4, 8, 20, 40])
    G = rng.choice([1, 1, 2, 3, 5, 8]) if Hkv <= 20 else 1
    kv = _log(rng, 1, 30000)
    q = 1 if rng.random() < 0.4 else _log(rng, 1, min(kv, 6000))
    while B > 1 and B * (kv * Hkv * D + q * kv * Hkv * G) > 1 << 30:
        B = (B + 1) // 2
    while B * q * kv * Hkv * G > 1 << 31 and q > 1:
        q = (q + 1) // 2
    return dict(op=op, B=B, q=q, kv=kv, Hq=Hkv * G, Hkv=Hkv, D=D, causal=rng.random() < 0.5,
                ragged=rng.random() < 0.6)


# ------------------------------------------------------------------------------------------
# the cache's layout and number format (plain)
# ------------------------------------------------------------------------------------------

def k_place(D, dev):
    """Byte offset of K's code (token, d) within one page of one head: [64, D]."""
    t = torch.arange(PAGE, device=dev)[:, None]
    d = torch.arange(D, device=dev)[None, :]
    frag = ((t // 32) * (D // 64) + d // 64) * 2 + (d // 16) % 2
    return (frag * 64 + ((d // 32) % 2) * 32 + t % 32) * 16 + d % 16


def v_place(D, dev):
    """Byte offset of V's code (token, d) within one page of one head: [64, D]."""
    t = torch.arange(PAGE, device=dev)[:, None]
    d = torch.arange(D, device=dev)[None, :]
    frag = (d // 32) * 2 + t // 32
    byte = 8 * ((t // 16) % 2) + 4 * ((t // 8) % 2) + t % 4
    return (frag * 64 + ((t // 4) % 2) * 32 + d % 32) * 16 + byte


def _two(e):
    """2^e exactly, in 64 bits (a power function may be off in its last bit)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e, within [E_MIN, E_MAX]."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _codes(x, e):
    """E4M3 codes (uint8) of x / 2^e."""
    y = (x.float() * _two(-e).float()).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes, e):
    return codes.view(torch.float8_e4m3fn).float() * _two(e).float()


def _write_pages(codes, scales, pages, valid, new, is_new, is_old, place, D):
    """Pages [P] of the cache get the values new [P, H, 64, D] at the slots is_new [P, 64];
    slots is_old are rounded again where the scale grows; the others keep their bytes."""
    H = codes.shape[1]
    at = place.reshape(-1)
    raw = codes[pages][:, :, at].reshape(-1, H, PAGE, D)
    e_old = scales[pages].int() - 127
    nm = is_new[:, None, :, None]
    om = is_old[:, None, :, None]
    e_new = _exponent(torch.where(nm, new, torch.zeros_like(new)).abs().amax(dim=(2, 3)).float())
    keep = is_old.any(dim=1)[:, None]
    e = torch.where(keep, torch.maximum(e_old, e_new), e_new)
    ee, eo = e[:, :, None, None], e_old[:, :, None, None]
    old = torch.where(om, raw, torch.zeros_like(raw))
    out = torch.where(nm, _codes(new, ee), torch.where(om, _codes(_values(old, eo), ee), raw))
    packed = torch.empty(out.shape[0], H, PAGE * D, dtype=torch.uint8, device=out.device)
    packed[:, :, at] = out.reshape(-1, H, PAGE * D)
    codes[pages[valid]] = packed[valid]
    scales[pages[valid]] = (e + 127).to(torch.uint8)[valid]


def _plain_write(s, K, V):
    c, B, D, H = s["cache"], s["B"], s["D"], s["H"]
    dev = K.device
    T = (s["max_new"] + PAGE - 1) // PAGE + 1
    start, n = s["start"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    j = (start // PAGE)[:, None] + torch.arange(T, device=dev)[None, :]           # [B, T]
    pos = j[:, :, None] * PAGE + torch.arange(PAGE, device=dev)                   # [B, T, 64]
    is_new = (pos >= start[:, None, None]) & (pos < (start + n)[:, None, None])
    is_old = (pos < start[:, None, None]) & is_new.any(dim=2, keepdim=True)
    row = (s["cu"][:-1].long()[:, None, None] + pos - start[:, None, None]).clamp(0, K.shape[0] - 1)
    pages = torch.gather(s["table"].long(), 1, j.clamp(max=s["table"].shape[1] - 1)).reshape(-1)
    valid = is_new.any(dim=2).reshape(-1)
    for_rows = row.reshape(-1, PAGE)
    new, old = is_new.reshape(-1, PAGE), is_old.reshape(-1, PAGE)
    for X, codes, scales, place in ((K, c["kc"], c["ks"], k_place(D, dev)),
                                    (V, c["vc"], c["vs"], v_place(D, dev))):
        tile = X[for_rows].reshape(-1, PAGE, H, D).transpose(1, 2)
        _write_pages(codes, scales, pages, valid, tile, new, old, place, D)


def _plain_gather(c, table, H, D):
    """Values of all pages of the table: K, V [B, H, blocks * 64, D] fp32."""
    B, nb = table.shape
    dev = table.device
    out = []
    for codes, scales, place in ((c["kc"], c["ks"], k_place(D, dev)),
                                 (c["vc"], c["vs"], v_place(D, dev))):
        raw = codes[table.long().reshape(-1)][:, :, place.reshape(-1)].reshape(-1, H, PAGE, D)
        e = scales[table.long().reshape(-1)].int()[:, :, None, None] - 127
        v = _values(raw, e).reshape(B, nb, H, PAGE, D).transpose(1, 2)
        out.append(v.reshape(B, H, nb * PAGE, D))
    return out


def _row_index(cu, start, max_n, dev):
    """For packed rows: sequence and position of every row."""
    n = (cu[1:] - cu[:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=dev), n)
    i = torch.arange(seq.numel(), device=dev) - cu[:-1].long()[seq]
    return seq, i + start.long()[seq], i


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _lengths(B, most, ragged):
    """Host lengths of B sequences, the first the longest; ragged ones down to a quarter."""
    if not ragged:
        return [most] * B
    return [most if b == 0 else max(1, int(most * (0.25 + 0.75 * (0.618034 * b % 1.0))))
            for b in range(B)]


def _attn_lengths(case):
    """Query rows and cached tokens of every sequence (the rows' own tokens are in the cache)."""
    q = _lengths(case["B"], case["q"], case["ragged"])
    kv = _lengths(case["B"], case["kv"], case["ragged"])
    return q, [max(a, b) for a, b in zip(q, kv)]


def _cum(v, dev):
    t = torch.zeros(len(v) + 1, dtype=torch.int32)
    t[1:] = torch.cumsum(torch.tensor(v, dtype=torch.int64), 0).int()
    return t.to(dev)


def _fresh_cache(gd, B, blocks, H, D, dev):
    """A cache full of earlier tokens and a block table over shuffled pages."""
    n_pages = B * blocks + 3
    order = torch.randperm(n_pages, generator=gd, device=dev)[: B * blocks]
    table = order.reshape(B, blocks).int().contiguous()
    c = {}
    for codes, scales, spread in (("kc", "ks", 1.0), ("vc", "vs", 0.7)):
        c[codes] = torch.empty(n_pages, H, PAGE * D, dtype=torch.uint8, device=dev)
        c[scales] = torch.empty(n_pages, H, dtype=torch.uint8, device=dev)
        at = (k_place if codes == "kc" else v_place)(D, dev).reshape(-1)
        step = max(1, (1 << 26) // (H * PAGE * D))
        for p in range(0, n_pages, step):
            m = min(step, n_pages - p)
            x = torch.randn(m, H, PAGE, D, generator=gd, device=dev) * spread
            e = _exponent(x.abs().amax(dim=(2, 3)))
            q = _codes(x, e[:, :, None, None]).reshape(m, H, PAGE * D)
            c[codes][p:p + m, :, at] = q
            c[scales][p:p + m] = (e + 127).to(torch.uint8)
    return c, table


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gd, device=dev)  # noqa: E731
    bf = torch.bfloat16
    op = case["op"]
    s = dict(op=op, case=case)
    if op == "norm":
        M, K, r = case["M"], case["K"], case["r"]
        profile = torch.exp(0.75 * rnd(K))
        s["X"] = (rnd(M, K + case["pad"]).mul_(0.3)).to(bf)[:, :K]
        s["res"] = None
        if case["residual"]:
            s["res"] = torch.empty(M, K, dtype=bf, device=dev)
            for a in range(0, M, 4096):
                s["res"][a:a + 4096] = rnd(min(4096, M - a), K) * profile
        s["gamma"] = (1.0 + 0.2 * rnd(K)).to(bf)
        s["lam"] = torch.exp(0.5 * rnd(K)) if case["smooth"] else None
        s["down"] = (0.02 * rnd(r, K)).to(bf) if r else None
        s["eps"] = 1e-6
    elif op == "rope":
        M, H, D = case["M"], case["heads"], case["D"]
        axes = [int(v) for v in case["axes"].split(",")]
        s["X"] = rnd(M, (H + case["tail"]) * D).to(bf)[:, :H * D]
        if case["far"]:    # long streams: the time axis runs into the millions
            top = torch.tensor([4_000_000, 4096, 4096][:len(axes)], device=dev)
            pos = (torch.rand(M, len(axes), generator=gd, device=dev, dtype=torch.float64) * top).int()
        else:              # raster order of a 24 x 42 grid
            i = torch.arange(M, device=dev) + int(torch.randint(0, 4096, (1,), generator=g))
            pos = torch.stack([i // 1008, i // 42 % 24, i % 42], 1)[:, :len(axes)].int()
        s["pos"] = pos.contiguous()
        s["freq"] = torch.cat([10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
                               for d in axes]).to(dev)
        s["axes"] = axes
    elif op == "cache":
        B, H, D = case["B"], case["H"], case["D"]
        n = _lengths(B, case["new"], case["ragged"])
        prior = _lengths(B, case["prior"], case["ragged"]) if case["prior"] else [0] * B
        s.update(B=B, H=H, D=D, max_new=max(n))
        blocks = max((a + b + PAGE - 1) // PAGE for a, b in zip(prior, n))
        s["cache"], s["table"] = _fresh_cache(gd, B, blocks, H, D, dev)
        s["cu"], s["start"] = _cum(n, dev), torch.tensor(prior, dtype=torch.int32, device=dev)
        N = sum(n)
        qkv = rnd(N, 2 * H * D).to(bf)   # the k | v columns of a packed buffer
        s["K"], s["V"] = qkv[:, :H * D], qkv[:, H * D:]
        back = [a // PAGE * PAGE for a in prior]
        m = [a + b - c for a, b, c in zip(prior, n, back)]
        s["back"], s["cu_back"] = torch.tensor(back, dtype=torch.int32, device=dev), _cum(m, dev)
        s["rows_back"], s["max_back"] = sum(m), max(m)
    else:
        B, Hq, H, D = case["B"], case["Hq"], case["Hkv"], case["D"]
        q, kv = _attn_lengths(case)
        s.update(B=B, H=H, Hq=Hq, D=D, max_q=max(q), max_kv=max(kv))
        blocks = (max(kv) + PAGE - 1) // PAGE
        s["cache"], s["table"] = _fresh_cache(gd, B, blocks, H, D, dev)
        s["cu"], s["len"] = _cum(q, dev), torch.tensor(kv, dtype=torch.int32, device=dev)
        s["Q"] = (1.5 * rnd(sum(q), Hq * D)).to(bf)
        s["scale"] = D ** -0.5
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _norm_out(s, codes, scales, D, H):
    """The element values (E4M3), their scales' exponent bytes, D and the new residual."""
    out = dict(q=codes.view(torch.float8_e4m3fn), e=scales)
    if D is not None:
        out["D"] = D
    if s["res"] is not None:
        out["H"] = H
    return out


def _run_own(s):
    from w4a4_quantized_dit_amd import layer as L
    op = s["op"]
    if op == "norm":
        return _norm_out(s, *L.norm_quantize_activation(s["X"], s["gamma"], s["lam"], s["down"],
                                                        eps=s["eps"], residual=s["res"]))
    if op == "rope":
        c = s["case"]
        return L.rope(s["X"], s["pos"], s["freq"], s["axes"], c["D"],
                      interleaved=c["interleaved"], inverse=c["inverse"])
    c = s["cache"]
    kv = L.KVCache(c["kc"], c["vc"], c["ks"], c["vs"], s["D"])
    if op == "cache":
        L.kv_write(kv, s["K"], s["V"], s["table"], s["cu"], s["start"], s["max_new"])
        return L.kv_read(kv, s["table"], s["cu_back"], s["back"], s["rows_back"], s["max_back"])
    O, lse = L.attention(s["Q"], kv, s["table"], s["cu"], s["len"], s["max_q"], s["max_kv"],
                         scale=s["scale"], causal=s["case"]["causal"], return_lse=True)
    return dict(O=O, lse=lse)


def _plain_norm(s):
    X, res = s["X"], s["res"]
    H = (X.float() + res.float()).to(torch.bfloat16) if res is not None else X
    K = X.shape[1]
    # the codes sit next to rounding borders: the sum in 64 bits, the products one by one in 32
    mean = H.double().square().sum(dim=1, keepdim=True) / K
    inv = (1.0 / torch.sqrt(mean + s["eps"])).float()
    x = H.float() * inv * s["gamma"].float()
    if s["lam"] is not None:
        x = x * (1.0 / s["lam"])
    blk = x.reshape(x.shape[0], K // 32, 32)
    a = blk.abs().amax(dim=2)
    e = torch.where(a > 0, torch.frexp(a)[1] - 9, torch.full_like(a, -127).int()).clamp(-127, 127)
    y = (blk.double() * _two(-e)[:, :, None]).float().clamp(-448.0, 448.0)
    codes = y.to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape)
    D = x.to(torch.bfloat16).float() @ s["down"].float().T if s["down"] is not None else None
    return codes, (e + 127).to(torch.uint8), D, H


def _plain_rope(X, pos, freq, axes, D, interleaved, inverse):
    M = X.shape[0]
    H, rot = X.shape[1] // D, 2 * freq.numel()
    axis = torch.repeat_interleave(torch.arange(len(axes), device=X.device),
                                   torch.tensor(axes, device=X.device) // 2)
    # far positions: the angle and its functions in 64 bits
    ang = pos.double()[:, axis] * freq
    cos, sin = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]
    sin = -sin if inverse else sin
    x = X.reshape(M, H, D).float()
    if interleaved:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).reshape(M, H, rot)
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
    return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16).reshape(M, H * D)


def _plain_attn(s):
    B, H, Hq, D = s["B"], s["H"], s["Hq"], s["D"]
    G, mq = Hq // H, s["max_q"]
    dev = s["Q"].device
    K, V = _plain_gather(s["cache"], s["table"], H, D)
    K, V = K[:, :, :s["max_kv"]], V[:, :, :s["max_kv"]]
    kv = s["len"].long()
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq, _, i = _row_index(s["cu"], torch.zeros_like(s["len"]), mq, dev)
    Q = torch.zeros(B, mq, Hq, D, device=dev)
    Q[seq, i] = s["Q"].float().reshape(-1, Hq, D)
    Q = Q.reshape(B, mq, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * mq, D)
    S = torch.matmul(Q, K.transpose(2, 3)).mul_(s["scale"])
    t = torch.arange(s["max_kv"], device=dev)
    last = kv[:, None].expand(B, mq)
    if s["case"]["causal"]:
        last = torch.minimum(last, (kv - n)[:, None] + torch.arange(mq, device=dev)[None, :] + 1)
    dead = (t[None, None, :] >= last[:, :, None])[:, None].repeat(1, 1, G, 1)
    S.masked_fill_(dead, float("-inf"))
    del dead
    m = S.amax(dim=3, keepdim=True)
    S.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    l = S.sum(dim=3, keepdim=True)
    O = torch.matmul(S, V) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l)).reshape(B, H, G, mq).permute(0, 3, 1, 2).reshape(B, mq, Hq)
    O = O.reshape(B, H, G, mq, D).permute(0, 3, 1, 2, 4).reshape(B, mq, Hq * D)
    return dict(O=O[seq, i].to(torch.bfloat16), lse=lse[seq, i])


def _run_plain(s):
    op = s["op"]
    if op == "norm":
        return _norm_out(s, *_plain_norm(s))
    if op == "rope":
        c = s["case"]
        return _plain_rope(s["X"], s["pos"], s["freq"], s["axes"], c["D"], c["interleaved"],
                           c["inverse"])
    if op == "cache":
        _plain_write(s, s["K"], s["V"])
        K, V = _plain_gather(s["cache"], s["table"], s["H"], s["D"])
        seq, pos, _ = _row_index(s["cu_back"], s["back"], s["max_back"], K.device)
        flat = (s["rows_back"], s["H"] * s["D"])
        return [T[seq, :, pos].reshape(flat).to(torch.bfloat16) for T in (K, V)]
    return _plain_attn(s)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        M, K, r = case["M"], case["K"], case["r"]
        b = 2 * M * K * (3 if case["residual"] else 1) + M * K + M * K // 32 + 4 * M * r
        return dict(bytes=b + 2 * K + 4 * K + 2 * r * K, flops=2 * M * K * r + 10 * M * K)
    if op == "rope":
        n = case["M"] * case["heads"] * case["D"]
        return dict(bytes=4 * n + 12 * case["M"], flops=3 * n)
    B, D = case["B"], case["D"]
    if op == "cache":
        n = sum(_lengths(B, case["new"], case["ragged"])) * case["H"] * D
        return dict(bytes=2 * n * (2 + 1 + 1 + 2), flops=4 * n)
    q, kv = _attn_lengths(case)
    pairs = sum(a * b - (a * (a - 1) // 2 if case["causal"] else 0) for a, b in zip(q, kv))
    return dict(bytes=sum(q) * case["Hq"] * (4 * D + 4) + 2 * sum(kv) * case["Hkv"] * D,
                flops=4 * pairs * case["Hq"] * D)


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------

def _e4m3_64(y):
    """Nearest E4M3 value of y in 64 bits, ties to even, at most 448."""
    a = y.abs().clamp(max=448.0)
    _, x = torch.frexp(a)
    quantum = _two((x - 1).clamp(min=-6) - 3)
    q = torch.round(a / quantum) * quantum
    return torch.where(y < 0, -q, q)


@functools.lru_cache(None)
def _places_64(D, is_v):
    """The byte of each code of a page, digit by digit."""
    def one(token, d):
        if is_v:
            half, lane, frag = token >> 2 & 1, d & 31, (d >> 5) * 2 + (token >> 5)
            byte = (token >> 4 & 1) << 3 | (token >> 3 & 1) << 2 | token & 3
        else:
            half, lane, byte = d >> 5 & 1, token & 31, d & 15
            frag = ((token >> 5) * (D >> 6) + (d >> 6)) * 2 + (d >> 4 & 1)
        return (((frag << 1 | half) << 5) | lane) << 4 | byte
    return [[one(t, d) for d in range(D)] for t in range(PAGE)]


def _tokens_64(s, b, n, head, which):
    """The first n cached tokens of sequence b and a head, [n, D] in 64 bits."""
    c, D = s["cache"], s["D"]
    codes, scales = (c["vc"], c["vs"]) if which else (c["kc"], c["ks"])
    blocks = (n + PAGE - 1) // PAGE
    page = s["table"][b, :blocks].long()
    at = torch.tensor(_places_64(D, which), device=codes.device)
    raw = codes[page, head][:, at].view(torch.float8_e4m3fn).double()
    scale = _two(scales[page, head].int() - 127)
    return (raw * scale[:, None, None]).reshape(blocks * PAGE, D)[:n]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "norm":
        return _exact_norm(s)
    if op == "rope":
        return _exact_rope(s, case)
    if op == "cache":
        return _exact_cache(s)
    if case["B"] * case["Hkv"] > 400:
        return None
    return _exact_attn(s, case)


def _exact_norm(s):
    X, K = s["X"], s["X"].shape[1]
    out = dict(e=None)
    h = X.double()
    if s["res"] is not None:
        h = (h + s["res"].double()).to(torch.bfloat16)
        out["H"] = h.clone()
        h = h.double()
    # by definition the reciprocal norm and each product are rounded to 32 bits
    inv = torch.rsqrt((h * h).mean(dim=1) + s["eps"]).float().double()
    x = (h * inv[:, None]).float().double()
    x = (x * s["gamma"].double()).float().double()
    if s["lam"] is not None:
        x = (x * (1.0 / s["lam"].double()).float().double()).float().double()
    blk = x.reshape(x.shape[0], K // 32, 32)
    a = blk.abs().amax(dim=2, keepdim=True)
    e = (torch.frexp(a)[1] - 9).clamp(min=-127)
    unit = _two(torch.where(a > 0, e, torch.full_like(e, -127)))
    out["q"] = _e4m3_64(blk / unit).reshape(x.shape)
    if s["down"] is not None:
        out["D"] = x.to(torch.bfloat16).double() @ s["down"].double().T
    return out


def _exact_rope(s, case):
    D, axes = case["D"], s["axes"]
    M = s["X"].shape[0]
    x = s["X"].double().reshape(M, -1, D)
    y = x.clone()
    pair, half = 0, s["freq"].numel()
    for a, width in enumerate(axes):
        for _ in range(width // 2):
            i, j = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + half)
            turn = torch.polar(torch.ones(M, device=x.device, dtype=torch.float64),
                               s["pos"][:, a].double() * float(s["freq"][pair]))
            if case["inverse"]:
                turn = turn.conj()
            z = torch.complex(x[:, :, i], x[:, :, j]) * turn[:, None]
            y[:, :, i], y[:, :, j] = z.real, z.imag
            pair += 1
    return y.reshape(M, -1)


def _exact_cache(s):
    B, H, D = s["B"], s["H"], s["D"]
    cu, start = s["cu"].tolist(), s["start"].tolist()
    res = []
    for which, X in ((0, s["K"]), (1, s["V"])):
        scales = s["cache"]["vs" if which else "ks"]
        parts = []
        for b in range(B):
            n, first = cu[b + 1] - cu[b], start[b] // PAGE * PAGE
            new = X[cu[b]:cu[b + 1]].double().reshape(n, H, D)
            done, at = [], start[b]
            while at < start[b] + n:
                page0 = at // PAGE * PAGE
                upto = min(page0 + PAGE, start[b] + n)
                v = new[at - start[b]:upto - start[b]]                       # [m, H, D]
                top = v.abs().amax(dim=(0, 2))
                e = torch.ceil(torch.log2(top / 448.0)).clamp(E_MIN, E_MAX).int()
                # a logarithm next to a whole number may fall on its wrong side
                e = torch.where(top > 448.0 * _two(e), e + 1, e)
                e = torch.where(top <= 448.0 * _two(e - 1), e - 1, e).clamp(E_MIN, E_MAX)
                if at > page0:
                    e = torch.maximum(e, scales[s["table"][b, page0 // PAGE].long()].int() - 127)
                    old = torch.stack([_tokens_64(s, b, at, h, which)[page0:at] for h in range(H)], 1)
                    v = torch.cat([old, v])
                unit = _two(e)[None, :, None]
                done.append(_e4m3_64(v / unit) * unit)
                at = upto
            parts.append(torch.cat(done).reshape(-1, H * D))
        res.append(torch.cat(parts))
    return res


def _exact_attn(s, case):
    D, Hq, H = s["D"], s["Hq"], s["H"]
    G, N = Hq // H, s["Q"].shape[0]
    cu, lens = s["cu"].tolist(), s["len"].tolist()
    dev = s["Q"].device
    O = torch.zeros(N, Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((N, Hq), float("-inf"), dtype=torch.float64, device=dev)
    Q = s["Q"].reshape(N, Hq, D)
    for b, kv in enumerate(lens):
        n = cu[b + 1] - cu[b]
        for h in range(H):
            k, v = _tokens_64(s, b, kv, h, 0), _tokens_64(s, b, kv, h, 1)
            for g in range(G):
                for a in range(0, n, 4096):
                    m = min(4096, n - a)
                    rows = slice(cu[b] + a, cu[b] + a + m)
                    z = (Q[rows, h * G + g].double() @ k.T) * s["scale"]
                    if case["causal"]:
                        see = kv - n + a + torch.arange(m, device=dev)[:, None]
                        z = z.masked_fill(torch.arange(kv, device=dev)[None] > see, float("-inf"))
                    lse[rows, h * G + g] = torch.logsumexp(z, 1)
                    O[rows, h * G + g] = torch.softmax(z, 1).nan_to_num(0.0) @ v
    return dict(O=O.reshape(N, Hq * D), lse=lse)
