"""The single-token and 4-bit side of a packed [text | video | audio] transformer block: cases,
inputs, plain forms and 64-bit values of

  qk     root-mean-square norm of every query and key head of a packed row with the rotary
         positions in the same pass;
  cache  tokens appended to a paged 4-bit key / value cache and the touched pages read back;
  attn   softmax attention of ragged query rows over that cache;
  gemv   the quantised projection of a few rows with 16-bit activations: 4-bit weights with
         group scales, smoothing and the low-rank branch.

With `own` false the plain torch form runs, with `own` true the calls a user makes of
w4a4_quantized_dit_amd.layer.  Both read the same buffers, the cache's page layout included:
64 tokens a page; the tensors of nibbles and scales follow the index maps below (code_places,
scale_places), a block of 32 channels of a token is MXFP4: E2M1 elements under one power of two.
"""
import math

import torch

own = False

PAGE = 64
E_MIN, E_MAX = -110, 85           # exponents of a block's power-of-two scale
FMT = dict(nvfp4=0, int4=1, mxfp4=2)
GROUP = dict(nvfp4=16, int4=64, mxfp4=32)


# ------------------------------------------------------------------------------------------
# cases (5120 = 40 heads of 128, 13824 the width of the feed-forward projections; 31 x 24 x 42
# is the grid of the DeltaQuant workload)
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # query and key heads of one new token of each of 32 streams: latency counts
        dict(name="qk-token", op="qk", M=32, Hq=40, Hk=8, tail=8, D=128, axes="44,42,42",
             interleaved=True, far=True),
        # a text prompt: narrow heads, one axis, halves turned against each other
        dict(name="qk-prompt", op="qk", M=4001, Hq=32, Hk=8, tail=8, D=64, axes="64",
             interleaved=False, far=False),
        # query and key heads of the whole grid
        dict(name="qk-grid", op="qk", M=31688, Hq=40, Hk=40, tail=40, D=128, axes="44,42,42",
             interleaved=True, far=False),
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
        # a clip against itself
        dict(name="attn-clip", op="attn", B=1, q=16384, kv=16384, Hq=40, Hkv=40, D=128,
             causal=False, ragged=False),
        # the attention projection of a single conditioning token
        dict(name="gemv-token", op="gemv", fmt="nvfp4", M=1, K=5120, N=5120, r=32, smooth=True,
             pad=0),
        # the feed-forward up-projection of one token of each of 32 streams
        dict(name="gemv-streams", op="gemv", fmt="int4", M=32, K=5120, N=13824, r=32, smooth=True,
             pad=0),
        # the feed-forward down-projection of a handful of strided rows, the wide branch
        dict(name="gemv-rows", op="gemv", fmt="mxfp4", M=5, K=13824, N=5120, r=128, smooth=False,
             pad=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "cache", "attn", "gemv"])
    if op == "qk":
        D, axes = rng.choice([(128, "44,42,42"), (128, "16,56,56"), (64, "16,24,24"),
                              (128, "32,32"), (64, "64"), (256, "64,96,96"), (96, "96")])
        return dict(op=op, M=_log(rng, 1, 12000), Hq=rng.randint(1, 48), Hk=rng.randint(0, 40),
                    tail=rng.randint(0, 40), D=D, axes=axes, interleaved=rng.random() < 0.5,
                    far=rng.random() < 0.3)
    if op == "gemv":
        return dict(op=op, fmt=rng.choice(["nvfp4", "int4", "mxfp4"]), M=_log(rng, 1, 64),
                    K=256 * _log(rng, 1, 54), N=8 * _log(rng, 1, 1728),
                    r=rng.choice([0, 8, 32, 64, 128]), smooth=rng.random() < 0.7,
                    pad=rng.choice([0, 8, 256]))
    B = _log(rng, 1, 32)
    D = rng.choice([64, 128])
    if op == "cache":
        new = _log(rng, 1, max(1, 12000 // B))
        return dict(op=op, B=B, new=new, prior=rng.choice([0, rng.randint(1, 4000)]),
                    H=rng.choice([1, 5, 8, 24, 40]), D=D, ragged=rng.random() < 0.6)
    Hkv = rng.choice([1, 4, 8, 20, 40])
    G = rng.choice([1, 1, 2, 3, 5, 8]) if Hkv <= 20 else 1
    kv = _log(rng, 1, 30000)
    q = 1 if rng.random() < 0.4 else _log(rng, 1, 6000)
    causal = rng.random() < 0.5
    if not causal or rng.random() < 0.8:
        q = min(q, kv)       # a causal call of more rows than tokens leaves the first rows empty
    while B > 1 and B * (kv * Hkv * D + q * kv * Hkv * G) > 1 << 30:
        B = (B + 1) // 2
    while B * q * kv * Hkv * G > 1 << 31 and q > 1:
        q = (q + 1) // 2
    return dict(op=op, B=B, q=q, kv=kv, Hq=Hkv * G, Hkv=Hkv, D=D, causal=causal,
                ragged=rng.random() < 0.6)


# ------------------------------------------------------------------------------------------
# the cache's layout and number format (plain)
# ------------------------------------------------------------------------------------------

def code_places(D, is_v, dev):
    """Byte, within one page of one head, of the codes of channels (2j, 2j + 1) of token t (the
    even channel in the low nibble): [64, D / 2]."""
    t = torch.arange(PAGE, device=dev)[:, None]
    d = 2 * torch.arange(D // 2, device=dev)[None, :]
    if is_v:
        frag, lane = (d // 64) * 2 + t // 32, ((t // 4) % 2) * 32 + (d // 2) % 32
        byte = ((t // 16) % 2) * 8 + ((t // 8) % 2) * 4 + t % 4
    else:
        frag, lane = (t // 32) * (D // 64) + d // 64, ((d // 32) % 2) * 32 + t % 32
        byte = (d % 32) // 2
    return (frag * 64 + lane) * 16 + byte


def scale_places(D, is_v, dev):
    """Byte, within one page of one head, of the scale of token t's channels 32b on: [64, D / 32]."""
    t = torch.arange(PAGE, device=dev)[:, None]
    b = torch.arange(D // 32, device=dev)[None, :]
    if is_v:
        return (b * 2 + (t // 4) % 2) * 32 + (t // 16) * 8 + ((t // 8) % 2) * 4 + t % 4
    return ((b % 2) * 32 + t % 32) * (D // 32) + (t // 32) * (D // 64) + b // 2


def _two(e):
    """2^e exactly, in 64 bits (a power function may be off in its last bit)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e2m1_code(y):
    """Codes of the nearest E2M1 values, ties to the even code, at most 6."""
    a = y.abs()
    c = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
         + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
    return c | (torch.signbit(y).byte() << 3)


def _e2m1_value(c):
    """Values of E2M1 codes in 32 bits."""
    m = (c & 7).float()
    mag = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2.0, 2.0 * m - 8.0))
    return torch.where((c & 8) > 0, -mag, mag)


def _pair(lo, hi):
    return lo | (hi << 4)


def _nibbles(b):
    """The two codes of every byte of the last dimension, in order."""
    return torch.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], 2 * b.shape[-1])


def _quantise(x):
    """Bytes [..., D / 2] and scale bytes [..., D / 32] of tokens x [..., D]."""
    blk = x.float().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    a = blk.abs().amax(dim=-1)
    e = torch.where(a > 0, torch.frexp(a)[1] - 3, torch.full_like(a, E_MIN).int())
    e = e.clamp(E_MIN, E_MAX)
    c = _e2m1_code(blk * _two(-e).float()[..., None]).reshape(x.shape)
    return _pair(c[..., 0::2], c[..., 1::2]), (e + 127).to(torch.uint8)


def _values(b, s):
    """The values [..., D] in 32 bits of bytes [..., D / 2] and scale bytes [..., D / 32]."""
    v = _e2m1_value(_nibbles(b))
    blk = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    return (blk * _two(s.int() - 127).float()[..., None]).reshape(v.shape)


def _plain_append(codes, scales, X, page, slot, D, is_v):
    """Rows X [N, H·D] become the tokens `slot` of the pages `page`."""
    H = codes.shape[1]
    b, s = _quantise(X.reshape(-1, H, D))
    at = page[:, None, None]
    head = torch.arange(H, device=X.device)[None, :, None]
    codes[at, head, code_places(D, is_v, X.device)[slot][:, None, :]] = b
    scales[at, head, scale_places(D, is_v, X.device)[slot][:, None, :]] = s


def _plain_gather(codes, scales, table, D, is_v):
    """Values of all pages of the table: [B, H, blocks * 64, D] fp32."""
    B, nb = table.shape
    H, dev = codes.shape[1], codes.device
    pages = table.long().reshape(-1)
    b = codes[pages][:, :, code_places(D, is_v, dev).reshape(-1)].reshape(-1, H, PAGE, D // 2)
    s = scales[pages][:, :, scale_places(D, is_v, dev).reshape(-1)].reshape(-1, H, PAGE, D // 32)
    v = _values(b, s).reshape(B, nb, H, PAGE, D).transpose(1, 2)
    return v.reshape(B, H, nb * PAGE, D)


def _row_index(cu, start):
    """For packed rows: sequence, position in the cache and position in the call of every row."""
    n = (cu[1:] - cu[:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=cu.device), n)
    i = torch.arange(seq.numel(), device=cu.device) - cu[:-1].long()[seq]
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


def _cum(v, dev):
    t = torch.zeros(len(v) + 1, dtype=torch.int32)
    t[1:] = torch.cumsum(torch.tensor(v, dtype=torch.int64), 0).int()
    return t.to(dev)


def _fresh_cache(gd, B, blocks, H, D, dev):
    """A cache full of earlier tokens and a block table over shuffled pages."""
    n_pages = B * blocks + 3
    order = torch.randperm(n_pages, generator=gd, device=dev)[: B * blocks]
    table = order.reshape(B, blocks).int().contiguous()
    step = max(1, (1 << 26) // (H * PAGE * D))

    def fill(spread, is_v):
        codes = torch.empty(n_pages, H, PAGE * D // 2, dtype=torch.uint8, device=dev)
        scales = torch.empty(n_pages, H, PAGE * D // 32, dtype=torch.uint8, device=dev)
        at_c = code_places(D, is_v, dev).reshape(-1)
        at_s = scale_places(D, is_v, dev).reshape(-1)

        def some(p):
            m = min(step, n_pages - p)
            b, s = _quantise(torch.randn(m, H, PAGE, D, generator=gd, device=dev) * spread)
            codes[p:p + m, :, at_c] = b.reshape(m, H, -1)
            scales[p:p + m, :, at_s] = s.reshape(m, H, -1)

        [some(p) for p in range(0, n_pages, step)]
        return codes, scales

    (kc, ks), (vc, vs) = fill(1.0, False), fill(0.7, True)
    return dict(kc=kc, ks=ks, vc=vc, vs=vs), table


def _positions(case, g, gd, n_axes, dev):
    M = case["M"]
    if case["far"]:    # long streams: the time axis runs into the millions
        top = torch.tensor([4_000_000, 4096, 4096][:n_axes], device=dev)
        return (torch.rand(M, n_axes, generator=gd, device=dev, dtype=torch.float64) * top).int()
    # raster order of a 24 x 42 grid
    i = torch.arange(M, device=dev) + int(torch.randint(0, 4096, (1,), generator=g))
    cols = [i] if n_axes == 1 else [i // 1008, i // 42 % 24, i % 42][:n_axes]
    return torch.stack(cols, 1).int().contiguous()


def _weight(fmt, N, K, rnd, dev):
    """Codes [N, K / 2], scales and tensor scale of a random residual weight."""
    R = rnd(N, K) * K ** -0.5
    blk = R.reshape(N, K // GROUP[fmt], GROUP[fmt])
    a = blk.abs().amax(dim=2)
    g = None
    if fmt == "int4":
        scales = (a / 7.0).half()
        c = torch.round(blk / scales.float()[..., None]).clamp(-8, 7).to(torch.int8).view(torch.uint8)
        c = (c & 15).reshape(N, K)
    elif fmt == "nvfp4":
        g = (a.amax() / 2688.0).reshape(1)
        sv = (a / (6.0 * g)).to(torch.float8_e4m3fn)
        scales = sv.view(torch.uint8)
        unit = (sv.float() * g)[..., None]
        c = _e2m1_code(torch.where(unit > 0, blk / unit, torch.zeros_like(blk))).reshape(N, K)
    else:
        e = torch.where(a > 0, torch.frexp(a)[1] - 3, torch.full_like(a, -127).int())
        scales = (e + 127).to(torch.uint8)
        c = _e2m1_code(blk * _two(-e).float()[..., None]).reshape(N, K)
    return _pair(c[:, 0::2], c[:, 1::2]).contiguous(), scales, g


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gd, device=dev)  # noqa: E731
    bf = torch.bfloat16
    op = case["op"]
    s = dict(op=op, case=case)
    if op == "qk":
        M, H, D = case["M"], case["Hq"] + case["Hk"], case["D"]
        axes = [int(v) for v in case["axes"].split(",")]
        # heads of different sizes, as a projection leaves them
        size = torch.exp(0.5 * rnd(H + case["tail"]))[:, None].expand(-1, D).reshape(-1)
        s["X"] = torch.cat([(rnd(min(4096, M - a), (H + case["tail"]) * D) * size).to(bf)
                            for a in range(0, M, 4096)])[:, :H * D]
        s["pos"] = _positions(case, g, gd, len(axes), dev)
        s["freq"] = torch.cat([10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
                               for d in axes]).to(dev)
        s["axes"], s["eps"] = axes, 1e-6
        s["gq"], s["gk"] = [(1.0 + 0.2 * rnd(D)).to(bf) for _ in range(2)]
    elif op == "cache":
        B, H, D = case["B"], case["H"], case["D"]
        n = _lengths(B, case["new"], case["ragged"])
        prior = _lengths(B, case["prior"], case["ragged"]) if case["prior"] else [0] * B
        s.update(B=B, H=H, D=D, max_new=max(n))
        blocks = max((a + b + PAGE - 1) // PAGE for a, b in zip(prior, n))
        s["cache"], s["table"] = _fresh_cache(gd, B, blocks, H, D, dev)
        s["cu"], s["start"] = _cum(n, dev), torch.tensor(prior, dtype=torch.int32, device=dev)
        qkv = rnd(sum(n), 2 * H * D).to(bf)   # the k | v columns of a packed buffer
        s["K"], s["V"] = qkv[:, :H * D], qkv[:, H * D:]
        back = [a // PAGE * PAGE for a in prior]
        m = [a + b - c for a, b, c in zip(prior, n, back)]
        s["back"], s["cu_back"] = torch.tensor(back, dtype=torch.int32, device=dev), _cum(m, dev)
        s["rows_back"], s["max_back"] = sum(m), max(m)
    elif op == "attn":
        B, Hq, H, D = case["B"], case["Hq"], case["Hkv"], case["D"]
        q, kv = [_lengths(B, case[k], case["ragged"]) for k in ("q", "kv")]
        s.update(B=B, H=H, Hq=Hq, D=D, max_q=max(q), max_kv=max(kv))
        s["cache"], s["table"] = _fresh_cache(gd, B, (max(kv) + PAGE - 1) // PAGE, H, D, dev)
        s["cu"], s["len"] = _cum(q, dev), torch.tensor(kv, dtype=torch.int32, device=dev)
        s["Q"] = (1.5 * rnd(sum(q), Hq * D)).to(bf)
        s["scale"] = D ** -0.5
    else:
        M, N, K, r = case["M"], case["N"], case["K"], case["r"]
        # channels of different sizes, 2 % of them thirty times as large
        profile = torch.exp(0.75 * rnd(K))
        profile = torch.where(torch.rand(K, generator=gd, device=dev) < 0.02, 30 * profile, profile)
        s["X"] = torch.cat([rnd(M, K) * profile, rnd(M, case["pad"])], 1).to(bf)[:, :K]
        s["lam"] = profile.sqrt() if case["smooth"] else None
        s["down"] = (0.02 * rnd(r, K)).to(bf) if r else None
        s["up"] = (0.2 * rnd(N, r)).to(bf) if r else None
        s["codes"], s["scales"], s["g"] = _weight(case["fmt"], N, K, rnd, dev)
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from w4a4_quantized_dit_amd import layer as L
    op, case = s["op"], s["case"]
    if op == "qk":
        return L.qk_norm_rope(s["X"], s["pos"], s["freq"], s["axes"], s["case"]["D"], case["Hq"],
                              s["gq"], s["gk"], eps=s["eps"], interleaved=case["interleaved"])
    if op == "gemv":
        pw = L.PreparedWeight(FMT[case["fmt"]], case["N"], case["K"], case["r"], s["codes"],
                              s["scales"], s["g"], s["up"])
        return L.gemv(s["X"], pw, s["lam"], s["down"])
    c = s["cache"]
    kv = L.KVCache(c["kc"], c["vc"], c["ks"], c["vs"], s["D"], bits=4)
    if op == "cache":
        L.kv_write(kv, s["K"], s["V"], s["table"], s["cu"], s["start"], s["max_new"])
        return L.kv_read(kv, s["table"], s["cu_back"], s["back"], s["rows_back"], s["max_back"])
    O, lse = L.attention(s["Q"], kv, s["table"], s["cu"], s["len"], s["max_q"], s["max_kv"],
                         scale=s["scale"], causal=case["causal"], return_lse=True)
    return dict(O=O, lse=lse)


def _plain_qk(s):
    case, axes, freq = s["case"], s["axes"], s["freq"]
    M, D, Hq, Hk = case["M"], case["D"], case["Hq"], case["Hk"]
    rot, dev = 2 * freq.numel(), s["X"].device
    x = s["X"].reshape(M, Hq + Hk, D).float()
    inv = 1.0 / torch.sqrt((x * x).mean(dim=2, keepdim=True) + s["eps"])
    gamma = torch.cat([s["gq"].float().expand(Hq, D), s["gk"].float().expand(Hk, D)])
    x = x * inv * gamma
    axis = torch.repeat_interleave(torch.arange(len(axes), device=dev),
                                   torch.tensor(axes, device=dev) // 2)
    # far positions: the angle and its functions in 64 bits
    ang = s["pos"].double()[:, axis] * freq
    cos, sin = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]
    if case["interleaved"]:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).reshape(M, Hq + Hk, rot)
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
    return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16).reshape(M, (Hq + Hk) * D)


def _plain_cache(s):
    c, D = s["cache"], s["D"]
    seq, pos, _ = _row_index(s["cu"], s["start"])
    page, slot = s["table"][seq, pos // PAGE].long(), pos % PAGE
    _plain_append(c["kc"], c["ks"], s["K"], page, slot, D, False)
    _plain_append(c["vc"], c["vs"], s["V"], page, slot, D, True)
    seq, pos, _ = _row_index(s["cu_back"], s["back"])
    K = _plain_gather(c["kc"], c["ks"], s["table"], D, False)[seq, :, pos]
    V = _plain_gather(c["vc"], c["vs"], s["table"], D, True)[seq, :, pos]
    flat = (s["rows_back"], s["H"] * D)
    return [K.reshape(flat).to(torch.bfloat16), V.reshape(flat).to(torch.bfloat16)]


def _plain_attn(s):
    B, H, Hq, D = s["B"], s["H"], s["Hq"], s["D"]
    G, mq, c = Hq // H, s["max_q"], s["cache"]
    dev = s["Q"].device
    K = _plain_gather(c["kc"], c["ks"], s["table"], D, False)[:, :, :s["max_kv"]]
    V = _plain_gather(c["vc"], c["vs"], s["table"], D, True)[:, :, :s["max_kv"]]
    kv = s["len"].long()
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    seq, _, i = _row_index(s["cu"], torch.zeros_like(s["len"]))
    Q = torch.zeros(B, mq, Hq, D, device=dev)
    Q[seq, i] = s["Q"].float().reshape(-1, Hq, D)
    Q = Q.reshape(B, mq, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * mq, D)
    S = torch.matmul(Q, K.transpose(2, 3).contiguous()).mul_(s["scale"])
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
    O = torch.matmul(S, V.contiguous()) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l)).reshape(B, H, G, mq).permute(0, 3, 1, 2).reshape(B, mq, Hq)
    O = O.reshape(B, H, G, mq, D).permute(0, 3, 1, 2, 4).reshape(B, mq, Hq * D)
    return dict(O=O[seq, i].to(torch.bfloat16), lse=lse[seq, i])


def _plain_gemv(s):
    fmt, N, K = s["case"]["fmt"], s["case"]["N"], s["case"]["K"]
    x = s["X"].float()
    if s["lam"] is not None:    # the 16-bit activations of the layer
        x = (x * (1.0 / s["lam"])).to(torch.bfloat16).float()
    c = _nibbles(s["codes"])
    if fmt == "int4":
        w, scale = ((c ^ 8).float() - 8.0), s["scales"].float()
    elif fmt == "nvfp4":
        w, scale = _e2m1_value(c), s["scales"].view(torch.float8_e4m3fn).float() * s["g"]
    else:
        w, scale = _e2m1_value(c), _two(s["scales"].int() - 127).float()
    w = (w.reshape(N, K // GROUP[fmt], GROUP[fmt]) * scale[..., None]).reshape(N, K)
    y = x @ w.T
    if s["down"] is not None:
        y = y + (x @ s["down"].float().T) @ s["up"].float().T
    return y.to(torch.bfloat16)


def _run_plain(s):
    return dict(qk=_plain_qk, cache=_plain_cache, attn=_plain_attn, gemv=_plain_gemv)[s["op"]](s)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "qk":
        n = case["M"] * (case["Hq"] + case["Hk"]) * case["D"]
        return dict(bytes=4 * n + 4 * case["M"] * len(case["axes"].split(",")) + 4 * case["D"],
                    flops=7 * n)
    if op == "gemv":
        M, K, N, r, fmt = case["M"], case["K"], case["N"], case["r"], case["fmt"]
        scale = dict(nvfp4=1 / 16, int4=2 / 64, mxfp4=1 / 32)[fmt]
        return dict(bytes=int(N * K * (0.5 + scale)) + 2 * M * (K + N) + 2 * r * (K + N)
                    + (4 * K if case["smooth"] else 0), flops=2 * M * (N * K + r * (K + N)))
    B, D = case["B"], case["D"]
    if op == "cache":
        n = sum(_lengths(B, case["new"], case["ragged"])) * case["H"] * D
        return dict(bytes=int(2 * n * (2 + 2 * (0.5 + 1 / 32) + 2)), flops=4 * n)
    q, kv = [_lengths(B, case[k], case["ragged"]) for k in ("q", "kv")]
    # causal row i of n sees kv - n + i + 1 tokens, rows before the first token none
    pairs = sum(a * b - (a * (a - 1) // 2 if a <= b else a * b - b * (b + 1) // 2)
                if case["causal"] else a * b for a, b in zip(q, kv))
    return dict(bytes=sum(q) * case["Hq"] * (4 * D + 4)
                + int(2 * sum(kv) * case["Hkv"] * D * (0.5 + 1 / 32)),
                flops=4 * pairs * case["Hq"] * D)


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    dev, f64 = s["X" if "X" in s else "table"].device, torch.float64
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=f64, device=dev)
    grid = torch.cat([grid, -grid])

    def nearest(y):
        """Nearest E2M1 value of y, ties to the even code, at most 6."""
        a = y.abs().clamp(max=6.0)
        step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).to(f64)
        q = torch.round(a / step) * step
        return torch.where(y < 0, -q, q)

    def digits(D, is_v):
        """(byte, nibble, scale byte) of every code of a page, digit by digit."""
        out = []
        for t in range(PAGE):
            row = []
            for d in range(D):
                if is_v:
                    frag, half, lane = d >> 6 << 1 | t >> 5, t >> 2 & 1, d >> 1 & 31
                    byte = (t >> 4 & 1) << 3 | (t >> 3 & 1) << 2 | t & 3
                    scale = (d >> 5) << 6 | half << 5 | (t >> 4) << 3 | (t >> 3 & 1) << 2 | t & 3
                else:
                    frag, half, lane = (t >> 5) * (D >> 6) + (d >> 6), d >> 5 & 1, t & 31
                    byte, scale = d >> 1 & 15, (half << 5 | lane) * (D >> 5) + frag
                row.append([((frag << 1 | half) << 5 | lane) << 4 | byte, 4 * (d & 1), scale])
            out.append(row)
        return torch.tensor(out, device=dev).unbind(-1)

    def tokens(b, n, head, is_v, place):
        """The first n cached tokens of sequence b and a head, [n, D]."""
        codes, scales = (s["cache"][k] for k in (("vc", "vs") if is_v else ("kc", "ks")))
        byte, shift, at = place
        page = s["table"][b, :(n + PAGE - 1) // PAGE].long()
        nib = (codes[page, head][:, byte].long() >> shift) & 15
        unit = _two(scales[page, head][:, at].long() - 127)
        return (grid[nib] * unit).reshape(-1, s["D"])[:n]

    def of_qk():
        D, Hq, M = case["D"], case["Hq"], case["M"]
        x = s["X"].double().reshape(M, -1, D)
        x = x / torch.sqrt((x * x).sum(dim=2, keepdim=True) / D + s["eps"])
        x[:, :Hq] *= s["gq"].double()
        x[:, Hq:] *= s["gk"].double()
        y = x.clone()
        pair, half = 0, s["freq"].numel()
        for a, width in enumerate(s["axes"]):
            for _ in range(width // 2):
                i, j = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + half)
                turn = torch.polar(torch.ones(M, device=dev, dtype=f64),
                                   s["pos"][:, a].double() * float(s["freq"][pair]))
                z = torch.complex(x[:, :, i], x[:, :, j]) * turn[:, None]
                y[:, :, i], y[:, :, j] = z.real, z.imag
                pair += 1
        return y.reshape(M, -1)

    def of_cache():
        H, D = s["H"], s["D"]
        cu, start, res = s["cu"].tolist(), s["start"].tolist(), []
        for is_v, X in ((False, s["K"]), (True, s["V"])):
            place, parts = digits(D, is_v), []
            for b, at in enumerate(start):
                first = at // PAGE * PAGE
                if at > first:
                    old = torch.stack([tokens(b, at, h, is_v, place)[first:] for h in range(H)], 1)
                    parts.append(old.reshape(-1, H * D))
                x = X[cu[b]:cu[b + 1]].double().reshape(-1, 32)
                top = x.abs().amax(dim=1, keepdim=True)
                e = torch.floor(torch.log2(top))
                # a logarithm next to a whole number may fall on its wrong side
                e = torch.where(_two(e) > top, e - 1, e)
                e = torch.where(_two(e + 1) <= top, e + 1, e) - 2
                unit = _two(torch.where(top > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX))
                parts.append((nearest(x / unit) * unit).reshape(-1, H * D))
            res.append(torch.cat(parts))
        return res

    def of_attn():
        D, Hq, H = s["D"], s["Hq"], s["H"]
        G, N = Hq // H, s["Q"].shape[0]
        cu, lens = s["cu"].tolist(), s["len"].tolist()
        O = torch.zeros(N, Hq, D, dtype=f64, device=dev)
        lse = torch.full((N, Hq), float("-inf"), dtype=f64, device=dev)
        Q, places = s["Q"].reshape(N, Hq, D), [digits(D, False), digits(D, True)]
        for b, kv in enumerate(lens):
            n = cu[b + 1] - cu[b]
            for h in range(H):
                k, v = [tokens(b, kv, h, w, places[w]) for w in (False, True)]
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

    def of_gemv():
        fmt, N = case["fmt"], case["N"]
        x = s["X"].double()
        if s["lam"] is not None:   # by definition 16-bit activations: the product in 32 bits, then bf16
            x = (x * (1.0 / s["lam"].double()).float().double()).float().to(torch.bfloat16).double()
        nib = torch.empty(N, case["K"], dtype=torch.long, device=dev)
        nib[:, 0::2], nib[:, 1::2] = s["codes"].long() % 16, s["codes"].long() // 16
        if fmt == "int4":
            w, unit = torch.where(nib > 7, nib - 16, nib).double(), s["scales"].double()
        elif fmt == "nvfp4":
            w, unit = grid[nib], s["scales"].view(torch.float8_e4m3fn).double() * s["g"].double()
        else:
            w, unit = grid[nib], _two(s["scales"].long() - 127)
        y = x @ (w * torch.repeat_interleave(unit, GROUP[fmt], dim=1)).T
        if s["down"] is not None:
            y += x @ s["down"].double().T @ s["up"].double().T
        return y

    if case["op"] == "attn" and case["B"] * case["Hkv"] > 400:
        return None
    return dict(qk=of_qk, cache=of_cache, attn=of_attn, gemv=of_gemv)[case["op"]]()
