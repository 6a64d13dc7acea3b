"""Cases that time the transformer-block operators: RMS norm (forward with the residual's addition and an 8-bit output,
and its gradient), rotary positions, the append to a 4-bit paged cache, and the attention that reads that cache.

``own`` false: elementary torch operations in 32 bits (64 where 32 lose: angles, codes next to a rounding border).
``own`` true: the calls of ``masking_tm_affine_gb300.tm``.  ``exact`` gives the same outputs from the definitions in
64 bits, written apart from the plain form.

The cache is a pool of pages of ``page`` tokens (a multiple of 16).  A page holds, for each KV head, page/16 blocks of
16 tokens, and a block of head size D is 16*(D+8) bytes:

    K codes   16 tokens x D/2 bytes, a token's D nibbles in order (low nibble first)
    V codes   8 token pairs x 8 slices x 2 tokens x D/16 bytes: slice r of a token is its dims [r*D/8, (r+1)*D/8)
    K scales  16 x (step, low) in 16-bit floats
    V scales  16 x (step, low)

and a code c stands for low + c*step.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a small batch: the latency of a norm whose output feeds an 8-bit product
        {"name": "norm_decode_e4m3", "op": "norm", "M": 32, "N": 4096, "type": "bf16", "residual": True, "out": "e4m3",
         "group": 0},
        # a long prompt through the same norm, a scale for each 128 columns
        {"name": "norm_prompt_e4m3", "op": "norm", "M": 8192, "N": 8192, "type": "bf16", "residual": True,
         "out": "e4m3", "group": 128},
        # a training step's norm, forward and gradient, with the residual stream's own gradient joining
        {"name": "norm_train", "op": "norm_train", "M": 8192, "N": 4096, "type": "bf16", "residual": True},
        # the same in fp32 on ragged extents
        {"name": "norm_train_ragged", "op": "norm_train", "M": 4100, "N": 1000, "type": "f32", "residual": False},
        # queries and keys of a training batch (32 + 8 heads rotated in one call)
        {"name": "rope_train", "op": "rope", "T": 8192, "H": 40, "D": 128, "rot": 128, "inter": False,
         "inverse": False, "type": "bf16", "base": 500000.0, "far": 8192},
        # the gradient of an interleaved rotation of part of the head, far positions, an odd count of tokens
        {"name": "rope_grad_partial", "op": "rope", "T": 1001, "H": 9, "D": 96, "rot": 48, "inter": True,
         "inverse": True, "type": "f32", "base": 10000.0, "far": 1000000},
        # one new token for each of 64 sequences: rotate q and k, write k and v to the cache, read them back
        {"name": "append_step", "op": "append", "T": 64, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "inter": False,
         "type": "bf16", "page": 16, "far": 131072, "run": 1},
        # a prompt of 8192 tokens written to the cache and read back in 16 bits, as the next chunk's dense pass does
        {"name": "append_prompt", "op": "append", "T": 8192, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "inter": False,
         "type": "bf16", "page": 64, "far": 8192, "run": 2731},
        # one short sequence in fp32, as many KV heads as query heads: the latency of a single call
        {"name": "attn_short_f32", "op": "attn", "B": 1, "q": 1, "max": 1000, "min": 1000, "Hq": 8, "Hkv": 8,
         "D": 64, "page": 16, "type": "f32", "window": 0, "idle": False},
        # a decode step of 64 sequences of ragged lengths
        {"name": "attn_decode", "op": "attn", "B": 64, "q": 1, "max": 8192, "min": 1000, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "type": "bf16", "window": 0, "idle": False},
        # one sequence with a very long context: the work has to be split over the cache
        {"name": "attn_long", "op": "attn", "B": 1, "q": 1, "max": 131071, "min": 131071, "Hq": 64, "Hkv": 8,
         "D": 128, "page": 16, "type": "f16", "window": 0, "idle": False},
        # the next chunk of two prompts over what the cache holds already
        {"name": "attn_chunk", "op": "attn", "B": 2, "q": 256, "max": 8192, "min": 4100, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "type": "bf16", "window": 0, "idle": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm_train", "rope", "append", "attn", "attn"])
    typ = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind in ("norm", "norm_train"):
        N = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            N = max(64, N // 64 * 64)
        M = min(_log(rng, 1, 16384), (1 << 25) // N)
        c = {"op": kind, "M": M, "N": N, "type": typ, "residual": rng.random() < 0.7}
        if kind == "norm":
            c["out"] = rng.choice(["e4m3", "e4m3", "same"])
            c["group"] = rng.choice([0, 0, 64, 128]) if c["out"] == "e4m3" else 0
        return c
    if kind == "rope":
        D = rng.choice([64, 80, 96, 128, 256])
        H = rng.randint(1, 48)
        T = min(_log(rng, 1, 16384), (1 << 25) // (H * D))
        rot = D if rng.random() < 0.5 else rng.choice([D // 2, D // 4])
        return {"op": "rope", "T": T, "H": H, "D": D, "rot": rot, "inter": rng.random() < 0.5,
                "inverse": rng.random() < 0.5, "type": typ, "base": rng.choice([10000.0, 500000.0]),
                "far": _log(rng, 1000, 1000000)}
    if kind == "append":
        D, Hkv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
        T = min(_log(rng, 1, 8192), (1 << 23) // (Hkv * D))
        return {"op": "append", "T": T, "Hq": Hkv * rng.choice([1, 3, 4, 8]), "Hkv": Hkv, "D": D,
                "rot": D if rng.random() < 0.7 else D // 2, "inter": rng.random() < 0.3, "type": typ,
                "page": rng.choice([16, 32, 64, 128]), "far": _log(rng, 8192, 1000000), "run": _log(rng, 1, T)}
    D, Hkv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
    q = 1 if rng.random() < 0.6 else _log(rng, 2, 256)
    B = _log(rng, 1, 64) if q < 16 else rng.randint(1, 2)
    longest = _log(rng, 16, 8192 if B > 4 else 65536 if q == 1 else 8192)
    longest = max(longest, q)
    group = rng.choice([1, 3, 4, 8])
    return {"op": "attn", "B": B, "q": q, "max": longest, "min": rng.randint(max(1, longest // 8), longest),
            "Hq": Hkv * min(group, 32 // Hkv), "Hkv": Hkv, "D": D, "page": rng.choice([16, 32, 64, 128]), "type": typ,
            "window": rng.choice([0, 0, 0, 1000]), "idle": B > 1 and rng.random() < 0.3}


def _lengths(c):
    """Cache lengths and query counts of the sequences of an attention case: spread evenly between min and max."""
    B, lo, hi = c["B"], c["min"], c["max"]
    lens = [hi - i * (hi - lo) // max(1, B - 1) for i in range(B)]
    qs = [min(n, c["q"] if i % 2 == 0 else max(1, c["q"] - c["q"] // 3)) for i, n in enumerate(lens)]
    if c["idle"]:
        lens[-1] = 0  # a slot of the batch that is empty for now: its query is answered with zeros
    return lens, qs


def _size(t):
    return {"f32": 4, "f16": 2, "bf16": 2}[t]


def work(c):
    e = _size(c["type"])
    if c["op"] == "norm":
        MN = c["M"] * c["N"]
        out = 1 if c["out"] == "e4m3" else e
        per = e + out + (2 * e if c["residual"] else 0)
        scales = 4 * c["M"] * (-(-c["N"] // c["group"]) if c["group"] else 1) if c["out"] == "e4m3" else 0
        return {"bytes": MN * per + e * c["N"] + scales, "flops": 5 * MN}
    if c["op"] == "norm_train":
        MN = c["M"] * c["N"]
        fwd = (4 if c["residual"] else 2) * e
        bwd = (4 if c["residual"] else 3) * e  # h, dy (and the stream's gradient) read, dx written
        return {"bytes": MN * (fwd + bwd) + 3 * e * c["N"] + 8 * c["M"], "flops": 15 * MN}
    if c["op"] == "rope":
        n = c["T"] * c["H"] * c["D"]
        return {"bytes": 2 * e * n + 8 * c["T"] + 4 * c["rot"], "flops": 3 * n}
    if c["op"] == "append":
        q, kv = c["T"] * c["Hq"] * c["D"], c["T"] * c["Hkv"] * c["D"]
        cache = c["T"] * c["Hkv"] * (c["D"] + 8)
        return {"bytes": 2 * e * q + 2 * e * kv + cache + cache + 2 * e * kv + 24 * c["T"], "flops": 3 * q + 12 * kv}
    lens, qs = _lengths(c)
    seen = pairs = 0
    for n, q in zip(lens, qs):
        if not n:
            continue
        w = c["window"] or n + q
        seen += min(n, w + q - 1)
        pairs += sum(min(n - q + t + 1, w) for t in range(q))
    rows = sum(qs) * c["Hq"]
    return {"bytes": seen * c["Hkv"] * (c["D"] + 8) + rows * (2 * c["D"] * e + 4) + 4 * seen // c["page"],
            "flops": 4 * pairs * c["Hq"] * c["D"]}


# ------------------------------------------------------------------------------------------------ inputs
def _inv_freq(c):
    """Angular frequencies of the rotation, radians a position, in 64 bits."""
    i = torch.arange(0, c["rot"], 2, dtype=torch.float64)
    return torch.exp(-i / c["rot"] * math.log(c.get("base", 10000.0)))


def _turns(inv_freq):
    """The same as turns a position in units of 2^-64, the form the kernels take."""
    t = [int(round(f / (2.0 * math.pi) * 2.0 ** 64)) for f in inv_freq.tolist()]
    return torch.from_numpy(np.array(t, dtype=np.uint64).view(np.int64))


def _quantise(x):
    """Codes (uint8, one each) and (step, low) of the vectors along the last dimension, from values in 64 bits."""
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    step = ((high - low) / 15).float().half()
    low = low.float().half()
    d = step.double()
    c = torch.where(d > 0, (x.double() - low.double()) / torch.where(d > 0, d, 1.0), 0.0).round().clamp(0, 15)
    return c.to(torch.uint8), torch.cat([step, low], -1)


def _vectors(tokens, channels, gen, dev, keys):
    """Vectors [*tokens, D] as they come in a cache: about normal, with some wide and some shifted channels among keys
    (``channels``: the shape over which those differ, D last)."""
    x = torch.randn(tokens, generator=gen, device=dev)
    if keys:
        wide = 1.0 + 2.0 * (torch.rand(channels, generator=gen, device=dev) < 0.03)
        x = x * wide + 0.5 * torch.randn(channels, generator=gen, device=dev)
    return x


def _pool(pages, Hkv, page, D, gen, dev):
    """A filled cache: every slot of every page, in the layout of this file's head."""
    n = pages * Hkv * page // 16
    out = torch.empty((n, 16 * (D + 8)), dtype=torch.uint8, device=dev)
    for i in range(0, n, 1 << 15):
        m = min(n, i + (1 << 15)) - i
        kc, kp = _quantise(_vectors((m, 16, D), (m, 1, D), gen, dev, True))
        vc, vp = _quantise(_vectors((m, 16, D), None, gen, dev, False))
        kb = (kc[..., 0::2] | (kc[..., 1::2] << 4)).view(m, 8 * D)
        vb = (vc[..., 0::2] | (vc[..., 1::2] << 4)).view(m, 8, 2, 8, D // 16).transpose(2, 3).reshape(m, 8 * D)
        out[i:i + m] = torch.cat([kb, vb, kp.reshape(m, -1).view(torch.uint8), vp.reshape(m, -1).view(torch.uint8)], 1)
    return out.view(pages, Hkv, page // 16, 16 * (D + 8))


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    t = TYPES[c["type"]]
    s = {"case": c}

    def randn(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * scale).to(t)

    def empty(*shape, dtype=t):
        return torch.empty(shape, dtype=dtype, device=dev)

    if c["op"] in ("norm", "norm_train"):
        M, N = c["M"], c["N"]
        s["x"] = randn(M, N)
        s["r"] = randn(M, N, scale=3.0) if c["residual"] else None
        s["w"] = (1.0 + 0.2 * torch.randn(N, generator=gen, device=dev)).to(t)
        s["h"] = empty(M, N) if c["residual"] else None
        if c["op"] == "norm":
            e4 = c["out"] == "e4m3"
            s["y"] = empty(M, N, dtype=torch.float8_e4m3fn if e4 else t)
            s["scale"] = empty(M, -(-N // c["group"]) if c["group"] else 1, dtype=torch.float32) if e4 else None
        else:
            s["y"], s["dx"], s["dw"] = empty(M, N), empty(M, N), empty(N)
            s["rstd"] = empty(M, dtype=torch.float32)
            s["dy"] = randn(M, N, scale=0.1)
            s["dr"] = randn(M, N, scale=0.1) if c["residual"] else None
            s["scratch"] = empty(8 << 20, dtype=torch.float32)
        return s
    if c["op"] == "rope":
        s["x"] = randn(c["T"], c["H"], c["D"])
        s["y"] = empty(c["T"], c["H"], c["D"])
        s["pos"] = torch.randint(0, c["far"], (c["T"],), generator=gen, device=dev)
        s["inv_freq"] = _inv_freq(c).to(dev)
        s["turns"] = _turns(_inv_freq(c)).to(dev)
        return s
    if c["op"] == "append":
        T, Hq, Hkv, D, page = c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
        s["qkv"] = torch.cat([randn(T, Hq, D), _vectors((T, Hkv, D), (Hkv, D), gen, dev, True).to(t), randn(T, Hkv, D)], 1)
        s["inv_freq"] = _inv_freq(c).to(dev)
        s["turns"] = _turns(_inv_freq(c)).to(dev)
        runs = -(-T // c["run"])  # sequences of `run` new tokens each, at a place of their own in pages of their own
        per = -(-(c["run"] + page - 1) // page)
        perm = torch.randperm(runs * per, generator=gen, device=dev).view(runs, per)
        first = torch.randint(0, page, (runs,), generator=gen, device=dev)
        begin = torch.randint(0, max(1, c["far"] - c["run"]), (runs,), generator=gen, device=dev)
        i = torch.arange(T, device=dev)
        seq, at = i // c["run"], first[i // c["run"]] + i % c["run"]
        s["slots"] = perm[seq, at // page] * page + at % page
        s["pos"] = begin[seq] + i % c["run"]
        s["pool"] = torch.zeros((runs * per, Hkv, page // 16, 16 * (D + 8)), dtype=torch.uint8, device=dev)
        s["q"], s["k"], s["v"] = empty(T, Hq, D), empty(T, Hkv, D), empty(T, Hkv, D)
        return s
    lens, qs = _lengths(c)
    B, page, Hkv, D = c["B"], c["page"], c["Hkv"], c["D"]
    per = -(-c["max"] // page)
    s["pool"] = _pool(B * per, Hkv, page, D, gen, dev)
    s["table"] = torch.randperm(B * per, generator=gen, device=dev).view(B, per).int()
    order = torch.randperm(B, generator=gen, device=dev).tolist() if c["q"] == 1 else list(range(B))
    lens, qs = [lens[i] for i in order], [qs[i] for i in order]
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["qstart"] = torch.tensor([0] + list(np.cumsum(qs)), dtype=torch.int32, device=dev)
    s["total"], s["max_q"] = sum(qs), max(qs)
    s["q"] = randn(s["total"], c["Hq"], D)
    s["o"] = empty(s["total"], c["Hq"], D)
    s["lse"] = empty(s["total"], c["Hq"], dtype=torch.float32)
    s["scratch"] = empty(64 << 20, dtype=torch.float32)
    return s


# ------------------------------------------------------------------------------------------------ plain form
def _plain_norm(s):
    c = s["case"]
    t = TYPES[c["type"]]
    h = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    y = h * rstd * s["w"].float()
    out = {} if s["r"] is None else {"h": h.to(t)}
    if c.get("out") != "e4m3":
        return {**out, "y": y.to(t)}, h, rstd
    M, N = y.shape
    g = c["group"] or N
    pad = torch.nn.functional.pad(y, (0, -N % g)).view(M, -1, g)
    amax = pad.abs().amax(2, keepdim=True)
    inv = torch.where(amax > 0, 448.0 / amax, 1.0)
    out["scale"] = torch.where(amax > 0, amax / 448.0, 1.0).view(M, -1)
    out["y"] = (pad * inv).view(M, -1)[:, :N].to(torch.float8_e4m3fn)
    return out, h, rstd


def _plain_norm_train(s):
    t = TYPES[s["case"]["type"]]
    out, h, rstd = _plain_norm(s)
    # the gradient is taken at what the forward pass stored
    h = h if s["r"] is None else out["h"].float()
    dy, w = s["dy"].float(), s["w"].float()
    xhat = h * rstd
    g = dy * w
    dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dr"] is not None:
        dx = dx + s["dr"].float()
    return {**out, "rstd": rstd.view(-1), "dx": dx.to(t), "dw": (dy * xhat).sum(0).to(t)}


def _rotate(x, pos, inv_freq, rot, inter, sign):
    """x [T, H, D] in 64 bits, rotated by pos * inv_freq (sign -1: back)."""
    angle = pos.double()[:, None] * inv_freq[None, :]
    cos, sin = torch.cos(angle)[:, None, :], sign * torch.sin(angle)[:, None, :]
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        ab = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        ab = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([ab, x[..., rot:]], -1)


def _plain_rope(s):
    c = s["case"]
    y = _rotate(s["x"].double(), s["pos"], s["inv_freq"], c["rot"], c["inter"], -1.0 if c["inverse"] else 1.0)
    return {"y": y.to(s["x"].dtype)}


def _plain_append(s):
    c = s["case"]
    T, Hq, Hkv, D, page = c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    t = TYPES[c["type"]]
    qk = _rotate(s["qkv"][:, :Hq + Hkv].double(), s["pos"], s["inv_freq"], c["rot"], c["inter"], 1.0)
    kc, kp = _quantise(qk[:, Hq:])
    vc, vp = _quantise(s["qkv"][:, Hq + Hkv:].double())
    at, pool = s["slots"], s["pool"]
    page_i, block, row = at // page, at % page // 16, at % 16
    k, v, kps, vps = _views(pool, D)
    k[page_i, :, block, row] = kc[..., 0::2] | (kc[..., 1::2] << 4)
    v[page_i, :, block, row // 2, :, row % 2] = (vc[..., 0::2] | (vc[..., 1::2] << 4)).view(T, Hkv, 8, D // 16)
    kps[page_i, :, block, row] = kp.view(torch.uint8)
    vps[page_i, :, block, row] = vp.view(torch.uint8)
    # read back
    kk = _values(k[page_i, :, block, row], kps[page_i, :, block, row])
    vv = _values(v[page_i, :, block, row // 2, :, row % 2].reshape(T, Hkv, D // 2), vps[page_i, :, block, row])
    return {"q": qk[:, :Hq].to(t), "k": kk.to(t), "v": vv.to(t)}


def _views(pool, D):
    """K codes, V codes and the two sets of scales of a pool, as strided views."""
    P, H, S, _ = pool.shape
    k = pool[..., :8 * D].view(P, H, S, 16, D // 2)
    v = pool[..., 8 * D:16 * D].view(P, H, S, 8, 8, 2, D // 16)
    kp = pool[..., 16 * D:16 * D + 64].view(P, H, S, 16, 4)
    vp = pool[..., 16 * D + 64:].view(P, H, S, 16, 4)
    return k, v, kp, vp


def _values(codes, params):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    p = params.contiguous().view(torch.float16).float()
    return c * p[..., :1] + p[..., 1:]


def _plain_attn(s):
    c = s["case"]
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    G, dev = c["Hq"] // Hkv, s["q"].device
    k, v, kp, vp = _views(s["pool"][s["table"].long()].flatten(0, 1), D)
    flat = (B, -1, Hkv, D)
    kk = _values(k, kp).transpose(1, 2).transpose(2, 3).reshape(flat)
    vv = _values(v.transpose(-2, -3).flatten(-4, -2).unflatten(-1, (-1,)).reshape(*v.shape[:3], 16, D // 2),
                 vp).transpose(1, 2).transpose(2, 3).reshape(flat)
    L, Q = kk.shape[1], s["max_q"]
    qn = s["qstart"][1:] - s["qstart"][:-1]
    t = torch.arange(Q, device=dev)
    rows = (s["qstart"][:-1, None] + t).clamp(max=s["total"] - 1).long()
    q = s["q"][rows].float().view(B, Q, Hkv, G, D)
    score = torch.einsum("bthgd,blhd->bhgtl", q, kk) * (D ** -0.5)
    at = (s["lens"] - qn)[:, None] + t
    j = torch.arange(L, device=dev)
    seen = (j <= at[..., None]) & (j < s["lens"][:, None, None])
    if c["window"]:
        seen = seen & (j > at[..., None] - c["window"])
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgtl,blhd->bthgd", p / torch.where(total > 0, total, 1.0), vv)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2)
    live = t < qn[:, None]
    return {"o": o.reshape(B, Q, -1, D)[live].to(s["q"].dtype), "lse": lse.reshape(B, Q, -1)[live]}


# ------------------------------------------------------------------------------------------------ the framework's
def _own(s):
    from masking_tm_affine_gb300 import tm
    c = s["case"]
    code = {"f32": tm.TM_F32, "f16": tm.TM_F16, "bf16": tm.TM_BF16}[c["type"]]
    if c["op"] in ("norm", "norm_train"):
        M, N = c["M"], c["N"]
        e4 = c.get("out") == "e4m3"
        tm.tm_rmsnorm(s["x"], N, s["r"], N, s["h"], N, s["w"], M, N, EPS, s["y"], N, s.get("scale"), s.get("rstd"),
                      code, code, tm.TM_E4M3 if e4 else code, c.get("group", 0))
        out = {"y": s["y"]}
        if s["r"] is not None:
            out["h"] = s["h"]
        if e4:
            out["scale"] = s["scale"]
        if c["op"] == "norm":
            return out
        h = s["x"] if s["r"] is None else s["h"]
        tm.tm_rmsnorm_bwd(s["dy"], N, h, N, s["w"], s["rstd"], s["dr"], N, s["dx"], N, s["dw"], M, N, code, code,
                          s["scratch"], s["scratch"].numel() * 4)
        return {**out, "rstd": s["rstd"], "dx": s["dx"], "dw": s["dw"]}
    if c["op"] == "rope":
        H, D = c["H"], c["D"]
        flags = (tm.TM_ROPE_INTERLEAVED if c["inter"] else 0) | (tm.TM_ROPE_INVERSE if c["inverse"] else 0)
        tm.tm_rope(s["x"], H * D, D, s["y"], H * D, D, s["pos"], s["turns"], c["T"], H, D, c["rot"], 1.0, code, flags)
        return {"y": s["y"]}
    if c["op"] == "append":
        T, Hq, Hkv, D, page = c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
        x, row = s["qkv"], (Hq + 2 * Hkv) * D
        flags = tm.TM_ROPE_INTERLEAVED if c["inter"] else 0
        tm.tm_kv4_append(x, row, D, s["q"], Hq * D, D, Hq, x[:, Hq:], row, D, x[:, Hq + Hkv:], row, D, s["pos"],
                         s["turns"], s["slots"], s["pool"], s["pool"].shape[0], page, T, Hkv, D, c["rot"], 1.0, code,
                         flags)
        tm.tm_kv4_gather(s["pool"], s["pool"].shape[0], page, s["slots"], s["k"], Hkv * D, D, s["v"], Hkv * D, D, T,
                         Hkv, D, code)
        return {"q": s["q"], "k": s["k"], "v": s["v"]}
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    tm.tm_kv4_attention(s["q"], Hq * D, D, s["o"], Hq * D, D, s["lse"], s["pool"], s["pool"].shape[0], c["page"],
                        s["table"], s["table"].shape[1], s["lens"], s["qstart"], c["B"], s["total"], s["max_q"],
                        c["max"], Hq, Hkv, D, D ** -0.5, c["window"], code, s["scratch"], s["scratch"].numel() * 4)
    return {"o": s["o"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)[0]
    return {"norm_train": _plain_norm_train, "rope": _plain_rope, "append": _plain_append, "attn": _plain_attn}[op](state)


# ------------------------------------------------------------------------------------------------ 64 bits
def _np(x):
    return x.detach().to(torch.float64).cpu().numpy()


def _exact_norm(s):
    c = s["case"]
    h = _np(s["x"])
    out = {}
    if s["r"] is not None:
        h = h + _np(s["r"])
        out["h"] = h
    w = _np(s["w"])[None]
    ms = np.einsum("ij,ij->i", h, h)[:, None] / h.shape[1] + EPS
    y = h / np.sqrt(ms) * w
    if c["op"] == "norm_train":
        stored = h if s["r"] is None else _np(torch.from_numpy(h).to(TYPES[c["type"]]))
        dy = _np(s["dy"])
        n = stored / np.sqrt(ms)
        along = np.einsum("ij,ij->i", dy * w, n)[:, None] / h.shape[1]
        dx = (dy * w - n * along) / np.sqrt(ms)
        if s["dr"] is not None:
            dx = dx + _np(s["dr"])
        return {**out, "y": y, "rstd": 1 / np.sqrt(ms[:, 0]), "dx": dx, "dw": np.einsum("ij,ij->j", dy, n)}
    if c["out"] != "e4m3":
        return {**out, "y": y}
    M, N = y.shape
    g = c["group"] or N
    edges = np.arange(0, N, g)
    top = np.maximum.reduceat(np.abs(y), edges, axis=1)
    scale = np.where(top > 0, top / 448, 1.0)
    z = y / np.repeat(scale, np.diff(np.append(edges, N)), axis=1)
    # e4m3: 3 bits after the leading one down to exponent -6, steps of 2^-9 below
    ulp = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(z), 1e-30))), -6) - 3)
    return {**out, "y": np.rint(z / ulp) * ulp, "scale": scale}


def _exact_turn(x, pos, c, sign):
    """Rotation as a product of complex numbers, angles reduced in whole turns' fractions with extended precision."""
    half = c["rot"] // 2
    f = np.exp(-2.0 * np.arange(half, dtype=np.longdouble) / c["rot"] * np.log(np.longdouble(c.get("base", 10000.0))))
    z = np.exp(1j * sign * np.fmod(pos[:, None].astype(np.longdouble) * f, 2 * np.longdouble(np.pi)).astype(np.float64))
    y = x.copy()
    if c["inter"]:
        w = (x[..., 0:c["rot"]:2] + 1j * x[..., 1:c["rot"]:2]) * z[:, None]
        y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2] = w.real, w.imag
    else:
        w = (x[..., :half] + 1j * x[..., half:c["rot"]]) * z[:, None]
        y[..., :half], y[..., half:c["rot"]] = w.real, w.imag
    return y


def _exact_held(x):
    """What a vector's 4-bit form stands for."""
    low, high = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    step = ((high - low) / 15).astype(np.float32).astype(np.float16).astype(np.float64)
    low = low.astype(np.float32).astype(np.float16).astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(step > 0, np.clip(np.rint((x - low) / step), 0, 15), 0)
    return low + c * step


def _exact_attn(s):
    """Sequence by sequence, the cache decoded block by block through its bytes."""
    c = s["case"]
    D, G = c["D"], c["Hq"] // c["Hkv"]
    table, lens, start = s["table"].cpu().tolist(), s["lens"].cpu().tolist(), s["qstart"].cpu().tolist()
    blocks = c["page"] // 16
    o = torch.zeros((s["total"], c["Hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.full((s["total"], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        n, q0, q1 = lens[b], start[b], start[b + 1]
        if n == 0:
            continue
        pages = torch.tensor(table[b][:-(-n // c["page"])], device="cuda")
        raw = s["pool"].index_select(0, pages).permute(1, 0, 2, 3).reshape(c["Hkv"], -1, 16 * (D + 8))
        held = raw[..., 16 * D:].contiguous().view(torch.float16).double().view(c["Hkv"], -1, 2, 16, 2)
        tok = torch.arange(raw.shape[1] * 16, device="cuda")[:n]
        blk, r = tok // 16, tok % 16
        d = torch.arange(D, device="cuda")
        k_at = r[:, None] * (D // 2) + d // 2
        v_at = 8 * D + (r // 2)[:, None] * D + (d // (D // 8)) * (D // 8) + (r % 2)[:, None] * (D // 16) \
            + d % (D // 8) // 2
        assert blocks * len(pages) == raw.shape[1]
        for hd in range(c["Hkv"]):
            kb, vb = raw[hd][blk[:, None], k_at].int(), raw[hd][blk[:, None], v_at].int()
            shift = (d % 2 * 4).int()
            kk = (kb >> shift & 15).double() * held[hd, blk, 0, r, :1] + held[hd, blk, 0, r, 1:]
            vv = (vb >> shift & 15).double() * held[hd, blk, 1, r, :1] + held[hd, blk, 1, r, 1:]
            heads = slice(hd * G, (hd + 1) * G)
            sc = s["q"][q0:q1, heads].double() @ kk.T / math.sqrt(D)
            where = (n - (q1 - q0) + torch.arange(q1 - q0, device="cuda"))[:, None, None]
            hidden = tok > where
            if c["window"]:
                hidden |= tok <= where - c["window"]
            sc = sc.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(sc, -1, keepdim=True)
            dead = z == -math.inf
            o[q0:q1, heads] = torch.exp(sc - z.masked_fill(dead, 0.0)) @ vv
            lse[q0:q1, heads] = z[..., 0]
    return {"o": o, "lse": lse}


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] in ("norm", "norm_train"):
        return _exact_norm(s)
    if c["op"] == "rope":
        return {"y": _exact_turn(_np(s["x"]), s["pos"].cpu().numpy(), c, -1.0 if c["inverse"] else 1.0)}
    if c["op"] == "append":
        x, Hq, Hkv = _np(s["qkv"]), c["Hq"], c["Hkv"]
        qk = _exact_turn(x[:, :Hq + Hkv], s["pos"].cpu().numpy(), c, 1.0)
        return {"q": qk[:, :Hq], "k": _exact_held(qk[:, Hq:]), "v": _exact_held(x[:, Hq + Hkv:])}
    return _exact_attn(s)
