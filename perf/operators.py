"""Timed cases of the quantised serving operators: MXFP4 quantisation and product, rotary positions, the
8-bit key/value cache and the attention that reads it.

`run` computes each operator in its plain form (elementary torch operations in 32 bits), or, with `own`
true, through the framework's calls; `exact` gives the values of the operators' definitions in 64 bits.
Sizes are those of Llama-2-7B and -70B decoder blocks (hidden 4096 / 8192, MLP 11008 / 28672, heads of
128) and of smaller, odd ones between.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the activations of one decode step of 16 sequences, quantised before a product
        {"name": "quant 16x4096 bf16", "op": "quant", "rows": 16, "cols": 4096, "dtype": "bf16"},
        # a master weight (the 7B gate projection, fp32) laid out for deployment, with its values
        {"name": "quant 11008x4096 fp32", "op": "quant", "rows": 11008, "cols": 4096, "dtype": "fp32"},
        # the 7B gate projection of one decoded token, activations quantised in the call
        {"name": "linear 1x4096x11008", "op": "linear", "m": 1, "k": 4096, "n": 11008, "dtype": "bf16"},
        # the 7B down projection of a short ragged prompt
        {"name": "linear 77x11008x4096", "op": "linear", "m": 77, "k": 11008, "n": 4096, "dtype": "fp16"},
        # the 70B gate projection of a 4096-token prompt, activations already in codes
        {"name": "gemm 4096x8192x28672", "op": "gemm", "m": 4096, "k": 8192, "n": 28672, "dtype": "bf16"},
        # one decode step of 16 sequences, 7B heads, far positions
        {"name": "rope 16 tokens", "op": "rope", "t": 16, "hq": 32, "hk": 32, "d": 128, "rot": 128, "half": True,
         "far": 131072, "dtype": "bf16"},
        # a 4096-token prompt with 70B heads, three quarters of each head rotated as interleaved pairs
        {"name": "rope 4096 tokens", "op": "rope", "t": 4096, "hq": 64, "hk": 8, "d": 128, "rot": 96, "half": False,
         "far": 32768, "dtype": "fp16"},
        # one decode step of 64 sequences of different lengths into pages of 64 tokens
        {"name": "append 64x1", "op": "append", "b": 64, "nq": 1, "kv": 1021, "hk": 8, "d": 128, "page": 64,
         "dtype": "bf16"},
        # two prompts of about 2048 tokens
        {"name": "append 2x2048", "op": "append", "b": 2, "nq": 2048, "kv": 2048, "hk": 32, "d": 128, "page": 64,
         "dtype": "fp16"},
        # one decoded token of one short conversation: latency
        {"name": "attn 1x1 over 257", "op": "attn", "b": 1, "nq": 1, "kv": 257, "hq": 32, "hk": 32, "d": 128,
         "page": 16, "dtype": "bf16"},
        # one decode step of 32 long conversations, grouped heads
        {"name": "attn 32x1 over 16381", "op": "attn", "b": 32, "nq": 1, "kv": 16381, "hq": 64, "hk": 8, "d": 128,
         "page": 64, "dtype": "bf16"},
        # two prompts of about 2048 tokens attending to themselves
        {"name": "attn 2x2048", "op": "attn", "b": 2, "nq": 2048, "kv": 2048, "hq": 32, "hk": 32, "d": 128,
         "page": 64, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "gemm", "rope", "append", "attn"])
    dt = rng.choice(["bf16", "fp16"])
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": 32 * _log(rng, 1, 170),
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op in ("linear", "gemm"):
        return {"op": op, "m": _log(rng, 1, 4096), "k": 32 * _log(rng, 2, 350), "n": _log(rng, 16, 12000), "dtype": dt}
    d = rng.choice([64, 128])
    hk = rng.choice([1, 2, 4, 8, 16, 32])
    hq = hk * rng.choice([1, 2, 4, 7, 8])
    if op == "rope":
        return {"op": op, "t": _log(rng, 1, 4096), "hq": min(hq, 64), "hk": hk, "d": d,
                "rot": rng.choice([d, d // 2, 3 * d // 4]), "half": rng.random() < 0.5, "far": _log(rng, 4096, 1 << 20),
                "dtype": dt}
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        nq = rng.choice([1, 1, _log(rng, 2, 2048)])
        return {"op": op, "b": _log(rng, 1, max(1, min(128, 4096 // nq))), "nq": nq, "kv": nq + _log(rng, 1, 2048),
                "hk": hk, "d": d, "page": page, "dtype": dt}
    hq, hk = min(hq, 64), min(hk, 8) if hq > 64 else hk
    hq -= hq % hk
    nq = rng.choice([1, 1, _log(rng, 2, 1024)])
    kv = nq + _log(rng, 1, 8192 if nq == 1 else 1024)
    b = _log(rng, 1, max(1, min(64, (1 << 20) // (kv * max(1, hk // 4)), 4096 // nq)))
    return {"op": op, "b": b, "nq": nq, "kv": kv, "hq": hq, "hk": hk, "d": d, "page": page, "dtype": dt}


def _lens(case):
    """Per sequence (new tokens, cached length with them): ragged, the longest as the case says; from the case alone."""
    b, nq, kv = case["b"], case["nq"], case["kv"]
    new = [max(1, nq - (i * 7919) % max(1, nq // 4 + 1)) for i in range(b)]
    if nq == kv:
        return [(n, n) for n in new]
    old = [max(0, kv - nq - (i * 104729) % max(1, 3 * (kv - nq) // 4 + 1)) for i in range(b)]
    return [(n, n + o) for n, o in zip(new, old)]


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "quant":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * e + 0.5 + 1 / 32), "flops": 2 * n}
    if op in ("linear", "gemm"):
        m, n, k = case["m"], case["n"], case["k"]
        x = m * k * (2 if op == "linear" else 17 / 32)
        return {"bytes": x + n * k * 17 / 32 + 2 * m * n, "flops": 2 * m * n * k}
    if op == "rope":
        n = case["t"] * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": 2 * n * e + 4 * case["t"] + 2 * case["rot"], "flops": 3 * n}
    lens = _lens(case)
    row = case["hk"] * case["d"]
    if op == "append":
        t = sum(n for n, _ in lens)
        blocks = sum((l - 1) // case["page"] - (l - n) // case["page"] + 1 for n, l in lens)
        return {"bytes": 2 * t * row * (e + 1) + 8 * blocks * case["hk"], "flops": 4 * t * row}
    t = sum(n for n, _ in lens)
    pairs = sum(n * l - n * (n - 1) // 2 for n, l in lens)
    keys = sum(l for _, l in lens)
    return {"bytes": 2 * keys * row + 2 * t * case["hq"] * case["d"] * e, "flops": 4 * pairs * case["hq"] * case["d"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _spread(shape, g, dev):
    """Normal values with a few large channels, as a decoder's activations have."""
    x = torch.randn(shape, generator=g, device=dev)
    big = torch.rand(shape[-1], generator=g, device=dev)
    return x * torch.where(big < 0.01, 20.0, 1.0) * (0.5 + big)


def _codes(shape, g, dev):
    return torch.randint(0, 256, shape, generator=g, device=dev, dtype=torch.uint8)


def _pages(case, g, dev):
    """A cache with room to spare, its pages in no order, and the lengths of its sequences."""
    lens = _lens(case)
    p = case["page"]
    most = -(-max(l for _, l in lens) // p)
    used = [-(-l // p) for _, l in lens]
    n = sum(used) + 3
    order = torch.randperm(n, generator=torch.Generator().manual_seed(int(g.initial_seed()) + 1))
    table = torch.full((case["b"], most), -1, dtype=torch.int32)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u].to(torch.int32)
        at += u
    cu = torch.tensor([0] + [m for m, _ in lens]).cumsum(0).to(torch.int32)
    kv = torch.tensor([l for _, l in lens], dtype=torch.int32)
    h, d = case["hk"], case["d"]
    s = {"table": table.to(dev), "cu": cu.to(dev), "lens": kv.to(dev), "most_new": max(m for m, _ in lens),
         "most_kv": max(l for _, l in lens), "tokens": int(cu[-1])}
    for name, shape in (("k", (n, h, p, d)), ("v", (n, h, d, p))):
        x = torch.randn(shape, generator=g, device=dev)
        s[name + "_cache"] = (x * 100).clamp(-448, 448).to(F8)
        e = torch.randint(-8, -5, (n, h), generator=g, device=dev)
        s[name + "_scale"] = torch.exp2(e.float())
    return s


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    s = {"case": case, "dtype": dt}
    if op == "quant":
        s["x"] = _spread((case["rows"], case["cols"]), g, dev).to(dt)
    elif op in ("linear", "gemm"):
        m, n, k = case["m"], case["n"], case["k"]
        s["wc"] = _codes((n, k // 2), g, dev)
        s["ws"] = torch.randint(116, 122, (n, k // 32), generator=g, device=dev, dtype=torch.uint8)
        if op == "linear":
            s["x"] = _spread((m, k), g, dev).to(dt)
        else:
            s["xc"] = _codes((m, k // 2), g, dev)
            s["xs"] = torch.randint(122, 130, (m, k // 32), generator=g, device=dev, dtype=torch.uint8)
    elif op == "rope":
        t, d = case["t"], case["d"]
        s["q"] = torch.randn((t, case["hq"], d), generator=g, device=dev).to(dt)
        s["k"] = torch.randn((t, case["hk"], d), generator=g, device=dev).to(dt)
        start = torch.randint(0, case["far"] - t + 1, (1,), generator=g, device=dev)
        s["pos"] = (start + torch.arange(t, device=dev)).to(torch.int32)
        # linear interpolation of the positions by 4, as for a context stretched to four times its length
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"]) / 4).float().to(dev)
    else:
        s |= _pages(case, g, dev)
        if op == "append":
            shape = (s["tokens"], case["hk"], case["d"])
            s["k"], s["v"] = (_spread(shape, g, dev).to(dt) for _ in range(2))
        else:
            s["q"] = torch.randn((s["tokens"], case["hq"], case["d"]), generator=g, device=dev).to(dt)
            s["softmax_scale"] = case["d"] ** -0.5
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _plain_quant(x):
    """(values fp32, codes uint8 [rows, cols / 2], scales uint8 [rows, cols / 32])."""
    rows, cols = x.shape
    b = x.float().view(rows, cols // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp(-127, 125)
    e = torch.where(amax == 0, -127, e)
    y = torch.ldexp(b, -e)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    idx = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    idx = (idx + 8 * torch.signbit(y).to(torch.uint8)).view(rows, cols)
    values = torch.ldexp(torch.copysign(a, y), e).view(rows, cols)
    return values, idx[:, ::2] | (idx[:, 1::2] << 4), (e + 127).to(torch.uint8).view(rows, cols // 32)


def _plain_values(codes, scales):
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1)
    e = scales.int() - 127
    return torch.ldexp(v.view(*scales.shape, 32), e.unsqueeze(-1)).view(codes.shape[0], -1)


def _plain_rope(x, pos, inv_freq, half):
    a = pos.double()[:, None] * inv_freq.double()
    c, s = a.cos().float()[:, None], a.sin().float()[:, None]
    r = 2 * inv_freq.numel()
    y = x.float()
    p, q = (y[..., :r // 2], y[..., r // 2:r]) if half else (y[..., 0:r:2], y[..., 1:r:2])
    u, v = p * c - q * s, q * c + p * s
    z = torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([z, y[..., r:]], -1).to(x.dtype)


def _plain_append(x, cache, scale, s, page, transposed):
    """The blocks that new tokens reach, each held as its codes times one power of two."""
    b = s["lens"].numel()
    cu, lens = s["cu"].long(), s["lens"].long()
    start = lens - (cu[1:] - cu[:-1])
    nb = (s["most_new"] - 2) // page + 2
    blk = start[:, None] // page + torch.arange(nb, device=x.device)
    blk = torch.where(blk * page < lens[:, None], blk, start[:, None] // page)     # past the end: the first one again
    pid = s["table"].long().gather(1, blk)                                          # [b, nb]
    pos = blk[..., None] * page + torch.arange(page, device=x.device)               # [b, nb, page]
    new = (pos >= start[:, None, None]) & (pos < lens[:, None, None])
    old = pos < start[:, None, None]
    row = (cu[:b, None, None] + pos - start[:, None, None]).clamp(0, x.shape[0] - 1)
    fresh = x[row].float().permute(0, 1, 3, 2, 4)                                   # [b, nb, h, page, d]
    codes = cache[pid]
    held = (codes.transpose(-1, -2) if transposed else codes).float()
    amax = torch.where(new[:, :, None, :, None], fresh.abs(), 0).amax((-1, -2))    # [b, nb, h]
    m, ex = torch.frexp(amax)
    e = torch.where(m > 0.875, ex - 8, ex - 9).clamp(min=-126)
    e = torch.where(amax == 0, -126, e)
    e_old = torch.where(old.any(-1)[:, :, None], torch.frexp(scale[pid])[1] - 1, -126)
    e_new = torch.maximum(e, e_old)
    y = torch.where(new[:, :, None, :, None], torch.ldexp(fresh, -e_new[..., None, None]),
                    torch.where(old[:, :, None, :, None], torch.ldexp(held, (e_old - e_new)[..., None, None]), held))
    y = y.to(F8)
    cache.view(torch.uint8).index_put_((pid,), (y.transpose(-1, -2) if transposed else y).view(torch.uint8))
    scale.index_put_((pid,), torch.exp2(e_new.float()))


def _plain_attn(s, hk, page):
    q, table = s["q"], s["table"].long().clamp(min=0)
    b, (t, hq, d) = s["lens"].numel(), q.shape
    cu, lens = s["cu"].long(), s["lens"].long()
    n, grp, most = cu[1:] - cu[:-1], hq // hk, s["most_new"]
    k = (s["k_cache"][table].float() * s["k_scale"][table][..., None, None]).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    v = s["v_cache"][table].float() * s["v_scale"][table][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(b, hk, -1, d)
    i = torch.arange(most, device=q.device)
    row = (cu[:b, None] + i).clamp(max=t - 1)
    qp = q[row].float().view(b, most, hk, grp, d).permute(0, 2, 3, 1, 4).reshape(b, hk, grp * most, d)
    sc = torch.matmul(qp, k.transpose(-1, -2)).view(b, hk, grp, most, -1) * s["softmax_scale"]
    last = (lens - n)[:, None] + i                                                  # [b, most]
    key = torch.arange(sc.shape[-1], device=q.device)
    seen = (key <= last[..., None]) & (key < lens[:, None, None])                   # [b, most, keys]
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True).clamp(min=-3e38))
    v = torch.where((key < lens[:, None])[:, None, :, None], v, 0)
    o = torch.matmul(p.view(b, hk, grp * most, -1), v).view(b, hk, grp, most, d)
    o = o / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.permute(0, 3, 1, 2, 4).reshape(b * most, hq, d).to(q.dtype)
    tok = torch.arange(t, device=q.device)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    return o[seq * most + tok - cu[seq]]


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        return _own(state, case, op)
    if op == "quant":
        v, c, e = _plain_quant(state["x"])
        return {"values": v.to(state["dtype"]), "codes": c, "scales": e}
    if op in ("linear", "gemm"):
        x = _plain_quant(state["x"])[0] if op == "linear" else _plain_values(state["xc"], state["xs"])
        return (x @ _plain_values(state["wc"], state["ws"]).t()).to(state["dtype"])
    if op == "rope":
        return [_plain_rope(state[n], state["pos"], state["inv_freq"], case["half"]) for n in ("q", "k")]
    if op == "append":
        _plain_append(state["k"], state["k_cache"], state["k_scale"], state, case["page"], False)
        _plain_append(state["v"], state["v_cache"], state["v_scale"], state, case["page"], True)
        return [state[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")]
    return _plain_attn(state, case["hk"], case["page"])


def _workspace(state, need):
    """The workspace that a program keeps beside its weights or its cache."""
    if need and state.get("workspace") is None:
        state["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return state["workspace"] if need else None


def _own(state, case, op):
    from weight_quantization_aware_amd import _lib as Q
    if op == "quant":
        x = state["x"]
        v = torch.empty_like(x)
        c = torch.empty(x.shape[0], x.shape[1] // 2, dtype=torch.uint8, device=x.device)
        e = torch.empty(x.shape[0], x.shape[1] // 32, dtype=torch.uint8, device=x.device)
        Q.qat_mx_quant(x, codes=c, scales=e, X_hat=v)
        return {"values": v, "codes": c, "scales": e}
    if op in ("linear", "gemm"):
        y = torch.empty(case["m"], case["n"], dtype=state["dtype"], device="cuda")
        ws = _workspace(state, Q.mx_ws_bytes(case["m"], case["n"], case["k"]))
        if op == "linear":
            Q.qat_mx_linear(state["x"], state["wc"], state["ws"], y, ws=ws)
        else:
            Q.qat_mx_gemm(state["xc"], state["xs"], state["wc"], state["ws"], y, ws=ws)
        return y
    if op == "rope":
        q, k = torch.empty_like(state["q"]), torch.empty_like(state["k"])
        Q.qat_rope(state["q"], state["pos"], state["inv_freq"], q, k=state["k"], k_out=k, half=case["half"])
        return [q, k]
    cache = [state[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")]
    if op == "append":
        Q.qat_kv_append(state["k"], state["v"], state["cu"], state["lens"], state["table"], *cache,
                        max_new=state["most_new"])
        return cache
    o = torch.empty_like(state["q"])
    ws = _workspace(state, Q.kv_attn_ws_bytes(state["tokens"], case["b"], case["hq"], case["hk"], case["d"],
                                              state["most_new"], state["most_kv"]))
    Q.qat_kv_attn(state["q"], state["cu"], state["lens"], state["table"], *cache, o, state["softmax_scale"],
                  max_new=state["most_new"], max_len=state["most_kv"], ws=ws)
    return o


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_quant(x):
    """Nearest element of the e2m1 grid by counting the midpoints below; a tie goes to the even code."""
    b = x.double().view(x.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0)))
    e = torch.where(torch.pow(2.0, e) > amax, e - 1, e)
    e = torch.where(torch.pow(2.0, e + 1) <= amax, e + 1, e) - 2
    e = torch.where(amax > 0, e, -127.0).clamp(-127, 125)
    a = b.abs() / torch.pow(2.0, e)
    idx = torch.zeros_like(a, dtype=torch.int32)
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        idx += ((a >= mid) if i % 2 else (a > mid)).int()
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    neg = torch.signbit(b)
    v = (torch.where(neg, -grid[idx], grid[idx]) * torch.pow(2.0, e)).view(x.shape)
    c = (idx + 8 * neg.int()).view(x.shape[0], -1, 2)
    return v, (c[..., 0] + 16 * c[..., 1]).to(torch.uint8), (e + 127).squeeze(-1).to(torch.uint8)


def _exact_values(codes, scales):
    c = torch.stack([codes % 16, codes // 16], -1).view(codes.shape[0], -1).long()
    m = c % 8
    mag = torch.where(m < 2, m * 0.5, (1 + (m % 2) * 0.5) * torch.pow(2.0, (m // 2 - 1).double()))
    w = torch.pow(2.0, scales.double() - 127).repeat_interleave(32, 1)
    return torch.where(c >= 8, -mag, mag) * w


def _exact_rope(x, pos, freq, half):
    r = 2 * freq.numel()
    a = pos.double().view(-1, 1, 1) * freq.double()
    i = torch.arange(r // 2, device=x.device)
    first, second = (i, i + r // 2) if half else (2 * i, 2 * i + 1)
    z = torch.polar(torch.ones_like(a), a) * torch.complex(x.double()[..., first], x.double()[..., second])
    out = x.double().clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_append(s, case):
    """Sequence by sequence and block by block on the host."""
    page = case["page"]
    got = []
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    for name in ("k", "v"):
        cache = s[name + "_cache"].cpu().double()
        cache = cache.transpose(-1, -2).contiguous() if name == "v" else cache
        scale, x = s[name + "_scale"].cpu().double(), s[name].cpu().double()
        for i, n in enumerate(lens):
            first = n - (cu[i + 1] - cu[i])
            for j in range(first // page, (n - 1) // page + 1):
                lo, hi, p = max(first, j * page), min(n, (j + 1) * page), table[i][j]
                new = x[cu[i] + lo - first:cu[i] + hi - first].transpose(0, 1)      # [h, tokens, d]
                amax = new.abs().amax((1, 2))
                e = torch.ceil(torch.log2(torch.where(amax > 0, amax / 448, 1.0)))
                e = torch.where(torch.pow(2.0, e) * 448 < amax, e + 1, e)
                e = torch.where(torch.pow(2.0, e - 1) * 448 >= amax, e - 1, e)
                e = torch.where(amax > 0, e.clamp(min=-126), -126.0)
                before = lo - j * page
                if before:
                    was = torch.log2(scale[p])
                    e = torch.maximum(e, was)
                    cache[p, :, :before] = _e4m3(cache[p, :, :before] * torch.pow(2.0, was - e)[:, None, None])
                cache[p, :, before:before + hi - lo] = _e4m3(new / torch.pow(2.0, e)[:, None, None])
                scale[p] = torch.pow(2.0, e)
        got.append((cache.transpose(-1, -2).contiguous() if name == "v" else cache, scale))
    return [got[0][0], got[1][0], got[0][1], got[1][1]]


def _e4m3(y):
    """Rounded to three bits behind the leading one, or to multiples of 2^-9 below 2^-6; ties to even."""
    step = torch.pow(2.0, torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _exact_attn(s, case):
    page, hk = case["page"], case["hk"]
    grp = case["hq"] // hk
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for i, n in enumerate(lens):
        new = cu[i + 1] - cu[i]
        ids = s["table"][i, :-(-n // page)].long()
        k = (s["k_cache"][ids].double() * s["k_scale"][ids].double()[..., None, None]).transpose(1, 2)
        v = (s["v_cache"][ids].double() * s["v_scale"][ids].double()[..., None, None]).permute(0, 3, 1, 2)
        k, v = (x.reshape(-1, hk, case["d"])[:n].transpose(0, 1) for x in (k, v))
        for j in range(0, new, 256):
            m = min(256, new - j)
            q = s["q"][cu[i] + j:cu[i] + j + m].double().view(m, hk, grp, -1).permute(1, 2, 0, 3).reshape(hk, grp * m, -1)
            x = (q @ k.transpose(1, 2).contiguous()).view(hk, grp, m, n) * s["softmax_scale"]
            late = torch.arange(n, device=x.device) > torch.arange(n - new + j, n - new + j + m, device=x.device)[:, None]
            x = torch.softmax(x.masked_fill(late, -math.inf), -1).view(hk, grp * m, n) @ v
            out[cu[i] + j:cu[i] + j + m] = x.view(hk, grp, m, -1).permute(2, 0, 1, 3).reshape(m, case["hq"], -1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        v, c, e = _exact_quant(s["x"])
        return {"values": v, "codes": c, "scales": e}
    if op in ("linear", "gemm"):
        x = _exact_quant(s["x"])[0] if op == "linear" else _exact_values(s["xc"], s["xs"])
        return x @ _exact_values(s["wc"], s["ws"]).t()
    if op == "rope":
        return [_exact_rope(s[n], s["pos"], s["inv_freq"], case["half"]) for n in ("q", "k")]
    if op == "append":
        return _exact_append(s, case)
    return _exact_attn(s, case)
