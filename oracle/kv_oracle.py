"""Plain fp64 numpy forms of include/qat_kv.h: rotary positions, the paged
e4m3 cache and the attention over it. Test infrastructure only; shares no code
with the kernels."""
import numpy as np

# value of every e4m3 (OCP FP8 E4M3) code
_c = np.arange(256)
_e, _m = (_c >> 3) & 15, _c & 7
E4M3 = np.where(_e == 0, _m / 8 * 2.0 ** -6, (1 + _m / 8) * 2.0 ** (_e - 7.0)) * np.where(_c & 128, -1.0, 1.0)
E4M3[[0x7F, 0xFF]] = np.nan
_POS = E4M3[:0x7F]                                          # 0 .. 448, ascending with the code


def e4m3(y):
    """Codes of y rounded to nearest, ties to even; NaN and infinities give 0x7F. |y| <= 448 otherwise."""
    y = np.asarray(y, np.float64)
    a = np.where(np.isfinite(y), np.abs(y), 0.0)
    hi = np.clip(np.searchsorted(_POS, a), 1, len(_POS) - 1)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = c | (np.signbit(y).astype(np.int64) << 7)
    return np.where(np.isfinite(y), c, 0x7F).astype(np.uint8)


def inv_freq(rot, base=10000.0, scaling="plain", factor=1.0, original=1, beta_fast=32.0, beta_slow=1.0):
    i = np.arange(rot // 2)
    f = base ** (-2.0 * i / rot)
    if scaling == "plain":
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    turns = lambda n: rot * np.log(original / (n * 2 * np.pi)) / (2 * np.log(base))
    lo, hi = max(np.floor(turns(beta_fast)), 0), min(np.ceil(turns(beta_slow)), rot - 1)
    if hi <= lo:
        hi = lo + 0.001
    keep = 1 - np.clip((i - lo) / (hi - lo), 0, 1)
    return f / factor * (1 - keep) + f * keep, (0.1 * np.log(factor) + 1 if factor > 1 else 1.0)


def rope(x, pos, freq, half, mscale=1.0, inverse=False):
    """x [tokens, heads, d] fp64, pos [tokens], freq [rot / 2] (the fp32 values, as fp64)."""
    r = 2 * len(freq)
    i = np.arange(r // 2)
    p, q = (i, i + r // 2) if half else (2 * i, 2 * i + 1)
    a = pos.astype(np.longdouble)[:, None] * freq.astype(np.longdouble)
    c, s = np.cos(a).astype(np.float64)[:, None], np.sin(a).astype(np.float64)[:, None]
    if inverse:
        s = -s
    out = np.array(x, np.float64)
    out[..., p] = mscale * (x[..., p] * c - x[..., q] * s)
    out[..., q] = mscale * (x[..., q] * c + x[..., p] * s)
    return out


def scale_exp(amax):
    """The smallest e >= -126 with 448 2^e >= amax."""
    e = -126
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return e


def append(x, cu, lens, table, codes, scale, max_new=None):
    """x [tokens, heads, d] into codes [pages, heads, page, d] and scale [pages, heads], in place."""
    n_pages, heads, page, _ = codes.shape
    cols = table.shape[1]
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        start = int(lens[b]) - n
        blocks = {}
        for i in range(n if max_new is None else min(n, max_new)):
            p = start + i
            if 0 <= p < cols * page and 0 <= table[b][p // page] < n_pages:
                blocks.setdefault(p // page, []).append(i)
        for blk, toks in blocks.items():
            pid, slot0 = int(table[b][blk]), start + toks[0] - blk * page
            for h in range(heads):
                new = np.asarray(x[[cu[b] + i for i in toks], h], np.float64)
                fin = np.abs(new[np.isfinite(new)])
                e = scale_exp(fin.max() if fin.size else 0.0)
                if slot0 > 0:
                    old = int(np.frexp(scale[pid, h])[1]) - 1
                    if e > old:
                        held = codes[pid, h, :slot0]
                        nan = np.isnan(E4M3[held])
                        codes[pid, h, :slot0] = np.where(nan, held, e4m3(np.nan_to_num(E4M3[held]) * 2.0 ** (old - e)
                                                                         * 1.0) | (held & 128))
                    e = max(e, old)
                scale[pid, h] = 2.0 ** e
                codes[pid, h, slot0:slot0 + len(toks)] = e4m3(new * 2.0 ** -e)


def attend(q, cu, lens, table, k, ks, v, vs, softmax_scale, causal):
    """q [tokens, hq, d] fp64; k, v codes [pages, hk, page, d]. Per token and head: the output and the terms of its
    error bound: (out, sum p |v|, largest |score| term sum, sum |code| max scale)."""
    hk, page, d = k.shape[1:]
    hq = q.shape[1]
    out = np.zeros(q.shape)
    absv, sabs, tail = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape)
    for b in range(len(lens)):
        n, ln = int(cu[b + 1] - cu[b]), int(lens[b])
        pos = np.arange(max(0, min(ln, table.shape[1] * page)))
        pid = table[b][pos // page] if len(pos) else np.zeros(0, int)
        ok = (pid >= 0) & (pid < k.shape[0])
        pos, pid = pos[ok], pid[ok]
        for i in range(n):
            at = ln - n + i
            use = pos <= at if causal else np.ones(len(pos), bool)
            p_, id_ = pos[use], pid[use]
            if not len(p_):
                continue
            for h in range(hq):
                g = h // (hq // hk)
                kk = E4M3[k[id_, g, p_ % page]] * ks[id_, g][:, None].astype(np.float64)
                code = E4M3[v[id_, g, p_ % page]]
                vv = code * vs[id_, g][:, None].astype(np.float64)
                s = kk @ q[cu[b] + i, h] * softmax_scale
                w = np.exp(s - s.max())
                w /= w.sum()
                t = cu[b] + i
                out[t, h] = w @ vv
                absv[t, h] = w @ np.abs(vv)
                sabs[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * softmax_scale
                tail[t, h] = np.abs(code).sum(0) * vs[id_, g].max()
    return out, absv, sabs, tail
