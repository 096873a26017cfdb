"""GPU parity of rotary positions, the 8-bit cache and its attention against the fp64 oracle, through the C ABI.

Bounds, u = eps / 2 of the activations' type, v = 2^-24:
- rotary: cosine and sine of the reduced fp32 angle are off by at most pi v
  (the angle) + 3 v (the function) and mscale's product adds v of their
  magnitude <= mscale; the two products and the sum add 3 v of their terms, so
  |got - ref| <= u |ref| + (1 + u) 12 v mscale (|x_p| + |x_q|) + least;
- append: every step but one rounding is exact: codes and scales bit for bit;
- attention: with E = gamma(head_dim + 8) * 2 * max_j (scale sum |q k_j|) the
  error of a score, a weight is off by a factor e^(2 E) at most, by 2^-11 for
  its rounding to fp16 and by 16 v for exponentials and products; fp16's
  spacing below 2^-14 adds 2^-25 of a weight of 1, in units of the largest
  value scale; the sums over n keys add 2 gamma(n + 64). With A = sum p |v| and
  T = sum |code| max scale:
  |got - ref| <= u |ref| + (1 + u) ((2^-11 + 2 (e^(4 E) - 1) + 4 gamma(n + 64) + 32 v) A + 2^-25 T) + least.
"""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as KV
from weight_quantization_aware_amd import _lib as Q
from tests.helpers import check_bound, gamma, say

pytestmark = pytest.mark.gpu

V = 2.0 ** -24
LEAST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


def host(t):
    return t.detach().cpu().double().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rand(shape, seed, dtype):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

def check_rope(x, y, pos, f, half, mscale, inverse):
    xv, fv = host(x), f.double().numpy()
    ref = KV.rope(xv, pos, fv, half, mscale, inverse)
    r = 2 * len(fv)
    pair = np.arange(r)
    pair = (pair + r // 2) % r if half else pair ^ 1
    mag = np.zeros(ref.shape)
    mag[..., :r] = np.abs(xv[..., :r]) + np.abs(xv[..., pair])
    u = torch.finfo(x.dtype).eps / 2
    bound = np.where(mag > 0, u * np.abs(ref) + (1 + u) * 12 * V * mscale * mag + LEAST[x.dtype], 0)
    check_bound("rope", host(y), ref, bound)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("T,hq,hk,d,rot,far", [(1, 1, 0, 64, 16, 10), (1, 32, 32, 128, 128, 1 << 20), (3, 7, 1, 128, 96, 4096),
                                               (300, 8, 2, 64, 64, 131072), (65, 40, 8, 128, 32, 2 ** 31 - 100)])
def test_rope(T, hq, hk, d, rot, far, half, dtype):
    say(f"rope T={T} heads={hq}+{hk} d={d} rot={rot} half={half} far={far} {dtype}")
    f, ms = Q.rope_inv_freq(rot, scaling="parts", factor=8.0, original=4096)
    pos = np.arange(T) + far - T
    q, k = rand((T, hq, d), T, dtype), rand((T, hk, d), T + 1, dtype) if hk else None
    qo, ko = torch.empty_like(q), torch.empty_like(k) if hk else None
    Q.qat_rope(q, i32(pos.tolist()), f.cuda(), qo, k=k, k_out=ko, half=half, mscale=ms)
    check_rope(q, qo, pos, f, half, ms, False)
    if hk:
        check_rope(k, ko, pos, f, half, ms, False)
    Q.qat_rope(q, i32(pos.tolist()), f.cuda(), qo, half=half, mscale=ms, inverse=True)
    check_rope(q, qo, pos, f, half, ms, True)


def test_rope_in_place_on_slices_of_one_projection():
    T, hq, hk, d = 9, 6, 2, 64
    qkv = rand((T, (hq + 2 * hk) * d), 5, BF)
    was = qkv.clone()
    q, k = (qkv[:, :hq * d].view(T, hq, d), qkv[:, hq * d:(hq + hk) * d].view(T, hk, d))
    f, _ = Q.rope_inv_freq(d)
    pos = np.array([0, 1, 2, 77, 5, -3, 0, 0, 9])
    Q.qat_rope(q, i32(pos.tolist()), f.cuda(), q, k=k, k_out=k)
    check_rope(was[:, :hq * d].view(T, hq, d), q, pos, f, True, 1.0, False)
    check_rope(was[:, hq * d:(hq + hk) * d].view(T, hk, d), k, pos, f, True, 1.0, False)
    assert torch.equal(qkv[:, (hq + hk) * d:], was[:, (hq + hk) * d:])
    Q.qat_rope(q[:0], i32([]), f.cuda(), q[:0])


@pytest.mark.parametrize("half", [True, False])
def test_rope_inverse_is_the_gradient(half):
    # d(sum g . rope(x)) / dx against differences, and against the formula R^T g
    T, d, rot = 4, 64, 48
    f, _ = Q.rope_inv_freq(rot)
    pos = np.array([3, 1000, 0, 17])
    g = rand((T, 2, d), 1, HF)
    dx = torch.empty_like(g)
    Q.qat_rope(g, i32(pos.tolist()), f.cuda(), dx, half=half, mscale=1.25, inverse=True)
    x, fv, gv = np.random.default_rng(0).standard_normal((T, 2, d)), f.double().numpy(), host(g)
    for t, h, e in [(0, 0, 0), (1, 1, 5), (1, 0, 30), (3, 1, 47), (2, 0, 50)]:
        step = np.zeros_like(x)
        step[t, h, e] = 0.5                                  # linear in x: a difference is exact up to fp64
        diff = ((KV.rope(x + step, pos, fv, half, 1.25) - KV.rope(x - step, pos, fv, half, 1.25)) * gv).sum()
        mag = np.abs(gv[t, h]).max() * 2
        assert abs(host(dx)[t, h, e] - diff) <= 2.0 ** -11 * abs(diff) + 12 * V * 1.25 * mag + LEAST[HF]


# ---------------------------------------------------------------------------
# The cache
# ---------------------------------------------------------------------------

class Cache:
    """A device cache and its host copy, pages in random order, everything outside the sequences poisoned."""

    def __init__(self, lens, heads, d, page, seed=0, spare=2, cols=None):
        rng = np.random.default_rng(seed)
        used = [max(0, -(-l // page)) for l in lens] if cols is None else [min(cols, -(-l // page)) for l in lens]
        n = sum(used) + spare
        order = rng.permutation(n)
        cols = max(1, max(used, default=1)) if cols is None else cols
        self.table = np.full((len(lens), cols), -1, np.int64)
        at = 0
        for i, u in enumerate(used):
            self.table[i, :u] = order[at:at + u]
            at += u
        # codes of NaN and scales that are not numbers wherever no token is
        self.k = np.full((n, heads, page, d), 0x7F, np.uint8)
        self.v = np.full((n, heads, page, d), 0xFF, np.uint8)
        self.ks, self.vs = (np.full((n, heads), np.nan, np.float32) for _ in range(2))
        self.lens, self.page, self.rng = lens, page, rng

    def fill(self, wide=3):
        heads = self.k.shape[1]
        for b, l in enumerate(self.lens):
            for j in range(-(-max(l, 0) // self.page)):
                p, m = self.table[b, j], min(self.page, l - j * self.page)
                for c, s in ((self.k, self.ks), (self.v, self.vs)):
                    c[p, :, :m] = KV.e4m3(np.clip(self.rng.standard_normal((heads, m, c.shape[-1])) * 100, -448, 448))
                    s[p] = 2.0 ** self.rng.integers(-8 - wide, -5, heads)
        return self

    def device(self):
        f8 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda().view(torch.float8_e4m3fn)
        return [f8(self.k), f8(self.v.transpose(0, 1, 3, 2)), torch.from_numpy(self.ks).cuda(),
                torch.from_numpy(self.vs).cuda()]

    def tab(self):
        return torch.from_numpy(self.table.astype(np.int32)).cuda()


def same_codes(got, want):
    """Bit for bit, but the NaN code has either sign."""
    got = got.view(torch.uint8).cpu().numpy()
    return np.array_equal(np.where(got & 0x7F == 0x7F, 0x7F, got), np.where(want & 0x7F == 0x7F, 0x7F, want))


def check_append(c, k, v, cu, lens, dev, max_new=None):
    Q.qat_kv_append(k, v, i32(cu), i32(lens), c.tab(), *dev, max_new=max_new)
    KV.append(host(k), cu, lens, c.table, c.k, c.ks, max_new)
    KV.append(host(v), cu, lens, c.table, c.v, c.vs, max_new)
    torch.cuda.synchronize()
    assert same_codes(dev[0], c.k)
    assert same_codes(dev[1].view(torch.uint8).transpose(-1, -2), c.v)
    assert np.array_equal(dev[2].cpu().numpy(), c.ks, equal_nan=True)
    assert np.array_equal(dev[3].cpu().numpy(), c.vs, equal_nan=True)


APPEND = [
    # new tokens and lengths of each sequence, heads, d, page
    ([1], [1], 1, 64, 16),
    ([1, 1, 1, 1], [1, 16, 17, 64], 2, 128, 16),
    ([1, 0, 1], [65, 0, 128], 2, 64, 64),
    ([3, 70, 0, 16], [3, 75, 9, 32], 2, 64, 32),
    ([130, 5], [130, 200], 1, 128, 128),
    ([2, 33], [129, 33], 3, 128, 64),
    ([4, 9], [19, 130], 1, 128, 128),
    ([7], [5], 1, 64, 16),                      # two tokens before position 0: left out
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("new,lens,heads,d,page", APPEND)
def test_append(new, lens, heads, d, page, dtype):
    say(f"append new={new} lens={lens} heads={heads} d={d} page={page} {dtype}")
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    c = Cache(lens, heads, d, page).fill()
    dev = c.device()
    T = cu[-1] + 2                              # two rows behind the last sequence
    base = rand((T, 3 * heads * d), T, dtype)
    k, v = (base[:, i * heads * d:(i + 1) * heads * d].view(T, heads, d) for i in (0, 2))
    k[0, 0, 0], k[0, 0, 1] = 300.0, -0.0        # grows a scale
    check_append(c, k, v, cu, lens, dev)
    check_append(c, k, v, cu, lens, dev)        # again: nothing changes
    check_append(c, (k * 64).to(dtype), (v * 0).to(dtype), cu, lens, dev)


def test_append_step_by_step():
    c = Cache([40, 23], 2, 64, 16)
    dev = c.device()
    lens = [0, 0]
    for step, new in enumerate([[9, 0], [1, 1], [1, 20], [0, 1], [29, 1]]):
        lens = [a + b for a, b in zip(lens, new)]
        cu = [0, new[0], sum(new)]
        k, v = (rand((cu[-1], 2, 64), 10 * step + i, BF) * 4.0 ** (step % 3) for i in range(2))
        check_append(c, k, v, cu, lens, dev, max_new=max(new))
    assert lens == [40, 23]


def test_append_non_finite_and_tiny():
    c = Cache([33], 1, 64, 16)
    dev = c.device()
    k = rand((33, 1, 64), 1, BF)
    k[3, 0, 5], k[4, 0, 6], k[20, 0, 0] = float("inf"), float("nan"), -float("inf")
    k[32] = 0
    v = (rand((33, 1, 64), 2, BF) * 2.0 ** -130).to(BF)
    v[16:32] *= 2.0 ** 120
    v[31, 0, 63] = 3e38
    check_append(c, k, v, [0, 33], [33], dev)
    assert np.isnan(KV.E4M3[c.k[c.table[0, 0], 0, 3, 5]])


def test_append_leaves_out_what_has_no_slot():
    # pages out of range, positions beyond the table, cu and lens that make no sense
    c = Cache([64, 64], 1, 64, 16, cols=3)
    c.table[0, 1], c.table[1, 2] = 10 ** 6, -5
    dev = c.device()
    k, v = rand((128, 1, 64), 1, HF), rand((128, 1, 64), 2, HF)
    check_append(c, k, v, [0, 64, 128], [64, 64], dev)
    was = [t.clone() for t in dev]
    for cu, lens in [([0, -7, 500], [64, 64]), ([0, 64, 128], [-5, -2 ** 31]), ([0, 64, 128], [2 ** 31 - 1, 10 ** 9]),
                     ([2 ** 31 - 1, -2 ** 31, 3], [7, 7]), ([100, 50, 20], [16, 16])]:
        Q.qat_kv_append(k, v, i32(cu), i32(lens), c.tab(), *dev)
    torch.cuda.synchronize()
    spare = [p for p in range(c.k.shape[0]) if p not in set(c.table.ravel().tolist())]
    for a, b in zip(was, dev):
        assert torch.equal(a.view(torch.uint8)[spare], b.view(torch.uint8)[spare])


def test_append_max_new_leaves_later_tokens_out():
    c = Cache([50], 2, 64, 32)
    dev = c.device()
    check_append(c, rand((50, 2, 64), 1, BF), rand((50, 2, 64), 2, BF), [0, 50], [50], dev, max_new=20)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def check_attn(c, q, cu, lens, scale, causal, out=None, dev=None, **kw):
    dev = c.device() if dev is None else dev
    T, hq, d = q.shape
    max_new = max([b - a for a, b in zip(cu, cu[1:])] + [0])
    kw.setdefault("max_new", max_new)
    kw.setdefault("max_len", max(max(lens), 0))
    ws = Q.workspace(Q.kv_attn_ws_bytes(T, len(lens), hq, c.k.shape[1], d, kw["max_new"], kw["max_len"]))
    ws.fill_(0xFF)
    o = torch.full((T, hq, d), 3.0, dtype=q.dtype, device="cuda") if out is None else out
    Q.qat_kv_attn(q, i32(cu), i32(lens), c.tab(), *dev, o, scale, causal=causal, ws=ws, **kw)
    torch.cuda.synchronize()
    ref, A, S, T_ = KV.attend(host(q), cu, lens, c.table, c.k, c.ks, c.v, c.vs, scale, causal)
    n = max(max(lens), 1)
    E = 2 * gamma(d + 8) * S
    u = torch.finfo(q.dtype).eps / 2
    rel = 2.0 ** -11 + 2 * np.expm1(4 * E) + 4 * gamma(n + 64) + 32 * V
    bound = u * np.abs(ref) + (1 + u) * (rel[..., None] * A + 2.0 ** -25 * T_) + LEAST[q.dtype]
    live = slice(0, cu[-1])
    check_bound("attention", host(o)[live], ref[live], bound[live])
    return o, host(o), ref


ATTN = [
    # new tokens and lengths of each sequence, hq, hk, d, page
    ([1], [1], 1, 1, 64, 16),
    ([1], [257], 4, 4, 128, 16),
    ([1, 1, 1, 1, 1], [15, 16, 17, 63, 65], 8, 2, 64, 16),
    ([1, 1, 1], [64, 128, 129], 7, 1, 128, 64),
    ([1, 0, 1, 1], [0, 5, 200, 1], 16, 2, 64, 128),
    ([1, 1], [1500, 700], 8, 1, 128, 32),
    ([1, 1, 1], [2100, 3, 513], 24, 2, 64, 128),
    ([2, 1, 5], [300, 70, 5], 8, 2, 128, 64),
    ([3, 17], [33, 17], 2, 2, 64, 32),
    ([16, 1], [700, 650], 4, 1, 128, 16),
    ([40, 0, 9], [40, 77, 100], 4, 2, 128, 64),
    ([130], [130], 2, 1, 64, 16),
    ([128, 64], [192, 64], 3, 3, 128, 128),
    ([70, 33], [600, 33], 10, 5, 64, 64),
    ([200], [1000], 8, 8, 128, 64),
    # enough workgroups of 128 rows for the prompts' kernel: ragged, empty and short sequences in one batch
    ([40, 33, 64], [40, 100, 64], 64, 64, 64, 16),
    ([70, 0, 130, 1], [70, 0, 300, 50], 96, 48, 128, 64),
    ([129, 5], [191, 500], 80, 80, 128, 128),
    ([35, 128, 2], [90, 128, 1], 320, 64, 64, 32),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,lens,hq,hk,d,page", ATTN)
def test_attn(new, lens, hq, hk, d, page, causal, dtype):
    say(f"attn new={new} lens={lens} heads={hq}/{hk} d={d} page={page} causal={causal} {dtype}")
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    c = Cache(lens, hk, d, page).fill()
    T = cu[-1] + 3
    base = rand((T, 2 * hq * d), T, dtype)
    q = base[:, hq * d:].view(T, hq, d)
    outb = torch.full((T, hq + 1, d), 3.0, dtype=dtype, device="cuda")
    o, _, _ = check_attn(c, q, cu, lens, d ** -0.5, causal, out=outb[:, :hq])
    assert (outb[cu[-1]:] == 3).all() and (outb[:, hq] == 3).all()     # rows and columns of others


def test_attn_split_over_a_long_cache():
    c = Cache([9000, 1, 2500], 1, 64, 64).fill()
    check_attn(c, rand((3, 2, 64), 1, HF), [0, 1, 2, 3], [9000, 1, 2500], 0.125, True)


def test_attn_many_sequences():
    lens = [(37 * i) % 300 for i in range(150)]
    c = Cache(lens, 1, 64, 16).fill()
    check_attn(c, rand((150, 2, 64), 1, BF), list(range(151)), lens, 0.125, True)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_attn_large_scores_and_spread_scales(dtype):
    # probabilities that reach one key only, and value scales 2^12 apart
    for hk, cu in ((2, [0, 1, 2]), (96, [0, 40, 80])):
        c = Cache([700, 90], hk, 64, 32).fill()
        for p in range(c.vs.shape[0]):
            c.vs[p] *= 2.0 ** (p % 13)
        check_attn(c, rand((cu[-1], max(hk, 4), 64), 1, dtype) * 8, cu, [700, 90], 1.0, True)


@pytest.mark.parametrize("new,hk", [(1, 1), (5, 1), (90, 1), (90, 96)])
def test_attn_masked_nan_stays_out(new, hk):
    # a key and a value that are not numbers, in the middle of the new tokens: rows before them see
    # neither, rows from them on see both; pages left out and slots behind the end are poison too
    n, d = 200, 64
    for what in ("k", "v"):
        c = Cache([n], hk, d, 16).fill()
        at = n - 1 - new // 2
        getattr(c, what)[c.table[0, at // 16], :, at % 16, 7] = 0x7F
        q = rand((new, 2 * hk, d), 3, BF)
        dev, out = c.device(), torch.empty(new, 2 * hk, d, dtype=BF, device="cuda")
        Q.qat_kv_attn(q, i32([0, new]), i32([n]), c.tab(), *dev, out, 0.125, ws=Q.workspace(1 << 24))
        first = at - (n - new)                  # the first row that sees position `at`
        o = host(out)
        assert np.isfinite(o[:first]).all(), what
        bad = np.isnan(o[first:])
        assert bad.all() if what == "k" else (bad[..., 7].all() and not bad[..., :7].any())


def test_attn_bad_pages_are_left_out():
    for page in (16, 64):
        c = Cache([300, 130], 2, 64, page).fill()
        c.table[0, 1], c.table[0, -1], c.table[1, 0] = -1, 10 ** 7, c.k.shape[0]
        check_attn(c, rand((4, 4, 64), 1, HF), [0, 3, 4], [300, 130], 0.125, True)
        check_attn(c, rand((4, 4, 64), 1, HF), [0, 3, 4], [300, 130], 0.125, False)
    big = Cache([300, 130], 96, 64, 32).fill()  # the prompts' kernel
    big.table[0, 1], big.table[0, -1], big.table[1, 0] = -1, 10 ** 7, big.k.shape[0]
    check_attn(big, rand((75, 96, 64), 1, HF), [0, 40, 75], [300, 130], 0.125, True)
    check_attn(big, rand((75, 96, 64), 1, HF), [0, 40, 75], [300, 130], 0.125, False)
    big.table[:] = -1
    _, o, _ = check_attn(big, rand((75, 96, 64), 1, HF), [0, 40, 75], [300, 130], 0.125, True)
    assert (o == 0).all()
    c.table[:] = -1                             # nothing is left
    _, o, _ = check_attn(c, rand((4, 4, 64), 1, HF), [0, 3, 4], [300, 130], 0.125, True)
    assert (o == 0).all()


def test_attn_rows_without_keys_are_zero():
    c = Cache([3, 0, 20], 1, 64, 16).fill()
    _, o, _ = check_attn(c, rand((9, 2, 64), 1, BF), [0, 7, 8, 9], [3, 0, 20], 0.125, True)
    assert (o[:4] == 0).all() and (o[4:7] != 0).any() and (o[7] == 0).all()


def test_attn_device_lengths_out_of_range():
    # lengths, offsets and bounds that make no sense stay inside every buffer
    c = Cache([64, 64], 1, 64, 16).fill()
    dev, q = c.device(), rand((8, 2, 64), 1, BF)
    guard = torch.full((10, 2, 64), 3.0, dtype=BF, device="cuda")
    for cu, lens, mn, ml in [([0, -7, 500], [64, 64], 4, 64), ([0, 4, 8], [2 ** 31 - 1, -2 ** 31], 4, 64),
                             ([8, 4, 0], [64, 64], 8, 1000), ([0, 4, 8], [64, 64], 2, 30),
                             ([2 ** 31 - 1, -2 ** 31, 8], [5, 5], 8, 64), ([0, 4, 8], [10 ** 9, 64], 4, 1 << 29)]:
        Q.qat_kv_attn(q, i32(cu), i32(lens), c.tab(), *dev, guard[1:9], 0.125, max_new=mn, max_len=ml,
                      ws=Q.workspace(1 << 24))
    torch.cuda.synchronize()
    assert (guard[0] == 3).all() and (guard[9] == 3).all()
    # max_len and max_new cut: rows beyond max_new stay, keys beyond max_len are not seen
    out = torch.full((8, 2, 64), 3.0, dtype=BF, device="cuda")
    Q.qat_kv_attn(q, i32([0, 4, 8]), i32([64, 64]), c.tab(), *dev, out, 0.125, causal=False, max_new=2, max_len=30,
                  ws=Q.workspace(1 << 24))
    ref, *_ = KV.attend(host(q), [0, 4, 8], [30, 30], c.table, c.k, c.ks, c.v, c.vs, 0.125, False)
    o = host(out)
    assert (o[[2, 3, 6, 7]] == 3).all() and np.abs(o[[0, 1, 4, 5]] - ref[[0, 1, 4, 5]]).max() < 0.05


def test_attn_of_a_cache_past_32_bit_offsets():
    # 40000 pages of 64 x 8 x 128 bytes: 2.6 GB of keys; the sequence lives in the last pages
    n, heads, d, page = 40000, 8, 128, 64
    k = torch.zeros(n, heads, page, d, dtype=torch.uint8, device="cuda")
    v = torch.zeros(n, heads, d, page, dtype=torch.uint8, device="cuda")
    ks, vs = torch.ones(n, heads, device="cuda"), torch.ones(n, heads, device="cuda")
    c = Cache([150], heads, d, page, spare=0).fill()
    ids = n - 1 - c.table[0] * 7
    kk, vv, a, b = c.device()
    src = torch.from_numpy(c.table[0]).cuda()
    dst = torch.from_numpy(ids).cuda()
    k[dst], v[dst], ks[dst], vs[dst] = kk.view(torch.uint8)[src], vv.view(torch.uint8)[src], a[src], b[src]
    q, tab = rand((1, 16, d), 1, BF), torch.from_numpy(ids.astype(np.int32)[None]).cuda()
    new = rand((1, heads, d), 2, BF)
    for dev, t in (((k, v, ks, vs), tab), ((kk, vv, a, b), c.tab())):
        Q.qat_kv_append(new, new, i32([0, 1]), i32([150]), t, *dev)
    outs = [torch.empty_like(q) for _ in range(2)]
    Q.qat_kv_attn(q, i32([0, 1]), i32([150]), tab, k, v, ks, vs, outs[0], 0.1, ws=Q.workspace(1 << 24))
    Q.qat_kv_attn(q, i32([0, 1]), i32([150]), c.tab(), kk, vv, a, b, outs[1], 0.1, ws=Q.workspace(1 << 24))
    assert torch.equal(outs[0], outs[1]) and torch.isfinite(outs[0].float()).all()


@pytest.mark.parametrize("new,lens,hk", [([1, 1, 1], [1500, 900, 40], 2), ([100, 20, 3], [100, 300, 3], 2),
                                         ([100, 20, 3], [100, 300, 3], 32)])
def test_attn_replayed_graphs_share_a_workspace(new, lens, hk):
    hq, d = 4 * hk, 64
    c = Cache([l + 8 for l in lens], hk, d, 32).fill()
    dev, tab, cu = c.device(), c.tab(), i32(np.concatenate([[0], np.cumsum(new)]).tolist())
    ln = i32(lens)
    q = rand((sum(new), hq, d), 1, BF)
    top = max(lens) + 8
    ws = Q.workspace(Q.kv_attn_ws_bytes(sum(new), 3, hq, hk, d, max(new), top))
    call = lambda o, causal: Q.qat_kv_attn(q, cu, ln, tab, *dev, o, 0.125, causal=causal, max_new=max(new), max_len=top,
                                           ws=ws)
    outs = [torch.empty_like(q) for _ in range(2)]
    graphs = []
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for i, o in enumerate(outs):
        with torch.cuda.stream(st):
            call(o, i == 0)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                call(o, i == 0)
        graphs.append(g)
    torch.cuda.current_stream().wait_stream(st)
    want = torch.empty_like(q)
    for step in range(4):
        q.copy_(rand(q.shape, 50 + step, BF))
        ln.add_(1)
        for i, g in enumerate(graphs):
            outs[i].fill_(5)
            g.replay()
            call(want, i == 0)
            torch.cuda.synchronize()
            assert torch.equal(outs[i], want), (step, i)


def test_attn_is_the_same_twice():
    c = Cache([3000, 100], 2, 128, 64).fill()
    dev, q = c.device(), rand((2, 16, 128), 1, BF)
    outs = [torch.empty_like(q) for _ in range(2)]
    for o in outs:
        Q.qat_kv_attn(q, i32([0, 1, 2]), i32([3000, 100]), c.tab(), *dev, o, 0.09, ws=Q.workspace(1 << 24))
    assert torch.equal(*outs)


def test_workspace_too_small_is_refused():
    c = Cache([3000], 1, 64, 64).fill()
    q = rand((1, 1, 64), 1, BF)
    out = torch.full_like(q, 3.0)
    for ws in (None, Q.workspace(64)):
        with pytest.raises(Q.QatError) as e:
            Q.qat_kv_attn(q, i32([0, 1]), i32([3000]), c.tab(), *c.device(), out, 0.1, ws=ws)
        assert e.value.status == 6
    torch.cuda.synchronize()
    assert (out == 3).all()


@pytest.mark.parametrize("new,hk", [(1, 2), (40, 96)])
def test_attn_page_scales_that_are_not_numbers_or_zero(new, hk):
    # a NaN scale of a page that is seen shows; zero scales give scores of zero and values of zero
    n, d = 100, 64
    q = rand((new, hk, d), 3, BF)
    run = lambda c, o: Q.qat_kv_attn(q, i32([0, new]), i32([n]), c.tab(), *c.device(), o, 0.125,
                                     ws=Q.workspace(1 << 24))
    for what in ("ks", "vs"):
        c = Cache([n], hk, d, 32).fill()
        getattr(c, what)[c.table[0, 0]] = np.nan
        o = torch.zeros_like(q)
        run(c, o)
        assert torch.isnan(o).all(), what
    c = Cache([n], hk, d, 32).fill()
    c.vs[c.table[0]] = 0
    o = torch.ones_like(q)
    run(c, o)
    assert (o == 0).all()
    c = Cache([n], hk, d, 32).fill()
    c.ks[c.table[0, 1]] = 0
    check_attn(c, q, [0, new], [n], 0.125, True)


def test_decode_step_captured_and_replayed():
    # rope, append and attention of three sequences as one graph; lengths and positions move on the device
    hq, hk, d, page, start = 8, 2, 64, 16, [30, 5, 61]
    c = Cache([l + 6 for l in start], hk, d, page).fill()
    for b, l in enumerate(start):               # only the first `start` positions are there
        for p in range(l, l + 6):
            c.k[c.table[b, p // page], :, p % page] = 0x7F
            c.v[c.table[b, p // page], :, p % page] = 0x7F
    devs = [c.device(), c.device()]
    cu, tab, f = i32([0, 1, 2, 3]), c.tab(), Q.rope_inv_freq(d)[0].cuda()
    qkv = torch.empty(3, (hq + 2 * hk) * d, dtype=BF, device="cuda")
    top = max(start) + 6
    ws = Q.workspace(Q.kv_attn_ws_bytes(3, 3, hq, hk, d, 1, top))
    lens, pos = i32(start), i32([l - 1 for l in start])

    def step(dev, x, out):
        q, k, v = (x[:, a * d:b * d].view(3, b - a, d) for a, b in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
        Q.qat_rope(q, pos, f, q, k=k, k_out=k)
        Q.qat_kv_append(k, v, cu, lens, tab, *dev, max_new=1)
        Q.qat_kv_attn(q, cu, lens, tab, *dev, out, 0.125, max_new=1, max_len=top, ws=ws)

    outs = [torch.empty(3, hq, d, dtype=BF, device="cuda") for _ in range(2)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step(devs[0], qkv, outs[0])
    torch.cuda.current_stream().wait_stream(st)
    for i in range(5):
        x = rand(qkv.shape, 70 + i, BF)
        lens.add_(1)
        pos.add_(1)
        qkv.copy_(x)
        graph.replay()
        step(devs[1], x, outs[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.isfinite(outs[0].float()).all(), i
        for a, b in zip(*devs):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
