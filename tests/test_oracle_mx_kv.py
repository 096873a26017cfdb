"""Pins of the MXFP4 and 8-bit cache oracles, and the argument checks of their calls (CPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv_oracle as KV
from oracle import mx_oracle as MX
from tests.test_isa_hazard import _device_asm, _hipcc, accumulator_hazards
from weight_quantization_aware_amd import _lib as Q

FAKE = 1 << 20


def test_mx_known_block():
    # largest magnitude 7 -> e = 0; ties go to the even code, above 6 saturates
    x = np.zeros((1, 32))
    x[0, :12] = [7, -7, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, 0.26, -5.01]
    codes, scales = MX.quantize(x)
    assert scales.tolist() == [[127]]
    assert MX.values(codes, scales)[0, :12].tolist() == [6, -6, 4, 4, 2, 2, 1, 1, 0, 0, 0.5, -6]
    assert codes[0, 9] == 8                       # the sign of zero is kept
    assert np.array_equal(MX.unpack(MX.pack(codes)), codes)


def test_mx_scale_range():
    x = np.zeros((4, 32))
    x[1, 3] = 2.0 ** -149                         # e clamps at -127
    x[2, 0] = np.inf
    x[3, 0] = 2.0 ** 127 * 1.9
    codes, scales = MX.quantize(x)
    assert scales[:, 0].tolist() == [0, 0, 255, 252]
    assert np.isnan(MX.values(codes, scales)[2]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_mx_values_are_exact_in_the_input_type(dtype):
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    x = bits[torch.isfinite(bits.float())].double().numpy()
    x = np.concatenate([x, np.zeros(-len(x) % 32)]).reshape(-1, 32)
    v = MX.values(*MX.quantize(x))
    assert np.array_equal(torch.from_numpy(v).to(dtype).double().numpy(), v)


def test_e4m3_codes_are_torchs():
    y = np.concatenate([np.linspace(-448, 448, 20001), KV.E4M3[:127], (KV.E4M3[:126] + KV.E4M3[1:127]) / 2,
                        np.geomspace(1e-5, 448, 5000)])
    want = torch.from_numpy(y).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    y = torch.from_numpy(y).float().double().numpy()
    assert np.array_equal(KV.e4m3(y), want)
    assert np.array_equal(KV.E4M3[want], torch.from_numpy(want).view(torch.float8_e4m3fn).double().numpy())


def test_scale_exponent_never_saturates():
    for a in (448.0, 448.001, 449.0, 1.0, 1.75, 1.7501, 0.0, 2.0 ** -140, 3.3e38):
        e = KV.scale_exp(a)
        assert 448 * 2.0 ** e >= a and (e == -126 or 448 * 2.0 ** (e - 1) < a)


def test_append_rescales_earlier_tokens():
    codes, scale = np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1), np.float32)
    x = np.full((1, 1, 64), 1.0)
    KV.append(x, [0, 1], [1], np.array([[0]]), codes, scale)
    assert scale[0, 0] == 2.0 ** -8 and (KV.E4M3[codes[0, 0, 0]] == 256).all()
    KV.append(x * 100, [0, 1], [2], np.array([[0]]), codes, scale)
    # 100 / 2^-2 = 400 lies halfway between 384 and 416; 384 has the even code
    assert scale[0, 0] == 2.0 ** -2 and (KV.E4M3[codes[0, 0, 0]] == 4).all() and (KV.E4M3[codes[0, 0, 1]] == 384).all()


@pytest.mark.parametrize("kw", [{}, {"scaling": "linear", "factor": 4.0},
                                {"scaling": "parts", "factor": 8.0, "original": 4096},
                                {"scaling": "parts", "factor": 32.0, "original": 2048, "beta_fast": 16.0,
                                 "beta_slow": 2.0, "base": 500000.0}])
@pytest.mark.parametrize("rot", [32, 96, 128])
def test_rope_inv_freq(rot, kw):
    f, m = Q.rope_inv_freq(rot, **kw)
    g, n = KV.inv_freq(rot, **kw)
    assert f.shape == (rot // 2,)
    # pow and log of the host library against numpy's: a few units of 2^-53, then one rounding to fp32
    assert np.all(np.abs(f.numpy() - g) <= g * (2.0 ** -24 + 2.0 ** -48)) and abs(m - n) <= 2.0 ** -24 * n
    if kw.get("scaling") == "parts":
        plain = KV.inv_freq(rot, kw.get("base", 10000.0))[0]
        assert f[0] == np.float32(plain[0])                      # the fastest pair keeps its angle
        assert abs(f[-1] * kw["factor"] / plain[-1] - 1) < 1e-6  # the slowest is interpolated


@pytest.mark.parametrize("args,status", [
    ((63, 10000.0, 0, 1.0, 1, 32.0, 1.0), 2), ((64, 1.0, 0, 1.0, 1, 32.0, 1.0), 2),
    ((64, 10000.0, 3, 1.0, 1, 32.0, 1.0), 11), ((64, 10000.0, 1, 0.5, 1, 32.0, 1.0), 2),
    ((64, 10000.0, 2, 2.0, 0, 32.0, 1.0), 2), ((64, 10000.0, 2, 2.0, 4096, 1.0, 32.0), 2),
    ((64, float("nan"), 0, 1.0, 1, 32.0, 1.0), 2),
])
def test_rope_inv_freq_refusals(args, status):
    f, m = (ctypes.c_float * 64)(), ctypes.c_float()
    assert Q.lib().qat_rope_inv_freq(*args, ctypes.addressof(f), ctypes.addressof(m)) == status
    assert Q.lib().qat_rope_inv_freq(64, 1e4, 0, 1.0, 1, 32.0, 1.0, None, ctypes.addressof(m)) == 1


def refused(name, good, changes):
    """Every change of the valid argument list is refused with its status before a device is touched."""
    fn = getattr(Q.lib(), name)
    for at, value, status in changes:
        args = list(good)
        for i, v in zip(at if isinstance(at, tuple) else (at,), value if isinstance(at, tuple) else (value,)):
            args[i] = v
        assert fn(*args) == status, (at, value)


M1 = 1 << 24      # addresses far enough apart for the sizes below


def test_mx_quant_refusals():
    #       X    type rows cols ldx codes      scales     X_hat     stream
    good = (FAKE, 1, 4, 64, 64, FAKE + M1, FAKE + 2 * M1, FAKE + 3 * M1, None)
    refused("qat_mx_quant", good, [
        (1, 3, 11), (1, -1, 11), (2, -1, 2), (3, 48, 2), (3, 0, 2), (4, 56, 2), (4, 68, 5), (0, None, 1),
        (5, None, 1), (6, None, 1), ((5, 6, 7), (None, None, None), 1), (0, FAKE + 8, 5), (5, FAKE + M1 + 4, 5),
        (7, FAKE, 8), (5, FAKE + 16, 8), (6, FAKE + M1 + 16, 8), (2, 1 << 30, 2)])
    assert Q.lib().qat_mx_quant(None, 1, 0, 64, 64, None, None, None, None) == 0


def test_mx_product_refusals():
    good = (FAKE, FAKE + M1, FAKE + 2 * M1, FAKE + 3 * M1, 4, 40, 64, 1, FAKE + 4 * M1, 40, None, 0, None)
    refused("qat_mx_gemm", good, [
        (7, 0, 11), (7, 3, 11), (4, -1, 2), (5, 0, 2), (6, 48, 2), (9, 39, 2), (0, None, 1), (1, None, 1),
        (2, None, 1), (3, None, 1), (8, None, 1), (3, FAKE + 3 * M1 + 1, 5), (8, FAKE, 8), (8, FAKE + 3 * M1, 8),
        (4, 1 << 29, 2), (5, 1 << 30, 2)])
    assert Q.lib().qat_mx_gemm(None, None, None, None, 0, 40, 64, 1, None, 40, None, 0, None) == 0
    M = 40
    need = Q.mx_ws_bytes(M, 48, 64)
    good = (FAKE, 64, FAKE + M1, FAKE + 2 * M1, M, 48, 64, 1, FAKE + 3 * M1, 48, FAKE + 4 * M1, need, None)
    refused("qat_mx_linear", good, [
        (7, 0, 11), (1, 32, 2), (1, 68, 5), (0, None, 1), (2, None, 1), (3, None, 1), (8, None, 1), (10, None, 6),
        (11, need - 1, 6), (10, FAKE, 8), (8, FAKE, 8), (10, FAKE + 3 * M1, 8), (10, FAKE + 4 * M1 + 8, 5),
        (6, 72, 2)])
    assert Q.mx_ws_bytes(4, 40, 48) == 0 and Q.mx_ws_bytes(-1, 40, 64) == 0


def test_rope_refusals():
    # q k pos inv tokens hq hk d rot half inverse mscale dtype ldq ldk q_out ldqo k_out ldko stream
    good = (FAKE, FAKE + M1, FAKE + 2 * M1, FAKE + 3 * M1, 4, 8, 2, 128, 64, 1, 0, 1.0, 1, 1024, 256, FAKE + 4 * M1,
            1024, FAKE + 5 * M1, 256, None)
    refused("qat_rope", good, [
        (12, 0, 11), (9, 2, 11), (10, -1, 11), (7, 96, 2), (8, 24, 2), (8, 144, 2), (8, 0, 2), (5, 0, 2), (6, -1, 2),
        (13, 1016, 2), (13, 1028, 5), (16, 512, 2), (18, 128, 2), (0, None, 1), (1, None, 1), (2, None, 1),
        (3, None, 1), (15, None, 1), (17, None, 1), (6, 0, 1), (0, FAKE + 8, 5), (2, FAKE + 2 * M1 + 2, 5),
        (15, FAKE + 128, 8),              # q_out inside q, not q itself
        (15, FAKE + M1, 8), (17, FAKE + 4 * M1, 8), (15, FAKE + 2 * M1, 8), (17, FAKE + 3 * M1, 8)])
    # heads of one packed projection may interleave; the same with overlapping heads may not
    ld = 1024 + 256
    args = list(good)
    args[0] = args[15] = FAKE
    args[1] = args[17] = FAKE + 2048 - 256
    args[13] = args[14] = args[16] = args[18] = ld
    assert Q.lib().qat_rope(*args) == 8
    assert Q.lib().qat_rope(*(list(good[:4]) + [0] + list(good[5:]))) == 0


def test_kv_append_refusals():
    # k v dtype ldk ldv cu lens table cols tokens batch heads d page n_pages max_new kc vc ks vs stream
    P = [FAKE + i * M1 for i in range(10)]
    good = (P[0], P[1], 1, 256, 256, P[2], P[3], P[4], 8, 4, 2, 2, 128, 64, 16, 4, P[5], P[6], P[7], P[8], None)
    refused("qat_kv_append", good, [
        (2, 0, 11), (2, 3, 11), (3, 128, 2), (3, 260, 5), (4, 260, 5), (8, 0, 2), (9, -1, 2), (10, -1, 2),
        (10, 70000, 2), (11, 0, 2), (12, 96, 2), (13, 48, 2), (13, 256, 2), (14, 0, 2), (15, -1, 2),
        *[(i, None, 1) for i in (0, 1, 5, 6, 7, 16, 17, 18, 19)], (0, P[0] + 8, 5), (16, P[5] + 4, 5),
        (18, P[7] + 2, 5), (17, P[5], 8), (16, P[0], 8), (18, P[4], 8)])
    assert Q.lib().qat_kv_append(*(list(good[:9]) + [0] + list(good[10:]))) == 0


def test_kv_attn_refusals():
    # q dtype ldq cu lens table cols tokens batch hq hk d page n_pages kc vc ks vs scale causal max_new max_len out ldo
    P = [FAKE + i * M1 for i in range(12)]
    need = Q.kv_attn_ws_bytes(4, 2, 8, 2, 128, 4, 4096)
    assert need > 0
    good = (P[0], 1, 1024, P[1], P[2], P[3], 64, 4, 2, 8, 2, 128, 64, 16, P[4], P[5], P[6], P[7], 0.1, 1, 4, 4096, P[8],
            1024, P[9], need, None)
    refused("qat_kv_attn", good, [
        (1, 0, 11), (2, 1000, 2), (2, 1028, 5), (6, 0, 2), (9, 7, 2), (9, 0, 2), (10, 0, 2), (11, 32, 2), (12, 8, 2),
        (13, 0, 2), (18, 0.0, 2), (18, float("nan"), 2), (18, float("inf"), 2), (19, 2, 11), (20, -1, 2), (21, -1, 2),
        (23, 1020, 2), (23, 1028, 5), *[(i, None, 1) for i in (0, 3, 4, 5, 14, 15, 16, 17, 22)], (24, None, 6),
        (25, need - 1, 6), (22, P[0], 8), (22, P[4], 8), (24, P[8], 8), (24, P[5], 8), (24, P[9] + 4, 5)])
    assert Q.lib().qat_kv_attn(*(list(good[:7]) + [0] + list(good[8:]))) == 0
    assert Q.kv_attn_ws_bytes(4, 2, 7, 2, 128, 4, 4096) == 0 and Q.kv_attn_ws_bytes(4, 2, 8, 2, 96, 4, 4096) == 0


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        Q.qat_mx_quant(x, c, s)
    with pytest.raises(ValueError, match="multiple of 32"):
        Q.qat_mx_quant(x[:, :40].contiguous(), c, s)
    with pytest.raises(ValueError, match="shape"):
        Q.qat_mx_quant(x, c[:3], s)
    with pytest.raises(TypeError):
        Q.qat_mx_quant(x.double(), c, s)
    with pytest.raises(ValueError, match="behind its first dimension"):
        Q.qat_mx_quant(torch.zeros(64, 4, dtype=torch.bfloat16).t(), c, s)
    with pytest.raises(ValueError, match="overlap"):
        Q.qat_mx_quant(x[:1].expand(4, 64), c, s)
    y = torch.zeros(4, 8, dtype=torch.bfloat16)
    w, ws = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    with pytest.raises(TypeError):
        Q.qat_mx_linear(x, w, ws, y.half())
    with pytest.raises(ValueError, match="shape"):
        Q.qat_mx_gemm(c, s, w, ws[:, :1], y)
    q = torch.zeros(4, 2, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        Q.qat_rope(q, torch.zeros(4, dtype=torch.int64), torch.zeros(32), q)
    with pytest.raises(ValueError):
        Q.qat_rope(q, torch.zeros(4, dtype=torch.int32), torch.zeros(32), q, k=q)
    cache = (torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.zeros(3, 2, 64, 16, dtype=torch.uint8),
             torch.zeros(3, 2), torch.zeros(3, 2))
    meta = (torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        Q.qat_kv_append(q, q, *meta, *cache)
    with pytest.raises(ValueError, match="v_cache must have shape"):
        Q.qat_kv_append(q, q, *meta, cache[0], cache[0], *cache[2:])
    with pytest.raises(ValueError, match="cu must have shape"):
        Q.qat_kv_attn(q, meta[0][:1], *meta[1:], *cache, q, 0.1)


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not available")
def test_mx_tiles_wait_before_reading_accumulators():
    # the tiled product issues its MFMAs from inline asm, like the bf16 GEMM
    asm = _device_asm("qat_mx.hip")
    assert asm.count("k_mx_tile") and asm.count("v_mfma_scale_f32_16x16x128_f8f6f4 a[") > 500
    assert not accumulator_hazards(asm)
