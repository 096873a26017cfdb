"""The serving operators together, as one attention half of a served decoder block uses them: MXFP4 projection to
q, k, v; rotary positions in place; append to the 8-bit cache; attention; MXFP4 projection back. A ragged prompt and
then single tokens; every step is checked against the fp64 oracle on that step's own inputs."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as KV
from oracle import mx_oracle as MX
from weight_quantization_aware_amd import _lib as Q
from tests.test_gpu_kv import Cache, check_append, check_attn, check_rope, i32
from tests.test_gpu_mx import check_y, host, operand, quant

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_and_decode(dtype):
    H, hq, hk, d, page = 512, 8, 2, 64, 32
    wc, ws, wv = operand((hq + 2 * hk) * d, H, 1, 118, 122)
    oc, os_, ov = operand(H, hq * d, 2, 118, 122)
    f, ms = Q.rope_inv_freq(d, scaling="linear", factor=2.0)
    c = Cache([90, 60, 33], hk, d, page)
    dev = c.device()
    lens = [0, 0, 0]
    g = torch.Generator("cuda").manual_seed(0)
    for new in ([80, 37, 0], [1, 1, 1], [1, 1, 0], [3, 2, 1], [1, 1, 1]):
        lens = [a + b for a, b in zip(lens, new)]
        cu = [0, *np.cumsum(new).tolist()]
        T = cu[-1]
        pos = np.concatenate([np.arange(l - n, l) for l, n in zip(lens, new)])
        x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
        qkv = torch.empty(T, (hq + 2 * hk) * d, dtype=dtype, device="cuda")
        work = Q.workspace(max(Q.mx_ws_bytes(T, qkv.shape[1], H), Q.mx_ws_bytes(T, H, hq * d)))
        Q.qat_mx_linear(x, wc, ws, qkv, ws=work)
        check_y(qkv, host(quant(x)[2]), wv)
        q, k, v = (qkv[:, a * d:b * d].view(T, b - a, d) for a, b in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
        q0, k0 = q.clone(), k.clone()
        Q.qat_rope(q, i32(pos.tolist()), f.cuda(), q, k=k, k_out=k, mscale=ms)
        check_rope(q0, q, pos, f, True, ms, False)
        check_rope(k0, k, pos, f, True, ms, False)
        check_append(c, k, v, cu, lens, dev, max_new=max(new))
        o, _, _ = check_attn(c, q, cu, lens, d ** -0.5, True, dev=dev)
        y = torch.empty(T, H, dtype=dtype, device="cuda")
        Q.qat_mx_linear(o.view(T, hq * d), oc, os_, y, ws=work)
        check_y(y, host(quant(o.view(T, hq * d))[2]), ov)
