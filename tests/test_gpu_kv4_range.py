"""The range of the attention's weights over the 4-bit cache (fastar_kv4_attn): weak keys under a strong one,
and logits so large that fp32 counts them in twos."""
import math

import numpy as np
import pytest
import torch

import test_gpu_kv4 as T
from kv_cache_tempcache_gb300 import _lib as L
from oracle import kv4_oracle as K

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _run(q, c, n, scale, with_ws):
    H, nq, d = q.shape
    nb = L.workspace_bytes(L.OP_KV4_ATTN, H, nq, c[0].shape[1], d, 1) if with_ws else 0
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV) if nb else None
    out, lse, status = torch.empty_like(q), torch.empty(H, nq, device=DEV), T._i32([0])
    L.fastar_kv4_attn(q, *c, T._i32([n]), scale, out, lse, dev_status=status, workspace=ws)
    torch.cuda.synchronize()
    assert status.item() == 0
    return out, lse


@pytest.mark.parametrize("dtype,G,nq,d", [("bf16", 1, 1, 128), ("bf16", 4, 3, 64), ("bf16", 1, 40, 128),
                                          ("bf16", 1, 129, 64), ("bf16", 1, 300, 128), ("f32", 1, 3, 128)])
def test_weak_keys_under_a_strong_one(dtype, G, nq, d):
    """The strong keys' V are 0, so the output is nothing but weak keys, 16 to 19 nats below.

    The bound is test_gpu_kv4's but for one term, what small weights lose for good: a bf16 call's weights are
    fp16 numbers on a scale on which the row's largest was at least 2^10 when the scale was set, so a
    weight below 2^-14 is off by half the spacing of fp16's subnormals, 2^-25, over a sum of at least
    2^10: 2^-35 sum_j |v_j|.  (fp32: 2^-38, as there.)  For 39,984 weak keys that is 1.2e-6, of an
    output of 39,984 e^-19 / 16 = 1.4e-5 at the least.  A weight of 2^-25 or less on a scale of the
    largest itself would be 0, and the output with it."""
    n = 40000
    x = torch.zeros(2, 1, n, d, device=DEV)
    x[1] = 1.0
    strong = torch.arange(0, 512, 32, device=DEV)             # one in each of the first blocks of 32 keys
    x[0, 0, strong, 0], x[1, 0, strong] = 6.0, 0.0            # their logit is 6 q_0 scale, the others' 0
    c = T._empty_cache(1, n, d)
    L.fastar_kv4_append(x[0].bfloat16(), x[1].bfloat16(), *c)
    kv, vv = [K.values(c[2 * i].cpu().numpy(), c[2 * i + 1].cpu().numpy()) for i in range(2)]
    scale = 0.125
    q = torch.zeros(G * nq, d, device=DEV)
    q[:, 0] = (16 + torch.arange(G * nq, device=DEV) % 7 * 0.5) / (6 * scale)
    q = q.view(G, nq, d).to(T.DT[dtype])
    want, wl, A, E = K.attention(T._np(q), kv, vv, [n], scale)
    e = (d * 2.0 ** -23 + 2.0 ** -22) * E + 2.0 ** -22
    bf16 = dtype == "bf16"
    tol = (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(want)
    tol += A * (4 * e + n * 2.0 ** -22 + (2.0 ** -11 if bf16 else 0))[..., None]
    tol += np.abs(vv[0]).sum(0) * (2.0 ** -35 if bf16 else 2.0 ** -38)
    for with_ws in (False, True):
        out, lse = _run(q, c, n, scale, with_ws)
        ratio = np.abs(T._np(out) - want) / tol
        assert (ratio <= 1).all(), f"worst {ratio.max():.2f} of the bound"
        assert (np.abs(T._np(lse) - wl) <= 2 * e + n * 2.0 ** -22 + 2.0 ** -22 * (1 + np.abs(wl))).all()


@pytest.mark.parametrize("dtype,nq,d", [("f32", 2, 128), ("bf16", 2, 64), ("bf16", 12, 128), ("bf16", 40, 128),
                                        ("bf16", 300, 64)])
def test_logits_that_fp32_counts_in_twos(dtype, nq, d):
    """Half the keys' logits, in units of log 2, are some 2^24, where fp32's numbers lie 2 apart; the other half,
    1024 rows later, are j 4/3 scale' above.  Dot products are exact here (24576 and 24576 + j 2^-9), so the
    weights are w = 2^(the difference) to 1, and the output (6 w - 3) / (w + 1): off by its own
    rounding, fp16's of the weights (2^-11, two of them: the quotient's), and 2^-16 for the
    exponentials' arguments, a 2^-24th of at most 2^7, times 9, the distance of the values.  Whether
    a weight passes fp16's end must not be decided by numbers that are rounded to twos."""
    n = 2048
    x = torch.zeros(2, 1, n, d, device=DEV)
    x[0, 0, :, 0] = 6.0
    x[0, 0, :, 17] = 6.0                                       # q is 0 there; it makes the block's scale 1
    x[0, 0, n // 2:, 16] = 1.0
    x[1, 0, :n // 2], x[1, 0, n // 2:] = -3.0, 6.0
    c = T._empty_cache(1, n, d)
    L.fastar_kv4_append(x[0].bfloat16(), x[1].bfloat16(), *c)
    kv = K.values(c[0].cpu().numpy(), c[1].cpu().numpy())
    assert np.array_equal(kv, T._np(x[0]))          # stored exactly
    q = torch.zeros(1, nq, d, device=DEV)
    q[..., 0] = 4096.0
    for up in (1.0625, 1.3, 1.9):
        for first in (1, 9):
            j = first + torch.arange(nq, device=DEV) % 8
            q[..., 16] = j * 2.0 ** -9
            scale = float(np.float32(up * 2.0 ** 24 / 24576 * math.log(2.0)))
            out, _ = _run(q.to(T.DT[dtype]), c, n, scale, False)
            w = 2.0 ** (j.cpu().double().numpy() * 2.0 ** -9 * scale / math.log(2.0))
            want = ((6 * w - 3) / (w + 1))[None, :, None]
            half, p = (2.0 ** -8, 2.0 ** -11) if dtype == "bf16" else (2.0 ** -24, 2.0 ** -22)
            got = T._np(out)
            assert np.isfinite(got).all(), (up, first)
            assert (np.abs(got - want) <= half * np.abs(want) + 9 * (2 * p + 2.0 ** -16)).all(), (up, first)
