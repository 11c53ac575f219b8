"""Paged attention on values that stretch its arithmetic, against 64 bits."""

import math

import numpy as np
import pytest
import torch

import decode_attention_04_gb300 as fd
import paged_ref as ref
from test_paged_gpu import BF16, E4M3, d

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("B", [1, 310])
@pytest.mark.parametrize("n,sink", [(32768, 0), (32768, 16300), (5001, 4999)])
@pytest.mark.parametrize("bits", [18, 22.5, 26])
@pytest.mark.parametrize("kv,HS,G", [(BF16, 64, 4), (BF16, 512, 16), (E4M3, 64, 4), (E4M3, 128, 8), (E4M3, 256, 16),
                                     (E4M3, 512, 5), (E4M3, 512, 16)])
def test_small_weights_behind_a_large_one(kv, HS, G, bits, n, sink, B):
    """One position has 2^bits times the weight of each of the others, and V = 0: the output is the sum of the small ones.
    310 sequences (of the same pages) put whole bands into one share, one sequence is cut into many.

    Bound: a score is one product, and its way to the weight has at most six roundings of a number below 32 (the two factors
    of the multiplier, the product, the reference, the difference) and exp2's two last places: 6 * 2^5 * 2^-24 * ln 2 + 2^-22
    < 2^-16 of the weight; six terms hold a weight to 2^-24 of itself or 2^-32 of the largest (2^-30 where terms share a
    column: head dim 512, more than 8 rows; bf16 has no such floor), two bf16 terms to 2^-16;
    the sums of n products, 32 an addition, are off by at most 2^-23 an addition."""
    P = 64
    N = -(-n // P)
    gen = torch.Generator().manual_seed(n)
    v = (0.5 + 0.25 * torch.randn(N, 1, P, HS, generator=gen)).clamp(0, 2)
    k = torch.zeros(N, 1, P, HS)
    v[sink // P, 0, sink % P] = 0
    gap = bits * math.log(2)
    ks = vs = None
    if kv == BF16:
        k[sink // P, 0, sink % P, 0] = gap
        k, v = k.bfloat16(), v.bfloat16()
        top, values = float(k[sink // P, 0, sink % P, 0]), v.double()
    else:
        k[sink // P, 0, sink % P, 0] = 256
        k, v = (x.to(torch.float8_e4m3fn) for x in (k, v))
        ks, vs = torch.ones(N, 1), torch.ones(N, 1)
        ks[sink // P] = gap / 256
        top, values = 256 * float(ks[sink // P, 0]), v.double()
        k, v = k.view(torch.uint8), v.view(torch.uint8)
    flat = values.reshape(-1, HS)[:n]
    part = 1 - torch.arange(G) / 128.0  # each row's share of the gap
    q = torch.zeros(B, G, HS)
    q[:, :, 0] = part
    q = q.bfloat16()
    table = np.tile(np.arange(N, dtype=np.int32), (B, 1))
    plan = fd.fd_paged_plan(B, G, 1, HS, P, N, 0, kv_dtype=kv)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    out = torch.empty(B, G, HS, dtype=torch.bfloat16, device=DEV)
    out32 = torch.empty(B, G, HS, device=DEV)
    fd.fd_get_device_error()
    fd.fd_paged_attn_ex(plan, ws, plan.workspace_bytes, out32, d(q), d(k), d(v), d(ks), d(vs), out, d(table),
                        torch.full((B,), n, dtype=torch.int32, device=DEV), B, G, 1, HS, P, N, N, 0, 1.0)
    assert fd.fd_get_device_error() == 0
    w = torch.exp(-part.double() * top)[:, None]
    want = w * flat.sum(0) / (1 + (n - 1) * w)
    floor = 0.0 if kv == BF16 else 2.0 ** -30 if HS == 512 and G > 8 else 2.0 ** -32
    rel = 2.0 ** -16 + (n / 32 + 64) * 2.0 ** -23 + (2.0 ** -16 if kv == BF16 else 2.0 ** -24)
    lim = rel * want + n * floor * flat.max()
    err = (out32.double().cpu() - want).abs()
    assert (err <= lim).all(), f"{(err / lim).max():.2f} of the bound, {(err / want).max():.2e} of the output"
    assert ((out.double().cpu() - want).abs() <= lim + want * 2.0 ** -8).all()
