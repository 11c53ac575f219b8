"""Paged attention on values that stretch its arithmetic, against 64 bits."""

import math

import numpy as np
import pytest
import torch

import decode_attention_04_gb300 as fd
import paged_ref as ref
from test_paged_gpu import BF16, E4M3, _values, d, make_pool, make_table, run_attn

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
    column: head dim 512, more than 8 rows; bf16 has no such floor), three bf16 terms to 2^-24;
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
    rel = 2.0 ** -16 + (n / 32 + 64) * 2.0 ** -23 + 2.0 ** -24
    lim = rel * want + n * floor * flat.max()
    err = (out32.double().cpu() - want).abs()
    assert (err <= lim).all(), f"{(err / lim).max():.2f} of the bound, {(err / want).max():.2e} of the output"
    assert ((out.double().cpu() - want).abs() <= lim + want * 2.0 ** -8).all()


@pytest.mark.parametrize("kv,HS,G", [(BF16, 64, 3), (BF16, 128, 8), (BF16, 512, 16), (E4M3, 64, 3), (E4M3, 128, 8),
                                     (E4M3, 256, 16), (E4M3, 512, 16)])
def test_weights_hold_24_bits(kv, HS, G):
    """Two positions whose values are 0 and 1: the fp32 output is the second's weight over their sum.

    Bound, relative to the output: a score is one product of at most 2 in size in powers of two, with at most six roundings on
    its way to the weight (6 * 2 * 2^-24 * ln 2 = 2^-20.9) and exp2's two last places (2^-22); three roundings (the weight's terms,
    the sum, the quotient) of 2^-24. Together below 2^-20; both weights take part, so twice that."""
    P, B = 16, 40
    k, v = torch.zeros(1, 1, P, HS), torch.zeros(1, 1, P, HS)
    k[0, 0, 1, 0], v[0, 0, 1] = 1.0, 1.0
    ks = vs = None
    if kv == E4M3:
        k, v = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
        ks, vs = torch.ones(1, 1), torch.ones(1, 1)
    else:
        k, v = k.bfloat16(), v.bfloat16()
    q = torch.zeros(B, G, HS)
    q[:, :, 0] = 2 * torch.rand(B, G, generator=torch.Generator().manual_seed(HS + G)) - 1
    q = q.bfloat16()
    _, out32, err = run_attn(kv, q, k, ks, v, vs, np.zeros((B, 1), dtype=np.int32), [2] * B, 0, 1.0)
    assert err == 0
    w = torch.exp(q[:, :, :1].double())
    want = w / (1 + w)
    off = ((out32.double() - want) / want).abs().max().item()
    assert off <= 2.0 ** -19, f"2^{math.log2(off):.1f}"


@pytest.mark.parametrize("kv,HS,G", [(BF16, 128, 4), (E4M3, 64, 3), (E4M3, 128, 8), (E4M3, 128, 16), (E4M3, 256, 12),
                                     (E4M3, 512, 8), (E4M3, 512, 16)])
def test_small_elements_of_q_beside_a_large_one(kv, HS, G):
    """A query row whose largest element meets zeros in K; the others, 2^-13.3 of it, make the score, 2 at the second of two
    positions, whose values are 0 and 1.

    Bound, relative to the output: that of test_weights_hold_24_bits; the score's sum, 2 HS 2^-23; with two terms of q (head dim
    512, more than 8 rows) 2 * 2^-21 of the largest element over the others."""
    P, B, top, small = 16, 3, 128.0, 201 * 2.0 ** -14
    k, v = torch.zeros(1, 1, P, HS), torch.zeros(1, 1, P, HS)
    k[0, 0, 1, 1:], v[0, 0, 1] = 64.0, 1.0
    want_k = 2 / (small * (HS - 1))
    ks = vs = None
    if kv == E4M3:
        k, v = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
        ks, vs = torch.full((1, 1), want_k / 64), torch.ones(1, 1)
        each = 64 * float(ks)
    else:
        k[0, 0, 1, 1:] = want_k
        k, v = k.bfloat16(), v.bfloat16()
        each = float(k[0, 0, 1, 1])
    q = torch.full((B, G, HS), small)
    q[:, :, 0] = top
    q = q.bfloat16()
    assert float(q[0, 0, 1]) == small
    _, out32, err = run_attn(kv, q, k, ks, v, vs, np.zeros((B, 1), dtype=np.int32), [2] * B, 0, 1.0)
    assert err == 0
    want = 1 / (1 + math.exp(-small * each * (HS - 1)))
    rel = 2.0 ** -19 + 2 * HS * 2.0 ** -23 + (2 * 2.0 ** -21 * top / small if kv == E4M3 and HS == 512 and G > 8 else 0.0)
    off = ((out32.double() - want) / want).abs().max().item()
    assert off <= rel, f"2^{math.log2(off):.1f} against 2^{math.log2(rel):.1f}"


@pytest.mark.parametrize("HS,G", [(64, 4), (128, 8), (512, 16)])
@pytest.mark.parametrize("n,at", [(300, 280), (9000, 8990)])
def test_largest_values_behind_a_lagging_reference(HS, G, n, at):
    """bf16: a value of the type's largest size at a position whose score lies 7.2 powers of two above those of the group's tiles
    before it, too few to move the reference; the other values are 0. The output is its part of the softmax, which is finite.
    320 sequences of the same pages, so that most bands lie in one share.
    Bound: that of test_weights_hold_24_bits, for a score of 7.2 instead of 2, and the sum of n weights."""
    P, B = 16, 320
    N = -(-n // P)
    k, v = torch.zeros(N, 1, P, HS), torch.zeros(N, 1, P, HS)
    top = torch.finfo(torch.bfloat16).max
    k[at // P, 0, at % P, 0], v[at // P, 0, at % P] = 5.0, top
    q = torch.zeros(B, G, HS)
    q[:, :, 0] = 1
    out16, out32, err = run_attn(BF16, q.bfloat16(), k.bfloat16(), None, v.bfloat16(), None,
                                 np.tile(np.arange(N, dtype=np.int32), (B, 1)), [n] * B, 0, 1.0)
    assert err == 0
    want = math.exp(5) / (math.exp(5) + n - 1) * float(torch.tensor(top).bfloat16())
    off = (out32.double() / want - 1).abs().max().item()
    assert off <= 2.0 ** -17 + (n / 128 + 64) * 2.0 ** -24, f"{off}"
    assert torch.isfinite(out16).all()


def check(kv, q, k, ks, v, vs, table, lens, out16, out32, e2, window=0):
    """Against the 64-bit reference; e2 bounds what the weights and the sums lose, relative to the largest value of the row.
    Below 2^-126 fp32 and bf16 round to multiples of their least values, by at most 2^-150 and 2^-134: fp32 once where a share's
    mean is made and twice for each share that is merged (the product with its factor is added to a sum, sums are added), and a
    share has 64 KB of K and V at least."""
    HS = q.shape[2]
    kr, vr = (k.double().numpy(), v.double().numpy()) if kv == BF16 else (k.numpy(), v.numpy())
    want, big, mass = ref.attend(q.double().numpy(), kr, vr, None if ks is None else ks.numpy(),
                                 None if vs is None else vs.numpy(), table, lens, window, HS ** -0.5, k.shape[0])
    shares = max(lens) * HS * (2 if kv == BF16 else 1) // 32768 + 2
    lim = ((4 * HS * 2.0 ** -23 * mass + e2 + 2.0 ** -20) * big)[..., None] + (1 + 2 * shares) * 2.0 ** -150
    got = out32.double().numpy()
    assert np.isfinite(got).all(), f"{(~np.isfinite(got)).sum()} of {got.size} are not finite"
    err = np.abs(got - want)
    assert (err <= lim).all(), f"{(err / lim).max():.2f} of the bound"
    assert (np.abs(out16.double().numpy() - want) <= lim + np.abs(want) * 2.0 ** -8 + 2.0 ** -134).all()
    return want


def lost(n):
    """For n positions: weights are off by 2^-24 of themselves or 2^-30 of the largest weight times the largest scale, which
    counts 2^5 times where the largest code under that scale is 448 / 2^5 (the pools here have larger ones); sums of n
    products, 32 an addition, by 2^-23 an addition."""
    return 2.0 ** -24 + n * 2.0 ** -25 + (n / 32 + 64) * 2.0 ** -23


def spans(n, P):
    """Runs of positions that are zeroed, by what they are to the kernel: its tiles are 128 positions long, taken by two
    groups in turn, and a share begins at any multiple of 32."""
    yield "first tile", (0, 128)
    yield "second tile", (128, 256)
    yield "third tile", (256, 384)
    yield "first two", (0, 256)
    yield "last page", ((n - 1) // P * P, n)
    yield "all but the last page", (0, (n - 1) // P * P)
    yield "a piece", (n // 2 // P * P, n // 2 // P * P + max(P, 32))
    yield "all", (0, n)


@pytest.mark.parametrize("codes", ["zero codes", "codes"])
@pytest.mark.parametrize("level", [-6, 0, 20, -120])
@pytest.mark.parametrize("HS,G,P", [(64, 1, 16), (128, 4, 16), (128, 8, 32), (256, 9, 16), (512, 16, 128), (512, 3, 16)])
def test_blocks_of_v_scale_zero(HS, G, P, level, codes):
    """Blocks whose V scale is zero - what the writer makes of zeros - count in the softmax's sum and add nothing: in any tile
    of a band that lies in one share or in several, beside scales of 2^level."""
    for n in (129, 200, 400, 257 * P // 16 + 2300):
        for what, (lo, hi) in spans(n, P):
            N = -(-n // P) + 1
            k, ks, _ = make_pool(E4M3, N, 2, P, HS, n)
            v, vs, _ = make_pool(E4M3, N, 2, P, HS, n + 1)
            table = make_table([n], P, N, N, n)
            vs = torch.exp2(torch.randint(level, level + 2, vs.shape, generator=torch.Generator().manual_seed(n)).float())
            pages = table[0][lo // P:-(-min(hi, n) // P)]
            vs[pages, 0] = 0.0
            if codes == "zero codes":
                v[pages, 0] = 0
            q = _values((1, 2 * G, HS), 7).bfloat16()
            out16, out32, err = run_attn(E4M3, q, k, ks, v, vs, table, [n], 0)
            assert err == 0
            want = check(E4M3, q, k, ks, v, vs, table, [n], out16, out32, lost(n))
            if what == "all":
                assert (want[0, :G] == 0).all() and (out32[0, :G] == 0).all()


@pytest.mark.parametrize("tiny", [0.0, 2.0 ** -149, 2.0 ** -126, 2.0 ** -124, 2.0 ** -60])
@pytest.mark.parametrize("HS,G,P", [(128, 4, 16), (512, 16, 128)])
def test_one_token_of_a_tiny_v_scale(HS, G, P, tiny):
    """A last token alone in its page and its tile; and the same scale in every block."""
    n = 2 * P + 1 if P == 128 else 129
    N = -(-n // P)
    k, ks, _ = make_pool(E4M3, N, 1, P, HS, 3)
    v, vs, _ = make_pool(E4M3, N, 1, P, HS, 4)
    table = make_table([n], P, N, N, 5)
    q = _values((1, G, HS), 7).bfloat16()
    vs[table[0, -1], 0] = tiny
    out16, out32, err = run_attn(E4M3, q, k, ks, v, vs, table, [n], 0)
    assert err == 0
    check(E4M3, q, k, ks, v, vs, table, [n], out16, out32, lost(n))
    vs[:] = tiny
    out16, out32, err = run_attn(E4M3, q, k, ks, v, vs, table, [n], 0)
    assert err == 0
    check(E4M3, q, k, ks, v, vs, table, [n], out16, out32, lost(n))


@pytest.mark.parametrize("P,HS,G", [(16, 128, 4), (32, 256, 16)])
def test_v_scales_far_apart_in_any_order(P, HS, G):
    """Scales from 2^-126 to 2^110, rising, falling and mixed, in bands of one share and of several."""
    for order in ("rising", "falling", "mixed"):
        for n in (300, 3000):
            N = -(-n // P)
            k, ks, _ = make_pool(E4M3, N, 1, P, HS, 3)
            v, _, _ = make_pool(E4M3, N, 1, P, HS, 4)
            e = torch.linspace(-126, 110, N).round()
            e = e.flip(0) if order == "falling" else e[torch.randperm(N, generator=torch.Generator().manual_seed(n))] if order == "mixed" else e
            table = np.arange(N, dtype=np.int32)[None]
            q = _values((1, G, HS), 7).bfloat16()
            vs = torch.exp2(e)[:, None].contiguous()
            out16, out32, err = run_attn(E4M3, q, k, ks, v, vs, table, [n], 0)
            assert err == 0
            check(E4M3, q, k, ks, v, vs, table, [n], out16, out32, lost(n))


def test_zeros_that_the_writer_stored():
    """A prompt whose first 150 values are zero, written by fd_paged_append and attended to."""
    B, NKV, G, HS, P, n = 1, 2, 4, 128, 16, 400
    N = n // P
    rows = _values((n, 2, NKV, HS), 3).bfloat16()
    rows[:150, 1] = 0
    rows[n - 1, 1, 0] = 0
    k, v = (torch.full((N, NKV, P, HS), ref.NAN_CODE, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((N, NKV), float("nan"), device="cuda") for _ in range(2))
    table, lens = np.arange(N, dtype=np.int32)[None], torch.tensor([n], dtype=torch.int32, device="cuda")
    new = rows.cuda()
    fd.fd_paged_append(new, new[:, 1], k, v, ks, vs, d(table), lens, torch.tensor([0, n], dtype=torch.int32, device="cuda"), None,
                       B, n, NKV, HS, P, N, N, new.stride(0), new.stride(0), E4M3)
    torch.cuda.synchronize()
    assert (vs[:9].cpu() == 0).all()
    q = _values((B, NKV * G, HS), 7).bfloat16()
    k, ks, v, vs = (x.cpu() for x in (k, ks, v, vs))
    out16, out32, err = run_attn(E4M3, q, k, ks, v, vs, table, [n], 0)
    assert err == 0
    check(E4M3, q, k, ks, v, vs, table, [n], out16, out32, lost(n))


@pytest.mark.parametrize("HS,G,NKV,P,window", [(64, 4, 3, 16, 0), (128, 8, 2, 32, 0), (256, 16, 1, 16, 100), (512, 16, 2, 16, 0)])
def test_far_scales_in_many_short_bands(HS, G, NKV, P, window):
    """A batch of short sequences, several bands to a block, whose blocks have scales of their own: a third zero, the others
    from 2^-126 to 2^100. A band's scales have no effect on the next one's."""
    rng = np.random.default_rng(HS)
    lens = [int(x) for x in rng.integers(0, 330, 60)] + [0, 1, P]
    wide = 330 // P + 1
    N = sum(-(-n // P) for n in lens) + 1
    k, ks, _ = make_pool(E4M3, N, NKV, P, HS, 3)
    v, _, _ = make_pool(E4M3, N, NKV, P, HS, 4)
    table = make_table(lens, P, wide, N, 5)
    e = rng.integers(-126, 101, (N, NKV))
    vs = torch.from_numpy(np.where(rng.random((N, NKV)) < 1 / 3, 0.0, np.exp2(e.astype(np.float64)))).float()
    q = _values((len(lens), NKV * G, HS), 7).bfloat16()
    out16, out32, err = run_attn(E4M3, q, k, ks, v, vs, table, lens, window)
    assert err == 0
    check(E4M3, q, k, ks, v, vs, table, lens, out16, out32, lost(330), window)
