"""The paged cache on the GPU, through the public entry points, against the
64-bit reference of paged_ref.py.

Tolerances of the attention, from the arithmetic that fd_paged_attn.h states. With
A = scale * sum_d |q_d k_d| of a score and n the products summed in fp32:
  * a score is off by at most n 2^-23 A (a sum of n terms in fp32, in any order,
    each addition off by at most 2^-23 of the partial sums' bound, which also holds
    where the adder truncates), and a weight by twice that, relatively, as its
    softmax's sum is off as well: e1 = 2 * 2 * HS * 2^-23 * A;
  * E4M3: q enters as E4M3 terms that leave at most 2^-21 of the row's largest element, which for
    the test's values (elements above 2^-13 of the largest are exact) is inside e1;
    a weight leaves at most 2^-24 of itself or 2^-30 of the largest: e2 = 2^-11 is wide for any n below 2^18;
    bf16: 2^-24, and e2 = 2^-16 is wide as well (test_paged_values_gpu.py has the close bounds);
  * the output is a mean of values of at most |V|: |error| <= (e1 + e2 + 2^-20) |V|;
  * the bf16 output adds half a step, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import decode_attention_04_gb300 as fd
import paged_ref as ref
from harness import Guarded

pytestmark = pytest.mark.gpu
BF16, E4M3 = fd.FD_KV_BF16, fd.FD_KV_E4M3
DEV = "cuda"


def _values(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g)


def make_pool(kv, N, NKV, P, HS, seed):
    """One tensor of a pool on the CPU: (bf16 tensor or uint8 codes, scale or None, the form paged_ref takes)."""
    x = _values((N, NKV, P, HS), seed)
    if kv == BF16:
        x = x.bfloat16()
        return x, None, x.double().numpy()
    g = torch.Generator().manual_seed(seed + 1)
    scale = torch.exp2(torch.randint(-9, -3, (N, NKV), generator=g).float()) * (1 + 0.5 * torch.rand(N, NKV, generator=g))
    codes = (x / scale[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scale, codes.numpy().copy()


def make_table(lens, P, wide, N, seed):
    order = np.random.default_rng(seed).permutation(N)
    table, at = np.full((len(lens), wide), -1, dtype=np.int32), 0
    for b, n in enumerate(lens):
        m = min(-(-max(n, 0) // P), wide)
        table[b, :m] = order[at:at + m]
        at += m
    assert at <= N
    return table


def dead_slots_nan(k, v, table, lens, window, P):
    """NaN in every slot that holds no live position."""
    live = np.zeros((k.shape[0], P), dtype=bool)
    for b, n in enumerate(lens):
        for p in range(max(0, n - window) if window > 0 else 0, min(max(n, 0), table.shape[1] * P)):
            if 0 <= table[b][p // P] < k.shape[0]:
                live[table[b][p // P], p % P] = True
    dead = torch.from_numpy(~live)[:, None, :, None].expand(k.shape)
    for x in (k, v):
        x[dead] = float("nan") if x.dtype == torch.bfloat16 else ref.NAN_CODE


def d(x):
    return None if x is None else (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(DEV)


def run_attn(kv, q, k, ks, v, vs, table, lens, window, scale=0.0, edit_plan=None):
    """One fd_paged_attn_ex call with guarded outputs and a workspace of NaN bytes."""
    B, NH, HS = q.shape
    N, NKV, P, _ = k.shape
    wide = table.shape[1]
    plan = fd.fd_paged_plan(B, NH, NKV, HS, P, wide, window, kv_dtype=kv)
    o16, o32 = Guarded(B * NH * HS * 2, DEV, fill=0xFF), Guarded(B * NH * HS * 4, DEV, fill=0xFF)
    ws = Guarded(plan.workspace_bytes, DEV, fill=0xFF)
    t = [d(x) for x in (q, k, v, ks, vs, table, torch.tensor(lens, dtype=torch.int32))]
    fd.fd_get_device_error()
    fd.fd_paged_attn_ex(plan, ws.ptr(), plan.workspace_bytes, o32.ptr(), *t[:5], o16.ptr(), *t[5:], B, NH, NKV, HS, P, N,
                        wide, window, scale)
    torch.cuda.synchronize()
    assert o16.canaries_intact() and o32.canaries_intact() and ws.canaries_intact()
    return (o16.view(torch.bfloat16, (B, NH, HS)).cpu(), o32.view(torch.float32, (B, NH, HS)).cpu(),
            fd.fd_get_device_error())


def check_attn(kv, q, kr, ks, vr, vs, table, lens, window, out16, out32, scale=None, N=None):
    HS = q.shape[2]
    want, big, mass = ref.attend(q.double().numpy(), kr, vr, None if ks is None else ks.numpy(),
                                 None if vs is None else vs.numpy(), table, lens, window, scale or HS ** -0.5,
                                 N or kr.shape[0])
    e1 = 4 * HS * 2.0 ** -23 * mass
    e2 = 2.0 ** -11 if kv == E4M3 else 2.0 ** -16
    lim = ((e1 + e2 + 2.0 ** -20) * big)[..., None]
    got = out32.double().numpy()
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= lim).all(), f"fp32 error {err.max():.3e}, {(err / np.maximum(lim, 1e-30)).max():.2f} of the bound"
    got16 = out16.double().numpy()
    assert (np.abs(got16 - want) <= lim + np.abs(want) * 2.0 ** -8).all()
    return err.max()


def case(kv, HS, NKV, G, P, lens, window=0, seed=0, spare=2, scale=0.0, poison=True):
    wide = max(1, -(-max(max(lens), 1) // P)) + 1
    N = sum(-(-max(n, 0) // P) for n in lens) + spare
    k, ks, _ = make_pool(kv, N, NKV, P, HS, seed)
    v, vs, _ = make_pool(kv, N, NKV, P, HS, seed + 100)
    table = make_table(lens, P, wide, N, seed)
    if window > 0:  # pages outside the band may be gone
        for b, n in enumerate(lens):
            table[b, :max(0, n - window) // P] = -1
    if poison:
        dead_slots_nan(k, v, table, lens, window, P)
    q = _values((len(lens), NKV * G, HS), seed + 7).bfloat16()
    kr = k.double().numpy() if kv == BF16 else k.numpy()
    vr = v.double().numpy() if kv == BF16 else v.numpy()
    out16, out32, err = run_attn(kv, q, k, ks, v, vs, table, lens, window, scale)
    assert err == 0
    check_attn(kv, q, kr, ks, vr, vs, table, lens, window, out16, out32, scale if scale > 0 else None)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("HS", [64, 128, 256, 512])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_attn_every_head_dim_and_page_size(kv, HS, P):
    case(kv, HS, 2, 3, P, [1, 0, P - 1, P, P + 1, 200, 3 * P + 5], seed=HS + P)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("G", list(range(1, 17)))
def test_attn_every_group_size(kv, G):
    case(kv, 128, 2, G, 16, [77, 130], seed=G)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("HS,G", [(64, 16), (256, 9), (512, 16), (512, 1)])
def test_attn_group_and_head_dim_extremes(kv, HS, G):
    case(kv, HS, 1, G, 32, [513, 31], seed=HS + G)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 4095, 4097])
def test_attn_lengths_around_tiles(kv, n):
    case(kv, 64, 1, 4, 16, [n], seed=n)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n,w", [(1, 1), (5, 1), (100, 1), (100, 7), (100, 16), (100, 99), (100, 100), (100, 101), (300, 130),
                                 (1000, 128), (1001, 33), (777, 2 ** 31 - 1)])
def test_attn_windows(kv, n, w):
    case(kv, 128, 2, 2, 16, [n, max(1, n - 3), 0], window=w, seed=n + w % 1000)
    case(kv, 256, 1, 8, 64, [n, 1], window=w, seed=n + w % 1000)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attn_many_short_sequences(kv):
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 90, 300)]
    case(kv, 64, 3, 2, 16, lens, seed=11)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attn_ragged_batch(kv):
    case(kv, 128, 8, 4, 16, [2000, 3, 0, 129, 5000, 1, 640, 31], seed=12)
    case(kv, 512, 1, 16, 64, [3000, 1, 500], seed=13)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attn_explicit_scale_and_peaked_scores(kv):
    case(kv, 128, 2, 4, 32, [300, 40], seed=14, scale=0.9)
    case(kv, 64, 2, 4, 32, [700, 40], seed=15, scale=0.001)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attn_one_position_gives_its_value(kv):
    """A single live position has weight 1 (bf16: up to one division's rounding). E4M3: the product with V's codes takes the
    weight 2^(t - m), t = s + log2(vs), exactly, and the row's sum takes 2^(s - m) = 1 / vs, so the scale passes through
    an exponent. With |log2 vs| <= 9 and |t| < 32 that exponent is off by at most 2^-20 (log2's last place, [8, 16)) +
    2^-20 (half a last place of t) + 2^-21 (of s - m); times ln 2, with two last places of exp2 (2^-22) and the
    division's half: 1.74 * 2^-20 + 2^-22 + 2^-24 < 2^-18."""
    P, N = 16, 3
    k, ks, _ = make_pool(kv, N, 2, P, 128, 3)
    v, vs, vr = make_pool(kv, N, 2, P, 128, 4)
    table = np.array([[2], [0]], dtype=np.int32)
    q = _values((2, 8, 128), 5).bfloat16()
    out16, out32, err = run_attn(kv, q, k, ks, v, vs, table, [1, 1], 0)
    assert err == 0
    for b, page in ((0, 2), (1, 0)):
        for h in range(8):
            want = vr[page, h // 4, 0] if kv == BF16 else ref.TABLE[vr[page, h // 4, 0]] * float(vs[page, h // 4])
            rtol = 2.0 ** -22 if kv == BF16 else 2.0 ** -18
            assert np.allclose(out32[b, h].double().numpy(), want, rtol=rtol, atol=0)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attn_extreme_scales_and_magnitudes(kv):
    """Blocks whose scales differ by 2^20 and query rows by 2^40."""
    P, N, HS = 32, 8, 128
    k, ks, _ = make_pool(kv, N, 1, P, HS, 6)
    v, vs, _ = make_pool(kv, N, 1, P, HS, 7)
    q = _values((1, 4, HS), 8)
    q = (q * torch.tensor([1.0, 2.0 ** -20, 2.0 ** -30, 3.0])[None, :, None]).bfloat16()
    if kv == E4M3:
        vs = vs * torch.exp2(torch.arange(N).float() * 3 - 12)[:, None]
    else:
        v = (v.float() * torch.exp2(torch.arange(N).float() * 3 - 12)[:, None, None, None]).bfloat16()
    table, lens = np.arange(N, dtype=np.int32)[None], [N * P - 3]
    o16, o32, err = run_attn(kv, q, k, ks, v, vs, table, lens, 0)
    assert err == 0
    kr, vr = (k.double().numpy(), v.double().numpy()) if kv == BF16 else (k.numpy(), v.numpy())
    check_attn(kv, q, kr, ks, vr, vs, table, lens, 0, o16, o32)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attn_nan_inside_the_band_reaches_only_its_group(kv):
    P, N = 16, 5
    k, ks, _ = make_pool(kv, N, 2, P, 128, 3)
    v, vs, _ = make_pool(kv, N, 2, P, 128, 4)
    table = np.arange(N, dtype=np.int32)[None]
    v[2, 1, 3, 5] = float("nan") if kv == BF16 else ref.NAN_CODE
    _, o32, err = run_attn(kv, _values((1, 8, 128), 5).bfloat16(), k, ks, v, vs, table, [70], 0)
    assert err == 0
    assert torch.isfinite(o32[0, :4]).all() and torch.isnan(o32[0, 4:, 5]).all()
    assert torch.isfinite(o32[0, 4:, :5]).all()


def test_attn_rows_without_a_finite_score():
    """Scores of -infinity have weight 0; a row of nothing else is zero, and beside a finite score they change nothing."""
    P, HS = 16, 64
    k, v = torch.zeros(3, 1, P, HS), torch.ones(3, 1, P, HS)
    k[0, :, :, 0] = float("-inf")
    k[1, :, 3:, 0] = float("-inf")
    v[1, 0, :3] = torch.arange(3.0)[:, None]
    k, v = k.bfloat16(), v.bfloat16()
    q = torch.zeros(2, 1, HS).bfloat16()
    q[:, :, 0] = 1
    table = np.array([[0, -1], [0, 1]], dtype=np.int32)
    _, o32, err = run_attn(BF16, q, k, None, v, None, table, [16, 32], 0)
    assert err == 0 and (o32[0] == 0).all() and torch.allclose(o32[1], torch.ones(1, HS))


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attn_repairs_lengths_and_leaves_bad_pages_out(kv):
    P, N, HS = 16, 6, 64
    k, ks, _ = make_pool(kv, N, 1, P, HS, 3)
    v, vs, _ = make_pool(kv, N, 1, P, HS, 4)
    kr, vr = (k.double().numpy(), v.double().numpy()) if kv == BF16 else (k.numpy(), v.numpy())
    q = _values((3, 4, HS), 5).bfloat16()
    table = np.array([[0, 1, -1], [2, 3, 4], [5, 0, 1]], dtype=np.int32)
    o16, o32, err = run_attn(kv, q, k, ks, v, vs, table, [-5, 100, 40], 0)
    assert err == fd.FD_DEVERR_LEN_NEGATIVE | fd.FD_DEVERR_LEN_CLAMPED
    check_attn(kv, q, kr, ks, vr, vs, table, [-5, 100, 40], 0, o16, o32)
    table = np.array([[0, -1, 1], [2, 3, 99], [-1, -7, N]], dtype=np.int32)
    o16, o32, err = run_attn(kv, q, k, ks, v, vs, table, [40, 48, 33], 0)
    assert err == fd.FD_DEVERR_PAGE_ID
    check_attn(kv, q, kr, ks, vr, vs, table, [40, 48, 33], 0, o16, o32)
    assert (o32[2] == 0).all()


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_attn_forms_agree_on_streams_and_in_graphs(kv):
    """The library-owned workspace, the convenience form, another stream and a replayed graph (with lengths and pages
    changed between replays) give the bits of the explicit form."""
    P, HS, lens = 16, 128, [700, 33, 1, 0]
    N, wide = 60, 48
    k, ks, _ = make_pool(kv, N, 4, P, HS, 3)
    v, vs, _ = make_pool(kv, N, 4, P, HS, 4)
    q = _values((4, 16, HS), 5).bfloat16()
    table = make_table(lens, P, wide, N, 9)
    want, _, _ = run_attn(kv, q, k, ks, v, vs, table, lens, 0)
    qd, kd, ksd, vd, vsd, td = (d(x) for x in (q, k, ks, v, vs, table))
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got = fd.paged_attention(qd, kd, vd, td, ld, k_scale=ksd, v_scale=vsd)
    assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
    s, g, out = torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.zeros_like(qd)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fd.paged_attention(qd, kd, vd, td, ld, k_scale=ksd, v_scale=vsd, out=out)
        s.synchronize()
        assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))
        with torch.cuda.graph(g, stream=s):
            fd.paged_attention(qd, kd, vd, td, ld, k_scale=ksd, v_scale=vsd, out=out)
    for n in ([700, 33, 1, 0], [12, 100, 300, 5], [0, 0, 0, 0]):
        t2 = make_table(n, P, wide, N, sum(n))
        td.copy_(d(t2))
        ld.copy_(torch.tensor(n, dtype=torch.int32))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want, _, _ = run_attn(kv, q, k, ks, v, vs, t2, n, 0)
        assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))
    assert fd.fd_get_device_error() == 0


def test_attn_refuses_to_allocate_during_capture():
    P, HS = 16, 64
    k, _, _ = make_pool(BF16, 2, 1, P, HS, 3)
    a = [d(_values((1, 1, HS), 5).bfloat16()), d(k), d(k), torch.zeros(1, 2, dtype=torch.int32, device=DEV),
         torch.ones(1, dtype=torch.int32, device=DEV)]
    out = torch.zeros_like(a[0])
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    fd.fd_release()
    with torch.cuda.stream(s):
        g.capture_begin()
        try:
            with pytest.raises(fd.FdError) as e:
                fd.paged_attention(*a, out=out)
        finally:
            g.capture_end()
    assert e.value.status == fd.FD_ERR_WORKSPACE
    assert torch.isfinite(fd.paged_attention(*a, out=out).float()).all()


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("HS,G", [(128, 4), (512, 16)])
@pytest.mark.parametrize("tile", [0, 1])
def test_attn_waits_are_bounded(kv, HS, G, tile):
    """Copies that are never issued: the waits for them give up, the call returns with the error bit, and the next call is
    right again."""
    P, lens = 32, [900, 40, 2000]
    N, wide = 100, 63
    k, ks, _ = make_pool(kv, N, 1, P, HS, 3)
    v, vs, _ = make_pool(kv, N, 1, P, HS, 4)
    q = _values((3, G, HS), 5).bfloat16()
    table = make_table(lens, P, wide, N, 9)
    want, _, err = run_attn(kv, q, k, ks, v, vs, table, lens, 0)
    assert err == 0
    try:
        fd.fd_debug_withhold_copies(tile, 100_000)
        _, _, err = run_attn(kv, q, k, ks, v, vs, table, lens, 0)
    finally:
        fd.fd_debug_withhold_copies(-1)
    assert err & ~fd.FD_DEVERR_WAIT_TIMEOUT == 0
    assert err or tile > 0  # a share may have a single tile
    got, _, err = run_attn(kv, q, k, ks, v, vs, table, lens, 0)
    assert err == 0 and torch.equal(got.view(torch.int16), want.view(torch.int16))


# ------------------------------------------------------------------- the writer

def append_both(kv, lens, start, count, T, NKV, HS, P, table, N, seed=0, new=None, pad=0, pools=None):
    """fd_paged_append against the reference, every byte of the pool and every scale; returns the library's pools."""
    k, ks, _ = make_pool(kv, N, NKV, P, HS, seed + 1) if pools is None else pools[0]
    v, vs, _ = make_pool(kv, N, NKV, P, HS, seed + 2) if pools is None else pools[1]
    if new is None:
        new = (_values((T, 2, NKV, HS), seed + 3) * torch.exp(_values((T, 1, NKV, 1), seed + 4))).bfloat16()
    wide_rows = torch.full((max(T, 1), 2 * NKV * HS + pad), float("nan"), dtype=torch.bfloat16)
    wide_rows[:T, :2 * NKV * HS] = new.reshape(T, -1)
    rows = wide_rows.to(DEV)
    kd, vd, ksd, vsd = (None if x is None else x.to(DEV).clone() for x in (k, v, ks, vs))
    fd.fd_get_device_error()
    fd.fd_paged_append(rows, rows.data_ptr() + 2 * NKV * HS, kd, vd, ksd, vsd, d(table), d(np.asarray(lens, dtype=np.int32)),
                       None if start is None else d(np.asarray(start, dtype=np.int32)),
                       None if count is None else d(np.asarray(count, dtype=np.int32)), len(lens), T, NKV, HS, P, N,
                       table.shape[1], rows.stride(0), rows.stride(0), kv)
    torch.cuda.synchronize()
    for i, (pool, scale, got, gots) in enumerate(((k, ks, kd, ksd), (v, vs, vd, vsd))):
        x = new[:, i].double().numpy()
        if kv == BF16:
            bits = pool.clone()
            ids = np.arange(pool.numel(), dtype=np.float64).reshape(pool.shape)  # where each value comes from
            src = -1.0 - np.arange(x.size, dtype=np.float64).reshape(x.shape)
            ref.append(src, ids, None, table, lens, start, count, N)
            flat = torch.cat([bits.view(-1), new[:, i].reshape(-1)]).view(torch.int16)
            at = torch.from_numpy(np.where(ids < 0, pool.numel() - 1 - ids, ids).astype(np.int64))
            differ = int((got.cpu().view(torch.int16) != flat[at]).sum())
            assert differ == 0, f"{differ} elements differ"
        else:
            want, wants = pool.numpy().copy(), scale.numpy().copy()
            ref.append(x, want, wants, table, lens, start, count, N)
            assert np.array_equal(gots.cpu().numpy(), wants), "scales"
            a, b = ref.TABLE[got.cpu().numpy()], ref.TABLE[want]
            assert np.array_equal(a, b, equal_nan=True), f"{(a != b).sum()} codes differ"
    return (kd.cpu(), None if ks is None else ksd.cpu(), None), (vd.cpu(), None if vs is None else vsd.cpu(), None)


def _starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("HS", [64, 128, 256, 512])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_append_ragged(kv, HS, P):
    new = [1, 0, P, 2 * P + 3, 5, P + 1, 130]
    held = [0, 7, 0, 5, P - 1, P - 2, 3 * P]
    lens = [a + b for a, b in zip(new, held)]
    N = sum(-(-n // P) for n in lens) + 2
    table = make_table(lens, P, max(lens) // P + 2, N, HS + P)
    append_both(kv, lens, _starts(new), None, sum(new), 2, HS, P, table, N, seed=HS + P, pad=8)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("HS", [64, 128, 256, 512])
@pytest.mark.parametrize("P", [16, 128])
def test_append_token_by_token(kv, HS, P):
    """Each token of three pages by a call of its own, scales rising and blocks re-rounded on the way; an empty sequence
    beside it writes nothing."""
    N, NKV = 12, 3
    table = make_table([3 * P, 3 * P, 0], P, 4, N, 1)
    pools = make_pool(kv, N, NKV, P, HS, 1), make_pool(kv, N, NKV, P, HS, 2)
    for n in list(range(1, 20)) + [P, P + 1, 2 * P, 3 * P]:
        pools = append_both(kv, [n, 3 * P + 1 - n, 0], None, None, 3, NKV, HS, P, table, N, seed=n, pools=pools)
    assert fd.fd_get_device_error() == 0


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_append_counts_take_tokens_away(kv):
    new, P = [20, 20, 20, 1, 0], 16
    lens, count = [23, 40, 9, 8, 5], [20, 0, 7, -3, 4]
    table = make_table([64] * 5, P, 4, 20, 3)
    append_both(kv, lens, _starts(new), count, sum(new), 2, 64, P, table, 20, seed=5)
    append_both(kv, [5, 17, 1], None, [1, 0, 9], 3, 2, 64, P, table[:3], 20, seed=6)
    assert fd.fd_get_device_error() == 0


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_append_edge_values(kv):
    """Largest values on both sides of 448 powers of two, zeros, blocks of zeros, subnormals, the type's largest and
    lowest value, infinities and NaN."""
    P, HS, NKV = 16, 64, 2
    top = float(torch.finfo(torch.bfloat16).max)
    rows = []
    for a in (0.0, 448.0, 450.0, 1.75, 1.7578125, 0.875, 2.0 ** -133, 2.0 ** -126, 2.0 ** -118, top, -top, 1.0, 3.5):
        x = torch.zeros(NKV, HS)
        x[0, 3], x[0, 4], x[1, 9] = a, a / 2, -a
        rows.append(x)
    for bad in (float("inf"), float("-inf"), float("nan")):
        x = torch.ones(NKV, HS)
        x[0, 1], x[1, 2] = bad, 0.25
        rows.append(x)
    new = torch.stack(rows).bfloat16()
    new = torch.stack([new, new.flip(2)], 1)
    T = new.shape[0]
    for per in (1, 3, T):  # a token of each kind for itself, and together
        n = [per] * (T // per) + ([T % per] if T % per else [])
        table = make_table(n, P, 2, 20, 4)
        append_both(kv, n, _starts(n), None, T, NKV, HS, P, table, 20, new=new)
    # and behind tokens that are there already, where some scales rise and others stay
    n = [1] * T
    append_both(kv, [6] * T, _starts(n), None, T, NKV, HS, P, make_table([6] * T, P, 1, T, 5), T, new=new)


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_append_leaves_out_what_has_no_place(kv):
    P, N = 16, 8
    table = np.array([[0, 1], [2, -1], [99, 3], [4, 5]], dtype=np.int32)
    append_both(kv, [20, 20, 20, 40], _starts([20, 20, 20, 8]), None, 68, 1, 64, P, table, N, seed=1)
    assert fd.fd_get_device_error() == fd.FD_DEVERR_PAGE_ID
    append_both(kv, [4, 3, 8, 8], [-2, 2, 5, 50, 60], None, 20, 1, 64, P, np.array([[0, 1], [2, 3], [4, 5], [6, 7]], dtype=np.int32),
                N, seed=2)  # rows outside [0, T)
    assert fd.fd_get_device_error() == fd.FD_DEVERR_PAGE_ID
    append_both(kv, [0, -3, 2, 1], None, None, 4, 1, 64, P, np.array([[0], [1], [2], [3]], dtype=np.int32), N, seed=3)
    assert fd.fd_get_device_error() == 0


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_append_many_sequences(kv):
    rng = np.random.default_rng(5)
    new = rng.integers(0, 40, 400)
    held = rng.integers(0, 50, 400)
    lens = (new + held).tolist()
    N = sum(-(-n // 16) for n in lens) + 1
    append_both(kv, lens, _starts(new), None, int(new.sum()), 1, 64, 16, make_table(lens, 16, 8, N, 6), N)
    append_both(kv, [n + 1 for n in lens], None, None, 400, 1, 64, 16, make_table([n + 1 for n in lens], 16, 8, N + 400, 6),
                N + 400)


# -------------------------------------------------------------- the bookkeeping

class Device:
    """The library's bookkeeping beside the reference's, compared after each call."""

    def __init__(self, table, lens, refs, P, room=None):
        self.book = ref.Book(table, lens, refs, P)
        self.table, self.lens, self.refs = d(table.copy()), d(lens.copy()), d(refs.copy())
        self.P, self.N = P, len(refs)
        self.room = max(len(lens), self.N // 2) + 4 if room is None else room
        self.moves = torch.full((2 * (self.room + 1),), -77, dtype=torch.int32, device=DEV)

    def ws(self):
        n = fd.fd_pages_workspace_bytes(len(self.book.lens), self.N)
        self._ws = Guarded(n, DEV, fill=0xFF)
        return self._ws.ptr(), n

    def same(self, moves=None, left=None):
        torch.cuda.synchronize()
        assert np.array_equal(self.table.cpu().numpy(), self.book.table)
        assert np.array_equal(self.lens.cpu().numpy(), self.book.lens)
        assert np.array_equal(self.refs.cpu().numpy(), self.book.refs)
        if moves is not None:
            assert self._ws.canaries_intact()
            m = self.moves.cpu().numpy()
            assert m[0] == len(moves) and m[1] == left
            assert m[2:2 + 2 * len(moves)].reshape(-1, 2).tolist() == [list(x) for x in moves]
            assert (m[2 + 2 * len(moves):] == -77).all(), "entries behind the list are left as they were"
            self.moves.fill_(-77)

    def reserve(self, grow):
        B, wide = self.book.table.shape
        granted = torch.full((B,), -5, dtype=torch.int32, device=DEV)
        g = None if grow is None else d(np.asarray(grow, dtype=np.int32))
        fd.fd_pages_reserve(self.table, self.lens, self.refs, g, granted, self.moves, *self.ws(), B, wide, self.N, self.P)
        want, moves, left = self.book.reserve([1] * B if grow is None else grow)
        self.same(moves, left)
        assert granted.cpu().tolist() == want
        return want, moves

    def fork(self, parent):
        B, wide = self.book.table.shape
        n = len(parent)
        t2, l2 = torch.full((n, wide), -9, dtype=torch.int32, device=DEV), torch.full((n,), -9, dtype=torch.int32, device=DEV)
        fd.fd_pages_fork(self.table, self.lens, d(np.asarray(parent, dtype=np.int32)), t2, l2, self.refs, B, n, wide, self.N)
        self.table, self.lens = t2, l2
        self.book.fork(parent)
        self.same()

    def free(self, keep, window=0):
        B, wide = self.book.table.shape
        fd.fd_pages_free(self.table, self.lens, self.refs, None if keep is None else d(np.asarray(keep, dtype=np.int32)),
                         window, B, wide, self.N, self.P)
        self.book.free(keep, window)
        self.same()

    def compact(self):
        B, wide = self.book.table.shape
        fd.fd_pages_compact(self.table, self.refs, self.moves, *self.ws(), B, wide, self.N)
        moves, left = self.book.compact()
        self.same(moves, left)
        return moves


def empty(B, wide, N, P):
    return Device(np.full((B, wide), -1, dtype=np.int32), np.zeros(B, dtype=np.int32), np.zeros(N, dtype=np.int32), P)


@pytest.mark.parametrize("N", [1, 7, 500, 8192, 8193, 40000])
def test_bookkeeping_random_runs(N):
    rng = np.random.default_rng(N)
    for P, B in ((16, 5), (128, 33)):
        dev = empty(B, 12, N, P)
        fd.fd_get_device_error()
        for step in range(14):
            op = rng.integers(0, 6)
            if op <= 2:
                dev.reserve(None if op == 0 else rng.integers(-2, 3 * P if op == 1 else 4, len(dev.book.lens)))
            elif op == 3:
                dev.fork(rng.integers(-1, len(dev.book.lens), rng.integers(1, B + 5)))
            elif op == 4:
                dev.free(rng.integers(-1, 6 * P, len(dev.book.lens)), int(rng.integers(0, 2)) * int(rng.integers(1, 3 * P)))
            else:
                dev.compact()
        assert fd.fd_get_device_error() & fd.FD_DEVERR_PAGE_ID == 0


def test_reserve_denies_in_order_and_says_so():
    dev = empty(4, 10, 10, 16)
    fd.fd_get_device_error()
    assert dev.reserve([100, 16, 50, 1])[0] == [100, 16, 0, 0]  # 7 + 1 pages; 4 do not fit, and nothing passes them
    assert fd.fd_get_device_error() == fd.FD_DEVERR_PAGES_EXHAUSTED
    assert dev.reserve([1, 0, 32, 0])[0] == [1, 0, 32, 0]       # room in the last page, then the last two pages
    assert dev.reserve([10, 0, 1, 1])[0] == [10, 0, 0, 0]       # none is left: only what needs none
    assert fd.fd_get_device_error() == fd.FD_DEVERR_PAGES_EXHAUSTED
    dev.free([0, 16, 32, 0])
    assert dev.reserve([200, 1, 1, 0])[0] == [0, 1, 1, 0]       # a row that is too short stops nobody
    assert fd.fd_get_device_error() == fd.FD_DEVERR_PAGES_EXHAUSTED


def test_reserve_copies_shared_pages_once_for_each_writer():
    dev = empty(1, 6, 20, 16)
    dev.reserve([20])
    dev.fork([0, 0, 0])
    granted, moves = dev.reserve([1, 0, 13])   # the third also enters a new page
    assert granted == [1, 0, 13] and len(moves) == 2 and moves[0][0] == moves[1][0]
    _, moves = dev.reserve(None)               # now everyone has a page alone
    assert moves == []
    dev.free([16, 16, 16])
    _, moves = dev.reserve([4, 4, 4])          # whole pages stay shared: nothing is copied
    assert moves == []


def test_free_twice_and_bad_entries_do_no_harm():
    dev = empty(3, 4, 9, 16)
    dev.reserve([40, 16, 1])
    dev.free([0, 16, 1])
    dev.free([0, 16, 1])
    dev.free(None)
    fd.fd_get_device_error()
    dev.table[2, 3] = 50
    fd.fd_pages_free(dev.table, dev.lens, dev.refs, None, 0, 3, 4, 9, 16)
    dev.same()
    assert fd.fd_get_device_error() == fd.FD_DEVERR_PAGE_ID
    t2, l2 = torch.zeros(2, 4, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    fd.fd_pages_fork(dev.table, dev.lens, d(np.array([7, -2], dtype=np.int32)), t2, l2, dev.refs, 3, 2, 4, 9)
    assert fd.fd_get_device_error() == fd.FD_DEVERR_PAGE_ID
    assert (t2 == -1).all() and (l2 == 0).all() and (dev.refs == 0).all()


def test_reserve_denies_a_row_whose_last_page_is_gone():
    dev = empty(2, 4, 9, 16)
    dev.reserve([5, 5])
    fd.fd_get_device_error()
    dev.table[0, 0] = -1
    dev.book.table[0, 0] = -1
    assert dev.reserve([1, 1])[0] == [0, 1]
    assert fd.fd_get_device_error() == fd.FD_DEVERR_PAGE_ID | fd.FD_DEVERR_PAGES_EXHAUSTED


def test_bookkeeping_without_sequences():
    refs = np.zeros(5, dtype=np.int32)
    refs[[1, 4]] = 1  # pages that somebody else holds
    dev = Device(np.full((0, 3), -1, dtype=np.int32), np.zeros(0, dtype=np.int32), refs, 16)
    dev.table, dev.lens = torch.zeros(0, 3, dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV)
    dev.book.table = np.zeros((0, 3), dtype=np.int32)
    n = fd.fd_pages_workspace_bytes(0, 5)
    ws = Guarded(n, DEV, fill=0xFF)
    fd.fd_pages_compact(None, dev.refs, dev.moves, ws.ptr(), n, 0, 3, 5)
    torch.cuda.synchronize()
    assert dev.moves[:4].tolist() == [1, 3, 4, 0] and dev.refs.tolist() == [1, 1, 0, 0, 0]
    fd.fd_pages_reserve(None, None, dev.refs, None, None, dev.moves, ws.ptr(), n, 0, 3, 5, 16)
    torch.cuda.synchronize()
    assert dev.moves[:2].tolist() == [0, 3] and ws.canaries_intact()
    fd.fd_pages_free(None, None, None, None, 0, 0, 3, 5, 16)
    fd.fd_pages_fork(None, None, None, None, None, dev.refs, 0, 0, 3, 5)


# --------------------------------------------------------------------- copying

@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("HS,P,NKV,layers,N,n,room", [
    (64, 16, 1, 1, 5, 2, 2), (64, 16, 3, 2, 9, 4, 100), (128, 32, 5, 3, 40, 20, 20), (512, 128, 2, 1, 6, 3, 3),
    (256, 64, 1, 2, 300, 150, 150), (128, 16, 8, 4, 64, 0, 32), (128, 16, 8, 4, 64, 20, 7)])
def test_copy(kv, HS, P, NKV, layers, N, n, room):
    shape = (layers, N, NKV, P, HS)
    g = torch.Generator().manual_seed(N)
    dt = torch.uint8 if kv else torch.int16
    pools = [torch.randint(0, 127, shape, generator=g).to(dt) for _ in range(2)]
    scales = [torch.rand((layers, N, NKV), generator=g) if kv else None for _ in range(2)]
    ids = torch.randperm(N, generator=g)[:2 * n].view(n, 2).int()
    moves = torch.cat([torch.tensor([n, 99]), ids.view(-1), torch.zeros(200)]).int()
    dev = [d(x) for x in pools + scales]
    fd.fd_get_device_error()
    fd.fd_pages_copy(dev[0], dev[1], dev[2], dev[3], d(moves), room, layers, N, NKV, P, HS, kv)
    torch.cuda.synchronize()
    ids = ids[:room].long()
    for x, y in zip(pools + scales, dev):
        if x is not None:
            x[:, ids[:, 1]] = x[:, ids[:, 0]]
            assert torch.equal(x, y.cpu())
    assert fd.fd_get_device_error() == 0


def test_copy_leaves_out_moves_that_name_no_page():
    x = torch.arange(6 * 16 * 64, dtype=torch.int32).to(torch.int16).view(1, 6, 1, 16, 64)
    k, v = x.to(DEV), x.to(DEV)
    moves = torch.tensor([4, 0, 0, 1, -1, 2, 3, 6, 4, 5], dtype=torch.int32, device=DEV)
    fd.fd_get_device_error()
    fd.fd_pages_copy(k, v, None, None, moves, 4, 1, 6, 1, 16, 64, BF16)
    assert fd.fd_get_device_error() == fd.FD_DEVERR_PAGE_ID
    x[:, 1], x[:, 5] = x[:, 0].clone(), x[:, 4].clone()
    assert torch.equal(k.cpu(), x) and torch.equal(v.cpu(), x)
    moves[0] = -3
    fd.fd_pages_copy(k, v, None, None, moves, 4, 1, 6, 1, 16, 64, BF16)
    assert torch.equal(k.cpu(), x)


# ------------------------------------------------------------- all of it together

@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("HS,P,NKV,G", [(128, 16, 2, 4), (64, 32, 1, 8), (512, 64, 1, 16)])
def test_serving_run(kv, HS, P, NKV, G):
    """Prompts, decode steps, forks, endings and compactions on two layers; after each step the attention of every layer
    against the reference, whose cache is kept by sequence, without pages."""
    rng = np.random.default_rng(HS)
    layers, B, wide, N = 2, 5, 10, 30
    pool = [torch.zeros(layers, N, NKV, P, HS, dtype=torch.uint8 if kv else torch.bfloat16, device=DEV) for _ in range(2)]
    pool = [x.fill_(ref.NAN_CODE if kv else float("nan")) for x in pool]
    scale = [torch.full((layers, N, NKV), float("nan"), device=DEV) if kv else None for _ in range(2)]
    dev = empty(B, wide, N, P)
    fd.fd_get_device_error()

    # the reference's cache: for each layer and of K and V a pool of its own, in which sequence b has pages b * wide ...
    own = np.array([[b * wide + j for j in range(wide)] for b in range(B)], dtype=np.int32)
    rpool = [[np.zeros((B * wide, NKV, P, HS), dtype=np.uint8 if kv else np.float64) for _ in range(2)] for _ in range(layers)]
    rscale = [[np.zeros((B * wide, NKV)) if kv else None for _ in range(2)] for _ in range(layers)]

    def copy():
        fd.fd_pages_copy(*pool, *scale, dev.moves, dev.room, layers, N, NKV, P, HS, kv)

    def reserve(grow):
        granted = torch.zeros(B, dtype=torch.int32, device=DEV)
        fd.fd_pages_reserve(dev.table, dev.lens, dev.refs, d(np.asarray(grow, dtype=np.int32)), granted, dev.moves, *dev.ws(), B,
                            wide, N, P)
        copy()
        want, moves, left = dev.book.reserve(grow)
        dev.same(moves, left)
        assert granted.cpu().tolist() == want
        return granted

    for step in range(10):
        grow = rng.integers(0, 2 * P, B) if step % 4 == 0 else np.ones(B, dtype=np.int64)
        granted = reserve(grow)
        start, T = _starts(grow), int(np.sum(grow))
        for n in range(layers):
            new = torch.from_numpy(rng.standard_normal((T, 2, NKV, HS)) * 2).bfloat16()
            rows = new.to(DEV)
            fd.fd_paged_append(rows, rows.data_ptr() + 2 * NKV * HS, pool[0][n], pool[1][n], None if kv == BF16 else scale[0][n],
                               None if kv == BF16 else scale[1][n], dev.table, dev.lens, d(start), granted, B, T, NKV, HS, P,
                               N, wide, 2 * NKV * HS, 2 * NKV * HS, kv)
            for i in range(2):
                ref.append(new[:, i].double().numpy(), rpool[n][i], rscale[n][i], own, dev.book.lens, start,
                           granted.cpu().numpy(), B * wide)
            q = torch.from_numpy(rng.standard_normal((B, NKV * G, HS))).bfloat16()
            w = (0, 3 * P + 1)[step % 2]
            plan = fd.fd_paged_plan(B, NKV * G, NKV, HS, P, wide, w, kv_dtype=kv)
            ws, o16 = Guarded(plan.workspace_bytes, DEV), torch.zeros(B, NKV * G, HS, dtype=torch.bfloat16, device=DEV)
            o32 = torch.zeros(B, NKV * G, HS, device=DEV)
            fd.fd_paged_attn_ex(plan, ws.ptr(), plan.workspace_bytes, o32, d(q), pool[0][n], pool[1][n],
                                None if kv == BF16 else scale[0][n], None if kv == BF16 else scale[1][n], o16, dev.table,
                                dev.lens, B, NKV * G, NKV, HS, P, N, wide, w, 0.0)
            torch.cuda.synchronize()
            ks, vs = (None if s is None else torch.from_numpy(s) for s in rscale[n])
            check_attn(kv, q, rpool[n][0], ks, rpool[n][1], vs, own, dev.book.lens, w, o16.cpu(), o32.cpu())
        if step % 3 == 2:  # a beam step: rows change parents
            parent = rng.integers(0, B, B)
            dev.fork(parent)
            at = own[parent].reshape(-1)
            rpool = [[x[at].copy() for x in layer] for layer in rpool]
            rscale = [[None if x is None else x[at].copy() for x in layer] for layer in rscale]
        if step % 4 == 3:  # endings and rollbacks, then the pages move together
            keep = [0, 10 ** 6, int(dev.book.lens[2]) - 3, 10 ** 6, 5]
            dev.free(keep)
            fd.fd_pages_compact(dev.table, dev.refs, dev.moves, *dev.ws(), B, wide, N)
            copy()
            moves, left = dev.book.compact()
            dev.same(moves, left)
    assert fd.fd_get_device_error() & ~fd.FD_DEVERR_PAGES_EXHAUSTED == 0


def test_decode_step_in_a_graph():
    """A whole decode step captured once and replayed: growing, copying shared pages, writing, attending."""
    HS, P, NKV, G, B, wide, N = 128, 16, 2, 2, 3, 6, 18
    pool = [torch.zeros(N, NKV, P, HS, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scale = [torch.zeros(N, NKV, device=DEV) for _ in range(2)]
    dev = empty(1, wide, N, P)
    dev.reserve([21])
    new = torch.randn(21, 2, NKV, HS, device=DEV).bfloat16()
    args = (B, NKV, HS, P, N, wide)

    def write(rows, start, B, T):
        fd.fd_paged_append(rows, rows.data_ptr() + 2 * NKV * HS, *pool, *scale, dev.table, dev.lens, start, None, B, T, *args[1:],
                           2 * NKV * HS, 2 * NKV * HS, E4M3)

    write(new, d(np.array([0, 21], dtype=np.int32)), 1, 21)
    dev.fork([0, 0, 0])
    q = torch.randn(B, NKV * G, HS, device=DEV).bfloat16()
    out, row = torch.zeros_like(q), torch.zeros(B, 2, NKV, HS, dtype=torch.bfloat16, device=DEV)
    granted = torch.zeros(B, dtype=torch.int32, device=DEV)
    wsn = fd.fd_pages_workspace_bytes(B, N)
    ws = torch.empty(wsn, dtype=torch.uint8, device=DEV)

    def step():
        fd.fd_pages_reserve(dev.table, dev.lens, dev.refs, None, granted, dev.moves, ws, wsn, B, wide, N, P)
        fd.fd_pages_copy(*pool, *scale, dev.moves, dev.room, 1, N, NKV, P, HS, E4M3)
        write(row, None, B, B)
        fd.paged_attention(q, *pool, dev.table, dev.lens, k_scale=scale[0], v_scale=scale[1], out=out)

    hist = [[new[:, i].double().cpu().numpy()] * B for i in range(2)]
    hist = [[h.copy() for h in x] for x in hist]
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        fd.paged_attention(q, *pool, dev.table, dev.lens, k_scale=scale[0], v_scale=scale[1], out=out)  # makes the workspace
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            step()
    for i in range(30):
        x = torch.randn(B, 2, NKV, HS, device=DEV).bfloat16() * (1 + i)
        row.copy_(x)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _, moves, left = dev.book.reserve([1] * B)
        m = dev.moves.cpu()
        assert m[0] == len(moves) and m[1] == left
        dev.moves.fill_(-77)
        dev.same()
        for b in range(B):
            for j in range(2):
                hist[j][b] = np.concatenate([hist[j][b], x[b, j][None].double().cpu().numpy()])
    # the cache holds what was written, to the steps of its codes: two roundings of at most 2^-4, and the scale's least value
    for b in range(B):
        n = int(dev.book.lens[b])
        assert n == 51
        for j in range(2):
            pages = dev.book.table[b][:-(-n // P)]
            codes, sc = pool[j].cpu().numpy()[pages], scale[j].cpu().numpy()[pages]
            got = (ref.TABLE[codes] * sc[..., None, None]).transpose(0, 2, 1, 3).reshape(-1, NKV, HS)[:n]
            least = np.repeat(sc, P, 0)[:n][..., None] * 2.0 ** -9
            want = hist[j][b]
            assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -4 + 2.0 ** -8) + least).all()
    kr, vr = (p.cpu().numpy() for p in pool)
    want, big, _ = ref.attend(q.double().cpu().numpy(), kr, vr, scale[0].cpu().numpy(), scale[1].cpu().numpy(), dev.book.table,
                              dev.book.lens, 0, HS ** -0.5, N)
    assert (np.abs(out.double().cpu().numpy() - want) <= np.abs(want) * 2.0 ** -8 + 2.0 ** -10 * big[..., None]).all()
    assert fd.fd_get_device_error() == 0


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("HS,NKV,G,P,lens", [
    (64, 8, 4, 16, [131000, 70001, 63, 59000]), (128, 8, 4, 16, [120000, 1, 90007]), (512, 1, 16, 128, [262144, 200001]),
    (256, 4, 9, 32, [100000, 64, 101, 99999])])
def test_attn_long_shares(kv, HS, NKV, G, P, lens):
    """Shares of many tiles, run several times without a pause: against 64-bit attention of some heads, made on the GPU, and
    bit for bit the same every time."""
    wide = -(-max(lens) // P)
    N = sum(-(-n // P) for n in lens)
    table = make_table(lens, P, wide, N, 5)
    gen = torch.Generator(device=DEV).manual_seed(HS)
    shape = (N, NKV, P, HS)
    k, v = (torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    ks = vs = None
    if kv == E4M3:
        ks, vs = (torch.exp2(torch.randint(-8, -5, (N, NKV), generator=gen, device=DEV).float()) for _ in range(2))
        k, v = ((x * 64).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
    B, NH = len(lens), NKV * G
    q = torch.randn(B, NH, HS, generator=gen, device=DEV).bfloat16()
    td, ld = d(table), torch.tensor(lens, dtype=torch.int32, device=DEV)
    fd.fd_get_device_error()
    outs = [fd.paged_attention(q, k, v, td, ld, k_scale=ks, v_scale=vs) for _ in range(6)]
    assert fd.fd_get_device_error() == 0
    assert all(torch.equal(outs[0].view(torch.int16), x.view(torch.int16)) for x in outs[1:])
    val = torch.from_numpy(ref.TABLE).to(DEV)
    for b, n in enumerate(lens):
        pos = torch.arange(n, device=DEV)
        page, slot = td[b].long()[pos // P], pos % P
        for h in (0, NKV - 1):
            kk, vv = k[page, h, slot], v[page, h, slot]
            if kv == E4M3:
                kk, vv = val[kk.long()] * ks[page, h].double()[:, None], val[vv.long()] * vs[page, h].double()[:, None]
            kk, vv, qq = kk.double(), vv.double(), q[b, h * G:(h + 1) * G].double()
            want = torch.softmax(qq @ kk.T * HS ** -0.5, 1) @ vv
            mass = (qq.abs() @ kk.abs().T).amax(1, keepdim=True) * HS ** -0.5
            lim = (4 * HS * 2.0 ** -23 * mass + (2.0 ** -11 if kv == E4M3 else 2.0 ** -16) + 2.0 ** -20) * vv.abs().max()
            got = outs[0][b, h * G:(h + 1) * G].double()
            assert ((got - want).abs() <= lim + want.abs() * 2.0 ** -8).all()


@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_pages_behind_four_billion_elements(kv):
    """Append, attention and copy on pages at both ends of a pool of more than 2^32 elements: bit for bit what the same calls
    give on a pool of a few pages. The pages between are never read."""
    HS, NKV, P, G, lens, new = 512, 8, 128, 2, [300, 129], [130, 3]
    far = 2 ** 32 // (NKV * P * HS) + 9
    dt = torch.uint8 if kv == E4M3 else torch.bfloat16
    small = np.array([[0, 1, 2], [3, 4, -1]], dtype=np.int32)
    ids = np.array([far - 1, 2, far - 4, far - 2, 0])  # where the pages of the small pool lie in the large one
    q = _values((2, NKV * G, HS), 1).bfloat16().to(DEV)
    rows = _values((sum(new), 2, NKV, HS), 2).bfloat16().to(DEV)
    old = [make_pool(kv, 5, NKV, P, HS, s)[:2] for s in (3, 4)]
    results = []
    fd.fd_get_device_error()
    for N, at in ((6, np.arange(5)), (far, ids)):
        where = torch.from_numpy(at).to(DEV)
        spare = 5 if N == 6 else far - 3
        pools, scales = [], []
        for pages, scale in old:
            pools.append(torch.empty((N, NKV, P, HS), dtype=dt, device=DEV))
            pools[-1][where] = pages.to(DEV)
            scales.append(None if scale is None else torch.zeros((N, NKV), device=DEV))
            if scale is not None:
                scales[-1][where] = scale.to(DEV)
        table = d(np.where(small < 0, -1, at[np.maximum(small, 0)]).astype(np.int32))
        ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
        fd.fd_paged_append(rows, rows.data_ptr() + 2 * NKV * HS, *pools, *scales, table, ld, d(_starts(new)), None, 2, sum(new),
                           NKV, HS, P, N, 3, 2 * NKV * HS, 2 * NKV * HS, kv)
        out = torch.empty_like(q)
        fd.fd_paged_attn(q, *pools, *scales, out, table, ld, 2, NKV * G, NKV, HS, P, N, 3, 0, 0.0, kv)
        moves = torch.tensor([2, 0, int(at[0]), spare, int(at[4]), int(at[3])], dtype=torch.int32, device=DEV)
        fd.fd_pages_copy(*pools, *scales, moves, 2, 1, N, NKV, P, HS, kv)
        held = torch.cat([where, torch.tensor([spare], device=DEV)])
        results.append([x[held].cpu() for x in pools + scales if x is not None] + [out.cpu()])
        del pools
    assert fd.fd_get_device_error() == 0
    for x, y in zip(*results):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(results[1][0][5].view(torch.uint8), results[1][0][0].view(torch.uint8))
