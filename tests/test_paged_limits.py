"""The paged cache at the ends of its ranges: many heads, many sequences, the largest batches of positions, several threads, codes next
to ties."""

import threading

import numpy as np
import pytest
import torch

import decode_attention_04_gb300 as fd
import paged_ref as ref
from test_paged_gpu import case, empty

BF16, E4M3 = fd.FD_KV_BF16, fd.FD_KV_E4M3
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def lib():
    from decode_attention_04_gb300 import build
    build.build()
    return fd.load_library()


@pytest.mark.parametrize("B,P,wide", [(32768, 32, 65504), (32768, 16, 131008), (65535, 128, 8185), (1, 16, 134217472)])
def test_bound_on_positions(B, P, wide):
    """B * (max_pages * page_size / 32 + 32) is below 2^31 and max_pages * page_size at most 2^31 - 4097: one page less than
    each of these is taken, each is refused. The writer, given no token, shows the same bound."""
    per = wide * P
    assert B * (per // 32 + 32) >= 2 ** 31 or per > 2 ** 31 - 4097
    assert B * ((per - P) // 32 + 32) < 2 ** 31 and per - P <= 2 ** 31 - 4097

    def append(pages):
        fd.fd_paged_append(*[None] * 8, 16, None, B, 0, 1, 64, P, 1, pages, 64, 64, BF16, 0)

    assert fd.fd_paged_plan_sms(B, 2, 1, 64, P, wide - 1, 0, 152, BF16).max_pages == wide - 1
    append(wide - 1)
    for call in (lambda: fd.fd_paged_plan_sms(B, 2, 1, 64, P, wide, 0, 152, BF16), lambda: append(wide)):
        with pytest.raises(fd.FdError) as e:
            call()
        assert e.value.status == fd.FD_ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
def test_append_more_heads_than_a_grid_is_high(kv):
    """40,000 heads whose blocks take eight warps an item: 80,000 items of one page."""
    NKV, HS, P, T = 40000, 128, 128, 3
    gen = torch.Generator(device=DEV).manual_seed(1)
    new = torch.randn(T, 2, NKV, HS, generator=gen, device=DEV).bfloat16()
    dt = torch.uint8 if kv else torch.bfloat16
    pools = [torch.zeros(1, NKV, P, HS, dtype=dt, device=DEV) for _ in range(2)]
    scales = [torch.full((1, NKV), -1.0, device=DEV) if kv else None for _ in range(2)]
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.full((1,), T, dtype=torch.int32, device=DEV)
    start = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    fd.fd_get_device_error()
    fd.fd_paged_append(new, new[:, 1], *pools, *scales, table, lens, start, None, 1, T, NKV, HS, P, 1, 1, new.stride(0),
                       new.stride(0), kv)
    assert fd.fd_get_device_error() == 0
    for i in range(2):
        x = new[:, i].transpose(0, 1)  # [NKV, T, HS]
        if kv:
            top = x.double().abs().amax((1, 2))
            s = torch.exp2(torch.ceil(torch.log2(top / 448)))
            assert (top <= 448 * s).all() and (top > 224 * s).all()
            assert torch.equal(scales[i][0], s.float())
            x = (x.float() / s.float()[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(pools[i][0, :, :T].view(torch.uint8), x.contiguous().view(torch.uint8))
        assert not pools[i][0, :, T:].view(torch.uint8).any()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("B", [128, 129, 1024, 1025, 3001])
def test_attn_many_sequences(kv, B):
    """On both sides of 128 sequences (a warp finds its share by itself) and of 1024 (lengths are kept in shared memory)."""
    lens = [int(x) for x in np.random.default_rng(B).integers(0, 60, B)]
    case(kv, 64, 1, 2, 16, lens, seed=B)
    case(kv, 64, 2, 1, 16, [max(n - 20, 0) for n in lens], window=13, seed=B)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1500, 20000])
@pytest.mark.parametrize("B", [1024, 1025, 2500])
def test_bookkeeping_many_sequences(B, N):
    """More than 1024 sequences: their lists lie in the workspace and are made in chunks of 1024, whose pages, grants and moves
    go on from one to the next; in one block and in a cluster."""
    P, rng = 16, np.random.default_rng(B + N)
    dev = empty(B, 8, N, P)
    fd.fd_get_device_error()
    dev.reserve(rng.integers(-1, 4, B))               # with 1500 pages some sequences of a later chunk get none
    dev.reserve(None)
    dev.fork(rng.integers(0, B, B))                   # shared last pages in every chunk
    _, moves = dev.reserve(rng.integers(0, 3, B))
    assert N < 2 * B or len(moves) > 100
    dev.free(rng.integers(0, 8, B))
    dev.compact()
    dev.reserve(rng.integers(0, 40, B))               # denied from the middle of a chunk on, where pages run out
    dev.fork(rng.integers(-1, B, B + 3))
    dev.free(None, 5)
    dev.compact()
    assert fd.fd_get_device_error() & fd.FD_DEVERR_PAGE_ID == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 130])
def test_attn_one_sequence_of_more_than_two_billion_pieces(B):
    """2^31 pieces of 32 positions in one sequence (65535 heads, each of a band of 2^20 positions over the same four pages):
    shares begin behind 2^31. Attention over pages that repeat is attention over them once. The other sequences are empty."""
    NKV, HS, P, n = 65535, 64, 16, 1 << 20
    assert NKV * (n // 32 + 16) > 2 ** 31
    gen = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(4, NKV, P, HS, generator=gen, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.ones(4, NKV, device=DEV) for _ in range(2))
    q = torch.randn(B, NKV, HS, generator=gen, device=DEV).bfloat16()
    table = torch.zeros(B, n // P, dtype=torch.int32, device=DEV)
    table[B - 1] = torch.arange(n // P, device=DEV) % 4
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    lens[B - 1] = n
    out = torch.full_like(q, float("nan"))
    fd.fd_get_device_error()
    fd.paged_attention(q, k, v, table, lens, k_scale=ks, v_scale=vs, out=out)
    assert fd.fd_get_device_error() == 0
    assert not out[:B - 1].any()
    for h in range(0, NKV, 4096):
        kk, vv = (x[:, h:h + 4096].double().transpose(0, 1).reshape(-1, 4 * P, HS) for x in (k, v))
        qq = q[B - 1, h:h + 4096].double()[:, None]
        s = (qq @ kk.transpose(1, 2)) * HS ** -0.5
        want = (torch.softmax(s, 2) @ vv)[:, 0]
        mass = (qq.abs() @ kk.abs().transpose(1, 2)).amax(2) * HS ** -0.5
        # the score's sum, weights of 24 bits, the sums over n positions (32 an addition, in two groups), and bf16's half step
        lim = (4 * HS * 2.0 ** -23 * mass + 2.0 ** -20 + (n / 64) * 2.0 ** -23) * vv.abs().amax((1, 2))[:, None]
        assert ((out[B - 1, h:h + 4096].double() - want).abs() <= lim + want.abs() * 2.0 ** -8).all()


@pytest.mark.gpu
def test_threads_on_their_default_streams_have_a_workspace_each():
    """The per-thread default stream has one handle (2) for as many streams as there are threads, which may run at the same
    time: the library's workspace (10 MB on 152 SMs) is allocated for each."""
    P, HS, n = 16, 128, 4000
    k = torch.randn(n // P, 2, P, HS, device=DEV).bfloat16()
    q = torch.randn(1, 8, HS, device=DEV).bfloat16()
    table = torch.arange(n // P, dtype=torch.int32, device=DEV)[None]
    lens = torch.full((1,), n, dtype=torch.int32, device=DEV)
    want = fd.paged_attention(q, k, k, table, lens)
    outs = [torch.zeros_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    free, failed = [torch.cuda.mem_get_info()[0]], []

    def call(out):
        try:
            torch.cuda.set_device(q.device)
            for _ in range(2):
                fd.fd_paged_attn(q, k, k, None, None, out, table, lens, 1, 8, 2, HS, P, n // P, n // P, 0, 0.0, BF16, 2)
            torch.cuda.synchronize()
        except Exception as e:
            failed.append(e)

    for out in outs:
        t = threading.Thread(target=call, args=(out,))
        t.start()
        t.join()
        free.append(torch.cuda.mem_get_info()[0])
    assert not failed
    assert free[0] - free[1] >= 9 << 20 and free[1] - free[2] >= 9 << 20
    assert all(torch.equal(out.view(torch.int16), want.view(torch.int16)) for out in outs)


@pytest.mark.gpu
def test_reserve_counts_free_pages_that_were_not_handed_out():
    """Two owners of one begun page, and both write: each gets a copy, the original is free, and moves[1] does not count it."""
    dev = empty(1, 3, 8, 16)
    dev.reserve([5])
    dev.fork([0, 0])
    _, moves = dev.reserve([1, 1])
    assert moves == [(0, 1), (0, 2)] and dev.book.refs.tolist() == [0, 1, 1, 0, 0, 0, 0, 0]
    refs = dev.refs.clone()
    fd.fd_pages_reserve(dev.table, dev.lens, dev.refs, torch.zeros(2, dtype=torch.int32, device=DEV),
                        torch.empty(2, dtype=torch.int32, device=DEV), dev.moves, *dev.ws(), 2, 3, 8, 16)
    assert dev.moves[:2].tolist() == [0, 6] and torch.equal(dev.refs, refs)  # the next call does


def _near_ties():
    """(x, s): bf16 values and fp32 scales whose quotient is within 2^-24 of the middle of two codes, but not on it."""
    out = []
    for middle in range(17, 33, 2):
        for x in range(128, 256):
            s = np.float32(x / middle)
            if float(s) * middle != x:
                out.append((float(x), float(s)))
    return out


@pytest.mark.gpu
def test_append_codes_next_to_the_middle_of_two():
    """Scales that are no powers of two, as a cache from elsewhere has them: x / scale next to a tie goes to the nearer code, not
    to the one that a quotient rounded onto the tie gives."""
    cases = _near_ties()
    assert len(cases) > 500
    HS, P, NKV = 64, 16, len(cases)  # a head for each case, as each has a scale
    x = torch.tensor([c[0] for c in cases], dtype=torch.float64)
    s = torch.tensor([c[1] for c in cases], dtype=torch.float64)
    sign = torch.where(torch.arange(HS) % 2 == 0, 1.0, -1.0)
    new = (x[:, None] * sign)[None].bfloat16()
    assert torch.equal(new.double()[0, :, 0], x)
    codes = torch.full((1, NKV, P, HS), 0x38, dtype=torch.uint8)  # earlier tokens: ones
    want = ref.e4m3_code((new[0].double() / s[:, None]).numpy())
    pools, scales = [codes.to(DEV) for _ in range(2)], [s.float()[None].to(DEV) for _ in range(2)]
    rows = torch.stack([new, new], 1).to(DEV)
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.full((1,), 2, dtype=torch.int32, device=DEV)
    fd.fd_paged_append(rows, rows[:, 1], *pools, *scales, table, lens, None, None, 1, 1, NKV, HS, P, 1, 1, rows.stride(0),
                       rows.stride(0), E4M3)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(scales[i].cpu()[0], s.float())  # no scale rose
        got = pools[i][0, :, 1].cpu().numpy()
        assert np.array_equal(got, want), f"{(got != want).sum()} of {got.size} codes differ"


@pytest.mark.gpu
def test_append_rounds_earlier_codes_next_to_the_middle_of_two():
    """Codes whose product with old scale / new scale is next to a tie, where a new token raises a scale that is no power of two."""
    HS, P = 64, 16
    held = [c for c in range(9, 0x78) if c & 7 in (3, 5, 7)]  # codes of odd significands 11, 13, 15
    pairs = []
    for c in held:
        for middle in range(17, 33, 2):
            old = np.float32(middle / (8 + (c & 7)) / 4)
            if float(old) * (8 + (c & 7)) * 4 != middle and 0.25 < old < 0.9:
                pairs.append((c, float(old)))
    NKV = len(pairs)
    assert NKV > 300
    old = torch.tensor([p[1] for p in pairs], dtype=torch.float64)
    codes = torch.zeros(1, NKV, P, HS, dtype=torch.uint8)
    codes[0, :, 0] = torch.tensor([p[0] for p in pairs], dtype=torch.uint8)[:, None]
    codes[0, :, 0, 1::2] |= 0x80
    want = ref.e4m3_code(ref.TABLE[codes[0, :, 0].numpy()] * old[:, None].numpy())
    pools, scales = [codes.to(DEV) for _ in range(2)], [old.float()[None].to(DEV) for _ in range(2)]
    rows = torch.full((1, 2, NKV, HS), 448.0, device=DEV).bfloat16()  # the new scale is 1
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.full((1,), 2, dtype=torch.int32, device=DEV)
    fd.fd_paged_append(rows, rows[:, 1], *pools, *scales, table, lens, None, None, 1, 1, NKV, HS, P, 1, 1, rows.stride(0),
                       rows.stride(0), E4M3)
    torch.cuda.synchronize()
    for i in range(2):
        assert (scales[i] == 1).all()
        got = pools[i][0, :, 0].cpu().numpy()
        assert np.array_equal(got, want), f"{(got != want).sum()} of {got.size} codes differ"
