"""The paged cache at the ends of its ranges: many heads, many sequences, the largest batches of positions."""

import numpy as np
import pytest
import torch

import decode_attention_04_gb300 as fd

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
