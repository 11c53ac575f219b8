"""The paged cache's C ABI without a GPU: plans, refused arguments (before any
CUDA call), and the reference of the GPU tests against independent values."""

import ctypes

import numpy as np
import pytest
import torch

import decode_attention_04_gb300 as fd
import paged_ref as ref


@pytest.fixture(scope="module", autouse=True)
def lib():
    from decode_attention_04_gb300 import build
    build.build()
    return fd.load_library()


def _aligned(n=4096):
    raw = np.zeros(n + 256, dtype=np.uint8)
    return raw, (raw.ctypes.data + 255) // 256 * 256


_KEEP, P0 = _aligned()  # an address for calls that are refused before anything reads it


def _status(f, *args, **kw):
    with pytest.raises(fd.FdError) as e:
        f(*args, **kw)
    return e.value.status


def _attn(**kw):
    a = dict(q=P0, k=P0, v=P0, ks=P0, vs=P0, out=P0, table=P0, lens=P0, B=1, NH=8, NKV=2, HS=128, P=16, N=4, mp=4, w=0,
             kv=fd.FD_KV_E4M3)
    a.update(kw)
    return (a["q"], a["k"], a["v"], a["ks"], a["vs"], a["out"], a["table"], a["lens"], a["B"], a["NH"], a["NKV"], a["HS"],
            a["P"], a["N"], a["mp"], a["w"], 0.0, a["kv"], 0)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), fd.FD_ERR_INVALID_ARG), (dict(B=65536), fd.FD_ERR_INVALID_ARG), (dict(NH=0), fd.FD_ERR_INVALID_ARG),
    (dict(NKV=0), fd.FD_ERR_INVALID_ARG), (dict(kv=2), fd.FD_ERR_INVALID_ARG), (dict(mp=0), fd.FD_ERR_INVALID_ARG),
    (dict(N=0), fd.FD_ERR_INVALID_ARG), (dict(HS=96), fd.FD_ERR_UNSUPPORTED), (dict(HS=1024), fd.FD_ERR_UNSUPPORTED),
    (dict(P=8), fd.FD_ERR_UNSUPPORTED), (dict(P=48), fd.FD_ERR_UNSUPPORTED), (dict(P=256), fd.FD_ERR_UNSUPPORTED),
    (dict(NH=9), fd.FD_ERR_UNSUPPORTED), (dict(NH=34), fd.FD_ERR_UNSUPPORTED),
    (dict(mp=1 << 27), fd.FD_ERR_UNSUPPORTED), (dict(B=65535, mp=1 << 16), fd.FD_ERR_UNSUPPORTED),
    *[({n: None}, fd.FD_ERR_INVALID_ARG) for n in ("q", "k", "v", "ks", "vs", "out", "table", "lens")],
])
def test_attn_refuses(kw, want):
    assert _status(fd.fd_paged_attn, *_attn(**kw)) == want


def _ex(plan, ws=P0, ws_bytes=None, out32=None, **kw):
    a = list(_attn(**kw))
    del a[17]
    return fd.fd_paged_attn_ex(plan, ws, plan.workspace_bytes if ws_bytes is None else ws_bytes, out32, *a)


def test_attn_ex_refuses_plans_workspaces_and_alignment():
    plan = fd.fd_paged_plan_sms(1, 8, 2, 128, 16, 4, 0, 152, fd.FD_KV_E4M3)
    up = lambda x: -(-x // 256) * 256
    assert plan.blocks == 152 and plan.granule == 32
    assert plan.workspace_bytes == up(2 * 152 * 4 * 128 * 4) + up(2 * 152 * 4 * 8) + up(152 * 16)
    # a share is 64 KB of K and V at least
    for HS, kv, want in ((64, fd.FD_KV_E4M3, 16), (128, fd.FD_KV_E4M3, 8), (128, fd.FD_KV_BF16, 4), (512, fd.FD_KV_BF16, 1)):
        assert fd.fd_paged_plan_sms(1, 8, 2, HS, 16, 4, 0, 152, kv).min_share == want
    assert _status(fd.fd_paged_plan_sms, 1, 8, 2, 128, 16, 4, 0, 1025, fd.FD_KV_BF16) == fd.FD_ERR_INVALID_ARG
    for name, value in (("B", 2), ("NH", 16), ("NKV", 4), ("HS", 64), ("page_size", 32), ("max_pages", 5), ("window", 7),
                        ("blocks", plan.blocks + 1), ("granule", 1), ("min_share", plan.min_share + 1), ("kv_dtype", 7),
                        ("num_sms", 0), ("workspace_bytes", 0)):
        bad = fd.fd_paged_plan_t.from_buffer_copy(plan)
        setattr(bad, name, value)
        assert _status(_ex, bad, ws_bytes=plan.workspace_bytes) == fd.FD_ERR_INVALID_ARG, name
    assert _status(_ex, plan, ws=None) == fd.FD_ERR_WORKSPACE
    assert _status(_ex, plan, ws_bytes=plan.workspace_bytes - 1) == fd.FD_ERR_WORKSPACE
    assert _status(_ex, plan, ws=P0 + 8) == fd.FD_ERR_ALIGNMENT
    assert _status(_ex, plan, out32=P0 + 4) == fd.FD_ERR_ALIGNMENT
    for name, off in (("q", 8), ("k", 8), ("v", 8), ("out", 2), ("table", 2), ("lens", 1), ("ks", 2), ("vs", 2)):
        assert _status(_ex, plan, **{name: P0 + off}) == fd.FD_ERR_ALIGNMENT, name
    empty = fd.fd_paged_plan_sms(0, 8, 2, 128, 16, 4, 0, 152, fd.FD_KV_E4M3)
    _ex(empty, ws=None, B=0, q=None)  # nothing to do


def _append(**kw):
    a = dict(kn=P0, vn=P0, k=P0, v=P0, ks=P0, vs=P0, table=P0, lens=P0, start=P0, count=None, B=2, T=3, NKV=2, HS=64, P=16,
             N=4, mp=4, sk=128, sv=128, kv=fd.FD_KV_E4M3)
    a.update(kw)
    return (*(a[n] for n in ("kn", "vn", "k", "v", "ks", "vs", "table", "lens", "start", "count", "B", "T", "NKV", "HS", "P",
                             "N", "mp", "sk", "sv", "kv")), 0)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), fd.FD_ERR_INVALID_ARG), (dict(T=-1), fd.FD_ERR_INVALID_ARG), (dict(start=None), fd.FD_ERR_INVALID_ARG),
    (dict(N=0), fd.FD_ERR_INVALID_ARG), (dict(sk=120), fd.FD_ERR_INVALID_ARG), (dict(sv=0), fd.FD_ERR_INVALID_ARG),
    (dict(sk=132), fd.FD_ERR_ALIGNMENT), (dict(sv=129), fd.FD_ERR_ALIGNMENT), (dict(kn=P0 + 2), fd.FD_ERR_ALIGNMENT),
    (dict(k=P0 + 8), fd.FD_ERR_ALIGNMENT), (dict(start=P0 + 2), fd.FD_ERR_ALIGNMENT), (dict(HS=100), fd.FD_ERR_UNSUPPORTED),
    (dict(P=24), fd.FD_ERR_UNSUPPORTED), (dict(kv=5), fd.FD_ERR_INVALID_ARG), (dict(count=P0 + 1), fd.FD_ERR_ALIGNMENT),
    *[({n: None}, fd.FD_ERR_INVALID_ARG) for n in ("kn", "vn", "k", "v", "ks", "vs", "table", "lens")],
])
def test_append_refuses(kw, want):
    assert _status(fd.fd_paged_append, *_append(**kw)) == want


def test_append_of_nothing_is_a_no_op():
    fd.fd_paged_append(*_append(T=0, kn=None, vn=None))
    fd.fd_paged_append(*_append(B=0, T=0, start=None, table=None))


def test_append_into_a_table_without_columns():
    """Empty sequences that get nothing: their table has no columns and no address."""
    fd.fd_paged_append(*_append(T=0, kn=None, vn=None, table=None, mp=0))
    assert _status(fd.fd_paged_append, *_append(mp=0)) == fd.FD_ERR_INVALID_ARG
    assert _status(fd.fd_paged_append, *_append(T=0, mp=-1)) == fd.FD_ERR_INVALID_ARG


def test_bookkeeping_refuses():
    need = fd.fd_pages_workspace_bytes(2, 8)
    assert need == 4 * (8 + 4 * 2 + 256)
    INV, UNS, ALI, WSP = fd.FD_ERR_INVALID_ARG, fd.FD_ERR_UNSUPPORTED, fd.FD_ERR_ALIGNMENT, fd.FD_ERR_WORKSPACE

    def reserve(table=P0, lens=P0, refs=P0, grow=P0, granted=P0, moves=P0, ws=P0, nb=need, B=2, mp=4, N=8, P=16):
        return _status(fd.fd_pages_reserve, table, lens, refs, grow, granted, moves, ws, nb, B, mp, N, P, 0)

    for n in ("table", "lens", "refs", "granted", "moves"):
        assert reserve(**{n: None}) == INV
        assert reserve(**{n: P0 + 2}) == ALI
    assert reserve(B=-1) == INV and reserve(B=65536) == INV and reserve(mp=0) == INV and reserve(N=0) == INV
    assert reserve(N=2 ** 31 - 1) == INV
    assert reserve(P=17) == UNS and reserve(mp=1 << 28) == UNS
    assert reserve(ws=None) == WSP and reserve(nb=need - 1) == WSP and reserve(ws=P0 + 8) == ALI

    def fork(table=P0, lens=P0 + 1024, parent=P0, to=P0 + 2048, lto=P0 + 1536, refs=P0, B=2, Bo=3, mp=4, N=8):
        return _status(fd.fd_pages_fork, table, lens, parent, to, lto, refs, B, Bo, mp, N, 0)

    for n in ("table", "lens", "parent", "to", "lto", "refs"):
        assert fork(**{n: None}) == INV
    assert fork(to=P0) == INV and fork(to=P0 + 16) == INV and fork(lto=P0 + 1024) == INV  # overlapping
    assert fork(Bo=-1) == INV and fork(Bo=65536) == INV and fork(parent=P0 + 1) == ALI

    def free(table=P0, lens=P0, refs=P0, keep=P0, w=0, B=2, mp=4, N=8, P=16):
        return _status(fd.fd_pages_free, table, lens, refs, keep, w, B, mp, N, P, 0)

    assert free(table=None) == INV and free(lens=None) == INV and free(refs=None) == INV and free(keep=P0 + 2) == ALI
    assert free(P=0) == UNS and free(N=-4) == INV

    def compact(table=P0, refs=P0, moves=P0, ws=P0, nb=need, B=2, mp=4, N=8):
        return _status(fd.fd_pages_compact, table, refs, moves, ws, nb, B, mp, N, 0)

    assert compact(table=None) == INV and compact(refs=None) == INV and compact(moves=None) == INV
    assert compact(ws=None) == WSP and compact(nb=need - 4) == WSP and compact(moves=P0 + 2) == ALI

    def copy(k=P0, v=P0, ks=P0, vs=P0, moves=P0, room=2, layers=1, N=8, NKV=2, P=16, HS=64, kv=1):
        return _status(fd.fd_pages_copy, k, v, ks, vs, moves, room, layers, N, NKV, P, HS, kv, 0)

    for n in ("k", "v", "ks", "vs", "moves"):
        assert copy(**{n: None}) == INV
    assert copy(room=-1) == INV and copy(layers=-1) == INV and copy(kv=3) == INV and copy(NKV=0) == INV
    assert copy(P=1) == UNS and copy(HS=65) == UNS and copy(k=P0 + 8) == ALI and copy(vs=P0 + 1) == ALI
    fd.fd_pages_copy(None, None, None, None, None, 0, 1, 8, 2, 16, 64, 1, 0)  # no room, no move


def test_plan_struct_matches_the_header():
    assert ctypes.sizeof(fd.fd_paged_plan_t) == 5 * 4 + 4 + 8 + 7 * 4 + 4


def test_convenience_form_refuses_what_bare_addresses_would_not_show():
    x = torch.zeros(2, 8, 64, dtype=torch.bfloat16)  # not on a GPU
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(Exception):
        fd.paged_attention(x, pages, pages, torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


# --------------------------------------------------------- the tests' reference

def test_reference_codes_are_those_of_the_format():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.TABLE, want, equal_nan=True)
    x = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * torch.exp2(torch.randint(-14, 10, (20000,)).float())
    x = x.clamp(-448, 448)
    got = ref.e4m3_code(x.double().numpy())
    assert np.array_equal(got, x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    mids = (ref._MAG[:-1] + ref._MAG[1:]) / 2  # ties
    assert np.array_equal(ref.e4m3_code(mids), torch.tensor(mids).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_block_scale():
    assert ref.block_scale(0.0) == 0 and ref.block_scale(448.0) == 1 and ref.block_scale(449.0) == 2
    assert ref.block_scale(224.0) == 0.5 and ref.block_scale(225.0) == 1 and ref.block_scale(1e-45) == 2.0 ** -126
    assert ref.block_scale(float(torch.finfo(torch.bfloat16).max)) == 2.0 ** 120


def test_reference_attention_is_a_softmax():
    g = np.random.default_rng(0)
    k, v = g.standard_normal((6, 2, 16, 64)), g.standard_normal((6, 2, 16, 64))
    q = g.standard_normal((1, 4, 64))
    table, lens = np.array([[4, 1, 3]], dtype=np.int32), np.array([37])
    out, _, _ = ref.attend(q, k, v, None, None, table, lens, 0, 0.125, 6)
    kk = np.concatenate([k[4], k[1], k[3]], 1)[:, :37]
    vv = np.concatenate([v[4], v[1], v[3]], 1)[:, :37]
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.tensor(q).view(1, 4, 1, 64), torch.tensor(kk).repeat_interleave(2, 0)[None],
        torch.tensor(vv).repeat_interleave(2, 0)[None], scale=0.125)
    assert np.allclose(out[0], want[0, :, 0].numpy(), atol=1e-12)
