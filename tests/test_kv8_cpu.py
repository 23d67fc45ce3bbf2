"""The paged 8-bit cache's calls on a machine without a GPU: refusals, sizes, and the
plain reference the GPU tests compare with.

Nothing here launches a kernel: every library call below is refused by its argument checks.
"""
import ctypes
import math

import pytest
import torch

import post_token_sparse_b200 as ds
from tests import kv8_ref as ref

P = ctypes.c_void_p(0x7000_0000_0000)  # aligned, never dereferenced
MIS = ctypes.c_void_p(0x7000_0000_0004)
NUL = None
BAD, UNS = ds.DS_ERR_INVALID_ARG, ds.DS_ERR_UNSUPPORTED


def dims(**kw):
    base = dict(B=2, Hq=8, Hkv=2, d=128, pages=100, page=64, table=10, format=0)
    base.update(kw)
    return ds.PageDims(*(base[n] for n, _ in ds.PageDims._fields_))


def calls(d, n=5):
    """Status of every call that takes these sizes, with pointers that are never read."""
    lib = ds.lib()
    yield lib.ds_page_assign(P, P, P, P, P, MIS, P, P, P, n, d, NUL)
    yield lib.ds_page_release(P, P, P, P, P, MIS, P, d, NUL)
    yield lib.ds_kv8_append(P, P, 256, MIS, P, P, P, n, 5, NUL, NUL, NUL, 0, 0, d, NUL)
    yield lib.ds_kv8_decode(MIS, P, P, P, P, P, NUL, d, 1.0, NUL, 0, NUL)
    yield lib.ds_kv8_sparse_decode(MIS, P, P, P, P, P, P, NUL, d, 5, 1.0, NUL, 0, NUL)
    yield lib.ds_kv8_group_sparse_decode(MIS, P, P, P, P, P, P, NUL, d, 5, 1.0, NUL, 0, NUL)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), BAD), (dict(pages=0), BAD), (dict(table=0), BAD), (dict(page=0), BAD),
    (dict(page=8), UNS), (dict(page=48), UNS), (dict(page=256), UNS),
    (dict(pages=1 << 28, page=16), UNS), (dict(table=1 << 27, page=16), UNS),
])
def test_sizes_of_the_pool(kw, want):
    assert list(calls(dims(**kw))) == [want] * 6
    assert ds.lib().ds_kv8_workspace_size(dims(**kw)) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(Hq=7), BAD), (dict(format=2), BAD),
    (dict(format=-1), BAD), (dict(d=0), BAD), (dict(d=64), UNS), (dict(B=20000), UNS),
    (dict(pages=1 << 25), UNS),
])
def test_sizes_of_the_heads(kw, want):
    assert list(calls(dims(**kw)))[2:] == [want] * 4


def test_limits_of_the_calls():
    lib, q = ds.lib(), ctypes.c_void_p(0x7000_0001_0000)
    many = (1 << 30) + 1
    assert lib.ds_page_assign(P, P, P, P, P, q, q, P, P, many, dims(), NUL) == UNS
    assert lib.ds_kv8_append(P, P, 256, P, P, P, P, many, many, NUL, NUL, NUL, 0, 0, dims(),
                             NUL) == UNS
    ok = (P, P, P, P, P)
    wide = dims(B=4000, Hq=16, Hkv=4, pages=1000, page=128, table=1 << 23)  # rows of all lists
    assert lib.ds_kv8_decode(*ok, P, NUL, wide, 1.0, P, 1 << 40, NUL) == UNS
    assert lib.ds_kv8_sparse_decode(*ok, P, P, NUL, dims(B=4000, Hq=16), 1 << 30, 1.0, P, 1 << 40,
                                    NUL) == UNS


@pytest.mark.parametrize("k,want", [((1 << 30) + 1, "UNS"), ((1 << 31) - 31, "UNS"),
                                    ((1 << 31) - 1, "UNS"), (1 << 30, "WS")])
def test_longest_list(k, want):
    """A list is at most 2^30 long, as a sequence is: the number of its tiles fits 32 bits on the
    GPU.  A list of that length comes to the next check, that of the workspace."""
    want = dict(UNS=UNS, WS=ds.DS_ERR_WORKSPACE)[want]
    d, ok = dims(B=1, Hq=1, Hkv=1), (P, P, P, P, P, P, P)
    for call in (ds.lib().ds_kv8_sparse_decode, ds.lib().ds_kv8_group_sparse_decode):
        assert call(*ok, NUL, d, k, 1.0, NUL, 0, NUL) == want


@pytest.mark.parametrize("Hq,Hkv,heads", [(8, 8, 1), (8, 2, 4), (64, 4, 8), (34, 2, 6),
                                          (64, 1, 8)])
def test_workspace(Hq, Hkv, heads):
    """Two partials a CTA and one a warp for the heads of a list, whatever the lengths."""
    lib, ok = ds.lib(), (P, P, P, P, P)
    d = dims(Hq=Hq, Hkv=Hkv)
    need = lib.ds_kv8_workspace_size(d)
    assert need == 1024 + (2 + 12) * 148 * heads * 132 * 4
    assert lib.ds_kv8_workspace_size(dims(B=7, Hq=Hq, Hkv=Hkv, table=9999)) == need
    for ws, n in ((NUL, need), (P, need - 1), (MIS, need)):
        assert lib.ds_kv8_decode(*ok, P, NUL, d, 1.0, ws, n, NUL) == ds.DS_ERR_WORKSPACE
        assert lib.ds_kv8_sparse_decode(*ok, P, P, NUL, d, 5, 1.0, ws, n, NUL) == \
            ds.DS_ERR_WORKSPACE


def test_pointers_and_counts():
    lib, d = ds.lib(), dims()
    assert list(calls(d)) == [BAD] * 6  # each has one misaligned pointer
    assert lib.ds_page_assign(P, P, P, P, P, P, P, P, P, 5, d, NUL) == BAD  # lens_out is lens
    q = ctypes.c_void_p(0x7000_0001_0000)
    assert lib.ds_page_assign(P, P, P, P, P, q, P, P, P, 5, d, NUL) == BAD  # n_free_out is n_free
    assert lib.ds_page_assign(P, P, P, P, P, q, q, P, P, -1, d, NUL) == BAD
    assert lib.ds_page_assign(P, P, P, P, P, q, q, P, NUL, 5, d, NUL) == BAD
    assert lib.ds_page_release(P, P, P, P, P, P, q, d, NUL) == BAD
    assert lib.ds_page_release(P, P, P, P, P, q, P, d, NUL) == BAD

    def append(K=P, stride=256, slots=P, n=5, most=5, C=NUL, label=NUL, lens=NUL, T=0, r=0):
        return lib.ds_kv8_append(K, P, stride, P, P, slots, P, n, most, C, label, lens, T, r, d,
                                 NUL)
    assert append(n=-1) == BAD
    assert append(most=0) == BAD
    assert append(K=NUL) == BAD
    assert append(K=MIS) == BAD
    assert append(slots=NUL) == BAD
    assert append(stride=255) == BAD      # below Hkv * d
    assert append(stride=260) == BAD      # rows not 16-byte aligned
    assert append(label=P, C=P, lens=P, T=10, r=0) == BAD
    assert append(label=P, C=P, lens=P, T=10, r=129) == BAD
    assert append(label=P, C=P, lens=P, T=0, r=8) == BAD
    assert append(label=P, C=NUL, lens=P, T=10, r=8) == BAD
    assert append(label=P, C=P, lens=NUL, T=10, r=8) == BAD
    assert append(n=0, K=NUL, slots=NUL, most=0) == ds.DS_OK  # nothing to do, nothing launched
    for k in (0, -3):
        assert lib.ds_kv8_sparse_decode(P, P, P, P, P, P, P, NUL, d, k, 1.0, NUL, 0, NUL) == BAD
        assert lib.ds_kv8_group_sparse_decode(P, P, P, P, P, P, P, NUL, d, k, 1.0, NUL, 0,
                                              NUL) == BAD
    assert lib.ds_kv8_sparse_decode(P, P, P, P, P, NUL, P, NUL, d, 5, 1.0, NUL, 0, NUL) == BAD
    assert lib.ds_kv8_decode(P, P, P, P, P, P, MIS, d, 1.0, NUL, 0, NUL) == BAD


def test_binding_refuses_wrong_tensors():
    KV = torch.zeros((4, 2, 16, 2, 128), dtype=torch.int8)
    with pytest.raises(TypeError, match="int8 or"):
        ds.kv8_workspace(torch.zeros(1, 2, 128), KV.to(torch.uint8))
    with pytest.raises(TypeError, match="KV must be"):
        ds.kv8_workspace(torch.zeros(1, 2, 128), KV[0])
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(TypeError, match="CUDA"):
        ds.page_release(i(2), i(2), i(2, 3), i(4), i(1), i(2), i(1), 16)
    with pytest.raises(TypeError, match="done must have shape"):
        ds.page_release(i(2), i(3), i(2, 3), i(4), i(1), i(2), i(1), 16)
    with pytest.raises(TypeError, match="slots must be"):
        ds.page_assign(i(2), i(2), i(4), i(1), i(2, 3), i(2), i(1), i(3), i(5).long(), 16)
    with pytest.raises(TypeError, match="block_table must be contiguous"):
        ds.page_release(i(2), i(2), i(3, 2).t(), i(4), i(1), i(2), i(1), 16)
    K = torch.zeros((5, 2, 128), dtype=torch.bfloat16)
    sc = torch.zeros((4, 2, 2))
    with pytest.raises(TypeError, match="heads of a token"):
        ds.kv8_append(K.transpose(1, 2).contiguous().transpose(1, 2), K, KV, sc, i(5), i(2), 5)
    with pytest.raises(TypeError, match="same token stride"):
        ds.kv8_append(K, torch.zeros((5, 4, 128), dtype=torch.bfloat16)[:, :2], KV, sc, i(5), i(2),
                      5)
    with pytest.raises(TypeError, match="label needs"):
        ds.kv8_append(K, K, KV, sc, i(5), i(2), 5, label=torch.zeros((1, 2, 9, 8)))


# ---- the reference itself ------------------------------------------------------

def test_reference_codes():
    x = torch.tensor([0.5, 1.5, -2.5, 126.5, 500.0, -500.0, math.inf, -math.inf, math.nan],
                     dtype=torch.float64)
    assert ref.codes(x, torch.int8).tolist() == [0, 2, -2, 126, 127, -127, 127, -127, 0]
    e = ref.codes(x, torch.float8_e4m3fn).float().tolist()
    # e4m3 steps: 1/16 at 0.5, 8 at 126.5; 2^-9 the smallest value, half of it rounds to 0
    assert e == [0.5, 1.5, -2.5, 128.0, 448.0, -448.0, 448.0, -448.0, 0.0]
    tiny = torch.tensor([2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10], dtype=torch.float64)
    assert ref.codes(tiny, torch.float8_e4m3fn).float().tolist() == [2.0 ** -9, 0.0, 2.0 ** -8]


@pytest.mark.parametrize("dtype,half", [(torch.int8, None), (torch.float8_e4m3fn, 2.0 ** -4)])
def test_reference_append_is_within_half_a_step(dtype, half):
    g = torch.Generator().manual_seed(1)
    page, N = 16, 37
    K, V = (torch.randn((N, 2, 128), generator=g).bfloat16() for _ in range(2))
    KV = torch.zeros((4, 2, page, 2, 128), dtype=torch.int8).view(dtype)
    sc = torch.zeros((4, 2, 2))
    slots = torch.tensor([(2 - i // page) * page + i % page for i in range(N)])
    KV, sc = ref.append(K, V, KV, sc, slots, torch.tensor([0, N]), page)
    table = torch.tensor([[2, 1, 0]])
    for h in range(2):
        k, v = ref.rows(KV, sc, table, 0, h, list(range(N)), page)
        for got, x in ((k, K[:, h].double()), (v, V[:, h].double())):
            step = sc[table[0, torch.arange(N) // page], h].double()[:, 0 if got is k else 1]
            if half is None:
                lim = step[:, None] * (0.5 + 127 * 2.0 ** -22)
            else:  # relative, or half the smallest step
                lim = torch.maximum(x.abs() * half, step[:, None] * 2.0 ** -10) * (1 + 2.0 ** -20)
            assert (got - x).abs().le(lim).all()


def test_reference_attention_is_torch_attention():
    g = torch.Generator().manual_seed(2)
    q, K, V = torch.randn(128, generator=g), torch.randn(9, 128, generator=g), \
        torch.randn(9, 128, generator=g)
    o, lse, _, _ = ref.attend(q, K.double(), V.double(), 0.3)
    want = torch.nn.functional.scaled_dot_product_attention(
        q.double()[None, None], K.double()[None], V.double()[None], scale=0.3)[0, 0]
    assert (o - want).abs().max() < 1e-12
    assert abs(lse - torch.logsumexp((K.double() @ q.double()) * 0.3, 0)) < 1e-12


def test_reference_assign_and_release_are_inverse():
    page, free = 16, list(range(20, 0, -1)) + [0]
    table = [[-1] * 6 for _ in range(3)]
    t, lens, nf, cu, slots, bits = ref.assign([0, 0, 0], [17, 0, 40], free, 21, table, 60, page)
    assert bits == 0 and nf == 21 - 5 and cu == [0, 17, 17, 57] and lens == [17, 0, 40]
    assert t[0][:2] == [0, 1] and t[2][:3] == [2, 3, 4]
    assert slots[:17] == [*range(16), 16] and slots[17] == 32 and slots[57:] == [-1] * 3
    f2, lens2, nf2, bits = ref.release(lens, [1, 1, 1], t, free, nf, page)
    assert nf2 == 21 and lens2 == [0, 0, 0] and sorted(f2) == sorted(free) and bits == 0
