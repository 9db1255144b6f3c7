"""The verification pass's entry points refuse bad arguments on the host, before any launch,
and the plain implementations that the GPU tests compare with do what they define."""
import ctypes as C

import numpy as np
import pytest

import speculative_decoding_drafter_head_b200 as ds
import verify_pass_ref as ref

F = C.c_void_p(0x10000)          # never dereferenced: every call below fails its host checks
ODD = C.c_void_p(0x10002)
HALF = C.c_void_p(0x10008)
OK, INVALID, SHAPE, SMALL = 0, 1, 2, 3


def layout(**kw):
    a = dict(L=F, anchor=F, x=F, accepted=None, context=F, rows=F, pages=F, held=F, free_pages=F,
             free_count=F, B=4, gamma=7, ps=16, max_pages=64, num_pages=256, cap=32, row_start=F,
             position=F, slot=F, token=F, stream=None)
    a.update(kw)
    return ds.load().dspark_verify_layout(*a.values())


@pytest.mark.parametrize("kw, status", [
    (dict(L=None), INVALID), (dict(context=None), INVALID), (dict(rows=None), INVALID),
    (dict(pages=None), INVALID), (dict(held=None), INVALID), (dict(free_pages=None), INVALID),
    (dict(free_count=None), INVALID), (dict(row_start=None), INVALID),
    (dict(position=None), INVALID), (dict(slot=None), INVALID),
    (dict(anchor=None), INVALID), (dict(x=None), INVALID),      # with a token output
    (dict(L=ODD), INVALID), (dict(accepted=ODD), INVALID), (dict(token=ODD), INVALID),
    (dict(cap=31), INVALID),                                    # below B (gamma + 1)
    (dict(B=0), SHAPE), (dict(B=4097, cap=1 << 30), SHAPE), (dict(gamma=-1), SHAPE),
    (dict(gamma=(1 << 20) + 1, cap=1 << 30), SHAPE), (dict(ps=0), SHAPE), (dict(ps=65537), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(num_pages=0), SHAPE), (dict(max_pages=1 << 30), SHAPE),
    (dict(num_pages=1 << 28), SHAPE),
])
def test_layout_refusals(kw, status):
    assert layout(**kw) == status


def norm(**kw):
    a = dict(qkv=F, stride=6144, qw=F, kw=F, eps=1e-6, inv=F, rot=128, inter=0, rs=1.0, pos=F, slot=F,
             n=F, cap=8, Hq=32, Hkv=8, D=128, ps=16, num_pages=64, q_out=F, kc=F, vc=F, stream=None)
    a.update(kw)
    return ds.load().dspark_qk_norm_rope_store(*a.values())


@pytest.mark.parametrize("kw, status", [
    (dict(qkv=None), INVALID), (dict(pos=None), INVALID), (dict(slot=None), INVALID),
    (dict(n=None), INVALID), (dict(q_out=None), INVALID), (dict(kc=None), INVALID),
    (dict(vc=None), INVALID), (dict(inv=None), INVALID), (dict(qkv=HALF), INVALID),
    (dict(qw=HALF), INVALID), (dict(kc=HALF), INVALID), (dict(pos=ODD), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(rs=float("inf")), INVALID),
    (dict(inter=2), INVALID), (dict(stride=6136), INVALID),
    (dict(stride=6148), SHAPE), (dict(D=96), SHAPE), (dict(D=256), SHAPE), (dict(rot=8), SHAPE),
    (dict(rot=144), SHAPE), (dict(rot=-16), SHAPE), (dict(Hq=0), SHAPE), (dict(Hkv=0), SHAPE),
    (dict(cap=0), SHAPE), (dict(ps=0), SHAPE), (dict(num_pages=1 << 28), SHAPE),
])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


def attention(**kw):
    a = dict(q=F, kc=F, vc=F, pages=F, context=F, row_start=F, B=4, cap=8, Hq=32, Hkv=8, D=128,
             ps=16, max_pages=64, num_pages=64, scale=0.1, out=F, ws=F, wsb=1 << 40, stream=None)
    a.update(kw)
    return ds.load().dspark_verify_attention(*a.values())


@pytest.mark.parametrize("kw, status", [
    (dict(q=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID),
    (dict(pages=None), INVALID), (dict(context=None), INVALID), (dict(row_start=None), INVALID),
    (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(q=HALF), INVALID),
    (dict(out=HALF), INVALID), (dict(vc=HALF), INVALID), (dict(ws=HALF), INVALID),
    (dict(pages=ODD), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(D=96), SHAPE), (dict(Hkv=0), SHAPE),
    (dict(Hq=12), SHAPE), (dict(Hq=4), SHAPE), (dict(Hq=113, Hkv=1), SHAPE), (dict(ps=8), SHAPE),
    (dict(ps=24), SHAPE), (dict(ps=256), SHAPE), (dict(B=0), SHAPE), (dict(B=4097), SHAPE),
    (dict(cap=0), SHAPE), (dict(max_pages=0), SHAPE), (dict(num_pages=0), SHAPE),
    (dict(num_pages=1 << 25), SHAPE), (dict(max_pages=1 << 30), SHAPE), (dict(wsb=16), SMALL),
])
def test_attention_refusals(kw, status):
    assert attention(**kw) == status


def test_workspace_bytes():
    assert ds.verify_attention_workspace_bytes(32, 8, 128) >= 256
    assert ds.verify_attention_workspace_bytes(32, 5, 128) == 0
    assert ds.verify_attention_workspace_bytes(32, 8, 96) == 0


def test_status_strings():
    assert ds.STATUS[9] == "OUT_OF_PAGES" and "pages" in ds.status_string(9)
    assert ds.STATUS[10] == "INVALID_PAGE" and "page" in ds.status_string(10)


def test_binding_refuses_cpu_tensors():
    import torch
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(TypeError):
        ds.verify_layout(z(2), z(2), z(2), z(2, 4), z(2), z(8), z(1), z(3), z(4), z(4), 16, 1)
    with pytest.raises(ValueError):       # drafts without a place for the tokens
        ds.verify_layout(z(2), z(2), z(2), z(2, 4), z(2), z(8), z(1), z(3), z(4), z(4), 16, 1,
                         anchor=z(2))
    bf = torch.bfloat16
    with pytest.raises(TypeError):
        ds.qk_norm_rope_store(torch.zeros(1, 384, dtype=bf), z(1), z(1), z(1),
                              torch.zeros(1, 1, 128, dtype=bf), torch.zeros(1, 1, 16, 128, dtype=bf),
                              torch.zeros(1, 1, 16, 128, dtype=bf))


def test_reference_layout_by_hand():
    # pages of 4: request 0 grows from 3 to 6 tokens (one page more), request 1 is idle and
    # gives its two pages back, request 2 needs one page of its three, request 3 starts
    pages = np.array([[5, -1, -1], [7, 8, -1], [1, 2, 3], [-1, -1, -1]])
    r = ref.layout(L=[2, 0, 1, 0], context=[3, -1, 0, 0], held=[1, 2, 3, 0], pages=pages,
                   free_pages=[9, 4, 0, 0, 0, 0, 0, 0, 0, 0], free_count=2, ps=4,
                   anchor=[10, 11, 12, 13], x=[[20, 21], [22, 23], [24, 25], [26, 27]])
    # the stack 9 4 takes 7 8 (request 1), then 2 3 (request 2); 3 goes to 0, 2 to 3
    assert r["free_pages"][:4].tolist() == [9, 4, 7, 8] and r["free_count"] == [4]
    assert r["pages"][0].tolist() == [5, 3, -1] and r["pages"][3].tolist() == [2, -1, -1]
    assert r["held"].tolist() == [2, 0, 1, 1] and r["rows"] == [3, 0, 2, 1]
    assert r["row_start"] == [0, 3, 3, 5, 6]
    assert r["position"] == [3, 4, 5, 0, 1, 0]
    assert r["slot"] == [23, 12, 13, 4, 5, 8]
    assert r["token"] == [10, 20, 21, 12, 24, 13] and not r["cut"]


def test_reference_layout_out_of_pages():
    r = ref.layout(L=[7, 7, 7], context=[2, 2, 4], held=[1, 1, 1], pages=np.zeros((3, 4), int),
                   free_pages=[3, 2, 0, 0], free_count=2, ps=4)
    # request 0 wants 3 pages and gets both; request 1 keeps two rows of its page, 2 has none
    assert r["rows"] == [8, 2, 0] and r["L"].tolist() == [7, 1, 0] and r["cut"]


def test_reference_attention_by_hand():
    # one query head, two keys with scores 0 and ln 3: weights 1/4 and 3/4
    k = np.zeros((1, 1, 16, 2)); v = np.zeros((1, 1, 16, 2))
    k[0, 0, 1, 0] = np.log(3.0)
    v[0, 0, 0], v[0, 0, 1] = [4, 0], [0, 4]
    q = np.ones((2, 1, 2))
    out, _ = ref.attention(q, k, v, np.array([[0]]), [0], [0, 2], 1.0)
    np.testing.assert_allclose(out[0, 0], [4, 0])
    np.testing.assert_allclose(out[1, 0], [1, 3])
