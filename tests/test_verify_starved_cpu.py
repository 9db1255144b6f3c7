"""Verification by rows refuses bad arguments on the host, before any launch."""
import ctypes as C
import inspect

import pytest

import speculative_decoding_drafter_head_b200 as ds
from speculative_decoding_drafter_head_b200.pipeline import VerifyPass

F = C.c_void_p(0x10000)          # never dereferenced: every call below fails its host checks
ODD = C.c_void_p(0x10002)
INVALID, SHAPE = 1, 2


def verify(**kw):
    a = dict(x=F, L=F, rows=F, anchor=F, target=F, B=4, gamma=7, accepted=F, bonus=F, stream=None)
    a.update(kw)
    return ds.load().dspark_verify_prefix_rows(*a.values())


@pytest.mark.parametrize("kw, status", [
    (dict(x=None), INVALID), (dict(L=None), INVALID), (dict(rows=None), INVALID),
    (dict(anchor=None), INVALID), (dict(target=None), INVALID), (dict(accepted=None), INVALID),
    (dict(bonus=None), INVALID), (dict(x=ODD), INVALID), (dict(rows=ODD), INVALID),
    (dict(anchor=ODD), INVALID), (dict(bonus=ODD), INVALID), (dict(B=0), SHAPE),
    (dict(gamma=-1), SHAPE), (dict(gamma=4097), SHAPE),
])
def test_refusals(kw, status):
    assert verify(**kw) == status


def test_rows_and_anchor_go_together():
    import torch
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for kw in (dict(rows=z(2)), dict(anchor=z(2)), dict(rows=z(3), anchor=z(2)),
               dict(rows=z(2), anchor=z(1))):
        with pytest.raises(ValueError):
            ds.verify_prefix(z(2, 3), z(2), z(2, 4), z(2), z(2), **kw)


def test_the_pass_says_what_to_look_at():
    """The documented step verifies by rows, and says how requests come, go and bring prompts."""
    import speculative_decoding_drafter_head_b200.pipeline as pipeline
    assert "vp.verify(" in pipeline.__doc__
    assert "rows" in inspect.getdoc(VerifyPass.verify)
    text = inspect.getdoc(VerifyPass)
    for word in ("context[b]", "accepted[b]", "prompt"):
        assert word in text
