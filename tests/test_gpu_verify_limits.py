"""The verification pass at the ends of its range: references that rise in every tile, values that
are not finite, scores and contexts of extreme size, launches in a shape that cannot run."""
import numpy as np
import pytest

from test_gpu_verify_pass import (check_attention, ds, host, i32, make_attention,  # noqa: F401
                                  reference_attention, torch_nan_to, with_workspace)

pytestmark = pytest.mark.gpu


def slots_of(s, b, count):
    """(page, offset) of request b's first `count` tokens."""
    import torch
    ps = s["k_cache"].shape[2]
    j = torch.arange(count, device="cuda")
    return s["pages"][b].long()[j // ps], j % ps


def set_keys(s, b, keys):
    """The first len(keys) keys of request b, the same for every key head: [n, D]."""
    page, off = slots_of(s, b, len(keys))
    s["k_cache"][page, :, off] = keys[:, None].to(s["k_cache"].dtype).expand(
        -1, s["k_cache"].shape[1], -1)


# Query tiles of up to 64 rows, and of up to 112 where the row capacity asks for more; 3 and 17
# tokens leave the last 16 columns in part empty, 16 and 28 fill the tile.
@pytest.mark.parametrize("tokens", [3, 16, 17, 28])
@pytest.mark.parametrize("D", [64, 128])
def test_reference_rises_in_every_tile(ds, D, tokens):  # noqa: F811
    """One row's scores jump by 2^29 in weight from tile to tile, so that every tile raises the
    references of all rows; the others' rise by factors of 0.13 to 0.8, so that O and l of the
    tiles before, scaled, are much of the result.  Some twelve tiles to a segment: both softmax
    groups raise, and find weights that the other has made stale."""
    import torch
    rng = np.random.default_rng(D + tokens)
    B, Hq, Hkv = 37, 16, 4
    ctx = 1400 + 5 * rng.integers(0, 60, B)
    s, start = make_attention(ctx, [tokens] * B, Hq, Hkv, D, 16, D + tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    for b in range(B):
        n = int(ctx[b]) + tokens
        k = torch.zeros(n, D, device="cuda")
        k[:, 0] = torch.arange(n, device="cuda") // 128
        k[:, 1] = torch.rand(n, generator=g, device="cuda") * 2 - 1
        set_keys(s, b, k)
    q = torch.zeros(s["q"].shape, device="cuda")
    r = torch.arange(q.shape[0] * Hq, device="cuda").reshape(-1, Hq)
    q[:, :, 0] = 0.25 + 0.25 * (r % 8)
    q[:, :, 1] = torch.rand(r.shape, generator=g, device="cuda") * 2 - 1
    # the row that jumps: one of each request's, in every key head
    at = torch.from_numpy(start[:-1] + rng.integers(0, tokens, B)).cuda()
    q[at, 1::4, 0] = 20.0
    s["q"] = q.bfloat16()
    with_workspace(ds, s)
    ds.verify_attention(**s, scale=1.0)
    assert ds.get_error() == 0
    # scores of two exact products, below 20 x 14: fp32 is off by 2^-15 in one of them, and the
    # scaling of O and l by 2^-22 of a factor a tile, far within check_attention's 2^-9
    check_attention(s, int(start[-1]), 1.0)
    out, _ = reference_attention(s, 1.0)
    last = out.clone()                                 # without the first ten tiles
    for b in range(B):
        page, off = slots_of(s, b, 1280)
        s["k_cache"][page, :, off, 0] = -200.0
    last, _ = reference_attention(s, 1.0)
    slow = s["q"][:, :, 0].float() == 0.25
    assert float((out - last).abs()[slow].mean()) > 0.02     # the tiles before do count


@pytest.mark.parametrize("others", [0, 230])               # units in parts, and whole ones
@pytest.mark.parametrize("D, tokens", [(64, 8), (64, 20), (128, 8), (128, 20)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_hidden_values_everywhere(ds, value, D, tokens, others):  # noqa: F811
    """A later row's key or value that is not finite reaches the rows that see it, no other: both
    head sizes, both query tiles, with and without a join."""
    rng = np.random.default_rng(5)
    ctx = [250, 100] + list(rng.integers(0, 300, others))
    s, start = make_attention(ctx, [tokens] * len(ctx), 8, 2, D, 16, 4)
    pages = host(s["pages"])
    for cache, b, pos in (("v_cache", 0, 254), ("k_cache", 1, 103), ("v_cache", 1, 106)):
        s[cache][int(pages[b, pos // 16]), 1, pos % 16, 17] = value
    with_workspace(ds, s)
    ds.verify_attention(**s)
    assert ds.get_error() == 0
    got = s["out"].double()
    clean = dict(s)
    clean["k_cache"], clean["v_cache"] = (torch_nan_to(s[k]) for k in ("k_cache", "v_cache"))
    out, mag = reference_attention(clean, D ** -0.5)
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -7 + 2.0 ** -9) * mag
    ok = (got - out).abs() <= tol
    assert bool(ok[:, :4].all())                            # the other key head
    assert bool(ok[:4].all())                               # request 0, rows before the value
    rest = ok[4:tokens, 4:]
    assert bool(rest[..., :17].all()) and bool(rest[..., 18:].all())
    bad = got[4:tokens, 4:, 17]
    assert bool(bad.isnan().all()) if value != value else bool((bad == value).all())
    assert bool(ok[tokens:tokens + 3].all())                # request 1, rows before the key
    assert bool(ok[2 * tokens:].all())                      # the other requests


@pytest.mark.parametrize("low", [0.0, float("-inf")])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_seen_value_in_a_part_of_no_weight(ds, value, D, low):  # noqa: F811
    """A value that is not finite reaches the rows that see it, whatever its key's weight rounds
    to: zero times it is NaN.  So also where a part of a cut unit has no weight beside the others,
    or none at all."""
    import torch
    s, start = make_attention([2000], [2], 2, 1, D, 16, 8)
    k = torch.zeros(2002, D, device="cuda")
    k[:, 0] = low
    k[1000:, 0] = 300.0
    set_keys(s, 0, k)
    s["q"].zero_()
    s["q"][:, :, 0] = 1.0
    page, off = slots_of(s, 0, 11)
    s["v_cache"][page[10], 0, off[10], 5] = value
    with_workspace(ds, s)
    ds.verify_attention(**s, scale=1.0)
    assert ds.get_error() == 0
    got = s["out"].double()
    assert not bool(got[:, :, 5].isfinite().any())
    s["v_cache"] = torch_nan_to(s["v_cache"])
    out, mag = reference_attention(s, 1.0)
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -7 + 2.0 ** -9) * mag
    ok = (got - out).abs() <= tol
    assert bool(ok[:, :, :5].all()) and bool(ok[:, :, 6:].all())


@pytest.mark.parametrize("others", [0, 230])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 14, 2.0 ** 17, 2.0 ** 40, -2.0 ** 14, -2.0 ** 40])
@pytest.mark.parametrize("D, tokens", [(64, 3), (128, 20)])
def test_scores_of_any_size(ds, D, tokens, size, others):  # noqa: F811
    """Scores far beyond 2^24, where a score's own rounding is more than a weight's range: the
    largest take all, in equal shares."""
    import torch
    ctx = [700, 40] + [50] * others
    s, start = make_attention(ctx, [tokens] * len(ctx), 8, 2, D, 16, 31)
    g = torch.Generator(device="cuda").manual_seed(1)
    for b in range(len(ctx)):
        n = ctx[b] + tokens
        k = torch.zeros(n, D, device="cuda")
        k[:, 0] = abs(size) * (1 + torch.randint(0, 40, (n,), generator=g, device="cuda") / 64)
        set_keys(s, b, k)
    s["q"].zero_()
    s["q"][:, :, 0] = size * (1 + torch.arange(8, device="cuda") / 8)
    with_workspace(ds, s)
    ds.verify_attention(**s, scale=1.0)
    assert ds.get_error() == 0
    # scores are single products of two bf16, exact, and differ by 2^-7 of their size at least:
    # 2^17 in natural logarithms from 2^24 on, so the weights are 1 or 0 in any arithmetic
    check_attention(s, int(start[-1]), 1.0)


def test_scores_below_any_reference(ds):  # noqa: F811
    """Finite scores of -1e36 behind keys whose scores are -inf."""
    import torch
    D, others = 128, 230
    ctx = [256, 200] + [40] * others
    s, start = make_attention(ctx, [1] * len(ctx), 4, 2, D, 16, 32)
    for b in range(2):
        n = ctx[b] + 1
        k = torch.zeros(n, D, device="cuda")
        k[:, 0] = 2.0 ** 60
        k[:160, 0] = float("inf")
        set_keys(s, b, k)
    for b in range(2, len(ctx)):
        set_keys(s, b, torch.full((41, D), 2.0 ** 60, device="cuda"))
    s["q"].zero_()
    s["q"][:, :, 0] = -2.0 ** 60
    with_workspace(ds, s)
    ds.verify_attention(**s, scale=1.0)
    assert ds.get_error() == 0
    # every weight that is not nothing is the same
    check_attention(s, int(start[-1]), 1.0)


def test_negative_context_with_rows(ds):  # noqa: F811
    """A length out of range is recorded and clamped, a context below zero as well."""
    s, start = make_attention([0, 40], [2, 1], 4, 2, 64, 16, 6)
    with_workspace(ds, s)
    s["context"][0] = -5
    ds.verify_attention(**s)
    assert ds.get_error() == 7
    s["context"][0] = 0
    check_attention(s, int(start[-1]), 64 ** -0.5)
    # without rows any context will do
    s["context"][0], s["row_start"] = -5, i32([0, 0, 1])
    ds.verify_attention(**s)
    assert ds.get_error() == 0


def test_longest_context(ds):  # noqa: F811
    """A context of 2^31 - 2 tokens (its pages are the same few over and over): the last tile's
    end is past 32 bits, and the key behind the last one stays hidden."""
    import torch
    D, ps = 64, 16
    pages = torch.zeros(1, (1 << 31) // ps, dtype=torch.int32, device="cuda")
    pages[0, -1] = 1
    k, v = (torch.zeros(2, 1, ps, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[1, 0, 14, 0], k[1, 0, 15, 0] = 60.0, 120.0
    v[1, 0, 14], v[1, 0, 15] = 3.0, 100.0
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 1.0
    s = dict(q=q, k_cache=k, v_cache=v, pages=pages, context=i32([2 ** 31 - 2]),
             row_start=i32([0, 1]), out=torch.full_like(q, 9.0))
    with_workspace(ds, s)
    ds.verify_attention(**s, scale=1.0)
    assert ds.get_error() == 0
    # e^60 beside 2^31 keys of weight 1: three, to 2^-55
    assert bool((s["out"] == 3.0).all())


@pytest.mark.parametrize("B, gamma", [(64, 16), (600, 4)])
def test_layout_without_its_cluster(ds, B, gamma):  # noqa: F811
    """A grid of several CTAs whose cluster is missing: reported, and nothing is touched."""
    from test_gpu_verify_pass import STATE, check_layout, make_layout, run_layout
    import verify_pass_ref as ref
    s = make_layout(B, gamma, 16, 500, B, spare=2 * B)
    d = {k: i32(s[k]) for k in STATE}
    for k, n in (("row_start", B + 1), *((k, B * (gamma + 1)) for k in ("position", "slot", "token"))):
        d[k] = i32(np.full(n, -7))
    before = {k: t.clone() for k, t in d.items()}
    ds.debug_barrier_extra(1)
    try:
        run_layout(ds, s, gamma, 16, out=d)
        assert ds.get_error() == 8
    finally:
        ds.debug_barrier_extra(0)
    for k, t in before.items():
        assert bool((d[k] == t).all()), k
    run_layout(ds, s, gamma, 16, out=d)
    assert ds.get_error() == 0
    check_layout(d, ref.layout(*(s[k] for k in ("L", "context", "held", "pages", "free_pages",
                                                "free_count")), 16, s["anchor"], s["x"]))
