"""The verification pass on the GPU against plain 64-bit implementations."""
import numpy as np
import pytest

import verify_pass_ref as ref
from helpers import dev

pytestmark = pytest.mark.gpu

NAN_BITS = 0x7FC0                 # a bf16 NaN, in every cache slot that no token owns


@pytest.fixture(scope="module")
def ds():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import speculative_decoding_drafter_head_b200 as m
    m.load()
    assert m.get_error() == 0
    return m


def i32(a):
    import torch
    return dev(np.asarray(a, np.int32), torch.int32)


def host(t):
    return t.cpu().numpy()


# ------------------------------------------------------------------------------- layout
STATE = ("L", "context", "rows", "pages", "held", "free_pages", "free_count")


def make_layout(B, gamma, ps, ctx_hi, seed, spare=1000, idle=0.1):
    """A cache between two steps, and the step's lengths and drafts."""
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_hi + 1, B)
    ctx[rng.random(B) < idle] = -1
    held = -(-np.maximum(ctx, 0) // ps)
    more = rng.random(B) < 0.5
    held[more] += rng.integers(0, gamma // ps + 3, B)[more]
    width = int(-(-(ctx_hi + gamma + 1) // ps) + gamma // ps + 3)
    n = int(held.sum())
    ids = rng.permutation(n + spare)
    pages = np.full((B, width), -1)
    pages[np.arange(width)[None] < held[:, None]] = ids[:n]
    free = np.full(n + spare, -1)
    free[:spare] = ids[n:]
    return dict(L=rng.integers(0, gamma + 1, B), context=ctx, rows=np.zeros(B), pages=pages,
                held=held, free_pages=free, free_count=np.array([spare]),
                anchor=rng.integers(0, 1 << 20, B), x=rng.integers(0, 1 << 20, (B, gamma)))


def run_layout(ds, s, gamma, ps, accepted=None, tokens=True, stream=None, out=None):
    import torch
    B = len(s["L"])
    cap = B * (gamma + 1)
    d = out or {k: i32(s[k]) for k in STATE}
    if out is None:
        for k, n in (("row_start", B + 1), ("position", cap), ("slot", cap), ("token", cap)):
            d[k] = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    more = dict(anchor=i32(s["anchor"]), x=i32(s["x"]), token=d["token"]) if tokens else {}
    ds.verify_layout(*(d[k] for k in STATE), d["row_start"], d["position"], d["slot"], ps, gamma,
                     accepted=None if accepted is None else i32(accepted), stream=stream, **more)
    return d


def check_layout(d, want, tokens=True):
    for k in STATE + ("row_start",):
        np.testing.assert_array_equal(host(d[k]), np.asarray(want[k]), err_msg=k)
    n = want["row_start"][-1]
    for k in ("position", "slot") + (("token",) if tokens else ()):
        np.testing.assert_array_equal(host(d[k])[:n], want[k], err_msg=k)
        assert (host(d[k])[n:] == -7).all(), k           # entries behind the last row


@pytest.mark.parametrize("B, gamma, ps, ctx_hi, seed", [
    (1, 0, 1, 0, 0), (1, 16, 16, 900, 1), (3, 4, 4, 9, 2), (31, 7, 16, 300, 3), (33, 16, 3, 100, 4),
    (64, 16, 16, 8000, 5), (511, 1, 32, 50, 6), (512, 8, 16, 2000, 7), (513, 5, 128, 4000, 8),
    (1024, 24, 32, 16000, 9), (4096, 3, 16, 700, 10), (2500, 0, 7, 100, 11),
])
def test_layout(ds, B, gamma, ps, ctx_hi, seed):
    s = make_layout(B, gamma, ps, ctx_hi, seed, spare=B * (gamma // ps + 2))
    want = ref.layout(*(s[k] for k in ("L", "context", "held", "pages", "free_pages", "free_count")),
                      ps, s["anchor"], s["x"])
    d = run_layout(ds, s, gamma, ps)
    check_layout(d, want)
    assert ds.get_error() == 0 and not want["cut"]
    # the same lengths again: nothing moves
    run_layout(ds, s, gamma, ps, out=d)
    check_layout(d, want)
    # without drafts, and with every request ended: the pages go back
    s2 = {k: host(d[k]) for k in STATE} | dict(anchor=s["anchor"], x=s["x"])
    s2["context"] = np.full(B, -1)
    want = ref.layout(*(s2[k] for k in ("L", "context", "held", "pages", "free_pages", "free_count")),
                      ps)
    d = run_layout(ds, s2, gamma, ps, tokens=False)
    check_layout(d, want, tokens=False)
    assert want["row_start"][-1] == 0 and sum(want["held"]) == 0 and ds.get_error() == 0


@pytest.mark.parametrize("spare", [0, 1, 5, 40])
@pytest.mark.parametrize("B, gamma, ps", [(7, 9, 4), (600, 6, 4)])
def test_layout_out_of_pages(ds, spare, B, gamma, ps):
    s = make_layout(B, gamma, ps, 60, 20 + spare, spare=spare, idle=0.0)
    s["held"] = np.minimum(s["held"], -(-s["context"] // ps))     # nothing to give back
    want = ref.layout(*(s[k] for k in ("L", "context", "held", "pages", "free_pages", "free_count")),
                      ps, s["anchor"], s["x"])
    d = run_layout(ds, s, gamma, ps)
    check_layout(d, want)
    assert ds.get_error() == (9 if want["cut"] else 0)
    assert want["cut"] or spare == 40


def test_layout_block_table_ends(ds):
    # the table has room for 8 tokens: request 0 stands at 6 and wants 4, request 1 is full
    s = dict(L=[3, 2], context=[6, 8], rows=[0, 0], pages=[[0, 1], [2, 3]], held=[2, 2],
             free_pages=[4, 5, 6, 7], free_count=[4], anchor=[1, 2], x=np.ones((2, 3)))
    want = ref.layout(*(s[k] for k in ("L", "context", "held", "pages", "free_pages")), 4, 4,
                      s["anchor"], s["x"])
    check_layout(run_layout(ds, s, 3, 4), want)
    assert want["rows"] == [2, 0] and ds.get_error() == 9


@pytest.mark.parametrize("change, status", [
    (dict(L=[9, 0]), 7), (dict(L=[-1, 0]), 7), (dict(context=[-5, 0]), 7),
    (dict(context=[1 << 30, 0]), 7), (dict(held=[-3, 0]), 7), (dict(free_count=[-1]), 7),
    (dict(free_count=[99]), 7), (dict(free_pages=[0, 99, 99, 99]), 10),
    (dict(free_pages=[0, -4, -4, -4]), 10),
])
def test_layout_bad_state(ds, change, status):
    s = dict(L=[3, 0], context=[2, 0], rows=[0, 0], pages=[[3, -1, -1], [-1, -1, -1]], held=[1, 0],
             free_pages=[0, 1, 2, 3], free_count=[3], anchor=[1, 2], x=np.ones((2, 3)))
    s.update(change)
    run_layout(ds, s, 3, 4)
    assert ds.get_error() == status


def test_layout_prompt_then_steps(ds):
    """A prompt, then steps that keep part of their drafts, against the plain form step by step."""
    rng = np.random.default_rng(5)
    B, ps, width, num = 9, 16, 90, 500
    s = dict(L=rng.integers(0, 1000, B), context=np.zeros(B), rows=np.zeros(B),
             pages=np.full((B, width), -1), held=np.zeros(B), free_pages=rng.permutation(num),
             free_count=[num], anchor=np.zeros(B), x=np.zeros((B, 0)))
    accepted = None
    for step in range(8):
        gamma = 1000 if step == 0 else 12
        want = ref.layout(*(s[k] for k in ("L", "context", "held", "pages", "free_pages")),
                          s["free_count"][0], ps, accepted=accepted, rows=s["rows"])
        d = run_layout(ds, s, gamma, ps, accepted=accepted, tokens=False)
        check_layout(d, want, tokens=False)
        assert ds.get_error() == 0
        s = {k: host(d[k]) for k in STATE}
        accepted = s["L"] if step == 0 else rng.integers(-1, 13, B)
        s["L"] = rng.integers(0, 13, B)
        s["anchor"], s["x"] = np.zeros(B), np.zeros((B, 0))
        if step == 4:
            s["context"] = np.where(np.arange(B) == 3, -1, s["context"])   # request 3 ended
        if step == 5:                                                      # and another came
            s["context"] = np.where(np.arange(B) == 3, 0, s["context"])
            accepted[3] = -1


# ---------------------------------------------------------------- norm, rotation, cache write
def make_norm(cap, n, Hq, Hkv, D, rot, seed, gap=0, weights=(True, True), ps=16, far=5000):
    import torch
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    width = (Hq + 2 * Hkv) * D
    num = -(-cap // ps) + 2
    s = dict(qkv=(torch.randn(cap, width + gap, generator=g) * 1.5).bfloat16().cuda()[:, :width],
             position=i32(rng.integers(0, far + 1, cap)), slot=i32(rng.permutation(num * ps)[:cap]),
             n_rows=i32([n]), q_out=torch.full((cap, Hq, D), 5.0).bfloat16().cuda(),
             k_cache=torch.full((num, Hkv, ps, D), 6.0).bfloat16().cuda(),
             v_cache=torch.full((num, Hkv, ps, D), 7.0).bfloat16().cuda())
    w = [(torch.randn(D, generator=g) * 0.3 + 1).bfloat16().cuda() if on else None for on in weights]
    inv = (1e6 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)).float().cuda() \
        if rot else None
    return s, w, inv


def check_norm(s, w, inv, before, eps, interleaved, rope_scale, skip=()):
    n, cap = int(s["n_rows"].item()), s["position"].numel()
    Hq, D = s["q_out"].shape[1:]
    Hkv, ps = s["k_cache"].shape[1:3]
    x = s["qkv"][:n].double().cpu().numpy().reshape(n, Hq + 2 * Hkv, D)
    pos, slot = host(s["position"])[:n], host(s["slot"])[:n]
    f = None if inv is None else inv.cpu().numpy()
    wf = [None if t is None else t.double().cpu().numpy() for t in w]
    q = ref.head(x[:, :Hq], wf[0], eps, pos, f, interleaved, rope_scale)
    k = ref.head(x[:, Hq:Hq + Hkv], wf[1], eps, pos, f, interleaved, rope_scale)

    def near(got, want):
        # one rounding to bf16, half a step: 2^-8 relative; before it fp32 work on the pair:
        # the norm's sum, root and products (under 16 roundings of 2^-24 and the 2-ulp root),
        # the sines (4 x 2^-24 and the angle's 2^-23), the products: under 64 x 2^-24 of the
        # pair's larger member, itself at most the head's largest channel
        big = np.abs(want).max(-1, keepdims=True) * 2.0
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * big + 1e-30).all()

    got_q = s["q_out"].double().cpu().numpy()
    near(got_q[:n], q)
    assert (got_q[n:] == before["q_out"][n:]).all()       # rows behind the count
    keep = np.ones(n, bool)
    keep[list(skip)] = False
    for name, want, exact in (("k_cache", k, False), ("v_cache", x[:, Hq + Hkv:], True)):
        got = s[name].double().cpu().numpy()
        at = (slot[keep] // ps, slice(None), slot[keep] % ps)
        if exact:
            assert (got[at] == want[keep]).all()
        else:
            near(got[at], want[keep])
        untouched = np.ones(got.shape[:1] + got.shape[2:3], bool)
        untouched[slot[keep] // ps, slot[keep] % ps] = False
        assert (got.transpose(0, 2, 1, 3)[untouched] ==
                before[name].transpose(0, 2, 1, 3)[untouched]).all(), name


def copies(s):
    return {k: s[k].double().cpu().numpy() for k in ("q_out", "k_cache", "v_cache")}


@pytest.mark.parametrize("cap, n, Hq, Hkv, D, rot, interleaved, gap, weights, far", [
    (1, 1, 1, 1, 64, 64, False, 0, (True, True), 0),
    (1, 1, 32, 8, 128, 128, False, 0, (True, True), 900),
    (5, 3, 3, 1, 64, 32, True, 8, (True, False), 50),
    (9, 0, 4, 2, 128, 128, False, 0, (True, True), 50),
    (70, 69, 15, 5, 64, 16, False, 40, (False, True), 5000),
    (33, 33, 7, 7, 128, 96, True, 0, (False, False), 1 << 20),
    (33, 32, 8, 1, 128, 64, False, 200, (True, True), (1 << 31) - 1),
    (17, 17, 6, 2, 128, 0, False, 0, (True, True), 10),
    (1203, 1190, 14, 2, 128, 128, False, 0, (True, True), 131072),
    (2001, 1999, 9, 3, 64, 48, True, 0, (True, True), 131072),
    (1901, 1877, 25, 3, 128, 96, True, 0, (True, True), 131072),   # two warps to a row
    (3701, 3655, 13, 5, 128, 128, False, 8, (True, False), 131072),   # and one
    (1500, 2000, 2, 2, 64, 64, False, 0, (True, True), 100),     # the count is clamped
])
def test_norm_rope_store(ds, cap, n, Hq, Hkv, D, rot, interleaved, gap, weights, far):
    s, w, inv = make_norm(cap, n, Hq, Hkv, D, rot, cap + rot, gap, weights, far=far)
    if n > 4:                                              # tiny, huge and constant heads
        s["qkv"][1] *= 1e-6
        s["qkv"][2] *= 1e6
        s["qkv"][3] = 0.5
    before = copies(s)
    ds.qk_norm_rope_store(**s, q_weight=w[0], k_weight=w[1], eps=1e-6, inv_freq=inv,
                          interleaved=interleaved, rope_scale=1.25)
    assert ds.get_error() == 0
    s["n_rows"].clamp_(max=cap)
    check_norm(s, w, inv, before, 1e-6, interleaved, 1.25)


def test_norm_bad_slots(ds):
    s, w, inv = make_norm(20, 20, 4, 2, 128, 128, 3)
    s["slot"][4], s["slot"][11] = -1, s["k_cache"].shape[0] * 16
    before = copies(s)
    ds.qk_norm_rope_store(**s, q_weight=w[0], k_weight=w[1], inv_freq=inv)
    assert ds.get_error() == 10
    check_norm(s, w, inv, before, 1e-6, False, 1.0, skip=(4, 11))


# ---------------------------------------------------------------------------- attention
def make_attention(ctx, rows, Hq, Hkv, D, ps, seed, cap_more=0, q_scale=2.0, spread=True):
    """Caches whose unowned slots are NaN, block tables with ids past their end."""
    import torch
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    ctx, rows = np.asarray(ctx, np.int64), np.asarray(rows, np.int64)
    B = len(ctx)
    length = np.where(rows > 0, np.maximum(ctx, 0) + rows, 0)
    count = -(-length // ps)
    num = int(count.sum()) + 3
    width = max(int(count.max()), 1) + 2
    pages = np.full((B, width), num + 5)
    ids = rng.permutation(num) if spread else np.arange(num)
    pages[np.arange(width)[None] < count[:, None]] = ids[:int(count.sum())]
    start = np.zeros(B + 1, np.int64)
    np.cumsum(rows, out=start[1:])
    cap = int(start[-1]) + cap_more
    caches = []
    for _ in range(2):
        c = torch.randn(num, Hkv, ps, D, generator=g, device="cuda").bfloat16()
        owned = np.zeros((num, ps), bool)
        for b in range(B):
            for j in range(int(count[b])):
                owned[pages[b, j], :max(0, min(ps, int(length[b]) - j * ps))] = True
        c.permute(0, 2, 1, 3)[~torch.from_numpy(owned).cuda()] = float("nan")
        caches.append(c)
    q = (torch.randn(max(cap, 1), Hq, D, generator=g, device="cuda") * q_scale).bfloat16()
    return dict(q=q, k_cache=caches[0], v_cache=caches[1], pages=i32(pages), context=i32(ctx),
                row_start=i32(start), out=torch.full_like(q, 9.0),
                workspace=torch.empty(0, dtype=torch.uint8, device="cuda")), start


def with_workspace(ds, s):
    import torch
    Hq, D = s["q"].shape[1:]
    size = ds.verify_attention_workspace_bytes(Hq, s["k_cache"].shape[1], D)
    s["workspace"] = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    return s


def reference_attention(s, scale):
    """(out, sum p |v|) in fp64 on the GPU, row group by row group, from the definition."""
    import torch
    D = s["q"].shape[2]
    Hkv, ps = s["k_cache"].shape[1:3]
    start, ctx = host(s["row_start"]), host(s["context"])
    out = s["q"].double() * 0
    mag = out.clone()
    for b in range(len(ctx)):
        a, e = int(start[b]), int(start[b + 1])
        if a == e:
            continue
        n, rows = int(ctx[b]) + e - a, e - a
        at = s["pages"][b, :-(-n // ps)].long()
        k, v = (c[at].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].double()
                for c in (s["k_cache"], s["v_cache"]))
        q = s["q"][a:e].double().reshape(rows, Hkv, -1, D).permute(1, 2, 0, 3)
        sc = torch.einsum("hgid,hjd->hgij", q, k) * scale
        hidden = torch.ones(rows, n, dtype=torch.bool, device="cuda").triu(int(ctx[b]) + 1)
        p = torch.softmax(sc.masked_fill(hidden, float("-inf")), -1)
        for dst, val in ((out, v), (mag, v.abs())):
            dst[a:e] = torch.einsum("hgij,hjd->ihgd", p, val).reshape(rows, -1, D)
    return out, mag


def check_attention(s, total, scale):
    out, mag = reference_attention(s, scale)
    got = s["out"].double()
    # the output's rounding (2^-8 of it), the weights' (2^-8 each, at most 2^-8 sum p|v - o|,
    # below 2 x 2^-8 sum p|v|), and fp32 scores: |score| stays under 2^7 here, so their error
    # under D x 2^-24 x 2^7 < 2^-10 (as a weight's relative error, of either sign, like the
    # rounding)
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -7 + 2.0 ** -9) * mag
    err = (got - out).abs()
    assert bool((err <= tol)[:total].all()), float((err / tol)[:total].max())
    assert bool((s["out"][total:] == 9.0).all())           # rows behind the last request


CASES = [
    # ctx, rows, Hq, Hkv, D, ps
    ([0], [1], 1, 1, 64, 16),                               # one token, no history
    ([0], [1], 32, 8, 128, 16),
    ([699], [1], 32, 8, 128, 16),
    ([126, 127, 128], [1, 1, 1], 8, 8, 128, 128),           # around a tile's end
    ([127, 126, 120, 0], [2, 2, 17, 17], 8, 2, 128, 16),    # rows across a tile's end
    ([5, -1, 300, -1, 40], [3, 0, 1, 0, 2], 10, 5, 64, 32),  # idle slots
    ([-1, -1], [0, 0], 4, 4, 64, 16),                       # nothing at all
    ([9000, 70, 1 << 30], [0, 3, 0], 4, 4, 64, 16),         # any context without rows
    ([1000, 3, 77], [17, 9, 1], 32, 8, 128, 16),            # 68 rows to a key head
    ([513], [25], 64, 8, 128, 64),                          # 200 rows to a key head
    ([63, 260], [7, 8], 112, 1, 128, 32),                   # every token a tile of rows
    ([33, 1029], [5, 3], 111, 1, 64, 16),                   # an odd group that fills no tile
    ([0], [300], 4, 2, 64, 16),                             # a prompt
    ([200], [129], 7, 1, 128, 128),                         # a piece of a prompt
    ([20011], [4], 12, 4, 128, 16),                         # one long request
    ([9000, 17, 4500, 1], [2, 17, 6, 1], 24, 3, 64, 64),    # long and short together
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(ds, case):
    ctx, rows, Hq, Hkv, D, ps = CASES[case]
    s, start = make_attention(ctx, rows, Hq, Hkv, D, ps, 40 + case, cap_more=case % 3)
    with_workspace(ds, s)
    ds.verify_attention(**s)
    assert ds.get_error() == 0
    check_attention(s, int(start[-1]), D ** -0.5)


@pytest.mark.parametrize("B, gamma, hi, Hq, Hkv, D, ps", [
    (200, 0, 300, 8, 4, 128, 16), (64, 16, 2000, 32, 8, 128, 16), (1000, 3, 40, 4, 2, 64, 16),
    (4096, 0, 5, 2, 1, 64, 16), (37, 24, 700, 15, 5, 64, 128), (150, 8, 900, 5, 5, 128, 32),
])
def test_attention_batches(ds, B, gamma, hi, Hq, Hkv, D, ps):
    rng = np.random.default_rng(B)
    ctx, rows = rng.integers(0, hi + 1, B), rng.integers(0, gamma + 2, B)
    s, start = make_attention(ctx, rows, Hq, Hkv, D, ps, B, cap_more=5)
    with_workspace(ds, s)
    ds.verify_attention(**s)
    assert ds.get_error() == 0
    check_attention(s, int(start[-1]), D ** -0.5)
    first = s["out"].clone()
    s["workspace"].fill_(0x3C)
    ds.verify_attention(**s)                                # the same bits every time
    assert bool((s["out"] == first).all())


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.02])
def test_attention_scales(ds, scale):
    s, start = make_attention([300, 5], [3, 9], 8, 2, 128, 16, 3)
    with_workspace(ds, s)
    ds.verify_attention(**s, scale=scale)
    check_attention(s, int(start[-1]), scale)


def test_attention_rising_scores(ds):
    """Scores that climb along the keys, by far more than fp32's exponent holds in one step:
    the running maximum has to follow."""
    import torch
    s, start = make_attention([1500, 900], [4, 2], 8, 2, 128, 16, 9, spread=False)
    n = s["k_cache"].shape[0] * 16
    k = s["k_cache"].permute(0, 2, 1, 3).reshape(n, 2, 128)
    k[:, :, 1:] = torch.where(k[:, :, 1:].isnan(), k[:, :, 1:], torch.zeros_like(k[:, :, 1:]))
    ramp = torch.arange(n, device="cuda").float().bfloat16()[:, None].expand(n, 2)
    k[:, :, 0] = torch.where(k[:, :, 0].isnan(), k[:, :, 0], ramp)
    s["k_cache"] = k.reshape(-1, 16, 2, 128).permute(0, 2, 1, 3).contiguous()
    s["q"][:, :, 0] = torch.tensor([8.0, -8.0, 1.0, 0.0, 40.0, 0.125, -0.5, 3.0]).cuda().bfloat16()
    with_workspace(ds, s)
    ds.verify_attention(**s, scale=1.0)
    assert ds.get_error() == 0
    out, mag = reference_attention(s, 1.0)
    # scores are exact here (bf16 times small integers' sums of one product), so only the
    # weights' and the output's roundings and exp's argument remain: the largest kept
    # argument is under 2^7, where its rounding is 2^-18
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -7 + 2.0 ** -9) * mag
    assert bool(((s["out"].double() - out).abs() <= tol).all())


@pytest.mark.parametrize("D", [64, 128])
def test_attention_scores_minus_infinity(ds, D):
    """Keys whose scores are -inf weigh nothing, however low the others are, in whole tiles too."""
    import torch
    s, start = make_attention([400, 60], [3, 2], 4, 2, D, 16, 12, spread=False)
    n = s["k_cache"].shape[0] * 16
    k = s["k_cache"].permute(0, 2, 1, 3).reshape(n, 2, D).nan_to_num(0.0)
    k[:, :, 0] = -300.0 - 4.0 * (torch.arange(n, device="cuda") % 8)[:, None]
    k[:300, 0, 0] = float("-inf")                           # request 0: two whole tiles and more
    k[410:450, :, 0] = float("-inf")                        # request 1
    s["k_cache"] = k.reshape(-1, 16, 2, D).permute(0, 2, 1, 3).contiguous()
    s["q"].zero_()
    s["q"][:, :, 0] = 1.0
    with_workspace(ds, s)
    ds.verify_attention(**s, scale=1.0)
    assert ds.get_error() == 0
    out, mag = reference_attention(s, 1.0)
    assert bool(out[:int(start[-1])].isfinite().all())
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -7 + 2.0 ** -9) * mag
    assert bool(((s["out"].double() - out).abs() <= tol).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_attention_hidden_values(ds, value):
    """A later row's key or value that is not finite reaches the rows that see it, no other."""
    s, start = make_attention([250, 100], [8, 8], 8, 2, 128, 16, 4)
    pages = host(s["pages"])
    for cache, b, pos in (("v_cache", 0, 254), ("k_cache", 1, 103), ("v_cache", 1, 106)):
        s[cache][int(pages[b, pos // 16]), 1, pos % 16, 17] = value
    with_workspace(ds, s)
    ds.verify_attention(**s)
    got = s["out"].double()
    clean = {k: t for k, t in s.items()}
    clean["k_cache"], clean["v_cache"] = (torch_nan_to(s[k]) for k in ("k_cache", "v_cache"))
    out, mag = reference_attention(clean, 128 ** -0.5)
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -7 + 2.0 ** -9) * mag
    ok = (got - out).abs() <= tol
    assert bool(ok[:, :4].all())                            # the other key head
    assert bool(ok[:4].all())                               # request 0, rows before the value
    assert bool(ok[4:8, 4:, :17].all()) and bool(ok[4:8, 4:, 18:].all())
    bad = got[4:8, 4:, 17]
    assert bool(bad.isnan().all()) if value != value else bool((bad == value).all())
    assert bool(ok[8:11].all())                             # request 1, rows before the key


def torch_nan_to(t):
    import torch
    return torch.nan_to_num(t, nan=0.0, posinf=0.0, neginf=0.0)


def test_attention_bad_pages(ds):
    import torch
    s, start = make_attention([100, 40], [2, 2], 4, 2, 64, 16, 6)
    s["k_cache"], s["v_cache"] = (torch_nan_to(s[k]) for k in ("k_cache", "v_cache"))
    good = s["pages"].clone()
    s["pages"][0, 2], s["pages"][1, 1] = -3, s["k_cache"].shape[0]
    with_workspace(ds, s)
    ds.verify_attention(**s)
    assert ds.get_error() == 10
    s["pages"] = torch.where(s["pages"] == -3, 0, s["pages"])
    s["pages"][1, 1] = 0
    check_attention(s, int(start[-1]), 64 ** -0.5)          # read as page 0
    # lengths past the block table are clamped to it
    s["pages"], s["context"] = good, i32([1 << 20, 40])
    ds.verify_attention(**s)
    assert ds.get_error() == 7


def test_attention_offsets_past_32_bits(ds):
    """A cache of more than 2^32 elements: a request in its last pages."""
    import torch
    num, Hkv, ps, D = 70000, 8, 64, 128                     # 4.6e9 elements, 9 GB each
    k = torch.empty(num, Hkv, ps, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    for c in (k, v):
        c[-4:] = torch.randn(4, Hkv, ps, D, generator=g, device="cuda").bfloat16()
    q = torch.randn(3, 16, D, generator=g, device="cuda").bfloat16()
    s = dict(q=q, k_cache=k, v_cache=v, pages=i32([[num - 1, num - 3, num - 2, num - 4]]),
             context=i32([200]), row_start=i32([0, 3]), out=torch.full_like(q, 9.0))
    with_workspace(ds, s)
    ds.verify_attention(**s)
    assert ds.get_error() == 0
    check_attention(s, 3, D ** -0.5)


# ------------------------------------------------------------------- the pass as it is used
def test_pass_together_captured(ds):
    """schedule -> layout -> norm/rope/store -> attention -> verify, captured once and
    replayed with other lengths and inputs, against the plain forms chained."""
    import torch
    rng = np.random.default_rng(8)
    B, gamma, ps, Hq, Hkv, D, width, num = 12, 8, 16, 8, 2, 128, 20, 200
    cap = B * (gamma + 1)
    s = dict(L=np.zeros(B), context=np.zeros(B), rows=np.zeros(B), pages=np.full((B, width), -1),
             held=np.zeros(B), free_pages=rng.permutation(num), free_count=[num])
    d = {k: i32(s[k]) for k in STATE}
    for k, n in (("row_start", B + 1), ("position", cap), ("slot", cap), ("token", cap)):
        d[k] = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    anchor, x, accepted = i32(np.zeros(B)), i32(np.zeros((B, gamma))), i32(np.full(B, -1))
    target, bonus = i32(np.zeros((B, gamma + 1))), i32(np.zeros(B))
    P = torch.zeros(B, gamma, dtype=torch.float32, device="cuda")
    Tstep = dev(np.where(np.arange(B * (gamma + 1) + 1) < 60, 10.0,
                         10.0 + 0.3 * (np.arange(B * (gamma + 1) + 1) - 60)))
    N, F = i32([0]), torch.zeros(1, dtype=torch.float64, device="cuda")
    ws = torch.empty(ds.workspace_bytes(B, gamma, 8), dtype=torch.uint8, device="cuda")
    aws = torch.empty(ds.verify_attention_workspace_bytes(Hq, Hkv, D), dtype=torch.uint8,
                      device="cuda")
    qkv = torch.zeros(cap, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda")
    w = (torch.randn(D) * 0.3 + 1).bfloat16().cuda()
    inv = (1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    kc, vc = (torch.full((num, Hkv, ps, D), float("nan")).bfloat16().cuda() for _ in range(2))
    q, out = (torch.full((cap, Hq, D), 9.0).bfloat16().cuda() for _ in range(2))

    def step():
        ds.schedule_prefix(P, Tstep, d["L"], N, F, ws)
        ds.verify_layout(*(d[k] for k in STATE), d["row_start"], d["position"], d["slot"], ps,
                         gamma, anchor=anchor, x=x, token=d["token"], accepted=accepted)
        ds.qk_norm_rope_store(qkv, d["position"], d["slot"], d["row_start"][B:], q, kc, vc,
                              q_weight=w, k_weight=w, inv_freq=inv)
        ds.verify_attention(q, kc, vc, d["pages"], d["context"], d["row_start"], out, aws)
        ds.verify_prefix(x, d["L"], target, accepted, bonus)

    ds.schedule_prefix(P, Tstep, i32(np.zeros(B)), N, F, ws)      # loads the kernels
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    state = dict(s)
    acc_prev = np.full(B, -1)
    hist = {}                                                     # (request, position) -> (k, v)
    for t in range(9):
        xs = rng.integers(0, 50, (B, gamma))
        tg = np.concatenate([xs, rng.integers(0, 50, (B, 1))], 1)
        tg[:, :-1] = np.where(rng.random((B, gamma)) < 0.8, tg[:, :-1], 60)
        scores = np.cumprod(rng.uniform(0.6, 1.0, (B, gamma)), 1).astype(np.float32)
        an = rng.integers(0, 50, B)
        for dst, src in ((x, xs), (target, tg), (anchor, an)):
            dst.copy_(i32(src))
        P.copy_(dev(scores))
        qkv.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert ds.get_error() == 0
        L = host(d["L"])                                          # never cut here
        want = ref.layout(L, state["context"], state["held"], state["pages"], state["free_pages"],
                          state["free_count"][0], ps, an, xs, accepted=acc_prev, rows=state["rows"])
        assert not want["cut"]
        n = want["row_start"][-1]
        for k in STATE + ("row_start",):
            np.testing.assert_array_equal(host(d[k]), np.asarray(want[k]), err_msg=k)
        for k in ("position", "slot", "token"):
            np.testing.assert_array_equal(host(d[k])[:n], want[k], err_msg=k)
        # keys and values as the cache holds them, by request and position
        rows = qkv[:n].double().cpu().numpy().reshape(n, Hq + 2 * Hkv, D)
        pos = np.asarray(want["position"])
        k64 = ref.head(rows[:, Hq:Hq + Hkv], w.double().cpu().numpy(), 1e-6, pos,
                       inv.cpu().numpy(), False, 1.0)
        at = np.asarray(want["slot"])
        kg = kc.double().cpu().numpy()[at // ps, :, at % ps]
        assert (np.abs(kg - k64) <= 2.0 ** -8 * np.abs(k64) + 2.0 ** -16).all()
        req = np.repeat(np.arange(B), want["rows"])
        for r in range(n):
            hist[int(req[r]), int(pos[r])] = (kg[r], rows[r, Hq + Hkv:])
        qg = q.double().cpu().numpy()
        og = out.double().cpu().numpy()
        for r in rng.permutation(n)[:12]:
            keys = [hist[int(req[r]), j] for j in range(int(pos[r]) + 1)]
            for h in range(Hq):
                kk = np.stack([a[0][h // 4] for a in keys])
                vv = np.stack([a[1][h // 4] for a in keys])
                sc = kk @ qg[r, h] * D ** -0.5
                p = np.exp(sc - sc.max())
                p /= p.sum()
                tol = 2.0 ** -8 * np.abs(p @ vv) + (2.0 ** -7 + 2.0 ** -9) * (p @ np.abs(vv))
                assert (np.abs(og[r, h] - p @ vv) <= tol).all()
        first = np.array([next((i for i in range(L[b]) if xs[b, i] != tg[b, i]), L[b])
                          for b in range(B)])
        np.testing.assert_array_equal(host(accepted), first)
        acc_prev = first
        state = {k: host(d[k]) for k in STATE}
    assert max(p for _, p in hist) > 20


def test_verify_pass_steps(ds):
    """pipeline.VerifyPass over two layers, with requests that come and go, against the plain
    forms: every row attends to all of its request's tokens that stuck, and to its own step's."""
    import torch
    from speculative_decoding_drafter_head_b200.pipeline import VerifyPass
    rng = np.random.default_rng(3)
    B, gamma, layers, Hq, Hkv, D, ps = 5, 3, 2, 6, 2, 64, 16
    inv = (1e4 ** (-torch.arange(16, dtype=torch.float64) / 16)).float().cuda()
    vp = VerifyPass(B, gamma, layers, Hq, Hkv, D, ps, num_pages=24, max_pages=6, inv_freq=inv,
                    interleaved=True, scale=0.2)
    side = torch.cuda.Stream()
    hist = [{} for _ in range(layers)]
    accepted, ctx, rows = None, np.full(B, -1), np.zeros(B, int)
    for t in range(10):
        if t == 0:
            vp.context.copy_(i32([0, 0, -1, 0, -1]))
            ctx = np.array([0, 0, -1, 0, -1])
        elif t == 4:                                           # request 1 ends, slot 4 starts
            vp.context[1], vp.context[4] = -1, 0
            ctx[1], ctx[4] = -1, 0
            hist = [{k: v for k, v in h.items() if k[0] not in (1, 4)} for h in hist]
            accepted[4] = -1
        if accepted is not None:
            ctx = np.where(ctx >= 0, ctx + np.minimum(accepted + 1, rows), ctx)
        L = rng.integers(0, gamma + 1, B)
        x, anchor = rng.integers(0, 99, (B, gamma)), rng.integers(0, 99, B)
        acc_d = None if accepted is None else i32(accepted)
        d = i32(L), i32(anchor), i32(x)
        torch.cuda.synchronize()
        vp.layout(*d, acc_d, stream=side)
        rows = np.where(ctx >= 0, L + 1, 0)
        req = np.repeat(np.arange(B), rows)
        n = len(req)
        pos = np.concatenate([np.arange(ctx[b], ctx[b] + rows[b]) for b in range(B)])
        side.synchronize()
        np.testing.assert_array_equal(host(vp.position)[:n], pos)
        np.testing.assert_array_equal(host(vp.context), ctx)
        assert int(vp.row_start[-1]) == n
        for layer in range(layers):
            qkv = torch.randn(B * (gamma + 1), (Hq + 2 * Hkv) * D, device="cuda").bfloat16()
            torch.cuda.synchronize()
            out = vp.attend(layer, qkv, stream=side)
            side.synchronize()
            assert ds.get_error() == 0
            r64 = qkv[:n].double().cpu().numpy().reshape(n, Hq + 2 * Hkv, D)
            q = vp.q.double().cpu().numpy()
            want_q = ref.head(r64[:, :Hq], None, 0, pos, inv.cpu().numpy(), True, 1.0)
            assert (np.abs(q[:n] - want_q) <= 2.0 ** -8 * np.abs(want_q) + 2.0 ** -16).all()
            k64 = ref.head(r64[:, Hq:Hq + Hkv], None, 0, pos, inv.cpu().numpy(), True, 1.0)
            k64 = torch.from_numpy(k64).bfloat16().double().numpy()    # one rounding, as stored
            for r in range(n):
                hist[layer][int(req[r]), int(pos[r])] = (k64[r], r64[r, Hq + Hkv:])
            got = out.double().cpu().numpy()
            for r in range(n):
                keys = [hist[layer][int(req[r]), j] for j in range(int(pos[r]) + 1)]
                for h in range(Hq):
                    kk, vv = (np.stack([a[i][h // 3] for a in keys]) for i in range(2))
                    sc = kk @ q[r, h] * 0.2
                    p = np.exp(sc - sc.max())
                    p /= p.sum()
                    # as elsewhere, and a key that rounds the other way: 2^-8 of it, which moves
                    # a score by up to 0.2 x 2^-8 |q| |k| < 2^-2 here, for a few keys of many
                    tol = 2.0 ** -8 * np.abs(p @ vv) + 2.0 ** -5 * (p @ np.abs(vv)) + 1e-6
                    assert (np.abs(got[r, h] - p @ vv) <= tol).all()
        accepted = np.array([rng.integers(0, L[b] + 1) for b in range(B)])
    assert int(vp.free_count) + int(vp.held.sum()) == 24       # no page lost


def test_graphs_that_share_a_workspace(ds):
    """Two captured calls with one workspace, replayed in turn and with other lengths between."""
    import torch
    calls, graphs = [], []
    for i in range(2):
        s, start = make_attention([5000, 700 + i], [3, 17], 16, 2, 128, 32, 90 + i)
        calls.append((with_workspace(ds, s), int(start[-1])))
    calls[1][0]["workspace"] = calls[0][0]["workspace"]
    for s, _ in calls:
        ds.verify_attention(**s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ds.verify_attention(**s)
        graphs.append(g)
    short = i32([100, 9])
    for ctx in (None, short):
        for s, _ in calls:
            if ctx is not None:
                s["context"].copy_(ctx)
            s["out"].fill_(9.0)
        for g in graphs * 2:
            g.replay()
        torch.cuda.synchronize()
        assert ds.get_error() == 0
        for s, total in calls:
            check_attention(s, total, 128 ** -0.5)


def test_two_streams_at_once(ds):
    """Two calls at once with a workspace each, on streams of their own."""
    import torch
    calls = []
    for i in range(2):
        s, start = make_attention([3000 + i, 50], [5, 2], 32, 8, 128, 16, 70 + i)
        calls.append((with_workspace(ds, s), int(start[-1])))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for (s, _), st in zip(calls, streams):
            ds.verify_attention(**s, stream=st)
    torch.cuda.synchronize()
    assert ds.get_error() == 0
    for s, total in calls:
        check_attention(s, total, 128 ** -0.5)


@pytest.mark.parametrize("Hq, rows", [(8, 3), (32, 17)])      # both query tile sizes
def test_attention_reports_timeout(ds, Hq, rows):
    """An arrival that never comes: every wait runs out or sees the abort, the call reports it,
    and the next one is right."""
    import torch
    s, start = make_attention([3000, 40, 700], [rows, 1, rows], Hq, 2, 128, 16, 21)
    with_workspace(ds, s)
    ds.verify_attention(**s)
    assert ds.get_error() == 0
    clean = s["out"].clone()
    ds.set_wait_timeout_ns(200_000_000)
    ds.debug_barrier_extra(1)
    try:
        ds.verify_attention(**s)
        assert ds.get_error() == 6
    finally:
        ds.debug_barrier_extra(0)
        ds.set_wait_timeout_ns(2_000_000_000)
    s["out"].fill_(9.0)
    ds.verify_attention(**s)
    assert ds.get_error() == 0
    assert bool((s["out"] == clean).all())
    check_attention(s, int(start[-1]), 128 ** -0.5)
