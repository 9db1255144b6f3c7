"""The operators of the target model's verification pass, measured.

``verify_layout`` lays the ragged batch of one verification step over a paged key-value
cache, ``qk_norm_rope_store`` normalises and rotates its queries and keys and writes keys
and values into the cache, ``verify_attention`` is the attention of its rows over the cache.
Each is here in its plain form (elementary torch operations in 32 bits, angles in 64) and
as the library's call; ``exact`` computes the same in 64 bits from the definitions.
"""
import math
import zlib

import numpy as np
import torch

own = False

VOCAB = 151936


# ------------------------------------------------------------------------------ cases
def listed():
    layout = dict(op="layout")
    norm = dict(op="norm", weights=True, rope_scale=1.0, gap=0)
    attn = dict(op="attention")
    return [
        # one interactive request: latency only
        dict(layout, name="layout-1", B=1, gamma=16, page=16, ctx_lo=900, ctx_hi=900),
        # the benchmark's batch of 64 requests with blocks of 16 drafts
        dict(layout, name="layout-64", B=64, gamma=16, page=16, ctx_lo=100, ctx_hi=8000),
        # the large batch: 1024 requests, blocks of 24 drafts, wide block tables
        dict(layout, name="layout-1024", B=1024, gamma=24, page=32, ctx_lo=1, ctx_hi=16000),
        # one token of one request: latency only
        dict(norm, name="norm-1", B=1, gamma=0, hq=32, hkv=8, D=128, page=16, rot=128,
             interleaved=False, ctx_lo=900, ctx_hi=900),
        # the benchmark's batch: some 580 rows of 4096 query channels
        dict(norm, name="norm-64", B=64, gamma=16, hq=32, hkv=8, D=128, page=16, rot=128,
             interleaved=False, ctx_lo=100, ctx_hi=8000),
        # interleaved pairs in a part of small heads, no norm, far positions, padded rows of qkv
        dict(norm, name="norm-part", B=96, gamma=8, hq=15, hkv=5, D=64, page=32, rot=32,
             interleaved=True, ctx_lo=20000, ctx_hi=900000, weights=False, rope_scale=1.25, gap=40),
        # the large batch: some 13000 rows
        dict(norm, name="norm-1024", B=1024, gamma=24, hq=32, hkv=8, D=128, page=32, rot=128,
             interleaved=False, ctx_lo=1, ctx_hi=16000),
        # one token of one request with a short history: latency only
        dict(attn, name="attn-1", B=1, gamma=0, hq=32, hkv=8, D=128, page=16, ctx_lo=700,
             ctx_hi=700),
        # one request with a long history: the cache's length is all there is to split
        dict(attn, name="attn-long", B=1, gamma=16, hq=32, hkv=8, D=128, page=16,
             ctx_lo=131000, ctx_hi=131000),
        # small heads without grouping, lengths from one token on
        dict(attn, name="attn-mha", B=40, gamma=7, hq=16, hkv=16, D=64, page=32, ctx_lo=1,
             ctx_hi=5000),
        # the benchmark's batch with its ragged verify lengths
        dict(attn, name="attn-64", B=64, gamma=16, hq=32, hkv=8, D=128, page=16, ctx_lo=500,
             ctx_hi=8000),
        # plain decoding of a large batch, one token each, eight query heads to a key head
        dict(attn, name="attn-decode", B=256, gamma=0, hq=32, hkv=4, D=128, page=64, ctx_lo=500,
             ctx_hi=8000),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("layout", "norm", "attention"))
    page = rng.choice((16, 32, 64, 128))
    if op == "layout":
        hi = _spread(rng, 1, 16000)
        return dict(op=op, B=_spread(rng, 1, 1024), gamma=rng.randint(0, 24), page=page,
                    ctx_lo=rng.randint(1, hi), ctx_hi=hi)
    D = rng.choice((64, 128))
    hkv = rng.choice((1, 2, 3, 4, 5, 8))
    group = rng.choice((1, 2, 3, 4, 5, 7, 8))
    if op == "norm":
        hi = _spread(rng, 1, 900000)
        B = _spread(rng, 1, 1024)
        rows = max(1, min(25, (1024 * 25 * 48 * 128) // (B * (group + 2) * hkv * D)))
        return dict(op=op, B=B, gamma=rng.randint(0, rows - 1), hq=group * hkv, hkv=hkv, D=D,
                    page=page, rot=rng.choice((0, 16, 32, 48, 64, D)), interleaved=rng.random() < 0.5,
                    ctx_lo=rng.randint(1, hi), ctx_hi=hi, weights=rng.random() < 0.7,
                    rope_scale=rng.choice((1.0, 1.0, 1.25)), gap=rng.choice((0, 0, 8, 200)))
    B = _spread(rng, 1, 256)
    gamma = rng.choice((0, 0, rng.randint(1, 24)))
    # at most half the largest case's cache, and less where many rows share a key head
    most = 256 * 8000 * 4 * 128 // (2 * B * hkv * D * max(1, group * (gamma + 1) // 64))
    hi = _spread(rng, 1, max(1, min(131000, most)))
    return dict(op=op, B=B, gamma=gamma, hq=group * hkv, hkv=hkv, D=D, page=page,
                ctx_lo=rng.randint(max(1, hi // 20), hi), ctx_hi=hi)


def _lengths(case):
    """(context, L) of a case's requests, the same for every seed but for their order."""
    text = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    rng = np.random.RandomState(zlib.crc32(text.encode()))
    B = case["B"]
    ctx = rng.randint(case["ctx_lo"], case["ctx_hi"] + 1, B)
    L = rng.randint(0, case["gamma"] + 1, B)
    return ctx.astype(np.int64), L.astype(np.int64)


def _pages_of(n, page):
    return -(-n // page)


# --------------------------------------------------------------------------- preparing
def _i32(a, device):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(device)


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed * 7919 + 17)
    rng = np.random.RandomState(seed % (1 << 31))
    ctx, L = _lengths(case)
    order = rng.permutation(case["B"])
    ctx, L = ctx[order], L[order]
    make = {"layout": _prepare_layout, "norm": _prepare_norm, "attention": _prepare_attention}
    return make[case["op"]](case, ctx, L, rng, gen, device)


def _prepare_layout(case, ctx, L, rng, gen, device):
    B, gamma, page = case["B"], case["gamma"], case["page"]
    table = _pages_of(case["ctx_hi"] + 2 * gamma + 2, page)
    # pages held from the step before: some requests have pages of drafts that were
    # rejected, some ended (idle slots that still hold pages), some are new to their pages
    held = _pages_of(ctx, page)
    tail = rng.random_sample(B) < 0.5
    held = np.where(tail, _pages_of(ctx + rng.randint(0, gamma + 1, B), page), held)
    ended = rng.random_sample(B) < (0.03 if B > 8 else 0.0)
    num = int(_pages_of(ctx + 2 * gamma + 1, page).sum() + 16)
    ctx = np.where(ended, -1, ctx)
    ids = rng.permutation(num)
    pages = np.full((B, table), -1, np.int64)
    place = np.arange(table)[None, :] < held[:, None]
    n = int(held.sum())
    pages[place] = ids[:n]
    free = np.full(num, -1, np.int64)
    free[:num - n] = ids[n:]
    cap = B * (gamma + 1)
    s = dict(case=case, page=page, gamma=gamma, cap=cap, num=num,
             L=_i32(L, device), context=_i32(ctx, device), pages=_i32(pages, device),
             held=_i32(held, device), free_pages=_i32(free, device),
             free_count=_i32([num - n], device),
             anchor=_i32(rng.randint(0, VOCAB, B), device),
             x=_i32(rng.randint(0, VOCAB, (B, max(gamma, 1)))[:, :gamma], device))
    for name, count in (("rows", B), ("row_start", B + 1), ("position", cap), ("slot", cap),
                        ("token", cap)):
        s[name] = torch.full((count,), -1, dtype=torch.int32, device=device)
    return s


def _rows(ctx, L):
    """row_start, and each row's request and place in it."""
    start = np.zeros(len(L) + 1, np.int64)
    np.cumsum(L + 1, out=start[1:])
    b = np.repeat(np.arange(len(L)), L + 1)
    return start, b, np.arange(start[-1]) - start[b]


def _prepare_norm(case, ctx, L, rng, gen, device):
    B, gamma, page, D = case["B"], case["gamma"], case["page"], case["D"]
    hq, hkv, rot = case["hq"], case["hkv"], case["rot"]
    start, b, i = _rows(ctx, L)
    n, cap = int(start[-1]), B * (gamma + 1)
    num = B * (gamma // page + 2)
    # every request's new rows in pages of its own, from wherever its context ends in one
    own_pages = rng.permutation(num).reshape(B, -1)
    at = ctx[b] % page + i
    position = np.full(cap, -1, np.int64)
    slot = np.full(cap, -1, np.int64)
    position[:n] = ctx[b] + i
    slot[:n] = own_pages[b, at // page] * page + at % page
    width = (hq + 2 * hkv) * D
    qkv = torch.randn(cap, width + case["gap"], generator=gen, device=device).mul_(1.7)
    s = dict(case=case, position=_i32(position, device), slot=_i32(slot, device),
             n_rows=_i32([n], device), qkv=qkv.to(torch.bfloat16)[:, :width], eps=1e-6,
             interleaved=case["interleaved"], rope_scale=case["rope_scale"],
             q_out=torch.zeros(cap, hq, D, dtype=torch.bfloat16, device=device),
             k_cache=torch.zeros(num, hkv, page, D, dtype=torch.bfloat16, device=device),
             v_cache=torch.zeros(num, hkv, page, D, dtype=torch.bfloat16, device=device),
             q_weight=None, k_weight=None, inv_freq=None)
    if case["weights"]:
        for name in ("q_weight", "k_weight"):
            w = torch.randn(D, generator=gen, device=device).mul_(0.3).add_(1.0)
            s[name] = w.to(torch.bfloat16)
    if rot:
        j = torch.arange(rot // 2, dtype=torch.float64)
        s["inv_freq"] = (1e6 ** (-2.0 * j / rot)).float().to(device)
    return s


def _prepare_attention(case, ctx, L, rng, gen, device):
    B, gamma, page, D = case["B"], case["gamma"], case["page"], case["D"]
    hq, hkv = case["hq"], case["hkv"]
    start, _, _ = _rows(ctx, L)
    cap = B * (gamma + 1)
    count = _pages_of(ctx + L + 1, page)
    table = int(count.max())
    num = int(count.sum()) + 3
    pages = np.full((B, table), -1, np.int64)
    pages[np.arange(table)[None, :] < count[:, None]] = rng.permutation(num)[:int(count.sum())]
    cache = lambda: torch.randn(num, hkv, page, D, generator=gen, device=device,  # noqa: E731
                                dtype=torch.bfloat16)
    return dict(case=case, k_cache=cache(), v_cache=cache(), pages=_i32(pages, device),
                context=_i32(ctx, device), row_start=_i32(start, device), scale=D ** -0.5,
                longest=int((ctx + L + 1).max()), workspace=None,
                q=torch.randn(cap, hq, D, generator=gen, device=device).mul_(2.0).to(torch.bfloat16),
                out=torch.zeros(cap, hq, D, dtype=torch.bfloat16, device=device))


# ------------------------------------------------------------------------------- passes
def run(state):
    op = state["case"]["op"]
    if op == "layout":
        return _own_layout(state) if own else _plain_layout(state)
    if op == "norm":
        return _own_norm(state) if own else _plain_norm(state)
    return _own_attention(state) if own else _plain_attention(state)


def _own_layout(s):
    import speculative_decoding_drafter_head_b200 as ds
    ds.verify_layout(s["L"], s["context"], s["rows"], s["pages"], s["held"], s["free_pages"],
                     s["free_count"], s["row_start"], s["position"], s["slot"], s["page"],
                     s["gamma"], anchor=s["anchor"], x=s["x"], token=s["token"])
    return {k: s[k] for k in ("L", "rows", "pages", "held", "free_pages", "free_count", "row_start",
                              "position", "slot", "token")}


def _own_norm(s):
    import speculative_decoding_drafter_head_b200 as ds
    ds.qk_norm_rope_store(s["qkv"], s["position"], s["slot"], s["n_rows"], s["q_out"], s["k_cache"],
                          s["v_cache"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                          eps=s["eps"], inv_freq=s["inv_freq"], interleaved=s["interleaved"],
                          rope_scale=s["rope_scale"])
    return {k: s[k] for k in ("q_out", "k_cache", "v_cache")}


def _own_attention(s):
    import speculative_decoding_drafter_head_b200 as ds
    if s["workspace"] is None:   # a program makes it with the cache and keeps it
        size = ds.verify_attention_workspace_bytes(s["case"]["hq"], s["case"]["hkv"], s["case"]["D"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["q"].device)
    ds.verify_attention(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["context"],
                        s["row_start"], s["out"], s["workspace"], scale=s["scale"])
    return s["out"]


def _plain_layout(s):
    ps, num, cap = s["page"], s["num"], s["cap"]
    L, ctx, held, pages = (s[k].long() for k in ("L", "context", "held", "pages"))
    F = s["free_count"].long()
    B, table = pages.shape
    live = ctx >= 0
    want = torch.where(live, torch.minimum(L + 1, table * ps - ctx), 0)
    need = torch.where(live, (ctx + want + ps - 1) // ps, 0)
    back, ask = (held - need).clamp(min=0), (need - held).clamp(min=0)
    back0, ask0 = back.cumsum(0) - back, ask.cumsum(0) - ask
    place = torch.arange(table, device=L.device)[None, :]
    # pages past the need go back on the stack, in request order
    gone = (place >= need[:, None]) & (place < held[:, None])
    to = torch.where(gone, F + back0[:, None] + place - need[:, None], num)
    stack = torch.cat([s["free_pages"].long(), s["free_pages"].new_zeros(1).long()])
    stack = stack.scatter(0, to.reshape(-1), pages.reshape(-1))[:num]
    top = F + back.sum()
    # missing pages come from its top, in request order, as long as it holds any
    grant = torch.minimum(ask, (top - ask0).clamp(min=0))
    kept = torch.minimum(held, need)
    new = (place >= kept[:, None]) & (place < (kept + grant)[:, None])
    take = (top - 1 - ask0[:, None] - (place - kept[:, None])).clamp(0, num - 1)
    pages = torch.where(new, stack[take], pages)
    held = kept + grant
    rows = torch.minimum(want, (held * ps - ctx).clamp(min=0))
    L = torch.where(rows < want, (rows - 1).clamp(min=0), L)
    start = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
    r = torch.arange(cap, device=L.device)
    b = torch.searchsorted(start[1:].contiguous(), r, right=True).clamp(max=B - 1)
    i = (r - start[b]).clamp(0, s["gamma"])
    position = (ctx[b] + i).clamp(0, table * ps - 1)
    slot = pages[b, position // ps] * ps + position % ps
    x = torch.cat([s["anchor"][:, None], s["x"]], 1)
    live_row = r < start[-1]
    keep = lambda new, old: torch.where(live_row, new.int(), old)  # noqa: E731
    return dict(L=L.int(), rows=rows.int(), pages=pages.int(), held=held.int(),
                free_pages=stack.int(), free_count=(top - grant.sum()).int(),
                row_start=start.int(), position=keep(position, s["position"]),
                slot=keep(slot, s["slot"]), token=keep(x[b, i], s["token"]))


def _plain_norm(s):
    case = s["case"]
    hq, hkv, D, rot, page = case["hq"], case["hkv"], case["D"], case["rot"], case["page"]
    cap = s["position"].numel()
    x = s["qkv"].float().reshape(cap, hq + 2 * hkv, D)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if s["q_weight"] is not None:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + s["eps"]) * s["q_weight"].float()
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + s["eps"]) * s["k_weight"].float()
    if rot:
        angle = s["position"].double()[:, None, None] * s["inv_freq"].double()
        cos, sin = (f(angle).mul(s["rope_scale"]).float() for f in (torch.cos, torch.sin))
        q, k = (_rotate(t, cos, sin, rot, s["interleaved"]) for t in (q, k))
    r = torch.arange(cap, device=x.device)
    live = r < s["n_rows"]
    # rows past the count repeat row 0, so that only the count's slots change
    at = torch.where(live, s["slot"], s["slot"][0]).long()
    first = live[:, None, None]
    s["k_cache"][at // page, :, at % page] = torch.where(first, k, k[:1]).to(torch.bfloat16)
    s["v_cache"][at // page, :, at % page] = torch.where(first, v, v[:1]).to(torch.bfloat16)
    s["q_out"].copy_(torch.where(first, q.to(torch.bfloat16), s["q_out"]))
    return {k: s[k] for k in ("q_out", "k_cache", "v_cache")}


def _rotate(t, cos, sin, rot, interleaved):
    turned, rest = t[..., :rot], t[..., rot:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        out = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = turned[..., :rot // 2], turned[..., rot // 2:]
        out = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([out, rest], -1)


def _plain_attention(s):
    case = s["case"]
    hq, hkv, D, most = case["hq"], case["hkv"], case["D"], case["gamma"] + 1
    ctx, start = s["context"].long(), s["row_start"].long()
    B = ctx.numel()
    cap = s["q"].shape[0]
    i = torch.arange(most, device=ctx.device)
    row = (start[:-1, None] + i).clamp(max=cap - 1)
    q = s["q"].float()[row].reshape(B, most, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4)
    count = (start[1:] - start[:-1])[:, None, None, None, None]

    def keys(cache):   # [B, hkv, 1, longest, D] in request order
        t = cache[s["pages"].clamp(min=0).long()].transpose(1, 2).reshape(B, hkv, 1, -1, D)
        return t[:, :, :, :s["longest"]].float()

    j = torch.arange(s["longest"], device=ctx.device)
    seen = j <= ctx[:, None, None, None, None] + i[:, None]
    known = j[:, None] < ctx[:, None, None, None, None] + count
    score = torch.matmul(q.flatten(2, 3)[:, :, None], keys(s["k_cache"]).transpose(-1, -2))
    score = score.reshape(B, hkv, hq // hkv, most, -1).mul_(s["scale"])
    score = score.masked_fill_(~(seen & known.transpose(-1, -2)), -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    value = keys(s["v_cache"]).masked_fill_(~known, 0.0)
    out = torch.matmul(p.flatten(2, 3)[:, :, None], value).reshape(B, hkv, hq // hkv, most, D)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, most, hq, D)
    r = torch.arange(cap, device=ctx.device)
    b = torch.searchsorted(start[1:].contiguous(), r, right=True).clamp(max=B - 1)
    got = out[b, (r - start[b]).clamp(max=most - 1)].to(torch.bfloat16)
    return torch.where((r < start[-1])[:, None, None], got, s["out"])


# -------------------------------------------------------------------------------- floors
def work(case):
    ctx, L = _lengths(case)
    rows = int((L + 1).sum())
    if case["op"] == "layout":
        # L, context, held in, held, rows, row_start out, drafts in, three words a row out
        return {"bytes": 4.0 * (7 * case["B"] + 4 * rows), "flops": 0.0}
    width = (case["hq"] + 2 * case["hkv"]) * case["D"]
    if case["op"] == "norm":
        return {"bytes": float(rows * (2 * width * 2 + 8)), "flops": 8.0 * rows * width}
    keys = int((ctx + L + 1).sum())
    seen = int(((L + 1) * ctx + (L + 1) * (L + 2) // 2).sum())
    return {"bytes": float(keys * case["hkv"] * case["D"] * 4 + 2 * rows * case["hq"] * case["D"] * 2),
            "flops": 4.0 * case["D"] * case["hq"] * seen}


# --------------------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    make = {"layout": _exact_layout, "norm": _exact_norm, "attention": _exact_attention}
    return make[case["op"]](s)


def _exact_layout(s):
    ps, gamma = s["page"], s["gamma"]
    L, ctx, held, anchor = (s[k].tolist() for k in ("L", "context", "held", "anchor"))
    pages, x = s["pages"].tolist(), s["x"].tolist()
    stack, top = s["free_pages"].tolist(), s["free_count"].item()
    rows, start, position, slot, token = [], [0], [], [], []
    want, need = [], []
    for b in range(len(L)):
        w = 0 if ctx[b] < 0 else min(L[b] + 1, len(pages[b]) * ps - ctx[b])
        want.append(w)
        need.append(0 if ctx[b] < 0 else math.ceil((ctx[b] + w) / ps))
        for at in range(need[b], held[b]):
            stack[top] = pages[b][at]
            top += 1
        held[b] = min(held[b], need[b])
    for b in range(len(L)):
        while held[b] < need[b] and top:
            top -= 1
            pages[b][held[b]] = stack[top]
            held[b] += 1
        n = max(0, min(want[b], held[b] * ps - ctx[b]))
        if n < want[b]:
            L[b] = max(n - 1, 0)
        rows.append(n)
        start.append(start[-1] + n)
        for i in range(n):
            at = ctx[b] + i
            position.append(at)
            slot.append(pages[b][at // ps] * ps + at % ps)
            token.append(x[b][i - 1] if i else anchor[b])
    fill = [-1] * (s["cap"] - len(position))
    i32 = lambda a: np.asarray(a, np.int32)  # noqa: E731
    return dict(L=i32(L), rows=i32(rows), pages=i32(pages), held=i32(held), free_pages=i32(stack),
                free_count=i32([top]), row_start=i32(start), position=i32(position + fill),
                slot=i32(slot + fill), token=i32(token + fill))


def _exact_norm(s):
    case = s["case"]
    hq, hkv, D, rot, page = case["hq"], case["hkv"], case["D"], case["rot"], case["page"]
    n = int(s["n_rows"].item())
    x = s["qkv"][:n].double().view(n, -1, D) if s["qkv"].is_contiguous() else \
        s["qkv"][:n].double().reshape(n, hq + 2 * hkv, D)
    turn = None
    if rot:   # as complex numbers: one factor for each pair
        angle = s["position"][:n].double()[:, None] * s["inv_freq"].double()[None]
        turn = torch.polar(torch.full_like(angle, s["rope_scale"]), angle)[:, None]

    def head(t, w):
        if w is not None:
            t = t / (t.pow(2).mean(-1, keepdim=True) + s["eps"]).sqrt() * w.double()
        if turn is not None:
            t = t.clone()
            pairs = t[..., :rot]
            pairs = pairs.reshape(n, -1, rot // 2, 2) if s["interleaved"] else \
                pairs.reshape(n, -1, 2, rot // 2).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            t[..., :rot] = (z if s["interleaved"] else z.transpose(-1, -2)).reshape(n, -1, rot)
        return t

    q_out, kc, vc = (s[k].double() for k in ("q_out", "k_cache", "v_cache"))
    q_out[:n] = head(x[:, :hq], s["q_weight"])
    page_of, off = s["slot"][:n].long() // page, s["slot"][:n].long() % page
    kc[page_of, :, off] = head(x[:, hq:hq + hkv], s["k_weight"])
    vc[page_of, :, off] = x[:, hq + hkv:]
    return dict(q_out=q_out, k_cache=kc, v_cache=vc)


def _exact_attention(s):
    case = s["case"]
    hq, hkv, D, page = case["hq"], case["hkv"], case["D"], case["page"]
    out = s["out"].double()
    start, ctx = s["row_start"].tolist(), s["context"].tolist()
    for b in range(len(ctx)):
        a, e = start[b], start[b + 1]
        n, rows = ctx[b] + e - a, e - a
        at = s["pages"][b, :_pages_of(n, page)].long()
        k, v = (c[at].transpose(0, 1).reshape(hkv, -1, D)[:, :n].double()
                for c in (s["k_cache"], s["v_cache"]))
        q = s["q"][a:e].double().reshape(rows, hkv, hq // hkv, D).permute(1, 2, 0, 3)
        score = torch.einsum("hgid,hjd->hgij", q, k) * s["scale"]
        hidden = torch.ones(rows, n, dtype=torch.bool, device=q.device).triu(ctx[b] + 1)
        p = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
        out[a:e] = torch.einsum("hgij,hjd->ihgd", p, v).reshape(rows, hq, D)
    return out
