"""Plain 64-bit implementations of the verification pass, from the definitions, on the CPU."""
from __future__ import annotations

import numpy as np


def layout(L, context, held, pages, free_pages, free_count, ps, anchor=None, x=None, accepted=None,
           rows=None):
    """The step's state and batch, request by request, page by page."""
    L, ctx, held, pages, stack = (np.array(a, np.int64) for a in (L, context, held, pages,
                                                                  free_pages))
    top, B, room = int(np.ravel(free_count)[0]), len(L), pages.shape[1] * ps
    if accepted is not None:
        for b in range(B):
            if ctx[b] >= 0:
                ctx[b] += min(int(accepted[b]) + 1, int(rows[b]))
    need = np.zeros(B, np.int64)
    for b in range(B):
        if ctx[b] >= 0:
            need[b] = -(-(ctx[b] + min(L[b] + 1, room - ctx[b])) // ps)
        for at in range(need[b], held[b]):
            stack[top] = pages[b, at]
            top += 1
        held[b] = min(held[b], need[b])
    start, n, position, slot, token, cut = [0], [], [], [], [], False
    for b in range(B):
        while held[b] < need[b] and top > 0:
            top -= 1
            pages[b, held[b]] = stack[top]
            held[b] += 1
        want = L[b] + 1 if ctx[b] >= 0 else 0
        k = int(min(want, max(0, held[b] * ps - ctx[b])))
        if k < want:
            L[b] = max(k - 1, 0)
            cut = True
        n.append(k)
        start.append(start[-1] + k)
        for i in range(k):
            at = ctx[b] + i
            position.append(at)
            slot.append(pages[b, at // ps] * ps + at % ps)
            if anchor is not None:
                token.append(x[b][i - 1] if i else anchor[b])
    return dict(L=L, context=ctx, rows=n, pages=pages, held=held, free_pages=stack,
                free_count=[top], row_start=start, position=position, slot=slot, token=token,
                cut=cut)


def head(x, weight, eps, position, inv_freq, interleaved, rope_scale):
    """One query or key tensor [rows, heads, D] in fp64 -> normalised and rotated."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    if inv_freq is not None:
        n = len(inv_freq)
        angle = position[:, None].astype(np.float64) * inv_freq.astype(np.float64)[None]
        c, s = rope_scale * np.cos(angle)[:, None], rope_scale * np.sin(angle)[:, None]
        ia = 2 * np.arange(n) if interleaved else np.arange(n)
        ib = ia + 1 if interleaved else ia + n
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia] = a * c - b * s
        y[..., ib] = a * s + b * c
    return y


def attention(q, k_cache, v_cache, pages, context, row_start, scale):
    """(out, sum_j p_j |v_j|) of the rows [row_start[0], row_start[B]), fp64."""
    q = q.astype(np.float64)
    total, Hq, D = q.shape
    Hkv, ps = k_cache.shape[1], k_cache.shape[2]
    out, mag = np.zeros_like(q), np.zeros_like(q)
    for b in range(len(context)):
        for r in range(row_start[b], row_start[b + 1]):
            n = int(context[b]) + r - row_start[b] + 1
            at = pages[b, np.arange(n) // ps]
            off = np.arange(n) % ps
            k = k_cache[at, :, off].astype(np.float64)      # [n, Hkv, D]
            v = v_cache[at, :, off].astype(np.float64)
            for h in range(Hq):
                kh = h // (Hq // Hkv)
                s = k[:, kh] @ q[r, h] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[r, h] = p @ v[:, kh]
                mag[r, h] = p @ np.abs(v[:, kh])
    return out, mag
