"""Requests that get no rows in a step, from layout to verification: nothing that no row of the
step computed may come out, and nothing may be lost."""
import numpy as np
import pytest

from test_gpu_verify_pass import ds, host, i32  # noqa: F401

pytestmark = pytest.mark.gpu

STALE = 999                       # a target token that no row of the step computed


def after(token, position):
    """A target model: the token that follows `token` at `position`."""
    return (7 * token + 3 * position + 1) % 50


def chain(token, position, count):
    """`count` tokens that follow `token` at `position`."""
    out = []
    for p in range(position, position + count):
        token = after(token, p)
        out.append(token)
    return out


@pytest.mark.parametrize("captured", [False, True])
def test_starved_requests_stay_lossless(ds, captured):  # noqa: F811
    """More requests than the pages hold: whatever the drafts and however often a request gets no
    row, what is emitted is the target's own sequence."""
    import torch
    from speculative_decoding_drafter_head_b200.pipeline import VerifyPass
    rng = np.random.default_rng(6)
    B, gamma, ps = 4, 4, 4
    vp = VerifyPass(B, gamma, 1, 2, 1, 64, ps, num_pages=5, max_pages=6)
    vp.context.copy_(i32([0, 0, 0, -1]))                       # slot 3 idle
    first = rng.integers(0, 50, B)
    emitted = [[int(t)] for t in first]
    anchor, accepted = i32(first), i32(np.full(B, -1))
    L, x, target = i32(np.zeros(B)), i32(np.zeros((B, gamma))), i32(np.zeros((B, gamma + 1)))

    def layout():
        vp.layout(L, anchor, x, accepted)

    def verify():
        # in place: a request's bonus token is the next step's anchor
        vp.verify(L, anchor, x, target, accepted, anchor)

    calls = [layout, verify]
    if captured:
        state = [t.clone() for t in (vp.context, anchor, accepted)]
        layout(), verify()                                     # loads the kernels
        ds.get_error()
        for t, s in zip((vp.context, anchor, accepted), state):
            t.copy_(s)
        for t, s in ((vp.rows, 0), (vp.held, 0), (vp.free_count, 5)):
            t.fill_(s)
        vp.free_pages.copy_(torch.arange(5))
        torch.cuda.synchronize()
        graphs = []
        for call in calls:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call()
            graphs.append(g)
        calls = [g.replay for g in graphs]
    ctx = np.array([0, 0, 0, -1])
    starved, after_starved = 0, 0
    was = np.zeros(B, bool)
    for step in range(16):
        if step == 7:                                          # request 0 ends: its pages go round
            vp.context[0] = -1
            ctx[0] = -1
        an = host(anchor)
        xs = rng.integers(0, 50, (B, gamma))
        for b in range(B):
            right = int(rng.integers(0, gamma + 1))
            xs[b, :right] = chain(int(an[b]), max(ctx[b], 0), right)
        L.copy_(i32(rng.integers(0, gamma + 1, B)))
        x.copy_(i32(xs))
        calls[0]()
        assert ds.get_error() in (0, 9)
        rows, start = host(vp.rows), host(vp.row_start)
        token, position = host(vp.token), host(vp.position)
        tg = np.full((B, gamma + 1), STALE)
        for b in range(B):
            for i in range(rows[b]):
                tg[b, i] = after(int(token[start[b] + i]), int(position[start[b] + i]))
        target.copy_(i32(tg))
        calls[1]()
        assert ds.get_error() == 0
        acc, bonus = host(accepted), host(anchor)
        for b in range(B):
            if rows[b] == 0:
                assert acc[b] == -1 and bonus[b] == an[b]
                starved += ctx[b] >= 0
                was[b] = ctx[b] >= 0
                continue
            assert 0 <= acc[b] < rows[b]
            emitted[b] += [int(t) for t in xs[b, :acc[b]]] + [int(bonus[b])]
            ctx[b] += acc[b] + 1
            after_starved += was[b]
            was[b] = False
    assert starved and after_starved
    for b in range(3):
        assert emitted[b] == emitted[b][:1] + chain(emitted[b][0], 0, len(emitted[b]) - 1)
        assert len(emitted[b]) > 4
    assert len(emitted[3]) == 1


@pytest.mark.parametrize("B, gamma", [(1, 20), (130, 20), (5, 0)])
def test_verify_by_rows(ds, B, gamma):  # noqa: F811
    """Against the definition: lengths are cut to the rows, and no row means no token."""
    rng = np.random.default_rng(B)
    x = rng.integers(0, 9, (B, gamma))
    target = np.concatenate([x, rng.integers(0, 9, (B, 1))], 1)
    target[rng.random((B, gamma + 1)) < 0.1] = 10
    L, rows = rng.integers(0, gamma + 1, B), rng.integers(0, gamma + 3, B)
    rows[0] = 0
    anchor = rng.integers(100, 200, B)
    acc, bonus = i32(np.full(B, -9)), i32(np.full(B, -9))
    ds.verify_prefix(i32(x), i32(L), i32(target), acc, bonus, rows=i32(rows), anchor=i32(anchor))
    assert ds.get_error() == 0
    for b in range(B):
        n = min(L[b], rows[b] - 1)
        a = next((i for i in range(n) if x[b, i] != target[b, i]), n)
        want = (-1, anchor[b]) if rows[b] == 0 else (a, target[b, a])
        assert (int(acc[b]), int(bonus[b])) == want
    if gamma == 0:
        return
    # without rows: the lengths alone, as ever
    ds.verify_prefix(i32(x), i32(L), i32(target), acc, bonus)
    assert ds.get_error() == 0
    a = [next((i for i in range(L[b]) if x[b, i] != target[b, i]), L[b]) for b in range(B)]
    np.testing.assert_array_equal(host(acc), a)
    np.testing.assert_array_equal(host(bonus), target[np.arange(B), a])


def test_prompt_by_pieces(ds):  # noqa: F811
    """A prompt through VerifyPass, gamma + 1 tokens a step, beside a request that decodes: every
    token at its position, in a slot of its own."""
    import torch
    from speculative_decoding_drafter_head_b200.pipeline import VerifyPass
    rng = np.random.default_rng(1)
    B, gamma, ps = 2, 6, 16
    vp = VerifyPass(B, gamma, 1, 2, 1, 64, ps, num_pages=20, max_pages=10)
    prompt = rng.integers(0, 99, 40)
    vp.context.copy_(i32([0, 0]))
    accepted = i32([-1, -1])
    done, seen, slots = 0, [], set()
    while done < len(prompt):
        piece = prompt[done:done + gamma + 1]
        anchor, x, L = [piece[0], 5], np.zeros((B, gamma)), [len(piece) - 1, 2]
        x[0, :len(piece) - 1] = piece[1:]
        vp.layout(i32(L), i32(anchor), i32(x), accepted)
        assert ds.get_error() == 0
        n = len(piece)
        assert host(vp.context)[0] == done and host(vp.rows)[0] == n
        np.testing.assert_array_equal(host(vp.position)[:n], done + np.arange(n))
        seen += host(vp.token)[:n].tolist()
        slots |= set(host(vp.slot)[:n].tolist())
        accepted = i32([len(piece) - 1, 0])                    # all of the piece sticks
        done += n
    assert seen == prompt.tolist() and len(slots) == len(prompt)
    torch.cuda.synchronize()
