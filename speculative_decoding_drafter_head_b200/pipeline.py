"""Asynchronous prefix scheduling from the scores of two steps earlier.

wispaper.ai, "DSpark: Overcoming the Efficiency Wall in LLM Speculative Decoding",
section "Critical Insights & Conclusion", key takeaway on asynchrony: so that scheduling
never stalls the GPU, the verify lengths of step t are decided from the confidence
predictions of step t - 2, which leaves a causal barrier between what is being drafted
and what decides how much of it is verified.
Verification stays a strict prefix match, so any lengths are lossless; the lag only
changes how many drafted tokens are sent to the target.

Here the scheduler kernel of step t reads the survival scores written by the
confidence kernel of step t - lag and runs on a side stream, so it no longer waits for
the confidence kernel of step t.  The draft kernel is a cooperative launch that holds
every SM, so nothing runs beside it; callers fork the side stream right after the draft
launch (``begin_step``), and the scheduler then overlaps the confidence kernel of the
same step.  Before `lag` steps exist, a step schedules on its own scores on the caller's
stream.

Buffers are rings of lag + 1 slots indexed by step: the confidence kernel of step t
writes ``scores(t)``, the scheduler of step t reads ``scores(t - lag)`` and writes the
lengths slot of step t, and verification of step t reads it.  Two events order the
streams, and each step uses them once:
  - fork: at ``begin_step(t)`` the side stream waits for everything already enqueued on
    the caller's stream (all of step t - 1, hence the scores of step t - lag);
  - join: the caller's stream waits for the scheduler of step t before verifying step t.
So scores slot (t - lag) mod (lag + 1), next written by the confidence kernel of step
t + 1, is no longer read by then, and every lengths slot is read by its own step's
verification before the next fork.  Both dependencies live inside one step, so a step
can be captured as one CUDA graph (one graph per ring phase) and replayed.

``VerifyPass`` keeps what the target's verification pass needs between the scheduler and the
verification: the paged cache of every layer, its block tables and free pages, and the
buffers of one step's ragged batch.  A step is

    L = sched.lengths(t)                              # or schedule_prefix's L_out
    vp.layout(L, anchor, x, accepted)                 # batch of this step, pages, slots
    for layer in range(layers):                       # the target's own products around it
        out = vp.attend(layer, qkv(layer), q_weight, k_weight)
    vp.verify(L, anchor, x, target, accepted, bonus)  # bonus: the next step's anchor

with every length on the device, so the whole step can be captured as one CUDA graph.

This module only orders launches of the library's kernels; it computes nothing.
"""
from __future__ import annotations

from . import (qk_norm_rope_store, schedule_prefix, verify_attention,
               verify_attention_workspace_bytes, verify_layout, verify_prefix, workspace_bytes)


def scores_slot(t: int, lag: int) -> int:
    """Ring slot holding the survival scores of step t."""
    return t % (lag + 1)


def source_step(t: int, lag: int) -> int:
    """The step whose scores decide the verify lengths of step t."""
    return t - lag if lag >= 1 and t >= lag else t


class LaggedScheduler:
    """Verify lengths for step t from the survival scores of step t - lag (default 2)."""

    def __init__(self, B: int, gamma: int, Tstep_us, lag: int = 2, device=None):
        import torch
        if lag < 0:
            raise ValueError("lag must be >= 0")
        device = device or Tstep_us.device
        self.B, self.gamma, self.lag = B, gamma, lag
        n = lag + 1
        self.Tstep = Tstep_us
        self.P = torch.empty(n, B, gamma, dtype=torch.float32, device=device)
        self.L = torch.empty(n, B, dtype=torch.int32, device=device)
        self.N = torch.empty(n, 1, dtype=torch.int32, device=device)
        self.obj = torch.empty(n, 1, dtype=torch.float64, device=device)
        # the side stream's own scheduler workspace: it runs concurrently with the draft
        # kernel, which uses the caller's workspace
        self.ws = torch.empty(workspace_bytes(B, gamma, 8), dtype=torch.uint8, device=device)
        self.side = torch.cuda.Stream(device=device)
        self.ev_fork = torch.cuda.Event()
        self.ev_join = torch.cuda.Event()

    def scores(self, t: int):
        """The [B, gamma] fp32 buffer that the confidence kernel of step t writes."""
        return self.P[scores_slot(t, self.lag)]

    def asynchronous(self, t: int) -> bool:
        """Whether step t is scheduled on the side stream (lag >= 1 and t >= lag)."""
        return self.lag >= 1 and t >= self.lag

    def begin_step(self, t: int, stream=None):
        """Launch the scheduler of step t on the side stream (if asynchronous).

        Call it after the draft launch of step t and before ``lengths(t)``."""
        import torch
        if not self.asynchronous(t):
            return
        main = stream or torch.cuda.current_stream()
        s = scores_slot(t - self.lag, self.lag)
        o = scores_slot(t, self.lag)
        self.ev_fork.record(main)
        self.side.wait_event(self.ev_fork)
        schedule_prefix(self.P[s], self.Tstep, self.L[o], self.N[o], self.obj[o], self.ws,
                        stream=self.side)
        self.ev_join.record(self.side)

    def lengths(self, t: int, workspace=None, stream=None):
        """Verify lengths [B] of step t, ordered before what the caller's stream runs next.

        Before `lag` steps exist (and always when lag = 0) this schedules step t on its own
        scores, on the caller's stream, with `workspace` or else the side workspace, which
        is idle then.
        """
        import torch
        main = stream or torch.cuda.current_stream()
        o = scores_slot(t, self.lag)
        if not self.asynchronous(t):
            schedule_prefix(self.P[o], self.Tstep, self.L[o], self.N[o], self.obj[o],
                            self.ws if workspace is None else workspace, stream=main)
        else:
            main.wait_event(self.ev_join)
        return self.L[o]

    def chosen(self, t: int):
        """(N*, objective) tensors of the schedule used at step t."""
        o = scores_slot(t, self.lag)
        return self.N[o], self.obj[o]


class VerifyPass:
    """Paged cache, block tables and batch buffers of the target's verification pass.

    All slots start idle.  Between steps the caller starts a request by context[b] = 0 and
    accepted[b] = -1 (nothing of the slot's last request sticks), its first token as anchor[b],
    and ends one by context[b] = -1: the next layout takes its pages back.  A prompt goes in by
    pieces of up to gamma + 1 tokens, a step each: the piece's first token as anchor[b], the others
    in x[b], L[b] their number, and accepted[b] = L[b] for the layout after it; context[b] says how
    far it has come.  Where pages run out a request gets fewer rows, or none (rows[b] = 0), and
    has to be sent again: verify() sees to it in the steps that verify."""

    def __init__(self, B: int, gamma: int, layers: int, Hq: int, Hkv: int, D: int, page_size: int,
                 num_pages: int, max_pages: int, inv_freq=None, interleaved: bool = False,
                 rope_scale: float = 1.0, eps: float = 1e-6, scale=None, device="cuda"):
        import torch
        i32 = dict(dtype=torch.int32, device=device)
        bf16 = dict(dtype=torch.bfloat16, device=device)
        rows = B * (gamma + 1)
        self.gamma, self.page_size = gamma, page_size
        self.rope = dict(eps=eps, inv_freq=inv_freq, interleaved=interleaved, rope_scale=rope_scale)
        self.scale = scale
        # the cache's state: all request slots idle, all pages free
        self.context = torch.full((B,), -1, **i32)
        self.rows = torch.zeros(B, **i32)
        self.pages = torch.zeros(B, max_pages, **i32)
        self.held = torch.zeros(B, **i32)
        self.free_pages = torch.arange(num_pages, **i32)
        self.free_count = torch.full((1,), num_pages, **i32)
        cache = (layers, num_pages, Hkv, page_size, D)
        self.k_cache, self.v_cache = torch.zeros(cache, **bf16), torch.zeros(cache, **bf16)
        # one step's batch
        self.row_start = torch.zeros(B + 1, **i32)
        self.position, self.slot, self.token = (torch.zeros(rows, **i32) for _ in range(3))
        self.q, self.out = (torch.zeros(rows, Hq, D, **bf16) for _ in range(2))
        self.workspace = torch.empty(verify_attention_workspace_bytes(Hq, Hkv, D),
                                     dtype=torch.uint8, device=device)

    def layout(self, L, anchor, x, accepted=None, stream=None):
        """Lay out this step's batch (see dspark_verify_layout): L [B] (cut in place where pages
        run out), anchor [B], x [B, gamma], and, from the second step of a request on, the
        accepted counts of the last step.  Fills row_start, position, slot and token."""
        verify_layout(L, self.context, self.rows, self.pages, self.held, self.free_pages,
                      self.free_count, self.row_start, self.position, self.slot, self.page_size,
                      self.gamma, anchor=anchor, x=x, token=self.token, accepted=accepted,
                      stream=stream)

    def verify(self, L, anchor, x, target, accepted_out, bonus_out, stream=None):
        """Verification of the step that layout() laid out, by its rows: a request without rows
        accepts -1 drafts and keeps its anchor as bonus token (see dspark_verify_prefix_rows).
        target [B, gamma + 1]: row row_start[b] + i's token at [b, i]."""
        verify_prefix(x, L, target, accepted_out, bonus_out, stream=stream, rows=self.rows,
                      anchor=anchor)

    def attend(self, layer: int, qkv, q_weight=None, k_weight=None, stream=None):
        """One layer's attention of the batch: qkv [B (gamma + 1), (Hq + 2 Hkv) D] normalised,
        rotated and stored, then attended.  Returns the buffer [B (gamma + 1), Hq, D], which the
        next call writes again."""
        k, v = self.k_cache[layer], self.v_cache[layer]
        qk_norm_rope_store(qkv, self.position, self.slot, self.row_start[-1:], self.q, k, v,
                           q_weight=q_weight, k_weight=k_weight, stream=stream, **self.rope)
        verify_attention(self.q, k, v, self.pages, self.context, self.row_start, self.out,
                         self.workspace, scale=self.scale, stream=stream)
        return self.out
