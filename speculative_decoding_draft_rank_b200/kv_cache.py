"""The target pass's paged 4-bit key/value cache.

Between scheduling and verification a round runs the target model over the
admitted tokens (paperlayer.ai summary of DSpark, §2: one target pass checks
the drafted tokens; menfem.com KB, "Key Contributions": the scheduler prunes
tokens from verification).  ``PagedCache`` keeps that pass's state for a batch
of seats and orders the library's calls:

  * ``plan(ell)`` after scheduling: rows, positions, slots and pages of the
    round's tokens (the last committed token and ell draft tokens per seat);
  * per layer ``write`` (head norms, rotation, cache write) and ``attend``;
  * ``commit(nout)`` after verification (``commit_round`` on a round's own
    outputs): the accepted tokens stay, the pages behind them go back to the
    pool.

``DeviceRound(..., cache=...)`` and ``ProductionRound`` call plan and commit
in their places.  Everything runs in libdspark's kernels on the given stream
and may be captured in a CUDA graph, except ``admit``, which seats prompts.
"""
from __future__ import annotations

import torch

from . import _lib


class Rows:
    """The packed rows of one plan: request b has rows q_start[b] .. q_start[b + 1] of arrays with `T` rows
    (by default as many as any plan can give; slot and pos may be longer, -1 behind the last row)."""

    MOST = 1 << 24     # rows that a plan or a pass takes

    def __init__(self, B: int, G: int, device, T: int | None = None):
        i32 = dict(dtype=torch.int32, device=device)
        self.B, self.G, self.T = B, G, B * (G + 1) if T is None else T
        self.q_start = torch.zeros(B + 1, **i32)
        self.n_rows = self.q_start[B:]
        self.kv_len = torch.zeros(B, **i32)
        entries = self.T if T is None else max(T, min(B * (G + 1), self.MOST))
        self.slot = torch.full((entries,), -1, **i32)
        self.pos = torch.full((entries,), -1, **i32)

    def used_on(self, stream):
        """Keep the arrays' memory from reuse until `stream` has done what it was given so far."""
        for t in (self.q_start, self.kv_len, self.slot, self.pos):
            t.record_stream(stream)


class PagedCache:
    """B seats, `n_layers` layers of Hkv key heads read by Hq query heads of
    `D` dims, a pool of n_pages pages of `page` tokens, at most max_pages of
    them per seat; draft blocks of up to G tokens.  `window` > 0 limits
    attention to the last `window` keys; `scale` defaults to D ** -0.5;
    k_scale and v_scale as in dspark_cache_attention."""

    def __init__(self, B: int, G: int, n_layers: int, Hq: int, Hkv: int, D: int, n_pages: int, max_pages: int,
                 page: int = 64, window: int = 0, scale: float | None = None, k_scale: float = 1.0,
                 v_scale: float = 1.0, inv_freq=None, interleaved: bool = False, eps: float = 1e-6, device="cuda"):
        dev = torch.device(device)
        rec = _lib.dspark_cache_record_bytes(page, D)
        need = _lib.dspark_cache_attention_workspace_size(B, Hq, Hkv, D)
        if rec == 0 or need == 0 or n_pages < 1 or max_pages < 1 or G < 0 or n_layers < 1:
            raise ValueError("cache shape outside the library's limits")
        self.B, self.G, self.Hq, self.Hkv, self.D = B, G, Hq, Hkv, D
        self.page, self.window, self.device = page, window, dev
        self.scale = D ** -0.5 if scale is None else float(scale)
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.eps, self.interleaved = float(eps), bool(interleaved)
        self.inv_freq = None if inv_freq is None else torch.as_tensor(inv_freq, dtype=torch.float32).to(dev).contiguous()
        self.layers = [torch.empty((n_pages, Hkv, rec), dtype=torch.uint8, device=dev) for _ in range(n_layers)]
        i32 = dict(dtype=torch.int32, device=dev)
        self.ctx = torch.full((B,), -1, **i32)                 # cached tokens per seat, -1: empty
        self.table = torch.full((B, max_pages), -1, **i32)
        self.held = torch.zeros(B, **i32)
        self.free_list = torch.arange(n_pages - 1, -1, -1, **i32)
        self.free_count = torch.full((1,), n_pages, **i32)
        self.rows = Rows(B, G, dev)
        # The round's calls follow one another on a stream, so they share a workspace.
        self.ws = torch.zeros((need + 255) // 256 * 256, dtype=torch.uint8, device=dev)

    # --------------------------------------------------------------- rounds
    def plan(self, ell, stream=None, ell_out=None) -> Rows:
        """Rows, slots and pages for the round's 1 + ell[b] tokens per seat.
        Where pages run out (the pool, or a seat's max_pages) a seat gets fewer
        rows or none, and the status word says CACHE_FULL; ell_out [B] (may be
        ell) receives the lengths that the rows cover, for verification."""
        r = self.rows
        _lib.dspark_cache_plan_rows(self.ctx, ell, r.G, self.table, self.held, self.free_list, self.free_count,
                                    self.page, self.ws, r.q_start, r.kv_len, r.slot, r.pos, ell_out, stream)
        return r

    def commit(self, nout, done=None, stream=None):
        """Keep nout[b] of the planned tokens; seats with done[b] are emptied."""
        _lib.dspark_cache_commit(self.ctx, self.rows.q_start, nout, done, self.table, self.held, self.free_list,
                                 self.free_count, self.page, self.ws, self.ctx, stream)

    def commit_round(self, nout, acc=None, tokens=None, done=None, stream=None):
        """commit after verification on the planned lengths: seats without rows
        (empty, or no page for their next token) emit nothing -- their nout and
        acc become 0 and their tokens -1, in place."""
        _lib.dspark_cache_commit_round(self.ctx, self.rows.q_start, nout, acc, tokens, done, self.table, self.held,
                                       self.free_list, self.free_count, self.page, self.ws, self.ctx, stream)

    def _rows(self, rows, stream) -> Rows:
        if rows is None or rows is self.rows:
            return self.rows
        rows.used_on(torch.cuda.current_stream(self.device) if stream is None else stream)
        return rows

    def write(self, layer: int, q, k, v, q_out, wq=None, wk=None, rows: Rows | None = None, k_out=None, stream=None):
        """Norm and turn the projections q, k [T, heads, D] of the planned rows
        and put keys and values v into the layer's cache; queries come back in
        q_out (which may be q where that is contiguous), keys in k_out where it
        is given."""
        r = self._rows(rows, stream)
        _lib.dspark_qk_norm_rope(q, k, wq, wk, self.eps, r.pos, self.inv_freq, self.interleaved, r.n_rows, q_out,
                                 k_out, self.ws, v=v, cache=self.layers[layer], slot=r.slot, page=self.page,
                                 k_scale=self.k_scale, v_scale=self.v_scale, stream=stream)

    def attend(self, layer: int, q, out, rows: Rows | None = None, stream=None):
        """out [T, Hq, D] = attention of the rows q over the layer's cache."""
        r = self._rows(rows, stream)
        _lib.dspark_cache_attention(q, self.layers[layer], self.table, r.q_start, r.kv_len, self.page, self.scale,
                                    self.window, self.ws, out, k_scale=self.k_scale, v_scale=self.v_scale,
                                    stream=stream)

    def read(self, layer: int, slot, k_out, v_out, stream=None):
        """Cached keys and values of the tokens `slot`."""
        _lib.dspark_cache_read(self.layers[layer], slot, self.page, k_out, v_out, self.ws, k_scale=self.k_scale,
                               v_scale=self.v_scale, stream=stream)

    # -------------------------------------------------------------- prompts
    def admit(self, lengths, stream=None) -> Rows:
        """Seat prompts: lengths[b] > 0 tokens into empty seat b (0: no
        change).  Returns the rows to run the prompt pass on (write and attend
        with rows=..., on arrays of rows.T rows, the prompts' tokens); the
        tokens count as cached from here on.  At most 2^20 tokens a prompt and
        2^24 a call.  Raises if a seat is taken or the pool is too small,
        leaving the cache as it was.
        Waits for the device before (rounds and graph replays on any stream
        have then left the tables) and after (any stream may go on from here);
        runs on `stream`, by default the current one.  No call on this cache
        may be made from another thread meanwhile."""
        want = torch.as_tensor(lengths, dtype=torch.int32).cpu()
        if want.shape != (self.B,) or int(want.min()) < 0 or int(want.max()) == 0:
            raise ValueError(f"lengths: {self.B} prompt lengths, one of them positive")
        total = int(want.sum(dtype=torch.int64))
        if total > Rows.MOST or int(want.max()) > 1 << 20:
            raise ValueError(f"{total} prompt tokens, the longest {int(want.max())}: at most 2^24 a call, 2^20 a prompt")
        torch.cuda.synchronize(self.device)
        ctx = self.ctx.cpu()
        if bool(((want > 0) & (ctx >= 0)).any()):
            raise ValueError("a prompt for a seat that is taken")
        need = int(((want + self.page - 1) // self.page).sum())
        if need > int(self.free_count) or int(want.max()) > self.table.shape[1] * self.page:
            raise RuntimeError(f"the prompts need {need} pages, {int(self.free_count)} are free, "
                               f"{self.table.shape[1]} at most per seat")
        st = torch.cuda.current_stream(self.device) if stream is None else stream
        with torch.cuda.stream(st):
            r = Rows(self.B, int(want.max()) - 1, self.device, total)
            new = (want > 0).to(self.device)
            want = want.to(self.device)
            none = torch.full_like(want, -1)
            _lib.dspark_cache_plan_rows(torch.where(new, 0, none), (want - 1).clamp(min=0), r.G, self.table, self.held,
                                        self.free_list, self.free_count, self.page, self.ws, r.q_start, r.kv_len,
                                        r.slot, r.pos, stream=st)
            self.ctx.copy_(torch.where(new, want, self.ctx))
        torch.cuda.synchronize(self.device)
        return r

    def device_status(self) -> int:
        """Data errors of the calls so far (0: none; synchronises)."""
        return _lib.dspark_get_device_status(self.ws)
