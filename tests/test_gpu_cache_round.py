"""The target pass's calls in a row, as a round uses them: plan, per layer
write and attend, commit; eager, on another stream, captured, and inside
DeviceRound."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from speculative_decoding_draft_rank_b200 import _lib, synth
from speculative_decoding_draft_rank_b200.kv_cache import PagedCache, Rows
from speculative_decoding_draft_rank_b200.round import DeviceRound

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _np(t):
    return t.detach().float().cpu().double().numpy()


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


class Model:
    """Random projections for the rows of a pass, a layer at a time."""

    def __init__(self, cache, T, seed):
        g = torch.Generator().manual_seed(seed)
        c = cache
        self.qkv = [(torch.randn(T, c.Hq + 2 * c.Hkv, c.D, generator=g) * 2).bfloat16().cuda() for _ in c.layers]
        self.out = [torch.full((T, c.Hq, c.D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in c.layers]
        self.q = [torch.full((T, c.Hq, c.D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in c.layers]
        self.w = [(1 + 0.2 * torch.randn(c.D, generator=g)).bfloat16().cuda() for _ in range(2)]

    def run(self, cache, rows=None, stream=None):
        for i, x in enumerate(self.qkv):
            q, k, v = x.split([cache.Hq, cache.Hkv, cache.Hkv], 1)
            cache.write(i, q, k, v, self.q[i], self.w[0], self.w[1], rows=rows, stream=stream)
            cache.attend(i, self.q[i], self.out[i], rows=rows, stream=stream)

    def check(self, cache, rows, table):
        """Against the oracle on the cache's own bytes (the write is checked against k and v)."""
        start, kv = rows.q_start.tolist(), rows.kv_len.tolist()
        m = start[-1]
        slot = rows.slot[:m].cpu().numpy()
        freq = cache.inv_freq.cpu().double().numpy()
        for i, x in enumerate(self.qkv):
            q, k, v = (_np(t) for t in x.split([cache.Hq, cache.Hkv, cache.Hkv], 1))
            bytes_ = cache.layers[i].cpu().numpy()
            gk, gv = oc.read(bytes_, slot, cache.page, cache.D)
            assert np.array_equal(gv, oc.dequantise(*oc.quantise(v[:m])))
            y = oc.norm_rope(k[:m], _np(self.w[1]), EPS, rows.pos[:m].cpu().numpy(), freq, False)
            near = oc.dequantise(*oc.quantise(y))
            # the nearest codes but where fp32 noise crosses a border: one step there
            assert (gk != near).mean() < 1e-3 and np.abs(gk - near).max() <= np.abs(y).max() / 2
            yq = oc.norm_rope(q[:m], _np(self.w[0]), EPS, rows.pos[:m].cpu().numpy(), freq, False)
            got_q = _np(self.q[i])
            assert (np.abs(got_q[:m] - yq) <= np.abs(yq) * 2.0 ** -8 + np.abs(yq).max() * 2.0 ** -17).all()
            ref, lim = oc.attention(got_q, bytes_, table, start, kv, cache.page, cache.scale, cache.window)
            out = _np(self.out[i])
            assert (np.abs(out[:m] - ref) <= lim * (1 + 2.0 ** -7) + np.abs(ref) * 2.0 ** -8).all()
            assert (out[m:] == 7.0).all()


def _freq(D):
    return 10000.0 ** (-np.arange(D // 2) / (D // 2))


@pytest.mark.parametrize("D,P,Hq,Hkv,window", [(64, 16, 6, 2, 0), (128, 32, 8, 1, 40)])
@pytest.mark.parametrize("side", [False, True])
def test_rounds_against_the_oracle(D, P, Hq, Hkv, window, side):
    B, G = 5, 4
    rng = np.random.default_rng(D)
    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        c = PagedCache(B, G, 2, Hq, Hkv, D, n_pages=60, max_pages=12, page=P, window=window, inv_freq=_freq(D))
        t = oc.Tables(B, 12, list(range(59, -1, -1)))
        prompt = np.array([37, 0, 3, 70, 1])
        rows = c.admit(prompt)
        start, kv, slot, pos, _ = t.plan(np.where(prompt > 0, 0, -1).tolist(), (prompt - 1).clip(0).tolist(), rows.G, P)
        assert rows.slot.tolist() == slot and rows.q_start.tolist() == start
        m = Model(c, rows.T, 1)
        m.run(c, rows)
        m.check(c, rows, t.table())
        ctx = np.where(prompt > 0, prompt, -1)
        assert c.ctx.tolist() == ctx.tolist()
        for rnd in range(4):
            ell = rng.integers(0, G + 1, B)
            rows = c.plan(_i32(ell))
            start, kv, slot, pos, full = t.plan(ctx.tolist(), ell.tolist(), G, P)
            assert rows.slot.tolist() == slot and rows.kv_len.tolist() == kv and not full
            m = Model(c, rows.T, 10 + rnd)
            m.run(c)
            m.check(c, rows, t.table())
            nout = np.minimum(rng.integers(1, G + 2, B), np.diff(start))
            done = (np.arange(B) == rnd).astype(np.int32)
            c.commit(_i32(nout), _i32(done))
            ctx = np.array(t.commit(ctx.tolist(), start, nout.tolist(), done.tolist(), P))
            assert c.ctx.tolist() == ctx.tolist() and c.free_list[: int(c.free_count)].tolist() == t.free
        assert c.device_status() == 0


def test_a_captured_round_replays():
    """plan, two layers and commit in one graph; a second graph shares the workspace; replays follow the tables."""
    B, G, D, P = 3, 3, 64, 16
    c = PagedCache(B, G, 2, 4, 2, D, n_pages=40, max_pages=10, page=P, inv_freq=_freq(D))
    t = oc.Tables(B, 10, list(range(39, -1, -1)))
    lengths = [20, 31, 5]
    rows = c.admit(lengths)
    t.plan([0] * 3, [x - 1 for x in lengths], rows.G, P)
    Model(c, rows.T, 0).run(c, rows)
    ell, nout = _i32([0] * B), _i32([0] * B)
    m = Model(c, B * (G + 1), 5)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        c.plan(ell)
        m.run(c)
    with torch.cuda.graph(g2):
        c.commit(nout)
    ctx = list(lengths)
    rng = np.random.default_rng(2)
    for _ in range(5):
        e = rng.integers(0, G + 1, B)
        n = np.minimum(rng.integers(1, G + 2, B), e + 1)
        ell.copy_(_i32(e))
        nout.copy_(_i32(n))
        for x in m.out:
            x.fill_(7.0)
        g1.replay()
        start, *_ = t.plan(ctx, e.tolist(), G, P)
        m.check(c, c.rows, t.table())
        g2.replay()
        ctx = t.commit(ctx, start, n.tolist(), None, P)
        assert c.ctx.tolist() == ctx
    assert c.device_status() == 0


def test_admit_refuses_and_leaves_the_cache_alone():
    c = PagedCache(3, 2, 1, 2, 2, 64, n_pages=6, max_pages=4, page=16)
    c.admit([20, 0, 0])
    before = [x.clone() for x in (c.ctx, c.table, c.held, c.free_count)]
    with pytest.raises(ValueError):
        c.admit([1, 0, 0])
    with pytest.raises(ValueError):
        c.admit([0, 0, 0])
    with pytest.raises(RuntimeError):
        c.admit([0, 64, 16])
    with pytest.raises(RuntimeError):
        c.admit([0, 65, 0])
    for x, y in zip(before, (c.ctx, c.table, c.held, c.free_count)):
        assert torch.equal(x, y)
    c.admit([0, 64, 0])
    assert c.ctx.tolist() == [20, 64, -1] and int(c.free_count) == 0
    c.commit(_i32([0, 0, 0]), _i32([1, 0, 0]))
    assert c.ctx.tolist()[0] == -1 and int(c.free_count) == 2
    with pytest.raises(ValueError):
        PagedCache(3, 2, 1, 3, 2, 64, n_pages=6, max_pages=4)


def test_offsets_past_32_bits():
    """A layer of 3 GB whose used pages lie at its ends."""
    Hq = Hkv = 8
    D, P, n_pages = 128, 64, 42000
    cache = torch.empty((n_pages, Hkv, _lib.dspark_cache_record_bytes(P, D)), dtype=torch.uint8, device="cuda")
    pages = np.array([n_pages - 1, 3, n_pages - 2])
    L = 150
    t = np.arange(L)
    g = torch.Generator().manual_seed(0)
    qkv = torch.randn(L, 3 * Hq, D, generator=g).bfloat16().cuda()
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    slot = _i32(pages[t // P] * P + t % P)
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda")
    qo = torch.empty(L, Hq, D, dtype=torch.bfloat16, device="cuda")
    _lib.dspark_qk_norm_rope(q, k, None, None, EPS, None, None, False, None, qo, None, ws, v=v, cache=cache, slot=slot,
                             page=P)
    ko, vo = torch.empty_like(qo), torch.empty_like(qo)
    _lib.dspark_cache_read(cache, slot, P, ko, vo, ws)
    assert np.array_equal(_np(ko), oc.dequantise(*oc.quantise(_np(k))))
    assert np.array_equal(_np(vo), oc.dequantise(*oc.quantise(_np(v))))
    out = torch.zeros(2, Hq, D, dtype=torch.bfloat16, device="cuda")
    _lib.dspark_cache_attention(q[:2], cache, _i32([pages]), _i32([0, 2]), _i32([L]), P, 0.1, 0, ws, out)
    small = cache[torch.from_numpy(pages).cuda()].cpu().numpy()
    ref, lim = oc.attention(_np(q[:2]), small, np.array([[0, 1, 2]]), [0, 2], [L], P, 0.1)
    assert (np.abs(_np(out) - ref) <= lim * (1 + 2.0 ** -7) + np.abs(ref) * 2.0 ** -8).all()
    assert _lib.dspark_get_device_status(ws) == 0


@pytest.mark.parametrize("production", [False, True])
def test_device_round_plans_and_commits(production):
    """A round with a cache and a target pass emits what it emits without, and the cache follows nout."""
    B, G, V, r, d = 6, 4, 4096, 32, 64
    kn, kt = np.array([0, 16], np.int32), np.array([8.0, 9.0])
    inp = synth.generate(B, G, V, r, d, "bf16", seed=5, hot=8)
    plain = DeviceRound(inp, kn, kt, -1, 1)
    c = PagedCache(B, G, 1, 4, 2, 64, n_pages=80, max_pages=12, page=16, inv_freq=_freq(64))
    rows = c.admit([30, 1, 17, 16, 5, 64])
    Model(c, rows.T, 3).run(c, rows)
    m = Model(c, B * (G + 1), 4)
    ran = []

    def target(dr, stream):
        ran.append(stream)
        m.run(c, stream=stream)

    dr = DeviceRound(inp, kn, kt, -1, 1, cache=c, target=target)
    if production:
        from speculative_decoding_draft_rank_b200.production import ProductionRound, ProductionScheduler
        run = ProductionRound(dr, ProductionScheduler(B, G, kn, kt)).run
        ref = ProductionRound(plain, ProductionScheduler(B, G, kn, kt)).run
    else:
        run, ref = dr.run, plain.run
    ctx = np.array([30, 1, 17, 16, 5, 64])
    for _ in range(3):
        run()
        ref()
        torch.cuda.synchronize()
        a, b = dr.outputs(), plain.outputs()
        for k in ("x", "ell", "tokens", "nout"):
            assert np.array_equal(a[k], b[k]), k
        assert c.rows.kv_len.tolist() == (ctx + a["ell"] + 1).tolist()
        m.check(c, c.rows, _planned_table(c, ctx, a["ell"]))
        for x in m.out:
            x.fill_(7.0)
        ctx = ctx + a["nout"]
        assert c.ctx.tolist() == ctx.tolist()
    assert len(ran) == 3 and c.device_status() == 0 and dr.device_status() == 0


def _planned_table(c, ctx, ell):
    """The table as it was before commit, from the slots (commit clears what it frees)."""
    table = c.table.cpu().numpy().copy()
    start, slot, pos = c.rows.q_start.tolist(), c.rows.slot.tolist(), c.rows.pos.tolist()
    for b in range(len(ctx)):
        for t in range(start[b], start[b + 1]):
            table[b, pos[t] // c.page] = slot[t] // c.page
    return table


def test_round_refuses_a_cache_of_another_batch():
    inp = synth.generate(4, 2, 4096, 32, 64, "bf16", seed=5, hot=8)
    kn, kt = np.array([0, 16], np.int32), np.array([8.0, 9.0])
    with pytest.raises(ValueError):
        DeviceRound(inp, kn, kt, -1, 1, cache=PagedCache(3, 2, 1, 2, 2, 64, n_pages=6, max_pages=4, page=16))
    with pytest.raises(ValueError):
        DeviceRound(inp, kn, kt, -1, 1, cache=PagedCache(4, 1, 1, 2, 2, 64, n_pages=6, max_pages=4, page=16))


@pytest.mark.parametrize("how", ["run", "host", "production", "graph"])
def test_a_round_whose_pages_run_out(how):
    """One free page and a seat at max_pages: requests are verified on the rows they got, a seat without rows emits
    nothing, and tokens and cache stay together.  The target fills the planned rows only; the others hold other logits."""
    from speculative_decoding_draft_rank_b200.production import ProductionRound, ProductionScheduler
    B, G, V, r, d, P = 8, 4, 4096, 32, 64, 16
    kn, kt = np.array([0, 64], np.int32), np.array([8.0, 8.1])
    inp = synth.generate(B, G, V, r, d, "bf16", seed=6, hot=8)
    lengths = [30, 1, 17, 16, 5, 64, 0, 47]
    c = PagedCache(B, G, 1, 4, 2, 64, n_pages=15, max_pages=4, page=P, inv_freq=_freq(64))
    t = oc.Tables(B, 4, list(range(14, -1, -1)))
    c.admit(lengths)
    ctx = [x if x else -1 for x in lengths]
    t.plan([0 if x else -1 for x in lengths], [max(x - 1, 0) for x in lengths], 63, P)
    plain = DeviceRound(inp, kn, kt, -1, 1)
    true = plain.t["Tlog"].clone()
    stale = true.roll(1, -1)

    def target(dr, stream):
        n = (c.rows.q_start[1:] - c.rows.q_start[:-1])[:, None]
        fresh = torch.arange(G + 1, device="cuda") < n
        dr.t["Tlog"].copy_(torch.where(fresh[..., None], true, dr.t["Tlog"]))

    dr = DeviceRound(inp, kn, kt, -1, 1, pinned_host=how == "host", cache=c, target=None if how == "host" else target)
    if how == "production":
        run = ProductionRound(dr, ProductionScheduler(B, G, kn, kt)).run
        ref = ProductionRound(plain, ProductionScheduler(B, G, kn, kt)).run
    else:
        run, ref = dr.run_from_host if how == "host" else dr.run, plain.run
    if how == "graph":
        ref()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dr.run()
        run = graph.replay
    starved = short = 0
    for _ in range(3):
        dr.t["Tlog"].copy_(stale)
        run()
        ref()
        ell = plain.o["ell"].tolist()
        start, kv, slot, pos, full = t.plan(ctx, ell, G, P)
        n = np.diff(start)
        plain.o["ell"].copy_(_i32(np.maximum(n - 1, 0)))
        plain.verify()
        torch.cuda.synchronize()
        a, b = dr.outputs(), plain.outputs()
        assert full and c.rows.slot.tolist() == slot and c.rows.q_start.tolist() == start
        assert a["ell"].tolist() == np.maximum(n - 1, 0).tolist()
        for k in ("acc", "tokens", "nout"):
            assert np.array_equal(a[k][n > 0], b[k][n > 0]), k
        assert (a["nout"][n == 0] == 0).all() and (a["acc"][n == 0] == 0).all() and (a["tokens"][n == 0] == -1).all()
        if how == "host":
            for k in ("ell", "tokens", "nout"):
                assert np.array_equal(dr.host_out[k].numpy(), a[k])
        starved += sum(int(m == 0 and x >= 0) for m, x in zip(n, ctx))
        short += sum(int(0 < m < e + 1) for m, e in zip(n, ell))
        ctx = t.commit(ctx, start, a["nout"].tolist(), None, P)
        assert c.ctx.tolist() == ctx and c.free_list[: int(c.free_count)].tolist() == t.free
        assert dr.device_status() == _lib.DEV_CACHE_FULL
    assert starved > 0 and short > 0


def test_admit_between_rounds_on_another_stream():
    """Rounds on a side stream that lags behind the host, admission from the default stream: admit sees what the last
    commit left, and the next round sees what admit did."""
    B, G, P = 3, 2, 16
    c = PagedCache(B, G, 1, 2, 1, 64, n_pages=12, max_pages=4, page=P, inv_freq=_freq(64))
    t = oc.Tables(B, 4, list(range(11, -1, -1)))
    side = torch.cuda.Stream()

    def seat(lengths, ctx, **kw):
        rows = c.admit(lengths, **kw)
        t.plan([0 if x else -1 for x in lengths], [max(x - 1, 0) for x in lengths], max(lengths) - 1, P)
        m = Model(c, rows.T, 1)
        side.wait_stream(torch.cuda.current_stream())
        m.run(c, rows, stream=side)
        side.synchronize()
        m.check(c, rows, t.table())
        return [x or y for x, y in zip(lengths, ctx)]

    ctx = seat([30, 5, 0], [-1, -1, -1])
    for rnd in range(3):
        ell, nout = _i32([2, 1, 0]), _i32([2, 1, 1])
        done = _i32([b == rnd for b in range(B)])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
        c.plan(ell, stream=side)
        c.commit(nout, done, stream=side)
        start, *_ = t.plan(ctx, [2, 1, 0], G, P)
        ctx = t.commit(ctx, start, [2, 1, 1], [b == rnd for b in range(B)], P)
        # the seat that the commit under way empties
        ctx = seat([30 if b == rnd else 0 for b in range(B)], ctx, **({"stream": side} if rnd == 2 else {}))
        c.plan(_i32([0, 0, 0]), stream=side)
        side.synchronize()
        start, kv, slot, *_ = t.plan(ctx, [0, 0, 0], G, P)
        assert c.ctx.tolist() == ctx and c.rows.kv_len.tolist() == kv and c.rows.slot.tolist() == slot
        assert c.free_list[: int(c.free_count)].tolist() == t.free
    assert c.device_status() == 0


def test_a_long_prompt_in_a_cache_of_many_seats():
    """Rows are the prompts' tokens, not seats times the longest prompt."""
    B, P, D, Hq = 256, 128, 64, 2
    lengths = [0] * B
    lengths[9], lengths[200] = 37, 70000
    c = PagedCache(B, 4, 1, Hq, 1, D, n_pages=600, max_pages=560, page=P, inv_freq=_freq(D))
    rows = c.admit(lengths)
    assert rows.T == 70037 and rows.slot.numel() >= rows.T
    assert rows.q_start.tolist() == [0] * 10 + [37] * 191 + [70037] * 56
    m = Model(c, rows.T, 2)
    m.run(c, rows)
    slot = rows.slot[: rows.T].cpu().numpy()
    q, k, v = (_np(x) for x in m.qkv[0].split([Hq, 1, 1], 1))
    cache = c.layers[0].cpu().numpy()
    gk, gv = oc.read(cache, slot, P, D)
    assert np.array_equal(gv, oc.dequantise(*oc.quantise(v)))
    at = np.array([0, 36, 37, 38, 165, 40000, 70035, 70036])            # rows as requests of one token each
    seat = np.where(at < 37, 9, 200)
    pos = np.where(at < 37, at, at - 37)
    assert rows.pos[torch.from_numpy(at).cuda()].tolist() == pos.tolist()
    ref, lim = oc.attention(_np(m.q[0])[at], cache, c.table.cpu().numpy()[seat], np.arange(len(at) + 1), pos + 1, P, c.scale)
    out = _np(m.out[0])[at]
    assert (np.abs(out - ref) <= lim * (1 + 2.0 ** -7) + np.abs(ref) * 2.0 ** -8).all()
    assert c.ctx.tolist() == [x or -1 for x in lengths] and c.device_status() == 0
    c.commit(_i32([0] * B), _i32([1] * B))
    assert int(c.free_count) == 600
    for bad in ([1 << 21] + [0] * (B - 1), [1 << 20] * 17 + [0] * (B - 17)):
        with pytest.raises(ValueError):
            c.admit(bad)


def test_many_seats_filled_at_once():
    """4096 prompts of 5000 tokens would be 2^24 padded rows and more; half the seats take short ones."""
    B, P = 4096, 16
    lengths = np.zeros(B, int)
    lengths[::2] = 1 + np.arange(B // 2) % 40
    lengths[1] = 5000
    c = PagedCache(B, 4, 1, 2, 1, 64, n_pages=9000, max_pages=320, page=P)
    rows = c.admit(lengths)
    t = oc.Tables(B, 320, list(range(8999, -1, -1)))
    start, kv, slot, pos, full = t.plan(np.where(lengths > 0, 0, -1).tolist(), np.maximum(lengths - 1, 0).tolist(), 4999, P)
    assert not full and rows.T == lengths.sum() == start[-1]
    assert rows.slot[: rows.T].tolist() == slot[: rows.T] and rows.pos[: rows.T].tolist() == pos[: rows.T]
    assert (rows.slot[rows.T:] == -1).all() and rows.q_start.tolist() == start and rows.kv_len.tolist() == kv
    assert c.device_status() == 0
