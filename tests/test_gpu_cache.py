"""The target pass's cache and attention on the GPU against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from speculative_decoding_draft_rank_b200 import _lib

pytestmark = pytest.mark.gpu

EPS1 = 1e-6


def _ws(n=256):
    return torch.zeros((n + 255) // 256 * 256, dtype=torch.uint8, device="cuda")


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def _np(t):
    return t.detach().float().cpu().double().numpy()


# ------------------------------------------------------------------ tables
class DeviceTables:
    """The device copy of an oracle Tables."""

    def __init__(self, t, n_pages, B, G, P):
        self.P, self.G, self.B = P, G, B
        self.table = _i32(t.table())
        self.held = _i32([len(r) for r in t.rows])
        self.free = _i32(t.free + [-1] * (n_pages - len(t.free)))
        self.count = _i32([len(t.free)])
        self.q_start, self.kv = _i32([7] * (B + 1)), _i32([7] * B)
        self.slot, self.pos = _i32([7] * (B * (G + 1))), _i32([7] * (B * (G + 1)))
        self.ctx_out = _i32([7] * B)
        self.ws = _ws()

    def plan(self, ctx, ell):
        _lib.dspark_cache_plan(ctx, ell, self.G, self.table, self.held, self.free, self.count, self.P, self.ws,
                               self.q_start, self.kv, self.slot, self.pos)

    def commit(self, ctx, nout, done=None, out=None):
        _lib.dspark_cache_commit(ctx, self.q_start, nout, done, self.table, self.held, self.free, self.count, self.P,
                                 self.ws, self.ctx_out if out is None else out)

    def check(self, t):
        assert np.array_equal(self.table.cpu().numpy(), t.table())
        assert self.held.tolist() == [len(r) for r in t.rows]
        assert int(self.count) == len(t.free)
        assert self.free[: len(t.free)].tolist() == t.free


@pytest.mark.parametrize("B,G,P,max_pages,pool", [
    (1, 0, 16, 3, 3), (5, 5, 16, 9, 30), (256, 5, 64, 8, 1200), (700, 8, 16, 12, 5000), (1024, 16, 32, 6, 2900),
    (4096, 3, 128, 3, 9000), (33, 200, 16, 40, 900)])
def test_tables_over_rounds(B, G, P, max_pages, pool):
    rng = np.random.default_rng(B * 31 + G)
    t = oc.Tables(B, max_pages, rng.permutation(pool).tolist())
    d = DeviceTables(t, pool, B, G, P)
    ctx = np.where(rng.random(B) < 0.1, -1, 0)
    ctx_d = _i32(ctx)
    for rnd in range(6):
        ell = rng.integers(0, G + 1, B)
        d.plan(ctx_d, _i32(ell))
        start, kv, slot, pos, full = t.plan(ctx.tolist(), ell.tolist(), G, P)
        d.check(t)
        assert d.q_start.tolist() == start and d.kv.tolist() == kv
        assert d.slot.tolist() == slot and d.pos.tolist() == pos
        st = _lib.dspark_get_device_status(d.ws)
        assert st == (_lib.DEV_CACHE_FULL if full else 0)
        _lib.dspark_clear_device_status(d.ws)
        if rnd == 2:       # the same plan again: the same rows, no further pages
            d.plan(ctx_d, _i32(ell))
            d.check(t)
            assert d.slot.tolist() == slot
        n = np.diff(start)
        nout = np.minimum(rng.integers(0, G + 2, B), n)
        done = rng.random(B) < 0.15
        out = t.commit(ctx.tolist(), start, nout.tolist(), done.tolist(), P)
        if rnd % 2:
            d.commit(ctx_d, _i32(nout), _i32(done), out=ctx_d)      # in place
            assert ctx_d.tolist() == out
        else:
            d.commit(ctx_d, _i32(nout), _i32(done))
            assert d.ctx_out.tolist() == out
            ctx_d = d.ctx_out.clone()
        d.check(t)
        # seats that emptied are taken again
        ctx = np.array(out)
        fresh = (ctx < 0) & (rng.random(B) < 0.7)
        ctx = np.where(fresh, 0, ctx)
        ctx_d = _i32(ctx)
    st = _lib.dspark_get_device_status(d.ws)
    assert st & ~_lib.DEV_CACHE_FULL == 0


def test_tables_report_bad_lengths():
    t = oc.Tables(3, 4, list(range(12)))
    d = DeviceTables(t, 12, 3, 2, 16)
    d.plan(_i32([0, 5, 3]), _i32([9, -4, 1]))
    start, kv, slot, pos, _ = t.plan([0, 5, 3], [9, -4, 1], 2, 16)
    assert d.slot.tolist() == slot and d.q_start.tolist() == start
    assert _lib.dspark_get_device_status(d.ws) == _lib.DEV_ELL_RANGE
    _lib.dspark_clear_device_status(d.ws)
    d.commit(_i32([0, 5, 3]), _i32([9, -1, 2]))
    assert d.ctx_out.tolist() == t.commit([0, 5, 3], start, [9, -1, 2], None, 16)
    assert _lib.dspark_get_device_status(d.ws) == _lib.DEV_LENGTH_RANGE
    # a context longer than its table: no tokens, and it says so
    _lib.dspark_clear_device_status(d.ws)
    d.plan(_i32([1000, 0, 0]), _i32([0, 0, 0]))
    assert d.q_start.tolist()[:2] == [0, 0]
    assert _lib.dspark_get_device_status(d.ws) == _lib.DEV_LENGTH_RANGE | _lib.DEV_CACHE_FULL


# -------------------------------------------------------- norm and rotation
def _tol_norm(ref, D, dtype):
    """fp32 sum of D squares (half of it in the root), a few fp32 products, the reduced angle's rounding, on the
    pair's length, at most sqrt(2) of the row's largest; then half a step of the output."""
    top = np.abs(ref).max(-1, keepdims=True) * np.sqrt(2.0)
    return top * (D * 2.0 ** -25 + 2.0 ** -20) + np.abs(ref) * torch.finfo(dtype).eps / 2 + 1e-30


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter", [
    (1, 1, 1, 64, 64, False), (7, 8, 2, 128, 128, False), (33, 10, 5, 64, 32, True), (5, 3, 3, 128, 64, True),
    (4, 64, 8, 128, 96, False), (3, 40, 1, 128, 0, False), (129, 6, 2, 64, 64, True)])
def test_norm_and_rotation(dtype, T, Hq, Hkv, D, rot, inter):
    g = torch.Generator().manual_seed(T * 7 + D + rot)
    qkv = (torch.randn(T + 2, Hq + 2 * Hkv, D, generator=g) * 3).to(dtype).cuda()
    q, k, _ = qkv.split([Hq, Hkv, Hkv], 1)
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2))
    pos = torch.randint(0, 1 << 20, (T + 2,), generator=g, dtype=torch.int32)
    pos[0] = 0
    freq = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).float()
    qo = torch.full((T + 2, Hq, D), 9.0, dtype=dtype, device="cuda")
    ko = torch.full((T + 2, Hkv, D), 9.0, dtype=dtype, device="cuda")
    ws = _ws()
    for weights in (True, False):
        _lib.dspark_qk_norm_rope(q, k, wq if weights else None, wk if weights else None, EPS1, pos.cuda(),
                                 freq.cuda() if rot else None, inter, _i32([T]), qo, ko, ws)
        for x, w, o in ((q, wq, qo), (k, wk, ko)):
            ref = oc.norm_rope(_np(x[:T]), _np(w) if weights else None, EPS1, pos[:T].numpy(), freq.double().numpy(),
                               inter)
            assert (np.abs(_np(o[:T]) - ref) <= _tol_norm(ref, D, dtype)).all()
            assert (o[T:] == 9.0).all()
    assert _lib.dspark_get_device_status(ws) == 0
    # in place on dense rows
    qd, kd = q.contiguous(), k.contiguous()
    _lib.dspark_qk_norm_rope(qd, kd, None, None, EPS1, pos.cuda(), freq.cuda() if rot else None, inter, _i32([T]), qd,
                             kd, ws)
    assert torch.equal(qd[:T], qo[:T]) and torch.equal(kd[:T], ko[:T]) and torch.equal(qd[T:], q[T:])


def _cache(n_pages, Hkv, P, D, fill=255):
    return torch.full((n_pages, Hkv, _lib.dspark_cache_record_bytes(P, D)), fill, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,P,g", [(1, 4, 1, 64, 64, 16, 1.0), (37, 8, 8, 128, 128, 64, 1.0),
                                                (9, 12, 3, 128, 64, 32, 0.25), (70, 2, 2, 64, 0, 128, 4.0)])
def test_cache_write_bytes(dtype, T, Hq, Hkv, D, rot, P, g):
    gen = torch.Generator().manual_seed(T + D + P)
    n_pages = T // P + 3
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=gen)
    qkv[:, :, :16] *= 50.0                                   # groups of very different scales, a zero one too
    qkv[:, :, 32:48] *= 1e-4
    qkv[0, :, 48:] = 0.0
    qkv = qkv.to(dtype).cuda()
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    wk = (1 + 0.3 * torch.randn(D, generator=gen)).to(dtype).cuda()
    pos = torch.randint(0, 9000, (T,), generator=gen, dtype=torch.int32).cuda()
    slot = torch.randperm(n_pages * P, generator=gen)[:T].int()
    slot[T // 2] = -1 if T > 1 else slot[0]
    freq = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).float().cuda()
    cache, ws = _cache(n_pages, Hkv, P, D), _ws()
    qo, ko = torch.empty(T, Hq, D, dtype=dtype, device="cuda"), torch.empty(T, Hkv, D, dtype=dtype, device="cuda")
    _lib.dspark_qk_norm_rope(q, k, None, wk, EPS1, pos, freq if rot else None, False, None, qo, ko, ws, v=v,
                             cache=cache, slot=slot.cuda(), page=P, k_scale=g, v_scale=2 * g)
    assert _lib.dspark_get_device_status(ws) == 0
    sl = slot.numpy()
    ref = np.full(cache.shape, 255, np.uint8)
    oc.write(ref, sl, _np(ko), _np(v), P, g, 2 * g)
    got = cache.cpu().numpy()
    half = got.shape[2] // 2
    assert np.array_equal(got[:, :, half:], ref[:, :, half:])            # values: every byte, untouched ones too
    if dtype == torch.float32:                                           # keys: k_out is what was quantised
        assert np.array_equal(got[:, :, :half], ref[:, :, :half])
    live = sl >= 0
    kv = [torch.full((T, Hkv, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    _lib.dspark_cache_read(cache, slot.cuda(), P, kv[0], kv[1], ws, k_scale=g, v_scale=2 * g)
    rk, rv = oc.read(got, sl[live], P, D, g, 2 * g)
    assert np.array_equal(_np(kv[0])[live], rk) and np.array_equal(_np(kv[1])[live], rv)
    assert (_np(kv[0])[~live] == 9.0).all()
    y = oc.norm_rope(_np(k), _np(wk), EPS1, pos.cpu().numpy(), freq.cpu().double().numpy(), False)[live]
    big = np.abs(y.reshape(len(rk), Hkv, -1, 16)).max(-1, keepdims=True)
    # half the widest step (1 of 6), half a step of the scale (2^-4), the scale's smallest step, fp32 noise
    lim = big * (1 / 6 + 2.0 ** -4) * (1 + 2.0 ** -15) + 6 * g * 2.0 ** -9
    assert (np.abs((rk - y).reshape(len(rk), Hkv, -1, 16)) <= lim).all()


def test_cache_write_of_nan_and_infinity():
    T, Hkv, D, P = 4, 2, 64, 16
    k = torch.randn(T, Hkv, D, generator=torch.Generator().manual_seed(0)).cuda()
    v = k.clone()
    v[1, 0, 3], v[2, 1, 20], v[3, 1, 63] = float("nan"), float("inf"), float("-inf")
    cache, ws = _cache(1, Hkv, P, D), _ws()
    slot = _i32([0, 5, 9, 15])
    _lib.dspark_qk_norm_rope(k, k, None, None, EPS1, None, None, False, None, torch.empty_like(k), None, ws, v=v,
                             cache=cache, slot=slot, page=P)
    assert _lib.dspark_get_device_status(ws) == _lib.DEV_BAD_VALUE
    ref = np.full(cache.shape, 255, np.uint8)
    oc.write(ref, slot.tolist(), _np(k), np.nan_to_num(_np(v), nan=0.0, posinf=1e30, neginf=-1e30), P)
    assert np.array_equal(cache.cpu().numpy(), ref)
    # a slot outside the pool is skipped and reported
    _lib.dspark_clear_device_status(ws)
    _lib.dspark_qk_norm_rope(k, k, None, None, EPS1, None, None, False, None, torch.empty_like(k), None, ws, v=k,
                             cache=cache, slot=_i32([16, -1, 1 << 30, -1]), page=P)
    assert _lib.dspark_get_device_status(ws) == _lib.DEV_PAGE_RANGE
    assert np.array_equal(cache.cpu().numpy(), ref)


@pytest.mark.parametrize("e", [-64, 64])
def test_cache_write_at_the_ends_of_the_layer_scales(e):
    """Powers of two go through every step exactly, so x * g stored with scale g has the bytes of x."""
    T, Hkv, D, P, g = 16, 2, 64, 16, 2.0 ** e
    gen = torch.Generator().manual_seed(3)
    k, v = (torch.randn(T, Hkv, D, generator=gen).cuda() for _ in range(2))
    slot, ws, caches = _i32(range(T)), _ws(), []
    for s in (1.0, g):
        cache = _cache(1, Hkv, P, D)
        _lib.dspark_qk_norm_rope(k * s, k * s, None, None, EPS1, None, None, False, None, torch.empty_like(k), None, ws,
                                 v=v * s, cache=cache, slot=slot, page=P, k_scale=s, v_scale=s)
        out = torch.empty_like(k), torch.empty_like(v)
        _lib.dspark_cache_read(cache, slot, P, *out, ws, k_scale=s, v_scale=s)
        caches.append((cache, out[0] / s, out[1] / s))
    assert _lib.dspark_get_device_status(ws) == 0
    for a, b in zip(*caches):
        assert torch.equal(a, b)


def test_calls_without_tokens():
    q, k = torch.empty(0, 4, 64, device="cuda", dtype=torch.bfloat16), torch.empty(0, 2, 64, device="cuda",
                                                                                  dtype=torch.bfloat16)
    cache = _cache(2, 2, 16, 64)
    ws = _ws(_lib.dspark_cache_attention_workspace_size(1, 4, 2, 64))
    none = _i32([])
    _lib.dspark_qk_norm_rope(q, k, None, None, EPS1, none, torch.ones(16, device="cuda"), False, None, q, None, ws, v=k,
                             cache=cache, slot=none, page=16)
    _lib.dspark_cache_read(cache, none, 16, k, torch.empty_like(k), ws)
    _lib.dspark_cache_attention(q, cache, _i32([[0]]), _i32([0, 0]), _i32([5]), 16, 0.1, 0, ws, torch.empty_like(q))
    assert _lib.dspark_get_device_status(ws) == 0 and (cache == 255).all()


# --------------------------------------------------------------- attention
def _fill(rng, B, Hkv, D, P, kv_len, kg=1.0, vg=1.0):
    """A cache of garbage bytes with the tokens of every request written by the oracle."""
    mp = max(1, max(-(-int(L) // P) for L in kv_len) + 1)
    n_pages = B * mp + 3
    table = rng.permutation(n_pages)[: B * mp].reshape(B, mp).astype(np.int32)
    cache = rng.integers(0, 256, (n_pages, Hkv, P * D // 8 * 9)).astype(np.uint8)
    cache[:, :, ::5] = 255
    for b, L in enumerate(kv_len):
        t = np.arange(L)
        if L:
            oc.write(cache, table[b][t // P].astype(np.int64) * P + t % P, rng.standard_normal((L, Hkv, D)) * kg,
                     rng.standard_normal((L, Hkv, D)) * vg, P, kg, vg)
    return cache, table


def _check_attention(q, cache, table, n, kv_len, P, scale, window=0, kg=1.0, vg=1.0, extra=2, ws=None):
    start = np.concatenate(([0], np.cumsum(n))).astype(np.int32)
    T, Hq, D = q.shape
    qd = torch.from_numpy(q).to(torch.bfloat16).cuda()
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    if ws is None:
        ws = _ws(_lib.dspark_cache_attention_workspace_size(len(n), Hq, cache.shape[1], D))
    args = (qd, torch.from_numpy(cache).cuda(), _i32(table), _i32(start), _i32(kv_len), P, scale, window, ws)
    _lib.dspark_cache_attention(*args, out, k_scale=kg, v_scale=vg)
    assert _lib.dspark_get_device_status(ws) == 0
    ref, lim = oc.attention(_np(qd), cache, table, start, kv_len, P, scale, window, kg, vg)
    got = _np(out)
    m = start[-1]
    err = np.abs(got[:m] - ref)
    bad = err > lim * (1 + 2.0 ** -7) + np.abs(ref) * 2.0 ** -8
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {err.max()} at {np.argwhere(bad)[:4].tolist()}"
    assert (got[m:] == 7.0).all()
    again = torch.full_like(out, 7.0)
    _lib.dspark_cache_attention(*args, again, k_scale=kg, v_scale=vg)
    assert torch.equal(out, again)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P,Hq,Hkv,n,kv_len,window", [
    (16, 1, 1, [1], [1], 0),
    (16, 4, 2, [1, 1], [0, 5], 0),
    (64, 8, 1, [1, 2, 3], [64, 128, 129], 0),
    (32, 6, 2, [3, 0, 2, 5], [127, 40, 300, 5], 0),
    (128, 5, 5, [4, 1], [257, 1000], 0),
    (16, 16, 2, [6, 1, 3], [33, 700, 250], 128),
    (32, 12, 4, [17, 9], [400, 131], 1),
    (64, 3, 1, [2, 4, 4], [3, 2, 640], 37),
    (16, 16, 1, [17, 3], [90, 500], 0),
    (64, 40, 1, [5], [333], 200),
    (32, 2, 1, [150, 70], [150, 400], 0),
    (16, 2, 2, [0, 0, 1], [9, 9, 9], 0)])
def test_attention(D, P, Hq, Hkv, n, kv_len, window):
    rng = np.random.default_rng(D + P + Hq + sum(kv_len))
    cache, table = _fill(rng, len(n), Hkv, D, P, kv_len)
    q = rng.standard_normal((sum(n) + 2, Hq, D)) * 2
    _check_attention(q, cache, table, n, kv_len, P, D ** -0.5, window)


def test_attention_splits_one_long_context():
    rng = np.random.default_rng(3)
    cache, table = _fill(rng, 2, 1, 128, 64, [30000, 4])
    q = rng.standard_normal((3, 4, 128)) * 2
    _check_attention(q, cache, table, [2, 1], [30000, 4], 64, 128 ** -0.5)


def test_attention_many_requests():
    rng = np.random.default_rng(4)
    n = rng.integers(0, 7, 520)
    kv = n + rng.integers(0, 90, 520)
    cache, table = _fill(rng, 520, 1, 64, 16, kv)
    q = rng.standard_normal((int(n.sum()) + 1, 2, 64))
    _check_attention(q, cache, table, n, kv.astype(np.int32), 16, 0.125)


@pytest.mark.parametrize("seed,B,Hq,Hkv,D,P,top,most,window", [
    (0, 40, 8, 2, 128, 64, 2500, 6, 0), (1, 150, 6, 3, 64, 16, 700, 17, 100), (2, 3, 48, 2, 64, 128, 9000, 4, 0),
    (3, 301, 4, 4, 64, 32, 260, 3, 0), (4, 17, 64, 1, 128, 32, 1500, 9, 513)])
def test_attention_ragged_batches(seed, B, Hq, Hkv, D, P, top, most, window):
    """Batches whose items are cut over the machine, every row against fp64 (torch, one request at a time)."""
    rng = np.random.default_rng(seed)
    n = rng.integers(0, most + 1, B)
    kv = n + (rng.random(B) ** 2 * top).astype(np.int64)
    mp = int(-(-kv.max() // P)) + 1
    n_pages = B * mp
    table = torch.from_numpy(rng.permutation(n_pages).reshape(B, mp).astype(np.int32)).cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = torch.randint(0, 256, (n_pages, Hkv, _lib.dspark_cache_record_bytes(P, D)), generator=g, device="cuda",
                          dtype=torch.uint8)
    half = cache.shape[2] // 2
    for at in (half, 2 * half):      # scale bytes of 2^-3 .. 2^0 so that softmax is neither flat nor a single key
        cache[:, :, at - P * D // 16:at] = torch.randint(32, 56, (n_pages, Hkv, P * D // 16), generator=g,
                                                         device="cuda", dtype=torch.uint8)
    start = np.concatenate(([0], np.cumsum(n))).astype(np.int32)
    T = int(start[-1]) + 1
    q = torch.randn(T, Hq, D, generator=g, device="cuda").bfloat16()
    out = torch.full_like(q, 7.0)
    ws = _ws(_lib.dspark_cache_attention_workspace_size(B, Hq, Hkv, D))
    _lib.dspark_cache_attention(q, cache, table, _i32(start), _i32(kv), P, D ** -0.5, window, ws, out)
    assert _lib.dspark_get_device_status(ws) == 0 and (out[-1] == 7.0).all()
    grid = torch.tensor(np.concatenate((oc.GRID, -oc.GRID)), device="cuda")
    e4m3 = torch.tensor(np.concatenate((oc.E4M3, oc.E4M3)), device="cuda")
    grp, m = Hq // Hkv, torch.finfo(torch.float64).min
    for b in range(B):
        if n[b] == 0:
            continue
        rec = cache[table[b, : -(-int(kv[b]) // P)].long()]
        kvs = []
        for part in (0, 1):
            r = rec[:, :, part * half:(part + 1) * half]
            c = r[:, :, :P * D // 2].reshape(-1, Hkv, D // 32, P, 16)
            v = grid[torch.stack((c & 15, c >> 4), -1).int()].permute(1, 0, 3, 2, 4, 5).reshape(Hkv, -1, D // 16, 16)
            s = e4m3[r[:, :, P * D // 2:].int()].reshape(-1, Hkv, P, D // 16).transpose(0, 1).reshape(Hkv, -1, D // 16, 1)
            kvs.append((v * s).reshape(Hkv, -1, D)[:, : kv[b]])
        K, V = kvs
        x = torch.einsum("nhgd,hsd->nhgs", q[start[b]:start[b + 1]].double().reshape(n[b], Hkv, grp, D), K) * D ** -0.5
        i = torch.arange(n[b], device="cuda")[:, None] + int(kv[b] - n[b])
        key = torch.arange(int(kv[b]), device="cuda")
        hide = (key > i) | ((key <= i - window) if window else torch.zeros_like(key > i))
        p = torch.softmax(x.masked_fill(hide[:, None, None], m), -1)
        ref = torch.einsum("nhgs,hsd->nhgd", p, V).reshape(n[b], Hq, D)
        mean = torch.einsum("nhgs,hsd->nhgd", p, V.abs()).reshape(n[b], Hq, D)
        # P's rounding (2^-11, twice), scores of D products in fp32 (|q||k| * scale * D * 2^-23, twice), exp2 and sums
        size = (q[start[b]:start[b + 1]].double().norm(dim=-1).max() * K.norm(dim=-1).max() * D ** -0.5).item()
        lim = mean * (2.0 ** -10 + 2 * D * 2.0 ** -23 * size + 2.0 ** -19 + len(key) * 2.0 ** -23) + \
            len(key) * 2.0 ** -24 * V.abs().max() * p.amax(-1).reshape(n[b], Hq, 1)
        err = (out[start[b]:start[b + 1]].double() - ref).abs()
        assert (err <= lim * (1 + 2.0 ** -7) + ref.abs() * 2.0 ** -8).all(), (b, n[b], kv[b], err.max().item())


@pytest.mark.parametrize("gain", [1e-30, 1e-3, 300.0, 1e30])
def test_attention_query_sizes(gain):
    """Queries far outside f16's range, and scores that grow along the context so that the running maximum rises."""
    rng = np.random.default_rng(5)
    D, P, L = 64, 16, 900
    cache, table = _fill(rng, 1, 1, D, P, [0])
    table = rng.permutation(L // P + 2)[None].astype(np.int32)
    cache = np.zeros((L // P + 2, 1, P * D // 8 * 9), np.uint8)
    t = np.arange(L)
    k = rng.standard_normal((L, 1, D)) * (0.2 + 3 * (t / L)[:, None, None])
    oc.write(cache, table[0][t // P].astype(np.int64) * P + t % P, k, rng.standard_normal((L, 1, D)), P)
    q = rng.standard_normal((3, 4, D)) * gain
    q[1] = np.abs(q[1])
    q[0, 0] = 0
    _check_attention(q, cache, table, [3], [L], P, 0.125 / gain * (4 if gain == 300.0 else 1))


def test_attention_layer_scales():
    rng = np.random.default_rng(6)
    cache, table = _fill(rng, 2, 2, 128, 32, [200, 77], kg=2.0 ** -9, vg=64.0)
    q = rng.standard_normal((5, 4, 128))
    _check_attention(q, cache, table, [2, 3], [200, 77], 32, 2.0 ** 6, kg=2.0 ** -9, vg=64.0)


def test_attention_strided_queries_and_negative_scale():
    rng = np.random.default_rng(7)
    cache, table = _fill(rng, 1, 2, 64, 16, [50])
    wide = torch.from_numpy(rng.standard_normal((2, 8, 64))).to(torch.bfloat16).cuda()
    q = wide[:, 2:6]
    out, ref = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), None
    ws = _ws(_lib.dspark_cache_attention_workspace_size(1, 4, 2, 64))
    args = (torch.from_numpy(cache).cuda(), _i32(table), _i32([0, 2]), _i32([50]), 16)
    _lib.dspark_cache_attention(q, *args, -0.3, 0, ws, out)
    ref, lim = oc.attention(_np(q), cache, table, [0, 2], [50], 16, -0.3)
    assert (np.abs(_np(out) - ref) <= lim * (1 + 2.0 ** -7) + np.abs(ref) * 2.0 ** -8).all()


def test_attention_nan_query_stays_in_its_row():
    rng = np.random.default_rng(8)
    cache, table = _fill(rng, 1, 1, 64, 16, [300])
    q = torch.from_numpy(rng.standard_normal((2, 4, 64))).to(torch.bfloat16).cuda()
    clean = torch.zeros_like(q)
    dirty = torch.zeros_like(q)
    ws = _ws(_lib.dspark_cache_attention_workspace_size(1, 4, 1, 64))
    args = (torch.from_numpy(cache).cuda(), _i32(table), _i32([0, 2]), _i32([300]), 16, 0.125, 0, ws)
    _lib.dspark_cache_attention(q, *args, clean)
    q[1, 2, 5] = float("nan")
    _lib.dspark_cache_attention(q, *args, dirty)
    assert torch.isnan(dirty[1, 2]).all()
    keep = torch.ones(2, 4, dtype=torch.bool, device="cuda")
    keep[1, 2] = False
    assert torch.equal(dirty[keep], clean[keep])


def test_attention_reports_bad_pages_and_lengths():
    rng = np.random.default_rng(9)
    cache, table = _fill(rng, 2, 1, 64, 16, [40, 40])
    cd = torch.from_numpy(cache).cuda()
    q = torch.from_numpy(rng.standard_normal((3, 2, 64))).to(torch.bfloat16).cuda()
    out = torch.zeros_like(q)
    ws = _ws(_lib.dspark_cache_attention_workspace_size(2, 2, 1, 64))
    bad = table.copy()
    bad[0, 1], bad[1, 0] = -1, len(cache)
    _lib.dspark_cache_attention(q, cd, _i32(bad), _i32([0, 1, 3]), _i32([40, 40]), 16, 0.125, 0, ws, out)
    assert _lib.dspark_get_device_status(ws) == _lib.DEV_PAGE_RANGE
    zero = np.where((bad < 0) | (bad >= len(cache)), 0, bad).astype(np.int32)     # page 0 is read instead
    ref, lim = oc.attention(_np(q), cache, zero, [0, 1, 3], [40, 40], 16, 0.125)
    assert (np.abs(_np(out) - ref) <= lim * (1 + 2.0 ** -7) + np.abs(ref) * 2.0 ** -8).all()
    for start, kv in (([0, 2, 1], [40, 40]), ([0, 1, 9], [40, 40]), ([0, 1, 3], [-3, 40]), ([0, 1, 3], [40, 1 << 20])):
        _lib.dspark_clear_device_status(ws)
        tb = np.zeros_like(table)          # every page is page 0: any clamped length stays readable
        _lib.dspark_cache_attention(q, cd, _i32(tb), _i32(start), _i32(kv), 16, 0.125, 0, ws, out)
        assert _lib.dspark_get_device_status(ws) == _lib.DEV_LENGTH_RANGE, (start, kv)


def test_attention_wait_that_runs_out(monkeypatch):
    rng = np.random.default_rng(10)
    kv = [3000, 500, 2000]
    cache, table = _fill(rng, 3, 1, 64, 16, kv)
    q = rng.standard_normal((9, 8, 64))
    ws = _ws(_lib.dspark_cache_attention_workspace_size(3, 8, 1, 64))
    qd = torch.from_numpy(q).to(torch.bfloat16).cuda()
    monkeypatch.setenv("DSPARK_WAIT_BUDGET_CYCLES", "200")
    _lib.dspark_cache_attention(qd, torch.from_numpy(cache).cuda(), _i32(table), _i32([0, 4, 5, 9]), _i32(kv), 16,
                                0.125, 0, ws, torch.empty_like(qd))
    assert _lib.dspark_get_device_status(ws) & _lib.DEV_TIMEOUT
    monkeypatch.delenv("DSPARK_WAIT_BUDGET_CYCLES")
    _lib.dspark_clear_device_status(ws)
    _check_attention(q, cache, table, [4, 1, 4], kv, 16, 0.125, ws=ws)


@pytest.mark.parametrize("tiles", [1, 2, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_runs_of_few_tiles(D, tiles):
    """As many equal items as CTAs: every CTA takes one item of 1, 2 or 3 tiles.  All values are 1.5 (the
    format holds it), so numerator and denominator are sums of the same probabilities: 1.5 after rounding to bf16."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(tiles)
    L, P = 128 * tiles - 5, 64
    k = rng.standard_normal((L, 1, D))
    cache = np.zeros((2 * tiles, 1, P * D // 8 * 9), np.uint8)
    oc.write(cache, np.arange(L), k, np.full((L, 1, D), 1.5), P)
    table = np.tile(np.arange(2 * tiles, dtype=np.int32), (sms, 1))
    q = torch.from_numpy(rng.standard_normal((sms, 2, D))).to(torch.bfloat16).cuda()
    ws = _ws(_lib.dspark_cache_attention_workspace_size(sms, 2, 1, D))
    for _ in range(20):
        out = torch.zeros_like(q)
        _lib.dspark_cache_attention(q, torch.from_numpy(cache).cuda(), _i32(table), _i32(np.arange(sms + 1)),
                                    _i32([L] * sms), P, D ** -0.5, 0, ws, out)
        assert (out == 1.5).all()
    assert _lib.dspark_get_device_status(ws) == 0


@pytest.mark.parametrize("start", [[0, 2, 1, 3], [0, 3, 0, 3], [3, 2, 1, 0], [0, 1, 3, -1]])
def test_attention_refuses_row_offsets_that_fall(start):
    """Two requests would write the same rows, and their work would not fit the sums made for T rows."""
    rng = np.random.default_rng(11)
    cache, table = _fill(rng, 3, 2, 64, 16, [40, 200, 40])
    q = torch.from_numpy(rng.standard_normal((3, 4, 64))).to(torch.bfloat16).cuda()
    ws = _ws(_lib.dspark_cache_attention_workspace_size(3, 4, 2, 64))
    args = (torch.from_numpy(cache).cuda(), _i32(table))
    out = torch.full_like(q, 7.0)
    _lib.dspark_cache_attention(q, *args, _i32(start), _i32([40, 200, 40]), 16, 0.125, 0, ws, out)
    assert _lib.dspark_get_device_status(ws) == _lib.DEV_LENGTH_RANGE
    assert (out == 7.0).all()
    _check_attention(q.float().cpu().numpy(), cache, table, [1, 1, 1], [40, 200, 40], 16, 0.125, extra=0,
                     ws=_ws(ws.nbytes))


@pytest.mark.parametrize("B,n,L", [(1, 20000, 1 << 20), (64, 20000, 1 << 17)])
def test_attention_of_a_long_prompt(B, n, L):
    """One long prompt alone, and in a batch of other seats; the first is more work than 32-bit sums hold.  Keys are
    zero, so all weights are equal; dim d of the values is 1.5 up to its own position and 0 behind it, so the result
    is 1.5 times a ratio of two counts, and every sum on the way is exact in fp32."""
    Hq, D, P, cap = 48, 64, 128, 1 << 20
    pages = L // P
    cut = torch.linspace(1, L, D, dtype=torch.float64).long().cuda()
    v = (torch.arange(L, device="cuda")[:, None] < cut).to(torch.bfloat16)[:, None] * 1.5
    k = torch.zeros_like(v)
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.zeros((B, cap // P), dtype=torch.int32, device="cuda")
    seat = B // 2
    table[seat, :pages] = torch.randperm(pages, generator=g, device="cuda").int()
    t = torch.arange(L, device="cuda")
    slot = table[seat, t // P] * P + (t % P).int()
    cache = torch.empty((pages, 1, _lib.dspark_cache_record_bytes(P, D)), dtype=torch.uint8, device="cuda")
    ws = _ws(_lib.dspark_cache_attention_workspace_size(B, Hq, 1, D))
    _lib.dspark_qk_norm_rope(k, k, None, None, EPS1, None, None, False, None, torch.empty_like(k), None, ws, v=v,
                             cache=cache, slot=slot, page=P)
    start = _i32([0] * (seat + 1) + [n] * (B - seat))
    kv = _i32([0] * seat + [L] + [0] * (B - seat - 1))
    q = torch.randn(n + 3, Hq, D, generator=g, device="cuda").bfloat16()
    out = torch.full_like(q, 7.0)
    _lib.dspark_cache_attention(q, cache, table, start, kv, P, D ** -0.5, 0, ws, out)
    assert _lib.dspark_get_device_status(ws) == 0
    see = torch.arange(L - n + 1, L + 1, device="cuda")[:, None]
    ref = (1.5 * torch.minimum(cut, see).double() / see)[:, None]
    # the reciprocal and the product in fp32, then half a step of bf16
    assert ((out[:n].double() - ref).abs() <= ref * (2.0 ** -8 + 2.0 ** -22)).all()
    assert (out[n:] == 7.0).all()


@pytest.mark.parametrize("B,G,T,max_pages,pool", [(5, 5, 12, 9, 30), (5, 5, 300, 9, 30), (300, 4, 1100, 8, 700),
                                                  (4096, 3, 9000, 3, 5000), (3, 70, 0, 20, 30), (64, 1 << 20, 2500, 8, 300)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_of_any_number_of_rows(B, G, T, max_pages, pool, in_place):
    """Arrays shorter or longer than the batch's rows, and the lengths that the rows cover."""
    P = 16
    rng = np.random.default_rng(B + T)
    t = oc.Tables(B, max_pages, rng.permutation(pool).tolist())
    d = DeviceTables(t, pool, B, 0, P)
    d.slot, d.pos = _i32([7] * T), _i32([7] * T)
    ctx = np.where(rng.random(B) < 0.2, -1, rng.integers(0, 9, B))
    ell = rng.integers(0, min(G, 60) + 1, B)
    ell_d = _i32(ell)
    granted = ell_d if in_place else _i32([7] * B)
    # contexts that are there already
    for b, x in enumerate(ctx):
        if x > 0 and t.free:
            t.rows[b].append(t.free.pop())
    d.table, d.held = _i32(t.table()), _i32([len(r) for r in t.rows])
    d.free, d.count = _i32(t.free + [-1] * (pool - len(t.free))), _i32([len(t.free)])
    _lib.dspark_cache_plan_rows(_i32(ctx), ell_d, G, d.table, d.held, d.free, d.count, P, d.ws, d.q_start, d.kv, d.slot,
                                d.pos, ell_out=granted)
    start, kv, slot, pos, full = t.plan(ctx.tolist(), ell.tolist(), min(G, 60), P)
    m = start[-1]
    slot, pos = slot[:m], pos[:m]
    cut = np.minimum(start, T)
    n = np.diff(cut)
    d.check(t)
    assert d.q_start.tolist() == cut.tolist()
    assert d.kv.tolist() == np.where(ctx < 0, 0, ctx + n).tolist()
    assert d.slot.tolist() == (slot + [-1] * T)[:T] and d.pos.tolist() == (pos + [-1] * T)[:T]
    assert granted.tolist() == np.maximum(n - 1, 0).tolist()
    assert _lib.dspark_get_device_status(d.ws) == (_lib.DEV_CACHE_FULL if full or m > T else 0)


def test_commit_of_a_round_clears_requests_without_rows():
    t = oc.Tables(4, 2, list(range(6)))
    d = DeviceTables(t, 6, 4, 2, 16)
    ctx = [3, -1, 32, 0]
    t.rows = [[5], [], [4, 3], []]
    t.free = [0, 1, 2]
    d.table, d.held = _i32(t.table()), _i32([1, 0, 2, 0])
    d.free, d.count = _i32([0, 1, 2, -1, -1, -1]), _i32([3])
    d.plan(_i32(ctx), _i32([2, 0, 1, 0]))
    start, *_ = t.plan(ctx, [2, 0, 1, 0], 2, 16)
    _lib.dspark_clear_device_status(d.ws)
    nout, acc = _i32([2, 1, 2, 1]), _i32([1, 0, 1, 0])
    tokens = _i32([[5, 6, -1], [7, -1, -1], [8, 9, -1], [4, -1, -1]])
    _lib.dspark_cache_commit_round(_i32(ctx), d.q_start, nout, acc, tokens, None, d.table, d.held, d.free, d.count, 16,
                                   d.ws, d.ctx_out)
    assert nout.tolist() == [2, 0, 0, 1] and acc.tolist() == [1, 0, 0, 0]
    assert tokens.tolist() == [[5, 6, -1], [-1] * 3, [-1] * 3, [4, -1, -1]]
    assert d.ctx_out.tolist() == t.commit(ctx, start, [2, 0, 0, 1], None, 16) == [5, -1, 32, 1]
    d.check(t)
    assert _lib.dspark_get_device_status(d.ws) == 0


@pytest.mark.parametrize("window", [0, 1 << 20, (1 << 31) - 5, (1 << 31) - 1])
def test_attention_windows_wider_than_the_context(window):
    """Five tokens of a request that holds one or three: the first have negative positions and see nothing."""
    rng = np.random.default_rng(12)
    cache, table = _fill(rng, 3, 1, 64, 16, [1, 3, 200])
    q = rng.standard_normal((15, 2, 64))
    _check_attention(q, cache, table, [5, 5, 5], [1, 3, 200], 16, 0.125, window)


@pytest.mark.parametrize("T", [1, 5])
def test_norm_in_place_beside_its_neighbours(T):
    """In place on rows that share one buffer: a single token's slices, and stacked dense arrays."""
    g = torch.Generator().manual_seed(T)
    Hq, Hkv, D = 4, 2, 64
    flat = torch.randn(T * (Hq + 2 * Hkv) * D, generator=g).bfloat16().cuda()
    q, k, v = (x.view(T, -1, D) for x in flat.split([T * Hq * D, T * Hkv * D, T * Hkv * D]))
    pos, freq = _i32(range(T)), torch.rand(32, generator=g).cuda()
    ref = torch.empty_like(q), torch.empty_like(k)
    caches = [_cache(1, Hkv, 16, D) for _ in range(2)]
    ws = _ws()
    for (qo, ko), cache in zip((ref, (q, k)), caches):
        _lib.dspark_qk_norm_rope(q, k, None, None, EPS1, pos, freq, False, None, qo, ko, ws, v=v, cache=cache, slot=pos,
                                 page=16)
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1]) and torch.equal(*caches)
    with pytest.raises(_lib.DsparkError):
        _lib.dspark_qk_norm_rope(q, k, None, None, EPS1, pos, freq, False, None, q, v, ws, v=v, cache=caches[0], slot=pos,
                                 page=16)
    assert _lib.dspark_get_device_status(ws) == 0


@pytest.mark.parametrize("down", [20.0, 22.5, 24.4, 25.6, 28.0])
def test_attention_of_one_key_over_a_flat_tail(down):
    """The first key's weight is 2^down times every other's, its value is 0, and one CTA has the whole context: the
    result is what the tail adds up to.  A weight is off by half a step of f16 at 2^7 times its size: 2^-32, or 2^-11
    of itself."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    D, P, pages = 64, 128, 1024
    N = pages * P - 1
    rec = _lib.dspark_cache_record_bytes(P, D)
    k, v = np.zeros((pages * P, 1, D)), np.full((pages * P, 1, D), 6.0)
    k[0, 0, 0], v[0] = 6.0, 0.0
    cache = np.zeros((pages, 1, rec), np.uint8)
    one = np.zeros((3, 1, rec), np.uint8)
    oc.write(one, np.arange(2 * P), k[:2 * P], v[:2 * P], P)
    cache[0], cache[1:] = one[0], one[1]
    q = torch.zeros(sms, 2, D, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 4.0
    out = torch.zeros_like(q)
    ws = _ws(_lib.dspark_cache_attention_workspace_size(sms, 2, 1, D))
    _lib.dspark_cache_attention(q, torch.from_numpy(cache).cuda(), _i32(np.tile(np.arange(pages), (sms, 1))),
                                _i32(np.arange(sms + 1)), _i32([pages * P] * sms), P, down * np.log(2.0) / 24, 0, ws, out)
    assert _lib.dspark_get_device_status(ws) == 0
    w = 2.0 ** -down
    ref = 6.0 * N * w / (1 + N * w)
    # ... the scale's and the score's rounding in fp32 (down * 2^-22), the output's half step
    tol = 6.0 * N * max(2.0 ** -32, w * 2.0 ** -11) + ref * (down * 2.0 ** -22 + 2.0 ** -8)
    assert (out.double() - ref).abs().max().item() <= tol


def _near_border(x, grid):
    """Is x within 2^-22 of a midpoint of the grid (where rounding the divisor to fp32 may turn the code)?"""
    mid = (grid[1:] + grid[:-1]) / 2
    i = np.clip(np.searchsorted(mid, x), 1, len(mid) - 1)
    return np.minimum(np.abs(x - mid[i]), np.abs(x - mid[i - 1])) <= x * 2.0 ** -22


@pytest.mark.parametrize("kg,vg", [(0.3, 1.7e-5), (1.0 / 3, 12345.678), (6.1e-17, 9.9e18)])
def test_cache_with_layer_scales_of_any_value(kg, vg):
    """Layer scales that are no powers of two: 6 g and scale * g round to fp32, so a code may turn at a border only."""
    T, Hkv, D, P = 200, 2, 128, 32
    kg, vg = float(np.float32(kg)), float(np.float32(vg))
    gen = torch.Generator().manual_seed(13)
    k, v = ((torch.randn(T, Hkv, D, generator=gen) * torch.exp(torch.randn(T, Hkv, 1, generator=gen)) * g).cuda()
            for g in (kg, vg))
    slot, ws, cache = _i32(np.random.default_rng(0).permutation(256)[:T]), _ws(), _cache(8, Hkv, P, D)
    _lib.dspark_qk_norm_rope(k, k, None, None, EPS1, None, None, False, None, torch.empty_like(k), None, ws, v=v,
                             cache=cache, slot=slot, page=P, k_scale=kg, v_scale=vg)
    out = torch.empty_like(k), torch.empty_like(v)
    _lib.dspark_cache_read(cache, slot, P, *out, ws, k_scale=kg, v_scale=vg)
    assert _lib.dspark_get_device_status(ws) == 0
    stored = oc.read(cache.cpu().numpy(), slot.cpu().numpy(), P, D)
    for x, g, y, o in zip((_np(k), _np(v)), (kg, vg), stored, out):
        code, sc = oc.quantise(x, g)
        off = (y != oc.dequantise(code, sc)).reshape(T, Hkv, -1, 16)
        top = np.abs(x).reshape(T, Hkv, -1, 16).max(-1) / (6 * g)
        with np.errstate(divide="ignore", invalid="ignore"):
            near = _near_border(np.abs(x).reshape(off.shape) / (oc.E4M3[sc] * g)[..., None], oc.GRID)
        assert not (off & ~near & ~_near_border(top, oc.E4M3[:127])[..., None]).any()
        assert off.mean() < 1e-3
        assert (np.abs(_np(o) - y * g) <= np.abs(y * g) * 2.0 ** -24).all()


def test_attention_layer_scales_of_any_value():
    rng = np.random.default_rng(14)
    kg, vg = float(np.float32(0.3)), float(np.float32(7.7))
    cache, table = _fill(rng, 2, 2, 64, 16, [300, 77], kg=kg, vg=vg)
    q = rng.standard_normal((5, 4, 64))
    _check_attention(q, cache, table, [2, 3], [300, 77], 16, 0.4, kg=kg, vg=vg)
