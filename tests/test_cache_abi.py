"""The cache and attention calls without a GPU: every documented refusal
comes back from the host checks, before any CUDA call."""
import ctypes
import math

import pytest
import torch

from speculative_decoding_draft_rank_b200 import _lib, build

A = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100008)
WS = ctypes.c_void_p(0x200000)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_sizes(lib):
    assert _lib.dspark_cache_record_bytes(64, 128) == 9216 and _lib.dspark_cache_record_bytes(16, 64) == 1152
    assert _lib.dspark_cache_record_bytes(48, 128) == 0 and _lib.dspark_cache_record_bytes(64, 96) == 0
    f = _lib.dspark_cache_attention_workspace_size
    assert 0 < f(1, 1, 1, 64) < f(4096, 64, 8, 128) < 16 << 20
    assert f(0, 8, 8, 64) == 0 and f(4097, 8, 8, 64) == 0 and f(1, 7, 2, 64) == 0 and f(1, 8, 8, 80) == 0
    assert f(1, 2048, 8, 64) == 0


def _plan(lib, B=4, G=5, P=64, mp=8, n=100, ws=WS, wsb=256, null=None):
    p = [A] * 10
    if null is not None:
        p[null] = None
    return lib.dspark_cache_plan(p[0], p[1], B, G, P, mp, n, p[2], p[3], p[4], p[5], ws, wsb, p[6], p[7], p[8], p[9],
                                 None)


def test_plan_refusals(lib):
    for bad in (dict(B=0), dict(B=4097), dict(G=-1), dict(G=(1 << 20) + 1), dict(B=4096, G=4096), dict(P=48),
                dict(mp=0), dict(n=0), dict(n=1 << 26), dict(mp=(1 << 24) + 1)):
        assert _plan(lib, **bad) == 1, bad
    for k in range(10):
        assert _plan(lib, null=k) == 1, k
    assert _plan(lib, ws=None) == 3 and _plan(lib, wsb=255) == 3 and _plan(lib, ws=ctypes.c_void_p(0x200010)) == 3


def test_commit_refusals(lib):
    f = lib.dspark_cache_commit

    def call(B=4, P=64, mp=8, n=100, ws=WS, wsb=256, null=None):
        p = [A] * 8
        if null is not None:
            p[null] = None
        return f(p[0], p[1], p[2], None, B, P, mp, n, p[3], p[4], p[5], p[6], ws, wsb, p[7], None)

    assert call(B=0) == 1 and call(P=8) == 1 and call(mp=0) == 1 and call(n=0) == 1
    for k in range(8):
        assert call(null=k) == 1, k
    assert call(ws=None) == 3 and call(wsb=0) == 3


def _norm(lib, q=A, qs=1024, k=A, ks=512, v=A, vs=512, wq=A, wk=A, eps=1e-6, pos=A, freq=A, rot=64, T=4, Hq=8, Hkv=4,
          D=128, dt=1, qo=A, ko=A, cache=A, slot=A, P=64, n=10, kg=1.0, vg=1.0, ws=WS, wsb=256):
    return lib.dspark_qk_norm_rope(q, qs, k, ks, v, vs, wq, wk, eps, pos, freq, rot, 0, None, T, Hq, Hkv, D, dt, qo,
                                   ko, cache, slot, P, n, kg, vg, ws, wsb, None)


def test_norm_refusals(lib):
    assert _norm(lib, dt=7) == 2
    for bad in (dict(T=-1), dict(T=(1 << 24) + 1), dict(Hq=6), dict(Hkv=0), dict(Hq=2048, Hkv=1024), dict(D=96),
                dict(rot=48), dict(rot=160), dict(rot=-32), dict(eps=-1.0), dict(eps=math.nan), dict(q=None),
                dict(k=None), dict(qo=None), dict(ko=None, cache=None), dict(pos=None), dict(freq=None),
                dict(v=None), dict(slot=None), dict(P=24), dict(n=0), dict(kg=0.0), dict(vg=-1.0),
                dict(kg=math.inf), dict(vg=math.nan), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(wq=ODD),
                dict(wk=ODD), dict(qo=ODD), dict(ko=ODD), dict(cache=ODD), dict(qs=1023), dict(qs=1028),
                dict(ks=511), dict(vs=500)):
        assert _norm(lib, **bad) == 1, bad
    assert _norm(lib, ws=None) == 3 and _norm(lib, wsb=128) == 3
    assert _norm(lib, T=0) == 0                     # nothing to do, nothing launched


def test_read_refusals(lib):
    def call(cache=A, slot=A, T=3, Hkv=4, D=64, P=16, n=9, kg=1.0, vg=1.0, dt=1, ko=A, vo=A, ws=WS, wsb=256):
        return lib.dspark_cache_read(cache, slot, T, Hkv, D, P, n, kg, vg, dt, ko, vo, ws, wsb, None)

    assert call(dt=3) == 2
    for bad in (dict(cache=None), dict(slot=None), dict(T=-1), dict(Hkv=0), dict(D=32), dict(P=0), dict(n=0),
                dict(kg=0.0), dict(vg=math.inf), dict(ko=None), dict(vo=ODD), dict(cache=ODD)):
        assert call(**bad) == 1, bad
    assert call(ws=None) == 3 and call(T=0) == 0


def _attend(lib, q=A, qs=1024, cache=A, table=A, start=A, kv=A, B=4, T=24, Hq=8, Hkv=4, D=128, P=64, mp=8, n=100,
            scale=0.1, kg=1.0, vg=1.0, window=0, dt=1, ws=WS, wsb=1 << 24, out=ctypes.c_void_p(0x900000)):
    return lib.dspark_cache_attention(q, qs, cache, table, start, kv, B, T, Hq, Hkv, D, P, mp, n, scale, kg, vg,
                                      window, dt, ws, wsb, out, None)


def test_attention_refusals(lib):
    assert _attend(lib, dt=0) == 2 and _attend(lib, dt=5) == 2
    for bad in (dict(B=0), dict(B=5000), dict(T=-1), dict(Hq=9), dict(Hkv=0), dict(D=256), dict(P=100), dict(mp=0),
                dict(n=0), dict(scale=math.nan), dict(scale=math.inf), dict(kg=0.0), dict(vg=-2.0), dict(window=-1),
                dict(q=None), dict(cache=None), dict(table=None), dict(start=None), dict(kv=None), dict(out=None),
                dict(q=ODD), dict(cache=ODD), dict(qs=1000), dict(qs=1028),
                dict(B=4096, T=1 << 20, Hq=64, Hkv=64, mp=1 << 20, P=128, n=1 << 20)):
        assert _attend(lib, **bad) == 1, bad
    assert _attend(lib, ws=None) == 3 and _attend(lib, wsb=4096) == 3
    for at in (0x100000, 0x100000 + 24 * 2048 - 16, 0x100000 - 24 * 2048 + 16):   # out over q
        assert _attend(lib, out=ctypes.c_void_p(at)) == 1
    assert _attend(lib, T=0) == 0


def test_injected_errors_come_back(lib, monkeypatch):
    monkeypatch.setenv("DSPARK_INJECT_ERROR", "dspark_cache_attention=4")
    assert _attend(lib) == 4
    monkeypatch.setenv("DSPARK_INJECT_ERROR", "dspark_cache_plan=4")
    assert _plan(lib) == 4


def test_binding_refuses_host_tensors_and_wrong_types(lib):
    i = torch.zeros(8, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        _lib.dspark_cache_plan(i[:2], i[:2], 1, torch.zeros(2, 4, dtype=torch.int32), i[:2], i, i[:1], 16, ws, i[:3],
                               i[:2], i[:4], i[:4])
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        _lib.dspark_qk_norm_rope(q, q, None, None, 1e-6, None, None, False, None, q, q, ws)
    with pytest.raises(ValueError):
        _lib.dspark_cache_attention(q, torch.zeros(4, 2, 99, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.int32),
                                    i[:2], i[:1], 16, 0.1, 0, ws, q)


@pytest.mark.parametrize("g", [2.0 ** -65, 1e-40, 2.0 ** 65, 3e38])
def test_layer_scales_out_of_range(lib, g):
    """Their reciprocals and products leave fp32's normal range."""
    assert _norm(lib, kg=g) == 1 and _norm(lib, vg=g) == 1
    assert _attend(lib, kg=g) == 1 and _attend(lib, vg=g) == 1
    assert lib.dspark_cache_read(A, A, 3, 4, 64, 16, 9, g, 1.0, 1, A, A, WS, 256, None) == 1
    assert _norm(lib, kg=2.0 ** -64, vg=2.0 ** 64, T=0) == 0


def test_score_scale_that_overflows(lib):
    assert _attend(lib, scale=1e38, kg=1e3) == 1 and _attend(lib, scale=-3e38) == 1
    assert _attend(lib, scale=1e30, kg=1e3, T=0) == 0


def test_empty_arrays_may_have_no_address(lib):
    assert _norm(lib, T=0, q=None, k=None, v=None, pos=None, slot=None, qo=None, ko=None) == 0
    assert lib.dspark_cache_read(A, None, 0, 4, 64, 16, 9, 1.0, 1.0, 1, None, None, WS, 256, None) == 0
    assert _attend(lib, T=0, q=None, out=None) == 0
    assert _norm(lib, T=0, D=96) == 1 and _attend(lib, T=0, cache=None) == 1


def test_attention_takes_long_prompts(lib):
    """The shape checks come before the workspace's: 3 says that the shape passed."""
    for ok in (dict(B=1, T=131072, Hq=64, Hkv=8, P=64, mp=2048, n=4096), dict(B=1, T=98304, Hq=64, Hkv=8, mp=1536),
               dict(B=256, T=1 << 21, Hq=64, Hkv=8, P=128, mp=1024), dict(B=1, T=1 << 20, Hq=64, Hkv=8, P=64, mp=1 << 14),
               dict(B=4096, T=36864, Hq=64, Hkv=8, P=64, mp=1 << 14)):
        assert _attend(lib, **{**dict(n=1 << 20, qs=8192, ws=None, out=ctypes.c_void_p(1 << 45)), **ok}) == 3, ok
    for bad in (dict(B=1, T=1 << 21, Hq=64, Hkv=8, P=64, mp=1 << 15), dict(B=4096, T=1 << 24, Hq=64, Hkv=8, P=128, mp=8192)):
        assert _attend(lib, **{**dict(n=1 << 20, qs=8192, ws=None, out=ctypes.c_void_p(1 << 45)), **bad}) == 1, bad


def test_plan_rows_and_commit_round_refusals(lib, monkeypatch):
    def plan(B=4, G=5, P=64, mp=8, n=100, T=24, ws=WS, wsb=256, null=None):
        p = [A] * 10
        if null is not None:
            p[null] = None
        return lib.dspark_cache_plan_rows(p[0], p[1], B, G, P, mp, n, p[2], p[3], p[4], p[5], T, ws, wsb, None, p[6],
                                          p[7], p[8], p[9], None)

    def commit(B=4, G=5, P=64, mp=8, n=100, ws=WS, wsb=256, null=None):
        p = [A] * 8
        if null is not None:
            p[null] = None
        return lib.dspark_cache_commit_round(p[0], p[1], p[2], None, None, None, B, G, P, mp, n, p[3], p[4], p[5], p[6],
                                             ws, wsb, p[7], None)

    for bad in (dict(B=0), dict(B=4097), dict(G=-1), dict(G=(1 << 20) + 1), dict(P=48), dict(mp=0), dict(n=0)):
        assert plan(**bad) == 1 and commit(**bad) == 1, bad
    assert plan(T=-1) == 1 and plan(T=(1 << 24) + 1) == 1
    for k in range(10):
        assert plan(null=k) == 1, k
    for k in range(8):
        assert commit(null=k) == 1, k
    assert plan(T=0, null=8, ws=None) == 3 and plan(T=0, null=9, ws=None) == 3      # no rows, no arrays
    assert plan(B=4096, G=1 << 20, ws=None) == 3
    assert plan(wsb=255) == 3 and commit(ws=None) == 3 and commit(wsb=0) == 3
    monkeypatch.setenv("DSPARK_INJECT_ERROR", "dspark_cache_plan_rows=4")
    assert plan() == 4
    monkeypatch.setenv("DSPARK_INJECT_ERROR", "dspark_cache_commit_round=4")
    assert commit() == 4


def test_norm_refuses_outputs_over_other_rows(lib):
    """T = 4, 8 query and 4 key heads of 128 bf16 dims: rows of 2048 and 1024 bytes."""
    at = lambda x: ctypes.c_void_p(0x1000000 + x)  # noqa: E731
    far = dict(q=at(0), k=at(0x10000), v=at(0x20000), qo=at(0x30000), ko=at(0x40000), cache=None, slot=None)
    for bad in (dict(qo=at(16)), dict(qo=at(0x10000)), dict(qo=at(0x10000 - 8192 + 16)), dict(ko=at(0)), dict(ko=at(0x10010)),
                dict(ko=at(0x30000 + 8176)), dict(ko=at(0x30000 - 4080)),
                dict(qs=2048, qo=at(0)), dict(ks=1024, ko=at(0x10000)),            # in place, but not dense
                dict(q=at(0), k=at(2048), v=at(2048 + 1024), qs=2048, ks=2048, vs=2048, qo=at(4 * 4096 - 2064)),
                dict(cache=at(0x80000), slot=at(0x70000), qo=at(0x20000)),
                dict(cache=at(0x80000), slot=at(0x70000), ko=at(0x20000))):
        assert _norm(lib, **{**far, **bad}) == 1, bad


def test_stride_of_a_single_token():
    """One token of a projection whose rows are not 16-byte multiples: there is no second row to be misaligned."""
    wide = torch.zeros(3, 4 * 64 + 3, dtype=torch.bfloat16)
    heads = wide[:, : 4 * 64].unflatten(1, (4, 64))
    one = heads[:1]
    assert one.stride(0) % 8 != 0
    assert _lib._rows(one, one.get_device(), "q") == (one.data_ptr(), 256)
    two = heads[:2]
    assert _lib._rows(two, two.get_device(), "q") == (two.data_ptr(), 259)
    with pytest.raises(ValueError):
        _lib._rows(two[:, :, ::2], two.get_device(), "q")
