"""The cache oracle against what fixes it: hand-worked tables, the number
formats' own values, and attention's limiting cases."""
import numpy as np
import pytest
import torch

from oracle import cache as oc


def test_tables_by_hand():
    t = oc.Tables(3, 4, free=[9, 8, 7, 6, 5])
    t.rows = [[1], [], [2, 3]]
    # pages of 16: request 0 grows from 15 to 18 tokens (one page), 1 is new with 1 token, 2 stays inside its pages
    start, kv, slot, pos, full = t.plan([15, 0, 20], [2, 0, 1], 2, 16)
    assert start == [0, 3, 4, 6] and kv == [18, 1, 22] and not full
    assert slot == [1 * 16 + 15, 5 * 16, 5 * 16 + 1, 6 * 16, 3 * 16 + 4, 3 * 16 + 5, -1, -1, -1]
    assert pos == [15, 16, 17, 0, 20, 21, -1, -1, -1]
    assert t.free == [9, 8, 7]
    assert t.commit([15, 0, 20], start, [0, 0, 2], None, 16) == [15, 0, 22]
    assert t.free == [9, 8, 7, 6, 5]          # nothing kept: the list is as before
    assert t.rows == [[1], [], [2, 3]]
    assert t.commit([15, -1, 22], [0, 0, 0, 0], [0, 0, 0], [0, 0, 1], 16) == [15, -1, -1]
    assert t.rows == [[1], [], []] and t.free == [9, 8, 7, 6, 5, 3, 2]


def test_tables_run_dry_in_request_order():
    t = oc.Tables(3, 4, free=[4, 3])
    start, kv, slot, pos, full = t.plan([0, 0, 0], [40, 0, 0], 40, 16)   # 3 pages, 1, 1
    assert full and start == [0, 0, 0, 0] and t.free == [4, 3]
    start, *_, full = t.plan([0, 0, 0], [16, 0, 0], 40, 16)
    assert full and start == [0, 17, 17, 17] and t.free == []


def test_formats_match_torch():
    x = np.concatenate([np.linspace(0, 460, 5001), 2.0 ** np.linspace(-12, 9, 4001)])
    ref = torch.from_numpy(np.minimum(x, 448)).to(torch.float32).to(torch.float8_e4m3fn).float().double().numpy()
    got = oc.E4M3[oc._nearest(np.minimum(x.astype(np.float32).astype(np.float64), 448.0), oc.E4M3[:127])]
    assert np.array_equal(got, ref)
    for v, want in ((0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0), (3.5, 4.0), (5.0, 4.0), (5.01, 6.0)):
        assert oc.GRID[oc._nearest(np.array([v]), oc.GRID)[0]] == want


@pytest.mark.parametrize("P,D", [(16, 64), (32, 128), (128, 64)])
def test_write_then_read_is_the_quantised_value(P, D):
    rng = np.random.default_rng(P + D)
    cache = np.full((5, 2, P * D // 8 * 9), 255, np.uint8)
    slot = rng.permutation(5 * P)[:23]
    k, v = rng.standard_normal((2, 23, 2, D))
    k[3, 0, :16] = 0.0
    oc.write(cache, slot, k, v, P)
    gk, gv = oc.read(cache, slot, P, D)
    for x, y in ((k, gk), (v, gv)):
        assert np.array_equal(oc.dequantise(*oc.quantise(x)), y)
        big = np.abs(x.reshape(23, 2, -1, 16)).max(-1, keepdims=True)
        # half the widest grid step (1 of 6) and half a step of the scale (2^-4)
        assert (np.abs((x - y).reshape(23, 2, -1, 16)) <= big * (1 / 6 + 2.0 ** -4)).all()


def test_attention_limits():
    rng = np.random.default_rng(0)
    P, D, L = 16, 64, 37
    cache = np.zeros((3, 1, P * D // 8 * 9), np.uint8)
    table = np.array([[2, 0, 1]], np.int32)
    t = np.arange(L)
    k, v = rng.standard_normal((2, L, 1, D))
    oc.write(cache, table[0][t // P] * P + t % P, k, v, P)
    _, vq = oc.read(cache, table[0][t // P] * P + t % P, P, D)
    q = np.zeros((3, 2, D))
    out, _ = oc.attention(q, cache, table, [0, 3], [L], P, 1.0)
    for j in range(3):      # zero queries: the mean over what the token sees
        assert np.allclose(out[j, 0], vq[: L - 2 + j, 0].mean(0))
    out, _ = oc.attention(q, cache, table, [0, 3], [L], P, 1.0, window=1)
    for j in range(3):      # a window of one: the token's own value
        assert np.allclose(out[j, 1], vq[L - 3 + j, 0])
    out, _ = oc.attention(q, cache, table, [0, 3], [2], P, 1.0)
    assert (out[0] == 0).all() and np.allclose(out[1, 0], vq[0, 0])   # the first token sees no key


def test_rotation_keeps_pairs_lengths_and_turns_by_the_angle():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 2, 64))
    f = 10000.0 ** (-np.arange(16) / 16)
    for inter in (False, True):
        y = oc.norm_rope(x, None, 0.0, [0, 1, 7, 1 << 20], f, inter)
        assert np.allclose(y[0], x[0]) and np.allclose(y[..., 32:], x[..., 32:])
        ia = np.arange(0, 32, 2) if inter else np.arange(16)
        ib = ia + 1 if inter else ia + 16
        z, w = x[..., ia] + 1j * x[..., ib], y[..., ia] + 1j * y[..., ib]
        assert np.allclose(w, z * np.exp(1j * np.array([0, 1, 7, 1 << 20])[:, None] * f)[:, None])
