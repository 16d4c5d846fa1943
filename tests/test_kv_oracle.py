"""The plain definitions of the KV cache's operators, pinned by hand-worked
cases and by properties (CPU)."""
import numpy as np

from oracle import kv_cache as kv


def test_plan_by_hand():
    # pages of 4; request 0 grows into a second page, 1 ends (returns 7, 8),
    # 2 starts, 3 does not fit any more, 4 asks for nothing
    table = np.array([[5, -1, -1], [7, 8, -1], [-1, -1, -1], [-1, -1, -1], [9, -1, -1]])
    r = kv.plan([4, 6, 0, 0, 2], [2, -1, 5, 9, 0], table, [1, 2, -1, -1, -1], 2, 16, 4)
    # the stack is 1 2 7 8: 8 to request 0, then 7 and 2 to request 2; 1 is left
    assert r["block_table"].tolist() == [[5, 8, -1], [7, 8, -1], [7, 2, -1], [-1, -1, -1], [9, -1, -1]]
    assert r["granted"].tolist() == [2, 0, 5, 0, 0]
    assert r["seq_len"].tolist() == [6, 0, 5, 0, 2]
    assert r["q_start"].tolist() == [0, 2, 2, 7, 7, 7]
    assert r["slots"].tolist() == [32, 33, 28, 29, 30, 31, 8] + [-1] * 9
    assert r["positions"].tolist() == [4, 5, 0, 1, 2, 3, 4] + [-1] * 9
    assert r["free_count"] == 1 and r["free_list"].tolist() == [1, 2, -1, -1, -1]


def test_plan_first_come_first_served():
    # 2 free pages of 4: the second request's 9 rows do not fit; nobody behind
    # it is served either, not even without a new page
    table = np.full((3, 4), -1)
    table[2, 0] = 3
    r = kv.plan([0, 0, 1], [4, 9, 1], table, [0, 1], 2, 99, 4)
    assert r["granted"].tolist() == [4, 0, 0] and r["free_count"] == 1
    # too few rows in the step's buffers does the same
    r = kv.plan([0, 0, 1], [4, 3, 1], table, [0, 1], 2, 6, 4)
    assert r["granted"].tolist() == [4, 0, 0]
    # outgrowing the block table row asks for nothing and blocks nobody
    r = kv.plan([0, 15, 1], [4, 2, 1], table, [0, 1], 2, 99, 4)
    assert r["granted"].tolist() == [4, 0, 1]


def test_append_by_hand():
    codes = np.zeros((2, 1, 4, 16), np.int8)
    codes[1, 0, 0] = 100
    scale = np.array([[0.5], [0.01]], np.float32)
    x = np.zeros((2, 1, 16), np.float32)
    x[0, 0, :4] = [2.54, -1.27, np.nan, np.inf]
    # one request holds a row on page 1 and adds two: top 2.54 -> scale 0.02
    c, s = kv.append(codes, scale, x, np.array([[1]]), [3], [0, 2], 4)
    assert np.isclose(s[1, 0], 0.02) and s[0, 0] == np.float32(0.5)
    assert (c[1, 0, 0] == 50).all()
    assert c[1, 0, 1, :5].tolist() == [127, -64, 0, 127, 0]  # -63.5 to even
    assert (c[0] == 0).all()
    # the same rows into a page without earlier rows: its old scale is gone
    c, s = kv.append(codes, np.array([[0.5], [9.0]], np.float32), x, np.array([[1]]), [2], [0, 2], 4)
    assert np.isclose(s[1, 0], 0.02)


def test_append_error_is_half_a_step():
    g = np.random.default_rng(1)
    x = g.standard_normal((40, 3, 32)).astype(np.float32)
    table = np.array([[4, 2, 0]])
    c, s = kv.append(np.zeros((5, 3, 16, 32), np.int8), np.zeros((5, 3), np.float32), x, table, [40], [0, 40], 16)
    slots = [int(table[0, i // 16]) * 16 + i % 16 for i in range(40)]
    back = kv.read(c, s, slots, 16)
    step = np.repeat(s[table[0]], 16, 0)[:40, :, None]
    assert (np.abs(back - x) <= step * 0.5 * (1 + 1e-6)).all()
    assert (kv.read(c, s, [-1, 5 * 16], 16) == 0).all()


def test_attention_by_hand():
    # two cached rows with equal logits, then one page missing: the mean, then the row left, then nothing
    k = np.zeros((2, 1, 16, 16), np.int8)
    v = np.zeros((2, 1, 16, 16), np.int8)
    v[0, 0, 0], v[0, 0, 1], v[1, 0, 0] = 10, 30, 50
    one = np.ones((2, 1), np.float32)
    q = np.ones((1, 2, 16), np.float32)
    out, lse, *_ = kv.attention(q, k, v, one, one, np.array([[0, 1]]), [2], [0, 1], 16, 0.25)
    assert np.allclose(out, 20) and np.allclose(lse, np.log(2))
    out, lse, *_ = kv.attention(q, k, v, one, one, np.array([[-1, 1]]), [17], [0, 1], 16, 0.25)
    assert np.allclose(out, 50) and np.allclose(lse, 0)
    out, lse, *_ = kv.attention(q, k, v, one, one, np.array([[-1, 7]]), [17], [0, 1], 16, 0.25)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_attention_is_causal_and_windowed():
    g = np.random.default_rng(2)
    k = g.integers(-127, 128, (3, 1, 16, 16)).astype(np.int8)
    v = g.integers(-127, 128, (3, 1, 16, 16)).astype(np.int8)
    s = np.full((3, 1), 0.01, np.float32)
    q = g.standard_normal((20, 1, 16))
    table = np.array([[2, 0, 1]])
    out, lse, *_ = kv.attention(q, k, v, s, s, table, [35], [0, 20], 16, 0.25, window=7)
    kk = np.concatenate([k[p, 0] for p in table[0]]) * 0.01
    vv = np.concatenate([v[p, 0] for p in table[0]]) * 0.01
    for i in range(20):
        pos = 15 + i
        x = kk[pos - 6:pos + 1] @ q[i, 0] * 0.25
        p = np.exp(x)
        assert np.allclose(out[i, 0], p @ vv[pos - 6:pos + 1] / p.sum(), rtol=1e-5)
        assert np.allclose(lse[i, 0], np.log(p.sum()), rtol=1e-5)
