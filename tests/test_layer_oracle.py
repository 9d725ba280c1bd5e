"""Pins of oracle/layer_oracle.py against closed forms, differences and the other oracle."""
import numpy as np
import pytest

from oracle import layer_oracle as lo
from oracle import muir_oracle as mo


def _inputs(B=2, T=7, H=2, dk=3, dv=4, seed=0):
    r = np.random.default_rng(seed)
    q, k = r.normal(size=(B, T, H, dk)), r.normal(size=(B, T, H, dk))
    return q, k, r.normal(size=(B, T, H, dv)), -r.uniform(0.01, 1.0, H), r.normal(size=(B, H, dk, dv)), r


def test_forward_is_the_decayed_sum_over_earlier_tokens():
    q, k, v, ld, S0, _ = _inputs()
    y, S = lo.lin_forward(q, k, v, ld, 0.5, None, S0)
    B, T, H, _ = q.shape
    for b in range(B):
        for h in range(H):
            for t in range(T):
                want = sum(np.exp(ld[h] * (t - s)) * (q[b, t, h] @ k[b, s, h]) * v[b, s, h] for s in range(t + 1))
                want = want + np.exp(ld[h] * (t + 1)) * (S0[b, h].T @ q[b, t, h])
                np.testing.assert_allclose(y[b, t, h], 0.5 * want, rtol=1e-12, atol=1e-12)


def test_forward_is_the_gated_delta_rule_without_erase_and_gates():
    q, k, v, ld, S0, _ = _inputs(dk=4)
    B, T, H, dk = q.shape
    one = np.ones_like(k)
    la = np.broadcast_to(ld[None, None, :, None], k.shape)
    y, S = mo.forward(q, k, v, 0 * one, np.ones_like(v), one, None, la, np.ones((H, dk)), S0=S0)
    y2, S2 = lo.lin_forward(q, k, v, ld, 1.0, None, S0)
    np.testing.assert_allclose(y2, y, rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(S2, S, rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("lengths", [None, [7, 3], [0, 9]])
def test_backward_against_differences(lengths):
    q, k, v, ld, S0, r = _inputs()
    dy, dS_T = r.normal(size=v.shape), r.normal(size=S0.shape)

    def loss(q, k, v, S0):
        y, S = lo.lin_forward(q, k, v, ld, 0.7, lengths, S0)
        return np.sum(y * dy) + np.sum(S * dS_T)
    g = lo.lin_backward(q, k, v, ld, dy, 0.7, lengths, S0, dS_T)
    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dS0", S0)):
        for _ in range(12):
            i = tuple(r.integers(0, n) for n in x.shape)
            old = x[i]
            x[i] = old + 1e-6
            up = loss(q, k, v, S0)
            x[i] = old - 1e-6
            down = loss(q, k, v, S0)
            x[i] = old
            assert abs((up - down) / 2e-6 - g[name][i]) < 1e-6 * (1 + abs(g[name][i])), (name, i)


def test_norm_backward_against_differences():
    r = np.random.default_rng(3)
    x, res, w, dy, dh = (r.normal(size=s) for s in ((5, 8), (5, 8), (8,), (5, 8), (5, 8)))

    def loss(x, w):
        y, h, _ = lo.rms_norm(x, w, res)
        return np.sum(y * dy) + np.sum(h * dh)
    _, h, rstd = lo.rms_norm(x, w, res)
    dx, dw = lo.rms_norm_backward(dy, h, w, rstd, dh)
    for g, a in ((dx, x), (dw, w)):
        for i in np.ndindex(a.shape):
            old = a[i]
            a[i] = old + 1e-6
            up = loss(x, w)
            a[i] = old - 1e-6
            down = loss(x, w)
            a[i] = old
            assert abs((up - down) / 2e-6 - g[i]) < 1e-6 * (1 + abs(g[i]))


def test_e4m3_table():
    # every e4m3 number is its own nearest; midpoints go to the even code
    vals = [(1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6 for e in range(16) for m in range(8)][:127]
    vals = np.array(vals)
    assert vals[-1] == 448.0
    np.testing.assert_array_equal(lo.e4m3(vals), vals)
    mid = (vals[:-1] + vals[1:]) / 2
    even = np.where(np.arange(126) % 2 == 0, vals[:-1], vals[1:])
    np.testing.assert_array_equal(lo.e4m3(mid), even)
    assert lo.e4m3(np.array([1e9, -1e9])).tolist() == [448.0, -448.0]


def test_w4_layout_reads_back():
    r = np.random.default_rng(5)
    codes, scales = r.integers(0, 16, (19, 256)).astype(np.uint8), r.normal(size=(19, 8))
    wq, ws = lo.w4_layout(codes, scales)
    assert wq.shape == (2, 2, 1024) and ws.shape == (2, 2, 4, 16)
    # output 17 = row 1 of tile 1, input 128 + 32*2 + 8*3 + 5: word 2 of lane (1, 3), nibble 5
    byte = (1 * 4 + 3) * 32 + 2 * 4 + 5 // 2
    assert wq[1, 1, byte] >> 4 == codes[17, 128 + 64 + 24 + 5]
    assert ws[1, 1, 2, 1] == scales[17, 4 + 2]
    assert (wq[1, 0, 16:32] != 0x88).sum() == 0  # outputs 24.. of 19 are padding
