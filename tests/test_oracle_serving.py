"""Pins of the float64 oracle of the serving operators (oracle/serving.py) against independent statements of
the same definitions: torch's e4m3 conversion, a search over the exponents, the bf16 MQA oracle."""
import numpy as np
import pytest
import torch

from oracle import mqa, serving as O


def test_e4m3_table_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(np.isnan(codes), np.isnan(O.TABLE))
    np.testing.assert_array_equal(codes[~np.isnan(codes)], O.TABLE[~np.isnan(codes)])


def test_round_e4m3_is_nearest_even_and_saturates():
    v = np.sort(O.TABLE[:127])
    mids = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9), [1e9, np.inf]])
    got = O.round_e4m3(np.concatenate([x, -x]))
    want = torch.from_numpy(np.minimum(x, 448.0)).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
    n = len(v) + len(mids)                      # the exact values and ties, which fp32 holds
    np.testing.assert_array_equal(got[:n], want[:n])
    np.testing.assert_array_equal(got[n:n + len(mids)], v[:-1])
    np.testing.assert_array_equal(got[n + len(mids):n + 2 * len(mids)], v[1:])
    np.testing.assert_array_equal(got[len(x) - 2:len(x)], [448.0, 448.0])
    np.testing.assert_array_equal(got[len(x):], -got[:len(x)])
    assert np.isnan(O.round_e4m3(np.nan))


@pytest.mark.parametrize("amax", [0.0, 1e-40, 448.0, 449.0, 447.9, 1.0, 1.75, 1.7500001, 3.3e38, np.inf, 2.0 ** -110])
def test_scale_is_the_smallest_that_holds(amax):
    s = O.scale_of(amax)
    fits = [e for e in range(-100, 121) if amax <= 448 * 2.0 ** e]
    assert s == 2.0 ** (fits[0] if fits else 120)


def test_append_then_attention_is_the_ring_oracle():
    """Values that e4m3 holds exactly: appending in chunks and attending gives the bf16 MQA oracle's rows."""
    rng = np.random.default_rng(0)
    H, D, ps, n, window = 2, 128, 16, 41, 20
    q = rng.integers(-4, 5, (n, H, D)) / 4.0
    v = rng.integers(-8, 8, (n, 1, D)) / 8.0
    k = np.zeros((n, 1, D))
    k[..., 0] = rng.integers(-8, 8, (n, 1))     # rotated by the oracle: rounded there, so read back from the pool
    qkv = np.concatenate([q.reshape(n, -1), k.reshape(n, -1), v.reshape(n, -1)], 1)
    P = 4
    table = np.array([[2, 0, 3]])
    kc, vc, ks, vs = np.zeros((P, 1, ps, D)), np.zeros((P, 1, ps, D)), np.ones((P, 1)), np.ones((P, 1))
    rows = []
    for a, b in ((0, 7), (7, 8), (8, 33), (33, 41)):
        qr, pools = O.append(qkv[a:b], [0, b - a], [a], table, kc, ks, vc, vs, H)
        kc, ks, vc, vs = pools["k"][0], pools["k"][1], pools["v"][0], pools["v"][1]
        o, _, _ = O.attention(qr, [0, b - a], [a], table, kc, ks, vc, vs, window, D ** -0.5)
        rows.append((qr, o))
    qr, got = (np.concatenate(x) for x in zip(*rows))
    p = np.arange(n)
    kd = (kc * ks[..., None, None])[table[0][p // ps], 0, p % ps]
    vd = (vc * vs[..., None, None])[table[0][p // ps], 0, p % ps]
    np.testing.assert_array_equal(vd, v[:, 0])
    want = mqa.attention_rows(qr[None], kd[None], vd[None], p[None], [(0, t) for t in range(n)], window)
    # the pool's scale rose while chunks came in only if a later one was larger; rows before see the earlier rounding
    np.testing.assert_allclose(got[-8:], want[-8:], rtol=1e-12, atol=1e-12)


def test_append_raises_the_scale_of_an_entered_page_only():
    ps, D = 16, 128
    kc = np.zeros((2, 1, ps, D))
    kc[:, :, :, 0] = 448.0
    qkv = np.zeros((1, 3 * D))
    qkv[0, 2 * D] = 4096.0                       # v; q and k are zero
    _, pools = O.append(qkv, [0, 1], [3], np.array([[1]]), kc, np.ones((2, 1)), kc, np.ones((2, 1)), 1)
    c, s, _ = pools["v"]
    assert s[1, 0] == 16 and s[0, 0] == 1
    np.testing.assert_array_equal(c[1, 0, :3, 0], 28.0)
    assert c[1, 0, 3, 0] == 256.0 and np.all(c[1, 0, 4:, 0] == 448.0)
    assert pools["k"][1][1, 0] == 1              # the key was zero: the page keeps its scale
