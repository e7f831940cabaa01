"""The oracle's rotary positions, cache rows and draws by hand and by identities."""
import numpy as np

import oracle


def test_rope_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    y = oracle.rope(x, [1], [np.pi / 2, np.pi])          # half layout: (1, 3), (2, 4)
    np.testing.assert_allclose(y[0, 0], [-3.0, -2.0, 1.0, -4.0, 9.0], atol=1e-15)
    y = oracle.rope(x, [1], [np.pi / 2, np.pi], rot_offset=1, interleaved=True)   # (2, 3), (4, 9)
    np.testing.assert_allclose(y[0, 0], [1.0, -3.0, 2.0, -4.0, -9.0], atol=2e-15)


def test_products_depend_on_distance_only():
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(2, 1, 1, 64))
    f = [10000.0 ** (-i / 32) for i in range(32)]
    dot = lambda p, j: float((oracle.rope(q, [p], f) * oracle.rope(k, [j], f)).sum())  # noqa: E731
    for p, j, d in ((5, 3, 1000), (100, 100, 77), (0, 40, 4096)):
        assert abs(dot(p, j) - dot(p + d, j + d)) < 1e-9
    y = oracle.rope(oracle.rope(q, [123], f), [123], f, inverse=True)
    np.testing.assert_allclose(y, q, atol=1e-12)


def test_latent_rows():
    rng = np.random.default_rng(1)
    kv = rng.normal(size=(3, 576))
    f = [10000.0 ** (-i / 32) for i in range(32)]
    w = rng.normal(size=512)
    r = oracle.latent_rows(kv, [7, 8, 9], f, w, 0.0)
    np.testing.assert_allclose(((r[:, :512] / w) ** 2).mean(axis=1), 1.0)
    np.testing.assert_allclose(r[:, 512:], oracle.rope(kv[:, None, 512:], [7, 8, 9], f)[:, 0])
    np.testing.assert_array_equal(oracle.latent_rows(kv, [7, 8, 9], f)[:, :512], kv[:, :512])


def test_draw_by_hand():
    p = np.array([0.1, 0.4, 0.2, 0.3])
    row = np.log(p)
    take = lambda u, **kw: oracle.draw(row, u, **kw)[0]  # noqa: E731
    assert [take(u) for u in (0.0, 0.05, 0.15, 0.45, 0.55, 0.65, 0.75, 0.999)] == \
        [0, 0, 1, 1, 2, 2, 3, 3]
    assert [take(u, top_k=2) for u in (0.0, 0.5, 0.6, 0.99)] == [1, 1, 3, 3]       # 0.4, 0.3
    assert [take(u, top_p=0.65) for u in (0.0, 0.57, 0.58, 0.99)] == [1, 1, 3, 3]   # 0.4 + 0.3
    assert [take(u, top_p=0.75) for u in (0.4, 0.5, 0.6, 0.7)] == [1, 2, 2, 3]      # and 0.2
    assert [take(u, min_p=0.6) for u in (0.5, 0.6)] == [1, 3]
    assert [take(u, top_k=3, top_p=0.5) for u in (0.5, 0.6)] == [1, 3]   # 0.4 of 0.9, then 0.7
    assert take(0.9, top_p=0.0) == 1 and take(0.9, temperature=0.0) == 1
    t, lp, _ = oracle.draw(row, 0.15)
    assert abs(lp - np.log(0.4)) < 1e-12
    assert abs(oracle.draw(row, 0.6, top_k=2)[1] - np.log(3 / 7)) < 1e-12
    # squared odds at half the temperature
    assert abs(oracle.draw(row, 0.3, temperature=0.5)[1] - np.log(0.16 / 0.30)) < 1e-12


def test_draw_ties_masks_and_margins():
    row = np.array([1.0, 2.0, 2.0, 2.0, -np.inf, np.nan])
    assert oracle.draw(row, 0.99, top_k=2)[0] == 2 and oracle.draw(row, 0.99, top_p=0.29)[0] == 1
    assert oracle.draw(row, 0.9999)[0] == 3 and oracle.draw(row, 1.0)[0] == 3
    assert oracle.draw(np.full(4, -np.inf), 0.5)[:2] == (0, -np.inf)
    assert oracle.draw(np.array([0.0, np.inf, 5.0, np.inf]), 0.6)[0] == 3
    w = np.log(np.array([0.25, 0.25, 0.5]))
    assert abs(oracle.draw(w, 0.3)[2] - 0.05) < 1e-9
    assert abs(oracle.draw(w, 0.3, top_p=0.76)[2] - 0.01) < 1e-9
