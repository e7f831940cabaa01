"""The oracle's rotary positions and cache rows by hand and by identities."""
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
