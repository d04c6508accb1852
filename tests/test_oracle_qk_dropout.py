"""Pins of the 64-bit reference of query/key norms with rotation and of dropout: central differences, rotations as
complex products, the generator's published test vectors."""
import numpy as np
import pytest

from oracle import transformer as T

STEP, BAR = 1e-5, 1e-5  # truncation ~STEP^2, rounding ~1e-16 / STEP, of functions of order 1 to 100


def diff(f, x, i):
    keep = x[i]
    x[i] = keep + STEP
    hi = f()
    x[i] = keep - STEP
    lo = f()
    x[i] = keep
    return (hi - lo) / (2 * STEP)


def angles(rng, positions, pairs):
    a = rng.uniform(-3, 3, (positions, pairs))
    return np.stack([np.cos(a), np.sin(a)], -1)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dim,rot,interleaved", [(8, 8, False), (8, 8, True), (10, 6, False), (10, 4, True), (6, 0, False)])
def test_norm_rope_backward_is_the_derivative_of_the_forward(dim, rot, interleaved, norm):
    rng = np.random.default_rng(dim * 10 + rot)
    x, dy = rng.normal(size=(4, 3, dim)), rng.normal(size=(4, 3, dim))
    gamma = rng.uniform(0.5, 1.5, dim) if norm else None
    table, pos = (angles(rng, 9, rot // 2), np.array([0, 8, 3, 20])) if rot else (None, np.zeros(4, int))
    kw = dict(norm=norm, interleaved=interleaved)

    def loss():
        return float((T.norm_rope_forward(x, gamma, table, pos, 1e-2, **kw) * dy).sum())

    dx, dgamma = T.norm_rope_backward(x, dy, gamma, table, pos, 1e-2, **kw)
    for _ in range(20):
        i = tuple(int(rng.integers(n)) for n in x.shape)
        assert abs(diff(loss, x, i) - dx[i]) < BAR
    if norm:
        for c in range(dim):
            assert abs(diff(loss, gamma, (c,)) - dgamma[c]) < BAR
    else:
        assert dgamma is None


def test_rotation_is_a_complex_product_and_its_inverse():
    rng = np.random.default_rng(1)
    x, a = rng.normal(size=(2, 1, 6)), rng.uniform(-3, 3, (2, 3))
    table = np.stack([np.cos(a), np.sin(a)], -1)
    z = (x[..., :3] + 1j * x[..., 3:]) * np.exp(1j * a)[:, None]
    y = T.rotate(x, table, [0, 1], False)
    assert np.allclose(y, np.concatenate([z.real, z.imag], -1))
    assert np.allclose(T.rotate(y, table, [0, 1], False, back=True), x)
    w = (x[..., 0::2] + 1j * x[..., 1::2]) * np.exp(1j * a)[:, None]
    y = T.rotate(x, table, [0, 1], True)
    assert np.allclose(y[..., 0::2], w.real) and np.allclose(y[..., 1::2], w.imag)


def test_normed_heads_have_unit_mean_square():
    x = np.random.default_rng(2).normal(size=(5, 2, 16)) * 7
    assert np.allclose((T.norm_rope_forward(x, None, None, None, 0.0) ** 2).mean(-1), 1)


def test_philox_words_of_the_published_vectors():
    """The known answers of the generator's authors for counters and keys of zeros, and of this key and counter in the
    low words; the upper words of the counter are always zero here."""
    assert [int(v) for v in T.philox(0, [0])[0]] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


def philox_of_four(key, counter):
    """Philox4x32-10 in whole numbers, with all four words of the counter."""
    k, x = list(key), list(counter)
    for _ in range(10):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [b >> 32 ^ x[1] ^ k[0], b & 0xFFFFFFFF, a >> 32 ^ x[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return x


def test_philox_has_the_order_of_the_published_words():
    """The known answers with a key and a counter in all words pin the order of both; the reference, whose counter has zeros
    in its upper words, agrees with the same steps on other seeds and counters, their low words first."""
    ones, pi = [0xFFFFFFFF] * 4, [0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344]
    assert philox_of_four(ones[:2], ones) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert philox_of_four([0xA4093822, 0x299F31D0], pi) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]
    rng = np.random.default_rng(7)
    for _ in range(50):
        key, low = ([int(v) for v in rng.integers(0, 1 << 32, 2)] for _ in range(2))
        words = T.philox(key[0] | key[1] << 32, [low[0] | low[1] << 32])[0]
        assert [int(v) for v in words] == philox_of_four(key, low + [0, 0])


def test_philox_uses_all_words_of_seed_and_counter():
    base = T.philox(5, [7])[0]
    for seed, c in ((5 | 1 << 40, 7), (5, 7 | 1 << 40), (6, 7), (5, 8)):
        assert not np.any(T.philox(seed, [c])[0] == base)
    assert T.philox(5, [7]).max() < 1 << 32


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9, 1.0])
def test_dropout_keeps_its_share(p):
    n = 40000
    keep = T.dropout_keep((200, 200), p, 11, 3)
    assert abs(keep.mean() - (1 - p)) <= 5 * np.sqrt(p * (1 - p) / n)  # five standard deviations
    x = np.random.default_rng(0).normal(size=(200, 200))
    y = T.dropout(x, p, 11, 3)
    # p is held in fp32, off by p 2^-24 at most: 1 / (1 - p) by p 2^-24 / (1 - p) of itself, 9 x 2^-24 < 6e-7 at 0.9
    assert np.all(y[~keep] == 0) and np.allclose(y[keep], x[keep] / (1 - p) if p < 1 else 0, rtol=6e-7, atol=0)
    assert np.allclose(T.dropout(x, p, 11, 3, residual=x), y + x)


def test_dropout_counters_go_on():
    """A call on n elements uses (n + 3) / 4 counters: the words of one on all of them are those of two in turn."""
    a, b = T.dropout_keep((10,), 0.5, 9, 100), T.dropout_keep((6,), 0.5, 9, 103)
    both = T.dropout_keep((18,), 0.5, 9, 100)
    assert np.array_equal(both[:10], a) and np.array_equal(both[12:], b)
