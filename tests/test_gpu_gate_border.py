"""The gate's kept groups where their ranks nearly meet and their errors in 32 bits differ: groups of two like
scores beside groups of a large and a small one, whose ranks are sums that cancel."""
import numpy as np
import pytest

from tests.test_gpu_gate import check, draw, run_gate

pytestmark = pytest.mark.gpu

# (E, K, groups, kept groups): every number of experts to a lane's instance, whole lanes and parts of them
SIZES = [(64, 6, 8, 3), (128, 6, 8, 4), (256, 8, 8, 2), (384, 8, 8, 1), (384, 8, 8, 4), (1024, 8, 8, 3), (1024, 8, 16, 9),
         (1020, 8, 17, 5), (1000, 8, 20, 4), (96, 4, 24, 7)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from token_dispatch_gb300 import build
    build.build()


def lane_of(E, G):
    """Experts of a lane that a group's experts are dealt out to."""
    gs, lanes = E // G, 32 // G
    n = -(-gs // lanes)
    return min((n + 3) // 4 * 4 if gs % 4 == 0 and n > 2 else n, gs)


def score(l, sigmoid):
    l = np.asarray(l, np.float64)
    return 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l)


def logit(s, sigmoid):
    return np.log(s) - np.log1p(-s) if sigmoid else np.log(s)


def group_ranks(l, b, G, sigmoid):
    """The groups' ranks in 64 bits (of a softmax without its sum, where there is no bias)."""
    c = score(l, sigmoid) if sigmoid or b is None else score(l, False) / score(l, False).sum(axis=1, keepdims=True)
    c = np.sort((c if b is None else c + b.astype(np.float64)).reshape(len(l), G, -1), axis=2)
    return c[:, :, -1] + c[:, :, -2]


def crowd(E, G, KG, B, sigmoid, T, seed):
    """Rows whose groups all rank within 1e-3 of each other, as near as 1e-9.  Every other group has one score
    near the ranks and one near zero, with biases of +B and -B where there are any, at the two ends of a lane."""
    rng = np.random.default_rng(seed)
    gs, n = E // G, lane_of(E, G)
    l = np.full((T, E), -12.0)
    b = None if B is None else np.zeros(E, np.float32)
    total = 0.9 + 0.2 * rng.random((T, 1))
    rank = total + np.exp(rng.uniform(np.log(1e-9), np.log(1e-3), (T, G))) * rng.choice([-1, 1], (T, G))
    wide = rng.random(G) < 0.5
    wide[rng.integers(G)] = True
    for g in range(G):
        one, two = (0, n - 1) if rng.random() < 0.5 else (n - 1, 0)
        share = rng.uniform(0.75, 0.85, T) if wide[g] else 0.5 + 1e-3 * rng.standard_normal(T)
        first = share * rank[:, g]
        if b is not None and wide[g]:
            b[g * gs:(g + 1) * gs] = -B
            b[g * gs + one] = B
        l[:, g * gs + one] = logit(first, sigmoid)
        # the rest by what the first became in 32 bits
        l[:, g * gs + two] = logit(rank[:, g] - score(l[:, g * gs + one].astype(np.float32), sigmoid), sigmoid)
    l = l.astype(np.float32)
    if b is not None and not sigmoid:  # a softmax's scores are those above over their sum: so the biases, too
        b *= np.float32(1 / G)
    r = np.sort(group_ranks(l, b, G, sigmoid), axis=1)
    # ranks in 64 bits are off by a few 2^-53 of |B| + 1 at most: under 1e-13 here
    return l[r[:, G - KG] - r[:, G - KG - 1] > 1e-12], b


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("B", [None, 2.0, 10.0, 100.0])
@pytest.mark.parametrize("size", SIZES, ids=["E%d_K%d_G%d_%d" % s for s in SIZES])
def test_gate_groups_of_unlike_errors(size, B, sigmoid):
    E, K, G, KG = size
    for seed in range(2):
        l, b = crowd(E, G, KG, B, sigmoid, 150, seed + E + KG)
        assert len(l) > 140
        check(l, K, G, KG, sigmoid, b, True, False)


def test_gate_group_above_the_border_only_in_32_bits():
    """One row by hand: group 1's ranks of 20.44 and -19.56 lose 4e-5 in 32 bits beside group 0's two halves."""
    l = np.full((1, 384), -8.0)
    b = np.zeros(384)
    l[0, :2] = 0
    b[48:96] = -20
    b[48] = 20
    l[0, 48], l[0, 48 + 11] = -0.45998737, 0.46007168
    idx, _ = check(l, 8, 8, 1, True, b, True, False)
    assert (idx // 48 == 1).all()


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,KG", [(1000, 20, 4), (1020, 17, 5)])
def test_gate_groups_of_unlike_logits(E, G, KG, sigmoid):
    """Without a bias the errors are those of the logits' places: many rows, the kept groups alone compared (the
    two high experts of each are the chosen ones)."""
    l, _ = crowd(E, G, KG, None, sigmoid, 30000, 1)
    idx, _ = run_gate(l, 2 * KG, G, KG, sigmoid, None, False, False, 1.0)
    ref = np.sort(np.argsort(-group_ranks(l, None, G, sigmoid), axis=1, kind="stable")[:, :KG], axis=1)
    assert np.array_equal(np.sort(idx // (E // G), axis=1)[:, ::2], ref)


@pytest.mark.parametrize("sigmoid", [True, False], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("size", SIZES[:6], ids=["E%d_K%d_G%d_%d" % s for s in SIZES[:6]])
def test_gate_finite_biases_up_to_the_highest_number(size, sigmoid):
    """Biases that differ far above 1e30 order their groups and experts by what they are."""
    E, K, G, KG = size
    rng = np.random.default_rng(E + KG)
    l = rng.standard_normal((60, E)).astype(np.float32)
    l[::4, ::3] = -np.inf
    for values in ([3e30, 0.9e30, 0, 0], [1e29, 2e29, 0.99e30, 1.01e30, -2e30, 0, 0, 0], [3.4e38, 3e38, 2e38, 1e35, -3e38, 0, 0]):
        for group_max in (False, True):
            check(l, K, G, KG, sigmoid, rng.choice(values, E), True, group_max)
    # one expert far above 1e30 in every other group, two below it in the rest
    b = np.zeros((G, E // G))
    b[::2, 1] = 3e30
    b[1::2, :2] = 0.9e30
    for group_max in (False, True):
        check(l, K, G, KG, sigmoid, b.ravel(), True, group_max)


@pytest.mark.parametrize("kind", ["plain", "ties", "near", "masked"])
@pytest.mark.parametrize("size", SIZES, ids=["E%d_K%d_G%d_%d" % s for s in SIZES])
def test_gate_softmax_by_logits_alone(size, kind):
    """Groups ranked by their largest logit and rescaled gates: nothing asks for the row's maximum or sum, in
    rows that 64 bits settle neither."""
    E, K, G, KG = size
    check(draw(100, E, kind, E + KG), K, G, KG, False, None, True, True)
