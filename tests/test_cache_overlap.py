"""Calls of the cache operators whose outputs lie over their inputs or over one
another are refused on the host, before the device is looked at: other thread
blocks still read, or also write, what one of them overwrites."""
import pytest
import torch

from tests.test_cache_abi import E4M3, call_commit, call_evict, call_tree, call_weights, fm  # noqa: F401  (fm: the fixture)

M = 1 << 24                                              # fake addresses, far apart: never dereferenced


def apart(*names):
    return {n: (i + 1) * M for i, n in enumerate(names)}


def clash(a, x, y, n):
    """Array y moved to where x, of n bytes, begins, and to its last 16 bytes."""
    return [{**a, y: a[x]}, {**a, y: a[x] + n - 16}]


# ---------------------------------------------------------------------------
# Eviction: B = 2 sequences, 2 heads, entries of 64 rows (out: 40), budget 32, bf16
# ---------------------------------------------------------------------------

EVICT = apart("kc", "vc", "acc", "ko", "vo", "ao", "sl", "bi", "oi", "kept", "ns")
ROWS_IN, ROWS_OUT = 2 * 64 * 2, 2 * 40 * 2               # rows of all heads and entries
EVICT_BYTES = dict(kc=ROWS_IN * 256, vc=ROWS_IN * 256, acc=ROWS_IN * 4, ko=ROWS_OUT * 256, vo=ROWS_OUT * 256,
                   ao=ROWS_OUT * 4, kept=2 * 2 * 32 * 4)


def in_place(**kw):
    a = {**EVICT, "oi": EVICT["bi"], **kw}
    return dict(a, ko=a["kc"], vo=a["vc"], ao=a["acc"], So=64)


@pytest.fixture
def past_the_checks(fm):  # noqa: F811
    """What a call that nothing is wrong with answers where there is no device."""
    if torch.cuda.is_available():
        pytest.skip("a device would be given the fake addresses")
    r = call_evict(fm, **EVICT)
    assert r != -1 and call_evict(fm, **in_place()) == r
    return r


@pytest.mark.parametrize("dt", [1, E4M3])
def test_evict_in_place_of_one_array_as_k_and_v(fm, past_the_checks, dt):  # noqa: F811
    """K's and V's thread blocks would move the same rows down, each at its own pace."""
    n = ROWS_IN * (128 if dt == E4M3 else 256)
    for vc in (EVICT["kc"], EVICT["kc"] + n - 16, EVICT["kc"] - n + 16):
        assert call_evict(fm, **in_place(vc=vc), dt=dt) == -1
    assert call_evict(fm, **in_place(vc=EVICT["kc"] + n), dt=dt) == past_the_checks      # next to one another


@pytest.mark.parametrize("x,y", [("ko", "vo"), ("ko", "ao"), ("vo", "ao"), ("ko", "kept"), ("vo", "kept"), ("ao", "kept"),
                                 ("ko", "ns"), ("vo", "ns"), ("ao", "ns"), ("kept", "ns")])
def test_evict_outputs_over_one_another(fm, past_the_checks, x, y):  # noqa: F811
    for a in clash(EVICT, x, y, EVICT_BYTES[x]):
        assert call_evict(fm, **a) == -1


@pytest.mark.parametrize("x,y", [(i, o) for i in ("kc", "vc", "acc") for o in ("kept", "ns")])
def test_evict_lists_over_the_input(fm, past_the_checks, x, y):  # noqa: F811
    for a in clash(EVICT, x, y, EVICT_BYTES[x]):
        assert call_evict(fm, **a) == -1
        assert call_evict(fm, **in_place(**{y: a[y]})) == -1


@pytest.mark.parametrize("x", ["ko", "vo", "ao", "kept"])
@pytest.mark.parametrize("y", ["sl", "bi", "oi"])
def test_evict_outputs_over_the_sequences(fm, past_the_checks, x, y):  # noqa: F811
    for a in clash(EVICT, x, y, EVICT_BYTES[x]):
        assert call_evict(fm, **a) == -1


@pytest.mark.parametrize("y", ["sl", "bi", "oi"])
def test_evict_new_lengths_over_the_sequences(fm, past_the_checks, y):  # noqa: F811
    for off in (-4, 0, 4):                               # int32 of two sequences: one element in common, or both
        assert call_evict(fm, **{**EVICT, "ns": EVICT[y] + off}) == -1
    for off in (-8, 8):
        assert call_evict(fm, **{**EVICT, "ns": EVICT[y] + off}) == past_the_checks


def test_evict_of_one_array_as_k_and_v_into_two_others(fm, past_the_checks):  # noqa: F811
    assert call_evict(fm, **{**EVICT, "vc": EVICT["kc"]}) == past_the_checks     # both only read it


# ---------------------------------------------------------------------------
# Weights: 2 sequences, 4 queries, 8 heads on 2, entries of 64 rows, bf16
# ---------------------------------------------------------------------------

WEIGHTS = apart("q", "kc", "lse", "ai", "ao", "sl", "bi", "nq", "ws")
WEIGHTS_BYTES = dict(q=2 * 4 * 8 * 256, kc=2 * 64 * 2 * 256, lse=2 * 8 * 4 * 4, ai=2 * 2 * 64 * 4, ao=2 * 2 * 64 * 4)


@pytest.fixture
def weights_past_the_checks(fm):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("a device would be given the fake addresses")
    r = call_weights(fm, **WEIGHTS)
    assert r != -1 and call_weights(fm, **{**WEIGHTS, "ai": WEIGHTS["ao"]}) == r
    return r


@pytest.mark.parametrize("x", ["q", "kc", "lse"])
def test_weights_scores_over_an_input(fm, weights_past_the_checks, x):  # noqa: F811
    """Blocks that are not done read the queries, keys and LSE that the first ones would overwrite."""
    for a in clash(WEIGHTS, x, "ao", WEIGHTS_BYTES[x]):
        assert call_weights(fm, **a) == -1
        assert call_weights(fm, **{**a, "ai": a["ao"]}) == -1
    assert call_weights(fm, **{**WEIGHTS, "ao": WEIGHTS[x] + WEIGHTS_BYTES[x]}) == weights_past_the_checks


@pytest.mark.parametrize("y", ["sl", "bi", "nq"])
def test_weights_scores_over_the_sequences(fm, weights_past_the_checks, y):  # noqa: F811
    for a in clash(WEIGHTS, "ao", y, WEIGHTS_BYTES["ao"]):
        assert call_weights(fm, **a) == -1


@pytest.mark.parametrize("x", ["q", "kc", "lse", "ai", "ao", "sl", "bi", "nq"])
def test_weights_scratch_over_an_array(fm, weights_past_the_checks, x):  # noqa: F811
    for off in (0, 256 - fm.fmha_cache_weights_workspace_size() // 256 * 256):
        assert call_weights(fm, **{**WEIGHTS, "ws": WEIGHTS[x] + off}) == -1


# ---------------------------------------------------------------------------
# Drafts: 2 sequences of 4, 8 heads on 2, entries of 64 rows, bf16
# ---------------------------------------------------------------------------

TREE = apart("q", "kc", "vc", "kn", "vn", "o", "lse", "sl", "bi", "nd", "mask", "ws")
TREE_BYTES = dict(q=2 * 4 * 8 * 256, o=2 * 4 * 8 * 256, kc=2 * 64 * 2 * 256, vc=2 * 64 * 2 * 256, kn=2 * 4 * 2 * 256,
                  vn=2 * 4 * 2 * 256, lse=2 * 8 * 4 * 4)


@pytest.fixture
def tree_past_the_checks(fm):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("a device would be given the fake addresses")
    r = call_tree(fm, **TREE)
    assert r != -1 and call_tree(fm, **{**TREE, "lse": None, "mask": None, "bi": None, "nd": None}) == r
    return r


@pytest.mark.parametrize("x", ["q", "kc", "vc", "kn", "vn", "o"])
def test_tree_lse_over_another_array(fm, tree_past_the_checks, x):  # noqa: F811
    for a in clash(TREE, x, "lse", TREE_BYTES[x]):
        assert call_tree(fm, **a) == -1
    assert call_tree(fm, **{**TREE, "lse": TREE[x] + TREE_BYTES[x]}) == tree_past_the_checks


@pytest.mark.parametrize("x", ["o", "lse"])
@pytest.mark.parametrize("y", ["sl", "bi", "nd"])
def test_tree_outputs_over_the_sequences(fm, tree_past_the_checks, x, y):  # noqa: F811
    for a in clash(TREE, x, y, TREE_BYTES[x]):
        assert call_tree(fm, **a) == -1


@pytest.mark.parametrize("x", ["o", "lse"])
def test_tree_outputs_over_the_mask(fm, tree_past_the_checks, x):  # noqa: F811
    """One mask of 4 x 4 bytes, or one for each of the two sequences, 100 bytes apart."""
    end = TREE[x] + TREE_BYTES[x]
    for ms in (0, 100):
        assert call_tree(fm, **{**TREE, "mask": TREE[x] - 15, "ms": ms}) == -1
        assert call_tree(fm, **{**TREE, "mask": TREE[x] - 100 - 15, "ms": ms}) == (-1 if ms else tree_past_the_checks)
        assert call_tree(fm, **{**TREE, "mask": end - 1, "ms": ms}) == -1
        assert call_tree(fm, **{**TREE, "mask": end, "ms": ms}) == tree_past_the_checks


@pytest.mark.parametrize("x", ["q", "kc", "vc", "kn", "vn", "o", "lse", "sl", "bi", "nd", "mask"])
def test_tree_scratch_over_an_array(fm, tree_past_the_checks, x):  # noqa: F811
    assert call_tree(fm, **{**TREE, "ws": TREE[x], "ws_bytes": 1 << 40}) == -1
    last = 256 - fm.fmha_tree_workspace_size(2, 4, 8, 2, 128, 64) // 256 * 256
    assert call_tree(fm, **{**TREE, "ws": TREE[x] + last}) == -1


# ---------------------------------------------------------------------------
# Commit: 2 sequences of 4 drafts, 3 accepted at most, 2 heads, entries of 64 rows, bf16
# ---------------------------------------------------------------------------

COMMIT = apart("kc", "vc", "kn", "vn", "sl", "bi", "path", "na")


@pytest.mark.parametrize("x", ["kc", "vc"])
@pytest.mark.parametrize("y", ["sl", "bi", "path", "na"])
def test_commit_cache_over_the_sequences(fm, x, y):  # noqa: F811
    """A thread block a draft: each reads its sequence's length, entry and path while others write rows."""
    if torch.cuda.is_available():
        pytest.skip("a device would be given the fake addresses")
    r = call_commit(fm, **COMMIT)
    assert r != -1 and call_commit(fm, **{**COMMIT, "bi": None}) == r
    for a in clash(COMMIT, x, y, 2 * 64 * 2 * 256):
        assert call_commit(fm, **a) == -1
    assert call_commit(fm, **{**COMMIT, y: COMMIT[x] + 2 * 64 * 2 * 256}) == r
