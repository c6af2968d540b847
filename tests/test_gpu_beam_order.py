"""pa_beam_select where ranks are equal or all but equal (needs a GPU): the lower beam comes first,
whatever the lengths the equal ranks come from."""
import numpy as np
import pytest
import torch

from cache_util import dev, host
from paged_fp8_kv_04_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _ended(scores, lengths, penalty):
    """Parents and tokens of requests all of whose beams have ended (end token 1 of three)."""
    N, W = scores.shape
    got = B.beam_select(torch.zeros(N, W, 3, device="cuda"), dev(scores.astype(np.float32)), eos=1,
                        finished=torch.ones(N, W, dtype=torch.uint8, device="cuda"),
                        lengths=dev(lengths.astype(np.int32)), length_penalty=penalty)
    return host(got[1]), host(got[0])


# ------------------------------------------------------------- beams of different lengths

def test_equal_ranks_of_two_lengths_go_to_the_lower_beam():
    """Scores and lengths of ended beams are exact, and so is -n / n: all these ranks are -1."""
    n = np.array([(a, b) for a in range(1, 100) for b in range(1, 100)])
    parents, tokens = _ended(-n, n, 1.0)
    assert np.array_equal(parents, np.tile([0, 1], (len(n), 1))) and (tokens == 1).all()


@pytest.mark.parametrize("W", [2, 5, 16, 32])
def test_equal_and_unequal_ranks_of_many_lengths(W):
    """Ranks -1, -1/2, ..., -1/64 (powers of two: the quotients are exact), several beams at each."""
    rng = np.random.default_rng(W)
    n = rng.integers(1, 2000, size=(300, W))
    level = rng.integers(0, 7, size=(300, W))
    n[:100], level[:100] = n[:100, :1], level[:100, :1]       # one length, one rank
    parents, _ = _ended(-n / 2.0 ** level, n, 1.0)
    assert np.array_equal(parents, np.argsort(-level, axis=1, kind="stable"))


@pytest.mark.parametrize("penalty", [0.25, 0.6, 1.0, 1.7, 2.0])
def test_ranks_within_the_tables_error(penalty):
    """The order is that of total / length ** penalty in fp64 down to its own roundings: the power is off by
    two units and the quotient by half of one here and in numpy (2^-52 each unit), 5 * 2^-52 together."""
    rng = np.random.default_rng(21)
    N = 60000
    n = rng.integers(1, 600, size=(N, 2))
    p = float(np.float32(penalty))
    t1 = (-1 - 40 * rng.random(N)).astype(np.float32)
    t2 = (t1 * (n[:, 1] / n[:, 0]) ** p).astype(np.float32)
    rank = np.stack([t1 / n[:, 0].astype(np.float64) ** p, t2 / n[:, 1].astype(np.float64) ** p], 1)
    gap = (rank[:, 0] - rank[:, 1]) / np.abs(rank[:, 0])
    clear = np.abs(gap) > 5 * 2.0 ** -52
    assert (clear & (np.abs(gap) < 1e-9)).sum() > 100
    parents, _ = _ended(np.stack([t1, t2], 1), n, penalty)
    assert np.array_equal((parents[:, 0] == 0)[clear], (gap > 0)[clear])


def test_ended_and_live_beams_of_equal_rank():
    """A live beam with one token to choose keeps its score: total = score + (x - x)."""
    n = np.array([(a, b) for a in range(1, 40) for b in range(1, 40)])
    N = len(n)
    for ended in (0, 1):
        fin = np.zeros((N, 2), np.uint8)
        fin[:, ended] = 1
        ln = n - (1 - fin)                                    # a live beam's length grows by one
        got = B.beam_select(torch.full((N, 2, 1), 3.25, device="cuda"), dev(-n.astype(np.float32)), eos=0, finished=dev(fin),
                            lengths=dev(ln.astype(np.int32)), length_penalty=1.0)
        assert np.array_equal(host(got[4]), n) and np.array_equal(host(got[1]), np.tile([0, 1], (N, 1))), ended


@pytest.mark.parametrize("penalty", [200.0, 1e4, 1e30])
def test_powers_near_and_beyond_the_largest_double(penalty):
    """Where length ** penalty is no finite double every rank is -0, and all are equal."""
    rng = np.random.default_rng(5)
    n = rng.integers(2, 4000, size=(200, 6))
    s = -rng.random((200, 6)).astype(np.float32) - 1
    with np.errstate(over="ignore"):
        rank = s.astype(np.float64) / n.astype(np.float64) ** float(np.float32(penalty)) + 0.0
    parents, _ = _ended(s, n, penalty)
    assert np.array_equal(parents, np.argsort(-rank, axis=1, kind="stable"))
