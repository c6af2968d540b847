"""pa_beam_select where ranks are equal or all but equal (needs a GPU): the lower beam comes first, then the
lower token, whatever the lengths and logits the equal ranks come from."""
import numpy as np
import pytest
import torch

from cache_util import dev, host
from oracle import cache_ops as C
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


# ------------------------------------------------------------ equal totals within a beam

def _same_as_definition(x, scores, lengths=None, penalty=0.0):
    got = B.beam_select(x, dev(scores), lengths=None if lengths is None else dev(lengths), length_penalty=penalty)
    want = C.beam_select(x.double().cpu().numpy(), scores, -1, None, lengths, penalty)
    assert np.array_equal(host(got[0]), want[0]) and np.array_equal(host(got[1]), want[1])
    # one rounding to fp32, and a log-sum-exp of some hundred thousand exponentials off by 2^-22 each
    assert np.allclose(host(got[2]).astype(np.float64), want[2], rtol=2.0 ** -23, atol=2.0 ** -18)
    if lengths is not None:
        assert np.array_equal(host(got[4]), want[4])


def test_a_score_that_swallows_the_logits():
    lowest = torch.finfo(torch.float32).min
    x = torch.tensor([[[0.0, 1.0, 2.0]] * 3], device="cuda")
    tokens, parents, _, _, _ = B.beam_select(x, torch.full((1, 3), lowest, device="cuda"))
    assert host(tokens).tolist() == [[0, 1, 2]] and host(parents).tolist() == [[0, 0, 0]]
    tokens, parents, _, _, _ = B.beam_select(x, torch.tensor([[lowest, lowest, -1.0]], device="cuda"))
    assert host(tokens).tolist() == [[2, 1, 0]] and host(parents).tolist() == [[2, 2, 2]]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [1, 3, 8, 32])
@pytest.mark.parametrize("V", [2, 7, 31, 300, 70001])
def test_beams_that_hardly_exist(dt, W, V):
    """The type's lowest value as the score of a beam that does not exist yet: all its tokens are equal."""
    rng = np.random.default_rng(V + W)
    lowest = np.finfo(np.float32).min
    scores = np.full((3, W), lowest, np.float32)
    scores[1, 0] = scores[2, W - 1] = -1.5                   # a first step
    big = torch.from_numpy(3 * rng.standard_normal((3, W, V + 3)).astype(np.float32)).to(dt).cuda()
    big[0, :, :] = big[0].sort(-1).values                    # the lowest tokens have the lowest logits
    for lo in (0, 1, 3):                                     # rows that begin at any alignment
        _same_as_definition(big[..., lo:lo + V], scores)


@pytest.mark.parametrize("dt,score,unit,base", [(torch.float32, -1e12, 2.0 ** -16, 200.0), (torch.bfloat16, -2.0 ** 60, 8.0, 1280.0)])
@pytest.mark.parametrize("W", [1, 4, 17, 32])
@pytest.mark.parametrize("V,cells", [(50, 2), (3000, 100), (40000, 3), (40000, 1000), (140001, 64)])
def test_totals_that_round_together(dt, score, unit, base, W, V, cells):
    """Logits within a rounding cell of the total: fp64 numbers of the score's size lie 8 (fp32) or 32 (bf16) units
    apart, the logits at most 3 or 12 units from a multiple of that, so that the last bits of the
    log-sum-exp decide nothing.  One token has logit 0 and all others e^-200 of its weight or less: its log is 0."""
    rng = np.random.default_rng(V + W)
    cell = 8 if dt == torch.float32 else 32
    cells = cells if dt == torch.float32 else min(cells, 3)
    at = cell * rng.integers(0, cells, size=(2, W, V)) + rng.integers(-(3 * cell // 8), 3 * cell // 8 + 1, size=(2, W, V))
    x = torch.from_numpy(-(base + unit * at)).to(dt)
    assert np.array_equal(x.double().numpy(), -(base + unit * at))
    x.scatter_(2, torch.from_numpy(rng.integers(0, V, size=(2, W, 1))), 0.0)
    scores = np.full((2, W), score, np.float32)
    scores[1, ::2] = 2 * score                               # whose cells are twice as wide
    scores[1, 0] = score
    x = x.cuda()
    _same_as_definition(x, scores)
    _same_as_definition(x, scores, np.full((2, W), 2, np.int32), 1.0)  # quotients by 3 round together what totals do not


@pytest.mark.parametrize("dt,cell", [(torch.float32, 2.0 ** -16), (torch.bfloat16, 2.0 ** -15)])
def test_scores_of_the_lower_tokens_of_equal_rank(dt, cell):
    """Totals just past the middle of two fp32 numbers: -2^40 - 2^16 + x (fp32) or -2^44 - 2^20 + x (bf16), x some 2^-9 or
    2^-7 below 0, where fp64 numbers lie 2^-12 or 2^-8 apart and the logits closer.  A score taken without its
    token's logit rounds to the beam's."""
    x = torch.full((1, 3, 70), -1e6)
    x[..., 40] = 65536.0
    base = 8 * 2.0 ** -12 if dt == torch.float32 else 8 * 2.0 ** -10
    x[..., 10:17] = -base + cell * torch.arange(-3, 4)         # rising: the highest logit is the highest token's
    x = x.to(dt).cuda()
    assert len(x[0, 0, 10:17].unique()) >= (7 if dt == torch.float32 else 3)
    score = np.full((1, 3), -2.0 ** 40 if dt == torch.float32 else -2.0 ** 44, np.float32)
    if dt == torch.bfloat16:
        x[..., 40] = 2.0 ** 20
    got = B.beam_select(x, dev(score))
    want = C.beam_select(x.double().cpu().numpy(), score)
    assert host(got[1]).tolist() == want[1].tolist() == [[0, 1, 2]] and host(got[0]).tolist() == want[0].tolist() == [[40, 40, 40]]
    score[:, 1:] = -np.inf
    got = B.beam_select(x, dev(score))
    want = C.beam_select(x.double().cpu().numpy(), score)
    assert np.array_equal(host(got[0]), want[0]) and want[0].tolist() == [[40, 10, 11]]
    assert np.array_equal(host(got[2]), want[2].astype(np.float32))
    assert host(got[2])[0, 1] < score[0, 0]                       # and not the score itself


@pytest.mark.parametrize("penalty", [0.0, 1.0])
def test_quotients_of_two_beams_that_round_together(penalty):
    """Second tokens of two beams of one length, with totals up to three fp64 steps (2^-13 at 10^12) apart: where their
    quotients are one number the lower beam comes first, and else the larger total's."""
    rng = np.random.default_rng(31)
    n = 4000
    x = torch.zeros(n, 3, 2)
    x[..., 1] = torch.from_numpy(-(200 + 2.0 ** -13 * rng.integers(0, 4, size=(n, 3)))).float()
    score = np.tile(np.array([-1e12, -1e12, -np.inf], np.float32), (n, 1))
    lengths = rng.integers(2, 40, size=(n, 1)).repeat(3, 1).astype(np.int32)
    got = B.beam_select(x.cuda(), dev(score), lengths=dev(lengths), length_penalty=penalty)
    want = C.beam_select(x.double().numpy(), score, -1, None, lengths, penalty)
    assert np.array_equal(host(got[0]), want[0]) and np.array_equal(host(got[1]), want[1])
    equal = x[:, 0, 1] < x[:, 1, 1]                                # the larger total is beam 1's
    assert (host(got[1])[:, 2][equal.numpy()] == 0).any() == (penalty == 1.0)


def test_more_tokens_of_the_lowest_logit_of_a_rank_than_the_list_holds():
    """-2^40 - 200 - 2^-13 lies in the middle of two fp64 numbers and rounds to -2^40 - 200, which is even: the
    lowest logit of that rank is -200 - 2^-13, of which the three best by logit hold one token of two."""
    x = torch.full((1, 3, 40), -1e6)
    x[..., 30], x[..., 33], x[..., 10], x[..., 20] = 0.0, -200.0, -200.0 - 2.0 ** -13, -200.0 - 2.0 ** -13
    score = np.array([[-2.0 ** 40, -np.inf, -np.inf]], np.float32)
    got, want = B.beam_select(x.cuda(), dev(score)), C.beam_select(x.double().numpy(), score)
    assert host(got[0]).tolist() == want[0].tolist() == [[30, 10, 20]] and (host(got[1]) == 0).all()


# --------------------------------------------------------------- the log-sum-exp in totals

@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,scale", [(3000, 1.0), (32001, 1.2), (131072, 1.5), (2000000, 1.5)])
def test_log_sum_exps_are_close_to_fp64(dt, V, scale):
    """A live beam's best total is set 2^-21 above or below an ended beam's score (through a live score of some 1e-6, in
    whose fp32 steps nothing is lost), and comes out on that side.  An exponential is off by 2^-22 of itself
    at most, at worst all in one direction; the roundings of its argument, of products and of partial sums, 2^-19 of it
    together, differ from term to term, and the sum is spread over 64 terms or more, which leaves an eighth of
    them: 2^-22 and 2^-22."""
    rng = np.random.default_rng(V)
    N = 24
    x = torch.from_numpy((scale * rng.standard_normal((N, V))).astype(np.float32)).to(dt)
    xd = x.double().numpy()
    top = xd.max(1)
    e = np.exp(xd - top[:, None])
    best = -np.log(e.sum(1))
    assert (e.sum(1) ** 2 / (e ** 2).sum(1)).min() > 64
    ended = best.astype(np.float32)
    live = x.cuda()[:, None].repeat(1, 2, 1)
    fin = torch.tensor([0, 1], dtype=torch.uint8, device="cuda").repeat(N, 1)
    for side in (1, -1):
        score = (ended - best + side * 1.01 * 2.0 ** -21).astype(np.float32)
        gap = score.astype(np.float64) + best - ended
        assert (side * gap > 2.0 ** -21).all() and np.abs(gap).max() < 2.0 ** -20
        got = B.beam_select(live, dev(np.stack([score, ended], 1)), eos=0, finished=fin)
        assert (host(got[1])[:, 0] == (0 if side > 0 else 1)).all()
