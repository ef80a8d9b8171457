"""GPU parity of the drafts' verification (draft_verify) with the oracle in integers and
fractions: tokens, counts and status bits, equal."""
import numpy as np
import pytest

from oracle import draft_verify as DV

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_indexer_gb300 import verify_drafts  # noqa: E402


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def make(seed, reqs, drafts, vocab, point=False, near=0.5):
    rng = np.random.default_rng(seed)
    z = 2.0 * rng.standard_normal((reqs, drafts + 1, vocab))
    p = softmax(z)
    q = softmax(z[:, :drafts] + near * rng.standard_normal((reqs, drafts, vocab)))
    tok = np.zeros((reqs, drafts), np.int32)
    for j in range(reqs):
        for i in range(drafts):
            w = q[j, i].astype(np.float64)
            tok[j, i] = np.argmax(w) if point else rng.choice(vocab, p=w / w.sum())
    return p, None if point else q, tok, rng.random((reqs, drafts + 1)).astype(np.float32)


def check(p, q, tok, u, n_drafts=None, strided=False):
    t = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    ro, rk, rs = DV.verify(p, q, tok, u, n_drafts)
    P, Q = t(p), t(q)
    if strided:  # rows at an odd stride inside a wider buffer
        def wide(x):
            b = torch.full((x.shape[0], x.shape[1], x.shape[2] + 3), 7.0, device="cuda")
            b[..., :x.shape[2]] = x
            return b[..., :x.shape[2]]
        P, Q = wide(P), None if Q is None else wide(Q)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    nd = None if n_drafts is None else t(np.asarray(n_drafts, np.int32))
    out, kept = verify_drafts(P, Q, t(tok), t(u), nd, st)
    torch.cuda.synchronize()
    assert np.array_equal(kept.cpu().numpy(), rk)
    assert np.array_equal(out.cpu().numpy(), ro)
    assert int(st.item()) == rs
    return ro, rk, rs


@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("reqs,drafts,vocab", [
    (1, 6, 5000), (1, 1, 1), (3, 2, 2), (2, 0, 100), (5, 31, 33), (40, 3, 31), (1, 7, 40001),
    (2, 3, 9999), (300, 2, 257), (7, 4, 12288)])
def test_sizes(reqs, drafts, vocab, point):
    check(*make(reqs * 100 + drafts, reqs, drafts, vocab, point))


@pytest.mark.parametrize("strided", [False, True])
def test_strides(strided):
    check(*make(3, 6, 3, 4097), strided=strided)


def test_ragged_draft_counts():
    p, q, tok, u = make(4, 8, 5, 700)
    check(p, q, tok, u, [0, 1, 2, 3, 4, 5, 5, 2])
    assert check(p, q, tok, u, [0, 6, -1, 3, 4, 5, 5, 2])[2] == DV.COUNT


@pytest.mark.parametrize("seed", range(4))
def test_draws_over_the_whole_row(seed):
    """Uniforms next to 0 and 1, and a few between; every request refuses its draft."""
    p, q, tok, u = make(20 + seed, 16, 1, 6007, near=3.0)
    u[:, 0] = np.float32(1 - 2.0 ** -24)
    u[:, 1] = np.linspace(0, 1, 16, endpoint=False)
    u[0, 1], u[15, 1] = 0.0, np.float32(1 - 2.0 ** -24)
    u[1, 1] = np.float32(2.0 ** -40)
    check(p, q, tok, u)


def above(x):
    """The least float32 that is not below x."""
    f = np.float32(x)
    return f if f >= x else np.nextafter(f, np.float32(np.inf))


@pytest.mark.parametrize("ones", [0, 9])
def test_uniforms_with_bits_below_2_to_the_64th(ones):
    """Tokens of 2^-60 each before those that have the rest: the drawn token is floor(r * sum),
    for the least r at which it is a given one, whose last bits lie below 2^-64."""
    rng = np.random.default_rng(ones)
    want = np.unique(np.concatenate([2 ** np.arange(13), rng.integers(1, 5900, 50)]))
    vocab, reqs = 6000, len(want) + 2
    p = np.full((reqs, 1, vocab), 2.0 ** -60, np.float32)
    p[:, 0, -1] = rng.uniform(0.5, 1, reqs)
    p[:, 0, vocab - 1 - ones:vocab - 1] = 0.75
    total = p[:, 0].astype(np.float64).sum(-1)
    u = np.zeros((reqs, 1), np.float32)
    u[:-2, 0] = [above(k * 2.0 ** -60 / t) for k, t in zip(want, total)]
    u[-2], u[-1] = 2.0 ** -149, 2.0 ** -62
    o, k, s = check(p, None, np.zeros((reqs, 0), np.int32), u)
    assert s == 0 and o[:-2, 0].tolist() == want.tolist()


def test_ties_of_the_test_and_of_the_draw():
    """u q equal to p refuses; a running sum equal to the point does not stop the draw."""
    p = np.full((4, 2, 8), 0.125, np.float32)
    q = np.full((4, 1, 8), 0.25, np.float32)
    tok = np.array([[3]] * 4, np.int32)
    u = np.array([[0.5, 0.5], [0.4999, 0.25], [0.5, 0.0], [0.25, 0.875]], np.float32)
    o, k, s = check(p, q, tok, u)
    assert k.tolist() == [0, 1, 0, 1]
    assert o[1].tolist() == [3, 2] and o[3].tolist() == [3, 7]


def test_zero_rows_and_points():
    p = np.zeros((5, 2, 300), np.float32)
    q = np.zeros((5, 1, 300), np.float32)
    p[0, 1, 299] = 1.0
    p[0, 0, 5], q[0, 0, 5] = 1.0, 1.0       # stands; the bonus row is one token
    p[1, 0, 7], q[1, 0, 7] = 0.5, 1.0       # nothing left of p - q: drawn from p
    p[2, 0, 9] = 1.0                        # the drafted token has no probability
    p[3, 0, 0], q[3, 0, 1] = 1.0, 1.0
    tok = np.array([[5], [7], [3], [1], [0]], np.int32)  # request 4: rows of zeros
    u = np.full((5, 2), 0.75, np.float32)
    o, k, s = check(p, q, tok, u)
    assert s == DV.EMPTY and o[4].tolist() == [-1, -1] and o[0].tolist() == [5, 299]


def test_values_outside_their_range():
    p, q, tok, u = make(6, 6, 2, 500, near=3.0)
    u[:, :2] = 0.999
    p[0, :, 3] = np.nan
    q[1, 0, 4] = -0.5
    p[2, :, 5] = 1.5
    assert check(p, q, tok, u)[2] == DV.PROB
    p, q, tok, u = make(7, 5, 2, 500)
    tok[0, 0], tok[1, 1] = 500, -1
    check(p, q, tok, u)  # the status bits too are compared inside
    p, q, tok, u = make(8, 4, 1, 60)
    u[0, 1], u[1, 0], u[2, 1], u[3, 0] = 1.0, np.nan, -0.25, 2.0
    assert check(p, q, tok, u)[2] == DV.UNIFORM


def test_rows_that_sum_to_more_than_eight():
    p = np.full((1, 1, 12), 1.0, np.float32)
    assert check(p, None, np.zeros((1, 0), np.int32), np.array([[0.5]], np.float32))[2] == DV.PROB


def test_rows_that_would_wrap_the_sums():
    p = np.full((2, 1, 4000), 1.0, np.float32)
    p[1] = 1.0 / 4096
    o, k, s = check(p, None, np.zeros((2, 0), np.int32), np.array([[0.5], [0.5]], np.float32))
    assert s == DV.PROB and o[0, 0] == -1 and o[1, 0] == 2000


@pytest.mark.parametrize("vocab", [300, 70000])
def test_rows_that_sum_to_fifteen(vocab):
    """No token from a sum of 15, wherever the tokens lie; one from the least sum below."""
    rng = np.random.default_rng(vocab)
    w = [1.0] * 14 + [2.0 ** -i for i in range(1, 29)]
    p = np.zeros((24, 1, vocab), np.float32)
    for j in range(24):
        at = rng.permutation(vocab)[:len(w) + 2]
        p[j, 0, at] = w + ([2.0 ** -29, 2.0 ** -29] if j < 12 else [2.0 ** -29, 2.0 ** -30])
    u = rng.random((24, 1)).astype(np.float32)
    o, k, s = check(p, None, np.zeros((24, 0), np.int32), u)
    assert (o[:12] == -1).all() and (o[12:] >= 0).all() and s == DV.PROB


@pytest.mark.parametrize("vocab", [255, 256, 257, 4095, 16384, 32768, 32769, 65537, 1100000])
def test_slices_and_steps(vocab):
    """One token's weight at a step's, a slice's and the row's ends."""
    at = sorted({0, vocab - 1, vocab // 2, *[x for s in (256, 2048, 16384, 131072)
                                             for x in (s - 1, s, s + 1) if x < vocab]})
    p = np.zeros((len(at), 1, vocab), np.float32)
    for j, x in enumerate(at):
        p[j, 0, x] = 0.75
        p[j, 0, 0] += 0.25
    u = np.tile(np.array([[0.25], [0.2499]], np.float32), (len(at), 1))[:len(at)]
    t = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    out, kept = verify_drafts(t(p), None, t(np.zeros((len(at), 0), np.int32)), t(u))
    want = [0 if u[j, 0] < 0.25 or x == 0 else x for j, x in enumerate(at)]
    assert out[:, 0].tolist() == want and kept.tolist() == [0] * len(at)


def test_every_run_and_a_graph_agree():
    p, q, tok, u = make(9, 4, 6, 20000)
    t = [torch.from_numpy(x).cuda() for x in (p, q, tok, u)]
    ref = verify_drafts(*t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out, kept = verify_drafts(*t)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(kept, ref[1])
