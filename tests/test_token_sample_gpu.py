"""GPU parity of token_sample with the oracle: tokens and status bits equal, the kept tokens (the
probabilities that are not 0) equal, each probability w / S within three roundings of fp32 (S,
its reciprocal's product with a power of two, and the product with w): 3 * 2^-24 of its value."""
import numpy as np
import pytest

from oracle import token_sample as TS

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_indexer_gb300 import sample_tokens, token_probs, verify_drafts  # noqa: E402

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def dev(a, dtype=torch.float32):
    return None if a is None else torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def check(logits, u, param_rows=1, rows=None, status=None, **settings):
    """logits a CUDA tensor [rows, vocab] (any strides of rows), settings lists."""
    args = {k: dev(v, torch.int32 if k == "top_k" else torch.float32) for k, v in settings.items()}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens, probs = sample_tokens(logits, dev(u), with_probs=True, status=st, param_rows=param_rows, **args)
    alone, none = sample_tokens(logits, dev(u), param_rows=param_rows, **args)
    only = token_probs(logits, param_rows=param_rows, **args)
    assert none is None and torch.equal(tokens, alone)
    assert torch.equal(probs, only) or torch.isnan(probs).any()
    tokens, probs = tokens.tolist(), probs.double().cpu().numpy()
    x = logits.float().cpu().numpy()
    want = 0
    for r in range(len(x)):
        mine = {k: v[r // param_rows] for k, v in settings.items()}
        if rows is not None and r not in rows:
            continue
        token, w, s = TS.row(x[r], u[r], **mine)
        want |= s
        assert tokens[r] == token, (r, mine)
        total = sum(w)
        p = np.array([a / total if total else 0.0 for a in w])
        assert ((probs[r] > 0) == (p > 0)).all(), (r, mine)
        assert (np.abs(probs[r] - p) <= 3 * 2.0 ** -24 * p).all(), (r, mine)
    if rows is None:
        assert int(st.item()) == (want if status is None else status)
    return tokens


def logits_of(rng, rows, vocab, dtype="fp32", spread=2.5, pad=0):
    x = torch.from_numpy((rng.standard_normal((rows, vocab + pad)) * spread).astype(np.float32))
    return x.to(TYPES[dtype]).cuda()[:, :vocab]


SETTINGS = [dict(), dict(top_k=1), dict(top_k=5), dict(top_p=0.9), dict(top_p=0.3), dict(min_p=0.05),
            dict(top_k=40, top_p=0.95), dict(top_k=300, top_p=0.6, min_p=0.01), dict(temperature=0.0),
            dict(temperature=0.5, top_p=0.99), dict(temperature=3.0, top_k=7, min_p=0.3)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 31, 33, 255, 1000, 1031, 4099])
def test_vocabularies(vocab, dtype):
    rng = np.random.default_rng(vocab)
    n = len(SETTINGS)
    full = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    s = {k: [x.get(k, full[k]) for x in SETTINGS] for k in full}
    check(logits_of(rng, n, vocab, dtype), rng.random(n).astype(np.float32).tolist(), **s)


@pytest.mark.parametrize("dtype,vocab", [("fp32", 20011), ("bf16", 33000), ("fp16", 50000)])
def test_large_vocabularies(dtype, vocab):
    rng = np.random.default_rng(vocab)
    n = 6
    check(logits_of(rng, n, vocab, dtype, 1.5), rng.random(n).astype(np.float32).tolist(),
          top_p=[0.95, 0.5, 0.999, 1.0, 0.95, 0.1], top_k=[0, 3000, 15000, 0, 50, 2049],
          temperature=[1.0, 0.7, 1.3, 1.0, 0.2, 5.0])


def test_many_rows():
    rng = np.random.default_rng(1)
    n = 600
    check(logits_of(rng, n, 501, "bf16"), rng.random(n).astype(np.float32).tolist(), rows=range(0, n, 29),
          top_p=rng.uniform(0.1, 1, n).astype(np.float32).tolist(), top_k=rng.integers(0, 60, n).tolist())


def test_a_row_too_long_to_keep():
    """More logits than the shared memory of a cluster holds: read from memory at every pass."""
    rng = np.random.default_rng(2)
    check(logits_of(rng, 1, 500001), [0.37], top_k=[50], top_p=[0.9])
    check(logits_of(rng, 1, 500001), [0.37], top_p=[0.999], temperature=[4.0])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_ties(dtype):
    """Equal logits are kept from the lowest index on: whole rows of them, and two values."""
    for vocab in (100, 3000, 9001):
        x = torch.zeros((6, vocab), dtype=TYPES[dtype], device="cuda")
        x[3:, ::3] = 1.0
        x[5, 1::3] = -0.0
        u = [0.0, 0.5, 0.9999, 0.2, 0.7, 0.999]
        check(x, u, top_k=[5, 17, vocab - 1, 20, vocab // 2, 0], top_p=[1.0, 0.5, 1.0, 0.9, 0.99, 0.6])


def test_borders_of_the_weights():
    """Logits whose z lies at whole numbers, at 16, 32 and around 40 and 41."""
    log2 = float(np.log(2))
    z = np.array([0, 0, 1, 15.999, 16, 16.001, 31.99, 32, 32.01, 39.99, 40, 40.0001, 40.5, 40.99, 41, 41.01, 60, 1e9])
    x = torch.from_numpy((-z * log2).astype(np.float32)).cuda()[None].repeat(8, 1).contiguous()
    check(x, [0.0, 0.3, 0.49, 0.51, 0.7, 0.99, 0.9999, 0.99999994],
          top_k=[0, 1, 2, 9, 11, 13, 15, 18], top_p=[1.0, 1.0, 0.9999999, 1.0, 1.0, 0.99999994, 1.0, 1.0])


def test_uniforms_at_the_ends():
    rng = np.random.default_rng(3)
    x = logits_of(rng, 4, 700)
    check(x, [0.0, 2.0 ** -149, float(np.nextafter(np.float32(1), np.float32(0))), 2.0 ** -24], top_p=[0.8] * 4)


def test_infinities_and_nan():
    rng = np.random.default_rng(4)
    x = logits_of(rng, 6, 300)
    x[0] = -np.inf
    x[1, 5:] = -np.inf
    x[2, 7] = np.inf
    x[3, 9] = x[3, 200] = np.inf
    x[4, 100:] = float("nan")
    x[5] = float("nan")
    u = rng.random(6).astype(np.float32).tolist()
    check(x, u)
    check(x, u, top_k=[3] * 6, top_p=[0.7] * 6)
    check(x, u, temperature=[0.0] * 6)
    check(x * 1e37, u, temperature=[1e-30, 1e30, 1.0, 1.0, 1.0, 1.0], top_p=[0.5] * 6)


def test_settings_out_of_range():
    rng = np.random.default_rng(5)
    nan, inf = float("nan"), float("inf")
    x = logits_of(rng, 9, 200)
    u = rng.random(9).astype(np.float32).tolist()
    check(x, u, temperature=[nan, -1.0, inf, 1.0, 1.0, 1.0, 1.0, 1e-45, 3e38],
          top_p=[0.5, 1.0, 1.0, nan, -1.0, 0.0, inf, 1.0, 1.0], min_p=[0, 0, 0, 0, 0, nan, 1.5, 1.0, -1.0],
          top_k=[0, -5, 200, 201, 1 << 30, 0, 0, 0, 0])
    check(x[:3], [-0.5, 1.0, nan], status=TS.UNIFORM)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_strides_shared_settings_and_canaries(dtype):
    """Rows that start off 16-byte boundaries, settings for every three rows, an output whose rows
    are strided: what lies between them stays."""
    rng = np.random.default_rng(6)
    x = logits_of(rng, 7, 777, dtype, pad=6)
    u = rng.random(7).astype(np.float32).tolist()
    check(x, u, param_rows=3, top_k=[5, 0, 50], top_p=[1.0, 0.9, 0.5], temperature=[1.0, 0.0, 2.0])
    out = torch.full((7, 800), -7.0, device="cuda")
    token_probs(x, top_p=dev([0.9] * 7), out=out[:, 3:780])
    assert (out[:, :3] == -7).all() and (out[:, 780:] == -7).all()
    assert torch.equal(out[:, 3:780], token_probs(x, top_p=dev([0.9] * 7)))


def test_nothing_and_refusals():
    x = torch.zeros((0, 50), device="cuda")
    tokens, probs = sample_tokens(x, torch.zeros(0, device="cuda"), with_probs=True)
    assert tokens.shape == (0,) and probs.shape == (0, 50)
    x = torch.zeros((3, 50), device="cuda")
    u = torch.zeros(3, device="cuda")
    for bad in (dict(logits=x.double()), dict(logits=x[0]), dict(uniforms=u[:2]), dict(uniforms=u.double()),
                dict(temperature=u[:2]), dict(top_k=u), dict(top_p=u.half()), dict(param_rows=0),
                dict(logits=x.t()), dict(min_p=u.cpu())):
        with pytest.raises(ValueError):
            sample_tokens(**{**dict(logits=x, uniforms=u), **bad})
    with pytest.raises(ValueError):
        token_probs(x, out=torch.zeros((3, 51), device="cuda"))


def test_runs_streams_and_graphs_agree():
    rng = np.random.default_rng(7)
    x = logits_of(rng, 9, 30000)
    u, k, p = dev(rng.random(9)), dev([50] * 9, torch.int32), dev([0.95] * 9)
    ref = sample_tokens(x, u, top_k=k, top_p=p, with_probs=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sample_tokens(x, u, top_k=k, top_p=p, with_probs=True, stream=s)
    s.synchronize()
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sample_tokens(x, u, top_k=k, top_p=p, with_probs=True)
    for _ in range(5):
        got[1].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


def test_drafts_that_verify():
    """sample_tokens draws drafts, token_probs gives both sides' probabilities, verify_drafts takes
    them: with the same logits on both sides every draft stands."""
    rng = np.random.default_rng(8)
    reqs, drafts, vocab = 5, 3, 1000
    x = logits_of(rng, reqs * (drafts + 1), vocab)
    settings = dict(top_k=dev([20] * reqs, torch.int32), top_p=dev([0.9] * reqs), param_rows=drafts + 1)
    target = token_probs(x, **settings).view(reqs, drafts + 1, vocab)
    mine = x.view(reqs, drafts + 1, vocab)[:, :drafts].reshape(-1, vocab)
    settings["param_rows"] = drafts
    tokens, q = sample_tokens(mine, dev(rng.random(reqs * drafts)), with_probs=True, **settings)
    out, kept = verify_drafts(target, q.view(reqs, drafts, vocab), tokens.view(reqs, drafts),
                              dev(rng.random((reqs, drafts + 1))))
    assert (kept == drafts).all()
    assert torch.equal(out[:, :drafts], tokens.view(reqs, drafts))
    last = target[torch.arange(reqs), drafts].gather(1, out[:, drafts:].long())
    assert (last > 0).all()
