"""token_sample of batches: from about 19 rows on it runs CTAs of 256 threads, up to eight to a row,
where a row alone runs 512. Some rows are compared with the oracle as in tests/test_token_sample_gpu.py;
all of them are equal bit for bit to the same row sampled alone (the results do not depend on the
split)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from sparse_attention_indexer_gb300 import sample_tokens, token_probs  # noqa: E402
from tests.test_token_sample_gpu import TYPES, check, dev, logits_of  # noqa: E402

N = 40  # more than SMs / 8 rows


def settings_of(rng, n, vocab):
    """Rows with each setting off and on; top-k lists below and above 256 and 2048 tokens."""
    f = lambda x: [float(np.float32(y)) for y in x]  # noqa: E731
    return dict(temperature=f(rng.choice([0.0, 0.3, 1.0, 1.3, 4.0], n)),
                top_k=[int(x) for x in rng.choice([0, 1, 40, 300, 1500, 2500, vocab - 1], n)],
                top_p=f(rng.choice([0.3, 0.9, 0.99, 1.0], n)), min_p=f(rng.choice([0.0, 0.0, 0.01, 0.2], n)))


def alone(x, u, s, param_rows=1):
    """Each row by itself."""
    tokens, probs = [], []
    for r in range(x.shape[0]):
        a = {k: dev([v[r // param_rows]], torch.int32 if k == "top_k" else torch.float32) for k, v in s.items()}
        t, p = sample_tokens(x[r:r + 1], dev(u[r:r + 1]), with_probs=True, **a)
        tokens.append(t)
        probs.append(p)
    return torch.cat(tokens), torch.cat(probs)


def batch(x, u, s, rows, param_rows=1):
    check(x, u, param_rows=param_rows, rows=rows, **s)
    a = {k: dev(v, torch.int32 if k == "top_k" else torch.float32) for k, v in s.items()}
    tokens, probs = sample_tokens(x, dev(u), with_probs=True, param_rows=param_rows, **a)
    t, p = alone(x, u, s, param_rows)
    assert torch.equal(tokens, t)
    assert torch.equal(probs, p)


# CTAs to a row of 256 threads: 1, 2, 4 and 8 (fp32: 1024 logits to a step of a CTA, else 2048)
@pytest.mark.parametrize("dtype,vocab", [("fp32", 1000), ("fp32", 2000), ("fp32", 4001), ("fp32", 20011),
                                         ("bf16", 2047), ("bf16", 4000), ("bf16", 8001), ("bf16", 33000),
                                         ("fp16", 3999), ("fp16", 50000)])
def test_clusters(dtype, vocab):
    rng = np.random.default_rng(vocab)
    x = logits_of(rng, N, vocab, dtype, 2.0)
    x[3, ::2] = x[3, 0]      # many ties
    x[4, vocab // 2:] = -np.inf
    x[5] = -np.inf
    x[6, 7] = np.inf
    u = rng.random(N).astype(np.float32).tolist()
    batch(x, u, settings_of(rng, N, vocab), rows=[0, 3, 4, 5, 6, 17, 29])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_ties_over_the_ctas_of_a_row(dtype):
    """Whole rows of one and of two values: the border's tokens lie in all CTAs of the row, and are
    more than its list holds."""
    rng = np.random.default_rng(1)
    vocab = 20011
    x = torch.zeros((N, vocab), dtype=TYPES[dtype], device="cuda")
    x[10:, ::3] = 1.0
    x[20:, 1::3] = -0.0
    u = rng.random(N).astype(np.float32).tolist()
    s = dict(top_k=[int(k) for k in rng.choice([0, 5, 2500, 7000, vocab - 1], N)],
             top_p=[float(np.float32(p)) for p in rng.choice([0.1, 0.6, 0.99, 1.0], N)])
    batch(x, u, s, rows=[0, 9, 12, 22, 39])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_flat_rows(dtype):
    """A threshold's bin holds more tokens than the list."""
    rng = np.random.default_rng(2)
    vocab = 30000
    x = logits_of(rng, N, vocab, dtype, 1.0)
    u = rng.random(N).astype(np.float32).tolist()
    s = dict(temperature=[20.0] * N, top_p=[float(np.float32(p)) for p in rng.choice([0.2, 0.7, 0.95], N)],
             top_k=[int(k) for k in rng.choice([0, 0, 9000], N)])
    batch(x, u, s, rows=[0, 13, 26])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rows_off_boundaries_and_shared_settings(dtype):
    """A verify step's target: settings for every five rows, rows that start off 16-byte boundaries."""
    rng = np.random.default_rng(3)
    x = logits_of(rng, N, 12345, dtype, 2.0, pad=2)
    u = rng.random(N).astype(np.float32).tolist()
    batch(x, u, settings_of(rng, N // 5, 12345), rows=[0, 4, 5, 39], param_rows=5)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rows_too_long_to_keep(dtype):
    """Read from memory at every pass, by CTAs of 256 and of 512 threads."""
    rng = np.random.default_rng(4)
    vocab, live = (500001, 20000) if dtype == "fp32" else (900001, 20000)
    x = torch.full((24, vocab), -np.inf, dtype=TYPES[dtype], device="cuda")
    at = torch.from_numpy(rng.permutation(vocab)[:live]).cuda()
    x[:, at] = logits_of(rng, 24, live, dtype, 2.0)
    u = rng.random(24).astype(np.float32).tolist()
    batch(x, u, settings_of(rng, 24, live), rows=[0, 23])


def test_target_of_a_verify_step():
    """Probabilities of many rows into a strided output: what lies between its rows stays."""
    rng = np.random.default_rng(5)
    x = logits_of(rng, N, 5003, "bf16", 2.0)
    p = dev([0.9] * (N // 8))
    out = torch.full((N, 5020), -7.0, device="cuda")
    token_probs(x, top_p=p, param_rows=8, out=out[:, 5:5008])
    assert (out[:, :5] == -7).all() and (out[:, 5008:] == -7).all()
    assert torch.equal(out[:, 5:5008], token_probs(x, top_p=p, param_rows=8))
