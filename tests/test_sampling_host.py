"""Shared prefixes, step maps and sampling without a GPU: pins of their oracles (hand-worked
values, invariants, planted mistakes), the host-side argument checks of their entry points
(every error is returned before any CUDA call), and the checks of the tensor-level front end."""
import math
import os

import numpy as np
import pytest

from oracle import kv_pages as KP
from oracle import token_sample as TS

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_attention_indexer_gb300")
B = S.binding

from tests.test_kv8_front_end import Library, Torch, dev, elsewhere  # noqa: E402


# ------------------------------------------------------------------ oracles
def test_weights_hand_worked():
    x = np.float32(np.log(2)) * -np.arange(5, dtype=np.float32)
    w = TS.weights(x, 1.0)
    assert w[0] == 1 << 40
    for i in range(1, 5):  # z is i but for the rounding of log 2 and of the product
        assert abs(w[i] - (1 << (40 - i))) <= 2.0 ** (40 - i) * 2.0 ** -20
    assert TS.weights(np.float32([0, -100]), 1.0)[1] == 0
    assert TS.weights(np.float32([np.inf, 1, -np.inf]), 1.0) == [1 << 40, 0, 0]
    assert TS.weights(np.float32([3, 3, -5]), 1e-30) == [1 << 40, 1 << 40, 0]


def test_weights_are_near_the_exponential():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(2000) * 5).astype(np.float32)
    for t in (0.3, 1.0, 2.5):
        w = np.array([float(a) for a in TS.weights(x, t)]) / 2.0 ** 40
        z = (x.max() - x.astype(np.float64)) / t / math.log(2)
        ref = 2.0 ** -z
        # the polynomial 2^-22.3; z itself, three roundings of 2^-24 times ln 2; 2^-40 cut off
        assert (np.abs(w - ref) <= ref * (2.0 ** -22.3 + 3 * 2.0 ** -24 * z) + 2.0 ** -40).all()


def test_rows_hand_worked():
    x = np.float32([1.0, 3.0, 2.0, 3.0])
    one = 1 << 40
    assert TS.row(x, 0.0, temperature=0.0) == (1, [0, one, 0, 0], 0)
    assert TS.row(x, 0.0, top_k=1) == (1, [0, one, 0, 0], 0)
    assert TS.row(x, 0.5, top_k=2) == (3, [0, one, 0, one], 0)
    assert TS.row(x, 0.49999, top_k=2)[0] == 1
    assert TS.row(x, 0.0, top_p=0.0)[1] == [0, one, 0, 0]
    # the weights are 1, 1, e^-1 and e^-2, 2.5032 together: 0.8 of that is 2.0026, 0.79 of it 1.9775
    assert [a > 0 for a in TS.row(x, 0.0, top_p=0.8)[1]] == [False, True, True, True]
    assert [a > 0 for a in TS.row(x, 0.0, top_p=0.79)[1]] == [False, True, False, True]
    assert [a > 0 for a in TS.row(x, 0.0, min_p=0.3)[1]] == [False, True, True, True]   # e^-1 = 0.37
    assert [a > 0 for a in TS.row(x, 0.0, min_p=0.4)[1]] == [False, True, False, True]
    # top-p of the first k: 0.9 of 2 needs both
    assert [a > 0 for a in TS.row(x, 0.0, top_k=2, top_p=0.9)[1]] == [False, True, False, True]


def test_rows_special():
    nan = float("nan")
    assert TS.row([-np.inf] * 3, 0.5) == (-1, [0, 0, 0], TS.EMPTY)
    assert TS.row([nan, 1.0], 0.5) == (1, [0, 1 << 40], TS.NAN)
    assert TS.row([1.0, 1.0], 1.0)[0::2] == (1, TS.UNIFORM) and TS.row([1.0, 1.0], nan)[0::2] == (0, TS.UNIFORM)
    for kw in (dict(temperature=-1.0), dict(temperature=nan), dict(top_p=nan), dict(min_p=nan), dict(min_p=1.5)):
        assert TS.row([2.0, 1.0], 0.1, **kw)[2] == TS.PARAM


@pytest.mark.parametrize("mutant", [1, 2, 3, 4, 5])
def test_planted_mistakes_of_sampling_show(mutant):
    rng = np.random.default_rng(1)
    seen = 0
    for i in range(60):
        x = np.round(rng.standard_normal(40) * 2).astype(np.float32)  # ties
        kw = dict(top_k=int(rng.integers(1, 20)), top_p=float(rng.uniform(0.2, 0.95)), min_p=float(rng.uniform(0, 0.2)))
        u = [0.0, 0.5, float(rng.random())][i % 3]
        seen += TS.row(x, u, **kw)[:2] != TS.row(x, u, mutant=mutant, **kw)[:2]
    assert seen


def test_tokens_come_as_often_as_their_weights_say():
    x = np.float32([0.0, 1.0, 2.0, 0.5])
    n = 4096
    counts = np.bincount([TS.row(x, (i + 0.5) / n)[0] for i in range(n)], minlength=4)
    p = np.exp(x - x.max()) / np.exp(x - x.max()).sum()
    assert (np.abs(counts - n * p) <= 1.5).all()  # uniforms on a grid: within one of the exact share


TABLE = np.array([[3, 1, -1], [3, 4, 9], [3, 1, 5]], np.int32)


def test_step_hand_worked():
    got = KP.step([2, 0], [1, 30], [3, 33], TABLE, 16, 8, 7)
    assert [x.tolist() for x in got[:5]] == [
        [1, 2, 30, 31, 32, -1, -1], [2, 2, 0, 0, 0, -1, -1], [49, 50, 30, 31, -1, -1, -1],
        [2, 3, 31, 32, 33, 0, 0], [0, 2, 5]]
    assert got[5] == KP.NO_PAGE
    got = KP.step([2, 7, 1], [0, 0, 32], [5, 5, 34], TABLE, 16, 8, 6)
    assert got[4].tolist() == [0, 5, 5, 6] and got[5] == KP.ROW | KP.PAGE | KP.TOKENS


def test_shared_hand_worked():
    assert KP.shared([0, 2], [48, 40], [0, 2], TABLE, 16, 8)[0].tolist() == [32]
    assert KP.shared([0, 2], [48, 31], [0, 2], TABLE, 16, 8)[0].tolist() == [16]
    assert KP.shared([0, 1, 2], [48, 0, 40], [0, 3, 3], TABLE, 16, 8)[0].tolist() == [32, 0]
    assert KP.shared([0, 1], [48, 40], [0, 2], TABLE, 16, 8)[0].tolist() == [16]
    assert KP.shared([0], [48], [0, 1], TABLE, 16, 8)[0].tolist() == [0]


def test_planted_mistakes_of_maps_show():
    a = KP.step([2, 0], [1, 30], [3, 33], TABLE, 16, 8, 7)
    for mutant in (6, 7):
        b = KP.step([2, 0], [1, 30], [3, 33], TABLE, 16, 8, 7, mutant)
        assert any(not np.array_equal(x, y) for x, y in zip(a[:5], b[:5]))
    assert KP.shared([0, 1, 2], [48, 0, 40], [0, 3], TABLE, 16, 8, 8)[0].tolist() != [32]


# ------------------------------------------------------------------ host checks of the library
def _lib():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("library not built")
    return B.lib()


A = 0x10000  # a pointer that is aligned and never read


def _call(name, defaults, kw):
    assert not set(kw) - set(defaults)
    return getattr(_lib(), name)(*{**defaults, **kw}.values())


def _shared_attention(**kw):
    return _call("kv8_attention_shared", dict(
        q=A, q_ld=512, dtype=0, rows=2, q_heads=4, kv_heads=2, dim=128, sm_scale=0.1, lens=A, max_len=100,
        group_rows=1, group_table=None, set_starts=A, n_sets=1, prefix_lens=A, max_prefix=200, block_table=A,
        n_tables=2, table_ld=4, page_size=64, block_tokens=32, k_cache=A, v_cache=A, k_scale=A, v_scale=A,
        num_slots=256, out=A, out_ld=512, lse=None, workspace=A, ws_bytes=1 << 40, status=None, stream=None), kw)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(rows=-1), dict(kv_heads=0), dict(q_heads=3), dict(q_heads=34), dict(dim=96), dict(max_len=-1),
    dict(group_rows=0), dict(group_rows=9), dict(n_sets=-1), dict(n_sets=B.KV8_MAX_SETS + 1), dict(max_prefix=-1),
    dict(n_tables=0), dict(table_ld=0), dict(page_size=0), dict(block_tokens=8), dict(block_tokens=48), dict(num_slots=100),
    dict(q_ld=504), dict(out_ld=516), dict(sm_scale=math.nan), dict(rows=1 << 30)])
def test_shared_attention_shapes(kw):
    assert _shared_attention(**kw) == B.KV8_ERR_SHAPE


def test_shared_attention_pointers():
    assert _shared_attention(rows=0, q=None) == 0
    for name in ("q", "lens", "set_starts", "prefix_lens", "block_table", "k_cache", "v_cache", "k_scale", "v_scale", "out",
                 "workspace"):
        assert _shared_attention(**{name: None}) == B.KV8_ERR_NULL, name
    for name, at in (("q", 8), ("out", 8), ("workspace", 8), ("k_cache", 8), ("lens", 2), ("set_starts", 2), ("prefix_lens", 1),
                     ("group_table", 2), ("lse", 2), ("status", 1), ("v_scale", 2)):
        assert _shared_attention(**{name: A + at}) == B.KV8_ERR_ALIGN, name
    assert _lib().kv8_attention_shared_workspace_bytes(-1, 4, 2, 128, 1) == B.KV8_ERR_SHAPE
    assert _lib().kv8_attention_shared_workspace_bytes(8, 4, 3, 128, 1) == B.KV8_ERR_SHAPE


def _step(**kw):
    return _call("kvpages_step", dict(
        rows=A, old_lens=A, new_lens=A, n=4, block_table=A, n_tables=2, table_ld=4, page_size=64, num_pages=10, tokens=9,
        positions=A, token_table=A, slots=A, lens=A, starts=A, status=None, stream=None), kw)


def _shared(**kw):
    return _call("kvpages_shared", dict(
        rows=A, lens=A, n=4, set_starts=A, n_sets=2, block_table=A, n_tables=2, table_ld=4, page_size=64, num_pages=10,
        prefix_lens=A, status=None, stream=None), kw)


def test_maps_shapes_and_pointers():
    for kw in (dict(n=-1), dict(n_tables=0), dict(table_ld=0), dict(page_size=0), dict(num_pages=-1),
               dict(num_pages=1 << 26, page_size=32)):
        assert _step(**kw) == B.KVPAGES_ERR_SHAPE and _shared(**kw) == B.KVPAGES_ERR_SHAPE, kw
    assert _step(tokens=-1) == B.KVPAGES_ERR_SHAPE and _shared(n_sets=-1) == B.KVPAGES_ERR_SHAPE
    assert _shared(n_sets=0, set_starts=None) == 0
    for name in ("rows", "old_lens", "new_lens", "block_table", "positions", "token_table", "slots", "lens", "starts"):
        assert _step(**{name: None}) == B.KVPAGES_ERR_NULL, name
        assert _step(**{name: A + 2}) == B.KVPAGES_ERR_ALIGN, name
    for name in ("rows", "lens", "set_starts", "block_table", "prefix_lens"):
        assert _shared(**{name: None}) == B.KVPAGES_ERR_NULL, name
        assert _shared(**{name: A + 2}) == B.KVPAGES_ERR_ALIGN, name


def _sample(**kw):
    return _call("token_sample", dict(
        logits=A, ld=100, dtype=2, rows=3, vocab=100, temperature=None, top_k=None, top_p=None, min_p=None, param_rows=1,
        uniforms=A, tokens=A, probs=A, probs_ld=100, status=None, stream=None), kw)


def test_sample_shapes_and_pointers():
    for kw in (dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(rows=1 << 28), dict(vocab=0), dict(vocab=(1 << 20) + 1, ld=1 << 21),
               dict(ld=99), dict(param_rows=0), dict(probs_ld=99)):
        assert _sample(**kw) == B.SAMPLE_ERR_SHAPE, kw
    assert _sample(rows=0, logits=None) == 0
    for kw in (dict(logits=None), dict(uniforms=None), dict(tokens=None, probs=None)):
        assert _sample(**kw) == B.SAMPLE_ERR_NULL, kw
    for name in ("logits", "temperature", "top_k", "top_p", "min_p", "uniforms", "tokens", "probs", "status"):
        assert _sample(**{name: A + 2}) == B.SAMPLE_ERR_ALIGN, name
    assert _sample(dtype=0, logits=A + 1) == B.SAMPLE_ERR_ALIGN


# ------------------------------------------------------------------ front end
@pytest.fixture
def library(monkeypatch):
    from sparse_attention_indexer_gb300 import api
    lib = Library()
    lib.kv8_attention_shared_workspace_bytes = lambda *a: 512 * (1 + a[0])
    monkeypatch.setattr(api.B, "lib", lambda: lib)
    monkeypatch.setattr(api.B, "_stream", lambda s: 7 if s is None else s or None)
    monkeypatch.setattr(api, "torch", Torch())
    monkeypatch.setattr(api, "_raw_stream", lambda device: 7)
    monkeypatch.setattr(api, "_current_device", lambda: api.torch.cuda.index)
    monkeypatch.setattr(api, "_capturing", lambda: api.torch.cuda.capturing)
    lib.cuda = api.torch.cuda
    return lib


def i32(*x):
    return dev(torch.tensor(x, dtype=torch.int32))


def _cache():
    codes = lambda: dev(torch.zeros((128, 2, 64), dtype=torch.uint8))  # noqa: E731
    scales = lambda: dev(torch.ones((4, 2)))  # noqa: E731
    return S.Kv8Cache(codes(), codes(), scales(), scales(), 64, 32)


def _shared_args(rows=3, **kw):
    a = dict(q=dev(torch.zeros((rows, 4, 64), dtype=torch.bfloat16)), lens=dev(torch.ones(rows, dtype=torch.int32)), max_len=10,
             block_table=dev(torch.zeros((rows, 2), dtype=torch.int32)), sm_scale=0.1, set_starts=i32(0, rows),
             prefix_lens=i32(128), max_prefix=128)
    a.update(kw)
    return a


def test_the_workspace_of_shared_attention_grows_with_the_rows(library):
    c = _cache()
    for rows, size in ((3, 4), (2, 4), (3, 4), (8, 9), (5, 9)):
        c.attention_shared(**_shared_args(rows))
        assert library.calls[-1][0] == "kv8_attention_shared" and library.calls[-1][1][-3] == 512 * size
    held = library.calls[-1][1][-4]
    library.cuda.capturing = True
    c.attention_shared(**_shared_args(5))
    assert library.calls[-1][1][-4] != held and library.calls[-1][1][-3] == 512 * 6


def test_front_end_refusals(library):
    c = _cache()
    for bad in (dict(set_starts=i32(0)), dict(prefix_lens=i32(1, 2)), dict(set_starts=elsewhere(torch.zeros(2, dtype=torch.int32))),
                dict(prefix_lens=dev(torch.zeros(1))), dict(lens=i32(1)), dict(group_table=i32(0))):
        with pytest.raises(ValueError):
            c.attention_shared(**_shared_args(**bad))
    pool = S.KvPages(dev(torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)), i32(1, 1, 1, 1), 16)
    library.calls.clear()
    for bad in (dict(rows=i32(1)), dict(old_lens=dev(torch.zeros(2))), dict(new_lens=elsewhere(torch.zeros(2, dtype=torch.int32))),
                dict(tokens=-1)):
        with pytest.raises(ValueError):
            pool.step(**{**dict(rows=i32(0, 1), old_lens=i32(0, 0), new_lens=i32(1, 1), tokens=2), **bad})
    for bad in (dict(lens=i32(1)), dict(set_starts=dev(torch.zeros(2))), dict(set_starts=dev(torch.zeros(0, dtype=torch.int32))),
                dict(rows=elsewhere(torch.zeros(2, dtype=torch.int32)))):
        with pytest.raises(ValueError):
            pool.shared(**{**dict(rows=i32(0, 1), lens=i32(1, 1), set_starts=i32(0, 2)), **bad})
    assert not library.calls
    s = pool.step(i32(0, 1), i32(0, 0), i32(1, 4), 5)
    assert [x.shape[0] for x in s] == [5, 5, 5, 5, 3]
    args = library.calls[-1][1]
    assert [x.data_ptr() for x in s] == list(args[10:15])  # the outputs, one behind another


def test_sampling_front_end_refusals(library):
    x, u = dev(torch.zeros((4, 9))), dev(torch.zeros(4))
    for bad in (dict(logits=torch.zeros((4, 9))), dict(logits=dev(torch.zeros((4, 9), dtype=torch.float64))),
                dict(logits=dev(torch.zeros((9, 4))).t()), dict(uniforms=u[:3]), dict(uniforms=elsewhere(torch.zeros(4))),
                dict(top_k=u), dict(top_p=dev(torch.zeros(3))), dict(temperature=elsewhere(torch.ones(4))), dict(param_rows=0),
                dict(param_rows=2, min_p=u), dict(status=u)):
        with pytest.raises(ValueError):
            S.sample_tokens(**{**dict(logits=x, uniforms=u), **bad})
    for out in (dev(torch.zeros((4, 8))), dev(torch.zeros((4, 9), dtype=torch.float16)), elsewhere(torch.zeros((4, 9)))):
        with pytest.raises(ValueError):
            S.token_probs(x, out=out)
    assert not library.calls
    library.cuda.index = 1
    with pytest.raises(ValueError):
        S.sample_tokens(x, u)
