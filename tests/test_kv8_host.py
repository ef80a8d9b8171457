"""Host-side argument checks of the 8-bit cache, the page operations and the drafts'
verification (no GPU needed: every error is returned before any CUDA call), and the checks
of the tensor-level front end."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_attention_indexer_gb300")
B = S.binding


def _lib():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("library not built")
    return B.lib()


A = 0x10000  # a pointer that is aligned and never read


def _store(**kw):
    a = dict(k=A, k_ld=256, v=A, v_ld=256, dtype=0, tokens=4, kv_heads=2, dim=128, positions=A,
             token_table=A, block_table=A, n_tables=1, table_ld=4, page_size=64, block_tokens=32,
             k_cache=A, v_cache=A, k_scale=A, v_scale=A, num_slots=256, status=None, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return _lib().kv8_store(*a.values())


def _attention(**kw):
    a = dict(q=A, q_ld=512, dtype=0, rows=2, q_heads=4, kv_heads=2, dim=128, sm_scale=0.1, lens=A,
             max_len=100, group_rows=1, group_table=None, block_table=A, n_tables=2, table_ld=4,
             page_size=64, block_tokens=32, k_cache=A, v_cache=A, k_scale=A, v_scale=A,
             num_slots=256, out=A, out_ld=512, lse=None, workspace=A, ws_bytes=1 << 40,
             status=None, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return _lib().kv8_attention(*a.values())


def _selected(**kw):
    a = dict(q=A, q_ld=512, dtype=0, rows=2, q_heads=4, kv_heads=2, dim=128, sm_scale=0.1,
             slots=A, k=16, slots_ld=16, block_tokens=32, k_cache=A, v_cache=A, k_scale=A,
             v_scale=A, num_slots=256, out=A, out_ld=512, lse=None, workspace=A,
             ws_bytes=1 << 40, status=None, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return _lib().kv8_attention_selected(*a.values())


SHAPE, NULL, ALIGN = B.KV8_ERR_SHAPE, B.KV8_ERR_NULL, B.KV8_ERR_ALIGN


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(tokens=-1), dict(kv_heads=0), dict(dim=96), dict(n_tables=0),
    dict(table_ld=0), dict(page_size=0), dict(block_tokens=0), dict(block_tokens=8),
    dict(block_tokens=24), dict(block_tokens=48), dict(block_tokens=128), dict(num_slots=-64),
    dict(num_slots=100), dict(num_slots=1 << 31), dict(k_ld=248), dict(v_ld=250)])
def test_store_shapes(kw):
    assert _store(**kw) == SHAPE


def test_store_pointers():
    assert _store(tokens=0, k=None) == 0
    for name in ("k", "v", "positions", "token_table", "block_table", "k_cache", "v_cache",
                 "k_scale", "v_scale"):
        assert _store(**{name: None}) == NULL, name
    for name in ("k", "v", "k_cache", "v_cache"):
        assert _store(**{name: A + 8}) == ALIGN, name
    for name in ("positions", "token_table", "block_table", "k_scale", "v_scale", "status"):
        assert _store(**{name: A + 2}) == ALIGN, name


@pytest.mark.parametrize("kw", [
    dict(dtype=-1), dict(rows=-1), dict(q_heads=3), dict(q_heads=0), dict(q_heads=34),
    dict(kv_heads=0), dict(dim=32), dict(sm_scale=float("nan")), dict(sm_scale=float("inf")),
    dict(max_len=-1), dict(group_rows=0), dict(group_rows=9), dict(n_tables=0), dict(table_ld=0),
    dict(page_size=0), dict(block_tokens=8), dict(block_tokens=48), dict(num_slots=100),
    dict(num_slots=-64), dict(num_slots=1 << 31), dict(q_ld=504), dict(q_ld=516),
    dict(out_ld=500), dict(out_ld=516)])
def test_attention_shapes(kw):
    assert _attention(**kw) == SHAPE


def test_attention_pointers():
    assert _attention(rows=0, q=None) == 0
    for name in ("q", "lens", "block_table", "k_cache", "v_cache", "k_scale", "v_scale", "out",
                 "workspace"):
        assert _attention(**{name: None}) == NULL, name
    for name in ("q", "k_cache", "v_cache", "out", "workspace"):
        assert _attention(**{name: A + 8}) == ALIGN, name
    for name in ("lens", "group_table", "block_table", "k_scale", "v_scale", "lse", "status"):
        assert _attention(**{name: A + 2}) == ALIGN, name


@pytest.mark.parametrize("kw", [dict(k=-1), dict(slots_ld=15), dict(block_tokens=20),
                                dict(num_slots=250), dict(rows=-1), dict(dim=256)])
def test_selected_shapes(kw):
    assert _selected(**kw) == SHAPE


def test_selected_pointers():
    assert _selected(rows=0, q=None) == 0
    for name in ("q", "slots", "k_cache", "out", "workspace"):
        assert _selected(**{name: None}) == NULL, name
    assert _selected(slots=A + 2) == ALIGN


def test_workspace_query_refuses():
    lib = _lib()
    for a in ((3, 2, 128, 1), (64, 2, 128, 1), (8, 8, 100, 1), (8, 8, 128, 0), (8, 8, 128, 9)):
        assert lib.kv8_attention_workspace_bytes(*a) == SHAPE


def _planes(*items):
    p = (B.KvPlane * max(1, len(items)))()
    for i, (base, n) in enumerate(items):
        p[i].base, p[i].page_bytes = base, n
    return p


def test_pages_refusals():
    lib = _lib()
    table = (A, 4, 8, 64, A, 100)  # block_table, n_tables, table_ld, page_size, refs, pages
    ok = _planes((A, 64))

    def reserve(rows=A, n=2, table=table, planes=ok, n_planes=1, ws=A, ws_bytes=1 << 30):
        return lib.kvpages_reserve(rows, A, A, n, *table, planes, n_planes, ws, ws_bytes, None,
                                   None)

    e = B
    assert reserve(n=-1) == e.KVPAGES_ERR_SHAPE
    for i, v in ((1, 0), (2, 0), (2, 1 << 31), (3, 0), (5, -1)):
        t = list(table)
        t[i] = v
        assert reserve(table=t) == e.KVPAGES_ERR_SHAPE
        assert lib.kvpages_fork(A, A, A, 2, *t, None, None) == e.KVPAGES_ERR_SHAPE
        assert lib.kvpages_free(A, None, 2, *t, None, None) == e.KVPAGES_ERR_SHAPE
    assert reserve(n_planes=241) == e.KVPAGES_ERR_SHAPE
    assert reserve(n_planes=-1) == e.KVPAGES_ERR_SHAPE
    assert reserve(planes=_planes((A, 0))) == e.KVPAGES_ERR_SHAPE
    assert reserve(planes=_planes((A, 6))) == e.KVPAGES_ERR_SHAPE
    assert reserve(planes=_planes((A + 2, 64))) == e.KVPAGES_ERR_ALIGN
    assert reserve(planes=_planes((None, 64))) == e.KVPAGES_ERR_NULL
    assert reserve(planes=None) == e.KVPAGES_ERR_NULL
    assert reserve(rows=None) == e.KVPAGES_ERR_NULL
    assert reserve(rows=A + 1) == e.KVPAGES_ERR_ALIGN
    assert reserve(ws=None) == e.KVPAGES_ERR_NULL
    assert reserve(ws=A + 4) == e.KVPAGES_ERR_ALIGN
    assert reserve(ws_bytes=lib.kvpages_workspace_bytes(2, 100) - 1) == e.KVPAGES_ERR_WORKSPACE
    assert reserve(n=0, rows=None) == 0
    assert lib.kvpages_workspace_bytes(-1, 5) == 0
    assert lib.kvpages_fork(None, A, A, 2, *table, None, None) == e.KVPAGES_ERR_NULL
    assert lib.kvpages_fork(A, A + 2, A, 2, *table, None, None) == e.KVPAGES_ERR_ALIGN
    assert lib.kvpages_free(None, None, 2, *table, None, None) == e.KVPAGES_ERR_NULL
    assert lib.kvpages_free(A, A + 2, 2, *table, None, None) == e.KVPAGES_ERR_ALIGN
    assert lib.kvpages_fork(A, A, A, 0, *table, None, None) == 0
    assert lib.kvpages_free(A, None, 0, *table, None, None) == 0

    def compact(ids=A, pages=100, ws_bytes=1 << 30):
        return lib.kvpages_compact(A, 4, 8, A, pages, ok, 1, ids, None, A, ws_bytes, None, None)

    assert compact(pages=-1) == e.KVPAGES_ERR_SHAPE
    assert compact(ids=None) == e.KVPAGES_ERR_NULL
    assert compact(ids=A + 2) == e.KVPAGES_ERR_ALIGN
    assert compact(ws_bytes=lib.kvpages_workspace_bytes(0, 100) - 1) == e.KVPAGES_ERR_WORKSPACE
    assert lib.kvpages_copy(A, A, -1, 100, ok, 1, None, None) == e.KVPAGES_ERR_SHAPE
    assert lib.kvpages_copy(None, A, 2, 100, ok, 1, None, None) == e.KVPAGES_ERR_NULL
    assert lib.kvpages_copy(A, A + 2, 2, 100, ok, 1, None, None) == e.KVPAGES_ERR_ALIGN
    assert lib.kvpages_copy(A, A, 0, 100, ok, 1, None, None) == 0
    assert ctypes.sizeof(B.KvPlane) == 16


def _verify(**kw):
    a = dict(target=A, target_req=300, target_row=100, draft=A, draft_req=200, draft_row=100,
             tokens=A, n_drafts=None, uniforms=A, reqs=2, drafts=2, vocab=100, out=A, kept=A,
             status=None, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return _lib().draft_verify(*a.values())


def test_verify_refusals():
    for kw in (dict(reqs=-1), dict(drafts=-1), dict(drafts=32), dict(vocab=0),
               dict(vocab=(1 << 30) + 1), dict(target_row=99), dict(draft_row=99),
               dict(target_req=-1), dict(draft_req=-1)):
        assert _verify(**kw) == B.VERIFY_ERR_SHAPE, kw
    for name in ("target", "tokens", "uniforms", "out", "kept"):
        assert _verify(**{name: None}) == B.VERIFY_ERR_NULL, name
    for name in ("target", "draft", "tokens", "n_drafts", "uniforms", "out", "kept", "status"):
        assert _verify(**{name: A + 2}) == B.VERIFY_ERR_ALIGN, name
    assert _verify(reqs=0, target=None) == 0


def test_front_end_refusals():
    """The front end's own checks: types, shapes and layouts (CPU tensors stand in where the
    check comes before any pointer is taken)."""
    c = torch.zeros((64, 2, 128), dtype=torch.uint8)
    with pytest.raises(ValueError):
        S.Kv8Cache(c, c, torch.ones(2, 2), torch.ones(2, 2), 32, 32)  # not CUDA
    i = torch.zeros((1, 2), dtype=torch.int32)
    t = torch.zeros((1, 3, 10))
    u = torch.zeros((1, 3))
    for args in ((t.double(), None, i, u), (t[:, :2], None, i, u), (t, t, i, u),
                 (t, None, i.long(), u), (t, None, i, u[:, :2]), (t, None, i, u.double()),
                 (t.transpose(1, 2), None, i, u)):
        with pytest.raises(ValueError):
            S.verify_drafts(*args)
    with pytest.raises(ValueError):
        S.KvPages(i, torch.zeros(4, dtype=torch.int32), 64)  # not CUDA
    with pytest.raises(ValueError):
        S.KvPages(i.long(), torch.zeros(4, dtype=torch.int32), 64)
