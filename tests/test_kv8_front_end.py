"""What the tensor-level front end of the 8-bit cache and the pages does around the library's
calls, on the CPU: the library is a stand-in that records how it is called, and CPU tensors
that say they are on a GPU stand for device memory."""
import contextlib
import threading
import time

import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_attention_indexer_gb300")
from sparse_attention_indexer_gb300 import api  # noqa: E402


class Device(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    is_cuda = True
    index = 0

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index

    def record_stream(self, stream):
        recorded.append((self.data_ptr(), stream))


recorded = []


class Elsewhere(Device):
    """The same on a second GPU."""
    index = 1


def dev(t):
    return t.as_subclass(Device)


def elsewhere(t):
    return t.as_subclass(Elsewhere)


class Torch:
    """torch for the front end: what it makes is on the CPU and says it is on a GPU."""

    def __init__(self):
        self.cuda = self.Cuda()

    class Cuda:
        capturing = False
        index = 0

        def current_device(self):
            return self.index

        def ExternalStream(self, handle):
            return handle

        def current_stream(self):
            return 7

        def default_stream(self):
            return 0

        def stream(self, stream):
            return contextlib.nullcontext()

        def is_current_stream_capturing(self):
            return self.capturing

        def __getattr__(self, name):
            return getattr(torch.cuda, name)

    def __getattr__(self, name):
        return getattr(torch, name)

    def empty(self, shape, dtype=None, device=None):
        return dev(torch.empty(shape, dtype=dtype))

    def zeros(self, shape, dtype=None, device=None):
        return dev(torch.zeros(shape, dtype=dtype))


class Library:
    """Records its calls; a call of two launches takes a while between them."""

    def __init__(self):
        self.launches = []
        self.calls = []

    def kvpages_workspace_bytes(self, n, pages):
        return 1024

    def kv8_attention_workspace_bytes(self, *a):
        return 512

    def __getattr__(self, name):
        def call(*a):
            me = (name, threading.get_ident(), len(self.calls))
            self.calls.append((name, a))
            self.launches.append(me)
            if name in ("kv8_attention", "kv8_attention_selected", "kvpages_reserve",
                        "kvpages_compact"):
                time.sleep(0.002)
                self.launches.append(me)
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(api.B, "lib", lambda: lib)
    monkeypatch.setattr(api.B, "_stream", lambda s: 7 if s is None else s or None)
    monkeypatch.setattr(api, "torch", Torch())
    monkeypatch.setattr(api, "_raw_stream", lambda device: 7)
    monkeypatch.setattr(api, "_current_device", lambda: api.torch.cuda.index)
    monkeypatch.setattr(api, "_capturing", lambda: api.torch.cuda.capturing)
    return lib


def cache():
    codes = lambda: dev(torch.zeros((64, 2, 64), dtype=torch.uint8))  # noqa: E731
    return S.Kv8Cache(codes(), codes(), dev(torch.ones(4, 2)), dev(torch.ones(4, 2)), 32, 16)


def attention_args(rows=2):
    return (dev(torch.zeros((rows, 4, 64), dtype=torch.bfloat16)),
            dev(torch.zeros(rows, dtype=torch.int32)), 32,
            dev(torch.zeros((rows, 1), dtype=torch.int32)), 0.1)


def in_pairs(launches):
    """Both launches of a call follow one another."""
    return len(launches) % 2 == 0 and all(a == b for a, b in zip(launches[::2], launches[1::2]))


def on_threads(*calls):
    failed = []

    def repeat(call):
        try:
            for _ in range(8):
                call()
        except BaseException as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=repeat, args=(c,)) for c in calls]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed


def test_attention_of_two_threads(library):
    """A call's two launches share a workspace with the next call's on the stream: no thread
    comes between them."""
    c, a = cache(), attention_args()
    q, slots = a[0], dev(torch.zeros((2, 3), dtype=torch.int32))
    on_threads(lambda: c.attention(*a), lambda: c.attention(*a),
               lambda: c.attention_selected(q, slots, 0.1))
    assert len(library.launches) == 48 and in_pairs(library.launches)


def pages():
    planes = [dev(torch.zeros((8, 16), dtype=torch.uint8))]
    return S.KvPages(dev(torch.full((4, 2), -1, dtype=torch.int32)),
                     dev(torch.zeros(8, dtype=torch.int32)), 16, planes)


def test_page_operations_of_two_threads(library):
    """reserve and compact leave a list of copies for their second launch: no other operation of
    the pool comes between."""
    p = pages()
    i = [dev(torch.zeros(2, dtype=torch.int32)) for _ in range(3)]
    on_threads(lambda: p.reserve(*i), lambda: p.compact(), lambda: p.reserve(*i))
    assert len(library.launches) == 48 and in_pairs(library.launches)
    library.launches.clear()
    on_threads(lambda: p.reserve(*i), lambda: (p.fork(*i), p.fork(*i)),
               lambda: (p.free(i[0]), p.free(i[0])), lambda: (p.copy(*i[:2]), p.copy(*i[:2])))
    two = [x for x in library.launches if x[0] == "kvpages_reserve"]
    at = [library.launches.index(x) for x in two[::2]]
    assert all(library.launches[j + 1] == library.launches[j] for j in at)


def test_a_captured_call_has_a_workspace_of_its_graph(library):
    """Streams are shared by captures, and graphs are replayed on any: a call in a capture takes
    memory of the graph's pool, which the call does not keep, and not the stream's workspace."""
    c, a = cache(), attention_args()
    q, slots = a[0], dev(torch.zeros((2, 3), dtype=torch.int32))

    def workspace():
        c.attention(*a)
        c.attention_selected(q, slots, 0.1)
        (_, x), (_, y) = library.calls[-2:]
        return x[-4], y[-4]

    eager = workspace()
    kept = dict(c._workspaces)
    api.torch.cuda.capturing = True
    made = []
    empty = api.torch.empty
    api.torch.empty = lambda *x, **k: made.append(empty(*x, **k)) or made[-1]
    captured = [workspace() for _ in range(2)]
    assert len({p for pair in captured for p in pair}) == 4  # `made` keeps them apart here
    assert not {p for pair in captured for p in pair} & set(eager)
    assert {p for pair in captured for p in pair} <= {t.data_ptr() for t in made}
    assert c._workspaces == kept
    api.torch.cuda.capturing = False
    assert workspace() == eager
    fresh = cache()
    api.torch.cuda.capturing = True
    fresh.attention(*a)  # the first call of a shape
    assert not fresh._workspaces


def each_elsewhere(call, args):
    """call(*args) is refused with any one tensor of args on another GPU, and works with none."""
    for i, t in enumerate(args):
        if isinstance(t, torch.Tensor):
            with pytest.raises(ValueError):
                call(*args[:i], elsewhere(t.as_subclass(torch.Tensor)), *args[i + 1:])
    call(*args)


def test_tensors_on_another_device_are_refused(library):
    c, a = cache(), attention_args()
    i = lambda *s: dev(torch.zeros(s, dtype=torch.int32))  # noqa: E731
    x = lambda: dev(torch.zeros((3, 2, 64), dtype=torch.bfloat16))  # noqa: E731
    out, lse = dev(torch.zeros((2, 4, 64), dtype=torch.bfloat16)), dev(torch.zeros(2, 4))
    each_elsewhere(c.store, (x(), x(), i(3), i(3), i(1, 2)))
    each_elsewhere(c.attention, (*a, 1, i(2), out, lse))
    each_elsewhere(c.attention_selected, (a[0], i(2, 5), 0.1, out, lse))
    codes = lambda: dev(torch.zeros((64, 2, 64), dtype=torch.uint8))  # noqa: E731
    ones = lambda: dev(torch.ones(4, 2))  # noqa: E731
    each_elsewhere(S.Kv8Cache, (codes(), codes(), ones(), ones(), 32, 16))
    p = pages()
    each_elsewhere(p.reserve, (i(2), i(2), i(2)))
    each_elsewhere(p.fork, (i(2), i(2), i(2)))
    each_elsewhere(p.free, (i(2), i(2)))
    each_elsewhere(p.copy, (i(2), i(2)))
    each_elsewhere(lambda t, r, x, y: S.KvPages(t, r, 16, [x, y]),
                   (i(4, 2), i(8), dev(torch.zeros(8, 16)), dev(torch.zeros(8, 4))))
    f = lambda *s: dev(torch.zeros(s))  # noqa: E731
    each_elsewhere(S.verify_drafts, (f(2, 3, 10), f(2, 2, 10), i(2, 2), f(2, 3), i(2), i(1)))


def test_another_current_device_is_refused(library):
    """The library launches on the current device."""
    c, a, p = cache(), attention_args(), pages()
    i = lambda *s: dev(torch.zeros(s, dtype=torch.int32))  # noqa: E731
    x = dev(torch.zeros((3, 2, 64), dtype=torch.bfloat16))
    f = lambda *s: dev(torch.zeros(s))  # noqa: E731
    api.torch.cuda.index = 1
    for call in (lambda: c.store(x, x, i(3), i(3), i(1, 2)), lambda: c.attention(*a),
                 lambda: c.attention_selected(a[0], i(2, 5), 0.1),
                 lambda: p.reserve(i(2), i(2), i(2)), lambda: p.fork(i(2), i(2), i(2)),
                 lambda: p.free(i(2)), lambda: p.compact(), lambda: p.copy(i(2), i(2)),
                 lambda: S.verify_drafts(f(2, 3, 10), None, i(2, 2), f(2, 3))):
        with pytest.raises(ValueError):
            call()
    assert not library.calls


def test_a_handles_own_buffers_are_recorded_on_the_streams_it_serves(library):
    """They come from the pool of the stream that the handle was made on, which would give them
    out again while another stream's work is on its way."""
    i = lambda *s: dev(torch.zeros(s, dtype=torch.int32))  # noqa: E731
    c, a, p = cache(), attention_args(), pages()
    x = dev(torch.zeros((3, 2, 64), dtype=torch.bfloat16))
    buffers = [t.data_ptr() for t in (p.workspace, p.new_ids, p.counts, p.status)]
    recorded.clear()
    p.reserve(i(2), i(2), i(2))
    c.store(x, x, i(3), i(3), i(1, 2))
    c.attention(*a)
    assert not recorded
    for call in (lambda s: p.reserve(i(2), i(2), i(2), stream=s), lambda s: p.compact(stream=s),
                 lambda s: p.free(i(2), stream=s), lambda s: p.copy(i(2), i(2), stream=s),
                 lambda s: p.fork(i(2), i(2), i(2), stream=s)):
        p = pages()
        buffers = [t.data_ptr() for t in (p.workspace, p.new_ids, p.counts, p.status)]
        for stream in (9, 9, 0, 7):
            call(stream)
        assert sorted(recorded, key=str) == sorted([(b, s) for b in buffers for s in (9, 0)], key=str)
        recorded.clear()
    for call in (lambda s: c.store(x, x, i(3), i(3), i(1, 2), stream=s),
                 lambda s: c.attention(*a, stream=s),
                 lambda s: c.attention_selected(a[0], i(2, 5), 0.1, stream=s)):
        c = cache()
        call(9)
        call(9)
        call(7)
        assert recorded == [(c.status.data_ptr(), 9)]
        recorded.clear()
