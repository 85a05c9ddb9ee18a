"""The attention's workspace: what calls that misuse it leave, who shares it."""

import threading
import time

import pytest

import memory_bound_gemv_gb300 as mbg
from memory_bound_gemv_gb300 import decode

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def make(lengths, heads=1, dim=64, page=16, seed=0, history=False, capacity=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    per = -(-(capacity or max(lengths)) // page)
    k, v = (torch.empty(len(lengths) * per, page, heads, dim, device="cuda").normal_(generator=g).half() for _ in range(2))
    table = torch.randperm(len(lengths) * per, generator=g, device="cuda").to(torch.int32).view(len(lengths), per)
    extra = dict(scores=torch.zeros(len(lengths), heads, per * page, device="cuda")) if history else {}
    return mbg.PagedKV(k, v, table, **extra), torch.tensor(lengths, dtype=torch.int32, device="cuda")


def query(cache, heads, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(cache.batch, heads, cache.head_dim, device="cuda").normal_(generator=g).half()


@pytest.mark.parametrize("lengths", [[70000], [20000] * 7, [3000, 0, 41, 900] * 60])
def test_attn_after_a_call_whose_lengths_changed(lengths):
    """Such a call can leave arrivals uncounted for; the calls after it count their own."""
    cache, n = make(lengths)
    queries = [query(cache, 4, seed) for seed in range(4)]
    good = [mbg.gemv_attn_paged(cache, q, n).clone() for q in queries]
    memory = cache._workspace(4, False, mbg._stream_ptr(None), None)[2]
    counters = memory[:decode._ATTN_COUNTER_BYTES].view(torch.int32)
    for step, q in enumerate(queries):
        counters[2::2] += 60  # more arrivals than are waited for
        out = mbg.gemv_attn_paged(cache, q, n, out=torch.full_like(q, 7.0))
        assert torch.equal(out, good[step]), step
    assert mbg.gemv_get_device_error() == mbg.OK


def test_attn_handles_of_one_size_share_a_workspace():
    """A model's layers on one stream: one workspace, not one each, and every layer its own answer."""
    lengths = [3000, 17, 900]
    layers = [make(lengths, heads=2, seed=s, history=True, capacity=20000) for s in range(4)]
    alone = []
    for cache, n in layers:
        alone.append(mbg.gemv_attn_paged(cache, query(cache, 8, 5), n, accumulate=True,
                                         scores_out=torch.zeros_like(cache.scores)).clone())
        cache.release_workspaces()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    outs = [mbg.gemv_attn_paged(cache, query(cache, 8, 5), n, accumulate=True) for cache, n in layers]
    held = torch.cuda.memory_allocated() - before
    need = max(w[1] for w in layers[0][0]._workspaces.values())
    assert need <= held < 2 * need  # (the outputs are small beside it)
    assert len({w[0] for cache, _ in layers for w in cache._workspaces.values()}) == 1
    assert all(torch.equal(a, b) for a, b in zip(outs, alone))
    del outs
    for cache, _ in layers:
        cache.release_workspaces()
    assert torch.cuda.memory_allocated() <= before
    small, n = make([50], heads=2)
    assert small._workspace(8, False, mbg._stream_ptr(None), None)[1] < need
    other = torch.cuda.Stream()
    first = layers[0][0]
    ptr = mbg._stream_ptr(None)
    assert first._workspace(8, True, ptr, None)[0] != first._workspace(8, True, mbg._stream_ptr(other), other)[0]


def test_attn_graphs_of_several_layers_and_their_release():
    """Layers captured into one graph share its workspace; graphs that are gone leave nothing behind."""
    lengths = [5000, 40]
    layers = [make(lengths, heads=2, seed=s, history=True) for s in range(3)]
    queries = [query(layers[0][0], 8, s) for s in range(3)]
    want = [mbg.gemv_attn_paged(cache, q, n).clone() for (cache, n), q in zip(layers, queries)]
    outs = [torch.empty_like(q) for q in queries]

    def captured():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for (cache, n), q, out in zip(layers, queries, outs):
                mbg.gemv_attn_paged(cache, q, n, out=out)
        return graph

    sizes = []
    for _ in range(4):
        for cache, _ in layers:
            cache.release_workspaces()
        graph = captured()
        assert len({w[0] for cache, _ in layers for w in cache._workspaces.values()}) == 1
        for out in outs:
            out.fill_(7.0)
        for _ in range(3):
            graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        torch.cuda.synchronize()
        sizes.append(torch.cuda.memory_allocated())
        del graph
    assert sizes[1:] == sizes[:-1]


@pytest.mark.parametrize("form", ["compiled checks", "Python checks"])
def test_attn_with_weights_from_several_threads(form, monkeypatch):
    """Threads on one stream: the attention of one call and its weights are not parted by another call's."""
    if form == "Python checks":
        decode._need_torch()

        class Absent:
            def __getattr__(self, name):
                return lambda *args: -1

        monkeypatch.setattr(decode, "_quick", Absent())
    cache, n = make([200, 100, 31, 77], heads=2, history=True)
    queries = [query(cache, 8, s) for s in range(4)]

    def call(i, out, sums):
        mbg.gemv_attn_paged(cache, queries[i], n, out=out, accumulate=True, scores_out=sums)

    want = []
    for i in range(4):
        want.append((torch.empty_like(queries[i]), torch.zeros_like(cache.scores)))
        call(i, *want[i])
    torch.cuda.synchronize()
    calls = 3000
    got = [[(torch.empty_like(queries[i]), torch.zeros_like(cache.scores)) for _ in range(calls)] for i in range(4)]
    go = threading.Barrier(4)

    def work(i):
        go.wait()
        for out, sums in got[i]:
            call(i, out, sums)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    wrong = sum(not (torch.equal(out, want[i][0]) and torch.equal(sums, want[i][1])) for i in range(4) for out, sums in got[i])
    assert wrong == 0


def test_attn_with_weights_is_one_call_at_a_time_per_workspace(monkeypatch):
    """What lets another thread's launches between a call's two: no two calls overlap on one workspace."""
    cache, n = make([20, 31], heads=2, history=True)
    other = mbg.PagedKV(cache.k, cache.v, cache.page_table, scores=torch.zeros_like(cache.scores))  # shares the workspace
    q = query(cache, 8, 1)
    for c in (cache, other):
        mbg.gemv_attn_paged(c, q, n, accumulate=True)
    state, guard = dict(inside=0, most=0, calls=0), threading.Lock()

    class Watched:
        """A library, or compiled checks, whose attention takes its time without holding the interpreter."""

        def __init__(self, real, name):
            self._real, self._name = real, name

        def __getattr__(self, name):
            f = getattr(self._real, name)
            if name != self._name:
                return f

            def watched(*args):
                with guard:
                    state["inside"] += 1
                    state["most"] = max(state["most"], state["inside"])
                    state["calls"] += 1
                time.sleep(0.002)
                result = f(*args)
                with guard:
                    state["inside"] -= 1
                return result

            return watched

    for c in (cache, other):
        c._lib = Watched(c._lib, "gemv_attn_paged")
    monkeypatch.setattr(decode, "_quick", Watched(decode._quick, "attn"))

    def work(i):
        for _ in range(10):
            mbg.gemv_attn_paged((cache, other)[i % 2], q, n, accumulate=True)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert state["calls"] == 40 and state["most"] == 1


def test_attn_calls_with_weights_or_a_new_output_take_the_compiled_checks(monkeypatch):
    cache, n = make([40, 31], heads=2, history=True)
    q, sums = query(cache, 8, 1), torch.zeros_like(cache.scores)
    want = mbg.gemv_attn_paged(cache, q, n, out=torch.empty_like(q))

    def refused(*args):
        raise AssertionError("not through the Python form")

    monkeypatch.setattr(decode, "_operand", refused)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert torch.equal(mbg.gemv_attn_paged(cache, q, n), want)
    assert torch.equal(mbg.gemv_attn_paged(cache, q, n, accumulate=True), want)
    assert torch.equal(mbg.gemv_attn_paged(cache, q, n, out=torch.empty_like(q), accumulate=True), want)
    streamed = mbg.gemv_attn_paged(cache, q, n, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(streamed, want)
    monkeypatch.undo()
    assert torch.equal(mbg.gemv_attn_paged(cache, q, n, accumulate=True, scores_out=sums), want)
    # two calls have added to the scores, and the third adds to a copy
    close = (sums - 1.5 * cache.scores).abs() <= 2.0 ** -21 * sums
    assert close.all() and (cache.scores[0, :, :40] > 0).all()
