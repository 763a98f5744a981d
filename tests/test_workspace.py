"""Which workspace a call without one of its own gets (CPU: the stream and
whether it is being captured are stood in for)."""
import gc
import threading
import weakref

import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api

CPU = torch.device("cpu")


@pytest.fixture
def stream(monkeypatch):
    state = {"id": 7, "capturing": False}
    monkeypatch.setattr(api, "_raw_stream", lambda device: state["id"])
    monkeypatch.setattr(api, "_capturing", lambda: state["capturing"])
    api.release_workspaces()
    yield state
    api.release_workspaces()


def test_kept_by_stream_and_grown(stream):
    a, n = api._workspace_of(1000, CPU)
    assert n >= 1000 and not a.any()
    assert api._workspace_of(500, CPU)[0] is a
    stream["id"] = 8
    assert api._workspace_of(500, CPU)[0] is not a
    stream["id"] = 7
    b, n = api._workspace_of(5000, CPU)
    assert b is not a and n >= 5000 and api._workspace_of(1000, CPU)[0] is b
    api.release_workspaces()
    assert api._workspace_of(1000, CPU)[0] is not b


def test_threads_on_one_stream_do_not_share(stream):
    got, hold = {}, threading.Barrier(2)

    def run(i):
        got[i] = api._workspace_of(1000, CPU)[0]
        hold.wait()
        assert api._workspace_of(1000, CPU)[0] is got[i]
        hold.wait()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    mine = api._workspace_of(1000, CPU)[0]
    assert len({x.data_ptr() for x in (*got.values(), mine)}) == 3
    ended = [weakref.ref(x) for x in got.values()]
    got.clear()
    del threads, t
    gc.collect()
    assert all(x() is None for x in ended)  # a thread's workspaces go with it
    assert api._workspace_of(1000, CPU)[0] is mine


def test_release_reaches_every_thread(stream):
    step, seen = threading.Barrier(2), []

    def run():
        seen.append(api._workspace_of(1000, CPU)[0])
        step.wait()
        step.wait()
        seen.append(api._workspace_of(1000, CPU)[0])

    t = threading.Thread(target=run)
    t.start()
    step.wait()
    api.release_workspaces()
    step.wait()
    t.join()
    assert seen[0] is not seen[1]


def test_calls_without_scratch_share_what_nobody_touches(stream):
    a, n = api._workspace_of(256, CPU, None, True)
    assert n == 256 and a.numel() >= 256 and api._workspace_of(256, CPU, None, True)[0] is a
    assert api._workspace_of(256, CPU)[0] is not a  # a header in use is the stream's own


@pytest.mark.parametrize("args", [(), (None, True)])
def test_a_captured_call_has_its_own(stream, args):
    before = api._workspace_of(1000, CPU)[0]
    kept = dict(api._thread.kept)
    stream["capturing"] = True
    a, n = api._workspace_of(1000, CPU, *args)
    b, _ = api._workspace_of(4000, CPU, *args)
    assert n >= 1000 and a.data_ptr() % 16 == 0
    assert len({x.data_ptr() for x in (before, a, b)}) == 3
    assert api._thread.kept.keys() == kept.keys() and all(api._thread.kept[k] is kept[k] for k in kept)
    if not args:
        assert not a.any()
    ws = torch.empty(4096 + 256, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:][:4096]
    assert api._workspace_of(1000, CPU, ws)[0] is ws  # the caller's, as ever
    stream["capturing"] = False
    assert api._workspace_of(1000, CPU)[0] is before
