"""Tensors on another device than the current one (CPU: the runtime's answers
are stood in for): a launch would go to the current device's default stream, so
the call is refused before one."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api


@pytest.fixture
def current(monkeypatch):
    state = {"device": 0}
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["device"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0 if index == 0 else 100 + index, raising=False)
    return state


def test_the_current_device_is_the_tensors(current):
    assert api._raw_stream(torch.device("cuda", 0)) == 0
    with pytest.raises(api.PararnnError, match="cuda:1.*cuda:0"):
        api._raw_stream(torch.device("cuda", 1))
    current["device"] = 1
    assert api._raw_stream(torch.device("cuda", 1)) == 101
    with pytest.raises(api.PararnnError):
        api._raw_stream(torch.device("cuda", 0))


def test_no_workspace_is_kept_for_a_refused_call(current, monkeypatch):
    monkeypatch.setattr(api, "_capturing", lambda: False)
    api.release_workspaces()
    with pytest.raises(api.PararnnError):
        api._workspace_of(1000, torch.device("cuda", 2), None, True)
    assert not api._thread.kept
