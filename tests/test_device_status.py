"""The sticky device status: which word a query reads and a reset clears.

On the CPU the library's calls are stood in for by ones that keep their words
in host memory, so that a word can be set without a kernel.
"""
import ctypes

import pytest
import torch

import deltanet_sequence_mixing_b200 as m


class HostLib:
    """The status calls on host memory."""

    def deltanet_workspace_init(self, ws, nbytes, stream):
        ctypes.memset(ws, 0, 256)
        return 0

    def deltanet_get_device_status(self, ws, stream):
        at = ws.value if isinstance(ws, ctypes.c_void_p) else ws
        return -5 if ctypes.c_uint.from_address(at).value else 0


@pytest.fixture
def host(monkeypatch):
    """The binding on host memory, device 1 of some current."""
    lib, empty = HostLib(), torch.empty
    monkeypatch.setattr(m, "lib", lambda: lib)
    monkeypatch.setattr(m, "_workspaces", {})
    monkeypatch.setattr(m, "_stream_workspaces", {})
    monkeypatch.setattr(m, "_stream", lambda device: None)
    monkeypatch.setattr(m, "_current_raw_stream", lambda index: 7)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return lib


def give_up(ws):
    ws[0] = 1


def test_a_device_has_one_word_whatever_it_is_called(host):
    ws = m.workspace_for(torch.device("cuda", 1))  # a tensor's device, as the calls pass it
    assert m.workspace_for("cuda") is ws and m.workspace_for("cuda:1") is ws
    assert m.workspace_for("cuda:0") is not ws
    give_up(ws)
    for device in (None, "cuda", "cuda:1", torch.device("cuda", 1)):
        assert m.deltanet_get_device_status(device) == m._lib.DN_ERR_DEVICE_TIMEOUT, device
    assert m.deltanet_get_device_status("cuda:0") == 0
    m.reset_device_status()
    assert m.deltanet_get_device_status("cuda:1") == 0


def test_reset_clears_all_that_the_query_reads(host):
    plain, kept = m.workspace_for("cuda:1"), m._own_workspace(torch.device("cuda", 1), 4096)
    other = m._own_workspace(torch.device("cuda", 0), 4096)
    for ws in (plain, kept):
        give_up(ws)
        assert m.deltanet_get_device_status() == m._lib.DN_ERR_DEVICE_TIMEOUT
        m.reset_device_status()
        assert m.deltanet_get_device_status() == 0
    give_up(other)
    m.reset_device_status("cuda:1")
    assert m.deltanet_get_device_status("cuda:0") == m._lib.DN_ERR_DEVICE_TIMEOUT
    mine = m._own_workspace(torch.device("cuda", 1), 4096)
    give_up(mine)
    m.reset_device_status(workspace=plain)  # a workspace's reset is its own
    assert m.deltanet_get_device_status() == m._lib.DN_ERR_DEVICE_TIMEOUT
