"""The sticky device status: which word a query reads and a reset clears.

On the CPU the library's calls are stood in for by ones that keep their words
in host memory, so that a word can be set without a kernel.
"""
import contextlib
import ctypes

import pytest
import torch

import deltanet_sequence_mixing_b200 as m


class HostLib:
    """The status calls on host memory; a device's own word by its index."""

    def __init__(self):
        self.current, self.words = 1, {0: 0, 1: 0}

    def deltanet_workspace_init(self, ws, nbytes, stream):
        ctypes.memset(ws, 0, 256)
        return 0

    def deltanet_get_device_status(self, ws, stream):
        at = ws.value if isinstance(ws, ctypes.c_void_p) else ws
        return -5 if ctypes.c_uint.from_address(at).value else 0

    def deltanet_get_recurrence_status(self, stream):
        return -5 if self.words[self.current] else 0

    def deltanet_clear_recurrence_status(self, stream):
        self.words[self.current] = 0
        return 0


@pytest.fixture
def host(monkeypatch):
    """The binding on host memory, device 1 of two current."""
    lib, empty = HostLib(), torch.empty

    @contextlib.contextmanager
    def device(d):
        before, lib.current = lib.current, d.index
        yield
        lib.current = before

    monkeypatch.setattr(m, "lib", lambda: lib)
    monkeypatch.setattr(m, "_workspaces", {})
    monkeypatch.setattr(m, "_stream_workspaces", {})
    monkeypatch.setattr(m, "_scratch_devices", set(), raising=False)
    monkeypatch.setattr(m, "_stream", lambda device: None)
    monkeypatch.setattr(m, "_current_raw_stream", lambda index: 7)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", device)
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
    plain = m.workspace_for("cuda:1")
    give_up(plain)
    assert m.deltanet_get_device_status() == m._lib.DN_ERR_DEVICE_TIMEOUT
    m.reset_device_status()
    assert m.deltanet_get_device_status() == 0
    host.words[0] = host.words[1] = 1
    assert m.deltanet_get_device_status() == m._lib.DN_ERR_DEVICE_TIMEOUT
    m.reset_device_status(workspace=plain)  # a workspace's reset is its own
    assert m.deltanet_get_device_status(workspace=plain) == 0
    assert m.deltanet_get_device_status() == m._lib.DN_ERR_DEVICE_TIMEOUT
    m.reset_device_status("cuda:1")
    assert m.deltanet_get_device_status() == 0
    assert m.deltanet_get_device_status("cuda:0") == m._lib.DN_ERR_DEVICE_TIMEOUT


def test_the_query_waits_for_other_streams_only_where_they_have_scratch(host, monkeypatch):
    """Waiting for the whole device would end another thread's graph capture."""
    waited = []
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: waited.append(torch.device(device).index))
    m._own_workspace(torch.device("cuda", 0), 4096)
    m.deltanet_get_device_status("cuda:1")
    m.reset_device_status("cuda:1")
    assert waited == []
    m._own_workspace(torch.device("cuda", 1), m._KEEP_BYTES + 1)
    m.deltanet_get_device_status()
    m.reset_device_status()
    assert waited == [1, 1]


def test_a_larger_workspace_keeps_the_status(host):
    give_up(m.workspace_for("cuda:1"))
    ws = m.workspace_for("cuda:1", 4096)
    assert ws.numel() == 4096 and m.deltanet_get_device_status() == m._lib.DN_ERR_DEVICE_TIMEOUT
    m.reset_device_status()
    assert m.workspace_for("cuda:1", 8192).numel() == 8192 and m.deltanet_get_device_status() == 0


def test_wait_selftest_refusals():
    from deltanet_sequence_mixing_b200 import _lib as E
    from deltanet_sequence_mixing_b200.build import build

    build()
    call = lambda ws=1 << 32, nb=256, polls=10: E.lib().deltanet_selftest_wait_polls(ws, nb, polls, None)
    assert call(ws=None) == E.DN_ERR_WORKSPACE
    assert call(nb=255) == E.DN_ERR_WORKSPACE
    for polls in (0, -1, 10001):
        assert call(polls=polls) == E.DN_ERR_INVALID_ARG


# ----------------------------------------------------------------- on the GPU --
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def dn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.lib()
    return m


@gpu
@pytest.mark.parametrize("polls", [1, 20])
def test_a_counted_wait_runs_out(dn, polls):
    """The recurrence's wait ends in a status that the host reads, and calls with
    the same workspace work again after a reset."""
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    assert dn.deltanet_selftest_wait_polls(polls, ws) == 0
    assert dn.deltanet_get_device_status(workspace=ws) == dn._lib.DN_ERR_DEVICE_TIMEOUT
    dn.reset_device_status()
    dn.reset_device_status(workspace=ws)
    assert dn.deltanet_get_device_status(workspace=ws) == 0
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(1, 2, 200, 64, generator=g, device="cuda").bfloat16() for _ in range(3))
    o, S = dn.gated_linear_attn_fwd(q, k, v, workspace=ws)
    want = dn.gated_linear_attn_fwd(q, k, v)
    assert torch.equal(o, want[0]) and torch.equal(S, want[1])
    assert dn.deltanet_get_device_status(workspace=ws) == 0 and dn.deltanet_get_device_status() == 0


@gpu
@pytest.mark.parametrize("kind", ["no scratch", "kept", "replaced", "large", "captured"])
def test_a_timeout_outlives_the_scratch(dn, kind):
    """A wait that runs out in any workspace that a call can be given is reported
    by the query without arguments, after the workspace is gone; a reset clears it."""
    dev = torch.device("cuda", torch.cuda.current_device())
    late = dn._lib.DN_ERR_DEVICE_TIMEOUT
    dn.reset_device_status()
    run = lambda nbytes: dn.deltanet_selftest_wait_polls(5, dn._own_workspace(dev, nbytes))
    if kind == "captured":
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            assert run(4096) == 0
        assert dn.deltanet_get_device_status() == 0
        g.replay()
    else:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            assert run({"no scratch": 256, "large": dn._KEEP_BYTES + 256}.get(kind, 4096)) == 0
            if kind == "replaced":
                dn._own_workspace(dev, 1 << 20)
        del s
    assert dn.deltanet_get_device_status() == late
    assert dn.deltanet_get_device_status() == late  # sticky
    dn.reset_device_status()
    assert dn.deltanet_get_device_status() == 0
    if kind == "captured":
        g.replay()
        assert dn.deltanet_get_device_status() == late
        dn.reset_device_status()


@gpu
def test_calls_leave_the_status_clear(dn):
    """Scratch of every kind, eager and captured."""
    dn.reset_device_status()
    gen = torch.Generator(device="cuda").manual_seed(2)
    for B, H, T in ((1, 2, 100), (1, 1, 3000), (2, 20, 2000)):
        q, k, v, dO = (torch.randn(B, H, T, 128, generator=gen, device="cuda").bfloat16() for _ in range(4))
        call = lambda: (dn.gated_linear_attn_fwd(q, k, v), dn.gated_linear_attn_bwd(q, k, v, dO))
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        g.replay()
    assert dn.deltanet_get_device_status() == 0
