"""Memory that the prefill calls take for themselves when the caller gives
none: which stream's pool it comes from.  CPU only: the allocations and the
library are stood in for."""

import types

import pytest
import torch

from paged_kv_cache_124_gb300 import api


class Handle:
    """A stream object of another library: its handle alone."""

    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


@pytest.fixture
def taken(monkeypatch):
    """What was allocated, and on which stream; `current`: the stack of current streams."""
    log = types.SimpleNamespace(current=["current"], took=[], called=[], captured=[])

    class use:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            log.current.append(self.stream)

        def __exit__(self, *_):
            log.current.pop()

    def took(what):
        def take(*a, **k):
            log.took.append((what, log.current[-1]))
            return torch.empty(16, dtype=torch.uint8) if what == "workspace" else torch.empty(2, dtype=torch.int32)
        return take

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Handle(77))
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: log.current[-1] in log.captured)
    monkeypatch.setattr(api, "prefill_workspace", took("workspace"))
    monkeypatch.setattr(api, "prefill_fp8_workspace", took("workspace"))
    monkeypatch.setattr(api, "_prefill_counters", {})
    monkeypatch.setattr(torch, "zeros", took("counters"))
    monkeypatch.setattr(api, "_dev", lambda t, dtype, name: t)
    monkeypatch.setattr(api, "_opt_dev", lambda t, dtype, name: t)
    call = lambda *a: log.called.append(a[-1].value or 0) or api.PA_OK  # noqa: E731
    monkeypatch.setattr(api, "_lib", types.SimpleNamespace(pa_prefill=call, pa_prefill_fp8=call))
    return log


def prefill(fp8, **kw):
    q, cache = torch.empty(3, 4, 64, dtype=torch.bfloat16), torch.empty(2, 2, 16, 64)
    tables, start, ctx = torch.empty(1, 2), torch.empty(2), torch.empty(1)
    if fp8:
        return api.pa_prefill_fp8(q, q, cache, cache, tables, start, ctx, 3, 16, 0.125, 1.0, 1.0, 4, 2, 64, **kw)
    return api.pa_prefill(q, q, cache, cache, tables, start, ctx, 3, 16, 0.125, 4, 2, 64, **kw)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("given,used", [(None, "current"), (0x5000, 0x5000), (Handle(0x6000), 0x6000), (0, "default"),
                                        (1, "default")])
def test_workspace_and_counters_come_from_the_pool_of_the_calls_stream(taken, fp8, given, used):
    """Else the call could write memory that the other stream still uses, or start before its counters are zeroed."""
    assert prefill(fp8, stream=given) == api.PA_OK
    assert sorted(taken.took) == [("counters", used), ("workspace", used)]
    assert taken.called == [77 if given is None else getattr(given, "cuda_stream", given)]
    assert taken.current == ["current"]


def test_the_per_thread_stream_takes_the_callers_memory(taken):
    """One handle for a stream of every thread: no pool is ordered with it."""
    with pytest.raises(ValueError, match="per-thread"):
        prefill(False, stream=2)
    with pytest.raises(ValueError, match="per-thread"):
        prefill(False, stream=2, counters=False)
    assert prefill(False, stream=2, counters=False, workspace=torch.empty(16)) == api.PA_OK


@pytest.mark.parametrize("given,used", [(None, "current"), (0x5000, 0x5000)])
def test_a_captured_call_has_counters_of_its_own(taken, given, used):
    """Those of the stream's calls would be zeroed in the graph alone, or shared by graphs that are replayed at once."""
    count = lambda: [s for what, s in taken.took if what == "counters"]  # noqa: E731
    taken.captured.append(used)
    prefill(False, stream=given)
    prefill(False, stream=given)
    assert count() == [used, used]
    taken.captured.clear()
    for _ in range(2):
        prefill(False, stream=given)
        assert count() == [used] * 3                     # then one pair for the stream, kept
    taken.captured.append(used)
    prefill(False, stream=given)
    assert count() == [used] * 4
