"""Calls given a stream allocate their results and workspaces in that stream's
pool and record the results on the caller's stream (no GPU needed: torch's
streams and the library are stood in for)."""
import contextlib
import types

import pytest
import torch

api = pytest.importorskip("combine_moe_dispatch_amd.api",
                          reason="libmoe_dispatch.so not built")

T, E, K = 20000, 64, 4


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream


class Cuda(torch.Tensor):
    """A CPU tensor that says it is on cuda:0."""
    device = torch.device("cuda", 0)


@pytest.fixture
def seen(monkeypatch):
    """What was allocated under which stream, recorded on which, launched on which."""
    log = types.SimpleNamespace(current=7, made=[], recorded=[], launched=[], pointers=[])

    @contextlib.contextmanager
    def on(s):
        before, log.current = log.current, s.cuda_stream
        yield
        log.current = before

    empty = torch.empty

    def make(*size, dtype=None, device=None):
        t = empty(*size, dtype=dtype).as_subclass(Cuda)
        log.made.append((t, log.current))
        return t

    def call(*args):
        log.launched.append(args[-1])
        log.pointers.append(args)
        return 0

    monkeypatch.setattr(torch, "empty", make)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(log.current))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(Cuda, "record_stream",
                        lambda t, s: log.recorded.append((t, s.cuda_stream)), raising=False)
    monkeypatch.setattr(api, "_raw_stream", lambda d: log.current)
    monkeypatch.setattr(api, "_all", lambda *a: 0)
    monkeypatch.setattr(api, "_gpu", lambda *a, **k: None)
    lib = api._lib
    monkeypatch.setattr(api, "_lib", types.SimpleNamespace(
        moe_balance_loss=call, moe_route_backward=call, moe_route_topk=call,
        moe_route_topk_grouped=call,
        moe_balance_loss_workspace_size=lib.moe_balance_loss_workspace_size,
        moe_route_backward_workspace_size=lib.moe_route_backward_workspace_size))
    return log


def cuda(t):
    return t.as_subclass(Cuda)


def balance(stream):
    return api.moe_balance_loss(cuda(torch.zeros(T, E)), None,
                                cuda(torch.zeros(T, K, dtype=torch.int32)), 0, 0.1, stream=stream)


def route_backward(stream):
    return api.moe_route_backward(cuda(torch.zeros(T, E)), None,
                                  cuda(torch.zeros(T, K, dtype=torch.int32)),
                                  cuda(torch.zeros(T, K)), cuda(torch.zeros(T, K)), 0,
                                  with_grad_bias=True, stream=stream)


def route(stream):
    return api.moe_route_topk(cuda(torch.zeros(T, E)), None, K, 0, stream=stream)


def route_grouped(stream):
    return api.moe_route_topk_grouped(cuda(torch.zeros(T, E)), None, K, 0, 8, 4, stream=stream)


@pytest.mark.parametrize("call,results,own", [(balance, 4, 5), (route_backward, 2, 3),
                                              (route, 2, 2), (route_grouped, 2, 2)])
@pytest.mark.parametrize("given", [lambda: Stream(9), lambda: 9])
def test_on_a_given_stream(seen, call, results, own, given):
    out = call(given())
    assert len(out) == results and len(seen.made) == own and seen.launched == [9]
    assert [s for _, s in seen.made] == [9] * own
    # every result, and it alone, is recorded on the stream of the caller
    assert all(s == 7 for _, s in seen.recorded)
    assert {id(t) for t, _ in seen.recorded} == {id(t) for t in out}
    # the library was given what was made there, the workspace among it
    assert {t.data_ptr() for t, _ in seen.made} <= set(seen.pointers[0])


@pytest.mark.parametrize("call,own", [(balance, 5), (route_backward, 3), (route, 2),
                                      (route_grouped, 2)])
def test_on_the_current_stream(seen, call, own):
    call(None)
    assert seen.launched == [7] and [s for _, s in seen.made] == [7] * own
    assert seen.recorded == []


@pytest.mark.parametrize("call", [balance, route_backward])
def test_a_stream_of_another_device_is_refused(seen, call):
    other = Stream(9)
    other.device_index = 1
    with pytest.raises(ValueError, match="stream is on cuda:1, tensors on cuda:0"):
        call(other)
    assert seen.launched == []
    other.device_index = 0
    call(other)
    assert seen.launched == [9]
