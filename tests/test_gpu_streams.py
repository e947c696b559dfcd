"""Calls given a stream while the current one still works on memory that was
freed there: results and workspaces must not share it."""
import pytest
import torch

from combine_moe_dispatch_amd import api

pytestmark = pytest.mark.gpu

T, E, K = 20000, 256, 8


@pytest.fixture(scope="module")
def routed():
    gen = torch.Generator().manual_seed(3)
    logits = torch.randn(T, E, generator=gen).cuda()
    ids, w = api.moe_route_topk(logits, None, K, 1)
    gw = torch.randn(T, K, generator=gen).cuda()
    _, counts, _, tokens = api.moe_balance_loss(logits, None, ids, 1, 0.1)
    return dict(logits=logits, ids=ids, w=w, gw=gw, counts=counts, tokens=tokens)


def balance(r, stream=None):
    return api.moe_balance_loss(r["logits"], None, r["ids"], 1, 0.1, stream=stream)


def route_backward(r, stream=None):
    return api.moe_route_backward(r["logits"], None, r["ids"], r["w"], r["gw"], 1, 0.1,
                                  expert_counts=r["counts"], seq_tokens=r["tokens"],
                                  with_grad_bias=True, stream=stream)


def route(r, stream=None):
    return api.moe_route_topk(r["logits"], None, K, 1, stream=stream)


def route_grouped(r, stream=None):
    return api.moe_route_topk_grouped(r["logits"], None, K, 1, 8, 4, stream=stream)


CALLS = [balance, route_backward, route, route_grouped]


def pending(sizes):
    """Queue a few milliseconds of products on the current stream, then writes to
    blocks of these sizes, and free them while all of it is pending."""
    x = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    for _ in range(10):
        torch.mm(x, x, out=y)
    for b in blocks:
        b.fill_(0x5A)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("as_handle", [False, True])
def test_blocks_freed_with_work_pending(routed, call, as_handle):
    want = call(routed)
    want_host = [t.cpu() for t in want]
    sizes = [t.numel() * t.element_size() for t in want]
    if call is balance:
        sizes.append(api.moe_balance_loss_workspace_size(T, E, 1))
    elif call is route_backward:
        sizes.append(api.moe_route_backward_workspace_size(T, E))
    st = torch.cuda.Stream()
    for _ in range(2):
        pending(sizes)
        got = call(routed, stream=st.cuda_stream if as_handle else st)
        torch.cuda.synchronize()
        for g, w in zip(got, want_host):
            assert torch.equal(g.cpu(), w)


@pytest.mark.parametrize("call", CALLS)
def test_dropped_results_are_not_reused_while_they_are_read(routed, call):
    want = [t.cpu() for t in call(routed)]
    st = torch.cuda.Stream()
    x = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    got = call(routed, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    for _ in range(10):
        torch.mm(x, x, out=y)
    copies = [t.clone() for t in got]    # reads behind the products
    del got
    with torch.cuda.stream(st):          # the pool the results came from
        again = [torch.full_like(t, 77) for t in copies for _ in range(2)]
    torch.cuda.synchronize()
    for c, w in zip(copies, want):
        assert torch.equal(c.cpu(), w)
    assert all((a == 77).all() for a in again)
