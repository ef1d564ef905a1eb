"""Memory of outputs and scratch that a call on another stream allocates: it
belongs to the stream that writes it, so nothing that is still queued on the
current stream uses it, and it is not given away before the current stream has
read it."""

import contextlib

import pytest
import torch

import moe_expert_layer_ep_gb300 as M

# ------------------------------------------------------------------ on the CPU, with streams that only have a name


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream


class Block:
    device = "cpu"

    def __init__(self, stream):
        self.stream, self.used_on = stream, []

    def record_stream(self, s):
        self.used_on.append(s.cuda_stream)


@pytest.fixture
def allocator(monkeypatch):
    now = [Stream(1)]

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch, "empty", lambda *a, **k: Block(now[-1].cuda_stream))


@pytest.mark.parametrize("handle,owner", [(None, 1), (1, 1), (2, 2)])
def test_memory_comes_from_the_pool_of_the_stream_that_writes_it(allocator, handle, owner):
    b = M._empty((4,), torch.float32, Block(1), None if handle is None else Stream(handle))
    assert b.stream == owner
    assert b.used_on == ([] if owner == 1 else [1])


def test_a_stream_given_by_its_handle(allocator):
    b = M._empty((4,), torch.float32, Block(1), 7)
    assert b.stream == 7 and b.used_on == [1]


# ------------------------------------------------------------------ on the GPU
T, K, I, E = 256, 256, 128, 2   # every expert's 128 rows carry a token


def _randn(*shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(sum(shape))).to(torch.bfloat16).cuda()


def _calls():
    """Calls that allocate all their outputs, by name."""
    ids = (torch.arange(T, dtype=torch.int32, device="cuda") % E).view(T, 1)
    src2dst, start, counts = M.moe_sort_plan(ids, E)
    w = torch.rand((T, 1), device="cuda")
    at = (start, counts, torch.zeros(4, dtype=torch.int32, device="cuda"))
    x, xi, gu = _randn(T, K), _randn(T, I), _randn(T, 2 * I)
    w13, w2 = _randn(E, 2 * I, K), _randn(E, K, I)
    planes = M.moe_router_prepare(torch.randn((E, K), device="cuda"))
    w32 = torch.randn((E, K), device="cuda")
    codes = torch.zeros((E, 128, 128), dtype=torch.uint8, device="cuda")
    scales = torch.ones((E, 1, 1), device="cuda")
    sf = torch.randint(100, 140, (E, 128, 4), device="cuda").to(torch.uint8)
    torch.cuda.synchronize()
    return {
        "plan": lambda s: M.moe_sort_plan(ids, E, stream=s),
        "sort": lambda s: M.moe_sort_tokens(x, src2dst, rows=T, stream=s),
        "unsort": lambda s: M.moe_unsort_tokens(x, src2dst, w, stream=s),
        "unsort_backward": lambda s: M.moe_unsort_tokens_backward(x, x, src2dst, w, stream=s),
        "gemm": lambda s: M.moe_expert_gemm(x, w13, *at, stream=s),
        "swiglu": lambda s: M.moe_expert_gemm_swiglu(x, w13, *at, stream=s),
        "dgrad": lambda s: M.moe_expert_gemm_dgrad(x, w2, *at, stream=s),
        "dgrad_swiglu": lambda s: M.moe_expert_gemm_dgrad_swiglu(x, w2, gu, *at, stream=s),
        "wgrad": lambda s: M.moe_expert_gemm_wgrad(x, xi, *at, stream=s),
        "route": lambda s: M.moe_route(x, planes, 1, stream=s),
        "router_prepare": lambda s: M.moe_router_prepare(w32, stream=s),
        "requant": lambda s: M.moe_requant_weights_ue8m0(codes, scales, stream=s),
        "pack_mx_scales": lambda s: M.moe_pack_mx_scales(sf, stream=s),
    }


NAMES = ("plan", "sort", "unsort", "unsort_backward", "gemm", "swiglu", "dgrad", "dgrad_swiglu", "wgrad", "route",
         "router_prepare", "requant", "pack_mx_scales")


def _outs(r):
    return list(r) if isinstance(r, tuple) else [r]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_a_call_on_another_stream_leaves_alone_what_is_queued(name):
    call = _calls()[name]
    want = [t.clone() for t in _outs(call(None))]
    side = torch.cuda.Stream()
    call(side)   # (its first use may set up what later ones find)
    torch.cuda.synchronize()
    old = [torch.full(t.shape, 3, dtype=t.dtype, device="cuda") for t in want for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)   # some 50 ms
    kept = [t.clone() for t in old]
    del old                          # free blocks of the current stream, which still has to read them
    got = _outs(call(side))
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for t in kept:
        assert torch.all(t == 3)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_outputs_of_another_stream_are_kept_until_they_were_read(name):
    call = _calls()[name]
    want = [t.clone() for t in _outs(call(None))]
    side = torch.cuda.Stream()
    got = _outs(call(side))
    side.synchronize()
    torch.cuda._sleep(100_000_000)
    read = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):    # what takes their memory now, does it write before they were read?
        new = [torch.full(t.shape, 5, dtype=t.dtype, device="cuda") for t in want for _ in range(3)]
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(read, want):
        assert torch.equal(a, b)
    assert len(new) == 3 * len(want)
