"""What a call allocates belongs to the stream that it is given: memory of the current stream, whose work may
still be under way, or that the current stream may hand out again, plays no part."""
import math

import numpy as np
import pytest
import torch

import mla_paged_decode_03_gb300 as M

pytestmark = pytest.mark.gpu

DEV = "cuda"
BUSY = 100_000_000                                   # clocks, some 50 ms


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def decode_inputs():
    g = torch.Generator().manual_seed(3)
    q = torch.randn(1, 1, 16, 576, generator=g).to(torch.bfloat16).to(DEV)
    cache = torch.randn(300, 16, 576, generator=g).to(torch.bfloat16).to(DEV)
    table = torch.randperm(300, generator=g).to(torch.int32).view(1, 300).to(DEV)
    lens = i32([4700])
    return q, cache, table, lens


def merge_call():
    g = torch.Generator().manual_seed(4)
    parts = torch.randn(3, 4096, 16, 128, generator=g).to(torch.bfloat16).to(DEV)
    lses = torch.randn(3, 4096, 16, generator=g).to(DEV)
    return (4096, 16, 128), lambda stream: M.lse_merge(parts, lses, stream=stream)[0]


def merge_call_512():
    g = torch.Generator().manual_seed(5)
    parts = torch.randn(3, 1024, 16, 512, generator=g).to(torch.bfloat16).to(DEV)
    lses = torch.randn(3, 1024, 16, generator=g).to(DEV)
    return (1024, 16, 512), lambda stream: M.lse_merge(parts, lses, stream=stream)[0]


def decode_call():
    q, cache, table, lens = decode_inputs()
    return (1, 16, 512), lambda stream: M.mla_decode(q, cache, table, lens, None, 1, 1, 0, 1 / math.sqrt(192), stream=stream)[0]


def shards_call():
    q, cache, table, lens = decode_inputs()
    t2, local, total = table.view(2, 150).contiguous(), i32([2300, 2300]), i32([4600])
    return (2, 1, 16, 512), lambda stream: M.mla_decode_shards(q, cache, t2, local, total, 1, 2, 1 / math.sqrt(192), stream=stream)[0]


def slot_call():
    pos = torch.arange(40000, device=DEV).view(2, -1)
    table = torch.randperm(4000, device=DEV).to(torch.int32).view(2, -1)
    return (2, 20000), lambda stream: M.cp_local_slot(pos, table, 16, 2, 1, stream=stream)


@pytest.mark.parametrize("case", [merge_call, merge_call_512, decode_call, shards_call, slot_call])
def test_outputs_are_not_memory_that_the_current_stream_still_writes(case):
    shape, call = case()
    want = call(None).clone()
    side = torch.cuda.Stream()
    side.synchronize()
    torch.cuda.synchronize()
    t = torch.empty(shape, dtype=want.dtype, device=DEV)
    torch.cuda._sleep(BUSY)
    t.fill_(9)                                       # still to run when the other stream's call is done
    del t
    got = call(side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert M.device_status() == 0


@pytest.mark.parametrize("case", [decode_call, shards_call])
def test_workspace_is_not_handed_out_while_the_call_runs(case):
    _, call = case()
    want = call(None).clone()
    side = torch.cuda.Stream()
    size = M.alloc_workspace(2 if case is shards_call else 1, 16, 1).numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = call(side)
    mine = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert all((m == 7).all() for m in mine)
    assert torch.equal(got, want)
