"""Calls with a stream of their own: what the binding allocates for them belongs
to that stream, whatever the caller's current stream has still to do."""
import pytest
import torch

import cache_util as cu
from sparse_mla_decode_partial_b200 import binding
from test_gpu_q4 import SCALE, clean_device, fill, lists_for  # noqa: F401

pytestmark = pytest.mark.gpu


def tensors(out):
    return [out] if isinstance(out, torch.Tensor) else [t for t in out if t is not None]


def check_beside_pending_work(call, scratch_bytes=0):
    """``call(stream)`` on a side stream gives what it gives by itself while the
    current stream has still to write to memory that it has let go of: blocks of
    the sizes the call asks for, which the allocator hands out again to the current
    stream at once, and must not hand to the side stream."""
    want = [t.clone() for t in tensors(call(None))]
    sizes = [max(t.numel() * t.element_size(), 16) for t in want]
    side = torch.cuda.Stream()
    torch.cuda._sleep(1)  # (loading a kernel waits for what runs, so this is done before)
    torch.empty(16, dtype=torch.uint8, device="cuda").fill_(1)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    pending = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes + [max(scratch_bytes, 16)]]
    torch.cuda._sleep(100_000_000)  # some 50 ms
    for t in pending:
        t.fill_(1)
    del pending, t
    got = call(side)
    torch.cuda.synchronize()
    for a, b in zip(tensors(got), want):
        assert torch.equal(torch.nan_to_num(a.float(), nan=-7.0), torch.nan_to_num(b.float(), nan=-7.0))


def q4_inputs():
    lens = [900, 700]
    paged = cu.Paged(lens, 2)
    cache, _ = fill(paged, lens, 3)
    return paged.cuda, cache, torch.from_numpy(lists_for(lens, 1, 300, 1)).cuda(), cu.queries(2, 1, 16, 4).cuda()


@pytest.mark.parametrize("nsplit", [1, 4])
def test_decode_q4(nsplit):
    table, cache, idx, q = q4_inputs()
    check_beside_pending_work(lambda s: binding.decode_q4(q, cache, table, idx, SCALE, nsplit, stream=s),
                              binding.q4_workspace_bytes(2, 1, 16, 300, nsplit))


@pytest.mark.parametrize("H", [16, 40])
def test_decode_dense_q4(H):
    table, cache, _, _ = q4_inputs()
    q, lens = cu.queries(2, 1, H, 4).cuda(), torch.tensor([[900], [700]], dtype=torch.int32).cuda()
    check_beside_pending_work(lambda s: binding.decode_dense_q4(q, cache, table, lens, SCALE, K=900, stream=s),
                              binding.dense_q4_workspace_bytes(2, 1, H, 900))


def test_q4_read():
    table, cache, idx, _ = q4_inputs()
    check_beside_pending_work(lambda s: binding.q4_read(cache, table, idx[:, 0].contiguous(), stream=s))


def test_evict_plan():
    acc = torch.rand(3, 900, generator=torch.Generator().manual_seed(1)).cuda()
    n = torch.tensor([900, 500, 20], dtype=torch.int32).cuda()
    check_beside_pending_work(lambda s: binding.evict_plan(acc, n, 300, stream=s))


def bf16_inputs():
    lens = [900, 700]
    paged = cu.Paged(lens, 2)
    cache = cu.latents(paged.pages * 64, 3).view(paged.pages, 64, 576).cuda()
    return paged.cuda, cache, torch.from_numpy(lists_for(lens, 1, 300, 1)).cuda(), cu.queries(2, 1, 16, 4).cuda()


@pytest.mark.parametrize("nsplit", [1, 4])
def test_decode(nsplit):
    table, cache, idx, q = bf16_inputs()
    check_beside_pending_work(lambda s: binding.decode(q, cache, table, idx, SCALE, nsplit, stream=s),
                              binding.workspace_bytes(2, 1, 16, nsplit))


def test_decode_partial_and_combine():
    table, cache, idx, q = bf16_inputs()
    call = lambda s: binding.decode_partial(q, cache, table, idx, SCALE, 4, stream=s)
    check_beside_pending_work(call)
    parts = call(None)
    check_beside_pending_work(lambda s: binding.lse_combine(*parts, stream=s))


def test_decode_dense():
    table, cache, _, q = bf16_inputs()
    lens = torch.tensor([[900], [700]], dtype=torch.int32).cuda()
    check_beside_pending_work(lambda s: binding.decode_dense(q, cache, table, lens, SCALE, 4, K=900, stream=s),
                              binding.dense_workspace_bytes(2, 1, 16, 900, 4))
    check_beside_pending_work(lambda s: binding.decode_dense_partial(q, cache, table, lens, SCALE, 4, K=900, stream=s))


def test_decode_host():
    table, cache, idx, q = [t.cpu().pin_memory() if t.dtype != torch.bfloat16 or t.dim() == 4 else t for t in bf16_inputs()]
    o, lse = torch.zeros(2, 1, 16, 512, dtype=torch.bfloat16).pin_memory(), torch.zeros(2, 1, 16).pin_memory()

    def call(s):
        binding.decode_host(q, cache, table, idx, SCALE, 4, o=o, lse=lse, stream=s)
        torch.cuda.synchronize() if s is None else s.synchronize()
        return o, lse

    check_beside_pending_work(call, binding.workspace_host_bytes(2, 1, 16, 300, table.shape[1], 4))


def test_indexer():
    table = bf16_inputs()[0]
    g = torch.Generator().manual_seed(5)
    keys = torch.randn(int(table.max()) + 1, 64, 128, generator=g).to(torch.bfloat16).cuda()
    q, w = torch.randn(2, 1, 8, 128, generator=g).to(torch.bfloat16).cuda(), torch.rand(2, 1, 8, generator=g).cuda()
    n = torch.tensor([[900], [700]], dtype=torch.int32).cuda()
    check_beside_pending_work(lambda s: binding.indexer_topk(q, w, keys, table, n, 128, 900, stream=s),
                              binding.indexer_workspace_bytes(2, 1, 900))
    check_beside_pending_work(lambda s: binding.indexer_scores(q, w, keys, table, n, 900, stream=s),
                              binding.indexer_workspace_bytes(2, 1, 0))
    scores = binding.indexer_scores(q, w, keys, table, n, 900)
    check_beside_pending_work(lambda s: binding.indexer_select(scores, n, 128, stream=s),
                              binding.indexer_select_workspace_bytes(2, 1, 900))


def test_the_default_stream_given_as_zero():
    table, cache, idx, q = bf16_inputs()
    want, got = (binding.decode(q, cache, table, idx, SCALE, 4, stream=s) for s in (None, 0))
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_a_stream_given_by_its_handle():
    table, cache, idx, q = q4_inputs()
    check_beside_pending_work(lambda s: binding.decode_q4(q, cache, table, idx, SCALE, 1,
                                                          stream=None if s is None else s.cuda_stream))


def test_outputs_that_the_caller_still_reads_stay_theirs():
    """An output dropped while the current stream has still to read it is not
    handed to the next call on the side stream."""
    table, cache, idx, q = q4_inputs()
    want = binding.decode_q4(q, cache, table, idx, SCALE, 1)[0].clone()
    other = -q
    side = torch.cuda.Stream()
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    o, _ = binding.decode_q4(q, cache, table, idx, SCALE, 1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(100_000_000)
    kept = o.clone()  # reads o when the current stream gets there
    del o
    binding.decode_q4(other, cache, table, idx, SCALE, 1, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


@pytest.mark.parametrize("H", [16, 40])
@pytest.mark.parametrize("q4", [False, True])
def test_lengths_that_the_side_stream_has_still_to_write(q4, H):
    """Without K the bound is read from the lengths as they stand on the call's stream."""
    table, cache = (q4_inputs() if q4 else bf16_inputs())[:2]
    decode = binding.decode_dense_q4 if q4 else binding.decode_dense
    q, lens = cu.queries(2, 1, H, 4).cuda(), torch.tensor([[900], [700]], dtype=torch.int32).cuda()
    want = decode(q, cache, table, lens, SCALE, 4)
    late, side = torch.ones_like(lens), torch.cuda.Stream()
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        late.copy_(lens)
    got = decode(q, cache, table, late, SCALE, 4, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
