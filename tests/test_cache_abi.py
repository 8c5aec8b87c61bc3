"""Host-side checks of the 4-bit cache and eviction entry points: bad arguments
return the documented status before any CUDA call, empty calls succeed,
workspaces are sized as documented, the binding refuses wrong tensors."""
import ctypes
import os
import re

import pytest
import torch

from sparse_mla_decode_partial_b200 import binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, MISALIGNED, SMALL = 0, 1, 2, 3, 4
FAKE = 0x10000000  # aligned, never dereferenced: every call fails its checks first
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def append(lib, rows=FAKE, n=4, cu=FAKE, start=FAKE, B=2, cache=FAKE, pages=8, pt=FAKE, stride=4, ps=64):
    return lib.smla_q4_append(rows, n, cu, start, B, cache, pages, pt, stride, ps, None)


def read(lib, cache=FAKE, pages=8, pt=FAKE, stride=4, positions=FAKE, B=2, K=3, ps=64, rows=FAKE):
    return lib.smla_q4_read(cache, pages, pt, stride, positions, B, K, ps, rows, None)


def sparse(lib, q=FAKE, cache=FAKE, pages=8, pt=FAKE, stride=4, idx=FAKE, B=1, T=1, H=16, K=64, ps=64, scale=0.1,
           S=2, ws=FAKE, wsb=BIG, o=FAKE, lse=FAKE):
    return lib.smla_decode_q4(q, cache, pages, pt, stride, idx, B, T, H, K, ps, scale, S, ws, wsb, o, lse, None)


def dense(lib, q=FAKE, cache=FAKE, pages=8, pt=FAKE, stride=4, lens=FAKE, B=1, T=1, H=16, K=256, ps=64, scale=0.1,
          S=2, ws=FAKE, wsb=BIG, o=FAKE, lse=FAKE):
    return lib.smla_decode_dense_q4(q, cache, pages, pt, stride, lens, B, T, H, K, ps, scale, S, ws, wsb, o, lse, None)


def weigh(lib, q=FAKE, cache=FAKE, pages=8, pt=FAKE, stride=4, lens=FAKE, lse=FAKE, B=1, T=1, H=16, ps=64, scale=0.1,
          acc=FAKE, max_n=100, name="smla_evict_accumulate"):
    return getattr(lib, name)(q, cache, pages, pt, stride, lens, lse, B, T, H, ps, scale, acc, max_n, None)


def plan(lib, acc=FAKE, pos=FAKE, n=FAKE, B=2, max_n=100, K=50, sink=4, recent=8, ws=FAKE, wsb=BIG, src=FAKE + 2048,
         n_new=FAKE + 4096, acc_new=FAKE + 8192, pos_new=FAKE + 16384):
    return lib.smla_evict_plan(acc, pos, n, B, max_n, K, sink, recent, ws, wsb, src, n_new, acc_new, pos_new, None)


def apply(lib, src=FAKE, B=2, K=50, pt=FAKE, stride=4, pages=8, ps=64, bufs=(FAKE,), rb=(416,), n=None):
    k = max(len(bufs), 1)
    return lib.smla_evict_apply(src, B, K, pt, stride, pages, ps, (ctypes.c_void_p * k)(*bufs),
                                (ctypes.c_int32 * k)(*rb), len(bufs) if n is None else n, None)


REFUSALS = [
    (append, dict(n=-1), INVALID), (append, dict(B=-1), INVALID), (append, dict(ps=32), UNSUPPORTED),
    (append, dict(n=0, ps=32), UNSUPPORTED), (append, dict(rows=None), INVALID), (append, dict(cu=None), INVALID),
    (append, dict(start=None), INVALID), (append, dict(cache=None), INVALID), (append, dict(pt=None), INVALID),
    (append, dict(pages=0), INVALID), (append, dict(stride=0), INVALID), (append, dict(pages=1 << 25), UNSUPPORTED),
    (append, dict(rows=FAKE + 8), MISALIGNED), (append, dict(cache=FAKE + 4), MISALIGNED),
    (append, dict(cu=FAKE + 2), MISALIGNED), (append, dict(start=FAKE + 1), MISALIGNED),
    (read, dict(B=-1), INVALID), (read, dict(K=-1), INVALID), (read, dict(ps=16), UNSUPPORTED),
    (read, dict(positions=None), INVALID), (read, dict(rows=None), INVALID), (read, dict(rows=FAKE + 2), MISALIGNED),
    (read, dict(positions=FAKE + 2), MISALIGNED), (read, dict(B=2**31 - 1, K=2**31 - 1), INVALID),
    (sparse, dict(H=65), UNSUPPORTED), (sparse, dict(B=-1), INVALID), (sparse, dict(K=-1), INVALID),
    (sparse, dict(scale=float("nan")), INVALID), (sparse, dict(S=-1), INVALID), (sparse, dict(S=1025), INVALID),
    (sparse, dict(K=2**30), INVALID), (sparse, dict(cache=None), INVALID), (sparse, dict(cache=FAKE + 8), MISALIGNED),
    (sparse, dict(q=FAKE + 2), MISALIGNED), (sparse, dict(o=None), INVALID), (sparse, dict(o=FAKE + 8), MISALIGNED),
    (sparse, dict(wsb=0), SMALL), (sparse, dict(ws=None), INVALID), (sparse, dict(ws=FAKE + 8), MISALIGNED),
    (sparse, dict(B=2**20, T=1024, H=1, S=8), INVALID), (sparse, dict(ps=128), UNSUPPORTED),
    (dense, dict(H=65), UNSUPPORTED), (dense, dict(lens=None), INVALID), (dense, dict(S=-1), INVALID),
    (dense, dict(scale=float("inf")), INVALID), (dense, dict(K=2**30), INVALID), (dense, dict(wsb=16), SMALL),
    (dense, dict(ws=None), INVALID), (dense, dict(ws=FAKE + 4), MISALIGNED), (dense, dict(lse=None), INVALID),
    (dense, dict(pages=0), INVALID), (dense, dict(ps=1), UNSUPPORTED),
    (weigh, dict(B=-1), INVALID), (weigh, dict(H=65), UNSUPPORTED), (weigh, dict(max_n=-1), INVALID),
    (weigh, dict(scale=float("inf")), INVALID), (weigh, dict(acc=None), INVALID), (weigh, dict(lse=None), INVALID),
    (weigh, dict(acc=FAKE + 2), MISALIGNED), (weigh, dict(q=FAKE + 8), MISALIGNED), (weigh, dict(ps=63), UNSUPPORTED),
    (weigh, dict(max_n=2**30), INVALID), (weigh, dict(B=2**20, T=2**10, H=2), INVALID), (weigh, dict(lens=None), INVALID),
    (plan, dict(B=-1), INVALID), (plan, dict(K=0), INVALID), (plan, dict(sink=-1), INVALID),
    (plan, dict(sink=40, recent=11), INVALID), (plan, dict(sink=2**31 - 1, recent=2**31 - 1), INVALID),
    (plan, dict(max_n=524289), UNSUPPORTED), (plan, dict(n=None), INVALID), (plan, dict(src=None), INVALID),
    (plan, dict(acc=None), INVALID), (plan, dict(n_new=None), INVALID), (plan, dict(wsb=799, pos_new=None), SMALL),
    (plan, dict(ws=None, pos_new=None), INVALID), (plan, dict(ws=FAKE + 4, pos_new=None), MISALIGNED), (plan, dict(acc_new=FAKE), INVALID),
    (plan, dict(acc_new=FAKE + 796), INVALID), (plan, dict(pos_new=FAKE), INVALID), (plan, dict(n_new=FAKE + 4), INVALID),
    (plan, dict(src=FAKE + 400), INVALID), (plan, dict(src=FAKE + 4096 - 4), INVALID), (plan, dict(acc_new=FAKE + 16384 + 796), INVALID),
    (plan, dict(pos=FAKE + 8192 + 796), INVALID), (plan, dict(n=FAKE + 4100), INVALID),
    (plan, dict(pos=FAKE + 2), MISALIGNED),
    (apply, dict(B=-1), INVALID), (apply, dict(src=None), INVALID), (apply, dict(src=FAKE + 1), MISALIGNED),
    (apply, dict(bufs=(FAKE,) * 5, rb=(16,) * 5), UNSUPPORTED), (apply, dict(rb=(24,)), MISALIGNED),
    (apply, dict(rb=(0,)), UNSUPPORTED), (apply, dict(rb=(65552,)), UNSUPPORTED), (apply, dict(bufs=(None,)), INVALID),
    (apply, dict(bufs=(FAKE + 8,)), MISALIGNED), (apply, dict(ps=32), UNSUPPORTED), (apply, dict(n=-1), INVALID),
    (apply, dict(pages=0), INVALID), (apply, dict(pt=None), INVALID),
]


@pytest.mark.parametrize("call,args,want", REFUSALS, ids=lambda v: v.__name__ if callable(v) else str(v))
def test_refusals(lib, call, args, want):
    assert call(lib, **args) == want
    if call is weigh:
        assert weigh(lib, name="smla_evict_accumulate_q4", **args) == want


@pytest.mark.parametrize("call,args", [
    (append, dict(n=0, rows=None)), (append, dict(B=0, cu=None)), (read, dict(K=0, rows=None)), (read, dict(B=0)),
    (sparse, dict(B=0, q=None)), (sparse, dict(H=0)), (dense, dict(T=0)), (weigh, dict(B=0)), (weigh, dict(max_n=0)),
    (plan, dict(B=0)), (apply, dict(K=0)), (apply, dict(bufs=(), n=0)),
])
def test_empty_calls_succeed_without_a_gpu(lib, call, args):
    assert call(lib, **args) == OK


def test_workspace_sizes_and_splits(lib):
    r = lambda x: (x + 255) // 256 * 256
    assert binding.evict_workspace_bytes(3, 1000) == r(3 * 1000 * 4)
    assert binding.evict_workspace_bytes(-1, 5) == 0
    assert binding.dense_q4_workspace_bytes(2, 1, 64, 4096, 1) == 0
    assert binding.dense_q4_workspace_bytes(2, 3, 8, 4096, 5) == binding.workspace_bytes(2, 3, 8, 5)
    for S in (1, 7):  # up to 16 query rows: pieces of (splits + 1) per unit, their maxima, the tiles before each unit
        assert binding.dense_q4_workspace_bytes(3, 2, 8, 4096, S) == r(3 * (S + 1) * 16 * 2048) + r(3 * (S + 1) * 16 * 8) + r(16)
    assert binding.q4_workspace_bytes(2, 1, 16, 2048, 1) == 0
    assert binding.q4_workspace_bytes(2, 3, 8, 2048, 5) == binding.workspace_bytes(2, 3, 8, 5)
    for B, T, H in [(1, 1, 16), (3, 5, 8), (60, 1, 64)]:  # 0: the default's
        assert binding.q4_workspace_bytes(B, T, H, 2048) == binding.q4_workspace_bytes(B, T, H, 2048, binding.q4_nsplit(B, T, H, 2048))
        assert binding.dense_q4_workspace_bytes(B, T, H, 9000) == binding.dense_q4_workspace_bytes(
            B, T, H, 9000, binding.dense_q4_nsplit(B, T, H, 9000))
    assert [binding.q4_nsplit(b, 1, 16, 2048) for b in (1, 15, 64, 1000)] == [32, 16, 4, 1]  # on 148 SMs
    for B, T, H, K in [(1, 1, 16, 2048), (64, 1, 16, 2048), (60, 1, 64, 2048), (3, 5, 8, 1999)]:
        assert 1 <= binding.q4_nsplit(B, T, H, K) <= 1024
        assert 1 <= binding.dense_q4_nsplit(B, T, H, 20 * K) <= 1024
    assert binding.q4_nsplit(1, 1, 16, 0) == 1 and binding.dense_q4_nsplit(0, 1, 16, 10) == 1


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "smla.h")).read()
    want = {name: int(v) for name, v in re.findall(r"#define (SMLA_\w+) (\d+)", text)}
    assert want["SMLA_Q4_ROW_BYTES"] == binding.Q4_ROW_BYTES == 416
    assert want["SMLA_EVICT_MAX_N"] == binding.EVICT_MAX_N
    assert want["SMLA_EVICT_MAX_CACHES"] == binding.EVICT_MAX_CACHES
    assert want["SMLA_EVICT_MAX_ROW_BYTES"] == binding.EVICT_MAX_ROW_BYTES


def test_binding_refuses_wrong_tensors():
    """Type and place are checked before anything is launched (CPU tensors never reach the library)."""
    rows, cache = torch.zeros(2, 576, dtype=torch.bfloat16), torch.zeros(1, 64, 416, dtype=torch.uint8)
    table, i32 = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.q4_append(rows, cache, table, torch.zeros(2, dtype=torch.int32), i32)
    with pytest.raises(TypeError):
        binding.q4_append(rows.float(), cache, table, torch.zeros(2, dtype=torch.int32), i32)
    with pytest.raises(TypeError):
        binding.q4_read(cache.float(), table, table)
    with pytest.raises(ValueError):
        binding.q4_read(cache[:, ::2], table, table)
    with pytest.raises(TypeError):
        binding.decode_q4(rows.float(), cache, table, table, 1.0)
    with pytest.raises(ValueError):
        binding.decode_dense_q4(rows.view(1, 1, 2, 576), cache, table, table, 1.0)
    with pytest.raises(TypeError):
        binding.evict_accumulate(rows.float(), cache, table, table, table, 1.0, table)
    with pytest.raises(TypeError):
        binding.evict_plan(table, i32, 4)
    with pytest.raises(TypeError):
        binding.evict_apply(table.long(), table, (cache,))


@pytest.mark.parametrize("at", [FAKE, FAKE + 2048 + 384, FAKE + 4096, FAKE + 8192 + 784, FAKE + 32768 - 768, FAKE + 65536 - 1008])
def test_plan_refuses_a_workspace_that_overlaps(lib, at):
    """acc (also pos), src, n_new, acc_new, pos and n, each in its first or last bytes; unused, it may lie anywhere."""
    args = dict(ws=at, pos=FAKE + 32768, n=FAKE + 65536)
    assert plan(lib, pos_new=None, **args) == INVALID
