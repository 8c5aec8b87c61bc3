"""The 4-bit latent cache on the GPU: quantise-and-append, read back, sparse and
dense decode, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import cache_util as cu
from sparse_mla_decode_partial_b200 import binding

pytestmark = pytest.mark.gpu
SCALE = 1.0 / 24.0


@pytest.fixture(autouse=True)
def clean_device():
    binding.check_device(clear=True)
    yield
    assert binding.check_device(clear=True) == (0, 0)


def fill(paged, lens, seed, std=0.7):
    """A 4-bit cache of random rows (every row of the pool), as bytes on both sides."""
    rows = cu.latents(paged.pages * 64, seed, std)
    table = torch.arange(paged.pages, dtype=torch.int32)[None].cuda()
    cache = torch.zeros(paged.pages, 64, cu.ROW, dtype=torch.uint8, device="cuda")
    n = rows.shape[0]
    binding.q4_append(rows.cuda(), cache, table, torch.tensor([0, n], dtype=torch.int32).cuda(),
                      torch.zeros(1, dtype=torch.int32).cuda())
    return cache, cu.values(cache.cpu().numpy().reshape(n, cu.ROW))


# ---------------------------------------------------------------- append, read
@pytest.mark.parametrize("new,start", [
    ([0], [0]), ([1], [0]), ([1], [63]), ([65], [1]), ([3, 0, 70, 1], [60, 5, 0, 127]), ([0, 0, 2], [1, 2, 3]),
    ([1] * 17, list(range(17))), ([200, 1, 33], [0, 64, 95]),
])
def test_append_writes_the_definition(new, start):
    paged = cu.Paged([a + n for a, n in zip(start, new)], seed=len(new))
    n = sum(new)
    rows = cu.latents(n + 5, 11)               # five rows behind the last sequence
    cache = torch.full((paged.pages, 64, cu.ROW), 0xA5, dtype=torch.uint8, device="cuda")
    offs = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    got = binding.q4_append(rows.cuda(), cache, paged.cuda, offs, torch.tensor(start, dtype=torch.int32).cuda())
    assert got is cache
    want = np.full((paged.pages * 64, cu.ROW), 0xA5, np.uint8)
    at, q = 0, cu.quantise(rows[:n])
    for b, k in enumerate(new):
        for t in range(k):
            want[paged.row(b, start[b] + t)] = q[at]
            at += 1
    np.testing.assert_array_equal(cache.cpu().numpy().reshape(-1, cu.ROW), want)


def special_rows():
    rows = cu.latents(12, 3).float()
    rows[0, :] = 0.0
    rows[1, :512] = torch.tensor(float("inf"))
    rows[2, 40] = float("nan")
    rows[3, :512] *= 2.0 ** -121            # around the smallest stored magnitude
    rows[4, :512] *= 2.0 ** 118             # around the largest
    rows[5, :32] = torch.arange(32) - 16.0  # ties: half steps of a scale of 16 / 7 rounded up
    rows[6, :32] = torch.linspace(-7, 7, 32)
    rows[6, 0] = 7.0                        # 7 times a scale exactly
    rows[7, :32] = torch.tensor([7.0] + [k + 0.5 for k in range(-7, 7)] + [0.5] * 17)  # exact ties at scale 1
    rows[8, 512:] = float("inf")
    rows[9, 512:] = float("nan")
    rows[10, 100] = -2.0 ** 120
    rows[11, 100] = 2.0 ** 120 * (1 - 2.0 ** -8)
    return rows.to(torch.bfloat16)


def test_append_special_values():
    rows = special_rows()
    paged = cu.Paged([len(rows)])
    cache = torch.zeros(paged.pages, 64, cu.ROW, dtype=torch.uint8, device="cuda")
    binding.q4_append(rows.cuda(), cache, paged.cuda, torch.tensor([0, len(rows)], dtype=torch.int32).cuda(),
                      torch.zeros(1, dtype=torch.int32).cuda())
    got = cache.cpu().numpy().reshape(-1, cu.ROW)[paged.rows(0, range(len(rows)))]
    want = cu.quantise(rows)
    for r in range(len(rows)):
        np.testing.assert_array_equal(got[r], want[r], err_msg=f"row {r}")


def test_append_error_is_at_most_half_a_step():
    rows = cu.latents(300, 5, std=3.0)
    raw = cu.quantise(rows)
    x, v = cu.f64(rows), cu.values(raw)
    scale = cu.f64(torch.from_numpy(raw[:, 256:288].copy()).view(torch.bfloat16))
    assert (np.abs(x - v)[:, :512] <= np.repeat(scale, 32, 1) / 2).all()
    assert (x[:, 512:] == v[:, 512:]).all()


def test_append_and_read_many_rows():
    """Enough rows for four per warp, ragged, with rows behind the last sequence."""
    new, start = [9001, 0, 13003, 1], [7, 0, 60, 63]
    paged = cu.Paged([a + n for a, n in zip(start, new)], seed=1)
    n = sum(new)
    rows = cu.latents(n + 3, 12)
    cache = torch.zeros(paged.pages, 64, cu.ROW, dtype=torch.uint8, device="cuda")
    offs = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    binding.q4_append(rows.cuda(), cache, paged.cuda, offs, torch.tensor(start, dtype=torch.int32).cuda())
    lists = torch.full((4, max(new) + 1), -1, dtype=torch.int32)
    for b in range(4):
        lists[b, :new[b]] = torch.arange(start[b], start[b] + new[b]).flip(0).int()
    out = cu.f64(binding.q4_read(cache, paged.cuda, lists.cuda()))
    raw = cache.cpu().numpy().reshape(-1, cu.ROW)
    at = 0
    assert not out[1].any()
    for b in (0, 2, 3):
        mine = raw[paged.rows(b, range(start[b], start[b] + new[b]))]
        some = np.unique(np.linspace(0, new[b] - 1, 97).astype(int))
        np.testing.assert_array_equal(mine[some], cu.quantise(rows[at + torch.from_numpy(some)]))
        np.testing.assert_array_equal(out[b, :new[b]], cu.values(mine)[::-1])
        assert not out[b, new[b]:].any()
        at += new[b]
    used = np.concatenate([paged.rows(b, range(start[b], start[b] + new[b])) for b in range(4)])
    left = np.ones(len(raw), bool)
    left[used] = False
    assert not raw[left].any()


def test_append_counts_rows_it_cannot_place():
    paged = cu.Paged([64, 64, 64])
    paged.table[1, 0] = -1
    paged.table[2, 0] = paged.pages
    rows = cu.latents(8, 7)
    cache = torch.zeros(paged.pages, 64, cu.ROW, dtype=torch.uint8, device="cuda")
    # sequence 0: positions 62 .. 65 (two past the table), 1: no page, 2: bad page
    binding.q4_append(rows.cuda(), cache, paged.cuda, torch.tensor([0, 4, 6, 8], dtype=torch.int32).cuda(),
                      torch.tensor([62, 0, 0], dtype=torch.int32).cuda())
    assert binding.check_device(clear=True) == (5, 6)
    got = cache.cpu().numpy().reshape(-1, cu.ROW)
    at = paged.rows(0, [62, 63])
    np.testing.assert_array_equal(got[at], cu.quantise(rows[:2]))
    got[at] = 0
    assert not got.any()
    # negative start, and offsets that do not ascend: counted, nothing written
    cache.zero_()
    binding.q4_append(rows.cuda(), cache, paged.cuda[:2].contiguous(), torch.tensor([0, 5, 3], dtype=torch.int32).cuda(),
                      torch.tensor([-9, -9], dtype=torch.int32).cuda())
    st, bad = binding.check_device(clear=True)
    assert st == 5 and bad == 3 and not cache.any()


def test_append_then_read_on_another_stream_and_in_a_graph():
    paged = cu.Paged([70, 3])
    rows = cu.latents(73, 8).cuda()
    cache = torch.zeros(paged.pages, 64, cu.ROW, dtype=torch.uint8, device="cuda")
    offs, start = torch.tensor([0, 70, 73], dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    lists = torch.full((2, 71), -1, dtype=torch.int32)
    lists[0, :70] = torch.randperm(70, generator=torch.Generator().manual_seed(1)).int()
    lists[1, 68:] = torch.arange(3).int()
    lists = lists.cuda()
    table = paged.cuda
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    binding.q4_append(rows, cache, table, offs, start, stream=side)
    out = binding.q4_read(cache, table, lists, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = cu.values(cu.quantise(rows.cpu()))
    full = np.zeros((2, 71, 576))
    full[0, :70] = want[:70][lists[0, :70].cpu().numpy()]
    full[1, 68:] = want[70:]
    np.testing.assert_array_equal(cu.f64(out), full)
    graph, again = torch.cuda.CUDAGraph(), torch.empty_like(out)
    cache.zero_()
    with torch.cuda.graph(graph):
        binding.q4_append(rows, cache, table, offs, start)
        binding.q4_read(cache, table, lists, out=again)
    for _ in range(2):
        again.zero_()
        graph.replay()
        np.testing.assert_array_equal(cu.f64(again), full)


def test_read_bad_positions_are_zero_rows_and_counted():
    paged = cu.Paged([100])
    cache, vals = fill(paged, [100], 4)
    lists = torch.tensor([[0, -1, 128, -2, 99, 2**31 - 1]], dtype=torch.int32).cuda()
    out = cu.f64(binding.q4_read(cache, paged.cuda, lists))
    assert binding.check_device(clear=True) == (5, 3)
    np.testing.assert_array_equal(out[0, [0, 4]], vals[paged.rows(0, [0, 99])])
    assert not out[0, [1, 2, 3, 5]].any()


# ---------------------------------------------------------------- sparse decode
def lists_for(lens, T, K, seed, hole=0.0):
    rng = np.random.default_rng(seed)
    idx = np.full((len(lens), T, K), -1, np.int32)
    for b, n in enumerate(lens):
        for t in range(T):
            k = min(n, K)
            idx[b, t, :k] = rng.permutation(n)[:k]
            idx[b, t, rng.random(K) < hole] = -1
    return idx


def run_sparse(lens, T, H, idx, nsplit, seed=0, what="", **kw):
    paged = cu.Paged(lens, seed)
    cache, vals = fill(paged, lens, seed + 1)
    q = cu.queries(len(lens), T, H, seed + 2)
    o, lse = binding.decode_q4(q.cuda(), cache, paged.cuda, torch.from_numpy(idx).cuda(), SCALE, nsplit, **kw)
    torch.cuda.synchronize()
    kv = lambda b, t: vals[paged.rows(b, idx[b, t][idx[b, t] >= 0])]
    cu.check_attention(o, lse, q, kv, SCALE, what or f"H {H} K {idx.shape[2]} S {nsplit}")


@pytest.mark.parametrize("H", [1, 3, 8, 15, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("nsplit", [0, 1, 2, 3, 16])
def test_sparse_heads(H, nsplit):
    run_sparse([300, 90], 2, H, lists_for([300, 90], 2, 130, H, hole=0.1), nsplit, seed=H)


@pytest.mark.parametrize("K", [0, 1, 7, 31, 32, 33, 63, 64, 65, 127, 200, 513])
@pytest.mark.parametrize("H,nsplit", [(16, 0), (16, 1), (16, 4), (16, 5), (7, 8), (64, 2), (5, 70)])
def test_sparse_widths(K, H, nsplit):
    run_sparse([600], 1, H, lists_for([600], 1, K, K), nsplit, seed=K + 1)


@pytest.mark.parametrize("H", [3, 16, 40])
def test_one_row_comes_out_as_it_is(H):
    """A softmax over one row is 1: o is the row's latents, bit for bit."""
    paged = cu.Paged([90, 70], 1)
    cache, vals = fill(paged, [90, 70], 2)
    q, idx = cu.queries(2, 1, H, 3).cuda(), torch.tensor([[[77]], [[3]]], dtype=torch.int32).cuda()
    want = binding.q4_read(cache, paged.cuda, idx[:, 0])[:, :, None, :512].expand(2, 1, H, 512)
    assert torch.equal(binding.decode_q4(q, cache, paged.cuda, idx, SCALE)[0], want)
    first = binding.q4_read(cache, paged.cuda, torch.zeros_like(idx[:, 0]))[:, :, None, :512].expand(2, 1, H, 512)
    one = torch.ones(2, 1, dtype=torch.int32).cuda()
    assert torch.equal(binding.decode_dense_q4(q, cache, paged.cuda, one, SCALE, K=1)[0], first)


@pytest.mark.parametrize("H", [8, 16, 48])
def test_sparse_long_lists_cross_resolve_chunks(H):
    run_sparse([5000, 4999], 1, H, lists_for([5000, 4999], 1, 4600, 3), 1, seed=5)


@pytest.mark.parametrize("H", [16, 64])
def test_sparse_duplicates_count_each_time(H):
    idx = np.array([[[5, 5, 5, 9, -1, 9, 64, 5]]], np.int32)
    run_sparse([70], 1, H, idx, 1)


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("nsplit", [1, 3])
def test_sparse_rows_that_select_nothing(H, nsplit):
    idx = lists_for([200, 200, 200], 2, 100, 9)
    idx[0, 1] = -1
    idx[2] = -1
    run_sparse([200, 200, 200], 2, H, idx, nsplit)


@pytest.mark.parametrize("H", [16, 64])
def test_sparse_bad_entries_are_masked_and_counted(H):
    lens = [128]
    paged = cu.Paged(lens, 2)
    cache, vals = fill(paged, lens, 3)
    idx = np.array([[[0, 5000, -7, 3, 127, 2**31 - 1]]], np.int32)
    q = cu.queries(1, 1, H, 4)
    o, lse = binding.decode_q4(q.cuda(), cache, paged.cuda, torch.from_numpy(idx).cuda(), SCALE, 1)
    assert binding.check_device(clear=True) == (5, 3)
    cu.check_attention(o, lse, q, lambda b, t: vals[paged.rows(0, [0, 3, 127])], SCALE, "bad entries")


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("nsplit", [1, 4])
def test_a_row_without_a_finite_value_reaches_only_who_attends_to_it(H, nsplit):
    """Row 10 was stored from infinities: token 0 selects it, token 1 does not."""
    lens = [256]
    paged = cu.Paged(lens, 2)
    cache, vals = fill(paged, lens, 3)
    bad = cu.latents(1, 1)
    bad[0, 77] = float("inf")
    binding.q4_append(bad.cuda(), cache, paged.cuda, torch.tensor([0, 1], dtype=torch.int32).cuda(),
                      torch.tensor([10], dtype=torch.int32).cuda())
    idx = lists_for(lens, 2, 150, 1)
    idx[0][idx[0] == 10] = 11
    idx[0, 0, 70] = 10
    q = cu.queries(1, 2, H, 4)
    o, lse = binding.decode_q4(q.cuda(), cache, paged.cuda, torch.from_numpy(idx).cuda(), SCALE, nsplit)
    assert torch.isnan(o[0, 0]).all() and torch.isnan(lse[0, 0]).all()
    ro, rl, to, tl = cu.attend(cu.f64(q)[0, 1], vals[paged.rows(0, idx[0, 1])], SCALE)
    cu.check(o[0, 1], ro, to, "o")
    cu.check(lse[0, 1], rl, tl, "lse")


def test_sparse_on_another_stream_in_two_graphs_and_twice_the_same():
    lens = [3000] * 4
    paged = cu.Paged(lens, 2)
    cache, vals = fill(paged, lens, 3)
    table = paged.cuda
    idx = lists_for(lens, 1, 700, 1)
    q = cu.queries(4, 1, 16, 4)
    qc, ic = q.cuda(), torch.from_numpy(idx).cuda()
    o, lse = binding.decode_q4(qc, cache, table, ic, SCALE)
    kv = lambda b, t: vals[paged.rows(b, idx[b, t])]
    cu.check_attention(o, lse, q, kv, SCALE, "plain call")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = binding.decode_q4(qc, cache, table, ic, SCALE, stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    graphs = []
    for k in range(2):
        g, out = torch.cuda.CUDAGraph(), (torch.empty_like(o), torch.empty_like(lse))
        with torch.cuda.graph(g):
            binding.decode_q4(qc, cache, table, ic, SCALE, o=out[0], lse=out[1])
        graphs.append((g, out))
    for g, out in graphs + graphs:
        out[0].zero_()
        g.replay()
        assert torch.equal(o, out[0]) and torch.equal(lse, out[1])


def test_calls_from_two_threads_on_two_streams():
    """Two host threads decode at once, each on a stream of its own, over one cache."""
    import threading
    lens = [900, 800]
    paged = cu.Paged(lens, 2)
    cache, vals = fill(paged, lens, 3)
    table = paged.cuda
    idx = torch.from_numpy(lists_for(lens, 1, 500, 1)).cuda()
    seq = torch.tensor([[900], [800]], dtype=torch.int32).cuda()
    qs = [cu.queries(2, 1, 16, 4 + k).cuda() for k in range(2)]
    want = [(binding.decode_q4(q, cache, table, idx, SCALE), binding.decode_dense_q4(q, cache, table, seq, SCALE, K=900)) for q in qs]
    torch.cuda.synchronize()
    bad = []

    def work(k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = (binding.decode_q4(qs[k], cache, table, idx, SCALE), binding.decode_dense_q4(qs[k], cache, table, seq, SCALE, K=900))
                stream.synchronize()
                bad.extend(not torch.equal(x, y) for a, b in zip(got, want[k]) for x, y in zip(a, b))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(bad) == 2 * 20 * 4 and not any(bad)


@pytest.mark.parametrize("T,H", [(1, 16), (2, 40)])
def test_dense_in_two_graphs(T, H):
    lens = [[700 - t for t in range(T)][::-1], [130 - t for t in range(T)][::-1]]
    paged = cu.Paged([700, 130], 2)
    cache, vals = fill(paged, lens, 3)
    table, q = paged.cuda, cu.queries(2, T, H, 4).cuda()
    seq = torch.tensor(lens, dtype=torch.int32).cuda()
    o, lse = binding.decode_dense_q4(q, cache, table, seq, SCALE, K=700)
    graphs = []
    for _ in range(2):
        g, out = torch.cuda.CUDAGraph(), (torch.empty_like(o), torch.empty_like(lse))
        with torch.cuda.graph(g):
            binding.decode_dense_q4(q, cache, table, seq, SCALE, K=700, o=out[0], lse=out[1])
        graphs.append((g, out))
    for g, out in graphs + graphs:
        out[0].zero_()
        g.replay()
        assert torch.equal(o, out[0]) and torch.equal(lse, out[1])


def test_binding_refuses_what_the_kernels_cannot_read():
    paged = cu.Paged([64])
    cache, _ = fill(paged, None, 1)
    q, table = cu.queries(1, 1, 8, 1).cuda(), paged.cuda
    idx, lens = torch.zeros(1, 1, 4, dtype=torch.int32).cuda(), torch.ones(1, 1, dtype=torch.int32).cuda()
    with pytest.raises(ValueError):
        binding.decode_q4(q, cache[:, :, :400].contiguous(), table, idx, SCALE)
    with pytest.raises(ValueError):
        binding.decode_q4(q, cache.transpose(0, 1), table, idx, SCALE)
    with pytest.raises(TypeError):
        binding.decode_q4(q, cache, table, idx.long(), SCALE)
    with pytest.raises(ValueError):
        binding.decode_q4(q, cache, table, idx[:, 0], SCALE)
    with pytest.raises(ValueError):
        binding.decode_q4(q, cache, torch.cat([table, table]), idx, SCALE)
    with pytest.raises(ValueError):
        binding.decode_q4(q, cache, table, idx.cpu(), SCALE)
    with pytest.raises(ValueError):
        binding.decode_q4(q, cache, table, idx, SCALE, o=torch.empty(1, 1, 8, 511, dtype=torch.bfloat16).cuda())
    with pytest.raises(binding.SmlaError):
        binding.decode_q4(q, cache, table, torch.zeros(1, 1, 400, dtype=torch.int32).cuda(), SCALE, 3, workspace=torch.empty(64, dtype=torch.uint8).cuda())
    with pytest.raises(binding.SmlaError):
        binding.decode_dense_q4(q, cache, table, lens, float("inf"))
    with pytest.raises(binding.SmlaError):
        shifted = torch.empty(8 * 576 + 1, dtype=torch.bfloat16).cuda()[1:].view(1, 1, 8, 576)
        binding.decode_dense_q4(shifted, cache, table, lens, SCALE)
    with pytest.raises(ValueError):
        binding.q4_append(q.view(8, 576), cache, table, torch.zeros(1, dtype=torch.int32).cuda(), lens[0])
    with pytest.raises(ValueError):
        binding.q4_read(cache, table, idx)


# ---------------------------------------------------------------- dense decode
def run_dense(lens, H, nsplit, seed=0, K=None, slack=0):
    lens = np.asarray(lens, np.int32)
    paged = cu.Paged([int(x.max()) for x in lens], seed, extra=slack)
    cache, vals = fill(paged, lens, seed + 1)
    q = cu.queries(*lens.shape, H, seed + 2)
    o, lse = binding.decode_dense_q4(q.cuda(), cache, paged.cuda, torch.from_numpy(lens).cuda(), SCALE, nsplit, K=K)
    torch.cuda.synchronize()
    cu.check_attention(o, lse, q, lambda b, t: vals[paged.rows(b, range(lens[b, t]))], SCALE,
                       f"H {H} S {nsplit} lens {lens.tolist()}")


@pytest.mark.parametrize("H", [1, 7, 8, 16, 17, 32, 40, 64])
@pytest.mark.parametrize("nsplit", [0, 1, 3])
def test_dense_heads(H, nsplit):
    run_dense([[198, 199, 200], [63, 64, 65]], H, nsplit, seed=H)


@pytest.mark.parametrize("lens", [
    [[0]], [[1]], [[0], [1], [0]], [[31], [32], [33]], [[63], [64], [65]], [[1000], [1], [129]],
    [[0, 0, 5]], [[900, 3, 0, 64, 511]], [[128], [0], [2000], [0], [77]],
])
@pytest.mark.parametrize("H,nsplit", [(16, 0), (16, 5), (64, 0), (8, 1)])
def test_dense_lengths(lens, H, nsplit):
    run_dense(lens, H, nsplit, seed=len(lens))


@pytest.mark.parametrize("H", [3, 40])
def test_dense_many_ragged_sequences(H):
    """More sequences than a block has threads, runs that cross many of them, empty ones between."""
    rng = np.random.default_rng(H)
    run_dense([[int(x)] for x in rng.integers(0, 200, 300) * (rng.random(300) < 0.7)], H, 0, seed=H)


def test_dense_one_long_sequence_among_many_empty():
    """Its pieces outnumber the combine's threads."""
    run_dense([[0]] * 400 + [[39000]] + [[1]] * 199, 2, 0, seed=1)


def test_dense_bound_above_every_length():
    run_dense([[70], [300]], 16, 0, K=4096)
    run_dense([[70], [300]], 64, 0, K=4096)


@pytest.mark.parametrize("T,H", [(9, 8), (4, 16), (5, 3), (33, 2), (3, 64)])
def test_dense_many_tokens(T, H):
    run_dense([[500 - T + t + 1 for t in range(T)], [90 + t for t in range(T)]], H, 0, seed=T)


def test_dense_clamps_and_counts_lengths_and_unmapped_positions():
    paged = cu.Paged([128, 128], 1)
    paged.table[1, 1] = -1
    cache, vals = fill(paged, None, 2)
    q = cu.queries(2, 1, 16, 3)
    lens = torch.tensor([[-4], [128]], dtype=torch.int32).cuda()
    o, lse = binding.decode_dense_q4(q.cuda(), cache, paged.cuda, lens, SCALE, 1, K=128)
    st, bad = binding.check_device(clear=True)
    assert st == 5 and bad == 1 + 64
    cu.check_attention(o, lse, q, lambda b, t: vals[paged.rows(b, range(64 * b))], SCALE, "unmapped")


@pytest.mark.parametrize("H", [4, 64])
def test_dense_a_draft_without_a_finite_value_leaves_earlier_tokens_alone(H):
    paged = cu.Paged([100], 1)
    cache, vals = fill(paged, None, 2)
    bad = cu.latents(1, 1)
    bad[0, 300] = float("nan")
    binding.q4_append(bad.cuda(), cache, paged.cuda, torch.tensor([0, 1], dtype=torch.int32).cuda(),
                      torch.tensor([99], dtype=torch.int32).cuda())
    q = cu.queries(1, 2, H, 4)
    lens = torch.tensor([[99, 100]], dtype=torch.int32).cuda()
    o, lse = binding.decode_dense_q4(q.cuda(), cache, paged.cuda, lens, SCALE, 0, K=100)
    ro, rl, to, tl = cu.attend(cu.f64(q)[0, 0], vals[paged.rows(0, range(99))], SCALE)
    cu.check(o[0, 0], ro, to, "o")
    cu.check(lse[0, 0], rl, tl, "lse")
    assert torch.isnan(o[0, 1]).all() and torch.isnan(lse[0, 1]).all()


def test_dense_equals_sparse_over_every_position():
    """The same rows by a list and by a length: both are held to the same bound."""
    lens = [700]
    paged = cu.Paged(lens, 4)
    cache, vals = fill(paged, lens, 5)
    q = cu.queries(1, 1, 16, 6)
    idx = torch.arange(700, dtype=torch.int32).view(1, 1, 700).cuda()
    for o, lse in (binding.decode_q4(q.cuda(), cache, paged.cuda, idx, SCALE),
                   binding.decode_dense_q4(q.cuda(), cache, paged.cuda, torch.tensor([[700]], dtype=torch.int32).cuda(), SCALE)):
        cu.check_attention(o, lse, q, lambda b, t: vals[paged.rows(0, range(700))], SCALE, "both")


@pytest.mark.parametrize("fill_value", [0.0, 1.0])
def test_extreme_scores(fill_value):
    """Scores of several hundred: one row takes all the weight; equal rows share it."""
    paged = cu.Paged([64], 0)
    rows = torch.full((64, 576), fill_value).to(torch.bfloat16)
    rows[17] = 24.0
    cache = torch.zeros(paged.pages, 64, cu.ROW, dtype=torch.uint8, device="cuda")
    binding.q4_append(rows.cuda(), cache, paged.cuda, torch.tensor([0, 64], dtype=torch.int32).cuda(),
                      torch.zeros(1, dtype=torch.int32).cuda())
    vals = cu.values(cache.cpu().numpy().reshape(-1, cu.ROW))[paged.rows(0, range(64))]
    for H in (16, 64):
        q = torch.ones(1, 1, H, 576).to(torch.bfloat16)
        o, lse = binding.decode_dense_q4(q.cuda(), cache, paged.cuda, torch.tensor([[64]], dtype=torch.int32).cuda(), 1.0)
        cu.check_attention(o, lse, q, lambda b, t: vals, 1.0, "extreme")


def one_row_of(cache, table, pos, H):
    """The latents at pos [B, T] as the o of queries that see only them."""
    B, T = pos.shape
    return binding.q4_read(cache, table, pos)[:, :, None, :512].expand(B, T, H, 512)


@pytest.mark.parametrize("H", [3, 16, 40])
@pytest.mark.parametrize("nsplit", [0, 1, 5])
def test_one_row_of_a_wide_list_comes_out_as_it_is(H, nsplit):
    """What a list of one row gives does not hang on the list's width or on where in it the row stands."""
    paged = cu.Paged([90, 70], 1)
    cache, _ = fill(paged, [90, 70], 2)
    idx = torch.full((2, 3, 2048), -1, dtype=torch.int32)
    pos = torch.tensor([[77, 3, 89], [0, 64, 69]], dtype=torch.int32)
    for b in range(2):
        for t, at in enumerate((0, 1000 + b, 2047)):
            idx[b, t, at] = pos[b, t]
    o, lse = binding.decode_q4(cu.queries(2, 3, H, 3).cuda(), cache, paged.cuda, idx.cuda(), SCALE, nsplit)
    assert torch.equal(o, one_row_of(cache, paged.cuda, pos.cuda(), H))


@pytest.mark.parametrize("T,H", [(1, 3), (1, 16), (2, 8), (1, 40), (2, 40)])
def test_one_visible_position_comes_out_as_it_is(T, H):
    """Neither a bound above every length nor a longer neighbour or a longer token of the same sequence changes it."""
    paged = cu.Paged([4000, 4000, 90], 1)
    cache, _ = fill(paged, None, 2)
    table, q = paged.cuda, cu.queries(3, T, H, 3).cuda()
    want = one_row_of(cache, table, torch.zeros(3, T, dtype=torch.int32).cuda(), H)
    one = torch.ones(3, T, dtype=torch.int32).cuda()
    assert torch.equal(binding.decode_dense_q4(q, cache, table, one, SCALE, K=4096)[0], want)
    one[1], one[0, -1] = 4000, 4000 if T > 1 else 1
    o = binding.decode_dense_q4(q, cache, table, one, SCALE, K=4096)[0]
    seen = one.cpu() == 1
    assert torch.equal(o[seen], want[seen])


@pytest.mark.parametrize("T,H", [(1, 16), (3, 4)])
def test_the_bound_alone_changes_nothing(T, H):
    """Up to 16 query rows: the same bits with the least bound and with larger ones."""
    lens = torch.tensor([[300 - T + t + 1 for t in range(T)], [70 + t for t in range(T)]], dtype=torch.int32).cuda()
    paged = cu.Paged([300, 80], 1, extra=1)
    cache, _ = fill(paged, None, 2)
    q = cu.queries(2, T, H, 3).cuda()
    want = binding.decode_dense_q4(q, cache, paged.cuda, lens, SCALE, 4, K=300)
    for K in (512, 513, 40000):
        got = binding.decode_dense_q4(q, cache, paged.cuda, lens, SCALE, 4, K=K)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_dense_more_pieces_than_the_combine_has_threads():
    """600 blocks share the 610 tiles of one sequence among empty ones: 600 pieces, where
    the combine's 512 threads take one each.  (Few rows, which four blocks join, have
    at most two blocks per SM to be cut by, so they never have as many.)"""
    blocks, tiles = 600, -(-39000 // 64)
    pieces = min(blocks, tiles)
    assert 2 * torch.cuda.get_device_properties(0).multi_processor_count <= blocks and pieces > 512
    run_dense([[0]] * 400 + [[39000]] + [[0]] * 199, 2, 0, seed=1)
    run_dense([[0, 0]] * 599 + [[38999, 39000]], 8, 0, seed=2)


@pytest.mark.parametrize("H", [24, 64])
def test_dense_clamps_lengths_and_masks_unmapped_positions_of_many_rows(H):
    paged = cu.Paged([128, 128], 1)
    paged.table[1, 1] = -1
    cache, vals = fill(paged, None, 2)
    q = cu.queries(2, 1, H, 3)
    o, lse = binding.decode_dense_q4(q.cuda(), cache, paged.cuda, torch.tensor([[-4], [128]], dtype=torch.int32).cuda(),
                                     SCALE, 1, K=128)
    assert binding.check_device(clear=True)[0] == 5
    cu.check_attention(o, lse, q, lambda b, t: vals[paged.rows(b, range(64 * b))], SCALE, "unmapped")
