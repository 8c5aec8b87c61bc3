"""Eviction on the GPU: accumulated weights, plans, moves, and a run of the
whole cache's life, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import cache_util as cu
from sparse_mla_decode_partial_b200 import binding
from test_gpu_q4 import SCALE, clean_device, fill  # noqa: F401

pytestmark = pytest.mark.gpu
INF = math.inf


def make_cache(paged, q4, seed):
    if q4:
        return fill(paged, None, seed)
    rows = cu.latents(paged.pages * 64, seed)
    return rows.view(paged.pages, 64, 576).cuda(), cu.f64(rows)


def check_weights(acc, before, q, lse, lens, rows_of, what):
    """acc against the definition.  A weight exp(x) with x off by dx (the score's
    bound of cache_util.attend and 2^-22 of |x| + |lse|, both parts of lse
    exact to 2^-48) is off by 2 dx of itself, ex2 adds 2^-21; the row sums and
    the addition to acc round once per term."""
    want, tol = before.copy(), np.zeros_like(before)
    B, T, H = lse.shape
    for b in range(B):
        for t in range(T):
            n = int(lens[b, t])
            if n == 0:
                continue
            kv = rows_of(b, n)
            s = q[b, t] @ kv.T * SCALE
            ds = 580 * 2.0 ** -23 * SCALE * (np.abs(q[b, t]) @ np.abs(kv).T) + 2.0 ** -22 * (np.abs(s) + np.abs(lse[b, t])[:, None] + 1)
            live = np.isfinite(lse[b, t])
            w = np.exp(s[live] - lse[b, t][live][:, None])
            want[b, :n] += w.sum(0)
            tol[b, :n] += (w * (2 * ds[live] + 2.0 ** -20 + 2.0 ** -23 * T * H)).sum(0)
    cu.check(acc, want, tol + 2.0 ** -23 * np.abs(want) + 1e-37, what)


def run_weigh(lens, H, q4, seed=0, max_n=None, lse_edit=None):
    lens = np.asarray(lens, np.int32)
    B, T = lens.shape
    most = int(lens.max()) if max_n is None else max_n
    paged = cu.Paged([max(int(x.max()), 1) for x in lens], seed)
    cache, vals = make_cache(paged, q4, seed + 1)
    q = cu.queries(B, T, H, seed + 2)
    qd = cu.f64(q)
    lse = np.full((B, T, H), -INF)
    for b in range(B):
        for t in range(T):
            if lens[b, t]:
                lse[b, t] = cu.attend(qd[b, t], vals[paged.rows(b, range(lens[b, t]))], SCALE)[1]
    if lse_edit:
        lse_edit(lse)
    lse32 = torch.from_numpy(lse).float()
    acc = torch.rand(B, most, generator=torch.Generator().manual_seed(seed)) * 0.01
    got = acc.cuda()
    out = binding.evict_accumulate(q.cuda(), cache, paged.cuda, torch.from_numpy(lens).cuda(), lse32.cuda(), SCALE, got)
    assert out is got
    check_weights(got, acc.double().numpy(), qd, lse32.double().numpy(), lens,
                  lambda b, n: vals[paged.rows(b, range(n))], f"lens {lens.tolist()} H {H} q4 {q4}")
    again = acc.cuda()
    binding.evict_accumulate(q.cuda(), cache, paged.cuda, torch.from_numpy(lens).cuda(), lse32.cuda(), SCALE, again)
    assert torch.equal(got, again)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 16), (1, 17), (2, 16), (3, 8), (9, 8), (1, 64), (5, 64), (2, 40)])
def test_weights_over_query_rows(T, H, q4):
    run_weigh([[200 + t for t in range(T)], [31 + t for t in range(T)]], H, q4, seed=T + H)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("lens", [[[0]], [[1]], [[0], [5], [0]], [[31], [32], [33]], [[64], [65], [1500]], [[0, 70, 3, 64]]])
def test_weights_over_lengths(lens, q4):
    run_weigh(lens, 16, q4, seed=len(lens), max_n=1600)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("H", [4, 24])
def test_weights_over_many_ragged_sequences(H, q4):
    """More sequences than a block has threads, runs that cross many of them, empty ones between."""
    rng = np.random.default_rng(H)
    run_weigh([[int(x)] for x in rng.integers(0, 200, 600) * (rng.random(600) < 0.7)], H, q4, seed=H)


@pytest.mark.parametrize("q4", [False, True])
def test_weights_of_rows_with_empty_and_infinite_lse(q4):
    def edit(lse):
        lse[0, 0, 3] = -INF
        lse[0, 1, 2] = INF
    run_weigh([[90, 100]], 8, q4, lse_edit=edit)


@pytest.mark.parametrize("H", [4, 16])
@pytest.mark.parametrize("q4", [False, True])
def test_weights_ignore_what_lies_behind_the_length(q4, H):
    """NaN rows in the masked part of a page and of the pool change nothing."""
    paged = cu.Paged([40], 1)
    cache, vals = make_cache(paged, q4, 2)
    q, lens = cu.queries(1, 2, H, 3), torch.tensor([[30, 37]], dtype=torch.int32).cuda()
    lse = torch.zeros(1, 2, H).cuda() + 4.0
    acc = torch.zeros(1, 40).cuda()
    binding.evict_accumulate(q.cuda(), cache, paged.cuda, lens, lse, SCALE, acc)
    flat = cache.view(-1, cache.shape[-1])
    keep = set(paged.rows(0, range(37)).tolist())
    dead = torch.tensor([r for r in range(flat.shape[0]) if r not in keep]).cuda()
    flat[dead] = 0xFF if q4 else float("nan")
    acc2 = torch.zeros(1, 40).cuda()
    binding.evict_accumulate(q.cuda(), cache, paged.cuda, lens, lse, SCALE, acc2)
    assert torch.equal(acc, acc2) and not acc[0, 37:].any()


@pytest.mark.parametrize("H", [4, 20])
@pytest.mark.parametrize("q4", [False, True])
def test_weights_of_a_sequence_ignore_its_neighbours_queries(q4, H):
    """NaN queries and statistics of one sequence stay out of the other's weights."""
    paged = cu.Paged([70, 70], 1)
    cache, vals = make_cache(paged, q4, 2)
    q, lse = cu.queries(2, 1, H, 3).cuda(), torch.zeros(2, 1, H).cuda() + 4.0
    lens = torch.tensor([[70], [70]], dtype=torch.int32).cuda()
    want = binding.evict_accumulate(q, cache, paged.cuda, lens, lse, SCALE, torch.zeros(2, 70).cuda())
    q[1], lse[1] = float("nan"), float("nan")
    got = binding.evict_accumulate(q, cache, paged.cuda, lens, lse, SCALE, torch.zeros(2, 70).cuda())
    assert torch.equal(got[0], want[0]) and got[1].isnan().all()


@pytest.mark.parametrize("H", [4, 20])
@pytest.mark.parametrize("q4", [False, True])
def test_weights_count_bad_lengths_and_pages(q4, H):
    paged = cu.Paged([128, 128], 1)
    paged.table[0, 1] = 10 ** 6
    cache, vals = make_cache(paged, q4, 2)
    q, lse = cu.queries(2, 1, H, 3).cuda(), torch.zeros(2, 1, H).cuda()
    acc = torch.zeros(2, 100).cuda()
    lens = torch.tensor([[100], [-3]], dtype=torch.int32).cuda()
    binding.evict_accumulate(q, cache, paged.cuda, lens, lse, SCALE, acc)
    assert binding.check_device(clear=True) == (5, 36 + 1)
    assert acc[0, :64].all() and not acc[0, 64:].any() and not acc[1].any()


# ---------------------------------------------------------------- plan
def run_plan(acc, n, K, pos=None, n_sink=0, n_recent=0):
    B, most = acc.shape
    p = binding.evict_plan(torch.from_numpy(acc).float().cuda(), torch.tensor(n, dtype=torch.int32).cuda(), K,
                           pos=None if pos is None else torch.from_numpy(pos).cuda(), n_sink=n_sink, n_recent=n_recent)
    src = np.full((B, K), -1, np.int32)
    a_new, p_new = np.zeros((B, most), np.float32), np.full((B, most), -1, np.int32)
    for b in range(B):
        ps = np.arange(most, dtype=np.int32) if pos is None else pos[b]
        s = cu.plan(acc[b].astype(np.float32).tolist(), ps.tolist(), n[b], K, n_sink, n_recent)
        src[b, :len(s)] = s
        a_new[b, :len(s)], p_new[b, :len(s)] = acc[b].astype(np.float32)[s], ps[s]
    np.testing.assert_array_equal(p.src.cpu().numpy(), src)
    np.testing.assert_array_equal(p.n.cpu().numpy(), np.minimum(n, K))
    np.testing.assert_array_equal(p.acc.cpu().numpy(), a_new)
    np.testing.assert_array_equal(p.pos.cpu().numpy(), p_new)


@pytest.mark.parametrize("most,n,K", [
    (1, [1], 1), (1, [0], 1), (5, [5, 4, 0, 1], 3), (64, [64, 33], 32), (100, [100, 99, 65], 64), (100, [100], 200),
    (1000, [1000, 1, 777], 1), (1000, [1000, 999], 998), (4097, [4097, 2048], 2048), (70001, [70001, 60000], 50000),
])
def test_plan_sizes(most, n, K):
    rng = np.random.default_rng(most + K)
    run_plan(rng.exponential(1.0, (len(n), most)), n, K)


@pytest.mark.parametrize("B,most,K", [(1, 8192, 8000), (2, 16385, 9000), (20, 9000, 8999), (40, 4100, 1000), (80, 2500, 2400),
                                      (1, 460001, 300000)])
def test_plan_batches_and_lengths_over_the_cluster_sizes(B, most, K):
    """Sequences shared by one to eight thread blocks, with positions, ragged, and
    too long for the keys to be kept in shared memory."""
    rng = np.random.default_rng(B)
    n = [most] + [int(x) for x in rng.integers(0, most + 1, B - 1)]
    pos = np.stack([rng.permutation(most) for _ in range(B)]).astype(np.int32)
    run_plan(np.round(rng.exponential(1.0, (B, most)), 3), n, K, pos=pos, n_sink=5, n_recent=100)


def test_plan_longest_sequences_one_thread_block_each():
    """As many slots as a call may have, in a batch whose sequences have one block each."""
    rng = np.random.default_rng(3)
    n = [0] * 80
    n[7], n[78], n[79] = 524288, 1, 300000
    run_plan(np.round(rng.exponential(1.0, (80, 524288)), 4), n, 250000, n_recent=77)


@pytest.mark.parametrize("kind", ["equal", "few", "zeros", "negative", "special"])
def test_plan_ties_and_special_weights(kind):
    rng = np.random.default_rng(1)
    acc = rng.exponential(1.0, (3, 500))
    if kind == "equal":
        acc[:] = 0.25
    elif kind == "few":
        acc = np.round(acc)
    elif kind == "zeros":
        acc = np.where(acc < 1, -0.0, np.where(acc < 2, 0.0, acc))
    elif kind == "negative":
        acc = 1 - acc
    else:
        acc[:, ::7], acc[:, 1::7], acc[:, 2::7], acc[:, 3::7] = np.nan, INF, -INF, 1e-45
    run_plan(acc, [500, 321, 40], 200)
    run_plan(acc, [500, 321, 40], 33, n_sink=4, n_recent=20)


@pytest.mark.parametrize("n_sink,n_recent", [(0, 0), (4, 0), (0, 30), (4, 30), (40, 60)])
def test_plan_keeps_sinks_and_recent_positions(n_sink, n_recent):
    rng = np.random.default_rng(2)
    B, most = 3, 400
    acc = rng.exponential(1.0, (B, most))
    pos = np.stack([rng.permutation(most * 3)[:most] for _ in range(B)]).astype(np.int32)
    run_plan(acc, [400, 399, 130], 100, pos=pos, n_sink=n_sink, n_recent=n_recent)
    run_plan(acc, [400, 399, 130], 100, n_sink=n_sink, n_recent=n_recent)


def test_plan_without_positions_out():
    """The C entry point without acc_new and pos_new: the list of movers goes to the workspace."""
    acc = torch.rand(3, 900, generator=torch.Generator().manual_seed(1)).cuda()
    n = torch.tensor([900, 500, 20], dtype=torch.int32).cuda()
    want = binding.evict_plan(acc, n, 300)
    src, m = torch.empty_like(want.src), torch.empty_like(n)
    ws = torch.empty(binding.evict_workspace_bytes(3, 900), dtype=torch.uint8, device="cuda")
    st = binding.lib().smla_evict_plan(acc.data_ptr(), None, n.data_ptr(), 3, 900, 300, 0, 0, ws.data_ptr(), ws.numel(),
                                       src.data_ptr(), m.data_ptr(), None, None, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(src, want.src) and torch.equal(m, want.n)


def test_plan_far_positions():
    acc = np.arange(40, dtype=np.float64)[None]
    pos = (np.arange(40)[None] + 2 ** 31 - 40).astype(np.int32)
    run_plan(acc, [40], 10, pos=pos, n_sink=2, n_recent=3)


def test_plan_clamps_and_counts_lengths():
    acc = torch.rand(2, 10).cuda()
    p = binding.evict_plan(acc, torch.tensor([-1, 11], dtype=torch.int32).cuda(), 20)
    assert binding.check_device(clear=True) == (5, 2)
    assert p.n.tolist() == [0, 10]


# ---------------------------------------------------------------- apply
@pytest.mark.parametrize("n,K", [([130, 64, 3], 50), ([700], 640), ([65, 66], 64)])
def test_apply_moves_rows_of_every_buffer(n, K):
    rng = np.random.default_rng(K)
    paged = cu.Paged(n, 3)
    bufs = [torch.randint(0, 256, (paged.pages, 64, w), dtype=torch.uint8, generator=torch.Generator().manual_seed(w)).cuda()
            for w in (1152, 416, 256, 16)]
    bufs[0] = bufs[0].view(torch.bfloat16)
    acc = torch.from_numpy(rng.exponential(1.0, (len(n), max(n)))).float().cuda()
    p = binding.evict_plan(acc, torch.tensor(n, dtype=torch.int32).cuda(), K)
    before = [b.view(torch.uint8).cpu().numpy().reshape(paged.pages * 64, -1).copy() for b in bufs]
    for _ in range(2):  # the second time changes nothing
        binding.evict_apply(p.src, paged.cuda, bufs)
        src = p.src.cpu().numpy()
        for buf, old in zip(bufs, before):
            want = old.copy()
            for b in range(len(n)):
                for i in range(min(n[b], K)):
                    want[paged.row(b, i)] = old[paged.row(b, src[b, i])]
            np.testing.assert_array_equal(buf.view(torch.uint8).cpu().numpy().reshape(paged.pages * 64, -1), want)


def test_apply_long_rows():
    """Rows of 20 KB: longer than the bulk form takes."""
    paged = cu.Paged([150], 3)
    buf = torch.randint(0, 256, (paged.pages, 64, 20480), dtype=torch.uint8, generator=torch.Generator().manual_seed(1)).cuda()
    old = buf.clone().view(-1, 20480)
    p = binding.evict_plan(torch.rand(1, 150, generator=torch.Generator().manual_seed(2)).cuda(), torch.tensor([150], dtype=torch.int32).cuda(), 70)
    binding.evict_apply(p.src, paged.cuda, (buf,))
    want = old.clone()
    to = torch.from_numpy(paged.rows(0, range(70))).cuda()
    want[to] = old[torch.from_numpy(paged.rows(0, p.src[0].tolist())).cuda()]
    assert torch.equal(buf.view(-1, 20480), want)


def test_apply_leaves_out_and_counts_unmapped_rows():
    paged = cu.Paged([128], 3)
    buf = torch.randint(0, 256, (paged.pages, 64, 32), dtype=torch.uint8).cuda()
    old = buf.cpu().numpy().reshape(-1, 32).copy()
    src = torch.tensor([[0, 127, 500, -2, 4, -1]], dtype=torch.int32).cuda()
    binding.evict_apply(src, paged.cuda, (buf,))
    assert binding.check_device(clear=True) == (5, 2)
    want = old.copy()
    want[paged.row(0, 1)] = old[paged.row(0, 127)]
    np.testing.assert_array_equal(buf.cpu().numpy().reshape(-1, 32), want)


def test_plan_of_empty_sequences():
    p = binding.evict_plan(torch.empty(2, 0).cuda(), torch.zeros(2, dtype=torch.int32).cuda(), 5)
    assert p.src.tolist() == [[-1] * 5] * 2 and p.n.tolist() == [0, 0] and p.acc.shape == (2, 0)


@pytest.mark.parametrize("q4", [False, True])
def test_accumulate_plan_apply_in_a_graph_and_on_another_stream(q4):
    paged = cu.Paged([500, 300], 1)
    start, _ = make_cache(paged, q4, 2)
    table, q = paged.cuda, cu.queries(2, 1, 16, 3).cuda()
    n = torch.tensor([500, 300], dtype=torch.int32).cuda()
    lens, lse = n[:, None].contiguous(), torch.full((2, 1, 16), 6.0).cuda()

    def steps(cache, acc, stream=None):
        binding.evict_accumulate(q, cache, table, lens, lse, SCALE, acc, stream=stream)
        p = binding.evict_plan(acc, n, 256, n_sink=4, n_recent=32, stream=stream)
        binding.evict_apply(p.src, table, (cache,), stream=stream)
        return p

    want_cache, want_acc = start.clone(), torch.zeros(2, 500).cuda()
    want = steps(want_cache, want_acc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache, acc = start.clone(), torch.zeros(2, 500).cuda()
    side.wait_stream(torch.cuda.current_stream())
    got = steps(cache, acc, stream=side)
    side.synchronize()
    assert torch.equal(cache.view(torch.uint8), want_cache.view(torch.uint8)) and all(torch.equal(a, b) for a, b in zip(got, want))
    cache, acc = start.clone(), torch.zeros(2, 500).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = steps(cache, acc)
    for _ in range(2):
        cache.copy_(start)
        acc.zero_()
        graph.replay()
        assert torch.equal(acc, want_acc) and torch.equal(cache.view(torch.uint8), want_cache.view(torch.uint8))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("q4", [False, True])
def test_pages_beyond_four_gigabytes(q4):
    """Every operator gives the same bits over the far pages of a pool larger than
    2^32 bytes as over a small pool."""
    far = 170000 if q4 else 60000
    lens = [300, 129]
    paged = cu.Paged(lens, 5)
    small, _ = make_cache(paged, q4, 6)
    big = torch.empty(far, *small.shape[1:], dtype=small.dtype, device="cuda")
    shift = far - paged.pages
    big[shift:] = small
    assert shift * small[0].numel() * small.element_size() > 2 ** 32
    near = paged.cuda
    table = torch.where(near >= 0, near + shift, near)
    q = cu.queries(2, 1, 16, 7).cuda()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    seq, lse = n[:, None].contiguous(), torch.full((2, 1, 16), 6.0).cuda()
    rows = cu.latents(9, 8).cuda()
    got = []
    for cache, pt in ((small, near), (big, table)):
        out = []
        if q4:
            binding.q4_append(rows, cache, pt, torch.tensor([0, 4, 9], dtype=torch.int32).cuda(), n - 5)
            every = torch.arange(300, dtype=torch.int32).expand(2, 300).cuda().where(torch.arange(300).cuda() < n[:, None], -1)
            idx = every.int().contiguous()
            out.append(binding.q4_read(cache, pt, idx))
            for H in (16, 40):
                qh = cu.queries(2, 1, H, 9).cuda()
                out.extend(binding.decode_q4(qh, cache, pt, idx[:, None], SCALE))
                out.extend(binding.decode_dense_q4(qh, cache, pt, seq, SCALE, K=300))
        acc = torch.zeros(2, 300).cuda()
        out.append(binding.evict_accumulate(q, cache, pt, seq, lse, SCALE, acc))
        p = binding.evict_plan(acc, n, 100)
        out.extend(p)
        binding.evict_apply(p.src, pt, (cache,))
        got.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert torch.equal(big[shift:].view(torch.uint8), small.view(torch.uint8))


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("q4", [False, True])
def test_a_cache_lives_through_steps_and_evictions(q4):
    """Rows enter, tokens decode over all of them, their weights accumulate, the
    cache is cut back to its budget, and the next step decodes over what is
    left: every step against 64 bits, on one stream without a synchronisation."""
    B, H, budget, room = 3, 8, 96, 256
    paged = cu.Paged([room] * B, 7)
    table = paged.cuda
    rng = np.random.default_rng(0)
    cache = (torch.zeros(paged.pages, 64, cu.ROW, dtype=torch.uint8) if q4 else
             torch.zeros(paged.pages, 64, 576, dtype=torch.bfloat16)).cuda()
    held = [[] for _ in range(B)]                 # (position, values) by slot
    acc = torch.zeros(B, room).cuda()
    pos = torch.full((B, room), -1, dtype=torch.int32).cuda()
    n = torch.zeros(B, dtype=torch.int32).cuda()
    nxt = [0] * B
    for step in range(4):
        new = [int(rng.integers(40, 90)) for _ in range(B)]
        rows = cu.latents(sum(new), 100 + step)
        at, cnt = 0, [len(h) for h in held]
        stored = cu.values(cu.quantise(rows)) if q4 else cu.f64(rows)
        offs = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
        if q4:
            binding.q4_append(rows.cuda(), cache, table, offs, n)
        for b in range(B):
            if not q4:
                flat = cache.view(-1, 576)
                flat[torch.from_numpy(paged.rows(b, range(cnt[b], cnt[b] + new[b]))).cuda()] = rows[at:at + new[b]].cuda()
            pos[b, cnt[b]:cnt[b] + new[b]] = torch.arange(nxt[b], nxt[b] + new[b]).int().cuda()
            held[b] += [(nxt[b] + k, stored[at + k]) for k in range(new[b])]
            nxt[b] += new[b]
            at += new[b]
        n = n + torch.tensor(new, dtype=torch.int32).cuda()
        q = cu.queries(B, 1, H, 200 + step)
        lens = n[:, None].contiguous()
        most = max(len(h) for h in held)
        decode = binding.decode_dense_q4 if q4 else binding.decode_dense
        o, lse = decode(q.cuda(), cache, table, lens, SCALE, K=most)
        before = acc.double().cpu().numpy()
        binding.evict_accumulate(q.cuda(), cache, table, lens, lse, SCALE, acc)
        p = binding.evict_plan(acc, n, budget, pos=pos, n_sink=4, n_recent=32)
        vals = [np.stack([v for _, v in h]) for h in held]
        if q4:
            cu.check_attention(o, lse, q, lambda b, t: vals[b], SCALE, f"step {step}")
        check_weights(acc, before, cu.f64(q), lse.double().cpu().numpy(), lens.cpu().numpy(),
                      lambda b, k: vals[b][:k], f"step {step}")
        for b in range(B):
            s = cu.plan(acc[b].cpu().tolist(), pos[b].tolist(), len(held[b]), budget, 4, 32)
            np.testing.assert_array_equal(p.src[b, :len(s)].cpu().numpy(), s)
            held[b] = [held[b][i] for i in s]
            assert p.pos[b, :len(s)].tolist() == [h[0] for h in held[b]]
        binding.evict_apply(p.src, table, (cache,))
        acc, pos, n = p.acc, p.pos, p.n
    raw = cache.cpu()
    for b in range(B):
        at = paged.rows(b, range(len(held[b])))
        got = cu.values(raw.numpy().reshape(-1, cu.ROW)[at]) if q4 else cu.f64(raw.view(-1, 576)[at])
        np.testing.assert_array_equal(got, np.stack([v for _, v in held[b]]))


# ---------------------------------------------------------------- long sequences
def check_weights_on_the_gpu(acc, before, q, lse, lens, values, what):
    """check_weights() for long sequences: the same definition and bound in 64 bits by
    torch, every position; values [B] of [n, 576]."""
    B, T, H = lse.shape
    q, lse = q.double(), lse.double()
    want, tol = before.double(), torch.zeros_like(before, dtype=torch.float64)
    for b in range(B):
        kv = values[b].double()
        for t in range(T):
            n = int(lens[b, t])
            s = q[b, t] @ kv[:n].T * SCALE
            ds = 580 * 2.0 ** -23 * SCALE * (q[b, t].abs() @ kv[:n].abs().T) + 2.0 ** -22 * (s.abs() + lse[b, t].abs()[:, None] + 1)
            w = torch.exp(s - lse[b, t][:, None])
            want[b, :n] += w.sum(0)
            tol[b, :n] += (w * (2 * ds + 2.0 ** -20 + 2.0 ** -23 * T * H)).sum(0)
    tol += 2.0 ** -23 * want.abs() + 1e-37
    off = (acc.double() - want).abs()
    assert (off <= tol).all(), f"{what}: {(off > tol).sum().item()} off, worst {(off / tol).max().item():.3g} x the bound"


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("T,H", [(1, 16), (3, 8), (4, 16), (9, 8), (2, 48), (16, 8), (25, 8), (5, 64)])
def test_weights_over_long_sequences(T, H, q4):
    """Every block walks several steps of a sequence: the ring, the accumulators and the
    parts of a score come round again, once and in further passes."""
    lens = torch.tensor([[65111 - T + t + 1 for t in range(T)], [30001 - 7 * t for t in range(T)]], dtype=torch.int32)
    paged = cu.Paged([65111, 30001], T)
    pages = sum(-(-n // 64) for n in (65111, 30001))
    assert pages >= 2 * 3 * torch.cuda.get_device_properties(0).multi_processor_count  # three steps of two pages each
    table = paged.cuda
    g = torch.Generator(device="cuda").manual_seed(T + H)
    rows = (torch.randn(paged.pages * 64, 576, device="cuda", generator=g) * 0.7).to(torch.bfloat16)
    if q4:
        cache = torch.zeros(paged.pages, 64, cu.ROW, dtype=torch.uint8, device="cuda")
        binding.q4_append(rows, cache, torch.arange(paged.pages, dtype=torch.int32)[None].cuda(),
                          torch.tensor([0, len(rows)], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda())
        values = [binding.q4_read(cache, table[b:b + 1], torch.arange(n, dtype=torch.int32)[None].cuda())[0]
                  for b, n in enumerate((65111, 30001))]
    else:
        cache = rows.view(paged.pages, 64, 576)
        values = [rows[torch.from_numpy(paged.rows(b, range(n))).cuda()] for b, n in enumerate((65111, 30001))]
    q = (torch.randn(2, T, H, 576, device="cuda", generator=g) * 1.5).to(torch.bfloat16)
    lse = torch.rand(2, T, H, device="cuda", generator=g) + 4.0
    before = torch.rand(2, 65111, device="cuda", generator=g)
    acc, again = before.clone(), before.clone()
    for x in (acc, again):
        binding.evict_accumulate(q, cache, table, lens.cuda(), lse, SCALE, x)
    assert torch.equal(acc, again) and torch.equal(acc[1, 30001:], before[1, 30001:])
    check_weights_on_the_gpu(acc, before, q, lse, lens, values, f"T {T} H {H} q4 {q4}")


@pytest.mark.parametrize("q4", [False, True])
def test_steps_and_evictions_queued_without_a_synchronisation(q4):
    """The device calls of all steps stand in the stream before the first of them
    runs; what each gave is checked afterwards."""
    B, H, budget, room, steps = 3, 8, 96, 256, 4
    paged = cu.Paged([room] * B, 7)
    table = paged.cuda
    rng = np.random.default_rng(5)
    new = [[int(rng.integers(40, 90)) for _ in range(B)] for _ in range(steps)]
    rows = [cu.latents(sum(k), 100 + s) for s, k in enumerate(new)]
    q = [cu.queries(B, 1, H, 200 + s) for s in range(steps)]
    count = [[0] * B]  # slots in use before each step
    for k in new:
        count.append([min(a + c, budget) for a, c in zip(count[-1], k)])
    seen = [sum(new[s][b] for s in range(step)) if step else 0 for step in range(steps + 1) for b in range(B)]
    seen = [seen[B * s:B * s + B] for s in range(steps + 1)]  # tokens before each step
    dev = []
    for s in range(steps):
        offs = torch.tensor(np.concatenate([[0], np.cumsum(new[s])]), dtype=torch.int32).cuda()
        start = torch.tensor(count[s], dtype=torch.int32).cuda()
        flat = torch.cat([torch.from_numpy(paged.rows(b, range(count[s][b], count[s][b] + new[s][b]))) for b in range(B)]).cuda()
        slot = torch.cat([b * room + count[s][b] + torch.arange(new[s][b]) for b in range(B)]).cuda()
        tok = torch.cat([seen[s][b] + torch.arange(new[s][b]) for b in range(B)]).int().cuda()
        dev.append((rows[s].cuda(), offs, start, flat, slot, tok, q[s].cuda(), start + torch.tensor(new[s], dtype=torch.int32).cuda()))
    cache = torch.zeros(paged.pages, 64, cu.ROW if q4 else 576, dtype=torch.uint8 if q4 else torch.bfloat16, device="cuda")
    acc, pos = torch.zeros(B, room).cuda(), torch.full((B, room), -1, dtype=torch.int32).cuda()
    got = []
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    torch.cuda.set_sync_debug_mode("error")
    try:
        torch.cuda._sleep(100_000_000)  # some 50 ms: the queue fills meanwhile
        for s, (r, offs, start, flat, slot, tok, qs, n) in enumerate(dev):
            if q4:
                binding.q4_append(r, cache, table, offs, start)
            else:
                cache.view(-1, 576).index_copy_(0, flat, r)
            pos.view(-1).index_copy_(0, slot, tok)
            lens, most = n[:, None].contiguous(), max(a + c for a, c in zip(count[s], new[s]))
            o, lse = (binding.decode_dense_q4 if q4 else binding.decode_dense)(qs, cache, table, lens, SCALE, K=most)
            before = acc.clone()
            binding.evict_accumulate(qs, cache, table, lens, lse, SCALE, acc)
            p = binding.evict_plan(acc, n, budget, pos=pos, n_sink=4, n_recent=32)
            binding.evict_apply(p.src, table, (cache,))
            got.append((o, lse, before, acc, pos, p))
            acc, pos = p.acc, p.pos
    finally:
        torch.cuda.set_sync_debug_mode("default")
    held = [[] for _ in range(B)]
    for s, (o, lse, before, acc, pos, p) in enumerate(got):
        stored = cu.values(cu.quantise(rows[s])) if q4 else cu.f64(rows[s])
        at = 0
        for b in range(B):
            held[b] += [(seen[s][b] + k, stored[at + k]) for k in range(new[s][b])]
            at += new[s][b]
            assert pos[b, :len(held[b])].tolist() == [h[0] for h in held[b]]
        vals = [np.stack([v for _, v in h]) for h in held]
        if q4:
            cu.check_attention(o, lse, q[s], lambda b, t: vals[b], SCALE, f"step {s}")
        check_weights(acc, before.double().cpu().numpy(), cu.f64(q[s]), lse.double().cpu().numpy(),
                      np.array([[len(h)] for h in held]), lambda b, k: vals[b][:k], f"step {s}")
        for b in range(B):
            src = cu.plan(acc[b].cpu().tolist(), pos[b].tolist(), len(held[b]), budget, 4, 32)
            np.testing.assert_array_equal(p.src[b, :len(src)].cpu().numpy(), src)
            held[b] = [held[b][i] for i in src]
    raw = cache.cpu()
    for b in range(B):
        at = paged.rows(b, range(len(held[b])))
        have = cu.values(raw.numpy().reshape(-1, cu.ROW)[at]) if q4 else cu.f64(raw.view(-1, 576)[at])
        np.testing.assert_array_equal(have, np.stack([v for _, v in held[b]]))
