"""The 4-bit latent cache and the eviction operators: their cases, their plain
forms, and the calls of the library that do the same work.

Five operators share one paged latent cache (pages of 64 rows, a page table per
sequence):

* ``store``   rows of 512 latents + 64 rope values are written into the 4-bit
              cache behind what each sequence holds, and read back;
* ``sparse``  split-K decode over index lists, reading the 4-bit cache;
* ``dense``   split-K decode over every visible position, reading it;
* ``weigh``   the attention weight each cached position has received is
              accumulated (over a bf16 or a 4-bit cache);
* ``evict``   the positions with the least of it leave: a plan of moves, and
              the moves applied to the paged buffers.

A row of the 4-bit cache has 416 bytes: 256 of codes, 16 bf16 scales, 64 bf16
rope values.  Group g holds latents 32 g .. 32 g + 31: value = (code - 8) *
scale[g], codes 1 .. 15.  The scale is the least number of four significant
bits that is at least max|x| / 7, and codes round x / scale to nearest even.
Eight codes share a little-endian 32-bit word: nibble k < 4 is value 2 k of the
eight, nibble k + 4 is value 2 k + 1.
"""
import math
import random

import torch

own = False

DC, DR, D, PAGE = 512, 64, 576, 64
GROUP, GROUPS = 32, 16
ROW_Q4 = DC // 2 + 2 * GROUPS + 2 * DR  # 416
IX_DIM = 128
DEV = "cuda"


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a batch of 64: each sequence gains one token
        {"name": "store_step", "op": "store", "B": 64, "rows": 64, "most": 1, "ctx": 16384, "lens_seed": 1},
        # a batch of prompts of unequal lengths enters the cache
        {"name": "store_prompts", "op": "store", "B": 7, "rows": 46080, "most": 32768, "ctx": 2048, "lens_seed": 2},
        # one request at a long context: latency counts
        {"name": "sparse_single", "op": "sparse", "B": 1, "T": 1, "H": 16, "K": 2048, "ctx_lo": 65536, "ctx_hi": 65536, "lens_seed": 3},
        # speculative verify of a few drafts, odd list width
        {"name": "sparse_verify", "op": "sparse", "B": 3, "T": 5, "H": 8, "K": 1999, "ctx_lo": 9000, "ctx_hi": 46080, "lens_seed": 4},
        # a full batch of decodes
        {"name": "sparse_batched", "op": "sparse", "B": 64, "T": 1, "H": 16, "K": 2048, "ctx_lo": 16384, "ctx_hi": 16384, "lens_seed": 5},
        # many heads, contexts log-uniform down to half a list
        {"name": "sparse_mixed", "op": "sparse", "B": 60, "T": 1, "H": 64, "K": 2048, "ctx_lo": 1024, "ctx_hi": 131072, "lens_seed": 6},
        # drafts of one long sequence verified against all of it
        {"name": "dense_verify", "op": "dense", "B": 1, "T": 9, "H": 8, "ctx_lo": 46089, "ctx_hi": 46089, "lens_seed": 7},
        # a ragged batch reading its whole contexts: bandwidth counts
        {"name": "dense_batched", "op": "dense", "B": 32, "T": 1, "H": 16, "ctx_lo": 4096, "ctx_hi": 65536, "lens_seed": 8},
        # the weights of a verify step over the bf16 cache
        {"name": "weigh_verify", "op": "weigh", "B": 1, "T": 9, "H": 8, "ctx_lo": 46089, "ctx_hi": 46089, "lens_seed": 9, "q4": False},
        # the weights of a ragged batch over the 4-bit cache
        {"name": "weigh_batched_q4", "op": "weigh", "B": 24, "T": 1, "H": 16, "ctx_lo": 4096, "ctx_hi": 65536, "lens_seed": 10, "q4": True},
        # one sequence that went a little over its budget
        {"name": "evict_single", "op": "evict", "B": 1, "ctx_lo": 8192 + 256, "ctx_hi": 8192 + 256, "K": 8192, "sink": 4, "recent": 512, "lens_seed": 11},
        # a batch cut back hard: half its rows leave
        {"name": "evict_batched", "op": "evict", "B": 16, "ctx_lo": 12000, "ctx_hi": 32768, "K": 8192, "sink": 64, "recent": 1024, "lens_seed": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "sparse", "sparse", "dense", "dense", "weigh", "weigh", "evict"])
    c = {"op": op, "lens_seed": rng.randrange(1 << 20)}
    if op == "store":
        c["B"] = _log(rng, 1, 64)
        c["rows"] = c["B"] * _log(rng, 1, 46080 // c["B"])
        c["most"] = min(46080, 4 * (c["rows"] // c["B"]))
        c["ctx"] = _log(rng, 1, 16384)
        return c
    c["B"] = _log(rng, 1, 64) if op in ("sparse", "dense") else _log(rng, 1, 24)
    if op == "evict":
        c["B"] = min(c["B"], 16)
        c["ctx_hi"] = _log(rng, 64, 32768)
        c["ctx_lo"] = max(1, c["ctx_hi"] // rng.choice([1, 2, 8]))
        c["K"] = max(1, int(c["ctx_hi"] * rng.uniform(0.2, 1.1)))
        c["sink"] = rng.randrange(0, 1 + min(64, c["K"] // 4))
        c["recent"] = rng.randrange(0, 1 + c["K"] // 4)
        return c
    c["H"] = rng.choice([1, 3, 8, 16, 16, 24, 32, 64])
    c["T"] = rng.choice([1, 1, 2, 4, 9]) if c["B"] <= 8 else 1
    most = 16 * 65536 // c["B"] * 16 // max(16, c["H"] * c["T"])
    c["ctx_hi"] = _log(rng, 65, min(131072, max(66, most)))
    c["ctx_lo"] = max(c["T"] + 1, c["ctx_hi"] // rng.choice([1, 4, 32]))
    if op == "sparse":
        c["K"] = _log(rng, 1, 2048)
    if op == "weigh":
        c["q4"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------- sizes of a case
def _lens(c):
    """Tokens that each sequence holds, log-uniform, from the case alone."""
    r = random.Random(c["lens_seed"])
    return [max(c.get("T", 1), _log(r, c["ctx_lo"], c["ctx_hi"])) for _ in range(c["B"])]


def _new_rows(c):
    """New rows per sequence (their sum is c["rows"], none over c["most"])."""
    r, B = random.Random(c["lens_seed"]), c["B"]
    w = [r.random() ** 2 + 0.02 for _ in range(B)]
    n = [min(c["most"], int(c["rows"] * x / sum(w))) for x in w]
    for b in range(B):
        n[b] += min(c["rows"] - sum(n), c["most"] - n[b])
    return n


def _starts(c):
    r = random.Random(c["lens_seed"] + 1)
    return [r.randrange(c["ctx"]) for _ in range(c["B"])]


def work(case):
    c = case
    if c["op"] == "store":
        n = c["rows"]
        return {"bytes": n * (2 * D + ROW_Q4) * 2, "flops": n * DC * 4}
    lens = _lens(c)
    if c["op"] == "evict":
        size = 0
        for n in lens:
            moved = max(0, n - c["K"]) * c["K"] / n
            size += n * 8 + (min(n, c["K"]) + max(lens) * 2) * 4 + moved * 2 * 2 * (D + IX_DIM)
        return {"bytes": size, "flops": sum(lens)}
    B, T, H = c["B"], c["T"], c["H"]
    if c["op"] == "sparse":
        seen = sum(min(c["K"], n) for n in lens) * T
        rows = sum(min(n, T * min(c["K"], n)) for n in lens)
        lists = B * T * c["K"] * 4 + rows * 4
    else:
        seen = sum(n - T + t + 1 for n in lens for t in range(T))
        rows = sum(lens)
        lists = B * T * 4 + rows // PAGE * 4
    q, o, stat = B * T * H * D * 2, B * T * H * DC * 2, B * T * H * 4
    if c["op"] == "weigh":
        return {"bytes": rows * (ROW_Q4 if c["q4"] else 2 * D) + lists + q + stat + rows * 8,
                "flops": 2.0 * seen * H * D}
    return {"bytes": rows * ROW_Q4 + lists + q + o + stat, "flops": 2.0 * seen * H * (D + DC)}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _pages(lens, g):
    """Page table int32 [B, most pages] over a shuffled pool (-1: no page), and the pool's size."""
    need = [(n + PAGE - 1) // PAGE for n in lens]
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    perm = torch.randperm(sum(need), generator=g, device=DEV).to(torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, sum(need)


def _latents(rows, g):
    """Latent rows: unit-scale values whose size varies from dimension to dimension, rope values beside them."""
    size = 0.3 + torch.rand(D, generator=g, device=DEV)
    x = torch.empty(rows, D, dtype=torch.bfloat16, device=DEV)
    for at in range(0, rows, 1 << 18):
        n = min(1 << 18, rows - at)
        x[at:at + n] = (torch.randn(n, D, generator=g, device=DEV) * size).to(torch.bfloat16)
    return x


def _cache(pages, q4, g):
    x = _latents(pages * PAGE, g)
    if not q4:
        return x.view(pages, PAGE, D)
    out = torch.empty(pages * PAGE, ROW_Q4, dtype=torch.uint8, device=DEV)
    for at in range(0, x.shape[0], 1 << 17):
        out[at:at + (1 << 17)] = _pack(x[at:at + (1 << 17)])
    return out.view(pages, PAGE, ROW_Q4)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "store":
        new, start = _new_rows(c), _starts(c)
        s["table"], pages = _pages([a + n for a, n in zip(start, new)], g)
        s["cache"] = torch.zeros(pages, PAGE, ROW_Q4, dtype=torch.uint8, device=DEV)
        s["rows"] = _latents(c["rows"], g)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
        # the positions that were written, as lists for the read
        width = max(new)
        i = torch.arange(width, device=DEV, dtype=torch.int32)[None]
        n = s["cu"].diff()[:, None]
        s["list"] = torch.where(i < n, s["start"][:, None] + i, -1).to(torch.int32).contiguous()
        s["out"] = torch.empty(c["B"], width, D, dtype=torch.bfloat16, device=DEV)
        return s
    lens = _lens(c)
    s["table"], pages = _pages(lens, g)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if c["op"] == "evict":
        B, most = c["B"], max(lens)
        s["n"], s["latents"] = n, _cache(pages, False, g)
        s["keys"] = torch.randn(pages, PAGE, IX_DIM, generator=g, device=DEV, dtype=torch.bfloat16)
        # weights received so far: few positions hold most of them, many tie at zero
        w = torch.rand(B, most, generator=g, device=DEV)
        s["acc"] = torch.where(w < 0.05, 0.0, (1 - w) ** -1.5 * 1e-3)
        # slots hold positions in order, but for a first part that earlier evictions shuffled
        gaps = torch.randint(1, 4, (B, most), generator=g, device=DEV)
        pos = gaps.cumsum(1).to(torch.int32) - 1
        for b, m in enumerate(lens):
            part = 3 * m // 4
            order = torch.randperm(max(part - c["sink"], 0), generator=g, device=DEV) + c["sink"]
            if part > c["sink"]:
                pos[b, c["sink"]:part] = pos[b, order]
        s["pos"] = pos.contiguous()
        return s
    B, T, H = c["B"], c["T"], c["H"]
    s["q"] = (torch.randn(B, T, H, D, generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(D)
    s["cache"] = _cache(pages, c["op"] != "weigh" or c["q4"], g)
    if c["op"] == "sparse":
        K, idx = c["K"], []
        for m in lens:
            order = torch.rand(T, m, generator=g, device=DEV).argsort(-1)[:, :K].to(torch.int32)
            idx.append(torch.nn.functional.pad(order, (0, K - order.shape[1]), value=-1))
        s["idx"] = torch.stack(idx).contiguous()
    else:
        s["lens"] = (n[:, None] - T + 1 + torch.arange(T, device=DEV, dtype=torch.int32)).to(torch.int32).contiguous()
        s["K"] = max(lens)
    if c["op"] == "weigh":
        s["acc"] = torch.rand(B, s["K"], generator=g, device=DEV) ** 4 * 0.01
        s["lse"] = _dense_lse(s)
        return s
    s["o"] = torch.empty(B, T, H, DC, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty(B, T, H, dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms
def _pack(x):
    """bf16 rows [N, 576] -> 4-bit rows uint8 [N, 416]."""
    v = x[:, :DC].float().view(-1, GROUPS, GROUP)
    most = v.abs().amax(-1)
    m, e = torch.frexp(most / torch.full_like(most, 7.0))  # a true quotient: 7 times a scale must give that scale
    scale = torch.ldexp((m * 16).ceil() / 16, e)
    code = (v / scale.clamp_min(1e-38)[..., None]).round() + 8
    w = code.to(torch.uint8).view(-1, DC // 8, 4, 2)          # [word, k, 0 / 1]: values 2 k, 2 k + 1
    nib = w.transpose(-1, -2).reshape(-1, DC // 8, 8)         # nibble k: 2 k; nibble 4 + k: 2 k + 1
    codes = (nib[..., 0::2] | (nib[..., 1::2] << 4)).reshape(-1, DC // 2)
    return torch.cat([codes, scale.to(torch.bfloat16).view(torch.uint8).view(-1, 2 * GROUPS),
                      x[:, DC:].contiguous().view(torch.uint8).view(-1, 2 * DR)], 1)


def _unpack(rows):
    """4-bit rows uint8 [..., 416] -> values fp32 [..., 576]."""
    lead = rows.shape[:-1]
    b = rows[..., :DC // 2]
    nib = torch.stack([b & 15, b >> 4], -1).reshape(*lead, DC // 8, 2, 4)
    code = nib.transpose(-1, -2).reshape(*lead, GROUPS, GROUP).float() - 8
    scale = rows[..., DC // 2:DC // 2 + 2 * GROUPS].contiguous().view(torch.bfloat16).float()
    rope = rows[..., DC // 2 + 2 * GROUPS:].contiguous().view(torch.bfloat16).float()
    return torch.cat([(code * scale[..., None]).reshape(*lead, DC), rope], -1)


def _row_of(table, pos):
    """Positions [B, ...] (-1: none) -> rows of the paged pool (row 0 for none)."""
    p = pos.clamp_min(0).long()
    flat = p.view(p.shape[0], -1)
    page = table.gather(1, flat // PAGE).long()
    return (page * PAGE + flat % PAGE).clamp_min(0).view(p.shape)


def _values(s, rows):
    cache = s["cache"].view(-1, s["cache"].shape[-1])[rows]
    return _unpack(cache) if s["cache"].dtype == torch.uint8 else cache.float()


def _attend(q, kv, seen, scale):
    """Plain attention in fp32: q [X, H, 576], kv [X, N, 576], seen [X, H or 1, N]; o and lse."""
    a = torch.matmul(q.float(), kv.transpose(1, 2)) * scale
    a = a.masked_fill(~seen, -math.inf)
    top = a.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(a - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, kv[..., :DC]) / total.clamp_min(1e-38)
    return o, (top + torch.log(total)).squeeze(-1)


def _dense_rows(s):
    c = s["case"]
    B, T, H, K = c["B"], c["T"], c["H"], s["K"]
    i = torch.arange(K, device=DEV)
    kv = _values(s, _row_of(s["table"], i[None].expand(B, K).clamp_max(s["table"].shape[1] * PAGE - 1)))
    seen = (i < s["lens"][..., None]).repeat_interleave(H, 1)  # [B, T H, K]
    # values behind a sequence's end belong to no one: they count as zeros
    kv = kv.masked_fill_((i >= s["lens"].amax(1)[:, None])[..., None], 0.0)
    return kv, seen


def _dense_lse(s):
    kv, seen = _dense_rows(s)
    q = s["q"].view(s["q"].shape[0], -1, D)
    a = (torch.matmul(q.float(), kv.transpose(1, 2)) * s["scale"]).masked_fill_(~seen, -math.inf)
    return torch.logsumexp(a, -1).view(s["q"].shape[:3]).contiguous()


def _plain_store(s):
    n = s["cu"].diff()
    b = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n.long())
    pos = s["start"][b] + torch.arange(s["rows"].shape[0], device=DEV) - s["cu"][b]
    rows = s["table"][b, pos // PAGE].long() * PAGE + pos % PAGE
    flat = s["cache"].view(-1, ROW_Q4)
    flat[rows] = _pack(s["rows"])
    got = _unpack(flat[_row_of(s["table"], s["list"])])
    return got.masked_fill(s["list"][..., None] < 0, 0.0).to(torch.bfloat16)


def _plain_sparse(s):
    B, T, H, K = *s["q"].shape[:3], s["idx"].shape[2]
    kv = _values(s, _row_of(s["table"], s["idx"]))
    o, lse = _attend(s["q"].view(B * T, H, D), kv.view(B * T, K, D), (s["idx"] >= 0).view(B * T, 1, K), s["scale"])
    return o.view(B, T, H, DC).to(torch.bfloat16), lse.view(B, T, H)


def _plain_dense(s):
    B, T, H = s["q"].shape[:3]
    kv, seen = _dense_rows(s)
    o, lse = _attend(s["q"].view(B, T * H, D), kv, seen, s["scale"])
    return o.view(B, T, H, DC).to(torch.bfloat16), lse.view(B, T, H)


def _plain_weigh(s):
    B = s["q"].shape[0]
    kv, seen = _dense_rows(s)
    a = torch.matmul(s["q"].view(B, -1, D).float(), kv.transpose(1, 2)) * s["scale"]
    w = torch.exp(a - s["lse"].view(B, -1, 1)).masked_fill(~seen, 0.0)
    s["acc"] += w.sum(1)
    return s["acc"]


def _plain_evict(s):
    c, acc, pos = s["case"], s["acc"], s["pos"]
    B, most = acc.shape
    K, i = c["K"], torch.arange(acc.shape[1], device=DEV)[None]
    n = s["n"].long()[:, None]
    live = i < n
    end = pos.masked_fill(~live, -1).amax(1, keepdim=True) + 1
    safe = live & ((pos < c["sink"]) | (pos >= end - c["recent"]))
    # protected rows first, then by weight; a stable sort leaves ties to the smaller slot
    key = torch.where(safe, math.inf, acc.nan_to_num(nan=-math.inf, posinf=3.4e38)).masked_fill(~live, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(live.gather(1, order).logical_not().to(torch.int8), dim=1, stable=True).indices)
    rank = torch.empty_like(order).scatter_(1, order, i.expand(B, most).contiguous())
    keep = live & (rank < K)
    m = n.clamp_max(K)
    hole, mover = (i < m) & ~keep, (i >= m) & keep
    by_rank = torch.zeros(B, most + 1, dtype=torch.long, device=DEV)
    at = torch.where(mover, mover.cumsum(1) - 1, most)
    by_rank.scatter_(1, at, i.expand(B, most).contiguous())
    fill = by_rank.gather(1, (hole.cumsum(1) - 1).clamp_min(0))
    src = torch.where(hole, fill, i.expand(B, most)).masked_fill(i >= m, -1)
    acc_new = acc.gather(1, src.clamp_min(0)).masked_fill(src < 0, 0.0)
    pos_new = pos.gather(1, src.clamp_min(0)).masked_fill(src < 0, -1)
    b, slot = torch.nonzero(hole, as_tuple=True)
    to = s["table"][b, slot // PAGE].long() * PAGE + slot % PAGE
    come = src[b, slot]
    come = s["table"][b, come // PAGE].long() * PAGE + come % PAGE
    for buf in (s["latents"], s["keys"]):
        flat = buf.view(-1, buf.shape[-1])
        flat[to] = flat[come]
    src = torch.nn.functional.pad(src, (0, max(0, K - most)), value=-1)[:, :K].to(torch.int32)
    return {"src": src, "n": m.squeeze(1).to(torch.int32), "acc": acc_new, "pos": pos_new.to(torch.int32),
            "latents": s["latents"], "keys": s["keys"]}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"store": _plain_store, "sparse": _plain_sparse, "dense": _plain_dense,
                "weigh": _plain_weigh, "evict": _plain_evict}[op](s)
    from sparse_mla_decode_partial_b200 import binding
    if op == "store":
        binding.q4_append(s["rows"], s["cache"], s["table"], s["cu"], s["start"])
        return binding.q4_read(s["cache"], s["table"], s["list"], out=s["out"])
    if op == "sparse":
        return binding.decode_q4(s["q"], s["cache"], s["table"], s["idx"], s["scale"],
                                 o=s["o"], lse=s["lse"])
    if op == "dense":
        return binding.decode_dense_q4(s["q"], s["cache"], s["table"], s["lens"], s["scale"], K=s["K"],
                                       o=s["o"], lse=s["lse"])
    if op == "weigh":
        return binding.evict_accumulate(s["q"], s["cache"], s["table"], s["lens"], s["lse"], s["scale"], s["acc"])
    c = s["case"]
    plan = binding.evict_plan(s["acc"], s["n"], c["K"], pos=s["pos"], n_sink=c["sink"], n_recent=c["recent"])
    binding.evict_apply(plan.src, s["table"], (s["latents"], s["keys"]))
    return {"src": plan.src, "n": plan.n, "acc": plan.acc, "pos": plan.pos, "latents": s["latents"], "keys": s["keys"]}


# ---------------------------------------------------------------- the definitions, in 64 bits
def _exact_rows(s, b, n):
    """Values of positions 0 .. n - 1 of sequence b, fp64 [n, 576]."""
    i = torch.arange(n, device=DEV)
    raw = s["cache"].view(-1, s["cache"].shape[-1])[s["table"][b].long()[i // PAGE] * PAGE + i % PAGE]
    return raw.double() if raw.dtype == torch.bfloat16 else _exact_decode(raw)


def _exact_decode(raw):
    out = torch.empty(raw.shape[0], D, dtype=torch.float64, device=DEV)
    word = raw[:, :DC // 2].contiguous().view(torch.int32).long()
    scale = raw[:, 256:288].contiguous().view(torch.bfloat16).double().repeat_interleave(4, 1)
    for j in range(8):
        out[:, j:DC:8] = (((word >> (4 * (j // 2 + 4 * (j % 2)))) & 15) - 8).double() * scale
    out[:, DC:] = raw[:, 288:].contiguous().view(torch.bfloat16).double()
    return out


def _exact_store(s):
    B, width = s["list"].shape
    out = torch.zeros(B, width, D, dtype=torch.float64, device=DEV)
    cu = s["cu"].tolist()
    for b in range(B):
        x = s["rows"][cu[b]:cu[b + 1]].double()
        v = x[:, :DC].reshape(-1, GROUPS, GROUP)
        bound = v.abs().max(-1).values / 7
        unit = torch.exp2(torch.floor(torch.log2(bound.clamp_min(1e-300))) - 3)  # one step of four significant bits
        unit = torch.where(bound / unit >= 16, 2 * unit, torch.where(bound / unit < 8, unit / 2, unit))
        scale = torch.ceil(bound / unit) * unit
        safe = torch.where(scale > 0, scale, 1.0)[..., None]
        low = torch.floor(v / safe)
        rest = v - low * safe
        up = (2 * rest > safe) | ((2 * rest == safe) & (low % 2 != 0))
        out[b, :cu[b + 1] - cu[b], :DC] = ((low + up) * scale[..., None]).reshape(-1, DC)
        out[b, :cu[b + 1] - cu[b], DC:] = x[:, DC:]
    return out


def _exact_attention(s):
    B, T, H = s["q"].shape[:3]
    o = torch.zeros(B, T, H, DC, dtype=torch.float64, device=DEV)
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device=DEV)
    lens = _lens(s["case"])
    for b in range(B):
        rows = _exact_rows(s, b, lens[b])
        for t in range(T):
            if "idx" in s:
                i = s["idx"][b, t].long()
                kv = rows[i[i >= 0]]
            else:
                kv = rows[:int(s["lens"][b, t])]
            if kv.shape[0]:
                a = s["q"][b, t].double() @ kv.T * s["scale"]
                lse[b, t] = torch.logsumexp(a, -1)
                o[b, t] = torch.softmax(a, -1) @ kv[:, :DC]
    return o, lse


def _exact_weigh(s):
    acc = s["acc"].double()
    lens = _lens(s["case"])
    for b in range(s["q"].shape[0]):
        rows = _exact_rows(s, b, lens[b])
        for t in range(s["q"].shape[1]):
            n = int(s["lens"][b, t])
            a = s["q"][b, t].double() @ rows[:n].T * s["scale"]
            acc[b, :n] += torch.exp(a - s["lse"][b, t].double()[:, None]).sum(0)
    return acc


def _exact_evict(s):
    c = s["case"]
    B, most = s["acc"].shape
    K = c["K"]
    src = torch.full((B, K), -1, dtype=torch.int32, device=DEV)
    acc = torch.zeros(B, most, dtype=torch.float64, device=DEV)
    pos = torch.full((B, most), -1, dtype=torch.int32, device=DEV)
    n_new = []
    latents, keys = s["latents"].double().view(-1, D), s["keys"].double().view(-1, IX_DIM)
    for b, n in enumerate(s["n"].tolist()):
        a, p = s["acc"][b, :n].tolist(), s["pos"][b, :n].tolist()
        end = max(p) + 1
        order = sorted(range(n), key=lambda i: (not (p[i] < c["sink"] or p[i] >= end - c["recent"]),
                                                -a[i] if not (p[i] < c["sink"] or p[i] >= end - c["recent"]) else 0.0, i))
        kept = set(order[:K])
        m = min(n, K)
        movers = iter(sorted(i for i in kept if i >= m))
        come = torch.tensor([i if i in kept else next(movers) for i in range(m)], device=DEV)
        n_new.append(m)
        src[b, :m] = come.to(torch.int32)
        acc[b, :m], pos[b, :m] = s["acc"][b, come].double(), s["pos"][b, come]
        slot = torch.arange(m, device=DEV)
        t = s["table"][b].long()
        for buf in (latents, keys):
            buf[t[slot // PAGE] * PAGE + slot % PAGE] = buf[t[come // PAGE] * PAGE + come % PAGE]
    return {"src": src, "n": torch.tensor(n_new, dtype=torch.int32, device=DEV), "acc": acc, "pos": pos,
            "latents": latents.view(s["latents"].shape), "keys": keys.view(s["keys"].shape)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "store":
        return _exact_store(s)
    if op == "weigh":
        return _exact_weigh(s)
    return _exact_evict(s) if op == "evict" else _exact_attention(s)
