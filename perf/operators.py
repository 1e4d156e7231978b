"""The full-attention layers' operators of a hybrid model's serving step, as they are measured.

Three operators work on one paged KV cache, k and v each [N][H_kv][page][d] with page 0 the null page, a
page table [R][width] whose row 0 is the null row, and the rows' lengths kv_len [R]:

  prologue   q/k RMS norm, rotary positions, and the write of the new tokens' k and v into their pages
  attention  of the new tokens of every sequence over its pages (causal, optionally over a window)
  pages      reserving, forking, freeing, copying and compacting pages

``run`` computes them from elementary torch operations in 32 bits where ``own`` is false, and through
the package's entry points where it is true.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

FP8_MAX = 448.0  # the largest finite e4m3 value
NORM_EPS = 1e-6
KINDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------ the cases

def _prologue(name, **kw):
    base = dict(name=name, op="prologue", B=1, n_min=1, n_max=1, past_min=0, past_max=0, H_q=16, H_kv=2, d=256,
                page=64, cache="bf16", rot=64, interleaved=False, norm=True, stretch=1.0)
    base.update(kw)
    return base


def _attention(name, **kw):
    base = dict(name=name, op="attention", B=1, n_min=1, n_max=1, past_min=0, past_max=0, H_q=16, H_kv=2, d=256,
                page=64, cache="bf16", window=0)
    base.update(kw)
    return base


def _pages(name, **kw):
    base = dict(name=name, op="pages", call="turnover", rows=64, past_max=2048, layers=2, H_kv=2, d=128, page=64,
                share=0.125)
    base.update(kw)
    return base


def listed():
    return [
        # one request decoding by itself: the latency of a launch
        _prologue("prologue 1 row", past_min=900, past_max=900, page=16),
        # a full decode batch into an 8-bit cache, the whole head rotated in adjacent pairs
        _prologue("prologue 64 rows e4m3", B=64, past_min=100, past_max=4000, H_q=32, H_kv=4, d=128, cache="e4m3",
                  rot=128, interleaved=True, norm=False),
        # a mixed step's prompt chunks far into a context that the frequencies were stretched for
        _prologue("prologue chunks", B=6, n_min=500, n_max=2500, past_min=0, past_max=20000, stretch=8.0),
        # one request with a short context: latency again
        _attention("attention 1 row", past_min=776, past_max=776, page=16),
        # a ragged decode batch of the size that the library's own decode step is quoted on
        _attention("attention 64 rows", B=64, past_min=200, past_max=8191, H_kv=4),
        # few rows over long contexts held in 8 bits
        _attention("attention long e4m3", B=8, past_min=40000, past_max=131000, H_q=32, H_kv=4, d=128, page=128,
                   cache="e4m3"),
        # the verify pass of speculative decoding: a few drafted tokens a row, over a sliding window
        _attention("attention verify 4 tokens", B=32, n_min=4, n_max=4, past_min=50, past_max=3000, H_q=32, H_kv=8,
                   d=128, page=32, window=1024),
        # a mixed step: prompt chunks beside single tokens
        _attention("attention mixed", B=12, n_min=1, n_max=701, past_min=0, past_max=6000),
        # long prompt chunks: the matrix-bound end
        _attention("attention chunks", B=2, n_min=3001, n_max=4096, past_min=8000, past_max=12000, d=128),
        # a scheduler's turn between two steps: finished rows freed, others forked, every row grown by its next tokens
        _pages("pages turnover", rows=256, past_max=4000),
        # prefix pages duplicated over every layer
        _pages("pages copy", call="copy", rows=32, past_max=4096, layers=8, share=0.5),
        # the pool packed to its low pages after half of its rows ended
        _pages("pages compact", call="compact", rows=128, past_max=4096, layers=8, share=0.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prologue", "prologue", "attention", "attention", "attention", "pages"])
    d = rng.choice([64, 128, 128, 256])
    H_kv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    cache = rng.choice(["bf16", "bf16", "e4m3"])
    if op == "prologue":
        n = _log_int(rng, 1, 2000)
        B = _log_int(rng, 1, max(1, min(128, 8000 // n)))
        past = _log_int(rng, 1, max(2, min(30000, 60000 // B)))
        rot = rng.choice([d, d // 2, d // 4, d - 2 * rng.randrange(1, d // 4)])
        return dict(op=op, B=B, n_min=1 if rng.random() < 0.5 else n, n_max=n, past_min=past // 3, past_max=past,
                    H_q=H_kv * G, H_kv=H_kv, d=d, page=page, cache=cache, rot=rot, interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.5, stretch=rng.choice([1.0, 4.0, 16.0]))
    if op == "attention":
        n = rng.choice([1, 1, _log_int(rng, 2, 16), _log_int(rng, 16, 2000)])
        B = _log_int(rng, 1, max(1, min(96, 4000 // n)))
        past = _log_int(rng, 20, max(40, min(60000, 300000 // B, 20_000_000 // (n * B))))
        return dict(op=op, B=B, n_min=1 if rng.random() < 0.5 else n, n_max=n, past_min=past // 8, past_max=past,
                    H_q=H_kv * G, H_kv=H_kv, d=d, page=page, cache=cache,
                    window=rng.choice([0, 0, _log_int(rng, 16, 4096)]))
    rows = _log_int(rng, 8, 256)
    return dict(op=op, call=rng.choice(["turnover", "copy", "compact"]), rows=rows,
                past_max=_log_int(rng, 50, min(20000, 400000 // rows)), layers=rng.choice([1, 2, 4]), H_kv=H_kv, d=d,
                page=page, share=rng.choice([0.1, 0.25, 0.5]))


def _lengths(case):
    """[(new tokens, tokens before them)] of the sequences: part of the case, not of its values."""
    r = random.Random("%(op)s %(B)d %(n_min)d %(n_max)d %(past_min)d %(past_max)d" % case)
    got = [(r.randint(case["n_min"], case["n_max"]), r.randint(case["past_min"], case["past_max"]))
           for _ in range(case["B"])]
    if case["B"] > 2 and case["n_max"] > 64:
        got[-1] = (1, case["past_max"])  # a decoding row beside the chunks
    return got


def _row_lengths(case):
    r = random.Random("%(rows)d %(past_max)d" % case)
    return [r.randint(1, case["past_max"]) for _ in range(case["rows"])]


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pool(g, N, case, layers=0):
    """k and v pages with the values that earlier steps left there."""
    shape = (N, case["H_kv"], case["page"], case["d"])
    dtype = KINDS[case.get("cache", "bf16")]
    make = lambda: torch.randn(((layers,) if layers else ()) + shape, generator=g, device="cuda",  # noqa: E731
                               dtype=torch.bfloat16).to(dtype)
    return make(), make()


def _table(seed, lengths, page, extra_rows, spare, width_spare=2):
    """A page table whose rows' pages are scattered over the pool; row i + 1 belongs to sequence i."""
    need = [_ceil(n, page) for n in lengths]
    N = 1 + sum(need) + spare
    ids = list(range(1, N))
    random.Random(seed).shuffle(ids)
    width = max(need) + width_spare
    table, at = [[0] * width], 0
    for n in need:
        table.append(ids[at:at + n] + [0] * (width - n))
        at += n
    table += [[0] * width] * extra_rows
    refs = [0] * N
    for i in ids[:at]:
        refs[i] = 1
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return N, i32(table), i32([0] + list(lengths) + [0] * extra_rows), i32(refs)


def prepare(case, seed):
    g = _gen(seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] == "pages":
        return _prepare_pages(case, seed, g)
    lens = _lengths(case)
    B, T = case["B"], sum(n for n, _ in lens)
    N, table, kv_len, _ = _table(seed, [n + p for n, p in lens], case["page"], 0, 3)
    order = list(range(1, B + 1))
    random.Random(seed + 1).shuffle(order)  # sequence b sits in some row of the table
    place = [0] * (B + 1)
    for b, r in enumerate(order):
        place[r] = b + 1
    at = torch.tensor(place, device="cuda")
    table, kv_len = table[at].contiguous(), kv_len[at].contiguous()
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    k, v = _pool(g, N, case)
    s = dict(case=case, k_pages=k, v_pages=v, page_table=table, kv_len=kv_len, row=i32(order), cu_seqlens=i32(cu),
             max_new=max(n for n, _ in lens))
    if case["cache"] == "e4m3":  # what one step of the 8-bit values stands for, a head
        s["k_scale"] = 0.5 + torch.rand(case["H_kv"], generator=g, device="cuda")
        s["v_scale"] = 0.5 + torch.rand(case["H_kv"], generator=g, device="cuda")
    else:
        s["k_scale"] = s["v_scale"] = None
    H_q, H_kv, d = case["H_q"], case["H_kv"], case["d"]
    if case["op"] == "attention":
        # queries long enough that some keys stand out, as they do in trained layers
        s["q"] = (2.0 * torch.randn(T, H_q, d, generator=g, device="cuda")).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(T, H_q, dtype=torch.float32, device="cuda")
        s["scale"] = d ** -0.5
        return s
    qkv = _normal(g, T, (H_q + 2 * H_kv) * d)  # the projection's packed output
    s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, d)) for t in qkv.split([H_q * d, H_kv * d, H_kv * d], 1))
    s["q_out"] = torch.empty(T, H_q, d, dtype=torch.bfloat16, device="cuda")
    rot = case["rot"]
    f = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot
    f = 1e6 ** -f
    if case["stretch"] != 1.0:  # long wavelengths stretched, short ones kept, a ramp between them
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        f = f * (keep + (1 - keep) / case["stretch"])
    s["freqs"] = f
    s["rope_scale"] = 1.0 if case["stretch"] == 1.0 else 0.1 * math.log(case["stretch"]) + 1.0
    s["q_norm"] = (0.2 * _normal(g, d, dtype=torch.float32)).to(torch.bfloat16) if case["norm"] else None
    s["k_norm"] = (0.2 * _normal(g, d, dtype=torch.float32)).to(torch.bfloat16) if case["norm"] else None
    return s


def _prepare_pages(case, seed, g):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, page, rows = _row_lengths(case), case["page"], case["rows"]
    n = max(1, int(rows * case["share"]))
    pick = random.Random(seed).sample(range(1, rows + 1), rows)
    spare = 2 * rows + 8
    if case["call"] == "copy":
        spare += _ceil(sum(_ceil(x, page) for x in lens), 2)
    N, table, kv_len, refs = _table(seed, lens, page, n, spare)
    k, v = _pool(g, N, case, case["layers"])
    s = dict(case=case, k_pages=k, v_pages=v, page_table=table, kv_len=kv_len, refs=refs)
    if case["call"] == "copy":
        m = max(1, int(case["share"] * sum(_ceil(x, page) for x in lens)))
        live = torch.nonzero(refs > 0)[:, 0]
        free = torch.nonzero(refs == 0)[1:, 0]  # without the null page
        m = min(m, live.numel(), free.numel())
        s["src"] = live[torch.randperm(live.numel(), generator=g, device="cuda")[:m]].int()
        s["dst"] = free[torch.randperm(free.numel(), generator=g, device="cuda")[:m]].int()
    elif case["call"] == "compact":
        # the rows that ended were freed before
        at = torch.tensor(pick[:n], device="cuda")
        refs[table[at].long().flatten()] = 0
        table[at] = 0
        kv_len[at] = 0
    else:
        s["free_rows"] = i32(pick[:n])
        s["src_rows"] = i32([pick[n + i % (rows - n)] for i in range(n)])
        s["dst_rows"] = i32([rows + 1 + i for i in range(n)])
        grow = pick[n:] + [rows + 1 + i for i in range(n)]
        s["grow_rows"] = i32(grow)
        s["grow_by"] = i32([1 + (7 * r) % 4 for r in grow])
    return s


# ------------------------------------------------------------------ the plain forms

def _sequence_of(s):
    """Sequence and cache position of every token."""
    cu = s["cu_seqlens"].long()
    n = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n, output_size=s["q"].shape[0])
    rows = s["row"].long()
    pos = s["kv_len"].long()[rows][seq] - n[seq] + torch.arange(seq.numel(), device="cuda") - cu[:-1][seq]
    return seq, rows, pos


def _norm(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + NORM_EPS) * (1.0 + w.float())


def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[1]
    c, n = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _store(pages, at, off, x, scale):
    if scale is not None:
        x = (x / scale[:, None]).clamp(-FP8_MAX, FP8_MAX)
        pages.view(torch.uint8)[at, :, off] = x.to(pages.dtype).view(torch.uint8)
    else:
        pages[at, :, off] = x.to(pages.dtype)


def _plain_prologue(s):
    c = s["case"]
    seq, rows, pos = _sequence_of(s)
    angle = pos.double()[:, None] * s["freqs"]
    cos = (angle.cos() * s["rope_scale"]).float()
    sin = (angle.sin() * s["rope_scale"]).float()
    q = _rotate(_norm(s["q"].float(), s["q_norm"]), cos, sin, c["interleaved"])
    k = _rotate(_norm(s["k"].float(), s["k_norm"]), cos, sin, c["interleaved"])
    at = s["page_table"].long()[rows[seq], pos // c["page"]]
    off = pos % c["page"]
    _store(s["k_pages"], at, off, k, s["k_scale"])
    _store(s["v_pages"], at, off, s["v"].float(), s["v_scale"])
    return q.to(torch.bfloat16), s["k_pages"], s["v_pages"]


def _gathered(pages, table, scale, L):
    """[B][H_kv][L][d] in 32 bits."""
    x = pages[table.long()] if pages.dtype != torch.float8_e4m3fn else pages.view(torch.uint8)[table.long()].view(pages.dtype)
    x = x.float().transpose(1, 2).flatten(2, 3)[:, :, :L]
    return x if scale is None else x * scale[:, None, None]


def _plain_attention(s):
    c = s["case"]
    seq, rows, pos = _sequence_of(s)
    B, H_q, H_kv, d = c["B"], c["H_q"], c["H_kv"], c["d"]
    n, G = s["max_new"], H_q // H_kv
    lens = s["kv_len"].long()[rows]
    L = s["page_table"].shape[1] * c["page"]
    table = s["page_table"][rows]
    slot = torch.arange(seq.numel(), device="cuda") - s["cu_seqlens"].long()[seq]
    q = torch.zeros(B, n, H_q, d, device="cuda")
    q[seq, slot] = s["q"].float()
    q = q.view(B, n, H_kv, G, d).permute(0, 2, 3, 1, 4).reshape(B, H_kv, G * n, d)
    at = torch.full((B, n), -1, dtype=torch.long, device="cuda")
    at[seq, slot] = pos
    k = _gathered(s["k_pages"], table, s["k_scale"], L)
    w = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"]).view(B, H_kv, G, n, L)
    key = torch.arange(L, device="cuda")
    seen = (key <= at[..., None]) & (key < lens[:, None, None])
    if c["window"]:
        seen &= key > at[..., None] - c["window"]
    w.masked_fill_(~seen[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True).clamp_min(-1e30)  # a row that sees no key keeps zeros
    w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    v = _gathered(s["v_pages"], table, s["v_scale"], L)
    o = torch.matmul(w.view(B, H_kv, G * n, L), v).view(B, H_kv, G, n, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + total.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, H_q, d)[seq, slot]
    return o.to(torch.bfloat16), lse.permute(0, 3, 1, 2).reshape(B, n, H_q)[seq, slot]


def _runs(starts, counts):
    """(which run, its next value) of runs of counts[i] whole numbers from starts[i] on, one after the other."""
    which = torch.repeat_interleave(torch.arange(counts.numel(), device="cuda"), counts)
    first = counts.cumsum(0) - counts
    return which, starts[which] + torch.arange(which.numel(), device="cuda") - first[which]


def _plain_free(table, kv_len, refs, rows):
    rows = rows.long()
    gone = torch.bincount(table[rows].long().flatten(), minlength=refs.numel()).int()
    gone[0] = 0
    refs -= gone
    table[rows] = 0
    kv_len[rows] = 0


def _plain_fork(s, table, kv_len, refs):
    page = s["case"]["page"]
    src, dst = s["src_rows"].long(), s["dst_rows"].long()
    n = kv_len[src].long()
    full, part = n // page, n % page > 0
    table[dst] = torch.where(torch.arange(table.shape[1], device="cuda") < full[:, None], table[src], 0)
    shared = torch.bincount(table[dst].long().flatten(), minlength=refs.numel()).int()
    shared[0] = 0
    refs += shared
    new = torch.nonzero(refs == 0)[1:, 0][:int(part.sum())]
    old = table[src[part], full[part]].long()
    table[dst[part], full[part]] = new.int()
    refs[new] = 1
    for pages in (s["k_pages"], s["v_pages"]):
        pages[:, new] = pages[:, old]
    kv_len[dst] = n.int()


def _plain_reserve(s, table, kv_len, refs):
    page, rows = s["case"]["page"], s["grow_rows"].long()
    had = kv_len[rows].long()
    to = had + s["grow_by"].long()
    first, last = (had + page - 1) // page, (to + page - 1) // page
    which, entry = _runs(first, last - first)
    new = torch.nonzero(refs == 0)[1:, 0][:which.numel()]
    table[rows[which], entry] = new.int()
    refs[new] = 1
    kv_len[rows] = to.int()


def _plain_compact(s, table, refs):
    live = refs > 0
    ids = torch.arange(refs.numel(), device="cuda")
    m = live.sum()
    src = ids[live & (ids > m)]
    dst = ids[~live & (ids <= m) & (ids > 0)]
    remap = torch.where(live, ids, 0)
    remap[src] = dst
    for pages in (s["k_pages"], s["v_pages"]):
        pages[:, dst] = pages[:, src]
    refs[dst] = refs[src]
    refs[src] = 0
    return remap.int()[table.long()], remap.int()


def _plain_pages(s):
    call = s["case"]["call"]
    if call == "copy":
        for pages in (s["k_pages"], s["v_pages"]):
            pages[:, s["dst"].long()] = pages[:, s["src"].long()]
        return s["k_pages"], s["v_pages"]
    table, kv_len, refs = s["page_table"].clone(), s["kv_len"].clone(), s["refs"].clone()
    if call == "compact":
        table, remap = _plain_compact(s, table, refs)
        return table, refs, remap, s["k_pages"], s["v_pages"]
    _plain_free(table, kv_len, refs, s["free_rows"])
    _plain_fork(s, table, kv_len, refs)
    _plain_reserve(s, table, kv_len, refs)
    return table, kv_len, refs, s["k_pages"], s["v_pages"]


# ------------------------------------------------------------------ the package's calls

def _scratch(s, nbytes):
    """The workspace that the program keeps beside its cache; nbytes() is asked once."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(nbytes(), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_prologue(s):
    import gated_deltanet_recurrent_decode_amd as gdn
    gdn.attn_prologue(s["q"], s["k"], s["v"], s["q_out"], s["k_pages"], s["v_pages"], s["page_table"], s["kv_len"],
                      s["row"], s["cu_seqlens"], s["freqs"], interleaved=s["case"]["interleaved"],
                      rope_scale=s["rope_scale"], q_norm=s["q_norm"], k_norm=s["k_norm"], norm_eps=NORM_EPS,
                      norm_add=1.0, k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s["q_out"], s["k_pages"], s["v_pages"]


def _own_attention(s):
    import gated_deltanet_recurrent_decode_amd as gdn
    c = s["case"]
    work = _scratch(s, lambda: gdn.attn_paged_workspace_bytes(c["B"], s["q"].shape[0], s["max_new"], c["H_q"],
                                                              c["H_kv"], c["d"]))
    gdn.attn_paged(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["kv_len"], s["row"], s["cu_seqlens"],
                   s["out"], work, max_new=s["max_new"], scale=s["scale"], window=c["window"], lse=s["lse"],
                   k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s["out"], s["lse"]


def _own_pages(s):
    import gated_deltanet_recurrent_decode_amd as gdn
    call, k, v = s["case"]["call"], s["k_pages"], s["v_pages"]
    if call == "copy":
        gdn.kv_page_copy(k, v, s["src"], s["dst"])
        return k, v
    table, kv_len, refs = s["page_table"].clone(), s["kv_len"].clone(), s["refs"].clone()
    if "result" not in s:
        s["result"] = torch.empty(2, dtype=torch.int32, device="cuda")
        s["remap"] = torch.empty_like(refs)
    n = 0 if call == "compact" else max(s["src_rows"].numel(), s["grow_rows"].numel())
    work = _scratch(s, lambda: gdn.kv_page_workspace_bytes(n, table.shape[0], refs.numel()))
    if call == "compact":
        gdn.kv_page_compact(k, v, table, refs, s["remap"], s["result"], work)
        return table, refs, s["remap"], k, v
    gdn.kv_page_free(table, kv_len, refs, s["free_rows"])
    gdn.kv_page_fork(k, v, table, kv_len, refs, s["src_rows"], s["dst_rows"], s["result"], work)
    gdn.kv_page_reserve(table, kv_len, refs, s["grow_rows"], s["grow_by"], s["result"], work,
                        page_size=s["case"]["page"])
    return table, kv_len, refs, k, v


def run(state):
    op = state["case"]["op"]
    if own:
        return {"prologue": _own_prologue, "attention": _own_attention, "pages": _own_pages}[op](state)
    return {"prologue": _plain_prologue, "attention": _plain_attention, "pages": _plain_pages}[op](state)


# ------------------------------------------------------------------ what a pass cannot do without

def _pairs(n, past, window):
    """(query, key) pairs of n new tokens behind `past` others."""
    if not window:
        return n * past + n * (n + 1) // 2
    return sum(min(past + i + 1, window) for i in range(n))


def work(case):
    d, H_kv = case["d"], case["H_kv"]
    if case["op"] == "pages":
        page_bytes = 2 * case["layers"] * H_kv * case["page"] * d * 2
        need = sum(_ceil(x, case["page"]) for x in _row_lengths(case))
        n = max(1, int(case["rows"] * case["share"]))
        if case["call"] == "copy":
            return {"bytes": 2 * page_bytes * max(1, int(case["share"] * need)), "flops": 0}
        table = 4 * need + 4 * (1 + need + 2 * case["rows"] + 8)
        if case["call"] == "compact":  # of the pages that stay, as many move as the share that ended
            return {"bytes": 2 * page_bytes * need * case["share"] * (1 - case["share"]) + 2 * table, "flops": 0}
        return {"bytes": 2 * page_bytes * n + table, "flops": 0}
    lens, H_q = _lengths(case), case["H_q"]
    T = sum(n for n, _ in lens)
    cell = 2 if case["cache"] == "bf16" else 1
    if case["op"] == "prologue":
        return {"bytes": T * d * (2 * (H_q + 2 * H_kv) + 2 * H_q + cell * 2 * H_kv), "flops": 8 * T * d * (H_q + H_kv)}
    seen = sum(min(p + n, case["window"] + n - 1) if case["window"] else p + n for n, p in lens)
    return {"bytes": 2 * seen * H_kv * d * cell + T * H_q * (4 * d + 4),
            "flops": 4 * d * H_q * sum(_pairs(n, p, case["window"]) for n, p in lens)}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_prologue(s):
    c = s["case"]
    T, R, page = s["q"].shape[0], c["rot"], c["page"]
    out = [s["q"].double().clone(), s["k_pages"].to(torch.float64), s["v_pages"].to(torch.float64)]
    cu, rows = s["cu_seqlens"].tolist(), s["row"].tolist()

    def turn(x, w, pos):
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + NORM_EPS).sqrt() * (1 + w.double())
        y = x.clone()
        for j in range(R // 2):
            a, b = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + R // 2)
            angle = (pos * s["freqs"][j])[:, None]
            y[..., a] = s["rope_scale"] * (x[..., a] * angle.cos() - x[..., b] * angle.sin())
            y[..., b] = s["rope_scale"] * (x[..., b] * angle.cos() + x[..., a] * angle.sin())
        return y

    for b, r in enumerate(rows):
        lo, hi = cu[b], cu[b + 1]
        first = int(s["kv_len"][r]) - (hi - lo)
        pos = torch.arange(first, first + hi - lo, dtype=torch.float64, device="cuda")
        out[0][lo:hi] = turn(s["q"][lo:hi].double(), s["q_norm"], pos)
        cells = ((s["k"], s["k_scale"], out[1], s["k_norm"]), (s["v"], s["v_scale"], out[2], None))
        for i, (x, scale, pages, w) in enumerate(cells):
            x = x[lo:hi].double()
            x = turn(x, w, pos) if i == 0 else x
            if scale is not None:
                x = (x / scale.double()[None, :, None]).clamp(-FP8_MAX, FP8_MAX)
            p = pos.long()
            pages[s["page_table"][r][p // page].long(), :, p % page] = x
    return tuple(out)


def _exact_attention(s):
    c = s["case"]
    T, H_q = s["q"].shape[:2]
    G, page = H_q // c["H_kv"], c["page"]
    out = torch.zeros(T, H_q, c["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((T, H_q), -math.inf, dtype=torch.float64, device="cuda")
    cu, rows = s["cu_seqlens"].tolist(), s["row"].tolist()
    for b, r in enumerate(rows):
        lo, hi, L = cu[b], cu[b + 1], int(s["kv_len"][r])
        ids = s["page_table"][r][:_ceil(L, page)].long()
        i = torch.arange(L - (hi - lo), L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None]
        off = (j > i) | ((j <= i - c["window"]) if c["window"] else torch.zeros_like(j > i))
        for h in range(c["H_kv"]):
            raw = lambda p: (p[ids, h] if p.dtype == torch.bfloat16 else  # noqa: E731
                             p.view(torch.uint8)[ids, h].view(p.dtype)).to(torch.float64).flatten(0, 1)[:L]
            k, v = raw(s["k_pages"]), raw(s["v_pages"])
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for g in range(h * G, h * G + G):
                z = torch.where(off, -math.inf, s["q"][lo:hi, g].double() @ k.T * s["scale"])
                lse[lo:hi, g] = torch.logsumexp(z, 1)
                out[lo:hi, g] = torch.softmax(z, 1) @ v
    return out, lse


def _exact_pages(s):
    """The bookkeeping one entry at a time, on the host; whole pages move as they are."""
    c, page = s["case"], s["case"]["page"]
    k, v = s["k_pages"].clone(), s["v_pages"].clone()
    if c["call"] == "copy":
        moves = list(zip(s["src"].tolist(), s["dst"].tolist()))
    table, kv_len, refs = (s[n].tolist() for n in ("page_table", "kv_len", "refs"))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    if c["call"] == "turnover":
        moves = []
        for r in s["free_rows"].tolist():
            for p in table[r]:
                refs[p] -= p > 0
            table[r], kv_len[r] = [0] * len(table[r]), 0
        for a, b in zip(s["src_rows"].tolist(), s["dst_rows"].tolist()):
            for e in range(_ceil(kv_len[a], page)):
                p = table[a][e]
                if (e + 1) * page > kv_len[a]:
                    p = refs.index(0, 1)
                    moves.append((table[a][e], p))
                table[b][e] = p
                refs[p] += 1
            kv_len[b] = kv_len[a]
        for r, n in zip(s["grow_rows"].tolist(), s["grow_by"].tolist()):
            for e in range(_ceil(kv_len[r], page), _ceil(kv_len[r] + n, page)):
                table[r][e] = refs.index(0, 1)
                refs[table[r][e]] = 1
            kv_len[r] += n
    elif c["call"] == "compact":
        live = [p for p in range(1, len(refs)) if refs[p]]
        holes = [p for p in range(1, len(live) + 1) if not refs[p]]
        moves = list(zip([p for p in live if p > len(live)], holes))
        to = {0: 0, **{p: p for p in live}, **dict(moves)}
        table = [[to[p] for p in r] for r in table]
        remap = [to.get(p, 0) for p in range(len(refs))]
        for a, b in moves:
            refs[a], refs[b] = 0, refs[a]
    if moves:
        a, b = (torch.tensor(x, device="cuda") for x in zip(*moves))
        k[:, b], v[:, b] = s["k_pages"][:, a], s["v_pages"][:, a]
    if c["call"] == "copy":
        return k, v
    if c["call"] == "compact":
        return i32(table), i32(refs), i32(remap), k, v
    return i32(table), i32(kv_len), i32(refs), k, v


def exact(case, seed):
    s = prepare(case, seed)
    return {"prologue": _exact_prologue, "attention": _exact_attention, "pages": _exact_pages}[case["op"]](s)
