"""Linear attention over state slots, and attention over a shared prefix, as they are measured.

The linear layers keep a state S [d_k][d_v] a value head in slots [N][H_v][d_k][d_v] (fp32, slot 0 the null
slot).  With a log decay g a head (fixed, or one for every token):

  S_t = exp(g_t) S_(t-1) + k_t v_t^T,   o_t = q_scale S_t^T q_t

  step     one token a row from its read slot to its write slot, or a few whose states are all kept
  prefill  packed prompts, each from its read slot (0: from zeros) to its write slot

The full-attention layers keep k and v in pages [N][H_kv][page][d].  Where the first positions of a group of
sequences are the same cells (rows forked from one prompt),

  shared   attention of every new token over its row, the common positions of a group computed once for all

``run`` computes them from elementary torch operations in 32 bits where ``own`` is false (decays are summed and
positions' weights formed in 64), and through the package's entry points where it is true.  ``exact`` is the
definition in 64 bits.
"""
import math
import random

import torch

own = False

KINDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
CHUNK = 64  # tokens of a chunk of the plain form


# ------------------------------------------------------------------ the cases

def _step(name, **kw):
    base = dict(name=name, op="step", B=1, T=1, H_k=16, H_v=16, d_k=128, d_v=128, per_token=False)
    base.update(kw)
    return base


def _prefill(name, **kw):
    base = dict(name=name, op="prefill", B=1, n_min=1, n_max=1, H_k=16, H_v=16, d_k=128, d_v=128, per_token=False,
                fresh=0.5)
    base.update(kw)
    return base


def _shared(name, **kw):
    base = dict(name=name, op="shared", B=8, K=1, n_min=1, n_max=1, prefix_min=1000, prefix_max=1000, own_min=1,
                own_max=100, H_q=16, H_kv=2, d=128, page=64, cache="bf16", window=0)
    base.update(kw)
    return base


def listed():
    return [
        # one request decoding by itself: the latency of a launch
        _step("step 1 row"),
        # a decode batch of the size that the library's own decode step is quoted on, twin slots
        _step("step 64 rows", B=64, per_token=True),
        # the verify pass of speculative decoding: the state after every drafted token is kept, heads in groups
        _step("step verify 4 tokens", B=24, T=4, H_k=8, H_v=32, d_v=64, per_token=True),
        # a short prompt alone: latency again
        _prefill("prefill short", n_min=77, n_max=77, fresh=1.0),
        # one long prompt, fixed decays: few heads to spread over the chip
        _prefill("prefill long", n_min=8191, n_max=8191, fresh=1.0),
        # a scheduler's batch of prompts and prompt chunks of all lengths
        _prefill("prefill 16 ragged", B=16, n_min=100, n_max=1500, per_token=True),
        # long prompts with key heads shared by four value heads of 64 columns
        _prefill("prefill grouped", B=4, n_min=5000, n_max=9000, H_k=8, H_v=32, d_v=64, per_token=True),
        # a few continuations of one short prompt: latency
        _shared("shared 8 rows", prefix_min=500, prefix_max=500, own_max=40, d=256, page=16),
        # a batch sampled from one long prompt
        _shared("shared 64 rows", B=64, prefix_min=8000, prefix_max=8000, own_min=50, own_max=800, H_q=32, H_kv=4),
        # three system prompts in an 8-bit cache, each with its requests
        _shared("shared 3 groups e4m3", B=48, K=3, prefix_min=4000, prefix_max=30000, own_min=100, own_max=1000,
                H_q=32, H_kv=8, page=128, cache="e4m3"),
        # drafted tokens verified behind one prompt
        _shared("shared verify 4 tokens", B=32, n_min=4, n_max=4, prefix_min=6001, prefix_max=6001, own_min=10,
                own_max=500, H_kv=4, d=256),
        # questions of some hundred tokens about one long document: the matrix-bound end
        _shared("shared chunks", n_min=100, n_max=600, prefix_min=12000, prefix_max=12000, own_min=0, own_max=200,
                H_q=32, H_kv=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "prefill", "prefill", "shared", "shared"])
    if op == "shared":
        d, H_kv, G = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
        n = rng.choice([1, 1, 1, _log_int(rng, 2, 8), _log_int(rng, 16, 500)])
        B = _log_int(rng, 2, max(3, min(96, 2400 // n)))
        prefix = _log_int(rng, 100, min(40000, 130_000_000_000 // (d * H_kv * G * n * B)))
        return dict(op=op, B=B, K=rng.randint(1, max(1, min(4, B // 2))), n_min=1 if rng.random() < 0.5 else n, n_max=n,
                    prefix_min=prefix // rng.choice([1, 1, 3]), prefix_max=prefix, own_min=0,
                    own_max=_log_int(rng, 4, max(8, min(3000, 60000 // B))), H_q=H_kv * G, H_kv=H_kv, d=d,
                    page=rng.choice([16, 32, 64, 128, 256]), cache=rng.choice(["bf16", "bf16", "e4m3"]),
                    window=rng.choice([0, 0, 0, _log_int(rng, 100, 8000)]))
    H_k, r = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 1, 2, 4])
    heads = dict(H_k=H_k, H_v=H_k * r, d_k=rng.choice([64, 128, 128]), d_v=rng.choice([64, 128, 128]),
                 per_token=rng.random() < 0.5)
    if op == "step":
        T = rng.choice([1, 1, 1, rng.randint(2, 6)])
        return dict(op=op, B=_log_int(rng, 1, max(2, min(160, 1000 // (H_k * r * T)))), T=T, **heads)
    most = min(24000, 7_000_000_000 // (H_k * r * heads["d_k"] * heads["d_v"]))  # tokens
    n = _log_int(rng, 1, min(9000, most))
    return dict(op=op, B=_log_int(rng, 1, min(32, most // n)), n_min=max(1, n // rng.choice([1, 2, 10])),
                n_max=n, fresh=rng.choice([0.0, 0.5, 1.0]), **heads)


def _lengths(case):
    """New tokens of each sequence: part of the case, not of its values."""
    r = random.Random("%(op)s %(B)d %(n_min)d %(n_max)d" % case)
    return [r.randint(case["n_min"], case["n_max"]) for _ in range(case["B"])]


def _groups(case):
    """(members of each group, common positions of each group, own tokens before the new ones of each sequence)."""
    r = random.Random("%(op)s %(B)d %(K)d %(prefix_max)d %(own_max)d" % case)
    B, K = case["B"], case["K"]
    cuts = [0] + sorted(r.sample(range(1, B), K - 1)) + [B]
    members = [b - a for a, b in zip(cuts, cuts[1:])]
    prefix = [r.randint(case["prefix_min"], case["prefix_max"]) for _ in range(K)]
    return members, prefix, [r.randint(case["own_min"], case["own_max"]) for _ in range(B)]


def _ceil(a, b):
    return -(-a // b)


def _fresh(case):
    """Which sequences of a prefill start from zeros."""
    r = random.Random("fresh %(B)d %(n_max)d" % case)
    return [r.random() < case["fresh"] for _ in range(case["B"])]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return _i32(cu)


def _prepare_linear(case, seed, g):
    """The projection's packed output with q, k and v as views of it, decays, and a pool of states in use."""
    B, H_k, H_v, d_k, d_v = (case[n] for n in ("B", "H_k", "H_v", "d_k", "d_v"))
    step = case["op"] == "step"
    lens = [case["T"]] * B if step else _lengths(case)
    T = sum(lens)
    qkv = _normal(g, T, 2 * H_k * d_k + H_v * d_v)
    qkv = torch.nn.functional.silu(qkv).to(torch.bfloat16)
    q, k, v = qkv.split([H_k * d_k, H_k * d_k, H_v * d_v], 1)
    s = dict(case=case, q=q.unflatten(1, (H_k, d_k)), k=k.unflatten(1, (H_k, d_k)), v=v.unflatten(1, (H_v, d_v)),
             q_scale=d_k ** -0.5)
    # slopes a factor apart from head to head, as trained decays have them; a gate of each token on top
    slope = -torch.exp2(-8.0 * (torch.arange(H_v, device="cuda") + 1) / H_v)
    s["g"] = slope * torch.nn.functional.softplus(2.0 * _normal(g, T, H_v)) if case["per_token"] else slope
    if step:
        shape = (B, T // B)
        s.update({n: s[n].unflatten(0, shape) for n in "qkv"})
        s["g"] = s["g"].unflatten(0, shape) if case["per_token"] else s["g"]
    N = 1 + B * (T // B + 1 if step else 2)
    s["state"] = 0.5 * _normal(g, N, H_v, d_k, d_v)
    s["state"][0] = 0
    ids = list(range(1, N))
    random.Random(seed).shuffle(ids)
    s["read_slot"] = _i32([0 if not step and new else i for i, new in zip(ids, [False] * B if step else _fresh(case))])
    if step and T > B:
        s["token_slots"] = _i32(ids[B:]).unflatten(0, shape)
    else:
        s["write_slot"] = _i32(ids[B:])
    s["cu_seqlens"] = _cu(lens)
    s["out"] = torch.empty(s["v"].shape, dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_shared(case, seed, g):
    lens, page, B = _lengths(case), case["page"], case["B"]
    members, prefix, past = _groups(case)
    H_q, H_kv, d, T = case["H_q"], case["H_kv"], case["d"], sum(lens)
    rows, copies, at, b = [], [], 0, 0

    def take(n):
        nonlocal at
        at += n
        return list(range(at - n + 1, at + 1))

    for m, p in zip(members, prefix):
        common, partly = take(p // page), None
        for _ in range(m):
            need = _ceil(p + past[b] + lens[b], page)
            mine = take(need - p // page)
            if p % page:  # the fork's copy of a page that is partly filled
                copies += [(partly, mine[0])] if partly else []
                partly = partly or mine[0]
            rows.append((common + mine, p + past[b] + lens[b]))
            b += 1
    N, width = at + 4, max(len(r) for r, _ in rows) + 2
    scatter = list(range(1, N))
    random.Random(seed).shuffle(scatter)
    to = lambda i: scatter[i - 1]  # noqa: E731
    order = list(range(1, B + 1))
    random.Random(seed + 1).shuffle(order)  # sequence b sits in some row of the table
    table, kv_len = [[0] * width for _ in range(B + 1)], [0] * (B + 1)
    for r, (pages, n) in zip(order, rows):
        table[r][:len(pages)] = [to(i) for i in pages]
        kv_len[r] = n
    dtype = KINDS[case["cache"]]
    make = lambda: torch.randn((N, H_kv, page, d), generator=g, device="cuda", dtype=torch.bfloat16).to(dtype)  # noqa: E731
    k, v = make(), make()
    if copies:
        src, dst = (torch.tensor([to(i) for i in x], device="cuda") for x in zip(*copies))
        for pages in (k, v):
            raw = pages.view(torch.uint8)
            raw[dst] = raw[src]
    s = dict(case=case, k_pages=k, v_pages=v, page_table=_i32(table), kv_len=_i32(kv_len), row=_i32(order),
             cu_seqlens=_cu(lens), cu_groups=_cu(members), shared_len=_i32(prefix), max_new=max(lens),
             members=max(members), own_max=max(n + x for n, x in zip(lens, past)), k_scale=None, v_scale=None)
    if case["cache"] == "e4m3":  # what one step of the 8-bit values stands for, a head
        s["k_scale"] = 0.5 + torch.rand(H_kv, generator=g, device="cuda")
        s["v_scale"] = 0.5 + torch.rand(H_kv, generator=g, device="cuda")
    # queries long enough that some keys stand out, as they do in trained layers
    s["q"] = (2.0 * _normal(g, T, H_q, d)).to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(T, H_q, dtype=torch.float32, device="cuda")
    s["scale"] = d ** -0.5
    return s


def prepare(case, seed):
    return (_prepare_shared if case["op"] == "shared" else _prepare_linear)(case, seed, _gen(seed))


# ------------------------------------------------------------------ the plain forms

def _chunked(q, k, v, g, S0, C):
    """q, k [B][L][H][d_k], v [B][L][H][d_v] in 32 bits, g [B][L][H] in 64, S0 [B][H][d_k][d_v], L a multiple of C:
    the read-outs [B][L][H][d_v] and the state behind each chunk [B][H][L/C + 1][d_k][d_v], S0 the first."""
    B, L, H, d_v = v.shape
    q, k, v = (x.view(B, L // C, C, H, -1).permute(0, 3, 1, 2, 4).contiguous() for x in (q, k, v))
    G = g.view(B, L // C, C, H).permute(0, 3, 1, 2).cumsum(-1)
    lower = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    w = (G[..., :, None] - G[..., None, :]).masked_fill_(~lower, -math.inf).exp_().float()
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(w), v)
    total = G[..., -1]
    left = (total[..., None] - G).exp().float()
    U = torch.matmul((k * left[..., None]).transpose(-1, -2).contiguous(), v)
    past = total.cumsum(-1)
    begin = torch.cat((torch.zeros_like(past[..., :1]), past), -1)
    before = torch.ones(L // C + 1, L // C, dtype=torch.bool, device="cuda").tril(-1)
    w = (begin[..., :, None] - past[..., None, :]).masked_fill_(~before, -math.inf).exp_().float()
    S = torch.matmul(w, U.flatten(-2)).unflatten(-1, S0.shape[-2:])
    S += begin.exp().float()[..., None, None] * S0[:, :, None]
    o += torch.matmul(q, S[:, :, :-1]) * G.exp().float()[..., None]
    return o.permute(0, 2, 3, 1, 4).reshape(B, L, H, d_v), S


def _plain_prefill(s):
    c = s["case"]
    r = c["H_v"] // c["H_k"]
    cu = s["cu_seqlens"].long()
    n = cu[1:] - cu[:-1]
    T, B, L = s["q"].shape[0], c["B"], _ceil(c["n_max"], CHUNK) * CHUNK
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), n, output_size=T)
    slot = torch.arange(T, device="cuda") - cu[seq]

    def padded(x, dtype):
        p = torch.zeros((B, L) + x.shape[1:], dtype=dtype, device="cuda")
        p[seq, slot] = x.to(dtype)
        return p

    q, k = (padded(s[x], torch.float32).repeat_interleave(r, 2) for x in "qk")
    g = padded(s["g"].expand(T, c["H_v"]), torch.float64)
    S0 = s["state"][s["read_slot"].long()] * (s["read_slot"] > 0)[:, None, None, None]
    o, S = _chunked(q, k, padded(s["v"], torch.float32), g, S0, CHUNK)
    s["state"][s["write_slot"].long()] = S[:, :, -1]
    return (o[seq, slot] * s["q_scale"]).to(torch.bfloat16), s["state"]


def _plain_step(s):
    c = s["case"]
    B, T, r = c["B"], c["T"], c["H_v"] // c["H_k"]
    q, k = (s[x].float().repeat_interleave(r, 2) for x in "qk")
    v, g = s["v"].float(), s["g"].double().expand(B, T, c["H_v"])
    S0 = s["state"][s["read_slot"].long()]
    if T == 1:
        S = S0 * g[:, 0].exp().float()[..., None, None] + k[:, 0, :, :, None] * v[:, 0, :, None]
        s["state"][s["write_slot"].long()] = S
        return (torch.matmul(q[:, 0, :, None], S)[:, None, :, 0] * s["q_scale"]).to(torch.bfloat16), s["state"]
    o, S = _chunked(q, k, v, g, S0, 1)
    s["state"][s["token_slots"].long()] = S[:, :, 1:].transpose(1, 2)
    return (o * s["q_scale"]).to(torch.bfloat16), s["state"]


def _cells(pages, page, off, scale):
    """[...][H_kv][d] in 32 bits."""
    raw = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
    x = raw[page.long(), :, off].view(pages.dtype).float()
    return x if scale is None else x * scale[:, None]


def _part(q, k, v, seen, scale):
    """Maximum, sum and product of a softmax over the seen keys: q [..][m][d], k and v [..][L][d], seen [..][m][L]."""
    w = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(scale).masked_fill_(~seen, -math.inf)
    top = w.amax(-1, keepdim=True).clamp_min(-1e30)  # a row that sees no key keeps zeros
    w.sub_(top).exp_()
    return top, w.sum(-1, keepdim=True), torch.matmul(w, v)


def _plain_shared(s):
    c = s["case"]
    B, K, H_q, H_kv, d, page, n, M = c["B"], c["K"], c["H_q"], c["H_kv"], c["d"], c["page"], s["max_new"], s["members"]
    G, T = H_q // H_kv, s["q"].shape[0]
    cu, cg, rows = s["cu_seqlens"].long(), s["cu_groups"].long(), s["row"].long()
    new, count, common = cu[1:] - cu[:-1], cg[1:] - cg[:-1], s["shared_len"].long()
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), new, output_size=T)
    group = torch.repeat_interleave(torch.arange(K, device="cuda"), count, output_size=B)
    slot, member = torch.arange(T, device="cuda") - cu[seq], torch.arange(B, device="cuda") - cg[group]
    pos = s["kv_len"].long()[rows][seq] - new[seq] + slot
    first = torch.full_like(pos, 0) if not c["window"] else pos - c["window"] + 1

    def laid(size, at):  # queries [.][H_kv][G * tokens][d], the positions of their tokens and the first that they see
        q = torch.zeros(size + (H_q, d), device="cuda")
        q[at] = s["q"].float()
        q = q.unflatten(2, (H_kv, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)
        p = torch.full(size, -1, dtype=torch.long, device="cuda")
        f = p.clone()
        p[at], f[at] = pos, first
        return q, p, f

    def back(x, size, at):  # [.][H_kv][G * tokens][y] as [T][H_q][y]
        return x.unflatten(2, (G, size[1])).permute(0, 3, 1, 2, 4).flatten(2, 3)[at]

    # the common positions, a group at a time with all its tokens
    size, at = (K, M * n), (group[seq], member[seq] * n + slot)
    q, p, f = laid(size, at)
    j = torch.arange(c["prefix_max"], device="cuda")
    last = s["page_table"].shape[1] - 1
    entry = s["page_table"][rows[cg[:-1]]][:, (j // page).clamp_max(last)]
    k, v = (_cells(s[x + "_pages"], entry, j % page, s[x + "_scale"]).transpose(1, 2) for x in "kv")
    seen = (j < common[:, None, None]) & (j <= p[..., None]) & (j >= f[..., None])
    a = [back(x, size, at) for x in _part(q, k, v, seen[:, None].repeat(1, 1, G, 1), s["scale"])]
    # each row's own positions
    size, at = (B, n), (seq, slot)
    q, p, f = laid(size, at)
    j = common[group][:, None] + torch.arange(s["own_max"], device="cuda")
    entry = s["page_table"][rows[:, None], (j // page).clamp_max(last)]
    k, v = (_cells(s[x + "_pages"], entry, j % page, s[x + "_scale"]).transpose(1, 2) for x in "kv")
    seen = (j[:, None] <= p[..., None]) & (j[:, None] >= f[..., None])
    b = [back(x, size, at) for x in _part(q, k, v, seen[:, None].repeat(1, 1, G, 1), s["scale"])]
    top = torch.maximum(a[0], b[0])
    fa, fb = (a[0] - top).exp(), (b[0] - top).exp()
    total = a[1] * fa + b[1] * fb
    return ((a[2] * fa + b[2] * fb) / total).to(torch.bfloat16), (top + total.log())[..., 0]


# ------------------------------------------------------------------ the package's calls

def _scratch(s, nbytes):
    """The workspace that the program keeps beside its cache; nbytes() is asked once."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(nbytes(), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_step(s):
    import gated_deltanet_recurrent_decode_amd as gdn
    if "token_slots" in s:
        gdn.lin_attn_step_tokens(s["q"], s["k"], s["v"], s["g"], s["state"], s["read_slot"], s["token_slots"],
                                 s["out"], q_scale=s["q_scale"])
    else:
        gdn.lin_attn_step(s["q"], s["k"], s["v"], s["g"], s["state"], s["read_slot"], s["write_slot"], s["out"],
                          q_scale=s["q_scale"])
    return s["out"], s["state"]


def _own_prefill(s):
    import gated_deltanet_recurrent_decode_amd as gdn
    c = s["case"]
    work = _scratch(s, lambda: gdn.lin_attn_prefill_workspace_bytes(c["B"], s["q"].shape[0], c["H_k"], c["H_v"],
                                                                    c["d_k"], c["d_v"]))
    gdn.lin_attn_prefill(s["q"], s["k"], s["v"], s["g"], s["cu_seqlens"], s["state"], s["read_slot"],
                         s["write_slot"], s["out"], work, q_scale=s["q_scale"])
    return s["out"], s["state"]


def _own_shared(s):
    import gated_deltanet_recurrent_decode_amd as gdn
    c = s["case"]
    work = _scratch(s, lambda: gdn.attn_shared_workspace_bytes(c["B"], s["q"].shape[0], c["K"], s["max_new"],
                                                               c["H_q"], c["H_kv"], c["d"]))
    gdn.attn_shared(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["kv_len"], s["row"], s["cu_seqlens"],
                    s["cu_groups"], s["shared_len"], s["out"], work, max_new=s["max_new"], scale=s["scale"],
                    window=c["window"], lse=s["lse"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s["out"], s["lse"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"step": _own_step, "prefill": _own_prefill, "shared": _own_shared}[op](state)
    return {"step": _plain_step, "prefill": _plain_prefill, "shared": _plain_shared}[op](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "shared":
        lens, H_q, H_kv, d, w = _lengths(case), case["H_q"], case["H_kv"], case["d"], case["window"]
        members, prefix, past = _groups(case)
        cell = 2 if case["cache"] == "bf16" else 1
        keys = pairs = b = 0
        for m, p in zip(members, prefix):
            reach = 0  # of the common positions, those that some member sees
            for n, x in zip(lens[b:b + m], past[b:b + m]):
                L = p + x + n
                pairs += sum(min(L - i, w or L) for i in range(n))
                low = max(0, L - n - w + 1) if w else 0
                keys += L - max(p, low)
                reach = max(reach, p - low)
            keys += reach
            b += m
        return {"bytes": 2 * keys * H_kv * d * cell + sum(lens) * H_q * (4 * d + 4), "flops": 4 * d * H_q * pairs}
    B, H_k, H_v, d_k, d_v = (case[n] for n in ("B", "H_k", "H_v", "d_k", "d_v"))
    step = case["op"] == "step"
    T = B * case["T"] if step else sum(_lengths(case))
    states = B + T if step else 2 * B - sum(_fresh(case))
    token = 2 * (2 * H_k * d_k + 2 * H_v * d_v) + (4 * H_v if case["per_token"] else 0)
    return {"bytes": T * token + 4 * states * H_v * d_k * d_v, "flops": 4 * T * H_v * d_k * d_v}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_linear(s):
    """Token by token, all sequences side by side."""
    c = s["case"]
    step, r = c["op"] == "step", c["H_v"] // c["H_k"]
    q, k, v = (x.flatten(0, 1) if step else x for x in (s["q"], s["k"], s["v"]))
    g = s["g"].reshape(-1, c["H_v"]).double()
    cu, read = s["cu_seqlens"].tolist(), s["read_slot"].long()
    pool = s["state"].double()
    out = torch.zeros(v.shape, dtype=torch.float64, device="cuda")
    S = pool[read] * (read > 0).double()[:, None, None, None]
    ends = [b - a for a, b in zip(cu, cu[1:])]
    for t in range(max(ends)):
        live = [b for b, n in enumerate(ends) if t < n]
        at, b = torch.tensor([cu[x] + t for x in live], device="cuda"), torch.tensor(live, device="cuda")
        decay = torch.exp(g[at] if c["per_token"] else g)
        now = S[b] * decay[..., None, None]
        now += k[at].double().repeat_interleave(r, 1)[..., None] * v[at].double()[:, :, None]
        out[at] = (q[at].double().repeat_interleave(r, 1)[..., None] * now).sum(2) * s["q_scale"]
        S[b] = now
        if "token_slots" in s:
            pool[s["token_slots"][:, t].long()] = now
    if "write_slot" in s:
        pool[s["write_slot"].long()] = S
    return out.view(s["v"].shape), pool


def _exact_shared(s):
    """Each sequence by itself over its own row of the table."""
    c = s["case"]
    T, H_q = s["q"].shape[:2]
    G, page = H_q // c["H_kv"], c["page"]
    out = torch.zeros(T, H_q, c["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((T, H_q), -math.inf, dtype=torch.float64, device="cuda")
    cu, rows, lens = s["cu_seqlens"].tolist(), s["row"].tolist(), s["kv_len"].tolist()
    for b, r in enumerate(rows):
        lo, hi, L = cu[b], cu[b + 1], lens[r]
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
            for y in range(h * G, h * G + G):
                z = torch.where(off, -math.inf, s["q"][lo:hi, y].double() @ k.T * s["scale"])
                lse[lo:hi, y] = torch.logsumexp(z, 1)
                out[lo:hi, y] = torch.softmax(z, 1) @ v
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_shared if case["op"] == "shared" else _exact_linear)(s)
