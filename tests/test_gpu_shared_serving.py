"""GPU: one prompt, many continuations, as a server runs them: the prompt once through both kinds of layers, its pages
forked and its linear state read by every continuation, then steps of one token (eager, captured and replayed) and a
step that verifies drafted tokens, against 64 bits (attn_helpers.py and lin_helpers.py derive the bounds)."""
import pytest
import torch

import gated_deltanet_recurrent_decode_amd as gdn
from tests import attn_helpers as H
from tests import lin_helpers as L

pytestmark = pytest.mark.gpu

ROWS, PROMPT, STEPS, DRAFT = 24, 1100, 4, 3
H_Q, H_KV, D, PAGE = 4, 2, 64, 16           # the attention layer
H_K, H_V, D_K, D_V = 2, 4, 64, 64           # the linear layer


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    def __init__(self):
        gen = torch.Generator().manual_seed(17)
        new = STEPS + DRAFT

        def bf(*shape):
            return torch.randn(*shape, generator=gen).to(L.BF)

        # one projection of each layer: the prompt's tokens, then every row's
        self.attn = bf(PROMPT, H_Q + 2 * H_KV, D), bf(ROWS, new, H_Q + 2 * H_KV, D)
        self.lin = bf(PROMPT, 2 * H_K * D_K + H_V * D_V), bf(ROWS, new, 2 * H_K * D_K + H_V * D_V)
        self.g = -0.2 * torch.rand(PROMPT, H_V, generator=gen), -0.2 * torch.rand(ROWS, new, H_V, generator=gen)
        pages = (PROMPT + PAGE - 1) // PAGE + ROWS * 3 + 4
        width = (PROMPT + new) // PAGE + 2
        self.k = torch.zeros(pages, H_KV, PAGE, D, dtype=L.BF, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.table = torch.zeros(ROWS + 2, width, dtype=torch.int32, device="cuda")
        self.kv_len = torch.zeros(ROWS + 2, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.result = torch.zeros(2, dtype=torch.int32, device="cuda")
        self.page_ws = torch.empty(gdn.kv_page_workspace_bytes(ROWS, ROWS + 2, pages), dtype=torch.uint8, device="cuda")
        # slot 1 the prompt's, then one a row, then DRAFT a row
        self.state = torch.full((2 + ROWS * (1 + DRAFT), H_V, D_K, D_V), 3.0, device="cuda")
        self.state[0] = 0
        self.rows = i32(list(range(2, 2 + ROWS)))
        self.served = []

    def cells(self, x, rows, cu, add):
        """Grows the rows and writes their new tokens' k and v."""
        gdn.kv_page_reserve(self.table, self.kv_len, self.refs, rows, add, self.result, self.page_ws, page_size=PAGE)
        q = torch.empty(x.shape[0], H_Q, D, dtype=L.BF, device="cuda")
        gdn.attn_prologue(x[:, :H_Q], x[:, H_Q:H_Q + H_KV], x[:, H_Q + H_KV:], q, self.k, self.v, self.table,
                          self.kv_len, rows, cu, None)
        return q

    @staticmethod
    def heads(x):
        a, b = H_K * D_K, 2 * H_K * D_K
        return (x[..., :a].unflatten(-1, (H_K, D_K)), x[..., a:b].unflatten(-1, (H_K, D_K)),
                x[..., b:].unflatten(-1, (H_V, D_V)))

    def step(self, ax, lx, g, n, slots, out, lin_out, ws, read, cu, add, groups, shared):
        """n tokens a row through both layers."""
        q = self.cells(ax, self.rows, cu, add)
        gdn.attn_shared(q, self.k, self.v, self.table, self.kv_len, self.rows, cu, groups, shared, out, ws, max_new=n,
                        least=512)
        step = gdn.lin_attn_step_tokens if n > 1 else gdn.lin_attn_step
        step(*self.heads(lx), g, self.state, read, slots, lin_out, q_scale=D_K ** -0.5)


def test_one_prompt_many_continuations():
    s = Server()
    cu1 = i32([0, PROMPT])
    lin_prompt, attn_prompt, g_prompt = s.lin[0].cuda(), s.attn[0].cuda(), s.g[0].cuda()
    # the prompt, once
    q = s.cells(attn_prompt, i32([1]), cu1, i32([PROMPT]))
    out0 = torch.empty(PROMPT, H_Q, D, dtype=L.BF, device="cuda")
    ws0 = torch.empty(gdn.attn_paged_workspace_bytes(1, PROMPT, PROMPT, H_Q, H_KV, D), dtype=torch.uint8, device="cuda")
    gdn.attn_paged(q, s.k, s.v, s.table, s.kv_len, i32([1]), cu1, out0, ws0, max_new=PROMPT)
    lin0 = torch.empty(PROMPT, H_V, D_V, dtype=L.BF, device="cuda")
    wsl = torch.empty(gdn.lin_attn_prefill_workspace_bytes(1, PROMPT, H_K, H_V, D_K, D_V), dtype=torch.uint8,
                      device="cuda")
    gdn.lin_attn_prefill(*s.heads(lin_prompt), g_prompt, cu1, s.state, i32([0]), i32([1]), lin0, wsl,
                         q_scale=D_K ** -0.5)
    # its continuations
    gdn.kv_page_fork(s.k, s.v, s.table, s.kv_len, s.refs, i32([1] * ROWS), s.rows, s.result, s.page_ws)
    assert s.result.tolist() == [0, -1]
    groups, shared = i32([0, ROWS]), i32([PROMPT])
    own, prompt_slot = i32(list(range(2, 2 + ROWS))), i32([1] * ROWS)
    outs = torch.zeros(STEPS + DRAFT, ROWS, H_Q, D, dtype=L.BF, device="cuda")
    lin_outs = torch.zeros(STEPS + DRAFT, ROWS, H_V, D_V, dtype=L.BF, device="cuda")
    attn_new, lin_new, g_new = s.attn[1].cuda(), s.lin[1].cuda(), s.g[1].cuda()
    ws = torch.empty(gdn.attn_shared_workspace_bytes(ROWS, ROWS * DRAFT, 1, DRAFT, H_Q, H_KV, D), dtype=torch.uint8,
                     device="cuda")
    ax, lx, g = (torch.empty_like(x[:, :1]).contiguous() for x in (attn_new, lin_new, g_new))
    out, lin_out = torch.empty(ROWS, H_Q, D, dtype=L.BF, device="cuda"), torch.empty(ROWS, 1, H_V, D_V, dtype=L.BF,
                                                                                     device="cuda")
    read, cu, one = prompt_slot.clone(), i32(list(range(ROWS + 1))), i32([1] * ROWS)

    def call(write=None):
        s.step(ax[:, 0], lx, g, 1, write, out, lin_out, ws, read, cu, one, groups, shared)

    graph = None
    for t in range(STEPS):
        for to, x in ((ax, attn_new), (lx, lin_new), (g, g_new)):
            to.copy_(x[:, t:t + 1])
        if t == 0:  # from the prompt's state into the row's own, then in place
            call(own)
            read.copy_(own)
        elif t == 1:
            call()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    call()
            graph.replay()
        torch.cuda.synchronize()
        outs[t], lin_outs[t] = out, lin_out[:, 0]
    # drafted tokens: every state is kept, each row's own stays
    kept = i32([[2 + ROWS + r * DRAFT + t for t in range(DRAFT)] for r in range(ROWS)])
    before = s.state[2:2 + ROWS].clone()
    out3 = torch.empty(ROWS * DRAFT, H_Q, D, dtype=L.BF, device="cuda")
    lin3 = torch.empty(ROWS, DRAFT, H_V, D_V, dtype=L.BF, device="cuda")
    s.step(attn_new[:, STEPS:].reshape(ROWS * DRAFT, -1, D), lin_new[:, STEPS:].contiguous(),
           g_new[:, STEPS:].contiguous(), DRAFT, kept, out3, lin3, ws, own,
           i32(list(range(0, ROWS * DRAFT + 1, DRAFT))), i32([DRAFT] * ROWS), groups, shared)
    torch.cuda.synchronize()
    outs[STEPS:] = out3.view(ROWS, DRAFT, H_Q, D).transpose(0, 1)
    lin_outs[STEPS:] = lin3.transpose(0, 1)
    assert torch.equal(before, s.state[2:2 + ROWS]) and s.kv_len[2:].tolist() == [PROMPT + STEPS + DRAFT] * ROWS

    # attention: a cache of every row's tokens side by side, the last STEPS + DRAFT of them new
    new = STEPS + DRAFT
    c = H.Cache([(new, PROMPT)] * ROWS, H_q=H_Q, H_kv=H_KV, d=D, page=PAGE, seed=0)
    c.q = s.attn[1][:, :, :H_Q].reshape(ROWS * new, H_Q, D)
    for b in range(ROWS):
        both = torch.cat([s.attn[0], s.attn[1][b]])
        for j in range(PROMPT + new):
            at = int(c.table[int(c.row[b])][j // PAGE]), slice(None), j % PAGE
            c.k[at], c.v[at] = both[j, H_Q:H_Q + H_KV], both[j, H_Q + H_KV:]
    o, _, tol, _ = H.attention(c, D ** -0.5)
    H.check(outs.transpose(0, 1).reshape(ROWS * new, H_Q, D), o, tol, "o of attention")

    # linear attention: the prompt and a row's tokens as one sequence
    for b in (0, 7, ROWS - 1):
        x, gg = torch.cat([s.lin[0], s.lin[1][b]]), torch.cat([s.g[0], s.g[1][b]])
        o, tol, states = L.recurrence(*s.heads(x), gg, torch.zeros(H_V, D_K, D_V), D_K ** -0.5)
        if b == 0:
            L.close(lin0, o[:PROMPT], tol[:PROMPT], "o of the prompt")
            L.close(s.state[1], states[PROMPT][0], states[PROMPT][1], "the prompt's state")
        L.close(lin_outs[:, b], o[PROMPT:], tol[PROMPT:], f"o of row {b}")
        L.close(s.state[2 + b], states[PROMPT + STEPS][0], states[PROMPT + STEPS][1], f"row {b}'s state")
        for t in range(DRAFT):
            S, err = states[PROMPT + STEPS + t + 1]
            L.close(s.state[2 + ROWS + b * DRAFT + t], S, err, f"row {b}'s state after drafted token {t}")
