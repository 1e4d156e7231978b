"""GPU: linear attention with a decay for each head (lin_attn_step, lin_attn_step_tokens, lin_attn_prefill)
against the recurrence in 64 bits, with bounds derived in lin_helpers.py."""
import math

import pytest
import torch

import gated_deltanet_recurrent_decode_amd as gdn
from tests.lin_helpers import BF, Layer, close

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prefill(c, lens, read, write, *, state=None, first=0, T=None, ws=None, out=None, qkv=None, g=None):
    """Runs the prompts; returns out and the pool."""
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    state = c.state.cuda() if state is None else state
    q, k, v = c.heads((c.qkv if qkv is None else qkv).cuda())
    out = torch.full((c.T, c.H_v, c.d_v), 7.0, dtype=BF, device="cuda") if out is None else out
    if ws is None:
        n = gdn.lin_attn_prefill_workspace_bytes(len(lens), c.T, c.H_k, c.H_v, c.d_k, c.d_v)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    gdn.lin_attn_prefill(q, k, v, (c.g if g is None else g).cuda(), i32(cu), state, i32(read),
                         None if write is None else i32(write), out, ws, q_scale=c.scale)
    torch.cuda.synchronize()
    return out, state


def check_prefill(c, lens, read, write, out, state, first=0):
    a = first
    to = read if write is None else write
    written = set()
    for b, n in enumerate(lens):
        r, w = read[b], to[b]
        if r == 0 and w == 0:
            assert torch.equal(out[a:a + n].cpu(), torch.zeros_like(out[a:a + n].cpu())), f"padding sequence {b}"
        else:
            S0 = c.state[r] if r else torch.zeros_like(c.state[0])
            o, tol, states = c.reference(a, a + n, S0)
            close(out[a:a + n], o, tol, f"out of sequence {b}")
            close(state[w], states[-1][0], states[-1][1], f"state of sequence {b}")
            written.add(w)
        a += n
    for s in range(c.N):
        if s not in written:
            assert torch.equal(state[s].cpu(), c.state[s]), f"slot {s} changed"
    assert bool((out[:first] == 7).all()) and bool((out[a:] == 7).all()), "tokens outside the sequences"


@pytest.mark.parametrize("d_k,d_v", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 77])
def test_prefill_one_prompt(d_k, d_v, per_token, n):
    c = Layer(n, H_k=1, H_v=2, d_k=d_k, d_v=d_v, N=4, per_token=per_token, seed=n)
    out, state = prefill(c, [n], [2], [3])
    check_prefill(c, [n], [2], [3], out, state)


@pytest.mark.parametrize("d_k,d_v,H_k,H_v", [(128, 128, 1, 1), (128, 64, 1, 2), (64, 128, 2, 2), (64, 64, 1, 4)])
@pytest.mark.parametrize("per_token", [False, True])
def test_prefill_several_segments(d_k, d_v, H_k, H_v, per_token):
    # prompts of no token, of one, of one segment and of many, from zeros, in place and to another slot
    lens = [0, 300, 1, 128, 129, 700, 0, 257]
    read, write = [1, 2, 3, 0, 5, 6, 0, 8], [9, 2, 10, 4, 5, 11, 7, 8]
    c = Layer(sum(lens) + 5, H_k=H_k, H_v=H_v, d_k=d_k, d_v=d_v, N=12, per_token=per_token, seed=3)
    out, state = prefill(c, lens, read, write, first=2)
    check_prefill(c, lens, read, write, out, state, first=2)


def test_prefill_in_place_padding_and_unusable_sequences():
    c = Layer(600, H_k=2, H_v=4, N=6, seed=4)
    lens = [200, 50, 300, 20, 30]
    out, state = prefill(c, lens, [1, 0, 2, 9, -1], None)
    # the unusable ones (slots 9 and -1 of 6) are NaN and touch nothing
    assert bool(out[550:].isnan().all())
    check_prefill(c, lens[:3], [1, 0, 2], None, torch.cat((out[:550], torch.full_like(out[550:], 7))), state)
    # reading a slot and writing the null slot is refused, a write slot outside too
    out, state = prefill(c, lens, [1, 2, 3, 4, 0], [0, 6, -2, 3, 0])
    assert bool(out[:550].isnan().all()) and bool((out[570:] == 0).all())
    o, tol, states = c.reference(550, 570, c.state[4])
    close(out[550:570], o, tol, "out")
    close(state[3], *states[-1], "state")
    for s in (0, 1, 2, 4, 5):
        assert torch.equal(state[s].cpu(), c.state[s])


def test_prefill_shared_read_slot_and_token_ranges_outside():
    # forks of one prefix state; a sequence whose range passes T, and one that runs backwards, are left as they were
    c = Layer(400, H_k=2, H_v=2, N=8, seed=5)
    out, state = prefill(c, [100, 150, 150], [1, 1, 1], [2, 3, 4])
    check_prefill(c, [100, 150, 150], [1, 1, 1], [2, 3, 4], out, state)
    q, k, v = c.heads(c.qkv.cuda())
    out = torch.full((400, 2, 64), 7.0, dtype=BF, device="cuda")
    state = c.state.cuda()
    ws = torch.empty(gdn.lin_attn_prefill_workspace_bytes(3, 400, 2, 2, 64, 64), dtype=torch.uint8, device="cuda")
    gdn.lin_attn_prefill(q, k, v, c.g.cuda(), i32([0, 90, 401, 380]), state, i32([1, 2, 3]), i32([4, 5, 6]), out, ws,
                         q_scale=c.scale)
    o, tol, states = c.reference(0, 90, c.state[1])
    close(out[:90], o, tol, "out")
    close(state[4], *states[-1], "state")
    assert bool((out[90:] == 7).all()) and torch.equal(state[5:].cpu(), c.state[5:])


@pytest.mark.parametrize("spread", [0.001, 1.0, 30.0, 400.0])
@pytest.mark.parametrize("per_token", [False, True])
def test_prefill_decays_from_none_to_all(spread, per_token):
    c = Layer(300, H_k=2, H_v=4, d_k=128, d_v=64, N=3, per_token=per_token, spread=spread, seed=6)
    out, state = prefill(c, [300], [1], [2])
    check_prefill(c, [300], [1], [2], out, state)


def test_prefill_resets_and_growth():
    # -inf forgets everything before its token; 0 keeps all; small positive logarithms let it grow
    c = Layer(200, H_k=1, H_v=2, N=3, seed=7)
    c.g[40], c.g[41], c.g[120, 0] = -math.inf, 0.0, -math.inf
    c.g[60:70] = 0.05
    out, state = prefill(c, [200], [1], [2])
    o, tol, states = c.reference(0, 200, c.state[1])
    close(out, o, tol.nan_to_num(posinf=0.0), "out")
    close(state[2], states[-1][0], states[-1][1], "state")


@pytest.mark.parametrize("which", ["q", "k", "v", "g"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("at", [0, 37, 63, 199])
def test_prefill_values_that_are_not_finite(which, value, at):
    if which == "g" and value == -math.inf:
        pytest.skip("a reset, tested above")
    c = Layer(200, H_k=1, H_v=2, N=5, seed=8)
    clean, state0 = prefill(c, [200], [1], [2])
    qkv, g = c.qkv.clone(), c.g.clone()
    q, k, v = c.heads(qkv)
    if which == "g":
        g[at, 1] = value
    else:
        {"q": q, "k": k, "v": v}[which][at, 0, 5] = value
    out, state = prefill(c, [200], [1], [2], qkv=qkv, g=g)
    assert torch.equal(out[:at].view(torch.int16), clean[:at].view(torch.int16)), "a token before it changed"
    if which == "q":  # q never enters the state
        assert not out[at].isfinite().any() and torch.equal(state, state0)
        assert torch.equal(out[at + 1:].view(torch.int16), clean[at + 1:].view(torch.int16))
    elif which == "v":  # one column of one head from there on
        assert not out[at:, 0, 5].isfinite().any() and not state[2, 0, :, 5].isfinite().any()
        rest = torch.ones(2, 64, dtype=torch.bool, device="cuda")
        rest[0, 5] = False
        assert torch.equal(out[:, rest], clean[:, rest])
        assert torch.equal(state[2].transpose(1, 2)[rest], state0[2].transpose(1, 2)[rest])
    elif which == "k":
        assert not out[at:].isfinite().any() and not state[2, :, 5].isfinite().any()
    else:
        assert not out[at:, 1].isfinite().any() and not state[2, 1].isfinite().any()
        assert torch.equal(out[:, 0], clean[:, 0]) and torch.equal(state[2, 0], state0[2, 0])


def test_prefill_same_bits_again_and_after_other_work():
    c = Layer(900, H_k=2, H_v=4, d_k=128, d_v=128, N=6, seed=9)
    a, sa = prefill(c, [500, 400], [1, 2], [3, 4])
    ws = torch.full((gdn.lin_attn_prefill_workspace_bytes(2, 900, 2, 4, 128, 128),), 0x7F, dtype=torch.uint8,
                    device="cuda")
    for _ in range(2):
        b, sb = prefill(c, [500, 400], [1, 2], [3, 4], ws=ws)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(sa, sb)


def test_prefill_many_sequences():
    # more than a wave holds: 150 sequences, some empty
    gen = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 12, (150,), generator=gen).tolist()
    lens[70] = 300
    c = Layer(sum(lens), H_k=1, H_v=1, N=301, seed=10)
    ids = (1 + torch.randperm(300, generator=gen)).tolist()
    out, state = prefill(c, lens, ids[:150], ids[150:])
    check_prefill(c, lens, ids[:150], ids[150:], out, state)


def test_prefill_without_tokens():
    c = Layer(0, N=5, seed=11)
    out, state = prefill(c, [0, 0, 0], [1, 0, 2], [3, 4, 2])
    assert torch.equal(state[3].cpu(), c.state[1]) and bool((state[4] == 0).all())
    assert torch.equal(state[:3].cpu(), c.state[:3])


# ------------------------------------------------------------------ single tokens

def step(c, B, T, read, write=None, tokens=None, state=None, stream=None):
    state = c.state.cuda() if state is None else state
    q, k, v = (x.unflatten(0, (B, T)) for x in c.heads(c.qkv.cuda()))
    g = c.g.cuda().unflatten(0, (B, T)) if c.per_token else c.g.cuda()
    out = torch.full((B, T, c.H_v, c.d_v), 7.0, dtype=BF, device="cuda")
    if tokens is not None:
        gdn.lin_attn_step_tokens(q, k, v, g, state, i32(read), i32(tokens), out, q_scale=c.scale, stream=stream)
    else:
        gdn.lin_attn_step(q, k, v, g, state, i32(read), None if write is None else i32(write), out, q_scale=c.scale,
                          stream=stream)
    torch.cuda.synchronize()
    return out, state


@pytest.mark.parametrize("d_k,d_v", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("twin", [False, True])
def test_step(d_k, d_v, per_token, T, twin):
    B, read = 4, [3, 0, 5, 1]
    write = [2, 7, 4, 6] if twin else None
    c = Layer(B * T, H_k=2, H_v=4, d_k=d_k, d_v=d_v, N=9, per_token=per_token, seed=T)
    out, state = step(c, B, T, read, write)
    written = set()
    for r in range(B):
        if read[r] == 0:
            assert bool((out[r] == 0).all())
            continue
        o, tol, states = c.reference(r * T, r * T + T, c.state[read[r]])
        close(out[r], o, tol, f"out of row {r}")
        w = write[r] if twin else read[r]
        close(state[w], *states[-1], f"state of row {r}")
        written.add(w)
    for s in set(range(9)) - written:
        assert torch.equal(state[s].cpu(), c.state[s]), f"slot {s} changed"


@pytest.mark.parametrize("d_k,d_v", [(64, 128), (128, 64)])
def test_step_tokens(d_k, d_v):
    B, T, read = 3, 4, [1, 0, 2]
    tokens = [[3, 0, 4, 5], [0, 0, 0, 0], [6, 7, 8, 0]]
    c = Layer(B * T, H_k=1, H_v=3, d_k=d_k, d_v=d_v, N=10, seed=2)
    out, state = step(c, B, T, read, tokens=tokens)
    assert bool((out[1] == 0).all())
    for r in (0, 2):
        o, tol, states = c.reference(r * T, r * T + T, c.state[read[r]])
        close(out[r], o, tol, "out")
        for t, s in enumerate(tokens[r]):
            if s:
                close(state[s], *states[t + 1], f"state after token {t} of row {r}")
    for s in (0, 1, 2, 9):
        assert torch.equal(state[s].cpu(), c.state[s])


def test_step_unusable_rows():
    c = Layer(6, H_k=1, H_v=2, N=5, seed=3)
    out, state = step(c, 6, 1, [9, -1, 1, 2, 0, 3], [1, 2, 0, 2, 9, 4])
    assert bool(out[:4].isnan().all()) and bool((out[4] == 0).all())
    o, tol, states = c.reference(5, 6, c.state[3])
    close(out[5], o, tol, "out")
    close(state[4], *states[-1], "state")
    assert torch.equal(state[:4].cpu(), c.state[:4])
    out, state = step(c, 3, 2, [1, 2, 4], tokens=[[2, 9], [2, 3], [-1, 0]])
    assert bool(out.isnan().all()) and torch.equal(state.cpu(), c.state)


def test_step_values_that_are_not_finite():
    # a NaN or infinity of a row's v stays in its column, of other rows and heads nothing changes
    c = Layer(4, H_k=1, H_v=2, N=9, seed=4)
    clean, s0 = step(c, 4, 1, [1, 2, 3, 4], [5, 6, 7, 8])
    c.heads(c.qkv)[2][2, 1, 9] = math.nan
    out, s1 = step(c, 4, 1, [1, 2, 3, 4], [5, 6, 7, 8])
    assert bool(out[2, 0, 1, 9].isnan()) and bool(s1[7, 1, :, 9].isnan().all())
    same = torch.ones_like(out, dtype=torch.bool)
    same[2, 0, 1, 9] = False
    assert torch.equal(out[same], clean[same])


# ------------------------------------------------------------------ together

def test_prompt_then_steps_equal_one_long_prompt():
    c = Layer(260, H_k=2, H_v=4, d_k=128, d_v=128, N=6, seed=12)
    out, state = prefill(c, [250], [0], [1])
    q, k, v = c.heads(c.qkv.cuda())
    here, there = i32([1]), i32([2])
    for t in range(250, 260):
        gdn.lin_attn_step(q[t:t + 1, None], k[t:t + 1, None], v[t:t + 1, None], c.g.cuda()[t:t + 1, None], state, here,
                          there, out[t:t + 1, None], q_scale=c.scale)
        gdn.slot_commit(here, there)
    torch.cuda.synchronize()
    o, tol, states = c.reference(0, 260, torch.zeros(4, 128, 128))
    close(out, o, tol, "out")
    close(state[1 if here.item() == 1 else 2], *states[-1], "state")


def test_calls_on_another_stream_and_in_a_graph():
    c = Layer(500, H_k=2, H_v=2, d_k=64, d_v=128, N=6, seed=13)
    want, want_state = prefill(c, [300, 200], [1, 0], [3, 4])
    state = c.state.cuda()
    q, k, v = (x.contiguous() for x in c.heads(c.qkv.cuda()))
    g, cu, read, write = c.g.cuda(), i32([0, 300, 500]), i32([1, 0]), i32([3, 4])
    out = torch.zeros(500, 2, 128, dtype=BF, device="cuda")
    ws = torch.empty(gdn.lin_attn_prefill_workspace_bytes(2, 500, 2, 2, 64, 128), dtype=torch.uint8, device="cuda")
    so = torch.zeros(1, 1, 2, 128, dtype=BF, device="cuda")

    def both():
        gdn.lin_attn_prefill(q, k, v, g, cu, state, read, write, out, ws, q_scale=c.scale)
        gdn.lin_attn_step(q[None, :1], k[None, :1], v[None, :1], g[None, :1], state, write[:1], i5, so,
                          q_scale=c.scale)

    i5 = i32([5])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(state[3:5], want_state[3:5])
    first = so.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for n in (500, 421, 300):  # a captured call follows the lengths on the device
        cu[2] = n
        out.zero_()
        so.zero_()
        state.copy_(c.state)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:n], want[:n]) and bool((out[n:] == 0).all()) and torch.equal(so, first)
        assert torch.equal(state[3], want_state[3])


def test_slots_past_eight_gib():
    c = Layer(300, H_k=8, H_v=16, d_k=128, d_v=128, N=3, seed=14)
    N = 8300  # slots of 1 MiB
    state = torch.empty(N, 16, 128, 128, device="cuda")
    state[N - 1] = c.state[1].cuda()
    q, k, v = c.heads(c.qkv.cuda())
    g, out = c.g.cuda(), torch.zeros(300, 16, 128, dtype=BF, device="cuda")
    ws = torch.empty(gdn.lin_attn_prefill_workspace_bytes(1, 299, 8, 16, 128, 128), dtype=torch.uint8, device="cuda")
    gdn.lin_attn_prefill(q[:299], k[:299], v[:299], g[:299], i32([0, 299]), state, i32([N - 1]), i32([N - 2]),
                         out[:299], ws, q_scale=c.scale)
    kept = i32([[N - 3]])
    gdn.lin_attn_step_tokens(q[None, 299:], k[None, 299:], v[None, 299:], g[None, 299:], state, i32([N - 2]), kept,
                             out[None, 299:], q_scale=c.scale)
    torch.cuda.synchronize()
    o, tol, states = c.reference(0, 300, c.state[1])
    close(out, o, tol, "out")
    close(state[N - 2], states[299][0], states[299][1], "the prompt's state")
    close(state[N - 3], states[300][0], states[300][1], "the state after a token")
    assert torch.equal(state[N - 1].cpu(), c.state[1])


def test_two_prompts_at_once():
    # each on its own stream with its own workspace: the bits of one after the other
    layers = [Layer(1500, H_k=2, H_v=4, d_k=64, d_v=64, N=4, seed=15),
              Layer(900, H_k=2, H_v=2, d_k=128, d_v=128, N=4, seed=16)]
    alone = [prefill(c, [c.T - 400, 400], [1, 0], [2, 3]) for c in layers]
    calls = []
    for c in layers:
        out = torch.zeros(c.T, c.H_v, c.d_v, dtype=BF, device="cuda")
        ws = torch.empty(gdn.lin_attn_prefill_workspace_bytes(2, c.T, c.H_k, c.H_v, c.d_k, c.d_v), dtype=torch.uint8,
                         device="cuda")
        calls.append(((*c.heads(c.qkv.cuda()), c.g.cuda(), i32([0, c.T - 400, c.T]), c.state.cuda(), i32([1, 0]),
                       i32([2, 3]), out, ws), c.scale, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for args, scale, stream in calls:
            gdn.lin_attn_prefill(*args, q_scale=scale, stream=stream)
    torch.cuda.synchronize()
    for (out, state), (args, _, _) in zip(alone, calls):
        assert torch.equal(out, args[8]) and torch.equal(state, args[5])
