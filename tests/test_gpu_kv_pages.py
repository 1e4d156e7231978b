"""GPU: the pages of a KV cache (kv_page_*, through the binding) against the
same rules restated one entry at a time, and a serving loop over all calls."""
import pytest
import torch

from tests import attn_helpers as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_recurrent_decode_amd as m
    m.lib()
    return m


class Model:
    """The rules in plain Python."""

    def __init__(self, R, width, N, page):
        self.R, self.width, self.N, self.page = R, width, N, page
        self.table = [[0] * width for _ in range(R)]
        self.len = [0] * R
        self.refs = [0] * N

    def free_pages(self):
        return [p for p in range(1, self.N) if self.refs[p] == 0]

    def reserve(self, rows, add):
        left, seen, missed, short = self.free_pages(), set(), [], False
        for i, (r, n) in enumerate(zip(rows, add)):
            again = r in seen
            seen.add(r)
            if not 0 < r < self.R or again or n < 0 or self.len[r] + n > self.width * self.page:
                missed.append(i)
                continue
            e0 = -(-self.len[r] // self.page)
            need = -(-(self.len[r] + n) // self.page) - e0
            if need and (short or need > len(left)):
                short = True
                missed.append(i)
                continue
            for e in range(e0, e0 + need):
                self.table[r][e] = p = left.pop(0)
                self.refs[p] = 1
            self.len[r] += n
        return missed

    def fork(self, src, dst):
        """Returns the entries not served and the page copies."""
        left, seen, missed, moves, short = self.free_pages(), set(), [], [], False
        had = list(self.len)
        for i, (a, b) in enumerate(zip(src, dst)):
            inside = 0 < a < self.R and 0 < b < self.R and a != b
            again = b in seen
            seen.add(b)
            if not inside or again or had[b] != 0:
                missed.append(i)
                continue
            n = had[a]
            part = n % self.page > 0
            if part and (short or not left):
                short = True
                missed.append(i)
                continue
            for e in range(n // self.page):
                self.table[b][e] = self.table[a][e]
                self.refs[self.table[a][e]] += 1
            if part:
                p = left.pop(0)
                self.table[b][n // self.page] = p
                self.refs[p] = 1
                moves.append((self.table[a][n // self.page], p))
            self.len[b] = n
        return missed, moves

    def free(self, rows):
        for r in rows:
            if not 0 < r < self.R:
                continue
            for p in self.table[r]:
                if 0 < p < self.N:
                    self.refs[p] -= 1
            self.table[r] = [0] * self.width
            self.len[r] = 0

    def compact(self):
        live = [p for p in range(1, self.N) if self.refs[p] > 0]
        holes = [p for p in range(1, len(live) + 1) if self.refs[p] == 0]
        moves = list(zip([p for p in live if p > len(live)], holes))
        to = {p: p for p in live}
        to.update(moves)
        self.table = [[to.get(p, 0) for p in r] for r in self.table]
        for a, b in moves:
            self.refs[a], self.refs[b] = 0, self.refs[a]
        return [to.get(p, 0) for p in range(self.N)], len(live), moves


class Device:
    def __init__(self, gdn, m, layers=1, H_kv=1, d=64, seed=0, n=64, kind="bf16"):
        g = torch.Generator().manual_seed(seed)
        self.gdn, self.m = gdn, m
        shape = (layers, m.N, H_kv, m.page, d) if layers > 1 else (m.N, H_kv, m.page, d)
        self.k = torch.randn(shape, generator=g).to(A.KINDS[kind]).cuda()
        self.v = torch.randn(shape, generator=g).to(A.KINDS[kind]).cuda()
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table, self.len, self.refs = (torch.tensor(x, **i32) for x in (m.table, m.len, m.refs))
        self.result = torch.full((2,), -9, **i32)
        self.ws = torch.full((gdn.kv_page_workspace_bytes(n, m.R, m.N),), 0xFF, dtype=torch.uint8, device="cuda")

    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def reserve(self, rows, add):
        self.gdn.kv_page_reserve(self.table, self.len, self.refs, self.ints(rows), self.ints(add), self.result,
                                 self.ws, page_size=self.m.page)

    def fork(self, src, dst):
        self.gdn.kv_page_fork(self.k, self.v, self.table, self.len, self.refs, self.ints(src), self.ints(dst),
                              self.result, self.ws)

    def free(self, rows):
        self.gdn.kv_page_free(self.table, self.len, self.refs, self.ints(rows))

    def agree(self, missed=None):
        torch.cuda.synchronize()
        m = self.m
        assert self.table.cpu().tolist() == m.table
        assert self.len.cpu().tolist() == m.len
        assert self.refs.cpu().tolist() == m.refs
        if missed is not None:
            assert self.result.cpu().tolist() == [len(missed), missed[0] if missed else -1]

    def moved(self, k, v, moves):
        """The pools are k and v with these copies, bit for bit."""
        bits = torch.uint8 if k.dtype == A.F8 else torch.int16
        axis = k.dim() - 4
        for got, want in ((self.k, k.clone()), (self.v, v.clone())):
            w = want.view(bits)
            for a, b in moves:
                w.select(axis, b).copy_(want.view(bits).select(axis, a))
            assert torch.equal(got.view(bits), w)


def test_reserve_in_the_order_of_the_list(gdn):
    m = Model(R=9, width=6, N=14, page=16)
    dev = Device(gdn, m)
    for rows, add in (([3, 1, 2], [1, 16, 17]), ([3, 1, 2, 5], [15, 0, 15, 33]), ([3, 4], [1, 0])):
        dev.reserve(rows, add)
        dev.agree(m.reserve(rows, add))


def test_reserve_refuses_rows_one_by_one(gdn):
    m = Model(R=9, width=4, N=12, page=16)
    dev = Device(gdn, m)
    # null row, outside, twice, negative, past the table, served ones between them
    rows, add = [0, 9, -1, 3, 3, 4, 5, 6], [1, 1, 1, 20, 1, -1, 65, 64]
    dev.reserve(rows, add)
    dev.agree(m.reserve(rows, add))
    # four pages left of eleven: the second row does not fit, the third would but comes behind it,
    # the fourth needs none
    rows, add = [1, 2, 7, 3], [33, 33, 5, 12]
    dev.reserve(rows, add)
    missed = m.reserve(rows, add)
    assert missed == [1, 2]
    dev.agree(missed)
    dev.reserve([2**31 - 1, 7], [2**31 - 1, 2**31 - 1])
    dev.agree(m.reserve([2**31 - 1, 7], [2**31 - 1, 2**31 - 1]))


@pytest.mark.parametrize("n", [0, 1, 1023, 1025, 2500])
def test_reserve_long_lists(gdn, n):
    m = Model(R=3001, width=5, N=6000, page=16)
    dev = Device(gdn, m, n=2500)
    rows = [1 + (7 * i) % 3000 for i in range(n)]
    add = [(13 * i) % 50 for i in range(n)]
    dev.reserve(rows, add)
    dev.agree(m.reserve(rows, add))
    dev.reserve(rows[::-1], add)
    dev.agree(m.reserve(rows[::-1], add))
    dev.free(rows[: n // 2])
    m.free(rows[: n // 2])
    dev.agree()


@pytest.mark.parametrize("layers,kind", [(1, "bf16"), (3, "bf16"), (2, "e4m3")])
def test_fork_shares_whole_pages_and_copies_the_last(gdn, layers, kind):
    m = Model(R=12, width=6, N=30, page=16)
    dev = Device(gdn, m, layers=layers, H_kv=2, d=64, kind=kind)
    rows, add = [1, 2, 3], [40, 32, 5]
    dev.reserve(rows, add)
    m.reserve(rows, add)
    k, v = dev.k.clone(), dev.v.clone()
    # the same source twice, a whole-paged one, an empty one, then refusals: full, itself, twice, outside, null
    src, dst = [1, 1, 2, 9, 3, 3, 3, 1, 12, 0], [4, 5, 6, 7, 2, 3, 4, 0, 8, 8]
    dev.fork(src, dst)
    missed, moves = m.fork(src, dst)
    dev.agree(missed)
    dev.moved(k, v, moves)
    # forks grow apart and end
    dev.reserve([1, 4, 5, 6], [30, 1, 17, 1])
    dev.agree(m.reserve([1, 4, 5, 6], [30, 1, 17, 1]))
    dev.free([1, 5, 5, 0, -3, 99])
    m.free([1])
    m.free([5])
    dev.agree()


def test_fork_without_enough_pages(gdn):
    m = Model(R=12, width=4, N=6, page=16)
    dev = Device(gdn, m)
    dev.reserve([1, 2], [20, 32])
    m.reserve([1, 2], [20, 32])
    k, v = dev.k.clone(), dev.v.clone()
    src, dst = [1, 1, 2, 1], [3, 4, 5, 6]   # one free page: the first takes it, whole pages still go
    dev.fork(src, dst)
    missed, moves = m.fork(src, dst)
    assert missed == [1, 3]
    dev.agree(missed)
    dev.moved(k, v, moves)


@pytest.mark.parametrize("layers,H_kv,page,d,kind", [(1, 1, 16, 64, "bf16"), (3, 2, 64, 128, "bf16"),
                                                     (2, 3, 32, 64, "e4m3"), (1, 1, 16, 64, "e4m3")])
def test_copy(gdn, layers, H_kv, page, d, kind):
    m = Model(R=2, width=2, N=40, page=page)
    dev = Device(gdn, m, layers=layers, H_kv=H_kv, d=d, kind=kind)
    k, v = dev.k.clone(), dev.v.clone()
    src, dst = [1, 1, 5, 0, 40, -1, 7], [10, 11, 12, 13, 14, 15, 0]
    gdn.kv_page_copy(dev.k, dev.v, dev.ints(src), dev.ints(dst))
    torch.cuda.synchronize()
    dev.moved(k, v, [(1, 10), (1, 11), (5, 12), (0, 13)])
    gdn.kv_page_copy(dev.k, dev.v, dev.ints([]), dev.ints([]))
    gdn.kv_page_copy(dev.k, dev.v, dev.ints(list(range(1, 20))), dev.ints(list(range(39, 20, -1))))
    torch.cuda.synchronize()
    assert torch.equal(dev.k.view(torch.uint8).select(int(layers > 1), 39),
                       dev.k.view(torch.uint8).select(int(layers > 1), 1))


@pytest.mark.parametrize("N,layers", [(2, 1), (60, 2), (1024, 1), (5000, 1)])
def test_compact(gdn, N, layers):
    m = Model(R=N // 2 + 2, width=4, N=N, page=16)
    dev = Device(gdn, m, layers=layers, n=N)
    rows = list(range(1, N // 2 + 1))
    add = [1 + (11 * i) % 40 for i in range(len(rows))]
    dev.reserve(rows, add)
    m.reserve(rows, add)
    dev.free(rows[::3] + rows[: len(rows) // 4])
    m.free(set(rows[::3] + rows[: len(rows) // 4]))
    dev.agree()
    k, v = dev.k.clone(), dev.v.clone()
    remap = torch.full((N,), -7, dtype=torch.int32, device="cuda")
    gdn.kv_page_compact(dev.k, dev.v, dev.table, dev.refs, remap, dev.result, dev.ws)
    want, live, moves = m.compact()
    dev.agree()
    assert dev.result.cpu().tolist() == [live, len(moves)] and remap.cpu().tolist() == want
    dev.moved(k, v, moves)
    gdn.kv_page_compact(dev.k, dev.v, dev.table, dev.refs, remap, dev.result, dev.ws)
    torch.cuda.synchronize()
    assert dev.result.cpu().tolist() == [live, 0]
    dev.agree()


def test_a_captured_turn(gdn):
    """Free, fork and reserve in one graph, replayed over other lists and tables."""
    m = Model(R=40, width=6, N=120, page=16)
    dev = Device(gdn, m)
    gone, src, dst, grow, add = (dev.ints(x) for x in ([0] * 4, [0] * 4, [0] * 4, [0] * 8, [0] * 8))

    def turn():
        gdn.kv_page_free(dev.table, dev.len, dev.refs, gone)
        gdn.kv_page_fork(dev.k, dev.v, dev.table, dev.len, dev.refs, src, dst, dev.result, dev.ws)
        gdn.kv_page_reserve(dev.table, dev.len, dev.refs, grow, add, dev.result, dev.ws, page_size=16)
    turn()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn()
    for step in range(5):
        rows = [1 + (8 * step + i) % 39 for i in range(8)]
        lists = ([rows[0], 1 + 3 * step, 0, 0], rows[:4], [30 - step, 20 + step, 0, 7], rows,
                 [9 + 5 * i for i in range(8)])
        for t, x in zip((gone, src, dst, grow, add), lists):
            t.copy_(dev.ints(x))
        torch.cuda.synchronize()
        graph.replay()
        for r in sorted(set(lists[0])):
            m.free([r])
        m.fork(lists[1], lists[2])
        dev.agree(m.reserve(lists[3], lists[4]))


def test_a_serving_loop(gdn):
    """Reserve, prologue, attention, fork, free and compact as a server uses them, on a mixed batch: each step's
    outputs against attention in 64 bits over what the prologue was given."""
    H_q, H_kv, d, page, R, width, N = 4, 2, 64, 16, 10, 8, 40
    m = Model(R, width, N, page)
    dev = Device(gdn, m, H_kv=H_kv, d=d)
    g = torch.Generator().manual_seed(11)
    freqs = gdn.rope_freqs(32, 10000.0, device="cpu")
    fd = freqs.cuda()
    remap = torch.empty(N, dtype=torch.int32, device="cuda")
    ws = torch.empty(gdn.attn_paged_workspace_bytes(4, 64, 32, H_q, H_kv, d), dtype=torch.uint8, device="cuda")
    history = {}  # row -> [(k, v)] as the cache holds them, bf16

    def step(batch):
        rows, n = [r for r, _ in batch], [x for _, x in batch]
        dev.reserve(rows, n)
        missed = m.reserve(rows, n)
        assert not missed
        dev.agree(missed)
        T = sum(n)
        q, k, v = (torch.randn(T, h, d, generator=g).to(A.BF) for h in (H_q, H_kv, H_kv))
        cu = [0]
        for x in n:
            cu.append(cu[-1] + x)
        qd, out = q.cuda(), torch.empty(T, H_q, d, dtype=A.BF, device="cuda")
        rd, cd = dev.ints(rows), dev.ints(cu)
        gdn.attn_prologue(qd, k.cuda(), v.cuda(), qd, dev.k, dev.v, dev.table, dev.len, rd, cd, fd)
        gdn.attn_paged(qd, dev.k, dev.v, dev.table, dev.len, rd, cd, out, ws, max_new=32)
        torch.cuda.synchronize()
        for b, (r, x) in enumerate(batch):
            c = A.Cache([(x, m.len[r] - x)], H_q=H_q, H_kv=H_kv, d=d, page=page)
            ks, fp32 = A.prologue(c, k[cu[b]:cu[b + 1]], freqs)
            qs, _ = A.prologue(c, q[cu[b]:cu[b + 1]], freqs)
            # q and k as the kernel rounded them (each within a bf16 step of its reference), so
            # that the attention's own tolerance holds
            got_q = qd[cu[b]:cu[b + 1]].cpu()
            A.check(got_q, qs, A.U_BF * qs.abs() + 1e-5, "q")
            for i in range(x):
                p = m.len[r] - x + i
                cell = m.table[r][p // page], p % page
                got_k = dev.k[cell[0], :, cell[1]].cpu()
                A.check(got_k, ks[i], A.U_BF * ks[i].abs() + 1e-5, "k")
                history.setdefault(r, []).append((got_k, v[cu[b] + i]))
            c.q = got_q
            flat_k = torch.stack([a for a, _ in history[r]])
            flat_v = torch.stack([a for _, a in history[r]])
            c.gather = lambda _, h, w: (flat_k if w == "k" else flat_v)[:, h].double()
            want, _, tol, _ = A.attention(c, d ** -0.5)
            A.check(out[cu[b]:cu[b + 1]], want, tol, f"row {r}")

    step([(1, 20), (2, 1), (3, 17)])
    step([(3, 1), (1, 1), (2, 5)])
    dev.fork([1, 3], [5, 6])
    m.fork([1, 3], [5, 6])
    history[5], history[6] = list(history[1]), list(history[3])
    step([(5, 1), (1, 3), (6, 16)])
    dev.free([1, 2])
    m.free([1, 2])
    del history[1], history[2]
    gdn.kv_page_compact(dev.k, dev.v, dev.table, dev.refs, remap, dev.result, dev.ws)
    m.compact()
    dev.agree()
    step([(5, 1), (6, 1), (3, 1), (7, 32)])
    step([(7, 1), (5, 1)])
