"""The paged 8-bit cache as a server uses it: decode steps of the two-launch form, whose long requests are shared out among
blocks, captured and replayed with new tokens, from several threads and in graphs that run at the same time; allocator steps
that cannot serve a request."""
import threading

import pytest
import torch

import causal_sliding_window_swa_b200 as swa
from tests import kv8_plain
from tests.test_kv8_gpu import Batch, GpuCache, bf16, f64, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield


WIDE = 4096       # entries of a block table for requests so long that a step takes the two-launch form


class Server:
    """Requests with prompts in the cache, and their next tokens."""

    def __init__(self, prompts, H, Hkv, D, P, steps, seed):
        g = torch.Generator().manual_seed(seed)
        B, self.P, self.H, self.Hkv, self.D = len(prompts), P, H, Hkv, D
        n_pages = sum(-(-(n + steps) // P) for n in prompts) + 2
        self.table = torch.full((B, WIDE), -1, dtype=torch.int32, device="cuda")
        self.kv_len, self.first, self.pool = i32([0] * B), i32([0] * B), i32([0, n_pages])
        self.ring = torch.randperm(n_pages, generator=g).int().cuda()
        self.cache = GpuCache(n_pages, Hkv, P, D)
        self.one = i32([1] * B)
        T = max(prompts)
        slots, _ = swa.kv_pages(self.table, self.kv_len, self.first, self.ring, self.pool, i32(prompts), P, T=T)
        kh = torch.randn((B, T, Hkv, D), generator=g)
        kh = (kh * torch.rsqrt(kh.square().mean(-1, keepdim=True))).to(torch.bfloat16).cuda()
        vp = torch.randn((B, T, Hkv, D), generator=g).to(torch.bfloat16).cuda()
        swa.kv8_write(kh, vp, slots, *self.cache.all())
        mk = lambda h: torch.randn((steps, B, h, D), generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        self.q, self.k, self.v = mk(H), mk(Hkv), mk(Hkv)
        self.ws = torch.full((swa.swa_attn_kv8_decode_workspace_bytes(B, H, Hkv, D),), 255, dtype=torch.uint8, device="cuda")

    def step(self, q, k, v, **kw):
        _, n = swa.kv_pages(self.table, self.kv_len, self.first, self.ring, self.pool, self.one, self.P)
        return swa.decode_kv8(q, k, v, *self.cache.all(), self.table, n, **kw)

    def capture(self, stream=None):
        """Graph of one step on the buffers self.buf, and its results."""
        self.buf = [t[0].clone() for t in (self.q, self.k, self.v)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            res = self.step(*self.buf, workspace=self.ws)
        return graph, res

    def state(self):
        return [t.clone() for t in (self.table, self.kv_len, self.ring, self.pool, self.cache.k.view(torch.uint8),
                                    self.cache.v.view(torch.uint8), torch.nan_to_num(self.cache.ks), torch.nan_to_num(self.cache.vs))]


# long requests whose chunks several blocks share, beside short ones; one group of heads to a warp, two, and sets of warps
SERVERS = [([1500, 1100, 70, 1], 4, 4, 64, 16), ([2100, 333], 16, 2, 128, 32), ([1800, 64], 12, 1, 128, 64), ([1300, 40], 32, 1, 128, 128)]
STEPS = 20


def _eager(case, seed):
    s = Server(*case, STEPS, seed)
    out = [[t.clone() for t in s.step(s.q[i], s.k[i], s.v[i])] for i in range(STEPS)]
    swa.check_device_status()
    return out, s.state()


@pytest.mark.parametrize("case", SERVERS, ids=[f"H{c[1]}/{c[2]} D{c[3]} P{c[4]}" for c in SERVERS])
def test_replays_of_two_launch_steps_with_new_tokens(case):
    want, end = _eager(case, 1)
    s = Server(*case, STEPS, 1)
    graph, res = s.capture()
    for i in range(STEPS):
        for d, t in zip(s.buf, (s.q, s.k, s.v)):
            d.copy_(t[i])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(res, want[i])), i
    assert all(torch.equal(a, b) for a, b in zip(s.state(), end))
    # and the last step is what 64-bit attention over the cached rows gives
    out, lse = want[-1]
    for b, n in enumerate(n0 + STEPS for n0 in case[0]):
        pos = torch.arange(n, device="cuda")
        slots = (s.table[b, pos // s.P].long() * s.P + pos % s.P).int()[None].contiguous()
        k, v = (t[0].double().cpu().numpy() for t in swa.kv8_read(slots, *s.cache.all()))
        qh = bf16(kv8_plain.prologue(f64(s.q[-1, b]), n - 1)).double().numpy()
        ref, ref_l, mag = kv8_plain.attend(qh, k, v)
        assert (abs(f64(out[b]) - ref) <= kv8_plain.out_tolerance(ref, mag)).all()
        assert (abs(f64(lse[b]) - ref_l) <= kv8_plain.lse_tolerance(ref_l, s.D)).all()
    swa.check_device_status()


def test_graphs_of_two_launch_steps_that_run_at_the_same_time():
    """Two servers' steps, captured with workspaces of their own, replayed on two streams without waiting for one another."""
    cases = [SERVERS[0], SERVERS[1]]
    want = [_eager(c, 2 + i) for i, c in enumerate(cases)]
    servers = [Server(*c, STEPS, 2 + i) for i, c in enumerate(cases)]
    streams = [torch.cuda.Stream() for _ in cases]
    graphs = [s.capture(st) for s, st in zip(servers, streams)]
    kept = [[], []]
    torch.cuda.synchronize()
    for i in range(STEPS):
        for x, (s, st, (graph, res)) in enumerate(zip(servers, streams, graphs)):
            with torch.cuda.stream(st):
                for d, t in zip(s.buf, (s.q, s.k, s.v)):
                    d.copy_(t[i])
                graph.replay()
                kept[x].append([t.clone() for t in res])
    torch.cuda.synchronize()
    for x, (out, end) in enumerate(want):
        assert all(torch.equal(a, b) for got, w in zip(kept[x], out) for a, b in zip(got, w))
        assert all(torch.equal(a, b) for a, b in zip(servers[x].state(), end))
    swa.check_device_status()


@pytest.mark.parametrize("H,Hkv,D,P", [(4, 2, 128, 32), (12, 1, 64, 64), (3, 3, 64, 128)])
def test_two_launch_steps_from_threads_and_streams(H, Hkv, D, P):
    x = Batch([2000, 20, 1111], H, Hkv, D, P, 0, seed=22)
    out, lse = x.run(wide=WIDE)
    x.append_plain()
    x.check(out, lse)
    torch.cuda.synchronize()
    got = [[] for _ in range(4)]
    go = threading.Barrier(4)

    def work(i):
        torch.cuda.set_device(0)
        st = torch.cuda.Stream()
        go.wait()
        for _ in range(10):
            with torch.cuda.stream(st):
                got[i].append(x.run(append=False, wide=WIDE))
        st.synchronize()

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert all(len(r) == 10 and torch.equal(o, out) and torch.equal(l, lse) for r in got for o, l in r)
    swa.check_device_status()


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("T", [1, 40, 2000])
def test_requests_that_cannot_be_served_still_give_back_what_their_window_has_passed(T, in_place):
    """Window 20, pages of 16, 5 table entries.  Requests: more new tokens than T; more pages than the table has; idle; served; a
    first_page that is not possible; a kv_len that is not possible; an impossible one that has ended."""
    L, F = [64, 80, 64, 64, 50, 81, -1], [1, 0, 0, 0, 5, 0, 0]
    news = [T + 1, 1, 0, 1, 1, 1, -1]
    table = torch.full((7, 5), -1, dtype=torch.int32)
    page = iter(range(100))
    for b in range(7):
        for j in range(max(0, F[b]), min(5, -(-max(0, L[b]) // 16))):
            table[b, j] = next(page)
    held = next(page)
    N = held + 6
    ring = torch.arange(N, dtype=torch.int32).roll(-held).cuda()          # free: pages held .. N - 1
    state = [table.cuda(), i32(L), i32(F), i32([0, 6])]
    out = None if in_place else tuple(torch.full_like(t, -7) for t in state)
    slots, step_len = swa.kv_pages(state[0], state[1], state[2], ring, state[3], i32(news), 16, 20, T, out=out)
    got = [t.tolist() for t in (out or state)]
    # pages before max(0, L - 19) // 16 go back: entries 1 of the first, 0 .. 2 of the second, 0 and 1 of the next two
    want = table.clone()
    back = []
    for b, upto in ((0, 2), (1, 3), (2, 2), (3, 2)):
        back += want[b, F[b]:upto].tolist()
        want[b, F[b]:upto] = -1
    want[3, 4] = held
    assert got[0] == want.tolist() and got[1] == [64, 80, 64, 65, 50, 81, -1] and got[2] == [2, 3, 2, 2, 5, 0, 0]
    assert got[3] == [1, 6 - 1 + len(back)] and len(back) == 8
    assert ring.tolist()[6:14] == back and ring.tolist()[:6] == list(range(held, N))
    assert step_len.tolist() == [0, 0, 0, 65, 0, 0, 0] and slots[3, 0] == held * 16
    assert (slots.cpu().flatten() >= 0).sum() == 1
    swa.check_device_status()
