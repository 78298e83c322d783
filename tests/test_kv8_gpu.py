"""The paged 8-bit cache and the decode step over it on the GPU, against the plain 64-bit statements of
``tests/kv8_plain.py`` (tolerances derived there): the allocator and the cached codes have to be equal, outputs are held
to the rounding of their type and of the weights."""
import os
import random
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import causal_sliding_window_swa_b200 as swa
import oracle
import workloads
from tests import kv8_plain

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def bf16(x):
    """64-bit values to bf16 in one rounding (a cast by way of 32 bits may round twice)."""
    m, e = np.frexp(x)
    return torch.from_numpy(np.ldexp(np.rint(m * 256), e - 8)).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


class GpuCache:
    """The tensors of a cache; codes and scales start as NaNs, which no result may show."""

    def __init__(self, n_pages, Hkv, P, D):
        self.P = P
        self.k = torch.full((n_pages, Hkv, P, D), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        self.v = self.k.clone()
        self.ks = torch.full((n_pages, Hkv), float("nan"), device="cuda")
        self.vs = self.ks.clone()
        self.plain = kv8_plain.Cache(n_pages, Hkv, P, D), kv8_plain.Cache(n_pages, Hkv, P, D)

    def all(self):
        return self.k, self.v, self.ks, self.vs

    def write(self, kh, vp, slots, **kw):
        swa.kv8_write(kh, vp, slots, *self.all(), **kw)
        self.write_plain(kh, vp, slots)

    def write_plain(self, kh, vp, slots):
        for c, x in zip(self.plain, (kh, vp)):
            c.write(f64(x).reshape(-1, *x.shape[2:]), slots.reshape(-1).tolist())

    def check(self, slots):
        """Codes and scales of the given slots, bit by bit (0 and -0 are one value)."""
        slots = [int(s) for s in slots if s >= 0]
        page, off = np.array(slots) // self.P, np.array(slots) % self.P
        for codes, scale, c in ((self.k, self.ks, self.plain[0]), (self.v, self.vs, self.plain[1])):
            got = kv8_plain.TABLE[codes.view(torch.uint8).cpu().numpy()[page, :, off]]
            np.testing.assert_array_equal(got, c.codes[page, :, off])
            np.testing.assert_array_equal(np.log2(f64(scale)[page]), c.e[page])


# ------------------------------------------------------------------------------------------ allocator

def _state(B, M, N):
    return [torch.full((B, M), -1, dtype=torch.int32, device="cuda"), i32([0] * B), i32([0] * B), i32([0, N])], \
        torch.arange(N, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,M,N,P,W,T,steps", [
    (1, 1, 1, 16, 0, 1, 20), (3, 5, 9, 16, 0, 40, 30), (9, 12, 60, 16, 70, 50, 60), (40, 7, 130, 32, 33, 1, 80),
    (5, 33, 100, 128, 1, 700, 20), (1030, 4, 2500, 16, 20, 3, 25), (2500, 3, 4000, 64, 0, 64, 12), (70, 40, 1500, 64, 1024, 300, 30),
])
@pytest.mark.parametrize("in_place", [True, False])
def test_allocator_steps_equal_the_plain_ones(B, M, N, P, W, T, steps, in_place):
    r = random.Random(B + N)
    a = kv8_plain.Pages(B, M, N, P, W)
    state, ring = _state(B, M, N)
    for _ in range(steps):
        news = [-r.randint(1, 9) if r.random() < 0.06 else r.choice([0, 1, 1, r.randint(0, T + 1)]) for _ in range(B)]
        out = None if in_place else tuple(torch.full_like(t, -7) for t in state)
        slots, step_len = swa.kv_pages(state[0], state[1], state[2], ring, state[3], i32(news), P, W, T, out=out)
        if not in_place:      # the inputs are as they were, and the step can be repeated from them
            again = tuple(torch.empty_like(t) for t in state)
            ring1 = ring.clone()
            s2, l2 = swa.kv_pages(state[0], state[1], state[2], ring, state[3], i32(news), P, W, T, out=again)
            assert torch.equal(ring, ring1) and torch.equal(s2, slots) and torch.equal(l2, step_len)
            assert all(torch.equal(x, y) for x, y in zip(out, again))
            state = list(out)
        want_slots, want_len = a.step(news, T)
        assert slots.tolist() == want_slots and step_len.tolist() == want_len
        assert state[0].tolist() == a.table and state[1].tolist() == a.kv_len and state[2].tolist() == a.first
        assert state[3].tolist() == [a.head, a.free] and ring.tolist() == a.ring
    swa.check_device_status()


@pytest.mark.parametrize("T", [1, 2000])
def test_allocator_leaves_impossible_requests_alone(T):
    # no length; more than 4 pages of 16 hold; fine; no first page; pages given back that it never had; an ended one of those
    state, ring = _state(6, 4, 20)
    state[1].copy_(i32([-5, 100, 3, 0, 20, 65]))
    state[2].copy_(i32([0, 0, 0, -1, 3, 0]))
    state[0][2, 0] = 19
    state[3].copy_(i32([0, 19]))
    was = [t.tolist() for t in state]
    slots, step_len = swa.kv_pages(state[0], state[1], state[2], ring, state[3], i32([1, 1, 1, 1, 1, -1]), 16, T=T)
    assert step_len.tolist() == [0, 0, 4, 0, 0, 0]
    assert slots[:, 0].tolist() == [-1, -1, 19 * 16 + 3, -1, -1, -1] and (slots[:, 1:] == -1).all()
    was[1][2] = 4
    assert [t.tolist() for t in state] == was and ring.tolist() == list(range(20))


# ---------------------------------------------------------------------------------------- write, read

@pytest.mark.parametrize("D,P,Hkv,lens", [
    (64, 16, 1, [1]), (128, 16, 3, [5, 16, 17, 1, 40]), (64, 32, 2, [31, 33, 64]), (128, 32, 2, [100, 7]), (64, 64, 5, [1, 63, 130]),
    (128, 64, 12, [200, 64, 65]), (64, 128, 2, [127, 1, 300]), (128, 128, 1, [129, 256, 5]), (128, 64, 1, [1500, 3]),
])
def test_write_and_read(D, P, Hkv, lens):
    g = torch.Generator().manual_seed(P + D + len(lens))
    B = len(lens)
    n_pages = sum(-(-n // P) + 1 for n in lens) + 2
    a = kv8_plain.Pages(B, max(lens) // P + 2, n_pages, P, 0)
    cache = GpuCache(n_pages, Hkv, P, D)
    used = []
    for news in (lens, [1] * B, [0 if b == 1 else 3 for b in range(B)], [P + 1] * B, [1] * B):
        T = max(news)
        if sum(-(-(n + m) // P) - -(-n // P) for n, m in zip(a.kv_len, news)) > a.free:
            break
        slots, _ = a.step(news, T)
        kh = torch.randn((B, T, Hkv, D), generator=g).to(torch.bfloat16).cuda()
        vp = (torch.randn((B, T, Hkv, D), generator=g) * torch.exp(2 * torch.randn((B, T, Hkv, 1), generator=g))).to(torch.bfloat16).cuda()
        cache.write(kh, vp, i32(slots))
        used += [s for row in slots for s in row if s >= 0]
        cache.check(used)
    assert len(used) > sum(lens)
    # what was not written is as it was
    left = np.setdiff1d(np.arange(n_pages * P), used)
    page, off = left // P, left % P
    for t in (cache.k, cache.v):
        assert (t.view(torch.uint8).cpu().numpy()[page, :, off] == 0x7f).all()
    assert torch.isnan(cache.ks[sorted(set(range(n_pages)) - {s // P for s in used})]).all()
    # read back: any order, repeated slots, empty rows
    rows = torch.tensor(used + [-1, used[0], -5])[torch.randperm(len(used) + 3, generator=g)]
    kh, vp = swa.kv8_read(rows.int().cuda()[None].contiguous(), *cache.all())
    for got, c in ((kh, cache.plain[0]), (vp, cache.plain[1])):
        np.testing.assert_array_equal(f64(got)[0], c.values(rows.tolist()))
    swa.check_device_status()


@pytest.mark.parametrize("B,T", [(1, 500), (9, 47), (60, 2), (300, 1), (5, 130)])
@pytest.mark.parametrize("D,P,Hkv", [(64, 16, 2), (128, 16, 1), (64, 32, 1), (128, 32, 2), (64, 64, 1), (128, 64, 2), (64, 128, 2), (128, 128, 1)])
def test_write_runs_anywhere(B, T, D, P, Hkv):
    """Runs of all lengths at all offsets, wherever they lie in a call's rows: between skipped rows, from one request's row into
    the next one's, several in a page's worth of tokens; three calls into the same pages, each page by one run a call."""
    r = random.Random(B * T + D + P)
    g = torch.Generator().manual_seed(P + D)
    n_pages = B * T // 2 + 4
    cache = GpuCache(n_pages, Hkv, P, D)
    fill = [0] * n_pages
    for _ in range(3):
        free = r.sample(range(n_pages), n_pages)
        flat = []
        while len(flat) < B * T:
            what = r.choice(["skip", "one", "short", "rest", "rest"])
            if what == "skip" or not free:
                flat += [-r.randint(1, 9)] * r.choice([1, 1, 2, r.randint(1, 2 * P)])
                continue
            page = free.pop()
            off = fill[page] if fill[page] < P else 0            # a full page is begun again
            n = min(P - off, {"one": 1, "short": r.randint(1, 5), "rest": P}[what], B * T - len(flat))
            flat += range(page * P + off, page * P + off + n)
            fill[page] = off + n
        slots = torch.tensor(flat[:B * T], dtype=torch.int32).view(B, T)
        kh = torch.randn((B, T, Hkv, D), generator=g).to(torch.bfloat16).cuda()
        vp = (torch.randn((B, T, Hkv, D), generator=g) * torch.exp(2 * torch.randn((B, T, Hkv, 1), generator=g))).to(torch.bfloat16).cuda()
        cache.write(kh, vp, slots.cuda())
        cache.check([p * P + i for p, n in enumerate(fill) for i in range(n)])
    swa.check_device_status()


def test_read_rows_written_elsewhere_are_the_same_values():
    # a request that moves: its rows as bf16, into other pages of another page size
    g = torch.Generator().manual_seed(5)
    a, b = GpuCache(6, 2, 32, 128), GpuCache(9, 2, 16, 128)
    slots = torch.arange(70, dtype=torch.int32, device="cuda")[None] + 64
    kh, vp = (torch.randn((1, 70, 2, 128), generator=g).to(torch.bfloat16).cuda() for _ in "kv")
    a.write(kh, vp, slots)
    k1, v1 = swa.kv8_read(slots, *a.all())
    swa.kv8_write(k1, v1, slots - 32, *b.all())
    k2, v2 = swa.kv8_read(slots - 32, *b.all())
    assert torch.equal(k1, k2) and torch.equal(v1, v2)


def test_infinities_nans_zeros_and_extremes():
    x = torch.zeros((1, 5, 1, 64), dtype=torch.bfloat16)
    x[0, 0, 0, :3] = torch.tensor([1.0, float("nan"), -2.0])
    x[0, 2, 0, :2] = torch.tensor([3e38, -1e-38])
    x[0, 3, 0, :2] = torch.tensor([float("inf"), float("-inf")])
    x[0, 4, 0, :4] = torch.tensor([1e-20, -1e-40, 0.0, 1e-19])
    cache = GpuCache(6, 1, 16, 64)
    slots = i32([[5, 16, 32, 48, 64]])
    slots[0, 0] = 0
    swa.kv8_write(x.cuda(), x.cuda(), slots, *cache.all())
    assert torch.log2(cache.ks[:5, 0]).tolist() == [-7, -60, kv8_plain.exponent(f64(x[0, 2])), 120, -60]
    kh, vp = swa.kv8_read(slots, *cache.all())
    kh = kh.cpu()[0, :, 0]
    assert kh[0, 0] == 1 and torch.isnan(kh[0, 1]) and kh[0, 2] == -2 and (kh[0, 3:] == 0).all()
    assert (kh[1] == 0).all() and abs(kh[2, 0].double() / 3e38 - 1) <= 2 ** -4 + 2 ** -8
    assert kh[3, 0] == float("inf") and kh[3, 1] == float("-inf")
    assert abs(kh[4, 0].double() - 1e-20) <= 2.0 ** -70 and abs(kh[4, 3].double() / 1e-19 - 1) <= 2 ** -4 + 2 ** -8
    assert torch.equal(kh.view(torch.int16), vp.cpu()[0, :, 0].view(torch.int16))


def test_slots_past_the_cache_are_recorded_and_skipped():
    swa.check_device_status()
    x = torch.ones((1, 3, 1, 64), dtype=torch.bfloat16, device="cuda")
    cache = GpuCache(2, 1, 16, 64)
    slots = i32([[0, 32, 2 ** 31 - 1]])
    swa.kv8_write(x, x, slots, *cache.all())
    rc, detail = swa.swa_attn_last_device_status()
    assert rc == swa.SWA_ERR_INVALID_ARG and (detail >> 8) & 0xff == 80
    kh, vp = swa.kv8_read(slots, *cache.all())
    assert swa.swa_attn_last_device_status()[0] == swa.SWA_ERR_INVALID_ARG
    assert kh[0, :, 0, 0].tolist() == [1, 0, 0] and vp[0, :, 0, 5].tolist() == [1, 0, 0]
    assert (cache.k.view(torch.uint8)[1] == 0x7f).all()


# --------------------------------------------------------------------------------------------- decode

class Batch:
    """Requests with cached tokens in shuffled pages, held only from the first page that the window needs."""

    def __init__(self, lens, H, Hkv, D, P, window, seed, ve=False, doc=False):
        self.g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.Hkv, self.D, self.P, self.window = lens, H, Hkv, D, P, window
        B = len(lens)
        first = [(max(0, n - window) if window > 0 else 0) // P for n in lens]
        last = [-(-n // P) for n in lens]
        n_pages = sum(max(0, z - a) for a, z in zip(first, last)) + 3
        perm = torch.randperm(n_pages, generator=self.g).tolist()
        width = max(1, max(last))
        self.table = torch.full((B, width), -1, dtype=torch.int32)
        for b in range(B):
            for j in range(first[b], last[b]):
                self.table[b, j] = perm.pop()
        self.cache = GpuCache(n_pages, Hkv, P, D)
        # the tokens before the new one, as rows of unit root mean square and as values of changing size
        T = max(max(lens) - 1, 1)
        slots = torch.full((B, T), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            for t in range(first[b] * P, n - 1):
                slots[b, t] = int(self.table[b, t // P]) * P + t % P
        kh = torch.randn((B, T, Hkv, D), generator=self.g)
        kh = kh * torch.rsqrt(kh.square().mean(-1, keepdim=True))
        vp = torch.randn((B, T, Hkv, D), generator=self.g) * torch.exp(torch.randn((B, T, Hkv, 1), generator=self.g))
        self.cache.write(kh.to(torch.bfloat16).cuda(), vp.to(torch.bfloat16).cuda(), slots.cuda())
        mk = lambda *s: torch.randn(s, generator=self.g).to(torch.bfloat16).cuda()  # noqa: E731
        self.q, self.k, self.v = mk(B, H, D), mk(B, Hkv, D), mk(B, Hkv, D)
        self.ve, self.gate_x, self.Wg = (mk(B, Hkv, D), mk(B, 32), mk(32, Hkv)) if ve else (None,) * 3
        self.start = [0 if n < 2 else int(torch.randint(0, n + 3, (1,), generator=self.g)) for n in lens] if doc else None

    def run(self, append=True, **kw):
        seq = kw.pop("seq_len", None)
        seq = i32(self.lens) if seq is None else seq
        k, v, ve, gx, wg = (self.k, self.v, self.ve, self.gate_x, self.Wg) if append else (None,) * 5
        # a table for much longer requests: the call cannot count on short ones, and goes another way
        table = torch.nn.functional.pad(self.table, (0, kw.pop("wide", 0)), value=-1)
        return swa.decode_kv8(self.q, k, v, *self.cache.all(), table.cuda(), seq, self.window, ve, gx, wg,
                              doc_start=None if self.start is None else i32(self.start), **kw)

    def token(self, b):
        """khat and v' of request b's new token, rounded to bf16, and its slot."""
        pos = self.lens[b] - 1
        kh = bf16(kv8_plain.prologue(f64(self.k[b]), pos))
        vp = f64(self.v[b])
        if self.ve is not None:
            z = f64(self.gate_x[b]) @ f64(self.Wg)
            vp = vp + (2 / (1 + np.exp(-z)))[:, None] * f64(self.ve[b])
        return kh, bf16(vp), int(self.table[b, pos // self.P]) * self.P + pos % self.P

    def append_plain(self):
        for b, n in enumerate(self.lens):
            if n > 0:
                kh, vp, slot = self.token(b)
                self.cache.write_plain(kh[None, None], vp[None, None], torch.tensor([[slot]]))

    def check(self, out, lse, bad_pages=()):
        out, lse = f64(out), f64(lse)
        for b, n in enumerate(self.lens):
            if n <= 0:
                assert (out[b] == 0).all() and (lse[b] == -np.inf).all()
                continue
            lo = kv8_plain.visible(n, self.window, self.start[b] if self.start else 0)
            slots = [int(self.table[b, t // self.P]) * self.P + t % self.P for t in range(lo, n)
                     if int(self.table[b, t // self.P]) not in bad_pages]
            k, v = (c.values(slots) for c in self.cache.plain)
            q = f64(bf16(kv8_plain.prologue(f64(self.q[b]), n - 1)))
            ref, ref_l, mag = kv8_plain.attend(q, k, v)
            tol = kv8_plain.out_tolerance(ref, mag)
            worst = np.abs(out[b] - ref) / tol
            assert worst.max() <= 1, (b, n, worst.max())
            err = np.abs(lse[b] - ref_l)
            assert (err <= kv8_plain.lse_tolerance(ref_l, self.D)).all(), (b, n, err.max())


CASES = [
    # lens, H, Hkv, D, P, window, ve, doc
    ([1], 1, 1, 64, 16, 0, False, False),
    ([2, 0, 1], 2, 2, 128, 16, 0, True, False),
    ([16, 17, 15, 33], 3, 3, 64, 16, 0, False, False),
    ([300], 12, 12, 64, 16, 0, False, False),
    ([129, 1, 0, 128, 127, 257], 4, 2, 128, 64, 100, True, False),
    ([700, 5, 64, 65, 1000], 8, 1, 128, 32, 0, False, True),
    ([513, 90], 16, 2, 64, 128, 1, False, False),
    ([400, 31, 32], 20, 4, 128, 16, 300, True, True),
    ([1111, 222], 24, 2, 64, 64, 0, False, False),          # 12 heads to a key/value head
    ([640, 3], 66, 2, 128, 32, 257, False, True),           # 33
    ([200, 600], 64, 1, 128, 16, 0, False, False),          # 64
    ([150] * 40, 5, 5, 64, 64, 128, False, False),
    ([3000, 2999, 10, 2048], 12, 12, 128, 64, 1024, True, False),
    ([449, 500, 512, 1], 4, 4, 128, 128, 300, True, False),
    ([5000], 2, 1, 128, 128, 0, False, False),
    ([257 + 13 * i for i in range(30)], 6, 3, 64, 32, 0, False, True),
]


@pytest.mark.parametrize("wide", [0, 4096])
@pytest.mark.parametrize("case", CASES, ids=[f"{len(c[0])}x{max(c[0])} H{c[1]}/{c[2]} D{c[3]} P{c[4]} W{c[5]}" for c in CASES])
def test_decode_matches_the_plain_statement(case, wide):
    lens, H, Hkv, D, P, window, ve, doc = case
    window = window or (1 << 30 if wide else 0)
    x = Batch(lens, H, Hkv, D, P, window, seed=sum(lens) + H, ve=ve, doc=doc)
    out, lse = x.run(wide=wide)
    x.append_plain()
    used = [x.token(b)[2] for b, n in enumerate(lens) if n > 0]
    x.cache.check([p * P + i for s in used for p, o in [divmod(s, P)] for i in range(o + 1)])
    x.check(out, lse)
    # the token is there now: the same step without it, with the caller's outputs and workspace; and repeated, bit for bit
    o2, l2 = torch.full_like(out, float("nan")), torch.full_like(lse, float("nan"))
    ws = torch.full((swa.swa_attn_kv8_decode_workspace_bytes(len(lens), H, Hkv, D),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        x.run(append=False, out=o2, lse=l2, workspace=ws, wide=wide)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    o3, l3 = x.run(wide=wide)          # the same token again: it takes the place it has
    assert torch.equal(o3, out) and torch.equal(l3, lse)
    swa.check_device_status()


@pytest.mark.parametrize("B,H,Hkv,D,P,window,most", [
    (24, 8, 8, 128, 64, 0, 3000), (40, 8, 8, 64, 16, 0, 2500), (60, 16, 2, 128, 32, 2000, 4000), (30, 12, 6, 64, 128, 0, 5000),
    (50, 30, 2, 128, 64, 0, 6000), (90, 24, 1, 64, 16, 5000, 9000), (60, 32, 1, 128, 128, 0, 9000), (60, 48, 1, 128, 64, 0, 5000),
    (100, 64, 1, 64, 32, 0, 4000), (256, 12, 12, 128, 64, 0, 129), (1000, 3, 3, 64, 16, 100, 200),
    (24, 8, 1, 128, 64, 0, 9000), (20, 4, 4, 128, 16, 0, 7000), (64, 12, 12, 128, 64, 1500, 3500), (13, 12, 12, 128, 64, 0, 2040),
    (12, 12, 12, 64, 64, 0, 1000), (7, 24, 12, 128, 32, 0, 1000), (5, 12, 12, 64, 64, 0, 900), (4, 12, 12, 128, 16, 0, 1500),
    (1, 12, 12, 64, 16, 0, 2900),
])
def test_decode_many_units_for_each_block(B, H, Hkv, D, P, window, most):
    """Many chunks of keys for each block, so that the ring of stages goes round many times: all requests against 64-bit
    attention over what kv8_read returns of the cache (which the tests above hold to the plain codes)."""
    g = torch.Generator("cuda").manual_seed(B + D)
    r = random.Random(B)
    lens = [most] + [r.choice([0, 1, 64, 65, r.randint(1, most), r.randint(most // 2, most)]) for _ in range(B - 1)]
    cnt = [-(-n // P) for n in lens]
    n_pages = sum(cnt) + 1
    perm = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.full((B, max(cnt)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(cnt):
        table[b, :c] = perm[at:at + c]
        at += c
    cache = []
    for _ in "kv":
        x = torch.randn((n_pages, Hkv, P, D), generator=g, device="cuda") * 64
        cache.append(x.to(torch.float8_e4m3fn))
    ks = torch.full((n_pages, Hkv), 2.0 ** -6, device="cuda")
    vs = torch.exp2(torch.randint(-9, 3, (n_pages, Hkv), generator=g, device="cuda").float())
    q = torch.randn((B, H, D), generator=g, device="cuda").to(torch.bfloat16)
    for _ in range(3):
        out, lse = swa.decode_kv8(q, None, None, *cache, ks, vs, table, i32(lens), window)
    swa.check_device_status()
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all() and (lse[b] == float("-inf")).all()
            continue
        lo = kv8_plain.visible(n, window, 0)
        pos = torch.arange(lo, n, device="cuda")
        slots = (table[b, pos // P].long() * P + pos % P).int()[None].contiguous()
        k, v = (t[0].double().transpose(0, 1) for t in swa.kv8_read(slots, *cache, ks, vs))      # (Hkv, n, D)
        qh = bf16(kv8_plain.prologue(f64(q[b]), n - 1)).double().cuda().view(Hkv, H // Hkv, D)
        s = qh @ k.transpose(1, 2) / D ** 0.5
        p = torch.softmax(s, -1)
        ref, mag = (p @ v).reshape(H, D).cpu().numpy(), (p @ v.abs()).reshape(H, D).cpu().numpy()
        ref_l = torch.logsumexp(s, -1).reshape(H).cpu().numpy()
        worst = np.abs(f64(out[b]) - ref) / kv8_plain.out_tolerance(ref, mag)
        assert worst.max() <= 1, (b, n, worst.max())
        # the keys here are rows of root mean square up to 1.3
        assert (np.abs(f64(lse[b]) - ref_l) <= 2 * kv8_plain.lse_tolerance(ref_l, D)).all(), (b, n)


@pytest.mark.parametrize("wide", [0, 4096])
def test_adversarial_scores_and_scales(wide):
    # keys along the query and against it, so that probabilities span the whole range; values of very different size in
    # neighbouring pages
    H, D, P, n = 2, 128, 16, 200
    x = Batch([n, n], H, H, D, P, 0, seed=9)
    q = np.stack([kv8_plain.prologue(f64(x.q[b]), n - 1) for b in range(2)])
    t = np.arange(n - 1)
    sign = np.where(t < 100, -1.0, np.where(t == 150, 1.0, -0.5))
    kh = bf16(q[:, None] * sign[None, :, None, None]).cuda()
    size = 2.0 ** (((t // P) * 7) % 23 - 11)
    vp = (torch.randn((2, n - 1, H, D), generator=x.g).double() * torch.from_numpy(size)[None, :, None, None]).to(torch.bfloat16).cuda()
    vp[0, :64] = 0
    slots = torch.stack([torch.tensor([int(x.table[b, u // P]) * P + u % P for u in t]) for b in range(2)]).int().cuda()
    x.cache.write(kh, vp, slots.contiguous())
    out, lse = x.run(wide=wide)
    x.append_plain()
    x.check(out, lse)


@pytest.mark.parametrize("wide", [0, 4096])
@pytest.mark.parametrize("P", [16, 64, 128])
def test_the_scale_of_the_last_page_grows_under_the_step(P, wide):
    # new tokens far larger than what their pages hold: the codes that are there move to the new scale in the same step
    x = Batch([P + P // 2 + 3, 2 * P, 5, P + 1], 4, 4, 128, P, 0, seed=P)
    x.v *= 64
    x.k *= 0
    x.k[:, :, 0] = 8             # khat has one large element
    out, lse = x.run(wide=wide)
    before = x.cache.plain[1].e.copy()
    x.append_plain()
    assert (x.cache.plain[1].e > before).any()
    x.cache.check([int(x.table[b, t // P]) * P + t % P for b, n in enumerate(x.lens) for t in range(n)])
    x.check(out, lse)


@pytest.mark.parametrize("wide", [0, 4096])
def test_values_that_are_not_visible_do_not_matter(wide):
    # NaN codes and scales in pages outside the window, behind the last token, and in rows before the document start
    x = Batch([100, 77], 4, 2, 64, 16, 40, seed=3, doc=True)
    x.start = [70, 0]
    out, lse = x.run(wide=wide)
    for b, n in enumerate(x.lens):
        lo = kv8_plain.visible(n, 40, x.start[b])
        for t in range(lo // 16 * 16, lo):
            page, off = int(x.table[b, t // 16]), t % 16
            x.cache.k.view(torch.uint8)[page, :, off] = 0x7f
            x.cache.v.view(torch.uint8)[page, :, off] = 0xff
        for t in range(n, -(-n // 16) * 16):
            page, off = int(x.table[b, t // 16]), t % 16
            x.cache.v.view(torch.uint8)[page, :, off] = 0x7f
    o2, l2 = x.run(append=False, wide=wide)
    assert torch.isfinite(out.float()).all() and torch.equal(out, o2) and torch.equal(lse, l2)
    # a NaN that is visible to one key/value head's queries stays with them
    lo = kv8_plain.visible(100, 40, 70)
    x.cache.v.view(torch.uint8)[int(x.table[0, lo // 16]), 1, lo % 16, 5] = 0x7f
    o3, _ = x.run(append=False, wide=wide)
    assert torch.isnan(o3[0, 2:, 5].float()).all()
    o3[0, 2:, 5] = out[0, 2:, 5]
    assert torch.equal(o3, out)


@pytest.mark.parametrize("wide", [0, 4096])
def test_bad_pages_and_lengths_are_recorded_and_skipped(wide):
    x = Batch([90, 40, 33], 2, 2, 64, 16, 0, seed=4)
    swa.check_device_status()
    n_pages = x.cache.k.shape[0]
    out, lse = x.run(wide=wide)
    x.append_plain()
    x.check(out, lse)
    swa.check_device_status()
    for bad in (-1, n_pages, 2 ** 31 - 1, -2 ** 31):
        was = int(x.table[0, 2])
        x.table[0, 2] = bad
        out, lse = x.run(append=False, wide=wide)
        rc, detail = swa.swa_attn_last_device_status()
        assert rc == swa.SWA_ERR_INVALID_ARG and (detail >> 8) & 0xff == 81
        x.check(out, lse, bad_pages=(bad,))
        x.table[0, 2] = was
    # the page of the new token: it is not stored, its key is not visible
    was = int(x.table[2, 2])
    x.table[2, 2] = n_pages
    before = x.cache.k.view(torch.uint8).clone()
    out, lse = x.run(wide=wide)
    assert swa.swa_attn_last_device_status()[0] == swa.SWA_ERR_INVALID_ARG
    assert torch.equal(before, x.cache.k.view(torch.uint8))
    x.check(out, lse, bad_pages=(n_pages,))
    # no page at all: nothing is visible
    x.table[2, :] = -1
    out, lse = x.run(wide=wide)
    assert swa.swa_attn_last_device_status()[0] == swa.SWA_ERR_INVALID_ARG
    assert (out[2] == 0).all() and (lse[2] == float("-inf")).all()
    # a length that the table cannot hold: an empty row
    out, lse = x.run(append=False, wide=wide, seq_len=i32([90, 40, 16 * (x.table.shape[1] + wide) + 1]))
    rc, detail = swa.swa_attn_last_device_status()
    assert rc == swa.SWA_ERR_INVALID_ARG and (detail >> 8) & 0xff == 82
    assert (out[2] == 0).all() and (lse[2] == float("-inf")).all()
    x.table[2, 2] = was
    # negative lengths are empty rows too, and nothing to record
    out, lse = x.run(append=False, wide=wide, seq_len=i32([90, -7, -2 ** 31]))
    swa.check_device_status()
    assert (out[1:] == 0).all() and (lse[1:] == float("-inf")).all()


def test_requests_may_share_pages():
    # a common prompt of two pages, own pages behind it
    x = Batch([50, 41], 2, 2, 128, 16, 0, seed=6)
    x.table[1, :2] = x.table[0, :2]
    out, lse = x.run()
    x.append_plain()
    x.check(out, lse)


def test_offsets_past_32_bits():
    # codes beyond 2^32 bytes from the start: 2 heads x 64 x 128 bytes a page
    P, Hkv, D = 64, 2, 128
    n_pages = (2 ** 32) // (P * Hkv * D) + 40
    k = torch.zeros((n_pages, Hkv, P, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.zeros_like(k.view(torch.uint8)).view(torch.float8_e4m3fn)
    ks, vs = torch.ones((n_pages, Hkv), device="cuda"), torch.ones((n_pages, Hkv), device="cuda")
    x = Batch([150], 4, Hkv, D, P, 0, seed=8)
    far = i32([[n_pages - 1, n_pages - 20, n_pages - 7]])
    near = x.table.cuda()
    out, lse = x.run()
    old = torch.cat([near[0, t // P:t // P + 1].long() * P + t % P for t in range(149)]).int()[None].contiguous()
    new = torch.cat([far[0, t // P:t // P + 1].long() * P + t % P for t in range(149)]).int()[None].contiguous()
    kh, vp = swa.kv8_read(old, *x.cache.all())
    swa.kv8_write(kh, vp, new, k, v, ks, vs)
    k2, v2 = swa.kv8_read(new, k, v, ks, vs)
    assert torch.equal(kh, k2) and torch.equal(vp, v2)
    o2, l2 = swa.decode_kv8(x.q, x.k, x.v, k, v, ks, vs, far, i32([150]))
    x.append_plain()
    x.check(o2, l2)
    swa.check_device_status()


# ------------------------------------------------------------------------------- together, as they are used

def _prompt_rows(d, T):
    """khat and v' (B, T, Hkv, D) of a layer's prompts from the forward's workspace."""
    B, _, H, D = d["q"].shape
    ws = torch.empty(swa.swa_attn_workspace_bytes(B, T, H, D, 1), dtype=torch.uint8, device="cuda")
    args = [d[n][:, :T].contiguous() for n in ("q", "k", "v")]
    out, lse = swa.forward(*args, 0, d["ve"][:, :T].contiguous(), d["gate_x"][:, :T].contiguous(), d["Wg"], workspace=ws)
    at = [swa.swa_attn_workspace_offset(B, T, H, D, 1, s) for s in (swa.SWA_WS_KHAT, swa.SWA_WS_VPRIME)]
    rows = [ws[o:o + B * T * H * D * 2].view(torch.bfloat16).view(B, T, H, D) for o in at]
    return out, lse, rows[0], rows[1]


@pytest.mark.parametrize("D,P,window", [(64, 16, 0), (128, 32, 48)])
def test_prompts_then_steps_with_requests_that_end(D, P, window):
    """Prompts through the forward, their khat and v' into pages, then decode steps in which requests end and a new one
    takes a row: every step against the plain attention over the cached values, every code against the oracle's rounded
    khat and v', and the outputs near the oracle's unquantised rows."""
    B, H, T0, steps = 3, 2, 70, 60
    Ttot = T0 + steps + 1
    s = workloads.LayerShape(B=B, T=Ttot, H=H, D=D, window=window, ve=True, seed=D, vocab=512, model_dim=64)
    host = workloads.make_layer(s)
    dev = {n: t.cuda() for n, t in workloads.gpu_side_inputs(host).items()}
    _, kh_ref, vp_ref = oracle.prologue(host, eps=float(np.float32(1e-6)), parity=True)
    q_ref = oracle.prologue(host, eps=float(np.float32(1e-6)), parity=True)[0]
    far_ref, _ = oracle.forward(host, window, parity=True)
    M, N = -(-Ttot // P), 40
    state, ring = _state(B, M, N)
    plain = kv8_plain.Pages(B, M, N, P, window)
    cache = GpuCache(N, H, P, D)
    lens = [T0, 1, T0 - 9]

    def admit(news, T):
        slots, step_len = swa.kv_pages(state[0], state[1], state[2], ring, state[3], i32(news), P, window, T)
        want = plain.step(news, T)
        assert slots.tolist() == want[0] and step_len.tolist() == want[1]
        return slots, step_len

    slots, _ = admit(lens, T0)
    _, _, kh, vp = _prompt_rows(dev, T0)
    cache.write(kh, vp, slots)
    worst = 0.0
    for step in range(steps):
        news = [1, 1, 1]
        if step == 20:
            news[2] = -1
        elif step == 21:
            news[2] = 0
        slots, step_len = admit(news, 1)
        cur = step_len.tolist()
        at = [max(0, n - 1) for n in cur]
        tok = {n: torch.stack([dev[n][b, at[b]] for b in range(B)]).contiguous() for n in ("q", "k", "v", "ve", "gate_x")}
        out, lse = swa.decode_kv8(tok["q"], tok["k"], tok["v"], *cache.all(), state[0], step_len, window, tok["ve"],
                                  tok["gate_x"], dev["Wg"])
        o, l = f64(out), f64(lse)
        for b, n in enumerate(cur):
            if n == 0:
                assert (o[b] == 0).all() and (l[b] == -np.inf).all()
                continue
            cache.write_plain(bf16(kh_ref[b, n - 1])[None, None], bf16(vp_ref[b, n - 1])[None, None], slots[b:b + 1])
            lo = kv8_plain.visible(n, window, 0)
            sl = [plain.table[b][t // P] * P + t % P for t in range(lo, n)]
            k, v = (c.values(sl) for c in cache.plain)
            ref, ref_l, mag = kv8_plain.attend(q_ref[b, n - 1], k, v)
            assert (np.abs(o[b] - ref) <= kv8_plain.out_tolerance(ref, mag)).all()
            assert (np.abs(l[b] - ref_l) <= kv8_plain.lse_tolerance(ref_l, D)).all()
            if step < 20 or b < 2:
                worst = max(worst, np.linalg.norm(o[b] - far_ref[b, n - 1]) / np.linalg.norm(far_ref[b, n - 1]))
        cache.check([x for row in slots.tolist() for x in row])
    # codes are off by at most 2^-4 of a value: a row of few keys is off by that in v', and by what the scores' errors move
    assert 0 < worst < 0.25
    swa.check_device_status()


def test_steps_in_a_captured_graph():
    """The allocator step and the decode step captured together: each replay is the next step (the state is updated in
    place), equal to eager calls; two graphs with workspaces of their own in turn."""
    B, H, D, P, N = 3, 4, 64, 16, 30
    g = torch.Generator().manual_seed(12)
    mk = lambda *sh: torch.randn(sh, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    toks = [(mk(B, H, D), mk(B, H, D), mk(B, H, D)) for _ in range(20)]

    def fresh():
        state, ring = _state(B, 8, N)
        return state, ring, GpuCache(N, H, P, D)

    state, ring, cache = fresh()
    eager = []
    one = i32([1, 1, 1])
    for q, k, v in toks:
        _, n = swa.kv_pages(state[0], state[1], state[2], ring, state[3], one, P)
        eager.append([t.clone() for t in swa.decode_kv8(q, k, v, *cache.all(), state[0], n, 0)])

    state, ring, cache = fresh()
    buf = [torch.empty_like(t) for t in toks[0]]
    graphs = []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):          # warm up outside the state
        st2, r2, c2 = fresh()
        _, n2 = swa.kv_pages(st2[0], st2[1], st2[2], r2, st2[3], one, P)
        swa.decode_kv8(*toks[0], *c2.all(), st2[0], n2, 0)
    side.synchronize()
    for _ in range(2):
        ws = torch.empty(swa.swa_attn_kv8_decode_workspace_bytes(B, H, H, D), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _, n = swa.kv_pages(state[0], state[1], state[2], ring, state[3], one, P)
            res = swa.decode_kv8(*buf, *cache.all(), state[0], n, 0, workspace=ws)
        graphs.append((graph, res))
    for i, tok in enumerate(toks):
        for d, t in zip(buf, tok):
            d.copy_(t)
        graph, res = graphs[i % 2]
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(res, eager[i])), i
    assert state[1].tolist() == [20] * 3
    swa.check_device_status()


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing that the first calls set up (launch limits, attributes, the library itself) is in the way of a capture."""
    code = """
import torch, causal_sliding_window_swa_b200 as swa
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
B, H, D, P, N = 2, 3, 64, 16, 9
table, ring = torch.full((B, 4), -1, dtype=torch.int32, device="cuda"), torch.arange(N, dtype=torch.int32, device="cuda")
kv_len, first, pool, one = i32([0] * B), i32([0] * B), i32([0, N]), i32([1] * B)
wide = torch.full((B, 4096), -1, dtype=torch.int32, device="cuda")
q, k, v = (torch.randn((B, H, D), device="cuda").to(torch.bfloat16) for _ in range(3))
cache = [torch.zeros((N, H, P, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"]
cache += [torch.ones((N, H), device="cuda") for _ in "kv"]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    slots, n = swa.kv_pages(table, kv_len, first, ring, pool, one, P)
    out, lse = swa.decode_kv8(q, k, v, *cache, table, n)
    wide[:, :4].copy_(table)
    out2, lse2 = swa.decode_kv8(q, None, None, *cache, wide, n)
    kh, vp = swa.kv8_read(slots, *cache)
    swa.kv8_write(kh, vp, slots, *cache)
for _ in range(3):
    graph.replay()
swa.check_device_status()
assert kv_len.tolist() == n.tolist() == [3, 3] and not torch.isnan(out).any()
assert (out.float() - out2.float()).abs().max() <= (2 ** -7 + 2 ** -10) * out.float().abs().max() and (lse - lse2).abs().max() < 1e-5
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]


def test_streams_and_threads():
    """Calls from four threads on streams of their own, and a call given another stream than the current one, have the
    results of a call by itself."""
    x = Batch([300, 20, 111], 4, 2, 128, 32, 0, seed=21)
    out, lse = x.run()
    torch.cuda.synchronize()
    got = [None] * 4
    go = threading.Barrier(4)

    def work(i):
        torch.cuda.set_device(0)
        st = torch.cuda.Stream()
        go.wait()
        for _ in range(5):
            with torch.cuda.stream(st):
                got[i] = x.run(append=False)
        st.synchronize()

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert all(torch.equal(o, out) and torch.equal(l, lse) for o, l in got)
    st = torch.cuda.Stream()
    for stream in (st, st.cuda_stream):
        o, l = x.run(append=False, stream=stream)
        junk = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(8)]    # what the call allocated is not taken again
        st.synchronize()
        assert torch.equal(o, out) and torch.equal(l, lse)
        del junk
    swa.check_device_status()
