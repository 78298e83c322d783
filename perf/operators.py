"""The paged 8-bit key/value cache and the decode step over it: the cases that are measured, and each operator in its
plain form.

Four operators, as a server uses them one after the other:

* ``pages``: one allocator step of a paged cache for B requests.  Every request has ``kv_len`` cached tokens and asks
  for ``n_new`` more (0: idle, negative: it has ended and gives its pages back); with a window, pages that no later
  query can see go back too.  Results: the block table, the lengths, the ring of free pages and the slot of every new
  token.
* ``write``: khat and v' rows (bf16) go into e4m3 pages with a power-of-two scale for each page and head, and are then
  read back, as when a request is moved.
* ``read``: rows of the cache as bf16.
* ``decode``: one new token for each request: RoPE, RMS QK-norm, the gated value embedding, the token's khat and v'
  into the cache (unless it is there already), and attention over the cached keys in the window.

The sizes are those of this repository's workloads (12 heads of 64 or 128, T = 1024 and 2048, windows of 1024 and 2048,
sequences up to 16384) and generic ones around them.
"""
import math
import random

import torch

own = False

EPS = 1e-6
ROPE_BASE = 10000.0
E_MIN = -60            # the smallest scale is 2^-60
CODE_MAX = 448.0       # the largest e4m3 value


# ------------------------------------------------------------------------------------------ cases

def listed():
    d = dict(op="decode", ve=False, append=True, doc=False)
    w = dict(op="write")
    r = dict(op="read")
    p = dict(op="pages")
    return [
        # the allocator: a decode step of a small batch; prompts that come in together; a crowded server in which
        # requests end, windows slide past pages and the last requests find no page
        dict(p, name="pages step 16", B=16, T=1, P=64, window=0, len=2048, tight=False, mix=1),
        dict(p, name="pages prompts 64x2048", B=64, T=2048, P=64, window=0, len=0, tight=False, mix=2),
        dict(p, name="pages crowded 1000", B=1000, T=1, P=16, window=1024, len=4096, tight=True, mix=3),
        # the prompts of the d24 layer; one token each for odd requests of a grouped-query layer with 64 features
        dict(w, name="write d24 prompts", B=16, T=2048, H=12, D=128, P=64, len=0, mix=4),
        dict(w, name="write tokens 33", B=33, T=1, H=4, D=64, P=16, len=1000, mix=5),
        # a batch of d24 requests taken out of the cache; ragged short ones
        dict(r, name="read d24", B=16, T=2048, H=12, D=128, P=64, len=2048, mix=6),
        dict(r, name="read ragged 7", B=7, T=333, H=6, D=64, P=32, len=333, mix=7),
        # one request of the GPT-2 124M layer whose token is in the cache already: latency
        dict(d, name="decode one", B=1, H=12, Hkv=12, D=64, P=16, window=0, len=301, append=False, mix=8),
        # the d24 layers: the short window with ragged lengths, the full window with value embeddings
        dict(d, name="decode d24 S", B=16, H=12, Hkv=12, D=128, P=64, window=1024, len=2048, mix=9),
        dict(d, name="decode d24 L VE", B=32, H=12, Hkv=12, D=128, P=64, window=2048, len=4096, ve=True, mix=10),
        # grouped queries, 8 heads to a key/value head, packed documents
        dict(d, name="decode grouped", B=48, H=16, Hkv=2, D=128, P=32, window=0, len=8192, doc=True, mix=11),
        # the longest sequences of the SSSL stack, many requests
        dict(d, name="decode 16384", B=32, H=12, Hkv=12, D=128, P=128, window=0, len=16384, append=False, mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["pages", "write", "read", "decode", "decode"])
    P = rng.choice([16, 32, 64, 128])
    mix = rng.randrange(1 << 20)
    if op == "pages":
        T = rng.choice([1, 1, _log(rng, 1, 2048)])
        return dict(op=op, B=_log(rng, 1, 1000), T=T, P=P, window=rng.choice([0, _log(rng, 1, 4096)]),
                    len=_log(rng, 1, 4096) if T == 1 else rng.choice([0, _log(rng, 1, 2048)]), tight=rng.random() < 0.4,
                    mix=mix)
    D = rng.choice([64, 128])
    Hkv, G = rng.choice([(1, 1), (1, 32), (2, 8), (3, 2), (4, 1), (4, 3), (5, 5), (8, 4), (12, 1)])
    most = 32 * 16384 * 12 // 4
    if op in ("write", "read"):
        T = rng.choice([1, _log(rng, 1, 2048)])
        B = max(1, min(_log(rng, 1, 256), 400000 // (T * Hkv)))
        return dict(op=op, B=B, T=T, H=Hkv, D=D, P=P, len=rng.choice([0, _log(rng, 1, 2048)]) if op == "write" else max(1, T),
                    mix=mix)
    length = _log(rng, 1, 16384)
    B = max(1, min(_log(rng, 1, 256), most // (length * Hkv)))
    return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, D=D, P=P, window=rng.choice([0, 1024, _log(rng, 1, 16384)]), len=length,
                ve=rng.random() < 0.4, append=rng.random() < 0.6, doc=rng.random() < 0.3, mix=mix)


# ----------------------------------------------------------------------------- lengths of a case

def _lens(case):
    """Tokens in the cache of each request (the new one of a decode step among them): mostly long ones, some short,
    with an empty row now and then.  Written from the case alone, so that the work is known."""
    r = random.Random(case["mix"])
    top = case["len"]
    if case["op"] == "decode":
        if case["B"] == 1:
            return [top]
        return [top] + [0 if r.random() < 0.03 else max(1, int(top * (1.0 - 0.75 * r.random() ** 2)))
                        for _ in range(case["B"] - 1)]
    if case["op"] == "read":
        return [top] + [r.randint(top // 2, top) for _ in range(case["B"] - 1)]
    return [r.randint(top // 2, top) for _ in range(case["B"])]


def _news(case):
    """New tokens of each request."""
    r = random.Random(case["mix"] + 1)
    B, T = case["B"], case["T"]
    if case["op"] == "write":
        return [T] + [T if T == 1 else r.randint(max(1, T // 2), T) for _ in range(B - 1)]
    if T == 1:
        return [1] + [-1 if u < 0.03 else 0 if u < 0.06 else 1 for u in (r.random() for _ in range(B - 1))]
    return [T] + [0 if r.random() < 0.05 else r.randint(max(1, T // 8), T) for _ in range(B - 1)]


def _first(length, window):
    return max(0, length - window) if window > 0 else 0


def _starts(case, lens):
    """First position of each request's document."""
    r = random.Random(case["mix"] + 2)
    return [int(n * 0.5 * r.random() ** 3) if n > 0 else 0 for n in lens]


# ----------------------------------------------------------------------------------------- inputs

def _table(held_from, held_to, width, perm):
    """A block table whose row b holds pages for entries [held_from, held_to), taken in turn from perm."""
    a = torch.tensor(held_from, device="cuda")[:, None]
    z = torch.tensor(held_to, device="cuda")[:, None]
    n = (z - a).clamp_min(0)
    j = torch.arange(width, device="cuda")[None]
    at = (torch.cumsum(n, 0) - n + j - a).clamp(0, perm.numel() - 1)
    return torch.where((j >= a) & (j < z), perm[at], -1).to(torch.int32).contiguous()


def _cache(n_pages, H, P, D, gen):
    """Pages of khat (rows of unit root mean square) and v' (normal) as they are kept: codes and scales."""
    out = []
    for which in (0, 1):
        codes = torch.empty((n_pages, H, P, D), dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.empty((n_pages, H), dtype=torch.float32, device="cuda")
        step = max(1, (1 << 26) // (H * P * D))
        for i in range(0, n_pages, step):
            x = torch.randn((min(step, n_pages - i), H, P, D), generator=gen, device="cuda")
            if which == 0:
                x = x * torch.rsqrt(x.square().mean(-1, keepdim=True))
            else:
                x = x * torch.exp2(torch.randint(-2, 3, (x.shape[0], H, 1, 1), generator=gen, device="cuda").float())
            amax = x.to(torch.bfloat16).float().abs().amax((-1, -2))
            s = torch.exp2(_exponent(amax).float())
            codes[i:i + step] = (x.to(torch.bfloat16).float() / s[:, :, None, None]).to(torch.float8_e4m3fn)
            scale[i:i + step] = s
        out += [codes, scale]
    return out[0], out[2], out[1], out[3]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case}
    lens, B, P = _lens(case), case["B"], case["P"]
    cdiv = lambda a: -(-a // P)  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] == "pages":
        news, W = _news(case), case["window"]
        first = [_first(n, W) // P for n in lens]
        held = sum(max(0, cdiv(n) - f) for n, f in zip(lens, first))
        need = sum(max(0, cdiv(n + max(0, m)) - cdiv(n)) for n, m in zip(lens, news))
        free = need * 2 // 3 if case["tight"] else need + 5
        n_pages = held + free + 3
        perm = torch.randperm(n_pages, generator=gen, device="cuda")
        width = max(1, cdiv(case["len"] + case["T"]))
        head = seed % n_pages
        s["ring"] = torch.roll(perm, head - held).to(torch.int32).contiguous()
        s["pool"] = i32([head, free])
        s["table"] = _table(first, [cdiv(n) for n in lens], width, perm)
        s["kv_len"], s["first"], s["n_new"] = i32(lens), i32(first), i32(news)
        s["to"] = tuple(torch.empty_like(s[k]) for k in ("table", "kv_len", "first", "pool"))
        s["slots"] = torch.empty((B, case["T"]), dtype=torch.int32, device="cuda")
        s["step_len"] = torch.empty((B,), dtype=torch.int32, device="cuda")
        return s
    D, T = case["D"], case.get("T", 1)
    H = case["Hkv"] if case["op"] == "decode" else case["H"]
    news = _news(case) if case["op"] == "write" else [0] * B
    W = case.get("window", 0)
    first = [_first(n, W) // P for n in lens]
    last = [cdiv(n + m) for n, m in zip(lens, news)]
    n_pages = sum(max(0, z - a) for a, z in zip(first, last)) + 2      # the last page is never used
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _cache(n_pages, H, P, D, gen)
    s["table"] = _table(first, last, max(1, max(last)), torch.randperm(n_pages - 1, generator=gen, device="cuda"))
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    if case["op"] != "decode":
        def slots(start, count, width):
            t = torch.arange(width, device="cuda")[None]
            pos = torch.tensor(start, device="cuda")[:, None] + t
            page = s["table"].long().gather(1, (pos // P).clamp_max(s["table"].shape[1] - 1))
            return torch.where(t < torch.tensor(count, device="cuda")[:, None], page * P + pos % P, -1).to(torch.int32)
        if case["op"] == "read":
            s["rows"] = slots([0] * B, lens, T).contiguous()
            return s
        kh = normal(B, T, H, D)
        s["kh"] = (kh * torch.rsqrt(kh.square().mean(-1, keepdim=True))).to(torch.bfloat16)
        s["vp"] = (normal(B, T, H, D) * torch.exp(0.5 * normal(B, T, H, 1))).to(torch.bfloat16)
        s["slots"] = slots(lens, news, T).contiguous()
        from_page = [n // P * P for n in lens]
        whole = [n + m - a for n, m, a in zip(lens, news, from_page)]
        s["rows"] = slots(from_page, whole, max(whole)).contiguous()
        return s
    bf = lambda *shape: normal(*shape).to(torch.bfloat16)  # noqa: E731
    s["q"], s["seq_len"] = bf(B, case["H"], D), i32(lens)
    s["k"], s["v"] = (bf(B, H, D), bf(B, H, D)) if case["append"] else (None, None)
    ve = case["ve"] and case["append"]
    s["ve"], s["gate_x"], s["Wg"] = (bf(B, H, D), bf(B, 32), (0.02 * normal(32, H)).to(torch.bfloat16)) if ve else (None,) * 3
    s["start"] = i32(_starts(case, lens)) if case["doc"] else None
    tail = [max(0, n - 1) // P * P for n in lens]
    if case["append"]:   # the rows of the pages that take the new tokens
        t = torch.arange(P, device="cuda")[None]
        pos = torch.tensor(tail, device="cuda")[:, None] + t
        page = s["table"].long().gather(1, (pos // P).clamp_max(s["table"].shape[1] - 1))
        s["rows"] = torch.where(pos < s["seq_len"][:, None], page * P + pos % P, -1).to(torch.int32).contiguous()
    return s


# ------------------------------------------------------------------------------------ plain forms

def _exponent(amax):
    """The smallest integer e >= E_MIN with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax.float() / CODE_MAX)
    return torch.where(m == 0.5, e - 1, e).clamp(E_MIN, 120).where(amax > 0, E_MIN)


def _fp8(x):
    return x.to(torch.float8_e4m3fn)


def _pages(s):
    case = s["case"]
    P, W, T = case["P"], case["window"], case["T"]
    L, n, F, table, ring = (s[k].long() for k in ("kv_len", "n_new", "first", "table", "ring"))
    head, free = s["pool"].long()[0], s["pool"].long()[1]
    N, M = ring.numel(), table.shape[1]
    have = (L + P - 1) // P
    ended = n < 0
    low = (L - W + 1).clamp_min(0) // P if W > 0 else torch.zeros_like(L)
    upto = torch.where(ended, have, torch.maximum(F, low))
    fits = (n >= 0) & (n <= T) & ((L + n + P - 1) // P <= M)
    need = torch.where(fits, (L + n + P - 1) // P - have, 0)
    S = torch.cumsum(need, 0)
    ok = fits & (n > 0) & ((need == 0) | (S <= free))
    take = torch.where(ok, need, 0)
    j = torch.arange(M, device="cuda")[None]
    fresh = ring[(head + (S - need)[:, None] + j - have[:, None]) % N]
    gone = (j >= F[:, None]) & (j < upto[:, None])
    out = torch.where((j >= have[:, None]) & (j < (have + take)[:, None]), fresh, torch.where(gone, -1, table))
    given = (upto - F).clamp_min(0)
    at = (head + free + (torch.cumsum(given, 0) - given)[:, None] + j - F[:, None]) % N
    ring = torch.cat([ring, ring[:1]]).scatter(0, torch.where(gone, at, N).reshape(-1), table.reshape(-1))[:N]
    taken = take.sum()
    pool = torch.stack([(head + taken) % N, free - taken + given.sum()])
    after = torch.where(ended, 0, torch.where(ok, L + n, L))
    pos = L[:, None] + torch.arange(T, device="cuda")[None]
    page = out.gather(1, (pos // P).clamp_max(M - 1))
    slots = torch.where(ok[:, None] & (pos < after[:, None]), page * P + pos % P, -1)
    answer = (out, after, torch.where(ended, 0, torch.maximum(F, upto)), pool, ring, slots, torch.where(ok, after, 0))
    return [t.to(torch.int32) for t in answer]


def _read(slots, P, k_cache, v_cache, k_scale, v_scale):
    sl = slots.long().clamp_min(0)
    page, off = sl // P, sl % P
    got = []
    for codes, scale in ((k_cache, k_scale), (v_cache, v_scale)):
        x = codes.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).float() * scale[page][..., None]
        got.append(torch.where((slots >= 0)[..., None, None], x, 0.0).to(torch.bfloat16))
    return got


def _store(x, slots, P, codes, scale):
    """Rows x (tokens, heads, features) into their slots; rows with a negative slot go to the last page, which is unused."""
    n_pages = codes.shape[0]
    sl = torch.where(slots < 0, (n_pages - 1) * P, slots.long())
    page, off = sl // P, sl % P
    e = _exponent(x.float().abs().amax(-1))
    want = torch.full(scale.shape, E_MIN - 1, device="cuda").scatter_reduce(0, page[:, None].expand_as(e), e.long(), "amax")
    fresh = torch.zeros(n_pages, dtype=torch.int32, device="cuda").index_put((page,), (off == 0).int(), accumulate=True)[:, None] > 0
    old = torch.log2(scale).round().long()
    new = torch.where(want < E_MIN, old, torch.where(fresh, want, torch.maximum(want, old)))
    old = torch.where(fresh, new, old)
    codes.copy_(_fp8(codes.float() * torch.exp2((old - new).float())[:, :, None, None]))
    scale.copy_(torch.exp2(new.float()))
    q = _fp8(x.float() / scale[page][..., None])
    heads = torch.arange(x.shape[1], device="cuda")[None]
    codes.view(torch.uint8).index_put_((page[:, None], heads, off[:, None]), q.view(torch.uint8))


def _bf16(x):
    """64-bit values to bf16 in one rounding (a cast by way of 32 bits may round twice)."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256.0), e - 8).to(torch.bfloat16)


def _rotate(x, pos):
    """RMS(RoPE(x)) of rows x (B, heads, D) at positions pos (B,), in 64 bits, rounded to bf16."""
    D = x.shape[-1]
    theta = ROPE_BASE ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device="cuda") / D)
    ang = (pos.double()[:, None] * theta)[:, None]
    a, b = x[..., :D // 2].double(), x[..., D // 2:].double()
    y = torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1)
    return _bf16(y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS))


def _decode(s):
    case = s["case"]
    B, H, Hkv, D, P = case["B"], case["H"], case["Hkv"], case["D"], case["P"]
    kc, vc, ks, vs = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    table, n = s["table"].long(), s["seq_len"].long()
    dummy = kc.shape[0] - 1
    pos = (n - 1).clamp_min(0)
    lens = _lens(case)
    if s["k"] is not None:
        kh = _rotate(s["k"], pos)
        vp = s["v"]
        if s["ve"] is not None:
            g = 2.0 * torch.sigmoid((s["gate_x"].double()[:, :, None] * s["Wg"].double()[None]).sum(1))
            vp = _bf16(vp.double() + g[..., None] * s["ve"].double())
        page = torch.where(n > 0, table.gather(1, (pos // P)[:, None])[:, 0], dummy)
        off = pos % P
        heads = torch.arange(Hkv, device="cuda")[None]
        row = torch.arange(P, device="cuda")[None, None, :, None]
        at = off[:, None, None, None]
        for x, codes, scale in ((kh, kc, ks), (vp, vc, vs)):
            old = torch.log2(scale[page]).round().long()
            tok = _exponent(x.float().abs().amax(-1)).long()
            new = torch.where(off[:, None] == 0, tok, torch.maximum(old, tok))
            held = codes.view(torch.uint8)[page].view(torch.float8_e4m3fn).float()
            moved = held * torch.exp2((old - new).float())[..., None, None]
            fresh = x.float()[:, :, None] / torch.exp2(new.float())[..., None, None]
            both = _fp8(torch.where(row < at, moved, torch.where(row == at, fresh, held)))
            codes.view(torch.uint8).index_put_((page[:, None], heads), both.view(torch.uint8))
            scale.index_put_((page[:, None], heads), torch.exp2(new.float()))
    q = _rotate(s["q"], pos).float().view(B, Hkv, H // Hkv, D)
    lo = (n - case["window"]).clamp_min(0) if case["window"] > 0 else torch.zeros_like(n)
    if s["start"] is not None:
        lo = torch.maximum(lo, torch.minimum(s["start"].long(), pos))
    width = max(1, max(m - _first(m, case["window"]) for m in lens))
    at = lo[:, None] + torch.arange(width, device="cuda")[None]
    seen = at < n[:, None]
    at = torch.where(seen, at, pos[:, None])
    page = torch.where(n[:, None] > 0, table.gather(1, at // P), dummy)
    off = at % P
    k = kc.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).float().mul_(ks[page][..., None])
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(D)
    del k
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = vc.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).float().mul_(vs[page][..., None])
    out = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0].masked_fill(n[:, None, None] <= 0, -math.inf)
    return out.reshape(B, H, D).to(torch.bfloat16), lse.reshape(B, H)


def run(s):
    case = s["case"]
    op, P = case["op"], case["P"]
    if own:
        import causal_sliding_window_swa_b200 as swa
        if op == "pages":
            slots, step_len = swa.kv_pages(s["table"], s["kv_len"], s["first"], s["ring"], s["pool"], s["n_new"], P,
                                           case["window"], out=s["to"], slots=s["slots"], step_len=s["step_len"])
            return [*s["to"], s["ring"], slots, step_len]
        cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if op == "read":
            return swa.kv8_read(s["rows"], *cache)
        if op == "write":
            swa.kv8_write(s["kh"], s["vp"], s["slots"], *cache)
            return swa.kv8_read(s["rows"], *cache)
        got = swa.decode_kv8(s["q"], s["k"], s["v"], *cache, s["table"], s["seq_len"], case["window"], s["ve"], s["gate_x"],
                             s["Wg"], ROPE_BASE, EPS, doc_start=s["start"])
        return [*got, *swa.kv8_read(s["rows"], *cache)] if case["append"] else list(got)
    if op == "pages":
        return _pages(s)
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if op == "read":
        return _read(s["rows"], P, *cache)
    if op == "write":
        sl = s["slots"].reshape(-1)
        _store(s["kh"].flatten(0, 1), sl, P, s["k_cache"], s["k_scale"])
        _store(s["vp"].flatten(0, 1), sl, P, s["v_cache"], s["v_scale"])
        return _read(s["rows"], P, *cache)
    got = _decode(s)
    return [*got, *_read(s["rows"], P, *cache)] if case["append"] else list(got)


# ------------------------------------------------------------------------------------------- work

def work(case):
    lens, P = _lens(case), case["P"]
    if case["op"] == "pages":
        news = _news(case)
        B, T, W = case["B"], case["T"], case["window"]
        width = max(1, -(-(case["len"] + T) // P))
        # lengths, first pages, new tokens in; lengths, first pages, step lengths out; both tables; the slots; what moves
        # through the ring (each entry once)
        moved = sum(-(-(n + max(0, m)) // P) - -(-n // P) for n, m in zip(lens, news))
        if W == 0:
            moved += sum(-(-n // P) for n, m in zip(lens, news) if m < 0)
        return {"bytes": 4.0 * (6 * B + 2 * B * width + B * T + moved), "flops": 8.0 * B}
    D = case["D"]
    if case["op"] == "read":
        n = sum(lens) * case["H"] * D * 2
        return {"bytes": 3.0 * n + 4.0 * case["B"] * case["T"], "flops": float(n)}
    if case["op"] == "write":
        news = _news(case)
        n = sum(news) * case["H"] * D * 2
        back = sum(a % P + m for a, m in zip(lens, news)) * case["H"] * D * 2
        return {"bytes": 3.0 * n + 3.0 * back, "flops": 3.0 * n + back}
    B, H, Hkv = case["B"], case["H"], case["Hkv"]
    starts = _starts(case, lens) if case["doc"] else [0] * B
    keys = sum(n - max(_first(n, case["window"]), min(a, n - 1) if n else 0) for n, a in zip(lens, starts))
    small = B * (2 * H * D * 2 + 4 * H)
    if case["append"]:
        small += B * Hkv * D * 2 * (2 + 1 + (1 if case["ve"] else 0))
        small += sum((n - 1) % P + 1 for n in lens if n > 0) * Hkv * D * 2 * 3
    return {"bytes": keys * Hkv * 2.0 * D + small, "flops": 4.0 * D * H * keys}


# ---------------------------------------------------------------------------- the definition in 64 bits

def _nearest(x):
    """e4m3 of 64-bit values: four significant bits, ties to even, 2^-9 the smallest step, at most 448."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -30))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(x / step) * step).clamp(-CODE_MAX, CODE_MAX)


def _eight(x):
    """64-bit values with eight significant bits, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(1e-30))) - 7.0)
    return torch.round(x / step) * step


def _fit(amax):
    """The exponent of the smallest power of two that brings amax within 448, one element at a time."""
    def one(a):
        if not a > 0:
            return E_MIN
        e = math.ceil(math.log2(a / CODE_MAX))
        e += 1 if a > CODE_MAX * 2.0 ** e else -1 if a <= CODE_MAX * 2.0 ** (e - 1) else 0
        return max(e, E_MIN)
    return torch.tensor([one(a) for a in amax.reshape(-1).tolist()], dtype=torch.float64, device=amax.device).view(amax.shape)


def _held(s, which, page, upto):
    """The first `upto` rows of a page, all heads, as values (64 bits)."""
    return s[which + "_cache"][page, :, :upto].double() * s[which + "_scale"][page].double()[:, None, None]


def _append(s, which, page, off, rows):
    """The values of a page's rows [0, off + n) after rows (n, heads, D) are appended at `off`."""
    want = _fit(rows.double().abs().amax((0, 2)))
    if off > 0:
        old = s[which + "_scale"][page].double()
        want = torch.maximum(want, torch.log2(old).round())
    scale = torch.exp2(want)[:, None, None]
    new = _nearest(rows.double().transpose(0, 1) / scale) * scale
    if off == 0:
        return new
    return torch.cat([_nearest(_held(s, which, page, off) / scale) * scale, new], 1)


def _turned(x, pos):
    """RMS(RoPE(x)) of rows (heads, D) at one position, as a rotation of complex numbers."""
    D = x.shape[-1]
    w = torch.tensor([pos * ROPE_BASE ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64, device="cuda")
    z = torch.complex(x[:, :D // 2].double(), x[:, D // 2:].double()) * torch.polar(torch.ones_like(w), w)
    y = torch.cat([z.real, z.imag], 1)
    return _eight(y * (y.square().mean(1, keepdim=True) + EPS) ** -0.5)


def exact(case, seed):
    """What run() returns, request by request, from the definition."""
    if case["op"] == "pages":
        return None           # whole numbers
    s = prepare(case, seed)
    P, lens = case["P"], _lens(case)
    table = s["table"].tolist()
    if case["op"] == "read":
        B, T = s["rows"].shape
        got = {}
        for which in "kv":
            x = torch.zeros((B, T, case["H"], case["D"]), dtype=torch.float64, device="cuda")
            for b, n in enumerate(lens):
                for j in range(0, n, P):
                    m = min(P, n - j)
                    x[b, j:j + m] = _held(s, which, table[b][j // P], m).transpose(0, 1)
            got[which] = x
        return [got["k"], got["v"]]
    if case["op"] == "write":
        if sum(_news(case)) * case["H"] > 500000:
            return None       # page by page it takes too long
        back = []
        for which, rows in (("k", s["kh"]), ("v", s["vp"])):
            x = torch.zeros((*s["rows"].shape, case["H"], case["D"]), dtype=torch.float64, device="cuda")
            for b, (n, m) in enumerate(zip(lens, _news(case))):
                base = n // P * P
                at = n
                while at < n + m:
                    k = min(P - at % P, n + m - at)
                    now = _append(s, which, table[b][at // P], at % P, rows[b, at - n:at - n + k])
                    x[b, at // P * P - base:at // P * P - base + now.shape[1]] = now.transpose(0, 1)
                    at += k
            back.append(x)
        return back
    H, Hkv, D, W = case["H"], case["Hkv"], case["D"], case["window"]
    starts = _starts(case, lens) if case["doc"] else [0] * case["B"]
    out = torch.zeros((case["B"], H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], H), -math.inf, dtype=torch.float64, device="cuda")
    kept = [torch.zeros((case["B"], P, Hkv, D), dtype=torch.float64, device="cuda") for _ in "kv"]
    for b, n in enumerate(lens):
        if n == 0:
            continue
        lo = max(_first(n, W), min(starts[b], n - 1))
        pages = torch.tensor(table[b][lo // P:(n - 1) // P + 1], device="cuda")
        whole = {}
        for which in "kv":
            codes = s[which + "_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn)
            whole[which] = (codes.double() * s[which + "_scale"][pages].double()[:, :, None, None]).transpose(0, 1).flatten(1, 2)
        last = (n - 1) // P * P - lo // P * P      # where the last page's rows begin
        if s["k"] is not None:
            vp = s["v"][b].double()
            if s["ve"] is not None:
                z = s["gate_x"][b].double() @ s["Wg"].double()
                vp = _eight(vp + (2.0 / (1.0 + torch.exp(-z)))[:, None] * s["ve"][b].double())
            for i, (which, row) in enumerate((("k", _turned(s["k"][b], n - 1)), ("v", vp))):
                now = _append(s, which, table[b][(n - 1) // P], (n - 1) % P, row[None])
                whole[which][:, last:last + now.shape[1]] = now
                kept[i][b, :now.shape[1]] = now.transpose(0, 1)
        k, v = (whole[c][:, lo % P:n - lo // P * P] for c in "kv")
        q = _turned(s["q"][b], n - 1).view(Hkv, H // Hkv, D)
        x = torch.einsum("hgd,hnd->hgn", q, k) / math.sqrt(D)
        lse[b] = torch.logsumexp(x, -1).reshape(H)
        out[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), v).reshape(H, D)
    return [out, lse, *kept] if case["append"] else [out, lse]
