"""The decode step over the paged 8-bit cache where weights and value scales span many powers of two: keys that weigh little
beside one that contributes nothing, pages whose large values lie in features of their own, pages of zeros beside pages of
very large values.  In 64 bits against the cached values, as kv8_read returns them; tolerances as in ``tests/kv8_plain.py``,
which counts an error of 2^-11 for each weight, whatever its size."""
import numpy as np
import pytest
import torch

import causal_sliding_window_swa_b200 as swa
from tests import kv8_plain

pytestmark = pytest.mark.gpu

P = 16                                    # a page for each tile of 16 keys


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield


def bf16(x):
    """64-bit values to bf16 in one rounding."""
    m, e = np.frexp(x)
    return torch.from_numpy(np.ldexp(np.rint(m * 256), e - 8)).to(torch.bfloat16)


def run(alpha, v, D, G, wide, seed=0, change=None):
    """One request of n keys, one key/value head: key j is alpha[j] times the query's direction, its values v[j] (n, D).
    The step's out (G, D) and lse (G), and those in 64 bits with the tolerances of each."""
    n = len(alpha)
    g = torch.Generator().manual_seed(seed)
    base = torch.randn((1, D), generator=g)
    q = (base + 0.02 * torch.randn((G, D), generator=g)).to(torch.bfloat16)[None].cuda()
    qh = bf16(kv8_plain.prologue(q[0].double().cpu().numpy(), n - 1)).double().numpy()
    along = qh.mean(0)
    kh = torch.from_numpy(along)[None] * torch.as_tensor(alpha, dtype=torch.float64)[:, None]
    n_pages = -(-n // P)
    order = torch.randperm(n_pages, generator=g)
    pos = torch.arange(n)
    slots = (order[pos // P] * P + pos % P).int()[None].contiguous().cuda()
    cache = [torch.full((n_pages, 1, P, D), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"]
    cache += [torch.full((n_pages, 1), float("nan"), device="cuda") for _ in "kv"]
    swa.kv8_write(kh.to(torch.bfloat16)[None, :, None].contiguous().cuda(), v.to(torch.bfloat16)[None, :, None].contiguous().cuda(),
                  slots, *cache)
    if change is not None:
        change(order, *cache)
    table = torch.full((1, n_pages + wide), -1, dtype=torch.int32)
    table[0, :n_pages] = order.int()
    out, lse = swa.decode_kv8(q, None, None, *cache, table.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"))
    k, vv = (t[0].double().cpu().numpy() for t in swa.kv8_read(slots, *cache))       # (n, 1, D)
    ref, ref_l, mag = kv8_plain.attend(qh, k, vv)
    swa.check_device_status()
    return (out[0].double().cpu().numpy(), lse[0].double().cpu().numpy(), ref, ref_l, kv8_plain.out_tolerance(ref, mag),
            kv8_plain.lse_tolerance(ref_l, D))


def check(*a, **kw):
    out, lse, ref, ref_l, tol, tol_l = run(*a, **kw)
    worst, worst_l = (np.abs(out - ref) / tol).max(), (np.abs(lse - ref_l) / tol_l).max()
    assert worst <= 1 and worst_l <= 1, (worst, worst_l)
    return ref


# One launch (a narrow table, few keys) or two; one group of eight heads, several in a warp, several sets of warps.
FORMS = [(128, 1, 0, 700), (128, 1, 8192, 700), (128, 1, 0, 16384), (64, 2, 0, 1500), (64, 8, 8192, 16384), (128, 12, 0, 3000),
         (128, 32, 0, 3000), (128, 64, 0, 2000), (64, 32, 0, 3000), (64, 64, 0, 2000)]


@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("bits", [12.0, 20.4, 25.5, 31.0])
@pytest.mark.parametrize("D,G,wide,n", FORMS)
def test_a_key_without_values_outweighs_the_others(D, G, wide, n, bits, where):
    # one key with values of zero scores `bits` powers of two above all others (rows of unit root mean square
    # score 16 above and below zero at most, 12 with 64 features): the others are all that the output consists of.  Their values are
    # positive, so that errors of their weights, all alike, do not cancel
    g = torch.Generator().manual_seed(n + G)
    top = D ** 0.5 * 1.4426950408889634                    # score of the query's direction itself, in powers of two
    alpha = torch.full((n,), 1 - bits / top)
    v = torch.rand((n, D), generator=g) + 0.5
    at = {"first": 0, "middle": n // 2 + 5, "last": n - 1}[where]
    alpha[at], v[at] = 1.0, 0.0
    ref = check(alpha, v, D, G, wide)
    assert (ref > 0).all()


@pytest.mark.parametrize("exponent", [10, 24, 33])
@pytest.mark.parametrize("page", [0, 7, -1])
@pytest.mark.parametrize("D,G,wide,n", FORMS)
def test_pages_whose_values_lie_in_other_features(D, G, wide, n, page, exponent):
    # equal scores; one page has a value of 2^exponent in one feature and zeros elsewhere, all others have nothing there
    g = torch.Generator().manual_seed(n + G + 1)
    v = torch.rand((n, D), generator=g) + 0.5
    v[:, 5] = 0.0
    at = page % (n // P) * P
    v[at:at + P] = 0.0
    v[at + 3, 5] = 2.0 ** exponent
    ref = check(torch.full((n,), 0.1), v, D, G, wide)
    assert (ref[:, [f for f in range(D) if f != 5]] > 0.4).all()


@pytest.mark.parametrize("kind", ["zeros first", "zeros last", "zeros in every second chunk", "zeros in every second page",
                                  "zeros in every second pair of chunks"])
@pytest.mark.parametrize("exponent", [60, 107])
@pytest.mark.parametrize("D,G,wide,n", [(128, 1, 0, 32), (128, 1, 8192, 32), *FORMS])
def test_pages_of_zeros_beside_pages_of_large_values(D, G, wide, n, exponent, kind):
    # equal scores; a page of zeros has the scale 2^-60, the others one up to 2^99: all keys count alike in the sum of the
    # exponentials, in whatever order, warp or block they are met
    pos = torch.arange(n)
    zero = {"zeros first": pos < n // 2 // P * P, "zeros last": pos >= n // 2 // P * P, "zeros in every second chunk": pos // 64 % 2 == 0,
            "zeros in every second page": pos // P % 2 == 0, "zeros in every second pair of chunks": pos // 128 % 2 == 0}[kind]
    g = torch.Generator().manual_seed(n + G + 2)
    v = (torch.rand((n, D), generator=g) + 0.5) * 2.0 ** exponent
    v[zero] = 0.0
    check(torch.full((n,), 0.1), v, D, G, wide)


@pytest.mark.parametrize("D,G,wide,n", FORMS)
def test_pages_whose_scale_is_zero_have_values_of_zero(D, G, wide, n):
    # no write leaves such a scale, but a cache that starts as zeros has it, and value = code * scale as in kv8_read
    g = torch.Generator().manual_seed(n + G + 3)

    def change(order, k_cache, v_cache, k_scale, v_scale):
        v_scale[order[::2]] = 0.0
        k_scale[order[::3]] = 0.0

    ref = check(torch.full((n,), 0.1), torch.rand((n, D), generator=g) + 0.5, D, G, wide, change=change)
    assert (ref > 0.4).all()
    ref = check(torch.full((n,), 0.1), torch.rand((n, D), generator=g), D, G, wide, change=lambda order, *c: c[3].zero_())
    assert (ref == 0).all()
