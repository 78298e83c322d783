"""The paged 8-bit cache without a GPU: the plain statements the GPU results are compared with are pinned, and every
entry point refuses bad arguments before it touches the device (the fake addresses are never used)."""
import random

import numpy as np
import pytest
import torch

import causal_sliding_window_swa_b200 as swa
from tests import kv8_plain

A = 0x7f0000000000


# ------------------------------------------------------------------------------- the plain statements

def test_plain_codes_match_torch():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(kv8_plain.TABLE, codes)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * s for s in (1e-3, 1e-2, 1.0, 30.0, 100.0)])
    mags = kv8_plain.TABLE[:127]
    mid = (mags[1:] + mags[:-1]) / 2                       # every tie
    x = np.concatenate([x, mid, -mid, mags, -mags])
    x = x[np.abs(x) <= 448].astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(kv8_plain.e4m3(x), want)
    assert kv8_plain.e4m3(1e9) == 448 and kv8_plain.e4m3(-np.inf) == -448 and np.isnan(kv8_plain.e4m3(np.nan))


def test_plain_exponent_is_the_smallest_that_fits():
    for top, want in ((448.0, 0), (448.5, 1), (224.0, -1), (7.0, -6), (7.0625, -5), (11.3, -5), (0.0, -60), (1e-30, -60),
                      (np.inf, 120)):
        assert kv8_plain.exponent(np.array([0.0, -top, np.nan])) == want


@pytest.mark.parametrize("P", [16, 64])
def test_a_page_filled_token_by_token_is_one_write_up_to_tiny_values(P):
    # the scale grows with the page; codes above 2^-6 move exactly, smaller ones are rounded again (each time by at
    # most half of 2^-9, the next scale being at least twice as large: together below 2^-9)
    rng = np.random.default_rng(P)
    x = rng.standard_normal((P, 2, 64)) * np.exp(rng.standard_normal((P, 1, 1)))
    one, many = kv8_plain.Cache(2, 2, P, 64), kv8_plain.Cache(2, 2, P, 64)
    slots = np.arange(P) + P
    one.write(x, slots)
    for t in range(P):
        many.write(x[t:t + 1], slots[t:t + 1])
    np.testing.assert_array_equal(one.e, many.e)
    big = np.abs(one.codes) >= 2.0 ** -5
    np.testing.assert_array_equal(one.codes[big], many.codes[big])
    assert np.abs(one.codes - many.codes).max() <= 2.0 ** -8
    # and a cached value is within half a step of what was written
    err = np.abs(one.values(slots) - x)
    assert (err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * 2.0 ** one.e[1].astype(float)[None, :, None])).all()


def test_plain_allocator_keeps_every_page_once():
    r = random.Random(3)
    B, M, N, P, W = 9, 12, 60, 16, 70
    a = kv8_plain.Pages(B, M, N, P, W)
    served = 0
    for step in range(300):
        T = r.choice([1, 1, 1, 50])
        news = [-1 if r.random() < 0.05 else r.randint(0, T) for _ in range(B)]
        before = list(a.kv_len)
        slots, step_len = a.step(news, T)
        held = [p for row in a.table for p in row if p >= 0]
        free = [a.ring[(a.head + i) % N] for i in range(a.free)]
        assert sorted(held + free) == list(range(N))
        for b in range(B):
            have = -(-a.kv_len[b] // P)
            assert all((a.table[b][j] >= 0) == (a.first[b] <= j < have) for j in range(M))
            got = [s for s in slots[b] if s >= 0]
            assert len(got) == (news[b] if step_len[b] else 0)
            assert a.kv_len[b] == (0 if news[b] < 0 else before[b] + len(got))
            # every key that a query from now on can see is still there
            assert a.first[b] * P <= max(0, before[b] - W + 1)
            served += step_len[b] > 0
    assert served > 500


# ------------------------------------------------------------------------------------------- refusals

def _pages(**kw):
    a = dict(block_table=A, kv_len=A, first_page=A, pool=A, n_new=A, ring=A, block_table_out=A, kv_len_out=A,
             first_page_out=A, pool_out=A, slots=A, step_len=A, B=2, T=1, max_pages=8, n_pages=16, page_size=16, window=0,
             stream=None)
    a.update(kw)
    return swa.swa_attn_kv_pages(*a.values())


@pytest.mark.parametrize("name", ["block_table", "kv_len", "first_page", "pool", "n_new", "ring", "block_table_out",
                                  "kv_len_out", "first_page_out", "pool_out", "slots", "step_len"])
def test_pages_refuses_null_and_misaligned_arrays(name):
    assert _pages(**{name: None}) == swa.SWA_ERR_INVALID_ARG
    assert _pages(**{name: A + 2}) == swa.SWA_ERR_MISALIGNED


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), swa.SWA_ERR_INVALID_ARG), (dict(T=0), swa.SWA_ERR_INVALID_ARG),
    (dict(max_pages=0), swa.SWA_ERR_INVALID_ARG), (dict(n_pages=0), swa.SWA_ERR_INVALID_ARG),
    (dict(page_size=0), swa.SWA_ERR_UNSUPPORTED), (dict(page_size=8), swa.SWA_ERR_UNSUPPORTED),
    (dict(page_size=48), swa.SWA_ERR_UNSUPPORTED), (dict(page_size=256), swa.SWA_ERR_UNSUPPORTED),
    (dict(n_pages=1 << 27), swa.SWA_ERR_UNSUPPORTED), (dict(max_pages=1 << 27), swa.SWA_ERR_UNSUPPORTED),
    (dict(B=1 << 20, T=1 << 11), swa.SWA_ERR_UNSUPPORTED), (dict(B=1 << 20, max_pages=1 << 11), swa.SWA_ERR_UNSUPPORTED),
])
def test_pages_refuses_bad_sizes(kw, code):
    assert _pages(**kw) == code


def _rows(fn, **kw):
    a = dict(kh=A, vp=A, slots=A, k_cache=A, v_cache=A, k_scale=A, v_scale=A, B=2, T=3, Hkv=2, D=64, n_pages=16,
             page_size=16, stream=None)
    a.update(kw)
    if fn == "read":
        order = ["slots", "k_cache", "v_cache", "k_scale", "v_scale", "kh", "vp"]
        return swa.swa_attn_kv8_read(*[a[k] for k in order], *list(a.values())[7:])
    return swa.swa_attn_kv8_write(*a.values())


@pytest.mark.parametrize("fn", ["write", "read"])
@pytest.mark.parametrize("kw,code", [
    *[({n: None}, swa.SWA_ERR_INVALID_ARG) for n in ("kh", "vp", "slots", "k_cache", "v_cache", "k_scale", "v_scale")],
    *[({n: A + 8}, swa.SWA_ERR_MISALIGNED) for n in ("kh", "vp", "k_cache", "v_cache")],
    *[({n: A + 2}, swa.SWA_ERR_MISALIGNED) for n in ("slots", "k_scale", "v_scale")],
    (dict(B=0), swa.SWA_ERR_INVALID_ARG), (dict(T=0), swa.SWA_ERR_INVALID_ARG), (dict(Hkv=0), swa.SWA_ERR_INVALID_ARG),
    (dict(D=96), swa.SWA_ERR_UNSUPPORTED), (dict(page_size=24), swa.SWA_ERR_UNSUPPORTED),
    (dict(n_pages=0), swa.SWA_ERR_INVALID_ARG), (dict(n_pages=1 << 26), swa.SWA_ERR_UNSUPPORTED),
    (dict(Hkv=65536), swa.SWA_ERR_UNSUPPORTED), (dict(B=1 << 16, T=1 << 15), swa.SWA_ERR_UNSUPPORTED),
])
def test_write_and_read_refuse_bad_arguments(fn, kw, code):
    assert _rows(fn, **kw) == code


def _decode(**kw):
    a = dict(q=A, k=A, v=A, ve=None, gate_x=None, Wg=None, k_cache=A, v_cache=A, k_scale=A, v_scale=A, block_table=A,
             seq_len=A, doc_start=None, out=A, lse=A, B=2, H=4, Hkv=2, D=64, n_pages=16, page_size=16, max_pages=8,
             window=0, rope_base=1e4, eps=1e-6, workspace=A, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return swa.swa_attn_kv8_decode(*a.values())


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, swa.SWA_ERR_INVALID_ARG) for n in ("q", "k", "v", "k_cache", "v_cache", "k_scale", "v_scale",
                                                     "block_table", "seq_len", "out", "workspace")],
    *[({n: A + 8}, swa.SWA_ERR_MISALIGNED) for n in ("q", "k", "v", "k_cache", "v_cache", "out", "workspace")],
    *[({n: A + 2}, swa.SWA_ERR_MISALIGNED) for n in ("k_scale", "v_scale", "block_table", "seq_len", "doc_start", "lse")],
    (dict(ve=A), swa.SWA_ERR_INVALID_ARG), (dict(ve=A, gate_x=A), swa.SWA_ERR_INVALID_ARG),
    (dict(k=None, v=None, ve=A, gate_x=A, Wg=A), swa.SWA_ERR_INVALID_ARG),
    (dict(B=0), swa.SWA_ERR_INVALID_ARG), (dict(H=3), swa.SWA_ERR_INVALID_ARG), (dict(Hkv=0), swa.SWA_ERR_INVALID_ARG),
    (dict(H=130, Hkv=2), swa.SWA_ERR_UNSUPPORTED), (dict(D=80), swa.SWA_ERR_UNSUPPORTED),
    (dict(B=65536), swa.SWA_ERR_UNSUPPORTED), (dict(page_size=100), swa.SWA_ERR_UNSUPPORTED),
    (dict(n_pages=0), swa.SWA_ERR_INVALID_ARG), (dict(n_pages=1 << 26), swa.SWA_ERR_UNSUPPORTED),
    (dict(max_pages=0), swa.SWA_ERR_INVALID_ARG), (dict(max_pages=1 << 27), swa.SWA_ERR_UNSUPPORTED),
    (dict(rope_base=0.0), swa.SWA_ERR_INVALID_ARG), (dict(eps=-1.0), swa.SWA_ERR_INVALID_ARG),
    (dict(ws_bytes=0), swa.SWA_ERR_NO_MEMORY),
])
def test_decode_refuses_bad_arguments(kw, code):
    assert _decode(**kw) == code


def test_decode_workspace_bytes():
    n = swa.swa_attn_kv8_decode_workspace_bytes(16, 12, 12, 128)
    assert n >= 16 * 12 * 128 * 2 and n % 1024 == 0
    assert swa.swa_attn_kv8_decode_workspace_bytes(16, 12, 5, 128) == 0
    assert swa.swa_attn_kv8_decode_workspace_bytes(16, 12, 12, 96) == 0
    assert swa.swa_attn_kv8_decode_workspace_bytes(1, 128, 1, 64) == 0
    assert _decode(ws_bytes=swa.swa_attn_kv8_decode_workspace_bytes(2, 4, 2, 64) - 1) == swa.SWA_ERR_NO_MEMORY


def test_valid_calls_reach_the_device_check():
    if torch.cuda.is_available():
        pytest.skip("the fake addresses must not reach a GPU")
    assert _pages() == _rows("write") == _rows("read") == _decode() == swa.SWA_ERR_NO_DEVICE
    assert _decode(k=None, v=None) == _decode(ve=A, gate_x=A, Wg=A, doc_start=A, lse=None) == swa.SWA_ERR_NO_DEVICE
    assert _decode(H=128) == swa.SWA_ERR_NO_DEVICE


def test_tensor_calls_refuse_what_the_c_calls_cannot_see():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    x = torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16)
    codes, scale = torch.zeros((4, 2, 16, 64), dtype=torch.float8_e4m3fn), torch.zeros((4, 2))
    with pytest.raises(ValueError, match="contiguous CUDA"):
        swa.kv_pages(i(2, 4), i(2), i(2), i(4), i(2), i(2), 16)
    with pytest.raises(ValueError, match=r"block_table must be \(B, max_pages\)"):
        swa.kv_pages(i(8), i(2), i(2), i(4), i(2), i(2), 16)
    with pytest.raises(ValueError, match="must be contiguous|contiguous CUDA"):
        swa.kv8_write(x, x, i(2, 3), codes, codes, scale, scale)
    with pytest.raises(ValueError, match="kh and vp must be"):
        swa.kv8_write(x[0], x[0], i(2, 3), codes, codes, scale, scale)
    with pytest.raises(ValueError, match="slots must be"):
        swa.kv8_read(i(6), codes, codes, scale, scale)
    with pytest.raises(ValueError, match="block_table"):
        swa.decode_kv8(x[0], None, None, codes, codes, scale, scale, i(3), i(3))
