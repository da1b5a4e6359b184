"""Refusals and host helpers of the paged-cache operators: every call here is
host-only or fails its checks before any HIP call."""
import ctypes

import numpy as np
import pytest

from scatter_tile_gather_amd._binding import _HOW, StgTensor

F32, BF16, F16, I32, U8 = range(5)
OK, INVALID, UNSUPPORTED, RANGE = range(4)
P = 0x1000  # a pointer that no check reads through
B = ctypes.byref


def t(shape, dtype=BF16, data=P, stride=None):
    d = StgTensor()
    d.data, d.dtype, d.rank = data, dtype, len(shape)
    st = stride or [int(np.prod(shape[i + 1:])) for i in range(len(shape))]
    for i in range(4):
        d.shape[i] = shape[i] if i < len(shape) else 1
        d.stride[i] = st[i] if i < len(shape) else 0
    return d


@pytest.fixture(scope="module")
def lib(stg):
    return stg.load_library()


def attention(lib, **kw):
    a = dict(q=t([4, 8, 64]), k=t([10, 16, 2, 64]), v=t([10, 16, 2, 64]), table=t([4, 3], I32), lens=P, ks=None, vs=None,
             scale=1.0, window=0, max_len=0, out=t([4, 8, 64]), lse=None, ws=None, wn=0)
    a.update(kw)
    ref = lambda x: None if x is None else B(x)  # noqa: E731
    return lib.paged_attention(ref(a["q"]), ref(a["k"]), ref(a["v"]), ref(a["table"]), a["lens"], a["ks"], a["vs"],
                               a["scale"], a["window"], a["max_len"], ref(a["out"]), a["lse"], a["ws"], a["wn"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(table=None), INVALID), (dict(out=None), INVALID),
    (dict(lens=None), INVALID),
    (dict(q=t([4, 8, 64], F32)), UNSUPPORTED), (dict(q=t([4, 512])), INVALID), (dict(q=t([4, 8, 64], stride=[1024, 128, 2])), INVALID),
    (dict(q=t([4, 8, 64], data=0)), INVALID),
    (dict(k=t([10, 16, 2, 64], F32)), UNSUPPORTED), (dict(k=t([10, 16, 2, 64], F16)), INVALID),
    (dict(v=t([10, 16, 2, 64], F16)), INVALID), (dict(v=t([10, 8, 2, 64])), INVALID), (dict(k=t([10, 32, 64])), INVALID),
    (dict(k=t([10, 16, 2, 64], stride=[4096, 256, 128, 2])), INVALID),
    (dict(k=t([10, 16, 2, 32]), v=t([10, 16, 2, 32])), INVALID), (dict(k=t([10, 16, 3, 64]), v=t([10, 16, 3, 64])), INVALID),
    (dict(k=t([10, 16, 0, 64]), v=t([10, 16, 0, 64])), INVALID),
    (dict(table=t([4, 3], BF16)), UNSUPPORTED), (dict(table=t([5, 3], I32)), INVALID), (dict(table=t([12], I32)), INVALID),
    (dict(table=t([4, 3], I32, stride=[6, 2])), INVALID), (dict(table=t([4, 3], I32, stride=[2, 1])), INVALID),
    (dict(out=t([4, 8, 64], F16)), INVALID), (dict(out=t([4, 4, 64])), INVALID),
    (dict(ks=P), INVALID), (dict(vs=P), INVALID), (dict(window=-1), INVALID), (dict(max_len=-1), INVALID),
    (dict(q=t([4, 8, 7]), k=t([10, 16, 2, 7]), v=t([10, 16, 2, 7]), out=t([4, 8, 7])), UNSUPPORTED),
    (dict(q=t([4, 8, 257]), k=t([10, 16, 2, 257]), v=t([10, 16, 2, 257]), out=t([4, 8, 257])), UNSUPPORTED),
    (dict(q=t([4, 1 << 17, 64]), out=t([4, 1 << 17, 64])), RANGE),
    (dict(k=t([1 << 31, 16, 2, 64]), v=t([1 << 31, 16, 2, 64])), RANGE),
    (dict(table=t([4, 5000], I32)), INVALID),                      # long rows: a workspace is missing
    (dict(table=t([4, 5000], I32), ws=0x1100, wn=16), INVALID),      # too small
    (dict(table=t([4, 5000], I32), ws=0x1010, wn=1 << 40), INVALID),  # unaligned
], ids=lambda x: None if isinstance(x, dict) else str(x))
def test_attention_refuses(lib, kw, code):
    assert attention(lib, **kw) == code
    assert lib.stg_last_error()


def test_attention_of_nothing_and_workspace(lib):
    assert attention(lib, q=t([0, 8, 64], data=0), table=t([0, 3], I32, data=0), out=t([0, 8, 64], data=0)) == OK
    q, k = t([4, 8, 64]), t([10, 16, 2, 64])
    need = lambda width, window, hint: lib.paged_attention_workspace(B(q), B(k), B(t([4, width], I32)), window, hint)  # noqa: E731
    assert need(1, 0, 0) == 0
    full = need(5000, 0, 0)
    assert full >= (64 + 2) * 4 * 4 * 8  # at least depth + 2 floats per row and head
    assert need(5000, 100, 0) == 0 and need(5000, 0, 200) == 0
    assert 0 < need(5000, 0, 2000) <= full
    assert need(5000, -1, 0) == -INVALID
    assert lib.paged_attention_workspace(None, B(k), B(t([4, 3], I32)), 0, 0) == -INVALID


def how(freq=P, qw=P, kw=P, rotary=64, interleaved=0, norm=1, wd=F32, gain=1.0, eps=1e-6):
    return _HOW.pack(freq or 0, qw or 0, kw or 0, rotary, interleaved, norm, wd, gain, eps)


Q, K = [5, 4, 64], [5, 2, 64]


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(how=None), INVALID), (dict(q_out=None), INVALID), (dict(k_out=None), INVALID),
    (dict(pos=None), INVALID), (dict(q=t(Q, I32), q_out=t(Q, I32)), UNSUPPORTED), (dict(q=t(Q, F16), q_out=t(Q, F16)), INVALID),
    (dict(q=t([5, 256])), INVALID), (dict(q=t(Q, stride=[512, 128, 2])), INVALID), (dict(q=t([6, 4, 64]), q_out=t([6, 4, 64])), INVALID),
    (dict(k=t([5, 2, 32]), k_out=t([5, 2, 32])), INVALID), (dict(q_out=t(Q, F16)), INVALID), (dict(k_out=t(Q)), INVALID),
    (dict(q=t([5, 4, 1025]), k=t([5, 2, 1025]), q_out=t([5, 4, 1025]), k_out=t([5, 2, 1025])), UNSUPPORTED),
    (dict(q=t([5, 4, 0]), k=t([5, 2, 0]), q_out=t([5, 4, 0]), k_out=t([5, 2, 0])), UNSUPPORTED),
    (dict(how=how(rotary=63)), INVALID), (dict(how=how(rotary=66)), INVALID), (dict(how=how(rotary=-2)), INVALID),
    (dict(how=how(freq=None)), INVALID), (dict(how=how(norm=0)), INVALID), (dict(how=how(wd=F16)), UNSUPPORTED),
    (dict(how=how(wd=U8)), UNSUPPORTED), (dict(how=how(eps=-1.0)), INVALID), (dict(how=how(eps=float("nan"))), INVALID),
    (dict(q=t([5, 65537, 64]), q_out=t([5, 65537, 64])), RANGE),
], ids=lambda x: None if isinstance(x, dict) else str(x))
def test_norm_rope_refuses(lib, kw, code):
    a = dict(q=t(Q), k=t(K), pos=P, how=how(), q_out=t(Q), k_out=t(K))
    a.update(kw)
    ref = lambda x: None if x is None else B(x)  # noqa: E731
    assert lib.qk_norm_rope(ref(a["q"]), ref(a["k"]), a["pos"], a["how"], ref(a["q_out"]), ref(a["k_out"]), None) == code
    assert lib.stg_last_error()
    # the same operands through the backward call
    if "q_out" not in kw and "k_out" not in kw:
        assert lib.qk_norm_rope_backward(ref(a["q"]), ref(a["k"]), ref(a["q"]), ref(a["k"]), a["pos"], a["how"], ref(a["q"]),
                                         ref(a["k"]), None, None, None, 0, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(v=None), INVALID), (dict(v=t(Q)), INVALID), (dict(v=t(K, F16)), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID),
    (dict(table=None), INVALID), (dict(table=t([4, 3], F16)), UNSUPPORTED), (dict(kc=t([9, 16, 2, 64], F16)), INVALID),
    (dict(kc=t([9, 16, 2, 64], F16), vc=t([9, 16, 2, 64], F16)), INVALID), (dict(vc=t([9, 16, 2, 32])), INVALID),
    (dict(kc=t([9, 16, 1, 64]), vc=t([9, 16, 1, 64])), INVALID), (dict(ks=P), INVALID), (dict(vs=P), INVALID),
    (dict(q_out=t(K)), INVALID), (dict(pos=None), INVALID),
    (dict(q=t(Q, F32), k=t(K, F32), v=t(K, F32), q_out=t(Q, F32)), UNSUPPORTED),
], ids=lambda x: None if isinstance(x, dict) else str(x))
def test_append_refuses(lib, kw, code):
    a = dict(q=t(Q), k=t(K), v=t(K), pos=P, kc=t([9, 16, 2, 64]), vc=t([9, 16, 2, 64]), table=t([4, 3], I32), ks=None,
             vs=None, q_out=t(Q))
    a.update(kw)
    ref = lambda x: None if x is None else B(x)  # noqa: E731
    assert lib.qk_norm_rope_append(ref(a["q"]), ref(a["k"]), ref(a["v"]), a["pos"], how(), None, ref(a["kc"]), ref(a["vc"]),
                                   ref(a["table"]), a["ks"], a["vs"], ref(a["q_out"]), None) == code
    assert lib.stg_last_error()


def test_backward_refuses(lib):
    q, k = t(Q), t(K)
    call = lambda how_, dqw, ws, wn, dq=q, g=q: lib.qk_norm_rope_backward(  # noqa: E731
        B(g), B(k), B(q), B(k), P, how_, B(dq), B(k), dqw, None, ws, wn, None)
    need = lib.qk_norm_rope_backward_workspace(B(q), B(k))
    assert need > 0
    assert call(how(), P, None, 0) == INVALID
    assert call(how(), P, 0x1100, need - 1) == INVALID
    assert call(how(), P, 0x1010, need) == INVALID
    assert call(how(qw=None, kw=None, norm=0), P, 0x1100, need) == INVALID
    assert call(how(qw=None, kw=None, wd=I32), P, 0x1100, need) == UNSUPPORTED
    assert call(how(), None, None, 0, dq=k) == INVALID
    assert call(how(), None, None, 0, g=t(Q, F16)) == INVALID
    assert lib.qk_norm_rope_backward_workspace(B(q), None) == -INVALID
    assert lib.qk_norm_rope_backward_workspace(B(q), B(t([5, 2, 32]))) == -INVALID


def test_page_calls_refuse(lib):
    cache, table = t([2, 10, 100], U8), t([4, 3], I32)
    need = lib.pages_workspace(10, 4)
    ws = 0x1100
    assert need > 0 and lib.pages_workspace(-1, 0) == -INVALID and lib.pages_workspace(1 << 31, 0) == -RANGE
    assert lib.pages_workspace(10, -1) == -INVALID
    copy = lambda c=cache, s=P, d=P, n=1: lib.pages_copy(B(c), s, d, n, None)  # noqa: E731
    assert copy(s=None) == copy(d=None) == copy(n=-1) == INVALID
    assert copy(c=t([20, 100], U8)) == INVALID and copy(c=t([2, 10, 100], U8, stride=[1000, 100, 2])) == INVALID
    assert copy(c=t([2, 10, 100], U8, stride=[1000, 50, 1])) == INVALID and copy(c=t([2, 10, 100], 17)) == UNSUPPORTED
    assert copy(n=1 << 31) == RANGE and copy(n=0) == OK and lib.pages_copy(None, P, P, 1, None) == INVALID
    reserve = lambda tb=table, lens=P, new=P, refs=P, n=10, slots=16, w=ws, wn=need: lib.pages_reserve(  # noqa: E731
        B(tb), lens, new, refs, n, slots, None, w, wn, None)
    assert reserve(lens=None) == reserve(new=None) == reserve(refs=None) == reserve(slots=0) == reserve(n=-1) == INVALID
    assert reserve(w=None) == reserve(wn=need - 1) == reserve(w=0x1010) == INVALID
    assert reserve(tb=t([4, 3], U8)) == UNSUPPORTED and reserve(slots=1 << 31) == RANGE
    fork = lambda c=cache, tb=table, lens=P, refs=P, slots=16, p=P, k=P, n=4, w=ws, wn=need: lib.pages_fork(  # noqa: E731
        B(c), B(tb), lens, refs, slots, p, k, n, None, w, wn, None)
    assert fork(lens=None) == fork(refs=None) == fork(p=None) == fork(k=None) == fork(n=-1) == fork(slots=0) == INVALID
    assert fork(w=None) == fork(wn=need - 1) == fork(w=0x1010) == INVALID
    assert fork(c=t([20, 100], U8)) == INVALID and fork(tb=t([4, 3], F32)) == UNSUPPORTED
    free = lambda tb=table, lens=P, refs=P, pages=10, rows=P, n=1: lib.pages_free(B(tb), lens, refs, pages, rows, n, None)  # noqa: E731
    assert free(lens=None) == free(refs=None) == free(rows=None) == free(n=-1) == free(pages=-1) == INVALID
    assert free(n=0) == OK and free(tb=t([4, 3], U8)) == UNSUPPORTED
    compact = lambda c=cache, tb=table, refs=P, remap=P, w=ws, wn=need: lib.pages_compact(  # noqa: E731
        B(c), B(tb), refs, remap, w, wn, None)
    assert compact(refs=None) == compact(remap=None) == compact(w=None) == compact(wn=100) == compact(w=0x1010) == INVALID
    assert compact(c=t([2, 0, 100], U8, data=0), refs=None, remap=None) == OK


def test_rope_frequencies(stg):
    f, g = stg.rope_frequencies(64, 10000.0)
    np.testing.assert_array_equal(f, (10000.0 ** (-np.arange(32) / 32.0)).astype(np.float32))
    assert g == 1.0
    lin, _ = stg.rope_frequencies(64, 10000.0, "linear", 4.0)
    np.testing.assert_array_equal(lin, (10000.0 ** (-np.arange(32) / 32.0) / 4).astype(np.float32))
    ntk, _ = stg.rope_frequencies(64, 10000.0, "ntk", 4.0)
    np.testing.assert_allclose(ntk[0], 1.0)
    np.testing.assert_allclose(ntk[-1], f[-1] / 4.0, rtol=1e-6)  # the lowest frequency is the one divided by factor
    yarn, gain = stg.rope_frequencies(64, 10000.0, "yarn", 4.0, original_len=4096)
    turns = 4096 * f / (2 * np.pi)
    np.testing.assert_allclose(gain, 0.1 * np.log(4.0) + 1, rtol=1e-6)
    np.testing.assert_array_equal(yarn[turns > 45], f[turns > 45])  # well past 32 turns: unchanged
    np.testing.assert_allclose(yarn[turns < 0.7], f[turns < 0.7] / 4, rtol=1e-6)
    assert np.all(np.diff(yarn) < 0) and np.all(yarn <= f) and np.all(yarn >= f / 4 * (1 - 1e-6))
    for same in ("linear", "ntk", "yarn"):
        np.testing.assert_allclose(stg.rope_frequencies(64, 10000.0, same, 1.0)[0], f, rtol=1e-6)
    assert stg.rope_frequencies(0)[0].size == 0 and stg.rope_frequencies(2, scaling="ntk", factor=8.0)[0][0] == 1.0
    for bad in (dict(rotary_dim=7), dict(rotary_dim=-2), dict(rotary_dim=8, base=1.0), dict(rotary_dim=8, base=float("nan")),
                dict(rotary_dim=8, scaling="linear", factor=0.5), dict(rotary_dim=8, scaling="yarn", factor=2.0, beta_fast=1.0),
                dict(rotary_dim=8, scaling="yarn", factor=2.0, beta_slow=0.0),
                dict(rotary_dim=8, scaling="yarn", factor=2.0, original_len=0.0)):
        with pytest.raises(stg.StgError):
            stg.rope_frequencies(**bad)
    assert stg.load_library().rope_frequencies(8, 10000.0, 9, 1.0, 1.0, 2.0, 1.0, P, None) == INVALID


def test_binding_refuses_host_tensors_and_shapes(stg):
    import torch

    q, cache = torch.zeros(4, 8, 64), torch.zeros(10, 16, 2, 64)
    i = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: stg.paged_attention(q, cache, cache, i.view(4, 1), i),
                 lambda: stg.qk_norm_rope(q, q, i, torch.ones(32)),
                 lambda: stg.qk_norm_rope_append(q, q, q, i, torch.ones(32), cache, cache, i.view(4, 1)),
                 lambda: stg.qk_norm_rope_backward(q, q, q, q, i, torch.ones(32)),
                 lambda: stg.pages_copy(torch.zeros(2, 3, 4), i, i),
                 lambda: stg.pages_reserve(i.view(4, 1), i, i, i, 4),
                 lambda: stg.pages_fork(torch.zeros(2, 4, 4), i.view(4, 1), i, i, 4, i, i),
                 lambda: stg.pages_free(i.view(4, 1), i, i, i),
                 lambda: stg.pages_compact(torch.zeros(2, 4, 4), i.view(4, 1), i)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    for call in (lambda: stg.paged_attention(q[0], cache, cache, i.view(4, 1), i), lambda: stg.qk_norm_rope(q[0], q, i, i),
                 lambda: stg.pages_copy(q[0], i, i), lambda: stg.pages_free(i, i, i, i)):
        with pytest.raises(ValueError, match="must be"):
            call()
