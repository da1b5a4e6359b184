"""Norm and rotation of queries and keys on the GPU against the fp64 oracle:
forward, into a cache, and backward.

Tolerances, u = 2^-24, from the fp32 computation: the sum of D squares is off
by at most D u relative, its root by half of that, the products by a few u; cos
and sin of an angle reduced in fp64 and rounded to fp32 (at most pi, so off by
at most 2^-23) by 8 u together.  So a result is off by at most (D / 2 + 24) u
times the magnitudes that enter it (the oracle's `bound`), plus half a rounding
step of the output's type.  A backward result has two such sums (of the squares
and of u w x): (3 D / 2 + 48) u.  A weight's gradient of n terms: (n + D / 2 +
48) u times the terms' magnitudes."""
import numpy as np
import pytest
import torch

from gpu_util import say
from paged_util import HALF_STEP, TINY, TYPES, U32, f64, random_table

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(seed, tokens, hq, hk, depth, rotary, kind, weight="f32", fused=True):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[kind]
    x = torch.randn((tokens, hq + 2 * hk, depth), generator=g).to(dt).to(DEV)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    w = [(1 + 0.3 * torch.randn(depth, generator=g)).to(torch.float32 if weight == "f32" else dt).to(DEV) for _ in range(2)]
    pos = torch.randint(0, 1 << 17, (tokens,), generator=g, dtype=torch.int32)
    if tokens > 3:
        pos[0], pos[1], pos[2], pos[3] = 0, 1, -5, (1 << 28) - 1
    f = (10000.0 ** (-torch.arange(rotary // 2) / max(1, rotary // 2))).float()
    return q, k, v, w, pos.to(DEV), f.to(DEV)


def check(got, want, bound, kind, factor):
    err = np.abs(f64(got) - want)
    tol = factor * U32 * bound * 1.01 + HALF_STEP[kind] * np.abs(want) * (1 + 1e-3) + TINY[kind]
    assert np.all(err <= tol), float((err / tol).max())


# (tokens, q heads, k heads, depth, rotary): pairs in a lane, pairs across
# lanes, part of a head, nothing; chunks that end inside a head; one token; one
# head; more heads than a wave's groups; the largest depth
SHAPES = [(5, 4, 2, 128, 128), (1, 1, 1, 64, 64), (33, 6, 3, 96, 64), (7, 3, 1, 80, 80), (9, 5, 5, 80, 60),
          (6, 7, 1, 100, 100), (4, 2, 2, 33, 14), (3, 1, 1, 1, 0), (2, 2, 1, 2, 2), (8, 40, 8, 256, 192),
          (5, 3, 2, 1024, 1024), (5, 2, 1, 520, 518), (300, 16, 4, 64, 32), (4, 3, 2, 128, 0), (11, 2, 0, 72, 24)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(stg, orc, shape, interleaved, kind):
    tokens, hq, hk, depth, rotary = shape
    weight = "same" if tokens % 2 else "f32"
    q, k, _, w, pos, f = make(1, tokens, hq, hk, depth, rotary, kind, weight)
    say("qk_norm_rope", shape, interleaved, kind)
    got = stg.qk_norm_rope(q, k, pos, f, w[0], w[1], eps=1e-5, interleaved=interleaved, rope_scale=1.25)
    for y, x, wt in ((got[0], q, w[0]), (got[1], k, w[1])):
        want, bound = orc.norm_rope(f64(x), f64(wt), pos.cpu().numpy(), f.cpu().numpy(), interleaved, 1.25, True, 1e-5)
        check(y, want, bound, kind, depth / 2 + 24)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,weighted", [(False, False), (True, False)])
def test_forward_without_weights(stg, orc, norm, weighted, interleaved, kind):
    q, k, _, _, pos, f = make(2, 19, 5, 2, 112, 50, kind)
    say("qk_norm_rope without weights", norm, interleaved, kind)
    got = stg.qk_norm_rope(q, k, pos, f, norm=norm, interleaved=interleaved)
    for y, x in zip(got, (q, k)):
        want, bound = orc.norm_rope(f64(x), None, pos.cpu().numpy(), f.cpu().numpy(), interleaved, 1.0, norm, 1e-6)
        check(y, want, bound, kind, 112 / 2 + 24)


def test_forward_in_place_and_strided(stg):
    """Outputs may be the inputs, or views with strides of their own; nothing between them is written."""
    q, k, _, w, pos, f = make(3, 21, 6, 2, 96, 40, "bf16")
    say("qk_norm_rope in place and into views")
    want = stg.qk_norm_rope(q, k, pos, f, *w)
    room = torch.full((21, 11, 101), 7.0, dtype=torch.bfloat16, device=DEV)
    stg.qk_norm_rope(q, k, pos, f, *w, q_out=room[:, 1:7, 3:99], k_out=room[:, 8:10, 3:99])
    assert torch.equal(room[:, 1:7, 3:99], want[0]) and torch.equal(room[:, 8:10, 3:99], want[1])
    room[:, 1:7, 3:99] = 7.0
    room[:, 8:10, 3:99] = 7.0
    assert bool((room == 7.0).all())
    v = stg.qk_norm_rope(q, k, pos, f, *w, q_out=q, k_out=k)
    assert v[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_unaligned_rows(stg, orc):
    """Rows that start at every odd element."""
    base = torch.randn((9, 700), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(DEV)
    pos = torch.arange(9, dtype=torch.int32, device=DEV)
    f = torch.ones(32, device=DEV)
    for off in (1, 3, 7):
        q = base[:, off:off + 3 * 64].unflatten(1, (3, 64))
        k = base[:, off + 201:off + 201 + 2 * 64].unflatten(1, (2, 64))
        say("qk_norm_rope at offset", off)
        got = stg.qk_norm_rope(q, k, pos, f)
        for y, x in zip(got, (q, k)):
            want, bound = orc.norm_rope(f64(x), None, pos.cpu().numpy(), f.cpu().numpy())
            check(y, want, bound, "bf16", 64 / 2 + 24)


def test_special_values(stg):
    """A zero head stays zero, NaN and infinity stay in their head, empty calls do nothing."""
    q, k, _, w, pos, f = make(5, 4, 3, 2, 64, 64, "bf16", fused=False)
    want = stg.qk_norm_rope(q, k, pos, f, *w)
    q[1, 0] = 0
    q[2, 1, 5] = float("nan")
    k[3, 1, 7] = float("inf")
    say("qk_norm_rope with zeros, NaN and infinity")
    got = stg.qk_norm_rope(q, k, pos, f, *w)
    assert bool((got[0][1, 0] == 0).all()) and bool(got[0][2, 1].isnan().all()) and bool(got[1][3, 1].isnan().any())
    keep = torch.ones(4, 3, dtype=torch.bool, device=DEV)
    keep[1, 0] = keep[2, 1] = False
    assert torch.equal(got[0][keep], want[0][keep])
    none = stg.qk_norm_rope(q[:0], k[:0], pos[:0], f, *w)
    assert none[0].shape == (0, 3, 64)


# ---- into a cache -----------------------------------------------------------

def e4m3_error(got, want, fp32):
    """Codes' values against exact values: half a step (2^-4 relative, 2^-10 in
    the subnormals) plus the fp32 error; saturated at 448."""
    want = np.clip(want, -448, 448)
    return np.all(np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) * (1 + 1e-6) + fp32)


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", [(1, 8, 2, 128, 128, 16), (40, 6, 3, 80, 60, 5), (23, 3, 1, 100, 100, 1),
                                   (64, 32, 8, 128, 128, 16), (9, 2, 2, 256, 64, 100)], ids=str)
def test_append(stg, orc, shape, interleaved, kind, cache):
    tokens, hq, hk, depth, rotary, slots = shape
    rng = np.random.default_rng(6)
    q, k, v, w, _, f = make(6, tokens, hq, hk, depth, rotary, kind)
    rows_n = 3
    lens = rng.integers(0, 50, rows_n)
    n = np.bincount(rng.integers(0, rows_n, tokens), minlength=rows_n)
    rows = np.repeat(np.arange(rows_n), n).astype(np.int32)
    pos = np.concatenate([lens[b] + np.arange(n[b]) for b in range(rows_n)]).astype(np.int32)
    width = -(-int((lens + n).max()) // slots)
    pages = width * rows_n + 2
    table = random_table(rng, lens + n, slots, pages, width)
    mix = rng.permutation(tokens)  # tokens in any order
    rows, pos = rows[mix], pos[mix]
    skip = np.zeros(tokens, bool)
    if tokens > 8:  # none of these is written: rows, positions and pages out of range
        rows[0], rows[1], pos[2], pos[3] = -1, rows_n, -1, width * slots
        table[rows[4], pos[4] // slots] = pages
        skip[:4] = True
        skip |= (rows == rows[4]) & (pos // slots == pos[4] // slots)
    store = torch.randn((2, pages, slots, hk, depth), generator=torch.Generator().manual_seed(7)).to(TYPES[cache]).to(DEV)
    before = store.clone()
    ks = vs = None
    if cache == "e4m3":
        ks = torch.linspace(0.01, 0.3, hk, device=DEV)
        vs = torch.linspace(0.2, 0.002, hk, device=DEV)  # the last head saturates
    say("qk_norm_rope_append", shape, interleaved, kind, cache)
    got = stg.qk_norm_rope_append(q, k, v, torch.from_numpy(pos).to(DEV), f, store[0], store[1],
                                  torch.from_numpy(table).to(DEV), rows=torch.from_numpy(rows).to(DEV), k_scale=ks,
                                  v_scale=vs, q_weight=w[0], k_weight=w[1], interleaved=interleaved)
    want, bound = orc.norm_rope(f64(q), f64(w[0]), pos, f.cpu().numpy(), interleaved)
    check(got, want, bound, kind, depth / 2 + 24)
    kw, kb = orc.norm_rope(f64(k), f64(w[1]), pos, f.cpu().numpy(), interleaved)
    now, was = f64(store.float()), f64(before.float())
    for t in np.flatnonzero(~skip):
        page, slot = table[rows[t], pos[t] // slots], pos[t] % slots
        if cache == "e4m3":
            sk, sv = f64(ks)[:, None], f64(vs)[:, None]
            fp32 = (depth / 2 + 26) * U32 * kb[t] / sk
            assert e4m3_error(now[0, page, slot], kw[t] / sk, fp32)
            assert e4m3_error(now[1, page, slot], f64(v)[t] / sv, 2 * U32 * np.abs(f64(v)[t] / sv))
        else:
            err = np.abs(now[0, page, slot] - kw[t])
            assert np.all(err <= (depth / 2 + 24) * U32 * kb[t] * 1.01 + HALF_STEP[kind] * np.abs(kw[t]) * 1.001 + TINY[kind])
            np.testing.assert_array_equal(now[1, page, slot], f64(v)[t])
        now[:, page, slot] = was[:, page, slot]
    np.testing.assert_array_equal(now, was)  # nothing else was written


def test_append_keeps_bits_of_values(stg):
    """Values pass unchanged into a cache of their type (NaN payloads aside, which no test fixes), and
    e4m3 codes of NaN and infinity are NaN and 448."""
    v = torch.tensor([[[1.5, -0.0, float("inf"), float("-inf"), float("nan"), 1e-30, 448.0, 460.0]]], device=DEV)
    v = v.to(torch.bfloat16)
    q = torch.ones_like(v)
    cache = torch.zeros((2, 1, 2, 1, 8), dtype=torch.bfloat16, device=DEV)
    table, pos = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    f = torch.ones(4, device=DEV)
    say("qk_norm_rope_append of special values")
    stg.qk_norm_rope_append(q, q, v, pos, f, cache[0], cache[1], table)
    got = cache[1, 0, 1]
    assert torch.equal(got.isnan(), v[0].isnan()) and torch.equal(got[~got.isnan()], v[0][~v[0].isnan()])
    assert bool(torch.signbit(got[0, 1]))
    codes = torch.zeros((2, 1, 2, 1, 8), dtype=torch.float8_e4m3fn, device=DEV)
    stg.qk_norm_rope_append(q, q, v, pos, f, codes[0], codes[1], table)
    got = codes[1, 0, 1, 0].float().cpu()
    assert got[:4].tolist() == [1.5, 0.0, 448.0, -448.0] and bool(got[4].isnan()) and got[5:].tolist() == [0.0, 448.0, 448.0]


def test_append_past_32_bits(stg):
    """Pages whose offsets pass 2^32 bytes."""
    slots, hk, depth = 16, 8, 128
    pages = (5 << 30) // (slots * hk * depth * 2)
    q, k, v, w, _, f = make(8, 2, 4, hk, depth, depth, "bf16")
    cache = torch.zeros((2, pages, slots, hk, depth), dtype=torch.bfloat16, device=DEV)
    table = torch.tensor([[pages - 1], [pages - 2]], dtype=torch.int32, device=DEV)
    pos = torch.tensor([15, 3], dtype=torch.int32, device=DEV)
    say("qk_norm_rope_append into a 10 GiB cache")
    got = stg.qk_norm_rope_append(q, k, v, pos, f, cache[0], cache[1], table, q_weight=w[0], k_weight=w[1])
    want = stg.qk_norm_rope(q, k, pos, f, *w)
    assert torch.equal(got, want[0])
    for t, (p, s) in enumerate(((pages - 1, 15), (pages - 2, 3))):
        assert torch.equal(cache[0, p, s], want[1][t]) and torch.equal(cache[1, p, s], v[t])
        cache[:, p, s] = 0
    assert not bool(cache[:, -2:].any()) and not bool(cache[:, :2].any())


# ---- backward ---------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES + [(2000, 8, 2, 64, 64), (700, 1, 1, 128, 96)], ids=str)
def test_backward(stg, orc, shape, interleaved, kind):
    tokens, hq, hk, depth, rotary = shape
    weight = "same" if tokens % 2 else "f32"
    q, k, _, w, pos, f = make(9, tokens, hq, hk, depth, rotary, kind, weight)
    gq, gk, gv, *_ = make(10, tokens, hq, hk, depth, rotary, kind)
    say("qk_norm_rope_backward", shape, interleaved, kind)
    got = stg.qk_norm_rope_backward(gq, gk, q, k, pos, f, w[0], w[1], eps=1e-5, interleaved=interleaved, rope_scale=1.25)
    again = stg.qk_norm_rope_backward(gq, gk, q, k, pos, f, w[0], w[1], eps=1e-5, interleaved=interleaved, rope_scale=1.25)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    wk = kind if weight == "same" else "f32"
    for i, (g, x, wt) in enumerate(((gq, q, w[0]), (gk, k, w[1]))):
        dx, bound, dw, abs_dw = orc.norm_rope_backward(f64(g), f64(x), f64(wt), pos.cpu().numpy(), f.cpu().numpy(),
                                                       interleaved, 1.25, True, 1e-5)
        check(got[i], dx, bound, kind, 1.5 * depth + 48)
        assert got[2 + i].dtype == wt.dtype
        check(got[2 + i], dw, abs_dw, wk, x.shape[0] * x.shape[1] + depth / 2 + 48)


@pytest.mark.parametrize("norm", [True, False])
def test_backward_without_weights(stg, orc, norm):
    q, k, _, _, pos, f = make(11, 13, 4, 2, 96, 50, "f32")
    gq, gk, *_ = make(12, 13, 4, 2, 96, 50, "f32")
    say("qk_norm_rope_backward without weights", norm)
    dq, dk, dqw, dkw = stg.qk_norm_rope_backward(gq, gk, q, k, pos, f, norm=norm, workspace=None)
    assert dqw is None and dkw is None
    for got, g, x in ((dq, gq, q), (dk, gk, k)):
        dx, bound, _, _ = orc.norm_rope_backward(f64(g), f64(x), None, pos.cpu().numpy(), f.cpu().numpy(), False, 1.0, norm)
        check(got, dx, bound, "f32", 1.5 * 96 + 48)


def test_backward_one_weight_and_no_tokens(stg, orc):
    """A weight on one side only; a batch of no tokens has zero weight gradients."""
    q, k, _, w, pos, f = make(13, 6, 4, 2, 64, 64, "bf16")
    say("qk_norm_rope_backward with a query weight only")
    dq, dk, dqw, dkw = stg.qk_norm_rope_backward(q, k, q, k, pos, f, q_weight=w[0])
    assert dkw is None
    _, _, dw, mag = orc.norm_rope_backward(f64(q), f64(q), f64(w[0]), pos.cpu().numpy(), f.cpu().numpy())
    check(dqw, dw, mag, "f32", 24 + 32 + 48)
    got = stg.qk_norm_rope_backward(q[:0], k[:0], q[:0], k[:0], pos[:0], f, *w)
    assert bool((got[2] == 0).all()) and bool((got[3] == 0).all())


def test_backward_against_differences(stg):
    """Directional differences of the forward call itself, in fp32: for L = sum
    g . y, (L(x + h e) - L(x - h e)) / 2h against dx . e, for steps on the
    inputs and on both weights.  The third-order term is h^2 / 6 times a third
    derivative of order 1 per unit of |L|'s terms; rounding is 2 u |terms| / h."""
    q, k, _, w, pos, f = make(14, 50, 4, 2, 64, 48, "f32", fused=False)
    gq, gk, *_ = make(15, 50, 4, 2, 64, 48, "f32", fused=False)
    dirs = [torch.randn(x.shape, generator=torch.Generator().manual_seed(i)).to(DEV) for i, x in enumerate((q, k, *w))]
    say("qk_norm_rope_backward against differences")
    dq, dk, dqw, dkw = stg.qk_norm_rope_backward(gq, gk, q, k, pos, f, *w)

    def terms(at):
        y = stg.qk_norm_rope(at[0], at[1], pos, f, at[2], at[3])
        return torch.cat([(y[0] * gq).flatten(), (y[1] * gk).flatten()]).double()

    h = 2.0 ** -7
    for i, grad in enumerate((dq, dk, dqw, dkw)):
        at = [q, k, *w]
        plus, minus = ([x + s * h * dirs[j] if j == i else x for j, x in enumerate(at)] for s in (1, -1))
        tp, tm = terms(plus), terms(minus)
        diff = (tp - tm).sum() / (2 * h)
        slope = (grad.double() * dirs[i].double()).sum()
        scale = tp.abs().sum()
        # the terms' fp32 errors are independent in sign, but the bound takes them all one way
        tol = scale * (60 * U32 / h + 4 * h * h)
        assert abs(float(diff - slope)) <= float(tol), (i, float(diff), float(slope), float(tol))


def test_captured_forward_and_backward_replay_like_eager(stg):
    q, k, v, w, pos, f = make(16, 70, 6, 2, 128, 128, "bf16")
    gq, gk, *_ = make(17, 70, 6, 2, 128, 128, "bf16")
    outs = [torch.empty(x.shape, dtype=x.dtype, device=DEV) for x in (q, k, q, k, w[0], w[1])]
    ws = torch.empty(stg.qk_norm_rope_backward_workspace(q, k), dtype=torch.uint8, device=DEV)

    def step():
        stg.qk_norm_rope(q, k, pos, f, *w, q_out=outs[0], k_out=outs[1])
        stg.qk_norm_rope_backward(gq, gk, q, k, pos, f, *w, dq=outs[2], dk=outs[3], dq_weight=outs[4],
                                  dk_weight=outs[5], workspace=ws)

    say("norm and rotation: eager, then captured")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    want = [x.clone() for x in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        say("replay", i)
        for x in outs:
            x.fill_(3.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_prepared_on_a_side_stream(stg):
    q, k, _, w, pos, f = make(18, 9, 4, 2, 64, 64, "f16", fused=False)
    say("prepared qk_norm_rope on a side stream")
    want = stg.qk_norm_rope(q, k, pos, f, *w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = stg.prepare(stg.qk_norm_rope, q, k, pos, f, *w, stream=side)
    got = call()
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q.mul_(0.5).add_(1)
    torch.cuda.synchronize()
    call()
    side.synchronize()
    want = stg.qk_norm_rope(q, k, pos, f, *w)
    assert torch.equal(got[0], want[0])
