"""Attention over a paged cache on the GPU against the fp64 oracle.

Tolerance, u = 2^-24, N attended tokens, D depth.  A score's products are exact
in fp32 and its D terms are summed in it: off by at most 2 D u of the sum of
their magnitudes, plus 4 u of the score for the scale factors; the largest of
these over the row is delta (an absolute error of an exponent, so a relative
one of a probability).  A probability is fed as two 16-bit terms (2^-16 of it
is left, at most), exp2 and the sums of N terms are fp32.  So out is off by at
most (2 delta + 2^-16 + 4 (N + 16) u) times the average of |v|, plus half a
step of its type; lse by delta + (N + 16) u + 4 u |lse| + 2^-22 (the log)."""
import numpy as np
import pytest
import torch

from gpu_util import say
from paged_util import HALF_STEP, TINY, TYPES, U32, f64, random_cache, random_table

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def close(orc, got, lse, q, k, v, table, lens, scale, window, kind, ks=None, vs=None):
    """out and lse against the oracle, within the tolerance above."""
    kk, vv = f64(k.float()), f64(v.float())
    if ks is not None:
        kk, vv = kk * f64(ks)[:, None], vv * f64(vs)[:, None]
    # what lies in unattended slots may be NaN: the oracle never reads it
    out, want_lse, abs_out, mag = orc.paged_attention(f64(q.float()), kk, vv, table, lens, scale, window)
    depth = q.shape[2]
    n = np.maximum(np.asarray(lens), 0).max() if len(lens) else 0
    delta = (2 * depth + 4) * U32 * mag
    rel = 2 * delta + 2.0 ** -16 + 4 * (n + 16) * U32
    tol = rel[..., None] * abs_out + HALF_STEP[kind] * np.abs(out) * (1 + rel[..., None]) + TINY[kind]
    err = np.abs(f64(got.float()) - out)
    assert np.all(err <= tol), float(np.nanmax(err / np.maximum(tol, 1e-300)))
    if lse is not None:
        a = f64(lse)
        none = np.isneginf(want_lse)
        np.testing.assert_array_equal(np.isneginf(a), none)
        ltol = delta + (n + 16) * U32 + 4 * U32 * np.abs(np.where(none, 0, want_lse)) + 2.0 ** -22
        assert np.all(np.abs(a[~none] - want_lse[~none]) <= ltol[~none])


def setup(seed, lens, hq, h, depth, slots, kind, cache="same", slack=3, width=None):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    lens = np.asarray(lens, np.int32)
    width = width or max(1, -(-int(max(lens.max(), 1)) // slots))
    used = int(sum(min(width, -(-max(0, int(n)) // slots)) for n in lens))
    pages = used + slack
    ckind = kind if cache == "same" else cache
    scale = 16.0 if ckind == "e4m3" else 1.0
    kc, vc = (random_cache(g, pages, slots, h, depth, ckind, scale) for _ in range(2))
    q = (2 * torch.randn((len(lens), hq, depth), generator=g)).to(TYPES[kind])
    table = random_table(rng, lens, slots, pages, width)
    ks = vs = None
    if ckind == "e4m3":
        ks, vs = torch.linspace(0.03, 0.1, h), torch.linspace(0.2, 0.05, h)
    return rng, q, kc, vc, table, lens, ks, vs


def dev(x):
    return None if x is None else (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(DEV)


def run(stg, q, kc, vc, table, lens, ks, vs, **kw):
    lse = torch.full(q.shape[:2], 9.0, dtype=torch.float32, device=DEV)
    out = stg.paged_attention(dev(q), dev(kc), dev(vc), dev(table), dev(lens), k_scale=dev(ks), v_scale=dev(vs), lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 64, 127, 129, 300, 700]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("depth", [8, 33, 64, 72, 80, 96, 100, 128, 129, 160, 192, 200, 256])
def test_depths(stg, orc, depth, cache, kind):
    _, q, kc, vc, table, lens, ks, vs = setup(depth, LENS, 6, 2, depth, 16, kind, cache)
    say("paged_attention depth", depth, cache, kind)
    out, lse = run(stg, q, kc, vc, table, lens, ks, vs)
    close(orc, out, lse, q, kc, vc, table, lens, depth ** -0.5, 0, kind, ks, vs)


@pytest.mark.parametrize("heads,group", [(1, 1), (3, 1), (2, 5), (1, 16), (2, 17), (1, 40), (8, 4)])
@pytest.mark.parametrize("slots", [1, 5, 16, 64, 100, 1024])
def test_heads_and_pages(stg, orc, heads, group, slots):
    _, q, kc, vc, table, lens, ks, vs = setup(slots + group, LENS, heads * group, heads, 64, slots, "bf16")
    say("paged_attention", heads, "heads of", group, "slots", slots)
    out, lse = run(stg, q, kc, vc, table, lens, ks, vs, scale=0.2)
    close(orc, out, lse, q, kc, vc, table, lens, 0.2, 0, "bf16")


@pytest.mark.parametrize("window", [1, 7, 32, 100, 299, 5000])
def test_windows(stg, orc, window):
    """Only the last `window` tokens count; pages before them may be gone."""
    _, q, kc, vc, table, lens, ks, vs = setup(window, LENS, 4, 2, 128, 16, "f16")
    gone = table.copy()
    for b, n in enumerate(lens):
        gone[b, :max(0, int(n) - window) // 16] = -1
    say("paged_attention window", window)
    for t in (table, gone):
        out, lse = run(stg, q, kc, vc, t, lens, ks, vs, window=window)
        close(orc, out, lse, q, kc, vc, table, lens, 128 ** -0.5, window, "f16")


@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_holes_and_what_lies_in_them(stg, orc, cache):
    """Table entries that name no page, lengths past the table, negative
    lengths; NaN and infinity in every slot that no row attends to."""
    rng, q, kc, vc, table, lens, ks, vs = setup(3, [40, 0, 100, 64, 7, 200], 4, 2, 96, 8, "bf16", cache, slack=5)
    table[0, 1], table[2, 0], table[2, 12], table[3, :] = -1, kc.shape[0], 1 << 30, -9
    lens[4], lens[5], lens[1] = -5, 1 << 30, -1
    used = np.zeros((kc.shape[0], 8), bool)
    for b, n in enumerate(lens):
        for j in range(min(max(0, int(n)), table.shape[1] * 8)):
            if 0 <= table[b, j // 8] < kc.shape[0]:
                used[table[b, j // 8], j % 8] = True
    for c in (kc, vc):
        bad = torch.tensor([float("nan"), float("inf"), float("-inf")])[torch.randint(0, 3, (int((~used).sum()),))]
        if cache == "e4m3":
            bad = torch.full_like(bad, float("nan"))
        bits = c.view(torch.uint8 if cache == "e4m3" else torch.int16)
        fill = bad.to(c.dtype).view(bits.dtype)
        bits[torch.from_numpy(~used)] = fill[:, None, None].expand(-1, 2, 96)
    say("paged_attention with holes", cache)
    for hint in (0, 8):
        out, lse = run(stg, q, kc, vc, table, lens, ks, vs, max_len=hint)
        close(orc, out, lse, q, kc, vc, table, np.minimum(lens, 1000), 96 ** -0.5, 0, "bf16", ks, vs)
        assert bool((out[[1, 3, 4]] == 0).all()) and bool(lse[[1, 3, 4]].isneginf().all())


@pytest.mark.parametrize("kind,cache,depth,group", [("bf16", "same", 128, 4), ("f16", "e4m3", 80, 1), ("bf16", "e4m3", 256, 9),
                                                    ("f16", "same", 64, 2)])
@pytest.mark.parametrize("lens", [[5000], [1, 4999, 0], [4096, 300, 5200, 17]], ids=str)
def test_split_rows(stg, orc, lens, kind, cache, depth, group):
    """Rows long enough to be split over workgroups and joined; the hint on the
    longest row changes the split, not the result."""
    _, q, kc, vc, table, lens, ks, vs = setup(7, lens, 2 * group, 2, depth, 16, kind, cache)
    say("paged_attention, split", lens.tolist(), kind, cache, depth)
    dq, dk, dt = dev(q), dev(kc), dev(table)
    assert stg.paged_attention_workspace(dq, dk, dt) > 0
    assert stg.paged_attention_workspace(dq, dk, dt, max_len=32) == 0
    for hint in (0, 32, 600, 5200):
        out, lse = run(stg, q, kc, vc, table, lens, ks, vs, max_len=hint)
        close(orc, out, lse, q, kc, vc, table, lens, depth ** -0.5, 0, kind, ks, vs)


def test_layouts(stg, orc):
    """Caches stored head-major, keys and values side by side, queries and
    results as views, page tables as views."""
    _, q, kc, vc, table, lens, _, _ = setup(9, LENS, 6, 3, 80, 16, "bf16")
    head_major = torch.stack([kc, vc]).permute(0, 1, 3, 2, 4).contiguous().to(DEV).transpose(2, 3)
    beside = torch.cat([kc, vc], -1).to(DEV)
    apart = (kc.to(DEV), head_major[1])
    wide_q = torch.zeros((len(lens), 9, 83), dtype=torch.bfloat16, device=DEV)
    wide_q[:, 2:8, 3:] = q.to(DEV)
    room = torch.full((len(lens), 8, 90), 5.0, dtype=torch.bfloat16, device=DEV)
    tables = torch.full((len(lens), table.shape[1] + 5), 7, dtype=torch.int32, device=DEV)
    tables[:, 2:-3] = dev(table)
    for name, (k, v) in {"head-major": head_major, "side by side": (beside[..., :80], beside[..., 80:]), "unlike": apart}.items():
        say("paged_attention layout", name)
        stg.paged_attention(wide_q[:, 2:8, 3:], k, v, tables[:, 2:-3], dev(lens), out=room[:, 1:7, 4:84])
        close(orc, room[:, 1:7, 4:84], None, q, kc, vc, table, lens, 80 ** -0.5, 0, "bf16")
        room[:, 1:7, 4:84] = 5.0
        assert bool((room == 5.0).all())


def test_scores_far_apart(stg, orc):
    """Running maxima that rise late, by far, and fall short of the row's end;
    scores of -1000 and 1000 in one row."""
    _, q, kc, vc, table, lens, ks, vs = setup(11, [700, 650, 33], 2, 1, 64, 16, "bf16")
    g = torch.Generator().manual_seed(1)
    ramp = torch.linspace(-1000, 1000, 700)
    for b in range(2):
        order = ramp if b == 0 else ramp[torch.randperm(700, generator=g)]
        u = q[b, 0].float() / q[b, 0].float().square().sum()
        for j in range(int(lens[b])):
            kc[table[b, j // 16], j % 16, 0] = (u * order[j]).to(torch.bfloat16)
    say("paged_attention, scores from -1000 to 1000")
    out, lse = run(stg, q, kc, vc, table, lens, ks, vs, scale=1.0)
    close(orc, out, lse, q, kc, vc, table, lens, 1.0, 0, "bf16")


def test_not_a_number_and_infinity(stg):
    """NaN in a query, key or value shows in the rows and heads that use it and
    nowhere else; a score of -inf weighs nothing; a row of them is empty."""
    _, q, kc, vc, table, lens, ks, vs = setup(13, [40, 40, 40, 40, 40, 700], 4, 2, 64, 8, "bf16")
    clean, _ = run(stg, q, kc, vc, table, lens, ks, vs)
    q[0, 1, 3] = float("nan")
    kc[table[1, 2], 4, 1, 9] = float("nan")
    vc[table[2, 0], 0, 0, 5] = float("nan")
    q[3] = 1.0
    kc[table[3, 1], 3, 0] = float("-inf")
    q[4] = 1.0
    kc[torch.from_numpy(table[4][:5].astype(np.int64))] = float("-inf")
    q[5, 0] = float("nan")
    say("paged_attention with NaN and infinity")
    out, lse = run(stg, q, kc, vc, table, lens, ks, vs)
    nan = out.isnan()
    assert bool(nan[0, 1].all()) and int(nan[0].sum()) == 64 and bool(lse[0, 1].isnan())
    assert bool(nan[1, 2:].all()) and int(nan[1].sum()) == 128
    assert bool(nan[2, :2, 5].all()) and int(nan[2].sum()) == 2 and not bool(lse[2].isnan().any())
    assert not bool(nan[3].any())
    assert bool((out[4] == 0).all()) and bool(lse[4].isneginf().all())
    assert bool(nan[5, 0].all()) and int(nan[5].sum()) == 64
    assert torch.equal(out[0, 0], clean[0, 0]) and torch.equal(out[0, 2:], clean[0, 2:])


def test_pages_past_32_bits(stg, orc):
    """Pages whose offsets pass 2^32 bytes."""
    slots, h, depth = 16, 8, 128
    pages = (5 << 30) // (slots * h * depth * 2)
    rng, q, kc, vc, table, lens, _, _ = setup(15, [50, 33], 16, h, depth, slots, "bf16", slack=1)
    big = torch.zeros((2, pages, slots, h, depth), dtype=torch.bfloat16, device=DEV)
    n = kc.shape[0]
    big[0, -n:], big[1, -n:] = kc.to(DEV), vc.to(DEV)
    far = np.where(table >= 0, table + pages - n, table).astype(np.int32)
    say("paged_attention over a 10 GiB cache")
    out = stg.paged_attention(dev(q), big[0], big[1], dev(far), dev(lens))
    close(orc, out, None, q, kc, vc, table, lens, depth ** -0.5, 0, "bf16")


def test_empty_calls(stg):
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros((3, 8, 2, 64), dtype=torch.bfloat16, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    say("paged_attention of no rows, no pages, no table")
    assert stg.paged_attention(q, cache, cache, torch.zeros((0, 5), **i32), torch.zeros(0, **i32)).shape == (0, 4, 64)
    q = torch.ones((2, 4, 64), dtype=torch.bfloat16, device=DEV)
    lens = torch.full((2,), 9, **i32)
    for c, width in ((cache[:0], 5), (cache[:, :0], 5), (cache, 0)):
        out = stg.paged_attention(q, c, c, torch.zeros((2, width), **i32), lens)
        assert bool((out == 0).all())


def test_captured_and_prepared_calls(stg):
    """Under capture and as prepared calls, with lengths, tables and contents
    that change between the passes."""
    _, q, kc, vc, table, lens, ks, vs = setup(17, [900, 3, 411, 1200], 8, 2, 128, 16, "bf16")
    dq, dk, dv, dt, dl = dev(q), dev(kc), dev(vc), dev(table), dev(lens)
    lse = torch.zeros((4, 8), device=DEV)
    ws = torch.empty(stg.paged_attention_workspace(dq, dk, dt), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(dq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stg.paged_attention(dq, dk, dv, dt, dl, out=out, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    say("paged_attention captured and prepared")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stg.paged_attention(dq, dk, dv, dt, dl, out=out, lse=lse, workspace=ws)
    call = stg.prepare(stg.paged_attention, dq, dk, dv, dt, dl, stream=side)
    for i in range(4):
        dl.copy_(torch.from_numpy(np.roll(lens, i)).to(DEV).clamp(max=int(lens.min()) + 5) if i == 3 else dev(lens) - i)
        dq.mul_(0.9)
        torch.cuda.synchronize()
        want_lse = torch.empty_like(lse)
        want = stg.paged_attention(dq, dk, dv, dt, dl, lse=want_lse)
        out.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        got = call()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse) and torch.equal(got, want)
