"""Attention over long batches (tokens of all rows cut into chunks), joins of
every kind, and the wide strides of qk_norm_rope.  Tolerances as in the tests
of the operators themselves."""
import numpy as np
import pytest
import torch

from gpu_util import say
from paged_util import TYPES, f64
from test_gpu_norm_rope import check, make
from test_gpu_paged_attention import DEV, close, run, setup

pytestmark = pytest.mark.gpu


def ragged(seed, rows, longest):
    """Lengths of every kind: none, one, short, around a chunk's end, long."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 400 if rows < 100 else 60, rows)
    lens[rng.permutation(rows)[:rows // 4]] = 0
    lens[rng.permutation(rows)[:2]] = longest, longest - 255
    lens[-3:] = 0, 1, 0
    return lens


# (rows, cache heads, group, depth, type, cache): plans by row and by chunk
# (more rows than chunks), joins of 16 and of 4 waves, pairs of heads, heads
# that do not pair, more queries than a tile, one chunk per workgroup only
CASES = [(5, 8, 4, 128, "bf16", "same"), (40, 8, 4, 128, "bf16", "e4m3"), (300, 4, 1, 256, "bf16", "same"),
         (130, 3, 2, 64, "f16", "same"), (70, 2, 17, 80, "f16", "e4m3"), (33, 64, 1, 32, "bf16", "same"),
         (600, 16, 1, 96, "f16", "same")]


@pytest.mark.parametrize("rows,heads,group,depth,kind,cache", CASES)
def test_ragged_batches(stg, orc, rows, heads, group, depth, kind, cache):
    lens = ragged(rows, rows, 2500)
    _, q, kc, vc, table, lens, ks, vs = setup(rows, lens, heads * group, heads, depth, 16, kind, cache)
    say("paged_attention chunks", rows, heads, group, depth, kind, cache)
    out, lse = run(stg, q, kc, vc, table, lens, ks, vs)
    close(orc, out, lse, q, kc, vc, table, lens, depth ** -0.5, 0, kind, ks, vs)


@pytest.mark.parametrize("depth,kind,cache", [(128, "bf16", "same"), (128, "f16", "e4m3"), (64, "f16", "same"),
                                              (100, "bf16", "same")])
def test_hints_and_room(stg, orc, depth, kind, cache):
    """A wide table lets the host expect long rows (pairs of heads), a small hint short ones; the result is the same
    attention, also for rows longer than the hint."""
    lens = ragged(9, 64, 3000)
    _, q, kc, vc, table, lens, ks, vs = setup(depth, lens, 16, 8, depth, 8, kind, cache, width=1024)
    for hint in (0, 3000, 8):
        say("paged_attention", depth, kind, cache, "hint", hint)
        out, lse = run(stg, q, kc, vc, table, lens, ks, vs, max_len=hint)
        close(orc, out, lse, q, kc, vc, table, lens, depth ** -0.5, 0, kind, ks, vs)


def test_batches_without_tokens(stg):
    """Chunks of nothing: every row is written."""
    _, q, kc, vc, table, lens, _, _ = setup(4, [3000] * 5, 8, 2, 64, 16, "bf16")
    for rows in (lens * 0, lens * 0 - 1):
        say("paged_attention of empty rows with room for long ones")
        out, lse = run(stg, q, kc, vc, table, rows.astype(np.int32), None, None)
        assert bool((out == 0).all()) and bool(lse.isneginf().all())


def test_pages_that_are_not_there_across_chunks(stg, orc):
    """Holes of whole chunks within a row, and a row of holes only."""
    _, q, kc, vc, table, lens, _, _ = setup(5, [4000, 900, 2000], 16, 8, 128, 16, "f16")
    table[0, 5:200] = -1
    table[1] = 1 << 30
    kc[table[2, 3], 2], vc[table[2, 3], 2] = float("nan"), float("nan")
    table[2, 3] = -7
    say("paged_attention with holes across chunks")
    out, lse = run(stg, q, kc, vc, table, lens, None, None)
    assert bool((out[1] == 0).all()) and bool(lse[1].isneginf().all())
    close(orc, out, lse, q, kc, vc, table, lens, 128 ** -0.5, 0, "f16")


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_infinite_values_stay_infinite(stg, kind):
    """An attended value of infinity gives infinity, in its dimension alone, and opposite ones NaN."""
    _, q, kc, vc, table, lens, _, _ = setup(6, [40, 3000, 40], 4, 2, 64, 8, kind)
    vc[table[0, 1], 3, 0, 7] = float("inf")
    vc[table[1, 9], 0, 1, 20] = float("-inf")
    vc[table[2, 0], 0, 0, 1], vc[table[2, 4], 5, 0, 1] = float("inf"), float("-inf")
    q[:] = 0.125  # no probability vanishes
    say("paged_attention with infinite values", kind)
    out, lse = run(stg, q, kc, vc, table, lens, None, None)
    assert bool((out[0, :2, 7] == float("inf")).all()) and int(out[0].isinf().sum()) == 2
    assert bool((out[1, 2:, 20] == float("-inf")).all()) and int(out[1].isinf().sum()) == 2
    assert bool(out[2, :2, 1].isnan().all()) and int(out.isnan().sum()) == 2 and bool(lse.isfinite().all())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_many_small_terms_beside_a_large_one(stg, orc, kind):
    """One token far above 30,000 equal ones: they weigh as much as it does."""
    n = 30000
    _, q, kc, vc, table, lens, _, _ = setup(7, [n], 1, 1, 64, 64, kind)
    kc[:] = 0
    q[:] = 1
    kc[table[0, 3], 5, 0] = float(np.log(n) / 8)  # score ln n
    say("paged_attention of a large term and many small ones", kind)
    out, lse = run(stg, q, kc, vc, table, lens, None, None, scale=0.125)
    close(orc, out, lse, q, kc, vc, table, lens, 0.125, 0, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_far_apart(stg, orc, kind, interleaved):
    """Token strides past 2^23 bytes, where offsets no longer fit 24-bit products."""
    tokens, hq, hk, depth = 5, 3, 2, 96
    q0, k0, _, w, pos, f = make(11, tokens, hq, hk, depth, 64, kind)
    stride = (1 << 23) // q0.element_size() + 8
    room = torch.zeros(tokens * stride, dtype=TYPES[kind], device=DEV)
    q = room.as_strided((tokens, hq, depth), (stride, depth, 1))
    k = room.as_strided((tokens, hk, depth), (stride, depth, 1), 4096)
    q.copy_(q0), k.copy_(k0)
    say("qk_norm_rope with far rows", kind, interleaved)
    got = stg.qk_norm_rope(q, k, pos, f, *w, interleaved=interleaved)
    for y, x, wt in ((got[0], q0, w[0]), (got[1], k0, w[1])):
        want, bound = orc.norm_rope(f64(x), f64(wt), pos.cpu().numpy(), f.cpu().numpy(), interleaved)
        check(y, want, bound, kind, depth / 2 + 24)
    near = stg.qk_norm_rope_backward(q0, k0, q0, k0, pos, f, *w, interleaved=interleaved)
    far = stg.qk_norm_rope_backward(q, k, q, k, pos, f, *w, interleaved=interleaved)
    for a, b in zip(near, far):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shape", [(60000, 1, 1, 64, 64), (60000, 2, 1, 16, 10), (50001, 3, 1, 24, 24)], ids=str)
def test_long_backward_runs(stg, orc, shape):
    """Waves that walk over more tokens than they hold angles for."""
    tokens, hq, hk, depth, rotary = shape
    q, k, _, w, pos, f = make(12, tokens, hq, hk, depth, rotary, "f32")
    dq, dk = torch.randn_like(q.contiguous()), torch.randn_like(k.contiguous())
    say("qk_norm_rope_backward", shape)
    got = stg.qk_norm_rope_backward(dq, dk, q, k, pos, f, *w)
    for y, dw, g, x, wt in ((got[0], got[2], dq, q, w[0]), (got[1], got[3], dk, k, w[1])):
        dx, bound, want, abs_dw = orc.norm_rope_backward(f64(g), f64(x), f64(wt), pos.cpu().numpy(), f.cpu().numpy())
        check(y, dx, bound, "f32", 1.5 * depth + 48)
        check(dw, want, abs_dw, "f32", tokens * x.shape[1] + depth / 2 + 48)


def test_codes_at_every_scale(stg):
    """e4m3 codes are those of the fp32 quotient, whatever the scale: ordinary, tiny, huge, zero, infinite."""
    heads = 6
    scales = torch.tensor([0.07, 3e-39, 1e-31, 2e38, 0.0, float("inf")])
    g = torch.Generator().manual_seed(13)
    v = (torch.randn((50, heads, 16), generator=g) * torch.exp(4 * torch.randn((50, heads, 16), generator=g))).to(torch.bfloat16)
    v[0, :, 0], v[0, :, 1], v[0, :, 2] = 0.0, float("inf"), float("nan")
    cache = torch.zeros((2, 50, 1, heads, 16), dtype=torch.float8_e4m3fn, device=DEV)
    table = torch.arange(50, dtype=torch.int32, device=DEV)[:, None].contiguous()
    q = torch.ones((50, heads, 16), dtype=torch.bfloat16, device=DEV)
    say("qk_norm_rope_append at odd scales")
    stg.qk_norm_rope_append(q, q, v.to(DEV), torch.zeros(50, dtype=torch.int32, device=DEV), torch.ones(8, device=DEV),
                            cache[0], cache[1], table, v_scale=scales.to(DEV))
    want = (v.float() / scales[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    got = cache[1, :, 0].cpu().float()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~got.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("pages", [65536, 65537, 70000])
def test_large_pools(stg, orc, pages):
    """Pools that scan workgroups count themselves, and larger ones counted first: reserve, fork, compact."""
    rng = np.random.default_rng(pages)
    refs = np.zeros(pages, np.int32)
    live = np.sort(rng.permutation(pages)[:pages // 2])
    refs[live] = 1
    table = np.full((4, pages // 8 + 600), -1, np.int32)
    table[:, :pages // 8] = rng.permutation(live)[:4 * (pages // 8)].reshape(4, -1)
    lens = np.full(4, pages // 8 * 3 - 1, np.int32)
    table[3], lens[3] = -1, 0
    cache = rng.integers(0, 1 << 30, (1, pages, 4)).astype(np.int32)
    c, t, n, r = (torch.from_numpy(x.copy()).to(DEV) for x in (cache, table, lens, refs))
    more = np.array([500, 0, 7, 3], np.int32)
    say("pools of", pages)
    stg.pages_reserve(t, n, torch.from_numpy(more).to(DEV), r, 3)
    orc.pages_reserve(table, lens, more, refs, 3)
    table[3], t[3] = -1, -1
    i32 = dict(dtype=torch.int32, device=DEV)
    stg.pages_fork(c, t, n, r, 3, torch.tensor([1], **i32), torch.tensor([3], **i32))
    orc.pages_fork(cache, table, lens, refs, 3, np.array([1], np.int32), np.array([3], np.int32))
    remap = stg.pages_compact(c, t, r)
    want = orc.pages_compact(cache, table, refs)
    for a, b in ((remap, want), (t, table), (n, lens), (r, refs), (c, cache)):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
