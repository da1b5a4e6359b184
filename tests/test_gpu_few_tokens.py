"""qk_norm_rope where tokens have many heads or few (runs of the backward that
start inside a token, rounds that cross tokens), half layouts that exchange
elements, and attention over 8-bit pages of the depths between the usual ones.
Tolerances as in the tests of the operators themselves."""
import pytest
import torch

from gpu_util import say
from paged_util import f64
from test_gpu_norm_rope import check, make
from test_gpu_paged_attention import close, run, setup
from test_gpu_paged_chunks import ragged

pytestmark = pytest.mark.gpu

# (tokens, q heads, k heads, depth, rotary)
SHAPES = [(1, 192, 12, 128, 128), (4, 240, 10, 112, 112), (1, 112, 16, 160, 28), (2, 1, 70, 64, 48), (3, 1, 1, 32, 32),
          (17, 65, 0, 16, 12), (509, 8, 2, 64, 64), (1500, 1, 3, 40, 36), (300, 100, 1, 192, 124), (7, 33, 9, 516, 500),
          (2300, 5, 5, 24, 20), (1, 1, 1, 1024, 1024)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward_runs(stg, orc, shape, interleaved, kind):
    tokens, hq, hk, depth, rotary = shape
    q, k, _, w, pos, f = make(21, tokens, hq, hk, depth, rotary, kind)
    dq, dk = torch.randn_like(q.contiguous()), torch.randn_like(k.contiguous())
    say("qk_norm_rope_backward", shape, interleaved, kind)
    got = stg.qk_norm_rope_backward(dq, dk, q, k, pos, f, *w, interleaved=interleaved)
    for y, dw, g, x, wt in ((got[0], got[2], dq, q, w[0]), (got[1], got[3], dk, k, w[1])):
        if not x.shape[1]:
            assert bool((dw == 0).all())
            continue
        dx, bound, want, abs_dw = orc.norm_rope_backward(f64(g), f64(x), f64(wt), pos.cpu().numpy(), f.cpu().numpy(),
                                                         interleaved)
        check(y, dx, bound, kind, 1.5 * depth + 48)
        check(dw, want, abs_dw, "f32", tokens * x.shape[1] + depth / 2 + 48)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(2782, 6, 3, 192, 124), (1033, 14, 7, 128, 116), (5, 2, 1, 72, 30), (900, 1, 1, 20, 18),
                                   (40, 3, 2, 17, 2), (33, 4, 4, 1000, 998)], ids=str)
def test_exchanged_halves(stg, orc, shape, kind):
    """Halves that are no multiple of 8 elements, of which partners lie in other lanes."""
    tokens, hq, hk, depth, rotary = shape
    q, k, _, w, pos, f = make(22, tokens, hq, hk, depth, rotary, kind)
    say("qk_norm_rope", shape, kind)
    got = stg.qk_norm_rope(q, k, pos, f, *w)
    for y, x, wt in ((got[0], q, w[0]), (got[1], k, w[1])):
        want, bound = orc.norm_rope(f64(x), f64(wt), pos.cpu().numpy(), f.cpu().numpy(), False)
        check(y, want, bound, kind, depth / 2 + 24)


def test_exchange_keeps_infinities_in_their_pairs(stg):
    """Without the norm an infinity stays in its pair; what a lane reads beside it does not leak."""
    depth, rotary = 64, 28
    x = torch.ones((3, 2, depth), device="cuda")
    x[1, 1, 5] = float("inf")
    pos = torch.tensor([3, 1, 2], dtype=torch.int32, device="cuda")
    f = torch.full((rotary // 2,), 0.3, device="cuda")
    say("qk_norm_rope with an infinity")
    y, _ = stg.qk_norm_rope(x, x, pos, f, norm=False)
    bad = (~y.isfinite()).nonzero().tolist()
    assert bad == [[1, 1, 5], [1, 1, 5 + rotary // 2]]


@pytest.mark.parametrize("heads,group,depth,kind", [(15, 3, 160, "f16"), (10, 24, 32, "bf16"), (4, 2, 40, "f16"),
                                                    (2, 5, 180, "bf16"), (6, 1, 192, "bf16"), (3, 8, 64, "f16")])
def test_8_bit_pages_of_other_depths(stg, orc, heads, group, depth, kind):
    lens = ragged(depth, 45, 1900)
    _, q, kc, vc, table, lens, ks, vs = setup(depth, lens, heads * group, heads, depth, 32, kind, "e4m3")
    say("paged_attention e4m3", heads, group, depth, kind)
    out, lse = run(stg, q, kc, vc, table, lens, ks, vs)
    close(orc, out, lse, q, kc, vc, table, lens, depth ** -0.5, 0, kind, ks, vs)
