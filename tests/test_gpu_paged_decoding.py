"""The decode loop of examples/paged_decoding.py: its operators together."""
import importlib.util
import os

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda:0")


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decoding.py")
    spec = importlib.util.spec_from_file_location("paged_decoding", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def started(example, n=21):
    d = example.Decoder(rows=4)
    g = torch.Generator(device="cuda:0").manual_seed(3)
    tokens = torch.randint(0, 512, (n, 4), generator=g, **I32)
    on = torch.tensor([1, 0, 1, 0], **I32)
    for t in tokens:
        d.step(t, on)
    return d, tokens[0], on


def test_main_runs(example):
    say("paged decoding")
    example.main()


def test_a_fork_continues_as_its_parent(example):
    d, tok, on = started(example)
    d.fork(torch.tensor([0], **I32), torch.tensor([3], **I32))
    on[3], tok[3] = 1, tok[0]
    say("fork, then the same tokens")
    for _ in range(15):  # past the page that both write on
        logits = d.step(tok, on)
        assert torch.equal(logits[0], logits[3])
        tok = logits.argmax(1).to(torch.int32)
    # then other tokens: the shared pages stay the parent's
    before = d.step(tok, on)
    other = tok.clone()
    other[3] = (tok[3] + 1) % 512
    assert not torch.equal(d.step(other, on)[0], before[0]) and int(d.refs.max()) == 2


def test_compaction_moves_nothing_that_shows(example):
    a, tok, on = started(example)
    b, _, _ = started(example)
    for d in (a, b):  # row 0's pages become holes in the pool
        d.fork(torch.tensor([0], **I32), torch.tensor([1], **I32))
        d.free(torch.tensor([0], **I32))
    on = torch.tensor([0, 1, 1, 0], **I32)
    b.compact()
    live = int((b.refs > 0).sum())
    assert bool((b.refs[:live] > 0).all())
    say("the same steps with and without compaction")
    for _ in range(20):
        x, y = a.step(tok, on), b.step(tok, on)
        assert torch.equal(x[1:3], y[1:3])
        tok = x.argmax(1).to(torch.int32)
