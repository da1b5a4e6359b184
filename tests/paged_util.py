"""Inputs shared by the paged-cache tests: caches, page tables and the values that codes stand for."""
import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
# half a rounding step, relative
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
# half the step of the smallest subnormals, absolute
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}
U32 = 2.0 ** -24


def f64(t) -> np.ndarray:
    """A tensor's values in fp64 on the host."""
    return t.detach().to("cpu").double().numpy()


def random_cache(gen, pages, slots, heads, depth, kind, scale=1.0):
    """(pages, slots, heads, depth) on the host in the cache's type."""
    x = torch.randn((pages, slots, heads, depth), generator=gen) * scale
    return x.to(TYPES[kind])


def random_table(rng, lens, slots, pages, width):
    """Page table with distinct random pages for every row's tokens, -1 elsewhere."""
    order = rng.permutation(pages)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(lens):
        c = min(width, -(-max(0, n) // slots))
        table[b, :c] = order[at:at + c]
        at += c
    assert at <= pages
    return table
