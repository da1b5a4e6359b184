"""The paged key-value cache's operators as workloads: their inputs, their plain
forms in elementary torch operations, and their definitions in 64 bits.

Five kinds of case (the key "kind"):

* attention   one new token per sequence attends to its cached keys and values;
* append      the step before it: queries and keys normalised per head and
              rotated, keys and values written into the cache's pages;
* norm_rope   the same normalisation and rotation without a cache (training);
* backward    its gradients, the weights' among them;
* fork        finished sequences freed, others forked into their rows;
* compact     live pages moved to the front of the pool.

A cache is (pages, slots, heads, depth); a sequence's pages are a row of an
int32 page table, -1 where it has none.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one user's chat: the smallest decode step, bound by latency
        dict(name="decode_one", kind="attention", batch=1, q_heads=32, heads=8, depth=128, page=16, longest=57,
             window=0, dtype="bf16", cache="bf16", empty=False),
        # a server's ordinary batch: 64 sequences of 1 .. 8192 tokens, 8 heads of 128
        dict(name="decode_ragged", kind="attention", batch=64, q_heads=32, heads=8, depth=128, page=16, longest=8192,
             window=0, dtype="bf16", cache="bf16", empty=False),
        # few users with very long contexts, the cache held in 8 bits
        dict(name="decode_long_e4m3", kind="attention", batch=8, q_heads=64, heads=8, depth=128, page=64,
             longest=131072, window=0, dtype="bf16", cache="e4m3", empty=False),
        # one key head per query head, an odd depth and page, a sliding window
        # whose left pages were freed, and some rows of the batch idle
        dict(name="decode_window_odd", kind="attention", batch=37, q_heads=12, heads=12, depth=80, page=24,
             longest=5001, window=1000, dtype="f16", cache="f16", empty=True),
        # the decode step's own append: one token per sequence, 8-bit cache, idle slots
        dict(name="append_step", kind="append", batch=64, tokens=64, q_heads=32, heads=8, depth=128, rotary=128,
             page=16, start=2000, interleaved=False, scaling="none", norm=True, weight="same", dtype="bf16",
             cache="e4m3", padded=5),
        # prefill of four prompts on top of cached prefixes, interleaved pairs, long-context frequencies
        dict(name="append_prefill", kind="append", batch=4, tokens=16384, q_heads=32, heads=8, depth=128, rotary=128,
             page=16, start=4096, interleaved=True, scaling="yarn", norm=True, weight="f32", dtype="bf16",
             cache="bf16", padded=0),
        # a training batch, an odd number of tokens, part of each head rotated
        dict(name="norm_rope_part", kind="norm_rope", tokens=8191, q_heads=16, heads=4, depth=96, rotary=64,
             interleaved=False, scaling="linear", norm=True, weight="f32", dtype="f16"),
        # gradients of a short batch in 32 bits
        dict(name="backward_short", kind="backward", tokens=509, q_heads=8, heads=2, depth=64, rotary=64,
             interleaved=True, scaling="none", norm=True, weight="f32", dtype="f32"),
        # gradients of a long batch
        dict(name="backward_long", kind="backward", tokens=16384, q_heads=32, heads=8, depth=128, rotary=128,
             interleaved=False, scaling="ntk", norm=True, weight="same", dtype="bf16"),
        # a beam step of eight hypotheses on a small cache
        dict(name="fork_beams", kind="fork", batch=8, forks=4, planes=4, page=16, heads=8, depth=128, longest=700,
             dtype="bf16"),
        # parallel sampling on a server: 128 of 256 rows refilled
        dict(name="fork_server", kind="fork", batch=256, forks=128, planes=16, page=16, heads=8, depth=128,
             longest=700, dtype="bf16"),
        # a pool half empty after many sequences ended, packed before it shrinks
        dict(name="compact_pool", kind="compact", batch=64, planes=16, pages=4096, live=2401, moves=997, page=16,
             heads=8, depth=128, dtype="bf16"),
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], spread over the logarithm, odd ones as often as even ones."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "append", "norm_rope", "backward", "fork", "compact"])
    depth = rng.choice([32, 64, 72, 80, 96, 100, 112, 128, 128, 160, 192, 256])
    heads = _spread(rng, 1, 16)
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 24])
    page = rng.choice([2, 5, 8, 16, 16, 24, 32, 64, 100, 128])
    half = rng.choice(["bf16", "f16"])
    if kind == "attention":
        batch = _spread(rng, 1, 256)
        # keys and values of at most 1 Gi elements, as the longest listed case
        most = min(131072, (1 << 29) // (batch * heads * depth))
        longest = _spread(rng, 1, max(1, most))
        return dict(kind=kind, batch=batch, q_heads=heads * group, heads=heads, depth=depth, page=page,
                    longest=longest, window=rng.choice([0, 0, 0, _spread(rng, 1, 4096)]), dtype=half,
                    cache=rng.choice([half, half, "e4m3"]), empty=rng.random() < 0.3)
    if kind == "fork":
        batch = _spread(rng, 2, 256)
        planes = min(_spread(rng, 2, 16), max(1, (1 << 28) // (batch * page * heads * depth)))
        most = max(1, min(2000, (1 << 30) // (batch * planes * heads * depth)))
        return dict(kind=kind, batch=batch, forks=rng.randint(1, batch // 2), planes=planes, page=page, heads=heads,
                    depth=depth, longest=_spread(rng, 1, most), dtype=rng.choice([half, "e4m3"]))
    if kind == "compact":
        planes = min(_spread(rng, 2, 64), max(1, (1 << 29) // (64 * page * heads * depth)))
        pages = _spread(rng, 64, max(64, min(1 << 17, (1 << 29) // (planes * page * heads * depth))))
        live = rng.randint(pages // 4, pages - pages // 4)
        moves = rng.randint(0, min(live, pages - live))
        return dict(kind=kind, batch=_spread(rng, 1, 256), planes=planes, pages=pages, live=live, moves=moves,
                    page=page, heads=heads, depth=depth, dtype=rng.choice([half, "e4m3"]))
    interleaved = rng.random() < 0.5
    rotary = depth if rng.random() < 0.6 else 2 * rng.randint(1, depth // 2)
    case = dict(kind=kind, q_heads=heads * group, heads=heads, depth=depth, rotary=rotary, interleaved=interleaved,
                scaling=rng.choice(["none", "linear", "ntk", "yarn"]), norm=rng.random() < 0.8,
                weight=rng.choice(["f32", "same"]), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    # queries and keys of at most 64 Mi elements
    most = min(20000, (1 << 26) // (heads * (group + 2) * depth))
    case["tokens"] = _spread(rng, 1, most)
    if kind == "append":
        case["dtype"] = half
        batch = rng.randint(1, min(256, case["tokens"]))
        case.update(batch=batch, page=page, start=_spread(rng, 1, max(1, min(4096, (1 << 27) // (batch * heads * depth)))),
                    cache=rng.choice([half, half, "e4m3"]), padded=rng.choice([0, case["tokens"] // 16]))
    return case


def _lengths(case):
    """The batch's lengths: spread evenly over 1 .. longest, every sixth row idle where the case says so."""
    n, longest = case["batch"], case["longest"]
    got = [max(1, -(-longest * (i + 1) // n)) for i in range(n)]
    if case.get("empty"):
        got = [0 if i % 6 == 3 else x for i, x in enumerate(got)]
    return got


def _attended(case, length):
    return min(length, case["window"]) if case["window"] else length


def _fork_lengths(case):
    """Lengths of a forking batch: as above, and no last page is full, so that every fork copies one."""
    page = case["page"]
    return [x if x % page else (x - 1 if x > 1 else x + 1) for x in _lengths(case)]


def work(case):
    kind = case["kind"]
    if kind == "attention":
        tokens = sum(_attended(case, x) for x in _lengths(case))
        d, rows = case["depth"], case["batch"] * case["q_heads"]
        pages = sum(-(-_attended(case, x) // case["page"]) for x in _lengths(case))
        return {"bytes": 2 * tokens * case["heads"] * d * _BYTES[case["cache"]] + 2 * rows * d * _BYTES[case["dtype"]]
                + 4 * rows + 4 * pages + 4 * case["batch"], "flops": 4 * tokens * case["q_heads"] * d}
    if kind in ("fork", "compact"):
        size = case["planes"] * case["page"] * case["heads"] * case["depth"] * _BYTES[case["dtype"]]
        if kind == "fork":
            return {"bytes": 2 * case["forks"] * size + 4 * case["forks"] * 2 * -(-case["longest"] // case["page"]),
                    "flops": 0}
        return {"bytes": 2 * case["moves"] * size + 12 * case["pages"] + 8 * _entries(case), "flops": 0}
    t, d, e = case["tokens"], case["depth"], _BYTES[case["dtype"]]
    qk = t * (case["q_heads"] + case["heads"]) * d
    kv = t * case["heads"] * d
    if kind == "append":
        return {"bytes": (qk + kv) * e + t * case["q_heads"] * d * e + 2 * kv * _BYTES[case["cache"]] + 12 * t,
                "flops": 10 * qk}
    return {"bytes": qk * e * (2 if kind == "norm_rope" else 3) + 4 * t, "flops": (10 if kind == "norm_rope" else 20) * qk}


# ---- inputs -----------------------------------------------------------------

def _randn(shape, dtype, gen, times=1.0):
    if dtype == torch.float8_e4m3fn:
        return _randn(shape, torch.bfloat16, gen, times).to(dtype)
    x = torch.randn(shape, dtype=dtype, device="cuda", generator=gen)
    return x if times == 1.0 else x.mul_(times)


def _table(counts, first, width, slack, gen):
    """A page table of `counts[b]` pages a row, the first first[b] of them without a page; pages in random order."""
    counts, first = (torch.tensor(x, device="cuda") for x in (counts, first))
    at = torch.arange(width, device="cuda")
    used = (at < counts[:, None]) & (at >= first[:, None])
    n = int(used.sum())
    pages = n + slack
    order = torch.randperm(pages, device="cuda", generator=gen)
    table = torch.full(used.shape, -1, dtype=torch.int32, device="cuda")
    table[used] = order[:n].to(torch.int32)
    return table, pages


def _frequencies(case):
    """Rotation frequencies (rotary / 2) and the factor on cos and sin, for four times the trained 4096 positions."""
    n, base, factor, trained = case["rotary"], 10000.0, 4.0, 4096.0
    if case["scaling"] == "ntk" and n > 2:
        base *= factor ** (n / (n - 2.0))
    f = [base ** (-2.0 * i / n) for i in range(n // 2)]
    gain = 1.0
    if case["scaling"] == "linear":
        f = [x / factor for x in f]
    elif case["scaling"] == "yarn":
        gain = 0.1 * math.log(factor) + 1.0
        at = lambda turns: n * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), n - 1)
        ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 0.001))) for i in range(n // 2)]
        f = [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)]
    return torch.tensor(f, dtype=torch.float32, device="cuda"), gain


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = random.Random(int(seed))
    kind = case["kind"]
    make = {"attention": _prepare_attention, "fork": _prepare_fork, "compact": _prepare_compact}.get(kind, _prepare_rows)
    state = make(case, gen, rng)
    state["case"] = case
    if own:
        state["calls"] = _calls(state)
    return state


def _prepare_attention(case, gen, rng):
    page, heads, d = case["page"], case["heads"], case["depth"]
    lens = _lengths(case)
    rng.shuffle(lens)
    counts = [-(-x // page) for x in lens]
    first = [(x - _attended(case, x)) // page for x in lens]  # pages that the window has left were freed
    width = max(1, -(-case["longest"] // page))
    table, pages = _table(counts, first, width, 1 + sum(counts) // 16, gen)
    cache, dtype = _TYPES[case["cache"]], _TYPES[case["dtype"]]
    scales = case["cache"] == "e4m3"
    kv = _randn((2, pages, page, heads, d), cache, gen, 16.0 if scales else 1.0)
    return {
        "q": _randn((case["batch"], case["q_heads"], d), dtype, gen, 2.0),
        "k_cache": kv[0], "v_cache": kv[1], "table": table,
        "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
        "k_scale": torch.linspace(0.05, 0.08, heads, device="cuda") if scales else None,
        "v_scale": torch.linspace(0.08, 0.05, heads, device="cuda") if scales else None,
        "scale": d ** -0.5,
    }


def _prepare_rows(case, gen, rng):
    """Rows of queries, keys and values as the projection leaves them: one tensor, a token's heads side by side."""
    t, d, hq, h = case["tokens"], case["depth"], case["q_heads"], case["heads"]
    dtype = _TYPES[case["dtype"]]
    qkv = _randn((t, hq + 2 * h, d), dtype, gen)
    freq, gain = _frequencies(case)
    state = {"q": qkv[:, :hq], "k": qkv[:, hq:hq + h], "v": qkv[:, hq + h:], "freq": freq, "gain": gain, "eps": 1e-6,
             "qw": None, "kw": None}
    if case["norm"]:
        wt = torch.float32 if case["weight"] == "f32" else dtype
        state["qw"], state["kw"] = ((1 + 0.2 * torch.randn(d, device="cuda", generator=gen)).to(wt) for _ in range(2))
    if case["kind"] == "append":
        n, page, b = -(-t // case["batch"]), case["page"], case["batch"]
        rows = torch.arange(t, device="cuda") // n
        start = torch.tensor([rng.randint(0, case["start"]) for _ in range(b)], device="cuda")
        state["positions"] = (start[rows] + torch.arange(t, device="cuda") % n).to(torch.int32)
        rows[t - case["padded"]:] = -1  # slots of a captured batch that no request fills
        state["rows"] = rows.to(torch.int32)
        width = -(-(case["start"] + n) // page)
        state["table"], pages = _table([width] * b, [0] * b, width, 1 + b, gen)
        cache = _TYPES[case["cache"]]
        kv = _randn((2, pages, page, h, d), cache, gen, 16.0 if case["cache"] == "e4m3" else 1.0)
        scales = case["cache"] == "e4m3"
        state.update(k_cache=kv[0], v_cache=kv[1], k_scale=torch.linspace(0.05, 0.08, h, device="cuda") if scales else None,
                     v_scale=torch.linspace(0.08, 0.05, h, device="cuda") if scales else None)
    else:
        state["positions"] = torch.randint(0, 16384, (t,), device="cuda", generator=gen, dtype=torch.int32)
    if case["kind"] == "backward":
        state["dq"], state["dk"] = _randn((t, hq, d), dtype, gen), _randn((t, h, d), dtype, gen)
    return state


def _meta(parts):
    """The tables of a cache as a program keeps them (one buffer) and a second buffer that a pass works on."""
    flat = torch.cat([p.reshape(-1).to(torch.int32) for p in parts.values()])
    work_on, views, at = torch.empty_like(flat), {}, 0
    for name, p in parts.items():
        views[name] = work_on[at:at + p.numel()].view(p.shape)
        at += p.numel()
    return {"given": flat, "work": work_on, **views}


def _prepare_fork(case, gen, rng):
    lens = _fork_lengths(case)
    rng.shuffle(lens)
    page = case["page"]
    counts = [-(-x // page) for x in lens]
    table, pages = _table(counts, [0] * len(lens), max(counts), case["forks"] + 1 + sum(counts) // 16, gen)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[table[table >= 0].long()] = 1
    children = rng.sample(range(case["batch"]), case["forks"])
    stay = [b for b in range(case["batch"]) if b not in set(children)]
    parents = [rng.choice(stay) for _ in children]
    state = _meta({"table": table, "lens": torch.tensor(lens, device="cuda"), "refs": refs})
    state.update(
        parents=torch.tensor(parents, dtype=torch.int32, device="cuda"),
        children=torch.tensor(children, dtype=torch.int32, device="cuda"),
        cache=_randn((case["planes"], pages, page * case["heads"] * case["depth"]), _TYPES[case["dtype"]], gen))
    return state


def _entries(case):
    return case["batch"] * (-(-case["live"] * 9 // (8 * case["batch"])) + 1)


def _prepare_compact(case, gen, rng):
    pages, live, moves = case["pages"], case["live"], case["moves"]
    low = torch.randperm(live, device="cuda", generator=gen)[: live - moves]
    high = torch.randperm(pages - live, device="cuda", generator=gen)[:moves] + live
    ids = torch.cat([low, high])[torch.randperm(live, device="cuda", generator=gen)]
    table = torch.full((_entries(case),), -1, dtype=torch.int32, device="cuda")
    table[:live] = ids.to(torch.int32)
    shared = ids[torch.randint(0, live, (live // 16,), device="cuda", generator=gen)]  # a prefix that two rows share
    table[live:live + live // 16] = shared.to(torch.int32)
    refs = torch.bincount(table[table >= 0].long(), minlength=pages)
    state = _meta({"table": table.view(case["batch"], -1), "refs": refs})
    state["cache"] = _randn((case["planes"], pages, case["page"] * case["heads"] * case["depth"]), _TYPES[case["dtype"]], gen)
    return state


# ---- one pass ---------------------------------------------------------------

def _calls(s):
    """The framework's calls on a state, prepared once as a serving loop keeps them."""
    import scatter_tile_gather_amd as stg

    case, kind = s["case"], s["case"]["kind"]
    if kind == "attention":
        s["lse"] = torch.empty((case["batch"], case["q_heads"]), dtype=torch.float32, device="cuda")
        return [stg.prepare(stg.paged_attention, s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                            scale=s["scale"], window=case["window"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                            max_len=case["longest"], lse=s["lse"])]
    if kind == "fork":
        return [stg.prepare(stg.pages_free, s["table"], s["lens"], s["refs"], s["children"]),
                stg.prepare(stg.pages_fork, s["cache"], s["table"], s["lens"], s["refs"], case["page"], s["parents"],
                            s["children"])]
    if kind == "compact":
        return [stg.prepare(stg.pages_compact, s["cache"], s["table"], s["refs"])]
    turn = dict(q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"], norm=case["norm"], interleaved=case["interleaved"],
                rope_scale=s["gain"])
    if kind == "append":
        return [stg.prepare(stg.qk_norm_rope_append, s["q"], s["k"], s["v"], s["positions"], s["freq"], s["k_cache"],
                            s["v_cache"], s["table"], rows=s["rows"], k_scale=s["k_scale"], v_scale=s["v_scale"], **turn)]
    if kind == "norm_rope":
        return [stg.prepare(stg.qk_norm_rope, s["q"], s["k"], s["positions"], s["freq"], **turn)]
    return [stg.prepare(stg.qk_norm_rope_backward, s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["freq"], **turn)]


def run(s):
    case, kind = s["case"], s["case"]["kind"]
    if kind in ("fork", "compact"):
        s["work"].copy_(s["given"])
    if own:
        for call in s["calls"]:
            got = call()
        if kind == "attention":
            return {"out": got, "lse": s["lse"]}
        if kind == "append":
            return {"q": got, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if kind == "norm_rope":
            return {"q": got[0], "k": got[1]}
        if kind == "backward":
            return {"dq": got[0], "dk": got[1], "dqw": got[2], "dkw": got[3]}
        if kind == "fork":
            return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], "cache": s["cache"]}
        return {"table": s["table"], "refs": s["refs"], "remap": got, "cache": s["cache"]}
    plain = {"attention": _plain_attention, "append": _plain_append, "norm_rope": _plain_norm_rope,
             "backward": _plain_backward, "fork": _plain_fork, "compact": _plain_compact}
    return plain[kind](s)


def _plain_attention(s):
    case, table, lens = s["case"], s["table"], s["lens"]
    page, h, d = case["page"], case["heads"], case["depth"]
    b, width = table.shape
    n, g = width * page, case["q_heads"] // h
    at = table.clamp(min=0)
    k, v = (x[at].permute(0, 3, 1, 2, 4).reshape(b, h, n, d).float() for x in (s["k_cache"], s["v_cache"]))
    q = s["q"].float().view(b, h, g, d).transpose(2, 3).contiguous()
    scores = torch.matmul(k, q) * s["scale"]
    if s["k_scale"] is not None:
        scores = scores * s["k_scale"][:, None, None]
    j = torch.arange(n, device="cuda")
    here = (j < lens[:, None]) & (table >= 0).repeat_interleave(page, 1)
    if case["window"]:
        here &= j >= lens[:, None] - case["window"]
    scores = scores.masked_fill(~here[:, None, :, None], -math.inf)
    top = scores.amax(2, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(2, keepdim=True)
    out = torch.matmul(p.transpose(2, 3).contiguous(), v) / total.clamp(min=1e-38).transpose(2, 3)
    if s["v_scale"] is not None:
        out = out * s["v_scale"][:, None, None]
    lse = (top + torch.log(total)).reshape(b, h * g)
    return {"out": out.reshape(b, h * g, d).to(s["q"].dtype), "lse": lse}


def _cos_sin(s):
    angle = s["positions"].double()[:, None] * s["freq"].double()
    return (angle.cos() * s["gain"]).float()[:, None], (angle.sin() * s["gain"]).float()[:, None]


def _rotate(x, cos, sin, interleaved):
    n = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _turned(s, x, w, cos, sin):
    x = x.float()
    if s["case"]["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
    return _rotate(x, cos, sin, s["case"]["interleaved"])


def _plain_norm_rope(s):
    cos, sin = _cos_sin(s)
    return {"q": _turned(s, s["q"], s["qw"], cos, sin).to(s["q"].dtype),
            "k": _turned(s, s["k"], s["kw"], cos, sin).to(s["k"].dtype)}


def _plain_append(s):
    cos, sin = _cos_sin(s)
    q, k, v = _turned(s, s["q"], s["qw"], cos, sin), _turned(s, s["k"], s["kw"], cos, sin), s["v"].float()
    page, pos = s["case"]["page"], s["positions"].long()
    at = s["table"][s["rows"].clamp(min=0).long(), pos // page].long()
    slot = pos % page
    if s["k_scale"] is not None:
        k = (k / s["k_scale"][:, None]).clamp(-448.0, 448.0)
        v = (v / s["v_scale"][:, None]).clamp(-448.0, 448.0)
    if s["case"]["padded"]:
        keep = s["rows"] >= 0
        at, slot, k, v = at[keep], slot[keep], k[keep], v[keep]
    s["k_cache"][at, slot] = k.to(s["k_cache"].dtype)
    s["v_cache"][at, slot] = v.to(s["v_cache"].dtype)
    return {"q": q.to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_backward(s):
    cos, sin = _cos_sin(s)
    dq, dqw = _gradient(s, s["dq"], s["q"], s["qw"], cos, sin)
    dk, dkw = _gradient(s, s["dk"], s["k"], s["kw"], cos, sin)
    return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}


def _gradient(s, g, x, w, cos, sin):
    u = _rotate(g.float(), cos, -sin, s["case"]["interleaved"])
    if not s["case"]["norm"]:
        return u.to(x.dtype), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
    xn = x * r
    uw = u * w.float()
    dx = r * (uw - xn * (uw * xn).mean(-1, keepdim=True))
    return dx.to(g.dtype), (u * xn).sum((0, 1)).to(w.dtype)


def _plain_fork(s):
    table, lens, refs, cache, page = s["table"], s["lens"], s["refs"], s["cache"], s["case"]["page"]
    parents, children = s["parents"].long(), s["children"].long()
    gone = table[children]
    refs.index_add_(0, gone.clamp(min=0).flatten(), -(gone >= 0).int().flatten())
    table[children] = -1
    lens[children] = 0
    n = lens[parents]
    full, part = n // page, n % page > 0
    order = torch.argsort((refs > 0).int(), stable=True).int()
    fresh = order[(part.cumsum(0) - 1).clamp(min=0)]
    rows = table[parents]
    j = torch.arange(table.shape[1], device="cuda")
    shared = (j < full[:, None]) & (rows >= 0)
    refs.index_add_(0, rows.clamp(min=0).flatten(), shared.int().flatten())
    refs[fresh[part].long()] = 1
    last = rows.gather(1, full[:, None].long().clamp(max=table.shape[1] - 1))[:, 0]
    table[children] = torch.where(shared, rows, torch.where((j == full[:, None]) & part[:, None], fresh[:, None], -1))
    lens[children] = n
    bits = cache.view(torch.uint8)
    bits[:, fresh[part].long()] = bits[:, last[part].long()]
    return {"table": table, "lens": lens, "refs": refs, "cache": cache}


def _plain_compact(s):
    table, refs, cache = s["table"], s["refs"], s["cache"]
    ids = torch.arange(refs.numel(), device="cuda")
    live = refs > 0
    n = live.sum()
    src, dst = (live & (ids >= n)).nonzero()[:, 0], (~live & (ids < n)).nonzero()[:, 0]
    remap = torch.where(live, ids, -1).int()
    remap[src] = dst.int()
    table.copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()], table))
    refs[dst] = refs[src]
    refs[src] = 0
    bits = cache.view(torch.uint8)
    bits[:, dst] = bits[:, src]
    return {"table": table, "refs": refs, "remap": remap, "cache": cache}


# ---- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    kind = case["kind"]
    if kind == "attention":
        return _exact_attention(s)
    if kind == "fork":
        return _exact_fork(s)
    if kind == "compact":
        return _exact_compact(s)
    return _exact_rows(s)


def _exact_attention(s):
    case = s["case"]
    page, h, d, hq = case["page"], case["heads"], case["depth"], case["q_heads"]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    out = torch.zeros((case["batch"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        at = [j for j in range(n - _attended(case, n), n) if table[b][j // page] >= 0]
        if not at:
            continue
        j = torch.tensor(at, device="cuda")
        where = s["table"][b].long()[j // page] * page + j % page
        for i in range(h):
            k = s["k_cache"].view(-1, h, d)[:, i].view(torch.uint8)[where].view(s["k_cache"].dtype).double()
            v = s["v_cache"].view(-1, h, d)[:, i].view(torch.uint8)[where].view(s["v_cache"].dtype).double()
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][i].double(), v * s["v_scale"][i].double()
            own_heads = slice(i * (hq // h), (i + 1) * (hq // h))
            z = s["q"][b, own_heads].double() @ k.t().contiguous() * case["depth"] ** -0.5
            lse[b, own_heads] = torch.logsumexp(z, 1)
            out[b, own_heads] = torch.softmax(z, 1) @ v
    return {"out": out, "lse": lse}


def _exact_rows(s):
    case = s["case"]
    n = case["rotary"] // 2
    turn = torch.polar(torch.full((1,), float(s["gain"]), dtype=torch.float64, device="cuda"),
                       torch.outer(s["positions"].double(), s["freq"].double()))  # (tokens, n): gain e^(i angle)
    first = torch.arange(n, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else n)

    def rotated(x, by):
        y = x.clone()
        z = torch.complex(x[..., first], x[..., second]) * by[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def forward(x, w):
        x = x.double()
        if case["norm"]:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.double()
        return rotated(x, turn)

    if case["kind"] != "backward":
        q, k = forward(s["q"], s["qw"]), forward(s["k"], s["kw"])
        if case["kind"] == "norm_rope":
            return {"q": q, "k": k}
        if case["cache"] == "e4m3":
            return {"q": q, "k_cache": None, "v_cache": None}
        caches = []
        pos, rows = s["positions"].long(), s["rows"].long()
        t = torch.nonzero(rows >= 0)[:, 0]
        at = s["table"].long()[rows[t], pos[t] // case["page"]] * case["page"] + pos[t] % case["page"]
        for cache, x in ((s["k_cache"], k), (s["v_cache"], s["v"].double())):
            c = cache.double()
            c.view(-1, case["heads"], case["depth"]).index_copy_(0, at, x[t])
            caches.append(c)
        return {"q": q, "k_cache": caches[0], "v_cache": caches[1]}
    got = []
    for g, x, w in ((s["dq"], s["q"], s["qw"]), (s["dk"], s["k"], s["kw"])):
        u = rotated(g.double(), turn.conj())
        if not case["norm"]:
            got.append((u, None))
            continue
        x = x.double()
        size = torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"])
        uw = u * w.double()
        inner = (uw * x).sum(-1, keepdim=True) / (case["depth"] * size * size)
        got.append(((uw - x * inner) / size, (u * x / size).sum(0).sum(0)))
    return {"dq": got[0][0], "dk": got[1][0], "dqw": got[0][1], "dkw": got[1][1]}


def _exact_fork(s):
    s["work"].copy_(s["given"])
    page = s["case"]["page"]
    table, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    for c in s["children"].tolist():
        for p in table[c]:
            if p >= 0:
                refs[p] -= 1
        table[c], lens[c] = [-1] * len(table[c]), 0
    free = [p for p, r in enumerate(refs) if r <= 0]
    src, dst = [], []
    for a, c in zip(s["parents"].tolist(), s["children"].tolist()):
        for j in range(lens[a] // page):
            table[c][j] = table[a][j]
            refs[table[a][j]] += 1
        if lens[a] % page:
            j = lens[a] // page
            table[c][j] = free.pop(0)
            refs[table[c][j]] = 1
            src.append(table[a][j])
            dst.append(table[c][j])
        lens[c] = lens[a]
    return {"table": torch.tensor(table), "lens": torch.tensor(lens), "refs": torch.tensor(refs),
            "cache": _moved(s["cache"], src, dst)}


def _moved(cache, src, dst):
    got = cache.view(torch.uint8).clone()
    old = cache.view(torch.uint8)
    for a, b in zip(src, dst):
        got[:, b] = old[:, a]
    return got.view(cache.dtype)


def _exact_compact(s):
    s["work"].copy_(s["given"])
    refs = s["refs"].tolist()
    live = [p for p, r in enumerate(refs) if r > 0]
    src = [p for p in live if p >= len(live)]
    dst = [p for p in range(len(live)) if refs[p] <= 0]
    remap = [p if r > 0 else -1 for p, r in enumerate(refs)]
    for a, b in zip(src, dst):
        remap[a], refs[b], refs[a] = b, refs[a], 0
    table = [[remap[p] if p >= 0 else p for p in row] for row in s["table"].tolist()]
    return {"table": torch.tensor(table), "refs": torch.tensor(refs), "remap": torch.tensor(remap),
            "cache": _moved(s["cache"], src, dst)}
