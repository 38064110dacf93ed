"""Cases of a serving step's attention over a paged cache, and their plain forms.

Between the q, k and v projections of a step and its output projection every
new token's keys and values go into the cache and its queries read what is
there.  `run` computes one of the two:

  append  q and k turned by their positions' angles,
              pair (a, b) at angle t -> (a cos t - b sin t, b cos t + a sin t),
          the pairs being halves of the turned columns or neighbours; k and v
          put into their places of the cache, in bf16 or, divided by a scale a
          head, in e4m3; the turned q returned
  attend  per row and head of q: o = sum_j p_j v_j, p = softmax(scale q k_j),
          over the keys of the prefix that the row's request shares with
          others (each prefix is in the cache once) and of the request itself;
          with `causal` the rows of a request are its last tokens and see no
          later key; lse = ln sum exp(scale q k_j) beside it

With `own` false in plain torch operations in 32 bits, with `own` true by the
framework's kernels.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
BASE = 500000.0


def _append(name, n, heads, kv, dim, rot, cache, layout, **more):
    case = {"op": "append", "n": n, "heads": heads, "kv": kv, "dim": dim, "rot": rot, "neighbours": False, "cache": cache,
            "layout": layout, "page": 16, "idle": 0, "pad": 0, **more}
    return {"name": name, **case} if name else case


def _attend(name, requests, rows, keys, heads, kv, dim, cache, layout, **more):
    lo, hi = keys
    case = {"op": "attend", "requests": requests, "rows": rows, "keys_lo": lo, "keys_hi": hi, "heads": heads, "kv": kv,
            "dim": dim, "cache": cache, "layout": layout, "page": 16, "causal": True, "idle": 0, "prefixes": 0,
            "prefix_lo": 0, "prefix_hi": 0, "bare": 0, "lse": False, "pad": 0, **more}
    return {"name": name, **case} if name else case


def listed():
    return [
        # one sequence being decoded: a token's keys and values appended (32 query heads over 8 of 128, as all of
        # this framework's decode and prompt workloads have)
        _append("append_token", 1, 32, 8, 128, 128, "bf16", "apart"),
        # the decode batch of 256 requests, four of them places kept free in a captured step, an 8-bit cache
        _append("append_decode", 256, 32, 8, 128, 128, "e4m3", "heads", idle=4),
        # the prompts of one prefill step
        _append("append_prompt", 6947, 32, 8, 128, 128, "bf16", "joint", pad=64),
        # one sequence being decoded at some thousand tokens
        _attend("attend_token", 1, 0, (4999, 4999), 32, 8, 128, "bf16", "apart"),
        # the decode batch: requests of very different age, a few places free
        _attend("attend_decode", 256, 0, (64, 4096), 32, 8, 128, "bf16", "apart", idle=4),
        # the same from an 8-bit cache
        _attend("attend_decode_8bit", 256, 0, (64, 4096), 32, 8, 128, "e4m3", "apart", idle=4),
        # a few dozen requests to a model whose query heads have keys of their own, on pages of an odd size
        _attend("attend_decode_heads", 37, 0, (10, 3001), 12, 12, 64, "bf16", "heads", page=24, lse=True),
        # the decode batch where the requests of a tenant share its instructions, some requests without any
        _attend("attend_prefix", 256, 0, (16, 512), 32, 8, 128, "bf16", "apart", prefixes=8, prefix_lo=700, prefix_hi=6000,
                bare=11),
        # 64 questions to one long document
        _attend("attend_prefix_document", 64, 0, (8, 100), 32, 8, 128, "e4m3", "joint", prefixes=1, prefix_lo=20011,
                prefix_hi=20011, lse=True),
        # whole prompts of very different length
        _attend("attend_prompt", 9, 6947, (0, 0), 32, 8, 128, "bf16", "joint", pad=64),
        # pieces of prompts at the end of long conversations that share their instructions
        _attend("attend_chunk", 4, 2048, (4000, 24000), 32, 8, 128, "bf16", "apart", prefixes=2, prefix_lo=900, prefix_hi=1500),
        # a decoder's queries to an encoder's states of another length
        _attend("attend_cross", 13, 1111, (300, 1500), 16, 16, 64, "bf16", "heads", page=32, causal=False, lse=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    dim = rng.choice([64, 80, 96, 112, 128, 128, 128, 256])
    kv, each = rng.choice([1, 2, 4, 8, 8, 12]), rng.choice([1, 2, 3, 4, 4, 8, 16])
    kv = min(kv, max(1, 64 // each))
    common = {"page": rng.choice([1, 8, 16, 16, 24, 32, 64, 128, 256]), "pad": 16 * rng.choice([0, 0, 1, 5])}
    cache, layout = rng.choice(["bf16", "e4m3"]), rng.choice(["apart", "joint", "heads"])
    kind = rng.choice(["append", "token", "token", "prefix", "prefix", "rows", "rows"])
    if kind == "append":
        n = _log_int(rng, 1, 8192 * 48 * 128 // (max(48, kv * (each + 2)) * max(dim, 128)))
        return _append(None, n, kv * each, kv, dim, 16 * rng.choice([0, dim // 16, dim // 16, rng.randint(1, dim // 16)]),
                       cache, layout, neighbours=rng.random() < 0.4, idle=rng.choice([0, n // 16]), **common)
    common["lse"] = rng.random() < 0.3
    row = kv * dim * 4                                   # bytes of a key and its value in bf16
    if kind == "rows":
        n = _log_int(rng, 2, 4096)
        requests = _log_int(rng, 1, min(n, 32))
        # pairs of rows and keys, and the plain form's scores
        most = int(min(24000, 2.0e9 * 64 / (n * kv * each * (dim / 128)) / 8, 2e9 / row / requests,
                       1.5e9 / (kv * each * requests * min(n, 4.0 * n / requests))))
        causal = rng.random() < 0.7
        hi = _log_int(rng, 1, max(2, most))
        lo = _log_int(rng, 1, hi)
        if causal and rng.random() < 0.4:
            lo = hi = 0
    else:
        n, causal = 0, True
        requests = _log_int(rng, 1, 512)
        hi = _log_int(rng, 8, max(16, min(32768, int(1.2e9 / row / requests))))
        lo = _log_int(rng, 1, hi)
        common["idle"] = rng.choice([0, 0, requests // 9])
    if kind == "prefix" or (kind == "rows" and rng.random() < 0.3):
        most = max(16, min(24000, int(1.2e9 / row / requests), int(2.0e9 * 8 / (max(n, requests) * kv * each))))
        if n:
            most = min(most, max(16, int(1e9 / (kv * each * requests * min(n, 4.0 * n / requests)))))
        common["prefixes"] = _log_int(rng, 1, requests)
        common["prefix_hi"] = _log_int(rng, 16, most)
        common["prefix_lo"] = _log_int(rng, 1, common["prefix_hi"])
        common["bare"] = rng.choice([0, 0, (requests - common["prefixes"]) // 5])
    return _attend(None, requests, n, (lo, hi), kv * each, kv, dim, cache, layout, causal=causal, **common)


# ---------------------------------------------------------------- lengths
def _spread(count, lo, hi):
    """`count` lengths from lo to hi, even over their logarithm."""
    return [int(round(lo * (hi / lo) ** ((i + 0.5) / count))) if lo > 0 else lo + (hi - lo) * (2 * i + 1) // (2 * count)
            for i in range(count)]


def _share(total, count, spread):
    """`total` cut into `count` parts of at least 1, the largest about `spread` times the smallest."""
    w = _spread(count, 1000, 1000 * spread)
    parts = [1 + (total - count) * x // sum(w) for x in w]
    parts[-1] += total - sum(parts)
    return parts


def _lengths(case):
    """(rows, keys) of every request and the prefixes' lengths, in no order."""
    live = case["requests"] - case["idle"]
    rows = _share(case["rows"], live, 20) if case["rows"] else [1] * live
    keys = _spread(live, case["keys_lo"], case["keys_hi"])
    if case["causal"]:                                   # the rows' own keys are in the cache too
        keys = [k + r for k, r in zip(keys, rows)]
    pairs = list(zip(rows, keys)) + [(0 if case["rows"] else 1, 0)] * case["idle"]
    return pairs, _spread(case["prefixes"], case["prefix_lo"], case["prefix_hi"]) if case["prefixes"] else []


def _groups(case):
    """Sizes of the groups of requests that share a prefix."""
    return _share(case["requests"] - case["bare"], case["prefixes"], 4)


# ---------------------------------------------------------------- inputs
def _pool(case, pages, normal):
    """The cache of keys and of values, [pages, page, kv, dim], as a server may lay it out, and the scales of e4m3."""
    page, kv, dim = case["page"], case["kv"], case["dim"]
    if case["layout"] == "joint":                        # a page's keys and values side by side
        both = normal(pages, 2, page, kv, dim)
    elif case["layout"] == "heads":                      # a head's tokens side by side
        both = normal(2, pages, kv, page, dim)
    else:
        both = normal(2, pages, page, kv, dim)
    if case["cache"] == "e4m3":
        both = (both / 0.02).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    else:
        both = both.bfloat16()
    if case["layout"] == "joint":
        return both[:, 0], both[:, 1]
    if case["layout"] == "heads":
        return both[0].transpose(1, 2), both[1].transpose(1, 2)
    return both[0], both[1]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    host = random.Random(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    heads, kv, dim, page, pad = case["heads"], case["kv"], case["dim"], case["page"], case["pad"]
    state = {"case": case}
    if case["op"] == "append":
        n, rot = case["n"], case["rot"]
        # the projection's result, q, k and v side by side, in a buffer that may be wider
        qkv = normal(n, (heads + 2 * kv) * dim + pad).bfloat16()
        state["q"] = qkv[:, :heads * dim].unflatten(1, (heads, dim))
        state["k"] = qkv[:, heads * dim:(heads + kv) * dim].unflatten(1, (kv, dim))
        state["v"] = qkv[:, (heads + kv) * dim:(heads + 2 * kv) * dim].unflatten(1, (kv, dim))
        pages = 2 * -(-n // page) + 64 // page + 1
        state["k_cache"], state["v_cache"] = _pool(case, pages, normal)
        place = torch.randperm(pages * page, generator=g, device="cuda")[:n]
        free = torch.randperm(n, generator=g, device="cuda")[:case["idle"]]
        place[free] = -1
        state["place"] = place.to(torch.int32)
        state["positions"] = state["rotation"] = None
        if rot:
            # cosines and sines of positions up to 131072, from angles in 64 bits
            angles = torch.arange(131072, device="cuda", dtype=torch.float64)[:, None] \
                * BASE ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)[None, :]
            state["rotation"] = torch.cat([angles.cos(), angles.sin()], dim=1).float()
            state["positions"] = torch.randint(0, 131072, (n,), generator=g, device="cuda").to(torch.int32)
        values = 2 * kv
    else:
        pairs, prefix_lens = _lengths(case)
        host.shuffle(pairs)
        host.shuffle(prefix_lens)
        rows, lens = [r for r, _ in pairs], [k for _, k in pairs]
        n = sum(rows)
        wide = max(1, -(-max(lens) // page))
        wide_prefix = -(-max(prefix_lens, default=0) // page)
        own_pages, pre_pages = sum(-(-k // page) for k in lens), sum(-(-k // page) for k in prefix_lens)
        order = torch.randperm(own_pages + pre_pages, generator=g, device="cuda").to(torch.int32)
        state["k_cache"], state["v_cache"] = _pool(case, max(1, own_pages + pre_pages), normal)
        state["lens"] = ints(lens)
        state["pages"] = _table(order, ints([-(-k // page) for k in lens]), wide, 0)
        state["starts"], state["most_rows"] = None, 1
        if case["rows"]:
            state["starts"], state["most_rows"] = ints([sum(rows[:i]) for i in range(len(rows) + 1)]), max(rows)
        state["most_keys"] = wide * page
        state["prefix_lens"] = None
        if prefix_lens:
            sizes = _groups(case)
            first = host.randint(0, case["bare"])        # requests without a prefix before the groups and behind them
            state["prefix_starts"] = ints([first + sum(sizes[:i]) for i in range(len(sizes) + 1)])
            state["prefix_lens"] = ints(prefix_lens)
            state["prefix_pages"] = _table(order, ints([-(-k // page) for k in prefix_lens]), wide_prefix, own_pages)
        state["q"] = normal(n, heads * dim + pad, std=1.5).bfloat16()[:, :heads * dim].unflatten(1, (heads, dim))
        values = 2
    # an 8-bit cache holds values over a scale a head
    state["k_scale"] = state["v_scale"] = None
    if case["cache"] == "e4m3":
        scales = 0.02 * (0.75 + 0.5 * torch.rand(2, kv, generator=g, device="cuda"))
        state["k_scale"], state["v_scale"] = scales[0], scales[1]
    return state


def _table(order, counts, wide, first):
    """Rows of page numbers, taken from `order` from `first` on; -1 behind a row's last page."""
    ends = first + counts.cumsum(0)
    at = (ends - counts)[:, None] + torch.arange(max(wide, 1), device=order.device)[None, :]
    return torch.where(at < ends[:, None], order[at.clamp_max(max(order.numel() - 1, 0))] if order.numel() else -1,
                       -1).to(torch.int32)


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return (_plain_append if case["op"] == "append" else _plain_attend)(case, state)


def _run_own(case, state):
    from tenant_lora_serving_amd import step
    if case["op"] == "append":
        q = step.kv_append(state["k"], state["v"], state["k_cache"], state["v_cache"], state["place"], q=state["q"],
                           positions=state["positions"], rotation=state["rotation"], neighbours=case["neighbours"],
                           k_scale=state["k_scale"], v_scale=state["v_scale"])
        return {"q": q, "k_cache": state["k_cache"], "v_cache": state["v_cache"]}
    prefix = None
    if case["prefixes"]:
        prefix = step.Prefixes(state["prefix_pages"], state["prefix_lens"], state["prefix_starts"])
    # one workspace for every step, as a server keeps it
    if "ws" not in state:
        state["ws"] = step.attention_workspace(state["q"].shape[0], case["heads"], case["kv"], case["dim"],
                                               prefixes=case["prefixes"] > 0)
    r = step.paged_attention(state["q"], state["k_cache"], state["v_cache"], state["pages"], state["lens"],
                             starts=state["starts"], max_rows=state["most_rows"], causal=case["causal"], prefix=prefix,
                             k_scale=state["k_scale"], v_scale=state["v_scale"], lse=case["lse"], ws=state["ws"])
    return {"out": r.out, "lse": r.lse}


def _turn(x, case, state):
    """x [n, heads, dim] in 32 bits, its first `rot` columns turned."""
    rot = case["rot"]
    if not rot:
        return x
    table = state["rotation"][state["positions"].long()][:, None, :]
    cos, sin = table[..., :rot // 2], table[..., rot // 2:]
    if case["neighbours"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _bytes(t):
    """The same cache with its 8-bit values as plain bytes, which torch can index."""
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _plain_append(case, state):
    page = case["page"]
    q, k = _turn(state["q"].float(), case, state), _turn(state["k"].float(), case, state)
    live = state["place"] >= 0
    place = state["place"][live].long()
    for cache, values, scale in ((state["k_cache"], k, state["k_scale"]),
                                 (state["v_cache"], state["v"].float(), state["v_scale"])):
        if scale is not None:
            values = (values / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        _bytes(cache)[place // page, place % page] = _bytes(values[live].to(cache.dtype))
    return {"q": q.bfloat16(), "k_cache": state["k_cache"], "v_cache": state["v_cache"]}


def _gather(cache, scale, table, keys):
    """Every request's keys or values in 32 bits, [requests, kv, keys, dim]."""
    page = cache.shape[1]
    j = torch.arange(keys, device=cache.device)
    at = table[:, j // page].long().clamp_min(0)
    x = _bytes(cache)[at, (j % page)[None, :]].view(cache.dtype).float()
    if scale is not None:
        x = x * scale[:, None]
    return x.transpose(1, 2)


def _plain_attend(case, state):
    q, lens, dim = state["q"], state["lens"].long(), case["dim"]
    dev, n, B, kv = q.device, q.shape[0], lens.shape[0], case["kv"]
    each, T = case["heads"] // kv, state["most_rows"]
    starts = state["starts"].long() if state["starts"] is not None else torch.arange(B + 1, device=dev)
    rows = starts[1:] - starts[:-1]
    # the rows of every request side by side
    t = torch.arange(T, device=dev)[None, :]
    at = (starts[:-1, None] + t).clamp_max(n - 1)
    x = q[at].float().reshape(B, T, kv, each, dim).permute(0, 2, 1, 3, 4).reshape(B, kv, T * each, dim)
    caches = [(state["k_cache"], state["k_scale"]), (state["v_cache"], state["v_scale"])]
    k, v = (_gather(c, s, state["pages"], state["most_keys"]) for c, s in caches)
    j = torch.arange(state["most_keys"], device=dev)
    seen = (lens[:, None] - rows[:, None] + t + 1).minimum(lens[:, None]) if case["causal"] else lens[:, None].expand(B, T)
    open_ = j[None, None, :] < seen[:, :, None]
    if state["prefix_lens"] is not None:
        groups = state["prefix_lens"].shape[0]
        group = torch.bucketize(torch.arange(B, device=dev), state["prefix_starts"].long(), right=True) - 1
        inside = (group >= 0) & (group < groups)
        group = group.clamp(0, groups - 1)
        most = state["prefix_pages"].shape[1] * case["page"]
        k, v = (torch.cat([_gather(c, s, state["prefix_pages"][group], most), own_], dim=2)
                for (c, s), own_ in zip(caches, (k, v)))
        shared = torch.where(inside, state["prefix_lens"].long()[group], 0)
        there = torch.arange(most, device=dev)[None, :] < shared[:, None]
        open_ = torch.cat([there[:, None, :].expand(B, T, most), open_], dim=2)
    s = x @ k.transpose(2, 3) * dim ** -0.5
    s = s.masked_fill_(~open_[:, None, :, None, :].expand(B, 1, T, each, -1).reshape(B, 1, T * each, -1), -math.inf)
    m = s.amax(dim=3, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = s.sub_(m).exp_()
    total = p.sum(dim=3, keepdim=True)
    o = p @ v / torch.where(total > 0, total, torch.ones_like(total))
    # back to the batch's rows
    i = torch.arange(n, device=dev)
    b = torch.bucketize(i, starts, right=True) - 1
    o = o.reshape(B, kv, T, each, dim).permute(0, 2, 1, 3, 4).reshape(B, T, kv * each, dim)[b, i - starts[b]]
    lse = None
    if case["lse"]:
        lse = (m + total.log()).reshape(B, kv, T, each).permute(0, 2, 1, 3).reshape(B, T, kv * each)[b, i - starts[b]]
    return {"out": o.bfloat16(), "lse": lse}


# ---------------------------------------------------------------- the least a pass has to do
def work(case):
    heads, kv, dim = case["heads"], case["kv"], case["dim"]
    size = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        n, live = case["n"], case["n"] - case["idle"]
        moved = 4 * n * heads * dim + live * 2 * kv * dim * (2 + size) + 4 * n
        moved += n * (4 + 4 * case["rot"]) if case["rot"] else 0
        return {"bytes": moved, "flops": 3 * (n * heads + live * kv) * case["rot"] + 1}
    pairs, prefix_lens = _lengths(case)
    n = sum(r for r, _ in pairs)
    keys = sum(k for _, k in pairs) + sum(prefix_lens)
    moved = keys * kv * dim * 2 * size + n * heads * (4 * dim + 4 * case["lse"]) + 4 * -(-keys // case["page"])
    met = sum(r * k - (r * (r - 1) // 2 if case["causal"] else 0) for r, k in pairs)
    # (which prefix a group has, and how many rows, goes by the seed: on average)
    if prefix_lens:
        met += n * (1.0 - case["bare"] / case["requests"]) * sum(prefix_lens) / len(prefix_lens)
    return {"bytes": moved, "flops": 4.0 * dim * heads * met}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    return _exact_append(case, state) if case["op"] == "append" else _exact_attend(case, state)


def _exact_append(case, state):
    rot, page = case["rot"], case["page"]
    q, k, v = state["q"].double(), state["k"].double(), state["v"].double()
    if rot:
        half = rot // 2
        turn = torch.complex(*state["rotation"].double().split(half, dim=1))[state["positions"].long()][:, None, :]
        i = torch.arange(half, device=q.device)
        first, second = (2 * i, 2 * i + 1) if case["neighbours"] else (i, i + half)
        for x in (q, k):
            z = torch.complex(x[:, :, first], x[:, :, second]) * turn
            x[:, :, first], x[:, :, second] = z.real, z.imag
    out = {"q": q}
    for name, x in (("k", k), ("v", v)):
        if state[name + "_scale"] is not None:
            x = (x / state[name + "_scale"].double()[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        cache = state[name + "_cache"].double()
        flat = cache.reshape(-1, *cache.shape[2:]).clone()
        keep = state["place"] >= 0
        flat.index_copy_(0, state["place"][keep].long(), x[keep])
        out[name + "_cache"] = flat.view(cache.shape)
    return out


def _exact_attend(case, state):
    q, page, kv, dim = state["q"].double(), case["page"], case["kv"], case["dim"]
    each = case["heads"] // kv
    lens = state["lens"].tolist()
    starts = state["starts"].tolist() if state["starts"] is not None else list(range(len(lens) + 1))
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    group = [-1] * len(lens)
    if case["prefixes"]:
        ends, prefix_lens = state["prefix_starts"].tolist(), state["prefix_lens"].tolist()
        for p in range(len(prefix_lens)):
            group[ends[p]:ends[p + 1]] = [p] * (ends[p + 1] - ends[p])

    def read(cache, scale, table, length):
        pages = table[:-(-length // page)].long()
        x = _bytes(cache)[pages].view(cache.dtype).double().flatten(0, 1)[:length]
        return x if scale is None else x * scale.double()[None, :, None]

    for b, length in enumerate(lens):
        r0, r1 = starts[b], starts[b + 1]
        keys = [read(state["k_cache"], state["k_scale"], state["pages"][b], length)]
        values = [read(state["v_cache"], state["v_scale"], state["pages"][b], length)]
        before = 0
        if group[b] >= 0:
            before = prefix_lens[group[b]]
            table = state["prefix_pages"][group[b]]
            keys.insert(0, read(state["k_cache"], state["k_scale"], table, before))
            values.insert(0, read(state["v_cache"], state["v_scale"], table, before))
        if r0 == r1 or before + length == 0:
            continue
        keys, values = torch.cat(keys), torch.cat(values)
        hidden = None
        if case["causal"] and r1 - r0 > 1:
            hidden = torch.ones(r1 - r0, before + length, dtype=torch.bool, device=q.device)
            hidden = hidden.triu(before + length - (r1 - r0) + 1)
        for h in range(kv):
            for e in range(each):
                s = (q[r0:r1, h * each + e] @ keys[:, h].T) / math.sqrt(dim)
                if hidden is not None:
                    s.masked_fill_(hidden, -math.inf)
                out[r0:r1, h * each + e] = torch.softmax(s, dim=1) @ values[:, h]
                lse[r0:r1, h * each + e] = torch.logsumexp(s, dim=1)
    return {"out": out, "lse": lse if case["lse"] else None}
