"""Cases of the serving-step operators around the routed LoRA delta, and their plain forms.

A decode or prompt step of a multi-tenant server runs, beside the adapters'
deltas: the norm in front of a projection (with the residual's addition and
an 8-bit copy of its result), the shared projection itself with every
request's adapter added to it, and, after the LM head, the log probabilities
that are answered to the clients.  `run` computes one of the three:

  norm    s = x + residual;  y = s / sqrt(mean(s^2) + eps) * weight, as bf16
          and / or as e4m3 with one scale a row (the row's largest |y| / 448)
  proj    y[i] = x[i] W^T + scale[s] (x[i] A_s^T) B_s^T for s = slot[i], the
          second term absent for a negative slot; W in bf16, or x and W in
          e4m3 with a scale per row of each (the adapters read the bf16 x)
  score   per row of logits: log p(token), the token's rank, the entropy,
          and the `top` most likely tokens with their log probabilities

With `own` false in plain torch operations in 32 bits, with `own` true by the
framework's kernels.
"""
import math

import torch

own = False

QKV = "4096,1024,1024"      # Llama-3-8B's q, k and v projections (the decode workload's output)
GATE_UP = "14336,14336"     # its gate and up projections (the prompt workload's output)
EPS = 1e-5
E4M3_MAX = 448.0


def listed():
    return [
        # the norm in front of a layer's projections: one sequence being decoded
        {"name": "norm_token", "op": "norm", "n": 1, "h": 4096, "residual": True, "bf16": True, "quant": True, "pad": 0},
        # the decode batch of 256 requests
        {"name": "norm_decode", "op": "norm", "n": 256, "h": 4096, "residual": True, "bf16": True, "quant": True, "pad": 0},
        # the prompts of one prefill step, rows cut out of a wider buffer
        {"name": "norm_prompt", "op": "norm", "n": 6947, "h": 4096, "residual": True, "bf16": True, "quant": True, "pad": 64},
        # q, k and v of one sequence being decoded
        {"name": "proj_token", "op": "proj", "form": "bf16", "n": 1, "k": 4096, "slices": QKV, "slots": 32, "rank": 16,
         "route": "zipf", "bare": 0.0, "pad": 0},
        # q, k and v of the decode batch: 256 requests over 32 adapters, a few on the shared model alone
        {"name": "proj_decode", "op": "proj", "form": "bf16", "n": 256, "k": 4096, "slices": QKV, "slots": 32, "rank": 16,
         "route": "zipf", "bare": 0.05, "pad": 0},
        # the same from 8-bit activations and weights
        {"name": "proj_decode_8bit", "op": "proj", "form": "e4m3", "n": 256, "k": 4096, "slices": QKV, "slots": 32,
         "rank": 16, "route": "zipf", "bare": 0.05, "pad": 0},
        # an LM head over a ragged vocabulary for a few dozen sampled rows
        {"name": "proj_head", "op": "proj", "form": "bf16", "n": 37, "k": 4096, "slices": "32008", "slots": 8, "rank": 8,
         "route": "zipf", "bare": 0.2, "pad": 8},
        # gate and up of a prefill step: whole sequences, one adapter each
        {"name": "proj_prompt", "op": "proj", "form": "bf16", "n": 6947, "k": 4096, "slices": GATE_UP, "slots": 16,
         "rank": 64, "route": "runs", "bare": 0.0, "pad": 0},
        {"name": "proj_prompt_8bit", "op": "proj", "form": "e4m3", "n": 6947, "k": 4096, "slices": GATE_UP, "slots": 16,
         "rank": 64, "route": "runs", "bare": 0.0, "pad": 0},
        # the answer to one client's token: its log probability and five alternatives
        {"name": "score_token", "op": "score", "n": 1, "v": 128256, "dtype": "bf16", "top": 5, "masked": 0.0, "pad": 0},
        # the decode batch, the twenty alternatives that clients may ask for
        {"name": "score_decode", "op": "score", "n": 256, "v": 128256, "dtype": "bf16", "top": 20, "masked": 0.0, "pad": 0},
        # the log probabilities of prompts, 32-bit logits over a ragged vocabulary under a mask
        {"name": "score_prompt", "op": "score", "n": 6947, "v": 32003, "dtype": "fp32", "top": 1, "masked": 0.1, "pad": 5},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "proj", "proj", "score"])
    if op == "norm":
        h = 8 * _log_int(rng, 8, 2048)
        bf16 = rng.random() < 0.7
        return {"op": op, "n": _log_int(rng, 1, min(20000, 6947 * 4096 // h)), "h": h, "residual": rng.random() < 0.7,
                "bf16": bf16, "quant": not bf16 or rng.random() < 0.7, "pad": 8 * rng.choice([0, 0, 1, 17])}
    if op == "proj":
        k = 16 * _log_int(rng, 4, 896)
        slices = [8 * _log_int(rng, 2, 1792) for _ in range(rng.choice([1, 1, 2, 3]))]
        rows = int(6947 * 4096 * 28672 // (k * sum(slices)))
        return {"op": op, "form": rng.choice(["bf16", "e4m3"]), "n": _log_int(rng, 1, min(8192, rows)), "k": k,
                "slices": ",".join(str(s) for s in slices), "slots": _log_int(rng, 1, 64),
                "rank": rng.choice([8, 8, 16, 16, 24, 32, 64, 128]), "route": rng.choice(["zipf", "runs", "mixed"]),
                "bare": rng.choice([0.0, 0.05, 0.5]), "pad": 16 * rng.choice([0, 0, 1, 3])}
    v = _log_int(rng, 500, 262144)
    return {"op": op, "n": _log_int(rng, 1, min(8192, 6947 * 32003 // v)), "v": v, "dtype": rng.choice(["bf16", "fp32"]),
            "top": rng.choice([0, 1, 5, 20, 32]), "masked": rng.choice([0.0, 0.1, 0.99]), "pad": rng.choice([0, 0, 1, 56])}


# ---------------------------------------------------------------- inputs
def _rows(values, pad):
    """The same rows inside a buffer with `pad` more columns."""
    if not pad:
        return values
    wide = torch.zeros(values.shape[0], values.shape[1] + pad, dtype=values.dtype, device=values.device)
    wide[:, :values.shape[1]] = values
    return wide[:, :values.shape[1]]


def _to_8bit(t):
    """e4m3 values and one scale a row, as a quantized checkpoint and the norm hand them over."""
    scale = t.abs().amax(dim=1).clamp_min(1e-12) / E4M3_MAX
    return (t / scale[:, None]).to(torch.float8_e4m3fn), scale


def _slots(case, g):
    n, S, dev = case["n"], case["slots"], "cuda"
    if case["route"] == "zipf":        # a few popular adapters, requests in any order
        p = 1.0 / torch.arange(1, S + 1, device=dev, dtype=torch.float32)
        slot = torch.multinomial(p, n, replacement=True, generator=g)
    elif case["route"] == "runs":      # whole sequences of some hundred rows, one adapter each
        seqs = max(1, n // 434)
        owner = torch.randint(0, S, (seqs,), generator=g, device=dev)
        ends = torch.sort(torch.randint(0, n, (seqs,), generator=g, device=dev)).values
        slot = owner[torch.bucketize(torch.arange(n, device=dev), ends, right=True).clamp_max(seqs - 1)]
    else:                              # every row its own draw
        slot = torch.randint(0, S, (n,), generator=g, device=dev)
    bare = torch.rand(n, generator=g, device=dev) < case["bare"]
    return torch.where(bare, -1, slot).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    n, pad = case["n"], case["pad"]
    state = {"case": case}
    if case["op"] == "norm":
        h = case["h"]
        loud = 1.0 + 19.0 * (torch.rand(h, generator=g, device="cuda") < 0.01)   # a few channels stand out
        state["x"] = _rows((normal(n, h) * loud).bfloat16(), pad)
        state["residual"] = _rows((normal(n, h, std=2.0) * loud).bfloat16(), pad) if case["residual"] else None
        state["weight"] = (1.0 + normal(h, std=0.1)).bfloat16()
    elif case["op"] == "proj":
        k, S, R = case["k"], case["slots"], case["rank"]
        widths = [int(s) for s in case["slices"].split(",")]
        N = sum(widths)
        x, w = normal(n, k), normal(N, k, std=k ** -0.5)
        state["widths"] = widths
        state["x"] = _rows(x.bfloat16(), pad)
        if case["form"] == "e4m3":
            xq, state["x_scale"] = _to_8bit(x)
            state["xq"] = _rows(xq.view(torch.uint8), pad).view(torch.float8_e4m3fn)
            state["w"], state["w_scale"] = _to_8bit(w)
        else:
            state["w"] = w.bfloat16()
        state["a"] = normal(S, len(widths), R, k, std=k ** -0.5).bfloat16()
        state["b"] = normal(S, N, R, std=R ** -0.5).bfloat16()
        state["scale"] = 0.25 + torch.rand(S, generator=g, device="cuda")
        state["slot"] = _slots(case, g)
    else:
        v = case["v"]
        logits = normal(n, v, std=2.5)
        peaks = torch.randint(0, v, (n, 4), generator=g, device="cuda")
        logits.scatter_add_(1, peaks, 10.0 * torch.rand(n, 4, generator=g, device="cuda"))
        if case["masked"]:
            logits.masked_fill_(torch.rand(n, v, generator=g, device="cuda") < case["masked"], -math.inf)
        state["logits"] = _rows(logits.bfloat16() if case["dtype"] == "bf16" else logits, pad)
        # most answered tokens are likely ones; some rows (a prompt's first, padding) ask for none
        other = torch.randint(0, v, (n,), generator=g, device="cuda")
        pick = torch.rand(n, generator=g, device="cuda")
        token = torch.where(pick < 0.7, peaks[:, 0], other)
        state["tokens"] = torch.where(pick > 0.95, -1, token).to(torch.int32)
    return state


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"norm": _plain_norm, "proj": _plain_proj, "score": _plain_score}[case["op"]](case, state)


def _run_own(case, state):
    from tenant_lora_serving_amd import step
    if case["op"] == "norm":
        r = step.rms_norm(state["x"], state["weight"], EPS, residual=state["residual"], bf16=case["bf16"],
                          quant=case["quant"])
        return {"y": r.y, "residual": r.residual, "q": r.q, "q_scale": r.q_scale}
    # one workspace for every step, as a server keeps it
    if case["op"] == "proj":
        if "ws" not in state:
            state["ws"] = step.linear_workspace(case["n"], case["k"], sum(state["widths"]), len(state["widths"]),
                                                case["rank"])
        return step.lora_linear(state["x"], state["w"], state["a"], state["b"], state["scale"], state["widths"],
                                state["slot"], xq=state.get("xq"), x_scale=state.get("x_scale"),
                                w_scale=state.get("w_scale"), ws=state["ws"])
    if "ws" not in state:
        state["ws"] = step.logprobs_workspace(case["n"], case["v"], case["top"])
    r = step.token_logprobs(state["logits"], state["tokens"], case["top"], ws=state["ws"])
    return {"logprob": r.logprob, "rank": r.rank, "entropy": r.entropy, "top_ids": r.top_ids,
            "top_logprobs": r.top_logprobs}


def _plain_norm(case, state):
    s = state["x"].float()
    if case["residual"]:
        s = s + state["residual"].float()
    y = s * torch.rsqrt((s * s).mean(dim=1, keepdim=True) + EPS) * state["weight"].float()
    out = {"y": y.bfloat16() if case["bf16"] else None, "residual": s.bfloat16() if case["residual"] else None,
           "q": None, "q_scale": None}
    if case["quant"]:
        scale = y.abs().amax(dim=1) / E4M3_MAX
        out["q"] = torch.where(scale[:, None] > 0, y / scale[:, None], torch.zeros_like(y)).to(torch.float8_e4m3fn)
        out["q_scale"] = scale
    return out


def _plain_proj(case, state):
    x, a, b = state["x"].float(), state["a"].float(), state["b"].float()
    S, L, R, k = a.shape
    if case["form"] == "e4m3":
        y = (state["xq"].float() @ state["w"].float().T) * state["x_scale"][:, None] * state["w_scale"][None, :]
    else:
        y = x @ state["w"].float().T
    # every adapter's shrink on every row, all but the row's own set to zero
    mine = (state["slot"][:, None] == torch.arange(S, device=x.device)[None, :]).float() * state["scale"][None, :]
    xa = (x @ a.reshape(S * L * R, k).T).reshape(-1, S, L, R) * mine[:, :, None, None]
    parts = b.split(state["widths"], dim=1)
    delta = [xa[:, :, l].reshape(-1, S * R) @ p.transpose(1, 2).reshape(S * R, -1) for l, p in enumerate(parts)]
    return (y + torch.cat(delta, dim=1)).bfloat16()


def _plain_score(case, state):
    z, tokens = state["logits"].float(), state["tokens"].long()
    open_ = z > -math.inf                                # a masked token; a row may have no other
    m = z.amax(dim=1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    total = torch.exp(z - m).sum(dim=1, keepdim=True)
    logp = torch.where(open_, z - m - torch.log(total), -math.inf)
    entropy = -(torch.exp(logp) * torch.where(open_, logp, 0.0)).sum(dim=1)
    given = tokens >= 0
    at = tokens.clamp_min(0)[:, None]
    logprob = torch.where(given, logp.gather(1, at)[:, 0], torch.zeros_like(entropy))
    rank = torch.where(given, 1 + (z > z.gather(1, at)).sum(dim=1), torch.zeros_like(tokens))
    top = case["top"]
    best = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top]   # ties: the lowest index first
    best_logp = logp.gather(1, best)
    ids = torch.where(best_logp > -math.inf, best, -1)
    return {"logprob": logprob, "rank": rank.int(), "entropy": entropy, "top_ids": ids.int() if top else None,
            "top_logprobs": best_logp if top else None}


# ---------------------------------------------------------------- the least a pass has to do
def _present(case):
    """Expected number of adapters that at least one row names."""
    n, S = case["n"] * (1.0 - case["bare"]), case["slots"]
    if case["route"] == "zipf":
        total = sum(1.0 / i for i in range(1, S + 1))
        return sum(1.0 - (1.0 - 1.0 / i / total) ** n for i in range(1, S + 1))
    draws = max(1, case["n"] // 434) if case["route"] == "runs" else n
    return S * (1.0 - (1.0 - 1.0 / S) ** draws)


def work(case):
    n = case["n"]
    if case["op"] == "norm":
        h = case["h"]
        reads = 2 * n * h * (2 if case["residual"] else 1) + 2 * h
        writes = n * h * (2 * case["bf16"] + 2 * case["residual"] + case["quant"]) + 4 * n * case["quant"]
        return {"bytes": reads + writes, "flops": 6 * n * h}
    if case["op"] == "proj":
        k, R, L = case["k"], case["rank"], case["slices"].count(",") + 1
        N = sum(int(s) for s in case["slices"].split(","))
        rows, adapters = n * (1.0 - case["bare"]), _present(case)
        size = 1 if case["form"] == "e4m3" else 2
        moved = size * (n * k + N * k) + (2 * rows * k + 4 * (n + N) if size == 1 else 0)
        moved += 2 * adapters * R * (L * k + N) + 2 * n * N + 4 * n
        return {"bytes": moved, "flops": 2.0 * n * N * k + 2.0 * rows * R * (L * k + N)}
    v = case["v"]
    return {"bytes": n * v * (2 if case["dtype"] == "bf16" else 4) + n * (16 + 8 * case["top"]), "flops": 6 * n * v}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "norm":
        s = state["x"].double()
        if case["residual"]:
            s += state["residual"].double()
        length = torch.linalg.vector_norm(s, dim=1, keepdim=True)
        y = s / torch.sqrt(length ** 2 / case["h"] + EPS) * state["weight"].double()
        scale = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / E4M3_MAX
        q = y / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
        return {"y": y if case["bf16"] else None, "residual": s if case["residual"] else None,
                "q": q if case["quant"] else None, "q_scale": scale if case["quant"] else None}
    if case["op"] == "proj":
        x = state["x"].double()
        if case["form"] == "e4m3":
            xd = state["xq"].double() * state["x_scale"].double()[:, None]
            y = xd @ (state["w"].double() * state["w_scale"].double()[:, None]).T
        else:
            y = x @ state["w"].double().T
        for s in state["slot"].unique().tolist():       # adapter by adapter, on its own rows
            if s < 0:
                continue
            rows = (state["slot"] == s).nonzero()[:, 0]
            lo = 0
            for l, width in enumerate(state["widths"]):
                xa = x[rows] @ state["a"][s, l].double().T
                part = xa @ state["b"][s, lo:lo + width].double().T * state["scale"][s].double()
                y[rows, lo:lo + width] += part
                lo += width
        return y
    z, tokens = state["logits"].double(), state["tokens"].long()
    logp = torch.where(z == -math.inf, z, torch.log_softmax(z, dim=1))
    entropy = torch.special.entr(logp.exp()).sum(dim=1)
    place = torch.arange(case["v"], device=z.device)
    hit = place[None, :] == tokens[:, None]
    logprob = torch.where(hit, logp, torch.zeros_like(logp)).sum(dim=1)
    mine = torch.where(hit, z, torch.full_like(z, -math.inf)).amax(dim=1, keepdim=True)
    rank = torch.where(tokens >= 0, 1 + (z > mine).sum(dim=1), 0)
    ids, left = [], z.clone()
    for _ in range(case["top"]):                        # the largest left, at its lowest place
        big = left.amax(dim=1, keepdim=True)
        at = torch.where(left == big, place[None, :], case["v"]).amin(dim=1)
        ids.append(torch.where(big[:, 0] > -math.inf, at, -1))
        left.scatter_(1, at[:, None], -math.inf)
    best = torch.stack(ids, dim=1) if ids else None
    best_logp = None
    if ids:
        best_logp = torch.where(best >= 0, logp.gather(1, best.clamp_min(0)), torch.full_like(logp[:, :1], -math.inf))
    return {"logprob": logprob, "rank": rank.int(), "entropy": entropy,
            "top_ids": best.int() if ids else None, "top_logprobs": best_logp}
