"""The training objectives' operators as a user's program calls them, each
with a plain form in elementary torch operations beside it.

Four operators:
  logprobs    log probability of each token under its row of logits
  policy      clipped policy loss with a KL term: loss and gradient of the logits
  preference  preference loss of (chosen, rejected) pairs: loss and gradient
  route       a mixture-of-experts router: top-k choice, gates, per-expert
              counts and balance loss; with backward, the logits' gradient too

A case is a dict of sizes and options; ``own`` selects the framework's
operators (True) or the plain forms (False) in ``run``.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# Tokens come in spans of this many, each a response followed by what is not
# trained on (masked): the next prompt, or padding.
SPAN = 512
# The most bytes of logits in a case (the largest listed one has them).
MOST_BYTES = 8192 * 131072 * 2


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the log probabilities of a few tokens just sampled, one decoding step
        {"name": "logprobs_step", "op": "logprobs", "tokens": 8, "vocab": 32000, "dtype": "bf16",
         "live": 1.0, "pad": 0, "temperature": 1.0},
        # a reference model's pass over a batch of rollouts, large vocabulary
        {"name": "logprobs_reference", "op": "logprobs", "tokens": 4096, "vocab": 131072,
         "dtype": "bf16", "live": 0.75, "pad": 0, "temperature": 1.0},
        # one short response, no KL term, summed
        {"name": "policy_short", "op": "policy", "tokens": 48, "vocab": 32000, "dtype": "bf16",
         "live": 1.0, "pad": 0, "temperature": 1.0, "beta": 0.0, "mean": False},
        # a micro-batch of rollouts on the 32000-word vocabulary
        {"name": "policy_batch", "op": "policy", "tokens": 4096, "vocab": 32000, "dtype": "bf16",
         "live": 0.75, "pad": 0, "temperature": 1.0, "beta": 0.04, "mean": True},
        # a large micro-batch on a large vocabulary
        {"name": "policy_large", "op": "policy", "tokens": 8192, "vocab": 131072, "dtype": "bf16",
         "live": 1.0, "pad": 0, "temperature": 1.0, "beta": 0.04, "mean": True},
        # fp32 logits, odd vocabulary in rows of an odd stride, sampling temperature
        {"name": "policy_odd_fp32", "op": "policy", "tokens": 777, "vocab": 50021, "dtype": "fp32",
         "live": 0.9, "pad": 3, "temperature": 0.8, "beta": 0.1, "mean": True},
        # two short pairs
        {"name": "preference_short", "op": "preference", "pairs": 2, "length": 48, "vocab": 32000,
         "dtype": "bf16", "live": 1.0, "pad": 0, "temperature": 1.0, "beta": 0.1, "kind": 0,
         "average": False, "smoothing": 0.0},
        # a batch of pairs with masked prompts
        {"name": "preference_batch", "op": "preference", "pairs": 16, "length": 384,
         "vocab": 32000, "dtype": "bf16", "live": 0.75, "pad": 0, "temperature": 1.0,
         "beta": 0.1, "kind": 0, "average": False, "smoothing": 0.1},
        # fp32, odd vocabulary and stride, squared loss of length-averaged ratios
        {"name": "preference_odd_fp32", "op": "preference", "pairs": 5, "length": 301,
         "vocab": 65537, "dtype": "fp32", "live": 0.9, "pad": 2, "temperature": 1.0, "beta": 0.2,
         "kind": 1, "average": True, "smoothing": 0.0},
        # serving: the choice of a few tokens, forward only
        {"name": "route_step", "op": "route", "tokens": 8, "experts": 32, "top_k": 4,
         "dtype": "bf16", "score": 0, "renorm": True, "bias": False, "sequences": 1, "live": 1.0,
         "backward": False},
        # training: the 32-expert layer, softmax gates, both directions
        {"name": "route_batch", "op": "route", "tokens": 8192, "experts": 32, "top_k": 4,
         "dtype": "bf16", "score": 0, "renorm": True, "bias": False, "sequences": 1, "live": 0.9,
         "backward": True},
        # training: 256 experts, sigmoid scores with a choice bias, ragged sequences
        {"name": "route_large", "op": "route", "tokens": 65536, "experts": 256, "top_k": 8,
         "dtype": "fp32", "score": 1, "renorm": True, "bias": True, "sequences": 33, "live": 1.0,
         "backward": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["logprobs", "policy", "preference", "route"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    live = rng.choice([1.0, 0.9, 0.75, 0.5])
    if op == "route":
        experts = _log_int(rng, 2, 512)
        backward = rng.random() < 0.7
        tokens = _log_int(rng, 1, 65536 if backward else 16384)
        return {"op": op, "tokens": tokens, "experts": experts,
                "top_k": rng.randint(1, min(8, experts)), "dtype": dtype,
                "score": rng.randint(0, 1), "renorm": rng.random() < 0.7,
                "bias": rng.random() < 0.5, "sequences": _log_int(rng, 1, 64), "live": live,
                "backward": backward}
    vocab = _log_int(rng, 1000, 200000)
    if rng.random() < 0.5:
        vocab = max(1024, vocab // 128 * 128)
    pad = rng.choice([0, 0, 0, 1, 5, 64])
    rows = min(8192, MOST_BYTES // 2 // ((vocab + pad) * (2 if dtype == "bf16" else 4)))
    rest = {"vocab": vocab, "dtype": dtype, "live": live, "pad": pad,
            "temperature": rng.choice([1.0, 1.0, 0.7]), "beta": rng.choice([0.02, 0.1, 0.3])}
    if op == "preference":
        pairs = _log_int(rng, 1, 24)
        return {"op": op, "pairs": pairs, "length": _log_int(rng, 2, max(2, min(512, rows // pairs // 2))),
                **rest, "kind": rng.randint(0, 1), "average": rng.random() < 0.5,
                "smoothing": rng.choice([0.0, 0.1])}
    case = {"op": op, "tokens": _log_int(rng, 1, rows), **rest}
    if op == "logprobs":
        del case["beta"]
    else:
        case["beta"] = rng.choice([0.0, 0.04, 0.2])
        case["mean"] = rng.random() < 0.7
    return case


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """Sequence lengths of a preference case (2 * pairs of them: the chosen,
    then the rejected), ragged; with three pairs or more one is empty."""
    n, top = 2 * case["pairs"], case["length"]
    got = [max(1, top - (top * ((7 * s) % 11)) // 22) for s in range(n)]
    if case["pairs"] >= 3:
        got[1] = 0
    return got


def _seq_starts(case):
    """Starts of a route case's sequences: ragged cuts of the token axis, one
    empty sequence among three or more."""
    n, t = case["sequences"], case["tokens"]
    cuts = [t * (s * n + (s * s) % n) // (n * n) for s in range(n)] + [t]
    if n >= 3:
        cuts[1] = cuts[2]
    return [0] + sorted(cuts[1:])


def _kept(case):
    """Tokens at the head of each span that are not masked."""
    return int(round(SPAN * case["live"]))


def _masked(case, tokens):
    """How many of the tokens are masked: the tail of each span."""
    kept = _kept(case)
    return tokens - (tokens // SPAN * kept + min(tokens % SPAN, kept))


def _tokens(case):
    return sum(_lengths(case)) if case["op"] == "preference" else case["tokens"]


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _logprobs64(x, y, inv_t):
    """Log probabilities of y under rows of x, in 64 bits, some rows at a time."""
    out = torch.empty(x.shape[0], dtype=torch.float64, device=x.device)
    step = max(1, (1 << 27) // max(1, x.shape[1]))
    for r in range(0, x.shape[0], step):
        z = x[r:r + step].double() * inv_t
        out[r:r + step] = z.gather(1, y[r:r + step, None]).squeeze(1) - torch.logsumexp(z, 1)
    return out


def _prepare_logits(case, seed, state):
    g = _generator(seed)
    tokens, vocab = _tokens(case), case["vocab"]
    wide = torch.randn(tokens, vocab + case["pad"], generator=g, device="cuda",
                       dtype=DTYPES[case["dtype"]]).mul_(2.5)
    logits = wide[:, :vocab]
    targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    # the sampled word is mostly a likely one
    rows = torch.arange(tokens, device="cuda")
    logits[rows, targets] += (9.0 + 3.0 * torch.randn(tokens, generator=g, device="cuda")).to(wide.dtype)
    live = rows % SPAN < _kept(case)
    state.update(logits=logits, inv_t=1.0 / case["temperature"])
    if case["op"] == "logprobs":
        state["targets"] = torch.where(live, targets, -100)
        return
    lp = _logprobs64(logits, targets, state["inv_t"])
    noise = torch.randn(2, tokens, generator=g, device="cuda", dtype=torch.float64)
    state["targets"] = torch.where(live, targets, -100)
    state["weights"] = (0.5 + torch.rand(tokens, generator=g, device="cuda")) * live
    state["ref_logp"] = (lp + 0.2 * noise[0]).float()
    if case["op"] == "policy":
        # ratios spread over the clipping range; none within 1e-3 of its ends,
        # where rounding alone decides the side
        ratio = torch.exp(0.15 * noise[1])
        for end in (1.0 - CLIP[0], 1.0 + CLIP[1]):
            ratio = torch.where((ratio - end).abs() < 1e-3, ratio + 2.5e-3, ratio)
        state["old_logp"] = (lp - torch.log(ratio)).float()
        state["advantages"] = torch.randn(tokens, generator=g, device="cuda")
    else:
        lengths = _lengths(case)
        state["seq_starts"] = torch.tensor(np.cumsum([0] + lengths), device="cuda")


def _prepare_route(case, seed, state):
    g = _generator(seed)
    tokens, experts = case["tokens"], case["experts"]
    dt = DTYPES[case["dtype"]]

    def rows(n):
        return (1.5 * torch.randn(n, experts, generator=g, device="cuda")).to(dt)

    logits = rows(tokens)
    bias = None
    if case["bias"]:
        bias = 0.05 * torch.randn(experts, generator=g, device="cuda")
        # where two scores in the choice differ by rounding alone, draw the row again
        at = torch.arange(tokens, device="cuda")
        for _ in range(20):
            x = logits[at].double()
            key = (torch.sigmoid(x) if case["score"] else torch.softmax(x, 1)) + bias.double()
            top = torch.sort(key, 1, descending=True).values[:, :case["top_k"] + 1]
            at = at[(top[:, :-1] - top[:, 1:]).amin(1) < 2e-6] if top.shape[1] > 1 else at[:0]
            if not at.numel():
                break
            logits[at] = rows(at.numel())
    live = torch.arange(tokens, device="cuda") % SPAN < _kept(case)
    state.update(logits=logits, bias=bias, live=live.to(torch.uint8) if case["live"] < 1 else None)
    state["seq_starts"] = torch.tensor(_seq_starts(case), device="cuda") if case["sequences"] > 1 else None
    if case["backward"]:
        state["d_gates"] = 1e-3 * torch.randn(tokens, case["top_k"], generator=g, device="cuda")


CLIP = (0.2, 0.28)    # the policy ratio is clipped to [1 - 0.2, 1 + 0.28]
SCALE = 0.5           # e.g. one of two accumulated micro-batches
MARGIN = 0.3          # preference margin
ROUTE_SCALE = 2.5     # factor on the gates
BALANCE = 0.01        # weight of the balance loss


def prepare(case, seed):
    state = {"case": case}
    if case["op"] == "route":
        _prepare_route(case, seed, state)
    else:
        _prepare_logits(case, seed, state)
    if own:
        from fsdp_buffer_layout_gb300 import objectives
        tokens, inv_t = _tokens(case), state.get("inv_t")
        dt = DTYPES[case["dtype"]]
        if case["op"] == "logprobs":
            state["call"] = objectives.TokenLogprobs(tokens, case["vocab"], dtype=dt, inv_temperature=inv_t)
        elif case["op"] == "policy":
            state["call"] = objectives.PolicyLoss(
                tokens, case["vocab"], dtype=dt, clip_low=CLIP[0], clip_high=CLIP[1],
                kl_beta=case["beta"], inv_temperature=inv_t, scale=SCALE, mean=case["mean"])
        elif case["op"] == "preference":
            state["call"] = objectives.PreferenceLoss(
                case["pairs"], tokens, case["vocab"], dtype=dt,
                kind=("sigmoid", "squared")[case["kind"]], beta=case["beta"],
                smoothing=case["smoothing"], margin=MARGIN, average=case["average"],
                inv_temperature=inv_t, scale=SCALE)
        else:
            state["call"] = objectives.Router(
                tokens, case["experts"], case["top_k"], dtype=dt,
                score=("softmax", "sigmoid")[case["score"]], renorm=case["renorm"],
                route_scale=ROUTE_SCALE, balance=BALANCE, sequences=case["sequences"])
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_logprobs(s):
    return {"logp": s["call"](s["logits"], s["targets"])}


def _own_policy(s):
    stats, logp, grad = s["call"](s["logits"], s["targets"], s["old_logp"], s["advantages"],
                                  ref_logp=s["ref_logp"], weights=s["weights"])
    return {"stats": stats, "logp": logp, "grad": grad}


def _own_preference(s):
    stats, rewards, logp, grad = s["call"](s["logits"], s["targets"], s["seq_starts"],
                                           ref_logp=s["ref_logp"], weights=s["weights"])
    return {"stats": stats, "rewards": rewards, "logp": logp, "grad": grad}


def _own_route(s):
    idx, gates, counts, loss = s["call"].forward(s["logits"], bias=s["bias"], live=s["live"],
                                                 seq_starts=s["seq_starts"])
    out = {"idx": idx, "gates": gates, "counts": counts, "loss": loss}
    if "d_gates" in s:
        out["grad"] = s["call"].backward(s["logits"], s["d_gates"], live=s["live"],
                                         seq_starts=s["seq_starts"])
    return out


def _plain_softmax(s):
    """Probabilities, log probabilities of the targets and the live tokens."""
    x = s["logits"].float() * s["inv_t"]
    x = x - x.amax(1, keepdim=True)
    e = torch.exp(x)
    total = e.sum(1, keepdim=True)
    live = s["targets"] >= 0
    if s.get("weights") is not None:
        live = live & (s["weights"] != 0)
    at = s["targets"].clamp(min=0)[:, None]
    logp = torch.where(live, (x.gather(1, at) - torch.log(total)).squeeze(1), 0.0)
    return e / total, logp, live, at


def _plain_grad(s, p, at, coef):
    """coef_t (1[v = target_t] - p) / temperature in the logits' type."""
    grad = p * -coef[:, None]
    grad.scatter_add_(1, at, coef[:, None])
    return (grad * s["inv_t"]).to(s["logits"].dtype)


def _plain_logprobs(s):
    return {"logp": _plain_softmax(s)[1]}


def _plain_policy(s):
    case = s["case"]
    p, logp, live, at = _plain_softmax(s)
    w = torch.where(live, s["weights"], 0.0)
    total = w.sum()
    n = total if case["mean"] else torch.ones_like(total)
    n = torch.where(n == 0, 1.0, n)
    ratio = torch.exp(logp - s["old_logp"])
    free = ratio * s["advantages"]
    held = ratio.clamp(1.0 - CLIP[0], 1.0 + CLIP[1]) * s["advantages"]
    u = s["ref_logp"] - logp
    kl = torch.expm1(u) - u
    policy = SCALE * (w * torch.where(live, -torch.minimum(free, held), 0.0)).sum() / n
    kl_sum = SCALE * (w * torch.where(live, kl, 0.0)).sum() / n
    slope = torch.where(free <= held, -free, 0.0) - case["beta"] * torch.expm1(u)
    coef = torch.where(live, SCALE * w / n * slope, 0.0)
    stats = torch.stack([policy + case["beta"] * kl_sum, policy, kl_sum, total])
    if not case["beta"]:
        stats = torch.stack([policy, policy, torch.zeros_like(policy), total])
    return {"stats": stats, "logp": logp, "grad": _plain_grad(s, p, at, coef)}


def _plain_preference(s):
    case = s["case"]
    pairs, starts = case["pairs"], s["seq_starts"]
    p, logp, live, at = _plain_softmax(s)
    w = torch.where(live, s["weights"], 0.0)
    rows = torch.arange(logp.numel(), device=logp.device)
    member = ((rows >= starts[:-1, None]) & (rows < starts[1:, None])).float()
    ratio = (member * (w * (logp - s["ref_logp"]))).sum(1)
    length = (member * w).sum(1) if case["average"] else torch.ones_like(ratio)
    length = torch.where(length == 0, 1.0, length)
    ratio = ratio / length
    h = ratio[:pairs] - ratio[pairs:]
    if case["kind"] == 0:
        z = case["beta"] * h - MARGIN
        tail = torch.log1p(torch.exp(-z.abs()))
        good, bad = z.clamp(max=0) - tail, (-z).clamp(max=0) - tail
        loss = -(1 - case["smoothing"]) * good - case["smoothing"] * bad
        slope = case["beta"] * (torch.sigmoid(z) - (1 - case["smoothing"]))
    else:
        loss = (h - 1 / (2 * case["beta"])) ** 2
        slope = 2 * (h - 1 / (2 * case["beta"]))
    per_seq = SCALE / pairs * torch.cat([slope, -slope]) / length
    coef = (member * per_seq[:, None]).sum(0) * w
    stats = torch.stack([SCALE * loss.mean(), case["beta"] * h.mean()])
    return {"stats": stats, "rewards": case["beta"] * ratio, "logp": logp,
            "grad": _plain_grad(s, p, at, coef)}


def _plain_route(s):
    case = s["case"]
    k, experts = case["top_k"], case["experts"]
    x = s["logits"].float()
    tokens = x.shape[0]
    live = torch.ones(tokens, dtype=torch.bool, device=x.device) if s["live"] is None else s["live"] != 0
    if case["score"]:
        sc = torch.sigmoid(x)
        z = sc.sum(1, keepdim=True) + 1e-20
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        sc = e / e.sum(1, keepdim=True)
        z = torch.ones_like(sc[:, :1])
    q = sc / z
    key = x if s["bias"] is None else sc + s["bias"]
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    picked = sc.gather(1, idx)
    down = picked.sum(1, keepdim=True) + 1e-20 if case["renorm"] else torch.ones_like(z)
    gates = torch.where(live[:, None], ROUTE_SCALE * picked / down, 0.0)
    chosen = torch.zeros_like(x).scatter_(1, idx, 1.0) * live[:, None]
    starts = s["seq_starts"]
    if starts is None:
        starts = torch.tensor([0, tokens], device=x.device)
    rows = torch.arange(tokens, device=x.device)
    member = ((rows >= starts[:-1, None]) & (rows < starts[1:, None]) & live).float()
    n = member @ chosen                 # whole numbers below 2^24: exact
    length = member.sum(1)
    full = (length > 0).float()
    safe = torch.where(length > 0, length, 1.0)
    per = full * BALANCE * experts / (k * safe * safe * full.sum().clamp(min=1.0))
    loss = (per * (n * (member @ q)).sum(1)).sum()
    out = {"idx": torch.where(live[:, None], idx, -1).to(torch.int32), "gates": gates,
           "counts": n.sum(0).to(torch.int32), "loss": loss}
    if "d_gates" in s:
        dg = s["d_gates"]
        if case["renorm"]:
            dot = (dg * picked).sum(1, keepdim=True) / down
            ds_picked = ROUTE_SCALE * (dg - dot) / down
        else:
            ds_picked = ROUTE_SCALE * dg
        ds = torch.zeros_like(x).scatter_(1, idx, ds_picked)
        b = member.t() @ (per[:, None] * n)
        if case["score"]:
            ds = ds + (b - (b * q).sum(1, keepdim=True)) / z
            grad = ds * sc * (1 - sc)
        else:
            ds = ds + b
            grad = sc * (ds - (sc * ds).sum(1, keepdim=True))
        out["grad"] = torch.where(live[:, None], grad, 0.0).to(s["logits"].dtype)
    return out


_OWN = {"logprobs": _own_logprobs, "policy": _own_policy, "preference": _own_preference,
        "route": _own_route}
_PLAIN = {"logprobs": _plain_logprobs, "policy": _plain_policy, "preference": _plain_preference,
          "route": _plain_route}


# ------------------------------------------------------------------ work
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "route":
        n, t, k = case["tokens"] * case["experts"], case["tokens"], case["top_k"]
        seen = n * (t - _masked(case, t)) / t
        moved = seen * size + 8 * t * k + 8 * case["experts"] + 4
        ops = 8 * seen
        if case["backward"]:
            moved += n * size + 4 * t * k
            ops += 10 * seen
        return {"bytes": moved, "flops": ops}
    t, v = _tokens(case), case["vocab"]
    seen = (t - _masked(case, t)) * v
    if case["op"] == "logprobs":
        return {"bytes": seen * size + 12 * t, "flops": 4 * seen}
    # targets, weights, ref_logp, logp; the policy's old_logp and advantages
    moved = seen * size + t * v * size + (28 if case["op"] == "policy" else 20) * t
    return {"bytes": moved, "flops": 8 * seen}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """What run() returns, from the definitions, in 64 bits."""
    s = prepare(case, seed)
    return _exact_route(s) if case["op"] == "route" else _exact_logits(s)


def _exact_logits(s):
    case, x, y = s["case"], s["logits"], s["targets"]
    t, v = x.shape
    dev = x.device
    w = s["weights"].double() if case["op"] != "logprobs" else torch.ones(t, dtype=torch.float64, device=dev)
    live = torch.nonzero((y >= 0) & (w != 0)).flatten()
    inv_t = 1.0 / case["temperature"]
    logp = torch.zeros(t, dtype=torch.float64, device=dev)
    logp[live] = _logprobs64(x[live], y[live], inv_t)
    if case["op"] == "logprobs":
        return {"logp": logp}
    coef = torch.zeros(t, dtype=torch.float64, device=dev)
    ref = s["ref_logp"].double()
    if case["op"] == "policy":
        a, beta = s["advantages"].double()[live], case["beta"]
        lw, lr = w[live], torch.exp(logp[live] - s["old_logp"].double()[live])
        n = float(lw.sum()) if case["mean"] and live.numel() and float(lw.sum()) else 1.0
        clipped = torch.where(a >= 0, lr > 1 + CLIP[1], lr < 1 - CLIP[0])
        bound = torch.where(a >= 0, 1 + CLIP[1], 1 - CLIP[0]).double()
        gain = torch.where(clipped, bound * a, lr * a)
        back = torch.exp(ref[live] - logp[live])
        kl = back - 1 - torch.log(back)
        policy = -SCALE / n * float((lw * gain).sum())
        kls = SCALE / n * float((lw * kl).sum()) if beta else 0.0
        coef[live] = SCALE / n * lw * (torch.where(clipped, 0.0, -lr * a) + beta * (1 - back))
        out = {"stats": np.array([policy + beta * kls, policy, kls, float(lw.sum())]), "logp": logp}
    else:
        pairs, starts = case["pairs"], s["seq_starts"].tolist()
        ratio, length = [], []
        wl = torch.zeros_like(w)
        wl[live] = w[live]
        for q in range(2 * pairs):
            part = slice(starts[q], starts[q + 1])
            total = float(wl[part].sum())
            length.append(total if case["average"] and total else 1.0)
            ratio.append(float((wl[part] * (logp[part] - ref[part])).sum()) / length[-1])
        loss, wide = 0.0, 0.0
        for q in range(pairs):
            h = ratio[q] - ratio[pairs + q]
            wide += case["beta"] * h / pairs
            if case["kind"] == 0:
                z = case["beta"] * h - MARGIN
                up = 1 / (1 + math.exp(-z))
                loss += -(1 - case["smoothing"]) * math.log(up) - case["smoothing"] * math.log(1 - up)
                slope = case["beta"] * (up - 1 + case["smoothing"])
            else:
                gap = h - 0.5 / case["beta"]
                loss, slope = loss + gap * gap, 2 * gap
            for side, q2 in ((1, q), (-1, pairs + q)):
                part = slice(starts[q2], starts[q2 + 1])
                coef[part] = side * SCALE / pairs * slope / length[q2] * wl[part]
        out = {"stats": np.array([SCALE * loss / pairs, wide]),
               "rewards": np.array([case["beta"] * r for r in ratio]), "logp": logp}
    grad = torch.zeros(t, v, dtype=torch.float64, device=dev)
    step = max(1, (1 << 27) // v)
    for r in range(0, live.numel(), step):
        at = live[r:r + step]
        z = torch.softmax(x[at].double() * inv_t, 1).mul_(-inv_t * coef[at, None])
        z[torch.arange(at.numel(), device=dev), y[at]] += inv_t * coef[at]
        grad[at] = z
    out["grad"] = grad
    return out


def _exact_route(s):
    case, k, experts = s["case"], s["case"]["top_k"], s["case"]["experts"]
    x = s["logits"].double().cpu().numpy()
    t = x.shape[0]
    live = np.ones(t, bool) if s["live"] is None else s["live"].cpu().numpy() != 0
    if case["score"]:
        sc = 1 / (1 + np.exp(-x))
        q = sc / sc.sum(1, keepdims=True)
    else:
        e = np.exp(x - x.max(1, keepdims=True))
        sc = q = e / e.sum(1, keepdims=True)
    key = x if s["bias"] is None else sc + s["bias"].double().cpu().numpy()
    idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
    picked = np.take_along_axis(sc, idx, 1)
    down = picked.sum(1, keepdims=True) if case["renorm"] else np.ones((t, 1))
    gates = np.where(live[:, None], ROUTE_SCALE * picked / down, 0)
    starts = [0, t] if s["seq_starts"] is None else s["seq_starts"].tolist()
    parts = [np.nonzero(live[a:b])[0] + a for a, b in zip(starts[:-1], starts[1:])]
    filled = sum(len(p) > 0 for p in parts)
    loss, counts, b = 0.0, np.zeros(experts, np.int64), np.zeros((t, experts))
    for p in parts:
        if len(p):
            n = np.bincount(idx[p].ravel(), minlength=experts)
            per = BALANCE * experts / (k * len(p) ** 2 * filled)
            loss += per * float((n * q[p].sum(0)).sum())
            counts += n
            b[p] = per * n
    out = {"idx": np.where(live[:, None], idx, -1).astype(np.int32), "gates": gates,
           "counts": counts.astype(np.int32), "loss": loss}
    if "d_gates" in s:
        dg = s["d_gates"].double().cpu().numpy()
        pull = np.zeros((t, experts))
        if case["renorm"]:
            dg = dg - (dg * picked).sum(1, keepdims=True) / down
        np.put_along_axis(pull, idx, ROUTE_SCALE * dg / down, 1)
        if case["score"]:
            pull += (b - (b * q).sum(1, keepdims=True)) / sc.sum(1, keepdims=True)
            grad = pull * sc * (1 - sc)
        else:
            pull += b
            grad = sc * (pull - (sc * pull).sum(1, keepdims=True))
        out["grad"] = np.where(live[:, None], grad, 0)
    return out
