"""What a mixture-of-experts model's post-training calls between the router and
the losses, as a user's program calls it, each with a plain form in elementary
torch operations beside it.

Three operators:
  scores   log probability of each token under its row of logits, the row's
           entropy and its top alternatives; with backward, the logits' gradient
  tokens   tokens sorted by expert (rows in the experts' order) and the experts'
           outputs combined with their gates; with backward, all gradients
  experts  the products of the sorted rows with their experts' weights; with
           backward, the gradients of rows and weights

A case is a dict of sizes and options; ``own`` selects the framework's
operators (True) or the plain forms (False) in ``run``.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# Tokens come in spans of this many, each a response followed by what is masked:
# the next prompt, or padding.
SPAN = 512
# The most a drawn case may move or compute: what the largest listed ones do.
MOST_LOGITS = 4096 * 131072 * 2
MOST_ROWS = 32768 * 8 * 2048 * 2
MOST_WEIGHTS = 32 * 5760 * 2880
MOST_PRODUCT = 8192 * 4 * 5760 * 2880


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a few tokens just sampled, one decoding step, with alternatives for display
        {"name": "scores_step", "op": "scores", "tokens": 8, "vocab": 32000, "dtype": "bf16",
         "top_k": 5, "live": 1.0, "pad": 0, "temperature": 1.0, "backward": False},
        # a teacher's or reference model's pass over a batch of rollouts, large vocabulary
        {"name": "scores_reference", "op": "scores", "tokens": 4096, "vocab": 131072,
         "dtype": "bf16", "top_k": 20, "live": 0.75, "pad": 0, "temperature": 1.0, "backward": False},
        # a training micro-batch: entropy bonus and distillation on the alternatives
        {"name": "scores_train", "op": "scores", "tokens": 4096, "vocab": 32000, "dtype": "bf16",
         "top_k": 8, "live": 0.75, "pad": 0, "temperature": 1.0, "backward": True},
        # fp32 logits, odd vocabulary in rows of an odd stride, sampling temperature
        {"name": "scores_odd_fp32", "op": "scores", "tokens": 777, "vocab": 50021, "dtype": "fp32",
         "top_k": 3, "live": 0.9, "pad": 3, "temperature": 0.8, "backward": True},
        # serving: a few tokens to the experts of the 32-expert layer and back
        {"name": "tokens_step", "op": "tokens", "tokens": 8, "experts": 32, "top_k": 4,
         "hidden": 2880, "dtype": "bf16", "live": 1.0, "pad": 0, "backward": False},
        # training: a micro-batch of the same layer, both directions
        {"name": "tokens_batch", "op": "tokens", "tokens": 8192, "experts": 32, "top_k": 4,
         "hidden": 2880, "dtype": "bf16", "live": 0.9, "pad": 0, "backward": True},
        # training: 256 experts, 8 a token, a large micro-batch
        {"name": "tokens_large", "op": "tokens", "tokens": 32768, "experts": 256, "top_k": 8,
         "hidden": 2048, "dtype": "bf16", "live": 1.0, "pad": 0, "backward": True},
        # fp32, odd width in rows of an odd stride, odd numbers of experts and choices
        {"name": "tokens_odd_fp32", "op": "tokens", "tokens": 5001, "experts": 61, "top_k": 7,
         "hidden": 1001, "dtype": "fp32", "live": 0.75, "pad": 2, "backward": True},
        # serving: the same few tokens through the layer's first product
        {"name": "experts_step", "op": "experts", "tokens": 8, "experts": 32, "top_k": 4,
         "out": 5760, "in": 2880, "live": 1.0, "backward": False},
        # a prompt of some hundred tokens through the second product
        {"name": "experts_prompt", "op": "experts", "tokens": 500, "experts": 32, "top_k": 4,
         "out": 2880, "in": 2880, "live": 1.0, "backward": False},
        # training: small experts of odd widths, a masked part, both directions
        {"name": "experts_odd", "op": "experts", "tokens": 1003, "experts": 13, "top_k": 3,
         "out": 1001, "in": 523, "live": 0.9, "backward": True},
        # training: the layer's first product on a micro-batch, both directions
        {"name": "experts_large", "op": "experts", "tokens": 8192, "experts": 32, "top_k": 4,
         "out": 5760, "in": 2880, "live": 1.0, "backward": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["scores", "tokens", "experts"])
    live = rng.choice([1.0, 0.9, 0.75, 0.5])
    backward = rng.random() < 0.6
    if op == "scores":
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        vocab = _log_int(rng, 1000, 200000)
        if rng.random() < 0.5:
            vocab = max(1024, vocab // 128 * 128)
        pad = rng.choice([0, 0, 0, 1, 5, 64])
        size = 2 if dtype == "bf16" else 4
        rows = min(8192, MOST_LOGITS // (2 if backward else 1) // ((vocab + pad) * size))
        return {"op": op, "tokens": _log_int(rng, 1, rows), "vocab": vocab, "dtype": dtype,
                "top_k": rng.randint(0, 20), "live": live, "pad": pad,
                "temperature": rng.choice([1.0, 1.0, 0.7]), "backward": backward}
    if op == "tokens":
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        experts = _log_int(rng, 2, 512)
        top_k = rng.randint(1, min(8, experts))
        hidden = _log_int(rng, 64, 8192)
        pad = rng.choice([0, 0, 1, 8])
        if rng.random() < 0.6:
            hidden, pad = max(64, hidden // 64 * 64), pad // 8 * 8
        size = 2 if dtype == "bf16" else 4
        most = min(32768, MOST_ROWS // ((hidden + pad) * size * top_k))
        return {"op": op, "tokens": _log_int(rng, 1, most), "experts": experts, "top_k": top_k,
                "hidden": hidden, "dtype": dtype, "live": live, "pad": pad, "backward": backward}
    n, k = _log_int(rng, 64, 8192), _log_int(rng, 64, 8192)
    if rng.random() < 0.6:
        n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
    experts = _log_int(rng, 2, max(2, min(64, MOST_WEIGHTS // (n * k))))
    top_k = rng.randint(1, min(8, experts))
    most = max(1, min(16384, MOST_PRODUCT // (n * k * top_k)))
    return {"op": op, "tokens": _log_int(rng, 1, most), "experts": experts, "top_k": top_k,
            "out": n, "in": k, "live": live, "backward": backward}


# ------------------------------------------------------------------ inputs
def _kept(case):
    """Tokens at the head of each span that are not masked."""
    return int(round(SPAN * case["live"]))


def _live(case):
    """How many tokens are not masked."""
    kept, tokens = _kept(case), case["tokens"]
    return tokens // SPAN * kept + min(tokens % SPAN, kept)


def _cuts(case):
    """Where each expert's rows start (experts + 1 of them): uneven loads, one
    expert without a row among three or more."""
    share = [2 + 3 * ((7 * e) % 5) for e in range(case["experts"])]
    if case["experts"] >= 3:
        share[1] = 0
    rows, total, cuts, seen = _live(case) * case["top_k"], sum(share), [0], 0
    for s in share:
        seen += s
        cuts.append(rows * seen // total)
    return cuts


def _wide(n):
    """Row strides of the products' operands: whole pieces of 16 bytes."""
    return (n + 7) // 8 * 8


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _prepare_scores(case, seed, state):
    g = _generator(seed)
    tokens, vocab, k = case["tokens"], case["vocab"], case["top_k"]
    wide = torch.randn(tokens, vocab + case["pad"], generator=g, device="cuda",
                       dtype=DTYPES[case["dtype"]]).mul_(2.5)
    logits = wide[:, :vocab]
    targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    # the sampled word is mostly a likely one
    rows = torch.arange(tokens, device="cuda")
    logits[rows, targets] += (9.0 + 3.0 * torch.randn(tokens, generator=g, device="cuda")).to(wide.dtype)
    state["targets"] = torch.where(rows % SPAN < _kept(case), targets, -100)
    state.update(logits=logits, inv_t=1.0 / case["temperature"])
    if case["backward"]:
        state["d_logp"] = 1e-3 * torch.randn(tokens, generator=g, device="cuda")
        state["d_entropy"] = 1e-4 * torch.randn(tokens, generator=g, device="cuda")
        state["d_top"] = 1e-3 * torch.randn(tokens, k, generator=g, device="cuda") if k else None


def _prepare_tokens(case, seed, state):
    g = _generator(seed)
    tokens, experts, k, hidden = case["tokens"], case["experts"], case["top_k"], case["hidden"]
    dt = DTYPES[case["dtype"]]

    def rows(n):
        return torch.randn(n, hidden + case["pad"], generator=g, device="cuda", dtype=dt)[:, :hidden]

    # a router's choice: some experts are taken more often than others
    lean = 0.7 * torch.randn(experts, generator=g, device="cuda")
    score = torch.randn(tokens, experts, generator=g, device="cuda") + lean
    idx = torch.topk(score, k, dim=1).indices.to(torch.int32)
    live = torch.arange(tokens, device="cuda") % SPAN < _kept(case)
    state["idx"] = torch.where(live[:, None], idx, -1)
    gates = torch.rand(tokens, k, generator=g, device="cuda") + 0.1
    state["gates"] = torch.where(live[:, None], gates / gates.sum(1, keepdim=True), 0.0)
    state["x"], state["y"] = rows(tokens), rows(tokens * k)
    if case["backward"]:
        state["d_out"], state["d_rows"] = rows(tokens), rows(tokens * k)


def _prepare_experts(case, seed, state):
    g = _generator(seed)
    rows, experts, n, k = case["tokens"] * case["top_k"], case["experts"], case["out"], case["in"]

    def made(*shape):
        return torch.randn(*shape[:-1], _wide(shape[-1]), generator=g, device="cuda",
                           dtype=torch.bfloat16)[..., :shape[-1]]

    state["starts"] = torch.tensor(_cuts(case), dtype=torch.int32, device="cuda")
    state["x"] = made(rows, k)
    state["w"] = made(experts, n, k).mul_(k ** -0.5)
    if case["backward"]:
        state["d_y"] = made(rows, n)


def prepare(case, seed):
    state = {"case": case}
    {"scores": _prepare_scores, "tokens": _prepare_tokens, "experts": _prepare_experts}[case["op"]](
        case, seed, state)
    if own:
        from fsdp_buffer_layout_gb300 import experts, objectives
        if case["op"] == "scores":
            state["call"] = objectives.TokenScores(
                case["tokens"], case["vocab"], top_k=case["top_k"], dtype=DTYPES[case["dtype"]],
                inv_temperature=state["inv_t"])
        elif case["op"] == "tokens":
            state["call"] = experts.Dispatch(case["tokens"], case["experts"], case["top_k"],
                                             case["hidden"], dtype=DTYPES[case["dtype"]])
        else:
            state["call"] = experts.ExpertLinear(case["tokens"] * case["top_k"], case["experts"],
                                                 case["out"], case["in"])
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_scores(s):
    logp, entropy, top_idx, top_logp = s["call"].forward(s["logits"], s["targets"])
    out = {"logp": logp, "entropy": entropy, "top_idx": top_idx, "top_logp": top_logp}
    if "d_logp" in s:
        out["grad"] = s["call"].backward(s["logits"], s["targets"], d_logp=s["d_logp"],
                                         d_entropy=s["d_entropy"], d_top=s["d_top"])
    return out


def _own_tokens(s):
    call = s["call"]
    starts, source, place = call.sort(s["idx"])
    out = {"starts": starts, "source": source, "place": place, "rows": call.gather(s["x"]),
           "out": call.combine(s["y"], s["gates"])}
    if "d_out" in s:
        out["d_y"], out["d_gates"] = call.combine_backward(s["d_out"], s["y"], s["gates"])
        out["d_x"] = call.gather_backward(s["d_rows"])
    return out


def _own_experts(s):
    call = s["call"]
    out = {"y": call.forward(s["x"], s["w"], s["starts"])}
    if "d_y" in s:
        out["d_x"] = call.backward_input(s["d_y"], s["w"], s["starts"])
        out["d_w"] = call.backward_weight(s["d_y"], s["x"], s["starts"])
    return out


def _plain_scores(s):
    case = s["case"]
    k, vocab = case["top_k"], case["vocab"]
    x = s["logits"].float()
    z = x * s["inv_t"]
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    p, lnp = e / total, z - torch.log(total)
    live = s["targets"] >= 0
    at = s["targets"].clamp(min=0)[:, None]
    logp = torch.where(live, lnp.gather(1, at).squeeze(1), 0.0)
    entropy = -torch.where(p > 0, p * lnp, 0.0).sum(1)
    # value and then position as one whole number: equal values in their order
    bits = x.view(torch.int32).long()
    bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    key = (bits << 32) + (vocab - 1 - torch.arange(vocab, device=x.device))
    top = torch.topk(key, k, dim=1).indices
    out = {"logp": logp, "entropy": torch.where(live, entropy, 0.0),
           "top_idx": torch.where(live[:, None], top, -1).to(torch.int32),
           "top_logp": torch.where(live[:, None], lnp.gather(1, top), 0.0)}
    if "d_logp" in s:
        d_top = s["d_top"] if k else torch.zeros_like(logp)[:, None][:, :0]
        pull = s["d_logp"] + d_top.sum(1)
        grad = -p * (pull[:, None] + s["d_entropy"][:, None] * (lnp + entropy[:, None]))
        grad.scatter_add_(1, at, s["d_logp"][:, None])
        grad.scatter_add_(1, top, d_top)
        out["grad"] = torch.where(live[:, None], grad * s["inv_t"], 0.0).to(s["logits"].dtype)
    return out


def _plain_tokens(s):
    case = s["case"]
    k, experts = case["top_k"], case["experts"]
    idx = s["idx"].flatten()
    n = idx.numel()
    key = torch.where(idx < 0, experts, idx)
    source = torch.sort(key, stable=True).indices
    starts = torch.zeros(experts + 2, dtype=torch.long, device=idx.device)
    starts = starts.index_add(0, key.long() + 1, torch.ones_like(source)).cumsum(0)[:experts + 1]
    at = torch.arange(n, device=idx.device)
    here = (at < starts[-1])[:, None]              # rows that hold a token
    place = torch.zeros_like(source).scatter_(0, source, at)
    routed = (idx >= 0).view(-1, k, 1)
    x, y, gates = s["x"], s["y"].float(), s["gates"]
    taken = torch.where(routed, y[place].view(-1, k, y.shape[1]), 0.0)
    out = {"starts": starts.to(torch.int32),
           "source": torch.where(here[:, 0], source, -1).to(torch.int32),
           "place": torch.where(routed.view(-1, k), place.view(-1, k), -1).to(torch.int32),
           "rows": torch.where(here, x[source // k], 0.0),
           "out": (gates[:, :, None] * taken).sum(1).to(x.dtype)}
    if "d_out" in s:
        d_out = s["d_out"].float()
        d_y = gates.flatten()[source][:, None] * d_out[source // k]
        out["d_y"] = torch.where(here, d_y, 0.0).to(x.dtype)
        out["d_gates"] = (d_out[:, None] * taken).sum(2)
        d_rows = s["d_rows"].float()[place].view(-1, k, y.shape[1])
        out["d_x"] = torch.where(routed, d_rows, 0.0).sum(1).to(x.dtype)
    return out


def _plain_experts(s):
    case = s["case"]
    experts, cuts, starts = case["experts"], _cuts(case), s["starts"].long()
    x, w = s["x"].float(), s["w"].float()
    rows = x.shape[0]
    # each expert's rows padded to the longest; rows of no expert behind them
    most = max([b - a for a, b in zip(cuts, cuts[1:])] + [rows - cuts[-1], 1])
    at = torch.arange(rows, device=x.device)
    expert = (at[:, None] >= starts[1:]).sum(1)
    place = at - starts[expert]
    here = (expert < experts)[:, None]

    def padded(v):
        out = torch.zeros(experts + 1, most, v.shape[1], device=v.device)
        out[expert, place] = v
        return out[:experts]

    def rows_of(v):
        return torch.where(here, v[expert.clamp(max=experts - 1), place], 0.0).to(s["x"].dtype)

    px = padded(x)
    out = {"y": rows_of(torch.bmm(px, w.transpose(1, 2)))}
    if "d_y" in s:
        pd = padded(s["d_y"].float())
        out["d_x"] = rows_of(torch.bmm(pd, w))
        out["d_w"] = torch.bmm(pd.transpose(1, 2), px).to(s["w"].dtype)
    return out


_OWN = {"scores": _own_scores, "tokens": _own_tokens, "experts": _own_experts}
_PLAIN = {"scores": _plain_scores, "tokens": _plain_tokens, "experts": _plain_experts}


# ------------------------------------------------------------------ work
def work(case):
    t = case["tokens"]
    if case["op"] == "scores":
        size, v = 2 if case["dtype"] == "bf16" else 4, case["vocab"]
        seen = _live(case) * v
        moved, ops = seen * size + 16 * t + 8 * t * case["top_k"], 6 * seen
        if case["backward"]:
            moved += t * v * size + 8 * t + 4 * t * case["top_k"]
            ops += 8 * seen
        return {"bytes": moved, "flops": ops}
    if case["op"] == "tokens":
        size, h, c = 2 if case["dtype"] == "bf16" else 4, case["hidden"], t * case["top_k"]
        n = _live(case) * case["top_k"]
        # idx, gates, starts, source, place; x, rows, y, out
        moved = 16 * c + 4 * case["experts"] + (_live(case) + 2 * n + t) * h * size
        ops = 2 * n * h
        if case["backward"]:
            # d_gates; d_out, d_y, d_rows, d_x (y has been read)
            moved += 4 * c + (_live(case) + 2 * n + t) * h * size
            ops += 4 * n * h
        return {"bytes": moved, "flops": ops}
    cuts, n, k = _cuts(case), case["out"], case["in"]
    used = sum(a < b for a, b in zip(cuts, cuts[1:]))
    moved = 2 * (used * n * k + cuts[-1] * (n + k))
    if case["backward"]:
        moved += 2 * (case["experts"] * n * k + cuts[-1] * (n + k))
    return {"bytes": moved, "flops": 2 * cuts[-1] * n * k * (3 if case["backward"] else 1)}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """What run() returns, from the definitions, in 64 bits."""
    s = prepare(case, seed)
    return {"scores": _exact_scores, "tokens": _exact_tokens, "experts": _exact_experts}[case["op"]](s)


def _exact_scores(s):
    case, x, y = s["case"], s["logits"], s["targets"]
    t, v = x.shape
    k, inv_t, dev = case["top_k"], 1.0 / case["temperature"], x.device
    f64 = {"dtype": torch.float64, "device": dev}
    out = {"logp": torch.zeros(t, **f64), "entropy": torch.zeros(t, **f64),
           "top_idx": torch.full((t, k), -1, dtype=torch.int32, device=dev),
           "top_logp": torch.zeros(t, k, **f64)}
    if "d_logp" in s:
        out["grad"] = torch.zeros(t, v, **f64)
    live = torch.nonzero(y >= 0).flatten()
    step = max(1, (1 << 26) // v)
    for r in range(0, live.numel(), step):
        at = live[r:r + step]
        one = torch.arange(at.numel(), device=dev)
        z = x[at].double() * inv_t
        lp = z - torch.logsumexp(z, 1, keepdim=True)
        p = torch.exp(lp)
        h = -torch.special.xlogy(p, p).sum(1)
        best = torch.sort(x[at], dim=1, descending=True, stable=True).indices[:, :k]
        out["logp"][at] = lp[one, y[at]]
        out["entropy"][at] = h
        out["top_idx"][at] = best.to(torch.int32)
        out["top_logp"][at] = lp.gather(1, best)
        if "d_logp" in s:
            # d logp_u = 1(v = u) - p, d entropy = -p (ln p + entropy)
            dl = torch.zeros(at.numel(), v, **f64)
            dl[one, y[at]] = s["d_logp"].double()[at]
            if k:
                dl.scatter_add_(1, best, s["d_top"].double()[at])
            lp += h[:, None]
            lp *= s["d_entropy"].double()[at, None]
            lp += dl.sum(1, keepdim=True)
            out["grad"][at] = inv_t * (dl - p * lp)
    return out


def _exact_tokens(s):
    case, idx = s["case"], s["idx"]
    t, k, experts, h = case["tokens"], case["top_k"], case["experts"], case["hidden"]
    dev = idx.device
    starts = [0]
    source = torch.full((t * k,), -1, dtype=torch.int32, device=dev)
    place = torch.full((t, k), -1, dtype=torch.int32, device=dev)
    back = "d_out" in s

    def zeros(*shape):
        return torch.zeros(*shape, dtype=torch.float64, device=dev)

    out = {"rows": zeros(t * k, h), "out": zeros(t, h)}
    if back:
        out.update(d_y=zeros(t * k, h), d_gates=zeros(t, k), d_x=zeros(t, h))
    for e in range(experts):
        token, slot = torch.nonzero(idx == e, as_tuple=True)
        a, b = starts[-1], starts[-1] + token.numel()
        starts.append(b)
        source[a:b] = (token * k + slot).to(torch.int32)
        place[token, slot] = torch.arange(a, b, dtype=torch.int32, device=dev)
        gate, y = s["gates"][token, slot].double()[:, None], s["y"][a:b].double()
        out["rows"][a:b] = s["x"][token].double()
        out["out"].index_add_(0, token, gate * y)
        if back:
            pull = s["d_out"][token].double()
            out["d_y"][a:b] = gate * pull
            out["d_gates"][token, slot] = (pull * y).sum(1)
            out["d_x"].index_add_(0, token, s["d_rows"][a:b].double())
    out.update(starts=torch.tensor(starts, dtype=torch.int32), source=source, place=place)
    return out


def _exact_experts(s):
    case, cuts = s["case"], s["starts"].tolist()
    rows, dev = s["x"].shape[0], s["x"].device

    def zeros(*shape):
        return torch.zeros(*shape, dtype=torch.float64, device=dev)

    out = {"y": zeros(rows, case["out"])}
    if "d_y" in s:
        out.update(d_x=zeros(rows, case["in"]), d_w=zeros(case["experts"], case["out"], case["in"]))
    for e, (a, b) in enumerate(zip(cuts, cuts[1:])):
        if a == b:
            continue
        x, w = s["x"][a:b].double(), s["w"][e].double()
        out["y"][a:b] = x @ w.t()
        if "d_y" in s:
            d_y = s["d_y"][a:b].double()
            out["d_x"][a:b] = d_y @ w
            out["d_w"][e] = d_y.t() @ x
    return out
