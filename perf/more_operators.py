"""The operators that adapt a shared model and read its logits, as their users call them:
low-rank adapters of many requests beside a shared projection (out = base + scale * up (down x),
every row with its own request's adapter) and their gradients; the log probability of each row's
given token with the row's entropy and its likeliest alternatives, and the gradient of the two.

`own` chooses between the plain form (elementary torch operations in 32 bits) and this
repository's operators; `exact` is the definition in 64 bits."""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
IDS = {"int32": torch.int32, "int64": torch.int64}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token's log probability and alternatives over a large vocabulary while a request
        # is decoded: latency counts
        {"name": "logprobs 1x128000 fp32 top 5", "kind": "logprobs", "rows": 1, "vocab": 128000,
         "logits": "fp32", "ids": "int64", "top": 5, "scale": 1.0, "keep": 1.0, "pad": 0.0},
        # a decode batch under a grammar's mask (-inf), a temperature of 0.8, sizes that divide
        # nothing, some slots without a request
        {"name": "logprobs 48x50001 fp16 top 20 masked", "kind": "logprobs", "rows": 48,
         "vocab": 50001, "logits": "fp16", "ids": "int32", "top": 20, "scale": 1.25, "keep": 0.1,
         "pad": 0.1},
        # the prompt's log probabilities with alternatives, asked for with a request
        {"name": "logprobs 700x128000 bf16 top 20", "kind": "logprobs", "rows": 700,
         "vocab": 128000, "logits": "bf16", "ids": "int64", "top": 20, "scale": 1.0, "keep": 1.0,
         "pad": 0.0},
        # log probabilities and entropies of sampled sequences, scored for a policy's update
        {"name": "logprobs 4096x128000 bf16", "kind": "logprobs", "rows": 4096, "vocab": 128000,
         "logits": "bf16", "ids": "int64", "top": 0, "scale": 1.0, "keep": 1.0, "pad": 0.1},
        # a small model's training step
        {"name": "logprobs gradient 512x8192 fp32", "kind": "logprobs_grad", "rows": 512,
         "vocab": 8192, "logits": "fp32", "ids": "int64", "scale": 1.0, "keep": 1.0, "pad": 0.0,
         "entropy": False},
        # a policy's update: log probabilities and entropies weighted by row, padded batch
        {"name": "logprobs gradient 2048x128000 bf16", "kind": "logprobs_grad", "rows": 2048,
         "vocab": 128000, "logits": "bf16", "ids": "int64", "scale": 1.0, "keep": 1.0, "pad": 0.1,
         "entropy": True},
        # a decode batch, each row a request with one of 64 loaded adapters: latency counts
        {"name": "adapt 32 of 4096 to 4096 rank 16", "kind": "adapt", "rows": 32, "in": 4096,
         "out": 4096, "rank": 16, "adapters": 64, "type": "bf16", "to": "bf16", "base": True,
         "ids": "int64", "order": "shuffled", "pad": 0.0},
        # prompts of a few requests packed one behind another, odd sizes, some without adapter
        {"name": "adapt 5001 of 2750 to 11000 rank 8 fp16", "kind": "adapt", "rows": 5001,
         "in": 2750, "out": 11000, "rank": 8, "adapters": 12, "type": "fp16", "to": "fp16",
         "base": True, "ids": "int32", "order": "runs", "pad": 0.1},
        # long prompts through a wide projection with adapters of a large rank
        {"name": "adapt 16384 of 4096 to 12288 rank 64", "kind": "adapt", "rows": 16384,
         "in": 4096, "out": 12288, "rank": 64, "adapters": 8, "type": "bf16", "to": "bf16",
         "base": True, "ids": "int64", "order": "runs", "pad": 0.0},
        # a small model's training step, one adapter in full precision
        {"name": "adapt gradient 512 of 512 to 2048 rank 8 fp32", "kind": "adapt_grad",
         "rows": 512, "in": 512, "out": 2048, "rank": 8, "adapters": 1, "type": "fp32",
         "to": "fp32", "base": False, "ids": "int64", "order": "runs", "pad": 0.0},
        # odd sizes, adapters of several users trained side by side, gradients kept in 16 bits
        {"name": "adapt gradient 3001 of 2750 to 5001 rank 20 fp16", "kind": "adapt_grad",
         "rows": 3001, "in": 2750, "out": 5001, "rank": 20, "adapters": 6, "type": "fp16",
         "to": "fp16", "base": True, "ids": "int32", "order": "shuffled", "pad": 0.1},
        # a training step of adapters beside a square projection
        {"name": "adapt gradient 8192 of 4096 to 4096 rank 16", "kind": "adapt_grad",
         "rows": 8192, "in": 4096, "out": 4096, "rank": 16, "adapters": 4, "type": "bf16",
         "to": "fp32", "base": True, "ids": "int64", "order": "runs", "pad": 0.0},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["logprobs", "logprobs", "logprobs_grad", "adapt", "adapt", "adapt_grad"])
    sixteen = rng.choice(["fp16", "bf16", "bf16"])
    ids = rng.choice(["int32", "int64"])
    if kind.startswith("logprobs"):
        vocab = _spread(rng, 1000, 131072)
        most = (1 << 28) // vocab
        rows = _spread(rng, 1, min(8192, most))
        case = {"kind": kind, "rows": rows, "vocab": vocab,
                "logits": rng.choice(["fp32", sixteen]), "ids": ids,
                "scale": rng.choice([1.0, 1.25, 0.7]), "keep": rng.choice([1.0, 1.0, 0.1]),
                "pad": rng.choice([0.0, 0.1]) if rows >= 16 else 0.0}
        if kind == "logprobs":
            case["top"] = rng.choice([0, 1, 5, 20])
        else:
            case["entropy"] = rng.random() < 0.5
        return case
    inner, outer = _spread(rng, 96, 12288), _spread(rng, 96, 12288)
    rank = rng.choice([4, 8, 16, 16, 20, 32, 64])
    most = (1 << (28 if kind == "adapt" else 26)) // (inner + outer)
    rows = _spread(rng, 1 if kind == "adapt" else 64, min(16384, most))
    kinds = rng.choice(["fp32", sixteen, sixteen])
    return {"kind": kind, "rows": rows, "in": inner, "out": outer, "rank": rank,
            "adapters": _spread(rng, 1, 64 if kind == "adapt" else 8), "type": kinds,
            "to": rng.choice([kinds, "fp32"]), "base": rng.random() < 0.7, "ids": ids,
            "order": rng.choice(["shuffled", "runs"]) if rows <= 256 else "runs",
            "pad": rng.choice([0.0, 0.1]) if rows >= 16 else 0.0}


def work(case):
    size = {"fp32": 4, "fp16": 2, "bf16": 2, "int32": 4, "int64": 8}
    n = case["rows"]
    ids = n * size[case["ids"]]
    if case["kind"] == "logprobs":
        top = case["top"]
        return {"bytes": ids + n * case["vocab"] * size[case["logits"]] + 16 * n
                + n * top * (4 + size[case["ids"]]), "flops": 4.0 * n * case["vocab"]}
    if case["kind"] == "logprobs_grad":
        given = 8 * n + 4 * n + (8 * n if case["entropy"] else 0)
        return {"bytes": ids + given + 2 * n * case["vocab"] * size[case["logits"]],
                "flops": 4.0 * n * case["vocab"]}
    inner, outer, rank = case["in"], case["out"], case["rank"]
    unit, to = size[case["type"]], size[case["to"]]
    used = min(case["adapters"], n)  # an adapter of several rows is read once
    weights = used * rank * (inner + outer) * unit
    if case["kind"] == "adapt":
        return {"bytes": ids + weights + n * inner * unit + n * outer * to
                * (2 if case["base"] else 1), "flops": 2.0 * n * rank * (inner + outer)}
    return {"bytes": ids + weights + n * (inner + outer) * unit
            + n * inner * unit * (2 if case["base"] else 1)
            + case["adapters"] * rank * (inner + outer) * to,
            "flops": 2.0 * n * rank * (3 * inner + 2 * outer)}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _tokens(case, g):
    """Token ids, frequent ones far more often than rare ones (a frequency of 1 over the rank);
    -1 where a padded batch has no token."""
    vocab, n = case["vocab"], case["rows"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ids = (float(vocab) ** u).long().sub_(1).clamp_(0, vocab - 1)
    if case["pad"]:
        ids[torch.rand(n, generator=g, device="cuda") < case["pad"]] = -1
    return ids.to(IDS[case["ids"]])


def _logits(case, ids, g):
    """A model's logits: a wide base, and the given token raised by up to 20, so that some rows
    are sure of it and others are not.  `keep` of the others are left by a mask."""
    vocab, n = case["vocab"], case["rows"]
    out = torch.empty(n, vocab, dtype=DTYPES[case["logits"]], device="cuda")
    step = max(1, (1 << 27) // vocab)
    for r in range(0, n, step):
        part = torch.randn(min(step, n - r), vocab, generator=g, device="cuda").mul_(2.0)
        given = ids[r:r + step].long()
        at = given.clamp(0, vocab - 1)[:, None]
        if case["keep"] < 1.0:
            left = torch.rand(part.shape, generator=g, device="cuda") < case["keep"]
            left.scatter_(1, at, True)
            part.masked_fill_(~left, -math.inf)
        rise = torch.rand(part.shape[0], 1, generator=g, device="cuda").mul_(20.0)
        part.scatter_(1, at, (part.gather(1, at) + rise).clamp_(-30.0, 30.0))
        out[r:r + step].copy_(part)
    return out


def _requests(case, g):
    """The adapter of each row: rows of a request lie together ("runs") or a batch has one row
    of each ("shuffled"); -1 for requests that use the shared model as it is."""
    n, adapters = case["rows"], case["adapters"]
    if case["order"] == "shuffled":
        ids = torch.randint(0, adapters, (n,), generator=g, device="cuda")
        bare = torch.rand(n, generator=g, device="cuda") < case["pad"]
    else:
        runs = max(1, min(2 * adapters, n // 64))
        of = torch.rand(n, generator=g, device="cuda").mul_(runs).long().clamp_(0, runs - 1)
        of = of.sort().values
        ids = torch.randint(0, adapters, (runs,), generator=g, device="cuda")[of]
        bare = (torch.rand(runs, generator=g, device="cuda") < case["pad"])[of]
    ids[bare] = -1
    return ids.to(IDS[case["ids"]])


def _normal(shape, dtype, g, by=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(by).to(DTYPES[dtype])


def _inputs(case, seed):
    g = _generator(seed)
    kind, n = case["kind"], case["rows"]
    s = {"case": case}
    if kind.startswith("logprobs"):
        s["ids"] = _tokens(case, g)
        s["logits"] = _logits(case, s["ids"], g)
        if kind == "logprobs_grad":
            # the weights of a policy's update (advantages) and of its entropies
            s["grad"] = torch.randn(n, generator=g, device="cuda")
            if case["entropy"]:
                s["grad_entropy"] = torch.full((n,), 0.01, device="cuda")
        return s
    inner, outer, rank, adapters = case["in"], case["out"], case["rank"], case["adapters"]
    s["ids"] = _requests(case, g)
    s["x"] = _normal((n, inner), case["type"], g)
    s["down"] = _normal((adapters, rank, inner), case["type"], g, inner ** -0.5)
    s["up"] = _normal((adapters, outer, rank), case["type"], g, rank ** -0.5)
    s["scales"] = torch.rand(adapters, generator=g, device="cuda").add_(0.5)
    if kind == "adapt":
        if case["base"]:
            s["base"] = _normal((n, outer), case["to"], g)
        return s
    s["grad"] = _normal((n, outer), case["type"], g)
    if case["base"]:
        s["base"] = _normal((n, inner), case["type"], g)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["kind"] == "logprobs_grad":
        # what the forward pass left: each row's largest logit and the logarithm of its sum, and
        # its entropy
        logits, stats, entropy = s["logits"], [], []
        step = max(1, (1 << 26) // case["vocab"])
        for r in range(0, case["rows"], step):
            m, total, h = _statistics64(logits[r:r + step], case["scale"])
            stats.append(torch.stack((m, total), 1).float())
            entropy.append(h.float())
        s["stats"] = torch.cat(stats)
        if case["entropy"]:
            s["entropy"] = torch.cat(entropy)
    return s


# ------------------------------------------------------------------ one pass

def _plain_logprobs(s):
    case = s["case"]
    vocab, scale, top = case["vocab"], case["scale"], case["top"]
    ids = s["ids"].long()
    there = (ids >= 0) & (ids < vocab)
    x = s["logits"].float()
    m = x.max(1).values
    z = (x - m[:, None]) * scale
    e = torch.exp(z)
    total = e.sum(1)
    log_total = torch.log(total)
    # a masked logit has no share in the entropy
    entropy = log_total - torch.where(e > 0, e * z, 0.0).sum(1) / total
    given = z.gather(1, ids.clamp(0, vocab - 1)[:, None])[:, 0] - log_total
    out = [torch.where(there, given, 0.0), entropy, torch.stack((m, log_total), 1)]
    if top:
        # order by value, then by the lower index: whole numbers that hold both
        bits = x.view(torch.int32).long()
        order = torch.where(bits >= 0, bits, -(bits & 0x7fffffff))
        keys = (order << 32) - torch.arange(vocab, device="cuda")
        at = (-keys.topk(top, 1).values) & 0xffffffff
        out += [at.to(s["ids"].dtype), z.gather(1, at) - log_total[:, None]]
    return out


def _plain_logprobs_grad(s):
    case = s["case"]
    vocab, scale = case["vocab"], case["scale"]
    ids = s["ids"].long()
    there = (ids >= 0) & (ids < vocab)
    weight = torch.where(there, s["grad"], 0.0)[:, None]
    lp = (s["logits"].float() - s["stats"][:, :1]) * scale - s["stats"][:, 1:]
    p = torch.exp(lp)
    d = -weight * p
    if case["entropy"]:
        d = d - s["grad_entropy"][:, None] * torch.where(
            p > 0, p * (lp + s["entropy"][:, None]), 0.0)
    d.scatter_add_(1, ids.clamp(0, vocab - 1)[:, None], weight)
    return (d * scale).to(DTYPES[case["logits"]])


def _plain_adapt(s):
    """All adapters' products, those of other adapters than the row's set to zero."""
    case = s["case"]
    n, adapters, rank = case["rows"], case["adapters"], case["rank"]
    of = s["ids"].long()[:, None] == torch.arange(adapters, device="cuda")
    pick = of[:, :, None].expand(n, adapters, rank).reshape(n, adapters * rank)
    wide = s["scales"].repeat_interleave(rank)
    down = s["down"].float().view(adapters * rank, case["in"])
    up = s["up"].float().transpose(1, 2).reshape(adapters * rank, case["out"])
    x = s["x"].float()
    hidden = torch.where(pick, (x @ down.t()) * wide, 0.0)
    if case["kind"] == "adapt":
        y = hidden @ up
        if case["base"]:
            y = y + s["base"].float()
        return y.to(DTYPES[case["to"]])
    grad = s["grad"].float()
    inner = torch.where(pick, (grad @ up.t()) * wide, 0.0)
    dx = inner @ down
    if case["base"]:
        dx = dx + s["base"].float()
    ddown = (inner.t() @ x).view(adapters, rank, case["in"])
    dup = (grad.t() @ hidden).view(case["out"], adapters, rank).transpose(0, 1).contiguous()
    to = DTYPES[case["to"]]
    return dx.to(s["x"].dtype), ddown.to(to), dup.to(to)


def run(state):
    case = state["case"]
    kind = case["kind"]
    if not own:
        if kind == "logprobs":
            return _plain_logprobs(state)
        if kind == "logprobs_grad":
            return _plain_logprobs_grad(state)
        return _plain_adapt(state)
    import spmv_storage_formats_amd as spmv
    if kind == "logprobs":
        r = spmv.token_logprobs(state["logits"], state["ids"], scale=case["scale"],
                                top=case["top"])
        out = [r.logprobs, r.entropy, r.stats]
        if case["top"]:
            out += [r.top_ids, r.top_logprobs]
        return out
    if kind == "logprobs_grad":
        return spmv.token_logprobs_grad(state["grad"], state["logits"], state["ids"],
                                        state["stats"], entropy=state.get("entropy"),
                                        grad_entropy=state.get("grad_entropy"),
                                        scale=case["scale"])
    if kind == "adapt":
        return spmv.adapt(state["x"], state["down"], state["up"], state["ids"],
                          base=state.get("base"), scales=state["scales"],
                          dtype=DTYPES[case["to"]])
    return spmv.adapt_grad(state["grad"], state["x"], state["down"], state["up"], state["ids"],
                           base=state.get("base"), scales=state["scales"],
                           dtype=DTYPES[case["to"]])


# ------------------------------------------------------------------ the definition in 64 bits

def _statistics64(logits, scale):
    """Largest logit, logarithm of the sum of exp(scale * (x - largest)), entropy, by row."""
    x = logits.double()
    m = x.amax(1)
    z = x.sub_(m[:, None]).mul_(scale)
    p = z.exp()
    total = p.sum(1)
    z.masked_fill_(p == 0, 0.0)
    rest = (p * z).sum(1)
    return m, total.log(), total.log() - rest / total


def _exact_logprobs(s):
    case = s["case"]
    vocab, scale, top = case["vocab"], case["scale"], case["top"]
    ids = s["ids"].cpu().tolist()
    logprobs, entropy, stats, top_ids, top_logprobs = [], [], [], [], []
    step = max(1, (1 << 26) // vocab)
    for r in range(0, case["rows"], step):
        part = s["logits"][r:r + step]
        m, total, h = _statistics64(part, scale)
        entropy.append(h)
        stats.append(torch.stack((m, total), 1))
        for t in range(part.shape[0]):
            if 0 <= ids[r + t] < vocab:
                logprobs.append((part[t, ids[r + t]].double() - m[t]) * scale - total[t])
            else:
                logprobs.append(torch.zeros((), dtype=torch.float64, device="cuda"))
        if top:
            # the first of the largest, `top` times, those found before left out
            left = part.double()
            for_row = torch.arange(part.shape[0], device="cuda")
            index = torch.arange(vocab, device="cuda")
            found, values = [], []
            for _ in range(top):
                best = left.amax(1)
                first = torch.where(left == best[:, None], index, vocab).amin(1)
                found.append(first)
                values.append((best - m) * scale - total)
                left[for_row, first] = -math.inf
            top_ids.append(torch.stack(found, 1))
            top_logprobs.append(torch.stack(values, 1))
    out = [torch.stack(logprobs), torch.cat(entropy), torch.cat(stats)]
    if top:
        out += [torch.cat(top_ids).to(s["ids"].dtype), torch.cat(top_logprobs)]
    return out


def _exact_logprobs_grad(s):
    case = s["case"]
    vocab, scale = case["vocab"], case["scale"]
    ids = s["ids"].cpu().tolist()
    out = torch.empty(case["rows"], vocab, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // vocab)
    for r in range(0, case["rows"], step):
        part = s["logits"][r:r + step]
        m, total, h = _statistics64(part, scale)
        lp = (part.double() - m[:, None]) * scale - total[:, None]
        p = lp.exp()
        d = out[r:r + step]
        d.zero_()
        if case["entropy"]:
            lp.masked_fill_(p == 0, 0.0)
            d -= s["grad_entropy"][r:r + step, None].double() * p * (lp + h[:, None])
        for t in range(part.shape[0]):
            v = ids[r + t]
            if 0 <= v < vocab:
                w = s["grad"][r + t].double()
                d[t] -= w * p[t]
                d[t, v] += w
        d *= scale
    return out


def _exact_adapt(s):
    case = s["case"]
    n, inner, outer = case["rows"], case["in"], case["out"]
    ids = s["ids"].cpu().tolist()
    rows = {}
    for t, a in enumerate(ids):
        if 0 <= a < case["adapters"]:
            rows.setdefault(a, []).append(t)
    backward = case["kind"] == "adapt_grad"
    width = inner if backward else outer
    y = torch.zeros(n, width, dtype=torch.float64, device="cuda")
    if case["base"]:
        y += s["base"].double()
    if backward:
        ddown = torch.zeros(s["down"].shape, dtype=torch.float64, device="cuda")
        dup = torch.zeros(s["up"].shape, dtype=torch.float64, device="cuda")
    for a, of in rows.items():
        at = torch.tensor(of, device="cuda")
        x, down, up = s["x"][at].double(), s["down"][a].double(), s["up"][a].double()
        scale = s["scales"][a].double()
        hidden = x @ down.t()
        if not backward:
            y[at] += scale * (hidden @ up.t())
            continue
        grad = s["grad"][at].double()
        back = scale * (grad @ up)
        y[at] += back @ down
        ddown[a] = back.t() @ x
        dup[a] = scale * (grad.t() @ hidden)
    return (y, ddown, dup) if backward else y


def exact(case, seed):
    s = _inputs(case, seed)
    if case["kind"] == "logprobs":
        return _exact_logprobs(s)
    if case["kind"] == "logprobs_grad":
        return _exact_logprobs_grad(s)
    return _exact_adapt(s)
