"""The operators of a model's token table, as their users call them: products with a 4-bit matrix
with group scales (a decode step's projections and logits), rows of a dense or a 4-bit table by
token with a scale (the input of a model), and the gradient of such a lookup by sorted tokens.

`own` chooses between the plain form (elementary torch operations in 32 bits) and this
repository's operators; `exact` is the definition in 64 bits."""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token through a square projection of a 4-bit model: latency counts
        {"name": "product 4096x4096 n1", "kind": "product", "rows": 4096, "cols": 4096, "n": 1,
         "group": 128, "zeros": False, "x": "bf16", "y": "bf16", "scales": "bf16", "add": False},
        # the repository's own contract, y += A x in fp32, at sizes that divide nothing
        {"name": "product 5001x2750 n3 fp32", "kind": "product", "rows": 5001, "cols": 2750, "n": 3,
         "group": 32, "zeros": True, "x": "fp32", "y": "fp32", "scales": "fp32", "add": True},
        # one token's logits over a large vocabulary, kept in fp32 for sampling
        {"name": "product 128000x4096 n1", "kind": "product", "rows": 128000, "cols": 4096, "n": 1,
         "group": 128, "zeros": False, "x": "bf16", "y": "fp32", "scales": "bf16", "add": False},
        # a decode batch of 16 through a wide projection, smaller groups and zero points
        {"name": "product 12288x8192 n16", "kind": "product", "rows": 12288, "cols": 8192, "n": 16,
         "group": 64, "zeros": True, "x": "fp16", "y": "fp16", "scales": "fp16", "add": False},
        # 48 rows of a batch with drafted tokens, added to the residual
        {"name": "product 8192x11000 n48", "kind": "product", "rows": 8192, "cols": 11000, "n": 48,
         "group": 128, "zeros": True, "x": "bf16", "y": "bf16", "scales": "bf16", "add": True},
        # a decode batch's input rows: latency counts
        {"name": "lookup 7 of 128000x4096", "kind": "lookup", "rows": 128000, "cols": 4096, "n": 7,
         "table": "bf16", "out": "bf16", "ids": "int64", "scale": 64.0, "pad": 0.0},
        # the prompts of a serving step, packed
        {"name": "lookup 16384 of 128000x4096", "kind": "lookup", "rows": 128000, "cols": 4096,
         "n": 16384, "table": "bf16", "out": "bf16", "ids": "int64", "scale": 1.0, "pad": 0.0},
        # rows of a tied 4-bit table, a padded batch
        {"name": "lookup 4-bit 5000 of 50001x2750", "kind": "lookup4", "rows": 50001, "cols": 2750,
         "n": 5000, "group": 32, "zeros": True, "scales": "fp16", "out": "fp16", "ids": "int32",
         "scale": 52.5, "pad": 0.1},
        {"name": "lookup 4-bit 8192 of 32768x4096", "kind": "lookup4", "rows": 32768, "cols": 4096,
         "n": 8192, "group": 128, "zeros": False, "scales": "bf16", "out": "bf16", "ids": "int64",
         "scale": 1.0, "pad": 0.0},
        # a small model's training step: few tokens, a small table
        {"name": "gradient 512 into 8192x512", "kind": "gradient", "rows": 8192, "cols": 512,
         "n": 512, "grad": "fp32", "out": "fp32", "ids": "int64", "scale": 1.0, "pad": 0.0},
        # odd sizes, a padded batch, gradients kept in 16 bits
        {"name": "gradient 5001 into 50001x1000", "kind": "gradient", "rows": 50001, "cols": 1000,
         "n": 5001, "grad": "fp16", "out": "fp16", "ids": "int32", "scale": 31.5, "pad": 0.1},
        # a large model's step: tokens as a language draws them, fp32 gradients
        {"name": "gradient 32768 into 128000x2048", "kind": "gradient", "rows": 128000,
         "cols": 2048, "n": 32768, "grad": "bf16", "out": "fp32", "ids": "int64", "scale": 1.0,
         "pad": 0.0},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["product", "product", "lookup", "lookup4", "gradient", "gradient"])
    cols = _spread(rng, 96, 12288)
    if kind == "product":
        case = {"kind": kind, "rows": _spread(rng, 64, min(131072, (1 << 28) // cols)),
                "cols": cols, "n": _spread(rng, 1, 64), "group": rng.choice([32, 64, 128, 256]),
                "zeros": rng.random() < 0.5, "add": rng.random() < 0.3}
        case["x"] = rng.choice(["fp32", "fp16", "bf16", "bf16"])
        case["y"] = rng.choice([case["x"], "fp32"])
        case["scales"] = rng.choice([case["x"], "fp32"])
        return case
    rows = _spread(rng, 1000, min(131072, (1 << 28) // cols))
    n = _spread(rng, 1, min(65536, (1 << 26) // cols))
    case = {"kind": kind, "rows": rows, "cols": cols, "n": n,
            "ids": rng.choice(["int32", "int64"]),
            "scale": rng.choice([1.0, round(math.sqrt(cols), 3)]), "pad": rng.choice([0.0, 0.1]) if n >= 16 else 0.0}
    sixteen = rng.choice(["fp16", "bf16", "bf16"])
    if kind == "lookup":
        case["table"] = rng.choice(["fp32", sixteen])
        case["out"] = rng.choice([case["table"], sixteen])
    elif kind == "lookup4":
        case["group"] = rng.choice([32, 64, 128, 256])
        case["zeros"] = rng.random() < 0.5
        case["scales"] = sixteen
        case["out"] = rng.choice([sixteen, "fp32"])
    else:
        case["grad"] = rng.choice(["fp32", sixteen])
        case["out"] = rng.choice([case["grad"], "fp32"])
    return case


def work(case):
    size = {"fp32": 4, "fp16": 2, "bf16": 2, "int32": 4, "int64": 8}
    rows, cols, n = case["rows"], case["cols"], case["n"]
    if case["kind"] in ("product", "lookup4"):
        row = (cols + 1) // 2
        row += -(-cols // case["group"]) * (size[case["scales"]] + (1 if case["zeros"] else 0))
    if case["kind"] == "product":
        return {"bytes": rows * row + n * cols * size[case["x"]]
                + n * rows * size[case["y"]] * (2 if case["add"] else 1),
                "flops": 2.0 * n * rows * cols}
    ids = n * size[case["ids"]]
    read = min(n, rows)  # a row asked for twice is read once
    if case["kind"] == "lookup4":
        return {"bytes": ids + read * row + n * cols * size[case["out"]], "flops": 2.0 * n * cols}
    if case["kind"] == "lookup":
        return {"bytes": ids + read * cols * size[case["table"]] + n * cols * size[case["out"]],
                "flops": 1.0 * n * cols}
    return {"bytes": ids + n * cols * size[case["grad"]] + rows * cols * size[case["out"]],
            "flops": 1.0 * n * cols}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _quantised(case, g):
    """A 4-bit matrix as a checkpoint holds it: two codes per byte (the even column in the low
    half), a scale per row and group, and, with `zeros`, a zero point per row and group."""
    rows, cols = case["rows"], case["cols"]
    groups = -(-cols // case["group"])
    # codes spread over the 16 values as those of normally distributed weights are
    codes = torch.empty(rows, (cols + 1) // 2, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // codes.shape[1])
    for r in range(0, rows, step):
        part = codes[r:r + step]
        low, high = (torch.randn(part.shape, generator=g, device="cuda").mul_(3).add_(8).round_()
                     .clamp_(0, 15).to(torch.uint8) for _ in range(2))
        part.copy_(low | (high << 4))
    scales = torch.rand(rows, groups, generator=g, device="cuda").mul_(0.01).add_(0.005)
    zeros = None
    if case["zeros"]:
        zeros = torch.randint(4, 12, (rows, groups), generator=g, device="cuda", dtype=torch.uint8)
    return {"codes": codes, "scales": scales.to(DTYPES[case["scales"]]), "zeros": zeros}


def _tokens(case, g):
    """Token ids, frequent ones far more often than rare ones (a frequency of 1 over the rank);
    -1 where a padded batch has no token."""
    rows, n = case["rows"], case["n"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ids = (float(rows) ** u).long().sub_(1).clamp_(0, rows - 1)
    if case["pad"]:
        ids[torch.rand(n, generator=g, device="cuda") < case["pad"]] = -1
    return ids.to(torch.int32 if case["ids"] == "int32" else torch.int64)


def _normal(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda").to(DTYPES[dtype])


def _inputs(case, seed):
    g = _generator(seed)
    kind, rows, cols, n = case["kind"], case["rows"], case["cols"], case["n"]
    s = {"case": case}
    if kind in ("product", "lookup4"):
        s.update(_quantised(case, g))
    if kind == "product":
        s["x"] = _normal((n, cols), case["x"], g)
        if case["add"]:
            s["y"] = _normal((n, rows), case["y"], g)
        return s
    s["ids"] = _tokens(case, g)
    if kind == "lookup":
        s["table"] = _normal((rows, cols), case["table"], g)
    elif kind == "gradient":
        s["grad"] = _normal((n, cols), case["grad"], g)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and "codes" in s:
        # a program that serves a 4-bit model lays its weights out once, when it loads them
        import spmv_storage_formats_amd as spmv
        s["matrix"] = spmv.build_quant_packed(s["codes"], s["scales"], case["cols"],
                                              group_size=case["group"], zero_points=s["zeros"])
    return s


# ------------------------------------------------------------------ one pass

def _dense(codes, scales, zeros, case):
    """The values that 4-bit rows stand for, in 32 bits."""
    cols, group = case["cols"], case["group"]
    q = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)[:, :cols].float()
    wide = scales.float().repeat_interleave(group, 1)[:, :cols]
    if zeros is None:
        return (q - 8.0) * wide
    return (q - zeros.float().repeat_interleave(group, 1)[:, :cols]) * wide


def _plain(s):
    case = s["case"]
    kind, rows = case["kind"], case["rows"]
    if kind == "product":
        y = s["x"].float() @ _dense(s["codes"], s["scales"], s["zeros"], case).t()
        if case["add"]:
            y = y + s["y"].float()
        return y.to(DTYPES[case["y"]])
    ids = s["ids"].long()
    there = (ids >= 0) & (ids < rows)
    if kind == "gradient":
        total = torch.zeros(rows + 1, case["cols"], device="cuda")
        total.index_add_(0, torch.where(there, ids, rows), s["grad"].float())
        return (total[:rows] * case["scale"]).to(DTYPES[case["out"]])
    at = ids.clamp(0, rows - 1)
    if kind == "lookup":
        values = s["table"][at].float()
    else:
        zeros = None if s["zeros"] is None else s["zeros"][at]
        values = _dense(s["codes"][at], s["scales"][at], zeros, case)
    return torch.where(there[:, None], values * case["scale"], 0.0).to(DTYPES[case["out"]])


def run(state):
    if own:
        import spmv_storage_formats_amd as spmv
        case = state["case"]
        kind = case["kind"]
        if kind == "product":
            x = state["x"]
            if case["add"]:
                y = state["y"].clone()
            else:
                y = torch.empty(case["n"], case["rows"], dtype=DTYPES[case["y"]], device="cuda")
            return state["matrix"].run(x, y, accumulate=case["add"])
        if kind == "lookup":
            return spmv.lookup(state["table"], state["ids"], scale=case["scale"],
                               dtype=DTYPES[case["out"]])
        if kind == "lookup4":
            return state["matrix"].lookup(state["ids"], scale=case["scale"],
                                          dtype=DTYPES[case["out"]])
        return spmv.lookup_grad(state["grad"], state["ids"], case["rows"], scale=case["scale"],
                                dtype=DTYPES[case["out"]])
    return _plain(state)


# ------------------------------------------------------------------ the definition in 64 bits

def _row64(s, case, at):
    """Rows `at` of the 4-bit matrix, column by column as the layout defines them."""
    c = torch.arange(case["cols"], device="cuda")
    q = (s["codes"][at][:, c // 2] >> ((c % 2) * 4).to(torch.uint8)) & 15
    g = c // case["group"]
    z = 8.0 if s["zeros"] is None else s["zeros"][at][:, g].double()
    return s["scales"][at][:, g].double() * (q.double() - z)


def exact(case, seed):
    s = _inputs(case, seed)
    kind, rows, cols, n = case["kind"], case["rows"], case["cols"], case["n"]
    if kind == "product":
        x = s["x"].double()
        y = torch.empty(n, rows, dtype=torch.float64, device="cuda")
        for r in range(0, rows, 8192):
            at = torch.arange(r, min(rows, r + 8192), device="cuda")
            w = _row64(s, case, at)
            for v in range(n):
                y[v, at] = (w * x[v]).sum(1)
        return y + s["y"].double() if case["add"] else y
    ids = s["ids"].cpu().tolist()
    if kind == "gradient":
        # the tokens of each row, one after another: the t-th use of every row in one step
        turn, uses = {}, []
        for t, v in enumerate(ids):
            if 0 <= v < rows:
                k = turn.get(v, 0)
                turn[v] = k + 1
                if k == len(uses):
                    uses.append(([], []))
                uses[k][0].append(v)
                uses[k][1].append(t)
        out = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
        for to, of in uses:
            to, of = (torch.tensor(a, device="cuda") for a in (to, of))
            out[to] = out[to] + s["grad"][of].double()
        return out * case["scale"]
    out = torch.zeros(n, cols, dtype=torch.float64, device="cuda")
    kept = [t for t, v in enumerate(ids) if 0 <= v < rows]
    if kept:
        at = torch.tensor([ids[t] for t in kept], device="cuda")
        values = s["table"][at].double() if kind == "lookup" else _row64(s, case, at)
        out[torch.tensor(kept, device="cuda")] = values * case["scale"]
    return out
