"""Cases that measure the operators around the LM head: log-probabilities of given tokens with
entropy and top alternatives, the norm before the head with its gradients, and 8-bit activation
checkpoints. Where `own` is false, run() computes them in elementary torch operations; where it
is true, it makes the calls a user of this package makes."""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 32          # elements of an 8-bit checkpoint that share one power-of-two scale


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of one sequence on an 8B-class head: the weight's read is the time
        dict(name="stats one token", op="stats_rows", n=1, d=4096, v=128256, top=8, dtype="bf16", pad=0),
        # one step of a small server: hidden rows strided inside a wider buffer, 20 alternatives
        dict(name="stats 48 tokens", op="stats_rows", n=48, d=2048, v=151936, top=20, dtype="bf16", pad=64),
        # the smallest preference batch, exact fp32 route
        dict(name="stats tiny f32", op="stats_batch", r=4, l=32, d=64, v=1000, top=5, dtype="f32", ragged=1),
        # scoring a small model's batch, greedy alternative only, ragged rows and an empty one
        dict(name="stats small batch", op="stats_batch", r=16, l=512, d=2048, v=32000, top=1, dtype="bf16", ragged=2),
        # scoring a full preference batch at the 8B head
        dict(name="stats 8B batch", op="stats_batch", r=8, l=2048, d=4096, v=128256, top=8, dtype="bf16", ragged=3),
        # the final norm of a full batch: layer norm with bias
        dict(name="norm fwd 16384x4096", op="norm_fwd", rows=16384, d=4096, kind="layer", dtype="bf16", bias=True, pad=0),
        # the final norm of one decoding step
        dict(name="norm fwd 64x2048 rms", op="norm_fwd", rows=64, d=2048, kind="rms", dtype="bf16", bias=False, pad=0),
        # its backward on the fp32 dH that the head's backward writes
        dict(name="norm bwd 16384x4096", op="norm_bwd", rows=16384, d=4096, kind="layer", dtype="bf16", dy="f32", bias=True, pad=0),
        # odd sizes, fp32 throughout, strided input
        dict(name="norm bwd 1003x1000 f32", op="norm_bwd", rows=1003, d=1000, kind="layer", dtype="f32", dy="f32", bias=True, pad=24),
        # forward that keeps x in 8 bits, and the backward that reads it
        dict(name="norm 8-bit 16384x2048", op="norm_ckpt", rows=16384, d=2048, kind="rms", dtype="bf16", dy="f32", bias=False, pad=0),
        # hidden states of the offline scoring batch put away in 8 bits and brought back
        dict(name="8-bit 131072x4096", op="ckpt", rows=131072, d=4096, dtype="bf16", pad=0),
        # a few odd fp32 rows
        dict(name="8-bit 129x2056 f32", op="ckpt", rows=129, d=2056, dtype="f32", pad=8),
    ]


def _spread(rng, lo, hi, step=1):
    """A size of [lo, hi] spread over its logarithm, a multiple of step."""
    x = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(x) // step * step))


def draw(rng):
    op = rng.choice(["stats_rows", "stats_batch", "norm_fwd", "norm_bwd", "norm_ckpt", "ckpt"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    pad = rng.choice([0, 0, 8, 64])
    if op == "stats_rows":
        if dtype == "f32":
            return dict(op=op, n=_spread(rng, 1, 64), d=_spread(rng, 8, 512, 8), v=_spread(rng, 2, 4000),
                        top=rng.randint(0, 32), dtype=dtype, pad=pad)
        return dict(op=op, n=_spread(rng, 1, 512), d=_spread(rng, 64, 4096, 8), v=_spread(rng, 300, 151936),
                    top=rng.randint(0, 32), dtype=dtype, pad=pad)
    if op == "stats_batch":
        r = 2 * rng.randint(1, 6)
        ragged = rng.randint(1, 1 << 20)
        if dtype == "f32":
            return dict(op=op, r=r, l=_spread(rng, 3, 40), d=_spread(rng, 8, 256, 8), v=_spread(rng, 2, 4000),
                        top=rng.randint(0, 32), dtype=dtype, ragged=ragged)
        return dict(op=op, r=r, l=_spread(rng, 16, 900), d=_spread(rng, 64, 4096, 8), v=_spread(rng, 300, 151936),
                    top=rng.randint(0, 32), dtype=dtype, ragged=ragged)
    d = _spread(rng, 8, 8192, 8)
    rows = _spread(rng, 1, max(1, min(65536, (1 << 25) // d)))
    if op == "ckpt":
        return dict(op=op, rows=rows, d=d, dtype=dtype, pad=pad)
    kind = rng.choice(["layer", "rms"])
    case = dict(op=op, rows=rows, d=d, kind=kind, dtype=dtype, bias=kind == "layer" and rng.random() < 0.7, pad=pad)
    if op != "norm_fwd":
        case["dy"] = rng.choice(["bf16", "f32"])
    return case


def _lengths(case):
    """Prompt and completion lengths of a preference batch: the shape belongs to the case, not the seed."""
    rng = random.Random(case["ragged"])
    r, l = case["r"], case["l"]
    prompt = [rng.randint(1, max(1, l // 2)) for _ in range(r)]
    done = [rng.randint(max(0, int(0.95 * l) - p), l - p) if l >= 1024 else rng.randint(0, l - p) for p in prompt]
    done[0] = l - prompt[0]          # one row runs to its end
    if l < 1024:
        done[-1] = 0                 # one row scores nothing
    return prompt, done


def _bytes_of(name):
    return 4 if name == "f32" else 2


def work(case):
    op, e = case["op"], _bytes_of(case["dtype"])
    if op.startswith("stats"):
        n = case["n"] if op == "stats_rows" else sum(_lengths(case)[1])
        d, v = case["d"], case["v"]
        out = n * (12 + 8 * case["top"]) + (4 * case["r"] if op == "stats_batch" else 0)
        return {"bytes": (v * d + n * d) * e + 4 * n + out, "flops": 2.0 * n * v * d}
    cells = case["rows"] * case["d"]
    held = 1 + 1 / BLOCK
    if op == "ckpt":                 # packed once, read once
        return {"bytes": cells * (2 * e + 2 * held), "flops": 4.0 * cells}
    stats = case["rows"] * (4 if case["kind"] == "rms" else 8)
    vec = case["d"] * e * (2 if case["bias"] else 1)
    fwd = cells * 2 * e + stats + vec
    if op == "norm_fwd":
        return {"bytes": fwd, "flops": 8.0 * cells}
    grads = case["d"] * 4 * (2 if case["bias"] else 1)
    dy = _bytes_of(case["dy"])
    if op == "norm_bwd":
        return {"bytes": cells * (2 * e + dy) + stats + vec + grads, "flops": 12.0 * cells}
    return {"bytes": fwd + cells * held + cells * (held + dy + e) + stats + vec + grads, "flops": 24.0 * cells}


# ------------------------------------------------------------------ inputs
def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _grid(gen, shape, std, dtype):
    """Normal values on a grid of an eighth of the power of two next to std, cut at four of it: a dot product
    of two such vectors is a sum of few enough bits that 32-bit arithmetic holds it exactly in any order, so
    that which alternative comes first has one answer, ties included."""
    step = 2.0 ** (round(math.log2(std)) - 3)
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    return x.mul_(std / step).round_().clamp_(-32, 32).mul_(step).to(dtype)


def _rows(gen, rows, d, pad, dtype, channel):
    """Rows of a residual stream: normal values with some large channels, row stride d + pad."""
    x = torch.randn(rows, d + pad, generator=gen, device=DEV, dtype=torch.float32)
    x[:, :d] *= channel
    return x.to(dtype)[:, :d]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, d, dtype = case["op"], case["d"], _dtype(case["dtype"])
    s = dict(case=case)
    if op.startswith("stats"):
        s["w"] = _grid(gen, (case["v"], d), d ** -0.5, dtype)
        if op == "stats_rows":
            s["h"] = _grid(gen, (case["n"], d + case["pad"]), 1.0, dtype)[:, :d]
            s["tokens"] = torch.randint(0, case["v"], (case["n"],), generator=gen, device=DEV).int()
        else:
            s["prompt"], s["done"] = _lengths(case)
            s["h"] = _grid(gen, (case["r"], case["l"], d), 1.0, dtype)
            s["tokens"] = torch.randint(0, case["v"], (case["r"], case["l"]), generator=gen, device=DEV).int()
            # what the plain form indexes with: the flat position and the row of each scored token
            row = torch.tensor([i for i, c in enumerate(s["done"]) for _ in range(c)], dtype=torch.long)
            t = torch.tensor([p - 1 + j for p, c in zip(s["prompt"], s["done"]) for j in range(c)], dtype=torch.long)
            s["row"], s["at"] = row.to(DEV), (row * case["l"] + t).to(DEV)
        return s
    channel = torch.where(torch.rand(d, generator=gen, device=DEV) < 0.01, 20.0, 1.0)
    s["x"] = _rows(gen, case["rows"], d, case["pad"], dtype, channel)
    if op == "ckpt":
        return s
    s["eps"] = 1e-5
    s["weight"] = (1 + 0.1 * torch.randn(d, generator=gen, device=DEV)).to(dtype)
    s["bias"] = (0.1 * torch.randn(d, generator=gen, device=DEV)).to(dtype) if case["bias"] else None
    if op != "norm_fwd":
        dy = torch.randn(case["rows"], d, generator=gen, device=DEV) * 1e-3
        dy *= torch.rand(case["rows"], 1, generator=gen, device=DEV) < 0.75      # prompt and padding rows get no gradient
        s["dy"] = dy.to(_dtype(case["dy"]))
    if op == "norm_bwd":
        x = s["x"].double()
        mean = x.mean(1) if case["kind"] == "layer" else torch.zeros_like(x[:, 0])
        s["rstd"] = ((x - mean[:, None]).square().mean(1) + s["eps"]).rsqrt().float()
        s["mean"] = mean.float() if case["kind"] == "layer" else None
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _own(state)
    return globals()["_plain_" + state["case"]["op"].split("_")[0]](state)


def _plain_stats(s):
    case = s["case"]
    if case["op"] == "stats_rows":
        h, y = s["h"], s["tokens"].long()
    else:
        h, y = s["h"].reshape(-1, case["d"])[s["at"]], s["tokens"].reshape(-1)[s["at"] + 1].long()
    z = h.float() @ s["w"].float().T
    m = z.amax(1, keepdim=True)
    c = z - m
    e = c.exp()
    total = e.sum(1)
    lse = m[:, 0] + total.log()
    logp = z.gather(1, y[:, None])[:, 0] - lse
    out = dict(logp=logp, entropy=total.log() - e.mul_(c).sum(1) / total, lse=lse)
    del c, e
    if case["top"]:
        n = min(case["top"], case["v"])
        # a key orders the logits, equal ones by their id; its low half gives the id back
        bits = (z + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() << 32
        key += torch.arange(case["v"] - 1, -1, -1, device=z.device)
        best = case["v"] - 1 - (key.topk(n, dim=1).values & 0xFFFFFFFF)
        ids = torch.full((len(z), case["top"]), -1, dtype=torch.int32, device=z.device)
        top = torch.full((len(z), case["top"]), -math.inf, device=z.device)
        ids[:, :n] = best.int()
        top[:, :n] = z.gather(1, best) - lse[:, None]
        out.update(top_ids=ids, top_logp=top)
    if case["op"] == "stats_batch":
        out["seq_logp"] = torch.zeros(case["r"], dtype=torch.float64, device=z.device).index_add_(0, s["row"], logp.double()).float()
    return out


def _held(x):
    """x as an 8-bit checkpoint holds it: blocks of 32 along the row, codes of -127 to 127 times a power of two."""
    rows, d = x.shape
    b = torch.nn.functional.pad(x.float(), (0, -d % BLOCK)).view(rows, -1, BLOCK)
    m, k = torch.frexp(b.abs().amax(2, keepdim=True))
    power = torch.where(m > 127 / 128, k - 6, k - 7).clamp(-126, 121)
    up, down = (((127 + sign * power) << 23).view(torch.float32) for sign in (1, -1))
    return ((b * down).round() * up).view(rows, -1)[:, :d]


def _plain_ckpt(s):
    return dict(x=_held(s["x"]).to(s["x"].dtype))


def _forward(x, s):
    mean = x.mean(1) if s["case"]["kind"] == "layer" else None
    c = x - mean[:, None] if mean is not None else x
    rstd = (c.square().mean(1) + s["eps"]).rsqrt()
    y = c * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y, mean, rstd


def _backward(x, mean, rstd, s):
    dy = s["dy"].float()
    xh = (x - mean[:, None] if mean is not None else x) * rstd[:, None]
    g = dy * s["weight"].float()
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if mean is not None:
        dx = dx - g.mean(1, keepdim=True)
    out = dict(dx=(dx * rstd[:, None]).to(s["x"].dtype), dweight=(dy * xh).sum(0))
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


def _plain_norm(s):
    op = s["case"]["op"]
    out = {}
    if op != "norm_bwd":
        y, mean, rstd = _forward(s["x"].float(), s)
        out = dict(y=y.to(s["x"].dtype), rstd=rstd)
        if mean is not None:
            out["mean"] = mean
    if op == "norm_bwd":
        out = _backward(s["x"].float(), s["mean"], s["rstd"], s)
    elif op == "norm_ckpt":
        out.update(_backward(_held(s["x"]), mean, rstd, s))
    return out


# ------------------------------------------------------------------ the package's calls
def _plan(s):
    """What a user's program keeps for one shape: its output buffers, its workspace and the batch's description."""
    from preference_alignment_b200 import libdpo
    case = s["case"]
    op, d = case["op"], case["d"]

    def f32(*shape):
        return torch.empty(shape, device=DEV)

    def space(n):
        return torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)

    if op.startswith("stats"):
        if op == "stats_rows":
            n = case["n"]
            ws, _ = libdpo.token_stats_rows_size(n, d, case["v"], case["top"], dtype=case["dtype"])
            p = {}
        else:
            n = sum(s["done"])
            p = dict(batch=libdpo.BatchArgs(s["h"], s["w"], s["tokens"], s["prompt"], s["done"], dtype=case["dtype"]))
            ws, _ = libdpo.token_stats_size(p["batch"], case["top"])
        p["ws"] = space(ws)
        p["out"] = dict(logp=f32(n), entropy=f32(n), lse_state=f32(n))
        if case["top"]:
            p["out"].update(top_ids=torch.empty(n, case["top"], dtype=torch.int32, device=DEV), top_logp=f32(n, case["top"]))
        if op == "stats_batch":
            p["out"]["seq_logp"] = f32(case["r"])
        return p
    rows, x = case["rows"], s["x"]
    p = {}
    if op in ("ckpt", "norm_ckpt"):
        p["held"] = libdpo.Checkpoint(torch.empty(rows, d, dtype=torch.int8, device=DEV),
                                      torch.empty(rows, -(-d // BLOCK), dtype=torch.uint8, device=DEV))
    if op == "ckpt":
        p["out"] = dict(x=torch.empty(rows, d, dtype=x.dtype, device=DEV))
        return p
    layer = case["kind"] == "layer"
    if op != "norm_bwd":
        p["fwd"] = dict(y=torch.empty(rows, d, dtype=x.dtype, device=DEV), rstd=f32(rows))
        if layer:
            p["fwd"]["mean"] = f32(rows)
    if op != "norm_fwd":
        p["ws"] = space(libdpo.norm_workspace_size(rows, d))
        p["bwd"] = dict(dx=torch.empty(rows, d, dtype=x.dtype, device=DEV), dweight=f32(d))
        if s["bias"] is not None:
            p["bwd"]["dbias"] = f32(d)
    return p


def _own(s):
    from preference_alignment_b200 import libdpo
    if "plan" not in s:
        s["plan"] = _plan(s)
    case, p = s["case"], s["plan"]
    op = case["op"]
    if op == "stats_rows":
        libdpo.token_stats_rows(s["h"], s["w"], s["tokens"], case["top"], ws=p["ws"], **p["out"])
    elif op == "stats_batch":
        libdpo.token_stats(p["batch"], case["top"], ws=p["ws"], **p["out"])
    elif op == "ckpt":
        libdpo.checkpoint_pack(s["x"], p["held"])
        libdpo.checkpoint_unpack(p["held"], p["out"]["x"])
    if op in ("stats_rows", "stats_batch", "ckpt"):
        out = dict(p["out"])
        if "lse_state" in out:
            out["lse"] = out.pop("lse_state")
        return out
    kind, w = case["kind"], s["weight"]
    if op == "norm_fwd":
        libdpo.norm_forward(s["x"], weight=w, bias=s["bias"], kind=kind, eps=s["eps"], **p["fwd"])
        return p["fwd"]
    if op == "norm_bwd":
        libdpo.norm_backward(s["x"], s["dy"], s["mean"], s["rstd"], weight=w, kind=kind, ws=p["ws"], **p["bwd"])
        return p["bwd"]
    fwd = p["fwd"]
    libdpo.norm_forward(s["x"], weight=w, bias=s["bias"], kind=kind, eps=s["eps"], save=p["held"], **fwd)
    libdpo.norm_backward(p["held"], s["dy"], fwd.get("mean"), fwd["rstd"], weight=w, kind=kind, ws=p["ws"], **p["bwd"])
    return {**fwd, **p["bwd"]}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exact_stats(case, s):
    d = case["d"]
    h = s["h"].double().reshape(-1, d)
    if case["op"] == "stats_rows":
        y, rows = s["tokens"].long(), None
    else:
        keep, y, rows = [], [], []
        tokens = s["tokens"].cpu()
        for r, (p, c) in enumerate(zip(s["prompt"], s["done"])):
            for j in range(p, p + c):
                keep.append(r * case["l"] + j - 1)
                y.append(int(tokens[r, j]))
                rows.append(r)
        h, y = h[torch.tensor(keep, dtype=torch.long, device=DEV)], torch.tensor(y, dtype=torch.long, device=DEV)
    w = s["w"].double()
    parts = []
    for a in range(0, len(h), 2048):
        lp = torch.log_softmax(h[a:a + 2048] @ w.T, dim=1)
        z0 = h[a:a + 2048] @ w[0]
        best = lp.topk(min(case["top"], case["v"]), dim=1).values
        best = torch.nn.functional.pad(best, (0, case["top"] - best.shape[1]), value=-math.inf)
        parts.append((lp.gather(1, y[a:a + 2048, None])[:, 0], -(lp.exp() * lp).sum(1), z0 - lp[:, 0], best))
    if not parts:
        return None
    logp, entropy, lse, best = (torch.cat(p) for p in zip(*parts))
    out = dict(logp=logp, entropy=entropy, lse=lse)
    if case["top"]:
        out.update(top_ids=None, top_logp=best)
    if rows is not None:
        total = [0.0] * case["r"]
        for r, v in zip(rows, logp.tolist()):
            total[r] += v
        out["seq_logp"] = torch.tensor(total, dtype=torch.float64)
    return out


def _exact_held(x):
    rows, d = x.shape
    out = torch.zeros(rows, d, dtype=torch.float64, device=x.device)
    for a in range(0, d, BLOCK):
        b = x[:, a:a + BLOCK].double()
        scale = torch.exp2(torch.ceil(torch.log2(b.abs().amax(1, keepdim=True).clamp_min(2.0 ** -119) / 127)))
        scale = torch.where(b.abs().amax(1, keepdim=True) <= 127 * scale / 2, scale / 2, scale)
        scale = torch.where(b.abs().amax(1, keepdim=True) > 127 * scale, scale * 2, scale)
        out[:, a:a + BLOCK] = torch.round(b / scale) * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("stats"):
        return _exact_stats(case, s)
    if case["op"] == "ckpt":
        return dict(x=_exact_held(s["x"]))
    x, w = s["x"].double(), s["weight"].double()
    layer, out = case["kind"] == "layer", {}
    if case["op"] != "norm_bwd":
        mean = x.sum(1) / case["d"] if layer else torch.zeros(len(x), dtype=torch.float64, device=DEV)
        rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).sum(1) / case["d"] + s["eps"])
        out = dict(y=(x - mean[:, None]) * rstd[:, None] * w + (s["bias"].double() if s["bias"] is not None else 0), rstd=rstd)
        if layer:
            out["mean"] = mean
    if case["op"] == "norm_fwd":
        return out
    if case["op"] == "norm_bwd":
        rstd = s["rstd"].double()
        mean = s["mean"].double() if layer else torch.zeros_like(rstd)
    else:
        x = _exact_held(s["x"])
    dy = s["dy"].double()
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    along = (g * xh).sum(1, keepdim=True) / case["d"]
    out["dx"] = rstd[:, None] * (g - xh * along - (g.sum(1, keepdim=True) / case["d"] if layer else 0))
    out["dweight"] = torch.einsum("rd,rd->d", dy, xh)
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out
