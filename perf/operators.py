"""Gradient-norm clipping around the shard step: the cases that are timed, their plain forms and their definitions in 64 bits.

Four operators:
  norm    squares of many gradient tensors: per tensor, in all, and the global norm
  clip    that norm, then every tensor times the clipping coefficient into its place in another buffer
  reduce  the mean of N gradient partials of one shard, and its square in the same pass
  step    a whole clipped optimizer step of one shard: reduce, coefficient over all ranks' squares, AdamW, bf16 parameters

With `own` false, run() computes in elementary torch operations; with `own` true it calls the library.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6                      # added to the norm in the coefficient
BETA1, BETA2, ADAM_EPS, DECAY, LR, STEP = 0.9, 0.999, 1e-8, 0.1, 1e-3, 100


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the smallest: a few dozen odd tensors (adapters, norms, biases), where latency is all
        {"name": "norm of 37 small tensors fp32", "op": "norm", "form": "ragged", "count": 37, "low": 1, "high": 20000, "sizes": 1, "types": "fp32", "sigma": 1e-2, "max_norm": 1.0, "scale": 1.0},
        # GPT-2 small's whole gradient on one GPU, as plain data parallelism clips it
        {"name": "norm of GPT-2 small bf16", "op": "norm", "form": "gpt2", "layers": 12, "width": 768, "vocab": 50257, "types": "bf16", "sigma": 1e-3, "max_norm": 1.0, "scale": 1.0},
        # many tensors of every size whose types differ (fp32 norms beside 16-bit weights), packed with no padding
        {"name": "norm of 1200 ragged mixed", "op": "norm", "form": "ragged", "count": 1200, "low": 64, "high": 1 << 20, "sizes": 2, "types": "mixed", "sigma": 1e-3, "max_norm": 1.0, "scale": 1.0},
        # fine-tuning with loss scaling: few small tensors unscaled and clipped
        {"name": "clip of 24 small tensors mixed", "op": "clip", "form": "ragged", "count": 24, "low": 1, "high": 5000, "sizes": 3, "types": "mixed", "to": "same", "sigma": 1e-2, "max_norm": 0.05, "scale": 1.0 / 16},
        # 16-bit gradients clipped into the fp32 main gradients that an optimizer reads
        {"name": "clip of GPT-2 small bf16 to fp32", "op": "clip", "form": "gpt2", "layers": 12, "width": 768, "vocab": 50257, "types": "bf16", "to": "fp32", "sigma": 1e-3, "max_norm": 1.0, "scale": 1.0},
        # four layers and both embeddings of a 7B Llama, clipped into the communication buffer in their own type
        {"name": "clip of Llama-7B 4 layers bf16", "op": "clip", "form": "llama", "layers": 4, "width": 4096, "ff": 11008, "vocab": 32000, "types": "bf16", "to": "same", "sigma": 1e-4, "max_norm": 1.0, "scale": 1.0},
        # one shard of a 1M-parameter model on four ranks
        {"name": "reduce tiny 4 ranks bf16", "op": "reduce", "numel": 262144, "ranks": 4, "type": "bf16", "group": 0, "micro": 1, "sigma": 1e-3, "max_norm": 0.1},
        # a 2B ragged model on 32 ranks with fp32 communication: the most bytes read an element
        {"name": "reduce ragged 32 ranks fp32", "op": "reduce", "numel": 62500000, "ranks": 32, "type": "fp32", "group": 0, "micro": 1, "sigma": 1e-4, "max_norm": 0.05},
        # the whole clipped step at the smallest shard
        {"name": "step tiny 4 ranks bf16", "op": "step", "state": "fp32", "numel": 262144, "ranks": 4, "type": "bf16", "skew": 0, "sigma": 1e-3, "max_norm": 0.1},
        # GPT-2 small's shard on 8 ranks, pure bf16 state, its slot at an odd element
        {"name": "step GPT-2 small 8 ranks kahan", "op": "step", "state": "kahan", "numel": 15554976, "ranks": 8, "type": "bf16", "skew": 3, "sigma": 1e-3, "max_norm": 1.0},
        # a 512-GPU shard of a 70B model reduced over 16 replicas, 12 bytes of state a parameter
        {"name": "step 70B shard 16 ranks bf16m", "op": "step", "state": "bf16m", "numel": 137800208, "ranks": 16, "type": "bf16", "skew": 0, "sigma": 1e-4, "max_norm": 1.0},
        # Llama-7B's rank-0 shard of 8: the largest
        {"name": "step Llama-7B shard 8 ranks fp32", "op": "step", "state": "fp32", "numel": 842301952, "ranks": 8, "type": "bf16", "skew": 0, "sigma": 1e-4, "max_norm": 1.0},
    ]


def _spread(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm", "clip", "reduce", "step"])
    max_norm = rng.choice([0.05, 0.5, 1.0, 100.0])          # the last leaves most gradients as they are
    if op in ("norm", "clip"):
        scale = rng.choice([1.0, 1.0, 1.0 / 64])
        case = {"op": op, "types": rng.choice(["bf16", "fp16", "fp32", "mixed"]), "sigma": 1e-3 / scale, "max_norm": max_norm, "scale": scale}
        if op == "clip":
            case["to"] = rng.choice(["same", "fp32", "bf16"])
            if case["to"] == "same" and case["types"] in ("fp16", "mixed"):
                case["max_norm"] = max(max_norm, 1.0)   # so that the results stay among fp16's normal numbers
        if rng.random() < 0.7:
            case.update(form="ragged", count=_spread(rng, 1, 1500), low=1, high=_spread(rng, 100, 1 << 20), sizes=rng.randrange(1 << 20))
        else:
            case.update(form="gpt2", layers=rng.randrange(1, 13), width=64 * rng.randrange(2, 13), vocab=_spread(rng, 1000, 50257))
        return case
    ranks = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 32])
    kind = rng.choice(["bf16", "bf16", "fp32"])
    # at most 8 GB of partials
    numel = _spread(rng, 70001, min(100000000, 8000000000 // (ranks * (2 if kind == "bf16" else 4))))
    case = {"op": op, "numel": numel, "ranks": ranks, "type": kind, "sigma": 10 ** rng.uniform(-4, -2), "max_norm": max_norm}
    if op == "reduce":
        case.update(group=rng.choice([0, 1] + ([ranks // 2] if ranks % 2 == 0 else [])), micro=rng.choice([1, 1, 3]))
    else:
        case.update(state=rng.choice(["fp32", "bf16m", "kahan"]), skew=rng.randrange(0, 8))
    return case


def _sizes(case):
    """The tensors' element counts, in model order."""
    if case["form"] == "ragged":
        r = random.Random(case["sizes"])
        return [_spread(r, case["low"], case["high"]) for _ in range(case["count"])]
    d, layers, vocab = case["width"], case["layers"], case["vocab"]
    if case["form"] == "gpt2":
        block = [d, d, 3 * d * d, 3 * d, d * d, d, d, d, 4 * d * d, 4 * d, 4 * d * d, d]
        return [vocab * d, 1024 * d] + layers * block + [d, d]
    ff = case["ff"]
    block = [d] + 4 * [d * d] + [d] + 3 * [d * ff]
    return [vocab * d] + layers * block + [d, vocab * d]


def _type_names(case, count):
    if case["types"] == "mixed":
        r = random.Random(count)
        return [r.choice(["bf16", "fp16", "fp32"]) for _ in range(count)]
    return [case["types"]] * count


# ------------------------------------------------------------------ inputs

def _packed(sizes, names, fill=None):
    """One flat buffer for each type, with no padding between its tensors, and the tensors as views in order."""
    flat = {n: torch.empty(sum(s for s, t in zip(sizes, names) if t == n), dtype=TYPES[n], device="cuda") for n in sorted(set(names))}
    if fill is not None:
        for n in flat:
            fill(flat[n])
    views, at = [], dict.fromkeys(flat, 0)
    for s, n in zip(sizes, names):
        views.append(flat[n][at[n]:at[n] + s])
        at[n] += s
    return flat, views


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = {"case": case}

    def normal(n, dtype, sigma):
        return torch.empty(n, dtype=dtype, device="cuda").normal_(0.0, sigma, generator=gen)

    if case["op"] in ("norm", "clip"):
        sizes = _sizes(case)
        names = _type_names(case, len(sizes))
        _, state["grads"] = _packed(sizes, names, lambda t: t.normal_(0.0, case["sigma"], generator=gen))
        if case["op"] == "clip":
            to = names if case["to"] == "same" else [case["to"]] * len(sizes)
            state["out"], state["places"] = _packed(sizes, to)
        if own:
            import sharded_optimizer_step_shard_amd as zs
            table = zs.zero_build_pieces(state["grads"], state.get("places"))
            state["n_pieces"], state["pieces"] = len(table), zs.pieces_to_device(table)
            state["work"] = torch.empty(zs.zero_norm_workspace(len(table)), dtype=torch.uint8, device="cuda")
            state["tensor_sq"] = torch.empty(len(sizes), dtype=torch.float64, device="cuda")
            state["sq"] = torch.empty(1, dtype=torch.float64, device="cuda")
            state["result"] = torch.empty(2, dtype=torch.float64, device="cuda")
            state["spec"] = zs.clip_spec(state["result"], case["max_norm"], EPS, case["scale"])
        return state

    n, ranks = case["numel"], case["ranks"]
    kind = TYPES[case["type"]]
    state["partials"] = [normal(n, kind, case["sigma"]) for _ in range(ranks)]
    if case["op"] == "reduce":
        state["acc"] = normal(n, torch.float32, case["sigma"] * math.sqrt(ranks * (case["micro"] - 1.0))) if case["micro"] > 1 else None
    else:
        narrow = torch.float32 if case["state"] == "fp32" else torch.bfloat16
        # this rank's slot lies `skew` elements into an aligned buffer
        state["param"] = normal(n + case["skew"], torch.bfloat16, 0.02)[case["skew"]:]
        state["weight"] = normal(n, torch.float32, 0.02) if case["state"] != "kahan" else torch.zeros(n, dtype=torch.bfloat16, device="cuda")
        state["m"] = normal(n, narrow, 0.1 * case["sigma"])
        state["v"] = normal(n, narrow, 0.3 * case["sigma"]).square_()
        # the other ranks' squares, as their all-gather brings them; this rank's comes first
        state["squares"] = n * case["sigma"] ** 2 / ranks * (0.9 + 0.2 * torch.rand(ranks, dtype=torch.float64, device="cuda", generator=gen))
    if own:
        import sharded_optimizer_step_shard_amd as zs
        state["work"] = torch.empty(zs.zero_norm_workspace(), dtype=torch.uint8, device="cuda")
        state["result"] = torch.empty(2, dtype=torch.float64, device="cuda")
        state["spec"] = zs.clip_spec(state["result"], case["max_norm"], EPS)
        # up to 4 bytes of partials an element are cheaper to reduce twice than to write and read as fp32
        keep = case["op"] == "reduce" or ranks * kind.itemsize > 4
        state["grad"] = torch.empty(n, dtype=torch.float32, device="cuda") if keep else None
        if case["op"] == "reduce":
            state["sq"] = torch.empty(1, dtype=torch.float64, device="cuda")
        else:
            table, _ = zs.zero_build_chunks([n], 1, 0, slot_dst=state["param"].data_ptr(), max_chunk=zs.ZERO_DEFAULT_MAX_CHUNK_REDUCED)
            state["n_chunks"], state["chunks"] = len(table), zs.chunks_to_device(table)
            state["mine"] = state["squares"][:1]
    return state


# ------------------------------------------------------------------ the plain forms

def _coefficient(sq, case):
    """[norm, coefficient] from the sum of squares, 64 bits."""
    scale = case.get("scale", 1.0)
    norm = sq.sqrt() * scale
    return torch.stack([norm, (case["max_norm"] / (norm + EPS)).clamp(max=1.0) * scale])


def _mean(state):
    """The mean of the partials in 64 bits, rounded once."""
    case = state["case"]
    k = case.get("group", 0) or case["ranks"]
    sums = [sum(p.double() for p in state["partials"][i:i + k]) for i in range(0, case["ranks"], k)]
    s = sum(sums)
    if state.get("acc") is not None:
        s = s + state["acc"].double()
    return (s / (case["ranks"] * case.get("micro", 1))).float()


def _adamw(g, m, v):
    """AdamW's new moments and direction, in the type of the arguments."""
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * g * g
    return m, v, (m / (1.0 - BETA1 ** STEP)) / ((v / (1.0 - BETA2 ** STEP)).sqrt() + ADAM_EPS)


def _plain_step(state):
    case = state["case"]
    g = _mean(state)
    state["squares"][0] = g.double().square().sum()
    result = _coefficient(state["squares"].sum(), case)
    g = (g.double() * result[1]).float()
    weight, m, v, param = (state[k] for k in ("weight", "m", "v", "param"))
    if case["state"] == "kahan":
        # 64 bits: what the compensation holds turns on the parameter's rounding
        m1, v1, u = _adamw(g.double(), m.double(), v.double())
        y = -LR * (u + DECAY * param.double()) + weight.double()
        moved = _bf16(param.double() + y)
        weight.copy_(_bf16(y - (moved.double() - param.double())))
        param.copy_(moved)
        m.copy_(_bf16(m1))
        v.copy_(_bf16(v1))
    else:
        m1, v1, u = _adamw(g, m.float(), v.float())
        weight.copy_(weight * (1.0 - LR * DECAY) - LR * u)
        m.copy_(m1)
        v.copy_(v1)
        param.copy_(weight)
    return result


def _bf16(x):
    """64 bits to bf16 in one rounding: by way of 32 bits rounded to odd."""
    f = x.float()
    up = f.double().abs() > x.abs()
    odd = (f.view(torch.int32) - up.int()) | (f.double() != x).int()
    return odd.view(torch.float32).bfloat16()


def _plain(state):
    case = state["case"]
    if case["op"] in ("norm", "clip"):
        tensor_sq = torch.stack([g.double().square().sum() for g in state["grads"]])
        result = _coefficient(tensor_sq.sum(), case)
        if case["op"] == "clip":
            [p.copy_(g.float() * result[1]) for g, p in zip(state["grads"], state["places"])]
        return tensor_sq, result
    if case["op"] == "reduce":
        g = _mean(state)
        return g, _coefficient(g.double().square().sum(), case)
    return None, _plain_step(state)


# ------------------------------------------------------------------ the library's calls

def _library(state):
    import sharded_optimizer_step_shard_amd as zs
    case = state["case"]
    if case["op"] in ("norm", "clip"):
        zs.zero_norm_pieces(state["pieces"], state["n_pieces"], state["sq"], state["work"], tensor_sq=state["tensor_sq"], spec=state["spec"])
        if case["op"] == "clip":
            zs.zero_scale_pieces(state["pieces"], state["n_pieces"], state["result"])
        return state["tensor_sq"], state["result"]
    n, grad = case["numel"], state["grad"]
    if case["op"] == "reduce":
        zs.zero_reduce_norm_shard(state["partials"], n, state["sq"], state["work"], grad_out=grad, group=case["group"], micro_batches=case["micro"], acc=state["acc"], spec=state["spec"])
        return grad, state["result"]
    zs.zero_reduce_norm_shard(state["partials"], n, state["mine"], state["work"], grad_out=grad)
    zs.zero_clip_coef(state["squares"], case["ranks"], state["spec"])
    step = {"fp32": zs.zero_shard_step_clipped, "bf16m": zs.zero_shard_step_bf16_moments_clipped, "kahan": zs.zero_shard_step_kahan_clipped}[case["state"]]
    step(state["partials"] if grad is None else [grad], state["weight"], state["m"], state["v"], n, state["chunks"], state["n_chunks"],
         zs.hparams(STEP, LR, BETA1, BETA2, ADAM_EPS, DECAY), state["result"])
    return None, state["result"]


def run(state):
    case = state["case"]
    first, result = _library(state) if own else _plain(state)
    if case["op"] == "norm":
        return {"squares": first, "norm": result}
    if case["op"] == "clip":
        return {"squares": first, "norm": result, "clipped": state["out"]}
    if case["op"] == "reduce":
        return {"gradient": first, "norm": result}
    return {"norm": result, **{k: state[k] for k in ("weight", "m", "v", "param")}}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"] in ("norm", "clip"):
        sizes = _sizes(case)
        names = _type_names(case, len(sizes))
        total = sum(sizes)
        moved = sum(s * size[n] for s, n in zip(sizes, names)) + 8 * len(sizes)
        if case["op"] == "clip":
            moved += sum(s * size[n if case["to"] == "same" else case["to"]] for s, n in zip(sizes, names))
        return {"bytes": moved, "flops": total * (2 if case["op"] == "norm" else 3)}
    n, ranks = case["numel"], case["ranks"]
    read = ranks * size[case["type"]]
    if case["op"] == "reduce":
        return {"bytes": n * (read + 4 + (4 if case["micro"] > 1 else 0)), "flops": n * (ranks + 3)}
    return {"bytes": n * (read + {"fp32": 26, "bf16m": 18, "kahan": 16}[case["state"]]), "flops": n * (ranks + 20)}


# ------------------------------------------------------------------ the definitions in 64 bits

def _clipping(sq, case):
    s = case.get("scale", 1.0)
    norm = s * math.sqrt(sq)
    c = s if norm + EPS <= case["max_norm"] else s * case["max_norm"] / (norm + EPS)
    return norm, c, torch.tensor([norm, c], dtype=torch.float64)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] in ("norm", "clip"):
        wide = [g.to(torch.float64) for g in state["grads"]]
        per = torch.stack([torch.dot(w, w) for w in wide])
        _, c, norm = _clipping(math.fsum(per.tolist()), case)
        if case["op"] == "norm":
            return {"squares": per, "norm": norm}
        names = _type_names(case, len(wide))
        into = names if case["to"] == "same" else [case["to"]] * len(wide)
        return {"squares": per, "norm": norm, "clipped": {n: torch.cat([c * w for w, t in zip(wide, into) if t == n]) for n in sorted(set(into))}}
    n, ranks = case["numel"], case["ranks"]
    g = torch.zeros(n, dtype=torch.float64, device="cuda")
    for p in state["partials"]:
        g += p
    if case.get("micro", 1) > 1:
        g += state["acc"]
    g /= ranks * case.get("micro", 1)
    mine = float(torch.dot(g, g))
    if case["op"] == "reduce":
        return {"gradient": g, "norm": _clipping(mine, case)[2]}
    _, c, norm = _clipping(math.fsum([mine] + state["squares"][1:].tolist()), case)
    g *= c
    m = torch.lerp(g, state["m"].double(), BETA1)
    v = torch.lerp(g * g, state["v"].double(), BETA2)
    u = m / (torch.sqrt(v / (1 - BETA2 ** STEP)) + ADAM_EPS) / (1 - BETA1 ** STEP)
    old = (state["param"] if case["state"] == "kahan" else state["weight"]).double()
    new = old - LR * (u + DECAY * old)
    if case["state"] == "kahan":   # the compensation starts at zero; what it is left with is the parameter's own rounding
        return {"norm": norm, "weight": None, "m": m, "v": v, "param": new}
    return {"norm": norm, "weight": new, "m": m, "v": v, "param": new}
