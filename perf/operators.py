"""Workloads of the Muon operators: orthogonalisation of a batch of matrices,
the sharded Muon step with its momentum in fp32 or in 8-bit blocks, and the
conversion of a momentum state between the two.

`own` selects what run() calls: the plain form (elementary torch operations
in fp32) or the package's operators.
"""
import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
STEPS = 5
MU, WEIGHT_DECAY = 0.95, 0.1
BLOCK = 256            # elements that share one scale of an 8-bit momentum
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One small matrix (an adapter, a toy model): what a call costs at least.
        {"name": "ortho 1x128x128 bf16", "op": "ortho", "batch": 1, "m": 128, "n": 128, "dtype": "bf16", "pad": 0, "steps": 5},
        # Odd extents and padded rows: views into a larger gradient buffer.
        {"name": "ortho 6x777x1025 f32", "op": "ortho", "batch": 6, "m": 777, "n": 1025, "dtype": "f32", "pad": 3, "steps": 5},
        # The up projections of three blocks of the 1.3B set, as one batch.
        {"name": "ortho 3x2048x8192 bf16", "op": "ortho", "batch": 3, "m": 2048, "n": 8192, "dtype": "bf16", "pad": 0, "steps": 5},
        # One gate matrix of the 7B set: tall, the largest matrix of its block.
        {"name": "ortho 1x11008x4096 f32", "op": "ortho", "batch": 1, "m": 11008, "n": 4096, "dtype": "f32", "pad": 0, "steps": 5},
        # The matrices of the tiny set, two replicas: a launch-bound step.
        {"name": "muon tiny w2", "op": "muon", "set": "tiny", "blocks": 1, "world": 2, "rank": 0, "state": "f32", "lr": 3e-4},
        # Odd matrices and a batch of experts, three replicas: nothing is aligned.
        {"name": "muon odd w3", "op": "muon", "set": "odd", "blocks": 2, "world": 3, "rank": 1, "state": "f32", "lr": 3e-4},
        # One rank's matrices of the 7B set at 64 replicas: the fold weighs as much as the products.
        {"name": "muon 7b w64", "op": "muon", "set": "7b", "blocks": 32, "world": 64, "rank": 0, "state": "f32", "lr": 3e-4},
        # The same steps with the momentum in 8 bits.
        {"name": "muon8 tiny w2", "op": "muon", "set": "tiny", "blocks": 1, "world": 2, "rank": 0, "state": "int8", "lr": 3e-4},
        {"name": "muon8 odd w3", "op": "muon", "set": "odd", "blocks": 2, "world": 3, "rank": 1, "state": "int8", "lr": 3e-4},
        # One rank's matrices of the 1.3B set at 8 replicas.
        {"name": "muon8 1p3b w8", "op": "muon", "set": "1p3b", "blocks": 24, "world": 8, "rank": 3, "state": "int8", "lr": 3e-4},
        # An fp32 momentum taken into 8 bits and back (resuming from and saving an fp32 state).
        {"name": "convert odd", "op": "convert", "set": "odd", "blocks": 2, "world": 3, "rank": 1},
        {"name": "convert 1p3b", "op": "convert", "set": "1p3b", "blocks": 24, "world": 8, "rank": 3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        while True:
            m, n, batch = _log(rng, 16, 11008), _log(rng, 16, 11008), _log(rng, 1, 24)
            if batch * min(m, n) ** 2 * max(m, n) <= 1.5e11 and batch * m * n <= 1e8:
                break
        return {"op": "ortho", "batch": batch, "m": m, "n": n, "dtype": rng.choice(["f32", "bf16", "f16"]),
                "pad": rng.choice([0, 0, 1, 8]), "steps": rng.choice([3, 5, 5, 6])}
    name, most = rng.choice([("tiny", 1), ("odd", 8), ("1p3b", 24), ("7b", 8)])
    world = rng.choice([1, 2, 3, 5, 8, 16])
    # at most two blocks' matrices of the 1.3B set on one rank, and half a block's of the 7B set
    if name == "7b":
        world = max(world, 2)
    most = min(most, 2 * world if name == "1p3b" else world // 2 if name == "7b" else most)
    case = {"op": rng.choice(["muon", "muon", "muon", "convert"]), "set": name, "blocks": rng.randint(1, most), "world": world}
    case["rank"] = rng.randrange(min(world, len(_shapes(case))))        # every one of these owns a matrix
    if case["op"] == "muon":
        case["state"] = rng.choice(["f32", "int8"])
        case["lr"] = rng.uniform(3e-5, 3e-4)
    return case


def _shapes(case):
    name, blocks = case["set"], case["blocks"]
    if name == "tiny":
        return [(512, 512), (512, 1024), (1024, 512)]
    if name == "odd":
        return [(333, 517), (1001, 77), (5, 130, 66), (1, 2000), (640, 1)] * blocks
    if name == "1p3b":
        return [(2048, 6144), (2048, 2048), (2048, 8192), (8192, 2048)] * blocks
    return [(4096, 4096)] * (4 * blocks) + [(11008, 4096)] * (2 * blocks) + [(4096, 11008)] * blocks


def _owned(case):
    """The rank's tensors, in declaration order: largest first (ties by
    index) to the least loaded rank (ties by the lowest)."""
    shapes = _shapes(case)
    size = [math.prod(s) for s in shapes]
    load, mine = [0] * case["world"], []
    for t in sorted(range(len(shapes)), key=lambda t: (-size[t], t)):
        r = load.index(min(load))
        load[r] += size[t]
        if r == case["rank"]:
            mine.append(t)
    return [shapes[t] for t in sorted(mine)]


def work(case):
    def products(batch, m, n, steps):
        g, l = min(m, n), max(m, n)
        return float(batch) * steps * (3 * g * g * l + g ** 3)      # the two Gram products are symmetric

    if case["op"] == "ortho":
        b, m, n = case["batch"], case["m"], case["n"]
        return {"bytes": float(b) * m * n * ({"f32": 4}.get(case["dtype"], 2) + 2), "flops": products(b, m, n, case["steps"])}
    owned = _owned(case)
    numel = float(sum(math.prod(s) for s in owned))
    scales = numel / BLOCK * 4
    if case["op"] == "convert":
        return {"bytes": numel * 10 + 2 * scales + 16, "flops": 0.0}
    momentum = 8 * numel if case["state"] == "f32" else 2 * numel + 2 * scales
    return {"bytes": numel * (2 * case["world"] + 8 + 2) + momentum + 16,
            "flops": sum(products(math.prod(s[:-2]), s[-2], s[-1], STEPS) for s in owned) + 16}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _low_rank_plus_noise(gen, batch, m, n, sigma):
    """What a weight's gradient looks like: a few strong directions and noise."""
    r = min(8, m, n)
    u = torch.randn(batch, m, r, generator=gen, device="cuda")
    v = torch.randn(batch, r, n, generator=gen, device="cuda")
    x = torch.randn(batch, m, n, generator=gen, device="cuda")
    return x.add_(torch.bmm(u, v), alpha=0.25).mul_(sigma)


def _inputs(case, seed):
    gen = _gen(seed)
    if case["op"] == "ortho":
        b, m, n = case["batch"], case["m"], case["n"]
        x = torch.zeros(b, m, n + case["pad"], dtype=DTYPES[case["dtype"]], device="cuda")[..., :n]
        x.copy_(_low_rank_plus_noise(gen, b, m, n, 1e-2))
        return {"x": x}
    owned = _owned(case)
    numel = sum(math.prod(s) for s in owned)

    def flat(sigma):
        parts = [_low_rank_plus_noise(gen, math.prod(s[:-2]), s[-2], s[-1], sigma).reshape(-1) for s in owned]
        return torch.cat(parts) if parts else torch.zeros(0, device="cuda")

    momentum = flat(1e-2)
    if case["op"] == "convert":
        return {"numel": numel, "shapes": owned, "momentum": momentum}
    base = flat(1e-3)
    grads = [(base + torch.randn(numel, generator=gen, device="cuda") * 5e-4).to(torch.bfloat16) for _ in range(case["world"])]
    master = torch.randn(numel, generator=gen, device="cuda") * 0.02
    return {"numel": numel, "shapes": owned, "momentum": momentum, "grads": grads, "master": master}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "ortho":
        return s
    n = s["numel"]
    if case["op"] == "muon":
        s["param"] = torch.zeros(n, dtype=torch.bfloat16, device="cuda")      # the rank's shard
    if case["op"] == "convert" or case["state"] == "int8":
        sizes = [math.prod(x[-2:]) for x in s["shapes"] for _ in range(math.prod(x[:-2]))]
        n_scales = sum(-(-k // BLOCK) for k in sizes)
        s["codes"] = torch.zeros(n, dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros(n_scales, dtype=torch.float32, device="cuda")
        if case["op"] == "muon":                                             # the state a running job holds
            codes, scales = _quantize(s["momentum"], s["shapes"])
            s["codes"].copy_(codes)
            s["scales"].copy_(scales)
        else:
            s["back"] = torch.zeros(n, dtype=torch.float32, device="cuda")
    if own:         # the handle that a training loop makes once; the inputs are the same either way
        from sharded_optimizer_step_zr_b200 import ZR_PARAMS_OWNED, ZR_PARTITION_WHOLE_TENSOR
        from sharded_optimizer_step_zr_b200.muon import ZrMuon
        from sharded_optimizer_step_zr_b200.plan import ZrPlan
        plan = ZrPlan(_shapes(case), case["world"], case["rank"], ZR_PARTITION_WHOLE_TENSOR)
        plan.set_param_layout(ZR_PARAMS_OWNED)
        s["muon"] = ZrMuon(plan, lr=case.get("lr", 3e-4), momentum=MU, weight_decay=WEIGHT_DECAY, nesterov=True, ns_steps=STEPS,
                           ns_coeffs=COEFFS, eps=EPS, scale="rms",
                           momentum_format="f32" if case.get("state", "int8") == "f32" else "int8")
    return s


# ---------------------------------------------------------------------------
# plain form (fp32, rounded once)
# ---------------------------------------------------------------------------

def _orthogonalize(x, steps):
    """Newton-Schulz of a batch [..., m, n], fp32 in and out."""
    norm = x.double().square().sum(dim=(-2, -1), keepdim=True).sqrt()
    x = (x.double() / (norm + EPS)).float()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    a, b, c = COEFFS
    for _ in range(steps):
        g = x @ x.mT
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.mT if tall else x


def _blocks(flat, shapes):
    """[n_blocks, 256] view of the values, each matrix padded to whole blocks."""
    parts, at = [], 0
    for s in shapes:
        count, size = math.prod(s[:-2]), math.prod(s[-2:])
        part = flat[at:at + count * size].view(count, size)
        parts.append(torch.nn.functional.pad(part, (0, -size % BLOCK)).reshape(-1, BLOCK))
        at += count * size
    return torch.cat(parts) if parts else flat.new_zeros(0, BLOCK)


def _unblock(blocks, shapes):
    parts, at = [], 0
    for s in shapes:
        count, size = math.prod(s[:-2]), math.prod(s[-2:])
        rows = -(-size // BLOCK) * count
        parts.append(blocks[at:at + rows].view(count, -1)[:, :size].reshape(-1))
        at += rows
    return torch.cat(parts) if parts else blocks.reshape(-1)


def _quantize(flat, shapes):
    x = _blocks(flat, shapes)
    scales = x.abs().amax(dim=1) / torch.full((), 127.0, device=x.device) if x.shape[0] else x.new_zeros(0)
    q = torch.where(scales[:, None] > 0, torch.round(x / scales[:, None]).clamp(-127, 127), torch.zeros_like(x))
    return _unblock(q.to(torch.int8), shapes), scales


def _dequantize(codes, scales, shapes):
    return _unblock(_blocks(codes, shapes).float() * scales[:, None], shapes)


def _scale(m, n):
    return 0.2 * math.sqrt(max(m, n))


def _plain_step(s):
    case, shapes = s["case"], s["shapes"]
    g = s["grads"][0].float()
    for more in s["grads"][1:]:
        g = g + more.float()
    g = g / torch.full((), float(case["world"]), device=g.device)      # a division, not a product with 1/W
    old = s["momentum"] if case["state"] == "f32" else _dequantize(s["codes"], s["scales"], shapes)
    new = old * MU + g
    u = g + new * MU
    if case["state"] == "f32":
        s["momentum"].copy_(new)
        momentum = s["momentum"]
    else:
        codes, scales = _quantize(new, shapes)
        s["codes"].copy_(codes)
        s["scales"].copy_(scales)
        momentum = _dequantize(s["codes"], s["scales"], shapes)
    at = 0
    for shape in shapes:
        size = math.prod(shape)
        o = _orthogonalize(u[at:at + size].view(shape), STEPS).reshape(-1)
        p = s["master"][at:at + size]
        step = case["lr"] * _scale(shape[-2], shape[-1])
        p.copy_(p * (1.0 - case["lr"] * WEIGHT_DECAY) - step * o)
        at += size
    s["param"].copy_(s["master"])
    return {"master": s["master"], "momentum": momentum, "param": s["param"]}


def run(state):
    s, case = state, state["case"]
    if case["op"] == "ortho":
        if own:
            from sharded_optimizer_step_zr_b200.muon import orthogonalize
            return orthogonalize(s["x"], steps=case["steps"], coeffs=COEFFS, eps=EPS)
        return _orthogonalize(s["x"].float(), case["steps"]).to(torch.bfloat16)
    if case["op"] == "convert":
        if own:
            s["muon"].quantize_momentum(s["momentum"], s["codes"], s["scales"])
            s["muon"].dequantize_momentum(s["codes"], s["scales"], s["back"])
            return {"scales": s["scales"], "momentum": s["back"]}
        codes, scales = _quantize(s["momentum"], s["shapes"])
        return {"scales": scales, "momentum": _dequantize(codes, scales, s["shapes"])}
    if not own:
        return _plain_step(s)
    if case["state"] == "f32":
        s["muon"].step(s["grads"], s["master"], s["momentum"], s["param"])
        return {"master": s["master"], "momentum": s["momentum"], "param": s["param"]}
    s["muon"].step(s["grads"], s["master"], (s["codes"], s["scales"]), s["param"])
    if "read" not in s:
        s["read"] = torch.empty(s["numel"], dtype=torch.float32, device="cuda")
    s["muon"].dequantize_momentum(s["codes"], s["scales"], s["read"])
    return {"master": s["master"], "momentum": s["read"], "param": s["param"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_orthogonal(u, steps):
    """p_k(...p_1(.)) of the singular values, one Newton-Schulz step at a time
    on the smaller side: X <- (aI + bG + cG^2) X with G = X X^T."""
    u = u.to(torch.float64)
    flip = u.shape[0] > u.shape[1]
    x = u.t() if flip else u
    x = x / (torch.linalg.vector_norm(x) + EPS)
    a, b, c = (float(v) for v in COEFFS)
    one = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
    for _ in range(steps):
        gram = torch.mm(x, x.t())
        x = torch.mm(a * one + torch.mm(gram, b * one + c * gram), x)
    return x.t() if flip else x


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "ortho":
        return torch.stack([_exact_orthogonal(x, case["steps"]) for x in s["x"]])
    if case["op"] == "convert":
        top, at = [torch.zeros(0, dtype=torch.float64, device="cuda")], 0
        m = s["momentum"].to(torch.float64).abs()
        for shape in s["shapes"]:
            size = shape[-2] * shape[-1]
            whole = size // BLOCK * BLOCK
            for _ in range(math.prod(shape[:-2])):
                if whole:
                    top.append(m[at:at + whole].view(-1, BLOCK).max(dim=1).values)
                if whole < size:
                    top.append(m[at + whole:at + size].max()[None])
                at += size
        # a code may fall on either side of a tie: the read-back values have no exact counterpart
        return {"scales": torch.cat(top) / 127, "momentum": None}
    g = sum(x.to(torch.float64) for x in s["grads"]) / case["world"]
    if case["state"] == "f32":
        old = s["momentum"].to(torch.float64)
    else:
        codes, scales = _quantize(s["momentum"], s["shapes"])
        old = _dequantize(codes.double(), scales.double(), s["shapes"]).to(torch.float64)
    new = MU * old + g
    u = g + MU * new
    master, at = s["master"].to(torch.float64), 0
    for shape in s["shapes"]:
        m, n = shape[-2:]
        for _ in range(math.prod(shape[:-2])):
            o = _exact_orthogonal(u[at:at + m * n].reshape(m, n), STEPS).reshape(-1)
            p = master[at:at + m * n]
            master[at:at + m * n] = p - case["lr"] * (WEIGHT_DECAY * p + 0.2 * max(m, n) ** 0.5 * o)
            at += m * n
    return {"master": master, "momentum": new if case["state"] == "f32" else None, "param": master}
