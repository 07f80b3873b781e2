"""The Muon optimizer step on Shard(0) parameter groups: what is timed and compared.

Muon updates a matrix parameter with an orthogonalised momentum.  On a group
whose matrices are sharded along dim 0 it is three operators, with collectives
between them:

* ``momentum``: m = mu m + (1 - mu) g on this rank's fp32 shards, and the bf16
  update u (m, or with Nesterov mu m + (1 - mu) g) packed into the rank's
  all-gather segment, zeros in the padding.  With ``reduce`` the gradient is
  the mean of the N bf16 rows of the reduce-scatter input, in the same pass.
* ``orthogonalize``: every full matrix U -> the quintic Newton-Schulz iterate
  X <- a X + b (X X^T) X + c (X X^T)^2 X, five times from U / (|U|_F + eps).
* ``update``: p = p (1 - lr wd) - lr s o on the fp32 master shards, o the bf16
  orthogonalised update (this rank's segment, or its rows of the full matrices)
  and s a factor for each parameter, and the bf16 copy-in of the new p.

``run`` computes them with elementary torch operations in 32 bits, or, where
``own`` is set, through the package's entry points; ``exact`` in 64 bits.
"""
import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
MU = 0.95
LR = 0.02
WD = 0.1

# The matrices of the repository's workloads (norms, biases and embeddings
# stay with AdamW).
PROBE = "32x16,4x32"
BLOCK = "4096x4096*4,14336x4096*2,4096x14336"
GQA = "8192x8192,1024x8192*2,8192x8192"
EXPERTS = "1408x2048*32,2048x1408*16,64x2048,1x2048"


def listed():
    return [
        # the two-layer probe: a step of a few hundred elements, all latency
        {"name": "momentum probe", "op": "momentum", "shapes": PROBE, "world": 2, "rank": 0, "align": 1,
         "reduce": False, "nesterov": True},
        # one decoder block on 8 ranks, gradients already reduced
        {"name": "momentum block n8", "op": "momentum", "shapes": BLOCK, "world": 8, "rank": 3, "align": 8,
         "reduce": False, "nesterov": True},
        # the same block straight from the reduce-scatter's rows
        {"name": "reduce momentum block n8", "op": "momentum", "shapes": BLOCK, "world": 8, "rank": 0, "align": 8,
         "reduce": True, "nesterov": True},
        # ragged experts on 6 ranks: short last chunks, empty pieces, rows at any phase
        {"name": "reduce momentum experts n6", "op": "momentum", "shapes": EXPERTS, "world": 6, "rank": 5, "align": 1,
         "reduce": True, "nesterov": False},
        {"name": "update probe", "op": "update", "shapes": PROBE, "world": 2, "rank": 1, "align": 1, "full": False},
        # the orthogonalised update came back as this rank's segment (each matrix worked on by one rank)
        {"name": "update block n8", "op": "update", "shapes": BLOCK, "world": 8, "rank": 3, "align": 8, "full": False},
        # every rank orthogonalised every matrix and takes its own rows
        {"name": "update rows experts n6", "op": "update", "shapes": EXPERTS, "world": 6, "rank": 1, "align": 1,
         "full": True},
        # the probe's matrices: a handful of rows
        {"name": "orthogonalize probe", "op": "orthogonalize", "shapes": PROBE, "f32": False},
        # key and value projections of a grouped-query block: few rows, long ones
        {"name": "orthogonalize kv", "op": "orthogonalize", "shapes": "1024x8192*2", "f32": False},
        # one square projection by itself, from fp32 (one rank: the momentum is the full matrix)
        {"name": "orthogonalize square", "op": "orthogonalize", "shapes": "4096x4096", "f32": True},
        # some of a layer's experts at once, sizes that are no multiple of a power of two
        {"name": "orthogonalize experts", "op": "orthogonalize", "shapes": "1408x2048*8,2048x1408*4,65x2047",
         "f32": False},
        # all matrices of one decoder block
        {"name": "orthogonalize block", "op": "orthogonalize", "shapes": BLOCK, "f32": False},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: any operator, sizes from a few elements to those of a decoder block."""
    op = rng.choice(("momentum", "update", "orthogonalize", "orthogonalize"))
    if op == "orthogonalize":
        rows, cols = _log(rng, 1, 6000), _log(rng, 1, 6000)
        if rng.random() < 0.5:      # the framework's widths are multiples of 64 more often than not
            rows, cols = -(-rows // 64) * 64, -(-cols // 64) * 64
        most = max(1, min(32, int(2.5e11 / (min(rows, cols) ** 2 * max(rows, cols) + 1e9))))
        return {"op": op, "shapes": "%dx%d*%d" % (rows, cols, _log(rng, 1, most)), "f32": rng.random() < 0.25}
    world = rng.choice((1, 2, 4, 6, 8, 8, 16))
    shapes = []
    for _ in range(rng.randint(1, 4)):
        r, c = _log(rng, 1, 8192), _log(rng, 1, 8192)
        if rng.random() < 0.5:
            c = -(-c // 64) * 64
        shapes.append("%dx%d*%d" % (r, c, rng.randint(1, 3)))
    case = {"op": op, "shapes": ",".join(shapes), "world": world, "rank": rng.randrange(world),
            "align": rng.choice((1, 8))}
    if op == "momentum":
        case.update(reduce=rng.random() < 0.5, nesterov=rng.random() < 0.5)
    else:
        case.update(full=rng.random() < 0.5)
    return case


# ---- layout ------------------------------------------------------------------


def _shapes(case):
    out = []
    for part in case["shapes"].split(","):
        dims, _, times = part.partition("*")
        r, c = dims.split("x")
        out += [(int(r), int(c))] * int(times or 1)
    return out


def _pieces(case):
    """This rank's piece of each matrix, as the group lays it out: (valid elements, offset in the segment, elements
    in the segment, offset in the flat shards, offset of its first row in the flat full matrices); then the segment's
    length and the two flat lengths.  Shards start at multiples of 64 elements, full matrices of 128."""
    world, rank, align = case["world"], case["rank"], case["align"]
    out, seg, flat, full = [], 0, 0, 0
    for r, c in _shapes(case):
        chunk = -(-r // world)
        first = min(rank * chunk, r)
        valid = (min((rank + 1) * chunk, r) - first) * c
        size = -(-chunk * c // align) * align
        out.append((valid, seg, size, flat, full + first * c))
        seg, flat, full = seg + size, flat + -(-valid // 64) * 64, full + -(-r * c // 128) * 128
    return out, seg, max(flat, 1), max(full, 1)


def _randn(gen, n, std):
    return torch.randn(n, generator=gen, device="cuda") * std


def _shards(gen, flat, pieces, std):
    """Flat fp32 shards, zeros in the gaps between them."""
    x = _randn(gen, flat, std)
    for n, _, _, at, _ in pieces:
        x[at + n:at + n + -n % 64] = 0
    return x


def _gradient(gen, rows, cols):
    """A gradient's spectrum: a few strong directions that fall off, over noise from the rest of the batch."""
    rank = max(1, min(rows, cols) // 8)
    left = torch.randn(rows, rank, generator=gen, device="cuda") / torch.arange(1, rank + 1, device="cuda")
    right = torch.randn(rank, cols, generator=gen, device="cuda")
    return 1e-3 * (left @ right + 0.05 * torch.randn(rows, cols, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    shapes = _shapes(case)
    state = {"case": case, "shapes": shapes}
    if case["op"] == "orthogonalize":
        state["u"] = [_gradient(gen, r, c).to(torch.float32 if case["f32"] else torch.bfloat16) for r, c in shapes]
        state["o"] = [torch.empty(r, c, dtype=torch.bfloat16, device="cuda") for r, c in shapes]
        if own:
            from sharded_shard_amd.group import Orthogonalizer
            state["plan"] = Orthogonalizer(shapes, coeffs=[COEFFS] * STEPS, eps=EPS)
            state["plan"].bind(state["u"], state["o"])
            state["plan"].allocate()
        return state
    pieces, seg, flat, full = _pieces(case)
    state["pieces"], state["seg"] = pieces, seg
    state["ag_in"] = torch.empty(seg, dtype=torch.bfloat16, device="cuda")
    if case["op"] == "momentum":
        state["m"] = _shards(gen, flat, pieces, 1e-3)
        if case["reduce"]:
            state["rs_in"] = _randn(gen, case["world"] * seg, 1e-3).to(torch.bfloat16)
            state["g"] = torch.zeros(1, device="cuda")
        else:
            state["g"] = _shards(gen, flat, pieces, 1e-3)
    else:
        state["p"] = _shards(gen, flat, pieces, 0.02)
        n = full if case["full"] else seg
        state["o"] = _randn(gen, n, 0.02).to(torch.bfloat16)
        # max(1, rows / cols) ** 0.5: updates of equal size whatever the matrix's shape
        state["s"] = torch.tensor([max(1.0, r / c) ** 0.5 for r, c in shapes], device="cuda")
    if own:
        state["group"] = _group(state)
    return state


def _group(state):
    """The group's plan, bound to the state's tensors."""
    from sharded_shard_amd.group import ShardedGroup
    case = state["case"]
    group = ShardedGroup(state["shapes"], case["world"], case["rank"], case["align"], bind=False, optimizer="muon")
    if case["op"] == "momentum":
        group.m_flat = state["m"]
        group.grad_flat = None if case["reduce"] else state["g"]
    else:
        group.master_flat = state["p"]
        group.full_flat = state["o"].view(torch.int16) if case["full"] else None
    group.bind()
    return group


# ---- the plain forms ---------------------------------------------------------


def _segment(x, state):
    """The flat shards' values in the segment's order, zeros in the padding."""
    return torch.cat([t for n, _, size, at, _ in state["pieces"] for t in (x[at:at + n], x.new_zeros(size - n))])


def _flat(x, field, state):
    """The shards' values in the flat order, zeros in the gaps, from the offset that each piece has in `field`."""
    return torch.cat([t for p in state["pieces"] for t in (x[p[field]:p[field] + p[0]], x.new_zeros(-p[0] % 64))])


def _momentum(state):
    case, m = state["case"], state["m"]
    if case["reduce"]:
        mean = state["rs_in"].view(case["world"], -1).float().sum(0) / case["world"]
        g = _flat(mean, 1, state)
        n = g.numel()
        m[:n].mul_(MU).add_(g * (1 - MU))
    else:
        g, n = state["g"], m.numel()
        m.mul_(MU).add_(g * (1 - MU))
    u = m[:n] * MU + g * (1 - MU) if case["nesterov"] else m
    state["ag_in"].copy_(_segment(u, state))
    return state["m"], state["ag_in"]


def _orthogonal(u):
    a, b, c = COEFFS
    x = u.float()
    tall = x.shape[0] > x.shape[1]
    x = x.mT if tall else x
    x = x / (x.norm() + EPS)
    for _ in range(STEPS):
        gram = x @ x.mT
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return (x.mT if tall else x).to(torch.bfloat16)


def _update(state):
    case, p = state["case"], state["p"]
    o = _flat(state["o"], 4 if case["full"] else 1, state)
    n = o.numel()
    s = torch.cat([state["s"][k].expand(q[0] + -q[0] % 64) for k, q in enumerate(state["pieces"])])
    p[:n].mul_(1 - LR * WD).sub_(LR * s * o.float())
    state["ag_in"].copy_(_segment(p, state))
    return state["p"], state["ag_in"]


def run(state):
    case = state["case"]
    if case["op"] == "orthogonalize":
        if own:
            state["plan"].execute()
            return state["o"]
        return [_orthogonal(u) for u in state["u"]]
    if not own:
        return _momentum(state) if case["op"] == "momentum" else _update(state)
    group = state["group"]
    if case["op"] == "update":
        group.muon_update(None if case["full"] else state["o"], state["ag_in"], scales=state["s"], lr=LR,
                          weight_decay=WD)
        return state["p"], state["ag_in"]
    if case["reduce"]:
        group.muon_reduce_momentum(state["rs_in"], state["ag_in"], momentum=MU, nesterov=case["nesterov"])
    else:
        group.muon_momentum(state["ag_in"], momentum=MU, nesterov=case["nesterov"])
    return state["m"], state["ag_in"]


# ---- what a pass has to do, and what it has to give --------------------------


def work(case):
    shapes = _shapes(case)
    if case["op"] == "orthogonalize":
        # an iteration is X X^T and its square, symmetric and so half of each product, and the product with X
        flops = sum(STEPS * (3 * min(s) ** 2 * max(s) + min(s) ** 3) for s in shapes)
        return {"bytes": sum(r * c for r, c in shapes) * (6 if case["f32"] else 4), "flops": flops}
    pieces, seg, _, _ = _pieces(case)
    valid = sum(p[0] for p in pieces)
    if case["op"] == "momentum":
        grads = 2 * case["world"] * valid if case["reduce"] else 4 * valid
        return {"bytes": grads + 8 * valid + 2 * seg, "flops": (6 + (case["world"] if case["reduce"] else 0)) * valid}
    return {"bytes": 10 * valid + 2 * seg, "flops": 3 * valid}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "orthogonalize":
        return [_exact_orthogonal(u.double()) for u in state["u"]]
    out = state["m" if case["op"] == "momentum" else "p"].double()
    segment = torch.zeros(state["seg"], dtype=torch.float64, device="cuda")
    for k, (n, seg, _, at, full) in enumerate(state["pieces"]):
        here = slice(at, at + n)
        if case["op"] == "momentum":
            if case["reduce"]:
                g = state["rs_in"].view(case["world"], -1)[:, seg:seg + n].double().mean(0)
            else:
                g = state["g"][here].double()
            out[here] = g + MU * (out[here] - g)
            segment[seg:seg + n] = g + MU * (out[here] - g) if case["nesterov"] else out[here]
        else:
            src = full if case["full"] else seg
            step = state["s"][k].double() * state["o"][src:src + n].double()
            out[here] = out[here] - LR * (WD * out[here] + step)
            segment[seg:seg + n] = out[here]
    return out, segment


def _exact_orthogonal(u):
    if u.shape[0] < u.shape[1]:
        return _exact_orthogonal(u.T.contiguous()).T.contiguous()
    a, b, c = COEFFS
    x = u / (torch.sqrt((u * u).sum()) + EPS)
    for _ in range(STEPS):
        g = x.T @ x
        x = x @ (c * (g @ g) + b * g + a * torch.eye(len(g), dtype=g.dtype, device=g.device))
    return x
