"""Cases that measure the trained feed-forward block and the clipping of its gradients.

Five operators, each in two forms (`own` false: elementary torch operations in
32 bits, rounded once at the end; `own` true: the calls that a user makes of
this package):

  gated      gate and up projection, activation and product of a gated
             feed-forward block: silu(x Wg^T) * (x Wu^T)
  gated_bwd  its gradient through the block's down projection
  product    the rows' product with a weight matrix: the down projection, and
             with the matrix transposed the gradient of the rows
  wgrad      the gradient of a weight matrix, summed over the rows
  clip       the global norm of many gradients, and their clipping to it

The first four are in BF16 and take either all rows and one matrix (E = 0: a
shared expert) or the rows of a layout, sorted by expert, and one matrix per
expert.
"""
import math
import random

import torch

own = False

CLIP_EPS = 1e-6


# ---- cases ----------------------------------------------------------------------------------

def listed():
    # routing of the grouped cases: T tokens, K of E experts each, R ranks, segments aligned to A
    prefill = {"T": 4096, "K": 8, "E": 256, "R": 8, "A": 128, "drop": 0.0, "zipf": 0.0}
    skewed = {"T": 16384, "K": 6, "E": 64, "R": 8, "A": 1, "drop": 0.02, "zipf": 1.2}
    return [
        # one token of a decode step through the shared expert: reads the weights
        {"name": "gated 1 token", "op": "gated", "T": 1, "E": 0, "D": 7168, "F": 2048,
         "keep": False},
        # a training batch through the shared expert, inputs of the gradient kept
        {"name": "gated shared", "op": "gated", "T": 4096, "E": 0, "D": 7168, "F": 2048,
         "keep": True},
        # the same batch through its routed experts
        {"name": "gated experts", "op": "gated", **prefill, "D": 7168, "F": 2048, "keep": True},
        # backward of the shared expert, a wide one of a narrower model
        {"name": "gated gradient shared", "op": "gated_bwd", "T": 8192, "E": 0, "D": 4096,
         "F": 8192},
        # backward of routed experts whose load is uneven
        {"name": "gated gradient experts", "op": "gated_bwd", **skewed, "D": 4096, "F": 2048},
        # down projection of a decode step's tokens
        {"name": "product decode", "op": "product", "T": 128, "E": 0, "D": 2048, "N": 7168,
         "flip": False},
        # gradient of the rows that came into the routed experts
        {"name": "product experts", "op": "product", **prefill, "D": 4096, "N": 7168,
         "flip": True},
        # the shared expert's weights, gradient kept in 32 bits
        {"name": "weights shared", "op": "wgrad", "T": 4096, "E": 0, "N": 4096, "D": 7168,
         "f32": True},
        # routed experts' weights under an uneven load
        {"name": "weights experts", "op": "wgrad", **skewed, "N": 4096, "D": 4096, "f32": False},
        # what trains around frozen experts (norm gains, routers): launch latency
        {"name": "clip small", "op": "clip", "count": 24, "total": 400_000, "bf16": 0.5,
         "flat": False, "max": 1.0},
        # a whole small model's gradients as views of one bucket, at odd offsets
        {"name": "clip bucket", "op": "clip", "count": 500, "total": 60_000_000, "bf16": 1.0,
         "flat": True, "max": 1.0},
        # experts' weights in 32 bits beside small tensors
        {"name": "clip experts", "op": "clip", "count": 40, "total": 1_000_000_000, "bf16": 0.1,
         "flat": False, "max": 1.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_bwd", "product", "wgrad", "clip"])
    if op == "clip":
        return {"op": op, "count": _log(rng, 1, 800), "total": _log(rng, 1000, 400_000_000),
                "bf16": rng.choice([0.0, 0.3, 1.0]), "flat": rng.random() < 0.5,
                "max": rng.choice([1.0, 1.0, 0.01, 1e9])}

    def width(lo, hi):
        step = rng.choice([8, 64, 128])
        return step * rng.randint(lo // step, hi // step)

    c = {"op": op, "T": _log(rng, 1, 16384), "E": 0}
    if rng.random() < 0.5:
        most = 5 if op == "wgrad" else 7  # a gradient in 32 bits takes twice its weights' bytes
        E, R = rng.choice([(4, 1), (8, 1), (16, 4), (32, 8), (64, 8), (128, 8), (256, 8)][:most])
        c.update(T=_log(rng, 1, 8192), E=E, R=R, K=rng.randint(1, min(8, E)),
                 A=rng.choice([1, 1, 8, 16, 64, 128]), drop=rng.choice([0.0, 0.0, 0.02, 0.3]),
                 zipf=rng.choice([0.0, 0.0, 1.2]))
    c["D"] = width(256, 7168)
    if op in ("gated", "gated_bwd"):
        c["F"] = width(256, 2048 if c["E"] else 8192)
        inner = c["F"] * (2 if op == "gated" else 1)
    else:
        c["N"] = inner = width(256, 4096 if c["E"] else 7168)
    if op == "gated":
        c["keep"] = rng.random() < 0.5
    elif op == "product":
        c["flip"] = rng.random() < 0.5
    elif op == "wgrad":
        c["f32"] = rng.random() < 0.5
    per_token = 2.0 * c.get("K", 1) * inner * c["D"]
    c["T"] = max(1, min(c["T"], int(1e12 / per_token)))  # no more than the largest listed one
    return c


def _sizes(case):
    """(elements, whether BF16) of every tensor of a clip case: from one element to most of all."""
    rng = random.Random("%d %d" % (case["count"], case["total"]))
    share = [math.exp(rng.uniform(0.0, 9.0)) for _ in range(case["count"])]
    whole = sum(share)
    return [(max(1, int(case["total"] * s / whole)), rng.random() < case["bf16"]) for s in share]


def work(case):
    op = case["op"]
    if op == "clip":
        sizes = _sizes(case)
        return {"bytes": sum(2 * n * (2 if half else 4) for n, half in sizes),
                "flops": 3 * sum(n for n, _ in sizes)}
    T, D, E = case["T"], case["D"], case["E"]
    rows, busy = T, 1
    if E:  # rows, and experts that have some
        keep = case["K"] * (1.0 - case["drop"])
        rows, busy = T * keep, E * (1.0 - max(0.0, 1.0 - keep / E) ** T)
    if op == "gated":
        F = case["F"]
        return {"bytes": 4 * busy * F * D + rows * (2 * D + 2 * F + (4 * F if case["keep"] else 0)),
                "flops": 4 * rows * F * D}
    if op == "gated_bwd":
        F = case["F"]
        return {"bytes": 2 * busy * F * D + rows * (2 * D + 10 * F), "flops": 2 * rows * F * D}
    N = case["N"]
    if op == "product":
        return {"bytes": 2 * busy * N * D + 2 * rows * (N + D), "flops": 2 * rows * N * D}
    return {"bytes": (4 if case["f32"] else 2) * max(1, E) * N * D + 2 * rows * (N + D),
            "flops": 2 * rows * N * D}


# ---- inputs ---------------------------------------------------------------------------------

def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(std)


def _weights(case, g, n, k):
    """One matrix [n, k], or one per expert, as an initialisation draws them."""
    lead = (case["E"],) if case["E"] else ()
    return _normal(g, *lead, n, k, std=k ** -0.5)


def _routing(case, g):
    """Router output: distinct experts per token, some slots empty."""
    T, K, E = case["T"], case["K"], case["E"]
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    score = -torch.log(-torch.log(u))
    score = score - case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda"))
    idx = score.topk(K, dim=1).indices.to(torch.int64)
    if case["drop"]:
        empty = torch.rand(idx.shape, generator=g, device="cuda") < case["drop"]
        idx = idx.masked_fill(empty, -1)
    return idx.contiguous()


def _rows(case, s, g, hidden):
    """The rows of the case: s["alloc"] allocated ones and, as (expert, first, end), those in
    use; with `own` also the package's layout, which a program keeps across its calls."""
    T, E = case["T"], case["E"]
    s["handle"] = None
    if not E:
        s["alloc"], s["segments"] = T, [(0, 0, T)]
        return
    A, R, K = case["A"], case["R"], case["K"]
    idx = _routing(case, g)
    cnt = torch.bincount(idx.reshape(-1) + 1, minlength=E + 1)[1:].tolist()
    first, s["segments"] = 0, []
    for e, n in enumerate(cnt):
        if n:
            s["segments"].append((e, first, first + n))
        first += -(-n // A) * A
    # rows allocated without waiting for the counts: the layout's upper bound
    M = -(-T // R)
    up = lambda v: -(-v // A) * A  # noqa: E731
    s["alloc"] = min(R * up(R * M * min(K, E // R) + (A - 1) * (E // R)),
                     up(T * K + E * (A - 1)))
    if own:
        import combine_topk_idx_gb300 as ep
        cfg = ep.make_config(T, K, E, R, hidden, M, A, do_expand=True, do_zero_padding=True,
                             do_cpu_sync=False)
        s["handle"] = ep.ep_layout(cfg, idx)


def _filled(s, g, n, std=1.0):
    """Rows [alloc, n] with values in use, zeros in the alignment padding as a dispatch leaves it."""
    v = torch.zeros(s["alloc"], n, dtype=torch.bfloat16, device="cuda")
    for _, r0, r1 in s["segments"]:
        v[r0:r1] = _normal(g, r1 - r0, n, std=std)
    return v


def _empty(s, n):
    """An output buffer; what no row of this routing reaches stays zero."""
    return torch.zeros(s["alloc"], n, dtype=torch.bfloat16, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], dict(case)
    if op == "clip":
        return _prepare_clip(case, s, g)
    D = case["D"]
    _rows(case, s, g, D)
    if op == "gated":
        F = case["F"]
        s["x"], s["w"] = _filled(s, g, D), _weights(case, g, 2 * F, D)
        s["act"], s["gate_up"] = _empty(s, F), _empty(s, 2 * F) if case["keep"] else None
    elif op == "gated_bwd":
        F = case["F"]
        s["gy"], s["w"] = _filled(s, g, D, std=0.02), _weights(case, g, D, F)
        s["gate_up"] = _filled(s, g, 2 * F, std=1.5)
        s["ggu"], s["act"] = _empty(s, 2 * F), _empty(s, F)
    elif op == "product":
        N = case["N"]
        s["a"], s["out"] = _filled(s, g, D), _empty(s, N)
        s["w"] = _weights(case, g, *((D, N) if case["flip"] else (N, D)))
    else:
        N = case["N"]
        s["grad"], s["a"] = _filled(s, g, N, std=0.02), _filled(s, g, D)
        lead = (case["E"],) if case["E"] else ()
        s["gw"] = torch.empty(*lead, N, D, device="cuda",
                              dtype=torch.float32 if case["f32"] else torch.bfloat16)
    return s


def _prepare_clip(case, s, g):
    """Gradients, each with a scale of its own, and where the clipped ones go: a bucket per
    type. With "flat" the gradients are views of such buckets too."""
    sizes = _sizes(case)
    s["grads"], s["outs"], s["buckets"] = [], [], {}
    at, bucket = {}, {}
    for half, name in ((False, "f32"), (True, "bf16")):
        n = sum(m for m, h in sizes if h is half)
        if n:
            kind = torch.bfloat16 if half else torch.float32
            bucket[half] = torch.empty(n, device="cuda", dtype=kind)
            s["buckets"][name] = torch.empty(n, device="cuda", dtype=kind)
            at[half] = 0
    std = (0.02 * 10.0 ** (-2.0 * torch.rand(len(sizes), generator=g, device="cuda"))).tolist()
    for (n, half), v in zip(sizes, std):
        a, to = at[half], s["buckets"]["bf16" if half else "f32"]
        at[half] += n
        t = bucket[half][a:a + n] if case["flat"] else torch.empty_like(bucket[half][a:a + n])
        s["grads"].append(t.normal_(0.0, v, generator=g))
        s["outs"].append(to[a:a + n])
    if own:  # a trainer's gradients stay where they are: listed once
        import combine_topk_idx_gb300 as ep
        s["plan"] = ep.plan_grads(s["grads"], s["outs"])
    return s


# ---- plain forms ----------------------------------------------------------------------------

def _matrix(s, e):
    return (s["w"][e] if s["E"] else s["w"]).float()


# one product per expert with rows, below: a single batched one would have to pad every expert
# to the longest, ten times the work on a skewed load

def _plain_gated(s):
    F = s["F"]
    for e, r0, r1 in s["segments"]:
        h = s["x"][r0:r1].float() @ _matrix(s, e).t()
        s["act"][r0:r1] = h[:, :F] / (1 + torch.exp(-h[:, :F])) * h[:, F:]
        if s["keep"]:
            s["gate_up"][r0:r1] = h
    return {"act": s["act"], "gate_up": s["gate_up"]}


def _plain_gated_bwd(s):
    F = s["F"]
    for e, r0, r1 in s["segments"]:
        da = s["gy"][r0:r1].float() @ _matrix(s, e)
        h = s["gate_up"][r0:r1].float()
        g, u = h[:, :F], h[:, F:]
        sig = 1 / (1 + torch.exp(-g))
        s["ggu"][r0:r1, :F] = da * u * sig * (1 + g * (1 - sig))
        s["ggu"][r0:r1, F:] = da * g * sig
        s["act"][r0:r1] = g * sig * u
    return {"ggu": s["ggu"], "act": s["act"]}


def _plain_product(s):
    for e, r0, r1 in s["segments"]:
        w = _matrix(s, e)
        s["out"][r0:r1] = s["a"][r0:r1].float() @ (w if s["flip"] else w.t())
    return {"out": s["out"]}


def _plain_wgrad(s):
    out = s["gw"] if s["E"] else s["gw"][None]
    if len(s["segments"]) < out.shape[0]:
        out.zero_()
    for e, r0, r1 in s["segments"]:
        out[e] = s["grad"][r0:r1].float().t() @ s["a"][r0:r1].float()
    return {"gw": s["gw"]}


def _plain_clip(s):
    # a long sum: in 64 bits
    norm = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum().sqrt()
    scale = (s["max"] / (norm + CLIP_EPS)).clamp(max=1.0).float()
    for t, to in zip(s["grads"], s["outs"]):
        to.copy_(t.float() * scale)
    return {"norm": norm.float(), **s["buckets"]}


# ---- the package's calls --------------------------------------------------------------------

def _own_gated(ep, s):
    ep.ep_ffn_gated(s["handle"], s["x"], s["w"], act=s["act"], gate_up=s["gate_up"])
    return {"act": s["act"], "gate_up": s["gate_up"]}


def _own_gated_bwd(ep, s):
    ep.ep_ffn_gated_backward(s["handle"], s["gy"], s["w"], s["gate_up"], grad_gate_up=s["ggu"],
                             act=s["act"])
    return {"ggu": s["ggu"], "act": s["act"]}


def _own_product(ep, s):
    ep.ep_ffn_product(s["handle"], s["a"], s["w"], out=s["out"], transposed=s["flip"])
    return {"out": s["out"]}


def _own_wgrad(ep, s):
    ep.ep_ffn_weight_grad(s["handle"], s["grad"], s["a"], grad_w=s["gw"])
    return {"gw": s["gw"]}


def _own_clip(ep, s):
    norm = ep.ep_clip_grads(s["plan"], s["max"])
    return {"norm": norm, **s["buckets"]}


_PLAIN = {"gated": _plain_gated, "gated_bwd": _plain_gated_bwd, "product": _plain_product,
          "wgrad": _plain_wgrad, "clip": _plain_clip}
_OWN = {"gated": _own_gated, "gated_bwd": _own_gated_bwd, "product": _own_product,
        "wgrad": _own_wgrad, "clip": _own_clip}


def run(state):
    if own:
        import combine_topk_idx_gb300 as ep
        return _OWN[state["op"]](ep, state)
    return _PLAIN[state["op"]](state)


# ---- the definition in 64 bits --------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    if op == "clip":
        sums = [torch.linalg.vector_norm(t.double()).item() for t in s["grads"]]
        norm = math.sqrt(math.fsum(v * v for v in sums))
        by = case["max"] / (norm + CLIP_EPS) if norm + CLIP_EPS > case["max"] else 1.0
        got = {"norm": torch.tensor(norm, dtype=torch.float64)}
        for name, b in s["buckets"].items():
            got[name] = torch.cat([t.double() for t in s["grads"] if t.dtype == b.dtype]) * by
        return got
    wide = lambda n: torch.zeros(s["alloc"], n, dtype=torch.float64, device="cuda")  # noqa: E731
    if op == "wgrad":
        out = torch.zeros(max(1, case["E"]), case["N"], case["D"], dtype=torch.float64,
                          device="cuda")
        for e, r0, r1 in s["segments"]:
            out[e] = torch.einsum("rn,rd->nd", s["grad"][r0:r1].double(), s["a"][r0:r1].double())
        return {"gw": out if case["E"] else out[0]}
    w = s["w"] if case["E"] else s["w"][None]
    if op == "product":
        out, into = wide(case["N"]), "rd,dn->rn" if case["flip"] else "rd,nd->rn"
        for e, r0, r1 in s["segments"]:
            out[r0:r1] = torch.einsum(into, s["a"][r0:r1].double(), w[e].double())
        return {"out": out}
    F = case["F"]
    act, both = wide(F), wide(2 * F)
    for e, r0, r1 in s["segments"]:
        if op == "gated":
            x = s["x"][r0:r1].double()
            gate, up = (torch.einsum("rd,fd->rf", x, p.double()) for p in w[e].split(F))
            both[r0:r1] = torch.cat([gate, up], dim=1)
        else:
            gate, up = s["gate_up"][r0:r1].double().split(F, dim=1)
            slope = torch.sigmoid(gate) + gate * torch.sigmoid(gate) * torch.sigmoid(-gate)
            da = torch.einsum("rd,df->rf", s["gy"][r0:r1].double(), w[e].double())
            both[r0:r1] = torch.cat([da * up * slope, da * gate * torch.sigmoid(gate)], dim=1)
        act[r0:r1] = torch.sigmoid(gate) * gate * up
    if op == "gated":
        return {"act": act, "gate_up": both if case["keep"] else None}
    return {"ggu": both, "act": act}
