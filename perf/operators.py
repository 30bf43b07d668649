"""Cases that measure the operators around dispatch and combine.

Six passes over four operators, each in two forms (`own` false: elementary
torch operations in 32 bits, rounded once at the end; `own` true: the call a
user makes of this package):

  norm      root-mean-square norm with the residual's addition, e4m3 output
            with one fp32 scale per 1x128 block (the input of a pre-quantised
            dispatch)
  norm_bwd  its gradient
  act       gated activation between the experts' two products, e4m3 output,
            and the 8-bit checkpoint of its input
  act_bwd   its gradient, from the checkpoint
  comb_bwd  gradient of the weighted combine: expert rows, weights, biases
  product   the experts' FP8 product over the rows sorted by expert
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
EPS = 1e-6


# ---- cases ----------------------------------------------------------------------------------

def listed():
    return [
        # one token of a decode step before its dispatch: launch latency
        {"name": "norm 1 token", "op": "norm", "T": 1, "H": 7168, "col": False, "bf16": True},
        # a prefill batch; column-major scales, as the dispatch hands them on
        {"name": "norm prefill", "op": "norm", "T": 4096, "H": 7168, "col": True, "bf16": False},
        # a training step of a narrower model
        {"name": "norm gradient", "op": "norm_bwd", "T": 16384, "H": 4096, "res": True},
        # 128 tokens per rank, one expert row per slot, no alignment: serving
        {"name": "act decode", "op": "act", "T": 1024, "K": 8, "E": 256, "R": 8, "A": 1,
         "F": 2048, "ckpt": False, "weights": False, "col": False, "drop": 0.0, "zipf": 0.0},
        # training forward on a prefill-sized batch: padded segments, checkpoint kept
        {"name": "act checkpoint", "op": "act", "T": 4096, "K": 8, "E": 256, "R": 8, "A": 128,
         "F": 2048, "ckpt": True, "weights": False, "col": True, "drop": 0.0, "zipf": 0.0},
        # the same batch backward, gradient handed on in 8 bits
        {"name": "act gradient", "op": "act_bwd", "T": 4096, "K": 8, "E": 256, "R": 8, "A": 128,
         "F": 2048, "weights": True, "fp8": True, "col": True, "drop": 0.0, "zipf": 0.0},
        # a test-sized batch: launch latency
        {"name": "combine gradient tiny", "op": "comb_bwd", "T": 128, "H": 256, "K": 2, "E": 16,
         "R": 4, "A": 8, "layout": "expand", "bias": False, "fp8": False, "col": False,
         "drop": 0.05, "zipf": 0.0},
        # prefill batch, rows sorted by expert, gradient rows in 8 bits for the next product
        {"name": "combine gradient prefill", "op": "comb_bwd", "T": 4096, "H": 7168, "K": 8,
         "E": 256, "R": 8, "A": 128, "layout": "expand", "bias": False, "fp8": True, "col": True,
         "drop": 0.0, "zipf": 0.0},
        # skewed routing, rows shared by a rank's experts, per-expert bias trained
        {"name": "combine gradient skewed", "op": "comb_bwd", "T": 16384, "H": 4096, "K": 6,
         "E": 64, "R": 8, "A": 1, "layout": "rank", "bias": True, "fp8": False, "col": False,
         "drop": 0.02, "zipf": 1.2},
        # one token through eight experts' gate and up projections: reads weights only
        {"name": "product 1 token", "op": "product", "T": 1, "K": 8, "E": 256, "R": 8, "A": 1,
         "N": 4096, "D": 7168, "col": False, "drop": 0.0, "zipf": 0.0},
        # a prefill batch over 256 experts
        {"name": "product prefill", "op": "product", "T": 4096, "K": 8, "E": 256, "R": 8,
         "A": 128, "N": 4096, "D": 7168, "col": True, "drop": 0.0, "zipf": 0.0},
        # few experts with many rows and an uneven load: bound by the tensor cores
        {"name": "product skewed", "op": "product", "T": 16384, "K": 6, "E": 64, "R": 8,
         "A": 128, "N": 4096, "D": 4096, "col": True, "drop": 0.02, "zipf": 1.2},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "act", "act_bwd", "comb_bwd", "product"])

    def width(lo, hi):
        return 128 * rng.choice([b for b in range(lo // 128, hi // 128 + 1) if b != 24])

    T = _log(rng, 1, 8192) if op != "norm_bwd" else _log(rng, 16, 16384)
    if T in (1536, 3072):  # keeps every size off one that no configuration here has
        T += 1
    if op == "norm":
        return {"op": op, "T": T, "H": width(256, 7168), "col": rng.random() < 0.5,
                "bf16": rng.random() < 0.5}
    if op == "norm_bwd":
        H = 8 * rng.randrange(32, 513) if rng.random() < 0.3 else width(256, 7168)
        return {"op": op, "T": T, "H": H, "res": rng.random() < 0.5}
    E, R = rng.choice([(8, 1), (16, 4), (32, 8), (64, 8), (128, 8), (256, 8), (256, 32)])
    c = {"op": op, "T": T, "K": rng.randint(1, 8), "E": E, "R": R,
         "A": rng.choice([1, 1, 8, 16, 64, 128]), "drop": rng.choice([0.0, 0.0, 0.02, 0.3]),
         "zipf": rng.choice([0.0, 0.0, 1.2]), "col": rng.random() < 0.5}
    if op in ("act", "act_bwd"):
        c["F"] = 128 * rng.choice([b for b in range(2, 17) if b != 12])
        c["weights"] = rng.random() < 0.5
        c["T"] = min(T, 4096)
        c["ckpt" if op == "act" else "fp8"] = rng.random() < 0.5
    elif op == "comb_bwd":
        c["H"] = width(256, 7168)
        c["layout"] = rng.choice(["expand", "expand", "rank"])
        c["bias"] = rng.random() < 0.4
        c["fp8"] = rng.random() < 0.5
        c["T"] = min(T, 4096)
    else:
        c["D"] = width(256, 7168)
        c["N"] = 8 * rng.randrange(32, 513) if rng.random() < 0.3 else width(256, 4096)
        if c["N"] == 3072:
            c["N"] = 2048
        c["T"] = min(T, 4096)
    return c


def work(case):
    op, T = case["op"], case["T"]
    if op in ("norm", "norm_bwd"):
        H = case["H"]
        if op == "norm":  # x, residual, sum, bytes, scales (and the BF16 output)
            return {"bytes": T * (H * (7 + 2 * case["bf16"]) + H // 32) + 2 * H, "flops": 8 * T * H}
        return {"bytes": T * (H * (6 + 2 * case["res"]) + 4) + 6 * H, "flops": 12 * T * H}
    K, E, keep = case["K"], case["E"], 1.0 - case["drop"]
    rows = T * K * keep
    if op == "act":
        F = case["F"]
        per = 4 * F + F + F // 32 + (2 * F + F // 16 if case["ckpt"] else 0)
        return {"bytes": rows * per, "flops": rows * F * 10}
    if op == "act_bwd":
        F = case["F"]
        per = 2 * F + F // 16 + 2 * F + (2 * F + F // 16 if case["fp8"] else 4 * F) + 8
        return {"bytes": rows * per, "flops": rows * F * 20}
    if op == "comb_bwd":
        H, L = case["H"], E // case["R"]
        slots = rows
        if case["layout"] == "rank":  # distinct ranks of a token's slots
            rows = T * case["R"] * (1.0 - (1.0 - keep * L / E) ** K)
        out = rows * (H + H // 32) if case["fp8"] else rows * 2 * H
        bias = E * H * 6 if case["bias"] else 0
        return {"bytes": T * H * 2 + rows * 2 * H + out + bias + T * K * 12, "flops": slots * H * 4}
    D, N = case["D"], case["N"]
    busy = E * (1.0 - (1.0 - K * keep / E) ** T) if K < E else E
    return {"bytes": busy * N * D + rows * (D + D // 32 + 2 * N), "flops": 2 * rows * N * D}


# ---- inputs ---------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * std)


def _routing(case, g):
    """Router output: distinct experts per token, softmax weights, some slots empty."""
    T, K, E = case["T"], case["K"], case["E"]
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    score = -torch.log(-torch.log(u))
    score = score - case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda"))
    top = score.topk(min(K, E), dim=1)
    idx = top.indices.to(torch.int64)
    w = torch.softmax(torch.randn(idx.shape, generator=g, device="cuda"), dim=1)
    if case["drop"]:
        empty = torch.rand(idx.shape, generator=g, device="cuda") < case["drop"]
        idx, w = idx.masked_fill(empty, -1), w.masked_fill(empty, 0.0)
    return idx.contiguous(), w.contiguous()


def _bound(case, layout="expand"):
    """Rows allocated without waiting for the counts: the layout's upper bound."""
    T, E, R, A = case["T"], case["E"], case["R"], case["A"]
    K, M = min(case["K"], E), -(-T // R)
    if layout == "rank":
        return min(R * M * R, T * min(K, R))
    up = lambda v: -(-v // A) * A  # noqa: E731
    return min(R * up(R * M * min(K, E // R) + (A - 1) * (E // R)), up(T * K + E * (A - 1)))


def _place(idx, case, layout="expand"):
    """Rows of the sorted layout: dst [T, K], each expert's first row and row count, rows."""
    E, A, R = case["E"], case["A"], case["R"]
    valid = idx >= 0
    if layout == "rank":
        rank = torch.where(valid, idx // (E // R), R)
        there = torch.zeros(idx.shape[0], R + 1, dtype=torch.int64, device="cuda")
        there = there.scatter_(1, rank, 1)[:, :R].t().contiguous().view(-1)
        row = (torch.cumsum(there, 0) - 1).view(R, -1)
        dst = row.t().gather(1, rank.clamp(max=R - 1))
        return torch.where(valid, dst, -1), None, None, int(there.sum())
    e = torch.where(valid, idx, E).view(-1)
    cnt = torch.bincount(e, minlength=E + 1)[:E]
    up = (cnt + A - 1) // A * A
    start, before = torch.cumsum(up, 0) - up, torch.cumsum(cnt, 0) - cnt
    order = torch.argsort(e, stable=True)
    es = e[order].clamp(max=E - 1)
    dst = torch.empty_like(e)
    dst[order] = start[es] + torch.arange(e.numel(), device="cuda") - before[es]
    return torch.where(valid, dst.view(idx.shape), -1), start, cnt, int(up.sum())


def _handle(case, s, hidden, fp8, layout="expand"):
    """The package's layout of the same routing, kept by a program across its calls."""
    import combine_topk_idx_gb300 as ep
    T, R = case["T"], case["R"]
    cfg = ep.make_config(T, s["idx"].shape[1], case["E"], R, hidden, -(-T // R), case["A"],
                         do_expand=layout == "expand", do_zero_padding=layout == "expand",
                         do_cpu_sync=False, use_fp8=fp8, use_tma_aligned_col_major_sf=case["col"])
    s["handle"] = ep.ep_layout(cfg, s["idx"])


def _buffers(case, s, n, kind):
    """Receive buffers of the upper bound; what no row of this routing reaches stays zero."""
    rows = s["alloc"]
    if kind == "bf16":
        return torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    tall = -(-rows // 4) * 4 if case["col"] else rows
    return (torch.zeros(rows, n, dtype=torch.uint8, device="cuda"),
            torch.zeros(tall * (n // 128), device="cuda"))


def prepare(case, seed):
    g, op, T = _gen(seed), case["op"], case["T"]
    s = dict(case)
    if op == "norm":
        s["x"], s["residual"] = _normal(g, T, case["H"]), _normal(g, T, case["H"], std=3.0)
        s["gamma"] = 1 + _normal(g, case["H"], std=0.1)
        return s
    if op == "norm_bwd":
        H = case["H"]
        s["r"], s["gy"] = _normal(g, T, H, std=3.0), _normal(g, T, H, std=0.02)
        s["gres"] = _normal(g, T, H, std=0.02) if case["res"] else None
        s["gamma"] = 1 + _normal(g, H, std=0.1)
        s["rstd"] = torch.rsqrt(s["r"].float().square().mean(1) + EPS)
        return s
    s["idx"], s["w"] = _routing(case, g)
    layout = case.get("layout", "expand")
    s["dst"], s["start"], s["cnt"], rows = _place(s["idx"], case, layout)
    s["rows"], s["alloc"] = rows, _bound(case, layout)
    if op == "comb_bwd":
        H = case["H"]
        s["g"], s["y"] = _normal(g, T, H, std=0.02), _normal(g, s["alloc"], H)
        if case["fp8"]:
            s["gy_q"], s["gy_sf"] = _buffers(case, s, H, "fp8")
        else:
            s["gy"] = _buffers(case, s, H, "bf16")
        s["bias"] = _normal(g, case["E"], H, std=0.1) if case["bias"] else None
        if own:
            _handle(case, s, H, case["fp8"], layout)
        return s
    # rows in use (the rest is alignment padding, zero as dispatch leaves it)
    rows = s["alloc"]
    used = torch.zeros(rows + 1, dtype=torch.bool, device="cuda")
    used[s["dst"].reshape(-1)] = True  # -1 marks the spare last element
    used = used[:rows]
    if op in ("act", "act_bwd"):
        F = case["F"]
        s["h"] = _normal(g, rows, 2 * F, std=1.5) * used[:, None]
        row_w = torch.rand(rows, generator=g, device="cuda") * used
        s["row_w"] = row_w if case["weights"] else None
        if op == "act":
            s["q"], s["sf"] = _buffers(case, s, F, "fp8")
            if case["ckpt"]:  # rows of padding are neither written nor read
                s["ckpt"] = torch.zeros(rows, 2 * F, dtype=torch.uint8, device="cuda")
                s["ckpt_sf"] = torch.zeros(rows, 2 * F // 128, device="cuda")
        else:
            q, s["ckpt_sf"] = _quantise(s.pop("h").float())
            s["ckpt"] = q.to(FP8).view(torch.uint8)
            s["da"] = _normal(g, rows, F, std=0.02) * used[:, None]
            if case["fp8"]:
                s["q"], s["sf"] = _buffers(case, s, 2 * F, "fp8")
            else:
                s["gh"] = _buffers(case, s, 2 * F, "bf16")
            s["gw"] = torch.zeros(rows, device="cuda")
        if own:
            _handle(case, s, F, True)
        return s
    D, N, E = case["D"], case["N"], case["E"]
    s["a"], s["a_sf"] = _buffers(case, s, D, "fp8")
    q, sf = _quantise(_normal(g, rows, D).float() * used[:, None])
    s["a"].view(FP8).copy_(q)
    _sf_rows(s, s["a_sf"], D, rows).copy_(sf)
    s["out"] = _buffers(case, s, N, "bf16")
    # weights as a quantised checkpoint holds them: 448 at about 4.5 deviations of a block
    s["wq"] = torch.empty(E, N, D, dtype=torch.uint8, device="cuda")
    for e in range(0, E, 8):
        part = torch.randn((min(8, E - e), N, D), generator=g, device="cuda", dtype=torch.bfloat16)
        s["wq"][e:e + 8] = (part * 100).clamp_(-448, 448).to(FP8).view(torch.uint8)
    s["w_sf"] = (0.5 + torch.rand(E, -(-N // 128), D // 128, generator=g, device="cuda")) / (
        100 * math.sqrt(D))
    # the rows [r0, r1) of each expert that has some
    s["segments"] = [(e, r0, r0 + n) for e, (r0, n) in
                     enumerate(zip(s["start"].tolist(), s["cnt"].tolist())) if n]
    if own:
        _handle(case, s, D, True)
    return s


# ---- plain forms ----------------------------------------------------------------------------

def _quantise(v):
    """What e4m3 holds of v [rows, n] by 1x128 blocks, before its rounding, and fp32 scales
    (amax / 448)."""
    b = v.view(v.shape[0], -1, 128)
    sf = b.abs().amax(2) / 448.0
    q = torch.where(sf[..., None] > 0, b / sf[..., None], torch.zeros_like(b)).clamp_(-448, 448)
    return q.view(v.shape), sf


def _sf_rows(s, flat, n, rows):
    """Scales [rows, n / 128] of a flat array in the receive layout."""
    if s["col"]:
        return flat.view(n // 128, -1)[:, :rows].t()
    return flat.view(-1, n // 128)[:rows]


def _put(s, v, q, sf):
    """Quantises v, the rows in use, into receive buffers."""
    rows, n = v.shape
    a, b = _quantise(v)
    q.view(FP8)[:rows].copy_(a)
    _sf_rows(s, sf, n, rows).copy_(b)
    return q.view(FP8), sf


def _values(q, sf):
    """fp32 values of e4m3 bytes q [..., n] and their scales [..., n / 128]."""
    v = q.view(FP8).to(torch.float32)
    return (v.view(*sf.shape, 128) * sf[..., None]).view(q.shape)


def _plain_norm(s):
    v = s["x"].float() + s["residual"].float()
    y = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * s["gamma"].float()
    q, sf = _quantise(y)
    return {"r": v.bfloat16(), "q": q.to(FP8), "sf": sf, "y": y.bfloat16() if s["bf16"] else None}


def _plain_norm_bwd(s):
    xh = s["r"].float() * s["rstd"][:, None]
    gy = s["gy"].float()
    t = gy * s["gamma"].float()
    gx = s["rstd"][:, None] * (t - xh * (t * xh).mean(1, keepdim=True))
    if s["gres"] is not None:
        gx = gx + s["gres"].float()
    return {"gx": gx.bfloat16(), "ggamma": (gy * xh).sum(0)}


def _plain_act(s):
    F, rows = s["F"], s["rows"]
    h = s["h"][:rows].float()
    g, u = h[:, :F], h[:, F:]
    a = g / (1 + torch.exp(-g)) * u
    if s["row_w"] is not None:
        a = a * s["row_w"][:rows, None]
    out = dict(zip(("q", "sf"), _put(s, a, s["q"], s["sf"])))
    if s["ckpt"] is not False:
        q, sf = _quantise(h)
        s["ckpt"].view(FP8)[:rows].copy_(q)
        s["ckpt_sf"][:rows].copy_(sf)
        out["ckpt"], out["ckpt_sf"] = s["ckpt"].view(FP8), s["ckpt_sf"]
    return out


def _plain_act_bwd(s):
    F, rows = s["F"], s["rows"]
    h = _values(s["ckpt"][:rows], s["ckpt_sf"][:rows])
    g, u, da = h[:, :F], h[:, F:], s["da"][:rows].float()
    sig = 1 / (1 + torch.exp(-g))
    out = {}
    t = da
    if s["row_w"] is not None:
        s["gw"][:rows].copy_((da * g * sig * u).sum(1))
        out["gw"] = s["gw"]
        t = da * s["row_w"][:rows, None]
    gh = torch.cat([t * u * sig * (1 + g * (1 - sig)), t * g * sig], 1)
    if s["fp8"]:
        out["q"], out["sf"] = _put(s, gh, s["q"], s["sf"])
    else:
        s["gh"][:rows].copy_(gh)
        out["gh"] = s["gh"]
    return out


def _plain_comb_bwd(s):
    rows = s["rows"]
    valid = s["dst"] >= 0
    at = torch.where(valid, s["dst"], rows)
    g = s["g"].float()
    y = torch.cat([s["y"][:rows], s["y"].new_zeros(1, s["H"])])[at].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()[s["idx"].clamp(min=0)]
    out = {"gw": torch.where(valid, (y * g[:, None, :]).sum(2), 0.0)}
    del y
    w = torch.where(valid, s["w"], 0.0)
    row_w = torch.zeros(rows + 1, device="cuda").index_add_(0, at.view(-1), w.view(-1))[:-1]
    token = torch.zeros(rows + 1, dtype=torch.int64, device="cuda")
    token[at] = torch.arange(s["T"], device="cuda")[:, None].expand_as(at)
    token = token[:-1]
    if s["fp8"]:  # a row's bytes are its token's: the weight goes into the scale
        q, sf = _quantise(g)
        q = torch.where(row_w[:, None] != 0, q.to(FP8).float()[token] * row_w.sign()[:, None], 0.0)
        s["gy_q"].view(FP8)[:rows].copy_(q)
        _sf_rows(s, s["gy_sf"], s["H"], rows).copy_(sf[token] * row_w.abs()[:, None])
        out["q"], out["sf"] = s["gy_q"].view(FP8), s["gy_sf"]
    else:
        s["gy"][:rows].copy_(g[token] * row_w[:, None])
        out["gy"] = s["gy"]
    if s["bias"] is not None:
        dense = torch.zeros(s["T"], s["E"], device="cuda")
        dense.scatter_add_(1, s["idx"].clamp(min=0), w)
        out["gbias"] = dense.t() @ g
    return out


def _plain_product(s):
    D, N = s["D"], s["N"]
    a = _values(s["a"][:s["rows"]], _sf_rows(s, s["a_sf"], D, s["rows"]))
    # one product per expert with rows: a single batched one would have to pad every expert to
    # the longest, ten times the work on a skewed load
    for e, r0, r1 in s["segments"]:
        w = s["wq"][e].view(FP8).float().view(N, D // 128, 128)
        w.mul_(s["w_sf"][e].repeat_interleave(128, 0)[:N, :, None])
        s["out"][r0:r1].copy_(a[r0:r1] @ w.view(N, D).t())
    return {"out": s["out"]}


# ---- the package's calls --------------------------------------------------------------------

def _own_norm(ep, s):
    o = ep.alloc_rmsnorm(s["x"], residual=True, bf16=s["bf16"], fp8=True, col_major_sf=s["col"])
    ep.ep_rmsnorm(s["x"], s["gamma"], EPS, s["residual"], **o)
    return {"r": o["residual_out"], "q": o["y_fp8"].view(FP8), "sf": o["y_sf"], "y": o["y"]}


def _own_norm_bwd(ep, s):
    gx, gg = ep.ep_rmsnorm_backward(s["gy"], s["r"], s["gamma"], s["rstd"], s["gres"])
    return {"gx": gx, "ggamma": gg}


def _own_act(ep, s):
    kept = {} if s["ckpt"] is False else {"ckpt": s["ckpt"], "ckpt_sf": s["ckpt_sf"]}
    ep.ep_swiglu(s["handle"], s["h"], s["row_w"], act_fp8=s["q"], act_sf=s["sf"], **kept)
    out = {"q": s["q"].view(FP8), "sf": s["sf"]}
    if kept:
        out["ckpt"], out["ckpt_sf"] = s["ckpt"].view(FP8), s["ckpt_sf"]
    return out


def _own_act_bwd(ep, s):
    o = {"grad_fp8": s["q"], "grad_sf": s["sf"]} if s["fp8"] else {"grad_gate_up": s["gh"]}
    out = {"q": s["q"].view(FP8), "sf": s["sf"]} if s["fp8"] else {"gh": s["gh"]}
    if s["row_w"] is not None:
        out["gw"] = o["grad_row_weights"] = s["gw"]
    ep.ep_swiglu_backward(s["handle"], s["da"], s["ckpt"], s["ckpt_sf"], s["row_w"], **o)
    return out


def _own_comb_bwd(ep, s):
    o = {"grad_topk_weights": torch.empty(s["w"].shape, device="cuda")}
    out = {"gw": o["grad_topk_weights"]}
    if s["fp8"]:
        o["grad_y_fp8"], o["grad_y_sf"] = s["gy_q"], s["gy_sf"]
        out["q"], out["sf"] = s["gy_q"].view(FP8), s["gy_sf"]
    else:
        out["gy"] = o["grad_y"] = s["gy"]
    if s["bias"] is not None:
        out["gbias"] = o["grad_expert_bias"] = torch.empty(s["E"], s["H"], device="cuda")
    ep.ep_combine_weighted_backward(s["handle"], s["g"], s["y"], s["w"], s["bias"], **o)
    return out


def _own_product(ep, s):
    return {"out": ep.ep_expert_gemm(s["handle"], s["a"], s["a_sf"], s["wq"], s["w_sf"],
                                     out=s["out"])}


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "act": _plain_act,
          "act_bwd": _plain_act_bwd, "comb_bwd": _plain_comb_bwd, "product": _plain_product}
_OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "act": _own_act,
        "act_bwd": _own_act_bwd, "comb_bwd": _own_comb_bwd, "product": _own_product}


def run(state):
    if own:
        import combine_topk_idx_gb300 as ep
        return _OWN[state["op"]](ep, state)
    return _PLAIN[state["op"]](state)


# ---- the definition in 64 bits --------------------------------------------------------------

def _blocks64(v):
    """v / scale (what an e4m3 byte stands for, before its rounding) and the scales."""
    rows, n = v.shape
    sf = v.abs().unflatten(1, (n // 128, 128)).max(dim=2).values / 448
    full = sf.repeat_interleave(128, dim=1)
    return torch.nan_to_num(v / full, nan=0.0), sf


def _decode64(q, sf):
    return q.view(FP8).double() * sf.double().repeat_interleave(128, dim=-1)


def _spread64(s, q, sf):
    """q and sf of the rows in use, laid out like the receive buffers."""
    rows, n = q.shape
    whole = torch.zeros(s["alloc"], n, dtype=torch.float64, device="cuda")
    whole[:rows] = q
    tall = -(-s["alloc"] // 4) * 4 if s["col"] else s["alloc"]
    scales = torch.zeros(tall, n // 128, dtype=torch.float64, device="cuda")
    scales[:rows] = sf
    return whole, (scales.t() if s["col"] else scales).reshape(-1)


def _tall64(s, v):
    whole = torch.zeros(s["alloc"], *v.shape[1:], dtype=torch.float64, device="cuda")
    whole[:v.shape[0]] = v
    return whole


def exact(case, seed):
    op = case["op"]
    if op == "product" and 2.0 * case["T"] * case["K"] * case["N"] * case["D"] > 5e12:
        return None
    s = prepare(case, seed)
    rows = s.get("rows")
    if op == "norm":
        v = s["x"].double() + s["residual"].double()
        y = torch.sqrt(torch.einsum("th,th->t", v, v) / case["H"] + EPS)[:, None]
        y = s["gamma"].double() * v / y
        q, sf = _blocks64(y)
        return {"r": v, "q": q, "sf": sf, "y": y if case["bf16"] else None}
    if op == "norm_bwd":
        r, k = s["r"].double(), s["rstd"].double()[:, None]
        gy = s["gy"].double()
        gx = gy * s["gamma"].double() * k
        gx = gx - r * k * k * (gx * r).sum(1, keepdim=True) / case["H"]
        if s["gres"] is not None:
            gx = gx + s["gres"].double()
        return {"gx": gx, "ggamma": torch.einsum("th,th,to->h", gy, r, k)}
    if op == "act":
        h = s["h"][:rows].double()
        g, u = torch.chunk(h, 2, dim=1)
        a = torch.sigmoid(g) * g * u
        if s["row_w"] is not None:
            a = s["row_w"][:rows].double()[:, None] * a
        out = dict(zip(("q", "sf"), _spread64(s, *_blocks64(a))))
        if s["ckpt"] is not False:
            out |= {k: _tall64(s, v) for k, v in zip(("ckpt", "ckpt_sf"), _blocks64(h))}
        return out
    if op == "act_bwd":
        g, u = torch.chunk(_decode64(s["ckpt"][:rows], s["ckpt_sf"][:rows]), 2, dim=1)
        da, sig = s["da"][:rows].double(), torch.sigmoid(g)
        slope = sig + g * sig * (1 - sig)
        out = {}
        if s["row_w"] is not None:
            out["gw"] = _tall64(s, torch.einsum("rf,rf,rf->r", da, u, g * sig))
            da = da * s["row_w"][:rows].double()[:, None]
        gh = torch.cat([da * u * slope, da * sig * g], dim=1)
        if not case["fp8"]:
            return out | {"gh": _tall64(s, gh)}
        return out | dict(zip(("q", "sf"), _spread64(s, *_blocks64(gh))))
    if op == "comb_bwd":
        T, K, H = case["T"], s["w"].shape[1], case["H"]
        g, y = s["g"].double(), s["y"].double()
        gw = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        mix = torch.zeros(rows, dtype=torch.float64, device="cuda")
        src = torch.zeros(rows, dtype=torch.int64, device="cuda")
        bias = torch.zeros(case["E"], H, dtype=torch.float64, device="cuda")
        for k in range(K):  # slot by slot, over the tokens that have one
            t = torch.nonzero(s["dst"][:, k] >= 0).view(-1)
            d, e, w = s["dst"][t, k], s["idx"][t, k], s["w"][t, k].double()
            v = y[d]
            if s["bias"] is not None:
                v = v + s["bias"].double()[e]
                bias.index_add_(0, e, g[t] * w[:, None])
            gw[t, k] = (v * g[t]).sum(1)
            mix.index_add_(0, d, w)
            src[d] = t
        out = {"gw": gw}
        if case["fp8"]:
            q, sf = _blocks64(g)
            out["q"], out["sf"] = _spread64(s, q[src] * mix.sign()[:, None],
                                            sf[src] * mix.abs()[:, None])
        else:
            out["gy"] = _tall64(s, g[src] * mix[:, None])
        if s["bias"] is not None:
            out["gbias"] = bias
        return out
    sf = _sf_rows(s, s["a_sf"], case["D"], rows)
    out = torch.zeros(s["alloc"], case["N"], dtype=torch.float64, device="cuda")
    for e in torch.nonzero(s["cnt"]).view(-1).tolist():  # expert by expert
        mine = s["start"][e] + torch.arange(int(s["cnt"][e]), device="cuda")
        block = s["w_sf"][e].double().repeat_interleave(128, 0)[:case["N"]]
        w = s["wq"][e].view(FP8).double() * block.repeat_interleave(128, 1)
        out[mine] = _decode64(s["a"][mine], sf[mine]) @ w.t()
    return {"out": out}
