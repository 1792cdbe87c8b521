"""The 8-bit integer projections and the routed experts of a decode or prefill step: what they
compute, the sizes they are used at, and how they are called.

Four operators:

* ``int8``: a projection of 8-bit integers with a scale for each row of x and each output
  channel, with bias, activation, gate and residual in its epilogue. x comes as 8-bit integers
  (``x`` = "int8"), or as bfloat16 that the pass makes 8-bit integers of: as it is ("plain"),
  through its root-mean-square norm ("norm"), or through that of x + residual stream ("add"),
  where the new residual stream is returned too;
* ``route``: the k best experts of every token and their weights, from the router's logits;
* ``experts``: the routed experts of a few tokens, both projections and the weighted sum, on
  weights in bfloat16, e4m3 (block or row scales) or 8-bit integers (row scales);
* ``layer``: ``route`` and ``experts`` one after the other.

``run`` computes them plainly in 32 bits (the values that a ranking compares in 64), or, where
``own`` is true, with the framework's operators. ``exact`` computes them in 64 bits.
"""
import functools
import math

import torch

own = False

EPS = 1e-6
GROUP = 128
TOP8, TOP_E4M3 = 127.0, 448.0
LEAST = 2.0 ** -100    # the least largest magnitude a scale is made from


# ---- cases ------------------------------------------------------------------

def _int8(name, M, N, K, x="int8", gated=False, act="none", bias=False, residual=False, f32=False):
    return {"name": name, "op": "int8", "M": M, "N": N, "K": K, "x": x, "gated": gated, "act": act,
            "bias": bias, "residual": residual, "f32": f32}


def _route(name, M, E, k, score="softmax", bias=False, groups=1, kept=1, renormalize=True, scale=1.0):
    return {"name": name, "op": "route", "M": M, "E": E, "k": k, "score": score, "bias": bias,
            "groups": groups, "kept": kept, "renormalize": renormalize, "scale": scale}


def _experts(name, M, E, k, H, I, kind, residual=False, act="silu"):
    return {"name": name, "op": "experts", "M": M, "E": E, "k": k, "H": H, "I": I, "kind": kind,
            "residual": residual, "act": act}


def listed():
    return [
        # one token through the widest input projection, 8-bit weights
        _int8("int8_step", 1, 12576, 4096),
        # a shared expert's gate and up projections for four tokens, from the residual stream
        _int8("int8_gated_step", 4, 1024, 4096, x="add", gated=True, act="silu"),
        # the LM head for five drafted tokens: float32 logits
        _int8("int8_logits", 5, 77440, 4096, f32=True),
        # a batch of sequences through the deepest output projection, from its bfloat16 input
        _int8("int8_batch", 100, 4096, 8192, x="plain", residual=True),
        # a prompt through the same projection, 8-bit input, an odd number of rows
        _int8("int8_prefill", 4095, 4096, 8192, bias=True, residual=True),
        # one token's choice of experts, corrected by a bias
        _route("route_step", 1, 288, 8, score="sigmoid", bias=True, scale=2.5),
        # a prompt's choice of experts, limited to half of the groups of experts
        _route("route_prefill", 8191, 256, 8, score="sigmoid", bias=True, groups=8, kept=4, scale=2.5),
        # one token through its experts, unquantized
        _experts("experts_step", 1, 288, 8, 4096, 1024, "bf16"),
        # five drafted tokens, e4m3 weights with block scales, added to the residual stream
        _experts("experts_draft", 5, 288, 8, 4096, 1024, "block", residual=True),
        # a batch of sequences, 8-bit integer weights, an intermediate width that is no multiple
        # of the tiles'
        _experts("experts_batch", 61, 64, 6, 2048, 1408, "int8"),
        # few, wide experts that many tokens share, unquantized
        _experts("experts_shared", 37, 16, 2, 4096, 1536, "bf16"),
        # the routed half of a layer for three tokens: router and experts, one after the other
        dict(_experts("layer_step", 3, 64, 4, 2048, 768, "row", residual=True), op="layer"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def draw(rng):
    op = rng.choice(("int8", "int8", "route", "experts", "experts", "layer"))
    if op == "int8":
        gated = rng.random() < 0.35
        K = _log_int(rng, 128, 8192) // 16 * 16
        N = _log_int(rng, 64, 12576 if not gated else 6288)
        most = 4095 * 4096 * 8192 // (N * K * (2 if gated else 1))
        M = _log_int(rng, 1, max(1, min(4095, most)))
        x = rng.choice(("int8", "int8", "plain", "norm", "add"))
        return {"op": op, "M": M, "N": N, "K": K, "x": x, "gated": gated,
                "act": rng.choice(ACTS[1:]) if gated else rng.choice(ACTS),
                "bias": rng.random() < 0.5, "residual": not gated and rng.random() < 0.5,
                "f32": x == "int8" and rng.random() < 0.3}
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        E = groups * _log_int(rng, 8, 512 // groups)
        kept = rng.randint(1, groups)
        k = _log_int(rng, 1, min(16, E * kept // groups))
        return {"op": op, "M": _log_int(rng, 1, min(8191, 8191 * 256 // E)), "E": E, "k": k,
                "score": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5,
                "groups": groups, "kept": kept, "renormalize": rng.random() < 0.7,
                "scale": rng.choice((1.0, 2.5))}
    H = _log_int(rng, 512, 5120) // 16 * 16
    I = _log_int(rng, 128, 2048) // 16 * 16
    E = _log_int(rng, 8, max(8, min(288, 288 * 4096 * 1024 // (H * I))))
    k = _log_int(rng, 1, 8)
    most = 61 * 6 * 2048 * 1408 // (H * I * k)
    return {"op": op, "M": _log_int(rng, 1, max(1, min(128, most))), "E": E, "k": k, "H": H, "I": I,
            "kind": rng.choice(("bf16", "block", "row", "int8")), "residual": rng.random() < 0.5,
            "act": rng.choice(("silu", "gelu_tanh", "gelu"))}


def _work_int8(c):
    M, N, K, mats = c["M"], c["N"], c["K"], 2 if c["gated"] else 1
    read = mats * (N * K + 4 * N) + (2 * mats * N if c["bias"] else 0)
    read += 2 * M * N if c["residual"] else 0
    read += M * K + 4 * M if c["x"] == "int8" else 2 * M * K
    read += 2 * K if c["x"] in ("norm", "add") else 0
    read += 2 * M * K if c["x"] == "add" else 0
    wrote = M * N * (4 if c["f32"] else 2) + (2 * M * K if c["x"] == "add" else 0)
    return {"bytes": read + wrote, "flops": 2 * M * N * K * mats}


def _work_route(c):
    return {"bytes": 4 * c["M"] * c["E"] + 8 * c["M"] * c["k"], "flops": 10 * c["M"] * c["E"]}


def _work_experts(c):
    M, E, k, H, I = c["M"], c["E"], c["k"], c["H"], c["I"]
    used = E * (1.0 - (1.0 - k / E) ** M)   # experts that some token picks: each is read once
    size = 2 if c["kind"] == "bf16" else 1
    read = 3 * used * I * H * size + 2 * M * H * (2 if c["residual"] else 1) + 8 * M * k
    return {"bytes": read + 2 * M * H, "flops": 6 * M * k * I * H}


def work(case):
    if case["op"] == "int8":
        return _work_int8(case)
    if case["op"] == "route":
        return _work_route(case)
    w = _work_experts(case)
    return dict(w, bytes=w["bytes"] + 4 * case["M"] * case["E"]) if case["op"] == "layer" else w


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, M, D):
    """Normal values with every 97th channel 16 times as large, as hidden states have them."""
    x = _randn(g, M, D)
    x[:, ::97] *= 16.0
    return x


def _scale_of(x, top):
    return x.abs().amax(dim=-1).clamp_min(LEAST) / top


def _int8_rows(x):
    scale = _scale_of(x, TOP8)
    return torch.round(x / scale[..., None]).to(torch.int8), scale


def _e4m3_rows(x):
    scale = _scale_of(x, TOP_E4M3)
    return (x / scale[..., None]).clamp(-TOP_E4M3, TOP_E4M3).to(torch.float8_e4m3fn), scale


def _e4m3_blocks(x):
    """Scales over blocks of 128 x 128 of the last two dimensions."""
    *lead, N, K = x.shape
    p = torch.nn.functional.pad(x, (0, -K % GROUP, 0, -N % GROUP))
    b = p.view(*lead, p.shape[-2] // GROUP, GROUP, p.shape[-1] // GROUP, GROUP)
    scale = b.abs().amax(dim=(-3, -1)).clamp_min(LEAST) / TOP_E4M3
    q = (b / scale[..., :, None, :, None]).clamp(-TOP_E4M3, TOP_E4M3).view(p.shape)[..., :N, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), scale


_STORED = {"bf16": lambda x: (x.to(torch.bfloat16), None), "block": _e4m3_blocks, "row": _e4m3_rows,
           "int8": _int8_rows}


def _expert_weights(g, E, N, K, kind):
    """[E, N, K] weights of the kind with their scales."""
    return _STORED[kind](_randn(g, E, N, K) / math.sqrt(K))


def _prepare_int8(s, g, c):
    M, N, K, mats = c["M"], c["N"], c["K"], 2 if c["gated"] else 1
    x = _activations(g, M, K)
    if c["x"] == "int8":
        s["x"], s["xs"] = _int8_rows(x)
    else:
        s["x"] = x.to(torch.bfloat16)
        s["norm"] = (1.0 + 0.1 * _randn(g, K)).to(torch.bfloat16)
        s["stream"] = _activations(g, M, K).to(torch.bfloat16)
    q = [_int8_rows(_randn(g, N, K) / math.sqrt(K)) for _ in range(mats)]
    s["w"], s["ws"] = [v[0] for v in q], [v[1] for v in q]
    s["bias"] = [(0.5 * _randn(g, N)).to(torch.bfloat16) if c["bias"] else None for _ in range(mats)]
    s["residual"] = _activations(g, M, N).to(torch.bfloat16) if c["residual"] else None


def _prepare_route(s, g, c):
    s["logits"] = 2.0 * _randn(g, c["M"], c["E"])
    s["correct"] = 0.1 * _randn(g, c["E"]) if c["bias"] else None


def _prepare_experts(s, g, c):
    M, E, k, H, I = c["M"], c["E"], c["k"], c["H"], c["I"]
    s["x"] = _randn(g, M, H).to(torch.bfloat16)
    s["residual"] = _activations(g, M, H).to(torch.bfloat16) if c["residual"] else None
    s["logits"] = 2.0 * _randn(g, M, E)
    if c["op"] == "experts":  # chosen by a router that ran before
        v, ids = torch.topk(s["logits"], k, dim=1)
        s["ids"], s["weights"] = ids.to(torch.int32), torch.softmax(v, dim=1)
    s["gate"], s["gate_s"] = _expert_weights(g, E, I, H, c["kind"])
    s["up"], s["up_s"] = _expert_weights(g, E, I, H, c["kind"])
    s["down"], s["down_s"] = _expert_weights(g, E, H, I, c["kind"])


def prepare(case, seed):
    s = {"case": case}
    {"int8": _prepare_int8, "route": _prepare_route, "experts": _prepare_experts,
     "layer": _prepare_experts}[case["op"]](s, _gen(seed), case)
    return s


# ---- the framework's calls --------------------------------------------------

@functools.cache
def _ops():
    from bf16_skinny_gemm_amd import torch_op
    return torch_op


def _own_int8(s):
    c, ops, tail = s["case"], _ops(), ()
    if c["x"] == "int8":
        q, xs = s["x"], s["xs"]
    elif c["x"] == "plain":
        q, xs = ops.quantize_int8(s["x"])
    elif c["x"] == "norm":
        q, xs = ops.rms_norm_int8(s["x"], s["norm"], EPS)
    else:
        q, xs, *tail = ops.add_rms_norm_int8(s["x"], s["stream"], s["norm"], EPS)
    w, ws, b = s["w"], s["ws"], s["bias"]
    if c["gated"]:
        y = ops.linear_gated_int8(q, xs, w[0], ws[0], w[1], ws[1], b[0], b[1], c["act"], c["f32"])
    else:
        y = ops.linear_int8(q, xs, w[0], ws[0], b[0], s["residual"], c["act"], c["f32"])
    return (y, *tail)


def _own_route(s):
    c = s["case"]
    return _ops().route(s["logits"], c["k"], c["score"], s["correct"], c["groups"], c["kept"],
                        c["renormalize"], c["scale"])


def _own_experts(s, ids, weights):
    return _ops().experts(s["x"], ids, weights, s["gate"], s["up"], s["down"], s["gate_s"], s["up_s"],
                          s["down_s"], s["residual"], s["case"]["act"])


def _own(s):
    c = s["case"]
    if c["op"] == "int8":
        return _own_int8(s)
    if c["op"] == "route":
        return _own_route(s)
    if c["op"] == "experts":
        return _own_experts(s, s["ids"], s["weights"])
    ids, weights = _ops().route(s["logits"], c["k"])
    return _own_experts(s, ids, weights), ids, weights


# ---- the plain forms --------------------------------------------------------

def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_input(s):
    """The 8-bit x as 32-bit numbers, its scales, and the new residual stream."""
    x = s["x"].float()
    how = s["case"]["x"]
    if how == "int8":
        return x, s["xs"], ()
    tail = ()
    if how == "add":
        x = x + s["stream"].float()
        tail = (x.to(torch.bfloat16),)
    if how != "plain":
        x = x * torch.rsqrt(x.pow(2).mean(dim=1, keepdim=True) + EPS) * s["norm"].float()
    scale = _scale_of(x, TOP8)
    return torch.round(x / scale[:, None]), scale, tail


def _plain_product(s, q, xs, i):
    z = q @ s["w"][i].float().t() * xs[:, None] * s["ws"][i]
    return z if s["bias"][i] is None else z + s["bias"][i].float()


def _plain_int8(s):
    c = s["case"]
    q, xs, tail = _plain_input(s)
    y = _act(_plain_product(s, q, xs, 0), c["act"])
    if c["gated"]:
        y = y * _plain_product(s, q, xs, 1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return (y if c["f32"] else y.to(torch.bfloat16), *tail)


def _plain_route(logits, k, score="softmax", correct=None, groups=1, kept=1, renormalize=True,
                 scale=1.0):
    M, E = logits.shape
    v = logits.double()
    if score == "softmax":
        e = torch.exp(v - v.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-v))
    rank = v if correct is None else p + correct.double()
    if groups > 1:
        by = torch.sort(rank.view(M, groups, -1), dim=2, descending=True).values
        best = by[:, :, 0] if correct is None else by[:, :, :2].sum(dim=2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :kept]
        left = torch.zeros_like(best, dtype=torch.bool).scatter(1, order, True)
        rank = torch.where(left[:, :, None], rank.view(M, groups, -1), -math.inf).view(M, E)
    ids = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids).float()
    if renormalize:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), w * scale


def _picked(w, scale, ids, kind):
    """The weights of each pair's expert in 32 bits."""
    v = w[ids].float()
    if kind == "bf16":
        return v
    t = scale[ids]
    if kind != "block":
        return v * t[:, :, None]
    wide = t.repeat_interleave(GROUP, dim=1)[:, :v.shape[1]]
    return v * wide.repeat_interleave(GROUP, dim=2)[:, :, :v.shape[2]]


def _plain_experts(s, ids, weights):
    c = s["case"]
    M, k, H, kind = c["M"], c["k"], c["H"], c["kind"]
    at = ids.reshape(-1).long()
    x = s["x"].float().repeat_interleave(k, dim=0)[:, :, None]
    g = torch.bmm(_picked(s["gate"], s["gate_s"], at, kind), x)
    u = torch.bmm(_picked(s["up"], s["up_s"], at, kind), x)
    z = torch.bmm(_picked(s["down"], s["down_s"], at, kind), _act(g, c["act"]) * u)
    y = (z.view(M, k, H) * weights[:, :, None]).sum(dim=1)
    return (y if s["residual"] is None else y + s["residual"].float()).to(torch.bfloat16)


def _plain(s):
    c = s["case"]
    if c["op"] == "int8":
        return _plain_int8(s)
    if c["op"] == "route":
        return _plain_route(s["logits"], c["k"], c["score"], s["correct"], c["groups"], c["kept"],
                            c["renormalize"], c["scale"])
    if c["op"] == "experts":
        return _plain_experts(s, s["ids"], s["weights"])
    ids, weights = _plain_route(s["logits"], c["k"])
    return _plain_experts(s, ids, weights), ids, weights


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits ----------------------------------------------

def _exact_act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * z * (1.0 + 0.044715 * z ** 2))
    return z


def _exact_int8(s):
    c, tail = s["case"], ()
    x = s["x"].double()
    if c["x"] == "int8":
        xs = s["xs"].double()
    else:
        if c["x"] == "add":
            x = s["stream"].double() + x
            tail = (x,)
        if c["x"] != "plain":
            ms = torch.einsum("md,md->m", x, x) / c["K"]
            x = s["norm"].double()[None, :] * (x / torch.sqrt(ms + EPS)[:, None])
        xs = torch.maximum(x.abs().max(dim=1).values, torch.tensor(LEAST, device="cuda")) / TOP8
        x = torch.round(x / xs[:, None])

    def product(i):
        z = torch.outer(xs, s["ws"][i].double()) * (x @ s["w"][i].double().t())
        return z if s["bias"][i] is None else s["bias"][i].double() + z

    y = _exact_act(product(0), c["act"])
    if c["gated"]:
        y = y * product(1)
    return (y if s["residual"] is None else s["residual"].double() + y, *tail)


def _exact_route(logits, k, score="softmax", correct=None, groups=1, kept=1, renormalize=True,
                 scale=1.0):
    """One expert after the other: the best left, the lowest index among equals."""
    v = logits.double()
    M, E = v.shape
    rows = torch.arange(M, device="cuda")
    p = torch.softmax(v, dim=1) if score == "softmax" else torch.special.expit(v)
    rank = v.clone() if correct is None else correct.double()[None, :] + p
    if groups > 1:
        left = rank.view(M, groups, E // groups)
        total = left.max(dim=2).values
        if correct is not None and E > groups:
            total = total + left.kthvalue(E // groups - 1, dim=2).values
        dropped = torch.ones(M, groups, dtype=torch.bool, device="cuda")
        for _ in range(kept):
            best = (total == total.max(dim=1, keepdim=True).values).int().argmax(dim=1)
            dropped[rows, best] = False
            total[rows, best] = -math.inf
        left[dropped] = -math.inf
    ids = torch.empty(M, k, dtype=torch.int32, device="cuda")
    for j in range(k):
        best = (rank == rank.max(dim=1, keepdim=True).values).int().argmax(dim=1)
        ids[:, j] = best
        rank[rows, best] = -math.inf
    w = torch.gather(p, 1, ids.long())
    if renormalize:
        w = torch.nn.functional.normalize(w, p=1.0, dim=1)
    return ids, scale * w


def _exact_weight(s, name, e):
    w, t = s[name][e].double(), s[name + "_s"]
    if t is None:
        return w
    t = t[e].double()
    if t.dim() == 1:
        return t[:, None] * w
    n, m = w.shape
    return w * torch.kron(t, torch.ones(GROUP, GROUP, dtype=torch.float64, device="cuda"))[:n, :m]


def _exact_experts(s, ids, weights):
    c = s["case"]
    y = torch.zeros(c["M"], c["H"], dtype=torch.float64, device="cuda")
    x = s["x"].double()
    for e in torch.unique(ids).tolist():
        m, j = torch.nonzero(ids == e, as_tuple=True)
        gate = x[m] @ _exact_weight(s, "gate", e).t()
        h = _exact_act(gate, c["act"]) * (x[m] @ _exact_weight(s, "up", e).t())
        y.index_add_(0, m, weights[m, j].double()[:, None] * (h @ _exact_weight(s, "down", e).t()))
    return y if s["residual"] is None else s["residual"].double() + y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "int8":
        return _exact_int8(s)
    if case["op"] == "route":
        return _exact_route(s["logits"], case["k"], case["score"], s["correct"], case["groups"],
                            case["kept"], case["renormalize"], case["scale"])
    if case["op"] == "experts":
        return _exact_experts(s, s["ids"], s["weights"])
    ids, weights = _exact_route(s["logits"], case["k"])
    return _exact_experts(s, ids, weights), ids, weights
