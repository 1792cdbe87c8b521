"""The fused operators of a decode or prefill step around the projections: what they
compute, the sizes they are used at, and how they are called.

Three operators, the parts of a transformer layer that touch a skinny GEMM's input and
output:

* ``norm``: root-mean-square norm of x, or of x + residual (which is also returned as the
  new residual), to bfloat16 or to 8-bit floats (e4m3) with one float32 scale per row or per
  128 consecutive columns;
* ``linear``: a bfloat16 projection with bias, activation and residual in its epilogue, or
  its gated form act(x Wg^T + bg) * (x Wu^T + bu);
* ``fp8``: the same two forms on 8-bit x and W, with scales per row of x and of W
  (``scales`` = "row") or per 128 columns of x and 128 x 128 block of W ("block").

``run`` computes them plainly in 32 bits, or, where ``own`` is true, with the framework's
operators. ``exact`` computes them in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
GROUP = 128
TOP = 448.0            # the largest e4m3 value
LEAST = 2.0 ** -100    # the least largest magnitude a scale is made from


# ---- cases ------------------------------------------------------------------

def _norm(name, M, D, out, residual, stride=0):
    return {"name": name, "op": "norm", "M": M, "D": D, "out": out, "residual": residual,
            "stride": stride or D}


def _linear(name, op, M, N, K, gated=False, scales="", act="none", bias=False, residual=False,
            f32=False):
    return {"name": name, "op": op, "M": M, "N": N, "K": K, "gated": gated, "scales": scales,
            "act": act, "bias": bias, "residual": residual, "f32": f32}


def listed():
    return [
        # one token's norm before a layer's input projection: latency is everything
        _norm("norm_step", 1, 4096, "bf16", True),
        # a few tokens' norm feeding an 8-bit projection with block scales
        _norm("norm_fp8_step", 4, 4096, "group", True),
        # the norm of the latent half of a merged projection's output: a strided input
        _norm("norm_latent", 515, 1536, "bf16", False, 2048),
        # a long prompt's norm feeding an 8-bit projection with row scales
        _norm("norm_fp8_prefill", 8192, 4096, "row", True),
        # attention's output projection for one token, added to the residual stream
        _linear("linear_step", "linear", 1, 4096, 4096, residual=True),
        # a shared expert's gate and up projections for three tokens (speculative decoding)
        _linear("gated_step", "linear", 3, 1024, 4096, gated=True, act="silu"),
        # a batch of sequences, an odd number of outputs kept in float32
        _linear("linear_batch", "linear", 48, 8191, 1536, act="gelu", bias=True, f32=True),
        # a prompt through a biased layer with its activation and residual
        _linear("linear_prefill", "linear", 4096, 4096, 4096, act="gelu_tanh", bias=True,
                residual=True),
        # one token through the widest input projection, 8-bit weights with row scales
        _linear("fp8_step", "fp8", 1, 12576, 4096, scales="row"),
        # a shared expert's gate and up projections, 8-bit weights with block scales
        _linear("fp8_gated_step", "fp8", 8, 1024, 4096, gated=True, scales="block", act="silu"),
        # a batch of sequences through the deepest output projection
        _linear("fp8_batch", "fp8", 100, 4096, 8192, scales="block", residual=True),
        # a prompt through the same projection with row scales
        _linear("fp8_prefill", "fp8", 4096, 4096, 8192, scales="row", bias=True, residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "linear", "fp8"))
    if op == "norm":
        D = _log_int(rng, 64, 16384)
        if rng.random() < 0.6:
            D = max(8, D // 8 * 8)
        M = _log_int(rng, 1, max(1, min(16384, 8192 * 4096 // D)))
        stride = D + rng.choice((0, 0, 8, 512))
        return {"op": op, "M": M, "D": D, "out": rng.choice(("bf16", "row", "group")),
                "residual": rng.random() < 0.6, "stride": stride}
    gated = rng.random() < 0.35
    K = _log_int(rng, 128, 8192) // 16 * 16
    N = _log_int(rng, 64, 12576 if not gated else 6288)
    most = 4096 * 4096 * (4096 if op == "linear" else 8192) // (N * K * (2 if gated else 1))
    M = _log_int(rng, 1, max(1, min(4096, most)))
    return {"op": op, "M": M, "N": N, "K": K, "gated": gated,
            "scales": rng.choice(("row", "block")) if op == "fp8" else "",
            "act": rng.choice(("silu", "gelu_tanh", "relu")) if gated
            else rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")),
            "bias": rng.random() < 0.5, "residual": not gated and rng.random() < 0.5,
            "f32": rng.random() < 0.2}


def work(case):
    M = case["M"]
    if case["op"] == "norm":
        D = case["D"]
        read = 2 * M * D * (2 if case["residual"] else 1) + 2 * D
        wrote = M * D * (2 if case["out"] == "bf16" else 1) + (2 * M * D if case["residual"] else 0)
        wrote += {"bf16": 0, "row": 4 * M, "group": 4 * M * -(-D // GROUP)}[case["out"]]
        return {"bytes": read + wrote, "flops": 5 * M * D}
    N, K = case["N"], case["K"]
    mats = 2 if case["gated"] else 1
    size = 2 if case["op"] == "linear" else 1
    read = size * (M * K + mats * N * K) + (2 * mats * N if case["bias"] else 0)
    read += 2 * M * N if case["residual"] else 0
    if case["scales"] == "row":
        read += 4 * (M + mats * N)
    elif case["scales"] == "block":
        read += 4 * (M * -(-K // GROUP) + mats * -(-N // GROUP) * -(-K // GROUP))
    return {"bytes": read + M * N * (4 if case["f32"] else 2), "flops": 2 * M * N * K * mats}


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


def _to_fp8_rows(x):
    scale = x.abs().amax(dim=1).clamp_min(LEAST) / TOP
    return (x / scale[:, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn), scale


def _to_fp8_blocks(x, rows):
    """Scales over blocks of `rows` x 128."""
    M, K = x.shape
    p = torch.nn.functional.pad(x, (0, -K % GROUP, 0, -M % rows))
    b = p.view(p.shape[0] // rows, rows, p.shape[1] // GROUP, GROUP)
    scale = b.abs().amax(dim=(1, 3)).clamp_min(LEAST) / TOP
    q = (b / scale[:, None, :, None]).clamp(-TOP, TOP).view(p.shape)[:M, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), scale


def prepare(case, seed):
    g = _gen(seed)
    M = case["M"]
    s = {"case": case}
    if case["op"] == "norm":
        D = case["D"]
        s["x"] = _activations(g, M, case["stride"]).to(torch.bfloat16)[:, :D]
        s["weight"] = (1.0 + 0.1 * _randn(g, D)).to(torch.bfloat16)
        s["residual"] = _activations(g, M, D).to(torch.bfloat16) if case["residual"] else None
        if own:
            from bf16_skinny_gemm_amd import torch_op
            s["ops"] = torch_op
        return s
    N, K = case["N"], case["K"]
    mats = 2 if case["gated"] else 1
    x = _activations(g, M, K) if case["op"] == "fp8" else _randn(g, M, K)
    w = [_randn(g, N, K) / math.sqrt(K) for _ in range(mats)]
    if case["op"] == "linear":
        s["x"], s["w"] = x.to(torch.bfloat16), [v.to(torch.bfloat16) for v in w]
    else:
        x = x / x.pow(2).mean(dim=1, keepdim=True).sqrt()
        if case["scales"] == "row":
            s["x"], s["xs"] = _to_fp8_rows(x)
            q = [_to_fp8_rows(v) for v in w]
        else:
            s["x"], s["xs"] = _to_fp8_blocks(x, 1)
            q = [_to_fp8_blocks(v, GROUP) for v in w]
        s["w"], s["ws"] = [v[0] for v in q], [v[1] for v in q]
    s["bias"] = [(0.5 * _randn(g, N)).to(torch.bfloat16) if case["bias"] else None
                 for _ in range(mats)]
    s["residual"] = _activations(g, M, N).to(torch.bfloat16) if case["residual"] else None
    if own:
        from bf16_skinny_gemm_amd import torch_op
        s["ops"] = torch_op
    return s


# ---- the framework's calls --------------------------------------------------

def _own_norm(s):
    c, ops = s["case"], s["ops"]
    x, w, r = s["x"], s["weight"], s["residual"]
    if c["out"] == "bf16":
        return ops.rms_norm(x, w, EPS) if r is None else ops.add_rms_norm(x, r, w, EPS)
    group = 0 if c["out"] == "row" else GROUP
    if r is None:
        return ops.rms_norm_fp8(x, w, EPS, group)
    return ops.add_rms_norm_fp8(x, r, w, EPS, group)


def _own_linear(s):
    c, ops = s["case"], s["ops"]
    x, w, b = s["x"], s["w"], s["bias"]
    if c["op"] == "linear":
        if c["gated"]:
            return ops.linear_gated(x, w[0], w[1], b[0], b[1], c["act"], c["f32"])
        return ops.linear_act(x, w[0], b[0], s["residual"], c["act"], c["f32"])
    xs, ws = s["xs"], s["ws"]
    if c["gated"]:
        return ops.linear_gated_fp8(x, xs, w[0], ws[0], w[1], ws[1], b[0], b[1], c["act"], c["f32"])
    return ops.linear_fp8(x, xs, w[0], ws[0], b[0], s["residual"], c["act"], c["f32"])


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


def _plain_norm(s):
    c = s["case"]
    M, D = c["M"], c["D"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.pow(2).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    if c["out"] == "bf16":
        got = [y.to(torch.bfloat16)]
    elif c["out"] == "row":
        scale = y.abs().amax(dim=1).clamp_min(LEAST) / TOP
        got = [(y / scale[:, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn), scale]
    else:
        p = torch.nn.functional.pad(y, (0, -D % GROUP)).view(M, -1, GROUP)
        scale = p.abs().amax(dim=2).clamp_min(LEAST) / TOP
        q = (p / scale[:, :, None]).clamp(-TOP, TOP).view(M, -1)[:, :D].to(torch.float8_e4m3fn)
        got = [q.contiguous(), scale]
    if s["residual"] is not None:
        got.append(h.to(torch.bfloat16))
    return got[0] if len(got) == 1 else tuple(got)


def _wide(q, scale, rows):
    """8-bit values times the scale of their rows x 128 block, in 32 bits."""
    M, K = q.shape
    full = scale.repeat_interleave(GROUP, dim=1)[:, :K]
    if rows > 1:
        full = full.repeat_interleave(rows, dim=0)[:M]
    return q.float() * full


def _plain_product(s, i):
    c = s["case"]
    if c["op"] == "linear":
        z = s["x"].float() @ s["w"][i].float().t()
    elif c["scales"] == "row":
        z = s["x"].float() @ s["w"][i].float().t() * s["xs"][:, None] * s["ws"][i]
    else:
        z = _wide(s["x"], s["xs"], 1) @ _wide(s["w"][i], s["ws"][i], GROUP).t()
    return z if s["bias"][i] is None else z + s["bias"][i].float()


def _plain_linear(s):
    c = s["case"]
    y = _act(_plain_product(s, 0), c["act"])
    if c["gated"]:
        y = y * _plain_product(s, 1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y if c["f32"] else y.to(torch.bfloat16)


def run(state):
    if state["case"]["op"] == "norm":
        return _own_norm(state) if own else _plain_norm(state)
    return _own_linear(state) if own else _plain_linear(state)


# ---- the definition in 64 bits ----------------------------------------------

def _e4m3(v):
    """The nearest e4m3 value, ties to even, |v| <= 448: 3 fraction bits down to 2^-6, then
    multiples of 2^-9."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return torch.round(v / step).mul(step).clamp(-TOP, TOP)


def _exact_norm(s):
    c = s["case"]
    h = s["x"].double()
    r = s["residual"]
    h = h if r is None else h + r.double()
    ms = torch.einsum("md,md->m", h, h) / c["D"]
    y = s["weight"].double()[None, :] * (h / torch.sqrt(ms + EPS)[:, None])
    tail = () if r is None else (h,)
    if c["out"] == "bf16":
        return (y,) + tail if tail else y
    width = c["D"] if c["out"] == "row" else GROUP
    parts = torch.split(y, width, dim=1)
    scales = [torch.maximum(p.abs().max(dim=1).values, torch.tensor(LEAST, device="cuda")) / TOP
              for p in parts]
    q = torch.cat([_e4m3(p / t[:, None]) for p, t in zip(parts, scales)], dim=1)
    scale = scales[0] if c["out"] == "row" else torch.stack(scales, dim=1)
    return (q, scale) + tail


def _exact_product(s, i):
    c = s["case"]
    x, w = s["x"].double(), s["w"][i].double()
    if c["op"] == "fp8" and c["scales"] == "block":
        z = torch.zeros(c["M"], c["N"], dtype=torch.float64, device="cuda")
        of = torch.arange(c["N"], device="cuda") // GROUP
        for k in range(0, c["K"], GROUP):
            b = k // GROUP
            part = x[:, k:k + GROUP] @ w[:, k:k + GROUP].t().contiguous()
            z += part * s["xs"][:, b].double()[:, None] * s["ws"][i][of, b].double()
    else:
        z = x @ w.t()
        if c["op"] == "fp8":
            z = torch.outer(s["xs"].double(), s["ws"][i].double()) * z
    return z if s["bias"][i] is None else s["bias"][i].double() + z


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    z = _exact_product(s, 0)
    if case["act"] == "relu":
        z = z.clamp_min(0.0)
    elif case["act"] == "silu":
        z = z * torch.special.expit(z)
    elif case["act"] == "gelu":
        z = z * torch.special.ndtr(z)
    elif case["act"] == "gelu_tanh":
        z = z * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * z * (1.0 + 0.044715 * z ** 2))
    if case["gated"]:
        z = z * _exact_product(s, 1)
    return z if s["residual"] is None else s["residual"].double() + z
