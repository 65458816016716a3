"""The norm that feeds the MoE layer and its 8-bit integer experts: cases, plain forms and calls.

Three operators (`op` of a case):
  norm  residual addition, RMS norm and an optional 8-bit output with scales
            s = x + r, n = s * g / sqrt(mean(s^2) + eps) per row; outputs round(s), round(n) and the codes of n
  gemm  grouped matrix product of int8 codes with a scale per token and per output channel
            y[i] = (x[i] . w[e(i)]^T) * x_scale[i] * w_scale[e(i)], rows grouped by expert
  ffn   the SwiGLU experts on it, from bf16 activations: int8 per token, gate and up product, SiLU(gate) * up,
        int8 per row, down product; the rows of y are grouped by expert

`own` false: the plain forms in torch operations (fp32, each output rounded once). `own` true: the calls of the
framework's operators. `exact` computes the same from the definitions in 64 bits.
"""
import math
import random  # noqa: F401  (draw() takes a random.Random)

import torch

own = False
DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token of a DeepSeek-V3-shaped fp8 layer: latency
        dict(name="norm-1-fp8", op="norm", rows=1, cols=7168, x="bf16", res="bf16", y="bf16", quant="fp8", pad=0),
        # a decode batch whose input is the fp32 output of the layer before (bf16 layers write fp32), int8 experts next
        dict(name="norm-128-int8", op="norm", rows=128, cols=7168, x="f32", res="bf16", y="bf16", quant="int8", pad=0),
        # an odd row length and odd strides: no 16-byte loads possible; norm alone
        dict(name="norm-1027-odd", op="norm", rows=1027, cols=4099, x="bf16", res="bf16", y="bf16", quant="none", pad=2),
        # the prefill batch of a DeepSeek-V3-shaped MX layer
        dict(name="norm-8192-mx", op="norm", rows=8192, cols=7168, x="bf16", res="bf16", y="bf16", quant="mx", pad=0),
        # one token through one dense projection (the shared expert's gate and up): the weight stream
        dict(name="gemm-1-dense", op="gemm", rows=1, E=1, N=4096, K=7168, out="bf16", skew=0.0),
        # 83 tokens (the grouped top-K operator's batch) down from the intermediate size, fp32 rows out
        dict(name="gemm-83-dense", op="gemm", rows=83, E=1, N=7168, K=2048, out="f32", skew=0.0),
        # the shared expert's gate and up over a prefill batch: one large dense product
        dict(name="gemm-8192-dense", op="gemm", rows=8192, E=1, N=4096, K=7168, out="bf16", skew=0.0),
        # the down projection of a skewed decode batch: 1024 rows over 256 experts, many of them empty
        dict(name="gemm-1024-zipf", op="gemm", rows=1024, E=256, N=7168, K=2048, out="bf16", skew=1.2),
        # one decoded token and its 8 experts
        dict(name="ffn-1", op="ffn", T=1, H=7168, I=2048, E=256, K=8, skew=0.0),
        # a skewed decode batch
        dict(name="ffn-128-zipf", op="ffn", T=128, H=7168, I=2048, E=256, K=8, skew=1.2),
        # a Mixtral-shaped prefill batch: few large experts
        dict(name="ffn-4096-mixtral", op="ffn", T=4096, H=4096, I=14336, E=8, K=2, skew=0.1),
        # a DeepSeek-V3-shaped prefill batch: many ragged experts
        dict(name="ffn-8192-dsv3", op="ffn", T=8192, H=7168, I=2048, E=256, K=8, skew=0.7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "gemm", "ffn"))
    if op == "norm":
        quant = rng.choice(("none", "fp8", "mx", "int8"))
        rows = _log(rng, 1, 8192)
        cols = 128 * rng.randint(1, 64) if quant != "none" else rng.randint(64, 8192)
        return dict(op=op, rows=rows, cols=cols, x=rng.choice(("bf16", "f32")), res=rng.choice(("bf16", "f32", "none")),
                    y=rng.choice(("bf16", "f32")), quant=quant, pad=rng.choice((0, 0, 2, 64)))
    if op == "gemm":
        rows, E = _log(rng, 1, 8192), rng.choice((1, 1, rng.randint(2, 96)))
        return dict(op=op, rows=rows, E=E, N=rng.randint(64, 7168), K=16 * rng.randint(4, 448), out=rng.choice(("bf16", "f32")),
                    skew=round(rng.uniform(0.0, 1.3), 2))
    E = rng.randint(2, 64)
    return dict(op=op, T=_log(rng, 1, 4096), H=128 * rng.randint(1, 40), I=128 * rng.randint(1, 24), E=E, K=rng.randint(1, min(E, 8)),
                skew=round(rng.uniform(0.0, 1.3), 2))


def group_counts(rows, E, skew, most):
    """Rows of each expert: shares (e + 1)^-skew of `rows`, at most `most` each; they add up to `rows`."""
    w = [(e + 1.0) ** -skew for e in range(E)]
    left, total, got = rows, sum(w), []
    for e in range(E):
        n = min(most, left, int(round(rows * w[e] / total)))
        got.append(n)
        left -= n
    e = 0
    while left:  # what the caps and roundings left over, one row at a time from the front
        if got[e] < most:
            got[e] += 1
            left -= 1
        e = (e + 1) % E
    return got


def work(case):
    size = {"bf16": 2, "f32": 4, "none": 0}
    if case["op"] == "norm":
        n, c = case["rows"] * case["cols"], case["cols"]
        per = size[case["x"]] + size[case["y"]] + 2 * size[case["res"]]
        q = {"none": 0, "fp8": n + n // 128 * 4, "mx": n + n // 32, "int8": n + case["rows"] * 4}[case["quant"]]
        return {"bytes": n * per + q + c * 2, "flops": 6 * n}
    if case["op"] == "gemm":
        rows, N, K = case["rows"], case["N"], case["K"]
        active = sum(c > 0 for c in group_counts(rows, case["E"], case["skew"], rows))
        return {"bytes": rows * (K + 4) + active * N * (K + 4) + rows * N * (4 if case["out"] == "f32" else 2),
                "flops": 2 * rows * N * K}
    T, H, I, P = case["T"], case["H"], case["I"], case["T"] * case["K"]
    active = sum(c > 0 for c in group_counts(P, case["E"], case["skew"], T))
    return {"bytes": T * H * 2 + active * (3 * H * I + (2 * I + H) * 4) + P * H * 2, "flops": 6 * P * H * I}


# ----------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _weights(E, N, K, g):
    """int8 codes [E, N, K] of normal weights (a channel's largest near 127) and the channels' scales [E, N]."""
    w = torch.empty((E, N, K), dtype=torch.int8, device=DEV)
    for e in range(E):
        w[e] = torch.randn((N, K), generator=g, device=DEV).mul_(30.0).round_().clamp_(-127, 127).to(torch.int8)
    scale = torch.randn((E, N), generator=g, device=DEV).mul_(0.2).exp_() / (30.0 * K ** 0.5)
    return w, scale


def _offsets(counts):
    o = [0]
    for c in counts:
        o.append(o[-1] + c)
    return o


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "norm":
        R, C, pad = case["rows"], case["cols"], case["pad"]

        def rows(t, spread):
            # activations of a residual stream: some channels are much larger than the others
            v = torch.randn((R, C + pad), generator=g, device=DEV) * spread
            v[:, : C // 64] *= 8.0
            return v.to(t)[:, :C]

        s["x"] = rows(TYPES[case["x"]], 1.0)
        s["r"] = rows(TYPES[case["res"]], 2.0) if case["res"] != "none" else None
        s["g"] = (1.0 + 0.2 * torch.randn(C, generator=g, device=DEV)).to(torch.bfloat16)
        s["y"] = torch.empty((R, C), dtype=TYPES[case["y"]], device=DEV)
        s["r_out"] = torch.empty((R, C), dtype=s["r"].dtype, device=DEV) if s["r"] is not None else None
        q = case["quant"]
        s["codes"] = s["scales"] = None
        if q != "none":
            s["codes"] = torch.empty((R, C), dtype=torch.int8 if q == "int8" else torch.uint8, device=DEV)
            shape, t = {"fp8": ((R, C // 128), torch.float32), "mx": ((C // 128, R, 4), torch.uint8), "int8": ((R,), torch.float32)}[q]
            s["scales"] = torch.empty(shape, dtype=t, device=DEV)
        return s
    if case["op"] == "gemm":
        rows, N, K = case["rows"], case["N"], case["K"]
        counts = group_counts(rows, case["E"], case["skew"], rows)
        at = torch.randperm(case["E"], generator=g, device=DEV).tolist()
        counts = [counts[e] for e in at]
        a = torch.randn((rows, K), generator=g, device=DEV)
        scale = a.abs().amax(1) / 127.0
        s["x"] = (a / scale[:, None]).round().to(torch.int8)
        s["x_scale"] = scale
        s["w"], s["w_scale"] = _weights(case["E"], N, K, g)
        s["counts"] = counts
        s["offsets"] = torch.tensor(_offsets(counts), dtype=torch.int32, device=DEV)
        s["y"] = torch.empty((rows, N), dtype=TYPES[case["out"]], device=DEV)
        if own:  # the workspace a caller keeps beside its buffers
            from mixture_experts_layer_07_amd import binding as B
            s["ws"] = torch.empty(B.moe_gemm_int8_workspace_size(), dtype=torch.uint8, device=DEV)
        return s
    T, H, I, E, K = case["T"], case["H"], case["I"], case["E"], case["K"]
    P = T * K
    counts = group_counts(P, E, case["skew"], T)
    at = torch.randperm(E, generator=g, device=DEV).tolist()
    counts = [counts[e] for e in at]
    # row i of the grouped order is pair (token perm[i mod T], choice i / T): no token twice at one expert
    perm = torch.randperm(T, generator=g, device=DEV)
    i = torch.arange(P, device=DEV)
    s["sorted_pair"] = (perm[i % T] * K + i // T).to(torch.int32)
    s["counts"] = counts
    s["offsets"] = torch.tensor(_offsets(counts), dtype=torch.int32, device=DEV)
    s["x"] = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    s["w13"], s["w13_scale"] = _weights(E, 2 * I, H, g)
    s["w2"], s["w2_scale"] = _weights(E, H, I, g)
    s["xq"] = torch.empty((T, H), dtype=torch.int8, device=DEV)
    s["xq_scale"] = torch.empty(T, dtype=torch.float32, device=DEV)
    s["y"] = torch.empty((P, H), dtype=torch.bfloat16, device=DEV)
    if own:  # the layer's config and workspace, which a caller keeps beside its buffers
        from mixture_experts_layer_07_amd import binding as B
        from mixture_experts_layer_07_amd.configs import LayerConfig
        s["cfg"] = B.make_config(LayerConfig("int8", T=T, H=H, I=I, E=E, K=K, score="softmax", renorm=True, route_scale=1.0, n_group=1,
                                             topk_group=1, group_rule="max", bias=None, dtype="int8", I_shared=0, seed=0))
        s["ws"] = torch.empty(B.moe_workspace_size(s["cfg"]), dtype=torch.uint8, device=DEV)
    return s


# ----------------------------------------------------------------------------------- plain forms
def _plain_norm(s):
    v = s["x"].float()
    out = {}
    if s["r"] is not None:
        v = v + s["r"].float()
        out["residual"] = v.to(s["r"].dtype)
    n = v * s["g"].float() * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
    out["y"] = n.to(s["y"].dtype)
    R, C = n.shape
    if s["quant"] == "fp8":
        b = n.view(R, C // 128, 128)
        scale = b.abs().amax(2) / 448.0
        out["codes"] = (b / scale.clamp(min=1e-38)[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(R, C)
        out["scales"] = scale
    elif s["quant"] == "mx":
        b = n.view(R, C // 32, 32)
        e = torch.frexp(b.abs().amax(2))[1] - 1  # floor(log2 absmax)
        code = (e - 8 + 127).clamp(0, 254)
        out["codes"] = torch.ldexp(b, (127 - code)[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(R, C)
        out["scales"] = code.to(torch.uint8).view(R, C // 128, 4).transpose(0, 1).contiguous().view(torch.float8_e8m0fnu)
    elif s["quant"] == "int8":
        scale = n.abs().amax(1) / 127.0
        out["codes"] = (n / scale.clamp(min=1e-38)[:, None]).round().clamp(-127, 127).to(torch.bfloat16)
        out["scales"] = scale
    return out


def _plain_product(a, a_scale, w, w_scale):
    """(a . w^T) with both scales, in fp32: a [M, K], w [N, K]."""
    return (a.float() @ w.float().t()) * a_scale[:, None] * w_scale[None, :]


def _plain_gemm(s):
    # the groups are ragged, so one product per non-empty expert is the shortest plain form
    y = torch.empty_like(s["y"])
    lo = 0
    for e, c in enumerate(s["counts"]):
        if c:
            y[lo:lo + c] = _plain_product(s["x"][lo:lo + c], s["x_scale"][lo:lo + c], s["w"][e], s["w_scale"][e])
        lo += c
    return y


def _plain_int8(v):
    scale = v.abs().amax(1) / 127.0
    return (v / scale.clamp(min=1e-38)[:, None]).round().clamp(-127, 127), scale


def _plain_ffn(s):
    q, qs = _plain_int8(s["x"].float())
    tok = s["sorted_pair"].long() // s["K"]
    I = s["I"]
    y = torch.empty_like(s["y"])
    lo = 0
    for e, c in enumerate(s["counts"]):  # ragged groups: one expert after the other
        if c:
            t = tok[lo:lo + c]
            z = _plain_product(q[t], qs[t], s["w13"][e], s["w13_scale"][e])
            h = z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:]
            hq, hs = _plain_int8(h)
            y[lo:lo + c] = _plain_product(hq, hs, s["w2"][e], s["w2_scale"][e])
        lo += c
    return y


# ----------------------------------------------------------------------------------- a pass
def run(state):
    s = state
    if not own:
        if s["op"] == "norm":
            return _plain_norm(s)
        return _plain_gemm(s) if s["op"] == "gemm" else _plain_ffn(s)
    from mixture_experts_layer_07_amd import binding as B
    if s["op"] == "norm":
        q = s["quant"]
        B.moe_rmsnorm(s["x"], s["g"], EPS, y=s["y"], residual=s["r"], residual_out=s["r_out"], quant=None if q == "none" else q,
                      codes=s["codes"], scales=s["scales"])
        out = {"y": s["y"]}
        if s["r"] is not None:
            out["residual"] = s["r_out"]
        if q != "none":  # the values that the codes stand for, in units of their scales
            out["codes"] = s["codes"].to(torch.bfloat16) if q == "int8" else s["codes"].view(torch.float8_e4m3fn)
            out["scales"] = s["scales"].view(torch.float8_e8m0fnu) if q == "mx" else s["scales"]
        return out
    if s["op"] == "gemm":
        B.moe_gemm_int8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["y"], s["ws"], offsets=s["offsets"])
        return s["y"]
    B.moe_quantize_int8(s["T"], s["H"], s["x"], s["xq"], s["xq_scale"])
    B.moe_expert_ffn_gather(s["cfg"], s["E"], s["T"] * s["K"], s["I"], s["offsets"], s["sorted_pair"], s["xq"], s["xq_scale"], s["w13"],
                            s["w13_scale"], s["w2"], s["w2_scale"], s["y"], s["ws"])
    return s["y"]


# ----------------------------------------------------------------------------------- 64 bits
def _grid_e4m3(v):
    """v on the e4m3 grid: 3 mantissa bits, exponents from -6, subnormals below, at most 448."""
    v = v.clamp(-448.0, 448.0)
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.pow(2.0, e - 3.0)
    return torch.round(v / step) * step


def _exact_int8(v):
    scale = v.abs().max(dim=1).values / 127.0
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    return torch.round(v / safe[:, None]), scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        v = s["x"].double()
        out = {}
        if s["r"] is not None:
            v = v + s["r"].double()
            out["residual"] = v
        n = v / torch.sqrt((v * v).mean(dim=1) + EPS)[:, None] * s["g"].double()
        out["y"] = n
        R, C = n.shape
        if case["quant"] == "fp8":
            b = n.reshape(R, -1, 128)
            scale = b.abs().max(dim=2).values / 448.0
            out["codes"] = _grid_e4m3(b / scale[:, :, None]).reshape(R, C)
            out["scales"] = scale
        elif case["quant"] == "mx":
            b = n.reshape(R, -1, 32)
            scale = torch.pow(2.0, torch.floor(torch.log2(b.abs().max(dim=2).values)) - 8.0)
            out["codes"] = _grid_e4m3(b / scale[:, :, None]).reshape(R, C)
            out["scales"] = scale.reshape(R, C // 128, 4).permute(1, 0, 2).contiguous()
        elif case["quant"] == "int8":
            out["codes"], out["scales"] = _exact_int8(n)
        return out
    lo, parts = 0, []
    if case["op"] == "gemm":
        for e, c in enumerate(s["counts"]):
            z = torch.mm(s["x"][lo:lo + c].double(), s["w"][e].double().t().contiguous())
            parts.append(s["x_scale"][lo:lo + c].double()[:, None] * z * s["w_scale"][e].double())
            lo += c
        return torch.cat(parts)
    q, scale = _exact_int8(s["x"].double())
    v, I = q * scale[:, None], case["I"]
    tok = torch.div(s["sorted_pair"].long(), case["K"], rounding_mode="floor")
    for e, c in enumerate(s["counts"]):
        if not c:
            continue
        up = torch.mm(v[tok[lo:lo + c]], (s["w13"][e].double() * s["w13_scale"][e].double()[:, None]).t().contiguous())
        h = up[:, I:] * up[:, :I] / (1.0 + torch.exp(-up[:, :I]))
        hq, hs = _exact_int8(h)
        parts.append(torch.mm(hq * hs[:, None], (s["w2"][e].double() * s["w2_scale"][e].double()[:, None]).t().contiguous()))
        lo += c
    return torch.cat(parts)
