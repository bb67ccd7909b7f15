"""The feed-forward side of a layer in a language model, as it is timed and compared.

The root-mean-square norm with the residual's addition (in the layer's type or in 8 bits with
a scale for each row; backward), the matrix product in 8-bit integers that reads such rows, and
the gated block (two projections, an activation and their product; backward).

Norm.  v = x + r, held in the layer's type (the residual stream), and of a row of v

    y_j = v_j * w_j / sqrt(mean(v^2) + eps)

In 8 bits a row is scale = max|y| / 127 and q_j = y_j / scale rounded to the nearest integer,
ties to even: q_j = rint(127 * v_j w_j / max|v w|).  Backward, with g = dy * w and c = mean(g v)
/ (mean(v^2) + eps), s the gradient that reaches v by its other way:

    dv_j = s_j + (g_j - c v_j) / sqrt(mean(v^2) + eps),   dw_j = sum over the rows of dy_j v_j / sqrt(...)

Product.  y_ij = scale_i * wscale_j * sum_k q_ik w_kj + bias_j, q and w int8; the rows come in
8 bits or are brought to them on the way, by the rule above.

Gated block.  g = x Wg, u = x Wu, h = act(g) * u.  Backward, dg = dh * u * act'(g) and du = dh *
act(g): dx = dg Wg^T + du Wu^T, dWg = x^T dg, dWu = x^T du.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one token of one request before an 8-bit projection: pure latency
        dict(name="norm8_decode_1_bf16", op="norm", type="bf16", M=1, K=4096, residual=True, out="q"),
        # a long batch, the stream kept, the norm in both forms (a layer that feeds 8-bit and other products)
        dict(name="norm_both_8192_bf16", op="norm", type="bf16", M=8192, K=8192, residual=True, out="both"),
        # a training step's norm, with the gradient that comes along the residual stream
        dict(name="norm_backward_bf16", op="norm_backward", type="bf16", M=8192, K=4096, stream=True),
        # the same at sizes that fit no vector, in float32
        dict(name="norm_backward_odd_f32", op="norm_backward", type="f32", M=4097, K=1023, stream=True),
        # one token through an 8-bit projection
        dict(name="linear8_decode_1_bf16", op="linear8", type="bf16", M=1, K=4096, N=4096, x="q", bias=False),
        # a decode step of 64 requests, whose rows the call brings to 8 bits itself
        dict(name="linear8_decode_64_bf16", op="linear8", type="bf16", M=64, K=4096, N=4096, x="type", bias=False),
        # a long prefill
        dict(name="linear8_prefill_8192_bf16", op="linear8", type="bf16", M=8192, K=4096, N=4096, x="q", bias=True),
        # a decode step of 8 requests through the gated block
        dict(name="gated_decode_8_bf16", op="gated", type="bf16", M=8, K=4096, N=8192, act="silu", save=False),
        # a training forward in float32 at sizes that fit no tile, what the backward pass needs kept
        dict(name="gated_train_odd_f32", op="gated", type="f32", M=1025, K=1023, N=3001, act="gelu", save=True),
        # a long training forward
        dict(name="gated_train_8192_bf16", op="gated", type="bf16", M=8192, K=4096, N=8192, act="silu", save=True),
        # its backward pass, all gradients
        dict(name="gated_backward_bf16", op="gated_backward", type="bf16", M=4096, K=4096, N=8192, act="silu"),
        # the same in float32 at odd sizes
        dict(name="gated_backward_odd_f32", op="gated_backward", type="f32", M=1025, K=1023, N=3001, act="gelu"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A row length: as it falls, or rounded to the multiples that models have."""
    n = _log_int(rng, low, high)
    return n if rng.random() < 0.4 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "linear8", "linear8", "gated", "gated", "gated_backward"])
    case = dict(op=op, type=rng.choice(["f32", "bf16"]))
    if op in ("norm", "norm_backward"):
        case["K"] = _width(rng, 64, 16384)
        case["M"] = _log_int(rng, 1, min(8192, 8192 * 4096 // case["K"]))
        if op == "norm":
            case["residual"], case["out"] = rng.random() < 0.7, rng.choice(["type", "q", "both"])
        else:
            case["stream"] = rng.random() < 0.7
        return case
    case["K"], case["N"] = _width(rng, 64, 8192), _width(rng, 64, 8192)
    most = 8192 if op == "gated" else 4096
    most = min(8192, most * 4096 * (4096 if op == "linear8" else 8192) // (case["K"] * case["N"]))
    case["M"] = _log_int(rng, 64 if op == "gated_backward" else 1, most)
    if op == "linear8":
        case["x"], case["bias"] = rng.choice(["q", "type"]), rng.random() < 0.5
        return case
    case["act"] = rng.choice(["silu", "silu", "gelu", "relu"])
    if op == "gated":
        case["save"] = case["M"] >= 64 and rng.random() < 0.6
    return case


# ------------------------------------------------------------------ inputs
def _activations(rows, cols, g):
    """Normal values with a few columns that are much larger, as hidden states have."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    outlier = torch.rand(cols, generator=g, device="cuda") < 0.004
    return x * torch.where(outlier, 20.0, 1.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, t, M, K = case["op"], TYPES[case["type"]], case["M"], case["K"]
    s = dict(case=case, op=op, type=t)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(t)

    def empty(*shape, dtype=t):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op in ("norm", "norm_backward"):
        s["w"] = (1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")).to(t)
    if op == "norm":
        s["X"] = _activations(M, K, g).to(t)
        s["R"] = _activations(M, K, g).to(t) if case["residual"] else None
        s["S"] = empty(M, K) if case["residual"] else None
        s["Y"] = empty(M, K) if case["out"] != "q" else None
        kept = case["out"] != "type"
        s["q"] = empty(M, K, dtype=torch.int8) if kept else None
        s["scale"] = empty(M, dtype=torch.float32) if kept else None
        s["back"] = empty(M, K) if kept else None
    elif op == "norm_backward":
        s["V"], s["dY"] = _activations(M, K, g).to(t), normal(M, K)
        s["dS"] = normal(M, K) if case["stream"] else None
        s["dX"], s["dw"] = empty(M, K), empty(K)
    elif op == "linear8":
        N = case["N"]
        x = _activations(M, K, g).to(t)
        if case["x"] == "q":
            top = x.float().abs().amax(dim=1)
            s["scale"] = top / 127.0
            s["q"] = torch.round(x.float() * (127.0 / top).unsqueeze(1)).to(torch.int8)
        else:
            s["X"] = x
        w = torch.randn(K, N, generator=g, device="cuda") * K ** -0.5
        s["wscale"] = w.abs().amax(dim=0) / 127.0
        s["W"] = torch.round(w / s["wscale"]).to(torch.int8)
        s["bias"] = normal(N) if case["bias"] else None
        s["Y"] = empty(M, N)
    else:
        N = case["N"]
        s["X"] = _activations(M, K, g).to(t)
        s["Wg"], s["Wu"] = normal(K, N, scale=K ** -0.5), normal(K, N, scale=K ** -0.5)
        if op == "gated":
            s["H"] = empty(M, N)
            s["G"], s["U"] = (empty(M, N), empty(M, N)) if case["save"] else (None, None)
        else:
            s["G"], s["U"], s["dH"] = normal(M, N, scale=1.5), normal(M, N, scale=1.5), normal(M, N)
            s["dX"], s["dWg"], s["dWu"] = empty(M, K), empty(K, N), empty(K, N)
    return s


# ------------------------------------------------------------------ plain forms
def _rows8(p):
    """(q, largest magnitude) of each row of p, in 64 bits: which side of a tie a value is on."""
    top = p.abs().amax(dim=1, keepdim=True)
    q = torch.round(127.0 * p / torch.where(top > 0, top, 1.0))
    return q.float(), top.squeeze(1).float()


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sigma = 1.0 / (1.0 + torch.exp(-z))
        return sigma * (1.0 + z * (1.0 - sigma))
    return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
            + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))


def _plain(s):
    op, t, case = s["op"], s["type"], s["case"]
    if op == "norm":
        v = s["X"].float()
        if s["R"] is not None:
            v = (v + s["R"].float()).to(t).float()
        w = s["w"].float()
        rstd = torch.rsqrt(v.square().mean(dim=1) + EPS)
        out = {"S": v.to(t) if s["R"] is not None else None, "Y": None, "back": None, "scale": None}
        if s["Y"] is not None:
            out["Y"] = (v * rstd.unsqueeze(1) * w).to(t)
        if s["q"] is not None:
            q, top = _rows8(v.double() * w.double())
            out["scale"] = top * rstd / 127.0
            out["back"] = (q * out["scale"].unsqueeze(1)).to(t)
        return out
    if op == "norm_backward":
        v, dy = s["V"].float(), s["dY"].float()
        rstd = torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS)
        g = dy * s["w"].float()
        dx = (g - v * ((g * v).mean(dim=1, keepdim=True) * rstd.square())) * rstd
        if s["dS"] is not None:
            dx = dx + s["dS"].float()
        return {"dX": dx.to(t), "dw": (dy * v * rstd).sum(dim=0).to(t)}
    if op == "linear8":
        if case["x"] == "q":
            q, scale = s["q"].float(), s["scale"]
        else:
            q, scale = _rows8(s["X"].double())
            scale = scale / 127.0
        y = (q @ s["W"].float()) * scale.unsqueeze(1) * s["wscale"]
        return (y if s["bias"] is None else y + s["bias"].float()).to(t)
    Wg, Wu, X = s["Wg"].float(), s["Wu"].float(), s["X"].float()
    if op == "gated":
        g, u = X @ Wg, X @ Wu
        save = s["G"] is not None
        return {"H": (_act(g, case["act"]) * u).to(t), "G": g.to(t) if save else None, "U": u.to(t) if save else None}
    g, u, dh = s["G"].float(), s["U"].float(), s["dH"].float()
    dg, du = dh * u * _act_slope(g, case["act"]), dh * _act(g, case["act"])
    return {"dX": (dg @ Wg.t() + du @ Wu.t()).to(t), "dWg": (X.t() @ dg).to(t), "dWu": (X.t() @ du).to(t)}


# ------------------------------------------------------------------ the framework's operators
def _own(s):
    from dense_fp32_gemm_02_gb300 import binding
    op, case = s["op"], s["case"]
    if op == "norm":
        binding.rmsnorm_into(s["X"], s["w"], Y=s["Y"], q=s["q"], scale=s["scale"], R=s["R"], S=s["S"], eps=EPS)
        if s["q"] is not None:
            torch.mul(s["q"], s["scale"].unsqueeze(1), out=s["back"])   # the values that the rows stand for
        return {"S": s["S"], "Y": s["Y"], "back": s["back"], "scale": s["scale"]}
    if op == "norm_backward":
        binding.rmsnorm_backward_into(s["dY"], s["V"], s["w"], s["dX"], dw=s["dw"], dS=s["dS"], eps=EPS)
        return {"dX": s["dX"], "dw": s["dw"]}
    if op == "linear8":
        X = (s["q"], s["scale"]) if case["x"] == "q" else s["X"]
        return binding.linear8_into(X, s["W"], s["wscale"], s["Y"], bias=s["bias"])
    if op == "gated":
        binding.gated_into(s["X"], s["Wg"], s["Wu"], s["H"], act=case["act"], G=s["G"], U=s["U"])
        return {"H": s["H"], "G": s["G"], "U": s["U"]}
    binding.gated_backward_into(s["dH"], s["X"], s["Wg"], s["Wu"], s["G"], s["U"], dX=s["dX"], dWg=s["dWg"],
                                dWu=s["dWu"], act=case["act"])
    return {"dX": s["dX"], "dWg": s["dWg"], "dWu": s["dWu"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, size, M, K = case["op"], SIZE[case["type"]], case["M"], case["K"]
    if op == "norm":       # x, r and w in; v, y, q and scale out, and q in again for the values
        matrices = 1 + (2 if case["residual"] else 0) + (case["out"] != "q") + (case["out"] != "type")
        kept = 0 if case["out"] == "type" else 2 * (M * K + 4 * M)
        return {"bytes": matrices * M * K * size + K * size + kept, "flops": M * K * 6}
    if op == "norm_backward":
        return {"bytes": (3 + case["stream"]) * M * K * size + 2 * K * size, "flops": M * K * 12}
    N = case["N"]
    if op == "linear8":
        x = M * K + 4 * M if case["x"] == "q" else M * K * size
        b = x + K * N + 4 * N + M * N * size + (N * size if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * M * K * N}
    if op == "gated":
        return {"bytes": (M * K + 2 * K * N + M * N * (3 if case["save"] else 1)) * size, "flops": 4 * M * K * N}
    return {"bytes": (2 * M * K + 4 * K * N + 3 * M * N) * size, "flops": 8 * M * K * N}


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_act(z, act):
    """(act, act') in 64 bits."""
    if act == "relu":
        return torch.relu(z), torch.where(z > 0, 1.0, 0.0).double()
    if act == "silu":
        sigma = torch.sigmoid(z)
        return z * sigma, sigma + z * sigma * torch.sigmoid(-z)
    cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
    return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        v = s["X"].double()
        if s["R"] is not None:
            v = (v + s["R"].double()).to(s["type"]).double()     # the stream, as it is held
        y = v * s["w"].double() / torch.sqrt((v * v).sum(1, keepdim=True) / case["K"] + EPS)
        scale = y.abs().max(dim=1).values / 127.0
        kept = s["q"] is not None
        back = torch.round(y / scale.unsqueeze(1)) * scale.unsqueeze(1) if kept else None
        return {"S": v if s["R"] is not None else None, "Y": y if s["Y"] is not None else None,
                "back": back, "scale": scale if kept else None}
    if op == "norm_backward":
        v, dy, w = s["V"].double(), s["dY"].double(), s["w"].double()
        rms = torch.sqrt((v * v).sum(1, keepdim=True) / case["K"] + EPS)
        n = v / rms
        g = dy * w
        dx = (g - n * (g * n).sum(1, keepdim=True) / case["K"]) / rms
        return {"dX": dx if s["dS"] is None else dx + s["dS"].double(), "dw": torch.einsum("mk,mk->k", dy, n)}
    if op == "linear8":
        if case["x"] == "q":
            x = s["q"].double() * s["scale"].double().unsqueeze(1)
        else:
            x = s["X"].double()
            step = x.abs().max(dim=1, keepdim=True).values / 127.0
            x = torch.round(x / step) * step
        y = x @ (s["W"].double() * s["wscale"].double())
        return y if s["bias"] is None else y + s["bias"].double()
    X, Wg, Wu = s["X"].double(), s["Wg"].double(), s["Wu"].double()
    if op == "gated":
        g, u = X @ Wg, X @ Wu
        save = s["G"] is not None
        return {"H": _exact_act(g, case["act"])[0] * u, "G": g if save else None, "U": u if save else None}
    value, slope = _exact_act(s["G"].double(), case["act"])
    dh = s["dH"].double()
    dg, du = dh * s["U"].double() * slope, dh * value
    return {"dX": torch.cat((dg, du), 1) @ torch.cat((Wg, Wu), 1).t(), "dWg": X.t() @ dg, "dWu": X.t() @ du}
