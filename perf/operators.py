"""The linear layer's language-model operators, as they are timed and compared.

Low-rank adapters of many requests beside a shared projection (forward and
backward), and activation checkpoints in 8 bits (stored, read back, and used for
the gradient of an activation and of a weight).

Adapters.  Row i of X uses adapter a = ids[i], or none where ids[i] < 0:

    H[i] = X[i] @ A[a],   Y[i] = X[i] @ W + bias + scale[a] * H[i] @ B[a]

with the first ranks[a] of the R columns of A[a] (rows of B[a]); the rest of the
stack holds whatever was there before and is not used.  Backward, W being frozen:

    G[i] = scale[a] * dY[i] @ B[a].T,   dX = dY @ W.T + G[i] @ A[a].T
    dA[a] = sum_i X[i].T G[i],          dB[a] = sum_i scale[a] * H[i].T dY[i]

Checkpoints.  Each block of 32 columns of a row keeps an exponent e, the least
integer >= -126 with max|x| <= 127 * 2^e, and q = rint(x / 2^e) in int8; it stands
for q * 2^e.
"""
import math

import torch

own = False

BLOCK = 32
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one token of one request through a small projection: pure latency
        dict(name="lora_decode_1_f32", op="lora", type="f32", M=1, K=1024, N=1024, L=4, R=8,
             rows="decode", ranks="full", bias=False, save=False),
        # a decode step of 64 requests, each with its own choice among 32 adapters of unequal rank
        dict(name="lora_decode_64_bf16", op="lora", type="bf16", M=64, K=4096, N=4096, L=32, R=16,
             rows="decode", ranks="mixed", bias=False, save=False),
        # a long prefill of several requests, rank 64
        dict(name="lora_prefill_8192_bf16", op="lora", type="bf16", M=8192, K=4096, N=4096, L=8, R=64,
             rows="requests", ranks="full", bias=True, save=False),
        # a training forward at sizes that fit no tile, with the rank-side product kept for the backward pass
        dict(name="lora_train_odd_f32", op="lora", type="f32", M=4097, K=1023, N=3001, L=5, R=20,
             rows="requests", ranks="mixed", bias=True, save=True),
        # the backward pass of a projection fine-tuned for four tenants at once
        dict(name="lora_backward_bf16", op="lora_backward", type="bf16", M=4096, K=4096, N=4096, L=4,
             R=32, rows="requests", ranks="full", x8=False),
        # the same at odd sizes, the layer's input kept in 8 bits
        dict(name="lora_backward_odd_x8_f32", op="lora_backward", type="f32", M=3001, K=1024, N=1023,
             L=3, R=20, rows="requests", ranks="mixed", x8=True),
        # a handful of rows checkpointed and read back: latency
        dict(name="act8_store_16_bf16", op="act8_store", type="bf16", M=16, K=1024, act="none"),
        # the hidden layer of a wide MLP: activation and checkpoint of its input in one pass
        dict(name="act8_store_gelu_bf16", op="act8_store", type="bf16", M=8192, K=16384, act="gelu"),
        # the activation's gradient from the checkpoint: odd sizes in float32, then the wide MLP
        dict(name="act8_grad_odd_f32", op="act8_grad", type="f32", M=4097, K=3001, act="gelu"),
        dict(name="act8_grad_gelu_bf16", op="act8_grad", type="bf16", M=8192, K=16384, act="gelu"),
        # the weight gradient from the 8-bit input, square and odd
        dict(name="act8_wgrad_bf16", op="act8_wgrad", type="bf16", M=8192, K=4096, N=4096),
        dict(name="act8_wgrad_odd_f32", op="act8_wgrad", type="f32", M=4097, K=1023, N=3001),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A row length: as it falls, or rounded to the multiples that models have."""
    n = _log_int(rng, low, high)
    return n if rng.random() < 0.4 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["lora", "lora", "lora", "lora_backward", "act8_store", "act8_grad", "act8_wgrad"])
    case = dict(op=op, type=rng.choice(["f32", "bf16"]))
    if op in ("act8_store", "act8_grad"):
        case["K"] = _width(rng, 64, 16384)
        case["M"] = _log_int(rng, 1, 8192)
        case["act"] = rng.choice(["gelu", "relu"] if op == "act8_grad" else ["none", "gelu", "relu"])
        return case
    case["K"], case["N"] = _width(rng, 64, 8192), _width(rng, 64, 8192)
    most = min(8192, 8192 * 4096 * 4096 // (case["K"] * case["N"]))
    case["M"] = _log_int(rng, 1 if op == "lora" else 64, most)
    if op == "act8_wgrad":
        return case
    case["R"] = _log_int(rng, 4, 128)
    case["L"] = _log_int(rng, 1, max(1, min(64, 512 // case["R"])))
    mixed = case["M"] <= 128 or (case["M"] <= 512 and rng.random() < 0.5)
    case["rows"] = "decode" if mixed and op == "lora" else "requests"
    case["ranks"] = rng.choice(["full", "mixed"])
    if op == "lora":
        case["bias"], case["save"] = rng.random() < 0.5, rng.random() < 0.5
    else:
        case["x8"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs
def _power_of_two(e):
    """2^e in float32 for e >= -126, exactly: the exponent's bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantised(x):
    """The checkpoint of a float32 matrix, by its definition: (q int8, e int8, the values it stands for)."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    x = torch.nn.functional.pad(x, (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    mant, exp = torch.frexp(x.abs().amax(dim=2))              # max|x| = mant * 2^exp, mant in [0.5, 1)
    e = torch.where(mant <= 127.0 / 128.0, exp - 7, exp - 6)  # 127 * 2^(exp-7) is mant = 127/128
    e = torch.where(mant == 0, torch.full_like(e, -126), e.clamp(min=-126))
    step = _power_of_two(e).unsqueeze(2)
    q = torch.round(x / step)
    values = (q * step).view(rows, blocks * BLOCK)[:, :cols]
    q = q.view(rows, blocks * BLOCK)[:, :cols]
    return q.to(torch.int8).contiguous(), e.to(torch.int8).contiguous(), values.contiguous()


def _activations(rows, cols, g):
    """Normal values with a few columns that are much larger, as hidden states have."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    outlier = torch.rand(cols, generator=g, device="cuda") < 0.004
    return x * torch.where(outlier, 20.0, 1.0)


def _row_ids(case, g):
    """ids of the rows: a choice for each row, or runs of rows of one request; some without an adapter."""
    M, L = case["M"], case["L"]
    if case["rows"] == "decode":
        ids = torch.randint(-1, L, (M,), generator=g, device="cuda")
    else:
        requests = min(M, 2 * L)
        cuts = torch.randint(0, M, (requests - 1,), generator=g, device="cuda")
        of_row = torch.bucketize(torch.arange(M, device="cuda"), cuts.sort().values, right=True)
        ids = torch.randint(-1, L, (requests,), generator=g, device="cuda")[of_row]
    return ids.to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, t, M, K = case["op"], TYPES[case["type"]], case["M"], case["K"]
    s = dict(case=case, op=op, type=t)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(t)

    if op == "act8_store":
        s["Z"] = _activations(M, K, g).to(t)
        s["q"] = torch.empty(M, K, dtype=torch.int8, device="cuda")
        s["e"] = torch.empty(M, -(-K // BLOCK), dtype=torch.int8, device="cuda")
        s["back"] = torch.empty(M, K, dtype=t, device="cuda")
        s["Y"] = torch.empty(M, K, dtype=t, device="cuda") if case["act"] != "none" else None
    elif op == "act8_grad":
        s["q"], s["e"], _ = _quantised(_activations(M, K, g).to(t).float())
        s["dY"] = normal(M, K)
        s["dZ"] = torch.empty(M, K, dtype=t, device="cuda")
    elif op == "act8_wgrad":
        s["q"], s["e"], _ = _quantised(_activations(M, K, g).to(t).float())
        s["dY"] = normal(M, case["N"])
        s["dW"] = torch.empty(K, case["N"], dtype=t, device="cuda")
    else:
        N, L, R = case["N"], case["L"], case["R"]
        s["ids"] = _row_ids(case, g)
        s["W"] = normal(K, N, scale=K ** -0.5)
        s["A"] = normal(L, K, R, scale=K ** -0.5)
        s["B"] = normal(L, R, N, scale=R ** -0.5)
        s["scale"] = torch.rand(L, generator=g, device="cuda") * 1.5 + 0.5
        s["ranks"] = None
        if case["ranks"] == "mixed":
            s["ranks"] = torch.randint(1, R + 1, (L,), generator=g, device="cuda", dtype=torch.int32)
        X = _activations(M, K, g).to(t)
        if op == "lora":
            s["X"] = X
            s["bias"] = normal(N) if case["bias"] else None
            s["Y"] = torch.empty(M, N, dtype=t, device="cuda")
            s["H"] = torch.empty(M, R, device="cuda") if case["save"] else None
        else:
            values = X
            if case["x8"]:
                s["q"], s["e"], values = _quantised(X.float())
            else:
                s["X"] = X
            s["H"] = _rank_side(s, values.float()).sum(1)
            s["dY"] = normal(M, N)
            s["dX"] = torch.empty(M, K, dtype=t, device="cuda")
            s["dA"] = torch.empty(L, K, R, dtype=t, device="cuda")
            s["dB"] = torch.empty(L, R, N, dtype=t, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _uses(s):
    """(M, L, R) truth values: row i uses column r of adapter l."""
    L, R = s["A"].shape[0], s["A"].shape[2]
    keep = (s["ids"].unsqueeze(1) == torch.arange(L, device="cuda")).unsqueeze(2)
    if s["ranks"] is not None:
        keep = keep & (torch.arange(R, device="cuda") < s["ranks"].unsqueeze(1))
    return keep.expand(-1, -1, R)


def _rank_side(s, X):
    """X @ A of every adapter, kept where a row uses it: (M, L, R)."""
    L, K, R = s["A"].shape
    every = (X @ s["A"].float().permute(1, 0, 2).reshape(K, L * R)).view(-1, L, R)
    return torch.where(_uses(s), every, 0.0)


def _dequantised(s):
    q, step = s["q"].float(), _power_of_two(s["e"])
    return q * step.repeat_interleave(BLOCK, dim=1)[:, :q.shape[1]]


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
            + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))


def _plain(s):
    op, t = s["op"], s["type"]
    if op == "act8_store":
        z = s["Z"].float()
        y = None if s["Y"] is None else _act(z, s["case"]["act"]).to(t)
        return {"back": _quantised(z)[2].to(t), "Y": y}
    if op == "act8_grad":
        return (s["dY"].float() * _act_slope(_dequantised(s), s["case"]["act"])).to(t)
    if op == "act8_wgrad":
        return (_dequantised(s).t() @ s["dY"].float()).to(t)
    L, K, R = s["A"].shape
    N = s["W"].shape[1]
    Bf = s["B"].float().reshape(L * R, N)
    if op == "lora":
        X = s["X"].float()
        H = _rank_side(s, X)
        Y = X @ s["W"].float() + (H * s["scale"].view(1, L, 1)).reshape(-1, L * R) @ Bf
        if s["bias"] is not None:
            Y = Y + s["bias"].float()
        return {"Y": Y.to(t), "H": H.sum(1) if s["H"] is not None else None}
    X = _dequantised(s) if s["case"]["x8"] else s["X"].float()
    dY = s["dY"].float()
    G = torch.where(_uses(s), (dY @ Bf.t()).view(-1, L, R) * s["scale"].view(1, L, 1), 0.0)
    G = G.reshape(-1, L * R)
    H = torch.where(_uses(s), s["H"].unsqueeze(1) * s["scale"].view(1, L, 1), 0.0).reshape(-1, L * R)
    dX = dY @ s["W"].float().t() + G @ s["A"].float().permute(0, 2, 1).reshape(L * R, K)
    dA = (X.t() @ G).view(K, L, R).permute(1, 0, 2)
    dB = (H.t() @ dY).view(L, R, N)
    return {"dX": dX.to(t), "dA": dA.to(t).contiguous(), "dB": dB.to(t)}


# ------------------------------------------------------------------ the framework's operators
def _own(s):
    from dense_fp32_gemm_02_gb300 import binding
    op, case = s["op"], s["case"]
    if op == "act8_store":
        binding.act8_store_into(s["Z"], s["q"], s["e"], act=case["act"], Y=s["Y"])
        return {"back": binding.act8_load_into(s["q"], s["e"], s["back"]), "Y": s["Y"]}
    if op == "act8_grad":
        return binding.act8_grad_into(s["q"], s["e"], s["dY"], s["dZ"], act=case["act"])
    if op == "act8_wgrad":
        return binding.act8_weight_grad_into(s["q"], s["e"], s["dY"], s["dW"])
    if op == "lora":
        binding.lora_into(s["X"], s["W"], s["A"], s["B"], s["ids"], s["Y"], scale=s["scale"],
                          ranks=s["ranks"], bias=s["bias"], H=s["H"])
        return {"Y": s["Y"], "H": s["H"]}
    X = (s["q"], s["e"]) if case["x8"] else s["X"]
    binding.lora_backward_into(s["dY"], X, s["W"], s["A"], s["B"], s["ids"], s["H"], dX=s["dX"],
                               dA=s["dA"], dB=s["dB"], scale=s["scale"], ranks=s["ranks"])
    return {"dX": s["dX"], "dA": s["dA"], "dB": s["dB"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, size, M, K = case["op"], SIZE[case["type"]], case["M"], case["K"]
    kept = M * K + M * -(-K // BLOCK)                       # a checkpoint's bytes
    if op == "act8_store":                                  # Z in, q and e out and in, the values out (and Y)
        outs = 1 if case["act"] == "none" else 2
        return {"bytes": M * K * size * (1 + outs) + 2 * kept, "flops": M * K * 4}
    if op == "act8_grad":
        return {"bytes": 2 * M * K * size + kept, "flops": M * K * 12}
    N = case["N"]
    if op == "act8_wgrad":
        return {"bytes": kept + (M + K) * N * size, "flops": 2 * M * K * N}
    used = min(case["L"], M)
    rank = case["R"] if case["ranks"] == "full" else (case["R"] + 1) / 2
    adapters = used * rank * (K + N) * size
    if op == "lora":
        b = (M * K + K * N + M * N) * size + adapters + 4 * M
        b += (N * size if case["bias"] else 0) + (4 * M * case["R"] if case["save"] else 0)
        return {"bytes": b, "flops": 2 * M * K * N + 2 * M * rank * (K + N)}
    b = (M * N + K * N + M * K) * size + (kept if case["x8"] else M * K * size)
    b += adapters + case["L"] * case["R"] * (K + N) * size + 4 * M * (case["R"] + 1)
    return {"bytes": b, "flops": 2 * M * K * N + 4 * M * rank * (K + N)}


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_power(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(s):
    """q * 2^e in 64 bits."""
    e = s["e"].double().repeat_interleave(BLOCK, dim=1)[:, :s["q"].shape[1]]
    return s["q"].double() * _exact_power(e)


def _exact_store(z):
    back = torch.zeros_like(z)
    for c in range(0, z.shape[1], BLOCK):
        block = z[:, c:c + BLOCK]
        top = block.abs().amax(dim=1, keepdim=True)
        e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 127.0))
        e = torch.where(top > 127.0 * _exact_power(e), e + 1, e)             # log2's own rounding
        e = torch.where(top <= 127.0 * _exact_power(e - 1), e - 1, e).clamp(min=-126)
        back[:, c:c + BLOCK] = torch.round(block / _exact_power(e)) * _exact_power(e)
    return back


def _exact_cdf(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2.0))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "act8_store":
        z = s["Z"].double()
        y = {"none": lambda: None, "relu": lambda: torch.relu(z), "gelu": lambda: z * _exact_cdf(z)}[case["act"]]()
        return {"back": _exact_store(z), "Y": y}
    if op == "act8_grad":
        z, dy = _exact_values(s), s["dY"].double()
        if case["act"] == "relu":
            return torch.where(z > 0, dy, 0.0)
        return dy * (_exact_cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    if op == "act8_wgrad":
        return torch.einsum("mk,mn->kn", _exact_values(s), s["dY"].double())
    L, K, R = s["A"].shape
    X = _exact_values(s) if case.get("x8") else s["X"].double()
    W = s["W"].double()
    if op == "lora":
        H = torch.zeros(X.shape[0], R, dtype=torch.float64, device="cuda")
        Y = X @ W
        if s["bias"] is not None:
            Y += s["bias"].double()
    else:
        dY = s["dY"].double()
        dX = dY @ W.t()
        dA, dB = torch.zeros_like(s["A"], dtype=torch.float64), torch.zeros_like(s["B"], dtype=torch.float64)
    for a in range(L):
        rows = torch.nonzero(s["ids"] == a).flatten()
        r = R if s["ranks"] is None else int(s["ranks"][a])
        f, A, B = float(s["scale"][a]), s["A"][a, :, :r].double(), s["B"][a, :r].double()
        if op == "lora":
            h = X[rows] @ A
            H[rows, :r] = h
            Y[rows] += f * (h @ B)
        else:
            g = f * (dY[rows] @ B.t())
            dX[rows] += g @ A.t()
            dA[a, :, :r] = X[rows].t() @ g
            dB[a, :r] = f * (s["H"][rows, :r].double().t() @ dY[rows])
    if op == "lora":
        return {"Y": Y, "H": H if s["H"] is not None else None}
    return {"dX": dX, "dA": dA, "dB": dB}
