"""Cases, plain forms and exact values of the operators around the MoE layer.

Three families, each through the package's public functions when `own` is true:

* products grouped by expert over ragged row groups (`grouped_matmul`, forward and
  transposed, and `grouped_matmul_wgrad`, the weight gradient of each expert);
* the dense layer beside the experts (`linear` with bias, activation and residual in its
  epilogue, and `linear_backward`);
* the orthogonalised update of a batch of weight gradients (`orthogonalize`, five
  Newton-Schulz steps of an odd quintic polynomial).

With `own` false, `run` computes the same values from elementary torch operations in
32 bits, rounded once at the end.
"""
import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decode step of the fine-grained layer: 32 tokens to 8 of 256 experts, gate projection
        dict(name="grouped decode", op="grouped", transpose=False, rows=256, E=256, active=163, K=7168, N=2048,
             skew=0.0, dtype="bf16"),
        # the smallest layer the repository configures, one odd row more than its 64 x 2 pairs, one idle expert
        dict(name="grouped tiny", op="grouped", transpose=False, rows=129, E=8, active=7, K=128, N=256, skew=0.0,
             dtype="fp16"),
        # prefill of 16384 tokens to 8 of 128 small experts under a skewed routing, gate projection
        dict(name="grouped skewed prefill", op="grouped", transpose=False, rows=131072, E=128, active=120, K=2048,
             N=768, skew=1.2, dtype="bf16"),
        # input gradient of the same product on eight wide experts (4096 tokens, two experts each)
        dict(name="grouped input gradient", op="grouped", transpose=True, rows=8192, E=8, active=8, K=14336, N=4096,
             skew=0.3, dtype="bf16"),
        # weight gradients of 128 small experts, a few idle, over a micro-batch of 4096 tokens to 8 experts each
        dict(name="grouped weight gradient", op="wgrad", rows=32768, E=128, active=120, K=2048, N=768, skew=1.0,
             dtype="bf16"),
        # weight gradients of the small layer, odd group sizes
        dict(name="weight gradient tiny", op="wgrad", rows=129, E=8, active=7, K=128, N=256, skew=0.5, dtype="fp16"),
        # one token through a dense layer's first projection
        dict(name="linear one token", op="linear", T=1, K=4096, N=14336, act="silu", bias=True, residual=False,
             save=False, dtype="bf16"),
        # a ragged batch of decode tokens through the down projection onto the residual stream
        dict(name="linear few tokens", op="linear", T=37, K=14336, N=4096, act=None, bias=False, residual=True,
             save=False, dtype="bf16"),
        # training forward of a dense layer, pre-activations kept for the backward
        dict(name="linear training", op="linear", T=4096, K=4096, N=14336, act="gelu", bias=True, residual=False,
             save=True, dtype="bf16"),
        # its backward at an odd token count
        dict(name="linear backward", op="linear_backward", T=4093, K=2048, N=7168, act="gelu", bias=True,
             dtype="bf16"),
        # update of one small odd-sized gradient, where latency counts
        dict(name="orthogonalize small", op="orthogonalize", B=1, m=129, n=250, dtype="fp32"),
        # update of the gate projections of 64 of the small experts
        dict(name="orthogonalize experts", op="orthogonalize", B=64, m=2048, n=768, dtype="bf16"),
    ]


#: A drawn case costs no more than these (flops as work() counts them, weight elements).
MOST_FLOPS, MOST_WEIGHTS = 9e11, 1 << 30


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["grouped", "grouped", "wgrad", "linear", "linear", "linear_backward", "orthogonalize",
                         "orthogonalize"])
        if op in ("grouped", "wgrad"):
            E, rows = _log(rng, 1, 256), _log(rng, 1, 65536)
            case = dict(op=op, rows=rows, E=E, active=rng.randint(1, min(E, rows)), K=8 * _log(rng, 8, 1024),
                        N=8 * _log(rng, 8, 1024), skew=round(rng.uniform(0.0, 1.5), 2),
                        dtype=rng.choice(["bf16", "bf16", "fp16"]))
            if op == "grouped":
                case["transpose"] = rng.random() < 0.5
            weights = E * case["K"] * case["N"]
        elif op == "orthogonalize":
            case = dict(op=op, B=_log(rng, 1, 64), m=_log(rng, 16, 4096), n=_log(rng, 16, 4096),
                        dtype=rng.choice(["bf16", "fp32"]))
            weights = case["B"] * case["m"] * case["n"]
        else:
            case = dict(op=op, T=_log(rng, 1, 16384), K=8 * _log(rng, 8, 1792), N=8 * _log(rng, 8, 1792),
                        act=rng.choice([None, "relu", "gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.5,
                        dtype=rng.choice(["bf16", "bf16", "fp16"]))
            if op == "linear":
                case["residual"], case["save"] = rng.random() < 0.5, rng.random() < 0.5
            weights = case["K"] * case["N"]
        if weights <= MOST_WEIGHTS and work(case)["flops"] <= MOST_FLOPS:
            return case


def _counts(case, seed):
    """Rows of each expert: `active` of the E experts get at least one, the others none; shares follow 1 / rank^skew."""
    g = torch.Generator().manual_seed(seed * 7 + 1)
    E, active, rows = case["E"], case["active"], case["rows"]
    chosen = torch.randperm(E, generator=g)[:active]
    share = (1.0 + torch.arange(active, dtype=torch.float64)) ** -case["skew"]
    counts = torch.zeros(E, dtype=torch.int64)
    counts[chosen] = 1
    if rows > active:
        picks = torch.multinomial(share / share.sum(), rows - active, replacement=True, generator=g)
        counts[chosen] += torch.bincount(picks, minlength=active)
    return counts


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        # one leading index at a time, so that a large set of weights needs no 32-bit copy of itself
        out = torch.empty(shape, dtype=dtype, device="cuda")
        for part in (out if len(shape) > 2 else [out]):
            part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(std))
        return out

    s = dict(case)
    op = case["op"]
    if op in ("grouped", "wgrad"):
        counts = _counts(case, seed)
        s["counts"] = counts.tolist()
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).cuda()
        s["x"] = normal(case["rows"], case["K"])
        if op == "grouped":
            shape = (case["N"], case["K"]) if case["transpose"] else (case["K"], case["N"])
            s["W"] = normal(case["E"], *shape, std=case["K"] ** -0.5)
        else:
            s["dy"] = normal(case["rows"], case["N"], std=0.05)
    elif op in ("linear", "linear_backward"):
        T, K, N = case["T"], case["K"], case["N"]
        s["x"], s["W"] = normal(T, K), normal(K, N, std=K ** -0.5)
        s["b"] = normal(N, std=0.1) if case["bias"] else None
        if op == "linear":
            s["r"] = normal(T, N) if case["residual"] else None
        else:
            s["dy"] = normal(T, N, std=0.05)
            s["z"] = normal(T, N) if case["act"] is not None else None
    else:
        # a gradient: a few strong directions over a noisy floor
        B, m, n = case["B"], case["m"], case["n"]
        r = max(1, min(m, n) // 16)
        strong = torch.arange(1, r + 1, device="cuda", dtype=torch.float32) ** -1.0
        G = torch.empty((B, m, n), dtype=dtype, device="cuda")
        for part in G:
            u, v = (torch.randn(k, r, generator=g, device="cuda") for k in (m, n))
            part.copy_((u * strong) @ v.T * 1e-3 + torch.randn(m, n, generator=g, device="cuda") * 3e-4)
        s["G"] = G
    return s


# ---------------------------------------------------------------- plain forms


def _act(z, act):
    if act is None:
        return z
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _plain_grouped(s):
    # one product for each expert that has rows; the group sizes are the program's own
    parts, at = [], 0
    for e, c in enumerate(s["counts"]):
        if c:
            W = s["W"][e].float()
            parts.append(s["x"][at:at + c].float() @ (W.T if s["transpose"] else W))
        at += c
    return torch.cat(parts).to(s["x"].dtype)


def _plain_wgrad(s):
    dW, at = torch.zeros((s["E"], s["K"], s["N"]), dtype=s["x"].dtype, device="cuda"), 0
    for e, c in enumerate(s["counts"]):
        if c:
            dW[e] = (s["x"][at:at + c].float().T @ s["dy"][at:at + c].float()).to(dW.dtype)
        at += c
    return dW


def _plain_linear(s):
    z = s["x"].float() @ s["W"].float()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    y = y.to(s["x"].dtype)
    return (y, z.to(y.dtype)) if s["save"] else y


def _plain_linear_backward(s):
    dz = s["dy"].float()
    if s["act"] is not None:
        dz = dz * _act_slope(s["z"].float(), s["act"])
    t = s["x"].dtype
    out = dict(dx=(dz @ s["W"].float().T).to(t), dW=(s["x"].float().T @ dz).to(t))
    if s["bias"]:
        out["dbias"] = dz.sum(0).to(t)
    return out


def _plain_orthogonalize(s):
    a, b, c = COEFFS
    X = s["G"].float()
    tall = s["m"] > s["n"]
    if tall:
        X = X.mT
    X = X / ((X * X).sum((-2, -1), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X.mT if tall else X).to(torch.bfloat16)


def run(s):
    op = s["op"]
    if not own:
        return {"grouped": _plain_grouped, "wgrad": _plain_wgrad, "linear": _plain_linear,
                "linear_backward": _plain_linear_backward, "orthogonalize": _plain_orthogonalize}[op](s)
    import moe_megakernel_b200 as mk
    if op == "grouped":
        return mk.grouped_matmul(s["x"], s["W"], s["offsets"], transpose=s["transpose"])
    if op == "wgrad":
        return mk.grouped_matmul_wgrad(s["x"], s["dy"], s["offsets"])
    if op == "linear":
        return mk.linear(s["x"], s["W"], bias=s["b"], activation=s["act"], residual=s["r"], save_preact=s["save"])
    if op == "linear_backward":
        g = mk.linear_backward(s["dy"], s["x"], s["W"], preact=s["z"], activation=s["act"], bias_grad=s["bias"])
        return {k: v for k, v in g.items() if v is not None}
    return mk.orthogonalize(s["G"], steps=STEPS, coeffs=COEFFS, eps=EPS)


def work(case):
    op = case["op"]
    if op in ("grouped", "wgrad"):
        rows, K, N = case["rows"], case["K"], case["N"]
        held = case["active"] if op == "grouped" else case["E"]   # weights read, or gradients written
        return {"bytes": 2.0 * (rows * (K + N) + held * K * N) + 4.0 * (case["E"] + 1), "flops": 2.0 * rows * K * N}
    if op == "orthogonalize":
        p, q = sorted((case["m"], case["n"]))
        size = 4 if case["dtype"] == "fp32" else 2
        # the two symmetric products need half of their entries
        return {"bytes": float(case["B"] * p * q * (size + 2)),
                "flops": float(case["B"] * STEPS * (p * p * q + p ** 3 + 2 * p * p * q))}
    T, K, N = case["T"], case["K"], case["N"]
    if op == "linear":
        rows = T * (K + N + (N if case["residual"] else 0) + (N if case["save"] else 0))
        return {"bytes": 2.0 * (rows + K * N + (N if case["bias"] else 0)), "flops": 2.0 * T * K * N}
    # dy, x, W and the pre-activations in, dx, dW and the bias gradient out
    rows = T * (N + K + K + (N if case["act"] is not None else 0))
    return {"bytes": 2.0 * (rows + 2 * K * N + (N if case["bias"] else 0)), "flops": 4.0 * T * K * N}


# ---------------------------------------------------------------- exact values in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op, f = case["op"], torch.float64
    if op in ("grouped", "wgrad"):
        ends = s["offsets"].tolist()
        spans = [(e, ends[e], ends[e + 1]) for e in range(case["E"])]
        if op == "grouped":
            y = torch.empty((case["rows"], case["N"]), dtype=f, device="cuda")
            for e, lo, hi in spans:
                y[lo:hi] = torch.einsum("rk,nk->rn" if case["transpose"] else "rk,kn->rn", s["x"][lo:hi].to(f),
                                        s["W"][e].to(f))
            return y
        return torch.stack([torch.einsum("rk,rn->kn", s["x"][lo:hi].to(f), s["dy"][lo:hi].to(f))
                            for _, lo, hi in spans])
    if op == "orthogonalize":
        a, b, c = COEFFS
        out = torch.empty((case["B"], case["m"], case["n"]), dtype=f, device="cuda")
        for i in range(case["B"]):
            X = s["G"][i].to(f)
            X = X / (torch.linalg.vector_norm(X) + EPS)
            eye = torch.eye(case["n"], dtype=f, device="cuda")
            if case["m"] < case["n"]:
                X, eye = X.T, eye[:case["m"], :case["m"]]
            for _ in range(STEPS):   # X p(X^T X) with p(t) = a + t (b + c t), the short side inside
                S = X.T @ X
                X = X @ (a * eye + S @ (b * eye + c * S))
            out[i] = X.T if case["m"] < case["n"] else X
        return out
    x, W, act = s["x"].to(f), s["W"].to(f), case["act"]
    z = (x @ W if op == "linear" else s["z"].to(f) if act is not None else None)
    if op == "linear" and case["bias"]:
        z = z + s["b"].to(f)
    if act is None:
        y, slope = z, 1.0
    elif act == "relu":
        y, slope = torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).to(f)
    elif act == "silu":
        q = torch.sigmoid(z)
        y, slope = z * q, q + z * q * torch.sigmoid(-z)
    elif act == "gelu":
        phi = 0.5 * torch.erfc(-z / math.sqrt(2))
        y, slope = z * phi, phi + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    else:
        k = 2 * math.sqrt(2 / math.pi)
        q = torch.sigmoid(k * (z + 0.044715 * z ** 3))   # (1 + tanh(u)) / 2 = sigmoid(2 u)
        y, slope = z * q, q + z * q * (1 - q) * k * (1 + 0.134145 * z.square())
    if op == "linear":
        if case["residual"]:
            y = y + s["r"].to(f)
        return (y, z) if case["save"] else y
    dz = s["dy"].to(f) * slope
    out = dict(dx=dz @ W.T, dW=x.T @ dz)
    if case["bias"]:
        out["dbias"] = dz.sum(0)
    return out
