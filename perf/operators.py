"""The feed-forward operators of a transformer layer, in their plain form and through the library.

Four operators, on row-major activations [tokens, features] and weights W [K, N] stored either
way ("kn": N contiguous, "nk": K contiguous, the transposed storage of a [N, K] parameter):

  linear         Z = X W + b,  Y = act(Z) + R
  linear_grad    dZ = dY act'(Z),  dX = dZ W^T,  dW = X^T dZ,  db = sum over rows of dZ
  gated          G = X Wg + bg,  U = X Wu + bu,  H = act(G) U
  gated_grad     dG = dH U act'(G),  dU = dH act(G),  dX = dG Wg^T + dU Wu^T,
                 dWg = X^T dG,  dWu = X^T dU,  dbg and dbu their column sums

`run` takes the plain form (32-bit torch operations, rounded once at the end) where `own` is
false and the library's calls where it is true; `exact` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
MATRICES = {"linear": 1, "linear_grad": 2, "gated": 2, "gated_grad": 4}  # products of M x N x K


def case(op, name, dtype, M, N, K, store, act, bias=True, residual=False, keep=False, pad=0):
    """keep: the forward pass also writes what the backward pass reads (Z, or G and U);
    pad: extra elements between the rows of the activations."""
    c = dict(op=op, dtype=dtype, M=M, N=N, K=K, store=store, act=act, bias=bias, residual=residual, keep=keep,
             pad=pad)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token's output projection while answering: the weights are read once
        case("linear", "linear_token", "bf16", 1, 4096, 4096, "nk", "none", bias=False, residual=True),
        # the down projection of a small serving batch, with the skip connection added
        case("linear", "linear_rows16", "f16", 16, 4096, 16384, "kn", "none", residual=True),
        # the smallest fp32 product of the library's benchmark: latency
        case("linear", "linear_f32_256", "f32", 256, 256, 256, "kn", "gelu"),
        # a training step's first projection at sizes that divide nothing, kept for the backward pass
        case("linear", "linear_ragged", "bf16", 4000, 3968, 4001, "kn", "gelu", residual=True, keep=True),
        # a prompt's projection
        case("linear", "linear_4096", "bf16", 4096, 4096, 4096, "nk", "gelu_tanh", residual=True),
        # one token through the gated block while answering
        case("gated", "gated_token", "bf16", 1, 16384, 4096, "nk", "silu", bias=False),
        # a few users' tokens, sizes that divide nothing, rows with padding between them
        case("gated", "gated_rows33", "f16", 33, 8190, 4001, "kn", "gelu_tanh", pad=7),
        # a training step's gated block, kept for the backward pass
        case("gated", "gated_4096", "bf16", 4096, 8192, 4096, "kn", "silu", bias=False, keep=True),
        # the backward pass of a projection
        case("linear_grad", "linear_grad_4096", "bf16", 4096, 4096, 4096, "kn", "gelu_tanh"),
        # the same in fp32, small and odd
        case("linear_grad", "linear_grad_f32", "f32", 777, 1025, 513, "kn", "relu"),
        # the backward pass of the gated block
        case("gated_grad", "gated_grad_2048", "bf16", 2048, 8192, 4096, "kn", "silu", bias=False),
        # the same for few tokens of odd sizes, in fp16 with transposed weights
        case("gated_grad", "gated_grad_odd", "f16", 1000, 2003, 1001, "nk", "gelu", pad=3),
    ]


def draw(rng):
    def size(low, high):
        n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
        return n if rng.random() < 0.4 else max(8, n // 8 * 8)

    op = rng.choice(("linear", "gated", "linear_grad", "gated_grad"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    most = (4e11 if dtype != "f32" else 2e10) / (2 * MATRICES[op])
    while True:
        M = size(1, 8192) if op in ("linear", "gated") else size(64, 8192)
        if op in ("linear", "gated") and rng.random() < 0.4:
            M = rng.randint(1, 48)  # single tokens and small batches
        N, K = size(128, 16384), size(128, 16384)
        if M * N * K <= most:
            break
    act = rng.choice(ACTS if op in ("linear", "linear_grad") else ("silu", "gelu", "gelu_tanh", "relu"))
    return case(op, None, dtype, M, N, K, rng.choice(("kn", "nk")), act, bias=rng.random() < 0.6,
                residual=op == "linear" and rng.random() < 0.5, keep=op in ("linear", "gated") and rng.random() < 0.4,
                pad=rng.choice((0, 0, 0, 1, 8)))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t, M, N, K, pad = TYPES[case["dtype"]], case["M"], case["N"], case["K"], case["pad"]

    def rows(r, c, scale=1.0):
        """r x c activations, `pad` elements apart."""
        whole = torch.randn(r, c + pad, generator=gen, device="cuda").mul_(scale).to(t)
        return whole[:, :c]

    def weight():
        n, k = (N, K)
        w = torch.randn(*((k, n) if case["store"] == "kn" else (n, k)), generator=gen, device="cuda")
        w = w.mul_(K ** -0.5).to(t)
        return w if case["store"] == "kn" else w.t()

    def empty(r, c):
        return torch.empty(r, c + pad, dtype=t, device="cuda")[:, :c]

    def like(w):
        return torch.empty_like(w)  # the weight's own storage order

    def vector():
        return torch.randn(N, generator=gen, device="cuda").mul_(0.5).to(t) if case["bias"] else None

    def vector_out():
        return torch.empty(N, dtype=t, device="cuda") if case["bias"] else None

    s = dict(case=case, X=rows(M, K))
    if case["op"] == "linear":
        s.update(W=weight(), b=vector(), R=rows(M, N) if case["residual"] else None, Y=empty(M, N),
                 Z=empty(M, N) if case["keep"] else None)
    elif case["op"] == "gated":
        s.update(Wg=weight(), Wu=weight(), bg=vector(), bu=vector(), H=empty(M, N),
                 G=empty(M, N) if case["keep"] else None, U=empty(M, N) if case["keep"] else None)
    elif case["op"] == "linear_grad":
        s.update(W=weight(), Z=rows(M, N), dY=rows(M, N), dX=empty(M, K), db=vector_out())
        s.update(dW=like(s["W"]))
    else:
        s.update(Wg=weight(), Wu=weight(), G=rows(M, N), U=rows(M, N), dH=rows(M, N), dX=empty(M, K),
                 dbg=vector_out(), dbu=vector_out())
        s.update(dWg=like(s["Wg"]), dWu=like(s["Wu"]))
    return s


# ---- the plain form ------------------------------------------------------------------------


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _slope(z, act):
    """The derivative of _act."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        h = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + h) + 0.5 * z * (1 - h * h) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain(s):
    c = s["case"]
    t, act, X = TYPES[c["dtype"]], c["act"], s["X"].float()
    if c["op"] == "linear":
        Z = X @ s["W"].float()
        if s["b"] is not None:
            Z = Z + s["b"].float()
        Y = _act(Z, act)
        if s["R"] is not None:
            Y = Y + s["R"].float()
        return {"Y": Y.to(t), "Z": Z.to(t)} if c["keep"] else {"Y": Y.to(t)}
    if c["op"] == "gated":
        G, U = X @ s["Wg"].float(), X @ s["Wu"].float()
        if s["bg"] is not None:
            G, U = G + s["bg"].float(), U + s["bu"].float()
        H = (_act(G, act) * U).to(t)
        return {"H": H, "G": G.to(t), "U": U.to(t)} if c["keep"] else {"H": H}
    if c["op"] == "linear_grad":
        dZ = s["dY"].float() * _slope(s["Z"].float(), act)
        out = {"dX": (dZ @ s["W"].float().t()).to(t), "dW": (X.t() @ dZ).to(t)}
        if c["bias"]:
            out["db"] = dZ.sum(0).to(t)
        return out
    G, U, dH = s["G"].float(), s["U"].float(), s["dH"].float()
    dG, dU = dH * U * _slope(G, act), dH * _act(G, act)
    out = {"dX": (dG @ s["Wg"].float().t() + dU @ s["Wu"].float().t()).to(t), "dWg": (X.t() @ dG).to(t),
           "dWu": (X.t() @ dU).to(t)}
    if c["bias"]:
        out.update(dbg=dG.sum(0).to(t), dbu=dU.sum(0).to(t))
    return out


# ---- the library's calls -------------------------------------------------------------------


def _own(s):
    from software_pipelined_tiled_loop_amd import binding as pg
    c = s["case"]
    act = c["act"]
    if c["op"] == "linear":
        pg.linear(s["X"], s["W"], s["Y"], bias=s["b"], residual=s["R"], act=act, Z=s["Z"])
        return {"Y": s["Y"], "Z": s["Z"]} if c["keep"] else {"Y": s["Y"]}
    if c["op"] == "gated":
        pg.gated(s["X"], s["Wg"], s["Wu"], s["H"], bias_g=s["bg"], bias_u=s["bu"], act=act, G=s["G"], U=s["U"])
        return {"H": s["H"], "G": s["G"], "U": s["U"]} if c["keep"] else {"H": s["H"]}
    if c["op"] == "linear_grad":
        pg.linear_backward(s["dY"], s["X"], s["W"], Z=s["Z"], act=act, dX=s["dX"], dW=s["dW"], dbias=s["db"])
        return {k: s[k] for k in ("dX", "dW", "db") if s[k] is not None}
    pg.gated_backward(s["dH"], s["X"], s["Wg"], s["Wu"], s["G"], s["U"], act=act, dX=s["dX"], dWg=s["dWg"],
                      dWu=s["dWu"], dbias_g=s["dbg"], dbias_u=s["dbu"])
    return {k: s[k] for k in ("dX", "dWg", "dWu", "dbg", "dbu") if s[k] is not None}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without, and its exact values -------------------------------------


def work(case):
    M, N, K, e = case["M"], case["N"], case["K"], BYTES[case["dtype"]]
    x, w, y, b = M * K, K * N, M * N, N if case["bias"] else 0
    values = {"linear": x + w + b + y * (1 + case["residual"] + case["keep"]),
              "gated": x + 2 * w + 2 * b + y * (1 + 2 * case["keep"]),
              "linear_grad": 2 * x + 2 * w + b + y * 2,
              "gated_grad": 2 * x + 4 * w + 2 * b + y * 3}[case["op"]]
    return {"bytes": e * values, "flops": 2 * MATRICES[case["op"]] * M * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    name = case["act"]

    def f(z):
        if name == "none":
            return z * 1.0
        if name == "relu":
            return z.clamp_min(0)
        if name == "silu":
            return z * torch.special.expit(z)
        if name == "gelu":
            return z * torch.special.ndtr(z)
        # (1 + tanh a) / 2 is the logistic function of 2a
        return z * torch.special.expit(math.sqrt(8 / math.pi) * z * (1 + 0.044715 * z.square()))

    def project(w, b):
        z = torch.mm(d["X"], d[w])
        return z.add_(d[b]) if b in d else z

    if case["op"] == "linear":
        z = project("W", "b")
        y = f(z)
        y = y.add_(d["R"]) if "R" in d else y
        return {"Y": y, "Z": z} if case["keep"] else {"Y": y}
    if case["op"] == "gated":
        g, u = project("Wg", "bg"), project("Wu", "bu")
        h = f(g).mul_(u)
        return {"H": h, "G": g, "U": u} if case["keep"] else {"H": h}

    def back(dz, w):
        """Gradients of sum(dz * (X w + b)) from its own definition."""
        return torch.mm(dz, d[w].t()), torch.mm(dz.t(), d["X"]).t(), torch.mv(dz.t(), dz.new_ones(dz.shape[0]))

    if case["op"] == "linear_grad":
        z = d["Z"].requires_grad_()
        dz, = torch.autograd.grad(f(z), z, d["dY"])
        dx, dw, db = back(dz, "W")
        return {"dX": dx, "dW": dw, "db": db} if case["bias"] else {"dX": dx, "dW": dw}
    g, u = d["G"].requires_grad_(), d["U"].requires_grad_()
    dg, du = torch.autograd.grad(f(g) * u, (g, u), d["dH"])
    (xg, wg, bg), (xu, wu, bu) = back(dg, "Wg"), back(du, "Wu")
    out = {"dX": xg + xu, "dWg": wg, "dWu": wu}
    return dict(out, dbg=bg, dbu=bu) if case["bias"] else out
