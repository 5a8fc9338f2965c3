"""Workloads of the operators that train the layer's experts: products grouped
by expert with both gradients, the gated activation with the routing weight,
and the orthogonalised update of stacked weights.

Each case is one call as a training (or serving) program makes it.  ``own``
selects the side: False computes the plain form (elementary torch operations
in 32 bits, rounded once at the end), True calls the package's entry points.

Shapes are those of the package's own configurations (d = 5120, d_ff = 2560,
256 experts, top 8; the small layer d = 512, d_ff = 256, 64 experts) and
generic ones between and beside them.  Group sizes are drawn the way a router
produces them: uneven, some groups empty.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_COEFFS = (3.4445, -4.7750, 2.0315)   # the usual quintic of the Muon optimiser
_EPS = 1e-7


# ------------------------------------------------------------------- cases
def _grouped(op, rows, E, N, K, dt, out, skew):
    return {"op": op, "rows": rows, "E": E, "N": N, "K": K, "dt": dt, "out": out, "skew": skew}


def _gate(op, rows, F, dt, weighted):
    return {"op": op, "rows": rows, "F": F, "dt": dt, "weighted": weighted}


def _ortho(batch, R, C, dt):
    return {"op": "orthogonalize", "batch": batch, "R": R, "C": C, "dt": dt, "out": "bf16"}


def listed():
    return [
        # the gate projection of a decode batch: 32 tokens, top 8 of 256 experts
        {"name": "product, decode T=32"} | _grouped("product", 256, 256, 2560, 5120, "bf16", "bf16", 0.3),
        # the small layer's gate projection, 64 tokens of 64 experts: latency counts
        {"name": "product, small layer"} | _grouped("product", 512, 64, 256, 512, "f16", "f16", 0.3),
        # the down projection of a training batch of 32768 tokens
        {"name": "product, batch T=32768"} | _grouped("product", 262144, 256, 5120, 2560, "bf16", "bf16", 0.3),
        # the input gradient of the gate projection over a chunk of 8192 tokens
        {"name": "input grad, T=8192"} | _grouped("product_dx", 65536, 256, 2560, 5120, "bf16", "bf16", 0.3),
        # sizes that no vector width divides, uneven groups, gradient kept in 32 bits
        {"name": "input grad, odd sizes"} | _grouped("product_dx", 3001, 24, 1365, 2047, "f16", "f32", 1.0),
        # the weight gradient of the down projection over the chunk, as 32-bit master gradients
        {"name": "weight grad, T=8192"} | _grouped("product_dw", 65536, 256, 5120, 2560, "bf16", "f32", 0.3),
        # the weight gradient of a few local experts (expert parallelism), 16-bit, very uneven
        {"name": "weight grad, 32 experts"} | _grouped("product_dw", 8191, 32, 2560, 5120, "bf16", "bf16", 1.0),
        # the activation between the products: a small batch forward, a training chunk backward
        {"name": "gated activation, T=64"} | _gate("gate", 512, 2560, "bf16", True),
        {"name": "gated activation grad"} | _gate("gate_grad", 65536, 2560, "bf16", True),
        # updates: the small layer's router, eight experts' projections, odd tall ones in 32 bits
        {"name": "update, small router"} | _ortho(1, 64, 512, "bf16"),
        {"name": "update, 8 experts"} | _ortho(8, 2560, 5120, "bf16"),
        {"name": "update, odd and tall"} | _ortho(3, 1001, 777, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Mostly multiples of 8, as model widths are; one in five as it falls."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.2 else max(8, (v + 4) // 8 * 8)


def draw(rng):
    kind = rng.choice(["product", "product_dx", "product_dw", "gate", "gate_grad", "orthogonalize"])
    if kind == "orthogonalize":
        R, C = _width(rng, 32, 5120), _width(rng, 32, 5120)
        most = work(_ortho(8, 2560, 5120, "bf16"))["flops"] / work(_ortho(1, R, C, "bf16"))["flops"]
        return _ortho(max(1, min(_log(rng, 1, 16), int(most))), R, C, rng.choice(["bf16", "f16", "f32"]))
    if kind in ("gate", "gate_grad"):
        rows, F = _log(rng, 1, 65536), _width(rng, 64, 5120)
        rows = min(rows, 65536 * 2560 // F)
        return _gate(kind, rows, F, rng.choice(["bf16", "f16"]), rng.random() < 0.7)
    E, N, K = _log(rng, 4, 256), _width(rng, 128, 5120), _width(rng, 128, 5120)
    rows = _log(rng, 8, 65536)
    dt = rng.choice(["bf16", "bf16", "f16"])
    return _grouped(kind, rows, E, N, K, dt, rng.choice([dt, dt, "f32"]), rng.choice([0.3, 1.0]))


# ------------------------------------------------------------------- inputs
def _offsets(case, seed):
    """Group boundaries as a router leaves them: shares with a log-normal
    spread, multinomial counts, now and then an expert that nothing chose."""
    r = np.random.default_rng(seed)
    share = np.exp(case["skew"] * r.standard_normal(case["E"]))
    share[r.random(case["E"]) < 0.03] = 0.0
    share = share if share.sum() > 0 else np.ones(case["E"])
    return np.concatenate([[0], np.cumsum(r.multinomial(case["rows"], share / share.sum()))])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dt=None):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt or _DT[case["dt"]]).mul_(scale)

    s = {"case": case}
    if case["op"].startswith("product"):
        off = _offsets(case, seed)
        rows, E, N, K = (case[k] for k in ("rows", "E", "N", "K"))
        s["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
        # where each row sits in a padded batch [E, longest] (the plain form's plan)
        group = np.repeat(np.arange(E), np.diff(off))
        s["group"] = torch.tensor(group, device="cuda")
        s["place"] = torch.tensor(np.arange(rows) - off[group], device="cuda")
        s["longest"] = int(np.diff(off).max())
        if case["op"] != "product_dx":
            s["x"] = normal(rows, K)
        if case["op"] != "product":
            s["dy"] = normal(rows, N, scale=1e-2)
        if case["op"] != "product_dw":
            s["w"] = normal(E, N, K, scale=0.02)
        if own:
            import group_limited_routed_gb300 as pkg
            call = {"product": pkg.grouped_matmul, "product_dx": pkg.grouped_matmul_dx,
                    "product_dw": pkg.grouped_matmul_dw}[case["op"]]
            s["call"] = call
            s["ws"] = pkg.OpWorkspace(pkg.grouped_matmul_workspace_size(rows, E, N, K, dtype=_DT[case["dt"]]))
    elif case["op"].startswith("gate"):
        s["g"] = normal(case["rows"], case["F"])
        s["u"] = normal(case["rows"], case["F"])
        if case["op"] == "gate_grad":
            s["dh"] = normal(case["rows"], case["F"], scale=1e-2)
        # routing weights: positive, 2.5 over 8 experts on average
        s["w"] = torch.rand(case["rows"], generator=g, device="cuda").mul_(0.5).add_(0.06) if case["weighted"] else None
        if own:
            import group_limited_routed_gb300 as pkg
            s["call"] = pkg.swiglu if case["op"] == "gate" else pkg.swiglu_grad
    else:
        # a momentum buffer: a few strong directions over a broad floor
        b, R, C = case["batch"], case["R"], case["C"]
        k = max(1, min(R, C) // 16)
        m = torch.bmm(normal(b, R, k, dt=torch.float32), normal(b, k, C, dt=torch.float32)).mul_(k ** -0.5)
        s["m"] = m.add_(normal(b, R, C, scale=0.3, dt=torch.float32)).mul_(1e-3).to(_DT[case["dt"]])
        if own:
            import group_limited_routed_gb300 as pkg
            s["call"] = pkg.orthogonalize
            s["ws"] = pkg.OpWorkspace(pkg.orthogonalize_workspace_size(b, R, C))
    return s


# ------------------------------------------------------------------- one pass
def _padded(s, rows):
    """[E, longest, width] in 32 bits, zero where a group has no row."""
    out = rows.new_zeros((s["case"]["E"], s["longest"], rows.shape[1]), dtype=torch.float32)
    out[s["group"], s["place"]] = rows.float()
    return out


def _run_own(s):
    c = s["case"]
    if c["op"] == "gate":
        return s["call"](s["g"], s["u"], s["w"])
    if c["op"] == "gate_grad":
        return s["call"](s["dh"], s["g"], s["u"], s["w"])
    if c["op"] == "orthogonalize":
        return s["call"](s["m"], steps=5, coeffs=_COEFFS, eps=_EPS, out_dtype=_DT[c["out"]], ws=s["ws"])
    if c["op"] == "product_dw":
        return s["call"](s["dy"], s["x"], s["offsets"], out_dtype=_DT[c["out"]], ws=s["ws"])
    return s["call"](s["dy"] if c["op"] == "product_dx" else s["x"], s["w"], s["offsets"],
                     out_dtype=_DT[c["out"]], ws=s["ws"])


def _steps(x):
    a, b, c = _COEFFS
    gram = torch.bmm(x, x.mT)
    poly = torch.baddbmm(gram, gram, gram, beta=b, alpha=c)
    return torch.baddbmm(x, poly, x, beta=a)


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "product":
        return torch.bmm(_padded(s, s["x"]), s["w"].float().mT)[s["group"], s["place"]].to(_DT[c["out"]])
    if c["op"] == "product_dx":
        return torch.bmm(_padded(s, s["dy"]), s["w"].float())[s["group"], s["place"]].to(_DT[c["out"]])
    if c["op"] == "product_dw":
        return torch.bmm(_padded(s, s["dy"]).mT, _padded(s, s["x"])).to(_DT[c["out"]])
    if c["op"] == "orthogonalize":
        x = s["m"].float()
        x = x.mT if c["R"] > c["C"] else x
        x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + _EPS)
        x = _steps(_steps(_steps(_steps(_steps(x)))))
        return (x.mT if c["R"] > c["C"] else x).to(_DT[c["out"]]).contiguous()
    dt = _DT[c["dt"]]
    g, u = s["g"].float(), s["u"].float()
    w = 1.0 if s["w"] is None else s["w"][:, None]
    sig = 1.0 / (1.0 + torch.exp(-g))
    if c["op"] == "gate":
        return (w * g * sig * u).to(dt)
    dh = s["dh"].float()
    dg = (dh * w * u * sig * (1.0 + g * (1.0 - sig))).to(dt)
    du = (dh * w * g * sig).to(dt)
    return (dg, du) if s["w"] is None else (dg, du, (dh * g * sig * u).sum(1))


# ------------------------------------------------------------------- work
def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    i = size[case["dt"]]
    if case["op"].startswith("product"):
        rows, E, N, K, o = *(case[k] for k in ("rows", "E", "N", "K")), size[case["out"]]
        touched = min(E, rows)   # weights no row needs are not read
        if touched < E or rows < 8 * E:
            touched = E * (1.0 - (1.0 - 1.0 / E) ** rows)
        flops = 2.0 * rows * N * K
        if case["op"] == "product":
            return {"bytes": rows * K * i + touched * N * K * i + rows * N * o, "flops": flops}
        if case["op"] == "product_dx":
            return {"bytes": rows * N * i + touched * N * K * i + rows * K * o, "flops": flops}
        return {"bytes": rows * (N + K) * i + E * N * K * o, "flops": flops}
    if case["op"].startswith("gate"):
        n, grad = case["rows"] * case["F"], case["op"] == "gate_grad"
        per_row = 4 * case["rows"] * (2 if grad else 1) if case["weighted"] else 0
        return {"bytes": n * i * (5 if grad else 3) + per_row, "flops": n * (16 if grad else 6)}
    m, n = sorted((case["R"], case["C"]))
    # both Gram products are symmetric: half of each is enough
    flops = 5.0 * (m * m * n + m ** 3 + 2.0 * m * m * n)
    return {"bytes": case["batch"] * m * n * (i + size[case["out"]]), "flops": case["batch"] * flops}


# ------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits, group by group and matrix by matrix."""
    s = prepare(case, seed)
    if case["op"].startswith("product"):
        off = s["offsets"].tolist()
        E, N, K = case["E"], case["N"], case["K"]
        shape = {"product": (case["rows"], N), "product_dx": (case["rows"], K), "product_dw": (E, N, K)}[case["op"]]
        out = torch.zeros(shape, dtype=torch.float64, device="cuda")
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            if case["op"] == "product":
                out[lo:hi] = s["x"][lo:hi].double() @ s["w"][e].double().t()
            elif case["op"] == "product_dx":
                out[lo:hi] = s["dy"][lo:hi].double() @ s["w"][e].double()
            else:
                out[e] = s["dy"][lo:hi].double().t() @ s["x"][lo:hi].double()
        return out
    if case["op"] == "orthogonalize":
        a, b, c = _COEFFS
        out = torch.empty(s["m"].shape, dtype=torch.float64, device="cuda")
        for i, m in enumerate(s["m"].double()):
            x = m / (torch.linalg.matrix_norm(m) + _EPS)
            for _ in range(5):
                # the odd polynomial by the smaller Gram matrix, from whichever side it sits on
                if x.shape[0] <= x.shape[1]:
                    q = x @ x.t()
                    x = a * x + b * (q @ x) + c * (q @ (q @ x))
                else:
                    q = x.t() @ x
                    x = a * x + b * (x @ q) + c * ((x @ q) @ q)
            out[i] = x
        return out
    g, u = s["g"].double(), s["u"].double()
    w = torch.ones(case["rows"], 1, dtype=torch.float64, device="cuda") if s["w"] is None else s["w"].double()[:, None]
    sig = torch.sigmoid(g)
    if case["op"] == "gate":
        return w * u * g * sig
    dh = s["dh"].double()
    dg, du = dh * w * u * (sig + g * sig * torch.sigmoid(-g)), dh * w * g * sig
    return (dg, du) if s["w"] is None else (dg, du, torch.einsum("rf,rf->r", dh, g * sig * u))
