"""What is measured of a transformer layer's operators around its experts: the root-mean-square norm with the
residual's addition (in the rows' type, in 8-bit integers for the products, and its gradient), the gated feed-forward
product (8-bit integers for serving, 16-bit types with gradients for training) and the experts' products in 16-bit
types with their gradients.

A case's "op" says which operator one pass runs; run() has both the plain form (elementary torch operations in 32
bits) and the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
TINY = 2.0 ** -119  # rows whose largest magnitude is below this quantise to zeros


# ------------------------------------------------------------------ cases
# op "norm":     T rows of H values; direction "forward" (x, residual -> norm, sum) or "backward" (gradient of both)
# op "linear":   the norm of T rows of K values in 8 bits, then the product with N x K int8 weights that reads it
# op "gated8":   T tokens of k slots through E experts' gated products in int8 (E = 0: one matrix)
# op "gated":    the same in 16 bits; direction "forward" (with the pre-activations kept) or "backward"
# op "product":  T tokens' k slots through E experts' products in 16 bits; direction "forward" or "backward"
# N is the width after the gate: a gated case's matrices have 2 N rows.  "dropped" is the share of slots routed nowhere.
def listed():
    return [
        # one generated token between two layers: nothing but latency
        dict(name="norm, one token", op="norm", direction="forward", T=1, H=4096, dtype="bf16", wtype="bf16", residual=True),
        # a training step's tokens
        dict(name="norm, training", op="norm", direction="forward", T=16384, H=4096, dtype="bf16", wtype="bf16", residual=True),
        # the gradient of the same, with the gradient that the residual stream brings
        dict(name="norm gradient, training", op="norm", direction="backward", T=16384, H=4096, dtype="bf16", wtype="f32", residual=True),
        # rows that no vector load fits, a norm without a residual
        dict(name="norm gradient, odd", op="norm", direction="backward", T=1021, H=2045, dtype="f32", wtype="f32", residual=False),
        # a decode batch into an 8-bit projection
        dict(name="norm and projection, decode", op="linear", T=16, K=4096, N=4096, dtype="bf16", wtype="bf16", out="bf16"),
        # a prefill batch into a narrow projection (keys and values of grouped heads)
        dict(name="norm and projection, prefill", op="linear", T=8192, K=4096, N=1024, dtype="bf16", wtype="bf16", out="bf16"),
        # a decode batch through the experts: their weights are read for a few rows each
        dict(name="gated int8, decode", op="gated8", T=32, k=8, E=64, K=4096, N=1024, out="bf16", dropped=0.0),
        # a prefill batch through one dense block
        dict(name="gated int8, dense prefill", op="gated8", T=4096, k=1, E=0, K=4096, N=8192, out="bf16", dropped=0.0),
        # a training step's experts, tokens gathered by the product
        dict(name="gated, training", op="gated", direction="forward", T=8192, k=4, E=32, K=2048, N=1408, dtype="bf16", dropped=0.0),
        dict(name="gated gradient, training", op="gated", direction="backward", T=8192, k=4, E=32, K=2048, N=1408, dtype="bf16", dropped=0.05),
        # a decode batch through the experts' second matrix
        dict(name="experts, decode", op="product", direction="forward", T=16, k=4, E=32, K=1408, N=2048, dtype="bf16", dropped=0.0),
        # no size fits a tile, a vector or a line
        dict(name="experts' gradient, odd", op="product", direction="backward", T=777, k=3, E=7, K=1111, N=513, dtype="f16", dropped=0.1),
    ]


def _spread(rng, lo, hi, odd=0.5):
    """A whole number from lo to hi, spread over its logarithm; half of them multiples of 64 where there is room."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() >= odd and v >= 64:
        v -= v % 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "norm", "linear", "gated8", "gated", "gated", "product", "product"])
    c = {"op": op}
    if op == "norm":
        c["direction"] = rng.choice(["forward", "backward"])
        c["H"] = _spread(rng, 64, 16384)
        c["T"] = _spread(rng, 1, min(65536, (1 << 26) // c["H"]), odd=0.7)
        c["dtype"] = rng.choice(["f32", "bf16", "f16"])
        c["wtype"] = rng.choice([c["dtype"], "f32"])
        c["residual"] = rng.random() < 0.7
        return c
    c["K"], c["N"] = _spread(rng, 64, 8192), _spread(rng, 64, 8192)
    if op == "linear":
        c["dtype"] = rng.choice(["bf16", "f16"])
        c["wtype"], c["out"] = rng.choice([c["dtype"], "f32"]), rng.choice(["bf16", "f16"])
        c["T"] = _spread(rng, 1, min(16384, max(1, (1 << 37) // (c["K"] * c["N"]))), odd=0.7)
        return c
    c["k"] = rng.randint(1, 8)
    c["E"] = _spread(rng, c["k"], 128, odd=0.7)
    c["dropped"] = rng.choice([0.0, 0.0, 0.05, 0.3])
    if rng.random() < 0.25:  # one matrix
        c["k"], c["E"], c["dropped"] = 1, 0, 0.0
    if op == "gated8":
        c["out"] = rng.choice(["bf16", "f16"])
    else:
        c["direction"], c["dtype"] = rng.choice(["forward", "backward"]), rng.choice(["bf16", "f16"])
    while c["E"] * c["K"] * c["N"] > 1 << 28:
        c["E"] = max(c["k"], c["E"] // 2)
        if c["E"] == c["k"]:
            c["K"], c["N"] = max(64, c["K"] // 2), max(64, c["N"] // 2)
    # the plain form pads every expert to the longest: a third of the largest listed case's products at most
    most = (1 << 36) // (c["k"] * c["K"] * c["N"])
    c["T"] = _spread(rng, 1, max(1, min(most, 32768 // c["k"])), odd=0.7)
    return c


# ------------------------------------------------------------------ inputs
def _route(c, g):
    """Expert ids as a router draws them: the k best of scores that favour some experts, a share of the slots routed
    nowhere (padding tokens, all k of them; single slots over an expert's capacity)."""
    favour = torch.randn(c["E"], generator=g, device="cuda")
    score = torch.randn(c["T"], c["E"], generator=g, device="cuda") + 0.7 * favour
    ids = score.topk(c["k"], dim=1).indices
    if c["dropped"]:
        u = torch.rand(c["T"], c["k"], generator=g, device="cuda") < c["dropped"] / 2
        v = torch.rand(c["T"], 1, generator=g, device="cuda") < c["dropped"] / 2
        ids = torch.where(u | v, -1, ids)
    return ids


def _sorted(ids, E):
    """offsets [E + 1] and src (sorted place -> slot, -1 behind the last) of a stable sort by expert."""
    flat = torch.where(ids < 0, E, ids).reshape(-1)
    keys, order = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(keys, torch.arange(E + 1, device=flat.device))
    return offsets.int(), torch.where(keys < E, order, -1).int()


def _normal(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _codes(shape, g):
    """int8 values as a quantiser leaves them: a normal distribution whose largest value in a row is about 127."""
    return (torch.randn(shape, generator=g, device="cuda") * 34).round_().clamp_(-127, 127).to(torch.int8)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("norm", "linear"):
        H = c["H"] if c["op"] == "norm" else c["K"]
        dt = DTYPES[c["dtype"]]
        s["x"] = _normal((c["T"], H), g, dt)
        s["w"] = (1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(DTYPES[c["wtype"]])
        if c["op"] == "linear" or c["residual"]:
            s["r"] = _normal((c["T"], H), g, dt, 3.0)
        if c["op"] == "linear":
            s["b"] = _codes((c["N"], H), g)
            s["sb"] = (torch.rand(c["N"], generator=g, device="cuda") + 0.5) * (1.0 / (34 * math.sqrt(H)))
        elif c["direction"] == "backward":
            s["dy"] = _normal((c["T"], H), g, dt)
        return s
    S, rows, experts = c["T"] * c["k"], c["N"] * (1 if c["op"] == "product" else 2), max(c["E"], 1)
    if c["E"]:
        s["offsets"], s["src"] = _sorted(_route(c, g), c["E"])
    if c["op"] == "gated8":
        s["x"] = _codes((c["T"], c["K"]), g)
        s["sx"] = torch.rand(c["T"], generator=g, device="cuda") * 0.02 + 0.02
        b = torch.empty(experts, rows, c["K"], dtype=torch.int8, device="cuda")
        sb = (torch.rand(experts, rows, generator=g, device="cuda") + 0.5) * (1.0 / (34 * math.sqrt(c["K"])))
        s["sb"] = sb if c["E"] else sb[0]
        dt = DTYPES[c["out"]]
    else:
        dt = DTYPES[c["dtype"]]
        gathered = c["op"] == "gated" and c["E"]  # the second matrix reads what the first has left in order
        s["x"] = _normal((c["T"] if gathered else S, c["K"]), g, dt)
        b = torch.empty(experts, rows, c["K"], dtype=dt, device="cuda")
    for e in range(experts):
        b[e] = _codes((rows, c["K"]), g) if c["op"] == "gated8" else _normal((rows, c["K"]), g, dt, 1.0 / math.sqrt(c["K"]))
    s["b"] = b if c["E"] else b[0]
    if c.get("direction") == "backward":
        s["dy"] = _normal((S, c["N"]), g, dt)
        s["dx"] = torch.zeros(S, c["K"], dtype=dt, device="cuda")  # buffers that the program keeps
        if c["op"] == "gated":
            s["pre"] = _normal((S, rows), g, dt)
    else:
        s["out"] = torch.zeros(S, c["N"], dtype=dt, device="cuda")
        if c["op"] == "gated":
            s["pre"] = torch.zeros(S, rows, dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _norm(s):
    """The rows' sum as it is stored, and its norm in 32 bits."""
    x = (s["x"].float() + s["r"].float()).to(s["x"].dtype) if "r" in s else s["x"]
    v = x.float()
    return x, v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["w"].float()


def _norm_backward(s):
    x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
    i = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    n, dn = x * i, dy * w
    dx = i * (dn - n * (dn * n).mean(1, keepdim=True))
    if "r" in s:  # here the gradient that the residual stream brings
        dx = dx + s["r"].float()
    return dx.to(s["x"].dtype), (dy * n).sum(0)


def _quantize(x):
    """Codes (whole numbers, held as float) and scales of every row."""
    a = x.abs().amax(1)
    live = a >= TINY
    q = (127.0 * x / torch.where(live, a, 1.0).unsqueeze(1)).round()
    return torch.where(live.unsqueeze(1), q, 0.0), torch.where(live, a / 127.0, 0.0)


class _Padded:
    """Every expert's rows side by side, padded to the longest of them; one spare row takes what is routed nowhere."""

    def __init__(self, s):
        c = s["case"]
        self.S = c["T"] * c["k"]
        self.E = max(c["E"], 1)
        if not c["E"]:
            self.cap, self.at, self.live = self.S, None, None
            return
        offsets = s["offsets"].long()
        self.cap = max(int((offsets[1:] - offsets[:-1]).max()), 1)
        place = torch.arange(self.S, device=offsets.device)
        e = torch.searchsorted(offsets[1:].contiguous(), place, right=True)
        self.live = (e < self.E).unsqueeze(1)
        self.at = torch.where(e < self.E, e * self.cap + place - offsets[e.clamp_max(self.E)], self.E * self.cap)
        self.e = e.clamp_max(self.E - 1)

    def put(self, rows):
        if self.at is None:
            return rows.unsqueeze(0)
        out = torch.zeros(self.E * self.cap + 1, rows.shape[1], device=rows.device).index_copy_(0, self.at, rows)
        out[-1] = 0.0
        return out[:-1].view(self.E, self.cap, -1)

    def take(self, padded):
        if self.at is None:
            return padded[0]
        rows = padded.reshape(self.E * self.cap, -1)[self.at.clamp_max(self.E * self.cap - 1)]
        return torch.where(self.live, rows, 0.0)


def _activated(g):
    return g * torch.sigmoid(g)


def _run_plain(s):
    c = s["case"]
    back = c.get("direction") == "backward"
    if c["op"] == "norm":
        if back:
            return _norm_backward(s)
        x, y = _norm(s)
        return (y.to(x.dtype), x) if "r" in s else y.to(x.dtype)
    if c["op"] == "linear":
        x, y = _norm(s)
        q, sq = _quantize(y)
        return ((q @ s["b"].float().t()) * sq.unsqueeze(1) * s["sb"]).to(DTYPES[c["out"]]), sq, x
    pad = _Padded(s)
    rows = (s["src"].clamp_min(0) // c["k"]).long() if c["E"] and c["op"] != "product" else slice(None)
    x, b = pad.put(s["x"].float()[rows]), s["b"].float().view(pad.E, -1, c["K"])
    if back:
        dy = s["dy"].float()
        if c["op"] == "gated":
            g, u = s["pre"].float().chunk(2, 1)
            sig = torch.sigmoid(g)
            dy = torch.cat([dy * u * sig * (1.0 + g * (1.0 - sig)), dy * g * sig], 1)
        dy = pad.put(dy)
        dx = pad.take(torch.bmm(dy, b))
        db = torch.bmm(dy.transpose(1, 2).contiguous(), x)
        return dx.to(s["x"].dtype), db.to(s["x"].dtype).view(s["b"].shape)
    y = pad.take(torch.bmm(x, b.transpose(1, 2).contiguous()))
    if c["op"] == "product":
        return y.to(s["x"].dtype)
    if c["op"] == "gated8":
        y = y * s["sx"][rows].unsqueeze(1) * (s["sb"][pad.e] if c["E"] else s["sb"])
    g, u = y.chunk(2, 1)
    h = (_activated(g) * u).to(s["out"].dtype)
    return h if c["op"] == "gated8" else (h, y.to(h.dtype))


# ------------------------------------------------------------------ the framework's calls
def _run_own(s):
    import spmm_csr_spmv_amd as sp

    c = s["case"]
    back = c.get("direction") == "backward"
    if c["op"] == "norm":
        if back:
            return sp.rms_norm_backward(s["dy"], s["x"], s["w"], eps=EPS, dsum=s.get("r"))
        return sp.rms_norm(s["x"], s["w"], residual=s.get("r"), eps=EPS)
    if c["op"] == "linear":
        q, sq, x = sp.rms_norm_i8(s["x"], s["w"], residual=s["r"], eps=EPS)
        return sp.gemm_i8(q, sq, s["b"], s["sb"], dtype=DTYPES[c["out"]]), sq, x
    if c["op"] == "gated8":
        if not c["E"]:
            return sp.gated_i8(s["x"], s["sx"], s["b"], s["sb"], out=s["out"])
        return sp.moe_gated_i8(s["x"], s["sx"], s["b"], s["sb"], s["offsets"], src=s["src"], slots=c["k"], out=s["out"])
    offsets = s.get("offsets")
    if c["op"] == "product":
        if back:
            return sp.moe_gemm_backward(s["dy"], s["x"], s["b"], offsets, dA=s["dx"])
        return sp.moe_gemm(s["x"], s["b"], offsets, out=s["out"])
    if back:
        return sp.moe_gated_backward(s["dy"], s["pre"], s["x"], s["b"], offsets, src=s.get("src"), slots=c["k"], dA=s["dx"])
    return sp.moe_gated(s["x"], s["b"], offsets, src=s.get("src"), slots=c["k"], pre=s["pre"], out=s["out"]), s["pre"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ bytes and operations
def work(case):
    c = case
    if c["op"] == "norm":
        n, b = c["T"] * c["H"], BYTES[c["dtype"]]
        weights = c["H"] * BYTES[c["wtype"]]
        if c["direction"] == "backward":
            return {"bytes": n * b * (4 if c["residual"] else 3) + weights + 4 * c["H"], "flops": 10 * n}
        return {"bytes": n * b * (4 if c["residual"] else 2) + weights, "flops": 5 * n}
    if c["op"] == "linear":
        n = c["T"] * c["K"]
        read = 2 * n * BYTES[c["dtype"]] + c["K"] * BYTES[c["wtype"]] + c["N"] * c["K"] + 4 * c["N"]
        return {"bytes": read + n * BYTES[c["dtype"]] + 4 * c["T"] + c["T"] * c["N"] * BYTES[c["out"]],
                "flops": 2 * n * c["N"]}
    S = c["T"] * c["k"]
    kept = S * (1.0 - c["dropped"] + c["dropped"] ** 2 / 4)
    live = c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"]) if c["E"] else 1  # experts that get a token, about
    rows = c["N"] * (1 if c["op"] == "product" else 2)
    tokens = c["T"] if c["op"] != "product" else kept
    index = 4 * (kept + c["E"] + 1) if c["E"] else 0
    flops = 2 * kept * rows * c["K"]
    if c["op"] == "gated8":
        read = c["T"] * (c["K"] + 4) + live * rows * (c["K"] + 4)
        return {"bytes": read + kept * c["N"] * BYTES[c["out"]] + index, "flops": flops}
    b = BYTES[c["dtype"]]
    if c["direction"] == "forward":
        wrote = kept * (c["N"] + (rows if c["op"] == "gated" else 0))
        return {"bytes": (tokens * c["K"] + live * rows * c["K"] + wrote) * b + index, "flops": flops}
    read = kept * (c["N"] + (rows if c["op"] == "gated" else 0)) + tokens * c["K"] + live * rows * c["K"]
    return {"bytes": (read + kept * c["K"] + max(c["E"], 1) * rows * c["K"]) * b + index, "flops": 2 * flops}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    back = c.get("direction") == "backward"
    if c["op"] in ("norm", "linear"):
        x = s["x"].double()
        if "r" in s and not back:
            x = (x + s["r"].double()).to(s["x"].dtype).double()  # the sum is what is stored
        w = s["w"].double()
        length = torch.linalg.vector_norm(x, dim=1, keepdim=True) / math.sqrt(x.shape[1])
        unit = x / torch.hypot(length, torch.full_like(length, math.sqrt(EPS)))
        if back:
            dy = s["dy"].double()
            along = torch.linalg.vecdot(dy * w, unit).unsqueeze(1) / x.shape[1]
            dx = (dy * w - unit * along) / torch.hypot(length, torch.full_like(length, math.sqrt(EPS)))
            return dx + s["r"].double() if "r" in s else dx, torch.linalg.vecdot(dy.t().contiguous(), unit.t().contiguous())
        y = unit * w
        if c["op"] == "norm":
            return (y, x) if "r" in s else y
        a = y.abs().max(dim=1).values
        q = torch.round(127 * y / a.clamp_min(TINY).unsqueeze(1))
        return torch.matmul(q, s["b"].double().t()) * torch.outer(a / 127, s["sb"].double()), a / 127, x
    S, rows = c["T"] * c["k"], c["N"] * (1 if c["op"] == "product" else 2)
    at = s["offsets"].tolist() if c["E"] else [0, S]
    y = torch.zeros(S, rows, dtype=torch.float64, device="cuda")
    h = torch.zeros(S, c["N"], dtype=torch.float64, device="cuda")
    dx = torch.zeros(S, c["K"], dtype=torch.float64, device="cuda")
    db = torch.zeros(len(at) - 1, rows, c["K"], dtype=torch.float64, device="cuda")
    for e in range(len(at) - 1):
        mine = torch.arange(at[e], at[e + 1], device="cuda")
        row = s["src"][mine].long() // c["k"] if c["E"] and c["op"] != "product" else mine
        x, b = s["x"][row].double(), s["b"].view(-1, rows, c["K"])[e].double()
        if back:
            d = s["dy"][mine].double()
            if c["op"] == "gated":
                g, u = s["pre"][mine, :c["N"]].double(), s["pre"][mine, c["N"]:].double()
                t = torch.tanh(g / 2)  # sigmoid(g) = (1 + t) / 2
                d = torch.cat([d * u * ((1 + t) / 2 + g * (1 - t * t) / 4), d * g * (1 + t) / 2], 1)
            dx[mine] = torch.matmul(d, b)
            db[e] = torch.matmul(d.t().contiguous(), x)
            continue
        y[mine] = torch.matmul(x, b.t())
        if c["op"] == "gated8":
            y[mine] *= torch.outer(s["sx"][row].double(), s["sb"].view(-1, rows)[e].double())
        if c["op"] != "product":
            g, u = y[mine, :c["N"]], y[mine, c["N"]:]
            h[mine] = g * u / (1 + torch.exp(-g))
    if back:
        return dx, db.view(s["b"].shape)
    return y if c["op"] == "product" else h if c["op"] == "gated8" else (h, y)
