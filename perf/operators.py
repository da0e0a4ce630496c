"""What is measured of the mixture-of-experts operators: sorting tokens by expert,
moving their rows there and back with weights (and the gradients of both), and
products in 8-bit integers with a scale per token and per channel.

A case's "op" says which operator one pass runs; run() has both the plain form
(elementary torch operations in 32 bits) and the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
TINY = 2.0 ** -119  # rows whose largest magnitude is below this quantise to zeros


# ------------------------------------------------------------------ cases
# op "sort":     T tokens of k slots over E experts
# op "dispatch": rows of H values; direction "forward" (X -> sorted rows) or "backward" (their gradient -> X's)
# op "combine":  direction "forward" (sorted rows, weights -> tokens) or "backward" (gradients of both)
# op "linear":   rows of `dtype` quantised per token, then the product with int8 weights (E = 0: one matrix)
# op "product":  the product alone, operands already in int8
# "dropped" is the share of slots routed nowhere; "out" the type of the product.
def listed():
    return [
        # one generated token: nothing but latency
        dict(name="sort, one token", op="sort", T=1, k=8, E=64, dropped=0.0),
        # a long prefill batch, part of it padding
        dict(name="sort, long batch", op="sort", T=65536, k=8, E=128, dropped=0.1),
        # a training step's tokens on their way to the experts
        dict(name="dispatch, training", op="dispatch", direction="forward", T=16384, k=4, E=32, H=4096, dtype="bf16", dropped=0.0),
        # the gradient on its way back, odd sizes, rows that no vector load fits
        dict(name="dispatch gradient, odd", op="dispatch", direction="backward", T=1021, k=3, E=9, H=1001, dtype="f32", dropped=0.1),
        # a small decode batch
        dict(name="combine, decode", op="combine", direction="forward", T=16, k=8, E=64, H=4096, dtype="bf16", dropped=0.0),
        # a training step's tokens on their way back
        dict(name="combine, prefill", op="combine", direction="forward", T=16384, k=8, E=64, H=2048, dtype="f16", dropped=0.05),
        dict(name="combine gradient, training", op="combine", direction="backward", T=16384, k=4, E=32, H=4096, dtype="bf16", dropped=0.0),
        dict(name="combine gradient, odd", op="combine", direction="backward", T=777, k=5, E=11, H=2045, dtype="f16", dropped=0.2),
        # a decode batch through the experts' first matrix: every expert's weights are read for a few rows
        dict(name="experts, decode", op="linear", T=32, k=8, E=64, K=4096, N=2048, dtype="bf16", out="bf16", dropped=0.0),
        # a prefill batch through the same matrix
        dict(name="experts, prefill", op="linear", T=4096, k=8, E=64, K=4096, N=2048, dtype="bf16", out="bf16", dropped=0.0),
        # a dense layer of a prefill batch, operands already in int8
        dict(name="product, large", op="product", T=8192, k=1, E=0, K=4096, N=8192, dtype="bf16", out="bf16", dropped=0.0),
        # no size fits a tile, a vector or a line
        dict(name="linear, odd", op="linear", T=333, k=1, E=0, K=1111, N=1001, dtype="f16", out="f32", dropped=0.0),
    ]


def _spread(rng, lo, hi, odd=0.5):
    """A whole number from lo to hi, spread over its logarithm; half of them multiples of 64 where there is room."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() >= odd and v >= 64:
        v -= v % 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "dispatch", "combine", "combine", "linear", "linear", "product"])
    c = {"op": op, "T": _spread(rng, 1, 65536, odd=0.7), "k": rng.randint(1, 8)}
    c["E"] = _spread(rng, c["k"], 256, odd=0.7)
    c["dropped"] = rng.choice([0.0, 0.0, 0.05, 0.3])
    if op == "sort":
        return c
    if op in ("dispatch", "combine"):
        c["direction"] = rng.choice(["forward", "backward"])
        c["H"] = _spread(rng, 64, 8192)
        c["dtype"] = rng.choice(["f32", "bf16", "f16"])
        c["T"] = max(1, min(c["T"], (1 << 28) // (c["k"] * c["H"])))
        return c
    c["K"], c["N"] = _spread(rng, 64, 8192), _spread(rng, 64, 8192)
    c["dtype"] = rng.choice(["bf16", "f16"])
    c["out"] = rng.choice(["bf16", "f16", "f32"])
    if op == "product" or rng.random() < 0.4:  # one matrix
        c["k"], c["E"], c["dropped"] = 1, 0, 0.0
    most = 1 << 37  # multiplications, half of the largest listed case's
    c["T"] = max(1, min(c["T"], 32768 // c["k"], most // (c["k"] * c["K"] * c["N"])))
    while c["E"] * c["K"] * c["N"] > 1 << 29:
        c["E"] = max(c["k"], c["E"] // 2)
        if c["E"] == c["k"]:
            c["K"], c["N"] = max(64, c["K"] // 2), max(64, c["N"] // 2)
    return c


# ------------------------------------------------------------------ inputs
def _route(c, g):
    """Expert ids as a router draws them: the k best of scores that favour some experts, a share of the slots routed
    nowhere (padding tokens, all k of them; single slots over an expert's capacity)."""
    favour = torch.randn(c["E"], generator=g, device="cuda")
    score = torch.randn(c["T"], c["E"], generator=g, device="cuda") + 0.7 * favour
    top = score.topk(c["k"], dim=1)
    ids = top.indices.to(torch.int32)
    if c["dropped"]:
        u = torch.rand(c["T"], c["k"], generator=g, device="cuda") < c["dropped"] / 2
        v = torch.rand(c["T"], 1, generator=g, device="cuda") < c["dropped"] / 2
        ids = torch.where(u | v, -1, ids)
    return ids.contiguous(), torch.softmax(top.values, 1).contiguous()


def _sorted(ids, E):
    """offsets [E + 1], src (sorted place -> slot), pos (slot -> sorted place) of a stable sort by expert."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    kept = (flat >= 0) & (flat < E)
    keys, order = torch.sort(torch.where(kept, flat, E), stable=True)
    offsets = torch.searchsorted(keys, torch.arange(E + 1, device=flat.device))
    place = torch.arange(n, device=flat.device)
    src = torch.where(place < offsets[E], order, -1)
    pos = torch.empty_like(order).scatter_(0, order, place)
    pos = torch.where(kept, pos, -1)
    return offsets.int(), src.int(), pos.int().reshape(ids.shape)


def _normal(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _codes(shape, g):
    """int8 values as a quantiser leaves them: a normal distribution whose largest value in a row is about 127."""
    return (torch.randn(shape, generator=g, device="cuda") * 34).round_().clamp_(-127, 127).to(torch.int8)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["E"]:
        s["ids"], w = _route(c, g)
        if c["op"] == "sort":
            return s
        s["offsets"], s["src"], s["pos"] = _sorted(s["ids"], c["E"])
    dt = DTYPES[c["dtype"]]
    S = c["T"] * c["k"]
    if c["op"] in ("dispatch", "combine"):
        if c["op"] == "combine":
            s["w"] = w
        if (c["op"] == "dispatch") == (c["direction"] == "forward"):  # token-ordered rows come in
            s["x"] = _normal((c["T"], c["H"]), g, dt)
            s["out"] = torch.zeros(S, c["H"], dtype=dt, device="cuda")  # a buffer that the program keeps
        if c["op"] == "combine" or c["direction"] == "backward":
            s["ys"] = _normal((S, c["H"]), g, dt)
        return s
    experts = max(c["E"], 1)
    s["x"] = _normal((c["T"], c["K"]), g, dt) if c["op"] == "linear" else _codes((c["T"], c["K"]), g)
    if c["op"] == "product":
        s["sx"] = torch.rand(c["T"], generator=g, device="cuda") * 0.02 + 0.02
    b = torch.empty(experts, c["N"], c["K"], dtype=torch.int8, device="cuda")
    for e in range(experts):
        b[e] = _codes((c["N"], c["K"]), g)
    sb = (torch.rand(experts, c["N"], generator=g, device="cuda") + 0.5) * (1.0 / (34 * math.sqrt(c["K"])))
    s["b"], s["sb"] = (b, sb) if c["E"] else (b[0], sb[0])
    s["out"] = torch.zeros(S, c["N"], dtype=DTYPES[c["out"]], device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _by_slot(rows, pos):
    """rows[pos] in 32 bits, zero where a slot is routed nowhere."""
    r = rows[pos.clamp_min(0).long()].float()
    return torch.where((pos >= 0).unsqueeze(-1), r, 0.0)


def _by_place(tokens, src, k):
    """The token's row (or weight) of every sorted place, zero behind the last routed one."""
    r = tokens[(src.clamp_min(0) // k).long()]
    return torch.where((src >= 0).reshape(-1, *[1] * (r.dim() - 1)), r, 0)


def _quantize(x):
    """Codes (whole numbers, held as float) and scales of every row."""
    x = x.float()
    a = x.abs().amax(1)
    bad = ~torch.isfinite(a)
    live = (a >= TINY) & ~bad
    # 127 x is exact in 32 bits for 16-bit inputs, so that halves round to even as they do in 64 bits
    q = (127.0 * x / torch.where(live, a, 1.0).unsqueeze(1)).round()
    q = torch.where(live.unsqueeze(1), q, 0.0)
    return q, torch.where(bad, float("nan"), torch.where(live, a / 127.0, 0.0))


def _plain_product(c, q, sq, s):
    if not c["E"]:
        return ((q @ s["b"].float().t()) * sq.unsqueeze(1) * s["sb"]).to(s["out"].dtype)
    # every expert's rows side by side, padded to the longest of them
    E, S = c["E"], s["src"].numel()
    offsets = s["offsets"].long()
    cap = int((offsets[1:] - offsets[:-1]).max())
    place = torch.arange(S, device=q.device)
    e = torch.searchsorted(offsets[1:].contiguous(), place, right=True)
    at = torch.where(e < E, e * cap + place - offsets[e.clamp_max(E)], E * cap)  # what is routed nowhere goes to one spare row
    row = (s["src"].clamp_min(0) // c["k"]).long()
    rows = torch.zeros(E * cap + 1, c["K"], device=q.device).index_copy_(0, at, q[row])
    y = torch.bmm(rows[:-1].view(E, cap, c["K"]), s["b"].float().transpose(1, 2))
    y = y.view(E * cap, c["N"])[at.clamp_max(max(E * cap - 1, 0))] * sq[row].unsqueeze(1) * s["sb"][e.clamp_max(E - 1)]
    return torch.where((e < E).unsqueeze(1), y, 0.0).to(s["out"].dtype)


def _run_plain(s):
    c = s["case"]
    op, back = c["op"], c.get("direction") == "backward"
    if op == "sort":
        return _sorted(s["ids"], c["E"])
    if op == "dispatch" and not back:
        return _by_place(s["x"], s["src"], c["k"])
    if op == "dispatch":
        return _by_slot(s["ys"], s["pos"]).sum(1).to(s["ys"].dtype)
    if op == "combine" and not back:
        return (s["w"].unsqueeze(-1) * _by_slot(s["ys"], s["pos"])).sum(1).to(s["ys"].dtype)
    if op == "combine":
        dys = _by_place(s["w"].reshape(-1, 1), s["src"], 1) * _by_place(s["x"].float(), s["src"], c["k"])
        dw = (s["x"].float().unsqueeze(1) * _by_slot(s["ys"], s["pos"])).sum(-1)
        return dys.to(s["ys"].dtype), dw
    if op == "product":
        return _plain_product(c, s["x"].float(), s["sx"], s)
    q, sq = _quantize(s["x"])
    return _plain_product(c, q, sq, s), sq


# ------------------------------------------------------------------ the framework's calls
def _run_own(s):
    import spmm_csr_spmv_amd as sp

    c = s["case"]
    op, back = c["op"], c.get("direction") == "backward"
    if op == "sort":
        return sp.moe_sort(s["ids"], c["E"])
    if op == "dispatch" and not back:
        return sp.moe_dispatch(s["x"], s["pos"], out=s["out"])
    if op == "dispatch":
        return sp.moe_combine(s["ys"], s["pos"])
    if op == "combine" and not back:
        return sp.moe_combine(s["ys"], s["pos"], s["w"])
    if op == "combine":
        return sp.moe_combine_backward(s["x"], s["ys"], s["pos"], s["w"], dYs=s["out"])
    if op == "product":
        return sp.gemm_i8(s["x"], s["sx"], s["b"], s["sb"], out=s["out"])
    q, sq = sp.quantize_rows_i8(s["x"])
    if c["E"]:
        y = sp.moe_gemm_i8(q, sq, s["b"], s["sb"], s["offsets"], src=s["src"], slots=c["k"], out=s["out"])
    else:
        y = sp.gemm_i8(q, sq, s["b"], s["sb"], out=s["out"])
    return y, sq


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ bytes and operations
def work(case):
    c = case
    n = c["T"] * c["k"]
    kept = n * (1.0 - c["dropped"] + c["dropped"] ** 2 / 4)
    if c["op"] == "sort":
        return {"bytes": 12 * n + 4 * (c["E"] + 1), "flops": n}
    b = BYTES[c["dtype"]]
    if c["op"] in ("dispatch", "combine"):
        rows, tokens = kept * c["H"], c["T"] * c["H"]
        weights = 4 * n if c["op"] == "combine" else 0
        if c["op"] == "combine" and c["direction"] == "backward":
            return {"bytes": (tokens + 2 * rows) * b + 4 * n + 2 * weights, "flops": 3 * rows}
        per_row = 0 if c["op"] == "dispatch" and c["direction"] == "forward" else 1 if c["op"] == "dispatch" else 2
        return {"bytes": (tokens + rows) * b + 4 * n + weights, "flops": per_row * rows}
    live = _used(c["E"], c["T"], c["k"]) if c["E"] else 1
    read = c["T"] * c["K"] * (b if c["op"] == "linear" else 1) + 4 * c["T"] + live * (c["N"] * c["K"] + 4 * c["N"])
    return {"bytes": read + kept * c["N"] * BYTES[c["out"]] + (4 * n if c["E"] else 0), "flops": 2 * kept * c["N"] * c["K"]}


def _used(E, T, k):
    """How many experts T tokens of k slots reach, about: only their weights have to be read."""
    return E * (1.0 - (1.0 - k / E) ** T)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    k, op, back = c["k"], c["op"], c.get("direction") == "backward"
    if op == "sort":
        flat = s["ids"].cpu().reshape(-1).tolist()
        lists = [[] for _ in range(c["E"])]
        for f, e in enumerate(flat):
            if 0 <= e < c["E"]:
                lists[e].append(f)
        src = [f for one in lists for f in one]
        pos = [-1] * len(flat)
        for p, f in enumerate(src):
            pos[f] = p
        offsets = [0]
        for one in lists:
            offsets.append(offsets[-1] + len(one))
        whole = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
        return whole(offsets), whole(src + [-1] * (len(flat) - len(src))), whole(pos).reshape(s["ids"].shape)
    if op in ("dispatch", "combine"):
        pos = s["pos"].long()
        rows = torch.zeros(pos.numel(), c["H"], dtype=torch.float64, device="cuda")
        tokens = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(c["T"], k, dtype=torch.float64, device="cuda")
        for j in range(k):  # slot by slot: the tokens whose slot j is routed somewhere
            t = (pos[:, j] >= 0).nonzero().reshape(-1)
            p = pos[t, j]
            w = s["w"][t, j].double().unsqueeze(1) if op == "combine" else 1.0
            if "x" in s:
                rows[p] = w * s["x"][t].double()
                if back:
                    dw[t, j] = torch.linalg.vecdot(s["x"][t].double(), s["ys"][p].double())
            else:
                tokens[t] += w * s["ys"][p].double()
        if op == "combine" and back:
            return rows, dw
        return rows if "x" in s else tokens
    x = s["x"].double()
    if op == "linear":
        a = x.abs().max(dim=1).values
        sq = a / 127
        x = torch.round(127 * x / a.clamp_min(TINY).unsqueeze(1))
    else:
        sq = s["sx"].double()
    y = torch.zeros(c["T"] * k, c["N"], dtype=torch.float64, device="cuda")
    if c["E"]:
        at = s["offsets"].tolist()
        for e in range(c["E"]):
            mine = torch.arange(at[e], at[e + 1], device="cuda")
            row = s["src"][mine].long() // k
            y[mine] = torch.matmul(x[row], s["b"][e].double().t()) * torch.outer(sq[row], s["sb"][e].double())
    else:
        y = torch.matmul(x, s["b"].double().t()) * torch.outer(sq, s["sb"].double())
    return y if op == "product" else (y, sq)
