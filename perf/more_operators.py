"""Work of the experts' products over rows in expert order, and of their gradients.

Four operators, each over rows grouped by expert (``E`` > 0: row r of the
expert-sorted order belongs to the expert whose range holds it, rows behind the
last valid pair stay as they are) or over plain rows with one matrix (``E`` = 0:
a shared expert), each as elementary torch operations in fp32 (``own`` false)
and as the library's calls (``own`` true):

* ``linear``: z[r] = W[e] x[r] + b[e], y[r] = residual[r] + act(z[r]); act is none, SiLU, GELU (z times the
  normal distribution function) or SwiGLU: SiLU(z[m]) z[M + m] with N = 2 M.  z is an output where it is kept for the
  backward pass.
* ``grad_x``: d[r] = dy[r] W[e]; with the pre-activation z of the product before, dz = d act'(z) in its place.
* ``grad_w``: dW[e] = sum over the expert's rows of dy[r] x[r]^T, db[e] = sum of dy[r]; zero for an expert without rows.
* ``act_grad``: dz = dy act'(z).
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
#: (E, H, I, k, routing) of the layers this repository is configured for: DeepSeek-V3- (a GPU's 32 of the
#: 256 experts, eight-way expert parallel), Mixtral-8x7B-, Qwen3-30B-A3B- and Qwen2-57B-shaped (TP=4 slice)
LAYERS = {"dsv3": (32, 7168, 2048, 8, "even"), "mixtral": (8, 4096, 14336, 2, "even"),
          "qwen3": (128, 2048, 768, 8, "biased"), "qwen2": (64, 3584, 640, 8, "hot")}
MOST = 2 * 8192 * 28672 * 4096   # operations of the largest listed case


def listed():
    return [
        # one decode token through the shared expert's gate and up rows: the weights' read, latency
        linear_case(dense(1), 4096, 7168, "bf16", "swiglu", name="linear_bf16_1_shared_up"),
        # a small serving batch on many small experts, some idle
        linear_case(layer("qwen3", 64), 1536, 2048, "bf16", "swiglu", name="linear_bf16_qwen3_T64_up"),
        # training, few large experts: gate-up with its sums kept for the backward pass
        linear_case(layer("mixtral", 4096), 28672, 4096, "bf16", "swiglu", keep=True, name="linear_bf16_mixtral_T4096_up"),
        # the down product of many experts, 256 rows each on average
        linear_case(layer("dsv3", 1024), 7168, 2048, "bf16", "none", name="linear_bf16_dsv3_T1024_down"),
        # a dense layer of odd sizes with everything its epilogue can do
        linear_case(dense(1234), 1000, 1048, "fp16", "gelu", bias=True, residual=True, keep=True, name="linear_fp16_1234_gelu"),
        # backward through the down product and the SwiGLU before it
        grad_x_case(layer("qwen2", 4096), 3584, 640, "bf16", "swiglu", name="grad_x_bf16_qwen2_T4096_down_swiglu"),
        # ... and through the gate-up product to the dispatched rows
        grad_x_case(layer("dsv3", 1024), 4096, 7168, "bf16", "none", name="grad_x_bf16_dsv3_T1024_up"),
        # gradient of large weights in fp32, as an optimizer of fp32 master weights takes it
        grad_w_case(layer("mixtral", 2048), 28672, 4096, "bf16", "fp32", name="grad_w_bf16_mixtral_T2048_up"),
        # odd and ragged: 61 experts, some pairs dropped by capacity, biases
        grad_w_case(groups(777, 6, 61, "biased", 0.02), 1000, 520, "fp16", "fp16", bias=True, name="grad_w_fp16_777_odd"),
        # the shared expert's down weights over a whole batch
        grad_w_case(dense(8192), 7168, 2048, "bf16", "bf16", name="grad_w_bf16_8192_shared_down"),
        # gradient of the activation by itself, where no product follows it
        act_case(layer("qwen2", 4096), 640, "bf16", "swiglu", name="act_grad_bf16_qwen2_T4096"),
        # ... of a small dense batch
        act_case(dense(100), 1000, "fp16", "gelu", name="act_grad_fp16_100x1000"),
    ]


def dense(rows):
    return {"T": rows, "k": 1, "E": 0, "routing": "", "drop": 0.0}


def groups(T, k, E, routing, drop=0.0):
    return {"T": T, "k": k, "E": E, "routing": routing, "drop": drop}


def layer(shape, T, drop=0.0):
    E, _, _, k, routing = LAYERS[shape]
    return groups(T, k, E, routing, drop)


def linear_case(rows, N, K, kind, act, bias=False, residual=False, keep=False, **more):
    return {"op": "linear", **rows, "N": N, "K": K, "type": kind, "act": act, "bias": bias, "residual": residual,
            "keep": keep, **more}


def grad_x_case(rows, N, K, kind, act, **more):
    return {"op": "grad_x", **rows, "N": N, "K": K, "type": kind, "act": act, **more}


def grad_w_case(rows, N, K, kind, out, bias=False, **more):
    return {"op": "grad_w", **rows, "N": N, "K": K, "type": kind, "out": out, "bias": bias, **more}


def act_case(rows, M, kind, act, **more):
    return {"op": "act_grad", **rows, "M": M, "type": kind, "act": act, **more}


def spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "grad_x", "grad_w", "act_grad"))
    kind = rng.choice(("bf16", "fp16"))
    act = rng.choice(("none", "silu", "gelu", "swiglu"))
    yes = lambda: rng.random() < 0.3
    if rng.random() < 0.5:     # a product of one of the layers, gate-up or down
        name = rng.choice(tuple(LAYERS))
        E, H, I, k, routing = LAYERS[name]
        up = rng.random() < 0.5
        N, K = (2 * I, H) if up else (H, I)
        if up == (op == "linear"):
            act = "swiglu"
        most = min(8192, MOST // (2 * k * N * K))
        rows = layer(name, spread(rng, 1, most), rng.choice((0.0, 0.0, 0.1)))
    else:
        N, K = 16 * spread(rng, 2, 512), 8 * spread(rng, 4, 1024)
        if rng.random() < 0.4:
            rows = dense(spread(rng, 1, 16384))
        else:
            E = rng.randint(1, 96)
            k = rng.randint(1, min(E, 8))
            rows = groups(spread(rng, 1, 4096), k, E, rng.choice(("even", "biased", "hot")), rng.choice((0.0, 0.05, 0.5)))
            while E * N * K > 1 << 30:   # experts of the largest listed case hold about as much
                N, K = max(32, N // 32 * 16), max(32, K // 16 * 8)
    if op == "linear":
        return linear_case(rows, N, K, kind, act, bias=yes(), residual=yes(), keep=yes())
    if op == "grad_x":
        return grad_x_case(rows, N, K, kind, act)
    if op == "grad_w":
        return grad_w_case(rows, N, K, kind, rng.choice((kind, "fp32")), bias=yes())
    return act_case(rows, K, kind, "gelu" if act == "none" else act)


# ---- inputs

def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def routes(g, T, k, E, routing, drop):
    """k distinct expert ids of every token, the highest of random scores first; `drop`: the share of
    pairs that are dropped (id -1)."""
    scores = normal(g, T, E)
    if routing == "biased":
        scores = scores + 1.5 * normal(g, E)
    if routing == "hot":
        scores[::2, 0] = 10.0
    ids = torch.topk(scores, k, dim=1).indices
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < drop, -1, ids)
    return ids.to(torch.int32).contiguous()


def ranges(ids, E):
    """Where each expert's rows begin in expert order, and where the last one's end."""
    flat = ids.flatten().long()
    count = torch.bincount(flat[flat >= 0], minlength=E)
    return [0] + torch.cumsum(count, 0).tolist()


def matrices(g, case, kind):
    """N(0, 1/K) weights, matrix by matrix."""
    E, N, K = max(1, case["E"]), case["N"], case["K"]
    w = torch.empty(E, N, K, dtype=kind, device="cuda")
    for e in range(E):
        w[e] = normal(g, N, K) / math.sqrt(K)
    return w if case["E"] else w[0]


def prepare(case, seed):
    g = generator(seed)
    st = dict(case)
    T, k, E, op, act = case["T"], case["k"], case["E"], case["op"], case.get("act")
    R, kind = T * k, TYPES[case["type"]]
    if E:
        ids = routes(g, T, k, E, case["routing"], case["drop"])
        if own:   # a layer has its routing from the step before
            import mixture_experts_layer_lds_amd as moe
            st["routing"] = moe.alloc_routing(T, k, E, 64, 64, "bf16")
            moe.moe_build_routing_bf16(ids, E, 64, 64, st["routing"])
        else:
            st["ranges"] = ranges(ids, E)
    else:
        st["ranges"] = [0, R]
    new = lambda cols, t=kind: torch.zeros(R, cols, dtype=t, device="cuda")   # buffers that are kept from call to call
    if op == "linear":
        st["x"] = normal(g, R, case["K"]).to(kind)
        st["w"] = matrices(g, case, kind)
        M = case["N"] // 2 if act == "swiglu" else case["N"]
        if case["bias"]:
            st["b"] = (0.5 * normal(g, max(1, E), case["N"])).to(kind)
            st["b"] = st["b"] if E else st["b"][0]
        if case["residual"]:
            st["r"] = normal(g, R, M).to(kind)
        st["y"] = new(M)
        if case["keep"]:
            st["z"] = new(case["N"])
    elif op == "grad_x":
        st["dy"] = normal(g, R, case["N"]).to(kind)
        st["w"] = matrices(g, case, kind)
        Z = case["K"] * (2 if act == "swiglu" else 1)
        if act != "none":
            st["z"] = normal(g, R, Z).to(kind)
        st["dx"] = new(Z)
    elif op == "grad_w":
        st["dy"], st["x"] = normal(g, R, case["N"]).to(kind), normal(g, R, case["K"]).to(kind)
        shape = (E, case["N"], case["K"]) if E else (case["N"], case["K"])
        st["dw"] = torch.empty(shape, dtype=TYPES[case["out"]], device="cuda")
        if case["bias"]:
            st["db"] = torch.empty(shape[:-1], dtype=TYPES[case["out"]], device="cuda")
    else:
        Z = case["M"] * (2 if act == "swiglu" else 1)
        st["dy"], st["z"] = normal(g, R, case["M"]).to(kind), normal(g, R, Z).to(kind)
        st["dz"] = new(Z)
    return st


# ---- the plain forms

def sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def phi(z):
    return 0.5 * torch.erfc(z * -math.sqrt(0.5))


def activated(z, act):
    if act == "none":
        return z
    if act == "gelu":
        return z * phi(z)
    if act == "silu":
        return z * sigmoid(z)
    M = z.shape[1] // 2
    return z[:, :M] * sigmoid(z[:, :M]) * z[:, M:]


def back(d, z, act):
    """d times the derivative of the activation at z."""
    if act == "none":
        return d
    if act == "gelu":
        return d * (phi(z) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    M = z.shape[1] // 2 if act == "swiglu" else z.shape[1]
    g = z[:, :M]
    s = sigmoid(g)
    slope = s * (1 + g * (1 - s))
    if act == "silu":
        return d * slope
    return torch.cat((d * z[:, M:] * slope, d * g * s), 1)


def spans(st):
    """(expert, first row, row behind the last) of every expert that has rows."""
    r = st["ranges"]
    return [(e, r[e], r[e + 1]) for e in range(len(r) - 1) if r[e + 1] > r[e]]


def of(t, st, e):
    """The matrix or vector of expert e; of plain rows, the one there is."""
    return (t[e] if st["E"] else t).float()


def plain_linear(st):
    y, z = st["y"], st.get("z")
    for e, a, b in spans(st):
        s = st["x"][a:b].float() @ of(st["w"], st, e).t()
        if "b" in st:
            s = s + of(st["b"], st, e)
        out = activated(s, st["act"])
        if "r" in st:
            out = out + st["r"][a:b].float()
        y[a:b] = out.to(y.dtype)
        if z is not None:
            z[a:b] = s.to(z.dtype)
    return y if z is None else (y, z)


def plain_grad_x(st):
    dx = st["dx"]
    for e, a, b in spans(st):
        d = st["dy"][a:b].float() @ of(st["w"], st, e)
        dx[a:b] = back(d, st["z"][a:b].float() if "z" in st else None, st["act"]).to(dx.dtype)
    return dx


def plain_grad_w(st):
    dw, db, r = st["dw"], st.get("db"), st["ranges"]
    for e in range(len(r) - 1):
        dy = st["dy"][r[e]:r[e + 1]].float()
        (dw[e] if st["E"] else dw).copy_(dy.t() @ st["x"][r[e]:r[e + 1]].float())
        if db is not None:
            (db[e] if st["E"] else db).copy_(dy.sum(0))
    return dw if db is None else (dw, db)


def plain_act_grad(st):
    n, dz = st["ranges"][-1], st["dz"]
    dz[:n] = back(st["dy"][:n].float(), st["z"][:n].float(), st["act"]).to(dz.dtype)
    return dz


def run(st):
    op, E = st["op"], st["E"]
    if not own:
        return {"linear": plain_linear, "grad_x": plain_grad_x, "grad_w": plain_grad_w, "act_grad": plain_act_grad}[op](st)
    import mixture_experts_layer_lds_amd as moe
    if op == "linear":
        more = {"bias": st.get("b"), "act": st["act"], "residual": st.get("r"), "z": st.get("z"), "out": st["y"]}
        if E:
            return moe.moe_grouped_linear(st["x"], st["w"], st["routing"], st["k"], **more)
        return moe.moe_linear(st["x"], st["w"], **more)
    if op == "grad_x":
        more = {"z": st.get("z"), "act": st["act"], "dx": st["dx"]}
        if E:
            return moe.moe_grouped_linear_grad_x(st["dy"], st["w"], st["routing"], st["k"], **more)
        return moe.moe_linear_grad_x(st["dy"], st["w"], **more)
    if op == "grad_w":
        more = {"dw": st["dw"], "dbias": st.get("db")}
        if E:
            return moe.moe_grouped_linear_grad_w(st["dy"], st["x"], st["routing"], st["k"], E, **more)
        return moe.moe_linear_grad_w(st["dy"], st["x"], **more)
    if E:
        return moe.moe_grouped_act_grad(st["dy"], st["z"], st["routing"], st["k"], E, st["act"], dz=st["dz"])
    return moe.moe_act_grad(st["dy"], st["z"], st["act"], dz=st["dz"])


def work(case):
    op, T, k, E, act = case["op"], case["T"], case["k"], case["E"], case.get("act")
    R = round(T * k * (1 - case["drop"]))
    b = BYTES[case["type"]]
    both = 2 if act == "swiglu" else 1
    if op == "act_grad":
        return {"bytes": b * R * case["M"] * (1 + 2 * both), "flops": 10 * R * case["M"]}
    N, K = case["N"], case["K"]
    flops = 2 * R * N * K
    # experts that get a row (the expected number of an even choice): their weights once
    active = 1 if not E else min(R, E * (1 - (1 - k / E) ** (T * (1 - case["drop"])))) if k < E else E
    weights = round(b * active * N * K)
    if op == "linear":
        total = weights + b * R * (K + N // both) + (b * R * N if case["keep"] else 0)
        total += (b * R * N // both if case["residual"] else 0) + (round(b * active * N) if case["bias"] else 0)
    elif op == "grad_x":
        total = weights + b * R * (N + K * both) + (b * R * K * both if act != "none" else 0)
    else:
        total = b * R * (N + K) + BYTES[case["out"]] * max(1, E) * N * (K + (1 if case["bias"] else 0))
    return {"bytes": total, "flops": flops}


# ---- the definition in 64 bits

def value(z, act):
    if act == "swiglu":
        gate, up = z.chunk(2, dim=1)
        return torch.sigmoid(gate) * gate * up
    return {"none": lambda: z, "silu": lambda: torch.sigmoid(z) * z, "gelu": lambda: torch.special.ndtr(z) * z}[act]()


def slope(z, act):
    """The derivative of z sigma(z), sigma the logistic or the normal distribution function."""
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    return torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)


def upstream(d, z, act):
    if act == "none":
        return d
    if act == "swiglu":
        gate, up = z.double().chunk(2, dim=1)
        return torch.cat((slope(gate, "silu") * up * d, value(gate, "silu") * d), dim=1)
    return slope(z.double(), act) * d


def exact(case, seed):
    st = prepare(case, seed)
    op, E, act = case["op"], case["E"], case.get("act")
    if E:
        g = generator(seed)
        begin = ranges(routes(g, case["T"], case["k"], E, case["routing"], case["drop"]), E)
    else:
        begin = [0, case["T"]]
    n = begin[-1]
    wide = lambda name: torch.zeros(st[name].shape, dtype=torch.float64, device="cuda")
    if op == "act_grad":
        dz = wide("dz")
        dz[:n] = upstream(st["dy"][:n].double(), st["z"][:n], act)
        return dz
    parts = [(e, slice(begin[e], begin[e + 1])) for e in range(max(1, E)) if begin[e + 1] > begin[e]]
    pick = lambda name, e: (st[name][e] if E else st[name]).double()
    if op == "linear":
        y, z = wide("y"), torch.zeros(case["T"] * case["k"], case["N"], dtype=torch.float64, device="cuda")
        for e, rows in parts:
            z[rows] = torch.mm(pick("w", e), st["x"][rows].double().t()).t()
            if case["bias"]:
                z[rows] += pick("b", e)
        y[:n] = value(z[:n], act)
        if case["residual"]:
            y[:n] += st["r"][:n].double()
        return (y, z) if case["keep"] else y
    if op == "grad_x":
        dx = wide("dx")
        for e, rows in parts:
            d = torch.mm(pick("w", e).t(), st["dy"][rows].double().t()).t()
            dx[rows] = upstream(d, st["z"][rows] if act != "none" else None, act)
        return dx
    dw = wide("dw")
    db = torch.zeros(dw.shape[:-1], dtype=torch.float64, device="cuda")
    for e, rows in parts:
        dy = st["dy"][rows].double()
        product, total = torch.mm(st["x"][rows].double().t(), dy).t(), dy.t() @ torch.ones(dy.shape[0], dtype=torch.float64, device="cuda")
        if E:
            dw[e], db[e] = product, total
        else:
            dw[:], db[:] = product, total
    return (dw, db) if case["bias"] else dw
