"""Work of the microscaled 4-bit (MXFP4) layer and of the expert-order row operators.

Five operators of the Mixture-of-Experts layer, each as elementary torch
operations in fp32 (``own`` false) and as the library's calls (``own`` true):

* ``quantize``: rows to OCP MXFP4 and back to the values the codes stand for.
  A block of 32 consecutive values of a row shares the scale 2^s,
  s = floor(log2 max|v|) - 2 (at least -127); each value is v 2^-s rounded to
  the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6 (ties to the even code), at most 6.
* ``layer``: out[t] = sum_j w[t][j] W2[e_j] q(SiLU(W1g[e_j] q(x[t])) * (W1u[e_j] q(x[t])))
  with W1, W2 in MXFP4 and q the rounding above; a pair whose id is outside
  [0, E) adds nothing.
* ``dispatch``: xs[r] = w[p] x[p // k] at the sorted row r of every valid pair p
  (pairs in the stable order of their expert; w left out: 1); backward
  dx[t] = sum_j w[p] dxs[r], dw[p] = <dxs[r], x[t]>.
* ``combine``: out[t] = sum_j w[p] y[r]; backward dy[r] = w[p] dout[t],
  dw[p] = <y[r], dout[t]>.
* ``router_grad``: the gradient of the fp32 expert scores from that of the
  routing weights of a softmax top-k choice.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
#: (E, H, I, k, routing) of the layers this repository is configured for:
#: DeepSeek-V3-, Mixtral-8x7B-, Qwen3-30B-A3B- and Qwen2-57B-shaped (TP=4 slice)
LAYERS = {"dsv3": (256, 7168, 2048, 8, "even"), "mixtral": (8, 4096, 14336, 2, "even"),
          "qwen3": (128, 2048, 768, 8, "biased"), "qwen2": (64, 3584, 640, 8, "hot")}


def listed():
    return [
        # the activations of a decode batch, quantised and read back
        quantize_case(16, 7168, "bf16", name="quantize_bf16_16x7168"),
        # one-time quantisation of fp32 master weights: the gate and up rows of 32 experts
        quantize_case(131072, 7168, "fp32", name="quantize_fp32_131072x7168"),
        # one decode token: the weights of eight experts, every launch counts
        layer_case("dsv3", 1, name="layer_dsv3_T1"),
        # a small serving batch on many small experts, some idle
        layer_case("qwen3", 64, name="layer_qwen3_T64"),
        # prefill of few large experts: many rows per expert, bound by arithmetic
        layer_case("mixtral", 2048, name="layer_mixtral_T2048"),
        # prefill of many experts: every expert's weights once, 128 rows each
        layer_case("dsv3", 4096, name="layer_dsv3_T4096"),
        # a decode batch sent to its experts
        move_case("dispatch", "forward", 64, 8, 256, 7168, "bf16", False, 0.0, name="dispatch_bf16_T64"),
        # training: the gradient of fp32 rows weighted on the way in, some pairs dropped by capacity
        move_case("dispatch", "backward", 4096, 8, 64, 3584, "fp32", True, 0.05, name="dispatch_back_fp32_T4096"),
        # the largest batch of the routing build, back to token order
        move_case("combine", "forward", 8192, 8, 256, 7168, "bf16", True, 0.0, name="combine_bf16_T8192"),
        # training, odd sizes: gradients of the expert rows and of the routing weights
        move_case("combine", "backward", 777, 6, 61, 1000, "fp16", True, 0.02, name="combine_back_fp16_T777"),
        # the router's gradient of a small batch, weights renormalised over the chosen
        router_case(64, 64, 8, True, name="router_grad_T64_E64"),
        # ... and of the largest batch over the softmax of every expert
        router_case(8192, 256, 8, False, name="router_grad_T8192_E256"),
    ]


def quantize_case(rows, cols, kind, **more):
    return {"op": "quantize", "rows": rows, "cols": cols, "type": kind, **more}


def layer_case(shape, T, drop=0.0, **more):
    E, H, I, k, routing = LAYERS[shape]
    return {"op": "layer", "T": T, "E": E, "H": H, "I": I, "k": k, "routing": routing, "drop": drop, **more}


def move_case(op, way, T, k, E, H, kind, weighted, drop, **more):
    return {"op": op, "way": way, "T": T, "k": k, "E": E, "H": H, "type": kind, "weighted": weighted, "drop": drop,
            **more}


def router_case(T, E, k, renormalize, **more):
    return {"op": "router_grad", "T": T, "E": E, "k": k, "renormalize": renormalize, **more}


def spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(("quantize", "layer", "layer", "dispatch", "combine", "router_grad"))
    if op == "quantize":
        cols = 32 * spread(rng, 1, 448)
        return quantize_case(spread(rng, 1, min(131072, 131072 * 7168 // cols)), cols, rng.choice(("bf16", "fp16", "fp32")))
    if op == "layer":
        drop = rng.choice((0.0, 0.0, 0.1))
        if rng.random() < 0.5:
            name = rng.choice(tuple(LAYERS))
            return layer_case(name, spread(rng, 1, 2048 if name == "mixtral" else 4096), drop)
        E = rng.randint(1, 96)
        return {"op": "layer", "T": spread(rng, 1, 2048), "E": E, "H": 128 * rng.randint(1, 32), "I": 128 * rng.randint(1, 16),
                "k": rng.randint(1, min(E, 8)), "routing": rng.choice(("even", "biased", "hot")), "drop": drop}
    if op == "router_grad":
        E = rng.randint(2, 256)
        return router_case(spread(rng, 1, 8192), E, rng.randint(1, min(E, 16)), rng.random() < 0.5)
    k = rng.randint(1, 16)
    E = rng.randint(max(2, k), 256)
    T = spread(rng, 1, 8192 * 8 // max(k, 8))
    kind = rng.choice(("bf16", "fp16", "fp32"))
    H = 8 * spread(rng, 4, 896 if kind != "fp32" else 448)
    return move_case(op, rng.choice(("forward", "backward")), T, k, E, H, kind, rng.random() < 0.7,
                     rng.choice((0.0, 0.05, 0.5)))


# ---- inputs

def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def routes(g, T, k, E, routing, drop):
    """k distinct expert ids of every token, the highest of random scores
    first, and their softmax weights; `drop`: the share of pairs that are
    dropped (id -1)."""
    scores = normal(g, T, E)
    if routing == "biased":
        scores = scores + 1.5 * normal(g, E)
    if routing == "hot":
        scores[::2, 0] = 10.0
    top, ids = torch.topk(scores, k, dim=1)
    w = torch.softmax(torch.where(top > 9, top - 8, top), dim=1)
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < drop, -1, ids)
    return ids.to(torch.int32).contiguous(), w.contiguous()


def expert_order(ids, E):
    """The sorted row of every pair (dropped pairs last) and the number of valid pairs."""
    flat = ids.flatten().long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device="cuda")
    return pos, key < E


def weights(g, E, rows, cols):
    """N(0, 1/cols) weights in MXFP4, expert by expert: codes, two a byte, and scale codes."""
    codes = torch.empty(E, rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, rows, cols // 32, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (rows * cols))
    for e in range(0, E, step):
        n = min(step, E - e)
        codes[e:e + n], scales[e:e + n] = encode(normal(g, n, rows, cols) / math.sqrt(cols))
    return codes, scales


def prepare(case, seed):
    g = generator(seed)
    op = case["op"]
    st = dict(case)
    if op == "quantize":
        # rows of differing magnitude, with a few large values, as hidden states have
        x = normal(g, case["rows"], case["cols"])
        x *= torch.exp(normal(g, case["rows"], 1))
        x *= torch.where(torch.rand(case["cols"], generator=g, device="cuda") < 0.002, 30.0, 1.0)
        st["x"] = x.to(TYPES[case["type"]])
        return st
    T, k, E = case["T"], case["k"], case["E"]
    if op == "router_grad":
        st["logits"] = normal(g, T, E)
        top, ids = torch.topk(st["logits"], k, dim=1)
        lse = 0.0 if case["renormalize"] else torch.logsumexp(st["logits"], 1, keepdim=True)
        st["w"] = torch.softmax(top, 1) if case["renormalize"] else torch.exp(top - lse)
        st["ids"], st["dw"] = ids.to(torch.int32).contiguous(), normal(g, T, k)
        return st
    st["ids"], st["w"] = routes(g, T, k, E, case.get("routing", "even"), case["drop"])
    H = case["H"]
    if op == "layer":
        st["x"] = normal(g, T, H).to(torch.bfloat16)
        w1 = weights(g, E, 2 * case["I"], H)
        w2 = weights(g, E, H, case["I"])
        if own:   # packed once, when weights are loaded; the buffers are kept from call to call
            import mixture_experts_layer_lds_amd as moe
            st["weights"] = moe.pack_weights({"w1": w1[0], "w1_scale": w1[1], "w2": w2[0], "w2_scale": w2[1]}, "mxfp4")
            st["routing"] = moe.alloc_routing(T, k, E, H, case["I"], "mxfp4")
            st["workspace"] = moe.alloc_workspace(T, k, E, H, case["I"], "mxfp4")
            st["out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        else:
            st["w1"], st["w2"] = w1, w2
            # rows that the busiest expert gets: the plain form's batch height
            flat = st["ids"].flatten()
            st["height"] = int(torch.bincount(flat[flat >= 0].long(), minlength=E).max()) if (flat >= 0).any() else 0
        return st
    # rows in token order and in expert order; a step has its routing from the layer
    kind = TYPES[case["type"]]
    st["tokens"] = normal(g, T, H).to(kind)
    pos, valid = expert_order(st["ids"], E)
    if op == "combine" or case["way"] == "backward":
        st["rows"] = normal(g, T * k, H).to(kind)
    if own:
        import mixture_experts_layer_lds_amd as moe
        st["routing"] = moe.alloc_routing(T, k, E, 64, 64, "bf16")
        moe.moe_build_routing_bf16(st["ids"], E, 64, 64, st["routing"])
    else:
        st["pos"], st["valid"] = pos, valid
    if (op == "dispatch") == (case["way"] == "forward"):
        st["out"] = torch.zeros(T * k, H, dtype=kind, device="cuda")   # rows behind the last valid pair stay
    return st


def two_to(e):
    """2^e in fp64, from its bits: exact, for whole e of [-1022, 1023]."""
    return ((e.long() + 1023) << 52).view(torch.float64)


# ---- the plain forms

def block_scales(v):
    """2^s of every 32-value block of fp32 v, as a float and as its e8m0 code."""
    top = v.unflatten(-1, (-1, 32)).abs().amax(-1)
    s = (torch.floor(torch.frexp(top).exponent.float()) - 1 - 2).clamp(min=-127)
    s = torch.where(top > 0, s, -127.0)
    return two_to(s).float(), (s + 127).to(torch.uint8)


def rounded(v):
    """fp32 v rounded to MXFP4: the values, 2^s of every block, its code, and the values over 2^s."""
    scale, code = block_scales(v)
    u = v.unflatten(-1, (-1, 32)) / scale.unsqueeze(-1)
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    u = torch.copysign((torch.round(a / step) * step).clamp(max=6.0), u)
    return (u * scale.unsqueeze(-1)).flatten(-2), scale, code, u.flatten(-2)


def encode(v):
    """MXFP4 codes, two a byte (the lower column in the low nibble), and scale codes of fp32 v."""
    _, _, code, u = rounded(v)
    a = u.abs()
    m = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = m | (torch.signbit(u).to(torch.uint8) << 3)
    return c[..., 0::2] | (c[..., 1::2] << 4), code


def decode(codes, scales):
    """fp32 values of MXFP4 codes."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    m = (c & 7).to(torch.bfloat16)   # small whole and half numbers: exact
    m = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    m = torch.where(c > 7, -m, m).float()
    s = two_to(scales.int() - 127).float()
    return (m.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def plain_layer(st):
    T, k, E, H, I = st["T"], st["k"], st["E"], st["H"], st["I"]
    xq = rounded(st["x"].float())[0]
    P = T * k
    ids = st["ids"].flatten().long()
    valid = (ids >= 0) & (ids < E)
    token = torch.arange(T, device="cuda").repeat_interleave(k)
    if P <= E:   # every pair with its own expert's weights
        batch, row, height, pick = torch.arange(P, device="cuda"), torch.zeros(P, dtype=torch.long, device="cuda"), 1, ids.clamp(min=0)
        at = [tuple(t.index_select(0, pick) for t in st[n]) for n in ("w1", "w2")]
    else:        # every expert with its rows, as many as the busiest has
        pos, _ = expert_order(st["ids"], E)
        batch = torch.where(valid, ids, 0)
        count = torch.zeros(E + 1, dtype=torch.long, device="cuda").scatter_add_(0, torch.where(valid, ids, E), torch.ones_like(ids))
        row = torch.where(valid, pos - (torch.cumsum(count, 0) - count)[batch], 0)
        height, at = max(1, st["height"]), [st["w1"], st["w2"]]
    n = at[0][0].shape[0]
    a = torch.zeros(n, height, H, device="cuda")
    a.index_put_((batch, row), torch.where(valid.unsqueeze(1), xq[token], 0.0), accumulate=True)
    gu = torch.bmm(decode(*at[0]), a.transpose(1, 2).contiguous())
    g, u = gu[:, :I], gu[:, I:]
    h = (g / (1 + torch.exp(-g)) * u).transpose(1, 2).contiguous()
    hq = rounded(h)[0].transpose(1, 2).contiguous()
    y = torch.bmm(decode(*at[1]), hq)
    rows = y.transpose(1, 2)[batch, row] * torch.where(valid, st["w"].flatten(), 0.0).unsqueeze(1)
    return rows.view(T, k, H).sum(1).to(torch.bfloat16)


def plain_move(st):
    T, k, H = st["T"], st["k"], st["H"]
    kind = TYPES[st["type"]]
    w = st["w"].flatten() if st["weighted"] else torch.ones(T * k, device="cuda")
    token = torch.arange(T, device="cuda").repeat_interleave(k)
    valid, pos = st["valid"], st["pos"]
    if (st["op"] == "dispatch") == (st["way"] == "forward"):   # token rows to expert order
        out = st["out"]
        out[pos] = torch.where(valid.unsqueeze(1), st["tokens"].float()[token] * w.unsqueeze(1), 0.0).to(kind)
        moved = out
    else:                                                      # expert rows to token order
        take = torch.where(valid.unsqueeze(1), st["rows"].float()[pos] * w.unsqueeze(1), 0.0)
        moved = take.view(T, k, H).sum(1).to(kind)
    if st["way"] == "forward":
        return moved
    if not st["weighted"]:
        return moved
    dw = (st["rows"].float()[pos] * st["tokens"].float()[token]).sum(1)
    return moved, torch.where(valid, dw, 0.0).view(T, k)


def plain_router(st):
    w, dw, ids = st["w"], st["dw"], st["ids"].long()
    s = (w * dw).sum(1, keepdim=True)
    if st["renormalize"]:
        return torch.zeros_like(st["logits"]).scatter_add_(1, ids, w * (dw - s))
    e = torch.exp(st["logits"] - st["logits"].amax(1, keepdim=True))
    return (-(e / e.sum(1, keepdim=True)) * s).scatter_add_(1, ids, w * dw)


def run(st):
    op = st["op"]
    if not own:
        if op == "quantize":
            return rounded(st["x"].float())[0].to(st["x"].dtype)
        return {"layer": plain_layer, "router_grad": plain_router}.get(op, plain_move)(st)
    import mixture_experts_layer_lds_amd as moe
    if op == "quantize":
        codes, scales = moe.moe_quantize_mxfp4(st["x"])
        return moe.moe_dequantize_mxfp4(codes, scales, st["x"].dtype)
    if op == "layer":
        return moe.route_forward(st["ids"], st["x"], st["w"], st["routing"], st["weights"], st["workspace"], st["out"], "mxfp4")
    if op == "router_grad":
        return moe.moe_router_topk_grad(st["logits"], st["ids"], st["w"], st["dw"], renormalize=st["renormalize"])
    w = st["w"] if st["weighted"] else None
    k, E = st["k"], st["E"]
    if op == "dispatch":
        if st["way"] == "forward":
            return moe.moe_dispatch(st["tokens"], st["routing"], k, E, topk_w=w, out=st["out"])
        return moe.moe_dispatch_grad(st["rows"], st["routing"], k, E, x=st["tokens"] if st["weighted"] else None, topk_w=w)
    if st["way"] == "forward":
        return moe.moe_combine(st["rows"], st["routing"], k, E, topk_w=w)
    return moe.moe_combine_grad(st["tokens"], st["routing"], k, E, y=st["rows"] if st["weighted"] else None, topk_w=w, dy=st["out"])


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * BYTES[case["type"]] * n, "flops": 4 * n}
    T, k, E = case["T"], case["k"], case["E"]
    if op == "router_grad":
        both = 1 if case["renormalize"] else 2
        return {"bytes": 4 * T * E * both + 12 * T * k, "flops": (6 if both == 2 else 1) * T * E + 4 * T * k}
    H = case["H"]
    P = round(T * k * (1 - case["drop"]))
    if op == "layer":
        # experts that get a row (the expected number of an even choice), their weights once
        active = min(P, E * (1 - (1 - k / E) ** (T * (1 - case["drop"]))) if k < E else E)
        return {"bytes": round(active * 3 * H * case["I"] * 17 / 32) + 4 * T * H + 8 * T * k, "flops": 6 * P * H * case["I"]}
    b = BYTES[case["type"]]
    total, flops = b * H * (T + P) + 4 * T * k, 2 * P * H
    if case["weighted"]:
        total += 4 * T * k
        if case["way"] == "backward":
            total, flops = total + 4 * T * k + b * H * (T if case["op"] == "dispatch" else P), 2 * flops
    return {"bytes": total, "flops": flops}


# ---- the definition in 64 bits

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def nearest(v):
    """fp64 v rounded to MXFP4 by comparison with the borders between neighbours: a border itself
    goes to the neighbour of even code."""
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
    border = (grid[1:] + grid[:-1]) / 2
    b = v.reshape(-1, 32)
    top = b.abs().amax(1, keepdim=True)
    _, e = torch.frexp(top)
    e = torch.where(top > 0, (e - 3).clamp(min=-127), -127)
    a = b.abs() * two_to(-e)
    low, high = torch.bucketize(a, border), torch.bucketize(a, border, right=True)
    code = torch.where(low % 2 == 0, low, high)
    return torch.copysign(grid[code] * two_to(e), b).view(v.shape)


def values(codes, scales):
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
    table = torch.cat((grid, -grid))
    both = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).flatten(-2)
    return both * two_to(scales.int() - 127).repeat_interleave(32, -1)


def exact_layer(case, seed):
    g = generator(seed)
    T, k, E, H, I = (case[n] for n in ("T", "k", "E", "H", "I"))
    ids, w = routes(g, T, k, E, case["routing"], case["drop"])
    x = nearest(normal(g, T, H).to(torch.bfloat16).double())
    w1, w2 = weights(g, E, 2 * I, H), weights(g, E, H, I)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            gu = x[t] @ values(w1[0][e], w1[1][e]).t()
            h = nearest(gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:])
            out.index_add_(0, t, (h @ values(w2[0][e], w2[1][e]).t()) * w[t, j].double().unsqueeze(1))
    return out


def exact(case, seed):
    op = case["op"]
    if op == "layer":
        return exact_layer(case, seed)
    if op == "quantize":
        x = prepare(case, seed)["x"]
        step = max(1, (1 << 26) // case["cols"])
        return torch.cat([nearest(x[r:r + step].double()) for r in range(0, case["rows"], step)])
    st = prepare(case, seed)
    T, k, E = case["T"], case["k"], case["E"]
    w = st["w"].double()
    if op == "router_grad":
        dw = st["dw"].double()
        chosen = torch.zeros(T, E, dtype=torch.bool, device="cuda").scatter_(1, st["ids"].long(), True)
        up = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, st["ids"].long(), dw)
        l = st["logits"].double()
        p = torch.softmax(l.masked_fill(~chosen, -math.inf) if case["renormalize"] else l, 1)
        return p * (up - (p * up).sum(1, keepdim=True))
    H = case["H"]
    pos, valid = expert_order(st["ids"], E)
    pos, valid = pos.view(T, k), valid.view(T, k)
    scale = (w if case["weighted"] else torch.ones_like(w)) * valid
    tokens = st["tokens"].double()
    if (op == "dispatch") == (case["way"] == "forward"):
        moved = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            moved[pos[:, j]] = tokens * scale[:, j:j + 1]
    else:
        moved = sum(st["rows"][pos[:, j]].double() * scale[:, j:j + 1] for j in range(k))
    if case["way"] == "forward" or not case["weighted"]:
        return moved
    dw = torch.stack([(st["rows"][pos[:, j]].double() * tokens).sum(1) for j in range(k)], 1)
    return moved, dw * valid
