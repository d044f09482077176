"""The mixture-of-experts and MXFP4 operators: what is measured, and their plain forms.

Five operators, by the `op` of a case:

  route     the router: top-k experts of every token, their weights, and the
            plan that groups the (token, choice) slots by expert; with `train`
            also the weighted sum of the experts' rows, its gradients and the
            router's
  moe       the gated MLP over sharded experts, its ragged products grouped by
            expert (gate|up with SwiGLU, down, the weighted sum over a token's
            experts)
  backward  the gradients of one grouped layer (input rows and weights), the
            SwiGLU gradient ahead of it for the gate|up layer
  quantize  values to MXFP4 (E2M1 codes, one E8M0 scale for 32 inputs) and back
  mxfp4     products with MXFP4 experts: the gated MLP on 16-bit activations
            (`acts` 16), or one gate|up layer on MXFP4 activations (`acts` 4)

`own` False computes them in elementary torch operations in 32 bits, rounded
once at the end; True calls the package's entry points.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one decoding step's routing for a small batch: launch latency is all there is
        {"name": "route-decode", "op": "route", "train": False, "T": 8, "E": 64, "k": 8, "D": 0, "dtype": "f32",
         "normalize": True, "masked": False},
        # a training step's routing: many tokens, masked experts, padded tokens, gradients
        {"name": "route-train", "op": "route", "train": True, "T": 8192, "E": 128, "k": 8, "D": 2048, "dtype": "bf16",
         "normalize": False, "masked": True},
        # one token through eight experts of the decode MLP's shape
        {"name": "moe-token", "op": "moe", "T": 1, "E": 8, "k": 2, "D": 4096, "F": 14336, "P": 8, "dtype": "bf16",
         "masked": False},
        # a decoding batch over many small experts: a few rows for each
        {"name": "moe-decode", "op": "moe", "T": 32, "E": 64, "k": 4, "D": 2048, "F": 1024, "P": 4, "dtype": "f16",
         "masked": False},
        # the prefill's tokens over eight experts of the MLP's shape
        {"name": "moe-prefill", "op": "moe", "T": 4096, "E": 8, "k": 2, "D": 4096, "F": 14336, "P": 4, "dtype": "bf16",
         "masked": False},
        # sizes that fill no tile, on padded batches
        {"name": "moe-odd", "op": "moe", "T": 777, "E": 20, "k": 3, "D": 1000, "F": 726, "P": 2, "dtype": "bf16",
         "masked": True},
        # gradients of the gate|up layer of the prefill's tokens
        {"name": "backward-column", "op": "backward", "mode": "column", "T": 4096, "E": 8, "k": 2, "D": 4096,
         "F": 14336, "P": 4, "dtype": "bf16"},
        # gradients of the down layer over many small experts, ragged
        {"name": "backward-row", "op": "backward", "mode": "row", "T": 1500, "E": 32, "k": 4, "D": 1024, "F": 704,
         "P": 2, "dtype": "f16"},
        # the gate|up weights of the decode MLP, quantized once when loaded
        {"name": "quantize-weights", "op": "quantize", "rows": 28672, "cols": 4096, "dtype": "bf16"},
        # a few tokens' activations, quantized at every step
        {"name": "quantize-tokens", "op": "quantize", "rows": 17, "cols": 14336, "dtype": "f32"},
        # a decoding batch through MXFP4 experts of the decode MLP's shape
        {"name": "mxfp4-decode", "op": "mxfp4", "acts": 16, "T": 16, "E": 8, "k": 2, "D": 4096, "F": 14336, "P": 8,
         "dtype": "bf16"},
        # the prefill's gate|up product with quantized activations, one expert
        {"name": "mxfp4-prefill", "op": "mxfp4", "acts": 4, "T": 4096, "E": 1, "k": 1, "D": 4096, "F": 14336, "P": 4,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "backward", "quantize", "mxfp4"])
    if op == "route":
        train = rng.random() < 0.5
        E = _log(rng, 4, 256)
        return {"op": "route", "train": train, "T": _log(rng, 1, 8192), "E": E, "k": rng.randint(1, min(8, E)),
                "D": 8 * _log(rng, 8, 256) if train else 0, "dtype": rng.choice(["bf16", "f16", "f32"]),
                "normalize": rng.random() < 0.5, "masked": rng.random() < 0.5}
    if op == "quantize":
        rows = _log(rng, 1, 28672)
        return {"op": "quantize", "rows": rows, "cols": 32 * _log(rng, 1, min(448, 3670016 // rows)),
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    E = _log(rng, 1, 64)
    k = rng.randint(1, min(6, E))
    P = rng.choice([1, 2, 4, 8])
    T = _log(rng, 1, 4096)
    if op == "mxfp4":
        D, F = 32 * _log(rng, 2, 128), 32 * P * _log(rng, 1, 448 // P)
    else:
        D, F = rng.choice([8, 2, 64]) * _log(rng, 16, 64), P * _log(rng, 16, 2048 // P)
        if rng.random() < 0.5:
            F = 64 * P * max(1, F // (64 * P))
    # no dearer than the largest listed case: weights to 1.4e9 values, products to 1.4e12
    E = max(k, min(E, int(1.4e9 // (3 * D * F))))
    T = max(1, min(T, int(1.4e12 // (6.0 * D * F * k))))
    c = {"op": op, "T": T, "E": E, "k": k, "D": D, "F": F, "P": P,
         "dtype": "bf16" if op == "mxfp4" else rng.choice(["bf16", "f16"])}
    if op == "moe":
        c["masked"] = rng.random() < 0.5
    elif op == "backward":
        c["mode"] = rng.choice(["column", "row"])
    else:
        c["acts"] = rng.choice([16, 4])
    return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _uniform(g, shape, bound, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").uniform_(-bound, bound, generator=g)


def _normal(g, shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def _logits(g, c):
    """Router logits: some experts drawn more often than others; masked: a few
    experts closed for each token, and the last tokens of the batch padding
    that no expert takes."""
    z = _normal(g, (c["T"], c["E"]), torch.float32) + 0.7 * _normal(g, (c["E"],), torch.float32)
    z = z.to(DT[c["dtype"]])
    if c.get("masked"):
        closed = torch.rand(z.shape, generator=g, device="cuda") < 0.1
        closed[:, 0] = False  # a token that is no padding has one expert at least
        closed[c["T"] - c["T"] // 9:] = True
        z[closed] = -math.inf
    return z


def _choose(z, k, normalize):
    """The k largest logits of each token (ties: the lowest expert), their
    weights, and the plan; slots whose logit is -inf are dropped (expert -1,
    weight 0)."""
    T, E = z.shape
    v, e = torch.sort(z.float(), dim=1, descending=True, stable=True)
    top = v[:, :1]
    kept = v[:, :k] > -math.inf
    p = torch.where(v > -math.inf, torch.exp(v - top), 0.0)
    w = torch.where(kept, p[:, :k] / (p[:, :k] if normalize else p).sum(1, keepdim=True), 0.0)
    e = torch.where(kept, e[:, :k], -1).to(torch.int32)
    return w, e, *_plan(e, E)


def _plan(e, E):
    """offsets (E + 1): where each expert's rows begin; rows (T k): the slot of
    each row, in slot order for each expert, -1 behind the last; slots (T, k):
    the row of each slot, -1 if dropped."""
    flat = e.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True)[1]
    ends = (key[:, None] == torch.arange(E, device=e.device)).sum(0).cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    at = torch.arange(flat.numel(), device=e.device)
    rows = torch.where(at < ends[-1], order, -1)
    slots = torch.empty_like(at).scatter_(0, order, at)
    slots = torch.where(flat < 0, -1, slots).view(e.shape)
    return offsets.to(torch.int32), rows.to(torch.int32), slots.to(torch.int32)


def _weights(g, E, n, m, dtype, mx):
    """E weights (n, m), U(+-1/sqrt m); MXFP4: random codes, scales that give about that size."""
    if not mx:
        return _uniform(g, (E, n, m), 1 / math.sqrt(m), dtype)
    codes = torch.randint(0, 256, (E, n, m // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(124, 127, (E, n, m // 32), dtype=torch.uint8, device="cuda", generator=g)
    return codes, scales - int(round(math.log2(m) / 2))


def _shard(w, sharding, segments, P):
    import sharded_gemm_alltosharded_amd as sg
    if isinstance(w, tuple):
        return sg.shard_mxfp4_experts(*w, sharding, segments=segments, P=P)
    return sg.shard_experts(w, sharding, segments=segments, P=P)


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = DT[c["dtype"]]
    if c["op"] == "quantize":
        # rows of different sizes, a few outliers
        x = _normal(g, (c["rows"], c["cols"]), torch.float32) * torch.exp(_normal(g, (c["rows"], 1), torch.float32))
        x[torch.rand(x.shape, generator=g, device="cuda") < 0.002] *= 20
        return {"case": c, "x": x.to(dt)}
    s = {"case": c}
    T, E, k = c["T"], c["E"], c["k"]
    s["logits"] = _logits(g, c)
    if c["op"] == "route":
        if c["train"]:
            s["y"] = _normal(g, (T * k, c["D"]), dt)
            s["dout"] = _normal(g, (T, c["D"]), dt)
            s["dy"] = torch.zeros_like(s["y"])  # rows of no slot stay as they are
        return s
    D, F, P = c["D"], c["F"], c["P"]
    w, e, offsets, rows, slots = _choose(s["logits"], k, True)
    s.update(weights=w, experts=e, offsets=offsets, rows=rows, slots=slots)
    s["ends"] = offsets.tolist()
    R = s["ends"][-1]
    s["x"] = _normal(g, (T, D), dt)
    mx = c["op"] == "mxfp4"
    if c["op"] in ("moe", "mxfp4"):
        s["gu"] = _weights(g, E, 2 * F, D, dt, mx)
        if not mx or c["acts"] == 16:
            s["dn"] = _weights(g, E, D, F, dt, mx)
        if own:
            s["lgu"] = _shard(s["gu"], "all-to-sharded", 2, P)
            if "dn" in s:
                s["ldn"] = _shard(s["dn"], "sharded-to-all", 1, P)
    elif c["mode"] == "column":
        s["gu"] = _weights(g, E, 2 * F, D, dt, False)
        s["pre"] = _normal(g, (P, R, 2 * F // P), dt)  # gate|up outputs, kept by the forward pass
        s["dh"] = _normal(g, (P, R, F // P), dt)
        if own:
            s["lgu"] = _shard(s["gu"], "all-to-sharded", 2, P)
    else:
        s["dn"] = _weights(g, E, D, F, dt, False)
        s["h"] = _normal(g, (P, R, F // P), dt)
        s["dy"] = _normal(g, (R, D), dt)
        if own:
            s["ldn"] = _shard(s["dn"], "sharded-to-all", 1, P)
    if own:
        import sharded_gemm_alltosharded_amd as sg
        s["route"] = sg.Route(w, e, offsets, rows, slots)
    return s


# ---- plain forms -----------------------------------------------------------

def _silu(z):
    return z / (1 + torch.exp(-z))


def _wide(w, e, to=torch.float32):
    """Expert e's weight in 32 bits."""
    if isinstance(w, tuple):
        return _decode(w[0][e], w[1][e])
    return w[e].to(to)


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _decode(codes, scales):
    """MXFP4 -> 32 bits: element 2i of a row in the low half of byte i."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], device=codes.device)
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    s = torch.where(scales == 255, math.nan, torch.exp2(scales.double() - 127)).float()
    return v * s.repeat_interleave(32, -1)


def _encode(x):
    """32 bits -> MXFP4 codes and scales: for each block of 32 the exponent of
    its largest magnitude less 2; nearest code, ties to the even one, the
    largest magnitude 6."""
    b = x.unflatten(-1, (-1, 32))
    m = b.abs().amax(-1)
    ex = (torch.frexp(m)[1] - 3).clamp(-127, 127)  # frexp's mantissa is in [1/2, 1)
    ex = torch.where(m > 0, ex, -127)
    q = (b.double() * torch.exp2(-ex.double())[..., None]).float()
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    r = (torch.round(a / step) * step).clamp(max=6.0)
    code = torch.searchsorted(torch.tensor(E2M1, device=x.device), r.contiguous()) + 8 * torch.signbit(q)
    code = code.to(torch.uint8).flatten(-2)
    bad = ~torch.isfinite(m)
    scales = torch.where(bad, 255, ex + 127).to(torch.uint8)
    return code[..., ::2] | (code[..., 1::2] << 4), scales


def _ranks(h, P):
    """(R, n) columns of P ranks -> (P, R, n / P)."""
    return h.unflatten(1, (P, -1)).transpose(0, 1)


def _columns(h):
    """(P, R, n / P) -> (R, n)."""
    return h.transpose(0, 1).flatten(1)


def _gate_up(x, w, floc):
    """Expert weight rows [gate; up] on the rows x: gate and up outputs."""
    return x @ w[:floc].T, x @ w[floc:].T


def _grouped(s, f):
    """f(expert, its rows' range) over the experts that have rows, joined."""
    ends = s["ends"]
    return torch.cat([f(e, slice(ends[e], ends[e + 1])) for e in range(len(ends) - 1) if ends[e] < ends[e + 1]])


def _sum_slots(y, slots, weights):
    """out[t] = sum over a token's kept slots of weight * row."""
    y = torch.cat([y, y.new_zeros(1, y.shape[1])])
    return (weights[:, :, None] * y[slots.long()]).sum(1)


def run(state):
    s = state
    c = s["case"]
    if own:
        return _run_own(s)
    dt = DT[c["dtype"]]
    if c["op"] == "quantize":
        return _decode(*_encode(s["x"].float())).to(dt)
    if c["op"] == "route":
        w, e, offsets, rows, slots = _choose(s["logits"], c["k"], c["normalize"])
        if not c["train"]:
            return w, e, offsets, rows, slots
        y, dout = s["y"].float(), s["dout"].float()
        out = _sum_slots(y, slots, w)
        kept = rows >= 0
        r = rows.clamp(min=0).long()
        t = r // c["k"]
        dy = torch.where(kept[:, None], w.flatten()[r][:, None] * dout[t], s["dy"].float())
        dots = (y * dout[t]).sum(1)
        dw = torch.where(slots < 0, 0.0, dots[slots.clamp(min=0).long()])
        back = (w * dw).sum(1, keepdim=True)
        z = s["logits"].float()
        chosen = torch.zeros_like(z).scatter_add(1, e.clamp(min=0).long(), torch.where(e < 0, 0.0, w * dw))
        if c["normalize"]:
            p = torch.zeros_like(z).scatter_add(1, e.clamp(min=0).long(), w)
        else:
            top = z.amax(1, keepdim=True)
            p = torch.where(z > -math.inf, torch.exp(z - top), 0.0)
            p = torch.where(top > -math.inf, p / p.sum(1, keepdim=True), 0.0)
        dz = chosen - p * back
        return w, e, offsets, rows, slots, out.to(dt), dy.to(dt), dw, dz.to(dt)
    D, F, P, k = c["D"], c["F"], c["P"], c["k"]
    R = s["ends"][-1]
    token = s["rows"][:R].long() // k
    if c["op"] == "backward" and c["mode"] == "column":
        # the layer's rows of rank r: [gate_r; up_r]
        g, u = (v.transpose(0, 1) for v in s["pre"].float().chunk(2, -1))  # (R, P, F / P)
        dh = s["dh"].float().transpose(0, 1)
        sig = 1 / (1 + torch.exp(-g))
        dg, du = dh * u * sig * (1 + g * (1 - sig)), dh * g * sig
        d = torch.cat([dg.flatten(1), du.flatten(1)], 1)  # columns [gate; up], as the unsharded rows
        x = s["x"].float()[token]
        dx = _grouped(s, lambda e, r: d[r] @ s["gu"][e].float())
        dw = torch.stack([d[s["ends"][e]:s["ends"][e + 1]].T @ x[s["ends"][e]:s["ends"][e + 1]]
                          for e in range(c["E"])])
        dw = dw.unflatten(1, (2, P, F // P)).transpose(1, 2).flatten(2, 3)  # (E, P, 2F / P, D)
        return torch.cat([dg, du], -1).transpose(0, 1).to(dt), dx.to(dt), dw.to(dt)
    if c["op"] == "backward":
        h, dy = _columns(s["h"].float()), s["dy"].float()
        dh = _grouped(s, lambda e, r: dy[r] @ s["dn"][e].float())
        dw = torch.stack([dy[s["ends"][e]:s["ends"][e + 1]].T @ h[s["ends"][e]:s["ends"][e + 1]]
                          for e in range(c["E"])])
        return _ranks(dh, P).to(dt), dw.unflatten(2, (P, F // P)).transpose(1, 2).to(dt)
    x = s["x"].float()
    if c["op"] == "mxfp4" and c["acts"] == 4:
        x = _decode(*_encode(x))
    x = x[token]

    def h_of(e, r):
        gate, up = _gate_up(x[r], _wide(s["gu"], e), F)
        return _silu(gate) * up

    h = _grouped(s, h_of)
    if c["op"] == "mxfp4" and c["acts"] == 4:
        return _ranks(h, P).to(dt)
    y = _grouped(s, lambda e, r: h[r] @ _wide(s["dn"], e).T)
    return _sum_slots(y, s["slots"], s["weights"]).to(dt)


# ---- the package's calls ---------------------------------------------------

def _run_own(s):
    import sharded_gemm_alltosharded_amd as sg
    c = s["case"]
    if c["op"] == "quantize":
        codes, scales = sg.quantize_mxfp4(s["x"])
        return sg.dequantize_mxfp4(codes, scales, out_dtype=s["x"].dtype)
    if c["op"] == "route":
        r = sg.moe_route(s["logits"], c["k"], normalize=c["normalize"])
        if not c["train"]:
            return r.weights, r.experts, r.offsets, r.rows, r.slots
        out = sg.moe_combine(s["y"], r.slots, r.weights)
        dy, dw = sg.moe_combine_backward(s["dout"], s["y"], r.slots, r.weights, dy=s["dy"])
        dz = sg.moe_route_backward(s["logits"], r, dw, normalize=c["normalize"])
        return r.weights, r.experts, r.offsets, r.rows, r.slots, out, dy, dw, dz
    if c["op"] == "backward" and c["mode"] == "column":
        d = sg.swiglu_backward(s["pre"], s["dh"])
        dx, dw = sg.experts_all_to_sharded_backward(s["lgu"], s["x"], d, s["offsets"], rows=s["rows"][:d.shape[1]],
                                                    k=c["k"], dw_dtype=d.dtype)
        return d, dx, dw
    if c["op"] == "backward":
        return sg.experts_sharded_to_all_backward(s["ldn"], s["h"], s["dy"], s["offsets"], dw_dtype=s["h"].dtype)
    if c["op"] == "mxfp4" and c["acts"] == 4:
        codes, scales = sg.quantize_mxfp4(s["x"])
        return sg.experts_all_to_sharded(s["lgu"], codes, s["offsets"], rows=s["rows"][:s["ends"][-1]], k=c["k"],
                                         swiglu=True, x_scales=scales, out_dtype=s["x"].dtype)
    return sg.moe_mlp(s["lgu"], s["ldn"], s["x"], s["route"])


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (2 * size + 2 * (0.5 + 1 / 32)), "flops": 4 * n}
    T, E, k = c["T"], c["E"], c["k"]
    plan = T * k * 16 + 4 * (E + 1)
    if c["op"] == "route":
        b = T * E * size + plan
        if c["train"]:
            b += (4 * T * k + 2 * T) * c["D"] * size + T * E * size + 8 * T * k
        return {"bytes": b, "flops": 8 * T * E + 4 * T * k * c["D"]}
    D, F = c["D"], c["F"]
    rows = T * k
    taken = E * (1 - (1 - k / E) ** T)  # experts that have rows, on average
    if c["op"] == "backward":
        n = 2 * F if c["mode"] == "column" else F
        acts = 2 * rows * (2 * n + D) + 2 * (T if c["mode"] == "column" else rows) * D
        return {"bytes": acts + 2 * D * n * (taken + E), "flops": 4.0 * rows * D * n}
    per = 0.5 + 1 / 32 if c["op"] == "mxfp4" else 2
    if c["op"] == "mxfp4" and c["acts"] == 4:
        return {"bytes": taken * 2 * F * D * per + 2 * T * D + 2 * rows * F, "flops": 4.0 * rows * D * F}
    return {"bytes": taken * 3 * F * D * per + 4 * T * D, "flops": 6.0 * rows * D * F}


# ---- the definitions in 64 bits --------------------------------------------

def _exact_route(z, k, normalize):
    """Ranks by counting: expert e stands behind every larger logit and every equal one of a lower number."""
    z = z.double()
    T, E = z.shape
    idx = torch.arange(E, device=z.device)
    rank = torch.zeros((T, E), dtype=torch.long, device=z.device)
    for f in range(E):
        other = z[:, f:f + 1]
        rank += (other > z) | ((other == z) & (f < idx))
    open_ = torch.isfinite(z)
    p = torch.softmax(z, 1).nan_to_num(0.0) * open_
    e = torch.full((T, k), -1, device=z.device)
    w = torch.zeros((T, k), dtype=torch.float64, device=z.device)
    for j in range(k):
        at = (rank == j) & open_
        has = at.any(1)
        e[:, j] = torch.where(has, at.int().argmax(1), -1)
        w[:, j] = (p * at).sum(1)
    if normalize:
        w = (w / w.sum(1, keepdim=True)).nan_to_num(0.0)
    flat = e.flatten()
    hit = [torch.nonzero(flat == f).flatten() for f in range(E)]
    offsets = torch.tensor([0] + [len(h) for h in hit], device=z.device).cumsum(0)
    order = torch.cat(hit)
    rows = torch.full((T * k,), -1, device=z.device)
    rows[:len(order)] = order
    slots = torch.full((T * k,), -1, device=z.device)
    slots[order] = torch.arange(len(order), device=z.device)
    return p, w, e, offsets, rows, slots.view(T, k)


def _power(n):
    """2^n in 64 bits, by its exponent field."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_mx(codes, scales):
    c = torch.stack([codes % 16, codes // 16], -1).flatten(-2).long()
    man, ex = c % 2, c // 2 % 4
    mag = torch.where(ex > 0, (2 + man) * _power(ex - 2), man * 0.5)
    v = torch.where(c >= 8, -mag, mag)
    return v.unflatten(-1, (-1, 32)).mul(_power(scales.long() - 127)[..., None]).flatten(-2)


def _exact_round(x):
    """The nearest values that MXFP4 can hold, by distance to each of its magnitudes."""
    b = x.double().unflatten(-1, (-1, 32))
    m = b.abs().amax(-1, keepdim=True)
    top = torch.where(m > 0, torch.floor(torch.log2(m.clamp(min=1e-300))), -125.0)
    top = torch.where(_power(top) > m, top - 1, torch.where(_power(top + 1) <= m, top + 1, top))
    s = _power((top - 2).clamp(-127, 127))
    a = b.abs() / s
    best = torch.zeros_like(a)
    for i in (2, 4, 6, 1, 3, 5, 7):  # a tie between neighbours goes to the even code
        nearer = (a - E2M1[i]).abs() < (a - best).abs()
        best = torch.where(nearer, E2M1[i], best)
    return (torch.copysign(best, b) * s).flatten(-2)


def exact(case, seed):
    global own
    c, was = case, own
    own = False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    if c["op"] == "quantize":
        n = max(1, (1 << 24) // c["cols"])
        return torch.cat([_exact_round(x) for x in s["x"].split(n)])
    if c["op"] == "route":
        p, w, e, offsets, rows, slots = _exact_route(s["logits"], c["k"], c["normalize"])
        plan = (w, e.int(), offsets.int(), rows.int(), slots.int())
        if not c["train"]:
            return plan
        T, k, D = c["T"], c["k"], c["D"]
        out = torch.zeros((T, D), dtype=torch.float64, device="cuda")
        dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        dy = torch.zeros_like(s["y"], dtype=torch.float64)
        for j in range(k):
            t = torch.nonzero(slots[:, j] >= 0).flatten()
            r = slots[t, j]
            out[t] += w[t, j:j + 1] * s["y"][r].double()
            dw[t, j] = torch.linalg.vecdot(s["y"][r].double(), s["dout"][t].double())
            dy[r] = w[t, j:j + 1] * s["dout"][t].double()
        q = torch.zeros_like(p)
        grad = torch.zeros_like(p)  # of the probabilities that the weights are
        for j in range(k):
            t = torch.nonzero(e[:, j] >= 0).flatten()
            grad[t, e[t, j]] = dw[t, j]
            q[t, e[t, j]] = w[t, j]
        q = q if c["normalize"] else p
        dz = q * (grad - (q * grad).sum(1, keepdim=True))
        return (*plan, out, dy, dw, dz)
    D, F, P, k = c["D"], c["F"], c["P"], c["k"]
    ends = s["ends"]
    R = ends[-1]
    f = F // P
    if c["op"] == "backward":
        dw = torch.zeros((c["E"], P, 2 * f, D) if c["mode"] == "column" else (c["E"], P, D, f), dtype=torch.float64,
                         device="cuda")
        if c["mode"] == "column":
            z, up = s["pre"][..., :f].double(), s["pre"][..., f:].double()
            th = torch.tanh(z / 2)  # sigmoid(z) = (1 + tanh(z / 2)) / 2
            sig, slope = (1 + th) / 2, (1 - th * th) / 4
            d = torch.cat([s["dh"].double() * up * (sig + z * slope), s["dh"].double() * z * sig], -1)
            dx = torch.zeros((R, D), dtype=torch.float64, device="cuda")
        else:
            dx = torch.zeros((P, R, f), dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            a, b = ends[e], ends[e + 1]
            for r in range(P):
                if c["mode"] == "column":
                    w = torch.cat([s["gu"][e, r * f:(r + 1) * f], s["gu"][e, F + r * f:F + (r + 1) * f]]).double()
                    dx[a:b] += d[r, a:b] @ w
                    dw[e, r] = d[r, a:b].T @ s["x"][s["rows"][a:b].long() // k].double()
                else:
                    dx[r, a:b] = s["dy"][a:b].double() @ s["dn"][e, :, r * f:(r + 1) * f].double()
                    dw[e, r] = s["dy"][a:b].double().T @ s["h"][r, a:b].double()
        return (d, dx, dw) if c["mode"] == "column" else (dx, dw)
    x = s["x"].double()
    four = c["op"] == "mxfp4" and c["acts"] == 4
    if four:
        x = _exact_round(x)
    wide = (lambda w, e: _exact_mx(w[0][e], w[1][e])) if c["op"] == "mxfp4" else (lambda w, e: w[e].double())
    h = torch.zeros((R, F), dtype=torch.float64, device="cuda")
    out = torch.zeros((c["T"], D), dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        slot = s["rows"][a:b].long()
        w = wide(s["gu"], e)
        gu = torch.matmul(w, x[slot // k].T).T
        h[a:b] = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        if not four:
            y = torch.matmul(wide(s["dn"], e), h[a:b].T).T
            out.index_add_(0, slot // k, s["weights"].double().flatten()[slot][:, None] * y)
    if four:
        return torch.stack([h[:, r * f:(r + 1) * f] for r in range(P)])
    return out
