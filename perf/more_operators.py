"""Measured cases of the experts' layer in 8-bit integers: rows cast as they are
dispatched and between the products, the products with scales per token and
channel, and the whole layer for a few tokens.

Each case is one call as a user's program makes it.  With `own` false, `run`
computes the operator in elementary torch operations; with `own` true it calls
the library.  Sizes are those of the repository's workloads (4096 x 7168 top-8
of 256, 8192 x 4096 top-6 of 64, 128 x 7168 top-8) and one to 64 tokens.
Codes are whole numbers: they have to be equal.
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"


def listed():
    return [
        # 128 tokens being generated, cast to the padded receive layout.
        _dispatch("dispatch_small", 128, 7168, 8, 256, 16, 0.0),
        # A training or prompt batch, packed.
        _dispatch("dispatch_dsv3", 4096, 7168, 8, 256, 0, 0.0),
        # A ragged batch with empty slots.
        _dispatch("dispatch_ragged", 8191, 4096, 6, 64, 0, 0.05),
        # Between the products of the 128 and the 4096 tokens.
        _quantize("quantize_small", 128, 8, 256, 2048, 16),
        _quantize("quantize_dsv3", 4096, 8, 256, 2048, 0),
        # Down products of 128 tokens being generated: every weight for a few rows.
        _linear("linear_small", 128, 8, 256, 2048, 7168, "none", 16),
        # Gate and up products of a prompt over 64 experts.
        _linear("linear_prompt", 8192, 6, 64, 4096, 1024, "silu_mul", 0),
        # Gate and up products of 4096 tokens over 256 experts: 128 rows an expert.
        _linear("linear_dsv3", 4096, 8, 256, 7168, 2048, "silu_mul", 0),
        # Down products of an odd batch.
        _linear("linear_ragged", 1111, 6, 60, 1408, 2048, "none", 0),
        # The layer for one token being generated, for 16 users at once, and for 64
        # over fewer and smaller experts.
        _moe("moe_token", 1, 8, 256, 7168, 2048, 0.0),
        _moe("moe_few", 16, 8, 256, 7168, 2048, 0.0),
        _moe("moe_batch", 64, 6, 64, 4096, 1024, 0.05),
    ]


def _dispatch(name, T, H, k, E, capacity, empty):
    return dict(name=name, op="dispatch", T=T, H=H, k=k, E=E, capacity=capacity, empty=empty)


def _quantize(name, T, k, E, K, capacity):
    return dict(name=name, op="quantize", T=T, k=k, E=E, K=K, capacity=capacity)


def _linear(name, T, k, E, K, N, epilogue, capacity):
    return dict(name=name, op="linear", T=T, k=k, E=E, K=K, N=N, epilogue=epilogue, capacity=capacity)


def _moe(name, T, k, E, H, F, empty):
    return dict(name=name, op="moe", T=T, k=k, E=E, H=H, F=F, empty=empty)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dispatch", "quantize", "linear", "moe"])
    k, E = rng.randint(1, 8), rng.choice([8, 16, 60, 64, 128, 256])
    if op == "dispatch":
        H = 16 * _log(rng, 4, 512)
        T = min(_log(rng, 1, 16384), 4096 * 8 * 7168 // (k * H))
        # A padded region holds a few times its mean load; later slots are dropped.
        c = _dispatch("", T, H, k, E, rng.choice([0, 0, 1]) * (4 + 2 * T * k // E), rng.choice([0.0, 0.05]))
    elif op == "quantize":
        K = 16 * _log(rng, 4, 512)
        T = min(_log(rng, 1, 16384), 4096 * 8 * 2048 // (k * K))
        c = _quantize("", T, k, E, K, rng.choice([0, 0, 1]) * (4 + 2 * T * k // E))
    elif op == "linear":
        epilogue = rng.choice(["none", "silu_mul"])
        K, N = 128 * _log(rng, 1, 56), 8 * _log(rng, 8, 896)
        wide = 2 * N if epilogue == "silu_mul" else N
        while E * wide * K > 1 << 32:
            E //= 2
        T = _log(rng, 1, 8192)
        T = max(1, min(T, 49152 // k, int(4e11 / (k * wide * K))))
        c = _linear("", T, k, E, K, N, epilogue, rng.choice([0, 0, 1]) * (4 + 2 * T * k // E))
    else:
        H, F = 128 * _log(rng, 1, 56), 128 * _log(rng, 1, 32)
        while E * H * F > 1 << 32:
            E //= 2
        c = _moe("", _log(rng, 1, 64), k, E, H, F, rng.choice([0.0, 0.0, 0.1]))
    del c["name"]
    return c


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _routing(g, c):
    """k distinct experts per token, uniform (the law of the repository's
    workloads), some slots empty."""
    idx = torch.rand(c["T"], c["E"], generator=g, device=DEV).argsort(dim=1)[:, : c["k"]].contiguous()
    if c.get("empty"):
        idx = torch.where(torch.rand(idx.shape, generator=g, device=DEV) < c["empty"], -1, idx)
    return idx


def _weights(g, E, rows, K):
    """Codes with a peak at zero that reach +-126, and scales that bring products of
    unit inputs to about one."""
    w = torch.randint(-63, 64, (E, rows, K), dtype=torch.int8, generator=g, device=DEV)
    w += torch.randint(-63, 64, (E, rows, K), dtype=torch.int8, generator=g, device=DEV)
    return w, torch.exp(0.2 * _normal(g, E, rows)) / (52.0 * math.sqrt(K))


def _order(idx, E, capacity):
    """Receive order: token_row [T, k] and offsets [E + 1], or for the padded
    layout slots and counts [E]."""
    ids = torch.where((idx < 0) | (idx >= E), E, idx).reshape(-1)
    order = torch.argsort(ids, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=DEV)
    count = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    count.scatter_add_(0, ids, torch.ones_like(ids))
    start = count.cumsum(0) - count
    if capacity:
        at = place - start[ids]
        row = torch.where((ids < E) & (at < capacity), ids * capacity + at, -1)
        return row.view(idx.shape).int(), count[:E].clamp(max=capacity).int()
    return torch.where(ids < E, place, -1).view(idx.shape).int(), start.int()


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    T, k, E, cap = c["T"], c["k"], c["E"], c.get("capacity", 0)
    idx = _routing(g, c)
    rows = E * cap if cap else T * idx.shape[1]
    if c["op"] == "dispatch":
        H = c["H"]
        # Activations: channels of different sizes.
        c["x"] = (_normal(g, T, H) * torch.exp(0.5 * _normal(g, H))).bfloat16()
        c["idx"], c["w"] = idx, torch.softmax(_normal(g, T, idx.shape[1]), dim=1)
        # A user's own buffers; rows that no slot maps to stay as they are.
        shape = (E, cap) if cap else (rows,)
        c["out"] = dict(recv_x_i8=torch.zeros(*shape, H, dtype=torch.int8, device=DEV),
                        recv_scales=torch.zeros(shape, device=DEV),
                        recv_src_idx=torch.zeros(shape, dtype=torch.int32, device=DEV),
                        recv_topk_weights=torch.zeros(shape, device=DEV))
        if cap:
            c["out"]["recv_count"] = torch.zeros(E, dtype=torch.int32, device=DEV)
            c["out"]["token_slot"] = torch.zeros(idx.shape, dtype=torch.int32, device=DEV)
        else:
            c["out"]["recv_expert_offset"] = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
            c["out"]["token_row"] = torch.zeros(idx.shape, dtype=torch.int32, device=DEV)
    elif c["op"] == "quantize":
        _, c["rows"] = _order(idx, E, cap)
        gate, up = _normal(g, rows, c["K"]), _normal(g, rows, c["K"])
        c["x"] = (gate * torch.sigmoid(gate) * up).bfloat16()
        c["out"] = dict(x_i8=torch.zeros(rows, c["K"], dtype=torch.int8, device=DEV), x_scales=torch.zeros(rows, device=DEV))
    elif c["op"] == "linear":
        K, N = c["K"], c["N"]
        _, c["rows"] = _order(idx, E, cap)
        c["x"] = (32 * _normal(g, rows, K)).round().clamp(-127, 127).to(torch.int8)
        c["xs"] = torch.exp(0.1 * _normal(g, rows)) / 32
        c["w"], c["ws"] = _weights(g, E, 2 * N if c["epilogue"] == "silu_mul" else N, K)
        c["y"] = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV)
        # What the plain form needs to lay the rows out one expert after the
        # other: the experts that have rows and the largest count.
        count = c["rows"].long() if cap else (c["rows"][1:] - c["rows"][:-1]).long()
        c["used"], c["most"] = count.nonzero().reshape(-1), int(count.max())
        c["start"] = (c["used"] * cap if cap else c["rows"][:-1][c["used"]].long())
        c["count"] = count[c["used"]]
    else:
        c["x"] = (_normal(g, T, c["H"]) * torch.exp(0.5 * _normal(g, c["H"]))).bfloat16()
        c["idx"], c["w"] = idx, torch.softmax(_normal(g, T, idx.shape[1]), dim=1)
        c["up"], c["us"] = _weights(g, E, 2 * c["F"], c["H"])
        c["down"], c["ds"] = _weights(g, E, c["H"], c["F"])
        # For the plain form: the experts that some slot chose, the slots of each
        # and the largest count.
        ids = torch.where(idx < 0, E, idx).reshape(-1)
        count = torch.bincount(ids, minlength=E + 1)
        c["used"], c["most"] = count[:E].nonzero().reshape(-1), int(count[:E].max())
        c["count"] = count[c["used"]]
        c["slots"] = torch.argsort(ids, stable=True)
        c["start"] = (count.cumsum(0) - count)[c["used"]]
    return c


# ---- the library's calls ---------------------------------------------------------


def _own(c):
    from combine_get_dispatch_02_amd import ep

    if c["op"] == "dispatch":
        if c["capacity"]:
            return ep.ep_dispatch_ll_i8(c["x"], c["idx"], c["w"], c["E"], c["capacity"], out=c["out"])
        return ep.ep_dispatch_i8(c["x"], c["idx"], c["w"], c["E"], 1, out=c["out"])
    if c["op"] == "quantize":
        return ep.ep_quantize_i8(c["x"], c["rows"], capacity=c["capacity"], out=c["out"])
    if c["op"] == "linear":
        return ep.ep_expert_linear_i8(c["x"], c["xs"], c["rows"], c["w"], c["ws"], capacity=c["capacity"], epilogue=c["epilogue"],
                                      out=c["y"])
    return ep.ep_moe_i8(c["x"], c["idx"], c["w"], c["up"], c["us"], c["down"], c["ds"])


# ---- the plain forms ---------------------------------------------------------------


def _cast(x):
    """Codes and scales of rows.  127 x and the largest magnitude of bf16 rows are exact
    in 32 bits, and so is a quotient halfway between two codes."""
    a = x.abs().amax(dim=1, keepdim=True)
    q = torch.where(a > 0, x * 127.0 / a, 0.0)
    return torch.round(q).to(torch.int8), (a / 127.0).reshape(-1)


def _plain_dispatch(c):
    row, bounds = _order(c["idx"], c["E"], c["capacity"])
    codes, scales = _cast(c["x"].float())
    to = row[row >= 0].long()
    token = torch.arange(c["T"], device=DEV)[:, None].expand(row.shape)[row >= 0]
    out = {name: torch.zeros_like(t) for name, t in c["out"].items()}
    flat = {name: out[name].view(-1, *out[name].shape[2 if c["capacity"] else 1:])
            for name in ("recv_x_i8", "recv_scales", "recv_src_idx", "recv_topk_weights")}
    flat["recv_x_i8"][to] = codes[token]
    flat["recv_scales"][to] = scales[token]
    flat["recv_src_idx"][to] = token.int()
    flat["recv_topk_weights"][to] = c["w"][row >= 0]
    out["token_slot" if c["capacity"] else "token_row"] = row
    out["recv_count" if c["capacity"] else "recv_expert_offset"] = bounds
    return out


def _plain_quantize(c):
    codes, scales = _cast(c["x"].float())
    rows, at = c["x"].shape[0], torch.arange(c["x"].shape[0], device=DEV)
    if c["capacity"]:
        filled = at % c["capacity"] < c["rows"].repeat_interleave(c["capacity"], output_size=rows)
    else:
        filled = at < c["rows"][-1]
    return dict(x_i8=torch.where(filled[:, None], codes, 0), x_scales=torch.where(filled, scales, 0.0))


def _plain_linear(c):
    used, start, count, most = c["used"], c["start"], c["count"], c["most"]
    # One block of `most` rows for each expert; rows past its count repeat row 0.
    at = torch.arange(most, device=DEV)
    filled = at < count[:, None]
    rows = torch.where(filled, start[:, None] + at, 0)
    v = torch.bmm(c["x"][rows].float(), c["w"][used].float().transpose(1, 2))
    v *= c["xs"][rows][:, :, None] * c["ws"][used][:, None, :]
    if c["epilogue"] == "silu_mul":
        gate, up = v[..., : c["N"]], v[..., c["N"]:]
        v = gate * torch.sigmoid(gate) * up
    y = torch.zeros_like(c["y"])
    y[rows[filled]] = v[filled].bfloat16()
    return y


def _plain_moe(c):
    used, start, count, most = c["used"], c["start"], c["count"], c["most"]
    T, F, H = c["T"], c["F"], c["H"]
    k = c["idx"].shape[1]
    at = torch.arange(most, device=DEV)
    filled = at < count[:, None]
    slots = c["slots"][torch.where(filled, start[:, None] + at, 0)]
    codes, scales = _cast(c["x"].float())
    v = torch.bmm(codes[slots // k].float(), c["up"][used].float().transpose(1, 2))
    v *= scales[slots // k][:, :, None] * c["us"][used][:, None, :]
    gate, up = v[..., :F], v[..., F:]
    h = gate * torch.sigmoid(gate) * up
    a = h.abs().amax(dim=2, keepdim=True)
    q = torch.round(torch.where(a > 0, h * 127.0 / a, 0.0))
    y = torch.bmm(q, c["down"][used].float().transpose(1, 2)) * (a / 127.0 * c["ds"][used][:, None, :])
    each = torch.zeros(T * k, H, device=DEV)
    each[slots[filled]] = y[filled]
    return (each.view(T, k, H) * torch.where(c["idx"] < 0, 0.0, c["w"])[:, :, None]).sum(dim=1).bfloat16()


def run(state):
    if own:
        return _own(state)
    return {"dispatch": _plain_dispatch, "quantize": _plain_quantize, "linear": _plain_linear, "moe": _plain_moe}[state["op"]](state)


def work(case):
    T, E = case["T"], case["E"]
    k = min(case["k"], E)
    n = T * k * (1 - case.get("empty", 0.0))
    # Experts that some slot chose, of uniform routing.
    used = E * (1 - (1 - n / (T * E)) ** T)
    if case["op"] == "dispatch":
        return {"bytes": (2 * T + n) * case["H"] + 12 * T * k + 16 * n + 4 * T * k, "flops": 4 * T * case["H"]}
    if case["op"] == "quantize":
        return {"bytes": n * (3 * case["K"] + 4) + 4 * E, "flops": 4 * n * case["K"]}
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        wide = 2 * N if case["epilogue"] == "silu_mul" else N
        return {"bytes": used * wide * (K + 4) + n * (K + 4 + 2 * N) + 4 * E, "flops": 2 * n * wide * K}
    H, F = case["H"], case["F"]
    return {"bytes": used * (3 * F * H + 8 * F + 4 * H) + 4 * T * H + 12 * T * k, "flops": 6 * n * F * H}


# ---- the definitions in 64 bits -------------------------------------------------------


def _codes64(x):
    """x [rows, K] fp64 -> codes and scales."""
    most = torch.maximum(x.max(dim=1).values, -x.min(dim=1).values)
    some = most > 0
    q = torch.zeros_like(x)
    q[some] = x[some] * 127 / most[some][:, None]
    low = torch.floor(q)
    over = q - low
    up = (over > 0.5) | ((over == 0.5) & (low % 2 != 0))
    return low + up.double(), most / 127


def _exact_dispatch(c):
    idx, w, E, cap = c["idx"].cpu().numpy(), c["w"].double().cpu().numpy(), c["E"], c["capacity"]
    T, k = idx.shape
    flat = idx.reshape(-1)
    valid = np.flatnonzero((flat >= 0) & (flat < E))
    valid = valid[np.argsort(flat[valid], kind="stable")]              # by expert, then slot
    e = flat[valid]
    count = np.bincount(e, minlength=E)
    offset = np.concatenate([[0], np.cumsum(count)])
    to = np.arange(len(valid))
    if cap:
        position = to - offset[e]
        valid, to = valid[position < cap], (e * cap + position)[position < cap]
    rows = E * cap if cap else T * k
    row = np.full(T * k, -1, np.int64)
    row[valid] = to
    src, rw = np.zeros(rows, np.int64), np.zeros(rows)
    src[to], rw[to] = valid // k, w.reshape(-1)[valid]
    q, s = _codes64(c["x"].double())
    q = q.to(torch.int8)
    at, token = torch.from_numpy(to).to(DEV), torch.from_numpy(valid // k).to(DEV)
    x, xs = torch.zeros(rows, c["H"], dtype=torch.int8, device=DEV), torch.zeros(rows, dtype=torch.float64, device=DEV)
    x[at], xs[at] = q[token], s[token]
    shape = (E, cap) if cap else (rows,)
    out = dict(recv_x_i8=x.view(*shape, c["H"]), recv_scales=xs.view(shape), recv_src_idx=src.reshape(shape),
               recv_topk_weights=rw.reshape(shape))
    if cap:
        out.update(recv_count=np.minimum(count, cap), token_slot=row.reshape(T, k))
    else:
        out.update(recv_expert_offset=offset, token_row=row.reshape(T, k))
    return out


def _exact_quantize(c):
    q, s = _codes64(c["x"].double())
    q = q.to(torch.int8)
    if c["capacity"]:
        for e, n in enumerate(c["rows"].tolist()):
            q[e * c["capacity"] + n: (e + 1) * c["capacity"]] = 0
            s[e * c["capacity"] + n: (e + 1) * c["capacity"]] = 0
    else:
        q[int(c["rows"][-1]):] = 0
        s[int(c["rows"][-1]):] = 0
    return dict(x_i8=q, x_scales=s)


def _exact_linear(c):
    y = torch.zeros_like(c["y"], dtype=torch.float64)
    for e, at, n in zip(c["used"].tolist(), c["start"].tolist(), c["count"].tolist()):
        v = (c["x"][at: at + n].double() * c["xs"][at: at + n].double()[:, None]) @ (c["w"][e].double() * c["ws"][e].double()[:, None]).t()
        if c["epilogue"] == "silu_mul":
            v = v[:, : c["N"]] / (1 + torch.exp(-v[:, : c["N"]])) * v[:, c["N"]:]
        y[at: at + n] = v
    return y


def _exact_moe(c):
    T, F = c["T"], c["F"]
    q, s = _codes64(c["x"].double())
    out = torch.zeros(T, c["H"], dtype=torch.float64, device=DEV)
    ids = c["idx"].cpu()
    for e in c["used"].tolist():
        up, down = c["up"][e].double(), c["down"][e].double()
        for t, j in (ids == e).nonzero().tolist():
            v = (up @ q[t]) * s[t] * c["us"][e].double()
            h = v[:F] / (1 + torch.exp(-v[:F])) * v[F:]
            hq, hs = _codes64(h[None])
            out[t] += c["w"][t, j].double() * (down @ hq[0]) * hs[0] * c["ds"][e].double()
    return out


def exact(case, seed):
    c = prepare(case, seed)
    return {"dispatch": _exact_dispatch, "quantize": _exact_quantize, "linear": _exact_linear, "moe": _exact_moe}[case["op"]](c)
