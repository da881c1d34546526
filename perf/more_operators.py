"""Performance cases of the operators that a training run of the MoE layer takes besides its experts.

Three operators: routing by scores (softmax or sigmoid, a balancing bias, groups
of experts; forward with the routing metadata and the bias update, and
backward), the dense product of a shared expert (bias, activation and residual
in its epilogue; forward and backward), and the AdamW step of a list of tensors
(states in 32 or 8 bits).

``run`` computes them with elementary torch operations (``own`` False) or
through the framework's entry points (``own`` True); ``exact`` computes the same
outputs from the definitions in fp64.  Sizes are the layer workloads' (T up to
16384 tokens, d up to 4096, f up to 1536, E up to 256) and odd ones in between.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
RATE = 1e-3
LR, BETAS, EPS, DECAY, STEP = 1e-3, (0.9, 0.999), 1e-8, 0.1, 1000
M32 = 0xFFFFFFFF


# ----------------------------------------------------------------------------- cases

def _route(op, T, E, k, score, bias=False, groups=1, top_groups=1, best=1, renorm=True, scale=1.0, zipf=False):
    return dict(op=op, T=T, E=E, k=k, score=score, bias=bias, groups=groups, top_groups=top_groups, best=best,
                renorm=renorm, scale=scale, zipf=zipf)


def listed():
    return [
        # a single trailing token over the E = 8 layer's experts: pure latency
        dict(_route("route_fwd", 1, 8, 2, "softmax"), name="route_fwd_1tok"),
        # a ragged batch over an odd number of experts, gates not renormalised
        dict(_route("route_fwd", 5003, 60, 6, "softmax", renorm=False, zipf=True), name="route_fwd_odd"),
        # fine-grained experts as balanced by a bias, chosen from half of their groups; the bias update included
        dict(_route("route_fwd", 16384, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5), name="route_fwd_16k_e256"),
        # the router's gradient at the E = 128 workloads: softmax scores as gates, so every expert gets some
        dict(_route("route_bwd", 16384, 128, 4, "softmax", renorm=False), name="route_bwd_16k_e128"),
        # one token through a shared expert's first product
        dict(name="linear_fwd_1tok_bf16", op="linear_fwd", M=1, K=2048, N=1024, act="silu", bias=True, residual=False,
             save=False, dtype="bf16"),
        # the largest workload's tokens through a shared expert's second product, added to the routed output
        dict(name="linear_fwd_16k_bf16", op="linear_fwd", M=16384, K=1536, N=4096, act="none", bias=True, residual=True,
             save=False, dtype="bf16"),
        # the E = 8 workload's first product backward: activation, all gradients, dx joining the routed one
        dict(name="linear_bwd_8k_bf16", op="linear_bwd", M=8192, K=2048, N=1024, act="silu", in_act="none",
             residual=True, dtype="bf16"),
        # odd sizes in fp32, the gradient taken on through the activation before this product
        dict(name="linear_bwd_odd_f32", op="linear_bwd", M=1001, K=777, N=333, act="none", in_act="gelu",
             residual=False, dtype="f32"),
        # everything but the experts of the tiny fp32 workload: router, norm weight and bias
        dict(name="adamw_tiny_f32", op="adamw", shapes="64x8,64,64", dtype="f32", bits=32, master=False),
        # many odd tensors (a shared expert's, norms', routers' of several layers), 8-bit states
        dict(name="adamw_odd_8bit", op="adamw", shapes=",".join(["777x333", "333", "333x777", "777", "777x60"] * 8),
             dtype="f32", bits=8, master=False),
        # the whole E = 8 bf16 layer with fp32 weights beside the bf16 ones
        dict(name="adamw_e8_master", op="adamw", shapes="8x2048x1024,8x2048x1024,8x1024x2048,2048x8,2048,2048",
             dtype="bf16", bits=32, master=True),
        # one projection of all experts of the E = 128 bf16 workload, states in 8 bits
        dict(name="adamw_e128_8bit", op="adamw", shapes="128x2048x1024", dtype="bf16", bits=8, master=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route_fwd", "route_bwd", "linear_fwd", "linear_bwd", "adamw", "adamw"])
    if op.startswith("route"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log_int(rng, 4, 256 // groups)
        top = rng.randint(1, groups)
        k = rng.randint(1, min(8, E // groups * top))
        return _route(op, _log_int(rng, 1, 16384), E, k, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6, groups,
                      top, rng.randint(1, 2), k > 1 and rng.random() < 0.6, rng.choice([1.0, 2.5]), rng.random() < 0.5)
    if op.startswith("linear"):
        M, K, N = _log_int(rng, 1, 16384), _log_int(rng, 8, 4096), _log_int(rng, 8, 4096)
        if rng.random() < 0.6:
            K, N = -(-K // 64) * 64, -(-N // 64) * 64
        dtype = rng.choice(["bf16", "bf16", "f32"])
        cap = 2 * 8192 * 2048 * 1024 // (8 if dtype == "f32" else 1)
        M = max(1, min(M, cap // (K * N)))
        act = rng.choice(["none", "relu", "silu", "gelu"])
        c = dict(op=op, M=M, K=K, N=N, act=act, residual=rng.random() < 0.5, dtype=dtype)
        if op == "linear_fwd":
            c.update(bias=rng.random() < 0.7, save=rng.random() < 0.5)
        else:
            c["in_act"] = rng.choice(["none", "relu", "silu", "gelu"])
        return c
    dtype, bits = rng.choice(["bf16", "f32"]), rng.choice([32, 8])
    shapes, left = [], _log_int(rng, 100, 1 << 26)
    for _ in range(_log_int(rng, 1, 40)):
        n = max(1, min(left, _log_int(rng, 1, 1 << 24)))
        cols = min(n, _log_int(rng, 1, 4096))
        shapes.append("%dx%d" % (n // cols, cols) if rng.random() < 0.7 else "%d" % n)
        left -= n
        if left <= 0:
            break
    return dict(op=op, shapes=",".join(shapes), dtype=dtype, bits=bits, master=dtype == "bf16" and rng.random() < 0.5)


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _pad32(n):
    return -(-n // 32) * 32


def work(case):
    c = case
    if c["op"] == "route_fwd":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * 4 + T * k * 16 + E * 16, "flops": T * E * (4 + 2 * c["bias"]) + 8 * T * k}
    if c["op"] == "route_bwd":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 2 * T * E * 4 + 8 * T * k, "flops": 8 * T * E}
    if c["op"] == "linear_fwd":
        M, K, N, es = c["M"], c["K"], c["N"], 2 if c["dtype"] == "bf16" else 4
        n_out = 1 + c["residual"] + (c["save"] and c["act"] != "none")
        return {"bytes": es * (M * K + K * N + M * N * n_out + N * c["bias"]), "flops": 2 * M * K * N}
    if c["op"] == "linear_bwd":
        M, K, N, es = c["M"], c["K"], c["N"], 2 if c["dtype"] == "bf16" else 4
        per_n, per_k = 1 + (c["act"] != "none"), 2 + (c["in_act"] != "none") + c["residual"]
        return {"bytes": es * (per_n * M * N + per_k * M * K + 2 * K * N + N), "flops": 4 * M * K * N}
    sizes = [math.prod(s) for s in _shapes(c)]
    n, p, es = sum(sizes), sum(_pad32(v) for v in sizes), 2 if c["dtype"] == "bf16" else 4
    # 8 bits: states in, and out again as the values they stand for
    states = 4 * (1 + 1 / 32 + 2 / 2) * p / 2 if c["bits"] == 8 else 16 * p
    return {"bytes": 3 * es * n + states + 8 * n * c["master"], "flops": 14 * n}


# ----------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV, dtype=torch.float32)


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    st = {"case": c}
    if c["op"].startswith("route"):
        T, E, k = c["T"], c["E"], c["k"]
        lg = _randn(g, T, E)
        if c["zipf"]:                                        # a few hot experts, as the Zipf workload
            lg = lg - 3.0 * torch.log(torch.randperm(E, generator=g, device=DEV).float() + 1)
        st["logits"] = lg
        if c["bias"]:                                        # what some hundred updates leave
            st["bias"] = 0.05 * _randn(g, E)
        if c["op"] == "route_bwd":
            st["idx"] = _rand(g, T, E).argsort(1)[:, :k].to(torch.int32).contiguous()
            st["dgates"] = 0.1 * _randn(g, T, k)
    elif c["op"].startswith("linear"):
        M, K, N, dt = c["M"], c["K"], c["N"], DT[c["dtype"]]
        st["x"], st["w"] = _randn(g, M, K).to(dt), (0.02 * _randn(g, K, N)).to(dt)
        if c["op"] == "linear_fwd":
            if c["bias"]:
                st["b"] = (0.1 * _randn(g, N)).to(dt)
            if c["residual"]:
                st["res"] = _randn(g, M, N).to(dt)
        else:
            st["dy"] = _randn(g, M, N).to(dt)
            if c["act"] != "none":                           # what the forward saved
                st["z"] = (0.02 * math.sqrt(K) * _randn(g, M, N)).to(dt)
            if c["in_act"] != "none":
                st["in_z"] = _randn(g, M, K).to(dt)
            if c["residual"]:
                st["dres"] = _randn(g, M, K).to(dt)
    else:
        _prepare_adamw(st, g)
    if own:
        _prepare_own(st)
    return st


def _prepare_adamw(st, g):
    """Parameters, gradients whose size differs by orders of magnitude, and states as earlier steps left them."""
    c = st["case"]
    dt, shapes = DT[c["dtype"]], _shapes(c)
    sizes = [math.prod(s) for s in shapes]
    st["off"] = [0] + np.cumsum([_pad32(n) for n in sizes]).tolist()
    p = st["off"][-1]
    st["w"], st["g"] = [], []
    m, u = torch.zeros(p, device=DEV), torch.zeros(p, device=DEV)
    if c["master"]:
        st["master"] = torch.zeros(p, device=DEV)
    for s, n, o in zip(shapes, sizes, st["off"]):
        size = 1e-3 * torch.exp2(-8.0 * _rand(g, s[-1])).expand(s).reshape(-1)
        w = 0.02 * _randn(g, n)
        st["w"].append(w.to(dt).view(s))
        st["g"].append((size * _randn(g, n)).to(dt).view(s))
        m[o:o + n] = 0.3 * size * _randn(g, n)
        u[o:o + n] = size * (0.5 + _rand(g, n))
        if c["master"]:
            st["master"][o:o + n] = w
    if c["bits"] == 8:
        st["m"], st["ms"] = _encode(m, None)
        st["v"], st["vs"] = _encode(u, None)
    else:
        st["m"], st["v"] = m, u.square_()
    st["seed"] = 12345
    st["gscale"] = torch.tensor([0.7], device=DEV)           # the clipping of the gradients' norm


def _prepare_own(st):
    """Plans, workspaces and output buffers, which a training loop makes once."""
    from mixture_experts_layer_17_amd import binding as B
    c = st["case"]
    if c["op"] == "route_fwd":
        st["ws"] = B._ws(B.lib().moe_route_scored_workspace(c["T"], c["E"], c["k"]), DEV)
    elif c["op"].startswith("linear"):
        st["ws"] = B.moe_linear_workspace(st["x"], st["w"], bwd=c["op"] == "linear_bwd")
    elif c["op"] == "adamw":
        state = B.moe_adamw_state(st["w"], bits=c["bits"], master=c["master"])
        for key, name in (("m", "m"), ("v", "v"), ("m_scale", "ms"), ("v_scale", "vs"), ("master", "master")):
            if state.get(key) is not None:
                state[key].copy_(st[name])
        # not in place: every pass gives the same step
        out = ([torch.empty_like(w) for w in st["w"]], B.moe_adamw_state(st["w"], bits=c["bits"], master=c["master"]))
        st["plan"] = B.moe_adamw_plan(st["w"], st["g"], state, weight_decay=DECAY, out=out)


# ----------------------------------------------------------------------------- the operators

def run(state):
    return _own(state) if own else _plain(state)


def _own(st):
    from mixture_experts_layer_17_amd import binding as B
    c = st["case"]
    op = c["op"]
    if op == "route_fwd":
        r = B.moe_route_scored(st["logits"], c["k"], score=c["score"], bias=st.get("bias"), groups=c["groups"],
                               top_groups=c["top_groups"], group_best=c["best"], renorm=c["renorm"], scale=c["scale"],
                               ws=st["ws"])
        if "bias" in st:
            r["bias"] = B.moe_route_bias_update(r["counts"], st["bias"], RATE, inplace=False)
        return r
    if op == "route_bwd":
        return B.moe_route_scored_bwd(st["logits"], st["idx"], st["dgates"], score=c["score"], renorm=c["renorm"],
                                      scale=c["scale"])
    if op == "linear_fwd":
        return B.moe_linear(st["x"], st["w"], bias=st.get("b"), act=c["act"], residual=st.get("res"),
                            save=c["save"] and c["act"] != "none", ws=st["ws"])
    if op == "linear_bwd":
        return B.moe_linear_bwd(st["dy"], st["x"], st["w"], z=st.get("z"), act=c["act"], in_z=st.get("in_z"),
                                in_act=c["in_act"], dres=st.get("dres"), ws=st["ws"])
    w, state = B.moe_adamw_step(st["plan"], LR, STEP, betas=BETAS, eps=EPS, seed=st["seed"], grad_scale=st["gscale"])
    out = {"w": w}
    if c["bits"] == 8:
        out.update(B.moe_adamw_state_values(state))
    else:
        out.update(m=state["m"], v=state["v"])
    if c["master"]:
        out["master"] = state["master"]
    return out


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "route_fwd":
        return _plain_route(st)
    if op == "route_bwd":
        lg, idx, dg = st["logits"], st["idx"].long(), st["dgates"] * c["scale"]
        s = torch.softmax(lg, 1) if c["score"] == "softmax" else torch.sigmoid(lg)
        sk = s.gather(1, idx)
        if c["renorm"]:
            tot = sk.sum(1, keepdim=True)
            dg = (dg - (dg * sk).sum(1, keepdim=True) / tot) / tot
        if c["score"] == "sigmoid":
            return torch.zeros_like(lg).scatter_(1, idx, dg * sk * torch.sigmoid(-lg.gather(1, idx)))
        ds = torch.zeros_like(lg).scatter_(1, idx, dg)
        return s * (ds - (dg * sk).sum(1, keepdim=True))
    if op == "linear_fwd":
        z = st["x"].float() @ st["w"].float()
        if "b" in st:
            z = z + st["b"].float()
        y = _act(z, c["act"])
        if "res" in st:
            y = y + st["res"].float()
        out = {"y": y.to(st["x"].dtype)}
        if c["save"] and c["act"] != "none":
            out["z"] = z.to(st["x"].dtype)
        return out
    if op == "linear_bwd":
        dz = st["dy"].float()
        if c["act"] != "none":
            dz = dz * _dact(st["z"].float(), c["act"])
        dx = dz @ st["w"].float().T
        if c["in_act"] != "none":
            dx = dx * _dact(st["in_z"].float(), c["in_act"])
        if "dres" in st:
            dx = dx + st["dres"].float()
        dt = st["x"].dtype
        return {"dx": dx.to(dt), "dw": (st["x"].float().T @ dz).to(dt), "db": dz.sum(0).to(dt)}
    return _plain_adamw(st)


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _dact(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))


def _plain_route(st):
    c = st["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    lg = st["logits"].double()                               # in 32 bits near ties would be settled by rounding
    s = torch.softmax(lg, 1) if c["score"] == "softmax" else torch.sigmoid(lg)
    choice = s + st["bias"].double() if "bias" in st else s
    if G > 1:
        best = choice.view(T, G, E // G).topk(c["best"], 2).values.sum(2)
        keep = best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        on = torch.zeros((T, G), dtype=torch.bool, device=DEV).scatter_(1, keep, True)
        choice = choice.masked_fill(~on.repeat_interleave(E // G, 1), -math.inf)
    idx = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    gates = s.gather(1, idx)
    if c["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    flat = idx.reshape(-1)
    counts = torch.zeros(E, dtype=torch.int64, device=DEV).index_add_(0, flat, torch.ones_like(flat))
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    src = flat.sort(dim=0, stable=True).indices
    dst = torch.empty_like(src).scatter_(0, src, torch.arange(T * k, device=DEV))
    out = {"topk_idx": idx, "counts": counts, "offsets": torch.cat([zero, counts.cumsum(0)]), "perm_src": src,
           "perm_dst": dst, "mx_blk_offsets": torch.cat([zero, ((counts + 31) // 32).cumsum(0)])}
    out = {key: v.to(torch.int32) for key, v in out.items()}
    out["gates"] = (gates * c["scale"]).float()
    if "bias" in st:
        out["bias"] = st["bias"] + RATE * torch.sign(T * k - E * counts).float()
    return out


# states in 8 bits: blocks of 32 values, E4M3 codes times a power of two (the byte b stands for 2^(b - 127))

def _encode(x, bits16):
    """Codes and scales of x (a multiple of 32 long), rounded to nearest or up with the chance that bits16 / 2^16 gives."""
    b = x.view(-1, 32)
    frac, exp = torch.frexp(b.abs().amax(1))                 # |x| = frac 2^exp, frac in [0.5, 1)
    e = torch.where(frac > 0, exp - 9 + (frac > 0.875).int(), -127).clamp(-127, 127)
    y = torch.ldexp(b, -e[:, None])                          # at most 448
    if bits16 is not None:
        y = y.abs()
        step = torch.ldexp(torch.ones_like(y), (torch.frexp(y).exponent - 4).clamp(min=-9))
        y = torch.floor(y / step + (bits16.view(-1, 32).float() + 0.5) / 65536.0) * step
        y = torch.copysign(y, b)
    return y.to(torch.float8_e4m3fn).view(torch.uint8).view(-1), (e + 127).to(torch.uint8)


def _decode(q, s):
    return torch.ldexp(q.view(torch.float8_e4m3fn).float().view(-1, 32), s.int()[:, None] - 127).view(-1)


def _mix(h):
    """A hash of 32 bits (numbers or int64 tensors below 2^32)."""
    h = h ^ (h >> 16)
    h = (h * 0x7FEB352D) & M32
    h = h ^ (h >> 15)
    h = (h * 0x846CA68B) & M32
    return h ^ (h >> 16)


def _random_bits(st, p):
    """32 random bits for each state value: a hash of the seed, the step, the tensor's place in the list and the index."""
    keys = [_mix((_mix((st["seed"] + 0x9E3779B9 * t) & M32) + 0x9E3779B9 * STEP) & M32)
            for t in range(len(st["w"]))]
    off = torch.tensor(st["off"], device=DEV)
    i = torch.arange(p, device=DEV)
    t = torch.searchsorted(off[1:], i, right=True)
    return _mix(((i - off[t]) * 0x9E3779B9 + torch.tensor(keys, device=DEV)[t]) & M32)


def _flat(tensors):
    return torch.cat([torch.nn.functional.pad(t.reshape(-1).float(), (0, _pad32(t.numel()) - t.numel())) for t in tensors])


def _plain_adamw(st):
    c = st["case"]
    (b1, b2), eight = BETAS, c["bits"] == 8
    w = st["master"] if c["master"] else _flat(st["w"])
    g = _flat(st["g"]) * st["gscale"]
    m = _decode(st["m"], st["ms"]) if eight else st["m"]
    v = _decode(st["v"], st["vs"]).square() if eight else st["v"]
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g * g
    u = v.sqrt()
    den = u / math.sqrt(1.0 - b2 ** STEP) + EPS
    w = (1.0 - LR * DECAY) * w - (LR / (1.0 - b1 ** STEP)) * (m / den)
    out = {"w": [w[o:o + t.numel()].view(t.shape).to(t.dtype) for t, o in zip(st["w"], st["off"])]}
    if eight:
        h = _random_bits(st, g.numel())
        out["m"] = _decode(*_encode(m, h >> 16)).bfloat16()
        code, s = _encode(u, h & 0xFFFF)
        code = torch.where((code == 0) & (u > 0), 1, code)   # a root above zero is not stored as zero
        out["root"] = _decode(code.to(torch.uint8), s).bfloat16()
    else:
        out.update(m=m, v=v)
    if c["master"]:
        out["master"] = w
    return out


# ----------------------------------------------------------------------------- the definitions in fp64

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"route_fwd": _exact_route, "route_bwd": _exact_route_bwd, "linear_fwd": _exact_linear,
            "linear_bwd": _exact_linear_bwd, "adamw": _exact_adamw}[case["op"]](st)


def _exact_scores(st):
    lg = st["logits"].cpu().numpy().astype(np.float64)
    if st["case"]["score"] == "sigmoid":
        return 1.0 / (1.0 + np.exp(-lg))
    e = np.exp(lg - lg.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def _exact_route(st):
    c = st["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    s = _exact_scores(st)
    choice = s + st["bias"].cpu().numpy().astype(np.float64) if "bias" in st else s.copy()
    rows = np.arange(T)
    if G > 1:
        part = np.sort(choice.reshape(T, G, E // G), axis=2)[:, :, -c["best"]:].sum(2)
        order = np.argsort(-part, axis=1, kind="stable")
        for j in range(c["top_groups"], G):
            gone = order[:, j]
            for e in range(E // G):
                choice[rows, gone * (E // G) + e] = -np.inf
    idx = np.empty((T, k), np.int64)
    for j in range(k):
        idx[:, j] = choice.argmax(1)                         # the first of equal ones
        choice[rows, idx[:, j]] = -np.inf
    gates = s[rows[:, None], idx]
    if c["renorm"]:
        gates = gates / gates.sum(1, keepdims=True)
    counts = np.bincount(idx.ravel(), minlength=E)
    slots = [np.nonzero(idx.ravel() == e)[0] for e in range(E)]
    src = np.concatenate(slots)
    dst = np.empty_like(src)
    dst[src] = np.arange(T * k)
    out = {"topk_idx": idx, "counts": counts, "offsets": np.concatenate([[0], np.cumsum(counts)]), "perm_src": src,
           "perm_dst": dst, "mx_blk_offsets": np.concatenate([[0], np.cumsum(-(-counts // 32))])}
    out = {key: torch.from_numpy(v.astype(np.int32)) for key, v in out.items()}
    out["gates"] = torch.from_numpy(gates * c["scale"])
    if "bias" in st:
        out["bias"] = st["bias"].cpu().double() + RATE * torch.from_numpy(np.sign(T * k / E - counts))
    return out


def _exact_route_bwd(st):
    c = st["case"]
    T, k, scale = c["T"], c["k"], c["scale"]
    rows = np.arange(T)[:, None]
    s, idx, dg = _exact_scores(st), st["idx"].cpu().numpy(), st["dgates"].cpu().numpy().astype(np.float64)
    sk = s[rows, idx]
    # d gate_j / d score_i, for the chosen i and j
    if c["renorm"]:
        tot = sk.sum(1)
        jac = np.eye(k)[None] / tot[:, None, None] - sk[:, :, None] / (tot * tot)[:, None, None]
    else:
        jac = np.broadcast_to(np.eye(k), (T, k, k))
    ds = np.zeros_like(s)
    ds[rows, idx] = scale * np.matmul(dg[:, None, :], jac)[:, 0]
    if c["score"] == "sigmoid":
        lg = st["logits"].cpu().numpy().astype(np.float64)
        return torch.from_numpy(ds * np.exp(-np.abs(lg)) / (1.0 + np.exp(-np.abs(lg))) ** 2)
    return torch.from_numpy(s * ds - s * (s * ds).sum(1, keepdims=True))


def _exact_act(z, act, d=False):
    if act == "none":
        return torch.ones_like(z) if d else z
    if act == "relu":
        return (z > 0).double() if d else torch.where(z > 0, z, 0.0)
    if act == "silu":
        return torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z) if d else z * torch.sigmoid(z)
    phi = 0.5 * torch.erfc(-z / math.sqrt(2.0))
    return phi + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi) if d else z * phi


def _exact_linear(st):
    c = st["case"]
    z = torch.mm(st["x"].double(), st["w"].double())
    if "b" in st:
        z += st["b"].double()
    y = _exact_act(z, c["act"])
    if "res" in st:
        y = y + st["res"].double()
    return {"y": y, "z": z} if c["save"] and c["act"] != "none" else {"y": y}


def _exact_linear_bwd(st):
    c = st["case"]
    dz = st["dy"].double()
    if "z" in st:
        dz = dz * _exact_act(st["z"].double(), c["act"], True)
    dx = torch.mm(st["w"].double(), dz.T).T
    if "in_z" in st:
        dx = dx * _exact_act(st["in_z"].double(), c["in_act"], True)
    if "dres" in st:
        dx = dx + st["dres"].double()
    return {"dx": dx, "dw": torch.mm(dz.T, st["x"].double()).T, "db": torch.mv(dz.T, dz.new_ones(c["M"]))}


def _exact_round8(x, r):
    """x in fp64 [n], n at most 32, as its block holds it: E4M3 times 2^e, up with the chance r."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    e = e - 8 + (top > 1.75 * torch.exp2(e))
    e = torch.where(top > 0, e, -127.0).clamp(-127, 127)
    y = x.abs() * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
    low = torch.floor(y / step)
    y = (low + (y / step - low + r >= 1.0)) * step
    return torch.sign(x) * y * torch.exp2(e), torch.exp2(e - 9)


def _exact_hash(i, key):
    h = (i * 0x9E3779B9 + key) % 2 ** 32
    for shift, mul in ((16, 0x7FEB352D), (15, 0x846CA68B), (16, 1)):
        h = torch.bitwise_xor(h, torch.div(h, 2 ** shift, rounding_mode="floor")) * mul % 2 ** 32
    return h


def _exact_adamw(st):
    c = st["case"]
    (b1, b2), eight = BETAS, c["bits"] == 8
    p = st["off"][-1]
    out = {"w": []}
    for name in ("m", "root" if eight else "v") + (("master",) if c["master"] else ()):
        out[name] = torch.zeros(p, dtype=torch.float64, device=DEV)
    for t, (w, g, o) in enumerate(zip(st["w"], st["g"], st["off"])):
        n, parts = w.numel(), []
        for a in range(0, n, 1 << 25):                       # a part at a time: fp64 takes room
            b = min(n, a + (1 << 25))
            lo, hi = o + a, o + _pad32(b) if b == n else o + b
            gg = g.reshape(-1)[a:b].double() * st["gscale"].double()
            if eight:
                block = lambda codes, s: (codes[lo:hi].view(torch.float8_e4m3fn).double().view(-1, 32)  # noqa: E731
                                          * torch.exp2(s[lo // 32:hi // 32].double() - 127.0)[:, None]).view(-1)[:b - a]
                m, v = block(st["m"], st["ms"]), block(st["v"], st["vs"]) ** 2
            else:
                m, v = st["m"][lo:lo + b - a].double(), st["v"][lo:lo + b - a].double()
            m, v = m + (1.0 - b1) * (gg - m), v + (1.0 - b2) * (gg * gg - v)
            ww = (st["master"][lo:lo + b - a] if c["master"] else w.reshape(-1)[a:b]).double()
            ww = ww - LR * (DECAY * ww + m / (1.0 - b1 ** STEP) / (torch.sqrt(v / (1.0 - b2 ** STEP)) + EPS))
            parts.append(ww)
            if c["master"]:
                out["master"][lo:lo + b - a] = ww
            if eight:
                key = _exact_hash(torch.tensor(STEP), _exact_hash(torch.tensor(t), st["seed"]))
                h = _exact_hash(torch.arange(a, a + hi - lo, device=DEV), int(key))
                m, u = (torch.nn.functional.pad(s, (0, hi - lo - (b - a))).view(-1, 32) for s in (m, torch.sqrt(v)))
                out["m"][lo:hi] = _exact_round8(m, ((h // 65536) + 0.5).double().view(-1, 32) / 65536.0)[0].view(-1)
                root, least = _exact_round8(u, ((h % 65536) + 0.5).double().view(-1, 32) / 65536.0)
                out["root"][lo:hi] = torch.where((root == 0) & (u > 0), least, root).view(-1)
            else:
                out["m"][lo:lo + b - a], out["v"][lo:lo + b - a] = m, v
        out["w"].append(torch.cat(parts).view(w.shape))
    return out
