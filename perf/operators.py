"""Cases of the operators around the layer: the block's norms, tokens sorted by
expert and back, and products with 4-bit weights.

Each case runs either the plain form (elementary torch operations in 32 bits)
or, with `own`, this framework's kernels on the same inputs.

  norm       out = x + c * gate * RMSNorm(y) * g_post, h = RMSNorm(out) * g_pre
  norm_bwd   its gradients
  dispatch   (token, expert) pairs in expert order, and the tokens' rows copied
             into that order
  combine    back to token order, weighted and added to a base
  combine_bwd  gradients of the rows and of the weights
  q4         y = x W^T, W[n][k] = scale[n][k / group] * (code[n][k] - zero[n][k / group])
  q4_experts the same with each row's own expert's W

Packed codes: K is padded to Kp, a multiple of 128; a block of 128 codes is 16
little-endian 32-bit words of 8 codes, word w of the block (codes 8 w .. 8 w + 7)
stored at place 4 (w % 4) + w // 4; in a word, code 2 i sits in bits 4 i .. 4 i + 3
and code 2 i + 1 in bits 16 + 4 i .. 19 + 4 i.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token through the norms around the layer at the edge layer's width: a decode step, latency alone
        dict(name="norm_decode", kind="norm", T=1, D=2048, dtype="bf16", gate="channel"),
        # a prompt through the larger layer's block, with a gate of its own for every token and channel
        dict(name="norm_prompt", kind="norm", T=4096, D=4096, dtype="bf16", gate="full"),
        # a ragged batch of an odd width in fp32 (no row starts on a 16-byte boundary but the first), one gate a token
        dict(name="norm_odd_f32", kind="norm", T=777, D=1001, dtype="f32", gate="token"),
        # the backward pass of a training step over the edge layer's block, per-channel gate
        dict(name="norm_train", kind="norm_bwd", T=8192, D=2048, dtype="bf16", gate="channel"),
        # 16 tokens of a decode batch routed by a ReLU router (a mask, about 20 % of 64 experts)
        dict(name="dispatch_decode", kind="dispatch", T=16, D=2048, E=64, K=0, ratio=0.2, dtype="bf16"),
        # a prompt of 4096 tokens, 13 experts each (20 % of 64), as lists of expert numbers
        dict(name="dispatch_prompt", kind="dispatch", T=4096, D=2048, E=64, K=13, ratio=1.0, dtype="bf16"),
        # the larger layer's rows back to token order, 26 of 128 experts each, added to the shared expert's output
        dict(name="combine_prompt", kind="combine", T=2048, D=4096, E=128, K=26, ratio=1.0, dtype="bf16"),
        # the backward pass of that for a ragged fp32 batch under a ReLU router's mask
        dict(name="combine_train", kind="combine_bwd", T=1021, D=2048, E=64, K=0, ratio=0.2, dtype="f32"),
        # one token through a small 4-bit matrix: the shared expert's down-projection
        dict(name="q4_one_token", kind="q4", T=1, N=2048, K=1024, group=128, zero=False, dtype="bf16"),
        # 16 tokens through the equal-parameter dense FFN's up-projection
        dict(name="q4_dense", kind="q4", T=16, N=17408, K=2048, group=64, zero=False, dtype="bf16"),
        # 16 tokens through the up-projections of the experts that a ReLU router activates
        dict(name="q4_experts", kind="q4_experts", T=16, E=64, N=256, K=2048, group=64, zero=False, ratio=0.2, dtype="bf16"),
        # odd sizes, fp32 activations, small groups with zero points, experts without rows
        dict(name="q4_experts_odd", kind="q4_experts", T=37, E=10, N=333, K=1056, group=32, zero=True, ratio=0.3, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: a multiple of 64 two times in three, else any number."""
    d = _log_int(rng, lo, hi)
    return max(64, d // 64 * 64) if rng.random() < 2 / 3 else d


def draw(rng):
    kind = rng.choice(["norm", "norm_bwd", "dispatch", "combine", "combine_bwd", "q4", "q4_experts"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("norm", "norm_bwd"):
        D = _width(rng, 64, 8192)
        T = _log_int(rng, 1, min(16384, (1 << 23) // D))
        return dict(kind=kind, T=T, D=D, dtype=dtype, gate=rng.choice(["none", "channel", "token", "full"]))
    if kind in ("dispatch", "combine", "combine_bwd"):
        D, E = _width(rng, 64, 4096), _log_int(rng, 4, 256)
        mask = rng.random() < 0.5
        K = 0 if mask else rng.randint(1, min(E, 32))
        T = _log_int(rng, 1, max(1, min(8192, (1 << 25) // (D * (E if mask else K)))))
        return dict(kind=kind, T=T, D=D, E=E, K=K, ratio=rng.choice([0.05, 0.2, 0.4]) if mask else rng.choice([0.8, 1.0]), dtype=dtype)
    K = _width(rng, 64, 8192)
    group, zero = rng.choice([32, 64, 128]), rng.random() < 0.5
    if kind == "q4":
        N = _log_int(rng, 16, min(20000, (1 << 25) // K))
        return dict(kind=kind, T=_log_int(rng, 1, 32), N=N, K=K, group=group, zero=zero, dtype=dtype)
    E = _log_int(rng, 4, 128)
    N = _log_int(rng, 16, max(16, min(4096, (1 << 25) // (K * E))))
    return dict(kind=kind, T=_log_int(rng, 1, 48), E=E, N=N, K=K, group=group, zero=zero, ratio=rng.choice([0.1, 0.2, 0.5]), dtype=dtype)


# ---- inputs ---------------------------------------------------------------

def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _pairs(c, g):
    """The routing of a batch: a mask [T][E], or expert numbers [T][K] (-1: an
    empty slot); and the expert of every slot, -1 where there is none."""
    T, E, K = c["T"], c["E"], c["K"]
    if K == 0:
        active = (_rand(g, T, E) < c["ratio"]).to(torch.uint8)
        return {"active": active}, torch.where(active > 0, torch.arange(E, device="cuda"), -1)
    ids = _rand(g, T, E).topk(K, dim=1).indices
    ids = torch.where(_rand(g, T, K) < c["ratio"], ids, -1)
    return {"experts": ids.to(torch.int32)}, ids


def _order(expert, E):
    """Sorted row of every slot (-1: none), slot of every row, offsets, number of pairs."""
    e = expert.reshape(-1)
    n = e.numel()
    key = torch.where(e < 0, E, e)
    order = torch.sort(key, stable=True).indices
    rank = torch.empty_like(order)
    rank[order] = torch.arange(n, device=e.device)
    counts = (key[:, None] == torch.arange(E, device=e.device)).sum(0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=e.device), counts.cumsum(0)])
    return torch.where(e < 0, -1, rank).to(torch.int32), order.to(torch.int32), counts.to(torch.int32), offsets.to(torch.int32)


def _pack(codes):
    """codes [..][Kp] (0..15) in the packed layout, [..][Kp / 2] bytes."""
    w = codes.to(torch.int32).unflatten(-1, (-1, 4, 4, 4, 2))         # block, w // 4, w % 4, i, code 2 i + (0 or 1)
    bits = torch.arange(4, device=w.device, dtype=torch.int32) * 4
    lo, hi = (w[..., 0] << bits).sum(-1), (w[..., 1] << bits).sum(-1)
    words = (lo + (hi << 16)).to(torch.int32).transpose(-1, -2).contiguous()   # 4 (w % 4) + w // 4
    return words.view(torch.uint8).flatten(-3)


def _codes(q):
    """The codes of the packed layout, [..][Kp], as 32-bit floats."""
    w = q.unflatten(-1, (-1, 64)).view(torch.int32).unflatten(-1, (4, 4)).transpose(-1, -2)
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=q.device, dtype=torch.int32)
    return ((w.unsqueeze(-1) >> shift) & 15).flatten(-4).float()


def _weights(c, g, *lead):
    """4-bit weights [..][N][K] of about unit gain, as their packed form."""
    K, group = c["K"], c["group"]
    Kp = -(-K // 128) * 128
    codes = (_randn(g, *lead, Kp) * 2.4 + 8).round_().clamp_(0, 15)
    codes[..., K:] = 0
    scale = ((_rand(g, *lead, Kp // group) + 0.5) / (2.4 * math.sqrt(K))).to(torch.bfloat16)
    zero = torch.randint(5, 11, (*lead, Kp // group), generator=g, device="cuda").to(torch.uint8) if c["zero"] else None
    return dict(q=_pack(codes), scale=scale, zero=zero, K=K, group=group)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, kind = DT[c["dtype"]], c["kind"]
    s = dict(case=c)
    if kind in ("norm", "norm_bwd"):
        T, D = c["T"], c["D"]
        s["x"], s["y"] = _randn(g, T, D, std=3.0, dtype=dt), _randn(g, T, D, dtype=dt)
        s["g_pre"], s["g_post"] = 1 + _randn(g, D, std=0.1), 1 + _randn(g, D, std=0.1)
        shape = {"none": None, "channel": (D,), "token": (T,), "full": (T, D)}[c["gate"]]
        s["gate"] = None if shape is None else _randn(g, *shape, std=0.3, dtype=dt if c["gate"] == "full" else torch.float32)
        s["branch_scale"] = 0.5
        if kind == "norm_bwd":      # x is the sum that the forward pass stored
            s["dout"], s["dh"] = _randn(g, T, D, dtype=dt), _randn(g, T, D, dtype=dt)
    elif kind in ("dispatch", "combine", "combine_bwd"):
        T, D, E = c["T"], c["D"], c["E"]
        how, expert = _pairs(c, g)
        S = expert.shape[1]
        if kind == "dispatch":
            s["x"], s["how"] = _randn(g, T, D, dtype=dt), how
            i32 = dict(dtype=torch.int32, device="cuda")
            # buffers that a program keeps from call to call; rows behind the last pair keep what they held
            s["out"] = dict(xs=torch.zeros(T * S, D, dtype=dt, device="cuda"), counts=torch.zeros(E, **i32), offsets=torch.zeros(E + 1, **i32),
                            row_of=torch.zeros(T, S, **i32), slot_of=torch.zeros(T * S, **i32), n_pairs=torch.zeros(1, **i32))
        else:
            row_of = _order(expert, E)[0].view(T, S)
            n = min(T * S, int(1.5 * T * S * c["ratio"]) + 64)          # room for more pairs than a ReLU router is likely to make
            s["row_of"], s["ys"], s["w"] = row_of, _randn(g, n, D, dtype=dt), _rand(g, T, S) + 0.1
            if kind == "combine":
                s["base"] = _randn(g, T, D, dtype=dt)
            else:
                s["dy"], s["dys"] = _randn(g, T, D, dtype=dt), torch.zeros(n, D, dtype=dt, device="cuda")
    elif kind == "q4":
        s["x"], s["W"] = _randn(g, c["T"], c["K"], dtype=dt), _weights(c, g, c["N"])
        s["y"] = torch.zeros(c["T"], c["N"], dtype=dt, device="cuda")
    else:
        T, E, N = c["T"], c["E"], c["N"]
        s["x"], s["W"] = _randn(g, T, c["K"], dtype=dt), _weights(c, g, E, N)
        active = _rand(g, T, E) < c["ratio"]
        active[:, E // 2] = False                                   # an expert without rows
        expert = torch.where(active, torch.arange(E, device="cuda"), -1)
        _, slot_of, _, s["offsets"] = _order(expert, E)
        s["perm"] = slot_of // E                                    # token of every sorted row, as the router's tables give it
        s["y"] = torch.zeros(T * E, N, dtype=torch.float32, device="cuda")   # rows behind the last pair keep what they held
    return s


# ---- plain forms ------------------------------------------------------------

def _rms(v, eps=EPS):
    return v * (v.square().mean(-1, keepdim=True) + eps).rsqrt()


def _gate(s, f):
    gate = s["gate"]
    if gate is None:
        return 1.0
    return gate.to(f)[:, None] if s["case"]["gate"] == "token" else gate.to(f)


def _plain_norm(s):
    f, dt = torch.float32, s["x"].dtype
    out = (s["x"].to(f) + s["branch_scale"] * _gate(s, f) * _rms(s["y"].to(f)) * s["g_post"]).to(dt)
    return {"out": out, "h": (_rms(out.to(f)) * s["g_pre"]).to(dt)}


def _rms_bwd(v, dn):
    """The gradient of RMSNorm at v, given that of its output, and the output."""
    r = (v.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = v * r
    return r * (dn - n * (dn * n).mean(-1, keepdim=True)), n


def _plain_norm_bwd(s):
    f, dt = torch.float32, s["x"].dtype
    dh, c, kind = s["dh"].to(f), s["branch_scale"], s["case"]["gate"]
    dx, n = _rms_bwd(s["x"].to(f), dh * s["g_pre"])
    dx = dx + s["dout"].to(f)
    gate = _gate(s, f)
    y = s["y"].to(f)
    dy, m = _rms_bwd(y, c * dx * gate * s["g_post"])
    r = {"dx": dx.to(dt), "dy": dy.to(dt), "dg_pre": (dh * n).sum(0), "dg_post": (c * dx * gate * m).sum(0)}
    full = c * dx * m * s["g_post"]
    if kind != "none":
        r["dgate"] = full.sum(0) if kind == "channel" else full.sum(1) if kind == "token" else full.to(dt)
    return r


def _plain_dispatch(s):
    c, how, o = s["case"], s["how"], s["out"]
    E = c["E"]
    expert = torch.where(how["active"] > 0, torch.arange(E, device="cuda"), -1) if "active" in how else how["experts"].long()
    row_of, order, counts, offsets = _order(expert, E)
    n = offsets[-1:]
    ok = torch.arange(order.numel(), device="cuda") < n
    xs = torch.where(ok[:, None], s["x"][(order // expert.shape[1]).long()], o["xs"])
    return dict(xs=xs, counts=counts, offsets=offsets, row_of=row_of.view(expert.shape), slot_of=torch.where(ok, order, o["slot_of"]), n_pairs=n)


def _plain_combine(s):
    row_of, f = s["row_of"], torch.float32
    ok = row_of >= 0
    rows = s["ys"][row_of.clamp(min=0).long()].to(f)
    w = torch.where(ok, s["w"], 0)
    return {"y": (s["base"].to(f) + (w[:, :, None] * rows).sum(1)).to(s["ys"].dtype)}


def _plain_combine_bwd(s):
    row_of, f, dt = s["row_of"], torch.float32, s["ys"].dtype
    T, S = row_of.shape
    ok = row_of >= 0
    rows = s["ys"][row_of.clamp(min=0).long()].to(f)
    dw = torch.where(ok, (rows * s["dy"].to(f)[:, None, :]).sum(-1), 0)
    n = s["ys"].shape[0]
    slot = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    slot[torch.where(ok, row_of, n).reshape(-1).long()] = torch.arange(T * S, device="cuda")
    slot = slot[:n]
    dys = (s["w"].reshape(-1)[slot][:, None] * s["dy"].to(f)[slot // S]).to(dt)
    return {"dys": torch.where((torch.arange(n, device="cuda") < ok.sum())[:, None], dys, s["dys"]), "dw": dw}


def _plain_weights(W):
    codes = _codes(W["q"]).unflatten(-1, (-1, W["group"]))
    w = W["scale"].float()[..., None] * (codes - (8.0 if W["zero"] is None else W["zero"].float()[..., None]))
    return w.flatten(-2)[..., : W["K"]]


def _plain_q4(s):
    return {"y": (s["x"].float() @ _plain_weights(s["W"]).T).to(s["y"].dtype)}


def _plain_q4_experts(s):
    c, off = s["case"], s["offsets"].long()
    T, E = c["T"], c["E"]
    i = torch.arange(T * E, device="cuda")
    ok = i < off[-1]
    e = torch.searchsorted(off, i, right=True).sub(1).clamp(0, E - 1)   # expert of every row
    at = e * T + (i - off[e]).clamp(0, T - 1)                           # its place among at most T rows of that expert
    xp = torch.zeros(E * T + 1, c["K"], device="cuda")
    xp[torch.where(ok, at, E * T)] = s["x"].float()[s["perm"].long()]
    y = torch.bmm(xp[:-1].view(E, T, -1), _plain_weights(s["W"]).transpose(1, 2)).reshape(E * T, -1)
    return {"y": torch.where(ok[:, None], y[at], s["y"])}


# ---- this framework's kernels -------------------------------------------------

def _gate_kind(c):
    """The gate's kind, where a batch of as many tokens as channels leaves it open."""
    return {"gate_kind": c["gate"]} if c["T"] == c["D"] and c["gate"] in ("channel", "token") else {}


def _own(s):
    import sparse_moe_ffn_relu_b200 as deco

    kind = s["case"]["kind"]
    if kind == "norm":
        out, h = deco.block_norm(s["x"], s["g_pre"], y=s["y"], g_post=s["g_post"], gate=s["gate"], branch_scale=s["branch_scale"], eps=EPS,
                                **_gate_kind(s["case"]))
        return {"out": out, "h": h}
    if kind == "norm_bwd":
        return deco.block_norm_backward(s["x"], s["g_pre"], y=s["y"], g_post=s["g_post"], gate=s["gate"], branch_scale=s["branch_scale"], eps=EPS,
                                        dout=s["dout"], dh=s["dh"], **_gate_kind(s["case"]))
    if kind == "dispatch":
        return deco.dispatch(s["x"], E=s["case"]["E"], out=s["out"], **s["how"])
    if kind == "combine":
        return {"y": deco.combine(s["ys"], s["row_of"], w=s["w"], base=s["base"])}
    if kind == "combine_bwd":
        dys, dw = deco.combine_backward(s["ys"], s["row_of"], s["w"], s["dy"], dys=s["dys"])
        return {"dys": dys, "dw": dw}
    if kind == "q4":
        return {"y": deco.q4_matvec(s["x"], s["W"], out=s["y"])}
    return {"y": deco.q4_expert_matvec(s["x"], s["W"], s["offsets"], perm=s["perm"], out=s["y"])}


_PLAIN = dict(norm=_plain_norm, norm_bwd=_plain_norm_bwd, dispatch=_plain_dispatch, combine=_plain_combine, combine_bwd=_plain_combine_bwd,
              q4=_plain_q4, q4_experts=_plain_q4_experts)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["kind"]](state)


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    c = case
    kind, b = c["kind"], 4 if c["dtype"] == "f32" else 2
    if kind in ("norm", "norm_bwd"):
        n = c["T"] * c["D"]
        gate = {"none": 0, "channel": 4 * c["D"], "token": 4 * c["T"], "full": n * b}[c["gate"]]
        if kind == "norm":
            return {"bytes": 4 * n * b + 8 * c["D"] + gate, "flops": 12 * n}
        return {"bytes": 6 * n * b + 16 * c["D"] + 2 * gate, "flops": 30 * n}
    if kind in ("dispatch", "combine", "combine_bwd"):
        slots = c["T"] * (c["K"] or c["E"])
        rows, row = slots * c["ratio"], c["D"] * b
        if kind == "dispatch":
            return {"bytes": c["T"] * row + rows * row + slots * (1 if c["K"] == 0 else 4) + 4 * (slots + rows), "flops": 0}
        if kind == "combine":
            return {"bytes": 2 * c["T"] * row + rows * row + 8 * slots, "flops": 2 * rows * c["D"]}
        return {"bytes": c["T"] * row + 2 * rows * row + 12 * slots, "flops": 3 * rows * c["D"]}
    w = c["N"] * c["K"] * (0.5 + (3 if c["zero"] else 2) / c["group"])
    if kind == "q4":
        return {"bytes": w + c["T"] * (c["K"] + c["N"]) * b, "flops": 2 * c["T"] * c["N"] * c["K"]}
    rows = c["T"] * (c["E"] - 1) * c["ratio"]
    used = (c["E"] - 1) * (1 - (1 - c["ratio"]) ** c["T"])
    return {"bytes": used * w + c["T"] * c["K"] * b + rows * (4 * c["N"] + 4), "flops": 2 * rows * c["N"] * c["K"]}


# ---- the definition in 64 bits ----------------------------------------------------

def _exact_norm(s):
    d = torch.float64
    x, y = s["x"].to(d), s["y"].to(d)
    gate = s["gate"]
    gate = torch.ones((), dtype=d, device="cuda") if gate is None else gate.to(d).reshape(-1, 1) if s["case"]["gate"] == "token" else gate.to(d)
    D = x.shape[1]
    ry = torch.sqrt(torch.linalg.vector_norm(y, dim=1, keepdim=True) ** 2 / D + EPS)
    return x, y, gate, ry, x + s["branch_scale"] * (gate * (s["g_post"].to(d) * (y / ry)))


def exact(case, seed):
    s = prepare(case, seed)
    d, kind = torch.float64, case["kind"]
    if kind == "norm":
        x, y, gate, ry, out = _exact_norm(s)
        ro = torch.sqrt((out * out).sum(1, keepdim=True) / case["D"] + EPS)
        return {"out": out, "h": out / ro * s["g_pre"].to(d)}
    if kind == "norm_bwd":
        # gradients by the chain rule, written with the Jacobian of v / |v|_rms: (I - v v^T / (D r^2)) / r
        x, y, gate, ry, _ = _exact_norm(s)
        D, c = case["D"], s["branch_scale"]
        rx = torch.sqrt((x * x).sum(1, keepdim=True) / D + EPS)
        a = s["dh"].to(d) * s["g_pre"].to(d)
        dx = s["dout"].to(d) + a / rx - x * ((a * x).sum(1, keepdim=True) / (D * rx ** 3))
        b = dx * gate * s["g_post"].to(d) * c
        r = {"dx": dx, "dy": b / ry - y * ((b * y).sum(1, keepdim=True) / (D * ry ** 3))}
        r["dg_pre"] = torch.einsum("td,td->d", s["dh"].to(d), x / rx)
        r["dg_post"] = torch.einsum("td,td->d", dx * gate, y / ry) * c
        u = dx * (y / ry) * s["g_post"].to(d) * c
        if case["gate"] != "none":
            r["dgate"] = {"channel": lambda: u.sum(0), "token": lambda: u.sum(1), "full": lambda: u}[case["gate"]]()
        return r
    if kind == "dispatch":
        E, how, o = case["E"], s["how"], s["out"]
        T, S = o["row_of"].shape
        hit = [(how["active"][:, e] > 0).nonzero()[:, 0] * S + e if "active" in how else (how["experts"].reshape(-1) == e).nonzero()[:, 0] for e in range(E)]
        slots = torch.cat(hit)
        counts = torch.tensor([len(h) for h in hit], device="cuda")
        row_of = torch.full((T * S,), -1, device="cuda")
        row_of[slots] = torch.arange(len(slots), device="cuda")
        xs, slot_of = o["xs"].clone(), o["slot_of"].clone()
        xs[: len(slots)] = s["x"][slots // S]
        slot_of[: len(slots)] = slots.to(torch.int32)
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
        return dict(xs=xs.to(d), counts=counts.int(), offsets=offsets.int(), row_of=row_of.view(T, S).int(), slot_of=slot_of, n_pairs=offsets[-1:].int())
    if kind in ("combine", "combine_bwd"):
        row_of, ys = s["row_of"], s["ys"]
        t, k = (row_of >= 0).nonzero(as_tuple=True)
        rows = row_of[t, k].long()
        w = s["w"][t, k].to(d)
        if kind == "combine":
            y = s["base"].to(d)
            for at in range(0, len(t), 1 << 14):           # a slice of pairs at a time: the rows in 64 bits are large
                m = slice(at, at + (1 << 14))
                y.index_add_(0, t[m], ys[rows[m]].to(d) * w[m, None])
            return {"y": y}
        dys, dw = s["dys"].to(d), torch.zeros(row_of.shape, dtype=d, device="cuda")
        for at in range(0, len(t), 1 << 14):
            m = slice(at, at + (1 << 14))
            dy = s["dy"][t[m]].to(d)
            dys[rows[m]] = w[m, None] * dy
            dw[t[m], k[m]] = torch.einsum("pd,pd->p", dy, ys[rows[m]].to(d))
        return {"dys": dys, "dw": dw}
    W, K, group = s["W"], case["K"], case["group"]
    b = W["q"].to(torch.int64)
    k = torch.arange(K, device="cuda")
    word, i = k % 128 // 8, k % 8
    bit = (k // 128 * 16 + 4 * (word % 4) + word // 4) * 32 + 4 * (i // 2) + 16 * (i % 2)    # of a row
    code = (b[..., bit // 8] >> (bit % 8)) & 15
    zero = torch.tensor(8, device="cuda") if W["zero"] is None else W["zero"].to(torch.int64)[..., k // group]
    w = (code - zero).to(d) * W["scale"].to(d)[..., k // group]
    if kind == "q4":
        return {"y": torch.einsum("tk,nk->tn", s["x"].to(d), w)}
    y, off = s["y"].to(d), s["offsets"].tolist()
    for e in range(case["E"]):
        y[off[e]:off[e + 1]] = s["x"][s["perm"][off[e]:off[e + 1]].long()].to(d) @ w[e].T
    return {"y": y}
