"""Cases of two operators for serving a few tokens at a time, their plain form and their definition.

* ``few``: the whole mixture-of-experts layer for 1 to 32 tokens (``Layer.forward_few``): two-level routing, the
  shared base of each chosen group once per group, the rank-r residual of each chosen expert, and the gate-weighted
  sum.  The base is held in 32 or 16 bits, or in 4 bits with one fp16 scale per 32 input rows.
* ``matvec``: y = x W for 1 to 32 rows x, W held in 4 bits with one fp16 scale per ``group`` input rows
  (``QuantLinear.matvec``).

A case of ``few`` names the layer (T tokens, width d, hidden width f, G groups of K experts, kg groups and ke experts
per group chosen for a token, residual rank r, activation, storage types); ``prior`` scales the expert-logit prior
log(1 / (i + 1)) that makes some experts popular.  A case of ``matvec`` names T, n_in, n_out, group and the type.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases --
def _few(name, T, d, f, G, K, kg, ke, r, act, x, base, resid, prior=0.0):
    c = dict(op="few", T=T, d=d, f=f, G=G, K=K, kg=kg, ke=ke, r=r, act=act, x=x, base=base, resid=resid, prior=prior)
    return dict(c, name=name) if name else c


def _matvec(name, T, n_in, n_out, group, x):
    c = dict(op="matvec", T=T, n_in=n_in, n_out=n_out, group=group, x=x)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through a small full-precision layer: a test model's step, all latency
        _few("tiny_fp32_gelu_1", 1, 64, 128, 2, 4, 1, 2, 4, "gelu_tanh", "f32", "f32", "f32"),
        # one sequence decoding through the 256-expert layer with popular experts
        _few("decode_fp16_1", 1, 4096, 1536, 16, 16, 2, 4, 16, "swiglu", "f16", "f16", "int4_g32", 1.0),
        # sixteen sequences decoding together: most groups are touched
        _few("decode_fp16_16", 16, 4096, 1536, 16, 16, 2, 4, 16, "swiglu", "f16", "f16", "int4_g32", 1.0),
        # a few sequences on the medium layer with 16-bit residual factors
        _few("medium_fp16_5", 5, 1024, 2816, 4, 4, 1, 2, 16, "swiglu", "f16", "f16", "f16"),
        # drafted tokens of one sequence on the fine-grained layer, bf16 activations on an fp16 base
        _few("fine_bf16_7", 7, 2048, 1408, 8, 8, 1, 4, 16, "swiglu", "bf16", "f16", "int4_g32"),
        # the uncompressed top-2-of-8 layer, two sequences: the largest weights
        _few("flat_bf16_2", 2, 4096, 14336, 8, 1, 2, 1, 0, "swiglu", "bf16", "bf16", "none", 0.5),
        # one sequence decoding, the base in 4 bits too
        _few("decode_int4_base_1", 1, 4096, 1536, 16, 16, 2, 4, 16, "swiglu", "f16", "int4_g32", "int4_g32", 1.0),
        # a full batch of 32 on the fine-grained layer with a 4-bit base and bf16 activations
        _few("fine_int4_base_32", 32, 2048, 1408, 8, 8, 1, 4, 16, "swiglu", "bf16", "int4_g32", "int4_g32"),
        # a square projection of one decoded token
        _matvec("square_fp16_1", 1, 4096, 4096, 32, "f16"),
        # the wide input projection of a feed-forward block, one token, coarse groups
        _matvec("wide_bf16_1", 1, 4096, 14336, 128, "bf16"),
        # its output projection for a batch
        _matvec("deep_fp16_32", 32, 14336, 4096, 64, "f16"),
        # odd sizes: columns that end inside a tile and rows that end inside a group
        _matvec("odd_bf16_3", 3, 1419, 2005, 128, "bf16"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    T = min(32, spread(1, 33))
    if rng.random() < 0.4:
        n_in, n_out = spread(64, 16384), spread(48, 16384)
        return _matvec(None, T, n_in, n_out, rng.choice([32, 64, 128]), rng.choice(["f16", "bf16"]))
    d, f = 64 * spread(1, 64), 64 * spread(1, 48)
    G = rng.randint(1, 16)
    K = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    kg = rng.randint(1, min(G, 4))
    ke = rng.randint(1, min(K, 4))
    act = rng.choice(["swiglu", "swiglu", "gelu_tanh"])
    x, base, kinds = rng.choice([
        ("f32", "f32", ["none", "f32"]), ("f16", "f16", ["none", "f16", "int4_g32"]),
        ("bf16", "bf16", ["none", "int4_g32"]), ("bf16", "f16", ["none", "f16", "int4_g32"]),
        ("f16", "int4_g32", ["none", "int4_g32"]), ("bf16", "int4_g32", ["none", "int4_g32"])])
    resid = rng.choice(kinds)
    r = 0 if resid == "none" else rng.randint(1, 16)
    # weights up to a gigabyte
    f = min(f, 64 * max(1, int(1e9 / (3 * G * d * 64 * {"f32": 4, "f16": 2, "bf16": 2, "int4_g32": 4}[base]))))
    return _few(None, T, d, f, G, K, kg, ke, r, act, x, base, resid, rng.choice([0.0, 0.5, 1.0]))


def _dims(c):
    inputs = [(c["d"], c["f"])] * (2 if c["act"] == "swiglu" else 1)
    return inputs + [(c["f"], c["d"])]


def work(case):
    c, T = case, case["T"]
    if c["op"] == "matvec":
        groups = -(-c["n_in"] // c["group"])
        return {"bytes": c["n_in"] * c["n_out"] / 2 + groups * c["n_out"] * 2 + T * (c["n_in"] + c["n_out"]) * 2,
                "flops": 2 * T * c["n_in"] * c["n_out"]}
    size = {"f32": 4, "f16": 2, "bf16": 2, "int4_g32": 0.5 + 2 / 32, "none": 0}
    G, K, kg, ke, r = c["G"], c["K"], c["kg"], c["ke"], c["r"]
    # groups and experts that T tokens touch when every choice is as likely
    groups = G * (1 - (1 - kg / G) ** T)
    experts = G * K * (1 - (1 - kg * ke / (G * K)) ** T)
    entries = sum(a * b for a, b in _dims(c))
    edges = sum(a + b for a, b in _dims(c))
    scores = G + (groups * K if K > 1 else 0)
    return {"bytes": groups * entries * size[c["base"]] + experts * edges * r * size[c["resid"]] +
            c["d"] * scores * 4 + 2 * T * c["d"] * size[c["x"]],
            "flops": 2 * T * (kg * entries + kg * ke * (r * edges + c["f"]) + c["d"] * (G + (kg * K if K > 1 else 0)))}


# ----------------------------------------------------------------- inputs --
def _quantise(m, group=32):
    """Codes and scales of a float32 matrix [..., n, cols], n a multiple of group: scale = fp16(amax / 7), codes
    rounded half to even and clamped to [-8, 7]; a scale of zero has zero codes."""
    n, cols = m.shape[-2:]
    b = m.reshape(*m.shape[:-2], n // group, group, cols)
    scale = (b.abs().amax(dim=-2) / 7.0).to(torch.float16)
    s = scale.float().unsqueeze(-2)
    q = torch.where(s > 0, torch.round(b / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(b))
    return q.clamp(-8, 7).to(torch.int8).reshape(m.shape), scale


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        t = torch.empty(shape, dtype=dtype, device=dev)
        return t.normal_(0.0, std, generator=g)

    T, st = c["T"], {"case": c}
    if c["op"] == "matvec":
        groups = -(-c["n_in"] // c["group"])
        q = torch.randint(-8, 8, (c["n_in"], c["n_out"]), generator=g, device=dev, dtype=torch.int8)
        scale = (normal(groups, c["n_out"]).abs() * 0.2 + 0.05).div_(math.sqrt(c["n_in"])).to(torch.float16)
        st["X"] = normal(T, c["n_in"]).to(DT[c["x"]])
        if own:
            from compressed_expert_ffn_amd import _lib as L
            st["linear"] = L.QuantLinear(c["n_in"], c["n_out"], c["group"], c["x"], q=q, scale=scale)
            st["Y"] = torch.empty((T, c["n_out"]), dtype=DT[c["x"]], device=dev)
        else:
            st["q"], st["scale"] = q, scale
        return st

    d, f, G, K, r = c["d"], c["f"], c["G"], c["K"], c["r"]
    E = G * K
    st["X"] = normal(T, d).to(DT[c["x"]])
    st["W_grp"] = normal(d, G, std=1 / math.sqrt(d))
    st["W_exp"] = normal(G, d, K, std=1 / math.sqrt(d)) if K > 1 else None
    prior = c["prior"] * torch.log(1.0 / torch.arange(1, E + 1, device=dev, dtype=torch.float32))
    st["group_bias"] = torch.logsumexp(prior.reshape(G, K), dim=1) if c["prior"] else torch.zeros(G, device=dev)
    st["expert_bias"] = prior if K > 1 else None
    base_dt = torch.float32 if c["base"] == "int4_g32" else DT[c["base"]]
    fac_dt = torch.float16 if c["resid"] == "f16" else torch.float32
    st["base"] = [normal(G, a, b, std=1 / math.sqrt(a), dtype=base_dt) for a, b in _dims(c)]
    st["A"] = [normal(E, a, r, std=0.05).to(fac_dt) for a, b in _dims(c)] if r else None
    st["B"] = [normal(E, b, r, std=0.05).to(fac_dt) for a, b in _dims(c)] if r else None
    if own:
        from compressed_expert_ffn_amd import _lib as L
        cfg = L.make_config(T, d, f, G, K, c["kg"], c["ke"], r, c["act"], c["x"], c["base"], c["resid"])
        inputs = {k: st.pop(k) for k in ("W_grp", "W_exp", "group_bias", "expert_bias", "base", "A", "B")}
        # codes and scales as the plain form has them: the layer rounds their values to themselves, where it may
        # round the floats to a neighbour (a tie, or a scale's last bit)
        for k, kind in (("base", c["base"]), ("A", c["resid"]), ("B", c["resid"])):
            if kind == "int4_g32":
                inputs[k] = [_values(_quantise(m)) for m in inputs[k]]
        st["layer"] = L.Layer(cfg, inputs, on_device=True)
        st["Y"] = torch.empty((T, d), dtype=DT[c["x"]], device=dev)
        k = c["kg"] * c["ke"]
        st["route"] = {"idx": torch.empty((T, k), dtype=torch.int32, device=dev),
                       "w": torch.empty((T, k), dtype=torch.float32, device=dev)}
        return st
    if c["base"] == "int4_g32":
        st["base"] = [_quantise(b) for b in st["base"]]
    if c["resid"] == "int4_g32":
        st["A"] = [_quantise(a) for a in st["A"]]
        st["B"] = [_quantise(b) for b in st["B"]]
    return st


# ------------------------------------------------------------- plain form --
def _values(m, group=32):
    """float32 values of a stored matrix: floats, or codes with their scales."""
    if not isinstance(m, tuple):
        return m.float()
    q, s = m
    return q.float() * s.float().repeat_interleave(group, dim=-2)[..., :q.shape[-2], :]


def _take(m, at):
    return tuple(x[at] for x in m) if isinstance(m, tuple) else m[at]


def _best(v, n):
    """The n largest of each row, best first, equal ones in index order."""
    order = torch.sort(v.float(), dim=-1, descending=True, stable=True).indices[..., :n]
    return order, torch.softmax(torch.gather(v, -1, order), dim=-1)


def _plain_route(st, c):
    """idx [T, k] and gate weights [T, k]; scores in 64 bits, for they decide which expert is taken."""
    K, kg, ke, T = c["K"], c["kg"], c["ke"], c["T"]
    x = st["X"].double()
    groups, pg = _best(x @ st["W_grp"].double() + st["group_bias"].double(), kg)
    if K == 1:
        return groups, groups.to(torch.int32), pg.float()
    W = st["W_exp"].double()[groups]  # [T, kg, d, K]
    e = torch.matmul(x[:, None, None, :], W).squeeze(2) + st["expert_bias"].double().reshape(-1, K)[groups]
    pick, pe = _best(e, ke)
    idx = groups[:, :, None] * K + pick
    return groups, idx.reshape(T, kg * ke).to(torch.int32), (pg[:, :, None] * pe).reshape(T, kg * ke).float()


def _plain_few(st):
    c = st["case"]
    T, G, K, kg, ke, r = c["T"], c["G"], c["K"], c["kg"], c["ke"], c["r"]
    groups, idx, w = _plain_route(st, c)
    x, dev = st["X"].float(), st["X"].device
    # gate weight of every expert for every token, [T, G, K]
    gate = torch.zeros((T, G * K), device=dev).scatter_(1, idx.long(), w).reshape(T, G, K)
    if T * kg < G:  # one entry per (token, chosen group)
        sel = groups.reshape(-1)
        mine = torch.arange(T, device=dev).repeat_interleave(kg)[:, None] == torch.arange(T, device=dev)[None]
    else:  # one entry per group, shared by its tokens
        sel = torch.arange(G, device=dev)
        mine = torch.ones((G, T), dtype=torch.bool, device=dev)
    share = (gate[:, sel] * mine.t()[:, :, None]).permute(1, 2, 0)  # [S, K, T]
    S = sel.shape[0]
    experts = (sel[:, None] * K + torch.arange(K, device=dev)).reshape(-1)
    zs = [torch.matmul(x, _values(_take(b, sel)))[:, None].expand(S, K, T, c["f"]) for b in st["base"][:-1]]
    if r:
        rest = [torch.matmul(torch.matmul(x, _values(_take(a, experts))), _values(_take(b, experts)).transpose(1, 2).contiguous())
                for a, b in zip(st["A"][:-1], st["B"][:-1])]
        zs = [z + u.reshape(S, K, T, c["f"]) for z, u in zip(zs, rest)]
    if c["act"] == "swiglu":
        h = zs[0] / (1 + torch.exp(-zs[0])) * zs[1]
    else:
        z = zs[0]
        h = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    h = h * share[..., None]
    y = torch.matmul(h.sum(dim=1), _values(_take(st["base"][-1], sel))).sum(dim=0)
    if r:
        v = torch.matmul(h.reshape(S * K, T, c["f"]), _values(_take(st["A"][-1], experts)))
        y = y + torch.matmul(v, _values(_take(st["B"][-1], experts)).transpose(1, 2).contiguous()).sum(dim=0)
    return {"y": y.to(st["X"].dtype), "idx": idx, "w": w}


def run(state):
    c = state["case"]
    if c["op"] == "matvec":
        if own:
            return {"y": state["linear"].matvec(state["X"], state["Y"])}
        return {"y": torch.matmul(state["X"].float(), _values((state["q"], state["scale"]), c["group"])).to(DT[c["x"]])}
    if own:
        y = state["layer"].forward_few(state["X"], state["Y"], route_bufs=state["route"])
        return {"y": y, "idx": state["route"]["idx"], "w": state["route"]["w"]}
    return _plain_few(state)


# ------------------------------------------------------------- definition --
def _stored64(m, i, group=32):
    """Matrix i of a stored stack, in 64 bits."""
    if isinstance(m, tuple):
        q, s = m[0][i].double(), m[1][i].double()
        rows = torch.arange(q.shape[0], device=q.device) // group
        return q * s[rows]
    return m[i].double()


def _top64(v, n):
    left, out = v.clone(), []
    for _ in range(n):
        i = int(torch.argmax(left))
        out.append(i)
        left[i] = -math.inf
    p = torch.exp(v[out] - v[out].max())
    return out, p / p.sum()


def exact(case, seed):
    global own
    c, kept, own = case, own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    x = st["X"].double()
    if c["op"] == "matvec":
        rows = torch.arange(c["n_in"], device=x.device) // c["group"]
        return {"y": x @ (st["q"].double() * st["scale"].double()[rows])}
    K, T = c["K"], c["T"]
    y, w = torch.zeros_like(x), torch.zeros((T, c["kg"] * c["ke"]), dtype=torch.float64, device=x.device)
    W = {}
    for t in range(T):
        groups, pg = _top64(x[t] @ st["W_grp"].double() + st["group_bias"].double(), c["kg"])
        for a, g in enumerate(groups):
            picks, pe = [0], torch.ones(1, dtype=torch.float64, device=x.device)
            if K > 1:
                picks, pe = _top64(x[t] @ st["W_exp"][g].double() + st["expert_bias"][g * K:(g + 1) * K].double(), c["ke"])
            if len(W) > 24:
                W.clear()
            if g not in W:
                W[g] = [_stored64(b, g) for b in st["base"]]
            for b, j in enumerate(picks):
                # the expert's residual, materialised: row vectors times (base + A B^T)
                def through(v, p):
                    out = v @ W[g][p]
                    if c["r"]:
                        out = out + v @ (_stored64(st["A"][p], g * K + j) @ _stored64(st["B"][p], g * K + j).T)
                    return out
                z = through(x[t], 0)
                if c["act"] == "swiglu":
                    h = z * torch.sigmoid(z) * through(x[t], 1)
                else:
                    h = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
                w[t, a * c["ke"] + b] = pg[a] * pe[b]
                y[t] += w[t, a * c["ke"] + b] * through(h, len(W[g]) - 1)
    return {"y": y, "w": w, "idx": None}
