"""Measured cases of two feed-forward operators: the whole mixture-of-experts layer
for a few tokens (router, routed experts, shared expert, residual in one call) and
the dense matrix product with bias, activation, gate and residual in its epilogue.

``run`` computes a case in plain torch operations where ``own`` is false, and by
the library's entry points (``MoELayer.few``, ``Linear``) where it is true.
"""
import math

import torch

own = False

# Layer widths: the sigmoid-router layer with 256 experts, the softmax-router layer
# with 128, and the small fp32 layer, as in the library's workloads.
WIDE = dict(H=2304, I=2048, E=256, k=8, router="sigmoid", scale=2.446)
SLIM = dict(H=2048, I=768, E=128, k=8, router="softmax", scale=1.0)
TINY = dict(H=256, I=128, E=16, k=4, router="sigmoid", scale=2.446)


def _few(name, base, T, wfmt, xfmt="bf16", act="silu", shared=0, residual=False, active=0):
    return dict(name=name, op="few", T=T, wfmt=wfmt, xfmt=xfmt, act=act, shared=shared, residual=residual,
                active=active, **base)


def _linear(name, M, K, N, wfmt, xfmt="bf16", yfmt="bf16", act="none", gated=False, bias=False, residual=False):
    return dict(name=name, op="linear", M=M, K=K, N=N, wfmt=wfmt, xfmt=xfmt, yfmt=yfmt, act=act, gated=gated,
                bias=bias, residual=residual)


def listed():
    return [
        # one sequence being decoded, bf16 weights, the whole block of a layer
        _few("few-1-bf16-block", WIDE, 1, "bf16", shared=2048, residual=True),
        # a few sequences decoded together, int8 weights, the whole block
        _few("few-4-int8-block", WIDE, 4, "int8", shared=2048, residual=True),
        # a small serving batch on a layer whose mask keeps 160 of the 256 experts
        _few("few-16-int8-masked", WIDE, 16, "int8", active=160),
        # one sequence, int4 weights: little to read, so latency counts
        _few("few-1-int4", SLIM, 1, "int4"),
        # a small serving batch, int4 weights
        _few("few-16-int4", SLIM, 16, "int4", residual=True),
        # the small fp32 layer: launches and latency alone
        _few("few-5-f32", TINY, 5, "f32", xfmt="f32"),
        # the dense first layer's gate and up projections for one token
        _linear("linear-1-int8-gated", 1, 2304, 9216, "int8", act="silu", gated=True),
        # its down projection into the residual stream for a few tokens
        _linear("linear-8-bf16-down", 8, 9216, 2304, "bf16", residual=True),
        # a biased, activated projection with an odd width for a batch of decoded tokens
        _linear("linear-48-int4-gelu", 48, 2048, 4999, "int4", act="gelu_tanh", bias=True),
        # the first layer's gate and up projections for a long prompt
        _linear("linear-4096-bf16-gated", 4096, 2304, 9216, "bf16", act="silu", gated=True),
        # its down projection for a prompt of odd length, quantised weights
        _linear("linear-1999-int8-down", 1999, 9216, 2304, "int8", bias=True, residual=True),
        # an fp32 projection with a ragged width
        _linear("linear-333-f32", 333, 2304, 1153, "f32", xfmt="f32", yfmt="f32", act="silu", bias=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        T = rng.randint(1, 16)
        wfmt = rng.choice(("bf16", "bf16", "int8", "int8", "int4", "int4", "int4b128", "f32"))
        kind = rng.random()
        if kind < 0.3:
            base = dict(WIDE)
        elif kind < 0.6:
            base = dict(SLIM)
        else:
            E = _log_int(rng, 8, 256)
            base = dict(H=128 * rng.randint(2, 24), I=128 * rng.randint(1, 16), E=E, k=rng.randint(1, min(8, E)),
                        router=rng.choice(("sigmoid", "softmax")), scale=rng.choice((1.0, 2.446)))
        if wfmt == "f32":
            base.update(H=128 * rng.randint(2, 12), I=128 * rng.randint(1, 6), E=min(base["E"], 64))
            base["k"] = min(base["k"], base["E"])
        active = rng.choice((0, 0, max(base["k"], base["E"] * 5 // 8)))
        case = _few("", base, T, wfmt, xfmt="f32" if wfmt == "f32" else "bf16",
                    act=rng.choice(("silu", "silu", "gelu_tanh")),
                    shared=rng.choice((0, 128 * rng.randint(1, 16))) if wfmt != "f32" else rng.choice((0, 256)),
                    residual=rng.random() < 0.5, active=0 if active >= base["E"] else active)
        while work(case)["bytes"] > 1.25e9:  # no more than the largest listed case of this operator
            case["T"] -= 1
    else:
        wfmt = rng.choice(("bf16", "bf16", "int8", "int8", "int4", "int4", "int4b128", "f32"))
        step = 128 if wfmt == "int4b128" else 64
        K = step * max(1, _log_int(rng, 128, 9216) // step)
        N = _log_int(rng, 64, 16384)
        gated = rng.random() < 0.4
        top = 16e9 if wfmt == "f32" else 1.7e11  # multiply-adds: no more than the largest listed cases
        M = _log_int(rng, 1, max(1, min(8192, int(top / 2 / (K * N * (2 if gated else 1))))))
        case = _linear("", M, K, N, wfmt, xfmt="f32" if wfmt == "f32" else "bf16",
                       yfmt="f32" if wfmt == "f32" else rng.choice(("bf16", "bf16", "f32")),
                       act=rng.choice(("none", "silu", "gelu_tanh")), gated=gated, bias=rng.random() < 0.5,
                       residual=rng.random() < 0.5)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = {"int4": 32, "int4b128": 128}


def _weights(shape, wfmt, gen, std):
    """Weights of the given standard deviation in a storage format: (values, scales).
    int8 and int4 codes have the spread that a largest-magnitude scale leaves."""
    dev = "cuda"
    if wfmt == "f32":
        return torch.empty(shape, device=dev).normal_(0, std, generator=gen), None
    if wfmt == "bf16":
        return torch.empty(shape, device=dev, dtype=torch.bfloat16).normal_(0, std, generator=gen), None
    if wfmt == "int8":
        q = torch.empty(shape, device=dev, dtype=torch.bfloat16).normal_(0, 36, generator=gen)
        s = torch.empty(shape[:-1], device=dev).uniform_(0.9, 1.1, generator=gen) * (std / 36)
        return q.round_().clamp_(-127, 127).to(torch.int8), s
    q = torch.empty(shape, device=dev, dtype=torch.bfloat16).normal_(0, 3, generator=gen)
    q = q.round_().clamp_(-8, 7).to(torch.int8).view(torch.uint8)
    s = torch.empty(shape[:-1] + (shape[-1] // BLOCK[wfmt],), device=dev).uniform_(0.6, 1.4, generator=gen) * (std / 3)
    return (q[..., 0::2] & 15) | (q[..., 1::2] << 4), s


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dev = "cuda"
    rows = c["T"] if c["op"] == "few" else c["M"]
    wide = c["H"] if c["op"] == "few" else c["K"]
    st = {"case": c, "x": torch.empty((rows, wide), device=dev).normal_(generator=gen).to(DTYPE[c["xfmt"]])}
    if c["op"] == "few":
        H, I, E, k = c["H"], c["I"], c["E"], c["k"]
        st["W_r"] = torch.empty((E, H), device=dev).normal_(0, 0.02, generator=gen)
        st["b"] = (torch.empty(E, device=dev).normal_(0, 0.05, generator=gen) if c["router"] == "sigmoid" else None)
        st["mask"] = None
        if c["active"]:
            st["mask"] = torch.zeros(E, device=dev, dtype=torch.uint8)
            st["mask"][torch.randperm(E, device=dev, generator=gen)[: c["active"]]] = 1
        for part, shape in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I))):
            st["W_" + part], st["s_" + part] = _weights((E,) + shape, c["wfmt"], gen, 0.02)
        if c["shared"]:
            for part, shape in (("gate", (c["shared"], H)), ("up", (c["shared"], H)), ("down", (H, c["shared"]))):
                st["Ws_" + part], st["ss_" + part] = _weights(shape, c["wfmt"], gen, 0.02)
        st["y"] = torch.empty((rows, H), device=dev, dtype=DTYPE[c["xfmt"]])
        st["idx"] = torch.empty((rows, k), device=dev, dtype=torch.int32)
        st["w"] = torch.empty((rows, k), device=dev)
    else:
        K, N = c["K"], c["N"]
        st["W"], st["s"] = _weights((N, K), c["wfmt"], gen, 0.02)
        st["W_up"], st["s_up"] = _weights((N, K), c["wfmt"], gen, 0.02) if c["gated"] else (None, None)
        st["b"] = torch.empty(N, device=dev).normal_(0, 0.5, generator=gen) if c["bias"] else None
        st["b_up"] = torch.empty(N, device=dev).normal_(0, 0.5, generator=gen) if c["bias"] and c["gated"] else None
        st["y"] = torch.empty((rows, N), device=dev, dtype=DTYPE[c["yfmt"]])
    st["residual"] = (torch.empty(st["y"].shape, device=dev).normal_(generator=gen).to(st["y"].dtype)
                      if c["residual"] else None)
    return st


# ---------------------------------------------------------------- the plain form

def _nibbles(q):
    """int4 pairs -> values, the even column in the low nibble."""
    both = torch.stack((q & 15, q >> 4), -1).flatten(-2).to(torch.int8)
    return torch.where(both > 7, both - 16, both)


def _dense(W, s, wfmt):
    """Stored weights -> fp32 values."""
    if wfmt in ("f32", "bf16"):
        return W.float()
    if wfmt == "int8":
        return W.float() * s[..., None]
    return _nibbles(W).float() * s.repeat_interleave(BLOCK[wfmt], -1)


def _act(v, act):
    if act == "none":
        return v
    z = v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)
    return v / (1 + torch.exp(-z))


def _plain_route(st):
    """Top k of the keys and the renormalised weights: 64 bits, since neighbouring
    keys can lie closer than fp32 sums resolve; equal keys go to the lower index."""
    c = st["case"]
    logits = st["x"].double() @ st["W_r"].double().T
    if c["router"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
        key = score + st["b"].double()
    else:
        score = torch.exp(logits - logits.max(-1, keepdim=True).values)
        key = logits
    if st["mask"] is not None:
        key = key.masked_fill(st["mask"] == 0, -math.inf)
    idx = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, : c["k"]]
    w = score.gather(-1, idx)
    w = w / w.sum(-1, keepdim=True) * c["scale"]
    return idx.to(torch.int32), w.float()


def _plain_few(st):
    c = st["case"]
    idx, w = _plain_route(st)
    x = st["x"].float()
    at = idx.long()

    def weight(part):
        s = st["s_" + part]
        return _dense(st["W_" + part][at], None if s is None else s[at], c["wfmt"])  # [T, k, rows, columns]

    gate = torch.matmul(weight("gate"), x[:, None, :, None])
    up = torch.matmul(weight("up"), x[:, None, :, None])
    out = torch.matmul(weight("down"), _act(gate, c["act"]) * up).squeeze(-1)
    y = (w[..., None] * out).sum(1)
    if c["shared"]:
        gate = x @ _dense(st["Ws_gate"], st["ss_gate"], c["wfmt"]).T
        up = x @ _dense(st["Ws_up"], st["ss_up"], c["wfmt"]).T
        y = y + (_act(gate, c["act"]) * up) @ _dense(st["Ws_down"], st["ss_down"], c["wfmt"]).T
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return {"y": y.to(st["y"].dtype), "idx": idx, "w": w}


def _plain_linear(st):
    c = st["case"]
    x = st["x"].float()
    v = x @ _dense(st["W"], st["s"], c["wfmt"]).T
    if st["b"] is not None:
        v = v + st["b"]
    y = _act(v, c["act"])
    if c["gated"]:
        u = x @ _dense(st["W_up"], st["s_up"], c["wfmt"]).T
        if st["b_up"] is not None:
            u = u + st["b_up"]
        y = y * u
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(st["y"].dtype)


# ---------------------------------------------------------------- the library's operators

def _own(st):
    import mixture_experts_layer_31_b200 as moe

    c = st["case"]
    op = st.get("handle")  # descriptors of the weights, as a program keeps them
    if op is None and c["op"] == "few":
        op = moe.MoELayer(H=c["H"], I=c["I"], E=c["E"], k=c["k"], router=c["router"], scale=c["scale"], wfmt=c["wfmt"],
                          xfmt=c["xfmt"], act=c["act"], W_r=st["W_r"], b=st["b"], expert_mask=st["mask"],
                          W_gate=st["W_gate"], W_up=st["W_up"], W_down=st["W_down"], s_gate=st["s_gate"],
                          s_up=st["s_up"], s_down=st["s_down"], I_s=c["shared"], Ws_gate=st.get("Ws_gate"),
                          Ws_up=st.get("Ws_up"), Ws_down=st.get("Ws_down"), ss_gate=st.get("ss_gate"),
                          ss_up=st.get("ss_up"), ss_down=st.get("ss_down"))
    elif op is None:
        op = moe.Linear(K=c["K"], N=c["N"], wfmt=c["wfmt"], xfmt=c["xfmt"], yfmt=c["yfmt"], act=c["act"], W=st["W"],
                        s=st["s"], b=st["b"], W_up=st["W_up"], s_up=st["s_up"], b_up=st["b_up"])
    st["handle"] = op
    if c["op"] == "few":
        y, idx, w = op.few(st["x"], residual=st["residual"], out=(st["y"], st["idx"], st["w"]))
        return {"y": y, "idx": idx, "w": w}
    return op(st["x"], residual=st["residual"], y=st["y"])


def run(st):
    if own:
        return _own(st)
    return _plain_few(st) if st["case"]["op"] == "few" else _plain_linear(st)


# ---------------------------------------------------------------- what a pass cannot do without

def _stored(rows, cols, wfmt):
    """Bytes of rows x cols stored weights with their scales."""
    n = rows * cols
    if wfmt == "f32":
        return 4.0 * n
    if wfmt == "bf16":
        return 2.0 * n
    if wfmt == "int8":
        return n + 4.0 * rows
    return 0.5 * n + 4.0 * n / BLOCK[wfmt]


def work(case):
    c = case
    if c["op"] == "few":
        T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
        among = c["active"] or E
        # experts that T tokens with k of `among` each are expected to touch
        touched = among * (1 - (1 - k / among) ** T)
        item = 4 if c["xfmt"] == "f32" else 2
        one = 2 * _stored(I, H, c["wfmt"]) + _stored(H, I, c["wfmt"])
        shared = (2 * _stored(c["shared"], H, c["wfmt"]) + _stored(H, c["shared"], c["wfmt"])) if c["shared"] else 0
        return {"bytes": touched * one + shared + 4.0 * E * H + T * H * item * (2 + bool(c["residual"])) + 8.0 * T * k,
                "flops": 2.0 * T * (E * H + 3 * H * (k * I + c["shared"]))}
    M, K, N = c["M"], c["K"], c["N"]
    sides = 2 if c["gated"] else 1
    xb, yb = (4 if c["xfmt"] == "f32" else 2), (4 if c["yfmt"] == "f32" else 2)
    return {"bytes": sides * (_stored(N, K, c["wfmt"]) + 4.0 * N * bool(c["bias"])) + M * K * xb
            + M * N * yb * (1 + bool(c["residual"])),
            "flops": 2.0 * M * N * K * sides}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_matrix(W, s, wfmt):
    if wfmt == "int8":
        return W.double() * s.double().unsqueeze(-1)
    if wfmt in BLOCK:
        v = torch.empty(W.shape[:-1] + (2 * W.shape[-1],), dtype=torch.float64, device=W.device)
        code = W.to(torch.int64)
        v[..., 0::2] = ((code % 16) + 8) % 16 - 8
        v[..., 1::2] = ((code // 16) + 8) % 16 - 8
        return (v.unflatten(-1, (-1, BLOCK[wfmt])) * s.double().unsqueeze(-1)).flatten(-2)
    return W.double()


def _exact_act(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    x = st["x"].double()
    if c["op"] == "linear":
        y = torch.nn.functional.linear(x, _exact_matrix(st["W"], st["s"], c["wfmt"]),
                                       None if st["b"] is None else st["b"].double())
        y = _exact_act(y, c["act"])
        if c["gated"]:
            y *= torch.nn.functional.linear(x, _exact_matrix(st["W_up"], st["s_up"], c["wfmt"]),
                                            None if st["b_up"] is None else st["b_up"].double())
        return y if st["residual"] is None else y + st["residual"].double()
    T, k = c["T"], c["k"]
    logits = (st["W_r"].double() @ x.T).T.cpu()
    bias = st["b"].double().cpu() if st["b"] is not None else torch.zeros(c["E"], dtype=torch.float64)
    open_ = [e for e in range(c["E"]) if st["mask"] is None or int(st["mask"][e])]
    idx = torch.zeros((T, k), dtype=torch.int32)
    w = torch.zeros((T, k), dtype=torch.float64)
    for t in range(T):
        score = torch.sigmoid(logits[t]) if c["router"] == "sigmoid" else torch.softmax(logits[t], 0)
        rank = (score + bias if c["router"] == "sigmoid" else logits[t]).tolist()
        best = sorted(open_, key=lambda e: (-rank[e], e))[:k]
        idx[t] = torch.tensor(best, dtype=torch.int32)
        w[t] = score[best] / score[best].sum() * c["scale"]

    def ffn(rows, parts):
        g, u, d = (_exact_matrix(W, s, c["wfmt"]) for W, s in parts)
        return (_exact_act(rows @ g.T, c["act"]) * (rows @ u.T)) @ d.T

    y = torch.zeros((T, c["H"]), dtype=torch.float64, device=x.device)
    for e in sorted(set(idx.flatten().tolist())):
        t, j = (idx == e).nonzero(as_tuple=True)
        at = t.to(x.device)
        one = ffn(x[at], [(st["W_" + p][e], None if st["s_" + p] is None else st["s_" + p][e])
                          for p in ("gate", "up", "down")])
        y[at] += w[t, j].to(x.device)[:, None] * one
    if c["shared"]:
        y += ffn(x, [(st["Ws_" + p], st["ss_" + p]) for p in ("gate", "up", "down")])
    if st["residual"] is not None:
        y += st["residual"].double()
    return {"y": y, "idx": idx, "w": w}
