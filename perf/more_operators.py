"""What scored routing and bf16 products with an epilogue cost, case by case.

Three families:

* ``select``: experts chosen from given router logits: sigmoid or softmax
  scores, a bias that takes part in the choice alone (load balance), groups of
  experts of which the best few stay, top-k, weights renormalised and scaled;
* ``gemm``: bf16 products with bias, activation and residual in the epilogue,
  for one weight matrix or for ragged expert segments;
* ``layer``: both as one decode step uses them: a rank's share of an MoE layer
  with scored routing, plus the expert that every token shares.

``run`` computes a case in plain torch operations, or, where ``own`` is true,
through the package's entry points.
"""
import torch

own = False


def _select(name, T, E, k, score, G=1, top=1, rule="max", bias=True, renorm=True, scale=1.0):
    return {"name": name, "op": "select", "T": T, "E": E, "k": k, "score": score, "G": G, "top": top, "rule": rule,
            "bias": bias, "renorm": renorm, "scale": scale}


def _gemm(name, M, K, N, act="none", bias=False, res="none", out="bf16", El=0, even=True):
    """El = 0: one matrix; else M rows in segments of El experts. N outputs."""
    return {"name": name, "op": "gemm", "M": M, "K": K, "N": N, "act": act, "bias": bias, "res": res, "out": out,
            "El": El, "even": even}


def listed():
    return [
        # one decode token of the DeepSeek-R1-shaped router: 8 groups, 4 stay
        _select("select_dsr1_t1", 1, 256, 8, "sigmoid", 8, 4, "top2", scale=2.5),
        # a prefill batch of it
        _select("select_dsr1_t16384", 16384, 256, 8, "sigmoid", 8, 4, "top2", scale=2.5),
        # an odd batch, an expert count that is no power of two, plain softmax
        # probabilities of the groups' best experts
        _select("select_e160_t1001", 1001, 160, 6, "softmax", 8, 3, "max", bias=False, renorm=False, scale=16.0),
        # a decode token through a shared expert's gate and up projections
        _gemm("gemm_gate_up_m1", 1, 7168, 2048, act="swiglu"),
        # its down projection for a small batch, onto the float32 share
        _gemm("gemm_down_m16", 16, 2048, 7168, res="f32", out="f32"),
        # an odd batch through a GPT-OSS-20B-shaped slice with bias (EP=2 x TP=4)
        _gemm("gemm_bias_gelu_m333", 333, 2880, 1536, act="gelu", bias=True, res="bf16"),
        # a prefill chunk through a dense gate and up projection
        _gemm("gemm_gate_up_m8192", 8192, 7168, 2048, act="swiglu"),
        # and its down projection onto the bf16 residual stream
        _gemm("gemm_down_m8192", 8192, 2048, 7168, res="bf16"),
        # a decode batch's rows on the GPT-OSS-20B-shaped EP=2 x TP=4 experts, with bias
        _gemm("gemm_experts_r61", 61, 2880, 768, act="swiglu", bias=True, El=16, even=False),
        # a prefill chunk's rows on the DeepSeek-R1-shaped EP=8 rank's experts, with bias
        _gemm("gemm_experts_r16384", 16384, 7168, 2048, act="swiglu", bias=True, El=32),
        # one token through the DeepSeek-R1-shaped layer, every expert cut to an
        # eighth of its intermediate size (EP=1 x TP=8), the shared one too
        {"name": "layer_dsr1_tp8_t1", "op": "layer", "T": 1, "H": 7168, "I": 256, "Is": 256, "E": 256, "El": 256,
         "e0": 0, "k": 8, "score": "sigmoid", "G": 8, "top": 4, "rule": "top2", "scale": 2.5},
        # a decode batch on its EP=8 rank share
        {"name": "layer_dsr1_ep8_t16", "op": "layer", "T": 16, "H": 7168, "I": 2048, "Is": 2048, "E": 256, "El": 32,
         "e0": 64, "k": 8, "score": "sigmoid", "G": 8, "top": 4, "rule": "top2", "scale": 2.5},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return max(lo, min(hi, int(round(v))))


def _groups(rng, E, most):
    """Groups, how many stay, and the rule, for E experts; at most `most` groups."""
    G = rng.choice([g for g in range(1, most + 1) if E % g == 0])
    return G, rng.randint(1, G), rng.choice(["max", "top2"])


def _used(T, E, El, k):
    """Local experts that at least one of T tokens selects, expected for even routing."""
    return El * (1.0 - (1.0 - k / E) ** T)


def draw(rng):
    op = rng.choice(["select", "select", "gemm", "gemm", "gemm", "experts", "experts", "layer"])
    if op == "select":
        T = _log_int(rng, 1, 16384)
        E = rng.choice([32, 64, 128, 256, rng.randint(8, 256), 8 * rng.randint(1, 64)])
        if T * E > 16384 * 256:
            T = 16384 * 256 // E
        G, top, rule = _groups(rng, E, min(E, 32))
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(16, E // G * top)),
                "score": rng.choice(["sigmoid", "softmax"]), "G": G, "top": top, "rule": rule,
                "bias": rng.random() < 0.7, "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5])}
    if op == "layer":
        while True:
            T = _log_int(rng, 1, 32)
            H, I, Is = 8 * _log_int(rng, 16, 896), 8 * _log_int(rng, 4, 352), 8 * _log_int(rng, 4, 352)
            E = 8 * rng.randint(1, 32)
            El = max(1, E // rng.choice([1, 2, 4, 8]))
            G, top, rule = _groups(rng, E, 8)
            k = rng.randint(1, min(8, E // G * top))
            # at most the largest listed case's weights
            if El * H * I <= 32 * 7168 * 2048 and _used(T, E, El, k) * H * I + H * Is <= 13.5 * 7168 * 2048:
                break
        return {"op": op, "T": T, "H": H, "I": I, "Is": Is, "E": E, "El": El, "e0": El * rng.randrange(E // El), "k": k,
                "score": rng.choice(["sigmoid", "softmax"]), "G": G, "top": top, "rule": rule,
                "scale": rng.choice([1.0, 2.5])}
    act = rng.choice(["none", "none", "swiglu", "swiglu", "silu", "gelu", "gelu_tanh", "relu"])
    c = {"op": "gemm", "act": act, "bias": rng.random() < 0.5, "res": rng.choice(["none", "bf16", "f32"]),
         "out": rng.choice(["bf16", "bf16", "f32"]), "El": 0, "even": True}
    if op == "gemm":
        while True:
            c.update(M=_log_int(rng, 1, 8192), K=8 * _log_int(rng, 8, 896), N=8 * _log_int(rng, 8, 896))
            if c["M"] * c["K"] * c["N"] <= 8192 * 7168 * 2048:
                break
        return c
    while True:
        c.update(M=_log_int(rng, 1, 8192), K=8 * _log_int(rng, 8, 896), N=8 * _log_int(rng, 8, 896),
                 El=_log_int(rng, 1, 64), even=rng.random() < 0.5)
        if c["M"] * c["K"] * c["N"] <= 8192 * 7168 * 2048 and c["El"] * c["K"] * c["N"] <= 32 * 7168 * 2048:
            break
    return c


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    bf = torch.bfloat16

    def randn(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype) * scale

    st = {"case": case}
    op = case["op"]
    if op == "select":
        T, E = case["T"], case["E"]
        # some experts are liked by every token; the bias works against that
        liked = randn(E, scale=0.5)
        st["logits"] = randn(T, E) + liked
        st["bias"] = randn(E, scale=0.05) - 0.1 * liked if case["bias"] else None
    elif op == "gemm":
        M, K, N, El = case["M"], case["K"], case["N"], case["El"]
        cols = 2 * N if case["act"] == "swiglu" else N
        st["a"] = randn(M, K).to(bf)
        st["w"] = randn(max(El, 1), K, cols, scale=K ** -0.5, dtype=bf)
        st["bias"] = randn(max(El, 1), cols, scale=0.2) if case["bias"] else None
        st["residual"] = None if case["res"] == "none" else randn(M, N).to(_TYPES[case["res"]])
        st["offsets"] = None
        if El:
            p = torch.rand(El, generator=g, device=dev) ** (0.0 if case["even"] else 2.0) + 1e-3
            pick = torch.multinomial(p, M, replacement=True, generator=g)
            ends = torch.bincount(pick, minlength=El).cumsum(0)
            st["offsets"] = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    else:
        T, H, I, Is, E, El = (case[n] for n in ("T", "H", "I", "Is", "E", "El"))
        st["x"] = randn(T, H, scale=H ** -0.5).to(bf)
        st["w_router"] = randn(E, H)
        st["choice_bias"] = randn(E, scale=0.05)
        st["w_gate_up"] = randn(El, H, 2 * I, scale=H ** -0.5, dtype=bf)
        st["w_down"] = randn(El, I, H, scale=I ** -0.5, dtype=bf)
        st["s_gate_up"] = randn(H, 2 * Is, scale=H ** -0.5, dtype=bf)
        st["s_down"] = randn(Is, H, scale=Is ** -0.5, dtype=bf)
    return st


# --------------------------------------------------------------------------- #
# The plain forms                                                              #
# --------------------------------------------------------------------------- #
def _plain_choice(logits, bias, c):
    """Chosen experts [T, k] and their weights. The choice compares neighbouring
    scores: 64 bits."""
    T, E = logits.shape
    k, G, top = c["k"], c["G"], c["top"]
    l = logits.double()
    if c["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        s = torch.exp(l - l.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    choice = s if bias is None else s + bias.double()
    if top < G:
        per = torch.sort(choice.view(T, G, E // G), dim=2, descending=True).values
        value = per[:, :, 0] if c["rule"] == "max" else per[:, :, :2].sum(2)
        best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :top]
        keep = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter(1, best, True)
        choice = torch.where(keep[:, :, None], choice.view(T, G, E // G), -torch.inf).view(T, E)
    idx = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, idx)
    if c.get("renorm", True):
        w = w / w.sum(1, keepdim=True)
    return idx.to(torch.int32), (w * c["scale"]).float()


def _silu(g):
    return g / (1 + torch.exp(-g))


def _plain_act(z, act):
    if act == "swiglu":
        n = z.shape[-1] // 2
        return _silu(z[..., :n]) * z[..., n:]
    if act == "silu":
        return _silu(z)
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z


def _plain_gemm(st):
    c = st["case"]
    a, w, bias = st["a"].float(), st["w"], st["bias"]
    if st["offsets"] is None:
        z = a @ w[0].float()
        z = z if bias is None else z + bias[0]
        z = _plain_act(z, c["act"])
    else:
        # the ragged rows in a padded [expert, row] grid
        off = st["offsets"].long()
        row = torch.arange(c["M"], device=off.device)
        e = torch.searchsorted(off[1:], row, right=True)
        at = row - off[e]
        most = int((off[1:] - off[:-1]).max())
        grid = a.new_zeros((c["El"], most, c["K"])).index_put((e, at), a)
        z = torch.matmul(grid, w.float())
        z = z if bias is None else z + bias[:, None]
        z = _plain_act(z, c["act"])[e, at]
    if st["residual"] is not None:
        z = z + st["residual"].float()
    return z.to(_TYPES[c["out"]])


def _plain_layer(st):
    c = st["case"]
    x = st["x"]
    logits = x.double() @ st["w_router"].double().T
    idx, p = _plain_choice(logits, st["choice_bias"], c)
    w = torch.zeros((c["T"], c["E"]), device=x.device).scatter(1, idx.long(), p)[:, c["e0"]:c["e0"] + c["El"]]
    x = x.float()
    # every local expert on every token, weighted with zero where not selected
    h = _plain_act(torch.matmul(x, st["w_gate_up"].float()), "swiglu")
    y = (w.T[:, :, None] * torch.matmul(h, st["w_down"].float())).sum(0)
    h = _plain_act(x @ st["s_gate_up"].float(), "swiglu")
    return (y + h @ st["s_down"].float()).to(torch.bfloat16)


# --------------------------------------------------------------------------- #
# One pass                                                                     #
# --------------------------------------------------------------------------- #
def _choice_args(c):
    return dict(score=c["score"], n_group=c["G"], topk_group=c["top"], group_score=c["rule"],
                renormalize=c.get("renorm", True), scale=c["scale"])


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        import expert_token_routing_amd as M
        if op == "select":
            return M.moe_select(st["logits"], c["k"], st["bias"], **_choice_args(c))
        if op == "gemm":
            return M.moe_gemm(st["a"], st["w"], st["bias"], st["offsets"], activation=c["act"],
                              residual=st["residual"], out_dtype=_TYPES[c["out"]])
        return M.moe_layer_forward(st["x"], st["w_router"], None, st["choice_bias"], st["w_gate_up"], st["w_down"],
                                   c["k"], c["e0"], st["s_gate_up"], st["s_down"], **_choice_args(c))[0]
    if op == "select":
        return _plain_choice(st["logits"], st["bias"], c)
    return _plain_gemm(st) if op == "gemm" else _plain_layer(st)


def work(case):
    """Each input once, each output once; of the layer's experts, the ones that
    even routing is expected to use."""
    op = case["op"]
    if op == "select":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 8 * T * E}
    size = {"none": 0, "bf16": 2, "f32": 4}
    if op == "gemm":
        M, K, N, El = case["M"], case["K"], case["N"], case["El"]
        cols = 2 * N if case["act"] == "swiglu" else N
        used = _used(M, El, El, 1) if El else 1
        return {"bytes": 2 * M * K + used * cols * (2 * K + (4 if case["bias"] else 0)) +
                M * N * (size[case["res"]] + size[case["out"]]), "flops": 2 * M * K * cols}
    T, H, I, Is, E, El, k = (case[n] for n in ("T", "H", "I", "Is", "E", "El", "k"))
    return {"bytes": 4 * E * H + (_used(T, E, El, k) * I + Is) * 6 * H + 4 * T * H,
            "flops": 2 * T * H * E + 6 * T * H * (k * El / E * I + Is)}


# --------------------------------------------------------------------------- #
# The definitions in 64 bits                                                   #
# --------------------------------------------------------------------------- #
def _exact_choice(logits, bias, c):
    import numpy as np
    l = logits.double().cpu().numpy()
    T, E = l.shape
    k, G, top = c["k"], c["G"], c["top"]
    if c["score"] == "sigmoid":
        s = np.reciprocal(1.0 + np.exp(-l))
    else:
        s = np.exp(l - l.max(1)[:, None])
        s /= s.sum(1)[:, None]
    choice = s + (0.0 if bias is None else bias.double().cpu().numpy()[None])
    idx = np.empty((T, k), dtype=np.int64)
    n = E // G
    for t in range(T):
        groups = []
        for g in range(G):
            part = np.sort(choice[t, g * n:(g + 1) * n])[::-1]
            groups.append(part[0] if c["rule"] == "max" else part[:2].sum())
        kept = sorted(range(G), key=lambda g: (-groups[g], g))[:top]
        among = np.concatenate([np.arange(g * n, (g + 1) * n) for g in sorted(kept)])
        idx[t] = among[np.argsort(-choice[t, among], kind="stable")[:k]]
    w = np.take_along_axis(s, idx, 1)
    if c.get("renorm", True):
        w = w / w.sum(1)[:, None]
    return torch.from_numpy(idx).to(logits.device), torch.from_numpy(w * c["scale"]).to(logits.device)


def _exact_mlp(x, gate_up, down):
    gu = x @ gate_up.double()
    I = gu.shape[-1] // 2
    return (gu[..., :I] * torch.sigmoid(gu[..., :I]) * gu[..., I:]) @ down.double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "select":
        idx, w = _exact_choice(st["logits"], st["bias"], case)
        return idx.to(torch.int32), w
    if op == "gemm":
        import torch.nn.functional as F
        M, N = case["M"], case["N"]
        act = {"none": lambda z: z, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
               "gelu_tanh": lambda z: F.gelu(z, approximate="tanh"),
               "swiglu": lambda z: F.silu(z[:, :N]) * z[:, N:]}[case["act"]]
        out = torch.zeros((M, N), dtype=torch.float64, device=st["a"].device)
        off = [0, M] if st["offsets"] is None else st["offsets"].tolist()
        for e in range(len(off) - 1):
            a, b = off[e], off[e + 1]
            if a < b:
                z = st["a"][a:b].double() @ st["w"][e].double()
                out[a:b] = act(z if st["bias"] is None else z + st["bias"][e].double())
        return out if st["residual"] is None else out + st["residual"].double()
    x = st["x"].double()
    logits = (x[:, None, :] * st["w_router"].double()[None]).sum(-1)
    idx, w = _exact_choice(logits, st["choice_bias"], case)
    y = _exact_mlp(x, st["s_gate_up"], st["s_down"])
    for t, (es, ws) in enumerate(zip(idx.tolist(), w.tolist())):
        for e, p in zip(es, ws):
            if case["e0"] <= e < case["e0"] + case["El"]:
                y[t] += p * _exact_mlp(x[t], st["w_gate_up"][e - case["e0"]], st["w_down"][e - case["e0"]])
    return y
