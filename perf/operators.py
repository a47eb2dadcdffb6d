"""Cases of the grouped BF16 products and of the many-adapter projection.

Grouped products (rows sorted by expert, offsets [E+1] as moe_group_tokens
writes them, one weight matrix [N][K] per expert):
  fwd    y[r]  = x[r] W_e^T          reduction over K
  dgrad  dx[r] = dy[r] W_e           reduction over N
  wgrad  dW_e  = sum_r dy[r]^T x[r]  reduction over the expert's rows
Many-adapter projection (rows in segments, one low-rank adapter per segment,
adapter -1 for none, beside one projection W [N][K] shared by all rows):
  fwd    u[t]  = scale_a x[t] A_a^T,  y[t] = x[t] W^T + u[t] B_a^T
  bwd    du[t] = scale_a dy[t] B_a,   dx[t] = dy[t] W + du[t] A_a,
         dA_a  = sum_t du[t]^T x[t],  dB_a = sum_t dy[t]^T u[t]
"""
import math

import torch

own = False

F32 = torch.float32
BF16 = torch.bfloat16


def listed():
    return [
        # one token of a top-8 layer: eight experts of one row each, latency and the weight stream
        dict(name="fwd one token", op="grouped", dir="fwd", T=1, k=8, E=64, K=2048, N=1024, zipf=0.0, drop=0.0, out="bf16"),
        # a decode batch through the down matrices, fp32 rows as the combine takes them
        dict(name="fwd decode 16", op="grouped", dir="fwd", T=16, k=8, E=64, K=1024, N=2048, zipf=0.0, drop=0.0, out="f32"),
        # a prefill batch through the gate matrices
        dict(name="fwd prefill 2048", op="grouped", dir="fwd", T=2048, k=8, E=64, K=2048, N=1024, zipf=0.0, drop=0.0,
             out="bf16"),
        # skewed routing with dropped pairs and sizes that fill no tile: empty and large groups together
        dict(name="fwd skewed odd", op="grouped", dir="fwd", T=509, k=8, E=64, K=2056, N=1000, zipf=1.2, drop=0.03, out="bf16"),
        # few wide experts, a long prefill: the largest product
        dict(name="fwd wide 8192", op="grouped", dir="fwd", T=8192, k=2, E=8, K=4096, N=14336, zipf=0.0, drop=0.0, out="bf16"),
        # training: the gradient that goes back to the rows, fp32 for the sum over a token's experts
        dict(name="dgrad 2048", op="grouped", dir="dgrad", T=2048, k=8, E=64, K=2048, N=1024, zipf=0.0, drop=0.0, out="f32"),
        # training: the weights' gradient in fp32, as an optimizer's main gradient holds it
        dict(name="wgrad 2048", op="grouped", dir="wgrad", T=2048, k=8, E=64, K=2048, N=1024, zipf=0.0, drop=0.0, out="f32"),
        # training of few wide experts with skewed groups
        dict(name="wgrad wide skewed", op="grouped", dir="wgrad", T=2047, k=2, E=8, K=4096, N=14336, zipf=1.2, drop=0.0,
             out="bf16"),
        # one token of one request
        dict(name="adapters one token", op="lora", dir="fwd", T=1, S=1, n=8, r=16, K=2048, N=2048, none=0.0, pad=0),
        # a decode batch, each token another request, some without an adapter, a padded batch
        dict(name="adapters decode 61", op="lora", dir="fwd", T=61, S=58, n=48, r=16, K=2048, N=4096, none=0.1, pad=3),
        # a mixed prefill batch of ragged requests
        dict(name="adapters prefill 8192", op="lora", dir="fwd", T=8192, S=13, n=8, r=64, K=4096, N=4096, none=0.1, pad=0),
        # a fine-tuning step of several adapters at once
        dict(name="adapters backward 2041", op="lora", dir="bwd", T=2041, S=11, n=6, r=16, K=2048, N=2048, none=0.1, pad=5),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    if rng.random() < 0.55:
        d = rng.choice(["fwd", "fwd", "dgrad", "wgrad"])
        E = rng.choice([8, 16, 27, 64, 128])
        k = rng.choice([1, 2, 4, 8])
        case = dict(op="grouped", dir=d, T=_log_int(rng, 1, 8192), k=k, E=E, K=_log_int(rng, 128, 4096, 8),
                    N=_log_int(rng, 128, 14336, 8), zipf=rng.choice([0.0, 0.0, 0.8, 1.2]),
                    drop=rng.choice([0.0, 0.0, 0.05, 0.5]), out=rng.choice(["bf16", "f32"]))
        while case["E"] * case["K"] * case["N"] > 8 * 4096 * 14336:  # no more weights than the largest listed case
            case["E"] = max(8, case["E"] // 2)
        while case["T"] * case["k"] * case["K"] * case["N"] > 16384 * 4096 * 14336:
            case["T"] = max(1, case["T"] // 2)
        if case["T"] * case["k"] < 16:
            case["drop"] = 0.0  # a pair is left
        return case
    T = _log_int(rng, 1, 8192)
    S = T if rng.random() < 0.3 and T <= 256 else min(T, _log_int(rng, 1, 64))  # one token a request, or prompts
    return dict(op="lora", dir=rng.choice(["fwd", "fwd", "bwd"]), T=T, S=S, n=_log_int(rng, 1, 64),
                r=rng.choice([8, 16, 16, 32, 64, 128]), K=_log_int(rng, 256, 4096, 8), N=_log_int(rng, 256, 4096, 8),
                none=rng.choice([0.0, 0.1, 0.5]), pad=rng.choice([0, 0, 1, 7]) if T >= 16 else 0)


# ------------------------------------------------------------------ inputs

def _group_counts(case, seed):
    """Rows per expert when each of T tokens picks k distinct experts (by a
    Gumbel top-k over log Zipf weights) and a share of the pairs is dropped."""
    g = torch.Generator().manual_seed(seed * 7919 + 11)
    T, k, E = case["T"], case["k"], case["E"]
    logit = -case["zipf"] * torch.log(torch.arange(1, E + 1, dtype=torch.float64))
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)))
    ids = torch.topk(logit + noise, k, dim=1).indices.flatten()
    keep = torch.rand(T * k, generator=g) >= case["drop"]
    return torch.bincount(ids[keep], minlength=E)


def _segments(case, seed):
    """Segment starts [S+1] and adapters [S]; the last `pad` rows lie behind the last segment."""
    g = torch.Generator().manual_seed(seed * 104729 + 5)
    S, n = case["S"], case["n"]
    rows = max(case["T"] - case["pad"], 0)
    if S >= rows:
        lens = torch.ones(S, dtype=torch.int64)
        lens[rows:] = 0  # requests that have ended
    else:
        cut = torch.sort(torch.randint(0, rows + 1, (S - 1,), generator=g)).values
        lens = torch.diff(torch.cat([torch.zeros(1, dtype=torch.int64), cut, torch.full((1,), rows)]))
    off = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(lens, 0)])
    ad = torch.randint(0, n, (S,), generator=g)
    ad[torch.rand(S, generator=g) < case["none"]] = -1
    return off, ad


def _normal(shape, std, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=BF16).mul_(std)


def _grouped_inputs(case, seed):
    E, N, K = case["E"], case["N"], case["K"]
    R = case["T"] * case["k"]
    off = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(_group_counts(case, seed), 0)])
    d = {"off": off}
    if case["dir"] != "dgrad":
        d["x"] = _normal((R, K), 1.0, 4 * seed + 1)
    if case["dir"] != "fwd":
        d["dy"] = _normal((R, N), 1.0, 4 * seed + 2)
    if case["dir"] != "wgrad":
        d["w"] = _normal((E, N, K), 0.02, 4 * seed + 3)
    return d


def _lora_inputs(case, seed):
    T, n, r, K, N = (case[c] for c in ("T", "n", "r", "K", "N"))
    off, ad = _segments(case, seed)
    d = {"off": off, "ad": ad, "x": _normal((T, K), 1.0, 8 * seed + 1), "w": _normal((N, K), 0.02, 8 * seed + 2),
         "a": _normal((n, r, K), 1.0 / math.sqrt(K), 8 * seed + 3), "b": _normal((n, N, r), 0.02, 8 * seed + 4)}
    g = torch.Generator().manual_seed(8 * seed + 5)
    d["scale"] = (0.5 + 1.5 * torch.rand(n, generator=g)).cuda()
    if case["dir"] == "bwd":
        d["dy"] = _normal((T, N), 1.0, 8 * seed + 6)
        u = torch.zeros(T, r, device="cuda")  # what the forward pass kept
        for s in range(len(ad)):
            lo, hi, q = int(off[s]), int(off[s + 1]), int(ad[s])
            if q >= 0 and hi > lo:
                u[lo:hi] = (d["x"][lo:hi].float() @ d["a"][q].float().T) * d["scale"][q]
        d["u"] = u.to(BF16)
    return d


def prepare(case, seed):
    st = {"case": case, **(_grouped_inputs if case["op"] == "grouped" else _lora_inputs)(case, seed)}
    st["host_off"] = st["off"].tolist()
    st["off"] = st["off"].to(torch.int32).cuda()
    if case["op"] == "grouped":
        R = case["T"] * case["k"]
        shape = {"fwd": (R, case["N"]), "dgrad": (R, case["K"]), "wgrad": (case["E"], case["N"], case["K"])}[case["dir"]]
        st["out"] = torch.zeros(shape, device="cuda", dtype=F32 if case["out"] == "f32" else BF16)
    else:
        st["host_ad"] = st["ad"].tolist()
        st["ad"] = st["ad"].to(torch.int32).cuda()
        T, n, r, K, N = (case[c] for c in ("T", "n", "r", "K", "N"))
        if case["dir"] == "fwd":
            st["u"] = torch.zeros(T, r, device="cuda", dtype=BF16)
            st["y"] = torch.zeros(T, N, device="cuda", dtype=BF16)
        else:
            st["du"] = torch.zeros(T, r, device="cuda", dtype=BF16)
            st["dx"] = torch.zeros(T, K, device="cuda", dtype=BF16)
            st["da"] = torch.zeros(n, r, K, device="cuda", dtype=BF16)
            st["db"] = torch.zeros(n, N, r, device="cuda", dtype=BF16)
    if own:
        import w4a16_mixture_experts_moe_b200 as moe
        size = (moe.moe_grouped_gemm_workspace_size(case["T"] * case["k"], case["E"], case["N"], case["K"])
                if case["op"] == "grouped" else
                moe.moe_lora_workspace_size(case["T"], case["S"], case["n"], case["r"], case["N"], case["K"]))
        st["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ one pass

def _run_own(st):
    import w4a16_mixture_experts_moe_b200 as moe
    c = st["case"]
    N, K, ws = c["N"], c["K"], st["ws"]
    if c["op"] == "grouped":
        R, E = c["T"] * c["k"], c["E"]
        flags = moe.MOE_GEMM_OUT_F32 if c["out"] == "f32" else 0
        if c["dir"] == "fwd":
            moe.moe_grouped_gemm(st["x"], K, st["off"], st["w"], N * K, R, E, N, K, flags, st["out"], N, ws, ws.numel())
        elif c["dir"] == "dgrad":
            moe.moe_grouped_gemm_dgrad(st["dy"], N, st["off"], st["w"], N * K, R, E, N, K, flags, st["out"], K, ws,
                                       ws.numel())
        else:
            moe.moe_grouped_gemm_wgrad(st["dy"], N, st["x"], K, st["off"], R, E, N, K, flags, st["out"], N * K, ws,
                                       ws.numel())
        return st["out"]
    T, S, n, r = c["T"], c["S"], c["n"], c["r"]
    if c["dir"] == "fwd":
        moe.moe_lora_linear(st["x"], K, st["w"], st["off"], st["ad"], st["a"], st["b"], st["scale"], T, S, n, r, N, K,
                            st["u"], st["y"], N, ws, ws.numel())
        return {"y": st["y"], "u": st["u"]}
    moe.moe_lora_linear_backward(st["dy"], N, st["x"], K, st["w"], st["u"], st["off"], st["ad"], st["a"], st["b"],
                                 st["scale"], T, S, n, r, N, K, st["du"], st["dx"], K, st["da"], st["db"], ws, ws.numel())
    return {"dx": st["dx"], "da": st["da"], "db": st["db"]}


def run(st):
    if own:
        return _run_own(st)
    c, off = st["case"], st["host_off"]
    if c["op"] == "grouped":
        out = torch.zeros_like(st["out"])
        for e in range(c["E"]):
            lo, hi = off[e], off[e + 1]
            if hi == lo:
                continue
            if c["dir"] == "fwd":
                out[lo:hi] = st["x"][lo:hi].float() @ st["w"][e].float().T
            elif c["dir"] == "dgrad":
                out[lo:hi] = st["dy"][lo:hi].float() @ st["w"][e].float()
            else:
                out[e] = st["dy"][lo:hi].float().T @ st["x"][lo:hi].float()
        return out
    end = off[-1]
    segs = [(off[s], off[s + 1], q) for s, q in enumerate(st["host_ad"]) if q >= 0 and off[s + 1] > off[s]]
    if c["dir"] == "fwd":
        y = torch.zeros(c["T"], c["N"], device="cuda")
        u = torch.zeros(c["T"], c["r"], device="cuda")
        y[:end] = st["x"][:end].float() @ st["w"].float().T
        for lo, hi, q in segs:
            u[lo:hi] = (st["x"][lo:hi].float() @ st["a"][q].float().T) * st["scale"][q]
            y[lo:hi] += u[lo:hi] @ st["b"][q].float().T
        return {"y": y.to(BF16), "u": u.to(BF16)}
    dx = torch.zeros(c["T"], c["K"], device="cuda")
    da = torch.zeros(st["a"].shape, device="cuda")
    db = torch.zeros(st["b"].shape, device="cuda")
    dx[:end] = st["dy"][:end].float() @ st["w"].float()
    for lo, hi, q in segs:
        g = st["dy"][lo:hi].float()
        du = (g @ st["b"][q].float()) * st["scale"][q]
        dx[lo:hi] += du @ st["a"][q].float()
        da[q] += du.T @ st["x"][lo:hi].float()
        db[q] += g.T @ st["u"][lo:hi].float()
    return {"dx": dx.to(BF16), "da": da.to(BF16), "db": db.to(BF16)}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    K, N = case["K"], case["N"]
    if case["op"] == "grouped":
        counts = _group_counts(case, 0)
        rows, active = int(counts.sum()), int((counts > 0).sum())
        o = 4 if case["out"] == "f32" else 2
        if case["dir"] == "fwd":
            b = 2 * rows * K + 2 * active * N * K + o * rows * N
        elif case["dir"] == "dgrad":
            b = 2 * rows * N + 2 * active * N * K + o * rows * K
        else:
            b = 2 * rows * (N + K) + o * case["E"] * N * K  # every expert's gradient is written
        return {"bytes": b + 4 * (case["E"] + 1), "flops": 2 * rows * N * K}
    off, ad = _segments(case, 0)
    lens = torch.diff(off)
    rows, arows = int(off[-1]), int(lens[ad >= 0].sum())
    active = len(set(ad[(ad >= 0) & (lens > 0)].tolist()))
    r, n = case["r"], case["n"]
    lora = 2 * active * r * (N + K)
    if case["dir"] == "fwd":
        return {"bytes": 2 * rows * (K + N) + 2 * N * K + lora + 2 * rows * r, "flops": 2 * rows * N * K + 2 * arows * r * (N + K)}
    return {"bytes": 2 * rows * (N + 2 * K) + 2 * N * K + lora + 2 * rows * r + 2 * n * r * (N + K),
            "flops": 2 * rows * N * K + 4 * arows * r * (N + K)}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    f64 = torch.float64
    if case["op"] == "grouped":
        d = _grouped_inputs(case, seed)
        starts, ends = d["off"][:-1].tolist(), d["off"][1:].tolist()
        if case["dir"] == "wgrad":
            res = torch.empty(case["E"], case["N"], case["K"], dtype=f64, device="cuda")
            for e, (i, j) in enumerate(zip(starts, ends)):
                res[e] = torch.einsum("rn,rk->nk", d["dy"][i:j].to(f64), d["x"][i:j].to(f64))
            return res
        src, eq, width = (d["x"], "rk,nk->rn", case["N"]) if case["dir"] == "fwd" else (d["dy"], "rn,nk->rk", case["K"])
        res = torch.zeros(src.shape[0], width, dtype=f64, device="cuda")
        for e, (i, j) in enumerate(zip(starts, ends)):
            if j > i:
                res[i:j] = torch.einsum(eq, src[i:j].to(f64), d["w"][e].to(f64))
        return res
    d = _lora_inputs(case, seed)
    T, n = case["T"], case["n"]
    owner = torch.full((T,), -2, dtype=torch.int64)  # -2: behind the last segment
    for s in range(case["S"]):
        owner[int(d["off"][s]):int(d["off"][s + 1])] = int(d["ad"][s])
    owner = owner.cuda()
    live = (owner >= -1).to(f64)[:, None]
    x, w, scale = d["x"].to(f64), d["w"].to(f64), d["scale"].to(f64)
    if case["dir"] == "fwd":
        y = torch.einsum("tk,nk->tn", x, w) * live
        u = torch.zeros(T, case["r"], dtype=f64, device="cuda")
        for q in range(n):
            t = torch.nonzero(owner == q).flatten()
            if t.numel():
                u[t] = scale[q] * torch.einsum("tk,jk->tj", x[t], d["a"][q].to(f64))
                y[t] += torch.einsum("tj,nj->tn", u[t], d["b"][q].to(f64))
        return {"y": y, "u": u}
    dy, uu = d["dy"].to(f64), d["u"].to(f64)
    dx = torch.einsum("tn,nk->tk", dy, w) * live
    da = torch.zeros(d["a"].shape, dtype=f64, device="cuda")
    db = torch.zeros(d["b"].shape, dtype=f64, device="cuda")
    for q in range(n):
        t = torch.nonzero(owner == q).flatten()
        if t.numel():
            du = scale[q] * torch.einsum("tn,nj->tj", dy[t], d["b"][q].to(f64))
            dx[t] += torch.einsum("tj,jk->tk", du, d["a"][q].to(f64))
            da[q] = torch.einsum("tj,tk->jk", du, x[t])
            db[q] = torch.einsum("tn,tj->nj", dy[t], uu[t])
    return {"dx": dx, "da": da, "db": db}
