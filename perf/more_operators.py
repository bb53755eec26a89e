"""Timing cases of the open expert layer and of the update of its weights.

moe_ffn fuses dispatch, SwiGLU experts and combine.  These are the pieces for a
layer whose experts are something else, with their gradients, and the step that
an orthogonalising optimiser takes on the stacked expert weights:

dispatch        the rows of x in expert order: the slots s = t*K + k of topk_ids
                sorted by expert, stable, rows[r] = x[t]; offsets[e] = first row of
                expert e; slot2row = the row of each slot.
dispatch_train  the same and dx[t] = sum_k d_rows[slot2row[t, k]].
combine         y[t] = sum_k topk_weights[t, k] * rows[slot2row[t, k]].
combine_train   the same, d_rows[slot2row[t, k]] = topk_weights[t, k] * dy[t] and
                d_topk_weights[t, k] = <rows[slot2row[t, k]], dy[t]>.
gmm             y[r] = x[r] . w[e] for the rows offsets[e] <= r < offsets[e + 1] of
                expert e, 0 for rows of no expert.
gmm_train       the same, dx[r] = dy[r] . w[e]^T and dw[e] = x_e^T . dy_e.
orthogonalize   scale * X_n for each matrix G of a stack, with X_0 = G / (|G|_F + eps)
                and X <- a X + (b A + c A A) X, A = X X^T (n steps).

`run` computes a case either through the library (`own`) or in a plain form of
elementary torch operations in 32 bits; `exact` computes it again in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-7
QUINTIC = (3.4445, -4.7750, 2.0315)


# ------------------------------------------------------------------- the cases
def listed():
    """The smallest calls, ordinary ones and the largest, for each operator."""
    return [
        # one decode token to its experts: latency only
        dict(name="dispatch, 1 token, 256 experts", op="dispatch", T=1, H=7168, E=256, K=8,
             routing="uniform", dtype="bfloat16"),
        # a training step's dispatch of a long batch with hot experts
        dict(name="dispatch step, 16384 tokens", op="dispatch_train", T=16384, H=7168, E=32, K=8,
             routing="zipf", dtype="bfloat16"),
        # a decode batch's merge of its experts' rows
        dict(name="combine, 128 tokens", op="combine", T=128, H=7168, E=256, K=8,
             routing="uniform", dtype="bfloat16", wdtype="float32"),
        # a training step's merge: an odd number of tokens, fp32 routing weights
        dict(name="combine step, 4097 tokens", op="combine_train", T=4097, H=2048, E=64, K=6,
             routing="uniform", dtype="bfloat16", wdtype="float32"),
        # one decode token: its eight experts' up-projections are streamed
        dict(name="gmm, 8 rows, 256 experts", op="gmm", R=8, K=7168, N=4096, E=256,
             routing="few", tail=0, dtype="bfloat16", transposed=False),
        # a decode batch: nearly every expert's down-projection is streamed
        dict(name="gmm, 1024 rows, 256 experts", op="gmm", R=1024, K=2048, N=7168, E=256,
             routing="uniform", tail=0, dtype="bfloat16", transposed=False),
        # a prompt, weights kept with the contraction contiguous, as a checkpoint of
        # linear layers has them
        dict(name="gmm, 24576 rows, 64 experts", op="gmm", R=24576, K=2048, N=2816, E=64,
             routing="uniform", tail=0, dtype="bfloat16", transposed=True),
        # a training step with hot and empty experts, fp16, and a batch padded at its end
        dict(name="gmm step, 24570 rows, 64 experts", op="gmm_train", R=24570, K=1408, N=2048,
             E=64, routing="zipf", tail=37, dtype="float16", transposed=False),
        # the down-projections of a long batch, all gradients
        dict(name="gmm step, 131072 rows, 32 experts", op="gmm_train", R=131072, K=2048, N=7168,
             E=32, routing="uniform", tail=0, dtype="bfloat16", transposed=False),
        # a few small matrices: the fifteen products depend on each other, latency counts
        dict(name="orthogonalize, 4 x 128 x 250", op="orthogonalize", B=4, M=128, N=250, steps=5,
             scale=1.0, dtype="float32"),
        # the down-projections of a 64-expert layer
        dict(name="orthogonalize, 64 x 1408 x 2048", op="orthogonalize", B=64, M=1408, N=2048,
             steps=5, scale=0.2, dtype="bfloat16"),
        # up-projections of large experts: more rows than columns
        dict(name="orthogonalize, 8 x 7168 x 4096", op="orthogonalize", B=8, M=7168, N=4096,
             steps=5, scale=1.0, dtype="bfloat16"),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, n))


def _multiple(rng, lo, hi, step):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    return max(lo, _log_int(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_train", "combine", "combine_train", "gmm", "gmm",
                     "gmm_train", "gmm_train", "orthogonalize", "orthogonalize"])
    if op.startswith(("dispatch", "combine")):
        E = rng.choice([8, 30, 64, 256])
        H, K = _multiple(rng, 64, 7168, 8), rng.randint(1, 8)
        T = _log_int(rng, 1, 16383) | 1
        c = dict(op=op, T=T, H=H, E=E, K=K, routing=rng.choice(["uniform", "zipf"]),
                 dtype=rng.choice(["bfloat16", "bfloat16", "float16", "float32"]))
        if op.startswith("combine"):
            c["wdtype"] = rng.choice(["float32", "bfloat16"])
        return c
    if op.startswith("gmm"):
        E = rng.choice([1, 4, 8, 30, 64, 96])
        K, N = _multiple(rng, 64, 7168, 8), _multiple(rng, 64, 7168, 8)
        while E * K * N > 64 * 2048 * 4096:
            E //= 2
        R = _log_int(rng, 1, 131071) | 1
        routing = rng.choice(["uniform", "zipf"])
        pad = max(1.5, 0.35 * E) if routing == "zipf" else 1.5  # (the plain form's padding)
        while pad * R * max(K * N, 1024 * (K + N)) > 1.5 * 131072 * 2048 * 7168:
            R = R // 2 | 1
        return dict(op=op, R=R, K=K, N=N, E=E, routing=routing,
                    tail=rng.choice([0, 0, 1, 77]) if R > 200 else 0,
                    dtype=rng.choice(["bfloat16", "bfloat16", "float16"]),
                    transposed=rng.random() < 0.4)
    M, N, B = _log_int(rng, 16, 7168), _log_int(rng, 16, 7168), _log_int(rng, 1, 64)
    while B > 1 and B * min(M, N) ** 2 * max(M, N) > 8 * 4096 * 4096 * 7168:
        B //= 2
    while B * min(M, N) ** 2 * max(M, N) > 8 * 4096 * 4096 * 7168:
        M, N = M * 3 // 4, N * 3 // 4
    return dict(op=op, B=B, M=M, N=N, steps=rng.choice([4, 5, 5, 6]),
                scale=rng.choice([1.0, 0.2]),
                dtype=rng.choice(["bfloat16", "bfloat16", "float16", "float32"]))


_BYTES = dict(bfloat16=2, float16=2, float32=4)


def work(c):
    op = c["op"]
    if op == "orthogonalize":
        m, n = min(c["M"], c["N"]), max(c["M"], c["N"])
        out = 2
        # A and A A are symmetric: one triangle of each
        per_step = m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n
        return dict(bytes=c["B"] * c["M"] * c["N"] * (_BYTES[c["dtype"]] + out),
                    flops=c["B"] * c["steps"] * per_step)
    if op.startswith("gmm"):
        R, K, N, E = c["R"] - c["tail"], c["K"], c["N"], c["E"]
        touched = E if R >= 8 * E else E * (1.0 - (1.0 - 1.0 / E) ** R)
        if c["routing"] == "few":
            touched = min(E, R)
        w = touched * K * N * 2
        d = dict(bytes=w + 2 * R * K + 2 * c["R"] * N + 4 * (E + 1), flops=2 * R * K * N)
        if op == "gmm_train":
            # dy read, dx written, every dw written
            d["bytes"] += 2 * R * N + 2 * c["R"] * K + 2 * E * K * N
            d["flops"] *= 3
        return d
    T, H, K, b = c["T"], c["H"], c["K"], _BYTES[c["dtype"]]
    x, rows, ids = T * H * b, T * K * H * b, 4 * T * K
    if op == "dispatch":
        return dict(bytes=x + rows + 2 * ids + 4 * (c["E"] + 1), flops=0)
    if op == "dispatch_train":
        return dict(bytes=2 * (x + rows) + 2 * ids + 4 * (c["E"] + 1), flops=T * K * H)
    w = T * K * _BYTES[c["wdtype"]]
    if op == "combine":
        return dict(bytes=x + rows + ids + w, flops=2 * T * K * H)
    return dict(bytes=2 * (x + rows) + ids + 2 * w, flops=5 * T * K * H)


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _popularity(g, c):
    """Probability of each expert: equal, or Zipf's with the last ones empty."""
    E = c["E"]
    if c["routing"] != "zipf":
        return torch.full((E,), 1.0 / E, device=DEVICE)
    p = torch.arange(1, E + 1, device=DEVICE, dtype=torch.float32).pow(-1.2)
    empty = min(3, E - c.get("K", 1)) if "T" in c else min(3, E - 1)
    if empty > 0:
        p[E - empty:] = 0
    p = p[torch.randperm(E, generator=g, device=DEVICE)]
    return p / p.sum()


def _topk_ids(g, c):
    u = torch.rand((c["T"], c["E"]), generator=g, device=DEVICE).clamp_min_(1e-12)
    key = -torch.log(-torch.log(u).clamp_min_(1e-12)) + torch.log(_popularity(g, c))
    return torch.argsort(key, dim=1, descending=True)[:, :c["K"]].to(torch.int32).contiguous()


def _offsets(g, c):
    """First row of each expert, and the rows of the largest."""
    R, E = c["R"] - c["tail"], c["E"]
    if c["routing"] == "few":
        counts = torch.zeros(E, dtype=torch.long, device=DEVICE)
        counts[torch.randperm(E, generator=g, device=DEVICE)[:R]] = 1
    else:
        p = _popularity(g, c)
        counts = torch.bincount(torch.multinomial(p, R, replacement=True, generator=g),
                                minlength=E)
    o = torch.zeros(E + 1, dtype=torch.int32, device=DEVICE)
    o[1:] = counts.cumsum(0)
    return o, int(counts.max())


def prepare(c, seed):
    g, op = _gen(seed), c["op"]
    dt = getattr(torch, c["dtype"])

    def normal(*shape, std=1.0, dtype=dt):
        out = torch.empty(shape, dtype=dtype, device=DEVICE)
        return out.normal_(0.0, std, generator=g)

    if op == "orthogonalize":
        # a gradient: a few strong directions over noise, as sums over tokens have them
        B, M, N = c["B"], c["M"], c["N"]
        r = max(1, min(M, N) // 16)
        strong = torch.bmm(normal(B, M, r, dtype=torch.float32),
                           normal(B, r, N, dtype=torch.float32))
        noise = normal(B, M, N, dtype=torch.float32)
        return dict(case=c, g=(strong.mul_(0.5 / r ** 0.5).add_(noise).mul_(1e-3)).to(dt))
    if op.startswith("gmm"):
        o, most = _offsets(g, c)
        E, K, N, R = c["E"], c["K"], c["N"], c["R"]
        w = normal(E, N, K, std=K ** -0.5) if c["transposed"] else normal(E, K, N, std=K ** -0.5)
        s = dict(case=c, x=normal(R, K), w=w, offsets=o, most=most)
        if op == "gmm_train":
            s["dy"] = normal(R, N)
        return s
    T, H, K = c["T"], c["H"], c["K"]
    ids = _topk_ids(g, c)
    s = dict(case=c, ids=ids)
    if op.startswith("dispatch"):
        s["x"] = normal(T, H)
        if op == "dispatch_train":
            s["d_rows"] = normal(T * K, H)
        return s
    # the routing is in hand: the forward's dispatch made it
    flat = ids.flatten().long()
    row2slot = torch.argsort(flat, stable=True)
    slot2row = torch.empty_like(row2slot)
    slot2row[row2slot] = torch.arange(T * K, device=DEVICE)
    counts = torch.bincount(flat, minlength=c["E"])
    o = torch.zeros(c["E"] + 1, dtype=torch.int32, device=DEVICE)
    o[1:] = counts.cumsum(0)
    s.update(rows=normal(T * K, H), offsets=o, counts=counts.int(),
             slot2row=slot2row.int().view(T, K), row2slot=row2slot.int())
    s["w"] = torch.softmax(normal(T, K, dtype=torch.float32), 1).to(getattr(torch, c["wdtype"]))
    if op == "combine_train":
        s["dy"] = normal(T, H)
    return s


# -------------------------------------------------------------- the plain form
def _plain_dispatch(c, s):
    T, K = c["T"], c["K"]
    flat = s["ids"].flatten().long()
    row2slot = torch.argsort(flat, stable=True)
    slot2row = torch.empty_like(row2slot)
    slot2row[row2slot] = torch.arange(T * K, device=flat.device)
    experts = torch.arange(c["E"] + 1, device=flat.device)
    out = dict(rows=s["x"][row2slot // K],
               offsets=torch.searchsorted(flat[row2slot], experts).int(),
               slot2row=slot2row.int().view(T, K))
    if c["op"] == "dispatch_train":
        out["dx"] = s["d_rows"].float()[slot2row].view(T, K, -1).sum(1).to(s["x"].dtype)
    return out


def _plain_combine(c, s):
    T, K = c["T"], c["K"]
    at = s["slot2row"].long()
    w = s["w"].float().unsqueeze(2)
    rows = s["rows"][at.flatten()].view(T, K, -1).float()
    out = dict(y=(w * rows).sum(1).to(s["rows"].dtype))
    if c["op"] == "combine_train":
        dy = s["dy"].float().unsqueeze(1)
        d_rows = torch.empty_like(s["rows"])
        d_rows[at.flatten()] = (w * dy).to(d_rows.dtype).view(T * K, -1)
        out.update(d_rows=d_rows, d_w=(rows * dy).sum(2).to(s["w"].dtype))
    return out


def _plain_gmm(c, s):
    R, E, o, most = c["R"], c["E"], s["offsets"].long(), s["most"]
    x, w, dev = s["x"], s["w"], s["x"].device
    r = torch.arange(R, device=dev)
    e = torch.searchsorted(o, r, right=True) - 1  # E behind the last expert's rows
    if c["op"] == "gmm" and R <= E:  # few rows: their experts' weights alone, a row each
        w, at, E, most = w[e], r, R, 1
    else:
        at = torch.where(e < E, e * most + r - o[e], E * most)
    wf = w.float()
    if c["transposed"]:
        wf = wf.transpose(1, 2)

    def padded(v):
        """Rows to [E, most, columns]; those of no expert behind them."""
        p = torch.zeros((E * most + 1, v.shape[1]), device=dev)
        p[at] = v.float()
        return p[:-1].view(E, most, -1)

    def rows(p):
        v = p.reshape(E * most, -1)[at.clamp(max=E * most - 1)].to(x.dtype)
        return v.masked_fill_((at == E * most).unsqueeze(1), 0.0)

    xp = padded(x)
    out = dict(y=rows(torch.bmm(xp, wf)))
    if c["op"] == "gmm_train":
        dyp = padded(s["dy"])
        out.update(dx=rows(torch.bmm(dyp, wf.transpose(1, 2))),
                   dw=torch.bmm(xp.transpose(1, 2), dyp).to(x.dtype))
    return out


def _plain_step(x, coefficients):
    a, b, c = coefficients
    if x.shape[1] <= x.shape[2]:
        s = torch.bmm(x, x.transpose(1, 2))
        return torch.bmm(b * s + c * torch.bmm(s, s), x) + a * x
    s = torch.bmm(x.transpose(1, 2), x)
    return torch.bmm(x, b * s + c * torch.bmm(s, s)) + a * x


def _plain_orthogonalize(c, s):
    x = s["g"].float()
    # (sums of squares of millions of elements: in 64 bits)
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt().float()
    x = x / (norm + EPS)
    for _ in range(c["steps"]):
        x = _plain_step(x, QUINTIC)
    return dict(x=(x * c["scale"]).to(_result_type(c)))


def _result_type(c):
    return torch.float16 if c["dtype"] == "float16" else torch.bfloat16


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op.startswith("dispatch"):
        return _plain_dispatch(c, s)
    if op.startswith("combine"):
        return _plain_combine(c, s)
    return _plain_gmm(c, s) if op.startswith("gmm") else _plain_orthogonalize(c, s)


# --------------------------------------------------------- through the library
def _own(s):
    import dispatch_grouped_gemm_gb300 as hmm

    c = s["case"]
    op = c["op"]
    if op == "orthogonalize":
        return dict(x=hmm.orthogonalize(s["g"], steps=c["steps"], coefficients=QUINTIC, eps=EPS,
                                        scale=c["scale"], out_dtype=_result_type(c)))
    if op.startswith("gmm"):
        w = s["w"].detach()
        if op == "gmm":
            return dict(y=hmm.moe_grouped_mm(s["x"], w.transpose(1, 2) if c["transposed"] else w,
                                             s["offsets"]))
        x, w = s["x"].detach().requires_grad_(), w.requires_grad_()
        y = hmm.moe_grouped_mm(x, w.transpose(1, 2) if c["transposed"] else w, s["offsets"])
        dx, dw = torch.autograd.grad(y, (x, w), s["dy"])
        return dict(y=y.detach(), dx=dx, dw=dw.transpose(1, 2) if c["transposed"] else dw)
    if op.startswith("dispatch"):
        routing = hmm.moe_route(s["ids"], c["E"])
        x = s["x"]
        if op == "dispatch_train":
            x = x.detach().requires_grad_()
        rows = hmm.moe_dispatch(x, routing)
        out = dict(rows=rows.detach(), offsets=routing.offsets, slot2row=routing.slot2row)
        if op == "dispatch_train":
            (out["dx"],) = torch.autograd.grad(rows, x, s["d_rows"])
        return out
    routing = hmm.MoeRouting(s["counts"], s["offsets"], s["slot2row"], s["row2slot"])
    if op == "combine":
        return dict(y=hmm.moe_combine(s["rows"], routing, s["w"]))
    rows, w = s["rows"].detach().requires_grad_(), s["w"].detach().requires_grad_()
    y = hmm.moe_combine(rows, routing, w)
    d_rows, d_w = torch.autograd.grad(y, (rows, w), s["dy"])
    return dict(y=y.detach(), d_rows=d_rows, d_w=d_w)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- in 64 bits
def _exact_gmm(c, s):
    x, w, o = s["x"].double(), s["w"], s["offsets"].tolist()
    out = dict(y=torch.zeros((c["R"], c["N"]), dtype=torch.float64, device=x.device))
    if c["op"] == "gmm_train":
        dy = s["dy"].double()
        out["dx"] = torch.zeros_like(x)
        out["dw"] = torch.zeros((c["E"], c["K"], c["N"]), dtype=torch.float64, device=x.device)
    for e in range(c["E"]):
        i, j = o[e], o[e + 1]
        if i == j:
            continue
        we = w[e].double().T if c["transposed"] else w[e].double()
        out["y"][i:j] = x[i:j] @ we
        if c["op"] == "gmm_train":
            out["dx"][i:j] = torch.einsum("rn,kn->rk", dy[i:j], we)
            out["dw"][e] = torch.einsum("rk,rn->kn", x[i:j], dy[i:j])
    return out


def _exact_orthogonalize(c, s):
    out = []
    a, b, d = QUINTIC
    for g in s["g"]:
        x = g.double()
        wide = x if c["M"] <= c["N"] else x.T
        x = wide / (torch.linalg.vector_norm(wide) + EPS)
        for _ in range(c["steps"]):
            # a X + b A X + c A (A X)
            s2 = x @ x.T
            ax = s2 @ x
            x = a * x + b * ax + d * (s2 @ ax)
        out.append((x if c["M"] <= c["N"] else x.T) * c["scale"])
    return dict(x=torch.stack(out))


def exact(c, seed):
    op = c["op"]
    # (the 64-bit rate of this card is about a TFLOP/s)
    if op.startswith("gmm") and work(c)["flops"] > 1.2e13:
        return None
    if op == "orthogonalize" and work(c)["flops"] > 6e12:
        return None
    s = prepare(c, seed)
    if op == "orthogonalize":
        return _exact_orthogonalize(c, s)
    if op.startswith("gmm"):
        return _exact_gmm(c, s)
    if op.startswith("dispatch"):
        out = dict(rows=None, offsets=None, slot2row=None)
        ids = s["ids"]
        place = torch.argsort(torch.argsort(ids.flatten().long(), stable=True))
        out["rows"] = torch.empty((c["T"] * c["K"], c["H"]), dtype=torch.float64, device=ids.device)
        out["rows"][place] = s["x"].double().repeat_interleave(c["K"], 0)
        if op == "dispatch_train":
            out["dx"] = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=ids.device)
            out["dx"].index_add_(0, torch.arange(c["T"], device=ids.device)
                                 .repeat_interleave(c["K"]), s["d_rows"].double()[place])
        return out
    token = s["row2slot"].long() // c["K"]
    w = s["w"].double().flatten()[s["row2slot"].long()].unsqueeze(1)
    rows = s["rows"].double()
    y = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=rows.device)
    out = dict(y=y.index_add_(0, token, w * rows))
    if op == "combine_train":
        dy = s["dy"].double()[token]
        out["d_rows"] = w * dy
        d_w = torch.empty(c["T"] * c["K"], dtype=torch.float64, device=rows.device)
        d_w[s["row2slot"].long()] = torch.einsum("rh,rh->r", rows, dy)
        out["d_w"] = d_w.view(c["T"], c["K"])
    return out
