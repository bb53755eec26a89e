"""Timing cases of the router and of the microscaled 4-bit expert operators.

Each case is one call that a user's program makes, over the sizes that the
library is used at: a few decode tokens, where the call's latency counts, up to
prompts and training batches of many thousand tokens.  `run` computes a case
either through the library (`own`) or in a plain form of elementary torch
operations in 32 bits; `exact` computes it again in 64 bits.

The operators:

gate          router scores to (topk_ids, topk_weights):  scores p = softmax(l)
              or sigmoid(l) over E experts; selection by the logit (softmax) or
              by sigmoid(l) + bias; optionally only inside the topk_groups best
              of `groups` groups of experts, a group counting by the sum of its
              group_top best keys; ties go to the lowest index; weights are
              scale * p, or scale * p / sum of the selected p.
gate_train    the same with the gradient of the logits, from d_topk_weights and
              (scores) the gradient of the full scores [T, E].
mx4_rows      rows [R, C] to microscaled 4-bit form (blocks of 32 along C: e2m1
              elements, one power-of-two scale per block) and back to values.
mx4_experts   the same for a stack of expert weights [E, K, N], blocks along K.
mx4_ffn       the experts' products with 4-bit operands:
              y = sum_k w_k Q(silu(Q(x) W1g) * (Q(x) W1u)) W2, with W1, W2 held
              in 4-bit form and Q the rounding to microscaled 4-bit blocks.

The storage of a 4-bit operand [N rows, K columns], K padded to a multiple of 32:
codes   uint8 [N, K/2], two e2m1 codes a byte, the even column in the low half;
scales  uint8 [ceil(N/128), ceil(K/128), 512], the scale 2^(s - 127) of row n and
        block c (32 columns) at byte (n % 32) * 16 + (n / 32 % 4) * 4 + c % 4 of
        tile (n / 128, c / 4); bytes of no block are 0.
The rows of an up-projection are 32 gate rows, the matching 32 up rows, and so on
(the intermediate size padded to a multiple of 32 with zero rows).
"""
import math

import torch

own = False

DEVICE = "cuda"
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- the cases
def listed():
    """The smallest calls, ordinary ones and the largest, for each operator."""
    return [
        # one decode token through a grouped sigmoid router of 256 experts: latency only
        dict(name="gate, 1 token, 256 experts", op="gate", T=1, E=256, K=8, score="sigmoid",
             groups=8, topk_groups=4, group_top=2, bias=True, renorm=True, scale=2.5,
             dtype="float32"),
        # a long prompt's worth of tokens through the same router
        dict(name="gate, 65537 tokens, 256 experts", op="gate", T=65537, E=256, K=8,
             score="sigmoid", groups=8, topk_groups=4, group_top=2, bias=True, renorm=True,
             scale=2.5, dtype="float32"),
        # a training step's router: softmax over 64 experts, 6 each, bf16 logits, the full
        # scores kept for a balance loss, some experts masked out
        dict(name="gate step, 4096 tokens, 64 experts", op="gate_train", T=4096, E=64, K=6,
             score="softmax", groups=1, topk_groups=1, group_top=1, bias=False, renorm=False,
             scale=1.0, dtype="bfloat16", scores=True, masked=True),
        # the largest router step: 131072 tokens, 160 experts in 8 groups, renormalised softmax
        dict(name="gate step, 131072 tokens, 160 experts", op="gate_train", T=131072, E=160, K=6,
             score="softmax", groups=8, topk_groups=3, group_top=1, bias=False, renorm=True,
             scale=16.0, dtype="float32", scores=False, masked=False),
        # activations of a decode batch
        dict(name="mx4 rows, 128 x 7168", op="mx4_rows", R=128, C=7168, dtype="bfloat16"),
        # activations of a long prompt with an odd row count and a ragged last block
        dict(name="mx4 rows, 32767 x 2056", op="mx4_rows", R=32767, C=2056, dtype="bfloat16"),
        # the down-projections of a 64-expert layer, converted once when a model is loaded
        dict(name="mx4 experts, 64 x 1408 x 2048", op="mx4_experts", E=64, K=1408, N=2048,
             gate_up=False),
        # the up-projections of a layer of large experts
        dict(name="mx4 experts, 32 x 7168 x 4096", op="mx4_experts", E=32, K=7168, N=4096,
             gate_up=True),
        # one decode token: eight experts' weights are streamed
        dict(name="mx4 ffn, 1 token, 256 experts", op="mx4_ffn", T=1, H=7168, I=2048, E=256, K=8,
             routing="uniform", wdtype="float32"),
        # a decode batch: nearly every expert's weights are streamed
        dict(name="mx4 ffn, 128 tokens, 256 experts", op="mx4_ffn", T=128, H=7168, I=2048, E=256,
             K=8, routing="uniform", wdtype="bfloat16"),
        # a prompt: uniform routing, an intermediate size that is no multiple of 128 elements x 2
        dict(name="mx4 ffn, 4096 tokens, 64 experts", op="mx4_ffn", T=4096, H=2048, I=1408, E=64,
             K=6, routing="uniform", wdtype="bfloat16"),
        # a long prompt with hot and empty experts
        dict(name="mx4 ffn, 16384 tokens, 32 experts", op="mx4_ffn", T=16384, H=7168, I=2048,
             E=32, K=8, routing="zipf", wdtype="bfloat16"),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, n))


def _multiple(rng, lo, hi, step):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    n = max(lo, _log_int(rng, lo, hi) // step * step)
    return n - step if n in (1536, 3072) else n


def draw(rng):
    op = rng.choice(["gate", "gate_train", "mx4_rows", "mx4_experts", "mx4_ffn", "mx4_ffn"])
    if op in ("gate", "gate_train"):
        groups = rng.choice([1, 1, 4, 8])
        E = groups * (rng.randint(4, 64) if groups > 1 else rng.randint(4, 384))
        topk_groups = 1 if groups == 1 else rng.randint(2, groups)
        score, renorm = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6
        # (one renormalised expert always has weight 1 and no gradient)
        K = min(rng.randint(2 if renorm else 1, 8), E // groups * topk_groups)
        T = _log_int(rng, 1, 131071) | 1
        while T * E > 131072 * 160:
            T //= 2
        c = dict(op=op, T=T, E=E, K=K, score=score, groups=groups, topk_groups=topk_groups,
                 group_top=1 if score == "softmax" else rng.choice([1, 2]),
                 bias=score == "sigmoid" and rng.random() < 0.7, renorm=renorm,
                 scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["float32", "bfloat16"]))
        if op == "gate_train":
            c.update(scores=rng.random() < 0.4, masked=rng.random() < 0.3)
        return c
    if op == "mx4_rows":
        return dict(op=op, R=_log_int(rng, 1, 32767) | 1, C=_multiple(rng, 64, 7168, 8),
                    dtype=rng.choice(["bfloat16", "float32"]))
    if op == "mx4_experts":
        gate_up = rng.random() < 0.5
        N = _multiple(rng, 64, 4096, 8)
        if gate_up:
            N = N // 16 * 16
        return dict(op=op, E=rng.randint(1, 32), K=_multiple(rng, 64, 7168, 8), N=N, gate_up=gate_up)
    E = rng.choice([8, 16, 30, 64, 96])
    H = _multiple(rng, 256, 7168, 8)
    I = _multiple(rng, 128, 2048, 8)
    while E * H * I > 96 * 2048 * 2048:
        E //= 2
    K = min(rng.randint(1, 8), E)
    return dict(op=op, T=_log_int(rng, 1, 8191) | 1, H=H, I=I, E=E, K=K,
                routing=rng.choice(["uniform", "zipf"]),
                wdtype=rng.choice(["float32", "bfloat16"]))


def _touched(c):
    """Experts that receive a token, on average, for uniform routing."""
    return c["E"] * (1.0 - (1.0 - c["K"] / c["E"]) ** c["T"])


def work(c):
    op = c["op"]
    if op in ("gate", "gate_train"):
        b = 4 if c["dtype"] == "float32" else 2
        n = c["T"] * c["E"]
        d = dict(bytes=n * b + c["T"] * c["K"] * 8 + (c["E"] * 4 if c["bias"] else 0), flops=5 * n)
        if op == "gate_train":
            d["bytes"] += n * b + c["T"] * c["K"] * 4 + (n * 8 if c["scores"] else 0)
            d["flops"] += 4 * n
        return d
    if op == "mx4_rows":
        n, b = c["R"] * c["C"], 4 if c["dtype"] == "float32" else 2
        return dict(bytes=n * (2 * b + 0.53125), flops=4 * n)
    if op == "mx4_experts":
        n = c["E"] * c["K"] * c["N"]
        return dict(bytes=n * (4 + 0.53125), flops=4 * n)
    weights = _touched(c) * 3 * c["H"] * c["I"] * 0.53125
    wb = 4 if c["wdtype"] == "float32" else 2
    return dict(bytes=weights + 4 * c["T"] * c["H"] + c["T"] * c["K"] * (4 + wb),
                flops=6 * c["T"] * c["K"] * c["H"] * c["I"])


# ------------------------------------------------------------------ the inputs
def _round_up(n, m):
    return (n + m - 1) // m * m


def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _pack(v):
    """fp32 values [E, N, K], K a multiple of 32, to stored codes and scales."""
    E, N, K = v.shape
    blocks = v.view(E, N, K // 32, 32)
    amax = blocks.abs().amax(-1)
    exp = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)
    m = (blocks * ((127 - exp) << 23).view(torch.float32).unsqueeze(-1)).abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5)
            + (m >= 3.5) + (m > 5.0) + (blocks < 0).to(torch.uint8) * 8)
    code = code.view(E, N, K // 2, 2)
    codes = code[..., 0] + code[..., 1] * 16
    nb, kb = _round_up(N, 128) // 128, _round_up(K, 128) // 128
    s = torch.zeros((E, nb * 128, kb * 4), dtype=torch.uint8, device=v.device)
    s[:, :N, :K // 32] = (exp + 127).to(torch.uint8)
    s = s.view(E, nb, 4, 32, kb, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, nb, kb, 512)
    return codes, s


def _routing(g, c):
    T, E, K = c["T"], c["E"], c["K"]
    u = torch.rand((T, E), generator=g, device=DEVICE).clamp_min_(1e-12)
    key = -torch.log(-torch.log(u).clamp_min_(1e-12))
    if c["routing"] == "zipf":
        p = torch.arange(1, E + 1, device=DEVICE, dtype=torch.float32).pow(-1.2)
        empty = min(3, E - K)
        if empty > 0:
            p[E - empty:] = 0
        key = key + torch.log(p[torch.randperm(E, generator=g, device=DEVICE)])
    ids = torch.argsort(key, dim=1, descending=True)[:, :K].to(torch.int32).contiguous()
    w = torch.softmax(torch.randn((T, K), generator=g, device=DEVICE), dim=1)
    return ids, w.to(getattr(torch, c["wdtype"]))


def prepare(c, seed):
    g, op = _gen(seed), c["op"]

    def expert_weights(E, rows, cols, gate_up, std):
        """A stored stack of E operands [rows, cols], made a few experts at a time."""
        kp = _round_up(cols, 32)
        half = rows // 2 if gate_up else rows
        hp = _round_up(half, 32) if gate_up else half
        parts = []
        step = max(1, (1 << 27) // (rows * cols))
        for e0 in range(0, E, step):
            n = min(E, e0 + step) - e0
            w = torch.randn((n, rows, cols), generator=g, device=DEVICE) * std
            if gate_up:
                both = torch.zeros((n, 2, hp, kp), device=DEVICE)
                both[:, :, :half, :cols] = w.view(n, 2, half, cols)
                v = both.view(n, 2, hp // 32, 32, kp).transpose(1, 2).reshape(n, 2 * hp, kp)
            else:
                v = torch.zeros((n, rows, kp), device=DEVICE)
                v[:, :, :cols] = w
            parts.append(_pack(v))
        return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])

    if op in ("gate", "gate_train"):
        T, E, K = c["T"], c["E"], c["K"]
        logits = 1.5 * torch.randn((T, E), generator=g, device=DEVICE)
        s = dict(case=c)
        if c.get("masked"):
            # a tenth of the experts closed to a token, and one token that has none left
            logits = logits.masked_fill(
                torch.rand((T, E), generator=g, device=DEVICE) < 0.1, -math.inf)
            logits[T // 2] = -math.inf
        s["logits"] = logits.to(getattr(torch, c["dtype"]))
        # balance biases move in fixed small steps
        s["bias"] = (torch.randint(-50, 51, (E,), generator=g, device=DEVICE).float() * 1e-3
                     if c["bias"] else None)
        if op == "gate_train":
            s["d_weights"] = torch.randn((T, K), generator=g, device=DEVICE)
            s["d_scores"] = (torch.randn((T, E), generator=g, device=DEVICE) * 0.01
                             if c["scores"] else None)
        return s
    if op == "mx4_rows":
        x = torch.randn((c["R"], c["C"]), generator=g, device=DEVICE)
        return dict(case=c, x=x.to(getattr(torch, c["dtype"])))
    if op == "mx4_experts":
        w = torch.empty((c["E"], c["K"], c["N"]), dtype=torch.bfloat16, device=DEVICE)
        return dict(case=c, w=w.normal_(0.0, c["K"] ** -0.5, generator=g))
    ids, w = _routing(g, c)
    counts = torch.bincount(ids.flatten().long(), minlength=c["E"])
    up = expert_weights(c["E"], 2 * c["I"], c["H"], True, c["H"] ** -0.5)
    down = expert_weights(c["E"], c["H"], c["I"], False, c["I"] ** -0.5)
    x = torch.randn((c["T"], c["H"]), generator=g, device=DEVICE).to(torch.bfloat16)
    return dict(case=c, x=x, ids=ids, w=w, up=up, down=down,
                most=int(counts.max()))  # the plain form's room for an expert


# -------------------------------------------------------------- the plain form
def _plain_scores(logits, score):
    l = logits.float()
    if score == "sigmoid":
        return l, 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(torch.isinf(top), 0.0, top))
    total = e.sum(1, keepdim=True)
    return l, e / torch.where(total == 0, 1.0, total)


def _plain_gate(c, s):
    l, p = _plain_scores(s["logits"], c["score"])
    key = l if c["score"] == "softmax" else p
    if s["bias"] is not None:
        key = key + s["bias"]
    T, E, G = c["T"], c["E"], c["groups"]
    if G > 1:
        best = key.view(T, G, E // G).sort(dim=2, descending=True)[0]
        group = best[:, :, 0] if c["group_top"] == 1 else best[:, :, 0] + best[:, :, 1]
        rank = group.sort(dim=1, descending=True, stable=True)[1][:, :c["topk_groups"]]
        open_ = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, rank, True)
        # experts of closed groups come after every expert of an open one
        order = torch.where(open_.repeat_interleave(E // G, 1),
                            key.clamp_min(torch.finfo(torch.float32).min), -math.inf)
    else:
        order = key
    ids = order.sort(dim=1, descending=True, stable=True)[1][:, :c["K"]]
    w = p.gather(1, ids)
    total = w.sum(1, keepdim=True)
    if c["renorm"]:
        w = w / torch.where(total == 0, 1.0, total)
    return p, ids, w * c["scale"], total


def _plain_gate_train(c, s):
    p, ids, w, total = _plain_gate(c, s)
    dw = s["d_weights"] * c["scale"]
    if c["renorm"]:
        n = w / c["scale"]
        dw = (dw - (dw * n).sum(1, keepdim=True)) / torch.where(total == 0, 1.0, total)
    dp = torch.zeros_like(p).scatter_(1, ids, dw)
    if s["d_scores"] is not None:
        dp = dp + s["d_scores"]
    if c["score"] == "sigmoid":
        dl = dp * p * (1.0 - p)
    else:
        dl = p * (dp - (dp * p).sum(1, keepdim=True))
    return p, ids, w, dl.to(s["logits"].dtype)


def _plain_blocks(b):
    """Blocks [..., 32] rounded to 4-bit values (fp32)."""
    amax = b.abs().amax(-1, keepdim=True)
    exp = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)
    up = ((127 - exp) << 23).view(torch.float32)  # 2^-exp
    down = torch.where(exp == -127, 2.0 ** -127, ((exp + 127) << 23).view(torch.float32))
    m = (b * up).abs()
    r = (0.5 * (m > 0.25) + 0.5 * (m >= 0.75) + 0.5 * (m > 1.25) + 0.5 * (m >= 1.75)
         + (m > 2.5) + (m >= 3.5) + 2.0 * (m > 5.0))
    return torch.where(b < 0, -r, r) * down


def _plain_rows(v):
    R, C = v.shape
    cp = _round_up(C, 32)
    f = v.float() if cp == C else torch.cat([v.float(), v.new_zeros((R, cp - C)).float()], 1)
    return _plain_blocks(f.view(R, cp // 32, 32)).view(R, cp)


def _plain_stored(codes, scales):
    """Stored codes and scales to fp32 values [E, N, K]."""
    E, N, half = codes.shape
    t = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    pairs = torch.stack([t.repeat(16), t.repeat_interleave(16)], 1)
    v = pairs[codes.int()].view(E, N, half // 16, 32)
    nb, kb = scales.shape[1:3]
    s = scales.view(E, nb, kb, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, nb * 128, kb * 4)
    s = s[:, :N, :half // 16].int()
    s = torch.where(s == 0, 2.0 ** -127, (s << 23).view(torch.float32))
    return v.mul_(s.unsqueeze(-1)).view(E, N, half * 2)


def _plain_ffn(c, s):
    T, H, E, K = c["T"], c["H"], c["E"], c["K"]
    flat, most, up, down = s["ids"].flatten().long(), s["most"], s["up"], s["down"]
    if T * K <= E:  # few slots: their experts' weights alone, one slot each
        up, down = [t[flat] for t in up], [t[flat] for t in down]
        flat, most, E = torch.arange(T * K, device=flat.device), 1, T * K
    by_expert = torch.argsort(flat, stable=True)
    in_order = flat[by_expert]
    first = torch.searchsorted(in_order, torch.arange(E, device=flat.device))
    place = torch.empty_like(flat)
    place[by_expert] = torch.arange(T * K, device=flat.device) - first[in_order]
    x = _plain_rows(s["x"])
    rows = torch.zeros((E, most, x.shape[1]), device=x.device)
    rows[flat, place] = x.repeat_interleave(K, 0)
    h = torch.bmm(rows, _plain_stored(*up).transpose(1, 2)).view(E, most, -1, 2, 32)
    g, u = h[:, :, :, 0], h[:, :, :, 1]
    a = _plain_blocks(g / (1.0 + torch.exp(-g)) * u).view(E, most, -1)
    o = torch.bmm(a, _plain_stored(*down).transpose(1, 2))
    o = o[flat, place].view(T, K, H)
    return (o * s["w"].float().unsqueeze(-1)).sum(1).to(torch.bfloat16)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "gate":
        p, ids, w, _ = _plain_gate(c, s)
        return dict(ids=ids.int(), weights=w)
    if op == "gate_train":
        p, ids, w, dl = _plain_gate_train(c, s)
        out = dict(ids=ids.int(), weights=w, d_logits=dl)
        if c["scores"]:
            out["scores"] = p
        return out
    if op == "mx4_rows":
        return dict(values=_plain_rows(s["x"])[:, :c["C"]].to(s["x"].dtype))
    if op == "mx4_experts":
        E, K, N = s["w"].shape
        kp = _round_up(K, 32)
        w = s["w"].float()
        if kp != K:
            w = torch.cat([w, w.new_zeros((E, kp - K, N))], 1)
        v = _plain_blocks(w.view(E, kp // 32, 32, N).transpose(2, 3))
        return dict(values=v.transpose(2, 3).reshape(E, kp, N)[:, :K].to(torch.bfloat16))
    return dict(y=_plain_ffn(c, s))


# --------------------------------------------------------- through the library
def _own(s):
    import dispatch_grouped_gemm_gb300 as hmm

    c = s["case"]
    op = c["op"]
    if op in ("gate", "gate_train"):
        kw = dict(score=c["score"], bias=s["bias"], groups=c["groups"],
                  topk_groups=c["topk_groups"], group_top=c["group_top"],
                  renormalize=c["renorm"], scale=c["scale"])
        if op == "gate":
            ids, w = hmm.moe_gate(s["logits"], c["K"], **kw)
            return dict(ids=ids, weights=w)
        logits = s["logits"].detach().requires_grad_()
        out = hmm.moe_gate(logits, c["K"], return_scores=c["scores"], **kw)
        if c["scores"]:
            (dl,) = torch.autograd.grad((out[1], out[2]), logits, (s["d_weights"], s["d_scores"]))
            return dict(ids=out[0], weights=out[1].detach(), d_logits=dl, scores=out[2].detach())
        (dl,) = torch.autograd.grad(out[1], logits, s["d_weights"])
        return dict(ids=out[0], weights=out[1].detach(), d_logits=dl)
    if op == "mx4_rows":
        return dict(values=hmm.mx4_quantize(s["x"]).dequantize(s["x"].dtype))
    if op == "mx4_experts":
        q = hmm.mx4_quantize_experts(s["w"], gate_up=c["gate_up"])
        return dict(values=q.dequantize(torch.bfloat16))
    up = hmm.Mx4Tensor.experts(*s["up"], K=c["H"], N=2 * c["I"], gate_up=True)
    down = hmm.Mx4Tensor.experts(*s["down"], K=c["I"], N=c["H"])
    return dict(y=hmm.moe_ffn_mx4(s["x"], s["ids"], s["w"], up, down))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- in 64 bits
def _exact_gate(c, s):
    l = s["logits"].double()
    if c["score"] == "sigmoid":
        p = torch.special.expit(l)
        key = p.clone()
    else:
        dead = torch.isneginf(l).all(1, keepdim=True)
        p = torch.where(dead, 0.0, torch.softmax(torch.where(dead, 0.0, l), 1))
        key = l.clone()
    if s["bias"] is not None:
        key += s["bias"].double()
    n = c["E"] // c["groups"]
    if c["groups"] > 1:
        per = key.unflatten(1, (c["groups"], n))
        worth = per.topk(c["group_top"], dim=2).values.sum(2)
        cut = worth.argsort(dim=1, descending=True, stable=True)[:, c["topk_groups"]:]
        per.clamp_(min=torch.finfo(torch.float64).min)
        per.scatter_(1, cut.unsqueeze(2).expand(-1, -1, n), -math.inf)
    ids = key.argsort(dim=1, descending=True, stable=True)[:, :c["K"]]
    w = torch.gather(p, 1, ids)
    out = dict(ids=None)
    total = w.sum(1, keepdim=True)
    safe = torch.where(total > 0, total, 1.0)
    out["weights"] = c["scale"] * (w / safe if c["renorm"] else w)
    if c["op"] == "gate":
        return out
    # gradient with respect to p, then through p's own derivative
    up = c["scale"] * s["d_weights"].double()
    if c["renorm"]:
        up = up / safe - (up * w).sum(1, keepdim=True) / safe ** 2
    dp = s["d_scores"].double().clone() if s["d_scores"] is not None else torch.zeros_like(p)
    dp.scatter_add_(1, ids, up)
    if c["score"] == "sigmoid":
        out["d_logits"] = dp * p * torch.special.expit(-l)
    else:
        out["d_logits"] = dp * p - p * torch.einsum("te,te->t", dp, p).unsqueeze(1)
    if c["scores"]:
        out["scores"] = p
    return out


def _exact_round(v, dim):
    """Blocks of 32 along dim (the last ones short), in 64 bits."""
    v = v.double().movedim(dim, -1)
    n = v.shape[-1]
    b = torch.nn.functional.pad(v, (0, -n % 32)).unflatten(-1, (-1, 32))
    big = b.abs().max(-1, keepdim=True).values
    e = torch.floor(torch.log2(torch.where(big > 0, big, 1.0)))
    e = torch.where(torch.exp2(e + 1) <= big, e + 1, torch.where(torch.exp2(e) > big, e - 1, e))
    scale = torch.exp2((e - 2).clamp(-127, 127))
    q = b / scale
    step = torch.where(q.abs() < 2, 0.5, torch.where(q.abs() < 4, 1.0, 2.0))
    q = (torch.round(q / step) * step).clamp(-6, 6)
    return (q * scale).flatten(-2)[..., :n].movedim(-1, dim)


def _exact_stored(codes, scales, rows, cols):
    """One expert's stored operand [rows, cols] in 64 bits."""
    low, high = (codes & 15).long(), (codes >> 4).long()
    c = torch.stack([low, high], -1).flatten(-2)[:rows, :cols]
    m, e = c & 1, (c >> 1) & 3
    v = torch.where(e == 0, 0.5 * m.double(), (1 + 0.5 * m.double()) * torch.exp2(e.double() - 1))
    v = torch.where(c >= 8, -v, v)
    r = torch.arange(rows, device=codes.device).unsqueeze(1)
    b = (torch.arange(cols, device=codes.device) // 32).unsqueeze(0)
    s = scales[r // 128, b // 4, r % 32 * 16 + r // 32 % 4 * 4 + b % 4]
    return v * torch.exp2(s.double() - 127)


def exact(c, seed):
    op = c["op"]
    if op == "mx4_ffn" and c["T"] * c["K"] * c["H"] * c["I"] > 5e11:
        return None  # minutes in 64 bits
    s = prepare(c, seed)
    if op in ("gate", "gate_train"):
        return _exact_gate(c, s)
    if op == "mx4_rows":
        return dict(values=_exact_round(s["x"], 1))
    if op == "mx4_experts":
        if s["w"].numel() > 3e8:
            return None  # tens of GB in 64 bits
        return dict(values=_exact_round(s["w"], 1))
    x = _exact_round(s["x"], 1)
    y = torch.zeros_like(x)
    j = torch.arange(c["I"], device=x.device)
    gate_rows = j // 32 * 64 + j % 32
    ip = _round_up(c["I"], 32)
    for e in range(c["E"]):
        t, k = torch.nonzero(s["ids"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        w1 = _exact_stored(s["up"][0][e], s["up"][1][e], 2 * ip, c["H"])
        g, u = x[t] @ w1[gate_rows].T, x[t] @ w1[gate_rows + 32].T
        a = _exact_round(g * torch.special.expit(g) * u, 1)
        w2 = _exact_stored(s["down"][0][e], s["down"][1][e], c["H"], c["I"])
        y.index_add_(0, t, (a @ w2.T) * s["w"][t, k].double().unsqueeze(1))
    return dict(y=y)
