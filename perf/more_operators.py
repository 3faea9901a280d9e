"""The expert layer's router, products with 4-bit weights and orthogonalised updates, as cases
that can be timed and checked.

Three families, each in its plain form (elementary torch operations in 32 bits, in 64 where a
choice or a long sum hangs on the last bits, rounded once at the end) and as the calls of this
library:

  gate  the experts that each token takes: the k largest scores, their weights, the slots per
        expert and the balance loss; and the logits' gradient (gate_back)
  w4    the forward product of expert rows with 4-bit weights: whole-number codes with one scale
        (and zero point) per group of 32, 64 or 128, or e2m1 codes with a power of two per 32
  orth  the nearest-to-orthogonal form of a weight update by five Newton-Schulz steps

`own` chooses between the two. The inputs come from the case and a seed alone.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
TINY = 1e-20  # beside the sum of a token's chosen scores


def _ceil(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decoding step of a few sequences: scores by sigmoid, a bias that evens out the load;
        # no statistics; latency
        dict(name="gate_step", op="gate", T=8, G=256, k=8, dtype="bf16", sigmoid=True, norm=True,
             bias=True, mask=False, stats=False),
        # a training step's tokens, with the balance loss: bandwidth
        dict(name="gate_train", op="gate", T=65536, G=256, k=8, dtype="f32", sigmoid=False,
             norm=True, bias=False, mask=False, stats=True),
        # odd sizes; experts that are switched off and padding rows without any
        dict(name="gate_odd", op="gate", T=5003, G=37, k=3, dtype="f32", sigmoid=True, norm=False,
             bias=True, mask=True, stats=True),
        # the same training step's gradient
        dict(name="gate_back", op="gate_back", T=65536, G=256, k=8, dtype="f32", sigmoid=False,
             norm=True, bias=False, mask=False, stats=True),
        # one token through one linear layer: latency
        dict(name="w4_token", op="w4", M=1, G=1, N=4096, K=7168, kind="int", group=128, zero=True,
             scale="bf16", out="bf16", pad=0),
        # a decoding step through 32 experts: every weight is read for a few rows
        dict(name="w4_step", op="w4", M=64, G=32, N=4096, K=7168, kind="int", group=128, zero=False,
             scale="bf16", out="bf16", pad=0),
        # more experts and sequences, the float format
        dict(name="w4_float", op="w4", M=256, G=64, N=2048, K=7168, kind="e2m1", group=32,
             zero=False, scale="e8m0", out="bf16", pad=0),
        # a prompt's tokens on one rank's experts
        dict(name="w4_prompt", op="w4", M=16384, G=8, N=4096, K=7168, kind="e2m1", group=32,
             zero=False, scale="e8m0", out="bf16", pad=0),
        # odd sizes, fp32 scales and results, rows of a wider matrix
        dict(name="w4_odd", op="w4", M=517, G=5, N=1000, K=1056, kind="int", group=32, zero=True,
             scale="f32", out="f32", pad=40),
        # small experts
        dict(name="orth_small", op="orth", G=8, R=384, C=256, dtype="f32"),
        # odd sizes
        dict(name="orth_odd", op="orth", G=3, R=777, C=1000, dtype="bf16"),
        # one rank's expert weights
        dict(name="orth_experts", op="orth", G=8, R=4096, C=7168, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "gate", "gate_back", "w4", "w4", "w4", "orth", "orth"])
    if op in ("gate", "gate_back"):
        G = _log_int(rng, 2, 1024)
        return dict(op=op, T=_log_int(rng, 1, min(65536, 65536 * 256 // G)), G=G,
                    k=rng.randint(1, min(8, G)), dtype=rng.choice(["f32", "bf16"]),
                    sigmoid=rng.choice([True, False]), norm=rng.choice([True, False]),
                    bias=op == "gate" and rng.choice([True, False]),
                    mask=rng.choice([True, False, False]), stats=op == "gate_back" or
                    rng.choice([True, True, False]))
    if op == "w4":
        kind = rng.choice(["int", "int", "e2m1"])
        group = 32 if kind == "e2m1" else rng.choice([32, 64, 128])
        G = _log_int(rng, 1, 64)
        K = group * _log_int(rng, max(1, 128 // group), 8192 // group)
        N = _log_int(rng, 64, max(65, min(8192, 900_000_000 // (G * K))))
        M = _log_int(rng, 1, max(2, min(16384, 450_000_000_000 // (N * K))))
        return dict(op=op, M=M, G=G, N=N, K=K, kind=kind, group=group,
                    zero=kind == "int" and rng.choice([True, False]),
                    scale="e8m0" if kind == "e2m1" else rng.choice(["bf16", "f32"]),
                    out=rng.choice(["bf16", "bf16", "f32"]),
                    pad=rng.choice([0, 0, 8 * rng.randint(1, 40)]))
    R, C = _log_int(rng, 16, 7168), _log_int(rng, 16, 7168)
    n, m = min(R, C), max(R, C)
    G = _log_int(rng, 1, max(2, min(64, 3_000_000_000_000 // (4 * n * n * m + 2 * n ** 3))))
    return dict(op=op, G=G, R=R, C=C, dtype=rng.choice(["f32", "bf16"]))


def work(case):
    if case["op"] in ("gate", "gate_back"):
        T, G, k, e = case["T"], case["G"], case["k"], TYPES[case["dtype"]].itemsize
        if case["op"] == "gate":  # logits in; idx and w out
            return dict(bytes=T * G * e + T * k * 8 + (G * 8 if case["stats"] else 0),
                        flops=8 * T * G)
        return dict(bytes=2 * T * G * e + T * k * 8 + G * 4, flops=12 * T * G)
    if case["op"] == "w4":
        M, G, N, K = (case[x] for x in "MGNK")
        live = G * (1 - (1 - 1 / G) ** M)  # experts that get a row, of even chances
        per = {"bf16": 2, "f32": 4, "e8m0": 1}[case["scale"]] + (1 if case["zero"] else 0)
        return dict(bytes=int(live * N * (K // 2 + K // case["group"] * per) + M * K * 2 +
                              M * N * TYPES[case["out"]].itemsize), flops=2 * M * N * K)
    n, m = sorted((case["R"], case["C"]))  # X X^T and A A are symmetric: half of each
    return dict(bytes=case["G"] * n * m * (TYPES[case["dtype"]].itemsize + 2),
                flops=case["G"] * 5 * (3 * n * n * m + n ** 3))


# --------------------------------------------------------------------------------- inputs

def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda")


def _prepare_gate(case, gen, s):
    T, G, k = case["T"], case["G"], case["k"]
    x = 1.5 * _randn(gen, T, G) + 0.7 * _randn(gen, G)
    if case["mask"]:  # one expert at least stays on
        off = _rand(gen, G) < 0.125
        off[0] = False
        x[:, off] = -math.inf
        x[_rand(gen, T) < 0.0625] = -math.inf
    s["x"] = x.to(TYPES[case["dtype"]])
    s["bias"] = 0.05 * _randn(gen, G) if case["bias"] else None
    s["scale"] = 2.5 if case["norm"] and case["sigmoid"] else 1.0
    s["coef"] = 0.01 * G / (k * T * T)
    if case["op"] == "gate_back":  # what the forward pass left, and the loss's gradients
        idx = _plain_choice(s["x"].double(), k)
        s["idx"] = idx.to(torch.int32)
        s["counts"] = (idx.view(-1, 1) == torch.arange(G, device="cuda")).sum(0).to(torch.int32)
        s["dw"] = _randn(gen, T, k) * 1e-3
        s["dloss"] = 0.5 + _rand(gen, 1)
    if own:
        import fp8_grouped_gemm_tn_amd as kg
        new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")
        s["flags"] = (kg.KG_GATE_SIGMOID if case["sigmoid"] else 0) | \
            (kg.KG_GATE_NORM if case["norm"] else 0)
        if case["op"] == "gate":
            stats = case["stats"]
            s["idx"], s["w"] = new((T, k), torch.int32), new((T, k), torch.float32)
            s["counts"] = new((G,), torch.int32) if stats else None
            s["psum"] = new((G,), torch.float32) if stats else None
            s["loss"] = new((1,), torch.float32) if stats else None
            s["ws"] = kg.new_gate_workspace(T, G, "cuda") if stats else None
        else:
            s["dx"] = torch.empty_like(s["x"])


def _counts(case, gen):
    """Rows per expert: a skewed draw that adds up to M (an expert may have none)."""
    M, G = case["M"], case["G"]
    p = torch.softmax(0.35 * _randn(gen, G), dim=0)
    to = torch.multinomial(p, M, replacement=True, generator=gen)
    return (to[:, None] == torch.arange(G, device="cuda")).sum(0).to(torch.int32)


def _prepare_w4(case, gen, s):
    M, G, N, K, group = (case[x] for x in ("M", "G", "N", "K", "group"))
    s["A"] = torch.zeros((M, K + case["pad"]), dtype=torch.bfloat16, device="cuda")[:, :K]
    s["A"].copy_(_randn(gen, M, K))
    # codes as rounding normal weights gives them, two in a byte, the even channel's low
    q = torch.empty((G, N, K // 2), dtype=torch.uint8, device="cuda")
    sw = torch.empty((G, N, K // group), device="cuda")
    zp = torch.empty((G, N, K // group), dtype=torch.uint8, device="cuda")
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for g in range(G):
        w = (_randn(gen, N, K) * K ** -0.5).view(N, -1, group)
        if case["kind"] == "e2m1":
            e = torch.floor(torch.log2(w.abs().amax(2))) - 2
            sw[g] = e + 127
            y = w / torch.exp2(e)[..., None]
            c = (torch.bucketize(y.abs(), edges) + 8 * (y < 0)).to(torch.uint8)
        else:
            lo, hi = w.amin(2), w.amax(2)
            if case["zero"]:
                sw[g] = (hi - lo) / 15
                zp[g] = (-lo / sw[g]).round().clamp(0, 15).to(torch.uint8)
            else:
                sw[g] = torch.maximum(-lo, hi) / 7.5
                zp[g] = 8
            sw[g] = sw[g].to(TYPES[case["scale"]]).float()
            c = (w / sw[g][..., None]).round() + zp[g][..., None]
            c = c.clamp(0, 15).to(torch.uint8)
        c = c.view(N, K // 2, 2)
        q[g] = c[..., 0] | (c[..., 1] << 4)
    s["W"], s["sw"] = q, sw.to(torch.uint8 if case["scale"] == "e8m0" else TYPES[case["scale"]])
    s["zp"] = zp if case["zero"] else None
    s["ms"] = _counts(case, gen)
    s["most"] = int(s["ms"].max())
    s["D"] = torch.empty((M, N), dtype=TYPES[case["out"]], device="cuda")


def _prepare_orth(case, gen, s):
    # a gradient's momentum: noise, a few directions that stand out, channels of unlike size
    G, R, C = case["G"], case["R"], case["C"]
    u = _randn(gen, G, R, C) * torch.exp(0.5 * _randn(gen, G, 1, C))
    few = min(4, R, C)
    u += 2 * torch.bmm(_randn(gen, G, R, few), _randn(gen, G, few, C))
    s["U"] = (u * 1e-3).to(TYPES[case["dtype"]])
    if own:
        import fp8_grouped_gemm_tn_amd as kg
        s["O"] = torch.empty((G, R, C), dtype=torch.bfloat16, device="cuda")
        s["ws"] = kg.new_orthogonalize_workspace(G, R, C, "cuda")


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(int(seed))
    s = dict(case=case)
    if case["op"] in ("gate", "gate_back"):
        _prepare_gate(case, gen, s)
    elif case["op"] == "w4":
        _prepare_w4(case, gen, s)
    else:
        _prepare_orth(case, gen, s)
    return s


# ----------------------------------------------------------------------------- plain forms

def _plain_choice(key, k):
    """The k largest per row, descending, ties to the lower index; -1 for a key of -inf."""
    top, idx = torch.sort(key, dim=1, descending=True, stable=True)
    return torch.where(top[:, :k] == -math.inf, -1, idx[:, :k])


def _plain_scores(x, sigmoid):
    """Scores and the probabilities of the balance loss; zeros for a row without experts."""
    if sigmoid:
        s = 1 / (1 + torch.exp(-x))
        total = s.sum(1, keepdim=True)
        return s, torch.where(total > 0, s / total, 0.0), total
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(1, keepdim=True)
    p = torch.where(total > 0, e / total, 0.0)
    return p, p, total


def _plain_gate(s):
    c, x = s["case"], s["x"].float()
    p, prob, _ = _plain_scores(x, c["sigmoid"])
    key = x.double()
    if s["bias"] is not None:  # a choice may hang on the last bit: 64 bits
        key = _plain_scores(key, c["sigmoid"])[0] + s["bias"].double()
        key = torch.where(x == -math.inf, -math.inf, key)
    idx = _plain_choice(key, c["k"])
    w = torch.where(idx < 0, 0.0, p.gather(1, idx.clamp(min=0)))
    if c["norm"]:
        w = w / (w.sum(1, keepdim=True) + TINY)
    out = dict(idx=idx.to(torch.int32), w=w * s["scale"])
    if c["stats"]:
        counts = torch.zeros(c["G"] + 1, dtype=torch.int64, device="cuda")
        flat = torch.where(idx < 0, c["G"], idx).view(-1)
        counts = counts.scatter_add_(0, flat, torch.ones_like(flat))[:c["G"]]
        psum = prob.double().sum(0)
        loss = (s["coef"] * counts * psum).sum().view(1)
        out.update(counts=counts.to(torch.int32), psum=psum.float(), loss=loss.float())
    return out


def _plain_gate_back(s):
    c, x = s["case"], s["x"].float()
    p, prob, total = _plain_scores(x, c["sigmoid"])
    idx = s["idx"].long()
    chosen = torch.where(idx < 0, 0.0, p.gather(1, idx.clamp(min=0)))
    dw = torch.where(idx < 0, 0.0, s["dw"])
    if c["norm"]:
        sum_ = chosen.sum(1, keepdim=True) + TINY
        d = (dw - (dw * chosen).sum(1, keepdim=True) / sum_) / sum_
    else:
        d = dw
    d = torch.where(idx < 0, 0.0, d * s["scale"])
    ds = torch.zeros_like(x).scatter_add_(1, idx.clamp(min=0), d)
    db = s["dloss"] * s["coef"] * s["counts"].float()[None]
    if c["sigmoid"]:
        even = (db - (db * prob).sum(1, keepdim=True)) / total
        dx = p * (1 / (1 + torch.exp(x))) * (ds + torch.where(total > 0, even, 0.0))
        dx = torch.where(x == -math.inf, 0.0, dx)
    else:
        dp = ds + db
        dx = p * (dp - (p * dp).sum(1, keepdim=True))
    return dict(dx=dx.to(s["x"].dtype))


def _plain_w4(s):
    c, ms = s["case"], s["ms"].long()
    M, G, N, K, group = (c[x] for x in ("M", "G", "N", "K", "group"))
    q = torch.stack((s["W"] & 15, s["W"] >> 4), dim=3).view(G, N, K // group, group)
    if c["kind"] == "e2m1":
        table = torch.tensor(E2M1 + [-v for v in E2M1], device="cuda")
        w = table[q.int()]
        w *= torch.exp2(s["sw"].float() - 127)[..., None]
    else:
        w = q.float()
        w -= 8.0 if s["zp"] is None else s["zp"].float()[..., None]
        w *= s["sw"].float()[..., None]
    row = torch.arange(M, device="cuda")
    end = ms.cumsum(0)
    g = (row[:, None] >= end).sum(1)  # the expert of each row
    at = row - (end - ms)[g]
    padded = torch.zeros((G, s["most"], K), device="cuda")
    padded[g, at] = s["A"].float()
    y = torch.bmm(padded, w.view(G, N, K).transpose(1, 2).contiguous())
    return dict(y=y[g, at].to(TYPES[c["out"]]))


def _plain_orth(s):
    u = s["U"].float()
    wide = s["case"]["R"] <= s["case"]["C"]
    x = u if wide else u.transpose(1, 2).contiguous()
    size = x.double().square().sum((1, 2), keepdim=True).sqrt().float()
    x = torch.where(size > 0, x / size, 0.0)
    for _ in range(5):
        a = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = NS_A * x + torch.bmm(NS_B * a + NS_C * torch.bmm(a, a), x)
    x = x if wide else x.transpose(1, 2)
    return dict(o=x.to(torch.bfloat16).contiguous())


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "gate":
        return _plain_gate(s)
    if op == "gate_back":
        return _plain_gate_back(s)
    return _plain_w4(s) if op == "w4" else _plain_orth(s)


# ------------------------------------------------------------------------ the library's calls

def _run_own(s, op):
    import fp8_grouped_gemm_tn_amd as kg
    if op == "gate":
        kg.kg_gate(s["x"], s["case"]["k"], s["bias"], s["flags"], s["scale"], s["coef"], s["idx"],
                   s["w"], s["counts"], s["psum"], s["loss"], s["ws"])
        out = dict(idx=s["idx"], w=s["w"])
        return dict(out, counts=s["counts"], psum=s["psum"], loss=s["loss"]) \
            if s["case"]["stats"] else out
    if op == "gate_back":
        kg.kg_gate_bwd(s["x"], s["idx"], s["dw"], s["counts"], s["dloss"], s["flags"], s["scale"],
                       s["coef"], s["dx"])
        return dict(dx=s["dx"])
    if op == "w4":
        kg.kg_fprop_w4(s["A"], s["W"], s["sw"], s["D"], s["ms"], s["zp"])
        return dict(y=s["D"])
    kg.kg_orthogonalize(s["U"], s["O"], 5, s["ws"])
    return dict(o=s["O"])


# ---------------------------------------------------------------------- the definitions in 64 bits

def _exact_probs(x, sigmoid):
    """Scores, balance probabilities and the sum of the scores: by logarithms."""
    dead = torch.isneginf(x).all(1, keepdim=True)
    if sigmoid:
        s = torch.special.expit(x)
        total = s.sum(1, keepdim=True)
        return s, torch.where(dead, 0.0, s / torch.where(dead, 1.0, total)), total
    p = torch.where(dead, 0.0, torch.exp(x - torch.logsumexp(torch.where(dead, 0.0, x), 1, keepdim=True)))
    return p, p, None


def _exact_gate(s):
    c, x = s["case"], s["x"].double()
    T, G, k = c["T"], c["G"], c["k"]
    p, prob, _ = _exact_probs(x, c["sigmoid"])
    left = (x if s["bias"] is None else p + s["bias"].double()).masked_fill(torch.isneginf(x), -math.inf)
    idx, w = [], []
    for _ in range(k):  # the largest that is left, the first of equals
        top = left.amax(1, keepdim=True)
        at = (left == top).int().argmax(1, keepdim=True)
        none = torch.isneginf(top)
        idx.append(torch.where(none, -1, at))
        w.append(torch.where(none, 0.0, p.gather(1, at)))
        left.scatter_(1, at, -math.inf)
    idx, w = torch.cat(idx, 1), torch.cat(w, 1)
    if c["norm"]:
        w = w / (w.sum(1, keepdim=True) + TINY)
    out = dict(idx=idx.to(torch.int32), w=w * s["scale"])
    if c["stats"]:
        counts = torch.stack([(idx == g).sum() for g in range(G)])
        psum = prob.sum(0)
        out.update(counts=counts.to(torch.int32), psum=psum,
                   loss=s["coef"] * torch.dot(counts.double(), psum).view(1))
    return out


def _exact_gate_back(s):
    """Through the Jacobian products of w and of the loss, slot by slot."""
    c, x = s["case"], s["x"].double()
    p, prob, total = _exact_probs(x, c["sigmoid"])
    idx, dw = s["idx"].long(), s["dw"].double()
    hot = [(idx[:, j, None] == torch.arange(c["G"], device="cuda")).double() for j in range(c["k"])]
    score = [(h * p).sum(1, keepdim=True) for h in hot]
    ds = torch.zeros_like(x)
    if c["norm"]:
        sum_ = sum(score) + TINY
        mean = sum(dw[:, j, None] * score[j] for j in range(c["k"])) / sum_
        for j, h in enumerate(hot):
            ds += h * (dw[:, j, None] - mean) / sum_
    else:
        for j, h in enumerate(hot):
            ds += h * dw[:, j, None]
    ds *= s["scale"]
    db = s["dloss"].double() * s["coef"] * s["counts"].double()
    if c["sigmoid"]:
        dead = total == 0
        db = db - (prob @ db)[:, None]
        ds = ds + torch.where(dead, 0.0, db / torch.where(dead, 1.0, total))
        return dict(dx=ds * p * torch.special.expit(-x))
    ds = ds + db
    return dict(dx=p * ds - p * (p * ds).sum(1, keepdim=True))


def _exact_w4(s):
    c = s["case"]
    K, group, at = c["K"], c["group"], 0
    y = torch.empty((c["M"], c["N"]), dtype=torch.float64, device="cuda")
    value = torch.tensor([math.copysign(v, 1 - 2 * n) for n in (0, 1) for v in E2M1],
                         dtype=torch.float64, device="cuda")
    for g, n in enumerate(s["ms"].tolist()):
        if n == 0:
            continue
        w = torch.empty((c["N"], K), dtype=torch.float64, device="cuda")
        for half in (0, 1):
            q = (s["W"][g] // 16 if half else s["W"][g] % 16).long()
            w[:, half::2] = value[q] if c["kind"] == "e2m1" else q.double()
        w = w.view(c["N"], -1, group)
        sw = s["sw"][g].double()[..., None]
        if c["kind"] == "e2m1":
            w = w * 2.0 ** (sw - 127)
        else:
            w = (w - (8 if s["zp"] is None else s["zp"][g].double()[..., None])) * sw
        y[at:at + n] = s["A"][at:at + n].double() @ w.view(c["N"], K).t()
        at += n
    return dict(y=y)


def _exact_orth(s):
    outs = []
    for u in s["U"]:
        x = u.double()
        norm = torch.linalg.vector_norm(x)
        x = x / norm if float(norm) > 0 else x
        for _ in range(5):
            if x.shape[0] <= x.shape[1]:
                a = x @ x.t()
                x = NS_A * x + NS_B * (a @ x) + NS_C * (a @ (a @ x))
            else:
                a = x.t() @ x
                x = NS_A * x + NS_B * (x @ a) + NS_C * ((x @ a) @ a)
        outs.append(x)
    return dict(o=torch.stack(outs))


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "gate":
            return _exact_gate(s)
        if case["op"] == "gate_back":
            return _exact_gate_back(s)
        return _exact_w4(s) if case["op"] == "w4" else _exact_orth(s)
