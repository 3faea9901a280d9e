"""The operators around an expert layer's products, as cases that can be timed and checked.

Three families, each in its plain form (elementary torch operations in 32 bits, rounded once at
the end) and as the calls of this library:

  route    tokens put into expert order and back: the sort plan, the gathered rows (as they
           are, or as e4m3 codes with one scale per row and 128 channels), the weighted sum
           back per token, and the gradients of both
  product  the forward product of expert rows with e4m3 weights: one fp32 scale per row and
           128 channels, one per 128 x 128 block of the weight
  adamw    one AdamW step over many tensors, states in fp32 or as e4m3 codes with one scale
           per 128 elements

`own` chooses between the two. The inputs come from the case and a seed alone.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
LR, BETA1, BETA2, EPS, DECAY, STEP = 3e-4, 0.9, 0.95, 1e-8, 0.1, 100
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _ceil(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decoding step of a few sequences: the sort and two short row copies; latency
        dict(name="route_step", op="route", T=8, k=8, G=256, H=7168, dtype="bf16", drop=0.0),
        # a training step's rows of one layer: bandwidth
        dict(name="route_rows", op="route", T=16384, k=8, G=256, H=7168, dtype="bf16", drop=0.0),
        # odd sizes in fp32, some slots dropped (experts held by other ranks)
        dict(name="route_odd", op="route", T=1021, k=3, G=37, H=1000, dtype="f32", drop=0.3),
        # the gathered rows as fp8 operands of the forward product
        dict(name="route_fp8", op="route8", T=8192, k=8, G=32, H=7168, dtype="bf16", drop=0.0),
        # the gradients of the same layer's rows
        dict(name="back_rows", op="back", T=8192, k=8, G=256, H=7168, dtype="bf16", drop=0.0),
        # gradients at an odd width (rows that are no whole number of 16-byte units)
        dict(name="back_odd", op="back", T=777, k=2, G=8, H=1235, dtype="bf16", drop=0.1),
        # a decoding step through 32 experts: every weight is read for a few rows
        dict(name="product_step", op="product", M=64, G=32, N=4096, K=7168, mode="fp8",
             out="bf16", pad=0),
        # one plain linear layer
        dict(name="product_dense", op="product", M=4096, G=1, N=7168, K=2048, mode="fp8",
             out="bf16", pad=0),
        # one rank's share of a training step's tokens
        dict(name="product_share", op="product", M=32768, G=8, N=4096, K=7168, mode="fp8",
             out="bf16", pad=0),
        # odd sizes with exact products and fp32 results, rows of a wider matrix
        dict(name="product_odd", op="product", M=5003, G=37, N=1000, K=1040, mode="exact",
             out="f32", pad=48),
        # a model's small tensors, one after the other without gaps: latency
        dict(name="adamw_small", op="adamw", count=160, lo=1, hi=40000, shape_seed=1, bits=32,
             grad="f32", gap=False),
        # one rank's expert weights, states in 8 bits
        dict(name="adamw_experts", op="adamw", count=8, lo=7168 * 4096, hi=7168 * 4096,
             shape_seed=1, bits=8, grad="bf16", gap=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route8", "back", "product", "product", "adamw", "adamw"])
    if op in ("route", "route8", "back"):
        G = _log_int(rng, 2, 512)
        k = min(G, rng.randint(1, 8))
        H = _log_int(rng, 64, 8192)
        if op == "route8":
            H = max(64, H // 16 * 16)
        T = _log_int(rng, 1, max(2, min(65536, 8192 * 8 * 7168 // (k * H))))
        return dict(op=op, T=T, k=k, G=G, H=H, dtype="bf16" if op == "route8" else
                    rng.choice(["bf16", "bf16", "f32"]), drop=rng.choice([0.0, 0.0, 0.25]))
    if op == "product":
        mode = rng.choice(["fp8", "fp8", "exact"])
        G = _log_int(rng, 1, 64)
        K = max(128, _log_int(rng, 128, 8192) // 16 * 16)
        N = _log_int(rng, 64, max(65, min(8192, 500_000_000 // (G * K))))
        M = _log_int(rng, 1, max(2, min(32768, 600_000_000_000 // (2 * N * K) * 2)))
        return dict(op=op, M=M, G=G, N=N, K=K, mode=mode,
                    out="bf16" if mode == "fp8" else rng.choice(["bf16", "f32"]),
                    pad=rng.choice([0, 0, 16 * rng.randint(1, 20)]))
    bits = rng.choice([8, 32])
    count = _log_int(rng, 1, 300)
    hi = _log_int(rng, 64, max(65, min(30_000_000, 120_000_000 // count)))
    return dict(op=op, count=count, lo=rng.choice([1, max(1, hi // 100)]), hi=hi,
                shape_seed=rng.randint(0, 1 << 30), bits=bits, grad=rng.choice(["f32", "bf16"]),
                gap=True if bits == 8 else rng.choice([True, False]))


def _sizes(case):
    rng = random.Random(case["shape_seed"])
    return [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["count"])]


def _starts(case):
    """Start of every tensor in the flat storage, and its length; tensors start at multiples
    of 128 elements, or (no gap) right behind each other."""
    starts, at = [], 0
    for n in _sizes(case):
        starts.append(at)
        at += n if not case["gap"] else _ceil(n, 128) * 128
    return starts, max(at, 1)


def work(case):
    if case["op"] in ("route", "route8", "back"):
        T, k, H = case["T"], case["k"], case["H"]
        R, e = T * k, TYPES[case["dtype"]].itemsize
        if case["op"] == "route":  # idx, plan; X in, Xp out; Y, w in, out out
            return dict(bytes=R * 12 + case["G"] * 4 + (2 * T + 2 * R) * H * e + R * 4,
                        flops=2 * R * H)
        if case["op"] == "route8":
            return dict(bytes=R * 12 + case["G"] * 4 + T * H * e + R * H +
                        R * _ceil(H, 128) * 4, flops=2 * T * H)
        # pos, w, dOut, Y, dXp in; dY, dw, dX out
        return dict(bytes=R * 12 + (2 * T + 3 * R) * H * e, flops=4 * R * H)
    if case["op"] == "product":
        M, G, N, K = (case[x] for x in "MGNK")
        live = G * (1 - (1 - 1 / G) ** M)  # experts that get a row, of even chances
        kb, nb = _ceil(K, 128), _ceil(N, 128)
        return dict(bytes=int(M * K + live * N * K + M * kb * 4 + live * nb * kb * 4 +
                            M * N * TYPES[case["out"]].itemsize), flops=2 * M * N * K)
    n = sum(_sizes(case))
    state = 4 * 4 if case["bits"] == 32 else 4 + 16 / 128
    return dict(bytes=int(n * (8 + TYPES[case["grad"]].itemsize + state + 2)), flops=20 * n)


# --------------------------------------------------------------------------------- inputs

def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _routing(case, gen):
    """k different experts per token from scores with a bias per expert, so that some experts
    get far more tokens than others; a dropped slot holds -1."""
    T, k, G = case["T"], case["k"], case["G"]
    score = _randn(gen, T, G) + 0.7 * _randn(gen, G)
    idx = score.topk(k, dim=1).indices.to(torch.int32)
    if case["drop"]:
        idx[torch.rand((T, k), generator=gen, device="cuda") < case["drop"]] = -1
    w = torch.softmax(_randn(gen, T, k), dim=1)
    return idx.contiguous(), w


def _rows_1x128(x):
    """e4m3 codes and scales [ceil(K / 128), rows] of fp32 rows."""
    M, K = x.shape
    xb = torch.nn.functional.pad(x, (0, -K % 128)).view(M, -1, 128)
    amax = xb.abs().amax(dim=2)
    s = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    q = (xb / s[..., None]).clamp(-448, 448).view(M, -1)[:, :K].to(E4M3)
    return q.contiguous(), s.t().contiguous()


def _weight(case, gen):
    """e4m3 codes [G, N, K] and 128 x 128 block scales of normal weights."""
    G, N, K = case["G"], case["N"], case["K"]
    nb, kb = _ceil(N, 128), _ceil(K, 128)
    q = torch.empty((G, N, K), dtype=E4M3, device="cuda")
    s = torch.empty((G, nb, kb), device="cuda")
    for g in range(G):
        w = torch.nn.functional.pad(_randn(gen, N, K) * K ** -0.5, (0, -K % 128, 0, -N % 128))
        w = w.view(nb, 128, kb, 128)
        s[g] = w.abs().amax(dim=(1, 3)) / 448
        q[g] = (w / s[g][:, None, :, None]).clamp(-448, 448).view(nb * 128, -1)[:N, :K].to(E4M3)
    return q, s


def _counts(case, gen):
    """Rows per expert: a skewed draw that adds up to M (an expert may have none)."""
    M, G = case["M"], case["G"]
    p = torch.softmax(0.35 * _randn(gen, G), dim=0)
    to = torch.multinomial(p, M, replacement=True, generator=gen)
    return (to[:, None] == torch.arange(G, device="cuda")).sum(0).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(int(seed))
    s = dict(case=case)
    new = lambda shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")
    if case["op"] in ("route", "route8", "back"):
        T, k, G, H = case["T"], case["k"], case["G"], case["H"]
        R, dt = T * k, TYPES[case["dtype"]]
        s["idx"], s["w"] = _routing(case, gen)
        x = _randn(gen, T, H)
        if case["op"] == "route8":  # activations with a few far channels
            x *= 1 + 30 * (torch.rand((H,), generator=gen, device="cuda") < 0.01)
        s["X"] = x.to(dt)
        s["ks"], s["pos"], s["src"] = new(G, torch.int32), new((T, k), torch.int32), new(R, torch.int32)
        if case["op"] == "route8":
            s["Q"], s["sa"] = new((R, H), torch.uint8), new((_ceil(H, 128), R))
        else:
            s["Y"] = _randn(gen, R, H).to(dt)
            s["Xp"], s["out"] = new((R, H), dt), new((T, H), dt)
        if case["op"] == "back":
            s["dXp"] = (_randn(gen, R, H) * 1e-3).to(dt)
            s["dw"] = new((T, k))
            s["ks"], s["pos"], s["src"] = _plain_route(s["idx"], G)  # the forward pass's plan
        elif own:
            import fp8_grouped_gemm_tn_amd as kg
            s["ws"] = kg.new_route_workspace(T, k, G, "cuda")
    elif case["op"] == "product":
        M, N, K, pad = case["M"], case["N"], case["K"], case["pad"]
        a, s["sa"] = _rows_1x128(_randn(gen, M, K))
        wide = torch.zeros((M, K + pad), dtype=torch.uint8, device="cuda")
        wide[:, :K] = a.view(torch.uint8)
        s["A"] = wide.view(E4M3)[:, :K]
        s["W"], s["sw"] = _weight(case, gen)
        s["ms"] = _counts(case, gen)
        s["most"] = int(s["ms"].max())
        s["D"] = new((M, N), TYPES[case["out"]])
    else:
        starts, total = _starts(case)
        sizes = _sizes(case)
        live = torch.zeros(total, device="cuda")
        at = torch.tensor(starts, device="cuda")
        live[at] += 1
        end = at + torch.tensor(sizes, device="cuda")
        live.index_put_((end[end < total],), torch.tensor(-1.0, device="cuda"), accumulate=True)
        live = live.cumsum(0) > 0.5 if case["gap"] else torch.ones_like(live, dtype=torch.bool)
        s["p"] = _randn(gen, total) * 0.02 * live
        s["g"] = (_randn(gen, total) * 1e-3 * live).to(TYPES[case["grad"]])
        m = _randn(gen, total) * 3e-4 * live
        r = (_randn(gen, total).abs() * 1e-3 + 1e-5) * live
        s["copy"] = s["p"].to(torch.bfloat16)
        if case["bits"] == 8:
            s["m"], s["ms"] = _pack(m)
            s["v"], s["vs"] = _pack(r, up=True)
        else:
            s["m"], s["v"] = m, r * r
        s["clip"] = torch.rand(1, generator=gen, device="cuda") * 0.5 + 0.5
        if own:
            import fp8_grouped_gemm_tn_amd as kg
            cut = lambda t: [t[a:a + n] for a, n in zip(starts, sizes)]
            blk = lambda t: [t[a // 128:a // 128 + _ceil(n, 128)] for a, n in zip(starts, sizes)]
            packed = case["bits"] == 8
            s["table"] = kg.AdamWTable(cut(s["p"]), cut(s["g"]), cut(s["m"]), cut(s["v"]),
                                       blk(s["ms"]) if packed else None,
                                       blk(s["vs"]) if packed else None, cut(s["copy"]))
    return s


# ----------------------------------------------------------------------------- plain forms

def _plain_route(idx, G):
    key = idx.reshape(-1).long()
    kept = (key >= 0) & (key < G)
    key = torch.where(kept, key, G)
    order = torch.argsort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=order.device)
    ks = (key[:, None] == torch.arange(G, device=key.device)).sum(0)
    pos = torch.where(kept, row, ~row).view(idx.shape)
    src = torch.where(kept[order], order, ~order)
    return ks.to(torch.int32), pos.to(torch.int32), src.to(torch.int32)


def _gather(X, src, k):
    src = src.long()
    x = X[torch.where(src < 0, ~src, src) // k].float()
    return torch.where((src < 0)[:, None], 0.0, x)


def _weighted_sum(Y, pos, w):
    pos = pos.long()
    y = torch.where((pos < 0)[..., None], 0.0, Y[pos.clamp(min=0)].float())
    if w is not None:
        y = y * torch.where(pos < 0, 0.0, w)[..., None]
    return y.sum(1).to(Y.dtype)


def _plain_product(s):
    c, ms = s["case"], s["ms"].long()
    M, G, N, K = c["M"], c["G"], c["N"], c["K"]
    nb, kb = _ceil(N, 128), _ceil(K, 128)
    a = s["A"].float() * s["sa"].t().repeat_interleave(128, 1)[:, :K]
    sw = s["sw"].repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    w = s["W"].float() * sw
    row = torch.arange(M, device="cuda")
    end = ms.cumsum(0)
    g = (row[:, None] >= end).sum(1)  # the expert of each row
    at = row - (end - ms)[g]
    padded = torch.zeros((G, s["most"], K), device="cuda")
    padded[g, at] = a
    y = torch.bmm(padded, w.transpose(1, 2).contiguous())
    return y[g, at].to(TYPES[c["out"]])


def _pack(x, up=False):
    """e4m3 codes and one scale per 128 elements; `up`: what is above zero stays above zero."""
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % 128)).view(-1, 128)
    amax = b.abs().amax(dim=1)
    kept = ~(amax < 2.0 ** -118)
    inv = torch.where(kept, 448 / amax, 0.0)
    y = b * inv[:, None]
    q = y.to(E4M3)
    if up:
        q = torch.where((y > 0) & (q.float() == 0), torch.tensor(2.0 ** -9, device="cuda"), q.float()).to(E4M3)
    return q.view(-1)[:n].contiguous(), torch.where(kept, amax / 448, 0.0)


def _unpack(q, s):
    n = q.numel()
    return (torch.nn.functional.pad(q.float(), (0, -n % 128)).view(-1, 128) * s[:, None]).view(-1)[:n]


def _plain_adamw(s):
    packed = s["case"]["bits"] == 8
    g = s["g"].float() * s["clip"]
    m = _unpack(s["m"], s["ms"]) if packed else s["m"]
    v = _unpack(s["v"], s["vs"]).square() if packed else s["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    root = v.sqrt()
    step = m / (root * (1 - BETA2 ** STEP) ** -0.5 + EPS)
    s["p"].copy_(s["p"] * (1 - LR * DECAY) - step * (LR / (1 - BETA1 ** STEP)))
    s["copy"].copy_(s["p"])
    if packed:
        for (q, scale), name in ((_pack(m), "m"), (_pack(root, up=True), "v")):
            s[name].copy_(q)
            s[name + "s"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "route":
        ks, pos, src = _plain_route(s["idx"], s["case"]["G"])
        rows = _gather(s["X"], src, s["case"]["k"]).to(s["X"].dtype)
        return dict(ks=ks, pos=pos, src=src, rows=rows, out=_weighted_sum(s["Y"], pos, s["w"]))
    if op == "route8":
        ks, pos, src = _plain_route(s["idx"], s["case"]["G"])
        q, sa = _rows_1x128(_gather(s["X"], src, s["case"]["k"]))
        return dict(ks=ks, pos=pos, src=src, q=q, sa=sa)
    if op == "back":
        pos, src, k = s["pos"].long(), s["src"].long(), s["case"]["k"]
        w = torch.where(src < 0, 0.0, s["w"].view(-1)[torch.where(src < 0, ~src, src)])
        d_rows = (_gather(s["X"], src, k) * w[:, None]).to(s["X"].dtype)
        y = torch.where((pos < 0)[..., None], 0.0, s["Y"][pos.clamp(min=0)].float())
        dw = (y * s["X"].float()[:, None]).sum(2)
        return dict(d_rows=d_rows, dw=dw, dx=_weighted_sum(s["dXp"], s["pos"], None))
    if op == "product":
        return dict(y=_plain_product(s))
    _plain_adamw(s)
    return _adamw_out(s)


def _adamw_out(s):
    out = dict(p=s["p"], copy=s["copy"], m=s["m"], v=s["v"])
    return dict(out, ms=s["ms"], vs=s["vs"]) if s["case"]["bits"] == 8 else out


# ------------------------------------------------------------------------ the library's calls

def _run_own(s, op):
    import fp8_grouped_gemm_tn_amd as kg
    if op in ("route", "route8"):
        kg.kg_route(s["idx"], s["ks"], s["pos"], s["src"], s["ws"])
        if op == "route8":
            kg.kg_dispatch_fp8(s["X"], s["pos"], s["Q"], s["sa"])
            return dict(ks=s["ks"], pos=s["pos"], src=s["src"], q=s["Q"].view(E4M3), sa=s["sa"])
        kg.kg_dispatch(s["X"], s["pos"], s["Xp"])
        kg.kg_combine(s["Y"], s["pos"], s["w"], s["out"])
        return dict(ks=s["ks"], pos=s["pos"], src=s["src"], rows=s["Xp"], out=s["out"])
    if op == "back":
        kg.kg_combine_bwd(s["X"], s["Y"], s["pos"], s["w"], s["Xp"], s["dw"])
        kg.kg_combine(s["dXp"], s["pos"], None, s["out"])
        return dict(d_rows=s["Xp"], dw=s["dw"], dx=s["out"])
    if op == "product":
        flags = kg.KG_FLAG_FP8_MFMA if s["case"]["mode"] == "fp8" else 0
        kg.kg_fprop(s["A"], s["sa"], s["W"], s["sw"], s["D"], s["ms"], flags)
        return dict(y=s["D"])
    kg.kg_adamw(s["table"], LR, BETA1, BETA2, EPS, DECAY, STEP, gscale=s["clip"])
    return _adamw_out(s)


# ---------------------------------------------------------------------- the definitions in 64 bits

def _exact_route(idx, G):
    """Ranks by counting: an expert's rows start behind all smaller experts', its slots in order."""
    key = idx.reshape(-1).long()
    key = torch.where((key < 0) | (key >= G), G, key)
    hot = torch.zeros((key.numel(), G + 1), dtype=torch.int32, device="cuda")
    hot.scatter_(1, key[:, None], 1)
    n = hot.sum(0)
    rank = (n.cumsum(0) - n)[key] + hot.cumsum(0).gather(1, key[:, None])[:, 0] - 1
    return key, n[:G], rank


def _e4m3_64(y, up=False):
    """The nearest e4m3 value of 64-bit numbers within +-448, ties to the even one."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    q = torch.round(y / step) * step
    return torch.where((y > 0) & (q == 0), 2.0 ** -9, q) if up else q


def _blocks_64(x, up=False):
    n = x.shape[-1]
    b = torch.nn.functional.pad(x, (0, -n % 128)).unflatten(-1, (-1, 128))
    s = b.abs().amax(dim=-1) / 448
    y = torch.where(s[..., None] > 0, b / s[..., None], 0.0)
    return _e4m3_64(y, up).flatten(-2)[..., :n], s


def exact(case, seed):
    if case["op"] == "product" and 2.0 * case["M"] * case["N"] * case["K"] > 3e14:
        return None
    s = prepare(case, seed)
    if case["op"] in ("route", "route8", "back"):
        T, k, G = case["T"], case["k"], case["G"]
        key, n, rank = _exact_route(s["idx"], G)
        lost = key == G
        token = torch.arange(T * k, device="cuda") // k
        pos, src = torch.where(lost, -1 - rank, rank), torch.empty_like(rank)
        src[rank] = torch.where(lost, -1 - torch.arange(T * k, device="cuda"), torch.arange(T * k, device="cuda"))
        plan = dict(ks=n.to(torch.int32), pos=pos.view(T, k).to(torch.int32), src=src.to(torch.int32))
        if case["op"] == "route8":
            x = s["X"].double()
            q, sc = _blocks_64(x)
            sc = torch.where(sc > 0, sc, 1.0)
            Q = torch.empty((T * k, x.shape[1]), dtype=torch.float32, device="cuda")
            Q[rank] = torch.where(lost[:, None], 0.0, q[token]).float()  # e4m3 values: exact
            sa = torch.empty((T * k, sc.shape[1]), dtype=torch.float64, device="cuda")
            sa[rank] = torch.where(lost[:, None], 1.0, sc[token])
            return dict(plan, q=Q, sa=sa.t().contiguous())
        add = lambda rows, w: sum(torch.where(lost.view(T, k)[:, j, None], 0.0, rows[rank.view(T, k)[:, j]].double()) *
                                  (1.0 if w is None else w[:, j, None].double()) for j in range(k))
        if case["op"] == "route":
            rows = torch.empty_like(s["Y"])
            rows[rank] = torch.where(lost[:, None], torch.zeros((), dtype=s["X"].dtype, device="cuda"), s["X"][token])
            return dict(plan, rows=rows, out=add(s["Y"], s["w"]))
        d_rows = torch.empty(s["Y"].shape, dtype=torch.float64, device="cuda")
        x = s["X"].double()
        for j in range(k):
            at = rank.view(T, k)[:, j]
            d_rows[at] = torch.where(lost.view(T, k)[:, j, None], 0.0, x * s["w"][:, j, None].double())
        dw = torch.stack([torch.where(lost.view(T, k)[:, j], 0.0, (x * s["Y"][rank.view(T, k)[:, j]].double()).sum(1))
                          for j in range(k)], 1)
        return dict(d_rows=d_rows, dw=dw, dx=add(s["dXp"], None))
    if case["op"] == "product":
        K, at, y = case["K"], 0, torch.empty((case["M"], case["N"]), dtype=torch.float64, device="cuda")
        for g, n in enumerate(s["ms"].tolist()):
            part = torch.zeros((n, case["N"]), dtype=torch.float64, device="cuda")
            for kb in range(_ceil(K, 128)):
                c = slice(kb * 128, min(K, kb * 128 + 128))
                col = s["sw"][g, :, kb].double().repeat_interleave(128)[:case["N"]]
                part += (s["A"][at:at + n, c].double() @ s["W"][g, :, c].double().t()) * \
                    s["sa"][kb, at:at + n, None].double() * col
            y[at:at + n] = part
            at += n
        return dict(y=y)
    wide = lambda q, sc: (torch.nn.functional.pad(q.double(), (0, -q.numel() % 128)).view(-1, 128) *
                          sc.double()[:, None]).view(-1)[:q.numel()]
    packed = case["bits"] == 8
    g = s["g"].double() * s["clip"].double()
    m = wide(s["m"], s["ms"]) if packed else s["m"].double()
    v = wide(s["v"], s["vs"]) ** 2 if packed else s["v"].double()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    p = s["p"].double() * (1 - LR * DECAY) - LR * (m / (1 - BETA1 ** STEP)) / (torch.sqrt(v / (1 - BETA2 ** STEP)) + EPS)
    if not packed:
        return dict(p=p, copy=p, m=m, v=v)
    (qm, sm), (qv, sv) = _blocks_64(m), _blocks_64(torch.sqrt(v), up=True)
    return dict(p=p, copy=p, m=qm.float(), v=qv.float(), ms=sm, vs=sv)
