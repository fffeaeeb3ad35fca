"""The operators of a training step around the routed experts, as measured
cases: the router's balance loss, the softmax cross entropy of the rows that
leave the model, and AdamW over the weights.

Every case has a plain form in elementary torch operations (``own`` False),
the calls into the library (``own`` True) and an exact form in 64 bits.

balance  p = softmax of a token's router logits z, c_be the slots of sequence b
         on expert e, n_b its tokens with any slot
         loss_b = E / (k n_b^2) sum_e c_be sum_t p_te
         back: dz_te = dloss_b E / (k n_b^2) p_te (c_be - sum_j p_tj c_bj),
         and the gradients of the token's own slots added to their experts
xent     z = scale h w^T, loss = log sum_v e^z_v - z_target; a target outside
         [0, V) takes no part
         back: ds = dloss scale (e^(z - lse) - [v = target]), dh = ds w, dw = ds^T h
adamw    g' = s g, s = min(1, max_norm / |g|) over all tensors
         m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
         p = p - lr (wd p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
         states in 32 bits, or m and sqrt(v) as E4M3 with a scale per 256 values;
         what is positive of sqrt(v) is held as one code at least
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
FP8 = torch.float8_e4m3fn
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.95, 1e-8, 0.1, 7


def listed():
    balance = dict(op="balance", E=256, k=6, z="f32", seqs=1, dead=0.0, back=True)
    xent = dict(op="xent", x="bf16", scale=1.0, dead=0.0, back=True)
    adamw = dict(op="adamw", p="f32", g="f32", master=False, fp8=False, clip=True)
    return [
        # the loads of a few sessions' tokens, watched while they are served
        dict(balance, name="balance_watch", T=16, back=False),
        # a chunk of 2048 tokens through the layer's router
        dict(balance, name="balance_chunk", T=2048),
        # a packed batch of ragged sequences with padding and dropped slots, bf16 logits
        dict(balance, name="balance_packed", T=16381, z="bf16", seqs=13, dead=0.1),
        # a large batch over fewer experts
        dict(balance, name="balance_large", T=262144, E=64, k=4, seqs=64),
        # scoring 16 drafted tokens
        dict(xent, name="xent_score", N=16, V=65536, d=4096, back=False),
        # a small model's step in fp32, an odd vocabulary
        dict(xent, name="xent_small", N=127, V=1003, d=256, x="f32", dead=0.1),
        # a ragged batch with masked prompts, an odd vocabulary
        dict(xent, name="xent_train", N=2047, V=50001, d=2048, dead=0.1),
        # a whole batch over a large vocabulary
        dict(xent, name="xent_large", N=4096, V=65536, d=4096),
        # the norm weights of 43 layers, three a layer
        dict(adamw, name="adamw_norms", tensors=129, n=4096, spread=False),
        # tensors of all sizes with fp32 states, bf16 weights and gradients
        dict(adamw, name="adamw_mixed", tensors=61, n=5000011, p="bf16", g="bf16", spread=True),
        # adapters of 256 experts, two a matrix, in bf16 with fp32 masters and 8-bit states
        dict(adamw, name="adamw_adapters", tensors=512, n=32768, p="bf16", g="bf16", master=True, fp8=True, spread=False),
        # a head and a shared expert, 8-bit states
        dict(adamw, name="adamw_head", tensors=4, n=65536 * 4096, p="bf16", g="bf16", fp8=True, spread=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "xent", "adamw"])
    types = ["f32", "bf16"]
    if op == "balance":
        E = _log_int(rng, 2, 256)
        T = _log_int(rng, 1, 65536)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), z=rng.choice(types),
                    seqs=rng.choice([1, _log_int(rng, 1, 64)]), dead=rng.choice([0.0, 0.1, 0.5]),
                    back=rng.random() < 0.7)
    if op == "xent":
        x = rng.choice(types)
        N, V, d = _log_int(rng, 1, 4096), _log_int(rng, 2, 65536), 256 * rng.randint(1, 16)
        while N * V * d > (2 ** 40 if x == "bf16" else 2 ** 37):
            N = max(1, N // 2)
        return dict(op=op, N=N, V=V, d=d, x=x, scale=rng.choice([1.0, 0.125]), dead=rng.choice([0.0, 0.1, 0.5]),
                    back=rng.random() < 0.7)
    p = rng.choice(types)
    tensors = _log_int(rng, 1, 512)
    spread = rng.random() < 0.5
    n = _log_int(rng, 1, 2 ** 27 // (1 if spread else tensors))
    return dict(op=op, tensors=tensors, n=n, p=p, g=rng.choice(types), master=p == "bf16" and rng.random() < 0.5,
                fp8=rng.random() < 0.5, clip=rng.random() < 0.5, spread=spread)


# ------------------------------------------------------------------ inputs

class _Rand:
    """Seeded draws on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, scale=1.0, dtype="f32"):
        return (torch.randn(*shape, generator=self.g, device="cuda") * scale).to(TYPES[dtype])

    def uniform(self, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda")


def _sizes(case):
    """Elements of each tensor: `tensors` of n, or sizes falling from most of n by halves (odd ones), n in all."""
    if not case["spread"]:
        return [case["n"]] * case["tensors"]
    left, sizes = case["n"], []
    for i in range(case["tensors"] - 1):
        take = max(1, left * 5 // 8 - i) if left > case["tensors"] else 1
        sizes.append(take)
        left = max(1, left - take)
    return sizes + [left]


def _pad(n):
    return (n + 255) // 256 * 256


def prepare(case, seed):
    r = _Rand(seed)
    s = dict(case)
    if case["op"] == "balance":
        T, k, E, B = (case[n] for n in ("T", "k", "E", "seqs"))
        popular = r.normal(E, scale=0.5)
        z = r.normal(T, E) + popular
        idx = torch.topk(z - torch.log(-torch.log(r.uniform(T, E).clamp(1e-6, 1 - 1e-6))) * 0.1, k, dim=1).indices
        idx = idx.sort(dim=1).values.to(torch.int32)
        if case["dead"]:
            off = (r.uniform(T, k) < case["dead"]) | (r.uniform(T, 1) < case["dead"])
            idx = torch.where(off, torch.full_like(idx, -1), idx)
        s["idx"] = idx.contiguous()
        s["in_z"] = z.to(TYPES[case["z"]])
        cut = (r.uniform(B - 1) * (T + 1)).int().clamp(max=T).sort().values
        ends = torch.full((1,), T, dtype=torch.int32, device="cuda")
        s["seq"] = torch.cat([torch.zeros_like(ends), cut, ends])
        if case["back"]:
            s["in_dloss"] = 0.01 * (0.5 + r.uniform(B))
            s["in_dslots"] = torch.where(s["idx"] >= 0, r.normal(T, k, scale=1e-3), torch.zeros((), device="cuda"))
    elif case["op"] == "xent":
        N, V, d = (case[n] for n in ("N", "V", "d"))
        w = r.normal(V, d, scale=1.5 / (case["scale"] * math.sqrt(d)))
        y = (V * r.uniform(N) ** 3).int().clamp(max=V - 1)  # some words far more often than others
        # rows that know their target a little
        h = r.normal(N, d) + w[y.long()] * (r.uniform(N, 1) * 3 * case["scale"])
        s["target"] = torch.where(r.uniform(N) < case["dead"], torch.full_like(y, -100), y)
        s["in_h"], s["in_w"] = h.to(TYPES[case["x"]]), w.to(TYPES[case["x"]])
        if case["back"]:
            live = (s["target"] >= 0).sum().clamp(min=1)
            s["in_dloss"] = torch.ones(N, device="cuda") / live
    else:
        sizes = _sizes(case)
        places, at = [], 0
        for n in sizes:
            places.append((at, n))
            at += _pad(n)
        s["places"], s["total"] = places, at
        used = torch.ones(at, dtype=torch.bool, device="cuda")
        for (a, n) in places:
            if n % 256:
                used[a + n:a + _pad(n)] = False
        # every tensor a piece of one buffer, on a border of 256 values; zeros between them
        row = torch.exp(r.normal(at // 256, 1))  # gradients of unequal size
        g = (r.normal(at // 256, 256) * row * 1e-3).reshape(-1) * used
        s["in_g"] = g.to(TYPES[case["g"]])
        p = r.normal(at, scale=0.02) * used
        s["p"] = p.to(TYPES[case["p"]])
        s["master"] = p if case["master"] else None
        m = (g + (r.normal(at // 256, 256) * row * 5e-4).reshape(-1)) * used
        v = g * g * 0.7 + (r.uniform(at // 256, 256) * row * row * 1e-6).reshape(-1) * used
        del p, g
        if case["fp8"]:
            s["m"], s["m_scale"] = _to_fp8(m, False)
            s["v"], s["v_scale"] = _to_fp8(torch.sqrt(v), True)
        else:
            s["m"], s["v"] = m, v
    return s


# ------------------------------------------------------------------ plain

def _round(v, kind):
    return v.to(TYPES[kind])


def _sequence_of(s):
    """The sequence of every token (those are contiguous and cover all tokens)."""
    t = torch.arange(s["T"], device="cuda")
    return torch.searchsorted(s["seq"][1:].long(), t, right=True)


def _balance(s):
    E, k = s["E"], s["k"]
    b = _sequence_of(s)
    z = s["in_z"].float()
    e = torch.exp(z - z.amax(1, keepdim=True))
    p = e / e.sum(1, keepdim=True)
    on = s["idx"] >= 0
    live = on.any(1)
    column = torch.where(on, s["idx"].long(), torch.full_like(b, E)[:, None])  # one more column takes what has no expert
    chosen = torch.zeros(s["T"], E + 1, device="cuda", dtype=torch.float64).scatter_(1, column, 1.0)[:, :E]
    edge = s["seq"].long()
    # running sums in 64 bits, of which a sequence's is a difference
    def total(a):
        run = a.t().contiguous().cumsum(1)
        return torch.diff(torch.cat([run.new_zeros(a.shape[1], 1), run], dim=1)[:, edge], dim=1).t()

    counts, mass = total(chosen), total(p.double() * live[:, None])
    tokens = total(live[:, None].double()).squeeze(1)
    n = tokens.clamp(min=1)
    factor = E / (k * n * n)
    out = dict(counts=counts.int(), tokens=tokens.int(), loss=(factor * (counts * mass).sum(1)).float())
    if s["back"]:
        c = counts.float()[b]
        dz = (s["in_dloss"] * factor.float())[b][:, None] * p * (c - (p * c).sum(1, keepdim=True))
        dz = torch.where(live[:, None], dz, torch.zeros((), device="cuda"))
        add = torch.where(on, s["in_dslots"], torch.zeros((), device="cuda"))
        dz = dz.scatter_add(1, torch.where(on, s["idx"].long(), torch.zeros_like(b)[:, None]), add)
        out["dz"] = _round(dz, s["z"])
    return out


def _xent(s):
    h, w = s["in_h"].float(), s["in_w"].float()
    z = (h @ w.t()) * s["scale"]
    top = z.amax(1, keepdim=True)
    lse = (top + torch.log(torch.exp(z - top).sum(1, keepdim=True))).squeeze(1)
    live = (s["target"] >= 0) & (s["target"] < s["V"])
    y = torch.where(live, s["target"], torch.zeros_like(s["target"])).long()[:, None]
    zero = torch.zeros((), device="cuda")
    out = dict(loss=torch.where(live, lse - z.gather(1, y).squeeze(1), zero), lse=lse)
    if s["back"]:
        ds = torch.exp(z - lse[:, None])
        ds.scatter_add_(1, y, torch.full_like(lse, -1.0)[:, None])
        ds *= (torch.where(live, s["in_dloss"], zero) * s["scale"])[:, None]
        out["dh"] = _round(ds @ w, s["x"])
        out["dw"] = _round(ds.t() @ h, s["x"])
    return out


def _to_fp8(x, positive):
    """E4M3 codes and scales of blocks of 256 fp32 values."""
    b = x.reshape(-1, 256)
    scale = b.abs().amax(1) / 448
    y = b / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
    if positive:
        y = torch.where(b > 0, y.clamp(min=2.0 ** -9), y)
    return y.to(FP8).reshape(-1), scale


def _from_fp8(q, scale):
    return (q.float().reshape(-1, 256) * scale[:, None]).reshape(-1)


def _adamw(s):
    g = s["in_g"].float()
    out = {}
    if s["clip"]:
        norm = torch.sqrt((g.double() * g.double()).sum()).float()
        out["norm"] = norm
        g = g * torch.where(norm > 1.0, 1.0 / norm, torch.ones_like(norm))
    if s["fp8"]:
        m = _from_fp8(s["m"], s["m_scale"])
        r = _from_fp8(s["v"], s["v_scale"])
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    p = (s["master"] if s["master"] is not None else s["p"]).float()
    p = p - LR * (DECAY * p + (m / (1 - BETA1 ** STEP)) / (torch.sqrt(v / (1 - BETA2 ** STEP)) + EPS))
    s["p"].copy_(p)
    if s["master"] is not None:
        s["master"].copy_(p)
    if s["fp8"]:
        for name, x, positive in (("m", m, False), ("v", torch.sqrt(v), True)):
            q, scale = _to_fp8(x, positive)
            s[name].copy_(q)
            s[name + "_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return out | _weights(s)


def _weights(s):
    return {n: s[n] for n in ("p", "master", "m", "v", "m_scale", "v_scale") if s.get(n) is not None}


def run(state):
    if own:
        return {"balance": _balance_own, "xent": _xent_own, "adamw": _adamw_own}[state["op"]](state)
    return {"balance": _balance, "xent": _xent, "adamw": _adamw}[state["op"]](state)


# ------------------------------------------------------------------ library

def _hold(s):
    """What a program holds between calls: outputs, workspaces, the optimizer's table.  Made by the first pass."""
    if "held" in s:
        return s["held"]
    from bit_quantized_routed_router_amd import ds4moe as D
    dt = {"f32": D.DT_F32, "bf16": D.DT_BF16}

    def new(*shape, kind="f32"):
        return torch.zeros(*shape, dtype=TYPES[kind], device="cuda")

    def space(n):
        return torch.empty(n, dtype=torch.uint8, device="cuda"), n

    if s["op"] == "balance":
        T, E, B = s["T"], s["E"], s["seqs"]
        out = dict(counts=new(B, E).int(), tokens=new(B).int(), loss=new(B))
        if s["back"]:
            out["dz"] = new(T, E, kind=s["z"])
        held = (D, dt, out, space(D.balance_workspace_bytes(T, E, B)))
    elif s["op"] == "xent":
        N, V, d = s["N"], s["V"], s["d"]
        out = dict(loss=new(N), lse=new(N))
        if s["back"]:
            out.update(dh=new(N, d, kind=s["x"]), dw=new(V, d, kind=s["x"]))
        held = (D, dt, out, space(D.xent_workspace_bytes(dt[s["x"]], N, V, d, s["back"])))
    else:
        def views(name, block=1):
            a = s.get(name)
            return None if a is None else [a[at // block:at // block + -(-n // block)] for at, n in s["places"]]

        opt = D.AdamW(views("p"), views("in_g"), views("m"), views("v"), m_scale=views("m_scale", 256),
                      v_scale=views("v_scale", 256), master=views("master"), lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS,
                      weight_decay=DECAY)
        clip = torch.zeros(2, device="cuda")  # the norm, and what it scales the gradients by
        held = (D, opt, clip, clip[0], clip[1:], space(opt.workspace_bytes()))
    s["held"] = held
    return held


def _balance_own(s):
    D, dt, o, (ws, nb) = _hold(s)
    z, T, E, k, B = dt[s["z"]], s["T"], s["E"], s["k"], s["seqs"]
    D.balance(s["in_z"], z, T, E, s["idx"], k, s["seq"], B, o["counts"], o["tokens"], o["loss"], ws, nb)
    if s["back"]:
        D.balance_grad(s["in_z"], z, T, E, s["idx"], k, s["seq"], B, o["counts"], o["tokens"], s["in_dloss"],
                       s["in_dslots"], o["dz"])
    return o


def _xent_own(s):
    D, dt, o, (ws, nb) = _hold(s)
    x, N, V, d = dt[s["x"]], s["N"], s["V"], s["d"]
    D.xent(s["in_h"], s["in_w"], x, N, V, d, s["scale"], s["target"], o["loss"], o["lse"], ws, nb)
    if s["back"]:
        D.xent_grad(s["in_h"], s["in_w"], x, N, V, d, s["scale"], s["target"], o["lse"], s["in_dloss"], o["dh"],
                    o["dw"], ws, nb)
    return o


def _adamw_own(s):
    D, opt, clip, norm, scale, (ws, nb) = _hold(s)
    out = {}
    if s["clip"]:
        D.adamw_norm(opt, 1.0, clip, ws, nb)
        out["norm"] = norm
    D.adamw_step(opt, STEP, scale if s["clip"] else None)
    return out | _weights(s)


# ------------------------------------------------------------------ work

def work(case):
    if case["op"] == "balance":
        T, E, k, B = (case[n] for n in ("T", "E", "k", "seqs"))
        b = T * E * SIZE[case["z"]] + T * k * 4 + B * (E + 3) * 4
        f = 6 * T * E
        if case["back"]:  # the softmax again or kept: the logits once, their gradients out
            b += T * E * SIZE[case["z"]] + T * k * 4
            f += 6 * T * E
        return {"bytes": b, "flops": f}
    if case["op"] == "xent":
        N, V, d = (case[n] for n in ("N", "V", "d"))
        once = (N + V) * d * SIZE[case["x"]]
        if not case["back"]:
            return {"bytes": once + N * 12, "flops": 2 * N * V * d}
        # the logits are not kept, so the gradient forms them again
        return {"bytes": 2 * once + N * 16, "flops": 8 * N * V * d}
    n = sum(_sizes(case))
    state = 2 * (1 + 4 / 256) if case["fp8"] else 8
    b = SIZE[case["g"]] + 2 * state + SIZE[case["p"]] + (8 if case["master"] else SIZE[case["p"]])
    return {"bytes": n * b, "flops": n * (18 if case["clip"] else 16)}


# ------------------------------------------------------------------ exact

def _exact_balance(s):
    T, E, k, B = (s[n] for n in ("T", "E", "k", "seqs"))
    edge = s["seq"].cpu().tolist()
    z = s["in_z"].double()
    prob = torch.exp(torch.log_softmax(z, dim=1))
    names = (s["idx"].long()[:, :, None] == torch.arange(E, device="cuda")[None, None, :]) if T * k * E <= 2 ** 26 else None
    chosen = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    grad = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    for j in range(k):
        hit = names[:, j] if names is not None else s["idx"][:, j, None].long() == torch.arange(E, device="cuda")
        chosen += hit
        if s["back"]:
            grad += hit * s["in_dslots"][:, j, None].double()
    counts = torch.zeros(B, E, dtype=torch.int32, device="cuda")
    tokens = torch.zeros(B, dtype=torch.int32, device="cuda")
    loss = torch.zeros(B, dtype=torch.float64, device="cuda")
    for b, (lo, hi) in enumerate(zip(edge, edge[1:])):
        part = chosen[lo:hi]
        alive = part.sum(1) > 0
        n = int(alive.sum())
        c = part.sum(0)
        counts[b] = c.int()
        tokens[b] = n
        if n:
            q = prob[lo:hi] * alive[:, None]
            share = E * c / (k * n)  # 1 for every expert where the loads are even
            loss[b] = torch.dot(share, q.mean(0) * ((hi - lo) / n))
            if s["back"]:
                grad[lo:hi] += s["in_dloss"][b].double() / n * q * (share - (q @ share)[:, None])
    out = dict(counts=counts, tokens=tokens, loss=loss)
    if s["back"]:
        out["dz"] = grad
    return out


def _exact_xent(s):
    N, V, d = s["N"], s["V"], s["d"]
    f64 = torch.float64
    w = s["in_w"].to(f64)
    loss = torch.zeros(N, dtype=f64, device="cuda")
    norm = torch.zeros(N, dtype=f64, device="cuda")
    dh = torch.zeros(N, d, dtype=f64, device="cuda")
    dw = torch.zeros(V, d, dtype=f64, device="cuda")
    wt = w.t().contiguous()
    for lo in range(0, N, 512):
        h = s["in_h"][lo:lo + 512].to(f64)
        logp = torch.mm(h, wt) * s["scale"]
        norm[lo:lo + 512] = torch.logsumexp(logp, 1)
        logp -= norm[lo:lo + 512, None]
        y = s["target"][lo:lo + 512].long()
        rows = torch.nonzero((y >= 0) & (y < V)).squeeze(1)
        loss[lo + rows] = -logp[rows, y[rows]]
        if s["back"]:
            up = torch.zeros_like(logp)
            up[rows] = torch.exp(logp[rows])
            up[rows, y[rows]] -= 1
            up *= s["in_dloss"][lo:lo + 512, None].to(f64) * s["scale"]
            dh[lo:lo + 512] = torch.mm(up, w)
            dw += torch.mm(up.t().contiguous(), h)
    out = dict(loss=loss, lse=norm)
    if s["back"]:
        out.update(dh=dh, dw=dw)
    return out


def _exact_adamw(s):
    f64 = torch.float64
    g = s["in_g"].to(f64)
    out = {}
    if s["clip"]:
        out["norm"] = torch.linalg.vector_norm(g)
        g = g / max(1.0, float(out["norm"]))
    if s["fp8"]:
        m = s["m"].to(f64) * s["m_scale"].to(f64).repeat_interleave(256)
        v = (s["v"].to(f64) * s["v_scale"].to(f64).repeat_interleave(256)) ** 2
    else:
        m, v = s["m"].to(f64), s["v"].to(f64)
    m = m + (1 - BETA1) * (g - m)
    v = v + (1 - BETA2) * (g * g - v)
    start = s["p"] if s["master"] is None else s["master"]
    p = start.to(f64) * (1 - LR * DECAY)
    p -= LR / (1 - BETA1 ** STEP) * m / ((v / (1 - BETA2 ** STEP)) ** 0.5 + EPS)
    out["p"] = p
    if s["master"] is not None:
        out["master"] = p
    if not s["fp8"]:
        return out | dict(m=m, v=v)
    # the codes are steps of the values: next to a border 32 and 64 bits take different ones
    top = lambda x: x.abs().reshape(-1, 256).amax(1) / 448  # noqa: E731
    return out | dict(m=None, v=None, m_scale=top(m), v_scale=top(v ** 0.5))


def exact(case, seed):
    s = prepare(case, seed)
    return {"balance": _exact_balance, "xent": _exact_xent, "adamw": _exact_adamw}[case["op"]](s)
