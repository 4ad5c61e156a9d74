"""The operators around the expert products, measured: rows sorted by expert and brought
back with their weights (and the gradients of both), activations kept in 8 bits for a
backward pass, the SwiGLU that uses such checkpoints, and low-rank adapters of many
requests beside a layer.

``listed()`` names the cases, ``draw()`` makes more of the same ranges, ``run()`` makes
one pass: in elementary torch operations, or with ``own`` through the library.
``exact()`` computes the same from the definitions in 64 bits.
"""
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
GROUP = 32  # values that share one scale in an 8-bit checkpoint


# ------------------------------------------------------------------ cases
def listed():
    return [
        # decode step of the 256-expert NVFP4 layer: 16 tokens, top-6; latency counts
        dict(name="dispatch decode", op="dispatch", T=16, k=6, E=256, H=2048, dtype="bf16", pad=0),
        # prefill of the same layer at its benchmark batch
        dict(name="dispatch prefill", op="dispatch", T=8192, k=6, E=256, H=2048, dtype="bf16", pad=0),
        # a padded training batch of the hot/cold layer: gradient of its dispatch
        dict(name="dispatch gradient", op="dispatch_grad", T=4096, k=8, E=256, H=2048, dtype="bf16", pad=301),
        # decode step of the 12288-wide layer: fp32 expert outputs brought back
        dict(name="collect decode", op="collect", T=64, k=2, E=128, H=12288, dtype="f32", pad=0),
        # the Mixtral-like layer's prefill batch: gradient of rows and weights
        dict(name="collect gradient", op="collect_grad", T=2048, k=2, E=8, H=4096, dtype="bf16", pad=77),
        # layer inputs of one training batch kept in 8 bits and restored in the backward pass
        dict(name="checkpoint batch", op="checkpoint", R=8192, F=4096, dtype="bf16"),
        # a short ragged one in fp16: rows that are no multiple of the group
        dict(name="checkpoint ragged", op="checkpoint", R=515, F=1001, dtype="f16"),
        # hidden layer of the Mixtral-like experts: forward with checkpoints, then the backward pass from them
        dict(name="swiglu step", op="swiglu", R=4096, F=14336, dtype="bf16"),
        # fp32 training of a small layer, ragged width
        dict(name="swiglu ragged", op="swiglu", R=333, F=778, dtype="f32"),
        # one request decoding beside a 4096-wide layer
        dict(name="adapters single token", op="adapters", T=1, K=4096, N=4096, r=16, n=32, requests=1, dtype="bf16"),
        # a decode batch: every row its own request
        dict(name="adapters decode", op="adapters", T=64, K=4096, N=4096, r=16, n=48, requests=64, dtype="bf16"),
        # prompts of many requests at once beside the 2048-wide layer, wide rank
        dict(name="adapters prefill", op="adapters", T=8192, K=2048, N=2048, r=64, n=24, requests=29, dtype="f16"),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, even over the logarithm."""
    import math
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "collect", "collect_grad", "checkpoint", "swiglu", "adapters"])
    if op == "adapters":
        c = dict(op=op, T=_log(rng, 1, 8192), K=8 * _log(rng, 16, 640), N=8 * _log(rng, 16, 640), r=8 * _log(rng, 1, 16),
                 n=_log(rng, 1, 64), dtype=rng.choice(["bf16", "f16"]))
        c["requests"] = _log(rng, 1, min(c["T"], 128))
        return c
    if op in ("checkpoint", "swiglu"):
        R, F = _log(rng, 1, 8192), _log(rng, 8, 14336)
        return dict(op=op, R=R, F=min(F, max(8, 32_000_000 // R)), dtype=rng.choice(["bf16", "f16", "f32"]))
    k = rng.randint(1, 8)
    T, H = _log(rng, 1, 8192), rng.choice([1, 8, 8]) * _log(rng, 8, 1536)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    H = min(H, max(8, (1 << 28) // SIZE[dtype] // (T * k)))
    return dict(op=op, T=T, k=k, E=_log(rng, k, 256), H=H, dtype=dtype,
                pad=rng.choice([0, T // 10, rng.randint(0, T - 1)]))


# ------------------------------------------------------------------ inputs
def _order(idx, E):
    """Stable order of the entries by expert: perm (dropped entries last), inv (-1: dropped), offsets."""
    key = torch.where((idx >= 0) & (idx < E), idx, E).reshape(-1)
    perm = torch.argsort(key, stable=True)
    row = torch.empty_like(perm)
    row[perm] = torch.arange(perm.numel(), device=perm.device)
    inv = torch.where(key < E, row, -1)
    offsets = (key[:, None] < torch.arange(E + 1, device=key.device)[None]).sum(0)
    return perm.int(), inv.int(), offsets.int()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[c["dtype"]]

    def normal(*shape, sigma=1.0, to=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * sigma).to(to)

    if c["op"] in ("checkpoint", "swiglu"):
        R, F = c["R"], c["F"]
        s = dict(case=c, g=normal(R, F))
        # every row has a magnitude of its own, as tokens have
        s["g"].mul_(torch.exp(normal(R, 1, sigma=0.7, to=torch.float32)).to(dt))
        if c["op"] == "swiglu":
            s["u"], s["dh"] = normal(R, F), normal(R, F, sigma=0.05)
        return s
    if c["op"] == "adapters":
        T, K, N, r, n = c["T"], c["K"], c["N"], c["r"], c["n"]
        # consecutive rows of one request share its adapter; every eighth request or so has none
        cuts = torch.randint(0, c["requests"], (T,), generator=gen, device="cuda").sort().values
        of = torch.randint(0, n, (c["requests"],), generator=gen, device="cuda")
        if c["requests"] > 1:
            of = torch.where(torch.rand(c["requests"], generator=gen, device="cuda") < 0.125, -1, of)
        ids = of[cuts].int()
        perm, inv, offsets = _order(ids[:, None].long(), n)
        return dict(case=c, x=normal(T, K), y=normal(T, N), A=normal(n, r, K, sigma=K ** -0.5), B=normal(n, N, r, sigma=0.3 * r ** -0.5),
                    scale=torch.rand(n, generator=gen, device="cuda") + 0.5, ids=ids, perm=perm, inv=inv, offsets=offsets,
                    out=torch.empty(T, N, dtype=dt, device="cuda"))
    T, k, E, H = c["T"], c["k"], c["E"], c["H"]
    # some experts are hotter than others; the tokens behind the batch's end have no expert
    logits = normal(T, E, to=torch.float32) + normal(1, E, to=torch.float32)
    top, idx = logits.topk(k, dim=1)
    w = torch.softmax(top, dim=1)
    idx[T - c["pad"]:] = -1
    s = dict(case=c, idx=idx.int(), w=w)
    R = T * k
    if c["op"] == "dispatch":
        s["x"] = normal(T, H)
        s["xs"] = torch.zeros(R, H, dtype=dt, device="cuda")
        s["perm"], s["inv"] = (torch.empty(R, dtype=torch.int32, device="cuda") for _ in range(2))
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        return s
    s["perm"], s["inv"], s["offsets"] = _order(idx, E)
    rows = normal(R, H)
    rows[(T - c["pad"]) * k:] = float("nan")  # rows behind the last expert's: never written, never read
    if c["op"] == "dispatch_grad":
        s["dxs"], s["dx"] = rows, torch.empty(T, H, dtype=dt, device="cuda")
    else:
        s["o"] = rows
        if c["op"] == "collect":
            s["y"] = torch.empty(T, H, dtype=dt, device="cuda")
        else:
            s["dy"] = normal(T, H, sigma=0.05)
            s["do"] = torch.zeros(R, H, dtype=dt, device="cuda")
            s["dw"] = torch.empty(T, k, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _keep8(x):
    """The values that an 8-bit checkpoint of x holds, in 32 bits."""
    R, F = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -F % GROUP)).reshape(R, -1, GROUP)
    top = {torch.float16: 9}.get(x.dtype, 121)
    m, p = torch.frexp(v.abs().amax(2, keepdim=True))
    e = (p - torch.where(m <= 127 / 128, 7, 6)).clamp(-126, top)
    two = lambda n: ((n.int() + 127) << 23).view(torch.float32)  # 2^n, exactly  # noqa: E731
    q = torch.round(v * two(-e)).clamp(-127, 127)
    return (q * two(e)).reshape(R, -1)[:, :F]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "checkpoint":
        return {"x": _keep8(s["g"]).to(s["g"].dtype)}
    if op == "swiglu":
        dt = s["g"].dtype
        g, u = s["g"].float(), s["u"].float()
        h = (g / (1 + torch.exp(-g)) * u).to(dt)
        g, u, dh = _keep8(s["g"]), _keep8(s["u"]), s["dh"].float()
        sig = 1 / (1 + torch.exp(-g))
        act = g * sig
        return {"h": h, "dg": (dh * u * sig * (1 + g * (1 - sig))).to(dt), "du": (dh * act).to(dt), "h_again": (act * u).to(dt)}
    if op == "adapters":
        n, r, K = s["A"].shape
        ids = s["ids"].long()
        mine = ids[:, None] == torch.arange(n, device=ids.device)[None]
        p = (s["x"].float() @ s["A"].float().reshape(n * r, K).T).reshape(-1, n, r)
        p = torch.where(mine[:, :, None], p * s["scale"][None, :, None], 0.0).reshape(-1, n * r)
        return {"out": (s["y"].float() + p @ s["B"].float().transpose(1, 2).reshape(n * r, -1)).to(s["y"].dtype)}
    T, k, E = c["T"], c["k"], c["E"]
    if op == "dispatch":
        perm, inv, offsets = _order(s["idx"].long(), E)
        real = torch.arange(T * k, device=perm.device) < offsets[E]
        return {"xs": torch.where(real[:, None], s["x"][perm.long() // k], s["xs"]), "perm": perm, "inv": inv, "offsets": offsets}
    inv = s["inv"].long().reshape(T, k)
    real = inv >= 0
    if op == "dispatch_grad":
        rows = torch.where(real[:, :, None], s["dxs"].float()[inv.clamp(min=0)], 0.0)
        return {"dx": rows.sum(1).to(s["dxs"].dtype)}
    rows = torch.where(real[:, :, None], s["o"].float()[inv.clamp(min=0)], 0.0)
    w = torch.where(real, s["w"], 0.0)
    if op == "collect":
        return {"y": (w[:, :, None] * rows).sum(1).to(s["o"].dtype)}
    dy = s["dy"].float()
    perm = s["perm"].long()
    back = (w.reshape(-1)[perm][:, None] * dy[perm // k]).to(s["o"].dtype)
    kept = torch.arange(T * k, device=perm.device) < s["offsets"][E]
    return {"do": torch.where(kept[:, None], back, s["do"]), "dw": (dy[:, None] * rows).sum(2)}


# ------------------------------------------------------------------ the library's calls
def _library(s):
    import mixed_precision_quantized_fp32_b200 as moe
    c = s["case"]
    op = c["op"]
    if op == "checkpoint":
        return {"x": moe.moe_act_load(moe.moe_act_save(s["g"]))}
    if op == "swiglu":
        h, kept = moe.moe_swiglu_save(s["g"], s["u"])
        dg, du, again = moe.moe_swiglu_backward(s["dh"], kept, rebuild_h=True)
        return {"h": h, "dg": dg, "du": du, "h_again": again}
    if op == "adapters":
        routes = moe.Routes(c["T"], 1, c["n"], s["perm"], s["inv"], s["offsets"])
        return {"out": moe.moe_adapters(s["x"], s["y"], s["A"], s["B"], s["scale"], routes, out=s["out"])}
    routes = moe.Routes(c["T"], c["k"], c["E"], s["perm"], s["inv"], s["offsets"])
    if op == "dispatch":
        xs, _ = moe.moe_dispatch(s["x"], s["idx"], c["E"], xs=s["xs"], routes=routes)
        return {"xs": xs, "perm": s["perm"], "inv": s["inv"], "offsets": s["offsets"]}
    if op == "dispatch_grad":
        return {"dx": moe.moe_dispatch_backward(s["dxs"], routes, dx=s["dx"])}
    if op == "collect":
        return {"y": moe.moe_collect(s["o"], s["w"], routes, y=s["y"])}
    do, dw = moe.moe_collect_backward(s["dy"], s["o"], s["w"], routes, do=s["do"], dw=s["dw"])
    return {"do": do, "dw": dw}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    es = SIZE[c["dtype"]]
    op = c["op"]
    if op == "checkpoint":  # values in and out; codes and exponents written once and read once
        n = c["R"] * c["F"]
        return {"bytes": n * (2 * es + 2) + 2 * c["R"] * -(-c["F"] // GROUP), "flops": 3 * n}
    if op == "swiglu":  # g, u, dh in; h, dg, du, h again out; two checkpoints written and read
        n = c["R"] * c["F"]
        return {"bytes": n * (7 * es + 4) + 4 * c["R"] * -(-c["F"] // GROUP), "flops": 25 * n}
    if op == "adapters":
        T, K, N, r = c["T"], c["K"], c["N"], c["r"]
        used = min(c["n"], c["requests"])
        return {"bytes": es * (T * (K + 2 * N) + used * r * (K + N)) + 4 * (T + 2 * c["n"]), "flops": 2 * T * r * (K + N)}
    T, k, H = c["T"], c["k"], c["H"]
    R, t = T * k, T - c["pad"]
    rows = t * k
    if op == "dispatch":
        return {"bytes": es * H * (t + rows) + 12 * R + 4 * c["E"], "flops": 0}
    if op == "dispatch_grad":
        return {"bytes": es * H * (T + rows) + 4 * R, "flops": rows * H}
    if op == "collect":
        return {"bytes": es * H * (T + rows) + 8 * R, "flops": 2 * rows * H}
    return {"bytes": es * H * (t + 2 * rows) + 12 * R, "flops": 3 * rows * H}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    op = c["op"]
    f64 = torch.float64

    def kept(x):
        """Group by group: the smallest power of two that brings the largest value to at most 127 steps."""
        R, F = x.shape
        v = x.to(f64)
        got = torch.empty_like(v)
        low, top = -126, 9 if x.dtype == torch.float16 else 121

        def two(e):  # 2^e, exactly: a value halfway between two steps stays there
            return ((e.long() + 1023) << 52).view(f64)

        for at in range(0, F, GROUP):
            part = v[:, at:at + GROUP]
            big = part.abs().max(dim=1, keepdim=True).values
            e = torch.ceil(torch.log2(big.clamp(min=2.0 ** -140) / 127))
            e = torch.where(127 * two(e - 1) >= big, e - 1, e)  # log2 may be an ulp off at a border
            e = torch.where(127 * two(e) < big, e + 1, e).clamp(low, top)
            step = two(e)
            got[:, at:at + GROUP] = (part / step).round().clamp(-127, 127) * step
        return got

    if op == "checkpoint":
        return {"x": kept(s["g"])}
    if op == "swiglu":
        def silu(v):
            return v * torch.sigmoid(v)
        g, u, dh = s["g"].to(f64), s["u"].to(f64), s["dh"].to(f64)
        h = silu(g) * u
        g, u = kept(s["g"]), kept(s["u"])
        sg = torch.sigmoid(g)
        return {"h": h, "dg": dh * u * (sg + g * sg * (1 - sg)), "du": dh * silu(g), "h_again": silu(g) * u}
    if op == "adapters":
        out = s["y"].to(f64)
        for a in range(c["n"]):
            at = torch.nonzero(s["ids"] == a).reshape(-1)
            if at.numel():
                out[at] += s["scale"][a].to(f64) * ((s["x"][at].to(f64) @ s["A"][a].to(f64).T) @ s["B"][a].to(f64).T)
        return {"out": out}
    T, k, E = c["T"], c["k"], c["E"]
    flat = s["idx"].reshape(-1).long()
    if op == "dispatch":
        lists = [torch.nonzero(flat == e).reshape(-1) for e in range(E)] + [torch.nonzero(flat < 0).reshape(-1)]
        perm = torch.cat(lists)
        offsets, at = [0], 0
        for part in lists[:-1]:
            at += part.numel()
            offsets.append(at)
        inv = torch.full_like(flat, -1)
        inv[perm[:at]] = torch.arange(at, device=flat.device)
        xs = torch.zeros(T * k, c["H"], dtype=f64, device="cuda")
        xs[:at] = s["x"].to(f64)[torch.div(perm[:at], k, rounding_mode="floor")]
        return {"xs": xs, "perm": perm, "inv": inv, "offsets": torch.tensor(offsets, device=flat.device)}
    inv = s["inv"].long().reshape(T, k)
    t = T - c["pad"]
    if op in ("dispatch_grad", "collect"):
        rows = s["dxs" if op == "dispatch_grad" else "o"]
        got = torch.zeros(T, c["H"], dtype=f64, device="cuda")
        for j in range(k):
            w = 1.0 if op == "dispatch_grad" else s["w"][:t, j:j + 1].to(f64)
            got[:t] += w * rows[inv[:t, j]].to(f64)
        return {"dx" if op == "dispatch_grad" else "y": got}
    do = torch.zeros(T * k, c["H"], dtype=f64, device="cuda")
    dw = torch.zeros(T, k, dtype=f64, device="cuda")
    dy = s["dy"][:t].to(f64)
    for j in range(k):
        do[inv[:t, j]] = s["w"][:t, j:j + 1].to(f64) * dy
        dw[:t, j] = torch.einsum("th,th->t", dy, s["o"][inv[:t, j]].to(f64))
    return {"do": do, "dw": dw}
