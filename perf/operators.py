"""Cases of the operators around the expert layer, with their plain forms.

Three operators that a training or serving program runs next to the Switch layer:

  grouped_fwd / grouped_bwd   products grouped by expert over ragged row ranges (experts of the
                              caller's own design, between a dispatch and a combine)
  norm_fwd / norm_bwd         the norms before and after the layer, with the token's gate, the
                              residual scale and the residual addition
  adamw                       one AdamW step over all tensors of the layer, states in 32 or 8 bits

`run` computes an operator in elementary torch operations in 32 bits, or (`own`) through the package.
"""
import math

import torch

own = False

EPS = 1e-6
LR, BETA1, BETA2, ADAM_EPS = 3e-4, 0.9, 0.999, 1e-8
BLOCK = 256                      # elements that share a scale in the 8-bit states
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
MASK32 = 0xFFFFFFFF


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token of each of 8 requests, routed over 128 experts: latency counts
        dict(name="fwd_decode8", op="grouped_fwd", dtype="bf16", M=8, K=1024, O=4096, N=128, cf=8.0,
             skew=0.0, spare=0, bias=True),
        # the first product of the large layer's experts, one training batch
        dict(name="fwd_large", op="grouped_fwd", dtype="bf16", M=16384, K=1024, O=4096, N=128, cf=1.5,
             skew=0.3, spare=512, bias=True),
        # a skewed router: popular experts hold many times the rows of the others
        dict(name="fwd_skewed", op="grouped_fwd", dtype="bf16", M=32768, K=2048, O=5120, N=64, cf=4.0,
             skew=0.8, spare=0, bias=False),
        # a float32 layer with odd widths
        dict(name="fwd_f32_odd", op="grouped_fwd", dtype="f32", M=4095, K=765, O=1021, N=60, cf=2.0,
             skew=0.4, spare=33, bias=True),
        # the gradients of a training batch's first product
        dict(name="bwd_large", op="grouped_bwd", dtype="bf16", M=16384, K=1024, O=4096, N=128, cf=1.5,
             skew=0.3, spare=512, bias=True),
        # float32 gradients, few experts
        dict(name="bwd_f32", op="grouped_bwd", dtype="f32", M=2050, K=512, O=1030, N=17, cf=2.0,
             skew=0.5, spare=0, bias=True),
        # one token between two sublayers: latency
        dict(name="norm_token", op="norm_fwd", dtype="bf16", T=1, d=1024, kind="rms", y=True, pre=True,
             post=True, gate=True, scale=True, bias=False),
        # a training batch of the skewed workload's width, norms on both sides
        dict(name="norm_batch", op="norm_fwd", dtype="bf16", T=32768, d=2048, kind="rms", y=True, pre=True,
             post=True, gate=True, scale=True, bias=False),
        # layer norm with bias in float32 at an odd width
        dict(name="norm_bwd_f32_odd", op="norm_bwd", dtype="f32", T=4099, d=771, kind="layer", y=True,
             pre=True, post=True, gate=False, scale=True, bias=True),
        # the backward pass of the training batch
        dict(name="norm_bwd_batch", op="norm_bwd", dtype="bf16", T=32768, d=2048, kind="rms", y=True,
             pre=True, post=True, gate=True, scale=True, bias=False),
        # a small float32 layer's tensors, the first step: launch latency
        dict(name="adamw_small_f32", op="adamw", dtype="f32", bits=32, master=False, N=4, d=96, d_ff=250,
             step=0, clip=False),
        # the base layer's expert weights in bf16 with float32 masters and 8-bit states
        dict(name="adamw_base_8bit", op="adamw", dtype="bf16", bits=8, master=True, N=64, d=768, d_ff=2048,
             step=1000, clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grouped_fwd", "grouped_fwd", "grouped_bwd", "norm_fwd", "norm_bwd", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("grouped_fwd", "grouped_bwd"):
        f32 = dtype == "f32"
        step = 1 if f32 else 8
        K = step * _log(rng, 64 / step, 2048 / step)
        O = step * _log(rng, 64 / step, 5120 / step)
        N = _log(rng, 2, min(256, 6.0e8 / (K * O)))
        most = (1.2e10 if f32 else 2.0e11) / (2 if op == "grouped_bwd" else 1) / (K * O)
        M = _log(rng, 1, max(2, min(32768, most)))
        return dict(op=op, dtype=dtype, M=M, K=K, O=O, N=N, cf=rng.choice([1.25, 2.0, 4.0]),
                    skew=rng.choice([0.0, 0.4, 0.8]), spare=rng.choice([0, 1, 77]),
                    bias=rng.random() < 0.6)
    if op in ("norm_fwd", "norm_bwd"):
        d = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            d = (d + 7) // 8 * 8
        T = _log(rng, 1, min(65536, 6.0e7 / d))
        kind = rng.choice(["rms", "layer"])
        y = rng.random() < 0.8
        pre = rng.random() < 0.8 or not y
        return dict(op=op, dtype=dtype, T=T, d=d, kind=kind, y=y, pre=pre,
                    post=y and rng.random() < 0.6, gate=y and rng.random() < 0.5,
                    scale=y and rng.random() < 0.5, bias=kind == "layer" and rng.random() < 0.7)
    return dict(op=op, dtype=dtype, bits=rng.choice([8, 32]), master=dtype == "bf16" and rng.random() < 0.5,
                N=_log(rng, 2, 48), d=_log(rng, 32, 768), d_ff=_log(rng, 32, 2048),
                step=rng.choice([0, 7, 30000]), clip=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    return g


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _capacity(c):
    return max(1, min(c["M"], math.ceil(c["cf"] * c["M"] / c["N"])))


def _group_sizes(c, g):
    """Rows per expert: draws from a skewed router, cut at the capacity, the overflow moved to the
    experts with free slots in expert order; they add up to M."""
    M, N, C = c["M"], c["N"], _capacity(c)
    w = (torch.arange(N, device="cuda", dtype=torch.float64) + 1) ** -c["skew"]
    w = w[torch.randperm(N, generator=g, device="cuda")]
    n = torch.bincount(torch.multinomial(w, M, replacement=True, generator=g), minlength=N)
    kept = n.clamp(max=C)
    free = C - kept
    before = free.cumsum(0) - free
    return kept + (M - kept.sum() - before).clamp(min=0).minimum(free)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] in ("grouped_fwd", "grouped_bwd"):
        dt, R, K, O, N = DTYPES[c["dtype"]], c["M"] + c["spare"], c["K"], c["O"], c["N"]
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"),
                                  _group_sizes(c, g).cumsum(0)]).to(torch.int32)
        s["x"] = _normal(g, (R, K), 1.0, dt)
        s["W"] = _normal(g, (N, O, K), K ** -0.5, dt)
        s["bias"] = _normal(g, (N, O), 0.1, dt) if c["bias"] else None
        s["cap"] = _capacity(c)
        if c["op"] == "grouped_fwd":
            s["out"] = torch.zeros((R, O), dtype=dt, device="cuda")
        else:
            s["dy"] = _normal(g, (R, O), 0.1, dt)
            s["dx"] = torch.zeros((R, K), dtype=dt, device="cuda")
            s["dW"] = torch.empty((N, O, K), dtype=dt, device="cuda")
            s["db"] = torch.empty((N, O), dtype=dt, device="cuda") if c["bias"] else None
        return s
    if c["op"] in ("norm_fwd", "norm_bwd"):
        dt, T, d = DTYPES[c["dtype"]], c["T"], c["d"]
        f = torch.float32
        wide = torch.exp(torch.randn(d, generator=g, device="cuda") * 0.5)    # channels differ in scale
        s["x"] = (_normal(g, (T, d), 1.0, f) * wide + 0.1).to(dt)
        s["y"] = s["gate"] = None
        if c["y"]:
            kept = (torch.rand(T, generator=g, device="cuda") > 0.1).to(f)    # dropped tokens: zero rows
            s["y"] = (_normal(g, (T, d), 0.5, f) * kept[:, None]).to(dt)
            if c["gate"]:
                s["gate"] = torch.rand(T, generator=g, device="cuda") * kept
        s["scale"] = 0.2 + _normal(g, (d,), 0.05, f) if c["scale"] else None
        s["w_pre"] = 1 + _normal(g, (d,), 0.1, f) if c["pre"] else None
        s["w_post"] = 1 + _normal(g, (d,), 0.1, f) if c["post"] else None
        s["b_pre"] = _normal(g, (d,), 0.1, f) if c["pre"] and c["bias"] else None
        s["b_post"] = _normal(g, (d,), 0.1, f) if c["post"] and c["bias"] else None
        if c["op"] == "norm_fwd":
            s["r"] = torch.empty((T, d), dtype=dt, device="cuda") if c["y"] else None
            s["h"] = torch.empty((T, d), dtype=dt, device="cuda") if c["pre"] else None
        else:
            s["dr"] = _normal(g, (T, d), 0.01, dt)
            s["dh"] = _normal(g, (T, d), 0.01, dt) if c["pre"] else None
        return s
    # adamw: the layer's tensors lie in one flat buffer, each from a multiple of BLOCK on; the bf16
    # layer's float32 router lies in a second one
    dt, N, d, d_ff = DTYPES[c["dtype"]], c["N"], c["d"], c["d_ff"]
    experts = [N * d_ff * d, N * d_ff, N * d * d_ff, N * d]
    decays = [0.1, 0.0, 0.1, 0.0]
    s["groups"] = [_flat_group(c, g, experts + ([N * d, N] if dt == torch.float32 else []),
                               decays + ([0.1, 0.0] if dt == torch.float32 else []), dt)]
    if dt != torch.float32:
        s["groups"].append(_flat_group(c, g, [N * d, N], [0.1, 0.0], torch.float32))
    s["step"] = torch.tensor([c["step"], 0], dtype=torch.int32, device="cuda")
    s["grad_scale"] = torch.full((1,), 0.37, device="cuda") if c["clip"] else None
    s["seed"] = 12345
    s["params"] = [t for q in s["groups"] for t in q["params"]]
    s["grads"] = [t for q in s["groups"] for t in q["grads"]]
    s["decays"] = [v for q in s["groups"] for v in q["decays"]]
    s["state"] = {"step": s["step"]}
    for k in ("m", "v", "m_scale", "v_scale", "master"):
        s["state"][k] = [t for q in s["groups"] for t in q["views"][k]]
    return s


def _flat_group(c, g, sizes, decays, dt):
    blocks = [-(-n // BLOCK) for n in sizes]
    nb, dev = sum(blocks), "cuda"
    begin = [sum(blocks[:i]) * BLOCK for i in range(len(sizes))]
    which = torch.repeat_interleave(torch.arange(len(sizes), device=dev), torch.tensor(blocks, device=dev))
    q = {"sizes": sizes, "decays": decays, "dt": dt}
    q["wd"] = torch.tensor(decays, device=dev, dtype=torch.float64)[which][:, None]
    q["block"] = torch.arange(nb, device=dev) - torch.tensor([b // BLOCK for b in begin], device=dev)[which]
    at = q["block"][:, None] * BLOCK + torch.arange(BLOCK, device=dev)
    inside = at < torch.tensor(sizes, device=dev)[which][:, None]

    def fill(std):
        return torch.randn((nb, BLOCK), generator=g, device=dev) * std * inside

    value = fill(0.02)
    q["p"] = value.to(dt)
    q["g"] = (fill(1.0) * torch.exp(torch.randn((nb, 1), generator=g, device=dev)) * 1e-3).to(dt)
    q["master"] = value.clone() if c["master"] and dt != torch.float32 else None
    m = fill(2e-4) if c["step"] else torch.zeros((nb, BLOCK), device=dev)
    r = fill(1.0).abs() * 1e-3 if c["step"] else torch.zeros((nb, BLOCK), device=dev)
    q["m_scale"] = q["v_scale"] = None
    if c["bits"] == 8:
        q["m_scale"], q["v_scale"] = m.abs().amax(1) / 448, r.amax(1) / 448
        q["m"] = (m / q["m_scale"].clamp(min=1e-30)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        q["v"] = (r / q["v_scale"].clamp(min=1e-30)[:, None]).clamp(0, 448).to(torch.float8_e4m3fn)
    else:
        q["m"], q["v"] = m, r * r

    def views(t, per=1):
        if t is None:
            return [None] * len(sizes)
        t = t.reshape(-1)
        return [t[b // per:b // per + -(-n // per)] for b, n in zip(begin, sizes)]

    q["params"], q["grads"] = views(q["p"]), views(q["g"])
    q["views"] = {"m": views(q["m"]), "v": views(q["v"]), "master": views(q["master"]),
                  "m_scale": views(q["m_scale"], BLOCK), "v_scale": views(q["v_scale"], BLOCK)}
    return q


# ---------------------------------------------------------------- one pass
def run(s):
    return {"grouped_fwd": _grouped_fwd, "grouped_bwd": _grouped_bwd, "norm_fwd": _norm_fwd,
            "norm_bwd": _norm_bwd, "adamw": _adamw}[s["case"]["op"]](s)


def _slots(s):
    """Row r of expert e goes to slot e * cap + (r - offsets[e]) of a padded batch; rows of no expert
    to a spare slot behind it."""
    c, off = s["case"], s["offsets"].long()
    r = torch.arange(s["x"].shape[0], device="cuda")
    e = torch.searchsorted(off[1:].contiguous(), r, right=True)
    real = (e < c["N"]) & (r >= off[0])
    return torch.where(real, e * s["cap"] + r - off[e.clamp(max=c["N"])], c["N"] * s["cap"]), real


def _padded(rows, slot, c, cap, t):
    p = torch.zeros((c["N"] * cap + 1, rows.shape[1]), dtype=t, device="cuda")
    p[slot] = rows.to(t)
    return p[:-1].view(c["N"], cap, rows.shape[1])


def _rows(p, slot, real, before):
    flat = p.reshape(-1, p.shape[2])
    return torch.where(real[:, None], flat[slot.clamp(max=flat.shape[0] - 1)].to(before.dtype), before)


def _grouped_fwd(s):
    if own:
        import sparse_mixture_experts_argmax_b200 as swl
        return swl.grouped_matmul(s["x"], s["offsets"], s["W"], bias=s["bias"], out=s["out"], check=False)
    slot, real = _slots(s)
    y = torch.bmm(_padded(s["x"], slot, s["case"], s["cap"], torch.float32), s["W"].float().transpose(1, 2))
    if s["bias"] is not None:
        y = y + s["bias"].float()[:, None]
    return _rows(y, slot, real, s["out"])


def _grouped_bwd(s):
    if own:
        import sparse_mixture_experts_argmax_b200 as swl
        return swl.grouped_matmul_backward(s["dy"], s["x"], s["offsets"], s["W"], dx=s["dx"], dW=s["dW"],
                                           db=s["db"], check=False)
    slot, real = _slots(s)
    dy = _padded(s["dy"], slot, s["case"], s["cap"], torch.float32)
    x = _padded(s["x"], slot, s["case"], s["cap"], torch.float32)
    got = {"dx": _rows(torch.bmm(dy, s["W"].float()), slot, real, s["dx"]),
           "dW": torch.bmm(dy.transpose(1, 2), x).to(s["x"].dtype)}
    got["db"] = dy.sum(1).to(s["x"].dtype) if s["db"] is not None else None
    return got


def _normed(t, kind):
    if kind == "layer":
        t = t - t.mean(1, keepdim=True)
    rho = 1 / torch.sqrt((t * t).mean(1, keepdim=True) + EPS)
    return t * rho, rho


def _norm_fwd(s):
    c = s["case"]
    if own:
        import sparse_mixture_experts_argmax_b200 as swl
        return swl.norm_residual(s["x"], y=s["y"], w_pre=s["w_pre"], b_pre=s["b_pre"], w_post=s["w_post"],
                                 b_post=s["b_post"], gate=s["gate"], scale=s["scale"], kind=c["kind"],
                                 eps=EPS, r=s["r"], h=s["h"])
    r = s["x"].float()
    if c["y"]:
        u = s["y"].float()
        if c["post"]:
            u = _normed(u, c["kind"])[0] * s["w_post"]
            u = u + s["b_post"] if s["b_post"] is not None else u
        u = u * s["scale"] if c["scale"] else u
        u = u * s["gate"][:, None] if c["gate"] else u
        r = r + u
    got = {"r": r.to(s["x"].dtype), "h": None}
    if c["pre"]:
        h = _normed(r, c["kind"])[0] * s["w_pre"]
        got["h"] = (h + s["b_pre"] if s["b_pre"] is not None else h).to(s["x"].dtype)
    return got


def _norm_back(grad, w, hat, rho, kind):
    a = grad * w
    back = a - hat * (a * hat).mean(1, keepdim=True)
    if kind == "layer":
        back = back - a.mean(1, keepdim=True)
    return back * rho


def _norm_bwd(s):
    c, dt = s["case"], s["x"].dtype
    if own:
        import sparse_mixture_experts_argmax_b200 as swl
        return swl.norm_residual_backward(s["dr"], s["dh"], s["x"], y=s["y"], w_pre=s["w_pre"],
                                          b_pre=s["b_pre"], w_post=s["w_post"], b_post=s["b_post"],
                                          gate=s["gate"], scale=s["scale"], kind=c["kind"], eps=EPS)
    got = dict.fromkeys(("dx", "dy", "dgate", "dscale", "dw_pre", "db_pre", "dw_post", "db_post"))
    D = s["dr"].float()
    if c["pre"]:
        dh = s["dh"].float()
        hat, rho = _normed(s["x"].float(), c["kind"])
        D = D + _norm_back(dh, s["w_pre"], hat, rho, c["kind"])
        got["dw_pre"] = (dh * hat).sum(0)
        got["db_pre"] = dh.sum(0) if s["b_pre"] is not None else None
    got["dx"] = D.to(dt)
    if c["y"]:
        u = s["y"].float()
        if c["post"]:
            hat, rho = _normed(u, c["kind"])
            u = hat * s["w_post"]
            u = u + s["b_post"] if s["b_post"] is not None else u
        if c["gate"]:
            got["dgate"] = (D * u * s["scale"] if c["scale"] else D * u).sum(1)
            D = D * s["gate"][:, None]
        if c["scale"]:
            got["dscale"] = (D * u).sum(0)
            D = D * s["scale"]
        if c["post"]:
            got["dw_post"] = (D * hat).sum(0)
            got["db_post"] = D.sum(0) if s["b_post"] is not None else None
            D = _norm_back(D, s["w_post"], hat, rho, c["kind"])
        got["dy"] = D.to(dt)
    return got


def _adamw_out(s):
    return {"step": s["step"][:1], "groups": [{k: q[k] for k in ("p", "master", "m", "v", "m_scale", "v_scale")}
                                              for q in s["groups"]]}


def _adamw(s):
    if own:
        import sparse_mixture_experts_argmax_b200 as swl
        swl.adamw_step(s["params"], s["grads"], s["state"], lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS,
                       weight_decay=s["decays"], grad_scale=s["grad_scale"], seed=s["seed"])
        return _adamw_out(s)
    s["step"][0] += 1
    t = s["step"][0].double()
    rate = (LR / (1 - torch.pow(torch.full_like(t, BETA1), t))).float()
    root2 = (1 / torch.sqrt(1 - torch.pow(torch.full_like(t, BETA2), t))).float()
    _adamw_flat(s, s["groups"][0], rate, root2)
    if len(s["groups"]) > 1:
        _adamw_flat(s, s["groups"][1], rate, root2)
    return _adamw_out(s)


def _dither(s, q):
    """16 random bits per element from (index pair, step, seed)."""
    pair = q["block"][:, None] * (BLOCK // 2) + torch.arange(BLOCK // 2, device="cuda")
    x = (pair + s["step"][0].long() * 0x3C6EF373 + s["seed"] * 0xA54FF53B) & MASK32
    x = ((x ^ (x >> 16)) * 0x6A09E667) & MASK32
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & MASK32
    x = x ^ (x >> 16)
    return torch.stack([x & 0xFFFF, x >> 16], 2).reshape(-1, BLOCK)


def _adamw_flat(s, q, rate, root2):
    eight = q["m_scale"] is not None
    w = q["p"].float() if q["master"] is None else q["master"]
    g = q["g"].float()
    if s["grad_scale"] is not None:
        g = g * s["grad_scale"]
    if eight:
        m = q["m"].float() * q["m_scale"][:, None]
        r = q["v"].float() * q["v_scale"][:, None]
        v = r * r
    else:
        m, v = q["m"], q["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    r = torch.sqrt(v)
    w = w * (1 - LR * q["wd"]).float() - (m / (r * root2 + ADAM_EPS)) * rate
    q["p"].copy_(w)
    if q["master"] is not None:
        q["master"].copy_(w)
    if not eight:
        q["m"].copy_(m)
        q["v"].copy_(v)
        return
    least = 2.0 ** -100
    top_m, top_r = m.abs().amax(1, keepdim=True), r.amax(1, keepdim=True)
    code = torch.where(top_m < least, 0.0, (m * (448 / top_m.clamp(min=least))).clamp(-448, 448))
    x = r * (448 / top_r.clamp(min=least))
    x = ((x.view(torch.int32) + (_dither(s, q) * 16 + 8).int()) & -0x100000).view(torch.float32)
    root = torch.where((top_r < least) | (r <= 0), 0.0, x.clamp(2.0 ** -9, 448))
    q["m"].copy_(code.to(torch.float8_e4m3fn))
    q["v"].copy_(root.to(torch.float8_e4m3fn))
    q["m_scale"].copy_(torch.where(top_m < least, 0.0, top_m / 448)[:, 0])
    q["v_scale"].copy_(torch.where(top_r < least, 0.0, top_r / 448)[:, 0])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] in ("grouped_fwd", "grouped_bwd"):
        e = 2 if c["dtype"] == "bf16" else 4
        M, K, O, N = c["M"], c["K"], c["O"], c["N"]
        used = N * (1 - (1 - 1 / N) ** M)           # experts with rows, on average
        b = e * O if c["bias"] else 0
        if c["op"] == "grouped_fwd":
            return {"bytes": e * M * (K + O) + used * (e * O * K + b), "flops": 2.0 * M * K * O}
        return {"bytes": e * M * (2 * K + O) + used * e * O * K + N * (e * O * K + b),
                "flops": 4.0 * M * K * O}
    if c["op"] in ("norm_fwd", "norm_bwd"):
        e = 2 if c["dtype"] == "bf16" else 4
        T, d = c["T"], c["d"]
        vectors = c["pre"] + c["post"] + c["scale"] + (c["bias"] and c["pre"]) + (c["bias"] and c["post"])
        if c["op"] == "norm_fwd":
            arrays = 1 + 2 * c["y"] + c["pre"]
            return {"bytes": e * T * d * arrays + 4 * T * c["gate"] + 4 * d * vectors, "flops": 10.0 * T * d}
        arrays = 2 + 2 * c["pre"] + 2 * c["y"]      # dr, dx; x, dh; y, dy
        return {"bytes": e * T * d * arrays + 8 * T * c["gate"] + 8 * d * vectors, "flops": 25.0 * T * d}
    N, d, d_ff = c["N"], c["d"], c["d_ff"]
    n, n32 = N * (2 * d_ff * d + d_ff + d), N * (d + 1)
    states = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
    each = (12 if c["dtype"] == "f32" else 14 if c["master"] else 6) + states
    if c["dtype"] == "bf16" and c["master"]:
        each -= 2                                    # the bf16 copy is written, not read
    return {"bytes": n * each + n32 * (12 + states), "flops": 20.0 * (n + n32)}


# ---------------------------------------------------------------- the same from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    D = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"] in ("grouped_fwd", "grouped_bwd"):
        off = s["offsets"].tolist()
        if case["op"] == "grouped_fwd":
            out = D["out"]
            for e in range(case["N"]):
                a, b = off[e], off[e + 1]
                if b > a:
                    out[a:b] = D["x"][a:b] @ D["W"][e].T + (D["bias"][e] if case["bias"] else 0)
            return out
        dx, dW = D["dx"], torch.zeros_like(D["W"])
        db = torch.zeros((case["N"], case["O"]), dtype=torch.float64, device="cuda") if case["bias"] else None
        for e in range(case["N"]):
            a, b = off[e], off[e + 1]
            if b > a:
                dx[a:b] = D["dy"][a:b] @ D["W"][e]
                dW[e] = D["dy"][a:b].T @ D["x"][a:b]
                if case["bias"]:
                    db[e] = D["dy"][a:b].sum(0)
        return {"dx": dx, "dW": dW, "db": db}
    if case["op"] == "norm_fwd":
        return _exact_norm(D, case)
    if case["op"] == "norm_bwd":
        # the formulas' gradients by differentiating the 64-bit definition
        names = [k for k in ("x", "y", "gate", "scale", "w_pre", "b_pre", "w_post", "b_post") if D.get(k) is not None]
        leaf = {k: D[k].clone().requires_grad_() for k in names}
        # `x` holds the residual r = x0 + u that the backward pass reads: x0 = r - u as a constant
        with torch.no_grad():
            base = D["x"] - _exact_branch(D, case) if case["y"] else D["x"]
        x0 = base.clone().requires_grad_()
        r = x0 + _exact_branch({**D, **leaf}, case) if case["y"] else x0
        total = (D["dr"] * r).sum()
        if case["pre"]:
            total = total + (D["dh"] * _exact_affine(r, leaf["w_pre"], leaf.get("b_pre"), case["kind"])).sum()
        wanted = [x0] + [leaf[k] for k in names if k != "x"]
        got = dict(zip(["x"] + [k for k in names if k != "x"], torch.autograd.grad(total, wanted)))
        return {"d" + k: got.get(k) for k in ("x", "y", "gate", "scale", "w_pre", "b_pre", "w_post", "b_post")}
    t = case["step"] + 1
    groups = []
    for q in s["groups"]:
        g = q["g"].double() * (s["grad_scale"].double() if case["clip"] else 1.0)
        w = (q["p"] if q["master"] is None else q["master"]).double()
        if case["bits"] == 8:
            m = q["m"].double() * q["m_scale"].double()[:, None]
            v = (q["v"].double() * q["v_scale"].double()[:, None]).square()
        else:
            m, v = q["m"].double(), q["v"].double()
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g.square()
        w = w - LR * (q["wd"] * w + m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)).sqrt() + ADAM_EPS))
        one = {"p": w, "master": None if q["master"] is None else w, "m": m, "v": v, "m_scale": None, "v_scale": None}
        if case["bits"] == 8:
            one.update(m=None, v=None, m_scale=m.abs().amax(1) / 448, v_scale=v.amax(1).sqrt() / 448)
        groups.append(one)
    return {"step": torch.tensor([t], dtype=torch.int32, device="cuda"), "groups": groups}


def _exact_affine(t, w, b, kind):
    if kind == "layer":
        z = (t - t.mean(1, keepdim=True)) / (t.var(1, unbiased=False, keepdim=True) + EPS).sqrt()
    else:
        z = t / (t.square().mean(1, keepdim=True) + EPS).sqrt()
    return z * w if b is None else z * w + b


def _exact_branch(D, c):
    u = _exact_affine(D["y"], D["w_post"], D.get("b_post"), c["kind"]) if c["post"] else D["y"]
    if c["scale"]:
        u = u * D["scale"]
    return u * D["gate"][:, None] if c["gate"] else u


def _exact_norm(D, c):
    r = D["x"] + _exact_branch(D, c) if c["y"] else D["x"]
    return {"r": r, "h": _exact_affine(r, D["w_pre"], D.get("b_pre"), c["kind"]) if c["pre"] else None}
