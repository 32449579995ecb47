"""Cases and plain forms of the differential softmax anchor and the block norms.

`run` computes them with elementary torch operations in 32 bits, or, where
`own` is set, with the library's entry points. `exact` gives the same outputs
from the definitions in 64 bits (gradients by automatic differentiation).

Differential anchor ("diff"), per batch b and head h, with the head's q and k
columns split in two maps of d/2 and v whole:
    P_m = softmax_s(scale q_m . k_m)  over the keys s < key_lens[b],  m = 1, 2
    out = (P_1 v - lambda P_2 v) * sigmoid(gate)
Block norms ("norm"), per token, N an RMS or layer norm over the D channels:
    h'  = res_scale h + gate_b * (N(o) w_post)
    u   = N(h') w_pre (1 + scale_b) + shift_b
"""
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # one new query row against a 480p clip's keys, both CFG branches: latency of a single token
        dict(name="diff_one_query", op="diff", dtype="bf16", B=2, N=1, keys=8190, H=16, d=128,
             train=False, lam="token", ragged=False),
        # the fp32 four-head group of the small test configuration
        dict(name="diff_fp32_1024", op="diff", dtype="fp32", B=1, N=1024, keys=1024, H=4, d=64,
             train=False, lam="token", ragged=False),
        # a 480p clip, one anchor layer, inference
        dict(name="diff_480p", op="diff", dtype="bf16", B=1, N=8190, keys=8190, H=16, d=128,
             train=False, lam="token", ragged=False),
        # one eighth of a 720p clip's queries against all of its keys (a sequence shard)
        dict(name="diff_shard_720p", op="diff", dtype="bf16", B=1, N=2415, keys=19320, H=16, d=128,
             train=False, lam="head", ragged=False),
        # a padded batch of short clips of different lengths, one of them empty: a training step
        dict(name="diff_train_ragged", op="diff", dtype="bf16", B=4, N=1555, keys=1555, H=8, d=128,
             train=True, lam="head", ragged=True),
        # a training step of one anchor layer on a 480p clip
        dict(name="diff_train_480p", op="diff", dtype="bf16", B=1, N=8190, keys=8190, H=16, d=128,
             train=True, lam="token", ragged=False),
        # a training step in fp32 at an odd length
        dict(name="diff_train_fp32", op="diff", dtype="fp32", B=2, N=777, keys=777, H=4, d=128,
             train=True, lam="token", ragged=False),
        # between two layers for a handful of tokens: latency
        dict(name="norm_small", op="norm", dtype="bf16", B=2, N=16, D=2048, kind="rms", train=False,
             post=True, pre=True, mod=True),
        # between two layers of a 480p clip, inference, both CFG branches
        dict(name="norm_480p", op="norm", dtype="bf16", B=2, N=8190, D=2048, kind="rms", train=False,
             post=True, pre=True, mod=True),
        # the same in a training step
        dict(name="norm_train_480p", op="norm", dtype="bf16", B=2, N=8190, D=2048, kind="rms",
             train=True, post=True, pre=True, mod=True),
        # fp32, layer norm, an odd width and length, no modulation: a training step
        dict(name="norm_train_fp32_odd", op="norm", dtype="fp32", B=3, N=1001, D=1002, kind="layer",
             train=True, post=True, pre=True, mod=False),
        # the norm before a stack's first layer alone, a long clip in training
        dict(name="norm_train_pre_long", op="norm", dtype="bf16", B=1, N=37720, D=2048, kind="layer",
             train=True, post=False, pre=True, mod=True),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.6:
        bf16 = rng.random() < 0.75
        B, H = rng.randint(1, 4), rng.randint(1, 16)
        keys = _between(rng, 16, 19000)
        same = rng.random() < 0.6
        N = keys if same else 1 if rng.random() < 0.3 else _between(rng, 1, 8000)
        most = 1e9 if bf16 else 6e7  # B H N keys: scores that the plain form holds
        while B * H * N * keys > most:
            if B > 1:
                B -= 1
            elif H > 4:
                H -= 1
            elif same:
                N = keys = keys * 3 // 4
            else:
                N = max(1, N // 2)
        return dict(op="diff", dtype="bf16" if bf16 else "fp32", B=B, N=N, keys=keys, H=H,
                    d=128 if bf16 else rng.choice([64, 128]), train=rng.random() < 0.5,
                    lam=rng.choice(["token", "head"]), ragged=rng.random() < 0.4)
    D, B = _between(rng, 64, 8192), rng.randint(1, 4)
    N = _between(rng, 1, max(2, int(7.5e7 / (B * D))))
    part = rng.choice(["both", "both", "both", "pre", "post"])
    return dict(op="norm", dtype="bf16" if rng.random() < 0.75 else "fp32", B=B, N=N, D=D,
                kind=rng.choice(["rms", "layer"]), train=rng.random() < 0.5, post=part != "pre",
                pre=part != "post", mod=rng.random() < 0.7)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _up8(n):
    return (n + 7) // 8 * 8


def _lens(case, seed):
    """Key counts of a padded batch: one full row, one empty (of three or more), the rest between."""
    B, keys = case["B"], case["keys"]
    if not case["ragged"]:
        return None
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(1, keys + 1, (B,), generator=g)
    lens[0] = keys
    if B > 2:
        lens[1] = 0
    return lens.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(case)

    def normal(*shape, of=None, mean=0.0, std=1.0):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return (t * std + mean).to(dt if of is None else of)

    s = dict(case=case)
    B, N = case["B"], case["N"]
    if case["op"] == "diff":
        H, d, keys = case["H"], case["d"], case["keys"]
        D = H * d
        # q, k, v, gate and the per-token lambda logits are slices of one projection's output, as
        # are their gradients; queries of a shard have keys and values of their own length
        W = 4 * D + _up8(H)
        names = [("q", 0, D), ("k", D, D), ("v", 2 * D, D), ("gate", 3 * D, D), ("lam", 4 * D, H)]
        fused = normal(B, N, W)
        grads = torch.empty(B, N, W, device="cuda", dtype=dt) if case["train"] else None
        for n, at, w in names:
            s[n] = fused[..., at:at + w]
            if case["train"]:
                s["d" + n] = grads[..., at:at + w]
        if keys != N:
            kv = normal(B, keys, 2 * D)
            s["k"], s["v"] = kv[..., :D], kv[..., D:]
            if case["train"]:
                dkv = torch.empty(B, keys, 2 * D, device="cuda", dtype=dt)
                s["dk"], s["dv"] = dkv[..., :D], dkv[..., D:]
        if case["lam"] == "head":  # the learned weights themselves, shared by all tokens
            s["lam"] = normal(H, mean=0.5, std=0.2)
            if case["train"]:
                s["dlam"] = torch.empty(H, device="cuda", dtype=dt)
        lens = _lens(case, seed)
        s["key_lens"] = None if lens is None else lens.cuda()
        s["out"] = torch.empty(B, N, D, device="cuda", dtype=dt)
        if case["train"]:
            s["dout"] = normal(B, N, D)
            s["saved"] = (torch.empty(B, N, D, device="cuda", dtype=dt),
                          torch.empty(B, N, D, device="cuda", dtype=dt),
                          torch.empty(2, B, H, N, device="cuda", dtype=torch.float32))
        s["ws"] = s["ws_bwd"] = None
        return s
    D = case["D"]
    ld = _up8(D)
    f32 = torch.float32
    s["h"] = normal(B, N, ld, of=f32, std=2.0)[..., :D]
    s["res_scale"] = 1.0 if case["kind"] == "rms" else 0.9
    for n in ("o", "w_post", "gate", "w_pre", "scale", "shift"):
        s[n] = None
    if case["post"]:
        s["o"] = normal(B, N, ld, std=0.5)[..., :D]
        s["w_post"] = normal(D, mean=1.0, std=0.1)
        s["h_out"] = torch.empty(B, N, ld, device="cuda", dtype=f32)[..., :D]
        if case["mod"]:
            s["gate"] = normal(B, ld, std=0.5)[:, :D]
    if case["pre"]:
        s["w_pre"] = normal(D, mean=1.0, std=0.1)
        s["u"] = torch.empty(B, N, ld, device="cuda", dtype=dt)[..., :D]
        if case["mod"]:
            mod = normal(B, 2 * ld, std=0.3)
            s["scale"], s["shift"] = mod[:, :D], mod[:, ld:ld + D]
    if case["train"]:
        s["stats"] = torch.empty(B, N, 4, device="cuda", dtype=f32)
        s["dh_out"] = normal(B, N, ld, of=f32)[..., :D]
        s["dh"] = torch.empty(B, N, ld, device="cuda", dtype=f32)[..., :D]
        if case["post"]:
            s["do"] = torch.empty(B, N, ld, device="cuda", dtype=dt)[..., :D]
            s["dw_post"] = torch.empty(D, device="cuda", dtype=f32)
            if case["mod"]:
                s["dgate"] = torch.empty(B, D, device="cuda", dtype=f32)
        if case["pre"]:
            s["du"] = normal(B, N, ld)[..., :D]
            s["dw_pre"] = torch.empty(D, device="cuda", dtype=f32)
            if case["mod"]:
                s["dscale"] = torch.empty(B, D, device="cuda", dtype=f32)
                s["dshift"] = torch.empty(B, D, device="cuda", dtype=f32)
    s["ws"] = None
    return s


_DIFF_GRADS = ("dq", "dk", "dv", "dgate", "dlam")
_NORM_GRADS = ("dh", "do", "dw_post", "dgate", "dw_pre", "dscale", "dshift")


def _own_diff(s):
    import softmax_attention_video_gated_b200 as sva

    case = s["case"]
    flags = sva.SVA_FLAG_LAMBDA_VALUE if case["lam"] == "head" else 0
    more = dict(key_lens=s["key_lens"], flags=flags)
    if case["train"] and s["saved"][0].dtype != torch.float32:  # the two maps' outputs are kept in 32 bits
        s["saved"] = (*(torch.empty_like(o, dtype=torch.float32) for o in s["saved"][:2]), s["saved"][2])
    s["ws"] = sva.sva_diff_anchor_fwd(s["q"], s["k"], s["v"], s["gate"], s["lam"], s["out"], case["H"],
                                      saved=s.get("saved"), ws=s["ws"], **more)
    if not case["train"]:
        return dict(out=s["out"])
    s["ws_bwd"] = sva.sva_diff_anchor_bwd(s["q"], s["k"], s["v"], s["gate"], s["lam"], s["dout"],
                                          s["saved"], s["dq"], s["dk"], s["dv"], s["dgate"],
                                          s["dlam"], case["H"], ws=s["ws_bwd"], **more)
    return dict(out=s["out"], **{n: s[n] for n in _DIFF_GRADS})


def _own_norm(s):
    import softmax_attention_video_gated_b200 as sva

    case = s["case"]
    kind = sva.SVA_NORM_RMS if case["kind"] == "rms" else sva.SVA_NORM_LAYER
    more = dict(w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"], scale=s["scale"], kind=kind,
                eps=EPS, res_scale=s["res_scale"])
    sva.sva_block_norm_fwd(s["h"], o=s["o"], h_out=s.get("h_out"), u=s.get("u"), shift=s["shift"],
                           stats=s.get("stats"), **more)
    out = {n: s[n] for n in ("h_out", "u") if n in s}
    if not case["train"]:
        return out
    s["ws"] = sva.sva_block_norm_bwd(s["h_out"] if case["post"] else s["h"], s["stats"], s["dh"],
                                     dh_out=s["dh_out"], o=s["o"], do=s.get("do"), du=s.get("du"),
                                     dw_post=s.get("dw_post"), dgate=s.get("dgate"),
                                     dw_pre=s.get("dw_pre"), dscale=s.get("dscale"),
                                     dshift=s.get("dshift"), ws=s["ws"], **more)
    return dict(out, **{n: s[n] for n in _NORM_GRADS if n in s})


def _heads(t, H, maps=1):
    """[B, N, H*d] -> fp32 [B, H, maps, N, d / maps]"""
    B, N, D = t.shape
    return t.float().reshape(B, N, H, maps, D // H // maps).permute(0, 2, 3, 1, 4)


def _rows(t):
    """[B, H, maps, N, w] -> [B, N, H*maps*w]"""
    B, H, M, N, w = t.shape
    return t.permute(0, 3, 1, 2, 4).reshape(B, N, H * M * w)


def _plain_diff(s):
    case = s["case"]
    H, dt = case["H"], _dtype(case)
    q, k = _heads(s["q"], H, 2), _heads(s["k"], H, 2)
    v, gate = _heads(s["v"], H), torch.sigmoid(_heads(s["gate"], H))
    per_head = case["lam"] == "head"
    if per_head:
        lam = s["lam"].float().view(1, H, 1, 1, 1)
    else:
        lam = torch.sigmoid(s["lam"].float()).permute(0, 2, 1)[:, :, None, :, None]
    scale = 1.0 / math.sqrt(case["d"] / 2)
    p = q @ k.transpose(-1, -2) * scale                                 # [B, H, 2, N, keys]
    if s["key_lens"] is not None:
        at = torch.arange(case["keys"], device=p.device)
        p.masked_fill_(at >= s["key_lens"].view(-1, 1, 1, 1, 1), -math.inf)
    top = p.amax(-1, keepdim=True)
    p = torch.exp(p - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    o = p @ v
    a = o[:, :, :1] - lam * o[:, :, 1:]
    res = dict(out=_rows(a * gate).to(dt))
    if not case["train"]:
        return res
    dy = _heads(s["dout"], H)
    da = dy * gate
    dgate = dy * a * gate * (1 - gate)
    dv = (p[:, :, :1] - lam * p[:, :, 1:]).transpose(-1, -2) @ da
    dp = da @ v.transpose(-1, -2)
    delta = (dp * p).sum(-1, keepdim=True)                              # [B, H, 2, N, 1]
    ds = p * (dp - delta)
    ds[:, :, 1:] *= -lam
    dq, dk = ds @ k * scale, ds.transpose(-1, -2) @ q * scale
    dlam = -delta[:, :, 1, :, 0]                                        # [B, H, N]
    if per_head:
        dlam = dlam.sum((0, 2))
    else:
        lt = lam[:, :, 0, :, 0]
        dlam = (dlam * lt * (1 - lt)).permute(0, 2, 1)
    return dict(res, dq=_rows(dq).to(dt), dk=_rows(dk).to(dt), dv=_rows(dv).to(dt),
                dgate=_rows(dgate).to(dt), dlam=dlam.to(dt))


def _normed(x, layer):
    """(normalised x, reciprocal deviation)"""
    if layer:
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _norm_back(dx, x, r, layer):
    """The gradient before the norm, from the one behind it and the normalised x."""
    dx = dx - x * (dx * x).mean(-1, keepdim=True) - (dx.mean(-1, keepdim=True) if layer else 0.0)
    return dx * r


def _plain_norm(s):
    case, dt = s["case"], _dtype(s["case"])
    layer = case["kind"] == "layer"
    f = {n: None if s[n] is None else s[n].float() for n in ("w_post", "gate", "w_pre", "scale", "shift")}
    gate = 1.0 if f["gate"] is None else f["gate"][:, None]
    scale = 1.0 if f["scale"] is None else 1.0 + f["scale"][:, None]
    shift = 0.0 if f["shift"] is None else f["shift"][:, None]
    h, res = s["h"], {}
    if case["post"]:
        on, ro = _normed(s["o"].float(), layer)
        h = res["h_out"] = s["res_scale"] * h + gate * (on * f["w_post"])
    if case["pre"]:
        hn, rh = _normed(h, layer)
        res["u"] = (hn * f["w_pre"] * scale + shift).to(dt)
    if not case["train"]:
        return res
    dh = s["dh_out"]
    if case["pre"]:
        du = s["du"].float()
        col = (du * hn).sum(1)                                          # [B, D]
        if case["mod"]:
            res["dscale"], res["dshift"] = col * f["w_pre"], du.sum(1)
        res["dw_pre"] = (col[:, None] * scale).sum((0, 1))
        dh = dh + _norm_back(du * (f["w_pre"] * scale), hn, rh, layer)
    if case["post"]:
        col = (dh * on).sum(1)
        if case["mod"]:
            res["dgate"] = col * f["w_post"]
        res["dw_post"] = (col[:, None] * gate).sum((0, 1))
        res["do"] = _norm_back(dh * (gate * f["w_post"]), on, ro, layer).to(dt)
        dh = dh * s["res_scale"]
    res["dh"] = dh
    return res


def run(s):
    if own:
        return _own_diff(s) if s["case"]["op"] == "diff" else _own_norm(s)
    return _plain_diff(s) if s["case"]["op"] == "diff" else _plain_norm(s)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, N = case["B"], case["N"]
    if case["op"] == "diff":
        keys, D = case["keys"], case["H"] * case["d"]
        rows, cols = B * N, B * keys
        pairs = B * case["H"] * N * keys
        if case["ragged"]:  # the expected share of a padded batch's keys
            pairs = pairs * (1 if B == 1 else 0.75 if B == 2 else (1 + (B - 2) / 2) / B)
        # scores of two maps of d/2, two products with v
        flops = pairs * (2 * case["d"] + 4 * case["d"])
        moved = e * (D * (3 * rows + 2 * cols) + case["H"] * (rows if case["lam"] == "token" else 1))
        if case["train"]:
            # scores again, dP, dV, and dQ and dK of two maps of d/2
            flops += pairs * 10 * case["d"]
            # dout, the gradients, and the saved outputs of both maps and their statistics, once each way
            moved += e * D * (rows + 2 * rows + 2 * cols) + 2 * (2 * e * D + 8 * case["H"]) * rows
        return dict(bytes=moved, flops=flops)
    rows, D = B * N, case["D"]
    fwd = (4 + (e + 4 if case["post"] else 0) + (e if case["pre"] else 0)) * rows * D
    if not case["train"]:
        return dict(bytes=fwd, flops=12 * rows * D)
    bwd = (8 + (4 + e if case["pre"] else 0) + (2 * e if case["post"] else 0)) * rows * D
    return dict(bytes=fwd + bwd, flops=36 * rows * D)


def _exact_diff(s):
    case = s["case"]
    B, N, keys, H, d = (case[n] for n in ("B", "N", "keys", "H", "d"))
    m = d // 2
    names = ("q", "k", "v", "gate", "lam")
    x = {n: s[n].double() for n in names}
    lens = [keys] * B if s["key_lens"] is None else s["key_lens"].tolist()
    out = torch.zeros(B, N, H * d, dtype=torch.float64, device="cuda")
    grads = {"d" + n: torch.zeros_like(x[n]) for n in names} if case["train"] else {}
    for b in range(B):
        for h in range(H if lens[b] else 0):
            c, n = slice(h * d, (h + 1) * d), lens[b]
            lam_at = (h,) if case["lam"] == "head" else (b, slice(None), h)
            leaf = [x["q"][b, :, c], x["k"][b, :n, c], x["v"][b, :n, c], x["gate"][b, :, c], x["lam"][lam_at]]
            leaf = [t.clone().requires_grad_(case["train"]) for t in leaf]
            q, k, v, gate, lam = leaf
            if case["lam"] == "token":
                lam = (1 / (1 + torch.exp(-lam)))[:, None]
            maps = []
            for i in (slice(0, m), slice(m, d)):
                z = q[:, i] @ k[:, i].T / math.sqrt(m)
                maps.append(torch.exp(z - torch.logsumexp(z, 1, keepdim=True)))
            y = (maps[0] @ v - lam * (maps[1] @ v)) / (1 + torch.exp(-gate))
            out[b, :, c] = y.detach()
            if case["train"]:
                found = torch.autograd.grad(y, leaf, s["dout"][b, :, c].double())
                for name, at, gr in zip(names, ((b, slice(None), c), (b, slice(n), c), (b, slice(n), c),
                                                (b, slice(None), c), lam_at), found):
                    grads["d" + name][at] += gr
            del maps, y
    return dict(out=out, **grads)


def _exact_norm(s):
    case = s["case"]
    leaf = {n: s[n].double().requires_grad_(case["train"])
            for n in ("h", "o", "w_post", "gate", "w_pre", "scale", "shift") if s[n] is not None}

    def norm(x):
        y = x - x.mean(-1, keepdim=True) if case["kind"] == "layer" else x
        return y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + EPS)

    h, res, ends = leaf["h"], {}, []
    if case["post"]:
        branch = norm(leaf["o"]) * leaf["w_post"]
        if case["mod"]:
            branch = branch * leaf["gate"].unsqueeze(1)
        h = h * s["res_scale"] + branch
        res["h_out"] = h
    if case["train"]:
        ends.append((h * s["dh_out"].double()).sum())
    if case["pre"]:
        u = norm(h) * leaf["w_pre"]
        if case["mod"]:
            u = u * (1 + leaf["scale"].unsqueeze(1)) + leaf["shift"].unsqueeze(1)
        res["u"] = u
        if case["train"]:
            ends.append((u * s["du"].double()).sum())
    if case["train"]:
        found = torch.autograd.grad(sum(ends), list(leaf.values()))
        res.update(("d" + n, gr) for n, gr in zip(leaf, found))
    return {n: t.detach() for n, t in res.items()}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_diff(s) if case["op"] == "diff" else _exact_norm(s)
