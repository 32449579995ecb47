"""The block norms, forward and backward, against the fp64 oracle: widths of every
launch shape and odd ones, one token, missing parts, aliased buffers, and the
run of a whole layer (norm, projection, differential anchor, projection with
norm, gate and residual), forward and backward.

Tolerances: fp32 results rel-L2 <= 1e-5; bf16 results carry one rounding, half a
step or 2^-8 relative at most, rms 2^-8 / sqrt(3): rel-L2 <= 1e-2 leaves room for
nothing else of that size."""
import math

import numpy as np
import pytest

import oracle as O
import workloads as W
from oracle import differential as OD
from tests._util import assert_close, rel_l2, to_dev, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import softmax_attention_video_gated_b200 as sva  # noqa: E402

F32_OUT = ("h_out", "dh", "dw_post", "dgate", "dw_pre", "dscale", "dshift")
SUMS = {"dw_post": 0, "dgate": 1, "dw_pre": 0, "dscale": 1, "dshift": 1}


def make(B, N, D, dtype, seed, part="both", mod=True, weights=True, mean=0.0):
    rng = np.random.default_rng(seed)

    def r(*s, dt=dtype, scale=1.0, at=0.0):
        return W.round_to((rng.standard_normal(s) * scale + at).astype(np.float32), dt)

    x = dict(h=r(B, N, D, dt="f32", scale=2.0, at=mean), dh_out=r(B, N, D, dt="f32"))
    if part != "pre":
        x["o"] = r(B, N, D, scale=0.5, at=mean)
        if weights:
            x["w_post"] = r(D, at=1.0, scale=0.2)
        if mod:
            x["gate"] = r(B, D)
    if part != "post":
        x["du"] = r(B, N, D)
        if weights:
            x["w_pre"] = r(D, at=1.0, scale=0.2)
        if mod:
            x["scale"], x["shift"] = r(B, D, scale=0.3), r(B, D, scale=0.3)
    return x


def padded(t, fill=None):
    """The same values as a slice of a buffer whose rows are padded to 8 elements and 8 more."""
    w = (t.shape[-1] + 7) // 8 * 8 + 8
    buf = torch.full((*t.shape[:-1], w), 7.0, device="cuda", dtype=t.dtype)
    s = buf[..., :t.shape[-1]]
    s.copy_(t) if fill is None else s.fill_(fill)
    return s


def call(x, dtype, kind, eps, res_scale):
    t = {n: to_dev(v, "f32" if n in ("h", "dh_out") else dtype) for n, v in x.items()}
    t = {n: v if v.dim() == 1 else padded(v) for n, v in t.items()}
    B, N, D = t["h"].shape
    nan = float("nan")
    post, pre = "o" in t, "du" in t
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    r = {}
    if post:
        r["h_out"] = padded(t["h"], nan)
    if pre:
        r["u"] = padded(t["du"], nan)
    stats = torch.full((B, N, 4), nan, device="cuda")
    more = {n: t.get(n) for n in ("w_post", "gate", "w_pre", "scale")}
    more |= dict(kind=kind, eps=eps, res_scale=res_scale)
    sva.sva_block_norm_fwd(t["h"], o=t.get("o"), h_out=r.get("h_out"), u=r.get("u"),
                           shift=t.get("shift"), stats=stats, **more)
    plain = {n: torch.full_like(v, nan) for n, v in r.items()}
    if D % 8 == 0:  # without stats: the same bits
        sva.sva_block_norm_fwd(t["h"], o=t.get("o"), h_out=plain.get("h_out"), u=plain.get("u"),
                               shift=t.get("shift"), **more)
        assert all(torch.equal(plain[n], r[n]) for n in r)
    r["dh"] = padded(t["h"], nan)
    if post:
        r["do"] = padded(t["o"], nan)
    for n, per_batch in SUMS.items():
        if n in ("dw_post", "dgate") and post or n in ("dw_pre", "dscale", "dshift") and pre:
            r[n] = torch.full((B, D) if per_batch else (D,), nan, device="cuda")
    bwd = lambda: sva.sva_block_norm_bwd(  # noqa: E731
        r["h_out"] if post else t["h"], stats, r["dh"], dh_out=t.get("dh_out"), o=t.get("o"),
        do=r.get("do"), du=t.get("du"), **{n: r.get(n) for n in SUMS}, **more)
    ws = bwd()
    assert sva.sva_check_device_status(ws) == sva.SVA_OK
    first = {n: v.clone() for n, v in r.items()}
    bwd()
    assert all(torch.equal(first[n], r[n]) for n in r)       # no atomics: the same bits
    for n, v in r.items():                                   # rows' padding is left as it was
        if v.dim() == 3:
            assert torch.all(v.as_strided((B, N, v.stride(1)), (N * v.stride(1), v.stride(1), 1))[..., D:] == 7), n
    assert tdt == (r["u"] if pre else r["do"]).dtype
    return r


def compare(x, dtype, kind=sva.SVA_NORM_RMS, eps=1e-6, res_scale=1.0):
    r = call(x, dtype, kind, eps, res_scale)
    ref = OD.block_norm(**{n: v for n, v in x.items()}, pre="du" in x, layer=kind == sva.SVA_NORM_LAYER,
                        eps=eps, res_scale=res_scale)
    for n, v in r.items():
        assert_close(to_host(v), ref[n], "f32" if n in F32_OUT else dtype, n)


KINDS = [sva.SVA_NORM_RMS, sva.SVA_NORM_LAYER]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,N,D", [(1, 1, 64), (2, 3, 8), (1, 700, 256), (3, 129, 264), (2, 50, 1000),
                                   (1, 40, 1024), (2, 33, 2048), (1, 9, 4096), (1, 7, 4104), (1, 5, 8192),
                                   (2, 31, 101), (5, 1, 2049), (1, 17, 8191), (2, 4000, 130)])
def test_against_oracle(dtype, kind, B, N, D):
    compare(make(B, N, D, dtype, N + D), dtype, kind)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("part", ["pre", "post"])
@pytest.mark.parametrize("mod, weights", [(True, False), (False, True), (False, False)])
def test_parts(dtype, kind, part, mod, weights):
    compare(make(2, 77, 520, dtype, 3, part, mod, weights), dtype, kind, res_scale=0.5, eps=1e-5)


@pytest.mark.parametrize("kind", KINDS)
def test_one_channel_and_constant_rows(kind):
    # a layer norm of one channel, or of equal channels, is zero whatever the value; eps keeps it finite
    x = make(1, 6, 1, "f32", 8)
    x["h"][:] = 3.0
    x["o"][:] = -2.0
    r = call(x, "f32", kind, 1e-6, 1.0)
    ref = OD.block_norm(**x, layer=kind == sva.SVA_NORM_LAYER, eps=1e-6)
    for n in ("h_out", "u", "dshift"):
        np.testing.assert_allclose(to_host(r[n]), ref[n], rtol=1e-6, atol=1e-6)


def test_layer_norm_far_from_zero():
    # a mean of 300 deviations: the two-step variance keeps the row's own digits. x - mean is exact to
    # half an ulp of x, 300 * 2^-24 = 2e-5 deviations, the same for every value of the row's mean
    x = make(1, 64, 2048, "f32", 4, part="pre", mean=600.0)
    r = call(x, "f32", sva.SVA_NORM_LAYER, 1e-6, 1.0)
    ref = OD.block_norm(**x, layer=True)
    assert rel_l2(to_host(r["u"]), ref["u"]) < 4e-5


def test_no_upstream_gradient_and_aliases():
    # dh_out missing counts as zero; h_out over h, dh over dh_out and do over o give the same values
    B, N, D = 2, 50, 512
    x = make(B, N, D, "bf16", 6)
    t = {n: to_dev(v, "f32" if n in ("h", "dh_out") else "bf16") for n, v in x.items()}
    more = {n: t[n] for n in ("w_post", "gate", "w_pre", "scale")}
    h, u, stats = t["h"].clone(), torch.empty_like(t["o"]), torch.empty(B, N, 4, device="cuda")
    sva.sva_block_norm_fwd(h, o=t["o"], h_out=h, u=u, shift=t["shift"], stats=stats, **more)
    ref = OD.block_norm(**x)
    assert_close(to_host(h), ref["h_out"], "f32", "h_out")
    dh, do = t["dh_out"].clone(), t["o"].clone()
    sva.sva_block_norm_bwd(h, stats, dh, dh_out=dh, o=do, do=do, du=t["du"], **more)
    assert_close(to_host(dh), ref["dh"], "f32", "dh")
    assert_close(to_host(do), ref["do"], "bf16", "do")
    sva.sva_block_norm_bwd(h, stats, dh, o=t["o"], do=do, du=t["du"], **more)
    zero = OD.block_norm(**{**x, "dh_out": np.zeros_like(x["dh_out"])})
    assert_close(to_host(dh), zero["dh"], "f32", "dh without dh_out")


def test_offsets_past_32_bits():
    # a tensor of more than 2^31 values, zero but for its last rows: those rows, and the sums over all
    N, D, last = 300_000, 8192, 40
    assert (N - last) * D > 2 ** 31
    torch.manual_seed(5)
    h = torch.zeros(1, N, D, device="cuda")
    o = torch.zeros(1, N, D, device="cuda", dtype=torch.bfloat16)
    h[:, -last:].normal_()
    o[:, -last:].normal_()
    h_tail, o_tail = to_host(h[:, -last:]), to_host(o[:, -last:])
    u, stats = torch.empty_like(o), torch.empty(1, N, 4, device="cuda")
    sva.sva_block_norm_fwd(h, o=o, h_out=h, u=u, stats=stats)
    du_tail = to_host(u[:, -last:])                       # u, zero but for its last rows, stands for du
    ref = OD.block_norm(h_tail, o=o_tail, dh_out=np.zeros_like(h_tail), du=du_tail)
    assert_close(to_host(h[:, -last:]), ref["h_out"], "f32", "h_out")
    assert_close(du_tail, ref["u"], "bf16", "u")
    assert not u[:, :-last].any()
    dh, do, dw = torch.empty_like(h), torch.empty_like(o), torch.empty(D, device="cuda")
    sva.sva_block_norm_bwd(h, stats, dh, o=o, do=do, du=u, dw_pre=dw)
    # dh of u itself: u . h'^ is nearly its own length, so dh and do cancel to a share of du and are
    # held to it; dw_pre is a sum without cancellation
    for n, got in (("dh", dh), ("do", do)):
        e = np.abs(to_host(got[:, -last:]) - ref[n]).max()
        assert e <= 2.0 ** -8 * np.abs(du_tail).max(), (n, e)
    assert_close(to_host(dw), ref["dw_pre"], "f32", "dw_pre")
    assert not dh[:, :-last].any()


def test_capture_and_two_streams():
    xs = [make(2, 333, 1024, "bf16", 50 + i) for i in range(2)]
    want = [call(x, "bf16", sva.SVA_NORM_LAYER, 1e-6, 0.9) for x in xs]
    ts = [{n: to_dev(v, "f32" if n in ("h", "dh_out") else "bf16") for n, v in x.items()} for x in xs]

    def buffers(t):
        B, N, D = t["h"].shape
        r = dict(h_out=torch.empty_like(t["h"]), u=torch.empty_like(t["o"]), dh=torch.empty_like(t["h"]),
                 do=torch.empty_like(t["o"]), stats=torch.empty(B, N, 4, device="cuda"),
                 ws=sva.workspace(sva.sva_block_norm_bwd_workspace_bytes(B, N, D)))
        return r | {n: torch.empty((B, D) if b else (D,), device="cuda") for n, b in SUMS.items()}

    def step(t, r):
        more = {n: t[n] for n in ("w_post", "gate", "w_pre", "scale")}
        more |= dict(kind=sva.SVA_NORM_LAYER, res_scale=0.9)
        sva.sva_block_norm_fwd(t["h"], o=t["o"], h_out=r["h_out"], u=r["u"], shift=t["shift"],
                               stats=r["stats"], **more)
        sva.sva_block_norm_bwd(r["h_out"], r["stats"], r["dh"], dh_out=t["dh_out"], o=t["o"], do=r["do"],
                               du=t["du"], ws=r["ws"], **{n: r[n] for n in SUMS}, **more)

    rs, streams = [buffers(t) for t in ts], [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    for t, r, s in zip(ts, rs, streams):
        with torch.cuda.stream(s):
            step(t, r)
    torch.cuda.synchronize()
    for r, w in zip(rs, want):
        assert all(torch.equal(r[n], w[n]) for n in w)
    t, r = {n: v.clone() for n, v in ts[0].items()}, buffers(ts[0])
    step(t, r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(t, r)
    for i in (1, 0):
        for n in t:
            t[n].copy_(ts[i][n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(r[n], want[i][n]) for n in want[i])


def test_python_refusals():
    h = torch.zeros(1, 4, 64, device="cuda")
    o = torch.zeros(1, 4, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sva.sva_block_norm_fwd(h)
    with pytest.raises(TypeError):
        sva.sva_block_norm_fwd(h.bfloat16(), u=o)
    with pytest.raises(TypeError):
        sva.sva_block_norm_fwd(h, u=o, w_pre=torch.ones(64, device="cuda"))
    with pytest.raises(ValueError):
        sva.sva_block_norm_fwd(h, u=o, scale=torch.ones(2, 64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(sva.SvaError):
        sva.sva_block_norm_fwd(h, o=o)                  # no h_out


# ------------------------------------------------------------------ a layer as it is used

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_forward_and_backward(dtype):
    """u = norm(h); [Q|K|V|G|lambda] = u W^T; y = differential anchor; o = y W_o^T;
    h' = h + gate norm(o): one layer through the library's calls, then its backward pass."""
    B, N, H, d = 2, 150, 2, 128
    D = H * d
    W_in = 4 * D + 64
    rng = np.random.default_rng(77)
    r = lambda *s, scale=1.0, at=0.0, dt=dtype: W.round_to(  # noqa: E731
        (rng.standard_normal(s) * scale + at).astype(np.float32), dt)
    h, w_in, w_o = r(B, N, D, dt="f32"), r(W_in, D, scale=1 / math.sqrt(D)), r(D, D, scale=1 / math.sqrt(D))
    w_pre, w_post, scale, shift, gate = (r(D, at=1.0, scale=0.1), r(D, at=1.0, scale=0.1),
                                         r(B, D, scale=0.3), r(B, D, scale=0.3), r(B, D))
    dh_out = r(B, N, D, dt="f32")
    lens = [N, 97]
    t = {n: to_dev(v, "f32" if n in ("h", "dh_out") else dtype) for n, v in dict(
        h=h, w_in=w_in, w_o=w_o, w_pre=w_pre, w_post=w_post, scale=scale, shift=shift, gate=gate,
        dh_out=dh_out).items()}
    tdt = t["w_in"].dtype
    new = lambda *s, dt=tdt: torch.empty(*s, device="cuda", dtype=dt)  # noqa: E731
    f32 = torch.float32
    kl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cuts = [(i * D, (i + 1) * D) for i in range(4)] + [(4 * D, 4 * D + H)]

    u, st1 = new(B, N, D), new(B, N, 4, dt=f32)
    sva.sva_block_norm_fwd(t["h"], u=u, w_pre=t["w_pre"], scale=t["scale"], shift=t["shift"], stats=st1)
    fused = new(B, N, W_in)
    sva.sva_projection_fwd(u.view(-1, D), t["w_in"], fused.view(-1, W_in))
    q, k, v, g, lam = (fused[..., a:b] for a, b in cuts)
    y, saved = new(B, N, D), (new(B, N, D, dt=f32), new(B, N, D, dt=f32), new(2, B, H, N, dt=f32))
    sva.sva_diff_anchor_fwd(q, k, v, g, lam, y, H, key_lens=kl, saved=saved)
    o = new(B, N, D)
    sva.sva_projection_fwd(y.view(-1, D), t["w_o"], o.view(-1, D))
    hp, st2 = new(B, N, D, dt=f32), new(B, N, 4, dt=f32)
    sva.sva_block_norm_fwd(t["h"], o=o, h_out=hp, w_post=t["w_post"], gate=t["gate"], stats=st2)
    # backward: the norm behind the block, W_o, the anchor, W_in, the norm before it
    dres, do, dw_post, dgate = new(B, N, D, dt=f32), new(B, N, D), new(D, dt=f32), new(B, D, dt=f32)
    sva.sva_block_norm_bwd(hp, st2, dres, dh_out=t["dh_out"], o=o, do=do, w_post=t["w_post"],
                           gate=t["gate"], dw_post=dw_post, dgate=dgate)
    dy = new(B, N, D)
    sva.sva_projection_fwd(do.view(-1, D), t["w_o"].t().contiguous(), dy.view(-1, D))
    dfused = torch.zeros(B, N, W_in, device="cuda", dtype=tdt)
    sva.sva_diff_anchor_bwd(q, k, v, g, lam, dy, saved, *(dfused[..., a:b] for a, b in cuts), H, key_lens=kl)
    du = new(B, N, D)
    sva.sva_projection_fwd(dfused.view(-1, W_in), t["w_in"].t().contiguous(), du.view(-1, D))
    dh, dw_pre, dscale, dshift = new(B, N, D, dt=f32), new(D, dt=f32), new(B, D, dt=f32), new(B, D, dt=f32)
    ws = sva.sva_block_norm_bwd(t["h"], st1, dh, dh_out=dres, du=du, w_pre=t["w_pre"], scale=t["scale"],
                                dw_pre=dw_pre, dscale=dscale, dshift=dshift)
    assert sva.sva_check_device_status(ws) == sva.SVA_OK

    # the oracle's layer on the same inputs, without the intermediate roundings
    pre = OD.block_norm(h, w_pre=w_pre, scale=scale, shift=shift)
    F = O.project(pre["u"].reshape(-1, D), w_in).reshape(B, N, W_in)
    part = [F[..., a:b] for a, b in cuts]
    Y = OD.diff_anchor(*part, H, key_lens=lens)["out"]
    Oo = O.project(Y.reshape(-1, D), w_o).reshape(B, N, D)
    post = OD.block_norm(h, o=Oo, w_post=w_post, gate=gate, pre=False, dh_out=dh_out)
    dY = post["do"] @ w_o.astype(np.float64)
    ga = OD.diff_anchor(*part, H, key_lens=lens, dout=dY)
    dF = np.concatenate([ga[n] for n in ("dq", "dk", "dv", "dgate", "dlam")], axis=2) @ \
        w_in[:4 * D + H].astype(np.float64)
    end = OD.block_norm(h, w_pre=w_pre, scale=scale, shift=shift, dh_out=post["dh"], du=dF)
    # fp32: a chain of five steps, 1e-5 each; bf16: six roundings of intermediate tensors (u, the
    # projection, y, o, and backward do, dy, dfused, du) beside the anchor's own, 2^-9 rms each,
    # and the norms divide by the small spread of o, so 3e-2 where one step is held to 1e-2
    tol = 3e-2 if dtype == "bf16" else 5e-5
    for n, got, ref in (("u", u, pre["u"]), ("y", y, Y), ("o", o, Oo), ("h'", hp, post["h_out"]),
                        ("do", do, post["do"]), ("dgate", dgate, post["dgate"]),
                        ("dw_post", dw_post, post["dw_post"]), ("dfused q", dfused[..., :D], ga["dq"]),
                        ("du", du, dF), ("dh", dh, end["dh"]), ("dw_pre", dw_pre, end["dw_pre"]),
                        ("dscale", dscale, end["dscale"]), ("dshift", dshift, end["dshift"])):
        e = rel_l2(to_host(got), ref)
        assert e <= tol, f"{n}: rel-L2 {e:.2e} > {tol}"
