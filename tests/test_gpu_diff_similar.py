"""The differential anchor where its two maps resemble each other and lambda is near 1, so that the
result is a small difference of two outputs.

bf16: each map's weights P are rounded to bf16 on their own for the product with V, so the error is
one of O_1 and of lambda O_2, not of their difference A. Element by element a weight is off by 2^-8
of itself at most, hence A by 2^-8 (sum P_1 |V| + |lambda| sum P_2 |V|), and the result is rounded
once more, 2^-8 |out|; fp32 sums and exponentials add less than 2^-17 of the same sums. Values of V
that are independent of the weights turn a rounding that is uniform over half a step, 2^-8 / sqrt(3)
rms at most, into the same share of the 2-norms of O_1, lambda O_2 and out. dgate is made of the
same A. Everything else is made of each map's own weights, recomputed in fp32, and is held to the
library's bounds. fp32: 1e-5 in the place of 2^-8 / sqrt(3), and dv's W = P_1 - lambda P_2 cancels
too, in fp32: 1e-5 of its parts."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import softmax_attention_video_gated_b200 as sva  # noqa: E402

TDT = {"bf16": torch.bfloat16, "f32": torch.float32}
H, d = 2, 128
D = H * d


def inputs(N, keys, dtype, near, seed):
    """q and k whose second halves are the first ones and `near` times something else."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = dict(q=r(1, N, D), k=r(1, keys, D), v=r(1, keys, D), gate=r(1, N, D), dout=r(1, N, D))
    for n in "qk":
        x = t[n].view(1, -1, H, 2, d // 2)
        x[:, :, :, 1] = x[:, :, :, 0] + near * x[:, :, :, 1]
    return {n: x.to(TDT[dtype]) for n, x in t.items()}


def exact(t, lam):
    """In 64 bits: out, dgate, dq, dk, dv, dlam, the gated O_1 and lambda O_2, the same with |V|, and
    dv's parts P_1^T dA and lambda P_2^T dA."""
    x = {n: y.double()[0].view(-1, H, d) for n, y in t.items()}
    r = {n: torch.zeros_like(x["k" if n in ("dk", "dv", "dv1", "dv2") else "q"]) for n in
         ("out", "dgate", "dq", "dk", "dv", "o1", "o2", "a1", "a2", "dv1", "dv2")}
    r["dlam"] = torch.zeros(H, dtype=torch.float64, device="cuda")
    for h in range(H):
        q, k, v, dout = (x[n][:, h] for n in ("q", "k", "v", "dout"))
        s = torch.sigmoid(x["gate"][:, h])
        P = [torch.softmax(q[:, c] @ k[:, c].T / 8, 1) for c in (slice(0, 64), slice(64, 128))]
        o = [p @ v for p in P]
        a, da = o[0] - lam * o[1], dout * s
        r["out"][:, h], r["dgate"][:, h] = a * s, da * a * (1 - s)
        r["o1"][:, h], r["o2"][:, h] = s * o[0], s * lam * o[1]
        r["a1"][:, h], r["a2"][:, h] = s * (P[0] @ v.abs()), s * lam * (P[1] @ v.abs())
        r["dv1"][:, h], r["dv2"][:, h] = P[0].T @ da, lam * (P[1].T @ da)
        r["dv"][:, h] = r["dv1"][:, h] - r["dv2"][:, h]
        r["dlam"][h] = -(da * o[1]).sum()
        dp = da @ v.T
        for c, p, w in ((slice(0, 64), P[0], 1.0), (slice(64, 128), P[1], -lam)):
            ds = w * p * (dp - (p * dp).sum(1, keepdim=True))
            r["dq"][:, h, c], r["dk"][:, h, c] = ds @ k[:, c] / 8, ds.T @ q[:, c] / 8
    return r


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,keys", [(500, 500), (1100, 3000), (2, 700)])
@pytest.mark.parametrize("near", [0.1, 0.03])
@pytest.mark.parametrize("lam", [0.949, 1.0])
def test_similar_maps(dtype, N, keys, near, lam):
    t = inputs(N, keys, dtype, near, N + keys)
    lam_t = torch.full((H,), lam, device="cuda").to(TDT[dtype])
    lam = float(lam_t[0])
    saved = tuple(torch.empty(1, N, D, device="cuda") for _ in range(2)) + \
        (torch.empty(2, 1, H, N, device="cuda"),)
    got = {"out": torch.empty_like(t["q"])}
    more = dict(flags=sva.SVA_FLAG_LAMBDA_VALUE)
    sva.sva_diff_anchor_fwd(t["q"], t["k"], t["v"], t["gate"], lam_t, got["out"], H, saved=saved, **more)
    for n, like in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dgate", "gate")):
        got[n] = torch.empty_like(t[like])
    dlam = torch.empty_like(lam_t)
    sva.sva_diff_anchor_bwd(t["q"], t["k"], t["v"], t["gate"], lam_t, t["dout"], saved, got["dq"], got["dk"],
                            got["dv"], got["dgate"], dlam, H, **more)
    ref = exact(t, lam)
    got = {n: x.double()[0].view(-1, H, d) for n, x in got.items()}
    norm = lambda *names: sum(float(ref[n].norm()) for n in names)  # noqa: E731
    err = {n: float((x - ref[n]).norm()) for n, x in got.items()}
    unit = 2.0 ** -8 / math.sqrt(3) if dtype == "bf16" else 1e-5
    assert err["out"] <= unit * norm("o1", "o2", "out"), err["out"] / norm("out")
    slope = (t["dout"].double()[0].view(-1, H, d) * torch.sigmoid(-t["gate"].double()[0].view(-1, H, d))).abs()
    parts = sum(float((slope * ref[n]).norm()) for n in ("o1", "o2"))
    assert err["dgate"] <= unit * (parts + norm("dgate")), err["dgate"] / norm("dgate")
    if dtype == "bf16":
        bound = 2.0 ** -8 * (ref["a1"] + ref["a2"] + ref["out"].abs()) * (1 + 2.0 ** -8)
        assert ((got["out"] - ref["out"]).abs() <= bound).all()
    library = 1e-2 if dtype == "bf16" else 1e-5
    for n in ("dq", "dk"):
        assert err[n] <= library * norm(n), (n, err[n] / norm(n))
    assert err["dv"] <= (library * norm("dv") if dtype == "bf16" else library * norm("dv1", "dv2")), err["dv"]
    assert float((dlam.double() - ref["dlam"]).norm()) <= library * norm("dlam")
