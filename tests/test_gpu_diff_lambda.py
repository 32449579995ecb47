"""The gradient of the differential anchor's lambda where its sums cancel: a lambda shared by all
tokens, few heads, many seeds; single heads of a few tokens.

dlambda_t = -sum_c dA_c O_2c, and a shared lambda's gradient adds up the tokens: sums of terms of
both signs, so their errors are measured against the terms, T = (sum_t sum_c (dA_c O_2c)^2)^(1/2)
over a head. A bf16 result is off by its own rounding, 2^-8 of it at most, and by what the terms
bring: O_2 and dA are each off by 2^-8 at most where they were rounded, and only the product of the
two errors is left, 2^-16 of a term, of random sign over terms, so its sum is off by 2^-16 T in the
mean and 4 * 2^-16 T = 2^-14 T bounds it. fp32: the library's bound of 1e-5 on the terms."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import softmax_attention_video_gated_b200 as sva  # noqa: E402

TDT = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(B, N, keys, H, dtype, seed, shared, lens=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(TDT[dtype])  # noqa: E731
    D = H * 128
    t = dict(q=r(B, N, D), k=r(B, keys, D), v=r(B, keys, D), g=r(B, N, D), dout=r(B, N, D),
             lam=r(H) if shared else r(B, N, H))
    t["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    return t


def dlam_of(t, H, flags):
    B, N, _ = t["q"].shape
    saved = tuple(torch.empty_like(t["q"], dtype=torch.float32) for _ in range(2)) + \
        (torch.empty(2, B, H, N, device="cuda"),)
    more = dict(key_lens=t["lens"], flags=flags)
    sva.sva_diff_anchor_fwd(t["q"], t["k"], t["v"], t["g"], t["lam"], torch.empty_like(t["q"]), H,
                            saved=saved, **more)
    g = {n: torch.empty_like(t[n]) for n in ("q", "k", "v", "g")}
    got = []
    for _ in range(2):
        dlam = torch.full_like(t["lam"], float("nan"))
        ws = sva.sva_diff_anchor_bwd(t["q"], t["k"], t["v"], t["g"], t["lam"], t["dout"], saved, g["q"],
                                     g["k"], g["v"], g["g"], dlam, H, **more)
        got.append(dlam)
    assert sva.sva_check_device_status(ws) == sva.SVA_OK
    assert torch.equal(*got)  # the same bits
    return got[0].double()


def exact(t, H, flags):
    """(dlambda, T) in 64 bits: [H] each for a shared lambda, else dlambda [B, N, H] and T [B, N, H]"""
    B, N, _ = t["q"].shape
    keys = t["k"].shape[1]
    ref = torch.zeros(B, N, H, device="cuda", dtype=torch.float64)
    terms = torch.zeros_like(ref)
    for b in range(B):
        n = keys if t["lens"] is None else int(t["lens"][b])
        for h in range(H if n else 0):
            c = slice(h * 128, (h + 1) * 128)
            half = slice(h * 128 + 64, (h + 1) * 128)
            z = t["q"][b, :, half].double() @ t["k"][b, :n, half].double().T / 8
            o2 = torch.softmax(z, 1) @ t["v"][b, :n, c].double()
            each = t["dout"][b, :, c].double() * torch.sigmoid(t["g"][b, :, c].double()) * o2
            ref[b, :, h], terms[b, :, h] = -each.sum(1), each.square().sum(1)
    if t["lam"].ndim == 1:
        ref, terms = ref.sum((0, 1)), terms.sum((0, 1))
    if not flags:
        s = torch.sigmoid(t["lam"].double()) * torch.sigmoid(-t["lam"].double())
        ref, terms = ref * s, terms * s.square()
    return ref, terms.sqrt()


def assert_within(t, H, dtype, flags):
    got, (ref, terms) = dlam_of(t, H, flags), exact(t, H, flags)
    bound = 2.0 ** -8 * ref.abs() + 2.0 ** -14 * terms if dtype == "bf16" else 1e-5 * terms
    over = (got - ref).abs() - bound
    assert float(over.max()) <= 0, (float((got - ref).abs().max()), float(ref.abs().min()))
    return float((got - ref).norm() / ref.norm())


VALUE = sva.SVA_FLAG_LAMBDA_VALUE


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("flags", [0, VALUE])
@pytest.mark.parametrize("B,N,keys,H,lens", [
    (1, 200, 200, 1, None), (1, 1000, 1000, 1, None), (2, 1000, 1000, 2, [1000, 613]),
    (1, 2000, 2000, 2, None), (3, 453, 453, 1, [453, 0, 301]), (1, 3000, 70, 1, None),
    (1, 40, 6000, 1, None), (2, 40, 6000, 2, [5999, 65]), (4, 3, 500, 1, None)])
def test_shared_lambda_over_many_seeds(dtype, flags, B, N, keys, H, lens):
    rel = [assert_within(inputs(B, N, keys, H, dtype, 100 + s, True, lens), H, dtype, flags)
           for s in range(10)]
    if dtype == "bf16":
        assert np.median(rel) <= 2.0 ** -8, rel


@pytest.mark.parametrize("flags", [0, VALUE])
@pytest.mark.parametrize("H", [1, 2])
def test_shared_lambda_of_a_long_clip(flags, H):
    rel = [assert_within(inputs(1, 9000, 9000, H, "bf16", 200 + s, True), H, "bf16", flags)
           for s in range(10)]
    assert np.median(rel) <= 2.0 ** -8, rel


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("flags", [0, VALUE])
@pytest.mark.parametrize("B,N,keys,H,lens", [(1, 5, 300, 1, None), (1, 70, 200, 2, None),
                                             (2, 33, 5000, 1, [4999, 70])])
def test_lambda_per_token_over_many_seeds(dtype, flags, B, N, keys, H, lens):
    for s in range(10):
        assert_within(inputs(B, N, keys, H, dtype, 300 + s, False, lens), H, dtype, flags)


def test_shared_lambda_of_zero_as_a_value():
    # the second map takes no part, its gradient is still the map's
    t = inputs(1, 300, 400, 2, "bf16", 7, True)
    t["lam"][0] = 0.0
    assert_within(t, 2, "bf16", VALUE)
    t["lam"][1] = -0.0
    assert_within(t, 2, "bf16", VALUE)
    assert math.isfinite(float(dlam_of(t, 2, VALUE).sum()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("logit", [9.0, 15.0, -15.0, 40.0, -40.0])
@pytest.mark.parametrize("N", [2, 130])
def test_gates_and_lambdas_far_from_zero(dtype, shared, logit, N):
    # s (1 - s) keeps its digits where the sigmoid s is next to 1: the library's bounds, of gradients
    # that are all of one size
    H = 2
    t = inputs(1, N, 150, H, dtype, 17, shared)
    t["g"].fill_(logit)
    t["lam"].fill_(logit)
    for flags in (0, VALUE):
        lam = t["lam"] if not flags else torch.full_like(t["lam"], 0.8)
        assert_within({**t, "lam": lam}, H, dtype, flags)
    saved = tuple(torch.empty(1, N, H * 128, device="cuda") for _ in range(2)) + \
        (torch.empty(2, 1, H, N, device="cuda"),)
    sva.sva_diff_anchor_fwd(t["q"], t["k"], t["v"], t["g"], t["lam"], torch.empty_like(t["q"]), H, saved=saved)
    g = [torch.empty_like(t[n]) for n in ("q", "k", "v", "g", "lam")]
    sva.sva_diff_anchor_bwd(t["q"], t["k"], t["v"], t["g"], t["lam"], t["dout"], saved, *g, H)
    s, s1 = (torch.sigmoid(torch.tensor(x, dtype=torch.float64)) for x in (logit, -logit))
    ref = torch.empty(1, N, H, 128, device="cuda", dtype=torch.float64)
    for h in range(H):
        c = slice(h * 128, (h + 1) * 128)
        o = []
        for m in (0, 64):
            i = slice(h * 128 + m, h * 128 + m + 64)
            o.append(torch.softmax(t["q"][0, :, i].double() @ t["k"][0, :, i].double().T / 8, 1) @
                     t["v"][0, :, c].double())
        lam = (t["lam"][h] if shared else t["lam"][0, :, h, None]).double()
        ref[0, :, h] = t["dout"][0, :, c].double() * (o[0] - torch.sigmoid(lam) * o[1]) * (s * s1).item()
    ref = ref.reshape(1, N, -1)
    rel = float((g[3].double() - ref).norm() / ref.norm())
    assert rel <= (1e-2 if dtype == "bf16" else 1e-5), rel
