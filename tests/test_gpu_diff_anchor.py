"""The gated differential anchor, forward and backward, against the fp64 oracle:
lengths from one token, tile edges and odd sizes, padded batches with an empty
one, strided operands, both forms of lambda, and the ways a program calls it
(other streams, captured graphs, two calls at once).

Tolerances are the library's own: bf16 rel-L2 <= 1e-2 and max-abs <= 3e-2
max|ref|, fp32 rel-L2 <= 1e-5. A bf16 result carries its own rounding and those
of P (and, backward, of dA and dS): four roundings of at most half a step, 2^-8
relative each, independent over hundreds of summed terms, so 4 * 2^-8 / sqrt(3)
= 9e-3 bounds the relative L2 error even where all four are at their rms."""
import math

import numpy as np
import pytest

import workloads as W
from oracle import differential as OD
from tests._util import assert_close, to_dev, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import softmax_attention_video_gated_b200 as sva  # noqa: E402

TDT = {"bf16": torch.bfloat16, "f32": torch.float32}
GRADS = ("dq", "dk", "dv", "dgate", "dlam")


def make(B, N, keys, H, d, dtype, seed, shared=False, q_scale=1.0):
    rng = np.random.default_rng(seed)
    D = H * d
    shapes = dict(q=(B, N, D), k=(B, keys, D), v=(B, keys, D), g=(B, N, D),
                  lam=(H,) if shared else (B, N, H), dout=(B, N, D))
    x = {n: W.round_to(rng.standard_normal(s).astype(np.float32), dtype) for n, s in shapes.items()}
    x["q"] = W.round_to((x["q"] * q_scale).astype(np.float32), dtype)
    return x


def dev(x, dtype):
    return {n: to_dev(v, dtype) for n, v in x.items()}


def forward(t, H, saved=None, key_lens=None, flags=0, **kw):
    out = torch.full_like(t["q"], float("nan"))
    ws = sva.sva_diff_anchor_fwd(t["q"], t["k"], t["v"], t["g"], t["lam"], out, H, saved=saved,
                                 key_lens=key_lens, flags=flags, **kw)
    return out, ws


def new_saved(t, H):
    B, N, _ = t["q"].shape
    o = torch.full(t["q"].shape, float("nan"), device="cuda", dtype=torch.float32)
    return o, o.clone(), torch.full((2, B, H, N), float("nan"), device="cuda")


def backward(t, H, saved, key_lens=None, flags=0, **kw):
    g = {n: torch.full_like(t[s], float("nan")) if t[s] is not None else None
         for n, s in zip(GRADS, ("q", "k", "v", "g", "lam"))}
    ws = sva.sva_diff_anchor_bwd(t["q"], t["k"], t["v"], t["g"], t["lam"], t["dout"], saved,
                                 g["dq"], g["dk"], g["dv"], g["dgate"], g["dlam"], H,
                                 key_lens=key_lens, flags=flags, **kw)
    return g, ws


def oracle(x, H, **kw):
    return OD.diff_anchor(x["q"], x["k"], x["v"], x["g"], x["lam"], H, dout=x["dout"], **kw)


def cancelled(x, n, H, d):
    """Absolute error that dq or dk may carry where the result itself cancels (a map on one key:
    dS = P (dP - delta) = 0). dP and delta are sums of d products da v, each off by d 2^-24
    sum |da v| <= d 2^-24 |da| |v| at most (fp32 sums), and dS = 2 d 2^-24 |da| |v| P at most is
    multiplied by scale and a row of k or q and summed over the rows of weight P (sum over the keys
    at most 1; over the queries at most N)."""
    def longest(t):
        t = np.nan_to_num(np.asarray(t, np.float64), posinf=0.0)
        return np.sqrt((t.reshape(*t.shape[:2], H, d) ** 2).sum(-1)).max()
    other, rows = ("k", 1) if n == "dq" else ("q", x["q"].shape[1])
    lam = 1 + np.abs(x["lam"]).max()
    return 2 * d * 2.0 ** -24 * longest(x["dout"]) * longest(x["v"]) * lam * rows * \
        np.abs(x[other]).max() / math.sqrt(d / 2)


def assert_grad(got, x, ref, n, H, dtype):
    got = to_host(got)
    if n in ("dq", "dk") and np.abs(got - ref[n]).max() <= cancelled(x, n, H, x["q"].shape[2] // H):
        return
    assert_close(got, ref[n], dtype, n)


def compare(x, t, H, dtype, lens=None, flags=0, scale=0.0):
    kl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref = oracle(x, H, key_lens=lens, raw=bool(flags), scale=scale or None)
    saved = new_saved(t, H)
    out, ws = forward(t, H, saved, kl, flags, scale=scale)
    assert sva.sva_check_device_status(ws) == sva.SVA_OK
    plain, _ = forward(t, H, None, kl, flags, scale=scale)
    assert torch.equal(out, plain)                        # saving changes nothing
    assert_close(to_host(out), ref["out"], dtype, "out")
    for got, n in zip(saved, ("o1", "o2")):
        assert_close(to_host(got), ref[n], dtype, n)
    lse = to_host(saved[2])
    assert np.array_equal(np.isfinite(lse), np.isfinite(ref["lse"]))
    fin = np.isfinite(lse)
    # a sum of exponentials of fp32 dots: 1e-5 of the largest logit at hand
    assert np.abs(lse[fin] - ref["lse"][fin]).max(initial=0.0) <= 1e-5 * max(
        1.0, np.abs(ref["lse"][fin]).max(initial=0.0))
    g, ws = backward(t, H, saved, kl, flags, scale=scale)
    assert sva.sva_check_device_status(ws) == sva.SVA_OK
    for n in GRADS:
        if g[n] is not None:
            assert_grad(g[n], x, ref, n, H, dtype)
    again, _ = backward(t, H, saved, kl, flags, scale=scale)
    for n in GRADS:
        assert g[n] is None or torch.equal(g[n], again[n]), n   # no atomics: the same bits
    return ref


SHAPES = [
    # B, N, keys, H
    (1, 1, 1, 1),          # one token: both maps are 1, out = (1 - lambda) v
    (2, 1, 300, 2),        # one query against many keys
    (1, 1, 20000, 1),      # ... split over many CTAs
    (1, 300, 1, 2),        # one key
    (2, 2, 700, 2), (1, 4, 5000, 3), (1, 3, 33, 1), (3, 1, 4095, 1),  # a handful, cut over clusters
    (1, 64, 64, 1), (1, 128, 128, 2), (1, 65, 129, 3), (2, 127, 63, 2), (1, 256, 192, 1),
    (2, 257, 1000, 1), (3, 333, 333, 2), (1, 5, 4097, 2),
    (1, 3000, 70, 2), (2, 100, 9000, 1), (1, 2000, 2000, 1),  # few tiles, their streams cut over clusters
]


@pytest.mark.parametrize("dtype, d", [("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("B,N,keys,H", SHAPES)
def test_against_oracle(dtype, d, B, N, keys, H):
    x = make(B, N, keys, H, d, dtype, 7 * N + keys)
    compare(x, dev(x, dtype), H, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("flags", [0, sva.SVA_FLAG_LAMBDA_VALUE])
@pytest.mark.parametrize("shared", [False, True])
def test_lambda_forms(dtype, flags, shared):
    # as a value, lambda may be negative, zero or above one
    x = make(2, 150, 200, 3, 128, dtype, 5, shared=shared)
    x["lam"].ravel()[:2] = (0.0, -1.5)
    compare(x, dev(x, dtype), 3, dtype, flags=flags)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[200, 0, 1], [64, 65, 128], [129, 199, 63], [-5, 1000, 32]])
def test_padded_batch(dtype, lens):
    # a key count per batch: none, one, a tile's edge, below zero and past the end
    x = make(3, 140, 200, 2, 128, dtype, 9)
    t = dev(x, dtype)
    for b, n in enumerate(lens):                       # what lies behind counts for nothing
        t["k"][b, max(n, 0):] = float("nan")
        t["v"][b, max(n, 0):] = float("inf")
    ref = compare(x, t, 2, dtype, lens=lens)
    assert np.all(ref["dk"][0, max(lens[0], 0):] == 0)


@pytest.mark.parametrize("dtype, d", [("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("N", [1, 2, 4])
@pytest.mark.parametrize("lens", [[3000, 0, 1], [17, 2049, 2999], [-1, 9999, 8]])
def test_padded_batch_of_a_few_queries(dtype, d, N, lens):
    # key counts that leave some or all CTAs of a cluster without keys
    x = make(3, N, 3000, 2, d, dtype, 15)
    t = dev(x, dtype)
    for b, n in enumerate(lens):
        t["k"][b, max(n, 0):] = float("nan")
        t["v"][b, max(n, 0):] = float("inf")
    compare(x, t, 2, dtype, lens=lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[6000, 0, 700], [5999, 65, 3000]])
def test_padded_batch_of_cut_streams(dtype, lens):
    x = make(3, 40, 6000, 1, 128, dtype, 16)
    t = dev(x, dtype)
    for b, n in enumerate(lens):
        t["k"][b, n:] = float("nan")
        t["v"][b, n:] = float("inf")
    compare(x, t, 1, dtype, lens=lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_batch_is_zero(dtype):
    x = make(2, 40, 70, 1, 128, dtype, 3)
    t = dev(x, dtype)
    kl = torch.zeros(2, dtype=torch.int32, device="cuda")
    saved = new_saved(t, 1)
    out, _ = forward(t, 1, saved, kl)
    g, _ = backward(t, 1, saved, kl)
    assert all(float(v.float().abs().max()) == 0.0 for v in (out, *saved[:2], *g.values()))
    assert torch.all(saved[2] == -math.inf)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 3, 100])
def test_no_gate(dtype, N):
    x = make(1, N, 90, 2, 128, dtype, 4)
    x["g"] = None
    t = {n: None if v is None else to_dev(v, dtype) for n, v in x.items()}
    compare(x, t, 2, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [2, 70])
def test_given_scale(dtype, N):
    x = make(1, N, 130, 2, 128, dtype, 19)
    compare(x, dev(x, dtype), 2, dtype, scale=0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 40])
def test_offsets_past_32_bits(dtype, N):
    """Keys and values in rows so far apart that the last ones start behind 2^32 bytes and 2^31
    elements; all but the last 300 and the first 300 keys are far below in logit."""
    H, d, Nk = 1, 128, 1100
    ld = 1 << 21                                       # elements a row
    torch.manual_seed(3)
    dt = TDT[dtype]
    kv = torch.empty(1, Nk, ld, device="cuda", dtype=dt)
    k, v = kv[..., :d], kv[..., ld - d:]
    assert (Nk - 1) * ld > 2 ** 31
    x = make(1, N, Nk, H, d, dtype, 71)
    t = dev(x, dtype)
    k.copy_(t["k"])
    v.copy_(t["v"])
    out, _ = forward({**t, "k": k, "v": v}, H)
    saved = new_saved(t, H)
    near, _ = forward(t, H, saved)
    assert torch.equal(out, near)
    if N > 1:  # the gradients' rows as far apart
        dkv = torch.empty_like(kv)
        g, _ = backward(t, H, saved)
        far = {n: torch.empty_like(g[n]) for n in ("dq", "dgate", "dlam")}
        sva.sva_diff_anchor_bwd(t["q"], k, v, t["g"], t["lam"], t["dout"], saved, far["dq"],
                                dkv[..., :d], dkv[..., ld - d:], far["dgate"], far["dlam"], H)
        for n in far:
            assert torch.equal(far[n], g[n]), n
        assert torch.equal(dkv[..., :d], g["dk"]) and torch.equal(dkv[..., ld - d:], g["dv"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_scale", [0.0, 40.0])
def test_flat_and_peaked_maps(dtype, q_scale):
    # all logits equal; logits of several hundred, where one key takes all the weight and the
    # running maximum moves by more than its lazy threshold
    x = make(1, 130, 500, 1, 128, dtype, 6, q_scale=q_scale)
    t = dev(x, dtype)
    ref = oracle(x, 1)
    saved = new_saved(t, 1)
    out, _ = forward(t, 1, saved)
    g, _ = backward(t, 1, saved)
    if dtype == "f32" and q_scale > 1:
        # logits l of up to 40 * 4.5 * 8 / 8 in fp32: the exponents are off by l * 2^-22, here 4e-5
        for n, got in (("out", out), ("dv", g["dv"])):
            r = np.linalg.norm(to_host(got) - ref[n]) / np.linalg.norm(ref[n])
            assert r <= 2e-4, (n, r)
        return
    assert_close(to_host(out), ref["out"], dtype, "out")
    assert_close(to_host(g["dv"]), ref["dv"], dtype, "dv")
    if q_scale == 0.0:
        for n in ("dq", "dlam"):
            assert_close(to_host(g[n]), ref[n], dtype, n)
        assert float(g["dk"].abs().max()) == 0.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 8])
def test_nan_among_the_keys_is_not_lost(dtype, N):
    # a key that counts and is not a number leaves no finite result, wherever it stands in a block
    x = make(1, N, 160, 1, 128, dtype, 51)
    t = dev(x, dtype)
    for at in (0, 3, 6, 7, 70, 127, 128, 159):
        k = t["k"].clone()
        k[0, at] = float("nan")
        out, _ = forward({**t, "k": k}, 1)
        assert not torch.isfinite(out.float()).any(), at


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_wider_buffers(dtype):
    # q, k, v, gate, lambda and their gradients as column slices of one buffer, the result in
    # another's: what lies between is left as it was
    B, N, H, d = 2, 137, 2, 128
    D = H * d
    x = make(B, N, N, H, d, dtype, 12)
    cat = np.concatenate([x["q"], x["k"], x["v"], x["g"], x["lam"],
                          np.zeros((B, N, 14), np.float32)], axis=2)
    buf = to_dev(cat.astype(np.float32), dtype)
    cuts = dict(q=(0, D), k=(D, 2 * D), v=(2 * D, 3 * D), g=(3 * D, 4 * D), lam=(4 * D, 4 * D + H))
    t = {n: buf[..., a:b] for n, (a, b) in cuts.items()}
    t["dout"] = to_dev(x["dout"], dtype)
    wide = torch.full((B, N, D + 32), 7.0, device="cuda", dtype=TDT[dtype])
    out = wide[..., 16:16 + D]
    saved = new_saved(t, H)
    sva.sva_diff_anchor_fwd(t["q"], t["k"], t["v"], t["g"], t["lam"], out, H, saved=saved)
    grads = torch.full_like(buf, 7.0)
    g = {n: grads[..., a:b] for n, (a, b) in cuts.items()}
    sva.sva_diff_anchor_bwd(t["q"], t["k"], t["v"], t["g"], t["lam"], t["dout"], saved, g["q"],
                            g["k"], g["v"], g["g"], g["lam"], H)
    ref = oracle(x, H)
    assert_close(to_host(out), ref["out"], dtype, "out")
    for n, r in zip(("q", "k", "v", "g", "lam"), GRADS):
        assert_close(to_host(g[n]), ref[r], dtype, r)
    assert torch.all(wide[..., :16] == 7) and torch.all(wide[..., 16 + D:] == 7)
    assert torch.all(grads[..., 4 * D + H:] == 7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_against_differences(dtype):
    # the kernels' own forward pass, differenced along the gradient: a bf16 output hides steps
    # below its rounding, so the directions are taken whole
    H = 1
    x = make(1, 96, 96, H, 128, dtype, 21)
    t = dev(x, dtype)
    saved = new_saved(t, H)
    forward(t, H, saved)
    g, _ = backward(t, H, saved)
    dout = t["dout"].double()
    for n, gn in (("q", "dq"), ("v", "dv"), ("g", "dgate")):
        step = 0.05
        move = (step * torch.sign(g[gn])).to(t[n].dtype)
        ends = []
        for s in (1, -1):
            moved = t[n] + s * move
            out, _ = forward({**t, n: moved}, H)
            ends.append(((out.double() * dout).sum(), moved.double()))
        slope = float(ends[0][0] - ends[1][0])
        told = float((g[gn].double() * (ends[0][1] - ends[1][1])).sum())
        # third-order terms: step^2 = 2.5e-3 of the slope and its like; bf16 outputs round 96 * 128
        # products at random, 2^-9 each, against a slope of their coherent sum
        assert abs(slope - told) < 2e-2 * abs(told), (n, slope, told)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_stream_graph_capture_and_two_calls_at_once(dtype):
    H, d = 2, 128
    xs = [make(1, 200, 700, H, d, dtype, 30 + i) for i in range(2)]
    ts = [dev(x, dtype) for x in xs]
    eager = []
    for t in ts:
        saved = new_saved(t, H)
        out, _ = forward(t, H, saved)
        eager.append((out, backward(t, H, saved)[0]))
    torch.cuda.synchronize()
    # two streams, each call with a workspace of its own
    streams = [torch.cuda.Stream() for _ in ts]
    for _ in range(3):
        got = []
        for t, s in zip(ts, streams):
            with torch.cuda.stream(s):
                saved = new_saved(t, H)
                out, _ = forward(t, H, saved)
                got.append((out, backward(t, H, saved)[0]))
        torch.cuda.synchronize()
        for (o, g), (eo, eg) in zip(got, eager):
            assert torch.equal(o, eo) and all(torch.equal(g[n], eg[n]) for n in GRADS)
    # a captured step replayed on new inputs
    t = {n: v.clone() for n, v in ts[0].items()}
    saved = new_saved(t, H)
    out = torch.empty_like(t["q"])
    g = {n: torch.empty_like(t[s]) for n, s in zip(GRADS, ("q", "k", "v", "g", "lam"))}
    dt = sva._dtype_code(t["q"])
    ws = sva.workspace(sva.sva_diff_anchor_workspace_bytes(1, 200, H, d, 700, dt))
    wb = sva.workspace(sva.sva_diff_anchor_bwd_workspace_bytes(1, 200, H, d, 700, dt))

    def step():
        sva.sva_diff_anchor_fwd(t["q"], t["k"], t["v"], t["g"], t["lam"], out, H, saved=saved, ws=ws)
        sva.sva_diff_anchor_bwd(t["q"], t["k"], t["v"], t["g"], t["lam"], t["dout"], saved, g["dq"],
                                g["dk"], g["dv"], g["dgate"], g["dlam"], H, ws=wb)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (1, 0):
        for n in t:
            t[n].copy_(ts[i][n])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i][0])
        assert all(torch.equal(g[n], eager[i][1][n]) for n in GRADS)
    assert sva.sva_check_device_status(ws) == sva.SVA_OK


# one query, a handful, a tile of queries against many keys, keys against many queries: each has
# its kernel or its cuts
CUT = [(2, 1, 3000, 2), (1, 4, 5000, 1), (2, 40, 6000, 1), (1, 3000, 70, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("flags", [0, sva.SVA_FLAG_LAMBDA_VALUE])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,N,keys,H", CUT)
def test_lambda_forms_of_cut_work(dtype, flags, shared, B, N, keys, H):
    x = make(B, N, keys, H, 128, dtype, 61, shared=shared)
    x["lam"].ravel()[:2] = (-1.5, 0.0)[:x["lam"].size]
    compare(x, dev(x, dtype), H, dtype, flags=flags)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,keys,H", CUT)
def test_slices_of_cut_work(dtype, B, N, keys, H):
    # keys and values, and their gradients, as column slices of one buffer: the same bits as from
    # buffers of their own, and what lies between and behind is left as it was
    x = make(B, N, keys, H, 128, dtype, 62)
    t = dev(x, dtype)
    D = H * 128
    saved = new_saved(t, H)
    out, _ = forward(t, H, saved)
    g, _ = backward(t, H, saved)
    kv = torch.full((B, keys, 2 * D + 32), float("nan"), device="cuda", dtype=TDT[dtype])
    kv[..., :D], kv[..., D + 16:2 * D + 16] = t["k"], t["v"]
    s = {**t, "k": kv[..., :D], "v": kv[..., D + 16:2 * D + 16]}
    saved2 = new_saved(s, H)
    out2, _ = forward(s, H, saved2)
    assert torch.equal(out, out2) and all(torch.equal(a, b) for a, b in zip(saved, saved2))
    dkv = torch.full((B, keys, 2 * D + 32), 7.0, device="cuda", dtype=TDT[dtype])
    dq = torch.full((B, N, D + 16), 7.0, device="cuda", dtype=TDT[dtype])
    dk, dv = dkv[..., :D], dkv[..., D + 16:2 * D + 16]
    sva.sva_diff_anchor_bwd(s["q"], s["k"], s["v"], s["g"], s["lam"], s["dout"], saved2, dq[..., :D],
                            dk, dv, torch.empty_like(s["g"]), torch.empty_like(s["lam"]), H)
    for got, n in ((dq[..., :D], "dq"), (dk, "dk"), (dv, "dv")):
        assert torch.equal(got, g[n]), n
    assert torch.all(dkv[..., D:D + 16] == 7) and torch.all(dkv[..., 2 * D + 16:] == 7)
    assert torch.all(dq[..., D:] == 7)


@pytest.mark.parametrize("dtype, d", [("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("B,N,keys,H", CUT + [(1, 1024, 1024, 4)])
def test_capture_of_cut_work(dtype, d, B, N, keys, H):
    ts = [dev(make(B, N, keys, H, d, dtype, 63 + i), dtype) for i in range(2)]
    t = {n: v.clone() for n, v in ts[0].items()}
    saved = new_saved(t, H)
    out = torch.empty_like(t["q"])
    g = {n: torch.empty_like(t[s]) for n, s in zip(GRADS, ("q", "k", "v", "g", "lam"))}
    dt = sva._dtype_code(t["q"])
    ws = sva.workspace(sva.sva_diff_anchor_workspace_bytes(B, N, H, d, keys, dt))
    wb = sva.workspace(sva.sva_diff_anchor_bwd_workspace_bytes(B, N, H, d, keys, dt))

    def step():
        sva.sva_diff_anchor_fwd(t["q"], t["k"], t["v"], t["g"], t["lam"], out, H, saved=saved, ws=ws)
        sva.sva_diff_anchor_bwd(t["q"], t["k"], t["v"], t["g"], t["lam"], t["dout"], saved,
                                g["dq"], g["dk"], g["dv"], g["dgate"], g["dlam"], H, ws=wb)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new in (ts[1], ts[0]):
        for n in t:
            t[n].copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        own = new_saved(new, H)
        eo, _ = forward(new, H, own)
        eg, _ = backward(new, H, own)
        assert torch.equal(out, eo) and all(torch.equal(a, b) for a, b in zip(saved, own))
        assert all(torch.equal(g[n], eg[n]) for n in GRADS)


def test_python_refusals():
    t = dev(make(1, 8, 8, 1, 128, "bf16", 1), "bf16")
    out = torch.empty_like(t["q"])
    call = lambda **kw: forward({**t, **kw}, 1)  # noqa: E731
    with pytest.raises(TypeError):
        call(v=t["v"].float())
    with pytest.raises(ValueError):
        call(k=t["k"][..., :64])
    with pytest.raises(ValueError):
        call(lam=torch.zeros(3, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        sva.sva_diff_anchor_fwd(t["q"], t["k"], t["v"], t["g"], t["lam"], out, 1,
                                key_lens=torch.tensor([8], device="cuda"))
    with pytest.raises(ValueError):
        backward(t, 1, None)
    with pytest.raises(sva.SvaError):
        forward({**t, "lam": t["lam"].expand(1, 8, 2).contiguous()}, 2)  # two bf16 heads of 64
