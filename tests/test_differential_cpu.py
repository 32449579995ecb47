"""The differential anchor and the block norms without a GPU: the fp64 oracle's
forms pinned against other things than themselves (the single-map softmax core,
central differences, limits), and the entry points' refusals on the host."""
import ctypes

import numpy as np
import pytest

import oracle as O
import softmax_attention_video_gated_b200 as sva
from oracle import differential as OD


def rand(shape, seed, scale=1.0):
    return np.random.default_rng(seed).standard_normal(shape) * scale


def diff_inputs(B, N, keys, H, d, seed):
    D = H * d
    r = [rand(s, seed + i) for i, s in enumerate(
        ((B, N, D), (B, keys, D), (B, keys, D), (B, N, D), (B, N, H), (B, N, D)))]
    return dict(zip(("q", "k", "v", "g", "lam", "dout"), r))


# ------------------------------------------------------------ the oracle's pins

def test_oracle_diff_is_two_softmax_cores():
    B, N, keys, H, d = 2, 5, 5, 3, 8
    x = diff_inputs(B, N, keys, H, d, 1)
    r = OD.diff_anchor(x["q"], x["k"], x["v"], x["g"], x["lam"], H)
    # each map alone is the plain softmax core with half-width heads; torch's own attention does it
    import torch
    qh, kh, vh = (torch.from_numpy(O.split_heads(x[n], H)) for n in "qkv")
    maps = [torch.nn.functional.scaled_dot_product_attention(
        qh[..., c].contiguous(), kh[..., c].contiguous(), vh) for c in (slice(0, 4), slice(4, 8))]
    lam = 1 / (1 + np.exp(-x["lam"].transpose(0, 2, 1)))[..., None]
    a = maps[0].numpy() - lam * maps[1].numpy()
    y = O.merge_heads(a) / (1 + np.exp(-x["g"]))
    np.testing.assert_allclose(r["out"], y, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(r["o2"], O.merge_heads(maps[1].numpy()), rtol=1e-12, atol=1e-12)


def test_oracle_diff_equal_maps_cancel_and_empty_batch_is_zero():
    B, N, keys, H, d = 3, 4, 6, 2, 8
    x = diff_inputs(B, N, keys, H, d, 7)
    for n in "qk":  # both halves alike
        h = O.split_heads(x[n], H).copy()
        h[..., 4:] = h[..., :4]
        x[n] = O.merge_heads(h)
    one = OD.diff_anchor(x["q"], x["k"], x["v"], None, np.ones(H), H, raw=True)
    assert np.abs(one["out"]).max() < 1e-14
    r = OD.diff_anchor(x["q"], x["k"], x["v"], x["g"], x["lam"], H, key_lens=[6, 0, 3], dout=x["dout"])
    assert np.all(r["out"][1] == 0) and np.all(r["lse"][:, 1] == -np.inf)
    assert all(np.all(r[n][1] == 0) for n in ("dq", "dk", "dv", "dgate", "dlam"))
    assert np.all(r["dk"][2, 3:] == 0) and np.any(r["dk"][2, :3] != 0)


@pytest.mark.parametrize("raw, shared", [(False, False), (True, True), (False, True)])
def test_oracle_diff_gradients_against_differences(raw, shared):
    B, N, keys, H, d = 2, 3, 4, 2, 4
    x = diff_inputs(B, N, keys, H, d, 11)
    if shared:
        x["lam"] = np.array([0.4, -0.3])
    kw = dict(H=H, key_lens=[4, 3], raw=raw)

    def loss(**new):
        y = {**x, **new}
        return (OD.diff_anchor(y["q"], y["k"], y["v"], y["g"], y["lam"], **kw)["out"] * x["dout"]).sum()

    r = OD.diff_anchor(x["q"], x["k"], x["v"], x["g"], x["lam"], dout=x["dout"], **kw)
    check_gradients(loss, x, {"q": r["dq"], "k": r["dk"], "v": r["dv"], "g": r["dgate"], "lam": r["dlam"]})


def check_gradients(loss, x, grads, step=1e-5):
    # central differences: error about step^2 times a third derivative of order one, plus
    # rounding 1e-16 / step = 1e-11, so 1e-8 holds with room
    for n, g in grads.items():
        flat = x[n].ravel()
        for i in np.random.default_rng(3).choice(flat.size, min(12, flat.size), replace=False):
            e = np.zeros(flat.size)
            e[i] = step
            e = e.reshape(x[n].shape)
            num = (loss(**{n: x[n] + e}) - loss(**{n: x[n] - e})) / (2 * step)
            assert abs(num - g.ravel()[i]) < 1e-8 * max(1, abs(num)), (n, i, num, g.ravel()[i])


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("part", ["both", "pre", "post"])
def test_oracle_block_norm_gradients_against_differences(layer, part):
    B, N, D = 2, 3, 5
    shapes = dict(h=(B, N, D), o=(B, N, D), w_post=(D,), gate=(B, D), w_pre=(D,), scale=(B, D),
                  shift=(B, D))
    if part == "pre":
        shapes = {n: s for n, s in shapes.items() if n not in ("o", "w_post", "gate")}
    if part == "post":
        shapes = {n: s for n, s in shapes.items() if n not in ("w_pre", "scale", "shift")}
    x = {n: rand(s, 20 + i) for i, (n, s) in enumerate(shapes.items())}
    dh_out, du = rand((B, N, D), 40), rand((B, N, D), 41)
    kw = dict(pre=part != "post", layer=layer, eps=1e-3, res_scale=0.7)

    def loss(**new):
        r = OD.block_norm(**{**x, **new}, **kw)
        hp = r.get("h_out", {**x, **new}["h"])
        return (hp * dh_out).sum() + (r["u"] * du).sum() * (part != "post") if part != "post" \
            else (hp * dh_out).sum()

    r = OD.block_norm(**x, **kw, dh_out=dh_out, du=du)
    check_gradients(loss, x, {n: r["d" + n] for n in shapes})


def test_oracle_block_norm_against_torch():
    import torch
    h, w, b = rand((2, 3, 6), 1), rand(6, 2), rand((2, 6), 3)
    u = OD.block_norm(h, w_pre=w, layer=True, eps=1e-5)["u"]
    t = torch.nn.functional.layer_norm(torch.from_numpy(h), (6,), torch.from_numpy(w), eps=1e-5)
    np.testing.assert_allclose(u, t.numpy(), rtol=1e-12, atol=1e-12)
    u = OD.block_norm(h, w_pre=w, shift=b, eps=1e-5)["u"]
    t = torch.nn.functional.rms_norm(torch.from_numpy(h), (6,), torch.from_numpy(w), eps=1e-5)
    np.testing.assert_allclose(u, t.numpy() + b[:, None], rtol=1e-12, atol=1e-12)


# ------------------------------------------------------------ refusals on the host

def diff_args(**kw):
    a = sva.DiffArgs()
    a.B, a.N, a.H, a.d, a.dtype = 1, 256, 2, 128, sva.SVA_BF16
    for f in ("q", "k", "v", "gate", "lam", "out", "o1", "o2", "lse"):
        setattr(a, f, 0x10000)
    a.ldq = a.ldk = a.ldv = a.ldg = a.ldo = 256
    a.ldl = 2
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def diff_grads(**kw):
    g = sva.DiffGrads()
    for f, ld in (("dout", "lddo"), ("dq", "lddq"), ("dk", "lddk"), ("dv", "lddv"), ("dgate", "lddg")):
        setattr(g, f, 0x10000)
        setattr(g, ld, 256)
    g.dlam, g.lddl = 0x10000, 2
    for k, v in kw.items():
        setattr(g, k, v)
    return g


BAD, NO = sva.SVA_ERR_INVALID_ARGUMENT, sva.SVA_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad, expect", [
    (dict(q=None), BAD), (dict(k=0x10008), BAD), (dict(ldv=128), BAD), (dict(ldk=260), BAD),
    (dict(N=0), BAD), (dict(n_keys=-1), BAD), (dict(dtype=5), BAD), (dict(lam=None), BAD),
    (dict(lam=0x10001), BAD), (dict(ldl=1), BAD), (dict(ldg=100), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=float("nan")), BAD), (dict(flags=1), BAD), (dict(key_lens=0x10002), BAD),
    (dict(o2=None), BAD), (dict(lse=None), BAD),
    (dict(d=64), NO), (dict(d=256, ldq=512, ldk=512, ldv=512, ldg=512, ldo=512), NO),
    (dict(B=3, N=1 << 30), NO), (dict(B=3, n_keys=1 << 30), NO), (dict(B=40000), NO),
])
def test_diff_rejects_bad_arguments_on_host(bad, expect):
    lib, a = sva._lib(), diff_args(**bad)
    assert lib.sva_diff_anchor_fwd(ctypes.byref(a), 0x20000, 1 << 62, None) == expect
    g = diff_grads()
    assert lib.sva_diff_anchor_bwd(ctypes.byref(a), ctypes.byref(g), 0x20000, 1 << 62, None) == expect


@pytest.mark.parametrize("bad", [
    dict(dout=None), dict(dq=None), dict(dk=0x10004), dict(lddv=100), dict(dgate=None),
    dict(dlam=None), dict(lddl=0), dict(lddl=1), dict(dlam=0x10001),
])
def test_diff_backward_rejects_bad_gradients_on_host(bad):
    lib, a, g = sva._lib(), diff_args(), diff_grads(**bad)
    call = lambda a, g: lib.sva_diff_anchor_bwd(ctypes.byref(a), ctypes.byref(g), 0x20000,  # noqa: E731
                                                1 << 62, None)
    assert call(a, g) == BAD
    assert call(diff_args(gate=None), diff_grads()) == BAD              # dgate without a gate
    assert call(diff_args(ldl=0), diff_grads()) == BAD                  # dlam per token, lam shared
    assert call(diff_args(o1=None, o2=None, lse=None), diff_grads()) == BAD  # nothing saved


def test_diff_forward_needs_out_and_its_workspaces():
    lib = sva._lib()
    assert lib.sva_diff_anchor_fwd(None, 0x20000, 1 << 30, None) == BAD
    assert lib.sva_diff_anchor_fwd(ctypes.byref(diff_args(out=None)), 0x20000, 1 << 62, None) == BAD
    for a in (diff_args(), diff_args(N=1, n_keys=50000)):
        need = sva.sva_diff_anchor_workspace_bytes(a.B, a.N, a.H, a.d, a.n_keys, a.dtype)
        assert need >= 256
        for ws, n in ((None, need), (0x20008, need), (0x20000, need - 1)):
            assert lib.sva_diff_anchor_fwd(ctypes.byref(a), ws, n, None) == sva.SVA_ERR_WORKSPACE
        need = sva.sva_diff_anchor_bwd_workspace_bytes(a.B, a.N, a.H, a.d, a.n_keys, a.dtype)
        g = diff_grads()
        assert lib.sva_diff_anchor_bwd(ctypes.byref(a), ctypes.byref(g), 0x20000, need - 1,
                                       None) == sva.SVA_ERR_WORKSPACE
    assert sva.sva_diff_anchor_workspace_bytes(0, 1, 1, 128, 1, sva.SVA_BF16) == 0
    assert sva.sva_diff_anchor_bwd_workspace_bytes(1, 1, 1, 128, -1, sva.SVA_BF16) == 0


def norm_args(**kw):
    a = sva.BlockNormArgs()
    a.B, a.N, a.D, a.dtype, a.kind, a.eps, a.res_scale = 2, 16, 100, sva.SVA_BF16, 0, 1e-6, 1.0
    for f, ld in (("h", "ldh"), ("o", "ldo"), ("gate", "ldgate"), ("h_out", "ldho"),
                  ("scale", "ldscale"), ("shift", "ldshift"), ("u", "ldu")):
        setattr(a, f, 0x10000)
        setattr(a, ld, 104)
    a.w_post = a.w_pre = a.stats = 0x10000
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def norm_grads(**kw):
    g = sva.BlockNormGrads()
    for f, ld in (("dh_out", "lddho"), ("du", "lddu"), ("dh", "lddh"), ("d_o", "lddo")):
        setattr(g, f, 0x10000)
        setattr(g, ld, 104)
    g.dw_post = g.dgate = g.dw_pre = g.dscale = g.dshift = 0x10000
    for k, v in kw.items():
        setattr(g, k, v)
    return g


@pytest.mark.parametrize("bad, expect", [
    (dict(B=0), BAD), (dict(D=0), BAD), (dict(dtype=9), BAD), (dict(kind=2), BAD),
    (dict(eps=-1e-6), BAD), (dict(res_scale=float("inf")), BAD), (dict(ldo=99), BAD),
    (dict(ldo=100), BAD),                                     # 200-byte rows: not 16-byte aligned
    (dict(h_out=None), BAD), (dict(u=0x10002), BAD), (dict(w_pre=0x10002), BAD),
    (dict(ldgate=96), BAD), (dict(stats=0x10004), BAD),
    (dict(o=None, u=None), BAD), (dict(o=None), BAD),         # its weight and gate are still there
    (dict(u=None), BAD),
    (dict(D=8193, ldh=8200, ldo=8200, ldgate=8200, ldho=8200, ldscale=8200, ldshift=8200, ldu=8200), NO),
    (dict(B=3, N=1 << 30), NO),
])
def test_block_norm_rejects_bad_arguments_on_host(bad, expect):
    lib, a = sva._lib(), norm_args(**bad)
    assert lib.sva_block_norm_fwd(ctypes.byref(a), None) == expect
    assert lib.sva_block_norm_bwd(ctypes.byref(a), ctypes.byref(norm_grads()), 0x20000, 1 << 62,
                                  None) == expect


@pytest.mark.parametrize("bad", [
    dict(du=None), dict(dh=None), dict(d_o=None), dict(lddh=96), dict(dh_out=0x10004),
    dict(dscale=0x10002),
])
def test_block_norm_backward_rejects_bad_gradients_on_host(bad):
    lib = sva._lib()
    call = lambda a, g, n=1 << 62: lib.sva_block_norm_bwd(ctypes.byref(a), ctypes.byref(g),  # noqa: E731
                                                          0x20000, n, None)
    assert call(norm_args(), norm_grads(**bad)) == BAD
    assert call(norm_args(stats=None), norm_grads()) == BAD
    only_pre = dict(o=None, w_post=None, gate=None)
    assert call(norm_args(**only_pre), norm_grads()) == BAD   # d_o, dw_post and dgate without o
    only_post = dict(u=None, w_pre=None, scale=None, shift=None)
    assert call(norm_args(**only_post), norm_grads()) == BAD
    need = sva.sva_block_norm_bwd_workspace_bytes(2, 16, 100)
    assert need > 256 and call(norm_args(), norm_grads(), need - 1) == sva.SVA_ERR_WORKSPACE
    assert sva.sva_block_norm_bwd_workspace_bytes(0, 16, 100) == 0


def test_struct_layouts_match_the_header():
    # LP64 sizes of the C structs in include/sva.h, field by field
    assert ctypes.sizeof(sva.DiffArgs) == 6 * 4 + 5 * 16 + 8 + 16 + 8 + 3 * 8
    assert ctypes.sizeof(sva.DiffGrads) == 6 * 16
    assert ctypes.sizeof(sva.BlockNormArgs) == 7 * 4 + 4 + 16 + 16 + 8 + 16 + 16 + 8 + 3 * 16 + 8
    assert ctypes.sizeof(sva.BlockNormGrads) == 4 * 16 + 5 * 8
