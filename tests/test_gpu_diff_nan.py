"""NaN among the differential anchor's queries and keys that count: it stays NaN in the rows that it
reaches, in each plan of the work (whole units, key parts that are merged or joined in a cluster, a
handful of queries), and in no other row."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import softmax_attention_video_gated_b200 as sva  # noqa: E402

TDT = {"bf16": torch.bfloat16, "f32": torch.float32}

# dtype, d, B, N, keys, H; the last block of keys (128 in bf16, 16 or 32 in fp32) holds one
PLANS = [
    ("bf16", 128, 1, 2000, 897, 1),     # eight parts of a block each, merged
    ("bf16", 128, 2, 2000, 1153, 1),    # parts of one block and of two
    ("bf16", 128, 1, 128 * 150, 129, 1),  # whole units, and two more
    ("f32", 128, 2, 777, 769, 4),       # merged
    ("f32", 64, 2, 1500, 1025, 8),      # whole units, and merged ones
    ("f32", 64, 1, 512, 1025, 4),       # joined in clusters
    ("f32", 128, 1, 200, 1009, 2),
    ("bf16", 128, 2, 1, 3001, 2), ("f32", 128, 2, 3, 3001, 2), ("bf16", 128, 1, 2, 5, 1),
]


def make(dtype, d, B, N, keys, H, room=40):
    """Inputs whose batches have `keys` keys of keys + room; what lies behind is NaN."""
    g = torch.Generator(device="cuda").manual_seed(N + keys)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(TDT[dtype])  # noqa: E731
    D = H * d
    t = dict(q=r(B, N, D), k=r(B, keys + room, D), v=r(B, keys + room, D), gate=r(B, N, D),
             lam=r(B, N, H), dout=r(B, N, D))
    t["k"][:, keys:] = math.nan
    t["v"][:, keys:] = math.nan
    t["lens"] = torch.full((B,), keys, dtype=torch.int32, device="cuda")
    return t


def step(t, H):
    """out, lse and the gradients"""
    B, N, _ = t["q"].shape
    new = lambda x: torch.full_like(x, 7.0)  # noqa: E731
    r = dict(out=new(t["q"]), o1=new(t["q"].float()), o2=new(t["q"].float()),
             lse=torch.full((2, B, H, N), 7.0, device="cuda"))
    saved = (r["o1"], r["o2"], r["lse"])
    sva.sva_diff_anchor_fwd(t["q"], t["k"], t["v"], t["gate"], t["lam"], r["out"], H, saved=saved,
                            key_lens=t["lens"])
    for n in ("q", "k", "v", "gate", "lam"):
        r["d" + n] = new(t[n])
    sva.sva_diff_anchor_bwd(t["q"], t["k"], t["v"], t["gate"], t["lam"], t["dout"], saved,
                            *(r["d" + n] for n in ("q", "k", "v", "gate", "lam")), H, key_lens=t["lens"])
    return r


@pytest.mark.parametrize("dtype,d,B,N,keys,H", PLANS)
def test_a_query_row_that_is_not_a_number(dtype, d, B, N, keys, H):
    t = make(dtype, d, B, N, keys, H)
    clean = step(t, H)
    assert all(torch.isfinite(v).all() for v in clean.values())
    for row in {0, N // 2, N - 1}:
        q = t["q"].clone()
        q[0, row, :d] = math.nan           # one head of one batch
        r = step({**t, "q": q}, H)
        for n in ("out", "o1", "o2", "dq", "dgate"):
            want = clean[n].clone()
            want[0, row, :d] = math.nan
            assert torch.equal(r[n].isnan(), want.isnan()), n
            assert torch.equal(r[n].nan_to_num(0), want.nan_to_num(0)), n
        assert r["lse"][:, 0, 0, row].isnan().all() and int(r["lse"].isnan().sum()) == 2
        assert bool(r["dlam"][0, row, 0].isnan())
        for n in ("dk", "dv"):              # every key of that head and batch, and no other
            assert r[n][0, :keys, :d].isnan().all(), n
            assert torch.equal(r[n][1:], clean[n][1:]) and torch.equal(r[n][0, :, d:], clean[n][0, :, d:]), n


@pytest.mark.parametrize("dtype,d,B,N,keys,H", PLANS)
@pytest.mark.parametrize("half", [0, 1])
def test_a_key_that_is_not_a_number(dtype, d, B, N, keys, H, half):
    t = make(dtype, d, B, N, keys, H)
    clean = step(t, H)
    # the last key, alone in its block; others at the places of both exponentials of a block
    for at in {keys - 1, 0, keys // 2, keys // 2 + 6, keys // 2 + 7} - {keys}:
        if at >= keys:
            continue
        k = t["k"].clone()
        k[0, at, half * d // 2:(half + 1) * d // 2] = math.nan   # one map of head 0
        r = step({**t, "k": k}, H)
        assert r["out"][0, :, :d].isnan().all(), at
        assert r["lse"][half, 0, 0].isnan().all() and torch.equal(r["lse"][1 - half], clean["lse"][1 - half])
        assert r["dq"][0, :, half * d // 2:(half + 1) * d // 2].isnan().all(), at
        assert torch.equal(r["out"][1:], clean["out"][1:]) and torch.equal(r["out"][0, :, d:], clean["out"][0, :, d:])
        assert torch.equal(r["dv"][1:], clean["dv"][1:])


@pytest.mark.parametrize("dtype,d,B,N,keys,H", PLANS)
def test_no_keys_are_not_a_nan(dtype, d, B, N, keys, H):
    # a batch without keys stays zero whatever its keys hold, beside one that has them
    t = make(dtype, d, max(B, 2), N, keys, H)
    t["lens"][0] = 0
    r = step(t, H)
    assert all(float(r[n][0].abs().max()) == 0 for n in ("out", "o1", "o2", "dq", "dk", "dv", "dgate", "dlam"))
    assert torch.all(r["lse"][:, 0] == -math.inf) and torch.isfinite(r["lse"][:, 1]).all()


@pytest.mark.parametrize("what", ["q", "dout"])
@pytest.mark.parametrize("dtype,d,B,N,keys,H", PLANS)
def test_rows_behind_the_last_key_are_zero_whatever_the_queries_hold(dtype, d, B, N, keys, H, what):
    t = make(dtype, d, max(B, 2), N, keys, H)
    x = t[what].clone()
    x[:, N // 2] = math.nan
    for lens in ([keys, 0], [keys - 3, keys]):
        t["lens"][:2] = torch.tensor(lens)
        r = step({**t, what: x}, H)
        for b in range(2):
            for n in ("dk", "dv"):
                assert torch.all(r[n][b, lens[b]:] == 0), (n, b)
