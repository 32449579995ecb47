"""A call on a given stream: the workspace that it makes for itself belongs to that stream, whether or
not the caller keeps it."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import softmax_attention_video_gated_b200 as sva  # noqa: E402


def test_a_workspace_is_made_on_the_given_stream(monkeypatch):
    on, made = [], []

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()

    empty = torch.empty

    def recorded(*a, **kw):
        made.append(list(on))
        return empty(*a, **kw)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", recorded)
    assert sva.workspace(1000, "cpu").numel() == 1000
    ws = sva.workspace(10, "cpu", "side")
    assert ws.numel() == sva.SVA_STATUS_BYTES and ws.dtype == torch.uint8
    assert made == [[], ["side"]] and on == []


# ------------------------------------------------------------------ on a GPU

B, N, H, d = 1, 300, 2, 128
D = H * d


def rand(*s, dt=torch.bfloat16):
    return torch.randn(*s, device="cuda").to(dt)


def calls():
    """One call of every entry point that makes a workspace, as a function of the stream."""
    x = {n: rand(B, N, D) for n in ("q", "k", "v", "g", "out", "dout", "dq", "dk", "dv", "dg")}
    qkvg = (x["q"], x["k"], x["v"], x["g"], x["out"])
    f32 = torch.float32
    state = rand(B * H, d * d + d, dt=f32)
    lam, dlam = rand(H), rand(H)
    saved = (rand(B, N, D, dt=f32), rand(B, N, D, dt=f32), rand(2, B, H, N, dt=f32))
    h, dh, stats = rand(B, N, D, dt=f32), rand(B, N, D, dt=f32), rand(B, N, 4, dt=f32)
    w, y, dw = rand(D, D), rand(N, D), rand(D, dt=f32)
    st = sva.Stack([rand(4 * D, D) for _ in range(4)], [rand(D, D) for _ in range(4)], rand(D, D), B, N, H)
    hx, hy = torch.zeros(B, N, D, dtype=torch.bfloat16), torch.zeros(B, N, D, dtype=torch.bfloat16)
    return {
        "linear": lambda s: sva.sva_linear_attn_fwd(*qkvg, H, stream=s),
        "state": lambda s: sva.sva_linear_attn_state_fwd(x["k"], x["v"], state, H, stream=s),
        "readout": lambda s: sva.sva_linear_attn_readout_fwd(x["q"], x["g"], x["out"], state, H, stream=s),
        "anchor": lambda s: sva.sva_softmax_anchor_fwd(*qkvg, H, stream=s),
        "diff": lambda s: sva.sva_diff_anchor_fwd(*qkvg[:4], lam, x["out"], H, saved=saved, stream=s),
        "diff_bwd": lambda s: sva.sva_diff_anchor_bwd(*qkvg[:4], lam, x["dout"], saved, x["dq"], x["dk"],
                                                      x["dv"], x["dg"], dlam, H, stream=s),
        "norm_bwd": lambda s: sva.sva_block_norm_bwd(h, stats, dh, du=x["dout"], dw_pre=dw, stream=s),
        "projection": lambda s: sva.sva_projection_fwd(x["q"][0], w, y, stream=s),
        "projection_residual": lambda s: sva.sva_projection_residual_fwd(x["q"][0], w, h[0], stream=s),
        "keys": lambda s: sva.sva_attnres_keys(x["q"][0], w, y, stream=s),
        "stack": lambda s: sva.sva_hybrid_stack_fwd(st, x["q"], x["out"], stream=s),
        "stack_host": lambda s: sva.sva_hybrid_stack_fwd_host(st, [hx], [hy], stream=s),
    }


def owner(t):
    """The stream whose memory the tensor lies in."""
    at = t.data_ptr()
    return next(g["stream"] for g in torch.cuda.memory_snapshot()
                if g["address"] <= at < g["address"] + g["total_size"])


@pytest.mark.gpu
def test_every_calls_own_workspace_belongs_to_its_stream():
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for name, call in calls().items():
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        for s in (side, None):
            made = call(s)
            torch.cuda.synchronize()
            for ws in made if isinstance(made, tuple) else (made,):
                want = side.cuda_stream if s is not None else torch.cuda.current_stream().cuda_stream
                assert owner(ws) == want, name


@pytest.mark.gpu
def test_gradients_on_a_given_stream_while_the_current_one_makes_buffers():
    # the returned workspace is dropped at once; the current stream then fills buffers of its size
    n, keys = 1500, 1500
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    q, k, v, gate, dout = r(2, n, D), r(2, keys, D), r(2, keys, D), r(2, n, D), r(2, n, D)
    lam, f32 = r(H), torch.float32
    h, stats = r(2, n, D, dt=f32), torch.empty(2, n, 4, device="cuda")
    u = torch.empty_like(q)
    sva.sva_block_norm_fwd(h, u=u, stats=stats)

    def step(s):
        saved = (torch.empty_like(q, dtype=f32), torch.empty_like(q, dtype=f32),
                 torch.empty(2, 2, H, n, device="cuda"))
        out = torch.empty_like(q)
        grads = [torch.empty_like(t) for t in (q, k, v, gate, lam)]
        dh, dw = torch.empty_like(h), torch.empty(D, device="cuda")
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        sva.sva_diff_anchor_fwd(q, k, v, gate, lam, out, H, saved=saved, stream=s)
        sva.sva_diff_anchor_bwd(q, k, v, gate, lam, dout, saved, *grads, H, stream=s)
        sva.sva_block_norm_bwd(h, stats, dh, du=dout, dw_pre=dw, stream=s)
        if s is not None:
            need = sva.sva_diff_anchor_bwd_workspace_bytes(2, n, H, d, keys, sva.SVA_BF16)
            for size in (need, need // 2, 1 << 20, 1 << 16, need):
                for _ in range(4):
                    torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        return [out, *saved, *grads, dh, dw]

    want = step(None)
    side = torch.cuda.Stream()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(step(side), want))
