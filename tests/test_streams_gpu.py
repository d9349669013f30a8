"""Calls on a stream of their own (stream=) while the caller's current stream
goes on: what a call allocates, what the caller drops and what queued work still
uses stay apart.  A busy stream is one with a spin of some 50 ms in front."""
import pytest
import torch

import retention_scan_b200 as la

pytestmark = pytest.mark.gpu

SPIN = 100_000_000  # cycles


@pytest.fixture(scope="module", autouse=True)
def built():
    from retention_scan_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def inputs():
    g = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    B, H, T, D = 4, 8, 96, 128  # 1.5 MB and more a tensor: blocks of their own
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).bfloat16()  # noqa: E731
    i = dict(q=unit(rn(B, H, T, D)), k=unit(rn(B, H, T, D)), v=rn(B, H, T, D).bfloat16(), beta=torch.sigmoid(rn(B, H, T)),
             lg=torch.nn.functional.logsigmoid(3 + rn(B, H, T)), S=rn(B, H, D, D), w=1 + 0.1 * rn(D),
             freq=la.rotary_frequencies(D, device="cuda")[0], beta16=torch.sigmoid(rn(B, H, T, D)).bfloat16())
    # made here: what a call makes of its inputs on the current stream would not be ordered before a stream's kernels
    return dict(i, qa=i["q"].abs(), ka=i["k"].abs(), seg=i["S"][None].clone(), seg_lg=i["lg"][None, :, :, 0].clone(),
                w8=i["w"].repeat(8))


def token(t):
    return t[:, :, 0].contiguous()


CALLS = {
    "delta_forward": lambda i, **k: la.delta_forward(i["q"], i["k"], i["v"], i["beta"], 2, i["lg"], i["S"], **k),
    "delta_backward": lambda i, **k: la.delta_backward(i["q"], i["k"], i["v"], i["beta"], i["v"], 2, i["lg"], i["S"], **k),
    "gated_norm": lambda i, **k: la.gated_norm(i["v"], i["q"], i["w"], **k),
    "gated_norm_backward": lambda i, **k: la.gated_norm_backward(i["v"], i["q"], i["k"], i["w"], **k),
    "rotary": lambda i, **k: la.rotary(i["q"], i["freq"], None, i["k"], **k),
    "chunk_forward": lambda i, **k: la.chunk_forward(i["q"], i["k"], i["v"], 2, i["lg"], init_state=i["S"], **k),
    "chunk_forward_raw": lambda i, **k: la.chunk_forward(i["q"], i["k"], i["v"], 2, i["lg"], normalize=True,
                                                         feature_map=la.FEATURE_ELU1, **k),
    "chunk_reverse": lambda i, **k: la.chunk_forward(i["q"], i["k"], i["v"], 2, i["lg"], reverse=True, **k),
    "bidirectional": lambda i, **k: la.bidirectional(i["q"], i["k"], i["v"], 2, i["lg"], **k),
    "chunk_backward": lambda i, **k: la.chunk_backward(i["q"], i["k"], i["v"], i["v"], 2, i["lg"], i["S"], **k),
    "chunk_backward_normalized": lambda i, **k: la.chunk_backward_normalized(i["qa"], i["ka"], i["v"], i["v"], 2, i["lg"], **k),
    "chunk_state": lambda i, **k: la.chunk_state(i["k"], i["v"], 2, i["lg"], normalize=True, **k),
    "state_combine": lambda i, **k: la.state_combine(i["seg"], i["seg_lg"], init_state=i["S"], **k),
    "ema_scan": lambda i, **k: la.ema_scan(i["v"].view(4, 96, 1024), i["beta16"].view(4, 96, 1024), **k),
    "wkv4_forward": lambda i, **k: la.wkv4_forward(i["k"].view(4, 96, 1024), i["v"].view(4, 96, 1024), i["w8"], i["w8"], **k),
}


def flat(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


@pytest.mark.parametrize("name", CALLS)
def test_dropped_outputs_are_not_written_over_new_tensors(name):
    i = inputs()
    shapes = [(t.shape, t.dtype) for t in flat(CALLS[name](i))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(SPIN)
    CALLS[name](i, stream=s)  # every output dropped while the call has yet to write it
    new = [torch.full(shape, 7.0, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(3)]
    torch.cuda.synchronize()
    assert all((t == 7.0).all() for t in new)


@pytest.mark.parametrize("name", CALLS)
def test_memory_that_queued_work_uses_is_not_handed_out(name):
    i = inputs()
    old = [torch.full(t.shape, 3.0, dtype=t.dtype, device="cuda") for t in flat(CALLS[name](i))]
    old.append(torch.full((64 << 18,), 3.0, device="cuda"))  # a workspace's block
    torch.cuda.synchronize()
    torch.cuda._sleep(SPIN)
    kept = [t.clone() for t in old]  # queued behind the spin; the blocks then go back to the current stream's pool
    del old
    s = torch.cuda.Stream()
    CALLS[name](i, stream=s)
    torch.cuda.synchronize()
    assert all((t == 3.0).all() for t in kept)


@pytest.mark.parametrize("name", CALLS)
def test_outputs_read_on_the_callers_stream_and_dropped(name):
    i = inputs()
    want = flat(CALLS[name](i))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = flat(CALLS[name](i, stream=s))
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(SPIN)
    kept = [t.clone() for t in got]
    del got
    CALLS[name](dict(i, q=i["k"], k=i["q"]), stream=s)  # other values, on a stream that does not wait for the copies
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))


@pytest.mark.parametrize("name", CALLS)
def test_inputs_dropped_while_the_call_runs(name):
    i = inputs()
    want = flat(CALLS[name](i))
    s = torch.cuda.Stream()
    copies = {n: t.clone() for n, t in i.items()}
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(SPIN)
    got = flat(CALLS[name](copies, stream=s))
    del copies
    new = [torch.full_like(t, 7.0) for t in i.values() for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all((t == 7.0).all() for t in new)


def test_one_token_on_a_busy_stream():
    i = inputs()
    state = i["S"].clone()
    want = la.delta_decode_step(token(i["q"]), token(i["k"]), token(i["v"]), token(i["beta"]), state, 2, token(i["lg"]))
    s = torch.cuda.Stream()
    args = [token(i[n]) for n in ("q", "k", "v", "beta")] + [i["S"], 2, token(i["lg"])]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(SPIN)
    got = la.delta_decode_step(*args, stream=s)
    del args  # the token's tensors go while the call has yet to read them
    new = [torch.full_like(want, 7.0) for _ in range(16)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(i["S"], state) and all((t == 7.0).all() for t in new)
    # and the plain scan's
    want = la.decode_step(token(i["q"]), token(i["k"]), token(i["v"]), state, None, 2, token(i["lg"]))
    args = [token(i[n]) for n in ("q", "k", "v")] + [i["S"], None, 2, token(i["lg"])]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(SPIN)
    got = la.decode_step(*args, stream=s)
    del args
    new = [torch.full_like(want, 7.0) for _ in range(16)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(i["S"], state) and all((t == 7.0).all() for t in new)


def test_a_stream_of_another_device_is_refused():
    class Elsewhere:
        device = torch.device("cuda", torch.cuda.device_count())
        cuda_stream = 0
    i = inputs()
    for name, call in CALLS.items():
        with pytest.raises(ValueError, match="stream"):
            call(i, stream=Elsewhere())


@pytest.mark.parametrize("name", CALLS)
def test_a_capture_that_forks_to_a_stream_of_its_own(name):
    # the call's allocations come from the graph's pool, on the forked stream; what is dropped is not the next call's
    i = inputs()
    CALLS[name](i)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        CALLS[name](i, stream=s)  # dropped
        got = flat(CALLS[name](i, stream=s))
        torch.cuda.current_stream().wait_stream(s)
        new = torch.full((1 << 20,), 7.0, device="cuda")
    for scale in (1.0, -0.5):
        i["v"].mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, flat(CALLS[name](i)))) and (new == 7.0).all()
