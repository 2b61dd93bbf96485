"""Memory of the tensors that a call makes for another stream than the current one."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")


class FakeTorch:
    """torch.empty and the current stream, with a record of which stream each tensor was made on."""

    def __init__(self):
        self.current, self.made = "current", []
        self.cuda = types.SimpleNamespace(stream=self._stream, Stream=str, current_stream=lambda dev=None: self.current)

    @contextlib.contextmanager
    def _stream(self, s):
        before, self.current = self.current, s
        yield
        self.current = before

    def empty(self, shape, dtype=None, device=None):
        t = types.SimpleNamespace(on=self.current, recorded=[])
        t.record_stream = t.recorded.append
        self.made.append(t)
        return t


def test_tensors_are_made_on_the_stream_of_the_call(monkeypatch):
    import drafter_sampling_gb300 as vt
    fake = FakeTorch()
    monkeypatch.setattr(vt, "_TORCH", fake)
    monkeypatch.setattr(vt, "_DEVICES", ("cuda:0",))
    out = vt._new((2, 3), None, 0, "side")
    assert out.on == "side" and out.recorded == ["current"]
    out = vt._new((2, 3), None, 0, None)
    assert out.on == "current" and out.recorded == []
    out = vt._new((2, 3), None, 0, "side", returned=False)
    assert out.on == "side" and out.recorded == []


B, H, K = 20, 300, 5000


def _calls(vt):
    """(call(stream) -> tensors, sizes of what it allocates) of each entry point that makes its own outputs."""
    W = torch.randn((K, H), device="cuda").to(torch.bfloat16)
    W8, s, _ = vt.vt_quantize_head(W)
    hid = torch.randn((B, H), device="cuda").to(torch.bfloat16)
    ids = torch.arange(K, dtype=torch.int32, device="cuda")
    u = torch.rand(B, device="cuda")
    x = torch.randn((B, K), device="cuda")
    tok = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = vt.workspace_bytes("draft_fp8", B=B, H=H, K=K)
    return {
        "quantize": (lambda st: vt.vt_quantize_head(W, stream=st)[:2], [K * 304]),
        "logits": (lambda st: [vt.vt_draft_logits_fp8(hid, W8, s, stream=st)], [4 * B * K, ws]),
        "step": (lambda st: vt.vt_draft_step_fp8(hid, W8, s, ids, u, stream=st), [4 * B * K, ws]),
        "topk": (lambda st: vt.vt_draft_topk_fp8(hid, W8, s, ids, 8, stream=st),
                 [vt.workspace_bytes("draft_topk_fp8", B=B, H=H, K=K, k=8)]),
        "logprobs": (lambda st: vt.vt_token_logprobs(x, tok, k=8, stream=st), [32 * B, 4 * B]),
    }


def _bytes(tensors):
    """Copies of the tensors' bytes, made on the current stream."""
    return [t.view(torch.uint8).clone() for t in tensors]


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["quantize", "logits", "step", "topk", "logprobs"])
def test_a_busy_current_stream_writes_nothing_of_a_side_streams_call(name):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import drafter_sampling_gb300 as vt
    call, sizes = _calls(vt)[name]
    side = torch.cuda.Stream()
    want = _bytes(call(None))
    torch.cuda.synchronize()
    for _ in range(3):
        # blocks of the sizes that the call allocates, freed while their last owner's kernels have yet to run
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        torch.cuda._sleep(10_000_000)
        for b in blocks:
            b.fill_(0x7F)
        del blocks, b
        got = call(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(_bytes(got), want))
        # read late on the current stream and freed before: the side stream's next tensors lie elsewhere
        torch.cuda._sleep(10_000_000)
        late = _bytes(got)
        del got
        with torch.cuda.stream(side):
            others = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x55) for n in sizes for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(late, want))
        del others


@pytest.mark.gpu
def test_a_side_streams_calls_within_a_capture():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import drafter_sampling_gb300 as vt
    calls = _calls(vt)
    want = {n: _bytes(c(None)) for n, (c, _) in calls.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        got = {n: c(side) for n, (c, _) in calls.items()}
        cur.wait_stream(side)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        for n, w in want.items():
            assert all(torch.equal(a, b) for a, b in zip(_bytes(got[n]), w)), n
