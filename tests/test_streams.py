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


def test_the_older_calls_tensors_too(monkeypatch):
    import drafter_sampling_gb300 as vt
    fake = FakeTorch()
    fake.uint8 = "uint8"
    monkeypatch.setattr(vt, "_TORCH", fake)
    assert vt._empty(3, None, "cuda:0", "side").recorded == ["current"]
    assert vt._ws(100, "cuda:0", "side").recorded == []         # used by that stream alone
    assert vt._ws(100, "cuda:0").on == "current"
    assert [t.on for t in fake.made] == ["side", "side", "current"]


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
    trim = torch.randperm(2 * K, device="cuda")[:K].to(torch.int32)
    inv = torch.full((2 * K,), -1, dtype=torch.int32, device="cuda")
    inv[trim.sort().values.long()] = ids
    Wfull = torch.randn((2 * K, H), device="cuda").to(torch.bfloat16)
    stream_ids = torch.randint(0, 2 * K, (10000,), device="cuda", dtype=torch.int32)
    q = torch.full((B, 2, K), 1.0 / K, device="cuda")
    drafted = trim.sort().values[torch.randint(0, K, (B, 2), device="cuda")].contiguous()
    ua, ur = torch.rand((B, 2), device="cuda"), torch.rand((B, 3), device="cuda")
    z = torch.randn((B, 3, 2 * K), device="cuda")
    parent = torch.tensor([-1, 0], dtype=torch.int32, device="cuda")
    old = {
        "calibrate_topk": (lambda st: vt.vt_calibrate_topk(stream_ids, 2 * K, K, stream=st),
                           [vt.workspace_bytes("calibrate", n=10000, V=2 * K, K=K), 8 * K, 4 * K]),
        "calibrate_top_p": (lambda st: vt.vt_calibrate_top_p(stream_ids, 2 * K, 0.5, stream=st),
                            [vt.workspace_bytes("select", n=10000, V=2 * K), 8 * K]),
        "trim": (lambda st: vt.vt_trim_head(Wfull, trim, stream=st), [2 * K * H, 8 * K, 4 * K]),
        "bf16_logits": (lambda st: [vt.vt_draft_logits(hid, W, stream=st)], [4 * B * K]),
        "bf16_step": (lambda st: vt.vt_draft_step(hid, W, ids, u, stream=st),
                      [4 * B * K, vt.workspace_bytes("draft", B=B, H=H, K=K)]),
        "bf16_topk": (lambda st: vt.vt_draft_topk(hid, W, ids, 8, stream=st), [32 * B, 4 * B * K]),
        "verify": (lambda st: vt.vt_verify(z, q, inv, drafted, ua, ur, stream=st),
                   [vt.workspace_bytes("verify", B=B, gamma=2, V=2 * K, K=K), 12 * B, 8 * B, 4 * B]),
        "verify_tree": (lambda st: vt.vt_verify_tree(z, parent, drafted, stream=st), [12 * B, 8 * B, 4 * B]),
        "selftest": (lambda st: [vt.vt_selftest_wait(1, 1000, stream=st)], [4]),
    }
    return {
        **old,
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
@pytest.mark.parametrize("name", ["quantize", "logits", "step", "topk", "logprobs", "calibrate_topk", "calibrate_top_p",
                                  "trim", "bf16_logits", "bf16_step", "bf16_topk", "verify", "verify_tree",
                                  "selftest"])
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


@pytest.mark.gpu
def test_a_block_graph_made_while_its_stream_is_busy_and_launched_on_another():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import drafter_sampling_gb300 as vt
    gamma, V = 2, 2 * K
    ids = torch.arange(K, dtype=torch.int32, device="cuda")
    inv = torch.full((V,), -1, dtype=torch.int32, device="cuda")
    inv[:K] = ids
    args = (torch.randn((gamma, B, H), device="cuda").to(torch.bfloat16),
            torch.randn((K, H), device="cuda").to(torch.bfloat16), ids, inv,
            torch.randn((B, gamma + 1, V), device="cuda"), torch.rand((gamma, B), device="cuda"),
            torch.rand((B, gamma), device="cuda"), torch.rand((B, gamma + 1), device="cuda"), 8.0)
    outputs = lambda g: _bytes([g.q, g.draft_tokens, g.out_tokens, g.out_num_accepted, g.dev_status])
    first = vt.BlockGraph(*args)
    first.launch()
    want = outputs(first)
    sizes = [first.workspace.numel(), first.q.numel() * 4, first.out_tokens.numel() * 4]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        torch.cuda._sleep(10_000_000)
        for b in blocks:
            b.fill_(0x7F)
        del blocks, b
        g = vt.BlockGraph(*args)
        g.launch(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(outputs(g), want))
        # dropped while a replay has yet to run: the current stream's next tensors lie elsewhere
        with torch.cuda.stream(side):
            torch.cuda._sleep(10_000_000)
        out = g.out_tokens
        g.launch(side)
        del g
        others = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x7F) for n in sizes for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.uint8), want[2])
        del others, out


@pytest.mark.gpu
def test_a_block_graph_outlives_a_stream_of_the_callers_own():
    """A raw stream, destroyed after its replay and before the graph: the tensors' memory is freed without it."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ctypes
    import gc

    import drafter_sampling_gb300 as vt
    rt = ctypes.CDLL("libcudart.so.13" if torch.version.cuda.startswith("13") else "libcudart.so")
    raw = ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(raw), 1) == 0
    ids = torch.arange(K, dtype=torch.int32, device="cuda")
    inv = torch.cat([ids, torch.full((K,), -1, dtype=torch.int32, device="cuda")])
    g = vt.BlockGraph(torch.randn((1, B, H), device="cuda").to(torch.bfloat16),
                      torch.randn((K, H), device="cuda").to(torch.bfloat16), ids, inv,
                      torch.randn((B, 2, 2 * K), device="cuda"), temperature=0.0)
    torch.cuda.synchronize()
    g.launch(torch.cuda.ExternalStream(raw.value))
    assert rt.cudaStreamSynchronize(raw) == 0 and rt.cudaStreamDestroy(raw) == 0
    assert g.dev_status.tolist() == [0, 0]
    del g
    gc.collect()
    torch.empty(1 << 20, device="cuda").fill_(1.0)
    torch.cuda.synchronize()
