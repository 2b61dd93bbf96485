"""Calls from other host threads than the main one, and from two at once (the binding gives up the
interpreter's lock during a call)."""
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import drafter_sampling_gb300 as m
    from drafter_sampling_gb300 import build
    build.build()
    m.lib()
    return m


def _fp8(vt, i):
    B, H, K = 50, 300, (1003, 20000)[i]       # no block with a second item, and some with one
    W8, s, _ = vt.vt_quantize_head(torch.randn((K, H), device="cuda").to(torch.bfloat16))
    hid = torch.randn((B, H), device="cuda").to(torch.bfloat16)
    ids = torch.arange(K, dtype=torch.int32, device="cuda")
    out = dict(q=torch.empty((B, K), device="cuda"), tokens=torch.empty(B, dtype=torch.int32, device="cuda"),
               dev_status=torch.empty(1, dtype=torch.int32, device="cuda"),
               workspace=torch.empty(vt.workspace_bytes("draft_fp8", B=B, H=H, K=K), dtype=torch.uint8, device="cuda"))
    return lambda st: vt.vt_draft_step_fp8(hid, W8, s, ids, None, 0.0, stream=st, **out)


def _bf16(vt, i):
    B, H, K = 16, (2000, 2001, 4001)[i], 700  # 16-byte aligned rows (tensor cores), and others
    W = torch.randn((K, H), device="cuda").to(torch.bfloat16)
    hid = torch.randn((B, H), device="cuda").to(torch.bfloat16)
    out = dict(logits=torch.empty((B, K), device="cuda"),
               workspace=torch.empty(vt.workspace_bytes("draft", B=B, H=H, K=K), dtype=torch.uint8, device="cuda"))
    return lambda st: (vt.vt_draft_logits(hid, W, stream=st, **out),)


@pytest.mark.parametrize("make", [_fp8, _bf16])
@pytest.mark.parametrize("bound", [False, True])
def test_first_call_of_a_thread(vt, make, bound):
    # a thread that has made no CUDA call before has no current context yet
    fn = make(vt, 0)
    st = torch.cuda.Stream()
    want = [t.clone() for t in fn(None)]
    torch.cuda.synchronize()
    failed, got = [], []

    def run():
        try:
            if bound:
                torch.cuda.synchronize()
            got.extend(fn(st))
        except Exception as e:                # noqa: BLE001 (reported below, from the main thread)
            failed.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def _calibrate(vt, i):
    V, K = (3001, 400003)[i], 100
    ids = torch.randint(0, V, (20000,), dtype=torch.int32, device="cuda")
    out = dict(counts=torch.empty(V, dtype=torch.int32, device="cuda"),
               topk_ids=torch.empty(K, dtype=torch.int32, device="cuda"),
               dev_status=torch.empty(1, dtype=torch.int32, device="cuda"),
               workspace=torch.empty(vt.workspace_bytes("calibrate", n=20000, V=V, K=K), dtype=torch.uint8,
                                     device="cuda"))
    return lambda st: vt.vt_calibrate_topk(ids, V, K, stream=st, **out)


@pytest.mark.parametrize("make,calls", [(_fp8, 20000), (_bf16, 20000), (_calibrate, 5000)])
def test_two_threads_at_once(vt, make, calls):
    """Of sizes for which one kernel is launched with different amounts of shared memory."""
    fns = [make(vt, i) for i in ((1, 2) if make is _bf16 else (0, 1))]
    want = [[t.clone() for t in f(None)] for f in fns]
    torch.cuda.synchronize()
    failed, got = [], [None, None]

    def run(i):
        st = torch.cuda.Stream()
        try:
            for n in range(calls):
                got[i] = fns[i](st)
                if n % 100 == 99:             # no more in flight than the launch queue takes
                    st.synchronize()
        except Exception as e:                # noqa: BLE001 (reported below, from the main thread)
            failed.append((i, n, e))
        st.synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
