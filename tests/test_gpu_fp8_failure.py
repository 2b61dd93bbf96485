"""The 8-bit product when a wait of its promoting threads runs out: vt_selftest_draft_fp8 makes them give up
at a chosen item of each thread block.  Nothing faults or hangs: the other waits are bounded (about a second),
the status word says so, and the next call is right.
"""
import pytest

torch = pytest.importorskip("torch")

# (B, H, K, other scales): a narrow tile, one CTA and a pair of CTAs an item, with scales that the tensor cores
# apply and others; more than one item for some blocks
CASES = [(3, 300, 45000, False), (100, 300, 45000, False), (100, 300, 45000, True), (256, 4500, 41000, False),
         (256, 300, 41000, True)]


def _run(vt, give_up, B, H, K, other):
    g = torch.Generator(device="cuda")
    g.manual_seed(B + H)
    hid = torch.randn((B, H), generator=g, device="cuda").to(torch.bfloat16)
    W8, s, _ = vt.vt_quantize_head(torch.randn((K, H), generator=g, device="cuda").to(torch.bfloat16))
    if other:
        s = s * 1.5
    z = torch.full((B, K), -7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(vt.workspace_bytes("draft_fp8", B=B, H=H, K=K), dtype=torch.uint8, device="cuda")
    rc = vt.lib().vt_selftest_draft_fp8(give_up, hid.data_ptr(), B, H, W8.data_ptr(), W8.stride(0), s.data_ptr(), K,
                                        1.0, z.data_ptr(), K, st.data_ptr(), ws.data_ptr(), ws.numel(),
                                        torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    return z, int(st.item()), vt.vt_draft_logits_fp8(hid, W8, s)


def _first_rows(B):
    """Rows of the head that are some block's item 0."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return 2 * sms * 128 if B <= 64 else sms * 256 if B <= 128 else sms // 2 * 256


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,K,other", CASES)
def test_items_after_a_wait_that_ran_out_are_not_stored(B, H, K, other):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import drafter_sampling_gb300 as vt
    z, status, want = _run(vt, -1, B, H, K, other)
    assert status == 0 and torch.equal(z, want)
    z, status, want = _run(vt, 1, B, H, K, other)
    n = _first_rows(B)
    assert status == vt.VT_DEV_TIMEOUT and n < K
    assert torch.equal(z[:, :n], want[:, :n])
    assert bool(((z[:, n:] == -7.0) | z[:, n:].isnan()).all())


def test_selftest_refusals():
    import ctypes

    from drafter_sampling_gb300 import _lib, build
    build.build()
    lib, fake = _lib.load(), ctypes.c_void_p(256)

    def call(give_up=0, z=fake, st=fake, n=1 << 20, ld=16):
        return lib.vt_selftest_draft_fp8(give_up, fake, 2, 64, fake, 64, fake, 16, 1.0, z, ld, st, fake, n, None)
    for kw in (dict(give_up=-2), dict(give_up=65536), dict(z=None), dict(st=None), dict(ld=15)):
        assert call(**kw) == _lib.VT_ERR_INVALID_ARG, kw
    assert call(n=16) == _lib.VT_ERR_WORKSPACE


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,K,other", CASES + [(64, 300, 300, False), (200, 300, 333, False)])
def test_logits_that_were_not_computed_are_nan(B, H, K, other):
    # vt_draft_logits_fp8 has no status word to say so
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import drafter_sampling_gb300 as vt
    n = _first_rows(B)
    z, status, want = _run(vt, 1 if n < K else 0, B, H, K, other)
    n = n if n < K else 0
    assert status == vt.VT_DEV_TIMEOUT
    assert torch.equal(z[:, :n], want[:, :n]) and bool(z[:, n:].isnan().all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0.0, 1.0])
@pytest.mark.parametrize("B", [3, 100, 256])
def test_a_long_predecessor_is_no_timeout(B, T):
    """The product may start while a kernel ahead of the call, which let its successors start, has two seconds to
    run; the limits of its waits, about a second, count from that kernel's end."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import drafter_sampling_gb300 as vt
    H, K = 300, 5000
    g = torch.Generator(device="cuda")
    g.manual_seed(B)
    hid = torch.randn((B, H), generator=g, device="cuda").to(torch.bfloat16)
    W8, s, _ = vt.vt_quantize_head(torch.randn((K, H), generator=g, device="cuda").to(torch.bfloat16))
    ids = torch.arange(K, dtype=torch.int32, device="cuda")
    u = torch.rand(B, generator=g, device="cuda")
    want = vt.vt_draft_step_fp8(hid, W8, s, ids, u, T)
    got = [torch.empty_like(t) for t in want]
    ws = torch.empty(vt.workspace_bytes("draft_fp8", B=B, H=H, K=K), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert vt.lib().vt_selftest_overlap(1 << 19, torch.cuda.current_stream().cuda_stream) == 0
    vt.vt_draft_step_fp8(hid, W8, s, ids, u, T, q=got[0], tokens=got[1], dev_status=got[2], workspace=ws)
    torch.cuda.synchronize()
    assert int(got[2].item()) == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_overlap_refusals():
    from drafter_sampling_gb300 import _lib, build
    build.build()
    lib = _lib.load()
    assert lib.vt_selftest_overlap(0, None) == _lib.VT_ERR_INVALID_ARG
    assert lib.vt_selftest_overlap((1 << 20) + 1, None) == _lib.VT_ERR_INVALID_ARG
