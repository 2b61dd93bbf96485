"""Refusals of the 8-bit head and the log probabilities that the host decides
before any device work (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from drafter_sampling_gb300 import build
    build.build()
    from drafter_sampling_gb300 import _lib
    return _lib.load()


FAKE = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(264)       # 8-byte aligned only
BIG = 1 << 30


def _bad():
    from drafter_sampling_gb300 import _lib
    return _lib.VT_ERR_INVALID_ARG, _lib.VT_ERR_UNSUPPORTED, _lib.VT_ERR_WORKSPACE


def test_quantize_head_refusals(lib):
    bad, unsupported, _ = _bad()
    for args in [(None, 4, 64, FAKE, 64, FAKE, FAKE), (FAKE, 4, 64, None, 64, FAKE, FAKE),
                 (FAKE, 4, 64, FAKE, 64, None, FAKE), (FAKE, 4, 64, FAKE, 64, FAKE, None),
                 (FAKE, 0, 64, FAKE, 64, FAKE, FAKE), (FAKE, 4, 0, FAKE, 64, FAKE, FAKE),
                 (FAKE, 4, 65537, FAKE, 65552, FAKE, FAKE),
                 (FAKE, 4, 64, FAKE, 48, FAKE, FAKE),        # stride shorter than a row
                 (FAKE, 4, 60, FAKE, 60, FAKE, FAKE),        # stride not a multiple of 16
                 (FAKE, 4, 64, ODD, 64, FAKE, FAKE)]:        # misaligned W8
        assert lib.vt_quantize_head(*args, None) == bad, args
    assert lib.vt_quantize_head(FAKE, 65535 * 128 + 1, 64, FAKE, 64, FAKE, FAKE, None) == unsupported


def test_fp8_draft_refusals(lib):
    bad, _, ws = _bad()
    assert lib.vt_draft_fp8_workspace_bytes(16, 2048, 32768) > 0
    for B, H, K in [(0, 64, 10), (4097, 64, 10), (4, 0, 10), (4, 65537, 10), (4, 64, 0)]:
        assert lib.vt_draft_fp8_workspace_bytes(B, H, K) == 0
    ok = dict(hidden=FAKE, B=2, H=64, W8=FAKE, ldw=64, sc=FAKE, K=16, T=1.0, out=FAKE, ld=16,
              ws=FAKE, n=BIG)

    def logits(**kw):
        a = {**ok, **kw}
        return lib.vt_draft_logits_fp8(a["hidden"], a["B"], a["H"], a["W8"], a["ldw"], a["sc"],
                                       a["K"], a["T"], a["out"], a["ld"], a["ws"], a["n"], None)
    for kw in [dict(hidden=None), dict(W8=None), dict(sc=None), dict(out=None), dict(B=0),
               dict(B=4097), dict(H=0), dict(K=0), dict(ldw=48), dict(ldw=72), dict(W8=ODD),
               dict(T=0.0), dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")), dict(ld=15)]:
        assert logits(**kw) == bad, kw
    assert logits(ws=None) == ws and logits(ws=ODD) == ws and logits(n=16) == ws

    def step(T=1.0, u=FAKE, ids=FAKE, q=FAKE, ldq=16, tok=FAKE, ldt=1, st=FAKE, w=FAKE, n=BIG):
        return lib.vt_draft_step_fp8(FAKE, 2, 64, FAKE, 64, FAKE, ids, 16, u, T, q, ldq, tok, ldt, st,
                                     w, n, None)
    for kw in [dict(u=None), dict(ids=None), dict(q=None), dict(ldq=15), dict(tok=None), dict(ldt=0),
               dict(st=None), dict(T=-1.0)]:
        assert step(**kw) == bad, kw
    assert step(T=0.0, u=None, w=None) == ws            # greedy: no uniforms needed

    def topk(k=4, K=16, T=1.0, ids=FAKE, n=BIG):
        return lib.vt_draft_topk_fp8(FAKE, 2, 64, FAKE, 64, FAKE, ids, K, k, T, FAKE, FAKE, FAKE, FAKE,
                                     n, None)
    for kw in [dict(k=0), dict(k=33, K=100), dict(k=17), dict(T=0.0), dict(ids=None)]:
        assert topk(**kw) == bad, kw
    assert topk(n=16) == ws
    assert lib.vt_draft_topk_fp8_workspace_bytes(2, 64, 16, 17) == 0


def test_fp8_block_refusals(lib):
    from drafter_sampling_gb300 import _lib
    bad, _, _ = _bad()
    h = ctypes.c_void_p()
    d = _lib.BlockDesc()
    assert lib.vt_block_graph_create_fp8(None, FAKE, 64, FAKE, ctypes.byref(h)) == bad
    assert lib.vt_block_graph_create_fp8(ctypes.byref(d), None, 64, FAKE, ctypes.byref(h)) == bad
    assert lib.vt_block_graph_create_fp8(ctypes.byref(d), FAKE, 64, None, ctypes.byref(h)) == bad
    assert lib.vt_block_graph_create_fp8(ctypes.byref(d), FAKE, 64, FAKE, ctypes.byref(h)) == bad
    assert lib.vt_block_fp8_workspace_bytes(16, 2048, 32768, 128256, 6) >= \
        lib.vt_verify_workspace_bytes(16, 6, 128256, 32768)
    assert lib.vt_block_fp8_workspace_bytes(0, 2048, 32768, 128256, 6) == 0


def test_token_logprobs_refusals(lib):
    bad, _, _ = _bad()
    ok = dict(l=FAKE, dt=0, R=2, V=10, ld=10, tok=FAKE, k=3, T=1.0, lp=FAKE, en=FAKE, ids=FAKE, top=FAKE,
              st=FAKE)

    def call(**kw):
        a = {**ok, **kw}
        return lib.vt_token_logprobs(a["l"], a["dt"], a["R"], a["V"], a["ld"], a["tok"], a["k"], a["T"],
                                     a["lp"], a["en"], a["ids"], a["top"], a["st"], None)
    for kw in [dict(l=None), dict(tok=None), dict(lp=None), dict(st=None), dict(ids=None), dict(top=None),
               dict(dt=2), dict(R=0), dict(R=(1 << 24) + 1), dict(V=0), dict(V=(1 << 22) + 1, ld=1 << 23),
               dict(ld=9), dict(k=-1), dict(k=33, V=100, ld=100), dict(k=11), dict(T=0.0), dict(T=-1.0),
               dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-40),
               dict(l=ctypes.c_void_p(258))]:                  # not aligned to a float
        assert call(**kw) == bad, kw


def test_binding_refusals_name_the_argument():
    torch = pytest.importorskip("torch")
    import drafter_sampling_gb300 as vt
    cpu = torch.zeros((4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        vt.vt_token_logprobs(cpu, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError, match="logits"):
        vt.vt_token_logprobs([0.0], None)
    with pytest.raises(ValueError, match="CUDA"):
        vt.vt_quantize_head(cpu.to(torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        vt.vt_draft_logits_fp8(cpu.to(torch.bfloat16), None, None)
    assert vt.workspace_bytes("draft_fp8", B=2, H=64, K=100) > 0
    assert vt.workspace_bytes("draft_topk_fp8", B=2, H=64, K=100, k=8) > \
        vt.workspace_bytes("draft_fp8", B=2, H=64, K=100)


@pytest.mark.parametrize("K", [65535 * 128 + 1, 2 ** 31 - 256, 2 ** 31 - 100, 2 ** 31 - 1])
def test_heads_of_too_many_rows_are_refused(lib, K):
    # rows beyond the quantiser's, up to where 32-bit counts of their blocks overflow
    _, unsupported, _ = _bad()
    huge = 1 << 50
    assert lib.vt_quantize_head(FAKE, K, 64, FAKE, 64, FAKE, FAKE, None) == unsupported
    for B in (2, 100, 200):
        assert lib.vt_draft_fp8_workspace_bytes(B, 64, K) == 0
        assert lib.vt_draft_topk_fp8_workspace_bytes(B, 64, K, 8) == 0
        assert lib.vt_draft_logits_fp8(FAKE, B, 64, FAKE, 64, FAKE, K, 1.0, FAKE, K, FAKE, huge, None) == unsupported
        for T in (0.0, 1.0):
            assert lib.vt_draft_step_fp8(FAKE, B, 64, FAKE, 64, FAKE, FAKE, K, FAKE, T, FAKE, K, FAKE, 1, FAKE, FAKE,
                                         huge, None) == unsupported
        assert lib.vt_draft_topk_fp8(FAKE, B, 64, FAKE, 64, FAKE, FAKE, K, 8, 1.0, FAKE, FAKE, FAKE, FAKE, huge,
                                     None) == unsupported
    assert lib.vt_draft_fp8_workspace_bytes(2, 64, 65535 * 128) > 0
