"""Refusals of the scored and shared-prefix calls on the host (none of these reaches a launch)."""
import ctypes
import math

import pytest

import long_context_decode_swa_b200 as rswa
from long_context_decode_swa_b200.binding import Dims, Score

INVALID, UNSUPPORTED = 1, 2
A = ctypes.c_void_p(0x10000)  # aligned stand-in, never dereferenced by a call that fails
MIS = ctypes.c_void_p(0x10008)
DIMS = Dims(2, 4, 128, 128, 64)


def _err():
    return rswa.load().rswa_last_error().decode()


def _scored(**kw):
    lib = rswa.load()
    a = dict(dims=DIMS, score=Score(30.0, None, None, None), q=A, pk=A, pv=A, prefix_len=A, ring_k=A, ring_v=A, wp=A,
             fill=A, scale=0.088, out=A, lse=None, ws=A,
             ws_bytes=lib.rswa_workspace_bytes(ctypes.byref(DIMS), rswa.OP_DECODE_SCORED))
    a.update(kw)
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    code = lib.rswa_decode_scored(ref(a["dims"]), ref(a["score"]), a["q"], a["pk"], a["pv"], a["prefix_len"],
                                  a["ring_k"], a["ring_v"], a["wp"], a["fill"], a["scale"], a["out"], a["lse"],
                                  a["ws"], a["ws_bytes"], None)
    return code, _err()


def _shared(**kw):
    lib = rswa.load()
    a = dict(dims=DIMS, P=3, cap=1000, q=A, sk=A, sv=A, shared_len=A, share_of=A, pk=A, pv=A, prefix_len=A, ring_k=A,
             ring_v=A, wp=A, fill=A, scale=0.088, out=A, lse=None, ws=A,
             ws_bytes=lib.rswa_decode_shared_workspace_bytes(ctypes.byref(DIMS), 3))
    a.update(kw)
    code = lib.rswa_decode_shared(None if a["dims"] is None else ctypes.byref(a["dims"]), a["P"], a["cap"], a["q"],
                                  a["sk"], a["sv"], a["shared_len"], a["share_of"], a["pk"], a["pv"], a["prefix_len"],
                                  a["ring_k"], a["ring_v"], a["wp"], a["fill"], a["scale"], a["out"], a["lse"],
                                  a["ws"], a["ws_bytes"], None)
    return code, _err()


COMMON = [(dict(dims=None), INVALID, "dims"), (dict(dims=Dims(0, 4, 128, 128, 64)), INVALID, "batch"),
          (dict(dims=Dims(65536, 4, 128, 128, 64)), UNSUPPORTED, "batch"),
          (dict(dims=Dims(2, 129, 128, 128, 64)), INVALID, "heads"), (dict(dims=Dims(2, 4, 64, 128, 64)), UNSUPPORTED, "head_dim"),
          (dict(dims=Dims(2, 4, 128, 1025, 64)), INVALID, "ring"), (dict(dims=Dims(2, 4, 128, 128, -1)), INVALID, "prefix_cap"),
          (dict(q=None), INVALID, "q must"), (dict(q=MIS), INVALID, "aligned"), (dict(pk=None), INVALID, "pk"),
          (dict(pv=MIS), INVALID, "aligned"), (dict(prefix_len=None), INVALID, "prefix_len"), (dict(ring_k=None), INVALID, "ring_k"),
          (dict(ring_v=MIS), INVALID, "aligned"), (dict(wp=None), INVALID, "wp"), (dict(fill=None), INVALID, "fill"),
          (dict(out=None), INVALID, "out"), (dict(ws=None), INVALID, "workspace"), (dict(scale=0.0), INVALID, "scale"),
          (dict(scale=math.nan), INVALID, "scale"), (dict(scale=math.inf), INVALID, "scale"),
          (dict(ws_bytes=255), INVALID, "workspace")]


@pytest.mark.parametrize("kw,code,word", COMMON + [
    (dict(score=None), INVALID, "score"), (dict(score=Score(-1.0, None, None, None)), INVALID, "softcap"),
    (dict(score=Score(math.nan, None, None, None)), INVALID, "softcap"),
    (dict(score=Score(math.inf, None, None, None)), INVALID, "softcap"),
    (dict(score=Score(1e-4, None, None, None)), INVALID, "softcap"), (dict(score=Score(1e7, None, None, None)), INVALID, "softcap"),
    (dict(score=Score(0.0, 0x10000, None, None)), INVALID, "slope and pos"),
    (dict(score=Score(0.0, None, 0x10000, None)), INVALID, "slope and pos"),
    (dict(score=Score(0.0, None, None, 0x10004)), INVALID, "range"),
    (dict(dims=Dims(65535, 128, 128, 128, 2 ** 14)), UNSUPPORTED, "2^31 tiles"),
])
def test_decode_scored_refusals(kw, code, word):
    got, msg = _scored(**kw)
    assert got == code and word in msg, (got, msg)


@pytest.mark.parametrize("kw,code,word", COMMON + [
    (dict(sk=None), INVALID, "sk"), (dict(sv=MIS), INVALID, "aligned"), (dict(shared_len=None), INVALID, "shared_len"),
    (dict(share_of=None), INVALID, "share_of"), (dict(P=0), INVALID, "n_shared"), (dict(P=8193), INVALID, "n_shared"),
    (dict(cap=0), INVALID, "shared_cap"), (dict(cap=2 ** 30 + 1), INVALID, "shared_cap"),
    (dict(P=8192, cap=2 ** 20), UNSUPPORTED, "2^31 shared rows"),
    (dict(dims=Dims(65535, 128, 128, 128, 0), P=1, cap=2 ** 24 - 1), UNSUPPORTED, "units"),
])
def test_decode_shared_refusals(kw, code, word):
    got, msg = _shared(**kw)
    assert got == code and word in msg, (got, msg)


def test_workspace_sizes():
    lib = rswa.load()
    need = lib.rswa_workspace_bytes(ctypes.byref(DIMS), rswa.OP_DECODE_SCORED)
    assert need >= 256 and _scored(ws_bytes=need - 1)[0] == INVALID
    shared = lib.rswa_decode_shared_workspace_bytes(ctypes.byref(DIMS), 3)
    assert shared > need and _shared(ws_bytes=shared - 1)[0] == INVALID
    for P in (0, 8193):
        assert lib.rswa_decode_shared_workspace_bytes(ctypes.byref(DIMS), P) == 0 and "n_shared" in _err()
    assert lib.rswa_decode_shared_workspace_bytes(ctypes.byref(Dims(2, 4, 96, 128, 64)), 3) == 0
    with pytest.raises(rswa.RswaError):
        rswa.shared_workspace_bytes(DIMS, 0)
    # one record a (sequence, head) and 256 a CTA, of 132 floats
    assert shared >= 2 * 4 * 132 * 4


def _prefill(**kw):
    lib = rswa.load()
    a = dict(dims=DIMS, score=Score(30.0, None, None, None), T=16, q=A, k_out=A, v_out=A, pk=A, pv=A, prefix_len=A,
             ring_k=A, ring_v=A, wp=A, fill=A, scale=0.088, out=A, lse=None, write_ring=0, ws=A, ws_bytes=256)
    a.update(kw)
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    code = lib.rswa_prefill_scored(ref(a["dims"]), ref(a["score"]), a["T"], a["q"], a["k_out"], a["v_out"], a["pk"],
                                   a["pv"], a["prefix_len"], a["ring_k"], a["ring_v"], a["wp"], a["fill"], a["scale"],
                                   a["out"], a["lse"], a["write_ring"], a["ws"], a["ws_bytes"], None)
    return code, _err()


@pytest.mark.parametrize("kw,code,word", COMMON + [
    (dict(score=None), INVALID, "score"), (dict(score=Score(-0.5, None, None, None)), INVALID, "softcap"),
    (dict(score=Score(0.0, 0x10000, None, None)), INVALID, "slope and pos"),
    (dict(score=Score(0.0, None, None, 0x10004)), INVALID, "range"), (dict(T=0), INVALID, "T must"),
    (dict(k_out=None), INVALID, "k_out"), (dict(v_out=MIS), INVALID, "aligned"), (dict(lse=MIS), INVALID, "aligned"),
    (dict(ring_k=None, ring_v=None, wp=None, fill=None, write_ring=1), INVALID, "write_ring"),
    (dict(T=2 ** 29), UNSUPPORTED, "2^31"), (dict(dims=Dims(64, 64, 128, 128, 2 ** 20)), UNSUPPORTED, "2^31"),
])
def test_prefill_scored_refusals(kw, code, word):
    got, msg = _prefill(**kw)
    assert got == code and word in msg, (got, msg)


def test_integers_past_32_bits_are_refused():
    # (cut to 32 bits they would be a size of 3)
    for n in (2 ** 32 + 3, -2 ** 32 + 3, 2 ** 31):
        with pytest.raises(ValueError, match="n_shared"):
            rswa.shared_workspace_bytes(DIMS, n)
    assert rswa.shared_workspace_bytes(DIMS, 3) == rswa.load().rswa_decode_shared_workspace_bytes(ctypes.byref(DIMS), 3)
