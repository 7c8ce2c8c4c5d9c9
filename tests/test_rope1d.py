"""rswa_rope_1d on the host: its refusals (no call here reaches a launch) and the frequency tables."""
import ctypes
import math

import pytest
import torch

import long_context_decode_swa_b200 as rswa
from long_context_decode_swa_b200.binding import Rope1d

INVALID, UNSUPPORTED = 1, 2
A = ctypes.c_void_p(0x10000)  # aligned stand-in, never dereferenced by a call that fails
MIS = ctypes.c_void_p(0x10008)


def _desc(**kw):
    d = Rope1d(2, 4, 2, 8, 128, 64, 0, 0, 0, 1.0)
    d.q_stride[:] = d.q_out_stride[:] = (4 * 8 * 128, 8 * 128, 128)
    d.k_stride[:] = d.k_out_stride[:] = (2 * 8 * 128, 8 * 128, 128)
    for name, value in kw.items():
        if isinstance(value, tuple):
            getattr(d, name)[:] = value
        else:
            setattr(d, name, value)
    return d


def _call(desc=None, freq="ok", pos=A, q=A, q_out=A, k=A, k_out=A):
    f = (ctypes.c_double * 64)(*([0.5] * 64))
    if isinstance(freq, float):
        f[5] = freq
    lib = rswa.load()
    code = lib.rswa_rope_1d(ctypes.byref(desc or _desc()), None if freq is None else f, pos, q, q_out, k, k_out, None)
    return code, lib.rswa_last_error().decode()


@pytest.mark.parametrize("kw,code,word", [
    (dict(batch=-1), INVALID, "batch"), (dict(tokens=-1), INVALID, "tokens"),
    (dict(heads_q=0), INVALID, "heads_q"), (dict(heads_q=129), INVALID, "heads_q"), (dict(heads_k=129), INVALID, "heads_k"),
    (dict(head_dim=8), UNSUPPORTED, "head_dim"), (dict(head_dim=272), UNSUPPORTED, "head_dim"),
    (dict(head_dim=120), UNSUPPORTED, "head_dim"), (dict(rot_dim=24), UNSUPPORTED, "rot_dim"),
    (dict(rot_dim=144), UNSUPPORTED, "rot_dim"), (dict(rot_dim=0), UNSUPPORTED, "rot_dim"),
    (dict(layout=2), INVALID, "layout"), (dict(dtype=2), UNSUPPORTED, "dtype"),
    (dict(mscale=math.inf), INVALID, "mscale"), (dict(mscale=math.nan), INVALID, "mscale"),
    (dict(q_stride=(4096, 1024, 124)), INVALID, "strides of q "),
    (dict(k_out_stride=(2048, 1020, 128)), INVALID, "strides of k_out"),
    (dict(q_out_stride=(4096, 0, 128)), INVALID, "overlap"),
    (dict(dtype=1, q_stride=(4096, 1024, 126)), INVALID, "strides of q "),
    (dict(q_out_stride=(4096, 2048, 256)), INVALID, "q_out in place"),  # q and q_out are one address here
    (dict(k_stride=(2048, 128, 256)), INVALID, "k_out in place"),
])
def test_descriptor_refusals(kw, code, word):
    got, msg = _call(_desc(**kw))
    assert got == code and word in msg, (got, msg)


@pytest.mark.parametrize("kw,word", [
    (dict(freq=None), "inv_freq"), (dict(freq=math.nan), "inv_freq[5]"), (dict(freq=math.inf), "inv_freq[5]"),
    (dict(pos=None), "pos"), (dict(q=None), "q"), (dict(q_out=MIS), "aligned"), (dict(k=MIS), "aligned"),
    (dict(k_out=None), "k_out"),
])
def test_argument_refusals(kw, word):
    got, msg = _call(**kw)
    assert got == INVALID and word in msg, (got, msg)
    assert rswa.load().rswa_rope_1d(None, None, A, A, A, None, None, None) == INVALID


def test_nothing_to_encode_launches_nothing():
    # empty buffers may be NULL once the descriptor holds
    assert _call(_desc(batch=0), q=None, q_out=None, k=None, k_out=None, pos=None)[0] == 0
    assert _call(_desc(tokens=0), q=None, q_out=None, k=None, k_out=None, pos=None)[0] == 0


def test_binding_refusals():
    x = torch.zeros(1, 2, 3, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rswa.rswa_rope_1d(x, torch.zeros(1, 3, dtype=torch.int32), rswa.rope_freqs(128)[0])
    with pytest.raises(TypeError, match="torch.Tensor"):
        rswa.rswa_rope_1d([1.0], None, None)


def test_rope_freqs_tables():
    f, m = rswa.rope_freqs(64, 10000.0)
    assert m == 1.0 and f.dtype == torch.float64 and f.shape == (32,)
    for i in (0, 7, 31):
        assert math.isclose(f[i].item(), 10000.0 ** (-i / 32), rel_tol=1e-14)
    lin, m = rswa.rope_freqs(64, scaling="linear", factor=4.0)
    assert m == 1.0 and torch.equal(lin, f / 4.0)
    ntk, m = rswa.rope_freqs(64, scaling="ntk", factor=4.0)
    # the fastest pair is kept, the slowest divided by the factor
    assert m == 1.0 and ntk[0] == 1.0 and math.isclose(ntk[31].item(), f[31].item() / 4.0, rel_tol=1e-12)
    parts, m = rswa.rope_freqs(64, scaling="by_parts", factor=8.0, trained=4096)
    assert math.isclose(m, 0.1 * math.log(8.0) + 1.0)
    turns = 4096 * f / (2 * math.pi)
    for i in range(32):
        if turns[i] >= 32:
            assert parts[i] == f[i]
        elif turns[i] <= 1:
            assert parts[i] == f[i] / 8.0
        else:
            assert f[i] / 8.0 < parts[i] < f[i]
    assert (turns >= 32).any() and (turns <= 1).any() and ((turns > 1) & (turns < 32)).any()


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(base=0.0), dict(base=math.inf),
                                dict(scaling="cubic"), dict(scaling="linear", factor=0.5), dict(scaling="ntk", rot_dim=2, factor=2.0),
                                dict(scaling="linear", factor=math.nan), dict(scaling="by_parts", factor=2.0),
                                dict(scaling="by_parts", factor=2.0, trained=0),
                                dict(scaling="by_parts", factor=2.0, trained=64, slow=4.0, fast=4.0)])
def test_rope_freqs_refusals(kw):
    with pytest.raises(ValueError):
        rswa.rope_freqs(**{"rot_dim": 64, **kw})
