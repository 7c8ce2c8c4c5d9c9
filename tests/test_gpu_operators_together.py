"""The rotary, scored and shared-prefix calls used together, as a decoder layer uses them, against plain
64-bit attention over the same rows; their bounded waits; and tensors past 2^31 elements.

Tolerances: those of the calls' own test files (bf16 outputs: 2 * 2^-8 sum w |v| from rounded weights and
2^-8 of the result; f32 outputs: 1e-4 sum w |v|; lse 1e-4)."""
import math
import time

import numpy as np
import pytest
import torch

import long_context_decode_swa_b200 as pkg
from long_context_decode_swa_b200 import binding as bind
from tests import plain64 as P64
from tests.plain64 import D, ints, randn

pytestmark = pytest.mark.gpu


def turn64(x, pos, freq, mscale):
    """Half-layout rotary encoding of the kernel's bf16 rows in f64, rounded to bf16 as the cache holds it."""
    ang = pos.double()[:, None, :, None] * freq.cuda()
    c, s = ang.cos() * mscale, ang.sin() * mscale
    h = freq.shape[0]
    a, b = x[..., :h].double(), x[..., h:2 * h].double()
    return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * h:].double()], -1)


def test_a_layer_generates(cuda_lib):
    # a document of two pages of unequal length for two sequences; a prompt chunk through the scored
    # prefill, then tokens one by one, every key rotated at its position, scores capped and biased
    B, H, n, T, steps = 2, 3, 48, 70, 5
    m, cap = [150, 90], 160
    g = P64.gen(77)
    freq, mscale = pkg.rope_freqs(96, scaling="by_parts", factor=4.0, trained=64)
    m32 = float(np.float32(mscale))
    slopes = torch.tensor([0.5, 0.1, 0.02], device="cuda")
    plen = ints(m)
    raw_pk, pv = randn((B, H, cap, D), g), randn((B, H, cap, D), g)
    pk = torch.empty_like(raw_pk)
    prefix_pos = torch.arange(cap, dtype=torch.int32, device="cuda").expand(B, cap).contiguous()
    pkg.rswa_rope_1d(raw_pk, prefix_pos, freq, q_out=pk, mscale=m32)
    raw_q, raw_k, v = (randn((B, H, T + steps, D), g, s) for s in (2.0, 1.0, 1.0))
    pos = plen[:, None] + torch.arange(T + steps, dtype=torch.int32, device="cuda")
    q, k = torch.empty_like(raw_q), torch.empty_like(raw_k)
    # the chunk in one call, each later token on its own: the same rows either way
    pkg.rswa_rope_1d(raw_q, pos, freq, q_out=q, k=raw_k, k_out=k, mscale=m32)
    for t in range(T, T + steps):
        a, b = pkg.rswa_rope_1d(raw_q[:, :, t].contiguous(), pos[:, t].contiguous(), freq, k=raw_k[:, :, t].contiguous(),
                                mscale=m32)
        assert torch.equal(a, q[:, :, t]) and torch.equal(b, k[:, :, t])
    # the encoded rows are the f64 ones to bf16
    ref_q = turn64(raw_q, pos, freq, m32)
    assert ((q.double() - ref_q).abs() <= 2.0 ** -8 * ref_q.abs() + 2.0 ** -18 * 20).all()

    ranges = ints([[(0, 100) if i % 2 else (60, 150) for i in range(T)], [(10, 90)] * T])
    rk, rv = torch.zeros((B, H, n, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((B, H, n, D), dtype=torch.bfloat16, device="cuda")
    wp, fill = ints([0, 0]), ints([0, 0])
    out = torch.empty((B, H, T, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, H, T), device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = dict(softcap=20.0, slopes=slopes)
    pkg.rswa_prefill_scored(q[:, :, :T].contiguous(), k[:, :, :T].contiguous(), v[:, :, :T].contiguous(), pk, pv, plen,
                            out, ws, pos=plen, ranges=ranges, lse=lse, ring_k=rk, ring_v=rv, wp=wp, fill=fill,
                            write_ring=True, **args)
    assert pkg.check_status(ws) == 0
    got = {t: (out[:, :, t].double(), lse[:, :, t].double(), 2 * 2.0 ** -8 + 2e-4, 2.0 ** -8) for t in range(T)}
    ws = pkg.new_workspace(pkg.dims_of(pk, rk), pkg.OP_DECODE_SCORED)
    step_range = ints([[0, 150], [10, 10]])
    for t in range(T, T + steps):
        pkg.rswa_append(rk, rv, k[:, :, t].contiguous(), v[:, :, t].contiguous(), wp, fill)
        o, e = torch.empty((B, H, D), device="cuda"), torch.empty((B, H), device="cuda")
        pkg.rswa_decode_scored(q[:, :, t].contiguous(), pk, pv, plen, rk, rv, wp, fill, o, ws, pos=pos[:, t].contiguous(),
                               ranges=step_range, lse=e, **args)
        got[t] = (o.double(), e.double(), 2e-4, 0.0)
    assert pkg.check_status(ws) == 0
    for t in range(T + steps):
        for b in range(B):
            lo, hi = (ranges[b, t] if t < T else step_range[b]).tolist()
            first = max(0, t - n + 1)
            at = torch.cat([torch.arange(lo, hi), m[b] + torch.arange(first, t + 1)]).cuda()
            for h in range(H):
                kk = torch.cat([pk[b, h, lo:hi], k[b, h, first:t + 1]]).double()
                vv = torch.cat([pv[b, h, lo:hi], v[b, h, first:t + 1]]).double()
                bias = -slopes[h].double() * (m[b] + t - at).double()[None]
                ref, e, size = P64.attend(q[b, h, t][None].double(), kk, vv, bias, 20.0)
                o, l, by_size, by_ref = got[t]
                assert ((o[b, h] - ref[0]).abs() <= by_size * size[0] + by_ref * ref[0].abs()).all(), (t, b, h)
                assert abs(l[b, h] - e[0]) <= 1e-4 + 2.0 ** -20 * abs(e[0]), (t, b, h)


def test_readers_of_one_document(cuda_lib):
    # steps of several sequences over one shared document, each with its own prompt: rotary, append and
    # shared decode against the same keys as private prefixes, through a captured graph
    B, H, n, m, prompt, steps = 5, 4, 32, 700, 9, 4
    g = P64.gen(78)
    freq, _ = pkg.rope_freqs(128)
    sk, sv = randn((1, H, m, D), g), randn((1, H, m, D), g)
    pkg.rswa_rope_1d(sk, torch.arange(m, dtype=torch.int32, device="cuda")[None], freq)
    pk, pv = randn((B, H, prompt, D), g), randn((B, H, prompt, D), g)
    plen, slen, share = ints([prompt - b for b in range(B)]), ints([m]), ints([0, 0, -1, 0, 0])
    rk, rv = torch.zeros((B, H, n, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((B, H, n, D), dtype=torch.bfloat16, device="cuda")
    wp, fill, pos = ints([0] * B), ints([0] * B), ints([m + prompt] * B)
    q, k, v = (torch.empty((B, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    raw = [randn((steps, B, H, D), g) for _ in range(3)]
    out, lse = torch.empty((B, H, D), dtype=torch.bfloat16, device="cuda"), torch.empty((B, H), device="cuda")
    ws = pkg.new_shared_workspace(pkg.Dims(B, H, D, n, prompt), 1)

    def step():
        pkg.rswa_rope_1d(q, pos, freq, k=k)
        pkg.rswa_append(rk, rv, k, v, wp, fill)
        pkg.rswa_decode_shared(q, sk, sv, slen, share, rk, rv, wp, fill, out, ws, pk=pk, pv=pv, prefix_len=plen, lse=lse)
        pos.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # warm up: its token is overwritten below
    torch.cuda.current_stream().wait_stream(side)
    wp.zero_(), fill.zero_(), pos.fill_(m + prompt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    full_k = torch.zeros((B, H, m + prompt, D), dtype=torch.bfloat16, device="cuda")
    full_v = torch.zeros_like(full_k)
    full_len = []
    for b in range(B):
        s, p = (m if share[b] >= 0 else 0), prompt - b
        full_k[b, :, :s], full_k[b, :, s:s + p] = sk[0, :, :s], pk[b, :, :p]
        full_v[b, :, :s], full_v[b, :, s:s + p] = sv[0, :, :s], pv[b, :, :p]
        full_len.append(s + p)
    ws_d = pkg.new_workspace(pkg.Dims(B, H, D, n, m + prompt), pkg.OP_DECODE)
    ref, ref_lse = torch.empty((B, H, D), device="cuda"), torch.empty((B, H), device="cuda")
    for t in range(steps):
        q.copy_(raw[0][t]), k.copy_(raw[1][t]), v.copy_(raw[2][t])
        graph.replay()
        pkg.rswa_decode(q, full_k, full_v, ints(full_len), rk, rv, wp, fill, ref, ws_d, lse=ref_lse)
        assert fill.tolist() == [t + 1] * B and pos.tolist() == [m + prompt + t + 1] * B
        assert (out.float() - ref).norm() <= 5e-3 * ref.norm()
        assert (lse - ref_lse).abs().max() <= 1e-4
    assert pkg.check_status(ws) == 0


@pytest.mark.parametrize("B,H,cap,drop,dropped", [
    (2, 4, 300, 0, True),      # items cut over CTAs: records and counters in use
    (60, 16, 32, 1, True),     # short items, whole
    (1, 16, 8000, 7, True),    # a warp's second tile (16 x 254 tiles over 296 CTAs: 14 each)
    (1, 16, 4000, 7, False),   # past the first CTA's share (16 x 129 tiles: 7 each, the last is number 6)
])
def test_scored_decode_wait_timeout(cuda_lib, B, H, cap, drop, dropped):
    # the first CTA leaves one tile's copy out (no fault: the bounded wait runs out); the call returns, its
    # status says so, the workspace is restored, and the next call is right
    g = P64.gen(79)
    q, pk, pv = randn((B, H, D), g), randn((B, H, cap, D), g), randn((B, H, cap, D), g)
    rk, rv, wp, fill = P64.ring(B, H, 128, [128] * B, g)
    plen, ws = ints([cap] * B), pkg.new_workspace(pkg.Dims(B, H, D, 128, cap), pkg.OP_DECODE_SCORED)
    out, lse = torch.empty((B, H, D), device="cuda"), torch.empty((B, H), device="cuda")
    run = lambda: pkg.rswa_decode_scored(q, pk, pv, plen, rk, rv, wp, fill, out, ws, softcap=30.0, lse=lse)  # noqa: E731
    run()
    ref = out.clone(), lse.clone()
    pkg.test_arm_wait_timeout(drop, 20_000_000)
    t0 = time.perf_counter()
    run()
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 2.0
    assert pkg.check_status(ws) == (bind.DEVICE_WAIT_TIMEOUT if dropped else 0)
    if not dropped:
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
        return
    assert int(ws.count_nonzero()) == 0
    run()
    assert pkg.check_status(ws) == 0
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_shared_decode_wait_timeout(cuda_lib):
    g = P64.gen(80)
    B, H, m = 6, 4, 300
    q, sk, sv = randn((B, H, D), g), randn((2, H, m, D), g), randn((2, H, m, D), g)
    rk, rv, wp, fill = P64.ring(B, H, 128, [128] * B, g)
    ws = pkg.new_shared_workspace(pkg.Dims(B, H, D, 128, 0), 2)
    out = torch.empty((B, H, D), dtype=torch.bfloat16, device="cuda")
    slen, share = ints([m, m]), ints([b % 2 for b in range(B)])
    run = lambda: pkg.rswa_decode_shared(q, sk, sv, slen, share, rk, rv, wp, fill, out, ws)  # noqa: E731
    run()
    ref = out.clone()
    pkg.test_arm_wait_timeout(0, 20_000_000)
    run()
    assert pkg.check_status(ws) & bind.DEVICE_WAIT_TIMEOUT
    assert int(ws.count_nonzero()) == 0
    run()
    assert pkg.check_status(ws) == 0 and torch.equal(out, ref)


class TestPast32Bits:
    """Offsets past 2^31 elements and 2^32 bytes: the same rows, far into a large buffer and on their own."""

    def test_scored_decode(self, cuda_lib):
        cap, lo, hi = 2 ** 24 + 5000, 2 ** 24 + 4000, 2 ** 24 + 4900
        g = P64.gen(81)
        pk = torch.zeros((1, 1, cap, D), dtype=torch.bfloat16, device="cuda")
        pv = torch.zeros_like(pk)
        pk[:, :, lo:hi], pv[:, :, lo:hi] = randn((1, 1, hi - lo, D), g), randn((1, 1, hi - lo, D), g)
        q = randn((1, 1, D), g)
        rk, rv, wp, fill = P64.ring(1, 1, 128, [0], g)
        outs = []
        for k, v, r, c in ((pk, pv, [lo, hi], cap), (pk[:, :, lo:hi].contiguous(), pv[:, :, lo:hi].contiguous(), [0, hi - lo], hi - lo)):
            ws = pkg.new_workspace(pkg.Dims(1, 1, D, 128, c), pkg.OP_DECODE_SCORED)
            out, lse = torch.empty((1, 1, D), device="cuda"), torch.empty((1, 1), device="cuda")
            pkg.rswa_decode_scored(q, k, v, ints([c]), rk, rv, wp, fill, out, ws, softcap=20.0, ranges=ints([r]), lse=lse)
            assert pkg.check_status(ws) == 0
            outs.append((out, lse))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])

    def test_shared_decode_and_prefill(self, cuda_lib):
        # the second prefix (sequence) starts 2^31 elements in
        cap, m, T = 2 ** 24 + 128, 700, 40
        g = P64.gen(82)
        sk = torch.zeros((2, 1, cap, D), dtype=torch.bfloat16, device="cuda")
        sv = torch.zeros_like(sk)
        sk[1, :, :m], sv[1, :, :m] = randn((1, m, D), g), randn((1, m, D), g)
        small_k, small_v = sk[:, :, :m].contiguous(), sv[:, :, :m].contiguous()
        q = randn((2, 1, D), g)
        rk, rv, wp, fill = P64.ring(2, 1, 128, [3, 128], g)
        share, slen = ints([1, 1]), ints([0, m])
        ws = pkg.new_shared_workspace(pkg.Dims(2, 1, D, 128, 0), 2)
        outs = []
        for k, v in ((sk, sv), (small_k, small_v)):
            out = torch.empty((2, 1, D), dtype=torch.bfloat16, device="cuda")
            pkg.rswa_decode_shared(q, k, v, slen, share, rk, rv, wp, fill, out, ws)
            assert pkg.check_status(ws) == 0
            outs.append(out)
        assert torch.equal(outs[0], outs[1])
        qt, ko, vo = (randn((2, 1, T, D), g) for _ in range(3))
        outs = []
        for k, v in ((sk, sv), (small_k, small_v)):
            out = torch.empty((2, 1, T, D), dtype=torch.bfloat16, device="cuda")
            pkg.rswa_prefill_scored(qt, ko, vo, k, v, slen, out, torch.zeros(256, dtype=torch.uint8, device="cuda"),
                                    softcap=20.0, ring=128, ranges=ints([[(0, 0)] * T, [(5, m)] * T]))
            outs.append(out)
        # the two calls may cut the keys over clusters differently (by capacity): bf16 outputs to a step
        assert (outs[0].float() - outs[1].float()).abs().max() <= 2.0 ** -7 * outs[1].float().abs().max()

    def test_rope(self, cuda_lib):
        far = 2 ** 31 + 4096
        x = torch.zeros(far + 2 * 128, dtype=torch.bfloat16, device="cuda")
        g = P64.gen(83)
        view = x.as_strided((2, 1, 2, 128), (far, 128, 128, 1))
        view.copy_(randn((2, 1, 2, 128), g))
        freq, _ = pkg.rope_freqs(64)
        pos = ints([[1, 2], [3, 4]])
        near, _ = pkg.rswa_rope_1d(view.contiguous(), pos, freq)
        pkg.rswa_rope_1d(view, pos, freq)
        assert torch.equal(view, near)


def _gives_up_and_recovers(run, ws, drop):
    """run(): the outputs of a call on workspace ws. One dropped tile, then the call as before."""
    ref = [t.clone() for t in run()]
    assert pkg.check_status(ws) == 0
    pkg.test_arm_wait_timeout(drop, 20_000_000)
    t0 = time.perf_counter()
    run()
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 2.0
    assert pkg.check_status(ws) == bind.DEVICE_WAIT_TIMEOUT
    assert int(ws.count_nonzero()) == 0
    for got, want in zip(run(), ref):
        assert torch.equal(got, want)
    assert pkg.check_status(ws) == 0


@pytest.mark.parametrize("B,P,H,m,drop", [
    (6, 2, 4, 300, 0),       # 24 key tiles over 24 CTAs
    (40, 16, 12, 300, 1),    # four tiles a CTA in two segments: the second of the first segment,
    (40, 16, 12, 300, 3),    # the last of all: every copy has been issued when its wait runs out
    (200, 1, 5, 9000, 2),    # both query tiles: 355 key tiles, three a CTA
    (420, 2, 2, 5000, 0),    # the same, grouped by a launch of its own
])
def test_shared_part_wait_timeout(cuda_lib, B, P, H, m, drop):
    g = P64.gen(84)
    q, sk, sv = randn((B, H, D), g), randn((P, H, m, D), g), randn((P, H, m, D), g)
    rk, rv, wp, fill = P64.ring(B, H, 16, [16] * B, g)
    ws = pkg.new_shared_workspace(pkg.Dims(B, H, D, 16, 0), P)
    slen, share = ints([m] * P), ints([b % P for b in range(B)])

    def run():
        out, lse = torch.empty((B, H, D), dtype=torch.bfloat16, device="cuda"), torch.empty((B, H), device="cuda")
        pkg.rswa_decode_shared(q, sk, sv, slen, share, rk, rv, wp, fill, out, ws, lse=lse)
        return out, lse

    _gives_up_and_recovers(run, ws, bind.TEST_SHARED_PART + drop)


@pytest.mark.parametrize("softcap,bias", [(0.0, False), (50.0, True)])
@pytest.mark.parametrize("B,H,T,cap,drop", [
    (1, 1, 100, 300, 0), (1, 1, 100, 300, 1),   # two key tiles a CTA, one a stream
    (1, 3, 130, 2000, 0),                       # over a cluster of eight: two or three key tiles a CTA
    (1, 3, 130, 2000, 1),
    (2, 80, 300, 400, 0), (2, 80, 300, 400, 2),  # paired query tiles and, started early, a split rest
    (2, 80, 300, 400, 5),                       # the last key tile: every copy has been issued when its wait runs out
])
def test_prefill_wait_timeout(cuda_lib, B, H, T, cap, drop, softcap, bias):
    g = P64.gen(85)
    q, ko, vo = (randn((B, H, T, D), g) for _ in range(3))
    pk, pv = randn((B, H, cap, D), g), randn((B, H, cap, D), g)
    ws, plen = torch.zeros(256, dtype=torch.uint8, device="cuda"), ints([cap] * B)
    score = dict(slopes=torch.full((H,), 0.02, device="cuda"), pos=plen) if bias else {}

    def run():
        out, lse = torch.empty((B, H, T, D), dtype=torch.bfloat16, device="cuda"), torch.empty((B, H, T), device="cuda")
        pkg.rswa_prefill_scored(q, ko, vo, pk, pv, plen, out, ws, softcap=softcap, lse=lse, ring=128, **score)
        return out, lse

    _gives_up_and_recovers(run, ws, drop)
