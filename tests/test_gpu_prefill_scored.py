"""GPU parity of rswa_prefill_scored with plain 64-bit attention.

Tolerances: P is rounded to bf16 (half a step: 2^-8 of a weight) in P V and in the normaliser alike, so an
output moves by at most 2 * 2^-8 sum w |v|, and the result is rounded to bf16 (2^-8 of it). A score
errs by less than 1e-4: 2^-20 of sum |q k| scale (|q| about 4 |k|: 44) for the dot, 4 * 2^-23 * cap log2(e)
for the capped form at cap 50, and 2^-23 of a bias that matters. Over a tensor the two independent
roundings have a relative 2-norm near sqrt(2) 2^-8 / sqrt(3) = 3.2e-3: 5e-3 is asserted where rows
average over many keys. lse comes from unrounded weights: 1e-4."""
import math
import time

import pytest
import torch

import long_context_decode_swa_b200 as pkg
from long_context_decode_swa_b200 import binding as bind
from tests import plain64 as P64
from tests.plain64 import D, ints, nan_past, randn

pytestmark = pytest.mark.gpu


def slopes_of(H):
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


class Case:
    def __init__(self, B, H, T, cap, n=128, plen=None, fill=None, softcap=0.0, slopes=None, pos=None, ranges=None,
                 qstd=4.0, seed=0, scale=None):
        g = P64.gen(3000 + seed)
        self.scale = scale
        self.B, self.H, self.T, self.cap, self.n, self.softcap = B, H, T, cap, n, softcap
        self.q, self.ko, self.vo = randn((B, H, T, D), g, qstd), randn((B, H, T, D), g), randn((B, H, T, D), g)
        self.plen = ints(plen if plen is not None else [cap] * B)
        self.pk, self.pv = (nan_past(randn((B, H, cap, D), g), self.plen) for _ in range(2))
        self.has_ring = fill is not None
        if self.has_ring:
            self.rk, self.rv, self.wp, self.fill = P64.ring(B, H, n, fill, g)
        self.slopes = None if slopes is None else torch.tensor(slopes, device="cuda", dtype=torch.float32)
        self.pos = None if pos is None else ints(pos)
        self.ranges = None if ranges is None else ints(ranges)
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def run(self, stream=None, write_ring=False, ws=None):
        out = torch.full((self.B, self.H, self.T, D), math.nan, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.B, self.H, self.T), math.nan, device="cuda")
        ring = dict(ring_k=self.rk, ring_v=self.rv, wp=self.wp, fill=self.fill) if self.has_ring else dict(ring=self.n)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        pkg.rswa_prefill_scored(self.q, self.ko, self.vo, self.pk, self.pv, self.plen, out, self.ws if ws is None else ws,
                                softcap=self.softcap, slopes=self.slopes, pos=self.pos, ranges=self.ranges, lse=lse,
                                write_ring=write_ring, stream=stream, scale=self.scale, **ring)
        return out, lse

    def check(self, out, lse, rel=5e-3):
        out, lse = out.double(), lse.double()
        T, n = self.T, self.n
        i = torch.arange(T, device="cuda")[:, None]
        worst, total, off = 0.0, 0.0, 0.0
        for b in range(self.B):
            m = self.plen[b].item()
            f = self.fill[b].item() if self.has_ring else 0
            at = torch.cat([torch.arange(m) - 10 ** 9, torch.arange(-f, T)]).cuda()[None]  # the band's line from the chunk
            seen = (at <= i) & (at > i - n)
            row = torch.arange(m, device="cuda")[None]
            if self.ranges is None:
                seen[:, :m] = True
            else:
                seen[:, :m] = (row >= self.ranges[b, :, :1]) & (row < self.ranges[b, :, 1:])
            for h in range(self.H):
                k, v = [self.pk[b, h, :m]], [self.pv[b, h, :m]]
                if f:
                    slots = P64.slots_oldest_first(self.wp[b].item(), f, n)
                    k.append(self.rk[b, h][slots]), v.append(self.rv[b, h][slots])
                k, v = torch.cat(k + [self.ko[b, h]]).double(), torch.cat(v + [self.vo[b, h]]).double()
                bias = torch.zeros(seen.shape, dtype=torch.float64, device="cuda")
                if self.slopes is not None:
                    away = torch.cat([self.pos[b] + i - row, i - at[:, m:]], 1)
                    bias = -self.slopes[h].double() * away.double()
                bias = bias.masked_fill(~seen, -math.inf)
                # rows of the prefix that nobody sees may hold anything
                dead = ~seen.any(0)
                k, v = k.masked_fill(dead[:, None], 0.0), v.masked_fill(dead[:, None], 0.0)
                o, e, size = P64.attend(self.q[b, h].double(), k, v, bias, self.softcap, self.scale)
                err = (out[b, h] - o).abs()
                bound = (2 * 2.0 ** -8 + 2e-4) * size + 2.0 ** -8 * o.abs() + 1e-30
                assert (err <= bound).all(), (b, h, (err - bound).max().item(), torch.nonzero(err > bound)[0].tolist())
                assert ((lse[b, h] - e).abs() <= 1e-4 + 2.0 ** -22 * e.abs()).all(), (b, h, (lse[b, h] - e).abs().max().item())
                total, off = total + o.square().sum().item(), off + err.square().sum().item()
        assert math.sqrt(off) <= rel * math.sqrt(total)
        assert pkg.check_status(self.ws) == 0


@pytest.mark.parametrize("B,H,T,cap,n,fill", [
    (1, 1, 1, 1, 1, None), (1, 1, 1, 1, 1, [1]), (1, 2, 5, 127, 7, [3]), (2, 1, 128, 128, 128, [128, 0]),
    (1, 2, 129, 129, 128, [77]), (2, 2, 257, 300, 100, [100, 1]), (1, 1, 700, 1000, 300, [299]),
    (1, 1, 300, 500, 1024, [1000]), (2, 3, 64, 2592, 128, None),
    (1, 1, 10, 5000, 128, [128]), (1, 3, 130, 2000, 64, [9]),   # one query tile's keys over a cluster
    (5, 16, 300, 400, 128, [128, 0, 64, 1, 127]),               # more 256-query tiles than SMs
])
@pytest.mark.parametrize("softcap,bias", [(0.0, False), (20.0, False), (0.0, True), (50.0, True)])
def test_matches_plain_attention(cuda_lib, B, H, T, cap, n, fill, softcap, bias):
    plen = [cap - (b * 37) % cap for b in range(B)]
    c = Case(B, H, T, cap, n, plen, fill, softcap, slopes_of(H) if bias else None,
             [m + 9 * b for b, m in enumerate(plen)] if bias else None, seed=B * 7 + T + cap)
    c.check(*c.run(), rel=5e-3 if T * H > 100 else 8e-3)


def documents(T, cuts, order, each):
    docs = list(zip(cuts, cuts[1:]))
    return [docs[order[min(i // each, len(order) - 1)]] for i in range(T)]


@pytest.mark.parametrize("softcap,bias", [(0.0, False), (30.0, False), (0.0, True), (50.0, True)])
def test_documents(cuda_lib, softcap, bias):
    T, cap = 520, 1500
    cuts = [0, 100, 101, 400, 777, 900, 1200, 1500]
    ranges = [
        documents(T, cuts, [0, 1, 2, 3, 4, 5, 6], 75),     # in order
        documents(T, cuts, [6, 0, 5, 1, 4, 2, 3], 40),     # six documents in a query tile, out of order
        [(min(3 * i, 1400), min(3 * i, 1400) + (i % 3) * 40) for i in range(T)],  # a moving window, every third empty
        documents(T, [0, 1500], [0], T),
    ]
    c = Case(4, 2, T, cap, ranges=ranges, fill=[128, 5, 0, 128], softcap=softcap, slopes=slopes_of(2) if bias else None,
             pos=[1500, 1700, 1500, 40000] if bias else None, seed=50)
    c.check(*c.run())


@pytest.mark.parametrize("softcap,bias", [(0.0, False), (30.0, True)])
def test_documents_of_many_sequences(cuda_lib, softcap, bias):
    # as many 256-query tiles as the chip takes at once: tiles of queries share their key tiles
    B, T, cap = 12, 300, 700
    cuts = [0, 100, 101, 400, 650, 700]
    orders = [[0, 1, 2, 3, 4], [4, 0, 3, 1, 2], [2, 2, 2, 2, 2], [3, 0, 3, 0, 3]]
    c = Case(B, 16, T, cap, ranges=[documents(T, cuts, orders[b % 4], 61 + b) for b in range(B)],
             fill=[(11 * b) % 129 for b in range(B)], softcap=softcap, slopes=slopes_of(16) if bias else None,
             pos=[700 + b for b in range(B)] if bias else None, seed=60)
    c.check(*c.run())


@pytest.mark.parametrize("qscale", [1.0, 4.0, 30.0])
@pytest.mark.parametrize("softcap", [5.0, 20.0, 1000.0])
def test_caps_from_barely_to_fully_saturated(cuda_lib, softcap, qscale):
    # |scale q.k| / cap from 0.01 to 50: both polynomials and the exponential form, within one warp too
    c = Case(1, 2, 150, 300, softcap=softcap, fill=[100], qstd=qscale, seed=61)
    c.q[:, :, ::3] *= 0.05
    out, lse = c.run()
    # a score of s errs by at most 2^-20 sum |q k| scale before the cap, which only shrinks it
    extra = 2.0 ** -20 * qscale * 2 * math.sqrt(D) if softcap == 1000.0 else 0.0
    if extra < 1e-4:
        c.check(out, lse, rel=8e-3)
    else:
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_what_lies_outside_the_documents_stays_there(cuda_lib):
    # NaN and infinities in prefix rows that no query of a 256-query tile sees: before, between
    # and after the documents, in the same key tiles as seen rows; more than four separate runs too
    T, cap = 400, 1400
    ranges = [[(130, 200) if i < 100 else (260, 300) for i in range(T)],
              [(50 + 200 * (i % 7), 90 + 200 * (i % 7)) for i in range(T)],
              [(0, 0)] * T]
    c = Case(3, 2, T, cap, ranges=ranges, softcap=30.0, seed=51)
    for b, r in enumerate(ranges):
        seen = torch.zeros(cap, dtype=torch.bool, device="cuda")
        for lo, hi in set(r):
            seen[lo:hi] = True
        c.pk[b].masked_fill_(~seen[None, :, None], math.nan)
        c.pv[b].masked_fill_(~seen[None, :, None], math.inf)
    c.check(*c.run())


@pytest.mark.parametrize("slope", [0.7, -0.02])
def test_bias_across_a_far_document(cuda_lib, slope):
    # the document lies after the query (negative distances), far before it, and around it
    T = 40
    c = Case(3, 1, T, 600, n=16, fill=[16, 3, 0], slopes=[slope], pos=[100, 10 ** 6, 300], ranges=[[(200, 600)] * T] * 3,
             seed=52)
    c.check(*c.run(), rel=8e-3)


@pytest.mark.parametrize("softcap", [0.0, 50.0])
def test_gentle_and_steep_slopes_of_many_queries(cuda_lib, softcap):
    # more 256-query tiles than SMs; where a slope moves the bias little along a tile, the tile's largest
    # score is bounded rather than found
    slopes = [0.7, -0.7, 0.34, -0.34, 0.36, -0.36, 0.02, -0.02, 0.0, 4.0, -4.0] * 7
    c = Case(1, 77, 511, 290, fill=[100], softcap=softcap, slopes=slopes, pos=[290], seed=61, qstd=4.0)
    c.check(*c.run())


@pytest.mark.parametrize("softcap,scale", [(1e-3, None), (0.5, None), (1e6, None), (30.0, 1e-9), (1e-3, 3.0), (1e6, 1e-4)])
def test_extreme_caps_and_scales(cuda_lib, softcap, scale):
    # scores far above and far below the cap, and products of the two far from 1
    c = Case(1, 2, 200, 300, fill=[60], softcap=softcap, seed=62, qstd=1.0, scale=scale)
    c.check(*c.run())


def test_rows_far_below_their_maximum(cuda_lib):
    # weights from 1 down past the least of f32, in whole tiles
    c = Case(1, 80, 300, 700, fill=[128], seed=63, qstd=20.0)
    c.check(*c.run(), rel=8e-3)  # outputs are one row of V: no averaging, rounding alone


@pytest.mark.parametrize("softcap,bias,B,H", [(0.0, False, 1, 8), (20.0, False, 1, 8), (0.0, True, 1, 8), (20.0, True, 1, 8),
                                              (0.0, False, 2, 80)])
def test_a_nan_key_that_is_seen_shows(cuda_lib, softcap, bias, B, H):
    # one key of each head, in each place of eight: no query's output hides it
    c = Case(B, H, 150, 400, fill=[128] * B, softcap=softcap, slopes=slopes_of(H) if bias else None,
             pos=[400] * B if bias else None, seed=64)
    for h in range(H):
        c.pk[:, h, 128 + h % 8, 5] = math.nan
    out, lse = c.run()
    assert not torch.isfinite(out).any() and not torch.isfinite(lse).any()


def test_plain_scores_agree_with_rswa_prefill(cuda_lib):
    c = Case(2, 3, 300, 700, plen=[700, 333], fill=[128, 60], qstd=1.0, seed=53)
    out, lse = c.run()
    ref = torch.empty(out.shape, device="cuda")
    ref_lse = torch.empty_like(lse)
    pkg.rswa_prefill(c.q, c.ko, c.vo, c.pk, c.pv, c.plen, ref, torch.zeros_like(c.ws), lse=ref_lse, ring_k=c.rk,
                     ring_v=c.rv, wp=c.wp, fill=c.fill)
    assert (out.float() - ref).norm() <= 3e-3 * ref.norm()
    assert (lse - ref_lse).abs().max() <= 1e-5


@pytest.mark.parametrize("T,n", [(1, 128), (50, 128), (128, 128), (300, 128), (5, 3)])
def test_write_ring_equals_appends_and_the_next_chunk(cuda_lib, T, n):
    c = Case(3, 2, T, 200, n=n, fill=[0, n, n // 2], softcap=20.0, seed=54 + T)
    rk, rv, wp, fill = c.rk.clone(), c.rv.clone(), c.wp.clone(), c.fill.clone()
    keep = c.run()
    out, lse = c.run(write_ring=True)
    assert torch.equal(out, keep[0]) and torch.equal(lse, keep[1])
    for t in range(T):
        pkg.rswa_append(rk, rv, c.ko[:, :, t].contiguous(), c.vo[:, :, t].contiguous(), wp, fill)
    assert torch.equal(c.wp, wp) and torch.equal(c.fill, fill)
    assert torch.equal(c.rk.view(torch.int16), rk.view(torch.int16)) and torch.equal(c.rv.view(torch.int16), rv.view(torch.int16))


def test_last_query_equals_a_decode_step(cuda_lib):
    # prefill of T outputs against rswa_decode_scored after appending them
    T = 70
    c = Case(2, 3, T, 500, fill=[128, 20], softcap=40.0, slopes=slopes_of(3), pos=[500, 800],
             ranges=[[(10, 400)] * T, [(100, 101)] * T], seed=55)
    out, lse = c.run(write_ring=True)
    d_out, d_lse = torch.empty((2, 3, D), device="cuda"), torch.empty((2, 3), device="cuda")
    ws = pkg.new_workspace(pkg.dims_of(c.pk, c.rk), pkg.OP_DECODE_SCORED)
    pkg.rswa_decode_scored(c.q[:, :, -1].contiguous(), c.pk, c.pv, c.plen, c.rk, c.rv, c.wp, c.fill, d_out, ws,
                           softcap=40.0, slopes=c.slopes, pos=c.pos + T - 1, ranges=c.ranges[:, -1].contiguous(), lse=d_lse)
    assert (out[:, :, -1].float() - d_out).norm() <= 8e-3 * d_out.norm()
    assert (lse[:, :, -1] - d_lse).abs().max() <= 1e-4


def test_streams_graph_and_repeats(cuda_lib):
    c = Case(2, 2, 300, 600, fill=[128, 128], softcap=50.0, slopes=slopes_of(2), pos=[600, 700],
             ranges=[[(0, 300)] * 150 + [(300, 600)] * 150] * 2, seed=56)
    ref = c.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [c.run(stream=s1), c.run(stream=s2, ws=torch.zeros_like(c.ws))]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], ref[0]) and torch.equal(o[1], ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = c.run()
    c.ranges[:, :200] = ints([7, 500])
    c.pos += 3
    graph.replay()
    torch.cuda.synchronize()
    c.check(out, lse)


def test_device_checks(cuda_lib):
    T = 20
    c = Case(4, 2, T, 300, fill=[128] * 4, slopes=[0.5, 0.25], pos=[300] * 4, ranges=[[(0, 300)] * T] * 4, seed=57)
    c.ranges[0, 3] = ints([-1, 50])
    c.ranges[0, 4] = ints([0, 301])
    c.pos[1] = -5
    c.plen[2] = -1
    c.wp[3] = -1
    out, lse = c.run()
    assert pkg.check_status(c.ws) == bind.DEVICE_BAD_RANGE | bind.DEVICE_BAD_POS | bind.DEVICE_BAD_PREFIX_LEN | \
        bind.DEVICE_BAD_RING_STATE
    c.ranges[0, 3:5] = 0
    c.ranges[1:3] = 0
    c.pos[1] = 300
    c.plen[2] = 0
    c.wp[3] = c.fill[3] = 0
    c.check(out, lse)


def test_no_prefix_at_all(cuda_lib):
    c = Case(2, 2, 200, 0, fill=[128, 4], softcap=20.0, seed=58)
    c.check(*c.run())


def test_binding_refusals(cuda_lib):
    T = 8
    c = Case(2, 2, T, 64, slopes=[0.5, 0.25], pos=[64] * 2, ranges=[[(0, 64)] * T] * 2, fill=[5, 5], seed=59)
    out, lse = c.run()
    base = dict(q=c.q, k_out=c.ko, v_out=c.vo, pk=c.pk, pv=c.pv, prefix_len=c.plen, out=out, workspace=c.ws, ring=128,
                slopes=c.slopes, pos=c.pos, ranges=c.ranges)
    for kw, err in [(dict(out=out.float()), TypeError), (dict(pos=None), ValueError), (dict(ranges=c.ranges[:, 0]), ValueError),
                    (dict(ring=None), ValueError), (dict(softcap=-1.0), pkg.RswaError), (dict(write_ring=True), pkg.RswaError),
                    (dict(ring=0), pkg.RswaError), (dict(ring_k=c.rk), TypeError), (dict(k_out=c.ko[:, :, 1:]), ValueError),
                    (dict(q=c.q[0]), ValueError), (dict(workspace=c.ws[:128]), pkg.RswaError),
                    (dict(lse=lse[0]), ValueError), (dict(scale=math.inf), pkg.RswaError)]:
        with pytest.raises(err):
            pkg.rswa_prefill_scored(**{**base, **kw})


@pytest.mark.parametrize("softcap,bias", [(0.0, False), (0.0, True), (20.0, False), (20.0, True)])
@pytest.mark.parametrize("H,T,cap", [(80, 300, 400), (4, 300, 400), (2, 40, 1500)])
def test_scores_of_minus_infinity(cuda_lib, H, T, cap, softcap, bias):
    # every key of the even heads scores -inf: without a cap such a query has no weight to give, like one that
    # sees no row (out 0, lse -inf), in whole tiles as in masked ones; with a cap every score is -cap. Odd heads
    # are what they are without such neighbours.
    c = Case(1, H, T, cap, fill=[128], softcap=softcap, slopes=[0.0] * H if bias else None, pos=[cap] if bias else None,
             seed=65, qstd=1.0)
    before = c.run()
    c.q[..., 0] = c.q[..., 0].abs() + 1.0
    after = c.run()
    for k in (c.pk, c.ko, c.rk):
        k[:, ::2, :, 0] = -math.inf
    out, lse = c.run()
    assert not torch.equal(before[0], after[0])
    o, o0, e, e0 = (t[:, 1::2].double() for t in (out, after[0], lse, after[1]))
    if softcap == 0.0:
        assert torch.equal(o, o0) and torch.equal(e, e0)
    else:
        # a warp's form of the tanh goes by all scores of its 32 columns, and a head's last key tile runs into the
        # next head's rows: any form's score is within 7e-7 cap (1.4e-5), so two runs' lse within 2.8e-5 and a last
        # rounding, and weights within 5.6e-5 of each other, each then rounded to bf16, as the outputs are
        assert (e - e0).abs().max().item() <= 4e-5
        most = max(t.float().nan_to_num(0.0).abs().max().item() for t in (c.pv, c.vo, c.rv))
        assert ((o - o0).abs() <= (2 * 2.0 ** -8 + 6e-5) * most + 2 * 2.0 ** -8 * o0.abs()).all()
        assert (o - o0).norm() <= 5e-3 * o0.norm()
    if softcap == 0.0:
        assert (out[:, ::2] == 0).all() and torch.isneginf(lse[:, ::2]).all()
    else:
        seen = cap + torch.clamp(128 - 1 - torch.arange(T, device="cuda"), min=0) + torch.clamp(torch.arange(T, device="cuda") + 1, max=128)
        ref = seen.double().log() - softcap
        assert (lse[:, ::2].double() - ref).abs().max().item() <= 1e-4
    assert pkg.check_status(c.ws) == 0


@pytest.mark.parametrize("B,H,T", [(2, 80, 600), (2, 8, 300)])
def test_a_workspace_that_says_timeout_costs_no_waits(cuda_lib, B, H, T):
    # three waves of paired query tiles and a split rest, or split tiles alone, on a workspace whose status word
    # already holds a give-up: the CTAs do no work and wait for nothing, the flag stays until it is read, and then
    # the workspace serves as before
    c = Case(B, H, T, 300, fill=[128] * B, softcap=20.0, seed=66)
    ref = c.run()
    c.ws.view(torch.int32)[0] = bind.DEVICE_WAIT_TIMEOUT
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    c.run()
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 1.0
    assert pkg.check_status(c.ws) == bind.DEVICE_WAIT_TIMEOUT
    out, lse = c.run()
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    c.check(out, lse)


def test_a_window_past_32_bits_is_refused(cuda_lib):
    c = Case(1, 1, 4, 8, seed=67)
    for n, err in ((2 ** 32 + 128, ValueError), (2 ** 31, ValueError), (1025, pkg.RswaError), (128.5, ValueError)):
        c.n = n
        with pytest.raises(err):
            c.run()
    c.n = 128.0
    c.run()


@pytest.mark.parametrize("largest", [0.399, 0.999, 12.0])
def test_capped_scores_by_each_form_of_the_tanh(cuda_lib, largest):
    # Queries that see only themselves (a window of one): lse is the score. The rows of a head are multiples of unit
    # vectors, so that every other score is 0, and a warp takes the form that its largest |u| = |scale q.k| / cap calls
    # for. In units of the cap: the polynomials are within 2e-8; ten f32 roundings (cap log2(e) 2, scale / cap 1, the
    # coefficient 2, Horner's last steps and the product 3, ln 2 and its product 2) of a value of at most tanh(largest).
    # The exponential form adds ex2's and rcp's errors (2^-22 of e^2u: 2^-23; 2^-23 of 2 / (e^2u + 1): 2^-22), the
    # argument's three roundings (u sech^2 u <= 0.45: 0.45 * 3 * 2^-24) and the sum's (2^-24).
    H, T, cap, scale = 96, 128, 50.0, 0.125
    g = torch.Generator("cuda")
    g.manual_seed(71)
    u = (torch.rand((1, H, T), generator=g, device="cuda", dtype=torch.float64) * 2 - 1) * largest
    a = (torch.rand((1, H, T), generator=g, device="cuda", dtype=torch.float64) + 1).bfloat16()
    b = (u * cap / scale / a.double()).bfloat16()
    over = (a.double() * b.double()).abs() * scale / cap > largest
    b = torch.where(over, (b.double() * 0.99).bfloat16(), b)
    eye = torch.eye(D, device="cuda", dtype=torch.bfloat16)[None, None]
    q, k = eye * a[..., None], eye * b[..., None]
    none = torch.empty((1, H, 0, D), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((1, H, T), device="cuda")
    pkg.rswa_prefill_scored(q.contiguous(), k.contiguous(), q.contiguous(), none, none, ints([0]), out,
                            torch.zeros(256, dtype=torch.uint8, device="cuda"), softcap=cap, scale=scale, ring=1, lse=lse)
    u = a.double() * b.double() * scale / cap
    err = ((lse.double() / cap) - torch.tanh(u)).abs().max().item()
    print(f"largest |u| {largest}: error {err:.2e} of the cap")
    bound = 2e-8 + 10 * 2.0 ** -24 * math.tanh(largest)
    if largest > 1:
        bound += 2.0 ** -23 + 2.0 ** -22 + 0.45 * 3 * 2.0 ** -24 + 2.0 ** -24
    assert u.abs().max().item() > 0.97 * largest
    assert err <= bound, (err, bound)


@pytest.mark.parametrize("softcap,bias", [(0.0, False), (30.0, True)])
def test_a_nan_value_row_stays_in_its_256_queries(cuda_lib, softcap, bias):
    # a NaN row of V that some query sees reaches at most the 256 queries of that query's tile (0 x NaN): queries of
    # other tiles, of the same and of other documents, are what they are without it
    T, cap = 700, 900
    ranges = [[(0, 300) if i < 100 else (300, 900) for i in range(T)]]
    c = Case(1, 3, T, cap, ranges=ranges, softcap=softcap, slopes=slopes_of(3) if bias else None, pos=[cap] if bias else None, seed=68)
    ref = c.run()
    c.pv[:, :, 77] = math.nan
    out, lse = c.run()
    assert out[:, :, :100].isnan().all()
    assert torch.equal(out[:, :, 256:], ref[0][:, :, 256:]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("captured", [False, True])
def test_chunks_with_an_early_started_rest(cuda_lib, captured):
    # Two launches a chunk, the second started early beside the first: inputs written just before them (by a copy, and
    # by a rotary call that starts early itself), the ring moved right after them, chunk upon chunk without a pause,
    # eagerly and from a graph, against the same calls one at a time
    B, H, T, n, cap = 2, 80, 300, 128, 300
    c = Case(B, H, T, cap, n=n, fill=[128, 60], softcap=30.0, slopes=slopes_of(H), pos=[cap, cap + 9],
             ranges=[[(0, 200)] * 150 + [(100, 300)] * 150] * B, seed=69)
    g = P64.gen(70)
    chunks = [tuple(randn((B, H, T, D), g, s) for s in (2.0, 1.0, 1.0)) for _ in range(4)]
    freq, _ = pkg.rope_freqs(128)
    at = torch.arange(T, dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    state = [t.clone() for t in (c.rk, c.rv, c.wp, c.fill, c.pos, c.ranges)]
    src = [torch.empty_like(x) for x in chunks[0]]
    q, k = torch.empty_like(c.q), torch.empty_like(c.ko)
    out, lse = torch.empty_like(c.q), torch.empty((B, H, T), device="cuda")

    def chunk(wait=lambda: None):
        c.vo.copy_(src[2])
        wait()
        pkg.rswa_rope_1d(src[0], at, freq, q_out=q, k=src[1], k_out=k)
        wait()
        pkg.rswa_prefill_scored(q, k, c.vo, c.pk, c.pv, c.plen, out, c.ws, softcap=30.0, slopes=c.slopes, pos=c.pos,
                                ranges=c.ranges, lse=lse, ring_k=c.rk, ring_v=c.rv, wp=c.wp, fill=c.fill, write_ring=True)
        wait()
        c.pos.add_(T)
        c.ranges.copy_(torch.roll(c.ranges, 40, 1))

    def restart():
        for t, s in zip((c.rk, c.rv, c.wp, c.fill, c.pos, c.ranges), state):
            t.copy_(s)

    refs = []
    for x in chunks:
        for s, t in zip(src, x):
            s.copy_(t)
        chunk(torch.cuda.synchronize)
        refs.append((out.clone(), lse.clone(), c.rk.clone(), c.rv.clone(), c.wp.clone(), c.fill.clone()))
    restart()
    step = chunk
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chunk()
        step = graph.replay
    for _ in range(3):
        got = []
        restart()
        for x in chunks:
            for s, t in zip(src, x):
                s.copy_(t)
            step()
            got.append((out.clone(), lse.clone(), c.rk.clone(), c.rv.clone(), c.wp.clone(), c.fill.clone()))
        torch.cuda.synchronize()
        for a, b in zip(got, refs):
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
    assert pkg.check_status(c.ws) == 0
