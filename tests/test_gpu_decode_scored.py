"""GPU parity of rswa_decode_scored with plain 64-bit attention.

Tolerances: everything is f32. A score is a dot of 128 bf16 products (chains of at most 16 additions:
2^-20 of sum |q k| scale), a tanh good to a few ulp of a value at most softcap, and a bias that counts
only where it is small against the row's favoured key: with |q| about 4 |k| a score errs by at most
5e-5, so weights and outputs are within 1e-4 sum w |v| and lse within 1e-4 (plus 2^-23 of its size)."""
import math

import pytest
import torch

import long_context_decode_swa_b200 as pkg
from long_context_decode_swa_b200 import binding as bind
from tests import plain64 as P64
from tests.plain64 import D, ints, nan_past, randn

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, B, H, cap, n=128, plen=None, fill=None, softcap=0.0, slopes=None, pos=None, ranges=None,
                 qstd=4.0, seed=0):
        g = P64.gen(2000 + seed)
        self.B, self.H, self.cap, self.n, self.softcap = B, H, cap, n, softcap
        self.q = randn((B, H, D), g, qstd)
        self.plen = ints(plen if plen is not None else [cap] * B)
        self.pk, self.pv = (nan_past(randn((B, H, cap, D), g), self.plen) for _ in range(2))
        self.rk, self.rv, self.wp, self.fill = P64.ring(B, H, n, fill if fill is not None else [n] * B, g)
        self.slopes = None if slopes is None else torch.tensor(slopes, device="cuda", dtype=torch.float32)
        self.pos = None if pos is None else ints(pos)
        self.ranges = None if ranges is None else ints(ranges)
        self.ws = pkg.new_workspace(pkg.Dims(B, H, D, n, cap), pkg.OP_DECODE_SCORED)

    def run(self, ws=None, stream=None):
        out = torch.full((self.B, self.H, D), math.nan, device="cuda")
        lse = torch.full((self.B, self.H), math.nan, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        pkg.rswa_decode_scored(self.q, self.pk, self.pv, self.plen, self.rk, self.rv, self.wp, self.fill, out,
                               self.ws if ws is None else ws, softcap=self.softcap, slopes=self.slopes, pos=self.pos,
                               ranges=self.ranges, lse=lse, stream=stream)
        return out, lse

    def check(self, out, lse):
        out, lse = out.double(), lse.double()
        for b in range(self.B):
            lo, hi = (0, self.plen[b].item()) if self.ranges is None else self.ranges[b].tolist()
            hi = max(lo, hi)
            f = self.fill[b].item()
            slots = P64.slots_oldest_first(self.wp[b].item(), f, self.n)
            for h in range(self.H):
                k = torch.cat([self.pk[b, h, lo:hi], self.rk[b, h][slots]]).double()
                v = torch.cat([self.pv[b, h, lo:hi], self.rv[b, h][slots]]).double()
                bias = None
                if self.slopes is not None:
                    at = torch.cat([torch.arange(lo, hi), self.pos[b].item() - f + 1 + torch.arange(f)]).cuda()
                    bias = -self.slopes[h].double() * (self.pos[b] - at).double()[None]
                o, e, size = P64.attend(self.q[b, h][None].double(), k, v, bias, self.softcap)
                err = (out[b, h] - o[0]).abs()
                assert (err <= 1e-4 * size[0] + 1e-30).all(), (b, h, err.max().item())
                if torch.isneginf(e[0]):
                    assert torch.isneginf(lse[b, h]) and (out[b, h] == 0).all()
                else:
                    assert abs(lse[b, h] - e[0]) <= 1e-4 + 2.0 ** -22 * abs(e[0]), (b, h, lse[b, h].item(), e[0].item())
        assert pkg.check_status(self.ws) == 0


def slopes_of(H):
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


@pytest.mark.parametrize("B,H,cap,n", [
    (1, 1, 1, 1), (1, 1, 31, 2), (1, 2, 32, 32), (2, 3, 33, 100), (1, 16, 288, 128), (5, 7, 1000, 128),
    (3, 2, 6000, 1024),   # long items cut over many CTAs
    (700, 2, 40, 128),    # several sequences a thread, many short items a CTA
    (1, 1, 20000, 128),   # one item over the whole grid
])
@pytest.mark.parametrize("softcap,bias", [(0.0, False), (20.0, False), (0.0, True), (50.0, True)])
def test_matches_plain_attention(cuda_lib, B, H, cap, n, softcap, bias):
    plen = [cap - (b * 13) % max(1, cap // 2) for b in range(B)]
    c = Case(B, H, cap, n, plen=plen, fill=[n - (b * 7) % n for b in range(B)], softcap=softcap,
             slopes=slopes_of(H) if bias else None, pos=[m + 5 * b for b, m in enumerate(plen)] if bias else None, seed=B + cap)
    c.check(*c.run())


def test_plain_scores_equal_rswa_decode(cuda_lib):
    c = Case(6, 4, 700, plen=[700, 0, 1, 333, 64, 65], fill=[128, 0, 5, 128, 127, 1], qstd=1.0, seed=3)
    out, lse = c.run()
    ref, ref_lse = torch.empty_like(out), torch.empty_like(lse)
    ws = pkg.new_workspace(pkg.dims_of(c.pk, c.rk), pkg.OP_DECODE)
    pkg.rswa_decode(c.q, c.pk, c.pv, c.plen, c.rk, c.rv, c.wp, c.fill, ref, ws, lse=ref_lse)
    assert (out - ref).norm() <= 1e-5 * ref.norm()
    assert torch.equal(torch.isneginf(lse), torch.isneginf(ref_lse))
    some = ~torch.isneginf(lse)
    assert (lse - ref_lse)[some].abs().max() <= 1e-5


def test_documents_and_what_lies_outside_them(cuda_lib):
    # ranges: unaligned, one row, empty, whole; NaN and infinities outside stay outside
    ranges = [[37, 205], [5, 6], [9, 9], [0, 300], [299, 300], [200, 3], [0, 0], [64, 96]]
    c = Case(8, 3, 300, ranges=ranges, fill=[128, 0, 128, 3, 0, 77, 0, 128], softcap=30.0, slopes=slopes_of(3),
             pos=[300, 290, 900, 300, 10 ** 9, 300, 300, 5000], seed=4)
    for b, (lo, hi) in enumerate(ranges):
        outside = torch.ones(300, dtype=torch.bool, device="cuda")
        outside[lo:max(lo, hi)] = False
        for x, bad in ((c.pk, math.inf), (c.pv, math.nan)):
            x[b].masked_fill_(outside[None, :, None], bad)
    out, lse = c.run()
    c.check(out, lse)
    assert torch.isneginf(lse[6]).all()  # no rows at all


@pytest.mark.parametrize("slope", [1.0, 0.707, -0.01, -1.0])
def test_far_documents_keep_their_precision(cuda_lib, slope):
    # an empty ring and a document a billion tokens back: the bias is about -1e9, equal up to
    # small differences for its rows; and queries inside, before and after the document
    c = Case(5, 2, 400, fill=[0, 0, 0, 128, 4], slopes=[slope, slope / 3], ranges=[[100, 400]] * 5,
             pos=[2 ** 30, 250, 0, 10 ** 9, 401], seed=5)
    c.check(*c.run())


def test_extreme_scores(cuda_lib):
    # scores of +-1e4 saturate the cap; without a cap one key takes all
    for softcap in (0.0, 50.0):
        c = Case(2, 2, 100, softcap=softcap, qstd=1.0, seed=6)
        c.q *= 1000.0
        out, lse = c.run()
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        if softcap:
            assert (lse <= 50.0 + math.log(228) + 1e-3).all() and (lse >= 49.0).all()


def test_nan_in_a_row_that_is_seen_comes_through(cuda_lib):
    c = Case(2, 2, 200, seed=7)
    c.pv[0, 1, 77, 5] = math.nan
    c.pk[1, 0, 3, 0] = math.nan
    out, _ = c.run()
    nan = torch.isnan(out)
    assert nan[0, 1, 5] and nan[0].sum() == 1 and nan[1, 0].all() and not nan[1, 1].any()


def test_streams_graph_and_repeats(cuda_lib):
    c = Case(9, 4, 900, softcap=50.0, slopes=slopes_of(4), pos=[900 + b for b in range(9)],
             ranges=[[b * 50, 900 - b] for b in range(9)], seed=8)
    ref = c.run()
    other = torch.zeros_like(c.ws)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [c.run(stream=s1), c.run(ws=other, stream=s2)]
    torch.cuda.synchronize()
    outs.append(c.run())
    for o in outs:  # which CTA joins the records last does not show
        assert torch.equal(o[0], ref[0]) and torch.equal(o[1], ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = c.run()
    c.ranges.copy_(ints([[3, 3 + 90 * b] for b in range(9)]))
    c.pos += 11
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    c.check(out, lse)


def test_device_checks(cuda_lib):
    c = Case(6, 2, 100, slopes=[0.5, 0.25], pos=[100] * 6, ranges=[[0, 100]] * 6, seed=9)
    c.ranges[0] = ints([-1, 50])
    c.ranges[1] = ints([0, 101])
    c.pos[2], c.pos[3] = -1, 2 ** 30 + 1
    c.plen[4] = 101
    c.wp[5] = 128
    out, lse = c.run()
    assert pkg.check_status(c.ws) == bind.DEVICE_BAD_RANGE | bind.DEVICE_BAD_POS | bind.DEVICE_BAD_PREFIX_LEN | \
        bind.DEVICE_BAD_RING_STATE
    c.ranges[:5] = 0
    c.ranges[5] = ints([0, 100])
    c.pos[2] = c.pos[3] = 100
    c.plen[4] = 100
    c.wp[5] = c.fill[5] = 0
    c.check(out, lse)


def test_binding_refusals(cuda_lib):
    c = Case(3, 2, 64, slopes=[0.5, 0.25], pos=[64] * 3, ranges=[[0, 64]] * 3, seed=10)
    out, lse = c.run()
    base = dict(q=c.q, pk=c.pk, pv=c.pv, prefix_len=c.plen, ring_k=c.rk, ring_v=c.rv, wp=c.wp, fill=c.fill, out=out,
                workspace=c.ws, slopes=c.slopes, pos=c.pos, ranges=c.ranges)
    for kw, err in [(dict(out=out.bfloat16()), TypeError), (dict(pos=None), ValueError), (dict(slopes=c.slopes[:1]), ValueError),
                    (dict(slopes=c.slopes.double()), TypeError), (dict(ranges=c.ranges[:, :1]), ValueError),
                    (dict(ranges=c.ranges.long()), TypeError), (dict(pos=c.pos[:2]), ValueError),
                    (dict(softcap=-1.0), pkg.RswaError), (dict(softcap=math.inf), pkg.RswaError),
                    (dict(softcap=math.nan), pkg.RswaError), (dict(scale=-1.0), pkg.RswaError),
                    (dict(workspace=c.ws[:256]), pkg.RswaError), (dict(pk=c.pk[:, :1]), ValueError),
                    (dict(ring_v=c.rv[:, :, :5]), ValueError), (dict(lse=lse.cpu()), ValueError)]:
        with pytest.raises(err):
            pkg.rswa_decode_scored(**{**base, **kw})
