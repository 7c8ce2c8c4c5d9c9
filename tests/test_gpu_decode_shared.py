"""GPU parity of rswa_decode_shared with plain 64-bit attention over each sequence's own keys.

Tolerances. Weights of shared rows are rounded to bf16 (half a step: 2^-8 of the weight) in the
products with V and in the normaliser alike, so an output moves by at most 2 * 2^-8 sum w |v|; the
result is rounded to bf16 (2^-8 of it); f32 scores and sums add below 1e-4 sum w |v| (a dot of 128
products of N(0, 1) has |q||k| / sqrt(D) about 11 and an f32 error below 2^-20 of that). Rounding
errors are independent, so over a whole tensor the relative 2-norm is near sqrt(2) 2^-8 / sqrt(3) =
3.2e-3: 5e-3 is asserted. lse is summed from unrounded weights: 1e-4 absolute."""
import math

import pytest
import torch

import long_context_decode_swa_b200 as pkg
from tests import plain64 as P64
from tests.plain64 import D, ints, nan_past, randn

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, B, P, H, scap, n=128, cap=0, share=None, slen=None, plen=None, fill=None, seed=0):
        g = P64.gen(1000 + seed)
        self.B, self.P, self.H, self.n, self.cap = B, P, H, n, cap
        self.q = randn((B, H, D), g, 1.5)
        self.slen = ints(slen if slen is not None else [scap] * P)
        self.share = ints(share if share is not None else [b % P for b in range(B)])
        self.sk = nan_past(randn((P, H, scap, D), g), self.slen)
        self.sv = nan_past(randn((P, H, scap, D), g), self.slen)
        self.plen = ints(plen if plen is not None else [cap] * B)
        self.pk, self.pv = (nan_past(randn((B, H, cap, D), g), self.plen) for _ in range(2))
        self.rk, self.rv, self.wp, self.fill = P64.ring(B, H, n, fill if fill is not None else [n] * B, g)
        self.ws = pkg.new_shared_workspace(pkg.Dims(B, H, D, n, cap), P)

    def run(self, ws=None, stream=None):
        out = torch.full((self.B, self.H, D), math.nan, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.B, self.H), math.nan, device="cuda")
        private = dict(pk=self.pk, pv=self.pv, prefix_len=self.plen) if self.cap else {}
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        pkg.rswa_decode_shared(self.q, self.sk, self.sv, self.slen, self.share, self.rk, self.rv, self.wp, self.fill,
                               out, self.ws if ws is None else ws, lse=lse, stream=stream, **private)
        return out, lse

    def check(self, out, lse, rel=5e-3):
        out, lse = out.double(), lse.double()
        share, slen, plen, fill, wp = (t.tolist() for t in (self.share, self.slen, self.plen, self.fill, self.wp))
        ref, size = torch.empty_like(out), torch.empty_like(out)
        ref_lse = torch.empty_like(lse)
        for b in range(self.B):
            p = share[b]
            s = slen[p] if 0 <= p < self.P else 0
            slots = P64.slots_oldest_first(wp[b], fill[b], self.n)
            for h in range(self.H):
                k = torch.cat([self.sk[p, h, :s], self.pk[b, h, :plen[b]], self.rk[b, h][slots]]).double()
                v = torch.cat([self.sv[p, h, :s], self.pv[b, h, :plen[b]], self.rv[b, h][slots]]).double()
                o, e, z = P64.attend(self.q[b, h][None].double(), k, v)
                ref[b, h], ref_lse[b, h], size[b, h] = o[0], e[0], z[0]
        bound = (2 * 2.0 ** -8 + 1e-4) * size + 2.0 ** -8 * ref.abs()
        err = (out - ref).abs()
        assert (err <= bound).all(), f"error {(err - bound).max().item():.3e} above its bound"
        none = torch.isneginf(ref_lse)
        assert torch.equal(torch.isneginf(lse), none) and (out[none] == 0).all()
        assert (lse[~none] - ref_lse[~none]).abs().max().item() <= 1e-4 if (~none).any() else True
        norm = ref.norm().item()
        assert (out - ref).norm().item() <= rel * norm + 1e-30
        assert pkg.check_status(self.ws) == 0


@pytest.mark.parametrize("B,P,H,scap", [
    (1, 1, 1, 1),          # one key
    (1, 1, 2, 128),        # one whole key tile
    (2, 1, 3, 129),        # one key past it
    (8, 1, 16, 288),       # fewer units than SMs
    (33, 2, 4, 700),       # a second warp's rows
    (128, 1, 2, 1000),     # a whole query tile
    (129, 1, 2, 1000),     # the second tile's first row
    (256, 1, 1, 300),
    (257, 1, 1, 300),      # a second pass over the prefix
    (600, 1, 2, 520),      # three
    (384, 1, 1, 200),      # as many sequences as the attention groups by itself
    (385, 2, 1, 200),      # one more
    (384, 384, 1, 3), (5, 384, 1, 40), (5, 385, 1, 40),
    (64, 16, 16, 900),     # several segments a CTA
    (40, 3, 5, 5000),      # a prefix cut over many CTAs
])
def test_matches_plain_attention(cuda_lib, B, P, H, scap):
    c = Case(B, P, H, scap, seed=B + scap)
    c.check(*c.run())


def test_ragged_everything(cuda_lib):
    # prefixes of length 0 and 1, one that nobody reads, sequences with none, private rows, part-filled rings
    share = [3, -1, 0, 1, 3, 2, 5, -1, 3, 0, 1, 1, 5, 5, 3, 2]
    B = len(share)
    c = Case(B, 6, 3, 333, n=100, cap=77, share=share, slen=[333, 1, 0, 257, 50, 128],
             plen=[(7 * b) % 78 for b in range(B)], fill=[(13 * b) % 101 for b in range(B)], seed=5)
    c.check(*c.run())


def test_sequences_that_see_nothing(cuda_lib):
    c = Case(4, 2, 2, 64, n=1, share=[-1, 0, 1, -1], slen=[64, 0], fill=[0, 0, 0, 1], seed=6)
    out, lse = c.run()
    c.check(out, lse)
    assert torch.isneginf(lse[0]).all() and torch.isneginf(lse[2]).all() and not torch.isneginf(lse[3]).any()


def test_many_prefixes(cuda_lib):
    # more prefixes and sequences than the grouping has threads
    B = P = 1500
    share = [(b * 7) % P if b % 3 else (b % 11) for b in range(B)]
    c = Case(B, P, 1, 40, n=3, share=share, slen=[(p * 5) % 41 for p in range(P)], seed=7)
    c.check(*c.run())


def test_the_most_prefixes(cuda_lib):
    c = Case(70, 8192, 1, 2, n=2, share=[(b * 117) % 8192 for b in range(69)] + [8191], seed=14)
    c.check(*c.run())


def test_one_workspace_for_calls_of_many_sizes(cuda_lib):
    # tables, records and counters of one call lie where the next one's do, or elsewhere
    cases = [Case(3, 1, 2, 300, n=5, seed=15), Case(420, 7, 1, 200, cap=9, seed=16), Case(40, 3, 4, 4000, seed=17),
             Case(1, 1, 1, 1, n=1, seed=18), Case(257, 1, 1, 129, seed=19)]
    ws = max((c.ws for c in cases), key=lambda w: w.numel())
    refs = [c.run() for c in cases]
    got = [c.run(ws=ws) for c in cases + cases[::-1]]
    for (o, e), (ro, re) in zip(got, refs + refs[::-1]):
        assert torch.equal(o, ro) and torch.equal(e, re)
    for c, r in zip(cases, refs):
        c.check(*r)
    assert pkg.check_status(ws) == 0


def test_one_peaked_key_and_large_scores(cuda_lib):
    # one key far above the rest, first in a late tile: the running maximum moves by hundreds
    c = Case(9, 1, 2, 900, seed=8)
    c.sk[0, :, 700] = c.q[3] * 8
    c.sk[0, :, 5] = c.q[4] * 8
    c.check(*c.run(), rel=6e-3)  # some outputs are one row of V: no averaging, rounding alone


def test_agrees_with_rswa_decode(cuda_lib):
    # the same keys laid out as private prefixes: rswa_decode in f32 throughout
    c = Case(12, 2, 4, 500, seed=9)
    out, lse = c.run()
    pk, pv = c.sk[c.share.long()].contiguous(), c.sv[c.share.long()].contiguous()
    ref = torch.empty((12, 4, D), device="cuda")
    ref_lse = torch.empty((12, 4), device="cuda")
    ws = pkg.new_workspace(pkg.dims_of(pk, c.rk), pkg.OP_DECODE)
    pkg.rswa_decode(c.q, pk, pv, c.slen[c.share.long()].contiguous(), c.rk, c.rv, c.wp, c.fill, ref, ws, lse=ref_lse)
    assert (out.float() - ref).norm() <= 5e-3 * ref.norm()
    assert (lse - ref_lse).abs().max() <= 1e-4


def test_repeats_are_bit_equal(cuda_lib):
    c = Case(300, 3, 2, 700, cap=33, seed=10)
    a = c.run()
    b = c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(*a)


def test_streams_graph_and_changed_groups(cuda_lib):
    c = Case(20, 3, 4, 400, cap=10, seed=11)
    ref = c.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    other = pkg.new_shared_workspace(pkg.Dims(20, 4, D, 128, 10), 3)
    torch.cuda.synchronize()
    outs = [c.run(stream=s1), c.run(ws=other, stream=s2)]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], ref[0]) and torch.equal(o[1], ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = c.run()
    # groups, lengths and ring states are read at replay
    c.share.copy_(ints([2] * 19 + [-1]))
    c.slen.copy_(ints([10, 20, 399]))
    c.sk[2, :, 399:] = math.nan
    c.fill.fill_(128)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    c.check(out, lse)


def test_device_checks(cuda_lib):
    c = Case(6, 2, 2, 100, cap=20, seed=12)
    good = c.run()
    c.share[1], c.share[2] = 2, -2          # read as -1
    c.plen[3] = 21                          # its private rows skipped
    c.fill[4] = 129                         # its ring skipped
    out, lse = c.run()
    st = pkg.check_status(c.ws)
    from long_context_decode_swa_b200 import binding as b
    assert st == b.DEVICE_BAD_SHARE | b.DEVICE_BAD_PREFIX_LEN | b.DEVICE_BAD_RING_STATE
    assert torch.equal(out[0], good[0][0]) and torch.equal(out[5], good[0][5])
    c.share[1] = c.share[2] = -1
    c.plen[3] = 0
    c.fill[4] = 0
    c.check(out, lse)
    c.slen[0] = 101                         # a bad shared length is read as 0
    out, lse = c.run()
    assert pkg.check_status(c.ws) == b.DEVICE_BAD_PREFIX_LEN
    c.slen[0] = 0
    c.check(out, lse)


def test_binding_refusals(cuda_lib):
    c = Case(3, 2, 2, 64, cap=4, seed=13)
    out, lse = c.run()
    base = dict(q=c.q, sk=c.sk, sv=c.sv, shared_len=c.slen, share_of=c.share, ring_k=c.rk, ring_v=c.rv, wp=c.wp,
                fill=c.fill, out=out, workspace=c.ws)
    for kw, err in [(dict(out=out.float()), TypeError), (dict(q=c.q.float()), TypeError), (dict(sv=c.sv[:, :, :63]), ValueError),
                    (dict(shared_len=c.slen.long()), TypeError), (dict(share_of=c.share[:2]), ValueError),
                    (dict(sk=c.sk[0]), ValueError), (dict(pv=c.pv), ValueError), (dict(wp=c.wp.cpu()), ValueError),
                    (dict(workspace=c.ws[:256]), pkg.RswaError), (dict(workspace=c.ws.view(torch.int32)), TypeError),
                    (dict(scale=0.0), pkg.RswaError), (dict(scale=math.nan), pkg.RswaError),
                    (dict(lse=lse[:, :1]), ValueError), (dict(q=c.q.transpose(0, 1)), ValueError)]:
        with pytest.raises(err):
            pkg.rswa_decode_shared(**{**base, **kw})


@pytest.mark.parametrize("B,P,H,scap", [
    (40, 16, 12, 300),   # 576 key tiles, four a CTA: three and one, two and two, one and three
    (24, 24, 37, 250),   # 1,776 key tiles, twelve a CTA: six segments of two each
    (64, 64, 37, 100),   # sixteen segments of one tile a CTA
    (31, 31, 43, 140),   # 2,666 key tiles, nineteen a CTA: two and one, in turn about the cuts
])
def test_segments_of_one_key_tile_after_others(cuda_lib, B, P, H, scap):
    # at most 128 readers: a segment of one key tile leaves the second group of rows without a score, right
    # after a segment whose sums the groups told each other
    c = Case(B, P, H, scap, n=8, seed=2000 + scap)
    ref = c.run()
    c.check(*ref)
    for _ in range(20):
        out, lse = c.run()
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
