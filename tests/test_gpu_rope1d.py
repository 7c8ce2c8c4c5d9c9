"""GPU parity of rswa_rope_1d with the rotation in 80-bit host arithmetic.

Tolerance, from the kernel's arithmetic. Angle: the fixed-point turn is cut to 32 bits (2^-32 turns),
its step is off by at most 2^-65 turns a position (2^-34 over int32), and the cut turn, at most half a
turn, is rounded to f32 (2^-25 turns): together below 2 pi 2^-24.9 = 2.0e-7 rad. sincospif is good to
an ulp (2^-23 at most), the product with mscale and mscale's own f32 value round once each (2^-24),
the rotation's product and FMA once each (2^-24). An output is a sum of two terms no larger than
mscale (|x| + |y|), so before its last rounding it is within 2^-20 mscale (|x| + |y|) of the exact
value (2.0e-7 + 1.2e-7 + 4 * 0.6e-7 = 5.6e-7 < 2^-20 = 9.5e-7). bf16 adds half a step of the result."""
import numpy as np
import pytest
import torch

import long_context_decode_swa_b200 as pkg

pytestmark = pytest.mark.gpu


def exact(x, pos, freq, rot, layout, mscale, inverse):
    """x f64 [B][H][T][D] (numpy), pos [B][T]: the encoded rows, and |x| + |y| of each output's pair."""
    ang = pos.astype(np.longdouble)[:, None, :, None] * freq.astype(np.longdouble)
    c, s = np.cos(ang) * mscale, np.sin(ang) * (-mscale if inverse else mscale)
    y, size = x.astype(np.longdouble).copy(), np.zeros(x.shape)
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    xa, xb = x[..., a].astype(np.longdouble), x[..., b].astype(np.longdouble)
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    size[..., a] = size[..., b] = (np.abs(xa) + np.abs(xb)).astype(np.float64)
    return y.astype(np.float64), size


def half_step(v, dtype):
    bits = 7 if dtype == torch.bfloat16 else 23
    a = np.abs(v)
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    return np.where(a > 0, np.exp2(np.maximum(e - bits, -133)), 2.0 ** -133) / 2


def check(got, x, pos, freq, layout, mscale=1.0, inverse=False):
    ref, size = exact(x.double().cpu().numpy(), pos.cpu().numpy(), freq.numpy(), 2 * len(freq), layout, mscale, inverse)
    g = got.double().cpu().numpy()
    assert g.shape == ref.shape
    bound = 2.0 ** -20 * abs(mscale) * size + np.where(size > 0, half_step(g, got.dtype), 0.0)
    err = np.abs(g - ref)
    at = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), f"error {err[at]:.3e} above {bound[at]:.3e} at {at}"


def rows(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def positions(B, T, seed, lo=-2 ** 31, hi=2 ** 31):
    return torch.from_numpy(np.random.default_rng(seed).integers(lo, hi, (B, T)).astype(np.int32)).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,Hq,Hk,T,D,rot", [
    (1, 1, 0, 1, 16, 16),       # the smallest row
    (1, 16, 16, 1, 128, 128),   # one token
    (3, 5, 2, 77, 128, 64),     # half of each head, odd counts, fewer k heads
    (2, 3, 3, 130, 64, 48),     # rotated part not a power of two
    (1, 128, 128, 5, 256, 256),  # the widest: several passes a token
    (700, 2, 1, 1, 96, 32),     # more groups than SMs
])
def test_matches_the_rotation(cuda_lib, dtype, layout, B, Hq, Hk, T, D, rot):
    freq, _ = pkg.rope_freqs(rot, 10000.0)
    q, k = rows((B, Hq, T, D), 1, dtype), rows((B, Hk, T, D), 2, dtype)
    pos = positions(B, T, 3, 0, 200000)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    cuda_lib.rswa_rope_1d(q, pos, freq, q_out=qo, layout=layout, **(dict(k=k, k_out=ko) if Hk else {}))
    check(qo, q, pos, freq, layout)
    if Hk:
        check(ko, k, pos, freq, layout)


def test_far_and_negative_positions(cuda_lib):
    # every int32 position, and frequencies of more than a turn a token and of either sign
    freq = torch.tensor([1.0, 7.5, -0.3, 1e-4, 123.456, 0.0, 1e-9, 3.0], dtype=torch.float64)
    q = rows((2, 3, 64, 16), 5, torch.float32)
    pos = positions(2, 64, 6)
    pos[0, :4] = torch.tensor([-2 ** 31, 2 ** 31 - 1, 0, -1])
    qo, _ = cuda_lib.rswa_rope_1d(q, pos, freq, q_out=torch.empty_like(q))
    check(qo, q, pos, freq, "half")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_leaves_the_rest_alone(cuda_lib, layout):
    freq, mscale = pkg.rope_freqs(32, scaling="by_parts", factor=16.0, trained=4096)
    q, k = rows((2, 4, 33, 128), 7), rows((2, 1, 33, 128), 8)
    q[..., 32:] = float("nan")  # not read, not written
    q0, k0 = q.clone(), k.clone()
    pos = positions(2, 33, 9, 0, 60000)
    a, b = cuda_lib.rswa_rope_1d(q, pos, freq, k=k, layout=layout, mscale=mscale)
    assert a is q and b is k
    check(q[..., :32], q0[..., :32], pos, freq, layout, float(np.float32(mscale)))
    check(k, k0, pos, freq, layout, float(np.float32(mscale)))
    assert q[..., 32:].isnan().all()
    # q in place and k copied in one call: q's rest untouched, k's copied
    q1, k1 = q0.clone(), k0.clone()
    ko = torch.empty_like(k1)
    cuda_lib.rswa_rope_1d(q1, pos, freq, k=k1, k_out=ko, layout=layout, mscale=mscale)
    assert torch.equal(q1.view(torch.int16), q.view(torch.int16)) and torch.equal(ko, k)


def test_strided_views_and_one_token_form(cuda_lib):
    # q and k as views of one packed projection, outputs in another order of the axes
    B, T, Hq, Hk, D = 2, 37, 6, 2, 128
    freq, _ = pkg.rope_freqs(64)
    x = rows((B, T, Hq + 2 * Hk, D), 11)
    keep = x.clone()
    view = x.transpose(1, 2)
    pos = positions(B, T, 12, 0, 5000)
    qo = torch.empty((T, B, Hq, D), dtype=x.dtype, device="cuda").permute(1, 2, 0, 3)
    ko = torch.empty((B, Hk, T, D), dtype=x.dtype, device="cuda")
    cuda_lib.rswa_rope_1d(view[:, :Hq], pos, freq, q_out=qo, k=view[:, Hq:Hq + Hk], k_out=ko)
    assert torch.equal(x, keep)
    check(qo, view[:, :Hq], pos, freq, "half")
    check(ko, view[:, Hq:Hq + Hk], pos, freq, "half")
    # the same rows in place in the packed tensor: bit for bit, v untouched
    cuda_lib.rswa_rope_1d(view[:, :Hq], pos, freq, k=view[:, Hq:Hq + Hk])
    assert torch.equal(view[:, :Hq], qo) and torch.equal(view[:, Hq:Hq + Hk], ko)
    assert torch.equal(x[:, :, Hq + Hk:], keep[:, :, Hq + Hk:])
    # [B][H][D] with pos [B]; a broadcast (stride 0) input
    one = torch.empty((B, Hq, D), dtype=x.dtype, device="cuda")
    cuda_lib.rswa_rope_1d(keep[:, 3, :Hq], pos[:, 3].contiguous(), freq, q_out=one)
    assert torch.equal(one, qo[:, :, 3])
    wide = keep[:1, :1, :1].transpose(1, 2).expand(B, 4, T, D)
    wo, _ = cuda_lib.rswa_rope_1d(wide, pos, freq, q_out=torch.empty((B, 4, T, D), dtype=x.dtype, device="cuda"))
    check(wo, wide, pos, freq, "half")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_inverse_is_the_gradient(cuda_lib, layout):
    # d/dx <g, rope(x)> = rope^T g: by the formula, and by differences (rope is linear, so a
    # difference quotient of any step is the derivative, up to f32 rounding of the two values)
    freq, mscale = pkg.rope_freqs(64, scaling="by_parts", factor=8.0, trained=2048)
    m32 = float(np.float32(mscale))
    x, g = rows((1, 2, 9, 96), 21, torch.float32), rows((1, 2, 9, 96), 22, torch.float32)
    pos = positions(1, 9, 23, 0, 9000)
    grad, _ = cuda_lib.rswa_rope_1d(g, pos, freq, q_out=torch.empty_like(g), layout=layout, mscale=mscale, inverse=True)
    check(grad, g, pos, freq, layout, m32, inverse=True)

    def value(v):
        y, _ = cuda_lib.rswa_rope_1d(v, pos, freq, q_out=torch.empty_like(v), layout=layout, mscale=mscale)
        return (y.double() * g.double()).sum((-1, -2, -3))

    base = value(x)
    for h, t, d in [(0, 0, 0), (1, 4, 33), (0, 8, 63), (1, 2, 64), (1, 8, 95)]:
        up = x.clone()
        up[0, h, t, d] += 1.0
        step = (up[0, h, t, d] - x[0, h, t, d]).double()
        got = ((value(up) - base) / step).item()
        # each of the two values' affected outputs is within 2^-20 m (|x| + |y|) + 2^-24 |out|
        size = (up.abs().max().item() + x.abs().max().item()) * 2
        assert abs(got - grad[0, h, t, d].item()) <= 4 * 2.0 ** -20 * m32 * size * g.abs().max().item() / step.item()


def test_two_streams_and_a_graph(cuda_lib):
    freq, _ = pkg.rope_freqs(128)
    q = rows((2, 4, 50, 128), 31)
    pos = positions(2, 50, 32, 0, 4000)
    ref, _ = cuda_lib.rswa_rope_1d(q, pos, freq, q_out=torch.empty_like(q))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a, b = torch.empty_like(q), torch.empty_like(q)
    cuda_lib.rswa_rope_1d(q, pos, freq, q_out=a, stream=side)
    with torch.cuda.stream(side):
        cuda_lib.rswa_rope_1d(q, pos, freq, q_out=b)
    side.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, ref)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.rswa_rope_1d(q, pos, freq, q_out=out)
    freq.zero_()  # the table was read during the call
    pos += 17     # the positions are read at replay
    graph.replay()
    torch.cuda.synchronize()
    check(out, q, pos, pkg.rope_freqs(128)[0], "half")


def test_refusals_on_device_tensors(cuda_lib):
    freq, _ = pkg.rope_freqs(64)
    q = rows((2, 4, 6, 128), 41)
    pos = positions(2, 6, 42, 0, 100)
    call = cuda_lib.rswa_rope_1d
    for bad in (lambda: call(q.half(), pos, freq), lambda: call(q, pos.long(), freq), lambda: call(q, pos, freq.float()),
                lambda: call(q, pos, freq.cuda()), lambda: call(q, pos, freq, k=q.float())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: call(q, pos[:, :5].contiguous(), freq), lambda: call(q, pos.cpu(), freq),
                lambda: call(q, pos, freq, layout="both"), lambda: call(q, pos, freq, k_out=q),
                lambda: call(q, pos, freq, q_out=q[:, :3]), lambda: call(q, pos, freq, k=q[:1]),
                lambda: call(q[..., ::2], pos, freq), lambda: call(q.transpose(0, 1)[:2, :2], pos, freq,
                                                                   q_out=q[:2, :2]),
                lambda: call(q[0, 0], pos, freq)):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros(2 * 4 * 6 * 132, dtype=torch.bfloat16, device="cuda").view(2, 4, 6, 132)[..., :128]
    for bad in (lambda: call(odd, pos, freq), lambda: call(q, pos, pkg.rope_freqs(130)[0]),
                lambda: call(q, pos, pkg.rope_freqs(24)[0]),
                lambda: call(q, pos, freq, q_out=torch.empty_like(q)[:, :1].expand(2, 4, 6, 128))):
        with pytest.raises(cuda_lib.RswaError):
            bad()


def test_tensors_that_require_a_gradient(cuda_lib):
    # refused while autograd records, whichever tensor it is; taken where it does not; and the gradient of an
    # autograd.Function of the call and its transpose against the formula's
    freq, _ = pkg.rope_freqs(64)
    q, k = rows((1, 2, 9, 96), 51, torch.float32), rows((1, 1, 9, 96), 52, torch.float32)
    pos, out = positions(1, 9, 53, 0, 9000), torch.empty_like(q)
    leaf, leaf_k = q.clone().requires_grad_(), k.clone().requires_grad_()
    for bad in (lambda: cuda_lib.rswa_rope_1d(leaf, pos, freq, q_out=out), lambda: cuda_lib.rswa_rope_1d(leaf, pos, freq),
                lambda: cuda_lib.rswa_rope_1d(leaf * 2, pos, freq, q_out=out),
                lambda: cuda_lib.rswa_rope_1d(q, pos, freq, q_out=leaf),
                lambda: cuda_lib.rswa_rope_1d(q, pos, freq, q_out=out, k=leaf_k, k_out=torch.empty_like(k)),
                lambda: cuda_lib.rswa_rope_1d(q, pos, freq, q_out=out, k=k, k_out=leaf_k)):
        with pytest.raises(ValueError, match="gradient"):
            bad()
    assert torch.equal(leaf, q) and torch.equal(leaf_k, k)
    with torch.no_grad():
        cuda_lib.rswa_rope_1d(leaf, pos, freq, q_out=out)
    check(out, q, pos, freq, "half")

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return cuda_lib.rswa_rope_1d(x, pos, freq, q_out=torch.empty_like(x))[0]

        @staticmethod
        def backward(ctx, g):
            return cuda_lib.rswa_rope_1d(g.contiguous(), pos, freq, q_out=torch.empty_like(g), inverse=True)[0]

    g = rows(q.shape, 54, torch.float32)
    (Rope.apply(leaf) * g).sum().backward()
    check(leaf.grad, g, pos, freq, "half", inverse=True)


def test_strides_of_axes_of_one_entry_do_not_matter(cuda_lib):
    # one sequence, one token, one head: such an axis may have any stride (views and slices give it odd ones), in
    # place too, where input and output may differ in it; and empty tensors of any strides
    freq, _ = pkg.rope_freqs(64)
    for shape, odd, other in [((1, 4, 6, 128), (7, 768, 128, 1), (3, 768, 128, 1)), ((2, 4, 1, 128), (512, 128, 5, 1), (512, 128, 128, 1)),
                              ((3, 1, 2, 128), (256, 13, 128, 1), (256, 0, 128, 1))]:
        x = rows((3 * 1024,), 61)
        keep = x.clone()
        pos = positions(shape[0], shape[2], 62, 0, 5000)
        plain = keep.as_strided(shape, (odd[0] if shape[0] > 1 else 4096, odd[1] if shape[1] > 1 else 4096,
                                        odd[2] if shape[2] > 1 else 4096, 1)).contiguous()
        want, _ = cuda_lib.rswa_rope_1d(plain, pos, freq, q_out=torch.empty_like(plain))
        got, _ = cuda_lib.rswa_rope_1d(x.as_strided(shape, odd), pos, freq, q_out=torch.empty_like(plain))
        assert torch.equal(got, want)
        got, gk = cuda_lib.rswa_rope_1d(x.as_strided(shape, odd), pos, freq, q_out=x.as_strided(shape, other),
                                        k=plain, k_out=plain.as_strided(shape, plain.stride()))
        assert torch.equal(got, want) and torch.equal(gk, want)
    empty = torch.empty((0, 4, 6, 128), dtype=torch.bfloat16, device="cuda")
    turned = torch.empty((0, 6, 4, 128), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    assert cuda_lib.rswa_rope_1d(empty, positions(0, 6, 63), freq, q_out=turned)[0] is turned
