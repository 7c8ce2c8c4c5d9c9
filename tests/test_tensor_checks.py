"""The binding's native tensor checks (csrc/tensors.cpp): refusals, without a GPU."""
import pytest
import torch

from long_context_decode_swa_b200 import binding

BF16 = torch.bfloat16


def _checks():
    return binding._tensors()


@pytest.mark.parametrize("fn", ["addresses", "strided"])
def test_refusals(fn):
    call = getattr(_checks(), fn)
    t = torch.zeros(2, 3, dtype=BF16)
    for spec, err, words in [
            ((t, "x", BF16, (2, 3)), ValueError, ["x:", "cuda:0", "cpu"]),
            ((t, "x", torch.float32, (2, 3)), TypeError, ["x:", "torch.float32"]),
            (([1.0], "x", BF16, (2, 3)), TypeError, ["x:", "torch.Tensor"]),
            ((None, "x", BF16, (2, 3)), TypeError, ["x:", "torch.Tensor"]),
            ((t, "x", "bf16", (2, 3)), TypeError, ["spec"]),
            ((t, "x", BF16, [2, 3]), TypeError, ["spec"]),
            ((t, "x"), TypeError, ["spec"]),
            (t, TypeError, ["spec"]),
            ((t.to_sparse(), "x", BF16, (2, 3)), ValueError, ["x:", "dense"]),
    ]:
        with pytest.raises(err) as e:
            call(0, spec)
        assert all(w in str(e.value) for w in words), str(e.value)
    with pytest.raises(TypeError):
        call()
    with pytest.raises(TypeError):
        call("cuda")


def test_optional_tensors():
    assert _checks().addresses(0, (None, "x", BF16, (1,), True)) == (None,)
    assert _checks().addresses(0) == ()


@pytest.mark.gpu
def test_addresses_and_strides(cuda_lib):
    t = torch.zeros(4, 3, 8, dtype=BF16, device="cuda")
    i = t.get_device()
    assert _checks().addresses(i, (t, "t", BF16, (4, 3, 8)), (t[1], "u", BF16, (3, 8))) == (t.data_ptr(), t[1].data_ptr())
    v = t.transpose(0, 1)
    assert _checks().strided(i, (v, "v", BF16, (3, 4, 8))) == ((t.data_ptr(), (8, 24, 1)),)
    for spec, word in [((v, "v", BF16, (3, 4, 8)), "contiguous"), ((t, "t", BF16, (4, 3)), "shape"), ((t, "t", BF16, (4, 3, 9)), "(4, 3, 8)")]:
        with pytest.raises(ValueError, match=word.replace("(", r"\(").replace(")", r"\)")):
            _checks().addresses(i, spec)
    with pytest.raises(ValueError, match=f"cuda:{i + 1}"):
        _checks().addresses(i + 1, (t, "t", BF16, (4, 3, 8)))
    empty = torch.zeros(2, 0, device="cuda")
    assert _checks().addresses(i, (empty, "e", torch.float32, (2, 0))) == (empty.data_ptr(),)
