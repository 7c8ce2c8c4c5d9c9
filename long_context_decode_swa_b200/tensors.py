"""binding.py's tensor checks in Python, where csrc/tensors.cpp, which does the same in a tenth of the time, cannot
be built: addresses(index, spec, ..) and strided(index, spec, ..), a spec being (tensor, name, dtype, shape[, optional])."""
from __future__ import annotations

import operator

import torch


def _checked(index: int, spec, dense: bool):
    """The spec's tensor, or None for an optional one that is not given."""
    if not isinstance(spec, tuple) or len(spec) < 4:
        raise TypeError("a spec is (tensor, name, torch dtype, shape tuple)")
    t, name, dtype, shape = spec[:4]
    if t is None and len(spec) > 4:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not isinstance(dtype, torch.dtype) or not isinstance(shape, tuple):
        raise TypeError(f"{name}: a spec is (tensor, name, torch dtype, shape tuple)")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.layout != torch.strided:
        raise ValueError(f"{name}: must be a dense (strided) tensor")
    if not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{name}: expected a tensor on cuda:{index}, got {t.device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if not dense and t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name}: requires a gradient, and the call records none (call it from an autograd.Function "
                         "or under torch.no_grad())")
    return t


def addresses(index, *specs):
    """Data pointers of contiguous tensors on CUDA device `index`."""
    index = operator.index(index)
    found = [_checked(index, s, True) for s in specs]
    return tuple(None if t is None else t.data_ptr() for t in found)


def strided(index, *specs):
    """(data pointer, strides) of tensors that need not be contiguous; none may require a gradient that autograd
    would record."""
    index = operator.index(index)
    found = [_checked(index, s, False) for s in specs]
    return tuple(None if t is None else (t.data_ptr(), t.stride()) for t in found)
