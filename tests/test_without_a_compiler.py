"""The package where csrc/tensors.cpp cannot be built: the library loads, every call checks its tensors in Python."""
import os
import subprocess
import sys

import pytest
import torch

from long_context_decode_swa_b200 import build, tensors

BF16 = torch.bfloat16


@pytest.fixture
def copy(tmp_path):
    """A copy of the package (by links) with the library and without the extension."""
    build.build_lib()
    pkg = tmp_path / os.path.basename(build.PKG)
    pkg.mkdir()
    for name in os.listdir(build.PKG):
        if not name.startswith(("_tensors", "_build", "__pycache__")):
            (pkg / name).symlink_to(os.path.join(build.PKG, name))
    (tmp_path / "include").symlink_to(build.INCLUDE)
    return tmp_path


def _run(copy, code):
    none = copy / "none"
    none.mkdir()
    return subprocess.run([sys.executable, "-c", code], cwd=copy, capture_output=True, text=True,
                          env={**os.environ, "PATH": str(none), "PYTHONPATH": str(copy), "PYTHONDONTWRITEBYTECODE": "1"})


def test_no_compiler(copy):
    r = _run(copy, """if True:
        import ctypes, warnings, torch
        import long_context_decode_swa_b200 as rswa
        from long_context_decode_swa_b200 import binding, build
        assert binding.__file__.startswith(%r), binding.__file__
        lib = rswa.load()                       # the older calls need nothing else
        assert lib.rswa_version() == 5
        assert lib.rswa_decode(None, *[None] * 8, 1.0, None, None, None, 0, None) == 1
        assert build.build() == build.LIB       # nothing to compile
        with warnings.catch_warnings(record=True) as told:
            warnings.simplefilter("always")
            checks = binding._tensors()
        assert checks.__name__.endswith(".tensors") and "Python" in str(told[0].message)
        assert binding._tensors() is checks and checks.addresses(0, (None, "x", torch.int32, (1,), True)) == (None,)
        print("fine")
    """ % str(copy))
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("fn", ["addresses", "strided"])
def test_refusals(fn):
    call = getattr(tensors, fn)
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


@pytest.mark.gpu
def test_python_and_native_checks_agree(cuda_lib):
    from long_context_decode_swa_b200 import binding
    native = binding._tensors()
    assert native is not tensors
    t = torch.zeros(4, 3, 8, dtype=BF16, device="cuda")
    i, v = t.get_device(), t.transpose(0, 1)
    good = [(t, "t", BF16, (4, 3, 8)), (t[1], "u", BF16, (3, 8)), (None, "n", BF16, (1,), True)]
    assert tensors.addresses(i, *good) == native.addresses(i, *good)
    assert tensors.strided(i, (v, "v", BF16, (3, 4, 8))) == native.strided(i, (v, "v", BF16, (3, 4, 8)))
    leaf = t.float().requires_grad_()
    for checks in (tensors, native):
        with pytest.raises(ValueError, match="gradient"):
            checks.strided(i, (leaf, "leaf", torch.float32, (4, 3, 8)))
        with torch.no_grad():
            checks.strided(i, (leaf, "leaf", torch.float32, (4, 3, 8)))
    for index, spec in [(i, (v, "v", BF16, (3, 4, 8))), (i, (t, "t", BF16, (4, 3))), (i + 1, good[0])]:
        for checks in (tensors, native):
            with pytest.raises(ValueError):
                checks.addresses(index, spec)


def test_the_extension_is_of_this_pytorch_python_and_source(monkeypatch, tmp_path):
    import sysconfig
    here = build.ext_path()
    assert build.ext_path() == here and os.path.dirname(here) == build.PKG
    seen = {here}
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", torch.__version__ + ".later")
        seen.add(build.ext_path())
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: ".cpython-399-x86_64-linux-gnu.so")
        seen.add(build.ext_path())
    with monkeypatch.context() as m:
        m.setattr(torch, "compiled_with_cxx11_abi", lambda: not torch._C._GLIBCXX_USE_CXX11_ABI)
        seen.add(build.ext_path())
    other = tmp_path / "tensors.cpp"
    with open(build.EXT_SRC) as f:
        other.write_text(f.read() + "\n// changed\n")
    monkeypatch.setattr(build, "EXT_SRC", str(other))
    seen.add(build.ext_path())
    assert len(seen) == 5
