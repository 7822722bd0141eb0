"""The binding's native argument checks answer as the Python functions do: the
same calls pass, the others raise the same error."""
import subprocess

import pytest
import torch

import unpermute_count_expert_amd as moe
from unpermute_count_expert_amd import _lib, build

BF = torch.bfloat16
py_arg, py_device, py_ptr = _lib.PYTHON_CHECKS
needs_native = pytest.mark.skipif(_lib._host is None, reason="_host.so is not built")


def outcome(f, *args, **kw):
    try:
        return f(*args, **kw)
    except Exception as e:   # noqa: BLE001 - the error itself is what is compared
        return type(e), str(e)


class Sub(torch.Tensor):
    pass


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


ARGS = [z(3, 4), z(3, 4, dtype=torch.int16), z(3, 4, dtype=torch.float32), z(4, 3).t(), z(6, 4)[::2], z(3, 8)[:, :4], z(5, 4),
        z(3, 4, 1), z(12), z(0, 4), z(1, 4).expand(3, 4), torch.nn.Parameter(z(3, 4)), z(3, 4).as_subclass(Sub), None, 5,
        "x", [z(3, 4)], torch.zeros(3, 4, dtype=BF, device="meta"), torch.eye(3).to_sparse(), z(3, 4).requires_grad_(),
        torch.zeros(3, 4, dtype=torch.complex64).conj()]


@needs_native
@pytest.mark.parametrize("i", range(len(ARGS)))
def test_check_arg(i):
    t = ARGS[i]
    for dtypes in (_lib.BF16, _lib.F32, (torch.complex64,), ()):
        assert outcome(_lib.check_arg, t, "t", dtypes) == outcome(py_arg, t, "t", dtypes)
        for shape in ((3, 4), (None, 4), (3, None), (None, None), (3,), (), (3, 4, 1), (12,), (0, 4), (None,), (5, 4)):
            assert outcome(_lib.check_arg, t, "t", dtypes, shape) == outcome(py_arg, t, "t", dtypes, shape)
            for kw in (dict(min_rows=2), dict(min_rows=3), dict(min_rows=4), dict(optional=True), dict(optional=False),
                       dict(min_rows=3, optional=True)):
                assert outcome(_lib.check_arg, t, "t", dtypes, shape, **kw) == outcome(py_arg, t, "t", dtypes, shape, **kw)
                assert outcome(_lib.check_arg, t, "t", dtypes, shape=shape, **kw) == \
                    outcome(py_arg, t, "t", dtypes, shape=shape, **kw)


@needs_native
def test_check_arg_called_wrongly():
    t = z(2)
    for args, kw in (((), {}), ((t,), {}), ((t, "t"), {}), ((t, "t", _lib.BF16, (2,), None, False, 1), {}),
                     ((t, "t", _lib.BF16), dict(nothing=1)), ((t, "t", _lib.BF16, (2,)), dict(shape=(2,))),
                     ((t, "t", BF), {}), ((t, "t", _lib.BF16, 2), {}), ((t, "t", _lib.BF16, ("2",)), {}),
                     ((t, "t", _lib.BF16, (2.0,)), {}), ((t, "t", _lib.BF16, (1 << 80,)), {}), ((t, "t", _lib.BF16, [2]), {})):
        got, want = outcome(_lib.check_arg, *args, **kw), outcome(py_arg, *args, **kw)
        assert got == want, (args, kw)


@needs_native
@pytest.mark.parametrize("args", [(), (None,), (None, None), (z(2),), (None, z(2)), (5,), (z(2), "x")])
def test_check_device_on_the_cpu(args):
    assert outcome(_lib.check_device, *args) == outcome(py_device, *args)


@needs_native
def test_ptr():
    for t in (None, z(3), z(3)[1:], z(0), 5, z(3).as_subclass(Sub), torch.nn.Parameter(z(2))):
        assert outcome(_lib._ptr, t) == outcome(py_ptr, t)


@needs_native
def test_gradient_lists_on_the_cpu_are_left_to_python():
    for lists in (([], []), ([z(2)], [z(2)]), ([z(2), 5], [z(2), 5]), ([None], [None])):
        assert _lib._host.grad_words(*lists) is None
    with pytest.raises(ValueError, match="current CUDA device"):
        moe.moe_grad_sumsq([z(3)], torch.zeros(1, dtype=torch.float64), torch.zeros(64, dtype=torch.uint8))


@needs_native
@pytest.mark.gpu
def test_on_the_gpu(monkeypatch):
    c = lambda *shape, dtype=BF: z(*shape, dtype=dtype).to("cuda")
    good = [c(3), c(4, 5, dtype=torch.float32), c(7, dtype=torch.int16), c(0), torch.nn.Parameter(c(9)), c(8)[3:], c(2, 1)]
    outs = [torch.empty_like(t) for t in good]
    outs[3], outs[5] = good[3], good[5]   # some in place
    for t in good:
        assert _lib.check_device(t, None, t) is None and _lib._ptr(t) == py_ptr(t)
    for bad in ((c(2), z(2)), (z(2), c(2)), (c(2), None, 7)):
        assert outcome(_lib.check_device, *bad) == outcome(py_device, *bad) != None   # noqa: E711
    lists = [(good, good), (good, outs), (good, outs[:-1]), ([], []), (good + [z(3)], good + [z(3)]),
             ([c(4, 4).t()], [c(4, 4)]), ([c(4)], [c(4, dtype=torch.float32)]), ([c(4)], [c(5)]),
             ([c(4).double()], [c(4).double()]), ([c(4), 5], [c(4), 5]), ([c(4).as_subclass(Sub)], [c(4)]), ([c(4)], [z(4)])]
    native = [outcome(_lib._grad_list, g, g if g is o else o) for g, o in lists]
    monkeypatch.setattr(_lib, "_host", None)
    for (g, o), got in zip(lists, native):
        assert got == outcome(_lib._grad_list, g, g if g is o else o)
    assert isinstance(native[0], bytes) and isinstance(native[1], bytes) and native[2][0] is ValueError


@pytest.mark.parametrize("error", [FileNotFoundError("no compiler"), subprocess.CalledProcessError(1, "c++"),
                                   ImportError("no torch headers")])
def test_build_without_the_native_checks(monkeypatch, tmp_path, capfd, error):
    """Where the module cannot be built the library still is, and a module of older sources is not left behind."""
    lib, host = tmp_path / "lib.so", tmp_path / "host.so"
    host.write_text("older")
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "HOST", str(host))
    monkeypatch.setenv("CXX", "the-cxx")

    def check_call(cmd):
        if cmd[0] == "the-cxx":
            raise error
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("library")

    monkeypatch.setattr(subprocess, "check_call", check_call)
    assert build.build() == str(lib)
    assert lib.read_text() == "library" and not host.exists()
    assert "argument checks" in capfd.readouterr().err


def test_build_fails_without_the_library(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "HIPCC", str(tmp_path / "no-hipcc"))
    with pytest.raises(FileNotFoundError):
        build.build()
