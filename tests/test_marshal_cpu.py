"""The binding's host library against the Python functions it stands for: the same
answers, the same exceptions, on tensors of every kind a call may be given (on the CPU:
nothing is dereferenced), and its calls against ctypes'."""
import itertools

import pytest
import torch

import sharded_mixed_precision_step_amd as zs
from sharded_mixed_precision_step_amd import _marshal, model, train

pytestmark = pytest.mark.cpu
CPU, GPU = torch.device("cpu"), torch.device("cuda:0")


def _outcome(f, *args):
    try:
        return f(*args)
    except Exception as e:  # noqa: BLE001
        return type(e), str(e)


def _same(fast, slow, *args):
    a, b = _outcome(fast, *args), _outcome(slow, *args)
    assert a == b, (args, a, b)
    return a


TENSORS = [torch.zeros(s, dtype=d) for s, d in itertools.product(
    [(), (3,), (0,), (4, 7), (1, 7), (7, 1), (0, 5), (5, 0), (1, 1), (2, 3, 4)],
    [torch.float32, torch.float16, torch.bfloat16, torch.int32, torch.int64, torch.uint8,
     torch.float64, torch.bool])]
TENSORS += [torch.zeros(6, 9)[:, 2:5], torch.zeros(6, 9).t(), torch.zeros(6, 9)[::2],
            torch.zeros(6, 9)[:1, 3:], torch.zeros(6, 9)[:, :1], torch.zeros(20)[::2],
            torch.zeros(4, 7).to_sparse(), torch.zeros(4, 7, requires_grad=True),
            torch.nn.Parameter(torch.zeros(4, 7))]
OTHERS = [None, 5, "x", [1, 2]]
KINDS = [train._ELEM, train._FP8, train._SCALE, train._INDEX, train._F32, train._BYTES, {}]


def test_matrices_and_vectors():
    answered = 0
    for t in TENSORS + OTHERS:
        for kinds in KINDS:
            for dev in (CPU, GPU):
                answered += isinstance(_same(_marshal.mat, train._mat_checked, t, kinds, dev, "x")
                                       [0], int)
                for n in (0, 1, 3, 7, 28, 27):
                    _same(_marshal.vec, train._vec_checked, t, n, kinds, dev, "v")
                for shape in ((4, 7), (4, 8), (7, 1), torch.Size((4, 7)), torch.Size((0, 5)),
                              torch.Size((1, 7)), torch.Size((3,))):
                    _same(_marshal.like, train._like_checked, t, shape, kinds, dev, "m")
    assert answered > 20


def test_q8_pairs():
    answered = 0
    for rows, cols in itertools.product((0, 1, 5), (0, 1, 127, 128, 129, 600)):
        for d8 in (torch.float8_e4m3fn, torch.float8_e5m2):
            q, s = zs.q8_empty(rows, cols, d8, "cpu")
            wide = torch.zeros(rows + 2, q.shape[1] + 128, dtype=d8)[1:rows + 1, 16:]
            for pair in ((q, s), (q, s.view(torch.uint8)), (None, None), (q, None), (None, s),
                         (s, q), (wide, s), (q.view(torch.uint8), s), (q[:, :-16], s),
                         (q, s[:, :-1])):
                for fmt in (None, 0, 1):
                    for r, c in ((rows, cols), (rows + 1, cols), (rows, cols + 128)):
                        got = _same(_marshal.q8, train._q8_checked, *pair, r, c, CPU, "q", fmt)
                        answered += len(got) == 5
                got = _same(_marshal.q8, train._q8_checked, *pair, rows, cols, CPU, "q")
                _same(_marshal.q8, train._q8_checked, *pair, rows, cols, GPU, "q")
    assert answered > 100


def test_wrong_numbers_of_arguments_are_refused():
    t = torch.zeros(4, 7)
    for f in (_marshal.mat, _marshal.like, _marshal.vec, _marshal.q8):
        with pytest.raises(TypeError):
            f(t)
    for name in ("init", "bind"):
        with pytest.raises((TypeError, KeyError)):
            getattr(_marshal, name)({})


def test_the_calls_take_what_ctypes_takes():
    """Refused at once, before anything is looked at: the same status and text."""
    args = [1, 7, 4096, None, 1, 4096, 1, None, 1, -1, 4096, 1e-5, None, 0, None, 1, 4096, None, 0,
            4096, None, 32, None, None, None]
    for call in (_marshal.zero_layernorm, zs.lib.zero_layernorm):
        assert call(*args) == -1
        assert "rows = -1" in zs.lib.zero_last_error_string().decode()
    for bad, error in ((args[:-1], TypeError), (args + [0], TypeError),
                       (["x"] + args[1:], TypeError), (args[:9] + [1 << 70] + args[10:],
                                                      OverflowError),
                       (args[:1] + [1 << 40] + args[2:], OverflowError),
                       (args[:11] + ["x"] + args[12:], TypeError)):
        with pytest.raises(error):
            _marshal.zero_layernorm(*bad)
    for name in model.EXPORTED:
        if not name.endswith(("workspace", "_ctl")):
            assert callable(getattr(_marshal, name)), name
