"""The gated recurrence, the experts' calls and the gradient norm refuse bad
arguments on the host, before any CUDA work (no GPU needed: none of these calls
reaches a kernel), and their plain test implementations agree with worked
examples and with differences."""
import ctypes

import numpy as np
import pytest

import model_ref as ref


@pytest.fixture(scope="module")
def lib():
    from stream_compaction_device_gb300 import build as b
    b.build()
    from stream_compaction_device_gb300 import _lib
    return _lib.load()


def at(i, by=0):
    """A pointer that is never dereferenced; 16 MiB apart from the others."""
    return ctypes.c_void_p(((i + 1) << 24) + by)


def refuser(fn, good):
    def call(**change):
        args = list(good)
        for k, v in change.items():
            args[int(k[1:])] = v
        return fn(*args)
    return call


def test_gated_scan_refusals(lib):
    from stream_compaction_device_gb300._lib import ERR_INVALID, GATED_SYMBOLS, OK
    for name in GATED_SYMBOLS:
        size = 4 if name.endswith("f32") else 2
        # x, strides, gate, strides, gate_f32, rows, tokens, channels, starts, initial, slots, pool, kind, out, strides, final
        call = refuser(getattr(lib, name), [at(0), 800, 8, at(1), 800, 8, 0, 4, 100, 8, None, at(2), None, 4, 0, at(3),
                                            800, 8, at(4), None])
        for i in (0, 3, 15):
            assert call(**{f"a{i}": None}) == ERR_INVALID, i           # a missing buffer
        assert call(a9=0) == ERR_INVALID                               # no channels
        assert call(a14=3) == ERR_INVALID and call(a14=-1) == ERR_INVALID
        assert call(a7=2**31) == ERR_INVALID and call(a8=2**31) == ERR_INVALID
        assert call(a9=2**31 - 2, a2=2**31, a17=2**31, a1=2**40, a16=2**40) == ERR_INVALID
        assert call(a7=2**20, a8=2**20) == ERR_INVALID                 # tokens past 32 bits
        assert call(a1=2**62) == ERR_INVALID and call(a2=2**62) == ERR_INVALID
        assert call(a17=7) == ERR_INVALID                              # output tokens overlap
        assert call(a16=700) == ERR_INVALID                            # output rows overlap
        assert call(a13=3) == ERR_INVALID                              # fewer states than rows
        assert call(a0=at(0, 1)) == ERR_INVALID                        # alignment
        assert call(a6=1, a3=at(1, 2)) == ERR_INVALID
        assert call(a11=at(2, 2)) == ERR_INVALID and call(a18=at(4, 1)) == ERR_INVALID
        assert call(a10=at(5, 2)) == ERR_INVALID and call(a12=at(5, 1)) == ERR_INVALID
        assert call(a15=at(1)) == ERR_INVALID                          # out on the gates
        assert call(a15=at(0, 4 * size)) == ERR_INVALID                # out shifted within x
        assert call(a15=at(2)) == ERR_INVALID                          # out on the states
        assert call(a18=at(2, 32)) == ERR_INVALID                      # final half on initial
        assert call(a18=at(0)) == ERR_INVALID                          # final on x
        assert call(a10=at(3), a7=4) == ERR_INVALID                    # starts on out
        assert call(a12=at(4)) == ERR_INVALID                          # slots on final
        assert call(a7=0) == OK                                        # no rows


def test_gated_backward_refusals(lib):
    from stream_compaction_device_gb300._lib import ERR_INVALID, GATED_BACKWARD_SYMBOLS, OK
    for name in GATED_BACKWARD_SYMBOLS:
        good = []
        for i in range(3):
            good += [at(i), 800, 8]                                    # grad, x, gate
        good += [0, at(3), 800, 8, 4, 100, 8, None, at(4), at(5), 2]   # gate_f32, y, sizes, starts, initial, grad_final, kind
        good += [at(6), 800, 8, at(7), 800, 8, at(8), None]
        call = refuser(getattr(lib, name), good)
        for i in (0, 3, 6, 10, 20, 23):
            assert call(**{f"a{i}": None}) == ERR_INVALID, i
        assert call(a19=5) == ERR_INVALID and call(a15=0) == ERR_INVALID
        assert call(a22=7) == ERR_INVALID and call(a24=3) == ERR_INVALID
        assert call(a20=at(0)) == ERR_INVALID and call(a23=at(3)) == ERR_INVALID    # outputs on inputs
        assert call(a23=at(6)) == ERR_INVALID                                       # both outputs at once
        assert call(a26=at(4)) == ERR_INVALID and call(a26=at(5)) == ERR_INVALID and call(a26=at(0)) == ERR_INVALID
        assert call(a20=at(4)) == ERR_INVALID
        assert call(a26=at(8, 1)) == ERR_INVALID
        assert call(a13=0) == OK


def test_expert_refusals(lib):
    from stream_compaction_device_gb300 import _lib
    from stream_compaction_device_gb300._lib import ERR_INVALID, OK
    for name in _lib.EXPERT_SORT_SYMBOLS:
        call = refuser(getattr(lib, name), [at(0), 100, 2, 8, 4, 300, at(1), at(2), at(3), at(4), None])
        for i in (0, 6, 7, 8, 9):
            assert call(**{f"a{i}": None}) == ERR_INVALID, i
        assert call(a2=0) == ERR_INVALID and call(a3=0) == ERR_INVALID and call(a3=1025) == ERR_INVALID
        assert call(a4=0) == ERR_INVALID and call(a1=2**31) == ERR_INVALID and call(a5=2**31) == ERR_INVALID
        assert call(a1=2**20, a2=2**12) == ERR_INVALID and call(a3=1024, a4=2**22) == ERR_INVALID
        assert call(a0=at(0, 2)) == ERR_INVALID and call(a8=at(3, 1)) == ERR_INVALID
        assert call(a9=at(0)) == ERR_INVALID and call(a7=at(1, 8)) == ERR_INVALID and call(a9=at(3, 400)) == ERR_INVALID
    call = refuser(lib.expert_dispatch, [at(0), 64, 64, 100, 2, at(1), 300, at(2), at(3), 64, None])
    for i in (0, 5, 8):
        assert call(**{f"a{i}": None}) == ERR_INVALID, i
    assert call(a1=63) == ERR_INVALID and call(a9=63) == ERR_INVALID and call(a2=0) == ERR_INVALID
    assert call(a4=0) == ERR_INVALID and call(a3=2**31) == ERR_INVALID and call(a6=2**31) == ERR_INVALID
    assert call(a1=2**61) == ERR_INVALID and call(a8=at(0)) == ERR_INVALID and call(a8=at(1)) == ERR_INVALID
    assert call(a8=at(2, 16)) == ERR_INVALID and call(a5=at(1, 2)) == ERR_INVALID
    assert call(a6=0) == OK
    for name in _lib.EXPERT_COMBINE_SYMBOLS:
        call = refuser(getattr(lib, name), [at(0), 32, 300, 100, 2, 32, at(1), at(2), at(3), 32, None])
        for i in (0, 6, 8):
            assert call(**{f"a{i}": None}) == ERR_INVALID, i
        assert call(a1=31) == ERR_INVALID and call(a9=31) == ERR_INVALID and call(a5=0) == ERR_INVALID
        assert call(a4=0) == ERR_INVALID and call(a8=at(0)) == ERR_INVALID and call(a8=at(2)) == ERR_INVALID
        assert call(a8=at(3, 1)) == ERR_INVALID and call(a7=at(2, 2)) == ERR_INVALID and call(a1=2**60) == ERR_INVALID
        assert call(a3=0) == OK
    for name in _lib.EXPERT_COMBINE_BACKWARD_SYMBOLS:
        call = refuser(getattr(lib, name), [at(0), 32, at(1), 32, 300, 100, 2, 32, at(2), at(3), at(4), at(5), 32, at(6), None])
        for i in (0, 2, 8, 11):
            assert call(**{f"a{i}": None}) == ERR_INVALID, i
        assert call(a1=31) == ERR_INVALID and call(a3=31) == ERR_INVALID and call(a12=31) == ERR_INVALID
        assert call(a11=at(0)) == ERR_INVALID and call(a11=at(1)) == ERR_INVALID and call(a13=at(3)) == ERR_INVALID
        assert call(a13=at(5)) == ERR_INVALID and call(a13=at(6, 2)) == ERR_INVALID


def test_norm_refusals(lib):
    from stream_compaction_device_gb300 import _lib
    from stream_compaction_device_gb300._lib import ERR_INVALID, Tensor
    assert _lib.norm_work_bytes(511) == 8192 and _lib.norm_work_bytes(512) == 16384

    def one(data=at(0), out=at(1), n=100, kind=0):
        return (Tensor * 1)(Tensor(data, out, n, kind))

    good = one()
    call = refuser(lib.clip_grad_norm, [good, 1, 1.0, at(2), at(3), 8192, None])
    assert call(a0=None) == ERR_INVALID and call(a3=None) == ERR_INVALID and call(a4=None) == ERR_INVALID
    assert call(a2=-1.0) == ERR_INVALID and call(a2=float("nan")) == ERR_INVALID and call(a5=8191) == ERR_INVALID
    assert call(a1=2**24 + 1) == ERR_INVALID and call(a3=at(2, 2)) == ERR_INVALID and call(a4=at(3, 4)) == ERR_INVALID
    assert call(a3=at(0)) == ERR_INVALID and call(a4=at(1)) == ERR_INVALID and call(a4=at(2)) == ERR_INVALID
    for bad in (one(data=None), one(out=None), one(kind=3), one(kind=-1), one(data=at(0, 2)), one(out=at(1, 1)),
                one(n=2**61), one(out=at(0, 4))):
        assert call(a0=bad) == ERR_INVALID
    assert lib.grad_norm(one(data=None), 1, at(2), at(3), 8192, None) == ERR_INVALID


def test_python_refuses_host_tensors():
    import torch
    import stream_compaction_device_gb300 as ds
    x = torch.ones(2, 4, 8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: ds.gated_scan(x, x), lambda: ds.gated_scan_backward(x, x, x, x),
                 lambda: ds.expert_sort(i, 4), lambda: ds.expert_dispatch(x[0], i, i[0]),
                 lambda: ds.expert_combine(x[0], i), lambda: ds.expert_combine_backward(x[0], x[0], i),
                 lambda: ds.grad_norm([x])):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("kind", ["decay", "log", "sigmoid"])
def test_reference_gradients_by_differences(kind):
    """The formulas of the backward reference against central differences of the
    forward one: (f(p + d) - f(p - d)) / 2d is off by d^2 f''' / 6, here below 1e-6."""
    rng = np.random.default_rng(7)
    spans, n, c, d = [(0, 1), (1, 1), (1, 6), (6, 9)], 9, 2, 1e-4
    p = {"x": rng.standard_normal((n, c)), "gate": -rng.random((n, c)) if kind != "sigmoid" else rng.standard_normal((n, c)),
         "initial": rng.standard_normal((4, c))}
    grad, grad_final = rng.standard_normal((n, c)), rng.standard_normal((4, c))

    def loss(q):
        h, _, final, _ = ref.scan(q["x"], q["gate"], kind, spans, q["initial"])
        return (h * grad).sum() + (final * grad_final).sum()

    h = ref.scan(p["x"], p["gate"], kind, spans, p["initial"])[0]
    got = ref.scan_backward(grad, p["x"], p["gate"], h, kind, spans, p["initial"], grad_final)
    for name in p:
        for i in np.ndindex(p[name].shape):
            up, down = {k: v.copy() for k, v in p.items()}, {k: v.copy() for k, v in p.items()}
            up[name][i] += d
            down[name][i] -= d
            assert abs((loss(up) - loss(down)) / (2 * d) - got[name][0][i]) < 1e-5, (name, i)


def test_reference_examples():
    h, _, final, _ = ref.scan(np.ones((4, 1)), np.full((4, 1), 0.5), "decay", [(0, 3), (3, 4)], np.array([[8.0], [0.0]]))
    assert h[:, 0].tolist() == [5.0, 3.5, 2.75, 1.0] and final[:, 0].tolist() == [2.75, 1.0]
    starts, counts, order, places = ref.sort([[2, 0], [2, -1], [0, 2]], 3, 2, 8)
    assert starts.tolist() == [0, 2, 2, 6] and counts.tolist() == [2, 0, 3]
    assert order.tolist() == [1, 4, 0, 2, 5, -1, -2, -2] and places.tolist() == [2, 0, 3, -1, 1, 4]
    y = np.arange(8.0)[:, None]
    out, _ = ref.combine(y, np.array([[2, 0], [3, -1], [1, 4]]), np.array([[1, 2], [3, 4], [5, 6.0]]))
    assert out[:, 0].tolist() == [2.0, 9.0, 29.0]
    gy, gw, _ = ref.combine_backward(np.array([[1.0], [2], [3]]), y, np.array([[2, 0], [3, -1], [1, 4]]),
                                     np.array([[1, 2], [3, 4], [5, 6.0]]), np.zeros((8, 1)))
    assert gy[:, 0].tolist() == [2, 15, 1, 6, 18, 0, 0, 0] and gw.tolist() == [[2, 0], [6, 0], [3, 12]]
