"""CPU checks of the binding's layer lists: descriptors of a class derived from the library's are taken, others are not."""
import ctypes

import pytest

from test_kv4_host import A, e3, kv4, kv16  # noqa: F401 (e3 is a fixture)
from test_kv8_host import kv8


@pytest.mark.parametrize("name", ["kv4", "kv8"])
def test_layer_lists(e3, name):  # noqa: F811
    make, base, other = (kv4, e3.e3_kv4_layer, e3.e3_kv8_layer) if name == "kv4" else (kv8, e3.e3_kv8_layer, e3.e3_kv4_layer)

    class Mine(base):
        """With what a program keeps beside a descriptor."""

    class Mine16(e3.e3_kv_layer):
        pass

    class Wider(base):
        _fields_ = [("more", ctypes.c_int * 4)]

    def as_(kind, d):
        x = kind()
        ctypes.memmove(ctypes.byref(x), ctypes.byref(d), ctypes.sizeof(d))
        return x
    a, b = make(e3), kv16(e3)
    plain = e3._layer_arrays("f", [a, a], [b, b], base)
    for layers, others in (([as_(Mine, a)] * 2, [b, b]), ([a, as_(Mine, a)], [as_(Mine16, b), b]), ((base * 2)(a, a), (e3.e3_kv_layer * 2)(b, b))):
        got = e3._layer_arrays("f", layers, others, base)
        assert [bytes(x) for x in got] == [bytes(x) for x in plain]
    for layers, others in (([as_(Wider, a)] * 2, [b, b]), ([as_(other, a)] * 2, [b, b]), ([a, a], [a, a]), ([b, b], [b, b]), ([a, b], [b, a]),
                           ([bytes(a)] * 2, [b, b])):
        with pytest.raises(TypeError):
            e3._layer_arrays("f", layers, others, base)
    with pytest.raises(ValueError):
        e3._layer_arrays("f", [a], [b, b], base)
    # to the entry point, where the host's own checks come next
    with pytest.raises(e3.E3Error):
        getattr(e3, name + "_append")([as_(Mine, a)], [as_(Mine16, b)], 0, 7, None, A, 0, A, None, stream=0)
