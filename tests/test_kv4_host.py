"""CPU checks of the verify pass over a 4-bit cache: refusals before any launch, the
rotary frequencies, and the plain forms that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest

import kv4_ref


@pytest.fixture(scope="module")
def e3():
    from eagle_speculative_decoding_round_gb300 import build
    build.build()
    from eagle_speculative_decoding_round_gb300 import eagle3
    return eagle3


def refused(e3, status, call, *args, **kw):
    n0 = e3.launch_count()
    with pytest.raises(e3.E3Error) as ei:
        call(*args, stream=0, **kw)
    assert ei.value.status == status, ei.value
    assert e3.last_error() and e3.launch_count() == n0


A = 4096  # a plausible aligned address; no call below reaches the device


def kv16(e3, hd=128, KVH=8, page=64, maxp=40, dt=None, flags=0, k=A):
    return e3.make_kv_layer(k, A, A, 10, page, maxp, KVH, hd, e3.E3_BF16 if dt is None else dt, flags)


def kv4(e3, hd=128, KVH=8, page=64, maxp=40, unit=1.0, flags=0, ks=A, n=10):
    return e3.make_kv4_layer(A, A, ks, A, A, n, page, maxp, KVH, hd, unit, 1.0, flags)


def test_qkv_append_refusals(e3):
    rope = e3.eagle3_rope_init(128, 10000.0)

    def call(qkv=A, ld=6144, B=1, R=61, H=32, qn=None, eps=1e-5, rp=rope, pos=A, kv=None, stream=0):
        e3.tree_qkv_append(qkv, ld, B, R, None, H, qn, None, eps, rp, pos, A, kv or kv16(e3), None, None, stream=stream)
    refused(e3, 1, call, qkv=None)
    refused(e3, 1, call, pos=None)                      # a rotation without positions
    refused(e3, 2, call, ld=6143)                       # rows shorter than their heads
    refused(e3, 2, call, B=0)
    refused(e3, 2, call, R=0)
    refused(e3, 2, call, B=1 << 16, R=1 << 15)          # 2^31 rows
    refused(e3, 2, call, H=0)
    refused(e3, 2, call, kv=kv16(e3, hd=64), ld=6144)   # rot_dim 128 in heads of 64
    refused(e3, 2, call, kv=kv16(e3, hd=100))
    refused(e3, 2, call, kv=kv16(e3, page=24))
    refused(e3, 1, call, kv=kv16(e3, k=A + 4))          # misaligned cache
    refused(e3, 1, call, kv=kv16(e3, dt=7))
    refused(e3, 1, call, kv=kv16(e3, flags=6))
    refused(e3, 1, call, qn=A, eps=-1.0)
    refused(e3, 1, call, qn=A, eps=float("nan"))


def test_kv4_row_refusals(e3):
    def append(layers=None, src=None, B=2, m=7, add=0, stream=0):
        e3.kv4_append(layers or [kv4(e3)], src or [kv16(e3)], B, m, None, A, add, A, None, None, stream=stream)

    def read(layers=None, dst=None, B=2, m=7, stream=0):
        e3.kv4_read(layers or [kv4(e3)], dst or [kv16(e3)], B, m, None, A, None, stream=stream)
    for call, other in ((append, "src"), (read, "dst")):
        refused(e3, 2, call, B=0)
        refused(e3, 2, call, B=65536)
        refused(e3, 2, call, m=0)
        refused(e3, 2, call, layers=[kv4(e3, hd=96)])
        refused(e3, 2, call, layers=[kv4(e3, page=8)])
        refused(e3, 2, call, layers=[kv4(e3, n=0)])
        refused(e3, 1, call, layers=[kv4(e3, ks=A + 8)])
        for unit in (0.0, -1.0, 3.0, 2.0 ** 61, 2.0 ** -61, float("inf"), float("nan")):
            refused(e3, 1, call, layers=[kv4(e3, unit=unit)])
        refused(e3, 1, call, layers=[kv4(e3, flags=2)])
        refused(e3, 3, call, **{other: [kv16(e3, dt=e3.E3_F32)]})
        refused(e3, 2, call, **{other: [kv16(e3, hd=64)]})
        refused(e3, 2, call, **{other: [kv16(e3, KVH=4)]})
        refused(e3, 2, call, layers=[kv4(e3), kv4(e3, page=128)], **{other: [kv16(e3)] * 2})
        refused(e3, 2, call, layers=[kv4(e3)] * 129, **{other: [kv16(e3)] * 129})
        with pytest.raises(ValueError):
            call(layers=[kv4(e3)] * 2)
    refused(e3, 2, append, add=2)
    refused(e3, 2, append, add=-1)


def test_verify4_refusals(e3):
    def call(Q=A, kv=None, tail=None, B=1, R=61, H=32, P=2048, scale=0.1, ws=A, n=1 << 40, stream=0):
        e3.tree_verify_attn4(Q, kv or kv4(e3), tail or kv16(e3), A, A, B, R, H, P, scale, A, A, None, ws, n, stream=stream)
    refused(e3, 1, call, Q=None)
    refused(e3, 1, call, Q=A + 2)
    refused(e3, 1, call, ws=None)
    refused(e3, 4, call, n=1000)                                # workspace too small
    refused(e3, 2, call, R=257)
    refused(e3, 2, call, R=0)
    refused(e3, 2, call, B=65536)
    refused(e3, 2, call, H=30)                                  # not a multiple of the KV heads
    refused(e3, 2, call, P=-1)
    refused(e3, 4, call, P=40 * 64 + 1)                         # beyond the pages
    refused(e3, 4, call, tail=kv16(e3, page=16, maxp=3))        # tail pages do not hold R
    refused(e3, 3, call, tail=kv16(e3, dt=e3.E3_F32))
    refused(e3, 2, call, tail=kv16(e3, hd=64))
    refused(e3, 2, call, tail=kv16(e3, KVH=4))
    refused(e3, 1, call, scale=0.0)
    refused(e3, 1, call, scale=float("nan"))
    refused(e3, 2, call, kv=kv4(e3, hd=32))
    assert e3.eagle3_verify4_workspace_bytes(0, 1, 1, 1, 128, 0) == 0
    assert e3.eagle3_verify4_workspace_bytes(1, 1, 3, 2, 128, 0) == 0


def test_logits_refusals(e3):
    def call(z=A, B=1, R=61, V=1000, tok=A, par=A, bt=None, nb=0, allow=None, na=0, out=A, stream=0):
        e3.tree_logits_process(z, B, R, V, A, None, tok, par, None, bt, bt, nb, allow, None, na, out, A, A, A, None,
                               stream=stream)
    refused(e3, 1, call, z=None)
    refused(e3, 1, call, out=None)
    refused(e3, 1, call, tok=None)                    # parents without tokens
    refused(e3, 2, call, B=0)
    refused(e3, 2, call, R=257)
    refused(e3, 2, call, V=0)
    refused(e3, 2, call, V=1 << 30)
    refused(e3, 2, call, bt=A, nb=1025)
    refused(e3, 2, call, nb=-1)
    refused(e3, 1, call, nb=3)                        # a count without a list
    refused(e3, 2, call, allow=A, na=0)
    for kw in (dict(V=0), dict(B=0), dict(m=0), dict(add=2)):
        d = dict(V=1000, B=1, m=7, add=1) | kw
        refused(e3, 2, e3.token_counts_add, A, d["V"], d["B"], A, A, d["add"], d["m"])
    refused(e3, 1, e3.token_counts_add, A + 2, 1000, 1, A, A, 0, 7)
    refused(e3, 1, e3.token_counts_add, None, 1000, 1, A, A, 0, 7)


@pytest.mark.parametrize("rot,base,scaling,kw", [
    (128, 10000.0, "plain", {}), (64, 500000.0, "linear", dict(factor=4.0)),
    (128, 500000.0, "wavelen", dict(factor=8.0, low=1.0, high=4.0, orig_len=8192.0)),
    (64, 10000.0, "yarn", dict(factor=16.0, low=1.0, high=32.0, orig_len=4096.0)), (2, 10.0, "plain", {}),
    (256, 1e6, "linear", dict(factor=0.01))])
def test_rope_frequencies(e3, rot, base, scaling, kw):
    kind = dict(plain=e3.E3_ROPE_PLAIN, linear=e3.E3_ROPE_LINEAR, wavelen=e3.E3_ROPE_WAVELEN, yarn=e3.E3_ROPE_YARN)[scaling]
    r = e3.eagle3_rope_init(rot, base, scaling=kind, **kw)
    f, amp = kv4_ref.rope_freqs(rot, base, scaling, **kw)
    got = np.array([r.turns[i] for i in range(rot // 2)], np.float64) * 2.0 ** -64
    want = (f / (2 * math.pi)) % 1.0
    # double arithmetic on both sides: a few roundings of values below 16 turns
    assert np.all(np.abs(got - want) <= 2.0 ** -46), np.abs(got - want).max()
    assert abs(r.amp - amp) <= 2.0 ** -23 * amp
    assert r.rot_dim == rot


def test_rope_refusals(e3):
    ok = dict(rot_dim=64, base=10000.0)
    e3.eagle3_rope_init(**ok)
    for status, kw in [(2, dict(rot_dim=63)), (2, dict(rot_dim=0)), (2, dict(rot_dim=258)), (1, dict(base=1.0)),
                       (1, dict(base=float("nan"))), (1, dict(scaling=4)), (1, dict(scaling=-1)), (1, dict(amp=-1.0)),
                       (1, dict(scaling=1, factor=0.0)), (1, dict(scaling=2, factor=8.0, low=4.0, high=4.0)),
                       (1, dict(scaling=3, factor=8.0, orig_len=0.0))]:
        with pytest.raises(e3.E3Error) as ei:
            e3.eagle3_rope_init(**(ok | kw))
        assert ei.value.status == status, kw
    assert e3.lib().eagle3_rope_init(None, ctypes.byref(e3.e3_rope())) == 1


def test_plain_quantizer():
    """The test's own quantizer: every value on the grid comes back, the nearest value is taken, ties go to even codes."""
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 16, (50, 128))
    codes[:, ::16] = 7  # the largest magnitude present: the scale is recovered
    full = np.concatenate([kv4_ref.GRID, -kv4_ref.GRID])
    scales = rng.integers(8, 100, (50, 8))
    x = full[codes] * np.repeat(kv4_ref.E4M3[scales], 16, 1)
    c, e = kv4_ref.quantize(x, 1.0)
    assert np.array_equal(e, scales) and np.array_equal(kv4_ref.dequantize(c, e, 1.0), x)
    mids = (kv4_ref.GRID[1:] + kv4_ref.GRID[:-1]) / 2
    assert np.array_equal(kv4_ref.nearest_even(mids, kv4_ref.GRID), [0, 2, 2, 4, 4, 6, 6])
    y = rng.normal(size=(20, 64)) * np.exp(rng.normal(size=(20, 1)))
    c, e = kv4_ref.quantize(y, 0.25)
    d = kv4_ref.dequantize(c, e, 0.25)
    step = np.repeat(kv4_ref.E4M3[e] * 0.25, 16, 1)
    # half the widest grid gap, or clipping by the scale's own rounding (half of 2^-3 of 6 steps)
    assert np.all(np.abs(d - y) <= step * 1.0 + 1e-12)


def test_pointers_off_their_elements_are_refused(e3):
    """Rows may start anywhere on their elements' grid (the scalar paths take those), but not off it."""
    def qkv(x=A, q=A, dt=None, hd=64):
        e3.tree_qkv_append(x, 3 * hd + 1, 1, 1, None, 1, None, None, 0.0, None, None, q, kv16(e3, hd=hd, KVH=1, dt=dt), None, None,
                           stream=0)

    def logits(z=A, counts=None, out=A):
        e3.tree_logits_process(z, 1, 1, 1000, A, counts, None, None, None, None, None, 0, None, None, 0, out, A, A, A, None, stream=0)
    n0 = e3.launch_count()
    for call, kw in ((qkv, dict(x=A + 1)), (qkv, dict(q=A + 1)), (qkv, dict(x=A + 2, dt=e3.E3_F32)), (qkv, dict(q=A + 2, dt=e3.E3_F32)),
                     (logits, dict(z=A + 2)), (logits, dict(out=A + 1)), (logits, dict(counts=A + 1))):
        with pytest.raises(e3.E3Error) as ei:
            call(**kw)
        assert ei.value.status == 1 and e3.launch_count() == n0, kw


def test_layer_lists_of_the_wrong_kind_are_refused(e3):
    """A descriptor of the other cache's kind would be read as pointers that it does not hold."""
    for call in (lambda a, b: e3.kv4_append(a, b, 1, 1, None, A, 0, A, None, None, stream=0),
                 lambda a, b: e3.kv4_read(a, b, 1, 1, None, A, None, stream=0)):
        for a, b in (([kv4(e3)], [kv4(e3)]), ([kv16(e3)], [kv16(e3)]), ([kv16(e3)], [kv4(e3)]), ([kv4(e3), kv16(e3)], [kv16(e3)] * 2)):
            n0 = e3.launch_count()
            with pytest.raises(TypeError):
                call(a, b)
            assert e3.launch_count() == n0


@pytest.mark.parametrize("missing", [(), ("_cuda_getCurrentRawStream",), ("_cuda_getDevice",)])
def test_current_stream_without_the_short_call(e3, monkeypatch, missing):
    """The stream of a call: by torch's short call where torch has it, else by its public one."""
    import sys
    import types
    fake = types.ModuleType("torch")
    short = {"_cuda_getCurrentRawStream": lambda d: 100 + d, "_cuda_getDevice": lambda: 1}
    fake._C = types.SimpleNamespace(**{k: v for k, v in short.items() if k not in missing})
    fake.cuda = types.SimpleNamespace(current_stream=lambda *a: types.SimpleNamespace(cuda_stream=77))
    monkeypatch.setitem(sys.modules, "torch", fake)
    for name in ("_torch_c", "_current_stream"):  # what the first call leaves
        if hasattr(e3, name):
            monkeypatch.setattr(e3, name, None)
    assert [e3._stream(None) for _ in range(2)] == ([77, 77] if missing else [101, 101])
    assert e3._stream(5) == 5 and e3._stream(types.SimpleNamespace(cuda_stream=9)) == 9


def test_workspace_is_asked_for_calls_that_are_taken(e3):
    """0 for what tree_verify_attn4 refuses, and no arithmetic that wraps on the way."""
    ok = dict(B=2, R=61, H=32, KVH=8, hd=128, P=4096)
    ask = lambda **kw: e3.eagle3_verify4_workspace_bytes(*(ok | kw).values())  # noqa: E731
    assert ask() > 0 and ask(hd=64) > 0 and ask(R=256, P=0) > 0 and ask(B=65535, R=1) > 0
    for kw in (dict(B=0), dict(B=65536), dict(R=0), dict(R=257), dict(R=70000, H=70000, KVH=1), dict(H=65536), dict(H=30), dict(KVH=0),
               dict(hd=96), dict(hd=0), dict(P=-1), dict(P=(1 << 30) + 1), dict(B=65535, R=256, H=65535, KVH=1)):
        assert ask(**kw) == 0, kw
