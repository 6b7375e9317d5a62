"""CPU checks of the 8-bit cache's calls: refusals before any launch, and the plain forms that the GPU tests
compare with."""
import numpy as np
import pytest
import torch

import kv8_ref
from test_kv4_host import A, e3, kv4, kv16, refused  # noqa: F401 (e3 is a fixture)


def kv8(e3, hd=128, KVH=8, page=64, maxp=40, block=64, flags=0, k=A, ke=A, n=10):  # noqa: F811
    return e3.make_kv8_layer(k, A, ke, A, A, n, page, maxp, KVH, hd, block, flags)


def test_kv8_row_refusals(e3):  # noqa: F811
    def append(layers=None, src=None, B=2, m=7, add=0, kv_len=A, stream=0):
        e3.kv8_append(layers or [kv8(e3)], src or [kv16(e3)], B, m, None, A, add, kv_len, None, None, stream=stream)

    def read(layers=None, dst=None, B=2, m=7, stream=0):
        e3.kv8_read(layers or [kv8(e3)], dst or [kv16(e3)], B, m, None, A, None, stream=stream)
    for call, other in ((append, "src"), (read, "dst")):
        refused(e3, 2, call, B=0)
        refused(e3, 2, call, B=65536)
        refused(e3, 2, call, m=0)
        refused(e3, 2, call, m=1 << 30)
        refused(e3, 2, call, layers=[kv8(e3, hd=96)])
        refused(e3, 2, call, layers=[kv8(e3, block=8)])
        refused(e3, 2, call, layers=[kv8(e3, block=48, page=48)])
        refused(e3, 2, call, layers=[kv8(e3, page=32)])          # pages of half a block
        refused(e3, 2, call, layers=[kv8(e3, page=96)])
        refused(e3, 2, call, layers=[kv8(e3, n=0)])
        refused(e3, 1, call, layers=[kv8(e3, k=A + 8)])
        refused(e3, 1, call, layers=[kv8(e3, ke=None)])
        refused(e3, 1, call, layers=[kv8(e3, flags=2)])
        refused(e3, 3, call, **{other: [kv16(e3, dt=e3.E3_F32)]})
        refused(e3, 2, call, **{other: [kv16(e3, hd=64)]})
        refused(e3, 2, call, **{other: [kv16(e3, KVH=4)]})
        refused(e3, 2, call, layers=[kv8(e3), kv8(e3, page=128)], **{other: [kv16(e3)] * 2})
        refused(e3, 2, call, layers=[kv8(e3), kv8(e3, block=32)], **{other: [kv16(e3)] * 2})
        refused(e3, 2, call, layers=[kv8(e3)] * 129, **{other: [kv16(e3)] * 129})
        with pytest.raises(ValueError):
            call(layers=[kv8(e3)] * 2)
        with pytest.raises(TypeError):
            call(layers=[kv4(e3)])                                # (a descriptor of the same size)
        with pytest.raises(TypeError):
            call(layers=[kv8(e3)], **{other: [kv8(e3)]})
    with pytest.raises(TypeError):
        e3.kv4_append([kv8(e3)], [kv16(e3)], 1, 1, None, A, 0, A, None, None, stream=0)
    refused(e3, 2, append, add=2)
    refused(e3, 2, append, add=-1)
    refused(e3, 1, append, kv_len=None)


def test_verify8_refusals(e3):  # noqa: F811
    def call(Q=A, kv=None, tail=None, B=1, R=61, H=32, P=2048, scale=0.1, ws=A, n=1 << 40, stream=0):
        e3.tree_verify_attn8(Q, kv or kv8(e3), tail or kv16(e3), A, A, B, R, H, P, scale, A, A, None, ws, n, stream=stream)
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
    refused(e3, 2, call, kv=kv8(e3, hd=32))
    assert e3.eagle3_verify8_workspace_bytes(0, 1, 1, 1, 128, 0) == 0
    assert e3.eagle3_verify8_workspace_bytes(1, 1, 3, 2, 128, 0) == 0
    assert e3.eagle3_verify8_workspace_bytes(1, 61, 32, 8, 128, 2048) > 0


def test_plain_codes_are_e4m3():
    """encode / decode against torch's e4m3 type; needed() at its borders."""
    x = np.concatenate([np.random.default_rng(0).normal(size=4000) * np.exp2(np.random.default_rng(1).integers(-12, 9, 4000)),
                        np.arange(-464, 465) / 2.0, np.arange(-64, 65) * 2.0 ** -11])
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn)
    got = kv8_ref.encode(x.astype(np.float32).astype(np.float64), 0)
    assert np.array_equal(kv8_ref.decode(got, 0), want.double().numpy())
    assert kv8_ref.needed(448.0) == 0 and kv8_ref.needed(449.0) == 1 and kv8_ref.needed(224.0) == -1
    assert kv8_ref.needed(0.0) == -100 and kv8_ref.needed(kv8_ref.TOP) == 120


def test_plain_rows_follow_a_growing_scale():
    """Rows appended one by one, each twice as large, end as rows appended at once, but for subnormal codes."""
    rng = np.random.default_rng(3)
    x = rng.integers(-15, 16, (20, 4)) * np.exp2(np.arange(20))[:, None] * 2.0 ** -6
    one, all_ = np.zeros((32, 4), np.uint8), np.zeros((32, 4), np.uint8)
    e1, e2 = np.zeros(2, np.int8), np.zeros(2, np.int8)
    for i in range(20):
        kv8_ref.append(one, e1, i, x[i:i + 1], 16)
    kv8_ref.append(all_, e2, 0, x, 16)
    assert np.array_equal(e1, e2)
    a, b = (kv8_ref.decode(c[:16], e[0]) for c, e in ((one, e1), (all_, e2)))
    assert np.all(np.abs(a - b) <= 2.0 ** (-10 + float(e1[0])) * 2)  # two roundings to a subnormal step
