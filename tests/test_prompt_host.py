"""CPU checks of prompt_attn: refusals before any launch."""
import pytest  # noqa: F401

from test_kv4_host import A, e3, kv16, refused  # noqa: F401 (e3 is a fixture)


def test_prompt_refusals(e3):  # noqa: F811
    def call(Q=A, start=A, rows=A, kv=None, kv_len=A, B=2, total=100, most=64, H=32, P=512, scale=0.1, O=A, lse=A, ws=A, n=1 << 40,  # noqa: E741
             stream=0):
        e3.prompt_attn(Q, start, rows, kv or kv16(e3), kv_len, B, total, most, H, P, scale, O, lse, None, ws, n, stream=stream)
    refused(e3, 1, call, Q=None)
    refused(e3, 1, call, O=None)
    refused(e3, 1, call, lse=None)
    refused(e3, 1, call, Q=A + 8)
    refused(e3, 1, call, O=A + 8)
    refused(e3, 1, call, lse=A + 2)
    refused(e3, 1, call, ws=A + 4)
    refused(e3, 2, call, B=0)
    refused(e3, 2, call, B=65536)
    refused(e3, 2, call, total=0)
    refused(e3, 2, call, most=0)
    refused(e3, 2, call, start=None)                    # 2 * 64 rows in 100
    refused(e3, 2, call, total=1 << 26)                 # 2^31 rows of heads
    refused(e3, 2, call, P=-1)
    refused(e3, 2, call, P=1 << 30)
    refused(e3, 2, call, most=1 << 30, P=1)
    refused(e3, 2, call, P=(1 << 25) - 63)              # bf16: 2^25 keys
    refused(e3, 2, call, H=30)                          # not a multiple of the KV heads
    refused(e3, 2, call, H=0)
    refused(e3, 2, call, kv=kv16(e3, hd=96))            # bf16 heads of 96
    refused(e3, 2, call, kv=kv16(e3, page=24))
    refused(e3, 1, call, kv=kv16(e3, flags=2))
    refused(e3, 1, call, kv=kv16(e3, k=A + 4))
    refused(e3, 1, call, kv=kv16(e3, dt=7))
    refused(e3, 1, call, scale=0.0)
    refused(e3, 1, call, scale=float("nan"))
    for bad in ((0, 1, 1, 1, 1, 64, 0), (1, 0, 1, 1, 1, 64, 0), (1, 1, 1, 3, 2, 64, 0), (1, 1, 1, 1, 1, 96, 0), (1, 1, 1, 1, 1, 64, -1)):
        assert e3.eagle3_prompt_workspace_bytes(*bad, e3.E3_BF16) == 0
