"""CPU checks: arrays off their elements' grid are refused before any launch (on the device they would fault)."""
import pytest

from test_kv4_host import A, e3, kv4, kv16, refused  # noqa: F401 (e3 is a fixture)
from test_kv8_host import kv8


def off(e3, make, *args, page_table=A + 2, **kw):  # noqa: F811
    d = make(e3, *args, **kw)
    d.page_table = page_table
    return d


def prompt(e3, start=A, rows=A, kv=None, kv_len=A, lse=A, err=A, stream=0):  # noqa: F811
    e3.prompt_attn(A, start, rows, kv or kv16(e3), kv_len, 2, 100, 64, 32, 512, 0.1, A, lse, err, A, 1 << 40, stream=stream)


def attn(name, make):
    def call(e3, kv=None, tail=None, lens=A, mask=A, lse=A, err=A, stream=0):  # noqa: F811
        getattr(e3, name)(A, kv or make(e3), tail or kv16(e3), lens, mask, 1, 61, 32, 2048, 0.1, A, lse, err, A, 1 << 40, stream=stream)
    return call


def append(name, make):
    def call(e3, kv=None, src=None, rows=A, n=A, lens=A, nxt=A, err=A, stream=0):  # noqa: F811
        getattr(e3, name)([kv or make(e3)], [src or kv16(e3)], 2, 7, rows, n, 0, lens, nxt, err, stream=stream)
    return call


def read(name, make):
    def call(e3, kv=None, dst=None, first=A, n=A, err=A, stream=0):  # noqa: F811
        getattr(e3, name)([kv or make(e3)], [dst or kv16(e3)], 2, 7, first, n, err, stream=stream)
    return call


def qkv(e3, n=A, qn=A, kn=A, pos=A, kv=None, lens=A, err=A, stream=0):  # noqa: F811
    e3.tree_qkv_append(A, 6144, 1, 61, n, 32, qn, kn, 1e-5, e3.eagle3_rope_init(128, 10000.0), pos, A, kv or kv16(e3), lens, err, stream=stream)


# call, its arrays of 32-bit and of 64-bit elements, its descriptors
CALLS = {
    "tree_qkv_append": (qkv, ("n", "qn", "kn", "pos", "lens", "err"), (), {"kv": kv16}),
    "prompt_attn": (prompt, ("start", "rows", "kv_len", "lse", "err"), (), {"kv": kv16}),
    "tree_verify_attn8": (attn("tree_verify_attn8", kv8), ("lens", "lse", "err"), ("mask",), {"kv": kv8, "tail": kv16}),
    "tree_verify_attn4": (attn("tree_verify_attn4", kv4), ("lens", "lse", "err"), ("mask",), {"kv": kv4, "tail": kv16}),
    "kv8_append": (append("kv8_append", kv8), ("rows", "n", "lens", "nxt", "err"), (), {"kv": kv8, "src": kv16}),
    "kv4_append": (append("kv4_append", kv4), ("rows", "n", "lens", "nxt", "err"), (), {"kv": kv4, "src": kv16}),
    "kv8_read": (read("kv8_read", kv8), ("first", "n", "err"), (), {"kv": kv8, "dst": kv16}),
    "kv4_read": (read("kv4_read", kv4), ("first", "n", "err"), (), {"kv": kv4, "dst": kv16}),
}


@pytest.mark.parametrize("name", CALLS)
def test_arrays_off_their_grid_are_refused(e3, name):  # noqa: F811
    call, words, longs, descriptors = CALLS[name]
    for arg in words + longs:
        for by in (1, 2, 3) + ((4, 6) if arg in longs else ()):
            refused(e3, 1, lambda stream, **kw: call(e3, stream=stream, **kw), **{arg: A + by})
    for arg, make in descriptors.items():
        for by in (1, 2, 3):
            refused(e3, 1, lambda stream, **kw: call(e3, stream=stream, **kw), **{arg: off(e3, make, page_table=A + by)})
