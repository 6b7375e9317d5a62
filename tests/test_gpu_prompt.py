"""GPU parity of prompt_attn with a plain 64-bit form.

Tolerances, from the arithmetic: scores are fp32 sums of hd products, off by 2^-18 of the largest sum |q||k| scale (fp32
operands: the same sums); weights are rounded to bf16 at most (2^-8; fp32: 2^-20 with the exponential), and carry twice
the scores' error; the output adds half a step of its type to the value reached.
"""
import math

import numpy as np
import pytest
import torch

from eagle_speculative_decoding_round_gb300 import synth
from gpu_util import host, to_dev

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from eagle_speculative_decoding_round_gb300 import eagle3 as e3
    from test_gpu_kv4 import err_word, i32

TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(seed, H, KVH, hd, rows, ctx, page, dt="bf16", gap=0, spread=1.3, fill=float("nan")):
    """Requests of `rows` rows behind `ctx` cached keys; `gap` rows between them that belong to none; slots that hold
    nothing hold `fill`."""
    rng = np.random.default_rng(seed)
    B = len(rows)
    order = rng.permutation(B)  # the requests' rows lie in no order
    start, at = np.zeros(B, np.int64), gap
    for b in order:
        start[b] = at
        at += rows[b] + gap
    pt, n = synth.page_table(seed, [max(1, r + c) for r, c in zip(rows, ctx)], page)
    rnd = (lambda a: synth.to_bf16_f32(a.astype(np.float32))) if dt == "bf16" else (lambda a: a.astype(np.float32))
    Q = rnd(spread * rng.normal(size=(max(at, 1), H, hd)))
    k, v = (np.full((n, KVH, page, hd), fill, np.float32) for _ in range(2))
    for b in range(B):
        t = np.arange(rows[b] + ctx[b])
        for x in (k, v):
            x[pt[b, t // page], :, t % page] = rnd(rng.normal(size=(len(t), KVH, hd)))
    return dict(B=B, H=H, KVH=KVH, hd=hd, rows=list(rows), ctx=list(ctx), page=page, dt=dt, start=start, total=max(at, 1), pt=pt, n=n,
                Q=Q, k=k, v=v)


def call(d, dev=None, ws=None, out=None, err=None, stream=None, max_rows=None, max_ctx=None, flags=0, n_rows=True, kv_len=True,
         row_start=True):
    dev = {} if dev is None else dev
    if not dev:
        dev.update(Q=to_dev(d["Q"], TD[d["dt"]]), k=to_dev(d["k"], TD[d["dt"]]), v=to_dev(d["v"], TD[d["dt"]]), pt=i32(d["pt"]),
                   start=i32(d["start"]), rows=i32(d["rows"]), ctx=i32(d["ctx"]))
    dt = e3.E3_BF16 if d["dt"] == "bf16" else e3.E3_F32
    kv = e3.make_kv_layer(dev["k"], dev["v"], dev["pt"], d["n"], d["page"], d["pt"].shape[1], d["KVH"], d["hd"], dt, flags)
    mr = max(1, max(d["rows"])) if max_rows is None else max_rows
    mc = max(d["ctx"]) if max_ctx is None else max_ctx
    need = e3.eagle3_prompt_workspace_bytes(d["B"], d["total"], mr, d["H"], d["KVH"], d["hd"], mc, dt)
    if ws is None:
        ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    O, lse = out or (torch.full((d["total"], d["H"], d["hd"]), 55.0, dtype=TD[d["dt"]], device="cuda"),
                     torch.full((d["total"], d["H"]), 55.0, device="cuda"))
    err = err_word() if err is None else err
    e3.prompt_attn(dev["Q"], dev["start"] if row_start else None, dev["rows"] if n_rows else None, kv, dev["ctx"] if kv_len else None,
                   d["B"], d["total"], mr, d["H"], mc, 1 / math.sqrt(d["hd"]), O, lse, err, ws, need, stream=stream)
    return O, lse, err


def check(d, O, lse, requests=None, rows_of=None):
    """Every row of the requests (or those that rows_of(n) names), and the rows of none, left as they were."""
    O, lse = host(O).astype(np.float64), host(lse).astype(np.float64)
    G, page, scale = d["H"] // d["KVH"], d["page"], 1 / math.sqrt(d["hd"])
    none = np.ones(d["total"], bool)
    for b in range(d["B"]):
        none[d["start"][b]:d["start"][b] + d["rows"][b]] = False
    if requests is None:
        assert np.all(O[none] == 55.0) and np.all(lse[none] == 55.0)
    w_err, half = (2.0 ** -8, 2.0 ** -8) if d["dt"] == "bf16" else (2.0 ** -20, 2.0 ** -24)
    for b in requests if requests is not None else range(d["B"]):
        n, c = d["rows"][b], d["ctx"][b]
        if n == 0:
            continue
        t = np.arange(c + n)
        k, v = (x[d["pt"][b, t // page], :, t % page].astype(np.float64) for x in (d["k"], d["v"]))
        r = np.arange(n) if rows_of is None else rows_of(n)
        at = d["start"][b] + r
        seen = t[None] <= c + r[:, None]
        for h in range(d["H"]):
            q, kh, vh = d["Q"][at, h].astype(np.float64), k[:, h // G], v[:, h // G]
            s = np.where(seen, q @ kh.T * scale, -np.inf)
            big = np.where(seen, np.abs(q) @ np.abs(kh).T * scale, 0.0).max(1)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            z = p.sum(1, keepdims=True)
            o, mag, l = p @ vh / z, p @ np.abs(vh) / z, (m + np.log(z))[:, 0]
            ds = 2.0 ** -18 * (big + 1.0)
            assert np.all(np.abs(lse[at, h] - l) <= ds + 2.0 ** -21 * np.abs(l)), (b, h, np.abs(lse[at, h] - l).max())
            e = (w_err + 2 * ds[:, None]) * mag
            bad = np.abs(O[at, h] - o) - (e + half * (np.abs(o) + e) + 2.0 ** -126)
            assert np.all(bad <= 0), (b, h, bad.max(), np.argwhere(bad > 0)[:3])


CASES = [
    # H, KVH, hd, rows, ctx, page, dt, gap
    (4, 4, 64, [1], [0], 16, "bf16", 0),
    (32, 8, 128, [1], [0], 64, "bf16", 1),
    (32, 8, 128, [300], [0], 64, "bf16", 0),
    (4, 4, 64, [1, 2, 0, 127, 128, 129, 257], [0] * 7, 16, "bf16", 2),
    (8, 2, 128, [31, 32, 33, 64, 65], [0, 1, 127, 128, 300], 64, "bf16", 0),
    (2, 2, 128, [255, 256, 513], [0, 1, 130], 128, "bf16", 3),          # a row tile is 256 rows of one head
    (6, 2, 64, [85, 86, 171], [0, 3, 64], 32, "bf16", 0),               # three heads: tiles end inside a row
    (5, 1, 128, [103, 52], [77, 0], 48, "bf16", 1),                     # pages that are no power of two
    (48, 1, 64, [9, 70], [500, 0], 16, "bf16", 0),
    (300, 1, 64, [3], [40], 16, "bf16", 0),                             # more heads than a tile has rows
    (64, 8, 128, [40, 3, 1], [2000, 1111, 4096], 64, "bf16", 0),        # few rows behind long contexts
    (16, 2, 128, [1, 1, 1], [640, 0, 127], 256, "bf16", 0),             # single tokens
    (8, 8, 128, [700], [0], 16, "bf16", 0),
    (8, 1, 128, [1000], [1000], 64, "bf16", 0),
    (4, 4, 64, [15, 131, 1], [128, 0, 3], 16, "f32", 1),
    (3, 1, 32, [70], [10], 16, "f32", 0),
    (4, 2, 128, [65, 64], [0, 63], 64, "f32", 0),
    (2, 1, 96, [33], [0], 48, "f32", 0),
    (2, 2, 256, [40, 5], [9, 200], 16, "f32", 0),
    (2, 1, 160, [20], [0], 16, "f32", 0),
    (2, 1, 192, [20], [70], 16, "f32", 0),
    (1, 1, 224, [66], [0], 32, "f32", 0),
]


@pytest.mark.parametrize("case", CASES)
def test_prompt_attn(case):
    H, KVH, hd, rows, ctx, page, dt, gap = case
    d = inputs(H + hd + sum(rows), H, KVH, hd, rows, ctx, page, dt, gap)
    O, lse, err = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(d, O, lse)


@pytest.mark.parametrize("H,KVH,hd,rows,ctx", [(32, 8, 128, [4000, 700], [0, 0]), (64, 8, 128, [257], [20000]), (4, 4, 64, [3000], [100])])
def test_prompt_attn_long(H, KVH, hd, rows, ctx):
    """Many key tiles; a sample of the rows is compared."""
    d = inputs(7 + H, H, KVH, hd, rows, ctx, 64)
    O, lse, err = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and not torch.any(lse == 55.0)
    check(d, O, lse, rows_of=lambda n: np.unique(np.concatenate([np.arange(0, n, 97), [n - 1, n // 2, min(n - 1, 255), min(n - 1, 256)]])))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_prompt_attn_sharp_rows(dt):
    """Scores that move the softmax base far, late maxima, rows of zeros, rows whose weight lies on one key."""
    d = inputs(5, 8, 2, 64, [400, 100], [0, 300], 64, dt)
    rng = np.random.default_rng(2)
    d["Q"] *= np.exp2(rng.integers(-12, 5, d["Q"].shape[:2]))[..., None].astype(np.float32)
    d["Q"][d["start"][0] + 5] = 0.0
    t = np.arange(400)
    late = d["k"][d["pt"][0, t // 64], :, t % 64] * np.linspace(0.1, 6.0, 400)[:, None, None]
    d["k"][d["pt"][0, t // 64], :, t % 64] = synth.to_bf16_f32(late.astype(np.float32))
    O, lse, err = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(d, O, lse)


@pytest.mark.parametrize("H,KVH,hd,dt", [(8, 2, 128, "bf16"), (4, 4, 64, "bf16"), (2, 1, 64, "f32")])
def test_prompt_attn_unseen_keys_have_no_effect(H, KVH, hd, dt):
    """A NaN or an Inf in K or V behind a row's position: the row stays exact; rows that see it get NaN or Inf."""
    for n, c, bad, which, x in ((200, 50, 170, "v", np.nan), (200, 0, 131, "v", np.inf), (300, 3, 190, "k", np.nan), (40, 0, 39, "v", -np.inf),
                                (130, 128, 256, "v", np.nan)):
        d = inputs(n + c, H, KVH, hd, [n], [c], 16, dt)
        clean = dict(d, k=d["k"].copy(), v=d["v"].copy())
        d[which][d["pt"][0, bad // 16], :, bad % 16, 3] = x
        O, lse, err = call(d)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        below = np.arange(0, bad - c)
        check(clean, O, lse, requests=[0], rows_of=lambda n: below)
        o = host(O)[d["start"][0] + np.arange(bad - c, n)]
        assert not np.isfinite(o[..., 3]).any(), (n, c, bad)


def test_prompt_attn_optional_arguments():
    """Without row_start, n_rows, kv_len: padded requests of max_rows rows without a context; looser bounds; the
    prefix promise; the same bits again on dirty scratch."""
    d = inputs(3, 16, 4, 128, [90, 90, 90], [0, 0, 0], 64)
    d["start"] = np.arange(3) * 90
    dev = {}
    O, lse, err = call(d, dev=dev)
    O2, lse2, _ = call(d, dev=dev, err=err, n_rows=False, kv_len=False, row_start=False)
    O3, lse3, _ = call(d, dev=dev, err=err, flags=e3.E3_KV_PREFIX_STABLE)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(d, O, lse)
    assert torch.equal(O, O2) and torch.equal(lse, lse2) and torch.equal(O, O3) and torch.equal(lse, lse3)
    O4, lse4, _ = call(d, dev=dev, err=err, max_rows=1000, max_ctx=5000)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(d, O4, lse4)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_prompt_attn_bad_requests_are_flagged(dt):
    """Rows or lengths out of bounds: that request's outputs stay, the others are exact; a bad page id is flagged."""
    base = inputs(9, 8, 2, 64, [70, 40, 33], [0, 100, 10], 16, dt, gap=1)
    for what, value in (("rows", 71), ("rows", -1), ("ctx", 101), ("ctx", -5), ("start", -1), ("start", base["total"] - 69), ("ctx", 2 ** 31 - 1)):
        dev = {}
        call(base, dev=dev)
        changed = list(base[what])
        changed[0] = value
        dev[what] = i32(changed)
        O, lse, err = call(base, dev=dev)
        torch.cuda.synchronize()
        assert int(err.item()) == e3.E3_DEV_ERR_CAPACITY, (what, value)
        s = base["start"][0]
        assert torch.all(O[s:s + 70] == 55.0) and torch.all(lse[s:s + 70] == 55.0)
        check(base, O, lse, requests=[1, 2])
    # slots beyond the pages: the table of request 1 ends before its last row
    dev = {}
    call(base, dev=dev)
    short = dict(base, pt=base["pt"][:, :8])
    dev["pt"] = i32(short["pt"])
    O, lse, err = call(short, dev=dev)
    torch.cuda.synchronize()
    assert int(err.item()) == e3.E3_DEV_ERR_CAPACITY
    s = base["start"][1]
    assert torch.all(O[s:s + 40] == 55.0)
    check(base, O, lse, requests=[0, 2])
    for page_id in (base["n"], -1):
        dev["pt"] = i32([base["pt"][0].tolist()[:1] + [page_id] * (base["pt"].shape[1] - 1)] + base["pt"].tolist()[1:])
        O, lse, err = call(base, dev=dev)
        torch.cuda.synchronize()
        assert int(err.item()) == e3.E3_DEV_ERR_CAPACITY
        check(base, O, lse, requests=[1, 2])


def test_prompt_attn_on_streams_and_in_a_graph():
    """Two calls on two streams with scratch of their own; a captured call replayed on changed inputs and lengths."""
    a = inputs(1, 16, 4, 128, [500, 33], [0, 900], 64)
    b = inputs(2, 8, 8, 64, [700, 10], [100, 0], 16)
    da, db = {}, {}
    call(a, dev=da)
    call(b, dev=db)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ra = call(a, dev=da)
        with torch.cuda.stream(s2):
            rb = call(b, dev=db)
    torch.cuda.synchronize()
    check(a, ra[0], ra[1])
    check(b, rb[0], rb[1])
    need = e3.eagle3_prompt_workspace_bytes(2, a["total"], 500, 16, 4, 128, 900, e3.E3_BF16)
    ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    out = (torch.full((a["total"], 16, 128), 55.0, dtype=torch.bfloat16, device="cuda"), torch.full((a["total"], 16), 55.0, device="cuda"))
    err = err_word()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(a, dev=da, ws=ws, out=out, err=err)
    a["rows"], a["ctx"] = [420, 12], [0, 321]
    a["Q"] = synth.to_bf16_f32(a["Q"] * 1.5)
    da["rows"].copy_(i32(a["rows"]))
    da["ctx"].copy_(i32(a["ctx"]))
    da["Q"].copy_(to_dev(a["Q"], torch.bfloat16))
    for t in out:
        t.fill_(55.0)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(a, *out)


def test_prompt_attn_many_requests():
    """More requests than lanes, a third of them empty."""
    rng = np.random.default_rng(4)
    rows = [int(x) for x in np.where(rng.random(75) < 0.3, 0, rng.integers(1, 90, 75))]
    ctx = [int(x) for x in np.where(rng.random(75) < 0.5, 0, rng.integers(1, 200, 75))]
    rows[40] = 600
    d = inputs(4, 8, 2, 128, rows, ctx, 16, gap=1)
    O, lse, err = call(d)
    O2, lse2, _ = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(d, O, lse)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)


def test_prompt_attn_wait_that_runs_out():
    """The self-test bit: keys that never come end the call with the error word set, after the waits' bound, and leave
    nothing behind that the next call on the same buffers meets."""
    d = inputs(6, 16, 4, 128, [700, 300], [0, 200], 64)
    dev = {}
    call(d, dev=dev)
    torch.cuda.synchronize()
    _, _, err = call(d, dev=dev, flags=e3.E3_KV_SELFTEST_STALL)
    torch.cuda.synchronize()
    assert int(err.item()) == e3.E3_DEV_ERR_TIMEOUT
    O, lse, err = call(d, dev=dev)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(d, O, lse)


SPLIT = [
    # H, KVH, hd, rows, ctx, page: few items behind long contexts, which are cut along their keys
    (8, 1, 128, [5], [20000], 16),                                      # one item in many parts
    (64, 8, 128, [100, 152, 204, 257], [3000, 2800, 2500, 2300], 64),   # more items than SMs
    (8, 8, 64, [1] * 5, [4000, 0, 2999, 129, 2500], 16),
    (5, 1, 128, [300, 52], [9000, 100], 48),                            # tiles end inside a row
    (2, 2, 128, [700, 1], [1500, 5000], 128),                           # diagonals in the last parts
    (40, 8, 128, [3, 0, 64], [2176, 5000, 2175], 64),
]


@pytest.mark.parametrize("H,KVH,hd,rows,ctx,page", SPLIT)
def test_prompt_attn_split_along_the_keys(H, KVH, hd, rows, ctx, page):
    d = inputs(11 + H + rows[0], H, KVH, hd, rows, ctx, page, gap=1)
    records = e3.eagle3_prompt_workspace_bytes(d["B"], d["total"], max(rows), H, KVH, hd, max(ctx), e3.E3_BF16)
    assert records > 0
    O, lse, err = call(d)
    O2, lse2, _ = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    check(d, O, lse)


def test_prompt_attn_split_with_many_requests_and_a_loose_bound():
    """More requests than lanes, lengths from none to far apart, the bounds above all of them."""
    rng = np.random.default_rng(14)
    rows = [int(x) for x in np.where(rng.random(45) < 0.3, 0, rng.integers(1, 60, 45))]
    ctx = [int(x) for x in np.where(rng.random(45) < 0.5, 0, rng.integers(1, 3000, 45))]
    ctx[7], rows[7], ctx[33], rows[33] = 6000, 0, 5000, 130
    d = inputs(14, 8, 2, 128, rows, ctx, 16, gap=1)
    assert e3.eagle3_prompt_workspace_bytes(45, d["total"], 200, 8, 2, 128, 9000, e3.E3_BF16) > 0
    O, lse, err = call(d, max_rows=200, max_ctx=9000)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(d, O, lse)


def test_prompt_attn_split_sharp_rows():
    """Parts whose bases differ widely, late maxima, rows of zeros."""
    d = inputs(15, 8, 2, 128, [40, 9], [4000, 2500], 64)
    rng = np.random.default_rng(3)
    d["Q"] *= np.exp2(rng.integers(-12, 5, d["Q"].shape[:2]))[..., None].astype(np.float32)
    d["Q"][d["start"][0] + 5] = 0.0
    t = np.arange(4000)
    late = d["k"][d["pt"][0, t // 64], :, t % 64] * np.linspace(0.1, 6.0, 4000)[:, None, None]
    d["k"][d["pt"][0, t // 64], :, t % 64] = synth.to_bf16_f32(late.astype(np.float32))
    O, lse, err = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(d, O, lse)


@pytest.mark.parametrize("bad,which,x", [(3010, "v", np.nan), (3001, "v", np.inf), (3039, "k", np.nan), (1234, "v", -np.inf)])
def test_prompt_attn_split_unseen_keys_have_no_effect(bad, which, x):
    """As above, with the items cut along their keys: in a part that some of the rows see, and in one that all see."""
    n, c = 50, 3000
    d = inputs(bad, 8, 2, 128, [n], [c], 16)
    clean = dict(d, k=d["k"].copy(), v=d["v"].copy())
    d[which][d["pt"][0, bad // 16], :, bad % 16, 3] = x
    O, lse, err = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    below = np.arange(0, max(0, bad - c))
    if len(below):
        check(clean, O, lse, requests=[0], rows_of=lambda n: below)
    o = host(O)[d["start"][0] + np.arange(max(0, bad - c), n)]
    assert not np.isfinite(o[..., 3]).any()


def test_prompt_attn_split_in_a_graph_and_with_bad_requests():
    """A captured split call replayed on other inputs and lengths; a request out of bounds beside ones that are cut."""
    a = inputs(21, 16, 4, 128, [30, 70], [3000, 1500], 64)
    dev = {}
    O, lse, err = call(a, dev=dev, max_rows=70, max_ctx=3000)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(a, O, lse)
    need = e3.eagle3_prompt_workspace_bytes(2, a["total"], 70, 16, 4, 128, 3000, e3.E3_BF16)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = (torch.full((100, 16, 128), 55.0, dtype=torch.bfloat16, device="cuda"), torch.full((100, 16), 55.0, device="cuda"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(a, dev=dev, ws=ws, out=out, err=err, max_rows=70, max_ctx=3000)
    # the same pages cut elsewhere: 70 rows of the first request behind 2960 keys, 30 of the second behind 1540
    rows = dict(a, rows=[70, 30], start=np.array([30, 0]), ctx=[2960, 1540])
    for key in ("rows", "start", "ctx"):
        dev[key].copy_(i32(rows[key]))
    g.replay()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(rows, *out)
    dev["ctx"].copy_(i32([3001, 1540]))
    out[0].fill_(55.0), out[1].fill_(55.0)
    g.replay()
    torch.cuda.synchronize()
    assert int(err.item()) == e3.E3_DEV_ERR_CAPACITY
    assert torch.all(out[0][30:] == 55.0) and torch.all(out[1][30:] == 55.0)
    check(rows, *out, requests=[1])


def test_prompt_attn_split_wait_that_runs_out():
    d = inputs(23, 16, 4, 128, [40, 30], [3000, 200], 64)
    dev = {}
    call(d, dev=dev)
    torch.cuda.synchronize()
    _, _, err = call(d, dev=dev, flags=e3.E3_KV_SELFTEST_STALL)
    torch.cuda.synchronize()
    assert int(err.item()) == e3.E3_DEV_ERR_TIMEOUT
    O, lse, err = call(d, dev=dev)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(d, O, lse)


@pytest.mark.parametrize("H,KVH,hd,rows,ctx", [
    (8, 8, 64, [1300], [0]), (16, 4, 128, [500, 620], [70, 0]), (160, 160, 32, [5], [9]), (40, 20, 96, [300], [10]), (80, 80, 160, [33, 70], [65, 0]),
    (80, 80, 192, [70], [3]), (160, 160, 224, [17], [64]), (80, 80, 256, [70, 65], [0, 128])])
def test_prompt_attn_fp32_enough_rows_for_every_sm(H, KVH, hd, rows, ctx):
    """Tiles of 64 rows."""
    d = inputs(H + hd, H, KVH, hd, rows, ctx, 16, "f32", gap=1)
    O, lse, err = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(d, O, lse, rows_of=None if hd < 128 else lambda n: np.unique(np.concatenate([np.arange(0, n, 7), [n - 1]])))


def test_prompt_attn_fp32_large_tiles_unseen_keys():
    """A NaN in V behind a row's position, with tiles of 64 rows."""
    n, c, bad = 700, 50, 330
    d = inputs(77, 16, 16, 64, [n], [c], 16, "f32")
    clean = dict(d, k=d["k"].copy(), v=d["v"].copy())
    d["v"][d["pt"][0, bad // 16], :, bad % 16, 3] = np.nan
    O, lse, err = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    below = np.arange(0, bad - c)
    check(clean, O, lse, requests=[0], rows_of=lambda m: below)
    assert not np.isfinite(host(O)[d["start"][0] + np.arange(bad - c, n)][..., 3]).any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_prompt_attn_thousands_of_requests(dt):
    """Short requests, many of them empty, far more than CTAs."""
    rng = np.random.default_rng(9)
    rows = [int(x) for x in rng.integers(0, 4, 3000)]
    ctx = [int(x) for x in np.where(rng.random(3000) < 0.8, 0, rng.integers(1, 40, 3000))]
    rows[1711] = 300
    d = inputs(9, 2, 1, 64, rows, ctx, 16, dt, gap=1)
    O, lse, err = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(d, O, lse)


def test_prompt_attn_split_on_two_streams_over_shared_pages():
    """Two split calls at once, each with scratch of its own; requests whose tables name the same pages."""
    a = inputs(31, 16, 4, 128, [20, 20], [3000, 3000], 64)
    k, v = a["k"], a["v"]
    for x in (k, v):  # both requests' contexts are the first one's pages; their own rows stay apart
        last = x[a["pt"][1, 3000 // 64]].copy()
        last[:, :3000 % 64] = x[a["pt"][0, 3000 // 64], :, :3000 % 64]
        x[a["pt"][1, 3000 // 64]] = last
    a["pt"][1, :3000 // 64] = a["pt"][0, :3000 // 64]
    dev = {}
    call(a, dev=dev)
    torch.cuda.synchronize()
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(call(a, dev=dev, stream=s))
    torch.cuda.synchronize()
    for O, lse, err in outs:
        assert int(err.item()) == 0
        assert torch.equal(O, outs[0][0]) and torch.equal(lse, outs[0][1])
    check(a, *outs[0][:2])


@pytest.mark.parametrize("ctx,dt", [([0, 3], "bf16"), ([5000, 0], "bf16"), ([9, 0], "f32")])
def test_prompt_attn_without_rows(ctx, dt):
    """Every request empty: nothing is written, nothing is flagged."""
    d = inputs(1, 8, 2, 64, [0, 0], ctx, 16, dt)
    O, lse, err = call(d, max_rows=30)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.all(O == 55.0) and torch.all(lse == 55.0)
