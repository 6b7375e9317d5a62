"""GPU parity of prompt_attn at the edges of its inputs: scores of -Inf, long sums.

Tolerances as in test_gpu_prompt, with what a test adds to them derived beside it.
"""
import math

import numpy as np
import pytest
import torch

from eagle_speculative_decoding_round_gb300 import synth
from gpu_util import host

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from eagle_speculative_decoding_round_gb300 import eagle3 as e3
    from test_gpu_prompt import call, check, inputs


def check_inf(d, O, lse):
    """As check() of test_gpu_prompt, with keys whose score is -Inf: they weigh 0, and a row that has no others gets 0 and -Inf."""
    O, lse = host(O).astype(np.float64), host(lse).astype(np.float64)
    G, page, scale = d["H"] // d["KVH"], d["page"], 1 / math.sqrt(d["hd"])
    w_err, half = (2.0 ** -8, 2.0 ** -8) if d["dt"] == "bf16" else (2.0 ** -20, 2.0 ** -24)
    for b in range(d["B"]):
        n, c = d["rows"][b], d["ctx"][b]
        t, r = np.arange(c + n), np.arange(n)
        k, v = (x[d["pt"][b, t // page], :, t % page].astype(np.float64) for x in (d["k"], d["v"]))
        at = d["start"][b] + r
        for h in range(d["H"]):
            q, kh, vh = d["Q"][at, h].astype(np.float64), k[:, h // G], v[:, h // G]
            kh0 = np.where(np.isinf(kh), 0.0, kh)
            seen = (t[None] <= c + r[:, None]) & ~np.isinf(kh).any(1)[None]
            s = np.where(seen, q @ kh0.T * scale, -np.inf)
            big = np.where(seen, np.abs(q) @ np.abs(kh0).T * scale, 0.0).max(1)
            none = ~seen.any(1)
            m = np.where(none, 0.0, s.max(1))[:, None]
            p = np.exp(s - m)
            z = p.sum(1, keepdims=True) + none[:, None]
            o, mag, l = p @ vh / z, p @ np.abs(vh) / z, (m + np.log(z))[:, 0]
            assert np.all(O[at[none], h] == 0) and np.all(np.isneginf(lse[at[none], h])), (b, h)
            some = ~none
            ds = 2.0 ** -18 * (big + 1.0)
            assert np.all((np.abs(lse[at, h] - l) <= ds + 2.0 ** -21 * np.abs(l))[some]), (b, h)
            e = (w_err + 2 * ds[:, None]) * mag
            bad = np.abs(O[at, h] - o) - (e + half * (np.abs(o) + e) + 2.0 ** -126)
            assert np.all(bad[some] <= 0), (b, h, bad[some].max())


def inf_keys(d, where):
    """Q positive in dim 0, K there -Inf for the keys that where(t, request) names: their scores are -Inf."""
    d["Q"][..., 0] = np.abs(d["Q"][..., 0]) + 0.5
    if d["dt"] == "bf16":
        d["Q"] = synth.to_bf16_f32(d["Q"])  # what the device holds
    for b in range(d["B"]):
        t = np.arange(d["rows"][b] + d["ctx"][b])
        gone = t[where(t, b)]
        d["k"][d["pt"][b, gone // d["page"]], :, gone % d["page"], 0] = -np.inf
    return d


WHERE = {"first 64": lambda t, b: t < 64, "first 130": lambda t, b: t < 130, "a stretch": lambda t, b: (t >= 40) & (t < 300),
         "all but one": lambda t, b: t != 200, "all": lambda t, b: t >= 0}


@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("H,KVH,hd,rows,ctx", [(4, 2, 64, [300, 5], [0, 250]), (32, 32, 128, [150], [100]), (2, 1, 96, [20], [220])])
def test_prompt_attn_fp32_scores_of_minus_inf(H, KVH, hd, rows, ctx, where):
    """Tiles of 16 and of 64 rows; rows with no other score in their first tiles, in later ones, in all."""
    d = inf_keys(inputs(H + hd, H, KVH, hd, rows, ctx, 16, "f32"), WHERE[where])
    O, lse, err = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check_inf(d, O, lse)


@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("H,KVH,hd,rows,ctx", [
    (4, 2, 64, [300, 5], [0, 250]), (8, 2, 128, [400], [100]), (5, 1, 128, [103, 300], [77, 0]),
    (8, 2, 128, [9, 130], [4000, 2500]), (16, 1, 64, [1], [20000])])  # (the last two are cut along their keys)
def test_prompt_attn_bf16_scores_of_minus_inf(H, KVH, hd, rows, ctx, where):
    """Rows with no other score in their first steps, in whole parts of a cut item, in all."""
    d = inf_keys(inputs(H + hd, H, KVH, hd, rows, ctx, 16), WHERE[where])
    O, lse, err = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check_inf(d, O, lse)


@pytest.mark.parametrize("dt,ctx", [("bf16", 130), ("bf16", 4000), ("f32", 130)])
def test_prompt_attn_bad_values_beside_scores_of_minus_inf(dt, ctx):
    """V with a NaN where the score is -Inf: the rows that see it get NaN (0 times NaN), whichever part holds it."""
    d = inf_keys(inputs(ctx, 8, 2, 64, [20], [ctx], 16, dt), WHERE["first 130"])
    d["v"][d["pt"][0, 7 // 16], :, 7 % 16, 3] = np.nan
    O, lse, err = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert np.isnan(host(O)[d["start"][0]:d["start"][0] + 20][..., 3]).all() and not np.isnan(host(lse)).any()


def long_inputs(seed, H, KVH, hd, rows, ctx, dt, page=64, n=5, zeros=True):
    """Contexts of any length over n pages that the tables name again and again; V of one sign, so that nothing of what a
    sum loses is lost in cancellation; rows of zeros in Q (equal weights), or ordinary ones."""
    rng = np.random.default_rng(seed)
    d = inputs(seed, H, KVH, hd, rows, [0] * len(rows), page, dt)
    rnd = (lambda a: synth.to_bf16_f32(a.astype(np.float32))) if dt == "bf16" else (lambda a: a.astype(np.float32))
    most = max(r + c for r, c in zip(rows, ctx))
    d.update(ctx=list(ctx), n=n, pt=np.stack([(np.arange(-(-most // page)) + b) % n for b in range(len(rows))]).astype(np.int32),
             k=rnd(rng.normal(size=(n, KVH, page, hd))), v=rnd(rng.uniform(0.5, 1.0, (n, KVH, page, hd))))
    if zeros:
        d["Q"][:] = 0.0
    return d


def check_long(d, O, lse, adds, heads=None, exact=False):
    """64-bit softmax over the pages' slots, each counted as often as a row sees it.  `adds(keys)` bounds the error of a sum of
    one sign, relative: it is added to the tolerance of test_gpu_prompt, once for the values' sum and once for the weights'.
    exact: the weights are 1, which no rounding changes."""
    O, lse = host(O).astype(np.float64), host(lse).astype(np.float64)
    G, page, scale = d["H"] // d["KVH"], d["page"], 1 / math.sqrt(d["hd"])
    w_err, half = (2.0 ** -8, 2.0 ** -8) if d["dt"] == "bf16" else (2.0 ** -20, 2.0 ** -24)
    if exact:
        w_err = 0.0
    worst = 0.0
    for b in range(d["B"]):
        for r in range(d["rows"][b]):
            keys = d["ctx"][b] + r + 1
            full, rest = divmod(keys, page)
            count = np.bincount(d["pt"][b, :full], minlength=d["n"])[:, None] * np.ones(page)
            if rest:
                count[d["pt"][b, full], :rest] += 1
            at, count = d["start"][b] + r, count.ravel()
            for h in range(d["H"]) if heads is None else heads:
                k, v = (x[:, h // G].reshape(-1, d["hd"]).astype(np.float64) for x in (d["k"], d["v"]))
                q = d["Q"][at, h].astype(np.float64)
                s, big = k @ q * scale, (np.abs(k) @ np.abs(q) * scale).max()
                m = s[count > 0].max()
                p = count * np.exp(s - m)
                z = p.sum()
                o, l = p @ v / z, m + np.log(z)
                ds, lost = 2.0 ** -18 * (big + 1.0), adds(keys)
                assert abs(lse[at, h] - l) <= ds + lost + 2.0 ** -21 * abs(l), (b, r, h, lse[at, h] - l)
                e = (w_err + 2 * ds + 2 * lost) * o
                bad = np.abs(O[at, h] - o) - (e + half * (o + e))
                worst = max(worst, (np.abs(O[at, h] - o) / o).max())
                assert np.all(bad <= 0), (b, r, h, worst, lost)
    return worst


def adds_fp32(keys):
    """64 keys of a tile one after another, then up to 2.5 sqrt(tiles) partial sums in two levels (64 or more in the first): 2^-24 each."""
    tiles = -(-keys // 64)
    span = max(64, 2 ** (((tiles - 1).bit_length() + 1) // 2))
    return (64 + min(tiles, span) + tiles // span) * 2.0 ** -24


@pytest.mark.parametrize("H,KVH,hd,rows,ctx,zeros", [
    (4, 2, 64, [3], [20000], True), (4, 2, 64, [3], [20000], False), (2, 2, 128, [1], [1 << 20], True), (2, 1, 256, [2, 1], [70001, 4095], False),
    (160, 160, 32, [2], [40000], True), (160, 160, 128, [1], [30000], False), (2, 1, 96, [1], [131072], True), (80, 80, 192, [70], [4200], True),
    (160, 160, 64, [1], [12345], True), (160, 160, 160, [1], [8200], False), (160, 160, 224, [1], [9000], True), (160, 160, 256, [1], [9000], True)])
def test_prompt_attn_fp32_long_sums(H, KVH, hd, rows, ctx, zeros):
    """Tens of thousands of keys of one sign, tiles of 16 and of 64 rows: the sums do not lose what is added late."""
    d = long_inputs(H + hd, H, KVH, hd, rows, ctx, "f32", zeros=zeros)
    O, lse, err = call(d)
    O2, lse2, _ = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(O, O2) and torch.equal(lse, lse2)
    check_long(d, O, lse, adds_fp32, heads=None if H < 10 else (0, 7, H - 1))


def adds_bf16(keys):
    """The tensor core sums 32768 keys at most, 16 a product, and cuts the sum off with each of up to four additions of a
    product, by one unit 2^-23 at most; then fp32 sums of these and of the steps' weights."""
    steps = -(-keys // 64)
    return (min(steps, 512) * 16 + min(steps, 512) // 2 + steps // 512) * 2.0 ** -23 if steps else 0.0


@pytest.mark.parametrize("H,KVH,hd,rows,ctx,zeros", [
    (152, 152, 128, [1], [1 << 20], True),             # whole items in a call that is cut
    (152, 152, 64, [3], [1 << 22], True),
    (152, 152, 128, [300], [33000], False),            # two waves, diagonals behind what has left tensor memory
    (2433, 2433, 64, [1], [40000], True),              # a call that is not cut
    (2433, 2433, 64, [1], [70000], False),
    (8, 1, 128, [5], [152 * 40000], True),             # one item in 152 parts, each longer than 32768 keys
    (8, 2, 128, [5, 40], [152 * 30000, 90001], False),
    (16, 2, 64, [1, 1], [40000, 20000], False)])
def test_prompt_attn_bf16_long_sums(H, KVH, hd, rows, ctx, zeros):
    """Contexts of tens of thousands to millions of keys, V of one sign."""
    d = long_inputs(H + hd, H, KVH, hd, rows, ctx, "bf16", zeros=zeros)
    O, lse, err = call(d)
    O2, lse2, _ = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(O, O2) and torch.equal(lse, lse2)
    if max(rows) > 50:  # (a sample of the rows)
        d = dict(d, start=d["start"] + rows[0] - 5, ctx=[ctx[0] + rows[0] - 5], rows=[5], B=1)
    check_long(d, O, lse, adds_bf16, heads=None if H < 10 else (0, 7, H - 1), exact=zeros)


@pytest.mark.parametrize("H,KVH,hd,ctx", [(152, 152, 64, 70000), (2433, 2433, 64, 40000), (4, 1, 128, 152 * 33000)])
def test_prompt_attn_bf16_long_sums_keep_what_they_have_met(H, KVH, hd, ctx):
    """A NaN in V of an early key reaches o behind the folded sums; late maxima move the base over them."""
    d = long_inputs(H, H, KVH, hd, [2], [ctx], "bf16", n=8)
    d["Q"][:] = 1.0
    d["pt"][0] = np.minimum(np.arange(d["pt"].shape[1]) * 8 // d["pt"].shape[1], 7)  # the pages one after another, repeated
    d["k"] = synth.to_bf16_f32((np.linspace(-1.0, 1.0, 8)[:, None, None, None] + 0.05 * d["k"]).astype(np.float32))
    O, lse, err = call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check_long(d, O, lse, adds_bf16, heads=None if H < 10 else (0, 7, H - 1))
    d["v"][0, :, 5, 3] = np.nan
    O2, lse2, _ = call(d)
    torch.cuda.synchronize()
    o = host(O2)
    assert np.isnan(o[..., 3]).all() and torch.equal(lse, lse2)
    assert np.array_equal(np.delete(o, 3, -1), np.delete(host(O), 3, -1))


def test_prompt_attn_bounds_of_long_contexts_over_short_ones():
    """A bound above 32768 keys takes the kernel for long items: on short requests (one call cut along its keys, one not) it answers the
    same, in a graph too, whose replay meets a long context; a wait that runs out in it ends the call."""
    for H, KVH, rows, ctx in ((16, 4, [70, 0, 3, 300], [10, 0, 2000, 0]), (8, 8, [20] * 320, [5] * 320)):
        d = inputs(H, H, KVH, 64, rows, ctx, 16, gap=1)
        dev = {}
        O, lse, err = call(d, dev=dev)
        O2, lse2, err2 = call(d, dev=dev, max_ctx=40000)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and int(err2.item()) == 0
        check(d, O2, lse2)
    _, _, err = call(d, dev=dev, max_ctx=40000, flags=e3.E3_KV_SELFTEST_STALL)
    torch.cuda.synchronize()
    assert int(err.item()) == e3.E3_DEV_ERR_TIMEOUT
    d = long_inputs(5, 152, 152, 64, [2], [40000], "bf16", zeros=False)
    dev = {}
    O, lse, err = call(d, dev=dev)
    need = e3.eagle3_prompt_workspace_bytes(1, d["total"], 2, 152, 152, 64, 40000, e3.E3_BF16)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = (torch.full_like(O, 55.0), torch.full_like(lse, 55.0))
    dev["ctx"].fill_(100)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(d, dev=dev, ws=ws, out=out, err=err)
    for ctx in (100, 40000, 32766, 32768, 700):
        dev["ctx"].fill_(ctx)
        g.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        check_long(dict(d, ctx=[ctx]), *out, adds_bf16, heads=(0, 151))
        if ctx == 40000:
            assert torch.equal(out[0], O) and torch.equal(out[1], lse)


def test_prompt_attn_long_sums_on_two_streams():
    """Two long calls at once, each with scratch of its own; fp32 beside them."""
    a = long_inputs(6, 152, 152, 64, [1], [70000], "bf16", zeros=False)
    b = long_inputs(7, 4, 2, 128, [2], [20000], "f32", zeros=False)
    da, db = {}, {}
    call(a, dev=da)
    call(b, dev=db)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    for _ in range(2):
        for s, d, dev in zip(streams, (a, a, b), (da, da, db)):
            with torch.cuda.stream(s):
                outs.append((d, call(d, dev=dev, stream=s)))
    torch.cuda.synchronize()
    for d, (O, lse, err) in outs:
        assert int(err.item()) == 0
        check_long(d, O, lse, adds_bf16 if d is a else adds_fp32, heads=(0, d["H"] - 1))
