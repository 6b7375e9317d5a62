"""GPU parity of the verify pass over an 8-bit cache with plain 64-bit forms (kv8_ref, kv4_ref.attend).

Rows of the cache and their exponents are equal bit for bit.  Attention, from the arithmetic: scores are fp32 sums of
128 products, off by 2^-18 of the largest sum |q||k| scale; weights are rounded to fp16 or bf16, 2^-8 at most, and carry
twice the scores' error; the output adds half a bf16 step of the value reached, 2^-8.  An fp16 weight below 2^-14 is off
by 2^-25 of a unit: with the largest at 2^7 or more, 2^-32 of it, times V in units of the request's largest block scale.
"""
import math

import numpy as np
import pytest
import torch

import kv4_ref
import kv8_ref
from eagle_speculative_decoding_round_gb300 import synth
from gpu_util import host, random_tree, to_dev

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from eagle_speculative_decoding_round_gb300 import eagle3 as e3
    from test_gpu_kv4 import ancestors, err_word, i32, mask_of


# ------------------------------------------------------------ rows of the cache

def kv8_buffers(L, n, KVH, page, hd, block, fill=0):
    codes = [torch.full((L, n, KVH, page, hd), fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
    exps = [torch.full((L, n, KVH, page // block), -77, dtype=torch.int8, device="cuda") for _ in range(2)]
    return codes + exps


def kv8_layers(bufs, pt, page, KVH, hd, block):
    return [e3.make_kv8_layer(*[b[l] for b in bufs], pt, bufs[0].shape[1], page, pt.shape[1], KVH, hd, block)
            for l in range(bufs[0].shape[0])]


def bf16_layers(bufs, pt, page, KVH, hd):
    return [e3.make_kv_layer(bufs[0][l], bufs[1][l], pt, bufs[0].shape[1], page, pt.shape[1], KVH, hd, e3.E3_BF16)
            for l in range(bufs[0].shape[0])]


@pytest.mark.parametrize("B,R,L,KVH,hd,page,block,path,in_place", [
    (1, 1, 1, 1, 64, 16, 16, False, False), (3, 7, 3, 8, 128, 64, 64, True, True), (2, 7, 2, 2, 64, 32, 16, True, False),
    (2, 9, 33, 1, 128, 128, 128, True, False), (2, 501, 2, 3, 128, 48, 16, False, True), (1, 1030, 1, 8, 128, 128, 128, False, False),
    (3, 130, 2, 2, 64, 128, 128, False, False), (2, 77, 2, 2, 128, 64, 32, False, True), (4, 64, 1, 5, 64, 64, 64, False, False)])
def test_kv8_append_and_read(B, R, L, KVH, hd, page, block, path, in_place):
    """Three appends in a row (blocks are filled in parts, scales grow and do not shrink), read back whole."""
    seed = B * 100 + R + hd
    rng = np.random.default_rng(seed)
    spt, sn = synth.page_table(seed + 1, [max(R, 40)] * B, 16)
    lens = [int(v) for v in rng.integers(0, 50, B)]
    lens[0] = 0
    pt, n = synth.page_table(seed, [p + 3 * R for p in lens], page)
    bufs = kv8_buffers(L, n, KVH, page, hd, block, fill=0x31)
    dpt, dspt, dlen, err = i32(pt), i32(spt), i32(lens), err_word()
    layers = kv8_layers(bufs, dpt, page, KVH, hd, block)
    # a row of positions for each request, layer, K/V and head, as the pages hold it
    T = pt.shape[1] * page
    at = np.arange(T)
    held = np.array([-(-(p + 3 * R) // page) * page for p in lens])
    codes = np.full((B, L, 2, KVH, T, hd), 0x31, np.uint8)
    exps = np.full((B, L, 2, KVH, T // block), -77, np.int8)
    for b in range(B):  # the rows that are there already: their exponents are what counts
        exps[b, :, :, :, :-(-lens[b] // block)] = rng.integers(-9, -4, (L, 2, KVH, -(-lens[b] // block)))
        for j in range(T // block):
            if j * block < held[b]:
                pg = pt[b, j * block // page]
                for w in range(2):
                    bufs[2 + w][:, pg, :, j * block % page // block] = to_dev(exps[b, :, w, :, j])
    for turn in range(3):
        x = [rng.normal(size=(L, sn, KVH, 16, hd)) * np.exp2(rng.integers(-3, 4, (L, 1, KVH, 1, 1)) + 2.0 * turn) for _ in range(2)]
        for w in range(2):  # rows of 0, ties between neighbouring codes, values far below the block's largest
            x[w][:, :, :, 1::5] = 0.0
            x[w][:, :, :, 2::5, :16] = np.array([17, 19, 21, 23, 25, 27, 29, 31, -17, -19, -21, -23, -25, -27, -29, -31]) * 0.25
            x[w][:, :, :, 3::5] *= 2.0 ** -13
        src = [to_dev(a.astype(np.float32), torch.bfloat16) for a in x]
        x = [host(t).astype(np.float64) for t in src]
        n_rows = rng.integers(0, R + 1, B)
        n_rows[turn % B] = R
        ids = np.stack([np.concatenate([[0], 1 + rng.permutation(38)])[:R] for _ in range(B)]) if path else None
        nxt = dlen if in_place else torch.full_like(dlen, -1)
        # (n_rows - 1 with n_add 1: a request without a row passes -1)
        e3.kv8_append(layers, bf16_layers(src, dspt, 16, KVH, hd), B, R, None if ids is None else i32(ids),
                      i32(n_rows - (1 if path else 0)), 1 if path else 0, dlen, nxt, err)
        torch.cuda.synchronize()
        for b in range(B):
            j = np.arange(n_rows[b])
            s = ids[b, j] if path else j
            for w in range(2):
                rows = x[w][:, spt[b, s // 16], :, s % 16]  # [n][L][KVH][hd]
                for l in range(L):
                    for h in range(KVH):
                        kv8_ref.append(codes[b, l, w, h], exps[b, l, w, h], lens[b], rows[:, l, h], block)
        lens = [p + int(k) for p, k in zip(lens, n_rows)]
        assert host(nxt).tolist() == lens
        dlen = nxt
    assert int(err.item()) == 0
    got = [host(b) for b in bufs]
    for b in range(B):
        t, j = at[:held[b]], at[:held[b]:block]
        for w in range(2):
            assert np.array_equal(got[w][:, pt[b, t // page], :, t % page], codes[b, :, w, :, :held[b]].transpose(2, 0, 1, 3))
            assert np.array_equal(got[2 + w][:, pt[b, j // page], :, j % page // block], exps[b, :, w, :, :len(j)].transpose(2, 0, 1))
    # read back, from the middle of a block
    first = np.minimum(rng.integers(0, 20, B), lens)
    n_back = np.array(lens) - first
    most = max(1, int(n_back.max()))
    bpt, bn = synth.page_table(seed + 5, [most] * B, 32)
    back = [torch.full((L, bn, KVH, 32, hd), 33.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dbpt = i32(bpt)
    e3.kv8_read(layers, bf16_layers(back, dbpt, 32, KVH, hd), B, most, i32(first), i32(n_back), err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for w in range(2):
        want = np.full(back[w].shape, 33.0)
        for b in range(B):
            r = np.arange(n_back[b])
            t = first[b] + r
            e = np.repeat(exps[b, :, w], block, -1)[:, :, t]
            want[:, bpt[b, r // 32], :, r % 32] = kv8_ref.decode(codes[b, :, w][:, :, t], e[..., None]).transpose(2, 0, 1, 3)
        assert np.array_equal(host(back[w]), want)


def test_kv8_append_ends_of_the_range():
    """NaN, Inf, the largest and the smallest bf16 values; a block of zeros; a scale that grows by its whole range."""
    KVH, hd, page, block = 1, 64, 16, 16
    x = torch.zeros((6, KVH, page, hd), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3.3895e38], device="cuda")
    x[0, 0, 1, 0] = -1.0
    x[1, 0, 0, 0] = 3.3895e38
    x[2, 0, 0, 0] = 1e-40
    x[2, 0, 1, 0] = 2.0 ** -100
    x[4, 0, 0] = 2.0 ** -90
    x[5, 0, 0] = 1.0
    bufs = kv8_buffers(1, 6, KVH, page, hd, block)
    pt = i32([[b] for b in range(6)])
    layers, src = kv8_layers(bufs, pt, page, KVH, hd, block), bf16_layers([x[None], x[None]], pt, page, KVH, hd)
    lens = torch.zeros(6, dtype=torch.int32, device="cuda")
    for b, flag in enumerate([e3.E3_DEV_ERR_NONFINITE, 0, 0, 0, 0, 0]):
        err = err_word()
        e3.kv8_append(layers, src, 6, 2, None, i32([2 if i == b else 0 for i in range(6)]), 0, lens, lens, err)
        torch.cuda.synchronize()
        assert int(err.item()) == flag, b
    err = err_word()
    # behind 2^-90, a row of 1.0: the exponent grows from -98 to -8, the old codes are 0 then
    s45 = i32([[5]] * 6)
    e3.kv8_append(layers, bf16_layers([x[None], x[None]], s45, page, KVH, hd), 6, 1, None, i32([0, 0, 0, 0, 1, 0]), 0, lens, lens, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and host(lens).tolist() == [2, 2, 2, 2, 3, 2]
    e = host(bufs[2])[0, :, 0, 0].tolist()
    assert e == [120, 120, -100, -100, -8, -8]
    v = kv8_ref.decode(host(bufs[0])[0, :, 0], host(bufs[2])[0, :, 0, :, None].astype(np.float64))
    top = kv8_ref.TOP
    assert v[0, 0, :4].tolist() == [0.0, top, -top, top] and v[0, 1, 0] == 0.0  # (-1 is far below the scale)
    assert v[1, 0, 0] == top and v[2, 0, 0] == 0.0 and v[2, 1, 0] == 2.0 ** -100
    assert np.all(v[4, :2] == 0.0) and np.all(v[4, 2] == 1.0) and np.all(v[5, 0] == 1.0)


def test_kv8_refused_requests_stay_as_they_were():
    """Too many rows, no room, a bad page on either side: flagged; the first two leave the request alone."""
    KVH, hd, page, block, B, R = 1, 64, 16, 16, 6, 4
    src = to_dev(np.random.default_rng(9).normal(size=(1, 8, KVH, page, hd)).astype(np.float32), torch.bfloat16)
    bufs = kv8_buffers(1, 8, KVH, page, hd, block)
    pt = i32([[0, 1], [2, 3], [4, -7], [5, 6], [7, 7], [3, 3]])
    spt = i32([[0], [1], [2], [3], [4], [8]])
    layers, s16 = kv8_layers(bufs, pt, page, KVH, hd, block), bf16_layers([src, src], spt, page, KVH, hd)
    lens = i32([0, 30, 14, 3, 2 ** 31 - 2, 0])
    expect = {0: (e3.E3_DEV_ERR_CAPACITY, 0), 1: (e3.E3_DEV_ERR_CAPACITY, 30), 2: (e3.E3_DEV_ERR_CAPACITY, 18), 3: (0, 3),
              4: (e3.E3_DEV_ERR_CAPACITY, 2 ** 31 - 2), 5: (e3.E3_DEV_ERR_CAPACITY, 4)}
    for b, (flag, after) in expect.items():
        n = [0] * B
        n[b] = {0: 5, 3: -2}.get(b, 4)
        nxt, err = torch.zeros_like(lens), err_word()
        for t in bufs:
            t.zero_()
        e3.kv8_append(layers, s16, B, R, None, i32(n), 0, lens, nxt, err)
        torch.cuda.synchronize()
        assert int(err.item()) == flag, b
        assert int(nxt[b]) == after and host(nxt).tolist()[:b] == host(lens).tolist()[:b]
        c = host(bufs[0])[0, :, 0]
        if b == 2:  # the rows on the good page are written
            assert c[4, 14:].any() and not c[:4].any() and not c[5:].any()
        else:
            assert not c.any()
    dst, err = torch.zeros_like(src), err_word()
    for first, n in ((None, [0, 0, 0, 0, 4, 0]), ([0, 0, 0, 31, 0, 0], [0, 0, 0, 2, 0, 0]), ([-1] * 6, [1, 0, 0, 0, 0, 0])):
        err = err_word()
        e3.kv8_read(layers, bf16_layers([dst, dst.clone()], spt, page, KVH, hd), B, 3, None if first is None else i32(first), i32(n), err)
        torch.cuda.synchronize()
        assert int(err.item()) == e3.E3_DEV_ERR_CAPACITY and not host(dst).any()


# -------------------------------------------------------------------- attention

def attn_inputs(seed, B, R, H, KVH, hd, lens, page, block, spread=1.0, exps=(-9, -4)):
    rng = np.random.default_rng(seed)
    pt, n = synth.page_table(seed, [max(p, 1) for p in lens], page)
    kv = []
    for _ in range(2):  # every slot holds something, beyond a request's length too: NaN
        c = (rng.integers(0, 2, (n, KVH, page, hd)) * 128 + rng.integers(0, 127, (n, KVH, page, hd))).astype(np.uint8)
        kv.append((c, rng.integers(*exps, (n, KVH, page // block)).astype(np.int8)))
    for b, p in enumerate(lens):
        for t in range(p, (p + page - 1) // page * page):
            for w in range(2):
                kv[w][0][pt[b, t // page], :, t % page] = 127 + 128 * (t & 1)
    nt = (R + page - 1) // page
    tpt = rng.permutation(B * nt).reshape(B, nt).astype(np.int32)
    tail = [synth.to_bf16_f32(rng.normal(size=(B * nt, KVH, page, hd)).astype(np.float32)) for _ in range(2)]
    Q = synth.to_bf16_f32((spread * rng.normal(size=(B, R, H, hd))).astype(np.float32))
    see = np.stack([ancestors(random_tree(rng, R, 6)[0]) for _ in range(B)])
    return dict(B=B, R=R, H=H, KVH=KVH, hd=hd, lens=lens, page=page, block=block, pt=pt, n=n, kv=kv, tpt=tpt, tail=tail, Q=Q, see=see)


def attn_call(d, max_kv_len=None, flags=0, tail_flags=0, ws=None, out=None, stream=None, err=None, dev=None):
    """Runs tree_verify_attn8; `dev` keeps device copies between calls."""
    dev = {} if dev is None else dev
    if not dev:
        dev.update(Q=to_dev(d["Q"], torch.bfloat16), pt=i32(d["pt"]), tpt=i32(d["tpt"]), lens=i32(d["lens"]),
                   mask=mask_of(d["see"]), tail=[to_dev(t, torch.bfloat16) for t in d["tail"]],
                   kv=[[to_dev(a) for a in w] for w in d["kv"]])
    B, R, H, KVH, hd, page = (d[k] for k in ("B", "R", "H", "KVH", "hd", "page"))
    kv = e3.make_kv8_layer(dev["kv"][0][0], dev["kv"][1][0], dev["kv"][0][1], dev["kv"][1][1], dev["pt"], d["n"], page,
                           d["pt"].shape[1], KVH, hd, d["block"], flags)
    tail = e3.make_kv_layer(*dev["tail"], dev["tpt"], dev["tail"][0].shape[0], page, d["tpt"].shape[1], KVH, hd, e3.E3_BF16, tail_flags)
    mx = max(d["lens"]) if max_kv_len is None else max_kv_len
    need = e3.eagle3_verify8_workspace_bytes(B, R, H, KVH, hd, mx)
    if ws is None:
        ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    O, lse = out or (torch.full((B, R, H, hd), 55.0, dtype=torch.bfloat16, device="cuda"),
                     torch.full((B, R, H), 55.0, device="cuda"))
    err = err_word() if err is None else err
    e3.tree_verify_attn8(dev["Q"], kv, tail, dev["lens"], dev["mask"], B, R, H, mx, 1 / math.sqrt(hd), O, lse, err, ws, need,
                         stream=stream)
    return O, lse, err


def attn_check(d, O, lse, requests=None):
    O, lse = host(O).astype(np.float64), host(lse).astype(np.float64)
    page, R, block = d["page"], d["R"], d["block"]
    for b in requests if requests is not None else range(d["B"]):
        t, j = np.arange(d["lens"][b]), np.arange(R)
        pg = d["pt"][b, t // page]
        exps = [d["kv"][w][1][pg, :, t % page // block].astype(np.float64)[..., None] for w in range(2)]
        k, v = (kv8_ref.decode(d["kv"][w][0][pg, :, t % page], exps[w]) for w in range(2))
        tk, tv = (d["tail"][w][d["tpt"][b, j // page], :, j % page].astype(np.float64) for w in range(2))
        o, l, mag, big = kv4_ref.attend(d["Q"][b].astype(np.float64), k, v, tk, tv, d["see"][b], 1 / math.sqrt(d["hd"]))
        ds = 2.0 ** -18 * (big + 1.0)
        dead = ~d["see"][b].any(-1) if d["lens"][b] == 0 else np.zeros(R, bool)
        assert np.all(O[b][dead] == 0) and np.all(np.isneginf(lse[b][dead]))
        live = ~dead
        assert np.all(np.abs(lse[b][live] - l[live]) <= (ds + 2.0 ** -21 * np.abs(l))[live]), np.abs(lse[b][live] - l[live]).max()
        # |e| <= the weights' error times mag; the output is then rounded by at most half a step of
        # that value: |e| + 2^-8 (|o| + |e|).  Weights below fp16's normal range: see the head of this file
        tiny = 0.0
        if len(t):
            codes = np.abs(v) * 2.0 ** (exps[1].max(0, keepdims=True) - exps[1])  # V where its block had the largest scale
            tiny = 2.0 ** -32 * np.repeat(codes.sum(0), d["H"] // d["KVH"], 0)[None]
        e = (2.0 ** -8 + 2 * ds[..., None]) * mag + tiny
        tol = e + 2.0 ** -8 * (np.abs(o) + e) + 2.0 ** -126
        bad = np.abs(O[b] - o)[live] - tol[live]
        assert np.all(bad <= 0), (b, bad.max())


ATTN = [
    # B, R, H, KVH, hd, page, block, lens
    (1, 1, 32, 8, 128, 64, 64, [1]),
    (2, 1, 4, 4, 64, 16, 16, [0, 17]),             # no prefix: the node alone
    (1, 1, 32, 8, 128, 64, 16, [2049]),
    (3, 1, 32, 8, 128, 16, 16, [15, 16, 700]),
    (1, 61, 32, 8, 128, 64, 64, [2048]),
    (2, 15, 4, 4, 64, 16, 16, [128, 1025]),
    (3, 33, 8, 1, 128, 64, 32, [63, 64, 65]),
    (2, 5, 6, 2, 64, 32, 32, [300, 0]),
    (1, 200, 8, 8, 128, 16, 16, [130]),
    (2, 256, 4, 1, 128, 128, 128, [129, 1000]),
    (2, 17, 5, 5, 128, 64, 16, [511, 1]),
    (1, 8, 64, 8, 128, 64, 64, [12345]),
    (4, 61, 32, 8, 128, 64, 64, [512, 0, 1777, 128]),
    (2, 64, 40, 8, 128, 128, 64, [640, 90]),       # five query heads per KV head
    (2, 3, 48, 1, 64, 48, 16, [97, 48]),
    (1, 2, 16, 1, 128, 256, 128, [40000]),
    (1, 130, 2, 1, 128, 96, 32, [1000]),
]


@pytest.mark.parametrize("case", ATTN)
def test_verify_attn8(case):
    B, R, H, KVH, hd, page, block, lens = case
    d = attn_inputs(R * 7 + H + hd + lens[0], B, R, H, KVH, hd, lens, page, block)
    O, lse, err = attn_call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    attn_check(d, O, lse)


def test_verify_attn8_repeats_bit_for_bit_and_with_looser_bounds():
    """Same inputs, same bits, on dirty workspaces and with the prefix promise; a larger length bound stays right."""
    for R in (2, 20):
        d = attn_inputs(11, 3, R, 16, 4, 128, [100, 1500, 64], 64, 32)
        dev = {}
        O, lse, _ = attn_call(d, dev=dev)
        O2, lse2, _ = attn_call(d, dev=dev, flags=e3.E3_KV_PREFIX_STABLE)
        torch.cuda.synchronize()
        assert torch.equal(O, O2) and torch.equal(lse, lse2)
        O3, lse3, err = attn_call(d, dev=dev, max_kv_len=d["pt"].shape[1] * 64)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        attn_check(d, O3, lse3)


@pytest.mark.parametrize("R,G,P", [(1, 4, 300), (33, 4, 300), (61, 4, 1000), (200, 1, 64), (80, 3, 500)])
def test_verify_attn8_scales_and_sharp_rows(R, G, P):
    """Blocks of very different scales, rows of very different magnitudes, scores that move the softmax base far."""
    d = attn_inputs(R + P, 2, R, 2 * G, 2, 128, [P, P // 2], 64, 16, spread=4.0, exps=(-14, -5))
    rng = np.random.default_rng(1)
    d["Q"] *= np.exp2(rng.integers(-20, 5, d["Q"].shape[:3]))[..., None].astype(np.float32)
    d["Q"][0, 0] = 0.0
    d["Q"] = synth.to_bf16_f32(d["Q"])
    O, lse, err = attn_call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    attn_check(d, O, lse)


@pytest.mark.parametrize("R", [1, 3, 20, 70])
def test_verify_attn8_ends_of_the_exponents(R):
    """K's scale against Q's magnitude at both ends; V's at both ends beside nodes of ordinary size."""
    for ke, qe, ve in ((-95, 92, -98), (100, -103, 88), (-6, 0, 90), (-6, 0, -99)):
        d = attn_inputs(R + 200 + ve, 1, R, 8, 2, 128, [200], 64, 64)
        d["kv"][0][1][:] = ke
        d["kv"][1][1][:] = ve
        d["Q"] = synth.to_bf16_f32((d["Q"] * 2.0 ** qe).astype(np.float32))
        # the nodes' scores stay moderate too
        d["tail"][0] = synth.to_bf16_f32((d["tail"][0] * 2.0 ** -qe).astype(np.float32))
        O, lse, err = attn_call(d)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        attn_check(d, O, lse)


@pytest.mark.parametrize("R,H", [(5, 4), (40, 16), (80, 8)])
def test_verify_attn8_masked_places_hold_anything(R, H):
    """NaN and Inf in tail slots: rows that do not see them are exact, rows that see a bad V get NaN;
    rows that see nothing (no prefix, empty mask) give 0 and -Inf; slots beyond R do not matter."""
    d = attn_inputs(R, 2, R, H, 2, 128, [0, 130], 64, 64)
    d["see"][0, 2:4] = False
    bad = R - 1
    d["see"][:, :bad, bad] = False
    clean = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in d.items()}
    clean["tail"] = [t.copy() for t in d["tail"]]
    page = d["page"]
    for b in range(2):
        d["tail"][0][d["tpt"][b, bad // page], :, bad % page] = np.nan
        d["tail"][1][d["tpt"][b, bad // page], :, bad % page, 7] = np.inf if b else np.nan
    if R % page:
        for w in range(2):
            d["tail"][w][d["tpt"][:, -1], :, R % page:] = np.nan
    O, lse, err = attn_call(d)
    clean["see"][:, bad] = False
    clean["see"][:, bad, 0] = True
    O2, lse2, _ = attn_call(clean)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    O, lse, O2, lse2 = (host(t).copy() for t in (O, lse, O2, lse2))
    assert np.isnan(O[:, bad]).all()
    O[:, bad], lse[:, bad] = O2[:, bad], lse2[:, bad]
    attn_check(clean, torch.from_numpy(O), torch.from_numpy(lse))
    # only V of the seen node is bad: the row's lse stays that of its scores
    d["tail"][0] = clean["tail"][0].copy()
    O3, lse3, _ = attn_call(d)
    torch.cuda.synchronize()
    assert np.isnan(host(O3)[:, bad]).all() and np.isfinite(host(lse3)[:, bad]).all()


def test_verify_attn8_capacity_is_flagged():
    """A length beyond the bound, a negative one: outputs of that request untouched, the others exact; a bad page id is flagged."""
    for lens_now, R in (([5000, 64, 100], 3), ([-1, 64, 100], 40)):
        d = attn_inputs(77 + R, 3, R, 8, 2, 128, [64, 64, 100], 64, 32)
        dev = {}
        attn_call(d, dev=dev)
        dev["lens"] = i32(lens_now)
        O, lse, err = attn_call(d, dev=dev)
        torch.cuda.synchronize()
        assert int(err.item()) == e3.E3_DEV_ERR_CAPACITY
        assert torch.all(O[0] == 55.0) and torch.all(lse[0] == 55.0)
        attn_check(d, O, lse, requests=[1, 2])
        dev["lens"] = i32(d["lens"])
        dev["pt"] = i32([[d["n"]] * d["pt"].shape[1]] + d["pt"].tolist()[1:])
        O, lse, err = attn_call(d, dev=dev)
        torch.cuda.synchronize()
        assert int(err.item()) == e3.E3_DEV_ERR_CAPACITY
        attn_check(d, O, lse, requests=[1, 2])


def test_verify_attn8_on_streams_and_in_a_graph():
    """Two calls on two streams with scratch of their own; a captured call replayed on changed inputs."""
    a = attn_inputs(1, 2, 40, 16, 4, 128, [900, 33], 64, 64)
    b = attn_inputs(2, 2, 1, 16, 4, 128, [700, 1000], 64, 16)
    da, db = {}, {}
    attn_call(a, dev=da)
    attn_call(b, dev=db)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ra = attn_call(a, dev=da)
        with torch.cuda.stream(s2):
            rb = attn_call(b, dev=db)
    torch.cuda.synchronize()
    attn_check(a, ra[0], ra[1])
    attn_check(b, rb[0], rb[1])
    need = e3.eagle3_verify8_workspace_bytes(2, 40, 16, 4, 128, 900)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = (torch.zeros((2, 40, 16, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 40, 16), device="cuda"))
    err = err_word()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn_call(a, dev=da, ws=ws, out=out, err=err)
    a["lens"] = [450, 20]
    da["lens"].copy_(i32(a["lens"]))
    a["Q"] = synth.to_bf16_f32(a["Q"] * 1.5)
    da["Q"].copy_(to_dev(a["Q"], torch.bfloat16))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    attn_check(a, *out)


@pytest.mark.parametrize("B,R,H,KVH,hd,most", [
    (48, 17, 32, 8, 128, 300), (48, 17, 32, 8, 128, 40), (40, 61, 32, 8, 128, 900), (24, 200, 16, 4, 128, 500), (64, 3, 16, 4, 64, 700)])
def test_verify_attn8_many_requests_of_differing_length(B, R, H, KVH, hd, most):
    """Shares that end inside a request, hold several, or begin behind one's last tile."""
    rng = np.random.default_rng(B + R + most)
    lens = [int(x) for x in np.where(rng.random(B) < 0.15, 0, rng.integers(1, most + 1, B))]
    lens[1] = 12 * most
    d = attn_inputs(R, B, R, H, KVH, hd, lens, 16, 16)
    dev = {}
    O, lse, err = attn_call(d, dev=dev)
    O2, lse2, _ = attn_call(d, dev=dev, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    assert not torch.any(O == 55.0) and not torch.any(lse == 55.0)
    attn_check(d, O, lse, requests=[0, 1, 2, B // 2, B - 1])


@pytest.mark.parametrize("R,H", [(20, 16), (40, 16)])
def test_verify_attn8_wait_that_runs_out(R, H):
    """The self-test bit on the tail: a tile that never comes ends the call with the error word set,
    after the waits' bound, and leaves nothing behind that the next call on the same buffers meets."""
    d = attn_inputs(R, 2, R, H, 4, 128, [900, 300], 64, 32)
    dev = {}
    need = e3.eagle3_verify8_workspace_bytes(2, R, H, 4, 128, 900)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    attn_call(d, dev=dev, ws=ws)
    torch.cuda.synchronize()
    _, _, err = attn_call(d, dev=dev, ws=ws, tail_flags=e3.E3_KV_SELFTEST_STALL)
    torch.cuda.synchronize()
    assert int(err.item()) == e3.E3_DEV_ERR_TIMEOUT
    O, lse, err = attn_call(d, dev=dev, ws=ws)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    attn_check(d, O, lse)


@pytest.mark.parametrize("R,H,KVH,hd", [(40, 4, 4, 64), (100, 6, 2, 64), (197, 6, 2, 64), (31, 8, 8, 128), (256, 2, 1, 64)])
def test_verify_attn8_granules_of_nodes_that_no_row_sees(R, H, KVH, hd):
    """Few rows per tile and many nodes: deep and shallow trees, tiles whose rows see no node at all (beside a prefix and
    without one), a NaN in V of a node that one row sees."""
    d = attn_inputs(R + hd, 3, R, H, KVH, hd, [0, 130, 517], 64, 16)
    d["see"][0, 16:32] = False             # no key at all
    d["see"][1, :] = np.eye(R, dtype=bool)  # each node itself alone
    d["see"][2, R // 2:] = False            # the prefix alone
    d["see"][2, R - 1, R - 1] = True
    O, lse, err = attn_call(d)
    O2, lse2, _ = attn_call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    attn_check(d, O, lse)
    bad = R - 1
    d["tail"][1][d["tpt"][2, bad // 64], :, bad % 64, 5] = np.nan
    O3, lse3, _ = attn_call(d)
    torch.cuda.synchronize()
    assert torch.isnan(O3[2, bad]).all() and torch.equal(lse3, lse)
    keep = torch.ones((3, R), dtype=torch.bool, device="cuda")
    keep[2, bad] = False
    if not d["see"][2, :bad, bad].any():
        assert torch.equal(O3[keep], O[keep])
