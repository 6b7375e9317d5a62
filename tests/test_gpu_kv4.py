"""GPU parity of the verify pass over a 4-bit cache with plain 64-bit forms (kv4_ref).

Tolerances, from the arithmetic:
  rotation   a position's phase is exact modulo a turn; as a float it is off by at most
             2^-25 half-turns, and sincospif and the products round a few times: 2^-18 of
             the head's largest value bounds the sum of all of it with the fp32 norm
             (256 squares: under 2^-20 relative).  The output adds half a step of its type.
  attention  scores: fp32 sums of 128 products, 2^-18 of the largest sum |q||k| scale.
             weights: rounded to fp16 (2^-11) or, for tree nodes, bf16 (2^-8), relative;
             twice the score error; output: half a bf16 step of the value reached, 2^-8.
  rows of the 4-bit cache, processed logits and statistics are equal bit for bit.
"""
import math

import numpy as np
import pytest
import torch

import kv4_ref
import oracle
from eagle_speculative_decoding_round_gb300 import synth
from gpu_util import host, random_tree, to_dev

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from eagle_speculative_decoding_round_gb300 import eagle3 as e3

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def ruled_out(z):
    """-Inf as the oracle takes it: finite, and without mass."""
    return np.where(np.isneginf(z), np.float32(-1e30), z).astype(np.float32)


def i32(a):
    return to_dev(np.asarray(a, np.int32))


def bits(*shape, seed=0, dt="bf16"):
    """Seeded N(0, 1) values on the grid of dt: (device tensor, float64 array)."""
    a = synth.normal(seed, "x" + str(shape), shape, 1.0)
    t = to_dev(a, TD[dt])
    return t, host(t).astype(np.float64)


def mask_of(see):
    R = see.shape[-1]
    W = (R + 63) // 64
    out = np.zeros(see.shape[:-1] + (W,), np.uint64)
    for j in range(R):
        out[..., j // 64] |= see[..., j].astype(np.uint64) << np.uint64(j % 64)
    return to_dev(out.view(np.int64))


def ancestors(parent):
    R = len(parent)
    see = np.eye(R, dtype=bool)
    for i in range(1, R):
        see[i] |= see[parent[i]]
        see[i, i] = True
    return see


# ------------------------------------------------------- norms, rotation, append

QKV = [
    # B, R, H, KVH, hd, page, dt, rot, inter, scaling, norm, pad, lens
    (1, 1, 32, 8, 128, 64, "bf16", 128, False, "plain", False, 0, [0]),
    (2, 61, 32, 8, 128, 64, "bf16", 128, False, "wavelen", True, 0, [2048, 77]),
    (3, 15, 4, 4, 64, 16, "f32", 32, True, "linear", True, 0, [128, 0, 31]),
    (2, 5, 6, 1, 64, 16, "bf16", 24, False, "yarn", True, 0, [15, 16]),       # pairs that no 16-byte piece holds
    (2, 5, 3, 1, 96, 32, "bf16", 96, False, "plain", True, 0, [5, 70]),       # a head of 96: the scalar path
    (1, 9, 2, 2, 256, 16, "f32", 256, False, "plain", True, 0, [1]),
    (1, 9, 5, 5, 32, 16, "bf16", 16, True, "plain", False, 0, [33]),
    (2, 33, 8, 2, 128, 64, "bf16", 64, False, "plain", True, 8, [100000, 3]),  # wide rows, far positions
    (2, 33, 8, 2, 128, 64, "bf16", 128, False, "plain", False, 3, [9, 3]),     # rows off the 16-byte grid
    (1, 300, 64, 8, 128, 128, "bf16", 128, False, "plain", False, 0, [40]),
    (4, 3, 2, 1, 224, 16, "f32", 0, False, "plain", True, 1, [0, 1, 2, 3]),    # no rotation
]


@pytest.mark.parametrize("case", QKV)
def test_qkv_append(case):
    B, R, H, KVH, hd, page, dt, rot, inter, scaling, norm, pad, lens = case
    seed = B * 1000 + R * 10 + hd
    ld = (H + 2 * KVH) * hd + pad
    qkv, q64 = bits(B * R, ld, seed=seed, dt=dt)
    rng = np.random.default_rng(seed)
    pt, n = synth.page_table(seed, [p + R for p in lens], page)
    pos = np.array(lens)[:, None] + rng.integers(0, 7, (B, R))
    n_rows = np.array([R - (b % 2) * (R // 2) for b in range(B)])
    kw = dict(linear=dict(factor=4.0), wavelen=dict(factor=8.0, low=1.0, high=4.0, orig_len=8192.0),
              yarn=dict(factor=16.0, low=1.0, high=32.0, orig_len=4096.0)).get(scaling, {})
    rope = ref_rope = None
    if rot:
        kind = ["plain", "linear", "wavelen", "yarn"].index(scaling)
        rope = e3.eagle3_rope_init(rot, 500000.0, interleaved=inter, scaling=kind, **kw)
        ref_rope = kv4_ref.rope_freqs(rot, 500000.0, scaling, **kw) + (rot, inter)
    norms = [None, None]
    if norm:
        norms = [1 + synth.normal(seed, f"n{i}", (hd,), 0.2) for i in range(2)]
    nd = [None if x is None else to_dev(x) for x in norms]
    K = torch.full((n, KVH, page, hd), 77.0, dtype=TD[dt], device="cuda")
    V, Q = K.clone(), torch.full((B, R, H, hd), 77.0, dtype=TD[dt], device="cuda")
    kv = e3.make_kv_layer(K, V, i32(pt), n, page, pt.shape[1], KVH, hd, e3.E3_BF16 if dt == "bf16" else e3.E3_F32)
    keep = [i32(pt), i32(lens), i32(pos), i32(n_rows)]
    kv.page_table = keep[0].data_ptr()
    err = err_word()
    e3.tree_qkv_append(qkv, ld, B, R, keep[3], H, nd[0], nd[1], 1e-5, rope, keep[2], Q, kv, keep[1], err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    x = q64[:, :(H + 2 * KVH) * hd]
    want = [p.reshape(B, R, -1, hd) for p in kv4_ref.qkv_heads(x, H, KVH, hd, *norms, 1e-5, ref_rope, pos.reshape(-1))]
    got = [host(t).astype(np.float64) for t in (Q, K, V)]
    hit = np.zeros((n, page), bool)

    def near(g, w, what):
        amax = np.abs(w).max(-1, keepdims=True) * (1.0 if ref_rope is None else max(1.0, ref_rope[1]) * math.sqrt(2))
        assert np.all(np.abs(g - w) <= HALF_STEP[dt] * np.abs(w) + 2.0 ** -18 * amax), what
    for b in range(B):
        for r in range(R):
            if r >= n_rows[b]:
                assert np.all(got[0][b, r] == 77.0)  # left as it was
                continue
            t = lens[b] + r
            pg, sl = pt[b, t // page], t % page
            hit[pg, sl] = True
            near(got[0][b, r], want[0][b, r], "q")
            near(got[1][pg, :, sl], want[1][b, r], "k")
            assert np.array_equal(got[2][pg, :, sl], want[2][b, r]), "v is copied"
    assert np.all(got[1].transpose(0, 2, 1, 3)[~hit] == 77.0) and np.all(got[2].transpose(0, 2, 1, 3)[~hit] == 77.0)


def test_qkv_append_bad_slots_are_flagged():
    """Rows without a page: past the table, a page id out of range, a negative length; Q is still written."""
    B, R, H, KVH, hd, page = 4, 20, 2, 1, 64, 16
    qkv, q64 = bits(B * R, (H + 2 * KVH) * hd, seed=5)
    K = torch.zeros((4, KVH, page, hd), dtype=torch.bfloat16, device="cuda")
    V, Q = K.clone(), torch.zeros((B, R, H, hd), dtype=torch.bfloat16, device="cuda")
    pt = i32([[0, 1], [2, 9], [-1, 3], [0, 1]])
    kv = e3.make_kv_layer(K, V, pt, 4, page, 2, KVH, hd, e3.E3_BF16)
    lens, err = i32([2 ** 31 - 5, 0, 0, -3]), err_word()
    e3.tree_qkv_append(qkv, (H + 2 * KVH) * hd, B, R, None, H, None, None, 0.0, None, None, Q, kv, lens, err)
    torch.cuda.synchronize()
    assert int(err.item()) == e3.E3_DEV_ERR_CAPACITY
    assert np.array_equal(host(Q).reshape(B * R, H * hd), q64[:, :H * hd])
    k = host(K)
    x = q64[:, H * hd:(H + 1) * hd].reshape(B, R, hd)
    assert np.array_equal(k[2, 0], x[1, :16]) and np.array_equal(k[3, 0, :4], x[2, 16:])
    assert np.all(k[0] == 0) and np.all(k[1] == 0) and np.all(k[3, 0, 4:] == 0)


# ------------------------------------------------------------ rows of the cache

def kv4_buffers(L, n, KVH, page, hd, fill=0):
    mk = lambda w: torch.full((L, n, KVH, page, w), fill, dtype=torch.uint8, device="cuda")  # noqa: E731
    return [mk(hd // 2), mk(hd // 2), mk(hd // 16), mk(hd // 16)]


def kv4_layers(bufs, pt, page, KVH, hd, units):
    return [e3.make_kv4_layer(*[b[l] for b in bufs], pt, bufs[0].shape[1], page, pt.shape[1], KVH, hd, *units[l])
            for l in range(bufs[0].shape[0])]


@pytest.mark.parametrize("B,R,L,KVH,hd,page,path,in_place", [
    (1, 1, 1, 1, 64, 16, False, False), (3, 7, 3, 8, 128, 64, True, True), (2, 7, 2, 2, 64, 16, True, False),
    (2, 501, 2, 3, 128, 16, False, True), (1, 1030, 1, 8, 128, 128, False, False)])
def test_kv4_append_and_read(B, R, L, KVH, hd, page, path, in_place):
    seed = B * 100 + R + hd
    rng = np.random.default_rng(seed)
    spt, sn = synth.page_table(seed + 1, [max(R, 40)] * B, page)
    x = [rng.normal(size=(L, sn, KVH, page, hd)) * np.exp(2 * rng.normal(size=(L, 1, KVH, 1, hd))) for _ in range(2)]
    for w in range(2):  # whole groups of 0, one tiny value, ties on every midpoint, values beyond the scale's range
        x[w][:, :, :, 1::4, :16] = 0.0
        x[w][:, :, :, 2::4, :16] = 0.0
        x[w][:, :, :, 2::4, 3] = 2.0 ** -12
        x[w][:, :, :, 3::4, :16] = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -0.0]) * 1.625
        x[w][:, :, :, ::8, 16:32] *= 2.0 ** 14
    src = [to_dev(a.astype(np.float32), torch.bfloat16) for a in x]
    x = [host(t).astype(np.float64) for t in src]
    lens = [int(v) for v in rng.integers(0, 50, B)]
    pt, n = synth.page_table(seed, [p + R for p in lens], page)
    n_rows = rng.integers(1, R + 1, B)
    n_rows[0] = R
    ids = np.stack([np.concatenate([[0], 1 + rng.permutation(38)])[:R] for _ in range(B)]) if path else None
    units = [(2.0 ** (l - 1), 2.0 ** -l) for l in range(L)]
    bufs = kv4_buffers(L, n, KVH, page, hd, fill=165)
    dpt, dspt, dlen, dn = i32(pt), i32(spt), i32(lens), i32(n_rows - (1 if path else 0))
    drows = None if ids is None else i32(ids)
    layers = kv4_layers(bufs, dpt, page, KVH, hd, units)
    sl = [e3.make_kv_layer(src[0][l], src[1][l], dspt, sn, page, spt.shape[1], KVH, hd, e3.E3_BF16) for l in range(L)]
    nxt = dlen if in_place else torch.full_like(dlen, -1)
    err = err_word()
    e3.kv4_append(layers, sl, B, R, drows, dn, 1 if path else 0, dlen, nxt, err)
    back = [torch.full_like(t, 33.0) for t in src]
    dst = [e3.make_kv_layer(back[0][l], back[1][l], dspt, sn, page, spt.shape[1], KVH, hd, e3.E3_BF16) for l in range(L)]
    first = i32(lens)
    e3.kv4_read(layers, dst, B, R, first, i32(n_rows), err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert np.array_equal(host(nxt), np.array(lens) + n_rows)
    if not in_place:
        assert np.array_equal(host(dlen), lens)
    got = [host(b) for b in bufs]
    want = [np.full_like(g, 165) for g in got]
    wback = [np.full(a.shape, 33.0) for a in x]
    for b in range(B):
        j = np.arange(n_rows[b])
        s = ids[b, j] if path else j
        t = lens[b] + j
        for w in range(2):
            for l in range(L):
                c, e = kv4_ref.quantize(x[w][l, spt[b, s // page], :, s % page], units[l][w])
                want[w][l, pt[b, t // page], :, t % page] = c
                want[2 + w][l, pt[b, t // page], :, t % page] = e
                wback[w][l, spt[b, j // page], :, j % page] = kv4_ref.dequantize(c, e, units[l][w])
    for g, w in zip(got, want):
        assert np.array_equal(g, w)  # codes and scales, and every untouched slot
    for w in range(2):
        assert np.array_equal(host(back[w]), wback[w])


def test_kv4_append_refused_requests_stay_as_they_were():
    """Too many rows, no room, a bad page, a non-finite value: flagged; the first two leave the request alone."""
    L, KVH, hd, page, B, R = 1, 1, 64, 16, 5, 4
    src, _ = bits(8, KVH, page, hd, seed=9)
    src[4, 0, 1, 5] = float("nan")
    src[4, 0, 2, 40] = float("inf")
    bufs = kv4_buffers(L, 8, KVH, page, hd)
    pt = i32([[0, 1], [2, 3], [4, -7], [5, 6], [7, 7]])
    spt = i32([[0], [1], [2], [3], [4]])
    layers = kv4_layers(bufs, pt, page, KVH, hd, [(1.0, 1.0)])
    s16 = [e3.make_kv_layer(src, src, spt, 8, page, 1, KVH, hd, e3.E3_BF16)]
    lens = i32([0, 30, 14, 3, 0])
    expect = {0: (e3.E3_DEV_ERR_CAPACITY, 0), 1: (e3.E3_DEV_ERR_CAPACITY, 30), 2: (e3.E3_DEV_ERR_CAPACITY, 18),
              3: (0, 3), 4: (e3.E3_DEV_ERR_NONFINITE, 4)}
    for b, (flag, after) in expect.items():
        n = [0] * B
        n[b] = {0: 5, 3: -2}.get(b, 4)
        nxt, err = torch.zeros_like(lens), err_word()
        for t in bufs:
            t.zero_()
        e3.kv4_append(layers, s16, B, R, None, i32(n), 0, lens, nxt, err)
        torch.cuda.synchronize()
        assert int(err.item()) == flag, b
        assert int(nxt[b]) == after and host(nxt).tolist()[:b] == host(lens).tolist()[:b]
        c = host(bufs[0])[0, :, 0]
        if b in (0, 1, 3):
            assert not c.any()
        if b == 2:  # the rows on the good page are written
            assert c[4, 14:].any() and not c[:4].any() and not c[5:].any()
        if b == 4:
            x = host(src[4, 0, :4]).astype(np.float64)
            assert np.array_equal(c[7, :4], kv4_ref.quantize(x, 1.0)[0])
    with_bad = i32([0, 0, 0, 0, 4])
    dst, err = torch.zeros_like(src), err_word()
    e3.kv4_read(layers, [e3.make_kv_layer(dst, dst.clone(), spt, 8, page, 1, KVH, hd, e3.E3_BF16)], B, 3, None, with_bad, err)
    torch.cuda.synchronize()
    assert int(err.item()) == e3.E3_DEV_ERR_CAPACITY and not host(dst).any()


# -------------------------------------------------------------------- attention

def attn_inputs(seed, B, R, H, KVH, hd, lens, page, tail_page=None, units=(1.0, 1.0), spread=1.0):
    rng = np.random.default_rng(seed)
    pt, n = synth.page_table(seed, [max(p, 1) for p in lens], page)
    q4 = []
    for w in range(2):  # every slot holds something, beyond a request's length too: NaN scales
        c = rng.integers(0, 256, (n, KVH, page, hd // 2)).astype(np.uint8)
        e = rng.integers(44, 60, (n, KVH, page, hd // 16)).astype(np.uint8)
        q4.append((c, e))
    for b, p in enumerate(lens):
        for t in range(p, (p + page - 1) // page * page):
            for w in range(2):
                q4[w][1][pt[b, t // page], :, t % page] = 127
    tp = tail_page or page
    nt = (R + tp - 1) // tp
    tpt = rng.permutation(B * nt).reshape(B, nt).astype(np.int32)
    tail = [synth.to_bf16_f32(rng.normal(size=(B * nt, KVH, tp, hd)).astype(np.float32)) for _ in range(2)]
    Q = synth.to_bf16_f32((spread * rng.normal(size=(B, R, H, hd))).astype(np.float32))
    see = np.stack([ancestors(random_tree(rng, R, 6)[0]) for _ in range(B)])
    return dict(B=B, R=R, H=H, KVH=KVH, hd=hd, lens=lens, page=page, pt=pt, n=n, q4=q4, tp=tp, tpt=tpt, tail=tail, Q=Q,
                see=see, units=units)


def attn_call(d, max_kv_len=None, flags=0, ws=None, out=None, stream=None, err=None, dev=None):
    """Runs tree_verify_attn4; `dev` keeps device copies between calls."""
    if dev is None:
        dev = {}
    if not dev:
        dev.update(Q=to_dev(d["Q"], torch.bfloat16), pt=i32(d["pt"]), tpt=i32(d["tpt"]), lens=i32(d["lens"]),
                   mask=mask_of(d["see"]), tail=[to_dev(t, torch.bfloat16) for t in d["tail"]],
                   q4=[[to_dev(a) for a in w] for w in d["q4"]])
    B, R, H, KVH, hd = (d[k] for k in ("B", "R", "H", "KVH", "hd"))
    kv = e3.make_kv4_layer(dev["q4"][0][0], dev["q4"][1][0], dev["q4"][0][1], dev["q4"][1][1], dev["pt"], d["n"], d["page"],
                           d["pt"].shape[1], KVH, hd, *d["units"], flags)
    tail = e3.make_kv_layer(*dev["tail"], dev["tpt"], dev["tail"][0].shape[0], d["tp"], d["tpt"].shape[1], KVH, hd, e3.E3_BF16)
    mx = max(d["lens"]) if max_kv_len is None else max_kv_len
    need = e3.eagle3_verify4_workspace_bytes(B, R, H, KVH, hd, mx)
    if ws is None:
        ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    O, lse = out or (torch.full((B, R, H, hd), 55.0, dtype=torch.bfloat16, device="cuda"),
                     torch.full((B, R, H), 55.0, device="cuda"))
    err = err_word() if err is None else err
    e3.tree_verify_attn4(dev["Q"], kv, tail, dev["lens"], dev["mask"], B, R, H, mx, 1 / math.sqrt(hd), O, lse, err, ws, need,
                         stream=stream)
    return O, lse, err


def attn_check(d, O, lse, requests=None):
    O, lse = host(O).astype(np.float64), host(lse).astype(np.float64)
    page, tp, R = d["page"], d["tp"], d["R"]
    for b in requests if requests is not None else range(d["B"]):
        t, j = np.arange(d["lens"][b]), np.arange(R)
        k, v = (kv4_ref.dequantize(d["q4"][w][0][d["pt"][b, t // page], :, t % page],
                                   d["q4"][w][1][d["pt"][b, t // page], :, t % page], d["units"][w]) for w in range(2))
        tk, tv = (d["tail"][w][d["tpt"][b, j // tp], :, j % tp].astype(np.float64) for w in range(2))
        o, l, mag, big = kv4_ref.attend(d["Q"][b].astype(np.float64), k, v, tk, tv, d["see"][b], 1 / math.sqrt(d["hd"]))
        ds = 2.0 ** -18 * (big + 1.0)
        dead = ~d["see"][b].any(-1) if d["lens"][b] == 0 else np.zeros(R, bool)
        assert np.all(O[b][dead] == 0) and np.all(np.isneginf(lse[b][dead]))
        live = ~dead
        assert np.all(np.abs(lse[b][live] - l[live]) <= (ds + 2.0 ** -21 * np.abs(l))[live]), np.abs(lse[b][live] - l[live]).max()
        # weights off by a relative w leave o + e, |e| <= w mag; the output is then rounded by at
        # most half a step OF THAT VALUE: |e| + 2^-8 (|o| + |e|).  An fp16 weight below 2^-14 is
        # off by half its subnormal step, 2^-25, whatever its size: with the largest weight at
        # 2^7 or more that is 2^-32 of it per prefix key
        G = d["H"] // d["KVH"]
        tiny = 2.0 ** -32 * np.repeat(np.abs(v).sum(0), G, 0)[None] if len(t) else 0.0
        e = (2.0 ** -8 + 2 * ds[..., None]) * mag + tiny
        tol = e + 2.0 ** -8 * (np.abs(o) + e) + 2.0 ** -126
        bad = np.abs(O[b] - o)[live] - tol[live]
        assert np.all(bad <= 0), (b, bad.max())


ATTN = [
    # B, R, H, KVH, hd, page, lens
    (1, 1, 32, 8, 128, 64, [1]),
    (2, 1, 4, 4, 64, 16, [0, 17]),                 # no prefix: the node alone
    (1, 1, 32, 8, 128, 64, [2049]),
    (3, 1, 32, 8, 128, 16, [15, 16, 700]),
    (1, 61, 32, 8, 128, 64, [2048]),
    (2, 15, 4, 4, 64, 16, [128, 1025]),
    (3, 33, 8, 1, 128, 64, [63, 64, 65]),
    (2, 5, 6, 2, 64, 32, [300, 0]),
    (1, 200, 8, 8, 128, 16, [130]),
    (2, 256, 4, 1, 128, 128, [129, 1000]),
    (2, 17, 5, 5, 128, 64, [511, 1]),
    (1, 8, 64, 8, 128, 64, [12345]),
    (4, 61, 32, 8, 128, 64, [512, 0, 1777, 128]),
    (2, 64, 40, 8, 128, 64, [640, 90]),            # five query heads per KV head
    (2, 3, 48, 1, 64, 48, [97, 48]),
    (1, 2, 16, 1, 128, 16, [40000]),
]


@pytest.mark.parametrize("case", ATTN)
def test_verify_attn4(case):
    B, R, H, KVH, hd, page, lens = case
    d = attn_inputs(R * 7 + H + hd + lens[0], B, R, H, KVH, hd, lens, page)
    O, lse, err = attn_call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    attn_check(d, O, lse)


def test_verify_attn4_repeats_bit_for_bit_and_with_looser_bounds():
    """Same inputs, same bits, on dirty workspaces and with the prefix promise; a larger length bound stays right."""
    d = attn_inputs(11, 3, 20, 16, 4, 128, [100, 1500, 64], 64)
    dev = {}
    O, lse, _ = attn_call(d, dev=dev)
    O2, lse2, _ = attn_call(d, dev=dev, flags=e3.E3_KV_PREFIX_STABLE)
    torch.cuda.synchronize()
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    O3, lse3, err = attn_call(d, dev=dev, max_kv_len=d["pt"].shape[1] * 64)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    attn_check(d, O3, lse3)


@pytest.mark.parametrize("R,G,P", [(1, 4, 300), (33, 4, 300), (61, 4, 1000), (200, 1, 64)])
def test_verify_attn4_units_and_sharp_rows(R, G, P):
    """Per-layer units, rows of very different magnitudes, scores that move the softmax base far."""
    d = attn_inputs(R + P, 2, R, 2 * G, 2, 128, [P, P // 2], 64, units=(2.0 ** -5, 2.0 ** 3), spread=4.0)
    rng = np.random.default_rng(1)
    d["Q"] *= np.exp2(rng.integers(-20, 5, d["Q"].shape[:3]))[..., None].astype(np.float32)
    d["Q"][0, 0] = 0.0
    d["Q"] = synth.to_bf16_f32(d["Q"])
    O, lse, err = attn_call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    attn_check(d, O, lse)


@pytest.mark.parametrize("R,H", [(5, 4), (40, 16), (80, 8)])
def test_verify_attn4_masked_places_hold_anything(R, H):
    """NaN and Inf in tail slots: rows that do not see them are exact, rows that see a bad V get NaN;
    rows that see nothing (no prefix, empty mask) give 0 and -Inf; slots beyond R do not matter."""
    d = attn_inputs(R, 2, R, H, 2, 128, [0, 130], 64)
    d["see"][0, 2:4] = False
    clean = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in d.items()}
    clean["tail"] = [t.copy() for t in d["tail"]]
    bad = R - 1
    d["see"][:, :bad, bad] = False
    clean["see"] = d["see"]
    tp = d["tp"]
    for b in range(2):
        d["tail"][0][d["tpt"][b, bad // tp], :, bad % tp] = np.nan
        d["tail"][1][d["tpt"][b, bad // tp], :, bad % tp, 7] = np.inf if b else np.nan
    if R % tp:
        for w in range(2):
            d["tail"][w][d["tpt"][:, -1], :, R % tp:] = np.nan
    O, lse, err = attn_call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    O, lse = host(O), host(lse)
    assert np.isnan(O[:, bad]).all()
    O[:, bad], lse[:, bad] = 0.0, 0.0
    clean["see"] = clean["see"].copy()
    clean["see"][:, bad] = False
    clean["see"][:, bad, 0] = True
    ref_rows = np.arange(R) != bad
    # compare every other row (the bad row is replaced by a finite stand-in that is not looked at)
    O2, lse2, _ = attn_call(clean)
    torch.cuda.synchronize()
    O[:, bad], lse[:, bad] = host(O2)[:, bad], host(lse2)[:, bad]
    attn_check(clean, torch.from_numpy(O), torch.from_numpy(lse))
    assert ref_rows.sum() == R - 1
    # only V of the seen node is bad: the row's lse stays that of its scores
    d2 = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in d.items()}
    d2["tail"] = [clean["tail"][0].copy(), d["tail"][1].copy()]
    O3, lse3, _ = attn_call(d2)
    torch.cuda.synchronize()
    assert np.isnan(host(O3)[:, bad]).all() and np.isfinite(host(lse3)[:, bad]).all()


def test_verify_attn4_capacity_is_flagged():
    """A length beyond the bound, a negative one: outputs of that request untouched, the others exact; a bad page id is flagged."""
    for lens_now, R in (([5000, 64, 100], 3), ([-1, 64, 100], 40)):
        d = attn_inputs(77 + R, 3, R, 8, 2, 128, [64, 64, 100], 64)
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


def test_verify_attn4_on_streams_and_in_a_graph():
    """Two calls on two streams with scratch of their own; a captured call replayed on changed inputs."""
    a = attn_inputs(1, 2, 40, 16, 4, 128, [900, 33], 64)
    b = attn_inputs(2, 2, 1, 16, 4, 128, [700, 1000], 64)
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
    need = e3.eagle3_verify4_workspace_bytes(2, 40, 16, 4, 128, 900)
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


@pytest.mark.parametrize("R,H", [(20, 16), (40, 16)])
def test_verify_attn4_wait_that_runs_out(R, H):
    """The self-test bit on the tail: a tile that never comes ends the call with the error word set,
    after the waits' bound, and leaves nothing behind that the next call on the same buffers meets."""
    d = attn_inputs(R, 2, R, H, 4, 128, [900, 300], 64)
    dev = {}
    need = e3.eagle3_verify4_workspace_bytes(2, R, H, 4, 128, 900)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    attn_call(d, dev=dev, ws=ws)
    torch.cuda.synchronize()
    make = e3.make_kv_layer
    try:
        e3.make_kv_layer = lambda *a: make(*a, flags=e3.E3_KV_SELFTEST_STALL)
        _, _, err = attn_call(d, dev=dev, ws=ws)
    finally:
        e3.make_kv_layer = make
    torch.cuda.synchronize()
    assert int(err.item()) == e3.E3_DEV_ERR_TIMEOUT
    O, lse, err = attn_call(d, dev=dev, ws=ws)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    attn_check(d, O, lse)


@pytest.mark.parametrize("B,R,H,KVH,hd,most", [
    (48, 17, 32, 8, 128, 300),    # 68 rows a KV head: parts of one tile and of several
    (48, 17, 32, 8, 128, 40),     # no more than the nodes' tile and one of the prefix
    (40, 61, 32, 8, 128, 900),    # 244 rows
    (24, 200, 16, 4, 128, 500),   # several row tiles, two tiles of nodes
    (64, 3, 16, 4, 64, 700),
])
def test_verify_attn4_many_requests_of_differing_length(B, R, H, KVH, hd, most):
    """Shares that end inside a request, hold several, or begin behind one's last tile."""
    rng = np.random.default_rng(B + R + most)
    lens = [int(x) for x in np.where(rng.random(B) < 0.15, 0, rng.integers(1, most + 1, B))]
    lens[1] = 12 * most
    d = attn_inputs(R, B, R, H, KVH, hd, lens, 16)
    dev = {}
    O, lse, err = attn_call(d, dev=dev)
    O2, lse2, _ = attn_call(d, dev=dev, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    assert not torch.any(O == 55.0) and not torch.any(lse == 55.0)
    attn_check(d, O, lse, requests=[0, 1, 2, B // 2, B - 1])


@pytest.mark.parametrize("R,H,KVH", [(9, 8, 4), (21, 16, 4), (40, 16, 4)])
def test_a_round_in_a_graph(R, H, KVH):
    """The round's calls captured once and replayed on other inputs: bit for bit the eager calls' results."""
    B, hd, V, D, page, lens = 2, 128, 2048, 4, 16, [130, 77]
    rng = np.random.default_rng(R)
    mp = 16
    pt = i32(rng.permutation(B * mp).reshape(B, mp))
    width = (H + 2 * KVH) * hd

    def values(seed):
        r = np.random.default_rng(seed)
        par = np.stack([random_tree(r, R, D)[0] for _ in range(B)]).astype(np.int32)
        path = np.zeros((B, D + 1), np.int32)
        acc = np.zeros(B, np.int32)
        for b in range(B):
            u, up = R - 1, []
            while u > 0:
                up.append(u)
                u = int(par[b, u])
            acc[b] = len(up)
            path[b, 1:len(up) + 1] = up[::-1]
        return dict(qkv=to_dev(synth.to_bf16_f32(r.normal(size=(B * R, width)).astype(np.float32)), torch.bfloat16),
                    pos=i32(r.integers(0, 9000, (B, R))), mask=mask_of(np.stack([ancestors(q) for q in par])),
                    par=i32(par), tok=i32(r.integers(0, V, (B, R))), path=i32(path), acc=i32(acc),
                    z=to_dev(r.normal(size=(B * R, V)).astype(np.float32) * 4.0))

    def state():
        r = np.random.default_rng(5)
        s = dict(q4=[torch.from_numpy(r.integers(0, 256, (B * mp, KVH, page, hd // 2), dtype=np.uint8)).cuda() for _ in range(2)],
                 e4=[torch.from_numpy(r.integers(40, 60, (B * mp, KVH, page, hd // 16), dtype=np.uint8)).cuda() for _ in range(2)],
                 tail=[torch.zeros((B, KVH, 64, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2)], tpt=i32([[0], [1]]),
                 lens=i32(lens), Q=torch.zeros((B, R, H, hd), dtype=torch.bfloat16, device="cuda"),
                 counts=torch.zeros(B * V, dtype=torch.int16, device="cuda"), err=err_word(),
                 back=[torch.zeros((B * mp, KVH, page, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2)],
                 out=torch.zeros((B * R, V), device="cuda"), mx=torch.zeros(B * R, device="cuda"),
                 Qs=torch.zeros(B * R, dtype=torch.int64, device="cuda"), am=torch.zeros(B * R, dtype=torch.int32, device="cuda"),
                 O=torch.zeros((B, R, H, hd), dtype=torch.bfloat16, device="cuda"), lse=torch.zeros((B, R, H), device="cuda"))
        s["need"] = e3.eagle3_verify4_workspace_bytes(B, R, H, KVH, hd, mp * page)
        s["ws"] = torch.full((s["need"],), 255, dtype=torch.uint8, device="cuda")
        return s

    rope = e3.eagle3_rope_init(hd, 10000.0)
    temp = torch.full((B * R,), 0.8, device="cuda")
    pen = to_dev(np.array([[1.2, 0.1, 0.1], [1.5, 0.0, 0.3]], np.float32))

    def run(s, x):
        kv = e3.make_kv4_layer(*s["q4"], *s["e4"], pt, B * mp, page, mp, KVH, hd)
        tail = e3.make_kv_layer(*s["tail"], s["tpt"], B, 64, 1, KVH, hd, e3.E3_BF16)
        back = e3.make_kv_layer(*s["back"], pt, B * mp, page, mp, KVH, hd, e3.E3_BF16)
        e3.tree_qkv_append(x["qkv"], width, B, R, None, H, None, None, 0.0, rope, x["pos"], s["Q"], tail, None, s["err"])
        e3.tree_verify_attn4(s["Q"], kv, tail, s["lens"], x["mask"], B, R, H, mp * page, hd ** -0.5, s["O"], s["lse"], s["err"],
                             s["ws"], s["need"])
        e3.tree_logits_process(x["z"], B, R, V, temp, s["counts"], x["tok"], x["par"], pen, None, None, 0, None, None, 0, s["out"],
                               s["mx"], s["Qs"], s["am"], s["err"])
        e3.kv4_append([kv], [tail], B, D + 1, x["path"], x["acc"], 1, s["lens"], s["lens"], s["err"])
        e3.token_counts_add(s["counts"], V, B, x["path"], x["acc"], 1, D + 1)
        e3.kv4_read([kv], [back], B, mp * page, None, s["lens"], s["err"])

    eager, held = state(), state()
    x = values(0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # (first calls set kernel attributes)
        run(state(), x)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(held, x)
    for seed in (1, 2):
        y = values(seed)
        for k in x:
            x[k].copy_(y[k])
        run(eager, y)
        g.replay()
        torch.cuda.synchronize()
        assert int(eager["err"].item()) == 0 and int(held["err"].item()) == 0
        for k in ("lens", "Q", "counts", "out", "mx", "Qs", "am", "O", "lse"):
            assert torch.equal(eager[k], held[k]), k
        for k in ("q4", "e4", "tail", "back"):
            assert all(torch.equal(a, b) for a, b in zip(eager[k], held[k])), k


# ----------------------------------------------------------------------- logits

LOGITS = [
    # B, R, V, n_bias, counts, paths, pen, grammar, in_place
    (1, 1, 1, 0, True, False, True, False, False),
    (2, 15, 1000, 3, True, True, True, True, False),
    (1, 61, 128256, 37, True, True, True, True, False),
    (2, 7, 50257, 300, True, True, True, True, True),   # odd rows: no 16-byte alignment
    (3, 4, 32003, 0, False, True, True, False, False),
    (1, 9, 4097, 1024, True, True, False, True, True),
    (2, 3, 33000, 0, False, False, False, False, False),
    (1, 2, 150001, 5, True, True, True, True, False),
    (1, 3, 200000, 5, True, True, True, True, True),
    (1, 2, 262148, 9, True, True, True, True, False),   # wider than a cluster holds
    (40, 8, 2052, 2, True, True, True, True, False),    # many rows
    (8, 40, 40000, 3, True, True, True, True, False),   # several rows to a cluster of several CTAs
    (4, 23, 128256, 300, True, True, True, True, True),
]


@pytest.mark.parametrize("case", LOGITS)
def test_logits_process(case):
    B, R, V, nb, has_counts, has_paths, has_pen, grammar, in_place = case
    rng = np.random.default_rng(V + nb)
    z = (rng.normal(size=(B * R, V)) * 3).astype(np.float32)
    z[:, rng.integers(0, V, 5)] = 0.0
    if V > 100:
        z[0, 50:60] = -np.inf  # ruled out before
    temps = np.repeat(rng.choice([0.0, 0.5, 1.0, 1.3], B), R).astype(np.float32)
    counts = None
    if has_counts:
        counts = np.zeros((B, V), np.uint16)
        hit = rng.integers(0, V, (B, min(V, 400)))
        for b in range(B):
            np.add.at(counts[b], hit[b], 1)
            counts[b, rng.integers(0, V, 200)] |= 32768
            counts[b, int(rng.integers(0, V))] = 32767
    par, tok, paths = None, None, [[] for _ in range(B * R)]
    if has_paths:
        par = np.stack([random_tree(rng, R, 6)[0] for _ in range(B)]).astype(np.int32)
        tok = rng.integers(0, min(V, 50), (B, R)).astype(np.int32)  # repeats along a path
        if R > 3:
            tok[0, 2], tok[0, 3] = -5, V + 3
        paths = []
        for b in range(B):
            for i in range(R):
                u, p = i, []
                while u > 0:
                    p.append(int(tok[b, u]))
                    u = par[b, u]
                paths.append(p)
    pen = np.stack([1 + rng.random(B), rng.random(B), rng.random(B) - 0.3], 1).astype(np.float32) if has_pen else None
    bt = rng.integers(-2, V + 2, (B, nb)).astype(np.int32)
    bv = (rng.normal(size=(B, nb)) * 4).astype(np.float32)
    if nb > 2:
        bt[:, 1], bt[:, 2] = bt[:, 0], bt[:, 0]  # one token three times
        bv[0, -1] = -np.inf
    W = (V + 31) // 32
    words = rng.integers(0, 2 ** 32, (5, W)).astype(np.uint32) if grammar else None
    arow = rng.integers(-1, 6, (B, R)).astype(np.int32) if grammar else None
    if grammar:
        words[:, 0] |= 1
    dz = to_dev(z)
    out = dz if in_place else torch.full((B * R, V), 9.0, device="cuda")
    mx, Qs = torch.zeros(B * R, device="cuda"), torch.zeros(B * R, dtype=torch.int64, device="cuda")
    am, err = torch.zeros(B * R, dtype=torch.int32, device="cuda"), err_word()
    dev = lambda a, v=None: None if a is None else to_dev(a if v is None else a.view(v))  # noqa: E731
    keep = [dev(temps), dev(counts, np.int16), dev(tok), dev(par), dev(pen), dev(bt) if nb else None, dev(bv) if nb else None,
            dev(words, np.int32), dev(arow)]
    e3.tree_logits_process(dz, B, R, V, keep[0], keep[1], keep[2], keep[3], keep[4], keep[5], keep[6], nb, keep[7], keep[8],
                           5 if grammar else 0, out, mx, Qs, am, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    got = host(out)
    for row in range(B * R):
        b, i = divmod(row, R)
        ok = None
        if grammar and 0 <= arow[b, i] < 5:
            v = np.arange(V)
            ok = ((words[arow[b, i], v // 32] >> (v % 32).astype(np.uint32)) & 1).astype(bool)
        want = kv4_ref.process(z[row], None if counts is None else counts[b], paths[row], None if pen is None else pen[b],
                               bt[b], bv[b], ok)
        assert np.array_equal(got[row], want), (row, np.nonzero(got[row] != want)[0][:5])
        ref = oracle.row_stats(ruled_out(want)[None], temps[row:row + 1])
        assert mx[row].item() == ref[0][0] and int(am[row]) == int(ref[2][0])
        assert int(Qs[row]) & (2 ** 64 - 1) == int(ref[1][0])


def test_logits_rows_without_a_token_and_bad_values():
    """A fully masked row, a NaN, an Inf: flagged rows carry the statistics that spec_accept reports;
    a NaN in a masked place does nothing."""
    R, V = 4, 500
    z = torch.randn((R, V), device="cuda")
    z[1, 7] = float("nan")
    z[2, 9] = float("nan")
    z[3, 11] = float("inf")
    allow = torch.full((R, 16), -1, dtype=torch.int32, device="cuda")
    allow[0] = 0
    allow[1, 0] &= ~(1 << 7)
    out = torch.zeros_like(z)
    mx, Qs = torch.zeros(R, device="cuda"), torch.ones(R, dtype=torch.int64, device="cuda")
    am, err = torch.zeros(R, dtype=torch.int32, device="cuda"), err_word()
    e3.tree_logits_process(z, 1, R, V, torch.ones(R, device="cuda"), None, None, None, None, None, None, 0, allow, None, R, out,
                           mx, Qs, am, err)
    torch.cuda.synchronize()
    assert int(err.item()) == e3.E3_DEV_ERR_MASKED | e3.E3_DEV_ERR_NONFINITE
    assert host(am).tolist()[0] == -1 and host(am)[1] >= 0 and host(am).tolist()[2:] == [-1, -1]
    assert host(Qs)[[0, 2, 3]].tolist() == [0, 0, 0] and np.isnan(host(mx)[[0, 2, 3]]).all()
    ref = oracle.row_stats(ruled_out(host(out)[1:2]), np.ones(1, np.float32))
    assert mx[1].item() == ref[0][0] and int(Qs[1]) == int(ref[1][0]) and torch.isneginf(out[1, 7])
    par, tok = i32([[-1, 0, 0, 1]]), i32([[1, 2, 3, 4]])
    acc, path, ot = (torch.zeros((1, n), dtype=torch.int32, device="cuda") for n in (1, 4, 4))
    st, u = i32([0]), torch.zeros((1, R), dtype=torch.int32, device="cuda")
    e3.spec_accept(tok, par, 1, R, 3, out, mx, Qs, am, V, torch.ones(1, device="cuda"), u, u, e3.E3_ACCEPT_TREE_DET, acc, path,
                   ot, st)
    torch.cuda.synchronize()
    assert int(st.item()) == e3.E3_DEV_ERR_NONFINITE


@pytest.mark.parametrize("V,B,n", [(1000, 3, 7), (33, 3, 40), (128256, 2, 3001)])
def test_token_counts(V, B, n):
    """Repeated tokens, neighbours in one word, saturation, skipped ids; the prompt's bit."""
    rng = np.random.default_rng(V)
    size = (B * V + 1) // 2 * 2
    base = np.zeros(size, np.uint16)
    base[5] = 32766
    tok = rng.integers(-1, min(V, 60) + 1, (B, n)).astype(np.int32)
    tok[0, :4] = 5
    cnt = rng.integers(0, n, B).astype(np.int32)
    cnt[0] = n
    d = to_dev(base.view(np.int16))
    e3.token_counts_add(d, V, B, i32(tok), i32(cnt), 1, n)
    e3.token_counts_add(d, V, B, i32(tok[:, ::-1].copy()), i32(np.minimum(cnt, 3)), 0, n, prompt=True)
    torch.cuda.synchronize()
    want = base.astype(np.int64)
    for b in range(B):
        for t in tok[b, :min(n, cnt[b] + 1)]:
            if 0 <= t < V:
                want[b * V + t] = min(want[b * V + t] + 1, 32767)
    for b in range(B):
        for t in tok[b, ::-1][:min(cnt[b], 3)]:
            if 0 <= t < V:
                want[b * V + t] |= 32768
    assert np.array_equal(host(d).view(np.uint16), want.astype(np.uint16))


# --------------------------------------------------------------------- together

def test_a_verify_pass_over_a_4bit_cache():
    """Two rounds as a server runs them: qkv rows -> tail and Q, attention over the 4-bit prefix and
    the tail, LM head, penalties and a grammar, accept, the accepted path committed in 4 bits, counts.
    Each round is compared with the plain forms on what the caches hold by then."""
    B, R, D, H, KVH, hd, page, V, P = 2, 15, 3, 4, 2, 64, 16, 256, [37, 0]
    seed = 31
    rng = np.random.default_rng(seed)
    maxp = 8
    pt = rng.permutation(B * maxp).reshape(B, maxp).astype(np.int32)
    bufs = kv4_buffers(1, B * maxp, KVH, page, hd)
    dpt = i32(pt)
    layers = kv4_layers(bufs, dpt, page, KVH, hd, [(1.0, 1.0)])
    tpt = i32(np.arange(B)[:, None])
    tk = torch.zeros((B, KVH, 64, hd), dtype=torch.bfloat16, device="cuda")
    tv = torch.zeros_like(tk)
    tail = e3.make_kv_layer(tk, tv, tpt, B, 64, 1, KVH, hd, e3.E3_BF16)
    rope = e3.eagle3_rope_init(hd, 10000.0)
    kvl, err = i32([0, 0]), err_word()
    Wlm, W64 = bits(V, H * hd, seed=8)
    # the prompt's rows enter through the tail, which is a bf16 cache like any other
    width = (H + 2 * KVH) * hd
    prompt, _ = bits(B * 40, width, seed=9)
    Q0 = torch.zeros((B, 40, H, hd), dtype=torch.bfloat16, device="cuda")
    e3.tree_qkv_append(prompt, width, B, 40, i32(P), H, None, None, 0.0, rope, i32(np.tile(np.arange(40), (B, 1))), Q0, tail, None, err)
    e3.kv4_append(layers, [tail], B, 40, None, i32(P), 0, kvl, kvl, err)
    counts = torch.zeros(B * V, dtype=torch.int16, device="cuda")
    lens = list(P)
    for rnd in range(2):
        par = np.stack([random_tree(rng, R, D)[0] for _ in range(B)]).astype(np.int32)
        tok = rng.integers(0, V, (B, R)).astype(np.int32)
        see = np.stack([ancestors(p) for p in par])
        depth = see.sum(-1) - 1
        pos = np.array(lens)[:, None] + depth
        qkv, q64 = bits(B * R, width, seed=100 + rnd)
        Q = torch.zeros((B, R, H, hd), dtype=torch.bfloat16, device="cuda")
        e3.tree_qkv_append(qkv, width, B, R, None, H, None, None, 0.0, rope, i32(pos), Q, tail, None, err)
        mx_len = 60
        O = torch.zeros((B, R, H, hd), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((B, R, H), device="cuda")
        need = e3.eagle3_verify4_workspace_bytes(B, R, H, KVH, hd, mx_len)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        e3.tree_verify_attn4(Q, layers[0], tail, kvl, mask_of(see), B, R, H, mx_len, hd ** -0.5, O, lse, err, ws, need)
        temp = torch.tensor([1.0, 0.0], device="cuda")
        trow = temp.repeat_interleave(R)
        z = torch.zeros((B * R, V), device="cuda")
        mx, Qs = torch.zeros(B * R, device="cuda"), torch.zeros(B * R, dtype=torch.int64, device="cuda")
        am = torch.zeros(B * R, dtype=torch.int32, device="cuda")
        e3.lmhead_logits(O, Wlm, B * R, H * hd, V, trow, z, mx, Qs, am, err, e3.E3_BF16)
        raw = host(z)
        pen = np.array([[1.2, 0.1, 0.1], [1.5, 0.0, 0.3]], np.float32)
        words = rng.integers(0, 2 ** 32, (1, V // 32)).astype(np.uint32)
        arow = np.where(rng.random((B, R)) < 0.5, 0, -1).astype(np.int32)
        held = host(counts).view(np.uint16).reshape(B, V).copy()
        e3.tree_logits_process(z, B, R, V, trow, counts, i32(tok), i32(par), to_dev(pen), None, None, 0,
                               to_dev(words.view(np.int32)), i32(arow), 1, z, mx, Qs, am, err)
        ua, ub = synth.uniforms(seed + rnd, synth.PURPOSE_ACCEPT, B, R), synth.uniforms(seed + rnd, synth.PURPOSE_BONUS, B, R)
        acc, path, ot = i32([0] * B), i32(np.zeros((B, D + 1))), i32(np.zeros((B, D + 1)))
        st = i32([0] * B)
        e3.spec_accept(i32(tok), i32(par), B, R, D, z, mx, Qs, am, V, temp, to_dev(ua.view(np.int32)), to_dev(ub.view(np.int32)),
                       e3.E3_ACCEPT_TREE_DET, acc, path, ot, st)
        e3.kv4_append(layers, [tail], B, D + 1, path, acc, 1, kvl, kvl, err)
        e3.token_counts_add(counts, V, B, ot, acc, 1, D + 1)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and not host(st).any()
        # attention on what the caches held, from the device's own bytes
        d = dict(B=B, R=R, H=H, KVH=KVH, hd=hd, lens=lens, page=page, pt=pt, tp=64, tpt=host(tpt), see=see, Q=host(Q),
                 tail=[host(tk), host(tv)], units=(1.0, 1.0), q4=[(host(bufs[w])[0], host(bufs[2 + w])[0]) for w in range(2)])
        attn_check(d, O, lse)
        zz = host(z)
        v = np.arange(V)
        ok = ((words[0, v // 32] >> (v % 32).astype(np.uint32)) & 1).astype(bool)
        for b in range(B):
            for i in range(R):
                p, u = [], i
                while u > 0:
                    p.append(tok[b, u])
                    u = par[b, u]
                want = kv4_ref.process(raw[b * R + i], held[b], p, pen[b], [], [], ok if arow[b, i] == 0 else None)
                assert np.array_equal(zz[b * R + i], want)
            a, pa = int(acc[b]), host(path)[b]
            ref = oracle.accept(dict(tok=tok[b], parent=par[b]), ruled_out(zz[b * R:(b + 1) * R]), float(temp[b]), ua[b], ub[b], D)
            assert a == ref[0] and pa[:a + 1].tolist() == list(ref[1][:a + 1])
            for j in range(a + 1):  # the committed rows are the tail's rows of the path, quantized
                t = lens[b] + j
                for w, src in enumerate((tk, tv)):
                    c, e = kv4_ref.quantize(host(src)[b, :, pa[j]].astype(np.float64), 1.0)
                    assert np.array_equal(host(bufs[w])[0, pt[b, t // page], :, t % page], c)
                    assert np.array_equal(host(bufs[2 + w])[0, pt[b, t // page], :, t % page], e)
                held[b, host(ot)[b, j]] += 1
            lens[b] += a + 1
        assert host(kvl).tolist() == lens
        assert np.array_equal(host(counts).view(np.uint16).reshape(B, V), held)
