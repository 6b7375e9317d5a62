"""GPU parity of tree_verify_attn8 at the edges of its inputs: bad rows of Q, rows of very uneven values, long sums.

Tolerances as in test_gpu_kv8, with what a test adds to them derived beside it.
"""
import numpy as np
import pytest
import torch

import kv8_ref
from eagle_speculative_decoding_round_gb300 import synth
from gpu_util import host

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from eagle_speculative_decoding_round_gb300 import eagle3 as e3
    from test_gpu_kv8 import attn_call, attn_check, attn_inputs


@pytest.mark.parametrize("R,G,hd", [(5, 1, 128), (8, 4, 128), (33, 1, 128), (40, 1, 128), (40, 4, 128), (70, 2, 128), (200, 1, 128), (6, 2, 64), (90, 4, 64)])
def test_verify_attn8_bad_query_row_that_sees_nothing(R, G, hd):
    """NaN or Inf in a row of Q: 0 and -Inf where it sees no key, NaN where it sees one; other rows are not touched.  Both kernels, both
    widths of the larger one's tile, with a prefix and without."""
    d = attn_inputs(R + G + 4, 2, R, 2 * G, 2, hd, [0, 20], 16, 16)
    d["see"][0, 1:3] = False
    good = d["Q"].copy()
    bad = [(0, 1), (0, 2), (0, 3), (1, 4)]
    d["Q"][0, 1], d["Q"][0, 2, :, 7], d["Q"][0, 3, :, 5], d["Q"][1, 4, :, 3] = np.nan, np.inf, np.nan, np.nan
    O, lse, err = attn_call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    O, lse = host(O).copy(), host(lse).copy()
    assert np.all(O[0, 1:3] == 0) and np.all(np.isneginf(lse[0, 1:3]))
    for b, i in bad[2:]:
        assert np.all(np.isnan(O[b, i])) and np.all(np.isnan(lse[b, i]))
    d["Q"] = good
    O2, lse2, _ = attn_call(d)
    torch.cuda.synchronize()
    for b, i in bad[2:]:
        O[b, i], lse[b, i] = host(O2)[b, i], host(lse2)[b, i]
    attn_check(d, torch.from_numpy(O), torch.from_numpy(lse))


def long_inputs(seed, B, R, H, KVH, hd, lens, page=64, n=5, late=False):
    """Prefixes of any length over n pages that the tables name again and again; V of one sign, so that nothing of what a sum
    loses is lost in cancellation.  late: the pages one after another, with ever larger scores."""
    rng = np.random.default_rng(seed)
    d = attn_inputs(seed, B, R, H, KVH, hd, [1] * B, page, 16, spread=0.5)
    k = (rng.integers(0x20, 0x38, (n, KVH, page, hd)) + 128 * rng.integers(0, 2, (n, KVH, page, hd))).astype(np.uint8)
    v = rng.integers(0x38, 0x40, (n, KVH, page, hd)).astype(np.uint8)
    exps = [rng.integers(-1, 2, (n, KVH, page // 16)).astype(np.int8) for _ in range(2)]
    m = -(-max(lens) // page)
    at = np.arange(m)[None] + np.arange(B)[:, None]
    pt = np.minimum(np.arange(m) * n // m, n - 1)[None].repeat(B, 0) if late else at % n
    if late:  # K along Q's rows, which are positive, from page to page
        d["Q"] = np.abs(d["Q"])
        k = (rng.integers(0x28, 0x30, (n, KVH, page, hd)) + 128 * (np.arange(n) < n // 2)[:, None, None, None]).astype(np.uint8)
        exps[0] = np.broadcast_to(np.abs(np.arange(n) - n // 2)[:, None, None] // 2, exps[0].shape).astype(np.int8).copy()
    d.update(lens=list(lens), n=n, pt=pt.astype(np.int32), kv=[(k, exps[0]), (v, exps[1])], tail=[d["tail"][0], np.abs(d["tail"][1])])
    return d


def check_long(d, O, lse, adds, heads, rows):
    """64-bit softmax over the pages' slots, each counted as often as a row sees it, and the nodes.  `adds(keys)` bounds the
    errors of the values' and of the weights' sums, relative, which join the tolerances of test_gpu_kv8."""
    O, lse = host(O).astype(np.float64), host(lse).astype(np.float64)
    page, R, G, scale = d["page"], d["R"], d["H"] // d["KVH"], 1 / np.sqrt(d["hd"])
    for b in range(d["B"]):
        keys = d["lens"][b]
        full, rest = divmod(keys, page)
        count = np.bincount(d["pt"][b, :full], minlength=d["n"])[:, None] * np.ones(page)
        if rest:
            count[d["pt"][b, full], :rest] += 1
        j = np.arange(R)
        lost_o, lost_l = adds(keys)
        for h in heads:
            k, v = (kv8_ref.decode(c[:, h // G], np.repeat(e[:, h // G].astype(np.float64), d["block"], -1)[..., None]).reshape(-1, d["hd"])
                    for c, e in d["kv"])
            tk, tv = (t[d["tpt"][b, j // page], h // G, j % page].astype(np.float64) for t in d["tail"])
            k, v = np.concatenate([k, tk]), np.concatenate([v, tv])
            for r in rows:
                q = d["Q"][b, r, h].astype(np.float64)
                c = np.concatenate([count.ravel(), d["see"][b, r].astype(float)])
                s, big = k @ q * scale, (np.abs(k) @ np.abs(q) * scale)[c > 0].max()
                m = s[c > 0].max()
                p = c * np.exp(s - m)
                z = p.sum()
                o, l = p @ v / z, m + np.log(z)
                ds = 2.0 ** -18 * (big + 1.0)
                assert abs(lse[b, r, h] - l) <= ds + lost_l + 2.0 ** -21 * abs(l), (b, r, h, lse[b, r, h] - l)
                e = (2.0 ** -8 + 2 * ds + lost_o + lost_l) * o
                bad = np.abs(O[b, r, h] - o) - (e + 2.0 ** -8 * (o + e))
                assert np.all(bad <= 0), (b, r, h, (np.abs(O[b, r, h] - o) / o).max())


def adds_tc(keys):
    """32768 keys at most in tensor memory, 16 a product, each cutting the sum off up to four times by at most a unit 2^-23;
    the weights' sum in steps of 64 keys; then fp32 sums of these."""
    n = min(keys, 32768)
    return (n / 4 + keys / 32768) * 2.0 ** -23, (n / 64 + keys / 32768) * 2.0 ** -24


@pytest.mark.parametrize("B,R,H,KVH,lens,late", [
    (1, 33, 152, 152, [1 << 20], False), (1, 200, 152, 152, [1 << 22], False),     # a part of every CTA; both widths of the tile
    (1, 33, 152, 152, [100001], True), (1, 150, 152, 152, [70000], True),          # late maxima over what has left tensor memory
    (2, 61, 32, 8, [2000000, 1300011], False),                                     # parts that begin and end inside a prefix
    (3, 40, 160, 80, [33000, 0, 90000], False)])
def test_verify_attn8_many_rows_long_sums(B, R, H, KVH, lens, late):
    d = long_inputs(R + H, B, R, H, KVH, 128, lens, late=late)
    O, lse, err = attn_call(d)
    O2, lse2, _ = attn_call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(O, O2) and torch.equal(lse, lse2)
    check_long(d, O, lse, adds_tc, heads=(0, H // 3, H - 1), rows=(0, R // 2, R - 1))


def adds_granules(keys):
    """The same in the granule kernel; a lane sums its two keys of 16 one after another."""
    n = min(keys, 32768)
    return (n / 4 + keys / 32768) * 2.0 ** -23, (n / 8 + keys / 32768) * 2.0 ** -24


@pytest.mark.parametrize("B,R,H,KVH,hd,lens,late", [
    (1, 1, 1824, 1824, 128, [1 << 20], False), (1, 16, 1216, 1216, 128, [1 << 20], False),     # a part of every warp
    (1, 1, 2432, 2432, 64, [1 << 20], False), (1, 40, 304, 304, 64, [1 << 20], False),
    (1, 1, 1824, 1824, 128, [100001], True), (1, 9, 1216, 1216, 128, [70000], True), (1, 2, 2432, 2432, 64, [100000], True),
    (2, 5, 480, 80, 128, [1000000, 777777], False), (3, 3, 800, 400, 64, [400000, 0, 290000], False)])  # parts that begin and end inside
def test_verify_attn8_few_rows_long_sums(B, R, H, KVH, hd, lens, late):
    d = long_inputs(R + H, B, R, H, KVH, hd, lens, late=late)
    O, lse, err = attn_call(d)
    O2, lse2, _ = attn_call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(O, O2) and torch.equal(lse, lse2)
    check_long(d, O, lse, adds_granules, heads=(0, H // 3, H - 1), rows=sorted({0, R // 2, R - 1}))


@pytest.mark.parametrize("top", [1.0, 1.75, 1.7578125, 1.9921875])
@pytest.mark.parametrize("R,G", [(40, 1), (40, 4), (6, 4)])
def test_verify_attn8_rows_of_uneven_values(R, G, top):
    """Q and the nodes' K with one large dim and the others far below it, each against keys, or queries, that are large in the
    others.  With more than 32 rows Q's values below 2^-9 of their row's largest are off by up to 2^-17 of it, the nodes' K
    below 2^-8 of theirs by 2^-16: times what they meet, that joins the scores' error.  Q's others from 2^-9 on are exact."""
    P, hd = 150, 128
    for f in (6, 7, 8, 9, 10, 12, 14):
        d = attn_inputs(R + f, 1, R, 2 * G, 2, hd, [P], 64, 16)
        rng = np.random.default_rng(f)
        q = rng.uniform(1.0, 1.99, d["Q"].shape) * 2.0 ** -f
        q[..., 0] = top
        d["Q"] = synth.to_bf16_f32(q.astype(np.float32))
        d["kv"][0][0][..., 0] = 0                                    # (K's codes positive, none in Q's large dim)
        d["kv"][0][0][..., 1:] = np.minimum(d["kv"][0][0][..., 1:] & 0x7F, 0x70)
        d["kv"][0][1][:] = f - 10
        tk = rng.uniform(-1.99, 1.99, d["tail"][0].shape) * 2.0 ** -f
        tk[..., 1] = top
        d["tail"][0] = synth.to_bf16_f32(tk.astype(np.float32))
        O, lse, err = attn_call(d)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        O, lse = host(O).astype(np.float64), host(lse).astype(np.float64)
        t, j, scale = np.arange(P), np.arange(R), 1 / np.sqrt(hd)
        pg = d["pt"][0, t // 64]
        k, v = (kv8_ref.decode(d["kv"][w][0][pg, :, t % 64], d["kv"][w][1][pg, :, t % 64 // 16].astype(np.float64)[..., None])
                for w in range(2))
        k, v = (np.concatenate([a, n[d["tpt"][0, j // 64], :, j % 64].astype(np.float64)]) for a, n in zip((k, v), d["tail"]))
        many = R * G > 32
        for h in range(2 * G):
            q, kh, vh = d["Q"][0, :, h].astype(np.float64), k[:, h // G], v[:, h // G]
            seen = np.concatenate([np.ones((R, P), bool), d["see"][0]], 1)
            qm, km = np.abs(q).max(1, keepdims=True), np.abs(kh).max(1, keepdims=True)
            eq = np.where(many & (np.abs(q) < 2.0 ** -9 * qm), 2.0 ** -17 * qm, 0.0)
            ek = np.where(many & (np.abs(kh) < 2.0 ** -8 * km) & (np.arange(P + R) >= P)[:, None], 2.0 ** -16 * km, 0.0)
            s = np.where(seen, q @ kh.T * scale, -np.inf)
            big = np.where(seen, np.abs(q) @ np.abs(kh).T * scale, 0.0).max(1)
            off = np.where(seen, (eq @ np.abs(kh).T + (np.abs(q) + eq) @ ek.T) * scale, 0.0).max(1)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            z = p.sum(1, keepdims=True)
            o, mag, l = p @ vh / z, p @ np.abs(vh) / z, (m + np.log(z))[:, 0]
            ds = 2.0 ** -18 * (big + 1.0) + off
            assert np.all(np.abs(lse[0, :, h] - l) <= ds + 2.0 ** -21 * np.abs(l)), (f, h, (np.abs(lse[0, :, h] - l) / ds).max())
            grow = np.expm1(2 * ds)[:, None]  # (the scores' error is not small against 1 everywhere)
            codes = np.abs(vh[:P]) * 2.0 ** (d["kv"][1][1].max() - d["kv"][1][1][pg, h // G, t % 64 // 16].astype(np.float64))[:, None]
            e = (2.0 ** -8 + grow) * mag + 2.0 ** -32 * codes.sum(0)[None]
            bad = np.abs(O[0, :, h] - o) - (e + 2.0 ** -8 * (np.abs(o) + e))
            assert np.all(bad <= 0), (f, h, bad.max())


@pytest.mark.parametrize("R,G,hd,page", [(6, 4, 128, 64), (40, 1, 128, 16), (40, 4, 128, 64), (70, 2, 128, 16), (200, 1, 128, 64), (256, 2, 128, 128),
                                         (90, 2, 64, 64)])
def test_verify_attn8_nodes_with_scores_of_minus_inf(R, G, hd, page):
    """-Inf in nodes' K where Q is positive: those nodes weigh 0, a row that sees no other key gets 0 and -Inf.  +Inf, a NaN: rows
    that see such a node get NaN, the others are exact.  Both kernels, both widths of the larger one's tile."""
    d = attn_inputs(R + G, 3, R, 2 * G, 2, hd, [0, 20, 300], page, 16)
    d["Q"] = np.abs(d["Q"])
    gone = np.zeros((3, R), bool)
    gone[0, :2], gone[1, [0, R // 2, R - 1]], gone[2] = True, True, np.arange(R) % 3 == 0
    d["see"][0, 2] = False
    d["see"][0, 2, :2] = True                          # (what it sees is gone)
    for b in range(3):
        for j in np.flatnonzero(gone[b]):
            d["tail"][0][d["tpt"][b, j // page], :, j % page, (5 * j) % hd] = -np.inf
    O, lse, err = attn_call(d)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    want = dict(d, see=d["see"] & ~gone[:, None], tail=[np.where(np.isinf(d["tail"][0]), 0.0, d["tail"][0]), d["tail"][1]])
    attn_check(want, O, lse)
    assert not want["see"][0, :3].any() and torch.all(O[0, :3] == 0)
    j = R - 2  # one node more, with scores that are no numbers' neighbours
    for value in (np.inf, np.nan):
        d["tail"][0][d["tpt"][2, j // page], :, j % page, 7] = value
        O2, lse2, _ = attn_call(d)
        torch.cuda.synchronize()
        see = torch.from_numpy(d["see"][2, :, j]).cuda()
        assert torch.isnan(O2[2][see]).all() and torch.isnan(lse2[2][see]).all() and see.any()
        assert torch.equal(O2[2][~see], O[2][~see]) and torch.equal(O2[:2], O[:2])


@pytest.mark.parametrize("R,KVH", [(33, 152), (140, 152), (1, 1824), (9, 1216)])
@pytest.mark.parametrize("P", [32640, 32768, 32769, 65536, 65600])
def test_verify_attn8_long_sums_borders(R, KVH, P):
    """Prefixes that end where the sums leave the accumulators, with the nodes behind: a fold before a tile of nodes, none, one more.
    The same call in a graph that was captured on a short prefix."""
    d = long_inputs(R + P, 1, R, KVH, KVH, 128, [P])
    dev = {}
    O, lse, err = attn_call(d, dev=dev)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    adds, at = adds_tc if R > 32 else adds_granules, dict(heads=(0, KVH - 1), rows=sorted({0, R - 1}))
    check_long(d, O, lse, adds, **at)
    need = e3.eagle3_verify8_workspace_bytes(1, R, KVH, KVH, 128, P)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = (torch.full_like(O, 55.0), torch.full_like(lse, 55.0))
    dev["lens"].fill_(70)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn_call(d, dev=dev, ws=ws, out=out, err=err)
    for keys in (70, P):
        dev["lens"].fill_(keys)
        g.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        check_long(dict(d, lens=[keys]), *out, adds, **at)
    assert torch.equal(out[0], O) and torch.equal(out[1], lse)
