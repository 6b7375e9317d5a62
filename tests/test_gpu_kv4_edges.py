"""The ends of the stated ranges of the verify pass over a 4-bit cache, against 64-bit forms.

Tolerances of the attention, from the arithmetic (check_attn):
  scores   fp32 sums of 128 products: 2^-18 of the largest sum |q||k| scale
  weights  of prefix keys rounded to fp16, half a step 2^-11; of tree nodes to bf16, 2^-8, or
           up to 32 query rows per KV head and for heads of 64 to two bf16 parts, 2^-16;
           each twice the score error on top
  output   half a bf16 step of the value reached, 2^-8 of it
"""
import math

import numpy as np
import pytest
import torch

import kv4_ref
import oracle
from eagle_speculative_decoding_round_gb300 import synth
from gpu_util import host, to_dev
from test_gpu_kv4 import ATTN, attn_inputs, err_word, i32, mask_of, ruled_out

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from eagle_speculative_decoding_round_gb300 import eagle3 as e3


def attn(d, scale):
    B, R, H, KVH, hd = (d[k] for k in ("B", "R", "H", "KVH", "hd"))
    q4 = [[to_dev(a) for a in w] for w in d["q4"]]
    tail16 = [to_dev(t, torch.bfloat16) for t in d["tail"]]
    pt, tpt, lens, mask, Q = i32(d["pt"]), i32(d["tpt"]), i32(d["lens"]), mask_of(d["see"]), to_dev(d["Q"], torch.bfloat16)
    kv = e3.make_kv4_layer(q4[0][0], q4[1][0], q4[0][1], q4[1][1], pt, d["n"], d["page"], d["pt"].shape[1], KVH, hd, *d["units"])
    tail = e3.make_kv_layer(*tail16, tpt, tail16[0].shape[0], d["tp"], d["tpt"].shape[1], KVH, hd, e3.E3_BF16)
    need = e3.eagle3_verify4_workspace_bytes(B, R, H, KVH, hd, max(d["lens"]))
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    O, lse, err = torch.full((B, R, H, hd), 55.0, dtype=torch.bfloat16, device="cuda"), torch.full((B, R, H), 55.0, device="cuda"), err_word()
    e3.tree_verify_attn4(Q, kv, tail, lens, mask, B, R, H, max(d["lens"]), scale, O, lse, err, ws, need)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return host(O).astype(np.float64), host(lse).astype(np.float64)


def parts(d, b):
    """K, V of request b's prefix and tail in 64 bits."""
    t, j = np.arange(d["lens"][b]), np.arange(d["R"])
    k, v = (kv4_ref.dequantize(d["q4"][w][0][d["pt"][b, t // d["page"]], :, t % d["page"]],
                               d["q4"][w][1][d["pt"][b, t // d["page"]], :, t % d["page"]], d["units"][w]) for w in range(2))
    tk, tv = (d["tail"][w][d["tpt"][b, j // d["tp"]], :, j % d["tp"]].astype(np.float64) for w in range(2))
    return k, v, tk, tv


def check_attn(d, O, lse, scale, skip=(), node=2.0 ** -8):
    for b in range(d["B"]):
        k, v, tk, tv = parts(d, b)
        Q, see, R = d["Q"][b].astype(np.float64), d["see"][b], d["R"]
        o, l, _, big = kv4_ref.attend(Q, k, v, tk, tv, see, scale)
        # sum p |v| over the prefix alone and over the nodes alone
        _, _, mag_p, _ = kv4_ref.attend(Q, k, np.abs(v), tk, 0 * tv, see, scale)
        _, _, mag_n, _ = kv4_ref.attend(Q, k, 0 * v, tk, np.abs(tv), see, scale)
        ds = 2.0 ** -18 * (big + 1.0)
        for i in range(R):
            if (b, i) in skip:
                continue
            if not d["lens"][b] and not see[i].any():
                assert np.all(O[b, i] == 0) and np.all(np.isneginf(lse[b, i])), (b, i)
                continue
            assert np.all(np.abs(lse[b, i] - l[i]) <= ds[i] + 2.0 ** -21 * np.abs(l[i])), (b, i, lse[b, i], l[i])
            # an fp16 weight below 2^-14 is off by up to 2^-25 whatever its size: 2^-32 of the row's largest
            G = d["H"] // d["KVH"]
            tiny = 2.0 ** -32 * np.repeat(np.abs(v).sum(0), G, 0) if len(v) else 0.0
            w = 2 * ds[i][:, None]
            e = (2.0 ** -11 + w) * mag_p[i] + (node + w) * mag_n[i] + tiny
            tol = e + 2.0 ** -8 * (np.abs(o[i]) + e) + 2.0 ** -126
            bad = np.abs(O[b, i] - o[i]) - tol
            assert np.all(bad <= 0), (b, i, bad.max(), np.abs(o[i]).max())


SIDES = [(5, 1, 128), (5, 4, 128), (40, 4, 128), (70, 4, 128), (5, 1, 64), (5, 4, 64), (40, 4, 64)]  # R, query heads per KV head, head_dim


@pytest.mark.parametrize("R,G,hd", SIDES)
@pytest.mark.parametrize("v_unit,top", [(2.0 ** -60, 2.0 ** 97), (2.0 ** -30, 2.0 ** 92), (2.0 ** 60, 2.0 ** 97), (2.0 ** 60, 1.0), (2.0 ** -60, 1.0)])
def test_large_nodes_beside_a_prefix_of_any_unit(R, G, hd, v_unit, top):
    """Nodes' V up to 2^100 with the ends of v_unit: finite and right, also for rows that see the prefix alone."""
    d = attn_inputs(R + G, 2, R, 2 * G, 2, hd, [150, 0], 16, units=(1.0, v_unit))
    d["tail"][1] = synth.to_bf16_f32(d["tail"][1] * np.float32(top))  # |N(0, 1)| < 2^3
    d["see"][:, R - 2] = False
    scale = 1 / math.sqrt(hd)
    check_attn(d, *attn(d, scale), scale)


@pytest.mark.parametrize("R,G,hd", SIDES)
def test_score_factors_that_leave_the_range(R, G, hd):
    """The smallest k_unit with a small scale, rows of zeros among them: every score is nothing, the keys weigh alike."""
    d = attn_inputs(R + G + 1, 2, R, 2 * G, 2, hd, [150, 3], 16, units=(2.0 ** -60, 1.0))
    d["Q"][:, ::3] = 0.0
    check_attn(d, *attn(d, 1e-9), 1e-9)


@pytest.mark.parametrize("R,G,hd", SIDES)
def test_score_factors_beyond_the_range(R, G, hd):
    """The largest k_unit with a scale of 1e29 and keys of zeros: every score is 0."""
    d = attn_inputs(R + G + 5, 2, R, 2 * G, 2, hd, [150, 3], 16, units=(2.0 ** 60, 1.0))
    d["q4"][0][0][:] = 0
    d["tail"][0][:] = 0.0
    check_attn(d, *attn(d, 1e29), 1e29)


@pytest.mark.parametrize("R,G,hd", SIDES)
@pytest.mark.parametrize("nodes", [2.0 ** 60, 1.0])
def test_small_queries_against_large_keys(R, G, hd, nodes):
    """Rows of Q from 2^-72 to 2^-62 against keys of 2^60: scores of ordinary size."""
    d = attn_inputs(R + G + 2, 2, R, 2 * G, 2, hd, [150, 20], 16, units=(2.0 ** 60, 1.0))
    at = np.random.default_rng(R).integers(-72, -61, d["Q"].shape[:3])
    d["Q"] = synth.to_bf16_f32(d["Q"] * np.exp2(at)[..., None].astype(np.float32))
    d["Q"][0, 0] = 0.0
    d["tail"][0] = synth.to_bf16_f32(d["tail"][0] * np.float32(nodes))
    check_attn(d, *attn(d, 1.0), 1.0)


@pytest.mark.parametrize("R,G,hd", SIDES)
def test_the_largest_nodes_against_the_smallest_queries(R, G, hd):
    """Nodes' K up to 2^127 with Q of 2^-121: scores of ordinary size.  (Values of Q below 2^-125 are left out.)"""
    d = attn_inputs(R + G + 3, 2, R, 2 * G, 2, hd, [0, 20], 16)
    q = d["Q"] * np.float32(2.0 ** -121)
    d["Q"] = synth.to_bf16_f32(np.where(np.abs(q) < 2.0 ** -125, 0.0, q).astype(np.float32))
    d["tail"][0] = synth.to_bf16_f32(d["tail"][0] * np.float32(2.0 ** 124))
    check_attn(d, *attn(d, 0.1), 0.1)


@pytest.mark.parametrize("R,G,hd", SIDES)
def test_a_bad_query_row_that_sees_nothing(R, G, hd):
    """NaN or Inf in a row of Q: 0 and -Inf where it sees no key, NaN where it sees one; other rows are not touched."""
    d = attn_inputs(R + G + 4, 2, R, 2 * G, 2, hd, [0, 20], 16)
    d["see"][0, 1:3] = False
    good = d["Q"].copy()
    bad = [(0, 1), (0, 2), (0, 3), (1, 4)]
    d["Q"][0, 1], d["Q"][0, 2, :, 7], d["Q"][0, 3, :, 5], d["Q"][1, 4, :, 3] = np.nan, np.inf, np.nan, np.nan
    O, lse = attn(d, 0.1)
    assert np.all(O[0, 1:3] == 0) and np.all(np.isneginf(lse[0, 1:3]))
    for b, i in bad[2:]:
        assert np.all(np.isnan(O[b, i])) and np.all(np.isnan(lse[b, i]))
    d["Q"] = good
    check_attn(d, O, lse, 0.1, skip=bad)


def logits_call(z, V, temp, counts=None, tok=None, par=None, pen=None, bias=None, allow=None, arow=None, B=1):
    """(out, row_max, row_Q, row_argmax, error word) of tree_logits_process on host arrays, as host arrays."""
    rows = len(z)
    dev = lambda a, v=None: None if a is None else to_dev(a if v is None else a.view(v))  # noqa: E731
    dz = to_dev(z)
    out, mx = torch.full((rows, V), 9.0, device="cuda"), torch.zeros(rows, device="cuda")
    Q, am = torch.ones(rows, dtype=torch.int64, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
    err = err_word()
    bt, bv = bias if bias is not None else (None, None)
    keep = [dev(temp), dev(counts, np.int16), dev(tok), dev(par), dev(pen), dev(bt), dev(bv), dev(allow, np.int32), dev(arow)]
    e3.tree_logits_process(dz, B, rows // B, V, *keep[:5], keep[5], keep[6], 0 if bt is None else bt.shape[1], keep[7], keep[8],
                           0 if allow is None else len(allow), out, mx, Q, am, err)
    torch.cuda.synchronize()
    return host(out), host(mx), host(Q).view(np.uint64), host(am), int(err.item())


def check_row(want, temp, mx, Q, am, row):
    """Statistics of the processed row `want` against the oracle."""
    ref = oracle.row_stats(ruled_out(want)[None], np.float32([temp]))
    assert mx == ref[0][0] and am == int(ref[2][0]) and int(Q) == int(ref[1][0]), row


@pytest.mark.parametrize("V", [500, 40000, 262148])
def test_paths_beyond_the_depth_limit_are_flagged(V):
    """A chain of nodes: rows whose path has at most 16 beside the root are exact, deeper ones carry the statistics of a bad row."""
    R = 20
    rng = np.random.default_rng(V)
    z = rng.normal(size=(R, V)).astype(np.float32)
    par = np.arange(-1, R - 1, dtype=np.int32)[None]
    tok = rng.integers(0, V, (1, R)).astype(np.int32)
    pen = np.float32([[1.3, 0.2, 0.1]])
    out, mx, Q, am, err = logits_call(z, V, np.ones(R, np.float32), None, tok, par, pen)
    for i in range(17):
        want = kv4_ref.process(z[i], None, [int(t) for t in tok[0, 1:i + 1]], pen[0], [], [], None)
        assert np.array_equal(out[i], want)
        check_row(want, 1.0, mx[i], Q[i], am[i], i)
    assert err == e3.E3_DEV_ERR_CAPACITY
    assert np.isnan(mx[17:]).all() and not Q[17:].any() and np.all(am[17:] == -1)


@pytest.mark.parametrize("V", [1000, 40000, 262148])
def test_rows_that_a_small_temperature_carries_past_the_range(V):
    """Finite logits whose quotient by the temperature overflows, either way: flagged, whichever kernel runs."""
    z = np.full((3, V), -1000.0, np.float32)
    z[1, 5] = 1000.0
    z[2] = -np.float32(1.5)
    out, mx, Q, am, err = logits_call(z, V, np.float32([1e-37, 1e-37, 0.5]))
    assert np.array_equal(out, z)
    assert err == e3.E3_DEV_ERR_NONFINITE
    assert np.isnan(mx[:2]).all() and not Q[:2].any() and np.all(am[:2] == -1)
    check_row(z[2], 0.5, mx[2], Q[2], am[2], 2)


@pytest.mark.parametrize("in_place", [False, True])
def test_append_of_the_largest_row_count(in_place):
    """n_rows + n_add past 31 bits is more rows than there are: flagged, the request as it was."""
    KVH, hd, page = 1, 64, 16
    src = torch.ones((2, KVH, page, hd), dtype=torch.bfloat16, device="cuda")
    bufs = [torch.zeros((2, KVH, page, w), dtype=torch.uint8, device="cuda") for w in (hd // 2, hd // 2, hd // 16, hd // 16)]
    pt = i32([[0], [1]])
    l4 = e3.make_kv4_layer(*bufs, pt, 2, page, 1, KVH, hd)
    l16 = e3.make_kv_layer(src, src, pt, 2, page, 1, KVH, hd, e3.E3_BF16)
    lens, n, err = i32([3, 2]), i32([2 ** 31 - 1, 3]), err_word()
    nxt = lens if in_place else torch.zeros_like(lens)
    e3.kv4_append([l4], [l16], 2, 4, None, n, 1, lens, nxt, err)
    torch.cuda.synchronize()
    assert int(err.item()) == e3.E3_DEV_ERR_CAPACITY
    assert host(nxt).tolist() == [3, 6] and not host(bufs[0])[0].any() and host(bufs[0])[1].any()


@pytest.mark.parametrize("first,n", [(30, 3), (-1, 2), (2 ** 31 - 2, 4), (0, 33)])
def test_read_beyond_the_pages_leaves_the_request(first, n):
    """Rows that the 4-bit cache's pages do not hold: flagged, nothing of the request is written; the other request is."""
    KVH, hd, page = 1, 64, 16
    bufs = [torch.full((4, KVH, page, w), 0x38 if w == hd // 16 else 0x22, dtype=torch.uint8, device="cuda")
            for w in (hd // 2, hd // 2, hd // 16, hd // 16)]
    l4 = e3.make_kv4_layer(*bufs, i32([[0, 1], [2, 3]]), 4, page, 2, KVH, hd)
    table = [i32([[0, 1], [2, 3]]), i32([[0, 1, 2], [3, 4, 5]])]
    l4.page_table = table[0].data_ptr()
    back = [torch.full((6, KVH, page, hd), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    l16 = e3.make_kv_layer(*back, table[1], 6, page, 3, KVH, hd, e3.E3_BF16)
    starts, count, err = i32([first, 31]), i32([n, 1]), err_word()
    e3.kv4_read([l4], [l16], 2, 40, starts, count, err)
    torch.cuda.synchronize()
    assert int(err.item()) == e3.E3_DEV_ERR_CAPACITY
    for t in back:
        assert torch.all(t[:3] == 9.0) and torch.all(t[3, 0, 0] == 1.0) and torch.all(t[3, 0, 1:] == 9.0) and torch.all(t[4:] == 9.0)


@pytest.mark.parametrize("rot,inter", [(64, False), (64, True), (24, False), (24, True)])
def test_rotation_close_to_whole_quarter_turns(rot, inter):
    """fp32 rows, unit vectors: cosine and sine are good to 2^-22 of themselves however close to 0 they are (half a
    step of the reduced phase, 2^-25, and sincospif's one unit in the last place, 2^-23)."""
    hd, R = 64, 96
    rng = np.random.default_rng(3)
    pos = np.concatenate([[0, 1, 355, 710, 103993, 104348, 208341, 312689, -355, 2 ** 31 - 1, -2 ** 31], rng.integers(-2 ** 31, 2 ** 31, R - 11)])
    rope = e3.eagle3_rope_init(rot, 10000.0, interleaved=inter)
    x = np.zeros((R, 3, hd), np.float32)
    low, high = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if inter else (np.arange(rot // 2), rot // 2 + np.arange(rot // 2))
    x[:, :2, low] = 1.0
    qkv = to_dev(x.reshape(R, -1))
    K = torch.zeros((6, 1, 16, hd), device="cuda")
    V, Q = torch.zeros_like(K), torch.zeros((R, hd), device="cuda")
    pt, dpos, err = i32([list(range(6))]), i32(pos.astype(np.int64).astype(np.int32)), err_word()
    kv = e3.make_kv_layer(K, V, pt, 6, 16, 6, 1, hd, e3.E3_F32)
    e3.tree_qkv_append(qkv, 3 * hd, 1, R, None, 1, None, None, 0.0, rope, dpos, Q, kv, None, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    hq, hk = host(Q), host(K)
    for r in range(R):
        for i in range(rot // 2):
            ph = rope.turns[i] * int(pos[r]) % 2 ** 64
            quarter, rest = (ph + 2 ** 61) >> 62, ((ph + 2 ** 61) & (2 ** 62 - 1)) - 2 ** 61
            c, s = math.cos(rest * math.pi * 2.0 ** -63), math.sin(rest * math.pi * 2.0 ** -63)
            c, s = [(c, s), (-s, c), (-c, -s), (s, -c)][quarter & 3]
            for got in (hq[r], hk[r // 16, 0, r % 16]):
                assert abs(got[low[i]] - c) <= 2.0 ** -22 * abs(c) and abs(got[high[i]] - s) <= 2.0 ** -22 * abs(s), (r, i)


@pytest.mark.parametrize("case", [c for c in ATTN if c[1] <= 64])
def test_attention_with_a_bound_for_each_part(case):
    """Prefix weights are good to fp16, the nodes' to bf16: the bounds of check_attn, which holds each part to its own."""
    B, R, H, KVH, hd, page, lens = case
    d = attn_inputs(R * 7 + H + hd + lens[0] + 1, B, R, H, KVH, hd, lens, page)
    scale = 1 / math.sqrt(hd)
    check_attn(d, *attn(d, scale), scale)


@pytest.mark.parametrize("V", [1500, 2052, 40000, 40003, 262148])
@pytest.mark.parametrize("seen", ["all", "list full", "list passed", "first part"])
def test_more_seen_tokens_than_the_list_holds(V, seen):
    """A part's list holds 1024 seen tokens: all seen, just as many, one more, and one part full while the others
    are not; path and bias tokens among the seen ones and beside them."""
    R, rng = 5, np.random.default_rng(V + len(seen))
    counts = np.zeros((1, V), np.uint16)
    hit = {"all": np.arange(V), "list full": np.arange(1024), "list passed": np.arange(1025),
           "first part": np.concatenate([np.arange(min(V, 5000)), rng.integers(0, V, 20)])}[seen]
    counts[0, hit] = rng.integers(1, 4, len(hit))
    counts[0, hit[::3]] |= 32768
    counts[0, hit[::5]] = 32768
    z = (rng.normal(size=(R, V)) * 3).astype(np.float32)
    par = np.int32([[-1, 0, 1, 1, 2]])
    tok = np.int32([[3, 7, V - 1, 7, 1023]])
    pen = np.float32([[1.3, 0.2, 0.1]])
    bt = np.int32([[7, 1023, 7, V - 1, V // 2, 1100]])
    bv = (rng.normal(size=bt.shape) * 2).astype(np.float32)
    out, mx, Q, am, err = logits_call(z, V, np.full(R, 0.7, np.float32), counts, tok, par, pen, (bt, bv))
    assert err == 0
    for i in range(R):
        path, u = [], i
        while u > 0:
            path.append(int(tok[0, u]))
            u = par[0, u]
        want = kv4_ref.process(z[i], counts[0], path, pen[0], bt[0], bv[0], None)
        assert np.array_equal(out[i], want), (i, np.nonzero(out[i] != want)[0][:5])
        check_row(want, 0.7, mx[i], Q[i], am[i], i)


@pytest.mark.parametrize("V", [2052, 40000, 40003, 128256, 262148])
def test_flagged_rows_of_wide_vocabularies(V):
    """A masked row, a NaN in a masked place, a NaN in the last token, an Inf in the middle, a good row."""
    R, W = 5, (V + 31) // 32
    z = np.random.default_rng(V).normal(size=(R, V)).astype(np.float32)
    z[1, V // 3] = np.nan
    z[2, V - 1] = np.nan
    z[3, V // 2] = np.inf
    allow = np.full((R, W), 0xFFFFFFFF, np.uint32)
    allow[0] = 0
    allow[1, V // 3 // 32] &= ~np.uint32(1 << (V // 3 % 32))
    out, mx, Q, am, err = logits_call(z, V, np.ones(R, np.float32), allow=allow, arow=np.arange(R, dtype=np.int32)[None])
    assert err == e3.E3_DEV_ERR_MASKED | e3.E3_DEV_ERR_NONFINITE
    assert np.isnan(mx[[0, 2, 3]]).all() and not Q[[0, 2, 3]].any() and np.all(am[[0, 2, 3]] == -1)
    assert np.all(np.isneginf(out[0]))
    for i in (1, 4):
        want = z[i].copy()
        if i == 1:
            want[V // 3] = -np.inf
        assert np.array_equal(out[i], want)
        check_row(want, 1.0, mx[i], Q[i], am[i], i)


@pytest.mark.parametrize("R,G,hd", [(15, 1, 64), (40, 4, 64), (8, 4, 128), (3, 2, 128)])
def test_rows_of_nodes_alone(R, G, hd):
    """No prefix: the nodes' weights are the row, and their two parts hold 2^-16 of it."""
    d = attn_inputs(R + G + 6, 3, R, 2 * G, 2, hd, [0, 0, 0], 16)
    scale = 1 / math.sqrt(hd)
    check_attn(d, *attn(d, scale), scale, node=2.0 ** -16)
