"""A request's whole way over an 8-bit cache: its prompt's attention in two pieces, the prompt committed to the cache, then
rounds of tree attention and commits.  Each step is compared with the plain forms on what the caches hold by then; the
tolerances are those of the operators' own tests."""
import numpy as np
import pytest
import torch

import kv8_ref
import oracle
import test_gpu_kv8 as kv8_tests
import test_gpu_prompt as prompt_tests
from eagle_speculative_decoding_round_gb300 import synth
from gpu_util import host, random_tree, to_dev

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from eagle_speculative_decoding_round_gb300 import eagle3 as e3
    from test_gpu_kv4 import ancestors, bits, err_word, i32, mask_of, ruled_out


def filled(shape, value, dtype=torch.bfloat16):
    return torch.full(shape, value, dtype=dtype, device="cuda")


def committed(bufs, pt, page, block, b, T):
    """(codes [2][KVH][T][hd], exps [2][KVH][T / block]) of one request, as its pages hold them."""
    t, j = np.arange(T), np.arange(0, T, block)
    return [[host(bufs[i + w])[0][pt[b, a // page], :, a % page // s].swapaxes(0, 1).copy() for w in range(2)]
            for i, a, s in ((0, t, 1), (2, j, block))]


def commit_check(bufs, pt, page, block, was, starts, rows):
    """The pages hold what the plain append makes of `was` and of rows[b] = (K, V) [n][KVH][hd] at starts[b]."""
    for b, kv in enumerate(rows):
        T = was[b][0][0].shape[1]
        codes, exps = was[b]
        for w in range(2):
            for h in range(codes[w].shape[0]):
                kv8_ref.append(codes[w][h], exps[w][h], starts[b], kv[w][:, h], block)
        got = committed(bufs, pt, page, block, b, T)
        for w in range(2):
            assert np.array_equal(got[0][w], codes[w]) and np.array_equal(got[1][w], exps[w])


@pytest.mark.parametrize("H,KVH,hd,R,page,block,first,second", [
    (8, 2, 64, 15, 32, 16, [70, 33, 1], [40, 0, 5]), (16, 2, 128, 15, 64, 64, [130, 1, 77], [65, 129, 1])])
def test_a_prompt_and_its_rounds_over_an_8bit_cache(H, KVH, hd, R, page, block, first, second):
    B, D, V, seed = 3, 3, 256, 41 + hd
    rng = np.random.default_rng(seed)
    total = [a + b for a, b in zip(first, second)]
    width, scale = (H + 2 * KVH) * hd, hd ** -0.5
    rope, err = e3.eagle3_rope_init(hd, 10000.0), err_word()
    # the prompt: a bf16 cache of its length, read and written in two pieces
    pt, n = synth.page_table(seed, total, page)
    k, v = filled((n, KVH, page, hd), float("nan")), filled((n, KVH, page, hd), float("nan"))
    dpt = i32(pt)
    cache = e3.make_kv_layer(k, v, dpt, n, page, pt.shape[1], KVH, hd, e3.E3_BF16)
    for rows, ctx in ((first, [0] * B), (second, first)):
        most = max(rows)
        qkv, _ = bits(B * most, width, seed=seed + most)
        Q, O, lse = filled((B * most, H, hd), 0.0), filled((B * most, H, hd), 55.0), filled((B * most, H), 55.0, torch.float32)
        pos = np.array(ctx)[:, None] + np.arange(most)
        e3.tree_qkv_append(qkv, width, B, most, i32(rows), H, None, None, 0.0, rope, i32(pos), Q, cache, i32(ctx), err)
        need = e3.eagle3_prompt_workspace_bytes(B, B * most, most, H, KVH, hd, max(ctx), e3.E3_BF16)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        e3.prompt_attn(Q, None, i32(rows), cache, i32(ctx), B, B * most, most, H, max(ctx), scale, O, lse, err, ws, need)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        prompt_tests.check(dict(B=B, H=H, KVH=KVH, hd=hd, rows=rows, ctx=ctx, page=page, dt="bf16", start=np.arange(B) * most,
                                total=B * most, pt=pt, n=n, Q=host(Q), k=host(k), v=host(v)), O, lse)
    # the prompt into the 8-bit cache, with room for the rounds
    pt8, n8 = synth.page_table(seed + 1, [t + 2 * (D + 1) for t in total], page)
    bufs = kv8_tests.kv8_buffers(1, n8, KVH, page, hd, block, fill=0x31)
    dpt8, kvl = i32(pt8), i32([0] * B)
    layer = kv8_tests.kv8_layers(bufs, dpt8, page, KVH, hd, block)
    held = [-(-(t + 2 * (D + 1)) // page) * page for t in total]
    was = [committed(bufs, pt8, page, block, b, held[b]) for b in range(B)]
    e3.kv8_append(layer, [cache], B, max(total), None, i32(total), 0, kvl, kvl, err)
    torch.cuda.synchronize()
    t = [np.arange(m) for m in total]
    rows = [[host(x)[pt[b, t[b] // page], :, t[b] % page].astype(np.float64) for x in (k, v)] for b in range(B)]
    commit_check(bufs, pt8, page, block, was, [0] * B, rows)
    # rounds
    tp = 64
    tpt = np.arange(B)[:, None].astype(np.int32)
    tk, tv, dtpt = filled((B, KVH, tp, hd), 0.0), filled((B, KVH, tp, hd), 0.0), i32(tpt)
    tail = e3.make_kv_layer(tk, tv, dtpt, B, tp, 1, KVH, hd, e3.E3_BF16)
    Wlm, _ = bits(V, H * hd, seed=8)
    lens = list(total)
    for rnd in range(2):
        par = np.stack([random_tree(rng, R, D)[0] for _ in range(B)]).astype(np.int32)
        tok = rng.integers(0, V, (B, R)).astype(np.int32)
        see = np.stack([ancestors(p) for p in par])
        pos = np.array(lens)[:, None] + see.sum(-1) - 1
        qkv, _ = bits(B * R, width, seed=100 + rnd)
        Q, O, lse = filled((B, R, H, hd), 0.0), filled((B, R, H, hd), 55.0), filled((B, R, H), 55.0, torch.float32)
        e3.tree_qkv_append(qkv, width, B, R, None, H, None, None, 0.0, rope, i32(pos), Q, tail, None, err)
        need = e3.eagle3_verify8_workspace_bytes(B, R, H, KVH, hd, max(lens))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        e3.tree_verify_attn8(Q, layer[0], tail, kvl, mask_of(see), B, R, H, max(lens), scale, O, lse, err, ws, need)
        torch.cuda.synchronize()
        was = [committed(bufs, pt8, page, block, b, held[b]) for b in range(B)]
        # (the reference reads pages of one size: the tail's 64 slots stand in pages of `page`)
        per = tp // page
        tails = [host(x).reshape(B, KVH, per, page, hd).swapaxes(1, 2).reshape(B * per, KVH, page, hd) for x in (tk, tv)]
        kv8_tests.attn_check(dict(B=B, R=R, H=H, KVH=KVH, hd=hd, lens=lens, page=page, block=block, pt=pt8, see=see, Q=host(Q), tail=tails,
                                  tpt=np.arange(B * per).reshape(B, per),
                                  kv=[(host(bufs[w])[0], host(bufs[2 + w])[0]) for w in range(2)]), O, lse)
        temp = torch.tensor([1.0, 0.0, 0.7], device="cuda")
        z, mx = torch.zeros((B * R, V), device="cuda"), torch.zeros(B * R, device="cuda")
        Qs, am = torch.zeros(B * R, dtype=torch.int64, device="cuda"), i32([0] * (B * R))
        e3.lmhead_logits(O, Wlm, B * R, H * hd, V, temp.repeat_interleave(R), z, mx, Qs, am, err, e3.E3_BF16)
        ua, ub = (synth.uniforms(seed + rnd, p, B, R) for p in (synth.PURPOSE_ACCEPT, synth.PURPOSE_BONUS))
        acc, path, ot, st = i32([0] * B), i32(np.zeros((B, D + 1))), i32(np.zeros((B, D + 1))), i32([0] * B)
        e3.spec_accept(i32(tok), i32(par), B, R, D, z, mx, Qs, am, V, temp, to_dev(ua.view(np.int32)), to_dev(ub.view(np.int32)),
                       e3.E3_ACCEPT_TREE_DET, acc, path, ot, st)
        e3.kv8_append(layer, [tail], B, D + 1, path, acc, 1, kvl, kvl, err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and not host(st).any()
        rows = []
        for b in range(B):
            a, pa = int(acc[b]), host(path)[b]
            ref = oracle.accept(dict(tok=tok[b], parent=par[b]), ruled_out(host(z)[b * R:(b + 1) * R]), float(temp[b]), ua[b], ub[b], D)
            assert a == ref[0] and pa[:a + 1].tolist() == list(ref[1][:a + 1])
            rows.append([host(x)[b][:, pa[:a + 1]].swapaxes(0, 1).astype(np.float64) for x in (tk, tv)])
        commit_check(bufs, pt8, page, block, was, lens, rows)
        lens = [p + len(r[0]) for p, r in zip(lens, rows)]
        assert host(kvl).tolist() == lens


@pytest.mark.parametrize("R,H,KVH", [(1, 8, 2), (15, 8, 4), (21, 16, 4)])
def test_a_prompt_and_a_round_in_a_graph(R, H, KVH):
    """The calls of a prompt's commit and of a round captured once and replayed on other inputs and lengths: bit for bit
    the eager calls' results."""
    B, hd, D, page, block, N, mp = 2, 128, 4, 32, 16, 150, 10
    width, need_len = (H + 2 * KVH) * hd, N + D + 1
    pt = i32(np.random.default_rng(R).permutation(B * mp).reshape(B, mp))
    rope = e3.eagle3_rope_init(hd, 10000.0)

    def values(seed):
        r = np.random.default_rng(seed)
        par = np.stack([random_tree(r, R, D)[0] for _ in range(B)]).astype(np.int32)
        path, acc = np.zeros((B, D + 1), np.int32), np.zeros(B, np.int32)
        for b in range(B):
            u, up = R - 1, []
            while u > 0:
                up.append(u)
                u = int(par[b, u])
            acc[b] = len(up)
            path[b, 1:len(up) + 1] = up[::-1]
        rows = r.integers(1, N + 1, B)
        return dict(prompt=bits(B * N, width, seed=seed)[0], qkv=bits(B * R, width, seed=seed + 50)[0], rows=i32(rows),
                    ppos=i32(np.tile(np.arange(N), (B, 1))), pos=i32(rows[:, None] + np.stack([ancestors(q) for q in par]).sum(-1) - 1),
                    mask=mask_of(np.stack([ancestors(q) for q in par])), path=i32(path), acc=i32(acc))

    def state():
        s = dict(cache=[filled((B * mp, KVH, page, hd), 0.0) for _ in range(2)], tail=[filled((B, KVH, 64, hd), 0.0) for _ in range(2)],
                 bufs=kv8_tests.kv8_buffers(1, B * mp, KVH, page, hd, block), tpt=i32([[0], [1]]), lens=i32([0, 0]), none=i32([0, 0]),
                 PQ=filled((B * N, H, hd), 0.0), PO=filled((B * N, H, hd), 0.0), plse=filled((B * N, H), 0.0, torch.float32),
                 Q=filled((B, R, H, hd), 0.0), O=filled((B, R, H, hd), 0.0), lse=filled((B, R, H), 0.0, torch.float32),
                 back=[filled((B * mp, KVH, page, hd), 0.0) for _ in range(2)], err=err_word())
        s["need"] = e3.eagle3_verify8_workspace_bytes(B, R, H, KVH, hd, need_len)
        s["pneed"] = e3.eagle3_prompt_workspace_bytes(B, B * N, N, H, KVH, hd, 0, e3.E3_BF16)
        s["ws"] = torch.full((max(s["need"], s["pneed"], 16),), 255, dtype=torch.uint8, device="cuda")
        return s

    def run(s, x):
        cache = e3.make_kv_layer(*s["cache"], pt, B * mp, page, mp, KVH, hd, e3.E3_BF16)
        tail = e3.make_kv_layer(*s["tail"], s["tpt"], B, 64, 1, KVH, hd, e3.E3_BF16)
        back = e3.make_kv_layer(*s["back"], pt, B * mp, page, mp, KVH, hd, e3.E3_BF16)
        layer = kv8_tests.kv8_layers(s["bufs"], pt, page, KVH, hd, block)
        e3.tree_qkv_append(x["prompt"], width, B, N, x["rows"], H, None, None, 0.0, rope, x["ppos"], s["PQ"], cache, s["none"], s["err"])
        e3.prompt_attn(s["PQ"], None, x["rows"], cache, None, B, B * N, N, H, 0, hd ** -0.5, s["PO"], s["plse"], s["err"], s["ws"],
                       s["pneed"])
        e3.kv8_append(layer, [cache], B, N, None, x["rows"], 0, s["none"], s["lens"], s["err"])
        e3.tree_qkv_append(x["qkv"], width, B, R, None, H, None, None, 0.0, rope, x["pos"], s["Q"], tail, None, s["err"])
        e3.tree_verify_attn8(s["Q"], layer[0], tail, s["lens"], x["mask"], B, R, H, need_len, hd ** -0.5, s["O"], s["lse"], s["err"],
                             s["ws"], s["need"])
        e3.kv8_append(layer, [tail], B, D + 1, x["path"], x["acc"], 1, s["lens"], s["lens"], s["err"])
        e3.kv8_read(layer, [back], B, need_len, None, s["lens"], s["err"])

    eager, held, x = state(), state(), values(0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # (first calls set kernel attributes)
        run(state(), x)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(held, x)
    for seed in (1, 2):
        y = values(seed)
        for key in x:
            x[key].copy_(y[key])
        run(eager, y)
        g.replay()
        torch.cuda.synchronize()
        assert int(eager["err"].item()) == 0 and int(held["err"].item()) == 0
        for key in ("lens", "PQ", "PO", "plse", "Q", "O", "lse"):
            assert torch.equal(eager[key], held[key]), key
        for key in ("cache", "tail", "bufs", "back"):
            assert all(torch.equal(a, b) for a, b in zip(eager[key], held[key])), key
