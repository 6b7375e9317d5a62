"""Measured cases of the operators that bring a prompt into the target's cache and verify over a cache held in 8 bits.

  prompt  prompt_attn: causal attention of whole prompts, or of a prompt's next piece, over the paged cache; grouped heads,
          sequences of different lengths packed in one call
  kv8     kv8_append + kv8_read: rows of a 16-bit cache committed to the 8-bit cache, whose scale is one power of two for
          each block of tokens and head (rows already in a block follow when its scale grows), and read back as values
  attn8   tree_verify_attn8: tree attention whose prefix is held in 8 bits

``run`` computes the plain form in elementary torch operations, or, where ``own`` is set,
makes the calls of this repository's library.
"""
import math

import torch

own = False

E_MIN, E_MAX = -100, 120  # exponents of a block's scale
TOP = 448.0               # largest e4m3 magnitude

# query heads, KV heads, head dim of the shapes that the rounds of this repository run with
TINY, MID, LARGE = (4, 4, 64), (32, 8, 128), (64, 8, 128)


def listed():
    return [
        # one request's prompt of the round's prefix length (latency counts)
        dict(name="prompt one", op="prompt", B=1, H=32, KVH=8, hd=128, lo=2048, hi=2048, ctx=0, page=64, dt="bf16", spare=0),
        # a batch's prompts, packed
        dict(name="prompt packed", op="prompt", B=16, H=32, KVH=8, hd=128, lo=512, hi=8192, ctx=0, page=64, dt="bf16", spare=5),
        # a long document in one piece (the largest)
        dict(name="prompt long", op="prompt", B=1, H=32, KVH=8, hd=128, lo=32768, hi=32768, ctx=0, page=64, dt="bf16", spare=0),
        # the next pieces of four long prompts: few rows behind a long cached context, wide groups
        dict(name="prompt piece", op="prompt", B=4, H=64, KVH=8, hd=128, lo=100, hi=257, ctx=16384, page=64, dt="bf16", spare=0),
        # narrow heads without groups, short pages, odd lengths down to one token
        dict(name="prompt narrow", op="prompt", B=9, H=4, KVH=4, hd=64, lo=1, hi=1021, ctx=0, page=16, dt="bf16", spare=3),
        # the fp32 target's prompts
        dict(name="prompt fp32", op="prompt", B=3, H=4, KVH=4, hd=64, lo=15, hi=131, ctx=128, page=16, dt="f32", spare=0),
        # the accepted paths of a batched round, every layer: most land in a block that holds rows already
        dict(name="kv8 accepted paths", op="kv8", B=32, R=7, L=32, KVH=8, hd=128, lo=512, hi=8192, page=64, block=64, path=True),
        # two prompts compressed into the 8-bit cache, four layers
        dict(name="kv8 prompts", op="kv8", B=2, R=8191, L=4, KVH=8, hd=128, lo=0, hi=77, page=64, block=32, path=False),
        # plain decoding of a batch: one node a request
        dict(name="attn8 decode", op="attn8", B=32, R=1, H=32, KVH=8, hd=128, lo=512, hi=8192, page=64, block=64),
        # one request's 60-node tree at a moderate prefix (latency)
        dict(name="attn8 tree", op="attn8", B=1, R=61, H=32, KVH=8, hd=128, lo=2048, hi=2048, page=64, block=64),
        # batched serving: 32 requests, each with its tree
        dict(name="attn8 batch", op="attn8", B=32, R=61, H=32, KVH=8, hd=128, lo=512, hi=8192, page=64, block=64),
        # long context: one request, a small tree, fine blocks
        dict(name="attn8 long", op="attn8", B=1, R=33, H=32, KVH=8, hd=128, lo=65536, hi=65536, page=64, block=16),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "kv8", "attn8", "attn8"])
    page = rng.choice([16, 64, 64, 128])
    block = rng.choice([b for b in (16, 32, 64, 128) if page % b == 0])
    if op == "prompt":
        H, KVH, hd = rng.choice([TINY, MID, MID, LARGE, (8, 1, 128), (6, 2, 64), (5, 5, 128), (12, 4, 64)])
        B = log_int(rng, 1, 32)
        ctx = rng.choice([0, 0, rng.randint(1, 300), log_int(rng, 100, 30000)])
        hi = log_int(rng, 1, 16000)
        dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
        # bounded by the largest listed case (an fp32 target is a small one)
        while B * H * hd * hi * (ctx + hi // 2) > (2e12 if dt == "bf16" else 2e10) or B * hi * H * hd > 1.5e9 or B * (ctx + hi) * KVH * hd > 1.5e9:
            hi, ctx, B = max(1, hi * 2 // 3), ctx * 2 // 3, max(1, B - 1)
        return dict(op=op, B=B, H=H, KVH=KVH, hd=hd, lo=rng.randint(1, hi), hi=hi, ctx=ctx, page=page, dt=dt, spare=rng.choice([0, 0, 9]))
    if op == "kv8":
        path = rng.random() < 0.5
        B = log_int(rng, 1, 32)
        R = rng.randint(1, 9) if path else log_int(rng, 1, max(1, 16000 // B))
        lo = rng.randint(0, 2000)
        return dict(op=op, B=B, R=R, L=rng.randint(1, 32) if path else rng.randint(1, 4), KVH=rng.choice([1, 2, 8]),
                    hd=rng.choice([64, 128]), lo=lo, hi=lo + rng.randint(0, 3000), page=page, block=block, path=path)
    H, KVH, hd = rng.choice([TINY, MID, MID, LARGE, (8, 1, 128), (6, 2, 64), (5, 5, 128)])
    B = log_int(rng, 1, 32)
    hi = log_int(rng, 16, max(64, min(65536, 130000 // B)))
    R = rng.choice([1, 2, rng.randint(3, 16), rng.randint(17, 64), rng.randint(65, 200)])
    R = max(1, min(R, 60000 // (B * H)))
    hi = max(16, min(hi, 250000000 // (B * R * H)))
    return dict(op=op, B=B, R=R, H=H, KVH=KVH, hd=hd, lo=rng.randint(0, hi), hi=hi, page=page, block=block)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def lengths(case):
    """A length for each request: spread over [lo, hi], in no order."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [lo + (hi - lo) * ((5 * b + 3) % B) // max(1, B - 1) for b in range(B)] if B > 1 else [hi]


def contexts(case):
    """(prompt) cached keys before each request's rows."""
    return [case["ctx"] - case["ctx"] * b // (3 * case["B"]) for b in range(case["B"])]


def path_rows(case):
    """(kv8) rows that each request appends."""
    B, R = case["B"], case["R"]
    return [1 + (3 * b + 1) % R for b in range(B)] if case["path"] else [R] * B


class Inputs:
    """Seeded draws on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda")

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.g, device="cuda")

    def ints(self, hi, *shape):
        return torch.randint(hi, shape, generator=self.g, device="cuda")

    def pages(self, lens, page):
        """(page table [B][max_pages] int32, number of pages): every request's pages drawn from one shuffled pool."""
        need = [max(1, -(-n // page)) for n in lens]
        total = sum(need)
        perm = torch.randperm(total, generator=self.g, device="cuda").to(torch.int32)
        start = torch.tensor([sum(need[:b]) for b in range(len(need))], device="cuda")
        at = start[:, None] + torch.arange(max(need), device="cuda")[None]
        held = torch.arange(max(need), device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
        return torch.where(held, perm[at.clamp(max=total - 1)], 0).to(torch.int32).contiguous(), total

    def tree(self, B, R):
        """Ancestor-or-self [B][R][R] of booleans of random trees, nodes in an order with parents first."""
        parent = torch.full((B, R), -1, dtype=torch.int64, device="cuda")
        if R > 1:
            last = torch.arange(R - 1, device="cuda")
            parent[:, 1:] = torch.minimum((last * self.uniform(B, R - 1).square()).long(), last)
        see = torch.eye(R, dtype=torch.bool, device="cuda").repeat(B, 1, 1)
        b, i = torch.arange(B, device="cuda")[:, None].expand(B, R), torch.arange(R, device="cuda")[None].expand(B, R)
        up = parent
        for _ in range(16):
            see[b, i, up.clamp(min=0)] |= up >= 0
            up = torch.where(up >= 0, parent.gather(1, up.clamp(min=0)), up)
        return see


def mask_words(see):
    """[B][R][R] booleans -> [B][R][ceil(R/64)] int64 bit rows."""
    B, R, _ = see.shape
    W = (R + 63) // 64
    wide = torch.zeros((B, R, W * 64), dtype=torch.int64, device=see.device)
    wide[:, :, :R] = see
    return (wide.view(B, R, W, 64) << torch.arange(64, device=see.device)).sum(-1)


def on_gpu(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    x, B, KVH, hd, page = Inputs(seed), case["B"], case["KVH"], case["hd"], case["page"]
    lens = lengths(case)
    s = {"case": case}
    if case["op"] == "prompt":
        H = case["H"]
        dt = torch.bfloat16 if case["dt"] == "bf16" else torch.float32
        ctx = contexts(case)
        s["rows"], s["ctx"] = lens, ctx
        s["first"] = [sum(lens[:b]) for b in range(B)]
        s["total"] = sum(lens) + case["spare"]  # rows behind the last sequence stay as they are
        s["row_start"], s["n_rows"], s["kv_len"] = on_gpu(s["first"]), on_gpu(lens), on_gpu(ctx)
        s["pages"], n = x.pages([c + r for c, r in zip(ctx, lens)], page)
        s["q"] = (x.normal(s["total"], H, hd) * 1.3).to(dt)
        s["k"], s["v"] = ((x.normal(n, KVH, page, hd) * torch.exp(0.3 * x.normal(1, KVH, 1, hd))).to(dt) for _ in range(2))
        s["o"] = torch.zeros((s["total"], H, hd), dtype=dt, device="cuda")
        s["lse"] = torch.zeros((s["total"], H), device="cuda")
        return s
    R, block = case["R"], case["block"]
    s["kv_len"], s["max_kv_len"] = on_gpu(lens), max(lens)
    if case["op"] == "kv8":
        L, rows = case["L"], path_rows(case)
        s["n_rows"] = on_gpu(rows)
        s["src_pages"], n = x.pages([max(R, 61) if case["path"] else R] * B, page)
        s["src"] = [(x.normal(L, n, KVH, page, hd) * torch.exp(0.5 * x.normal(1, 1, KVH, 1, hd))).to(torch.bfloat16) for _ in range(2)]
        s["path"] = None
        if case["path"]:  # node ids along a path: the root first, then increasing
            s["path"] = torch.cat([torch.zeros((B, 1), dtype=torch.int64, device="cuda"),
                                   1 + torch.cumsum(1 + x.ints(5, B, R - 1), 1)], 1).to(torch.int32).contiguous()
        s["n_given"] = s["n_rows"] - 1 if case["path"] else s["n_rows"]
        s["pages"], n8 = x.pages([p + R for p in lens], page)
        s["codes"] = [torch.zeros((L, n8, KVH, page, hd), dtype=torch.uint8, device="cuda") for _ in range(2)]
        s["exps"] = [torch.zeros((L, n8, KVH, page // block), dtype=torch.int8, device="cuda") for _ in range(2)]
        # the rows of each request's last block that are in the cache already
        s["open"] = s["kv_len"] % block
        s["back_first"], s["n_back"] = s["kv_len"] - s["open"], s["n_rows"] + s["open"]
        old = torch.arange(block, device="cuda")[None].expand(B, block)
        b, i = (old < s["open"][:, None]).nonzero(as_tuple=True)
        t = s["back_first"][b].long() + i
        if len(b):
            pg = s["pages"][b, t // page].long()
            for w in range(2):
                rows8 = torch.zeros((L, B, KVH, block, hd), device="cuda")
                rows8[:, b, :, i] = (x.normal(len(b), L, KVH, hd) * torch.exp(0.5 * x.normal(1, L, KVH, 1))).to(torch.bfloat16).float()
                e = needed(rows8.abs().amax((-2, -1)))
                s["codes"][w][:, pg, :, t % page] = to_codes(rows8, e[..., None, None])[:, b, :, i]
                s["exps"][w][:, pg, :, t % page // block] = e[:, b].to(torch.int8).permute(1, 0, 2)
        s["back_pages"], nb = x.pages([R + block] * B, page)
        s["back"] = [torch.zeros((L, nb, KVH, page, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        s["kv_len_next"] = torch.zeros_like(s["kv_len"])
        return s
    H = case["H"]
    s["pages"], n = x.pages(lens, page)
    s["codes"], s["exps"] = [], []
    for _ in range(2):
        v = x.normal(n, KVH, page, hd) * torch.exp(0.3 * x.normal(1, KVH, 1, hd)) * torch.exp(0.3 * x.normal(n, 1, page, 1))
        v = v.unflatten(2, (-1, block))
        e = needed(v.abs().amax((-2, -1)))
        s["codes"].append(to_codes(v, e[..., None, None]).flatten(2, 3))
        s["exps"].append(e.to(torch.int8))
    s["q"] = (x.normal(B, R, H, hd) * 1.5).to(torch.bfloat16)
    tp = -(-R // page)
    s["tail_pages"] = torch.arange(B * tp, dtype=torch.int32, device="cuda").view(B, tp).contiguous()
    s["tail"] = [x.normal(B * tp, KVH, page, hd).to(torch.bfloat16) for _ in range(2)]
    s["see"] = x.tree(B, R)
    s["mask"] = mask_words(s["see"])
    s["o"] = torch.zeros((B, R, H, hd), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros((B, R, H), device="cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def needed(amax):
    """Exponent of a block's scale: the smallest e with amax <= 448 * 2^e, within [E_MIN, E_MAX]."""
    m, ex = torch.frexp(amax.float())
    e = ex - 9 + (m > 0.875).to(ex.dtype)
    return torch.where(amax > 0, e.clamp(E_MIN, E_MAX), E_MIN)


def two_to(e):
    """2^e in fp32 from its exponent's bits (a power function may be off in its last one)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def to_codes(x, e):
    """Values -> e4m3 bytes of x / 2^e, to the nearest, ties to even."""
    return (x.float() * two_to(-e.int())).to(torch.float8_e4m3fn).view(torch.uint8)


def values(codes, e):
    return codes.view(torch.float8_e4m3fn).float() * two_to(e)


def slots(table, at, page):
    """(page id, slot) of the logical positions `at` [B][n] of each request."""
    return table.gather(1, at // page).long(), at % page


def run_prompt(s):
    case = s["case"]
    H, KVH, hd, page = (case[k] for k in ("H", "KVH", "hd", "page"))
    G = H // KVH
    for b in range(case["B"]):
        first, n, c = s["first"][b], s["rows"][b], s["ctx"][b]
        t = torch.arange(c + n, device="cuda")
        pg = s["pages"][b][t // page].long()
        k, v = (s[w][pg, :, t % page].float().transpose(0, 1) for w in "kv")  # [KVH][keys][hd]
        step = max(1, min(n, (1 << 29) // (H * (c + n))))
        for r0 in range(0, n, step):
            r1 = min(n, r0 + step)
            q = s["q"][first + r0:first + r1].float().view(r1 - r0, KVH, G, hd).permute(1, 2, 0, 3).flatten(1, 2)
            a = (q @ k.transpose(1, 2)).mul_(1.0 / math.sqrt(hd)).view(KVH, G, r1 - r0, c + n)
            a.masked_fill_(t[None] > c + torch.arange(r0, r1, device="cuda")[:, None], -math.inf)
            m = a.amax(-1, keepdim=True)
            p = a.sub_(m).exp_()
            z = p.sum(-1, keepdim=True)
            o = (p.flatten(1, 2) @ v).view(KVH, G, r1 - r0, hd) / z
            s["o"][first + r0:first + r1] = o.permute(2, 0, 1, 3).reshape(r1 - r0, H, hd).to(s["o"].dtype)
            s["lse"][first + r0:first + r1] = (m + torch.log(z))[..., 0].permute(2, 0, 1).reshape(r1 - r0, H)
    return {"o": s["o"], "lse": s["lse"]}


def run_kv8(s):
    case = s["case"]
    B, R, L, page, block = (case[k] for k in ("B", "R", "L", "page", "block"))
    # the blocks that change, from the one that each request's first new row lies in; every row of them
    W = (R + block - 1) // block + 1
    i = torch.arange(W * block, device="cuda")[None].expand(B, W * block)
    j = i - s["open"][:, None]  # number of the new row
    n = s["n_rows"][:, None]
    new, old = (j >= 0) & (j < n), j < 0
    cap = s["pages"].shape[1] * page
    t = (s["back_first"][:, None] + i).long().clamp(max=cap - 1)
    dp, ds = slots(s["pages"], t, page)
    r = j.clamp(0, R - 1).long()
    sp, ss = slots(s["src_pages"], s["path"].long().gather(1, r) if s["path"] is not None else r, page)
    bp, bs = slots(s["back_pages"], i.clamp(max=R + block - 1), page)
    keep = new | old
    for w in range(2):
        x = s["src"][w][:, sp, :, ss].float()  # [B][W block][L][KVH][hd]
        e_held = s["exps"][w][:, dp, :, ds // block].int()
        x = torch.where(new[..., None, None, None], x, torch.where(old[..., None, None, None],
                                                                   values(s["codes"][w][:, dp, :, ds], e_held[..., None]), 0.0))
        amax = (x.abs().amax(-1) * new[..., None, None]).unflatten(1, (W, block)).amax(2)  # of the new rows
        held = torch.where(old.unflatten(1, (W, block)).any(2)[..., None, None], e_held.unflatten(1, (W, block))[:, :, 0], E_MIN)
        e = torch.maximum(needed(amax), held).repeat_interleave(block, 1)
        codes = to_codes(x, e[..., None])
        back = values(codes, e[..., None]).to(torch.bfloat16)
        at = keep.nonzero(as_tuple=True)
        s["codes"][w][:, dp[at], :, ds[at]] = codes[at]
        s["exps"][w][:, dp[at], :, ds[at] // block] = e[at].to(torch.int8)
        s["back"][w][:, bp[at], :, bs[at]] = back[at]
    torch.add(s["kv_len"], s["n_rows"], out=s["kv_len_next"])
    return {"k": s["back"][0], "v": s["back"][1], "k_exp": s["exps"][0], "v_exp": s["exps"][1], "kv_len": s["kv_len_next"]}


def run_attn8(s):
    case = s["case"]
    B, R, H, KVH, hd, page, block = (case[k] for k in ("B", "R", "H", "KVH", "hd", "page", "block"))
    G = H // KVH
    T = -(-max(1, s["max_kv_len"]) // page)
    at = s["pages"][:, :T].long()
    k, v = (values(s["codes"][w][at], s["exps"][w][at].repeat_interleave(block, -1)[..., None]).transpose(1, 2).flatten(2, 3)
            for w in range(2))
    tail = s["tail_pages"].long()
    tk, tv = (s["tail"][w][tail].float().transpose(1, 2).flatten(2, 3)[:, :, :R] for w in range(2))
    q = s["q"].float().view(B, R, KVH, G, hd).permute(0, 2, 3, 1, 4).reshape(B, KVH, G * R, hd)
    live = torch.arange(k.shape[2], device="cuda")[None] < s["kv_len"][:, None]
    sp = (q @ k.transpose(2, 3) / math.sqrt(hd)).masked_fill_(~live[:, None, None], -math.inf)
    st = (q @ tk.transpose(2, 3) / math.sqrt(hd)).view(B, KVH, G, R, R)
    st = st.masked_fill_(~s["see"][:, None, None], -math.inf).view(B, KVH, G * R, R)
    m = torch.maximum(sp.amax(-1, keepdim=True), st.amax(-1, keepdim=True))
    p, t = torch.exp(sp - m), torch.exp(st - m)
    z = p.sum(-1, keepdim=True) + t.sum(-1, keepdim=True)
    o = (p @ v + t @ tv) / z
    o, lse = (y.view(B, KVH, G, R, -1).permute(0, 3, 1, 2, 4).reshape(B, R, H, -1) for y in (o, m + torch.log(z)))
    s["o"].copy_(o)
    s["lse"].copy_(lse[..., 0])
    return {"o": s["o"], "lse": s["lse"]}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def own_calls(s):
    """What a program keeps between its calls: descriptors and workspaces."""
    if "lib" not in s:
        from eagle_speculative_decoding_round_gb300 import eagle3 as e3
        case, s["lib"] = s["case"], e3
        B, KVH, hd, page = (case[k] for k in ("B", "KVH", "hd", "page"))
        s["dev_err"] = torch.zeros(1, dtype=torch.int32, device="cuda")

        def layer16(k, v, table, dt=e3.E3_BF16):
            return e3.make_kv_layer(k, v, table, k.shape[0], page, table.shape[1], KVH, hd, dt)

        def layer8(k, v, ke, ve):
            return e3.make_kv8_layer(k, v, ke, ve, s["pages"], k.shape[0], page, s["pages"].shape[1], KVH, hd, case["block"])
        if case["op"] == "prompt":
            dt = e3.E3_BF16 if case["dt"] == "bf16" else e3.E3_F32
            s["kv"], s["max_rows"], s["max_ctx"] = layer16(s["k"], s["v"], s["pages"], dt), max(s["rows"]), max(s["ctx"])
            s["ws_bytes"] = e3.eagle3_prompt_workspace_bytes(B, s["total"], s["max_rows"], case["H"], KVH, hd, s["max_ctx"], dt)
        elif case["op"] == "kv8":
            s["kv"] = [layer8(s["codes"][0][i], s["codes"][1][i], s["exps"][0][i], s["exps"][1][i]) for i in range(case["L"])]
            s["from"] = [layer16(s["src"][0][i], s["src"][1][i], s["src_pages"]) for i in range(case["L"])]
            s["to"] = [layer16(s["back"][0][i], s["back"][1][i], s["back_pages"]) for i in range(case["L"])]
            s["ws_bytes"] = 0
        else:
            s["kv"] = layer8(*s["codes"], *s["exps"])
            s["from"] = layer16(*s["tail"], s["tail_pages"])
            s["ws_bytes"] = e3.eagle3_verify8_workspace_bytes(B, case["R"], case["H"], KVH, hd, s["max_kv_len"])
        s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device="cuda")
    return s["lib"]


def own_prompt(s):
    e3, case = own_calls(s), s["case"]
    e3.prompt_attn(s["q"], s["row_start"], s["n_rows"], s["kv"], s["kv_len"], case["B"], s["total"], s["max_rows"], case["H"], s["max_ctx"],
                   1.0 / math.sqrt(case["hd"]), s["o"], s["lse"], s["dev_err"], s["ws"], s["ws_bytes"])
    return {"o": s["o"], "lse": s["lse"]}


def own_kv8(s):
    e3, case = own_calls(s), s["case"]
    e3.kv8_append(s["kv"], s["from"], case["B"], case["R"], s["path"], s["n_given"], 1 if case["path"] else 0, s["kv_len"],
                  s["kv_len_next"], s["dev_err"])
    e3.kv8_read(s["kv"], s["to"], case["B"], case["R"] + case["block"], s["back_first"], s["n_back"], s["dev_err"])
    return {"k": s["back"][0], "v": s["back"][1], "k_exp": s["exps"][0], "v_exp": s["exps"][1], "kv_len": s["kv_len_next"]}


def own_attn8(s):
    e3, case = own_calls(s), s["case"]
    e3.tree_verify_attn8(s["q"], s["kv"], s["from"], s["kv_len"], s["mask"], case["B"], case["R"], case["H"], s["max_kv_len"],
                         1.0 / math.sqrt(case["hd"]), s["o"], s["lse"], s["dev_err"], s["ws"], s["ws_bytes"])
    return {"o": s["o"], "lse": s["lse"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"prompt": own_prompt, "kv8": own_kv8, "attn8": own_attn8}[op](state)
    return {"prompt": run_prompt, "kv8": run_kv8, "attn8": run_attn8}[op](state)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------

def work(case):
    B, KVH, hd, lens = case["B"], case["KVH"], case["hd"], lengths(case)
    if case["op"] == "prompt":
        H, size, ctx = case["H"], 2 if case["dt"] == "bf16" else 4, contexts(case)
        rows, keys = sum(lens), sum(lens) + sum(ctx)
        return {"bytes": rows * H * (2 * hd * size + 4) + keys * KVH * 2 * hd * size,
                "flops": 4 * hd * H * sum(n * c + n * (n + 1) // 2 for n, c in zip(lens, ctx))}
    if case["op"] == "kv8":  # 16-bit rows in, 8-bit rows out, 16-bit values back; the rows of an open block are read back as well
        n = sum(path_rows(case))
        held = sum(p % case["block"] for p in lens)
        width = case["L"] * 2 * KVH * hd
        return {"bytes": n * width * (2 + 1 + 2) + held * width * (1 + 2), "flops": (n + held) * width * 2}
    R, H, prefix = case["R"], case["H"], sum(lens)
    return {"bytes": prefix * KVH * 2 * hd + sum(-(-p // case["block"]) for p in lens) * KVH * 2 +
            B * R * (KVH * hd * 4 + H * hd * 4 + H * 4) + B * R * ((R + 63) // 64) * 8,
            "flops": 4 * hd * H * R * (prefix + B * R // 2)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": exact_prompt, "kv8": exact_kv8, "attn8": exact_attn8}[case["op"]](s)


def exact_prompt(s):
    """One request and one query head at a time, in strips of rows that meet only the keys up to their last, in 64 bits."""
    case = s["case"]
    H, KVH, hd, page = (case[k] for k in ("H", "KVH", "hd", "page"))
    o, lse = s["o"].double(), s["lse"].double()
    for b, (first, n, c) in enumerate(zip(s["first"], s["rows"], s["ctx"])):
        where = torch.arange(c + n, device="cuda")
        table = s["pages"][b].long()
        k, v = (s[w][table[where // page], :, where % page].double() for w in "kv")  # [keys][KVH][hd]
        for r0 in range(0, n, 2048):
            r1 = min(n, r0 + 2048)
            unseen = torch.ones((r1 - r0, c + r1), dtype=torch.bool, device="cuda").triu(c + r0 + 1)
            at = slice(first + r0, first + r1)
            for h in range(H):
                a = s["q"][at, h].double() @ k[:c + r1, h * KVH // H].T * hd ** -0.5
                a[unseen] = -math.inf
                top = torch.logsumexp(a, 1)
                o[at, h] = torch.exp(a - top[:, None]) @ v[:c + r1, h * KVH // H]
                lse[at, h] = top
    return {"o": o, "lse": lse}


def exact_kv8(s):
    """Request by request and block by block; each value's nearest point of the scaled grid by distance, a tie to the even code."""
    case = s["case"]
    page, block = case["page"], case["block"]
    grid = torch.tensor([(m / 8 if x == 0 else 1 + m / 8) * 2.0 ** (max(x, 1) - 7) for x in range(16) for m in range(8)][:127],
                        dtype=torch.float64, device="cuda")
    two = torch.tensor([2.0 ** e for e in range(E_MIN, E_MAX + 1)], dtype=torch.float64, device="cuda")
    tops = TOP * two

    def nearest(v):
        hi = torch.searchsorted(grid, v.contiguous()).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        up, down = grid[hi] - v, v - grid[lo]
        return grid[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]
    back = [t.double() for t in s["back"]]
    exps = [t.clone() for t in s["exps"]]
    for b, (p, n) in enumerate(zip(lengths(case), path_rows(case))):
        ids = s["path"][b, :n].long() if s["path"] is not None else torch.arange(n, device="cuda")
        table, src, out = (s[name][b].long() for name in ("pages", "src_pages", "back_pages"))
        start = p - p % block
        for w in range(2):
            x = s["src"][w][:, src[ids // page], :, ids % page].double()  # [n][L][KVH][hd]
            held = torch.arange(start, p, device="cuda")
            e_held = exps[w][:, table[start // page], :, start % page // block].long()  # [L][KVH]
            c = s["codes"][w][:, table[held // page], :, held % page].long()
            old = grid[(c % 128).clamp(max=126)] * (1 - 2 * (c // 128)) * two[e_held - E_MIN][..., None]
            rows = torch.cat([old, x])
            full = torch.nn.functional.pad(rows, (0, 0, 0, 0, 0, 0, 0, -len(rows) % block)).unflatten(0, (-1, block))
            fresh = full.clone()
            fresh[0, :p - start] = 0
            e = torch.searchsorted(tops, fresh.abs().amax((1, 4)).contiguous()).clamp(max=len(tops) - 1) + E_MIN  # [blocks][L][KVH]
            if p > start:
                e[0] = torch.maximum(e[0], e_held)
            step = two[e - E_MIN][:, None, :, :, None]
            done = (nearest(full.abs() / step) * step * torch.sign(full)).flatten(0, 1)[:len(rows)]
            r = torch.arange(len(rows), device="cuda")
            back[w][:, out[r // page], :, r % page] = done
            at = start + block * torch.arange(len(full), device="cuda")
            exps[w][:, table[at // page], :, at % page // block] = e.to(torch.int8)
    return {"k": back[0], "v": back[1], "k_exp": exps[0], "v_exp": exps[1], "kv_len": s["kv_len"] + s["n_rows"]}


def exact_attn8(s):
    """One request at a time, its keys and values in one row of positions, in 64 bits."""
    case = s["case"]
    R, H, KVH, hd, page, block = (case[k] for k in ("R", "H", "KVH", "hd", "page", "block"))
    grid = torch.tensor([(m / 8 if x == 0 else 1 + m / 8) * 2.0 ** (max(x, 1) - 7) for x in range(16) for m in range(8)],
                        dtype=torch.float64, device="cuda")
    grid = torch.cat([grid, -grid])
    two = torch.tensor([2.0 ** e for e in range(E_MIN, E_MAX + 1)], dtype=torch.float64, device="cuda")
    o = torch.zeros((case["B"], R, H, hd), dtype=torch.float64, device="cuda")
    lse = torch.zeros((case["B"], R, H), dtype=torch.float64, device="cuda")
    for b, p in enumerate(lengths(case)):
        t, j = torch.arange(p, device="cuda"), torch.arange(R, device="cuda")
        rows = []
        for w in range(2):
            pg = s["pages"][b].long()[t // page]
            x = grid[s["codes"][w][pg, :, t % page].long()] * two[s["exps"][w][pg, :, t % page // block].long() - E_MIN][..., None]
            rows.append(torch.cat([x, s["tail"][w][s["tail_pages"][b].long()[j // page], :, j % page].double()]))
        seen = torch.cat([torch.ones((R, p), dtype=torch.bool, device="cuda"), s["see"][b]], 1)
        for h in range(H):
            a = s["q"][b, :, h].double() @ rows[0][:, h // (H // KVH)].T * hd ** -0.5
            a[~seen] = -math.inf
            lse[b, :, h] = torch.logsumexp(a, 1)
            o[b, :, h] = torch.exp(a - lse[b, :, h, None]) @ rows[1][:, h // (H // KVH)]
    return {"o": o, "lse": lse}
