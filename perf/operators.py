"""Measured cases of the operators around one verify pass over a 4-bit KV cache.

  qkv     tree_qkv_append: per-head norms of the projected queries and keys, rotary
          positions, and the append of K and V to a paged cache
  kv4     kv4_append + kv4_read: rows of a 16-bit cache committed to the 4-bit cache
          (the accepted path of a round, or a whole prompt), and read back as values
  attn4   tree_verify_attn4: tree attention whose prefix is held in 4 bits
  logits  tree_logits_process: penalties along the tree's paths, biases and grammar masks
          on the node logits, with the softmax statistics that the accept step reads

``run`` computes the plain form in elementary torch operations, or, where ``own`` is set,
makes the calls of this repository's library.
"""
import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of a 4-bit value (1 sign, 2 exponent, 1 mantissa bit)
EPS = 1e-5

# query heads, KV heads, head dim of the shapes that the rounds of this repository run with
TINY, MID, LARGE = (4, 4, 64), (32, 8, 128), (64, 8, 128)


def listed():
    return [
        # one round's tree nodes of a single request (the smallest serving call: launch latency)
        dict(name="qkv tree", op="qkv", B=1, R=61, H=32, KVH=8, hd=128, lo=2048, hi=2048, page=64, dt="bf16", rot=128,
             inter=False, scal="wavelen", norm=False, ragged=False),
        # a ragged batch of prompts entering the cache, with per-head norms
        dict(name="qkv prompts", op="qkv", B=4, R=4099, H=32, KVH=8, hd=128, lo=0, hi=1024, page=64, dt="bf16", rot=128,
             inter=False, scal="plain", norm=True, ragged=True),
        # fp32 target, interleaved pairs over half of each head
        dict(name="qkv tiny fp32", op="qkv", B=2, R=15, H=4, KVH=4, hd=64, lo=128, hi=133, page=16, dt="f32", rot=32,
             inter=True, scal="linear", norm=True, ragged=False),
        # the accepted paths of a batched round, every layer
        dict(name="kv4 accepted paths", op="kv4", B=32, R=7, L=32, KVH=8, hd=128, lo=512, hi=8192, page=64, path=True),
        # two prompts compressed into the 4-bit cache, four layers
        dict(name="kv4 prompts", op="kv4", B=2, R=8191, L=4, KVH=8, hd=128, lo=0, hi=77, page=64, path=False),
        # plain decoding of a batch: one node a request
        dict(name="attn4 decode", op="attn4", B=32, R=1, H=32, KVH=8, hd=128, lo=512, hi=8192, page=64),
        # one request's 60-node tree at a moderate prefix (latency)
        dict(name="attn4 tree", op="attn4", B=1, R=61, H=32, KVH=8, hd=128, lo=2048, hi=2048, page=64),
        # batched serving: 32 requests, each with its tree
        dict(name="attn4 batch", op="attn4", B=32, R=61, H=32, KVH=8, hd=128, lo=512, hi=8192, page=64),
        # long context: one request, a small tree
        dict(name="attn4 long", op="attn4", B=1, R=33, H=32, KVH=8, hd=128, lo=65536, hi=65536, page=64),
        # narrow heads, odd lengths, short pages, a request without a prefix
        dict(name="attn4 narrow", op="attn4", B=3, R=15, H=4, KVH=4, hd=64, lo=0, hi=1025, page=16),
        # one request's node logits: repetition, frequency and presence penalties, biases, a grammar
        dict(name="logits tree", op="logits", B=1, R=61, V=128256, bias=37, grammar=True, seen=900),
        # a batch's node logits
        dict(name="logits batch", op="logits", B=32, R=61, V=128256, bias=5, grammar=True, seen=3000),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qkv", "kv4", "attn4", "attn4", "logits"])
    if op == "qkv":
        H, KVH, hd = rng.choice([TINY, MID, LARGE, (8, 2, 128), (6, 1, 64)])
        B = log_int(rng, 1, 32)
        R = log_int(rng, 1, max(1, 16000 // B))
        lo = rng.randint(0, 100000)
        return dict(op=op, B=B, R=R, H=H, KVH=KVH, hd=hd, lo=lo, hi=lo + rng.randint(0, 3000), page=rng.choice([16, 64, 128]),
                    dt=rng.choice(["bf16", "bf16", "f32"]), rot=rng.choice([hd, hd, hd // 2, 24]), inter=rng.random() < 0.4,
                    scal=rng.choice(["plain", "linear", "wavelen", "yarn"]), norm=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if op == "kv4":
        path = rng.random() < 0.5
        B = log_int(rng, 1, 32)
        R = rng.randint(1, 9) if path else log_int(rng, 1, max(1, 16000 // B))
        lo = rng.randint(0, 2000)
        return dict(op=op, B=B, R=R, L=rng.randint(1, 32) if path else rng.randint(1, 4), KVH=rng.choice([1, 2, 8]),
                    hd=rng.choice([64, 128]), lo=lo, hi=lo + rng.randint(0, 3000), page=rng.choice([16, 64, 128]), path=path)
    if op == "attn4":
        H, KVH, hd = rng.choice([TINY, MID, MID, LARGE, (8, 1, 128), (6, 2, 64), (5, 5, 128)])
        B = log_int(rng, 1, 32)
        hi = log_int(rng, 16, max(64, min(65536, 130000 // B)))
        R = rng.choice([1, 2, rng.randint(3, 16), rng.randint(17, 64), rng.randint(65, 200)])
        R = max(1, min(R, 60000 // (B * H)))
        hi = max(16, min(hi, 250000000 // (B * R * H)))
        return dict(op=op, B=B, R=R, H=H, KVH=KVH, hd=hd, lo=rng.randint(0, hi), hi=hi, page=rng.choice([16, 64, 64, 128]))
    B = log_int(rng, 1, 32)
    R = rng.randint(1, max(1, min(64, 1600 // B)))
    return dict(op=op, B=B, R=R, V=rng.choice([1024, 32000, 128256, 50257, log_int(rng, 1000, 150000)]), bias=rng.choice([0, 3, 60, 300]),
                grammar=rng.random() < 0.6, seen=log_int(rng, 10, 900))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def lengths(case):
    """Prefix length of each request: spread over [lo, hi], in no order."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [lo + (hi - lo) * ((5 * b + 3) % B) // max(1, B - 1) for b in range(B)] if B > 1 else [hi]


def counts_of_rows(case):
    """Rows of each request that hold something: all of them, or a ragged part."""
    B, R = case["B"], case["R"]
    if case.get("path"):
        return [1 + (3 * b + 1) % R for b in range(B)]
    if case.get("ragged"):
        return [max(1, R * ((3 * b + 1) % B + 1) // B - (b & 1)) for b in range(B)]
    return [R] * B


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
        """(parent, depth, ancestor-or-self [B][R][R] of booleans) of random trees, nodes in an order with parents first."""
        parent = torch.full((B, R), -1, dtype=torch.int64, device="cuda")
        if R > 1:
            u = self.uniform(B, R - 1)
            first = (torch.arange(1, R, device="cuda") - 12).clamp(min=0)  # a window keeps the trees wide and of moderate depth
            span = torch.arange(1, R, device="cuda") - first
            parent[:, 1:] = (first // 3 + (u * (span + first - first // 3)).long()).clamp(max=torch.arange(0, R - 1, device="cuda"))
            parent[:, 1:] = parent[:, 1:] // 2 if R > 24 else parent[:, 1:]
        see = torch.eye(R, dtype=torch.bool, device="cuda").repeat(B, 1, 1)
        up = parent.clone()
        depth = torch.zeros((B, R), dtype=torch.int64, device="cuda")
        b = torch.arange(B, device="cuda")[:, None].expand(B, R)
        i = torch.arange(R, device="cuda")[None].expand(B, R)
        for _ in range(16):
            on = up >= 0
            see[b, i, up.clamp(min=0)] |= on
            depth += on
            up = torch.where(on, parent.gather(1, up.clamp(min=0)), up)
        return parent, depth, see


def mask_words(see):
    """[B][R][R] booleans -> [B][R][ceil(R/64)] int64 bit rows."""
    B, R, _ = see.shape
    W = (R + 63) // 64
    wide = torch.zeros((B, R, W * 64), dtype=torch.int64, device=see.device)
    wide[:, :, :R] = see
    return (wide.view(B, R, W, 64) << torch.arange(64, device=see.device)).sum(-1)


def frequencies(case, dev):
    """Angle per position of each rotated pair, in 64 bits, and the factor on the rotated part."""
    rot, base = case["rot"], 500000.0
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    if case["scal"] == "linear":
        return f / 4.0, 1.0
    if case["scal"] == "wavelen":  # long waves slowed by 8, short ones kept, a ramp between
        turns = 8192.0 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return f * ((1.0 - keep) / 8.0 + keep), 1.0
    if case["scal"] == "yarn":  # the same by the pair's index, with a factor on the rotated part
        at = [rot * math.log(4096.0 / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32.0, 1.0)]
        a, e = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        slow = ((torch.arange(rot // 2, dtype=torch.float64, device=dev) - a) / max(e - a, 0.001)).clamp(0.0, 1.0)
        return f * (slow / 16.0 + (1.0 - slow)), 0.1 * math.log(16.0) + 1.0
    return f, 1.0


def prepare(case, seed):
    x, B, R = Inputs(seed), case["B"], case["R"]
    s = {"case": case}
    if case["op"] == "logits":
        V = case["V"]
        s["logits"] = x.normal(B * R, V) * 2.5
        s["parent"], s["depth"], s["see"] = x.tree(B, R)
        s["tok"] = x.ints(V, B, R).to(torch.int32)
        s["parent"] = s["parent"].to(torch.int32)
        s["temp_rows"] = (0.6 + x.uniform(B, 1)).expand(B, R).reshape(-1).contiguous()
        n = x.ints(V, B, case["seen"])  # what the answer holds so far, and (the last third) the prompt
        cnt = torch.zeros((B, V), dtype=torch.int64, device="cuda")
        third = case["seen"] // 3
        cnt.scatter_add_(1, n[:, third:], torch.ones_like(n[:, third:]))
        prompt = torch.zeros((B, V), dtype=torch.int64, device="cuda").scatter_(1, n[:, :third], 1)
        s["counts"] = (cnt + 32768 * prompt - 65536 * prompt * (cnt + 32768 * prompt >= 32768)).to(torch.int16)
        s["pen"] = torch.stack([1.0 + 0.3 * x.uniform(B), 0.5 * x.uniform(B), 0.5 * x.uniform(B)], 1).contiguous()
        nb = case["bias"]
        s["bias_tok"] = x.ints(V, B, nb).to(torch.int32) if nb else None
        s["bias_val"] = x.normal(B, nb) * 3.0 if nb else None
        s["allow"] = s["allow_row"] = None
        if case["grammar"]:  # an eighth of the nodes are free, the others follow one of 16 masks
            W = (V + 31) // 32
            a, b2 = (x.ints(2 ** 32, 16, W) for _ in range(2))
            bits = a & torch.where(torch.arange(16, device="cuda")[:, None] % 2 == 0, b2, torch.full_like(b2, 2 ** 32 - 1))
            bits[:, 0] |= 1
            s["allow"] = (bits - 2 ** 32 * (bits >= 2 ** 31)).to(torch.int32)
            s["allow_row"] = torch.where(x.uniform(B, R) < 0.125, -1, x.ints(16, B, R)).to(torch.int32)
        s["out"] = torch.zeros((B * R, V), device="cuda")
        s["row_max"] = torch.zeros(B * R, device="cuda")
        s["row_Q"] = torch.zeros(B * R, dtype=torch.int64, device="cuda")
        s["row_argmax"] = torch.zeros(B * R, dtype=torch.int32, device="cuda")
        return s
    KVH, hd, page = case["KVH"], case["hd"], case["page"]
    lens, rows = lengths(case), counts_of_rows(case)
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["n_rows"] = torch.tensor(rows, dtype=torch.int32, device="cuda")
    s["max_kv_len"] = max(lens)
    # flat indices b * R + r of the rows that hold something
    s["valid"] = torch.tensor([b * R + r for b in range(B) for r in range(rows[b])], device="cuda")
    if case["op"] == "qkv":
        H = case["H"]
        dt = torch.bfloat16 if case["dt"] == "bf16" else torch.float32
        s["qkv"] = x.normal(B, R, (H + 2 * KVH) * hd).to(dt)
        _, depth, _ = x.tree(B, R) if R <= 256 else (None, torch.arange(R, device="cuda")[None].expand(B, R), None)
        s["pos"] = (s["kv_len"][:, None] + depth).to(torch.int32).contiguous()
        s["q_norm"] = 1.0 + 0.2 * x.normal(hd) if case["norm"] else None
        s["k_norm"] = 1.0 + 0.2 * x.normal(hd) if case["norm"] else None
        s["pages"], n = x.pages([p + R for p in lens], page)
        # rows are appended to pages that already hold the prefix; a prefix beyond 4096 tokens is not filled in here
        s["k"] = x.normal(n, KVH, page, hd).to(dt) if n * page <= 1 << 17 else torch.zeros((n, KVH, page, hd), dtype=dt, device="cuda")
        s["v"] = torch.zeros((n, KVH, page, hd), dtype=dt, device="cuda")
        s["q"] = torch.zeros((B, R, H, hd), dtype=dt, device="cuda")
        return s
    if case["op"] == "kv4":
        L = case["L"]
        s["src_pages"], n = x.pages([max(R, 61) if case["path"] else R] * B, page)
        s["src"] = [(x.normal(L, n, KVH, page, hd) * torch.exp(0.5 * x.normal(1, 1, KVH, 1, hd))).to(torch.bfloat16) for _ in range(2)]
        s["path"] = None
        if case["path"]:  # node ids along a path: the root first, then increasing
            s["path"] = torch.cat([torch.zeros((B, 1), dtype=torch.int64, device="cuda"),
                                   1 + torch.cumsum(1 + x.ints(5, B, R - 1), 1)], 1).to(torch.int32).contiguous()
        s["n_given"] = s["n_rows"] - 1 if case["path"] else s["n_rows"]
        s["pages"], n4 = x.pages([p + R for p in lens], page)
        s["codes"] = [torch.zeros((L, n4, KVH, page, hd // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
        s["scales"] = [torch.zeros((L, n4, KVH, page, hd // 16), dtype=torch.uint8, device="cuda") for _ in range(2)]
        s["back"] = [torch.zeros((L, n, KVH, page, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        s["kv_len_next"] = torch.zeros_like(s["kv_len"])
        return s
    H = case["H"]
    s["pages"], n = x.pages(lens, page)
    s["codes"], s["scales"] = [], []
    for which in range(2):
        c, e = quantize(x.normal(n, KVH, page, hd) * torch.exp(0.3 * x.normal(1, KVH, 1, hd)), 1.0)
        s["codes"].append(c)
        s["scales"].append(e)
    s["q"] = (x.normal(B, R, H, hd) * 1.5).to(torch.bfloat16)
    tp = -(-R // page)
    s["tail_pages"] = torch.arange(B * tp, dtype=torch.int32, device="cuda").view(B, tp).contiguous()
    s["tail"] = [x.normal(B * tp, KVH, page, hd).to(torch.bfloat16) for _ in range(2)]
    _, _, s["see"] = x.tree(B, R)
    s["mask"] = mask_words(s["see"])
    s["o"] = torch.zeros((B, R, H, hd), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros((B, R, H), device="cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def quantize(x, unit):
    """Values [..., hd] -> (codes [..., hd/2] uint8, scale bytes [..., hd/16] uint8): each 16 values share a scale
    e4m3(amax / (6 unit)), each value is the nearest of +-GRID times scale times unit (ties to the even code)."""
    g = x.float().unflatten(-1, (-1, 16))
    e = (g.abs().amax(-1) / g.new_full((), 6.0 * unit)).clamp(max=448.0).to(torch.float8_e4m3fn)  # (a true division)
    step = (e.float() * unit).unsqueeze(-1)
    y = torch.where(step > 0, g.abs() / step, 0.0)
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = (code | (torch.signbit(g).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), e.view(torch.uint8)


def dequantize(codes, scales, unit, dtype=torch.float32):
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=dtype, device=codes.device)
    v = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * (scales.view(torch.float8_e4m3fn).to(dtype) * unit).unsqueeze(-1)).flatten(-2)


def slots(table, at, page):
    """(page id, slot) of the logical positions `at` [B][n] of each request."""
    return table.gather(1, at // page).long(), at % page


def plain_qkv(s, dtype=torch.float32):
    case = s["case"]
    B, R, H, KVH, hd, rot = (case[k] for k in ("B", "R", "H", "KVH", "hd", "rot"))
    x = s["qkv"].to(dtype).view(B, R, H + 2 * KVH, hd)
    q, k, v = x[:, :, :H], x[:, :, H:H + KVH], x[:, :, H + KVH:]
    if case["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["q_norm"].to(dtype)
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["k_norm"].to(dtype)
    f, m = frequencies(case, x.device)
    a = s["pos"].double()[..., None] * f
    c, n = (torch.cos(a) * m).to(dtype)[:, :, None], (torch.sin(a) * m).to(dtype)[:, :, None]

    def turned(y):
        z = y[..., :rot]
        if case["inter"]:
            p, r = z[..., 0::2], z[..., 1::2]
            z = torch.stack([p * c - r * n, r * c + p * n], -1).flatten(-2)
        else:
            p, r = z[..., :rot // 2], z[..., rot // 2:]
            z = torch.cat([p * c - r * n, r * c + p * n], -1)
        return torch.cat([z, y[..., rot:]], -1)
    return turned(q), turned(k), v


def run_qkv(s):
    case = s["case"]
    B, R, page = case["B"], case["R"], case["page"]
    q, k, v = plain_qkv(s)
    pg, sl = slots(s["pages"], (s["kv_len"][:, None] + torch.arange(R, device="cuda")).long(), page)
    at = s["valid"]
    s["q"].view(B * R, -1)[at] = q.reshape(B * R, -1)[at].to(s["q"].dtype)
    pg, sl = pg.reshape(-1)[at], sl.reshape(-1)[at]
    s["k"][pg, :, sl] = k.flatten(0, 1)[at].to(s["k"].dtype)
    s["v"][pg, :, sl] = v.flatten(0, 1)[at].to(s["v"].dtype)
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def from_and_to(s):
    """Pages and slots of a kv4 case's rows: in the source, in the 4-bit cache, and where they are read back to."""
    case = s["case"]
    B, R, page = case["B"], case["R"], case["page"]
    r = torch.arange(R, device="cuda").expand(B, R)
    at = s["valid"]
    sides = [(s["src_pages"], s["path"].long() if s["path"] is not None else r), (s["pages"], s["kv_len"][:, None].long() + r),
             (s["src_pages"], r)]
    return [tuple(t.reshape(-1)[at] for t in slots(table, where, page)) for table, where in sides]


def run_kv4(s):
    (sp, ss), (dp, ds), (bp, bs) = from_and_to(s)
    for w in range(2):
        codes, scales = quantize(s["src"][w][:, sp, :, ss], 1.0)
        s["codes"][w][:, dp, :, ds] = codes
        s["scales"][w][:, dp, :, ds] = scales
        s["back"][w][:, bp, :, bs] = dequantize(s["codes"][w][:, dp, :, ds], s["scales"][w][:, dp, :, ds], 1.0).to(torch.bfloat16)
    torch.add(s["kv_len"], s["n_rows"], out=s["kv_len_next"])
    return {"k": s["back"][0], "v": s["back"][1], "kv_len": s["kv_len_next"]}


def attend(s, b0, b1, dtype):
    """Requests b0 .. b1: (o, lse) of the softmax over the prefix in 4 bits and the seen tree nodes."""
    case = s["case"]
    R, H, KVH, hd, page = (case[k] for k in ("R", "H", "KVH", "hd", "page"))
    n, G = b1 - b0, H // KVH
    T = -(-max(1, s["max_kv_len"]) // page)
    at = s["pages"][b0:b1, :T].long()
    k, v = (dequantize(s["codes"][w][at], s["scales"][w][at], 1.0, dtype).transpose(1, 2).flatten(2, 3) for w in range(2))
    tail = s["tail_pages"][b0:b1].long()
    tk, tv = (s["tail"][w][tail].to(dtype).transpose(1, 2).flatten(2, 3)[:, :, :R] for w in range(2))
    q = s["q"][b0:b1].to(dtype).view(n, R, KVH, G, hd).permute(0, 2, 3, 1, 4).reshape(n, KVH, G * R, hd)
    live = torch.arange(k.shape[2], device="cuda")[None] < s["kv_len"][b0:b1, None]
    sp = (q @ k.transpose(2, 3) / math.sqrt(hd)).masked_fill_(~live[:, None, None], -math.inf)
    st = (q @ tk.transpose(2, 3) / math.sqrt(hd)).view(n, KVH, G, R, R)
    st = st.masked_fill_(~s["see"][b0:b1, None, None], -math.inf).view(n, KVH, G * R, R)
    m = torch.maximum(sp.amax(-1, keepdim=True), st.amax(-1, keepdim=True))
    p, t = torch.exp(sp - m), torch.exp(st - m)
    z = p.sum(-1, keepdim=True) + t.sum(-1, keepdim=True)
    o = (p @ v + t @ tv) / z
    back = [y.view(n, KVH, G, R, -1).permute(0, 3, 1, 2, 4).reshape(n, R, H, -1) for y in (o, m + torch.log(z))]
    return back[0], back[1][..., 0]


def run_attn4(s):
    o, lse = attend(s, 0, s["case"]["B"], torch.float32)
    s["o"].copy_(o)
    s["lse"].copy_(lse)
    return {"o": s["o"], "lse": s["lse"]}


def processed(s, dtype):
    """The rows' logits after penalties, biases and masks."""
    case = s["case"]
    B, R, V = case["B"], case["R"], case["V"]
    z = s["logits"].to(dtype).view(B, R, V)
    c = s["counts"].int()
    count = (c & 32767)[:, None].expand(B, R, V).contiguous()
    # node j counts for the rows of node j and its descendants; the root is in the answer's counts already
    onward = s["see"].clone()
    onward[:, :, 0] = False
    count.scatter_add_(2, s["tok"].long()[:, None].expand(B, R, R), onward.int())
    pen = s["pen"].to(dtype)
    rep, freq, pres = (pen[:, j, None, None] for j in range(3))
    seen = (count > 0) | (c < 0)[:, None]
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = torch.where(count > 0, z - freq * count.to(dtype) - pres, z)
    if case["bias"]:
        add = torch.zeros((B, V), dtype=torch.float64, device="cuda")
        add.scatter_add_(1, s["bias_tok"].long(), s["bias_val"].double())
        z = z + add.to(dtype)[:, None]
    if case["grammar"]:
        v = torch.arange(V, device="cuda")
        ok = ((s["allow"][:, v // 32] >> (v % 32)) & 1).bool()
        z = z.masked_fill_(~(ok[s["allow_row"].long().clamp(min=0)] | (s["allow_row"] < 0)[..., None]), -math.inf)
    return z.reshape(B * R, V)


def run_logits(s):
    V = s["case"]["V"]
    z = processed(s, torch.float32)
    t = z * (1.0 / s["temp_rows"])[:, None]
    m = t.amax(1, keepdim=True)
    s["out"].copy_(z)
    mass = torch.exp((t - m).double()).sum(1).float()
    first = torch.where(t == m, torch.arange(V, device="cuda", dtype=torch.int32), V).amin(1).to(torch.int32)
    return {"logits": s["out"], "max": m[:, 0], "argmax": first, "mass": mass}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def own_calls(s):
    """What a program keeps between its calls: descriptors and workspaces."""
    if "lib" not in s:
        from eagle_speculative_decoding_round_gb300 import eagle3 as e3
        case, s["lib"] = s["case"], e3
        s["dev_err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["op"] == "qkv":
            dt = e3.E3_BF16 if case["dt"] == "bf16" else e3.E3_F32
            how = {"plain": {}, "linear": dict(scaling=e3.E3_ROPE_LINEAR, factor=4.0),
                   "wavelen": dict(scaling=e3.E3_ROPE_WAVELEN, factor=8.0, low=1.0, high=4.0, orig_len=8192.0),
                   "yarn": dict(scaling=e3.E3_ROPE_YARN, factor=16.0, low=1.0, high=32.0, orig_len=4096.0)}[case["scal"]]
            s["rope"] = e3.eagle3_rope_init(case["rot"], 500000.0, interleaved=case["inter"], **how)
            s["kv"] = e3.make_kv_layer(s["k"], s["v"], s["pages"], s["k"].shape[0], case["page"], s["pages"].shape[1],
                                       case["KVH"], case["hd"], dt)
        elif case["op"] in ("kv4", "attn4"):
            def layer4(k, v, ks, vs, n):
                return e3.make_kv4_layer(k, v, ks, vs, s["pages"], n, case["page"], s["pages"].shape[1], case["KVH"], case["hd"])

            def layer16(k, v, table, n):
                return e3.make_kv_layer(k, v, table, n, case["page"], table.shape[1], case["KVH"], case["hd"], e3.E3_BF16)
            if case["op"] == "kv4":
                s["kv"] = [layer4(s["codes"][0][i], s["codes"][1][i], s["scales"][0][i], s["scales"][1][i], s["codes"][0].shape[1])
                           for i in range(case["L"])]
                s["from"], s["to"] = ([layer16(t[0][i], t[1][i], s["src_pages"], t[0].shape[1]) for i in range(case["L"])]
                                      for t in (s["src"], s["back"]))
            else:
                s["kv"] = layer4(*s["codes"], *s["scales"], s["codes"][0].shape[0])
                s["from"] = layer16(*s["tail"], s["tail_pages"], s["tail"][0].shape[0])
                s["ws_bytes"] = e3.eagle3_verify4_workspace_bytes(case["B"], case["R"], case["H"], case["KVH"], case["hd"], s["max_kv_len"])
                s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device="cuda")
    return s["lib"]


def own_qkv(s):
    e3, case = own_calls(s), s["case"]
    e3.tree_qkv_append(s["qkv"], s["qkv"].shape[2], case["B"], case["R"], s["n_rows"], case["H"], s["q_norm"], s["k_norm"], EPS, s["rope"],
                       s["pos"], s["q"], s["kv"], s["kv_len"], s["dev_err"])
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def own_kv4(s):
    e3, case = own_calls(s), s["case"]
    e3.kv4_append(s["kv"], s["from"], case["B"], case["R"], s["path"], s["n_given"], 1 if case["path"] else 0, s["kv_len"],
                  s["kv_len_next"], s["dev_err"])
    e3.kv4_read(s["kv"], s["to"], case["B"], case["R"], s["kv_len"], s["n_rows"], s["dev_err"])
    return {"k": s["back"][0], "v": s["back"][1], "kv_len": s["kv_len_next"]}


def own_attn4(s):
    e3, case = own_calls(s), s["case"]
    e3.tree_verify_attn4(s["q"], s["kv"], s["from"], s["kv_len"], s["mask"], case["B"], case["R"], case["H"], s["max_kv_len"],
                         1.0 / math.sqrt(case["hd"]), s["o"], s["lse"], s["dev_err"], s["ws"], s["ws_bytes"])
    return {"o": s["o"], "lse": s["lse"]}


def own_logits(s):
    e3, case = own_calls(s), s["case"]
    e3.tree_logits_process(s["logits"], case["B"], case["R"], case["V"], s["temp_rows"], s["counts"], s["tok"], s["parent"], s["pen"],
                           s["bias_tok"], s["bias_val"], case["bias"], s["allow"], s["allow_row"], 16 if case["grammar"] else 0,
                           s["out"], s["row_max"], s["row_Q"], s["row_argmax"], s["dev_err"])
    return {"logits": s["out"], "max": s["row_max"], "argmax": s["row_argmax"], "mass": (s["row_Q"].double() * 2.0 ** -40).float()}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"qkv": own_qkv, "kv4": own_kv4, "attn4": own_attn4, "logits": own_logits}[op](state)
    return {"qkv": run_qkv, "kv4": run_kv4, "attn4": run_attn4, "logits": run_logits}[op](state)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------

def work(case):
    B, R = case["B"], case["R"]
    if case["op"] == "logits":
        V = case["V"]
        masks = 16 * ((V + 31) // 32) * 4 if case["grammar"] else 0
        return {"bytes": B * R * V * 8 + B * V * 2 + masks + B * R * 28 + B * case["bias"] * 8, "flops": B * R * V * 8}
    KVH, hd = case["KVH"], case["hd"]
    n = sum(counts_of_rows(case))
    if case["op"] == "qkv":
        values = n * (case["H"] + 2 * KVH) * hd
        return {"bytes": values * 2 * (2 if case["dt"] == "bf16" else 4) + n * 4, "flops": values * 6}
    if case["op"] == "kv4":  # 16-bit rows in, 4.5-bit rows out, 16-bit values back
        values = n * case["L"] * 2 * KVH * hd
        return {"bytes": values * 2 + values * 9 // 16 + values * 2, "flops": values * 4}
    H = case["H"]
    prefix = sum(lengths(case))
    return {"bytes": prefix * KVH * 2 * (hd // 2 + hd // 16) + B * R * (KVH * hd * 4 + H * hd * 4 + H * 4) + B * R * ((R + 63) // 64) * 8,
            "flops": 4 * hd * H * R * (prefix + B * R // 2)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qkv":
        return exact_qkv(s)
    if case["op"] == "kv4":
        return exact_kv4(s)
    if case["op"] == "attn4":
        return exact_attn4(s)
    return exact_logits(s)


def exact_qkv(s):
    """Each pair as a complex number times exp(i angle), row by row into the cache."""
    case = s["case"]
    B, R, H, KVH, hd, rot, page = (case[k] for k in ("B", "R", "H", "KVH", "hd", "rot", "page"))
    f, m = frequencies(case, "cuda")
    turn = torch.polar(torch.full((B, R, rot // 2), m, dtype=torch.float64, device="cuda"), s["pos"].double()[..., None] * f)[:, :, None]
    out = {"q": s["q"].double(), "k": s["k"].double(), "v": s["v"].double()}
    heads = dict(zip("qkv", s["qkv"].double().view(B, R, -1, hd).split([H, KVH, KVH], 2)))
    for name in "qk":
        y = heads[name]
        if case["norm"]:
            y = y / (torch.linalg.vector_norm(y, dim=-1, keepdim=True).square() / hd + EPS).sqrt() * s[name + "_norm"].double()
        pairs = y[..., :rot].unflatten(-1, (rot // 2, 2) if case["inter"] else (2, rot // 2))
        re, im = pairs.unbind(-1 if case["inter"] else -2)
        z = torch.complex(re, im) * turn
        heads[name] = torch.cat([torch.stack([z.real, z.imag], -1 if case["inter"] else -2).flatten(-2), y[..., rot:]], -1)
    rows = counts_of_rows(case)
    for b, p in enumerate(lengths(case)):
        n = rows[b]
        out["q"][b, :n] = heads["q"][b, :n]
        where = torch.arange(p, p + n, device="cuda")
        for name in "kv":
            out[name][s["pages"][b].long()[where // page], :, where % page] = heads[name][b, :n]
    return out


def exact_kv4(s):
    """Each value's nearest point of the scaled grid by distance; a tie goes to the even code."""
    case = s["case"]
    R, page = case["R"], case["page"]
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")
    scale_grid = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()

    def nearest(v, points):
        hi = torch.searchsorted(points, v.contiguous()).clamp(max=len(points) - 1)
        lo = (hi - 1).clamp(min=0)
        up, down = points[hi] - v, v - points[lo]
        return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    back = [t.double() for t in s["back"]]
    for b, n in enumerate(counts_of_rows(case)):
        ids = s["path"][b, :n].long() if s["path"] is not None else torch.arange(n, device="cuda")
        r = torch.arange(n, device="cuda")
        table = s["src_pages"][b].long()
        for w in range(2):
            x = s["src"][w][:, table[ids // page], :, ids % page].double().unflatten(-1, (-1, 16))
            step = scale_grid[nearest((x.abs().amax(-1) / x.new_full((), 6.0)).clamp(max=448), scale_grid)].unsqueeze(-1)
            y = torch.where(step > 0, x.abs() / step, 0.0)
            back[w][:, table[r // page], :, r % page] = (grid[nearest(y, grid)] * step * torch.sign(x)).flatten(-2)
    return {"k": back[0], "v": back[1], "kv_len": s["kv_len"] + s["n_rows"]}


def exact_attn4(s):
    """One request at a time, its keys and values in one row of positions, in 64 bits."""
    case = s["case"]
    R, H, KVH, hd, page = (case[k] for k in ("R", "H", "KVH", "hd", "page"))
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device="cuda")
    o = torch.zeros((case["B"], R, H, hd), dtype=torch.float64, device="cuda")
    lse = torch.zeros((case["B"], R, H), dtype=torch.float64, device="cuda")
    for b, p in enumerate(lengths(case)):
        t = torch.arange(p, device="cuda")
        j = torch.arange(R, device="cuda")
        rows = []
        for w in range(2):
            pg = s["pages"][b].long()[t // page]
            c = s["codes"][w][pg, :, t % page].long()  # [p][KVH][hd/2]
            e = s["scales"][w][pg, :, t % page].view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
            x = torch.empty((p, KVH, hd), dtype=torch.float64, device="cuda")
            x[..., 0::2], x[..., 1::2] = grid[c % 16], grid[c // 16]
            rows.append(torch.cat([x * e, s["tail"][w][s["tail_pages"][b].long()[j // page], :, j % page].double()]))
        seen = torch.cat([torch.ones((R, p), dtype=torch.bool, device="cuda"), s["see"][b]], 1)
        for h in range(H):
            a = s["q"][b, :, h].double() @ rows[0][:, h // (H // KVH)].T * hd ** -0.5
            a[~seen] = -math.inf
            lse[b, :, h] = torch.logsumexp(a, 1)
            o[b, :, h] = torch.exp(a - lse[b, :, h, None]) @ rows[1][:, h // (H // KVH)]
    return {"o": o, "lse": lse}


def exact_logits(s):
    """One request at a time; each node's path is walked up from the node."""
    case = s["case"]
    B, R, V = case["B"], case["R"], case["V"]
    out = torch.empty((B * R, V), dtype=torch.float64, device="cuda")
    top, mass = (torch.empty(B * R, dtype=torch.float64, device="cuda") for _ in range(2))
    parents, toks = s["parent"].tolist(), s["tok"].tolist()
    for b in range(B):
        held = s["counts"][b].long() & 32767
        count = held.repeat(R, 1)
        i, t = [], []
        for node in range(R):
            u = node
            while u > 0:
                i.append(node)
                t.append(toks[b][u])
                u = parents[b][u]
        if i:
            count.index_put_((torch.tensor(i, device="cuda"), torch.tensor(t, device="cuda")), torch.tensor(1, device="cuda"), accumulate=True)
        z = s["logits"][b * R:(b + 1) * R].double()
        rep, freq, pres = s["pen"][b].double()
        factor = torch.where(z > 0, 1.0 / rep, rep)
        z = torch.where((count > 0) | (s["counts"][b] < 0), z * factor, z) - freq * count - pres * (count > 0)
        if case["bias"]:
            z.index_add_(1, s["bias_tok"][b].long(), s["bias_val"][b].double().expand(R, -1))
        if case["grammar"]:
            bits = (s["allow"].long()[:, :, None] >> torch.arange(32, device="cuda")) & 1
            no = bits.flatten(1)[:, :V][s["allow_row"][b].long()] == 0
            no[s["allow_row"][b] < 0] = False
            z[no] = -math.inf
        at = slice(b * R, (b + 1) * R)
        out[at] = z
        t = z / s["temp_rows"][at, None].double()
        top[at] = t.amax(1)
        mass[at] = torch.exp(t - top[at, None]).sum(1)
    return {"logits": out, "max": top, "argmax": None, "mass": mass}
