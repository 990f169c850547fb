"""Key-value cache operators of a serving loop, as cases to be measured.

Three operators that a decode step runs one after the other:

* plan:   block tables and slot maps from request lengths, on the GPU;
* append: the new tokens' keys and values into the paged cache (16-bit, or
          e4m3 codes with one scale per kv head);
* attend: attention of one new token per request over the paged cache.

`run` computes each in a plain form with elementary torch operations (own is
false) or calls the library (own is true).  Caches are [pages, kv heads, page
size, head dim]; the slot of a token is page * page_size + offset.
"""

import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"fp16": 2, "bf16": 2, "e4m3": 1}


def listed():
    return [
        # one chat request with a short history: latency counts
        dict(name="attend one short", op="attend", batch=1, heads=32, kv_heads=8, dim=128, page=16,
             dtype="fp16", cache="fp16", lo=200, hi=260, window=0, empty=False),
        # a small batch with uneven lengths, some slots of the batch idle (length 0), a head size
        # that is no power of two and pages that end inside a tile
        dict(name="attend ragged odd", op="attend", batch=13, heads=24, kv_heads=8, dim=80, page=24,
             dtype="bf16", cache="bf16", lo=1, hi=1500, window=0, empty=True),
        # a busy server: 64 requests of very different lengths over an e4m3 cache
        dict(name="attend batch e4m3", op="attend", batch=64, heads=64, kv_heads=8, dim=128, page=64,
             dtype="fp16", cache="e4m3", lo=256, hi=8192, window=0, empty=False),
        # sliding-window layers, a head each, wide heads
        dict(name="attend window", op="attend", batch=32, heads=16, kv_heads=16, dim=256, page=16,
             dtype="bf16", cache="e4m3", lo=300, hi=6000, window=1024, empty=False),
        # one document of 128K tokens: all the parallelism is along the cache
        dict(name="attend long", op="attend", batch=1, heads=32, kv_heads=8, dim=128, page=16,
             dtype="bf16", cache="bf16", lo=131072, hi=131072, window=0, empty=False),
        # one decode step's tokens
        dict(name="append decode", op="append", tokens=64, chunk=1, heads=32, kv_heads=8, dim=128,
             page=16, dtype="fp16", cache="fp16"),
        # ragged prompt chunks into an e4m3 cache, odd sizes
        dict(name="append ragged", op="append", tokens=1537, chunk=97, heads=24, kv_heads=8, dim=80,
             page=24, dtype="fp16", cache="e4m3"),
        # a prompt into an e4m3 cache
        dict(name="append prompt e4m3", op="append", tokens=8192, chunk=2048, heads=32, kv_heads=8,
             dim=128, page=64, dtype="bf16", cache="e4m3"),
        # the largest prompt batch, 16-bit cache
        dict(name="append large", op="append", tokens=32768, chunk=8192, heads=8, kv_heads=8, dim=128,
             page=16, dtype="bf16", cache="bf16"),
        # a decode step of a few requests
        dict(name="plan decode", op="plan", batch=8, page=16, cached_lo=0, cached_hi=4000, added_lo=1,
             added_hi=1),
        # a decode step of a large batch, long histories
        dict(name="plan large batch", op="plan", batch=1000, page=16, cached_lo=1, cached_hi=16384,
             added_lo=1, added_hi=1),
        # prompts of very different lengths entering together
        dict(name="plan prompts", op="plan", batch=256, page=32, cached_lo=0, cached_hi=0, added_lo=0,
             added_hi=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "plan"])
    kv = rng.choice([1, 2, 4, 8, 16, 32])
    dim = rng.choice([64, 80, 96, 112, 128, 192, 256])
    page = rng.choice([16, 16, 24, 32, 48, 64, 128])
    dtype = rng.choice(["fp16", "bf16"])
    cache = rng.choice([dtype, "e4m3"])
    if op == "attend":
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        batch = _log(rng, 1, 200)
        # at most 240 MB of 16-bit keys at the longest length of every request
        most = max(2, int(240e6 / (batch * kv * dim * 2)))
        hi = _log(rng, 1, min(most, 131072))
        lo = _log(rng, 1, hi)
        window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        return dict(op=op, batch=batch, heads=kv * group, kv_heads=kv, dim=dim, page=page, dtype=dtype,
                    cache=cache, lo=lo, hi=hi, window=window, empty=rng.random() < 0.25)
    if op == "append":
        tokens = _log(rng, 1, min(32768, int(60e6 / (kv * dim * 2))))
        return dict(op=op, tokens=tokens, chunk=_log(rng, 1, tokens), heads=kv * rng.choice([1, 2, 4]),
                    kv_heads=kv, dim=dim, page=page, dtype=dtype, cache=cache)
    batch = _log(rng, 1, 2000)
    cached_hi = rng.choice([0, _log(rng, 1, 16384)])
    added_hi = rng.choice([1, _log(rng, 1, max(1, min(4096, 200000 // batch)))])
    return dict(op=op, batch=batch, page=page, cached_lo=rng.randint(0, cached_hi), cached_hi=cached_hi,
                added_lo=min(added_hi, rng.choice([0, 1])), added_hi=added_hi)


def _lens(case):
    """The lengths of an attend case's requests: fixed by the case, so that its work is known."""
    rng = random.Random(case["batch"] * 1000003 + case["lo"] * 31 + case["hi"])
    lens = [_log(rng, case["lo"], case["hi"]) for _ in range(case["batch"])]
    if case["empty"]:
        lens = [0 if i % 5 == 3 else n for i, n in enumerate(lens)]
    return lens


def _plan_lens(case):
    rng = random.Random(case["batch"] * 1000003 + case["cached_hi"] * 31 + case["added_hi"])
    cached = [rng.randint(case["cached_lo"], case["cached_hi"]) for _ in range(case["batch"])]
    added = [rng.randint(case["added_lo"], case["added_hi"]) for _ in range(case["batch"])]
    return cached, added


def _seen(case):
    """Tokens that each request of an attend case attends to."""
    return [min(n, case["window"]) if case["window"] else n for n in _lens(case)]


def _normal(shape, g, dtype=torch.float16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _cache(pages, case, g):
    """A cache pool as a server holds it: every slot carries some earlier token's values."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    if case["cache"] == "e4m3":   # codes of N(0, 1) values at a scale of 1/32 (a range of +-14)
        return (_normal(shape, g) * 32).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return _normal(shape, g, DTYPES[case["cache"]])


def _scales(case, g):
    if case["cache"] != "e4m3":
        return None, None
    s = (0.75 + 0.5 * torch.rand((2, case["kv_heads"]), generator=g, device="cuda")) / 32
    return s[0].clone(), s[1].clone()


def _qkv(rows, case, g):
    """The three parts of a fused QKV product's output, as views of it."""
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    y = _normal((rows, (hq + 2 * hk) * d), g, DTYPES[case["dtype"]])
    q, k, v = y.split([hq * d, hk * d, hk * d], dim=1)
    return q.unflatten(1, (hq, d)), k.unflatten(1, (hk, d)), v.unflatten(1, (hk, d))


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    P = case.get("page")
    if case["op"] == "attend":
        lens = _lens(case)
        blocks = [-(-n // P) for n in lens]
        width = max(1, max(blocks))
        pages = sum(blocks) + 8
        s["q"] = _qkv(case["batch"], case, g)[0]
        s["k_cache"], s["v_cache"] = _cache(pages, case, g), _cache(pages, case, g)
        s["k_scale"], s["v_scale"] = _scales(case, g)
        order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
        n = torch.tensor(blocks, device="cuda")[:, None]
        at = torch.arange(width, device="cuda")[None, :]
        first = torch.cumsum(n, 0) - n
        s["table"] = torch.where(at < n, order[(first + at).clamp_(max=pages - 1)], -1).contiguous()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["max_len"] = max(1, max(lens))
    elif case["op"] == "append":
        # requests of `chunk` new tokens each, from a random offset in their first page on
        T, chunk = case["tokens"], case["chunk"]
        req = -(-T // chunk)
        per = -(-(chunk + P - 1) // P)
        pages = req * per + 4
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int64)
        off = torch.randint(0, P, (req,), generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        pos = off[t // chunk] + t % chunk
        s["slots"] = order[t // chunk * per + pos // P] * P + pos % P
        _, s["k"], s["v"] = _qkv(T, case, g)
        s["k_cache"], s["v_cache"] = _cache(pages, case, g), _cache(pages, case, g)
        s["k_scale"], s["v_scale"] = _scales(case, g)
    else:
        cached, added = _plan_lens(case)
        B = case["batch"]
        width = max(1, -(-(max(cached) + max(added)) // P))
        have = [-(-c // P) for c in cached]
        total = sum(-(-(c + a) // P) for c, a in zip(cached, added))
        order = torch.randperm(total + 16, generator=g, device="cuda", dtype=torch.int32)
        n = torch.tensor(have, device="cuda")[:, None]
        at = torch.arange(width, device="cuda")[None, :]
        first = torch.cumsum(n, 0) - n
        s["table"] = torch.where(at < n, order[(first + at).clamp_(max=total)], -1).contiguous()
        s["free"] = order[sum(have):].contiguous()
        s["cached"] = torch.tensor(cached, dtype=torch.int32, device="cuda")
        s["added"] = torch.tensor(added, dtype=torch.int32, device="cuda")
        s["tokens"] = sum(added)
        s["out"] = (torch.empty(B, dtype=torch.int32, device="cuda"),
                    torch.empty(B + 1, dtype=torch.int32, device="cuda"),
                    torch.empty(B + 1, dtype=torch.int32, device="cuda"),
                    torch.empty(sum(added), dtype=torch.int64, device="cuda"))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:   # the library and the buffers that a serving loop keeps for it
        import bit_quantized_gemm_qgemm_amd as qg

        s["qg"] = qg
        if case["op"] == "attend":
            s["out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
            s["workspace"] = torch.empty(max(16, qg.qgemm_paged_attention_workspace_bytes(
                case["batch"], case["heads"], case["kv_heads"], case["dim"], s["max_len"],
                case["window"])), dtype=torch.uint8, device="cuda")
    return s


def _plain_plan(s):
    P, table, free = s["page"], s["table"], s["free"]
    W = table.shape[1]
    c, a = s["cached"].long().clamp(min=0), s["added"].long().clamp(min=0)
    lens = (c + a).clamp(max=W * P)
    have = ((c + P - 1) // P).clamp(max=W)
    take = ((lens + P - 1) // P - have).clamp(min=0)
    cu_tokens = torch.nn.functional.pad(torch.cumsum(a, 0), (1, 0))
    cu_pages = torch.nn.functional.pad(torch.cumsum(take, 0), (1, 0))
    at = torch.arange(W, device=table.device)[None, :]
    j = at - have[:, None]
    pick = cu_pages[:-1, None] + j
    new = torch.where(pick < len(free), free[pick.clamp(0, len(free) - 1)], -1)
    table.copy_(torch.where((j >= 0) & (j < take[:, None]), new, table))
    t = torch.arange(s["tokens"], device=table.device)
    req = torch.searchsorted(cu_tokens[1:], t, right=True).clamp(max=len(c) - 1)
    pos = c[req] + t - cu_tokens[req]
    page = table[req, (pos // P).clamp(max=W - 1)].long()
    ok = (t < cu_tokens[-1]) & (pos < W * P) & (page >= 0)
    slots = torch.where(ok, page * P + pos % P, -1)
    return lens.int(), cu_tokens.int(), cu_pages.int(), slots, table


def _plain_append(s):
    P = s["page"]
    page, off = s["slots"] // P, s["slots"] % P
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        if scale is None:
            cache[page, :, off] = x
        else:
            codes = (x.float() / scale[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            cache.view(torch.uint8)[page, :, off] = codes.view(torch.uint8)
    return s["k_cache"], s["v_cache"]


def _plain_attend(s):
    q, P, D, Hk = s["q"], s["page"], s["dim"], s["kv_heads"]
    B, Hq = q.shape[:2]
    blocks = -(-s["max_len"] // P)
    table = s["table"][:, :blocks].long()

    def tokens(cache, scale):   # [B, Hk, blocks * P, D] in 32 bits
        x = cache.view(torch.uint8)[table.clamp(min=0)].view(cache.dtype).float()
        x = x.permute(0, 2, 1, 3, 4).reshape(B, Hk, blocks * P, D)
        return x if scale is None else x * scale[None, :, None, None]

    t = torch.arange(blocks * P, device=q.device)[None, :]
    n = s["lens"].long()[:, None]
    seen = (t < n) & (table >= 0).repeat_interleave(P, dim=1)
    if s["window"]:
        seen &= t >= n - s["window"]
    qg = q.float().reshape(B, Hk, Hq // Hk, D).transpose(2, 3).contiguous()
    score = torch.matmul(tokens(s["k_cache"], s["k_scale"]), qg).transpose(2, 3) * D ** -0.5
    score = torch.where(seen[:, None, None, :], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = (p / torch.where(total == 0, 1.0, total)).contiguous()
    v = torch.where(seen[:, None, :, None], tokens(s["v_cache"], s["v_scale"]), 0.0)
    return torch.matmul(p, v).reshape(B, Hq, D).to(q.dtype)


def run(s):
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)
    qg = s["qg"]
    if s["op"] == "plan":
        lens, cu_tokens, cu_pages, slots = qg.qgemm_kv_plan(
            s["table"], s["cached"], s["added"], s["free"], s["page"], s["tokens"], out=s["out"])
        return lens, cu_tokens, cu_pages, slots, s["table"]
    if s["op"] == "append":
        qg.qgemm_kv_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"],
                           k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["k_cache"], s["v_cache"]
    return qg.qgemm_paged_attention(
        s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], k_scale=s["k_scale"],
        v_scale=s["v_scale"], window=s["window"], max_len=s["max_len"], out=s["out"],
        workspace=s["workspace"])


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "plan":
        return None   # whole numbers
    P, D, Hk = case["page"], case["dim"], case["kv_heads"]
    if case["op"] == "append":
        got = []
        for part in ("k", "v"):
            x, scale = s[part].double(), s[part + "_scale"]
            if scale is not None:
                # nearest multiple of the step of x's binade (ties to even): 2^(e-3), 2^-9 at least
                x = (x / scale.double()[:, None]).clamp(-448, 448)
                step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
                x = torch.round(x / step) * step
            whole = s[part + "_cache"].double().permute(0, 2, 1, 3).reshape(-1, Hk, D)
            whole[s["slots"]] = x
            got.append(whole.reshape(-1, P, Hk, D).permute(0, 2, 1, 3).contiguous())
        return tuple(got)
    q = s["q"].double()
    group = case["heads"] // Hk
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for b, n in enumerate(_lens(case)):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        t = torch.arange(first, n, device=q.device)
        page, off = s["table"][b].long()[t // P], t % P
        for h in range(Hk):
            def rows(cache, scale):
                x = cache.view(torch.uint8)[:, h] if cache.dtype == torch.float8_e4m3fn else cache[:, h]
                x = x[page, off]
                x = x.view(cache.dtype).double()
                return x if scale is None else x * scale[h].double()

            qh = q[b, h * group:(h + 1) * group] / math.sqrt(D)
            w = torch.softmax(qh @ rows(s["k_cache"], s["k_scale"]).t().contiguous(), dim=1)
            out[b, h * group:(h + 1) * group] = w @ rows(s["v_cache"], s["v_scale"])
    return out


def work(case):
    if case["op"] == "attend":
        seen = sum(_seen(case))
        heads, kv, d = case["heads"], case["kv_heads"], case["dim"]
        size = 2 * seen * kv * d * SIZE[case["cache"]] + 4 * case["batch"] * heads * d
        entries = sum(-(-n // case["page"]) for n in _seen(case))
        return {"bytes": size + 4 * entries + 4 * case["batch"], "flops": 4 * seen * heads * d}
    if case["op"] == "append":
        n = case["tokens"] * case["kv_heads"] * case["dim"]
        return {"bytes": 2 * n * (2 + SIZE[case["cache"]]) + 8 * case["tokens"], "flops": 0}
    cached, added = _plan_lens(case)
    P = case["page"]
    taken = sum(-(-(c + a) // P) - -(-c // P) for c, a in zip(cached, added))
    return {"bytes": 20 * case["batch"] + 8 * taken + 8 * sum(added), "flops": 0}
