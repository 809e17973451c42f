"""Cases for latent attention: a hybrid model's full-attention layers whose
keys and values all come from one vector of 512 per token (the latent) and a
key part of 64 that all heads share.

  prompt   causal attention in the expanded form (every head its own key of 128
           beside the shared part, and its own value of 128), whole prompts or
           the newest tokens of longer ones, packed one after another
  train    the same with its backward pass (one training step's attention)
  store    new tokens' latents written to a paged cache in 8 bits (e4m3) with
           one power-of-two scale for each token and 128 values, the shared key
           part beside them in bfloat16
  load     the cache read back, as bfloat16, the sequences packed: what the
           next part of a long prompt is expanded from
  decode   attention of one or a few new tokens of every request in the absorbed
           form: every head's query meets the cached latents themselves

`run` computes them with elementary torch operations, or, with `own` set,
through kda_gated_delta_amd's entry points.
"""

import math
import random

import torch

own = False

D = 128                 # a head's own key, and its value
S = 64                  # the shared key part
R = 512                 # the latent
BLOCK = 128             # of the latent: values under one scale
SCALE = (D + S) ** -0.5
TOP = 448.0             # the largest e4m3 value
LEAST, MOST = -64, 119  # exponents of a cache scale
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a short question to an idle server: latency
        dict(name="prompt_short", kind="prompt", seqs=1, longest=129, past=0, ragged=False, one_row=False, heads=8),
        # the next parts of a few prompts, of different lengths, over what the cache already holds of them; keys
        # and values read from the rows of their one projection
        dict(name="prompt_continued", kind="prompt", seqs=6, longest=1500, past=6000, ragged=True, one_row=True,
             heads=32),
        # one long document
        dict(name="prompt_long", kind="prompt", seqs=1, longest=8192, past=0, ragged=False, one_row=False, heads=32),
        # a training step over packed samples of odd lengths
        dict(name="train_packed", kind="train", seqs=7, longest=2011, past=0, ragged=True, one_row=True, heads=12),
        # a training step over one long sample
        dict(name="train_long", kind="train", seqs=1, longest=8192, past=0, ragged=False, one_row=False, heads=16),
        # the latents of one decode step of a full server
        dict(name="store_step", kind="store", seqs=256, cached=700, new=1, page=64),
        # the latents of a batch of prompts
        dict(name="store_prompts", kind="store", seqs=16, cached=100, new=8192, page=64),
        # one conversation goes on
        dict(name="load_one", kind="load", seqs=1, longest=1500, page=64),
        # many do
        dict(name="load_many", kind="load", seqs=16, longest=16384, page=16),
        # one user, a short history: latency
        dict(name="decode_one", kind="decode", seqs=1, longest=1000, queries=1, page=64, heads=32),
        # a full server, histories of very different lengths
        dict(name="decode_batch", kind="decode", seqs=64, longest=16384, queries=1, page=64, heads=32),
        # a layer of many heads
        dict(name="decode_wide", kind="decode", seqs=48, longest=8192, queries=1, page=32, heads=96),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["prompt", "train", "store", "load", "decode"])
    page = rng.choice([16, 32, 64, 128])
    case = dict(kind=kind, seqs=1)
    if kind in ("prompt", "train"):
        # at most the (query, key) pairs and heads of the long listed case of its kind
        room = {"prompt": 32, "train": 16}[kind] * 8192 ** 2
        heads = rng.choice([1, 2, 5, 8, 12, 16, 32, 64])
        # (one token alone has no gradient in q and k: nothing to compare)
        longest = _log(rng, 1 if kind == "prompt" else 2, 8192)
        past = _log(rng, 1, 8192) if rng.random() < 0.4 else 0
        while heads * longest * (longest + 2 * past) > room:
            longest, past = max(2, longest * 3 // 4), past * 3 // 4
        case["seqs"] = min(_log(rng, 1, 64), max(1, room // (heads * longest * (longest + 2 * past))))
        case.update(longest=longest, past=past, ragged=past > 0 or rng.random() < 0.7, one_row=rng.random() < 0.5,
                    heads=heads)
    elif kind == "store":
        new = 1 if rng.random() < 0.4 else _log(rng, 1, 8192)
        case.update(seqs=min(_log(rng, 1, 512), max(1, 65536 // new)), cached=_log(rng, 1, 4096), new=new, page=page)
        case["seqs"] = min(case["seqs"], max(1, 400000 // (case["cached"] + new)))
    elif kind == "load":
        longest = _log(rng, 1, 65536)
        case.update(seqs=min(_log(rng, 1, 256), max(1, 131072 // longest)), longest=longest, page=page)
    else:
        longest, heads = _log(rng, 1, 131072), rng.choice([4, 8, 12, 16, 20, 32, 64, 96, 128])
        queries = rng.choice([1, 1, 1, 2, 4])
        # at most the tokens that the listed batch holds, and its products
        room = min(32 * 16384, 32 * 16384 * 32 // (heads * queries))
        while longest > room:
            longest = longest * 3 // 4
        case.update(seqs=min(_log(rng, 1, 256), max(1, room // longest)), longest=longest, queries=queries, page=page,
                    heads=heads)
    return case


def _lengths(n, longest, ragged, salt):
    """Lengths in [1, longest], the first of them `longest`."""
    rng = random.Random("%d %d %s" % (n, longest, salt))
    return [longest if i == 0 or not ragged else rng.randint(1, longest) for i in range(n)]


def _shape(case):
    """What the kinds' sizes come to: prompt, train: (queries, keys) per sequence; store: (cached, new) tokens; else the
    cached tokens."""
    kind = case["kind"]
    if kind in ("prompt", "train"):
        new = _lengths(case["seqs"], case["longest"], case["ragged"], "new")
        past = _lengths(case["seqs"], case["past"], True, "past") if case["past"] else [0] * case["seqs"]
        return new, [a + b for a, b in zip(new, past)]
    if kind == "store":
        return (_lengths(case["seqs"], case["cached"], True, "cached"),
                _lengths(case["seqs"], case["new"], True, "new"))
    return _lengths(case["seqs"], case["longest"], True, "cached")


def _pages(tokens, page):
    return -(-tokens // page)


TOKEN = R + R // BLOCK + 2 * S       # bytes of a token in the cache


def work(case):
    kind = case["kind"]
    if kind in ("prompt", "train"):
        (lq, lk), h = _shape(case), case["heads"]
        T, K = sum(lq), sum(lk)
        pairs = h * sum(a * b - a * (a - 1) // 2 for a, b in zip(lq, lk))
        rows, keys = 2 * (D + S) * h * T, 2 * K * (2 * D * h + S)
        if kind == "prompt":
            return {"bytes": rows + keys + T * h * (2 * D + 4), "flops": 2 * (2 * D + S) * pairs}
        # q, k, v, the shared part and d_out in; o, lse and the gradients out; two products forward, five backward
        return {"bytes": 2 * rows + 2 * keys + T * h * (4 * D + 4),
                "flops": 2 * (4 * (D + S) + 3 * D) * pairs}
    if kind == "store":
        T = sum(_shape(case)[1])
        return {"bytes": T * (2 * (R + S) + 4 + TOKEN), "flops": 2 * T * R}
    lens = _shape(case)
    T, held = sum(lens), sum(_pages(x, case["page"]) for x in lens)
    if kind == "load":
        return {"bytes": T * (TOKEN + 2 * (R + S)) + 4 * (held + len(lens) + 1), "flops": T * R}
    rows = case["heads"] * case["queries"]
    return {"bytes": T * TOKEN + 4 * held + len(lens) * (4 + rows * (2 * (R + S) + 2 * R + 4)),
            "flops": 2 * (2 * R + S) * rows * T}


# ------------------------------------------------------------------ the inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _cache(g, pages, page):
    """A cache in use: codes of normalised latents under the scales that fit them (about 2^-7)."""
    codes = torch.empty(pages, page, R, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (page * R))
    for i in range(0, pages, step):
        part = torch.randn(min(step, pages - i), page, R, generator=g, device=DEV)
        codes[i:i + step] = (part * 100.0).clamp_(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.randint(127 - 8, 127 - 6, (pages, page, R // BLOCK), generator=g, device=DEV).to(torch.uint8)
    return {"c_cache": codes.view(torch.float8_e4m3fn), "c_scale": scale, "k_cache": _normal(g, pages, page, S)}


def _tables(order, lens, page, spare):
    """Page ids of each sequence, in no order, in rows as wide as the longest; and all pages."""
    held = [_pages(n, page) for n in lens]
    ids = list(range(sum(held) + spare))
    order.shuffle(ids)
    table, at = [], 0
    for n in held:
        table.append(ids[at:at + n] + [-1] * (max(held) - n))
        at += n
    return table, len(ids)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kind, s = case["kind"], {"case": dict(case)}
    if kind in ("prompt", "train"):
        (lq, lk), h = _shape(case), case["heads"]
        B, T, K = (1, sum(lq), sum(lk)) if case["ragged"] else (len(lq), max(lq), max(lk))
        s["q"], s["k_shared"] = _normal(g, B, T, h, D + S), _normal(g, B, K, S)
        if case["one_row"]:
            row = _normal(g, B, K, h, 2 * D)
            s["k"], s["v"] = row[..., :D], row[..., D:]
        else:
            s["k"], s["v"] = _normal(g, B, K, h, D), _normal(g, B, K, h, D)
        s["cu"] = _ints(_offsets(lq)) if case["ragged"] else None
        s["cu_kv"] = _ints(_offsets(lk)) if case["past"] else s["cu"]
        s["longest"] = max(lq), max(lk)
        if kind == "train":
            s["d_out"] = _normal(g, B, T, h, D)
        return s
    order, page = random.Random(seed), case["page"]
    if kind == "store":
        old, new = _shape(case)
        table, pages = _tables(order, [a + b for a, b in zip(old, new)], page, 50)
        slots = [row[p // page] * page + p % page for row, a, b in zip(table, old, new) for p in range(a, a + b)]
        row = _normal(g, len(slots), R + S)      # latent and shared part leave one projection together
        # some tokens' values larger than others'
        row[:, :R] *= 1 + 7 * (torch.rand(len(slots), 1, generator=g, device=DEV) < 0.1)
        s.update(_cache(g, pages, page), slots=_ints(slots), c=row[:, :R], k_shared=row[:, R:])
        return s
    lens = _shape(case)
    table, pages = _tables(order, lens, page, 3)
    s.update(_cache(g, pages, page), table=_ints(table))
    if kind == "load":
        s.update(cu=_ints(_offsets(lens)), tokens=sum(lens))
    else:
        s.update(lens=_ints(lens), longest=max(lens), q=_normal(g, len(lens), case["queries"], case["heads"], R + S))
    return s


# ------------------------------------------------------------------ the plain forms

def _spread(x, cu, L):
    """[B, T, ...] -> float32 [N, L, ...], each sequence from its first token (rows behind its last hold other tokens)."""
    if cu is None:
        return x.float()
    return x[0].float()[(cu[:-1, None] + torch.arange(L, device=x.device)).clamp_(max=x.shape[1] - 1)]


def _gather(x, cu, T):
    """[N, L, ...] -> [1, T, ...]: the sequences' rows, packed."""
    if cu is None:
        return x
    t = torch.arange(T, device=x.device)
    n = torch.searchsorted(cu, t, right=True) - 1
    return x[n, t - cu[n]][None]


def _heads(x):
    return x.transpose(1, 2)            # [N, L, H, ...] <-> [N, H, L, ...]


def _prompt(s):
    (Lq, Lk), cu, cu_kv = s["longest"], s["cu"], s["cu_kv"]
    q, v = _heads(_spread(s["q"], cu, Lq)), _heads(_spread(s["v"], cu_kv, Lk))
    k = _heads(_spread(s["k"], cu_kv, Lk))
    k = torch.cat((k, _spread(s["k_shared"], cu_kv, Lk)[:, None].expand(-1, k.shape[1], -1, -1)), -1)
    p = torch.matmul(q, k.transpose(2, 3)).mul_(SCALE)
    i, j = torch.arange(Lq, device=q.device)[:, None], torch.arange(Lk, device=q.device)
    if cu is None:
        seen = j <= i + Lk - Lq
    else:
        seen = j <= i + (cu_kv[1:] - cu_kv[:-1] - cu[1:] + cu[:-1])[:, None, None, None]
    p.masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(total)
    return q, k, v, p, torch.matmul(p, v), (top + total.log())[..., 0]


def _packed(x, cu, T):
    return _gather(_heads(x), cu, T).bfloat16()


def _prompt_plain(s):
    *_, o, lse = _prompt(s)
    T = s["q"].shape[1]
    return _packed(o, s["cu"], T), _heads(_gather(_heads(lse), s["cu"], T))


def _train_plain(s):
    q, k, v, p, o, lse = _prompt(s)
    cu, cu_kv, T, K = s["cu"], s["cu_kv"], s["q"].shape[1], s["k"].shape[1]
    do = _heads(_spread(s["d_out"], cu, s["longest"][0]))
    if cu is not None:                  # rows behind a sequence's end have no gradient
        real = torch.arange(do.shape[2], device=q.device) < (cu[1:] - cu[:-1])[:, None]
        do = do * real[:, None, :, None]
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(SCALE)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q)
    return (_packed(o, cu, T), _heads(_gather(_heads(lse), cu, T)), _packed(dq, cu, T),
            _packed(dk[..., :D], cu_kv, K), _gather(dk[..., D:].sum(1), cu_kv, K).bfloat16(), _packed(dv, cu_kv, K))


def _store_plain(s):
    slots, c = s["slots"].long(), s["c"].float().unflatten(1, (-1, BLOCK))
    top = c.abs().amax(-1)
    part, power = torch.frexp(top)
    e = torch.where(top > 0, power - 9 + (part > 0.875).int(), LEAST).clamp(LEAST, MOST)
    codes = (c * torch.exp2(-e.float())[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    s["c_cache"].view(torch.uint8).flatten(0, 1)[slots] = codes.flatten(1).view(torch.uint8)
    s["c_scale"].flatten(0, 1)[slots] = (e + 127).to(torch.uint8)
    s["k_cache"].flatten(0, 1)[slots] = s["k_shared"]
    return s["c_cache"], s["c_scale"], s["k_cache"]


def _values(s, at):
    """Latents [..., 512] and shared parts [..., 64] in float32 at places `at` of the cache."""
    codes = s["c_cache"].view(torch.uint8).flatten(0, 1)[at].view(torch.float8_e4m3fn).float()
    scale = torch.exp2(s["c_scale"].flatten(0, 1)[at].float() - 127.0)
    return (codes.unflatten(-1, (-1, BLOCK)) * scale[..., None]).flatten(-2), s["k_cache"].flatten(0, 1)[at].float()


def _load_plain(s):
    cu, P = s["cu"], s["c_cache"].shape[1]
    t = torch.arange(s["tokens"], device=cu.device)
    n = torch.searchsorted(cu, t, right=True) - 1
    at = t - cu[n]
    c, k = _values(s, s["table"][n, at // P].long() * P + at % P)
    return c.bfloat16(), k.bfloat16()


def _decode_plain(s):
    q, lens, P = s["q"].float(), s["lens"], s["c_cache"].shape[1]
    N, Q, H, _ = q.shape
    pages = s["table"].long().clamp(min=0)
    at = (pages[..., None] * P + torch.arange(P, device=q.device)).flatten(1)
    c, k = _values(s, at)
    L = c.shape[1]
    p = torch.matmul(q.flatten(1, 2), torch.cat((c, k), -1).transpose(1, 2)).mul_(SCALE).view(N, Q, H, L)
    seen = torch.arange(L, device=q.device) <= (lens[:, None] - Q + torch.arange(Q, device=q.device))[..., None]
    seen = seen[:, :, None, :]
    top = p.masked_fill(~seen, -math.inf).amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(p - torch.where(top > -math.inf, top, 0.0)), 0.0)
    total = p.sum(-1, keepdim=True)
    lse = top + total.log()
    p = p / torch.where(total > 0, total, 1.0)
    return torch.matmul(p.view(N, Q * H, L), c).view(N, Q, H, R).bfloat16(), lse[..., 0]


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import kda_gated_delta_amd as kda
    kind = s["case"]["kind"]
    if kind in ("prompt", "train"):
        more = dict(cu_seqlens=s["cu"], cu_seqlens_kv=s["cu_kv"])
        o, lse = kda.latent_prefill(s["q"], s["k"], s["k_shared"], s["v"], **more)
        if kind == "prompt":
            return o, lse
        return (o, lse, *kda.latent_backward(s["q"], s["k"], s["k_shared"], s["v"], o, lse, s["d_out"], **more))
    cache = s["c_cache"], s["c_scale"], s["k_cache"]
    if kind == "store":
        kda.latent_cache_store(s["c"], s["k_shared"], *cache, s["slots"])
        return cache
    if kind == "load":
        return kda.latent_cache_load(*cache, s["table"], s["cu"], s["tokens"])
    if "workspace" not in s:            # a server keeps one for all its steps
        s["workspace"] = torch.empty(kda.latent_decode_workspace_size(*s["q"].shape[:3]), dtype=torch.uint8, device=DEV)
    return kda.latent_decode(s["q"], *cache, s["table"], s["lens"], workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    return {"prompt": _prompt_plain, "train": _train_plain, "store": _store_plain, "load": _load_plain,
            "decode": _decode_plain}[state["case"]["kind"]](state)


# ------------------------------------------------------------------ the definitions, in 64 bits

def _softmax64(z, seen):
    """Weights and logarithm of their sum of scores z [r, n] where seen; rows that see nothing are zero."""
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, dim=1)
    return torch.where(seen, torch.exp(z - torch.where(torch.isfinite(lse), lse, 0.0)[:, None]), 0.0), lse


def _exact_prompt(s, train):
    q, k, v, shared = (s[x].double() for x in ("q", "k", "v", "k_shared"))
    B, T, H, _ = q.shape
    o, lse = q.new_zeros(B, T, H, D), q.new_zeros(B, H, T)
    dq, dk, dv, dshared = (torch.zeros_like(x) for x in (q, k, v, shared))
    cu = [0, T] if s["cu"] is None else s["cu"].tolist()
    cu_kv = [0, k.shape[1]] if s["cu_kv"] is None else s["cu_kv"].tolist()
    for b in range(B):
        for lo, hi, klo, khi in zip(cu, cu[1:], cu_kv, cu_kv[1:]):
            last = khi - klo - (hi - lo) + torch.arange(hi - lo, device=q.device)
            seen = torch.arange(khi - klo, device=q.device)[None, :] <= last[:, None]
            common = shared[b, klo:khi]
            for h in range(H):
                qn, qs = q[b, lo:hi, h, :D], q[b, lo:hi, h, D:]
                kh, vh = k[b, klo:khi, h], v[b, klo:khi, h]
                w, lse[b, h, lo:hi] = _softmax64((qn @ kh.t() + qs @ common.t()) / math.sqrt(D + S), seen)
                o[b, lo:hi, h] = w @ vh
                if train:
                    up = s["d_out"][b, lo:hi, h].double()
                    dv[b, klo:khi, h] = w.t() @ up
                    dw = up @ vh.t()
                    dz = w * (dw - (w * dw).sum(1, keepdim=True)) / math.sqrt(D + S)
                    dq[b, lo:hi, h, :D], dq[b, lo:hi, h, D:] = dz @ kh, dz @ common
                    dk[b, klo:khi, h] = dz.t() @ qn
                    dshared[b, klo:khi] += dz.t() @ qs
    return (o, lse, dq, dk, dshared, dv) if train else (o, lse)


def _exact_store(s):
    c, scale, k = s["c_cache"].float().double(), s["c_scale"].clone(), s["k_cache"].double()
    slots = s["slots"].long()
    for j in range(R // BLOCK):
        x = s["c"][:, j * BLOCK:(j + 1) * BLOCK].double()
        e = torch.ceil(torch.log2(x.abs().amax(1) / TOP)).clamp(LEAST, MOST)
        c.view(-1, R)[slots, j * BLOCK:(j + 1) * BLOCK] = x / torch.exp2(e)[:, None]
        scale.view(-1, R // BLOCK)[slots, j] = (e + 127).to(torch.uint8)
    k.view(-1, S)[slots] = s["k_shared"].double()
    return c, scale, k


def _exact_tokens(s, n, length):
    P = s["c_cache"].shape[1]
    ids = s["table"][n, :_pages(length, P)].long()
    c = s["c_cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).float().double()
    c = c.view(-1, R)[:length]
    scale = s["c_scale"][ids].view(-1, R // BLOCK)[:length].double()
    c = c * torch.exp2(scale - 127).repeat_interleave(BLOCK, 1)
    return c, s["k_cache"][ids].view(-1, S)[:length].double()


def _exact_load(s):
    got = [_exact_tokens(s, n, length) for n, length in enumerate(_shape(s["case"]))]
    return torch.cat([c for c, _ in got]), torch.cat([k for _, k in got])


def _exact_decode(s):
    q = s["q"].double()
    N, Q, H, _ = q.shape
    o, lse = q.new_zeros(N, Q, H, R), q.new_zeros(N, Q, H)
    for n, length in enumerate(s["lens"].tolist()):
        c, k = _exact_tokens(s, n, length)
        for i in range(Q):
            seen = (torch.arange(length, device=q.device) <= length - Q + i)[None, :]
            w, lse[n, i] = _softmax64((q[n, i, :, :R] @ c.t() + q[n, i, :, R:] @ k.t()) / math.sqrt(D + S), seen)
            o[n, i] = w @ c
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("prompt", "train"):
        return _exact_prompt(s, kind == "train")
    return {"store": _exact_store, "load": _exact_load, "decode": _exact_decode}[kind](s)
