"""Cases for the full-attention operators: what a hybrid model runs in the
layers between its gated-delta layers.

  prompt   causal attention over whole prompts, grouped heads, sequences of
           equal length or packed one after another
  train    the same with its backward pass (one training step's attention)
  tables   page tables, slot map and packed offsets of one serving step, made
           on the GPU from the requests' lengths
  store    new keys and values written to a paged cache in 8 bits (e4m3) with
           one power-of-two scale for each page and head
  decode   attention of one or a few new tokens of every request over that
           cache

`run` computes them with elementary torch operations, or, with `own` set,
through kda_gated_delta_amd's entry points.  Heads are 128 wide throughout, as
everywhere in this library.
"""

import math
import random

import torch

own = False

D = 128
TOP = 448.0             # the largest e4m3 value
LEAST = -64             # the smallest exponent of a cache scale
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a short question to an idle server: latency
        dict(name="prompt_short", kind="prompt", seqs=1, longest=129, ragged=False, one_row=False,
             hq=8, hkv=2),
        # a batch of prompts of different lengths, packed, read from the rows of one projection
        dict(name="prompt_packed", kind="prompt", seqs=16, longest=4096, ragged=True, one_row=True,
             hq=16, hkv=2),
        # one long document
        dict(name="prompt_long", kind="prompt", seqs=1, longest=8192, ragged=False, one_row=False,
             hq=32, hkv=8),
        # a training step over packed samples of odd lengths
        dict(name="train_packed", kind="train", seqs=7, longest=2011, ragged=True, one_row=False,
             hq=12, hkv=4),
        # a training step over one long sample
        dict(name="train_long", kind="train", seqs=1, longest=8192, ragged=False, one_row=False,
             hq=16, hkv=4),
        # the bookkeeping of one decode step of a full server
        dict(name="tables_step", kind="tables", seqs=256, cached=8192, new=1, page=64),
        # the bookkeeping of a batch of prompts that just arrived
        dict(name="tables_prompts", kind="tables", seqs=32, cached=0, new=8192, page=64),
        # the keys and values of one decode step
        dict(name="store_step", kind="store", seqs=256, cached=700, new=1, page=64, hkv=8),
        # the keys and values of a batch of prompts
        dict(name="store_prompts", kind="store", seqs=8, cached=0, new=8192, page=64, hkv=8),
        # one user, a short history: latency
        dict(name="decode_one", kind="decode", seqs=1, longest=1000, queries=1, page=64, hq=32, hkv=8),
        # a full server, histories of very different lengths
        dict(name="decode_batch", kind="decode", seqs=64, longest=16384, queries=1, page=64,
             hq=32, hkv=8),
        # two very long histories, four drafted tokens checked at once
        dict(name="decode_long", kind="decode", seqs=2, longest=131072, queries=4, page=16,
             hq=16, hkv=2),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["prompt", "train", "tables", "store", "decode"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128])
    case = dict(kind=kind, seqs=1)
    if kind in ("prompt", "train"):
        # at most the attention (query, key) pairs of the long listed case of its kind
        room = {"prompt": 32, "train": 16}[kind] * 8192 ** 2
        # (one token alone has no gradient in q and k: nothing to compare)
        longest = _log(rng, 1 if kind == "prompt" else 2, 8192)
        heads = hkv * group
        case.update(longest=longest, ragged=rng.random() < 0.7, one_row=rng.random() < 0.5, hq=heads, hkv=hkv)
        case["seqs"] = min(_log(rng, 1, 64), max(1, room // (heads * longest ** 2)))
        while heads * longest ** 2 > room:
            case["longest"] = longest = longest * 3 // 4
    elif kind in ("tables", "store"):
        new = 1 if rng.random() < 0.4 else _log(rng, 1, 8192)
        top = {"tables": 262144, "store": 65536}[kind]
        case.update(seqs=min(_log(rng, 1, 512), max(1, top // new)), cached=_log(rng, 1, 4096), new=new, page=page)
        if kind == "store":
            case["hkv"] = hkv
            case["seqs"] = min(case["seqs"], max(1, 400000 // (case["cached"] + new)))
    else:
        longest = _log(rng, 1, 131072)
        seqs = min(_log(rng, 1, 256), max(1, 2 ** 23 // (longest * hkv)))
        case.update(seqs=seqs, longest=longest, queries=rng.choice([1, 1, 1, 2, 4, 7]), page=page, hq=hkv * group, hkv=hkv)
    return case


def _lengths(n, longest, ragged, salt):
    """Lengths in [1, longest], the first of them `longest`."""
    rng = random.Random("%d %d %s" % (n, longest, salt))
    return [longest if i == 0 or not ragged else rng.randint(1, longest) for i in range(n)]


def _shape(case):
    """What the kinds' sizes come to: the requests' lengths before and in this step."""
    if case["kind"] in ("prompt", "train"):
        return _lengths(case["seqs"], case["longest"], case["ragged"], "new")
    if case["kind"] == "decode":
        return _lengths(case["seqs"], case["longest"], True, "cached")
    old = _lengths(case["seqs"], case["cached"], True, "cached") if case["cached"] else [0] * case["seqs"]
    return old, _lengths(case["seqs"], case["new"], True, "new")


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    kind = case["kind"]
    if kind in ("prompt", "train"):
        lens, hq, hkv = _shape(case), case["hq"], case["hkv"]
        T, pairs = sum(lens), sum(n * (n + 1) // 2 for n in lens) * hq
        if kind == "prompt":
            return {"bytes": T * (2 * D * (2 * hq + 2 * hkv) + 4 * hq), "flops": 4 * D * pairs}
        # q, k, v, d_out in; o, lse and the three gradients out; two products forward, five backward
        return {"bytes": T * (2 * D * (4 * hq + 4 * hkv) + 4 * hq), "flops": 14 * D * pairs}
    if kind == "decode":
        lens, hq, hkv, n = _shape(case), case["hq"], case["hkv"], case["queries"]
        held = sum(_pages(x, case["page"]) for x in lens)
        return {"bytes": sum(lens) * hkv * 2 * D + held * (4 + 8 * hkv) + len(lens) * (4 + n * hq * (4 * D + 4)),
                "flops": 4 * D * hq * n * sum(lens)}
    old, new = _shape(case)
    T, page = sum(new), case["page"]
    if kind == "tables":
        added = sum(_pages(a + b, page) - _pages(a, page) for a, b in zip(old, new))
        return {"bytes": 4 * (4 * len(old) + 3 + T + 2 * added), "flops": 0}
    touched = sum((a + b - 1) // page - a // page + 1 for a, b in zip(old, new))
    return {"bytes": T * (case["hkv"] * 2 * D * 3 + 4) + touched * case["hkv"] * 16, "flops": 2 * T * case["hkv"] * D * 2}


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


def _cache(g, pages, hkv, page):
    """A cache in use: codes of normal values under the scale that fits a page's largest value (about 2^-6)."""
    def codes():
        out = torch.empty(pages, hkv, page, D, dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 27) // (hkv * page * D))
        for i in range(0, pages, step):
            part = torch.randn(min(step, pages - i), hkv, page, D, generator=g, device=DEV)
            out[i:i + step] = (part * 64.0).clamp_(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)
        return out.view(torch.float8_e4m3fn)
    def scales():
        return torch.exp2(torch.randint(-7, -5, (pages, hkv), generator=g, device=DEV).float())
    return {"k_cache": codes(), "v_cache": codes(), "k_scale": scales(), "v_scale": scales()}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kind, s = case["kind"], {"case": dict(case)}
    if kind in ("prompt", "train"):
        lens, hq, hkv = _shape(case), case["hq"], case["hkv"]
        T, L = sum(lens), max(lens)
        B, S = (1, T) if case["ragged"] else (len(lens), L)
        if case["one_row"]:
            row = _normal(g, B, S, hq + 2 * hkv, D)
            s["q"], s["k"], s["v"] = row[:, :, :hq], row[:, :, hq:hq + hkv], row[:, :, hq + hkv:]
        else:
            s["q"], s["k"], s["v"] = _normal(g, B, S, hq, D), _normal(g, B, S, hkv, D), _normal(g, B, S, hkv, D)
        s["cu"] = _ints(_offsets(lens)) if case["ragged"] else None
        s["longest"] = L
        if kind == "train":
            s["d_out"] = _normal(g, B, S, hq, D)
        return s
    order = random.Random(seed)
    if kind == "decode":
        lens, page = _shape(case), case["page"]
        held = [_pages(n, page) for n in lens]
        total = sum(held) + 3
        ids = list(range(total))
        order.shuffle(ids)
        table, at = [], 0
        for n in held:
            table.append(ids[at:at + n] + [-1] * (max(held) - n))
            at += n
        s.update(_cache(g, total, case["hkv"], page), table=_ints(table), lens=_ints(lens), longest=max(lens),
                 q=_normal(g, len(lens), case["queries"], case["hq"], D))
        return s
    old, new = _shape(case)
    page, T = case["page"], sum(new)
    width = max(_pages(a + b, page) for a, b in zip(old, new))
    held = [_pages(a, page) for a in old]
    total = sum(_pages(a + b, page) for a, b in zip(old, new)) + 100
    ids = list(range(total))
    order.shuffle(ids)
    table, at = [], 0
    for n in held:
        table.append(ids[at:at + n] + [-1] * (width - n))
        at += n
    if kind == "tables":
        s.update(cached=_ints(old), new=_ints(new), table=_ints(table), free=_ints(ids[at:]), head=_ints([0]),
                 tokens=T, page=page)
        return s
    slots = []
    for row, a, b in zip(table, old, new):
        for c in range(_pages(a, page), _pages(a + b, page)):
            row[c] = ids[at]
            at += 1
        slots += [row[p // page] * page + p % page for p in range(a, a + b)]
    s.update(_cache(g, total, case["hkv"], page), slots=_ints(slots), k=_normal(g, T, case["hkv"], D),
             v=_normal(g, T, case["hkv"], D))
    # some heads of some tokens larger than what their pages have held so far
    s["k"] *= 1 + 3 * (torch.rand(T, case["hkv"], 1, generator=g, device=DEV) < 0.1)
    return s


# ------------------------------------------------------------------ the plain forms

def _spread(x, cu, L):
    """[B, S, H, D] -> float32 [N, H, L, D], each sequence from its first token (rows behind its last hold other tokens)."""
    if cu is None:
        return x.float().transpose(1, 2)
    at = (cu[:-1, None] + torch.arange(L, device=x.device)).clamp_(max=x.shape[1] - 1)
    return x[0].float()[at].transpose(1, 2)


def _gather(x, cu, T):
    """[N, H, L, ...] -> [1, T, H, ...]: the sequences' rows, packed."""
    if cu is None:
        return x.transpose(1, 2)
    t = torch.arange(T, device=x.device)
    n = torch.searchsorted(cu, t, right=True) - 1
    return x[n, :, t - cu[n]][None]


def _prompt(s):
    q, k, v, cu, L = s["q"], s["k"], s["v"], s["cu"], s["longest"]
    T, hq, hkv = q.shape[1], q.shape[2], k.shape[2]
    q, k, v = _spread(q, cu, L), _spread(k, cu, L), _spread(v, cu, L)
    N, G = q.shape[0], hq // hkv
    q = q.reshape(N, hkv, G * L, D)
    p = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).view(N, hkv, G, L, L)
    p.masked_fill_(torch.ones(L, L, dtype=torch.bool, device=q.device).triu(1), -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).view(N, hq, L)
    p = p.div_(total).view(N, hkv, G * L, L)
    o = torch.matmul(p, v)
    return q, k, v, p, o, lse, (N, hkv, G, L, T)


def _prompt_plain(s):
    *_, o, lse, (N, hkv, G, L, T) = _prompt(s)
    return (_gather(o.view(N, hkv * G, L, D), s["cu"], T).bfloat16(),
            lse if s["cu"] is None else _gather(lse, s["cu"], T).transpose(1, 2))


def _train_plain(s):
    q, k, v, p, o, lse, (N, hkv, G, L, T) = _prompt(s)
    cu, shape = s["cu"], (N, hkv, G * L, D)
    do = _spread(s["d_out"], cu, L)
    if cu is not None:   # rows behind a sequence's end have no gradient
        real = torch.arange(L, device=q.device) < (cu[1:] - cu[:-1])[:, None]
        do = do * real[:, None, :, None]
    do = do.reshape(shape)
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(D ** -0.5)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q)
    heads = (N, hkv * G, L, D)
    return (_gather(o.view(heads), cu, T).bfloat16(), lse if cu is None else _gather(lse, cu, T).transpose(1, 2),
            _gather(dq.view(heads), cu, T).bfloat16(), _gather(dk, cu, T).bfloat16(), _gather(dv, cu, T).bfloat16())


def _tables_plain(s):
    old, new, table, free, page = s["cached"], s["new"], s["table"], s["free"], s["page"]
    W = table.shape[1]
    cu = torch.zeros(old.numel() + 1, dtype=torch.int32, device=old.device)
    cu[1:] = new.cumsum(0)
    first = ((old + page - 1) // page).clamp(max=W)
    last = ((old + new + page - 1) // page).clamp(max=W)
    ends = (last - first).cumsum(0)
    col = torch.arange(W, device=old.device)
    at = s["head"] + (ends - (last - first))[:, None] + col - first[:, None]
    added = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    table.copy_(torch.where((col >= first[:, None]) & (col < last[:, None]), added, table))
    t = torch.arange(s["tokens"], device=old.device)
    n = torch.searchsorted(cu, t, right=True) - 1
    pos = old[n] + t - cu[n]
    held = table[n, pos // page]
    slots = torch.where(held >= 0, held * page + pos % page, -1)
    return cu, slots.int(), old + new, table, (s["head"] + ends[-1]).int()


def _store_plain(s):
    slots = s["slots"].long()
    out = []
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        pages, hkv, P, _ = cache.shape
        page, off = slots // P, slots % P
        x = x.float()
        top = torch.zeros(pages, hkv, device=x.device)
        top.scatter_reduce_(0, page[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
        first = torch.full((pages,), P, device=x.device).scatter_reduce_(0, page, off, "amin")
        part, power = torch.frexp(top)
        fits = torch.where(top > 0, power - 9 + (part > 0.875).int(), LEAST).clamp(min=LEAST)
        fits = torch.exp2(fits.float())
        now = torch.where((first == 0)[:, None], fits, torch.maximum(scale, fits))
        now = torch.where((first < P)[:, None], now, scale)
        begun = page[(off == first[page]) & (off > 0)]       # pages that hold earlier tokens
        codes = cache.view(torch.uint8)
        held = codes[begun].view(torch.float8_e4m3fn).float() * (scale[begun] / now[begun])[:, :, None, None]
        earlier = torch.arange(P, device=x.device)[None, :] < first[begun][:, None]
        codes[begun] = torch.where(earlier[:, None, :, None], held.to(torch.float8_e4m3fn).view(torch.uint8), codes[begun])
        codes[page, :, off] = (x / now[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale.copy_(now)
        out += [cache, scale]
    return out


def _decode_plain(s):
    q, lens, longest = s["q"].float(), s["lens"], s["longest"]
    N, Q, hq, _ = q.shape
    hkv, P = s["k_cache"].shape[1:3]
    pages = s["table"][:, :_pages(longest, P)].long().clamp(min=0)
    L = pages.shape[1] * P

    def values(cache, scale):
        x = cache.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * scale[pages][..., None, None]
        return x.transpose(1, 2).reshape(N, hkv, L, D)

    rows = q.view(N, Q, hkv, hq // hkv, D).permute(0, 2, 1, 3, 4).reshape(N, hkv, -1, D)
    p = torch.matmul(rows, values(s["k_cache"], s["k_scale"]).transpose(2, 3)).mul_(D ** -0.5).view(N, hkv, Q, -1, L)
    seen = torch.arange(L, device=q.device) <= (lens[:, None] - Q + torch.arange(Q, device=q.device))[..., None]
    seen = seen[:, None, :, None, :]
    top = p.masked_fill(~seen, -math.inf).amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(p - torch.where(top > -math.inf, top, 0.0)), 0.0)
    total = p.sum(-1, keepdim=True)
    lse = top + total.log()
    p = p / torch.where(total > 0, total, 1.0)
    o = torch.matmul(p.view(N, hkv, -1, L), values(s["v_cache"], s["v_scale"]))
    o = o.view(N, hkv, Q, -1, D).permute(0, 2, 1, 3, 4).reshape(N, Q, hq, D)
    return o.bfloat16(), lse[..., 0].permute(0, 2, 1, 3).reshape(N, Q, hq)


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import kda_gated_delta_amd as kda
    kind = s["case"]["kind"]
    if kind == "prompt":
        return kda.attn_prefill(s["q"], s["k"], s["v"], cu_seqlens=s["cu"])
    if kind == "train":
        o, lse = kda.attn_prefill(s["q"], s["k"], s["v"], cu_seqlens=s["cu"])
        return (o, lse, *kda.attn_backward(s["q"], s["k"], s["v"], o, lse, s["d_out"], cu_seqlens=s["cu"]))
    if kind == "tables":
        cu, slots, lens, head = kda.attn_tables(s["cached"], s["new"], s["table"], s["free"], s["head"], s["page"],
                                                s["tokens"])
        return cu, slots, lens, s["table"], head
    if kind == "store":
        kda.attn_cache_store(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"])
        return [s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"]]
    if "workspace" not in s:   # a server keeps one for all its steps
        s["workspace"] = torch.empty(kda.attn_decode_workspace_size(*s["q"].shape[:3], s["k_cache"].shape[1]),
                                     dtype=torch.uint8, device=DEV)
    return kda.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"],
                           workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    return {"prompt": _prompt_plain, "train": _train_plain, "tables": _tables_plain, "store": _store_plain,
            "decode": _decode_plain}[state["case"]["kind"]](state)


# ------------------------------------------------------------------ the definitions, in 64 bits

def _softmax64(q, k, v, seen):
    """q [r, D], k, v [n, D], seen [r, n] -> (weights, output, log of the weights' sum); rows that see nothing are zero."""
    z = (q @ k.t()) / math.sqrt(D)
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, dim=1)
    w = torch.where(seen, torch.exp(z - torch.where(torch.isfinite(lse), lse, 0.0)[:, None]), 0.0)
    return w, w @ v, lse


def _exact_prompt(s, train):
    q, k, v = (s[x].double() for x in "qkv")
    B, T, hq, _ = q.shape
    G = hq // k.shape[2]
    o, lse = torch.zeros_like(q), q.new_zeros(B, hq, T)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    cu = [0, T] if s["cu"] is None else s["cu"].tolist()
    for b in range(B):
        for lo, hi in zip(cu, cu[1:]):
            at = torch.arange(hi - lo, device=q.device)
            seen = at[None, :] <= at[:, None]
            for h in range(hq):
                qq, kk, vv = q[b, lo:hi, h], k[b, lo:hi, h // G], v[b, lo:hi, h // G]
                w, out, z = _softmax64(qq, kk, vv, seen)
                o[b, lo:hi, h], lse[b, h, lo:hi] = out, z
                if train:
                    up = s["d_out"][b, lo:hi, h].double()
                    dv[b, lo:hi, h // G] += w.t() @ up
                    dw = up @ vv.t()
                    dz = w * (dw - (w * dw).sum(1, keepdim=True)) / math.sqrt(D)
                    dq[b, lo:hi, h] = dz @ kk
                    dk[b, lo:hi, h // G] += dz.t() @ qq
    return (o, lse, dq, dk, dv) if train else (o, lse)


def _exact_store(s):
    out, slots = [], s["slots"].tolist()
    P = s["k_cache"].shape[2]
    runs = {}
    for t, slot in enumerate(slots):
        runs.setdefault(slot // P, []).append(t)
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        cache, scale, x = cache.float().double(), scale.double(), x.double()
        biggest = x.abs().amax(-1)
        ids = torch.tensor([p for p, ts in runs.items() for _ in ts], device=x.device)
        ts = torch.tensor([t for ts in runs.values() for t in ts], device=x.device)
        begin = torch.tensor([min(slots[t] % P for t in ts) for ts in runs.values()], device=x.device)
        pages = torch.tensor(list(runs), device=x.device)
        top = torch.zeros_like(scale).scatter_reduce(0, ids[:, None].expand(-1, scale.shape[1]), biggest[ts], "amax")[pages]
        need = torch.exp2(torch.ceil(torch.log2(top / TOP)).clamp(min=LEAST))
        then = scale[pages]
        now = torch.where((begin > 0)[:, None], torch.maximum(then, need), need)
        kept = (torch.arange(P, device=x.device)[None, :] < begin[:, None])[:, None, :, None]
        cache[pages] = torch.where(kept, cache[pages] * (then / now)[:, :, None, None], cache[pages])
        scale[pages] = now
        where = torch.tensor(slots, device=x.device)
        cache[where // P, :, where % P] = x / scale[where // P][:, :, None]
        out += [cache, scale]
    return out


def _exact_decode(s):
    q = s["q"].double()
    N, Q, hq, _ = q.shape
    hkv, P = s["k_cache"].shape[1:3]
    o, lse = torch.zeros_like(q), q.new_zeros(N, Q, hq)
    for n, length in enumerate(s["lens"].tolist()):
        ids = s["table"][n, :_pages(length, P)].long()
        kv = []
        for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
            x = cache.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float().double() * scale[ids].double()[:, :, None, None]
            kv.append(x.transpose(0, 1).reshape(hkv, -1, D)[:, :length])
        seen = torch.arange(length, device=q.device)[None, :] <= length - Q + torch.arange(Q, device=q.device)[:, None]
        for h in range(hq):
            _, o[n, :, h], lse[n, :, h] = _softmax64(q[n, :, h], kv[0][h * hkv // hq], kv[1][h * hkv // hq], seen)
    return o, lse


def exact(case, seed):
    if case["kind"] == "tables":
        return None          # whole numbers only
    s = prepare(case, seed)
    if case["kind"] == "store":
        return _exact_store(s)
    return _exact_decode(s) if case["kind"] == "decode" else _exact_prompt(s, case["kind"] == "train")
