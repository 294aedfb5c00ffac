"""Measured cases of the grouped-head attention path: the rotation that appends keys and
values to a paged cache, the paged attention of one new token, and the attention of a
whole packed prompt.

Every case is a dict of plain values.  ``run`` makes one pass through an operator, in the
plain form (elementary torch operations in fp32) where ``own`` is false and through the
library's entry points where it is true.  ``exact`` computes the same outputs from the
definition in fp64.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of a batch of 64 on a two-KV-head shard: the smallest call of the
        # path, where the launch is all there is.
        dict(name="append_step", op="append", tokens=64, q_heads=16, kv_heads=2, dim=128, rot=128,
             neox=True, page=128, fp8=False, k_out=False, idle=0),
        # The new keys of a whole prompt of 16,384 tokens into an e4m3 cache, the rotated keys
        # also kept for the prompt's own attention.
        dict(name="append_prompt_fp8", op="append", tokens=16384, q_heads=32, kv_heads=8, dim=128,
             rot=128, neox=True, page=128, fp8=True, k_out=True, idle=0),
        # 4,089 unique tokens behind a shared prefix, 64-wide heads of which 32 columns rotate
        # in interleaved pairs, small pages, some tokens without a slot (padding).
        dict(name="append_partial", op="append", tokens=4089, q_heads=25, kv_heads=5, dim=64, rot=32,
             neox=False, page=16, fp8=False, k_out=True, idle=7),
        # One request with a short history: latency alone.
        dict(name="decode_short", op="decode", requests=1, shortest=137, longest=137, mix=1,
             q_heads=32, kv_heads=8, dim=128, page=16, fp8=False),
        # A serving batch: 64 requests of 2,048 .. 65,536 positions, a two-KV-head shard.
        dict(name="decode_batch", op="decode", requests=64, shortest=2048, longest=65536, mix=2,
             q_heads=16, kv_heads=2, dim=128, page=128, fp8=False),
        # One conversation of 142,000 positions in an e4m3 cache: split over its length.
        dict(name="decode_long_fp8", op="decode", requests=1, shortest=142000, longest=142000, mix=3,
             q_heads=64, kv_heads=8, dim=128, page=128, fp8=True),
        # Ragged lengths, five query heads a KV head, 64-wide heads, pages of 16, e4m3.
        dict(name="decode_ragged_fp8", op="decode", requests=37, shortest=1, longest=4089, mix=4,
             q_heads=20, kv_heads=4, dim=64, page=16, fp8=True),
        # A short question on its own: one sequence, few tiles.
        dict(name="prompt_short", op="prompt", requests=1, shortest=133, longest=133, context=0, mix=5,
             q_heads=32, kv_heads=8, dim=128, dim_v=128),
        # Prompts of very different lengths packed into one call.
        dict(name="prompt_packed", op="prompt", requests=24, shortest=17, longest=4089, context=0,
             mix=6, q_heads=32, kv_heads=8, dim=128, dim_v=128),
        # One long prompt.
        dict(name="prompt_long", op="prompt", requests=1, shortest=16384, longest=16384, context=0,
             mix=7, q_heads=32, kv_heads=8, dim=128, dim_v=128),
        # A latent-attention layer's prompt with its keys and values expanded to heads (12 heads
        # of 192 / 128 columns): 4,089 unique tokens behind a prefix of 63,911.
        dict(name="prompt_prefix_192", op="prompt", requests=1, shortest=4089, longest=4089,
             context=63911, mix=8, q_heads=12, kv_heads=12, dim=192, dim_v=128),
        # Small ragged prompts of 64-wide heads, seven query heads a KV head.
        dict(name="prompt_ragged_64", op="prompt", requests=53, shortest=1, longest=700, context=300,
             mix=9, q_heads=14, kv_heads=2, dim=64, dim_v=64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges, no dearer than the largest listed one."""
    largest = {}
    for c in listed():
        w = work(c)
        for k in ("bytes", "flops"):
            key = (c["op"], k)
            largest[key] = max(largest.get(key, 0), w[k])
    while True:
        op = rng.choice(("append", "decode", "prompt"))
        kv_heads = rng.choice((1, 2, 3, 4, 5, 8))
        group = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 12, 16))
        case = dict(op=op, q_heads=kv_heads * group, kv_heads=kv_heads)
        if op == "append":
            dim = rng.choice((64, 128))
            case.update(tokens=_log_int(rng, 1, 16384), dim=dim,
                        rot=rng.choice([r for r in (16, 32, 64, 96, 128) if r <= dim]),
                        neox=rng.random() < 0.5, page=rng.choice((1, 16, 32, 64, 128)),
                        fp8=rng.random() < 0.5, k_out=rng.random() < 0.5,
                        idle=rng.choice((0, 0, 3, 10)))
        elif op == "decode":
            longest = _log_int(rng, 1, 142000)
            case.update(requests=_log_int(rng, 1, 256), longest=longest,
                        shortest=_log_int(rng, 1, longest), mix=rng.randrange(1, 10 ** 6),
                        dim=rng.choice((64, 128)), page=rng.choice((1, 16, 32, 64, 128)),
                        fp8=rng.random() < 0.5)
        else:
            longest = _log_int(rng, 1, 16384)
            dim = rng.choice((64, 128, 192))
            case.update(requests=_log_int(rng, 1, 64), longest=longest,
                        shortest=_log_int(rng, 1, longest), mix=rng.randrange(1, 10 ** 6),
                        context=rng.choice((0, 0, _log_int(rng, 1, 63911))), dim=dim,
                        dim_v=min(dim, 128))
        w = work(case)
        if all(w[k] <= largest[(op, k)] for k in ("bytes", "flops")):
            return case


def _lengths(case):
    """The requests' lengths, log-uniform between the shortest and the longest, the longest
    among them; a property of the case, not of the seed."""
    rng = random.Random(case["mix"])
    out = [_log_int(rng, case["shortest"], case["longest"]) for _ in range(case["requests"])]
    out[rng.randrange(len(out))] = case["longest"]
    return out


def _prompt_lengths(case):
    """(query tokens, key positions) of every request; a prompt behind a prefix attends the
    prefix too."""
    rng = random.Random(case["mix"] + 1)
    new = _lengths(case)
    if case["context"] == 0:
        return new, list(new)
    if case["requests"] == 1:
        return new, [new[0] + case["context"]]
    return new, [n + rng.randrange(0, case["context"] + 1) for n in new]


def work(case):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        t = case["tokens"]
        read = t * ((hq + 2 * hk) * d * 2 + 4 + 4 + 4 * case["rot"])
        written = t * hq * d * 2 + (t * hk * d * 2 if case["k_out"] else 0)
        written += _live(case) * 2 * hk * d * (1 if case["fp8"] else 2)
        return {"bytes": read + written, "flops": 3 * t * (hq + hk) * case["rot"]}
    if case["op"] == "decode":
        lens = _lengths(case)
        pages = sum(-(-n // case["page"]) for n in lens)
        size = 1 if case["fp8"] else 2
        b = len(lens)
        return {"bytes": sum(lens) * hk * d * 2 * size + 2 * b * hq * d * 2 + b * hq * 4 +
                         4 * (pages + 2 * b + 1),
                "flops": 4 * sum(lens) * hq * d}
    new, keys = _prompt_lengths(case)
    dv = case["dim_v"]
    pairs = sum(n * k - n * (n - 1) // 2 for n, k in zip(new, keys))
    return {"bytes": 2 * (sum(new) * hq * (d + dv) + sum(keys) * hk * (d + dv)) + 4 * sum(new) * hq +
                     8 * (len(new) + 1),
            "flops": 2 * pairs * hq * (d + dv)}


def _live(case):
    """Tokens that have a slot: every idle-th one has none."""
    n = case["tokens"]
    return n - (n // case["idle"] if case["idle"] else 0)


# ----------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    """N(0, std^2), made in slices so that large tensors need no fp32 copy."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        x = torch.randn(n, generator=g, device=DEV) * std
        flat[i:i + n] = x.clamp_(-448, 448).to(dtype)
    return out


def _indptr(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=DEV)


def _append_inputs(case, seed):
    g = _gen(seed)
    t, hq, hk, d, r = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim", "rot"))
    st = dict(case=case)
    st["q"] = _normal(g, (t, hq, d))
    st["k"] = _normal(g, (t, hk, d))
    st["v"] = _normal(g, (t, hk, d))
    st["positions"] = torch.randint(0, 73728, (t,), generator=g, device=DEV, dtype=torch.int32)
    # the rotary table of a serving engine: fp32 cosines and sines, the angles in fp64
    inv = 10000.0 ** (-torch.arange(r // 2, device=DEV, dtype=torch.float64) * 2 / r)
    ang = torch.arange(73728, device=DEV, dtype=torch.float64)[:, None] * inv
    st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
    pages = -(-(t + 64) // case["page"]) + 1
    slots = torch.randperm(pages * case["page"], generator=g, device=DEV)[:t].to(torch.int32)
    if case["idle"]:
        slots[case["idle"] - 1::case["idle"]] = -1
    st["slots"] = slots
    kind = torch.float8_e4m3fn if case["fp8"] else torch.bfloat16
    shape = (pages, case["page"], hk, d)
    st["k_cache"] = _normal(g, shape, dtype=kind)
    st["v_cache"] = _normal(g, shape, dtype=kind)
    if case["fp8"]:
        st["k_scale"] = torch.tensor(0.02, device=DEV)
        st["v_scale"] = torch.tensor(0.015, device=DEV)
    else:
        st["k_scale"] = st["v_scale"] = None
    st["q_out"] = torch.empty_like(st["q"])
    st["k_out"] = torch.empty_like(st["k"]) if case["k_out"] else None
    return st


def _decode_inputs(case, seed):
    g = _gen(seed)
    hq, hk, d, ps = (case[k] for k in ("q_heads", "kv_heads", "dim", "page"))
    lens = _lengths(case)
    n_pages = [-(-n // ps) for n in lens]
    total = sum(n_pages)
    pool = total + max(1, total // 16)
    st = dict(case=case, lens=lens)
    st["q"] = _normal(g, (len(lens), hq, d), 1.5)
    kind = torch.float8_e4m3fn if case["fp8"] else torch.bfloat16
    std = 50.0 if case["fp8"] else 1.0
    st["k_cache"] = _normal(g, (pool, ps, hk, d), std, kind)
    st["v_cache"] = _normal(g, (pool, ps, hk, d), std, kind)
    st["kv_indptr"] = _indptr(n_pages)
    st["kv_indices"] = torch.randperm(pool, generator=g, device=DEV)[:total].to(torch.int32)
    last = [n - (p - 1) * ps for n, p in zip(lens, n_pages)]
    st["kv_last_page_lens"] = torch.tensor(last, dtype=torch.int32, device=DEV)
    if case["fp8"]:
        st["k_scale"] = torch.tensor(0.02, device=DEV)
        st["v_scale"] = torch.tensor(0.015, device=DEV)
    else:
        st["k_scale"] = st["v_scale"] = None
    st["sm_scale"] = d ** -0.5
    st["o"] = torch.empty((len(lens), hq, d), dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.empty((len(lens), hq), dtype=torch.float32, device=DEV)
    return st


def _prompt_inputs(case, seed):
    g = _gen(seed)
    hq, hk, d, dv = (case[k] for k in ("q_heads", "kv_heads", "dim", "dim_v"))
    new, keys = _prompt_lengths(case)
    st = dict(case=case, new=new, keys=keys)
    st["q"] = _normal(g, (sum(new), hq, d), 1.5)
    st["k"] = _normal(g, (sum(keys), hk, d))
    st["v"] = _normal(g, (sum(keys), hk, dv))
    st["qo_indptr"] = _indptr(new)
    st["kv_indptr"] = _indptr(keys)
    st["sm_scale"] = d ** -0.5
    st["o"] = torch.empty((sum(new), hq, dv), dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.empty((sum(new), hq), dtype=torch.float32, device=DEV)
    return st


_INPUTS = {"append": _append_inputs, "decode": _decode_inputs, "prompt": _prompt_inputs}


def prepare(case, seed):
    st = _INPUTS[case["op"]](case, seed)
    if own:
        import paged_mla_latent_gb300 as pm
        if case["op"] == "decode":
            st["workspace"] = pm.make_gqa_decode_workspace(case["requests"], case["q_heads"],
                                                           case["kv_heads"], case["dim"], DEV)
        else:
            st["error_word"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return st


# ----------------------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _rotate(x, cos_sin, positions, neox):
    """fp32 (tokens, heads, dim) with its first columns rotated by the table's rows."""
    r = cos_sin.shape[1]
    row = cos_sin[positions.long()][:, None, :]
    c, s = row[..., :r // 2], row[..., r // 2:]
    rot, rest = x[..., :r], x[..., r:]
    if neox:
        a, b = rot[..., :r // 2], rot[..., r // 2:]
        return torch.cat([a * c - b * s, b * c + a * s, rest], dim=-1)
    a, b = rot[..., 0::2], rot[..., 1::2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2), rest], dim=-1)


def _stored(x, scale, kind):
    """fp32 values as the cache holds them."""
    if kind == torch.bfloat16:
        return x.to(kind)
    return (x / scale).clamp(-448, 448).to(kind)


def _plain_append(st):
    ps = st["case"]["page"]
    neox = st["case"]["neox"]
    q = _rotate(st["q"].float(), st["cos_sin"], st["positions"], neox)
    k = _rotate(st["k"].float(), st["cos_sin"], st["positions"], neox)
    live = torch.nonzero(st["slots"] >= 0)[:, 0]
    slot = st["slots"].long()[live]
    for cache, x, scale in ((st["k_cache"], k, st["k_scale"]),
                            (st["v_cache"], st["v"].float(), st["v_scale"])):
        new = _stored(x[live], scale, cache.dtype)
        if cache.dtype != torch.bfloat16:
            cache, new = cache.view(torch.uint8), new.view(torch.uint8)
        cache[slot // ps, slot % ps] = new
    out = dict(q=q.bfloat16(), k_cache=st["k_cache"], v_cache=st["v_cache"])
    if st["k_out"] is not None:
        out["k"] = k.bfloat16()
    return out


def _plain_decode(st):
    case = st["case"]
    hk, ps, d = case["kv_heads"], case["page"], case["dim"]
    group = case["q_heads"] // hk
    pages = st["kv_indices"].long()
    os, lses = [], []
    at = 0
    for b, n in enumerate(st["lens"]):
        ids = pages[at:at + -(-n // ps)]
        at += ids.numel()
        k = st["k_cache"].view(torch.uint8)[ids].view(st["k_cache"].dtype) if case["fp8"] else st["k_cache"][ids]
        v = st["v_cache"].view(torch.uint8)[ids].view(st["v_cache"].dtype) if case["fp8"] else st["v_cache"][ids]
        k = k.reshape(-1, hk, d)[:n].float()
        v = v.reshape(-1, hk, d)[:n].float()
        if case["fp8"]:
            k, v = k * st["k_scale"], v * st["v_scale"]
        q = st["q"][b].float().view(hk, group, d)
        s = torch.matmul(q, k.permute(1, 2, 0)) * st["sm_scale"]
        m = s.amax(dim=-1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(dim=-1, keepdim=True)
        os.append((torch.matmul(p, v.permute(1, 0, 2)) / z).reshape(-1, d))
        lses.append((m + torch.log(z)).reshape(-1))
    return dict(o=torch.stack(os).bfloat16(), lse=torch.stack(lses))


def _plain_prompt(st):
    case = st["case"]
    hk, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    o = torch.empty_like(st["o"])
    lse = torch.empty_like(st["lse"])
    q0 = k0 = 0
    for n, m in zip(st["new"], st["keys"]):
        step = max(64, min(2048, (1 << 28) // (group * m)))
        for h in range(hk):
            heads = slice(h * group, (h + 1) * group)
            k = st["k"][k0:k0 + m, h].float()
            v = st["v"][k0:k0 + m, h].float()
            for a in range(0, n, step):
                e = min(n, a + step)
                seen = m - n + e          # keys that the block's last query sees
                q = st["q"][q0 + a:q0 + e, heads].float().transpose(0, 1)
                s = torch.matmul(q, k[:seen].t()) * st["sm_scale"]
                at = torch.arange(m - n + a, seen, device=DEV)[:, None]
                s.masked_fill_(torch.arange(seen, device=DEV)[None, :] > at, -math.inf)
                top = s.amax(dim=-1, keepdim=True)
                s = s.sub_(top).exp_()
                z = s.sum(dim=-1, keepdim=True)
                o[q0 + a:q0 + e, heads] = (torch.matmul(s, v[:seen]) / z).transpose(0, 1).bfloat16()
                lse[q0 + a:q0 + e, heads] = (top + torch.log(z))[..., 0].t()
        q0 += n
        k0 += m
    return dict(o=o, lse=lse)


_plain = {"append": _plain_append, "decode": _plain_decode, "prompt": _plain_prompt}


def _own_append(st):
    import paged_mla_latent_gb300 as pm
    pm.mla_gqa_rope_and_cache(st["q"], st["k"], st["v"], st["positions"], st["cos_sin"],
                              int(st["case"]["neox"]), st["slots"], st["q_out"], st["k_cache"],
                              st["v_cache"], st["error_word"], k_scale=st["k_scale"],
                              v_scale=st["v_scale"], k_out=st["k_out"])
    out = dict(q=st["q_out"], k_cache=st["k_cache"], v_cache=st["v_cache"])
    if st["k_out"] is not None:
        out["k"] = st["k_out"]
    return out


def _own_decode(st):
    import paged_mla_latent_gb300 as pm
    pm.mla_gqa_decode(st["q"], st["k_cache"], st["v_cache"], st["o"], st["kv_indptr"],
                      st["kv_indices"], st["kv_last_page_lens"], st["sm_scale"],
                      k_scale=st["k_scale"], v_scale=st["v_scale"], lse_out=st["lse"],
                      workspace=st["workspace"])
    return dict(o=st["o"], lse=st["lse"])


def _own_prompt(st):
    import paged_mla_latent_gb300 as pm
    pm.mla_prompt_attention(st["q"], st["k"], st["v"], st["o"], st["qo_indptr"], st["kv_indptr"],
                            st["sm_scale"], error_word=st["error_word"], lse_out=st["lse"])
    return dict(o=st["o"], lse=st["lse"])


_own = {"append": _own_append, "decode": _own_decode, "prompt": _own_prompt}


# ----------------------------------------------------------------------------- fp64

def exact(case, seed):
    if case["op"] == "prompt" and work(case)["flops"] > 4e12:
        return None
    st = _INPUTS[case["op"]](case, seed)
    return {"append": _exact_append, "decode": _exact_decode, "prompt": _exact_prompt}[case["op"]](st)


def _exact_append(st):
    """Each pair as a complex number, turned by the table's unit (cos + i sin)."""
    case = st["case"]
    r, ps = case["rot"], case["page"]
    row = st["cos_sin"].double()[st["positions"].long()]
    turn = torch.complex(row[:, :r // 2], row[:, r // 2:])[:, None, :]
    first = torch.arange(r // 2, device=DEV) * (1 if case["neox"] else 2)
    second = first + (r // 2 if case["neox"] else 1)
    turned = []
    for x in (st["q"], st["k"]):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first] = z.real
        y[..., second] = z.imag
        turned.append(y)
    out = dict(q=turned[0])
    for name, new, scale in (("k_cache", turned[1], st["k_scale"]), ("v_cache", st["v"].double(), st["v_scale"])):
        cache = st[name].double().view(-1, case["kv_heads"], case["dim"])
        if scale is not None:
            new = (new / scale.double()).clamp(-448, 448)
        for some in torch.arange(case["tokens"], device=DEV).split(4096):
            some = some[st["slots"][some] >= 0]
            cache[st["slots"][some].long()] = new[some]
        out[name] = cache.view(-1, ps, case["kv_heads"], case["dim"])
    if st["k_out"] is not None:
        out["k"] = turned[1]
    return out


def _exact_decode(st):
    """One request and one KV head at a time; softmax through the log of the sum."""
    case = st["case"]
    hk = case["kv_heads"]
    group = case["q_heads"] // hk
    o = torch.empty(st["o"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(st["lse"].shape, dtype=torch.float64, device=DEV)
    ks = 1.0 if st["k_scale"] is None else st["k_scale"].double()
    vs = 1.0 if st["v_scale"] is None else st["v_scale"].double()
    start = st["kv_indptr"].tolist()
    for b, n in enumerate(st["lens"]):
        ids = st["kv_indices"][start[b]:start[b + 1]].long()
        some = {}
        for name in ("k_cache", "v_cache"):
            cache = st[name]
            bits = torch.uint8 if case["fp8"] else torch.int16
            some[name] = cache.view(bits).index_select(0, ids).view(cache.dtype).flatten(0, 1)[:n]
        for h in range(hk):
            k, v = some["k_cache"][:, h].double(), some["v_cache"][:, h].double()
            heads = slice(h * group, (h + 1) * group)
            s = torch.einsum("gd,nd->gn", st["q"][b, heads].double(), k) * (st["sm_scale"] * ks)
            l = torch.logsumexp(s, dim=1)
            lse[b, heads] = l
            o[b, heads] = torch.einsum("gn,nd->gd", torch.exp(s - l[:, None]), v) * vs
    return dict(o=o, lse=lse)


def _exact_prompt(st):
    """One request and one query head at a time, the keys that no query of a block sees left
    out; softmax through the log of the sum."""
    case = st["case"]
    group = case["q_heads"] // case["kv_heads"]
    o = torch.empty(st["o"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(st["lse"].shape, dtype=torch.float64, device=DEV)
    q0s, k0s = st["qo_indptr"].tolist(), st["kv_indptr"].tolist()
    for b, (n, m) in enumerate(zip(st["new"], st["keys"])):
        for h in range(case["q_heads"]):
            q = st["q"][q0s[b]:q0s[b + 1], h].double()
            k = st["k"][k0s[b]:k0s[b + 1], h // group].double()
            v = st["v"][k0s[b]:k0s[b + 1], h // group].double()
            for rows in torch.arange(n, device=DEV).split(1024):
                seen = m - n + int(rows[-1]) + 1
                s = st["sm_scale"] * (q[rows] @ k[:seen].T)
                future = torch.arange(seen, device=DEV) - (m - n) > rows[:, None]
                s = torch.where(future, torch.full_like(s, -math.inf), s)
                l = torch.logsumexp(s, dim=1, keepdim=True)
                o[q0s[b] + rows, h] = torch.exp(s - l) @ v[:seen]
                lse[q0s[b] + rows, h] = l[:, 0]
    return dict(o=o, lse=lse)
