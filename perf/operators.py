"""Serving over a paged key/value cache: the two operators of one step, as cases to be timed and compared.

``append``  rotates the step's new queries and keys by their positions and writes the keys and values into the pages of
            the cache, in BF16 or as E4M3 with one power-of-two scale for each page and key/value head
            (``attn_cache_append``).
``attend``  attention of the new queries over the pages of their sequences (``attn_fwd_cache``): single tokens, a few
            drafted tokens, chunks of a prompt; causal, with or without a window.

Where ``own`` is false ``run`` computes an operator in elementary torch operations in FP32 (angles in FP64); where it is
true it calls the framework.  ``exact`` computes it in FP64, sequence by sequence.

Heads are the package's own (16 query heads over 16, 2 or 1 key/value heads of 128), lengths run from its 256-token
case to several times its 32K one.
"""
import math
import random

import torch

own = False

D = 128
H_Q = 16
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One user, one token: what counts is the latency of the call.
        dict(name="append_b1_n1_kv2_e4m3_p64", op="append", batch=1, ctx=700, new=1, h_kv=2, page=64, kind="e4m3",
             rotary=128, interleaved=False, ragged=False),
        # A full serving batch, one token each.
        dict(name="append_b256_n1_kv2_e4m3_p16", op="append", batch=256, ctx=4096, new=1, h_kv=2, page=16, kind="e4m3",
             rotary=128, interleaved=False, ragged=True),
        # Drafted tokens: pages are entered in the middle, some scales grow and old tokens are coded again.
        dict(name="append_b64_n5_kv16_e4m3_p32", op="append", batch=64, ctx=1000, new=5, h_kv=16, page=32, kind="e4m3",
             rotary=128, interleaved=False, ragged=True),
        # Prompts of different lengths into a BF16 cache; half of each head rotates, in neighbouring pairs.
        dict(name="append_b8_ragged2048_kv16_bf16_p128", op="append", batch=8, ctx=2048, new=2048, h_kv=16, page=128,
             kind="bf16", rotary=64, interleaved=True, ragged=True),
        # One long prompt into an 8-bit cache.
        dict(name="append_b1_n32768_kv2_e4m3_p64", op="append", batch=1, ctx=32768, new=32768, h_kv=2, page=64,
             kind="e4m3", rotary=128, interleaved=False, ragged=False),
        # One user, one token, a short dialogue.
        dict(name="attend_b1_n1_ctx500_kv2_e4m3_p16", op="attend", batch=1, ctx=500, new=1, h_kv=2, page=16,
             kind="e4m3", window=-1, ragged=False),
        # A serving batch of dialogues of all lengths, grouped heads, 8 bits.
        dict(name="attend_b64_n1_ctx8192_kv2_e4m3_p64", op="attend", batch=64, ctx=8192, new=1, h_kv=2, page=64,
             kind="e4m3", window=-1, ragged=True),
        # One very long document: the keys are the only axis to divide.
        dict(name="attend_b1_n1_ctx262144_kv2_e4m3_p64", op="attend", batch=1, ctx=262144, new=1, h_kv=2, page=64,
             kind="e4m3", window=-1, ragged=False),
        # A head of keys for each head of queries, BF16 cache in small pages.
        dict(name="attend_b16_n1_ctx4096_kv16_bf16_p16", op="attend", batch=16, ctx=4096, new=1, h_kv=16, page=16,
             kind="bf16", window=-1, ragged=True),
        # Drafted tokens checked in one pass, one key/value head for all queries.
        dict(name="attend_b32_n5_ctx16384_kv1_e4m3_p32", op="attend", batch=32, ctx=16384, new=5, h_kv=1, page=32,
             kind="e4m3", window=-1, ragged=True),
        # Long dialogues under a sliding window.
        dict(name="attend_b128_n1_ctx32768_w2048_kv2_bf16_p128", op="attend", batch=128, ctx=32768, new=1, h_kv=2,
             page=128, kind="bf16", window=2048, ragged=True),
        # Chunks of prompts over what the cache already holds.
        dict(name="attend_b4_n1024_ctx16384_kv2_e4m3_p64", op="attend", batch=4, ctx=16384, new=1024, h_kv=2, page=64,
             kind="e4m3", window=-1, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    h_kv = rng.choice([1, 2, 4, 8, 16])
    page = rng.choice([8, 16, 24, 32, 48, 64, 128, 256])
    kind = rng.choice(["e4m3", "e4m3", "bf16"])
    ragged = rng.random() < 0.7
    if rng.random() < 0.4:
        if rng.random() < 0.5:
            batch, new = _log_int(rng, 1, 256), _log_int(rng, 1, 8)
        else:
            batch = _log_int(rng, 1, 16)
            new = _log_int(rng, 9, max(9, 16384 // batch))
        ctx = max(new, _log_int(rng, 1, 4096))
        # the caches of one case stay within the largest listed one's
        batch = max(1, min(batch, (1 << 19) // (ctx * h_kv) or 1))
        return dict(op="append", batch=batch, ctx=ctx, new=new, h_kv=h_kv, page=page, kind=kind,
                    rotary=rng.choice([0, 32, 64, 96, 128, 128]), interleaved=rng.random() < 0.4, ragged=ragged)
    if rng.random() < 0.7:
        new = rng.choice([1, 1, 1, 2, 3, 5, 8])
        ctx = max(new, _log_int(rng, 1, 131072))
        keys = (1 << 20) // (2 if kind == "bf16" else 1) // h_kv  # keys of one head in all sequences
        batch = max(1, min(_log_int(rng, 1, 128), keys // ctx))
    else:
        batch = _log_int(rng, 1, 8)
        new = _log_int(rng, 9, 1024)
        ctx = max(new, _log_int(rng, 16, 16384))
        batch = max(1, min(batch, (1 << 23) // (new * ctx)))
    return dict(op="attend", batch=batch, ctx=ctx, new=new, h_kv=h_kv, page=page, kind=kind,
                window=_log_int(rng, 1, 4096) if rng.random() < 0.25 else -1, ragged=ragged)


def _lengths(case):
    """(keys, new tokens) of each sequence: the case's own, whatever the seed."""
    rng = random.Random(case["batch"] * 1000003 + case["ctx"] * 101 + case["new"])
    lens, news = [], []
    for _ in range(case["batch"]):
        n = case["new"]
        if case["ragged"] and n > 8:
            n = rng.randint(1, n)
        lo = max(n, case["ctx"] // 4)
        lens.append(rng.randint(lo, max(lo, case["ctx"])) if case["ragged"] else max(n, case["ctx"]))
        news.append(n)
    return lens, news


def _visible(length, n, window):
    """(query, key) pairs that see each other in one sequence, and the keys that any query sees."""
    pairs = 0
    for i in range(n):
        last = length - n + i
        pairs += last + 1 if window < 0 else min(last + 1, window + 1)
    first = 0 if window < 0 else max(0, length - n - window)
    return pairs, length - first


def work(case):
    lens, news = _lengths(case)
    total, h_kv = sum(news), case["h_kv"]
    size = 1 if case["kind"] == "e4m3" else 2
    if case["op"] == "append":
        bytes_ = total * (h_kv * D * 2 * (2 + size) + H_Q * D * 4) + 8 * len(lens)
        if size == 1:  # a scale for each page entered, key and value
            bytes_ += 8 * h_kv * sum((n - 1) // case["page"] + 1 for n in news)
        return {"bytes": bytes_, "flops": total * (H_Q + h_kv) * 3 * case["rotary"]}
    bytes_, pairs = total * H_Q * (D * 4 + 4), 0
    for length, n in zip(lens, news):
        p, keys = _visible(length, n, case["window"])
        pairs += p
        pages = -(-keys // case["page"])
        bytes_ += keys * h_kv * D * 2 * size + pages * (4 + (8 * h_kv if size == 1 else 0))
    return {"bytes": bytes_, "flops": 4 * pairs * H_Q * D}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    lens, news = _lengths(case)
    batch, page, h_kv, total = len(lens), case["page"], case["h_kv"], sum(news)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    pages_of = [-(-n // page) for n in lens]
    max_pages, num_pages = max(pages_of), sum(pages_of) + 3
    # Pages are handed out in no order; a table's entries past a sequence's last page are never looked at.
    order = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    counts = torch.tensor(pages_of, device=dev)
    slot = torch.arange(max_pages, device=dev)[None]
    first = torch.cumsum(counts, 0) - counts
    held = slot < counts[:, None]
    table = torch.where(held, order[(first[:, None] + slot).clamp(max=num_pages - 1)], -1).contiguous()
    seqlens = torch.tensor(lens, dtype=torch.int32, device=dev)
    cu = torch.zeros(batch + 1, dtype=torch.int32, device=dev)
    cu[1:] = torch.cumsum(torch.tensor(news, device=dev), 0)
    uniform = len(set(news)) == 1

    # What the cache holds: each head's keys and values have a size of their own, a page varies around it.  The
    # slots past a sequence's end are whatever was there (zeros for append, NaN for attend).
    shape = (num_pages, page, h_kv, D)
    filled = torch.zeros(num_pages, dtype=torch.int64, device=dev)
    inside = (seqlens[:, None] - slot * page).clamp(0, page)
    filled[table[held].long()] = inside[held].long()
    if case["op"] == "append":  # only what the earlier steps wrote
        before = (seqlens - cu.diff()).long()
        filled.zero_()
        filled[table[held].long()] = (before[:, None] - slot * page).clamp(0, page)[held]
    empty = torch.arange(page, device=dev)[None] >= filled[:, None]
    state = {"op": case["op"], "kind": case["kind"], "page": page, "h_kv": h_kv, "total": total, "batch": batch,
             "table": table, "seqlens": seqlens, "cu": cu, "uniform": uniform, "max_new": max(news)}
    for name, size in (("k", 1.0), ("v", 0.7)):
        x = torch.randn(shape, generator=g, device=dev)
        x *= size * (0.5 + torch.rand((num_pages, 1, h_kv, 1), generator=g, device=dev))
        if case["kind"] == "e4m3":
            # the smallest power of two that holds the page, as it would be kept
            top = torch.where(empty[:, :, None, None], 0.0, x).abs().amax((1, 3))
            m, e = torch.frexp(top / E4M3_MAX)
            e = e - (m == 0.5).to(e.dtype)
            scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), 0.0)
            x = torch.where(scale[:, None, :, None] > 0, x / scale[:, None, :, None], 0.0)
            state[name + "_scale"] = scale.contiguous()
            rest = 0x7F  # NaN
        else:
            state[name + "_scale"], rest = None, 0x7FC0
        x = x.to(torch.float8_e4m3fn if case["kind"] == "e4m3" else torch.bfloat16).contiguous()
        bits = x.view(torch.uint8 if case["kind"] == "e4m3" else torch.int16)
        bits.masked_fill_(empty[:, :, None, None], 0 if case["op"] == "append" else rest)
        state[name + "_pages"] = x

    if case["op"] == "append":
        # the three are slices of one projection's result, as a model leaves them
        qkv = torch.randn((total, H_Q + 2 * h_kv, D), generator=g, device=dev)
        qkv *= 0.5 + 2 * torch.rand((total, 1, 1), generator=g, device=dev)
        qkv = qkv.to(torch.bfloat16)
        state.update(q=qkv[:, :H_Q], k=qkv[:, H_Q:H_Q + h_kv], v=qkv[:, H_Q + h_kv:], rotary=case["rotary"],
                     interleaved=case["interleaved"], q_out=torch.empty(total, H_Q, D, dtype=torch.bfloat16, device=dev))
        half = torch.arange(case["rotary"] // 2, device=dev, dtype=torch.float64)
        state["inv_freq"] = (10000.0 ** (-2 * half / max(case["rotary"], 1))).float() if case["rotary"] else None
    else:
        state["q"] = torch.randn((total, H_Q, D), generator=g, device=dev).to(torch.bfloat16)
        state.update(window=case["window"], scale=1.0 / math.sqrt(D),
                     o=torch.empty(total, H_Q, D, dtype=torch.bfloat16, device=dev),
                     lse=torch.empty(H_Q, total, dtype=torch.float32, device=dev))
    if own:
        # the handle and the workspace that a server keeps from step to step
        from scaled_dot_product_10_b200 import attn
        state["cache"] = attn.KVCache(state["k_pages"], state["v_pages"], state["k_scale"], state["v_scale"])
        if case["op"] == "attend":
            state["workspace"] = torch.empty(attn.cache_workspace_bytes(H_Q, h_kv, max(news)), dtype=torch.uint8,
                                             device=dev)
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _own_append(state) if state["op"] == "append" else _own_attend(state)
    return _plain_append(state) if state["op"] == "append" else _plain_attend(state)


def _own_append(s):
    from scaled_dot_product_10_b200 import attn
    q_out = attn.attn_cache_append(s["cache"], s["k"], s["v"], s["table"], s["seqlens"],
                                   cu_seqlens=None if s["uniform"] else s["cu"], max_seqlen=s["max_new"], q=s["q"],
                                   q_out=s["q_out"], inv_freq=s["inv_freq"], interleaved=s["interleaved"])
    return _cache_out(s, q_out)


def _own_attend(s):
    from scaled_dot_product_10_b200 import attn
    o, lse = attn.attn_fwd_cache(s["q"], s["cache"], s["table"], s["seqlens"],
                                 cu_seqlens_q=None if s["uniform"] else s["cu"], max_seqlen_q=s["max_new"],
                                 causal=True, window_left=s["window"], scale=s["scale"], o=s["o"], lse=s["lse"],
                                 workspace=s["workspace"])
    return {"o": o, "lse": lse}


def _cache_out(s, q_out):
    out = {"q": q_out, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["kind"] == "e4m3":
        out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


def _rotate(x, angle, rotary, interleaved):
    """x [tokens, heads, 128] FP32 rotated by angle [tokens, rotary / 2] (FP64)."""
    if rotary == 0:
        return x
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if interleaved:
        a, b = x[..., 0:rotary:2], x[..., 1:rotary:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :rotary // 2], x[..., rotary // 2:rotary]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., rotary:]), -1)


def _pow2_scale(bound):
    """The smallest power of two s with bound <= 448 s; 0 for 0."""
    m, e = torch.frexp(bound)  # bound = m 2^e with m in [1/2, 1); 448 = (7/8) 2^9
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(bound > 0, torch.ldexp(torch.ones_like(bound), e), 0.0)


def _plain_append(s):
    page, rot = s["page"], s["rotary"]
    token = torch.arange(s["total"], device=s["cu"].device)
    seq = torch.searchsorted(s["cu"][1:].contiguous().long(), token, right=True)
    ends = s["cu"][1:].long()
    pos = s["seqlens"].long()[seq] - (ends[seq] - token)
    pid = s["table"][seq, pos // page].long()
    slot = pos % page
    angle = pos.double()[:, None] * s["inv_freq"].double()[None] if rot else None
    q = _rotate(s["q"].float(), angle, rot, s["interleaved"]).to(torch.bfloat16)
    for name in ("k", "v"):
        x = s[name].float()
        pages, scale = s[name + "_pages"], s[name + "_scale"]
        y = _rotate(x, angle, rot, s["interleaved"]) if name == "k" else x
        if s["kind"] == "bf16":
            pages[pid, slot] = y.to(torch.bfloat16)
            continue
        # the bound of a key's rotated pair is |a| + |b|, which no rotation of it exceeds
        top = x.abs()
        if name == "k" and rot:
            if s["interleaved"]:
                pair = top[..., 0:rot:2] + top[..., 1:rot:2]
            else:
                pair = top[..., :rot // 2] + top[..., rot // 2:rot]
            top = torch.cat((pair, top[..., rot:]), -1)
        top = top.amax(-1)  # [tokens, heads]
        bound = torch.zeros_like(scale).scatter_reduce_(0, pid[:, None].expand_as(top), top, "amax")
        touched = torch.zeros_like(scale[:, 0], dtype=torch.bool)
        touched[pid] = True
        begin = torch.full((pages.shape[0],), page, device=pid.device).scatter_reduce_(0, pid, slot, "amin")
        old = torch.where((touched & (begin > 0))[:, None] | ~touched[:, None], scale, 0.0)
        new = torch.maximum(old, _pow2_scale(bound))
        factor = torch.where(new > 0, old / new, 1.0)
        # only where a scale has grown are the page's older tokens coded again
        grown = (touched[:, None] & (old > 0) & (factor < 1)).any(1)
        codes = pages.view(torch.uint8)
        again = codes[grown].view(pages.dtype).float() * factor[grown][:, None, :, None]
        codes[grown] = again.to(pages.dtype).view(torch.uint8)
        scale.copy_(new)
        ns = new[pid][..., None]
        code = torch.where(ns > 0, y / ns, 0.0).clamp(-E4M3_MAX, E4M3_MAX).to(pages.dtype)
        codes[pid, slot] = code.view(torch.uint8)
    return _cache_out(s, q)


def _gathered(s, name):
    """The pages of every sequence in order, [batch, keys, heads, 128] FP32, zeros past the sequence's end."""
    ids = s["table"].long().clamp(min=0)
    x = s[name + "_pages"][ids] if s["kind"] == "bf16" else s[name + "_pages"].view(torch.uint8)[ids].view(torch.float8_e4m3fn)
    x = x.float()
    if s["kind"] == "e4m3":
        x = x * s[name + "_scale"][ids][:, :, None, :, None]
    x = x.flatten(1, 2)
    there = torch.arange(x.shape[1], device=x.device)[None] < s["seqlens"][:, None]
    return torch.where(there[:, :, None, None], x, 0.0)


def _plain_attend(s):
    h_kv, group = s["h_kv"], H_Q // s["h_kv"]
    k, v = _gathered(s, "k"), _gathered(s, "v")
    batch, keys = k.shape[:2]
    n = s["max_new"]
    news = s["cu"].diff().long()
    row = torch.arange(n, device=k.device)[None]
    real = row < news[:, None]  # [batch, n]
    at = (s["cu"][:-1, None].long() + row).clamp(max=s["total"] - 1)
    q = s["q"].float()[at]  # [batch, n, heads, 128]
    q = q.view(batch, n, h_kv, group, D).permute(0, 2, 3, 1, 4).reshape(batch, h_kv, group * n, D)
    x = (q @ k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(batch, h_kv, group, n, keys)
    last = s["seqlens"].long()[:, None] - news[:, None] + row  # the last key each query sees
    j = torch.arange(keys, device=k.device)
    seen = j <= last[..., None]
    if s["window"] >= 0:
        seen &= j >= (last - s["window"])[..., None]
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = x.view(batch, h_kv, group * n, keys) @ v.permute(0, 2, 1, 3)
    o = o.view(batch, h_kv, group, n, D) / torch.where(total > 0, total, 1.0)
    lse = (m + total.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, n, H_Q, D)
    lse = lse.permute(0, 3, 1, 2).reshape(batch, n, H_Q)
    return {"o": o[real].to(torch.bfloat16), "lse": lse[real].T.contiguous()}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    lens, news = s["seqlens"].tolist(), s["cu"].diff().tolist()
    return _exact_append(s, lens, news) if case["op"] == "append" else _exact_attend(s, lens, news)


def _exact_turned(x, first, rot, inv_freq, interleaved):
    """Complex multiplication by exp(i position frequency), FP64."""
    if rot == 0:
        return x
    pos = torch.arange(first, first + x.shape[0], device=x.device, dtype=torch.float64)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos[:, None] * inv_freq.double())[:, None]
    y = x.clone()
    if interleaved:
        z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_append(s, lens, news):
    rot, page = s["rotary"], s["page"]
    out = {"q": torch.empty(s["total"], H_Q, D, dtype=torch.float64, device=s["q"].device)}
    values = {n: s[n + "_pages"].double() for n in ("k", "v")}
    scales = {n: s[n + "_scale"].double() for n in ("k", "v")} if s["kind"] == "e4m3" else None
    table, row = s["table"].tolist(), 0
    for b, (length, n) in enumerate(zip(lens, news)):
        first = length - n
        rows = slice(row, row + n)
        row += n
        out["q"][rows] = _exact_turned(s["q"][rows].double(), first, rot, s["inv_freq"], s["interleaved"])
        for name in ("k", "v"):
            x = s[name][rows].double()
            y = _exact_turned(x, first, rot, s["inv_freq"], s["interleaved"]) if name == "k" else x
            length_of = x.abs()
            if name == "k" and rot:
                a = length_of[..., 0:rot:2] if s["interleaved"] else length_of[..., :rot // 2]
                c = length_of[..., 1:rot:2] if s["interleaved"] else length_of[..., rot // 2:rot]
                length_of = torch.cat((a + c, length_of[..., rot:]), -1)
            for p in range(first // page, (length - 1) // page + 1):
                lo, hi = max(first, p * page), min(length, (p + 1) * page)
                part, pid = slice(lo - first, hi - first), table[b][p]
                here = slice(lo - p * page, hi - p * page)
                if scales is None:
                    values[name][pid, here] = y[part]
                    continue
                bound = length_of[part].amax((0, 2))
                want = torch.exp2(torch.round(torch.log2(bound / E4M3_MAX)))  # the power nearest, then the first to hold it
                want = torch.where(want * E4M3_MAX < bound, 2 * want, want)
                want = torch.where(bound > 0, want, 0.0)
                old = scales[name][pid] if lo > p * page else torch.zeros_like(bound)
                new = torch.maximum(old, want)
                old_rows = values[name][pid, :lo - p * page]
                old_rows *= torch.where(new > 0, old / torch.where(new > 0, new, 1.0), 1.0)[None, :, None]
                scales[name][pid] = new
                values[name][pid, here] = y[part] / torch.where(new > 0, new, 1.0)[None, :, None]
    out.update(k_pages=values["k"], v_pages=values["v"])
    if scales is not None:
        out.update(k_scale=scales["k"], v_scale=scales["v"])
    return out


def _exact_attend(s, lens, news):
    h_kv, group, page = s["h_kv"], H_Q // s["h_kv"], s["page"]
    dev = s["q"].device
    o = torch.zeros(s["total"], H_Q, D, dtype=torch.float64, device=dev)
    lse = torch.full((H_Q, s["total"]), float("-inf"), dtype=torch.float64, device=dev)
    row = 0
    for b, (length, n) in enumerate(zip(lens, news)):
        ids = s["table"][b, :-(-length // page)].long()
        last = torch.arange(length - n, length, device=dev)
        first = 0 if s["window"] < 0 else max(0, length - n - s["window"])
        j = torch.arange(first, length, device=dev)
        hidden = j[None] > last[:, None]
        if s["window"] >= 0:
            hidden |= j[None] < last[:, None] - s["window"]
        for h in range(h_kv):
            kv = []
            for name in ("k", "v"):
                x = s[name + "_pages"][:, :, h].view(torch.uint8 if s["kind"] == "e4m3" else torch.bfloat16)[ids]
                x = x.view(torch.float8_e4m3fn).double() if s["kind"] == "e4m3" else x.double()
                if s["kind"] == "e4m3":
                    x = x * s[name + "_scale"][ids, h].double()[:, None, None]
                kv.append(x.reshape(-1, D)[first:length])
            for e in range(h * group, (h + 1) * group):
                x = s["q"][row:row + n, e].double() @ kv[0].T * s["scale"]
                x[hidden] = float("-inf")
                lse[e, row:row + n] = torch.logsumexp(x, -1)
                o[row:row + n, e] = torch.softmax(x, -1) @ kv[1]
        row += n
    return {"o": o, "lse": lse}
