"""Attention and its key-value cache as measured cases: causal attention over packed prompts with
grouped heads (forward and backward), attention of one new token over a paged cache in bf16 or
8 bits, block tables and slot maps from request lengths, and new keys and values written into
the cache's pages.

`run` computes each operator in plain torch operations, or with `own` through the library's
entry points; `exact` is the same definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
F64 = torch.float64
NEG = float("-inf")


def listed():
    return [
        # one short chat prompt at the head size of small models, where launch latency counts
        {"name": "attention 37 tokens", "op": "attn", "n": 37, "seqs": 1, "heads": 16, "kv": 4, "d": 64, "causal": True, "prefix": 0},
        # a training batch at the 8B layer's heads: 8192 tokens of sixteen ragged rollouts
        {"name": "attention 8192 tokens of 16", "op": "attn", "n": 8192, "seqs": 16, "heads": 32, "kv": 8, "d": 128, "causal": True, "prefix": 0},
        # one long agentic rollout: the longest row the trainer packs
        {"name": "attention 16384 tokens", "op": "attn", "n": 16384, "seqs": 1, "heads": 32, "kv": 8, "d": 128, "causal": True, "prefix": 0},
        # a small client's step: an odd number of tokens in seven short datums
        {"name": "attention backward 1003 tokens of 7", "op": "attn_bwd", "n": 1003, "seqs": 7, "heads": 16, "kv": 2, "d": 64, "causal": True, "prefix": 0},
        # the training batch's backward, few long sequences among short ones
        {"name": "attention backward 8192 tokens of 6", "op": "attn_bwd", "n": 8192, "seqs": 6, "heads": 32, "kv": 8, "d": 128, "causal": True, "prefix": 0},
        # one sequence decoding: latency, the length split over the chip
        {"name": "decode 1x4001", "op": "decode", "n": 1, "len": 4001, "heads": 32, "kv": 8, "d": 128, "page": 16, "x8": False},
        # a rollout batch in bf16 at the 8B layer's heads
        {"name": "decode 64x8000", "op": "decode", "n": 64, "len": 8000, "heads": 32, "kv": 8, "d": 128, "page": 16, "x8": False},
        # the 30B-A3B layer's four key heads, a large rollout batch on an 8-bit cache
        {"name": "decode 8 bits 250x3000", "op": "decode", "n": 250, "len": 3000, "heads": 32, "kv": 4, "d": 128, "page": 64, "x8": True},
        # a decoding step's bookkeeping: one token each, a few requests ended
        {"name": "tables 64 requests", "op": "tables", "n": 64, "len": 4000, "new": 1, "page": 16},
        # a prefill wave: many requests' prompts enter the cache at once
        {"name": "tables 1000 requests of prompts", "op": "tables", "n": 1000, "len": 500, "new": 120, "page": 16},
        # a decoding step's rows into the cache
        {"name": "write 64 rows", "op": "write", "n": 64, "kv": 8, "d": 128, "page": 16, "x8": False},
        # a prefill's rows into an 8-bit cache, an odd count
        {"name": "write 8 bits 16381 rows", "op": "write", "n": 16381, "kv": 8, "d": 128, "page": 16, "x8": True},
    ]


def _log(rng, lo, hi):
    return lo * (hi / lo) ** rng.random()


def draw(rng):
    op = rng.choice(("attn", "attn", "attn_bwd", "attn_bwd", "decode", "decode", "tables", "write"))
    d, page = rng.choice((64, 128, 128)), rng.choice((16, 16, 32, 64, 128))
    kv = rng.choice((1, 2, 4, 8))
    heads = kv * rng.choice((1, 2, 4, 5, 8) if kv < 8 else (1, 2, 3, 4))
    if op in ("attn", "attn_bwd"):
        n = round(_log(rng, 1, 11000 if op == "attn" else 3300))
        return {"op": op, "n": n, "seqs": min(n, round(_log(rng, 1, 64))), "heads": heads, "kv": kv, "d": d,
                "causal": rng.random() < 0.8, "prefix": round(_log(rng, 1, 400)) if rng.random() < 0.25 else 0}
    if op == "decode":
        n = round(_log(rng, 1, 256))
        return {"op": op, "n": n, "len": round(_log(rng, 1, min(32000, 250000 // n))), "heads": heads, "kv": kv, "d": d, "page": page,
                "x8": rng.random() < 0.5}
    if op == "tables":
        n = round(_log(rng, 1, 1000))
        return {"op": op, "n": n, "len": round(_log(rng, 1, 500)), "new": rng.choice((1, round(_log(rng, 1, 100)))), "page": page}
    return {"op": op, "n": round(_log(rng, 1, 12000)), "kv": kv, "d": d, "page": page, "x8": rng.random() < 0.5}


# ---------------------------------------------------------------- layouts: the case's, not the seed's

def _layout(c):
    return np.random.default_rng([ord(ch) for ch in c["op"]] + [int(c[k]) for k in sorted(c) if k not in ("op", "name")])


def _split(rng, total, parts):
    """`total` in `parts` lengths of one or more whose sizes vary as those of rollouts do."""
    w = np.exp(rng.standard_normal(parts))
    sizes = 1 + np.floor(w / w.sum() * (total - parts)).astype(np.int64)
    sizes[int(np.argmax(sizes))] += total - int(sizes.sum())
    return sizes


def _attn_lens(c):
    rng = _layout(c)
    lq = _split(rng, c["n"], c["seqs"])
    # keys of earlier chunks in front of the queries, as where a prompt goes through in pieces
    return lq, lq + (rng.integers(0, 2 * c["prefix"] + 1, c["seqs"]) if c["prefix"] else 0)


def _decode_lens(c):
    rng = _layout(c)
    lens = np.maximum(1, (c["len"] * rng.uniform(0.3, 1.0, c["n"])).astype(np.int64))
    lens[0] = c["len"]
    return lens


def _table_lens(c):
    """Cached and new lengths: a few requests have ended (-1), a few wait (0), a few are new (cached 0)."""
    rng, n = _layout(c), c["n"]
    cached = rng.integers(0, 2 * c["len"], n)
    new = rng.integers(1, 2 * c["new"], n) if c["new"] > 1 else np.ones(n, np.int64)
    kind = rng.random(n)
    new = np.where(kind < 0.05, -1, np.where(kind < 0.1, 0, new))
    return np.where(kind > 0.8 if c["new"] > 1 else kind > 0.97, 0, cached), new


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _up(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype)).to(DEV)


def _cu(lens):
    return _up(np.concatenate([[0], np.cumsum(lens)]))


def _heads(g, n, heads, d, gain):
    """Rows of unit RMS for each head, as behind a norm over the head, times the head's gain."""
    return _randn(g, n, heads, d) * (gain[:, None] if gain is not None else 1.0)


def _gains(heads):
    return torch.linspace(0.5, 3.0, heads, device=DEV)  # flat heads and peaked ones


def _prepare_attn(c, g):
    n, hq, hk, d = c["n"], c["heads"], c["kv"], c["d"]
    lq, lk = _attn_lens(c)
    nk = int(lk.sum())
    s = {"lq": lq.tolist(), "lk": lk.tolist(), "cu_q": _cu(lq), "cu_k": _cu(lk), "scale": 1.0 / math.sqrt(d), "causal": c["causal"]}
    if nk == n:  # one fused projection's output, and one buffer for its gradient
        qkv = torch.empty(n, hq + 2 * hk, d, dtype=torch.bfloat16, device=DEV)
        s |= {"q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "v": qkv[:, hq + hk:]}
        grad = torch.empty_like(qkv)
        grads = {"dq": grad[:, :hq], "dk": grad[:, hq:hq + hk], "dv": grad[:, hq + hk:]}
    else:
        s |= {"q": torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV), "k": torch.empty(nk, hk, d, dtype=torch.bfloat16, device=DEV),
              "v": torch.empty(nk, hk, d, dtype=torch.bfloat16, device=DEV)}
        grads = {"d" + k: torch.empty_like(s[k]) for k in "qkv"}
    s["q"].copy_(_heads(g, n, hq, d, _gains(hq)))
    s["k"].copy_(_heads(g, nk, hk, d, None))
    s["v"].copy_(_randn(g, nk, hk, d))
    s |= {"o": torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV), "lse": torch.empty(hq, n, device=DEV),
          "ws": torch.zeros(256 + 8 * hq * n, dtype=torch.uint8, device=DEV)}
    if c["op"] == "attn_bwd":
        out = _plain_attn(s)
        s |= grads | {"o": out["o"], "lse": out["lse"], "dout": (0.01 * _randn(g, n, hq, d)).to(torch.bfloat16)}
    return s


def _pow2(b):
    return (b.to(torch.int32) << 23).view(torch.float32)


def _quantize8(v):
    """v fp32 [..., d] -> (e4m3 codes [..., d], scale bytes [..., d/32]): the least power of two with max|v| <= 448 scale."""
    blocks = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    bits = blocks.abs().amax(-1).contiguous().view(torch.int32)
    b = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)).clamp(min=1)
    return (blocks / _pow2(b)[..., None]).to(torch.float8_e4m3fn).reshape(v.shape), b.to(torch.uint8)


def _prepare_cache(c, g, n_pages):
    shape = (n_pages, c["kv"], c["page"], c["d"])
    s = {"k_scales": None, "v_scales": None}
    for name in ("k", "v"):
        if c["x8"]:
            codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
            scales = torch.empty(*shape[:3], c["d"] // 32, dtype=torch.uint8, device=DEV)
            step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
            for r in range(0, n_pages, step):
                m = min(step, n_pages - r)
                codes[r:r + m], scales[r:r + m] = _quantize8(_randn(g, m, *shape[1:]))
            s |= {name + "_cache": codes, name + "_scales": scales.view(torch.float8_e8m0fnu)}
        else:
            s[name + "_cache"] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    return s


def _perm(g, n):
    return torch.randperm(n, generator=g, device=DEV, dtype=torch.int32)


def _tables_of(counts, pages, width):
    """Block tables [n][width] from a list of pages, in request order; entries behind a request's pages are 0."""
    first = np.cumsum(counts) - counts
    j = np.arange(width)
    at = np.where(j < counts[:, None], first[:, None] + j, 0)
    return torch.where(_up(j < counts[:, None], np.bool_), pages[_up(at, np.int64)], 0)


def _prepare_decode(c, g):
    lens = _decode_lens(c)
    pages = -(-lens // c["page"])
    n_pages = int(pages.sum()) + 3
    width = int(pages.max()) + 1
    n, hq, d = c["n"], c["heads"], c["d"]
    return _prepare_cache(c, g, n_pages) | {
        "table": _tables_of(pages, _perm(g, n_pages), width), "lens": _up(lens), "q": _heads(g, n, hq, d, _gains(hq)).to(torch.bfloat16),
        "o": torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV), "lse": torch.empty(n, hq, device=DEV), "scale": 1.0 / math.sqrt(d),
        "max_len": c["len"], "kv": c["kv"], "page": c["page"], "n_pages": n_pages}


def _prepare_tables(c, g):
    cached, new = _table_lens(c)
    n, ps = c["n"], c["page"]
    owned = -(-cached // ps)
    after = np.where(new < 0, owned, -(-(cached + np.maximum(new, 0)) // ps))
    n_pages = int(after.sum()) + 5
    perm = _perm(g, n_pages)
    held, width = int(owned.sum()), int(max(after.max(), 1)) + 4
    # the free pages lie in the ring from some head on; the counters have run for a while
    head = 3 * n_pages + int(torch.randint(0, n_pages, (1,), generator=g, device=DEV))
    tail = head + n_pages - held
    ring = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
    ring[(head + torch.arange(n_pages - held, device=DEV)) % n_pages] = perm[held:]
    total = int(np.maximum(new, 0).sum())
    slots = max(64, -(-total // 64) * 64)  # a batch padded to whole tiles of rows
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"cached": _up(cached), "new": _up(new), "table": _tables_of(owned, perm, width), "ring": ring,
            "state": _up([head, tail], np.int64), "state_out": torch.zeros(2, dtype=torch.int64, device=DEV), "seq_lens": i32(n),
            "cu": i32(n + 1), "slots": i32(slots), "positions": i32(slots), "token_seqs": i32(slots), "page": ps, "n_pages": n_pages}


def _prepare_write(c, g):
    n, ps = c["n"], c["page"]
    n_pages = -(-n // ps) + 64
    s = _prepare_cache(c, g, n_pages)
    fused = torch.empty(n, 2 * c["kv"], c["d"], dtype=torch.bfloat16, device=DEV)
    fused.copy_(_randn(g, n, 2 * c["kv"], c["d"]))
    # runs of a page's slots in pages of any order; the last rows of a padded batch have none
    slots = (_perm(g, n_pages)[:, None] * ps + torch.arange(ps, dtype=torch.int32, device=DEV)).reshape(-1)[:n].contiguous()
    slots[n - n // 50:] = -1
    return s | {"k": fused[:, :c["kv"]], "v": fused[:, c["kv"]:], "slots": slots, "page": ps, "n_pages": n_pages}


def prepare(case, seed):
    g = _gen(seed)
    f = {"attn": _prepare_attn, "attn_bwd": _prepare_attn, "decode": _prepare_decode, "tables": _prepare_tables, "write": _prepare_write}
    return {**f[case["op"]](case, g), "op": case["op"]}


# ---------------------------------------------------------------- the plain forms

def _chunks(s):
    """(first query row, first key row, keys, first query of the chunk, its queries, queries) for each sequence."""
    heads, q0, k0 = s["q"].shape[1], 0, 0
    for lq, lk in zip(s["lq"], s["lk"]):
        step = max(1, (1 << 29) // (heads * max(lk, 1)))
        for r in range(0, lq, step):
            yield q0, k0, lk, r, min(step, lq - r), lq
        q0, k0 = q0 + lq, k0 + lk


def _kv_of(s, name, k0, lk):
    """Keys or values [kv heads][keys][d] of a sequence in 32 bits."""
    return s[name][k0:k0 + lk].float().transpose(0, 1).contiguous()


def _grouped(t, kv):
    """[rows][heads][d] -> [kv heads][group * rows][d] in 32 bits."""
    rows, heads, d = t.shape
    return t.float().reshape(rows, kv, heads // kv, d).permute(1, 2, 0, 3).reshape(kv, -1, d)


def _ungrouped(t, rows):
    """The way back: [kv heads][group * rows][d] -> [rows][heads][d]."""
    kv, d = t.shape[0], t.shape[-1]
    return t.reshape(kv, -1, rows, d).permute(2, 0, 1, 3).reshape(rows, -1, d)


def _scores(s, q, k, lk, r, rows, lq):
    """Masked scores [kv heads][group][rows][keys]."""
    z = torch.matmul(q, k.transpose(1, 2).contiguous()).mul_(s["scale"])
    z = z.view(k.shape[0], -1, rows, lk)
    if s["causal"]:
        i = torch.arange(r, r + rows, device=DEV)[:, None] + (lk - lq)
        z.masked_fill_(torch.arange(lk, device=DEV) > i, NEG)
    return z


def _plain_attn(s):
    o, lse = torch.zeros_like(s["o"]), torch.full_like(s["lse"], NEG)
    kv = s["k"].shape[1]
    for q0, k0, lk, r, rows, lq in _chunks(s):
        if lk == 0:
            continue
        at = slice(q0 + r, q0 + r + rows)
        z = _scores(s, _grouped(s["q"][at], kv), _kv_of(s, "k", k0, lk), lk, r, rows, lq)
        top = z.amax(-1, keepdim=True)
        p = (z - torch.where(top == NEG, 0.0, top)).exp_()
        total = p.sum(-1, keepdim=True)
        p = p.div_(torch.where(total == 0, 1.0, total)).view(kv, -1, lk)
        o[at] = _ungrouped(torch.matmul(p, _kv_of(s, "v", k0, lk)), rows).to(torch.bfloat16)
        lse[:, at] = (top + total.log()).view(-1, rows)
    return {"o": o, "lse": lse}


def _plain_attn_bwd(s):
    kv, d = s["k"].shape[1:]
    dk, dv = (torch.zeros(s["k"].shape[0], kv, d, device=DEV) for _ in range(2))
    for q0, k0, lk, r, rows, lq in _chunks(s):
        if lk == 0:
            continue
        at = slice(q0 + r, q0 + r + rows)
        q, do = _grouped(s["q"][at], kv), _grouped(s["dout"][at], kv)
        k, v = _kv_of(s, "k", k0, lk), _kv_of(s, "v", k0, lk)
        delta = (do * _grouped(s["o"][at], kv)).sum(-1, keepdim=True)
        lse = s["lse"][:, at].reshape(kv, -1, rows, 1)
        p = (_scores(s, q, k, lk, r, rows, lq) - torch.where(lse == NEG, 0.0, lse)).exp_().view(kv, -1, lk)
        dv[k0:k0 + lk] += torch.matmul(p.transpose(1, 2).contiguous(), do).transpose(0, 1)
        ds = torch.matmul(do, v.transpose(1, 2).contiguous()).sub_(delta).mul_(p).mul_(s["scale"])
        s["dq"][at] = _ungrouped(torch.matmul(ds, k), rows).to(torch.bfloat16)
        dk[k0:k0 + lk] += torch.matmul(ds.transpose(1, 2).contiguous(), q).transpose(0, 1)
    s["dk"].copy_(dk)
    s["dv"].copy_(dv)
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


def _gathered(s, name, table):
    """A cache's pages of some requests in 32 bits: [requests][kv heads][width * page][d]."""
    t = s[name + "_cache"].view(torch.uint8)[table.long()].view(s[name + "_cache"].dtype).float()
    if s[name + "_scales"] is not None:
        t = (t.unflatten(-1, (-1, 32)) * _pow2(s[name + "_scales"].view(torch.uint8)[table.long()])[..., None]).flatten(-2)
    return t.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_decode(s):
    n, heads, d = s["q"].shape
    kv, width = s["kv"], s["table"].shape[1]
    o, lse = [], []
    step = max(1, (1 << 28) // (kv * width * s["page"] * d))
    for b in range(0, n, step):
        table, lens = s["table"][b:b + step], s["lens"][b:b + step]
        m = table.shape[0]
        q = s["q"][b:b + step].float().view(m * kv, -1, d)
        z = torch.matmul(q, _gathered(s, "k", table).flatten(0, 1).transpose(1, 2).contiguous()) * s["scale"]
        z = z.view(m, heads, -1).masked_fill(torch.arange(z.shape[-1], device=DEV) >= lens[:, None, None], NEG)
        top = z.amax(-1, keepdim=True)
        p = (z - top).exp_()
        total = p.sum(-1, keepdim=True)
        v = _gathered(s, "v", table)
        o.append((torch.matmul(p.view(m * kv, -1, p.shape[-1]), v.flatten(0, 1)).view(m, heads, d) / total).to(torch.bfloat16))
        lse.append((top + total.log())[..., 0])
    return {"o": torch.cat(o), "lse": torch.cat(lse)}


def _plain_tables(s):
    ps, n_pages, cap = s["page"], s["n_pages"], s["slots"].numel()
    cached, new = s["cached"].long(), s["new"].long()
    head, tail = s["state"][0], s["state"][1]
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    run_of = lambda t: torch.cat((zero, t.cumsum(0)))  # noqa: E731
    ended = new < 0
    owned = (cached + ps - 1) // ps
    lens = cached + new.clamp(min=0)
    need = torch.where(ended, 0, (lens + ps - 1) // ps - owned)
    cu, taken, given = run_of(new.clamp(min=0)), run_of(need), run_of(torch.where(ended, owned, 0))
    served = (need == 0) | (taken[1:] <= tail - head)
    # pages: a new column of a request's table takes the ring's next page
    j = torch.arange(s["table"].shape[1], device=DEV)
    k = j - owned[:, None]
    fresh = (k >= 0) & (k < need[:, None]) & served[:, None]
    page = s["ring"][(head + taken[:-1, None] + torch.where(fresh, k, 0)) % n_pages]
    table = torch.where(fresh, page, s["table"])
    # tokens
    t = torch.arange(cap, device=DEV)
    seq = torch.searchsorted(cu, t, right=True).sub_(1).clamp_(max=s["new"].numel() - 1)
    live = t < cu[-1]
    pos = cached[seq] + t - cu[seq]
    slot = table[seq, torch.where(live, pos // ps, 0)].long() * ps + pos % ps
    # pages of ended requests go to the ring's tail
    i = (torch.arange(n_pages, device=DEV) - tail) % n_pages
    back = i < given[-1]
    owner = torch.searchsorted(given, torch.where(back, i, 0), right=True).sub_(1).clamp_(max=s["new"].numel() - 1)
    freed = s["table"][owner, torch.where(back, i - given[owner], 0)]
    used = torch.where(served, taken[1:], 0).amax()
    return {"seq_lens": torch.where(ended, 0, torch.where(served, lens, cached)).int(), "table": table, "cu": cu.int(),
            "ring": torch.where(back, freed, s["ring"]), "state": torch.stack((head + used, tail + given[-1])),
            "slots": torch.where(live & served[seq], slot, -1).int(), "positions": torch.where(live, pos, -1).int(),
            "token_seqs": torch.where(live, seq, -1).int()}


def _plain_write(s):
    slots = s["slots"].long()
    page, row = slots // s["page"], slots % s["page"]
    old = slots < 0
    out = {}
    for name in ("k", "v"):
        x = s[name]
        parts = [(name + "_cache", x)]
        if s[name + "_scales"] is not None:
            q, b = _quantize8(x.float())
            parts = [(name + "_cache", q.view(torch.uint8)), (name + "_scales", b)]
        for key, value in parts:
            cache = s[key].view(value.dtype)
            # rows without a slot write what the first live row writes
            first = (~old).to(torch.int8).argmax()
            pick = torch.where(old, first, torch.arange(len(slots), device=DEV))
            cache[page[pick], :, row[pick]] = value[pick]
            out[key] = s[key]
    return out


# ---------------------------------------------------------------- the library's calls

_loaded = []


def _lib():
    if not _loaded:
        from rl_lora_linear_amd import lib
        _loaded.append(lib)
    return _loaded[0]


def _attn_shape(s):
    if "shape" not in s:
        q, k = s["q"], s["k"]
        s["shape"] = _lib().make_attention_shape(q.shape[0], k.shape[0], len(s["lq"]), q.shape[1], k.shape[1], q.shape[2], s["scale"],
                                                 causal=s["causal"], q_stride=q.stride(0), k_stride=k.stride(0), v_stride=s["v"].stride(0))
    return s["shape"]


def _own_attn(s):
    _lib().attention_forward(_attn_shape(s), s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["o"], s["lse"], s["ws"])
    return {"o": s["o"], "lse": s["lse"]}


def _own_attn_bwd(s):
    _lib().attention_backward(_attn_shape(s), s["dout"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["cu_q"], s["cu_k"], s["dq"], s["dk"],
                              s["dv"], s["ws"])
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


def _kv_shape(s, n, kv, d, width):
    if "shape" not in s:
        s["shape"] = _lib().make_kv_shape(n, kv, d, s["page"], s["n_pages"], width)
    return s["shape"]


def _own_decode(s):
    L = _lib()
    n, heads, d = s["q"].shape
    shape = _kv_shape(s, n, s["kv"], d, s["table"].shape[1])
    if "ws" not in s:
        s["ws"] = L.empty_workspace(L.attention_decode_workspace_bytes(shape, heads, s["max_len"]))
    L.attention_decode(shape, s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["max_len"], s["scale"], s["o"], s["ws"],
                       k_scales=s["k_scales"], v_scales=s["v_scales"], lse=s["lse"])
    return {"o": s["o"], "lse": s["lse"]}


def _own_tables(s):
    L = _lib()
    shape = _kv_shape(s, s["new"].numel(), 1, 64, s["table"].shape[1])
    if "ws" not in s:
        s["ws"] = L.empty_workspace(L.kv_tables_workspace_bytes(shape))
    L.kv_tables(shape, s["cached"], s["new"], s["seq_lens"], s["table"], s["ring"], s["state"], s["state_out"], s["cu"], s["slots"], s["ws"],
                positions=s["positions"], token_seqs=s["token_seqs"])
    return {"seq_lens": s["seq_lens"], "table": s["table"], "cu": s["cu"], "ring": s["ring"], "state": s["state_out"], "slots": s["slots"],
            "positions": s["positions"], "token_seqs": s["token_seqs"]}


def _own_write(s):
    L = _lib()
    if "ws" not in s:
        s["ws"] = L.empty_workspace(256)
    shape = _kv_shape(s, 1, s["k"].shape[1], s["k"].shape[2], 1)
    L.kv_write(shape, s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["ws"], k_scales=s["k_scales"], v_scales=s["v_scales"])
    return {k: s[k] for k in ("k_cache", "v_cache", "k_scales", "v_scales") if s[k] is not None}


def run(state):
    if own:
        f = {"attn": _own_attn, "attn_bwd": _own_attn_bwd, "decode": _own_decode, "tables": _own_tables, "write": _own_write}
    else:
        f = {"attn": _plain_attn, "attn_bwd": _plain_attn_bwd, "decode": _plain_decode, "tables": _plain_tables, "write": _plain_write}
    return f[state["op"]](state)


# ---------------------------------------------------------------- work

def _pairs(c):
    """(query, key) pairs that the masks leave, over all sequences."""
    total = 0
    for lq, lk in zip(*(a.tolist() for a in _attn_lens(c))):
        total += lq * lk - (lq * (lq - 1) // 2 if c["causal"] else 0)
    return total


def work(case):
    c, op = case, case["op"]
    if op in ("attn", "attn_bwd"):
        q = c["n"] * c["heads"]
        k = int(_attn_lens(c)[1].sum()) * c["kv"]
        pairs = float(_pairs(c)) * c["heads"] * c["d"]
        if op == "attn":
            return {"bytes": 4 * c["d"] * (q + k) + 4 * q, "flops": 4.0 * pairs}
        return {"bytes": 8 * c["d"] * (q + k) + 4 * q, "flops": 10.0 * pairs}
    if op == "decode":
        rows = int(_decode_lens(c).sum())
        row = c["d"] + c["d"] // 32 if c["x8"] else 2 * c["d"]
        return {"bytes": 2 * rows * c["kv"] * row + c["n"] * c["heads"] * (4 * c["d"] + 4), "flops": 4.0 * rows * c["heads"] * c["d"]}
    if op == "tables":
        cached, new = _table_lens(c)
        owned = -(-cached // c["page"])
        moved = np.where(new < 0, owned, -(-(cached + np.maximum(new, 0)) // c["page"]) - owned)
        tokens = int(np.maximum(new, 0).sum())
        return {"bytes": 16 * c["n"] + 8 * int(moved.sum()) + 12 * tokens + 32, "flops": 4.0 * tokens}
    live = c["n"] - c["n"] // 50
    row = c["d"] + c["d"] // 32 if c["x8"] else 2 * c["d"]
    return {"bytes": 4 * c["n"] + 2 * live * c["kv"] * (2 * c["d"] + row), "flops": 4.0 * live * c["kv"] * c["d"]}


# ---------------------------------------------------------------- 64 bits

def _head_probs(c, s, h, q0, k0, r, rows, lq, lk):
    """Scores of one head's query rows against the keys they may see, and how many keys those are at most."""
    last = min(lk, max(0, r + rows + lk - lq)) if c["causal"] else lk
    g = h // (c["heads"] // c["kv"])
    q = s["q"][q0 + r:q0 + r + rows, h].double()
    k = s["k"][k0:k0 + last, g].double()
    z = (q @ k.t().contiguous()) / math.sqrt(c["d"])
    if c["causal"]:
        gone = torch.arange(last, device=DEV)[None, :] - torch.arange(r, r + rows, device=DEV)[:, None] > lk - lq
        z[gone] = NEG
    return g, last, q, k, z


def _walk(c):
    lq_all, lk_all = _attn_lens(c)
    q0 = k0 = 0
    for lq, lk in zip(lq_all.tolist(), lk_all.tolist()):
        for r in range(0, lq, 4096):
            yield q0, k0, r, min(4096, lq - r), lq, lk
        q0, k0 = q0 + lq, k0 + lk


def _exact_attn(c, s):
    o = torch.zeros(c["n"], c["heads"], c["d"], dtype=F64, device=DEV)
    lse = torch.full((c["heads"], c["n"]), NEG, dtype=F64, device=DEV)
    for q0, k0, r, rows, lq, lk in _walk(c):
        for h in range(c["heads"]):
            g, last, _, _, z = _head_probs(c, s, h, q0, k0, r, rows, lq, lk)
            if last:
                total = torch.logsumexp(z, 1)
                w = torch.exp(z - total.clamp(min=-1e300)[:, None])
                o[q0 + r:q0 + r + rows, h] = w @ s["v"][k0:k0 + last, g].double().contiguous()
                lse[h, q0 + r:q0 + r + rows] = total
    return {"o": o, "lse": lse}


def _exact_attn_bwd(c, s):
    dq = torch.zeros(s["q"].shape, dtype=F64, device=DEV)
    dk, dv = (torch.zeros(s["k"].shape, dtype=F64, device=DEV) for _ in range(2))
    for q0, k0, r, rows, lq, lk in _walk(c):
        at = slice(q0 + r, q0 + r + rows)
        for h in range(c["heads"]):
            g, last, q, k, z = _head_probs(c, s, h, q0, k0, r, rows, lq, lk)
            if not last:
                continue
            w = torch.exp(z - s["lse"][h, at].double().clamp(min=-1e300)[:, None])
            do = s["dout"][at, h].double()
            slope = do @ s["v"][k0:k0 + last, g].double().t().contiguous()
            slope -= torch.einsum("id,id->i", do, s["o"][at, h].double())[:, None]
            slope *= w / math.sqrt(c["d"])
            dq[at, h] = slope @ k
            dk[k0:k0 + last, g] += slope.t().contiguous() @ q
            dv[k0:k0 + last, g] += w.t().contiguous() @ do
    return {"dq": dq, "dk": dk, "dv": dv}


def _two_to(e):
    """2^e in 64 bits from the exponent's bits (a library power may be off by its last bit)."""
    return ((e.long() + 1023) << 52).view(F64)


def _exact_cache(s, name, pages):
    t = s[name + "_cache"].view(torch.uint8)[pages].view(s[name + "_cache"].dtype).to(torch.float32).double()
    if s[name + "_scales"] is not None:
        e = s[name + "_scales"].view(torch.uint8)[pages].long() - 127
        t = t * _two_to(e).repeat_interleave(32, dim=-1)
    return t.transpose(0, 1).reshape(t.shape[1], -1, t.shape[-1])


def _exact_decode(c, s):
    o = torch.empty(c["n"], c["heads"], c["d"], dtype=F64, device=DEV)
    lse = torch.empty(c["n"], c["heads"], dtype=F64, device=DEV)
    for b, length in enumerate(_decode_lens(c).tolist()):
        pages = s["table"][b, :-(-length // c["page"])].long()
        k, v = (_exact_cache(s, name, pages)[:, :length] for name in ("k", "v"))
        q = s["q"][b].double().view(c["kv"], -1, c["d"])
        z = (q @ k.transpose(1, 2).contiguous()) / math.sqrt(c["d"])
        lse[b] = torch.logsumexp(z, -1).reshape(-1)
        o[b] = (torch.softmax(z, -1) @ v).reshape(c["heads"], c["d"])
    return {"o": o, "lse": lse}


def _exact_tables(c, s):
    """Request by request, as a host's allocator would go."""
    ps, n_pages = c["page"], s["n_pages"]
    table, ring = s["table"].tolist(), s["ring"].tolist()
    (head, tail), back = s["state"].tolist(), []
    free = tail - head
    lens, cu, slots, positions, seqs, taken = [], [0], [], [], [], 0
    for b, (cached, new) in enumerate(zip(s["cached"].tolist(), s["new"].tolist())):
        held = (cached + ps - 1) // ps
        if new < 0:
            back += table[b][:held]
            lens.append(0)
            cu.append(cu[-1])
            continue
        for j in range(held, (cached + new + ps - 1) // ps):
            assert taken < free
            table[b][j] = ring[(head + taken) % n_pages]
            taken += 1
        for p in range(cached, cached + new):
            slots.append(table[b][p // ps] * ps + p % ps)
            positions.append(p)
            seqs.append(b)
        lens.append(cached + new)
        cu.append(cu[-1] + new)
    for i, page in enumerate(back):
        ring[(tail + i) % n_pages] = page
    pad = [-1] * (s["slots"].numel() - len(slots))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"seq_lens": i32(lens), "table": i32(table), "cu": i32(cu), "ring": i32(ring),
            "state": torch.tensor([head + taken, tail + len(back)], dtype=torch.int64, device=DEV), "slots": i32(slots + pad),
            "positions": i32(positions + pad), "token_seqs": i32(seqs + pad)}


def _to_e4m3(v):
    """v rounded (half to even) to three fraction bits, exponents from -6 on."""
    step = _two_to((torch.frexp(v).exponent - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_write(c, s):
    live = s["slots"] >= 0
    slots = s["slots"][live].long()
    out = {}
    for name in ("k", "v"):
        cache = s[name + "_cache"].to(torch.float32).double()
        rows = s[name][live].double()
        if c["x8"]:
            scales = _two_to(s[name + "_scales"].view(torch.uint8).long() - 127)
            blocks = rows.unflatten(-1, (-1, 32))
            f = torch.frexp(blocks.abs().amax(-1) / 448.0)
            e = (f.exponent - (f.mantissa == 0.5).to(torch.int32)).clamp(min=-126)
            scale = _two_to(e)
            rows = _to_e4m3(blocks / scale[..., None]).flatten(-2)
            scales[slots // c["page"], :, slots % c["page"]] = scale
            out[name + "_scales"] = scales
        cache[slots // c["page"], :, slots % c["page"]] = rows
        out[name + "_cache"] = cache
    return out


def exact(case, seed):
    s = prepare(case, seed)
    f = {"attn": _exact_attn, "attn_bwd": _exact_attn_bwd, "decode": _exact_decode, "tables": _exact_tables, "write": _exact_write}
    return f[case["op"]](case, s)
