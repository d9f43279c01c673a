"""Workloads of the calls around the key/value cache: rotary positions on the way
into it, its pages, and attention over the pages that a cheap score selects.

Three operators, by a case's "op":
  rope    qrope          rotary positions with one or several axes
  rope_w  qrope_write    the same for q, k and v of a layer, straight into the cache;
          qcache_read    and what the cache then holds, as a prompt's next chunk reads it
  beams   qcache_fork, qcache_reserve, qcache_copy
                         a step of a beam search over the cache's pages
  copy    qcache_copy    whole pages, all layers
  compact qcache_compact the kept tokens of each sequence follow its context
  bounds  qcache_bounds  the keys' bounds of each page, as new tokens come in
  sparse  qblock_select, qattn_blocks
                         pages by their bounds, attention over the picked ones

With `own` false, run() computes the same results from elementary torch
operations in 32 bits (angles in 64); with `own` true it calls the package.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # A decode step of 32 sequences: rotated and cached straight from the fp32 output of one q/k/v product.
        dict(name="rope_step_32", op="rope_w", tokens=32, heads=64, kv=8, dim=128, rot=128, axes=1, style="halves", src="fp32", far=131071, dense=False, page=16, codes="int8"),
        # A prompt of 8191 tokens with images among the text: time, height and width, dense keys and values for its attention too.
        dict(name="rope_prompt_8191", op="rope_w", tokens=8191, heads=64, kv=8, dim=128, rot=128, axes=3, style="halves", src="fp32", far=8191, dense=True, page=64, codes="fp8"),
        # The patches of an image of 77 x 53, two axes, heads of 64 channels, neighbouring channels as pairs.
        dict(name="rope_image", op="rope", tokens=4081, heads=32, dim=64, rot=64, axes=2, style="pairs", src="bf16", far=77),
        # A step of a beam search: 12 prompts, 8 beams each, every beam follows one of its prompt's and gets room for a token.
        dict(name="beams_96", op="beams", groups=12, beams=8, lo=300, hi=9000, kv=8, dim=128, page=16, codes="int8"),
        # A long conversation forked: its 601 pages copied in each of 6 layers.
        dict(name="copy_layers", op="copy", pages=601, layers=6, kv=8, dim=128, page=16, codes="int8"),
        # Accepting drafts: trees of 13 for 16 sequences, in each of 8 layers.
        dict(name="compact_drafts", op="compact", batch=16, lo=100, hi=2000, new=13, share=0.3, layers=8, kv=8, dim=128, page=16, codes="int8"),
        # Half of the tokens of two long contexts dropped, two layers.
        dict(name="compact_context", op="compact", batch=2, lo=20000, hi=30001, new=0, share=0.5, layers=2, kv=8, dim=128, page=64, codes="fp8"),
        # The bounds of a prompt of 30001 tokens, once it is in the cache.
        dict(name="bounds_prompt", op="bounds", batch=1, lo=30001, hi=30001, new=0, kv=8, dim=128, page=32, codes="fp8"),
        # One token of one user, a short conversation: latency.
        dict(name="sparse_b1", op="sparse", batch=1, lo=1000, hi=1000, new=1, count=24, heads=64, kv=8, dim=128, page=16, codes="int8"),
        # One token of one user with a very long document: 64 of 2048 pages.
        dict(name="sparse_long", op="sparse", batch=1, lo=131071, hi=131071, new=1, count=64, heads=64, kv=8, dim=128, page=64, codes="int8"),
        # A decode step of 48 sequences of very different lengths.
        dict(name="sparse_batch", op="sparse", batch=48, lo=17, hi=16000, new=1, count=64, heads=64, kv=8, dim=128, page=16, codes="int8"),
        # The next 255 tokens of two long prompts, each with pages of its own choice, heads of 64 channels.
        dict(name="sparse_chunk_d64", op="sparse", batch=2, lo=9000, hi=30000, new=255, count=40, heads=32, kv=8, dim=64, page=32, codes="fp8"),
    ]


def draw(rng):
    def log(a, b):
        return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))

    op = rng.choice(["rope_w", "rope_w", "rope", "beams", "copy", "compact", "bounds", "sparse", "sparse", "sparse"])
    kv = rng.choice([1, 2, 4, 8, 8])
    dim = rng.choice([64, 128, 128])
    heads = kv * rng.choice([1, 2, 4, 5, 7, 8])
    page = rng.choice([16, 16, 32, 64, 128])
    codes = rng.choice(["int8", "fp8"])
    if op in ("rope", "rope_w"):
        got = dict(op=op, tokens=log(1, 8191), heads=heads, kv=kv, dim=dim, rot=rng.choice([dim, dim, dim, 32, 16]),
                   axes=rng.choice([1, 1, 2, 3]), style=rng.choice(["halves", "halves", "pairs"]), src=rng.choice(["fp32", "bf16"]),
                   far=log(100, 1000000), dense=rng.random() < 0.5, page=page, codes=codes)
        return got if op == "rope_w" else {k: v for k, v in got.items() if k not in ("kv", "dense", "page", "codes")}
    if op == "beams":
        hi = log(20, 8000)
        return dict(op=op, groups=log(1, 16), beams=rng.choice([1, 2, 4, 5, 8]), lo=log(1, hi), hi=hi, kv=kv, dim=dim, page=page, codes=codes)
    if op == "copy":
        return dict(op=op, pages=log(1, 9000 // page), layers=log(1, 8), kv=kv, dim=dim, page=page, codes=codes)
    if op == "compact":
        if rng.random() < 0.6:
            hi = log(64, 4000)
            return dict(op=op, batch=log(1, 64), lo=log(64, hi), hi=hi, new=log(1, 64), share=rng.uniform(0.05, 0.95), layers=log(1, 8),
                        kv=kv, dim=dim, page=page, codes=codes)
        hi = log(1, 30000)
        return dict(op=op, batch=log(1, 3), lo=log(1, hi), hi=hi, new=0, share=rng.uniform(0.05, 0.95), layers=rng.choice([1, 2]), kv=kv,
                    dim=dim, page=page, codes=codes)
    batch = log(1, 64)
    hi = log(1, min(131071, 262144 // batch))
    lo = log(1, hi)
    if op == "bounds":
        return dict(op=op, batch=batch, lo=lo, hi=hi, new=rng.choice([0, 1, log(1, lo)]), kv=kv, dim=dim, page=page, codes=codes)
    new = rng.choice([1, 1, log(1, 200)])
    if new > 1:
        batch = min(batch, max(1, 500 // new))
        hi = max(new, min(hi, 40000 // batch))
        lo = max(new, min(lo, hi))
    return dict(op=op, batch=batch, lo=lo, hi=hi, new=new, count=log(2, max(2, min(1024 if new > 1 else 4096, 400000 // (batch * new)) // page)),
                heads=heads, kv=kv, dim=dim, page=page, codes=codes)


def lengths(case):
    """The sequences' lengths: the first is `hi`, the others spread over lo..hi by their logarithm."""
    lo, hi, n = case["lo"], case["hi"], case["groups" if case["op"] == "beams" else "batch"]
    got = [hi]
    for i in range(1, n):
        u = math.modf(0.5 + i * 0.6180339887498949)[0]
        got.append(max(lo, min(hi, int(round(lo * (hi / lo) ** u)))))
    return got


def fresh(case):
    """The new tokens of each sequence: `new` of them, or all."""
    return [min(case["new"], n) if case["new"] else n for n in lengths(case)]


def work(case):
    op, dim = case["op"], case["dim"]
    if op in ("rope", "rope_w"):
        size = 4 if case["src"] == "fp32" else 2
        row = case["tokens"] * dim
        if op == "rope":
            return {"bytes": row * case["heads"] * (size + 2), "flops": 3 * row * case["heads"]}
        cached = case["tokens"] * 2 * case["kv"]
        return {"bytes": row * case["heads"] * (size + 2) + cached * (dim * (size + (2 if case["dense"] else 0)) + 2 * (dim + 4) + 2 * dim),
                "flops": 3 * row * (case["heads"] + 2 * case["kv"])}
    page = case["kv"] * 2 * case["page"] * (dim + 4)  # bytes of one page of one layer
    if op == "copy":
        return {"bytes": 2 * case["pages"] * case["layers"] * page, "flops": 0}
    if op == "beams":
        rows = sum(-(-n // case["page"]) for n in lengths(case)) * case["beams"]
        partial = sum(n % case["page"] > 0 for n in lengths(case)) * max(1, case["beams"] // 2)
        return {"bytes": 8 * rows + 2 * partial * page, "flops": 0}
    if op == "compact":
        return {"bytes": 2 * case["share"] * sum(fresh(case)) * case["layers"] * case["kv"] * 2 * (dim + 4), "flops": 0}
    n = lengths(case)
    if op == "bounds":
        pages = sum(-(-x // case["page"]) - (x - f) // case["page"] for x, f in zip(n, fresh(case)))
        return {"bytes": pages * case["kv"] * (case["page"] * (dim + 4) + 2 * dim + 4), "flops": 3 * pages * case["kv"] * case["page"] * dim}
    held = [-(-x // case["page"]) for x in n]
    rows = case["new"] * len(n)
    picked = [min(case["count"], h) for h in held]
    seen = sum(min(h, p * case["new"]) for h, p in zip(held, picked))  # pages that some row may pick
    return {"bytes": sum(held) * case["kv"] * (2 * dim + 4) + seen * page + 4 * dim * case["heads"] * rows,
            "flops": case["new"] * sum(4 * dim * case["heads"] * p * case["page"] + 4 * dim * case["kv"] * h for h, p in zip(held, picked))}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 29)
    return g


def _heads(g, tokens, heads, dim, dtype):
    """Rows as projections give them: every head with a few channels larger than the rest."""
    x = torch.randn(tokens, heads, dim, device=DEV, generator=g)
    x *= torch.exp(0.5 * torch.randn(1, heads, dim, device=DEV, generator=g))
    return x.to(dtype)


def _starts(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)


def _ints(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device=DEV)


def _tables(rng, n, page, spare=3):
    """A block table [batch, pages of the longest] over pages in random order, and the number of pages."""
    need = [-(-x // page) for x in n]
    ids = rng.permutation(sum(need) + spare)
    table = np.zeros((len(n), max(need)), np.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = ids[at:at + c]
        at += c
    return _ints(table), sum(need) + spare


def _cache(g, pages, case, layers=0):
    """A filled cache: codes [pages, 2, kv, page, dim] and scales without the last, with the layers in front if there are any."""
    shape = ((layers,) if layers else ()) + (pages, 2, case["kv"], case["page"], case["dim"])
    if case["codes"] == "int8":
        codes = torch.empty(shape, device=DEV).normal_(0.0, 42.0, generator=g).round_().clamp_(-127, 127).to(torch.int8)
        step = 1 / 42
    else:
        codes = torch.empty(shape, device=DEV).normal_(0.0, 140.0, generator=g).clamp_(-448, 448).to(torch.float8_e4m3fn)
        step = 1 / 140
    scales = step * torch.exp(0.3 * torch.randn(shape[:-1], device=DEV, generator=g))
    return codes, scales


def prepare(case, seed):
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    s = dict(case=dict(case))
    return {"rope": _prepare_rope, "rope_w": _prepare_rope, "beams": _prepare_beams, "copy": _prepare_copy, "compact": _prepare_compact,
            "bounds": _prepare_cache, "sparse": _prepare_cache}[case["op"]](s, case, g, rng)


def _prepare_rope(s, case, g, rng):
    t, dim, half = case["tokens"], case["dim"], case["rot"] // 2
    src = torch.float32 if case["src"] == "fp32" else torch.bfloat16
    # positions: tokens one behind the other, or anywhere up to `far` in a decode step; further axes in rows of an image
    base = rng.integers(0, case["far"] + 1, t) if t <= 64 else int(rng.integers(0, max(1, case["far"] - t + 1))) + np.arange(t)
    axes = [base] + [(np.arange(t) // (1 if a else 53)) % (53 if a else max(1, case["far"])) for a in range(case["axes"] - 1)]
    # pairs of an axis lie together, or go round the axes where an image is rotated
    axis = np.arange(half) * case["axes"] // half if case["op"] == "rope_w" else np.arange(half) % case["axes"]
    s.update(positions=_ints(np.stack(axes)), axis=_ints(axis),
             rates=torch.tensor(500000.0 ** (-np.arange(half) / half), dtype=torch.float64, device=DEV))
    if case["op"] == "rope":
        s.update(x=_heads(g, t, case["heads"], dim, src))
        return s
    h, kv = case["heads"], case["kv"]
    y = _heads(g, t, h + 2 * kv, dim, src)  # views of the fused product's output
    table, pages = _tables(rng, [t], case["page"])
    at = torch.arange(t, device=DEV)
    slots = table[0].long()[at // case["page"]] * case["page"] + at % case["page"]
    code = torch.int8 if case["codes"] == "int8" else torch.float8_e4m3fn
    s.update(q=y[:, :h], k=y[:, h:h + kv], v=y[:, h + kv:], slots=slots, table=table, cu=_starts([t]), codes=torch.zeros(pages, 2, kv, case["page"], dim, device=DEV).to(code),
             scales=torch.zeros(pages, 2, kv, case["page"], device=DEV))
    return s


def _prepare_beams(s, case, g, rng):
    size, beams = case["page"], case["beams"]
    n = np.repeat(lengths(case), beams)
    width = max(-(-x // size) for x in n) + 2
    rows, refs_of = [], []
    at = 0
    for i, x in enumerate(lengths(case)):
        # the beams of a prompt share its pages up to where they parted; each has its last few for itself
        held = -(-x // size)
        common = max(0, held - 1 - i % 4)
        shared = np.arange(at, at + common)
        at += common
        for _ in range(beams):
            mine = np.arange(at, at + held - common)
            at += held - common
            row = np.full(width, -1)
            row[:held] = np.concatenate([shared, mine])
            rows.append(row)
    pages = at + len(rows) + 7
    ids = rng.permutation(pages)
    table = np.stack(rows)
    table = np.where(table >= 0, ids[table], -1)
    refs = np.bincount(table[table >= 0], minlength=pages)
    parents = np.concatenate([b * beams + rng.integers(0, beams, beams) for b in range(case["groups"])])
    codes, scales = _cache(g, pages, case)
    s.update(codes=codes, scales=scales, table=_ints(table), lens=_ints(n), refs=_ints(refs), parents=_ints(parents))
    return s


def _prepare_copy(s, case, g, rng):
    pages = 2 * case["pages"] + 5
    codes, scales = _cache(g, pages, case, case["layers"])
    ids = rng.permutation(pages)[:2 * case["pages"]]
    s.update(codes=codes, scales=scales, copies=_ints(ids.reshape(-1, 2)))
    return s


def _prepare_compact(s, case, g, rng):
    n, new = lengths(case), fresh(case)
    table, pages = _tables(rng, n, case["page"])
    codes, scales = _cache(g, pages, case, case["layers"])
    s.update(codes=codes, scales=scales, table=table, lens=_ints(n), cu=_starts(new), keep=_ints(rng.random(sum(new)) < case["share"], torch.bool))
    return s


def _prepare_cache(s, case, g, rng):
    n, new = lengths(case), fresh(case)
    table, pages = _tables(rng, n, case["page"])
    codes, scales = _cache(g, pages, case)
    s.update(codes=codes, scales=scales, table=table, lens=_ints(n), cu=_starts(new) if max(new) > 1 else None, total=sum(new), most=max(new),
             bounds=torch.zeros(pages, case["kv"], 2, case["dim"], dtype=torch.int8, device=DEV), bound_scales=torch.zeros(pages, case["kv"], device=DEV))
    if case["op"] == "sparse":
        s.update(q=_heads(g, sum(new), case["heads"], case["dim"], torch.bfloat16))
        # the bounds that the cache has by now: of every page, over all of its tokens
        used = torch.zeros(pages, case["page"], dtype=torch.bool, device=DEV)
        for b, x in enumerate(n):
            at = torch.arange(x, device=DEV)
            used[table[b].long()[at // case["page"]], at % case["page"]] = True
        for p in range(0, pages, 1024):
            s["bounds"][p:p + 1024], s["bound_scales"][p:p + 1024] = _bounds_of(codes[p:p + 1024, 0], scales[p:p + 1024, 0], used[p:p + 1024])
    return s


def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "rope_w": _plain_rope_write, "beams": _plain_beams, "copy": _plain_copy, "compact": _plain_compact,
            "bounds": _plain_bounds, "sparse": _plain_sparse}[s["case"]["op"]](s)


def _own(s):
    import dequant_gemv_qgemv_amd as q
    case, op = s["case"], s["case"]["op"]
    if op == "rope":
        return q.qrope(s["x"], s["positions"], s["rates"], axis=s["axis"], style=case["style"])
    if op == "rope_w":
        got = q.qrope_write(s["q"], s["k"], s["v"], s["positions"], s["rates"], s["slots"], s["codes"], s["scales"], axis=s["axis"],
                            style=case["style"], dense=case["dense"])
        got = got if case["dense"] else (got,)
        k, v = q.qcache_read(s["codes"], s["scales"], s["table"], s["cu"], case["tokens"])
        return {"dense": got, "k": k, "v": v, "scales": s["scales"]}
    if op == "beams":
        refs = s["refs"].clone()
        table, lens = q.qcache_fork(refs, s["table"], s["lens"], s["parents"], case["page"])
        slots, lens, copies = q.qcache_reserve(refs, table, lens, case["page"])
        q.qcache_copy(s["codes"], s["scales"], copies)
        return dict(refs=refs, table=table, lens=lens, slots=slots, copies=copies, codes=s["codes"], scales=s["scales"])
    if op == "copy":
        q.qcache_copy(s["codes"], s["scales"], s["copies"])
        return dict(codes=s["codes"], scales=s["scales"])
    if op == "compact":
        lens = q.qcache_compact(s["codes"], s["scales"], s["table"], s["lens"], s["keep"], s["cu"])
        return dict(lens=lens, codes=s["codes"], scales=s["scales"])
    if op == "bounds":
        q.qcache_bounds(s["codes"], s["scales"], s["table"], s["lens"], s["bounds"], s["bound_scales"], cu_q=s["cu"], total=s["total"])
        return dict(bounds=s["bounds"], scales=s["bound_scales"])
    picks = q.qblock_select(s["q"], s["bounds"], s["bound_scales"], s["table"], s["lens"], case["count"], case["page"], cu_q=s["cu"])
    return dict(picks=picks, out=q.qattn_blocks(s["q"], s["codes"], s["scales"], s["table"], s["lens"], picks, cu_q=s["cu"]))


# ------------------------------------------------------------ plain forms ---
def _angles(s):
    """cos and sin [tokens, 1, pairs]: the angles in 64 bits."""
    t = s["positions"][s["axis"].long()].double() * s["rates"][:, None]
    return t.cos().float().T[:, None], t.sin().float().T[:, None]


def _rotate(x, cos, sin, case):
    """Rows [tokens, heads, dim] in 32 bits, rotated."""
    x, rest = x.float()[..., :case["rot"]], x.float()[..., case["rot"]:]
    if case["style"] == "halves":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _plain_rope(s):
    return _rotate(s["x"], *_angles(s), s["case"]).to(torch.bfloat16)


def _plain_rope_write(s):
    case = s["case"]
    cos, sin = _angles(s)
    q, k, v = _rotate(s["q"], cos, sin, case).to(torch.bfloat16), _rotate(s["k"], cos, sin, case), s["v"].float()
    x = torch.stack([k, v], 1)  # [tokens, 2, kv, dim]
    limit = torch.full_like(x[..., :1], 127.0 if case["codes"] == "int8" else 448.0)
    scale = x.abs().amax(-1, keepdim=True) / limit
    y = torch.where(scale > 0, x / scale, torch.zeros_like(x))
    page, at = s["slots"] // case["page"], s["slots"] % case["page"]
    if case["codes"] == "int8":
        s["codes"][page, :, :, at] = y.round().clamp(-127, 127).to(torch.int8)
    else:
        s["codes"].view(torch.uint8)[page, :, :, at] = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s["scales"][page, :, :, at] = scale[..., 0]
    dense = (q, k.to(torch.bfloat16), v.to(torch.bfloat16)) if case["dense"] else (q,)
    back = s["codes"].view(torch.uint8)[page, :, :, at].view(s["codes"].dtype).float() * s["scales"][page, :, :, at][..., None]
    return {"dense": dense, "k": back[:, 0].to(torch.bfloat16), "v": back[:, 1].to(torch.bfloat16), "scales": s["scales"]}


def _plain_copy(s):
    copies = s["copies"].long()
    copies = copies[copies[:, 0] >= 0]
    raw = s["codes"].view(torch.uint8)
    if s["case"]["op"] == "copy":
        raw[:, copies[:, 1]] = raw[:, copies[:, 0]]
        s["scales"][:, copies[:, 1]] = s["scales"][:, copies[:, 0]]
    else:
        raw[copies[:, 1]] = raw[copies[:, 0]]
        s["scales"][copies[:, 1]] = s["scales"][copies[:, 0]]
    return dict(codes=s["codes"], scales=s["scales"])


def _plain_beams(s):
    size = s["case"]["page"]
    refs, table, lens, parents = s["refs"].clone(), s["table"], s["lens"], s["parents"].long()
    # fork: each row holds its parent's pages as far as those hold tokens
    col = torch.arange(table.shape[1], device=DEV)[None]
    kept = table.masked_fill(col >= (lens[:, None] + size - 1) // size, -1)
    new, lens = kept[parents], lens[parents]
    old, held = table.long().flatten(), new.long().flatten()
    refs.index_add_(0, old.clamp(min=0), -(old >= 0).to(torch.int32))
    refs.index_add_(0, held.clamp(min=0), (held >= 0).to(torch.int32))
    # reserve: one token each; a page that is not there or is shared is replaced by the lowest free ones in order
    end = lens + 1
    inside = (col >= (lens // size)[:, None]) & (col < ((end + size - 1) // size)[:, None])
    there = new >= 0
    shared = there & (refs[new.long().clamp(min=0)] > 1)
    need = inside & (~there | shared) & (end <= new.shape[1] * size)[:, None]
    count = need.sum(1)
    free, order = torch.sort((refs != 0).int(), dim=0, stable=True)
    served = (end <= new.shape[1] * size) & ((count == 0) | (count.cumsum(0) <= (free == 0).sum()))
    need = need & served[:, None]
    rank = need.flatten().cumsum(0).view(need.shape) - 1
    page = order[rank.clamp(min=0)].to(torch.int32)
    given = torch.where(need, page, new)
    gone = (need & there).flatten()
    refs.index_add_(0, held.clamp(min=0), -gone.to(torch.int32))
    refs.index_add_(0, given.long().flatten().clamp(min=0), need.flatten().to(torch.int32))
    at = (lens // size).long()[:, None]
    src, dst = new.gather(1, at)[:, 0], given.gather(1, at)[:, 0]
    slots = torch.where(served, dst.long() * size + lens % size, -1)
    moved = (need & there).gather(1, at)[:, 0] & (lens % size > 0)
    copies = torch.where(moved[:, None], torch.stack([src, dst], 1), -1)
    _plain_copy(dict(s, copies=copies))
    return dict(refs=refs, table=given, lens=torch.where(served, end, lens), slots=slots, copies=copies, codes=s["codes"], scales=s["scales"])


def _rows_of(cu, total):
    """Sequence and place within it of each packed row."""
    at = torch.arange(total, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), at, right=True)
    return b, at - cu.long()[b]


def _plain_compact(s):
    size, cu, lens, keep = s["case"]["page"], s["cu"], s["lens"].long(), s["keep"]
    b, i = _rows_of(cu, keep.shape[0])
    ctx = lens - (cu[1:] - cu[:-1])
    upto = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), keep.long().cumsum(0)])
    rank = upto[1:] - 1 - upto[cu.long()[b]]  # among the kept tokens of the sequence
    src, dst = (ctx[b] + i)[keep], (ctx[b] + rank)[keep]
    b = b[keep]
    table = s["table"].long()
    ps, pd = table[b, src // size], table[b, dst // size]
    raw = s["codes"].view(torch.uint8)
    raw[:, pd, :, :, dst % size] = raw[:, ps, :, :, src % size]
    s["scales"][:, pd, :, :, dst % size] = s["scales"][:, ps, :, :, src % size]
    return dict(lens=(ctx + upto[cu.long()[1:]] - upto[cu.long()[:-1]]).to(torch.int32), codes=s["codes"], scales=s["scales"])


def _bounds_of(codes, scales, used):
    """Bounds [pages, kv, 2, dim] and their scales [pages, kv] of keys [pages, kv, page, dim], over the places used [pages, page]."""
    x = codes.float() * scales[..., None]
    used = used[:, None, :, None]
    top, low = x.masked_fill(~used, -math.inf).amax(2), x.masked_fill(~used, math.inf).amin(2)
    y = torch.stack([top, low], 2)
    y = torch.where(used.any(2, keepdim=True), y, torch.zeros_like(y))
    step = y.abs().amax((2, 3), keepdim=True) / torch.full_like(y[:, :, :1, :1], 127.0)
    y = torch.where(step > 0, y / step, torch.zeros_like(y))
    return y.round().clamp(-127, 127).to(torch.int8), step[:, :, 0, 0]


def _plain_bounds(s):
    size, lens = s["case"]["page"], s["lens"].long()
    new = s["cu"][1:] - s["cu"][:-1] if s["cu"] is not None else torch.ones_like(s["lens"])
    col = torch.arange(s["table"].shape[1], device=DEV)[None]
    touched = (col >= ((lens - new) // size)[:, None]) & (col * size < lens[:, None])
    b, c = touched.nonzero(as_tuple=True)
    page = s["table"].long()[b, c]
    used = c[:, None] * size + torch.arange(size, device=DEV)[None] < lens[b][:, None]
    s["bounds"][page], s["bound_scales"][page] = _bounds_of(s["codes"].view(torch.uint8)[page, 0].view(s["codes"].dtype), s["scales"][page, 0], used)
    return dict(bounds=s["bounds"], scales=s["bound_scales"])


def _plain_select(s):
    case, size, count = s["case"], s["case"]["page"], s["case"]["count"]
    batch, new, kv, dim = case["batch"], case["new"], case["kv"], case["dim"]
    table = s["table"].long()
    q = s["q"].double().view(batch, new, kv, -1, dim)
    w = torch.cat([q.clamp(min=0).sum(3), q.clamp(max=0).sum(3)], -1).float()  # [batch, new, kv, 2 dim]
    step = w.abs().amax(-1, keepdim=True) / torch.full_like(w[..., :1], 127.0)
    w = torch.where(step > 0, w / step, torch.zeros_like(w)).round()
    # whole numbers below 2^24: the products' sums are exact
    keys = s["bounds"][table].view(batch, -1, kv, 2 * dim).permute(0, 2, 3, 1).float().contiguous()
    score = torch.matmul(w.transpose(1, 2).contiguous(), keys).transpose(1, 2)  # [batch, new, kv, pages]
    score = score * s["bound_scales"][table].transpose(1, 2)[:, None]
    seen = (s["lens"].long()[:, None] - new + torch.arange(new, device=DEV)[None]) // size + 1  # pages up to the row's own
    seen = seen[:, :, None, None]
    col = torch.arange(table.shape[1], device=DEV)
    score = score.masked_fill((col < 1) | (col == seen - 1), math.inf).masked_fill(col >= seen, -math.inf)
    if table.shape[1] < count:
        score = torch.nn.functional.pad(score, (0, count - table.shape[1]), value=-math.inf)
    picks = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :count]
    picks = picks.masked_fill(picks >= seen, 1 << 30).sort(-1)[0]
    return picks.masked_fill(picks == 1 << 30, -1).to(torch.int32).view(batch * new, kv, count)


def _plain_sparse(s):
    case, size = s["case"], s["case"]["page"]
    batch, new, kv, dim, heads = case["batch"], case["new"], case["kv"], case["dim"], case["heads"]
    picks = _plain_select(s)
    p = picks.long()
    b = torch.arange(batch, device=DEV).repeat_interleave(new)
    page = s["table"].long()[b[:, None, None], p.clamp(min=0)]  # [rows, kv, count]
    head = torch.arange(kv, device=DEV)[None, :, None]

    def values(which):
        c = s["codes"].view(torch.uint8)[page, which, head].view(s["codes"].dtype).float()
        return (c * s["scales"][page, which, head][..., None]).flatten(2, 3)  # [rows, kv, count page, dim]

    pos = s["lens"].long()[b] - new + torch.arange(new, device=DEV).repeat(batch)
    key = (p[..., None] * size + torch.arange(size, device=DEV)).flatten(2)
    seen = (p >= 0).repeat_interleave(size, 2) & (key <= pos[:, None, None])
    q = s["q"].float().view(-1, kv, heads // kv, dim)
    t = torch.matmul(q, values(0).transpose(2, 3).contiguous()) * (1 / math.sqrt(dim))
    t = t.masked_fill_(~seen[:, :, None], -math.inf)
    t = t.sub_(t.amax(-1, keepdim=True)).exp_()
    out = torch.matmul(t, values(1)) / t.sum(-1, keepdim=True)
    return dict(picks=picks, out=out.view(-1, heads, dim).to(torch.bfloat16))


# --------------------------------------------------- definition in 64 bits ---
def _e4m3(y):
    """The e4m3 value nearest to y, ties to the even mantissa."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    e = e - (torch.exp2(e) > y.abs().clamp(min=2.0 ** -6)).double()
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _turned(x, s):
    """x in 64 bits with each pair of channels turned by its angle, as a product of complex numbers."""
    case, half = s["case"], s["case"]["rot"] // 2
    angle = torch.stack([s["positions"][int(a)].double() * float(r) for a, r in zip(s["axis"].tolist(), s["rates"].tolist())], -1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    out = x.double().clone()
    first = torch.arange(half, device=DEV) * (1 if case["style"] == "halves" else 2)
    second = first + (half if case["style"] == "halves" else 1)
    z = torch.complex(out[..., first], out[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _turned(s["x"], s)
    if op == "rope_w":
        q, k, v = _turned(s["q"], s), _turned(s["k"], s), s["v"].double()
        back = []
        scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device=DEV)
        page, at = s["slots"] // case["page"], s["slots"] % case["page"]
        for which, x in enumerate((k, v)):
            t = x.abs().max(dim=2).values / (127 if case["codes"] == "int8" else 448)
            y = x / t[:, :, None]
            back.append((torch.round(y) if case["codes"] == "int8" else _e4m3(y)) * t[:, :, None])
            scales[page, which, :, at] = t
        return {"dense": (q, k, v) if case["dense"] else (q,), "k": back[0], "v": back[1], "scales": scales}
    if op == "beams":
        return None  # pages' numbers, and what is moved as it is
    if op == "copy":
        scales = s["scales"].double()
        scales[:, s["copies"][:, 1].long()] = s["scales"].double()[:, s["copies"][:, 0].long()]
        return dict(codes=None, scales=scales)
    if op in ("compact", "bounds"):
        size, cu = case["page"], s["cu"].tolist() if s["cu"] is not None else list(range(case["batch"] + 1))
        scales = s["scales"].double() if op == "compact" else s["bound_scales"].double()
        for b, n in enumerate(lengths(case)):
            at = torch.arange(n - cu[b + 1] + cu[b], n, device=DEV)
            if op == "compact":
                at, to = at[s["keep"][cu[b]:cu[b + 1]]], at
                to = to[:len(at)]
                page, first = s["table"][b].long()[at // size], s["table"][b].long()[to // size]
                scales[:, first, :, :, to % size] = s["scales"].double()[:, page, :, :, at % size]
            else:
                at = torch.arange(int(at[0]) // size * size, n, device=DEV)
                page = s["table"][b].long()[at // size]
                codes = s["codes"].view(torch.uint8)[page, 0, :, at % size].view(s["codes"].dtype).to(torch.float32).double()
                top = codes.abs().amax(-1) * s["scales"][page, 0, :, at % size].double()
                scales.index_reduce_(0, page, top / 127, "amax")
        return dict(lens=None, codes=None, scales=scales) if op == "compact" else dict(bounds=None, scales=scales)
    # attention in 64 bits over the pages that the rule picks, row by row
    rows = case["new"] * case["batch"]
    if rows * case["kv"] > 5000:
        return None
    size, kv, dim, group = case["page"], case["kv"], case["dim"], case["heads"] // case["kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    picks = torch.full((rows, kv, case["count"]), -1, dtype=torch.int32, device=DEV)
    lens, table = s["lens"].tolist(), s["table"].long()
    for b in range(case["batch"]):
        limits, steps = s["bounds"][table[b]].double(), s["bound_scales"][table[b]]
        for i in range(case["new"]):
            t, pos = b * case["new"] + i, lens[b] - case["new"] + i
            n = pos // size + 1
            for h in range(kv):
                q = s["q"][t, h * group:(h + 1) * group].double()
                w = torch.stack([torch.relu(q).sum(0), -torch.relu(-q).sum(0)]).float()
                top = w.abs().max() / torch.tensor(127.0, device=DEV)
                w = torch.round(w / top).double()
                if n <= case["count"]:
                    mine = torch.arange(n, device=DEV)
                else:
                    score = (limits[1:n - 1, h] * w).sum((1, 2)).float() * steps[1:n - 1, h]
                    best = torch.sort(-score, stable=True)[1][:case["count"] - 2] + 1
                    mine = torch.cat([torch.tensor([0, n - 1], device=DEV), best]).sort()[0]
                picks[t, h, :len(mine)] = mine.int()
                page = table[b][mine]
                key = (mine[:, None] * size + torch.arange(size, device=DEV)).view(-1) <= pos
                k, v = ((s["codes"].view(torch.uint8)[page, a, h].view(s["codes"].dtype).to(torch.float32).double()
                         * s["scales"][page, a, h].double()[..., None]).view(-1, dim)[key] for a in (0, 1))
                p = torch.softmax(q @ k.T.contiguous() / math.sqrt(dim), -1)
                out[t, h * group:(h + 1) * group] = p @ v
    return dict(picks=None, out=out)


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c, work(c))
