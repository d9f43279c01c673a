"""Workloads of the attention operators around the W3G128 products.

Four operators, by a case's "op":
  prompt  qattn_prompt   attention of packed sequences, causal, grouped heads
  write   qcache_write   quantise keys and values into a paged cache, and
          qcache_read    read them back (the round trip that a prompt's next
                         chunk makes)
  read    qcache_read    a long prefix read back dense
  cache   qattn_cache    attention over the quantised cache: single tokens, or
                         a tree of drafted tokens per sequence

With `own` false, run() computes the same results from elementary torch
operations in 32 bits; with `own` true it calls the package.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # A short question to one user: the prompt call whose launch time counts.
        dict(name="prompt_37", op="prompt", batch=1, lo=37, hi=37, prefix=0, heads=64, kv=8, dim=128, causal=True),
        # A whole prompt of 8192 tokens at the 70B layer's heads: the largest case, bound by the matrix unit.
        dict(name="prompt_8192", op="prompt", batch=1, lo=8192, hi=8192, prefix=0, heads=64, kv=8, dim=128, causal=True),
        # Twelve waiting requests of 3 to 2500 tokens packed into one call, at 16 heads over 4.
        dict(name="prompt_packed", op="prompt", batch=12, lo=3, hi=2500, prefix=0, heads=16, kv=4, dim=128, causal=True),
        # The next 511 tokens of two prompts against 6000 earlier ones, heads of 64 channels.
        dict(name="prompt_chunk_d64", op="prompt", batch=2, lo=511, hi=511, prefix=6000, heads=32, kv=8, dim=64, causal=True),
        # A decode step of 32 sequences: one new token each, straight from the fp32 outputs of the products.
        dict(name="write_step_32", op="write", tokens=32, kv=8, dim=128, page=16, codes="int8", src="fp32"),
        # A prompt of 8191 tokens goes into the cache and comes back for its next chunk.
        dict(name="write_prompt_8191", op="write", tokens=8191, kv=8, dim=128, page=64, codes="fp8", src="bf16"),
        # The cached prefixes of eight sequences, 500 to 30001 tokens, read back dense.
        dict(name="read_prefix", op="read", batch=8, lo=500, hi=30001, kv=8, dim=128, page=16, codes="int8"),
        # One token of one user, a short conversation: latency.
        dict(name="decode_b1", op="cache", batch=1, lo=1000, hi=1000, draft=1, tree=False, heads=64, kv=8, dim=128, page=16, codes="int8"),
        # One token of one user with a very long document: the cache read split over the whole card.
        dict(name="decode_long", op="cache", batch=1, lo=131071, hi=131071, draft=1, tree=False, heads=64, kv=8, dim=128, page=64, codes="int8"),
        # A decode step of 48 sequences of very different lengths.
        dict(name="decode_batch", op="cache", batch=48, lo=17, hi=16000, draft=1, tree=False, heads=64, kv=8, dim=128, page=16, codes="int8"),
        # Verifying a tree of 13 drafted tokens for four users, fp8 codes, heads of 64 channels.
        dict(name="tree_13_d64", op="cache", batch=4, lo=700, hi=5000, draft=13, tree=True, heads=32, kv=8, dim=64, page=32, codes="fp8"),
        # Verifying trees of 64 drafted tokens for eight users: 512 query rows share each cached key.
        dict(name="tree_64", op="cache", batch=8, lo=1500, hi=8000, draft=64, tree=True, heads=64, kv=8, dim=128, page=16, codes="int8"),
    ]


def draw(rng):
    def log(a, b):
        return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))

    op = rng.choice(["prompt", "prompt", "write", "read", "cache", "cache", "cache"])
    kv = rng.choice([1, 2, 4, 8, 8])
    dim = rng.choice([64, 128, 128])
    heads = kv * rng.choice([1, 2, 4, 5, 7, 8])
    if op == "prompt":
        batch = rng.choice([1, 1, 2, 5, 12])
        hi = log(1, 8192 if batch == 1 else 4000)
        prefix = rng.choice([0, 0, log(1, 6000)])
        return dict(op=op, batch=batch, lo=log(1, hi), hi=hi, prefix=prefix if hi <= 2048 else 0, heads=heads, kv=kv,
                    dim=dim, causal=rng.random() < 0.8)
    page = rng.choice([16, 16, 32, 64, 128])
    codes = rng.choice(["int8", "fp8"])
    if op == "write":
        return dict(op=op, tokens=log(1, 20000), kv=kv, dim=dim, page=page, codes=codes, src=rng.choice(["fp32", "bf16"]))
    batch = log(1, 64)
    hi = log(1, min(131071, 262144 // batch))
    lo = log(1, hi)
    if op == "read":
        return dict(op=op, batch=batch, lo=lo, hi=hi, kv=kv, dim=dim, page=page, codes=codes)
    draft = rng.choice([1, 1, log(2, 64)])
    if draft > 1:
        hi = min(hi, 16000)
        hi = max(draft, min(hi, 64000 // batch))
        lo = max(draft, min(lo, hi))
    return dict(op=op, batch=batch, lo=lo, hi=hi, draft=draft, tree=draft > 1 and rng.random() < 0.75, heads=heads, kv=kv,
                dim=dim, page=page, codes=codes)


def lengths(case):
    """The sequences' lengths: the first is `hi`, the others spread over lo..hi by their logarithm."""
    lo, hi, n = case["lo"], case["hi"], case["batch"]
    got = [hi]
    for i in range(1, n):
        u = math.modf(0.5 + i * 0.6180339887498949)[0]
        got.append(max(lo, min(hi, int(round(lo * (hi / lo) ** u)))))
    return got


def visible(case):
    """How many (query, key) pairs a case has, for one query head."""
    total = 0
    for n in lengths(case):
        if case["op"] == "prompt":
            k = n + case["prefix"]
            total += n * k - (n * (n - 1) // 2 if case["causal"] else 0)
        else:
            d = case["draft"]
            # a random tree of d nodes: about ln(d) + 1 ancestors each; a chain: (d + 1) / 2
            total += d * (n - d) + int(d * (math.log(d) + 1) if case["tree"] else d * (d + 1) // 2)
    return total


def work(case):
    op, kv, dim = case["op"], case["kv"], case["dim"]
    if op == "write":
        t = case["tokens"] * kv * 2
        size = 4 if case["src"] == "fp32" else 2
        return {"bytes": t * (dim * size + dim + 4) + t * (dim + 4 + 2 * dim) + case["tokens"] * 8, "flops": 3 * t * dim}
    n = lengths(case)
    if op == "read":
        t = sum(n) * kv * 2
        return {"bytes": t * (dim + 4 + 2 * dim), "flops": t * dim}
    flops = 4 * dim * case["heads"] * visible(case)
    if op == "prompt":
        q = sum(n)
        return {"bytes": 2 * dim * (2 * q * case["heads"] + 2 * (q + case["prefix"] * len(n)) * kv), "flops": flops}
    q = case["draft"] * len(n)
    return {"bytes": sum(n) * kv * 2 * (dim + 4) + 4 * dim * case["heads"] * q, "flops": flops}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)
    return g


def _heads(g, tokens, heads, dim, dtype):
    """Rows as projections give them: every head with a few channels larger than the rest."""
    x = torch.randn(tokens, heads, dim, device=DEV, generator=g)
    x *= torch.exp(0.5 * torch.randn(1, heads, dim, device=DEV, generator=g))
    return x.to(dtype)


def _starts(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)


def _tables(rng, n, page):
    """A block table [batch, pages of the longest] over pages in random order, and the number of pages."""
    need = [-(-x // page) for x in n]
    ids = rng.permutation(sum(need) + 3)
    table = np.zeros((len(n), max(need)), np.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = ids[at:at + c]
        at += c
    return torch.tensor(table, device=DEV), sum(need) + 3


def _ancestors(rng, batch, n):
    """One random tree of n drafted tokens for each sequence: bit j of row i says that i descends from j or is it."""
    rows = np.zeros((batch, n), np.uint64)
    for b in range(batch):
        for i in range(n):
            up = rows[b, rng.integers(0, i)] if i else np.uint64(0)
            rows[b, i] = up | (np.uint64(1) << np.uint64(i))
    return torch.tensor(rows.view(np.int64).reshape(-1), device=DEV)


def _cache(g, pages, case):
    """A filled cache: codes [pages, 2, kv, page, dim], scales [pages, 2, kv, page]."""
    shape = (pages, 2, case["kv"], case["page"], case["dim"])
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
    op, kv, dim = case["op"], case["kv"], case["dim"]
    s = dict(case=dict(case))
    if op == "prompt":
        n = lengths(case)
        m = [x + case["prefix"] for x in n]
        s.update(q=_heads(g, sum(n), case["heads"], dim, torch.bfloat16), k=_heads(g, sum(m), kv, dim, torch.bfloat16),
                 v=_heads(g, sum(m), kv, dim, torch.bfloat16), cu_q=_starts(n), cu_k=_starts(m), lq=max(n), lk=max(m))
        return s
    if op == "write":
        src = torch.float32 if case["src"] == "fp32" else torch.bfloat16
        t = case["tokens"]
        # one sequence whose pages lie in random order
        table, pages = _tables(rng, [t], case["page"])
        at = torch.arange(t, device=DEV)
        slots = table[0].long()[at // case["page"]] * case["page"] + at % case["page"]
        code = torch.int8 if case["codes"] == "int8" else torch.float8_e4m3fn
        s.update(k=_heads(g, t, kv, dim, src), v=_heads(g, t, kv, dim, src), slots=slots, table=table, cu=_starts([t]),
                 total=t, lk=t, codes=torch.zeros(pages, 2, kv, case["page"], dim, device=DEV).to(code),
                 scales=torch.zeros(pages, 2, kv, case["page"], device=DEV))
        return s
    n = lengths(case)
    table, pages = _tables(rng, n, case["page"])
    codes, scales = _cache(g, pages, case)
    s.update(table=table, codes=codes, scales=scales, lk=max(n))
    if op == "read":
        s.update(cu=_starts(n), total=sum(n))
        return s
    d = case["draft"]
    s.update(q=_heads(g, d * len(n), case["heads"], dim, torch.bfloat16), lens=torch.tensor(n, dtype=torch.int32, device=DEV),
             cu_q=_starts([d] * len(n)) if d > 1 else None, tree=_ancestors(rng, len(n), d) if case["tree"] else None)
    return s


def run(s):
    if own:
        return _own(s)
    return {"prompt": _plain_prompt, "write": _plain_write, "read": _plain_read, "cache": _plain_cache}[s["case"]["op"]](s)


def _own(s):
    import dequant_gemv_qgemv_amd as q
    op = s["case"]["op"]
    if op == "prompt":
        return q.qattn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=s["case"]["causal"])
    if op == "write":
        q.qcache_write(s["k"], s["v"], s["slots"], s["codes"], s["scales"])
        k, v = q.qcache_read(s["codes"], s["scales"], s["table"], s["cu"], s["total"])
        return {"k": k, "v": v, "scales": s["scales"]}
    if op == "read":
        return q.qcache_read(s["codes"], s["scales"], s["table"], s["cu"], s["total"])
    return q.qattn_cache(s["q"], s["codes"], s["scales"], s["table"], s["lens"], cu_q=s["cu_q"], tree=s["tree"])


# ------------------------------------------------------------ plain forms ---
def _attend(q, k, v, seen):
    """softmax(q k^T / sqrt(dim)) v over the keys seen.

    q [batch, rows, heads, dim], k and v [batch, keys, kv, dim] in fp32, seen [batch, rows, keys]; rows that see no key
    get zeros."""
    b, r, h, d = q.shape
    kv = k.shape[2]
    g = h // kv
    q = q.view(b, r, kv, g, d).permute(0, 2, 3, 1, 4).reshape(b, kv, g * r, d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * (1 / math.sqrt(d))
    s = s.view(b, kv, g, r, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, kv, g * r, -1), v.permute(0, 2, 1, 3).contiguous()).view(b, kv, g, r, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.permute(0, 3, 1, 2, 4).reshape(b, r, h, d)


def _padded(x, cu, most):
    """Packed rows [total, ...] as [batch, most, ...], rows past a sequence's end those of another (masked later)."""
    at = cu[:-1].long()[:, None] + torch.arange(most, device=DEV)[None]
    return x[at.clamp_(max=x.shape[0] - 1)]


def _packed(x, cu, total):
    """[batch, most, ...] back to the packed rows [total, ...]."""
    at = torch.arange(total, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), at, right=True)
    return x[b, at - cu.long()[b]]


def _plain_prompt(s):
    cu_q, cu_k = s["cu_q"], s["cu_k"]
    nq, nk = (cu_q[1:] - cu_q[:-1])[:, None, None], (cu_k[1:] - cu_k[:-1])[:, None, None]
    i = torch.arange(s["lq"], device=DEV)[None, :, None]
    j = torch.arange(s["lk"], device=DEV)[None, None, :]
    seen = (i < nq) & (j < nk)
    if s["case"]["causal"]:
        seen = seen & (j <= i + nk - nq)
    o = _attend(_padded(s["q"], cu_q, s["lq"]).float(), _padded(s["k"], cu_k, s["lk"]).float(),
                _padded(s["v"], cu_k, s["lk"]).float(), seen)
    return _packed(o, cu_q, s["q"].shape[0]).to(torch.bfloat16)


def _plain_write(s):
    case = s["case"]
    x = torch.stack([s["k"], s["v"]], 1).float()  # [tokens, 2, kv, dim]
    top = x.abs().amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(x).all(-1, keepdim=True), top, torch.full_like(top, math.nan))
    limit = torch.full_like(top, 127.0 if case["codes"] == "int8" else 448.0)
    scale = top / limit
    y = torch.where(scale > 0, x / scale, torch.zeros_like(x))
    page, at = s["slots"] // case["page"], s["slots"] % case["page"]
    if case["codes"] == "int8":
        s["codes"][page, :, :, at] = y.round().clamp(-127, 127).to(torch.int8)
    else:
        s["codes"].view(torch.uint8)[page, :, :, at] = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s["scales"][page, :, :, at] = scale[..., 0]
    k, v = _plain_read(s)
    return {"k": k, "v": v, "scales": s["scales"]}


def _values(codes, scales, page, at):
    """Keys and values [..., kv, dim] in fp32 of the tokens at (page, at)."""
    c = codes.view(torch.uint8)[page, :, :, at].view(codes.dtype).float()
    x = c * scales[page, :, :, at][..., None]
    return x.select(-3, 0), x.select(-3, 1)


def _plain_read(s):
    size = s["case"]["page"]
    row = torch.arange(s["total"], device=DEV)
    b = torch.searchsorted(s["cu"][1:].contiguous(), row, right=True)
    pos = row - s["cu"].long()[b]
    k, v = _values(s["codes"], s["scales"], s["table"].long()[b, pos // size], pos % size)
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _plain_cache(s):
    case = s["case"]
    size, d, batch = case["page"], case["draft"], case["batch"]
    lens = s["lens"].long()[:, None, None]
    j = torch.arange(s["lk"], device=DEV)
    page = s["table"].long()[:, j // size]
    k, v = _values(s["codes"], s["scales"], page, (j % size).expand(batch, -1))
    i = torch.arange(d, device=DEV)[None, :, None]
    j = j[None, None, :]
    if s["tree"] is None:
        seen = j <= lens - d + i
    else:
        bit = (j - (lens - d)).clamp(0, 63)
        seen = (j < lens - d) | ((j < lens) & ((s["tree"].view(batch, d, 1) >> bit) & 1 == 1))
    o = _attend(s["q"].float().view(batch, d, case["heads"], case["dim"]), k, v, seen)
    return o.reshape(batch * d, case["heads"], case["dim"]).to(torch.bfloat16)


# --------------------------------------------------- definition in 64 bits ---
def _e4m3(y):
    """The e4m3 value nearest to y, ties to the even mantissa."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    e = e - (torch.exp2(e) > y.abs().clamp(min=2.0 ** -6)).double()
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def exact(case, seed):
    if visible(case) * case["heads"] > 1.2e10 if case["op"] in ("prompt", "cache") else False:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "write":
        out = []
        scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device=DEV)
        for which, x in enumerate((s["k"].double(), s["v"].double())):
            t = x.abs().max(dim=2).values / (127 if case["codes"] == "int8" else 448)
            y = x / t[:, :, None]
            out.append((torch.round(y) if case["codes"] == "int8" else _e4m3(y)) * t[:, :, None])
            flat = scales[:, which].transpose(1, 2).contiguous().view(-1, case["kv"])  # by slot
            flat[s["slots"]] = t
            scales[:, which] = flat.view(-1, case["page"], case["kv"]).transpose(1, 2)
        return {"k": out[0], "v": out[1], "scales": scales}

    n = lengths(case)

    def keys(b, which):
        used = s["table"][b, :-(-n[b] // case["page"])].long()
        c = s["codes"].view(torch.uint8)[used, which].view(s["codes"].dtype).to(torch.float32).double()
        x = (c * s["scales"][used, which].double()[..., None]).transpose(1, 2)
        return x.reshape(-1, case["kv"], case["dim"])[:n[b]]

    if op == "read":
        return tuple(torch.cat([keys(b, which) for b in range(len(n))]) for which in (0, 1))
    g = case["heads"] // case["kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    q0 = k0 = 0
    for b, length in enumerate(n):
        if op == "prompt":
            nq, nk = length, length + case["prefix"]
            k, v = s["k"][k0:k0 + nk].double(), s["v"][k0:k0 + nk].double()
        else:
            nq, nk = case["draft"], length
            k, v = keys(b, 0), keys(b, 1)
        j = torch.arange(nk, device=DEV)
        for i0 in range(0, nq, 1024):
            i = torch.arange(i0, min(nq, i0 + 1024), device=DEV)
            if op == "prompt":
                hidden = (j[None] > i[:, None] + nk - nq) if case["causal"] else torch.zeros(len(i), nk, dtype=torch.bool, device=DEV)
            elif s["tree"] is None:
                hidden = j[None] > nk - nq + i[:, None]
            else:
                word = s["tree"][q0 + i][:, None]
                hidden = (j[None] >= nk - nq) & (((word >> (j - (nk - nq)).clamp(min=0, max=63)[None]) & 1) == 0)
            for h in range(case["heads"]):
                t = (s["q"][q0 + i, h].double() @ k[:, h // g].T.contiguous()) / math.sqrt(case["dim"])
                t = t.masked_fill(hidden, -math.inf)
                p = torch.exp(t - t.max(dim=1, keepdim=True).values.clamp(min=-1e300))
                out[q0 + i, h] = (p @ v[:, h // g].contiguous()) / p.sum(dim=1, keepdim=True).clamp(min=1e-300)
        q0, k0 = q0 + nq, k0 + nk
    return out


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c, work(c))
