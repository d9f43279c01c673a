"""The attention half of a decoder layer, with W3G128 projections and a quantised
cache whose pages are counted on the GPU: what a server runs for each layer.

  prompt   q/k/v products of all rows -> rotary embedding, and the new keys and
           values into the cache -> qattn_prompt -> o product.  A prompt may come
           in chunks: the cached prefix is read back dense for the next one.
  verify   a tree of drafted tokens for each sequence (or one token): q/k/v
           products -> rotary embedding by depth and cache -> qattn_cache with the
           tree's masks -> o product.
  accept   the accepted path's rows move to the end of the context.
  step     one token for each sequence over the pages that its query selects.
  fork     sequences that follow others, page by page, as beams and samples do.

Run on a GPU:  python3 examples/attention_block.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dequant_gemv_qgemv_amd as q3  # noqa: E402


def random_weight(rows, cols, generator):
    """A packed W3G128 matrix and its scales, as a checkpoint holds them."""
    p = torch.tensor([0.1, 0.2, 0.4, 0.2, 0.1], device="cuda")
    codes = 2 + torch.multinomial(p, rows * cols, replacement=True, generator=generator).to(torch.uint8)
    scales = torch.randn(rows, cols // 128, device="cuda", generator=generator).abs() / math.sqrt(cols) + 1e-4
    return q3.qpack_uint3(codes.view(rows, cols)), scales.to(torch.bfloat16)


class AttentionBlock:
    def __init__(self, hidden=8192, heads=64, kv_heads=8, dim=128, pages=64, page_size=16, codes=torch.int8, seed=0, longest=1024):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.page_size = heads, kv_heads, dim, page_size
        # one matrix for q, k and v: their rows one below the other
        self.qkv = random_weight((heads + 2 * kv_heads) * dim, hidden, g)
        self.o = random_weight(hidden, heads * dim, g)
        self.codes, self.scales = q3.new_cache(pages, page_size, kv_heads, dim, codes)
        self.bounds = q3.new_bounds(self.codes)
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")  # who holds each page
        self.table = torch.empty((0, longest // page_size), dtype=torch.int32, device="cuda")
        self.lens = torch.empty(0, dtype=torch.int32, device="cuda")
        self.counts = []  # the same lengths on the host, which decides them here
        self.rates = 10000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)

    # -------------------------------------------------------- bookkeeping --
    def add(self):
        """A new, empty sequence: its number."""
        self.fork(list(range(len(self.counts))) + [-1])
        return len(self.counts) - 1

    def fork(self, parents):
        """Sequence i becomes what parents[i] is now (-1: empty); sequences that nobody follows end."""
        self.table, self.lens = q3.qcache_fork(self.refs, self.table, self.lens, self.ints(parents), self.page_size)
        self.counts = [self.counts[p] if p >= 0 else 0 for p in parents]

    def reserve(self, new):
        """Room for new[b] more tokens of sequence b: their slots, and the sequences' lengths with them."""
        slots, lens, copies = q3.qcache_reserve(self.refs, self.table, self.lens, self.page_size, cu=self.starts(new), total=sum(new))
        q3.qcache_copy(self.codes, self.scales, copies)  # pages that were shared until now
        # The host decides lengths here and has to know. A server lets the sequences whose lens did not grow wait; the
        # others keep the pages that they got and find them at the next call.
        if slots.numel() and int(slots.min()) < 0:
            raise RuntimeError("no room for the new tokens: %d pages, contexts of up to %d tokens"
                               % (self.refs.numel(), self.table.shape[1] * self.page_size))
        return slots, lens

    def spread(self, seqs, new):
        """The number of new tokens of each sequence, 0 for those that are not in seqs."""
        if len(set(seqs)) != len(seqs):
            raise ValueError("a sequence is named twice: %s" % (seqs,))
        each = [0] * len(self.counts)
        for b, n in zip(seqs, new):
            each[b] = n
        return each

    @staticmethod
    def by_number(call, seqs, new, x):
        """call(places in seqs, rows), whose rows are packed by their sequences' numbers, for rows x packed as seqs are."""
        order = sorted(range(len(seqs)), key=lambda i: seqs[i])
        if order == list(range(len(seqs))):
            return call(order, x)
        part = x.split(list(new))
        out = call(order, torch.cat([part[i] for i in order])).split([new[i] for i in order])
        return torch.cat([out[order.index(i)] for i in range(len(seqs))])

    @staticmethod
    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    @classmethod
    def starts(cls, n):
        return cls.ints([sum(n[:i]) for i in range(len(n) + 1)])

    # ------------------------------------------------------------ the layer --
    def project(self, x, positions, slots, dense=False):
        """Rotated q (bf16) of rows x [T, hidden], whose keys and values go into the cache; with `dense` those too."""
        y = q3.qgemm_w3g128_smallM(x, *self.qkv).view(x.shape[0], self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = y.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        return q3.qrope_write(q, k, v, self.ints(positions), self.rates, slots, self.codes, self.scales, dense=dense)

    def output(self, attended):
        return q3.qgemm_w3g128_smallM(attended.view(attended.shape[0], -1), *self.o)

    def prompt(self, seqs, new, x):
        """The next new[i] prompt tokens of sequence seqs[i], packed in x [sum(new), hidden]."""
        return self.by_number(lambda order, rows: self.prompt_rows([seqs[i] for i in order], [new[i] for i in order], rows), seqs, new, x)

    def prompt_rows(self, seqs, new, x):
        each = self.spread(seqs, new)
        slots, self.lens = self.reserve(each)
        q, k, v = self.project(x, [t for n, c in zip(each, self.counts) for t in range(c, c + n)], slots, dense=True)
        later = any(self.counts[b] for b in seqs)  # not the first chunk
        self.counts = [c + n for c, n in zip(self.counts, each)]
        cu_q = cu_k = self.starts(each)
        q3.qcache_bounds(self.codes, self.scales, self.table, self.lens, *self.bounds, cu_q=cu_q, total=sum(each))
        if later:  # the prefix comes back from the cache, this chunk with it
            cu_k = self.starts(self.counts)
            k, v = q3.qcache_read(self.codes, self.scales, self.table, cu_k, sum(self.counts))
        return self.output(q3.qattn_prompt(q, k, v, cu_q, cu_k))

    def verify(self, seqs, parents, x):
        """Drafted tokens of each sequence, x packed [sum of drafts, hidden]. parents[i][j]: the draft that draft j of
        seqs[i] follows, -1 for the last cached token. The drafts lie behind the context until accept()."""
        return self.by_number(lambda order, rows: self.verify_rows([seqs[i] for i in order], [parents[i] for i in order], rows), seqs,
                              [len(up) for up in parents], x)

    def verify_rows(self, seqs, parents, x):
        depth, words = [], []
        for b, up in zip(seqs, parents):
            d, w = [], []
            for j, p in enumerate(up):
                d.append(0 if p < 0 else d[p] + 1)
                w.append((0 if p < 0 else w[p]) | 1 << j)
            depth += [self.counts[b] + i for i in d]
            words += [i - (1 << 64) if i >> 63 else i for i in w]
        each = self.spread(seqs, [len(up) for up in parents])
        slots, self.ahead = self.reserve(each)
        self.drafts = each
        q = self.project(x, depth, slots)
        attended = q3.qattn_cache(q, self.codes, self.scales, self.table, self.ahead, cu_q=self.starts(self.drafts),
                                  tree=torch.tensor(words, dtype=torch.int64, device="cuda"))
        return self.output(attended)

    def accept(self, paths):
        """Of the drafts of the last verify() keep those on paths[b] of sequence b: their cache rows follow the context."""
        keep = [j in paths.get(b, ()) for b, n in enumerate(self.drafts) for j in range(n)]
        cu = self.starts(self.drafts)
        self.lens = q3.qcache_compact(self.codes, self.scales, self.table, self.ahead, torch.tensor(keep, device="cuda"), cu_q=cu)
        self.counts = [c + len(paths.get(b, ())) for b, c in enumerate(self.counts)]
        kept = [len(paths.get(b, ())) for b in range(len(self.counts))]
        q3.qcache_bounds(self.codes, self.scales, self.table, self.lens, *self.bounds, cu_q=self.starts(kept), total=sum(kept))

    def step(self, x, count):
        """One token for every sequence, x [sequences, hidden], which attends to `count` pages for each kv head."""
        each = [1] * len(self.counts)
        slots, self.lens = self.reserve(each)
        q = self.project(x, self.counts, slots)
        self.counts = [c + 1 for c in self.counts]
        q3.qcache_bounds(self.codes, self.scales, self.table, self.lens, *self.bounds)
        picks = q3.qblock_select(q, *self.bounds, self.table, self.lens, count, self.page_size)
        return self.output(q3.qattn_blocks(q, self.codes, self.scales, self.table, self.lens, picks))


def demo(hidden=1024, heads=8, kv_heads=2, dim=128, codes=torch.int8, verbose=True):
    """Two prompts, the second in two chunks, then a drafted tree for each; the accepted path's outputs, and those of the
    next tokens of both sequences and of a fork of the first, against the same tokens as a plain prompt. Returns the largest
    relative difference (the cache holds 8 bits)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(2, 80, hidden, device="cuda", generator=g).to(torch.bfloat16)
    block = AttentionBlock(hidden, heads, kv_heads, dim, codes=codes)
    a, b = block.add(), block.add()
    block.prompt([a], [50], x[0, :50])
    block.prompt([b], [20], x[1, :20])
    block.prompt([b], [17], x[1, 20:37])
    #   0 -> 1 -> 3 and 0 -> 2: token 1 and 3 are the ones that follow in x, 2 is a wrong guess
    parents = [[-1, 0, 0, 1]] * 2
    wrong = torch.randn(1, hidden, device="cuda", generator=g).to(torch.bfloat16)
    drafts = torch.cat([torch.cat([x[i, n:n + 2], wrong, x[i, n + 2:n + 3]]) for i, n in ((0, 50), (1, 37))])
    got = block.verify([a, b], parents, drafts).view(2, 4, -1)[:, [0, 1, 3]]
    block.accept({a: [0, 1, 3], b: [0, 1, 3]})
    # one more token for each, and for a fork of the first, which goes on with another one
    block.fork([a, b, a])
    step = block.step(torch.stack([x[0, 53], x[1, 40], wrong[0]]), count=8)  # as many pages as there are

    plain = AttentionBlock(hidden, heads, kv_heads, dim, codes=codes)
    want = plain.prompt([plain.add(), plain.add(), plain.add()], [54, 41, 54], torch.cat([x[0, :54], x[1, :41], x[0, :53], wrong]))
    far = 0.0
    for i, end in ((0, 54), (1, 95), (2, 149)):
        w = want[end - 4:end] if i < 2 else want[end - 1:end]
        have = torch.cat([got[i], step[i:i + 1]]) if i < 2 else step[2:]
        far = max(far, float((have - w).norm() / w.norm()))
    if verbose:
        print("largest relative difference from the unquantised prompt: %.4f" % far)
    return far


if __name__ == "__main__":
    demo()
    demo(codes=torch.float8_e4m3fn)
    demo(8192, 64, 8, 128)
