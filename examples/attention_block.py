"""The attention half of a decoder layer, with W3G128 projections and a quantised
cache: what a server runs for each layer.

  prompt   q/k/v products of all rows -> rotary embedding -> the new keys and
           values into the cache -> qattn_prompt -> o product.  A prompt may come
           in chunks: the cached prefix is read back dense for the next one.
  verify   a tree of drafted tokens for each sequence (or one token): q/k/v
           products -> rotary embedding by depth -> cache -> qattn_cache with the
           tree's masks -> o product.
  accept   the accepted path's rows move to the end of the context.

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
    def __init__(self, hidden=8192, heads=64, kv_heads=8, dim=128, pages=64, page_size=16, codes=torch.int8, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.page_size = heads, kv_heads, dim, page_size
        # one matrix for q, k and v: their rows one below the other
        self.qkv = random_weight((heads + 2 * kv_heads) * dim, hidden, g)
        self.o = random_weight(hidden, heads * dim, g)
        self.codes, self.scales = q3.new_cache(pages, page_size, kv_heads, dim, codes)
        self.free = list(range(pages))
        self.tables = []   # the pages of each sequence
        self.lens = []     # its cached tokens
        self.rate = 10000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float32) / dim)

    # -------------------------------------------------------- bookkeeping --
    def add(self):
        self.tables.append([])
        self.lens.append(0)
        return len(self.lens) - 1

    def reserve(self, seqs, new):
        """Pages for `new` more tokens of each sequence; the slots of those tokens, in order."""
        slots = []
        for b, n in zip(seqs, new):
            table = self.tables[b]
            while len(table) * self.page_size < self.lens[b] + n:
                table.append(self.free.pop())
            slots += [table[t // self.page_size] * self.page_size + t % self.page_size
                      for t in range(self.lens[b], self.lens[b] + n)]
        return torch.tensor(slots, dtype=torch.int64, device="cuda")

    def block_table(self, seqs):
        most = max(len(self.tables[b]) for b in seqs)
        return torch.tensor([self.tables[b] + [0] * (most - len(self.tables[b])) for b in seqs], dtype=torch.int32,
                            device="cuda")

    @staticmethod
    def starts(n):
        return torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")

    # ------------------------------------------------------------ the layer --
    def project(self, x, positions):
        """q (bf16, rotated), k (float32, rotated) and v (a float32 view) of rows x [T, hidden]."""
        y = q3.qgemm_w3g128_smallM(x, *self.qkv).view(x.shape[0], self.heads + 2 * self.kv_heads, self.dim)
        qk, v = y[:, :self.heads + self.kv_heads], y[:, self.heads + self.kv_heads:]
        angle = positions.float()[:, None, None] * self.rate
        cos, sin = angle.cos(), angle.sin()
        a, b = qk[..., :self.dim // 2], qk[..., self.dim // 2:]
        qk = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return qk[:, :self.heads].to(torch.bfloat16), qk[:, self.heads:].contiguous(), v

    def output(self, attended):
        return q3.qgemm_w3g128_smallM(attended.view(attended.shape[0], -1), *self.o)

    def prompt(self, seqs, new, x):
        """The next new[i] prompt tokens of sequence seqs[i], packed in x [sum(new), hidden]."""
        at = [self.lens[b] for b in seqs]
        positions = torch.cat([torch.arange(p, p + n, device="cuda") for p, n in zip(at, new)])
        q, k, v = self.project(x, positions)
        q3.qcache_write(k, v, self.reserve(seqs, new), self.codes, self.scales)
        for b, n in zip(seqs, new):
            self.lens[b] += n
        cu_q = self.starts(new)
        if any(at):  # a later chunk: the prefix comes back from the cache, this chunk with it
            lens = [self.lens[b] for b in seqs]
            cu_k = self.starts(lens)
            kd, vd = q3.qcache_read(self.codes, self.scales, self.block_table(seqs), cu_k, sum(lens))
        else:
            cu_k, kd, vd = cu_q, k.to(torch.bfloat16), v.to(torch.bfloat16)
        return self.output(q3.qattn_prompt(q, kd, vd, cu_q, cu_k))

    def verify(self, seqs, parents, x):
        """Drafted tokens of each sequence, x packed [sum of drafts, hidden]. parents[i][j]: the draft that draft j of
        seqs[i] follows, -1 for the last cached token. The drafts lie behind the context until accept()."""
        depth, words = [], []
        for b, up in zip(seqs, parents):
            d, w = [], []
            for j, p in enumerate(up):
                d.append(0 if p < 0 else d[p] + 1)
                w.append((0 if p < 0 else w[p]) | 1 << j)
            depth += [self.lens[b] + i for i in d]
            words += [i - (1 << 64) if i >> 63 else i for i in w]
        new = [len(up) for up in parents]
        q, k, v = self.project(x, torch.tensor(depth, device="cuda"))
        q3.qcache_write(k, v, self.reserve(seqs, new), self.codes, self.scales)
        lens = torch.tensor([self.lens[b] + n for b, n in zip(seqs, new)], dtype=torch.int32, device="cuda")
        attended = q3.qattn_cache(q, self.codes, self.scales, self.block_table(seqs), lens,
                                  cu_q=None if all(n == 1 for n in new) else self.starts(new),
                                  tree=torch.tensor(words, dtype=torch.int64, device="cuda"))
        return self.output(attended)

    def accept(self, b, path):
        """Keep the drafts on `path` (ascending) of sequence b: their cache rows follow the context."""
        def place(t):
            return self.tables[b][t // self.page_size], t % self.page_size
        raw = self.codes.view(torch.uint8)
        for i, j in enumerate(path):
            (p0, s0), (p1, s1) = place(self.lens[b] + j), place(self.lens[b] + i)
            raw[p1, :, :, s1] = raw[p0, :, :, s0]
            self.scales[p1, :, :, s1] = self.scales[p0, :, :, s0]
        self.lens[b] += len(path)


def demo(hidden=1024, heads=8, kv_heads=2, dim=128, codes=torch.int8, verbose=True):
    """Two prompts, the second in two chunks, then a drafted tree for each; the accepted path's outputs against those of
    the same tokens as a plain prompt. Returns the largest relative difference (the cache holds 8 bits)."""
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
    for s in (a, b):
        block.accept(s, [0, 1, 3])
    step = block.verify([a, b], [[-1], [-1]], torch.stack([x[0, 53], x[1, 40]]))  # one more token for each

    plain = AttentionBlock(hidden, heads, kv_heads, dim, codes=codes)
    want = plain.prompt([plain.add(), plain.add()], [54, 41], torch.cat([x[0, :54], x[1, :41]]))
    far = 0.0
    for i, end in ((0, 54), (1, 95)):
        w = want[end - 4:end]
        have = torch.cat([got[i], step[i:i + 1]])
        far = max(far, float((have - w).norm() / w.norm()))
    if verbose:
        print("largest relative difference from the unquantised prompt: %.4f" % far)
    return far


if __name__ == "__main__":
    demo()
    demo(codes=torch.float8_e4m3fn)
    demo(8192, 64, 8, 128)
