"""examples/attention_block.py where its demo does not go: what a caller may hand to it, and what it has to refuse."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def block(**kwargs):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod.AttentionBlock(1024, 8, 2, 128, **kwargs)


def tokens(n):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    return torch.randn(n, 1024, device="cuda", generator=g).to(torch.bfloat16)


def test_no_room_is_an_error_and_loses_nothing():
    b = block(pages=5)
    first, second = b.add(), b.add()
    b.prompt([first], [40], tokens(40))
    b.fork([first, second, first])  # 3 pages, the last of them shared and partly filled
    with pytest.raises(RuntimeError, match="room"):
        b.prompt([second], [64], tokens(64))
    with pytest.raises(RuntimeError, match="room"):
        b.verify([second], [[-1] * 33], tokens(33))
    with pytest.raises(RuntimeError, match="room"):  # copies for both holders of the shared page, and a page for the empty one
        b.step(tokens(3), 4)
    assert b.counts == [40, 0, 40] == b.lens.tolist()
    # what got room above kept it, and its tokens
    b.fork([0, 2])
    out = b.step(tokens(2), 4)
    alone = block(pages=20)
    alone.add(), alone.add()
    alone.prompt([0, 1], [40, 40], torch.cat([tokens(40), tokens(40)]))
    assert torch.equal(out, alone.step(tokens(2), 4))


def test_a_context_longer_than_a_table_is_an_error():
    b = block(pages=40, longest=64)
    with pytest.raises(RuntimeError, match="room"):
        b.prompt([b.add()], [65], tokens(65))


def test_sequences_in_any_order():
    """Prompts, chunks and drafts packed in the caller's order, whatever numbers their sequences have."""
    x = tokens(150)
    parents = [[-1, 0, 0], [-1], [-1, 0, 1, 1]]
    straight, turned = block(), block()
    for b in (straight, turned):
        for _ in range(3):
            b.add()
    for new, at in (([30, 20, 40], 0), ([1, 7, 16], 90)):  # then a second chunk
        part = x[at:at + sum(new)].split(new)
        want = straight.prompt([0, 1, 2], new, torch.cat(part)).split(new)
        got = turned.prompt([2, 0, 1], [new[i] for i in (2, 0, 1)], torch.cat([part[i] for i in (2, 0, 1)])).split([new[i] for i in (2, 0, 1)])
        assert all(torch.equal(got[j], want[i]) for j, i in enumerate((2, 0, 1)))
    n = [3, 1, 4]
    part = x[114:122].split(n)
    want = straight.verify([0, 1, 2], parents, torch.cat(part)).split(n)
    got = turned.verify([1, 2, 0], [parents[i] for i in (1, 2, 0)], torch.cat([part[i] for i in (1, 2, 0)])).split([1, 4, 3])
    assert all(torch.equal(got[j], want[i]) for j, i in enumerate((1, 2, 0)))
    for b in (straight, turned):
        b.accept({0: [0, 2], 2: [0, 1, 3]})
    assert torch.equal(straight.step(x[122:125], 3), turned.step(x[122:125], 3))
    with pytest.raises(ValueError):
        turned.prompt([1, 1], [2, 2], x[:4])
