"""The counting check of oracle/attention.py sees what it is for: outputs that a
kernel would give if it lost a key, a run of keys, or counted one twice.  The
mistake is planted here, in the computed output."""
import numpy as np
import pytest

from oracle import attention as ref


def output(seen, values, weight=None):
    """What a kernel gives: rounded to bf16."""
    w = np.asarray(seen, np.float64) * (1.0 if weight is None else weight)
    o = (w @ values / np.maximum(w.sum(axis=1, keepdims=True), 1)).astype(np.float32)
    return ref.bf16_values(ref.to_bf16(o))


@pytest.mark.parametrize("n", [1, 64, 700, 5000, 9001, 20000, 30000])
@pytest.mark.parametrize("dim", [64, 128])
def test_one_lost_or_doubled_key_shows(n, dim):
    rng = np.random.default_rng(n + dim)
    parts = ref.counting_parts(n, dim)
    seen = np.ones((1, n))
    for part in range(parts):
        v = ref.counting_values(n, dim, part, parts)
        assert v.sum(axis=0).max() <= 96
        assert not ref.miscounted(output(seen, v), seen, v).any()
    for j in {0, n - 1} | set(rng.integers(0, n, 20).tolist()):
        v = ref.counting_values(n, dim, (j // (32 * dim)) % parts, parts)
        assert v[j, (j // 32) % dim] == 1
        for times in (0, 2):
            w = np.ones(n)
            w[j] = times
            if n > 1:
                assert ref.miscounted(output(seen, v, w), seen, v).any(), (j, times)


@pytest.mark.parametrize("n", [700, 4000, 9000, 20000])
@pytest.mark.parametrize("run", [16, 32, 64, 128, 512])
@pytest.mark.parametrize("times", [0, 2])
def test_a_lost_or_doubled_run_of_keys_shows(n, run, times):
    parts = ref.counting_parts(n, 128)
    seen = np.ones((1, n))
    for at in (0, n // 2 // run * run, n - run):
        w = np.ones(n)
        w[at:at + run] = times
        assert any(ref.miscounted(output(seen, v, w), seen, v).any()
                   for v in (ref.counting_values(n, 128, part, parts) for part in range(parts)))


def test_values_of_all_sets_cover_every_key():
    for n, dim in ((1, 64), (12801, 128), (30000, 64)):
        parts = ref.counting_parts(n, dim)
        assert sum(ref.counting_values(n, dim, p, parts).sum() for p in range(parts)) == n


def test_weights_of_one_bf16_leave_the_bound_of_two():
    q, k = np.zeros(64), np.zeros((40, 64))
    q[0], k[20:, 0] = 1.0, ref.HALF_WAY
    p = np.exp(ref.HALF_WAY)
    v = np.full((40, 64), 1.0)
    v[:20] = -p
    w = np.exp(k @ q)
    one = ref.bf16_values(ref.to_bf16(w.astype(np.float32)))
    two = one + ref.bf16_values(ref.to_bf16((w - one).astype(np.float32)))
    want, bound = ref.attend(q, k, v, np.arange(40), 1.0, 2.0 ** -16)
    for weights, inside in ((two, True), (one, False)):
        got = ref.bf16_values(ref.to_bf16((weights @ v / w.sum()).astype(np.float32)))
        assert (np.abs(got - want) <= bound).all() == inside
    assert (np.abs(got - want) > 20 * bound).all()
