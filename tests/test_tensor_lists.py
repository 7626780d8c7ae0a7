"""The compiled module that checks lists of tensors (CPU only)."""
import random

import pytest
import torch

from rank_randomized_gradient_amd import rgc


@pytest.fixture(scope="module")
def lists():
    return rgc._lists()


def _span(lists, ts):
    p, c, name, _ = lists.pack(ts, None, 1)
    return p, c, rgc._ITEM_BYTES[name]


def test_shared_memory(lists):
    x = torch.zeros(1024)
    span = lambda *ts: _span(lists, list(ts))  # noqa: E731
    far, other = torch.zeros(64), torch.zeros(64)
    free = span(far)
    assert lists.disjoint(free, span(x[:64], x[64:128]))
    assert lists.disjoint(free, span(x[64:128], x[:64]))
    assert not lists.disjoint(free, span(x[:64], x[63:128]))  # neighbours that share an element
    assert not lists.disjoint(free, span(x[64:128], x[:65]))
    assert not lists.disjoint(free, span(x[:64], x[:64]))
    assert not lists.disjoint(free, span(x[:64], other), span(x[32:64]))  # two lists
    assert not lists.disjoint(free, span(x), span(x[500:501]))  # one within the other
    assert lists.disjoint(free, span(x[:64]), span(x[64:65], other))
    assert not lists.disjoint(span(x[10:11]), span(x[:64]))  # read and written
    assert not lists.disjoint(span(x[63:70]), span(x[:64], x[100:101]))
    assert lists.disjoint(span(x[64:100], x[64:100], x[70:90]), span(x[:64], x[100:101]))  # only read
    assert lists.disjoint(free, span(x[:64], x[5:5], x[7:7]))  # tensors of nothing
    y = torch.zeros(64, dtype=torch.bfloat16)
    assert lists.disjoint(span(y[:32]), span(y[32:]))


def test_many_against_every_pair(lists):
    rng = random.Random(1)
    x = torch.zeros(4000)
    for _ in range(300):
        def some(n):
            cuts = [rng.randrange(3900) for _ in range(n)]
            return [(a, a + rng.choice([0, 1, 5, 40])) for a in cuts]

        read, w1, w2 = some(rng.randrange(1, 6)), some(rng.randrange(1, 6)), some(rng.randrange(1, 6))
        meet = lambda a, b: max(a[0], b[0]) < min(a[1], b[1])  # noqa: E731
        w = w1 + w2
        want = not any(meet(w[i], w[j]) for i in range(len(w)) for j in range(i)) and not any(meet(a, b) for a in read for b in w)
        assert lists.disjoint(*[_span(lists, [x[a:b] for a, b in part]) for part in (read, w1, w2)]) == want


def test_what_is_no_list_of_spans(lists):
    for bad in ((1,), ((b"12345678", b"", 4),), ((b"12345678", b"12345678"),)):
        with pytest.raises((TypeError, ValueError)):
            lists.disjoint(*bad)
