"""GPU tests of the verification of drafted tokens against the fp64 oracle.  The
outputs are whole numbers: equal.  Sums are in 64 bits on both sides; two orders
of adding V values differ by at most V 2^-53 of the sum, so a random number is
that near to a border between two tokens with a probability of about 1e-10 per
request in the random cases, and the cases on borders have exact sums.
"""
import numpy as np
import pytest
import torch

import oracle.drafts as od
from parity import need_gpu

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _bf():
    import bit_expert_ffn_top_amd as bf
    return bf


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(need_gpu())


def _check(p, q, draft, ua, us, n_draft=None, dtype=F32):
    bf = _bf()
    P = _dev(p, dtype)
    Q = None if q is None else _dev(q, dtype)
    D = _dev(draft, torch.int32)
    tokens, accepted = bf.verify_drafts(P, Q, D, _dev(ua, F32), _dev(us, F32),
                                        n_draft=None if n_draft is None else _dev(n_draft, torch.int32))
    want, count = od.verify(P.float().cpu().numpy(), None if Q is None else Q.float().cpu().numpy(), np.asarray(draft),
                            np.asarray(ua, np.float32), np.asarray(us, np.float32), n_draft)
    assert np.array_equal(accepted.cpu().numpy(), count)
    assert np.array_equal(tokens.cpu().numpy(), want)
    return want, count


def _random(B, n, V, seed=0, near=0.5):
    rng = np.random.default_rng(B * 1000 + n * 100 + V + seed)
    logits = 2 * rng.normal(size=(B, n + 1, V))
    p = np.exp(logits) / np.exp(logits).sum(-1, keepdims=True)
    lq = logits[:, :n] + near * rng.normal(size=(B, n, V))
    q = np.exp(lq) / np.exp(lq).sum(-1, keepdims=True)
    draft = np.array([[rng.choice(V, p=q[b, i]) for i in range(n)] for b in range(B)], np.int64).reshape(B, n)
    return p, q, draft, rng.random((B, n)), rng.random(B), rng


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("looked_up", [False, True])
@pytest.mark.parametrize("B,n,V", [(1, 0, 1), (1, 1, 1), (1, 3, 7), (3, 1, 2), (70, 2, 33), (5, 7, 1000), (2, 3, 4096),
                                   (9, 4, 4097), (3, 63, 257), (2, 3, 16384), (1, 5, 50001), (2, 2, 131073)])
def test_random(B, n, V, looked_up, dtype):
    p, q, draft, ua, us, rng = _random(B, n, V)
    _check(p, None if looked_up else q, draft, ua, us, dtype=dtype)
    ragged = rng.integers(-1, n + 2, B)
    _check(p, None if looked_up else q, draft, ua, us, ragged, dtype=dtype)


@pytest.mark.parametrize("B", [1, 17, 300, 3000])
def test_many_requests(B):
    p, q, draft, ua, us, rng = _random(B, 2, 37)
    _, count = _check(p, q, draft, ua, us, rng.integers(0, 3, B))
    if B > 100:
        assert set(count) == {0, 1, 2}


def test_every_border_of_a_uniform_row():
    """V a power of two and equal probabilities: sums are exact, and u = i / V
    lies on the border below token i."""
    V = 8192
    u = np.concatenate([np.arange(0, V, 61) / V, np.arange(1, V, 61) / V - 2.0 ** -24, [1 - 2.0 ** -24]])
    p = np.full((len(u), 1, V), 1.0 / V)
    want, _ = _check(p, None, np.zeros((len(u), 0)), np.zeros((len(u), 0)), u)
    assert want[0, 0] == 0 and want[1, 0] == 61 and want[-1, 0] == V - 1


def test_acceptance_on_the_border():
    """u q = p exactly is not accepted, one step of u below it is."""
    V = 4
    p, q = np.full((3, 2, V), 0.25), np.full((3, 1, V), 0.5)
    draft = np.ones((3, 1))
    ua = np.array([[0.5], [0.5 - 2.0 ** -25], [0.0]])
    _, count = _check(p, q, draft, ua, np.full(3, 0.3))
    assert count.tolist() == [0, 1, 1]
    # the product is exact where 32 bits would round it up to p
    u, qv = 1 - 2.0 ** -24, np.float32(1 / 3)
    p = np.full((1, 2, V), float(qv))
    _, count = _check(p, np.full((1, 1, V), float(qv)), np.ones((1, 1)), np.array([[u]]), np.array([0.1]))
    assert count.tolist() == [1]


def test_one_hot_rows_verify_a_greedy_choice():
    """p one at the target's choice: drafts that agree are accepted, the first
    that does not is replaced by that choice, whatever the random numbers."""
    rng = np.random.default_rng(3)
    B, n, V = 40, 4, 5003
    choice = rng.integers(0, V, (B, n + 1))
    p = np.zeros((B, n + 1, V))
    np.put_along_axis(p, choice[..., None], 1.0, -1)
    draft = np.where(rng.random((B, n)) < 0.7, choice[:, :n], rng.integers(0, V, (B, n)))
    q = np.full((B, n, V), 1.0 / V)
    ua, us = rng.random((B, n)), rng.random(B)
    for probs in (q, None):
        want, count = _check(p, probs, draft, ua, us)
        for b in range(B):
            j = 0
            while j < n and draft[b, j] == choice[b, j]:
                j += 1
            assert count[b] == j and want[b, :j + 1].tolist() == choice[b, :j + 1].tolist()


def test_nothing_left_of_p():
    """p = q with a draft that is refused (q of a token not drawn from it): the
    target's own row is drawn from; a row of zeros gives -1."""
    V = 300
    rng = np.random.default_rng(4)
    p = np.zeros((4, 2, V))
    p[:, :, :100] = rng.random((4, 2, 100))
    q = p[:, :1].copy()
    p[1, 0] = 0.0
    p[2, 1] = 0.0
    q[3] = 0.0
    draft = np.array([[200], [200], [5], [200]])
    ua = np.array([[0.5], [0.5], [0.0], [0.9]])
    want, count = _check(p, q, draft, ua, np.array([0.3, 0.3, 0.3, 0.999]))
    assert count.tolist() == [0, 0, 1, 0]
    assert want[1].tolist() == [-1, -1] and want[2].tolist() == [5, -1]
    want, _ = _check(p, None, draft, ua, np.array([0.0, 0.3, 0.3, 0.999]))
    assert want[0, 0] == 0
    # the looked-up draft is all that p holds, and refused
    only = np.zeros((1, 2, V))
    only[0, :, 7] = 0.5
    want, count = _check(only, None, np.array([[7]]), np.array([[0.75]]), np.array([0.5]))
    assert count.tolist() == [0] and want[0].tolist() == [7, -1]


def test_drafts_and_counts_out_of_range():
    p, q, draft, ua, us, _ = _random(6, 3, 50)
    draft[0, 0], draft[1, 1], draft[2, 2], draft[3, 0] = -1, 50, 2 ** 31 - 1, -2 ** 31
    ua[:] = 0.0
    for probs in (q, None):
        _, count = _check(p, probs, draft, ua, us)
        assert count.tolist() == [0, 1, 2, 0, 3, 3]
        _check(p, probs, draft, ua, us, np.array([2 ** 31 - 1, -2 ** 31, 99, 0, -1, 1]))


@pytest.mark.parametrize("u", [0.0, 1 - 2.0 ** -24, 1.0, -0.5, 2.0, float("nan"), float("inf")])
def test_ends_of_the_random_numbers(u):
    """Zeros at both ends of a row are never drawn, whatever u."""
    V = 9000
    p = np.zeros((2, 1, V))
    p[0, 0, 5000:5003] = [0.25, 0.5, 0.25]
    p[1, 0, [17, 8191]] = 0.5
    want, _ = _check(p, None, np.zeros((2, 0)), np.zeros((2, 0)), np.full(2, u))
    assert want[0, 0] in (5000, 5001, 5002) and want[1, 0] in (17, 8191)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), -1.0])
def test_values_that_are_no_probabilities(bad):
    """Where r is formed they count as 0; in front of the sampled token too."""
    p, q, draft, ua, us, rng = _random(40, 2, 400)
    for arr in (p, q):
        at = rng.random(arr.shape) < 0.05
        arr[at] = bad
    for probs in (q, None):
        _check(p, probs, draft, ua, us)


def test_the_result_is_distributed_as_the_target():
    """First tokens of 65,536 requests over one p and a different q: the share of
    every token is p's within 5 standard deviations."""
    bf = _bf()
    dev = need_gpu()
    B, V = 65536, 8
    p = torch.tensor([0.3, 0.05, 0.2, 0.0, 0.25, 0.1, 0.06, 0.04], device=dev)
    q = torch.tensor([0.1, 0.15, 0.05, 0.2, 0.3, 0.1, 0.05, 0.05], device=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    draft = torch.multinomial(q, B, True, generator=g).int()[:, None].contiguous()
    tokens, _ = bf.verify_drafts(p.expand(B, 2, V).contiguous(), q.expand(B, 1, V).contiguous(), draft,
                                 torch.rand((B, 1), generator=g, device=dev),
                                 torch.rand((B,), generator=g, device=dev))
    share = torch.bincount(tokens[:, 0].long(), minlength=V).double().cpu() / B
    pc = p.double().cpu()
    assert ((share - pc).abs() <= 5 * (pc * (1 - pc) / B).sqrt()).all()


def test_far_rows():
    """Rows whose byte offsets pass 2^32."""
    bf = _bf()
    dev = need_gpu()
    B, n, V = 70, 3, 4_000_001
    p = torch.zeros((B, n + 1, V), device=dev)
    q = torch.zeros((B, n, V), device=dev)
    assert B * n * V * 4 > 2 ** 31 and p.numel() * 4 > 2 ** 32
    draft = torch.full((B, n), V - 1, dtype=torch.int32, device=dev)
    p[-1, :, V - 1], q[-1, :, V - 1] = 0.5, 0.5
    p[-1, 2, V - 1], p[-1, 2, V - 3], p[-1, 2, 12] = 0.1, 0.4, 0.4
    ua = torch.full((B, n), 0.5, device=dev)
    us = torch.full((B,), 0.75, device=dev)
    tokens, accepted = bf.verify_drafts(p, q, draft, ua, us)
    assert accepted[-1].item() == 2 and tokens[-1].tolist() == [V - 1, V - 1, V - 3, -1]
    assert (accepted[:-1] == 0).all() and (tokens[:-1] == -1).all()
