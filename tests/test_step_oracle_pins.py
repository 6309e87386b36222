"""Pins of the fp64 statements of verification, the cache's table calls and the attention."""
import numpy as np

from oracle import step_oracle as S


def test_softmax_reads_odd_logits():
    p = S.softmax([0.0, np.nan, -np.inf, np.log(3.0)])
    assert np.allclose(p, [0.25, 0, 0, 0.75])
    assert np.allclose(S.softmax([1.0, np.inf, np.inf]), [0, 0.5, 0.5])
    assert not S.softmax([-np.inf, np.nan]).any()


def test_emitted_token_follows_the_target():
    # whatever the drafter's distribution, the first emitted token is distributed as p_0
    rng = np.random.default_rng(3)
    V, trials = 5, 4000
    target = rng.normal(size=(1, 2, V))
    draft = rng.normal(size=(1, V)) * 2
    p, q = S.softmax(target[0, 0]), S.softmax(draft[0])
    for given in (draft, None):
        seen = np.zeros(V)
        for _ in range(trials):
            # one-hot drafts are exact for any drafted token; a sampled one comes from q
            x = rng.choice(V, p=q)
            tok, count, _, _ = S.verify(target, given, np.array([[0, x]]), None, None,
                                        rng.random((1, 1)), rng.exponential(size=(1, V)))
            assert count[0] in (1, 2) and (tok[0, 0] == x) == (count[0] == 2)
            seen[tok[0, 0]] += 1
        # five standard deviations of a binomial share
        assert np.all(np.abs(seen / trials - p) < 5 * np.sqrt(p * (1 - p) / trials))


def test_verify_by_hand():
    # p = (1/2, 1/4, 1/4); the draft names id 1: accepted below u = 1/4
    t = np.log(np.array([[[2.0, 1, 1], [1, 1, 2]]]))
    e = np.array([[1.0, 9.0, 0.25]])
    tok, count, prob, _ = S.verify(t, None, np.array([[7, 1]]), None, None, np.array([[0.2]]), e)
    assert tok.tolist() == [[1, 2]] and count[0] == 2 and np.allclose(prob, 0.25)
    # rejected: residual (1/2, 0, 1/4) raced against e
    tok, count, _, _ = S.verify(t, None, np.array([[7, 1]]), None, None, np.array([[0.3]]), e)
    assert tok.tolist() == [[2, -1]] and count[0] == 1
    # greedy: the lowest of equal maxima
    tied = np.array([[[1.0, 3, 3], [0, 0, 0]]])
    tok, _, _, _ = S.verify(tied, None, np.array([[0, 1]]), None, np.zeros(1), np.zeros((1, 1)), e)
    assert tok.tolist() == [[1, 0]]
    tok, _, _, _ = S.verify(tied, None, np.array([[0, 2]]), None, np.zeros(1), np.zeros((1, 1)), e)
    assert tok.tolist() == [[1, -1]]


def test_pages_by_hand():
    table = np.array([[4, 1, -1], [2, -1, -1]], np.int32)
    refs = np.array([0, 1, 1, 0, 1, 0], np.int32)
    t, n, r = S.resize(table, np.array([7, 3]), np.array([2, 9]), refs, 4)
    assert t.tolist() == [[4, -1, -1], [2, 0, 1]] and n.tolist() == [2, 9]
    assert r.tolist() == [1, 1, 1, 0, 1, 0]
    c, n, r, moves = S.fork(table, np.array([7, 3]), [0, 1, 0], None, refs, 4)
    assert c.tolist() == [[4, 0, -1], [3, -1, -1], [4, 5, -1]] and n.tolist() == [7, 3, 7]
    assert r.tolist() == [1, 1, 1, 1, 3, 1] and moves == [(1, 0, 3), (2, 3, 3), (1, 5, 3)]
    t, r, new, live, moves = S.compact(table, np.array([7, 3]), refs, 4)
    assert t.tolist() == [[0, 1, -1], [2, -1, -1]] and live == 3 and moves == [(4, 0)]
    assert r.tolist() == [1, 1, 1, 0, 0, 0] and new.tolist() == [-1, 1, 2, -1, 0, -1]


def test_attention_by_hand():
    # two keys, equal scores: the mean of their values; the second token sees the tail too
    q = np.zeros((1, 2, 1, 2))
    kp, vp = np.ones((1, 1, 2)), np.array([[[2.0, 4.0]]])
    tail = (np.ones((1, 1, 2)), np.array([[[6.0, 0.0]]]))
    out, lse, _, _ = S.attention(q, kp, vp, [tail], 1.0)
    assert np.allclose(out[0, :, 0], [[2, 4], [4, 2]]) and np.allclose(lse[0, :, 0], [0, np.log(2)])
    out, lse, _, _ = S.attention(q, kp[:0], vp[:0], [tail], 1.0)
    assert np.allclose(out[0, :, 0], [[0, 0], [6, 0]]) and lse[0, 0, 0] == -np.inf


def test_temperatures_scale_differences():
    # the difference to the maximum is what is scaled: no clipping, however small the temperature
    p = S.softmax([20.0, 5.0, 20.0, -np.inf, 1e38], 1e-38)
    assert p.tolist() == [0, 0, 0, 0, 1]
    assert S.softmax([20.0, 5.0, 20.0], 1e-38).tolist() == [0.5, 0, 0.5]
    assert np.allclose(S.softmax([3e38, 3e38, -3e38], 10.0), [0.5, 0.5, 0])
    assert np.allclose(S.softmax([8.0, 8.0 - 1e-3 * np.log(3), -np.inf], 1e-3), [0.75, 0.25, 0])
    # the least temperature that is one
    t = np.array([[[5.0, 20.0, 20.0], [0, 0, 0]]])
    e = np.array([[1.0, 2.0, 1.0]])
    for heat, token in ((2e-38, 2), (1e-38, 1), (-1.0, 1), (np.nan, 1)):
        tok, count, prob, _ = S.verify(t, None, np.array([[0, 0]]), None, np.array([heat]),
                                       np.array([[0.0]]), e)
        assert tok.tolist() == [[token, -1]] and count[0] == 1 and prob[0, 0] == 0


def test_an_argmax_offered_with_its_logits_is_biased():
    # the condition of the law above: x has to be drawn from q.  q's argmax, which is certain, follows
    # the target when it is taken as one-hot and not when it is given with q
    rng = np.random.default_rng(4)
    V, trials = 4, 3000
    target, draft = np.log([[[0.4, 0.3, 0.2, 0.1], [1, 1, 1, 1]]]), np.log([[0.7, 0.1, 0.1, 0.1]])
    p = S.softmax(target[0, 0])
    off = []
    for given in (None, draft):
        seen = np.zeros(V)
        for _ in range(trials):
            tok, _, _, _ = S.verify(target, given, np.array([[0, 0]]), None, None, rng.random((1, 1)),
                                    rng.exponential(size=(1, V)))
            seen[tok[0, 0]] += 1
        off.append(np.abs(seen / trials - p) / np.sqrt(p * (1 - p) / trials))
    assert off[0].max() < 5 and off[1].max() > 15
