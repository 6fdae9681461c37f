"""What verification does with probabilities that are none: a draft whose p or q is negative or NaN is
refused, and a token whose p or q is has no part in the residual. The definition is written out here in
64 bits, with those rules of its own. The tokens have to be the same."""
import numpy as np
import pytest

import test_gpu_verify as base
from test_gpu_verify import env  # noqa: F401

gpu = pytest.mark.gpu


def defined(p, q, draft, u_accept, u_sample):
    """tokens, accepted of the definition; p [B][K + 1][V], q [B][K][V] or None."""
    B, K = draft.shape
    tokens, accepted = np.full((B, K + 1), -1, np.int32), np.zeros(B, np.int32)
    p, u_sample = p.astype(np.float64), u_sample.astype(np.float64)
    q = None if q is None else q.astype(np.float64)
    for b in range(B):
        a = 0
        for i in range(K):
            x = draft[b, i]
            px, qx = p[b, i, x], 1.0 if q is None else q[b, i, x]
            if not (px >= 0 and qx >= 0 and float(u_accept[b, i]) * qx < px):
                break
            tokens[b, a] = x
            a += 1
        positive = np.where(p[b, a] > 0, p[b, a], 0.0)
        r = positive
        if a < K:
            if q is None:
                r = positive.copy()
                r[draft[b, a]] = 0.0
            else:
                good = (p[b, a] >= 0) & (q[b, a] >= 0)
                r = np.where(good, np.maximum(np.where(good, p[b, a] - q[b, a], 0.0), 0.0), 0.0)
            if r.sum() <= 0:
                r = positive
        run = np.cumsum(r)
        accepted[b] = a
        if run[-1] > 0:
            past = np.nonzero((r > 0) & (run > u_sample[b] * run[-1]))[0]
            tokens[b, a] = past[0] if len(past) else np.nonzero(r)[0][-1]
    return tokens, accepted


def same(env, p, q, draft, ua, us):
    want = defined(p.float().cpu().numpy(), None if q is None else q.float().cpu().numpy(), draft, ua, us)
    got = base.run(env, p, q, draft, ua, us)
    assert np.array_equal(got[1], want[1]), (got[1], want[1])
    assert np.array_equal(got[0], want[0]), (got[0], want[0])
    return got


def test_the_definition_by_hand():
    """u = 0 and one draft of token 1, one thing wrong at a time."""
    u, s = np.zeros((1, 1)), np.full(1, 0.6)

    def one(p, q):
        t, a = defined(np.array([[p, [1.0, 0, 0]]]), np.array([[q]]), np.array([[1]]), u, s)
        return t[0].tolist(), int(a[0])
    assert one([0.5, 0.25, 0.25], [0.0, 0.5, 0.5]) == ([1, 0], 1)
    assert one([0.5, 0.25, 0.25], [0.0, -0.5, 0.125]) == ([0, -1], 0)   # r = 0.5, 0, 0.125: 0.375 is in the first
    assert one([0.25, 0.25, 0.5], [-0.5, -0.5, 0.25]) == ([2, -1], 0)   # r = 0, 0, 0.25
    assert one([-0.25, 0.0, 0.5], [-0.5, 0.5, 0.25]) == ([2, -1], 0)    # -0.25 is more than -0.5, and nothing
    assert one([0.25, np.nan, 0.5], [0.5, 0.5, np.nan]) == ([2, -1], 0)  # no residual: from p itself


@gpu
@pytest.mark.parametrize("bad", [-0.3, -1e-30, float("nan")])
@pytest.mark.parametrize("where", ["p", "q", "both"])
def test_a_draft_without_a_probability_is_refused(env, bad, where):
    """Also where u q < p holds: q negative under a p of zero or more, p negative over a q yet smaller."""
    pn, torch, dev = env
    for u in (0.0, 0.5):
        p, q, draft, ua, us = base.inputs(torch, dev, 21, 4, 3, 700, torch.float32, near=0.05)
        ua[:] = u
        for b in range(4):
            i, x = b % 3, int(draft[b, b % 3])
            if where != "q":
                p[b, i, x] = bad
            if where != "p":
                q[b, i, x] = 2 * bad
            elif b == 3:
                q[b, i, x] = 0.0
        if where == "q":
            p[0, 0, int(draft[0, 0])] = 0.0
        got = same(env, p, q, draft, ua, us)
        assert (got[1] <= np.arange(4) % 3).all()


@gpu
@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("V", [255, 2048, 6001, 6008])
def test_the_residual_leaves_out_what_is_no_probability(env, type_, V):
    """Whole ranges of negative and NaN numbers in p, in q and in both, in vector and in single loads; the
    first draft is refused, so that the residual is what is drawn from."""
    pn, torch, dev = env
    dt = getattr(torch, type_)
    rng = np.random.default_rng(V)
    for rep in range(6):
        p, q, draft, _, us = base.inputs(torch, dev, 30 + rep, 5, 2, V, dt, near=1.5)
        for t, scale in ((p, -1.0), (q, -3.0)):
            hit = torch.from_numpy(rng.random((5, t.shape[1], V))).to(dev)
            t[(hit < 0.3)] *= scale
            t[(hit > 0.9)] = float("nan")
        both = torch.from_numpy(rng.random((5, 2, V)) < 0.1).to(dev)
        p[:, :2][both] = -0.001
        q[both] = -0.002
        same(env, p, q, draft, np.ones((5, 2), np.float32), us)
        same(env, p, None, draft, np.ones((5, 2), np.float32), us)


@gpu
def test_a_residual_of_nothing_but_negative_q(env):
    """q negative where p is positive and larger than p elsewhere: no residual, the draw is from p."""
    pn, torch, dev = env
    p, q, draft, ua, us = base.inputs(torch, dev, 41, 3, 1, 5000, torch.float32)
    q[:, :, ::2] = -0.5
    q[:, :, 1::2] = 2.0
    same(env, p, q, draft, np.ones_like(ua), us)
