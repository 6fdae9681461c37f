"""Verification over one workspace that nobody clears: replays of a graph, whose call number is always the
same, calls of other sizes and eager calls between them; and vocabularies of more chunks than a workgroup
has threads. The same tokens as the 64-bit definition, each time from new inputs."""
import numpy as np
import pytest

import step_reference as ref
import test_gpu_verify as base
from test_gpu_verify import env  # noqa: F401

pytestmark = pytest.mark.gpu


class Call:
    """Device inputs and outputs of one size; the inputs can be replaced in place."""

    def __init__(self, env, B, K, V, work, certain=False):
        self.pn, self.torch, self.dev = env
        torch, dev = self.torch, self.dev
        self.size, self.work, self.certain = (B, K, V), work, certain
        self.p, self.q = torch.zeros(B, K + 1, V, device=dev), None if certain else torch.zeros(B, K, V, device=dev)
        self.draft = torch.zeros(B, K, dtype=torch.int32, device=dev)
        self.ua, self.us = torch.zeros(B, K, device=dev), torch.zeros(B, device=dev)
        self.tokens = torch.zeros(B, K + 1, dtype=torch.int32, device=dev)
        self.accepted = torch.zeros(B, dtype=torch.int32, device=dev)

    def fill(self, seed, near=0.5):
        """New inputs, outputs that nothing gives."""
        torch = self.torch
        p, q, draft, ua, us = base.inputs(torch, self.dev, seed, *self.size, torch.float32, self.certain, near)
        self.p.copy_(p)
        if q is not None:
            self.q.copy_(q)
        for d, h in ((self.draft, draft), (self.ua, ua), (self.us, us)):
            d.copy_(torch.from_numpy(h))
        self.tokens.fill_(-7)
        self.accepted.fill_(-7)
        self.want = ref.verify(p.cpu().numpy(), None if q is None else q.cpu().numpy(), draft, ua, us)

    def run(self, stream=None):
        self.pn.verify(self.p, self.q, self.draft, self.ua, self.us, self.tokens, self.accepted, self.work,
                       stream=stream)

    def check(self, what):
        self.torch.cuda.synchronize()
        assert np.array_equal(self.accepted.cpu().numpy(), self.want[1]), what
        assert np.array_equal(self.tokens.cpu().numpy(), self.want[0]), what


def workspace(env, sizes):
    pn, torch, dev = env
    need = max(pn.verify_workspace_bytes(B, V) for B, _, V in sizes)
    return torch.full((need,), 0xA5, dtype=torch.uint8, device=dev)


def captured(env, call):
    torch = env[1]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call.run(stream=s)
    return g


@pytest.mark.parametrize("certain", [False, True])
def test_replays_over_what_the_last_one_left(env, certain):
    """The word that counts arrivals is as the replay before left it."""
    size = (4, 3, 9001)
    work = workspace(env, [size])
    c = Call(env, *size, work, certain)
    c.fill(1)
    c.run()
    c.check("eager")
    g = captured(env, c)
    for rep in range(6):
        c.fill(2 + rep, near=(0.05, 1.5)[rep % 2])
        env[1].cuda.synchronize()
        g.replay()
        c.check(f"replay {rep}")


def test_other_calls_between_replays(env):
    """Eager calls of the same and of other sizes, and a second graph, over the graph's own workspace."""
    sizes = [(4, 3, 9001), (1, 2, 60000), (17, 1, 4096), (3, 0, 2049)]
    work = workspace(env, sizes)
    calls = [Call(env, *size, work) for size in sizes]
    for c in calls:
        c.fill(5)
    g, h = captured(env, calls[0]), captured(env, calls[1])
    for rep in range(4):
        for n, step in enumerate((g.replay, calls[0].run, g.replay, h.replay, calls[2].run, g.replay, h.replay,
                                  calls[3].run)):
            c = calls[(0, 0, 0, 1, 2, 0, 1, 3)[n]]
            c.fill(10 * rep + n)
            env[1].cuda.synchronize()
            step()
            c.check((rep, n))


def test_sizes_in_turn_over_one_workspace(env):
    """Sums of one call lie where the next one counts its arrivals."""
    sizes = [(1, 1, 248320), (32, 1, 2049), (7, 3, 3000), (1, 0, 1), (32, 2, 2048), (2, 2, 100000), (9, 1, 20000)]
    work = workspace(env, sizes)
    calls = [Call(env, *size, work) for size in sizes]
    for rep in range(2):
        for n, c in enumerate(calls):
            c.fill(100 + 10 * rep + n)
            c.run()
            c.check((rep, n))


@pytest.mark.parametrize("V", [524288, 524289, 700001])
def test_more_chunks_than_threads(env, V):
    """More than 256 chunks: a thread has several, in the search for the chunk too. Draws all over the row,
    into its first and its last token."""
    size = (3, 1, V)
    c = Call(env, *size, workspace(env, [size]))
    torch = env[1]
    for rep, us in enumerate(([0.0, 0.3, 0.6], [0.9, 0.99, float(np.nextafter(np.float32(1), np.float32(0)))])):
        c.fill(200 + rep)
        c.us.copy_(torch.tensor(us))
        p, q, draft, ua = (x.cpu().numpy() for x in (c.p, c.q, c.draft, c.ua))
        c.want = ref.verify(p, q, draft, ua, np.array(us, np.float32))
        c.run()
        c.check(rep)
