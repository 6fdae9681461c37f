"""A prompt's operators together: every call that the example makes, with its own views and strides, against the
64-bit definitions on the numbers that the call was given; and a decode step of them captured into a graph."""
import os
import sys

import numpy as np
import pytest

import prompt_reference as ref
import step_reference as step
import test_gpu_logprobs

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    return pn, torch, torch.device("cuda:0")


def f64(t):
    return t.double().cpu().numpy()


class Checked:
    """The library's calls, each checked after it is made; the names of those that were."""

    def __init__(self, pn, torch):
        self.pn, self.torch, self.calls = pn, torch, []

    def __getattr__(self, name):
        real = getattr(self.pn, name)
        check = getattr(type(self), "check_" + name, None)
        if check is None:
            return real

        def call(*args, **kw):
            self.calls.append(name)
            check(self, real, *args, **kw)
        return call

    @staticmethod
    def near(got, want, halves):
        """Within `halves` roundings to fp32 of the numbers."""
        assert (np.abs(got - want) <= halves * 2.0 ** -24 * np.abs(want) * (1 + 1e-6)).all()

    def check_int8_quantize_rows(self, real, x, codes, scales):
        real(x, codes, scales)
        want, want_scales = ref.int8_rows(f64(x))
        assert (codes.cpu().numpy() == want).all()
        self.near(f64(scales), want_scales, 1)

    def check_add_norm(self, real, x, weight, eps, codes, scales, residual, sum):
        real(x, weight, eps, codes=codes, scales=scales, residual=residual, sum=sum)
        h = x if residual is None else x + residual
        if residual is not None:
            assert self.torch.equal(sum, h)
        _, t, r = ref.norm(f64(h), f64(weight), eps)
        want, want_scales = ref.int8_rows(t, r)
        assert (codes.cpu().numpy() == want).all()
        self.near(f64(scales), want_scales, 1)

    def check_gemm_int8(self, real, a, a_scales, w, w_scales, out, work):
        real(a, a_scales, w, w_scales, out, work)
        sums = a.cpu().numpy().astype(np.float64) @ w.cpu().numpy().astype(np.float64).T
        self.near(f64(out), sums * f64(a_scales)[:, None] * f64(w_scales), 3)

    def check_cache_append(self, real, cache, k, v, slots, rotation, positions, q, q_out):
        host = step.Cache(cache.format, cache.heads, cache.dim, cache.page, cache.pages)
        host.data[:] = cache.data.cpu().numpy()
        row = rotation.cpu().numpy()[positions.cpu().numpy()]
        host.write(ref.turn(f64(k), row, False).astype(np.float64), f64(v), slots.cpu().numpy())
        turned = ref.turn(f64(q), row, False)
        kept = k.clone()
        real(cache, k, v, slots, rotation, positions=positions, q=q, q_out=q_out)
        assert (cache.data.cpu().numpy() == host.data).all()
        assert (q_out.cpu().numpy() == turned).all() and self.torch.equal(k, kept)

    def check_attend(self, real, cache, q, table, lens, out, workspace):
        real(cache, q, table, lens, out, workspace=workspace)
        host = step.Cache(cache.format, cache.heads, cache.dim, cache.page, cache.pages)
        host.data[:] = cache.data.cpu().numpy()
        want, _, mix, size, count = step.attend(host, f64(q), table.cpu().numpy(), lens.cpu().numpy(),
                                                np.zeros(0, np.int64), 0, cache.dim ** -0.5)
        # a score is a sum of dim + 2 roundings of its parts (three of q), its exponential and the sums over
        # the tokens take as many again as there are tokens
        room = (2 * cache.dim + 8) * size + 4 * count[:, :, None] + 64
        assert (np.abs(f64(out) - want) <= 2.0 ** -24 * room[..., None] * mix + 1e-30).all()

    def check_logprobs(self, real, logits, tokens, workspace, **got):
        lse = self.torch.empty(logits.shape[0], device=logits.device)
        real(logits, tokens, workspace=workspace, lse=lse, **got)
        test_gpu_logprobs.same(dict(got, lse=lse), f64(logits), tokens.cpu().numpy(), 1.0, got["top_ids"].shape[1])


@pytest.mark.parametrize("format", [step.MXFP8, step.MXFP4])
def test_every_call_of_the_example(env, format, monkeypatch):
    pn, torch, dev = env
    import score_prompt as ex
    checked = Checked(pn, torch)
    monkeypatch.setattr(ex, "pn", checked)
    layer = ex.Layer(60, format, seed=3)
    prompt = torch.randint(0, ex.VOCAB, (45,), generator=layer.gen, device=dev)
    got = layer.score(prompt, 5)
    assert got["rank"][-1] == -1 and got["logprob"][-1] == 0
    for n in range(3):  # and single tokens after it
        layer.score(got["top_ids"][-1:, 0].long(), 5)
    assert layer.length == 48
    assert {name: checked.calls.count(name) for name in set(checked.calls)} == {
        "int8_quantize_rows": 3 + 4, "add_norm": 8, "gemm_int8": 12, "cache_append": 4, "attend": 4, "logprobs": 4}


def test_a_step_in_a_graph(env):
    """One token's calls over buffers that stay, captured; each replay against eager calls on the same inputs."""
    pn, torch, dev = env
    g = torch.Generator(device=dev)
    g.manual_seed(9)
    K, H, G, D, V, page, T = 512, 2, 3, 64, 9001, 32, 4
    x, res = torch.empty(T, K, device=dev), torch.randn(T, K, generator=g, device=dev)
    norm = torch.rand(K, generator=g, device=dev) + 0.5
    table = torch.from_numpy(ref.table(500, D)).to(dev)

    def weights(rows, width):
        codes, scales = torch.empty(rows, width, dtype=torch.int8, device=dev), torch.empty(rows, device=dev)
        pn.int8_quantize_rows(torch.randn(rows, width, generator=g, device=dev) / width ** 0.5, codes, scales)
        return codes, scales
    wqkv, wo, head = weights(H * (G + 2) * D, K), weights(K, H * G * D), weights(V, K)
    place = torch.arange(T, device=dev)
    lens = torch.full((1,), T, dtype=torch.int32, device=dev)
    pages = torch.arange(4, dtype=torch.int32, device=dev)[None]
    tokens = torch.zeros(T, dtype=torch.int32, device=dev)
    works = [torch.randint(0, 256, (n + 16,), dtype=torch.uint8, device=dev) for n in (
        pn.gemm_int8_workspace_bytes(T, H * (G + 2) * D, K), pn.gemm_int8_workspace_bytes(T, K, H * G * D),
        pn.gemm_int8_workspace_bytes(T, V, K), pn.logprobs_workspace_bytes(T, V, 4))]

    def buffers():
        e = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=dev)  # noqa: E731
        return dict(sum=e(T, K), codes=e(T, K, dt=torch.int8), scales=e(T), qkv=e(T, H * (G + 2) * D), out=e(1, T, H * G, D),
                    ocodes=e(T, H * G * D, dt=torch.int8), oscales=e(T), o=e(T, K), logits=e(T, V), logprob=e(T), entropy=e(T),
                    ids=e(T, 4, dt=torch.int32), top=e(T, 4),
                    data=torch.zeros(4 * pn.cache_page_bytes(step.MXFP8, H, D, page), dtype=torch.uint8, device=dev))

    def run(b):
        pn.add_norm(x, norm, 1e-6, codes=b["codes"], scales=b["scales"], residual=res, sum=b["sum"])
        pn.gemm_int8(b["codes"], b["scales"], *wqkv, b["qkv"], works[0])
        q, k, v = b["qkv"].view(T, -1, D).split([H * G, H, H], 1)
        cache = pn.Cache(step.MXFP8, H, D, page, b["data"])
        pn.cache_append(cache, k, v, place, table, positions=place, q=q, q_out=q)
        pn.attend(cache, q[None], pages, lens, b["out"],
                  workspace=torch.empty(pn.attend_workspace_bytes(cache, q[None], pages), dtype=torch.uint8, device=dev))
        pn.int8_quantize_rows(b["out"].view(T, -1), b["ocodes"], b["oscales"])
        pn.gemm_int8(b["ocodes"], b["oscales"], *wo, b["o"], works[1])
        pn.add_norm(b["o"], norm, 1e-6, codes=b["codes"], scales=b["scales"], residual=b["sum"], sum=b["sum"])
        pn.gemm_int8(b["codes"], b["scales"], *head, b["logits"], works[2])
        pn.logprobs(b["logits"], tokens, b["logprob"], works[3], entropy=b["entropy"], top_ids=b["ids"], top_logprobs=b["top"])
    b, again = buffers(), buffers()
    x.normal_(generator=g)
    run(b)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run(b)
    for n in range(4):
        x.normal_(generator=g)
        tokens += 13
        place += T
        lens += T
        graph.replay()
        torch.cuda.synchronize()
        again["data"].copy_(b["data"])
        run(again)
        torch.cuda.synchronize()
        for name in b:
            assert torch.equal(b[name], again[name]), name
