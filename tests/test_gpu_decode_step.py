"""The example's decode step on the GPU against the same step on the host: its products from decoded
weights, its cache and attention from the 64-bit reference; and the step's place in the cache."""
import os
import sys

import numpy as np
import pytest

import oracle
import step_reference as ref

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("format", [ref.MXFP8, ref.MXFP4])
def test_steps_against_the_host(format):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decode_step as ex
    import block_quantized_weight_pn3t_amd as pn
    B, K, steps, prompt = 3, 2, 3, 45
    layer = ex.Layer(B, K + 1, format, prompt, steps, seed=5)
    tokens = torch.randint(0, ex.VOCAB, (prompt,), generator=layer.gen, device=layer.dev)
    layer.fill_prompt(tokens)

    def rows(w):
        type_, W, n = w
        k = {pn.PN3T: 80, pn.PN4T: 64}[type_] * (W.shape[1] // 34)
        return oracle.dequantize_rows(type_, W.cpu().numpy(), k).astype(np.float64)
    wq, wk, wv, wo = (rows(w) for w in (layer.wq, layer.wk, layer.wv, layer.wo))
    embed = layer.embed.cpu().numpy().astype(np.float64)
    head = oracle.fp8row_dequantize_rows(layer.head.cpu().numpy(), layer.head_scale.view(torch.int16).cpu().numpy()
                                         .view(np.uint16), ex.VOCAB, ex.HIDDEN).astype(np.float64)
    last = torch.tensor([1, 2, 3], dtype=torch.int32, device=layer.dev)
    for n in range(steps):
        guess = torch.randn(B, K, ex.VOCAB, generator=layer.gen, device=layer.dev).softmax(-1)
        draft = torch.multinomial(guess.view(B * K, -1), 1, generator=layer.gen).view(B, K).int()
        own = layer.own.cpu().numpy()
        step = torch.cat([last[:, None], draft], 1).long()
        got = layer.logits(step).cpu().double().numpy()
        # the host's step over the bytes that the device's cache holds now: a key's code may sit next
        # to a border that fp32 products and exact ones fall on either side of
        host = ref.Cache(format, ex.HEADS, ex.DIM, ex.PAGE, layer.cache.pages)
        host.data[:] = layer.cache.data.cpu().numpy()
        x = embed[step.cpu().numpy()]
        q = (x @ wq.T).reshape(B, K + 1, ex.HEADS * ex.GROUP, ex.DIM)
        out, _, mix, size, count = ref.attend(host, q, layer.table.cpu().numpy(), own + K + 1,
                                              layer.prefix_table.cpu().numpy(), prompt, ex.DIM ** -0.5)
        want = (x + out.reshape(B, K + 1, -1) @ wo.T) @ head.T
        # what the new tokens left in the cache is within one step of the type of their exact k and v
        rk, rv = host.read([s for b in range(B) for s in ref.slots_of(layer.table[b].cpu().numpy(), int(own[b]) + K + 1,
                                                                     ex.PAGE)[int(own[b]):]])
        for r, w in ((rk, wk), (rv, wv)):
            exact = (x @ w.T).reshape(B * (K + 1), ex.HEADS, ex.DIM)
            top = np.abs(exact).reshape(*exact.shape[:2], -1, 32).max(-1).repeat(32, -1)
            assert np.all(np.abs(r - exact) <= top * (2.0 ** -3 if format == ref.MXFP8 else 2.0 ** -1))
        # every product is within 1e-5 of its sum |w x|, and takes the error of its input on. In the
        # attention an error in q moves each score by at most scale * sum |dq k|, beside 2^-16 of
        # sum |scale q k| from q's two parts and under 2^-15 from sums and exponentials; scores and
        # the weights' two parts (2^-16) count twice against sum w |v| / sum w
        dq = 1e-5 * (np.abs(x) @ np.abs(wq).T).reshape(q.shape)
        _, _, _, moved, _ = ref.attend(host, dq, layer.table.cpu().numpy(), own + K + 1,
                                       layer.prefix_table.cpu().numpy(), prompt, ex.DIM ** -0.5)
        dout = (2 * ((moved + 2.0 ** -15 * (1 + size)) + 2.0 ** -16))[..., None] * mix
        flat, aw = out.reshape(B, K + 1, -1), np.abs(wo).T
        dx = dout.reshape(flat.shape) @ aw + 1e-5 * (np.abs(flat) @ aw) + 2.0 ** -24 * np.abs(x + flat @ wo.T)
        tol = dx @ np.abs(head).T + 1e-5 * (np.abs(x + flat @ wo.T) + dx) @ np.abs(head).T
        assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
        tokens, accepted = layer.step(last, draft, guess)
        a = accepted.cpu().numpy()
        assert np.array_equal(layer.own.cpu().numpy(), own + 1 + a)
        t = tokens.cpu().numpy()
        for b in range(B):
            assert np.array_equal(t[b, :a[b]], draft[b, :a[b]].cpu().numpy())
            assert 0 <= t[b, a[b]] < ex.VOCAB and (t[b, a[b] + 1:] == -1).all()
        last = tokens.gather(1, accepted[:, None].long())[:, 0]


def test_the_example_runs(capsys, monkeypatch):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decode_step as ex
    monkeypatch.setattr(sys, "argv", ["decode_step.py", "--steps", "2", "--format", "mxfp4"])
    ex.main()
    assert capsys.readouterr().out.count("step ") == 2
