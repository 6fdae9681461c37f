"""Pins of the references of a prompt's operators by hand, and the refusals of the C entry points and of the
binding, which are decided before anything runs."""
import ctypes as C

import numpy as np
import pytest
import torch  # first: the library takes its HIP runtime

import block_quantized_weight_pn3t_amd as pn
import prompt_reference as ref

P = C.c_void_p
fake = P(0x1000)
L = pn.lib()


def test_int8_rows_by_hand():
    codes, scales = ref.int8_rows([[0.0, 254.0, -254.0, 3.0, 1.0, 5.0, -1.0], [0.0] * 7,
                                   [1.0, np.nan, 0, 0, 0, 0, 0], [1.0, -np.inf, 0, 0, 0, 0, 0]])
    # ties at 1.5, 0.5 and 2.5 go to the even code
    assert codes[0].tolist() == [0, 127, -127, 2, 0, 2, 0]
    assert scales[0] == 2.0 and scales[1] == 0.0 and np.isnan(scales[2:]).all()
    assert not codes[1:].any()


def test_norm_by_hand():
    y, t, r = ref.norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(y, [[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]], rtol=1e-15)
    assert t.tolist() == [[3.0, 8.0]]


def test_turn_by_hand():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    quarter = np.array([[0, 0, 1, 1]], np.float32)  # by a right angle
    assert ref.turn(x, quarter, False)[0, 0].tolist() == [-3, -4, 1, 2, 5, 6, 7, 8]
    assert ref.turn(x, quarter, True)[0, 0].tolist() == [-2, 1, -4, 3, 5, 6, 7, 8]


def test_logprobs_by_hand():
    x = np.log(np.array([[1.0, 4.0, 2.0, 4.0, 5.0]]))
    got = ref.logprobs(x, [2], 1.0, 3)
    p = np.array([1, 4, 2, 4, 5]) / 16
    assert np.isclose(got["logprob"][0], np.log(2 / 16)) and got["rank"][0] == 3
    assert np.isclose(got["entropy"][0], -(p * np.log(p)).sum()) and np.isclose(got["lse"][0], np.log(16))
    assert got["top_ids"][0].tolist() == [4, 1, 3]
    # equal logits with different signs of zero: the lowest number first
    assert ref.logprobs(np.array([[-0.0, 0.0, -1.0]]), [5], 1.0, 2)["top_ids"][0].tolist() == [0, 1]


def add_norm(**kw):
    a = dict(type=0, weight_type=0, rows=2, K=64, x=0x1000, x_stride=64, residual=0, residual_stride=0, sum=0,
             sum_stride=0, weight=0x1000, eps=1e-6, out=0x2000, out_stride=64, codes=0, scales=0)
    a.update(kw)
    return L.pn_add_norm(C.byref(pn.AddNormArgs(**a)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=3), -9), (dict(weight_type=-1), -9), (dict(K=0), -2), (dict(K=65537), -2), (dict(rows=-1), -2),
    (dict(rows=1 << 31), -2), (dict(eps=-1e-9), -2), (dict(eps=float("nan")), -2), (dict(eps=float("inf")), -2),
    (dict(x=0), -4), (dict(weight=0), -4), (dict(out=0), -4), (dict(codes=0x1000), -4), (dict(scales=0x1000), -4),
    (dict(x=0x1002), -5), (dict(type=1, x=0x1001), -5), (dict(residual=0x1001), -5), (dict(sum=0x1002), -5),
    (dict(weight=0x1002), -5), (dict(out=0x1001), -5), (dict(codes=0x1000, scales=0x1002), -5), (dict(rows=0), 0)])
def test_add_norm_refusals(kw, status):
    assert add_norm(**kw) == status


def test_quantize_rows_refusals():
    f = L.pn_int8_quantize_rows
    assert f(9, fake, 64, 2, 64, fake, fake, None) == -9
    assert f(0, fake, 64, -1, 64, fake, fake, None) == -2
    assert f(0, fake, 64, 2, 0, fake, fake, None) == -2
    assert f(0, fake, 64, 2, 65537, fake, fake, None) == -2
    assert f(0, None, 64, 2, 64, fake, fake, None) == -4
    assert f(0, fake, 64, 2, 64, None, fake, None) == -4
    assert f(0, fake, 64, 2, 64, fake, None, None) == -4
    assert f(0, P(0x1002), 64, 2, 64, fake, fake, None) == -5
    assert f(2, P(0x1001), 64, 2, 64, fake, fake, None) == -5
    assert f(0, fake, 64, 2, 64, fake, P(0x1002), None) == -5
    assert f(0, None, 64, 0, 64, None, None, None) == 0
    assert L.pn_add_norm(None, None) == -4


def gemm(a=fake, sa=fake, M=4, w=fake, sw=fake, N=8, K=64, type=0, out=fake, stride=8, work=fake, bytes=1 << 40):
    return L.pn_gemm_int8(a, sa, M, w, sw, N, K, type, out, stride, work, bytes, None)


def test_gemm_int8_refusals():
    assert gemm(type=3) == -9
    for kw in (dict(M=-1), dict(N=-1), dict(K=0), dict(K=24), dict(K=-16), dict(K=131072), dict(M=1 << 40),
               dict(N=1 << 40)):
        assert gemm(**kw) == -2, kw
        assert L.pn_gemm_int8_workspace_bytes(kw.get("M", 4), kw.get("N", 8), kw.get("K", 64)) == 0
    for name in ("a", "sa", "w", "sw", "out"):
        assert gemm(**{name: None}) == -4, name
        assert gemm(**{name: P(0x1002) if name != "out" else P(0x1001)}) == -5, name
    assert gemm(a=P(0x1008)) == -5
    assert gemm(type=1, out=P(0x1001)) == -5
    assert gemm(M=0, a=None) == 0 and gemm(N=0, w=None) == 0


def cache_desc(**kw):
    c = dict(format=0, heads=2, dim=128, page=64, pages=2, data=0x1000)
    c.update(kw)
    return C.byref(pn.CacheDesc(**c))


def append(cache=None, **kw):
    a = dict(type=0, Hq=4, q=0x1000, q_token_stride=512, q_head_stride=128, q_out=0x2000, q_out_token_stride=512,
             q_out_head_stride=128, k=0x1000, k_token_stride=256, k_head_stride=128, v=0x1000, v_token_stride=256,
             v_head_stride=128, rotation=0x1000, rows=10, rot=128, interleaved=0, positions=0x1000, slots=0x1000, T=3)
    a.update(kw)
    return L.pn_cache_append(cache or cache_desc(), C.byref(pn.AppendArgs(**a)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=3), -9), (dict(T=-1), -2), (dict(rows=0), -2), (dict(rot=0), -2), (dict(rot=12), -2),
    (dict(rot=136), -2), (dict(interleaved=2), -2), (dict(Hq=0), -2), (dict(positions=0, rows=2), -2),
    (dict(T=1 << 41), -2), (dict(k=0), -4), (dict(v=0), -4), (dict(slots=0), -4), (dict(rotation=0), -4),
    (dict(q_out=0), -4), (dict(k=0x1002), -5), (dict(v=0x1001), -5), (dict(q=0x1002), -5), (dict(q_out=0x1002), -5),
    (dict(slots=0x1004), -5), (dict(positions=0x1004), -5), (dict(rotation=0x1008), -5), (dict(T=0), 0),
    (dict(T=0, k=0, v=0, slots=0), 0)])
def test_append_refusals(kw, status):
    assert append(**kw) == status


def test_append_cache_refusals():
    assert append(cache_desc(format=2)) == -9
    assert append(cache_desc(dim=96)) == -2
    assert append(cache_desc(data=0x1008)) == -5
    assert append(cache_desc(data=0)) == -4
    assert L.pn_cache_append(None, None, None) == -4 and L.pn_cache_append(cache_desc(), None, None) == -4


def logp(work=fake, bytes=1 << 40, **kw):
    a = dict(type=0, top=2, R=3, V=5000, stride=5000, logits=0x1000, tokens=0x1000, scale=1.0, logprob=0x1000,
             rank=0x1000, entropy=0x1000, lse=0x1000, top_ids=0x1000, top_logprobs=0x1000)
    a.update(kw)
    return L.pn_logprobs(C.byref(pn.LogprobsArgs(**a)), work, bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=-1), -9), (dict(R=-1), -2), (dict(V=0), -2), (dict(V=1 << 30), -2), (dict(top=-1), -2),
    (dict(top=65), -2), (dict(R=1 << 31), -2), (dict(scale=0.0), -2), (dict(scale=-1.0), -2),
    (dict(scale=float("nan")), -2), (dict(scale=float("inf")), -2), (dict(logits=0), -4), (dict(tokens=0), -4),
    (dict(top_ids=0), -4), (dict(top_logprobs=0), -4), (dict(logits=0x1002), -5), (dict(type=1, logits=0x1001), -5),
    (dict(tokens=0x1002), -5), (dict(logprob=0x1002), -5), (dict(rank=0x1002), -5), (dict(entropy=0x1002), -5),
    (dict(lse=0x1002), -5), (dict(top_ids=0x1002), -5), (dict(top_logprobs=0x1002), -5), (dict(work=None), -4),
    (dict(work=P(0x1008)), -5), (dict(bytes=16), -10), (dict(R=0), 0)])
def test_logprobs_refusals(kw, status):
    assert logp(**kw) == status


def test_logprobs_workspace_is_enough_for_less():
    for V in (1, 2048, 9000, 248320):
        for top in (0, 20):
            need = [pn.logprobs_workspace_bytes(R, V, top) for R in range(1, 1100)]
            assert need == sorted(need)
    for R in (1, 3, 255, 256, 511, 600):
        need = [pn.logprobs_workspace_bytes(R, V, 20) for V in range(1, 300000, 997)]
        assert need == sorted(need)


def test_logprobs_workspace():
    assert L.pn_logprobs(None, fake, 0, None) == -4
    for R, V, top in ((-1, 10, 0), (1, 0, 0), (1, 1 << 30, 0), (1, 10, 65), (1, 10, -1), (0, 10, 0)):
        assert pn.logprobs_workspace_bytes(R, V, top) == 0
    assert pn.logprobs_workspace_bytes(1, 248320, 20) > 0


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(4, 64)
    i8, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError):
        pn.add_norm(x, torch.ones(64), 1e-6, out=x)
    with pytest.raises(ValueError):
        pn.int8_quantize_rows(x, i8, s)
    with pytest.raises(ValueError):
        pn.gemm_int8(i8, s, i8, s, x)
    with pytest.raises(ValueError):
        pn.logprobs(x, entropy=s)
    assert pn.gemm_int8_workspace_bytes(4, 8, 20) == 0
