"""Limits of the prompt's entry points that are decided before anything runs: scales, sizes of launches, tensors that the
binding is given."""
import ctypes as C
import itertools

import pytest
import torch  # first: the library takes its HIP runtime

import block_quantized_weight_pn3t_amd as pn
from test_prompt_reference import append, cache_desc, gemm, logp


@pytest.mark.parametrize("V,scale,refused", [
    (1, 2.0 ** -121, False), (1, 2.0 ** -122, True), (5000, 1.881e-33, False), (5000, 1.880e-33, True), (5000, 1e-37, True),
    ((1 << 30) - 1, 4.1e-28, False), ((1 << 30) - 1, 4.0e-28, True)])
def test_logprobs_scales(V, scale, refused):
    """From V * 2^-121 on no sum of a row's differences passes fp32."""
    assert (logp(V=V, stride=V, scale=scale, logits=0x1000, R=1, tokens=0x1002) == -2) == refused


def test_logprobs_rows():
    assert logp(R=1 << 25, tokens=0x1002) == -2 and logp(R=(1 << 25) - 1, tokens=0x1002) == -5
    assert pn.logprobs_workspace_bytes(1 << 25, 5000, 2) == 0 < pn.logprobs_workspace_bytes((1 << 25) - 1, 5000, 2)


@pytest.mark.parametrize("M,N,refused", [
    (64 * ((1 << 25) - 1), 1, True), (256 * ((1 << 23) - 1), 1, False), (1, 256 * ((1 << 23) - 1), False),
    (64 << 12, 64 << 13, True), (64 << 12, 64 * ((1 << 13) - 1), False)])
def test_gemm_int8_tiles(M, N, refused):
    """Outputs of which one launch has tiles of 256 for all."""
    assert (gemm(M=M, N=N, K=16, a=C.c_void_p(0x1008)) == -2) == refused


def test_launches_of_the_cache():
    """2^24 workgroups of 256 threads are one too many for a launch. (The alignment is looked at after the sizes.)"""
    odd, fake = C.c_void_p(0x1001), C.c_void_p(0x1000)
    for T, heads, write, read in ((8192 - 32, 65536, False, True), (8192 - 31, 65536, True, True), (4096 - 16, 65536, False, False),
                                  (4096 - 15, 65536, False, True), (1 << 29, 1, True, True), ((1 << 29) - 32, 1, False, True)):
        c = cache_desc(heads=heads)
        assert (pn.lib().pn_cache_write(c, 0, odd, 0, 0, fake, 0, 0, fake, T, None) == -2) == write, (T, heads)
        assert (pn.lib().pn_cache_read(c, 0, fake, T, odd, fake, None) == -2) == read, (T, heads)
        assert (append(c, T=T, q=0, k=0x1001) == -2) == write, (T, heads)


def test_launches_of_the_queries():
    assert append(cache_desc(heads=1), T=1 << 20, Hq=1 << 16, positions=0x1000, rows=1) == -2


def test_launches_of_attention_and_verification():
    import test_step_reference as step
    fake = C.c_void_p(0x1000)

    def attend(B, **kw):
        a = step.attend_args(pn, B=B, Q=1, Hq=2, prefix_len=0, table_width=1, **kw)
        return pn.lib().pn_attend(C.byref(step.desc(pn, heads=2)), C.byref(a), None, 0, None)
    # two heads of eight waves a sequence; a missing workspace is looked at after the sizes
    assert attend(1 << 22) == -2
    for B, V, refused in ((1 << 20, 32768, True), ((1 << 20) - 1, 32768, False), (1 << 24, 100, True), ((1 << 24) - 1, 100, False)):
        st = pn.lib().pn_verify(0, fake, V, None, V, None, None, None, C.c_void_p(0x1002), B, 0, V, fake, fake, fake, 1 << 50, None)
        assert (st == -2) == refused, (B, V)


class Lib:
    """In the library's place: the names of the entry points that were called."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def on_host(monkeypatch):
    """The binding with host tensors as those of the current device; its calls go nowhere."""
    pn._names()
    monkeypatch.setattr(pn._Torch, "device", staticmethod(lambda: -1))
    monkeypatch.setattr(pn._Torch, "raw_stream", staticmethod(lambda device: 0))
    lib = Lib()
    monkeypatch.setattr(pn, "_lib", lib)
    return lib


def cache_on(device, heads=2, dim=64):
    c = pn.Cache.__new__(pn.Cache)
    c.format, c.heads, c.dim, c.page, c.pages, c.device, c.ref = pn.MXFP8, heads, dim, 32, 1, device, 0
    c.data = torch.zeros(1, dtype=torch.uint8)
    return c


def test_append_to_a_cache_of_another_device(on_host):
    k, slots, table = torch.zeros(3, 2, 64), torch.arange(3), torch.zeros(3, 64)
    pn.cache_append(cache_on(-1), k, k, slots, table)
    assert on_host.calls == ["pn_cache_append"]
    with pytest.raises(ValueError, match="cache"):
        pn.cache_append(cache_on(0), k, k, slots, table)
    assert on_host.calls == ["pn_cache_append"]


def test_overlaps_of_heads():
    """Against the numbers' own places, for every small shape and stride."""
    for n, heads, dim in itertools.product((0, 1, 2, 3, 4), (1, 2, 3), (1, 2, 4)):
        for token, head in itertools.product(range(14), range(14)):
            at = [t * token + h * head + d for t in range(n) for h in range(heads) for d in range(dim)]
            assert pn._overlap(n, heads, dim, token, head) == (len(set(at)) < len(at)), (n, heads, dim, token, head)


def test_append_to_queries_that_overlap(on_host):
    k, slots, table = torch.zeros(3, 2, 64), torch.arange(3), torch.zeros(3, 64)
    q = torch.zeros(3, 5, 64)
    wide = torch.zeros(4096)
    for q_out in (torch.zeros(3, 5, 64), torch.zeros(5, 3, 64).transpose(0, 1), torch.zeros(3, 9, 64)[:, 2:7], q,
                  wide.as_strided((3, 5, 64), (5 * 64 + 1, 64, 1)), wide.as_strided((3, 5, 64), (128, 384, 1))):
        pn.cache_append(cache_on(-1), k, k, slots, table, q=q, q_out=q_out)
    # read as they are, from one head or token too
    pn.cache_append(cache_on(-1), k, k, slots, table, q=q[:, :1].expand(3, 5, 64), q_out=q)
    made = len(on_host.calls)
    assert made == 7
    for q_out in (torch.zeros(3, 1, 64).expand(3, 5, 64), torch.zeros(1, 5, 64).expand(3, 5, 64),
                  wide.as_strided((3, 5, 64), (320, 63, 1)), wide.as_strided((3, 5, 64), (319, 64, 1)),
                  wide.as_strided((3, 5, 64), (128, 256, 1))):
        with pytest.raises(ValueError, match="overlap"):
            pn.cache_append(cache_on(-1), k, k, slots, table, q=q, q_out=q_out)
    assert len(on_host.calls) == made


@pytest.mark.parametrize("N,K", [(1, 17408), (64, 512), (200, 5120), (1024, 5120), (2560, 17408), (5120, 5120), (5120, 17408),
                                 (10240, 1024), (34816, 5120), (1024, 384)])
def test_gemm_int8_workspace_is_enough_for_fewer_rows(N, K):
    need = [pn.gemm_int8_workspace_bytes(M, N, K) for M in [*range(0, 3000, 7), *range(3000, 70000, 997)]]
    assert need == sorted(need)
    assert need[4] == 0  # up to 32 rows take none
    if K <= 384 or N > 32768:  # nor do short rows, or weights whose own tiles fill the machine
        assert need[-1] == 0


@pytest.mark.parametrize("args,pack", [(pn.AddNormArgs, pn._pack_add_norm), (pn.AppendArgs, pn._pack_append),
                                       (pn.LogprobsArgs, pn._pack_logprobs), (pn.AttendArgs, pn._pack_attend)])
def test_packed_arguments_are_the_structures(args, pack):
    """The calls pack by format strings what the structures name field by field."""
    values = [0.5 + n if kind is C.c_float else n + 1 for n, (_, kind) in enumerate(args._fields_)]
    packed = pack(*values)
    assert len(packed) == C.sizeof(args)
    fields = args.from_buffer_copy(packed)
    assert [getattr(fields, name) for name, _ in args._fields_] == values
