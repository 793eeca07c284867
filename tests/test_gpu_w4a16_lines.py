"""The few-row linear where its line of 256-element chunks is much longer than the grid: CTAs that go round their ring, sum over many
chunks, and cross from one unit of 256 weight rows to the next, for every number of rows that has a kernel of its own.
Definition, error bound and weights are those of the operator's other tests."""
import pytest
import torch

from epilogue_gemm_nvfp4_b200 import binding as B
from tests.test_gpu_w4a16 import assert_within, make_weight, reference

pytestmark = pytest.mark.gpu

CTAS = 160  # at least as many as the grid has


def operands(M, N, K, kind, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + M)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()
    more = {"residual": r(M, N), "gate": torch.randn(N, device="cuda", generator=gen)} if kind == "resid_gate" else {}
    return r(M, K), dict(kind=kind, bias=r(N), **more)


@pytest.mark.parametrize("N,K,rows", [
    (1536, 53248, [(8, "bias"), (16, "bias"), (32, "bias"), (31, "resid_gate")]),          # eight chunks per CTA, units shared by CTAs
    (6144, 4608, [(32, "gated_silu"), (16, "gated_silu"), (3, "gated_silu"), (2, "gated_silu"), (1, "gated_silu")]),
    (4608, 4608, [(17, "resid_gate"), (9, "resid_gate"), (5, "resid_gate"), (1, "resid_gate")]),
    # three units of one chunk and more per CTA
    (3 * 256 * CTAS + 1, 256, [(1, "bias"), (2, "bias"), (8, "bias"), (16, "bias"), (32, "bias")]),
    # units of two and a quarter chunks, the CTAs' ranges start anywhere in them: one and two rows' own digits serve several units
    (3 * 256 * CTAS, 576, [(1, "bias"), (2, "gated_silu"), (7, "gated_silu"), (16, "bias"), (32, "gated_silu")]),
])
def test_matches_definition(N, K, rows):
    w, value = make_weight(N, K, seed=N + K)
    for M, kind in rows:
        x, more = operands(M, N, K, kind)
        out = B.w4a16_linear(x, w, **more)
        B.check_device_error()
        assert_within(out, *reference(x, w, value, **more))


@pytest.mark.parametrize("N,K,kind", [(2048, 20480, "bias"), (3 * 256 * CTAS, 576, "gated_silu"), (2 * 256 * CTAS, 1088, "resid_gate")])
def test_rows_do_not_depend_on_their_number(N, K, kind):
    w, _ = make_weight(N, K, seed=5)
    x, more = operands(32, N, K, kind)
    whole = B.w4a16_linear(x, w, **more)
    part = lambda a, b: {n: t[a:b] if n == "residual" else t for n, t in more.items()}
    for a, b in ((0, 1), (0, 2), (0, 8), (0, 9), (0, 16), (0, 17), (0, 31), (30, 32), (20, 21), (5, 13)):
        assert torch.equal(B.w4a16_linear(x[a:b], w, **part(a, b)), whole[a:b]), (a, b)
    B.check_device_error()


def test_the_residual_may_be_the_output():
    for M, N, K in ((3, 300, 512), (32, 4608, 1024), (1, 130, 256)):
        w, _ = make_weight(N, K, seed=M)
        x, more = operands(M, N, K, "resid_gate")
        want = B.w4a16_linear(x, w, **more)
        got = B.w4a16_linear(x, w, **more, out=more["residual"])
        assert got.data_ptr() == more["residual"].data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("M", [1, 6, 32])
def test_silu_over_its_whole_range(M):
    """silu(x) for x from -100 to 30, block by block, against the bound that the header states for x': 2^-17 of the power of two of the
    block's largest (2^-34 of the row's), twice for an element that the first error takes to the other neighbour, (|x| + 4) 2^-22 of
    itself, and 2^-119 where the division gives 0.  The weights are positive, so that every element's error would show."""
    N, K = 64, 1024
    w, value = make_weight(N, K, seed=3)
    w.codes.bitwise_and_(0x77)
    value = value.abs()
    gen = torch.Generator(device="cuda").manual_seed(M)
    mid = torch.linspace(-97, 28, K // 16, device="cuda").repeat_interleave(16)
    x = (mid + torch.randn(M, K, device="cuda", generator=gen)).bfloat16()
    x[M // 2, 300:] = -90.5   # a row of the smallest values alone
    x[M // 2, :300] = -60.0
    xd = x.double()
    s = xd / (1.0 + torch.exp(-xd))
    power = lambda t: torch.exp2(torch.floor(torch.log2(t)))
    block = torch.maximum(power(s.abs().view(M, -1, 16).amax(-1)), power(s.abs().amax(1, keepdim=True)) * 2.0 ** -17)
    off = 2 * 2.0 ** -17 * block.repeat_interleave(16, dim=1) + s.abs() * (xd.abs() + 4) * 2.0 ** -22 + 2.0 ** -119
    g = w.g.double()
    ref = s @ value.t() * g
    err = (off @ value.t() + (s.abs() @ value.t()) * (K / 8 + 12) * 2.0 ** -23) * g
    out = B.w4a16_linear(x, w, silu_input=True)
    B.check_device_error()
    assert_within(out, ref, err + 2.0 ** -133)   # half of bf16's smallest step
