"""The operators around the linears at the ends of their ranges: exponents that leave fp32, heads whose squares do, one-row
views, calls whose operands do not belong together."""
import pytest
import torch

from epilogue_gemm_nvfp4_b200 import binding as B
from tests import test_gpu_norm_rope as norm_rope

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Mq,Mk,H", [(3, 900, 2), (200, 130, 1), (3000, 400, 8)])
@pytest.mark.parametrize("scale", [2.0 ** 20, 2.0 ** 28, 1.0e30, 1.0e36, 1.0e38])
def test_attention_to_the_largest_scores_alone(D, Mq, Mk, H, scale):
    """Scores that are whole numbers (exact in fp32) times a scale that leaves the largest of them alone: the output is the
    mean of v over the keys that share the largest score, which lie in different key tiles, and lse is that score plus the
    logarithm of their number.  Tolerance: half a bf16 step of the result; half a bf16 step of each p (one that comes from a
    product of score and scale below 2^24 is 1 only up to the rounding of that product, and the sum is of the unrounded p);
    their number (at most 2^10) times 2^-23 of mean |v| for the sum, 2^-20 for the reciprocal and the merge of a cluster;
    lse: 2^-21 of it for five roundings, 2^-20 for the logarithm."""
    gen = torch.Generator(device="cuda").manual_seed(D + Mq)
    q = torch.randint(-1, 2, (1, Mq, H, D), device="cuda", generator=gen).bfloat16()
    k = torch.randint(-1, 2, (1, Mk, H, D), device="cuda", generator=gen).bfloat16()
    k[:, Mk // 2:Mk // 2 * 2] = k[:, :Mk // 2]
    q[:, 1], k[:, :, H - 1] = 1, -k[:, :, H - 1].abs()  # rows without a positive score, one of small ones only
    v = torch.randn(1, Mk, H, D, device="cuda", generator=gen).bfloat16()
    out, lse = B.cross_attention(q, k, v, scale=scale, want_lse=True)
    B.check_device_error()
    s = torch.einsum("bqhd,bkhd->bhqk", q.double(), k.double())
    top = s.amax(-1, keepdim=True)
    w = (s == top).double()
    count = w.sum(-1, keepdim=True)
    assert count.max() <= 1024
    want = torch.einsum("bhqk,bkhd->bqhd", w / count, v.double())
    mag = torch.einsum("bhqk,bkhd->bqhd", w / count, v.double().abs())
    room = want.abs() * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -13 + 2.0 ** -20) * (1 + 2.0 ** -8)
    assert ((out.double() - want).abs() <= room).all()
    if scale < 1.0e37:  # the logarithm itself fits fp32
        ref = (top * scale + count.log())[..., 0]
        assert ((lse.double() - ref).abs() <= ref.abs() * 2.0 ** -21 + 2.0 ** -20).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows", [9, 4000])
def test_head_norm_of_heads_whose_squares_leave_fp32(D, interleaved, rows):
    """Heads of ordinary size beside heads of up to bf16's largest value (and of a few such elements), with a gamma that takes
    element times gamma past fp32 as well.  The formula and its tolerance are those of the operator's tests."""
    gen = torch.Generator(device="cuda").manual_seed(D)
    x = torch.randn(rows, 5, D, device="cuda", generator=gen)
    x[1::3, 1] *= 2.0 ** 100
    x[2::3, 2] = x[2::3, 2].clamp(-3, 3) * 2.0 ** 126
    x[::4, 3, ::9] *= 2.0 ** 80   # the others vanish beside these, but are not zero
    x = x.bfloat16()
    assert x.isfinite().all()
    cos, sin = norm_rope.table(rows, D // 2)
    gamma = (torch.rand(D, device="cuda", generator=gen) * 8 - 4).bfloat16()
    out, _ = B.qk_norm_rope(x, None, cos, sin, gamma_q=gamma, interleaved=interleaved)
    some = slice(0, rows) if rows < 100 else slice(1990, 2010)
    ref = norm_rope.reference(x[some], gamma, cos[some], sin[some], None, interleaved, 1e-6)
    norm_rope.assert_close(out[some], ref)
    # an infinity makes its head's other elements zeros and itself NaN; the heads beside it keep their bits
    y = x.clone()
    y[4, 1, 3] = float("inf")
    got = B.qk_norm_rope(y, None, None, None, gamma_q=gamma)[0]
    want = B.qk_norm_rope(x, None, None, None, gamma_q=gamma)[0]
    assert got[4, 1, 3].isnan() and (got[4, 1, :3] == 0).all() and (got[4, 1, 4:] == 0).all()
    got[4, 1] = want[4, 1]
    assert torch.equal(got, want)


def test_cleared_rows_of_every_last_tile():
    """Head_dim 256 on CTA pairs, thousands of pieces of work of one to three key tiles, each of which ends inside a tile with NaN
    and infinities behind it: every piece's zeros reach the other CTA's products, in many repeats."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()
    Bn, Mq, Mk, H, D = 24, 1100, 384, 24, 256
    q, k, v = r(Bn, Mq, H, D), r(Bn, Mk, H, D), r(Bn, Mk, H, D)
    n = torch.randint(1, Mk, (Bn,), device="cuda", generator=gen, dtype=torch.int32)
    gone = (torch.arange(Mk, device="cuda") >= n[:, None])[:, :, None, None]
    clean = B.cross_attention(q, torch.where(gone, 0, k), torch.where(gone, 0, v), kv_lens=n)
    k, v = torch.where(gone, float("nan"), k), torch.where(gone, float("inf"), v)
    out = torch.empty_like(q)
    for _ in range(50):
        B.cross_attention(q, k, v, kv_lens=n, out=out)
        assert torch.equal(out, clean)
    B.check_device_error()


def test_one_row_of_a_buffer_with_any_row_stride():
    """A single row's stride says nothing: rows of buffers whose stride no kernel could take give the contiguous row's bits."""
    K, N, D = 256, 96, 128
    w = B.quantize(torch.randn(N, K, device="cuda").bfloat16())

    def row(*shape, dtype=torch.bfloat16, extra=1):
        """The first of three rows of a buffer whose rows are `extra` elements longer."""
        n = shape[0] * shape[1] if len(shape) == 2 else shape[0]
        inner = (shape[1], 1) if len(shape) == 2 else (1,)
        return torch.randn(3, n + extra, device="cuda").to(dtype).as_strided((1, *shape), (n + extra, *inner))

    def plain(t):
        return torch.empty(t.shape, dtype=t.dtype, device="cuda").copy_(t)

    x, res, gate, out = row(K), row(N), torch.rand(N, device="cuda"), row(N, extra=3)
    assert x.stride(0) == K + 1
    B.w4a16_linear(x, w, "resid_gate", residual=res, gate=gate, out=out)
    assert torch.equal(out, B.w4a16_linear(plain(x), w, "resid_gate", residual=plain(res), gate=gate))
    q, k, out = row(4, D), row(2, D), row(4, D, extra=5)
    cos, sin = row(D // 2, dtype=torch.float32), row(D // 2, dtype=torch.float32, extra=3)
    qo, ko = B.qk_norm_rope(q, k, cos, sin, q_out=out)
    qc, kc = B.qk_norm_rope(plain(q), plain(k), plain(cos), plain(sin))
    assert torch.equal(qo, qc) and torch.equal(ko, kc)
    assert torch.equal(B.cross_attention(q[None], k[None], k[None]), B.cross_attention(plain(q)[None], plain(k)[None], plain(k)[None]))


def test_head_norm_refuses_operands_of_what_is_not_there():
    """An output for no k would come back unwritten; positions without tables would turn nothing."""
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos, gamma = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(k_out=torch.empty_like(q)), dict(gamma_k=gamma), dict(positions=pos)):
        with pytest.raises(ValueError):
            B.qk_norm_rope(q, None, None, None, **kw)


def test_few_row_linear_refuses_a_weight_smaller_than_it_says():
    """Codes or scale bytes of fewer rows or columns would be read past their end, and so would one row of codes for all."""
    q = B.quantize(torch.randn(256, 128, device="cuda").bfloat16())
    x = torch.randn(2, 128, device="cuda").bfloat16()
    want = B.w4a16_linear(x, q)
    # larger buffers than it says are fine: the first rows of a longer weight, codes with more columns
    assert torch.equal(B.w4a16_linear(x, B.QTensor(q.codes, q.scales, q.g, 128, 128)), want[:, :128])
    wide = torch.cat((q.codes, q.codes), 1)
    assert torch.equal(B.w4a16_linear(x, B.QTensor(wide, q.scales.view(2, -1), q.g, 256, 128)), want)
    for w in (B.QTensor(q.codes[:128], q.scales, q.g, 256, 128), B.QTensor(q.codes[:, :32], q.scales, q.g, 256, 128),
              B.QTensor(q.codes[:1].expand(256, 64), q.scales, q.g, 256, 128), B.QTensor(q.codes, q.scales[:1024], q.g, 256, 128),
              B.QTensor(q.codes.view(-1), q.scales, q.g, 256, 128), B.QTensor(q.codes, q.scales[::2], q.g, 256, 128)):
        with pytest.raises(ValueError):
            B.w4a16_linear(x, w)


def test_scalar_operands():
    """A weight whose scale is a tensor without dimensions, as nvfp4_linear takes it; any other such operand is refused."""
    q = B.quantize(torch.randn(256, 128, device="cuda").bfloat16())
    x = torch.randn(2, 128, device="cuda").bfloat16()
    scalar = torch.zeros((), dtype=torch.bfloat16, device="cuda")
    assert torch.equal(B.w4a16_linear(x, B.QTensor(q.codes, q.scales, q.g[0], 256, 128)), B.w4a16_linear(x, q))
    for call in (lambda: B.w4a16_linear(x, q, bias=scalar), lambda: B.w4a16_linear(scalar, q), lambda: B.qk_norm_rope(scalar, None, None, None),
                 lambda: B.qk_norm_rope(x.view(2, 2, 64), None, None, None, gamma_q=scalar),
                 lambda: B.cross_attention(x.view(1, 2, 2, 64), scalar, scalar)):
        with pytest.raises(ValueError):
            call()
