"""The operators around the linears at their largest: the tokens of a whole image and its prompt attending to each other, and
operands whose offsets pass 2^32 elements.  Compared with the definitions on sampled rows, heads and columns, by the references
and bounds of each operator's own tests."""
import numpy as np
import pytest
import torch

from epilogue_gemm_nvfp4_b200 import binding as B
from oracle import nvfp4_oracle as O
from tests import test_gpu_attention as attention
from tests import test_gpu_norm_rope as norm_rope
from tests import test_gpu_w4a16 as w4a16

pytestmark = pytest.mark.gpu


def normal(*shape, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", dtype=torch.bfloat16, generator=gen)


def check(q, k, v, got, lse, rows, heads, lens=None):
    """Sampled rows and heads (one key head each).  Beside the bound of the operator's tests, the running sums over the keys: one
    rounding, perhaps a cut, of 2^-23 per 16 keys."""
    for h in heads:
        kh = h * k.shape[2] // q.shape[2]
        part = [t[:, :, i:i + 1] for t, i in ((k, kh), (v, kh))]
        o, l, eo, el = attention.reference(q[:, rows, h:h + 1], *part, lens, q.shape[3] ** -0.5)
        weight = attention.reference(q[:, rows, h:h + 1], part[0], part[1].abs(), lens, q.shape[3] ** -0.5)[0]
        run = k.shape[1] / 16 * 2.0 ** -23
        room = o.abs() * 2.0 ** -8 + (eo + weight * 2 * run) * (1 + 2.0 ** -8)
        assert ((got[:, rows, h:h + 1].double() - o).abs() <= room).all(), h
        assert ((lse[:, h:h + 1, rows].double() - l).abs() <= el + run).all(), h


@pytest.mark.parametrize("n,H,D", [(4608, 18, 256), (16896, 18, 256), (16896, 36, 128), (16896, 72, 64)])
def test_attention_of_a_blocks_own_tokens(n, H, D):
    """q, k and v are the columns of one product of the block's 4096 or 16,384 image and 512 prompt tokens."""
    qkv = normal(1, n, 3, H, D, seed=n)
    q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    got, lse = B.cross_attention(q, k, v, want_lse=True)
    B.check_device_error()
    rows = torch.cat((torch.arange(5), torch.randint(0, n, (40,), generator=torch.Generator().manual_seed(1)), torch.arange(n - 5, n))).cuda()
    check(q, k, v, got, lse, rows, (0, H // 2, H - 1))
    assert torch.equal(B.cross_attention(q, k, v), got)


@pytest.mark.parametrize("Mq", [2, 1500])
def test_attention_to_keys_past_32_bit_offsets(Mq):
    Mk, H, D = (1 << 19) + 77, 32, 256     # 4.3e9 elements of k, and of v
    q, k, v = normal(1, Mq, H, D), normal(1, Mk, H, D, seed=1), normal(1, Mk, H, D, seed=2)
    lens = torch.tensor([Mk - 3], dtype=torch.int32, device="cuda")
    got, lse = B.cross_attention(q, k, v, kv_lens=lens, want_lse=True)
    B.check_device_error()
    check(q, k, v, got, lse, torch.tensor([0, Mq - 1], device="cuda"), (0, H - 1), lens)


def test_attention_with_queries_past_32_bit_offsets():
    Mq, H, D = (1 << 21) + 5, 8, 256
    q, k, v = normal(1, Mq, H, D), normal(1, 130, 2, D, seed=1), normal(1, 130, 2, D, seed=2)
    got, lse = B.cross_attention(q, k, v, want_lse=True)
    B.check_device_error()
    check(q, k, v, got, lse, torch.tensor([0, 1 << 20, Mq - 6, Mq - 1], device="cuda"), (0, 3, 7))


@pytest.mark.parametrize("interleaved", [False, True])
def test_head_norm_of_rows_past_32_bit_offsets(interleaved):
    rows, heads, D = 66000, 3, 128
    buf = torch.zeros(rows, 65536, dtype=torch.bfloat16, device="cuda")
    x = buf[:, 1024:1024 + heads * D].view(rows, heads, D)
    x.copy_(normal(rows, heads, D))
    last = slice(rows - 20, rows)
    before = x[last].clone()
    cos, sin = norm_rope.table(rows, D // 2)
    gamma = (torch.rand(D, device="cuda") + 0.5).bfloat16()
    B.qk_norm_rope(x, None, cos, sin, gamma_q=gamma, interleaved=interleaved, q_out=x)
    norm_rope.assert_close(x[last], norm_rope.reference(before, gamma, cos[last], sin[last], None, interleaved, 1e-6))
    assert (buf[last, :1024] == 0).all() and (buf[last, 1024 + heads * D:] == 0).all()


@pytest.mark.parametrize("M", [1, 5, 32])
def test_few_row_linear_on_codes_past_32_bit_offsets(M):
    N, K = (1 << 20) + 200, 8192          # 4.3e9 bytes of codes
    gen = torch.Generator(device="cuda").manual_seed(M)
    codes = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=torch.uint8, generator=gen)
    scales = torch.randint(0, 0x7F, (B.scale_bytes(N, K),), device="cuda", dtype=torch.uint8, generator=gen)
    w = B.QTensor(codes, scales, torch.tensor([1.0 / (64.0 * K ** 0.5)], device="cuda"), N, K)
    x = normal(M, K, seed=M)
    out = B.w4a16_linear(x, w)
    B.check_device_error()
    for first in (0, (N // 128 - 1) * 128, N // 128 * 128):   # whole row blocks, so that the scale atoms are theirs
        n = min(128, N - first)
        atoms = scales.view(-1, 512 * (K // 64))[first // 128:first // 128 + 1].reshape(-1)
        value = O.e2m1_decode(O.unpack_codes(codes[first:first + n].cpu().numpy())).astype(np.float64) * np.repeat(
            O.e4m3_decode(O.scales_from_mma_layout(atoms.cpu().numpy(), n, K)).astype(np.float64), 16, axis=1)
        w4a16.assert_within(out[:, first:first + n], *w4a16.reference(x, w, torch.from_numpy(value).cuda()))
