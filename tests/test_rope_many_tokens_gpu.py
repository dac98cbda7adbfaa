"""Rotation and head norms over thousands of tokens: blocks with several tokens
and several rounds of them, ragged last rounds, rows divided by odd numbers of
heads, the sharing of the gradient's blocks between queries and keys."""
import pytest
import torch

from tests import attention_reference as ref
from tests.test_rope_gpu import _positions, _rand, _within, ets  # noqa: F401

pytestmark = pytest.mark.gpu

# D, rot, offset: vectors of 16, 8 and 4 bytes and single elements
SHAPES = [(128, 128, 0), (64, 64, 0), (128, 64, 64), (96, 12, 0), (90, 30, 10), (37, 10, 3)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,offset", SHAPES)
@pytest.mark.parametrize("T,H,Hk", [(5003, 7, 1), (5003, 12, 5), (20011, 3, 2)])
def test_many_tokens(ets, dtype, interleaved, D, rot, offset, T, H, Hk):  # noqa: F811
    freqs, pos = ets.rope_freqs(rot), _positions(T)
    q, k = _rand((T, H, D), dtype, 1), _rand((T, Hk, D), dtype, 2)
    qw, kw = (1 + 0.3 * _rand((D,), dtype, s) for s in (3, 4))
    dy = [_rand(t.shape, dtype, 5 + i) for i, t in enumerate((q, k))]
    opt = {"interleaved": interleaved, "offset": offset, "scale": 0.75}
    x = ets.topk_rope(q, pos, freqs, **opt)
    want, mag = ref.rotate(q.double(), pos, freqs, interleaved, offset, 0.75)
    _within(x, want, ref.rope_bound(want, mag, dtype))
    got = ets.topk_qk_norm_rope(q, k, qw, kw, pos, freqs, **opt)
    grad = ets.topk_qk_norm_rope_backward(*dy, q, k, qw, kw, pos, freqs, **opt)
    for j, (x, w) in enumerate(((q, qw), (k, kw))):
        n, _ = ref.norm(x, w, 1e-6)
        want, mag = ref.rotate(n, pos, freqs, **opt)
        _within(got[j], want, ref.norm_bound(want, mag, dtype))
        dx, size, dw, terms = ref.norm_grad(dy[j], x, w, pos, freqs, 1e-6, **opt)
        _within(grad[j], dx, 2.0 ** -17 * size + ref.rounding(dx, dtype))
        # a lane adds a few dozen rows, then warps and blocks are joined: below 2^7 roundings
        _within(grad[2 + j], dw, 2.0 ** -17 * terms + 1e-37)


@pytest.mark.parametrize("T", [303, 305, 609, 1217, 4999])
@pytest.mark.parametrize("H,Hk", [(64, 1), (1, 9), (129, 2)])
def test_token_counts_around_the_blocks(ets, T, H, Hk):  # noqa: F811
    """Counts at which blocks go from one token to two and more."""
    D = 64
    freqs, pos = ets.rope_freqs(D), _positions(T)
    q, k = _rand((T, H, D), torch.bfloat16, 1), _rand((T, Hk, D), torch.bfloat16, 2)
    w = 1 + 0.3 * _rand((D,), torch.float32, 3)
    got = ets.topk_qk_norm_rope(q, k, w, w, pos, freqs)
    grad = ets.topk_qk_norm_rope_backward(q, k, q, k, w, w, pos, freqs)
    for j, x in enumerate((q, k)):
        n, _ = ref.norm(x, w, 1e-6)
        want, mag = ref.rotate(n, pos, freqs)
        _within(got[j], want, ref.norm_bound(want, mag, torch.bfloat16))
        dx, size, dw, terms = ref.norm_grad(x, x, w, pos, freqs, 1e-6)
        _within(grad[j], dx, 2.0 ** -17 * size + ref.rounding(dx, torch.bfloat16))
        _within(grad[2 + j], dw, 2.0 ** -17 * terms + 1e-37)
