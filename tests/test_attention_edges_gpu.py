"""Attention over selected keys at the edges of its inputs: values that are not
finite, very large or very small ones, rows with one key, clusters with several
items, other streams.  64-bit references and bounds: tests/attention_reference.py."""
import math

import pytest
import torch

from tests import attention_reference as ref
from tests.test_sparse_attention_gpu import _rand, _select, ets  # noqa: F401

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
# tokens: few (with five chunks of keys and more, clusters share their items) and
# more than SMs
TOKENS = [2, 400]


def _inputs(T, H, Hk, D, K, S, dtype=torch.bfloat16, fill=None):
    q, k, v = (_rand(s, dtype, i) for i, s in enumerate(((T, H, D), (S, Hk, D), (S, Hk, D))))
    return q, k, v, _select(T, K, S, fill=fill)


def _same_kind(got, want):
    """Equal where want is not finite (NaN with NaN, infinities by sign)."""
    got, want = got.double(), want.double()
    kind = lambda x: torch.where(x.isnan(), 2.0, torch.where(x.isinf(), x.sign(), 0.0))  # noqa: E731
    return torch.equal(kind(got), kind(want))


def _bad_head_and_key(T, H, D, dtype=torch.bfloat16):
    """q with a NaN in head 1 of token 1 and k with one in a key that only token
    0 selects."""
    q, k, v, idx = _inputs(T, H, 1, D, 600, 900, dtype)
    key = int(idx[0, 150])
    idx[1:][idx[1:] == key] = -1
    clean = q.clone(), k.clone()
    q[1, 1, 7] = math.nan
    k[key, 0, 3] = math.nan
    return q, k, v, idx, key, clean


@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("H", [4, 40, 100])
def test_nan_scores_stay_nan(ets, softcap, T, H):  # noqa: F811
    """Rows with a NaN score are NaN, with and without the cap; the others do not change."""
    q, k, v, idx, key, clean = _bad_head_and_key(T, H, 64)
    good = torch.ones((T, H), dtype=torch.bool, device=DEV)
    good[1, 1] = False
    good[0] = False
    out, lse = ets.topk_sparse_attention(q, k, v, idx, softcap=softcap, return_lse=True)
    want, wlse = ets.topk_sparse_attention(*clean, v, idx, softcap=softcap, return_lse=True)
    assert bool(out[~good].isnan().all()) and bool(lse[0].isnan().all())
    assert torch.equal(out[good], want[good]) and torch.equal(lse[good], wlse[good])
    dout = _rand(q.shape, q.dtype, 7)
    bad_lse = wlse.clone()
    bad_lse[~good] = math.nan
    dq, dk, dv = ets.topk_sparse_attention_backward(dout, q, k, v, idx, out, bad_lse,
                                                    softcap=softcap)
    assert bool(dq[~good].isnan().all()) and bool(dq[good].isfinite().all())
    hit = torch.zeros(900, dtype=torch.bool, device=DEV)
    hit[idx[:2][idx[:2] >= 0].long()] = True
    assert bool(dk[hit].isnan().all()) and bool(dv[hit].isnan().all())
    assert bool(dk[~hit].isfinite().all()) and bool(dv[~hit].isfinite().all())


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("H", [4, 40, 100])
def test_nan_scores_hidden_by_the_cap_in_the_gradient(ets, T, H):  # noqa: F811
    """The scores alone carry the NaN (lse and out are the clean call's)."""
    q, k, v, idx, key, clean = _bad_head_and_key(T, H, 64)
    out, lse = ets.topk_sparse_attention(*clean, v, idx, softcap=5.0, return_lse=True)
    dq, dk, _ = ets.topk_sparse_attention_backward(_rand(q.shape, q.dtype, 7), q, k, v, idx, out,
                                                   lse, softcap=5.0)
    assert bool(dq[1, 1].isnan().all()) and bool(dq[0].isnan().all())
    assert bool(dk[key].isnan().all())


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("H", [4, 40, 100])
def test_log_sum_of_nan_scores_is_nan(ets, T, H):  # noqa: F811
    """A head whose scores are all NaN has lse NaN: -inf means that no key is left."""
    q, k, v, idx = _inputs(T, H, 1, 128, 600, 900)
    want = ets.topk_sparse_attention(q, k, v, idx, return_lse=True)[1]
    q[1, 1, 7] = math.nan
    idx[0] = -1
    out, lse = ets.topk_sparse_attention(q, k, v, idx, return_lse=True)
    assert bool(lse[1, 1].isnan()) and bool(out[1, 1].isnan().all())
    assert bool((lse[0] == -math.inf).all()) and float(out[0].float().abs().max()) == 0.0
    rest = torch.ones((T, H), dtype=torch.bool, device=DEV)
    rest[0], rest[1, 1] = False, False
    assert torch.equal(lse[rest], want[rest])


def _infinite_values(v, keys):
    """Infinities and NaN in columns of their own: one +inf, one -inf, two +inf,
    both signs, a NaN, a NaN beside an infinity."""
    a, b = (int(x) for x in keys)
    v[a, :, 0] = math.inf
    v[b, :, 1] = -math.inf
    v[a, :, 2], v[b, :, 2] = math.inf, math.inf
    v[a, :, 3], v[b, :, 3] = math.inf, -math.inf
    v[a, :, 4] = math.nan
    v[a, :, 5], v[b, :, 5] = math.inf, math.nan


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", TOKENS + [160])
@pytest.mark.parametrize("H,Hk,D", [(4, 1, 64), (40, 1, 128), (100, 1, 64), (16, 2, 128)])
def test_infinite_values(ets, dtype, T, H, Hk, D):  # noqa: F811
    """A selected infinity gives an infinity, however many heads share the key and
    however small its weight; keys a and b lie in different tiles and parts of them."""
    K, S = (2048, 3000) if T == 160 else (600, 900)  # 160 items: clusters with several each
    q, k, v, idx = _inputs(T, H, Hk, D, K, S, dtype)
    _infinite_values(v, (idx[0, 5], idx[0, 450]))
    idx[1, :] = idx[0]  # a second row with both
    q[1] *= 8           # whose weights are far apart
    out, lse = ets.topk_sparse_attention(q, k, v, idx, return_lse=True)
    n = min(T, 24)
    r = ref.attend(q[:n], k, v, idx[:n], D ** -0.5)
    assert _same_kind(out[:n], r["out"]) and bool(lse.isfinite().all())
    bound, _ = ref.attend_bounds(r, v, idx[:n], dtype)
    fine = r["out"].isfinite()
    assert bool(((out[:n].double() - r["out"]).abs() <= bound)[fine].all())


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("H,Hk,D", [(4, 1, 64), (40, 1, 128), (100, 1, 64), (16, 2, 128)])
def test_infinite_output_gradients(ets, T, H, Hk, D):  # noqa: F811
    """dv of an infinite dout is infinite (with its sign), NaN where both signs or a NaN meet."""
    K, S = 200, 300
    q, k, v, idx = _inputs(T, H, Hk, D, K, S)
    dout = _rand(q.shape, q.dtype, 7)
    dout[0, 0, 0] = math.inf
    dout[1, H - 1, 1] = -math.inf
    dout[0, 0, 2], dout[1, 1, 2] = math.inf, -math.inf
    dout[1, 0, 3] = math.nan
    out, lse = ets.topk_sparse_attention(q, k, v, idx, return_lse=True)
    n = 2
    got = ets.topk_sparse_attention_backward(dout[:n].contiguous(), q[:n].contiguous(), k, v,
                                             idx[:n].contiguous(), out[:n].contiguous(),
                                             lse[:n].contiguous())
    r = ref.attend(q[:n], k, v, idx[:n], D ** -0.5)
    want, bound = ref.attend_grad(dout[:n], q[:n], k, v, idx[:n], out[:n], lse[:n], r, D ** -0.5)
    assert _same_kind(got[2], want[2])
    fine = want[2].isfinite() & bound[2].isfinite()
    assert bool(((got[2].double() - want[2]).abs() <= bound[2])[fine].all())
    if T > n:  # the other tokens' rows of the whole call
        dq = ets.topk_sparse_attention_backward(dout, q, k, v, idx, out, lse)[0]
        assert bool(dq[n:].isfinite().all())


@pytest.mark.parametrize("power", [-12, -4, 10, 12, 13])
@pytest.mark.parametrize("H,Hk,D", [(2, 1, 128), (8, 2, 128), (36, 1, 64)])
def test_float16_gradients_of_scaled_losses(ets, power, H, Hk, D):  # noqa: F811
    """dout times 2^power: P (dP - delta) passes float16's 65504 where dq, dk and dv
    do not.  dS is held times a power of two that puts the token's largest |dout|
    into [4, 8), so what its rounding may lose below the normal range is
    2^-25 / factor."""
    T, K, S = 5, 40, 400
    q = _rand((T, H, D), torch.float16, 1, 2.0)
    k, v = _rand((S, Hk, D), torch.float16, 2, 1.5), _rand((S, Hk, D), torch.float16, 3, 3.0)
    idx = _select(T, K, S)
    dout = (_rand((T, H, D), torch.float32, 4).clamp(-3, 3) * 2.0 ** power).half()
    scale = D ** -0.5
    out, lse = ets.topk_sparse_attention(q, k, v, idx, scale=scale, return_lse=True)
    got = ets.topk_sparse_attention_backward(dout, q, k, v, idx, out, lse, scale=scale)
    r = ref.attend(q, k, v, idx, scale)
    want, bound = ref.attend_grad(dout, q, k, v, idx, out, lse, r, scale)
    G = H // Hk
    top = dout.double().abs().view(T, Hk, -1).amax(-1)  # [T, Hk]
    lost = 2.0 ** -25 * 2.0 ** (torch.floor(torch.log2(top)) - 2)
    i = idx.long()
    bound[0] += scale * torch.einsum("tn,tknd->tnd", lost, k.double().abs()[i]).repeat_interleave(G, 1)
    heads = q.double().abs().view(T, Hk, G, D).sum(2) * lost[..., None]
    bound[1].index_add_(0, i.flatten(), scale * heads[:, None].expand(-1, K, -1, -1).reshape(-1, Hk, D))
    for g, w, b in zip(got, want, bound):
        keep = w.abs() < 65000  # what float16 holds
        assert float(keep.double().mean()) > 0.99
        err = (g.double() - w).abs()
        assert bool((err <= b)[keep].all()), float((err / b)[keep].max())


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("H", [4, 40, 100])
@pytest.mark.parametrize("power", [75, -60])
def test_large_and_small_values_under_growing_scores(ets, T, H, power):  # noqa: F811
    """Values near 2^power in bfloat16 while the scores' maximum climbs by 20 nats
    a tile: weights and values together stay inside FP32."""
    D, S = 64, 768
    q = _rand((T, H, D), torch.bfloat16, 4, 0.05)
    q[..., 0] = 1.0
    k = _rand((S, 1, D), torch.bfloat16, 5, 0.05)
    k[:, 0, 0] = torch.tensor([0.0, 20, 40], device=DEV).repeat_interleave(256).bfloat16()
    v = (_rand((S, 1, D), torch.float32, 6) * 2.0 ** power).bfloat16()
    idx = torch.arange(S, dtype=torch.int32, device=DEV)[None].repeat(T, 1)
    out, lse = ets.topk_sparse_attention(q, k, v, idx, scale=1.0, return_lse=True)
    n = 4
    r = ref.attend(q[:n], k, v, idx[:n], 1.0)
    ob, lb = ref.attend_bounds(r, v, idx[:n], torch.bfloat16)
    assert bool(((out[:n].double() - r["out"]).abs() <= ob).all())
    assert bool(((lse[:n].double() - r["lse"]).abs() <= lb).all())


@pytest.mark.parametrize("softcap", [300.0, 1e4, 1e6, 1e30])
@pytest.mark.parametrize("H", [8, 100])
def test_caps_far_above_the_scores(ets, softcap, H):  # noqa: F811
    """Such a cap changes next to nothing: its tanh is right relative to the score
    (2^-20 of it: below the product's own bound), not only to the cap."""
    T, D, K, S = 6, 64, 200, 400
    q, k, v, idx = _inputs(T, H, 1, D, K, S)
    out, lse = ets.topk_sparse_attention(q, k, v, idx, softcap=softcap, return_lse=True)
    r = ref.attend(q, k, v, idx, D ** -0.5, softcap)
    r["mag"] = ref.attend(q, k, v, idx, D ** -0.5)["mag"]  # without what a cap may add
    ob, lb = ref.attend_bounds(r, v, idx, q.dtype)
    assert bool(((out.double() - r["out"]).abs() <= ob).all())
    assert bool(((lse.double() - r["lse"]).abs() <= lb).all())
    dout = _rand(q.shape, q.dtype, 7)
    got = ets.topk_sparse_attention_backward(dout, q, k, v, idx, out, lse, softcap=softcap)
    want, bound = ref.attend_grad(dout, q, k, v, idx, out, lse, r, D ** -0.5, softcap)
    for g, w, b in zip(got, want, bound):
        assert bool(((g.double() - w).abs() <= b).all())


@pytest.mark.parametrize("H", [4, 40, 100])
def test_gradients_of_rows_whose_scores_are_all_minus_infinity(ets, H):  # noqa: F811
    """A bias below every finite score leaves nothing: out 0, lse -inf, gradients 0."""
    T, D, K, S = 5, 64, 150, 400
    q, k, v, idx = _inputs(T, H, 1, D, K, S)
    slopes = torch.zeros(H, device=DEV)
    slopes[1] = 2e38
    opt = {"slopes": slopes, "positions": torch.full((T,), 2000, dtype=torch.int32, device=DEV)}
    out, lse = ets.topk_sparse_attention(q, k, v, idx, return_lse=True, **opt)
    assert float(out[:, 1].float().abs().max()) == 0.0 and bool((lse[:, 1] == -math.inf).all())
    dout = _rand(q.shape, q.dtype, 7)
    dq, dk, dv = ets.topk_sparse_attention_backward(dout, q, k, v, idx, out, lse, **opt)
    assert float(dq[:, 1].float().abs().max()) == 0.0
    keep = [h for h in range(H) if h != 1]
    plain = [t[:, keep].contiguous() for t in (dout, q, out)]
    _, ek, ev = ets.topk_sparse_attention_backward(plain[0], plain[1], k, v, idx, plain[2],
                                                   lse[:, keep].contiguous())
    for a, b in ((dk, ek), (dv, ev)):
        assert bool(a.isfinite().all())
        assert float((a.double() - b.double()).abs().max()) <= 2.0 ** -7 * float(b.abs().max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,Hk,D", [(2, 128, 4, 64), (24, 128, 1, 64), (7, 32, 8, 128), (300, 8, 1, 128)])
def test_rows_with_one_key(ets, dtype, T, H, Hk, D):  # noqa: F811
    """One key: out is its value, dv its dout, and dq and dk are zero up to the
    rounding of dP - delta, two sums of the same D products: 2 D 2^-24 of their
    magnitudes each (4 where an accumulator truncates), times the scale and the
    other factor."""
    S = 500
    q, k, v, idx = _inputs(T, H, Hk, D, 17, S, dtype, fill=[t % 2 for t in range(T)])
    out, lse = ets.topk_sparse_attention(q, k, v, idx, return_lse=True)
    dout = _rand(q.shape, dtype, 7)
    dq, dk, dv = ets.topk_sparse_attention_backward(dout, q, k, v, idx, out, lse)
    G, scale = H // Hk, D ** -0.5
    slack = torch.zeros((S, Hk, D), dtype=torch.float64, device=DEV)
    sums = torch.zeros_like(slack)
    for t in range(T):
        if t % 2 == 0:
            assert not bool(out[t].any()) and not bool(dq[t].any())
            continue
        key = int(idx[t].max())
        vh, kh = (x[key].repeat_interleave(G, 0) for x in (v, k))
        assert torch.equal(out[t], vh)
        res = 4 * 2 * D * 2.0 ** -24 * (dout[t].double() * vh.double()).abs().sum(-1) * scale  # [H]
        tiny = 2.0 ** -24 if dtype == torch.float16 else 0.0
        assert bool((dq[t].double().abs() <= res[:, None] * 1.01 * kh.double().abs() + tiny).all())
        slack[key] += (res[:, None] * q[t].double().abs()).view(Hk, G, D).sum(1)
        sums[key] += dout[t].double().view(Hk, G, D).sum(1)
    assert bool((dk.double().abs() <= 1.01 * slack + (2.0 ** -24 if dtype == torch.float16 else 0)).all())
    # P is 1 to FP32's exponential and logarithm (2^-20), rounded to 16 bits: 1
    mag = torch.zeros_like(sums)
    for t in range(1, T, 2):
        mag[int(idx[t].max())] += dout[t].double().abs().view(Hk, G, D).sum(1)
    assert bool(((dv.double() - sums).abs() <= ref.rounding(sums, dtype) + 2.0 ** -18 * mag).all())


def _rounds(ets_, T, H, Hk, D, K, S, fill, dtype=torch.bfloat16):
    q, k, v, idx = _inputs(T, H, Hk, D, K, S, dtype, fill=fill)
    out, lse = ets_.topk_sparse_attention(q, k, v, idx, return_lse=True)
    for a in range(0, T, 4):
        b = min(a + 4, T)
        r = ref.attend(q[a:b], k, v, idx[a:b], D ** -0.5)
        ob, lb = ref.attend_bounds(r, v, idx[a:b], dtype)
        assert bool(((out[a:b].double() - r["out"]).abs() <= ob).all())
        none = torch.isinf(r["lse"])
        assert torch.equal(torch.isinf(lse[a:b]), none)
        assert bool(((lse[a:b].double() - r["lse"]).abs() <= lb)[~none].all())
    assert ets_.sparse_attention_read_status() == 0


# a little more items than SMs (or than SMs / 4) and many chunks: clusters of 2, 4
# and 8 CTAs with several items each, an odd last round among them
@pytest.mark.parametrize("D,G,Hk", [(64, 8, 8), (128, 8, 1), (128, 64, 4), (64, 128, 8), (128, 100, 5)])
@pytest.mark.parametrize("K,items", [(2048, 1.05), (2048, 1.3), (4096, 1.05), (8000, 0.3)])
def test_clusters_with_several_items(ets, D, G, Hk, K, items):  # noqa: F811
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = -(-int(sms * items) // Hk)
    # rows that leave CTAs of a cluster without a tile, empty rows, full ones
    fill = [(K, 0, 100, K - 1, 129, 1, K)[t % 7] for t in range(T)]
    _rounds(ets, T, G * Hk, Hk, D, K, 9000, fill)


def test_results_on_another_stream_wait_for_nobody(ets):  # noqa: F811
    """A call on another stream takes its memory from that stream: blocks that the
    current stream still uses are not written into."""
    T, H, D, K, S = 64, 16, 128, 300, 900
    q, k, v, idx = _inputs(T, H, 1, D, K, S)
    dout, x = _rand(q.shape, q.dtype, 7), _rand((T, 1, D), q.dtype, 8)
    w, pos = torch.ones(D, device=DEV), torch.arange(T, dtype=torch.int32, device=DEV)
    freqs = ets.rope_freqs(D)
    out, lse = ets.topk_sparse_attention(q, k, v, idx, return_lse=True)

    def calls(stream=None):
        return (*ets.topk_sparse_attention(q, k, v, idx, return_lse=True, stream=stream),
                ets.topk_sparse_attention_backward(dout, q, k, v, idx, out, lse, stream=stream)[0],
                ets.topk_rope(q, pos, freqs, stream=stream),
                *ets.topk_qk_norm_rope(q, x, w, w, pos, freqs, stream=stream),
                *ets.topk_qk_norm_rope_backward(dout, x, q, x, w, w, pos, freqs, stream=stream))

    want = calls()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of every size that the calls ask for, still to be written by this stream
    late = [torch.empty_like(t) for t in want for _ in range(4)]
    late += [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (1 << 17, 1 << 19, 1 << 20, 1 << 21)]
    for t in late:  # (loads the kernels)
        t.fill_(6)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for t in late:
        t.fill_(7)
    del late, t
    got = calls(s)
    s.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_inputs_of_another_stream_outlive_the_call(ets):  # noqa: F811
    """The caller may drop the inputs as soon as a call on another stream returns."""
    T, H, D, K, S = 64, 16, 128, 300, 900
    base = _inputs(T, H, 1, D, K, S)
    want = ets.topk_sparse_attention(*base)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    mine = [t.clone() for t in base]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    got = ets.topk_sparse_attention(*mine, stream=s)
    shapes = [(t.shape, t.dtype) for t in mine]
    del mine
    over = [torch.full(sh, 3, dtype=dt, device=DEV) for sh, dt in shapes for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del over


@pytest.mark.parametrize("T", [0, 1, 5])
def test_no_selected_keys_at_all(ets, T):  # noqa: F811
    """idx with no column: nothing is left in any row."""
    q, k, v, _ = _inputs(T, 8, 2, 64, 1, 30)
    idx = torch.empty((T, 0), dtype=torch.int32, device=DEV)
    out, lse = ets.topk_sparse_attention(q, k, v, idx, return_lse=True)
    assert out.shape == q.shape and not bool(out.any()) and bool((lse == -math.inf).all())
    grads = ets.topk_sparse_attention_backward(_rand(q.shape, q.dtype, 7), q, k, v, idx, out, lse)
    assert [g.shape for g in grads] == [q.shape, k.shape, v.shape]
    assert not any(bool(g.any()) for g in grads)


def test_one_row_of_keys_for_all_tokens(ets):  # noqa: F811
    """idx broadcast over the tokens (row stride 0)."""
    q, k, v, idx = _inputs(9, 8, 2, 64, 200, 300)
    row = idx[:1].expand(9, -1)
    assert row.stride(0) == 0
    dout = _rand(q.shape, q.dtype, 7)
    out, lse = ets.topk_sparse_attention(q, k, v, row, return_lse=True)
    want, wlse = ets.topk_sparse_attention(q, k, v, row.contiguous(), return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    a = ets.topk_sparse_attention_backward(dout, q, k, v, row, out, lse)[0]
    b = ets.topk_sparse_attention_backward(dout, q, k, v, row.contiguous(), out, lse)[0]
    assert torch.equal(a, b)


def test_outputs_that_overlap_themselves_are_refused(ets):  # noqa: F811
    """An expanded tensor as output would be written by many rows."""
    pos, freqs = torch.arange(4, dtype=torch.int32, device=DEV), ets.rope_freqs(64)
    x = _rand((4, 8, 64), torch.bfloat16)
    for out in (x[:1].expand(4, -1, -1), x[:, :1].expand(-1, 8, -1)):
        out = out.to(x.dtype)
        assert 0 in out.stride()
        with pytest.raises(ValueError, match="overlap"):
            ets.topk_rope(x, pos, freqs, out=out)
        with pytest.raises(ValueError, match="overlap"):
            ets.topk_qk_norm_rope(x, x, None, None, pos, freqs, q_out=out)
