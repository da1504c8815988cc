"""zo_distill_loss against its 64-bit definition (bounds: lm_more_ref)."""
import math

import pytest
import torch

import forward_only_amd as zo
import lm_more_ref as more
import lm_ref as ref

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ctx():
    c = zo.zo_init(3)
    yield c
    c.close()


def _case(rows, vocab, k, dtype, seed=0, std=2.5, pad=0):
    g = torch.Generator().manual_seed(seed + 7 * rows + vocab)
    x = (torch.randn(rows, vocab + pad, generator=g) * std).to(dtype)[:, :vocab]
    ids = torch.stack([torch.randperm(vocab, generator=g)[:k] if k <= vocab else
                       torch.randint(0, vocab, (k,), generator=g) for _ in range(rows)]) if rows else \
        torch.zeros(0, k, dtype=torch.int64)
    return x, ids.view(rows, k), torch.randn(rows, k, generator=g) * 2, torch.rand(rows, generator=g) + 0.5


def _on(x, shift=0):
    """x on the GPU with its row stride, its first element `shift` elements into an allocation."""
    if not x.shape[0]:
        return x.cuda()
    stride = x.stride(0) if x.shape[0] > 1 else x.shape[1]
    whole = torch.zeros(x.shape[0] * stride + shift + 16, dtype=x.dtype, device="cuda")
    view = whole[shift:shift + x.shape[0] * stride].view(x.shape[0], stride)[:, :x.shape[1]]
    view.copy_(x)
    return view


def _check(ctx, x, ids, t, w, targets=None, T=1.0, shift=0, out=None):
    want, grad, lb, gb = more.distill(x, ids, t, targets, T)
    dx = _on(x, shift)
    tc = None if targets is None else targets.cuda()
    got = zo.zo_distill_loss(ctx, dx, ids.cuda(), t.cuda(), targets=tc, temperature=T, grad=out is None,
                             row_grad=w.cuda(), out=out)
    torch.cuda.synchronize()
    ref.assert_close(got.loss, want, lb + ref.U32 * want.abs() + 1e-30, "loss")
    g = w.double()[:, None]
    half = ref.UBF if x.dtype == BF else ref.U32
    ref.assert_close(got.grad, g * grad, g.abs() * gb * 1.01 + (half + 4 * ref.U32) * (g * grad).abs() + 1e-38, "grad")
    alone = zo.zo_distill_loss(ctx, dx, ids.cuda(), t.cuda(), targets=tc, temperature=T)
    assert alone.grad is None
    ref.assert_close(alone.loss, want, lb + ref.U32 * want.abs() + 1e-30, "loss alone")
    return got, dx


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (1, 7, 3), (3, 64, 1), (5, 1000, 20), (2, 50272, 32),
                                          (4, 32003, 5), (7, 16387, 128), (2, 70001, 64), (2, 140009, 8),
                                          (1, 300000, 4), (260, 257, 2), (0, 40, 3)])
def test_matches_reference(ctx, rows, vocab, k, dtype):
    x, ids, t, w = _case(rows, vocab, k, dtype)
    _check(ctx, x, ids, t, w)
    _check(ctx, x, ids, t, -w, T=2.5)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shift", [1, 3, 5, 7])
@pytest.mark.parametrize("vocab,pad", [(1003, 2), (9, 0), (50001, 5)])
def test_any_alignment_and_stride(ctx, vocab, pad, shift, dtype):
    x, ids, t, w = _case(3, vocab, 4, dtype, pad=pad)
    _check(ctx, x, ids, t, w, T=0.5, shift=shift)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_that_count_for_nothing(ctx, dtype):
    x, ids, t, w = _case(8, 501, 5, dtype, seed=1)
    targets = torch.zeros(8, dtype=torch.int64)
    targets[2] = ref.IGNORE
    x[2] = math.nan
    t[2] = math.nan
    ids[3] = -1                         # no entries
    x[3] = math.inf
    ids[4, 2:] = -1                     # fewer entries
    t[4, 2:] = math.nan
    targets[5] = 10 ** 12               # any other target counts
    _check(ctx, x, ids, t, w, targets=targets)
    none = zo.zo_distill_loss(ctx, x.cuda(), torch.zeros(8, 0, dtype=torch.int64, device="cuda"),
                              torch.zeros(8, 0, device="cuda"), grad=True)
    assert not none.loss.any() and not none.grad.float().any()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("vocab", [300, 40000])
def test_masks_and_values_out_of_range(ctx, dtype, vocab):
    x, ids, t, w = _case(12, vocab, 4, dtype, seed=2)
    low = torch.finfo(dtype).min
    x[0, ::2] = -math.inf
    ids[0] = torch.tensor([1, 3, 5, 7])
    x[1, ::2] = low                     # the type's lowest value is a number
    ids[1] = torch.tensor([1, 3, 5, 7])
    x[2, 8:] = -math.inf
    ids[2] = torch.tensor([1, 2, 9, 3])  # an entry where the model has no probability
    t[3, 1] = -math.inf                 # a share of 0, one of them masked by the model
    x[3, ids[3, 1]] = -math.inf
    x[4] = -math.inf
    x[5, 17] = math.inf
    x[6, 18] = math.nan
    t[7] = -math.inf
    t[8, 0] = math.inf
    t[9, 2] = math.nan
    ids[10, 1] = vocab
    ids[11, 3] = -2
    got, _ = _check(ctx, x, ids, t, w)
    assert math.isinf(float(got.loss[2])) and torch.isfinite(got.grad[2]).all()
    assert torch.isfinite(got.loss[:2]).all() and torch.isfinite(got.loss[3])
    for r in range(4, 12):
        assert torch.isnan(got.loss[r]) and torch.isnan(got.grad[r]).all(), r


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("vocab", [100, 33000])
def test_an_id_that_comes_twice_has_both_shares(ctx, dtype, vocab):
    x, ids, t, w = _case(4, vocab, 70, dtype, seed=3)
    ids[0] = 5
    ids[1, ::2] = 0
    ids[2, 1:] = vocab - 1
    _check(ctx, x, ids, t, w)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("vocab,pad", [(640, 0), (50272, 0), (1003, 5), (300000, 0)])
def test_gradient_in_the_logits_place(ctx, dtype, vocab, pad):
    x, ids, t, w = _case(3, vocab, 6, dtype, seed=4, pad=pad)
    apart = zo.zo_distill_loss(ctx, _on(x), ids.cuda(), t.cuda(), grad=True, row_grad=w.cuda())
    place = _on(x)
    got = zo.zo_distill_loss(ctx, place, ids.cuda(), t.cuda(), row_grad=w.cuda(),
                             out=zo.DistillLoss(torch.empty(3, device="cuda"), place))
    assert torch.equal(got.loss, apart.loss) and torch.equal(place, apart.grad)


def test_gradient_against_differences(ctx):
    """Central differences of the loss itself, in 64 bits, along random directions."""
    x, ids, t, w = _case(6, 203, 5, F32, seed=5)
    got = zo.zo_distill_loss(ctx, x.cuda(), ids.cuda(), t.cuda(), temperature=2.0, grad=True, row_grad=w.cuda())
    g = torch.Generator().manual_seed(1)
    for _ in range(4):
        d, h = torch.randn(6, 203, generator=g).double(), 1e-5
        up = (w.double() * more.distill(x.double() + h * d, ids, t, None, 2.0)[0]).sum()
        down = (w.double() * more.distill(x.double() - h * d, ids, t, None, 2.0)[0]).sum()
        # 64-bit differences: truncation h^2, cancellation 1e-16 / h; the gradient's own error 1e-6
        assert abs(float((up - down) / (2 * h) - (got.grad.double().cpu() * d).sum())) < 1e-4


def test_teacher_from_token_alternatives(ctx):
    """A teacher's alternatives, ignored rows included, are the entries; a model that is its own
    teacher over the whole vocabulary loses nothing."""
    x, _, _, _ = _case(9, 32, 1, F32, seed=6)
    targets = torch.arange(9)
    targets[4] = ref.IGNORE
    top = zo.zo_token_logprobs(ctx, x.cuda(), targets.cuda(), top_k=32)
    got = zo.zo_distill_loss(ctx, x.cuda(), top.top_ids, top.top_logp, grad=True)
    # sums of 32 shares: |log p - log q| is at most a few roundings of values below 32
    assert float(got.loss.abs().max()) < 1e-5 and float(got.grad.abs().max()) < 1e-6
    assert float(got.loss[4]) == 0.0


def test_streams_and_replayed_graph(ctx):
    x, ids, t, w = _case(5, 5003, 7, BF, seed=7)
    d = [v.cuda() for v in (x, ids, t, w)]
    eager = zo.zo_distill_loss(ctx, d[0], d[1], d[2], grad=True, row_grad=d[3])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = zo.zo_distill_loss(ctx, d[0], d[1], d[2], grad=True, row_grad=d[3], stream=side)
    side.synchronize()
    assert torch.equal(other.loss, eager.loss) and torch.equal(other.grad, eager.grad)
    out = zo.DistillLoss(torch.empty(5, device="cuda"), torch.empty_like(d[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zo.zo_distill_loss(ctx, d[0], d[1], d[2], row_grad=d[3], out=out)
    for seed in range(3):
        d[0].copy_(_case(5, 5003, 7, BF, seed=20 + seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        eager = zo.zo_distill_loss(ctx, d[0], d[1], d[2], grad=True, row_grad=d[3])
        assert torch.equal(out.loss, eager.loss) and torch.equal(out.grad, eager.grad)


def test_rows_behind_the_last_are_left(ctx):
    x, ids, t, _ = _case(3, 1001, 4, BF, seed=8)
    whole = torch.full((5, 1010), 7.0, dtype=BF, device="cuda")
    loss = torch.full((5,), 7.0, device="cuda")
    zo.zo_distill_loss(ctx, x.cuda(), ids.cuda(), t.cuda(), out=zo.DistillLoss(loss[:3], whole[:3, 3:1004]))
    assert (whole[3:] == 7).all() and (whole[:, :3] == 7).all() and (whole[:, 1004:] == 7).all()
    assert (loss[3:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T", [2e-6, 0.01, 100.0, 1e6])
def test_temperatures(ctx, dtype, T):
    """A gradient's terms at any temperature; losses of a high one are roundings times T^2."""
    x, ids, t, w = _case(5, 600, 5, dtype, seed=9)
    _check(ctx, x, ids, t, w, T=float(torch.tensor(T)))


def test_more_rows_than_a_launch_holds(ctx):
    """Rows past 2^25, of 64 threads each, and past 2^32 bytes of the teacher's entries; the same 4096 again and
    again."""
    n, vocab, k, rows = 4096, 8, 16, (1 << 25) + 4096
    x, ids, t, w = _case(n, vocab, k, BF, seed=10)
    want, grad, lb, gb = more.distill(x, ids, t, None, 1.0)
    many = lambda v: v.cuda().repeat(rows // n, *([1] * (v.dim() - 1)))  # noqa: E731
    got = zo.zo_distill_loss(ctx, many(x), many(ids), many(t), grad=True, row_grad=many(w))
    g = w.double()[:, None]
    ref.assert_close(got.loss[-n:], want, lb + ref.U32 * want.abs() + 1e-30, "loss")
    ref.assert_close(got.grad[-n:], g * grad, g.abs() * gb * 1.01 + (ref.UBF + 4 * ref.U32) * (g * grad).abs() + 1e-38, "grad")
    assert torch.equal(got.loss.view(-1, n), got.loss[:n].expand(rows // n, n))
    assert torch.equal(got.grad.view(-1, n * vocab), got.grad[:n].reshape(1, -1).expand(rows // n, n * vocab))


def test_rows_past_32_bits_of_offsets(ctx):
    """Rows 2^31 elements apart, read and written past 2^32 bytes and elements."""
    x, ids, t, w = _case(3, 1003, 4, BF, seed=11)
    stride = (1 << 31) + 16
    whole = torch.empty(2 * stride + 1003, dtype=BF, device="cuda")
    place = whole.as_strided((3, 1003), (stride, 1))
    place.copy_(x)
    apart = zo.zo_distill_loss(ctx, x.cuda(), ids.cuda(), t.cuda(), grad=True, row_grad=w.cuda())
    got = zo.zo_distill_loss(ctx, place, ids.cuda(), t.cuda(), row_grad=w.cuda(),
                             out=zo.DistillLoss(torch.empty(3, device="cuda"), place))
    assert torch.equal(got.loss, apart.loss) and torch.equal(place, apart.grad)


def test_refusals(ctx):
    x, ids, t, w = (v.cuda() for v in _case(3, 40, 4, F32))
    call = lambda **kw: zo.zo_distill_loss(ctx, kw.pop("x", x), kw.pop("ids", ids), kw.pop("t", t), **kw)  # noqa: E731
    for bad in (0.0, -1.0, math.nan, math.inf, 1e-7, 1.1e6):
        with pytest.raises(ValueError):
            call(temperature=bad)
    with pytest.raises(ValueError):
        call(ids=ids[:2])
    with pytest.raises(ValueError):
        call(row_grad=w)
    with pytest.raises(ValueError):
        call(ids=torch.zeros(3, 129, dtype=torch.int64, device="cuda"), t=torch.zeros(3, 129, device="cuda"))
    with pytest.raises(TypeError):
        call(ids=ids.int())
    with pytest.raises(TypeError):
        call(x=x.half())
    with pytest.raises(ValueError):
        call(x=x.t())
    whole = torch.zeros(3, 80, device="cuda")
    with pytest.raises(zo.ZOError):      # within the logits, but not in their place
        call(x=whole[:, :40], out=zo.DistillLoss(torch.empty(3, device="cuda"), whole[:, 8:48]))
    with pytest.raises(zo.ZOError):
        call(x=torch.zeros(3, 0, device="cuda"))
