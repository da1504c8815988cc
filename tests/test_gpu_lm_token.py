"""zo_token_logprobs and zo_group_loss against 64-bit references (bounds: lm_ref)."""
import math

import pytest
import torch

import forward_only_amd as zo
import lm_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = zo.zo_init(5)
    yield c
    c.close()


def _logits(rows, vocab, dtype, seed, std=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g) * std).to(dtype)


def _check(ctx, x, targets, top_k, xd=None):
    xd = x.cuda() if xd is None else xd
    td = None if targets is None else targets.cuda()
    got = zo.zo_token_logprobs(ctx, xd, td, top_k=top_k)
    torch.cuda.synchronize()
    logp, entropy, ids, top = ref.token(x, targets, top_k)
    E = ref.token_bound(x.shape[1])
    m = x.double().max(dim=1, keepdim=True).values
    mag = (x.double() - m).nan_to_num(0.0, 0.0, 0.0)
    if targets is not None:
        at = targets.clamp(0, x.shape[1] - 1)
        b = E + ref.U32 * (mag.gather(1, at[:, None])[:, 0].abs() + logp.abs().nan_to_num(0, 0, 0))
        ref.assert_close(got.logp, logp, b, "logp")
    else:
        assert got.logp is None
    ref.assert_close(got.entropy, entropy, E * (1 + 2 * 13), "entropy")
    if top_k:
        assert torch.equal(got.top_ids.cpu(), ids)
        ref.assert_close(got.top_logp, top, E + ref.U32 * 2 * top.abs().nan_to_num(0, 0, 0) + 1e-30,
                         "top_logp")
    else:
        assert got.top_ids is None and got.top_logp is None
    again = zo.zo_token_logprobs(ctx, xd, td, top_k=top_k)
    for a, b in zip(got, again):
        assert a is None or torch.equal(a.view(torch.int32 if a.dtype == torch.float32 else a.dtype),
                                        b.view(torch.int32 if b.dtype == torch.float32 else b.dtype))
    return got


SIZES = [(1, 1), (3, 2), (5, 7), (2, 63), (4, 64), (3, 65), (2, 255), (2, 257), (7, 1000),
         (3, 2047), (2, 2049), (3, 4099), (2, 8191), (2, 16385), (3, 50272), (1, 131077)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_matches_reference(ctx, rows, vocab, dtype):
    x = _logits(rows, vocab, dtype, rows * 7 + vocab)
    g = torch.Generator().manual_seed(vocab)
    t = torch.randint(0, vocab, (rows,), generator=g)
    for k in sorted({0, 1, min(5, vocab), min(32, vocab)}):
        _check(ctx, x, t, k)


@pytest.mark.parametrize("rows", [1, 255, 256, 257, 700, 2100])
def test_row_counts(ctx, rows):
    x = _logits(rows, 1003, torch.bfloat16, rows)
    t = torch.arange(rows) * 17 % 1003
    t[::3] = zo.ZO_IGNORE_TOKEN
    _check(ctx, x, t, 4)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_without_targets_and_ignored(ctx, dtype):
    x = _logits(9, 777, dtype, 3)
    _check(ctx, x, None, 6)
    t = torch.full((9,), zo.ZO_IGNORE_TOKEN)
    got = _check(ctx, x, t, 6)
    assert (got.logp == 0).all() and (got.top_ids == -1).all()
    # an ignored row is not read: NaN there stays there
    x[4] = math.nan
    t[5] = 3
    _check(ctx, x, t, 2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("start,pad", [(0, 1), (1, 0), (3, 5), (8, 8), (7, 1)])
def test_strides_and_unaligned_rows(ctx, dtype, start, pad):
    rows, vocab = 6, 1001
    big = _logits(rows, vocab + start + pad, dtype, start * 10 + pad)
    view = big.cuda()[:, start:start + vocab]
    x = big[:, start:start + vocab].contiguous()
    t = torch.arange(rows) * 100
    _check(ctx, x, t, 5, xd=view)
    _check(ctx, x[1:], t[1:], 5, xd=view[1:])
    _check(ctx, x[::2].contiguous(), t[::2].contiguous(), 3, xd=view[::2])
    one = x[2:3].expand(4, vocab)
    _check(ctx, one.contiguous(), t[:4], 3, xd=view[2:3].expand(4, vocab))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [33, 4099])
def test_masks_infinities_nan_and_ties(ctx, dtype, vocab):
    low = torch.finfo(dtype).min
    x = _logits(16, vocab, dtype, vocab)
    x[0, 5:] = -math.inf                   # few survive
    x[1, :] = -math.inf                    # nothing survives
    x[2, 3:] = low                         # masked by the type's lowest value
    x[3, :] = low                          # every value the lowest
    x[4, 7] = math.nan
    x[5, 9] = math.inf
    x[6, :] = 1.5                          # all equal
    x[7, 1::2] = x[7, 0]                   # many ties
    x[8, :-1] = -math.inf                  # a single value
    x[9, 0] = torch.finfo(dtype).max       # differences overflow to -inf
    x[9, 1] = low
    x[10, 4] = 0.0                         # -0 and +0 are equal
    x[10, 2] = -0.0
    x[10, :][x[10] > 0] = -1.0
    x[11, 3] = -math.nan
    x[11, 1] = math.nan
    x[12, 6] = math.inf
    x[12, 2] = math.inf
    x[13, :] = torch.linspace(4, -4, vocab).to(dtype)      # sorted: the best in one place
    x[14, :] = torch.linspace(-4, 4, vocab).to(dtype)
    x[15, ::8] = 3.0
    t = torch.tensor([2, 0, 1, 4, 7, 9, 3, 1, vocab - 1, 1, 2, 1, 6, 0, vocab - 1, 8])
    for k in (1, 8, 32):
        _check(ctx, x, t, k)
    _check(ctx, x, None, 16)


@pytest.mark.parametrize("vocab", [5000, 50272])
def test_alternatives_in_adversarial_orders(ctx, vocab):
    """The best values close together, in every stride and block that a thread may own."""
    x = torch.zeros(12, vocab)
    base = torch.arange(vocab, dtype=torch.float32)
    x[0] = base % 256                       # each residue of 256 holds equal values
    x[1] = -(base % 256)
    x[2] = base // 2048
    x[3] = -(base // 2048)
    x[4] = (base % 8) * 10 + base / vocab
    x[5] = torch.where(base % 256 == 17, base / vocab + 5, -base / vocab)
    x[6] = torch.where((base // 8) % 256 == 3, base / vocab + 5, -base / vocab)
    x[7] = torch.where((base // 4) % 256 == 255, 9 - base / vocab, -base / vocab)
    x[8] = torch.where((base // 8) % 1024 == 1000, 9 - base / vocab, -base / vocab)
    x[9, -40:] = 1.0
    x[10, :40] = 1.0
    x[11] = base.remainder(997) * base.remainder(31)
    for dtype in (torch.float32, torch.bfloat16):
        for k in (1, 20, 32):
            _check(ctx, x.to(dtype), None, k)


def test_targets_out_of_range(ctx):
    x = _logits(6, 50, torch.float32, 1)
    t = torch.tensor([50, -1, -101, 2 ** 40, -2 ** 62, 49])
    got = _check(ctx, x, t, 2)
    assert torch.isnan(got.logp[:5]).all() and torch.isfinite(got.logp[5])


def test_refusals(ctx):
    x = torch.zeros(4, 10, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        zo.zo_token_logprobs(ctx, x, t, top_k=33)
    with pytest.raises(zo.ZOError):
        zo.zo_token_logprobs(ctx, x, t, top_k=11)          # more than the vocabulary
    with pytest.raises(TypeError):
        zo.zo_token_logprobs(ctx, x.half(), t)
    with pytest.raises(TypeError):
        zo.zo_token_logprobs(ctx, x, t.int())
    with pytest.raises(ValueError):
        zo.zo_token_logprobs(ctx, x, t[:3])
    with pytest.raises(ValueError):
        zo.zo_token_logprobs(ctx, x.t(), t)                # columns apart
    with pytest.raises(ValueError):
        zo.zo_token_logprobs(ctx, x[0], t)
    with pytest.raises(ValueError):
        zo.zo_token_logprobs(ctx, x.cpu(), t)
    with pytest.raises(zo.ZOError):
        zo.zo_token_logprobs(ctx, x[:, :0], t)
    with pytest.raises(ValueError):
        zo.zo_group_loss(ctx, x[:, 0].contiguous(), t[:2], t)
    L, h = zo._lib.lib(), ctx.handle
    p, q = x.data_ptr(), t.data_ptr()
    EINVAL, EUNSUP = zo.ZO_EINVAL, zo.ZO_EUNSUPPORTED
    assert L.zo_token_logprobs(h, p, 7, 4, 10, 10, q, p, p, 0, None, None, None) == EINVAL
    assert L.zo_token_logprobs(h, p, 0, 1 << 31, 10, 10, q, p, p, 0, None, None, None) == EUNSUP
    assert L.zo_token_logprobs(h, p, 0, 4, 1 << 31, 10, q, p, p, 0, None, None, None) == EUNSUP
    assert L.zo_token_logprobs(h, p + 2, 0, 4, 10, 10, q, p, p, 0, None, None, None) == EINVAL
    assert L.zo_token_logprobs(h, p, 0, 4, 10, 10, q + 4, p, p, 0, None, None, None) == EINVAL
    assert L.zo_token_logprobs(h, p, 0, 4, 10, 10, q, None, p, 0, None, None, None) == EINVAL
    assert L.zo_token_logprobs(h, p, 0, 4, 10, 10, None, p, p, 0, None, None, None) == EINVAL
    assert L.zo_token_logprobs(h, p, 0, 4, 10, 10, q, p, p, 2, None, p, None) == EINVAL
    assert L.zo_token_logprobs(h, p, 0, 4, 10, 1 << 63, q, p, p, 0, None, None, None) == EINVAL
    assert L.zo_group_loss(h, p, q, None, 2, 4, p, None) == EINVAL
    assert L.zo_group_loss(h, p, q, q, 1 << 31, 4, p, None) == EUNSUP
    # empty calls
    assert L.zo_token_logprobs(h, None, 0, 0, 10, 10, None, None, None, 0, None, None, None) == 0
    assert L.zo_group_loss(h, None, None, None, 0, 0, None, None) == 0
    e = zo.zo_token_logprobs(ctx, x[:0], t[:0], top_k=3)
    assert e.logp.numel() == 0 and e.top_ids.shape == (0, 3)


def _group_ref(logp, targets, starts):
    out = []
    for g in range(len(starts) - 1):
        lo, hi = int(starts[g]), int(starts[g + 1])
        p = logp[lo:hi].double()
        if targets is not None:
            p = p[targets[lo:hi] != zo.ZO_IGNORE_TOKEN]
        out.append(-p.sum().item() / p.numel() if p.numel() else math.nan)
    return torch.tensor(out, dtype=torch.float64)


@pytest.mark.parametrize("lengths", [[1], [0, 1, 0], [5, 0, 300, 1, 64], [256, 257, 255],
                                     [70000, 3], [2] * 700])
@pytest.mark.parametrize("given", [True, False])
def test_group_loss(ctx, lengths, given):
    rows = sum(lengths) + 5                     # rows behind the last group
    g = torch.Generator().manual_seed(rows)
    logp = -torch.rand(rows, generator=g) * 7
    targets = None
    if given:
        targets = torch.randint(0, 100, (rows,), generator=g)
        targets[torch.rand(rows, generator=g) < 0.4] = zo.ZO_IGNORE_TOKEN
    starts = torch.tensor([0] + lengths).cumsum(0)
    got = zo.zo_group_loss(ctx, logp.cuda(), None if targets is None else targets.cuda(),
                           starts.cuda()).cpu()
    want = _group_ref(logp, targets, starts)
    # fp64 sums of n fp32 values of one sign: n 2^-53 relative, both sides
    ref.assert_close(got, want, 2 * max(lengths) * 2.0 ** -53 * want.abs().nan_to_num(1) + 1e-18,
                     "loss")


def test_group_loss_takes_any_starts_and_values(ctx):
    logp = -torch.arange(1.0, 11.0)
    logp[3] = math.nan
    logp[8] = -math.inf
    starts = torch.tensor([-5, 2, 4, 4, 8, 2 ** 60, -2 ** 60, 3])
    got = zo.zo_group_loss(ctx, logp.cuda(), None, starts.cuda()).cpu()
    assert got[0] == 1.5 and math.isnan(got[1]) and math.isnan(got[2])
    assert got[3] == 6.5 and got[4] == math.inf
    assert math.isnan(got[5]) and got[6] == 2.0          # rows [10, 0) and [0, 3)


def test_streams_and_replayed_graph(ctx):
    x = [_logits(70, 5003, torch.bfloat16, s).cuda() for s in (1, 2)]
    t = (torch.arange(70) * 31 % 5003).cuda()
    starts = torch.tensor([0, 30, 70]).cuda()

    def both(a):
        r = zo.zo_token_logprobs(ctx, a, t, top_k=4)
        return list(r) + [zo.zo_group_loss(ctx, r.logp, t, starts)]

    want = [both(a) for a in x]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = zo.zo_token_logprobs(ctx, x[0], t, top_k=4, stream=side)
    side.synchronize()
    for a, b in zip(got, want[0]):
        assert torch.equal(a, b)
    buf = x[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(buf)
    for i in (0, 1, 0, 1):
        buf.copy_(x[i])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b)
        both(x[1 - i])


@pytest.mark.parametrize("rows", [2, 600])
@pytest.mark.parametrize("vocab", [40, 700, 2100, 4095, 16383, 16384, 20000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_most_alternatives_at_every_workgroup_size(ctx, rows, vocab, dtype):
    """32 alternatives where the row is short for its workgroup, with ties and masked values."""
    x = _logits(rows, vocab, dtype, vocab + rows, std=1.0)
    x[0, :] = -math.inf
    x[0, 3:30:2] = 1.0                       # fewer allowed than asked for
    x[1] = torch.round(x[1].float()).to(dtype)
    _check(ctx, x, None, 32)
    _check(ctx, x, torch.arange(rows) % 32 * 0 + 3, 7)


def test_stream_of_another_device_is_refused(ctx):
    class Other:
        device = torch.device("cuda", torch.cuda.current_device() + 1)
        cuda_stream = 0
    x = torch.zeros(2, 64, device="cuda")
    with pytest.raises(ValueError):
        zo.zo_token_logprobs(ctx, x, None, stream=Other())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [1e3, -1e3, 1e6, -1e6, 2.0 ** 20 - 4, 4 - 2.0 ** 20, -2.0 ** 20 - 90, -3e6, 1e9,
                                   -1e9, 1e30, -1e30, 3e38, -3e38])
def test_rows_far_from_zero(ctx, dtype, shift):
    """Logits around a large value, and some there beside ordinary ones."""
    vocab = 2085
    x = (_logits(9, vocab, torch.float32, 11) + shift).to(dtype)
    x[3, 700:] = _logits(1, vocab - 700, dtype, 12)[0]          # whole threads in either range
    x[4, ::2] = _logits(1, vocab, dtype, 13)[0, ::2]
    x[5, :] = shift
    x[6, 1:] = -math.inf
    x[7, 40:] = torch.finfo(dtype).min
    x[8, 900] = math.nan
    _check(ctx, x, torch.tensor([0, 1, 2, 3, 4, 5, 0, 7, 8]), 0)
    _check(ctx, x[:6], torch.tensor([vocab - 1, 699, 700, 701, 5, 9]), 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(6, 1), (6, 7), (6, 32), (6, 33), (6, 700), (6, 20011), (520, 33000)])
def test_nan_at_the_first_index(ctx, dtype, rows, vocab):
    """NaN ranks above all values wherever it stands: first of the row, all of it, beside +inf;
    up to as many alternatives as the row has values, at every workgroup size."""
    x = _logits(rows, vocab, dtype, vocab)
    x[0, 0] = math.nan
    x[1, :] = math.nan
    x[2, 0] = -math.nan
    x[2, vocab - 1] = math.inf
    x[3, 0] = math.inf
    x[3, vocab // 2] = math.nan
    x[4, ::2] = math.nan
    t = torch.arange(rows) % vocab
    for k in sorted({1, min(2, vocab), min(32, vocab)}):
        got = _check(ctx, x, t, k)
        assert int(got.top_ids.min()) >= 0 and int(got.top_ids.max()) < vocab
        assert torch.isnan(got.top_logp[:5]).all()


def test_stream_of_another_device_is_refused_with_all_outputs_given(ctx):
    class Other:
        device = torch.device("cuda", torch.cuda.current_device() + 1)
        cuda_stream = 0
    x, w = torch.zeros(2, 64, device="cuda"), torch.zeros(64, 64, device="cuda")
    t, starts = torch.zeros(2, dtype=torch.int64, device="cuda"), torch.tensor([0, 2], device="cuda")
    ids = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    rows, y, loss = torch.zeros(2, device="cuda"), x.clone(), torch.zeros(1, dtype=torch.float64, device="cuda")
    for call in (lambda **k: zo.zo_token_logprobs(ctx, x, t, out=zo.TokenLogprobs(rows, rows.clone(), None, None), **k),
                 lambda **k: zo.zo_head_logprobs(ctx, x, w, t, out=zo.HeadLogprobs(rows, rows.clone()), workspace=ws, **k),
                 lambda **k: zo.zo_group_loss(ctx, rows, t, starts, out=loss, **k),
                 lambda **k: zo.zo_adapter_project(ctx, x, w, x[:0], 0, starts, ids, out=y, workspace=ws, **k)):
        with pytest.raises(ValueError):
            call(stream=Other())
        torch.cuda.synchronize()
        call(stream=torch.cuda.Stream())
        torch.cuda.synchronize()
