"""The language-model operators where byte and element offsets pass 32 bits: far rows, far
adapters and their signs, weights beyond 4 GiB.  Most of each buffer is zero, so that the
references stay small."""
import math

import pytest
import torch

import forward_only_amd as zo
import lm_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def ctx():
    c = zo.zo_init(17)
    yield c
    c.close()
    torch.cuda.empty_cache()


def _rand(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF)


def _far_rows(x, reach):
    """A copy of x whose rows are spread over `reach` elements."""
    rows, cols = x.shape
    stride = reach // rows // 8 * 8
    view = torch.zeros(rows * stride, dtype=x.dtype, device="cuda").view(rows, stride)[:, :cols]
    view.copy_(x)
    return view


# few, middling and many rows; the last on tiles of 256 x 256
@pytest.mark.parametrize("rows,d_in,d_out", [(20, 256, 72), (50, 256, 72), (90, 256, 72), (700, 4104, 5000)])
def test_far_rows(ctx, rows, d_in, d_out):
    x, w, ad = _rand(1, rows, d_in), _rand(2, d_out, d_in, std=0.05), _rand(3, 16 * (d_in + d_out), std=0.1)
    starts, ids = torch.tensor([0, rows]).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    want = zo.zo_adapter_project(ctx, x, w, ad, 16, starts, ids)
    reach = (1 << 31) + (1 << 28)           # elements: 4.8 GB
    out = _far_rows(torch.zeros(rows, d_out, dtype=BF, device="cuda"), reach)
    got = zo.zo_adapter_project(ctx, _far_rows(x, reach), w, ad, 16, starts, ids, out=out)
    assert torch.equal(got, want)
    head = _rand(4, 999, d_in, std=0.1)
    t = torch.arange(rows, device="cuda") % 999
    t[::5] = zo.ZO_IGNORE_TOKEN
    a, b = (zo.zo_head_logprobs(ctx, v, head, t) for v in (x, _far_rows(x, reach)))
    assert torch.equal(a.logp, b.logp) and torch.equal(a.entropy, b.entropy)
    a, b = (zo.zo_token_logprobs(ctx, v, t % d_in, top_k=5) for v in (x, _far_rows(x, reach)))
    for p, q in zip(a, b):
        assert torch.equal(p, q)


@pytest.mark.parametrize("lengths", [[3, 4], [40, 60]])
def test_far_adapters_and_signs(ctx, lengths):
    d_in, d_out, rank = 64, 64, 8
    per = rank * (d_in + d_out)
    n = (1 << 32) // per + 3                # parameters pass 2^32
    ad = torch.zeros(n * per, dtype=BF, device="cuda")
    one = _rand(5, per, std=0.1)
    ad[-per:] = one
    x, w = _rand(6, sum(lengths), d_in), _rand(7, d_out, d_in, std=0.05)
    starts = torch.tensor([0] + lengths).cumsum(0).cuda()
    probes = torch.tensor([0, -1], dtype=torch.int32).cuda()
    al = torch.tensor([1e-2, 0.0]).cuda()
    ids = torch.full((2,), n - 1, dtype=torch.int32).cuda()
    got = zo.zo_adapter_project(ctx, x, w, ad, rank, starts, ids, probes=probes, alphas=al, step=1,
                                n_probes=1)
    # the same adapter alone in a buffer that begins at its global index
    zero = torch.zeros(2, dtype=torch.int32).cuda()
    assert (n - 1) * per % 128 == 0
    want = zo.zo_adapter_project(ctx, x, w, one, rank, starts, zero, probes=probes, alphas=al, step=1,
                                 n_probes=1, offset=(n - 1) * per)
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows", [4, 200])
def test_weights_beyond_4_gib(ctx, rows):
    vocab, d, live = 1_100_000, 2056, 1000  # 4.5 GB; all but the last rows give the logit 0
    w = torch.zeros(vocab, d, dtype=BF, device="cuda")
    w[-live:] = _rand(8, live, d, std=0.2)
    h = _rand(9, rows, d)
    t = vocab - 1 - torch.arange(rows, device="cuda") % live
    got = zo.zo_head_logprobs(ctx, h, w, t)
    x = h.double() @ w[-live:].double().t().contiguous()
    m = x.max(dim=1, keepdim=True).values.clamp(min=0.0)
    e = torch.exp(x - m)
    s = e.sum(dim=1) + (vocab - live) * torch.exp(-m[:, 0])
    mean = ((e * (x - m)).sum(dim=1) - (vocab - live) * m[:, 0] * torch.exp(-m[:, 0])) / s
    logp = (x.gather(1, (t - vocab + live)[:, None])[:, 0] - m[:, 0]) - torch.log(s)
    off = 8 * math.sqrt(d) * ref.U32 * (torch.linalg.vector_norm(h.double(), dim=1)
                                        * torch.linalg.vector_norm(w[-live:].double(), dim=1).max())
    E = ref.token_bound(vocab)
    spread = m[:, 0] - x.min(dim=1).values.clamp(max=0.0)
    ref.assert_close(got.logp, logp, 2 * off + E + 2 * ref.U32 * spread, "logp")
    # |t / s| <= log V + 1 < 15 here
    ref.assert_close(got.entropy, torch.log(s) - mean, 32 * off + 31 * E, "entropy")


def test_more_rows_and_groups_than_one_launch_holds(ctx):
    # 2^31 threads a launch: 2^25 rows of one wave each, 2^23 groups of 256 threads
    rows, vocab = (1 << 25) + 5, 2
    x = torch.zeros(rows, vocab, dtype=BF, device="cuda")
    x[-9:, 1] = 1.0
    t = torch.ones(rows, dtype=torch.int64, device="cuda")
    t[1 << 25] = zo.ZO_IGNORE_TOKEN
    got = zo.zo_token_logprobs(ctx, x, t, top_k=1)
    for p, q in zip(got, zo.zo_token_logprobs(ctx, x[-9:], t[-9:], top_k=1)):
        assert torch.equal(p[-9:], q)
    # two equal logits: -log 2, one fp32 logarithm
    assert (got.logp[:-9] - math.log(0.5)).abs().max().item() <= 1e-6
    assert not got.top_ids[:-9].any()
    groups = (1 << 23) + 3
    starts = torch.arange(groups + 1, device="cuda") * 3
    loss = zo.zo_group_loss(ctx, got.logp[:3 * groups], t[:3 * groups], starts)
    want = got.logp[:3 * groups].double().view(groups, 3).sum(dim=1) / -3.0
    # sums of three equal fp32 values are exact in fp64
    assert torch.allclose(loss, want, rtol=4 * torch.finfo(torch.float64).eps, atol=0.0)


def test_sizes_beyond_a_launch_are_refused(ctx):
    L, h = zo._lib.lib(), ctx.handle
    p = torch.zeros(64, device="cuda").data_ptr()
    UNSUP = zo.ZO_EUNSUPPORTED

    def head(rows, d, vocab):
        return L.zo_head_logprobs(h, p, d, p, 1, rows, d, vocab, p, p, p, p, 1 << 62, None)

    def project(rows, d_in, d_out, groups):
        return L.zo_adapter_project(h, p, d_in, p, None, 1, rows, d_in, d_out, p, 1, 8, 1.0, p, p, groups,
                                    None, None, 0, 0, 0, 0, None, p, 1 << 62, p, d_out, None)

    assert head(1, 8, (1 << 24) + 8) == UNSUP and head(1, (1 << 26) + 8, 8) == UNSUP
    assert head((1 << 31) - 1, 64, 8) == UNSUP      # 256 GiB of hidden states
    assert project((1 << 25) + 1, 8, 8, 1) == UNSUP and project(1, 8, 8, (1 << 22) + 1) == UNSUP
    assert project(1, (1 << 26) + 8, 8, 1) == UNSUP and project(1, 8, (1 << 24) + 8, 1) == UNSUP
    assert project(1 << 25, 8, 1032, 1) == UNSUP


def test_probe_rows_past_64_bits_are_refused(ctx):
    # 2^31 probes of 2^33 bytes each: 2^64, which is 0 in 64 bits
    L, h = zo._lib.lib(), ctx.handle
    p = torch.zeros(64, device="cuda").data_ptr()
    assert zo.zo_bits_stride(1 << 36) == 1 << 33
    assert L.zo_adapter_project(h, p, 1016, p, None, 1, 1, 1016, 8, p, 1 << 23, 8, 1.0, p, p, 1, p, p,
                                0, 0, 0, 1 << 31, None, p, 1 << 40, p, 8, None) == zo.ZO_EINVAL


def test_large_grids(ctx):
    """As many groups as one call takes, most of them empty, and many rows of few features."""
    groups, rows, d = 1 << 22, 5000, 64
    x, w, ad = _rand(1, rows, d), _rand(2, d, d, std=0.1), _rand(3, 8 * 2 * d, std=0.1)
    starts = torch.zeros(groups + 1, dtype=torch.int64, device="cuda")
    starts[groups // 2 + 1:] = rows
    ids = torch.full((groups,), -1, dtype=torch.int32, device="cuda")
    ids[groups // 2] = 0
    got = zo.zo_adapter_project(ctx, x, w, ad, 8, starts, ids)
    one = torch.tensor([0, rows], device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(got, zo.zo_adapter_project(ctx, x, w, ad, 8, *one))
    rows = 1 << 22
    far = torch.zeros(rows, 8, dtype=BF, device="cuda")
    far[-700:] = _rand(4, 700, 8)
    w, ad = _rand(5, 8, 8), _rand(6, 8 * 16)
    starts = torch.tensor([0, rows], device="cuda")
    got = zo.zo_adapter_project(ctx, far, w, ad, 8, starts, one[1])
    assert torch.equal(got[-700:], zo.zo_adapter_project(ctx, far[-700:], w, ad, 8,
                                                         torch.tensor([0, 700], device="cuda"), one[1]))
    assert not got[:-700].any()
