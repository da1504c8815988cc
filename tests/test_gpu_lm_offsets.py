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
@pytest.mark.parametrize("rows,d_in,d_out", [(20, 256, 72), (50, 256, 72), (700, 4104, 5000)])
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
