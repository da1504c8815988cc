"""zo_adapter_project and zo_head_logprobs at the sizes where the products run on tiles of
256 x 256: whole rounds of tiles, a rest cut along k, ragged edges; and sizes drawn at random
across the shapes.  References in 64 bits on the GPU (bounds: lm_ref)."""
import math
import random

import pytest
import torch

import forward_only_amd as zo
import lm_ref as ref

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ctx():
    c = zo.zo_init(13)
    yield c
    c.close()


def _rand(gen, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _project(ctx, lengths, d_in, d_out, rank, dtype, seed, probes=0, lead=0, tail=0):
    gen = _gen(seed)
    rows = lead + sum(lengths) + tail
    adapters, G = 3, len(lengths)
    x, w = _rand(gen, rows, d_in, dtype=dtype), _rand(gen, d_out, d_in, std=0.05, dtype=dtype)
    bias = _rand(gen, d_out, dtype=dtype)
    ad = _rand(gen, adapters * rank * (d_in + d_out), std=0.1, dtype=dtype)
    starts = torch.tensor([lead] + list(lengths)).cumsum(0)
    ids = torch.tensor([g % (adapters + 1) - 1 for g in range(G)], dtype=torch.int32)
    kw, extra = {}, {}
    if probes:
        which = torch.tensor([g % (probes + 1) - 1 for g in range(G)], dtype=torch.int32)
        al = torch.tensor([1e-2 * (-1) ** g for g in range(G)])
        bits = zo.zo_gen_probes(ctx, 1, 0, probes, 0, ad.numel())
        kw = {"probes": which.cuda(), "alphas": al.cuda(), "bits": bits}
        extra = {"probes": which, "alphas": al, "z": ref.signs(bits.cpu(), ad.numel()).cuda()}
    out = torch.full((rows, d_out), 5.0, dtype=dtype, device="cuda")
    got = zo.zo_adapter_project(ctx, x, w, ad, rank, starts.cuda(), ids.cuda(), scale=-1.5, bias=bias,
                                out=out, **kw)
    y, low, sums = ref.project(x, w, bias, ad, rank, starts, ids, -1.5, **extra)
    inside = slice(lead, lead + sum(lengths))
    half = ref.UBF if dtype == BF else ref.U32
    bound = half * y[inside].abs() + (2.0 ** -15 + 128 * ref.U32) * low[inside] + sums[inside] * 1.01
    ref.assert_close(got[inside], y[inside], bound, "y")
    assert (out[:lead] == 5).all() and (out[lead + sum(lengths):] == 5).all()
    again = zo.zo_adapter_project(ctx, x, w, ad, rank, starts.cuda(), ids.cuda(), scale=-1.5, bias=bias,
                                  **kw)
    assert torch.equal(again[inside], got[inside])


# (lengths, d_in, d_out): tiles of 256 x 256 -- a rest of 60 in four slices; 180, none sliced;
# 265, whole and sliced; one row of tiles with a ragged end; many short groups across tiles
LARGE = [([200, 1, 400, 99], 4104, 5000), ([1100], 136, 9000), ([555, 300, 245], 1032, 13504),
         ([37] * 30, 2056, 8008), ([1] * 300 + [500], 4104, 6152), ([130, 0, 126], 5120, 20480)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lengths,d_in,d_out", LARGE)
@pytest.mark.parametrize("rank,probes", [(16, 0), (40, 2)])
def test_project_on_large_tiles(ctx, lengths, d_in, d_out, rank, probes, dtype):
    _project(ctx, lengths, d_in, d_out, rank, dtype, sum(lengths) + d_out, probes, lead=3, tail=5)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d_in,d_out", [(4104, 5000), (136, 9000)])
def test_values_of_one_group_stay_in_it_on_large_tiles(ctx, dtype, d_in, d_out):
    gen = _gen(5)
    lengths, rank = [300, 333, 467], 16
    rows = sum(lengths)
    x, w = _rand(gen, rows, d_in, dtype=dtype), _rand(gen, d_out, d_in, std=0.05, dtype=dtype)
    per = rank * (d_in + d_out)
    ad = _rand(gen, 3 * per, std=0.1, dtype=dtype)
    starts = torch.tensor([0] + lengths).cumsum(0).cuda()
    ids = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    clean = zo.zo_adapter_project(ctx, x, w, ad, rank, starts, ids)
    ad[per + 3] = math.nan
    ad[per + rank * d_in + 5] = math.inf
    x[700, 7] = math.nan
    got = zo.zo_adapter_project(ctx, x, w, ad, rank, starts, ids)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[300:633] = False
    keep[700] = False
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[300:633]).all() and torch.isnan(got[700]).all()
    ids[1] = 3
    got = zo.zo_adapter_project(ctx, x, w, ad, rank, starts, ids)
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[300:633]).all()


def _head(ctx, rows, d, vocab, dtype, ignore, seed):
    gen = _gen(seed)
    h, w = _rand(gen, rows, d, dtype=dtype), _rand(gen, vocab, d, std=3 / math.sqrt(d), dtype=dtype)
    t = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    t[torch.rand(rows, generator=gen, device="cuda") < ignore] = zo.ZO_IGNORE_TOKEN
    got = zo.zo_head_logprobs(ctx, h, w, t)
    x = h.double() @ w.double().t().contiguous()
    m, logs, ts = ref.log_stats(x)
    skip = t == zo.ZO_IGNORE_TOKEN
    logp = ((x.gather(1, t.clamp(min=0)[:, None])[:, 0] - m) - logs).masked_fill(skip, 0)
    entropy = (logs - ts).masked_fill(skip, 0)
    e = 8 * math.sqrt(d) * ref.U32 * (torch.linalg.vector_norm(h.double(), dim=1)
                                      * torch.linalg.vector_norm(w.double(), dim=1).max())
    E = ref.token_bound(vocab)
    spread = x.max(dim=1).values - x.min(dim=1).values
    ref.assert_close(got.logp, logp, 2 * e + E + 2 * ref.U32 * spread, "logp")
    ref.assert_close(got.entropy, entropy, 28 * e + 27 * E, "entropy")
    only = zo.zo_head_logprobs(ctx, h, w, None)
    assert only.logp is None
    ref.assert_close(only.entropy, logs - ts, 28 * e + 27 * E, "entropy of all")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,d,vocab", [(700, 4104, 5003), (1100, 136, 9001), (1100, 1032, 13501),
                                          (2500, 520, 8000), (260, 5120, 20001)])
@pytest.mark.parametrize("ignore", [0.0, 0.7])
def test_head_on_large_tiles(ctx, rows, d, vocab, dtype, ignore):
    _head(ctx, rows, d, vocab, dtype, ignore, rows + vocab)


@pytest.mark.parametrize("seed", range(16))
def test_drawn_sizes(ctx, seed):
    rng = random.Random(seed)

    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    dtype = rng.choice([F32, BF])
    rows = size(1, 3000)
    cut = sorted(rng.randint(0, rows) for _ in range(rng.choice([0, 1, 5, 60])))
    lengths = [b - a for a, b in zip([0] + cut, cut + [rows])]
    print(f"[drawn] {seed}: {dtype} {lengths[:8]} ...", flush=True)
    _project(ctx, lengths, 8 * size(1, 400), 8 * size(1, 1200), rng.choice([8, 16, 24, 64, 128]), dtype,
             seed, probes=rng.choice([0, 0, 3]), lead=rng.choice([0, 7]), tail=rng.choice([0, 9]))
    _head(ctx, size(1, 2500), 8 * size(1, 300), size(1, 9000), dtype, rng.choice([0.0, 0.5]), seed)


def test_two_streams_at_once_and_graphs_on_large_tiles(ctx):
    gen = _gen(3)
    lengths = [200, 1, 400, 99]
    xs = [_rand(gen, 700, 4104, dtype=BF) for _ in range(2)]
    w, head = _rand(gen, 5000, 4104, std=0.05, dtype=BF), _rand(gen, 6001, 5000, std=0.01, dtype=BF)
    ad = _rand(gen, 2 * 16 * 9104, std=0.1, dtype=BF)
    starts = torch.tensor([0] + lengths).cumsum(0).cuda()
    ids = torch.tensor([0, 1, -1, 1], dtype=torch.int32).cuda()
    t = torch.randint(0, 6001, (700,), generator=gen, device="cuda")
    t[::3] = zo.ZO_IGNORE_TOKEN

    def both(x, stream=None):
        y = zo.zo_adapter_project(ctx, x, w, ad, 16, starts, ids, stream=stream)
        r = zo.zo_head_logprobs(ctx, y, head, t, stream=stream)
        return [y, r.logp, r.entropy, zo.zo_group_loss(ctx, r.logp, t, starts, stream=stream)]

    def same(a, b):
        return all(torch.equal(torch.nan_to_num(p, 9.0), torch.nan_to_num(q, 9.0)) for p, q in zip(a, b))

    want = [both(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [both(x, s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        assert same(got[0], want[0]) and same(got[1], want[1])
    bufs = [x.clone() for x in xs]
    graphs, outs = [], []
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both(b))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert same(outs[0], want[0]) and same(outs[1], want[1])
        both(xs[0])
    bufs[0].copy_(xs[1])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert same(outs[0], want[1])


# up to 16 and 32 rows beside many features, ragged, the last two beyond the 256 MB that the
# last cache holds
WIDE = [([16], 72, 16400), ([17], 72, 16384), ([9, 1, 14], 136, 16424), ([32], 264, 20000),
        ([3, 2], 4104, 33000), ([20, 0, 7], 4104, 33000)]


# 33 to 64 rows: all of them in a workgroup up to 8192 features
WIDE += [([33], 72, 40), ([5, 0, 43], 136, 8192), ([48], 1032, 8184), ([40, 9], 776, 72), ([1] * 64, 520, 8192),
         ([64], 16400, 8192), ([30, 33], 264, 8200), ([65], 264, 8192)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lengths,d_in,d_out", WIDE)
def test_few_rows_and_many_features(ctx, lengths, d_in, d_out, dtype):
    _project(ctx, lengths, d_in, d_out, 24, dtype, sum(lengths) + d_out, probes=2)
    _head(ctx, sum(lengths), d_in, d_out + 3, dtype, 0.2, d_out)


def test_logits_beyond_the_last_cache(ctx):
    """More than 256 MB: rows as short as one wave takes, and longer, equal to parts' results."""
    for rows, vocab in ((70001, 2003), (11000, 13001)):
        x = torch.randn(rows, vocab, generator=_gen(rows), device="cuda").mul_(3).to(BF)
        t = torch.arange(rows, device="cuda") % vocab
        t[::7] = zo.ZO_IGNORE_TOKEN
        got = zo.zo_token_logprobs(ctx, x, t)
        for r0 in range(0, rows, rows // 3):
            part = slice(r0, r0 + rows // 3)
            want = zo.zo_token_logprobs(ctx, x[part], t[part])
            assert torch.equal(got.logp[part], want.logp) and torch.equal(got.entropy[part], want.entropy)


# tiles of 64 x 64 that many short groups meet: a row each, empty ones between, a long one last
SHORT = [([1] * 70, 296, 240), ([1, 0, 2, 0, 0, 3] * 12 + [40], 136, 1000), ([5] * 30, 520, 264),
         ([0] * 300 + [1] * 40 + [0] * 70 + [90], 72, 72), ([1] * 100, 1032, 4104)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lengths,d_in,d_out", SHORT)
@pytest.mark.parametrize("rank,probes", [(8, 0), (64, 2)])
def test_short_groups(ctx, lengths, d_in, d_out, rank, probes, dtype):
    _project(ctx, lengths, d_in, d_out, rank, dtype, sum(lengths) + d_out, probes, lead=2, tail=3)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("most,d_in,d_out", [(300, 5120, 5120), (1100, 136, 9000), (40, 264, 20000)])
def test_one_workspace_for_the_largest_batch(ctx, dtype, most, d_in, d_out):
    """Fewer rows in the largest batch's workspace, which holds old values, as in their own."""
    gen = _gen(most)
    x, w = _rand(gen, most, d_in, dtype=dtype), _rand(gen, d_out, d_in, std=0.05, dtype=dtype)
    ad = _rand(gen, 2 * 16 * (d_in + d_out), std=0.1, dtype=dtype)
    t = torch.randint(0, d_out, (most,), generator=gen, device="cuda")
    t[::5] = zo.ZO_IGNORE_TOKEN
    ids, probes = torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([1, -1], dtype=torch.int32).cuda()
    kw = dict(probes=probes, alphas=torch.tensor([1e-2, 0.0]).cuda(), step=3, n_probes=2)
    project = torch.full((zo.zo_adapter_workspace_bytes(most, d_in, d_out, 2, 16, 2, 2),), 255,
                         dtype=torch.uint8, device="cuda")
    head = torch.full((zo.zo_head_workspace_bytes(most, d_in, d_out),), 255, dtype=torch.uint8, device="cuda")
    for rows in (most, 260, 257, 256, 129, 65, 64, 33, 32, 17, 16, 5):
        if rows > most:
            continue
        starts = torch.tensor([0, rows // 3, rows], device="cuda")
        a = zo.zo_adapter_project(ctx, x[:rows], w, ad, 16, starts, ids, workspace=project, **kw)
        b = zo.zo_adapter_project(ctx, x[:rows], w, ad, 16, starts, ids, **kw)
        assert torch.equal(a, b), rows
        a = zo.zo_head_logprobs(ctx, x[:rows], w, t[:rows], workspace=head)
        b = zo.zo_head_logprobs(ctx, x[:rows], w, t[:rows])
        assert torch.equal(a.logp, b.logp) and torch.equal(a.entropy, b.entropy), rows
