"""zo_adapter_project and zo_head_logprobs against 64-bit references (bounds: lm_ref)."""
import math

import pytest
import torch

import forward_only_amd as zo
import lm_ref as ref
from forward_only_amd.step import spsa_step_fused

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ctx():
    c = zo.zo_init(9)
    yield c
    c.close()


def _rand(gen, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=gen) * std).to(dtype)


def _problem(lengths, d_in, d_out, rank, adapters, dtype, seed=0, tail=0):
    gen = torch.Generator().manual_seed(seed + d_in + 3 * d_out)
    rows = sum(lengths) + tail
    p = {"x": _rand(gen, rows, d_in, dtype=dtype), "w": _rand(gen, d_out, d_in, std=0.05, dtype=dtype),
         "bias": _rand(gen, d_out, dtype=dtype),
         "ad": _rand(gen, adapters * rank * (d_in + d_out), std=0.1, dtype=dtype),
         "starts": torch.tensor([0] + list(lengths)).cumsum(0),
         "ids": torch.randint(-1, adapters, (len(lengths),), generator=gen, dtype=torch.int32)}
    return p


def _y_bound(y, low, sums, dtype):
    # one rounding to the type; the low-rank factor's 16 leading bits (2^-16) and fp32 sums of
    # at most 128 terms
    half = ref.UBF if dtype == BF else ref.U32
    return half * y.abs().nan_to_num(0) + (2.0 ** -15 + 128 * ref.U32) * low + sums * 1.01 + 1e-30


def _check(ctx, p, rank, scale=0.5, bias=True, dtype=F32, probes=None, alphas=None, bits=None, out=None,
           x=None):
    d = {k: v.cuda() for k, v in p.items()}
    kw = {}
    z = None
    if probes is not None:
        kw = {"probes": probes.cuda(), "alphas": alphas.cuda(), "bits": bits.cuda()}
        z = ref.signs(bits, p["ad"].numel())
    got = zo.zo_adapter_project(ctx, d["x"] if x is None else x, d["w"], d["ad"], rank, d["starts"],
                                d["ids"], scale=scale, bias=d["bias"] if bias else None, out=out, **kw)
    torch.cuda.synchronize()
    y, low, sums = ref.project(p["x"], p["w"], p["bias"] if bias else None, p["ad"], rank,
                               p["starts"], p["ids"], scale, probes, alphas, z)
    inside = ~torch.isnan(y[:, 0])
    ref.assert_close(got.cpu()[inside], y[inside], _y_bound(y, low, sums, dtype)[inside], "y")
    again = zo.zo_adapter_project(ctx, d["x"] if x is None else x, d["w"], d["ad"], rank, d["starts"],
                                  d["ids"], scale=scale, bias=d["bias"] if bias else None, **kw)
    assert torch.equal(again[inside.cuda()], got[inside.cuda()])         # deterministic
    return got


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lengths,d_in,d_out,rank,adapters", [
    ([1], 8, 8, 8, 1), ([1, 1, 1], 64, 72, 8, 2), ([3, 0, 5], 40, 16, 16, 3),
    ([17, 16, 15, 1], 136, 264, 24, 2), ([64], 256, 128, 32, 1), ([1] * 40, 96, 328, 8, 7),
    ([130, 70, 1, 0, 55], 72, 136, 40, 3), ([300], 520, 264, 64, 2), ([5, 9], 1032, 40, 128, 2),
    ([100, 33, 180], 768, 520, 16, 2), ([2] * 130, 64, 64, 8, 130), ([1000, 24], 200, 392, 8, 2),
    ([7], 5120, 1288, 16, 1), ([2] * 20, 2048, 640, 56, 9)])
def test_project_matches_reference(ctx, lengths, d_in, d_out, rank, adapters, dtype):
    p = _problem(lengths, d_in, d_out, rank, adapters, dtype)
    _check(ctx, p, rank, dtype=dtype)
    _check(ctx, p, rank, scale=-2.0, bias=False, dtype=dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 48, 64, 65, 100, 128, 129, 255, 257, 513, 777])
def test_project_row_counts(ctx, rows, dtype):
    lengths = [rows // 3, rows - rows // 3 - rows // 5, rows // 5]
    p = _problem(lengths, 264, 272, 16, 2, dtype, seed=rows)
    _check(ctx, p, 16, dtype=dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lengths", [[4, 0, 9, 1, 30], [1] * 9, [70, 200, 3]])
def test_probes_equal_perturb_in_place(ctx, lengths, dtype):
    """Stored rows, regenerated rows and adapters moved by zo_perturb give the same bits."""
    rank, adapters, d_in, d_out, offset, step, probe0 = 16, 2, 136, 72, 1280, 3, 5
    p = _problem(lengths, d_in, d_out, rank, adapters, dtype, seed=1)
    n = p["ad"].numel()
    G = len(lengths)
    probes = torch.tensor([(g % 4) - 1 for g in range(G)], dtype=torch.int32)
    alphas = torch.tensor([1e-3 * (-1) ** g * (1 + g) for g in range(G)])
    bits = zo.zo_gen_probes(ctx, step, probe0, 3, offset, n).cpu()
    got = _check(ctx, p, rank, dtype=dtype, probes=probes, alphas=alphas, bits=bits)
    d = {k: v.cuda() for k, v in p.items()}
    regen = zo.zo_adapter_project(ctx, d["x"], d["w"], d["ad"], rank, d["starts"], d["ids"], scale=0.5,
                                  bias=d["bias"], probes=probes.cuda(), alphas=alphas.cuda(),
                                  offset=offset, step=step, probe0=probe0, n_probes=3)
    assert torch.equal(got, regen)
    for g in range(G):
        th = d["ad"].clone()
        if probes[g] >= 0:
            zo.zo_perturb(ctx, th, offset, step, probe0 + int(probes[g]), float(alphas[g]))
        one = zo.zo_adapter_project(ctx, d["x"], d["w"], th, rank, d["starts"], d["ids"], scale=0.5,
                                    bias=d["bias"])
        lo, hi = int(p["starts"][g]), int(p["starts"][g + 1])
        assert torch.equal(one[lo:hi], got[lo:hi]), g


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows", [20, 200])
def test_rows_of_no_group_and_bad_indices(ctx, dtype, rows):
    rank, d_in, d_out = 8, 72, 136
    p = _problem([rows], d_in, d_out, rank, 3, dtype, seed=2, tail=9)
    n = rows // 10
    p["starts"] = torch.tensor([2, 2 + n, 2 + 2 * n, 2 + 3 * n, 2 + 4 * n, 2 + 5 * n])
    p["ids"] = torch.tensor([0, 3, -1, -2, 2], dtype=torch.int32)        # two outside the table
    d = {k: v.cuda() for k, v in p.items()}
    out = torch.full((rows + 9, d_out), 7.0, dtype=dtype, device="cuda")
    zo.zo_adapter_project(ctx, d["x"], d["w"], d["ad"], rank, d["starts"], d["ids"], out=out)
    s = p["starts"]
    assert (out[:2] == 7).all() and (out[int(s[5]):] == 7).all()
    assert torch.isnan(out[int(s[1]):int(s[2])]).all() and torch.isnan(out[int(s[3]):int(s[4])]).all()
    good = p["ids"].clone()
    good[1] = good[3] = -1
    y, low, sums = ref.project(p["x"], p["w"], None, p["ad"], rank, s, good, 1.0)
    for g in (0, 2, 4):
        r = slice(int(s[g]), int(s[g + 1]))
        ref.assert_close(out[r].cpu(), y[r], _y_bound(y, low, sums, dtype)[r], f"group {g}")
    # probes outside the table
    probes = torch.tensor([0, 1, -2, 0, 2], dtype=torch.int32).cuda()
    ids = torch.tensor([0, 0, 0, 1, 1], dtype=torch.int32).cuda()
    al = torch.full((5,), 1e-3, device="cuda")
    out = zo.zo_adapter_project(ctx, d["x"], d["w"], d["ad"], rank, d["starts"], ids, probes=probes,
                                alphas=al, n_probes=2)
    nan = [bool(torch.isnan(out[int(s[g]):int(s[g + 1])]).any()) for g in range(5)]
    assert nan == [False, False, True, False, True]
    # starts out of range and out of order stay inside the buffers
    for bad in ([-5, 3, 2 ** 60, 2 ** 61, 2 ** 62, 2 ** 62], [90, 3, 50, 1, 0, -7], [5, 5, 5, 5, 5, 5]):
        zo.zo_adapter_project(ctx, d["x"], d["w"], d["ad"], rank, torch.tensor(bad).cuda(), ids,
                              probes=probes, alphas=al, n_probes=2)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows", [12, 150])
def test_values_of_one_group_stay_in_it(ctx, dtype, rows):
    """NaN and infinities in one adapter or one row reach that group or row alone."""
    rank, d_in, d_out = 16, 64, 80
    p = _problem([rows // 3] * 3, d_in, d_out, rank, 3, dtype, seed=4)
    p["ids"] = torch.tensor([0, 1, 2], dtype=torch.int32)
    per = rank * (d_in + d_out)
    n = rows // 3
    clean = _check(ctx, p, rank, dtype=dtype)
    bad = dict(p, ad=p["ad"].clone(), x=p["x"].clone())
    bad["ad"][per + 3] = math.nan                      # A of adapter 1
    bad["ad"][per + rank * d_in + 5] = math.inf        # B of adapter 1
    bad["x"][2 * n + 1, 7] = math.nan
    d = {k: v.cuda() for k, v in bad.items()}
    got = zo.zo_adapter_project(ctx, d["x"], d["w"], d["ad"], rank, d["starts"], d["ids"], scale=0.5,
                                bias=d["bias"])
    keep = torch.ones(3 * n, dtype=torch.bool)
    keep[n:2 * n] = False
    keep[2 * n + 1] = False
    assert torch.equal(got.cpu()[keep], clean.cpu()[keep])
    assert torch.isnan(got[2 * n + 1]).all() and torch.isnan(got[n:2 * n]).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_project_strides_and_no_adapters(ctx, dtype):
    p = _problem([30, 41], 72, 88, 8, 2, dtype, seed=6)
    wide = torch.full((71, 120), math.nan, dtype=dtype, device="cuda")
    wide[:, 16:88] = p["x"].cuda()
    out = torch.full((71, 104), 3.0, dtype=dtype, device="cuda")
    if dtype == F32:
        x = wide[:, 16:88]
    else:
        x = wide[:, 16:88]
    got = _check(ctx, p, 8, dtype=dtype, x=x, out=out[:, 8:96])
    assert got.data_ptr() == out[:, 8:96].data_ptr()
    assert (out[:, :8] == 3).all() and (out[:, 96:] == 3).all()
    none = dict(p, ids=torch.full((2,), -1, dtype=torch.int32))
    base = _check(ctx, none, 8, dtype=dtype)
    d = {k: v.cuda() for k, v in p.items()}
    empty = zo.zo_adapter_project(ctx, d["x"], d["w"], d["ad"][:0], 0, d["starts"],
                                  none["ids"].cuda(), bias=d["bias"])
    assert torch.equal(base, empty)
    z = zo.zo_adapter_project(ctx, d["x"][:0], d["w"], d["ad"], 8, torch.zeros(1, dtype=torch.int64).cuda(),
                              d["ids"][:0])
    assert z.shape == (0, 88)


def test_project_refusals(ctx):
    p = {k: v.cuda() for k, v in _problem([4, 4], 64, 64, 8, 2, F32).items()}

    def call(**kw):
        a = dict(x=p["x"], weight=p["w"], adapters=p["ad"], rank=8, starts=p["starts"], ids=p["ids"])
        a.update(kw)
        return zo.zo_adapter_project(ctx, **a)

    call()
    with pytest.raises(TypeError):
        call(x=p["x"].half())
    with pytest.raises(TypeError):
        call(weight=p["w"].to(BF))
    with pytest.raises(ValueError):
        call(weight=p["w"][:, :32])
    with pytest.raises(ValueError):
        call(adapters=p["ad"][:-8])
    with pytest.raises(ValueError):
        call(ids=p["ids"][:1])
    with pytest.raises(TypeError):
        call(starts=p["starts"].int())
    with pytest.raises(ValueError):
        call(probes=p["ids"])
    with pytest.raises(ValueError):
        call(probes=p["ids"], alphas=torch.ones(2, device="cuda"))       # how many?
    with pytest.raises(ValueError):
        call(out=torch.empty(8, 72, device="cuda"))
    with pytest.raises(zo.ZOError):
        call(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(zo.ZOError):
        call(probes=p["ids"], alphas=torch.ones(2, device="cuda"), n_probes=2, offset=64)
    with pytest.raises(zo.ZOError):
        call(probes=p["ids"], alphas=torch.ones(2, device="cuda"), n_probes=2, probe0=2 ** 32 - 1)
    with pytest.raises(zo.ZOError):            # widths are multiples of 8
        zo.zo_adapter_project(ctx, p["x"][:, :60].contiguous(), p["w"][:, :60].contiguous(), p["ad"][:0],
                              0, p["starts"], p["ids"])
    with pytest.raises(zo.ZOError):
        call(rank=4, adapters=p["ad"][:4 * 128])
    with pytest.raises(zo.ZOError):
        call(rank=136, adapters=torch.zeros(136 * 128, device="cuda"))
    with pytest.raises(zo.ZOError):            # rows 4 elements apart in 16 bytes
        call(x=torch.zeros(8, 68, device="cuda")[:, :64])
    h = zo.zo_init(1)
    h.close()
    with pytest.raises(ValueError):
        zo.zo_adapter_project(h, p["x"], p["w"], p["ad"], 8, p["starts"], p["ids"])


# ---- the head ---------------------------------------------------------------------------

def _head_check(ctx, hidden, weight, targets, hd=None):
    hd = hidden.cuda() if hd is None else hd
    wd, td = weight.cuda(), None if targets is None else targets.cuda()
    got = zo.zo_head_logprobs(ctx, hd, wd, td)
    x = (hd.double() @ wd.double().t()).cpu()
    logp, entropy, _, _ = ref.token(x, targets, 0)
    d, vocab = hidden.shape[1], weight.shape[0]
    # logits off by at most e each move log s and the mean of x by at most e, and p_v by 2 e
    # relative, so the entropy by at most 2 e + 2 e max|d| over the mass (<= 13)
    e = 8 * math.sqrt(d) * ref.U32 * (torch.linalg.vector_norm(hidden.double(), dim=1)
                                      * torch.linalg.vector_norm(weight.double(), dim=1).max())
    E = ref.token_bound(vocab)
    if targets is not None:
        spread = (x.max(dim=1).values - x.min(dim=1).values).nan_to_num(0)
        ref.assert_close(got.logp, logp, (2 * e + E + 2 * ref.U32 * spread).nan_to_num(0), "logp")
    ref.assert_close(got.entropy, entropy, (e * 28 + E * 27).nan_to_num(0), "entropy")
    again = zo.zo_head_logprobs(ctx, hd, wd, td)
    for a, b in zip(got, again):
        assert a is None or torch.equal(a.view(torch.int32), b.view(torch.int32))
    return got


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,d,vocab", [
    (1, 8, 1), (1, 64, 2), (2, 72, 31), (3, 40, 33), (16, 128, 257), (17, 136, 1000), (33, 768, 4099),
    (64, 256, 515), (65, 520, 129), (100, 1032, 700), (200, 64, 2051), (257, 96, 300),
    (4, 5120, 2053), (300, 2048, 1027), (520, 264, 640)])
def test_head_matches_reference(ctx, rows, d, vocab, dtype):
    gen = torch.Generator().manual_seed(rows + d + vocab)
    hidden = _rand(gen, rows, d, dtype=dtype)
    weight = _rand(gen, vocab, d, std=3 / math.sqrt(d), dtype=dtype)
    t = torch.randint(0, vocab, (rows,), generator=gen)
    _head_check(ctx, hidden, weight, t)
    t[torch.rand(rows, generator=gen) < 0.6] = zo.ZO_IGNORE_TOKEN
    if rows > 3:
        t[0], t[2] = vocab, -1                        # outside the vocabulary
    _head_check(ctx, hidden, weight, t)
    _head_check(ctx, hidden, weight, None)
    _head_check(ctx, hidden, weight, torch.full((rows,), zo.ZO_IGNORE_TOKEN))


def test_head_of_many_rows(ctx):
    """More rows than one launch's partial statistics hold, most of them ignored or none."""
    gen = torch.Generator().manual_seed(8)
    rows = 2 * 16384 + 70
    hidden, weight = _rand(gen, rows, 64, dtype=BF), _rand(gen, 45, 64, std=0.4, dtype=BF)
    t = torch.randint(0, 45, (rows,), generator=gen)
    _head_check(ctx, hidden, weight, t)
    t[torch.rand(rows, generator=gen) < 0.4] = zo.ZO_IGNORE_TOKEN
    _head_check(ctx, hidden, weight, t)
    t[:] = zo.ZO_IGNORE_TOKEN
    t[rows - 1] = 44
    t[3] = 0
    _head_check(ctx, hidden, weight, t)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows", [9, 130])
def test_head_strides_nan_and_infinite_logits(ctx, dtype, rows):
    gen = torch.Generator().manual_seed(3)
    big = _rand(gen, rows, 200, dtype=dtype)
    weight = _rand(gen, 333, 64, std=0.5, dtype=dtype)
    t = torch.arange(rows) * 5 % 333
    view = big.cuda()[:, 8:72]
    _head_check(ctx, big[:, 8:72].contiguous(), weight, t, hd=view)
    bad = big[:, 8:72].contiguous()
    bad[1, 3] = math.nan
    bad[4, 0] = math.inf
    got = zo.zo_head_logprobs(ctx, bad.cuda(), weight.cuda(), t.cuda())
    clean = zo.zo_head_logprobs(ctx, view, weight.cuda(), t.cuda())
    keep = torch.ones(rows, dtype=torch.bool)
    keep[1] = keep[4] = False
    assert torch.equal(got.logp.cpu()[keep], clean.logp.cpu()[keep])
    assert torch.isnan(got.logp.cpu()[~keep]).all() and torch.isnan(got.entropy.cpu()[~keep]).all()


def test_head_refusals(ctx):
    h, w = torch.zeros(4, 64, device="cuda"), torch.zeros(10, 64, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        zo.zo_head_logprobs(ctx, h, w.to(BF), t)
    with pytest.raises(ValueError):
        zo.zo_head_logprobs(ctx, h, w[:, :32].contiguous(), t)
    with pytest.raises(ValueError):
        zo.zo_head_logprobs(ctx, h, w[:, ::2], t)
    with pytest.raises(ValueError):
        zo.zo_head_logprobs(ctx, h, w, t[:2])
    with pytest.raises(zo.ZOError):
        zo.zo_head_logprobs(ctx, h, w, None, entropy=False)
    with pytest.raises(zo.ZOError):
        zo.zo_head_logprobs(ctx, h, w, t, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(zo.ZOError):
        zo.zo_head_logprobs(ctx, h[:, :60].contiguous(), w[:, :60].contiguous(), t)
    with pytest.raises(zo.ZOError):
        zo.zo_head_logprobs(ctx, torch.zeros(4, 70, device="cuda")[:, :64], w, t)
    with pytest.raises(zo.ZOError):
        zo.zo_head_logprobs(ctx, h, w[:0], t)
    assert zo.zo_head_logprobs(ctx, h[:0], w, t[:0]).logp.numel() == 0


# ---- together ---------------------------------------------------------------------------

def _losses(ctx, p, rank, head, targets, starts, n, offset, step):
    """loss_probes_at of spsa_step_fused: every probe's both signs and the clean pass as groups
    of one batch of 2 n + 1 copies."""
    def at(probe0, n, alpha, rows, plus, minus, clean):
        G = 2 * n + 1
        which = torch.tensor([g // 2 if g < 2 * n else -1 for g in range(G)], dtype=torch.int32).cuda()
        al = torch.tensor([(alpha if g % 2 == 0 else -alpha) if g < 2 * n else 0.0
                           for g in range(G)]).cuda()
        ids = torch.zeros(G, dtype=torch.int32).cuda()
        y = zo.zo_adapter_project(ctx, p["x"].repeat(G, 1), p["w"], p["ad"], rank, starts, ids, scale=2.0,
                                  bias=p["bias"], probes=which, alphas=al, offset=offset, step=step,
                                  probe0=probe0, n_probes=n, bits=rows)
        lp = zo.zo_head_logprobs(ctx, y, head, targets, entropy=False).logp
        loss = zo.zo_group_loss(ctx, lp, targets, starts)
        plus.copy_(loss[0:2 * n:2])
        minus.copy_(loss[1:2 * n:2])
        clean.copy_(loss[2 * n:])
    return at


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("mode", ["bits", "regen"])
def test_step_with_adapters(ctx, dtype, mode):
    rank, d_in, d_out, vocab, T, n, offset, step = 8, 128, 72, 301, 13, 4, 256, 2
    p = _problem([T], d_in, d_out, rank, 1, dtype, seed=11)
    gen = torch.Generator().manual_seed(12)
    head = _rand(gen, vocab, d_out, std=0.3, dtype=dtype).cuda()
    t1 = torch.randint(0, vocab, (T,), generator=gen)
    t1[:5] = zo.ZO_IGNORE_TOKEN
    G = 2 * n + 1
    targets = t1.repeat(G).cuda()
    starts = (torch.arange(G + 1) * T).cuda()
    d = {k: v.cuda() for k, v in p.items()}
    theta = d["ad"].clone()
    d["ad"] = theta
    eps, eta, delta = 2.0 ** -7, 1e-3, 1e-6
    bits = zo.zo_gen_probes(ctx, step, 0, n, offset, theta.numel()) if mode == "bits" else None
    before = theta.clone()
    res = spsa_step_fused(ctx, theta, step=step, npert=n, eps=eps, eta=eta, delta=delta, offset=offset,
                          bits=bits, loss_probes_at=_losses(ctx, d, rank, head, targets, starts, n,
                                                            offset, step), probes_give_clean=True)
    # every loss against a forward in 64 bits at the moved adapters
    z = ref.signs(zo.zo_gen_probes(ctx, step, 0, n, offset, theta.numel()).cpu(), theta.numel())

    def forward(alpha, i):
        th = before.cpu()
        if i >= 0:
            th = (th.float() + alpha * z[i]).to(dtype)
        y, _, _ = ref.project(p["x"], p["w"], p["bias"], th, rank, [0, T], [0], 2.0)
        logits = y.to(dtype).double() @ head.cpu().double().t()
        lp = torch.log_softmax(logits, dim=1).gather(1, t1.clamp(min=0)[:, None])[:, 0]
        return -lp[t1 != zo.ZO_IGNORE_TOKEN].mean().item()

    # y's roundings may differ in the last bit next to a border: a bf16 step of a few y of each
    # row moves a logit by at most 2^-7 |y| |w| each
    tol = 2e-2 if dtype == BF else 2e-5
    for i in range(n):
        assert abs(res["Lp"][i].item() - forward(eps, i)) < tol
        assert abs(res["Lm"][i].item() - forward(-eps, i)) < tol
    assert abs(res["L0"].item() - forward(0.0, -1)) < tol
    want = before.clone()
    zo.zo_update(ctx, want, offset, step, res["c"], eta, bits)
    assert torch.equal(want, theta) and not torch.equal(theta, before)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("mode", ["bits", "regen"])
@pytest.mark.parametrize("npert,per", [(5, 32), (5, 2), (1, 1), (0, 4)])
def test_spsa_step_adapters(ctx, dtype, mode, npert, per):
    """The step in batches of probes equals one forward per probe and sign at adapters that
    zo_perturb moved, then the weights and zo_update."""
    from forward_only_amd.step import spsa_step_adapters
    rank, d_in, d_out, vocab, T, offset, step = 16, 64, 72, 211, 9, 128, 4
    p = _problem([T], d_in, d_out, rank, 1, dtype, seed=21)
    gen = torch.Generator().manual_seed(22)
    head = _rand(gen, vocab, d_out, std=0.3, dtype=dtype).cuda()
    t = torch.randint(0, vocab, (T,), generator=gen)
    t[:4] = zo.ZO_IGNORE_TOKEN
    t = t.cuda()
    d = {k: v.cuda() for k, v in p.items()}
    theta = d["ad"].clone()
    eps, eta, delta = 2.0 ** -6, 1e-3, 1e-6
    bits = None
    if mode == "bits" and npert:
        bits = zo.zo_gen_probes(ctx, step, 0, npert, offset, theta.numel())

    def logp_of(groups):
        G = groups.ids.numel()
        y = zo.zo_adapter_project(ctx, d["x"].repeat(G, 1), d["w"], theta, rank, bias=d["bias"],
                                  **groups.of_project())
        return zo.zo_head_logprobs(ctx, y, head, t.repeat(G), entropy=False).logp

    res = spsa_step_adapters(ctx, theta, step=step, npert=npert, eps=eps, eta=eta, delta=delta,
                             logp_of=logp_of, targets=t, offset=offset, bits=bits, probes_per_batch=per)
    one = torch.tensor([0, T]).cuda()
    none = torch.zeros(1, dtype=torch.int32).cuda()

    def loss(th):
        y = zo.zo_adapter_project(ctx, d["x"], d["w"], th, rank, one, none, bias=d["bias"])
        lp = zo.zo_head_logprobs(ctx, y, head, t, entropy=False).logp
        return zo.zo_group_loss(ctx, lp, t, one).item()

    # the same products in tiles of another shape: sums in another order (fp32, relative 1e-6 of
    # the logits), and in bf16 now and then the next value of y (2^-8 of a term of a logit)
    tol = 3e-2 if dtype == BF else 2e-5
    assert abs(res["L0"].item() - loss(d["ad"])) < tol
    for i in range(npert):
        for a, got in ((eps, res["Lp"]), (-eps, res["Lm"])):
            th = d["ad"].clone()
            zo.zo_perturb(ctx, th, offset, step, i, a)
            assert abs(got[i].item() - loss(th)) < tol
    want = d["ad"].clone()
    c = zo.zo_probe_weights(ctx, res["Lp"], res["Lm"], res["L0"], eps, delta)
    assert torch.equal(c, res["c"])
    zo.zo_update(ctx, want, offset, step, c, eta, bits)
    assert torch.equal(want, theta)


def test_streams_and_replayed_graph(ctx):
    p = [{k: v.cuda() for k, v in _problem([30, 50, 1], 264, 136, 16, 2, BF, seed=s).items()} for s in (1, 2)]
    gen = torch.Generator().manual_seed(5)
    head = _rand(gen, 1003, 136, std=0.2, dtype=BF).cuda()
    t = torch.randint(0, 1003, (81,), generator=gen)
    t[::4] = zo.ZO_IGNORE_TOKEN
    t = t.cuda()
    probes = torch.tensor([0, 1, -1], dtype=torch.int32).cuda()
    al = torch.tensor([1e-2, -1e-2, 0.0]).cuda()

    def both(x, **kw):
        y = zo.zo_adapter_project(ctx, x, p[0]["w"], p[0]["ad"], 16, p[0]["starts"], p[0]["ids"],
                                  bias=p[0]["bias"], probes=probes, alphas=al, n_probes=2, **kw)
        r = zo.zo_head_logprobs(ctx, y, head, t, **kw)
        return [y, r.logp, r.entropy, zo.zo_group_loss(ctx, r.logp, t, p[0]["starts"], **kw)]

    want = [both(p[i]["x"]) for i in (0, 1)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = both(p[1]["x"], stream=side)
    side.synchronize()
    for a, b in zip(got, want[1]):
        assert torch.equal(torch.nan_to_num(a, 99.0), torch.nan_to_num(b, 99.0))
    buf = p[0]["x"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(buf)
    for i in (0, 1, 0, 1):
        buf.copy_(p[i]["x"])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[i]):
            assert torch.equal(torch.nan_to_num(a, 99.0), torch.nan_to_num(b, 99.0))
        both(p[1 - i]["x"])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("mode", ["bits", "regen"])
def test_step_with_adapters_captured_and_replayed(ctx, dtype, mode):
    """A whole step in two batches, captured once and replayed, equals the eager step each time."""
    from forward_only_amd.step import spsa_step_adapters
    rank, d_in, d_out, vocab, T, npert = 8, 64, 72, 131, 11, 5
    p = {k: v.cuda() for k, v in _problem([T], d_in, d_out, rank, 1, dtype, seed=31).items()}
    gen = torch.Generator().manual_seed(32)
    head = _rand(gen, vocab, d_out, std=0.3, dtype=dtype).cuda()
    t = torch.randint(0, vocab, (T,), generator=gen)
    t[::4] = zo.ZO_IGNORE_TOKEN
    t = t.cuda()
    theta = p["ad"].clone()
    bits = zo.zo_gen_probes(ctx, 2, 0, npert, 0, theta.numel()) if mode == "bits" else None

    def logp_of(groups):
        n = groups.ids.numel()
        y = zo.zo_adapter_project(ctx, p["x"].repeat(n, 1), p["w"], theta, rank, **groups.of_project())
        return zo.zo_head_logprobs(ctx, y, head, t.repeat(n), entropy=False).logp

    def step():
        return spsa_step_adapters(ctx, theta, step=2, npert=npert, eps=2.0 ** -7, eta=1e-2, delta=1e-6,
                                  logp_of=logp_of, targets=t, bits=bits, probes_per_batch=3)

    def eager(start):
        theta.copy_(start)
        r = step()
        return [theta.clone()] + [r[k].clone() for k in ("L0", "Lp", "Lm", "c")]

    starts = [p["ad"], (p["ad"].float() * 0.5).to(dtype)]
    want = [eager(s) for s in starts]
    assert not torch.equal(want[0][0], starts[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in (0, 1, 1, 0):
        theta.copy_(starts[i])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([theta] + [out[k] for k in ("L0", "Lp", "Lm", "c")], want[i]):
            assert torch.equal(a, b)
        eager(starts[1 - i])


# few rows; 64 x 64 tiles, group by group and row by row; 256 x 256 tiles, whole and in slices
@pytest.mark.parametrize("lengths,d_in,d_out", [([3, 4], 64, 72), ([30, 50, 1], 264, 136), ([1] * 90, 72, 264),
                                                ([1100], 136, 9000), ([400, 300], 4104, 5000)])
@pytest.mark.parametrize("rank", [8, 64, 128])
def test_fp32_adapter_product_keeps_32_bits(ctx, lengths, d_in, d_out, rank):
    """fp32 alone, without the bound of bf16's two parts: W is 0 and each row of x has one value,
    so that x W^T is exact and x A^T rounds once.  What is left of y = scale u B^T rounds twice a
    term (product and sum), once for u, scale and the result each, and once per eight terms where
    parts are added: (2 + 1/8) rank + 3 half steps of the terms' magnitudes."""
    gen = torch.Generator().manual_seed(rank + d_out)
    rows, adapters = sum(lengths), 2
    x = torch.zeros(rows, d_in)
    x[torch.arange(rows), torch.arange(rows) * 7 % d_in] = torch.randn(rows, generator=gen)
    w = torch.zeros(d_out, d_in)
    ad = torch.randn(adapters * rank * (d_in + d_out), generator=gen)
    starts = torch.tensor([0] + lengths).cumsum(0)
    ids = torch.arange(len(lengths), dtype=torch.int32) % adapters
    got = zo.zo_adapter_project(ctx, x.cuda(), w.cuda(), ad.cuda(), rank, starts.cuda(), ids.cuda(), scale=0.3)
    y, low, _ = ref.project(x, w, None, ad, rank, starts, ids, float(torch.tensor(0.3)))
    ref.assert_close(got, y, (2.125 * rank + 3) * ref.U32 * low + 1e-30, "y")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("mode", ["bits", "regen"])
def test_adapters_of_two_projections_in_one_buffer(ctx, dtype, mode):
    """Each projection takes its part of the flat buffer, of its indices and of stored rows; every
    group's rows equal those at the whole buffer moved by zo_perturb."""
    from forward_only_amd.step import adapter_probe_groups
    rank, d, wide, T, n, offset, step = 8, 72, 112, 7, 3, 256, 6
    gen = torch.Generator().manual_seed(41)
    x, w1, w2 = (_rand(gen, *s, std=0.2, dtype=dtype).cuda() for s in ((T, d), (wide, d), (d, wide)))
    per = rank * (d + wide)
    begin = (per + 127) // 128 * 128            # where the second adapter begins
    assert begin > per
    theta = _rand(gen, begin + per, std=0.1, dtype=dtype).cuda()
    bits = zo.zo_gen_probes(ctx, step, 0, n, offset, theta.numel()) if mode == "bits" else None
    groups = adapter_probe_groups(n, T, 2.0 ** -6, offset=offset, step=step, bits=bits)
    G = groups.ids.numel()

    def model(th, moved):
        y = x.repeat(G, 1)
        for w, a, b in ((w1, 0, per), (w2, begin, begin + per)):
            kw = {"starts": groups.starts, "ids": groups.ids}
            if moved:
                kw = groups.of_project()
                kw["offset"] += a
                if bits is not None:
                    kw["bits"] = bits[:, a // 8:][:, :zo.zo_bits_stride(b - a)].contiguous()
            y = zo.zo_adapter_project(ctx, y, w, th[a:b], rank, **kw)
        return y

    got = model(theta, True)
    for g in range(G):
        th = theta.clone()
        p = int(groups.probes[g])
        if p >= 0:
            zo.zo_perturb(ctx, th, offset, step, p, float(groups.alphas[g]))
        want = model(th, False)
        assert torch.equal(got[g * T:(g + 1) * T], want[g * T:(g + 1) * T]), g


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows,d,vocab", [(9, 64, 333), (60, 64, 8000), (130, 64, 333), (700, 4104, 5003)])
def test_head_whatever_ignored_rows_hold(ctx, rows, d, vocab, dtype):
    """Padding of NaN and infinities: zeros for it, and not a bit of the other rows moves."""
    gen = torch.Generator().manual_seed(rows)
    hidden = _rand(gen, rows, d, dtype=dtype).cuda()
    weight = _rand(gen, vocab, d, std=0.1, dtype=dtype).cuda()
    t = torch.arange(rows, device="cuda") % vocab
    skip = torch.arange(rows, device="cuda") % 3 != 1
    t[skip] = zo.ZO_IGNORE_TOKEN
    clean = zo.zo_head_logprobs(ctx, hidden, weight, t)
    hidden[skip] = math.nan
    hidden[0] = math.inf
    got = zo.zo_head_logprobs(ctx, hidden, weight, t)
    for a, b in zip(got, clean):
        assert torch.equal(a, b) and not a[skip].any() and torch.isfinite(a).all()
    t[:] = zo.ZO_IGNORE_TOKEN
    got = zo.zo_head_logprobs(ctx, hidden, weight, t)
    assert not got.logp.any() and not got.entropy.any()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rows", [20, 90, 700])
def test_one_row_read_as_many(ctx, rows, dtype):
    """Rows no elements apart: the same row for every group."""
    d_in, d_out = 4104, 5000
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, w, ad = (torch.randn(*s, generator=gen, device="cuda").mul(0.05).to(dtype)
                for s in ((1, d_in), (d_out, d_in), (2 * 16 * (d_in + d_out),)))
    starts = torch.tensor([0, rows // 2, rows - 1, rows], device="cuda")
    ids = torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda")
    many = x.expand(rows, d_in)
    assert many.stride(0) == 0
    got = zo.zo_adapter_project(ctx, many, w, ad, 16, starts, ids)
    assert torch.equal(got, zo.zo_adapter_project(ctx, many.contiguous(), w, ad, 16, starts, ids))
    t = torch.arange(rows, device="cuda")
    head = w[:1001]
    a, b = (zo.zo_head_logprobs(ctx, v, head, t) for v in (many, many.contiguous()))
    assert torch.equal(a.logp, b.logp) and torch.equal(a.entropy, b.entropy)
