"""The language-model operators as a step uses them together: a teacher's alternatives, a student with 4-bit
weights and adapters that learns from them by probes, and the exact gradient of its unembedding matrix."""
import pytest
import torch

import forward_only_amd as zo
import lm_more_ref as more
import lm_ref as ref
from forward_only_amd.step import adapter_probe_groups, applied_eps, spsa_step_adapters

pytestmark = pytest.mark.gpu

ROWS, D, HID, VOCAB, RANK, TOP = 24, 128, 64, 512, 8, 12


@pytest.fixture(scope="module")
def ctx():
    c = zo.zo_init(21)
    yield c
    c.close()


@pytest.fixture(scope="module")
def model(ctx):
    g = torch.Generator().manual_seed(3)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std  # noqa: E731
    m = {"x": n(ROWS, D), "w": n(HID, D, std=0.1), "u": n(VOCAB, HID, std=0.3),
         "ad": n(RANK * (D + HID), std=0.05), "targets": torch.arange(ROWS) % 7}
    m["targets"][::5] = ref.IGNORE
    m = {k: v.cuda() for k, v in m.items()}
    m["w4"] = zo.zo_q4_quantize(ctx, m["w"], 64)
    m["u4"] = zo.zo_q4_quantize(ctx, m["u"], 32)
    # the teacher: the model before its weights lost bits
    logits = (m["x"] @ m["w"].t()) @ m["u"].t()
    top = zo.zo_token_logprobs(ctx, logits, m["targets"], top_k=TOP)
    m["ids"], m["logp"] = top.top_ids, top.top_logp
    return m


def _logits(ctx, m, ad, groups):
    G = groups.ids.numel()
    h = zo.zo_q4_project(ctx, m["x"].repeat(G, 1), m["w4"], ad, RANK, **groups.of_project())
    return h, zo.zo_q4_project(ctx, h, m["u4"])


def test_step_by_distillation(ctx, model):
    m, npert, eps, delta, eta = model, 6, 0.0625, 1e-6, 1e-3
    ad = m["ad"].clone()
    seen = []

    def logp_of(groups):
        G = groups.ids.numel()
        _, logits = _logits(ctx, m, ad, groups)
        loss = zo.zo_distill_loss(ctx, logits, m["ids"].repeat(G, 1), m["logp"].repeat(G, 1),
                                  targets=m["targets"].repeat(G)).loss
        seen.append(loss.view(G, ROWS))
        return -loss

    out = spsa_step_adapters(ctx, ad, step=4, npert=npert, eps=eps, eta=eta, delta=delta, logp_of=logp_of,
                             targets=m["targets"], probes_per_batch=4)
    torch.cuda.synchronize()
    # each probe's losses from the definitions in 64 bits, with the weights that the codes stand for
    w, u = zo.zo_q4_unpack(ctx, m["w4"]).double().cpu(), zo.zo_q4_unpack(ctx, m["u4"]).double().cpu()
    bits = zo.zo_gen_probes(ctx, 4, 0, npert, 0, ad.numel()).cpu()
    z, a = ref.signs(bits, ad.numel()), applied_eps(eps)
    count = m["targets"].cpu() != ref.IGNORE

    def loss_at(theta):
        t = theta.double()
        A, B = t[:RANK * D].view(RANK, D), t[RANK * D:].view(HID, RANK)
        x = m["x"].double().cpu()
        logits = (x @ w.t() + (x @ A.t()) @ B.t()) @ u.t()
        return more.distill(logits, m["ids"].cpu(), m["logp"].cpu(), m["targets"].cpu(), 1.0)[0][count].mean()

    th = m["ad"].cpu()
    # fp32 sums: products of 128 and 64 terms of norms below 60, a softmax of 512: 1e-4 is ten times their bounds
    assert abs(float(out["L0"]) - float(loss_at(th))) < 1e-4
    for i in range(npert):
        assert abs(float(out["Lp"][i]) - float(loss_at(th + a * z[i]))) < 1e-4
        assert abs(float(out["Lm"][i]) - float(loss_at(th - a * z[i]))) < 1e-4
    assert torch.isfinite(out["c"]).all() and not torch.equal(ad, m["ad"])
    assert len(seen) == 2 and not seen[0][:, ::5].any()          # ignored rows lose nothing


def test_exact_head_gradient_beside_probes(ctx, model):
    """The clean pass's hidden states give the unembedding's gradient and the mean loss."""
    m = model
    groups = adapter_probe_groups(0, ROWS, 0.0)
    h, _ = _logits(ctx, m, m["ad"], groups)
    n = int((m["targets"] != ref.IGNORE).sum())
    weight = torch.full((ROWS,), 1.0 / n, device="cuda")
    got = zo.zo_head_grad(ctx, h, m["u"], m["targets"], row_grad=weight)
    logp, dh, dw, bl, bh, bw = more.head_grad(h.cpu(), m["u"].cpu(), m["targets"].cpu(), weight.cpu(), torch.float32)
    ref.assert_close(got.logp, logp, bl + 1e-30, "logp")
    ref.assert_close(got.hidden_grad, dh, bh * 1.01 + 1e-30, "hidden_grad")
    ref.assert_close(got.weight_grad, dw, bw * 1.01 + 1e-30, "weight_grad")
    starts = torch.tensor([0, ROWS], device="cuda")
    assert abs(float(zo.zo_group_loss(ctx, got.logp, m["targets"], starts)) + float(logp.sum()) / n) < 1e-5


def test_adapter_and_4bit_projections_agree(ctx, model):
    """The same call with the weights that the codes stand for."""
    m = model
    groups = adapter_probe_groups(3, ROWS, 0.125, step=2)
    a = zo.zo_q4_project(ctx, m["x"].repeat(7, 1), m["w4"], m["ad"], RANK, **groups.of_project())
    b = zo.zo_adapter_project(ctx, m["x"].repeat(7, 1), zo.zo_q4_unpack(ctx, m["w4"]), m["ad"], RANK, **groups.of_project())
    # both within lm_ref's bound of a product of 128 terms
    x, w = m["x"].double(), zo.zo_q4_unpack(ctx, m["w4"]).double()
    bound = 4 * 8 * 128 ** 0.5 * ref.U32 * torch.linalg.vector_norm(x, dim=1).max() * torch.linalg.vector_norm(w, dim=1).max()
    assert float((a - b).abs().max()) < float(bound) + 1e-5
