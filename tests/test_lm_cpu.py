"""Host-side checks of the language-model operators: refusals that need no GPU, workspace sizes,
and that the references agree with torch's own float64 functions."""
import math

import pytest
import torch

import forward_only_amd as zo
import lm_ref as ref
from forward_only_amd import _lib


def test_null_context_is_refused():
    L = _lib.lib()
    assert L.zo_token_logprobs(None, None, 0, 1, 8, 8, None, None, None, 0, None, None,
                               None) == _lib.ZO_EINVAL
    assert L.zo_head_logprobs(None, None, 8, None, 0, 1, 8, 8, None, None, None, None, 0,
                              None) == _lib.ZO_EINVAL
    assert L.zo_group_loss(None, None, None, None, 1, 1, None, None) == _lib.ZO_EINVAL
    assert L.zo_adapter_project(None, None, 8, None, None, 0, 1, 8, 8, None, 0, 8, 1.0, None, None, 1,
                                None, None, 0, 0, 0, 0, None, None, 0, None, 8, None) == _lib.ZO_EINVAL


def test_workspace_sizes_grow_and_stay_bounded():
    assert zo.zo_head_workspace_bytes(1, 768, 50272) <= zo.zo_head_workspace_bytes(16384, 768, 50272)
    # beyond one launch's rows only the row list grows
    a, b = (zo.zo_head_workspace_bytes(r, 768, 50272) for r in (1 << 20, 1 << 21))
    assert 0 < b - a <= 4 * (1 << 20) + 256
    base = zo.zo_adapter_workspace_bytes(100, 64, 64, 2, 8, 3)
    assert zo.zo_adapter_workspace_bytes(100, 64, 64, 2, 8, 3, 5) == base + 5 * zo.zo_bits_stride(2048)
    assert zo.zo_adapter_workspace_bytes(0, 64, 64, 2, 8, 3) >= 0


def test_cpu_tensors_are_refused():
    x, t = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64)
    for call in (lambda: zo.zo_token_logprobs(None, x, t), lambda: zo.zo_head_logprobs(None, x, x, t),
                 lambda: zo.zo_group_loss(None, x[:, 0].contiguous(), t, t),
                 lambda: zo.zo_adapter_project(None, x, x, x, 8, t, t.int())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        zo.zo_token_logprobs(None, [1.0], t)


def test_references_agree_with_torch():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 40, generator=g)
    t = torch.tensor([3, -100, 39, 40, 0])
    logp, entropy, ids, top = ref.token(x, t, 4)
    p = torch.log_softmax(x.double(), dim=1)
    want = torch.stack([p[0, 3], torch.tensor(0.0).double(), p[2, 39], torch.tensor(math.nan).double(),
                        p[4, 0]])
    ref.assert_close(logp, want, 1e-13, "logp")
    h = -(p.exp() * p).sum(1)
    h[1] = 0
    ref.assert_close(entropy, h, 1e-13, "entropy")
    v, i = p.topk(4, dim=1)
    assert torch.equal(ids[0], i[0]) and (ids[1] == -1).all()
    ref.assert_close(top[2], v[2], 1e-13, "top")
    with pytest.raises(AssertionError):
        ref.assert_close(logp, want + 1e-6, 1e-7, "a planted mistake")


def test_project_reference_agrees_with_a_dense_adapter():
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn(6, 16, generator=g), torch.randn(24, 16, generator=g)
    ad = torch.randn(2 * 8 * 40, generator=g)
    y, low, bound = ref.project(x, w, None, ad, 8, [0, 2, 2, 5], [1, 0, -1], 0.5)
    per = 8 * 40
    a, b = ad[per:per + 128].view(8, 16).double(), ad[per + 128:].view(24, 8).double()
    dense = x[:2].double() @ (w.double() + 0.5 * b @ a).t()
    ref.assert_close(y[:2], dense, 1e-12, "adapter 1")
    ref.assert_close(y[2:5], x[2:5].double() @ w.double().t(), 1e-12, "none")
    assert torch.isnan(y[5]).all() and (bound > 0).all()


def test_probe_groups_of_a_batch():
    from forward_only_amd.step import adapter_probe_groups
    g = adapter_probe_groups(3, 5, 0.25, probe0=7, step=2, offset=128, device="cpu")
    assert g.starts.tolist() == [0, 5, 10, 15, 20, 25, 30, 35] and g.starts.dtype == torch.int64
    assert g.probes.tolist() == [0, 0, 1, 1, 2, 2, -1] and g.probes.dtype == torch.int32
    assert g.alphas.tolist() == [0.25, -0.25, 0.25, -0.25, 0.25, -0.25, 0.0]
    assert g.ids.tolist() == [0] * 7 and g.of_project()["n_probes"] == 3
    assert adapter_probe_groups(2, 4, 1.0, clean=False, device="cpu").probes.tolist() == [0, 0, 1, 1]
    only = adapter_probe_groups(0, 4, 1.0, device="cpu")
    assert only.probes.tolist() == [-1] and only.starts.tolist() == [0, 4]


@pytest.mark.parametrize("narrow,wide", [(5120, 5120), (768, 2304), (5120, 20480), (64, 64), (40008, 64),
                                         (7168, 7168), (2048, 520), (768, 50272), (5120, 50272), (4104, 5003)])
def test_a_workspace_for_many_rows_serves_fewer(narrow, wide):
    """Sizes never fall as rows grow, though the products' tiles change with them."""
    most = 0
    for rows in list(range(0, 1200)) + list(range(1200, 9000, 61)) + [1 << 20, 1 << 25]:
        need = zo.zo_adapter_workspace_bytes(rows, narrow, wide // 8 * 8, 1, 16, 8, 3)
        assert need >= most, rows
        most = need
    most = 0
    for rows in list(range(0, 1200)) + list(range(1200, 20000, 61)) + [1 << 20, 1 << 30]:
        need = zo.zo_head_workspace_bytes(rows, narrow, wide)
        assert need >= most, rows
        most = need
    # slices of tiles, 64 MiB, the list of rows, and at most one statistic of 32 features a row
    assert zo.zo_head_workspace_bytes(16384, narrow, wide) <= (1 << 26) + 16384 * (8 + 12 * (wide // 32 + 1)) + 2048


class _OtherStream:
    device = torch.device("cuda", 1)
    cuda_stream = 0


def test_stream_of_another_device_is_refused_without_allocations():
    with pytest.raises(ValueError):
        zo._stream(_OtherStream(), 0)
    assert zo._stream(_OtherStream(), 1) == 0


def test_probe_groups_are_made_on_their_device():
    """No tensor of the host takes part, so that a step can be captured into a graph."""
    from torch.utils._python_dispatch import TorchDispatchMode
    from torch.utils._pytree import tree_flatten

    from forward_only_amd.step import adapter_probe_groups
    seen = []

    class Watch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            seen.extend((str(func), t.device.type) for t in tree_flatten((args, kwargs, out))[0]
                        if isinstance(t, torch.Tensor))
            return out

    for n, clean in ((3, True), (2, False), (0, True)):
        with Watch():
            g = adapter_probe_groups(n, 5, 0.25, clean=clean, device="meta")
        assert g.starts.device.type == g.ids.device.type == "meta"
    assert seen and not [s for s in seen if s[1] != "meta"]
