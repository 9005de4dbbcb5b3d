"""FewTokenMoE takes tensors of the current device only: the library sees addresses.

Checked on the host with stand-ins for tensors of two devices; the library's calls are replaced by ones that record.
"""
import pytest

torch = pytest.importorskip("torch")
m = pytest.importorskip("moe_layer_dsv3_gb300")
few_module = pytest.importorskip("moe_layer_dsv3_gb300.few")

SHAPE = dict(d=256, E=8, k=2, n_groups=1, topk_groups=1, I=128, n_shared=1)


class Tensor:
    """What the class looks at of a dense CUDA tensor."""

    is_cuda = True

    def __init__(self, dev, dtype, *shape):
        self.device, self.dtype, self.shape = torch.device("cuda", dev), dtype, torch.Size(shape)

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 4096

    def __getitem__(self, rows):
        return Tensor(self.device.index, self.dtype, len(range(*rows.indices(self.shape[0]))), *self.shape[1:])


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    new = lambda shape, dtype=None, device=None: Tensor(torch.device(device).index or 0, dtype,
                                                        *(shape if isinstance(shape, tuple) else (shape,)))
    monkeypatch.setattr(torch, "zeros", new)
    monkeypatch.setattr(torch, "empty", new)
    for name in ("moe_few_forward", "moe_quantize_weights"):
        monkeypatch.setattr(few_module, name, lambda *a, name=name: made.append(name))
    return made


def weights(dev=0):
    return Tensor(dev, torch.uint8, m.moe_weights_size(m.config(4, *SHAPE.values())))


def inputs(dev=0):
    return dict(x=Tensor(dev, torch.bfloat16, 4, 256), w_router=Tensor(dev, torch.bfloat16, 8, 256), bias=Tensor(dev, torch.float32, 8))


def masters(dev=0):
    return dict(w_gu=Tensor(dev, torch.bfloat16, 8, 256, 256), w_d=Tensor(dev, torch.bfloat16, 8, 256, 128),
                ws_gu=Tensor(dev, torch.bfloat16, 1, 256, 256), ws_d=Tensor(dev, torch.bfloat16, 1, 256, 128))


def refused(f, *a, **kw):
    with pytest.raises(m.MoeError) as e:
        f(*a, **kw)
    assert e.value.code == m.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("own", [False, True])
def test_one_device(calls, own):
    few = few_module.FewTokenMoE(4, **SHAPE, wq=None if own else weights(), device="cuda")
    few.quantize_weights(**masters())
    few.forward(**inputs())
    assert calls == ["moe_quantize_weights", "moe_few_forward"]


def test_weights_of_another_device_are_refused(calls):
    refused(few_module.FewTokenMoE, 4, **SHAPE, wq=weights(1), device="cuda:0")
    few_module.FewTokenMoE(4, **SHAPE, wq=weights(1), device="cuda:1")     # of the layer's own device
    few = few_module.FewTokenMoE(4, **SHAPE, wq=weights(), device="cuda:0")
    few.wq = weights(1)                                                     # exchanged later
    refused(few.forward, **inputs())
    refused(few.quantize_weights, **masters())
    assert not calls


def test_tensors_of_another_device_are_refused(calls):
    few = few_module.FewTokenMoE(4, **SHAPE, device="cuda:0")
    for name, t in inputs(1).items():
        refused(few.forward, **{**inputs(), name: t})
    refused(few.forward, **inputs(), y=Tensor(1, torch.bfloat16, 4, 256))
    for name, t in masters(1).items():
        refused(few.quantize_weights, **{**masters(), name: t})
    other = few_module.FewTokenMoE(4, **SHAPE, device="cuda:1")            # the layer's device is not the current one
    refused(other.forward, **inputs())
    refused(other.forward, **inputs(1))
    refused(other.quantize_weights, **masters(1))
    assert not calls
