"""The binding of include/qlayer.h on the CPU: tensors that do not fit are
refused before the library is called."""
import os

import pytest
import torch

import compressed_gemv_amd as cg


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(cg.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return cg.load()


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(n):
    return torch.zeros(n, dtype=torch.int32)


def f64(n):
    return torch.zeros(n, dtype=torch.float64)


@pytest.mark.parametrize("A,B,scales,ranks", [
    (bf(2, 8, 64), bf(3, 40, 8), torch.ones(2), None), (bf(2, 8, 64), bf(2, 40, 16), torch.ones(2), None),
    (bf(2, 8, 64).float(), bf(2, 40, 8), torch.ones(2), None), (bf(8, 64), bf(2, 40, 8), torch.ones(2), None),
    (bf(2, 8, 64), bf(2, 40, 8), torch.ones(3), None), (bf(2, 8, 64), bf(2, 40, 8), torch.ones(2).double(), None),
    (bf(2, 8, 64), bf(2, 40, 8), torch.ones(2), i32(3)), (bf(2, 8, 64), bf(2, 40, 8), torch.ones(2), torch.zeros(2))])
def test_adapter_sets(A, B, scales, ranks):
    with pytest.raises(ValueError):
        cg.make_qadapters(A, B, scales, ranks)


def test_adapters_on_the_host_are_refused():
    with pytest.raises(ValueError, match="CUDA"):
        cg.make_qadapters(bf(2, 8, 64), bf(2, 40, 8), torch.ones(2))


def handle():
    a = cg.qadapters(2, 64, 40, 8, 0x10000, 0x10000, 0x10000, None)
    a._device, a._index = torch.device("cuda:0"), 0
    return a


@pytest.mark.parametrize("x,y,ids,starts,kw", [
    (bf(3, 56), bf(3, 40), i32(3), None, {}), (bf(3, 64).float(), bf(3, 40), i32(3), None, {}), (bf(64), bf(3, 40), i32(3), None, {}),
    (bf(3, 64), bf(2, 40), i32(3), None, {}), (bf(3, 64), bf(3, 41), i32(3), None, {}), (bf(3, 64), bf(3, 40).half(), i32(3), None, {}),
    (bf(3, 64), bf(3, 40), i32(2), None, {}), (bf(3, 64), bf(3, 40), i32(3).long(), None, {}), (bf(3, 64), bf(3, 40), i32(2), i32(4), {}),
    (bf(3, 64), bf(3, 40), i32(2), i32(3).long(), {}), (bf(3, 64), bf(3, 40), i32(3), None, {"out": bf(3, 40).float()}),
    (bf(3, 64), bf(3, 40), i32(3), None, {"out": bf(4, 40)}), (bf(64, 3).t(), bf(3, 40), i32(3), None, {}),
    (bf(3, 64), bf(40, 3).t(), i32(3), None, {}), (bf(1, 64).expand(3, 64), bf(3, 40), i32(3), None, {})])
def test_adapt(x, y, ids, starts, kw):
    with pytest.raises(ValueError):
        cg.qadapt(handle(), x, y, ids, starts, **kw)


def test_adapt_on_the_host_is_refused():
    with pytest.raises(ValueError, match="CUDA"):
        cg.qadapt(handle(), bf(3, 64), bf(3, 40), i32(3))


def test_workspace_sizes():
    a = handle()
    assert cg.qadapt_ws(a, 3, 3) == 3 * 16 * 4
    with pytest.raises(cg.QError):
        cg.qadapt_ws(a, 0, 0)


class Fake(torch.Tensor):
    """A host tensor that says it lies on the GPU, to reach the checks behind that one."""
    is_cuda = True

    def get_device(self):
        return 0

    @property
    def device(self):
        return torch.device("cuda:0")


def fake(t):
    return t.as_subclass(Fake)


@pytest.mark.parametrize("Q,K,lens,starts,kw", [
    (None, None, i32(3), None, {}), (bf(3, 64), bf(3, 2, 64), i32(3), None, {}), (bf(3, 4, 64), bf(2, 2, 64), i32(3), None, {}),
    (bf(3, 4, 64), bf(3, 2, 128), i32(3), None, {}), (bf(3, 4, 64), bf(3, 2, 64).float(), i32(3), None, {}),
    (bf(3, 4, 64).half(), None, i32(3), None, {}), (bf(3, 4, 64), None, i32(2), None, {}), (bf(3, 4, 64), None, i32(3).long(), None, {}),
    (bf(3, 4, 64), None, i32(2), i32(2), {}), (bf(3, 4, 64), None, i32(3), None, {"freqs": f64(32).float()}),
    (bf(3, 4, 64), None, i32(3), None, {"q_weight": bf(63)}), (bf(3, 4, 64), None, i32(3), None, {"q_weight": bf(64).half()}),
    (bf(3, 4, 64), bf(3, 2, 64), i32(3), None, {"q_weight": bf(64), "k_weight": torch.zeros(64)}),
    (bf(3, 4, 64), None, i32(3), None, {"out_dtype": torch.float16}), (bf(3, 4, 64), None, i32(3), None, {"Ko": bf(3, 2, 64)}),
    (bf(3, 4, 64), None, i32(3), None, {"Qo": bf(2, 4, 64)}), (bf(3, 64, 4).transpose(1, 2), None, i32(3), None, {}),
    (bf(3, 4, 64), bf(3, 2, 64), i32(3), None, {"Qo": bf(3, 4, 64), "Ko": bf(3, 2, 64).float()})])
def test_norm_rope(Q, K, lens, starts, kw):
    with pytest.raises(ValueError):
        cg.qnorm_rope(None if Q is None else fake(Q), None if K is None else fake(K), fake(lens), None if starts is None else fake(starts),
                      **{n: fake(v) if isinstance(v, torch.Tensor) else v for n, v in kw.items()})


def test_norm_rope_on_the_host_is_refused():
    with pytest.raises(ValueError, match="CUDA"):
        cg.qnorm_rope(bf(3, 4, 64), None, i32(3))


@pytest.mark.parametrize("Q,K,V,starts,kw", [
    (bf(3, 64), bf(3, 2, 64), bf(3, 2, 64), None, {}), (bf(3, 5, 64), bf(3, 2, 64), bf(3, 2, 64), None, {}),
    (bf(2, 4, 64), bf(3, 2, 64), bf(3, 2, 64), None, {}), (bf(3, 4, 64), bf(3, 2, 64), bf(2, 2, 64), None, {}),
    (bf(3, 4, 64), bf(3, 2, 64), bf(3, 1, 64), None, {}), (bf(3, 4, 64).float(), bf(3, 2, 64), bf(3, 2, 64), None, {}),
    (bf(3, 4, 64), bf(3, 2, 64), bf(3, 2, 64).half(), None, {}), (bf(3, 4, 64), bf(3, 2, 64), bf(3, 2, 64), i32(1), {}),
    (bf(3, 4, 64), bf(3, 2, 64), bf(3, 2, 64), i32(3).long(), {}), (bf(3, 4, 64), bf(3, 2, 64), bf(3, 2, 64), None, {"out": bf(2, 4, 64)}),
    (bf(3, 4, 64), bf(3, 2, 64), bf(3, 2, 64), None, {"out_dtype": torch.float16}),
    (bf(3, 4, 128), bf(3, 2, 64), bf(3, 2, 64), None, {})])
def test_prompt_attend(Q, K, V, starts, kw):
    with pytest.raises(ValueError):
        cg.qprompt_attend(fake(Q), fake(K), fake(V), None if starts is None else fake(starts),
                          **{n: fake(v) if isinstance(v, torch.Tensor) else v for n, v in kw.items()})


def test_prompt_attend_on_the_host_is_refused():
    with pytest.raises(ValueError, match="CUDA"):
        cg.qprompt_attend(bf(3, 4, 64), bf(3, 2, 64), bf(3, 2, 64))
