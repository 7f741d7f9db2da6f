"""The binding's one look at a call's tensors: what the compiled form and the Python form accept and refuse
has to be the same, and whatever they refuse has to reach the checks that say why."""
import pytest
import torch

from two_tower_block_b200 import ops

X = torch.zeros(4, 6, dtype=torch.bfloat16)
I = torch.zeros(3, dtype=torch.int32)
CASES = {
    "fits": (-1, (X, I), ((torch.bfloat16, 24), (torch.int32, 3)), True),
    "nothing": (-1, (), (), True),
    "parameter": (-1, (torch.nn.Parameter(X),), ((torch.bfloat16, 24),), True),
    "size": (-1, (X,), ((torch.bfloat16, 23),), False),
    "dtype": (-1, (X,), ((torch.float16, 24),), False),
    "device": (0, (X,), ((torch.bfloat16, 24),), False),
    "strided": (-1, (X.t(),), ((torch.bfloat16, 24),), False),
    "none": (-1, (X, None), ((torch.bfloat16, 24), (torch.int32, 3)), False),
    "address": (-1, (X.data_ptr(),), ((torch.bfloat16, 24),), False),
    "numpy": (-1, (X.float().numpy(),), ((torch.float32, 24),), False),
    "meta": (-1, (torch.zeros(24, dtype=torch.bfloat16, device="meta"),), ((torch.bfloat16, 24),), False),
    "sparse": (-1, (torch.zeros(24).to_sparse(),), ((torch.float32, 24),), False),
}


@pytest.mark.parametrize("name", list(CASES))
def test_compiled_and_python_form_agree(name):
    device, tensors, want, fits = CASES[name]
    for form in (ops._quick, ops._quick_py):
        if form is ops._quick_py and name in ("meta", "sparse"):
            continue   # (the Python form may fail on these in its own way)
        at = form(device, tensors, want)
        assert at == ([t.data_ptr() for t in tensors] if fits else None), form


def test_the_compiled_form_is_built_and_checks_its_own_arguments():
    assert ops._quick is not ops._quick_py
    for bad in ((), (0, [X], ()), ("0", (X,), ()), (0, (X,), ())):
        with pytest.raises(TypeError):
            ops._quick(*bad)


def test_odd_want_is_refused():
    assert ops._quick(-1, (X,), ((torch.bfloat16,),)) is None
    with pytest.raises((TypeError, OverflowError)):
        ops._quick(-1, (X,), ((torch.bfloat16, "24"),))


@pytest.mark.parametrize("form", ["_quick", "_quick_py"])
def test_a_copy_on_write_tensor_gets_memory_of_its_own(form):
    """A lazy clone shares its source's memory until someone writes: the address that a kernel may write to
    must not be the source's."""
    source = torch.arange(24, dtype=torch.float32)
    clone = torch._lazy_clone(source)
    at = getattr(ops, form)(-1, (clone,), ((torch.float32, 24),))
    assert at == [clone.data_ptr()] and at != [source.data_ptr()]
    assert torch.equal(clone, source)
