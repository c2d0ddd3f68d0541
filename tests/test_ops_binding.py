"""What the native binding of the operators around the layer refuses and shows
without a GPU: tensors here have a device and a shape, and no call gets as far
as their memory."""
import pytest
import torch

BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


@pytest.fixture(scope="module")
def bsq():
    from block_scaled_precision_03_gb300 import _build
    import block_scaled_precision_03_gb300 as b
    _build.build()
    b.lib()
    return b


def on(device, *shape, dtype=F32):
    """A tensor of that shape on cuda:`device` whose memory is not there."""
    stride = [1]
    for n in reversed(shape[1:]):
        stride.insert(0, stride[0] * n)
    nbytes = max(1, torch.Size(shape).numel()) * dtype.itemsize
    storage = torch._C._construct_storage_from_data_pointer(1 << 20, torch.device("cuda", device), nbytes)
    return torch._C._construct_CUDA_Tensor_From_Storage_And_Metadata(
        {"storage_offset": 0, "dtype": dtype, "size": shape, "stride": tuple(stride)}, storage)


T, C, V, E, K = 4, 16, 10, 3, 2
PLAN = (("offsets", (E + 1,), I64), ("slot_row", (T, K), I32), ("row_slot", (T * K,), I32))
# name: (tensor arguments in order: (shape, type); a number stands for itself; "plan" for a plan)
CALLS = {
    "moe_sort_into": [((T, K), I64), "plan"],
    "moe_dispatch_into": [((T, C), BF), ((T, K), I64), "plan", ((T * K, C), BF)],
    "moe_gather_into": [((T, C), BF), "plan", ((T * K, C), BF)],
    "moe_combine_into": [((T * K, C), BF), ((T, K), F32), "plan", ((T, C), BF)],
    "moe_combine_backward_into": [((T, C), BF), ((T * K, C), BF), ((T, K), F32), "plan", ((T * K, C), BF), ((T, K), F32)],
    "layer_norm_into": [((T, C), BF), ((C,), F32), ((C,), F32), 1e-5, ((T, C), BF), ((T,), F32), ((T,), F32)],
    "layer_norm_backward_into": [((T, C), BF), ((T, C), BF), ((C,), F32), ((T,), F32), ((T,), F32), ((T, C), BF),
                                 ((C,), F32), ((C,), F32)],
    "linear_cross_entropy_into": [((T, C), BF), ((V, C), BF), ((T,), I64), ((T,), F32), ((T,), F32)],
    "linear_cross_entropy_backward_into": [((T, C), BF), ((V, C), BF), ((T,), I64), ((T,), F32), ((T,), F32),
                                           ((T, C), BF), ((V, C), BF)],
}


def build(bsq, spec, other):
    """Arguments on cuda:0, but the tensor number `other` on cuda:1; returns (arguments, number of tensors)."""
    n, args = 0, []

    def one(shape, dtype):
        nonlocal n
        n += 1
        return on(1 if n - 1 == other else 0, *shape, dtype=dtype)
    for a in spec:
        if a == "plan":
            args.append(bsq.MoePlan(E, *(one(shape, dtype) for _, shape, dtype in PLAN)))
        else:
            args.append(one(*a) if isinstance(a, tuple) else a)
    return args, n


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_on_two_devices_are_refused(bsq, name):
    _, n = build(bsq, CALLS[name], -1)
    for other in range(n):
        args, _ = build(bsq, CALLS[name], other)
        with pytest.raises(bsq.BsqError, match="cuda:[01]") as e:
            getattr(bsq, name)(*args)
        assert e.value.status == 1, other


def test_gradient_lists_on_two_devices_are_refused(bsq):
    a, b = on(0, 8), on(1, 8)
    for grads, outs in (([a, b], None), ([a], [b]), ([a, a], [a, b])):
        with pytest.raises(bsq.BsqError, match="cuda:1"):
            bsq.GradList(grads, outs)
    assert bsq.GradList([b], [b]).count == 1
    from block_scaled_precision_03_gb300 import ops
    with pytest.raises(bsq.BsqError, match="cuda:1"):
        ops._native().grads_into(0, 1, 1.0, 0.0, on(0, 1), on(1, 16, dtype=torch.uint8), None)


def test_clipping_to_no_norm_is_refused(bsq):
    # None would otherwise mean "the norm only" and leave the outputs as they are
    grads = bsq.GradList([on(0, 8)], [on(0, 8)])
    for call in (lambda: bsq.clip_grad_norm(grads, None), lambda: bsq.clip_grad_norm([on(0, 8)], None),
                 lambda: bsq.clip_grad_norm_into(grads, None, on(0, 1))):
        with pytest.raises(bsq.BsqError, match="max_norm"):
            call()


def test_the_calls_keep_their_documentation(bsq):
    # the native functions take the places of the Python ones at the first call
    import subprocess
    import sys
    code = """
import inspect
import block_scaled_precision_03_gb300 as bsq
from block_scaled_precision_03_gb300 import ops
before = {n: (inspect.getdoc(getattr(bsq, n)), list(inspect.signature(getattr(bsq, n)).parameters.values())) for n in ops._BOUND}
ops._native()
for name, (doc, parameters) in before.items():
    f = getattr(bsq, name)
    assert f is getattr(ops, name) and type(f).__name__ == "builtin_function_or_method"
    assert doc and inspect.getdoc(f) == doc, (name, f.__doc__)
    got = list(inspect.signature(f).parameters.values())
    assert [(p.name, p.default) for p in got] == [(p.name, p.default) for p in parameters], (name, got)
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root)
