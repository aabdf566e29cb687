"""The binding's short way on tensors whose memory cannot be had."""
import pytest
import torch

from test_gpu_draft_binding import F, calls  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["attend", "attend_fp8"])
def test_an_address_that_raises_is_an_error_of_the_call(F, name):
    """A traced tensor has no address: asking for it raises, which must happen while the
    interpreter's lock is held, and reaches the caller."""
    from torch._subclasses import FakeTensorMode
    f, args = calls(F)[name]
    with FakeTensorMode():
        q = torch.empty(args["q"].shape, dtype=args["q"].dtype, device="cuda")
    torch._C._set_throw_on_mutable_data_ptr(q)
    with pytest.raises(RuntimeError):
        f(**{**args, "q": q})
    f(**args)
    torch.cuda.synchronize()
    assert F.fdllm_get_status(args["workspace"]) == F.OK
