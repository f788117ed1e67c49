"""Edges of the operators next to the owner step that need no GPU: the oracle's
special values, and calls that the host turns away."""
import numpy as np
import pytest

from oracle.ops import grad_clip_ref


def test_clip_oracle_at_an_infinite_limit():
    norm, coef, out = grad_clip_ref([[1.0, np.nan], [2.0]], np.inf, 1e-6)
    assert np.isnan(norm) and np.isnan(coef) and np.isnan(np.concatenate(out)).all()
    assert grad_clip_ref([[np.inf, 1.0]], np.inf, 1e-6)[:2] == (np.inf, 1.0)
    assert grad_clip_ref([[3.0, 4.0]], np.inf, 1e-6)[:2] == (5.0, 1.0)


def test_scales_that_fp32_does_not_hold_are_refused(mfsdp):
    """The kernels multiply in fp32: a scale that is infinite there would make every
    zero a NaN."""
    lib = mfsdp.raw_lib()
    a, b, c, ws = 0x10000000, 0x20000000, 0x30000000, 0x50000000      # fake, aligned, far apart
    wsb = lib.mfsdp_embedding_grad_workspace_bytes(10, 100, 64)

    def lookup(scale, out=c):
        return lib.mfsdp_embedding_lookup(a, 0, 100, 64, 64, b, mfsdp.ID_I32, 10, scale, out, 0, 64, None)

    def grad(scale, g=c):
        return lib.mfsdp_embedding_grad(a, 0, 64, b, mfsdp.ID_I32, 10, scale, g, 0, 100, 64, 64, 0, ws, wsb, None)
    for scale in (1e300, -1e300, 3.5e38, float("inf"), float("nan")):
        assert lookup(scale) == grad(scale) == mfsdp.ERR_INVALID_ARG, scale
    for scale in (3.4e38, 0.0, -1e-60):                                # turned away later, for the output's alignment
        assert lookup(scale, c + 4) == grad(scale, c + 4) == mfsdp.ERR_MISALIGNED, scale


def test_binding_refuses_workspaces_that_are_no_device_memory(mfsdp):
    """On fakes of CUDA tensors, so that each call comes as far as its workspace."""
    import torch

    class Cuda:
        """What the binding asks of a CUDA tensor."""
        is_cuda = True

        def __init__(self, *shape, dtype=torch.float32):
            self.t = torch.empty(shape, dtype=dtype)
            self.shape, self.dtype = self.t.shape, dtype

        def __getattr__(self, name):
            return getattr(self.t, name)

    host, gaps = torch.empty(1 << 20, dtype=torch.uint8), Cuda(8, 8, dtype=torch.uint8)
    gaps.t = gaps.t[:, :4]
    f, b, i = Cuda(4, 8), Cuda(4, 8, dtype=torch.bfloat16), Cuda(4, dtype=torch.int32)
    w, starts, out = Cuda(3, 8, 8, dtype=torch.bfloat16), Cuda(4, dtype=torch.int32), Cuda(2)
    calls = {
        "grad_norm": lambda ws: mfsdp.grad_norm(mfsdp.grad_set([f]), out, ws, stream=0),
        "grad_clip": lambda ws: mfsdp.grad_clip(mfsdp.grad_set([f]), out, ws, max_norm=1.0, stream=0),
        "sort_ids": lambda ws: mfsdp.sort_ids(i, 3, Cuda(4, dtype=torch.int32), starts, ws, stream=0),
        "embedding_grad": lambda ws: mfsdp.embedding_grad(f, i, Cuda(9, 8), ws, stream=0),
        "expert_matmul": lambda ws: mfsdp.expert_matmul(b, w, starts, Cuda(4, 8), ws, stream=0),
        "expert_weight_grad": lambda ws: mfsdp.expert_weight_grad(b, b, starts, Cuda(3, 8, 8), ws, stream=0),
        "op_device_status": lambda ws: mfsdp.op_device_status(ws, stream=0),
    }
    for name, call in calls.items():
        with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
            call(host)
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            call(gaps)
        if name != "op_device_status":
            with pytest.raises(mfsdp.MfsdpError):                      # none at all: the library's own check
                call(None)
    assert mfsdp._ws(Cuda(64, dtype=torch.float32))[1] == 256          # bytes, whatever the type
    assert mfsdp.op_device_status(None, stream=0)[0] == mfsdp.ERR_INVALID_ARG


@pytest.mark.parametrize("experts,n,rows,cols,cut", [
    (1, 4096, 512, 512, True), (1, 4095, 512, 512, False), (1, 4096, 1024, 2048, False), (1, 16_384, 1024, 1024, True),
    (4, 4096, 256, 1024, False), (4, 16_384, 256, 512, True), (8, 8192, 128, 512, False), (16, 32_768, 256, 512, False),
    (2, 8192, 512, 1024, True), (128, 32_768, 1408, 2048, False), (39, 1 << 20, 64, 64, False)])
def test_weight_gradients_are_cut_where_that_pays(mfsdp, experts, n, rows, cols, cut):
    """A cut contraction takes fp32 matrices in the workspace, beside the status word and the
    groups' padded ends: the sizes on both sides of the rule, as measured."""
    up = lambda b: -(-b // 256) * 256
    plain = 256 + up(16 * experts * rows * 2) + up(16 * experts * cols * 2)
    got = mfsdp.raw_lib().mfsdp_expert_workspace_bytes(experts, n, rows, cols, rows * cols, rows, cols)
    assert got == plain if not cut else got >= plain + experts * rows * cols * 4, (got, plain)
