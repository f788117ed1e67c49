"""The norms' gradient of an empty batch: what it leaves in its workspace, and what the binding takes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DIM = 64


def setup(mfsdp, gate_rows):
    ones = [torch.ones(DIM, device="cuda") for _ in range(3)]
    norm = mfsdp.BlockNorm(DIM, post=mfsdp.NORM_RMS, post_weight=ones[0], gate=ones[1], gate_rows=gate_rows,
                           pre=mfsdp.NORM_RMS, pre_weight=ones[2])
    ws = torch.full((mfsdp.block_norm_grad_workspace_bytes(norm, 0),), 0x55, dtype=torch.uint8, device="cuda")
    rows, stats = torch.empty(0, DIM, device="cuda"), torch.empty(0, 4, device="cuda")
    return norm, ws, rows, stats


@pytest.mark.parametrize("wanted", ["d_pre_weight", "d_post_weight"])
def test_status_word_is_cleared(mfsdp, wanted):
    """A call that launches leaves its own status, not what the memory held before."""
    norm, ws, rows, stats = setup(mfsdp, 5)
    assert mfsdp.op_device_status(ws)[0] != mfsdp.OK
    d = torch.full((DIM,), 7.0, device="cuda")
    mfsdp.block_norm_grad(norm, rows, stats, branch=rows, d_residual_out=rows, d_normed=rows, workspace=ws, **{wanted: d})
    assert not d.any()
    assert mfsdp.op_device_status(ws) == (mfsdp.OK, 0)


@pytest.mark.parametrize("accumulate", [False, True])
def test_binding_takes_the_usual_buffers(mfsdp, accumulate):
    """What a training step passes for any batch, d_gate of the gate's size among it, which stays as it is."""
    norm, ws, rows, stats = setup(mfsdp, 5)
    d_gate, d = (torch.full((DIM,), 7.0, device="cuda") for _ in range(2))
    mfsdp.block_norm_grad(norm, rows, stats, branch=rows, d_residual_out=rows, d_normed=rows, d_residual=rows, d_branch=rows,
                          d_gate=d_gate, d_pre_weight=d, accumulate=accumulate, workspace=ws)
    assert (d_gate == 7.0).all() and (d == (7.0 if accumulate else 0.0)).all()
    with pytest.raises(ValueError):
        mfsdp.block_norm_grad(norm, rows, stats, branch=rows, d_residual_out=rows, d_normed=rows,
                              d_gate=d_gate.bfloat16(), workspace=ws)
