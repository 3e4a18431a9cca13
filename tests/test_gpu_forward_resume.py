"""A calibration that resumes and then goes on from the cache, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

import test_forward_stack as fs  # noqa: E402
from transformer_sharding_affinity_gb300 import binding as B, forward as FW, stack as ST  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kept", [[], [2], [1, 2], [0, 1, 2]])
def test_tokens_after_a_resumed_calibration(tmp_path, kept):
    """Whatever layers' scores were already there, the next tokens see the whole step."""
    dev, _ = fs._rounded(fs._layers(8), torch.float32)
    lengths = [25, 40, 16]
    g = torch.Generator().manual_seed(9)
    x, more = torch.randn(sum(lengths), fs.D, generator=g).cuda(), torch.randn(6, fs.D, generator=g).cuda()
    d = B.dims(sum(lengths), fs.D, fs.H, fs.G, fs.DH, fs.I, dtype=B.AFF_FP32)

    def run(calibrate):
        fwd = FW.Forward(dev, fs.H, fs.G, fs.DH, n_pages=16, n_pos=64, page_size=16)
        seqs = [fwd.new_sequence() for _ in lengths]
        if calibrate:
            ST.calibrate_stack(fwd.layer_inputs(x, seqs, lengths), fs.N, d, checkpoint_dir=str(tmp_path))
        else:
            fwd.run(x, seqs, lengths)
        return fwd.run(more, seqs)

    want = run(False)
    assert torch.equal(run(True), want)
    for i in range(fs.N):
        if i not in kept:
            (tmp_path / f"layer_{i:03d}.npz").unlink()
    assert torch.equal(run(True), want)
