"""The calls on rows of logits and of tables at the edges of what they take.  Tolerances as in
test_gpu_rows."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ds = pytest.importorskip("speculative_decoding_03_gb300")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture
def ws():
    w = ds.Workspace.of_bytes(256)
    yield w
    assert w.status() == 0


# ------------------------------------------------------------------------------ no rows

@pytest.mark.parametrize("lead", [(0,), (0, 4)])
def test_distill_of_no_rows(lead, ws):
    z = torch.empty(lead + (1000,), device="cuda")
    ids = torch.empty(lead + (8,), dtype=torch.int32, device="cuda")
    t = torch.empty(lead + (8,), device="cuda")
    alone = ds.distill_loss(z, ids, t, ws, labels=ids[..., 0].contiguous(), weights=t[..., 0].contiguous())
    both = ds.distill_loss_grad(z, ids, t, ws, d_loss=t[..., 0].contiguous())
    assert alone["loss"].shape == alone["accept"].shape == both["loss"].shape == lead
    assert both["d_logits"].shape == z.shape
