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


@pytest.mark.parametrize("dtype,out_dtype,D", [(torch.float32, None, 512), (torch.float32, None, 516),
                                               (torch.float32, None, 2560), (torch.bfloat16, None, 1032),
                                               (torch.bfloat16, torch.float32, 2561), (torch.float16, None, 4096)], ids=str)
@pytest.mark.parametrize("layout", ["packed", "strided"])
def test_embed_grad_of_no_positions(dtype, out_dtype, D, layout):
    """Zeroes the table's gradient, rows of every width; adds nothing to one that is given."""
    V, pad = 300, {"packed": 0, "strided": 8}[layout]
    w = ds.Workspace.of_bytes(ds.embed_grad_workspace_bytes(0, V, D))
    d_out = torch.empty(0, D, dtype=dtype, device="cuda")
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    buf = torch.full((V, D + pad), 7.0, dtype=out_dtype or dtype, device="cuda")
    ds.embed_grad(d_out, ids, V, w, out=buf[:, :D], accumulate=True)
    assert (buf == 7).all()
    ds.embed_grad(d_out, ids, V, w, out=buf[:, :D])
    assert (buf[:, :D] == 0).all() and (buf[:, D:] == 7).all()
    assert w.status() == 0
