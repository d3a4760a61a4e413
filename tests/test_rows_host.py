"""What the calls on rows do on the host before they launch, in a process that sees no device: a
call that is not refused ends with the launch's error and touches none of its pointers."""
import os
import signal
import subprocess
import sys

import pytest

from test_rows_abi import INVALID, UNSUPPORTED, distill, logprobs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA_ERROR = 3


def status_of(call):
    """Exit status of a process without devices that makes `call` (of test_rows_abi)."""
    code = f"import sys; sys.path[:0] = [{os.path.join(ROOT, 'tests')!r}, {ROOT!r}]\n" \
           f"import test_rows_abi as t\nsys.exit(t.{call})"
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    return subprocess.run([sys.executable, "-c", code], env=env, timeout=300).returncode


@pytest.mark.parametrize("V,dtype", [(1, 0), (3, 0), (1, 1), (7, 2), (8, 1)])
def test_token_logprobs_grad_of_rows_shorter_than_a_chunk(V, dtype):
    """A row of fewer elements than 16 bytes hold has no chunk to cut into segments."""
    status = status_of(f"logprobs_grad(V={V}, ld={V}, ld_d={V}, dtype={dtype})")
    assert status != -signal.SIGFPE and status == CUDA_ERROR


@pytest.mark.parametrize("grad", [False, True])
def test_distill_refuses_a_temperature_whose_scale_overflows(grad):
    """The kernels form log2(e) / temperature, which passes fp32's largest number below 4.24e-39."""
    for tau in (3e-39, 4.2e-39):
        assert distill(grad, tau=tau) == INVALID
    assert status_of(f"distill({grad}, tau=4.3e-39)") == CUDA_ERROR      # taken
    assert status_of(f"distill({grad}, tau=3.4e38)") == CUDA_ERROR


def test_token_logprobs_bounds_the_rows_that_have_alternatives():
    """Logits in ascending order are taken up tile by tile: beyond 2^26 of them that could outlast
    the kernel's waits.  Without alternatives rows may be longer."""
    assert logprobs(V=(1 << 26) + 1, ld=1 << 27) == UNSUPPORTED
    assert logprobs(V=1 << 30, ld=1 << 30, K=1) == UNSUPPORTED
    assert status_of("logprobs(V=1 << 26, ld=1 << 26)") == CUDA_ERROR    # taken
    assert status_of("logprobs(V=1 << 30, ld=1 << 30, K=0, ids=None, top=None)") == CUDA_ERROR
