"""Workspaces and kept buffers of the caller, which kernels write by address and
size: those on another device, or whose size counts memory that is not theirs, are
refused by the binding before a pointer leaves it."""
import pytest
import torch

from linear_recurrent_sequence_shortconv_amd import prism as P


def _calls(device):
    """Every entry that takes a buffer, by name: a function of that buffer."""
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device=device)
    x, w, taps, h = z(2, 300, 64), z(64), z(64, 4), z(2, 300, 64)
    q, g = z(2, 32, 2, 64), z(2)
    ab, S = torch.full((2, 32, 2), 0.5, device=device), z(2, 2, 64, 64)
    return {
        "layer_norm_backward": lambda b: P.layer_norm_backward(x, x, w, workspace=b),
        "short_conv_backward": lambda b: P.short_conv_backward(x, taps, x, workspace=b),
        "gated_recurrence": lambda b: P.gated_recurrence(x, x, workspace=b),
        "gated_recurrence_backward": lambda b: P.gated_recurrence_backward(x, x, h, x, workspace=b),
        "forward": lambda b: P.forward(q, q, q, ab, ab, chunk=32, workspace=b),
        "forward saved": lambda b: P.forward(q, q, q, ab, ab, chunk=32, saved=b),
        "backward": lambda b: P.backward(q, q, q, ab, ab, dO=q, chunk=32, workspace=b),
        "backward saved": lambda b: P.backward(q, q, q, ab, ab, dO=q, chunk=32, saved=b),
        "step": lambda b: P.step(q, q, q, ab, ab, S=S, workspace=b),
        "qk_norm_backward": lambda b: P.qk_norm_backward(q, q, q, q, wq=w, workspace=b),
        "linear_attention": lambda b: P.linear_attention(q, q, q, g, workspace=b),
        "linear_attention_backward": lambda b: P.linear_attention_backward(q, q, q, g, q, workspace=b),
    }


@pytest.mark.parametrize("name", ["layer_norm_backward", "short_conv_backward", "gated_recurrence",
                                  "gated_recurrence_backward"])
def test_refused_on_the_host(name):
    call = _calls("cpu")[name]
    with pytest.raises(ValueError, match="workspace: expected device"):
        call(torch.empty(1 << 24, dtype=torch.uint8, device="meta"))
    for buf in (torch.zeros(1, dtype=torch.uint8).expand(1 << 24), torch.zeros(1 << 12, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            call(buf)
    with pytest.raises(ValueError, match="GPU"):
        call(torch.zeros(1 << 12, dtype=torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(_calls("meta")))
def test_refused_beside_tensors_on_the_gpu(name):
    call, what = _calls("cuda")[name], "saved" if "saved" in name else "workspace"
    print(f"\n[given buffer {name}]", flush=True)
    with pytest.raises(ValueError, match=f"{what}: expected device"):
        call(torch.zeros(1 << 24, dtype=torch.uint8))
    with pytest.raises(ValueError, match=f"{what} must be contiguous"):
        call(torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 28))
    if what == "workspace":
        call(torch.zeros(1 << 28, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
