"""GPU tests of the gated delta rule's step at its limits, and of states that went through the 8-bit cache."""
import pytest
import torch

import chunked_linear_scan_amd as cls
from oracle import delta as od
from test_gpu_delta import KEYS, delta_case, oracle_args
from test_gpu_selective import U, close, f64, on_gpu

pytestmark = pytest.mark.gpu


def test_step_of_very_many_rows():
    """2^26 rows of states (2 GiB): each sequence as on its own."""
    nb, H, dk, dv = 1 << 14, 16, 8, 256
    g = torch.Generator(device="cuda").manual_seed(60)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    h = rn(nb, H, dv, dk)
    q, k = (torch.nn.functional.normalize(rn(nb, 1, dk), dim=-1).bfloat16() for _ in range(2))
    v, gl, beta = rn(nb, H, dv).bfloat16(), -rn(nb, H).abs(), torch.sigmoid(rn(nb, H))
    for part in (slice(0, 3), slice(nb // 2, nb // 2 + 1), slice(nb - 5, nb)):
        want_h = h[part].clone()
        want = cls.gated_delta_step(want_h, *(t[part] for t in (q, k, v, gl, beta)))
        before = h[part].clone()
        every = cls.gated_delta_step(h, q, k, v, gl, beta)
        assert torch.equal(every[part], want) and torch.equal(h[part], want_h) and not torch.equal(before, want_h)


def test_a_state_from_the_cache_is_continued():
    """A prompt's state kept in 8 bits and read back: what follows it is what follows the state that was read."""
    c = delta_case(33, 2, 64, 1, 2, 64, 32)
    d = on_gpu(c)
    _, h = cls.gated_delta(*(d[k] for k in KEYS))
    cache = torch.zeros(4, 2, 32, 64, dtype=torch.int8, device="cuda")
    scales = torch.zeros(4, 2, 32, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    cls.state_cache_write(h, cache, scales, slots)
    back = cls.state_cache_read(cache, scales, slots)
    y, h2 = cls.gated_delta(*(d[k] for k in KEYS[:5]), h0=back)
    a = {**oracle_args(c), "h0": f64(back)}
    ry, rh = od.delta(**a)
    _, err = od.delta_bounds("bf16", 64, **a)
    close(y, ry, err["y"] / U, "y")
    close(h2, rh, err["h"] / U, "h")
