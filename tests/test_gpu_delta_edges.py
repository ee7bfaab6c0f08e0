"""GPU tests of the gated delta rule: orders of dimensions, the step at its limits, states from the 8-bit cache."""
import pytest
import torch

import chunked_linear_scan_amd as cls
from oracle import delta as od
from test_gpu_delta import KEYS, delta_case, oracle_args, run
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


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_orders_of_dimensions(kind):
    """Heads in front of tokens, tokens that overlap (windows of one signal), one key head for all: the same bits as
    contiguous tensors give."""
    c = on_gpu(delta_case(61, 2, 150, 2, 4, 64, 48, kind=kind))
    c = {k: v.contiguous() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    want = run(c)
    names = ("q", "k", "v", "dy")
    got = run({**c, **{k: c[k].transpose(1, 2).contiguous().transpose(1, 2) for k in names}})
    got2 = run({**c, **{k: c[k].permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3) for k in names}})
    for n in want:
        assert torch.equal(got[n], want[n]) and torch.equal(got2[n], want[n]), n
    signal = torch.randn(2, 2, 8 * 149 + 64, generator=torch.Generator().manual_seed(62)).to(c["q"].dtype).cuda() / 8
    over = signal.as_strided((2, 150, 2, 64), (signal.stride(0), 8, signal.stride(1), 1))
    shared = c["q"][:, :, :1].expand(2, 150, 2, 64)
    want = run({**c, "k": over.contiguous(), "q": shared.contiguous()})
    got = run({**c, "k": over, "q": shared})
    for n in want:
        assert torch.equal(got[n], want[n]), n
