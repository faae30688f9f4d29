"""Paths of the gated linear recurrence that depend on the call's size: stages
used again by later tiles; against the fp64 oracle, with the bounds of
tests/test_gpu_linrec.py."""
import threading

import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
from tests.test_gpu_linrec import DEV, F, TYPES, check_bwd, check_fwd, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load()


def shifted(t):
    """A copy whose first element lies one element behind a 16-byte boundary."""
    flat = torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)
    out = flat[1:1 + t.numel()].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 16
    return out


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(d)[6:] for d in t))
def test_unaligned_rows_through_a_stage_used_again(types):
    """Rows at the ends of unaligned tensors go into the stage element by
    element, and later tiles of the same CTA by bulk copies over them: more
    tiles than CTAs (three groups of channels by 200 rows of tiles and more)."""
    c = make(61, [15000, 1, 24999], 129, *types, g_lo=-0.5)
    x, g, y = (shifted(c[k].to(DEV)) for k in ("x", "g", "y"))
    cu, h0, df = (c[k].to(DEV) for k in ("cu", "h0", "df"))
    out, hT = gdr.linrec_fwd(x, g, cu, initial_state=h0)
    check_fwd(c, out.cpu(), hT.cpu())
    check_bwd(c, *(t.cpu() for t in gdr.linrec_bwd(x, g, y, cu, initial_state=h0, d_final_state=df)))
    assert gdr.device_status() == 0


def test_validation_of_a_step_reads_no_padding():
    """Gates of padding sequences are not looked at, whatever they hold; those
    of the others are, in the first row and the last."""
    lens = [2, 3, 0, 5, 1]
    c = make(62, lens, 40, F, F, pad=2)
    at = [int(v) for v in c["cu"]]
    dev = {k: c[k].to(DEV) for k in ("x", "g", "cu")}
    idx = torch.tensor([3, -1, 0, -7, 5], dtype=torch.int32, device=DEV)
    call = lambda g: gdr.linrec_step(dev["x"], g, torch.zeros(6, 40, device=DEV), idx, dev["cu"],  # noqa: E731
                                     flags=gdr.GDR_COMMIT | gdr.GDR_VALIDATE)
    g = dev["g"].clone()
    for a, b in ((at[1], at[2]), (at[3], at[4]), (at[5], c["T"])):
        g[a:b] = float("nan")
    call(g)
    for row in (at[0], at[1] - 1, at[4]):
        for value in (float("nan"), 0.5):
            bad = g.clone()
            bad[row, 39] = value
            with pytest.raises(gdr.GdrError, match="gate"):
                call(bad)


def test_validated_calls_from_two_threads():
    """One thread's input is good and the other's bad, over and over: neither
    takes the other's findings, or loses its own."""
    c = make(63, [60], 64, F, F)
    x, g, cu = (c[k].to(DEV) for k in ("x", "g", "cu"))
    bad = g.clone()
    bad[7, 9] = 1.0
    torch.cuda.synchronize()
    found = {}

    def many(name, gates):
        torch.cuda.set_device(0)
        stream = torch.cuda.Stream()
        found[name] = 0
        for _ in range(1000):
            try:
                gdr.linrec_fwd(x, gates, cu, flags=gdr.GDR_VALIDATE, stream=stream)
            except gdr.GdrError:
                found[name] += 1

    threads = [threading.Thread(target=many, args=a) for a in (("good", g), ("bad", bad), ("good too", g))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert found == {"good": 0, "bad": 1000, "good too": 0}
