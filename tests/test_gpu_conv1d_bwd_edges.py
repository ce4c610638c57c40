"""The convolution's gradient where it could go wrong: inputs that are not finite
next to the sequence's end."""
import pytest
import torch

import mamba_ssd_scan_b200 as ssd

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _grads(x, w, dy, st, df):
    to = lambda t: None if t is None else t.to(DEV)
    return ssd.ssd_causal_conv1d_bwd(to(x), to(w), to(dy), None, to(st), to(df), activation=False)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("K", [2, 4, 8])
def test_a_non_finite_input_stays_in_the_taps_that_read_it(dtype, value, K):
    """Without activation dweight[c, k] = sum_t dy[t] xin[t - (K-1) + k], t < L: an input
    i places before the end is not read by the taps k < K-1-i.  The others, every
    other channel, dx, dbias and d_init are bitwise what a finite input gives
    there, whatever the length."""
    g = torch.Generator().manual_seed(K)
    C = 16
    for L in list(range(1, 2 * K)) + [15, 16, 17, 24, 31, 33, 41, 47, 64, 500]:
        x, dy = (torch.randn((2, L, C), generator=g).to(dtype) for _ in range(2))
        st, df = (torch.randn((2, C, K - 1), generator=g) for _ in range(2))
        w = torch.randn((C, K), generator=g)
        ends = list(range(min(L, K - 1)))          # places from the end, in x
        carried = list(range(min(L, K - 1), K - 1))  # and in the carried inputs of a short sequence
        clean = _grads(x, w, dy, st, df)
        for i in ends + carried:
            xd, sd = x.clone(), st.clone()
            # column of [carried, x] that lies i places before its end
            if i < L:
                xd[1, L - 1 - i, 5] = value
            else:
                sd[1, 5, K - 1 - 1 - (i - L)] = value
            got = _grads(xd, w, dy, sd, df)
            taps = slice(K - 1 - i, K - 1 - i + min(L, i + 1))  # its taps: those of the tokens 0 .. L - 1
            same = torch.ones((C, K), dtype=torch.bool, device=DEV)
            same[5, taps] = False
            assert torch.equal(got["dweight"][same], clean["dweight"][same]), (L, i)
            assert not torch.isfinite(got["dweight"][5, taps]).any(), (L, i)
            for k in ("dx", "dbias", "d_init"):
                assert torch.equal(got[k], clean[k]), (k, L, i)
