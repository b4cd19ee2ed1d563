"""16-bit prompts hold states, sums and operands to binary32: what is rounded to
16 bits is o, once.

Bounds, for unit keys without a common direction, retentions below 1 and v of unit
size (no product is then much larger than its sum):
 * a state passes at most four chained products (K M, the system for U, K^T U, and
   the sum with the faded state).  Each is a sum of no more than 24 binary32 rounded
   additions of values the size of the result (matrix instructions add 16 or 32 terms at
   once), of 2^-24 / sqrt(3) each in the 2-norm: sqrt(4 * 24 / 3) * 2^-24 = 3.4e-7,
   and three times that for the terms of the chunks before that have not faded: 1e-6;
 * an output's own products add two more, 4.2e-7 of the size of its terms in the
   2-norm; the largest of 10^5 values of that spread lies within 5 of them: 2.1e-6.  So
   each value of o is within half a unit in the last place of the exact result, and
   2.1e-6 of the terms' size |q| |M| (the 2-norm of o's row over sqrt(D) is of it, so
   the row's size is used)."""
import numpy as np
import pytest

from linear_ref import recurrence
from test_linear import Run, far

STATE = 1e-6
BEYOND = 2.1e-6


def half_unit(x, dtype):
    """Half a unit in the last place of the 16-bit type at |x|, at least that of its smallest normal value."""
    bits, low = {"bf16": (8, -126), "f16": (11, -14)}[dtype]
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** low))) - bits)


@pytest.mark.gpu
@pytest.mark.parametrize("rule", ["delta", "additive"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,lengths,D", [((16, 8), [37], 128), ((4, 2), [700, 65], 128), ((4, 4), [300, 0, 1, 129], 64),
                                             ((3, 1), [260] * 90, 128), ((3, 3), [130] * 90, 64), ((2, 1), [260, 64], 32),
                                             ((2, 2), [200, 3], 16)], ids=str)
def test_states_and_outputs_have_binary32_accuracy(dtype, rule, heads, lengths, D):
    r = Run(dtype, *heads, D, rule, lengths, seed=21)
    resume = [b % 2 for b in range(len(lengths))]
    r.prefill(resume)
    q, k, v, beta, gate = r.host()
    o, state = r.o.double().cpu().numpy(), r.state.cpu().numpy()
    for b, slot in enumerate(r.slots):
        at = slice(r.cu[b], r.cu[b + 1])
        m = r.before[slot] if resume[b] else np.zeros_like(r.before[slot])
        ro, rm = recurrence(q[at], k[at], v[at], None if beta is None else beta[at], gate[at], m)
        assert far(state[slot], rm) <= STATE, b
        if lengths[b]:
            size = np.sqrt((ro ** 2).mean())
            over = np.abs(o[at] - ro) - half_unit(ro, dtype)
            assert over.max() <= BEYOND * size, (b, over.max() / size)


@pytest.mark.gpu
@pytest.mark.parametrize("rule", ["delta", "additive"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("close", [2.0 ** -9, 2.0 ** -14, 2.0 ** -20, 2.0 ** -23])
def test_retentions_close_to_one_over_a_long_prompt(dtype, rule, close):
    """Retentions within `close` of 1, for 3000 tokens: a relative error of 2^-23 in each
    logarithm leaves 3000 close 2^-23 of the state, far below the bound, an absolute one of
    that size 3.6e-4 of it.  States that hardly fade gather the rounding of 47 chunks' sums,
    sqrt(47 / 3) * 2^-24 = 2.4e-7, on top of a chunk's 3.4e-7 (above): within the same 1e-6."""
    import torch
    r = Run(dtype, 2, 1, 64, rule, [3000], seed=50)
    r.gate = 1.0 - close * torch.rand(3000, 2, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    r.prefill([1])
    q, k, v, beta, gate = r.host()
    ro, rm = recurrence(q, k, v, beta, gate, r.before[r.slots[0]])
    assert far(r.state[int(r.slots[0])].cpu().numpy(), rm) <= STATE
