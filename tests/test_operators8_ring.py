"""The 8-bit products' ring of stages: every order of events of a model of it, and the numbers of stages that calls get (no GPU needed).

The kernel (csrc/grouped8.cu): one warp loads slice g into stage g % stages once the slice there before has been used; two warps issue the
products of every other slice each, once its data have landed and its accumulator, g % accumulators, has been read; the sums follow in
order.  All waits are by parity: a wait for use u of a barrier passes while the number of finished phases differs from u by an odd
number, so a wait that is two phases late passes by mistake.
"""
import ctypes
import os
from collections import deque

import pytest

PAIR, SINGLE = 2, 1


def passes(done, use):
    """A wait for the end of phase `use` (-1: before the first) where `done` phases are over."""
    return (done - 1 - use) % 2 == 0


def search(stages, accs, n, accumulator_first):
    """Every order in which n slices can be loaded, land, be issued, be done and summed.  Returns what goes wrong, or None.

    A state is: loads started; slices landed (bits); for both issuing warps the next slice and which of its two tests has passed; slices issued,
    done, and reported to the sums and to the loads (bits); sums done.  The two tests of a slice are on their way at once, so either
    may be the older one."""
    def phases(bits, first, step):
        return sum(bits >> k & 1 for k in range(first, n, step))

    start = (0, 0, (0, 0), (1, 0), 0, 0, 0, 0, 0)
    seen, queue = {start}, deque([start])
    while queue:
        p, landed, w0, w1, issued, done, summable, free, e = state = queue.popleft()
        after = []
        if p < n and passes(phases(free, p % stages, stages), p // stages - 1):
            if p >= stages and not free >> (p - stages) & 1:
                return f"load {p} over a stage in use"
            after.append((p + 1, landed, w0, w1, issued, done, summable, free, e))
        for k in range(n):
            bit, previous = 1 << k, k < 2       # a warp's products are done, and reported, in the order that it issued them
            if k < p and not landed & bit:
                after.append((p, landed | bit, w0, w1, issued, done, summable, free, e))
            if issued & bit and not done & bit:
                after.append((p, landed, w0, w1, issued, done | bit, summable, free, e))
            if done & bit and not summable & bit and (previous or summable >> (k - 2) & 1):
                after.append((p, landed, w0, w1, issued, done, summable | bit, free, e))
            if done & bit and not free & bit and (previous or free >> (k - 2) & 1):
                after.append((p, landed, w0, w1, issued, done, summable, free | bit, e))
        if e < n and passes(phases(summable, e % accs, accs), e // accs):
            if not summable >> e & 1:
                return f"sum {e} too early"
            after.append((p, landed, w0, w1, issued, done, summable, free, e + 1))
        for i, (k, tested) in enumerate((w0, w1)):
            if k >= n:
                continue
            data = passes(phases(landed, k % stages, stages), k // stages)
            accumulator = passes(len(range(k % accs, e, accs)), k // accs - 1)
            if not ((accumulator, data) if accumulator_first else (data, accumulator))[tested]:
                continue
            now = issued
            if tested:
                if not landed >> k & 1:
                    return f"slice {k} issued before its data"
                if k >= accs and e <= k - accs:
                    return f"slice {k} over an accumulator in use"
                now |= 1 << k
            warp = (k + 2, 0) if tested else (k, 1)
            after.append((p, landed, *((warp, w1) if i == 0 else (w0, warp)), now, done, summable, free, e))
        if not after and not (e == n and free == (1 << n) - 1):
            return "nothing can happen"
        for s in after:
            if s not in seen:
                seen.add(s)
                queue.append(s)
    return None


def allowed(stages, accs):
    """Each warp has its own stages, or what was in the stage before has landed when the tests start."""
    return stages >= 2 and (stages % 2 == 0 or stages >= accs + 2)


@pytest.mark.parametrize("stages,accs,n", [(2, 2, 7), (3, 2, 8), (4, 2, 8), (5, 2, 9), (6, 2, 9), (2, 4, 8), (3, 4, 8), (4, 4, 9), (5, 4, 9), (6, 4, 9)])
def test_the_rule_is_what_every_order_of_events_asks_for(stages, accs, n):
    """n passes each stage and each accumulator again.  With more stages than these a stage's last use is longer over when its next one is tested."""
    sound = all(search(stages, accs, n, first) is None for first in (False, True))
    assert sound == allowed(stages, accs)


@pytest.fixture(scope="module")
def form():
    from serving_layer_moe_gb300 import build as b
    from serving_layer_moe_gb300 import load_library
    if not os.path.exists(b.LIB):
        b.build()
    lib, out = load_library(), (ctypes.c_int32 * 4)()

    def call(P, E, N, K=2048, act=0, quant=0, sms=152):
        lib.moe_product8_form(P, E, N, K, act, quant, sms, out)
        return tuple(out)
    return call


# rows of E experts, N, act, quant: calls of each form
FORMS = {
    (PAIR, 256): lambda E: [(1537 * E, 2048, 1, 0), (1537 * E, 2048, 1, 1), (705 * E, 2000, 0, 0), (4000 * E, 256, 0, 0)],
    (SINGLE, 256): lambda E: [(P, 1 << 20, 0, 0) for P in (1, 16, 17, 33, 64, 65, 97, 128, 300 * E)] + [(P, 128, 1, 1) for P in (1, 20, 40, 100, 128, 300 * E)],
    (SINGLE, 128): lambda E: [(P, 100 * 128 // min(P, E) // 128 * 128, 0, 0) for P in (1, 16, 17, 33, 64, 65, 97) if min(P, E) <= 64],
    (SINGLE, 64): lambda E: [(P, 64, 0, 0) for P in (1, 16, 17, 33, 64, 65) if min(P, E) < 76],
}


@pytest.mark.parametrize("kind", FORMS)
def test_every_call_gets_stages_that_the_rule_allows(form, kind):
    reached = set()
    for E in range(1, 4097):
        for P, N, act, quant in FORMS[kind](E):
            ctas, tile, stages, accs = form(P, E, N, act=act, quant=quant)
            if (ctas, tile) == kind:
                assert allowed(stages, accs) and stages <= 12, (P, E, N, stages, accs)
                reached.add((stages, accs))
    assert len(reached) > 1, reached       # small calls and large tables get other numbers


def test_the_form_follows_the_sizes(form):
    """Pairs from their thresholds on; smaller tiles where there are few; one tile for requantised results."""
    assert [form(P, 8, 1920, K=K, act=act)[0] for P, K, act in ((8 * 1536, 400, 1), (8 * 1536 + 1, 400, 1), (8 * 704, 4096, 1), (8 * 704 + 1, 4096, 1), (8 * 704 + 1, 4095, 1))] == [1, 2, 1, 2, 1]
    assert [form(P, 8, 1920, K=K)[0] for P, K in ((8 * 384, 1024), (8 * 384 + 1, 1024), (8 * 384 + 1, 1040), (8 * 704, 1040), (8 * 704 + 1, 1040))] == [1, 2, 1, 1, 2]
    assert [form(1, 1, N)[1] for N in (64, 4096, 9600, 9601, 19200, 19201)] == [64, 64, 64, 128, 128, 256]
    assert form(1, 1, 128, act=1, quant=1)[:2] == (1, 256)
