"""The barriers of the windowed attention kernel under drawn delays, on a host model: no wait passes
for another phase than the one it means, nothing is overwritten in use, no block gets stuck."""
import random

import pytest

import window_sync_model as model
from test_attn_sync import noticed

FORMS = {  # what launch_window_tc picks by tiles an item, elements a head and output type
    "one_d128": dict(stages=(3, 3), two=False),
    "one_d128_fp32_from_bf16": dict(stages=(3, 3), two=False, split=True, parted=True),
    "one_d128_fp32_from_fp16": dict(stages=(3, 3), two=False, split=True),
    "one_d64": dict(stages=(6, 6), two=False, apart=True),
    "one_d64_fp32": dict(stages=(6, 6), two=False, split=True),
    "two_d128": dict(stages=(2, 3), two=True),
    "two_d128_fp32_from_bf16": dict(stages=(2, 3), two=True, split=True, parted=True),
    "two_d128_fp32_from_fp16": dict(stages=(2, 3), two=True, split=True),
    "two_d64": dict(stages=(6, 6), two=True, apart=True),
    "two_d64_fp32": dict(stages=(6, 6), two=True, split=True),
}
TIMES = [dict(copy=2000, slow=20), dict(copy=3000, slow=5), dict(copy=300, slow=100)]


def segments(seed):
    """A block's parts of items, many of them short: which of their steps have masks."""
    r = random.Random(seed)
    return [[r.random() < 0.4 for _ in range(r.choice([1, 1, 2, 3, 4, 5, 9, 14]))] for _ in range(r.randint(1, 6))]


@pytest.mark.parametrize("form", FORMS)
def test_attention(form):
    for times in TIMES:
        for seed in range(60):
            model.window_tc(seed, segments(seed), **FORMS[form], **times)


def test_products_that_do_not_wait_for_the_look_at_values_are_noticed():
    assert noticed(lambda seed: model.window_tc(seed, segments(seed), **FORMS["two_d128"], copy=300, slow=100,
                                                wait_ready=False))


def test_new_weights_before_the_last_products_are_noticed():
    assert noticed(lambda seed: model.window_tc(seed, segments(seed), **FORMS["two_d64"], copy=300, slow=100,
                                                wait_done=False))


def test_both_halves_of_the_weights_at_one_barrier_are_noticed():
    assert noticed(lambda seed: model.window_tc(seed, segments(seed), **FORMS["two_d64_fp32"], copy=300, slow=100,
                                                one_barrier=True))
