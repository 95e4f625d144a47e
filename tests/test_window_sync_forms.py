"""The faulty protocols of test_window_sync in the windowed kernel's other forms: one tile of rows, whose
streams take alternate steps, and 128 elements a head."""
import pytest

import window_sync_model as model
from test_attn_sync import noticed
from test_window_sync import FORMS, segments


def found(form, **wrong):
    return noticed(lambda seed: model.window_tc(seed, segments(seed), **FORMS[form], copy=300, slow=100, **wrong))


@pytest.mark.parametrize("form", FORMS)
def test_products_that_do_not_wait_for_the_look_at_values_are_noticed(form):
    assert found(form, wait_ready=False)


@pytest.mark.parametrize("form", [f for f in FORMS if FORMS[f].get("apart")])
def test_new_weights_before_the_last_products_are_noticed(form):
    assert found(form, wait_done=False)


@pytest.mark.parametrize("form", [f for f in FORMS if FORMS[f].get("split")])
def test_both_halves_of_the_weights_at_one_barrier_are_noticed(form):
    assert found(form, one_barrier=True)
