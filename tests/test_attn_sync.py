"""The barriers of the tcgen05 attention kernels under drawn delays, on a host model: no wait
passes for another phase than the one it means, no slot is copied into before its last use,
no block gets stuck. (Such a fault shows on a GPU only when copies are late, if ever.)"""
import random

import pytest

import attn_sync_model as model

FORMS = {  # what run_tc picks by rows, elements a head and output type
    "rows128_d128": dict(stages=(3, 3), two=False),
    "rows128_d128_fp32_from_bf16": dict(stages=(3, 3), two=False, split=True, parted=True),
    "rows128_d128_fp32_from_fp16": dict(stages=(3, 3), two=False, split=True),
    "rows128_d64": dict(stages=(6, 6), two=False, apart=True),
    "rows128_d64_fp32": dict(stages=(6, 6), two=False, split=True),
    "rows256_d128": dict(stages=(2, 3), two=True),
    "rows256_d128_fp32_from_bf16": dict(stages=(2, 3), two=True, split=True, parted=True),
    "rows256_d128_fp32_from_fp16": dict(stages=(2, 3), two=True, split=True),
    "rows256_d64": dict(stages=(6, 6), two=True, apart=True),
    "rows256_d64_fp32": dict(stages=(6, 6), two=True, split=True),
}
TIMES = [dict(copy=2000, slow=20), dict(copy=3000, slow=5), dict(copy=300, slow=100)]


def segments(seed):
    """Key tiles of the parts of items that a block gets, many of them short."""
    r = random.Random(seed)
    return [r.choice([1, 1, 2, 3, 4, 5, 9, 14]) for _ in range(r.randint(1, 5))]


@pytest.mark.parametrize("form", FORMS)
def test_attention(form):
    for times in TIMES:
        for seed in range(60):
            model.attn_tc(seed, segments(seed), **FORMS[form], **times)


def noticed(run, seeds=1000):
    """Whether the model finds a fault for one of the seeds."""
    for seed in range(seeds):
        try:
            run(seed)
        except model.Broken:
            return True
    return False


def test_one_ring_for_keys_and_values_is_noticed():
    """Copiers that know of their own entries only run into entries of the other stream."""
    assert noticed(lambda seed: model.attn_tc(seed, segments(seed), **FORMS["rows128_d128_fp32_from_bf16"], copy=300,
                                              slow=100, rings=1))


def test_a_stream_that_does_not_answer_is_noticed():
    """In a part of one tile the second stream has none; nothing else holds it to that part."""
    assert noticed(lambda seed: model.attn_tc(seed, segments(seed), **FORMS["rows128_d128"], copy=300, slow=100,
                                              ack=False))


# Ring slots that run puts beside the queries of 1 to 4 row tiles.
RINGS = [(1, 5), (2, 4), (3, 3), (4, 2), (1, 12), (2, 11), (3, 10), (4, 9)]


def rows(seed, most):
    """Key tiles and row tiles of a block's parts: ragged trees have up to `most`."""
    r = random.Random(seed)
    return [(n, r.randint(1, most)) for n in segments(seed)]


@pytest.mark.parametrize("most,stages", RINGS)
def test_weights(most, stages):
    for times in TIMES:
        for seed in range(60):
            model.weights_tc(seed, rows(seed, most), stages, **times)
            model.weights_tc(seed, [(n, most) for n in segments(seed)], stages, **times)


def test_score_buffers_of_both_groups_by_turns_are_noticed():
    """Four products a tile: a group's buffers were last the other group's."""
    assert noticed(lambda seed: model.weights_tc(seed, [(n, 4) for n in segments(seed)], 2, own_buffers=False))


def test_parts_without_products_are_noticed():
    """(The plan leaves out sequences that have no rows in a launch.)"""
    assert noticed(lambda seed: model.weights_tc(seed, [(n, nq - 1) for n, nq in rows(seed, 3)], 3))
