"""How near windowed attention to fp32 comes: scores that are exact, so that nothing but the weights,
their products with the values and the sums is measured.

A query has one element, a power of two, and keys hold 32nds between -2 and 0: a score is one exact
product. The error's norm, relative to the output's (values are positive), adds up from

* cuts of the tensor core's sum: a step's products are 8 of 16 keys, each cutting less than two last
  places, 2 x 2^-23, off a sum that is on average half of the step's: 8 x 2^-23 (9.5e-7);
* a score's factor, |scale| * log2(e) in fp32 (two roundings, 2 x 2^-24 of at most 2, times ln 2), in
  the weights and in their sum: 3.3e-7;
* ex2, 2^-22 in both: 4.8e-7; two fp16 numbers for a weight: 2^-22, 2.4e-7 (three bf16 ones: none);
* roundings of either sign: a score's, and 32 + 512 additions at most for a weights' sum, 512 for the
  outputs, 0.29 x 2^-23 each: (1 + sqrt(544) + sqrt(512)) x 3.5e-8 = 1.6e-6;
* the division and the last rounding: 1.2e-7.

Added up 3.8e-6. Two bf16 numbers a weight, or sums that run on in the tensor core through all keys,
exceed it: that is tested on the oracle's side, without a GPU."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

BF, FP = torch.bfloat16, torch.float16
BOUND = 3.8e-6
SCALE = float(np.float32(math.log(2)))


def keys(rng, *shape):
    return -rng.integers(0, 64, shape) / 32.0


def values(rng, *shape):
    return np.abs(rng.standard_normal(shape)) + 0.5


# ------------------------------------------------------------------ the bound tells them apart (oracle's side)

def cut_bf16(x):
    return (x.astype(np.float32).view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)


def cut24(x):
    """Toward zero, to 24 bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(np.ldexp(m, 24)), e - 24)


def error(o, want):
    return float(np.linalg.norm(o - want) / np.linalg.norm(want))


@pytest.fixture(scope="module")
def row():
    rng = np.random.default_rng(0)
    p = np.exp2(keys(rng, 16384)).astype(np.float32).astype(np.float64)
    v = torch.from_numpy(values(rng, 16384, 128)).to(BF).double().numpy()
    return p, v, p @ v / p.sum()


def running(p, v, step):
    """Sums of 16 keys at a time that are cut, `step` keys long; those added up in fp32."""
    o = np.zeros(v.shape[1], np.float32)
    for a in range(0, len(p), step):
        s = np.zeros(v.shape[1])
        for k in range(a, a + step, 16):
            s = cut24(s + p[k:k + 16] @ v[k:k + 16])
        o = o + s.astype(np.float32)
    return o.astype(np.float64) / p.sum()


def test_two_bf16_numbers_a_weight_exceed_the_bound(row):
    p, v, want = row
    hi = cut_bf16(p)
    lo = cut_bf16(p - hi)
    third = cut_bf16(p - hi - lo)
    assert error((hi + lo) @ v / p.sum(), want) > 1.5 * BOUND
    assert error((hi + lo + third) @ v / p.sum(), want) < 1e-12


def test_sums_that_run_on_exceed_the_bound(row):
    p, v, want = row
    assert error(running(p, v, len(p)), want) > 1.5 * BOUND
    assert error(running(p, v, 128), want) < BOUND / 2


# ------------------------------------------------------------------ the kernels

# sequences that share their pages, tokens, query heads a head, keys: an item a block, or nearly
FORMS = {"rows": (40, 1, 4, 32768), "one": (20, 20, 4, 16384), "two": (20, 40, 4, 16384)}


@pytest.mark.gpu
@pytest.mark.parametrize("what", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_outputs_to_fp32(what, D, dt):
    import int4_group_quantized_gs64_gb300 as q
    B, T, G, n = FORMS[what]
    Hkv, page, N = 8, 64, B * T
    rng = np.random.default_rng(n + D)
    k = torch.from_numpy(keys(rng, n // page, Hkv, page, D)).to("cuda", dt)
    v = torch.from_numpy(values(rng, n // page, Hkv, page, D)).to("cuda", dt)
    x = np.zeros((N, Hkv * G, D))
    np.put_along_axis(x, rng.integers(0, D, (N, Hkv * G, 1)), rng.choice([0.5, 1.0], (N, Hkv * G, 1)), 2)
    x = torch.from_numpy(x).to("cuda", dt)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i32([list(range(n // page))] * B)
    o, lse = q.attn_window(q.AttnCache(k, v), x, table, i32([n - T] * B), i32([T * b for b in range(B + 1)]), T,
                           scale=SCALE, o_dtype=torch.float32)
    want = torch.zeros(o.shape, dtype=torch.float64, device="cuda")
    want_lse = torch.zeros(lse.shape, dtype=torch.float64, device="cuda")
    hidden = torch.arange(n, device="cuda") > torch.arange(n - T, n, device="cuda").repeat(B)[:, None]
    for h in range(Hkv):
        kk, vv = (z[:, h].reshape(n, D).double() for z in (k, v))
        for g in range(h * G, h * G + G):
            s = (x[:, g].double() @ kk.T * SCALE).masked_fill_(hidden, -math.inf)
            want_lse[:, g] = torch.logsumexp(s, 1)
            want[:, g] = torch.softmax(s, 1) @ vv
    assert float((o.double() - want).norm() / want.norm()) <= BOUND
    # (its rounding, 2^-24 of 12, log2's and the sum's)
    assert float((lse.double() - want_lse).abs().max()) <= 2.0 ** -20 + 544 * 2.0 ** -24
