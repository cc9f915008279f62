"""Products with adapters of more than 4096 rows, whose sums are made 64 rows at a time, and
results of 16 bits in many shapes, against the definitions in 64 bits with the tolerances
of the other tests of adapters."""
from __future__ import annotations

import random

import pytest

torch = pytest.importorskip("torch")

from mixed_precision_dense_02_gb300 import binding
from test_gpu_lora import Case, T, random_lengths, rnd, rows16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    yield
    binding.device_status()


MIXED = [1500, 1, 2, 7, 63, 65, 1, 1, 0, 3, 2000, 5, 8, 9, 4]
BATCHES = {
    "one": [4097], "mixed": MIXED + [5000 - sum(MIXED)], "singles": [1] * 900 + [3500],
    "many": [1, 0, 6, 7, 3] * 250 + [900], "prompts": [64, 128, 1000, 3200],
}


@pytest.mark.parametrize("row", [False, True])
@pytest.mark.parametrize("r", [16, 33, 65, 128])
@pytest.mark.parametrize("batch,kind,out", [
    ("one", "bf16", "bf16"), ("mixed", "bf16", "f32"), ("mixed", "f16", "f16"), ("singles", "f16", "f32"),
    ("many", "bf16", "f32"), ("many", "f16", "f16"), ("prompts", "f16", "f32"), ("prompts", "bf16", "bf16")])
def test_many_rows(batch, kind, out, r, row):
    lengths = BATCHES[batch]
    assert sum(lengths) > 4096
    rng = random.Random(r)
    adapters = [rng.choice([-1, 0, 1, 2, 3, 4]) for _ in lengths]
    c = Case(lengths, 136, 200, r, adapters, 5, kind, row, gap=(rng.choice([0, 5]), rng.choice([0, 70])), seed=r)
    addend = rows16(rnd(9, c.t, 136), T[out], 1) if r == 33 else None
    c.check(out, addend)


def test_long_sums_of_many_rows():
    """Several rounds of the ring, and its last stage in part."""
    for row in (False, True):
        for k in (1000, 4104):
            Case(BATCHES["mixed"], 72, k, 128, [i % 4 - 1 for i in range(16)], 3, "bf16", row, seed=k).check("f32")


def test_many_random_batches_in_16_bits():
    for seed in range(30):
        rng = random.Random(100 + seed)
        lengths = random_lengths(seed, rng.randint(1, 60), rng.choice([4, 40, 300]))
        if sum(lengths) == 0:
            lengths[0] = 1
        total, kind = rng.randint(1, 9), rng.choice(["bf16", "f16"])
        n, k, r = rng.randint(1, 700), rng.randint(1, 900), rng.choice([1, 8, 16, 33, 64, 100, 128])
        adapters = [rng.randint(-1, total) for _ in lengths]
        Case(lengths, n, k, r, adapters, total, kind, rng.random() < 0.4,
             gap=(rng.randint(0, 2), rng.randint(0, 70)), seed=seed).check(rng.choice([kind, kind, "f32"]))
